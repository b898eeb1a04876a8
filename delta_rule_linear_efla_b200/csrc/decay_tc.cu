// decay_tc.cu -- linear attention with a decay for each head on the tensor cores (tcgen05, TMEM, TMA):
// the walks of decay.h for bf16 inputs with a and b of 64 or 128.
//
// One CTA walks one stretch of one head, a chunk of 64 tokens at a time.  The state and value
// dimensions are the MMA's M, so that the state stays in tensor memory as S^T, fp32, and its 16-bit copy
// is a tensor-memory operand:
//
//   P        = X Y^T                        [64 x 64]
//   O2^T     = Z^T (D o P)^T                [b x 64]
//   O1^T     = S^T X^T                      [b x 64]     out = diag(q) O1 + O2
//   S^T      = e^{c_C} S^T + Z^T Yw         [b x a]      Yw = diag(w) Y
//
// What is rounded to bf16 on the way, and how often:
//   D o P   once: at most 2^-8 of terms that add like the bf16 output itself, whose own rounding is the same.
//   Yw      as two bf16 halves (Yw = hi + lo to 2^-16), two products into the fp32 state: the state is an
//           fp32 result, and a sequence's rounding errors would gather in it.  What is left is that (2.5e-6 of
//           S_final) and the tensor core's fp32 accumulation, which truncates: 3e-8 of the state a product, eight a
//           chunk, 5e-6 for heads that remember 2000 tokens.
//   S^T     once for o and for dv.  For dq and dk, whose dots with q and k give dl, as two halves: dl is
//           a suffix sum of q.dq - k.dk that cancels down to the pairs that straddle a token; errors of
//           D o P cancel with them (dq and dk round the same products), errors of two different state
//           copies would not, and would grow with the square root of the sequence.
// Decay factors and the sums of their logarithms are fp32.  The factors within a chunk take differences of
// running sums, off by at most 2^-10 where a chunk forgets everything at every token (sums of 18000) and 2^-15
// with one such token: below the rounding of D o P.
//
// What bounds it (4 x 16 x 4096 tokens, d = 128: forward 94 us with its first pass, 87 in a loop of that call alone;
// the three backward walks 309 to 322 us with theirs): the latency of a chunk's chain of hand-offs (the state's copy,
// its products, the state again), under which one CTA an SM has nothing else to run, and the bytes.  Loads and
// hand-offs alone take 63 of the 87 us and 163 of 305; leaving out any one role's arithmetic changes the forward by
// at most 6 %, the gradients by at most 12 %.  Issue slots are busy 42 to 52 % of the time, the tensor pipe 16 to 38 %.
// At 1 x 16 x 65536 the forward's two passes move 1.6 GB in 345 us (296 before the power limit takes the clock from
// 1965 to 1500 MHz).
//
// Warp roles (one CTA an SM, 24 warps):
//   0-3   weight:  Yw's halves from Y's tile
//   4-7   mask:    D o P from TMEM into its operand tile
//   8-11  state:   S^T after a chunk: its 16-bit copy, and scaled by the next chunk's e^{c_C}
//   12-19 output:  out^T from TMEM to global memory, and its dots; half a chunk's tokens each four warps
//   20    issues the state's products (S^T and O1^T)   21 those within the chunk (P and O2^T)
//   22    TMA producer   23 decays (sums and weights, up to four chunks ahead)
// The two issuers wait for different groups; one that waited for both ran the two loops one after the other.
// Role bodies are loops of 16 to 32 columns: each is run once a chunk by one warp a scheduler, and unrolled
// bodies were bound by instruction fetch (8 to 9 cycles an instruction against about 3).
// Every mbarrier wait is bounded; a wait that gives up sets the device error word, lets what is in flight
// land (again bounded), frees its tensor memory and exits.
#include <cudaTypedefs.h>

#include "decay_gate.cuh"
#include "launchers.h"
#include "tma_slabs.cuh"

namespace efla {
namespace decay {

static __device__ unsigned int g_decay_error = 0;

namespace {

constexpr int WARPS = 24, THREADS = WARPS * 32;
constexpr int W_STATE = 20, W_INTRA = 21, W_TMA = 22, W_GATE = 23;
constexpr int NS = 3;     // stages of X, Y, Z
constexpr int FL = 4;     // chunks that the first pass adds up on the tensor cores
constexpr int GB = 4, SLOTS = 2 * GB;  // chunks whose decay weights are made at once, and kept
constexpr long long WAIT_BUDGET = 2000000000LL;  // ~1 s of SM cycles

struct Maps {
    CUtensorMap x[MAX_WALKS], y[MAX_WALKS], z[MAX_WALKS], d[MAX_WALKS];
};

template <int A, int B, bool BWD>
struct Cfg {
    static constexpr int XB = (A / 64) * 8192, ZB = (B / 64) * 8192;
    static constexpr int OFF_X = 0, OFF_Y = XB, OFF_Z = 2 * XB, STAGE = 2 * XB + ZB;
    // Yw: two buffers of its hi half, one of its lo half (written when the product that read the last is done)
    static constexpr int OFF_W = NS * STAGE, OFF_L = OFF_W + 2 * XB;
    static constexpr int OFF_P = OFF_L + XB;           // D o P
    static constexpr int OFF_D = OFF_P + 8192;         // backwards: the dots' other factor, half a chunk for each output group
    static constexpr int SMEM = OFF_D + (BWD ? ZB : 0) + 1024;  // + alignment slack
    // tensor memory columns
    // P twice, so that the mask's loop does not wait for the next one; O1^T twice where it fits
    static constexpr int NO1 = BWD && A == 128 ? 1 : 2;
    static constexpr uint32_t T_S = 0, T_H = A, T_L = T_H + A / 2, T_P = T_L + (BWD ? A / 2 : 0), T_O1 = T_P + 128,
                              T_O2 = T_O1 + NO1 * 64;
    static_assert(T_O2 + 64 <= 512, "tensor memory");
};

struct Bars {
    // one arrival (a commit, a thread, or a TMA load)
    uint64_t full[NS], gready[2], y_free[2], pdone[2], d2done, o1done[2], o2done, o2read, drain[2], dfull[2], l_free;
    // one arrival from each of four warps
    uint64_t dread[2];          // backwards: an output group has read the dots' other factor
    uint64_t p_ready, s_ready;  // without output: an accumulator of the sum's parts is free again (pdone: it is full)
    // every warp that reads a batch's weights and that nothing else orders before it: the eight output warps and the
    // weights' four (without output the weights' sixteen).  The mask's and the state's warps have read a chunk's
    // before its p_ready and s_ready, which its output follows; the products that the output follows do not wait
    // for its y_ready.
    uint64_t gfree[2];
    uint64_t o_free[2];                // the eight output warps
    uint64_t y_ready[2];               // the weights' four warps, sixteen without output
    uint64_t free_s[NS];               // one from each issuer
};
constexpr int BARS = sizeof(Bars) / 8, BARS_ONE = NS + 2 + 2 + 2 + 1 + 2 + 2 + 2 + 3, BARS_FOUR = BARS_ONE + 4,
              BARS_GATE = BARS_FOUR + 2, BARS_OUT = BARS_GATE + 2, BARS_Y = BARS_OUT + 2;

struct Slot {
    float qw[C];
    float kw[C];
    float gw[C];  // 2^(c_end - c) within a token's group of eight (end: its last token in walking order)
    float c2[C];  // running sum in units of log 2 (its negative backwards)
    float tot, pad[3];
};

template <int M>
__device__ __forceinline__ int acc_row(int warp, int lane) {
    if constexpr (M == 128) return 32 * warp + lane;
    else return lane < 16 ? 16 * warp + lane : -1;
}

__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

// Bounded waits that also give up once another role has.  try_wait suspends the warp for a while: with
// test_wait, which does not, the polls of two dozen warps that mostly wait took issue slots from the working
// ones (105 us for a prefill of 90).
__device__ __forceinline__ bool try_wait(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    return ok != 0;
}
// By whole warps, whose lanes get one answer: a lane that gave up alone would leave the others of its warp behind, at
// the next instruction that takes all of them.
__device__ __noinline__ bool wait_longer(uint32_t addr, uint32_t parity, volatile int *abort_flag) {
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, try_wait(addr, parity))) {
        const bool late = clock64() - t0 > WAIT_BUDGET;
        if (late) *abort_flag = 1;
        if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    const uint32_t addr = tc::smem_u32(bar);
    return __all_sync(0xffffffffu, try_wait(addr, parity)) || wait_longer(addr, parity, abort_flag);
}

// 16 lanes x 16 columns of tensor memory, a row of eight columns on four threads: v[4 k + 2 e + i] is row
// lane / 4 + 8 e, column 8 k + 2 (lane % 4) + i.  Waits for completion.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 lanes x 16 columns of raw words into tensor memory, without the wait for completion.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 32 lanes x 16 columns from each of two places in tensor memory, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(ta), "r"(tb)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a[i] = __uint_as_float(r[i]);
        b[i] = __uint_as_float(r[16 + i]);
    }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Two fp32 in a 64-bit register: the packed arithmetic of sm_100 does both in one instruction.
struct F2 {
    uint64_t r;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 a;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a.r) : "f"(x), "f"(y));
    return a;
}
__device__ __forceinline__ float2 unpack(F2 a) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(a.r));
    return v;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.r) : "l"(a.r), "l"(b.r));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.r) : "l"(a.r), "l"(b.r), "l"(c.r));
    return d;
}
__device__ __forceinline__ uint32_t pack(F2 a) {
    const float2 v = unpack(a);
    return tc::pack_bf16(v.x, v.y);
}

// Two floats as packed bf16 halves: x = hi + lo to 2^-16 of |x|.
__device__ __forceinline__ void split2(F2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack(x);
    lo = pack(fma2(f2(bf_lo(hi), bf_hi(hi)), f2(-1.f, -1.f), x));
}

// The sums over a warp's lanes of 32 columns: lane l ends with column l's.
__device__ __forceinline__ float column_sums(float (&p)[32], int lane) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float keep = up ? p[i + off] : p[i], send = up ? p[i] : p[i + off];
            p[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    return p[0];
}

__device__ __forceinline__ void put2(float *p, float *q, float x, float y, bool on_p, bool on_q) {
    if (on_p) *p = x;
    if (on_q) *q = y;
}
__device__ __forceinline__ void put2(__nv_bfloat16 *p, __nv_bfloat16 *q, float x, float y, bool on_p, bool on_q) {
    const uint32_t u = tc::pack_bf16(x, y);
    if (on_p) *reinterpret_cast<unsigned short *>(p) = (unsigned short)u;
    if (on_q) *reinterpret_cast<unsigned short *>(q) = (unsigned short)(u >> 16);
}

// OUT = false: the stretch's own contribution to the state only (the segments' first pass).  BWD: walks
// that may have dots (w.dot), with the state's copy in two halves where they do.
template <int A, int B, typename TO, bool OUT, bool BWD>
__global__ void __launch_bounds__(THREADS, 1)
    walk_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Walks ws, const Shares sh, const Gate g,
                   int BH, int L) {
    using K = Cfg<A, B, BWD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = tc::smem_u32(smem_raw);
    uint8_t *base = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
    __shared__ Bars bars;
    __shared__ __align__(16) Slot slots[SLOTS];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2, gtid = tid & 127;
    // ---- walks in the order of their kind, then their head: the shares of two kinds that read the same tensors in
    // the same direction lie alike, so that the later of two readers finds its tiles in L2.
    // This CTA's chunks, [p0, p1) of the row of all walks' chunks, or a part of such a share's last stretch
    const int NC = (L + C - 1) / C;
    const int share = blockIdx.x;
    auto bound = [&](int c) { return c * sh.size + min(c, sh.more); };
    long long p0 = bound(share), p1 = bound(share + 1);
    // A place in it: the walk and its head, and the chunk's position in walking order.
    const uint32_t revs = ws.w[0].rev | ws.w[1].rev << 1 | ws.w[2].rev << 2;
    struct Place {
        int wi, bh, k;
        bool rev;
        __device__ __forceinline__ void walk(int n, uint32_t revs) {  // on to the next walk, n heads of each kind
            if (++bh == n) {
                bh = 0;
                ++wi;
            }
            rev = revs >> wi & 1;
        }
        __device__ __forceinline__ int chunk(int NC) const { return rev ? NC - 1 - k : k; }
    };
    Place at;
    {
        // whole walks: a share is one; shares of cut ones are counted in 32 bits (tc_shares)
        const uint32_t u = sh.cut ? (uint32_t)(OUT ? p0 : p1 - 1) / (uint32_t)NC : share;
        at.k = (int)(p0 - (long long)u * NC);
        if (!OUT) {
            const bool ends = p1 == (long long)(u + 1) * NC;  // the share ends with a walk's end: nothing to do
            if (at.k < 0) at.k = 0;
            p0 = ends ? p1 : (long long)u * NC + at.k;
        }
        at.wi = u / BH;
        at.bh = u - at.wi * BH;
        at.rev = revs >> at.wi & 1;
    }
    const int cnt = p1 > p0 ? (int)(p1 - p0) : 0;
    // Without output the state's weights are taken up to the stretch's end, from its last chunk backwards, so
    // that every product simply adds to the accumulator.
    if (!OUT) at.k += max(cnt - 1, 0);
    auto next = [&](Place &p) {
        if (!OUT) --p.k;
        else if (++p.k == NC) {
            p.k = 0;
            p.walk(BH, revs);
        }
    };

    if (tid == 0) {
        uint64_t *b = reinterpret_cast<uint64_t *>(&bars);
        for (int i = 0; i < BARS; ++i) 
            tc::mbar_init(b + i, i < BARS_ONE ? 1 : i < BARS_FOUR ? 4 : i < BARS_GATE ? (OUT ? 12 : 16) : i < BARS_OUT ? 8 : i < BARS_Y ? (OUT ? 4 : 16) : (OUT ? 2 : 1));
        tc::fence_mbar_init();
        abort_flag = 0;
        tc::tma_prefetch_desc(&maps.x[at.wi]);
        tc::tma_prefetch_desc(&maps.y[at.wi]);
        tc::tma_prefetch_desc(&maps.z[at.wi]);
    }
    if (warp == 0) {
        tc::tmem_alloc(&tmem_base, 512);
        tc::tmem_relinquish();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0), lane_base = (uint32_t)(32 * (warp & 3)) << 16, sb = tc::smem_u32(base);
    const long long budget = WAIT_BUDGET;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bar(bar, parity & 1, &abort_flag); };
    auto wait_gate = [&](int n) { return n % GB != 0 || wait(&bars.gready[n / GB & 1], n / SLOTS); };

    // The state that enters a walk, or a place in it over the stretches [f0, f1) before it, into tensor memory:
    // blocks of 16 columns from cb0 on, every `step`.
    auto load_state = [&](const Place &pl, int f0, int f1, int cb0, int step) {
        const int j = acc_row<B>(warp & 3, lane);
        const Walk &w = ws.w[pl.wi];
        const float *s0 = w.s0 ? w.s0 + (size_t)pl.bh * A * B : nullptr;
        const int di = w.s0_t ? 1 : B, dj = w.s0_t ? A : 1;
#pragma unroll 1
        for (int cb = cb0; cb < A; cb += step) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = s0 && j >= 0 ? s0[(cb + i) * di + j * dj] : 0.f;
#pragma unroll 1
            for (int f = f0; f < f1; ++f) {
                const float e = sh.e[f];
                const float *u = sh.u + (size_t)f * A * B + (size_t)cb * B + j;
                if (j >= 0)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = fmaf(e, v[i], u[i * B]);
            }
            tc::tmem_st16(tmem + lane_base + K::T_S + cb, v);
        }
    };
    auto store_state = [&](const Place &pl) {
        const int j = acc_row<B>(warp & 3, lane);
        float *out = ws.w[pl.wi].s_end ? ws.w[pl.wi].s_end + (size_t)pl.bh * A * B : nullptr;
        if (!out) return;
#pragma unroll 1
        for (int cb = 0; cb < A; cb += 16) {
            float v[16];
            tc::tmem_ld16(tmem + lane_base + K::T_S + cb, v);
            if (j >= 0)
#pragma unroll
                for (int i = 0; i < 16; ++i) out[(size_t)(cb + i) * B + j] = v[i];
        }
    };

    if (OUT) {
        cudaGridDependencySynchronize();
        if (wg >= 2 && wg < 5) {  // the three warpgroups that write and read the state and the outputs
            int c0 = share;       // the first share whose last stretch is of this walk
            if (at.k > 0)
                while (bound(c0) > p0 - at.k) --c0;
            load_state(at, c0, share, 16 * (wg - 2), 48);
            tc::tc_fence_before();
            tc::named_bar_sync(1, 384);
            tc::tc_fence_after();
        }
    }
    if (warp == W_TMA) {
        const bool leader = elect();
        int n = 0;
        for (; n < cnt; ++n) {
            const int st = n % NS, c0 = at.chunk(NC) * C, wi = at.wi, bh = at.bh;
            if (n >= NS && !wait(&bars.free_s[st], n / NS - 1)) break;
            uint8_t *s = base + st * K::STAGE;
            if (leader) {
                tc::mbar_expect_tx(&bars.full[st], (OUT ? 2 : 1) * K::XB + K::ZB);
                tc::tma_load_4d(s + K::OFF_Y, &maps.y[wi], &bars.full[st], 0, c0, 0, bh);
                if (OUT) tc::tma_load_4d(s + K::OFF_X, &maps.x[wi], &bars.full[st], 0, c0, 0, bh);
                tc::tma_load_4d(s + K::OFF_Z, &maps.z[wi], &bars.full[st], 0, c0, 0, bh);
            }
            __syncwarp();
            next(at);
        }
        if (abort_flag)  // let this CTA's own copies land before it exits (bounded)
            for (int m = n > NS ? n - NS : 0; m < n; ++m) tc::mbar_wait(&bars.full[m % NS], (m / NS) & 1, budget / 8);
    } else if (warp == W_STATE) {
        // The whole warp runs the loop and one elected lane issues, so that descriptors are warp-uniform.
        constexpr uint32_t id_s = tc::idesc_bf16(B, A, true, true), id_o1 = tc::idesc_bf16(B, 64, false, false);
        const uint64_t dx = tc::sdesc(sb + K::OFF_X, 16, 1024), dz = tc::sdesc(sb + K::OFF_Z, 8192, 1024);
        const uint64_t dh = tc::sdesc(sb + K::OFF_W, 8192, 1024), dl = tc::sdesc(sb + K::OFF_L, 8192, 1024);
        int st = 0, ph = 0;  // stage and its pass
        for (int n = 0; n < cnt; ++n) {
            const uint64_t o = (uint64_t)(st * (K::STAGE >> 4));
            if (!wait(&bars.full[st], ph) || (OUT && !wait(&bars.s_ready, n))) break;
            tc::tc_fence_after();
            if (OUT) {
                // O1^T = S^T X^T, before the state changes: its copy is then free when the new state is there
                const int ob = n % K::NO1, m = n - K::NO1;  // read by the output of chunk m
                if (m >= 0 && !wait(&bars.o_free[m & 1], m >> 1)) break;
                tc::tc_fence_after();
                const bool split = BWD && ws.w[at.wi].dot;
                if (elect()) {
                    const uint32_t o1 = tmem + K::T_O1 + ob * 64;
#pragma unroll
                    for (int kk = 0; kk < A / 16; ++kk) {
                        const uint64_t x = dx + o + ((kk >> 2) * 512 + (kk & 3) * 2);
                        tc::mma_tmem_a(o1, tmem + K::T_H + kk * 8, x, id_o1, kk > 0);
                        if (split) tc::mma_tmem_a(o1, tmem + K::T_L + kk * 8, x, id_o1, 1u);
                    }
                    tc::mma_commit(&bars.o1done[n & 1]);
                }
                __syncwarp();
            }
            if (!wait(&bars.y_ready[n & 1], n >> 1)) break;
            const int part = n / FL;  // first pass: of the sum, in one of two accumulators
            if (!OUT && n % FL == 0 && part >= 2 && !wait(part & 1 ? &bars.s_ready : &bars.p_ready, part / 2 - 1)) break;
            const uint32_t acc = tmem + K::T_S + (OUT ? 0 : (part & 1) * A);
            tc::tc_fence_after();
            if (elect()) {  // S^T += Z^T Yw
                const uint64_t yh = dh + (uint64_t)((n & 1) * (K::XB >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    tc::mma_bf16(acc, dz + o + kk * 128, yh + kk * 128, id_s, OUT || n % FL > 0 || kk > 0);
                    tc::mma_bf16(acc, dz + o + kk * 128, dl + kk * 128, id_s, 1u);
                }
                tc::mma_commit(&bars.d2done);
                tc::mma_commit(&bars.y_free[n & 1]);
                tc::mma_commit(&bars.l_free);
                if (!OUT && (n % FL == FL - 1 || n == cnt - 1)) tc::mma_commit(&bars.pdone[part & 1]);
            }
            if (elect()) tc::mma_commit(&bars.free_s[st]);
            __syncwarp();
            if (OUT) next(at);
            if (++st == NS) {
                st = 0;
                ++ph;
            }
        }
        // nothing of this CTA's is in flight when it exits (bounded)
        if (elect()) tc::mma_commit(&bars.drain[0]);
        __syncwarp();
        tc::mbar_wait(&bars.drain[0], 0, budget / 4);
    } else if (OUT && warp == W_INTRA) {
        constexpr uint32_t id_p = tc::idesc_bf16(64, 64, false, false), id_o2 = tc::idesc_bf16(B, 64, true, false);
        const uint64_t dx = tc::sdesc(sb + K::OFF_X, 16, 1024), dy = tc::sdesc(sb + K::OFF_Y, 16, 1024);
        const uint64_t dz = tc::sdesc(sb + K::OFF_Z, 8192, 1024), dp = tc::sdesc(sb + K::OFF_P, 16, 1024);
        auto issue_p = [&](int n, int st) {  // P = X Y^T
            if (elect()) {
                const uint64_t o = (uint64_t)(st * (K::STAGE >> 4));
#pragma unroll
                for (int kk = 0; kk < A / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * 512 + (kk & 3) * 2;
                    tc::mma_bf16(tmem + K::T_P + (n & 1) * 64, dx + o + off, dy + o + off, id_p, kk > 0);
                }
                tc::mma_commit(&bars.pdone[n & 1]);
            }
            __syncwarp();
        };
        int st = -1, cur = 0, ph = 0;
        for (int n = -1; n < cnt; ++n) {
            cur = st;
            if (++st == NS) {
                st = 0;
                ++ph;
            }
            if (n + 1 < cnt) {
                if (!wait(&bars.full[st], ph)) break;
                tc::tc_fence_after();
                issue_p(n + 1, st);
            }
            if (n < 0) continue;
            if (!wait(&bars.p_ready, n) || (n > 0 && !wait(&bars.o_free[(n - 1) & 1], (n - 1) >> 1))) break;
            tc::tc_fence_after();
            if (elect()) {  // O2^T = Z^T (D o P)^T
                const uint64_t z = dz + (uint64_t)(cur * (K::STAGE >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc::mma_bf16(tmem + K::T_O2, z + kk * 128, dp + kk * 2, id_o2, kk > 0);
                tc::mma_commit(&bars.o2done);
                tc::mma_commit(&bars.o2read);
                tc::mma_commit(&bars.free_s[cur]);
            }
            __syncwarp();
        }
        if (elect()) tc::mma_commit(&bars.drain[1]);
        __syncwarp();
        tc::mbar_wait(&bars.drain[1], 0, budget / 4);
    } else if (warp == W_GATE) {
        // Four chunks at once: eight lanes a chunk, eight tokens a lane.  A weight is 2 to the sum of the log-decays
        // between its token and the chunk's start or end, and each is summed from that side: fp32 rounds a sum
        // by 2^-24 of itself, and where that is much the weight is nothing.
        float sum = 0.f;
        float x[8] = {};
        const int gk = lane >> 3, tk = 8 * (lane & 7);  // this lane's chunk of the four, and its first token in it
        const __nv_bfloat16 *tokens = static_cast<const __nv_bfloat16 *>(g.p);
        const float *heads = static_cast<const float *>(g.p);
        Place pl = at;  // of the lane's chunk in the batch that is loaded
        bool rev;       // of its chunk in the batch that is worked on
        auto load = [&](int n, int skip) {
            if (!OUT) pl.k -= skip;
            else {
#pragma unroll 1
                for (pl.k += skip; pl.k >= NC; pl.k -= NC) pl.walk(BH, revs);
            }
            const int t = n + gk < cnt ? pl.chunk(NC) * C + tk : L;
            const float lh = g.per_head && t < L ? heads[pl.bh % g.H] : 0.f;
            const __nv_bfloat16 *row = tokens + (size_t)pl.bh * L;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = lh;
                if (!g.per_head && t + i < L) x[i] = __bfloat162float(row[t + i]);
                if (t + i >= L) x[i] = 0.f;
            }
        };
#pragma unroll 1
        for (int n = -GB; n < cnt; n += GB) {
            float c[8], d[8];  // sums up to and with the token, and behind it, in units of log 2, of this lane's eight
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float l = x[i] < L_MIN ? L_MIN : x[i] > -L_MIN ? -L_MIN : x[i];  // NaN stays NaN
                c[i] = l * 1.44269504f;
            }
            rev = pl.rev;
            if (n + GB < cnt) load(n + GB, n < 0 ? gk : GB);
            if (n < 0) continue;
            d[7] = 0.f;
#pragma unroll
            for (int i = 6; i >= 0; --i) d[i] = d[i + 1] + c[i + 1];
            const float own = d[0] + c[0], first = c[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) c[i] += c[i - 1];
            float before = own, behind = own;  // inclusive, over the chunk's eight lanes from either side
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, before, o, 8), v = __shfl_down_sync(0xffffffffu, behind, o, 8);
                if ((lane & 7) >= o) before += u;
                if ((lane & 7) < 8 - o) behind += v;
            }
            const float cC = __shfl_sync(0xffffffffu, before, 7, 8);
            before = __shfl_up_sync(0xffffffffu, before, 1, 8);
            behind = __shfl_down_sync(0xffffffffu, behind, 1, 8);
            if ((lane & 7) == 0) before = 0.f;
            if ((lane & 7) == 7) behind = 0.f;
            float after = 1.f;
            if (!OUT) {  // the decay of the chunks already walked, the batch's earlier ones among them
#pragma unroll
                for (int k = 0; k < GB; ++k) {
                    if (k == gk) after = ex2(sum);
                    sum += __shfl_sync(0xffffffffu, cC, 8 * k);
                }
            }
            const int bi = n / GB & 1;
            if (n >= SLOTS && !wait(&bars.gfree[bi], n / SLOTS - 1)) break;
            Slot &sl = slots[bi * GB + gk];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                float q[4], k[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float up = ex2(before + c[i + e]), down = ex2(behind + d[i + e]);
                    k[e] = after * (rev ? up : down);
                    q[e] = rev ? down : up;
                }
                *reinterpret_cast<float4 *>(sl.kw + tk + i) = make_float4(k[0], k[1], k[2], k[3]);
                if (OUT) *reinterpret_cast<float4 *>(sl.qw + tk + i) = make_float4(q[0], q[1], q[2], q[3]);
            }
            if (OUT) {
                const float sg = rev ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4 *>(sl.c2 + tk + i) = make_float4(sg * (before + c[i]), sg * (before + c[i + 1]),
                                                                              sg * (before + c[i + 2]), sg * (before + c[i + 3]));
                    // within the lane's eight: behind a token, or between the first and it
                    *reinterpret_cast<float4 *>(sl.gw + tk + i) = make_float4(ex2(rev ? c[i] - first : d[i]), ex2(rev ? c[i + 1] - first : d[i + 1]),
                                                                              ex2(rev ? c[i + 2] - first : d[i + 2]), ex2(rev ? c[i + 3] - first : d[i + 3]));
                }
                if ((lane & 7) == 0) sl.tot = ex2(cC);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.gready[bi]);
        }
        if (!OUT && lane == 0) sh.e[blockIdx.x] = ex2(sum);  // 1 for an empty stretch
    } else if (OUT ? wg == 0 : wg < 4) {
        // ---------------------------------------------------------- Yw
        for (int n = 0; n < cnt; ++n) {
            if (!wait_gate(n) || !wait(&bars.full[n % NS], n / NS)) break;
            if (n >= 2 && !wait(&bars.y_free[n & 1], (n >> 1) - 1)) break;
            constexpr int T = OUT ? 128 : 512, PIECES = K::XB / 16 / T;
            const int i0 = OUT ? gtid : tid;
            const uint4 *y = reinterpret_cast<const uint4 *>(base + (n % NS) * K::STAGE + K::OFF_Y) + i0;
            uint4 *hi = reinterpret_cast<uint4 *>(base + K::OFF_W + (n & 1) * K::XB) + i0;
            uint4 *lo = reinterpret_cast<uint4 *>(base + K::OFF_L) + i0;
            const float *kw = slots[n % SLOTS].kw;
            uint4 l[PIECES];
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {  // 8 pieces of 16 bytes a row of a 64-column slab
                const float w1 = kw[(i0 + i * T) >> 3 & 63];
                const F2 f = f2(w1, w1);
                const uint4 u = y[i * T];
                uint4 h;
                split2(f * f2(bf_lo(u.x), bf_hi(u.x)), h.x, l[i].x);
                split2(f * f2(bf_lo(u.y), bf_hi(u.y)), h.y, l[i].y);
                split2(f * f2(bf_lo(u.z), bf_hi(u.z)), h.z, l[i].z);
                split2(f * f2(bf_lo(u.w), bf_hi(u.w)), h.w, l[i].w);
                hi[i * T] = h;
            }
            if (n >= 1 && !wait(&bars.l_free, n - 1)) break;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) lo[i * T] = l[i];
            tc::fence_async_smem();
            warp_arrive(&bars.y_ready[n & 1], lane);
            if (lane == 0 && n % GB == GB - 1) tc::mbar_arrive(&bars.gfree[n / GB & 1]);
        }
    } else if (!OUT && wg == 4) {
        // The stretch's contribution.  The tensor core truncates its fp32 sums, and a stretch is up to a hundred
        // chunks of eight products, whose older ones add little or nothing to a large sum: off by 2e-4 in all.  So
        // it adds up four chunks at a time, and these are added here, rounded to nearest.
        const int j = acc_row<B>(warp & 3, lane), parts = (cnt + FL - 1) / FL;
        float *u = sh.u + (size_t)blockIdx.x * A * B;
        for (int f = 0; f < parts; ++f) {
            if (!wait(&bars.pdone[f & 1], f >> 1)) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < A; cb += 16) {
                float v[16];
                tc::tmem_ld16(tmem + lane_base + K::T_S + (f & 1) * A + cb, v);
                if (f > 0) {
                    float s[16];
                    tc::tmem_ld16(tmem + lane_base + K::T_S + 2 * A + cb, s);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += s[i];
                }
                if (f < parts - 1) {
                    tc::tmem_st16(tmem + lane_base + K::T_S + 2 * A + cb, v);
                } else if (j >= 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[(size_t)(cb + i) * B + j] = v[i];
                }
            }
            warp_arrive(f & 1 ? &bars.s_ready : &bars.p_ready, lane);
        }
    } else if (OUT && wg == 1) {
        // ---------------------------------------------------------- D o P
        // A warp's 16 rows; a thread holds rows r and r + 8, two columns of every eight.  The warp's diagonal
        // block (16 x 16) takes 2^(c_row - c_column) itself; the blocks on the diagonal's on side take it as
        // 2^(c_row - c_end) 2^(c_end - c_column), end the last token (in walking order) of a column's group of
        // eight: neither factor grows, and the second is made once a chunk.  The off side stays zero.
        const int r0 = 16 * (warp & 3), r = r0 + (lane >> 2), cq = 2 * (lane & 3);
        uint8_t *pt = base + K::OFF_P;
        bool rev = false;
        int on0 = 0, on1 = 0;  // columns of the on side's blocks
        for (int n = 0; n < cnt; ++n, next(at)) {
            if (n == 0 || at.rev != rev) {  // the other direction: the off side anew
                if (n > 0 && !wait(&bars.o2done, n - 1)) break;
                rev = at.rev;
#pragma unroll 1
                for (int c = rev ? 0 : 2 * (warp & 3) + 2; c < (rev ? 2 * (warp & 3) : 8); ++c)
                    *reinterpret_cast<uint4 *>(pt + tc::sw128_off(r0 + (lane & 15), c)) = make_uint4(0u, 0u, 0u, 0u);
                on0 = rev ? r0 + 16 : 0;
                on1 = rev ? 64 : r0;
                __syncwarp();
            }
            if (!wait_gate(n) || !wait(&bars.pdone[n & 1], n >> 1)) break;
            tc::tc_fence_after();
            const Slot &sl = slots[n % SLOTS];
            const float ca = sl.c2[r], cb = sl.c2[r + 8];
            const uint32_t tp = tmem + lane_base + K::T_P + (n & 1) * 64;
            uint32_t u[4];
            auto store = [&](int c0) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint32_t *>(pt + tc::sw128_off(r + 8 * e, (c0 >> 3) + k) + 2 * cq) = u[2 * k + e];
            };
            {
                float v[8];
                tmem_ld_16x256(tp + r0, v);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = r0 + 8 * k + cq;
                    const float2 cc = *reinterpret_cast<const float2 *>(&sl.c2[c]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // row r + 8 e, columns c and c + 1
                        const float cr = e ? cb : ca;
                        const int a = rev ? c - r - 8 * e : r + 8 * e - c, a1 = rev ? a + 1 : a - 1;  // on where >= 0
                        u[2 * k + e] = tc::pack_bf16(a >= 0 ? v[4 * k + 2 * e] * ex2(cr - cc.x) : 0.f,
                                                     a1 >= 0 ? v[4 * k + 2 * e + 1] * ex2(cr - cc.y) : 0.f);
                    }
                }
            }
            if (n > 0 && !wait(&bars.o2done, n - 1)) break;  // the tile's last reader
            store(r0);
#pragma unroll 1
            for (int c0 = on0; c0 < on1; c0 += 16) {
                float v[8];
                tmem_ld_16x256(tp + c0, v);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float ce = sl.c2[c0 + 8 * k + (rev ? 0 : 7)];
                    const F2 f = *reinterpret_cast<const F2 *>(&sl.gw[c0 + 8 * k + cq]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = ex2((e ? cb : ca) - ce);
                        u[2 * k + e] = pack(f2(v[4 * k + 2 * e], v[4 * k + 2 * e + 1]) * (f2(x, x) * f));
                    }
                }
                store(c0);
            }
            tc::fence_async_smem();
            warp_arrive(&bars.p_ready, lane);
        }
    } else if (OUT && wg == 2) {
        // ---------------------------------------------------------- S^T
        for (int n = 0;; ++n, next(at)) {
            if (n > 0) {
                if (!wait(&bars.d2done, n - 1)) break;
                tc::tc_fence_after();
                if (at.k == 0) {  // the end of a walk: its state leaves
                    Place last = at;
                    last.bh = at.bh > 0 ? at.bh - 1 : BH - 1;
                    last.wi = at.bh > 0 ? at.wi : at.wi - 1;
                    store_state(last);
                    if (n < cnt) load_state(at, 0, 0, 0, 16);
                }
            }
            if (n == cnt || !wait_gate(n)) break;
            const F2 tot2 = f2(slots[n % SLOTS].tot, slots[n % SLOTS].tot);
#pragma unroll 1
            for (int cb = 0; cb < A; cb += 32) {
                float v[32];
                tc::tmem_ld32(tmem + lane_base + K::T_S + cb, v);
                uint32_t h[16], l[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(f2(v[2 * i], v[2 * i + 1]), h[i], l[i]);
                tmem_st16(tmem + lane_base + K::T_H + cb / 2, h);
                if (BWD && ws.w[at.wi].dot) tmem_st16(tmem + lane_base + K::T_L + cb / 2, l);
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 t = unpack(tot2 * f2(v[e + i], v[e + i + 1]));
                        u[i] = __float_as_uint(t.x);
                        u[i + 1] = __float_as_uint(t.y);
                    }
                    tmem_st16(tmem + lane_base + K::T_S + cb + e, u);
                }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            warp_arrive(&bars.s_ready, lane);
        }
    } else if (OUT && (wg == 3 || wg == 4)) {
        // ---------------------------------------------------------- out
        const int j = acc_row<B>(warp & 3, lane), h0 = wg == 3 ? 0 : 32;  // tokens h0 .. h0 + 31 of a chunk
        int loads = 0;  // of the dots' other factor: the group's half of a chunk's tile, by its first lane
        const int half = wg - 3;
        const bool issuer = (warp & 3) == 0;
        uint8_t *dt = base + K::OFF_D + half * (K::ZB / 2);
#pragma unroll 1
        for (int n = 0; n < cnt; ++n) {
            const int t0 = at.chunk(NC) * C + h0, cl = min(32, L - t0), bh = at.bh, wi = at.wi;
            const Walk &w = ws.w[wi];
            const bool split = BWD && w.dot != nullptr;
            if (split) {  // once every warp has read the last one
                if (issuer && loads > 0 && !wait(&bars.dread[half], loads - 1)) break;
                if (gtid == 0) {
                    tc::mbar_expect_tx(&bars.dfull[half], K::ZB / 2);
                    tc::tma_load_4d(dt, &maps.d[wi], &bars.dfull[half], 0, t0, 0, bh);
                }
                ++loads;
            }
            const size_t row0 = (size_t)bh * L + t0;
            next(at);
            if (!wait_gate(n) || !wait(&bars.o1done[n & 1], n >> 1) || !wait(&bars.o2read, n)) break;
            tc::tc_fence_after();
            const float *qw = slots[n % SLOTS].qw + h0;
            const uint32_t o1 = tmem + lane_base + K::T_O1 + (n % K::NO1) * 64 + h0, o2 = tmem + lane_base + K::T_O2 + h0;
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
                float a[16], b[16];
                tmem_ld16x2(o1 + e, o2 + e, a, b);
                if (e == 16) warp_arrive(&bars.o_free[n & 1], lane);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(qw + e + i);
                    const float2 x = unpack(fma2(f2(f.x, f.y), f2(a[i], a[i + 1]), f2(b[i], b[i + 1])));
                    const float2 y = unpack(fma2(f2(f.z, f.w), f2(a[i + 2], a[i + 3]), f2(b[i + 2], b[i + 3])));
                    v[e + i] = x.x; v[e + i + 1] = x.y; v[e + i + 2] = y.x; v[e + i + 3] = y.y;
                }
            }
            __syncwarp();
            if (lane == 0 && n % GB == GB - 1) tc::mbar_arrive(&bars.gfree[n / GB & 1]);
            if (j >= 0) {
                TO *out = static_cast<TO *>(w.out) + row0 * B + j;
                if (!BWD && cl == 32) {  // (backwards the code that a second form takes costs more than its predicates)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) put2(out + i * B, out + (i + 1) * B, v[i], v[i + 1], true, true);
                } else {
#pragma unroll
                for (int i = 0; i < 32; i += 2) put2(out + i * B, out + (i + 1) * B, v[i], v[i + 1], i < cl, i + 1 < cl);
                }
            }
            if (split) {
                if (!wait(&bars.dfull[half], loads - 1)) break;
                const int c = (j < 0 ? 0 : j) & 63;
                const uint8_t *x = dt + (j >= 64 ? 4096 : 0) + (c & 7) * 2;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t u = *reinterpret_cast<const unsigned short *>(x + tc::sw128_off(i, c >> 3));
                    v[i] = B == 128 || j >= 0 ? v[i] * bf_lo(u) : 0.f;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.dread[half]);
                const float s = column_sums(v, lane);
                if (lane < cl) w.dot[((size_t)(warp & 3) * BH + bh) * L + t0 + lane] = s;
            }
        }
        if (issuer && loads > 0) tc::mbar_wait(&bars.dfull[half], (loads - 1) & 1, budget / 8);  // nothing in flight at the end
    }
    tc::tc_fence_before();
    __syncthreads();
    if (tid == 0 && abort_flag) atomicOr(&g_decay_error, 1u);
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int A, int B, typename TO, bool BWD>
cudaError_t launch_t(const Maps &maps, const Walks &ws, Gate g, int BH, int L, const Shares &sh, bool out, cudaStream_t s) {
    constexpr int smem = Cfg<A, B, BWD>::SMEM;
    auto *kernel = out ? walk_tc_kernel<A, B, TO, true, BWD> : walk_tc_kernel<A, B, TO, false, BWD>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (out && sh.stretches() > 0) return launch_after(kernel, dim3(sh.g), THREADS, smem, s, maps, ws, sh, g, BH, L);
    kernel<<<out ? sh.g : sh.stretches(), THREADS, smem, s>>>(maps, ws, sh, g, BH, L);
    return cudaGetLastError();
}

template <typename TO, bool BWD>
cudaError_t launch_ab(const Walks &ws, Gate g, int BH, int L, const Shares &sh, bool out, cudaStream_t s) {
    Maps maps;
    for (int i = 0; i < ws.n; ++i) {
        const Walk &w = ws.w[i];
        if (!tmap::make_slabs(&maps.x[i], w.x, w.a / 64, L, BH, C) || !tmap::make_slabs(&maps.y[i], w.y, w.a / 64, L, BH, C) ||
            !tmap::make_slabs(&maps.z[i], w.z, w.b / 64, L, BH, C) ||
            (w.dot && !tmap::make_slabs(&maps.d[i], w.dotx, w.b / 64, L, BH, C / 2)))
            return cudaErrorInvalidValue;
    }
    const int a = ws.w[0].a, b = ws.w[0].b;
    if (a == 128 && b == 128) return launch_t<128, 128, TO, BWD>(maps, ws, g, BH, L, sh, out, s);
    if (a == 128) return launch_t<128, 64, TO, BWD>(maps, ws, g, BH, L, sh, out, s);
    if (b == 128) return launch_t<64, 128, TO, BWD>(maps, ws, g, BH, L, sh, out, s);
    return launch_t<64, 64, TO, BWD>(maps, ws, g, BH, L, sh, out, s);
}

cudaError_t launch_pass(const Walks &ws, Gate g, int BH, int L, const Shares &sh, bool out_bf16, bool bwd, bool out,
                        cudaStream_t s) {
    if (bwd) return launch_ab<__nv_bfloat16, true>(ws, g, BH, L, sh, out, s);
    if (out_bf16) return launch_ab<__nv_bfloat16, false>(ws, g, BH, L, sh, out, s);
    return launch_ab<float, false>(ws, g, BH, L, sh, out, s);
}

}  // namespace

bool tc_sizes(int dk, int dv, bool bf16) { return bf16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

Shares tc_shares(int BH, int L, int n) {
    // In chunks of a walk: whole walks take as many rounds as the device needs for them; even shares take their
    // length, the first pass's, whose chunks cost 0.4 of a walk's and whose stretches are at most a share or most
    // of a walk, and some 6 for its launch and the states between.
    constexpr int SMS = 148;
    const long long units = (long long)BH * n, NC = (L + C - 1) / C, total = units * NC;
    Shares sh{};
    sh.g = (int)units;
    sh.size = NC;
    const long long g = (total / 4 < SMS ? total / 4 : SMS) / n * n;  // four chunks a share or more, walks alike
    if (g < 2 || total >= 1LL << 31) return sh;
    const double whole = (double)((units + SMS - 1) / SMS * NC), even = (double)total / g;
    if (even + 0.4 * (even < NC ? even : 0.7 * NC) + 6. >= whole) return sh;
    sh.g = (int)g;
    sh.size = total / g;
    sh.more = (int)(total % g);
    sh.cut = true;
    return sh;
}

cudaError_t launch_walks_tc(const Walks &ws, Gate g, int BH, int L, const Shares &sh, bool out_bf16, bool bwd,
                            cudaStream_t s) {
    if (sh.stretches() > 0) {
        const cudaError_t e = launch_pass(ws, g, BH, L, sh, out_bf16, bwd, false, s);
        if (e != cudaSuccess) return e;
    }
    return launch_pass(ws, g, BH, L, sh, out_bf16, bwd, true, s);
}

cudaError_t read_and_clear_error(unsigned int *out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_decay_error, sizeof(unsigned int));
    if (e != cudaSuccess || *out == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_decay_error, &zero, sizeof(unsigned int));
}

}  // namespace decay
}  // namespace efla
