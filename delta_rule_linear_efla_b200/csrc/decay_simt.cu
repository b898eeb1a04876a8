// decay_simt.cu -- linear attention with a decay for each head on CUDA cores: fp32 inputs, and
// head sizes that the tensor-core walks do not take.
//
// One CTA walks one stretch of one head for SIMT_BT = 32 value columns (columns of the state do not
// depend on one another), a chunk of 64 tokens at a time, everything in fp32:
//
//   P = D o (X Y^T) (64 x 64),   out = diag(q) X S + P Z,   S <- e^{c_C} S + Y^T diag(w) Z
//
// with D, q and w the decay weights of decay.h.  Every product is register-tiled out of shared
// memory (4 x 4 or 4 x 2 outputs a thread, 16-byte loads along the inner dimension).  32 columns keep
// a CTA at 113 KB, two to an SM, so that one's loads run under the other's arithmetic; P is computed
// again in each column block, up to its diagonal.
//
// What bounds it (fp32, 8 x 32 x 256 tokens, d = 128: 319 us): shared memory's wavefronts (68 % of their
// rate) and issue slots (59 %); a chunk of one column block takes 53,000 warp instructions, 29,000 of them FMAs.
// Short sequences of few heads wait for their chain of chunks: cut into segments of two or more chunks,
// 2 x 3 x 777 tokens take 43 us (76 with four or more, whose loads and joins waited for one another).
#include "decay_gate.cuh"
#include "launchers.h"

#include <type_traits>

namespace efla {
namespace decay {

namespace {

constexpr int NT = 256;
constexpr int BT = SIMT_BT;
constexpr int ZP = BT + 4, PP = C + 4;

struct Lay {
    int ap, xp;  // a rounded up to 4, and the row stride of X and Y
    int oX, oY, oZ, oP, oS, oG, total;
    __host__ __device__ explicit Lay(int a) {
        ap = (a + 3) & ~3;
        xp = ap + 4;
        oX = 0;
        oY = oX + C * xp;
        oZ = oY + C * xp;
        oP = oZ + C * ZP;
        oS = oP + C * PP;
        oG = oS + ap * ZP;
        total = (oG + 4 * C + 4) * (int)sizeof(float);
    }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(float *dst, const void *src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES), "r"(on ? BYTES : 0)
                 : "memory");
}

// V elements a thread and row, V * sizeof(T) bytes at once; d and n are multiples of V.
template <int V, typename T>
__device__ __forceinline__ void load_rows(float *dst, int pitch, const T *src, int d, int j0, int n, int cl, int tid) {
    const int per = n / V, step = NT / per, c = tid % per * V;  // per <= 128
    int r = tid / per;
    if (r >= step) return;
    dst += r * pitch + c;
    const bool in = j0 + c < d;
    const T *p = src + (in ? (size_t)r * d + j0 + c : 0);
    if constexpr (sizeof(T) == 4) {
        for (; r < C; r += step, dst += step * pitch, p += step * d)
            copy_async<4 * V>(dst, in && r < cl ? p : src, in && r < cl);
    } else {
        using U = std::conditional_t<V == 8, uint4, std::conditional_t<V == 4, uint2, std::conditional_t<V == 2, unsigned, unsigned short>>>;
#pragma unroll 8
        for (; r < C; r += step, dst += step * pitch, p += step * d) {
            U u{};
            if (in && r < cl) u = *reinterpret_cast<const U *>(p);
            const T *h = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int i = 0; i < V; ++i) dst[i] = to_f32(h[i]);
        }
    }
}

// Rows 0 .. C - 1 of src [][d], columns [j0, j0 + n), zero from row cl and column d on.  fp32 comes by asynchronous
// copies, all in flight at once; copies_done() waits for the thread's own.
template <typename T>
__device__ __forceinline__ void load_tile(float *dst, int pitch, const T *src, int d, int j0, int n, int cl, int tid) {
    const unsigned at = (unsigned)reinterpret_cast<uintptr_t>(src) / (unsigned)sizeof(T) | d | n;  // src, rows and n: multiples of V?
    if constexpr (sizeof(T) == 4) {
        if (at % 4 == 0) load_rows<4>(dst, pitch, src, d, j0, n, cl, tid);
        else load_rows<1>(dst, pitch, src, d, j0, n, cl, tid);
    } else {
        if (at % 8 == 0) load_rows<8>(dst, pitch, src, d, j0, n, cl, tid);
        else if (at % 4 == 0) load_rows<4>(dst, pitch, src, d, j0, n, cl, tid);
        else if (at % 2 == 0) load_rows<2>(dst, pitch, src, d, j0, n, cl, tid);
        else load_rows<1>(dst, pitch, src, d, j0, n, cl, tid);
    }
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void fma4(float (&acc)[4], float s, const float4 &v) {
    acc[0] = fmaf(s, v.x, acc[0]);
    acc[1] = fmaf(s, v.y, acc[1]);
    acc[2] = fmaf(s, v.z, acc[2]);
    acc[3] = fmaf(s, v.w, acc[3]);
}

// Rows r .. r + 3 of P = D o (X Y^T), at columns c, c + 16, .. (NJ of them).
template <int NJ>
__device__ __forceinline__ void scores(float *P, const float *X, const float *Y, int xp, int ap, const float *chi,
                                       const float *clo, int r, int c, bool rev) {
    float p[4][NJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[i][j] = 0.f;
#pragma unroll 2
    for (int k = 0; k < ap; k += 4) {
        float4 xv[4], yv[NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const float4 *>(X + (r + i) * xp + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) yv[j] = *reinterpret_cast<const float4 *>(Y + (c + 16 * j) * xp + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                p[i][j] = fmaf(xv[i].x, yv[j].x, fmaf(xv[i].y, yv[j].y, fmaf(xv[i].z, yv[j].z, fmaf(xv[i].w, yv[j].w, p[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int t = r + i, u = c + 16 * j;
            const float d = (chi[t] - chi[u]) + (clo[t] - clo[u]);
            P[t * PP + u] = (rev ? u >= t : u <= t) ? p[i][j] * exp2f(rev ? -d : d) : 0.f;
        }
}

// S <- e S + Y^T diag(kw) Z over n tokens: RT x 4 elements a thread, so that its 256 threads cover 32 RT rows.
template <int RT>
__device__ __forceinline__ void update_state(float *S, const float *Y, const float *Z, const float *kw, float e, int xp,
                                             int ap, int n, int tid) {
    const int si = (tid >> 3) * RT, sc = (tid & 7) * 4;
    if (si >= ap) return;
    float acc[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
        float yv[RT];
        if constexpr (RT == 4) *reinterpret_cast<float4 *>(yv) = *reinterpret_cast<const float4 *>(Y + t * xp + si);
        else *reinterpret_cast<float2 *>(yv) = *reinterpret_cast<const float2 *>(Y + t * xp + si);
        float4 zv = *reinterpret_cast<const float4 *>(Z + t * ZP + sc);
        const float f = kw[t];
        zv.x *= f; zv.y *= f; zv.z *= f; zv.w *= f;
#pragma unroll
        for (int i = 0; i < RT; ++i) fma4(acc[i], yv[i], zv);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float4 *s4 = reinterpret_cast<float4 *>(S + (si + i) * ZP + sc);
        float4 s = *s4;
        s.x = fmaf(e, s.x, acc[i][0]); s.y = fmaf(e, s.y, acc[i][1]);
        s.z = fmaf(e, s.z, acc[i][2]); s.w = fmaf(e, s.w, acc[i][3]);
        *s4 = s;
    }
}

// OUT = false: the stretch's own contribution to the state only (segments' first pass).
template <typename T, typename TO, bool OUT>
__global__ void __launch_bounds__(NT, 2)
    walk_simt_kernel(const __grid_constant__ Walks ws, const __grid_constant__ Segments sg, const Gate g, int BH, int L) {
    extern __shared__ __align__(16) float sm[];
    // ---- which walk, column block and head: blockIdx.x = (block of all walks) * BH + bh
    const int bh = blockIdx.x % BH;
    int blk = blockIdx.x / BH, wi = 0;
    while (wi + 1 < ws.n && blk >= (ws.w[wi].b + BT - 1) / BT) {
        blk -= (ws.w[wi].b + BT - 1) / BT;
        ++wi;
    }
    const Walk &w = ws.w[wi];
    const int a = w.a, b = w.b, j0 = blk * BT, nb = min(BT, b - j0);
    const bool rev = w.rev != 0;
    const Lay lay(a);
    float *X = sm + lay.oX, *Y = sm + lay.oY, *Z = sm + lay.oZ, *P = sm + lay.oP, *S = sm + lay.oS;
    float *qw = sm + lay.oG, *kw = qw + C, *chi = kw + C, *clo = chi + C, *tot = clo + C;
    const int xp = lay.xp, ap = lay.ap;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int NC = (L + C - 1) / C;
    const int seg = blockIdx.y;  // in walking order
    const int i0 = seg * sg.chunks, i1 = min(NC, i0 + sg.chunks);
    if (OUT) cudaGridDependencySynchronize();

    // ---- the state that enters
    const size_t sbh = (size_t)bh * a * b;
    const float *s0 = OUT && w.s0 ? w.s0 + sbh : nullptr;
    const float *eb = sg.e + ((size_t)(rev ? 1 : 0) * BH + bh) * (sg.n - 1), *ub = sg.u[wi] + (size_t)bh * (sg.n - 1) * a * b;
    if (OUT && s0 && w.s0_t) {
        for (int e = tid; e < a * nb; e += NT) {  // along the stored rows
            const int j = e / a, i = e - j * a;
            S[i * ZP + j] = s0[(size_t)(j0 + j) * a + i];
        }
        __syncthreads();
    }
    {
        constexpr int PER = 128 / (NT / BT);  // a <= 128
        const int i0 = tid / BT, j = tid % BT;
        float v[PER];
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int i = i0 + m * (NT / BT);
            v[m] = OUT && s0 && i < a && j < nb ? (w.s0_t ? S[i * ZP + j] : s0[(size_t)i * b + j0 + j]) : 0.f;
        }
        if (OUT && j < nb)
#pragma unroll 2
            for (int k = 0; k < seg; ++k) {
                const float e = eb[k], *u = ub + (size_t)k * a * b + (size_t)i0 * b + j0 + j;
#pragma unroll
                for (int m = 0; m < PER; ++m)
                    if (i0 + m * (NT / BT) < a) v[m] = fmaf(e, v[m], u[(size_t)m * (NT / BT) * b]);
            }
#pragma unroll
        for (int m = 0; m < PER; ++m)
            if (i0 + m * (NT / BT) < ap) S[(i0 + m * (NT / BT)) * ZP + j] = v[m];
    }
    Fixed seg_sum = 0;
    bool seg_good = true;

    // P: rows r4.., columns tc + 16 j up to the diagonal; out: columns 2 tc, 2 tc + 1.  Warps w and w + 4, which an
    // SM's scheduler holds together, have five column blocks of P between them.
    const int r4 = 8 * (warp < 4 ? warp : 11 - warp) + 4 * (lane >> 4), tc = tid & 15;
    const int jb = r4 / 16, j_lo = rev ? jb : 0, nj = rev ? 4 - jb : jb + 1;
    const size_t head = (size_t)bh * L;
    auto load_x = [&](int it) {
        const int t0 = (rev ? NC - 1 - it : it) * C;
        load_tile(X, xp, static_cast<const T *>(w.x) + (head + t0) * a, a, 0, ap, min(C, L - t0), tid);
    };
    if (OUT) load_x(i0);
    for (int it = i0; it < i1; ++it) {
        const int n = rev ? NC - 1 - it : it;
        const int t0 = n * C, cl = min(C, L - t0);
        const size_t row0 = head + t0;
        __syncthreads();  // the chunk before is done with every buffer
        load_tile(Y, xp, static_cast<const T *>(w.y) + row0 * a, a, 0, ap, cl, tid);
        load_tile(Z, ZP, static_cast<const T *>(w.z) + row0 * b, b, j0, BT, cl, tid);
        if (warp == 0) {
            const int t = t0 + 2 * lane;
            const PairSum c = chunk_sums(gate_or_zero(g, bh, L, t), gate_or_zero(g, bh, L, t + 1), lane);
            const Fixed cc[2] = {c.c0, c.c1};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const float up = if_good(exp2_fixed(cc[e]), t < c.bad), down = if_good(exp2_fixed(c.cC - cc[e]), c.bad == C || t >= c.bad);
                qw[t] = rev ? down : up;
                kw[t] = rev ? up : down;
                const float hi = __ll2float_rn(cc[e]);
                chi[t] = if_good(hi * (1.f / FIXED_ONE), t < c.bad);
                clo[t] = __ll2float_rn(cc[e] - __float2ll_rn(hi)) * (1.f / FIXED_ONE);
            }
            if (lane == 0) tot[0] = if_good(exp2_fixed(c.cC), c.bad == C);
            seg_sum = max(seg_sum + c.cC, FIXED_MIN);
            seg_good = seg_good && c.bad == C;
        }
        copies_done();
        __syncthreads();
        if (OUT) {
            if (r4 < cl) {
                const int c0 = tc + 16 * j_lo;
                if (nj == 1) scores<1>(P, X, Y, xp, ap, chi, clo, r4, c0, rev);
                else if (nj == 2) scores<2>(P, X, Y, xp, ap, chi, clo, r4, c0, rev);
                else if (nj == 3) scores<3>(P, X, Y, xp, ap, chi, clo, r4, c0, rev);
                else scores<4>(P, X, Y, xp, ap, chi, clo, r4, c0, rev);
            }
            __syncthreads();
            // ---- out = diag(q) X S + P Z: 4 rows x 2 columns a thread
            float o[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i][0] = o[i][1] = 0.f;
            const int cc = 2 * tc;
            const int ka = r4 < cl ? ap : 0;
#pragma unroll 2
            for (int k = 0; k < ka; k += 4) {
                float4 xv[4];
                float2 sv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const float4 *>(X + (r4 + i) * xp + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) sv[j] = *reinterpret_cast<const float2 *>(S + (k + j) * ZP + cc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i][0] = fmaf(xv[i].x, sv[0].x, fmaf(xv[i].y, sv[1].x, fmaf(xv[i].z, sv[2].x, fmaf(xv[i].w, sv[3].x, o[i][0]))));
                    o[i][1] = fmaf(xv[i].x, sv[0].y, fmaf(xv[i].y, sv[1].y, fmaf(xv[i].z, sv[2].y, fmaf(xv[i].w, sv[3].y, o[i][1]))));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i][0] *= qw[r4 + i];
                o[i][1] *= qw[r4 + i];
            }
            const int k0 = rev ? r4 : 0, k1 = r4 >= cl ? k0 : rev ? cl : r4 + 4;  // the rest of P's rows, or of Z, is zero
#pragma unroll 2
            for (int k = k0; k < k1; k += 4) {
                float4 pv[4];
                float2 zv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4 *>(P + (r4 + i) * PP + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) zv[j] = *reinterpret_cast<const float2 *>(Z + (k + j) * ZP + cc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i][0] = fmaf(pv[i].x, zv[0].x, fmaf(pv[i].y, zv[1].x, fmaf(pv[i].z, zv[2].x, fmaf(pv[i].w, zv[3].x, o[i][0]))));
                    o[i][1] = fmaf(pv[i].x, zv[0].y, fmaf(pv[i].y, zv[1].y, fmaf(pv[i].z, zv[2].y, fmaf(pv[i].w, zv[3].y, o[i][1]))));
                }
            }
            TO *out = static_cast<TO *>(w.out) + row0 * b + j0;
            const T *dx = w.dot ? static_cast<const T *>(w.dotx) + row0 * b + j0 : nullptr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r4 + i;
                double dd = 0.0;  // q.dq and k.dk cancel in dl's sums: their own rounding is kept out of them
                if (r < cl) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (cc + j < nb) {
                            out[(size_t)r * b + cc + j] = from_f32<TO>(o[i][j]);
                            if (dx) dd += (double)to_f32(dx[(size_t)r * b + cc + j]) * (double)o[i][j];
                        }
                }
                if (dx) {  // the row's 16 threads are half a warp
#pragma unroll
                    for (int off = 8; off > 0; off >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, off);
                    if (tc == 0 && r < cl) w.dot[((size_t)blk * BH + bh) * L + t0 + r] = (float)dd;
                }
            }
            __syncthreads();  // the state and X are read
            if (it + 1 < i1) load_x(it + 1);
        }
        if (ap > 64) update_state<4>(S, Y, Z, kw, tot[0], xp, ap, cl, tid);
        else update_state<2>(S, Y, Z, kw, tot[0], xp, ap, cl, tid);
    }
    __syncthreads();
    float *sout = nullptr;
    if (!OUT) sout = sg.u[wi] + ((size_t)bh * (sg.n - 1) + seg) * a * b;
    else if (seg == sg.n - 1 && w.s_end) sout = w.s_end + sbh;
    if (sout) {
        for (int e = tid; e < a * BT; e += NT) {
            const int i = e / BT, j = e % BT;
            if (j < nb) sout[(size_t)i * b + j0 + j] = S[i * ZP + j];
        }
    }
    // every walk in the same direction finds the same decay of a segment: its first one writes it
    if (!OUT && warp == 0 && lane == 0 && blk == 0 && (wi == 0 || ws.w[wi - 1].rev != w.rev))
        sg.e[((size_t)(rev ? 1 : 0) * BH + bh) * (sg.n - 1) + seg] = if_good(exp2_fixed(seg_sum), seg_good);
}

template <typename T, typename TO>
cudaError_t launch_t(const Walks &ws, Gate g, int BH, int L, const Segments &sg, cudaStream_t s) {
    int blocks = 0, smem = 0;
    for (int i = 0; i < ws.n; ++i) {
        blocks += (ws.w[i].b + BT - 1) / BT;
        const int t = Lay(ws.w[i].a).total;
        smem = t > smem ? t : smem;
    }
    auto *full = walk_simt_kernel<T, TO, true>;
    auto *part = walk_simt_kernel<T, TO, false>;
    // The most that any head size takes: the limit belongs to the kernel, and another thread's call of a smaller head
    // size must not lower it between here and the launch.
    const int most = Lay(128).total;
    cudaError_t e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && sg.n > 1) e = cudaFuncSetAttribute(part, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (sg.n == 1) {
        full<<<dim3(blocks * BH), NT, smem, s>>>(ws, sg, g, BH, L);
        count_launches(1);
        return cudaGetLastError();
    }
    part<<<dim3(blocks * BH, sg.n - 1), NT, smem, s>>>(ws, sg, g, BH, L);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_after(full, dim3(blocks * BH, sg.n), NT, smem, s, ws, sg, g, BH, L);
}

constexpr int DL_T = 512, DL_E = 8;  // tokens at once: 4096

// One CTA per head, 4096 tokens at a time from the end: a block-wide suffix sum in fp64 (the differences q.dq - k.dk
// of a long sequence cancel down to the pairs that straddle a token).  At a token that forgets everything the sum is
// zero by definition, and starts anew before it: the rounding of what is behind does not reach the documents in front.
template <typename T>
__global__ void __launch_bounds__(DL_T)
    dlog_kernel(const float *__restrict__ dotq, int nq, const float *__restrict__ dotk, int nk,
                const float *__restrict__ dS, const float *__restrict__ S_end, const Gate g, T *__restrict__ dlog,
                int BH, int L, int dk, int dv) {
    __shared__ double part[DL_T / 32];
    __shared__ int part_cut[DL_T / 32];
    __shared__ double carry_s;
    const int bh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    cudaGridDependencySynchronize();
    double carry = 0.0;
    if (dS) {  // <dS_final, S_final>
        const size_t base = (size_t)bh * dk * dv;
        double t = 0.0;
        for (int e = tid; e < dk * dv; e += DL_T) {
            const int i = e / dk, j = e - i * dk;  // S_end is [dv][dk]
            t += (double)S_end[base + e] * (double)dS[base + (size_t)j * dv + i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) part[warp] = t;
        __syncthreads();
        for (int i = 0; i < DL_T / 32; ++i) carry += part[i];
        __syncthreads();
    }
    const size_t row = (size_t)bh * L, plane = (size_t)BH * L;
    for (int lo = (L - 1) / (DL_T * DL_E) * (DL_T * DL_E); lo >= 0; lo -= DL_T * DL_E) {
        // thread tid holds tokens t0 .. t0 + DL_E - 1, and the sums behind them
        const int t0 = lo + tid * DL_E;
        double x[DL_E];
#pragma unroll
        for (int e = 0; e < DL_E; ++e) x[e] = 0.0;
        if (t0 < L) {
            const bool whole = t0 + DL_E <= L && L % 4 == 0;  // then every row of the planes is 16-byte aligned
            for (int i = 0; i < nq + nk; ++i) {
                const float *p = (i < nq ? dotq + i * plane : dotk + (i - nq) * plane) + row + t0;
                float v[DL_E];
                if (whole) {
#pragma unroll
                    for (int e = 0; e < DL_E; e += 4) *reinterpret_cast<float4 *>(v + e) = *reinterpret_cast<const float4 *>(p + e);
                } else {
#pragma unroll
                    for (int e = 0; e < DL_E; ++e) v[e] = t0 + e < L ? p[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < DL_E; ++e) x[e] += i < nq ? (double)v[e] : -(double)v[e];
            }
        }
        // sums within the thread, from its end or from the last forgetting token on
        unsigned forgets = 0;  // bit e: token t0 + e
#pragma unroll
        for (int e = 0; e < DL_E; ++e)
            if (t0 + e < L && gate_at(g, bh, L, t0 + e) == L_MIN) forgets |= 1u << e;
#pragma unroll
        for (int e = DL_E - 1; e >= 0; --e) x[e] = forgets >> e & 1 ? 0.0 : e + 1 < DL_E ? x[e] + x[e + 1] : x[e];
        // over the warp's threads from this one on; cut: up to a forgetting token among them
        double s = x[0];
        int cut = forgets != 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_down_sync(0xffffffffu, s, o);
            const int c = __shfl_down_sync(0xffffffffu, cut, o);
            if (lane + o < 32 && !cut) {
                s += y;
                cut = c;
            }
        }
        if (lane == 0) {
            part[warp] = s;
            part_cut[warp] = cut;
        }
        // what reaches this thread from behind: the rest of its warp, the warps behind, the tokens behind them
        double behind = __shfl_down_sync(0xffffffffu, s, 1);
        cut = __shfl_down_sync(0xffffffffu, cut, 1);
        if (lane == 31) {
            behind = 0.0;
            cut = 0;
        }
        __syncthreads();
        for (int i = warp + 1; i < DL_T / 32 && !cut; ++i) {
            behind += part[i];
            cut = part_cut[i];
        }
        if (!cut) behind += carry;
#pragma unroll
        for (int e = 0; e < DL_E; ++e) {
            const int t = t0 + e;
            if (forgets >> e == 0) x[e] += behind;
            if (t < L) dlog[row + t] = from_f32<T>((float)x[e]);
        }
        if (tid == 0) carry_s = x[0];
        __syncthreads();
        carry = carry_s;
    }
}

}  // namespace

Segments simt_segments(int BH, int L, const int *blocks, int n) {
    // In chunks of a walk: two CTAs an SM take rounds of n segments' chunks each, a first pass (the state update
    // alone) another 0.35 of them, joining the states of the segments before some 0.05 a segment, and the launch 1.
    constexpr int SLOTS = 2 * 148;
    Segments sg{};
    long long ctas = 0;
    for (int i = 0; i < n; ++i) ctas += (long long)blocks[i] * BH;
    const int NC = (L + C - 1) / C;
    sg.n = 1;
    sg.chunks = NC;
    double best = (double)((ctas + SLOTS - 1) / SLOTS) * NC;
    for (int k = 2; k <= NC / 2 && ctas * k <= 4 * SLOTS; ++k) {
        const int chunks = (NC + k - 1) / k, m = (NC + chunks - 1) / chunks;
        const double cost = (double)((ctas * m + SLOTS - 1) / SLOTS) * chunks * 1.35 + 0.05 * m + 1.;
        if (cost < best) {
            best = cost;
            sg.n = m;
            sg.chunks = chunks;
        }
    }
    return sg;
}

cudaError_t launch_walks_simt(const Walks &ws, Gate g, int BH, int L, const Segments &sg, bool in_bf16, bool out_bf16,
                              cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (in_bf16) return out_bf16 ? launch_t<bf, bf>(ws, g, BH, L, sg, s) : launch_t<bf, float>(ws, g, BH, L, sg, s);
    return out_bf16 ? launch_t<float, bf>(ws, g, BH, L, sg, s) : launch_t<float, float>(ws, g, BH, L, sg, s);
}

cudaError_t launch_dlog(const float *dotq, int nq, const float *dotk, int nk, const float *dS_final,
                        const float *S_end, Gate g, void *dlog, int BH, int L, int dk, int dv, cudaStream_t s) {
    count_launches(1);
    if (g.bf16)
        return launch_after(dlog_kernel<__nv_bfloat16>, dim3(BH), DL_T, 0, s, dotq, nq, dotk, nk, dS_final, S_end, g,
                            (__nv_bfloat16 *)dlog, BH, L, dk, dv);
    return launch_after(dlog_kernel<float>, dim3(BH), DL_T, 0, s, dotq, nq, dotk, nk, dS_final, S_end, g, (float *)dlog, BH,
                        L, dk, dv);
}

}  // namespace decay
}  // namespace efla
