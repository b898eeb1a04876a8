// norms.cu -- per-head norms before (head norm) and after (gated norm) the attention, with their
// gradients; the change between the projections' layout [B,L,H,d] and the kernels' [B,H,L,d] happens
// on the way.
//
// HBM-bound: every tensor is read or written once.  A row of d elements belongs to a group of G lanes
// of one warp, each with its elements in registers (16-byte pieces where d, the strides and the
// pointers allow it), so the row's sums are a few shuffles and nothing goes through shared memory.
// Rows are walked in the order (b, t, h): a warp's consecutive rows are consecutive in the
// projections' layout.  The weight's gradient is summed by each thread over its rows, then over the
// CTA and over the CTAs in a fixed order, all in fp32.
#include "common.cuh"
#include "launchers.h"
#include "norms.h"

namespace efla {
namespace norms {

namespace {

constexpr int NT = 256;
constexpr int MAX_CTAS = 148 * 8;

template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> { using V = uint4; };
template <> struct Piece<float, 4> { using V = uint4; };
template <> struct Piece<__nv_bfloat16, 4> { using V = uint2; };
template <> struct Piece<float, 1> { using V = uint32_t; };
template <> struct Piece<__nv_bfloat16, 1> { using V = uint16_t; };

// A piece as it was loaded; zeros where there is none.
template <typename T, int VEC>
struct Raw {
    typename Piece<T, VEC>::V u;
    __device__ __forceinline__ void load(const T *p, bool on) {
        u = on ? *reinterpret_cast<const typename Piece<T, VEC>::V *>(p) : typename Piece<T, VEC>::V{};
    }
    __device__ __forceinline__ void to(float (&f)[VEC]) const {
        const T *h = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f32(h[i]);
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void st(T *p, const float (&f)[VEC]) {
    typename Piece<T, VEC>::V u;
    T *h = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = from_f32<T>(f[i]);
    *reinterpret_cast<typename Piece<T, VEC>::V *>(p) = u;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float weight_at(const Weight &w, int i) {
    if (!w.p) return 1.f;
    return w.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w.p)[i]) : static_cast<const float *>(w.p)[i];
}

__device__ __forceinline__ unsigned div(unsigned n, const Div &d) {
    return (unsigned)(((unsigned long long)__umulhi(n, d.mul) + n) >> d.shift);
}

// Where row r = (b L + t) H + h lies: in the view's strides, and in the kernels' layout [B,H,L,d].
struct Row {
    unsigned b, t, h;
    __device__ __forceinline__ Row(unsigned r, const Sizes &n) {
        const unsigned bt = div(r, n.byH);
        h = r - bt * n.H;
        b = div(bt, n.byL);
        t = bt - b * n.L;
    }
    __device__ __forceinline__ size_t at(const View &v) const { return b * v.sb + t * v.sl + h * v.sh; }
    __device__ __forceinline__ size_t heads(const Sizes &n) const {
        return (((size_t)b * n.H + h) * n.L + t) * n.d;
    }
};

// The weight gradient's shares: acc of every thread -> part[blockIdx.x][d].
template <int VEC, int NV, int G>
__device__ __forceinline__ void store_dw(float (&acc)[NV][VEC], float *part, int d, int lane) {
    __shared__ float red[NT / 32][DMAX];
    // the groups of a warp, then the warps
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int o = G; o < 32; o <<= 1) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], o);
            const int i = (j * G + lane % G) * VEC + e;
            if (lane < G && i < d) red[threadIdx.x >> 5][i] = acc[j][e];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < d; i += NT) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) x += red[w][i];
        part[(size_t)blockIdx.x * d + i] = x;
    }
}

// dw[i] = sum of the CTAs' shares, in a fixed order: eight columns a CTA, 128 threads a column.
template <typename TW>
__global__ void __launch_bounds__(1024) sum_dw_kernel(const float *__restrict__ part, TW *__restrict__ dw, int rows, int d) {
    __shared__ float red[32][8];
    cudaGridDependencySynchronize();
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3, i = blockIdx.x * 8 + c;
    float x = 0.f;
    if (i < d) {
#pragma unroll 5
        for (int r = g; r < rows; r += 128) x += part[(size_t)r * d + i];
    }
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    if ((threadIdx.x & 31) < 8) red[threadIdx.x >> 5][c] = x;
    __syncthreads();
    if (threadIdx.x < 8 && i < d) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) s += red[r][c];
        dw[i] = from_f32<TW>(s);
    }
}

// Every kernel takes R rows a group at once: their loads are all on the way before the first is used.  Rows of
// one turn are neighbours (group g of a warp or block takes g, g + groups, ...), turns are a grid apart.
template <int VEC, int NV, int G>
struct Group {
    int gl;
    __device__ __forceinline__ Group() : gl(threadIdx.x % G) {}
    __device__ __forceinline__ int at(int j) const { return (j * G + gl) * VEC; }
    __device__ __forceinline__ void weights(float (&wv)[NV][VEC], const Weight &w, int d, float scale) const {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) wv[j][e] = at(j) + e < d ? scale * weight_at(w, at(j) + e) : 0.f;
    }
    template <typename T>
    __device__ __forceinline__ void load(Raw<T, VEC> (&f)[NV], const T *p, int d, bool on) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) f[j].load(p + at(j), on && at(j) < d);
    }
    template <typename T>
    __device__ __forceinline__ static void to(float (&f)[NV][VEC], const Raw<T, VEC> (&r)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) r[j].to(f[j]);
    }
    template <typename T>
    __device__ __forceinline__ void store(T *p, const float (&f)[NV][VEC], int d, bool on) const {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on && at(j) < d) st<T, VEC>(p + at(j), f[j]);
    }
    __device__ __forceinline__ float norm(const float (&f)[NV][VEC], float m, float eps) const {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(f[j][e], f[j][e], sum);
        return rsqrtf(fmaf(m, group_sum<G>(sum), eps));
    }
};

// ------------------------------------------------------------------ head norm
template <typename T, int VEC, int NV, int G, int R>
__global__ void __launch_bounds__(NT, 4)
    head_norm_kernel(const View x, const Weight w, T *__restrict__ y, const Sizes n, unsigned rows, float m, float scale, float eps) {
    const Group<VEC, NV, G> g;
    constexpr unsigned RPC = NT / G;
    float wv[NV][VEC];
    g.weights(wv, w, n.d, scale);
    for (unsigned r0 = blockIdx.x * RPC * R + threadIdx.x / G; r0 - threadIdx.x / G < rows; r0 += gridDim.x * RPC * R) {
        Raw<T, VEC> xr[R][NV];
        size_t out[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            const Row row(r < rows ? r : 0, n);
            g.load(xr[k], static_cast<const T *>(x.p) + row.at(x), n.d, r < rows);
            out[k] = row.heads(n);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float f[NV][VEC];
            g.to(f, xr[k]);
            const float rs = g.norm(f, m, eps);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[j][e] = f[j][e] * rs * wv[j][e];
            g.store(y + out[k], f, n.d, r0 + k * RPC < rows);
        }
    }
}

template <typename T, int VEC, int NV, int G, int R>
__global__ void __launch_bounds__(NT, 4)
    head_norm_bwd_kernel(const View x, const Weight w, const T *__restrict__ dy, T *__restrict__ dx,
                         float *__restrict__ part, const Sizes n, unsigned rows, float m, float scale, float eps) {
    const Group<VEC, NV, G> g;
    constexpr unsigned RPC = NT / G;
    float wv[NV][VEC], acc[NV][VEC];
    g.weights(wv, w, n.d, scale);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    for (unsigned r0 = blockIdx.x * RPC * R + threadIdx.x / G; r0 - threadIdx.x / G < rows; r0 += gridDim.x * RPC * R) {
        Raw<T, VEC> xr[R][NV], dr[R][NV];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            const Row row(r < rows ? r : 0, n);
            g.load(xr[k], static_cast<const T *>(x.p) + row.at(x), n.d, r < rows);
            g.load(dr[k], dy + row.heads(n), n.d, r < rows);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            float f[1][NV][VEC], gd[1][NV][VEC];
            g.to(f[0], xr[k]);
            g.to(gd[0], dr[k]);
            const float rs = g.norm(f[0], m, eps);
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float nn = f[0][j][e] * rs;
                    if (r < rows) acc[j][e] = fmaf(gd[0][j][e], nn, acc[j][e]);
                    const float dn = gd[0][j][e] * wv[j][e];
                    dot = fmaf(dn, nn, dot);
                    f[0][j][e] = nn;
                    gd[0][j][e] = dn;
                }
            dot = m * group_sum<G>(dot);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[0][j][e] = rs * fmaf(-dot, f[0][j][e], gd[0][j][e]);
            g.store(dx + (size_t)r * n.d, f[0], n.d, r < rows);
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] *= scale;
        store_dw<VEC, NV, G>(acc, part, n.d, threadIdx.x & 31);
    }
}

// ------------------------------------------------------------------ gated norm
// 1 / (1 + e^-x).  Where everything made from it is bf16, the fast exponential and division: off by 2 + 1.17 |x| ulp
// and 2 ulp (at most 1.3e-5 of the value, for gates near -87), far below bf16's rounding; and 0 below -87, where e^-x
// leaves the division's range.  An fp32 weight's gradient is summed from those values too: the relative error is that
// of its terms, and those of gates far below zero, whose error is large, count least.  Outputs in fp32 (a gate's
// own type forwards, the gate's or o's backwards) take the accurate ones.
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid_of(float x) {
    if constexpr (ACCURATE) return 1.f / (1.f + expf(-x));
    else return x < -87.f ? 0.f : __fdividef(1.f, 1.f + __expf(-x));
}

template <typename T, typename TO, int VEC, int NV, int G, int R>
__global__ void __launch_bounds__(NT, 4)
    gated_norm_kernel(const TO *__restrict__ o, const View gate, const Weight w, const View res, T *__restrict__ y,
                      const Sizes n, unsigned rows, bool silu, float scale, float eps) {
    constexpr bool ACC = sizeof(T) == 4;
    const Group<VEC, NV, G> g;
    constexpr unsigned RPC = NT / G;
    const float m = 1.f / n.d;
    float wv[NV][VEC];
    g.weights(wv, w, n.d, scale);
    for (unsigned r0 = blockIdx.x * RPC * R + threadIdx.x / G; r0 - threadIdx.x / G < rows; r0 += gridDim.x * RPC * R) {
        Raw<TO, VEC> fr[R][NV];
        Raw<T, VEC> gr[R][NV], rr[R][NV];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            const Row row(r < rows ? r : 0, n);
            g.load(fr[k], o + row.heads(n), n.d, r < rows);
            g.load(gr[k], static_cast<const T *>(gate.p) + row.at(gate), n.d, r < rows);
            g.load(rr[k], static_cast<const T *>(res.p) + row.at(res), n.d, res.p && r < rows);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            float f[1][NV][VEC], gv[1][NV][VEC], rv[1][NV][VEC];
            g.to(f[0], fr[k]);
            g.to(gv[0], gr[k]);
            g.to(rv[0], rr[k]);
            const float rs = g.norm(f[0], m, eps);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float sg = sigmoid_of<ACC>(gv[0][j][e]), a = silu ? gv[0][j][e] * sg : sg;
                    f[0][j][e] = fmaf(f[0][j][e] * rs * wv[j][e], a, rv[0][j][e]);
                }
            g.store(y + (size_t)r * n.d, f[0], n.d, r < rows);
        }
    }
}

template <typename T, typename TO, int VEC, int NV, int G, int R>
__global__ void __launch_bounds__(NT, 4)
    gated_norm_bwd_kernel(const TO *__restrict__ o, const View gate, const Weight w, const T *__restrict__ dy,
                          TO *__restrict__ d_o, T *__restrict__ dgate, float *__restrict__ part, const Sizes n,
                          unsigned rows, bool silu, float scale, float eps) {
    constexpr bool ACC = sizeof(T) == 4 || sizeof(TO) == 4;
    const Group<VEC, NV, G> g;
    constexpr unsigned RPC = NT / G;
    const float m = 1.f / n.d;
    float wv[NV][VEC], acc[NV][VEC];
    g.weights(wv, w, n.d, scale);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    for (unsigned r0 = blockIdx.x * RPC * R + threadIdx.x / G; r0 - threadIdx.x / G < rows; r0 += gridDim.x * RPC * R) {
        Raw<TO, VEC> fr[R][NV];
        Raw<T, VEC> gr[R][NV], dr[R][NV];
        size_t at_o[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            const Row row(r < rows ? r : 0, n);
            at_o[k] = row.heads(n);
            g.load(fr[k], o + at_o[k], n.d, r < rows);
            g.load(gr[k], static_cast<const T *>(gate.p) + row.at(gate), n.d, r < rows);
            g.load(dr[k], dy + (size_t)r * n.d, n.d, r < rows);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const unsigned r = r0 + k * RPC;
            float f[1][NV][VEC], gv[1][NV][VEC], gd[1][NV][VEC];
            g.to(f[0], fr[k]);
            g.to(gv[0], gr[k]);
            g.to(gd[0], dr[k]);
            const float rs = g.norm(f[0], m, eps);
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float x = gv[0][j][e], sg = sigmoid_of<ACC>(x);
                    const float a = silu ? x * sg : sg, da = silu ? sg * fmaf(x, 1.f - sg, 1.f) : sg * (1.f - sg);
                    const float nn = f[0][j][e] * rs, dyv = gd[0][j][e];
                    if (r < rows) acc[j][e] = fmaf(dyv * a, nn, acc[j][e]);
                    const float dyw = dyv * wv[j][e];
                    gv[0][j][e] = dyw * nn * da;  // dgate
                    gd[0][j][e] = dyw * a;        // dn
                    f[0][j][e] = nn;
                    dot = fmaf(gd[0][j][e], nn, dot);
                }
            dot = m * group_sum<G>(dot);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[0][j][e] = rs * fmaf(-dot, f[0][j][e], gd[0][j][e]);
            g.store(d_o + at_o[k], f[0], n.d, r < rows);
            g.store(dgate + (size_t)r * n.d, gv[0], n.d, r < rows);
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] *= scale;
        store_dw<VEC, NV, G>(acc, part, n.d, threadIdx.x & 31);
    }
}

// ------------------------------------------------------------------ dispatch
bool wide(const void *p, int bytes) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool wide(const View &v, int vec) { return v.p == nullptr || (v.sb % vec == 0 && v.sl % vec == 0 && v.sh % vec == 0); }

// Calls f(VEC, NV, G as constants): rows of d elements on G lanes with NV pieces of VEC elements each.
// VEC: elements of a 16-byte piece, or 1 where some pointer, stride or d is not a multiple of it.
template <int V> struct Int { static constexpr int value = V; };
template <int VEC, typename F>
cudaError_t by_width(int d, F f) {
    if constexpr (VEC == 1) {
        if (d <= 32) return f(Int<1>(), Int<1>(), Int<32>());
        if (d <= 64) return f(Int<1>(), Int<2>(), Int<32>());
        if (d <= 128) return f(Int<1>(), Int<4>(), Int<32>());
        return f(Int<1>(), Int<8>(), Int<32>());
    } else {
        const int p = (d + VEC - 1) / VEC;
        if (p <= 4) return f(Int<VEC>(), Int<1>(), Int<4>());
        if (p <= 8) return f(Int<VEC>(), Int<1>(), Int<8>());
        if (p <= 16) return f(Int<VEC>(), Int<1>(), Int<16>());
        if (p <= 32) return f(Int<VEC>(), Int<1>(), Int<32>());
        return f(Int<VEC>(), Int<2>(), Int<32>());
    }
}

// Blocks of R rows a group: at most eight a processor, which then take turns.
unsigned grid_for(const Sizes &n, int G, int R) {
    const long long rpc = (long long)(NT / G) * R, want = (n.rows() + rpc - 1) / rpc;
    return (unsigned)(want < MAX_CTAS ? want : MAX_CTAS);
}
// Rows at once: as many as keep a thread's pieces in registers; one where there are few (the blocks then spread).
template <int NV> constexpr int rows_at_once(int tensors) { return NV > 1 || tensors > 2 ? 1 : tensors == 1 ? 4 : 2; }
bool few(const Sizes &n, int G) { return n.rows() < (long long)(NT / G) * MAX_CTAS; }

cudaError_t finish_dw(void *dw, bool w_bf16, const float *ws, int rows, int d, cudaStream_t s) {
    const unsigned blocks = (d + 7) / 8;
    count_launches(1);
    if (w_bf16) return launch_after(sum_dw_kernel<__nv_bfloat16>, dim3(blocks), 1024, 0, s, ws, (__nv_bfloat16 *)dw, rows, d);
    return launch_after(sum_dw_kernel<float>, dim3(blocks), 1024, 0, s, ws, (float *)dw, rows, d);
}

template <typename T, int VEC>
cudaError_t head_fwd(View x, Weight w, void *y, Sizes n, float m, float scale, float eps, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        constexpr int R = rows_at_once<N>(1);
        if (few(n, G)) head_norm_kernel<T, V, N, G, 1><<<grid_for(n, G, 1), NT, 0, s>>>(x, w, (T *)y, n, (unsigned)n.rows(), m, scale, eps);
        else head_norm_kernel<T, V, N, G, R><<<grid_for(n, G, R), NT, 0, s>>>(x, w, (T *)y, n, (unsigned)n.rows(), m, scale, eps);
        count_launches(1);
        return cudaGetLastError();
    });
}
template <typename T, int VEC>
cudaError_t head_bwd(View x, Weight w, const void *dy, void *dx, void *dw, Sizes n, float m, float scale, float eps,
                     float *ws, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        constexpr int R = rows_at_once<N>(2);
        const bool one = few(n, G);
        const unsigned grid = grid_for(n, G, one ? 1 : R);
        if (one) head_norm_bwd_kernel<T, V, N, G, 1><<<grid, NT, 0, s>>>(x, w, (const T *)dy, (T *)dx, dw ? ws : nullptr, n, (unsigned)n.rows(), m, scale, eps);
        else head_norm_bwd_kernel<T, V, N, G, R><<<grid, NT, 0, s>>>(x, w, (const T *)dy, (T *)dx, dw ? ws : nullptr, n, (unsigned)n.rows(), m, scale, eps);
        count_launches(1);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess || !dw ? e : finish_dw(dw, w.bf16, ws, grid, n.d, s);
    });
}
template <typename T, typename TO, int VEC>
cudaError_t gated_fwd(const void *o, View gate, Weight w, View res, void *y, Sizes n, bool silu, float scale, float eps,
                      cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        constexpr int R = rows_at_once<N>(2);
        if (few(n, G)) gated_norm_kernel<T, TO, V, N, G, 1><<<grid_for(n, G, 1), NT, 0, s>>>((const TO *)o, gate, w, res, (T *)y, n, (unsigned)n.rows(), silu, scale, eps);
        else gated_norm_kernel<T, TO, V, N, G, R><<<grid_for(n, G, R), NT, 0, s>>>((const TO *)o, gate, w, res, (T *)y, n, (unsigned)n.rows(), silu, scale, eps);
        count_launches(1);
        return cudaGetLastError();
    });
}
template <typename T, typename TO, int VEC>
cudaError_t gated_bwd(const void *o, View gate, Weight w, const void *dy, void *d_o, void *dgate, void *dw, Sizes n,
                      bool silu, float scale, float eps, float *ws, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        constexpr int R = rows_at_once<N>(3);
        const bool one = few(n, G);
        const unsigned grid = grid_for(n, G, one ? 1 : R);
        auto *kernel = one ? gated_norm_bwd_kernel<T, TO, V, N, G, 1> : gated_norm_bwd_kernel<T, TO, V, N, G, R>;
        kernel<<<grid, NT, 0, s>>>((const TO *)o, gate, w, (const T *)dy, (TO *)d_o, (T *)dgate, dw ? ws : nullptr, n,
                                   (unsigned)n.rows(), silu, scale, eps);
        count_launches(1);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess || !dw ? e : finish_dw(dw, w.bf16, ws, grid, n.d, s);
    });
}

using bf = __nv_bfloat16;

}  // namespace

size_t bwd_workspace_bytes(int d) { return (size_t)MAX_CTAS * d * sizeof(float); }

cudaError_t launch_head_norm(View x, Weight w, void *y, Sizes n, bool l2, float scale, float eps, bool bf16,
                             cudaStream_t s) {
    const float m = l2 ? 1.f : 1.f / n.d;
    const int V = bf16 ? 8 : 4;
    const bool vec = n.d % V == 0 && wide(x.p, 16) && wide(x, V) && wide(y, 16);
    if (bf16) return vec ? head_fwd<bf, 8>(x, w, y, n, m, scale, eps, s) : head_fwd<bf, 1>(x, w, y, n, m, scale, eps, s);
    return vec ? head_fwd<float, 4>(x, w, y, n, m, scale, eps, s) : head_fwd<float, 1>(x, w, y, n, m, scale, eps, s);
}

cudaError_t launch_head_norm_bwd(View x, Weight w, const void *dy, void *dx, void *dw, Sizes n, bool l2, float scale,
                                 float eps, bool bf16, float *ws, cudaStream_t s) {
    const float m = l2 ? 1.f : 1.f / n.d;
    const int V = bf16 ? 8 : 4;
    const bool vec = n.d % V == 0 && wide(x.p, 16) && wide(x, V) && wide(dy, 16) && wide(dx, 16);
    if (bf16)
        return vec ? head_bwd<bf, 8>(x, w, dy, dx, dw, n, m, scale, eps, ws, s) : head_bwd<bf, 1>(x, w, dy, dx, dw, n, m, scale, eps, ws, s);
    return vec ? head_bwd<float, 4>(x, w, dy, dx, dw, n, m, scale, eps, ws, s) : head_bwd<float, 1>(x, w, dy, dx, dw, n, m, scale, eps, ws, s);
}

cudaError_t launch_gated_norm(const void *o, bool o_bf16, View gate, Weight w, View res, void *y, Sizes n, bool silu,
                              float scale, float eps, bool bf16, cudaStream_t s) {
    const int V = bf16 && o_bf16 ? 8 : 4;
    const bool vec = n.d % V == 0 && wide(o, 16) && wide(gate.p, 16) && wide(gate, V) && wide(res.p, 16) && wide(res, V) && wide(y, 16);
    if (bf16 && o_bf16) return vec ? gated_fwd<bf, bf, 8>(o, gate, w, res, y, n, silu, scale, eps, s) : gated_fwd<bf, bf, 1>(o, gate, w, res, y, n, silu, scale, eps, s);
    if (bf16) return vec ? gated_fwd<bf, float, 4>(o, gate, w, res, y, n, silu, scale, eps, s) : gated_fwd<bf, float, 1>(o, gate, w, res, y, n, silu, scale, eps, s);
    if (o_bf16) return vec ? gated_fwd<float, bf, 4>(o, gate, w, res, y, n, silu, scale, eps, s) : gated_fwd<float, bf, 1>(o, gate, w, res, y, n, silu, scale, eps, s);
    return vec ? gated_fwd<float, float, 4>(o, gate, w, res, y, n, silu, scale, eps, s) : gated_fwd<float, float, 1>(o, gate, w, res, y, n, silu, scale, eps, s);
}

cudaError_t launch_gated_norm_bwd(const void *o, bool o_bf16, View gate, Weight w, const void *dy, void *d_o,
                                  void *dgate, void *dw, Sizes n, bool silu, float scale, float eps, bool bf16,
                                  float *ws, cudaStream_t s) {
    const int V = bf16 && o_bf16 ? 8 : 4;
    const bool vec = n.d % V == 0 && wide(o, 16) && wide(gate.p, 16) && wide(gate, V) && wide(dy, 16) && wide(d_o, 16) && wide(dgate, 16);
#define EFLA_GB(T, TO, W) \
    return vec ? gated_bwd<T, TO, W>(o, gate, w, dy, d_o, dgate, dw, n, silu, scale, eps, ws, s) \
               : gated_bwd<T, TO, 1>(o, gate, w, dy, d_o, dgate, dw, n, silu, scale, eps, ws, s)
    if (bf16 && o_bf16) EFLA_GB(bf, bf, 8);
    if (bf16) EFLA_GB(bf, float, 4);
    if (o_bf16) EFLA_GB(float, bf, 4);
    EFLA_GB(float, float, 4);
#undef EFLA_GB
}

}  // namespace norms
}  // namespace efla
