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
constexpr int MAX_CTAS = 148 * 8;  // of the kernels that sum a weight gradient

template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> { using V = uint4; };
template <> struct Piece<float, 4> { using V = uint4; };
template <> struct Piece<__nv_bfloat16, 4> { using V = uint2; };
template <> struct Piece<float, 1> { using V = uint32_t; };
template <> struct Piece<__nv_bfloat16, 1> { using V = uint16_t; };

template <typename T, int VEC>
__device__ __forceinline__ void ld(float (&f)[VEC], const T *p) {
    const typename Piece<T, VEC>::V u = *reinterpret_cast<const typename Piece<T, VEC>::V *>(p);
    const T *h = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32(h[i]);
}
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

// Where row r = (b L + t) H + h lies: in the view's strides, and in the kernels' layout [B,H,L,d].
struct Row {
    int b, t, h;
    __device__ __forceinline__ Row(long long r, const Sizes &n) {
        const long long bt = r / n.H;
        h = (int)(r - bt * n.H);
        b = (int)(bt / n.L);
        t = (int)(bt - (long long)b * n.L);
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

// dw[i] = sum of the CTAs' shares, in their order: 32 columns a CTA, 32 rows of threads.
template <typename TW>
__global__ void __launch_bounds__(1024) sum_dw_kernel(const float *__restrict__ part, TW *__restrict__ dw, int rows, int d) {
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, i = blockIdx.x * 32 + c;
    float x = 0.f;
    if (i < d)
        for (int r = g; r < rows; r += 32) x += part[(size_t)r * d + i];
    red[g][c] = x;
    __syncthreads();
    if (g == 0 && i < d) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) s += red[r][c];
        dw[i] = from_f32<TW>(s);
    }
}

// ------------------------------------------------------------------ head norm
template <typename T, int VEC, int NV, int G>
__global__ void __launch_bounds__(NT)
    head_norm_kernel(const View x, const Weight w, T *__restrict__ y, const Sizes n, float m, float scale, float eps) {
    const int lane = threadIdx.x & 31, gl = lane % G;
    constexpr int RPC = NT / G;
    const long long rows = (long long)n.B * n.L * n.H, step = (long long)gridDim.x * RPC;
    float wv[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = (j * G + gl) * VEC + e;
            wv[j][e] = i < n.d ? scale * weight_at(w, i) : 0.f;
        }
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < rows; r0 += step) {
        const long long r = r0 + threadIdx.x / G;
        const bool on = r < rows;
        const Row row(on ? r : 0, n);
        const T *px = static_cast<const T *>(x.p) + row.at(x);
        float f[NV][VEC], sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
            if (on && i < n.d) ld<T, VEC>(f[j], px + i);
            else
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[j][e] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(f[j][e], f[j][e], sum);
        }
        const float rs = rsqrtf(fmaf(m, group_sum<G>(sum), eps));
        T *py = y + row.heads(n);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[j][e] = f[j][e] * rs * wv[j][e];
            if (on && i < n.d) st<T, VEC>(py + i, f[j]);
        }
    }
}

template <typename T, int VEC, int NV, int G>
__global__ void __launch_bounds__(NT)
    head_norm_bwd_kernel(const View x, const Weight w, const T *__restrict__ dy, T *__restrict__ dx,
                         float *__restrict__ part, const Sizes n, float m, float scale, float eps) {
    const int lane = threadIdx.x & 31, gl = lane % G;
    constexpr int RPC = NT / G;
    const long long rows = (long long)n.B * n.L * n.H, step = (long long)gridDim.x * RPC;
    float wv[NV][VEC], acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = (j * G + gl) * VEC + e;
            wv[j][e] = i < n.d ? scale * weight_at(w, i) : 0.f;
            acc[j][e] = 0.f;
        }
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < rows; r0 += step) {
        const long long r = r0 + threadIdx.x / G;
        const bool on = r < rows;
        const Row row(on ? r : 0, n);
        const T *px = static_cast<const T *>(x.p) + row.at(x);
        const T *pd = dy + row.heads(n);
        float f[NV][VEC], gd[NV][VEC], sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
            if (on && i < n.d) {
                ld<T, VEC>(f[j], px + i);
                ld<T, VEC>(gd[j], pd + i);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[j][e] = gd[j][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(f[j][e], f[j][e], sum);
        }
        const float rs = rsqrtf(fmaf(m, group_sum<G>(sum), eps));
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                f[j][e] *= rs;  // n
                if (on) acc[j][e] = fmaf(gd[j][e], f[j][e], acc[j][e]);
                gd[j][e] *= wv[j][e];  // dn
                dot = fmaf(gd[j][e], f[j][e], dot);
            }
        dot = m * group_sum<G>(dot);
        T *po = dx + (size_t)(on ? r : 0) * n.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[j][e] = rs * fmaf(-dot, f[j][e], gd[j][e]);
            if (on && i < n.d) st<T, VEC>(po + i, f[j]);
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] *= scale;
        store_dw<VEC, NV, G>(acc, part, n.d, lane);
    }
}

// ------------------------------------------------------------------ gated norm
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <typename T, typename TO, int VEC, int NV, int G>
__global__ void __launch_bounds__(NT)
    gated_norm_kernel(const TO *__restrict__ o, const View gate, const Weight w, const View res, T *__restrict__ y,
                      const Sizes n, bool silu, float scale, float eps) {
    const int lane = threadIdx.x & 31, gl = lane % G;
    constexpr int RPC = NT / G;
    const long long rows = (long long)n.B * n.L * n.H, step = (long long)gridDim.x * RPC;
    const float m = 1.f / n.d;
    float wv[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = (j * G + gl) * VEC + e;
            wv[j][e] = i < n.d ? scale * weight_at(w, i) : 0.f;
        }
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < rows; r0 += step) {
        const long long r = r0 + threadIdx.x / G;
        const bool on = r < rows;
        const Row row(on ? r : 0, n);
        const TO *po = o + row.heads(n);
        const T *pg = static_cast<const T *>(gate.p) + row.at(gate);
        const T *pr = res.p ? static_cast<const T *>(res.p) + row.at(res) : nullptr;
        float f[NV][VEC], gv[NV][VEC], rv[NV][VEC], sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[j][e] = gv[j][e] = rv[j][e] = 0.f;
            if (on && i < n.d) {
                ld<TO, VEC>(f[j], po + i);
                ld<T, VEC>(gv[j], pg + i);
                if (pr) ld<T, VEC>(rv[j], pr + i);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(f[j][e], f[j][e], sum);
        }
        const float rs = rsqrtf(fmaf(m, group_sum<G>(sum), eps));
        T *py = y + (size_t)(on ? r : 0) * n.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float sg = sigmoid(gv[j][e]), a = silu ? gv[j][e] * sg : sg;
                f[j][e] = fmaf(f[j][e] * rs * wv[j][e], a, rv[j][e]);
            }
            if (on && i < n.d) st<T, VEC>(py + i, f[j]);
        }
    }
}

template <typename T, typename TO, int VEC, int NV, int G>
__global__ void __launch_bounds__(NT)
    gated_norm_bwd_kernel(const TO *__restrict__ o, const View gate, const Weight w, const T *__restrict__ dy,
                          TO *__restrict__ d_o, T *__restrict__ dgate, float *__restrict__ part, const Sizes n,
                          bool silu, float scale, float eps) {
    const int lane = threadIdx.x & 31, gl = lane % G;
    constexpr int RPC = NT / G;
    const long long rows = (long long)n.B * n.L * n.H, step = (long long)gridDim.x * RPC;
    const float m = 1.f / n.d;
    float wv[NV][VEC], acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = (j * G + gl) * VEC + e;
            wv[j][e] = i < n.d ? scale * weight_at(w, i) : 0.f;
            acc[j][e] = 0.f;
        }
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < rows; r0 += step) {
        const long long r = r0 + threadIdx.x / G;
        const bool on = r < rows;
        const Row row(on ? r : 0, n);
        const size_t at_o = row.heads(n), at_y = (size_t)(on ? r : 0) * n.d;
        const T *pg = static_cast<const T *>(gate.p) + row.at(gate);
        float f[NV][VEC], gv[NV][VEC], gd[NV][VEC], sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[j][e] = gv[j][e] = gd[j][e] = 0.f;
            if (on && i < n.d) {
                ld<TO, VEC>(f[j], o + at_o + i);
                ld<T, VEC>(gv[j], pg + i);
                ld<T, VEC>(gd[j], dy + at_y + i);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(f[j][e], f[j][e], sum);
        }
        const float rs = rsqrtf(fmaf(m, group_sum<G>(sum), eps));
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float x = gv[j][e], sg = sigmoid(x);
                const float a = silu ? x * sg : sg, da = silu ? sg * fmaf(x, 1.f - sg, 1.f) : sg * (1.f - sg);
                const float nn = f[j][e] * rs, dyv = gd[j][e];
                if (on) acc[j][e] = fmaf(dyv * a, nn, acc[j][e]);
                const float dyw = dyv * wv[j][e];
                gv[j][e] = dyw * nn * da;  // dgate
                gd[j][e] = dyw * a;        // dn
                f[j][e] = nn;
                dot = fmaf(gd[j][e], nn, dot);
            }
        dot = m * group_sum<G>(dot);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * G + gl) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[j][e] = rs * fmaf(-dot, f[j][e], gd[j][e]);
            if (on && i < n.d) {
                st<TO, VEC>(d_o + at_o + i, f[j]);
                st<T, VEC>(dgate + at_y + i, gv[j]);
            }
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] *= scale;
        store_dw<VEC, NV, G>(acc, part, n.d, lane);
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

unsigned grid_for(const Sizes &n, int G, int most) {
    const long long rows = (long long)n.B * n.L * n.H, rpc = NT / G, want = (rows + rpc - 1) / rpc;
    return (unsigned)(want < most ? want : most);
}

cudaError_t finish_dw(void *dw, bool w_bf16, const float *ws, int rows, int d, cudaStream_t s) {
    const unsigned blocks = (d + 31) / 32;
    if (w_bf16) sum_dw_kernel<<<blocks, 1024, 0, s>>>(ws, (__nv_bfloat16 *)dw, rows, d);
    else sum_dw_kernel<<<blocks, 1024, 0, s>>>(ws, (float *)dw, rows, d);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t head_fwd(View x, Weight w, void *y, Sizes n, float m, float scale, float eps, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        head_norm_kernel<T, V, N, G><<<grid_for(n, G, 1 << 30), NT, 0, s>>>(x, w, (T *)y, n, m, scale, eps);
        count_launches(1);
        return cudaGetLastError();
    });
}
template <typename T, int VEC>
cudaError_t head_bwd(View x, Weight w, const void *dy, void *dx, void *dw, Sizes n, float m, float scale, float eps,
                     float *ws, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        const unsigned grid = grid_for(n, G, MAX_CTAS);
        head_norm_bwd_kernel<T, V, N, G><<<grid, NT, 0, s>>>(x, w, (const T *)dy, (T *)dx, dw ? ws : nullptr, n, m, scale, eps);
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
        gated_norm_kernel<T, TO, V, N, G><<<grid_for(n, G, 1 << 30), NT, 0, s>>>((const TO *)o, gate, w, res, (T *)y, n, silu, scale, eps);
        count_launches(1);
        return cudaGetLastError();
    });
}
template <typename T, typename TO, int VEC>
cudaError_t gated_bwd(const void *o, View gate, Weight w, const void *dy, void *d_o, void *dgate, void *dw, Sizes n,
                      bool silu, float scale, float eps, float *ws, cudaStream_t s) {
    return by_width<VEC>(n.d, [&](auto vec, auto nv, auto g) {
        constexpr int V = decltype(vec)::value, N = decltype(nv)::value, G = decltype(g)::value;
        const unsigned grid = grid_for(n, G, MAX_CTAS);
        gated_norm_bwd_kernel<T, TO, V, N, G><<<grid, NT, 0, s>>>((const TO *)o, gate, w, (const T *)dy, (TO *)d_o,
                                                                  (T *)dgate, dw ? ws : nullptr, n, silu, scale, eps);
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
