// decay_step.cu -- one decode token of linear attention with a decay for each head:
//   S <- e^l S + k v^T in place, then o = S^T q.
//
// HBM-bound: the fp32 state is read once and written once (q, k, v and o are negligible).  State
// columns do not depend on one another, so a CTA takes one head and a block of its columns, each
// thread a few rows of VEC columns in registers; the rows' shares of o are added through shared
// memory in a fixed order.
#include "decay_gate.cuh"
#include "launchers.h"

namespace efla {
namespace decay {

namespace {

constexpr int NT = 256, DMAX = 256;

template <int VEC> struct Cols;
template <> struct Cols<4> { using V = float4; };
template <> struct Cols<1> { using V = float; };
__device__ __forceinline__ void step_cols(float4 &s, float e, float k, const float4 &v, float q, float4 &o) {
    s.x = fmaf(k, v.x, e * s.x); s.y = fmaf(k, v.y, e * s.y);
    s.z = fmaf(k, v.z, e * s.z); s.w = fmaf(k, v.w, e * s.w);
    o.x = fmaf(q, s.x, o.x); o.y = fmaf(q, s.y, o.y); o.z = fmaf(q, s.z, o.z); o.w = fmaf(q, s.w, o.w);
}
__device__ __forceinline__ void step_cols(float &s, float e, float k, float v, float q, float &o) {
    s = fmaf(k, v, e * s);
    o = fmaf(q, s, o);
}

// CB columns a CTA; VEC columns a thread; ROWS: rows a thread keeps in flight.
template <typename T, typename TO, int VEC, int CB>
__global__ void __launch_bounds__(NT)
    step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const Gate g,
                float *__restrict__ S, TO *__restrict__ o, int BH, int dk, int dv) {
    using V = typename Cols<VEC>::V;
    constexpr int TPR = CB / VEC, RG = NT / TPR, ROWS = 4;
    __shared__ float ks[DMAX], qs[DMAX];
    __shared__ __align__(16) float vs[CB];
    __shared__ __align__(16) float red[RG * CB];
    const int bh = blockIdx.x, j0 = blockIdx.y * CB, tid = threadIdx.x;
    const int cg = tid % TPR, rg = tid / TPR, col = j0 + cg * VEC;
    float *Sh = S + (size_t)bh * dk * dv + col;
    const bool on = col < dv;
    // the state's loads do not wait for the vectors
    V st[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + i * RG;
        if (on && r < dk) st[i] = *reinterpret_cast<const V *>(Sh + (size_t)r * dv);
    }
    for (int i = tid; i < dk; i += NT) {
        ks[i] = to_f32(k[(size_t)bh * dk + i]);
        qs[i] = to_f32(q[(size_t)bh * dk + i]);
    }
    for (int i = tid; i < CB; i += NT) vs[i] = j0 + i < dv ? to_f32(v[(size_t)bh * dv + j0 + i]) : 0.f;
    const float e = expf(gate_at(g, bh, 1, 0));
    __syncthreads();
    V acc{};
    const V vv = *reinterpret_cast<const V *>(vs + cg * VEC);
    if (on) {
        for (int r0 = rg; r0 < dk; r0 += ROWS * RG) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int r = r0 + i * RG;
                if (r < dk) {
                    step_cols(st[i], e, ks[r], vv, qs[r], acc);
                    *reinterpret_cast<V *>(Sh + (size_t)r * dv) = st[i];
                }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int r = r0 + (ROWS + i) * RG;
                if (r < dk) st[i] = *reinterpret_cast<const V *>(Sh + (size_t)r * dv);
            }
        }
    }
    *reinterpret_cast<V *>(red + rg * CB + cg * VEC) = acc;
    __syncthreads();
    for (int c = tid; c < CB; c += NT) {
        float x = 0.f;
#pragma unroll 8
        for (int i = 0; i < RG; ++i) x += red[i * CB + c];
        if (j0 + c < dv) o[(size_t)bh * dv + j0 + c] = from_f32<TO>(x);
    }
}

template <typename T, typename TO>
void launch_t(const void *q, const void *k, const void *v, Gate g, float *S, void *o, int BH, int dk, int dv,
              cudaStream_t s) {
    // 64 columns a CTA: 24.7 us for 1024 heads of 128 x 128 (5.5 TB/s), against 26.7 with 32 and 26.8 with 128
    if (dv % 4 == 0 && dv > 32)  // S is 16-byte aligned: every row is
        step_kernel<T, TO, 4, 64><<<dim3(BH, (dv + 63) / 64), NT, 0, s>>>((const T *)q, (const T *)k, (const T *)v, g,
                                                                          S, (TO *)o, BH, dk, dv);
    else if (dv % 4 == 0)
        step_kernel<T, TO, 4, 32><<<dim3(BH, (dv + 31) / 32), NT, 0, s>>>((const T *)q, (const T *)k, (const T *)v, g,
                                                                          S, (TO *)o, BH, dk, dv);
    else
        step_kernel<T, TO, 1, 32><<<dim3(BH, (dv + 31) / 32), NT, 0, s>>>((const T *)q, (const T *)k, (const T *)v, g,
                                                                          S, (TO *)o, BH, dk, dv);
}

}  // namespace

cudaError_t launch_step(const void *q, const void *k, const void *v, Gate g, float *S, void *o, int BH, int dk,
                        int dv, bool in_bf16, bool o_bf16, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (in_bf16) {
        if (o_bf16) launch_t<bf, bf>(q, k, v, g, S, o, BH, dk, dv, s);
        else launch_t<bf, float>(q, k, v, g, S, o, BH, dk, dv, s);
    } else {
        if (o_bf16) launch_t<float, bf>(q, k, v, g, S, o, BH, dk, dv, s);
        else launch_t<float, float>(q, k, v, g, S, o, BH, dk, dv, s);
    }
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace decay
}  // namespace efla
