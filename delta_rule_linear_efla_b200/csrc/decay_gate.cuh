// decay_gate.cuh -- log-decays of a chunk and the weights made from them (device side).
#pragma once

#include "common.cuh"
#include "decay.h"

namespace efla {
namespace decay {

__device__ __forceinline__ float gate_at(const Gate &g, int bh, int L, int t) {
    float l;
    if (g.per_head) l = static_cast<const float *>(g.p)[bh % g.H];
    else if (g.bf16) l = __bfloat162float(static_cast<const __nv_bfloat16 *>(g.p)[(size_t)bh * L + t]);
    else l = static_cast<const float *>(g.p)[(size_t)bh * L + t];
    return l < L_MIN ? L_MIN : l;  // NaN stays NaN
}

// Running sums of a chunk's log-decays.  A sum of 64 of them can be in the thousands (tokens that
// forget everything), where fp32 would leave nothing of the small ones behind it, so they are added
// in fp64 and kept as hi + lo, two fp32; differences of two sums are exact to fp32 that way.
// One warp; lane holds tokens 2 lane and 2 lane + 1 (0 past the sequence's end).
struct PairSum {
    double c0, c1;
};
__device__ __forceinline__ PairSum chunk_sums(const Gate &g, int bh, int L, int t0, int lane) {
    const int t = t0 + 2 * lane;
    const double x0 = t < L ? (double)gate_at(g, bh, L, t) : 0.0;
    const double x1 = t + 1 < L ? (double)gate_at(g, bh, L, t + 1) : 0.0;
    double s = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    return {s - x1, s};
}
// e^x for a sum held in fp64: |lo| is at most half an ulp of hi, so e^lo = 1 + lo to fp32.
__device__ __forceinline__ float exp_sum(double x) {
    const float hi = (float)x, lo = (float)(x - (double)hi);
    const float e = expf(hi);
    return fmaf(e, lo, e);
}

}  // namespace decay
}  // namespace efla
