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
__device__ __forceinline__ float gate_or_zero(const Gate &g, int bh, int L, int t) {
    return t < L ? gate_at(g, bh, L, t) : 0.f;
}

// A sum of two fp32: hi + lo, lo at most about half an ulp of hi.  A chunk's running sum of log-decays can
// be in the thousands (tokens that forget everything), where fp32 alone would leave nothing of the small
// ones behind it; held like this, differences of two running sums are exact to fp32.  (fp64 does the same at
// 2900 cycles a chunk against 600: its adds are a long dependent chain.)
struct Sum {
    float hi, lo;
};
// Knuth's error-free sum: a + b = s + e.
__device__ __forceinline__ Sum two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Sum operator+(const Sum &a, const Sum &b) {
    const Sum s = two_sum(a.hi, b.hi);
    const float lo = s.lo + (a.lo + b.lo), hi = s.hi + lo;
    return {hi, lo - (hi - s.hi)};
}
__device__ __forceinline__ Sum operator-(const Sum &a, const Sum &b) { return a + Sum{-b.hi, -b.lo}; }

// Running sums of a chunk's log-decays in units of log 2.  One warp; lane holds tokens 2 lane and
// 2 lane + 1, l0 and l1 their log-decays (0 past the sequence's end).
struct PairSum {
    Sum c0, c1;
};
__device__ __forceinline__ Sum to_log2(float l) {  // l / ln 2
    const float p = l * 1.44269502f;
    return {p, fmaf(l, 1.92596299e-8f, fmaf(l, 1.44269502f, -p))};
}
__device__ __forceinline__ PairSum chunk_sums(float l0, float l1, int lane) {
    const Sum x0 = to_log2(l0), x1 = to_log2(l1);
    Sum s = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y = {__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
        const Sum t = s + y;
        if (lane >= o) s = t;
    }
    Sum before = {__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    return {before + x0, s};
}
__device__ __forceinline__ Sum last_sum(const PairSum &c) {
    return {__shfl_sync(0xffffffffu, c.c1.hi, 31), __shfl_sync(0xffffffffu, c.c1.lo, 31)};
}
// 2^x: |lo| is far below 1, so 2^lo = 1 + lo ln 2 to fp32.
__device__ __forceinline__ float exp2_sum(const Sum &x) {
    const float e = exp2f(x.hi);
    return fmaf(e, x.lo * 0.693147181f, e);
}

}  // namespace decay
}  // namespace efla
