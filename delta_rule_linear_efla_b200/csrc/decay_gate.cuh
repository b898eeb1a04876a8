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
    return l < L_MIN ? L_MIN : l > -L_MIN ? -L_MIN : l;  // NaN stays NaN; e^200 is infinite in fp32
}
__device__ __forceinline__ float gate_or_zero(const Gate &g, int bh, int L, int t) {
    return t < L ? gate_at(g, bh, L, t) : 0.f;
}

// A log-decay in units of log 2 / 2^32, as an integer, for the fp32 walks: sums are exact (64 tokens of -200
// take 47 bits), and a difference of two sums keeps all of its bits where the sums themselves are in the
// thousands (tokens that forget everything before tokens that forget little).
using Fixed = long long;
constexpr float FIXED_ONE = 4294967296.f;
constexpr Fixed FIXED_MIN = -(1LL << 60);  // a sum over many chunks stops here: 2^-(2^28) is 0
__device__ __forceinline__ Fixed to_fixed(float l) {
    // l / ln 2 in two parts, so that its rounding (2^-24 relative) is not what the sums keep
    const float p = l * 1.44269502f;
    const float e = fmaf(l, 1.92596299e-8f, fmaf(l, 1.44269502f, -p));
    return __float2ll_rn(p * FIXED_ONE) + __float2ll_rn(e * FIXED_ONE);
}
__device__ __forceinline__ float exp2_fixed(Fixed x) { return exp2f(__ll2float_rn(x) * (1.f / FIXED_ONE)); }

// Running sums of a chunk's log-decays.  One warp; lane holds tokens 2 lane and 2 lane + 1, l0 and l1 their
// log-decays (0 past the sequence's end).  bad: the first token of the chunk whose log-decay is not a number
// (64: none); from it on, every sum is to be taken as such.
struct PairSum {
    Fixed c0, c1, cC;
    int bad;
};
__device__ __forceinline__ PairSum chunk_sums(float l0, float l1, int lane) {
    const Fixed x0 = to_fixed(l0), x1 = to_fixed(l1);
    Fixed s = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Fixed y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    const unsigned n0 = __ballot_sync(0xffffffffu, l0 != l0), n1 = __ballot_sync(0xffffffffu, l1 != l1);
    const int b0 = n0 ? 2 * (__ffs(n0) - 1) : C, b1 = n1 ? 2 * __ffs(n1) - 1 : C;
    return {s - x1, s, __shfl_sync(0xffffffffu, s, 31), min(b0, b1)};
}
// The factors that a sum over tokens [from, to] gives: not a number where it takes a bad token in.
__device__ __forceinline__ float if_good(float x, bool good) { return good ? x : __int_as_float(0x7fffffff); }

}  // namespace decay
}  // namespace efla
