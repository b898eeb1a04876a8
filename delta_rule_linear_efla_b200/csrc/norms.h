// norms.h -- the per-head norms before and after the attention (internal to the library; the public
// ABI is include/efla.h).
//
//   head norm:   y[b,h,t,:] = scale w o x[b,t,h,:] r,          r = (m sum x^2 + eps)^(-1/2), m = 1 (l2) or 1/d (rms)
//   gated norm:  y[b,t,h,:] = res[b,t,h,:] + scale act(gate[b,t,h,:]) o w o n,  n = o[b,h,t,:] r (rms)
//
// and with dn the gradient of n: dx = r (dn - m n (dn . n)).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace efla {
namespace norms {

// A [B,L,H,d] tensor whose last dimension is dense; strides in elements.
struct View {
    const void *p;
    long long sb, sl, sh;
};
// Division by a number below 2^31 as a multiplication (Granlund and Montgomery): n / d for n < 2^31.
struct Div {
    unsigned mul, shift, d;
    Div() = default;
    explicit Div(unsigned dd) : d(dd) {
        shift = 0;
        while ((1ull << shift) < d) ++shift;
        mul = (unsigned)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
};
struct Sizes {
    int B, L, H, d;
    Div byH, byL;
    Sizes(int b, int l, int h, int dd) : B(b), L(l), H(h), d(dd), byH(h), byL(l) {}
    long long rows() const { return (long long)B * L * H; }
};
struct Weight {
    const void *p;  // [d], or null for ones
    bool bf16;
};

constexpr int DMAX = 256;
size_t bwd_workspace_bytes(int d);  // the weight gradient's shares

cudaError_t launch_head_norm(View x, Weight w, void *y, Sizes n, bool l2, float scale, float eps, bool bf16,
                             cudaStream_t s);
cudaError_t launch_head_norm_bwd(View x, Weight w, const void *dy, void *dx, void *dw, Sizes n, bool l2, float scale,
                                 float eps, bool bf16, float *ws, cudaStream_t s);
cudaError_t launch_gated_norm(const void *o, bool o_bf16, View gate, Weight w, View res, void *y, Sizes n, bool silu,
                              float scale, float eps, bool bf16, cudaStream_t s);
cudaError_t launch_gated_norm_bwd(const void *o, bool o_bf16, View gate, Weight w, const void *dy, void *d_o,
                                  void *dgate, void *dw, Sizes n, bool silu, float scale, float eps, bool bf16,
                                  float *ws, cudaStream_t s);

}  // namespace norms
}  // namespace efla
