// norms_api.cu -- extern "C" entry points of the per-head norms (include/efla.h).
#include <math.h>
#include <stdint.h>

#include "../../include/efla.h"
#include "norms.h"

namespace {

using efla::norms::Sizes;
using efla::norms::View;
using efla::norms::Weight;

constexpr long long MAX_ROWS = 0x7f000000LL;

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t elem(efla_dtype dt) { return dt == EFLA_BF16 ? 2 : 4; }
bool dtype_ok(efla_dtype d) { return d == EFLA_F32 || d == EFLA_BF16; }
efla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA; }
View view(const void *p, const long long *st) { return {p, st ? st[0] : 0, st ? st[1] : 0, st ? st[2] : 0}; }

// The checks that the four calls share; EFLA_OK with no rows left means there is nothing to do.
efla_status check(int B, int L, int H, int d, efla_dtype dt, efla_dtype w_dt, const void *w, bool option, float scale,
                  float eps) {
    if (!dtype_ok(dt) || (w && !dtype_ok(w_dt))) return EFLA_ERR_DTYPE;
    if (!option || !(eps >= 0.f) || !isfinite(eps) || !isfinite(scale)) return EFLA_ERR_OPTION;
    if (B < 0 || L < 0 || H < 0 || d < 1) return EFLA_ERR_SHAPE;
    if (d > efla::norms::DMAX) return EFLA_ERR_UNSUPPORTED;
    // rows are counted in 32 bits, a turn past the last one
    if ((long long)B * L >= MAX_ROWS || (long long)B * L * H >= MAX_ROWS) return EFLA_ERR_SHAPE;
    if (!aligned(w, w ? elem(w_dt) : 1)) return EFLA_ERR_ALIGN;
    return EFLA_OK;
}

efla_status no_rows(void *dw, efla_dtype w_dt, int d, void *stream) {
    return dw ? from_cuda(cudaMemsetAsync(dw, 0, elem(w_dt) * d, (cudaStream_t)stream)) : EFLA_OK;
}

efla_status check_ws(const void *dw, const void *w, int d, efla_dtype w_dt, const void *ws, size_t bytes) {
    if (!dw) return EFLA_OK;
    if (!w) return EFLA_ERR_NULL;
    if (!ws || bytes < efla_norm_bwd_workspace_size(d)) return EFLA_ERR_WORKSPACE;
    return aligned(dw, elem(w_dt)) && aligned(ws, 16) ? EFLA_OK : EFLA_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t efla_norm_bwd_workspace_size(int d) {
    return d < 1 || d > efla::norms::DMAX ? 0 : efla::norms::bwd_workspace_bytes(d);
}

efla_status efla_head_norm(const void *x, const long long *x_strides, const void *w, efla_dtype w_dt, void *y, int B,
                           int L, int H, int d, efla_dtype dt, efla_norm kind, float scale, float eps, void *stream) {
    const efla_status st = check(B, L, H, d, dt, w_dt, w, kind == EFLA_NORM_L2 || kind == EFLA_NORM_RMS, scale, eps);
    if (st != EFLA_OK) return st;
    if (B == 0 || L == 0 || H == 0) return EFLA_OK;
    if (!x || !x_strides || !y) return EFLA_ERR_NULL;
    if (!aligned(x, elem(dt)) || !aligned(y, elem(dt))) return EFLA_ERR_ALIGN;
    return from_cuda(efla::norms::launch_head_norm(view(x, x_strides), {w, w_dt == EFLA_BF16}, y, {B, L, H, d},
                                                   kind == EFLA_NORM_L2, scale, eps, dt == EFLA_BF16,
                                                   (cudaStream_t)stream));
}

efla_status efla_head_norm_bwd(const void *x, const long long *x_strides, const void *w, efla_dtype w_dt,
                               const void *dy, void *dx, void *dw, int B, int L, int H, int d, efla_dtype dt,
                               efla_norm kind, float scale, float eps, void *workspace, size_t workspace_bytes,
                               void *stream) {
    efla_status st = check(B, L, H, d, dt, w_dt, w, kind == EFLA_NORM_L2 || kind == EFLA_NORM_RMS, scale, eps);
    if (st != EFLA_OK) return st;
    if ((st = check_ws(dw, w, d, w_dt, workspace, workspace_bytes)) != EFLA_OK) return st;
    if (B == 0 || L == 0 || H == 0) return no_rows(dw, w_dt, d, stream);
    if (!x || !x_strides || !dy || !dx) return EFLA_ERR_NULL;
    if (!aligned(x, elem(dt)) || !aligned(dy, elem(dt)) || !aligned(dx, elem(dt))) return EFLA_ERR_ALIGN;
    return from_cuda(efla::norms::launch_head_norm_bwd(view(x, x_strides), {w, w_dt == EFLA_BF16}, dy, dx, dw,
                                                       {B, L, H, d}, kind == EFLA_NORM_L2, scale, eps,
                                                       dt == EFLA_BF16, (float *)workspace, (cudaStream_t)stream));
}

efla_status efla_gated_norm(const void *o, efla_dtype o_dt, const void *gate, const long long *gate_strides,
                            const void *w, efla_dtype w_dt, const void *residual, const long long *residual_strides,
                            void *y, int B, int L, int H, int d, efla_dtype dt, efla_act act, float scale, float eps,
                            void *stream) {
    const efla_status st = check(B, L, H, d, dt, w_dt, w, act == EFLA_ACT_SILU || act == EFLA_ACT_SIGMOID, scale, eps);
    if (st != EFLA_OK) return st;
    if (!dtype_ok(o_dt)) return EFLA_ERR_DTYPE;
    if (B == 0 || L == 0 || H == 0) return EFLA_OK;
    if (!o || !gate || !gate_strides || !y || (residual && !residual_strides)) return EFLA_ERR_NULL;
    if (!aligned(o, elem(o_dt)) || !aligned(gate, elem(dt)) || !aligned(residual, elem(dt)) || !aligned(y, elem(dt)))
        return EFLA_ERR_ALIGN;
    return from_cuda(efla::norms::launch_gated_norm(o, o_dt == EFLA_BF16, view(gate, gate_strides),
                                                    {w, w_dt == EFLA_BF16},
                                                    residual ? view(residual, residual_strides) : View{}, y,
                                                    {B, L, H, d}, act == EFLA_ACT_SILU, scale, eps, dt == EFLA_BF16,
                                                    (cudaStream_t)stream));
}

efla_status efla_gated_norm_bwd(const void *o, efla_dtype o_dt, const void *gate, const long long *gate_strides,
                                const void *w, efla_dtype w_dt, const void *dy, void *d_o, void *dgate, void *dw,
                                int B, int L, int H, int d, efla_dtype dt, efla_act act, float scale, float eps,
                                void *workspace, size_t workspace_bytes, void *stream) {
    efla_status st = check(B, L, H, d, dt, w_dt, w, act == EFLA_ACT_SILU || act == EFLA_ACT_SIGMOID, scale, eps);
    if (st != EFLA_OK) return st;
    if (!dtype_ok(o_dt)) return EFLA_ERR_DTYPE;
    if ((st = check_ws(dw, w, d, w_dt, workspace, workspace_bytes)) != EFLA_OK) return st;
    if (B == 0 || L == 0 || H == 0) return no_rows(dw, w_dt, d, stream);
    if (!o || !gate || !gate_strides || !dy || !d_o || !dgate) return EFLA_ERR_NULL;
    if (!aligned(o, elem(o_dt)) || !aligned(d_o, elem(o_dt)) || !aligned(gate, elem(dt)) || !aligned(dy, elem(dt)) ||
        !aligned(dgate, elem(dt)))
        return EFLA_ERR_ALIGN;
    return from_cuda(efla::norms::launch_gated_norm_bwd(o, o_dt == EFLA_BF16, view(gate, gate_strides),
                                                        {w, w_dt == EFLA_BF16}, dy, d_o, dgate, dw, {B, L, H, d},
                                                        act == EFLA_ACT_SILU, scale, eps, dt == EFLA_BF16,
                                                        (float *)workspace, (cudaStream_t)stream));
}

}  // extern "C"
