// decay_api.cu -- extern "C" entry points of linear attention with a decay for each head
// (include/efla.h): argument checks, workspace layout and the choice of kernels.
#include <stdint.h>

#include "../../include/efla.h"
#include "decay.h"
#include "launchers.h"

namespace {

using efla::decay::Gate;
using efla::decay::Segments;
using efla::decay::Shares;
using efla::decay::Walk;
using efla::decay::Walks;

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t elem(efla_dtype dt) { return dt == EFLA_BF16 ? 2 : 4; }
bool dtype_ok(efla_dtype d) { return d == EFLA_F32 || d == EFLA_BF16; }
bool form_ok(efla_decay_form f) { return f == EFLA_DECAY_TOKEN || f == EFLA_DECAY_HEAD; }
efla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA; }
size_t gate_elem(efla_decay_form f, efla_dtype dt) { return f == EFLA_DECAY_HEAD ? 4 : elem(dt); }

constexpr long long MAX_HEADS = 1 << 24;  // B * H: grids stay below 2^31 blocks

bool sizes_ok(int B, int H, long long L, int dk, int dv) {
    return B >= 1 && H >= 1 && L >= 0 && dk >= 1 && dv >= 1 && (long long)B * H <= MAX_HEADS && L <= 0x7fffff00LL &&
           (long long)B * H * L <= (1LL << 40);
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// A bump allocator over the caller's workspace; with a null base it only counts.
struct Arena {
    char *base;
    size_t used = 0;
    float *floats(size_t n) {
        float *p = base ? reinterpret_cast<float *>(base + used) : nullptr;
        used += up(n * sizeof(float));
        return p;
    }
};

int blocks_of(int b) { return (b + efla::decay::SIMT_BT - 1) / efla::decay::SIMT_BT; }

// How CUDA-core walks are cut, and their stretches' contributions.
Segments plan_segments(const Walks &ws, int BH, int L, Arena &ar) {
    int blocks[efla::decay::MAX_WALKS];
    for (int i = 0; i < ws.n; ++i) blocks[i] = blocks_of(ws.w[i].b);
    Segments sg = efla::decay::simt_segments(BH, L, blocks, ws.n);
    if (sg.n > 1) {
        for (int i = 0; i < ws.n; ++i) sg.u[i] = ar.floats((size_t)BH * (sg.n - 1) * ws.w[i].a * ws.w[i].b);
        sg.e = ar.floats((size_t)2 * BH * (sg.n - 1));
    }
    return sg;
}

// The same of tensor-core walks of the same head sizes.
Shares plan_shares(const Walks &ws, int BH, int L, Arena &ar) {
    Shares sh = efla::decay::tc_shares(BH, L, ws.n);
    if (const int n = sh.stretches()) {
        sh.u = ar.floats((size_t)n * ws.w[0].a * ws.w[0].b);
        sh.e = ar.floats(n);
    }
    return sh;
}

struct FwdPlan {
    Walks ws{};
    Segments sg{};
    Shares sh{};
    float *S0 = nullptr;  // a copy of S0 where S_final replaces it: every stretch of a cut walk starts from it
    size_t bytes = 0;
    FwdPlan(int BH, int L, int dk, int dv, bool tc, void *base) {
        Arena ar{static_cast<char *>(base)};
        ws.n = 1;
        ws.w[0].a = dk;
        ws.w[0].b = dv;
        if (tc) sh = plan_shares(ws, BH, L, ar);
        else sg = plan_segments(ws, BH, L, ar);
        if (tc ? sh.cut : sg.n > 1) S0 = ar.floats((size_t)BH * dk * dv);
        bytes = ar.used;
    }
};

struct BwdPlan {
    Walks ws{};              // dq, dk, dv
    Walks part[2]{};         // tensor-core launches: those of the same head sizes together
    int parts = 0;
    Segments sg{};
    Shares sh[2]{};
    float *S_end = nullptr, *dotq = nullptr, *dotk = nullptr;
    int planes = 1;
    size_t bytes = 0;
    BwdPlan(int BH, int L, int dk, int dv, bool tc, void *base) {
        Arena ar{static_cast<char *>(base)};
        ws.n = 3;
        ws.w[0].a = dv; ws.w[0].b = dk;
        ws.w[1].a = dv; ws.w[1].b = dk; ws.w[1].rev = 1;
        ws.w[2].a = dk; ws.w[2].b = dv; ws.w[2].rev = 1;
        planes = tc ? efla::decay::DOT_PLANES : blocks_of(dk);
        dotq = ar.floats((size_t)planes * BH * L);
        dotk = ar.floats((size_t)planes * BH * L);
        S_end = ar.floats((size_t)BH * dk * dv);
        if (!tc) {
            sg = plan_segments(ws, BH, L, ar);
        } else {
            parts = dk == dv ? 1 : 2;
            split();
            for (int i = 0; i < parts; ++i) sh[i] = plan_shares(part[i], BH, L, ar);
        }
        bytes = ar.used;
    }
    // The launches' walks, from ws as it is now.
    void split() {
        part[0] = part[1] = Walks{};
        for (int i = 0; i < 3; ++i) {
            Walks &p = part[parts == 2 && i == 2 ? 1 : 0];
            p.w[p.n++] = ws.w[i];
        }
    }
};

// The workspace of either path: which one runs also depends on the pointers' alignment.
template <typename Plan>
size_t plan_bytes(int BH, int L, int dk, int dv, bool bf16) {
    const size_t n = Plan(BH, L, dk, dv, false, nullptr).bytes;
    if (!efla::decay::tc_sizes(dk, dv, bf16)) return n;
    const size_t t = Plan(BH, L, dk, dv, true, nullptr).bytes;
    return n > t ? n : t;
}

}  // namespace

extern "C" {

size_t efla_decay_chunk_fwd_workspace_size(int B, int H, int L, int dk, int dv, efla_dtype dt) {
    if (!dtype_ok(dt) || !sizes_ok(B, H, L, dk, dv) || L == 0 || dk > 128 || dv > 128) return 0;
    return plan_bytes<FwdPlan>(B * H, L, dk, dv, dt == EFLA_BF16);
}

efla_status efla_decay_chunk_fwd(const void *q, const void *k, const void *v, const void *log_g,
                                 efla_decay_form form, const float *S0, void *o, float *S_final, int B, int H, int L,
                                 int dk, int dv, efla_dtype dt, efla_dtype o_dt, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dt) || !dtype_ok(o_dt)) return EFLA_ERR_DTYPE;
    if (!form_ok(form)) return EFLA_ERR_OPTION;
    if (!sizes_ok(B, H, L, dk, dv)) return EFLA_ERR_SHAPE;
    if (dk > 128 || dv > 128) return EFLA_ERR_UNSUPPORTED;
    if (L > 0 && (!q || !k || !v || !log_g || !o)) return EFLA_ERR_NULL;
    if (!aligned(q, elem(dt)) || !aligned(k, elem(dt)) || !aligned(v, elem(dt)) || !aligned(o, elem(o_dt)) ||
        !aligned(log_g, gate_elem(form, dt)) || !aligned(S0, 4) || !aligned(S_final, 4) || !aligned(workspace, 16))
        return EFLA_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const int BH = B * H;
    const size_t state = (size_t)BH * dk * dv * sizeof(float);
    if (L == 0) {
        if (!S_final || S0 == S_final) return EFLA_OK;
        return from_cuda(S0 ? cudaMemcpyAsync(S_final, S0, state, cudaMemcpyDeviceToDevice, s)
                            : cudaMemsetAsync(S_final, 0, state, s));
    }
    const size_t need = efla_decay_chunk_fwd_workspace_size(B, H, L, dk, dv, dt);
    if (need > 0 && (!workspace || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
    const bool tc = efla::decay::tc_sizes(dk, dv, dt == EFLA_BF16) && aligned(q, 16) && aligned(k, 16) && aligned(v, 16);
    FwdPlan p(BH, L, dk, dv, tc, workspace);
    Walk &w = p.ws.w[0];
    w.x = q; w.y = k; w.z = v;
    w.s0 = S0;
    if (S0 && S0 == S_final && p.S0) {
        const cudaError_t e = cudaMemcpyAsync(p.S0, S0, state, cudaMemcpyDeviceToDevice, s);
        if (e != cudaSuccess) return EFLA_ERR_CUDA;
        w.s0 = p.S0;
    }
    w.out = o;
    w.s_end = S_final;
    const Gate g{log_g, form == EFLA_DECAY_HEAD, dt == EFLA_BF16, H};
    if (tc) return from_cuda(efla::decay::launch_walks_tc(p.ws, g, BH, L, p.sh, o_dt == EFLA_BF16, false, s));
    return from_cuda(efla::decay::launch_walks_simt(p.ws, g, BH, L, p.sg, dt == EFLA_BF16,
                                                    o_dt == EFLA_BF16, s));
}

size_t efla_decay_bwd_workspace_size(int B, int H, int L, int dk, int dv, efla_dtype dt) {
    if (!dtype_ok(dt) || !sizes_ok(B, H, L, dk, dv) || L == 0 || dk > 128 || dv > 128) return 0;
    return plan_bytes<BwdPlan>(B * H, L, dk, dv, dt == EFLA_BF16);
}

efla_status efla_decay_bwd(const void *q, const void *k, const void *v, const void *log_g, efla_decay_form form,
                           const float *S0, const void *dO, const float *dS_final, void *dq, void *dkey, void *dval,
                           void *dlog_g, float *dS0, int B, int H, int L, int dk, int dv, efla_dtype dt,
                           void *workspace, size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dt)) return EFLA_ERR_DTYPE;
    if (!form_ok(form) || (form == EFLA_DECAY_HEAD && dlog_g)) return EFLA_ERR_OPTION;
    if (!sizes_ok(B, H, L, dk, dv)) return EFLA_ERR_SHAPE;
    if (dk > 128 || dv > 128) return EFLA_ERR_UNSUPPORTED;
    if (L > 0 && (!q || !k || !v || !log_g || !dO || !dq || !dkey || !dval)) return EFLA_ERR_NULL;
    const void *in[] = {q, k, v, dO, dq, dkey, dval, dlog_g};
    for (const void *p : in)
        if (!aligned(p, elem(dt))) return EFLA_ERR_ALIGN;
    if (!aligned(log_g, gate_elem(form, dt)) || !aligned(S0, 4) || !aligned(dS_final, 4) || !aligned(dS0, 4) ||
        !aligned(workspace, 16))
        return EFLA_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const int BH = B * H;
    const size_t state = (size_t)BH * dk * dv * sizeof(float);
    if (L == 0) {
        if (!dS0) return EFLA_OK;
        return from_cuda(dS_final ? cudaMemcpyAsync(dS0, dS_final, state, cudaMemcpyDeviceToDevice, s)
                                  : cudaMemsetAsync(dS0, 0, state, s));
    }
    if (!workspace || workspace_bytes < efla_decay_bwd_workspace_size(B, H, L, dk, dv, dt)) return EFLA_ERR_WORKSPACE;
    const bool tc = efla::decay::tc_sizes(dk, dv, dt == EFLA_BF16) && aligned(q, 16) && aligned(k, 16) && aligned(v, 16) &&
                    aligned(dO, 16);
    BwdPlan p(BH, L, dk, dv, tc, workspace);
    const bool want_dl = dlog_g != nullptr, tail = want_dl && dS_final;
    Walk &a = p.ws.w[0], &b = p.ws.w[1], &c = p.ws.w[2];
    a.x = dO; a.y = v; a.z = k;
    a.s0 = S0; a.s0_t = 1;
    a.out = dq;
    a.s_end = tail ? p.S_end : nullptr;
    b.x = v; b.y = dO; b.z = q;
    b.s0 = dS_final; b.s0_t = 1;
    b.out = dkey;
    c.x = k; c.y = q; c.z = dO;
    c.s0 = dS_final;
    c.out = dval;
    c.s_end = dS0;
    if (want_dl) {
        a.dotx = q; a.dot = p.dotq;
        b.dotx = k; b.dot = p.dotk;
    }
    const Gate g{log_g, form == EFLA_DECAY_HEAD, dt == EFLA_BF16, H};
    const bool bf16 = dt == EFLA_BF16;
    cudaError_t e = cudaSuccess;
    if (tc) {
        p.split();
        for (int i = 0; i < p.parts && e == cudaSuccess; ++i)
            e = efla::decay::launch_walks_tc(p.part[i], g, BH, L, p.sh[i], bf16, true, s);
    } else {
        e = efla::decay::launch_walks_simt(p.ws, g, BH, L, p.sg, bf16, bf16, s);
    }
    if (e != cudaSuccess || !want_dl) return from_cuda(e);
    return from_cuda(efla::decay::launch_dlog(p.dotq, p.planes, p.dotk, p.planes, dS_final, tail ? p.S_end : nullptr, g, dlog_g,
                                              BH, L, dk, dv, s));
}

efla_status efla_decay_recurrent_step(const void *q, const void *k, const void *v, const void *log_g,
                                      efla_decay_form form, float *S, void *o, int B, int H, int dk, int dv,
                                      efla_dtype dt, efla_dtype o_dt, void *stream) {
    if (!dtype_ok(dt) || !dtype_ok(o_dt)) return EFLA_ERR_DTYPE;
    if (!form_ok(form)) return EFLA_ERR_OPTION;
    if (!sizes_ok(B, H, 1, dk, dv)) return EFLA_ERR_SHAPE;
    if (dk > 256 || dv > 256) return EFLA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !log_g || !S || !o) return EFLA_ERR_NULL;
    if (!aligned(q, elem(dt)) || !aligned(k, elem(dt)) || !aligned(v, elem(dt)) || !aligned(o, elem(o_dt)) ||
        !aligned(log_g, gate_elem(form, dt)) || !aligned(S, 16))
        return EFLA_ERR_ALIGN;
    const Gate g{log_g, form == EFLA_DECAY_HEAD, dt == EFLA_BF16, H};
    return from_cuda(efla::decay::launch_step(q, k, v, g, S, o, B * H, dk, dv, dt == EFLA_BF16, o_dt == EFLA_BF16,
                                              (cudaStream_t)stream));
}

}  // extern "C"
