// decay.h -- linear attention with a decay for each head: what its kernels and its entry points
// share (internal to the library; the public ABI is include/efla.h).
//
//   S_t = e^{l_t} S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t.
//
// Forward and backward are runs of one "walk" over the tokens, with queries x and keys y of a
// elements, values z of b elements and a carried state of a x b:
//
//   forwards:   out_t = sum_{s <= t} e^{c_t - c_s} (x_t . y_s) z_s + e^{c_t} S^T x_t
//   backwards:  out_t = sum_{s >= t} e^{c_s - c_t} (x_t . y_s) z_s + e^{c_C - c_t} S^T x_t
//
// with c the running sum of l over a stretch of tokens (c_C at its end) and S the state that
// enters it (from before it, or from behind it).  The state that leaves is e^{c_C} S +
// sum_s w_s y_s z_s^T with w_s = e^{c_C - c_s} forwards and e^{c_s} backwards.
//
//   o  = forwards (q, k, v) from S0           dq = forwards (dO, v, k) from S0^T
//   dk = backwards (v, dO, q) from dS_final^T  dv = backwards (k, q, dO) from dS_final, ending in dS0
//   dl_t = sum_{u >= t} (q_u . dq_u - k_u . dk_u) + <dS_final, S_final>
//
// The last line: dl_t = e^{l_t} <dL/dS_t, S_{t-1}> = <dL/dS_t, S_t> - k_t . dk_t, and <dL/dS_t, S_t> =
// q_t . dq_t + dl_{t+1}.  The sum ends before the next token that forgets everything, whose dl is zero.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace efla {
namespace decay {

// The log-decay: [B,H,L] in the input type, or [H] fp32.
struct Gate {
    const void *p;
    int per_head;
    int bf16;
    int H;
};

// One walk.  dotx / dot: where dot is given, each token's dotx_t . out_t before out is rounded, as shares
// ([planes][BH][L] fp32, added by the gradient kernel).
struct Walk {
    const void *x, *y, *z;
    const float *s0;  // the state that enters, or null for zero
    int s0_t;         // s0 is stored transposed ([b][a])
    void *out;
    float *s_end;     // the state that leaves, or null
    int a, b, rev;
    const void *dotx;
    float *dot;
};

constexpr int MAX_WALKS = 3;
struct Walks {
    Walk w[MAX_WALKS];
    int n;
};

constexpr int C = 64;             // tokens in a chunk
constexpr float L_MIN = -200.f;   // e^L_MIN is 0 in fp32: lower log-decays (-inf) act as this one (above, 200 does)

// Where whole walks would leave processors idle (few heads, or a last round with few of them), sequences are
// cut: a first pass gives every stretch's own contribution to the state (u, fp32 [a][b]) and its whole decay
// (e), both for every stretch that does not end its sequence, and the walk proper starts a stretch from
// S = e_i S + u_i over the stretches before it.

// CUDA-core walks: any a, b <= 128, fp32 arithmetic; blocks of SIMT_BT value columns.  Every sequence is cut
// into n segments of `chunks` chunks.
constexpr int SIMT_BT = 32;
struct Segments {
    int n, chunks;
    float *u[MAX_WALKS];  // [BH][n - 1][a][b]
    float *e;             // [2][BH][n - 1]: forward walks, backward walks
};
Segments simt_segments(int BH, int L, const int *blocks, int n);
cudaError_t launch_walks_simt(const Walks &ws, Gate g, int BH, int L, const Segments &sg, bool in_bf16, bool out_bf16,
                              cudaStream_t s);

// Tensor-core walks (decay_tc.cu): bf16 inputs, a and b of 64 or 128, x, y and z 16-byte aligned.  bwd: walks
// with dots, given as DOT_PLANES shares (one for each warp of the output group); outputs are bf16.
// All walks (of the same head sizes) one after another, kind by kind, are one row of chunks, and each of g CTAs
// takes an even share of it: the end of one walk, whole ones, the start of another.  The stretch of a share
// that does not end its sequence is the last one.
constexpr int DOT_PLANES = 4;
struct Shares {
    int g;
    bool cut;         // false: shares are whole walks
    long long size;   // chunks in a share; the first `more` have one more
    int more;
    float *u;  // [g - 1][a][b]
    float *e;  // [g - 1]
    int stretches() const { return cut ? g - 1 : 0; }
};
bool tc_sizes(int dk, int dv, bool in_bf16);
Shares tc_shares(int BH, int L, int n);
cudaError_t launch_walks_tc(const Walks &ws, Gate g, int BH, int L, const Shares &sh, bool out_bf16, bool bwd,
                            cudaStream_t s);
cudaError_t read_and_clear_error(unsigned int *out);

// dl from the walks' dots: dotq [nq][BH][L], dotk [nk][BH][L] (shares of their column blocks);
// dS_final [BH][dk][dv] and the forward walk's end state S_end [BH][dv][dk], or both null.
cudaError_t launch_dlog(const float *dotq, int nq, const float *dotk, int nk, const float *dS_final,
                        const float *S_end, Gate g, void *dlog, int BH, int L, int dk, int dv, cudaStream_t s);

cudaError_t launch_step(const void *q, const void *k, const void *v, Gate g, float *S, void *o, int BH, int dk,
                        int dv, bool in_bf16, bool o_bf16, cudaStream_t s);

}  // namespace decay
}  // namespace efla
