/*
 * sequence_ops.h -- C ABI of the sequence operators of the MI355X (gfx950)
 * convolution library: a depthwise causal convolution, a selective state space
 * scan, and the norms between two residual blocks.  Same shared library,
 * status codes and error text as conv2d_grad_input.h.
 *
 * Layouts
 * -------
 * Activations are channel-first, [B, D, L] (batch, channel, position): NCHW
 * with H = 1, so that a 1x1 conv2d_forward projects them.  Positions are
 * contiguous; the batch and channel strides are the caller's (seq_tensor), so
 * an operand can be a slice of a wider tensor's channels.  An activation is
 * fp32, bf16 or fp16 (one type per call); learned parameters, scan states and
 * the residual stream are dense fp32.  Every output is overwritten, never
 * accumulated, and must not overlap an input unless an entry says so.
 *
 * Lengths and cache lines
 * -----------------------
 * lengths (device int32 [B], NULL: all L) gives each sequence's number of
 * positions, clamped to [0, L].  What inputs hold beyond it is not used (it may
 * be NaN), outputs are 0 there.  A length of 0 leaves the sequence's state as
 * it was given.
 * slots (device int32 [B], NULL: row b uses line b) names the line of a state
 * cache of `lines` lines that each row of a single-token call reads and
 * updates in place.  A row whose slot is outside [0, lines) is a padding row:
 * its output is 0 and no line changes.  Rows of one call name different lines.
 *
 * Calls
 * -----
 * Arguments travel in one struct per entry, read during the call.  Calls are
 * asynchronous on `stream`; everything is checked on the host first
 * (CONV2D_GI_EINVAL: null pointer, bad size, type or stride;
 * CONV2D_GI_EUNSUPPORTED: beyond the library's limits), nothing is enqueued on
 * a refusal, and no entry allocates: scratch is the caller's `workspace`, of the
 * size the *_workspace function gives, which may be reused once the call's work
 * is done.  That keeps a call's addresses fixed under graph capture.  All sums
 * are in a fixed order: the same call gives the same bits.
 */
#ifndef SEQUENCE_OPS_H
#define SEQUENCE_OPS_H

#include "conv2d_grad_input.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation types. */
enum { SEQ_F32 = 0, SEQ_BF16 = 1, SEQ_F16 = 2 };

/* Limits: taps of a causal convolution, states of a scan, channels of a norm.
   Of every entry: B <= 65535, B*D < 2^24 (single tokens: D < 2^24, B*D < 2^28),
   L <= 2^26, B*L < 2^31 (norms: about 2^27, block_norm_forward with 1025 .. 2048
   channels 2^26, in whole tiles of positions);
   of state_scan_backward also 2*B*G*N*(L+256) + D*(N+2) < 2^32 - 512. */
enum { SEQ_MAX_TAPS = 8, SEQ_MAX_STATES = 256, SEQ_MAX_NORM_CHANNELS = 65536 };

/* An activation [B, D, L]: element (b, d, t) at data[b*batch + d*channel + t].
   Strides in elements; they may be 0 (an input broadcast) or negative. */
typedef struct seq_tensor {
    void *data;
    int64_t batch, channel;
} seq_tensor;

/*
 * causal_conv: the depthwise causal convolution of K taps with its bias and
 * SiLU.  With full = the K-1 values of state_in followed by x,
 *
 *   p[b,d,t] = bias[d] + sum over k < K of w[d,k] * full[b,d,t+k]
 *   y = p * sigmoid(p)  (silu) or p        for t < len, 0 beyond
 *   state_out[b,d,:] = full[b,d,len .. len+K-2]
 *
 * state_in NULL: zeros; state_out NULL: not wanted.  Both [B, D, K-1] dense, of
 * x's type; state_out may be state_in.
 */
typedef struct causal_conv_args {
    int32_t dtype, B, D, L, K, silu;
    seq_tensor x, y;
    const float *w;      /* [D, K]                    */
    const float *bias;   /* [D] or NULL               */
    const void *state_in;
    void *state_out;
    const int32_t *lengths;
} causal_conv_args;
CONV2D_GI_API int causal_conv_forward(const causal_conv_args *a, hipStream_t stream);

/*
 * The gradients of causal_conv from a zero state, given gy, the gradient of y:
 *   dp = gy * (d y / d p) for t < len, 0 beyond
 *   dx[t] = sum over j < K of w[d,K-1-j] * dp[t+j]        (T, like x)
 *   dw[d,k] = sum over b, t of dp[t] * x[t-K+1+k],  db[d] = sum of dp   (fp32)
 * dx.data, dw or db NULL: not wanted.  workspace: causal_conv_workspace bytes.
 */
typedef struct causal_conv_backward_args {
    int32_t dtype, B, D, L, K, silu;
    seq_tensor gy, x, dx;
    const float *w, *bias;
    float *dw, *db;
    const int32_t *lengths;
    void *workspace;
    int64_t workspace_bytes;
} causal_conv_backward_args;
CONV2D_GI_API int causal_conv_backward(const causal_conv_backward_args *a, hipStream_t stream);
CONV2D_GI_API int64_t causal_conv_workspace(int32_t B, int32_t D, int32_t L, int32_t K);

/*
 * One position of causal_conv for every row: x and y [B, D] (seq_tensor with
 * position 0 only), state [lines, D, K-1] dense, updated in place.
 */
typedef struct causal_conv_step_args {
    int32_t dtype, B, D, K, silu, lines;
    seq_tensor x, y;   /* .channel is the element stride along D */
    const float *w, *bias;
    void *state;
    const int32_t *slots;
} causal_conv_step_args;
CONV2D_GI_API int causal_conv_step(const causal_conv_step_args *a, hipStream_t stream);

/*
 * state_scan: the selective state space scan.  With s = softplus(dt + dt_bias)
 * (softplus != 0) or dt + dt_bias, g = d / (D/G) the group of channel d,
 *
 *   h[b,d,t,n] = exp(s[b,d,t] * A[d,n]) * h[b,d,t-1,n] + s[b,d,t] * x[b,d,t] * Bm[b,g,n,t]
 *   y[b,d,t]   = sum over n of Cm[b,g,n,t] * h[b,d,t,n] + skip[d] * x[b,d,t]
 *   out        = y * z * sigmoid(z)  (z given) or y         for t < len, 0 beyond
 *
 * h before position 0 is state_in ([B, D, N], NULL: zeros); state_out [B, D, N]
 * (NULL: not wanted) is h after the last position.  Bm and Cm are [B, G, N, L]:
 * seq_tensor.channel is the stride between consecutive states, G*N of them.
 * checkpoints (NULL: not wanted) receives the state before every
 * SEQ_SCAN_CHECKPOINT-th position, [B, D, ceil(L / SEQ_SCAN_CHECKPOINT), N], for
 * the backward call.  The states are kept in fp32 registers throughout.
 * A is meant to be negative; -inf forgets the state at each position.  Where decays
 * above 1 multiply beyond fp32's range over up to 1024 positions, a state of 0 may
 * come out as NaN.
 */
enum { SEQ_SCAN_CHECKPOINT = 128 };
typedef struct state_scan_args {
    int32_t dtype, B, D, L, N, G, softplus, reserved;
    seq_tensor x, dt, z, Bm, Cm, y;   /* z.data NULL: no gate */
    const float *A;                   /* [D, N] */
    const float *skip, *dt_bias;      /* [D] or NULL */
    const float *state_in;
    float *state_out, *checkpoints;
    const int32_t *lengths;
} state_scan_args;
CONV2D_GI_API int state_scan_forward(const state_scan_args *a, hipStream_t stream);

/*
 * The gradients of state_scan.  gout is the gradient of out, gstate [B, D, N]
 * (NULL: zeros) that of state_out.  With gy = gout * silu(z) (or gout) and
 * q[t,n] the gradient of h[t,n]:
 *   q[t]  = Cm[t] * gy[t] + exp(s[t+1] A) * q[t+1]       (beyond len: gstate)
 *   dx    = skip * gy + s * sum over n of q Bm
 *   ds    = x * sum over n of q Bm + sum over n of A * q * exp(s A) h[t-1]
 *   ddt   = ds * sigmoid(dt + dt_bias)  (softplus) or ds;   ddt_bias = sum over b, t of ddt
 *   dA    = sum over b, t of q * s * exp(s A) h[t-1];       dskip = sum over b, t of gy * x
 *   dBm   = sum over the group's channels of q * s * x;     dCm = ... of gy * h
 *   dz    = gout * y * (d silu / d z);                      dstate = exp(s[0] A) q[0]
 * dx, ddt, dz have x's layout rules and type; dBm, dCm are dense [B, G, N, L] of
 * x's type; dA [D, N], dskip, ddt_bias [D], dstate [B, D, N] fp32.  dx, ddt, dA,
 * dBm and dCm are required, dz with z, the others may be NULL.  checkpoints: as
 * the forward call on the same inputs wrote them.
 */
typedef struct state_scan_backward_args {
    int32_t dtype, B, D, L, N, G, softplus, reserved;
    seq_tensor gout, x, dt, z, Bm, Cm, dx, ddt, dz;
    const float *A, *skip, *dt_bias, *checkpoints, *gstate;
    void *dBm, *dCm;
    float *dA, *dskip, *ddt_bias, *dstate;
    const int32_t *lengths;
    void *workspace;
    int64_t workspace_bytes;
} state_scan_backward_args;
CONV2D_GI_API int state_scan_backward(const state_scan_backward_args *a, hipStream_t stream);
CONV2D_GI_API int64_t state_scan_workspace(int32_t B, int32_t D, int32_t L, int32_t N, int32_t G);

/*
 * Host-only: how the work of a state_scan_forward (backward = 0) or _backward
 * call of these sizes is dealt, as text written into buf (NUL-terminated,
 * truncated to len): waves of a work-group, positions of a lane and, forward,
 * lanes of a row, waves that share a row's states and states staged at once;
 * backward, segments of a row and states whose sums over channels are joined at
 * once.  Returns a status code.
 */
CONV2D_GI_API int state_scan_plan(int32_t B, int32_t D, int32_t L, int32_t N, int32_t G,
                                  int32_t backward, char *buf, size_t len);

/*
 * One position of state_scan for every row: x, dt, z, out [B, D], Bm and Cm
 * [B, G, N] (seq_tensor.channel: the stride between consecutive states), state
 * [lines, D, N] dense fp32, updated in place.
 */
typedef struct state_scan_step_args {
    int32_t dtype, B, D, N, G, softplus, lines, reserved;
    seq_tensor x, dt, z, Bm, Cm, y;
    const float *A, *skip, *dt_bias;
    float *state;
    const int32_t *slots;
} state_scan_step_args;
CONV2D_GI_API int state_scan_step(const state_scan_step_args *a, hipStream_t stream);

/*
 * block_norm: what stands between two residual blocks.  Over the D channels of
 * each position, with rms(v) = v / sqrt(mean of v^2 + eps),
 *
 *   n     = rms(y) * w_post                 (w_post NULL: n = y)
 *   r_out = r + scale * sigmoid(gate) * n   (scale or gate NULL: without it)
 *   u     = rms(r_out) * w_pre              (w_pre NULL: no u)
 *
 * eps >= 0; at eps = 0 a position whose values are all 0 is 0/0.
 * y, gate and u have the call's type, r and r_out [B, D, L] are fp32 (r_out may
 * be r itself, same strides).  r_out and u are 0 beyond a sequence's length.
 */
typedef struct block_norm_args {
    int32_t dtype, B, D, L;
    float eps;
    int32_t reserved;
    seq_tensor y, gate, r, r_out, u;
    const float *scale, *w_post, *w_pre;   /* [D] or NULL */
    const int32_t *lengths;
    void *workspace;
    int64_t workspace_bytes;
} block_norm_args;
CONV2D_GI_API int block_norm_forward(const block_norm_args *a, hipStream_t stream);

/*
 * The gradients of block_norm: gr (fp32) of r_out, gu of u (each .data may be
 * NULL: zeros; gu only with w_pre), r_out as the forward call wrote it.
 *   dr = gr + the gradient of u's norm (fp32);   dy, dgate (T);
 *   dscale, dw_post, dw_pre [D] (fp32).
 * dr and dy are required; dgate with gate; each of the others may be NULL.
 */
typedef struct block_norm_backward_args {
    int32_t dtype, B, D, L;
    float eps;
    int32_t reserved;
    seq_tensor gr, gu, y, gate, r_out, dy, dr, dgate;
    const float *scale, *w_post, *w_pre;
    float *dscale, *dw_post, *dw_pre;
    const int32_t *lengths;
    void *workspace;
    int64_t workspace_bytes;
} block_norm_backward_args;
CONV2D_GI_API int block_norm_backward(const block_norm_backward_args *a, hipStream_t stream);
/* Bytes of scratch for block_norm_forward (backward 0) or _backward (1). */
CONV2D_GI_API int64_t block_norm_workspace(int32_t B, int32_t D, int32_t L, int32_t backward);

#ifdef __cplusplus
}
#endif

#endif /* SEQUENCE_OPS_H */
