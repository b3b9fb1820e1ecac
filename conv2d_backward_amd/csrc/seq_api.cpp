// seq_api.cpp -- entry points of the sequence operators: argument checks, then
// the launchers of seq_kernels.h.
//
// Entry points and their contract are declared in include/sequence_ops.h.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdint>

#include "api_internal.h"
#include "seq_kernels.h"
#include "sequence_ops.h"

namespace {

// Grid sizes: batch items are a grid's y, rows and row pieces its x.
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxStepRows = (int64_t)1 << 28;
constexpr int64_t kMaxPositions = (int64_t)1 << 26;
constexpr int64_t kMaxBatchPositions = (int64_t)1 << 31;  // of all batch items; counted in 32 bits
// A norm's work-groups have 1024 work-items at most, and a grid less than 2^32.
constexpr int64_t kMaxNormTiles = (int64_t)1 << 22;
constexpr int64_t kMaxCodeRows = (int64_t)1 << 22;
constexpr int64_t kMaxProduct = (int64_t)1 << 35;  // elements of a product's result
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;  // work-items of a grid along one axis

int check_sizes(int32_t dtype, int64_t B, int64_t D, int64_t L) {
    if (dtype != SEQ_F32 && dtype != SEQ_BF16 && dtype != SEQ_F16) return CONV2D_GI_EINVAL;
    if (B < 1 || D < 1 || L < 1) return CONV2D_GI_EINVAL;
    if (B > kMaxBatch || B * D >= kMaxRows || L > kMaxPositions || B * L >= kMaxBatchPositions)
        return CONV2D_GI_EUNSUPPORTED;
    return CONV2D_GI_OK;
}

// One position of each row: a batch item is a grid's y, and offsets are 64-bit, so that
// large batches of wide layers fit too.
int check_step(int32_t dtype, int64_t B, int64_t D) {
    const int rc = check_sizes(dtype, 1, D, 1);
    if (rc != CONV2D_GI_OK) return rc;
    if (B < 1) return CONV2D_GI_EINVAL;
    return B > kMaxBatch || B * D >= kMaxStepRows ? CONV2D_GI_EUNSUPPORTED : CONV2D_GI_OK;
}

int check_norm(int64_t B, int64_t D, int64_t L, bool backward, float eps) {
    if (D > SEQ_MAX_NORM_CHANNELS) return CONV2D_GI_EUNSUPPORTED;
    const int64_t columns = backward ? 32 : std::min<int64_t>(32, seq::norm_columns(B, D, L));
    if (B * ((L + columns - 1) / columns) >= kMaxNormTiles) return CONV2D_GI_EUNSUPPORTED;
    return eps >= 0.f ? CONV2D_GI_OK : CONV2D_GI_EINVAL;
}

int check_taps(int32_t K) {
    if (K < 1) return CONV2D_GI_EINVAL;
    return K > SEQ_MAX_TAPS ? CONV2D_GI_EUNSUPPORTED : CONV2D_GI_OK;
}

int check_states(int64_t D, int64_t N, int64_t G) {
    if (N < 1 || G < 1 || D % G != 0) return CONV2D_GI_EINVAL;
    return N > SEQ_MAX_STATES ? CONV2D_GI_EUNSUPPORTED : CONV2D_GI_OK;
}

int check_grid(int64_t items) {
    return items > kMaxItems ? CONV2D_GI_EUNSUPPORTED : CONV2D_GI_OK;
}

int check_scan_backward(int64_t B, int64_t D, int64_t L, int64_t N, int64_t G) {
    const int rc = check_states(D, N, G);
    // The join is one grid, the largest: over 4-position runs of dB and dC ([2, B, G, N]
    // rows padded to whole chunks), 64 to a work-group of 256, and behind them over dA,
    // dskip and ddt_bias, [D, N + 2].
    const int64_t left = kMaxItems - 512 - D * (N + 2);
    if (rc == CONV2D_GI_OK && (left < 0 || B * G * N > left / 2 / (L + 256)))
        return CONV2D_GI_EUNSUPPORTED;
    return rc;
}

// An output's rows must not share elements: dense positions, channels and batch
// items apart by at least what they hold.
bool is_apart(const seq_tensor &t, int64_t B, int64_t D, int64_t L) {
    const int64_t c = t.channel < 0 ? -t.channel : t.channel;
    const int64_t b = t.batch < 0 ? -t.batch : t.batch;
    const int64_t row = L, item = (D - 1) * c + L, all = (B - 1) * b + L;
    if (D == 1) return B == 1 || b >= row;
    if (B == 1) return c >= row;
    // Channels inside a batch item, or batch items inside a channel.
    return (c >= row && b >= item) || (b >= row && c >= all);
}

int64_t int8_row(int64_t D) { return (D + SEQ_INT8_ROW - 1) / SEQ_INT8_ROW * SEQ_INT8_ROW; }

// Of a quantization.  A work-group has 1024 work-items at most and one position at least, and a
// grid less than 2^32 work-items.
int check_codes(int32_t dtype, int64_t B, int64_t D, int64_t L) {
    if (dtype != SEQ_F32 && dtype != SEQ_BF16 && dtype != SEQ_F16) return CONV2D_GI_EINVAL;
    if (B < 1 || D < 1 || L < 1) return CONV2D_GI_EINVAL;
    return D > SEQ_MAX_INT8_CHANNELS || B * L >= kMaxCodeRows ? CONV2D_GI_EUNSUPPORTED
                                                              : CONV2D_GI_OK;
}

// Of a product.  K bounds the sums: 128^2 * 65536 is below 2^31.  The smallest tiles have 16
// work-items for each 256 elements of y, and a grid less than 2^32.
int check_product(int32_t dtype, int64_t B, int64_t E, int64_t L, int64_t K) {
    const int rc = check_codes(dtype, B, 1, L);
    if (rc != CONV2D_GI_OK) return rc;
    if (E < 1 || K < SEQ_INT8_ROW || K % SEQ_INT8_ROW != 0) return CONV2D_GI_EINVAL;
    return K > SEQ_MAX_INT8_CHANNELS || E >= kMaxRows || E * (B * L) >= kMaxProduct
               ? CONV2D_GI_EUNSUPPORTED
               : CONV2D_GI_OK;
}

bool is_codes(const void *p) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool is_workspace(const void *p, int64_t bytes, int64_t needed) {
    return needed == 0 || (p && bytes >= needed && reinterpret_cast<uintptr_t>(p) % 16 == 0);
}

int status(hipError_t e) { return e == hipSuccess ? CONV2D_GI_OK : gi::record_hip_error(e); }

}  // namespace

extern "C" {

int causal_conv_forward(const causal_conv_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_taps(a->K);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->y.data || !a->w) return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, a->L)) return CONV2D_GI_EINVAL;
    return status(seq::launch_conv_forward(*a, stream));
}

int64_t causal_conv_workspace(int32_t B, int32_t D, int32_t L, int32_t K) {
    if (check_sizes(SEQ_F32, B, D, L) != CONV2D_GI_OK || check_taps(K) != CONV2D_GI_OK) return -1;
    return seq::conv_backward_workspace(B, D, L, K);
}

int causal_conv_backward(const causal_conv_backward_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_taps(a->K);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->gy.data || !a->x.data || !a->w) return CONV2D_GI_EINVAL;
    if (a->dx.data && !is_apart(a->dx, a->B, a->D, a->L)) return CONV2D_GI_EINVAL;
    if (!a->dx.data && !a->dw && !a->db) return CONV2D_GI_OK;
    if ((a->dw || a->db) &&
        !is_workspace(a->workspace, a->workspace_bytes,
                      seq::conv_backward_workspace(a->B, a->D, a->L, a->K)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_conv_backward(*a, stream));
}

int causal_conv_step(const causal_conv_step_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_step(a->dtype, a->B, a->D);
    if (rc == CONV2D_GI_OK) rc = check_taps(a->K);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->y.data || !a->w || (!a->state && a->K > 1)) return CONV2D_GI_EINVAL;
    if (a->lines < 1 || (!a->slots && a->lines < a->B)) return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, 1)) return CONV2D_GI_EINVAL;
    return status(seq::launch_conv_step(*a, stream));
}

int state_scan_forward(const state_scan_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_states(a->D, a->N, a->G);
    if (rc == CONV2D_GI_OK) rc = check_grid(seq::scan_forward_items(*a));
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->dt.data || !a->Bm.data || !a->Cm.data || !a->y.data || !a->A)
        return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, a->L)) return CONV2D_GI_EINVAL;
    return status(seq::launch_scan_forward(*a, stream));
}

int64_t state_scan_workspace(int32_t B, int32_t D, int32_t L, int32_t N, int32_t G) {
    if (check_sizes(SEQ_F32, B, D, L) != CONV2D_GI_OK ||
        check_scan_backward(B, D, L, N, G) != CONV2D_GI_OK)
        return -1;
    return seq::scan_backward_workspace(B, D, L, N, G);
}

int state_scan_backward(const state_scan_backward_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_scan_backward(a->B, a->D, a->L, a->N, a->G);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->gout.data || !a->x.data || !a->dt.data || !a->Bm.data || !a->Cm.data || !a->A ||
        !a->checkpoints || !a->dx.data || !a->ddt.data || !a->dBm || !a->dCm || !a->dA)
        return CONV2D_GI_EINVAL;
    if (!a->z.data != !a->dz.data) return CONV2D_GI_EINVAL;
    if (!is_apart(a->dx, a->B, a->D, a->L) || !is_apart(a->ddt, a->B, a->D, a->L) ||
        (a->dz.data && !is_apart(a->dz, a->B, a->D, a->L)))
        return CONV2D_GI_EINVAL;
    if (!is_workspace(a->workspace, a->workspace_bytes,
                      seq::scan_backward_workspace(a->B, a->D, a->L, a->N, a->G)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_scan_backward(*a, stream));
}

int state_scan_plan(int32_t B, int32_t D, int32_t L, int32_t N, int32_t G, int32_t backward,
                    char *buf, size_t len) {
    if (!buf || len == 0) return CONV2D_GI_EINVAL;
    int rc = check_sizes(SEQ_F32, B, D, L);
    if (rc == CONV2D_GI_OK)
        rc = backward ? check_scan_backward(B, D, L, N, G) : check_states(D, N, G);
    if (rc != CONV2D_GI_OK) return rc;
    state_scan_args a = {};
    a.B = B, a.D = D, a.L = L, a.N = N, a.G = G;
    if (!backward && (rc = check_grid(seq::scan_forward_items(a))) != CONV2D_GI_OK) return rc;
    if (backward)
        seq::scan_backward_plan(B, D, L, N, G, buf, len);
    else
        seq::scan_forward_plan(a, buf, len);
    return CONV2D_GI_OK;
}

int state_scan_step(const state_scan_step_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_step(a->dtype, a->B, a->D);
    if (rc == CONV2D_GI_OK) rc = check_states(a->D, a->N, a->G);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->dt.data || !a->Bm.data || !a->Cm.data || !a->y.data || !a->A ||
        !a->state)
        return CONV2D_GI_EINVAL;
    if (a->lines < 1 || (!a->slots && a->lines < a->B)) return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, 1)) return CONV2D_GI_EINVAL;
    return status(seq::launch_scan_step(*a, stream));
}

int block_norm_forward(const block_norm_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_norm(a->B, a->D, a->L, false, a->eps);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->y.data || !a->r.data || !a->r_out.data) return CONV2D_GI_EINVAL;
    if (!a->w_pre != !a->u.data) return CONV2D_GI_EINVAL;
    if (!is_apart(a->r_out, a->B, a->D, a->L) ||
        (a->u.data && !is_apart(a->u, a->B, a->D, a->L)))
        return CONV2D_GI_EINVAL;
    if (!is_workspace(a->workspace, a->workspace_bytes,
                      seq::norm_workspace(a->B, a->D, a->L, 0)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_norm_forward(*a, stream));
}

int64_t block_norm_workspace(int32_t B, int32_t D, int32_t L, int32_t backward) {
    if (check_sizes(SEQ_F32, B, D, L) != CONV2D_GI_OK || check_norm(B, D, L, backward != 0, 0.f) != CONV2D_GI_OK)
        return -1;
    return seq::norm_workspace(B, D, L, backward != 0);
}

int block_norm_backward(const block_norm_backward_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc == CONV2D_GI_OK) rc = check_norm(a->B, a->D, a->L, true, a->eps);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->y.data || !a->r_out.data || !a->dy.data || !a->dr.data) return CONV2D_GI_EINVAL;
    if ((a->gu.data && !a->w_pre) || !a->gate.data != !a->dgate.data) return CONV2D_GI_EINVAL;
    if ((a->dscale && !a->scale) || (a->dw_post && !a->w_post) || (a->dw_pre && !a->w_pre))
        return CONV2D_GI_EINVAL;
    if (!is_apart(a->dy, a->B, a->D, a->L) || !is_apart(a->dr, a->B, a->D, a->L) ||
        (a->dgate.data && !is_apart(a->dgate, a->B, a->D, a->L)))
        return CONV2D_GI_EINVAL;
    if (!is_workspace(a->workspace, a->workspace_bytes,
                      seq::norm_workspace(a->B, a->D, a->L, 1)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_norm_backward(*a, stream));
}

int gated_scan_forward(const gated_scan_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    const int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->r.data || !a->i.data || !a->y.data || !a->A) return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, a->L)) return CONV2D_GI_EINVAL;
    return status(seq::launch_gated_forward(*a, stream));
}

int64_t gated_scan_workspace(int32_t B, int32_t D, int32_t L) {
    if (check_sizes(SEQ_F32, B, D, L) != CONV2D_GI_OK) return -1;
    return seq::gated_backward_workspace(B, D, L);
}

int gated_scan_backward(const gated_scan_backward_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    const int rc = check_sizes(a->dtype, a->B, a->D, a->L);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->gout.data || !a->x.data || !a->r.data || !a->i.data || !a->A || !a->checkpoints ||
        !a->dx.data || !a->dr.data || !a->di.data || !a->dA)
        return CONV2D_GI_EINVAL;
    if (!a->z.data != !a->dz.data) return CONV2D_GI_EINVAL;
    if ((a->dr_bias && !a->r_bias) || (a->di_bias && !a->i_bias)) return CONV2D_GI_EINVAL;
    if (!is_apart(a->dx, a->B, a->D, a->L) || !is_apart(a->dr, a->B, a->D, a->L) ||
        !is_apart(a->di, a->B, a->D, a->L) || (a->dz.data && !is_apart(a->dz, a->B, a->D, a->L)))
        return CONV2D_GI_EINVAL;
    if (!is_workspace(a->workspace, a->workspace_bytes, seq::gated_backward_workspace(a->B, a->D, a->L)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_gated_backward(*a, stream));
}

int gated_scan_plan(int32_t B, int32_t D, int32_t L, int32_t backward, char *buf, size_t len) {
    if (!buf || len == 0) return CONV2D_GI_EINVAL;
    const int rc = check_sizes(SEQ_F32, B, D, L);
    if (rc != CONV2D_GI_OK) return rc;
    seq::gated_plan((int64_t)B * D, L, backward, buf, len);
    return CONV2D_GI_OK;
}

int gated_scan_step(const gated_scan_step_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    const int rc = check_step(a->dtype, a->B, a->D);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !a->r.data || !a->i.data || !a->y.data || !a->A || !a->state)
        return CONV2D_GI_EINVAL;
    if (a->lines < 1 || (!a->slots && a->lines < a->B)) return CONV2D_GI_EINVAL;
    if (!is_apart(a->y, a->B, a->D, 1)) return CONV2D_GI_EINVAL;
    return status(seq::launch_gated_step(*a, stream));
}

int quantize_tokens(const quantize_tokens_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    const int rc = check_codes(a->dtype, a->B, a->D, a->L);
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !is_codes(a->codes) || !a->scales || a->K != int8_row(a->D))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_quantize(*a, stream));
}

int project_int8(const project_int8_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    const int rc = check_product(a->dtype, a->B, a->E, a->L, a->K);
    if (rc != CONV2D_GI_OK) return rc;
    if (!is_codes(a->codes) || !is_codes(a->w) || !a->scales || !a->w_scales || !a->y.data ||
        !is_apart(a->y, a->B, a->E, a->L))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_project(*a, stream));
}

int64_t project_int8_step_workspace_for(int32_t dtype, int32_t B, int32_t D, int32_t E) {
    if (check_codes(dtype, B, D, 1) != CONV2D_GI_OK ||
        check_product(dtype, B, E, 1, int8_row(D)) != CONV2D_GI_OK)
        return -1;
    return seq::project_step_workspace(dtype, B, D, E);
}

int64_t project_int8_step_workspace(int32_t B, int32_t D, int32_t E) {
    return std::max(project_int8_step_workspace_for(SEQ_F32, B, D, E),
                    project_int8_step_workspace_for(SEQ_BF16, B, D, E));
}

int project_int8_step(const project_int8_step_args *a, hipStream_t stream) {
    if (!a) return CONV2D_GI_EINVAL;
    int rc = check_codes(a->dtype, a->B, a->D, 1);
    if (rc == CONV2D_GI_OK) rc = check_product(a->dtype, a->B, a->E, 1, int8_row(a->D));
    if (rc != CONV2D_GI_OK) return rc;
    if (!a->x.data || !is_codes(a->w) || !a->w_scales || !a->y.data || a->K != int8_row(a->D) ||
        !is_apart(a->y, a->B, a->E, 1))
        return CONV2D_GI_EINVAL;
    if (!is_workspace(a->workspace, a->workspace_bytes,
                      seq::project_step_workspace(a->dtype, a->B, a->D, a->E)))
        return CONV2D_GI_EINVAL;
    return status(seq::launch_project_step(*a, stream));
}

}  // extern "C"
