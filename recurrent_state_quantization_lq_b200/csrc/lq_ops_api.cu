// C ABI of the stateless operators: checks of arguments and launches.  The
// declarations and the contract of every entry point are in include/lq.h.
#include <cmath>

#include "lq_host.h"
#include "lq_ops.h"

namespace {

using lq::aligned;
using lq::cuda_fail;
using lq::fail;
using lq::Range;

size_t element(int32_t dtype) { return dtype == LQ_DTYPE_BF16 ? 2 : 4; }

bool dtype_ok(int32_t t) { return t == LQ_DTYPE_F32 || t == LQ_DTYPE_BF16; }

const char *why_not(const lq_scan_config *c) {
    if (c == nullptr) return "config is NULL";
    if (c->batch < 1 || c->heads < 1) return "batch and heads must be >= 1";
    if ((long long)c->batch * c->heads > (1LL << 24)) return "batch * heads must be <= 2^24";
    if (c->d < 1 || c->d > 256) return "d must be in 1..256";
    if (c->gate != LQ_GATE_SCALAR && c->gate != LQ_GATE_CHANNEL) return "gate must be LQ_GATE_SCALAR or LQ_GATE_CHANNEL";
    if (!dtype_ok(c->in_dtype) || !dtype_ok(c->out_dtype)) return "in_dtype and out_dtype must be LQ_DTYPE_F32 or LQ_DTYPE_BF16";
    return nullptr;
}

// A tensor [T][batch][heads][d] of one call.
struct Extent {
    int64_t T, B, H;
    int d;
};

// Whether every row of a tensor is whole, aligned pieces of 16 bytes, and its
// rows are apart (as a tensor map wants them).
bool rows_of_16_bytes(const void *p, const lq_strides &s, const Extent &x, size_t e) {
    if (p == nullptr) return true;
    auto fits = [&](int64_t n, int64_t stride) {
        const int64_t bytes = stride * (int64_t)e;
        return n <= 1 || (bytes > 0 && bytes % 16 == 0 && bytes < (1LL << 40));
    };
    return aligned(p, 16) && x.d * e % 16 == 0 && fits(x.T, s.token) && fits(x.B, s.seq) && fits(x.H, s.head);
}

// Whether two elements of an output could have one address for want of a stride.
bool strides_cover(const void *p, const lq_strides &s, int64_t T, int64_t B, int64_t H) {
    return p == nullptr || !((T > 1 && s.token == 0) || (B > 1 && s.seq == 0) || (H > 1 && s.head == 0));
}

const char *why_not(const lq_scan_config &c, const lq_scan_args *a, bool *vec) {
    if (a == nullptr) return "args is NULL";
    if (a->n_tokens < 0) return "negative n_tokens";
    if (a->n_tokens > (1 << 30)) return "n_tokens must be <= 2^30";
    if (a->zero_past != 0 && a->zero_past != 1) return "zero_past must be 0 or 1";
    if (a->n_tokens > 0 && (a->v == nullptr || a->g == nullptr)) return "NULL v or g";
    if (!aligned(a->v, element(c.in_dtype)) || !aligned(a->out, element(c.out_dtype)) || !aligned(a->g, 4) ||
        !aligned(a->beta, 4) || !aligned(a->h0, 4) || !aligned(a->h_last, 4) || !aligned(a->checkpoints, 4) ||
        !aligned(a->lengths, 4))
        return "a pointer is not aligned to its element";
    const bool chan = c.gate == LQ_GATE_CHANNEL;
    const Extent x{a->n_tokens, c.batch, c.heads, c.d};
    *vec = c.d % 4 == 0 && rows_of_16_bytes(a->v, a->v_stride, x, element(c.in_dtype)) &&
           (!chan || rows_of_16_bytes(a->g, a->g_stride, x, 4)) && aligned(a->h0, 16) && aligned(a->checkpoints, 16);
    return nullptr;
}

const char *why_not(const lq_qk_norm_config *c) {
    if (c == nullptr) return "config is NULL";
    if (c->heads_q < 1 || c->heads_k < 0) return "heads_q must be >= 1 and heads_k >= 0";
    if (c->heads_q > (1 << 20) || c->heads_k > (1 << 20)) return "heads must be <= 2^20";
    if (c->d < 1 || c->d > 256) return "d must be in 1..256";
    if (c->norm != LQ_NORM_L2 && c->norm != LQ_NORM_RMS) return "norm must be LQ_NORM_L2 or LQ_NORM_RMS";
    if (c->rot_dim < 0 || c->rot_dim > c->d || c->rot_dim % 2 != 0) return "rot_dim must be even and in 0..d";
    if (c->pairs != LQ_PAIRS_HALF && c->pairs != LQ_PAIRS_NEIGHBOURS) return "pairs must be LQ_PAIRS_HALF or LQ_PAIRS_NEIGHBOURS";
    if (!dtype_ok(c->dtype)) return "dtype must be LQ_DTYPE_F32 or LQ_DTYPE_BF16";
    if (!std::isfinite(c->eps) || c->eps <= 0.0f) return "eps must be finite and > 0";
    if (!std::isfinite(c->q_scale)) return "q_scale must be finite";
    return nullptr;
}

const char *why_not(const lq_qk_norm_config &c, const lq_qk_norm_args *a) {
    if (a == nullptr) return "args is NULL";
    if (a->n_tokens < 0 || a->n_tokens > (1LL << 31) - 1) return "n_tokens must be in 0..2^31 - 1";
    if (a->n_tokens == 0) return nullptr;
    if (a->q == nullptr || (c.heads_k > 0 && a->k == nullptr)) return "NULL q or k";
    if (c.rot_dim > 0 && (a->positions == nullptr || a->inv_freq == nullptr)) return "a rotation needs positions and inv_freq";
    const size_t e = element(c.dtype);
    if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->positions, 4) || !aligned(a->inv_freq, 8) ||
        !aligned(a->weight_q, 4) || !aligned(a->weight_k, 4))
        return "a pointer is not aligned to its element";
    return nullptr;
}

const char *why_not(const lq_qk_norm_config &c, int64_t n_tokens, const lq_qk_pair *p, bool written) {
    if (p == nullptr) return "a pair of outputs or gradients is NULL";
    if (n_tokens == 0) return nullptr;
    if (p->q == nullptr || (c.heads_k > 0 && p->k == nullptr)) return "NULL output or gradient";
    if (!aligned(p->q, element(c.dtype)) || !aligned(p->k, element(c.dtype))) return "a pointer is not aligned to its element";
    if (written && ((n_tokens > 1 && (p->q_token == 0 || (c.heads_k > 0 && p->k_token == 0))) ||
                    (c.heads_q > 1 && p->q_head == 0) || (c.heads_k > 1 && p->k_head == 0)))
        return "an output dimension has stride 0";
    return nullptr;
}

// Whether every row of q and k is whole, aligned pieces of 16 bytes.
bool rows_of_16_bytes(const lq_qk_norm_config &c, const void *q, const void *k, int64_t q_token, int64_t q_head,
                      int64_t k_token, int64_t k_head) {
    const int64_t m = (int64_t)(16 / element(c.dtype));
    const bool keys = c.heads_k == 0 || (aligned(k, 16) && k_token % m == 0 && k_head % m == 0);
    return c.d % m == 0 && aligned(q, 16) && q_token % m == 0 && q_head % m == 0 && keys;
}
bool rows_of_16_bytes(const lq_qk_norm_config &c, const lq_qk_pair &p) {
    return rows_of_16_bytes(c, p.q, p.k, p.q_token, p.q_head, p.k_token, p.k_head);
}

}  // namespace

extern "C" {

size_t lq_gated_scan_checkpoint_bytes(const lq_scan_config *cfg, int32_t n_tokens) {
    const char *why = why_not(cfg);
    if (why == nullptr && (n_tokens < 0 || n_tokens > (1 << 30))) why = "n_tokens must be in 0..2^30";
    if (why != nullptr) {
        fail(LQ_ERR_INVALID_ARG, why);
        return 0;
    }
    const size_t every = (size_t)lq::scan_checkpoint_tokens(*cfg);
    return ((size_t)n_tokens + every - 1) / every * (size_t)cfg->batch * (size_t)cfg->heads * (size_t)cfg->d * 4;
}

lq_status lq_gated_scan(const lq_scan_config *cfg, const lq_scan_args *args, void *stream) {
    Range nvtx_range("lq_gated_scan");
    bool vec = false;
    if (const char *why = why_not(cfg)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args, &vec)) return fail(LQ_ERR_INVALID_ARG, why);
    if (!strides_cover(args->out, args->out_stride, args->n_tokens, cfg->batch, cfg->heads))
        return fail(LQ_ERR_INVALID_ARG, "an output dimension has stride 0");
    const Extent x{args->n_tokens, cfg->batch, cfg->heads, cfg->d};
    vec = vec && rows_of_16_bytes(args->out, args->out_stride, x, element(cfg->out_dtype)) && aligned(args->h_last, 16);
    const cudaError_t e = lq::launch_scan_forward(*cfg, *args, vec, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LQ_OK : cuda_fail(e, "launching the scan kernel");
}

lq_status lq_gated_scan_backward(const lq_scan_config *cfg, const lq_scan_args *args, const lq_scan_grads *grads,
                                 void *stream) {
    Range nvtx_range("lq_gated_scan_backward");
    bool vec = false;
    if (const char *why = why_not(cfg)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args, &vec)) return fail(LQ_ERR_INVALID_ARG, why);
    if (grads == nullptr) return fail(LQ_ERR_INVALID_ARG, "grads is NULL");
    if (args->n_tokens > 0 && args->checkpoints == nullptr) return fail(LQ_ERR_INVALID_ARG, "NULL checkpoints");
    if (grads->grad_beta != nullptr && args->beta == nullptr) return fail(LQ_ERR_INVALID_ARG, "grad_beta without beta");
    if (!aligned(grads->grad_out, element(cfg->out_dtype)) || !aligned(grads->grad_v, element(cfg->in_dtype)) ||
        !aligned(grads->grad_last, 4) || !aligned(grads->grad_g, 4) || !aligned(grads->grad_beta, 4) ||
        !aligned(grads->grad_h0, 4))
        return fail(LQ_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    const int64_t T = args->n_tokens, B = cfg->batch, H = cfg->heads;
    if (!strides_cover(grads->grad_v, grads->grad_v_stride, T, B, H) ||
        !strides_cover(grads->grad_g, grads->grad_g_stride, T, B, H) ||
        !strides_cover(grads->grad_beta, grads->grad_beta_stride, T, B, H))
        return fail(LQ_ERR_INVALID_ARG, "an output dimension has stride 0");
    const Extent x{T, B, H, cfg->d};
    // (a grad_out that is not there has rows in shared memory all the same, which the kernel clears)
    vec = vec && cfg->d * element(cfg->out_dtype) % 16 == 0 &&
          rows_of_16_bytes(grads->grad_out, grads->grad_out_stride, x, element(cfg->out_dtype)) &&
          rows_of_16_bytes(grads->grad_v, grads->grad_v_stride, x, element(cfg->in_dtype)) &&
          (cfg->gate != LQ_GATE_CHANNEL || rows_of_16_bytes(grads->grad_g, grads->grad_g_stride, x, 4));
    const cudaError_t e = lq::launch_scan_backward(*cfg, *args, *grads, vec, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LQ_OK : cuda_fail(e, "launching the scan's backward kernel");
}

lq_status lq_qk_norm_rotate(const lq_qk_norm_config *cfg, const lq_qk_norm_args *args, const lq_qk_pair *out,
                            void *stream) {
    Range nvtx_range("lq_qk_norm_rotate");
    if (const char *why = why_not(cfg)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args->n_tokens, out, true)) return fail(LQ_ERR_INVALID_ARG, why);
    const bool vec = rows_of_16_bytes(*cfg, args->q, args->k, args->q_token, args->q_head, args->k_token, args->k_head) &&
                     rows_of_16_bytes(*cfg, *out);
    const cudaError_t e = lq::launch_qk_norm(*cfg, *args, *out, vec, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LQ_OK : cuda_fail(e, "launching the norm kernel");
}

size_t lq_qk_norm_rotate_workspace_bytes(const lq_qk_norm_config *cfg) {
    if (const char *why = why_not(cfg)) {
        fail(LQ_ERR_INVALID_ARG, why);
        return 0;
    }
    return (size_t)2 * lq::kQkPartials * (size_t)cfg->d * 4;
}

lq_status lq_qk_norm_rotate_backward(const lq_qk_norm_config *cfg, const lq_qk_norm_args *args,
                                     const lq_qk_pair *grad_out, const lq_qk_pair *grad_in, float *grad_weight_q,
                                     float *grad_weight_k, void *workspace, void *stream) {
    Range nvtx_range("lq_qk_norm_rotate_backward");
    if (const char *why = why_not(cfg)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args->n_tokens, grad_out, false)) return fail(LQ_ERR_INVALID_ARG, why);
    if (const char *why = why_not(*cfg, args->n_tokens, grad_in, true)) return fail(LQ_ERR_INVALID_ARG, why);
    if ((grad_weight_q != nullptr && args->weight_q == nullptr) || (grad_weight_k != nullptr && args->weight_k == nullptr))
        return fail(LQ_ERR_INVALID_ARG, "a weight gradient without its weight");
    if (grad_weight_k != nullptr && cfg->heads_k == 0) return fail(LQ_ERR_INVALID_ARG, "a weight gradient of keys without keys");
    if (!aligned(grad_weight_q, 4) || !aligned(grad_weight_k, 4))
        return fail(LQ_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    if ((grad_weight_q != nullptr || grad_weight_k != nullptr) && (workspace == nullptr || !aligned(workspace, 16)))
        return fail(LQ_ERR_WORKSPACE, "a weight gradient needs a 16-byte aligned workspace");
    const bool vec = rows_of_16_bytes(*cfg, args->q, args->k, args->q_token, args->q_head, args->k_token, args->k_head) &&
                     rows_of_16_bytes(*cfg, *grad_out) && rows_of_16_bytes(*cfg, *grad_in);
    const cudaError_t e = lq::launch_qk_norm_backward(*cfg, *args, *grad_out, *grad_in, grad_weight_q, grad_weight_k,
                                                      static_cast<float *>(workspace), vec,
                                                      static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LQ_OK : cuda_fail(e, "launching the norm's backward kernel");
}

}  // extern "C"
