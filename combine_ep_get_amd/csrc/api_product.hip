// C ABI of the experts' products, the few-token expert layer and the
// combine's gradient (declared in include/ep_get.h): argument checks and
// launches.  As in api.hip, nothing here allocates, frees or synchronises.
#include <limits.h>

#include "../../include/ep_get.h"
#include "ep_internal.h"
#include "product_internal.h"

namespace {

using epget::check_problem;
using epget::check_shape;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether every pointer (null ones pass) is aligned to 16 bytes.
template <class... P>
bool aligned16(P... p) {
    return (aligned(p, 16) && ...);
}

int hip_rc(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

bool gated(const ep_product *q) { return q->activation == EP_ACT_SWIGLU || q->activation == EP_ACT_GEGLU; }

int32_t weight_rows(const ep_product *q) { return gated(q) ? 2 * q->out_features : q->out_features; }

int check_product(const ep_product *q, int32_t multiple) {
    if (!q || q->reserved != 0) return EP_ERR_INVALID_ARG;
    for (int32_t n : {q->in_features, q->out_features})
        if (n < 8 || n % multiple != 0 || n > EP_MAX_FEATURES) return EP_ERR_INVALID_ARG;
    if (q->activation < EP_ACT_NONE || q->activation > EP_ACT_GEGLU) return EP_ERR_INVALID_ARG;
    // the kernels reach into an expert's weight with 32-bit byte offsets
    if (static_cast<int64_t>(weight_rows(q)) * q->in_features > EP_MAX_WEIGHT) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// The experts' rows.  Null arrays are a dense product of T rows.
int segments(const ep_problem *p, const int32_t *expert_count, const int32_t *expert_offset, epget::Segments *s) {
    if (!expert_count != !expert_offset) return EP_ERR_INVALID_ARG;
    if (!aligned(expert_count, 4) || !aligned(expert_offset, 4)) return EP_ERR_INVALID_ARG;
    if (!expert_count && (p->num_experts != 1 || p->num_topk != 1 || p->rank_stride_rows < p->num_tokens))
        return EP_ERR_INVALID_ARG;
    s->count = expert_count;
    s->offset = expert_offset;
    s->E = p->num_experts;
    s->L = p->num_experts / p->num_ranks;
    s->dense = p->num_tokens;
    s->S = p->rank_stride_rows;
    return EP_OK;
}

int64_t mean_rows(const ep_problem *p) {
    return (static_cast<int64_t>(p->num_tokens) * p->num_topk + p->num_experts - 1) / p->num_experts;
}

int64_t grad_workspace(const ep_problem *p, const ep_product *q) {
    const int64_t splits = epget::grad_row_ranges(p->num_experts, q->out_features);
    const int64_t floats = splits > 1 ? p->num_experts * splits * weight_rows(q) : 0;
    return 256 + floats * 4;
}

// The status and the hidden rows.
int64_t tokens_workspace(const ep_problem *p, const ep_product *q) {
    return 256 + static_cast<int64_t>(p->num_tokens) * p->num_topk * q->out_features * 2;
}

// Behind them, 256-byte aligned, the entries' rows of a 4-bit layer that keeps them.
int64_t tokens_rows_offset(const ep_problem *p, const ep_product *q) { return (tokens_workspace(p, q) + 255) / 256 * 256; }

int64_t tokens_workspace_of(const ep_problem *p, const ep_product *q, epget::WeightType type) {
    if (type != epget::kFp4) return tokens_workspace(p, q);
    const int64_t rows =
        epget::tokens_fp4_rows_bytes(p->num_tokens, p->num_topk, p->num_experts, p->hidden, q->out_features);
    return rows ? tokens_rows_offset(p, q) + rows : tokens_workspace(p, q);
}

int check_tokens(const ep_problem *p, const ep_product *q, int32_t multiple) {
    int rc = check_shape(p);
    if (rc != EP_OK) return rc;
    if ((rc = check_product(q, multiple)) != EP_OK) return rc;
    if (p->num_tokens > EP_MOE_TOKENS_MAX || q->in_features != p->hidden) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Multiple that a weight's sizes have to be of: its blocks of one scale.
int32_t size_step(epget::WeightType w) { return w == epget::kFp8 ? 128 : w == epget::kFp4 ? 32 : 8; }

// Alignment of a weight's scales: fp32, or e8m0 as a whole array.
uintptr_t scale_alignment(epget::WeightType w) { return w == epget::kFp4 ? 16 : 4; }

int run_tokens(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *topk_idx,
               const float *topk_weights, const void *w1, const void *w1_sf, const float *b1, const void *w2,
               const void *w2_sf, const float *b2, const uint16_t *residual, uint16_t *out, void *workspace,
               size_t workspace_bytes, epget::WeightType type, void *stream) {
    const int rc = check_tokens(p, q, size_step(type));
    if (rc != EP_OK) return rc;
    const bool scaled = type != epget::kBf16;
    const int64_t need = tokens_workspace_of(p, q, type);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < static_cast<size_t>(need)) return EP_ERR_INVALID_ARG;
    if (p->num_tokens > 0 && (!x || !topk_idx || !w1 || !w2 || !out || (scaled && (!w1_sf || !w2_sf))))
        return EP_ERR_INVALID_ARG;
    if (!aligned16(x, w1, b1, w2, b2, residual, out) || !aligned(topk_idx, 4) || !aligned(topk_weights, 4) ||
        !aligned(w1_sf, scale_alignment(type)) || !aligned(w2_sf, scale_alignment(type)))
        return EP_ERR_INVALID_ARG;
    epget::TokensArgs a = {};
    a.T = p->num_tokens;
    a.H = p->hidden;
    a.I = q->out_features;
    a.M = weight_rows(q);
    a.E = p->num_experts;
    a.K = p->num_topk;
    a.act = q->activation;
    a.x = x;
    a.idx = topk_idx;
    a.w = topk_weights;
    a.w1 = w1;
    a.w2 = w2;
    a.w1_sf = w1_sf;
    a.w2_sf = w2_sf;
    a.b1 = b1;
    a.b2 = b2;
    a.residual = residual;
    a.out = out;
    a.status = static_cast<int32_t *>(workspace);
    a.h = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + 256);
    a.y = reinterpret_cast<float *>(static_cast<char *>(workspace) + tokens_rows_offset(p, q));
    if (type == epget::kFp4) return hip_rc(epget::launch_tokens_fp4(a, static_cast<hipStream_t>(stream)));
    return hip_rc(epget::launch_tokens(a, type == epget::kFp8, static_cast<hipStream_t>(stream)));
}

int run_product(const ep_problem *p, const ep_product *q, const void *x, const float *x_sf, int64_t sf_ts,
                int64_t sf_hs, const int32_t *expert_count, const int32_t *expert_offset, const void *weight,
                const void *w_sf, const float *bias, const uint16_t *residual, uint16_t *pre, uint16_t *out,
                epget::WeightType type, void *stream) {
    int rc = check_problem(p);
    if (rc != EP_OK) return rc;
    if ((rc = check_product(q, size_step(type))) != EP_OK) return rc;
    const bool fp8 = type == epget::kFp8;
    epget::ProductArgs a = {};
    if ((rc = segments(p, expert_count, expert_offset, &a.seg)) != EP_OK) return rc;
    if (fp8 && (sf_ts < 1 || sf_hs < 1)) return EP_ERR_INVALID_ARG;
    if (p->num_tokens == 0) return EP_OK;
    if (!x || !weight || !out || (fp8 && !x_sf) || (type != epget::kBf16 && !w_sf)) return EP_ERR_INVALID_ARG;
    if (!aligned16(x, weight, bias, residual, pre, out) || !aligned(x_sf, 4) ||
        !aligned(w_sf, scale_alignment(type)))
        return EP_ERR_INVALID_ARG;
    a.C = q->in_features;
    a.N = q->out_features;
    a.M = weight_rows(q);
    a.act = q->activation;
    a.x = x;
    a.weight = weight;
    a.x_sf = x_sf;
    a.w_sf = w_sf;
    a.sf_ts = sf_ts;
    a.sf_hs = sf_hs;
    a.bias = bias;
    a.residual = residual;
    a.pre = pre;
    a.out = out;
    a.entries = static_cast<int64_t>(p->num_tokens) * p->num_topk;
    a.mean_rows = mean_rows(p);
    if (type == epget::kFp4) return hip_rc(epget::launch_product_fp4(a, static_cast<hipStream_t>(stream)));
    return hip_rc(epget::launch_product(a, fp8, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int ep_combine_backward(const ep_problem *p, const uint16_t *dout, const uint16_t *y, const int32_t *token_slot,
                        const float *topk_weights, uint16_t *dy, float *dweights, void *stream) {
    const int rc = check_problem(p);
    if (rc != EP_OK) return rc;
    if (dweights && !y && p->num_tokens > 0) return EP_ERR_INVALID_ARG;
    if (p->num_tokens == 0 || (!dy && !dweights)) return EP_OK;
    if (!dout || !token_slot) return EP_ERR_INVALID_ARG;
    if (!aligned16(dout, y, dy) || !aligned(token_slot, 4) || !aligned(topk_weights, 4) || !aligned(dweights, 4))
        return EP_ERR_INVALID_ARG;
    epget::CopyParams c = {};
    c.T = p->num_tokens;
    c.H = p->hidden;
    c.K = p->num_topk;
    c.nvec = p->hidden / 8;
    c.num_rows = p->rank_stride_rows * p->num_ranks;
    return hip_rc(epget::launch_combine_backward(c, dout, y, token_slot, topk_weights, dy, dweights,
                                                 static_cast<hipStream_t>(stream)));
}

int ep_expert_product(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *expert_count,
                      const int32_t *expert_offset, const uint16_t *weight, const float *bias,
                      const uint16_t *residual, uint16_t *pre, uint16_t *out, void *stream) {
    return run_product(p, q, x, nullptr, 0, 0, expert_count, expert_offset, weight, nullptr, bias, residual, pre, out,
                       epget::kBf16, stream);
}

int ep_expert_product_fp8(const ep_problem *p, const ep_product *q, const uint8_t *x_fp8, const float *x_sf,
                          int64_t sf_token_stride, int64_t sf_hidden_stride, const int32_t *expert_count,
                          const int32_t *expert_offset, const uint8_t *w_fp8, const float *w_sf, const float *bias,
                          const uint16_t *residual, uint16_t *out, void *stream) {
    return run_product(p, q, x_fp8, x_sf, sf_token_stride, sf_hidden_stride, expert_count, expert_offset, w_fp8, w_sf,
                       bias, residual, nullptr, out, epget::kFp8, stream);
}

size_t ep_product_workspace_bytes(const ep_problem *p, const ep_product *q) {
    if (check_problem(p) != EP_OK || check_product(q, 8) != EP_OK) return 0;
    return static_cast<size_t>(grad_workspace(p, q));
}

int ep_expert_product_backward(const ep_problem *p, const ep_product *q, const uint16_t *dout, const uint16_t *pre,
                               const uint16_t *x, const int32_t *expert_count, const int32_t *expert_offset,
                               const uint16_t *weight, uint16_t *dpre, uint16_t *dx, uint16_t *dweight,
                               float *dweight_acc, float *dbias, void *workspace, size_t workspace_bytes,
                               void *stream) {
    int rc = check_problem(p);
    if (rc != EP_OK) return rc;
    if ((rc = check_product(q, 8)) != EP_OK) return rc;
    epget::ProductGradArgs a = {};
    if ((rc = segments(p, expert_count, expert_offset, &a.seg)) != EP_OK) return rc;
    if (q->activation == EP_ACT_NONE && (pre || dpre)) return EP_ERR_INVALID_ARG;
    if (dbias && (!workspace || workspace_bytes < static_cast<size_t>(grad_workspace(p, q)))) return EP_ERR_INVALID_ARG;
    if (!aligned16(dout, pre, x, weight, dpre, dx, dweight, dweight_acc, dbias) || !aligned(workspace, 256))
        return EP_ERR_INVALID_ARG;
    if (p->num_tokens == 0) {  // no rows, whatever the arrays hold: the weights' gradients are zeros
        a.seg.count = a.seg.offset = nullptr;
    } else {
        if (!dout || (q->activation != EP_ACT_NONE && (!pre || !dpre))) return EP_ERR_INVALID_ARG;
        if ((dx && !weight) || ((dweight || dweight_acc) && !x)) return EP_ERR_INVALID_ARG;
    }
    a.C = q->in_features;
    a.N = q->out_features;
    a.M = weight_rows(q);
    a.act = q->activation;
    a.dout = dout;
    a.pre = pre;
    a.x = x;
    a.weight = weight;
    a.dpre = q->activation == EP_ACT_NONE ? const_cast<uint16_t *>(dout) : dpre;  // read only then
    a.dx = dx;
    a.dweight = dweight;
    a.dweight_acc = dweight_acc;
    a.dbias = dbias;
    a.partial = dbias ? reinterpret_cast<float *>(static_cast<char *>(workspace) + 256) : nullptr;
    a.entries = static_cast<int64_t>(p->num_tokens) * p->num_topk;
    a.mean_rows = mean_rows(p);
    a.splits = epget::grad_row_ranges(p->num_experts, q->out_features);
    return hip_rc(epget::launch_product_grad(a, static_cast<hipStream_t>(stream)));
}

size_t ep_moe_tokens_workspace_bytes(const ep_problem *p, const ep_product *q) {
    if (check_tokens(p, q, size_step(epget::kBf16)) != EP_OK) return 0;
    const bool fp4 = check_tokens(p, q, size_step(epget::kFp4)) == EP_OK;  // the most of all
    return static_cast<size_t>(tokens_workspace_of(p, q, fp4 ? epget::kFp4 : epget::kBf16));
}

size_t ep_moe_tokens_weights_workspace_bytes(const ep_problem *p, const ep_product *q, int32_t weights) {
    static_assert(EP_WEIGHTS_BF16 == epget::kBf16 && EP_WEIGHTS_FP8 == epget::kFp8 && EP_WEIGHTS_FP4 == epget::kFp4);
    if (weights < EP_WEIGHTS_BF16 || weights > EP_WEIGHTS_FP4) return 0;
    const auto type = static_cast<epget::WeightType>(weights);
    return check_tokens(p, q, size_step(type)) == EP_OK ? static_cast<size_t>(tokens_workspace_of(p, q, type)) : 0;
}

int ep_moe_tokens(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *topk_idx,
                  const float *topk_weights, const uint16_t *w1, const float *b1, const uint16_t *w2, const float *b2,
                  const uint16_t *residual, uint16_t *out, void *workspace, size_t workspace_bytes, void *stream) {
    return run_tokens(p, q, x, topk_idx, topk_weights, w1, nullptr, b1, w2, nullptr, b2, residual, out, workspace,
                      workspace_bytes, epget::kBf16, stream);
}

int ep_moe_tokens_fp8(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *topk_idx,
                      const float *topk_weights, const uint8_t *w1_fp8, const float *w1_sf, const float *b1,
                      const uint8_t *w2_fp8, const float *w2_sf, const float *b2, const uint16_t *residual,
                      uint16_t *out, void *workspace, size_t workspace_bytes, void *stream) {
    return run_tokens(p, q, x, topk_idx, topk_weights, w1_fp8, w1_sf, b1, w2_fp8, w2_sf, b2, residual, out, workspace,
                      workspace_bytes, epget::kFp8, stream);
}

int ep_expert_product_fp4(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *expert_count,
                          const int32_t *expert_offset, const uint8_t *w_fp4, const uint8_t *w_sf, const float *bias,
                          const uint16_t *residual, uint16_t *out, void *stream) {
    if (p && p->num_tokens > EP_MOE_TOKENS_MAX) return EP_ERR_INVALID_ARG;
    return run_product(p, q, x, nullptr, 0, 0, expert_count, expert_offset, w_fp4, w_sf, bias, residual, nullptr, out,
                       epget::kFp4, stream);
}

int ep_moe_tokens_fp4(const ep_problem *p, const ep_product *q, const uint16_t *x, const int32_t *topk_idx,
                      const float *topk_weights, const uint8_t *w1_fp4, const uint8_t *w1_sf, const float *b1,
                      const uint8_t *w2_fp4, const uint8_t *w2_sf, const float *b2, const uint16_t *residual,
                      uint16_t *out, void *workspace, size_t workspace_bytes, void *stream) {
    return run_tokens(p, q, x, topk_idx, topk_weights, w1_fp4, w1_sf, b1, w2_fp4, w2_sf, b2, residual, out, workspace,
                      workspace_bytes, epget::kFp4, stream);
}

}  // extern "C"
