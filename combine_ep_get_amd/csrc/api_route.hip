// C ABI of the router, its balance loss and gradient, and of the gradients'
// norm and clipping (declared in include/ep_get.h): argument checks and
// launches.  As in api.hip, nothing here allocates, frees or synchronises.
#include <math.h>

#include "../../include/ep_get.h"
#include "ep_internal.h"
#include "grads_internal.h"
#include "route_internal.h"

namespace {

using epget::check_shape;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether every pointer (null ones pass) is aligned to 4 bytes.
template <class... P>
bool aligned4(P... p) {
    return (aligned(p, 4) && ...);
}

int hip_rc(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

int check_router(const ep_problem *p, const ep_router *r) {
    const int rc = check_shape(p);
    if (rc != EP_OK) return rc;
    if (!r || r->score < EP_SCORE_SOFTMAX || r->score > EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
    if ((r->normalise & ~1) || (r->logits_bf16 & ~1) || !isfinite(r->scale)) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

epget::RouteArgs route_args(const ep_problem *p, const ep_router *r, const void *logits, const uint8_t *mask) {
    epget::RouteArgs a = {};
    a.T = p->num_tokens;
    a.E = p->num_experts;
    a.K = p->num_topk;
    a.score = r->score;
    a.normalise = r->normalise;
    a.scale = r->scale;
    a.bf16 = r->logits_bf16 != 0;
    a.logits = logits;
    a.mask = mask;
    return a;
}

// The statistics' arrays and workspace into a: all of them.
int statistics(const ep_problem *p, int32_t *expert_count, int32_t *token_count, float *prob_sum, float *losses,
               void *workspace, size_t workspace_bytes, epget::RouteArgs *a) {
    if (!expert_count || !token_count || !prob_sum || !losses || !workspace) return EP_ERR_INVALID_ARG;
    if (!aligned4(expert_count, token_count, prob_sum, losses) || !aligned(workspace, 256)) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < static_cast<size_t>(epget::route_workspace(p->num_tokens, p->num_experts, p->num_topk)))
        return EP_ERR_INVALID_ARG;
    a->expert_count = expert_count;
    a->token_count = token_count;
    a->prob_sum = prob_sum;
    a->losses = losses;
    a->workspace = workspace;
    return EP_OK;
}

int check_grads(const ep_grad *grads, int32_t num, bool out) {
    if (num < 0 || (num > 0 && !grads)) return EP_ERR_INVALID_ARG;
    for (int32_t i = 0; i < num; ++i) {
        const ep_grad &g = grads[i];
        if (g.reserved != 0 || g.type < EP_GRAD_BF16 || g.type > EP_GRAD_FP32) return EP_ERR_INVALID_ARG;
        if (g.count < 0 || g.count >= int64_t{1} << 40) return EP_ERR_INVALID_ARG;
        const uintptr_t size = g.type == EP_GRAD_FP32 ? 4 : 2;
        if (!aligned(g.grad, size) || (out && !aligned(g.out, size))) return EP_ERR_INVALID_ARG;
        if (g.count > 0 && (!g.grad || (out && !g.out))) return EP_ERR_INVALID_ARG;
    }
    return EP_OK;
}

}  // namespace

extern "C" {

size_t ep_route_workspace_bytes(const ep_problem *p, const ep_router *r) {
    if (check_router(p, r) != EP_OK) return 0;
    return static_cast<size_t>(epget::route_workspace(p->num_tokens, p->num_experts, p->num_topk));
}

int ep_route(const ep_problem *p, const ep_router *r, const void *logits, const float *bias, const uint8_t *token_mask,
             int32_t *topk_idx, float *topk_weights, int32_t *expert_count, int32_t *token_count, float *prob_sum,
             float *losses, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_router(p, r);
    if (rc != EP_OK) return rc;
    epget::RouteArgs a = route_args(p, r, logits, token_mask);
    if (expert_count || token_count || prob_sum || losses) {
        rc = statistics(p, expert_count, token_count, prob_sum, losses, workspace, workspace_bytes, &a);
        if (rc != EP_OK) return rc;
    }
    if (p->num_tokens > 0 && (!logits || !topk_idx || !topk_weights)) return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned4(bias, topk_idx, topk_weights)) return EP_ERR_INVALID_ARG;
    a.bias = bias;
    a.idx = topk_idx;
    a.w = topk_weights;
    return hip_rc(epget::launch_route(a, static_cast<hipStream_t>(stream)));
}

int ep_balance_loss(const ep_problem *p, const ep_router *r, const void *logits, const int32_t *topk_idx,
                    const uint8_t *token_mask, int32_t *expert_count, int32_t *token_count, float *prob_sum,
                    float *losses, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_router(p, r);
    if (rc != EP_OK) return rc;
    epget::RouteArgs a = route_args(p, r, logits, token_mask);
    rc = statistics(p, expert_count, token_count, prob_sum, losses, workspace, workspace_bytes, &a);
    if (rc != EP_OK) return rc;
    if (p->num_tokens > 0 && (!logits || !topk_idx)) return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned4(topk_idx)) return EP_ERR_INVALID_ARG;
    a.idx = const_cast<int32_t *>(topk_idx);  // read only then
    return hip_rc(epget::launch_balance(a, static_cast<hipStream_t>(stream)));
}

int ep_route_backward(const ep_problem *p, const ep_router *r, const void *logits, const int32_t *topk_idx,
                      const uint8_t *token_mask, const int32_t *expert_count, const int32_t *token_count,
                      const float *dweights, const float *dlosses, void *dlogits, void *stream) {
    const int rc = check_router(p, r);
    if (rc != EP_OK) return rc;
    if (dlosses && (!expert_count || !token_count)) return EP_ERR_INVALID_ARG;
    if (p->num_tokens > 0 && (!logits || !dlogits || (dweights && !topk_idx))) return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(dlogits, 16) ||
        !aligned4(topk_idx, expert_count, token_count, dweights, dlosses))
        return EP_ERR_INVALID_ARG;
    epget::RouteArgs a = route_args(p, r, logits, token_mask);
    a.idx = const_cast<int32_t *>(topk_idx);  // read only, as the counts are
    a.expert_count = const_cast<int32_t *>(expert_count);
    a.token_count = const_cast<int32_t *>(token_count);
    a.dw = dweights;
    a.dlosses = dlosses;
    a.dlogits = dlogits;
    return hip_rc(epget::launch_route_backward(a, static_cast<hipStream_t>(stream)));
}

size_t ep_grad_workspace_bytes(const ep_grad *grads, int32_t num_grads) {
    if (check_grads(grads, num_grads, false) != EP_OK) return 0;
    return static_cast<size_t>(epget::grad_workspace_bytes(grads, num_grads));
}

int ep_grad_square_sum(const ep_grad *grads, int32_t num_grads, double *square_sum, void *workspace,
                       size_t workspace_bytes, void *stream) {
    const int rc = check_grads(grads, num_grads, false);
    if (rc != EP_OK) return rc;
    if (!square_sum || !aligned(square_sum, 8) || !workspace || !aligned(workspace, 256)) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < static_cast<size_t>(epget::grad_workspace_bytes(grads, num_grads))) return EP_ERR_INVALID_ARG;
    return hip_rc(epget::launch_square_sum(grads, num_grads, square_sum, workspace, static_cast<hipStream_t>(stream)));
}

int ep_grad_clip(const ep_grad *grads, int32_t num_grads, const double *square_sum, float max_norm, float *norm,
                 void *stream) {
    const int rc = check_grads(grads, num_grads, true);
    if (rc != EP_OK) return rc;
    if (!square_sum || !aligned(square_sum, 8) || !aligned(norm, 4) || !(max_norm >= 0.0f)) return EP_ERR_INVALID_ARG;
    return hip_rc(epget::launch_clip(grads, num_grads, square_sum, max_norm, norm, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
