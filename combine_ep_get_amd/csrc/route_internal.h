// Parameters of the router, its balance loss and its gradient.  Internal
// header; the public ABI is include/ep_get.h.
#pragma once

#include "ep_internal.h"

namespace epget {

struct RouteArgs {
    int32_t T, E, K;
    int32_t score;      // EP_SCORE_*
    int32_t normalise;  // weights over the chosen experts' sum
    float scale;
    bool bf16;          // element type of logits and dlogits: bf16, or fp32
    const void *logits;
    const float *bias;    // or null
    const uint8_t *mask;  // or null
    int32_t *idx;         // written by the router, else read
    float *w;
    // statistics (all null in a router call without them)
    int32_t *expert_count, *token_count;
    float *prob_sum, *losses;
    void *workspace;
    // the gradient's
    const float *dw, *dlosses;  // or null
    void *dlogits;
};

// Bytes of the partial sums that a call with statistics leaves.
int64_t route_workspace(int32_t T, int32_t E, int32_t K);

hipError_t launch_route(const RouteArgs &a, hipStream_t stream);
hipError_t launch_balance(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream);

}  // namespace epget
