// The global norm of many gradients, and clipping.  Internal header; the
// public ABI is include/ep_get.h.
#pragma once

#include "ep_internal.h"

struct ep_grad;

namespace epget {

// Bytes of workspace that the square sum of these (checked) gradients needs.
int64_t grad_workspace_bytes(const ep_grad *grads, int32_t num);

hipError_t launch_square_sum(const ep_grad *grads, int32_t num, double *square_sum, void *workspace, hipStream_t stream);
hipError_t launch_clip(const ep_grad *grads, int32_t num, const double *square_sum, float max_norm, float *norm,
                       hipStream_t stream);

}  // namespace epget
