// Host-side launchers of the stateless operators (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lq.h"

namespace lq {

// Tokens between two checkpoints of the gated scan: what one CTA of the
// backward pass takes in a step.
int scan_checkpoint_tokens(const lq_scan_config &c);

// `vec`: every row of every tensor of the call is whole, aligned pieces of 16 bytes.
cudaError_t launch_scan_forward(const lq_scan_config &c, const lq_scan_args &a, bool vec, cudaStream_t s);
cudaError_t launch_scan_backward(const lq_scan_config &c, const lq_scan_args &a, const lq_scan_grads &g, bool vec,
                                 cudaStream_t s);

// Partial weight gradients that the norm's backward pass writes at most: one
// for each CTA and each of q and k.
constexpr int kQkPartials = 1024;

cudaError_t launch_qk_norm(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &out, bool vec,
                           cudaStream_t s);
cudaError_t launch_qk_norm_backward(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &grad_out,
                                    const lq_qk_pair &grad_in, float *grad_wq, float *grad_wk, float *partials,
                                    bool vec, cudaStream_t s);

}  // namespace lq
