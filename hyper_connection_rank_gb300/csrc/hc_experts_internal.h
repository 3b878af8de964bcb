// Host-side interfaces of the experts' layer (include/hc_experts.h) and of the
// choice of tokens (include/hc_sample.h) between the C ABI layer and the kernel
// launchers. Arguments are validated before a launcher sees them.
#pragma once

#include "hc_experts.h"
#include "hc_internal.h"
#include "hc_sample.h"

namespace hc {

// Routing (hc_route.cu).
cudaError_t launch_expert_route(const hc_expert_route_t& a, cudaStream_t s);

// Choice of tokens (hc_sample.cu).
constexpr int kSampleMaxVocab = 409600;
cudaError_t launch_token_sample(const hc_token_sample_t& a, int num_sms, cudaStream_t s);

// The experts' products (hc_experts.cu). `aligned`: pointers and strides allow
// TMA copies of x and of the weights.
size_t expert_mlp_workspace(const hc_expert_mlp_t& a, bool aligned, int num_sms);
cudaError_t launch_expert_mlp(const hc_expert_mlp_t& a, bool aligned, int num_sms, cudaStream_t s);

}  // namespace hc
