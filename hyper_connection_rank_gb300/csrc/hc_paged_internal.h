// Host-side interfaces of the paged-cache operators (include/hc_paged.h)
// between the C ABI layer and the kernel launchers. Arguments are validated
// before a launcher sees them.
#pragma once

#include "hc_internal.h"
#include "hc_paged.h"

namespace hc {

// Rotary positions (hc_rotary.cu). `vec`: pointers and strides allow 16-byte
// accesses.
cudaError_t launch_rotary(const hc_rotary_t& a, bool vec, cudaStream_t s);
cudaError_t launch_rotary_append(const hc_rotary_append_t& a, bool vec, cudaStream_t s);

// Attention (hc_attn.cu). `aligned`: every pointer is 16-byte aligned and the
// strides are multiples of 16 bytes.
size_t attention_workspace(const hc_paged_attention_t& a, bool aligned, int num_sms);
cudaError_t launch_attention(const hc_paged_attention_t& a, bool aligned, int num_sms, cudaStream_t s);

// Pages (hc_pages.cu).
size_t pages_workspace(int64_t num_pages, int32_t seqs);
cudaError_t launch_page_copy(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t count, int num_sms, cudaStream_t s);
cudaError_t launch_page_fork(const hc_pages_t& p, const int32_t* parents, int32_t children, int32_t* missing,
                             void* cache, int64_t planes, int64_t page_bytes, void* ws, int num_sms, cudaStream_t s);
cudaError_t launch_page_extend(const hc_pages_t& p, const int32_t* new_tokens, int32_t* missing, void* ws,
                               int num_sms, cudaStream_t s);
cudaError_t launch_page_release(const hc_pages_t& p, const uint8_t* drop, int num_sms, cudaStream_t s);
cudaError_t launch_page_compact(const hc_pages_t& p, int32_t* remap, int32_t* live, void* cache, int64_t planes,
                                int64_t page_bytes, void* ws, int num_sms, cudaStream_t s);

}  // namespace hc
