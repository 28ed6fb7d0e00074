// attn_plan.h -- arguments, launch plans and dispatch of the softmax-attention
// kernels, shared by block_api.hip (validation) and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "gdn.h"

namespace gdn {

// How a forward call is laid out: blocks of `rows` query rows (a row is one
// token of one of the query heads that share a key head), `blocks` of them at
// most for any lengths, and at most `splits` pieces of the key axis, about as
// many as make `want` workgroups.
struct AttnPlan {
    bool small;  // 32-row blocks whose waves share out the keys; else 128-row blocks
    int rows, splits, want;
    long long blocks, jobs;  // jobs: workgroups a key head
    size_t ws_bytes;  // partial outputs [splits][T * Hq][D] and log-sums [splits][T * Hq], fp32
};

AttnPlan attn_plan(const gdn_attn_shape& s, bool paged);

gdn_status attn_forward_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const int* cu,
                                 const int* kv_len, const int* table, void* o, float* lse, void* ws, bool paged,
                                 hipStream_t st);

size_t attn_backward_ws(const gdn_attn_shape& s);
// whether the launches of the gradients stay below 2^32 work-items
bool attn_backward_fits(const gdn_attn_shape& s);
gdn_status attn_backward_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const int* cu,
                                  const void* o, const float* lse, const void* dO, void* dq, void* dk, void* dv,
                                  void* ws, hipStream_t st);

gdn_status attn_append_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const float* cos,
                                const float* sin, const int* cu, const int* kv_len, const int* table, void* k_cache,
                                void* v_cache, void* q_out, hipStream_t st);

}  // namespace gdn
