// pages.h -- dispatch of the page step of the paged cache (pages.hip), for
// mixer_api.hip.  Shapes are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>

#include "gdn.h"

namespace gdn {

gdn_status pages_release_dispatch(const gdn_pages_shape& s, const int* done, const int* kv_len, const int* table, int* free_pages,
                                  const int* free_count, int* kv_out, int* count_out, hipStream_t st);
gdn_status pages_take_dispatch(const gdn_pages_shape& s, const int* want, const int* kv_len, int* table, const int* free_pages,
                               const int* free_count, int* kv_out, int* count_out, int* cu, int* positions, long long* slots,
                               hipStream_t st);

}  // namespace gdn
