// norm.h -- launches of the norms around a block (norm.hip), for block_api.hip.
// Shapes are validated by the caller; gate_stride is filled in.
#pragma once

#include <hip/hip_runtime.h>

#include "gdn.h"

namespace gdn {

// rows of partial weight gradients the backward leaves in its workspace
int norm_partials(const gdn_norm_shape& s, bool gate);

gdn_status norm_block_dispatch(const gdn_norm_shape& s, const void* x, const void* y, const float* a, const float* w,
                               void* h, void* n, float* rstd, hipStream_t st);
gdn_status norm_block_bwd_dispatch(const gdn_norm_shape& s, const void* dn, const void* dh, const void* x,
                                   const void* y, const float* a, const float* w, const float* rstd, void* dx,
                                   void* dy, float* dw, float* da, float* part, hipStream_t st);
gdn_status norm_gate_dispatch(const gdn_norm_shape& s, const void* o, const void* z, const float* w, void* y,
                              float* rstd, hipStream_t st);
gdn_status norm_gate_bwd_dispatch(const gdn_norm_shape& s, const void* dy, const void* o, const void* z,
                                  const float* w, const float* rstd, void* dO, void* dz, float* dw, float* part,
                                  hipStream_t st);

}  // namespace gdn
