// conv.h -- arguments and dispatch of the short causal convolution (conv.hip), for
// mixer_api.hip.  Shapes are validated by the caller; x_stride is filled in.
#pragma once

#include <hip/hip_runtime.h>

#include "gdn.h"

namespace gdn {

struct ConvArgs {
    const void *x, *state, *dy, *dstate_out;
    const float *w, *bias;
    const int* cu;  // null: one row a sequence
    void *y, *state_out, *dx, *dstate;
    float* part;
    long long x_stride;
    int B, T, C, silu;
    int strip, head_blocks;  // filled in by the dispatch
};

// rows of partial weight gradients ([W + 1][C] each) the backward leaves in its workspace
int conv_partials(const gdn_conv_shape& s);

gdn_status conv_forward_dispatch(const gdn_conv_shape& s, const ConvArgs& a, hipStream_t st);
gdn_status conv_backward_dispatch(const gdn_conv_shape& s, const ConvArgs& a, float* dw, float* db, hipStream_t st);

}  // namespace gdn
