// bounds.h -- the sequences of packed rows, read alike by the short convolution
// (conv.hip) and the state space scan (ssm_*.hip): device code.
#pragma once

#include "common.h"

namespace gdn {

// Bounds of the lanes' sequences b0, b0 + 1 .., clamped to 0 <= start <= end <= T; a
// bound below an earlier one counts as that one, so that no row is two sequences':
// none is written twice, and the scan's workspace has the chunks of T rows.  top: the greatest bound so far, 0 at first.
// The search for it runs only where there is such a bound.
__device__ __forceinline__ void ordered_bounds(const int* __restrict__ cu, int B, int T, int b0, int& top, int& st, int& en)
{
    const int l = lane_id(), b = b0 + l < B ? b0 + l : B - 1;
    st = cu[b], en = cu[b + 1];
    st = st < 0 ? 0 : st > T ? T : st;
    en = en < 0 ? 0 : en > T ? T : en;
    if (__any(en < st || st < top)) {
        st = st < top ? top : st;
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(st, o);
            if (l >= o && up > st) st = up;
        }
        en = en < st ? st : en;
    }
    top = __builtin_amdgcn_readlane(en, 63);
}

}  // namespace gdn
