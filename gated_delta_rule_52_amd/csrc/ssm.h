// ssm.h -- arguments, plans and dispatch of the selective state space scan
// (ssm_*.hip), for mixer_api.hip.
//
// The scan, of head h in group h / (H / G):
//   delta = softplus(dt + bias) or dt + bias,  g = delta A,
//   S_t = exp(g_t) S_{t-1} + delta_t B_t x_t^T,   y_t = S_t^T C_t + D x_t
// is computed in chunks of L tokens.  With c the running sum of g in a chunk and
// E_ts = exp(c_t - c_s) for s <= t, 0 otherwise,
//   y = (E o C B^T) (delta x) + exp(c) C S_in + D x,
//   S_out = exp(c_L) S_in + B^T (exp(c_L - c) delta x):
// all of it matrix products.  A head's P values are independent of one another,
// so everything is done in slices of 64 of them.  The decays
// (ssm_prep.hip) and the states between chunks (ssm_walk.hip) are formed first; outputs (ssm_out.hip) and gradients
// (ssm_grad.hip) are then independent chunk by chunk.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "gdn.h"

namespace gdn {

constexpr int kSlice = 64;  // values of a head that are worked on together

struct SsmArgs {
    const void *x, *B, *C, *dy;
    const float *dt, *A, *D, *bias;
    const int* cu;
    const float *h0, *dhT;
    void* y;
    float *hT, *dh0;
    void *dx, *dB, *dC;
    float *ddt, *dA, *dD, *dbias;
    long long xs, bs, cs;  // elements between tokens of x, B, C
};

// How a call is laid out, from its sizes alone (the lengths are device data).
struct SsmPlan {
    int L;              // tokens of a chunk
    int slices;         // H P / 64
    int pairs;          // of slices in a group, the last of which may lack its second
    long long chunks;   // at most, over all sequences
    long long between;  // states between chunks, at most
    int seg;            // chunks of a segment; 0: a sequence is one segment
    long long segs;     // at most, over all sequences
    long long several;  // at most, of sequences that have several
    int splits;         // parts into which the heads of a group are dealt in the gradients
    size_t dec_at, seg_at, tot_at, fwd_at, back_at, token_at, sum_at, part_at, bytes;  // offsets in the workspace
};
SsmPlan ssm_plan(const gdn_ssm_shape& s, bool backward);  // ssm_plan.hip

// The most elements between two tokens of x, B or C.  The walk addresses the rows of half
// a chunk, and the other kernels runs of 16, with 32-bit byte offsets from their first.
constexpr long long kMostStride = 1LL << 24;

// The decays of every chunk and head; the walk over the chunks (states between them,
// and the last one into hT; for the gradients forward and backward, and dh0).
gdn_status ssm_prep(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& a, char* ws, hipStream_t st);
gdn_status ssm_walk(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& a, bool backward, char* ws, hipStream_t st);
gdn_status ssm_out(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& a, char* ws, hipStream_t st);
gdn_status ssm_grad(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& a, char* ws, hipStream_t st);
// the gradients of dt, A, D and dt_bias, behind ssm_grad
gdn_status ssm_finish(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& a, char* ws, hipStream_t st);
gdn_status ssm_step(const gdn_ssm_shape& s, const SsmArgs& a, float* state, hipStream_t st);

}  // namespace gdn
