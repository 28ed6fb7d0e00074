// mixer_api.hip -- the C ABI of the state-space layer's operators and of the page
// step (include/gdn.h): argument validation and dispatch of the short convolution
// (conv.hip), the selective state space scan (ssm_*.hip) and the pages (pages.hip).
// Nothing here allocates; every launch goes to the caller's stream.
#include <stdint.h>

#include "common.h"
#include "conv.h"
#include "pages.h"
#include "ssm.h"

using namespace gdn;

namespace {

bool off16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

template <typename... P> bool any_null(P... p) { return (... || (p == nullptr)); }
template <typename... P> bool any_of(const void* x, P... p) { return (... || (x == (const void*)p)); }
template <typename... P> bool any_off16(P... p) { return (... || off16((const void*)p)); }
template <typename... P> bool any_off4(P... p) { return (... || off4((const void*)p)); }

gdn_status check_conv(const gdn_conv_shape* sh, bool step, gdn_conv_shape& s)
{
    if (!sh) return GDN_ERR_INVALID_ARG;
    s = *sh;
    if (s.B < 1 || s.T < 0 || s.C < 1 || s.x_stride < 0) return GDN_ERR_INVALID_ARG;
    if (s.dtype != GDN_F32 && s.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (s.silu != 0 && s.silu != 1) return GDN_ERR_INVALID_ARG;
    if (step && s.T != s.B) return GDN_ERR_INVALID_ARG;
    if (s.W < 2 || s.W > 4) return GDN_ERR_UNSUPPORTED;
    const int ve = s.dtype == GDN_BF16 ? 8 : 4;
    // launches below 2^32 work-items, 4 sequences or 4 strips of 8 tokens or more (32
    // where there are many) a workgroup of 256, and rows of all channels in y
    if (s.C % ve || s.C > (1 << 20) || s.T > (1 << 28) || s.B > (1 << 25)) return GDN_ERR_UNSUPPORTED;
    if (!step && s.B > 65536) return GDN_ERR_UNSUPPORTED;  // every strip looks for its sequence along the bounds
    if (!s.x_stride) s.x_stride = s.C;
    if (s.x_stride < s.C) return GDN_ERR_INVALID_ARG;
    if (s.x_stride % ve) return GDN_ERR_ALIGNMENT;
    return GDN_OK;
}

size_t conv_ws(const gdn_conv_shape& s)
{
    const size_t n = (size_t)conv_partials(s) * (s.W + 1) * s.C * sizeof(float);
    return n < 256 ? 256 : n;
}

enum SsmCall { CALL_FORWARD, CALL_BACKWARD, CALL_STEP };

gdn_status check_ssm(const gdn_ssm_shape* sh, SsmCall call, gdn_ssm_shape& s)
{
    if (!sh) return GDN_ERR_INVALID_ARG;
    s = *sh;
    if (s.B < 1 || s.T < 0 || s.H < 1 || s.G < 1 || s.N < 1 || s.P < 1) return GDN_ERR_INVALID_ARG;
    if (s.H % s.G) return GDN_ERR_INVALID_ARG;
    if (s.dtype != GDN_F32 && s.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (s.softplus != 0 && s.softplus != 1) return GDN_ERR_INVALID_ARG;
    if (call == CALL_STEP && s.T != s.B) return GDN_ERR_INVALID_ARG;
    if ((s.N != 64 && s.N != 128) || (s.P != 64 && s.P != 128)) return GDN_ERR_UNSUPPORTED;
    // 32-bit launches: heads of one token, token-heads and sequence-heads of one call
    if (s.H > 1024 || (long long)s.T * s.H >= (1LL << 27) || (long long)s.B * s.H >= (1LL << 23)) return GDN_ERR_UNSUPPORTED;
    const long long e = s.dtype == GDN_BF16 ? 2 : 4, row[3] = {(long long)s.H * s.P, (long long)s.G * s.N, (long long)s.G * s.N};
    long long* st[3] = {&s.x_stride, &s.b_stride, &s.c_stride};
    for (int i = 0; i < 3; ++i) {
        if (!*st[i]) *st[i] = row[i];
        if (*st[i] < row[i]) return GDN_ERR_INVALID_ARG;
        if ((*st[i] * e) % 16) return GDN_ERR_ALIGNMENT;
        if (*st[i] > kMostStride) return GDN_ERR_UNSUPPORTED;
    }
    if (call != CALL_STEP) {
        // every workgroup looks for its chunk along the bounds, 64 sequences at a time
        if (s.B > 65536) return GDN_ERR_UNSUPPORTED;
        // below 2^32 work-items: 512 a chunk (or segment) and slice or part, in whole
        // eights of chunks and 32s of workgroups a die
        const SsmPlan p = ssm_plan(s, call == CALL_BACKWARD);
        const long long most = p.chunks > p.segs ? p.chunks : p.segs;
        const long long jobs = p.slices > s.G * p.splits ? p.slices : s.G * p.splits;
        if ((most + 8) * jobs + 256 >= (1LL << 23)) return GDN_ERR_UNSUPPORTED;
    }
    return GDN_OK;
}

gdn_status check_pages(const gdn_pages_shape* sh, gdn_pages_shape& s)
{
    if (!sh) return GDN_ERR_INVALID_ARG;
    s = *sh;
    if (s.B < 1 || s.num_pages < 1 || s.max_pages < 1 || s.page_size < 1 || s.rows < 0) return GDN_ERR_INVALID_ARG;
    if (s.page_size < 16 || s.page_size > 1024 || (s.page_size & (s.page_size - 1))) return GDN_ERR_UNSUPPORTED;
    if ((long long)s.max_pages * s.page_size > (1LL << 30)) return GDN_ERR_UNSUPPORTED;
    if (s.B > 8192) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_conv_workspace_bytes(const gdn_conv_shape* sh)
{
    gdn_conv_shape s;
    return check_conv(sh, false, s) == GDN_OK ? conv_ws(s) : 0;
}

gdn_status gdn_conv_forward(const gdn_conv_shape* sh, const void* x, const float* weight, const float* bias,
                            const int* cu_seqlens, const void* state, void* y, void* state_out, void* stream)
{
    gdn_conv_shape s;
    gdn_status r = check_conv(sh, false, s);
    if (r != GDN_OK) return r;
    if (any_null(weight) || !cu_seqlens) return GDN_ERR_INVALID_ARG;
    if (s.T && (any_null(x, (const void*)y) || x == y)) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, weight, bias, state, y, state_out) || off4(cu_seqlens)) return GDN_ERR_ALIGNMENT;
    ConvArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.cu = cu_seqlens; a.state = state; a.y = y; a.state_out = state_out;
    a.x_stride = s.x_stride; a.B = s.B; a.T = s.T; a.C = s.C; a.silu = s.silu;
    return conv_forward_dispatch(s, a, (hipStream_t)stream);
}

gdn_status gdn_conv_backward(const gdn_conv_shape* sh, const void* x, const float* weight, const float* bias,
                             const int* cu_seqlens, const void* state, const void* dy, const void* dstate_out, void* dx,
                             float* dweight, float* dbias, void* dstate, void* ws, size_t ws_bytes, void* stream)
{
    gdn_conv_shape s;
    gdn_status r = check_conv(sh, false, s);
    if (r != GDN_OK) return r;
    if (any_null(weight, (const float*)dweight) || !cu_seqlens) return GDN_ERR_INVALID_ARG;
    if (s.T && (any_null(x, dy, (const void*)dx) || x == dx || dy == dx)) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, weight, bias, state, dy, dstate_out, dx, dweight, dbias, dstate, ws) || off4(cu_seqlens))
        return GDN_ERR_ALIGNMENT;
    if (!ws || ws_bytes < conv_ws(s)) return GDN_ERR_WORKSPACE;
    // the launch of dstate reads these behind the outputs that they would be, or behind
    // its own earlier rows
    if (dweight == weight || (dbias && dbias == bias) || (dstate && dstate == dstate_out)) return GDN_ERR_INVALID_ARG;
    ConvArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.cu = cu_seqlens; a.state = state;
    a.dy = dy; a.dstate_out = dstate_out; a.dx = dx; a.dstate = dstate; a.part = (float*)ws;
    a.x_stride = s.x_stride; a.B = s.B; a.T = s.T; a.C = s.C; a.silu = s.silu;
    return conv_backward_dispatch(s, a, dweight, dbias, (hipStream_t)stream);
}

gdn_status gdn_conv_step(const gdn_conv_shape* sh, const void* x, const float* weight, const float* bias, void* state,
                         void* y, void* stream)
{
    gdn_conv_shape s;
    gdn_status r = check_conv(sh, true, s);
    if (r != GDN_OK) return r;
    if (any_null(x, (const void*)weight, (const void*)state, (const void*)y) || x == y) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, weight, bias, state, y)) return GDN_ERR_ALIGNMENT;
    ConvArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.state = state; a.state_out = state; a.y = y;
    a.x_stride = s.x_stride; a.B = s.B; a.T = s.T; a.C = s.C; a.silu = s.silu;
    return conv_forward_dispatch(s, a, (hipStream_t)stream);
}

size_t gdn_ssm_workspace_bytes(const gdn_ssm_shape* sh, int call)
{
    gdn_ssm_shape s;
    if (call != GDN_SSM_FORWARD && call != GDN_SSM_BACKWARD) return 0;
    const bool back = call == GDN_SSM_BACKWARD;
    return check_ssm(sh, back ? CALL_BACKWARD : CALL_FORWARD, s) == GDN_OK ? ssm_plan(s, back).bytes : 0;
}

gdn_status gdn_ssm_forward(const gdn_ssm_shape* sh, const void* x, const float* dt, const float* A, const void* B,
                           const void* C, const float* D, const float* dt_bias, const int* cu_seqlens, const float* h0,
                           void* y, float* hT, void* ws, size_t ws_bytes, void* stream)
{
    gdn_ssm_shape s;
    gdn_status r = check_ssm(sh, CALL_FORWARD, s);
    if (r != GDN_OK) return r;
    if (!A || !cu_seqlens) return GDN_ERR_INVALID_ARG;
    if (s.T && (any_null(x, B, C, (const void*)y) || !dt)) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, B, C, h0, y, hT, ws) || any_off4(dt, A, D, dt_bias) || off4(cu_seqlens)) return GDN_ERR_ALIGNMENT;
    const SsmPlan p = ssm_plan(s, false);
    if (!ws || ws_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    if (s.T && any_of(y, x, B, C)) return GDN_ERR_INVALID_ARG;  // another workgroup's operands
    SsmArgs a{};
    a.x = x; a.B = B; a.C = C; a.dt = dt; a.A = A; a.D = D; a.bias = dt_bias; a.cu = cu_seqlens;
    a.h0 = h0; a.y = y; a.hT = hT;
    a.xs = s.x_stride; a.bs = s.b_stride; a.cs = s.c_stride;
    r = ssm_prep(s, p, a, (char*)ws, (hipStream_t)stream);
    if (r != GDN_OK) return r;
    r = ssm_walk(s, p, a, false, (char*)ws, (hipStream_t)stream);
    if (r != GDN_OK || !s.T) return r;
    return ssm_out(s, p, a, (char*)ws, (hipStream_t)stream);
}

gdn_status gdn_ssm_backward(const gdn_ssm_shape* sh, const void* x, const float* dt, const float* A, const void* B,
                            const void* C, const float* D, const float* dt_bias, const int* cu_seqlens, const float* h0,
                            const void* dy, const float* dhT, void* dx, float* ddt, float* dA, void* dB, void* dC,
                            float* dD, float* ddt_bias, float* dh0, void* ws, size_t ws_bytes, void* stream)
{
    gdn_ssm_shape s;
    gdn_status r = check_ssm(sh, CALL_BACKWARD, s);
    if (r != GDN_OK) return r;
    if (!A || !cu_seqlens || !dA) return GDN_ERR_INVALID_ARG;
    if (s.T && (any_null(x, B, C, dy, (const void*)dx, (const void*)dB, (const void*)dC) || !dt || !ddt))
        return GDN_ERR_INVALID_ARG;
    if (any_off16(x, B, C, h0, dy, dhT, dx, dB, dC, dh0, ws) || any_off4(dt, A, D, dt_bias, ddt, dA, dD, ddt_bias) ||
        off4(cu_seqlens))
        return GDN_ERR_ALIGNMENT;
    const SsmPlan p = ssm_plan(s, true);
    if (!ws || ws_bytes < p.bytes) return GDN_ERR_WORKSPACE;
    // the gradients read h0 and dhT after the walk has written dh0, and one workgroup's
    // operands after another has written its results
    if (dh0 && (dhT == dh0 || h0 == dh0)) return GDN_ERR_INVALID_ARG;
    if (s.T && (any_of(dx, x, B, C, dy) || any_of(dB, x, B, C, dy, dx) || any_of(dC, x, B, C, dy, dx, dB)))
        return GDN_ERR_INVALID_ARG;
    SsmArgs a{};
    a.x = x; a.B = B; a.C = C; a.dy = dy; a.dt = dt; a.A = A; a.D = D; a.bias = dt_bias; a.cu = cu_seqlens;
    a.h0 = h0; a.dhT = dhT; a.dx = dx; a.dB = dB; a.dC = dC; a.ddt = ddt; a.dA = dA; a.dD = dD; a.dbias = ddt_bias; a.dh0 = dh0;
    a.xs = s.x_stride; a.bs = s.b_stride; a.cs = s.c_stride;
    r = ssm_prep(s, p, a, (char*)ws, (hipStream_t)stream);
    if (r != GDN_OK) return r;
    r = ssm_walk(s, p, a, true, (char*)ws, (hipStream_t)stream);
    if (r != GDN_OK) return r;
    r = ssm_grad(s, p, a, (char*)ws, (hipStream_t)stream);
    if (r != GDN_OK) return r;
    return ssm_finish(s, p, a, (char*)ws, (hipStream_t)stream);
}

gdn_status gdn_ssm_step(const gdn_ssm_shape* sh, const void* x, const float* dt, const float* A, const void* B,
                        const void* C, const float* D, const float* dt_bias, float* state, void* y, void* stream)
{
    gdn_ssm_shape s;
    gdn_status r = check_ssm(sh, CALL_STEP, s);
    if (r != GDN_OK) return r;
    if (any_null(x, B, C, (const void*)y) || !dt || !A || !state) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, B, C, state, y) || any_off4(dt, A, D, dt_bias)) return GDN_ERR_ALIGNMENT;
    if (any_of(y, x, B, C)) return GDN_ERR_INVALID_ARG;
    SsmArgs a{};
    a.x = x; a.B = B; a.C = C; a.dt = dt; a.A = A; a.D = D; a.bias = dt_bias; a.y = y;
    a.xs = s.x_stride; a.bs = s.b_stride; a.cs = s.c_stride;
    return ssm_step(s, a, state, (hipStream_t)stream);
}

gdn_status gdn_pages_release(const gdn_pages_shape* sh, const int* done, const int* kv_len, const int* page_table,
                             int* free_pages, const int* free_count, int* kv_out, int* count_out, void* stream)
{
    gdn_pages_shape s;
    gdn_status r = check_pages(sh, s);
    if (r != GDN_OK) return r;
    if (any_null(done, kv_len, page_table, (const int*)free_pages, free_count, (const int*)kv_out, (const int*)count_out))
        return GDN_ERR_INVALID_ARG;
    if (any_off4(done, kv_len, page_table, free_pages, free_count, kv_out, count_out)) return GDN_ERR_ALIGNMENT;
    return pages_release_dispatch(s, done, kv_len, page_table, free_pages, free_count, kv_out, count_out, (hipStream_t)stream);
}

gdn_status gdn_pages_take(const gdn_pages_shape* sh, const int* want, const int* kv_len, int* page_table,
                          const int* free_pages, const int* free_count, int* kv_out, int* count_out, int* cu_seqlens,
                          int* positions, long long* slots, void* stream)
{
    gdn_pages_shape s;
    gdn_status r = check_pages(sh, s);
    if (r != GDN_OK) return r;
    if (any_null(want, kv_len, (const int*)page_table, free_pages, free_count, (const int*)kv_out, (const int*)count_out,
                 (const int*)cu_seqlens))
        return GDN_ERR_INVALID_ARG;
    if (any_off4(want, kv_len, page_table, free_pages, free_count, kv_out, count_out, cu_seqlens, positions) ||
        ((uintptr_t)slots & 7u))
        return GDN_ERR_ALIGNMENT;
    return pages_take_dispatch(s, want, kv_len, page_table, free_pages, free_count, kv_out, count_out, cu_seqlens, positions,
                               slots, (hipStream_t)stream);
}

}  // extern "C"
