// block_api.hip -- the C ABI of the operators around the layer (include/gdn.h):
// argument validation and dispatch of the block norms (norm.hip) and of softmax
// attention (attn_*.hip).  Nothing here allocates; every launch goes to the
// caller's stream.
#include <stdint.h>

#include "attn_plan.h"
#include "common.h"
#include "norm.h"

using namespace gdn;

namespace {

bool off16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

template <typename... P> bool any_null(P... p) { return (... || (p == nullptr)); }
template <typename... P> bool any_off16(P... p) { return (... || off16((const void*)p)); }
template <typename... P> bool any_off4(P... p) { return (... || off4((const void*)p)); }

// Validate a norm's shape and fill in the dense gate stride.
gdn_status check_norm(const gdn_norm_shape* sh, bool gate, gdn_norm_shape& out)
{
    if (!sh) return GDN_ERR_INVALID_ARG;
    out = *sh;
    if (sh->tokens < 0 || sh->heads < 1 || sh->width < 1 || sh->gate_stride < 0) return GDN_ERR_INVALID_ARG;
    if (sh->dtype != GDN_F32 && sh->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (!(sh->eps > 0.f && sh->eps <= 1.f)) return GDN_ERR_INVALID_ARG;  // also NaN
    const int ve = sh->dtype == GDN_BF16 ? 8 : 4;
    // work-items of the largest launch (a workgroup of 256 a row at most) below
    // 2^32 by the launches' own caps; row indices and strides in int
    if ((long long)sh->tokens * sh->heads > (1LL << 29)) return GDN_ERR_UNSUPPORTED;
    if (gate) {
        if (sh->width != 16 && sh->width != 32 && sh->width != 64 && sh->width != 128) return GDN_ERR_UNSUPPORTED;
        const long long dense = (long long)sh->heads * sh->width;
        if (!out.gate_stride) out.gate_stride = dense;
        if (out.gate_stride < dense) return GDN_ERR_INVALID_ARG;
        if (out.gate_stride % ve) return GDN_ERR_ALIGNMENT;
    } else {
        if (sh->heads != 1 || sh->gate_stride != 0) return GDN_ERR_INVALID_ARG;
        if (sh->width % ve || sh->width > 2048 * ve) return GDN_ERR_UNSUPPORTED;
    }
    return GDN_OK;
}

size_t norm_ws(const gdn_norm_shape& s, bool gate)
{
    const size_t n = (size_t)(gate ? 1 : 2) * norm_partials(s, gate) * s.width * sizeof(float);
    return n < 256 ? 256 : n;
}

enum AttnCall { CALL_PROMPT, CALL_BACKWARD, CALL_PAGED, CALL_APPEND };

// Validate an attention shape and fill in the defaults.
gdn_status check_attn(const gdn_attn_shape* sh, AttnCall call, gdn_attn_shape& s)
{
    if (!sh) return GDN_ERR_INVALID_ARG;
    s = *sh;
    if (s.B < 1 || s.T < 0 || s.Hq < 1 || s.Hkv < 1 || s.D < 1) return GDN_ERR_INVALID_ARG;
    if (s.Hq % s.Hkv) return GDN_ERR_INVALID_ARG;
    if (s.dtype != GDN_F32 && s.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (!(s.scale >= 0.f && s.scale <= 1e30f)) return GDN_ERR_INVALID_ARG;  // also NaN
    if (s.D != 64 && s.D != 128) return GDN_ERR_UNSUPPORTED;
    if (s.scale == 0.f) s.scale = 1.0f / sqrtf((float)s.D);
    // heads and rows of one call: 32-bit row indices and launches below 2^32 work-items
    if (s.Hq > 1024 || (long long)s.T * s.Hq >= (1LL << 27)) return GDN_ERR_UNSUPPORTED;
    const long long e = s.dtype == GDN_BF16 ? 2 : 4, hd[3] = {s.Hq, s.Hkv, s.Hkv};
    long long* st[3] = {&s.q_stride, &s.k_stride, &s.v_stride};
    for (int i = 0; i < 3; ++i) {
        if (!*st[i]) *st[i] = hd[i] * s.D;
        if (*st[i] < hd[i] * s.D) return GDN_ERR_INVALID_ARG;
        if ((*st[i] * e) % 16) return GDN_ERR_ALIGNMENT;
        // a run of 16 token rows is addressed with 32-bit offsets from its first
        if (*st[i] > (1LL << 24)) return GDN_ERR_UNSUPPORTED;
    }
    if (call == CALL_PAGED || call == CALL_APPEND) {
        if (s.num_pages < 1 || s.max_pages < 1 || s.page_size < 1) return GDN_ERR_INVALID_ARG;
        if (s.page_size < 16 || s.page_size > 1024 || (s.page_size & (s.page_size - 1))) return GDN_ERR_UNSUPPORTED;
        if ((long long)s.max_pages * s.page_size > (1LL << 30)) return GDN_ERR_UNSUPPORTED;
    }
    if (call == CALL_APPEND) {
        if (s.rot_dim < 0 || s.rot_dim > s.D || s.rot_dim % 16) return GDN_ERR_INVALID_ARG;
        if (s.rot_dim && s.max_pos < 1) return GDN_ERR_INVALID_ARG;
        if (!s.rot_dim) s.max_pos = 0x7fffffff;
        // two tokens a workgroup of 256, below 2^32 work-items
        if (s.T > (1 << 25) - 2) return GDN_ERR_UNSUPPORTED;
    } else {
        const AttnPlan p = attn_plan(s, call == CALL_PAGED);
        if (p.jobs * s.Hkv >= (1LL << 24)) return GDN_ERR_UNSUPPORTED;
        if (call == CALL_BACKWARD && !attn_backward_fits(s)) return GDN_ERR_UNSUPPORTED;
    }
    return GDN_OK;
}

size_t at_least_256(size_t n) { return n < 256 ? 256 : n; }

}  // namespace

extern "C" {

size_t gdn_norm_workspace_bytes(const gdn_norm_shape* sh, int gate)
{
    gdn_norm_shape s;
    if (check_norm(sh, gate != 0, s) != GDN_OK) return 0;
    return norm_ws(s, gate != 0);
}

gdn_status gdn_norm_block(const gdn_norm_shape* sh, const void* x, const void* y, const float* res_scale,
                          const float* weight, void* h, void* n, float* rstd, void* stream)
{
    gdn_norm_shape s;
    gdn_status r = check_norm(sh, false, s);
    if (r != GDN_OK) return r;
    if (s.tokens == 0) return GDN_OK;
    if (res_scale && !y) return GDN_ERR_INVALID_ARG;
    if (any_null(x, (const void*)weight, (const void*)n)) return GDN_ERR_INVALID_ARG;
    if (any_off16(x, y, res_scale, weight, h, n) || off4(rstd)) return GDN_ERR_ALIGNMENT;
    return norm_block_dispatch(s, x, y, res_scale, weight, h, n, rstd, (hipStream_t)stream);
}

gdn_status gdn_norm_block_backward(const gdn_norm_shape* sh, const void* dn, const void* dh, const void* x,
                                   const void* y, const float* res_scale, const float* weight, const float* rstd,
                                   void* dx, void* dy, float* dweight, float* dres_scale, void* ws, size_t ws_bytes,
                                   void* stream)
{
    gdn_norm_shape s;
    gdn_status r = check_norm(sh, false, s);
    if (r != GDN_OK) return r;
    // with no rows the rows' pointers may be anything; the sums are still written
    if (!dweight || (res_scale && !dres_scale)) return GDN_ERR_INVALID_ARG;
    if (s.tokens && (any_null(dn, x, (const void*)weight, (const void*)rstd, (const void*)dx) ||
                     (res_scale && (!y || !dy))))
        return GDN_ERR_INVALID_ARG;
    if (any_off16(dn, dh, x, y, res_scale, weight, dx, dy, dweight, dres_scale, ws) || off4(rstd))
        return GDN_ERR_ALIGNMENT;
    if (!ws || ws_bytes < norm_ws(s, false)) return GDN_ERR_WORKSPACE;
    return norm_block_bwd_dispatch(s, dn, dh, x, y, res_scale, weight, rstd, dx, dy, dweight, dres_scale, (float*)ws,
                                   (hipStream_t)stream);
}

gdn_status gdn_norm_gate(const gdn_norm_shape* sh, const void* o, const void* gate, const float* weight, void* y,
                         float* rstd, void* stream)
{
    gdn_norm_shape s;
    gdn_status r = check_norm(sh, true, s);
    if (r != GDN_OK) return r;
    if (s.tokens == 0) return GDN_OK;
    if (any_null(o, gate, (const void*)weight, (const void*)y)) return GDN_ERR_INVALID_ARG;
    if (any_off16(o, gate, weight, y) || off4(rstd)) return GDN_ERR_ALIGNMENT;
    return norm_gate_dispatch(s, o, gate, weight, y, rstd, (hipStream_t)stream);
}

gdn_status gdn_norm_gate_backward(const gdn_norm_shape* sh, const void* dy, const void* o, const void* gate,
                                  const float* weight, const float* rstd, void* dO, void* dgate, float* dweight,
                                  void* ws, size_t ws_bytes, void* stream)
{
    gdn_norm_shape s;
    gdn_status r = check_norm(sh, true, s);
    if (r != GDN_OK) return r;
    if (!dweight) return GDN_ERR_INVALID_ARG;
    if (s.tokens && any_null(dy, o, gate, (const void*)weight, (const void*)rstd, (const void*)dO, (const void*)dgate))
        return GDN_ERR_INVALID_ARG;
    if (any_off16(dy, o, gate, weight, dO, dgate, dweight, ws) || off4(rstd)) return GDN_ERR_ALIGNMENT;
    if (!ws || ws_bytes < norm_ws(s, true)) return GDN_ERR_WORKSPACE;
    return norm_gate_bwd_dispatch(s, dy, o, gate, weight, rstd, dO, dgate, dweight, (float*)ws, (hipStream_t)stream);
}

size_t gdn_attn_workspace_bytes(const gdn_attn_shape* sh, int call)
{
    gdn_attn_shape s;
    if (call == GDN_ATTN_PAGED)
        return check_attn(sh, CALL_PAGED, s) == GDN_OK ? at_least_256(attn_plan(s, true).ws_bytes) : 0;
    if (call == GDN_ATTN_BACKWARD)
        return check_attn(sh, CALL_BACKWARD, s) == GDN_OK ? at_least_256(attn_backward_ws(s)) : 0;
    return 0;
}

gdn_status gdn_attn_forward(const gdn_attn_shape* sh, const void* q, const void* k, const void* v,
                            const int* cu_seqlens, void* o, float* lse, void* stream)
{
    gdn_attn_shape s;
    gdn_status r = check_attn(sh, CALL_PROMPT, s);
    if (r != GDN_OK) return r;
    if (s.T == 0) return GDN_OK;
    if (any_null(q, k, v, (const void*)cu_seqlens, (const void*)o)) return GDN_ERR_INVALID_ARG;
    if (any_off16(q, k, v, o) || any_off4(cu_seqlens, lse)) return GDN_ERR_ALIGNMENT;
    return attn_forward_dispatch(s, q, k, v, cu_seqlens, nullptr, nullptr, o, lse, nullptr, false,
                                 (hipStream_t)stream);
}

gdn_status gdn_attn_backward(const gdn_attn_shape* sh, const void* q, const void* k, const void* v,
                             const int* cu_seqlens, const void* o, const float* lse, const void* dO, void* dq,
                             void* dk, void* dv, void* ws, size_t ws_bytes, void* stream)
{
    gdn_attn_shape s;
    gdn_status r = check_attn(sh, CALL_BACKWARD, s);
    if (r != GDN_OK) return r;
    if (s.T == 0) return GDN_OK;
    if (any_null(q, k, v, (const void*)cu_seqlens, o, (const void*)lse, dO, (const void*)dq, (const void*)dk,
                 (const void*)dv))
        return GDN_ERR_INVALID_ARG;
    if (any_off16(q, k, v, o, dO, dq, dk, dv, ws) || any_off4(cu_seqlens, lse)) return GDN_ERR_ALIGNMENT;
    if (!ws || ws_bytes < attn_backward_ws(s)) return GDN_ERR_WORKSPACE;
    return attn_backward_dispatch(s, q, k, v, cu_seqlens, o, lse, dO, dq, dk, dv, ws, (hipStream_t)stream);
}

gdn_status gdn_attn_append(const gdn_attn_shape* sh, const void* q, const void* k, const void* v, const float* cos,
                           const float* sin, const int* cu_seqlens, const int* kv_len, const int* page_table,
                           void* k_cache, void* v_cache, void* q_out, void* stream)
{
    gdn_attn_shape s;
    gdn_status r = check_attn(sh, CALL_APPEND, s);
    if (r != GDN_OK) return r;
    if ((q == nullptr) != (q_out == nullptr)) return GDN_ERR_INVALID_ARG;
    if (s.T == 0) return GDN_OK;
    if (any_null(k, v, (const void*)cu_seqlens, (const void*)kv_len, (const void*)page_table, (const void*)k_cache,
                 (const void*)v_cache))
        return GDN_ERR_INVALID_ARG;
    if (s.rot_dim && any_null(cos, sin)) return GDN_ERR_INVALID_ARG;
    if (any_off16(q, k, v, cos, sin, k_cache, v_cache, q_out) || any_off4(cu_seqlens, kv_len, page_table))
        return GDN_ERR_ALIGNMENT;
    return attn_append_dispatch(s, q, k, v, cos, sin, cu_seqlens, kv_len, page_table, k_cache, v_cache, q_out,
                                (hipStream_t)stream);
}

gdn_status gdn_attn_paged(const gdn_attn_shape* sh, const void* q, const void* k_cache, const void* v_cache,
                          const int* page_table, const int* cu_seqlens, const int* kv_len, void* o, void* ws,
                          size_t ws_bytes, void* stream)
{
    gdn_attn_shape s;
    gdn_status r = check_attn(sh, CALL_PAGED, s);
    if (r != GDN_OK) return r;
    if (s.T == 0) return GDN_OK;
    if (any_null(q, k_cache, v_cache, (const void*)page_table, (const void*)cu_seqlens, (const void*)kv_len,
                 (const void*)o))
        return GDN_ERR_INVALID_ARG;
    if (any_off16(q, k_cache, v_cache, o, ws) || any_off4(page_table, cu_seqlens, kv_len)) return GDN_ERR_ALIGNMENT;
    const size_t need = attn_plan(s, true).ws_bytes;
    if (need && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    return attn_forward_dispatch(s, q, k_cache, v_cache, cu_seqlens, kv_len, page_table, o, nullptr, ws, true,
                                 (hipStream_t)stream);
}

}  // extern "C"
