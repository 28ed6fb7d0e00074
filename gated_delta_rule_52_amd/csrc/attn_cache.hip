// attn_cache.hip -- new keys and values into a paged cache (gdn_attn_append),
// keys and, where asked for, queries rotated by their position on the way:
//
//   x'_i = x_i cos_p,i - x_{i + R/2} sin_p,i,   x'_{i + R/2} = x_{i + R/2} cos_p,i + x_i sin_p,i
//
// for i < R / 2, R the rotated width (the rest of a head passes through), p the
// token's position in its sequence; fp32, rounded once.  Bound by HBM: q, k, v
// are read once and written once (17.7 thousand tokens of 16 + 2 x 4 heads of 128,
// bf16, 297 MB: 51 us a pass on data that no cache holds, 5.9 TB/s); single tokens
// are bound by the launch (256 tokens: 4.0 us).
#include "attn.h"

namespace gdn {

namespace {

struct AppendArgs {
    const void *q, *k, *v;
    const float *cos, *sin;
    const int *cu, *kv_len, *table;
    void *kc, *vc, *qo;
    long long q_stride, k_stride, v_stride;
    int B, T, Hq, Hkv, D;
    int num_pages, page_shift, max_pages, rot, max_pos;
};

template <typename T> __device__ __forceinline__ u32x4 load_word(const T* p) { return *reinterpret_cast<const u32x4*>(p); }
// PAST: not to be kept in the L2
template <bool PAST, typename T> __device__ __forceinline__ void store_word(T* p, u32x4 w)
{
    if constexpr (PAST)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<u32x4*>(p) = w;
}

__device__ __forceinline__ void rotate(u32x4& a, u32x4& b, const float* c, const float* s, bf16)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = __uint_as_float(a[i] << 16), a1 = __uint_as_float(a[i] & 0xffff0000u);
        const float b0 = __uint_as_float(b[i] << 16), b1 = __uint_as_float(b[i] & 0xffff0000u);
        const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
        a[i] = cvt2_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
        b[i] = cvt2_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
    }
}
__device__ __forceinline__ void rotate(u32x4& a, u32x4& b, const float* c, const float* s, float)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = __uint_as_float(a[i]), b0 = __uint_as_float(b[i]);
        a[i] = __float_as_uint(a0 * c[i] - b0 * s[i]);
        b[i] = __float_as_uint(b0 * c[i] + a0 * s[i]);
    }
}

// TPB tokens a workgroup; one wave finds a token's sequence and slot (the
// number of sequence ends at or before it, counted 64 at a time), then all
// threads take (token, head, word pair) items.
template <typename T, int TPB, bool PAST>
__global__ __launch_bounds__(256) void attn_append_kernel(AppendArgs a)
{
    constexpr int VE = 16 / (int)sizeof(T);
    __shared__ int pos_s[TPB];
    __shared__ long long slot_s[TPB];
    const int w = uniform(wave_id()), l = lane_id();
    for (int i = w; i < TPB; i += 4) {
        const int tok = blockIdx.x * TPB + i;
        int pos = -1;
        long long slot = -1;
        if (tok < a.T) {
            int b = 0;
            for (int b0 = 0; b0 < a.B; b0 += 64) {
                const int e = b0 + l < a.B ? a.cu[b0 + l + 1] : 0x7fffffff;
                b += __popcll(__ballot(e <= tok));
            }
            if (b < a.B) {
                // clamped as in the attention, so that both count a sequence's tokens alike
                int st = a.cu[b], en = a.cu[b + 1];
                st = st < 0 ? 0 : st;
                en = en > a.T ? a.T : en;
                if (tok >= st) {
                    const long long p = (long long)a.kv_len[b] - en + tok;  // kv_len - n + (tok - st)
                    if (p >= 0 && p < a.max_pos && p < ((long long)a.max_pages << a.page_shift)) {
                        pos = (int)p;
                        const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
                        if (page >= 0 && page < a.num_pages)
                            slot = ((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
                    }
                }
            }
        }
        if (l == 0) {
            pos_s[i] = pos;
            slot_s[i] = slot;
        }
    }
    __syncthreads();
    const int pairs = a.D / VE / 2, turned = a.rot / VE / 2;
    const int hq = a.qo ? a.Hq : 0;
    const int per = (hq + 2 * a.Hkv) * pairs;
    for (int x = threadIdx.x; x < TPB * per; x += 256) {
        const int i = x / per, y = x - i * per, hd = y / pairs, j = y - hd * pairs;
        const int pos = pos_s[i];
        const long long slot = slot_s[i];
        const size_t tok = (size_t)blockIdx.x * TPB + i;
        if (pos < 0) continue;  // no sequence's token, or no place for its position
        const bool rot = j < turned;
        const int at = rot ? j * VE : a.rot + (j - turned) * 2 * VE;
        const int gap = rot ? a.rot / 2 : VE;
        const T* src;
        T* dst;
        if (hd < hq) {
            src = (const T*)a.q + tok * a.q_stride + (size_t)hd * a.D;
            dst = (T*)a.qo + (tok * a.Hq + hd) * a.D;
        } else {
            if (slot < 0) continue;  // the table has no page for it
            const int kv = hd - hq, hh = kv < a.Hkv ? kv : kv - a.Hkv;
            src = kv < a.Hkv ? (const T*)a.k + tok * a.k_stride : (const T*)a.v + tok * a.v_stride;
            dst = (kv < a.Hkv ? (T*)a.kc : (T*)a.vc) + ((size_t)slot * a.Hkv + hh) * a.D;
            src += (size_t)hh * a.D;
        }
        u32x4 u = load_word(src + at), v = load_word(src + at + gap);
        if (rot && hd < hq + a.Hkv) {
            float c[VE], s[VE];
            const size_t p = (size_t)pos * (a.rot / 2) + at;
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                *reinterpret_cast<f32x4*>(c + e) = *reinterpret_cast<const f32x4*>(a.cos + p + e);
                *reinterpret_cast<f32x4*>(s + e) = *reinterpret_cast<const f32x4*>(a.sin + p + e);
            }
            rotate(u, v, c, s, T{});
        }
        store_word<PAST>(dst + at, u);
        store_word<PAST>(dst + at + gap, v);
    }
}

template <typename T>
gdn_status launch(const AppendArgs& a, hipStream_t st)
{
    // A workgroup a token while there are at most eight for a compute unit; then two
    // tokens share one, which few heads need (65536 tokens of one head of 64: 26 us,
    // one a workgroup 42) and many do not mind (17.7 thousand of 24 heads of 128: 35
    // and 33 us on warm caches, on cold ones 51.5 and 50.7, four a workgroup 54).
    // Where they write more than the L2 holds (4 MB on each of 8 dies), it is not kept
    // there (192 MB: 59 us, kept 71 us; with the attention that then reads it 624 and
    // 621 us).  Up to there it is kept: this kernel takes longer (24 MB: 9.9 us, not kept
    // 8.1) and the attention gains more (62.4 us together, not kept 63.8).
    const long long words = (long long)a.T * ((a.qo ? a.Hq : 0) + 2 * a.Hkv) * a.D;
    if (a.T <= 2048)
        GDN_LAUNCH("attn_append", (attn_append_kernel<T, 1, false>), dim3(a.T), dim3(256), st, a);
    else if (words * (long long)sizeof(T) <= (32LL << 20))
        GDN_LAUNCH("attn_append", (attn_append_kernel<T, 2, false>), dim3((a.T + 1) / 2), dim3(256), st, a);
    else
        GDN_LAUNCH("attn_append", (attn_append_kernel<T, 2, true>), dim3((a.T + 1) / 2), dim3(256), st, a);
    return GDN_OK;
}

}  // namespace

gdn_status attn_append_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const float* cos,
                                const float* sin, const int* cu, const int* kv_len, const int* table, void* k_cache,
                                void* v_cache, void* q_out, hipStream_t st)
{
    AppendArgs a{};
    a.q = q; a.k = k; a.v = v; a.cos = cos; a.sin = sin;
    a.cu = cu; a.kv_len = kv_len; a.table = table;
    a.kc = k_cache; a.vc = v_cache; a.qo = q_out;
    a.q_stride = s.q_stride; a.k_stride = s.k_stride; a.v_stride = s.v_stride;
    a.B = s.B; a.T = s.T; a.Hq = s.Hq; a.Hkv = s.Hkv; a.D = s.D;
    a.num_pages = s.num_pages; a.page_shift = __builtin_ctz((unsigned)s.page_size); a.max_pages = s.max_pages;
    a.rot = s.rot_dim; a.max_pos = s.max_pos;
    return s.dtype == GDN_BF16 ? launch<bf16>(a, st) : launch<float>(a, st);
}

}  // namespace gdn
