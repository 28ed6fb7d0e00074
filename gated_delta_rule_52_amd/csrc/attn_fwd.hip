// attn_fwd.hip -- causal softmax attention with grouped heads: packed prompts
// (gdn_attn_forward) and new tokens over a paged cache (gdn_attn_paged).
//
//   o_i = sum_{j <= i} p_ij v_j,  p_ij = exp(scale q_i . k_j - lse_i),
//   lse_i = log sum_{j <= i} exp(scale q_i . k_j);  o_i = 0 where no key is seen.
//
// One pass over the keys with a running maximum and sum, both fp32 and held per
// query row.  The G = Hq / Hkv query heads of one key head are rows of the same
// block (row = token * G + head), so a key is read once for all of them, for
// single tokens too.
#include "attn.h"

namespace gdn {

namespace {

struct FwdArgs {
    const void *q, *k, *v;
    void* o;
    float* lse;
    const int *cu, *kv_len, *table;
    long long q_stride;           // elements between tokens of q
    uint32_t k_bytes, v_bytes;    // bytes between tokens of k and v (slots of the cache)
    int B, T, Hq, Hkv, G;
    int num_pages, page_shift, max_pages;
    int splits;
    float scale;
    float *part_o, *part_l;
};

// What a wave keeps of its 32 query rows: lane l is row l % 32 in both halves.
template <typename T, int D>
struct Queries {
    static constexpr int KK = D / 16, DT = D / 32;
    Frag<T> q[KK];
    f32x16 o[DT];
    float m, l;   // running maximum of the raw scores; sum of this lane's own keys
    int limit;    // keys [0, limit) are seen

    __device__ __forceinline__ void load(const T* row)
    {
        const int h = lane_id() >> 5;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) q[kk] = load_frag<T>(row + 16 * kk + 8 * h);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = zero16();
        m = -INFINITY;
        l = 0.f;
    }

    // NK * 32 keys of the tables from row r0; key0 is the position of the first.
    // MASK: some key may lie behind some row's limit, or `gone` (a bit for each
    // run of CH keys) says that it is absent.
    template <int NK, bool MASK, int CH>
    __device__ __forceinline__ void step(const void* ktab, const void* vtab, int r0, int key0, unsigned gone, float sl2)
    {
        const int h = lane_id() >> 5;
        f32x16 s[NK];
#pragma unroll
        for (int t = 0; t < NK; ++t) s[t] = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int t = 0; t < NK; ++t) s[t] = mma32(Rows<T, D>::along(ktab, r0 + 32 * t, kk), q[kk], s[t]);
        if (MASK) {
#pragma unroll
            for (int t = 0; t < NK; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int key = 32 * t + 8 * (r >> 2) + 4 * h + (r & 3);
                    // CH >= 8: the four rows of a register group lie in one run
                    const bool out = key0 + key >= limit || ((gone >> ((32 * t + 8 * (r >> 2)) / CH)) & 1);
                    s[t][r] = out ? -INFINITY : s[t][r];
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[t][r]);
        mx = half_max(mx);
        // The maximum is moved, and what was summed rescaled, only when it grew
        // by more than 2^8: until then the exponentials stay below 256, which
        // costs neither bf16 nor fp32 any relative precision.
        if (__any(mx * sl2 > m * sl2 + 8.f || (m == -INFINITY && mx > m))) {
            const float mn = fmaxf(m, mx);
            const float al = mn == -INFINITY ? 1.f : exp2_hw((m - mn) * sl2);
            m = mn;
            l *= al;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[dt][r] *= al;
        }
        const float off = m == -INFINITY ? 0.f : m * sl2;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[t][r] = exp2_hw(s[t][r] * sl2 - off);
                sum += s[t][r];
            }
        l += sum;
        // The operand of the second product is rounded to the inputs' type: half
        // a step of bf16 a key, against the half step of the stored output; the
        // sum above takes the unrounded values.
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const Frag<T> p = acc_frag<T>(s[t], b);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt)
                    o[dt] = mma32(Rows<T, D>::down(vtab, r0 + 32 * t + 16 * b, 32 * dt), p, o[dt]);
            }
    }
};

// The keys of one (sequence, key head): where run `c` of CH keys lies.
template <typename T, int D, bool PAGED, int CH>
struct Keys {
    const char *k, *v;
    int len;    // keys there are
    int first;  // position of the sequence's first new token (negative: more new tokens than positions)
    const int* __restrict__ pages;

    __device__ __forceinline__ Keys(const FwdArgs& a, const Span& s, int hk)
    {
        if (PAGED) {
            int n = uniform(a.kv_len[s.b]);
            const long long cap = (long long)a.max_pages << a.page_shift;
            n = n < 0 ? 0 : n > (1 << 30) ? 1 << 30 : n;
            len = n > cap ? (int)cap : n;
            first = n - s.n;
            pages = a.table + (size_t)s.b * a.max_pages;
            k = (const char*)a.k + (size_t)hk * D * sizeof(T);
            v = (const char*)a.v + (size_t)hk * D * sizeof(T);
        } else {
            len = s.n;
            first = 0;
            pages = nullptr;
            k = (const char*)a.k + (size_t)s.start * a.k_bytes + (size_t)hk * D * sizeof(T);
            v = (const char*)a.v + (size_t)s.start * a.v_bytes + (size_t)hk * D * sizeof(T);
        }
    }
    // keys that new token `tok` sees
    __device__ __forceinline__ int seen(int tok) const
    {
        const int n = first + tok + 1;
        return n < 0 ? 0 : n < len ? n : len;
    }
    // page of the run that starts at key `key` (of the last key where it starts behind the end), -1: none.
    // A run never crosses a page: page sizes are powers of two, 16 at least, and runs are 8 or 16 keys from a multiple.
    __device__ __forceinline__ int page(const FwdArgs& a, int key) const
    {
        const int at = (key < len ? key : len - 1) >> a.page_shift;
        const int p = pages[at];
        return p >= 0 && p < a.num_pages ? p : -1;
    }
    // the run from `key` into rows r0 .. r0 + CH - 1 of both tables
    __device__ __forceinline__ void fetch(const FwdArgs& a, int key, int page, void* ktab, void* vtab, int r0) const
    {
        if (PAGED && page < 0) {
            Rows<T, D>::template clear<CH>(ktab, r0);
            Rows<T, D>::template clear<CH>(vtab, r0);
            return;
        }
        const int at = key < len ? key : len - 1;
        const int last = len - 1 - at;
        const long long row = PAGED ? ((long long)page << a.page_shift) + (at & ((1 << a.page_shift) - 1)) : at;
        Rows<T, D>::template fetch<CH>(ktab, r0, k + row * a.k_bytes, a.k_bytes, last);
        Rows<T, D>::template fetch<CH>(vtab, r0, v + row * a.v_bytes, a.v_bytes, last);
    }
};

// ---------------------------------------------------------------------------
// 128-row blocks: four waves of 32 rows; the workgroup's tiles of KT keys go
// through two LDS buffers, each wave fetching a quarter of a tile while the
// tile before it is multiplied.
// ---------------------------------------------------------------------------
template <typename T, int D, bool PAGED>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(FwdArgs a)
{
    constexpr int KT = sizeof(T) == 2 ? 64 : 32, CH = KT / 4, NK = KT / 32;
    constexpr int TAB = KT * Rows<T, D>::BYTES;
    __shared__ __align__(1024) char lds[2][2][TAB];

    const int hk = blockIdx.x % a.Hkv;
    const int rest = blockIdx.x / a.Hkv, split = rest % a.splits;
    Span s;
    if (!find_block(a.cu, a.B, a.T, a.G, 128, rest / a.splits, s)) return;
    const int R = s.n * a.G, nblk = (R + 127) / 128;
    const int row0 = (nblk - 1 - s.blk) * 128;  // the longest rows first
    const Keys<T, D, PAGED, CH> keys(a, s, hk);
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;

    const int wrow = row0 + 32 * w;
    const int row = wrow + (l & 31);
    const int rr = row < R ? row : R - 1;
    const int tok = rr / a.G, hq = hk * a.G + (rr - tok * a.G);
    Queries<T, D> qs;
    qs.load((const T*)a.q + (size_t)(s.start + tok) * a.q_stride + (size_t)hq * D);
    qs.limit = keys.seen(tok);
    // limits of the wave's first and last row, and of the workgroup's last row
    const int wmin = __builtin_amdgcn_readlane(qs.limit, 0), wmax = __builtin_amdgcn_readlane(qs.limit, 31);
    const int end = row0 + 127 < R ? row0 + 127 : R - 1;
    const int tiles = (keys.seen(end / a.G) + KT - 1) / KT;
    const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);
    const float sl2 = a.scale * kLog2e;

    int page[4] = {0, 0, 0, 0};
    auto lookup = [&](int t) {
#pragma unroll
        for (int c = 0; c < 4; ++c) page[c] = PAGED ? keys.page(a, t * KT + c * CH) : 0;
    };
    auto absent = [&]() -> unsigned {
        unsigned m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) m |= page[c] < 0 ? 1u << c : 0;
        return m;
    };
    auto fetch = [&](int t, int buf) {
        const int p = w == 0 ? page[0] : w == 1 ? page[1] : w == 2 ? page[2] : page[3];
        keys.fetch(a, t * KT + w * CH, p, lds[buf][0], lds[buf][1], w * CH);
    };

    unsigned gone = 0, gone_next = 0;
    if (t0 < t1) {
        lookup(t0);
        gone_next = absent();
        fetch(t0, 0);
        if (t0 + 1 < t1) lookup(t0 + 1);
    }
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        gone = gone_next;
        wait_vm<0>();
        __syncthreads();
        if (t + 1 < t1) {
            gone_next = absent();
            fetch(t + 1, buf ^ 1);
            if (t + 2 < t1) lookup(t + 2);
        }
        const int key0 = t * KT;
        if (key0 < wmax) {
            if (key0 + KT > wmin || gone)
                qs.template step<NK, true, CH>(lds[buf][0], lds[buf][1], 0, key0, gone, sl2);
            else
                qs.template step<NK, false, CH>(lds[buf][0], lds[buf][1], 0, key0, 0, sl2);
        }
    }

    const float sum = half_add(qs.l);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (row < R) {
        const size_t at = (size_t)(s.start + tok) * a.Hq + hq;
        const float lse2 = sum == 0.f ? -INFINITY : qs.m * sl2 + __builtin_amdgcn_logf(sum);
        if (a.splits > 1) {
            const size_t p = (size_t)split * a.T * a.Hq + at;
            if (h == 0) a.part_l[p] = lse2;
            if (sum != 0.f) {
                float* o = a.part_o + p * D;
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        store4<float>(o + 32 * dt + 8 * i + 4 * h, qs.o[dt][4 * i] * inv, qs.o[dt][4 * i + 1] * inv,
                                      qs.o[dt][4 * i + 2] * inv, qs.o[dt][4 * i + 3] * inv);
            }
        } else {
            if (a.lse && h == 0) a.lse[at] = lse2 * kLn2;
            T* o = (T*)a.o + at * D;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store4<T>(o + 32 * dt + 8 * i + 4 * h, qs.o[dt][4 * i] * inv, qs.o[dt][4 * i + 1] * inv,
                              qs.o[dt][4 * i + 2] * inv, qs.o[dt][4 * i + 3] * inv);
        }
    }
}

// ---------------------------------------------------------------------------
// 32-row blocks, for single tokens and short runs of them: the cost is the read
// of the cache, so each wave streams tiles of 32 keys of its own (every NW-th)
// through two LDS buffers of its own, with no barrier between waves, and the
// waves' results are joined at the end.
// ---------------------------------------------------------------------------
template <typename T, int D>
struct Small {
    static constexpr int STAGE = 2 * 32 * Rows<T, D>::BYTES;  // keys and values
    static constexpr int NW = STAGE > 16384 ? 2 : 4;
    static constexpr int NS = 2;
    static constexpr int OROW = D + 4;  // floats; the pad spreads the rows over the banks
    static constexpr int RING = NW * NS * STAGE;
    static constexpr int JOIN = NW * 32 * OROW * 4 + NW * 32 * 8;
    static constexpr int LDS = RING > JOIN ? RING : JOIN;
};

template <typename T, int D>
__global__ __launch_bounds__((Small<T, D>::NW * 64), 1) void attn_small_kernel(FwdArgs a)
{
    typedef Small<T, D> C;
    constexpr int NW = C::NW, NS = C::NS;
    constexpr int LOADS = 2 * 32 / Rows<T, D>::PER;
    __shared__ __align__(1024) char lds[C::LDS];

    const int hk = blockIdx.x % a.Hkv;
    const int rest = blockIdx.x / a.Hkv, split = rest % a.splits;
    Span s;
    if (!find_block(a.cu, a.B, a.T, a.G, 32, rest / a.splits, s)) return;
    const int R = s.n * a.G;
    const int row0 = s.blk * 32;
    const Keys<T, D, true, 16> keys(a, s, hk);
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;

    const int row = row0 + (l & 31);
    const int rr = row < R ? row : R - 1;
    const int tok = rr / a.G, hq = hk * a.G + (rr - tok * a.G);
    Queries<T, D> qs;
    qs.load((const T*)a.q + (size_t)(s.start + tok) * a.q_stride + (size_t)hq * D);
    qs.limit = keys.seen(tok);
    const int wmin = __builtin_amdgcn_readlane(qs.limit, 0), upto = __builtin_amdgcn_readlane(qs.limit, 31);
    const int tiles = (upto + 31) / 32;
    const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);
    const float sl2 = a.scale * kLog2e;

    char* ring = lds + w * NS * C::STAGE;
    auto fetch = [&](int t, int p0, int p1, int st) {
        char* tab = ring + st * C::STAGE;
        keys.fetch(a, t * 32, p0, tab, tab + C::STAGE / 2, 0);
        keys.fetch(a, t * 32 + 16, p1, tab, tab + C::STAGE / 2, 16);
    };
    int p0[NS], p1[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int t = t0 + w + i * NW;
        p0[i] = p1[i] = 0;
        if (t < t1) {
            p0[i] = keys.page(a, t * 32);
            p1[i] = keys.page(a, t * 32 + 16);
            fetch(t, p0[i], p1[i], i);
        }
    }
    for (int t = t0 + w; t < t1; t += NS * NW) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int tt = t + i * NW;
            if (tt < t1) {
                const int tn = tt + NS * NW;
                int n0 = 0, n1 = 0;
                if (tn < t1) {
                    n0 = keys.page(a, tn * 32);
                    n1 = keys.page(a, tn * 32 + 16);
                }
                // this tile has landed; the one behind it may be under way (an
                // absent run's tile issues fewer loads: then wait for all)
                const bool whole = tt + NW < t1 && p0[(i + 1) % NS] >= 0 && p1[(i + 1) % NS] >= 0;
                if (whole)
                    wait_vm<LOADS>();
                else
                    wait_vm<0>();
                const char* tab = ring + i * C::STAGE;
                const unsigned gone = (p0[i] < 0 ? 1u : 0u) | (p1[i] < 0 ? 2u : 0u);
                if (tt * 32 + 32 > wmin || gone)
                    qs.template step<1, true, 16>(tab, tab + C::STAGE / 2, 0, tt * 32, gone, sl2);
                else
                    qs.template step<1, false, 16>(tab, tab + C::STAGE / 2, 0, tt * 32, 0, sl2);
                // the table's reads are done before its next rows arrive
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                p0[i] = n0;
                p1[i] = n1;
                if (tn < t1) fetch(tn, n0, n1, i);
            }
        }
    }

    // join: out = sum_w 2^(m_w - m) o_w / sum_w 2^(m_w - m) l_w
    __syncthreads();
    float* ot = reinterpret_cast<float*>(lds);
    float* ml = ot + NW * 32 * C::OROW;
    const float sum = half_add(qs.l);
    if (h == 0) {
        ml[(w * 32 + l) * 2] = qs.m;
        ml[(w * 32 + l) * 2 + 1] = sum;
    }
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store4<float>(ot + (w * 32 + (l & 31)) * C::OROW + 32 * dt + 8 * i + 4 * h, qs.o[dt][4 * i],
                          qs.o[dt][4 * i + 1], qs.o[dt][4 * i + 2], qs.o[dt][4 * i + 3]);
    __syncthreads();
    constexpr int LPR = D / 4;  // lanes a row
    const int live = R - row0 < 32 ? R - row0 : 32;
    for (int i = threadIdx.x; i < live * LPR; i += NW * 64) {
        const int r = i / LPR, c = (i % LPR) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < NW; ++x) mx = fmaxf(mx, ml[(x * 32 + r) * 2]);
        float sm = 0.f;
        f32x4 acc = zero4();
#pragma unroll
        for (int x = 0; x < NW; ++x) {
            const float m = ml[(x * 32 + r) * 2];
            const float f = m == -INFINITY ? 0.f : exp2_hw((m - mx) * sl2);
            sm += f * ml[(x * 32 + r) * 2 + 1];
            const f32x4 v = *reinterpret_cast<const f32x4*>(ot + (x * 32 + r) * C::OROW + c);
            acc += f * v;
        }
        const float inv = sm == 0.f ? 0.f : 1.f / sm;
        const int tk = (row0 + r) / a.G;
        const size_t at = (size_t)(s.start + tk) * a.Hq + hk * a.G + (row0 + r - tk * a.G);
        if (a.splits > 1) {
            const size_t p = (size_t)split * a.T * a.Hq + at;
            if (c == 0) a.part_l[p] = sm == 0.f ? -INFINITY : mx * sl2 + __builtin_amdgcn_logf(sm);
            store4<float>(a.part_o + p * D + c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        } else {
            store4<T>((T*)a.o + at * D + c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        }
    }
}

// Join the splits of one row: weights 2^(l_s - max), in the order of the
// splits within each of the workgroup's row copies, then the copies in order.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(FwdArgs a)
{
    constexpr int LPR = D / 4, NG = 256 / LPR;
    __shared__ f32x4 acc_s[NG][LPR];
    __shared__ float sum_s[NG];
    const size_t row = blockIdx.x;
    const int tok = (int)(row / a.Hq);
    int lo = a.cu[0], hi = a.cu[a.B];
    if (tok < lo || tok >= hi) return;  // not a sequence's row
    const size_t rows = (size_t)a.T * a.Hq;
    const int g = threadIdx.x / LPR, c = threadIdx.x % LPR;
    float mx = -INFINITY;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, a.part_l[s * rows + row]);
    float sum = 0.f;
    f32x4 acc = zero4();
    for (int s = g; s < a.splits; s += NG) {
        const float p = a.part_l[s * rows + row];
        if (p == -INFINITY) continue;  // nothing was seen, nothing written
        const float f = exp2_hw(p - mx);
        sum += f;
        acc += f * *reinterpret_cast<const f32x4*>(a.part_o + (s * rows + row) * D + 4 * c);
    }
    acc_s[g][c] = acc;
    if (c == 0) sum_s[g] = sum;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int x = 1; x < NG; ++x) {
        acc += acc_s[x][c];
        sum += sum_s[x];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    store4<T>((T*)a.o + row * D + 4 * c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
}

template <typename T, int D>
gdn_status launch(const FwdArgs& a, const AttnPlan& p, bool paged, hipStream_t st)
{
    const dim3 grid((unsigned)((size_t)p.blocks * a.splits * a.Hkv));
    if (p.small)
        GDN_LAUNCH("attn_small", (attn_small_kernel<T, D>), grid, dim3(Small<T, D>::NW * 64), st, a);
    else if (paged)
        GDN_LAUNCH("attn_paged", (attn_fwd_kernel<T, D, true>), grid, dim3(256), st, a);
    else
        GDN_LAUNCH("attn_fwd", (attn_fwd_kernel<T, D, false>), grid, dim3(256), st, a);
    if (a.splits > 1)
        GDN_LAUNCH("attn_join", (attn_join_kernel<T, D>), dim3((unsigned)((size_t)a.T * a.Hq)), dim3(256), st, a);
    return GDN_OK;
}

}  // namespace

// 32-row blocks where the sequences have, on average, at most 64 rows.  The key axis is
// split where the blocks alone do not fill the card's 256 compute units.
AttnPlan attn_plan(const gdn_attn_shape& s, bool paged)
{
    AttnPlan p{};
    const long long G = s.Hq / s.Hkv, rows = (long long)s.T * G;
    p.small = paged && rows <= 64LL * s.B;
    p.rows = p.small ? 32 : 128;
    p.blocks = (int)(rows / p.rows + s.B);
    p.splits = 1;
    if (paged) {
        // blocks that can hold work: every sequence but the first of a block has less than a whole one
        const long long busy = (rows + p.rows - 1) / p.rows > s.B ? (rows + p.rows - 1) / p.rows : s.B;
        const long long items = busy * s.Hkv;
        const long long want = p.small ? 512 : 512;
        const long long keys = (long long)s.max_pages * s.page_size;
        const long long most = keys / (p.small ? 512 : 1024);  // at least so many keys a piece
        long long n = want / items;
        n = n > most ? most : n;
        p.splits = n < 1 ? 1 : n > 128 ? 128 : (int)n;
    }
    if (p.splits > 1) p.ws_bytes = (size_t)p.splits * s.T * s.Hq * (s.D + 1) * sizeof(float);
    return p;
}

gdn_status attn_forward_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const int* cu,
                                 const int* kv_len, const int* table, void* o, float* lse, void* ws, bool paged,
                                 hipStream_t st)
{
    const AttnPlan p = attn_plan(s, paged);
    const uint32_t e = s.dtype == GDN_BF16 ? 2 : 4;
    FwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.cu = cu; a.kv_len = kv_len; a.table = table;
    a.q_stride = s.q_stride;
    a.k_bytes = (uint32_t)(paged ? (long long)s.Hkv * s.D * e : s.k_stride * e);
    a.v_bytes = (uint32_t)(paged ? (long long)s.Hkv * s.D * e : s.v_stride * e);
    a.B = s.B; a.T = s.T; a.Hq = s.Hq; a.Hkv = s.Hkv; a.G = s.Hq / s.Hkv;
    a.num_pages = s.num_pages; a.max_pages = s.max_pages;
    a.page_shift = paged ? __builtin_ctz((unsigned)s.page_size) : 0;
    a.splits = p.splits;
    a.scale = s.scale;
    a.part_o = (float*)ws;
    a.part_l = (float*)ws + (size_t)p.splits * s.T * s.Hq * s.D;
    if (s.dtype == GDN_BF16)
        return s.D == 64 ? launch<bf16, 64>(a, p, paged, st) : launch<bf16, 128>(a, p, paged, st);
    return s.D == 64 ? launch<float, 64>(a, p, paged, st) : launch<float, 128>(a, p, paged, st);
}

}  // namespace gdn
