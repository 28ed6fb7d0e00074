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
    // the key axis is cut into pieces, at most `splits` of them, of such a length that
    // there are about `want` workgroups (for blocks of `block_rows` rows)
    int splits, want, block_rows;
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
    int rest0, rest1;  // uniform: the keys whose values the products may have left out (add_rest)

    __device__ __forceinline__ void load(const T* row)
    {
        const int h = lane_id() >> 5;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) q[kk] = load_frag<T>(row + 16 * kk + 8 * h);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = zero16();
        m = -INFINITY;
        l = 0.f;
        rest0 = 0x7fffffff, rest1 = 0;
    }

    // 32 keys of the tables from row r0; key0 is the position of the first.
    // mask (uniform): some key may lie behind some row's limit, or `gone` (a bit
    // for each run of CH keys) says that it is absent.
    template <int CH>
    __device__ __forceinline__ void step(const void* ktab, const void* vtab, int r0, int key0, bool mask, unsigned gone,
                                         float sl2)
    {
        const int h = lane_id() >> 5;
        f32x16 s = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) s = mma32(Rows<T, D>::along(ktab, r0, kk), q[kk], s);
        // the values are read now, to arrive under the exponentials
        Frag<T> v[2 * DT];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) v[b * DT + dt] = Rows<T, D>::down(vtab, r0 + 16 * b, 32 * dt);
        if (sizeof(T) == 2) {
            order_products<KK, 1, 4>();
            order_reads<4 * DT>();
        }
        if (mask) {
            // A value that a row does not see must not reach it, and 0 x infinity would:
            // where there is any, the products take finite ones, and what they leave out
            // is added in the end.
            if (__builtin_expect(!all_finite(v), 0)) {
                rest0 = rest0 < key0 ? rest0 : key0;
                rest1 = key0 + 32;
#pragma unroll
                for (int i = 0; i < 2 * DT; ++i) v[i] = finite_only(v[i]);
            }
            const int left = limit - key0 - 4 * h;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                // CH >= 8: the four rows of a register group lie in one run
                const bool out = 8 * (r >> 2) + (r & 3) >= left || ((gone >> (8 * (r >> 2) / CH)) & 1);
                s[r] = out ? -INFINITY : s[r];
            }
        }
        float mx = s[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
        mx = half_max(mx);
        // The maximum is moved, and what was summed rescaled, only when it grew
        // by more than 2^8: until then the exponentials stay below 256, which
        // costs neither bf16 nor fp32 any relative precision.
        if (__any(mx * sl2 > m * sl2 + 8.f)) {
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
        for (int r = 0; r < 16; ++r) {
            s[r] = exp2_hw(s[r] * sl2 - off);
            sum += s[r];
        }
        l += sum;
        // The operand of the second product is rounded to the inputs' type: half
        // a step of bf16 a key, against the half step of the stored output; the
        // sum above takes the unrounded values.
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const Frag<T> p = acc_frag<T>(s, b);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[dt] = mma32(v[b * DT + dt], p, o[dt]);
        }
    }

    // What the products left out of the values, below key `end`.  `at`: a key's
    // values, null for an absent one.
    template <typename F>
    __device__ __forceinline__ void add_rest(int end, F&& at)
    {
        end = end < rest1 ? end : rest1;
#pragma unroll 1
        for (int key = rest0; key < end; ++key) {
            const T* v = at(key);
            if (v) add_nonfinite<T, D>(o, v, key < limit);
        }
    }
};

constexpr int kLeastPiece = 256;

__device__ __forceinline__ int cached_len(const FwdArgs& a, int n)
{
    const long long cap = (long long)a.max_pages << a.page_shift;
    return n < 0 ? 0 : n > cap ? (int)cap : n;
}

// pieces of a sequence of len keys
__device__ __forceinline__ int pieces_of(int len, int piece) { return len > piece ? (len + piece - 1) / piece : 1; }

// 64 sequences from b0 on, lane l that of sequence b0 + l: its rows, its blocks
// and its keys (0 without new tokens).
struct Lengths {
    int st, en, nb, len;
    __device__ __forceinline__ Lengths(const FwdArgs& a, int b0)
    {
        const int l = lane_id(), b = b0 + l < a.B ? b0 + l : a.B - 1;
        st = a.cu[b], en = a.cu[b + 1], len = a.kv_len[b];
        st = st < 0 ? 0 : st > a.T ? a.T : st;
        en = en < st ? st : en > a.T ? a.T : en;
        if (b0 + l >= a.B) en = st;
        nb = (int)(((long long)(en - st) * a.G + a.block_rows - 1) / a.block_rows);
        len = en > st ? cached_len(a, len) : 0;
    }
};

// Keys a piece, the same in every wave of the call: the keys of all blocks over
// the workgroups wanted, for the table's width says little about the lengths (8
// sequences of 8192 keys in a table for 131072, 64 new tokens each, 16 heads over
// 2: 64 us, against 429 us with pieces from the table's width; one token each
// for 16 of them: 30 us, against 83 us).  A multiple of 128 and no more pieces
// than there is room for; below 1024 keys, where writing and joining the partial
// outputs begins to count, only as far as one workgroup for each compute unit
// asks for it.  The kernel and the join of its pieces each form it and have to
// find the same bits: nothing is contracted here, since whether a product (rounded
// from 2^24 on) goes into its sum unrounded would be the compiler's choice in each.
__device__ __forceinline__ int piece_keys(const FwdArgs& a, const Lengths& first)
{
#pragma clang fp contract(off)
    float work = wave_sum((float)first.nb * (float)first.len);
    int most = wave_max(first.len);
    for (int b0 = 64; b0 < a.B; b0 += 64) {
        const Lengths v(a, b0);
        work += wave_sum((float)v.nb * (float)v.len);
        const int m = wave_max(v.len);
        most = most > m ? most : m;
    }
    work *= (float)a.Hkv;
    const float even = fmaxf(work / (float)a.want, fminf(work * (1.f / 256.f), 1024.f));
    const int need = (most + a.splits - 1) / a.splits;
    int keys = even > (float)(1 << 29) ? 1 << 29 : (int)even + 1;
    keys = keys > need ? keys : need;
    keys = keys > kLeastPiece ? keys : kLeastPiece;
    return uniform((keys + 127) / 128 * 128);
}

// What a workgroup does: block `s`, and of its sequence's `pieces` pieces, of
// `piece` keys each (the sequence's own share, so that its last piece is no
// remnant), the `split`-th.  False: nothing.
struct Job {
    Span s;
    int split, pieces, piece;
    template <bool PAGED, int BR>
    __device__ __forceinline__ bool find(const FwdArgs& a, int id)
    {
        split = 0, pieces = 1, piece = 1 << 30;
        if (!PAGED || a.splits <= 1) return find_block<!PAGED>(a.cu, a.B, a.T, a.G, BR, id, s);
        // every (block, piece) there is, one after the other: nobody starts for nothing but at the end
        Lengths v(a, 0);
        const int most = piece_keys(a, v);
        for (int b0 = 0, before = 0;;) {
            const int np = pieces_of(v.len, most), n = v.nb * np, inc = wave_scan(n);
            const uint64_t hit = __ballot(before + inc > id);
            if (hit) {
                const int b = __builtin_ctzll(hit);
                const int at = id - before - __builtin_amdgcn_readlane(inc - n, b);
                pieces = __builtin_amdgcn_readlane(np, b);
                s.b = b0 + b;
                s.start = __builtin_amdgcn_readlane(v.st, b);
                s.n = __builtin_amdgcn_readlane(v.en, b) - s.start;
                s.blocks = __builtin_amdgcn_readlane(v.nb, b);
                split = at / s.blocks;  // blocks that read the same keys together
                s.level = s.blocks - 1 - at % s.blocks;
                piece = ((__builtin_amdgcn_readlane(v.len, b) + pieces - 1) / pieces + 127) / 128 * 128;
                return true;
            }
            before += __builtin_amdgcn_readlane(inc, 63);
            b0 += 64;
            if (b0 >= a.B) return false;
            v = Lengths(a, b0);
        }
    }
};

// The keys of one (sequence, key head): where a run of CH keys lies.
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
            len = cached_len(a, n);
            n = n < 0 ? 0 : n > (1 << 30) ? 1 << 30 : n;
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
    // Page of the run that starts at key `key` (of the last key where it starts behind the end), -1: none.  A run
    // never crosses a page: page sizes are powers of two from 16 on, and runs start at multiples of their 8 or 16 keys.
    __device__ __forceinline__ int page(const FwdArgs& a, int key) const
    {
        if (!PAGED || len == 0) return 0;
        const int p = pages[(key < len ? key : len - 1) >> a.page_shift];
        return p >= 0 && p < a.num_pages ? p : -1;
    }
    // the values of key `key`, below len; null: absent
    __device__ __forceinline__ const T* value(const FwdArgs& a, int key) const
    {
        const int p = page(a, key);
        if (PAGED && p < 0) return nullptr;
        const long long row = PAGED ? ((long long)p << a.page_shift) + (key & ((1 << a.page_shift) - 1)) : key;
        return (const T*)(v + row * a.v_bytes);
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
// tile before it is multiplied.  The waves take a tile 32 keys at a time, which
// keeps the scores, the outputs and the queries of a row within the 256
// registers that two waves a SIMD have (64 keys at once spilled: 412 us instead of
// 295 us).  Bound by the matrix units and the card's power: 8192 tokens, 16 heads
// over 4 of 128, bf16, take 297 to 312 us, 880 to 925 TFLOP/s.
// ---------------------------------------------------------------------------
template <typename T, int D, bool PAGED>
__global__ __launch_bounds__(256, (sizeof(T) == 4 && D == 128) ? 1 : 2) void attn_fwd_kernel(FwdArgs a)
{
    constexpr int KT = sizeof(T) == 2 ? 64 : 32, CH = KT / 4;
    constexpr int TAB = KT * Rows<T, D>::BYTES;
    constexpr int WIN = 16;  // tiles whose pages a wave holds: lane 4 i + c has run c of the i-th
    __shared__ __align__(1024) char lds[2][2][TAB];

    const int hk = blockIdx.x % a.Hkv;
    Job job;
    if (!job.find<PAGED, 128>(a, blockIdx.x / a.Hkv)) return;
    const Span& s = job.s;
    const int split = job.split, pieces = job.pieces, piece = job.piece;
    const int R = s.n * a.G, row0 = s.level * 128;
    const Keys<T, D, PAGED, CH> keys(a, s, hk);
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;

    const int row = row0 + 32 * w + (l & 31);
    const int rr = row < R ? row : R - 1;
    const int tok = rr / a.G, hq = hk * a.G + (rr - tok * a.G);
    Queries<T, D> qs;
    qs.load((const T*)a.q + (size_t)(s.start + tok) * a.q_stride + (size_t)hq * D);
    qs.limit = keys.seen(tok);
    // limits of the wave's first and last row, and of the workgroup's last row
    const int wmin = __builtin_amdgcn_readlane(qs.limit, 0), wmax = __builtin_amdgcn_readlane(qs.limit, 31);
    const int end = row0 + 127 < R ? row0 + 127 : R - 1;
    const int tiles = (keys.seen(end / a.G) + KT - 1) / KT;
    const int t0 = pieces > 1 ? split * (piece / KT) : 0;
    int t1 = pieces > 1 ? t0 + piece / KT : tiles;
    t1 = t1 < tiles ? t1 : tiles;
    const float sl2 = a.scale * kLog2e;

    int ids = 0, ids_next = 0;  // pages of the window's tiles, and of the next window's
    if (PAGED) {
        ids = keys.page(a, (t0 + (l >> 2)) * KT + (l & 3) * CH);
        ids_next = keys.page(a, (t0 + WIN + (l >> 2)) * KT + (l & 3) * CH);
    }
    auto fetch = [&](int t, int buf) -> unsigned {  // returns the runs that are absent
        unsigned gone = 0;
        int p = 0;
        if (PAGED) {
            const int i = (t - t0) % WIN;
            if (i == 0 && t > t0) {
                ids = ids_next;
                ids_next = keys.page(a, (t + WIN + (l >> 2)) * KT + (l & 3) * CH);
            }
            gone = (unsigned)(__ballot(ids < 0) >> (4 * i)) & 15u;
            p = __builtin_amdgcn_readlane(ids, 4 * i + w);
        }
        keys.fetch(a, t * KT + w * CH, p, lds[buf][0], lds[buf][1], w * CH);
        return gone;
    };

    unsigned gone = 0, gone_next = 0;
    // one tile: the buffers are compile-time constants, so that every LDS address
    // is a fixed register plus an immediate
    auto tile = [&](int t, auto BUF) {
        constexpr int buf = BUF();
        gone = gone_next;
        wait_vm<0>();
        __syncthreads();
        if (t + 1 < t1) gone_next = fetch(t + 1, buf ^ 1);
#pragma unroll
        for (int sub = 0; sub < KT / 32; ++sub) {
            const int key0 = t * KT + 32 * sub;
            if (key0 < wmax)
                qs.template step<CH>(lds[buf][0], lds[buf][1], 32 * sub, key0, key0 + 32 > wmin || gone,
                                     gone >> (sub * 32 / CH), sl2);
        }
    };
    if (t0 < t1) gone_next = fetch(t0, 0);
    for (int t = t0; t < t1; t += 2) {
        tile(t, std::integral_constant<int, 0>{});
        if (t + 1 < t1) tile(t + 1, std::integral_constant<int, 1>{});
    }

    if (__builtin_expect(qs.rest1, 0))
        qs.add_rest(t1 * KT < wmax ? t1 * KT : wmax, [&](int key) { return keys.value(a, key); });
    const float sum = half_add(qs.l);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (row < R) {
        const size_t at = (size_t)(s.start + tok) * a.Hq + hq;
        const float lse2 = sum == 0.f ? -INFINITY : qs.m * sl2 + __builtin_amdgcn_logf(sum);
        if (pieces > 1) {
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
// 32-row blocks, for single tokens and short runs of them, and for prompts too
// few to fill the card with 128-row blocks: the waves share out the keys.  Each
// wave streams tiles of 32 keys of its own (every NW-th) through two LDS
// buffers of its own, with no barrier between waves, and the waves' results
// are joined at the end.  Bound by HBM over a cache: 256 sequences of up to 4097
// keys, 16 heads over 4 of 128, bf16, take 264 us, 5.1 TB/s; two of up to 131073,
// heads over 2, 40 us, 6.1 TB/s.
// ---------------------------------------------------------------------------
template <typename T, int D>
struct Small {
    static constexpr int STAGE = 2 * 32 * Rows<T, D>::BYTES;  // keys and values
    // bf16: 64 KB a workgroup, two of them a compute unit; fp32, bound by its
    // matrix instructions, as many waves as fit 128 KB
    static constexpr int NW = (sizeof(T) == 2 ? 65536 : 131072) / (2 * STAGE);
    static constexpr int NS = 2;
    static_assert(NW == 2 || NW == 4, "waves");
    static constexpr int OROW = D + 4;  // floats; the pad spreads the rows over the banks
    static constexpr int RING = NW * NS * STAGE;
    static constexpr int JOIN = NW * 32 * OROW * 4 + NW * 32 * 8;
    static constexpr int LDS = RING > JOIN ? RING : JOIN;
};

template <typename T, int D, bool PAGED>
__global__ __launch_bounds__((Small<T, D>::NW * 64), 1) void attn_small_kernel(FwdArgs a)
{
    typedef Small<T, D> C;
    constexpr int NW = C::NW, NS = C::NS;
    constexpr int LOADS = 2 * 32 / Rows<T, D>::PER;
    constexpr int WIN = 32;  // tiles whose pages a wave holds: lane 2 i + c has run c of the wave's i-th tile
    __shared__ __align__(1024) char lds[C::LDS];

    const int hk = blockIdx.x % a.Hkv;
    Job job;
    if (!job.find<PAGED, 32>(a, blockIdx.x / a.Hkv)) return;
    const Span& s = job.s;
    const int split = job.split, pieces = job.pieces, piece = job.piece;
    const int R = s.n * a.G, row0 = s.level * 32;
    const Keys<T, D, PAGED, 16> keys(a, s, hk);
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;

    const int row = row0 + (l & 31);
    const int rr = row < R ? row : R - 1;
    const int tok = rr / a.G, hq = hk * a.G + (rr - tok * a.G);
    Queries<T, D> qs;
    qs.limit = keys.seen(tok);
    const int wmin = __builtin_amdgcn_readlane(qs.limit, 0), upto = __builtin_amdgcn_readlane(qs.limit, 31);
    const int tiles = (upto + 31) / 32;
    const int t0 = pieces > 1 ? split * (piece / 32) : 0;
    int t1 = pieces > 1 ? t0 + piece / 32 : tiles;
    t1 = t1 < tiles ? t1 : tiles;
    const float sl2 = a.scale * kLog2e;

    char* ring = lds + w * NS * C::STAGE;
    // the wave's tiles are t0 + w + i NW, i = 0 .. n - 1
    const int tw = t0 + w, n = t1 > tw ? (t1 - tw + NW - 1) / NW : 0;
    auto window = [&](int i) { return PAGED ? keys.page(a, (tw + (i + (l >> 1)) * NW) * 32 + (l & 1) * 16) : 0; };
    int ids = window(0), ids_next = 0;
    if (n > WIN) ids_next = window(WIN);
    qs.load((const T*)a.q + (size_t)(s.start + tok) * a.q_stride + (size_t)hq * D);
    unsigned gone[NS] = {};  // absent runs of the tile in each buffer
    auto fetch = [&](int i, int st) {
        const int t = tw + i * NW, at = i % WIN;
        int p0 = 0, p1 = 0;
        if (PAGED) {
            if (at == 0 && i > 0) {
                ids = ids_next;
                ids_next = window(i + WIN);
            }
            p0 = __builtin_amdgcn_readlane(ids, 2 * at);
            p1 = __builtin_amdgcn_readlane(ids, 2 * at + 1);
            gone[st] = (p0 < 0 ? 1u : 0u) | (p1 < 0 ? 2u : 0u);
        }
        char* tab = ring + st * C::STAGE;
        keys.fetch(a, t * 32, p0, tab, tab + C::STAGE / 2, 0);
        keys.fetch(a, t * 32 + 16, p1, tab, tab + C::STAGE / 2, 16);
    };
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (i < n) fetch(i, i);
    for (int i0 = 0; i0 < n; i0 += NS) {
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            const int i = i0 + st;
            if (i < n) {
                // this tile has landed; the one behind it may be under way (a
                // tile with absent runs has fewer loads: then all are waited for)
                if (i + 1 < n && gone[(st + 1) % NS] == 0)
                    wait_vm<LOADS>();
                else
                    wait_vm<0>();
                const int key0 = (tw + i * NW) * 32;
                const char* tab = ring + st * C::STAGE;
                qs.template step<16>(tab, tab + C::STAGE / 2, 0, key0, key0 + 32 > wmin || gone[st], gone[st], sl2);
                // the table's reads are done before its next rows arrive
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (i + NS < n) fetch(i + NS, st);
            }
        }
    }

    if (__builtin_expect(qs.rest1, 0))
        qs.add_rest(t1 * 32 < upto ? t1 * 32 : upto, [&](int key) { return keys.value(a, key); });
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
        const float lse2 = sm == 0.f ? -INFINITY : mx * sl2 + __builtin_amdgcn_logf(sm);
        if (pieces > 1) {
            const size_t p = (size_t)split * a.T * a.Hq + at;
            if (c == 0) a.part_l[p] = lse2;
            store4<float>(a.part_o + p * D + c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        } else {
            if (a.lse && c == 0) a.lse[at] = lse2 * kLn2;
            store4<T>((T*)a.o + at * D + c, acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        }
    }
}

// Join the pieces of a row: weights 2^(l_s - max).  Q waves share a row's pieces
// (every Q-th each), and their sums are added in order: the same in every run.
template <typename T, int D, int Q>
__global__ __launch_bounds__((Q > 4 ? Q : 4) * 64) void attn_join_kernel(FwdArgs a)
{
    constexpr int V = D / 64;  // values a lane
    constexpr int NW = Q > 4 ? Q : 4;
    __shared__ float acc_s[NW][D];
    __shared__ float sum_s[NW];
    const int w = uniform(wave_id()), l = lane_id(), q = w % Q;
    const size_t rows = (size_t)a.T * a.Hq;
    const size_t row = (size_t)blockIdx.x * (NW / Q) + w / Q;
    int np = 1;
    if (row < rows) {
        const int tok = (int)(row / a.Hq);
        Lengths v(a, 0);
        const int most = piece_keys(a, v);
        for (int b0 = 0;;) {
            const uint64_t hit = __ballot(tok >= v.st && tok < v.en);
            if (hit) {
                np = __builtin_amdgcn_readlane(pieces_of(v.len, most), __builtin_ctzll(hit));
                break;
            }
            b0 += 64;
            if (b0 >= a.B) break;
            v = Lengths(a, b0);
        }
    }
    float acc[V] = {}, sum = 0.f;
    if (np > 1) {
        float mx = -INFINITY;
        for (int s0 = 0; s0 < np; s0 += 64) {
            float p = s0 + l < np ? a.part_l[(s0 + l) * rows + row] : -INFINITY;
#pragma unroll
            for (int d = 32; d; d >>= 1) p = fmaxf(p, __shfl_xor(p, d));
            mx = fmaxf(mx, p);
        }
#pragma unroll 8
        for (int s = q; s < np; s += Q) {
            const float p = a.part_l[s * rows + row];
            // a piece that saw nothing wrote no output: its old contents are read and not used
            const float f = p == -INFINITY ? 0.f : exp2_hw(p - mx);
            sum += f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float x = a.part_o[(s * rows + row) * D + V * l + v];
                acc[v] += p == -INFINITY ? 0.f : f * x;
            }
        }
    }
    if (Q > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) acc_s[w][V * l + v] = acc[v];
        if (l == 0) sum_s[w] = sum;
        __syncthreads();
        if (q) return;
#pragma unroll
        for (int x = 1; x < Q; ++x) {
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += acc_s[w + x][V * l + v];
            sum += sum_s[w + x];
        }
    }
    if (np > 1) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T* o = (T*)a.o + row * D + V * l;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = from_f32<T>(acc[v] * inv);
    }
}

template <typename T, int D>
gdn_status launch(const FwdArgs& a, const AttnPlan& p, bool paged, hipStream_t st)
{
    const dim3 grid((unsigned)(p.jobs * a.Hkv));
    const dim3 threads(p.small ? Small<T, D>::NW * 64 : 256);
    if (p.small && paged)
        GDN_LAUNCH("attn_small_paged", (attn_small_kernel<T, D, true>), grid, threads, st, a);
    else if (p.small)
        GDN_LAUNCH("attn_small", (attn_small_kernel<T, D, false>), grid, threads, st, a);
    else if (paged)
        GDN_LAUNCH("attn_paged", (attn_fwd_kernel<T, D, true>), grid, threads, st, a);
    else
        GDN_LAUNCH("attn_fwd", (attn_fwd_kernel<T, D, false>), grid, threads, st, a);
    if (a.splits > 1) {
        const size_t rows = (size_t)a.T * a.Hq;
        if (rows <= 128)
            GDN_LAUNCH("attn_join", (attn_join_kernel<T, D, 16>), dim3((unsigned)rows), dim3(1024), st, a);
        else if (rows <= 2048)
            GDN_LAUNCH("attn_join", (attn_join_kernel<T, D, 4>), dim3((unsigned)rows), dim3(256), st, a);
        else
            GDN_LAUNCH("attn_join", (attn_join_kernel<T, D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), st, a);
    }
    return GDN_OK;
}

}  // namespace

// 32-row blocks over a cache where the sequences have, on average, at most 32
// rows (8 sequences of 4096 keys, 16 heads over 4: 8 tokens each take 24 us, with
// 128-row blocks 30 us; 16 tokens 33 us and 31 us, 32 sequences of them 54 us and
// 34 us), and for prompts whose 128-row blocks are fewer than the compute units
// (fp32, 2048 tokens, 8 heads over 2: 168 us against 279 us; bf16: 40 and 43;
// 4096 tokens, which have enough: 621 us against 554 us).
// The key axis of a cache is cut into pieces where the blocks alone do not fill
// the card: two workgroups of 32-row blocks fit a compute unit, and the 128-row
// ones, whose work is uneven, end together best with somewhat more (chunks of 512
// on 16384, 219 us for 896 workgroups: 768 take 4 % longer, 640 8 %).  The room for
// partial outputs bounds the pieces: it is laid out for all rows alike, so that a
// long sequence among many short ones is cut into no more pieces than their number
// leaves (none from 513 pairs of a sequence and a key head on).
AttnPlan attn_plan(const gdn_attn_shape& s, bool paged)
{
    AttnPlan p{};
    const long long G = s.Hq / s.Hkv, rows = (long long)s.T * G;
    const long long big = ((rows + 127) / 128) * s.Hkv;
    p.small = paged ? rows <= 32LL * s.B : big < 256;
    p.rows = p.small ? 32 : 128;
    p.blocks = rows / p.rows + s.B;
    p.splits = 1;
    const long long cap = (long long)s.max_pages * s.page_size;
    p.want = p.small ? 512 : 896;
    if (paged) {
        const long long full = (rows + p.rows - 1) / p.rows, busy = full > s.B ? full : s.B, items = busy * s.Hkv;
        // room for twice the pieces that equal lengths would make
        const long long most = (cap + kLeastPiece - 1) / kLeastPiece;
        long long n = 2 * p.want / items;
        n = n > most ? most : n;
        p.splits = n < 1 ? 1 : n > 128 ? 128 : (int)n;
    }
    p.jobs = p.blocks * p.splits;
    // The sum of ceil(len / piece) over the blocks is at most one a block more than
    // the sum of len / piece, which a piece's length holds to want / Hkv (or to 256
    // / Hkv, where it is below 1024).
    if (p.splits > 1 && p.jobs > p.want / s.Hkv + p.blocks + 2) p.jobs = p.want / s.Hkv + p.blocks + 2;
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
    a.splits = p.splits; a.want = p.want; a.block_rows = p.rows;
    a.scale = s.scale;
    a.part_o = (float*)ws;
    a.part_l = (float*)ws + (size_t)p.splits * s.T * s.Hq * s.D;
    if (s.dtype == GDN_BF16)
        return s.D == 64 ? launch<bf16, 64>(a, p, paged, st) : launch<bf16, 128>(a, p, paged, st);
    return s.D == 64 ? launch<float, 64>(a, p, paged, st) : launch<float, 128>(a, p, paged, st);
}

}  // namespace gdn
