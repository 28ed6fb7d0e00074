// attn_bwd.hip -- gradients of causal softmax attention over packed prompts.
//
//   p_ij = exp(scale q_i . k_j - lse_i),   delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
//
// The probabilities are formed again from the saved log-sums.  Two passes, one
// over the queries of a block of keys (dk, dv: a key's sum runs over all query
// heads of its group inside one workgroup) and one over the keys of a block of
// queries (dq): seven products where five would do, and in return no sum ever
// crosses workgroups, so there are no atomics and the order is the same in every
// run.  Both products that sum over an accumulator's rows take it as their
// operand without leaving the registers (attn.h).
#include "attn.h"

namespace gdn {

namespace {

struct BwdArgs {
    const void *q, *k, *v, *o, *dO;
    const float* lse;
    const int* cu;
    void *dq, *dk, *dv;
    // [Hq][T]: lse * log2 e and delta for the key pass, left by the query pass (bf16)
    // or by attn_delta_kernel (fp32)
    float *lse2, *delta;
    long long q_stride;
    uint32_t q_bytes, k_bytes, v_bytes, o_bytes;  // bytes between tokens
    int B, T, Hq, Hkv, G;
    float scale;
    int kparts, qparts;  // pieces that a key block's queries, a query block's keys are cut into
    float *part_k, *part_q;  // [2][kparts][T * Hkv][D] (dk, dv), [qparts][T * Hq][D]
};

// Four accumulator rows of one column times f: to the gradient, or to a piece's
// partial sums where the work is cut up.
template <typename T>
__device__ __forceinline__ void put4(T* out, float* part, size_t at, const f32x16& v, int i, float f)
{
    if (part)
        store4<float>(part + at, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else
        store4<T>(out + at, v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
}

// The key pass: dk, dv of 128 keys: four waves of 32 keys.  The keys stay in registers, the
// values in LDS (with both in registers a wave would need more than the 256 that
// two waves a SIMD have, and spills: 2.3 times the time); tiles of 32 tokens of one
// query head after the other go through two LDS buffers.  Four products for a pair:
// 8192 tokens, 16 heads over 4 of 128, bf16, take 530 us, 1.04 PFLOP/s.
template <typename T, int D>
struct KeyLds {
    static constexpr int QT = 32, TAB = QT * Rows<T, D>::BYTES;
    char lds[2][2][TAB];  // q, do
    float ld[2][2][64];   // lse2, delta of a tile (64 lanes' words; QT are read)
    __align__(1024) char vtab[128 * Rows<T, D>::BYTES];
};

template <typename T, int D>
__device__ __forceinline__ void key_pass(const BwdArgs& a, int id, KeyLds<T, D>& m)
{
    constexpr int KK = D / 16, DT = D / 32;
    constexpr int QT = KeyLds<T, D>::QT, RW = QT / 4;
    auto& vtab = m.vtab;
    auto& lds = m.lds;
    auto& ld = m.ld;

    const int hk = id % a.Hkv;
    const int rest = id / a.Hkv, part = rest % a.kparts;
    Span s;
    if (!find_block<true>(a.cu, a.B, a.T, 1, 128, rest / a.kparts, s)) return;
    const int key0 = (s.blocks - 1 - s.level) * 128;  // the first keys have the most queries: they come first
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;
    const int wkey = key0 + 32 * w;
    const int key = wkey + (l & 31);
    const int kc = key < s.n ? key : s.n - 1;
    const unsigned seen = key < s.n ? s.n - key : 0;  // queries that see the key

    Frag<T> kf[KK];
    {
        const T* kp = (const T*)((const char*)a.k + (size_t)(s.start + kc) * a.k_bytes) + (size_t)hk * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) kf[kk] = load_frag<T>(kp + 16 * kk + 8 * h);
        const int at = wkey < s.n ? wkey : s.n - 1;
        Rows<T, D>::template fetch<32>(vtab, 32 * w,
                                       (const char*)a.v + (size_t)(s.start + at) * a.v_bytes + (size_t)hk * D * sizeof(T),
                                       a.v_bytes, s.n - 1 - at);
    }
    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dk[dt] = dv[dt] = zero16();

    const float sl2 = a.scale * kLog2e;
    // tiles: the query tiles at or after the block, of one head after the other; this piece's are i0 .. i1 - 1
    const int tq0 = key0 / QT, ntq = (s.n + QT - 1) / QT - tq0;
    const int total = ntq * a.G;
    const int i0 = (int)((long long)total * part / a.kparts), i1 = (int)((long long)total * (part + 1) / a.kparts);
    int fg = i0 / ntq, fq = i0 - fg * ntq;  // head and query tile of the next fetch
    auto fetch = [&](int buf) {
        const int q0 = (tq0 + fq) * QT, hq = hk * a.G + fg;
        const int at = q0 + w * RW < s.n ? q0 + w * RW : s.n - 1;
        const int last = s.n - 1 - at;
        const size_t tok = (size_t)(s.start + at);
        Rows<T, D>::template fetch<RW>(lds[buf][0], w * RW, (const char*)a.q + tok * a.q_bytes + (size_t)hq * D * sizeof(T),
                                       a.q_bytes, last);
        Rows<T, D>::template fetch<RW>(lds[buf][1], w * RW, (const char*)a.dO + tok * a.o_bytes + (size_t)hq * D * sizeof(T),
                                       a.o_bytes, last);
        const int t = q0 + l < s.n ? q0 + l : s.n - 1;
        if (w == 0) dma4(a.lse2 + (size_t)hq * a.T + s.start + t, ld[buf][0]);
        if (w == 1) dma4(a.delta + (size_t)hq * a.T + s.start + t, ld[buf][1]);
        if (++fq == ntq) {
            fq = 0;
            ++fg;
        }
    };
    int cq = fq;  // query tile of the one being multiplied
    int later = i1;  // masked tiles from this one on are left for the end (attn.h)
    const uint32_t along = Rows<T, D>::along_at();
    auto tile = [&](int it, auto BUF) {
        constexpr int buf = BUF();
        wait_vm<0>();
        __syncthreads();
        if (it + 1 < i1) fetch(buf ^ 1);
        const int qs = (tq0 + cq) * QT;
        if (++cq == ntq) cq = 0;
        if (qs + 31 < wkey) return;  // every query stands before the wave's keys
        const void* qt = lds[buf][0];
        const void* ot = lds[buf][1];
        f32x16 sc = zero16(), dp = zero16();
        const uint32_t at = opaque(along);
        const char* vw = vtab + 32 * w * Rows<T, D>::BYTES;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) sc = mma32(Rows<T, D>::along(qt, at, 0, kk), kf[kk], sc);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            dp = mma32(Rows<T, D>::along(ot, at, 0, kk), Rows<T, D>::along(vw, at, 0, kk), dp);
        if (sizeof(T) == 2) {
            order_products<KK, 1, 4>();
            order_products<KK, 2, 2>();
            __builtin_amdgcn_sched_barrier(0);  // the statistics' reads stay behind
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 ls = *reinterpret_cast<const f32x4*>(&ld[buf][0][8 * i + 4 * h]);
            const f32x4 de = *reinterpret_cast<const f32x4*>(&ld[buf][1][8 * i + 4 * h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * i + e;
                sc[r] = exp2_hw(sc[r] * sl2 - ls[e]);
                dp[r] = sc[r] * (dp[r] - de[e]);
            }
        }
        if (qs < wkey + 31 || qs + 32 > s.n) {
            // a query's q that is not finite leaves its log-sum, its do its delta neither
            const bool finite = fabsf(ld[buf][h][l & 31]) < INFINITY;
            if (__builtin_expect(!__all(finite) || later < i1, 0)) {
                later = later < it ? later : it;
                return;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const bool in = (unsigned)(qs - key + 4 * h + 8 * (r >> 2) + (r & 3)) < seen;  // key <= query < s.n
                sc[r] = in ? sc[r] : 0.f;
                dp[r] = in ? dp[r] : 0.f;
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // both operands are rounded to the inputs' type, as in the forward
            const Frag<T> p = acc_frag<T>(sc, b), ds = acc_frag<T>(dp, b);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                dv[dt] = mma32(Rows<T, D>::down(ot, 16 * b, 32 * dt), p, dv[dt]);
                dk[dt] = mma32(Rows<T, D>::down(qt, 16 * b, 32 * dt), ds, dk[dt]);
            }
        }
        if (sizeof(T) == 2) order_products<4 * DT, 2, 3>();
    };
    if (i0 < i1) fetch(0);
    for (int it = i0; it < i1; it += 2) {
        tile(it, std::integral_constant<int, 0>{});
        if (it + 1 < i1) tile(it + 1, std::integral_constant<int, 1>{});
    }
    wait_vm<0>();  // a piece without tiles still has its values under way
    // The masked tiles that were left: the same steps, with finite operands in the
    // products and everything but v straight from memory.
#pragma unroll 1
    for (int it = later; it < i1; ++it) {
        const int h4 = opaque(4 * h);  // of this loop alone: nothing is formed ahead of the other
        const int g = it / ntq, qs = (tq0 + it - g * ntq) * QT, hq = hk * a.G + g;
        if (qs + 31 < wkey || !(qs < wkey + 31 || qs + 32 > s.n)) continue;
        auto row = [&](int q) { return (size_t)(s.start + (q < s.n ? q : s.n - 1)); };
        auto q_at = [&](int q) { return (const T*)((const char*)a.q + row(q) * a.q_bytes) + (size_t)hq * D; };
        auto o_at = [&](int q) { return (const T*)((const char*)a.dO + row(q) * a.o_bytes) + (size_t)hq * D; };
        f32x16 sc = zero16(), dp = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int c = 16 * kk + 2 * h4;
            sc = mma32(load_frag<T>(q_at(qs + (l & 31)) + c), kf[kk], sc);
            dp = mma32(load_frag<T>(o_at(qs + (l & 31)) + c), Rows<T, D>::along(vtab + 32 * w * Rows<T, D>::BYTES, along, 0, kk), dp);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int q = qs + 8 * (r >> 2) + h4 + (r & 3);
            const size_t st = (size_t)hq * a.T + row(q);
            const bool in = (unsigned)(q - key) < seen;
            const float p = exp2_hw(sc[r] * sl2 - a.lse2[st]), ds = p * (dp[r] - a.delta[st]);
            sc[r] = in ? p : 0.f;
            dp[r] = in ? ds : 0.f;
        }
        // columns d .. d + 31 of 16 rows from q0 on, as Rows::down reads them, one
        // after the other: no registers of the loop above are for this
        auto down = [&](auto at, int q0, int d) {
            Frag<T> v;
            __builtin_amdgcn_sched_barrier(0);
            q0 = opaque(q0);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = frag_value(at(q0 + 8 * (j >> 2) + h4 + (j & 3))[d + (l & 31)]);
            return finite_only(v);
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const Frag<T> p = acc_frag<T>(sc, b), ds = acc_frag<T>(dp, b);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                dv[dt] = mma32(down(o_at, qs + 16 * b, 32 * dt), p, dv[dt]);
                dk[dt] = mma32(down(q_at, qs + 16 * b, 32 * dt), ds, dk[dt]);
            }
        }
        // (of a query whose q is not finite no p is: dk has it from the products)
#pragma unroll 1
        for (int q = qs; q < qs + 32 && q < s.n; ++q) add_nonfinite<T, D>(dv, o_at(q), key <= q);
    }
    if (key < s.n) {
        const size_t at = ((size_t)(s.start + key) * a.Hkv + hk) * D, all = (size_t)a.T * a.Hkv * D;
        float* pk = a.kparts > 1 ? a.part_k + part * all : nullptr;
        float* pv = a.kparts > 1 ? a.part_k + (a.kparts + part) * all : nullptr;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 32 * dt + 8 * i + 4 * h;
                put4<T>((T*)a.dk, pk, at + c, dk[dt], i, a.scale);
                put4<T>((T*)a.dv, pv, at + c, dv[dt], i, 1.f);
            }
    }
}

// The query pass: dq of 128 rows (token * G + head): four waves of 32 rows; tiles
// of KT keys go through two LDS buffers.  Three products for a pair: 395 us, 1.04
// PFLOP/s at the sizes above.
//
// bf16: delta_i = do_i . o_i carries the rounding of the stored o, and an error
// e_i in it reaches every ds_ij as -p_ij e_i.  Since sum_j p_ij = 1, the row sum
// sum_j ds_ij, which is 0 for the true delta, is -e_i with the given one; so it is
// summed on the way and delta + sum_j ds_ij goes to the key pass.  Rows that see
// at most SHORT keys, where o is as large as the values it averages and its
// rounding counts most, take a first round over their keys for it and use it in
// their own dq too.  (Error of dq and dk against 64 bits, in units of the error of
// storing them: 1.7 and 1.8 at 16 tokens without this, 1.4 with it; two tokens,
// whose gradients are a product or two, have up to 2.2.)  Where the keys are cut
// into pieces no piece has the whole row sum, and the longer rows keep the given
// delta: 1.4 with scores of deviation 1, 2.0 with 4, where few keys take the weight.
template <typename T, int D>
struct QueryLds {
    static constexpr int KT = sizeof(T) == 2 ? 64 : 32;
    char lds[2][2][KT * Rows<T, D>::BYTES];  // k, v
};

template <typename T, int D>
__device__ __forceinline__ void query_pass(const BwdArgs& a, int id, QueryLds<T, D>& m)
{
    constexpr int KK = D / 16, DT = D / 32;
    constexpr int KT = QueryLds<T, D>::KT, RW = KT / 4;
    constexpr int SHORT = 512;
    auto& lds = m.lds;

    const int hk = id % a.Hkv;
    const int rest = id / a.Hkv, part = rest % a.qparts;
    Span s;
    if (!find_block<true>(a.cu, a.B, a.T, a.G, 128, rest / a.qparts, s)) return;
    const int R = s.n * a.G, row0 = s.level * 128;
    const int w = uniform(wave_id()), l = lane_id(), h = l >> 5;
    const int row = row0 + 32 * w + (l & 31);
    const int rr = row < R ? row : R - 1;
    const int tok = rr / a.G, hq = hk * a.G + (rr - tok * a.G);
    const size_t at = (size_t)(s.start + tok);
    Frag<T> qf[KK], df[KK];
    float delta = 0.f;
    {
        const T* qp = (const T*)a.q + at * a.q_stride + (size_t)hq * D;
        const T* dp = (const T*)a.dO + (at * a.Hq + hq) * D;
        const T* op = (const T*)a.o + (at * a.Hq + hq) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            qf[kk] = load_frag<T>(qp + 16 * kk + 8 * h);
            df[kk] = load_frag<T>(dp + 16 * kk + 8 * h);
            const Frag<T> of = load_frag<T>(op + 16 * kk + 8 * h);
#pragma unroll
            for (int j = 0; j < 8; ++j) delta += (float)of[j] * (float)df[kk][j];
        }
    }
    delta = half_add(delta);
    const float lse2 = a.lse[at * a.Hq + hq] * kLog2e;
    f32x16 dq[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dq[dt] = zero16();
    const float sl2 = a.scale * kLog2e;

    const int limit = tok + 1;
    const int wmin = __builtin_amdgcn_readlane(limit, 0), wmax = __builtin_amdgcn_readlane(limit, 31);
    const int end = row0 + 127 < R ? row0 + 127 : R - 1;
    const int tiles = (end / a.G + 1 + KT - 1) / KT;
    const char* kb = (const char*)a.k + (size_t)s.start * a.k_bytes + (size_t)hk * D * sizeof(T);
    const char* vb = (const char*)a.v + (size_t)s.start * a.v_bytes + (size_t)hk * D * sizeof(T);
    auto fetch = [&](int t, int buf) {
        const int k0 = t * KT + w * RW;
        const int kat = k0 < s.n ? k0 : s.n - 1;
        Rows<T, D>::template fetch<RW>(lds[buf][0], w * RW, kb + (size_t)kat * a.k_bytes, a.k_bytes, s.n - 1 - kat);
        Rows<T, D>::template fetch<RW>(lds[buf][1], w * RW, vb + (size_t)kat * a.v_bytes, a.v_bytes, s.n - 1 - kat);
    };
    float over = 0.f;  // sum_j ds_ij of this lane's keys
    int rest0 = 0x7fffffff;  // from which key on the products may have left out keys (attn.h)
    // one tile; FIRST: only the row sums
    auto tile = [&](int t, int end, auto BUF, auto FIRST) {
        constexpr int buf = BUF();
        wait_vm<0>();
        __syncthreads();
        if (t + 1 < end) fetch(t + 1, buf ^ 1);
#pragma unroll
        for (int sub = 0; sub < KT / 32; ++sub) {
            const int key0 = t * KT + 32 * sub;
            if (key0 >= wmax) continue;
            f32x16 sc = zero16(), dp = zero16();
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) sc = mma32(Rows<T, D>::along(lds[buf][0], 32 * sub, kk), qf[kk], sc);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) dp = mma32(Rows<T, D>::along(lds[buf][1], 32 * sub, kk), df[kk], dp);
            // the keys' columns are read now, to arrive under the exponentials
            Frag<T> kd[2 * DT];
            if (!FIRST()) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
                        kd[b * DT + dt] = Rows<T, D>::down(lds[buf][0], 32 * sub + 16 * b, 32 * dt);
            }
            if (sizeof(T) == 2) {
                order_products<2 * KK, 1, 4>();
                if (!FIRST()) order_reads<4 * DT>();
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) dp[r] = exp2_hw(sc[r] * sl2 - lse2) * (dp[r] - delta);
            if (key0 + 32 > wmin) {
                if (!FIRST()) {
                    // a key that is not finite shows in its scores
                    float z = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) z = fmaf(sc[r], 0.f, z);
                    if (__builtin_expect(__any(z != z), 0)) {
                        rest0 = rest0 < key0 ? rest0 : key0;
#pragma unroll
                        for (int i = 0; i < 2 * DT; ++i) kd[i] = finite_only(kd[i]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    dp[r] = key0 + 8 * (r >> 2) + 4 * h + (r & 3) < limit ? dp[r] : 0.f;
            }
            if (sizeof(T) == 2) {
#pragma unroll
                for (int r = 0; r < 16; ++r) over += dp[r];
            }
            if (!FIRST()) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const Frag<T> ds = acc_frag<T>(dp, b);
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) dq[dt] = mma32(kd[b * DT + dt], ds, dq[dt]);
                }
            }
        }
    };
    auto round = [&](int from, int end, auto FIRST) {
        if (from < end) fetch(from, 0);
        for (int t = from; t < end; t += 2) {
            tile(t, end, std::integral_constant<int, 0>{}, FIRST);
            if (t + 1 < end) tile(t + 1, end, std::integral_constant<int, 1>{}, FIRST);
        }
    };
    if (sizeof(T) == 2 && tiles * KT <= SHORT) {
        round(0, tiles, std::true_type{});
        delta += half_add(over);
        over = 0.f;
        __syncthreads();  // all waves are done with the buffers
    }
    const int t0 = (int)((long long)tiles * part / a.qparts), t1 = (int)((long long)tiles * (part + 1) / a.qparts);
    round(t0, t1, std::false_type{});
    if (__builtin_expect(rest0 < wmax, 0)) {
#pragma unroll 1
        for (int j = rest0; j < wmax; ++j) add_nonfinite<T, D>(dq, (const T*)(kb + (size_t)j * a.k_bytes), j < limit);
    }
    if (sizeof(T) == 2 && part == 0) {
        // a piece of the keys does not have the whole row sum
        if (a.qparts == 1) delta += half_add(over);
        if (row < R && h == 0) {
            a.lse2[(size_t)hq * a.T + at] = lse2;
            a.delta[(size_t)hq * a.T + at] = delta;
        }
    }
    if (row < R) {
        const size_t out = (at * a.Hq + hq) * D;
        float* pq = a.qparts > 1 ? a.part_q + part * ((size_t)a.T * a.Hq * D) : nullptr;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) put4<T>((T*)a.dq, pq, out + 32 * dt + 8 * i + 4 * h, dq[dt], i, a.scale);
    }
}

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(BwdArgs a)
{
    __shared__ __align__(1024) QueryLds<T, D> m;
    query_pass<T, D>(a, blockIdx.x, m);
}

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_dkdv_kernel(BwdArgs a)
{
    __shared__ __align__(1024) KeyLds<T, D> m;
    key_pass<T, D>(a, blockIdx.x, m);
}

// fp32, whose delta needs no correction: both passes in one launch, the first
// `kblocks` workgroups for the keys.  A small batch (three prompts of up to 333
// tokens, 6 heads of 64) does not fill the card with either: forward and backward
// take 47 us, and 55 us in two launches.
template <int D>
__global__ __launch_bounds__(256, 1) void attn_grads_kernel(BwdArgs a, unsigned kblocks)
{
    __shared__ __align__(1024) union {
        KeyLds<float, D> k;
        QueryLds<float, D> q;
    } m;
    if (blockIdx.x < kblocks)
        key_pass<float, D>(a, blockIdx.x, m.k);
    else
        query_pass<float, D>(a, blockIdx.x - kblocks, m.q);
}

// fp32: delta and the log-sums in base 2, by query head; a row by D / 4 lanes
template <int D>
__global__ __launch_bounds__(256) void attn_delta_kernel(BwdArgs a)
{
    constexpr int L = D / 4;
    const size_t rows = (size_t)a.T * a.Hq;
    const size_t row = (size_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int c = (threadIdx.x % L) * 4;
    const size_t at = (row < rows ? row : rows - 1) * D + c;
    const f32x4 x = *reinterpret_cast<const f32x4*>((const float*)a.o + at);
    const f32x4 y = *reinterpret_cast<const f32x4*>((const float*)a.dO + at);
    float sum = lane16_sum((x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]));
    if (L == 32) sum += __shfl_xor(sum, 16);
    if (c == 0 && row < rows) {
        const size_t t = row / a.Hq, h = row % a.Hq;
        a.delta[h * a.T + t] = sum;
        a.lse2[h * a.T + t] = a.lse[row] * kLog2e;
    }
}

// out = f * sum of the np pieces' partial sums, in their order, for the rows of
// sequences; four values a thread.  Up to three outputs of one call.
struct SumArgs {
    const float* part[3];
    void* out[3];
    float f[3];
    int np[3], per_token[3];
    size_t n[3];
};

template <typename T>
__global__ __launch_bounds__(256) void attn_sum_kernel(const int* __restrict__ cu, int B, SumArgs a)
{
    const int y = blockIdx.y;
    const float* part = y == 0 ? a.part[0] : y == 1 ? a.part[1] : a.part[2];
    T* out = (T*)(y == 0 ? a.out[0] : y == 1 ? a.out[1] : a.out[2]);
    const float f = y == 0 ? a.f[0] : y == 1 ? a.f[1] : a.f[2];
    const int np = y == 0 ? a.np[0] : y == 1 ? a.np[1] : a.np[2];
    const int per = y == 0 ? a.per_token[0] : y == 1 ? a.per_token[1] : a.per_token[2];
    const size_t n = y == 0 ? a.n[0] : y == 1 ? a.n[1] : a.n[2];
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int tok = (int)(i / per);
    if (tok < cu[0] || tok >= cu[B]) return;
    f32x4 s = *reinterpret_cast<const f32x4*>(part + i);
#pragma unroll 4
    for (int p = 1; p < np; ++p) s += *reinterpret_cast<const f32x4*>(part + p * n + i);
    store4<T>(out + i, s[0] * f, s[1] * f, s[2] * f, s[3] * f);
}

// workgroups of a pass over `heads` rows a token (query pass: the query heads of a
// key head, key pass: 1), each block's work cut into `parts`
long long pass_blocks(int T, int heads, int B, int Hkv, int parts)
{
    return ((long long)T * heads / 128 + B) * Hkv * parts;
}
// workgroups of attn_delta_kernel
long long delta_blocks(int T, int Hq, int D) { return ((long long)T * Hq + 1024 / D - 1) / (1024 / D); }

template <typename T, int D>
gdn_status launch(const BwdArgs& a, hipStream_t st)
{
    const unsigned qblocks = (unsigned)pass_blocks(a.T, a.G, a.B, a.Hkv, a.qparts);
    const unsigned kblocks = (unsigned)pass_blocks(a.T, 1, a.B, a.Hkv, a.kparts);
    if constexpr (sizeof(T) == 4) {
        GDN_LAUNCH("attn_delta", attn_delta_kernel<D>, dim3((unsigned)delta_blocks(a.T, a.Hq, D)), dim3(256), st, a);
        GDN_LAUNCH("attn_grads", attn_grads_kernel<D>, dim3(kblocks + qblocks), dim3(256), st, a, kblocks);
    } else {
        GDN_LAUNCH("attn_dq", (attn_dq_kernel<T, D>), dim3(qblocks), dim3(256), st, a);
        GDN_LAUNCH("attn_dkdv", (attn_dkdv_kernel<T, D>), dim3(kblocks), dim3(256), st, a);
    }
    SumArgs m{};
    int n = 0;
    size_t most = 0;
    auto add = [&](const float* part, void* out, float f, int np, int heads) {
        m.part[n] = part; m.out[n] = out; m.f[n] = f; m.np[n] = np; m.per_token[n] = heads * D;
        m.n[n] = (size_t)a.T * heads * D;
        most = most > m.n[n] ? most : m.n[n];
        ++n;
    };
    if (a.kparts > 1) {
        add(a.part_k, a.dk, a.scale, a.kparts, a.Hkv);
        add(a.part_k + (size_t)a.kparts * a.T * a.Hkv * D, a.dv, 1.f, a.kparts, a.Hkv);
    }
    if (a.qparts > 1) add(a.part_q, a.dq, a.scale, a.qparts, a.Hq);
    if (n)
        GDN_LAUNCH("attn_sum", attn_sum_kernel<T>, dim3((unsigned)((most / 4 + 255) / 256), n), dim3(256), st, a.cu, a.B, m);
    return GDN_OK;
}

// How the work of a block is cut up: until there are `want` workgroups (key pass of
// eight packed prompts, 288 blocks, 563 us in all with four pieces: with three 5 %
// longer, whole 39 %), but
// pieces of `least` tiles at least (on average: `tiles` are those of a middle block).
int parts_for(long long blocks, long long want, long long tiles, long long least, int most)
{
    long long p = (want + blocks - 1) / blocks;
    p = p > tiles / least ? tiles / least : p;
    return p < 1 ? 1 : p > most ? most : (int)p;
}

struct BwdPlan {
    int kparts, qparts;
    size_t o_delta, o_k, o_q, bytes;
};

BwdPlan bwd_plan(const gdn_attn_shape& s)
{
    BwdPlan p;
    const long long G = s.Hq / s.Hkv, len = s.T / s.B;
    const long long kb = ((long long)s.T + 127) / 128, qb = ((long long)s.T * G + 127) / 128;
    const int kt = s.dtype == GDN_BF16 ? 64 : 32;
    // a key block's work falls with its place in the sequence, so the first
    // blocks decide the end unless there are several workgroups a compute unit
    // (fp32, whose tiles take eight times as long, goes down to one tile a piece)
    const int least = s.dtype == GDN_BF16 ? 2 : 1;
    p.kparts = parts_for((kb > s.B ? kb : s.B) * s.Hkv, 1024, G * (len / 2 + 32) / 32, least, 16);
    p.qparts = parts_for((qb > s.B ? qb : s.B) * s.Hkv, 512, (len / 2 + kt) / kt, least, 16);
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const size_t f = sizeof(float), rows = (size_t)s.T * s.Hq;
    p.o_delta = up(rows * f);
    p.o_k = p.o_delta + up(rows * f);
    p.o_q = p.o_k + (p.kparts > 1 ? up(2 * p.kparts * (size_t)s.T * s.Hkv * s.D * f) : 0);
    p.bytes = p.o_q + (p.qparts > 1 ? up(p.qparts * rows * s.D * f) : 0);
    return p;
}

}  // namespace

size_t attn_backward_ws(const gdn_attn_shape& s) { return bwd_plan(s).bytes; }

bool attn_backward_fits(const gdn_attn_shape& s)
{
    const BwdPlan p = bwd_plan(s);
    const long long most = (1LL << 24) - 1;  // of 256 work-items each
    const long long kb = pass_blocks(s.T, 1, s.B, s.Hkv, p.kparts);
    const long long qb = pass_blocks(s.T, s.Hq / s.Hkv, s.B, s.Hkv, p.qparts);
    if (s.dtype == GDN_F32) return kb + qb <= most && delta_blocks(s.T, s.Hq, s.D) <= most;
    return kb <= most && qb <= most;
}

gdn_status attn_backward_dispatch(const gdn_attn_shape& s, const void* q, const void* k, const void* v, const int* cu,
                                  const void* o, const float* lse, const void* dO, void* dq, void* dk, void* dv,
                                  void* ws, hipStream_t st)
{
    const uint32_t e = s.dtype == GDN_BF16 ? 2 : 4;
    BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.dO = dO; a.lse = lse; a.cu = cu;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.lse2 = (float*)ws;
    const BwdPlan p = bwd_plan(s);
    a.delta = (float*)((char*)ws + p.o_delta);
    a.part_k = (float*)((char*)ws + p.o_k);
    a.part_q = (float*)((char*)ws + p.o_q);
    a.kparts = p.kparts;
    a.qparts = p.qparts;
    a.q_stride = s.q_stride;
    a.q_bytes = (uint32_t)(s.q_stride * e);
    a.k_bytes = (uint32_t)(s.k_stride * e);
    a.v_bytes = (uint32_t)(s.v_stride * e);
    a.o_bytes = (uint32_t)(s.Hq * s.D * e);
    a.B = s.B; a.T = s.T; a.Hq = s.Hq; a.Hkv = s.Hkv; a.G = s.Hq / s.Hkv;
    a.scale = s.scale;
    if (s.dtype == GDN_BF16) return s.D == 64 ? launch<bf16, 64>(a, st) : launch<bf16, 128>(a, st);
    return s.D == 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}

}  // namespace gdn
