// attn.h -- what the softmax-attention kernels share: 32 x 32 tiles on the
// matrix cores, row tables in LDS, and the way a workgroup finds its rows.
//
// Fragments.  An operand fragment holds 8 values a lane: lane l (m = l % 32,
// h = l / 32), element j, is operand row (A) or column (B) m at contraction
// index kappa(h, j) of a 16-long block.  Any kappa gives the same product as
// long as A and B agree on it; two are used:
//   plain:    kappa = 8 h + j                      (operands read along their rows)
//   permuted: kappa = 8 (j / 4) + 4 h + j % 4      (accumulators fed back as operands)
// bf16 takes one v_mfma_f32_32x32x16_bf16 a fragment pair, fp32 eight
// v_mfma_f32_32x32x2_f32, the j-th over element j of both.
// Accumulator: lane l holds column l % 32, rows 8 (r / 4) + 4 h + r % 4 in
// acc[r], r = 0..15: registers 8 b .. 8 b + 7 are, in the permuted order, the
// 16 rows from 16 b.  So with scores computed as S^T = K Q^T (a lane is one
// query, its registers are keys) a lane's probabilities are the next product's
// operand as they stand, and a row's maximum and sum need one exchange between
// the lane halves.
#pragma once

#include "common.h"
#include "attn_plan.h"

namespace gdn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <typename T> struct FragOf;
template <> struct FragOf<bf16> { typedef bf16x8 type; };
template <> struct FragOf<float> { typedef f32x8 type; };
template <typename T> using Frag = typename FragOf<T>::type;

__device__ __forceinline__ __bf16 frag_value(bf16 x) { return __builtin_bit_cast(__bf16, x.bits); }
__device__ __forceinline__ float frag_value(float x) { return x; }

__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f32x8 a, f32x8 b, f32x16 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 zero16()
{
    return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// registers 8 b .. 8 b + 7 of an accumulator as an operand (permuted order)
template <typename T> __device__ __forceinline__ Frag<T> acc_frag(const f32x16& s, int b);
template <> __device__ __forceinline__ bf16x8 acc_frag<bf16>(const f32x16& s, int b)
{
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt2_bf16(s[8 * b + 2 * i], s[8 * b + 2 * i + 1]);
    return __builtin_bit_cast(bf16x8, w);
}
template <> __device__ __forceinline__ f32x8 acc_frag<float>(const f32x16& s, int b)
{
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s[8 * b + i];
    return v;
}

// a fragment in plain order from 8 values in memory, 16-byte aligned
template <typename T> __device__ __forceinline__ Frag<T> load_frag(const T* p);
template <> __device__ __forceinline__ bf16x8 load_frag<bf16>(const bf16* p)
{
    return *reinterpret_cast<const bf16x8*>(p);
}
template <> __device__ __forceinline__ f32x8 load_frag<float>(const float* p)
{
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Masked pairs.  A value that a row does not depend on must not reach it, and a
// product of an infinity or a NaN with the pair's 0 would.  So where a masked tile
// holds such values, its products take finite ones instead (finite_only), and the
// rows that do depend on them get them after the last tile (add_nonfinite).  Tiles
// without a masked pair go through the products as they are.
//
// Whether all of a wave's fragments are finite.  bf16: by their products with 0,
// which are 0 or NaN (in any assignment of rows), a matrix instruction a fragment.
template <int N> __device__ __forceinline__ bool all_finite(const bf16x8 (&v)[N])
{
    f32x4 z = zero4();
#pragma unroll
    for (int i = 0; i < N; ++i)
        z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[i], __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}), z, 0, 0, 0);
    const float s = (z[0] + z[1]) + (z[2] + z[3]);
    return !__any(s != s);
}
// fp32: by the sum of the products with 0, an operation a value.
template <int N> __device__ __forceinline__ bool all_finite(const f32x8 (&v)[N])
{
    f32x4 z = zero4();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j & 3] = __builtin_fmaf(v[i][j], 0.f, z[j & 3]);
    const float s = (z[0] + z[1]) + (z[2] + z[3]);
    return !__any(s != s);
}

// a fragment with infinities and NaN as finite values of the largest magnitude,
// whose product with the 0 of a masked pair is 0
__device__ __forceinline__ bf16x8 finite_only(bf16x8 v)
{
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // without the sign bit a signed minimum, with it an unsigned one
        const uint32_t x = w[i];
        const s16x2 a = __builtin_elementwise_min(__builtin_bit_cast(s16x2, x), s16x2{0x7f7f, 0x7f7f});
        const u16x2 b = __builtin_elementwise_min(__builtin_bit_cast(u16x2, a), u16x2{0xff7f, 0xff7f});
        w[i] = __builtin_bit_cast(uint32_t, b);
    }
    return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ f32x8 finite_only(f32x8 v)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(v[i], -3.402823466e38f, 3.402823466e38f);
    return v;
}

// The infinities and NaN of a row of D values into the accumulators of the lanes
// whose column depends on it.  Where the products did take them, that changes nothing.
template <typename T, int D>
__device__ __forceinline__ void add_nonfinite(f32x16 (&acc)[D / 32], const T* row, bool depends)
{
    const int h = lane_id() >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
        __builtin_amdgcn_sched_barrier(0);  // rare: with few registers, not fast
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float x = to_f32(row[32 * dt + 8 * (r >> 2) + 4 * h + (r & 3)]);
            if (depends && !(fabsf(x) < INFINITY)) acc[dt][r] += x;
        }
    }
}

// four accumulator rows of one column, stored as four neighbours
template <typename T> __device__ __forceinline__ void store4(T* p, float a, float b, float c, float d);
template <> __device__ __forceinline__ void store4<bf16>(bf16* p, float a, float b, float c, float d)
{
    *reinterpret_cast<uint2*>(p) = uint2{cvt2_bf16(a, b), cvt2_bf16(c, d)};
}
template <> __device__ __forceinline__ void store4<float>(float* p, float a, float b, float c, float d)
{
    *reinterpret_cast<f32x4*>(p) = f32x4{a, b, c, d};
}

// the value of lane l and of lane l ^ 32, the same pair in both
__device__ __forceinline__ float2 half_pair(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return float2{__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ float half_max(float x)
{
    const float2 p = half_pair(x);
    return fmaxf(p.x, p.y);
}
__device__ __forceinline__ float half_add(float x)
{
    const float2 p = half_pair(x);
    return p.x + p.y;
}

// dma16 (common.h) from a wave-uniform base plus a 32-bit byte offset a lane
__device__ __forceinline__ void dma16_at(const void* base, uint32_t off, const void* lds_wave_base)
{
    const uint32_t m0v = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)lds_wave_base);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0v), "v"(off), "s"(base)
                 : "memory", "m0");
}

// ---------------------------------------------------------------------------
// row tables in LDS: rows of D elements, U = D sizeof(T) / 16 words of 16
// bytes; word u of row r sits at word r U + (u ^ f(r)).  f is a permutation of
// the row bits that decide a bank group, so that both reads below meet every
// bank group once: 16-byte reads of 16 of 32 consecutive rows (a phase is the
// lanes with equal bit 5 and equal parity of bits 2..4), and transposing reads
// of four consecutive rows.
// ---------------------------------------------------------------------------
template <typename T, int D>
struct Rows {
    static constexpr int U = D * (int)sizeof(T) / 16;
    static constexpr int BYTES = U * 16;
    static constexpr int PER = 64 / U;  // rows a wave's 64 words hold
    static_assert(U == 8 || U == 16 || U == 32, "head size");
    static __device__ __forceinline__ int f(int r)
    {
        return U == 8 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r & 3) << 2 | ((r >> 2) & 3);
    }
    static __device__ __forceinline__ int word(int r, int u) { return r * U + (u ^ f(r)); }

    // Operand rows r0 .. r0 + 31 (r0 a multiple of 16, so that f does not see it)
    // along their own values 16 kk .. + 15, plain order.  `at` is along_at(), the
    // lane's byte offset at kk = 0: the others differ from it in bits of the word
    // index alone.  A kernel short of registers keeps `at` opaque in its loop, so
    // that the offsets are formed on the way instead of being held.
    static __device__ __forceinline__ uint32_t along_at()
    {
        const int l = lane_id(), r = l & 31, h = l >> 5;
        return (uint32_t)word(r, sizeof(T) == 2 ? h : 2 * h) * 16;
    }
    static __device__ __forceinline__ Frag<T> along(const void* tab, uint32_t at, int r0, int kk)
    {
        const char* t = reinterpret_cast<const char*>(tab) + r0 * BYTES;
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const bf16x8*>(t + (at ^ (kk << 5)));
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(t + (at ^ (kk << 6)));
            const f32x4 b = *reinterpret_cast<const f32x4*>(t + (at ^ (kk << 6) ^ 16));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    static __device__ __forceinline__ Frag<T> along(const void* tab, int r0, int kk)
    {
        return along(tab, along_at(), r0, kk);
    }

    // operand columns d0 .. d0 + 31 down rows k0 .. k0 + 15 (k0 a multiple of 16), permuted order.
    // bf16: two transposing loads; in one, lane i of a group of 16 receives
    // element i % 4 of what lanes 4 e + i / 4 read, e = 0..3, so lane i reads
    // row i / 4 at columns 4 (i % 4) and gets column i of the four rows.
    static __device__ __forceinline__ Frag<T> down(const void* tab, int k0, int d0)
    {
        const int l = lane_id(), h = l >> 5;
        if constexpr (sizeof(T) == 2) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            const int i = l & 15, c = d0 + 16 * ((l >> 4) & 1) + 4 * (i & 3);
            s16x4 v[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int r = 8 * t + 4 * h + (i >> 2);
                const char* p = reinterpret_cast<const char*>(tab) + k0 * BYTES + word(r, c >> 3) * 16 + (c & 7) * 2;
                v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
            }
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int c = d0 + (l & 31);
            const float* t = reinterpret_cast<const float*>(tab) + k0 * U * 4;
            f32x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 8 * (j >> 2) + 4 * h + (j & 3);
                v[j] = t[word(r, c >> 2) * 4 + (c & 3)];
            }
            return v;
        }
    }

    // Rows r0 .. r0 + N - 1 of a table from global memory, by direct loads of the
    // calling wave (N / PER of them): row r comes from `base` + min(r - r0, last)
    // * stride bytes.  r0 is a multiple of N, N of PER; base, stride and last are
    // the same in all lanes.  Away from a sequence's end the lanes' offsets do
    // not change from call to call: only the scalar base moves.
    template <int N>
    static __device__ __forceinline__ void fetch(void* tab, int r0, const void* base, uint32_t stride, int last,
                                                 int l = lane_id())
    {
        char* to = reinterpret_cast<char*>(tab) + r0 * BYTES;
        if (last >= N - 1) {
#pragma unroll
            for (int i = 0; i < N / PER; ++i) {
                const int rr = i * PER + l / U;
                dma16_at(base, (uint32_t)rr * stride + (uint32_t)((l % U) ^ f(r0 + rr)) * 16, to + i * PER * BYTES);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / PER; ++i) {
                const int rr = i * PER + l / U;
                dma16_at(base, (uint32_t)(rr < last ? rr : last) * stride + (uint32_t)((l % U) ^ f(r0 + rr)) * 16,
                         to + i * PER * BYTES);
            }
        }
    }
    // zeros in the same places
    template <int N>
    static __device__ __forceinline__ void clear(void* tab, int r0)
    {
        u32x4* t = reinterpret_cast<u32x4*>(tab) + r0 * U;
#pragma unroll
        for (int i = 0; i < N / PER; ++i) t[i * 64 + lane_id()] = u32x4{0, 0, 0, 0};
    }
};

// 4-byte direct load into LDS: lane i's word lands at lds_wave_base + 4 i
__device__ __forceinline__ void dma4(const void* gptr, const void* lds_wave_base)
{
    warm_line(gptr, lds_wave_base);
}

// Order of issue within a block of code: the next N LDS reads, the next N matrix
// instructions.  Left alone the compiler reads an operand into the registers that
// the last one has just left, and every matrix instruction waits out an LDS
// latency; the kernels keep four operands ahead.
template <int N> __device__ __forceinline__ void order_reads() { __builtin_amdgcn_sched_group_barrier(0x100, N, 0); }
template <int N> __device__ __forceinline__ void order_mma() { __builtin_amdgcn_sched_group_barrier(0x008, N, 0); }
// N products of one read (R instructions) each, P operands ahead
template <int N, int R, int P> __device__ __forceinline__ void order_products()
{
    constexpr int A = P < N ? P : N;
    order_reads<A * R>();
#pragma unroll
    for (int i = 0; i < N - A; ++i) {
        order_mma<1>();
        order_reads<R>();
    }
    order_mma<A>();
}

// x, of which the compiler no longer knows where it comes from
__device__ __forceinline__ uint32_t opaque(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// value of a wave-uniform integer in a scalar register
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Sum and maximum over the wave, and the sum over the lanes up to and with the
// lane itself, by DPP moves (a workgroup begins with up to a dozen of these:
// through the LDS crossbar each kernel took 0.6 us longer).
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp_or_zero(int x)
{
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_sum(int x)
{
    x += dpp_or_zero<0xB1, 0xF>(x);   // quad_perm [1,0,3,2]
    x += dpp_or_zero<0x4E, 0xF>(x);   // quad_perm [2,3,0,1]
    x += dpp_or_zero<0x141, 0xF>(x);  // row_half_mirror
    x += dpp_or_zero<0x140, 0xF>(x);  // row_mirror
    return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) + __builtin_amdgcn_readlane(x, 32) +
           __builtin_amdgcn_readlane(x, 48);
}
__device__ __forceinline__ int wave_max(int x)  // of values >= 0
{
    auto up = [](int a, int b) { return a > b ? a : b; };
    x = up(x, dpp_or_zero<0xB1, 0xF>(x));
    x = up(x, dpp_or_zero<0x4E, 0xF>(x));
    x = up(x, dpp_or_zero<0x141, 0xF>(x));
    x = up(x, dpp_or_zero<0x140, 0xF>(x));
    return up(up(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
              up(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}
__device__ __forceinline__ float wave_sum(float x)
{
    x = lane16_sum(x);
    const int u = __builtin_bit_cast(int, x);
    auto at = [u](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, l)); };
    return (at(0) + at(16)) + (at(32) + at(48));
}
__device__ __forceinline__ int wave_scan(int x)
{
    x += dpp_or_zero<0x111, 0xF>(x);  // row_shr:1, 2, 4, 8: within the rows of 16
    x += dpp_or_zero<0x112, 0xF>(x);
    x += dpp_or_zero<0x114, 0xF>(x);
    x += dpp_or_zero<0x118, 0xF>(x);
    x += dpp_or_zero<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
    x += dpp_or_zero<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
    return x;
}

// ---------------------------------------------------------------------------
// Packed sequences: sequence b has the rows cu[b] .. cu[b + 1] - 1.  The bounds
// are device data: they are clamped to 0 <= start <= end <= T, so that no value
// of theirs reaches outside the buffers.
// ---------------------------------------------------------------------------
struct Span {
    int b, start, n;
    int level, blocks;  // the block's place and the number of the sequence's blocks
};

// Block `id` of all sequences' blocks of BR rows, a sequence of n tokens having
// n * G rows; every wave finds it by itself.  False: there is no such block.
// BY_LEVEL, up to 64 sequences: the blocks come in the order of their level, the
// highest first, across sequences: a causal prompt's block has work in
// proportion to its level, and the largest pieces first is what lets a grid end
// evenly (eight packed prompts of up to 4096 tokens, forward and backward, take 10 %
// longer with the sequences one after the other).  Otherwise the sequences come
// one after the other, each from its highest level down, which keeps the blocks
// that share keys together (chunks of new tokens over a cache take 22 % longer by
// level).
template <bool BY_LEVEL>
__device__ __forceinline__ bool find_block(const int* __restrict__ cu, int B, int T, int G, int BR, int id, Span& s)
{
    const int l = lane_id();
    auto bounds = [&](int b0, int& st, int& en) {
        const int b = b0 + l < B ? b0 + l : B - 1;
        st = cu[b], en = cu[b + 1];
        st = st < 0 ? 0 : st > T ? T : st;
        en = en < st ? st : en > T ? T : en;
        return b0 + l < B ? (int)(((long long)(en - st) * G + BR - 1) / BR) : 0;
    };
    auto take = [&](int b0, int lane, int level, int st, int en, int nb) {
        s.b = b0 + lane;
        s.start = __builtin_amdgcn_readlane(st, lane);
        s.n = __builtin_amdgcn_readlane(en, lane) - s.start;
        s.blocks = __builtin_amdgcn_readlane(nb, lane);
        s.level = level;
    };
    int st, en;
    if (BY_LEVEL && B <= 64) {
        const int nb = bounds(0, st, en);
        if (id >= wave_sum(nb)) return false;
        // the level j with above(j + 1) <= id < above(j), above(j) the number of blocks at level j and higher
        int lo = 0, hi = wave_max(nb), past = 0;
        while (hi - lo > 1) {  // above(lo) > id >= above(hi)
            const int mid = (lo + hi) >> 1;
            const int n = wave_sum(nb > mid ? nb - mid : 0);
            if (n > id) {
                lo = mid;
            } else {
                hi = mid;
                past = n;
            }
        }
        uint64_t have = __ballot(nb > lo);
        for (int i = id - past; i > 0; --i) have &= have - 1;
        take(0, __builtin_ctzll(have), lo, st, en, nb);
        return true;
    }
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int nb = bounds(b0, st, en);
        const int inc = wave_scan(nb);
        const uint64_t hit = __ballot(before + inc > id);
        if (hit) {
            const int first = __builtin_ctzll(hit);
            take(b0, first, before + __builtin_amdgcn_readlane(inc, first) - 1 - id, st, en, nb);
            return true;
        }
        before += __builtin_amdgcn_readlane(inc, 63);
    }
    return false;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace gdn
