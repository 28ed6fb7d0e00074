// ssm_tile.h -- device code that the state space scan's kernels share: chunks of
// packed sequences, the decays of a chunk, split operands.  Tiles, tables and
// fragments are those of attn.h.
#pragma once

#include "attn.h"
#include "bounds.h"
#include "ssm.h"

namespace gdn {

template <typename T> struct SsmTile;
template <> struct SsmTile<bf16> {
    static constexpr int L = 128;
    // An fp32 value as the sum of three bf16: 8 + 8 + 8 bits, so that the product with
    // a bf16 operand is as exact as in fp32.  The states are products of this kind.
    static constexpr int PARTS = 3;
};
template <> struct SsmTile<float> {
    static constexpr int L = 64;
    static constexpr int PARTS = 1;
};

// Units of `len` tokens (chunks, segments) of packed sequences, in the order of
// the sequences.  A sequence has `count` of them, of which count - drop are dealt out,
// `least` at least (drop < 0: one, if there are several).  Unit `id` of those: the at-th
// of sequence b, whose rows are start .. start + n - 1; chunks: of the sequence; first:
// the units of those with several, before, between: the chunks and the states between
// chunks, of all sequences before it.
struct Unit {
    int b, at, count, start, n, chunks;
    long long first, before, between;
};
template <int L>
__device__ __forceinline__ bool find_unit(const int* __restrict__ cu, int B, int T, int len, int drop, int least, long long id,
                                          Unit& u)
{
    const int l = lane_id();
    long long dealt = 0, first = 0, between = 0, chunks = 0;
    int top = 0, st, en;
    for (int b0 = 0; b0 < B; b0 += 64) {
        ordered_bounds(cu, B, T, b0, top, st, en);
        const bool real = b0 + l < B;
        const int n = en - st, ch = real ? (n + L - 1) / L : 0, count = real ? (n + len - 1) / len : 0;
        const int several = count > 1 ? count : 0, nbt = ch > 1 ? ch - 1 : 0;
        const int nu = !real ? 0 : drop < 0 ? several > 0 : count - drop < least ? least : count - drop;
        const int inc = wave_scan(nu), incf = wave_scan(several), incb = wave_scan(nbt), incc = wave_scan(ch);
        const uint64_t hit = __ballot(dealt + inc > id);
        if (hit) {
            const int k = __builtin_ctzll(hit);
            auto here = [&](int x) { return __builtin_amdgcn_readlane(x, k); };
            u.b = b0 + k;
            u.count = here(count);
            u.at = (int)(id - dealt) - (here(inc) - here(nu));
            u.start = here(st);
            u.n = here(n);
            u.chunks = here(ch);
            u.first = first + here(incf) - here(several);
            u.before = chunks + here(incc) - u.chunks;
            u.between = between + here(incb) - here(nbt);
            return true;
        }
        dealt += __builtin_amdgcn_readlane(inc, 63);
        first += __builtin_amdgcn_readlane(incf, 63);
        between += __builtin_amdgcn_readlane(incb, 63);
        chunks += __builtin_amdgcn_readlane(incc, 63);
    }
    return false;
}

// Workgroup -> (unit, slice).  Workgroups go to the 8 dies in turn; four slices of a
// unit, which read the same B and C, are one die's, and the dies have equal numbers (a
// unit's slices all on one: up to 72 of 480 workgroups on a die with room for 64 at a
// time, and nearly twice the time).  The grid is a multiple of 32.
__device__ __forceinline__ void deal(long long id, int slices, long long& unit, int& slice)
{
    const long long k = id >> 3, flat = ((k >> 2) * 8 + (id & 7)) * 4 + (k & 3);
    unit = flat / slices;
    slice = (int)(flat - unit * slices);
}
inline unsigned dealt(long long units, int slices) { return (unsigned)((units * slices + 31) / 32 * 32); }

// log(1 + exp(v)), v itself from where they agree in fp32
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// What ssm_prep.hip leaves of a chunk and head, a row of L values each, and behind
// them exp(c_L) and its logarithm.  c is the running sum of log2 exp(g): its
// differences are small and it is not, so it comes as two floats whose sum has
// 48 bits.  Blocks are of 32 tokens; E_ts of t in a later block than s is
// AHEAD_t exp(c at the start of t's block - c at the end of s's) BEHIND_s, factors
// that decay throughout, so that a pair costs a product and no exponential.
enum { DEC_HI, DEC_LO, DEC_DELTA, DEC_E, DEC_F, DEC_FD, DEC_AHEAD, DEC_BEHIND, DEC_ROWS };
template <int L> constexpr int kDecays = DEC_ROWS * L + 4;  // floats a chunk and head
enum { DEC_KEEP, DEC_TOTAL };
//   E: exp(c), F: exp(c_L - c), FD: that times delta, AHEAD: exp(c - c before the block), BEHIND: exp(c at
//   the block's end - c); behind the last token delta and E are 0 and c stays as it is

// What ssm_grad.hip leaves of a chunk and head for the steps' gradients, a row of L
// values each: sums of r from the state before and from earlier blocks, of q / delta
// into the state behind and into later blocks, the pairs of the token's own block
// that pass over it, x . du and x . dy.  Behind them <S, dS> by block, and, in chunks of
// four blocks, the sums of the pairs between blocks (2, 0), (3, 0), and (3, 0) + (3, 1).
enum { TOK_R_STATE, TOK_R_BLOCKS, TOK_Q_STATE, TOK_Q_BLOCKS, TOK_OWN, TOK_XDU, TOK_XDY, TOK_ROWS };
template <int L> constexpr int kTokens = TOK_ROWS * L + 8;  // floats a chunk and head

// v as three bf16 each: the upper 8 bits of its 24, the next, the rest.  Cut off and
// not rounded, which leaves all bits and takes fewer instructions; the first one
// rounded (NEAREST) where it also stands for v by itself.
__device__ __forceinline__ uint32_t upper_halves(float a, float b)  // of a in the low half
{
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float upper(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
template <bool NEAREST = false> __device__ __forceinline__ void split(const float (&v)[8], u32x4 (&w)[3])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
        if constexpr (NEAREST) {
            w[0][i] = cvt2_bf16(a, b);
            a -= __uint_as_float(w[0][i] << 16), b -= upper(__uint_as_float(w[0][i]));
        } else {
            w[0][i] = upper_halves(a, b);
            a -= upper(a), b -= upper(b);
        }
        w[1][i] = upper_halves(a, b);
        a -= upper(a), b -= upper(b);
        w[2][i] = upper_halves(a, b);
    }
}

// a wave-uniform address in LDS as its offset there, and dma16_at (attn.h) to one
__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p);
}
__device__ __forceinline__ void dma16_to(const void* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}

// A state of N rows of 64 values in memory, as the walk's lanes hold it: value p of
// row n at (n / 4) 256 + 4 p + n % 4.  Eight rows of one value, from the two runs of
// four, are a word of bf16 (or two of fp32) of a table of 64 rows p along n.
__device__ __forceinline__ void load_state8(const float* s, int n, int p, float (&v)[8])
{
    const f32x4 a = *reinterpret_cast<const f32x4*>(s + n * kSlice + 4 * p), b = *reinterpret_cast<const f32x4*>(s + (n + 4) * kSlice + 4 * p);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
}

// Reads of a row table (Rows) from a lane's byte offset, all others of a kind being
// that offset with bits of the word index flipped: a kernel short of registers keeps
// the offset opaque in its loops, so that the others are formed on the way.
//   along:  an operand's rows along their values          (plain order, Rows::along)
//   down:   an operand's columns down 16 rows             (permuted order, Rows::down)
//   plain:  the same in plain order, to go with along
//   row4:   four values of a lane's own row, those of accumulator registers 4 i .. + 3
template <typename T, int D> struct Reads {
    using R = Rows<T, D>;
    static constexpr int BYTES = R::BYTES;
    typedef short s16x4 __attribute__((ext_vector_type(4)));

    static __device__ __forceinline__ uint32_t down_at() { return lane_at(4 * (lane_id() >> 5)); }
    static __device__ __forceinline__ uint32_t plain_at() { return lane_at(8 * (lane_id() >> 5)); }
    static __device__ __forceinline__ Frag<T> down(const void* tab, uint32_t at, int k0, int d0)
    {
        if constexpr (sizeof(T) == 2)
            return pair<8, 2>(tab, at, k0, d0);  // rows 8 t + 4 h + .. : bit 1 of the row's flips is t
        else
            return R::down(tab, k0, d0);
    }
    static __device__ __forceinline__ Frag<T> plain(const void* tab, uint32_t at, int k0, int d0)
    {
        if constexpr (sizeof(T) == 2) {
            return pair<4, 1>(tab, at, k0, d0);  // rows 8 h + 4 t + ..
        } else {
            const int l = lane_id(), c = d0 + (l & 31);
            const float* t = reinterpret_cast<const float*>(tab) + k0 * R::U * 4;
            f32x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = t[R::word(8 * (l >> 5) + j, c >> 2) * 4 + (c & 3)];
            return v;
        }
    }
    static __device__ __forceinline__ uint32_t row_at(int r)
    {
        const uint32_t h = lane_id() >> 5;
        return sizeof(T) == 2 ? (uint32_t)R::word(r, 0) * 16 + 8 * h : (uint32_t)R::word(r, h) * 16;
    }
    // values 32 i + 8 q + 4 h .. + 3
    static __device__ __forceinline__ f32x4 row4(const void* tab, uint32_t at, int i, int q)
    {
        const char* p = reinterpret_cast<const char*>(tab);
        if constexpr (sizeof(T) == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + (at ^ ((4 * i + q) << 4)));
            return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u)};
        } else {
            return *reinterpret_cast<const f32x4*>(p + (at ^ ((8 * i + 2 * q) << 4)));
        }
    }

private:
    static __device__ __forceinline__ uint32_t lane_at(int row)
    {
        const int l = lane_id(), i = l & 15, c = 16 * ((l >> 4) & 1) + 4 * (i & 3);
        return (uint32_t)R::word(row + (i >> 2), c >> 3) * 16 + (c & 7) * 2;
    }
    template <int ROWS, int FLIP>
    static __device__ __forceinline__ bf16x8 pair(const void* tab, uint32_t at, int k0, int d0)
    {
        const char* p = reinterpret_cast<const char*>(tab) + k0 * BYTES;
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(p + t * ROWS * BYTES + (at ^ (uint32_t)(((d0 >> 3) ^ (t * FLIP)) << 4))));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Pairs within a block of 32 tokens are masked: a token may depend on the block's later
// (or earlier) ones through products with 0, and an infinity or a NaN times that would
// reach it.  Where a block has such rows, the products take finite ones (finite_only),
// and what those leave out is added here, times the lane's weight: w holds the weights
// of the block's rows (row0 .. + 31 of the table), `later`: the lane's token takes the
// rows from its own on, otherwise those up to its own.
template <typename T, int D>
__device__ __forceinline__ void add_masked_rest(f32x16 (&acc)[D / 32], const f32x16& w, const void* tab, int row0, bool later)
{
    const int l = lane_id(), t = l & 31;
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {  // rare: with few registers, not fast
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) mine = r == 4 * (j >> 3) + (j & 3) ? w[r] : mine;
        mine = __shfl(mine, t | (j & 4) << 3);
        const uint32_t at = Reads<T, D>::row_at(row0 + j);
        const bool takes = later ? j >= t : j <= t;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 x = Reads<T, D>::row4(tab, at, i, q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (takes && !(fabsf(x[k]) < INFINITY)) acc[i][4 * q + k] += mine * x[k];
            }
        }
    }
}

// rows of a tile's accumulator registers 4 i .. 4 i + 3: 8 i + 4 h + 0 .. 3
__device__ __forceinline__ int acc_rows(int i, int l = lane_id()) { return 8 * i + 4 * (l >> 5); }

}  // namespace gdn
