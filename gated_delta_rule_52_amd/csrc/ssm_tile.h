// ssm_tile.h -- device code that the state space scan's kernels share: chunks of
// packed sequences, the decays of a chunk, split operands.  Tiles, tables and
// fragments are those of attn.h.
#pragma once

#include "attn.h"
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
// the sequences.  Unit `id`: the at-th of `count` of sequence b, whose rows are
// start .. start + n - 1; chunks: of the sequence; between: states between chunks
// in all sequences before it.  Every sequence has `least` units or more.
struct Unit {
    int b, at, count, start, n, chunks;
    long long between;
};
template <int L>
__device__ __forceinline__ bool find_unit(const int* __restrict__ cu, int B, int T, int len, int least, long long id, Unit& u)
{
    const int l = lane_id();
    long long before = 0, between = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int b = b0 + l < B ? b0 + l : B - 1;
        int st = cu[b], en = cu[b + 1];
        st = st < 0 ? 0 : st > T ? T : st;
        en = en < st ? st : en > T ? T : en;
        const int n = en - st, ch = (n + L - 1) / L;
        int nu = (n + len - 1) / len;
        nu = b0 + l < B ? (nu < least ? least : nu) : 0;
        const int nbt = b0 + l < B && ch > 1 ? ch - 1 : 0;
        const int inc = wave_scan(nu), incb = wave_scan(nbt);
        const uint64_t hit = __ballot(before + inc > id);
        if (hit) {
            const int first = __builtin_ctzll(hit);
            u.b = b0 + first;
            u.count = __builtin_amdgcn_readlane(nu, first);
            u.at = (int)(id - before) - (__builtin_amdgcn_readlane(inc, first) - u.count);
            u.start = __builtin_amdgcn_readlane(st, first);
            u.n = __builtin_amdgcn_readlane(n, first);
            u.chunks = __builtin_amdgcn_readlane(ch, first);
            u.between = between + __builtin_amdgcn_readlane(incb, first) - __builtin_amdgcn_readlane(nbt, first);
            return true;
        }
        before += __builtin_amdgcn_readlane(inc, 63);
        between += __builtin_amdgcn_readlane(incb, 63);
    }
    return false;
}

// Workgroup -> (unit, slice), the slices of a unit on one die: they read the same
// B and C, and workgroups go to the 8 dies in turn.  The grid is a multiple of 8 units.
__device__ __forceinline__ void deal(long long id, int slices, long long& unit, int& slice)
{
    const long long j = id >> 3;
    unit = (j / slices) * 8 + (id & 7);
    slice = (int)(j % slices);
}

// log(1 + exp(v)), v itself from where they agree in fp32
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

__device__ __forceinline__ double shift_up(double x, int d) { return __shfl_up(x, d); }

// Decays of a chunk of L tokens, K of them a lane: token K l + k.  raw: dt + bias,
// d: delta (0 behind the chunk's end, where nothing changes), c: the running sum of
// log2 exp(g), in 64 bits: its differences are small, it is not.
template <int L> struct Decays {
    static constexpr int K = L / 64;
    float raw[K], d[K];
    double c[K], total;
    // `dt`: of the chunk's first token and the head, tokens H apart; live: tokens of the chunk
    __device__ __forceinline__ void load(const float* __restrict__ dt, int H, int live, float bias)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = K * lane_id() + k;
            raw[k] = dt[(size_t)(t < live ? t : live - 1) * H] + bias;
        }
    }
    __device__ __forceinline__ void scan(float A, int plus, int live)
    {
        const double a2 = (double)A * 1.4426950408889634;
        double run = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = K * lane_id() + k < live;
            d[k] = in ? (plus ? softplus(raw[k]) : raw[k]) : 0.f;
            run += in ? (double)d[k] * a2 : 0.0;
            c[k] = run;
        }
        double s = run;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double up = shift_up(s, o);
            if (lane_id() >= o) s += up;
        }
        total = __shfl(s, 63);
#pragma unroll
        for (int k = 0; k < K; ++k) c[k] += s - run;
    }
};

// v as PARTS fragments that sum up to it
__device__ __forceinline__ void split(const float (&v)[8], u32x4 (&w)[3])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t x = cvt2_bf16(a, b);
            w[p][i] = x;
            a -= __uint_as_float(x << 16);
            b -= __uint_as_float(x & 0xffff0000u);
        }
    }
}

// Rows::down, in plain order: to go with operands read along their rows
template <typename T, int D>
__device__ __forceinline__ Frag<T> down_plain(const void* tab, int k0, int d0)
{
    using R = Rows<T, D>;
    const int l = lane_id(), h = l >> 5;
    if constexpr (sizeof(T) == 2) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        const int i = l & 15, c = d0 + 16 * ((l >> 4) & 1) + 4 * (i & 3);
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r = 8 * h + 4 * t + (i >> 2);
            const char* p = reinterpret_cast<const char*>(tab) + k0 * R::BYTES + R::word(r, c >> 3) * 16 + (c & 7) * 2;
            v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
        }
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const int c = d0 + (l & 31);
        const float* t = reinterpret_cast<const float*>(tab) + k0 * R::U * 4;
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t[R::word(8 * h + j, c >> 2) * 4 + (c & 3)];
        return v;
    }
}

// four values of row r at column c (a multiple of 4) of a table
template <typename T, int D>
__device__ __forceinline__ f32x4 row4(const void* tab, int r, int c)
{
    using R = Rows<T, D>;
    if constexpr (sizeof(T) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const char*>(tab) + R::word(r, c >> 3) * 16 + (c & 7) * 2);
        return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u)};
    } else {
        return *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(tab) + R::word(r, c >> 2) * 16);
    }
}

// rows of a tile's accumulator registers 4 i .. 4 i + 3: 8 i + 4 h + 0 .. 3
__device__ __forceinline__ int acc_rows(int i) { return 8 * i + 4 * (lane_id() >> 5); }

}  // namespace gdn
