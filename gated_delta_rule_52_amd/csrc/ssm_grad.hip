// ssm_grad.hip -- gradients of the selective state space scan, chunk by chunk,
// from the states S before and the gradients dS behind every chunk (ssm_walk.hip).
// With G = C B^T, Z = dy x^T, E_ts = exp(c_t - c_s) for s <= t:
//
//   du_s = sum_t E_ts G_ts dy_t + exp(c_L - c_s) dS^T B_s,     dx = delta du + D dy
//   dB_s = delta_s (sum_t E_ts Z_ts C_t + exp(c_L - c_s) dS x_s)      summed over a group's heads
//   dC_t = sum_s E_ts Z_ts delta_s B_s + exp(c_t) S dy_t              summed over a group's heads
//   dg_t = sum_{t' >= t > s} M_t's + sum_{t' >= t} r_t' + sum_{s < t} q_s + exp(c_L) <S, dS>
//          with M = E G Z delta, r_t = exp(c_t) C_t . S dy_t, q_s = delta_s exp(c_L - c_s) x_s . dS^T B_s
//   ddelta = A dg + x . du,   dA = sum delta dg,   dD = sum dy . x
//
// (g_t scales everything that passes from before t to t or after it.)  dg and
// x . du are formed from E, G and Z themselves and from states split into bf16 that
// hold all their bits, so they are as exact as in fp32; where a result is stored as
// bf16, E G, E Z delta and, for dB, dS are rounded to it on the way (dB and dC are off by
// 0.0021 to 0.0024 in the 2-norm, dx by 0.0017 to 0.0020, where storing them alone is 0.0017;
// two parts of each would be twice the products).  The sums behind
// dg go to ssm_finish_kernel (ssm_prep.hip).  dg's weights add up along the tokens, so
// it must not be a difference of row and column sums of M, whose roundings would
// (dA 20 times as far off where it is small): pairs within a block of 32 tokens are
// summed up to and from every t by a product with 0s and 1s.
//
// A workgroup has a chunk, a group and some of its heads, whose slices of 64
// values it takes one after the other, and one of two parts: that of the t (dC, r)
// or that of the s (dx, dB, q), a wave each 32 of the chunk's tokens.  The sum over
// the heads stays in registers, and so do the wave's own rows of C and dy, or B and
// x; the other side's rows and half of a state at a time are in LDS, so that two
// workgroups share a compute unit and one computes while the other loads.  A t has
// the s before it and an s the t behind it, so the parts' waves complement one
// another on a SIMD.  Each sum is formed within a lane and its other half, in one
// order.  32768 tokens of 6 heads of 128, N = 128: 193 to 197 us.
//
// Masked pairs (s behind t within a block of 32) must not let an infinity or a NaN
// through: their factors are selected away, and where G or Z of a block has such a value
// the chunk's part is done again with care (CAREFUL).  The sums that find it take
// 1 % of a call of small heads (in line, the care took the registers of the hot loop).
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct GradArgs {
    const void *x, *B, *C, *dy;
    const float *dec, *D, *h0, *dhT;
    const int* cu;
    const float *fwd, *back;  // [states][slices] states
    void *dx, *dB, *dC;
    float *token, *part;  // token: [chunks][H][kTokens]; part: [2][splits][T][G][N]
    long long xs, bs, cs;
    int nb, T, H, G, P, slices, splits;
};

// order of issue of N products with one read of R instructions each, where the
// compiler's own has the reads wait
template <typename T, int N, int R> __device__ __forceinline__ void ordered()
{
    if constexpr (sizeof(T) == 2) order_products<N, R, 4>();
    __builtin_amdgcn_sched_barrier(0);
}

// registers 8 b .. 8 b + 7 of an accumulator as parts that hold all their bits
template <typename T> __device__ __forceinline__ void acc_parts(const f32x16& s, int b, Frag<T> (&f)[SsmTile<T>::PARTS])
{
    if constexpr (sizeof(T) == 2) {
        float v[8];
        u32x4 w[3];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s[8 * b + i];
        split(v, w);
#pragma unroll
        for (int p = 0; p < 3; ++p) f[p] = __builtin_bit_cast(bf16x8, w[p]);
    } else {
        f[0] = acc_frag<float>(s, b);
    }
}

// row m = l % 32 of the strictly lower triangle of ones (minus: of -1), columns
// 16 b .. + 15, permuted order
template <typename T> __device__ __forceinline__ Frag<T> ones_below(int b, int l, bool minus)
{
    const int m = l & 31, h = l >> 5;
    if constexpr (sizeof(T) == 2) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 16 * b + 8 * (i >> 1) + 4 * h + 2 * (i & 1);
            w[i] = ((s < m ? 0x3f80u : 0u) | (s + 1 < m ? 0x3f800000u : 0u)) ^ (minus ? 0x80008000u : 0u);
        }
        return __builtin_bit_cast(bf16x8, w);
    } else {
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 16 * b + 8 * (j >> 2) + 4 * h + (j & 3) < m ? (minus ? -1.f : 1.f) : 0.f;
        return v;
    }
}

// Whether a block's products G and Z of all pairs, masked ones among them, are finite: a
// row of either side that is not leaves none of its own finite.
__device__ __forceinline__ bool finite_pairs(const f32x16& g, const f32x16& z)
{
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += g[r] + z[r];
    return !__any(!(fabsf(s) < INFINITY));
}

// The pairs that are not finite, taken out of g (M of the lane's t' and the registers'
// s), as the products with ones_below would sum them: lane q of 16 gets the sum over
// t' >= t > s of register q's t.  Rare.
__device__ __forceinline__ float own_pairs(f32x16& g, int l)
{
    f32x16 out;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const bool finite = fabsf(g[r]) < INFINITY;
        out[r] = finite ? 0.f : g[r];
        g[r] = finite ? g[r] : 0.f;
    }
    float mine = 0.f;
#pragma unroll 1
    for (int t = 0; t < 32; ++t) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) v += acc_rows(r >> 2, l) + (r & 3) < t ? out[r] : 0.f;
        v = wave_sum((l & 31) >= t ? v : 0.f);
        if ((l & 15) == 4 * (t >> 3) + (t & 3) && l >> 5 == (t >> 2 & 1)) mine = v;
    }
    return mine;
}

// an operand in plain order as in permuted order (attn.h): 4 of each half's values change places
template <typename T> __device__ __forceinline__ Frag<T> permuted(const Frag<T>& f)
{
    constexpr int W = sizeof(Frag<T>) / 4;
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    words v = __builtin_bit_cast(words, f);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(v[i], v[i + W / 2], false, false);
        v[i] = r[0], v[i + W / 2] = r[1];
    }
    return __builtin_bit_cast(Frag<T>, v);
}

template <typename T, int N> struct GradLds {
    static constexpr int L = SsmTile<T>::L;
    char rows[L * Rows<T, N>::BYTES], vals[L * Rows<T, kSlice>::BYTES];  // B and x, or C and dy
    char st[SsmTile<T>::PARTS][64 * Rows<T, kSlice>::BYTES];              // half of a state
    float dec[DEC_ROWS * L];
};

// what both parts know of their chunk
struct Chunk {
    Unit u;
    long long id;
    size_t row0;
    int c, live, g, sp, h_first, h_last;
};

template <typename T, int N> struct Grad {
    static constexpr int L = SsmTile<T>::L, NB = L / 32, NTH = 64 * NB, PARTS = SsmTile<T>::PARTS, KN = N / 16, TN = N / 32, NH = N / 64;
    static constexpr int SW = 64 * 8 / NTH;  // runs of 8 values of half a state a thread stages
    using NTab = Rows<T, N>;
    using VTab = Rows<T, kSlice>;
    using NRead = Reads<T, N>;
    using VRead = Reads<T, kSlice>;
    using State = float[SW][8];

    template <typename R> static __device__ __forceinline__ void fetch(char* tab, const T* base, long long stride, int live, int l)
    {
        for (int r = 16 * uniform(wave_id()); r < L; r += 16 * NB) {
            const int rr = r < live ? r : live - 1;
            R::template fetch<16>(tab, r, base + (size_t)rr * stride, (uint32_t)(stride * sizeof(T)), live - 1 - rr, l);
        }
    }
    // Rows 64 hh .. + 63 of a state, as a table of its 64 values along them: run i of a
    // thread is 8 rows of value p.  At a sequence's edge a state is [N][P].
    static __device__ __forceinline__ void load_state(const GradArgs& a, const Chunk& k, const float* between, long long which,
                                                      const float* edge, int slice, int hh, int tid, State& v)
    {
        const int per_head = a.P / kSlice, head = slice / per_head;
        const float* s = edge ? edge + (((size_t)k.u.b * a.H + head) * N + 64 * hh) * a.P + (slice - head * per_head) * kSlice
                              : between + (((size_t)which * a.slices + slice) * N + 64 * hh) * kSlice;
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            const int x = i * NTH + tid, p = x & 63, n = x >> 6 << 3;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = s[(size_t)(n + j) * a.P + p];
            } else {
                load_state8(s, n, p, v[i]);
            }
        }
    }
    static __device__ __forceinline__ void put_state(GradLds<T, N>& m, int tid, const State& v)
    {
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            const int x = i * NTH + tid, p = x & 63, q = x >> 6;
            if constexpr (sizeof(T) == 2) {
                u32x4 parts[3];
                split<true>(v[i], parts);  // dB takes the first part alone
#pragma unroll
                for (int j = 0; j < 3; ++j) *reinterpret_cast<u32x4*>(m.st[j] + VTab::word(p, q) * 16) = parts[j];
            } else {
                *reinterpret_cast<f32x4*>(m.st[0] + VTab::word(p, 2 * q) * 16) = f32x4{v[i][0], v[i][1], v[i][2], v[i][3]};
                *reinterpret_cast<f32x4*>(m.st[0] + VTab::word(p, 2 * q + 1) * 16) = f32x4{v[i][4], v[i][5], v[i][6], v[i][7]};
            }
        }
    }
    // exp(c) from the end of block `from` to the start of block `to`
    static __device__ __forceinline__ float between(const float* dec, int from, int to)
    {
        const int e = 32 * from + 31, s = 32 * to - 1;
        return exp2_hw((dec[DEC_HI * L + s] - dec[DEC_HI * L + e]) + (dec[DEC_LO * L + s] - dec[DEC_LO * L + e]));
    }
    static __device__ __forceinline__ void store(const GradArgs& a, const Chunk& k, const f32x16 (&acc)[TN], bool is_s, int at)
    {
        if (at >= k.live) return;
        const size_t o = ((k.row0 + at) * a.G + k.g) * N;
        T* out = (T*)(is_s ? a.dB : a.dC) + o;
        float* part = a.part + ((size_t)(is_s ? 0 : a.splits) + k.sp) * a.T * a.G * N + o;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = 32 * i + acc_rows(q);
                const float v0 = acc[i][4 * q], v1 = acc[i][4 * q + 1], v2 = acc[i][4 * q + 2], v3 = acc[i][4 * q + 3];
                if (a.splits == 1)
                    store4<T>(out + n, v0, v1, v2, v3);
                else
                    store4<float>(part + n, v0, v1, v2, v3);
            }
    }

    // Both parts return whether a block's own pairs, the masked ones among them, had a value
    // that is not finite.  It would reach results that do not depend on it through products
    // with 0: the chunk's part is then done again with CAREFUL, which keeps such values
    // from the masked products and adds them where they belong.
    //
    // the part of the t: dC and r
    template <bool CAREFUL> static __device__ __forceinline__ bool of_t(const GradArgs& a, const Chunk& k, GradLds<T, N>& m)
    {
        const int w = uniform(wave_id()), rb = w, live = k.live, per_head = a.P / kSlice;
        const bool has_s = k.c > 0 || a.h0, has_d = k.c < k.u.chunks - 1 || a.dhT;
        fetch<NTab>(m.rows, (const T*)a.B + k.row0 * a.bs + (size_t)k.g * N, a.bs, live, lane_id());
        const uint32_t na = NTab::along_at(), va = VTab::along_at(), nd = NRead::down_at(), vp = VRead::plain_at();
        const int mine = 32 * rb + (lane_id() & 31), row = mine < live ? mine : live - 1;
        Frag<T> own[KN], val[4];  // the lane's rows of C and dy
#pragma unroll
        for (int kk = 0; kk < KN; ++kk)
            own[kk] = load_frag<T>((const T*)a.C + (k.row0 + row) * a.cs + (size_t)k.g * N + 16 * kk + 8 * (lane_id() >> 5));
        f32x16 acc[TN];
#pragma unroll
        for (int i = 0; i < TN; ++i) acc[i] = zero16();
        bool seen = false;
        float r_state = 0.f, r_blocks = 0.f, over_own = 0.f, dot = 0.f, cross0 = 0.f, cross1 = 0.f;

        for (int slice = k.h_first * per_head; slice < k.h_last * per_head; ++slice) {
            const int head = slice / per_head, sub = slice - head * per_head, p0 = sub * kSlice;
            // the lane, opaque: what follows from it is formed here and not held from slice to slice
            const int l = (int)opaque(lane_id()), h = l >> 5, tid = 64 * w + l, at = 32 * rb + (l & 31);
            fetch<VTab>(m.vals, (const T*)a.x + k.row0 * a.xs + (size_t)head * a.P + p0, a.xs, live, l);
            const float* dec = a.dec + ((size_t)k.id * a.H + head) * kDecays<L>;
            if (sub == 0) {
                r_state = r_blocks = over_own = dot = cross0 = cross1 = 0.f;
                for (int i = tid; i < DEC_ROWS * L; i += NTH) m.dec[i] = dec[i];
            }
            {
                const int t = at < live ? at : live - 1;
                const T* dy = (const T*)a.dy + ((k.row0 + t) * a.H + head) * a.P + p0 + 8 * h;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) val[kk] = load_frag<T>(dy + 16 * kk);
            }
            const float e_t = dec[DEC_E * L + at];
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                if (hh) __syncthreads();  // the half before is read
                if (has_s) {
                    State sv, dv;
                    load_state(a, k, a.fwd, k.u.between + k.c - 1, k.c > 0 ? nullptr : a.h0, slice, hh, tid, sv);
                    if (has_d) load_state(a, k, a.back, k.u.between + k.c, k.c < k.u.chunks - 1 ? nullptr : a.dhT, slice, hh, tid, dv);
                    put_state(m, tid, sv);
                    if (has_d) {
#pragma unroll
                        for (int i = 0; i < SW; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(sv[i][j], dv[i][j], dot);
                    }
                }
                if (hh == 0) wait_vm<0>();
                __syncthreads();
                if (!has_s) continue;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 2 * hh; i < 2 * hh + 2; ++i) {
                    f32x16 z = zero16();
                    const uint32_t pl = opaque(vp);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) z = mma32(VRead::plain(m.st[p], pl, 16 * kk, 32 * (i - 2 * hh)), val[kk], z);
                    ordered<T, 4 * PARTS, 2>();
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> cv = permuted<T>(own[2 * i + b]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = z[8 * b + j] * e_t;
                            acc[i][8 * b + j] += v;
                            r_state = __builtin_fmaf((float)cv[j], v, r_state);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (32 * rb < live) {
                const float *hi_s = m.dec + DEC_HI * L, *lo_s = m.dec + DEC_LO * L, *d_s = m.dec + DEC_DELTA * L,
                            *behind_s = m.dec + DEC_BEHIND * L;
                const float ahead = m.dec[DEC_AHEAD * L + at];
                float r = 0.f;
                for (int sb = 0; sb <= rb; ++sb) {
                    f32x16 gm = zero16(), z = zero16();
                    const uint32_t nal = opaque(na), val4 = opaque(va), ndn = opaque(nd);
#pragma unroll
                    for (int kk = 0; kk < KN; ++kk) gm = mma32(NTab::along(m.rows, nal, 32 * sb, kk), own[kk], gm);
                    ordered<T, KN, 1>();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(m.vals, val4, 32 * sb, kk), val[kk], z);
                    ordered<T, 4, 1>();
                    if (sb < rb) {
                        const float f = ahead * between(m.dec, sb, rb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 32 * sb + acc_rows(i, l);
                            const f32x4 bs = *reinterpret_cast<const f32x4*>(behind_s + s), ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                z[4 * i + j] *= f * bs[j] * ds[j];
                                r = __builtin_fmaf(z[4 * i + j], gm[4 * i + j], r);
                            }
                        }
                        if (NB == 4 && sb + 1 < rb) {  // pairs that pass over blocks 1 and 2
                            const float all = wave_sum(at < live ? r : 0.f);
                            cross0 += sb ? 0.f : all;
                            cross1 += sb ? all : 0.f;
                        }
                    } else {
                        if constexpr (!CAREFUL) seen |= !finite_pairs(gm, z);
                        const float hc = hi_s[at], lc = lo_s[at];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 32 * sb + acc_rows(i, l);
                            const f32x4 hs = *reinterpret_cast<const f32x4*>(hi_s + s), ls = *reinterpret_cast<const f32x4*>(lo_s + s),
                                        ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // selected: pairs that are none may be anything
                                const float e = exp2_hw((hc - hs[j]) + (lc - ls[j])) * ds[j];
                                z[4 * i + j] = s + j <= at ? z[4 * i + j] * e : 0.f;
                                gm[4 * i + j] = s + j < at && at < live ? gm[4 * i + j] * z[4 * i + j] : 0.f;
                            }
                        }
                        // over[t][t'] = sum_{s < t} M_t's, then for every t the sum over t' >= t.
                        // The bf16 products round their sums down a little on average, which
                        // sums over all tokens (dA, ddt_bias) would show: every other block of
                        // tokens sums -M, and the smallest parts come first.
                        if constexpr (CAREFUL) over_own += own_pairs(gm, l);
                        const bool minus = w & 1;
                        f32x16 over = zero16();
                        Frag<T> parts[2][PARTS];
#pragma unroll
                        for (int b = 0; b < 2; ++b) acc_parts<T>(gm, b, parts[b]);
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                            for (int b = 0; b < 2; ++b) over = mma32(ones_below<T>(b, l, minus), parts[b][p], over);
                        float mine = 0.f;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float v = lane16_sum((l & 31) >= acc_rows(q >> 2, l) + (q & 3) ? over[q] : 0.f);
                            mine = (l & 15) == q ? v : mine;
                        }
                        mine += __shfl_xor(mine, 16);
                        over_own += minus ? -mine : mine;
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> zv = acc_frag<T>(z, b);
                        if (CAREFUL && sb == rb) {
#pragma unroll
                            for (int i = 0; i < TN; ++i)
                                acc[i] = mma32(finite_only(NRead::down(m.rows, ndn, 32 * sb + 16 * b, 32 * i)), zv, acc[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < TN; ++i) acc[i] = mma32(NRead::down(m.rows, ndn, 32 * sb + 16 * b, 32 * i), zv, acc[i]);
                            ordered<T, TN, 2>();
                        }
                    }
                    if (CAREFUL && sb == rb) add_masked_rest<T, N>(acc, z, m.rows, 32 * sb, false);
                }
                r_blocks += r;
            }
            if (sub == per_head - 1) {  // the head's sums are complete
                float* o = a.token + ((size_t)k.id * a.H + head) * kTokens<L>;
                const float rs = half_add(r_state), rk = half_add(r_blocks), all = wave_sum(dot);
                if (h == 0) {
                    o[TOK_R_STATE * L + at] = rs;
                    o[TOK_R_BLOCKS * L + at] = rk;
                }
                // lane q of 16 has the sum of register q's t
                if (!(l & 16)) o[TOK_OWN * L + 32 * rb + acc_rows((l & 15) >> 2, l) + (l & 3)] = over_own;
                if (l == 0) {
                    o[TOK_ROWS * L + w] = all;
                    if (NB == 4 && rb == 2) o[TOK_ROWS * L + 4] = cross0;
                    if (NB == 4 && rb == 3) {
                        o[TOK_ROWS * L + 5] = cross0;
                        o[TOK_ROWS * L + 6] = cross1;
                    }
                }
            }
            __syncthreads();
        }
        store(a, k, acc, false, 32 * rb + (lane_id() & 31));
        return seen;
    }

    // the part of the s: dx, dB and q
    template <bool CAREFUL> static __device__ __forceinline__ bool of_s(const GradArgs& a, const Chunk& k, GradLds<T, N>& m)
    {
        const int w = uniform(wave_id()), rb = w, live = k.live, per_head = a.P / kSlice;
        const bool has_d = k.c < k.u.chunks - 1 || a.dhT;
        fetch<NTab>(m.rows, (const T*)a.C + k.row0 * a.cs + (size_t)k.g * N, a.cs, live, lane_id());
        const uint32_t na = NTab::along_at(), va = VTab::along_at(), nd = NRead::down_at(), vd = VRead::down_at(),
                       vp = VRead::plain_at();
        const int mine = 32 * rb + (lane_id() & 31), row = mine < live ? mine : live - 1;
        Frag<T> own[KN], val[4];  // the lane's rows of B and x
#pragma unroll
        for (int kk = 0; kk < KN; ++kk)
            own[kk] = load_frag<T>((const T*)a.B + (k.row0 + row) * a.bs + (size_t)k.g * N + 16 * kk + 8 * (lane_id() >> 5));
        f32x16 acc[TN];
#pragma unroll
        for (int i = 0; i < TN; ++i) acc[i] = zero16();
        bool seen = false;
        float q_blocks = 0.f, q_state = 0.f, xdu = 0.f, xdy = 0.f;

        for (int slice = k.h_first * per_head; slice < k.h_last * per_head; ++slice) {
            const int head = slice / per_head, sub = slice - head * per_head, p0 = sub * kSlice;
            const int l = (int)opaque(lane_id()), h = l >> 5, tid = 64 * w + l, at = 32 * rb + (l & 31);
            fetch<VTab>(m.vals, (const T*)a.dy + (k.row0 * a.H + head) * a.P + p0, (long long)a.H * a.P, live, l);
            const float* dec = a.dec + ((size_t)k.id * a.H + head) * kDecays<L>;
            if (sub == 0) {
                q_blocks = q_state = xdu = xdy = 0.f;
                for (int i = tid; i < DEC_ROWS * L; i += NTH) m.dec[i] = dec[i];
            }
            {
                const int s = at < live ? at : live - 1;
                const T* x = (const T*)a.x + (k.row0 + s) * a.xs + (size_t)head * a.P + p0 + 8 * h;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) val[kk] = load_frag<T>(x + 16 * kk);
            }
            const float f_s = dec[DEC_F * L + at], d_s = dec[DEC_DELTA * L + at];
            f32x16 du[2] = {zero16(), zero16()};
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                if (hh) __syncthreads();  // the half before is read
                if (has_d) {
                    State dv;
                    load_state(a, k, a.back, k.u.between + k.c, k.c < k.u.chunks - 1 ? nullptr : a.dhT, slice, hh, tid, dv);
                    put_state(m, tid, dv);
                }
                if (hh == 0) wait_vm<0>();
                __syncthreads();
                if (!has_d) continue;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int pt = 0; pt < 2; ++pt) {
                    f32x16 z = zero16();
                    const uint32_t al = opaque(va);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(m.st[p], al, 32 * pt, kk), own[4 * hh + kk], z);
                    ordered<T, 4 * PARTS, 1>();
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> xv = permuted<T>(val[2 * pt + b]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = z[8 * b + j] * f_s;
                            du[pt][8 * b + j] += v;
                            q_state = __builtin_fmaf((float)xv[j], v, q_state);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 2 * hh; i < 2 * hh + 2; ++i) {
                    f32x16 z = zero16();
                    const uint32_t pl = opaque(vp);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) z = mma32(VRead::plain(m.st[0], pl, 16 * kk, 32 * (i - 2 * hh)), val[kk], z);
                    ordered<T, 4, 2>();
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = __builtin_fmaf(z[j], f_s * d_s, acc[i][j]);
                }
            }
            if (32 * rb < live) {
                const float *hi_s = m.dec + DEC_HI * L, *lo_s = m.dec + DEC_LO * L, *ahead_s = m.dec + DEC_AHEAD * L;
                const float behind = m.dec[DEC_BEHIND * L + at];
                for (int tb = rb; tb < NB && 32 * tb < live; ++tb) {
                    f32x16 gm = zero16(), z = zero16();
                    const uint32_t nal = opaque(na), val4 = opaque(va), ndn = opaque(nd), vdn = opaque(vd);
#pragma unroll
                    for (int kk = 0; kk < KN; ++kk) gm = mma32(NTab::along(m.rows, nal, 32 * tb, kk), own[kk], gm);
                    ordered<T, KN, 1>();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(m.vals, val4, 32 * tb, kk), val[kk], z);
                    ordered<T, 4, 1>();
                    if (tb > rb) {
                        const float f = behind * between(m.dec, rb, tb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int t = 32 * tb + acc_rows(i, l);
                            const f32x4 as = *reinterpret_cast<const f32x4*>(ahead_s + t);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float e = t + j < live ? as[j] * f : 0.f;  // no copies of the last token
                                gm[4 * i + j] *= e;
                                q_blocks = __builtin_fmaf(gm[4 * i + j], z[4 * i + j], q_blocks);
                                z[4 * i + j] *= e * d_s;
                            }
                        }
                    } else {
                        if constexpr (!CAREFUL) seen |= !finite_pairs(gm, z);
                        const float hc = hi_s[at], lc = lo_s[at];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int t = 32 * tb + acc_rows(i, l);
                            const f32x4 ht = *reinterpret_cast<const f32x4*>(hi_s + t), lt = *reinterpret_cast<const f32x4*>(lo_s + t);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // selected: pairs that are none may be anything
                                const bool pair = at <= t + j && t + j < live;
                                const float e = exp2_hw((ht[j] - hc) + (lt[j] - lc));
                                const float eg = pair ? e * gm[4 * i + j] : 0.f, zv = z[4 * i + j];
                                xdu = pair ? __builtin_fmaf(eg, zv, xdu) : xdu;
                                xdy += t + j == at ? zv : 0.f;
                                gm[4 * i + j] = eg;
                                z[4 * i + j] = pair ? e * zv * d_s : 0.f;
                            }
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> mv = acc_frag<T>(gm, b), zv = acc_frag<T>(z, b);
                        if (CAREFUL && tb == rb) {
#pragma unroll
                            for (int pt = 0; pt < 2; ++pt)
                                du[pt] = mma32(finite_only(VRead::down(m.vals, vdn, 32 * tb + 16 * b, 32 * pt)), mv, du[pt]);
#pragma unroll
                            for (int i = 0; i < TN; ++i)
                                acc[i] = mma32(finite_only(NRead::down(m.rows, ndn, 32 * tb + 16 * b, 32 * i)), zv, acc[i]);
                        } else {
#pragma unroll
                            for (int pt = 0; pt < 2; ++pt) du[pt] = mma32(VRead::down(m.vals, vdn, 32 * tb + 16 * b, 32 * pt), mv, du[pt]);
#pragma unroll
                            for (int i = 0; i < TN; ++i) acc[i] = mma32(NRead::down(m.rows, ndn, 32 * tb + 16 * b, 32 * i), zv, acc[i]);
                            ordered<T, 2 + TN, 2>();
                        }
                    }
                    if (CAREFUL && tb == rb) {
                        add_masked_rest<T, kSlice>(du, gm, m.vals, 32 * tb, true);
                        add_masked_rest<T, N>(acc, z, m.rows, 32 * tb, true);
                    }
                }
            }
            if (at < live) {
                const float skip = a.D ? a.D[head] : 0.f;
                T* dx = (T*)a.dx + ((k.row0 + at) * a.H + head) * a.P + p0;
                const uint32_t vr = VRead::row_at(at);
#pragma unroll
                for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 yv = VRead::row4(m.vals, vr, pt, q);
                        float v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[j] = d_s * du[pt][4 * q + j];
                            if (a.D) v[j] = __builtin_fmaf(skip, yv[j], v[j]);
                        }
                        store4<T>(dx + 32 * pt + acc_rows(q, l), v[0], v[1], v[2], v[3]);
                    }
            }
            if (sub == per_head - 1) {  // the head's sums are complete
                float* o = a.token + ((size_t)k.id * a.H + head) * kTokens<L>;
                const float qb = half_add(q_blocks), qs = half_add(q_state), xd = half_add(xdu), xy = half_add(xdy);
                if (h == 0) {
                    o[TOK_Q_BLOCKS * L + at] = qb;
                    o[TOK_Q_STATE * L + at] = qs;
                    o[TOK_XDU * L + at] = (qb + xd) + qs;
                    o[TOK_XDY * L + at] = xy;  // the pair t = s is one half's
                }
            }
            __syncthreads();
        }
        store(a, k, acc, true, 32 * rb + (lane_id() & 31));
        return seen;
    }
};

template <typename T, int N>
__global__ __launch_bounds__(64 * (SsmTile<T>::L / 32), sizeof(T) == 2 ? 2 : 1) void ssm_grad_kernel(GradArgs a)
{
    constexpr int L = SsmTile<T>::L;
    __shared__ __align__(16) GradLds<T, N> m;
    // Parts in turn by 32 workgroups of a die: as many as it has compute units, each
    // of which then gets one of either.
    const long long j = blockIdx.x >> 3;
    const bool is_s = (j >> 5) & 1;
    const int jobs = a.G * a.splits;
    long long unit;
    int job;
    Chunk k;
    deal((((j >> 6) << 5 | (j & 31)) << 3) | (blockIdx.x & 7), jobs, unit, job);
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, 0, unit, k.u)) return;
    const int per_group = a.H / a.G;
    k.id = unit;
    k.c = k.u.at;
    k.live = k.u.n - k.c * L < L ? k.u.n - k.c * L : L;
    k.row0 = (size_t)k.u.start + (size_t)k.c * L;
    k.g = job / a.splits;
    k.sp = job - k.g * a.splits;
    k.h_first = k.g * per_group + (int)((long long)per_group * k.sp / a.splits);
    k.h_last = k.g * per_group + (int)((long long)per_group * (k.sp + 1) / a.splits);
    const bool seen = is_s ? Grad<T, N>::template of_s<false>(a, k, m) : Grad<T, N>::template of_t<false>(a, k, m);
    if (__builtin_expect(__syncthreads_or(seen), 0)) {
        if (is_s)
            Grad<T, N>::template of_s<true>(a, k, m);
        else
            Grad<T, N>::template of_t<true>(a, k, m);
    }
}

// dB and dC from the parts of a group's heads, in order: a word of 4 values a thread.
// The sequences' rows end at the greatest bound, which is the last one only where no
// bound decreases (ordered_bounds).
template <typename T>
__global__ __launch_bounds__(256) void ssm_join_kernel(const float* __restrict__ part, const int* __restrict__ cu, T* dB,
                                                       T* dC, int nb, int tokens, int splits, int width)
{
    __shared__ int red[4];
    int end = 0;
    for (int b = threadIdx.x; b <= nb; b += 256) end = cu[b] > end ? cu[b] : end;
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const int other = __shfl_xor(end, o);
        end = other > end ? other : end;
    }
    if (lane_id() == 0) red[wave_id()] = end;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) end = red[w] > end ? red[w] : end;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, total = (long long)tokens * width / 4;
    if (i >= total) return;
    const int row = (int)(i * 4 / width);
    if (row < cu[0] || row >= end) return;  // a row of no sequence
    const f32x4* p = reinterpret_cast<const f32x4*>(part) + (size_t)blockIdx.y * splits * total + i;
    f32x4 s = p[0];
    for (int k = 1; k < splits; ++k) s += p[(size_t)k * total];
    store4<T>((blockIdx.y ? dC : dB) + i * 4, s[0], s[1], s[2], s[3]);
}

template <typename T, int N> gdn_status grad(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, const GradArgs& a, hipStream_t st)
{
    constexpr int L = SsmTile<T>::L;
    if (p.chunks) {
        // whole 32s of workgroups a die, for both parts
        const long long a_die = dealt(p.chunks, s.G * p.splits) / 8;
        const dim3 grid((unsigned)((a_die + 31) / 32 * 32 * 8 * 2));
        GDN_LAUNCH("ssm_grad", (ssm_grad_kernel<T, N>), grid, dim3(2 * L), st, a);
    }
    if (p.splits > 1) {
        const int width = s.G * N;
        const dim3 grid((unsigned)(((long long)s.T * width / 4 + 255) / 256), 2);
        GDN_LAUNCH("ssm_join", (ssm_join_kernel<T>), grid, dim3(256), st, a.part, a.cu, (T*)x.dB, (T*)x.dC, s.B, s.T,
                   p.splits, width);
    }
    return GDN_OK;
}

}  // namespace

gdn_status ssm_grad(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, char* ws, hipStream_t st)
{
    GradArgs a{};
    a.x = x.x; a.B = x.B; a.C = x.C; a.dy = x.dy;
    a.dec = (const float*)(ws + p.dec_at);
    a.D = x.D; a.h0 = x.h0; a.dhT = x.dhT; a.cu = x.cu;
    a.fwd = (const float*)(ws + p.fwd_at);
    a.back = (const float*)(ws + p.back_at);
    a.dx = x.dx; a.dB = x.dB; a.dC = x.dC;
    a.part = (float*)(ws + p.part_at);
    a.token = (float*)(ws + p.token_at);
    a.xs = x.xs; a.bs = x.bs; a.cs = x.cs;
    a.nb = s.B; a.T = s.T; a.H = s.H; a.G = s.G; a.P = s.P; a.slices = p.slices; a.splits = p.splits;
    if (s.dtype == GDN_BF16) return s.N == 64 ? grad<bf16, 64>(s, p, x, a, st) : grad<bf16, 128>(s, p, x, a, st);
    return s.N == 64 ? grad<float, 64>(s, p, x, a, st) : grad<float, 128>(s, p, x, a, st);
}

}  // namespace gdn
