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
// bf16, E G, E Z delta and one operand are rounded to it on the way.  The sums behind
// dg go to ssm_finish_kernel (ssm_prep.hip).  dg's weights add up along the tokens, so
// it must not be a difference of row and column sums of M, whose roundings would
// (dA 20 times as far off where it is small): pairs within a block of 32 tokens are
// summed up to and from every t by a product with 0s and 1s.
//
// A workgroup has a chunk, a group and some of its heads, whose slices of 64
// values it takes one after the other: dB and dC stay in registers.  Half of the
// waves are a 32-token block of t each (dC, r), the others one of s (dx, dB, q);
// the states' parts share one table: first S, read by the former while the latter
// go through the chunk's pairs, then dS the other way round.  Each sum is formed
// within a lane and its other half, in one order.
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct GradArgs {
    const void *x, *B, *C, *dy;
    const float *dec, *D, *h0, *dhT;
    const int* cu;
    const float *fwd, *back;  // [states][slices][N][64]
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

// row m = l % 32 of the strictly lower triangle of ones, columns 16 b .. + 15, permuted order
template <typename T> __device__ __forceinline__ Frag<T> ones_below(int b, int l)
{
    const int m = l & 31, h = l >> 5;
    if constexpr (sizeof(T) == 2) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 16 * b + 8 * (i >> 1) + 4 * h + 2 * (i & 1);
            w[i] = (s < m ? 0x3f80u : 0u) | (s + 1 < m ? 0x3f800000u : 0u);
        }
        return __builtin_bit_cast(bf16x8, w);
    } else {
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 16 * b + 8 * (j >> 2) + 4 * h + (j & 3) < m ? 1.f : 0.f;
        return v;
    }
}

template <typename T, int N>
__global__ __launch_bounds__(128 * (SsmTile<T>::L / 32)) void ssm_grad_kernel(GradArgs a)
{
    constexpr int L = SsmTile<T>::L, NB = L / 32, NTH = 128 * NB, PARTS = SsmTile<T>::PARTS, KN = N / 16, TN = N / 32;
    constexpr bool HOLD = sizeof(T) == 2;  // operands that are used again stay in registers
    using NTab = Rows<T, N>;
    using VTab = Rows<T, kSlice>;
    using NRead = Reads<T, N>;
    using VRead = Reads<T, kSlice>;
    constexpr int SW = N * 8 / NTH;  // runs of 8 values of a state a thread stages
    __shared__ __align__(16) char b_s[L * NTab::BYTES], c_s[L * NTab::BYTES];
    __shared__ __align__(16) char x_s[L * VTab::BYTES], y_s[L * VTab::BYTES];
    __shared__ __align__(16) char st_s[PARTS][N * VTab::BYTES];
    __shared__ __align__(16) float dec_s[DEC_ROWS * L], tok_s[kTokens<L>];

    long long id;
    int job;
    deal(blockIdx.x, a.G * a.splits, id, job);
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, id, u)) return;
    const int c = u.at, live = u.n - c * L < L ? u.n - c * L : L;
    const size_t row0 = (size_t)u.start + (size_t)c * L;
    const int w = uniform(wave_id());
    const bool is_s = w >= NB;
    const int rb = is_s ? w - NB : w;  // the lanes' tokens: 32 rb + l % 32
    const int per_head = a.P / kSlice, per_group = a.H / a.G, g = job / a.splits, sp = job - g * a.splits;
    const int h_first = g * per_group + (int)((long long)per_group * sp / a.splits),
              h_last = g * per_group + (int)((long long)per_group * (sp + 1) / a.splits);
    const bool has_s = c > 0 || a.h0, has_d = c < u.chunks - 1 || a.dhT;

    auto rows_of = [&](char* tab, auto rows, const T* base, long long stride, int l) {
        using R = decltype(rows);
        for (int r = 16 * w; r < L; r += 32 * NB) {
            const int rr = r < live ? r : live - 1;
            R::template fetch<16>(tab, r, base + (size_t)rr * stride, (uint32_t)(stride * sizeof(T)), live - 1 - rr, l);
        }
    };
    rows_of(b_s, NTab{}, (const T*)a.B + row0 * a.bs + (size_t)g * N, a.bs, lane_id());
    rows_of(c_s, NTab{}, (const T*)a.C + row0 * a.cs + (size_t)g * N, a.cs, lane_id());

    f32x16 acc[TN];  // dC of 32 t or dB of 32 s
#pragma unroll
    for (int i = 0; i < TN; ++i) acc[i] = zero16();
    // a lane's offsets for the reads below; opaque, each loop's are formed in it
    const uint32_t na = NTab::along_at(), va = VTab::along_at(), nd = NRead::down_at(), vd = VRead::down_at(),
                   vp = VRead::plain_at(), nr = NRead::row_at(32 * rb + (lane_id() & 31)), vr = VRead::row_at(32 * rb + (lane_id() & 31));
    Frag<T> own[HOLD ? KN : 1], val[HOLD ? 4 : 1];  // the lane's rows of C or B, and of dy or x
    auto own_at = [&](int kk) {
        if constexpr (HOLD) return own[kk];
        else return NTab::along(is_s ? b_s : c_s, opaque(na), 32 * rb, kk);
    };
    auto val_at = [&](int kk) {
        if constexpr (HOLD) return val[kk];
        else return VTab::along(is_s ? x_s : y_s, opaque(va), 32 * rb, kk);
    };

    for (int slice = h_first * per_head; slice < h_last * per_head; ++slice) {
        const int head = slice / per_head, sub = slice - head * per_head, p0 = sub * kSlice;
        // the lane, opaque: what follows from it is formed here and not held from slice to slice
        const int l = (int)opaque(lane_id()), h = l >> 5, tid = 64 * w + l, at = 32 * rb + (l & 31);
        rows_of(x_s, VTab{}, (const T*)a.x + row0 * a.xs + (size_t)head * a.P + p0, a.xs, l);
        rows_of(y_s, VTab{}, (const T*)a.dy + (row0 * a.H + head) * a.P + p0, (long long)a.H * a.P, l);
        // run i of this thread: row n of the state, values 8 q .. 8 q + 7
        auto run = [&](int i, int& n, int& q) {
            const int x = i * NTH + tid;
            n = x >> 3, q = x & 7;
        };
        auto state_of = [&](const float* between, long long which, const float* edge, f32x4 (&v)[SW][2]) {
            // between chunks [N][64]; at a sequence's edge [N][P]
            const float* s = edge ? edge + ((size_t)u.b * a.H + head) * N * a.P + p0
                                  : between + ((size_t)which * a.slices + slice) * N * kSlice;
            const int stride = edge ? a.P : kSlice;
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int n, q;
                run(i, n, q);
                v[i][0] = *reinterpret_cast<const f32x4*>(s + (size_t)n * stride + 8 * q);
                v[i][1] = *reinterpret_cast<const f32x4*>(s + (size_t)n * stride + 8 * q + 4);
            }
        };
        auto put_state = [&](const f32x4 (&v)[SW][2]) {
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int n, q;
                run(i, n, q);
                if constexpr (sizeof(T) == 2) {
                    u32x4 parts[3];
                    const float f[8] = {v[i][0][0], v[i][0][1], v[i][0][2], v[i][0][3], v[i][1][0], v[i][1][1], v[i][1][2], v[i][1][3]};
                    split(f, parts);
#pragma unroll
                    for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4*>(st_s[p] + VTab::word(n, q) * 16) = parts[p];
                } else {
                    *reinterpret_cast<f32x4*>(st_s[0] + VTab::word(n, 2 * q) * 16) = v[i][0];
                    *reinterpret_cast<f32x4*>(st_s[0] + VTab::word(n, 2 * q + 1) * 16) = v[i][1];
                }
            }
        };
        // what put_state has put there, times v
        auto dot_state = [&](const f32x4 (&v)[SW][2]) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int n, q;
                run(i, n, q);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int p = PARTS - 1; p >= 0; --p) {
                        if constexpr (sizeof(T) == 2) {
                            const uint2 w = *reinterpret_cast<const uint2*>(st_s[p] + VTab::word(n, q) * 16 + 8 * j);
                            s += f32x4{__uint_as_float(w.x << 16), upper(__uint_as_float(w.x)), __uint_as_float(w.y << 16),
                                       upper(__uint_as_float(w.y))};
                        } else {
                            s = *reinterpret_cast<const f32x4*>(st_s[p] + VTab::word(n, 2 * q + j) * 16);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) dot = __builtin_fmaf(s[k], v[i][j][k], dot);
                }
            }
            return dot;
        };
        f32x4 sv[SW][2];
        if (has_s) {
            state_of(a.fwd, u.between + c - 1, c > 0 ? nullptr : a.h0, sv);
            put_state(sv);
        }
        if (sub == 0) {
            const float* dec = a.dec + ((size_t)id * a.H + head) * kDecays<L>;
            for (int i = tid; i < DEC_ROWS * L; i += NTH) dec_s[i] = dec[i];
        }
        if (has_d) state_of(a.back, u.between + c, c < u.chunks - 1 ? nullptr : a.dhT, sv);
        wait_vm<0>();
        __syncthreads();

        if constexpr (HOLD) {
            if (slice == h_first * per_head) {
#pragma unroll
                for (int kk = 0; kk < KN; ++kk) own[kk] = NTab::along(is_s ? b_s : c_s, na, 32 * rb, kk);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) val[kk] = VTab::along(is_s ? x_s : y_s, va, 32 * rb, kk);
        }
        const float *hi_s = dec_s + DEC_HI * L, *lo_s = dec_s + DEC_LO * L, *d_s = dec_s + DEC_DELTA * L,
                    *ahead_s = dec_s + DEC_AHEAD * L, *behind_s = dec_s + DEC_BEHIND * L;
        const float dc = d_s[at];
        // a sum of this slice onto those of the head's before it
        auto leave = [&](int i, float v) { tok_s[i] = sub ? tok_s[i] + v : v; };
        // exp(c) from the end of block `from` to the start of block `to`
        auto between = [&](int from, int to) {
            const int e = 32 * from + 31, s = 32 * to - 1;
            return exp2_hw((hi_s[s] - hi_s[e]) + (lo_s[s] - lo_s[e]));
        };
        f32x16 du[2] = {zero16(), zero16()};
        float qo = 0.f, xdu = 0.f, zd = 0.f;
        __builtin_amdgcn_sched_barrier(0);
        if (!is_s) {
            float r = 0.f;
            if (has_s) {
                const float e = dec_s[DEC_E * L + at];
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    f32x16 m = zero16();
                    const uint32_t al = opaque(va), row = opaque(nr);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) m = mma32(VTab::along(st_s[p], al, 32 * i, kk), val_at(kk), m);
                    ordered<T, 4 * PARTS, 1>();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 cv = NRead::row4(c_s, row, i, q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = m[4 * q + j] * e;
                            acc[i][4 * q + j] += v;
                            r = __builtin_fmaf(cv[j], v, r);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            r = half_add(r);
            if (h == 0) leave(TOK_R_STATE * L + at, r);
        } else if (32 * rb < live) {
            const float behind = behind_s[at];
            for (int tb = rb; tb < NB && 32 * tb < live; ++tb) {
                f32x16 m = zero16(), z = zero16();
                const uint32_t nal = opaque(na), val4 = opaque(va), ndn = opaque(nd), vdn = opaque(vd);
#pragma unroll
                for (int kk = 0; kk < KN; ++kk) m = mma32(NTab::along(c_s, nal, 32 * tb, kk), own_at(kk), m);
                ordered<T, KN, 1>();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(y_s, val4, 32 * tb, kk), val_at(kk), z);
                ordered<T, 4, 1>();
                if (tb > rb) {
                    const float f = behind * between(rb, tb);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = 32 * tb + acc_rows(i, l);
                        const f32x4 as = *reinterpret_cast<const f32x4*>(ahead_s + t);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e = t + j < live ? as[j] * f : 0.f;  // no copies of the last token
                            m[4 * i + j] *= e;
                            qo = __builtin_fmaf(m[4 * i + j], z[4 * i + j], qo);
                            z[4 * i + j] *= e * dc;
                        }
                    }
                } else {
                    const float hc = hi_s[at], lc = lo_s[at];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = 32 * tb + acc_rows(i, l);
                        const f32x4 ht = *reinterpret_cast<const f32x4*>(hi_s + t), lt = *reinterpret_cast<const f32x4*>(lo_s + t);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // pairs that are none: exp2(-inf)
                            const float e = exp2_hw(at <= t + j && t + j < live ? (ht[j] - hc) + (lt[j] - lc) : -INFINITY);
                            const float eg = e * m[4 * i + j], zv = z[4 * i + j];
                            xdu = __builtin_fmaf(eg, zv, xdu);
                            zd = t + j == at ? zv : zd;
                            m[4 * i + j] = eg;
                            z[4 * i + j] = e * zv * dc;
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const Frag<T> mv = acc_frag<T>(m, b), zv = acc_frag<T>(z, b);
#pragma unroll
                    for (int pt = 0; pt < 2; ++pt) du[pt] = mma32(VRead::down(y_s, vdn, 32 * tb + 16 * b, 32 * pt), mv, du[pt]);
#pragma unroll
                    for (int i = 0; i < TN; ++i) acc[i] = mma32(NRead::down(c_s, ndn, 32 * tb + 16 * b, 32 * i), zv, acc[i]);
                    ordered<T, 2 + TN, 2>();
                }
            }
            qo = half_add(qo);
            xdu = half_add(xdu) + qo;
            zd = half_add(zd);  // the pair t = s is one half's
        }
        __syncthreads();
        const float dot = wave_sum(has_s && has_d ? dot_state(sv) : 0.f);
        if (l == 0) leave(TOK_ROWS * L + w, dot);
        if (has_d) put_state(sv);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        if (!is_s) {
            float r = 0.f, own_sum = 0.f;
            if (32 * rb < live) {
                const float ahead = ahead_s[at];
                for (int sb = 0; sb <= rb; ++sb) {
                    f32x16 m = zero16(), z = zero16();
                    const uint32_t nal = opaque(na), val4 = opaque(va), ndn = opaque(nd);
#pragma unroll
                    for (int kk = 0; kk < KN; ++kk) m = mma32(NTab::along(b_s, nal, 32 * sb, kk), own_at(kk), m);
                    ordered<T, KN, 1>();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(x_s, val4, 32 * sb, kk), val_at(kk), z);
                    ordered<T, 4, 1>();
                    if (sb < rb) {
                        const float f = ahead * between(sb, rb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 32 * sb + acc_rows(i, l);
                            const f32x4 bs = *reinterpret_cast<const f32x4*>(behind_s + s), ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                z[4 * i + j] *= f * bs[j] * ds[j];
                                r = __builtin_fmaf(z[4 * i + j], m[4 * i + j], r);
                            }
                        }
                        if constexpr (NB == 4) {  // pairs that pass over blocks 1 and 2
                            if (sb + 1 < rb) {
                                const float all = wave_sum(at < live ? r : 0.f);
                                if (l == 0) leave(TOK_ROWS * L + 2 * NB + (sb ? 2 : rb - 2), all);
                            }
                        }
                    } else {
                        const float hc = hi_s[at], lc = lo_s[at];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 32 * sb + acc_rows(i, l);
                            const f32x4 hs = *reinterpret_cast<const f32x4*>(hi_s + s), ls = *reinterpret_cast<const f32x4*>(lo_s + s),
                                        ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                z[4 * i + j] *= exp2_hw(s + j <= at ? (hc - hs[j]) + (lc - ls[j]) : -INFINITY) * ds[j];
                                m[4 * i + j] *= s + j < at && at < live ? z[4 * i + j] : 0.f;
                            }
                        }
                        // over[t][t'] = sum_{s < t} M_t's, then for every t the sum over t' >= t
                        f32x16 over = zero16();
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            Frag<T> parts[PARTS];
                            acc_parts<T>(m, b, parts);
                            const Frag<T> ones = ones_below<T>(b, l);
#pragma unroll
                            for (int p = 0; p < PARTS; ++p) over = mma32(ones, parts[p], over);
                        }
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float v = lane16_sum((l & 31) >= acc_rows(k >> 2, l) + (k & 3) ? over[k] : 0.f);
                            own_sum = (l & 15) == k ? v : own_sum;
                        }
                        own_sum += __shfl_xor(own_sum, 16);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> zv = acc_frag<T>(z, b);
#pragma unroll
                        for (int i = 0; i < TN; ++i) acc[i] = mma32(NRead::down(b_s, ndn, 32 * sb + 16 * b, 32 * i), zv, acc[i]);
                        ordered<T, TN, 2>();
                    }
                }
            }
            if (NB == 4 && 32 * rb >= live && rb > 1 && l < rb - 1) leave(TOK_ROWS * L + 2 * NB + rb - 2 + l, 0.f);
            r = half_add(r);
            if (h == 0) leave(TOK_R_BLOCKS * L + at, r);
            // lane k of 16 has the sum of register k's t
            if (!(l & 16)) leave(TOK_OWN * L + 32 * rb + acc_rows((l & 15) >> 2, l) + (l & 3), own_sum);
        } else {
            float qi = 0.f;
            if (has_d) {
                const float e = dec_s[DEC_F * L + at];
#pragma unroll
                for (int pt = 0; pt < 2; ++pt) {
                    f32x16 m = zero16();
                    const uint32_t pl = opaque(vp), row = opaque(vr);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int kk = 0; kk < KN; ++kk) m = mma32(VRead::plain(st_s[p], pl, 16 * kk, 32 * pt), own_at(kk), m);
                    ordered<T, PARTS * KN, 2>();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 xv = VRead::row4(x_s, row, pt, q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = m[4 * q + j] * e;
                            du[pt][4 * q + j] += v;
                            qi = __builtin_fmaf(xv[j], v, qi);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    f32x16 m = zero16();
                    const uint32_t al = opaque(va);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) m = mma32(VTab::along(st_s[0], al, 32 * i, kk), val_at(kk), m);
                    ordered<T, 4, 1>();
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = __builtin_fmaf(m[j], e * dc, acc[i][j]);
                }
            }
            qi = half_add(qi);
            if (h == 0) {
                leave(TOK_Q_BLOCKS * L + at, qo);
                leave(TOK_Q_STATE * L + at, qi);
                leave(TOK_XDU * L + at, xdu + qi);
                leave(TOK_XDY * L + at, zd);
            }
            if (at < live) {
                const float skip = a.D ? a.D[head] : 0.f;
                T* dx = (T*)a.dx + ((row0 + at) * a.H + head) * a.P + p0;
                const uint32_t row = opaque(vr);
#pragma unroll
                for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int p = 32 * pt + acc_rows(q, l);
                        const f32x4 yv = VRead::row4(y_s, row, pt, q);
                        float v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[j] = dc * du[pt][4 * q + j];
                            if (a.D) v[j] = __builtin_fmaf(skip, yv[j], v[j]);
                        }
                        store4<T>(dx + p, v[0], v[1], v[2], v[3]);
                    }
            }
        }
        __syncthreads();
        if (sub == per_head - 1) {  // the head's sums are complete
            float* o = a.token + ((size_t)id * a.H + head) * kTokens<L>;
            for (int i = tid; i < kTokens<L>; i += NTH) o[i] = tok_s[i];
            if (slice + 1 < h_last * per_head) __syncthreads();
        }
    }
    const int at = 32 * rb + (lane_id() & 31);
    if (at < live) {
        const size_t o = ((row0 + at) * a.G + g) * N;
        if (a.splits == 1) {
            T* out = (T*)(is_s ? a.dB : a.dC) + o;
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    store4<T>(out + 32 * i + acc_rows(q), acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
        } else {
            float* out = a.part + ((size_t)(is_s ? 0 : a.splits) + sp) * a.T * a.G * N + o;
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    store4<float>(out + 32 * i + acc_rows(q), acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
        }
    }
}

// dB and dC from the parts of a group's heads, in order: a word of 4 values a thread
template <typename T>
__global__ __launch_bounds__(256) void ssm_join_kernel(const float* __restrict__ part, const int* __restrict__ cu, T* dB,
                                                       T* dC, int nb, int tokens, int splits, int width)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, total = (long long)tokens * width / 4;
    if (i >= total) return;
    const int row = (int)(i * 4 / width);
    if (row < cu[0] || row >= cu[nb]) return;  // a row of no sequence
    const f32x4* p = reinterpret_cast<const f32x4*>(part) + (size_t)blockIdx.y * splits * total + i;
    f32x4 s = p[0];
    for (int k = 1; k < splits; ++k) s += p[(size_t)k * total];
    store4<T>((blockIdx.y ? dC : dB) + i * 4, s[0], s[1], s[2], s[3]);
}

template <typename T, int N> gdn_status grad(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, const GradArgs& a, hipStream_t st)
{
    constexpr int L = SsmTile<T>::L;
    if (p.chunks) {
        const dim3 grid((unsigned)((p.chunks + 7) / 8 * 8 * s.G * p.splits));
        GDN_LAUNCH("ssm_grad", (ssm_grad_kernel<T, N>), grid, dim3(4 * L), st, a);
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
