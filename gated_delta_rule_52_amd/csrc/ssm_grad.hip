// ssm_grad.hip -- gradients of the selective state space scan, chunk by chunk,
// from the states S before and the gradients dS behind every chunk (ssm_walk.hip).
// With G = C B^T, Z = dy x^T, E_ts = exp(c_t - c_s) for s <= t:
//
//   du_s = sum_t E_ts G_ts dy_t + exp(c_L - c_s) dS^T B_s,     dx = delta du + D dy
//   dB_s = delta_s (sum_t E_ts Z_ts C_t + exp(c_L - c_s) dS x_s)      summed over a group's heads
//   dC_t = sum_s E_ts Z_ts delta_s B_s + exp(c_t) S dy_t              summed over a group's heads
//   dg_t = sum_{t' >= t > s} E G Z delta + sum_{t' >= t} r_t' + sum_{s < t} q_s + exp(c_L) <S, dS>
//          with r_t = exp(c_t) C_t . S dy_t,  q_s = delta_s exp(c_L - c_s) x_s . dS^T B_s
//   ddelta = A dg + x . du,   dA = sum delta dg,   dD = sum dy . x
//
// (g_t scales everything that passes from before t to t or after it.)  dg is formed
// from E, G and Z themselves and from states that are split into bf16 parts, so it
// is as exact as in fp32; where a result is stored as bf16, E G, E Z delta and one
// operand are rounded to it on the way.
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
    const float *dt, *A, *D, *bias, *h0, *dhT;
    const int* cu;
    const float *fwd, *back;  // [states][slices][N][64]
    void *dx, *dB, *dC;
    float *ddt, *part, *sums;  // part: [2][splits][T][G][N]; sums: [chunks][H][3]
    long long xs, bs, cs;
    int nb, T, H, G, P, slices, splits, plus;
};

template <typename T, int N>
__global__ __launch_bounds__(128 * (SsmTile<T>::L / 32)) void ssm_grad_kernel(GradArgs a)
{
    constexpr int L = SsmTile<T>::L, NB = L / 32, NTH = 128 * NB, PARTS = SsmTile<T>::PARTS, KN = N / 16, TN = N / 32;
    constexpr bool HOLD = sizeof(T) == 2;  // operands that are used again stay in registers
    using NTab = Rows<T, N>;
    using VTab = Rows<T, kSlice>;
    constexpr int SW = N * 8 / NTH;  // runs of 8 values of a state a thread stages
    __shared__ __align__(16) char b_s[L * NTab::BYTES], c_s[L * NTab::BYTES];
    __shared__ __align__(16) char x_s[L * VTab::BYTES], y_s[L * VTab::BYTES];
    __shared__ __align__(16) char st_s[PARTS][N * VTab::BYTES];
    __shared__ __align__(16) float hi_s[L], lo_s[L], d_s[L];
    __shared__ float ri_s[L], rp_s[L], qp_s[L], qd_s[L], qi_s[L], zd_s[L], tot_s[2], dot_s[2 * NB];

    long long id;
    int job;
    deal(blockIdx.x, a.G * a.splits, id, job);
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, id, u)) return;
    const int c = u.at, live = u.n - c * L < L ? u.n - c * L : L;
    const size_t row0 = (size_t)u.start + (size_t)c * L;
    const int l = lane_id(), h = l >> 5, w = uniform(wave_id()), tid = threadIdx.x;
    const bool is_s = w >= NB;
    const int rb = is_s ? w - NB : w, at = 32 * rb + (l & 31);  // the lane's token
    const int per_head = a.P / kSlice, per_group = a.H / a.G, g = job / a.splits, sp = job - g * a.splits;
    const int h_first = g * per_group + (int)((long long)per_group * sp / a.splits),
              h_last = g * per_group + (int)((long long)per_group * (sp + 1) / a.splits);
    const bool has_s = c > 0 || a.h0, has_d = c < u.chunks - 1 || a.dhT;

    auto rows_of = [&](char* tab, auto rows, const T* base, long long stride) {
        using R = decltype(rows);
        for (int r = 16 * w; r < L; r += 32 * NB) {
            const int rr = r < live ? r : live - 1;
            R::template fetch<16>(tab, r, base + (size_t)rr * stride, (uint32_t)(stride * sizeof(T)), live - 1 - rr);
        }
    };
    rows_of(b_s, NTab{}, (const T*)a.B + row0 * a.bs + (size_t)g * N, a.bs);
    rows_of(c_s, NTab{}, (const T*)a.C + row0 * a.cs + (size_t)g * N, a.cs);

    f32x16 acc[TN];  // dC of 32 t or dB of 32 s
#pragma unroll
    for (int i = 0; i < TN; ++i) acc[i] = zero16();
    Frag<T> own[HOLD ? KN : 1], val[HOLD ? 4 : 1];  // the lane's rows of C or B, and of dy or x
    auto own_at = [&](int kk) {
        if constexpr (HOLD) return own[kk];
        else return NTab::along(is_s ? b_s : c_s, 32 * rb, kk);
    };
    auto val_at = [&](int kk) {
        if constexpr (HOLD) return val[kk];
        else return VTab::along(is_s ? x_s : y_s, 32 * rb, kk);
    };
    bool loaded = false;

    for (int slice = h_first * per_head; slice < h_last * per_head; ++slice) {
        const int head = slice / per_head, sub = slice - head * per_head, p0 = sub * kSlice;
        rows_of(x_s, VTab{}, (const T*)a.x + row0 * a.xs + (size_t)head * a.P + p0, a.xs);
        rows_of(y_s, VTab{}, (const T*)a.dy + (row0 * a.H + head) * a.P + p0, (long long)a.H * a.P);
        // run i of this thread: row n of the state, values 8 q .. 8 q + 7
        auto run = [&](int i, int& n, int& q) {
            const int x = i * NTH + tid;
            n = x >> 3, q = x & 7;
        };
        auto state_of = [&](const float* between, long long which, const float* edge, float (&v)[SW][8]) {
            // between chunks [N][64]; at a sequence's edge [N][P]
            const float* s = edge ? edge + ((size_t)u.b * a.H + head) * N * a.P + p0
                                  : between + ((size_t)which * a.slices + slice) * N * kSlice;
            const int stride = edge ? a.P : kSlice;
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int n, q;
                run(i, n, q);
                const f32x4 e = *reinterpret_cast<const f32x4*>(s + (size_t)n * stride + 8 * q),
                            f = *reinterpret_cast<const f32x4*>(s + (size_t)n * stride + 8 * q + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = e[j], v[i][4 + j] = f[j];
            }
        };
        auto put_state = [&](const float (&v)[SW][8]) {
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int n, q;
                run(i, n, q);
                if constexpr (sizeof(T) == 2) {
                    u32x4 parts[3];
                    split(v[i], parts);
#pragma unroll
                    for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4*>(st_s[p] + VTab::word(n, q) * 16) = parts[p];
                } else {
                    *reinterpret_cast<f32x4*>(st_s[0] + VTab::word(n, 2 * q) * 16) = f32x4{v[i][0], v[i][1], v[i][2], v[i][3]};
                    *reinterpret_cast<f32x4*>(st_s[0] + VTab::word(n, 2 * q + 1) * 16) = f32x4{v[i][4], v[i][5], v[i][6], v[i][7]};
                }
            }
        };
        float sv[SW][8], dv[SW][8];
        if (has_s) {
            state_of(a.fwd, u.between + c - 1, c > 0 ? nullptr : a.h0, sv);
            put_state(sv);
        }
        if (has_d) state_of(a.back, u.between + c, c < u.chunks - 1 ? nullptr : a.dhT, dv);
        if (w == 0 && sub == 0) {
            Decays<L> dec;
            dec.load(a.dt + row0 * a.H + head, a.H, live, a.bias ? a.bias[head] : 0.f);
            dec.scan(a.A[head], a.plus, live);
#pragma unroll
            for (int k = 0; k < Decays<L>::K; ++k) {
                const int t = Decays<L>::K * l + k;
                const float hi = (float)dec.c[k];
                hi_s[t] = hi;
                lo_s[t] = (float)(dec.c[k] - (double)hi);
                d_s[t] = dec.d[k];
            }
            if (l == 0) {
                tot_s[0] = (float)dec.total;
                tot_s[1] = (float)(dec.total - (double)(float)dec.total);
            }
        }
        wait_vm<0>();
        __syncthreads();

        if constexpr (HOLD) {
            if (!loaded) {
#pragma unroll
                for (int kk = 0; kk < KN; ++kk) own[kk] = NTab::along(is_s ? b_s : c_s, 32 * rb, kk);
                loaded = true;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) val[kk] = VTab::along(is_s ? x_s : y_s, 32 * rb, kk);
        }
        const float hc = hi_s[at], lc = lo_s[at], dc = d_s[at];
        f32x16 du[2] = {zero16(), zero16()};
        float qp = 0.f, qd = 0.f, zd = 0.f;
        if (!is_s) {
            float r = 0.f;
            if (has_s) {
                const float e = exp2_hw(hc + lc);
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    f32x16 m = zero16();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) m = mma32(VTab::along(st_s[p], 32 * i, kk), val_at(kk), m);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 cv = row4<T, N>(c_s, at, 32 * i + acc_rows(q));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = m[4 * q + j] * e;
                            acc[i][4 * q + j] += v;
                            r = __builtin_fmaf(cv[j], v, r);
                        }
                    }
                }
            }
            r = half_add(r);
            if (h == 0) ri_s[at] = sub ? ri_s[at] + r : r;
        } else if (32 * rb < live) {
            for (int tb = rb; tb < NB; ++tb) {
                if (32 * tb >= live) break;
                f32x16 m = zero16(), z = zero16();
#pragma unroll
                for (int kk = 0; kk < KN; ++kk) m = mma32(NTab::along(c_s, 32 * tb, kk), own_at(kk), m);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(y_s, 32 * tb, kk), val_at(kk), z);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 32 * tb + acc_rows(i);
                    const f32x4 ht = *reinterpret_cast<const f32x4*>(hi_s + t), lt = *reinterpret_cast<const f32x4*>(lo_s + t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = at <= t + j && t + j < live;
                        const float e = in ? exp2_hw((ht[j] - hc) + (lt[j] - lc)) : 0.f;
                        const float mv = in ? m[4 * i + j] : 0.f, zv = in ? z[4 * i + j] : 0.f;
                        const float eg = e * mv, p = eg * zv;
                        if (t + j == at) {
                            qd = p;
                            zd = zv;
                        } else {
                            qp += p;
                        }
                        m[4 * i + j] = eg;
                        z[4 * i + j] = e * zv * dc;
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const Frag<T> mv = acc_frag<T>(m, b), zv = acc_frag<T>(z, b);
#pragma unroll
                    for (int pt = 0; pt < 2; ++pt) du[pt] = mma32(VTab::down(y_s, 32 * tb + 16 * b, 32 * pt), mv, du[pt]);
#pragma unroll
                    for (int i = 0; i < TN; ++i) acc[i] = mma32(NTab::down(c_s, 32 * tb + 16 * b, 32 * i), zv, acc[i]);
                }
            }
            qp = half_add(qp);
            qd = half_add(qd);  // the pair t = s is one half's
            zd = half_add(zd);
        }
        __syncthreads();
        float dot = 0.f;
        if (has_d) {
            put_state(dv);
            if (has_s) {
#pragma unroll
                for (int i = 0; i < SW; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(sv[i][j], dv[i][j], dot);
            }
        }
        dot = wave_sum(dot);
        if (l == 0) dot_s[w] = sub ? dot_s[w] + dot : dot;
        __syncthreads();
        if (!is_s) {
            float r = 0.f;
            if (32 * rb < live) {
                for (int sb = 0; sb <= rb; ++sb) {
                    f32x16 m = zero16(), z = zero16();
#pragma unroll
                    for (int kk = 0; kk < KN; ++kk) m = mma32(NTab::along(b_s, 32 * sb, kk), own_at(kk), m);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) z = mma32(VTab::along(x_s, 32 * sb, kk), val_at(kk), z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = 32 * sb + acc_rows(i);
                        const f32x4 hs = *reinterpret_cast<const f32x4*>(hi_s + s), ls = *reinterpret_cast<const f32x4*>(lo_s + s),
                                    ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e = exp2_hw((hc - hs[j]) + (lc - ls[j])) * ds[j];
                            const float ez = s + j <= at ? e * z[4 * i + j] : 0.f;
                            r += s + j < at ? ez * m[4 * i + j] : 0.f;
                            z[4 * i + j] = ez;
                        }
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const Frag<T> zv = acc_frag<T>(z, b);
#pragma unroll
                        for (int i = 0; i < TN; ++i) acc[i] = mma32(NTab::down(b_s, 32 * sb + 16 * b, 32 * i), zv, acc[i]);
                    }
                }
            }
            r = half_add(r);
            if (h == 0) rp_s[at] = sub ? rp_s[at] + r : r;
        } else {
            float qi = 0.f;
            if (has_d) {
                const float e = exp2_hw((tot_s[0] - hc) + (tot_s[1] - lc));
#pragma unroll
                for (int pt = 0; pt < 2; ++pt) {
                    f32x16 m = zero16();
#pragma unroll
                    for (int kk = 0; kk < KN; ++kk)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) m = mma32(down_plain<T, kSlice>(st_s[p], 16 * kk, 32 * pt), own_at(kk), m);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 xv = row4<T, kSlice>(x_s, at, 32 * pt + acc_rows(q));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = m[4 * q + j] * e;
                            du[pt][4 * q + j] += v;
                            qi = __builtin_fmaf(xv[j], v, qi);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    f32x16 m = zero16();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) m = mma32(VTab::along(st_s[0], 32 * i, kk), val_at(kk), m);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = __builtin_fmaf(m[j], e * dc, acc[i][j]);
                }
            }
            qi = half_add(qi);
            if (h == 0) {
                qp_s[at] = sub ? qp_s[at] + qp : qp;
                qd_s[at] = sub ? qd_s[at] + qd : qd;
                qi_s[at] = sub ? qi_s[at] + qi : qi;
                zd_s[at] = sub ? zd_s[at] + zd : zd;
            }
            if (at < live) {
                const float skip = a.D ? a.D[head] : 0.f;
                T* dx = (T*)a.dx + ((row0 + at) * a.H + head) * a.P + p0;
#pragma unroll
                for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int p = 32 * pt + acc_rows(q);
                        const f32x4 yv = row4<T, kSlice>(y_s, at, p);
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
        if (w == 0 && sub == per_head - 1) {  // the head's sums are complete
            constexpr int K = L / 64;
            double f[K], q[K], fs = 0, qs = 0;
            float d[K], xdu[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int t = K * l + k;
                const bool in = t < live;
                d[k] = d_s[t];
                xdu[k] = in ? qp_s[t] + qd_s[t] + qi_s[t] : 0.f;
                f[k] = in ? (double)ri_s[t] + (double)rp_s[t] - (double)d[k] * (double)qp_s[t] : 0.0;
                q[k] = in ? (double)d[k] * (double)qi_s[t] : 0.0;
                fs += f[k];
                qs += q[k];
            }
            double fi = fs, qi = qs;  // inclusive sums over the lanes
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double a1 = shift_up(fi, o), a2 = shift_up(qi, o);
                if (l >= o) fi += a1, qi += a2;
            }
            double run = __shfl(fi, 63) - (fi - fs), past = qi - qs;  // from the lane's first token on; before it
            float dot_all = 0.f;
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) dot_all += dot_s[k];
            const double through = has_s && has_d ? (double)(exp2_hw(tot_s[0] + tot_s[1]) * dot_all) : 0.0;
            const float A = a.A[head], bias = a.bias ? a.bias[head] : 0.f;
            double sa = 0, sd = 0, sb = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int t = K * l + k;
                const double dg = run + past + through;
                run -= f[k];
                past += q[k];
                if (t < live) {
                    const size_t o = (row0 + t) * a.H + head;
                    float dd = (float)((double)A * dg + (double)xdu[k]);
                    if (a.plus) dd *= 1.f / (1.f + expf(-(a.dt[o] + bias)));
                    a.ddt[o] = dd;
                    sa += (double)d[k] * dg;
                    sd += (double)zd_s[t];
                    sb += (double)dd;
                }
            }
#pragma unroll
            for (int o = 32; o; o >>= 1) {
                sa += __shfl_xor(sa, o);
                sd += __shfl_xor(sd, o);
                sb += __shfl_xor(sb, o);
            }
            if (l == 0) {
                float* s = a.sums + ((size_t)id * a.H + head) * 3;
                s[0] = (float)sa, s[1] = (float)sd, s[2] = (float)sb;
            }
        }
    }
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

// dA, dD and dbias of head blockIdx.x from the chunks' sums
template <int L>
__global__ __launch_bounds__(256) void ssm_sums_kernel(const float* __restrict__ sums, const int* __restrict__ cu, int nb,
                                                       int T, int H, float* dA, float* dD, float* dbias)
{
    __shared__ double red[4][3];
    const int l = lane_id(), head = blockIdx.x;
    long long chunks = 0;
    for (int b0 = 0; b0 < nb; b0 += 64) {
        const int b = b0 + l < nb ? b0 + l : nb - 1;
        int st = cu[b], en = cu[b + 1];
        st = st < 0 ? 0 : st > T ? T : st;
        en = en < st ? st : en > T ? T : en;
        chunks += wave_sum(b0 + l < nb ? (en - st + L - 1) / L : 0);
    }
    double s[3] = {0, 0, 0};
    for (long long i = threadIdx.x; i < chunks; i += 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += (double)sums[((size_t)i * H + head) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 32; o; o >>= 1) s[k] += __shfl_xor(s[k], o);
        if (l == 0) red[wave_id()][k] = s[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        const int k = threadIdx.x;
        float* out = k == 0 ? dA : k == 1 ? dD : dbias;
        if (out) out[head] = (float)((red[0][k] + red[1][k]) + (red[2][k] + red[3][k]));
    }
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
    GDN_LAUNCH("ssm_sums", (ssm_sums_kernel<L>), dim3(s.H), dim3(256), st, a.sums, a.cu, s.B, s.T, s.H, x.dA, x.dD, x.dbias);
    return GDN_OK;
}

}  // namespace

gdn_status ssm_grad(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, char* ws, hipStream_t st)
{
    GradArgs a{};
    a.x = x.x; a.B = x.B; a.C = x.C; a.dy = x.dy;
    a.dt = x.dt; a.A = x.A; a.D = x.D; a.bias = x.bias; a.h0 = x.h0; a.dhT = x.dhT; a.cu = x.cu;
    a.fwd = (const float*)(ws + p.fwd_at);
    a.back = (const float*)(ws + p.back_at);
    a.dx = x.dx; a.dB = x.dB; a.dC = x.dC; a.ddt = x.ddt;
    a.part = (float*)(ws + p.part_at);
    a.sums = (float*)(ws + p.sum_at);
    a.xs = x.xs; a.bs = x.bs; a.cs = x.cs;
    a.nb = s.B; a.T = s.T; a.H = s.H; a.G = s.G; a.P = s.P; a.slices = p.slices; a.splits = p.splits; a.plus = s.softplus;
    if (s.dtype == GDN_BF16) return s.N == 64 ? grad<bf16, 64>(s, p, x, a, st) : grad<bf16, 128>(s, p, x, a, st);
    return s.N == 64 ? grad<float, 64>(s, p, x, a, st) : grad<float, 128>(s, p, x, a, st);
}

}  // namespace gdn
