// ssm_out.hip -- outputs of the selective state space scan, chunk by chunk, from
// the states between them (ssm_walk.hip):
//
//   y_t = sum_{s <= t} exp(c_t - c_s) (C_t . B_s) delta_s x_s + exp(c_t) C_t S_in + D x_t
//
// A workgroup has a chunk and some of the slices (64 values of a head) of a group;
// a wave has 32 of the chunk's tokens.  It computes B C^T, so that a lane is one t
// and its registers are the s: the decay, the causal limit and delta are applied
// there, and the result is the next product's operand as it stands.  That product
// gives y^T, so that a lane stores neighbouring values of its token.  32768 tokens of 6
// heads of 128, N = 128: 55 us.  No unit is full (matrix units 13 %): a wave's loads,
// products and the vector work between them follow one another, and two workgroups share
// a compute unit.
//
// bf16: E C B^T delta is rounded to it for the product with x, and the states are read
// as bf16.  y is off by 0.0018 to 0.0020 in the 2-norm, where storing it alone is 0.0017;
// operands in two parts would be twice the products, and twice the states' bytes.
//
// A block's own pairs are masked: what is not finite in B or the steps is selected away,
// and in x kept from the products (add_masked_rest), 0.2 to 1.0 % of a call's time.
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct OutArgs {
    const void *x, *B, *C;
    const float *dec, *D;
    const int* cu;
    const void* between;  // [states][slices] states, then each sequence's first
    void* y;
    long long xs, bs, cs, firsts;
    int nb, T, H, P, per_group, slices, parts, first;
};

template <typename T, int N>
__global__ __launch_bounds__(64 * (SsmTile<T>::L / 32), 2) void ssm_out_kernel(OutArgs a)
{
    constexpr int L = SsmTile<T>::L, NW = L / 32, KN = N / 16;
    using NTab = Rows<T, N>;
    using VTab = Rows<T, kSlice>;
    using VRead = Reads<T, kSlice>;
    __shared__ __align__(16) char b_s[L * NTab::BYTES];
    __shared__ __align__(16) char x_s[L * VTab::BYTES];
    __shared__ __align__(16) char s_s[kSlice * NTab::BYTES];
    __shared__ __align__(16) float hi_s[L], lo_s[L], d_s[L], behind_s[L];

    long long id;
    int part;
    deal(blockIdx.x, a.parts, id, part);
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, 0, id, u)) return;
    const int c = u.at, live = u.n - c * L < L ? u.n - c * L : L;
    const size_t row0 = (size_t)u.start + (size_t)c * L;
    const int l = lane_id(), h = l >> 5, w = uniform(wave_id());
    // later rows have more to do: the order is turned round from block to block,
    // for the waves of two workgroups on one SIMD
    const int rb = (blockIdx.x >> 8) & 1 ? NW - 1 - w : w;
    const int per_head = a.P / kSlice, s_first = (int)((long long)part * a.slices / a.parts),
              s_last = (int)((long long)(part + 1) * a.slices / a.parts);

    Frag<T> cf[KN];
    int group = -1;
    for (int slice = s_first; slice < s_last; ++slice) {
        const int head = slice / per_head, p0 = (slice - head * per_head) * kSlice, g = head / a.per_group;
        const bool state = c > 0 || a.first;
        if (slice != s_first) __syncthreads();  // the tables are read
        if (g != group) {
            group = g;
            const T* b = (const T*)a.B + row0 * a.bs + (size_t)g * N;
            for (int r = 16 * w; r < L; r += 16 * NW) {
                const int rr = r < live ? r : live - 1;
                NTab::template fetch<16>(b_s, r, b + (size_t)rr * a.bs, (uint32_t)(a.bs * sizeof(T)), live - 1 - rr);
            }
            const int t = 32 * rb + (l & 31);
            const T* cp = (const T*)a.C + (row0 + (t < live ? t : live - 1)) * a.cs + (size_t)g * N + 8 * h;
#pragma unroll
            for (int kk = 0; kk < KN; ++kk) cf[kk] = load_frag<T>(cp + 16 * kk);
        }
        {
            const T* x = (const T*)a.x + row0 * a.xs + (size_t)head * a.P + p0;
            for (int r = 16 * w; r < L; r += 16 * NW) {
                const int rr = r < live ? r : live - 1;
                VTab::template fetch<16>(x_s, r, x + (size_t)rr * a.xs, (uint32_t)(a.xs * sizeof(T)), live - 1 - rr);
            }
        }
        if (state) {
            const T* s = (const T*)a.between + ((size_t)(c > 0 ? u.between + c - 1 : a.firsts + u.b) * a.slices + slice) * kSlice * N;
            constexpr int VE = 16 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < N / VE * kSlice / (64 * NW); ++i) {
                const int x = i * 64 * NW + threadIdx.x, p = x % kSlice, q = x / kSlice;  // word q of row p
                u32x4 word;
                if constexpr (sizeof(T) == 2) {
                    const uint2 lo = *reinterpret_cast<const uint2*>(s + (8 * q) * kSlice + 4 * p),
                                hi = *reinterpret_cast<const uint2*>(s + (8 * q + 4) * kSlice + 4 * p);
                    word = u32x4{lo.x, lo.y, hi.x, hi.y};
                } else {
                    word = *reinterpret_cast<const u32x4*>(s + (4 * q) * kSlice + 4 * p);
                }
                *reinterpret_cast<u32x4*>(s_s + NTab::word(p, q) * 16) = word;
            }
        }
        const float* dec = a.dec + ((size_t)id * a.H + head) * kDecays<L>;
        if (threadIdx.x < L) {
            const int t = threadIdx.x;
            const float d = dec[DEC_DELTA * L + t];
            hi_s[t] = dec[DEC_HI * L + t];
            lo_s[t] = dec[DEC_LO * L + t];
            d_s[t] = d;
            behind_s[t] = dec[DEC_BEHIND * L + t] * d;
        }
        const int t = 32 * rb + (l & 31);
        const float et = dec[DEC_E * L + t], ahead = dec[DEC_AHEAD * L + t];
        wait_vm<0>();
        __syncthreads();
        if (32 * rb >= live) continue;  // no token of this wave's

        const float ht = hi_s[t], lt = lo_s[t], skip = a.D ? a.D[head] : 0.f;
        f32x16 acc[2] = {zero16(), zero16()};
        if (state) {
#pragma unroll
            for (int kk = 0; kk < KN; ++kk)
#pragma unroll
                for (int pt = 0; pt < 2; ++pt) acc[pt] = mma32(NTab::along(s_s, 32 * pt, kk), cf[kk], acc[pt]);
            if (sizeof(T) == 2) order_products<2 * KN, 1, 4>();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[pt][r] *= et;
        }
        for (int sb = 0; sb <= rb; ++sb) {
            f32x16 m = zero16();
#pragma unroll
            for (int kk = 0; kk < KN; ++kk) m = mma32(NTab::along(b_s, 32 * sb, kk), cf[kk], m);
            if (sizeof(T) == 2) order_products<KN, 1, 4>();
            __builtin_amdgcn_sched_barrier(0);
            Frag<T> xf[4];  // read now, to arrive under the decays
#pragma unroll
            for (int i = 0; i < 4; ++i) xf[i] = VTab::down(x_s, 32 * sb + 16 * (i >> 1), 32 * (i & 1));
            if (sb < rb) {
                const int end = 32 * sb + 31, from = 32 * rb - 1;  // c from the one block's end to the other's start
                const float f = ahead * exp2_hw((hi_s[from] - hi_s[end]) + (lo_s[from] - lo_s[end]));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 bs = *reinterpret_cast<const f32x4*>(behind_s + 32 * sb + acc_rows(i));
#pragma unroll
                    for (int j = 0; j < 4; ++j) m[4 * i + j] *= f * bs[j];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = 32 * sb + acc_rows(i);
                    const f32x4 hs = *reinterpret_cast<const f32x4*>(hi_s + s), ls = *reinterpret_cast<const f32x4*>(lo_s + s),
                                ds = *reinterpret_cast<const f32x4*>(d_s + s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e = exp2_hw((ht - hs[j]) + (lt - ls[j])) * ds[j];
                        m[4 * i + j] = s + j <= t ? m[4 * i + j] * e : 0.f;  // selected: the others may be anything
                    }
                }
            }
            // a value that is not finite must not reach the block's earlier tokens
            const bool rest = sb == rb && !all_finite(xf);
            if (__builtin_expect(rest, 0)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) xf[i] = finite_only(xf[i]);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const Frag<T> v = acc_frag<T>(m, b);
#pragma unroll
                for (int pt = 0; pt < 2; ++pt) acc[pt] = mma32(xf[2 * b + pt], v, acc[pt]);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (__builtin_expect(rest, 0)) add_masked_rest<T, kSlice>(acc, m, x_s, 32 * sb, false);
        }
        if (t < live) {
            T* y = (T*)a.y + ((row0 + t) * a.H + head) * a.P + p0;
            const uint32_t xr = VRead::row_at(t);
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = 32 * pt + acc_rows(i);
                    f32x4 v{acc[pt][4 * i], acc[pt][4 * i + 1], acc[pt][4 * i + 2], acc[pt][4 * i + 3]};
                    if (a.D) {
                        const f32x4 x = VRead::row4(x_s, xr, pt, i);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(skip, x[j], v[j]);
                    }
                    store4<T>(y + p, v[0], v[1], v[2], v[3]);
                }
        }
    }
}

template <typename T, int N> gdn_status out(const SsmPlan& p, OutArgs a, hipStream_t st)
{
    // slices of a chunk that share its B and C: as many workgroups as there are
    // slices while they are few, then about four a compute unit
    int parts = a.slices;
    while (parts > 1 && p.chunks * (parts / 2) >= 1024) parts /= 2;
    a.parts = parts;
    const dim3 grid(dealt(p.chunks, parts));
    GDN_LAUNCH("ssm_out", (ssm_out_kernel<T, N>), grid, dim3(64 * (SsmTile<T>::L / 32)), st, a);
    return GDN_OK;
}

}  // namespace

gdn_status ssm_out(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, char* ws, hipStream_t st)
{
    OutArgs a{};
    a.x = x.x; a.B = x.B; a.C = x.C;
    a.dec = (const float*)(ws + p.dec_at);
    a.D = x.D; a.cu = x.cu;
    a.between = ws + p.fwd_at;
    a.firsts = p.between;
    a.first = x.h0 != nullptr;
    a.y = x.y;
    a.xs = x.xs; a.bs = x.bs; a.cs = x.cs;
    a.nb = s.B; a.T = s.T; a.H = s.H; a.P = s.P; a.per_group = s.H / s.G; a.slices = p.slices;
    if (s.dtype == GDN_BF16) return s.N == 64 ? out<bf16, 64>(p, a, st) : out<bf16, 128>(p, a, st);
    return s.N == 64 ? out<float, 64>(p, a, st) : out<float, 128>(p, a, st);
}

}  // namespace gdn
