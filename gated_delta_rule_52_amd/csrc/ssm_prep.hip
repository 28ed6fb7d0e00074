// ssm_prep.hip -- steps and decays of the selective state space scan, chunk by chunk
// (DEC_* in ssm_tile.h), which all its other kernels read; and, behind the
// gradients' products (ssm_grad.hip), the gradients of the steps from the sums that
// those leave of every token.  A wave has a chunk and a head; its running sums are
// in 64 bits.  Small: 6 heads of 32768 tokens have 0.8 MB of steps and 6.3 MB of decays
// (5 us, latency; the steps' gradients 9 us).
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

// sum over the lanes up to and with the lane itself
__device__ __forceinline__ double wave_scan(double x)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_up(x, o);
        if (lane_id() >= o) x += up;
    }
    return x;
}
// sums over the other lanes of a run of W, before the lane and behind it
template <int W> __device__ __forceinline__ double lanes_before(double x)
{
    const int at = lane_id() % W;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
        const double up = __shfl_up(x, o, W);
        if (at >= o) x += up;
    }
    x = __shfl_up(x, 1, W);
    return at ? x : 0.0;
}
template <int W> __device__ __forceinline__ double lanes_behind(double x)
{
    const int at = lane_id() % W;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
        const double down = __shfl_down(x, o, W);
        if (at + o < W) x += down;
    }
    x = __shfl_down(x, 1, W);
    return at < W - 1 ? x : 0.0;
}
__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

struct PrepArgs {
    const float *dt, *A, *bias;
    const int* cu;
    float* dec;  // [chunks][H][kDecays]
    int nb, T, H, plus;
};

// blockIdx.x: chunk, blockIdx.y: four heads
template <int L>
__global__ __launch_bounds__(256) void ssm_prep_kernel(PrepArgs a)
{
    constexpr int K = L / 64, LB = 32 / K;  // tokens a lane; lanes a block of 32 tokens
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, 0, blockIdx.x, u)) return;
    const int head = blockIdx.y * 4 + wave_id(), l = lane_id();
    if (head >= a.H) return;
    const int live = u.n - u.at * L < L ? u.n - u.at * L : L;
    const size_t row0 = (size_t)u.start + (size_t)u.at * L;
    const float bias = a.bias ? a.bias[head] : 0.f;
    const double a2 = (double)a.A[head] * 1.4426950408889634;
    float d[K];
    double c[K], run = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = K * l + k;
        const bool in = t < live;
        const float raw = a.dt[(row0 + (in ? t : live - 1)) * a.H + head] + bias;
        d[k] = in ? (a.plus ? softplus(raw) : raw) : 0.f;
        run += in ? (double)d[k] * a2 : 0.0;
        c[k] = run;
    }
    // of the lanes before: not a difference, in which a step that is not finite would
    // reach the lane's earlier tokens
    const double s = wave_scan(run), total = __shfl(s, 63), up = __shfl_up(s, 1), ahead = l ? up : 0.0;
    const double end = __shfl(s, (l / LB) * LB + LB - 1);
    const double before = __shfl(s, (l / LB) * LB - 1 < 0 ? 0 : (l / LB) * LB - 1);
    const double start = l < LB ? 0.0 : before;
    float* o = a.dec + ((size_t)blockIdx.x * a.H + head) * kDecays<L>;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = K * l + k;
        const double x = c[k] + ahead;
        const float hi = (float)x;
        o[DEC_HI * L + t] = hi;
        o[DEC_LO * L + t] = (float)(x - (double)hi);
        o[DEC_DELTA * L + t] = d[k];
        const float f = exp2_hw((float)(total - x));
        o[DEC_E * L + t] = t < live ? exp2_hw((float)x) : 0.f;
        o[DEC_F * L + t] = f;
        o[DEC_FD * L + t] = f * d[k];
        o[DEC_AHEAD * L + t] = exp2_hw((float)(x - start));
        o[DEC_BEHIND * L + t] = exp2_hw((float)(end - x));
    }
    if (l == 0) {
        o[DEC_ROWS * L + DEC_KEEP] = exp2_hw((float)total);
        o[DEC_ROWS * L + DEC_TOTAL] = (float)total;
    }
}

struct FinishArgs {
    const float *dt, *A, *bias, *dec, *token;
    const int* cu;
    float *ddt, *sums;  // sums: [chunks][H][3]
    int nb, T, H, plus;
};

// ddelta = A dg + x . du, dg of a token t of block b, over the pairs t' >= t > s:
// both in b; t' in b and s before it; s in b and t' behind it; neither; and what
// comes from the state before the chunk or goes into the one behind it.  No two of
// these cancel, so dg is as exact as its terms.
template <int L>
__global__ __launch_bounds__(256) void ssm_finish_kernel(FinishArgs a)
{
    constexpr int K = L / 64, LB = 32 / K, NB = L / 32;
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, L, 0, 0, blockIdx.x, u)) return;
    const int head = blockIdx.y * 4 + wave_id(), l = lane_id();
    if (head >= a.H) return;
    const int live = u.n - u.at * L < L ? u.n - u.at * L : L;
    const size_t row0 = (size_t)u.start + (size_t)u.at * L, at = (size_t)blockIdx.x * a.H + head;
    const float *v = a.token + at * kTokens<L>, *dec = a.dec + at * kDecays<L>;
    float d[K], xdu[K], zd[K], dgd[K];
    double ri[K], ro[K], qo[K], qi[K], sri = 0, sro = 0, sqo = 0, sqi = 0;  // of the lane
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = K * l + k;
        const bool in = t < live;
        d[k] = dec[DEC_DELTA * L + t];
        ri[k] = in ? (double)v[TOK_R_STATE * L + t] : 0.0;
        ro[k] = in ? (double)v[TOK_R_BLOCKS * L + t] : 0.0;
        qi[k] = in ? (double)d[k] * (double)v[TOK_Q_STATE * L + t] : 0.0;
        qo[k] = in ? (double)d[k] * (double)v[TOK_Q_BLOCKS * L + t] : 0.0;
        xdu[k] = v[TOK_XDU * L + t];
        zd[k] = in ? v[TOK_XDY * L + t] : 0.f;
        dgd[k] = v[TOK_OWN * L + t];
        sri += ri[k], sro += ro[k], sqo += qo[k], sqi += qi[k];
    }
    // of the lanes behind, to the chunk's and to the block's end, and of those before, from
    // their starts: no differences, in which a token that is not finite would reach others
    const double all_r = lanes_behind<64>(sri), own_r = lanes_behind<LB>(sro), own_q = lanes_before<LB>(sqo),
                 all_q = lanes_before<64>(sqi);
    const float* more = v + TOK_ROWS * L;
    double rest = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) rest += (double)more[b];  // <S, dS>
    rest *= (double)dec[DEC_ROWS * L + DEC_KEEP];
    if constexpr (NB == 4) {  // across blocks 1 and 2
        const int b = l / LB;
        if (b == 1) rest += (double)more[4] + (double)more[5];
        if (b == 2) rest += (double)more[6];
    }
    const float A = a.A[head], bias = a.bias ? a.bias[head] : 0.f;
    double sa = 0, sd = 0, sb = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = K * l + k;
        double dg = all_r + own_r + own_q + all_q + rest + (double)dgd[k];
#pragma unroll
        for (int j = 0; j < K; ++j) dg += j < k ? qi[j] + qo[j] : ri[j] + ro[j];
        if (t < live) {
            const size_t o = (row0 + t) * a.H + head;
            double dd = (double)A * dg + (double)xdu[k];
            if (a.plus) dd *= (double)(1.f / (1.f + expf(-(a.dt[o] + bias))));
            a.ddt[o] = (float)dd;
            sa += (double)d[k] * dg;
            sd += (double)zd[k];
            sb += dd;
        }
    }
    sa = wave_sum(sa), sd = wave_sum(sd), sb = wave_sum(sb);
    if (l == 0) {
        float* s = a.sums + at * 3;
        s[0] = (float)sa, s[1] = (float)sd, s[2] = (float)sb;
    }
}

// dA, dD and dbias of head blockIdx.x from the chunks' sums
template <int L>
__global__ __launch_bounds__(256) void ssm_sums_kernel(const float* __restrict__ sums, const int* __restrict__ cu, int nb,
                                                       int T, int H, float* dA, float* dD, float* dbias)
{
    __shared__ double red[4][3];
    const int l = lane_id(), head = blockIdx.x;
    long long chunks = 0;
    int top = 0, st, en;
    for (int b0 = 0; b0 < nb; b0 += 64) {
        ordered_bounds(cu, nb, T, b0, top, st, en);
        chunks += gdn::wave_sum(b0 + l < nb ? (en - st + L - 1) / L : 0);
    }
    double s[3] = {0, 0, 0};
    for (long long i = threadIdx.x; i < chunks; i += 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += (double)sums[((size_t)i * H + head) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = wave_sum(s[k]);
        if (l == 0) red[wave_id()][k] = s[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        const int k = threadIdx.x;
        float* out = k == 0 ? dA : k == 1 ? dD : dbias;
        if (out) out[head] = (float)((red[0][k] + red[1][k]) + (red[2][k] + red[3][k]));
    }
}

template <int L> gdn_status prep(const gdn_ssm_shape& s, const SsmPlan& p, const PrepArgs& a, hipStream_t st)
{
    GDN_LAUNCH("ssm_prep", (ssm_prep_kernel<L>), dim3((unsigned)p.chunks, (s.H + 3) / 4), dim3(256), st, a);
    return GDN_OK;
}

template <int L> gdn_status finish(const gdn_ssm_shape& s, const SsmPlan& p, const FinishArgs& a, const SsmArgs& x, hipStream_t st)
{
    if (p.chunks)
        GDN_LAUNCH("ssm_finish", (ssm_finish_kernel<L>), dim3((unsigned)p.chunks, (s.H + 3) / 4), dim3(256), st, a);
    GDN_LAUNCH("ssm_sums", (ssm_sums_kernel<L>), dim3(s.H), dim3(256), st, a.sums, a.cu, s.B, s.T, s.H, x.dA, x.dD, x.dbias);
    return GDN_OK;
}

}  // namespace

gdn_status ssm_prep(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, char* ws, hipStream_t st)
{
    if (!p.chunks) return GDN_OK;
    PrepArgs a{};
    a.dt = x.dt; a.A = x.A; a.bias = x.bias; a.cu = x.cu;
    a.dec = (float*)(ws + p.dec_at);
    a.nb = s.B; a.T = s.T; a.H = s.H; a.plus = s.softplus;
    return s.dtype == GDN_BF16 ? prep<SsmTile<bf16>::L>(s, p, a, st) : prep<SsmTile<float>::L>(s, p, a, st);
}

gdn_status ssm_finish(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, char* ws, hipStream_t st)
{
    FinishArgs a{};
    a.dt = x.dt; a.A = x.A; a.bias = x.bias; a.cu = x.cu;
    a.dec = (const float*)(ws + p.dec_at);
    a.token = (const float*)(ws + p.token_at);
    a.ddt = x.ddt;
    a.sums = (float*)(ws + p.sum_at);
    a.nb = s.B; a.T = s.T; a.H = s.H; a.plus = s.softplus;
    return s.dtype == GDN_BF16 ? finish<SsmTile<bf16>::L>(s, p, a, x, st) : finish<SsmTile<float>::L>(s, p, a, x, st);
}

}  // namespace gdn
