// ssm_step.hip -- one token of the selective state space scan for every sequence and
// head, the state updated in place, and the plan of the longer calls.
//
//   S <- exp(delta A) S + delta B x^T,   y = S^T C + D x
//
// The state is the whole cost: it is read once and written once, by a workgroup a
// (sequence, head) that holds it in registers in between; y is summed over N within
// the lanes that share four of the P values, then across the waves in LDS, in order.
// 256 sequences of 16 heads of 64, N = 128, bf16: 50 us, 5.3 TB/s of the state's bytes.
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct StepArgs {
    const void *x, *B, *C;
    const float *dt, *A, *D, *bias;
    float* state;
    void* y;
    long long xs, bs, cs;
    int H, per_group, plus;
};

template <typename T, int N, int P>
__global__ __launch_bounds__(256) void ssm_step_kernel(StepArgs a)
{
    constexpr int LANES = P / 4, ROWS = 256 / LANES, NP = N / ROWS;  // lanes a row, rows a pass, passes
    __shared__ float b_s[N], c_s[N];
    __shared__ __align__(16) float red[4][P];
    const int head = blockIdx.x % a.H, b = blockIdx.x / a.H, tid = threadIdx.x, g = head / a.per_group;
    const int p = tid % LANES * 4, n0 = tid / LANES;
    float* s = a.state + (size_t)blockIdx.x * N * P + p;
    f32x4 v[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = *reinterpret_cast<const f32x4*>(s + (size_t)(n0 + i * ROWS) * P);
    const float raw = a.dt[(size_t)b * a.H + head] + (a.bias ? a.bias[head] : 0.f), d = a.plus ? softplus(raw) : raw;
    const float keep = expf(d * a.A[head]);
    if (tid < N) {
        b_s[tid] = to_f32(((const T*)a.B)[(size_t)b * a.bs + (size_t)g * N + tid]);
        c_s[tid] = to_f32(((const T*)a.C)[(size_t)b * a.cs + (size_t)g * N + tid]);
    }
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = to_f32(((const T*)a.x)[(size_t)b * a.xs + (size_t)head * P + p + j]);
    __syncthreads();
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int n = n0 + i * ROWS;
        const float u = d * b_s[n], cn = c_s[n];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i][j] = __builtin_fmaf(v[i][j], keep, u * x[j]);
            y[j] = __builtin_fmaf(v[i][j], cn, y[j]);
        }
        *reinterpret_cast<f32x4*>(s + (size_t)n * P) = v[i];
    }
#pragma unroll
    for (int o = LANES; o < 64; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], o);
    if ((tid & 63) < LANES) *reinterpret_cast<f32x4*>(red[tid >> 6] + p) = f32x4{y[0], y[1], y[2], y[3]};
    __syncthreads();
    if (tid < LANES) {
        const float skip = a.D ? a.D[head] : 0.f;
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[j] = (red[0][p + j] + red[1][p + j]) + (red[2][p + j] + red[3][p + j]);
            if (a.D) o[j] = __builtin_fmaf(skip, x[j], o[j]);
        }
        store4<T>((T*)a.y + (size_t)blockIdx.x * P + p, o[0], o[1], o[2], o[3]);
    }
}

template <typename T> gdn_status step(const gdn_ssm_shape& s, const StepArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)(s.B * s.H));
    if (s.N == 64 && s.P == 64)
        GDN_LAUNCH("ssm_step", (ssm_step_kernel<T, 64, 64>), grid, dim3(256), st, a);
    else if (s.N == 64)
        GDN_LAUNCH("ssm_step", (ssm_step_kernel<T, 64, 128>), grid, dim3(256), st, a);
    else if (s.P == 64)
        GDN_LAUNCH("ssm_step", (ssm_step_kernel<T, 128, 64>), grid, dim3(256), st, a);
    else
        GDN_LAUNCH("ssm_step", (ssm_step_kernel<T, 128, 128>), grid, dim3(256), st, a);
    return GDN_OK;
}

}  // namespace

gdn_status ssm_step(const gdn_ssm_shape& s, const SsmArgs& x, float* state, hipStream_t st)
{
    StepArgs a{};
    a.x = x.x; a.B = x.B; a.C = x.C;
    a.dt = x.dt; a.A = x.A; a.D = x.D; a.bias = x.bias;
    a.state = state; a.y = x.y;
    a.xs = x.xs; a.bs = x.bs; a.cs = x.cs;
    a.H = s.H; a.per_group = s.H / s.G; a.plus = s.softplus;
    return s.dtype == GDN_BF16 ? step<bf16>(s, a, st) : step<float>(s, a, st);
}

SsmPlan ssm_plan(const gdn_ssm_shape& s, bool backward)
{
    SsmPlan p{};
    const long long e = s.dtype == GDN_BF16 ? 2 : 4;
    p.L = s.dtype == GDN_BF16 ? SsmTile<bf16>::L : SsmTile<float>::L;
    p.slices = s.H * (s.P / kSlice);
    p.pairs = (p.slices / s.G + 1) / 2;
    p.chunks = s.T ? s.T / p.L + (s.B < s.T ? s.B : s.T) : 0;
    p.between = s.T / p.L;  // n tokens have ceil(n / L) - 1 <= n / L states between their chunks
    // Segments: the first launch walks all but the last of a sequence's, the last one
    // all but the first.  As many as keep either launch within two workgroups a compute
    // unit, which is what fits; three at least (two are as long as one, in two
    // launches), none below 2 chunks.
    const long long whole = (long long)s.B * s.G * p.pairs * (backward ? 2 : 1), each = (p.between + s.B - 1) / s.B;
    long long want = 1 + 512 / whole, seg = 0;
    if (want > 32) want = 32;
    if (want > 2 && each > 6) {
        seg = (each + want - 1) / want;
        if (seg < 2) seg = 2;
    }
    // Where there are workgroups enough, or the mean sequence is short, one may still be
    // long (a prompt among single tokens): none walks more than 4 times the mean length,
    // or 32 chunks, in a row.  16 heads of 64, N = 128: 65536 tokens among 255 single ones
    // 512 us (in a row 2100); 256 sequences of 256, for which nothing is cut, 316 (299).
    if (!seg) {
        const long long most = 4 * each < 32 ? 32 : 4 * each;
        if (p.between > 2 * most) seg = most;
    }
    p.seg = (int)seg;
    p.segs = seg ? s.T / (seg * p.L) + s.B : s.B;
    // n tokens that are more than one segment's are less than 2 n / (seg L) of them
    p.several = seg ? 2LL * s.T / (seg * p.L) : 0;
    if (p.several > p.segs) p.several = p.segs;
    // Parts of a group's heads in the gradients: until there is a workgroup for every
    // compute unit (it takes nearly all of its LDS).
    p.splits = 1;
    const int per_group = s.H / s.G;
    while (backward && p.chunks && p.splits * 2 <= per_group && p.chunks * s.G * p.splits < 256) p.splits *= 2;
    size_t at = 0;
    auto take = [&](long long bytes) {
        const size_t was = at;
        at += (size_t)((bytes + 255) / 256 * 256);
        return was;
    };
    const long long state = (long long)p.slices * s.N * kSlice;
    const int ways = backward ? 2 : 1;
    p.dec_at = take(p.chunks * s.H * (p.L == 128 ? kDecays<128> : kDecays<64>) * 4);
    p.seg_at = take(ways * p.several * state * 4);
    p.tot_at = take(ways * p.several * p.slices * 4);
    p.fwd_at = take(backward ? p.between * state * 4 : (p.between + s.B) * state * e);
    if (backward) {
        p.back_at = take(p.between * state * 4);
        p.token_at = take(p.chunks * s.H * (p.L == 128 ? kTokens<128> : kTokens<64>) * 4);
        p.sum_at = take(p.chunks * s.H * 12);
        p.part_at = take(p.splits > 1 ? 2LL * p.splits * s.T * s.G * s.N * 4 : 0);
    }
    p.bytes = at < 256 ? 256 : at;
    return p;
}

}  // namespace gdn
