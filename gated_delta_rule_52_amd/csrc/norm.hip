// norm.hip -- the norms around a block: residual add with a residual scale and
// RMS norm before it (gdn_norm_block), RMS norm of every head with weight and
// silu gate after it (gdn_norm_gate), each with its gradients.
//
//   h = x + a o y,   r = 1 / sqrt(mean(h^2) + eps),   n = r h o w
//   dh' = dh + r (g - xh mean(g o xh)),  g = dn o w,  xh = r h
//   dx = dh',  dy = a o dh',  dw = sum_rows dn o xh,  da = sum_rows y o dh'
//
//   y = oh o w o s(z),  oh = r o_,  s(z) = z / (1 + exp(-z))
//   do = r (g - oh mean(g o oh)),  g = dy o s(z) o w
//   dz = dy o oh o w o s'(z),  dw = sum_rows dy o s(z) o oh
//
// Everything is computed in fp32 and rounded once, when stored; h enters the
// norm unrounded (the backward forms it again from x and y, which it reads
// anyway for da).  All of these are bound by HBM: each value is read once and
// written once, as 16-byte words.  Forward and backward together move 503 MB at
// 4.8 TB/s (block norm, 32768 x 768 bf16, 104 us) and 403 MB at 5.4 TB/s (gated
// norm, 32768 x 6 x 128 bf16, 75 us); a copy of 256 MB reaches 5.5 TB/s.
#include "common.h"
#include "norm.h"

namespace gdn {

namespace {

// A word of an output.  PAST: not to be kept in the L2, for outputs that it could
// not hold until the next kernel anyway (past_l2).  At 32768 x 768 bf16 the block
// norm forward and backward take 104 us with it and 113 us without, the gated
// norm at 32768 x 6 x 128 75 us and 84 us.
template <bool PAST> __device__ __forceinline__ void put(u32x4* p, u32x4 w)
{
    if constexpr (PAST)
        __builtin_nontemporal_store(w, p);
    else
        *p = w;
}

// VE elements in one 16-byte word
template <typename T> struct Vec;
template <> struct Vec<bf16> {
    static constexpr int VE = 8;
    static __device__ __forceinline__ void load(const bf16* p, float (&v)[8])
    {
        open(*reinterpret_cast<const u32x4*>(p), v);
    }
    static __device__ __forceinline__ void open(u32x4 w, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    template <bool PAST> static __device__ __forceinline__ void store(bf16* p, const float (&v)[8])
    {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = cvt2_bf16(v[2 * i], v[2 * i + 1]);
        put<PAST>(reinterpret_cast<u32x4*>(p), w);
    }
};
template <> struct Vec<float> {
    static constexpr int VE = 4;
    static __device__ __forceinline__ void load(const float* p, float (&v)[4])
    {
        open(*reinterpret_cast<const u32x4*>(p), v);
    }
    static __device__ __forceinline__ void open(u32x4 w, float (&v)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
    template <bool PAST> static __device__ __forceinline__ void store(float* p, const float (&v)[4])
    {
        put<PAST>(reinterpret_cast<u32x4*>(p), __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    }
};

template <int VE> __device__ __forceinline__ void load_f32(const float* p, float (&v)[VE])
{
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(p + i);
        v[i] = w[0], v[i + 1] = w[1], v[i + 2] = w[2], v[i + 3] = w[3];
    }
}
template <int VE> __device__ __forceinline__ void store_f32(float* p, const float (&v)[VE])
{
#pragma unroll
    for (int i = 0; i < VE; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// sum over aligned groups of L lanes, the same bits in every lane of the group;
// L = 256 is the whole workgroup of four waves (one LDS word a wave; `slot`
// alternates between two sets so that one barrier a sum is enough)
template <int L> __device__ __forceinline__ float group_sum(float x, float (*red)[4], int slot)
{
    if (L >= 2) x += dpp_mov<0xB1>(x);
    if (L >= 4) x += dpp_mov<0x4E>(x);
    if (L >= 8) x += dpp_mov<0x141>(x);
    if (L >= 16) x += dpp_mov<0x140>(x);
    if (L >= 32) x += __shfl_xor(x, 16);
    if (L >= 64) x += __shfl_xor(x, 32);
    if (L == 256) {
        if (lane_id() == 0) red[slot][wave_id()] = x;
        __syncthreads();
        x = (red[slot][0] + red[slot][1]) + (red[slot][2] + red[slot][3]);
    }
    return x;
}

// ---------------------------------------------------------------------------
// residual add and norm.  A row is held by L lanes, N words each.
// ---------------------------------------------------------------------------
// x and y are not __restrict__: h may be either of them.  A lane stores only the
// words of its own row that it has loaded; the groups behind the last row load that
// row without using it.
template <typename T, int L, int N, bool PAST>
__global__ __launch_bounds__(256) void norm_block_kernel(const T* x, const T* y, const float* __restrict__ a,
                                                         const float* __restrict__ w, T* h, T* n,
                                                         float* __restrict__ rstd, int rows, int width, float eps)
{
    constexpr int VE = Vec<T>::VE, R = 256 / L;
    __shared__ float red[2][4];
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const float inv = 1.0f / (float)width;
    int slot = 0;
    // the row index is the same for all lanes of a group and, at L = 256, for the workgroup
    for (int row0 = blockIdx.x * R; row0 < rows; row0 += gridDim.x * R, slot ^= 1) {
        const int row = row0 + sub;
        const bool live = row < rows;
        const size_t base = (size_t)(live ? row : rows - 1) * width;
        float v[N][VE];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * L + lane) * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = 0.f;
            if (c < width) {
                Vec<T>::load(x + base + c, v[i]);
                if (y) {
                    float u[VE], s[VE];
                    Vec<T>::load(y + base + c, u);
                    if (a) load_f32<VE>(a + c, s);
#pragma unroll
                    for (int e = 0; e < VE; ++e) v[i][e] += a ? s[e] * u[e] : u[e];
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) ss += v[i][e] * v[i][e];
            }
        }
        ss = group_sum<L>(ss, red, slot);
        const float r = 1.0f / sqrtf(ss * inv + eps);
        if (live) {
            if (rstd && lane == 0) rstd[row] = r;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (i * L + lane) * VE;
                if (c < width) {
                    float s[VE], out[VE];
                    load_f32<VE>(w + c, s);
#pragma unroll
                    for (int e = 0; e < VE; ++e) out[e] = v[i][e] * r * s[e];
                    if (h) Vec<T>::template store<PAST>(h + base + c, v[i]);
                    Vec<T>::template store<PAST>(n + base + c, out);
                }
            }
        }
    }
}

// The rows are dealt to a fixed number of workgroups; each lane sums its
// columns' dw and da over its rows in registers, the workgroup's row groups are
// added in LDS, and one row of partial sums a workgroup goes to `part`
// ([2][gridDim.x][width], dw then da), added up by norm_finish_kernel: the same
// order in every run.  A row's words are held as they were loaded and opened
// twice, for the row's sum and for its gradients: with four rows' worth of
// floats instead a lane took 192 registers and the card had too few loads in
// flight (32768 x 768 bf16, forward and backward: 131 us, against 113 us).  The
// bounds are as many waves as that leaves room for; <bf16, 16, 2> and <bf16, 16, 3>
// spill 8 registers each under them, which costs less than a wave (65536 rows of
// 256: 43 us, without 49; of 384: 60 and 71).  Eight words of bf16 a lane need more
// than the 256 registers of two waves (114 spilled): they have one (2048 rows of
// 16384: 142 us, with two waves 204).
template <typename T, int L, int N, bool PAST>
__global__ __launch_bounds__(256, N <= 2 ? 4 : N == 3 ? 3 : N == 8 && sizeof(T) == 2 ? 1 : 2) void norm_block_bwd_kernel(
    const T* __restrict__ dn, const T* __restrict__ dh, const T* __restrict__ x, const T* __restrict__ y,
    const float* __restrict__ a, const float* __restrict__ w, const float* __restrict__ rstd, T* dx, T* dy,
    float* __restrict__ part, int rows, int width)
{
    constexpr int VE = Vec<T>::VE, R = 256 / L;
    __shared__ float red[2][4];
    __shared__ __align__(16) float tot[R > 1 ? 256 * VE : 4];
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const float inv = 1.0f / (float)width;
    float dw[N][VE] = {}, da[N][VE] = {};
    int slot = 0;
    for (int row0 = blockIdx.x * R; row0 < rows; row0 += gridDim.x * R, slot ^= 1) {
        const int row = row0 + sub;
        const bool live = row < rows;
        const size_t base = (size_t)(live ? row : rows - 1) * width;
        const float r = rstd[live ? row : rows - 1];
        u32x4 xr[N], yr[N], nr[N], hr[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * L + lane) * VE;
            xr[i] = yr[i] = nr[i] = hr[i] = u32x4{0, 0, 0, 0};
            if (c < width) {
                xr[i] = *reinterpret_cast<const u32x4*>(x + base + c);
                nr[i] = *reinterpret_cast<const u32x4*>(dn + base + c);
                if (y) yr[i] = *reinterpret_cast<const u32x4*>(y + base + c);
                if (dh) hr[i] = *reinterpret_cast<const u32x4*>(dh + base + c);
            }
        }
        // word i's normalised values, the norm's g, and dn
        auto opened = [&](int i, int c, float (&xh)[VE], float (&g)[VE], float (&t)[VE]) {
            float s[VE];
            Vec<T>::open(xr[i], xh);
            Vec<T>::open(nr[i], t);
            if (y) {
                float u[VE];
                Vec<T>::open(yr[i], u);
                if (a) load_f32<VE>(a + c, s);
#pragma unroll
                for (int e = 0; e < VE; ++e) xh[e] += a ? s[e] * u[e] : u[e];
            }
            load_f32<VE>(w + c, s);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                xh[e] *= r;
                g[e] = t[e] * s[e];
            }
        };
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * L + lane) * VE;
            if (c < width) {
                float xh[VE], g[VE], t[VE];
                opened(i, c, xh, g, t);
#pragma unroll
                for (int e = 0; e < VE; ++e) dot += g[e] * xh[e];
            }
        }
        dot = group_sum<L>(dot, red, slot) * inv;
        if (live) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (i * L + lane) * VE;
                if (c < width) {
                    float xh[VE], g[VE], t[VE], o[VE];
                    opened(i, c, xh, g, t);
                    Vec<T>::open(hr[i], o);  // zeros without dh
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        dw[i][e] += t[e] * xh[e];
                        o[e] += r * (g[e] - xh[e] * dot);
                    }
                    if (a) {
                        float s[VE], q[VE], u[VE];
                        load_f32<VE>(a + c, s);
                        Vec<T>::open(yr[i], u);
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            da[i][e] += u[e] * o[e];
                            q[e] = s[e] * o[e];
                        }
                        Vec<T>::template store<PAST>(dy + base + c, q);
                    }
                    Vec<T>::template store<PAST>(dx + base + c, o);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && !a) break;
        float* out = part + ((size_t)k * gridDim.x + blockIdx.x) * width;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * L + lane) * VE;
            float s[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) s[e] = k ? da[i][e] : dw[i][e];
            if (R > 1) {  // add the row groups' sums, in order
                __syncthreads();
                store_f32<VE>(tot + threadIdx.x * VE, s);
                __syncthreads();
                if (sub == 0)
                    for (int q = 1; q < R; ++q) {
                        float t[VE];
                        load_f32<VE>(tot + (q * L + lane) * VE, t);
#pragma unroll
                        for (int e = 0; e < VE; ++e) s[e] += t[e];
                    }
            }
            if (sub == 0 && c < width) store_f32<VE>(out + c, s);
        }
    }
}

// out[c] = sum over the nb rows of part[.][c]: 16 columns a workgroup, 64 row
// strips (a strip's loads are what it waits for; with 16 the gated norm's training
// case took 1.6 % longer), then the strips in order
__global__ __launch_bounds__(1024) void norm_finish_kernel(const float* __restrict__ part, float* __restrict__ out0,
                                                           float* __restrict__ out1, int nb, int width)
{
    __shared__ float tot[64][17];
    const int i = threadIdx.x & 15, c = blockIdx.x * 16 + i, strip = threadIdx.x >> 4;
    const float* p = part + (size_t)blockIdx.y * nb * width;
    float s = 0.f;
    if (c < width) {
#pragma unroll 8
        for (int r = strip; r < nb; r += 64) s += p[(size_t)r * width + c];
    }
    tot[strip][i] = s;
    __syncthreads();
    if (strip < 4) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 16; ++q) s += tot[16 * strip + q][i];
    }
    __syncthreads();
    if (strip < 4) tot[strip][i] = s;
    __syncthreads();
    if (strip == 0 && c < width) (blockIdx.y ? out1 : out0)[c] = (tot[0][i] + tot[1][i]) + (tot[2][i] + tot[3][i]);
}

// ---------------------------------------------------------------------------
// gated norm of every head: a row of D values is held by L = D / VE lanes, one
// word each.  The gate's tokens are gate_stride elements apart.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + fast_exp(-z)); }

template <typename T, int L, bool PAST>
__global__ __launch_bounds__(256) void norm_gate_kernel(const T* __restrict__ o, const T* __restrict__ z,
                                                        const float* __restrict__ w, T* y, float* __restrict__ rstd,
                                                        int rows, int heads, long long gate_stride, float eps)
{
    constexpr int VE = Vec<T>::VE, R = 256 / L, D = L * VE;
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    float wv[VE];
    load_f32<VE>(w + lane * VE, wv);
    for (int row0 = blockIdx.x * R; row0 < rows; row0 += gridDim.x * R) {
        const int row = row0 + sub;
        const bool live = row < rows;
        const unsigned rr = live ? row : rows - 1;
        const unsigned tok = rr / (unsigned)heads;
        const size_t at = (size_t)rr * D + lane * VE;
        float v[VE], g[VE];
        Vec<T>::load(o + at, v);
        Vec<T>::load(z + (size_t)tok * gate_stride + (size_t)(rr - tok * heads) * D + lane * VE, g);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) ss += v[e] * v[e];
        ss = group_sum<L>(ss, nullptr, 0);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] = v[e] * r * wv[e] * (g[e] * sigmoid(g[e]));
        if (live) {
            if (rstd && lane == 0) rstd[row] = r;
            Vec<T>::template store<PAST>(y + at, v);
        }
    }
}

template <typename T, int L, bool PAST>
__global__ __launch_bounds__(256) void norm_gate_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ o,
                                                            const T* __restrict__ z, const float* __restrict__ w,
                                                            const float* __restrict__ rstd, T* dO, T* dz,
                                                            float* __restrict__ part, int rows, int heads,
                                                            long long gate_stride)
{
    constexpr int VE = Vec<T>::VE, R = 256 / L, D = L * VE;
    __shared__ __align__(16) float tot[256 * VE];
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    float wv[VE], dw[VE] = {};
    load_f32<VE>(w + lane * VE, wv);
    for (int row0 = blockIdx.x * R; row0 < rows; row0 += gridDim.x * R) {
        const int row = row0 + sub;
        const bool live = row < rows;
        const unsigned rr = live ? row : rows - 1;
        const unsigned tok = rr / (unsigned)heads;
        const size_t at = (size_t)rr * D + lane * VE;
        float v[VE], g[VE], d[VE], p[VE];
        Vec<T>::load(o + at, v);
        Vec<T>::load(z + (size_t)tok * gate_stride + (size_t)(rr - tok * heads) * D + lane * VE, g);
        Vec<T>::load(dy + at, d);
        const float r = rstd[rr];
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            v[e] *= r;
            const float s = sigmoid(g[e]), act = g[e] * s;
            const float t = d[e] * v[e];               // dy oh
            if (live) dw[e] += t * act;
            p[e] = d[e] * act * wv[e];                 // g of the norm
            dot += p[e] * v[e];
            g[e] = t * wv[e] * (s + act * (1.0f - s)); // dz
        }
        dot = group_sum<L>(dot, nullptr, 0) * (1.0f / D);
#pragma unroll
        for (int e = 0; e < VE; ++e) p[e] = r * (p[e] - v[e] * dot);
        if (live) {
            Vec<T>::template store<PAST>(dO + at, p);
            Vec<T>::template store<PAST>(dz + at, g);
        }
    }
    store_f32<VE>(tot + threadIdx.x * VE, dw);
    __syncthreads();
    // thread c < D adds its column over the row groups, in order
    for (int c = threadIdx.x; c < D; c += 256) {
        float s = 0.f;
        for (int q = 0; q < R; ++q) s += tot[q * D + c];
        part[(size_t)blockIdx.x * D + c] = s;
    }
}

// whether an output of this shape is larger than the card's L2 (4 MB on each of 8 dies)
template <typename T> bool past_l2(const gdn_norm_shape& s)
{
    return (long long)s.tokens * s.heads * s.width * (long long)sizeof(T) > (32LL << 20);
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Lanes and words a row of norm_block: the pair that wastes the fewest words;
// among equals the widest group when the rows are few (a whole workgroup a row
// ends sooner) and the narrowest when they are many (no barrier).
struct Split {
    int L, N;
};
Split pick_split(int words, int rows)
{
    static const Split all[] = {{16, 1}, {16, 2}, {16, 3}, {16, 4}, {32, 1}, {32, 2}, {32, 3}, {32, 4}, {64, 1}, {64, 2}, {64, 3}, {64, 4},
                                {256, 1}, {256, 2}, {256, 3}, {256, 4}, {256, 8}};
    const bool few = rows <= 2048;
    Split best{0, 0};
    for (const Split& s : all) {
        if (s.L * s.N < words) continue;
        const int have = best.L * best.N, now = s.L * s.N;
        if (!best.L || now < have || (now == have && (few ? s.L > best.L : s.L < best.L))) best = s;
    }
    return best;
}

// Call f(L, N, PAST) as compile-time constants.
template <typename F> gdn_status with_split(Split s, bool past, F&& f)
{
#define GDN_SPLIT(l, n) \
    if (s.L == l && s.N == n)       \
        return with_bool(past, [&](auto p) { return f(std::integral_constant<int, l>{}, std::integral_constant<int, n>{}, p); })
    GDN_SPLIT(16, 1); GDN_SPLIT(16, 2); GDN_SPLIT(16, 3); GDN_SPLIT(16, 4);
    GDN_SPLIT(32, 1); GDN_SPLIT(32, 2); GDN_SPLIT(32, 3); GDN_SPLIT(32, 4);
    GDN_SPLIT(64, 1); GDN_SPLIT(64, 2); GDN_SPLIT(64, 3); GDN_SPLIT(64, 4);
    GDN_SPLIT(256, 1); GDN_SPLIT(256, 2); GDN_SPLIT(256, 3); GDN_SPLIT(256, 4); GDN_SPLIT(256, 8);
#undef GDN_SPLIT
    return GDN_ERR_UNSUPPORTED;
}

template <typename F> gdn_status with_lanes(int L, bool past, F&& f)
{
    switch (L) {
    case 2: return with_bool(past, [&](auto p) { return f(std::integral_constant<int, 2>{}, p); });
    case 4: return with_bool(past, [&](auto p) { return f(std::integral_constant<int, 4>{}, p); });
    case 8: return with_bool(past, [&](auto p) { return f(std::integral_constant<int, 8>{}, p); });
    case 16: return with_bool(past, [&](auto p) { return f(std::integral_constant<int, 16>{}, p); });
    case 32: return with_bool(past, [&](auto p) { return f(std::integral_constant<int, 32>{}, p); });
    }
    return GDN_ERR_UNSUPPORTED;
}

template <typename T>
gdn_status block_fwd(const gdn_norm_shape& s, const void* x, const void* y, const float* a, const float* w, void* h,
                     void* n, float* rstd, hipStream_t st)
{
    const Split sp = pick_split(s.width / Vec<T>::VE, s.tokens);
    return with_split(sp, past_l2<T>(s), [&](auto L, auto N, auto PAST) -> gdn_status {
        const int blocks = ceil_div(s.tokens, 256 / L());
        GDN_LAUNCH("norm_block", (norm_block_kernel<T, L(), N(), PAST()>), dim3(blocks < 4096 ? blocks : 4096), dim3(256), st,
                   (const T*)x, (const T*)y, a, w, (T*)h, (T*)n, rstd, s.tokens, s.width, s.eps);
        return GDN_OK;
    });
}

template <typename T>
gdn_status block_bwd(const gdn_norm_shape& s, const void* dn, const void* dh, const void* x, const void* y,
                     const float* a, const float* w, const float* rstd, void* dx, void* dy, float* dw, float* da,
                     float* part, hipStream_t st)
{
    const Split sp = pick_split(s.width / Vec<T>::VE, s.tokens);
    const int nb = norm_partials(s, false);
    gdn_status r = with_split(sp, past_l2<T>(s), [&](auto L, auto N, auto PAST) -> gdn_status {
        if (!nb) return GDN_OK;  // no rows: the sums are zeros
        GDN_LAUNCH("norm_block_bwd", (norm_block_bwd_kernel<T, L(), N(), PAST()>), dim3(nb), dim3(256), st, (const T*)dn,
                   (const T*)dh, (const T*)x, (const T*)y, a, w, rstd, (T*)dx, (T*)dy, part, s.tokens, s.width);
        return GDN_OK;
    });
    if (r != GDN_OK) return r;
    GDN_LAUNCH("norm_finish", norm_finish_kernel, dim3(ceil_div(s.width, 16), a ? 2 : 1), dim3(1024), st, part, dw, da,
               nb, s.width);
    return GDN_OK;
}

template <typename T>
gdn_status gate_fwd(const gdn_norm_shape& s, const void* o, const void* z, const float* w, void* y, float* rstd,
                    hipStream_t st)
{
    const int rows = s.tokens * s.heads;
    return with_lanes(s.width / Vec<T>::VE, past_l2<T>(s), [&](auto L, auto PAST) -> gdn_status {
        const int blocks = ceil_div(rows, 256 / L());
        GDN_LAUNCH("norm_gate", (norm_gate_kernel<T, L(), PAST()>), dim3(blocks < 8192 ? blocks : 8192), dim3(256), st,
                   (const T*)o, (const T*)z, w, (T*)y, rstd, rows, s.heads, s.gate_stride, s.eps);
        return GDN_OK;
    });
}

template <typename T>
gdn_status gate_bwd(const gdn_norm_shape& s, const void* dy, const void* o, const void* z, const float* w,
                    const float* rstd, void* dO, void* dz, float* dw, float* part, hipStream_t st)
{
    const int rows = s.tokens * s.heads;
    const int nb = norm_partials(s, true);
    gdn_status r = with_lanes(s.width / Vec<T>::VE, past_l2<T>(s), [&](auto L, auto PAST) -> gdn_status {
        if (!nb) return GDN_OK;  // no rows: the sums are zeros
        GDN_LAUNCH("norm_gate_bwd", (norm_gate_bwd_kernel<T, L(), PAST()>), dim3(nb), dim3(256), st, (const T*)dy,
                   (const T*)o, (const T*)z, w, rstd, (T*)dO, (T*)dz, part, rows, s.heads, s.gate_stride);
        return GDN_OK;
    });
    if (r != GDN_OK) return r;
    GDN_LAUNCH("norm_finish", norm_finish_kernel, dim3(ceil_div(s.width, 16), 1), dim3(1024), st, part, dw,
               (float*)nullptr, nb, s.width);
    return GDN_OK;
}

}  // namespace

// Workgroups of the backward, each leaving one row of partial sums: as many as
// are on the card at once (its 256 compute units times what the registers
// allow).
int norm_partials(const gdn_norm_shape& s, bool gate)
{
    const int ve = s.dtype == GDN_BF16 ? 8 : 4;
    const Split sp = gate ? Split{s.width / ve, 1} : pick_split(s.width / ve, s.tokens);
    const int blocks = ceil_div((long long)s.tokens * s.heads, 256 / sp.L);
    const int most = sp.N <= 2 ? 1024 : sp.N == 3 ? 768 : sp.N == 8 && ve == 8 ? 256 : 512;
    return blocks < most ? blocks : most;
}

gdn_status norm_block_dispatch(const gdn_norm_shape& s, const void* x, const void* y, const float* a, const float* w,
                               void* h, void* n, float* rstd, hipStream_t st)
{
    return s.dtype == GDN_BF16 ? block_fwd<bf16>(s, x, y, a, w, h, n, rstd, st)
                               : block_fwd<float>(s, x, y, a, w, h, n, rstd, st);
}

gdn_status norm_block_bwd_dispatch(const gdn_norm_shape& s, const void* dn, const void* dh, const void* x,
                                   const void* y, const float* a, const float* w, const float* rstd, void* dx,
                                   void* dy, float* dw, float* da, float* part, hipStream_t st)
{
    return s.dtype == GDN_BF16 ? block_bwd<bf16>(s, dn, dh, x, y, a, w, rstd, dx, dy, dw, da, part, st)
                               : block_bwd<float>(s, dn, dh, x, y, a, w, rstd, dx, dy, dw, da, part, st);
}

gdn_status norm_gate_dispatch(const gdn_norm_shape& s, const void* o, const void* z, const float* w, void* y,
                              float* rstd, hipStream_t st)
{
    return s.dtype == GDN_BF16 ? gate_fwd<bf16>(s, o, z, w, y, rstd, st) : gate_fwd<float>(s, o, z, w, y, rstd, st);
}

gdn_status norm_gate_bwd_dispatch(const gdn_norm_shape& s, const void* dy, const void* o, const void* z,
                                  const float* w, const float* rstd, void* dO, void* dz, float* dw, float* part,
                                  hipStream_t st)
{
    return s.dtype == GDN_BF16 ? gate_bwd<bf16>(s, dy, o, z, w, rstd, dO, dz, dw, part, st)
                               : gate_bwd<float>(s, dy, o, z, w, rstd, dO, dz, dw, part, st);
}

}  // namespace gdn
