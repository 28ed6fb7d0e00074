// conv.hip -- the short causal convolution along the tokens that stands before a
// recurrent layer (gdn_conv_forward, gdn_conv_backward, gdn_conv_step): every
// channel by itself, W = 2..4 taps, over packed sequences.  With e the sequence's
// rows behind its state (the W - 1 rows before it, or zeros),
//
//   z_t = bias + sum_j w_j e_{t+j},   y = z / (1 + exp(-z)) or z,   state' = the last W - 1 rows of e
//   dz = dy s(z) (1 + z (1 - s(z))),  s(z) = 1 / (1 + exp(-z))
//   de_i = sum_j w_j dz_{i-j} (+ the gradient of state'),  dw_j = sum_t dz_t e_{t+j},  dbias = sum_t dz_t
//
// fp32, rounded once when stored.  Bound by HBM: a thread holds one 16-byte word of
// channels and walks down a strip of tokens with its window in registers, so that
// every row is read once (but for the W - 1 rows between strips).
//
// A workgroup is CW words of channels by 256 / CW strips.  Of 64 words a wave is one
// strip: its rows come as whole kilobytes, and where a sequence ends is a question for
// scalar registers; of 16 words where 64 would leave more than a fifth of the lanes
// without a channel.  32768 rows of 1024 bf16: forward 26 to 27 us, 5.0 TB/s;
// backward 46 us, 4.4 TB/s (traced; among others 34, with 16 words 41, and 50, without the
// rows to come on their way 58).
#include "conv.h"
#include "bounds.h"
#include "common.h"

namespace gdn {

namespace {

// a thread's word of channels in its workgroup, and its strip (or sequence)
template <int CW> __device__ __forceinline__ int lane_word() { return threadIdx.x & (CW - 1); }
template <int CW> __device__ __forceinline__ int lane_strip()
{
    return CW == 64 ? __builtin_amdgcn_readfirstlane(wave_id()) : (int)threadIdx.x / CW;
}

// one 16-byte word of channels
template <typename T> struct Word;
template <> struct Word<bf16> {
    static constexpr int VE = 8;
    static __device__ __forceinline__ void open(u32x4 w, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4 close(const float (&v)[8])
    {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = cvt2_bf16(v[2 * i], v[2 * i + 1]);
        return w;
    }
};
template <> struct Word<float> {
    static constexpr int VE = 4;
    static __device__ __forceinline__ void open(u32x4 w, float (&v)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ u32x4 close(const float (&v)[4])
    {
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
};

template <typename T> __device__ __forceinline__ u32x4 load_word(const T* p) { return *reinterpret_cast<const u32x4*>(p); }
// PAST: not to be kept in the L2
template <bool PAST, typename T> __device__ __forceinline__ void store_word(T* p, u32x4 w)
{
    if constexpr (PAST)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<u32x4*>(p) = w;
}

// a thread's channels: its word of every row, their taps and bias
template <typename T, int W> struct Taps {
    static constexpr int VE = Word<T>::VE;
    float w[W][VE], bias[VE];
    __device__ __forceinline__ void load(const ConvArgs& a, int c)
    {
        const f32x4* p = reinterpret_cast<const f32x4*>(a.w + (size_t)c * W);
        float flat[W * VE];
#pragma unroll
        for (int i = 0; i < W * VE / 4; ++i) {
            const f32x4 q = p[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) flat[4 * i + k] = q[k];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            bias[e] = a.bias ? a.bias[c + e] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
        }
    }
    // z of the window of which `last` is the newest row
    __device__ __forceinline__ void sum(const float (&win)[W - 1][VE], const float (&last)[VE], float (&z)[VE]) const
    {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            z[e] = bias[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z[e] = __builtin_fmaf(w[j][e], win[j][e], z[e]);
            z[e] = __builtin_fmaf(w[W - 1][e], last[e], z[e]);
        }
    }
};

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-z)); }

template <int VE> __device__ __forceinline__ void activate(float (&z)[VE], bool silu)
{
    if (silu) {
#pragma unroll
        for (int e = 0; e < VE; ++e) z[e] *= sigmoid(z[e]);
    }
}
// dz from dy and z
template <int VE> __device__ __forceinline__ void through(float (&dy)[VE], const float (&z)[VE], bool silu)
{
    if (silu) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float s = sigmoid(z[e]);
            dy[e] *= s * __builtin_fmaf(z[e], 1.f - s, 1.f);
        }
    }
}

template <int K, int VE> __device__ __forceinline__ void shift(float (&win)[K][VE], const float (&x)[VE])
{
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) win[j][e] = j < K - 1 ? win[j + 1 < K ? j + 1 : j][e] : x[e];
}
template <int VE> __device__ __forceinline__ void clear(float (&v)[VE])
{
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = 0.f;
}

__device__ __forceinline__ int clamped(const ConvArgs& a, int i)
{
    const int v = a.cu[i];
    return v < 0 ? 0 : v > a.T ? a.T : v;
}

__device__ __forceinline__ int wave_most(int x)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const int other = __shfl_xor(x, o);
        x = other > x ? other : x;
    }
    return __builtin_amdgcn_readfirstlane(x);
}

// The greatest of x and of 256 WORDS bounds from i on, a lane's share of them
template <int WORDS> __device__ __forceinline__ int most_of(const int* __restrict__ cu, int i, int x)
{
    typedef int i32x4 __attribute__((ext_vector_type(4), aligned(4)));
    i32x4 v[WORDS];
#pragma unroll
    for (int k = 0; k < WORDS; ++k) v[k] = *reinterpret_cast<const i32x4*>(cu + i + 256 * k + 4 * lane_id());
#pragma unroll
    for (int k = 0; k < WORDS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x = v[k][j] > x ? v[k][j] : x;
    return x;
}

// Rows st .. en - 1 of sequence b, as ordered_bounds has them: it begins at the greatest
// of the bounds up to its own.  Called by whole workgroups, whose sequences follow one
// another from `base` on; they read whole 8192s of the bounds before it together.
__device__ __forceinline__ void rows_of(const ConvArgs& a, int base, int b, int& st, int& en)
{
    if (!a.cu) {  // single tokens: row b is all of sequence b
        st = b, en = b + 1;
        return;
    }
    __shared__ int red[4];
    const int first = __builtin_amdgcn_readfirstlane(b);
    int i0 = 0;
    st = en = 0;
    if (base >= 8192) {
        const int w = __builtin_amdgcn_readfirstlane(wave_id());
        for (; i0 + 8192 <= base + 1; i0 += 8192) st = most_of<8>(a.cu, i0 + 2048 * w, st);
        red[w] = wave_most(st);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) st = red[k] > st ? red[k] : st;
    }
    if (first >= a.B) return;
    for (; i0 + 2048 <= first + 1; i0 += 2048) st = most_of<8>(a.cu, i0, st);
    for (; i0 + 256 <= first + 1; i0 += 256) st = most_of<1>(a.cu, i0, st);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = i0 + 64 * k + lane_id(), v = a.cu[i <= first ? i : first];
        st = v > st ? v : st;
    }
    st = wave_most(st);
    st = st > a.T ? a.T : st;
    if (b >= a.B) return;
    for (int i = first + 1; i <= b; ++i) {
        const int v = clamped(a, i);
        st = v > st ? v : st;
    }
    en = clamped(a, b + 1);
    en = en < st ? st : en;
}

// the sequence of a row, moved forward as the rows go on; end past every row where there is none
struct Seq {
    int b, st, en;
    // Called by whole waves, with one row t a CW lanes, ascending: 64 sequences at a time
    // along the ordered bounds, behind whole 2048s and 256s of them that end at or before
    // the first row.  (A bisection would find some rise past t, not the first.)
    template <int CW> __device__ __forceinline__ void find(const ConvArgs& a, int t)
    {
        constexpr int GROUPS = 64 / CW;
        const int l = lane_id(), t0 = __builtin_amdgcn_readfirstlane(t);
        b = a.B, st = en = 0x7fffffff;
        if (t0 >= a.T) return;
        int b0 = 0, top = 0, most = a.cu[0];
        auto skip = [&](auto words) {
            constexpr int WORDS = decltype(words)::value;
            for (; b0 + 256 * WORDS <= a.B; b0 += 256 * WORDS) {
                const int m = most_of<WORDS>(a.cu, b0 + 1, most);
                if (__any(m > t0)) break;
                most = m;
            }
        };
        if (most <= t0) {
            skip(std::integral_constant<int, 8>{});
            skip(std::integral_constant<int, 1>{});
            if (b0) top = wave_most(most < 0 ? 0 : most);
        }
        unsigned open = 0;  // groups of lanes whose row is yet to be found
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) open |= __builtin_amdgcn_readlane(t, g * CW) < a.T ? 1u << g : 0u;
        for (; b0 < a.B && open; b0 += 64) {
            int s, e;
            ordered_bounds(a.cu, a.B, a.T, b0, top, s, e);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const uint64_t hit = __ballot(e > __builtin_amdgcn_readlane(t, g * CW));
                if (hit && (open >> g & 1)) {
                    const int k = __builtin_ctzll(hit), sk = __builtin_amdgcn_readlane(s, k), ek = __builtin_amdgcn_readlane(e, k);
                    if (GROUPS == 1 || l / CW == g) b = b0 + k, st = sk, en = ek;
                    open &= ~(1u << g);
                }
            }
        }
    }
    __device__ __forceinline__ void move(const ConvArgs& a, int t)
    {
        while (t >= en && b < a.B) {
            if (++b < a.B) {
                st = en;
                const int e = clamped(a, b + 1);
                en = e < st ? st : e;
            } else {
                st = en = 0x7fffffff;
            }
        }
    }
};

// A sequence's first W - 1 rows (those whose window holds its state) and its new
// state, by the threads that have read the old one: state and state_out may be one.
template <typename T, int W>
__device__ __forceinline__ void head_rows(const ConvArgs& a, int b, int st, int n, int c)
{
    constexpr int VE = Word<T>::VE, K = W - 1;
    Taps<T, W> taps;
    taps.load(a, c);
    const T* x = (const T*)a.x + (size_t)st * a.x_stride + c;
    u32x4 old[K], rows[K], tail[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        old[j] = rows[j] = tail[j] = u32x4{0, 0, 0, 0};
        if (a.state) old[j] = load_word((const T*)a.state + ((size_t)b * K + j) * a.C + c);
        if (j < n) rows[j] = load_word(x + (size_t)j * a.x_stride);
        if (a.state_out && n + j >= K) tail[j] = load_word(x + (size_t)(n + j - K) * a.x_stride);
    }
    if (a.state_out) {
#pragma unroll
        for (int j = 0; j < K; ++j) {  // row n + j of the state and the sequence after it
            u32x4 w = tail[j];
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (n + j == i) w = old[i];
            *reinterpret_cast<u32x4*>((T*)a.state_out + ((size_t)b * K + j) * a.C + c) = w;
        }
    }
    float win[K][VE];
#pragma unroll
    for (int j = 0; j < K; ++j) Word<T>::open(old[j], win[j]);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (j < n) {
            float v[VE], z[VE];
            Word<T>::open(rows[j], v);
            taps.sum(win, v, z);
            activate(z, a.silu);
            store_word<false>((T*)a.y + (size_t)(st + j) * a.C + c, Word<T>::close(z));
            shift<K, VE>(win, v);
        }
    }
}

// blockIdx.y: channels.  The first a.head_blocks of blockIdx.x are sequences, the others strips.
template <typename T, int W, int CW, bool PAST>
__global__ __launch_bounds__(256) void conv_forward_kernel(ConvArgs a)
{
    constexpr int VE = Word<T>::VE, K = W - 1, AHEAD = 8;
    constexpr int NS = 256 / CW;
    const int c = (blockIdx.y * CW + lane_word<CW>()) * VE, sub = lane_strip<CW>();
    if ((int)blockIdx.x < a.head_blocks) {
        const int b = blockIdx.x * NS + sub;
        int st, en;
        rows_of(a, blockIdx.x * NS, b, st, en);
        if (b < a.B && c < a.C) head_rows<T, W>(a, b, st, en - st, c);
        return;
    }
    const long long first = ((long long)(blockIdx.x - a.head_blocks) * NS + sub) * a.strip;
    const int t0 = first < a.T ? (int)first : a.T, t1 = a.T - t0 < a.strip ? a.T : t0 + a.strip;
    Seq s;
    s.find<CW>(a, t0);
    if (s.b >= a.B || c >= a.C) return;  // behind the last sequence
    Taps<T, W> taps;
    taps.load(a, c);
    const T* x = (const T*)a.x + c;
    float win[K][VE];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int t = t0 - K + j;
        clear(win[j]);
        if (t >= 0) Word<T>::open(load_word(x + (size_t)t * a.x_stride), win[j]);
    }
    u32x4 next[AHEAD];  // the rows to come are on their way while these are worked on
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) next[i] = load_word(x + (size_t)(t + i < t1 ? t + i : t1 - 1) * a.x_stride);
    };
    fetch(t0);
    for (int t = t0; t < t1; t += AHEAD) {
        u32x4 r[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) r[i] = next[i];
        if (t + AHEAD < t1) fetch(t + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (t + i < t1) {
                s.move(a, t + i);
                float v[VE];
                Word<T>::open(r[i], v);
                // the first W - 1 rows of a sequence are head_rows'
                if (t + i - K >= s.st && t + i < s.en) {
                    float z[VE];
                    taps.sum(win, v, z);
                    activate(z, a.silu);
                    store_word<PAST>((T*)a.y + (size_t)(t + i) * a.C + c, Word<T>::close(z));
                }
                shift<K, VE>(win, v);
            }
        }
    }
}

// Gradients.  A thread walks its strip and the W - 1 rows behind it, forms dz of
// every row and with it dx of the row W - 1 before.  Its sums for the taps and the
// bias go to `part` [strip blocks][W + 1][C], a block's strips added in LDS, and
// are added up by conv_finish_kernel: the same order in every run.
template <typename T, int W, int CW, bool PAST>
__global__ __launch_bounds__(256) void conv_backward_kernel(ConvArgs a)
{
    constexpr int VE = Word<T>::VE, K = W - 1, AHEAD = 4, NS = 256 / CW;
    __shared__ float tot[NS][CW * VE + 1];
    const int cw = lane_word<CW>(), c = (blockIdx.y * CW + cw) * VE, sub = lane_strip<CW>();
    const long long first = ((long long)blockIdx.x * NS + sub) * a.strip;
    const int t0 = first < a.T ? (int)first : a.T;
    Seq s;
    s.find<CW>(a, t0);
    float dw[W][VE], db[VE];
    clear(db);
#pragma unroll
    for (int j = 0; j < W; ++j) clear(dw[j]);
    if (c < a.C && t0 < a.T) {
        const int t1 = a.T - t0 < a.strip ? a.T : t0 + a.strip;
        const int last = a.T - t1 < K ? a.T : t1 + K;  // rows whose dz this strip needs
        Taps<T, W> taps;
        taps.load(a, c);
        const T *x = (const T*)a.x + c, *dy = (const T*)a.dy + c;
        // win: the K rows before t as the window of row t has them; dzs, ends, seqs: dz, the sequence's end and its number of the K rows before
        float win[K][VE], dzs[K][VE];
        int ends[K], seqs[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int t = t0 - K + j;
            clear(win[j]);
            clear(dzs[j]);
            ends[j] = seqs[j] = -1;
            if (t >= s.st) {
                Word<T>::open(load_word(x + (size_t)t * a.x_stride), win[j]);
            } else if (a.state && s.b < a.B && t0 >= s.st) {  // row t - st + K of the state
                Word<T>::open(load_word((const T*)a.state + ((size_t)s.b * K + (t - s.st + K)) * a.C + c), win[j]);
            }
        }
        // up to row last - 1, then K - (last - t1) rows that do not exist: the end of the buffer
        u32x4 next_x[AHEAD], next_y[AHEAD];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int row = t + i < last ? t + i : last - 1;
                next_x[i] = load_word(x + (size_t)row * a.x_stride);
                next_y[i] = load_word(dy + (size_t)row * a.C);
            }
        };
        fetch(t0);
        for (int t = t0; t < t1 + K; t += AHEAD) {
            u32x4 rx[AHEAD], ry[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) rx[i] = next_x[i], ry[i] = next_y[i];
            if (t + AHEAD < last) fetch(t + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int row = t + i;
                if (row < t1 + K) {
                    float dz[VE], v[VE];
                    clear(dz);
                    clear(v);
                    int end = -1, seq = -1;
                    if (row < last) {
                        s.move(a, row);
                        Word<T>::open(rx[i], v);
                        if (row >= s.st && row < s.en) {
                            end = s.en, seq = s.b;
                            if (row == s.st && row != t0) {  // a sequence begins here: its window holds its state
#pragma unroll
                                for (int j = 0; j < K; ++j) {
                                    clear(win[j]);
                                    if (a.state) Word<T>::open(load_word((const T*)a.state + ((size_t)s.b * K + j) * a.C + c), win[j]);
                                }
                            }
                            float z[VE];
                            taps.sum(win, v, z);
                            Word<T>::open(ry[i], dz);
                            through(dz, z, a.silu);
                            if (row < t1) {
#pragma unroll
                                for (int e = 0; e < VE; ++e) {
                                    db[e] += dz[e];
#pragma unroll
                                    for (int j = 0; j < W; ++j)
                                        dw[j][e] = __builtin_fmaf(dz[e], j < K ? win[j < K ? j : 0][e] : v[e], dw[j][e]);
                                }
                            }
                        }
                    }
                    const int to = row - K;  // dx of row `to`: the dz up to its sequence's end
                    if (to >= t0 && ends[0] > to) {
                        float g[VE];
                        clear(g);
                        if (a.dstate_out && to >= ends[0] - K) {
                            const int j = to - (ends[0] - K);
                            Word<T>::open(load_word((const T*)a.dstate_out + ((size_t)seqs[0] * K + j) * a.C + c), g);
                        }
#pragma unroll
                        for (int k = 0; k < W; ++k) {  // dz of row to + k with tap K - k
                            if (to + k < ends[0]) {
#pragma unroll
                                for (int e = 0; e < VE; ++e)
                                    g[e] = __builtin_fmaf(taps.w[K - k][e], k < K ? dzs[k < K ? k : 0][e] : dz[e], g[e]);
                            }
                        }
                        store_word<PAST>((T*)a.dx + (size_t)to * a.C + c, Word<T>::close(g));
                    }
                    shift<K, VE>(win, v);
                    shift<K, VE>(dzs, dz);
#pragma unroll
                    for (int j = 0; j < K; ++j) {
                        ends[j] = j < K - 1 ? ends[j + 1 < K ? j + 1 : j] : end;
                        seqs[j] = j < K - 1 ? seqs[j + 1 < K ? j + 1 : j] : seq;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q <= W; ++q) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VE; ++e) tot[sub][cw * VE + e] = q < W ? dw[q < W ? q : 0][e] : db[e];
        __syncthreads();
        for (int i = threadIdx.x; i < CW * VE; i += 256) {
            const int ch = blockIdx.y * CW * VE + i;
            if (ch >= a.C) break;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < NS; ++k) sum += tot[k][i];
            a.part[((size_t)blockIdx.x * (W + 1) + q) * a.C + ch] = sum;
        }
    }
}

// dweight [C][W] and dbias [C] from the strip blocks' sums: 16 columns of
// [W + 1][C] a workgroup, 16 strips of blocks, then the strips in order
template <int W>
__global__ __launch_bounds__(256) void conv_finish_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                          float* __restrict__ db, int blocks, int C)
{
    __shared__ float tot[16][17];
    const int i = threadIdx.x & 15, strip = threadIdx.x >> 4;
    const long long col = (long long)blockIdx.x * 16 + i, width = (long long)(W + 1) * C;
    float s = 0.f;
    if (col < width) {
#pragma unroll 8
        for (int r = strip; r < blocks; r += 16) s += part[(size_t)r * width + col];
    }
    tot[strip][i] = s;
    __syncthreads();
    if (strip == 0 && col < width) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += tot[k][i];
        const int q = (int)(col / C), c = (int)(col - (long long)q * C);
        if (q < W)
            dw[(size_t)c * W + q] = s;
        else if (db)
            db[c] = s;
    }
}

// the gradient of the sequences' states: rows 0 .. W - 2 of de
template <typename T, int W>
__global__ __launch_bounds__(256) void conv_dstate_kernel(ConvArgs a)
{
    constexpr int VE = Word<T>::VE, K = W - 1;
    const int c = (blockIdx.y * 16 + (threadIdx.x & 15)) * VE, b = blockIdx.x * 16 + (threadIdx.x >> 4);
    int st, en;
    rows_of(a, blockIdx.x * 16, b, st, en);
    if (c >= a.C || b >= a.B) return;
    Taps<T, W> taps;
    taps.load(a, c);
    const int n = en - st;
    float win[K][VE], dzs[K][VE], z[VE], v[VE];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        clear(win[j]);
        clear(dzs[j]);
        if (a.state) Word<T>::open(load_word((const T*)a.state + ((size_t)b * K + j) * a.C + c), win[j]);
    }
#pragma unroll
    for (int t = 0; t < K; ++t) {
        if (t < n) {
            Word<T>::open(load_word((const T*)a.x + (size_t)(st + t) * a.x_stride + c), v);
            taps.sum(win, v, z);
            Word<T>::open(load_word((const T*)a.dy + (size_t)(st + t) * a.C + c), dzs[t]);
            through(dzs[t], z, a.silu);
            shift<K, VE>(win, v);
        }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
        float g[VE];
        clear(g);
        if (a.dstate_out && i >= n) Word<T>::open(load_word((const T*)a.dstate_out + ((size_t)b * K + (i - n)) * a.C + c), g);
#pragma unroll
        for (int t = 0; t <= i; ++t)
#pragma unroll
            for (int e = 0; e < VE; ++e) g[e] = __builtin_fmaf(taps.w[i - t][e], dzs[t][e], g[e]);
        store_word<false>((T*)a.dstate + ((size_t)b * K + i) * a.C + c, Word<T>::close(g));
    }
}

// words of channels a workgroup has
int channel_words(const gdn_conv_shape& s)
{
    const int words = s.C / (s.dtype == GDN_BF16 ? 8 : 4), idle = (words + 63) / 64 * 64 - words;
    return idle * 5 <= words ? 64 : 16;
}
int channel_blocks(const gdn_conv_shape& s, int cw)
{
    const int words = s.C / (s.dtype == GDN_BF16 ? 8 : 4);
    return (words + cw - 1) / cw;
}

// Tokens a thread walks: 32 where that leaves 512 threads a compute unit, fewer
// (down to 8, the rows it has in flight) for shorter calls
int conv_strip(const gdn_conv_shape& s)
{
    const long long words = s.C / (s.dtype == GDN_BF16 ? 8 : 4);
    for (int r = 32; r > 8; r /= 2)
        if ((long long)s.T * words / r >= 256 * 512) return r;
    return 8;
}

template <typename F> gdn_status with_taps(int W, F&& f)
{
    switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    default: return f(std::integral_constant<int, 4>{});
    }
}

// outputs larger than the L2 (4 MB on each of 8 dies) are not kept there
bool past_l2(const gdn_conv_shape& s) { return (long long)s.T * s.C * (s.dtype == GDN_BF16 ? 2 : 4) > (32LL << 20); }

template <typename F> gdn_status with_words(const gdn_conv_shape& s, F&& f)
{
    return channel_words(s) == 64 ? f(std::integral_constant<int, 64>{}) : f(std::integral_constant<int, 16>{});
}

template <typename T> gdn_status forward(const gdn_conv_shape& s, ConvArgs a, hipStream_t st)
{
    a.strip = conv_strip(s);
    const int strips = a.cu ? (s.T + a.strip - 1) / a.strip : 0;
    return with_taps(s.W, [&](auto w) -> gdn_status {
        constexpr int W = decltype(w)::value;
        return with_words(s, [&](auto cw) -> gdn_status {
            constexpr int CW = decltype(cw)::value, NS = 256 / CW;
            a.head_blocks = (s.B + NS - 1) / NS;
            const dim3 grid(a.head_blocks + (strips + NS - 1) / NS, channel_blocks(s, CW));
            return with_bool(past_l2(s), [&](auto past) -> gdn_status {
                GDN_LAUNCH("conv_forward", (conv_forward_kernel<T, W, CW, decltype(past)::value>), grid, dim3(256), st, a);
                return GDN_OK;
            });
        });
    });
}

template <typename T> gdn_status backward(const gdn_conv_shape& s, ConvArgs a, float* dw, float* db, hipStream_t st)
{
    a.strip = conv_strip(s);
    const int blocks = conv_partials(s), cols = (s.W + 1) * ((s.C + 15) / 16);
    return with_taps(s.W, [&](auto w) -> gdn_status {
        constexpr int W = decltype(w)::value;
        if (blocks) {
            const gdn_status r = with_words(s, [&](auto cw) -> gdn_status {
                constexpr int CW = decltype(cw)::value;
                return with_bool(past_l2(s), [&](auto past) -> gdn_status {
                    GDN_LAUNCH("conv_backward", (conv_backward_kernel<T, W, CW, decltype(past)::value>),
                               dim3(blocks, channel_blocks(s, CW)), dim3(256), st, a);
                    return GDN_OK;
                });
            });
            if (r != GDN_OK) return r;
        }
        GDN_LAUNCH("conv_finish", (conv_finish_kernel<W>), dim3(cols), dim3(256), st, a.part, dw, db, blocks, s.C);
        if (a.dstate)
            GDN_LAUNCH("conv_dstate", (conv_dstate_kernel<T, W>), dim3((s.B + 15) / 16, channel_blocks(s, 16)), dim3(256), st, a);
        return GDN_OK;
    });
}

}  // namespace

int conv_partials(const gdn_conv_shape& s)
{
    const long long rows = (long long)conv_strip(s) * (256 / channel_words(s));
    return (int)((s.T + rows - 1) / rows);
}

gdn_status conv_forward_dispatch(const gdn_conv_shape& s, const ConvArgs& a, hipStream_t st)
{
    return s.dtype == GDN_BF16 ? forward<bf16>(s, a, st) : forward<float>(s, a, st);
}

gdn_status conv_backward_dispatch(const gdn_conv_shape& s, const ConvArgs& a, float* dw, float* db, hipStream_t st)
{
    return s.dtype == GDN_BF16 ? backward<bf16>(s, a, dw, db, st) : backward<float>(s, a, dw, db, st);
}

}  // namespace gdn
