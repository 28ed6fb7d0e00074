// ssm_walk.hip -- the states between the chunks of the selective state space scan,
// forward and, for the gradients, backward:
//
//   S_out  = exp(c_L) S_in  + B^T (exp(c_L - c) delta x)     over a sequence's chunks
//   dS_in  = exp(c_L) dS_out + C^T (exp(c) dy)               over them in reverse
//
// A workgroup walks a segment of a sequence with two slices of 64 of its heads'
// values: a wave has 32 of them, whose N x 32 state it keeps in fp32 accumulators.
// It reads both operands down the tokens by transposing loads, scales its own (f x)
// and splits it into three bf16 that hold all its bits, so that the state is as
// exact as in fp32: three products for one.  Half a chunk is in LDS at a time, the
// other half on its way there by direct loads, so that two workgroups share a compute
// unit: a wave alone on its SIMD issues its products, its splitting and its reads one
// after the other (6.2 thousand cycles for 96 products that take 3.2).
//
// Where sequences are cut into segments, a first launch walks the first of them as
// it is and forms what the others but the last contribute from a zero state, a second
// adds these up along the sequence, and a third walks the segments but the first from
// there: most products are formed twice, fewer in a row.  8 sequences of 4096 tokens, 6
// heads of 128, N = 128: forward 28 + 10 + 28 us, both ways 47 + 10 + 65 us.  The given state is read by
// the first segment's workgroup alone and the last state written behind it, so they
// may be one.
#include <stddef.h>

#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct WalkArgs {
    const void *rows, *vals;  // B and x, or C and dy
    const float* init;        // h0 or dhT
    float* last;              // hT or dh0
    float *seg, *tot;         // [segs][slices] states and logarithms of decays
    void* between;            // [states][slices] states; for the outputs, then each sequence's first
    long long rs, vs;
};
struct WalkCall {
    WalkArgs way[2];  // forward, backward
    const float* dec;
    const int* cu;
    long long firsts;
    int nb, T, H, P, per_group, slices, pairs, seg_len;  // pairs: of slices, in a group
};

template <typename T, int N> struct WalkLds {
    static constexpr int L = SsmTile<T>::L;
    static constexpr int H = L / 2;
    char rows[2][H * Rows<T, N>::BYTES], vals[2][2][H * Rows<T, kSlice>::BYTES];
    float f[2][2][64];
};

// PHASE 0: all segments of a sequence but the last; 1: all but the first, or the only
// one.  OUT: states between chunks as T, rounded to nearest: they are operands of the
// outputs alone (ssm_out.hip), the walk goes on from its own in fp32, and they are half
// the bytes.  Otherwise fp32, for the gradients: those of the steps are sums of products
// with them that have to be as exact as in fp32.
template <typename T, int N, bool BACK, int PHASE, bool OUT>
__device__ __forceinline__ void walk_segment(const WalkCall& a, const WalkArgs& g, WalkLds<T, N>& m)
{
    constexpr int L = SsmTile<T>::L, HALF = L / 2, PARTS = SsmTile<T>::PARTS, NT = N / 32, KK = HALF / 16;
    using RT = Rows<T, N>;
    using VT = Rows<T, kSlice>;
    using Lds = WalkLds<T, N>;

    long long id;
    int pair;
    deal(blockIdx.x, a.H / a.per_group * a.pairs, id, pair);
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, a.seg_len * L, 1, PHASE, id, u)) return;
    if (u.count > 1 && (PHASE == 1) != BACK) ++u.at;  // the first of the walk is left out, or the last
    const int order = BACK && u.count ? u.count - 1 - u.at : u.at;
    const int w = uniform(wave_id()), l = lane_id(), which = w >> 1, pt = w & 1;
    const int group = pair / a.pairs, per_head = a.P / kSlice, in_group = a.per_group * per_head;
    const int at_group = 2 * (pair - group * a.pairs) + which;
    const bool live_slice = at_group < in_group;  // an odd slice has no neighbour: its waves take the other's place and write nothing
    const int slice = group * in_group + (live_slice ? at_group : at_group - 1);
    const int head = slice / per_head, p0 = (slice - head * per_head) * kSlice, col = 32 * pt + (l & 31);

    const int c0 = u.at * a.seg_len, c1 = u.chunks - c0 < a.seg_len ? u.chunks : c0 + a.seg_len, count = c1 - c0;
    const T* rows = (const T*)g.rows + (size_t)group * N;
    const T* vals = (const T*)g.vals + (size_t)head * a.P + p0;
    auto chunk_of = [&](int k) { return BACK ? c1 - 1 - k : c0 + k; };
    float keep_next = 1.f, total_next = 0.f;
    // Half a chunk into its buffer by direct loads, in KK shares: a wave loads a quarter
    // of the rows, and half of its slice's values and factors (0 behind the last token,
    // whose rows are copies).
    constexpr int RI = HALF / 4 / RT::PER, VI = HALF / 2 / VT::PER;  // direct loads of a wave
    // offsets of rows from the half's first fit 31 bits, also where they are not whole loads
    static_assert((HALF - 1) * kMostStride * (long long)sizeof(T) + RT::BYTES < (1LL << 31), "row offsets");
    const uint32_t r_row = (uint32_t)(g.rs * sizeof(T)), v_row = (uint32_t)(g.vs * sizeof(T));
    struct Source {
        const char *rows, *vals;
        const float* dec;
        int live;  // of the half's tokens
    };
    auto source_of = [&](int k, int half) {
        const int c = chunk_of(k), from = c * L + half * HALF, live = u.n - from;
        const size_t row0 = (size_t)u.start + (live < 1 ? u.n - 1 : from);
        return Source{(const char*)(rows + row0 * g.rs), (const char*)(vals + row0 * g.vs),
                      a.dec + ((size_t)(u.before + c) * a.H + head) * kDecays<L>, live < 1 ? 1 : live < HALF ? live : HALF};
    };
    const uint32_t lds = lds_offset(&m);
    const uint32_t r_off = (l / RT::U) * r_row, v_off = (l / VT::U) * v_row;
    auto load = [&](const Source& s, int buf, int part, bool full) {
#pragma unroll
        for (int i = VI * part / KK; i < VI * (part + 1) / KK; ++i) {
            const int r = HALF / 2 * pt + i * VT::PER, rr = r + l / VT::U;
            const uint32_t word = ((l % VT::U) ^ VT::f(rr)) * 16, to = lds + (uint32_t)offsetof(Lds, vals) + (2 * buf + which) * HALF * VT::BYTES + r * VT::BYTES;
            if (full)
                dma16_to(s.vals + (size_t)r * v_row, v_off + word, to);
            else
                dma16_to(s.vals, (uint32_t)(rr < s.live ? rr : s.live - 1) * v_row + word, to);
        }
#pragma unroll
        for (int i = RI * part / KK; i < RI * (part + 1) / KK; ++i) {
            const int r = HALF / 4 * w + i * RT::PER, rr = r + l / RT::U;
            const uint32_t word = ((l % RT::U) ^ RT::f(rr)) * 16, to = lds + (uint32_t)offsetof(Lds, rows) + buf * HALF * RT::BYTES + r * RT::BYTES;
            if (full)
                dma16_to(s.rows + (size_t)r * r_row, r_off + word, to);
            else
                dma16_to(s.rows, (uint32_t)(rr < s.live ? rr : s.live - 1) * r_row + word, to);
        }
        // 64 words for HALF factors: the rest is not read
        if (part == 0 && pt == 0)
            dma4(s.dec + (BACK ? DEC_E : DEC_FD) * L + HALF * buf + (HALF == 64 ? l : l & 31), m.f[buf][which]);
    };
    auto load_all = [&](const Source& s, int buf) {
#pragma unroll
        for (int part = 0; part < KK; ++part) load(s, buf, part, false);
    };
    if (count > 0) {
        const Source s = source_of(0, 0);
        keep_next = s.dec[DEC_ROWS * L + DEC_KEEP];
        total_next = s.dec[DEC_ROWS * L + DEC_TOTAL];
        load_all(s, 0);
    }

    f32x16 acc[NT];
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][r] = f(acc[i][r], 32 * i + acc_rows(r >> 2) + (r & 3), i, r);
    };
    each([&](float, int, int, int) { return 0.f; });
    if (order == 0) {
        if (g.init) {
            const float* s = g.init + ((size_t)u.b * a.H + head) * N * a.P + p0 + col;
            each([&](float, int n, int, int) { return s[(size_t)n * a.P]; });
        }
    } else if (PHASE == 1) {
        const size_t at = (size_t)(u.first + u.at + (BACK ? 1 : -1)) * a.slices + slice;
        const float* s = g.seg + at * N * kSlice + col * 4;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(s + (32 * i + acc_rows(r >> 2)) * kSlice);
                acc[i][r] = v[0], acc[i][r + 1] = v[1], acc[i][r + 2] = v[2], acc[i][r + 3] = v[3];
            }
    }

    // a state as four rows of N after the other, their values side by side: what a lane
    // holds is stored as it stands (load_state8 reads it)
    auto store_state = [&](auto* s) {
        typedef std::remove_reference_t<decltype(*s)> S;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                store4<S>(s + (32 * i + acc_rows(r >> 2)) * kSlice + col * 4, acc[i][r], acc[i][r + 1], acc[i][r + 2], acc[i][r + 3]);
    };
    auto store_between = [&](long long state) {
        typedef std::conditional_t<OUT, T, float> S;
        if (live_slice) store_state((S*)g.between + ((size_t)state * a.slices + slice) * N * kSlice);
    };
    float tot = 0.f;
    // half a chunk, from its buffer; the next one's loads on the way
    auto step = [&](int k, auto HALF_OF) {
        constexpr int buf = HALF_OF();
        wait_vm<0>();
        __syncthreads();
        // behind the last half it is loaded again
        const Source next = buf == 0 ? source_of(k, 1) : k + 1 < count ? source_of(k + 1, 0) : source_of(k, 1);
        if constexpr (buf == 0) {
            const float keep = keep_next;
            tot += total_next;
            if (PHASE == 1 || order == 0) {
                const int c = chunk_of(k);
                if (c != (BACK ? u.chunks - 1 : 0))
                    store_between(u.between + (BACK ? c : c - 1));
                else if (OUT && g.init)
                    store_between(a.firsts + u.b);
            }
            each([&](float v, int, int, int) { return v * keep; });
        } else {
            keep_next = next.dec[DEC_ROWS * L + DEC_KEEP];
            total_next = next.dec[DEC_ROWS * L + DEC_TOTAL];
        }
        const bool full = next.live == HALF;
        if (!full) load_all(next, buf ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        Frag<T> f[2][NT], raw;
        f32x4 f0, f1;
        auto read = [&](int kk, Frag<T> (&o)[NT]) {
            const float* fs = m.f[buf][which] + 16 * kk + acc_rows(0);  // permuted order
            raw = VT::down(m.vals[buf][which], 16 * kk, 32 * pt);
            f0 = *reinterpret_cast<const f32x4*>(fs);
            f1 = *reinterpret_cast<const f32x4*>(fs + 8);
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i] = RT::down(m.rows[buf], 16 * kk, 32 * i);
        };
        Frag<T> v[2][PARTS];
        auto scale = [&](Frag<T> (&o)[PARTS]) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)raw[j] * (j < 4 ? f0[j & 3] : f1[j & 3]);
            if constexpr (sizeof(T) == 2) {
                u32x4 p[3];
                split(x, p);
#pragma unroll
                for (int i = 0; i < 3; ++i) o[i] = __builtin_bit_cast(bf16x8, p[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[0][j] = x[j];
            }
        };
        read(0, f[0]);
        scale(v[0]);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if (kk + 1 < KK) read(kk + 1, f[(kk + 1) & 1]);
            if (full) load(next, buf ^ 1, kk, true);
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i] = mma32(f[kk & 1][i], v[kk & 1][p], acc[i]);
            if (kk + 1 < KK) scale(v[(kk + 1) & 1]);
        }
    };
    for (int k = 0; k < count; ++k) {
        step(k, std::integral_constant<int, 0>{});
        step(k, std::integral_constant<int, 1>{});
    }
    wait_vm<0>();  // the last half's second load
    if (!live_slice) return;
    if (PHASE == 0) {
        const size_t at = (size_t)(u.first + u.at) * a.slices + slice;
        if (pt == 0 && l == 0) g.tot[at] = tot;
        store_state(g.seg + at * N * kSlice);
    } else if (g.last && order >= u.count - 1) {
        float* s = g.last + ((size_t)u.b * a.H + head) * N * a.P + p0 + col;
        each([&](float v, int n, int, int) { return s[(size_t)n * a.P] = v; });
    }
}

template <typename T, int N, int PHASE, bool OUT>
__global__ __launch_bounds__(256, 2) void ssm_walk_kernel(WalkCall a)
{
    __shared__ __align__(16) WalkLds<T, N> m;
    if (OUT || blockIdx.y == 0)
        walk_segment<T, N, false, PHASE, OUT>(a, a.way[0], m);
    else
        walk_segment<T, N, true, PHASE, OUT>(a, a.way[1], m);
}

// The states at the segments' ends, in place, from what each contributes: four values
// a thread along a sequence's segments (blockIdx.y: of the sequences that have several),
// those to come on their way.
// blockIdx.x: slice and 1024 values of it; blockIdx.z: way.
template <int L, int N> __global__ __launch_bounds__(256) void ssm_segments_kernel(WalkCall a)
{
    constexpr int BLOCKS = N * kSlice / 1024, AHEAD = 4;
    const WalkArgs& g = a.way[blockIdx.z];
    const bool back = blockIdx.z != 0;
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, a.seg_len * L, -1, 0, blockIdx.y, u)) return;
    const int slice = blockIdx.x / BLOCKS, many = u.count - 1;  // those of the first launch
    const size_t at0 = (size_t)(u.first + (back ? u.count - 1 : 0)) * a.slices + slice;
    const long long step = (back ? -1LL : 1LL) * a.slices;
    float* s = g.seg + (blockIdx.x % BLOCKS * 256 + threadIdx.x) * 4;
    auto at = [&](int k) { return s + (at0 + k * step) * N * kSlice; };
    f32x4 v[AHEAD], acc{0.f, 0.f, 0.f, 0.f};
    float decay[AHEAD];
    auto fetch = [&](int k, int i) {
        v[i] = *reinterpret_cast<const f32x4*>(at(k));
        decay[i] = g.tot[at0 + k * step];
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (k < many) fetch(k, k);
    for (int k0 = 0; k0 < many; k0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = k0 + i;
            if (k < many) {
                const float e = exp2_hw(decay[i]);
                // the first is whole as it stands
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = k ? __builtin_fmaf(acc[j], e, v[i][j]) : v[i][j];
                if (k + AHEAD < many) fetch(k + AHEAD, i);
                if (k) *reinterpret_cast<f32x4*>(at(k)) = acc;
            }
        }
    }
}

template <typename T, int N, bool OUT> gdn_status walk(const SsmPlan& p, const WalkCall& a, hipStream_t st)
{
    // a sequence has one segment fewer in the first launch, and in the last one at least;
    // those that have several are at most as many as whole segments fit into the tokens
    const int jobs = a.H / a.per_group * a.pairs;
    const dim3 grid(dealt(p.segs, jobs), OUT ? 1 : 2);
    if (p.seg) {
        const long long whole = p.segs - a.nb;
        GDN_LAUNCH("ssm_walk_segments", (ssm_walk_kernel<T, N, 0, OUT>), dim3(dealt(whole, jobs), OUT ? 1 : 2), dim3(256), st, a);
        GDN_LAUNCH("ssm_segments", (ssm_segments_kernel<SsmTile<T>::L, N>),
                   dim3(a.slices * (N / 16), (unsigned)(whole < a.nb ? whole : a.nb), OUT ? 1 : 2), dim3(256), st, a);
    }
    GDN_LAUNCH("ssm_walk", (ssm_walk_kernel<T, N, 1, OUT>), grid, dim3(256), st, a);
    return GDN_OK;
}

template <typename T> gdn_status walk(int N, bool backward, const SsmPlan& p, const WalkCall& a, hipStream_t st)
{
    if (N == 64) return backward ? walk<T, 64, false>(p, a, st) : walk<T, 64, true>(p, a, st);
    return backward ? walk<T, 128, false>(p, a, st) : walk<T, 128, true>(p, a, st);
}

}  // namespace

gdn_status ssm_walk(const gdn_ssm_shape& s, const SsmPlan& p, const SsmArgs& x, bool backward, char* ws, hipStream_t st)
{
    WalkCall a{};
    const long long state = (long long)p.slices * s.N * kSlice;
    for (int back = 0; back < (backward ? 2 : 1); ++back) {
        WalkArgs& g = a.way[back];
        g.rows = back ? x.C : x.B;
        g.rs = back ? x.cs : x.bs;
        g.vals = back ? x.dy : x.x;
        g.vs = back ? (long long)s.H * s.P : x.xs;
        g.init = back ? x.dhT : x.h0;
        g.last = back ? x.dh0 : backward ? nullptr : x.hT;
        g.seg = (float*)(ws + p.seg_at) + back * p.several * state;
        g.tot = (float*)(ws + p.tot_at) + back * p.several * p.slices;
        g.between = ws + (back ? p.back_at : p.fwd_at);
    }
    a.dec = (const float*)(ws + p.dec_at);
    a.cu = x.cu;
    a.firsts = p.between;
    a.nb = s.B; a.T = s.T; a.H = s.H; a.P = s.P; a.per_group = s.H / s.G; a.slices = p.slices; a.pairs = p.pairs;
    a.seg_len = p.seg ? p.seg : s.T / p.L + 1;  // longer than any sequence
    return s.dtype == GDN_BF16 ? walk<bf16>(s.N, backward, p, a, st) : walk<float>(s.N, backward, p, a, st);
}

}  // namespace gdn
