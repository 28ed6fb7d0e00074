// ssm_walk.hip -- the states between the chunks of the selective state space scan,
// forward and, for the gradients, backward:
//
//   S_out  = exp(c_L) S_in  + B^T (exp(c_L - c) delta x)     over a sequence's chunks
//   dS_in  = exp(c_L) dS_out + C^T (exp(c) dy)               over them in reverse
//
// A workgroup walks a segment of a sequence with a slice of 64 of a head's values,
// its N x 64 state in fp32 accumulators: four waves, each 32 of the 64 values and
// half of N.  The scaled operand (f x) is split into three bf16 that hold all its
// bits, so the state is as exact as in fp32.  Rows of both operands are read down
// the tokens by transposing loads; the next chunk's are on their way in registers
// meanwhile, and two workgroups share a compute unit.
//
// Where sequences are cut into segments, a first launch walks the first of them as
// it is and forms what the others but the last contribute from a zero state; the
// second launch walks those with the sum of all before them: most products are
// formed twice, fewer in a row.  The given state is read by the first segment's
// workgroup alone and the last state written behind it, so they may be one.
#include "ssm_tile.h"

#include "common.h"

namespace gdn {

namespace {

struct WalkArgs {
    const void *rows, *vals;  // B and x, or C and dy
    const float* init;        // h0 or dhT
    float* last;              // hT or dh0
    float *seg, *tot;         // [segs][slices][N][64], [segs][slices]
    void* between;            // [states][slices][..]; for the outputs, then each sequence's first
    long long rs, vs;
};
struct WalkCall {
    WalkArgs way[2];  // forward, backward
    const float* dec;
    const int* cu;
    long long firsts;
    int nb, T, H, P, per_group, slices, seg_len;
};

template <typename T, int N> struct WalkLds {
    static constexpr int L = SsmTile<T>::L;
    char rows[L * Rows<T, N>::BYTES], vals[SsmTile<T>::PARTS][L * Rows<T, kSlice>::BYTES];
};

// PHASE 0: all segments of a sequence but the last; 1: all but the first, or the only
// one.  OUT: states as T [64][N] (operands of the outputs), otherwise fp32 [N][64].
template <typename T, int N, bool BACK, int PHASE, bool OUT>
__device__ __forceinline__ void walk_segment(const WalkCall& a, const WalkArgs& g, WalkLds<T, N>& m)
{
    constexpr int L = SsmTile<T>::L, PARTS = SsmTile<T>::PARTS, NT = N / 64;
    using RT = Rows<T, N>;
    using VT = Rows<T, kSlice>;
    constexpr int RW = L * RT::U / 256, VW = L * VT::U / 256;  // words a thread stages

    long long id;
    int slice;
    deal(blockIdx.x, a.slices, id, slice);
    Unit u;
    if (!find_unit<L>(a.cu, a.nb, a.T, a.seg_len * L, 1, id, u)) return;
    const int order = BACK ? u.count - 1 - u.at : u.at;
    if (PHASE == 0 ? order == u.count - 1 : order == 0 && u.count > 1) return;
    const int per_head = a.P / kSlice, head = slice / per_head, p0 = (slice - head * per_head) * kSlice;
    const int l = lane_id(), w = uniform(wave_id()), pt = w & 1, n0 = (w >> 1) * (N / 2), tid = threadIdx.x;
    const int col = 32 * pt + (l & 31);

    const int c0 = u.at * a.seg_len, c1 = u.chunks - c0 < a.seg_len ? u.chunks : c0 + a.seg_len;
    const T* rows = (const T*)g.rows + (size_t)(head / a.per_group) * N;
    const T* vals = (const T*)g.vals + (size_t)head * a.P + p0;
    u32x4 rw[RW], vw[VW];
    float fw[VW], keep, total;
    auto live_of = [&](int c) { return u.n - c * L < L ? u.n - c * L : L; };
    auto load = [&](int c) {
        const int live = live_of(c);
        const size_t row0 = (size_t)u.start + (size_t)c * L;
        const float* dec = a.dec + ((size_t)(u.before + c) * a.H + head) * kDecays<L>;
        keep = dec[DEC_ROWS * L + DEC_KEEP];
        total = dec[DEC_ROWS * L + DEC_TOTAL];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const int x = i * 256 + tid, r = x / VT::U, v = x % VT::U;
            vw[i] = *reinterpret_cast<const u32x4*>(vals + (row0 + (r < live ? r : live - 1)) * g.vs + v * (16 / sizeof(T)));
            fw[i] = BACK ? (r < live ? dec[DEC_E * L + r] : 0.f) : dec[DEC_F * L + r] * dec[DEC_DELTA * L + r];
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int x = i * 256 + tid, r = x / RT::U, v = x % RT::U;
            rw[i] = *reinterpret_cast<const u32x4*>(rows + (row0 + (r < live ? r : live - 1)) * g.rs + v * (16 / sizeof(T)));
        }
    };
    const int count = c1 - c0;
    if (count > 0) load(BACK ? c1 - 1 : c0);

    f32x16 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = zero16();
    if (order == 0) {
        if (g.init) {
            const float* s = g.init + (((size_t)u.b * a.H + head) * N + n0) * a.P + p0 + col;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][r] = s[(size_t)(32 * i + acc_rows(r >> 2) + (r & 3)) * a.P];
        }
    } else if (PHASE == 1) {
        const long long first = BACK ? id - u.at + u.count - 1 : id - u.at;
        for (int k = 0; k < order; ++k) {
            const size_t at = (size_t)(BACK ? first - k : first + k) * a.slices + slice;
            const float e = exp2_hw(g.tot[at]);
            const float* s = g.seg + (at * N + n0) * kSlice + col;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float v = s[(32 * i + acc_rows(r >> 2) + (r & 3)) * kSlice];
                    acc[i][r] = k ? __builtin_fmaf(acc[i][r], e, v) : v;
                }
        }
    }

    float tot = 0.f;
    for (int k = 0; k < count; ++k) {
        const int c = BACK ? c1 - 1 - k : c0 + k;
        __syncthreads();  // the tables of the chunk before are read
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const int x = i * 256 + tid, at = VT::word(x / VT::U, x % VT::U) * 16;
            if constexpr (sizeof(T) == 2) {
                float v[8];
                u32x4 parts[3];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = __uint_as_float(vw[i][j] << 16) * fw[i];
                    v[2 * j + 1] = upper(__uint_as_float(vw[i][j])) * fw[i];
                }
                split(v, parts);
#pragma unroll
                for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4*>(m.vals[p] + at) = parts[p];
            } else {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(__uint_as_float(vw[i][j]) * fw[i]);
                *reinterpret_cast<u32x4*>(m.vals[0] + at) = v;
            }
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int x = i * 256 + tid;
            *reinterpret_cast<u32x4*>(m.rows + RT::word(x / RT::U, x % RT::U) * 16) = rw[i];
        }
        __syncthreads();
        const float e = keep;
        tot += total;
        if (k + 1 < count) load(BACK ? c - 1 : c + 1);
        const bool edge = c == (BACK ? u.chunks - 1 : 0);
        if ((PHASE == 1 || order == 0) && (!edge || (OUT && g.init))) {
            const size_t at = (size_t)(edge ? a.firsts + u.b : u.between + (BACK ? c : c - 1)) * a.slices + slice;
            if constexpr (OUT) {
                T* s = (T*)g.between + (at * kSlice + col) * N + n0;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        store4<T>(s + 32 * i + acc_rows(r >> 2), acc[i][r], acc[i][r + 1], acc[i][r + 2], acc[i][r + 3]);
            } else {
                float* s = (float*)g.between + (at * N + n0) * kSlice + col;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[(32 * i + acc_rows(r >> 2) + (r & 3)) * kSlice] = acc[i][r];
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][r] *= e;
#pragma unroll
        for (int kk = 0; kk < L / 16; ++kk) {
            Frag<T> f[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) f[i] = RT::down(m.rows, 16 * kk, n0 + 32 * i);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const Frag<T> v = VT::down(m.vals[p], 16 * kk, 32 * pt);
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i] = mma32(f[i], v, acc[i]);
            }
        }
    }
    if (PHASE == 0) {
        const size_t at = (size_t)id * a.slices + slice;
        if (tid == 0) g.tot[at] = tot;
        float* s = g.seg + (at * N + n0) * kSlice + col;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[(32 * i + acc_rows(r >> 2) + (r & 3)) * kSlice] = acc[i][r];
    } else if (g.last && order == u.count - 1) {
        float* s = g.last + (((size_t)u.b * a.H + head) * N + n0) * a.P + p0 + col;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[(size_t)(32 * i + acc_rows(r >> 2) + (r & 3)) * a.P] = acc[i][r];
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

template <typename T, int N, bool OUT> gdn_status walk(const SsmPlan& p, const WalkCall& a, hipStream_t st)
{
    const dim3 grid((unsigned)((p.segs + 7) / 8 * 8 * p.slices), OUT ? 1 : 2);
    if (p.seg) GDN_LAUNCH("ssm_walk_segments", (ssm_walk_kernel<T, N, 0, OUT>), grid, dim3(256), st, a);
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
        g.seg = (float*)(ws + p.seg_at) + back * p.segs * state;
        g.tot = (float*)(ws + p.tot_at) + back * p.segs * p.slices;
        g.between = ws + (back ? p.back_at : p.fwd_at);
    }
    a.dec = (const float*)(ws + p.dec_at);
    a.cu = x.cu;
    a.firsts = p.between;
    a.nb = s.B; a.T = s.T; a.H = s.H; a.P = s.P; a.per_group = s.H / s.G; a.slices = p.slices;
    a.seg_len = p.seg ? p.seg : s.T / p.L + 1;  // longer than any sequence
    return s.dtype == GDN_BF16 ? walk<bf16>(s.N, backward, p, a, st) : walk<float>(s.N, backward, p, a, st);
}

}  // namespace gdn
