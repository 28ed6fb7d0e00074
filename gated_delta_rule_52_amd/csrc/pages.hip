// pages.hip -- one step of continuous batching over the paged cache: pages of
// finished sequences go back to a stack of free ones (gdn_pages_release), new
// tokens get pages from its top, and the step's sequence bounds, positions and
// cache slots are built (gdn_pages_take).  Whole numbers; everything follows from
// prefix sums over the sequences:
//
//   release   back_b = done_b ? ceil(len_b / S) : 0; its pages go to count + sum_{b' < b} back_b' ...
//   take      fresh_b = ceil((len_b + want_b) / S) - ceil(len_b / S); b is served if its table has room, the
//             stack holds sum_{b' <= b} fresh_b' (or fresh_b = 0), and the rows hold all tokens up to its own
//
// Bound by latency (256 sequences), then by the maps' bytes.  Every workgroup forms
// the sums for itself, 1024 sequences at a time, and keeps what it needs of them in
// LDS; the pages or tokens are then dealt to all threads, each finding its sequence
// by bisection in LDS.  The first workgroup writes the lengths and the count; where
// these replace the ones that were read, a launch of its own does, behind the others.
// 256 sequences: 5 and 8 us; 512 sequences that ask for 650 thousand tokens: 5 and 13 us.
#include "pages.h"

#include "common.h"

namespace gdn {

namespace {

typedef long long i64;

// sum over the lanes up to and with the lane itself, for all 1024 threads of the
// workgroup; `all` is the sum over them.  red: 16 values, free after the call's
// second barrier until the next call's first.
__device__ __forceinline__ i64 scan_1024(i64 x, i64* red, i64& all)
{
    const int l = lane_id(), w = wave_id();
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const i64 up = __shfl_up(x, o);
        if (l >= o) x += up;
    }
    __syncthreads();
    if (l == 63) red[w] = x;
    __syncthreads();
    i64 before = 0;
    all = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const i64 r = red[k];
        if (k < w) before += r;
        all += r;
    }
    return before + x;
}

// how many of the n ascending values are at or below x
__device__ __forceinline__ int at_or_below(const int* v, int n, int x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

struct PagesArgs {
    const int *flag, *kv_len, *free_count;  // flag: done or want
    int *table, *free_pages;
    int *kv_out, *count_out, *cu, *positions;
    i64* slots;
    int B, width, shift, pool, rows;
    int maps, counts;  // what this launch writes
};

__device__ __forceinline__ i64 pages_of(i64 len, int shift) { return (len + (1 << shift) - 1) >> shift; }
__device__ __forceinline__ int count_of(const PagesArgs& a)
{
    const int c = a.free_count[0];
    return c < 0 ? 0 : c > a.pool ? a.pool : c;
}

template <int CAP>
__global__ __launch_bounds__(1024) void pages_release_kernel(PagesArgs a)
{
    __shared__ i64 red[16];
    __shared__ int end_s[CAP];  // pages given back up to and with each sequence
    const int count = count_of(a);
    i64 carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        i64 back = 0;
        if (b < a.B) {
            const int len = a.kv_len[b], done = a.flag[b];
            if (done && len > 0) back = pages_of(len, a.shift);
            if (back > a.width) back = a.width;
            if (a.counts && blockIdx.x == 0) a.kv_out[b] = done || len < 0 ? 0 : len;
        }
        i64 all;
        const i64 inc = carry + scan_1024(back, red, all);
        // nothing lies past the stack's end
        if (b < a.B) end_s[b] = (int)(inc < a.pool - count ? inc : a.pool - count);
        carry += all;
    }
    __syncthreads();
    const int total = (int)(carry < a.pool - count ? carry : a.pool - count);
    if (a.counts && blockIdx.x == 0 && threadIdx.x == 0) a.count_out[0] = count + total;
    if (!a.maps) return;
    for (i64 i = (i64)blockIdx.x * 1024 + threadIdx.x; i < total; i += (i64)gridDim.x * 1024) {
        const int b = at_or_below(end_s, a.B, (int)i);
        a.free_pages[count + i] = a.table[(size_t)b * a.width + (i - (b ? end_s[b - 1] : 0))];
    }
}

template <int CAP>
__global__ __launch_bounds__(1024) void pages_take_kernel(PagesArgs a)
{
    __shared__ i64 red[16];
    __shared__ int end_s[CAP], len_s[CAP], top_s[CAP];  // tokens up to and with a sequence; its length before; the stack above its pages
    const int count = count_of(a);
    i64 asked = 0, wanted = 0, taken = 0, tokens = 0;
    for (int b0 = 0; b0 < a.B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        const bool real = b < a.B;
        i64 len = 0, want = 0;
        if (real) {
            len = a.kv_len[b], want = a.flag[b];
            len = len < 0 ? 0 : len;
            want = want < 0 ? 0 : want;
        }
        const i64 have = pages_of(len, a.shift), need = pages_of(len + want, a.shift);
        bool ok = real && need <= a.width;
        i64 fresh = ok ? need - have : 0, all;
        const i64 inc = asked + scan_1024(fresh, red, all);
        asked += all;
        ok = ok && (fresh == 0 || inc <= count);
        const i64 row = wanted + scan_1024(ok ? want : 0, red, all);
        wanted += all;
        ok = ok && row <= a.rows;
        fresh = ok ? fresh : 0;
        want = ok ? want : 0;
        const i64 below = taken + scan_1024(fresh, red, all) - fresh;
        taken += all;
        const i64 end = tokens + scan_1024(want, red, all);
        tokens += all;
        if (real) {
            end_s[b] = (int)end;
            len_s[b] = (int)len;
            top_s[b] = (int)(count - below);
            if (blockIdx.x == 0) {
                if (a.maps) a.cu[b + 1] = (int)end;
                if (a.counts) a.kv_out[b] = (int)(len + want);
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (a.maps) a.cu[0] = 0;
        if (a.counts) a.count_out[0] = (int)(count - taken);
    }
    __syncthreads();
    if (!a.maps) return;
    const int mask = (1 << a.shift) - 1;
    for (i64 i = (i64)blockIdx.x * 1024 + threadIdx.x; i < tokens; i += (i64)gridDim.x * 1024) {
        const int b = at_or_below(end_s, a.B, (int)i), first = b ? end_s[b - 1] : 0;
        const int len = len_s[b], pos = len + (int)(i - first), at = pos >> a.shift;
        const int k = at - (int)pages_of(len, a.shift);  // the k-th of the sequence's new pages
        int* entry = a.table + (size_t)b * a.width + at;
        const int page = k >= 0 ? a.free_pages[top_s[b] - 1 - k] : *entry;
        if (k >= 0 && (pos & mask) == 0) *entry = page;
        if (a.positions) a.positions[i] = pos;
        if (a.slots) a.slots[i] = page < 0 ? -1 : ((i64)page << a.shift) + (pos & mask);
    }
}

// LDS for the sequences a call may have: 1024 are the usual batch, and three words
// each of 8192 would leave one workgroup a compute unit
template <typename F> gdn_status with_capacity(int B, F&& f)
{
    return B <= 1024 ? f(std::integral_constant<int, 1024>{}) : f(std::integral_constant<int, 8192>{});
}

// workgroups for `items`, four a thread
unsigned groups(i64 items)
{
    const i64 n = (items + 4095) / 4096;
    return (unsigned)(n < 1 ? 1 : n > 256 ? 256 : n);
}

}  // namespace

gdn_status pages_release_dispatch(const gdn_pages_shape& s, const int* done, const int* kv_len, const int* table, int* free_pages,
                                  const int* free_count, int* kv_out, int* count_out, hipStream_t st)
{
    PagesArgs a{};
    a.flag = done; a.kv_len = kv_len; a.free_count = free_count;
    a.table = const_cast<int*>(table); a.free_pages = free_pages; a.kv_out = kv_out; a.count_out = count_out;
    a.B = s.B; a.width = s.max_pages; a.shift = __builtin_ctz((unsigned)s.page_size); a.pool = s.num_pages;
    const bool in_place = kv_out == kv_len || count_out == free_count;
    const i64 most = (i64)s.B * s.max_pages < s.num_pages ? (i64)s.B * s.max_pages : s.num_pages;
    return with_capacity(s.B, [&](auto cap) -> gdn_status {
        constexpr int CAP = decltype(cap)::value;
        a.maps = 1;
        a.counts = !in_place;
        GDN_LAUNCH("pages_release", (pages_release_kernel<CAP>), dim3(groups(most)), dim3(1024), st, a);
        if (in_place) {
            a.maps = 0;
            a.counts = 1;
            GDN_LAUNCH("pages_release_counts", (pages_release_kernel<CAP>), dim3(1), dim3(1024), st, a);
        }
        return GDN_OK;
    });
}

gdn_status pages_take_dispatch(const gdn_pages_shape& s, const int* want, const int* kv_len, int* table, const int* free_pages,
                               const int* free_count, int* kv_out, int* count_out, int* cu, int* positions, long long* slots,
                               hipStream_t st)
{
    PagesArgs a{};
    a.flag = want; a.kv_len = kv_len; a.free_count = free_count;
    a.table = table; a.free_pages = const_cast<int*>(free_pages); a.kv_out = kv_out; a.count_out = count_out;
    a.cu = cu; a.positions = positions; a.slots = slots;
    a.B = s.B; a.width = s.max_pages; a.shift = __builtin_ctz((unsigned)s.page_size); a.pool = s.num_pages; a.rows = s.rows;
    const bool in_place = kv_out == kv_len || count_out == free_count;
    return with_capacity(s.B, [&](auto cap) -> gdn_status {
        constexpr int CAP = decltype(cap)::value;
        a.maps = 1;
        a.counts = !in_place;
        GDN_LAUNCH("pages_take", (pages_take_kernel<CAP>), dim3(groups(s.rows)), dim3(1024), st, a);
        if (in_place) {
            a.maps = 0;
            a.counts = 1;
            GDN_LAUNCH("pages_take_counts", (pages_take_kernel<CAP>), dim3(1), dim3(1024), st, a);
        }
        return GDN_OK;
    });
}

}  // namespace gdn
