// ssm_plan.hip -- how a call of the state space scan over packed sequences is laid out
// (SsmPlan in ssm.h): chunks, segments, and the workspace.  Host code.
#include "ssm_tile.h"

namespace gdn {

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
