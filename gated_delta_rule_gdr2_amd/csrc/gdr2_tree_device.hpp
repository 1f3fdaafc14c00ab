// Device building blocks of trees of drafted tokens over a paged cache: spans, the line of rows, and a row's tree.
#pragma once
#include "gdr2_device.hpp"
#include "gdr2_tree.hpp"

namespace gdr2 {

struct TreeSpan {
    int start, lo, hi, u0, units;  // context tokens; first and last token that any draft may see; units
};
// U: tokens of a unit
template <int U>
__device__ __forceinline__ TreeSpan tree_span(const TreeArgs& a, int b) {
    const long long cap = (long long)a.c.max_pages << a.c.shift;
    const int st = a.starts[b];
    TreeSpan s;
    s.start = st < 0 ? 0 : (long long)st < cap ? st : (int)cap;
    s.hi = (int)min((long long)s.start + a.T, cap);
    s.lo = a.window > 0 && s.start >= a.window ? s.start + 1 - a.window : 0;
    s.u0 = s.lo / U;
    s.units = max(1, (s.hi + U - 1) / U - s.u0);
    return s;
}

// The line of all rows (gdr2_attn.hip): lane t holds the place before its run of `per` sequences.
struct TreeLine {
    unsigned before, total, share;
    int per;
};
template <int U>
__device__ __forceinline__ TreeLine tree_line(const TreeArgs& a) {
    const int l = lane_id(), HR = a.Hkv * a.nb;
    TreeLine p;
    p.per = (a.B + 63) / 64;
    unsigned own = 0;
    for (int i = 0; i < p.per; ++i) {
        const int b = l * p.per + i;
        if (b < a.B) own += (tree_span<U>(a, b).units + a.cost) * HR;
    }
    unsigned x = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const unsigned y = __shfl_up(x, o);
        if (l >= o) x += y;
    }
    p.before = x - own;
    p.total = __builtin_amdgcn_readlane(x, 63);
    p.share = max((p.total + a.wgs - 1) / a.wgs, (unsigned)a.share_min);
    return p;
}
struct TreeAt {
    int b;
    unsigned at;
    TreeSpan sp;
};
template <int U>
__device__ __forceinline__ TreeAt tree_find(const TreeArgs& a, const TreeLine& line, unsigned t) {
    const int HR = a.Hkv * a.nb;
    const int ln = __popcll(__ballot(line.before <= t && lane_id() * line.per < a.B)) - 1;
    TreeAt f;
    f.b = ln * line.per;
    f.at = __builtin_amdgcn_readlane(line.before, ln);
    f.sp = tree_span<U>(a, f.b);
    while (t >= f.at + (f.sp.units + a.cost) * HR) {
        f.at += (f.sp.units + a.cost) * HR;
        f.sp = tree_span<U>(a, ++f.b);
    }
    return f;
}

// The tree of sequence b, draft i in lane i: the drafts that it sees (itself and those above it, within the window),
// how many lie above it, and whether it is one (a chain of parents that ends at -1) or padding.
struct TreeLane {
    unsigned long long sees, all;  // all: the drafts of the tree
    int depth;
};
__device__ __forceinline__ TreeLane tree_lane(const TreeArgs& a, int b) {
    const int i = lane_id();
    const int p = i < a.T ? a.parents[(size_t)b * a.T + i] : -2;
    int ok = p >= -1 && p < i;
    const int up = ok && p >= 0 ? p : i;
    TreeLane t;
    t.depth = up != i;
    t.sees = 1ull << i;
    int hop = up;
    ok &= __shfl(ok, up);
    for (int n = 1; n < a.T; n *= 2) {
        t.sees |= __shfl(t.sees, hop);
        t.depth += __shfl(t.depth, hop);
        ok &= __shfl(ok, hop);
        hop = __shfl(hop, hop);
    }
    if (a.window > 0 && a.window < a.T) {  // the nearest ones only
        unsigned long long m = 0;
        int x = i;
        for (int n = 0; n < a.window; ++n) {
            m |= 1ull << x;
            x = __shfl(up, x);
        }
        t.sees = m;
    }
    t.all = __ballot(ok);
    if (!ok) t.sees = 0;
    return t;
}

}  // namespace gdr2
