// What the kernels for drafted tokens share: the lengths of a sequence's
// committed and drafted slots, and which drafts a query row sees.
#pragma once

#include "ic_device.cuh"

namespace ic {

constexpr int kMaxDrafts = 64;  // one bit each in a row's mask

struct TreeArgs {
    const int32_t* prefix_len;
    const int32_t* draft_len;           // null: T each
    const unsigned long long* mask;     // null: a chain
    int T;
    int cap;  // slots of a sequence's cache
};

// Committed and drafted slots of sequence b; m = 0 for lengths out of range
// (then nothing of the sequence is read or written).  Returns false for those.
__device__ __forceinline__ bool tree_lens(const TreeArgs& a, int b, int& n, int& m) {
    n = __ldg(a.prefix_len + b);
    m = a.draft_len ? __ldg(a.draft_len + b) : a.T;
    const bool ok = n >= 0 && m >= 0 && m <= a.T && n <= a.cap - m;
    if (!ok) n = m = 0;
    return ok;
}

// The drafts that row (b, t) sees, of the sequence's m.
__device__ __forceinline__ unsigned long long tree_bits(const TreeArgs& a, int b, int t, int m) {
    const unsigned long long all = m >= 64 ? ~0ull : (1ull << m) - 1ull;
    const unsigned long long bits =
        a.mask ? __ldg(a.mask + static_cast<long long>(b) * a.T + t) : (2ull << t) - 1ull;
    return bits & all;
}

// ------------------------------------------------------- the line of work
// Work of all sequences on one line: sequence b contributes groups * tiles
// items, a group being up to group_rows of its m * rows_per_draft query rows
// and a tile kLineTile keys.  The line is cut into equal ranges, one per CTA;
// lengths live on the device, so each CTA finds its own range.
constexpr int kLineTile = 128;

struct TreeLine {
    TreeArgs ta;
    int listed;  // keys before the drafts: that many, or prefix_len when < 0
    int rows_per_draft;
    int group_rows;
};
struct SeqWork {
    int n, m, rows, groups, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const TreeLine& a, int b) {
    SeqWork w;
    tree_lens(a.ta, b, w.n, w.m);
    w.rows = w.m * a.rows_per_draft;
    w.groups = (w.rows + a.group_rows - 1) / a.group_rows;
    const int keys = (a.listed >= 0 ? a.listed : w.n) + w.m;
    w.tiles = (keys + kLineTile - 1) / kLineTile;
    return w;
}
// Items of all sequences before `b_end` (called by one whole warp).  The
// host checks that all of them fit 32 bits (line_fits).
__device__ __forceinline__ int tiles_before(const TreeLine& a, int b_end) {
    int sum = 0;
    for (int b = threadIdx.x & 31; b < b_end; b += 32) {
        const SeqWork w = seq_work(a, b);
        sum += w.groups * w.tiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// Range [g0, g1) of CTA `cta`, and the sequence b0 that g0 lies in, whose
// first item is `base`.  No CTA up to min(ctas, items) is left without items.
struct LineRange {
    int g0, g1, base, b0;
};
__device__ __forceinline__ LineRange line_range(const TreeLine& a, int B, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    const long long total = tiles_before(a, B);
    const int parts = total < ctas ? static_cast<int>(total) : ctas;
    LineRange r{0, 0, 0, 0};
    if (cta >= parts) return r;
    r.g0 = static_cast<int>(total * cta / parts);
    r.g1 = static_cast<int>(total * (cta + 1) / parts);
    for (int c = 0; c < B; c += 32) {  // 32 sequences at a time
        int mine = 0;
        if (c + lane < B) {
            const SeqWork w = seq_work(a, c + lane);
            mine = w.groups * w.tiles;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, r.base + incl > r.g0);
        if (past) {
            const int l = __ffs(past) - 1;
            r.b0 = c + l;
            r.base += __shfl_sync(0xffffffffu, incl - mine, l);
            break;
        }
        r.base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}
// Whether the longest line that B sequences of these capacities could make
// (and one tile more per CTA) fits 32 bits.
inline bool line_fits(int B, long long groups_max, long long keys_max) {
    return static_cast<long long>(B) * groups_max * ((keys_max + kLineTile - 1) / kLineTile) < (1ll << 30);
}

// One part of a (sequence, row group): key tiles [t0, t1) of w.tiles.
struct Part {
    SeqWork w;
    int b, group, t0, t1;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == w.tiles; }
};

// Walks a CTA's range part by part.
struct PartWalk {
    int g, g_end, base, b;  // base: items before sequence b
    Part p;
    __device__ __forceinline__ explicit PartWalk(const LineRange& r)
        : g(r.g0), g_end(r.g1), base(r.base), b(r.b0) {}
    __device__ __forceinline__ bool next(const TreeLine& a) {
        if (g >= g_end) return false;
        SeqWork w = seq_work(a, b);
        while (g >= base + w.groups * w.tiles) {
            base += w.groups * w.tiles;
            w = seq_work(a, ++b);
        }
        const int off = g - base;
        p.w = w;
        p.b = b;
        p.group = off / w.tiles;
        p.t0 = off - p.group * w.tiles;
        p.t1 = min(w.tiles, p.t0 + (g_end - g));
        g += p.t1 - p.t0;
        return true;
    }
};

}  // namespace ic
