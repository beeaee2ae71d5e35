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
// and a tile kLineTile keys.  The CTAs share the line in one of two ways:
//  * by pieces: every (sequence, group) is cut into ceil(tiles / step) equal
//    pieces, one CTA each, with the smallest step that gives no more pieces
//    than CTAs; no CTA then changes its query rows;
//  * by equal ranges of the whole line, where that step would be more than
//    SLACK tiles above the mean (a change of rows costs a CTA about that).
// Lengths live on the device, so each CTA finds its own range.
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
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The work of sequence c + lane: `first` for the first 32, which every pass
// over the sequences needs again.
__device__ __forceinline__ SeqWork work_of_lane(const TreeLine& a, int B, int c, const SeqWork& first) {
    const int b = c + (threadIdx.x & 31);
    return c == 0 ? first : (b < B ? seq_work(a, b) : SeqWork{0, 0, 0, 0, 0});
}

// Range [g0, g1) of CTA `cta`, and the sequence b0 that g0 lies in, whose
// first item is `base`; step: of the pieces, 0 for equal ranges; total: items
// of the line; parts: CTAs that have any.  With equal ranges no CTA up to
// min(ctas, items) is left without items.
struct LineRange {
    int g0, g1, base, b0, step, total, parts;
};
template <int SLACK>
__device__ __forceinline__ LineRange line_range(const TreeLine& a, int B, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    LineRange r{0, 0, 0, 0, 0, 0, 0};
    const SeqWork first = lane < B ? seq_work(a, lane) : SeqWork{0, 0, 0, 0, 0};
    for (int c = 0; c < B; c += 32) {
        const SeqWork w = work_of_lane(a, B, c, first);
        r.total += w.groups * w.tiles;
    }
    r.total = warp_sum(r.total);
    r.parts = min(r.total, ctas);
    if (r.total == 0) return r;
    const int mean = (r.total + ctas - 1) / ctas;
    int n[SLACK + 1];  // pieces of steps mean, mean + 1, ..
#pragma unroll
    for (int s = 0; s <= SLACK; ++s) n[s] = 0;
    for (int c = 0; c < B; c += 32) {
        const SeqWork w = work_of_lane(a, B, c, first);
#pragma unroll
        for (int s = 0; s <= SLACK; ++s)
            n[s] += w.groups * static_cast<int>(static_cast<unsigned>(w.tiles + mean + s - 1) /
                                                static_cast<unsigned>(mean + s));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int s = 0; s <= SLACK; ++s) n[s] += __shfl_xor_sync(0xffffffffu, n[s], o);
#pragma unroll
    for (int s = SLACK; s >= 0; --s)
        if (n[s] <= ctas) {
            r.step = mean + s;
            r.parts = n[s];
        }
    if (cta >= r.parts) return r;
    // the sequence that holds this CTA's piece, or its range's first item
    const int want = r.step ? cta : static_cast<int>(static_cast<long long>(r.total) * cta / r.parts);
    int before = 0;  // pieces, or items, of the sequences before
    for (int c = 0; c < B; c += 32) {  // 32 sequences at a time
        const SeqWork w = work_of_lane(a, B, c, first);
        const int items = w.groups * w.tiles;
        const int cuts = r.step ? (w.tiles + r.step - 1) / r.step : w.tiles;
        int incl = w.groups * cuts, isum = items;
        const int mine = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o), x = __shfl_up_sync(0xffffffffu, isum, o);
            if (lane >= o) {
                incl += v;
                isum += x;
            }
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + incl > want);
        if (past) {
            const int l = __ffs(past) - 1;
            r.b0 = c + l;
            r.base += __shfl_sync(0xffffffffu, isum - items, l);
            const int off = want - before - __shfl_sync(0xffffffffu, incl - mine, l);
            if (r.step) {
                const int n = __shfl_sync(0xffffffffu, cuts, l), tiles = __shfl_sync(0xffffffffu, w.tiles, l);
                const int group = off / n, k = off - group * n;
                // below 2^24 tiles (2^31 keys) and 256 CTAs: 32 bits, unsigned
                const unsigned t = tiles, parts = n, first = k;
                r.g0 = r.base + group * tiles + static_cast<int>(t * first / parts);
                r.g1 = r.base + group * tiles + static_cast<int>(t * (first + 1) / parts);
            } else {
                r.g0 = want;
                r.g1 = static_cast<int>(static_cast<long long>(r.total) * (cta + 1) / r.parts);
            }
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        r.base += __shfl_sync(0xffffffffu, isum, 31);
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
