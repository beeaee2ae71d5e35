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

}  // namespace ic
