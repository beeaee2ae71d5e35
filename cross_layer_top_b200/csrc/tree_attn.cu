// Attention of drafted tokens over a cache:
//   o[b,t,h,:] = sum_s softmax_s(scale * Q[b,t,h,:].K[b,s,:]) V[b,s,:]
// over the committed slots (all, or the positions of one list per sequence)
// and the drafts that row (b, t) sees.  One K/V head is shared by all query
// heads and, here, by all drafts of a sequence: a key read once serves T*Hq
// query rows.
#include <math.h>

#include "ic_internal.h"
#include "tree.cuh"

using namespace ic;

namespace {

// A warp per query head and a block per (sequence, draft): lanes hold D/32
// values of q and of the running sum, keys come one by one.
template <int D>
__global__ void k_tree_attn(const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ K,
                            const __nv_bfloat16* __restrict__ V, const int32_t* __restrict__ idx,
                            TreeArgs ta, int Hq, int k, long long kv_stride, float scale_log2,
                            __nv_bfloat16* __restrict__ out, int* __restrict__ err) {
    constexpr int E = D / 32;
    const int b = blockIdx.x / ta.T, t = blockIdx.x % ta.T;
    const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int n, m;
    if (!tree_lens(ta, b, n, m) && threadIdx.x == 0) atomicCAS(err, 0, kDevBadTree);
    if (t >= m) return;
    const unsigned long long bits = tree_bits(ta, b, t, m);
    const long long qrow = (static_cast<long long>(blockIdx.x) * Hq + h) * D + lane * E;
    float qv[E], acc[E], mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(Q[qrow + e]) * scale_log2;
        acc[e] = 0.f;
    }
    const int listed = idx ? k : n;
    for (int i = 0; i < listed + m; ++i) {
        int s = i;
        if (i >= listed) {
            if (!((bits >> (i - listed)) & 1)) continue;
            s = n + i - listed;
        } else if (idx) {
            s = __ldg(idx + static_cast<long long>(b) * k + i);
            if (s < 0 || s >= n) {
                if (s != -1 && threadIdx.x == 0) atomicCAS(err, 0, kDevBadIndex);
                continue;
            }
        }
        const long long at = b * kv_stride + static_cast<long long>(s) * D + lane * E;
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(qv[e], __bfloat162float(K[at + e]), z);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float m2 = fmaxf(mx, z);
        const float f = m2 == -INFINITY ? 1.f : exp2f(mx - m2);
        const float p = m2 == -INFINITY ? 0.f : exp2f(z - m2);
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * __bfloat162float(V[at + e]);
        mx = m2;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) out[qrow + e] = __float2bfloat16(l > 0.f ? acc[e] / l : 0.f);
}

}  // namespace

extern "C" int ic_tree_attn(ic_ctx* ctx, const void* Q, const void* K, const void* V,
                            const int32_t* idx, const int32_t* prefix_len, const int32_t* draft_len,
                            const uint64_t* tree_mask, int B, int T, int Hq, int d, int k,
                            int64_t kv_seq_stride, int kv_len, float scale, void* out,
                            void* stream) {
    if (!ctx) return fail(nullptr, IC_ERR_INVALID_ARG, "context is NULL");
    if (B < 0 || T < 1 || Hq < 1 || Hq > 16 || kv_len < 1 || (idx ? (k < 1 || k > 2048) : k != 0))
        return fail(ctx, IC_ERR_SHAPE,
                    "tree_attn: B=%d T=%d Hq=%d kv_len=%d k=%d (k in [1,2048] with idx, else 0)", B,
                    T, Hq, kv_len, k);
    if (T > kMaxDrafts)
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree_attn: T=%d (at most %d)", T, kMaxDrafts);
    if (d != 64 && d != 128) return fail(ctx, IC_ERR_UNSUPPORTED, "tree_attn: d=%d", d);
    if (kv_len > (1 << 24))
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree_attn: kv_len=%d above 2^24", kv_len);
    if (kv_seq_stride % 8 != 0 || (B > 1 && kv_seq_stride < static_cast<int64_t>(kv_len) * d))
        return fail(ctx, IC_ERR_SHAPE, "tree_attn: kv_seq_stride=%lld", (long long)kv_seq_stride);
    if (static_cast<long long>(B) * T > (1 << 24))
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree_attn: B*T=%lld above 2^24",
                    static_cast<long long>(B) * T);
    if (B == 0) return IC_OK;
    if (!Q || !K || !V || !prefix_len || !out) return fail(ctx, IC_ERR_INVALID_ARG, "tree_attn: NULL");
    if (!aligned_to(Q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(out, 16))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree_attn: Q, K, V and out must be 16-byte aligned");
    if (!(scale > 0.f)) scale = 1.0f / sqrtf(static_cast<float>(d));
    DeviceGuard guard(ctx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const TreeArgs ta{prefix_len, draft_len, reinterpret_cast<const unsigned long long*>(tree_mask),
                      T, kv_len};
    auto* kern = d == 128 ? k_tree_attn<128> : k_tree_attn<64>;
    LaunchScope ls(ctx, IC_K_TREE_ATTN, s);
    kern<<<B * T, Hq * 32, 0, s>>>(
        static_cast<const __nv_bfloat16*>(Q), static_cast<const __nv_bfloat16*>(K),
        static_cast<const __nv_bfloat16*>(V), idx, ta, Hq, k, kv_seq_stride,
        scale * 1.4426950408889634f, static_cast<__nv_bfloat16*>(out), ctx->dev_err);
    cudaError_t e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "tree_attn launch");
    return IC_OK;
}
