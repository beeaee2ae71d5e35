// Lightning-indexer scores and selections of drafted tokens: T query tokens
// per sequence against the FP8 indexer-key cache, where query (b, t) sees
// the committed slots and its own ancestors among the drafts.
//   I[b,t,s] = scale[b,s] * sum_j w[b,t,j] * ReLU(q[b,t,j,:] . e4m3(k8[b,s,:]))
// which is the decode step's score ("IndexCache：跨层复用稀疏索引，以及它为什么
// 能被训练", §2.1) for every row of the tree; scale > 0 commutes with ReLU.
#include "ic_internal.h"
#include "tree.cuh"

using namespace ic;

namespace {

// ---- scores: a thread per key, its 128 values in registers, against every
// (token, head) query row of the sequence in shared memory
constexpr int kKeys = 128;

__global__ void __launch_bounds__(kKeys)
    k_index_score_tree(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ w,
                       const uint8_t* __restrict__ k8, const float* __restrict__ kscale,
                       TreeArgs ta, int S_max, int H_I, float* __restrict__ scores, long long ld,
                       int* __restrict__ err) {
    extern __shared__ float sq[];  // [H_I][128] of one token, then its weights
    float* sw = sq + H_I * 128;
    const int b = blockIdx.y, t = blockIdx.z;
    int n, m;
    if (!tree_lens(ta, b, n, m)) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && t == 0) atomicCAS(err, 0, kDevBadTree);
    }
    const int s = blockIdx.x * kKeys + threadIdx.x;
    if (t >= m || blockIdx.x * kKeys >= n + m) return;
    const long long row = static_cast<long long>(b) * ta.T + t;
    for (int i = threadIdx.x; i < H_I * 128; i += kKeys) sq[i] = __bfloat162float(q[row * H_I * 128 + i]);
    for (int i = threadIdx.x; i < H_I; i += kKeys) sw[i] = __bfloat162float(w[row * H_I + i]);
    __syncthreads();
    if (s >= n + m) return;
    const unsigned long long bits = tree_bits(ta, b, t, m);
    float* out = scores + row * ld + s;
    if (s >= n && !((bits >> (s - n)) & 1)) {
        *out = __int_as_float(0xff800000);
        return;
    }
    const long long key = static_cast<long long>(b) * S_max + s;
    float kv[128];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(k8 + key * 128) + c);
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 lo = float2_of_e4m3x2(w4[e] & 0xFFFFu), hi = float2_of_e4m3x2(w4[e] >> 16);
            kv[c * 16 + e * 4] = lo.x;
            kv[c * 16 + e * 4 + 1] = lo.y;
            kv[c * 16 + e * 4 + 2] = hi.x;
            kv[c * 16 + e * 4 + 3] = hi.y;
        }
    }
    float sum = 0.f;
    for (int h = 0; h < H_I; ++h) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 128; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sq + h * 128 + i);
            d = fmaf(x.x, kv[i], d);
            d = fmaf(x.y, kv[i + 1], d);
            d = fmaf(x.z, kv[i + 2], d);
            d = fmaf(x.w, kv[i + 3], d);
        }
        sum = fmaf(sw[h], fmaxf(d, 0.f), sum);
    }
    *out = sum * __ldg(kscale + key);
}

// ---- selections: each row's candidates for the top-k (0 for padding rows)
__global__ void k_tree_rows(TreeArgs ta, int rows, int32_t* __restrict__ row_len,
                            int* __restrict__ err) {
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= rows) return;
    int n, m;
    if (!tree_lens(ta, r / ta.T, n, m)) atomicCAS(err, 0, kDevBadTree);
    row_len[r] = r % ta.T < m ? n + m : 0;
}

// The drafts a row does not see carry -inf, so the top-k takes them only for
// want of others; they are taken out here.  Positions are ascending, so the
// drafts are among the last 64 of the row's min(k, n + m): one warp compacts
// those in place.
__global__ void k_tree_hide(TreeArgs ta, int rows, int k, int32_t* __restrict__ idx) {
    const int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= rows) return;
    int n, m;
    tree_lens(ta, r / ta.T, n, m);
    if (r % ta.T >= m) return;
    const unsigned long long bits = tree_bits(ta, r / ta.T, r % ta.T, m);
    const int have = min(k, n + m), first = max(0, have - kMaxDrafts);
    int32_t* row = idx + static_cast<long long>(r) * k;
    int v[2], kept = first;
    bool keep[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = first + 32 * i + lane;
        v[i] = at < have ? row[at] : -1;
        keep[i] = v[i] >= 0 && (v[i] < n || ((bits >> (v[i] - n)) & 1));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned ball = __ballot_sync(0xffffffffu, keep[i]);
        if (keep[i]) row[kept + __popc(ball & ((1u << lane) - 1u))] = v[i];
        kept += __popc(ball);
    }
    for (int at = kept + lane; at < have; at += 32) row[at] = -1;
}

int check_args(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8, const float* kI_scale,
               const int32_t* prefix_len, int B, int T, int S_max, int H_I, int d_I) {
    if (!ctx) return fail(nullptr, IC_ERR_INVALID_ARG, "context is NULL");
    if (!q || !w || !kI8 || !kI_scale || !prefix_len)
        return fail(ctx, IC_ERR_INVALID_ARG, "tree index: NULL input");
    if (!aligned_to(q, 16) || !aligned_to(kI8, 16))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree index: q and kI8 must be 16-byte aligned");
    if (B <= 0 || T <= 0 || S_max <= 0)
        return fail(ctx, IC_ERR_SHAPE, "tree index: B=%d T=%d S_max=%d", B, T, S_max);
    if (T > kMaxDrafts)
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree index: T=%d (at most %d)", T, kMaxDrafts);
    if ((H_I != 32 && H_I != 64) || d_I != 128)
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree index: H_I=%d d_I=%d (need {32,64}, 128)", H_I,
                    d_I);
    if (static_cast<long long>(B) * S_max > 0x7FFFF000ll || B > 65535)
        return fail(ctx, IC_ERR_SHAPE, "tree index: B=%d, B*S_max=%lld too large", B,
                    static_cast<long long>(B) * S_max);
    return IC_OK;
}

int launch_index_score_tree(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8,
                            const float* kI_scale, const TreeArgs& ta, int B, int H_I,
                            float* scores, int64_t ld, cudaStream_t s) {
    const dim3 grid((ta.cap + kKeys - 1) / kKeys, B, ta.T);
    const int smem = H_I * 129 * 4;
    LaunchScope ls(ctx, IC_K_INDEX_SCORE_TREE, s);
    k_index_score_tree<<<grid, kKeys, smem, s>>>(
        static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(w), kI8, kI_scale,
        ta, ta.cap, H_I, scores, static_cast<long long>(ld), ctx->dev_err);
    cudaError_t e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "index_score_tree launch");
    return IC_OK;
}

}  // namespace

extern "C" int ic_index_score_tree(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8,
                                   const float* kI_scale, const int32_t* prefix_len,
                                   const int32_t* draft_len, const uint64_t* tree_mask, int B,
                                   int T, int S_max, int H_I, int d_I, float* scores, int64_t ld,
                                   void* stream) {
    int rc = check_args(ctx, q, w, kI8, kI_scale, prefix_len, B, T, S_max, H_I, d_I);
    if (rc) return rc;
    if (!scores || !aligned_to(scores, 16))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree index: scores NULL or not 16-byte aligned");
    if (ld < S_max || ld % 4 != 0)
        return fail(ctx, IC_ERR_SHAPE, "tree index: ld=%lld (>= S_max, a multiple of 4)",
                    (long long)ld);
    DeviceGuard guard(ctx);
    const TreeArgs ta{prefix_len, draft_len, reinterpret_cast<const unsigned long long*>(tree_mask),
                      T, S_max};
    return launch_index_score_tree(ctx, q, w, kI8, kI_scale, ta, B, H_I, scores, ld,
                                   reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int ic_index_fp_tree(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8,
                                const float* kI_scale, const int32_t* prefix_len,
                                const int32_t* draft_len, const uint64_t* tree_mask, int B, int T,
                                int S_max, int H_I, int d_I, int k, int32_t* idx_out,
                                void* stream) {
    int rc = check_args(ctx, q, w, kI8, kI_scale, prefix_len, B, T, S_max, H_I, d_I);
    if (rc) return rc;
    if (!idx_out) return fail(ctx, IC_ERR_INVALID_ARG, "tree index: idx_out is NULL");
    if (k < 1 || k > 2048) return fail(ctx, IC_ERR_SHAPE, "tree index: k=%d not in [1,2048]", k);
    DeviceGuard guard(ctx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // fp32 score rows of a chunk of sequences, then their lengths
    const int64_t ld = (static_cast<int64_t>(S_max) + 63) / 64 * 64;
    const size_t per_seq = static_cast<size_t>(T) * (ld + 1) * 4;
    int64_t chunk = static_cast<int64_t>(ctx->scratch_limit / per_seq);
    if (chunk < 1)
        return fail(ctx, IC_ERR_NOMEM, "tree index: one sequence's scores need %zu bytes of scratch",
                    per_seq);
    if (chunk > B) chunk = B;
    rc = ensure_buffer(ctx, reinterpret_cast<void**>(&ctx->scores), &ctx->scores_cap,
                       chunk * per_seq);
    if (rc) return rc;
    for (int b0 = 0; b0 < B; b0 += static_cast<int>(chunk)) {
        const int nb = static_cast<int>(b0 + chunk < B ? chunk : B - b0), rows = nb * T;
        const long long r0 = static_cast<long long>(b0) * T;
        int32_t* row_len = reinterpret_cast<int32_t*>(ctx->scores + static_cast<int64_t>(rows) * ld);
        const TreeArgs ta{prefix_len + b0, draft_len ? draft_len + b0 : nullptr,
                          tree_mask ? reinterpret_cast<const unsigned long long*>(tree_mask) + r0
                                    : nullptr,
                          T, S_max};
        rc = launch_index_score_tree(
            ctx, static_cast<const __nv_bfloat16*>(q) + r0 * H_I * d_I,
            static_cast<const __nv_bfloat16*>(w) + r0 * H_I,
            kI8 + static_cast<long long>(b0) * S_max * d_I,
            kI_scale + static_cast<long long>(b0) * S_max, ta, nb, H_I, ctx->scores, ld, s);
        if (rc) return rc;
        {
            LaunchScope ls(ctx, IC_K_INDEX_SCORE_TREE, s);
            k_tree_rows<<<(rows + 255) / 256, 256, 0, s>>>(ta, rows, row_len, ctx->dev_err);
            cudaError_t e = ls.done();
            if (e != cudaSuccess) return cuda_fail(ctx, e, "tree_rows launch");
        }
        rc = launch_topk(ctx, ctx->scores, ld, rows, k, 0, row_len, S_max, idx_out + r0 * k, k, s);
        if (rc) return rc;
        LaunchScope ls(ctx, IC_K_TOPK, s);
        k_tree_hide<<<(rows + 7) / 8, 256, 0, s>>>(ta, rows, k, idx_out + r0 * k);
        cudaError_t e = ls.done();
        if (e != cudaSuccess) return cuda_fail(ctx, e, "tree_hide launch");
    }
    return IC_OK;
}
