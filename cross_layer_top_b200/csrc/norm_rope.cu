// Per-head norm, position rotation, quantisation and cache write, for all of
// a layer's projected tensors in one launch (ic_qk_norm_rope): the steps
// between the projections and the tensors the indexer and the attention
// take ("IndexCache：跨层复用稀疏索引，以及它为什么能被训练", the indexer's
// k_norm and rotation).
//
// Per head vector x of d values:
//   y = norm(x) * weight + bias;  z = rotation of y's first d_rot values;
//   bf16(z), or scale = max(max|z|, 1e-12)/448 and e4m3(z / scale).
// Every value is read once and written once, so HBM bytes bound it.
//
// Layout: d/8 lanes hold one vector, 8 values (16 bytes) each, so a warp
// holds G = 256/d vectors and every global access is 16 bytes per lane (8
// for e4m3 output).  The norm's and the scale's reductions are shuffles in
// those d/8 lanes; the half-split rotation takes its partner values from the
// lane d_rot/16 away, the interleaved one has them in the same lane.  A warp
// owns kIters * G consecutive vectors of one tensor (consecutive heads of a
// row, then the next row) and issues their loads before it uses the first.
// Sums, statistics and the rotation are fp32; the one rounding is the store.
#include "ic_device.cuh"
#include "ic_internal.h"

using namespace ic;

namespace {

constexpr int kWarps = 8;
constexpr int kIters = 4;

struct HeadDesc {
    const __nv_bfloat16* x;
    long long x_stride;
    const float* weight;
    const float* bias;
    const float* rope;
    void* out;  // bf16 or e4m3 bytes
    float* out_scale;  // e4m3 output when not null
    const long long* slot;
    long long out_rows;
    long long warp_begin;  // first warp of this tensor
    float eps;
    int H, d, norm, d_rot, interleaved;
};
struct HeadDescs {
    HeadDesc t[IC_MAX_HEAD_IO];
    int n;
};

// The vector of 8 values at lane position lg of a head of D values.
template <int D>
__device__ __forceinline__ void norm_rope_vectors(const HeadDesc& t, long long warp, int rows,
                                                  const int32_t* __restrict__ pos, int n_pos,
                                                  int* __restrict__ err) {
    constexpr int LG = D / 8;    // lanes per vector
    constexpr int G = 32 / LG;   // vectors per warp
    const int lane = threadIdx.x & 31, lg = lane % LG, g = lane / LG;
    const long long n_vec = static_cast<long long>(rows) * t.H;
    const long long v0 = warp * (G * kIters) + g;
    const int c0 = lg * 8;  // this lane's first value

    uint4 raw[kIters];
    int row[kIters], head[kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const long long v = v0 + i * G;
        row[i] = v < n_vec ? static_cast<int>(v / t.H) : -1;
        head[i] = static_cast<int>(v - static_cast<long long>(row[i]) * t.H);
        raw[i] = make_uint4(0, 0, 0, 0);
        if (row[i] >= 0)
            raw[i] = __ldg(reinterpret_cast<const uint4*>(t.x + row[i] * t.x_stride + head[i] * D + c0));
    }
    float wt[8], bs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        wt[e] = 1.f;
        bs[e] = 0.f;
    }
    if (t.weight) {
        *reinterpret_cast<float4*>(wt) = __ldg(reinterpret_cast<const float4*>(t.weight + c0));
        *reinterpret_cast<float4*>(wt + 4) = __ldg(reinterpret_cast<const float4*>(t.weight + c0 + 4));
    }
    if (t.bias) {
        *reinterpret_cast<float4*>(bs) = __ldg(reinterpret_cast<const float4*>(t.bias + c0));
        *reinterpret_cast<float4*>(bs + 4) = __ldg(reinterpret_cast<const float4*>(t.bias + c0 + 4));
    }
    const bool rotates = t.rope != nullptr;
    const int half = t.d_rot / 2;
    const bool in_rot = rotates && c0 < t.d_rot;
    const bool first = c0 < half;  // half-split: first or second value of the pairs
    // half-split partner lane; lanes past d_rot take their own values
    const int partner = !in_rot ? lane : (first ? lane + half / 8 : lane - half / 8);

#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const uint32_t w4[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] = __uint_as_float(w4[e] << 16);
            y[2 * e + 1] = __uint_as_float(w4[e] & 0xFFFF0000u);
        }
        if (t.norm != IC_NORM_NONE) {
            if (t.norm == IC_NORM_LAYER) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) s += y[e];
#pragma unroll
                for (int o = LG / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                s *= 1.f / D;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] -= s;
            }
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(y[e], y[e], q);
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
            const float r = 1.f / sqrtf(q * (1.f / D) + t.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e] * r, wt[e], bs[e]);
        }
        bool ok = row[i] >= 0;
        if (rotates) {
            const int p = ok ? __ldg(pos + row[i]) : 0;
            if (p < 0 || p >= n_pos) {
                if (ok && lg == 0) atomicCAS(err, 0, kDevBadPos);
                ok = false;
            }
            float c[8], s[8];
            if (ok && in_rot) {
                const float* tab = t.rope + static_cast<long long>(p) * t.d_rot;
                if (t.interleaved) {
                    const float4 cc = __ldg(reinterpret_cast<const float4*>(tab + c0 / 2));
                    const float4 ss = __ldg(reinterpret_cast<const float4*>(tab + half + c0 / 2));
                    c[0] = c[1] = cc.x, c[2] = c[3] = cc.y, c[4] = c[5] = cc.z, c[6] = c[7] = cc.w;
                    s[0] = s[1] = ss.x, s[2] = s[3] = ss.y, s[4] = s[5] = ss.z, s[6] = s[7] = ss.w;
                } else {
                    const int k = first ? c0 : c0 - half;
                    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(tab + k));
                    *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(tab + k + 4));
                    *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(tab + half + k));
                    *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(tab + half + k + 4));
                }
            }
            if (t.interleaved) {
                if (ok && in_rot)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float a = y[e], b = y[e + 1];
                        y[e] = a * c[e] - b * s[e];
                        y[e + 1] = b * c[e] + a * s[e];
                    }
            } else {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, y[e], partner);
                if (ok && in_rot)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = first ? y[e] * c[e] - o[e] * s[e] : y[e] * c[e] + o[e] * s[e];
            }
        }
        long long w = row[i];
        if (ok && t.slot) {
            w = __ldg(t.slot + row[i]);
            if (w < -1 || w >= t.out_rows) {
                if (lg == 0) atomicCAS(err, 0, kDevBadSlot);
                w = -1;
            }
            ok = w >= 0;
        }
        const long long at = (w * t.H + head[i]) * D + c0;
        if (t.out_scale == nullptr) {
            uint4 o;
            o.x = pack_bf16x2(y[0], y[1]);
            o.y = pack_bf16x2(y[2], y[3]);
            o.z = pack_bf16x2(y[4], y[5]);
            o.w = pack_bf16x2(y[6], y[7]);
            if (ok) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.out) + at) = o;
        } else {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, 1e-12f);
            const float scale = m / 448.f;
            // one division per vector: z * (1/scale) is within 1.5 fp32 ulps
            // of z / scale, 2^-19 of an e4m3 step (and saturates at 448)
            const float inv = 1.f / scale;
            uint2 o;
            o.x = e4m3x2_of(y[0] * inv, y[1] * inv) | e4m3x2_of(y[2] * inv, y[3] * inv) << 16;
            o.y = e4m3x2_of(y[4] * inv, y[5] * inv) | e4m3x2_of(y[6] * inv, y[7] * inv) << 16;
            if (ok) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.out) + at) = o;
                if (lg == 0) t.out_scale[w * t.H + head[i]] = scale;
            }
        }
    }
}

__global__ void __launch_bounds__(kWarps * 32)
    k_qk_norm_rope(const __grid_constant__ HeadDescs ds, int rows,
                   const int32_t* __restrict__ pos, int n_pos, int* __restrict__ err) {
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    int i = 0;
    while (i + 1 < ds.n && warp >= ds.t[i + 1].warp_begin) ++i;
    const HeadDesc& t = ds.t[i];
    const long long own = warp - t.warp_begin;
    if (t.d == 128)
        norm_rope_vectors<128>(t, own, rows, pos, n_pos, err);
    else if (t.d == 64)
        norm_rope_vectors<64>(t, own, rows, pos, n_pos, err);
    else
        norm_rope_vectors<32>(t, own, rows, pos, n_pos, err);
}

int check_head(ic_ctx* ctx, const ic_head_io& h, int i, int rows, const int32_t* pos, int n_pos) {
    if (!h.x || (!h.out && !h.out8))
        return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: tensor %d: NULL x or output", i);
    if ((h.out != nullptr) == (h.out8 != nullptr) || (h.out8 != nullptr) != (h.out_scale != nullptr))
        return fail(ctx, IC_ERR_INVALID_ARG,
                    "qk_norm_rope: tensor %d: give out, or out8 with out_scale", i);
    if (h.d != 32 && h.d != 64 && h.d != 128)
        return fail(ctx, IC_ERR_UNSUPPORTED, "qk_norm_rope: tensor %d: d=%d not in {32,64,128}", i,
                    h.d);
    if (h.H < 1 || h.H > 1024)
        return fail(ctx, IC_ERR_UNSUPPORTED, "qk_norm_rope: tensor %d: H=%d not in [1,1024]", i, h.H);
    if (h.x_stride < static_cast<int64_t>(h.H) * h.d || h.x_stride % 8 != 0)
        return fail(ctx, IC_ERR_SHAPE,
                    "qk_norm_rope: tensor %d: x_stride=%lld (need >= H*d, a multiple of 8)", i,
                    (long long)h.x_stride);
    if (!aligned_to(h.x, 16) || !aligned_to(h.out, 16) || !aligned_to(h.out8, 16) ||
        !aligned_to(h.weight, 16) || !aligned_to(h.bias, 16) || !aligned_to(h.rope, 16))
        return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: tensor %d: 16-byte alignment", i);
    if (h.norm != IC_NORM_NONE && h.norm != IC_NORM_RMS && h.norm != IC_NORM_LAYER)
        return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: tensor %d: norm=%d", i, h.norm);
    if (h.norm == IC_NORM_NONE ? (h.weight || h.bias) : (h.bias && h.norm != IC_NORM_LAYER))
        return fail(ctx, IC_ERR_INVALID_ARG,
                    "qk_norm_rope: tensor %d: weight needs a norm, bias the layer norm", i);
    if (h.norm != IC_NORM_NONE && !(h.eps > 0.f))
        return fail(ctx, IC_ERR_SHAPE, "qk_norm_rope: tensor %d: eps must be > 0", i);
    if (h.rope) {
        if (h.d_rot < 16 || h.d_rot > h.d || h.d_rot % 16 != 0)
            return fail(ctx, IC_ERR_UNSUPPORTED,
                        "qk_norm_rope: tensor %d: d_rot=%d (a multiple of 16, <= d)", i, h.d_rot);
        if (!pos || n_pos < 1)
            return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: tensor %d: rotation without pos", i);
    }
    if (h.out_rows < 0 || (!h.slot && h.out_rows < rows))
        return fail(ctx, IC_ERR_SHAPE, "qk_norm_rope: tensor %d: out_rows=%lld", i,
                    (long long)h.out_rows);
    return IC_OK;
}

}  // namespace

extern "C" int ic_qk_norm_rope(ic_ctx* ctx, const ic_head_io* heads, int n_heads, int rows,
                               const int32_t* pos, int n_pos, void* stream) {
    if (!ctx) return fail(nullptr, IC_ERR_INVALID_ARG, "context is NULL");
    if (!heads) return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: heads is NULL");
    if (n_heads < 1 || n_heads > IC_MAX_HEAD_IO || rows < 0 || rows > (1 << 24))
        return fail(ctx, IC_ERR_SHAPE, "qk_norm_rope: n_heads=%d (1..%d) rows=%d (0..2^24)", n_heads,
                    IC_MAX_HEAD_IO, rows);
    if (rows == 0) return IC_OK;  // nothing is read or written
    HeadDescs ds = {};
    long long warps = 0;
    for (int i = 0; i < n_heads; ++i) {
        const ic_head_io& h = heads[i];
        int rc = check_head(ctx, h, i, rows, pos, n_pos);
        if (rc) return rc;
        HeadDesc& t = ds.t[i];
        t.x = static_cast<const __nv_bfloat16*>(h.x);
        t.x_stride = h.x_stride;
        t.weight = h.weight;
        t.bias = h.bias;
        t.rope = h.rope;
        t.out = h.out8 ? static_cast<void*>(h.out8) : h.out;
        t.out_scale = h.out8 ? h.out_scale : nullptr;
        t.slot = reinterpret_cast<const long long*>(h.slot);
        t.out_rows = h.out_rows;
        t.eps = h.eps;
        t.H = h.H;
        t.d = h.d;
        t.norm = h.norm;
        t.d_rot = h.rope ? h.d_rot : 0;
        t.interleaved = h.interleaved != 0;
        t.warp_begin = warps;
        const long long per_warp = kIters * (256 / h.d);
        warps += (static_cast<long long>(rows) * h.H + per_warp - 1) / per_warp;
    }
    ds.n = n_heads;
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFFll) return fail(ctx, IC_ERR_SHAPE, "qk_norm_rope: too many heads");
    DeviceGuard guard(ctx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LaunchScope ls(ctx, IC_K_NORM_ROPE, s);
    k_qk_norm_rope<<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(ds, rows, pos, n_pos,
                                                                        ctx->dev_err);
    cudaError_t e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "qk_norm_rope launch");
    return IC_OK;
}
