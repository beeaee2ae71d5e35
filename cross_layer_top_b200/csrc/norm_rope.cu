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
// Layout: d/8 lanes hold one vector, 8 values each, so a warp holds G = 256/d
// vectors at once.  A lane's values are two runs of four chosen so that both
// values of every rotated pair are its own: runs 4 l.. of the two halves of
// the rotated part, or of the rest (lane l of those the part takes), and for
// the interleaved rotation 8 l .. 8 l + 7; only the norm's and the scale's
// reductions cross lanes, and every access of a warp covers whole 32-byte
// sectors.  A warp takes kIters * G consecutive vectors of one tensor
// (consecutive heads of a row, then the next row) at a time, loads them all
// and then does each step for all of them, so that the steps' latencies
// overlap.  Where the heads of a row are a multiple of kIters * G, it takes
// up to kChunks such chunks of the row: the next chunk's loads are under way
// while one is worked on, and the row's position, table values and output row
// are looked up once.
// Sums, statistics and the rotation are fp32; the one rounding is the store.
// Measured (B200): 16384 rows of 16 + 2 heads as bf16 and 64 + 1 as e4m3, all
// of 128 values (577 MB), 107 us = 5.4 TB/s, 0.83 of a plain copy's rate, each
// call with cold inputs; 99 us in a loop over one input.  64 rows of the same
// tensors: 4.9 us in a graph, launch and one round trip, and 8.2 us a
// call from Python.
#include "ic_device.cuh"
#include "ic_internal.h"

using namespace ic;

namespace {

// Blocks of one warp: nothing is shared, and a block's place is free as soon
// as its one warp is done (at 16384 rows 3 blocks of 8 warps took 115 us, 4 of
// 5 106, 22 of one 99).  22 leave 88 registers a thread: the kernel spills a
// little with fewer and hides less latency with more.
constexpr int kBlocksPerSm = 22;
constexpr int kIters = 4;   // vectors of a lane at a time
constexpr int kChunks = 4;  // chunks of a row a warp takes, at most

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
    int warp_begin;  // first warp of this tensor
    float eps;
    int H, d, norm, d_rot, interleaved;
    int chunks;  // of one row per warp; 0: vectors of any rows
    uint32_t ahead;  // warps from one to the one whose values it prefetches
    uint32_t magic, shift;  // v / H for v < 2^31 (magic 0: H = 1)
};
struct HeadDescs {
    HeadDesc t[IC_MAX_HEAD_IO];
    int n;
};

// The rotation of a lane's values with four cosines and sines: pairs
// (v[e], v[e + 4]), or (v[2 e], v[2 e + 1]).
__device__ __forceinline__ void rotate_halves(float (&v)[8], const float4& cs, const float4& sn) {
    const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = v[e], b = v[e + 4];
        v[e] = fmaf(a, c[e], -(b * s[e]));
        v[e + 4] = fmaf(b, c[e], a * s[e]);
    }
}
__device__ __forceinline__ void rotate_pairs(float (&v)[8], const float4& cs, const float4& sn) {
    const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = v[2 * e], b = v[2 * e + 1];
        v[2 * e] = fmaf(a, c[e], -(b * s[e]));
        v[2 * e + 1] = fmaf(b, c[e], a * s[e]);
    }
}

// A warp's vectors of one tensor: kIters * G, or with ONE_ROW t.chunks times
// as many of one row.
template <int D, bool ONE_ROW>
__device__ __forceinline__ void norm_rope_vectors(const HeadDesc& t, uint32_t warp, int rows,
                                                  const int32_t* __restrict__ pos, int n_pos,
                                                  int* __restrict__ err) {
    constexpr int LG = D / 8;    // lanes per vector
    constexpr int G = 32 / LG;   // vectors per warp
    constexpr int CHUNK = G * kIters;
    const int lane = threadIdx.x & 31, lg = lane % LG, g = lane / LG;
    const int H = t.H, d_rot = t.d_rot, norm = t.norm;
    const uint32_t magic = t.magic, shift = t.shift;
    const uint32_t n_vec = static_cast<uint32_t>(rows) * H;
    const int chunks = ONE_ROW ? t.chunks : 1;
    const uint32_t v0 = warp * (CHUNK * chunks) + g;
    const bool rot = lg * 8 < d_rot, pairs = t.interleaved;  // pairs: (2 i, 2 i + 1)
    // this lane's two runs of four values
    const int ca = pairs ? 8 * lg : rot ? 4 * lg : d_rot / 2 + 4 * lg;
    const int cb = pairs ? ca + 4 : ca + (rot ? d_rot : D - d_rot) / 2;
    auto load = [&](const __nv_bfloat16* x, uint2& a, uint2& b) {
        if (pairs) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(x + ca));
            a = make_uint2(v.x, v.y);
            b = make_uint2(v.z, v.w);
        } else {
            a = __ldcs(reinterpret_cast<const uint2*>(x + ca));
            b = __ldcs(reinterpret_cast<const uint2*>(x + cb));
        }
    };

    auto row_of = [&](uint32_t v) { return magic ? __umulhi(v, magic) >> shift : v; };
    const uint32_t row0 = row_of(v0), head0 = v0 - row0 * H;
    if (ONE_ROW && v0 >= n_vec) return;  // the same for the whole warp
    uint2 ra[kIters], rb[kIters];
    const __nv_bfloat16* x = t.x + row0 * t.x_stride + head0 * D;
    if (ONE_ROW) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) load(x + i * G * D, ra[i], rb[i]);
        // the values of a warp that starts a quarter of the resident warps
        // later go to L2 meanwhile (125 -> 118 us at 16384 rows)
        const uint32_t later = v0 + t.ahead * (CHUNK * chunks);
        if (lane == 0 && later < n_vec) {
            const uint32_t r = row_of(later);
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             t.x + r * t.x_stride + (later - r * H) * D),
                         "r"(CHUNK * chunks * D * 2));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const uint32_t v = v0 + i * G, r = row_of(v);
            ra[i] = rb[i] = make_uint2(0, 0);
            if (v < n_vec) {
                load(t.x + r * t.x_stride + (v - r * H) * D, ra[i], rb[i]);
            }
        }
    }
    // a row's table values, and the output row (-1: nothing to write)
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = cs;
    auto look_up = [&](uint32_t r) {
        long long to = r;
        if (d_rot) {
            const int p = __ldg(pos + r);
            if (p < 0 || p >= n_pos) {
                if (lg == 0) atomicCAS(err, 0, kDevBadPos);
                to = -1;
            } else if (rot) {
                const float* tab = t.rope + static_cast<long long>(p) * d_rot + 4 * lg;
                cs = __ldg(reinterpret_cast<const float4*>(tab));
                sn = __ldg(reinterpret_cast<const float4*>(tab + d_rot / 2));
            }
        }
        if (to >= 0 && t.slot) {
            const long long w = __ldg(t.slot + r);
            if (w < -1 || w >= t.out_rows) {
                if (lg == 0) atomicCAS(err, 0, kDevBadSlot);
                to = -1;
            } else {
                to = w;
            }
        }
        return to;
    };
    long long vec0 = 0;  // ONE_ROW: output vector of this lane's first
    if (ONE_ROW) {
        const long long to = look_up(row0);
        if (to < 0) return;  // the same for the whole warp
        vec0 = to * H + head0;
    }

#pragma unroll 1
    for (int j = 0; j < chunks; ++j) {
        // values: run a, then run b
        float y[kIters][8];
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const uint32_t w[4] = {ra[i].x, ra[i].y, rb[i].x, rb[i].y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][2 * e] = __uint_as_float(w[e] << 16);
                y[i][2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
        if (ONE_ROW && j + 1 < chunks) {
            x += CHUNK * D;
#pragma unroll
            for (int i = 0; i < kIters; ++i) load(x + i * G * D, ra[i], rb[i]);
        }
        // sums of all vectors over their lanes, together
        auto sum_lanes = [&](float (&v)[kIters]) {
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < kIters; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        };
        if (norm != IC_NORM_NONE) {
            float q[kIters];
            if (norm == IC_NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < kIters; ++i)
                    q[i] = ((y[i][0] + y[i][1]) + (y[i][2] + y[i][3])) + ((y[i][4] + y[i][5]) + (y[i][6] + y[i][7]));
                sum_lanes(q);
#pragma unroll
                for (int i = 0; i < kIters; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] -= q[i] * (1.f / D);
            }
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s0 = fmaf(y[i][e], y[i][e], s0);
                    s1 = fmaf(y[i][e + 4], y[i][e + 4], s1);
                }
                q[i] = s0 + s1;
            }
            sum_lanes(q);
            float w[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = 1.f;
                b[e] = 0.f;
            }
            if (t.weight) {
                *reinterpret_cast<float4*>(w) = __ldg(reinterpret_cast<const float4*>(t.weight + ca));
                *reinterpret_cast<float4*>(w + 4) = __ldg(reinterpret_cast<const float4*>(t.weight + cb));
            }
            if (t.bias) {
                *reinterpret_cast<float4*>(b) = __ldg(reinterpret_cast<const float4*>(t.bias + ca));
                *reinterpret_cast<float4*>(b + 4) = __ldg(reinterpret_cast<const float4*>(t.bias + cb));
            }
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                const float r = rsqrtf(q[i] * (1.f / D) + t.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = fmaf(y[i][e] * r, w[e], b[e]);
            }
        }
        // rotation, and where each vector goes (-1: nowhere)
        long long vec[kIters];
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            if (ONE_ROW) {
                vec[i] = vec0 + j * CHUNK + i * G;
            } else {
                const uint32_t v = v0 + i * G, r = row_of(v);
                const long long to = v < n_vec ? look_up(r) : -1;
                vec[i] = to < 0 ? -1 : to * H + (v - r * H);
            }
            if (rot) {
                if (pairs)
                    rotate_pairs(y[i], cs, sn);
                else
                    rotate_halves(y[i], cs, sn);
            }
        }
        // many-headed tensors are written once and read much later: their lines
        // are the first to leave L2 (118 -> 115 us at 16384 rows)
        auto put = [](auto* to, auto v) {
            if (ONE_ROW)
                __stcs(reinterpret_cast<decltype(v)*>(to), v);
            else
                *reinterpret_cast<decltype(v)*>(to) = v;
        };
        if (t.out_scale == nullptr) {
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out) + vec[i] * D;
                if (ONE_ROW || vec[i] >= 0) {
                    put(o + ca, make_uint2(pack_bf16x2(y[i][0], y[i][1]), pack_bf16x2(y[i][2], y[i][3])));
                    put(o + cb, make_uint2(pack_bf16x2(y[i][4], y[i][5]), pack_bf16x2(y[i][6], y[i][7])));
                }
            }
        } else {
            float m[kIters];
#pragma unroll
            for (int i = 0; i < kIters; ++i)
                m[i] = fmaxf(fmaxf(fmaxf(fabsf(y[i][0]), fabsf(y[i][1])), fmaxf(fabsf(y[i][2]), fabsf(y[i][3]))),
                             fmaxf(fmaxf(fabsf(y[i][4]), fabsf(y[i][5])), fmaxf(fabsf(y[i][6]), fabsf(y[i][7]))));
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < kIters; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                const float scale = fmaxf(m[i], 1e-12f) * (1.f / 448.f);
                // one reciprocal per vector (the scale is normal and so is it):
                // z * (1/scale) is within 2 fp32 ulps of z / scale, 2^-19 of an
                // e4m3 step, and saturates at 448
                float inv;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
                uint8_t* o = static_cast<uint8_t*>(t.out) + vec[i] * D;
                if (ONE_ROW || vec[i] >= 0) {
                    put(o + ca, e4m3x2_of(y[i][0] * inv, y[i][1] * inv) |
                                    e4m3x2_of(y[i][2] * inv, y[i][3] * inv) << 16);
                    put(o + cb, e4m3x2_of(y[i][4] * inv, y[i][5] * inv) |
                                    e4m3x2_of(y[i][6] * inv, y[i][7] * inv) << 16);
                    if (lg == 0) t.out_scale[vec[i]] = scale;
                }
            }
        }
    }
}

template <int D>
__device__ __forceinline__ void norm_rope_tensor(const HeadDesc& t, uint32_t warp, int rows,
                                                 const int32_t* pos, int n_pos, int* err) {
    if (t.chunks)
        norm_rope_vectors<D, true>(t, warp, rows, pos, n_pos, err);
    else
        norm_rope_vectors<D, false>(t, warp, rows, pos, n_pos, err);
}

__global__ void __launch_bounds__(32, kBlocksPerSm)
    k_qk_norm_rope(const __grid_constant__ HeadDescs ds, int rows,
                   const int32_t* __restrict__ pos, int n_pos, int* __restrict__ err) {
    const int warp = blockIdx.x;
    int i = 0;
    while (i + 1 < ds.n && warp >= ds.t[i + 1].warp_begin) ++i;
    const HeadDesc& t = ds.t[i];
    const uint32_t own = warp - t.warp_begin;
    if (t.d == 128)
        norm_rope_tensor<128>(t, own, rows, pos, n_pos, err);
    else if (t.d == 64)
        norm_rope_tensor<64>(t, own, rows, pos, n_pos, err);
    else
        norm_rope_tensor<32>(t, own, rows, pos, n_pos, err);
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

// Outputs (values, scales) share no byte with anything the call reads, nor
// with each other unless the slots of two tensors say which rows are whose:
// then rows of one size, on one grid of rows.
int check_overlap(ic_ctx* ctx, const ic_head_io* heads, int n, int rows, const int32_t* pos,
                  int n_pos) {
    struct Out {
        Span span;
        long long row;  // bytes
        int tensor;
    };
    Span in[5 * IC_MAX_HEAD_IO + 1];
    Out out[2 * IC_MAX_HEAD_IO];
    int n_in = 0, n_out = 0;
    if (pos) in[n_in++] = Span(pos, rows * 4ll);
    for (int i = 0; i < n; ++i) {
        const ic_head_io& h = heads[i];
        const long long row = static_cast<long long>(h.H) * h.d;
        in[n_in++] = Span(h.x, ((rows - 1ll) * h.x_stride + row) * 2);
        if (h.weight) in[n_in++] = Span(h.weight, h.d * 4);
        if (h.bias) in[n_in++] = Span(h.bias, h.d * 4);
        if (h.rope) in[n_in++] = Span(h.rope, static_cast<long long>(n_pos) * h.d_rot * 4);
        if (h.slot) in[n_in++] = Span(h.slot, rows * 8ll);
        const long long bytes = row * (h.out8 ? 1 : 2);
        out[n_out++] = Out{Span(h.out8 ? static_cast<void*>(h.out8) : h.out, h.out_rows * bytes), bytes, i};
        if (h.out8) out[n_out++] = Out{Span(h.out_scale, h.out_rows * h.H * 4), h.H * 4ll, i};
    }
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (out[o].span.meets(in[i]))
                return fail(ctx, IC_ERR_INVALID_ARG,
                            "qk_norm_rope: an output of tensor %d overlaps what the call reads",
                            out[o].tensor);
        for (int i = 0; i < o; ++i) {
            if (!out[o].span.meets(out[i].span)) continue;
            const bool by_slot = heads[out[o].tensor].slot && heads[out[i].tensor].slot &&
                                 out[o].tensor != out[i].tensor && out[o].row == out[i].row;
            const long long apart = static_cast<long long>(out[o].span.a - out[i].span.a);
            if (!by_slot || apart % out[o].row != 0)
                return fail(ctx, IC_ERR_INVALID_ARG, "qk_norm_rope: outputs of tensors %d and %d overlap",
                            out[i].tensor, out[o].tensor);
        }
    }
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
        t.warp_begin = static_cast<int>(warps);
        if (static_cast<long long>(rows) * h.H > 0x7FFF0000ll)
            return fail(ctx, IC_ERR_UNSUPPORTED, "qk_norm_rope: tensor %d: rows*H=%lld above 2^31", i,
                        static_cast<long long>(rows) * h.H);
        if (h.H > 1) {
            // v / H = (v * magic) >> (31 + l) exactly for v < 2^31, with
            // 2^(l-1) < H <= 2^l and magic = floor(2^(31+l) / H) + 1
            int l = 1;
            while ((1 << l) < h.H) ++l;
            t.magic = static_cast<uint32_t>((1ull << (31 + l)) / h.H + 1);
            t.shift = l - 1;
        }
        // whole chunks of a row where its heads allow it: as many per warp as
        // divide the row evenly
        const int chunk = kIters * (256 / h.d);
        t.ahead = ctx->num_sms * kBlocksPerSm / 4;
        t.chunks = 0;
        for (int c = kChunks; c >= 1 && !t.chunks; c /= 2)
            if (h.H % (chunk * c) == 0) t.chunks = c;
        const long long per_warp = static_cast<long long>(chunk) * (t.chunks ? t.chunks : 1);
        warps += (static_cast<long long>(rows) * h.H + per_warp - 1) / per_warp;
    }
    ds.n = n_heads;
    if (warps > 0x7FFFFF00ll) return fail(ctx, IC_ERR_UNSUPPORTED, "qk_norm_rope: too many heads");
    int rc = check_overlap(ctx, heads, n_heads, rows, pos, n_pos);
    if (rc) return rc;
    DeviceGuard guard(ctx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LaunchScope ls(ctx, IC_K_NORM_ROPE, s);
    k_qk_norm_rope<<<static_cast<unsigned>(warps), 32, 0, s>>>(ds, rows, pos, n_pos,
                                                                        ctx->dev_err);
    cudaError_t e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "qk_norm_rope launch");
    return IC_OK;
}
