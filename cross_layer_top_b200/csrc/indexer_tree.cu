// Lightning-indexer scores and selections of drafted tokens: T query tokens
// per sequence against the FP8 indexer-key cache, where query (b, t) sees
// the committed slots and its own ancestors among the drafts.
//   I[b,t,s] = scale[b,s] * sum_j w[b,t,j] * ReLU(q[b,t,j,:] . e4m3(k8[b,s,:]))
// which is the decode step's score ("IndexCache：跨层复用稀疏索引，以及它为什么
// 能被训练", §2.1) for every row of the tree; scale > 0 commutes with ReLU.
//
// Design (sm_100a).  A key is read from HBM once for all T tokens of its
// sequence, so the contraction (2 H_I d_I operations per token and key) is
// what bounds it from T = 3 on; below that, HBM.  "Keys as M": A = a tile of
// 128 keys, B = the (token, head) rows of a group of up to COLS columns, D =
// per-head dot products in TMEM, lane = key.  The thread that owns a key
// sums ReLU(.) w over the heads in its own registers.
//  * Queries stay bf16 and keys are exact in bf16, so the products are exact
//    and kind::f16 runs at the full bf16 rate on the queries as given; e4m3
//    operands would need the queries in two terms, the same tensor time and
//    twice the accumulator columns to read.  The keys are widened in shared
//    memory by four warps: e4m3's 7 magnitude bits shifted into a bf16's
//    exponent and mantissa are the value times 2^-120 (subnormals included),
//    and one packed multiplication by 2^120 makes it exact.
//  * Warp roles (one CTA per SM): 0 TMA (raw key tiles, query groups), 1 MMA,
//    2 TMEM, 3 finds the CTA's range of the work line, 4..7 widen, 8..15
//    epilogue (lane quarter warp % 4, token half (warp - 8) / 4).
//  * Up to 256 columns are one accumulator; two ping-pong, over the halves of
//    a 512-column group or over successive tiles.
// Work split: as tree.cuh says; a (sequence, token group, key tile) is an
// item and no two need joining.  Every wait is bounded.
#include "ic_internal.h"
#include "tree.cuh"

using namespace ic;

namespace {

template <int H_I, int COLS>
struct ScoreShape {
    static constexpr int TG = COLS / H_I;         // tokens per group
    static constexpr int JOBS = COLS / 256;       // accumulators per tile, at most
    static constexpr int JT = 256 / H_I;          // tokens per accumulator
    static constexpr int KT = kLineTile;          // keys per tile
    static constexpr int RAW = KT * 128;          // e4m3 tile
    static constexpr int ATOM = KT * 128;         // 64 bf16 columns of a key tile
    static constexpr int WIDE = 2 * ATOM;         // bf16 tile
    static constexpr int B_ATOM = 256 * 128;      // 64 columns of 256 query rows
    static constexpr int B_JOB = 2 * B_ATOM;
    static constexpr int NRAW = COLS == 512 ? 2 : 4;
    static constexpr int NWIDE = COLS == 512 ? 2 : 3;
    static constexpr int OFF_RAW = JOBS * B_JOB;
    static constexpr int OFF_WIDE = OFF_RAW + NRAW * RAW;
    static constexpr int OFF_W = OFF_WIDE + NWIDE * WIDE;
    static constexpr int OFF_BAR = OFF_W + COLS * 4;
    static constexpr int SMEM = OFF_BAR + 512;
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct ScoreArgs {
    TreeLine line;
    const __nv_bfloat16* w;
    const float* kscale;
    float* scores;
    int* err;
    long long ld;
    int B, S_max;
};

// Two e4m3 values (the two bytes of v that `sel` moves to the tops of the
// halves) as bf16; the NaN encodings read as +-480.
__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t v, uint32_t sel) {
    const uint32_t x = __byte_perm(v, 0u, sel);
    const uint32_t y = ((x & 0x7F007F00u) >> 4) | (x & 0x80008000u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7B807B80u));  // 2^120
    return r;
}

template <int H_I, int COLS>
__global__ void __launch_bounds__(512, 1)
    k_index_score_tree(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ ScoreArgs a) {
    using S = ScoreShape<H_I, COLS>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sB = smem;
    uint8_t* sRaw = smem + S::OFF_RAW;
    uint8_t* sWide = smem + S::OFF_WIDE;
    float* sW = reinterpret_cast<float*>(smem + S::OFF_W);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);  // [NRAW] TMA
    uint64_t* raw_empty = raw_full + S::NRAW;    // [NRAW] 4 widening warps
    uint64_t* wide_full = raw_empty + S::NRAW;   // [NWIDE] 4 widening warps
    uint64_t* wide_empty = wide_full + S::NWIDE; // [NWIDE] MMA commit
    uint64_t* q_full = wide_empty + S::NWIDE;
    uint64_t* q_empty = q_full + 1;
    uint64_t* acc_full = q_empty + 1;            // [2]
    uint64_t* acc_empty = acc_full + 2;          // [2] 8 epilogue warps
    uint64_t* w_full = acc_empty + 2;            // weights of a part written (8 warps)
    uint64_t* w_empty = w_full + 1;              // .. no longer read (8 warps)
    uint64_t* done_bar = w_empty + 1;
    LineRange* s_range = reinterpret_cast<LineRange*>(done_bar + 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_range + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* err = a.err;
    const int T = a.line.ta.T;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        if (smem_u32(smem) & 1023u) {
            *abort_flag = 1;
            atomicCAS(err, 0, kDevSmemMisaligned);
        }
        for (int i = 0; i < S::NRAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < S::NWIDE; ++i) {
            mbar_init(&wide_full[i], 4);
            mbar_init(&wide_empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 8);
        }
        mbar_init(w_full, 8);
        mbar_init(w_empty, 8);
        mbar_init(done_bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == 3) {
        const LineRange r = line_range(a.line, a.B, blockIdx.x, gridDim.x);
        if (lane == 0) *s_range = r;
        // lengths out of range are reported by the first CTA
        if (blockIdx.x == 0)
            for (int b = lane; b < a.B; b += 32) {
                int n, m;
                if (!tree_lens(a.line.ta, b, n, m)) atomicCAS(err, 0, kDevBadTree);
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool start_ok = (*abort_flag == 0);
    PartWalk walk(*s_range);
    // a part's tokens: groups of equal size, halved over two accumulators
    // where one does not hold them
    struct Tokens {
        int t0, n, jobs, first;  // first: tokens of the first accumulator
    };
    auto tokens = [&](const Part& p) {
        Tokens k;
        const int size = (p.w.m + p.w.groups - 1) / p.w.groups;
        k.t0 = p.group * size;
        k.n = max(0, min(size, p.w.m - k.t0));
        k.jobs = k.n > S::JT ? 2 : 1;
        k.first = (k.n + k.jobs - 1) / k.jobs;
        return k;
    };

    if (warp == 0 && lane == 0 && start_ok) {
        // ------------------------------------------------ TMA
        uint32_t it = 0, q_it = 0;
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const Tokens k = tokens(p);
            for (int t = p.t0; t < p.t1; ++t, ++it) {
                const uint32_t st = it % S::NRAW;
                if (!mbar_wait(&raw_empty[st], ((it / S::NRAW) & 1) ^ 1, abort_flag, err,
                               kDevTimeoutProducer)) {
                    ok = false;
                    break;
                }
                // keys past the sequence's last are read (zeros past the
                // cache's end) and their scores never stored
                mbar_arrive_expect_tx(&raw_full[st], S::RAW);
                tma_load_2d(sRaw + st * S::RAW, &tm_k, &raw_full[st], 0, p.b * a.S_max + t * S::KT);
                if (t != p.t0) continue;
                if (!mbar_wait(q_empty, (q_it & 1) ^ 1, abort_flag, err, kDevTimeoutProducer)) {
                    ok = false;
                    ++it;
                    break;
                }
                mbar_arrive_expect_tx(q_full, k.jobs * S::B_JOB);
                for (int j = 0; j < k.jobs; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_2d(sB + j * S::B_JOB + c * S::B_ATOM, &tm_q, q_full, c * 64,
                                    (p.b * T + k.t0 + j * k.first) * H_I);
                ++q_it;
            }
        }
        // no copy may still be landing at exit
        for (uint32_t i = it > S::NRAW ? it - S::NRAW : 0; i < it; ++i)
            mbar_wait_drain(&raw_full[i % S::NRAW], (i / S::NRAW) & 1);
        if (q_it > 0) mbar_wait_drain(q_full, (q_it - 1) & 1);
    } else if (warp == 1 && lane == 0 && start_ok) {
        // ------------------------------------------------ MMA issuer
        uint32_t it = 0, q_it = 0, job = 0;
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const Tokens k = tokens(p);
            if (!mbar_wait(q_full, q_it & 1, abort_flag, err, kDevTimeoutMma)) break;
            ++q_it;
            for (int t = p.t0; t < p.t1 && ok; ++t, ++it) {
                const uint32_t st = it % S::NWIDE;
                if (!mbar_wait(&wide_full[st], (it / S::NWIDE) & 1, abort_flag, err, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                const uint32_t k0 = smem_u32(sWide + st * S::WIDE);
                for (int j = 0; j < k.jobs; ++j, ++job) {
                    const uint32_t acc = job & 1;
                    if (!mbar_wait(&acc_empty[acc], ((job >> 1) & 1) ^ 1, abort_flag, err,
                                   kDevTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int cols = (j == 0 ? k.first : k.n - k.first) * H_I;
                    const uint32_t id = idesc_bf16_f32(S::KT, cols);
                    const uint32_t q0 = smem_u32(sB + j * S::B_JOB);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tmem + acc * 256, sdesc_k_sw128(k0 + c * S::ATOM + kk * 32),
                                      sdesc_k_sw128(q0 + c * S::B_ATOM + kk * 32), id,
                                      (c | kk) ? 1u : 0u);
                    umma_commit(&acc_full[acc]);
                }
                if (!ok) break;
                umma_commit(&wide_empty[st]);
            }
            if (ok) umma_commit(q_empty);
        }
        umma_commit(done_bar);
        if (!mbar_wait_drain(done_bar, 0)) atomicCAS(err, 0, kDevTimeoutDrain);
    } else if (warp >= 4 && warp < 8 && start_ok) {
        // ------------------------------------------------ widening
        const int id = threadIdx.x - 128;  // 16-byte piece id % 8 of key rows id / 8 + 16 i
        uint32_t it = 0;
        const uint32_t total = static_cast<uint32_t>(walk.g_end - walk.g);
        for (; it < total; ++it) {
            const uint32_t rs = it % S::NRAW, ws = it % S::NWIDE;
            bool got = mbar_wait(&raw_full[rs], (it / S::NRAW) & 1, abort_flag, err, kDevTimeoutProducer) &&
                       mbar_wait(&wide_empty[ws], ((it / S::NWIDE) & 1) ^ 1, abort_flag, err,
                                 kDevTimeoutProducer);
            if (!__all_sync(0xffffffffu, got)) break;
            const uint8_t* src = sRaw + rs * S::RAW;
            // piece c holds values 16 c .. 16 c + 15: 32 bytes of atom c / 4
            const int c = id & 7;
            uint8_t* dst = sWide + ws * S::WIDE + (c >> 2) * S::ATOM;
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = (id >> 3) + 16 * i;
                v[i] = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[rs]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = (id >> 3) + 16 * i;
                const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[2 * e] = bf16x2_of_e4m3x2(x[e], 0x1404);
                    o[2 * e + 1] = bf16x2_of_e4m3x2(x[e], 0x3424);
                }
                const int p0 = (c & 3) * 2;
                *reinterpret_cast<uint4*>(dst + row * 128 + ((p0 ^ (row & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dst + row * 128 + (((p0 + 1) ^ (row & 7)) << 4)) =
                    make_uint4(o[4], o[5], o[6], o[7]);
            }
            // generic-proxy writes must be visible to the tensor core
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&wide_full[ws]);
        }
    } else if (warp >= 8 && start_ok) {
        // ------------------------------------------------ epilogue
        const int lq = warp & 3, half = (warp - 8) >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(lq * 32) << 16);
        uint32_t job = 0, part = 0;
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const Tokens k = tokens(p);
            const int n = p.w.n, m = p.w.m;
            // weights of the part's columns, fp32: first accumulator's, then the second's
            bool got = mbar_wait(w_empty, (part & 1) ^ 1, abort_flag, err, kDevTimeoutEpilogue);
            if (!__all_sync(0xffffffffu, got)) break;
            const long long row0 = static_cast<long long>(p.b) * T + k.t0;
            for (int c = threadIdx.x - 256; c < k.n * H_I; c += 256) {
                const int at = c < k.first * H_I ? c : c - k.first * H_I + 256;
                sW[at] = __bfloat162float(a.w[row0 * H_I + c]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(w_full);
            got = mbar_wait(w_full, part & 1, abort_flag, err, kDevTimeoutEpilogue);
            if (!__all_sync(0xffffffffu, got)) break;
            ++part;
            for (int t = p.t0; t < p.t1 && ok; ++t) {
                const int s = t * S::KT + lq * 32 + lane;
                const float ks = s < n + m ? __ldg(a.kscale + static_cast<long long>(p.b) * a.S_max + s) : 0.f;
                for (int j = 0; j < k.jobs; ++j, ++job) {
                    const uint32_t acc = job & 1;
                    // this warp's tokens of the accumulator
                    const int nt = j == 0 ? k.first : k.n - k.first;
                    const int mid = (nt + 1) >> 1;
                    const int tb = half ? mid : 0, te = half ? nt : mid;
                    got = mbar_wait(&acc_full[acc], (job >> 1) & 1, abort_flag, err,
                                    kDevTimeoutEpilogue);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int chunks = (te - tb) * (H_I / 32);
                    const uint32_t col0 = acc * 256 + tb * H_I;
                    const float* wa = sW + j * 256 + tb * H_I;
                    float* out = a.scores + (row0 + j * k.first + tb) * a.ld + s;
                    // 32-column chunks: the next is loaded while one is scored
                    constexpr int MAXC = 128 / 32;
                    uint32_t buf[2][32];
                    if (chunks > 0) {
                        tmem_ld32(tl + col0, buf[0]);
                        tmem_ld_wait();
                    }
                    uint64_t p01 = 0, p23 = 0;
#pragma unroll
                    for (int c = 0; c < MAXC; ++c) {
                        if (c + 1 < chunks) tmem_ld32(tl + col0 + (c + 1) * 32, buf[(c + 1) & 1]);
                        if (c < chunks) {
                            const uint32_t(&v)[32] = buf[c & 1];
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const ulonglong2 wv = *reinterpret_cast<const ulonglong2*>(wa + c * 32 + e);
                                p01 = f2_fma(wv.x, f2_pack(fmaxf(__uint_as_float(v[e]), 0.f),
                                                           fmaxf(__uint_as_float(v[e + 1]), 0.f)), p01);
                                p23 = f2_fma(wv.y, f2_pack(fmaxf(__uint_as_float(v[e + 2]), 0.f),
                                                           fmaxf(__uint_as_float(v[e + 3]), 0.f)), p23);
                            }
                            if ((c + 1) % (H_I / 32) == 0) {  // a token's last head is in
                                const float2 x = f2_unpack(p01), y = f2_unpack(p23);
                                float sc = ((x.x + x.y) + (y.x + y.y)) * ks;
                                if (s < n + m) {
                                    if (s >= n) {
                                        const int tok = k.t0 + j * k.first + tb + c / (H_I / 32);
                                        const unsigned long long bits = tree_bits(a.line.ta, p.b, tok, m);
                                        if (!((bits >> (s - n)) & 1)) sc = __int_as_float(0xff800000);
                                    }
                                    out[static_cast<long long>(c / (H_I / 32)) * a.ld] = sc;
                                }
                                p01 = 0;
                                p23 = 0;
                            }
                        }
                        if (c + 1 < chunks) tmem_ld_wait();
                        // all of this accumulator that the warp reads is in registers
                        if (c == max(chunks, 1) - (chunks > 1 ? 2 : 1)) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&acc_empty[acc]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(w_empty);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
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

template <int H_I, int COLS>
int launch_t(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8, const float* kI_scale,
             const TreeArgs& ta, int B, float* scores, int64_t ld, cudaStream_t s) {
    using S = ScoreShape<H_I, COLS>;
    static PerDeviceOnce attr_once;
    cudaError_t e = attr_once.run(ctx->device, [] {
        return cudaFuncSetAttribute(k_index_score_tree<H_I, COLS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    });
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaFuncSetAttribute(index_score_tree)");
    CUtensorMap tm_q, tm_k;
    int rc = make_tmap_bf16_2d(ctx, &tm_q, q, static_cast<uint64_t>(B) * ta.T * H_I, 128, 256);
    if (rc == IC_OK)
        rc = make_tmap_u8_2d(ctx, &tm_k, kI8, static_cast<uint64_t>(B) * ta.cap, 128, 128, S::KT, true);
    if (rc) return rc;
    ScoreArgs a;
    a.line = TreeLine{ta, -1, 1, S::TG};
    a.w = static_cast<const __nv_bfloat16*>(w);
    a.kscale = kI_scale;
    a.scores = scores;
    a.err = ctx->dev_err;
    a.ld = ld;
    a.B = B;
    a.S_max = ta.cap;
    // no more CTAs than the longest caches could have items
    const long long most = static_cast<long long>(B) * ((ta.T + S::TG - 1) / S::TG) *
                           ((ta.cap + S::KT - 1) / S::KT);
    const int grid = most < ctx->num_sms ? static_cast<int>(most) : ctx->num_sms;
    LaunchScope ls(ctx, IC_K_INDEX_SCORE_TREE, s);
    k_index_score_tree<H_I, COLS><<<grid, 512, S::SMEM, s>>>(tm_q, tm_k, a);
    e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "index_score_tree launch");
    return IC_OK;
}

int launch_index_score_tree(ic_ctx* ctx, const void* q, const void* w, const uint8_t* kI8,
                            const float* kI_scale, const TreeArgs& ta, int B, int H_I,
                            float* scores, int64_t ld, cudaStream_t s) {
    // up to 256 (token, head) columns: half the query block, a deeper key ring
    const bool narrow = ta.T * H_I <= 256;
    if (H_I == 64)
        return narrow ? launch_t<64, 256>(ctx, q, w, kI8, kI_scale, ta, B, scores, ld, s)
                      : launch_t<64, 512>(ctx, q, w, kI8, kI_scale, ta, B, scores, ld, s);
    return narrow ? launch_t<32, 256>(ctx, q, w, kI8, kI_scale, ta, B, scores, ld, s)
                  : launch_t<32, 512>(ctx, q, w, kI8, kI_scale, ta, B, scores, ld, s);
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
