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
//  * kind::f16 at the full 16-bit rate: e4m3 keys are exact in f16, and each
//    (token, head) query row is scaled by the power of two that brings its
//    largest value into [2^14, 2^15), where f16 holds a bf16 exactly down to
//    2^-29 of the row's largest (and within 2^-39 of it below).  The scale
//    goes back into w[t,j], which ReLU commutes with.  e4m3 operands would
//    need the queries in two terms: the same tensor time and twice the
//    accumulator columns to read.
//  * The keys are widened in shared memory by four warps (one conversion per
//    two values); the epilogue warps convert a part's queries in place once
//    TMA has brought them.
//  * 2 ReLU(x) is x + |x| (exact; the weights carry the half): an addition on
//    the FMA pipe, where max(x, 0) would take two cycles of the ALU, which
//    the widening loads.  Of -inf it would be NaN, so a part with an infinite
//    query value puts 0 there first.
//  * Warp roles (one CTA per SM): 0 TMA (raw key tiles, query groups), 1 MMA,
//    2 TMEM, 3 finds the CTA's range of the work line, 4..7 widen, 8..23
//    epilogue: two sets of eight, one for each accumulator (lane quarter
//    warp % 4, half of its tokens each), so that one set's waits and loads
//    run beside the other's sums (all 16 on one accumulator at a time took 7%
//    more in short runs, 4% under the power cap; the last accumulator of a
//    part is drained by eight warps instead of sixteen, which costs a call of
//    a few tiles a CTA 1 us of 16 when its inputs are cold).
//  * Up to 256 columns are one accumulator; two ping-pong, over the halves of
//    a 512-column group or over successive tiles.
// Work split: as tree.cuh says; a (sequence, token group, key tile) is an
// item and no two need joining.  Every wait is bounded.
// Measured (B200, H_I = 64, repeated calls): 32 x 65537 keys, 4 tokens each
// 140-144 us = 0.95 PFLOP/s, 8 x 200001, 16 tokens each 355-360 us = 1.11
// PFLOP/s, both under the power cap at 1600 MHz; 20 calls after a pause, which
// end before it acts, take 126 and 311 us.  One and two tokens at 32 x 65537:
// 89 us (1965 MHz) and 107 us (1820 MHz), 2.1 and 2.5 times the bytes' time.
// That is 1570, 1750 and 2040 clocks a tile for 1, 2 and 4 tokens: most of it
// goes into bringing, widening and handing on a tile, for any number of them.
// Reading the accumulators, ReLU and the head sums bound it, and with two
// accumulators in TMEM the products cannot run far enough ahead of them: per
// 256 columns a set holds its accumulator 1600 clocks, the products take
// 1080.  One token at 777 keys: 7.1 us in a graph.
// Tried without gain: half the epilogue warps with 128 columns each in
// registers; widening by integer bit moves; sleeping waits; keys widened into
// TMEM as the A operand with three accumulators of 128 columns (30% slower:
// every accumulator costs its waits, whatever its size).
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
    static constexpr int EPI = 16;                // epilogue warps
    static constexpr int SET = EPI / 2;           // .. of one accumulator
    static constexpr int GROUPS = SET / 4;        // .. that share its tokens
    // tokens of a warp, at most (the epilogue has code for 1 to TOKS)
    static constexpr int TOKS = (JT + GROUPS - 1) / GROUPS;
    static_assert(TOKS == 2 || TOKS == 4, "no epilogue code for more tokens a warp");
    static constexpr int THREADS = (8 + EPI) * 32;
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

// Four e4m3 values as f16, exact.
__device__ __forceinline__ void f16x4_of_e4m3x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
// The power of two 2^s that brings a magnitude with bf16 bits M into
// [2^14, 2^15), clamped to normal floats.
__device__ __forceinline__ int f16_shift_of_max(uint32_t M) {
    const int s = M == 0 ? 0 : 14 - (static_cast<int>(M >> 7) - 127);
    return max(-126, min(126, s));
}

// One warp's share of an accumulator, TOK tokens of 32 keys (at most 64
// columns): the thread of TMEM lane s sums ReLU(dot) w over the heads of each
// token, 32 columns at a time (four such warps per scheduler hide each
// other's loads, and none may spill: beside 227 KB of shared memory the L1
// does not hold 768 threads' spills).  The accumulator is handed back once
// the last columns are in registers.
template <int H_I, int TOK, class Store>
__device__ __forceinline__ void score_columns(uint32_t taddr, const float* w, float ks,
                                              uint64_t* empty, Store&& store) {
    constexpr int CH = TOK * H_I / 32;
    uint64_t p01 = 0, p23 = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        uint32_t v[32];
        tmem_ld32(taddr + c * 32, v);
        tmem_ld_wait();
        if (c == CH - 1) {
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const ulonglong2 wv = *reinterpret_cast<const ulonglong2*>(w + c * 32 + e);
            const float x0 = __uint_as_float(v[e]), x1 = __uint_as_float(v[e + 1]);
            const float x2 = __uint_as_float(v[e + 2]), x3 = __uint_as_float(v[e + 3]);
            p01 = f2_fma(wv.x, f2_pack(x0 + fabsf(x0), x1 + fabsf(x1)), p01);
            p23 = f2_fma(wv.y, f2_pack(x2 + fabsf(x2), x3 + fabsf(x3)), p23);
        }
        if ((c + 1) % (H_I / 32) == 0) {  // a token's last head is in
            const float2 x = f2_unpack(p01), y = f2_unpack(p23);
            store(c / (H_I / 32), ((x.x + x.y) + (y.x + y.y)) * ks);
            p01 = 0;
            p23 = 0;
        }
    }
}

// The same where a query of the part holds an infinity: a dot product may be
// -inf, of which x + |x| would not make 0.  Any number of tokens, in the order
// of sums of score_columns.  (There, a test per 32 columns cost 3% of the time.)
template <int H_I, class Store>
__device__ __forceinline__ void score_columns_infinite(uint32_t taddr, int toks, const float* w,
                                                       float ks, uint64_t* empty, Store&& store) {
#pragma unroll 1
    for (int i = 0; i < toks; ++i) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = i * H_I; c < (i + 1) * H_I; c += 16) {
            uint32_t v[16];
            tmem_ld16(taddr + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = v[e] == 0xff800000u ? 0.f : __uint_as_float(v[e]);
                p[e & 3] = fmaf(w[c + e], x + fabsf(x), p[e & 3]);
            }
        }
        store(i, ((p[0] + p[1]) + (p[2] + p[3])) * ks);
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
}

template <int H_I, int COLS>
__global__ void __launch_bounds__(ScoreShape<H_I, COLS>::THREADS, 1)
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
    uint64_t* q_raw = wide_empty + S::NWIDE;     // a part's bf16 queries (TMA)
    uint64_t* q_full = q_raw + 1;                // .. in f16, and its weights (epilogue warps)
    uint64_t* q_empty = q_full + 1;              // .. no longer read (MMA commit)
    uint64_t* acc_full = q_empty + 1;            // [2]
    uint64_t* acc_empty = acc_full + 2;          // [2] epilogue warps
    uint64_t* w_empty = acc_empty + 2;           // its weights no longer read (epilogue warps)
    uint64_t* done_bar = w_empty + 1;
    LineRange* s_range = reinterpret_cast<LineRange*>(done_bar + 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_range + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // by part & 1: whether one of its queries holds an infinity (epilogue warps)
    volatile int* q_infinite = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* err = a.err;
    const int T = a.line.ta.T;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        q_infinite[0] = q_infinite[1] = 0;
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
        mbar_init(q_raw, 1);
        mbar_init(q_full, S::EPI);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], S::SET);
        }
        mbar_init(w_empty, S::EPI);
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
        const LineRange r = line_range<1>(a.line, a.B, blockIdx.x, gridDim.x);
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
                // the tile's scales go to L2 meanwhile (five lines hold 128
                // fp32 at any alignment; the last is the last key's)
                const float* sc = a.kscale + static_cast<long long>(p.b) * a.S_max;
                const int last = min((t + 1) * S::KT, a.S_max) - 1;
#pragma unroll
                for (int i = 0; i < 5; ++i)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(sc + min(t * S::KT + 32 * i, last)));
                if (t != p.t0) continue;
                // the part's queries, behind its first keys
                if (!mbar_wait(q_empty, (q_it & 1) ^ 1, abort_flag, err, kDevTimeoutProducer)) {
                    ok = false;
                    ++it;
                    break;
                }
                mbar_arrive_expect_tx(q_raw, k.jobs * S::B_JOB);
                for (int j = 0; j < k.jobs; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_2d(sB + j * S::B_JOB + c * S::B_ATOM, &tm_q, q_raw, c * 64,
                                    (p.b * T + k.t0 + j * k.first) * H_I);
                ++q_it;
            }
        }
        // no copy may still be landing at exit
        for (uint32_t i = it > S::NRAW ? it - S::NRAW : 0; i < it; ++i)
            mbar_wait_drain(&raw_full[i % S::NRAW], (i / S::NRAW) & 1);
        if (q_it > 0) mbar_wait_drain(q_raw, (q_it - 1) & 1);
    } else if (warp == 1 && lane == 0 && start_ok) {
        // ------------------------------------------------ MMA issuer
        // descriptors of the first stage and query block; the address field
        // counts 16 bytes and never overflows into the next
        const uint64_t k_desc = sdesc_k_sw128(smem_u32(sWide)), q_desc = sdesc_k_sw128(smem_u32(sB));
        uint32_t it = 0, q_it = 0, job = 0;
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const Tokens k = tokens(p);
            if (!mbar_wait(q_full, q_it & 1, abort_flag, err, kDevTimeoutMma)) break;
            ++q_it;
            const uint32_t id0 = idesc_f16_f32(S::KT, k.first * H_I);
            const uint32_t id1 = idesc_f16_f32(S::KT, (k.n - k.first) * H_I);
            for (int t = p.t0; t < p.t1 && ok; ++t, ++it) {
                const uint32_t st = it % S::NWIDE;
                if (!mbar_wait(&wide_full[st], (it / S::NWIDE) & 1, abort_flag, err, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                const uint64_t kd = k_desc + static_cast<uint64_t>(st * (S::WIDE >> 4));
                for (int j = 0; j < k.jobs; ++j, ++job) {
                    const uint32_t acc = job & 1;
                    if (!mbar_wait(&acc_empty[acc], ((job >> 1) & 1) ^ 1, abort_flag, err,
                                   kDevTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t id = j == 0 ? id0 : id1, d = tmem + acc * 256;
                    const uint64_t qd = q_desc + static_cast<uint64_t>(j * (S::B_JOB >> 4));
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16(d, kd + ((c * S::ATOM + kk * 32) >> 4),
                                     qd + ((c * S::B_ATOM + kk * 32) >> 4), id, (c | kk) ? 1u : 0u);
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
        // Eight lanes take four pieces (values 16 c .. 16 c + 15) of two rows
        // r and r ^ 5: with pieces XOR-swizzled by row, neither the loads (the
        // rows differ in bit 2) nor the stores of the two 16-byte halves (they
        // differ in bit 0) meet a bank group twice.
        const int c = (lane & 3) | ((lane >> 1) & 4);  // atom c / 4 is lane bit 3
        const int pair0 = (warp - 4) * 2 + (lane >> 4), second = (lane >> 2) & 1;
        uint32_t it = 0;
        const uint32_t total = static_cast<uint32_t>(walk.g_end - walk.g);
        for (; it < total; ++it) {
            const uint32_t rs = it % S::NRAW, ws = it % S::NWIDE;
            bool got = mbar_wait(&raw_full[rs], (it / S::NRAW) & 1, abort_flag, err, kDevTimeoutProducer) &&
                       mbar_wait(&wide_empty[ws], ((it / S::NWIDE) & 1) ^ 1, abort_flag, err,
                                 kDevTimeoutProducer);
            if (!__all_sync(0xffffffffu, got)) break;
            const uint8_t* src = sRaw + rs * S::RAW;
            uint8_t* dst = sWide + ws * S::WIDE + (c >> 2) * S::ATOM;
#pragma unroll 4
            for (int i = 0; i < 8; ++i) {
                const int pr = pair0 + 8 * i;  // row pair of the tile's 64
                const int row = (pr >> 2) * 8 + ((pr & 3) ^ (second * 5));
                const uint4 v = *reinterpret_cast<const uint4*>(src + row * 128 + ((c ^ (row & 7)) << 4));
                uint4 lo, hi;
                f16x4_of_e4m3x4(v.x, lo.x, lo.y);
                f16x4_of_e4m3x4(v.y, lo.z, lo.w);
                f16x4_of_e4m3x4(v.z, hi.x, hi.y);
                f16x4_of_e4m3x4(v.w, hi.z, hi.w);
                const int p0 = (c & 3) * 2;
                *reinterpret_cast<uint4*>(dst + row * 128 + ((p0 ^ (row & 7)) << 4)) = lo;
                *reinterpret_cast<uint4*>(dst + row * 128 + (((p0 + 1) ^ (row & 7)) << 4)) = hi;
            }
            // generic-proxy writes must be visible to the tensor core
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&raw_empty[rs]);
                mbar_arrive(&wide_full[ws]);
            }
        }
    } else if (warp >= 8 && start_ok) {
        // ------------------------------------------------ epilogue
        const int lq = warp & 3, group = ((warp - 8) >> 2) & 1;
        const uint32_t set = (warp - 8) >> 3;
        const uint32_t tl = tmem + (static_cast<uint32_t>(lq * 32) << 16);
        uint32_t job = 0, part = 0;
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const Tokens k = tokens(p);
            const int n = p.w.n, m = p.w.m;
            // The part's queries from bf16 to f16 in place (K-major, swizzled:
            // 64 columns per atom, an accumulator's rows from row 0 of its
            // block), and its weights: 16 lanes per (token, head) row.
            const long long row0 = static_cast<long long>(p.b) * T + k.t0;
            const int rows = k.n * H_I, rows0 = k.first * H_I, l16 = lane & 15;
            const int r_first = (warp - 8) * 2 + (lane >> 4);
            // lane l16 holds the weights of this half-warp's rows l16 and l16 + 16
            float wv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = r_first + (l16 + 16 * i) * 2 * S::EPI;
                wv[i] = r < rows ? __bfloat162float(a.w[row0 * H_I + r]) : 0.f;
            }
            bool got = mbar_wait(w_empty, (part & 1) ^ 1, abort_flag, err, kDevTimeoutEpilogue) &&
                       mbar_wait(q_raw, part & 1, abort_flag, err, kDevTimeoutEpilogue);
            if (!__all_sync(0xffffffffu, got)) break;
            // rows is a multiple of 32: the two rows of a warp go together
#pragma unroll 4
            for (int r = r_first, i = 0; r < rows; r += 2 * S::EPI, ++i) {
                const float w = __shfl_sync(0xffffffffu, i < 16 ? wv[0] : wv[1], (lane & 16) + (i & 15));
                const int j = r >= rows0, rr = r - j * rows0;
                uint4* at = reinterpret_cast<uint4*>(sB + j * S::B_JOB + (l16 >> 3) * S::B_ATOM +
                                                     rr * 128 + (((l16 & 7) ^ (rr & 7)) << 4));
                const uint4 v = *at;
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                uint32_t M = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) M = max(M, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) M = max(M, __shfl_xor_sync(0xffffffffu, M, o));
                const int sh = f16_shift_of_max(M);
                const float up = __int_as_float((127 + sh) << 23);
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 y = __floats2half2_rn(__uint_as_float(x[e] << 16) * up,
                                                        __uint_as_float(x[e] & 0xFFFF0000u) * up);
                    h[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *at = make_uint4(h[0], h[1], h[2], h[3]);
                // ReLU of a row with an infinity is 0, inf or NaN whatever it was
                // scaled by, and a weight scaled back up could pass fp32's range
                const bool inf = M == 0x7F80u;
                if (l16 == 0) {
                    sW[j * 256 + rr] = inf ? w : w * (0.5f * __int_as_float((127 - sh) << 23));
                    if (inf) q_infinite[part & 1] = 1;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            got = mbar_wait(q_full, part & 1, abort_flag, err, kDevTimeoutEpilogue);
            if (!__all_sync(0xffffffffu, got)) break;
            const bool infinite = q_infinite[part & 1] != 0;
            // the next part's: read a part ago, and set once w_empty says that
            // every warp is past this line
            if (threadIdx.x == 256) q_infinite[(part & 1) ^ 1] = 0;
            ++part;
            // This set's accumulators are the odd or the even ones: the same
            // one of every tile's two, or every second tile's one.
            const uint32_t turn = (set ^ job) & 1;
            const int j = k.jobs == 2 ? turn : 0, step = 3 - k.jobs;
            // .. and this warp's tokens of it
            const int nt = j == 0 ? k.first : k.n - k.first;
            const int per = (nt + S::GROUPS - 1) / S::GROUPS;
            const int tb = min(nt, group * per), toks = min(nt, tb + per) - tb;
            const int end = n + m;
            const uint32_t ta = tl + set * 256 + tb * H_I;
            const float* const wa = sW + j * 256 + tb * H_I;
            const int tok = j * k.first + tb;  // of the part
            float* const out = a.scores + (row0 + tok) * a.ld + lq * 32 + lane;
            const float* const scale = a.kscale + static_cast<long long>(p.b) * a.S_max + lq * 32 + lane;
            for (int t = p.t0 + (k.jobs == 1 ? turn : 0); t < p.t1; t += step) {
                const int s = t * S::KT + lq * 32 + lane;
                const bool inner = (t + 1) * S::KT <= n;  // every row sees the whole tile
                // in L2 since the tile's keys were asked for; used after the head sums
                const float ks = s < end ? __ldg(scale + t * S::KT) : 0.f;
                const uint32_t now = job + (t - p.t0) * k.jobs + j;
                got = mbar_wait(&acc_full[set], (now >> 1) & 1, abort_flag, err, kDevTimeoutEpilogue);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float* const row = out + t * S::KT;
                auto store = [&](int i, float sc) {
                    if (!inner) {
                        if (s >= end) return;
                        if (s >= n) {
                            const unsigned long long bits = tree_bits(a.line.ta, p.b, k.t0 + tok + i, m);
                            if (!((bits >> (s - n)) & 1)) sc = __int_as_float(0xff800000);
                        }
                    }
                    row[i * a.ld] = sc;
                };
                if (infinite) {
                    score_columns_infinite<H_I>(ta, toks, wa, ks, &acc_empty[set], store);
                    continue;
                }
                switch (toks) {  // straight-line code for each count a warp can have
                    case 1: score_columns<H_I, 1>(ta, wa, ks, &acc_empty[set], store); break;
                    case 2: score_columns<H_I, 2>(ta, wa, ks, &acc_empty[set], store); break;
                    case 3:
                        if constexpr (S::TOKS == 4)
                            score_columns<H_I, 3>(ta, wa, ks, &acc_empty[set], store);
                        break;
                    case 4:
                        if constexpr (S::TOKS == 4)
                            score_columns<H_I, 4>(ta, wa, ks, &acc_empty[set], store);
                        break;
                    default:
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[set]);
                }
            }
            job += static_cast<uint32_t>(p.t1 - p.t0) * k.jobs;
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

// Whether a call's output lies on anything it reads.
bool meets_input(const Span& out, const void* q, const void* w, const uint8_t* kI8,
                 const float* kI_scale, const int32_t* prefix_len, const int32_t* draft_len,
                 const uint64_t* tree_mask, int B, int T, int S_max, int H_I, int d_I) {
    const long long drafts = static_cast<long long>(B) * T, keys = static_cast<long long>(B) * S_max;
    return out.meets(Span(q, drafts * H_I * d_I * 2)) || out.meets(Span(w, drafts * H_I * 2)) ||
           out.meets(Span(kI8, keys * d_I)) || out.meets(Span(kI_scale, keys * 4)) ||
           out.meets(Span(prefix_len, B * 4ll)) || (draft_len && out.meets(Span(draft_len, B * 4ll))) ||
           (tree_mask && out.meets(Span(tree_mask, drafts * 8)));
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
    const int groups = (ta.T + S::TG - 1) / S::TG;
    if (!line_fits(B, groups, ta.cap))
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree index: B=%d sequences of up to %d keys are too many",
                    B, ta.cap);
    const long long most = static_cast<long long>(B) * groups * ((ta.cap + S::KT - 1) / S::KT);
    const int grid = most < ctx->num_sms ? static_cast<int>(most) : ctx->num_sms;
    LaunchScope ls(ctx, IC_K_INDEX_SCORE_TREE, s);
    k_index_score_tree<H_I, COLS><<<grid, S::THREADS, S::SMEM, s>>>(tm_q, tm_k, a);
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
    if (meets_input(Span(scores, ((static_cast<long long>(B) * T - 1) * ld + S_max) * 4), q, w, kI8, kI_scale,
                    prefix_len, draft_len, tree_mask, B, T, S_max, H_I, d_I))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree index: scores overlap an input");
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
    if (meets_input(Span(idx_out, static_cast<long long>(B) * T * k * 4), q, w, kI8, kI_scale, prefix_len,
                    draft_len, tree_mask, B, T, S_max, H_I, d_I))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree index: idx_out overlaps an input");
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
    rc = ensure_buffer_on(ctx, s, reinterpret_cast<void**>(&ctx->scores), &ctx->scores_cap,
                          chunk * per_seq, &ctx->scores_hold);
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
