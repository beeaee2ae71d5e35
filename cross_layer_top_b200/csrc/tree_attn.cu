// Attention of drafted tokens over a cache:
//   o[b,t,h,:] = sum_s softmax_s(scale * Q[b,t,h,:].K[b,s,:]) V[b,s,:]
// over the committed slots (all, or the positions of one list per sequence)
// and the drafts that row (b, t) sees.  One K/V head is shared by all query
// heads and, here, by all drafts of a sequence: a key read once serves T*Hq
// query rows.
//
// Design (sm_100a).  The T*Hq query rows of a sequence are the M rows of
// tcgen05 tiles (128 rows each; NM = 1 or 2 tiles per CTA), 128 keys the
// other side: S = Q K^T into TMEM, softmax in registers (one thread per row
// and tile, so no row reduction crosses threads), P as bf16 back into TMEM
// over its S, and O += P V with P as the A operand from TMEM and V as the
// MN-major B operand straight from the same [keys, d] tile that TMA or the
// gather wrote.
//  * Two streams of tiles take turns on the tensor core: with NM = 2 the two
//    row tiles of each key tile, with NM = 1 the even and the odd key tiles of
//    the one row tile (each with its own O, maximum and sum, joined at the
//    part's end).  While one stream is in its softmax, the other's products run.
//  * Warps 0..3 (loads): tiles that lie whole in the committed prefix come by
//    TMA; tiles with listed positions or drafts are gathered with cp.async,
//    rows that nobody sees (drafts outside every row's mask, list entries of
//    -1, what lies behind the last draft) filled with zeros, so that whatever
//    those slots hold takes no part.  K and V tiles alternate in one ring.
//  * Warp 4 issues the MMAs, warp 5 owns the TMEM allocation, warp 6 finds
//    the CTA's range of the work line.
//  * Warps 8..15 (softmax, four per stream) hold a whole row of S in
//    registers, which they take from the other warps.  The running maximum is
//    only a reference for exp2: it moves, and O in TMEM is rescaled, when a
//    logit passes it by 2^8 (lazy rescale).  P is rounded to bf16 for the
//    tensor core (relative 2^-8 of each weight, as in the one-token attention);
//    the row sum, of the weights as they were, and O stay fp32.  Against 64
//    bits outputs are off by 0.0021-0.0024 of their size, where rounding the
//    exact result to bf16 alone gives 0.0017.
// Work split (one CTA per SM): see tree.cuh.  A part that covers a whole
// (sequence, row-tile group) writes the output; the others write (O, m, l) to
// a workspace slot and a second, small kernel (launched as a programmatic
// dependent) joins them.  A CTA has at most two such parts, one that ends its
// unit (slot 0, only ever the CTA's first part) and one that another CTA
// continues (slot 1); each CTA notes which unit its slot 0 ends and which CTA
// began it.
// Every wait is bounded.
// Measured (B200, Hq = 16, d = 128, repeated calls), join included: 8 sequences
// of ragged lengths up to 200001, 8 drafts each 163-173 us = 4.5-4.8 TB/s of K
// and V; 32 x 65537 225 us = 4.8 TB/s; both under the power cap at 1600 MHz (20
// calls after a pause, before it acts: 146 and 196 us).  4 x 64 drafts at 16421
// 60 us = 0.55 PFLOP/s at 1965 MHz: a pair of 128 x 128 tiles takes 4900
// clocks, of which the products take 2700 (2050 at the full rate) and each
// stream's softmax 2050; each stream is one chain (S, the whole tile's softmax,
// P V, the next S), and the two do not hide all of each other's steps.  32 lists of 2048, 8 drafts each 26.6 us:
// start 4 us, five gathered tiles one after the other, the part's end, the
// join's launch.
// Tried without gain: exp2 as a polynomial on the FMA pipe, 3-input maxima,
// looking at the next barriers between products.
#include <math.h>

#include "ic_internal.h"
#include "tree.cuh"

using namespace ic;

namespace {

constexpr int kTile = kLineTile;  // keys per tile, rows per row tile
constexpr float kRescale = 8.f; // log2 units
constexpr int kWsRows = 256;    // workspace rows of one slot: two row tiles
// tiles that one more part costs a CTA (measured 5 us: O out, rows in, the
// pipeline's drain and fill; a key tile takes 1.2 us with one row tile, 2.5
// with two)
template <int NM>
constexpr int kPartTiles = NM == 1 ? 4 : 2;
// the unit whose last part lies in a CTA's slot 0 (b < 0: none), and the CTA
// of its first part
struct __align__(16) JoinNote {
    int b, group, first, rows;  // rows: of the sequence
};

template <int D, int NM>
struct AttnTile {
    static constexpr int NATOM = D / 64;
    static constexpr int ATOM = kTile * 128;          // 64 columns of a tile
    static constexpr int TILE = NATOM * ATOM;         // bytes of a Q, K or V tile
    static constexpr int BAR_BYTES = 512;
    static constexpr int XCH_BYTES = NM == 1 ? 2 * 2 * kTile * 8 : 0;  // [part & 1][stream][row] (m, l)
    static constexpr int NST_RAW = (232448 - NM * TILE - BAR_BYTES - XCH_BYTES) / TILE;
    static constexpr int NST = NST_RAW > 10 ? 10 : NST_RAW;
    static constexpr int OFF_KV = NM * TILE;
    static constexpr int OFF_BAR = OFF_KV + NST * TILE;
    static constexpr int OFF_XCH = OFF_BAR + BAR_BYTES;
    static constexpr int SMEM = OFF_XCH + XCH_BYTES;
    static constexpr int THREADS = 512;
    // registers: 128 a thread at launch; the softmax takes what the others need not
    static constexpr int REGS_LOW = 72, REGS_SOFT = 184;
    static_assert(256 * REGS_LOW + 256 * REGS_SOFT <= THREADS * 128, "register split");
    static_assert(NST >= 5 && SMEM <= 232448, "shared memory budget");
};

struct AttnArgs {
    TreeLine line;
    TreeArgs ta;
    const int32_t* idx;
    const __nv_bfloat16* K;
    const __nv_bfloat16* V;
    __nv_bfloat16* out;
    float* ws;
    JoinNote* notes;  // [CTAs]
    int* err;
    long long kv_stride;
    int B, Hq, k;
    float scale_log2;
};

template <int D, int NM>
__global__ void __launch_bounds__(AttnTile<D, NM>::THREADS, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs a) {
    using S = AttnTile<D, NM>;
    constexpr int NST = S::NST, TILE = S::TILE, ATOM = S::ATOM, NATOM = S::NATOM;
    constexpr int GROUP_ROWS = NM * kTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sQ = smem;
    uint8_t* sKV = smem + S::OFF_KV;
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);  // [NST] the load warps' threads
    uint64_t* kv_empty = kv_full + NST;  // [NST] MMA commit
    uint64_t* q_full = kv_empty + NST;
    uint64_t* q_empty = q_full + 1;
    // by stream:
    uint64_t* s_full = q_empty + 1;   // [2] S computed
    uint64_t* p_full = s_full + 2;    // [2] P written (four softmax warps)
    uint64_t* pv_done = p_full + 2;   // [2] O += P V complete
    uint64_t* o_empty = pv_done + 2;  // [2] O of a part read out (NM = 1: by both streams' warps)
    uint64_t* x_full = o_empty + 2;   // [2] NM = 1: the stream's (m, l) of a part written
    uint64_t* done_bar = x_full + 2;
    LineRange* s_range = reinterpret_cast<LineRange*>(done_bar + 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_range + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* err = a.err;
    griddep_launch_dependents();  // the join kernel may be set up early; it waits for this one

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        if (smem_u32(smem) & 1023u) {
            *abort_flag = 1;
            atomicCAS(err, 0, kDevSmemMisaligned);
        }
        for (int i = 0; i < NST; ++i) {
            mbar_init(&kv_full[i], 128);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_empty[i], NM == 1 ? 8 : 4);
            mbar_init(&x_full[i], 4);
        }
        mbar_init(done_bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 5) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == 6) {
        // this CTA's range of the line, and the sequence it starts in
        const LineRange r = line_range<kPartTiles<NM>>(a.line, a.B, blockIdx.x, gridDim.x);
        if (lane == 0) *s_range = r;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 6) {
        if (lane == 0) {
            const LineRange r = *s_range;
            JoinNote note{-1, 0, 0, 0};
            PartWalk first(r);
            if (first.next(a.line) && first.p.t0 > 0 && first.p.t1 == first.p.w.tiles) {
                const Part& p = first.p;
                note.b = p.b;
                note.group = p.group;
                note.rows = p.w.rows;
                // pieces follow each other; of equal ranges, the one that
                // holds item u is floor(((u + 1) parts - 1) / total)
                const long long u = first.base + p.group * p.w.tiles;
                note.first = r.step
                                 ? static_cast<int>(blockIdx.x) - ((p.w.tiles + r.step - 1) / r.step - 1)
                                 : static_cast<int>(((u + 1) * r.parts - 1) / r.total);
            }
            a.notes[blockIdx.x] = note;
        }
        // lengths out of range are reported by the first CTA
        if (blockIdx.x == 0)
            for (int b = lane; b < a.B; b += 32) {
                int n, m;
                if (!tree_lens(a.ta, b, n, m)) atomicCAS(err, 0, kDevBadTree);
            }
    }
    const uint32_t tmem = *tmem_slot;
    const bool start_ok = (*abort_flag == 0);
    PartWalk walk(*s_range);

    if (warp < 8) {
    regs_dec<S::REGS_LOW>();
    if (warp < 4 && start_ok) {
        // ------------------------------------------------ loads
        uint32_t item = 0, q_it = 0;   // ring items (K, V, K, V, ..) and parts so far
        uint32_t tma_used = 0, tma_ph = 0;  // per stage: last filled by TMA, with which parity
        bool ok = true;
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const int n = p.w.n, m = p.w.m;
            const int L = a.idx ? a.k : n;  // columns before the drafts
            const __nv_bfloat16* Kb = a.K + p.b * a.kv_stride;
            const __nv_bfloat16* Vb = a.V + p.b * a.kv_stride;
            unsigned long long any = 0;  // drafts that some row sees
            bool any_known = false;
            for (int t = p.t0; t < p.t1 && ok; ++t) {
                const int v0 = t * kTile;
                const bool tma = a.idx == nullptr && v0 + kTile <= n;
                int slot = -1;
                if (!tma) {
                    if (v0 + kTile > L && !any_known) {
                        any_known = true;
                        for (int r = lane; r < m; r += 32) any |= tree_bits(a.ta, p.b, r, m);
                        any = static_cast<unsigned long long>(
                                  __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32))) << 32 |
                              __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any));
                    }
                    const int v = v0 + warp * 32 + lane;
                    if (v < L) {
                        slot = a.idx ? __ldg(a.idx + static_cast<long long>(p.b) * a.k + v) : v;
                        if (slot < 0 || slot >= n) {
                            if (slot != -1) atomicCAS(err, 0, kDevBadIndex);
                            slot = -1;
                        }
                    } else if (v - L < m && ((any >> (v - L)) & 1)) {
                        slot = n + v - L;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t st = item % NST, par = (item / NST) & 1;
                    const bool got = mbar_wait(&kv_empty[st], par ^ 1, abort_flag, err, kDevTimeoutProducer);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dst = sKV + st * TILE;
                    if (tma) {
                        if (threadIdx.x == 0) {
                            mbar_arrive_expect_tx(&kv_full[st], TILE);
#pragma unroll
                            for (int c = 0; c < NATOM; ++c)
                                tma_load_3d(dst + c * ATOM, kv ? &tm_v : &tm_k, &kv_full[st], c * 64, v0, p.b);
                        } else {
                            mbar_arrive(&kv_full[st]);
                        }
                        tma_used |= 1u << st;
                        tma_ph = (tma_ph & ~(1u << st)) | (par << st);
                    } else {
                        tma_used &= ~(1u << st);
                        const __nv_bfloat16* src = kv ? Vb : Kb;
                        constexpr int PPR = D / 8;        // 16-byte pieces per row
                        constexpr int RPI = 32 / PPR;     // rows per instruction
                        const int piece = lane % PPR;
                        const uint32_t base = smem_u32(dst) + (piece >> 3) * ATOM;
#pragma unroll
                        for (int r = 0; r < 32; r += RPI) {
                            const int rr = r + lane / PPR;
                            const int s = __shfl_sync(0xffffffffu, slot, rr);
                            const int row = warp * 32 + rr;
                            cp_async16(base + row * 128 + (((piece & 7) ^ (row & 7)) << 4),
                                       src + static_cast<long long>(s < 0 ? 0 : s) * D + piece * 8,
                                       s >= 0);
                        }
                        cp_async_arrive(&kv_full[st]);
                    }
                    ++item;
                }
                if (t == p.t0 && ok) {
                    // the part's query rows, behind its first tile so that the
                    // wait for the previous part's last use costs no load time
                    if (warp == 0) {
                        const bool got = mbar_wait(q_empty, (q_it & 1) ^ 1, abort_flag, err, kDevTimeoutProducer);
                        if (!__all_sync(0xffffffffu, got)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full, NM * TILE);
                            const int row0 = p.b * a.ta.T * a.Hq + p.group * GROUP_ROWS;
#pragma unroll
                            for (int i = 0; i < NM; ++i)
#pragma unroll
                                for (int c = 0; c < NATOM; ++c)
                                    tma_load_2d(sQ + i * TILE + c * ATOM, &tm_q, q_full, c * 64,
                                                row0 + i * kTile);
                        }
                    }
                    ++q_it;
                }
            }
        }
        // no copy may still be landing at exit
        cp_async_wait_all();
        if (warp == 0 && lane == 0) {
            for (int i = 0; i < NST; ++i)
                if ((tma_used >> i) & 1) mbar_wait_drain(&kv_full[i], (tma_ph >> i) & 1);
            if (q_it > 0) mbar_wait_drain(q_full, (q_it - 1) & 1);
        }
    } else if (warp == 4 && start_ok) {
        // ------------------------------------------------ MMA issuer
        // The whole warp runs the loop, lane 0 issues: this thread's own
        // instructions lie between one tile's products and the next.
        constexpr uint32_t ID_S = idesc_bf16_f32(kTile, kTile);
        constexpr uint32_t ID_O = idesc_bf16_f32(kTile, D) | kIdescBMnMajor;
        const uint32_t lead = lane == 0;
        uint32_t q_it = 0;
        uint32_t uses[2] = {0, 0};      // S tiles of each stream so far
        uint32_t parts_of[2] = {0, 0};  // parts of each stream so far
        bool ok = true;
        // descriptors of the first tiles; the address field counts 16 bytes
        // and never overflows into the next
        const uint64_t q_desc = sdesc_k_sw128(smem_u32(sQ)), k_desc = sdesc_k_sw128(smem_u32(sKV));
        const uint64_t v_desc = sdesc_mn_sw128(smem_u32(sKV), ATOM);
        // ring stage and parity of the next K tile and the next V tile
        uint32_t ks = 0, kp = 0, vs = 1, vp = 0;
        auto wait = [&](uint64_t* bar, uint32_t par) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, err, kDevTimeoutMma)) != 0;
            return ok;
        };
        // a tile has landed; gathered ones came by the generic proxy
        auto full = [&](uint32_t stage, uint32_t par) {
            const bool got = wait(&kv_full[stage], par);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            return got;
        };
        auto step2 = [](uint32_t& stage, uint32_t& par) {  // two items on
            stage += 2;
            if (stage >= NST) {
                stage -= NST;
                par ^= 1;
            }
        };
        // S of stream st (rows of row tile rt) with the K tile in its stage
        auto issue_s = [&](int st, int rt) {
            const uint64_t qd = q_desc + static_cast<uint64_t>(rt * (TILE >> 4));
            const uint64_t kd = k_desc + static_cast<uint64_t>(ks * (TILE >> 4));
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NATOM; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f16_if(lead, tmem + st * 128, qd + ((c * ATOM + kk * 32) >> 4),
                                kd + ((c * ATOM + kk * 32) >> 4), ID_S, (c | kk) ? 1u : 0u);
            umma_commit_if(lead, &s_full[st]);
        };
        auto issue_o = [&](int st, bool acc) {
            const uint64_t vd = v_desc + static_cast<uint64_t>(vs * (TILE >> 4));
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
                umma_f16_ts_if(lead, tmem + 256 + st * 128, tmem + st * 128 + kk * 8,
                               vd + ((kk * 2048) >> 4), ID_O, (acc || kk) ? 1u : 0u);
            umma_commit_if(lead, &pv_done[st]);
        };
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const int nt = p.t1 - p.t0;
            if (!wait(q_full, q_it & 1)) break;
            ++q_it;
            if (NM == 1) {
                // stream j & 1: P V of tile j - 2, then S of tile j over that P
                for (int j = 0; j < nt + 2 && ok; ++j) {
                    const int st = j & 1;
                    if (j >= 2 && j - 2 < nt) {
                        if (!full(vs, vp)) break;
                        if (j < 4 && !wait(&o_empty[st], (parts_of[0] & 1) ^ 1)) break;
                        if (!wait(&p_full[st], (uses[st] - 1) & 1)) break;
                        issue_o(st, j >= 4);
                        umma_commit_if(lead, &kv_empty[vs]);
                        step2(vs, vp);
                    }
                    if (j < nt) {
                        if (!full(ks, kp)) break;
                        if (uses[st] > 0 && !wait(&pv_done[st], (uses[st] - 1) & 1)) break;
                        issue_s(st, 0);
                        umma_commit_if(lead, &kv_empty[ks]);
                        step2(ks, kp);
                        if (j == nt - 1) umma_commit_if(lead, q_empty);
                        ++uses[st];
                    }
                }
                ++parts_of[0];
            } else {
                const int live = p.w.rows - p.group * GROUP_ROWS > kTile ? 2 : 1;
                for (int j = 0; j <= nt && ok; ++j) {
                    for (int rt = 0; rt < live && ok; ++rt) {
                        if (j > 0) {
                            if (rt == 0 && !full(vs, vp)) break;
                            if (j == 1 && !wait(&o_empty[rt], (parts_of[rt] & 1) ^ 1)) break;
                            if (!wait(&p_full[rt], (uses[rt] - 1) & 1)) break;
                            issue_o(rt, j > 1);
                            if (rt == live - 1) umma_commit_if(lead, &kv_empty[vs]);
                        }
                        if (j < nt) {
                            if (rt == 0 && !full(ks, kp)) break;
                            // S overwrites P of this row tile's tile before
                            if (uses[rt] > 0 && !wait(&pv_done[rt], (uses[rt] - 1) & 1)) break;
                            issue_s(rt, rt);
                            if (rt == live - 1) {
                                umma_commit_if(lead, &kv_empty[ks]);
                                if (j == nt - 1) umma_commit_if(lead, q_empty);
                            }
                            ++uses[rt];
                        }
                    }
                    if (j > 0) step2(vs, vp);
                    if (j < nt) step2(ks, kp);
                }
                for (int rt = 0; rt < live; ++rt) ++parts_of[rt];
            }
        }
        // every MMA issued completes before TMEM and shared memory are released
        umma_commit_if(lead, done_bar);
        if (!mbar_wait_drain(done_bar, 0)) atomicCAS(err, 0, kDevTimeoutDrain);
    }
    } else {
        regs_inc<S::REGS_SOFT>();
        // ------------------------------------------------ softmax
        const int st = (warp - 8) >> 2;           // stream
        const int rt = NM == 2 ? st : 0;          // its row tile
        const int lq = warp & 3;                  // TMEM lanes 32 lq ..
        const uint32_t tl = tmem + (static_cast<uint32_t>(lq * 32) << 16);
        const uint32_t s_col = st * 128, o_col = 256 + st * 128;
        constexpr int STEP = NM == 1 ? 2 : 1;     // key tiles from one of the stream to the next
        float2* xch = reinterpret_cast<float2*>(smem + S::OFF_XCH);
        uint32_t it = 0, part = 0;  // tiles of this stream, and parts, so far
        bool ok = start_ok;
        const uint64_t scale2 = f2_pack(a.scale_log2, a.scale_log2);
        while (ok && walk.next(a.line)) {
            const Part& p = walk.p;
            const int row0 = p.group * GROUP_ROWS + rt * kTile;
            if (NM == 2 && row0 >= p.w.rows && rt == 1) continue;  // no such row tile
            const int row = row0 + lq * 32 + lane;
            const bool live = row < p.w.rows;
            const bool warp_live = row0 + lq * 32 < p.w.rows;
            const int n = p.w.n, m = p.w.m, L = a.idx ? a.k : n;
            const int32_t* list = a.idx ? a.idx + static_cast<long long>(p.b) * a.k : nullptr;
            const unsigned long long bits = live ? tree_bits(a.ta, p.b, row / a.Hq, m) : 0ull;
            const int t_first = p.t0 + (NM == 1 ? st : 0);
            float ref = -INFINITY, l = 0.f;  // reference of exp2, sum of weights
            // the list entries of a tile's 128 columns, loaded a tile ahead
            int ent[4] = {-1, -1, -1, -1};
            auto load_list = [&](int t) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int v = t * kTile + c * 32 + lane;
                    ent[c] = list && warp_live && t < p.t1 && v < L ? __ldg(list + v) : -1;
                }
            };
            load_list(t_first);
            for (int t = t_first; t < p.t1; t += STEP, ++it) {
                // visible columns of this row, 32 at a time
                uint32_t vis[4];
                bool all = !list && (t + 1) * kTile <= L;
                if (!all) {
                    all = true;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t listed =
                            list ? __ballot_sync(0xffffffffu, ent[c] >= 0 && ent[c] < n) : 0xffffffffu;
                        const int u = t * kTile + c * 32 - L;  // draft of the first column
                        uint32_t d;
                        if (u <= -32) d = 0u;
                        else if (u >= 64) d = 0u;
                        else if (u >= 0) d = static_cast<uint32_t>(bits >> u);
                        else d = static_cast<uint32_t>(bits << -u);
                        const uint32_t before = u <= -32 ? 0xffffffffu : (u >= 0 ? 0u : (1u << -u) - 1u);
                        vis[c] = (before & listed) | (d & ~before);
                        all = all && vis[c] == 0xffffffffu;
                    }
                    load_list(t + STEP);
                    all = __all_sync(0xffffffffu, all || !live);
                }
                bool got = mbar_wait(&s_full[st], it & 1, abort_flag, err, kDevTimeoutEpilogue);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (warp_live) {
                    // the tile's maximum; half of the row stays in registers,
                    // the other half is loaded again (a whole row spills)
                    auto mask = [&](uint32_t (&v)[32], uint32_t seen) {
                        if (!all)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((seen >> e) & 1)) v[e] = 0xff800000u;
                    };
                    auto max_of = [](const uint32_t (&v)[32]) {
                        float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[1]);
#pragma unroll
                        for (int e = 2; e < 32; e += 2) {
                            m0 = fmaxf(m0, __uint_as_float(v[e]));
                            m1 = fmaxf(m1, __uint_as_float(v[e + 1]));
                        }
                        return fmaxf(m0, m1);
                    };
                    uint32_t s[2][32], u[32];
                    tmem_ld32(tl + s_col, s[0]);
                    tmem_ld32(tl + s_col + 32, s[1]);
                    tmem_ld32(tl + s_col + 64, u);
                    tmem_ld_wait();
                    mask(s[0], vis[0]);
                    mask(s[1], vis[1]);
                    mask(u, vis[2]);
                    float mx = max_of(u);
                    tmem_ld32(tl + s_col + 96, u);
                    mx = fmaxf(mx, fmaxf(max_of(s[0]), max_of(s[1])));
                    tmem_ld_wait();
                    mask(u, vis[3]);
                    mx = fmaxf(mx, max_of(u)) * a.scale_log2;
                    const bool moves = mx > ref + kRescale || (ref == -INFINITY && mx > -INFINITY);
                    if (__any_sync(0xffffffffu, moves)) {
                        const float to = moves ? mx : ref;
                        const float f = ref == -INFINITY ? 0.f : ex2_approx(ref - to);
                        const float fl = to == -INFINITY ? 1.f : f;
                        ref = to;
                        l *= fl;
                        if (t > t_first) {
                            // O holds the stream's tiles before this one
                            got = mbar_wait(&pv_done[st], (it - 1) & 1, abort_flag, err, kDevTimeoutEpilogue);
                            if (!__all_sync(0xffffffffu, got)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(tl + o_col + c * 16, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fl);
                                tmem_st16(tl + o_col + c * 16, o);
                            }
                        }
                    }
                    const float sub = ref == -INFINITY ? 0.f : ref;
                    const uint64_t sub2 = f2_pack(-sub, -sub);
                    uint64_t sum[2] = {0, 0};
                    // P of 32 columns: in the first 64 columns of S, which are in registers
                    auto weights = [&](const uint32_t (&v)[32], int c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]),
                                                                      __uint_as_float(v[e + 1])),
                                                              scale2, sub2));
                            const float w0 = ex2_approx(x.x), w1 = ex2_approx(x.y);
                            sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2_pack(w0, w1));
                            pk[e / 2] = pack_bf16x2(w0, w1);
                        }
                        tmem_st16(tl + s_col + c * 16, pk);
                    };
                    weights(s[0], 0);
                    tmem_ld32(tl + s_col + 64, s[0]);
                    weights(s[1], 1);
                    tmem_ld_wait();
                    mask(s[0], vis[2]);
                    weights(s[0], 2);
                    weights(u, 3);
                    const float2 sa = f2_unpack(f2_add(sum[0], sum[1]));
                    l += sa.x + sa.y;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[st]);
            }
            if (!ok) break;
            // the part's result
            const bool mine = t_first < p.t1;  // this stream had a tile
            if (mine) {
                const bool got = mbar_wait(&pv_done[st], (it - 1) & 1, abort_flag, err, kDevTimeoutEpilogue);
                if (!__all_sync(0xffffffffu, got)) break;
                tc_fence_after();
            }
            // columns [c0, c1) of O are this warp's to write; f and g scale this
            // stream's O and the other's
            int c0 = 0, c1 = D / 16;
            float f = 1.f, g = 0.f;
            bool other = false;
            if (NM == 1) {
                // A stream without a tile in this part must not run ahead: its
                // arrival here could complete x_full's next phase before the
                // other stream has waited for this one.  Both have once the
                // part before is read out.
                if (part > 0) {
                    const bool got = mbar_wait(&o_empty[st], (part - 1) & 1, abort_flag, err, kDevTimeoutEpilogue);
                    if (!__all_sync(0xffffffffu, got)) break;
                }
                float2* mlp = xch + ((part & 1) * 2 + st) * kTile + lq * 32 + lane;
                *mlp = make_float2(ref, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x_full[st]);
                const bool got = mbar_wait(&x_full[st ^ 1], part & 1, abort_flag, err, kDevTimeoutEpilogue);
                if (!__all_sync(0xffffffffu, got)) break;
                tc_fence_after();
                const float2 ml = xch[((part & 1) * 2 + (st ^ 1)) * kTile + lq * 32 + lane];
                const float M = fmaxf(ref, ml.x);
                f = ref == -INFINITY ? 0.f : ex2_approx(ref - M);
                g = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                l = l * f + ml.y * g;
                ref = M;
                other = st == 1 || p.t1 - p.t0 > 1;
                c0 = st * (D / 32);
                c1 = c0 + D / 32;
            }
            if (warp_live) {
                const bool whole = p.whole();
                if (whole) {
                    const float inv = l != 0.f ? 1.f / l : 0.f;  // 0: nothing seen
                    f *= inv;
                    g *= inv;
                }
                __nv_bfloat16* o = a.out + (static_cast<long long>(p.b) * a.ta.T * a.Hq + row) * D;
                // slot 0: a part that ends its unit, slot 1: one that another CTA continues
                const long long sl = 2 * static_cast<long long>(blockIdx.x) + (p.t1 == p.w.tiles ? 0 : 1);
                float* w = a.ws + sl * (kWsRows * (D + 2)) + rt * kTile + lq * 32 + lane;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    uint32_t v[16], u[16];
                    if (mine) tmem_ld16(tl + o_col + c * 16, v);
                    if (other) tmem_ld16(tl + (256 + (st ^ 1) * 128) + c * 16, u);
                    tmem_ld_wait();
                    float r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        r[e] = mine ? __uint_as_float(v[e]) * f : 0.f;
                        if (other) r[e] = fmaf(__uint_as_float(u[e]), g, r[e]);
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[(c * 16 + e) * kWsRows] = r[e];
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint4 q;
                            q.x = pack_bf16x2(r[e], r[e + 1]);
                            q.y = pack_bf16x2(r[e + 2], r[e + 3]);
                            q.z = pack_bf16x2(r[e + 4], r[e + 5]);
                            q.w = pack_bf16x2(r[e + 6], r[e + 7]);
                            *reinterpret_cast<uint4*>(o + c * 16 + e) = q;
                        }
                    }
                }
                if (!whole && (NM == 2 || st == 0)) {
                    w[D * kWsRows] = ref;
                    w[(D + 1) * kWsRows] = l;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&o_empty[st]);
                if (NM == 1) mbar_arrive(&o_empty[st ^ 1]);
            }
            ++part;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of a (sequence, row-tile group) that several CTAs computed:
//   M = max m_i;  o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// Blocks z take the z-th unit that the notes name, 32 of its rows (lanes) and
// kJoinCols columns; a block's warps share the parts out and add up in shared
// memory, in a fixed order.  One warp looks for the unit, through the L1: all
// warps of all blocks asking the L2 for the same few notes took 20 us.
constexpr int kJoinCols = 16;
constexpr int kJoinWarps = 8;

template <int D, int NM>
__global__ void __launch_bounds__(kJoinWarps * 32)
    k_tree_attn_join(const __grid_constant__ AttnArgs a, int ctas) {
    constexpr int GROUP_ROWS = NM * kTile;
    __shared__ float acc_s[kJoinWarps][kJoinCols + 1][32];
    __shared__ float max_s[kJoinWarps][32];
    __shared__ int unit_s[5];  // b, group, first CTA, last CTA (< 0: no such unit), rows of the sequence
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    if (warp == 0) {
        // 160 notes at a time, all loads at once (every SM has one)
        constexpr int N = 5;
        int seen = 0;
        bool found = false;
        if (lane == 0) unit_s[3] = -1;
        __syncwarp();
        for (int c = 0; c < ctas && !found; c += 32 * N) {
            int4 n[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = c + 32 * i + lane;
                n[i] = k < ctas ? *reinterpret_cast<const int4*>(a.notes + k) : make_int4(-1, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const unsigned m = __ballot_sync(0xffffffffu, n[i].x >= 0);
                if (n[i].x >= 0 && seen + __popc(m & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.z)) {
                    unit_s[0] = n[i].x;
                    unit_s[1] = n[i].y;
                    unit_s[2] = n[i].z;
                    unit_s[3] = c + 32 * i + lane;
                    unit_s[4] = n[i].w;
                }
                seen += __popc(m);
            }
            found = seen > static_cast<int>(blockIdx.z);
        }
    }
    __syncthreads();
    const int last = unit_s[3];
    if (last < 0) return;
    const int b = unit_s[0], first = unit_s[2], rows = unit_s[4];
    const int wrow = blockIdx.y * 32, row_g = unit_s[1] * GROUP_ROWS + wrow;  // of the unit, of the sequence
    if (row_g >= rows) return;
    auto part = [&](int c) {
        return a.ws + (2 * static_cast<long long>(c) + (c == last ? 0 : 1)) * (kWsRows * (D + 2)) + wrow + lane;
    };
    const int col0 = blockIdx.x * kJoinCols;
    float acc[kJoinCols + 1] = {};
    float M = -INFINITY;  // of this warp's parts; acc is relative to it
    for (int c = first + warp; c <= last; c += kJoinWarps) {
        const float* q = part(c);
        float v[kJoinCols];
        const float ref = __ldcg(q + D * kWsRows), l = __ldcg(q + (D + 1) * kWsRows);
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) v[e] = __ldcg(q + (col0 + e) * kWsRows);
        const float to = fmaxf(M, ref);
        const float f = ref == -INFINITY ? 0.f : ex2_approx(ref - to);
        const float g = M == -INFINITY ? 0.f : ex2_approx(M - to);
        M = to;
        acc[kJoinCols] = acc[kJoinCols] * g + l * f;
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) acc[e] = fmaf(v[e], f, acc[e] * g);
    }
    max_s[warp][lane] = M;
#pragma unroll
    for (int e = 0; e <= kJoinCols; ++e) acc_s[warp][e][lane] = acc[e];
    __syncthreads();
    // warp e adds up columns 2 e and 2 e + 1; every warp needs the weights' sum
    float all = -INFINITY;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) all = fmaxf(all, max_s[i][lane]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
        const float m = max_s[i][lane], f = m == -INFINITY ? 0.f : ex2_approx(m - all);
        l = fmaf(acc_s[i][kJoinCols][lane], f, l);
        o0 = fmaf(acc_s[i][2 * warp][lane], f, o0);
        o1 = fmaf(acc_s[i][2 * warp + 1][lane], f, o1);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;  // 0: nothing seen
    __syncthreads();
    reinterpret_cast<uint32_t*>(acc_s)[lane * kJoinWarps + warp] = pack_bf16x2(o0 * inv, o1 * inv);
    __syncthreads();
    // 16 columns of 32 rows: 32 bytes a row, two threads
    const int r = threadIdx.x >> 1, h = threadIdx.x & 1;
    if (r < 32 && row_g + r < rows)
        *reinterpret_cast<uint4*>(a.out + (static_cast<long long>(b) * a.ta.T * a.Hq + row_g + r) * D + col0 +
                                  8 * h) =
            *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(acc_s) + r * kJoinWarps + 4 * h);
}
static_assert(kJoinCols == 2 * kJoinWarps && kJoinWarps == 8, "two columns per warp, 32 bytes per row");

template <int D, int NM>
int launch(ic_ctx* ctx, const AttnArgs& a, const void* Q, int kv_len, cudaStream_t s) {
    using S = AttnTile<D, NM>;
    static PerDeviceOnce attr_once;
    cudaError_t e = attr_once.run(ctx->device, [] {
        return cudaFuncSetAttribute(k_tree_attn<D, NM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::SMEM);
    });
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaFuncSetAttribute(tree_attn)");
    CUtensorMap tq, tk, tv;
    const uint64_t rows = static_cast<uint64_t>(a.B) * a.ta.T * a.Hq;
    const uint64_t stride = a.B > 1 ? a.kv_stride : static_cast<uint64_t>(kv_len) * D;
    int rc = make_tmap_bf16_2d(ctx, &tq, Q, rows, D, kTile);
    if (rc == IC_OK) rc = make_tmap_bf16_3d(ctx, &tk, a.K, a.B, kv_len, D, stride, kTile);
    if (rc == IC_OK) rc = make_tmap_bf16_3d(ctx, &tv, a.V, a.B, kv_len, D, stride, kTile);
    if (rc) return rc;
    // no more CTAs than the longest caches could have key tiles
    const int row_max = a.ta.T * a.Hq, groups = (row_max + NM * kTile - 1) / (NM * kTile);
    const long long keys = a.idx ? a.k + a.ta.T : kv_len;
    if (!line_fits(a.B, groups, keys))
        return fail(ctx, IC_ERR_UNSUPPORTED, "tree_attn: B=%d sequences of up to %lld keys are too many",
                    a.B, keys);
    const int tiles = static_cast<int>((keys + kTile - 1) / kTile);
    const long long units = static_cast<long long>(a.B) * groups, most = units * tiles;
    // one tile a unit: nothing to cut or to join.  (From two on, cutting pays:
    // three tiles took 11.9 us in one CTA, 10.6 us in three and a join.)
    const bool cut = tiles > 1 || units > ctx->num_sms;
    const int grid = !cut ? static_cast<int>(units)
                          : most < ctx->num_sms ? static_cast<int>(most) : ctx->num_sms;
    {
        LaunchScope ls(ctx, IC_K_TREE_ATTN, s);
        k_tree_attn<D, NM><<<grid, S::THREADS, S::SMEM, s>>>(tq, tk, tv, a);
        e = ls.done();
        if (e != cudaSuccess) return cuda_fail(ctx, e, "tree_attn launch");
    }
    cudaLaunchConfig_t cfg = {};
    // units of several parts: no more than units, nor than CTAs
    cfg.gridDim = dim3(D / kJoinCols, (row_max < NM * kTile ? row_max + 31 : NM * kTile) / 32,
                       static_cast<unsigned>(units < grid ? units : grid));
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LaunchScope ls(ctx, IC_K_TREE_ATTN, s);
    cudaLaunchKernelEx(&cfg, k_tree_attn_join<D, NM>, a, grid);
    e = ls.done();
    if (e != cudaSuccess) return cuda_fail(ctx, e, "tree_attn join launch");
    return IC_OK;
}

}  // namespace

extern "C" int ic_tree_attn(ic_ctx* ctx, const void* Q, const void* K, const void* V,
                            const int32_t* idx, const int32_t* prefix_len, const int32_t* draft_len,
                            const uint64_t* tree_mask, int B, int T, int Hq, int d, int k,
                            int64_t kv_seq_stride, int kv_len, float scale, void* out,
                            void* stream) {
    if (!ctx) return fail(nullptr, IC_ERR_INVALID_ARG, "context is NULL");
    if (B < 0 || B > 65535 || T < 1 || Hq < 1 || Hq > 16 || kv_len < 1 || (idx ? (k < 1 || k > 2048) : k != 0))
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
    // (sequences of one call may finish in any order)
    const long long q_bytes = static_cast<long long>(B) * T * Hq * d * 2;
    const long long kv_bytes = ((B - 1ll) * kv_seq_stride + static_cast<long long>(kv_len) * d) * 2;
    const Span o(out, q_bytes);
    if (o.meets(Span(Q, q_bytes)) || o.meets(Span(K, kv_bytes)) || o.meets(Span(V, kv_bytes)))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree_attn: out overlaps Q, K or V");
    // (every warp reads the lengths for itself: they must not change meanwhile)
    if (o.meets(Span(prefix_len, B * 4ll)) || (idx && o.meets(Span(idx, static_cast<long long>(B) * k * 4))) ||
        (draft_len && o.meets(Span(draft_len, B * 4ll))) ||
        (tree_mask && o.meets(Span(tree_mask, static_cast<long long>(B) * T * 8))))
        return fail(ctx, IC_ERR_INVALID_ARG, "tree_attn: out overlaps the lengths, the mask or the list");
    if (!(scale > 0.f)) scale = 1.0f / sqrtf(static_cast<float>(d));
    DeviceGuard guard(ctx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const TreeArgs ta{prefix_len, draft_len, reinterpret_cast<const unsigned long long*>(tree_mask),
                      T, kv_len};
    // fixed workspace: two slots of partial sums and a note per CTA
    const size_t slots = static_cast<size_t>(ctx->num_sms) * 2 * kWsRows * (128 + 2) * sizeof(float);  // 16-byte multiple
    const size_t ws = slots + static_cast<size_t>(ctx->num_sms) * sizeof(JoinNote);
    int rc = ensure_buffer_on(ctx, s, reinterpret_cast<void**>(&ctx->tree_ws), &ctx->tree_ws_cap, ws,
                              nullptr);
    if (rc) return rc;
    AttnArgs a;
    a.line = TreeLine{ta, idx ? k : -1, Hq, (T * Hq <= kTile ? 1 : 2) * kTile};
    a.ta = ta;
    a.idx = idx;
    a.K = static_cast<const __nv_bfloat16*>(K);
    a.V = static_cast<const __nv_bfloat16*>(V);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ws = ctx->tree_ws;
    a.notes = reinterpret_cast<JoinNote*>(reinterpret_cast<char*>(ctx->tree_ws) + slots);
    a.err = ctx->dev_err;
    a.kv_stride = kv_seq_stride;
    a.B = B;
    a.Hq = Hq;
    a.k = k;
    a.scale_log2 = scale * 1.4426950408889634f;
    if (T * Hq <= kTile)
        return d == 128 ? launch<128, 1>(ctx, a, Q, kv_len, s) : launch<64, 1>(ctx, a, Q, kv_len, s);
    return d == 128 ? launch<128, 2>(ctx, a, Q, kv_len, s) : launch<64, 2>(ctx, a, Q, kv_len, s);
}
