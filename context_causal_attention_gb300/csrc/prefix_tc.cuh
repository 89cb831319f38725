// prefix_tc.cuh -- the shared-prefix attention's kernel for many rows: tiles of
// 2 x 128 rows on tcgen05 (S and O in tensor memory, K and V pages by TMA).
//
// One block on an SM works through its share of the line (cp_prefix.cuh) with
// 12 warps:
//   warps 0, 2  loads of K and of V: the page numbers of 32 pages side by side in
//               the lanes, the next 32 on their way; pages of 64 tokens or more
//               by TMA (64 columns x a page's rows a copy), smaller ones by
//               cp.async (cp_prefix.cuh), into a ring of stages.  A page number
//               out of range becomes a coordinate outside the tensor, which TMA
//               fills with zeros.
//               Warp 2 also gathers Q: the rows of a tile are query heads of one
//               KV head from one or many sequences (16-byte cp.async, swizzled).
//   warps 1, 3  MMA issue of the two halves: S_i = Q_i K^T, O_i += P_i V with P_i
//               in tensor memory (512 columns: S0 | S1 | O0 | O1).
//   warps 4-7   softmax of rows 0..127, warps 8-11 of rows 128..255: one thread
//               a row, in the log2 domain with an integer running maximum that
//               moves only when a tile's sum passes 2^64 (as in attn.cu).
// The two halves keep the tensor cores and the exponentials busy in turn.  In a
// tile of up to 128 rows both hold the same rows and take the key tiles in turn;
// the first half joins the two results at the end (with one half alone the scores,
// the exponentials and the second product of a tile follow one another: 35 rows
// ran at half of this speed).
// Keys past the problem's length lie in a page's tail or in pages that were not
// loaded: their scores become -inf, and their V rows are zeros before the product
// reads them (zeroed in shared memory behind TMA, never copied by cp.async), so
// nothing that they hold (NaN included) is multiplied.
//
// What bounds it: the chain of a tile's scores, exponentials and second product, in
// which each half is one step behind the other.  8 ragged prompts of up to 1024
// tokens, 32 heads of 128, over 16384 shared keys (1.48 TFLOP): 1066 us for this
// launch, 1.39 PFLOP/s, the tensor pipe 58% active.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_prefix.cuh"
#include "cp_ptx.cuh"
#include "cp_softmax.cuh"

namespace cpattn {
namespace {

constexpr int kTcThreads = 384;
// Pages of this many tokens or more are copied by TMA, smaller ones by cp.async
// (see copy_tile).  64 rows over 32768 keys in pages of 16 take 62.6 us by TMA and 60.5
// by cp.async; prompts over pages of 64 359.5 by TMA and 367.7 by cp.async.
constexpr int kTmaPage = 64;

template <int D>
struct TcCfg {
    static constexpr int kAtom = 128 * 128;  // 128 rows x 64 columns
    static constexpr int kAtoms = D / 64;
    static constexpr int kTile = kAtom * kAtoms;
    // Stages of K and of V: a third of K (D = 128) or six of both (D = 64) measured the same.
    static constexpr int kStagesK = D == 128 ? 2 : 4, kStagesV = D == 128 ? 2 : 4;
    // even: a stage then serves the same half through a piece whose halves take turns
    static_assert(kStagesK % 2 == 0 && kStagesV % 2 == 0, "stages");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + kStagesK * kTile;
    static constexpr int kOffLine = kOffV + kStagesV * kTile;
    static constexpr int kOffStart = (kOffLine + static_cast<int>(sizeof(Line)) + 15) & ~15;
    static constexpr int kOffBar = (kOffStart + static_cast<int>(sizeof(Start)) + 15) & ~15;
    // q_full[2], s_full[2], p_full[2], o_full[2], o_empty[2], drain[2], ml_full, q_empty, turn[2], k_full[], v_full[], k_empty[], v_empty[]
    static constexpr int kWalks = kTcThreads / 32;
    static constexpr int kBars = 16 + 2 * (kStagesK + kStagesV);
    static constexpr int kOffMisc = kOffBar + kBars * 8;
    static_assert(kOffMisc % 16 == 0, "tensor memory's address is left on 16 bytes");
    static constexpr int kOffMl = (kOffMisc + 16 + 15) & ~15;        // [128] (m, l) of the second half
    static constexpr int kOffWalk = kOffMl + 128 * 8;   // [warps]
    static constexpr int kSmem = kOffWalk + kWalks * static_cast<int>(sizeof(Walk<kTcTM, kTcKT>)) + 1024;  // + alignment slack
    static_assert(kSmem <= 232448, "shared memory budget");
};

__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Scores of columns c0 .. c0+63 that the row does not see (column >= lim) become -inf.
__device__ __forceinline__ void hide_columns(int c0, int lim, uint32_t (&h)[64]) {
#pragma unroll
    for (int c = 0; c < 64; ++c)
        if (c0 + c >= lim) h[c] = 0xff800000u;
}

// One lane of the warp (non-zero there), the same at every call.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// D (+)= A B, one K step of 16, A and B in shared memory; takes effect where `lead`.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(lead)
        : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint64_t db, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(ta), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(lead)
        : "memory");
}
// umma_commit where `lead`.
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

// Starts the gather of 128 rows of a piece, the first of them row0, into a Q tile
// swizzled as TMA would (zeros behind the piece's rows).  By one warp.
template <int D, int kAtom>
__device__ __forceinline__ void copy_queries(const PrefixArgs &a, const Piece &x, int row0, uint32_t tile, int lane) {
    constexpr int kChunks = D / 8, kRpi = 32 / kChunks;  // 16-byte chunks of a row, rows of an instruction
    const int c = lane % kChunks, r0 = lane / kChunks;
    const uint32_t dst = tile + (c >> 3) * kAtom + r0 * 128;
#pragma unroll 1
    for (int g = 0; g < 128; g += 32) {
        // element offset of row g + lane, handed to the lanes that copy it
        const int row = row0 + g + lane, tok = static_cast<int>(fdiv(static_cast<uint32_t>(row), a.div_g));
        const long long mine =
            row < x.rows ? (static_cast<long long>(x.tok0 + tok) * a.N + x.kvh * a.G + row - tok * a.G) * D : -1;
#pragma unroll 8
        for (int j = 0; j < 32 / kRpi; ++j) {
            const long long at = __shfl_sync(0xffffffffu, mine, j * kRpi + r0);
            const uint32_t to = dst + (g + j * kRpi) * 128 + (((c & 7) ^ ((j * kRpi + r0) & 7)) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                         "l"(a.q + (at < 0 ? 0 : at + c * 8)), "r"(at < 0 ? 0 : 16)
                         : "memory");
        }
    }
}

// Barriers of a block's pipeline.  By one thread; a __syncthreads follows in tc_work.
template <int D, bool tma>
__device__ __forceinline__ void tc_init(uint8_t *smem, const CUtensorMap &tmK, const CUtensorMap &tmV) {
    using C = TcCfg<D>;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bar, *s_full = bar + 2, *p_full = bar + 4, *o_full = bar + 6, *o_empty = bar + 8;
    uint64_t *drain = bar + 10, *ml_full = bar + 12, *q_empty = bar + 13, *turn = bar + 14, *k_full = bar + 16,
             *v_full = k_full + C::kStagesK, *k_empty = v_full + C::kStagesV, *v_empty = k_empty + C::kStagesK;
    *reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4) = 0;  // abort flag
    for (int i = 0; i < 2; ++i) {
        mbar_init(q_full + i, 32);
        mbar_init(s_full + i, 1);
        mbar_init(p_full + i, 4);
        mbar_init(o_full + i, 1);
        mbar_init(o_empty + i, 4);
        mbar_init(drain + i, 1);
        mbar_init(turn + i, 4);
    }
    mbar_init(ml_full, 4);
    mbar_init(q_empty, 2);  // the MMA warps, each when it has seen that its half's products with Q are done
    for (int s = 0; s < C::kStagesK; ++s) {
        mbar_init(k_full + s, tma ? 1 : 32);
        mbar_init(k_empty + s, 2);
    }
    for (int s = 0; s < C::kStagesV; ++s) {
        mbar_init(v_full + s, tma ? 1 : 32);
        mbar_init(v_empty + s, 2);
    }
    fence_mbar_init();
    if (tma) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
}

// A block's share, behind the scan of its line.  tma: the pages are copied by TMA,
// else by cp.async.
template <int D, bool tma>
__device__ __forceinline__ void tc_work(const CUtensorMap &tmK, const CUtensorMap &tmV, const PrefixArgs &a,
                                        uint8_t *smem) {
    using C = TcCfg<D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Line &line = *reinterpret_cast<Line *>(smem + C::kOffLine);
    Start &start = *reinterpret_cast<Start *>(smem + C::kOffStart);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bar, *s_full = bar + 2, *p_full = bar + 4, *o_full = bar + 6, *o_empty = bar + 8;
    uint64_t *drain = bar + 10, *ml_full = bar + 12, *q_empty = bar + 13, *turn = bar + 14, *k_full = bar + 16, *v_full = k_full + C::kStagesK,
             *k_empty = v_full + C::kStagesV, *v_empty = k_empty + C::kStagesK;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    long long t0, t1;
    if (!share_of(a, line, &t0, &t1)) return;
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == 0) find_start<kTcTM, kTcKT>(a, line, t0, &start);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t *sQ = smem + C::kOffQ, *sK = smem + C::kOffK, *sV = smem + C::kOffV;

    Walk<kTcTM, kTcKT> &walk = reinterpret_cast<Walk<kTcTM, kTcKT> *>(smem + C::kOffWalk)[warp];
    const Piece &x = walk.x;
    walk.begin(a, line, start, t1 - t0);
    if (warp == 0 || warp == 2) {
        // -------------------------------------------------------- loads: K by warp 0, Q and V by warp 2
        const CUtensorMap *map = warp ? &tmV : &tmK;
        uint64_t *full = warp ? v_full : k_full, *empty = warp ? v_empty : k_empty;
        uint8_t *ring = warp ? sV : sK;
        const uint32_t stages = warp ? C::kStagesV : C::kStagesK;
        uint32_t st = 0, ph = 0;  // stage and phase of tile `it`
        const int shift = a.own.shift, rows = min(kTcKT, 1 << shift);  // rows of a copy
        uint32_t it = 0, items = 0;
        bool ok = warp != 0 || released(a, abort_flag);
        while (ok && walk.next(a, line)) {
            if (x.k0 >= x.k1) continue;
            if (warp == 2) {
                // Q, gathered: the last piece's scores have all been computed, and its V has
                // landed (its K has, or they would not)
                if (items && !mbar_wait_warp(q_empty, (items - 1) & 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                for (uint32_t i = it > stages ? it - stages : 0; i < it && ok; ++i)
                    ok = mbar_wait_warp(full + i % stages, (i / stages) & 1u, abort_flag, a.timeout_ns);
                if (!ok) break;
                ++items;
                for (int i = 0; i < 2 && x.row0 + i * 128 < x.rows; ++i) {
                    copy_queries<D, C::kAtom>(a, x, x.row0 + i * 128, smem_u32(sQ) + i * C::kTile, lane);
                    copies_arrive(q_full + i);
                }
            }
            PageWindow win;
            win.begin(a, x, (x.k0 * kTcKT) >> shift, lane);
            for (int kt = x.k0; kt < x.k1; ++kt, ++it) {
                const int key = kt * kTcKT;
                win.advance(key >> shift, lane);
                const int n = (min(kTcKT, x.keys - key) + rows - 1) / rows;
                if (it) {
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (!mbar_wait_warp(empty + st, ph ^ 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                if (!tma) {
                    copy_tile<D, kTcKT, C::kAtom>(a, x, win, warp ? a.v : a.k, smem_u32(ring) + st * C::kTile, key, lane);
                    copies_arrive(full + st);
                    continue;
                }
                if (lane == 0) mbar_arrive_expect_tx(full + st, n * rows * 128 * C::kAtoms);
                for (int i = 0; i < n; ++i) {
                    const int row = win.row(a, key + i * rows);
                    if (lane == 0)
#pragma unroll
                        for (int at = 0; at < C::kAtoms; ++at)
                            tma_load_4d(ring + st * C::kTile + at * C::kAtom + i * rows * 128, map, full + st, 64 * at,
                                        x.kvh, row, 0);
                }
            }
        }
        copies_drain();
        if (tma && lane == 0) {
            // Every copy already issued lands before shared memory goes away, also where this
            // warp has issued all of its own and a wait of another warp ends the block.
            volatile int no_abort = 0;
            for (uint32_t i = it > stages ? it - stages : 0; i < it; ++i)
                mbar_wait(full + i % stages, (i / stages) & 1u, &no_abort, 100000000ull);
        }
        __syncwarp();
    } else if (warp < 4) {
        // -------------------------------------------------------- MMA issue: half 0 by warp 1, half 1 by warp 3
        // One warp for both halves spent 1000 cycles on the instructions of a half's
        // tile (waits, 8 + 8 MMAs, commits) and was what a tile waited for.  The warp
        // runs whole and one lane's instructions take effect, so that the operands
        // stay in uniform registers.
        const int i = warp >> 1;
        const uint32_t lead = elect_lane();
        const uint32_t tS = tmem + i * 128, tP = tS + 64, tO = tmem + 256 + i * D;
        constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0), kIdescPV = idesc_bf16_f32(128, D, 0, 1);
        constexpr uint64_t kStageDesc = C::kTile >> 4;
        const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv = smem_desc_sw128(smem_u32(sV), C::kAtom, 1024);
        uint32_t kv = 0, items = 0, tiles = 0, pieces = 0, wide = 0;  // wide: pieces of more than 128 rows
        bool ok = true;
        while (ok && walk.next(a, line)) {
            const int n = x.k1 - x.k0;
            if (n <= 0) continue;
            // up to 128 rows: the halves take the key tiles in turn, both with Q's first tile
            const bool paired = x.rows - x.row0 <= 128;
            const int begin = paired ? i : 0, step = paired ? 2 : 1;
            const uint32_t base = kv;
            kv += n;
            // The waits that do not hang on the softmax come first, so that the
            // products follow its weights at once.
            auto v_wait = [&](uint32_t at) -> bool {
                return mbar_wait_warp(v_full + at % C::kStagesV, (at / C::kStagesV) & 1u, abort_flag, a.timeout_ns);
            };
            // O (+)= P V of tile `at`
            auto pv = [&](uint32_t at, bool first) -> bool {
                const uint32_t st = at % C::kStagesV;
                if (first && !mbar_wait_warp(o_empty + i, (items & 1u) ^ 1u, abort_flag, a.timeout_ns)) return false;
                if (!mbar_wait_warp(p_full + i, tiles & 1u, abort_flag, a.timeout_ns)) return false;
                tc_fence_after();
                ++tiles;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(tO, tP + 8 * k, dv + st * kStageDesc + 128 * k, kIdescPV, !first || k > 0, lead);
                commit(v_empty + st, lead);
                if (paired) commit(v_empty + st, lead);  // for the other half
                return true;
            };
            // Also with no tile for this half (a piece of one tile): Q of a piece is
            // loaded when both halves are done with the last one's, so that neither
            // waits for a stage or a query tile more than one phase ahead, where the
            // parity would tell it the opposite.
            if (!mbar_wait_warp(q_full, pieces++ & 1u, abort_flag, a.timeout_ns) ||
                (!paired && i && !mbar_wait_warp(q_full + 1, wide++ & 1u, abort_flag, a.timeout_ns))) {
                ok = false;
                break;
            }
            if (begin < n) {
                const uint64_t dqi = dq + (paired ? 0 : i) * kStageDesc;
                for (int j = begin; j < n && ok; j += step) {
                    const uint32_t st = (base + j) % C::kStagesK, ph = ((base + j) / C::kStagesK) & 1u;
                    if (!mbar_wait_warp(k_full + st, ph, abort_flag, a.timeout_ns) || (j > begin && !v_wait(base + j - step))) {
                        ok = false;
                        break;
                    }
                    fence_async_shared();  // Q (and without TMA K and V) was written by cp.async
                    if (j > begin && !pv(base + j - step, j == begin + step)) { ok = false; break; }
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(tS, dqi + (k / 4) * (C::kAtom >> 4) + (k % 4) * 2,
                               dk + st * kStageDesc + (k / 4) * (C::kAtom >> 4) + (k % 4) * 2, kIdescQK, k > 0, lead);
                    commit(s_full + i, lead);
                    commit(k_empty + st, lead);
                    if (paired) commit(k_empty + st, lead);  // for the other half
                }
                // Q has been read when the last scores are there.  (The weights that this warp
                // waits for next come after them.  Against a commit on q_empty in this place: 300
                // sequences of 30 tokens 174 and 171 us, 64 of 20 behind 16384 keys 312 and 312.)
                if (!ok || !mbar_wait_warp(s_full + i, tiles & 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                if (lane == 0) mbar_arrive(q_empty);
                const int last = begin + (n - 1 - begin) / step * step;
                if (!v_wait(base + last)) { ok = false; break; }
                fence_async_shared();
                if (!pv(base + last, last == begin)) { ok = false; break; }
                commit(o_full + i, lead);
                ++items;
            } else if (lane == 0) {
                // it multiplied nothing here and has nothing to wait for
                mbar_arrive(q_empty);
            }
        }
        // no MMA may still be running when tensor memory is released
        commit(drain + i, lead);
        volatile int no_abort = 0;
        mbar_wait(drain + i, 0, &no_abort, 100000000ull);
        __syncwarp();
    } else if (warp >= 4) {
        // -------------------------------------------------------- softmax
        const int half = (warp - 4) >> 2, in_tile = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + half * 128, tO = tmem + lane_off + 256 + half * D;
        const float sl2 = a.scale_log2;
        float2 *ml_s = reinterpret_cast<float2 *>(smem + C::kOffMl);
        uint32_t tiles = 0, items = 0, kv = 0, joins = 0, other = 0;  // other: items of the other half
        bool ok = true;
        // The first pass through the code of a tile is made on what tensor memory
        // happens to hold, while the first copies are under way: read cold, that
        // code took 8000 cycles, four times a tile's time.  Nothing is written in it and
        // no barrier touched.
        bool dry = true;
        // The first half's k-th turn (k > 0) follows the second half's turn k - 1,
        // which follows the first half's.
        uint32_t turns = half ? 0u : 0xffffffffu;
        auto my_turn = [&]() -> bool {
            const uint32_t k = turns++;
            return k == 0xffffffffu || mbar_wait_warp(turn + half, k & 1u, abort_flag, a.timeout_ns);
        };
        auto pass_turn = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(turn + (half ^ 1));
        };
        while (ok && walk.next(a, line)) {
            // up to 128 rows: both halves hold the same rows, tile j of the piece is half j & 1's
            const bool paired = x.rows - x.row0 <= 128;
            const int first_row = x.row0 + (paired ? 0 : half * 128), row = first_row + in_tile, all = x.k1 - x.k0;
            const bool valid = row < x.rows, write = valid && x.slot >= 0 && !(paired && half);
            const long long at = static_cast<long long>(max(x.slot, 0)) * kTcTM + row - x.row0;
            if (x.slot < 0 && in_tile == 0) report(a.status, CP_ERR_PAGE);
            if (all <= 0) {
                if (write) a.slot_ml[at] = make_float2(-INFINITY, 0.f);
                continue;
            }
            const int begin = paired ? half : 0, step = paired ? 2 : 1;
            uint32_t tile = kv + begin;
            kv += all;
            if (begin >= all) {  // one tile: nothing for the second half but its turn
                if (!my_turn()) { ok = false; break; }
                pass_turn();
                continue;
            }
            // counted from the current tile: keys of the problem, that this row sees, that all rows see
            int past = x.keys - (x.k0 + begin) * 128;
            int limit = (valid ? row_limit(a, x, row) : x.keys) - (x.k0 + begin) * 128;
            int whole = row_limit(a, x, first_row) - (x.k0 + begin) * 128;
            float m_run = -INFINITY, l_run = 0.f;
            for (int n = begin; n < all;) {
                if (!dry && !mbar_wait_warp(s_full + half, tiles & 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                // The halves take turns at the exponentials: left alone they fall into
                // step, and the tensor cores wait while both compute and the other way round.
                if (!dry && !my_turn()) { ok = false; break; }
                tc_fence_after();
                const bool mask = whole < 128;
                const int lim = limit;
                uint32_t sa[64], sb[64], pa[32], pb[32];
                tmem_ld64_nowait(tS, sa);
                tmem_wait_ld(sa);
                tmem_ld64_nowait(tS + 64, sb);
                if (mask) hide_columns(0, lim, sa);
                const bool first = !__all_sync(0xffffffffu, m_run != -INFINITY);
                if (first) {
                    // rows without a running maximum yet: set it
                    tmem_wait_ld(sb);
                    if (mask) hide_columns(64, lim, sb);
                    if (m_run == -INFINITY) {
                        const float top = row_max128(sa, sb) * sl2;
                        if (top > -INFINITY) m_run = ceilf(top);
                    }
                }
                const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
                const float s0 = exp_pack64(sa, sl2, neg_m, pa);
                tmem_wait_ld(sb);  // columns 64..127 are read: P may overwrite them
                if (!dry) tmem_st32_nowait(tS + 64, pa);
                if (mask && !first) hide_columns(64, lim, sb);
                const float s1 = exp_pack64(sb, sl2, neg_m, pb);
                if (!dry) tmem_st32_nowait(tS + 96, pb);
                float sum = s0 + s1;
                const bool big = !(sum <= 0x1p64f);  // also for inf and NaN
                if (!dry) pass_turn();
                tmem_wait_st();
                if (__any_sync(0xffffffffu, big) && !dry) {
                    // rare: the scores grew by more than 2^64 over the running maximum.
                    // Columns 0..63 of S are still in tensor memory, 64..127 in sb.
                    tmem_ld64(tS, sa);
                    if (mask) hide_columns(0, lim, sa);
                    float f = 1.f;
                    if (big) {
                        const float m_new = ceilf(row_max128(sa, sb) * sl2), d = m_run - m_new;
                        f = d >= -126.f ? __int_as_float((127 + static_cast<int>(d)) << 23) : 0.f;
                        l_run *= f;
                        m_run = m_new;
                    }
                    exp_pack128(sa, sb, sl2, m_run == -INFINITY ? 0.f : -m_run, pa, pb, &sum);
                    tmem_st64(tS + 64, pa, pb);
                    // O is quiet: this tile's product waits for p_full below.  Before a
                    // piece's first product (NaN or infinite scores) it is still the last
                    // piece's, which the first half may be joining.
#pragma unroll
                    for (int c0 = 0; c0 < D && n != begin; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32(tO + c0, ov);
#pragma unroll
                        for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f);
                        tmem_st32(tO + c0, ov);
                    }
                }
                l_run += sum;
                tc_fence_before();
                __syncwarp();
                if (dry) {
                    dry = false;
                    m_run = -INFINITY;
                    l_run = 0.f;
                    continue;
                }
                if (tma && past < 128) {
                    // The scores of this tile came after the product of the stage's last tile was
                    // issued, so that one's V has landed: the wait is for this tile's phase.
                    const uint32_t st = tile % C::kStagesV, ph = (tile / C::kStagesV) & 1u;
                    if (!mbar_wait_warp(v_full + st, ph, abort_flag, a.timeout_ns)) { ok = false; break; }
                    if (in_tile >= past) {
                        uint8_t *dst = sV + st * C::kTile + in_tile * 128;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kAtom + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_shared();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + half);
                n += step;
                tile += step;
                ++tiles;
                past -= 128 * step;
                limit -= 128 * step;
                whole -= 128 * step;
            }
            // a piece of an odd number of tiles: the second half's last turn is empty
            if (ok && paired && half && (all & 1)) {
                ok = my_turn();
                pass_turn();
            }
            if (!ok || !mbar_wait_warp(o_full + half, items & 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
            tc_fence_after();
            ++items;
            if (paired && half) {
                // the first half joins the two; this thread's row is the same lane of tensor memory there
                ml_s[in_tile] = make_float2(m_run, l_run);
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
                continue;
            }
            const bool join = paired && all > 1;
            float f0 = 1.f, f1 = 0.f;
            if (join) {
                if (!mbar_wait_warp(ml_full, joins++ & 1u, abort_flag, a.timeout_ns) ||
                    !mbar_wait_warp(o_full + 1, other & 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                tc_fence_after();
                const float2 other = ml_s[in_tile];
                const float m = fmaxf(m_run, other.x);
                f0 = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m);
                f1 = other.x == -INFINITY ? 0.f : fast_exp2(other.x - m);
                l_run = f0 * l_run + f1 * other.y;
                m_run = m;
            }
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t ov[32], ow[32];
                tmem_ld32(tO + c, ov);
                if (join) {
                    tmem_ld32(tO + D + c, ow);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ov[e] = __float_as_uint(f0 * __uint_as_float(ov[e]) + f1 * __uint_as_float(ow[e]));
                }
                if (c + 32 == D) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_empty + half);
                    if (lane == 0 && join) mbar_arrive(o_empty + 1);
                }
                if (write) {
                    float *dst = a.slot_o + at * D + c;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        st_global_v8(dst + e, __uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), __uint_as_float(ov[e + 2]),
                                     __uint_as_float(ov[e + 3]), __uint_as_float(ov[e + 4]), __uint_as_float(ov[e + 5]),
                                     __uint_as_float(ov[e + 6]), __uint_as_float(ov[e + 7]));
                }
            }
            if (write) a.slot_ml[at] = left_ml(m_run, l_run);
            if (!paired || join) ++other;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *abort_flag) report(a.status, CP_ERR_DEVICE_TIMEOUT);
}

template <int D, bool tma>
__global__ void __launch_bounds__(kTcThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PrefixArgs a) {
    using C = TcCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Line &line = *reinterpret_cast<Line *>(smem + C::kOffLine);
    if (threadIdx.x == 0) tc_init<D, tma>(smem, tmK, tmV);
    // its blocks may have started under the kernels that made its inputs
    wait_for_previous();
    launch_dependents();
    scan_line<kTcTM, kTcKT>(a, line, nullptr, 0);
    if (blockIdx.x == 0 && blockIdx.y == 0) leave_places<kTcTM, kTcKT>(a, line);
    tc_work<D, tma>(tmK, tmV, a, smem);
}

}  // namespace
}  // namespace cpattn
