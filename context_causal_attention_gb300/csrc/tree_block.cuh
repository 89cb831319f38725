// tree_block.cuh -- the tree attention of many sequences: a block takes an item -- up to 64 rows (tokens x the G query
// heads of a KV head) of one sequence -- over all of its keys, and two blocks share an SM.
//
// Items of many sequences are short beside what a block needs before its first key tile and behind its last one
// (lists, page numbers, the first tile's way, the last one's scores and products: 9 us, in which nothing is read).
// Two blocks of half an SM's shared memory and tensor memory cover that for each other, and the GPU deals out the
// items by itself as blocks end, the longest first.  No partials, no workspace, no second launch.  64 sequences of up to
// 4096 keys, 16 tokens of 32 / 8 heads of 128 each: 86 us (77 at the copy's rate for the keys alone; one block of 12 warps an
// SM 113, the line 126), none ragged 166 (161; 211, 217), 300 of up to 500 78 (51; 174, 174).  Where all items run at once a
// tile's chain (scores, weights, product: 0.75 us for 64 keys) bounds it.
//
// Inside: warps 0 and 1 softmax, a thread a row; warp 2 loads K, warp 4 V, by 16-byte cp.async (the softmax warps Q);
// warp 3 issues the products.  S = Q K^T and O += P V on tcgen05 with S, P and O in tensor memory (S0 | S1 | O).
// Rows 64 .. 127 of the product's tile have no place of their own: the matrix reads what lies behind the 64 rows of Q,
// and nobody reads those results.  A tile is 64 keys: its scores fit a thread's registers at once, and the next
// tile's are formed meanwhile (tiles of 128 keys, one buffer: 107 us, none ragged 174).  Two threads a row, each with
// half of a tile's keys, were slower (a sequence's 64 tiles 48 us for 43 at D = 64): what they tell each other costs
// more than the shorter turns save.
// The weights as in tree_cluster.cuh: relative to a maximum of the scores themselves, looked for before they are
// formed and moved only when a weight would pass 2^30.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_prefix.cuh"
#include "cp_ptx.cuh"
#include "cp_softmax.cuh"
#include "prefix_tc.cuh"
#include "tree_cluster.cuh"

namespace cpattn {
namespace {

constexpr int kBlThreads = 160;
constexpr int kBlRows = 64;
constexpr int kBlKeys = 64;  // of a tile

template <int D>
struct BlCfg {
    static constexpr int kAtom = kBlKeys * 128;    // 64 keys x 64 columns
    static constexpr int kAtomQ = kBlRows * 128;   // 64 rows x 64 columns
    static constexpr int kTile = kAtom * (D / 64);
    static constexpr int kStages = D == 128 ? 3 : 6;   // of K and of V
    static constexpr int kOffK = kAtomQ * (D / 64);    // behind Q
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffBar = kOffV + kStages * kTile;
    // q_full, s_full[2], p_full[2], o_full[2], drain, k_full[], k_empty[], v_full[], v_empty[]
    static constexpr int kBars = 8 + 4 * kStages;
    static constexpr int kOffMisc = (kOffBar + kBars * 8 + 15) & ~15;  // tensor memory's address, abort flag
    static constexpr int kSmem = kOffMisc + 16;
    // two blocks on an SM, of whose 228 KB each takes 1 KB more; the matrix reads 64 rows past Q
    static_assert(kSmem + 1024 <= 228 * 1024 / 2 && kStages * kTile >= kAtomQ, "shared memory budget");
};

// Whether the phase of parity `parity` is over, without a wait.
__device__ __forceinline__ bool mbar_test(const uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

struct BlockArgs {
    ClusterArgs c;
    int longest_first;  // the order of the items: the longest sequences' first (B up to kBlThreads)
};

template <int D>
__global__ void __launch_bounds__(kBlThreads, 2) tree_block_kernel(const __grid_constant__ BlockArgs args) {
    const ClusterArgs &c = args.c;
    using C = BlCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const PrefixArgs &a = c.p;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bar, *s_full = bar + 1, *p_full = bar + 3, *o_full = bar + 5, *drain = bar + 7, *k_full = bar + 8,
             *k_empty = k_full + C::kStages, *v_full = k_empty + C::kStages, *v_empty = v_full + C::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int rest = static_cast<int>(blockIdx.x);
    const int kvh = rest % a.Nkv;
    rest /= a.Nkv;
    const int tile0 = rest % c.tiles, place = rest / c.tiles;

    // (the tiles' swizzle counts from 1024-byte boundaries; there is no room to align them here)
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) report(a.status, CP_ERR_ALIGNMENT);
        return;
    }
    if (tid == 0) {
        *abort_flag = 0;
        mbar_init(q_full, 2 * 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 2);
            mbar_init(o_full + i, 1);
        }
        mbar_init(drain, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(k_full + s, 32);
            mbar_init(k_empty + s, 1);
            mbar_init(v_full + s, 32);
            mbar_init(v_empty + s, 1);
        }
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    wait_for_previous();
    launch_dependents();
    // the sequence, as the lists give it (those that make no sense are cut and reported, as in sequence_problem)
    int b = place;
    if (args.longest_first) {
        // the sequence with `place` longer ones (in Q's place, before Q)
        int *lengths = reinterpret_cast<int *>(smem), *found = lengths + kBlThreads;
        // (no two compare equal; beyond 2^22 tokens the order is the index's)
        const int mine = tid < a.B ? min(max(__ldcg(a.kv_len + tid), 0), 1 << 22) << 8 | (255 - tid) : -1;
        lengths[tid] = mine;
        __syncthreads();
        int before = 0;
        for (int i = 0; i < a.B; i += 4) {
            const int4 y = *reinterpret_cast<const int4 *>(lengths + i);
            before += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
        }
        if (tid < a.B && before == place) *found = tid;
        __syncthreads();
        b = *found;
    }
    const int c0 = __ldcg(a.cu + b), c1 = __ldcg(a.cu + b + 1);
    long long length = __ldcg(a.kv_len + b);
    int n = c1 - c0;
    const long long most = static_cast<long long>(a.own.max_pages) << a.own.shift;
    if (c0 < 0 || c1 < c0 || c1 > a.R) {
        n = 0;
        if (tid == 0) report(a.status, CP_ERR_PAGE);
    }
    if (length < 0 || length > most) {
        length = length < 0 ? 0 : most;
        if (tid == 0) report(a.status, CP_ERR_PAGE);
    }
    TreePiece x{};
    x.b = b;
    x.kvh = kvh;
    x.tok0 = c0;
    x.rows = n * a.G;
    x.keys = static_cast<int>(length);
    x.off = x.keys - n;
    x.tree = n <= 32 * a.words ? n : 0;
    const int prefix = static_cast<int>(a.P), prefix_tiles = static_cast<int>((a.P + kBlKeys - 1) / kBlKeys);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t *sK = smem + C::kOffK, *sV = smem + C::kOffV;

    // over all row tiles: tiles of keys so far, queries
    uint32_t kv = 0, queries = 0;
    for (int tile = tile0; tile * kBlRows < x.rows; tile += c.tiles) {
        x.row0 = tile * kBlRows;
        const int rows = min(kBlRows, x.rows - x.row0);
        const int last = x.tree ? x.keys : row_limit(a, x, x.row0 + rows - 1);
        const int tiles = prefix_tiles + (last + kBlKeys - 1) / kBlKeys;
        if (warp == 2 || warp == 4) {
            // -------------------------------------------------------- loads: K by warp 2, V by warp 4
            uint64_t *full = warp == 4 ? v_full : k_full, *empty = warp == 4 ? v_empty : k_empty;
            const __nv_bfloat16 *cache = warp == 4 ? a.v : a.k;
            const uint32_t ring = smem_u32(warp == 4 ? sV : sK);
            PageWindow win{};
            Piece y = x;
            int segment = -1;
            const int loads = tiles && released(a, abort_flag) ? tiles : 0;
            for (int j = 0; j < loads; ++j) {
                const bool pre = j < prefix_tiles;
                const int key = (j - (pre ? 0 : prefix_tiles)) * kBlKeys;
                if (segment != pre) {
                    segment = pre;
                    y.b = pre ? -1 : b;
                    y.keys = pre ? prefix : x.keys;
                    win.begin(a, y, key >> a.own.shift, lane);
                }
                win.advance(key >> a.own.shift, lane);
                const uint32_t it = kv + j, st = it % C::kStages;
                if (!mbar_wait_warp(empty + st, ((it / C::kStages) & 1u) ^ 1u, abort_flag, a.timeout_ns)) break;
                copy_tile<D, kBlKeys, C::kAtom, true>(a, y, win, cache, ring + st * C::kTile, key, lane);
                copies_arrive(full + st);
            }
        } else if (warp == 3) {
            // -------------------------------------------------------- products
            const uint32_t lead = elect_lane();
            const uint32_t tO = tmem + 128;
            constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kBlKeys, 0, 0), kIdescPV = idesc_bf16_f32(128, D, 0, 1);
            constexpr uint64_t kStageDesc = C::kTile >> 4;
            const uint64_t dq = smem_desc_sw128(smem_u32(smem), 16, 1024), dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t dv = smem_desc_sw128(smem_u32(sV), C::kAtom, 1024);
            // the scores of tile j, into the buffer that the product before last has read
            auto qk = [&](int j) -> bool {
                const uint32_t it = kv + j, st = it % C::kStages;
                if (!mbar_wait_warp(k_full + st, (it / C::kStages) & 1u, abort_flag, a.timeout_ns)) return false;
                fence_async_shared();  // Q and K were written by cp.async
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(tmem + (it & 1u) * 64, dq + (k / 4) * (C::kAtomQ >> 4) + (k % 4) * 2,
                           dk + st * kStageDesc + (k / 4) * (C::kAtom >> 4) + (k % 4) * 2, kIdescQK, k > 0, lead);
                commit(s_full + (it & 1u), lead);
                commit(k_empty + st, lead);
                return true;
            };
            bool ok = tiles == 0 || (mbar_wait_warp(q_full, queries & 1u, abort_flag, a.timeout_ns) && qk(0));
            for (int j = 0; j < tiles && ok; ++j) {
                const uint32_t it = kv + j, st = it % C::kStages;
                ok = (j + 1 == tiles || qk(j + 1)) &&
                     mbar_wait_warp(v_full + st, (it / C::kStages) & 1u, abort_flag, a.timeout_ns) &&
                     mbar_wait_warp(p_full + (it & 1u), (it >> 1) & 1u, abort_flag, a.timeout_ns);
                if (!ok) break;
                tc_fence_after();
                fence_async_shared();
                const bool pre = j < prefix_tiles;
                const int left = (pre ? prefix : x.keys) - (j - (pre ? 0 : prefix_tiles)) * kBlKeys;
#pragma unroll
                for (int k = 0; k < kBlKeys / 16; ++k)
                    if (16 * k < left) mma_ts(tO, tmem + (it & 1u) * 64 + 8 * k, dv + st * kStageDesc + 128 * k, kIdescPV, j > 0 || k > 0, lead);
                commit(v_empty + st, lead);
                commit(o_full + (it & 1u), lead);
            }
        } else {
            // -------------------------------------------------------- softmax
            const int mine = warp * 32 + lane, row = x.row0 + mine;
            const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
            const uint32_t tO = tmem + lane_off + 128;
            if (tiles > 0) {
                // Q: 32 rows a warp, the 16-byte pieces of D / 8 lanes a row (zeros behind the last)
                constexpr int kChunks = D / 8, kRpi = 32 / kChunks;
                const int piece = lane % kChunks;
#pragma unroll 8
                for (int j = 0; j < 32; j += kRpi) {
                    const int r = warp * 32 + j + lane / kChunks, i = x.row0 + r;
                    const int tok = static_cast<int>(fdiv(static_cast<uint32_t>(i), a.div_g));
                    const long long at = (static_cast<long long>(x.tok0 + tok) * a.N + kvh * a.G + i - tok * a.G) * D + piece * 8;
                    const uint32_t to = smem_u32(smem) + (piece >> 3) * C::kAtomQ + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(a.q + (r < rows ? at : 0)),
                                 "r"(r < rows ? 16 : 0)
                                 : "memory");
                }
                copies_arrive(q_full);
            }
            const bool valid = mine < rows, busy = warp * 32 < rows;
            const int tok = static_cast<int>(fdiv(static_cast<uint32_t>(valid ? row : x.row0), a.div_g));
            const int own_limit = valid ? row_limit(a, x, row) : x.keys;
            const int own_whole = x.tree ? max(x.off, 0) : row_limit(a, x, x.row0);
            const float sl2 = a.scale_log2;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            auto ended = [&](uint32_t it) { return mbar_wait_warp(o_full + (it & 1u), (it >> 1) & 1u, abort_flag, a.timeout_ns); };
            for (int j = 0; j < tiles; ++j) {
                const bool pre = j < prefix_tiles;
                const int key = (j - (pre ? 0 : prefix_tiles)) * kBlKeys;
                const bool mask = (pre ? prefix : own_whole) - key < kBlKeys;
                uint32_t seen0 = 0, seen1 = 0;
                if (mask && busy) {
                    const bool tree = !pre && x.tree && valid;
                    const int limit = pre ? prefix : own_limit;
                    seen0 = tree ? tree_bits(a, x, tok, key) : limit_bits(limit, key);
                    seen1 = tree ? tree_bits(a, x, tok, key + 32) : limit_bits(limit, key + 32);
                }
                const uint32_t it = kv + j, tS = tmem + lane_off + (it & 1u) * 64;
                // (the product before last has ended, as these scores came behind it; each phase is seen.  Both barriers are
                // asked at once: a wait for one that is over costs 130 clk of a tile's 1200.  Asked a tile ahead, beside the
                // exponentials, they are not over yet: 16 sequences of up to 4096 keys 53 us for 46.)
                const uint32_t ph = (it >> 1) & 1u;
                const bool there = mbar_test(s_full + (it & 1u), ph) & (j < 2 || mbar_test(o_full + (it & 1u), ph ^ 1u));
                ok = __all_sync(0xffffffffu, there) ||
                     (mbar_wait_warp(s_full + (it & 1u), ph, abort_flag, a.timeout_ns) && (j < 2 || ended(it - 2)));
                if (!ok) break;
                if (busy) {
                    tc_fence_after();
                    uint32_t h[64], pk[32];
                    tmem_ld64(tS, h);
                    if (mask) hide_columns(seen0, seen1, h);
                    const float top = row_max64(h) * sl2;
                    if (__any_sync(0xffffffffu, top > m + 30.f)) {
                        float f = 1.f;
                        if (top > m + 30.f) {
                            f = fast_exp2(m - top);  // 0 from -inf
                            l *= f;
                            m = top;
                        }
                        if (j > 0) {
                            // O is quiet when the last product has ended
                            ok = ended(it - 1);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int e = 0; e < D; e += 32) {
                                uint32_t ov[32];
                                tmem_ld32(tO + e, ov);
#pragma unroll
                                for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
                                tmem_st32(tO + e, ov);
                            }
                        }
                    }
                    l += exp_pack64(h, sl2, m == -INFINITY ? 0.f : -m, pk);
                    tmem_st32_nowait(tS, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(p_full + (it & 1u));  // (of two: a warp may be a tile ahead of the other)
            }
            // a thread's row: its D values and lse
            if (busy) ok = ok && (tiles < 2 || ended(kv + tiles - 2)) && (tiles < 1 || ended(kv + tiles - 1));
            if (ok && busy) {
                tc_fence_after();
                const float2 ml = left_ml(m, sum_of_one(m, l));
                const bool none = ml.x == -INFINITY;
                const float inv = none ? 0.f : 1.f / ml.y;
                const int head = kvh * a.G + row - tok * a.G;
                const long long to = (static_cast<long long>(x.tok0 + tok) * a.N + head) * D;
#pragma unroll 1
                for (int e = 0; e < D; e += 32) {
                    uint32_t ov[32];
                    if (tiles) tmem_ld32(tO + e, ov);
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = none ? 0.f : __uint_as_float(ov[i]) * inv;
                    if (valid && c.o_bf16) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(c.o) + to + e);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                                pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
                    } else if (valid) {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(c.o) + to + e);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                    __syncwarp();
                }
                if (valid)
                    c.lse[static_cast<long long>(head) * a.R + x.tok0 + tok] =
                        none ? -INFINITY : (ml.x + log2f(ml.y)) * 0.69314718055994530942f;
                tc_fence_before();
            }
        }
        kv += tiles;
        queries += tiles > 0;
        __syncthreads();  // Q's place, and O, are free
        tc_fence_after();
    }
    // no copy lands and no product runs when the block is gone
    copies_drain();
    if (warp == 3 && *abort_flag) {  // (else every product has been waited for)
        const uint32_t lead = elect_lane();
        commit(drain, lead);
        volatile int no_abort = 0;
        mbar_wait(drain, 0, &no_abort, 100000000ull);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
    if (tid == 0 && *abort_flag) report(a.status, CP_ERR_DEVICE_TIMEOUT);
}

}  // namespace
}  // namespace cpattn
