// tree_cluster.cuh -- the tree attention of few sequences: one launch of thread-block clusters, without a plan of
// the work, partials in global memory or a second launch.
//
// Few sequences are latency: a tree of 27 tokens over 4096 keys takes 19 us by the line of prefix_call.cuh (its scan, the
// search of a block's place, the partials' way through global memory, the join) and 13 so, where the keys take 3.  Here
// a cluster of up to 16 blocks takes one item -- 128 rows (tokens x the G query heads of a KV head) of one sequence --
// and its blocks an equal share of the item's key tiles each, first the prefix's and then the sequence's own.  Where a
// block works follows from its index alone, and the blocks join their partials through each other's shared memory.
//
// Inside a block, as in prefix_tc.cuh: two halves of four softmax warps take the key tiles in turn, S = Q K^T and
// O += P V on tcgen05 with S, P and O in tensor memory (S0 | S1 | O0 | O1), a thread a row.  K and V come by 16-byte
// cp.async whatever the page's size, Q is gathered by the softmax warps.  A row's maximum is looked for before its
// weights are formed (and moved only when a weight would pass 2^30), so nothing is computed twice.  It is the score itself, not
// a whole number above it: the output of a row that sees one key is that key's value then (sum_of_one).
// A tile's code is a loop over 64 columns, not unrolled over 128: a block goes through two to thirty tiles, and code
// that is read for the first time costs more than the loop (1.4 us less than with the weights of 128 columns in a row and
// the maximum looked for only when their sum asks for it).  16-key groups behind the last key are neither copied nor
// multiplied: the block with the end of the sequence was the one that all others waited for (2 us).
//
// All of S is read before P overwrites it: the upper 64 columns' weights are stored over columns 96 .. 127, which
// have been read, then the lower ones' over 64 .. 95.
//
// An item of up to 64 rows lies in the tile twice, for the first half in its first 64 rows and for the second in
// the others: the halves' busy warps are then on different parts of the SM (a warp reads its own 32 lanes of tensor
// memory), and each half leaves a partial of its own.  Warps without rows compute nothing.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_prefix.cuh"
#include "cp_ptx.cuh"
#include "cp_softmax.cuh"
#include "prefix_tc.cuh"

namespace cpattn {
namespace {

constexpr int kClThreads = 384;
constexpr int kClMost = 16;  // blocks of a cluster

template <int D>
struct ClCfg {
    static constexpr int kAtom = 128 * 128;  // 128 rows x 64 columns
    static constexpr int kTile = kAtom * (D / 64);
    static constexpr int kStagesK = D == 128 ? 3 : 6, kStagesV = D == 128 ? 2 : 5;
    static constexpr int kOffK = kTile;  // behind Q
    static constexpr int kOffV = kOffK + kStagesK * kTile;
    static constexpr int kOffHalves = kOffV + kStagesV * kTile;  // [2][128] (m, l) of the halves
    static constexpr int kOffMl = kOffHalves + 2 * 128 * 8;      // [128] (m, l) of the block
    static constexpr int kOffBar = kOffMl + 128 * 8;
    // q_full, s_full[2], p_full[2], o_full[2], drain[2], k_full[], k_empty[], v_full[], v_empty[]
    static constexpr int kBars = 9 + 2 * (kStagesK + kStagesV);
    static constexpr int kOffMisc = (kOffBar + kBars * 8 + 15) & ~15;  // tensor memory's address, abort flag
    static constexpr int kSmem = kOffMisc + 16 + 1024;                 // + alignment slack
    // the block's partial, [128][D] fp32, lies where K was
    static_assert(128 * D * 4 <= kStagesK * kTile && kSmem <= 232448, "shared memory budget");
};

struct ClusterArgs {
    PrefixArgs p;
    int tiles;  // row tiles of a sequence that have clusters of their own
    void *o;
    int o_bf16;
    float *lse;
};

__device__ __forceinline__ uint32_t cluster_rank32() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size32() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// By all threads of all blocks of the cluster: what they wrote before is seen behind it, and what they read before is read
// from what stood there before it (also a value that nobody waits for, as those of the join's pieces of weight 0).
// The release is 0.6 us of the 13 at the end of a row tile, before the results' stores as well as behind them.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Address of this block's shared address `a` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
// A barrier of the eight softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The maximum of 64 scores.
__device__ __forceinline__ float row_max64(const uint32_t (&h)[64]) {
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], __uint_as_float(h[c + 2 * u]), __uint_as_float(h[c + 2 * u + 1]));
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

template <int D>
__global__ void __launch_bounds__(kClThreads, 1) tree_cluster_kernel(const __grid_constant__ ClusterArgs c) {
    using C = ClCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PrefixArgs &a = c.p;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bar, *s_full = bar + 1, *p_full = bar + 3, *o_full = bar + 5, *drain = bar + 7, *k_full = bar + 9,
             *k_empty = k_full + C::kStagesK, *v_full = k_empty + C::kStagesK, *v_empty = v_full + C::kStagesV;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = static_cast<int>(cluster_size32()), rank = static_cast<int>(cluster_rank32());
    int rest = static_cast<int>(blockIdx.x) / blocks;
    const int kvh = rest % a.Nkv;
    rest /= a.Nkv;
    const int tile0 = rest % c.tiles, b = rest / c.tiles;

    if (tid == 0) {
        *abort_flag = 0;
        mbar_init(q_full, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(o_full + i, 1);
            mbar_init(drain + i, 1);
        }
        for (int s = 0; s < C::kStagesK; ++s) {
            mbar_init(k_full + s, 32);
            mbar_init(k_empty + s, 1);
        }
        for (int s = 0; s < C::kStagesV; ++s) {
            mbar_init(v_full + s, 32);
            mbar_init(v_empty + s, 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    wait_for_previous();
    launch_dependents();
    // the sequence, as the lists give it (those that make no sense are cut and reported, as in sequence_problem)
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
    const int prefix = static_cast<int>(a.P), prefix_tiles = static_cast<int>((a.P + 127) >> 7);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t *sQ = smem, *sK = smem + C::kOffK, *sV = smem + C::kOffV;
    float2 *ml_s = reinterpret_cast<float2 *>(smem + C::kOffMl), *halves = reinterpret_cast<float2 *>(smem + C::kOffHalves);

    // of this thread's role, over all row tiles: key tiles so far, of its half, queries, products' ends of the halves
    uint32_t kv = 0, mine = 0, queries = 0, ends0 = 0, ends1 = 0;
    for (int tile = tile0; tile * 128 < x.rows; tile += c.tiles) {
        x.row0 = tile * 128;
        const int rows = min(128, x.rows - x.row0);
        const bool twice = rows <= 64;
        const int last = x.tree ? x.keys : row_limit(a, x, x.row0 + rows - 1);
        const int all = prefix_tiles + ((last + 127) >> 7);
        const int k0 = static_cast<int>(static_cast<long long>(all) * rank / blocks);
        const int tiles = static_cast<int>(static_cast<long long>(all) * (rank + 1) / blocks) - k0;
        if (warp == 0 || warp == 2) {
            // -------------------------------------------------------- loads: K by warp 0, V by warp 2
            uint64_t *full = warp ? v_full : k_full, *empty = warp ? v_empty : k_empty;
            const uint32_t ring = smem_u32(warp ? sV : sK), stages = warp ? C::kStagesV : C::kStagesK;
            PageWindow win{};
            Piece y = x;
            int segment = -1;
            const int loads = tiles && released(a, abort_flag) ? tiles : 0;
            for (int j = 0; j < loads; ++j) {
                const bool pre = k0 + j < prefix_tiles;
                const int key = (k0 + j - (pre ? 0 : prefix_tiles)) * 128;
                if (segment != pre) {
                    segment = pre;
                    y.b = pre ? -1 : b;
                    y.keys = pre ? prefix : x.keys;
                    win.begin(a, y, key >> a.own.shift, lane);
                }
                win.advance(key >> a.own.shift, lane);
                const uint32_t it = kv + j, st = it % stages;
                if (!mbar_wait_warp(empty + st, ((it / stages) & 1u) ^ 1u, abort_flag, a.timeout_ns)) break;
                copy_tile<D, 128, C::kAtom, true>(a, y, win, warp ? a.v : a.k, ring + st * C::kTile, key, lane);
                copies_arrive(full + st);
            }
        } else if (warp < 4) {
            // -------------------------------------------------------- products: half 0 by warp 1, half 1 by warp 3
            const int i = warp >> 1;
            const uint32_t lead = elect_lane();
            const uint32_t tS = tmem + i * 128, tP = tS + 64, tO = tmem + 256 + i * D;
            constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0), kIdescPV = idesc_bf16_f32(128, D, 0, 1);
            constexpr uint64_t kStageDesc = C::kTile >> 4;
            const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024), dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t dv = smem_desc_sw128(smem_u32(sV), C::kAtom, 1024);
            // O (+)= P V of tile j
            auto pv = [&](int j) -> bool {
                const uint32_t it = kv + j, st = it % C::kStagesV;
                if (!mbar_wait_warp(v_full + st, (it / C::kStagesV) & 1u, abort_flag, a.timeout_ns) ||
                    !mbar_wait_warp(p_full + i, mine & 1u, abort_flag, a.timeout_ns))
                    return false;
                ++mine;
                tc_fence_after();
                fence_async_shared();
                const bool pre = k0 + j < prefix_tiles;
                const int left = (pre ? prefix : x.keys) - (k0 + j - (pre ? 0 : prefix_tiles)) * 128;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (16 * k < left) mma_ts(tO, tP + 8 * k, dv + st * kStageDesc + 128 * k, kIdescPV, j > i || k > 0, lead);
                commit(v_empty + st, lead);
                return true;
            };
            bool ok = i >= tiles || mbar_wait_warp(q_full, queries & 1u, abort_flag, a.timeout_ns);
            for (int j = i; j < tiles && ok; j += 2) {
                const uint32_t it = kv + j, st = it % C::kStagesK;
                ok = mbar_wait_warp(k_full + st, (it / C::kStagesK) & 1u, abort_flag, a.timeout_ns) && (j == i || pv(j - 2));
                if (!ok) break;
                fence_async_shared();  // Q and K were written by cp.async
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(tS, dq + (k / 4) * (C::kAtom >> 4) + (k % 4) * 2,
                           dk + st * kStageDesc + (k / 4) * (C::kAtom >> 4) + (k % 4) * 2, kIdescQK, k > 0, lead);
                commit(s_full + i, lead);
                commit(k_empty + st, lead);
            }
            if (ok && i < tiles && pv(i + (tiles - 1 - i) / 2 * 2)) commit(o_full + i, lead);
        } else {
            // -------------------------------------------------------- softmax
            const int half = (warp - 4) >> 2, in_tile = (warp & 3) * 32 + lane, mine0 = in_tile - (twice ? half * 64 : 0);
            const int row = x.row0 + mine0;  // mine0: of the item's rows here (negative: none)
            const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_off + half * 128, tO = tmem + lane_off + 256;
            if (tiles > 0) {
                // Q: 16 rows a warp, the 16-byte pieces of D / 8 lanes a row (zeros behind the last)
                constexpr int kChunks = D / 8, kRpi = 32 / kChunks;
                const int piece = lane % kChunks;
#pragma unroll
                for (int j = 0; j < 16; j += kRpi) {
                    const int r = (warp - 4) * 16 + j + lane / kChunks, q = twice ? r & 63 : r, i = x.row0 + q;
                    const int tok = static_cast<int>(fdiv(static_cast<uint32_t>(i), a.div_g));
                    const long long at = (static_cast<long long>(x.tok0 + tok) * a.N + kvh * a.G + i - tok * a.G) * D + piece * 8;
                    const uint32_t to = smem_u32(sQ) + (piece >> 3) * C::kAtom + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(a.q + (q < rows ? at : 0)),
                                 "r"(q < rows ? 16 : 0)
                                 : "memory");
                }
                copies_arrive(q_full);
            }
            const bool valid = mine0 >= 0 && mine0 < rows, busy = __any_sync(0xffffffffu, valid);
            const int tok = static_cast<int>(fdiv(static_cast<uint32_t>(valid ? row : x.row0), a.div_g));
            const int own_limit = valid ? row_limit(a, x, row) : x.keys;
            const int own_whole = x.tree ? max(x.off, 0) : row_limit(a, x, x.row0);
            const float sl2 = a.scale_log2;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = half; j < tiles; j += 2) {
                const bool pre = k0 + j < prefix_tiles;
                const int key = (k0 + j - (pre ? 0 : prefix_tiles)) * 128;
                if (!busy) {
                    ok = mbar_wait_warp(s_full + half, mine & 1u, abort_flag, a.timeout_ns);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(p_full + half);
                    ++mine;
                    continue;
                }
                const bool mask = (pre ? prefix : own_whole) - key < 128;
                uint32_t seen[4];
                if (mask) {
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        seen[w] = !pre && x.tree && valid ? tree_bits(a, x, tok, key + 32 * w)
                                                          : limit_bits(pre ? prefix : own_limit, key + 32 * w);
                }
                ok = mbar_wait_warp(s_full + half, mine & 1u, abort_flag, a.timeout_ns);
                if (!ok) break;
                tc_fence_after();
                float top = -INFINITY;
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    uint32_t h[64];
                    tmem_ld64(tS + 64 * u, h);
                    if (mask) hide_columns(u ? seen[2] : seen[0], u ? seen[3] : seen[1], h);
                    top = fmaxf(top, row_max64(h));
                }
                top *= sl2;
                if (__any_sync(0xffffffffu, top > m + 30.f)) {
                    float f = 1.f;
                    if (top > m + 30.f) {
                        f = fast_exp2(m - top);  // 0 from -inf
                        l *= f;
                        m = top;
                    }
                    // O is quiet: its last product was issued before these scores
#pragma unroll 1
                    for (int e = 0; e < D && j > half; e += 32) {
                        uint32_t ov[32];
                        tmem_ld32(tO + half * D + e, ov);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
                        tmem_st32(tO + half * D + e, ov);
                    }
                }
                const float neg_m = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
                for (int u = 1; u >= 0; --u) {
                    uint32_t h[64], pk[32];
                    tmem_ld64(tS + 64 * u, h);
                    if (mask) hide_columns(u ? seen[2] : seen[0], u ? seen[3] : seen[1], h);
                    l += exp_pack64(h, sl2, neg_m, pk);
                    tmem_st32_nowait(tS + 64 + 32 * u, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + half);
                ++mine;
            }
            // the block's partial into shared memory
            const uint32_t to = smem_u32(sK) + in_tile * D * 4;
            // 16-byte pieces of a row are swizzled by the row
            auto store = [&](int column, float v0, float v1, float v2, float v3) {
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((column >> 2) ^ (in_tile & (D / 4 - 1))) << 4)),
                             "f"(v0), "f"(v1), "f"(v2), "f"(v3)
                             : "memory");
            };
            if (!twice) halves[half * 128 + in_tile] = make_float2(m, l);
            softmax_sync();
            ok = ok && !*abort_flag;
            // (also where a half leaves its own: K's place is free when both are done)
            if (ok && tiles > 0) ok = mbar_wait_warp(o_full, ends0 & 1u, abort_flag, a.timeout_ns);
            if (ok && tiles > 1) ok = mbar_wait_warp(o_full + 1, ends1 & 1u, abort_flag, a.timeout_ns);
            tc_fence_after();
            if (twice) {
                const bool left = ok && half < tiles;
                if ((in_tile >> 6) == half) ml_s[in_tile] = left ? left_ml(m, sum_of_one(m, l)) : make_float2(-INFINITY, 0.f);
                if (left && busy) {
#pragma unroll 1
                    for (int e = 0; e < D; e += 32) {
                        uint32_t ov[32];
                        tmem_ld32(tO + half * D + e, ov);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            store(e + i, __uint_as_float(ov[i]), __uint_as_float(ov[i + 1]), __uint_as_float(ov[i + 2]),
                                  __uint_as_float(ov[i + 3]));
                    }
                }
            } else {
                // the two halves' results joined, each half half the columns
                const float2 h0 = halves[in_tile], h1 = halves[128 + in_tile];
                const float top = fmaxf(h0.x, h1.x);
                const float f0 = h0.x == -INFINITY ? 0.f : fast_exp2(h0.x - top);
                const float f1 = h1.x == -INFINITY ? 0.f : fast_exp2(h1.x - top);
                const float sum = f0 * h0.y + f1 * h1.y;  // (NaN where a half's is, also one of all NaN, without exponent)
                if (half == 0) ml_s[in_tile] = ok && tiles > 0 ? left_ml(top, sum_of_one(top, sum)) : make_float2(-INFINITY, 0.f);
                if (ok && tiles > 0 && busy) {
#pragma unroll 1
                    for (int e = half * (D / 2); e < (half + 1) * (D / 2); e += 32) {
                        uint32_t ov[32], ow[32];
                        tmem_ld32(tO + e, ov);
                        if (tiles > 1) tmem_ld32(tO + D + e, ow);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[k] = f0 * __uint_as_float(ov[i + k]);
                                if (tiles > 1) v[k] += f1 * __uint_as_float(ow[i + k]);
                            }
                            store(e + i, v[0], v[1], v[2], v[3]);
                        }
                    }
                }
            }
            tc_fence_before();
        }
        kv += tiles;
        queries += tiles > 0;
        ends0 += tiles > 0;
        ends1 += tiles > 1;
        cluster_sync();
        // -------------------------------------------------------- join: every blocks-th row, a warp a row
        const uint32_t ml_at = smem_u32(ml_s), o_at = smem_u32(sK);
        // pieces: one of each block, or its two halves'
        const int pieces = twice ? 2 * blocks : blocks, by = twice;
        for (int i = rank + blocks * warp; i < rows; i += blocks * (kClThreads / 32)) {
            constexpr int kV = D / 32;
            const uint32_t chunk = kV == 4 ? lane : lane >> 1;
            const uint32_t from = o_at + i * D * 4 + ((chunk ^ (i & (D / 4 - 1))) << 4) + (kV == 4 ? 0 : (lane & 1) * 8);
            const float2 ml = lane < pieces ? ld_cluster2(at_rank(ml_at + ((lane & by) * 64 + i) * 8, lane >> by))
                                            : make_float2(-INFINITY, 0.f);
            // eight pieces' rows on their way together, the first ones beside the sums
            constexpr int kAtOnce = 8;
            float v[kAtOnce][kV];
            auto fetch = [&](int r0) {
#pragma unroll
                for (int r = 0; r < kAtOnce; ++r)
                    // (64 rows further the swizzle is the same)
                    if (r0 + r < pieces) {
                        const uint32_t at = at_rank(from + ((r0 + r) & by) * 64 * D * 4, (r0 + r) >> by);
                        if (kV == 4) {
                            const float4 y = ld_cluster4(at);
                            v[r][0] = y.x, v[r][1] = y.y, v[r][2 % kV] = y.z, v[r][3 % kV] = y.w;
                        } else {
                            const float2 y = ld_cluster2(at);
                            v[r][0] = y.x, v[r][1] = y.y;
                        }
                    }
            };
            fetch(0);
            float top = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - top);
            float sum = w * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            float acc[kV];
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[e] = 0.f;
            for (int r0 = 0;;) {
#pragma unroll
                for (int r = 0; r < kAtOnce; ++r) {
                    const float f = __shfl_sync(0xffffffffu, w, r0 + r);  // (0 behind the last)
                    if (f != 0.f)                                         // (a piece that saw nothing may hold anything)
#pragma unroll
                        for (int e = 0; e < kV; ++e) acc[e] += f * v[r][e];
                }
                r0 += kAtOnce;
                if (r0 >= pieces) break;
                fetch(r0);
            }
            const float inv = top == -INFINITY ? 0.f : 1.f / sum;
            const int at = x.row0 + i, tok = static_cast<int>(fdiv(static_cast<uint32_t>(at), a.div_g));
            const int head = kvh * a.G + at - tok * a.G;
            const long long to = (static_cast<long long>(x.tok0 + tok) * a.N + head) * D + lane * kV;
            if (c.o_bf16) {
                uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(c.o) + to);
#pragma unroll
                for (int e = 0; e < kV; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
            } else {
                float *dst = static_cast<float *>(c.o) + to;
#pragma unroll
                for (int e = 0; e < kV; ++e) dst[e] = acc[e] * inv;
            }
            if (lane == 0)
                c.lse[static_cast<long long>(head) * a.R + x.tok0 + tok] =
                    top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
        }
        cluster_sync();  // nothing of this block is read any more
    }
    // no copy lands and no product runs when the block is gone
    copies_drain();
    if ((warp == 1 || warp == 3) && *abort_flag) {  // (else every product has been waited for)
        const uint32_t lead = elect_lane();
        commit(drain + (warp >> 1), lead);
        volatile int no_abort = 0;
        mbar_wait(drain + (warp >> 1), 0, &no_abort, 100000000ull);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *abort_flag) report(a.status, CP_ERR_DEVICE_TIMEOUT);
}

}  // namespace
}  // namespace cpattn
