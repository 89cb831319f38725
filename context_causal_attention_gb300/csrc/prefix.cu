// prefix.cu -- attention of a batch whose sequences share a long prefix, over
// the paged cache: every query row sees all prefix keys and the keys of its own
// sequence up to its own index.
//
// Softmax splits over any partition of the keys ("Context Parallelism & Ring
// Attention", "Softmax is decomposable"), so the prefix part is computed for the
// rows of ALL sequences together -- its keys and values leave memory once, not
// once for each sequence -- and each sequence's own part apart.  The partials
// (m, l, o) with m an exponent, l = sum 2^(x - m), o = sum 2^(x - m) v are
// joined as in cp_lse_merge: M = max m, lse = (M + log2 sum 2^(m-M) l) ln 2.
//
// Rows.  The G = N/Nkv query heads of a KV head read the same keys, so the rows
// of a problem (the prefix, or one sequence) for one KV head are its tokens
// times G heads, row i = token i / G, head i % G, cut into tiles of kTM rows.
//
// Work split.  Few rows and many keys: the parallelism is in the keys.  All
// (problem, KV head, row tile) items are laid end to end, each as long as its
// key tiles and kExtra more (cp_prefix.cuh), and every block takes an equal share of
// that line, whatever the lengths are.  Where a call has both kinds of tiles there are
// two lines, and the blocks are divided between them by their estimated cycles
// (prefix_workers).  A share that covers part of an item leaves a partial; the
// k-th piece of a line has slot (item + block), which is unique, so the slots need
// no counter.  A second launch joins the pieces of every row in their order:
// the result does not depend on timing.
//
// Inside a block of the 16-row kernel: four warps copy K and V into a ring of
// 64-key stages (16-byte cp.async, two warps for each of K and V), two groups of
// 4 warps take the block's pieces in turn, so that one group's epilogue and next
// queries run under the other's products and the ring never waits for them.  Each warp owns 16
// of a stage's 64 keys: every byte of K and V passes from shared memory to
// registers once.  Both products run on mma.sync m16n8k16: at 16 rows the tensor
// work is a tenth of what the SM can do while it waits for memory.  Running
// maximum and sum stay in fp32 registers; P is rounded to bf16 for the second
// product (off by 2^-8 of each weight at most, as in cp_attn_partial).  Keys past the
// length are never copied (zeros in their place), whatever the page holds there.
// Problems of more rows run in prefix_tc.cuh.
//
// What bounds it: few rows read each key and value once, so the bytes of the
// pages.  64 single-token sequences of 4096 keys and 8 KV heads of 128 (1.07 GB)
// take 190 us from a cold L2, 5.6 TB/s.  A call of one token over 4400 keys is latency:
// 15 us, of them 3.7 until the place on the line is found, 3 for the first tile,
// 6 for the join.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "cp_internal.h"
#include "cp_paged.cuh"
#include "cp_prefix.cuh"
#include "cp_ptx.cuh"
#include "prefix_tc.cuh"

namespace cpattn {
namespace {

__device__ int g_prefix_status = 0;
__device__ int g_prefix_hold = 0;  // never set

// A problem whose rows for one KV head are more than this runs in tiles of 256
// rows on the tensor memory, else in tiles of 16.  A second 16-row tile reads
// every key again: 16 sequences of 4096 keys (8 KV heads of 128) take 72.8 us with
// 16 rows each (74.9 on the wide tiles), 115.8 with 32 (wide: 78.9) and 187.5 with
// 64 (83.1); 64 single tokens 191.6 (199.8), 16 rows over a prefix of 32768 keys
// 48.3 (50.3).  At D = 64 the same: that prefix 33.9 (38.0), 32 rows of 4096 keys
// 70.8 (50.3).  Where the prefix is wide and the sequences are narrow but next to
// nothing (four of 64 keys), wide tiles for both would win: 52.4 against 60.5; the
// lengths are not known here.
constexpr int kTcRows = 16;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kMaxBlocks = 320;               // of a launch (a slot more for each)
constexpr int kGroups = 2;                    // consumer groups of 4 warps
constexpr int kLoaders = 4;                   // warps: K and V, the first and second half of a stage
constexpr int kMmaThreads = kLoaders * 32 + kGroups * 128;

template <int D>
struct MmaCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtom = kKT * 128;                // 64 rows x 64 columns, 128-byte swizzle
    static constexpr int kTile = kAtom * kAtoms;           // K or V of a stage
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kOffOut = kStages * 2 * kTile;    // [groups][4 warps][16 rows][D] fp32
    static constexpr int kOffMl = kOffOut + kGroups * 4 * 16 * D * 4;  // [groups][4][16] (m, l)
    static constexpr int kOffLine = kOffMl + kGroups * 4 * 16 * 8;
    static constexpr int kListed = 1024;                   // sequences whose lists are kept here
    static constexpr int kOffLists = kOffLine + static_cast<int>(sizeof(Line));
    static constexpr int kOffStart = (kOffLists + (2 * kListed + 1) * 4 + 15) & ~15;
    static constexpr int kOffBar = (kOffStart + static_cast<int>(sizeof(Start)) + 15) & ~15;
    static constexpr int kOffMisc = kOffBar + kStages * 16 + kGroups * 8;
    static constexpr int kOffWalk = (kOffMisc + 16 + 15) & ~15;  // [warps]
    static constexpr int kSmem = kOffWalk + kMmaThreads / 32 * static_cast<int>(sizeof(Walk<kTM, kKT>)) + 1024;  // + alignment slack
    static_assert(kSmem <= 232448, "shared memory budget");
};

// Shared-memory address of 16-byte chunk c (of D/8) of row r in a stage tile.
template <int D>
__device__ __forceinline__ uint32_t tile_at_chunk(uint32_t base, int r, int c) {
    return base + (c >> 3) * MmaCfg<D>::kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}

// group_sync that also tells every thread whether any of them has `v`.
__device__ __forceinline__ bool group_any(int group, bool v) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\tbar.red.or.pred p, %1, 128, q;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(group + 1), "r"(static_cast<int>(v))
        : "memory");
    return r != 0;
}

// Barriers of a block's pipeline.  By one thread; a __syncthreads follows in mma_work.
template <int D>
__device__ __forceinline__ void mma_init(uint8_t *smem) {
    using C = MmaCfg<D>;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *empty = full + C::kStages, *go = empty + C::kStages;
    *reinterpret_cast<volatile int *>(smem + C::kOffMisc) = 0;  // abort flag
    for (int s = 0; s < C::kStages; ++s) {
        mbar_init(full + s, 32 * kLoaders);
        mbar_init(empty + s, 4);
    }
    for (int i = 0; i < kGroups; ++i) mbar_init(go + i, 4);
    fence_mbar_init();
}
template <int D>
__device__ __forceinline__ void mma_scan(const PrefixArgs &a, uint8_t *smem) {
    using C = MmaCfg<D>;
    scan_line<kTM, kKT>(a, *reinterpret_cast<Line *>(smem + C::kOffLine), reinterpret_cast<int *>(smem + C::kOffLists),
                        C::kListed);
}

// A block's share, behind mma_scan.
template <int D>
__device__ __forceinline__ void mma_work(const PrefixArgs &a, uint8_t *smem) {
    using C = MmaCfg<D>;
    Line &line = *reinterpret_cast<Line *>(smem + C::kOffLine);
    Start &start = *reinterpret_cast<Start *>(smem + C::kOffStart);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *empty = full + C::kStages, *go = empty + C::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    long long t0, t1;
    if (!share_of(a, line, &t0, &t1)) return;
    if (warp == 0) find_start<kTM, kKT>(a, line, t0, &start);
    __syncthreads();

    Walk<kTM, kKT> &walk = reinterpret_cast<Walk<kTM, kKT> *>(smem + C::kOffWalk)[warp];
    const Piece &x = walk.x;
    walk.begin(a, line, start, t1 - t0);
    if (warp < kLoaders) {
        // -------------------------------------------------------- loads
        constexpr int kPart = kKT * 2 / kLoaders;  // keys of a warp
        const bool is_v = warp & 1;
        const __nv_bfloat16 *cache = is_v ? a.v : a.k;
        const int shift = a.own.shift, part = (warp >> 1) * kPart;
        const uint32_t ring = smem_u32(smem) + is_v * C::kTile + part * 128;
        uint32_t it = 0;
        bool ok = warp != 0 || released(a, abort_flag);
        while (ok && walk.next(a, line)) {
            if (x.k0 >= x.k1) continue;
            PageWindow win;
            win.begin(a, x, (x.k0 * kKT) >> shift, lane);
            for (int kt = x.k0; kt < x.k1; ++kt, ++it) {
                win.advance((kt * kKT) >> shift, lane);
                const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1u;
                if (!mbar_wait_warp(empty + st, ph ^ 1u, abort_flag, a.timeout_ns)) { ok = false; break; }
                copy_tile<D, kPart, C::kAtom>(a, x, win, cache, ring + st * 2 * C::kTile, kt * kKT + part, lane);
                copies_arrive(full + st);
            }
        }
        copies_drain();  // also where a wait was given up: no copy may land after the block is gone
    } else {
        // -------------------------------------------------------- products
        const int group = (warp - kLoaders) >> 2, w = (warp - kLoaders) & 3, gtid = tid - kLoaders * 32 - group * 128;
        const int g = lane >> 2, t4 = lane & 3;  // accumulator row (and row + 8), column pair
        float *out_s = reinterpret_cast<float *>(smem + C::kOffOut) + group * 4 * 16 * D;
        float2 *ml_s = reinterpret_cast<float2 *>(smem + C::kOffMl) + group * 4 * 16;
        const uint32_t sbase = smem_u32(smem);
        uint32_t it = 0, gone = 0;
        int turn = 0;
        bool ok = true;
        bool first = true;
        for (; ok && walk.next(a, line); turn ^= 1, first = false) {
            if (turn != group) {
                // the other group's piece
                it += static_cast<uint32_t>(x.k1 - x.k0);
                continue;
            }
            // this warp's copy of the rows as A operands
            uint32_t qf[D / 16][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = x.row0 + g + 8 * h;
                const bool in = row < x.rows;
                const int tok = static_cast<int>(fdiv(static_cast<uint32_t>(row), a.div_g));
                const __nv_bfloat16 *qp = a.q + (static_cast<long long>(x.tok0 + (in ? tok : 0)) * a.N + x.kvh * a.G +
                                                 (in ? row - tok * a.G : 0)) * D;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[kk][h] = in ? __ldcg(reinterpret_cast<const uint32_t *>(qp + kk * 16 + 2 * t4)) : 0u;
                    qf[kk][2 + h] = in ? __ldcg(reinterpret_cast<const uint32_t *>(qp + kk * 16 + 8 + 2 * t4)) : 0u;
                }
            }
            const int lim0 = x.row0 + g < x.rows ? row_limit(a, x, x.row0 + g) : 0;
            const int lim1 = x.row0 + g + 8 < x.rows ? row_limit(a, x, x.row0 + g + 8) : 0;
            // tiles from the first that some row does not see whole on are masked
            const int whole = x.row0 + kTM <= x.rows ? row_limit(a, x, x.row0) : 0;
            float o[D / 8][4];
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            // the other group has used up the stages before these: a wait for a stage
            // is then never more than one of its phases ahead
            if (!first && !mbar_wait_warp(go + group, gone++ & 1u, abort_flag, a.timeout_ns)) ok = false;
            for (int kt = x.k0; kt < x.k1 && ok; ++kt, ++it) {
                const uint32_t st = it % C::kStages, ph = (it / C::kStages) & 1u;
                if (!mbar_wait_warp(full + st, ph, abort_flag, a.timeout_ns)) { ok = false; break; }
                const uint32_t ks = sbase + st * 2 * C::kTile, vs = ks + C::kTile;
                const int key0 = w * 16;
                float s[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b[4];
                    // lanes 0-7: keys 0-7, low 8 columns; 8-15: high; 16-31: keys 8-15
                    ldsm4(tile_at_chunk<D>(ks, key0 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)), b);
                    mma16816(s[0], qf[kk], b[0], b[1]);
                    mma16816(s[1], qf[kk], b[2], b[3]);
                }
                const int kb = kt * kKT + key0 + 2 * t4;
                const bool masked = whole - kt * kKT < kKT;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[n][e] *= a.scale_log2;
                        if (masked && kb + 8 * n + (e & 1) >= ((e & 2) ? lim1 : lim0)) s[n][e] = -INFINITY;
                    }
                // the maximum is an integer, set by the first keys that a row sees and
                // moved only when a weight would pass 2^30: rescaling is exact and rare
                const float top0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                const float top1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
                if (__any_sync(0xffffffffu, top0 > m[0] + 30.f || top1 > m[1] + 30.f)) {
                    float top[2] = {top0, top1};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                        if (top[h] > m[h] + 30.f) {
                            const float mn = ceilf(top[h]), f = fast_exp2(m[h] - mn);  // 0 from -inf
                            m[h] = mn;
                            l[h] *= f;
#pragma unroll
                            for (int n = 0; n < D / 8; ++n) {
                                o[n][2 * h] *= f;
                                o[n][2 * h + 1] *= f;
                            }
                        }
                    }
                }
                const float n0 = m[0] == -INFINITY ? 0.f : m[0], n1 = m[1] == -INFINITY ? 0.f : m[1];
                uint32_t pf[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = fast_exp2(s[n][0] - n0), p1 = fast_exp2(s[n][1] - n0);
                    const float p2 = fast_exp2(s[n][2] - n1), p3 = fast_exp2(s[n][3] - n1);
                    l[0] += p0 + p1;
                    l[1] += p2 + p3;
                    pf[2 * n] = pack_bf16x2(p0, p1);
                    pf[2 * n + 1] = pack_bf16x2(p2, p3);
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t b[4];
                    // lanes 0-7: keys 0-7, 8-15: keys 8-15 of the low 8 columns; 16-31: of the high
                    ldsm4t(tile_at_chunk<D>(vs, key0 + (lane & 15), 2 * n + (lane >> 4)), b);
                    mma16816(o[2 * n], pf, b[0], b[1]);
                    mma16816(o[2 * n + 1], pf, b[2], b[3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st);
            }
            if (lane == 0) mbar_arrive(go + (group ^ 1));
            // join the four warps' keys and leave the piece's partial (a warp that gave
            // up a wait takes part, so that the group stays together, and all leave below)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                if (t4 == 0) ml_s[w * 16 + g + 8 * h] = make_float2(m[h], l[h]);
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(out_s + (w * 16 + g + 8 * h) * D + ((8 * n + 2 * t4) ^ ((g & 3) << 3))) =
                        make_float2(o[n][2 * h], o[n][2 * h + 1]);
            }
            group_sync(group);
            const int row = gtid >> 3, c0 = (gtid & 7) * 4;  // 8 threads a row, 4 values at a time
            if (x.row0 + row < x.rows && x.slot >= 0) {
                float2 ml[4];
                float f[4], mx = -INFINITY, ls = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ml[i] = ml_s[i * 16 + row];
                    mx = fmaxf(mx, ml[i].x);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - mx);
                    ls += f[i] * ml[i].y;
                }
                const long long at = static_cast<long long>(x.slot) * kTM + row;
#pragma unroll
                for (int c = c0; c < D; c += 32) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 y = *reinterpret_cast<const float4 *>(out_s + (i * 16 + row) * D + (c ^ ((row & 3) << 3)));
                        if (f[i] != 0.f) {  // a warp that saw nothing holds zeros
                            v.x += f[i] * y.x;
                            v.y += f[i] * y.y;
                            v.z += f[i] * y.z;
                            v.w += f[i] * y.w;
                        }
                    }
                    *reinterpret_cast<float4 *>(a.slot_o + at * D + c) = v;
                }
                if (c0 == 0) a.slot_ml[at] = left_ml(mx, ls);
            }
            if (x.slot < 0 && gtid == 0) report(a.status, CP_ERR_PAGE);
            if (group_any(group, !ok)) ok = false;
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) report(a.status, CP_ERR_DEVICE_TIMEOUT);
}

__device__ __forceinline__ uint8_t *aligned_shared() {
    extern __shared__ uint8_t smem_raw[];
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

template <int D>
__global__ void __launch_bounds__(kMmaThreads, 1)
    prefix_mma_kernel(const __grid_constant__ PrefixArgs a) {
    uint8_t *smem = aligned_shared();
    if (threadIdx.x == 0) mma_init<D>(smem);
    // its blocks may have started under the kernels that made its inputs
    wait_for_previous();
    launch_dependents();
    mma_scan<D>(a, smem);
    if (blockIdx.x == 0 && blockIdx.y == 0)
        leave_places<kTM, kKT>(a, *reinterpret_cast<Line *>(smem + MmaCfg<D>::kOffLine));
    mma_work<D>(a, smem);
}

// A block's beginning and end in cycles (lists, pages, queries, first tiles; the last
// rows' partials): a wide block had its first scores after 13 us and its last 6 us
// before its end, a narrow one its first tile after 6.6.
constexpr float kAroundWide = 36000.f, kAroundNarrow = 15000.f;

// Workers of a lane for the prefix, so that the slower of the two kinds is done
// soonest.  With the wide tile's cost (D = 128, small pages: 4250 cycles) a prefix of
// 32768 keys and 64 sequences of up to 2048, 32 / 8 heads, take 88 us; at 3000 100, at
// 3600 93.6, at 5000 88, at 5600 93.  In proportion
// to the costs alone (without what lies around the tiles, rounded) five tokens each
// of 7 sequences behind 100003 keys, 16 heads of 64, got one worker where they need
// two: 101 us, 95 so.  Warp-wide; at least two workers.
__device__ __forceinline__ int prefix_workers(float prefix, float own, int workers) {
    if (own == 0.f) return workers;
    uint32_t best = 0xffffffffu;
    for (int w = 1 + (threadIdx.x & 31); w < workers; w += 32) {
        const float t = fmaxf(kAroundWide + prefix / w, kAroundNarrow + own / (workers - w));
        best = min(best, (__float_as_uint(t) & ~511u) | w);  // t > 0: its bits are in its order
    }
    return static_cast<int>(__reduce_min_sync(0xffffffffu, best) & 511u);
}

// The prefix in tiles of 256 rows and the sequences in tiles of 16, side by side:
// the first are bound by their arithmetic and the second by memory, so a block does
// one kind (prefix_workers).  As two launches, each leaving the other's blocks idle, the
// idle blocks of the second waited for the first and the join for them: 93 us
// where this took 88.  a: the prefix; b: the sequences.
template <int D, bool tma>
__global__ void __launch_bounds__(kTcThreads, 1)
    prefix_both_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PrefixArgs a, const __grid_constant__ PrefixArgs b) {
    static_assert(kMmaThreads == kTcThreads && kMaxBlocks < 512, "one launch");
    uint8_t *smem = aligned_shared();
    wait_for_previous();
    launch_dependents();
    mma_scan<D>(b, smem);
    Line &line = *reinterpret_cast<Line *>(smem + MmaCfg<D>::kOffLine);
    const Problem p = prefix_problem<kTcTM, kTcKT>(a, line);
    const int items = a.heads * p.row_tiles;
    const long long tiles = items * p.key_tiles;
    const int w = prefix_workers(static_cast<float>(tiles) * a.cost, static_cast<float>(line.tile[kRuns]) * b.cost, gridDim.y);
    const int y = blockIdx.y, rows_end = line.rows_end;
    __syncthreads();
    if (y >= w) {
        if (threadIdx.x == 0) {
            mma_init<D>(smem);
            line.worker = y - w;
            line.workers = gridDim.y - w;
        }
        __syncthreads();
        if (blockIdx.x == 0 && y == w) leave_places<kTM, kKT>(b, line);
        mma_work<D>(b, smem);
        return;
    }
    // the prefix alone makes a line of one problem
    Line &own = *reinterpret_cast<Line *>(smem + TcCfg<D>::kOffLine);
    if (threadIdx.x <= kRuns) {
        own.tile[threadIdx.x] = tiles;
        own.item[threadIdx.x] = items;
    }
    if (threadIdx.x == 0) {
        own.worker = y;
        own.workers = w;
        own.rows_end = rows_end;
        own.listed = 0;
        tc_init<D, tma>(smem, tmK, tmV);
    }
    __syncthreads();
    tc_work<D, tma>(tmK, tmV, a, smem);
}

// What a launch left, as the join reads it.
struct JoinPart {
    const long long *head, *base_tile;
    const int *base_item;
    const float2 *slot_ml;
    const float *slot_o;
    int slots, tm, kt, lanes;  // slots: of a lane
};
struct JoinArgs {
    JoinPart part[2];  // the prefix; the sequences
    const int32_t *cu, *kv_len;
    int R, B, N, Nkv, G;
    long long P, most;  // most: keys that a sequence's table can hold
    void *o;
    int o_bf16;
    float *lse;
};

// Heads of a token that one warp of join_token_kernel takes: 4, 8, 16 and 32
// measured 1220, 1206, 1208 and 1223 us for 8 ragged prompts of up to 1024 tokens
// (32 heads of 128) over a prefix of 16384 keys, the whole call.
constexpr int kJoinHeads = 16;

// Where the pieces of a row of head h lie: the slots first .. first + n - 1, row r of each.
struct RowPieces {
    int first, n, r;
};

// Keys of sequence b, whose `count` new tokens begin at row `begin`, as the launch
// before the join takes them (sequence_problem): where the counts make no sense
// it has no rows there, and so no keys here (reported there).
__device__ __forceinline__ long long own_keys(const JoinArgs &a, int b, int *begin, int *count) {
    if (b < 0) return 0;
    if (*begin < 0 || *count > a.R - *begin) {
        *begin = *count = 0;
        return 0;
    }
    return min(max(static_cast<long long>(__ldcg(a.kv_len + b)), 0ll), a.most);
}

// A part of one token's rows, for all its heads.
struct TokenPart {
    const float2 *slot_ml;
    const float *slot_o;
    long long base_tile, key_tiles, share;
    int base_item, row_tiles, row0, tm, slots, lanes;
    // which: 0 the prefix, 1 the sequence b that begins at row `begin`, of n tokens' rows
    __device__ __forceinline__ TokenPart(const JoinArgs &a, int which, int b, int tok, int begin, int n, long long keys) {
        const JoinPart &p = a.part[which];
        slot_ml = p.slot_ml;
        slot_o = p.slot_o;
        slots = p.slots;
        lanes = p.lanes;
        tm = p.tm;
        key_tiles = keys ? div_floor(keys + p.kt - 1, p.kt) + kExtra : 0;
        row_tiles = (n * a.G + tm - 1) / tm;
        row0 = (tok - (which ? begin : 0)) * a.G;
        base_tile = which ? p.base_tile[b] : 0;
        base_item = which ? p.base_item[b] : 0;
        share = p.head[0];
        if (row0 >= n * a.G) key_tiles = 0;
    }
    __device__ __forceinline__ RowPieces row(int kvh, int gh) const {
        if (key_tiles == 0) return RowPieces{0, 0, 0};
        const int i = row0 + gh, pass = kvh / lanes;
        const long long at = static_cast<long long>(pass) * row_tiles + place_of(i / tm, row_tiles);
        const long long first = base_tile + at * key_tiles;
        const int c0 = static_cast<int>(div_floor(first, share));
        const int c1 = static_cast<int>(div_floor(first + key_tiles - 1, share));
        const int slot = base_item + static_cast<int>(at) + c0;
        if (slot < 0) return RowPieces{0, 0, 0};  // lists that make no sense (reported)
        return RowPieces{(kvh - pass * lanes) * slots + slot, max(0, min(c1 - c0 + 1, slots - slot)), i % tm};
    }
};

template <int kV>
__device__ __forceinline__ void store_row(const JoinArgs &a, long long row, int lane, const float (&v)[kV], float f) {
    const long long at = row * (32 * kV) + lane * kV;
    if (a.o_bf16) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.o) + at);
#pragma unroll
        for (int e = 0; e < kV; e += 2) dst[e / 2] = pack_bf16x2(v[e] * f, v[e + 1] * f);
    } else {
        float *dst = static_cast<float *>(a.o) + at;
#pragma unroll
        for (int e = 0; e < kV; ++e) dst[e] = v[e] * f;
    }
}
template <int kV>
__device__ __forceinline__ void add_row(float (&acc)[kV], const float *src, float f) {
    if (kV == 4) {
        const float4 y = *reinterpret_cast<const float4 *>(src);
        acc[0] += f * y.x, acc[1] += f * y.y, acc[2 % kV] += f * y.z, acc[3 % kV] += f * y.w;
    } else {
        const float2 y = *reinterpret_cast<const float2 *>(src);
        acc[0] += f * y.x, acc[1] += f * y.y;
    }
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Few rows of many pieces: a warp joins the pieces of one row, those of both
// parts in one list: a lane a piece's (m, l), then the pieces' rows, twelve on their
// way together.  One token's 19 pieces: the call 15.0 us, with eight or sixteen
// 15.8; 64 sequences' 10 to 12: 88.2, 87.6, 89.7.
constexpr int kAheadRows = 12;
template <int D>
__global__ void __launch_bounds__(128) join_row_kernel(const JoinArgs a) {
    constexpr int kV = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.R) * a.N) return;
    const int tok = static_cast<int>(row / a.N), h = static_cast<int>(row - static_cast<long long>(tok) * a.N);
    int begin, count;
    const int b = find_sequence<true>(a.cu, a.B, tok, lane, &begin, &count);
    // inputs, as the search: before the wait, and past L1
    const int all = min(max(__ldcg(a.cu + a.B), 0), a.R);
    const long long len = own_keys(a, b, &begin, &count);
    wait_for_previous();
    if (b < 0) return;
    float mx = -INFINITY, ls = 0.f, acc[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.f;
    const int kvh = h / a.G;
    const TokenPart p0(a, 0, b, tok, begin, all, a.P), p1(a, 1, b, tok, begin, count, len);
    const RowPieces x0 = p0.row(kvh, h - kvh * a.G), x1 = p1.row(kvh, h - kvh * a.G);
    for (int cb = 0; cb < x0.n + x1.n; cb += 32) {
        const int i = cb + lane;
        const bool one = i >= x0.n;
        const TokenPart &p = one ? p1 : p0;
        const long long at = static_cast<long long>(one ? x1.first + i - x0.n : x0.first + i) * p.tm + (one ? x1.r : x0.r);
        const bool in = i < x0.n + x1.n;
        const float2 ml = in ? p.slot_ml[at] : make_float2(-INFINITY, 0.f);
        const float *mine = in ? p.slot_o + at * D : nullptr;
        const int n = min(32, x0.n + x1.n - cb);
        const float top = warp_max(ml.x);
        if (top == -INFINITY) continue;
        if (top > mx) {
            const float f = mx == -INFINITY ? 0.f : fast_exp2(mx - top);
            ls *= f;
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[e] *= f;
            mx = top;
        }
        const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - mx);
        float add = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
        ls += add;
        for (int k0 = 0; k0 < n; k0 += kAheadRows) {
            float v[kAheadRows][kV];
#pragma unroll
            for (int k = 0; k < kAheadRows; ++k) {
                const float *src = reinterpret_cast<const float *>(__shfl_sync(
                    0xffffffffu, reinterpret_cast<unsigned long long>(mine), (k0 + k) & 31));
#pragma unroll
                for (int e = 0; e < kV; ++e) v[k][e] = 0.f;
                if (k0 + k < n) add_row<kV>(v[k], src + lane * kV, 1.f);
            }
#pragma unroll
            for (int k = 0; k < kAheadRows; ++k) {
                const float f = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                if (f != 0.f)  // a piece that saw nothing may hold anything
#pragma unroll
                    for (int e = 0; e < kV; ++e) acc[e] += f * v[k][e];
            }
        }
    }
    store_row<kV>(a, row, lane, acc, mx == -INFINITY ? 0.f : 1.f / ls);
    if (lane == 0) a.lse[static_cast<long long>(h) * a.R + tok] = lse_of(mx, ls);
}

// Many rows of few pieces: a warp joins kJoinHeads heads of one token, a lane a
// head's (m, l), then four heads' rows at a time with their loads in flight together.
template <int D>
__global__ void __launch_bounds__(128) join_token_kernel(const JoinArgs a) {
    constexpr int kV = D / 32;
    const int lane = threadIdx.x & 31, blocks = (a.N + kJoinHeads - 1) / kJoinHeads;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int tok = static_cast<int>(unit / blocks), h0 = static_cast<int>(unit - static_cast<long long>(tok) * blocks) * kJoinHeads;
    if (tok >= a.R) return;
    int begin, count;
    const int b = find_sequence<true>(a.cu, a.B, tok, lane, &begin, &count);
    // inputs, as the search: before the wait, and past L1
    const int all = min(max(__ldcg(a.cu + a.B), 0), a.R);
    const long long len = own_keys(a, b, &begin, &count);
    wait_for_previous();
    if (b < 0) return;
    const int heads = min(kJoinHeads, a.N - h0), h = h0 + min(lane, heads - 1), kvh = h / a.G;
    const TokenPart p0(a, 0, b, tok, begin, all, a.P), p1(a, 1, b, tok, begin, count, len);
    const RowPieces x0 = p0.row(kvh, h - kvh * a.G);
    const RowPieces x1 = p1.row(kvh, h - kvh * a.G);
    const float2 *s0 = p0.slot_ml + static_cast<long long>(x0.first) * p0.tm + x0.r;
    const float2 *s1 = p1.slot_ml + static_cast<long long>(x1.first) * p1.tm + x1.r;
    float mx = -INFINITY, ls = 0.f;
    for (int i = 0; i < x0.n; ++i) mx = fmaxf(mx, s0[static_cast<long long>(i) * p0.tm].x);
    for (int i = 0; i < x1.n; ++i) mx = fmaxf(mx, s1[static_cast<long long>(i) * p1.tm].x);
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int i = 0; i < x0.n; ++i) {
        const float2 ml = s0[static_cast<long long>(i) * p0.tm];
        ls += fast_exp2(ml.x - ref) * ml.y;
    }
    for (int i = 0; i < x1.n; ++i) {
        const float2 ml = s1[static_cast<long long>(i) * p1.tm];
        ls += fast_exp2(ml.x - ref) * ml.y;
    }
    const float inv = mx == -INFINITY ? 0.f : 1.f / ls;
    if (lane < heads) a.lse[static_cast<long long>(h) * a.R + tok] = lse_of(mx, ls);
    for (int k0 = 0; k0 < heads; k0 += 4) {
        float acc[4][kV];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[k][e] = 0.f;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const TokenPart &p = which ? p1 : p0;
            const RowPieces &x = which ? x1 : x0;
            const float2 *s = which ? s1 : s0;
            int n[4], most = 0;
            const float *src[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                n[k] = __shfl_sync(0xffffffffu, x.n, (k0 + k) & 31);
                if (k0 + k >= heads) n[k] = 0;
                most = max(most, n[k]);
                src[k] = p.slot_o + (static_cast<long long>(__shfl_sync(0xffffffffu, x.first, (k0 + k) & 31)) * p.tm +
                                     __shfl_sync(0xffffffffu, x.r, (k0 + k) & 31)) * D + lane * kV;
            }
            for (int i = 0; i < most; ++i) {
                const float w = i < x.n ? fast_exp2(s[static_cast<long long>(i) * p.tm].x - ref) * inv : 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                    if (i < n[k] && f != 0.f) add_row<kV>(acc[k], src[k] + static_cast<long long>(i) * p.tm * D, f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k0 + k < heads) store_row<kV>(a, static_cast<long long>(tok) * a.N + h0 + k0 + k, lane, acc[k], 1.f);
    }
}

// ---------------------------------------------------------------- host side
// Up to this many rows (tokens x heads) a warp joins one, beyond it kJoinHeads heads
// of a token.  Few rows have many pieces, many rows few.  The whole call, by rows and by
// tokens, 32 heads of 128, tokens of one behind 32768 keys: 2048 rows 106 and 163 us,
// 8192 237 and 263, 16384 362 and 374, 32768 594 and 575, 65536 (16384 keys) 767 and 692;
// prompts behind 16384 keys: 8192 rows 93 and 132, 16384 153 and 169, 32768 288
// and 276, 65536 515 and 454; one prompt with no prefix: 16384 51 and 48, 32768 77 and 54.
constexpr long long kJoinRows = 16384;

// Blocks of a launch for each lane.
int workers_of(int lanes) { return (sm_count() < kMaxBlocks ? sm_count() : kMaxBlocks) / lanes; }

// How a call is cut: which launches it makes and where they leave their pieces.
struct Shape {
    bool tc_prefix, tc_own;  // tensor-memory tiles of 256 rows, else tiles of 16 rows
    int lanes;               // of KV heads
    long long slots[2];      // of a lane of the 16-row launch and the 256-row launch (0: not made)
    size_t head[2], base_tile[2], base_item[2], slot_ml[2], slot_o[2], bytes;
};

Shape shape_of(int64_t R, int64_t B, int64_t max_new, int64_t P, int64_t N, int64_t Nkv, int64_t D) {
    const long long G = N / Nkv;
    Shape s{};
    s.tc_prefix = R * G > kTcRows;
    s.tc_own = max_new * G > kTcRows;
    // as many lanes as leave nearly no SM without work
    const int sms = sm_count();
    for (int d = 1; d <= Nkv && d <= sms; ++d)
        if (Nkv % d == 0 && sms / d * d * 25LL >= sms * 24LL) s.lanes = d;
    size_t at = 0;
    auto take = [&at](size_t n) {
        const size_t x = at;
        at = (at + n + 255) & ~size_t(255);
        return x;
    };
    for (int k = 0; k < 2; ++k) {
        const bool pre = P > 0 && s.tc_prefix == (k == 1), own = s.tc_own == (k == 1);
        const long long tm = k ? kTcTM : kTM, tiles = (R * G + tm - 1) / tm;
        if (!pre && !own) continue;
        // every row tile of the prefix and of the sequences (each may end a tile early), and a cut for each block
        s.slots[k] = Nkv / s.lanes * ((pre ? tiles : 0) + (own ? tiles + (B < R ? B : R) : 0)) + kMaxBlocks / s.lanes;
        s.head[k] = take(8);
        s.base_tile[k] = take(B * 8);
        s.base_item[k] = take(B * 4);
        s.slot_ml[k] = take(static_cast<size_t>(s.slots[k]) * s.lanes * tm * 8);
        s.slot_o[k] = take(static_cast<size_t>(s.slots[k]) * s.lanes * tm * D * 4);
    }
    s.bytes = at;
    return s;
}

// One launch: `wide` in tiles of 256 rows, `narrow` in tiles of 16, or both (either
// may be null).
template <int D>
cp_status launch_main(const PrefixArgs *wide, const PrefixArgs *narrow, cudaStream_t stream) {
    constexpr int both_smem = TcCfg<D>::kSmem > MmaCfg<D>::kSmem ? TcCfg<D>::kSmem : MmaCfg<D>::kSmem;
    const PrefixArgs &a = wide ? *wide : *narrow;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(prefix_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaCfg<D>::kSmem);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(prefix_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TcCfg<D>::kSmem);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(prefix_tc_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TcCfg<D>::kSmem);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(prefix_both_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, both_smem);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(prefix_both_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, both_smem);
    });
    if (err != cudaSuccess) return cuda_status(err);
    const dim3 grid(a.lanes, workers_of(a.lanes));
    if (!wide) return launch(prefix_mma_kernel<D>, grid, kMmaThreads, MmaCfg<D>::kSmem, stream, a);
    const int64_t rows = static_cast<int64_t>(a.own.n_pages) << a.own.shift;
    const int page = 1 << a.own.shift, box = page < kTcKT ? page : kTcKT;
    // at D = 64 a head's row is 128 bytes and its neighbour another head's
    const int l2 = D == 64 ? 128 : 256;
    CUtensorMap mk{}, mv{};  // read only with TMA
    if (page >= kTmaPage) {
        if (!make_map(&mk, a.k, D, a.Nkv, rows, 1, box, l2) || !make_map(&mv, a.v, D, a.Nkv, rows, 1, box, l2))
            return CP_ERR_CUDA;
        if (narrow) return launch(prefix_both_kernel<D, true>, grid, kTcThreads, both_smem, stream, mk, mv, a, *narrow);
        return launch(prefix_tc_kernel<D, true>, grid, kTcThreads, TcCfg<D>::kSmem, stream, mk, mv, a);
    }
    if (narrow) return launch(prefix_both_kernel<D, false>, grid, kTcThreads, both_smem, stream, mk, mv, a, *narrow);
    return launch(prefix_tc_kernel<D, false>, grid, kTcThreads, TcCfg<D>::kSmem, stream, mk, mv, a);
}

template <int D>
cp_status launch_call(const PrefixArgs &call, const Shape &s, uint8_t *w, JoinArgs j, cudaStream_t stream) {
    PrefixArgs args[2];  // tiles of 16 rows, of 256
    for (int k = 0; k < 2; ++k) {
        if (!s.slots[k]) continue;
        PrefixArgs &a = args[k];
        a = call;
        a.with_prefix = a.P > 0 && s.tc_prefix == (k == 1);
        a.with_own = s.tc_own == (k == 1);
        // Measured cycles of a tile, for the blocks' shares where both kinds run (a tile
        // of up to 128 rows by both halves in turn; small pages by cp.async).
        const bool half = static_cast<int64_t>(a.R) * a.G <= 128, small = (1 << a.own.shift) < kTmaPage;
        a.cost = !k ? (D == 128 ? 1200.f : 780.f)
                    : D == 128 ? (half ? (small ? 3400.f : 2900.f) : (small ? 4250.f : 4000.f))
                               : (half ? (small ? 2050.f : 1450.f) : 2700.f);
        a.head = reinterpret_cast<long long *>(w + s.head[k]);
        a.base_tile = reinterpret_cast<long long *>(w + s.base_tile[k]);
        a.base_item = reinterpret_cast<int *>(w + s.base_item[k]);
        a.slot_ml = reinterpret_cast<float2 *>(w + s.slot_ml[k]);
        a.slot_o = reinterpret_cast<float *>(w + s.slot_o[k]);
        a.slots = static_cast<int>(s.slots[k]);
        for (int which = 0; which < 2; ++which)
            if (which ? a.with_own : a.with_prefix)
                j.part[which] = JoinPart{a.head, a.base_tile, a.base_item, a.slot_ml, a.slot_o, a.slots,
                                         k ? kTcTM : kTM, k ? kTcKT : kKT, a.lanes};
    }
    if (call.P == 0) j.part[0] = j.part[1];  // not read into a result: no keys
    const PrefixArgs *narrow = s.slots[0] ? &args[0] : nullptr, *wide = s.slots[1] ? &args[1] : nullptr;
    cp_status st = CP_OK;
    if (narrow && wide && workers_of(s.lanes) < 2) {
        // a lane of one worker has none to share
        st = launch_main<D>(wide, nullptr, stream);
        wide = nullptr;
    }
    if (st == CP_OK) st = launch_main<D>(wide, narrow, stream);
    if (st != CP_OK) return st;
    const long long rows = static_cast<long long>(call.R) * call.N;
    const bool few = rows <= kJoinRows;
    const long long units = few ? rows : static_cast<long long>(call.R) * ((call.N + kJoinHeads - 1) / kJoinHeads);
    return launch(few ? join_row_kernel<D> : join_token_kernel<D>, dim3(static_cast<unsigned>((units + 3) / 4)), 128, 0,
                  stream, j);
}

cp_status check_sizes(int64_t R, int64_t B, int64_t max_new, int64_t P, int64_t N, int64_t Nkv, int64_t D,
                      int64_t page_size, int64_t max_pages) {
    if (R < 1 || N < 1 || N > 65535 || max_new < 1 || max_new > R || P < 0 || P > kMaxKeys) return CP_ERR_SHAPE;
    const cp_status st = check_pages(1, page_size, B, max_pages, Nkv, D);
    if (st != CP_OK) return st;
    if (N % Nkv) return CP_ERR_DIVISIBILITY;
    if (R * N > INT32_MAX / 4) return CP_ERR_SHAPE;
    return CP_OK;
}

}  // namespace

namespace {
// Device address of the status word in the current context (looked up at each
// call: a new context has another).
cp_status status_word(int **p) {
    return cuda_status(cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_prefix_status));
}
}  // namespace

cp_status read_prefix_device_status(int *code, bool clear) {
    if (cudaMemcpyFromSymbol(code, g_prefix_status, sizeof(int)) != cudaSuccess) return CP_ERR_CUDA;
    if (clear) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(int)) != cudaSuccess) return CP_ERR_CUDA;
    }
    return CP_OK;
}

}  // namespace cpattn

using namespace cpattn;

extern "C" cp_status cp_prefix_attn_workspace_size(int64_t R, int64_t B, int64_t max_new, int64_t prefix_len,
                                                   int64_t N, int64_t Nkv, int64_t D, int64_t page_size,
                                                   int64_t max_pages, size_t *bytes) {
    if (!bytes) return CP_ERR_NULL;
    const cp_status st = check_sizes(R, B, max_new, prefix_len, N, Nkv, D, page_size, max_pages);
    if (st != CP_OK) return st;
    *bytes = shape_of(R, B, max_new, prefix_len, N, Nkv, D).bytes;
    return CP_OK;
}

namespace {
// cp_prefix_attn_fwd, with the limit of its waits; stalled: its loads wait for a word that nothing sets.
cp_status prefix_call(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages, int64_t page_size,
                      const int32_t *prefix_pages, int64_t prefix_len, const int32_t *table, int64_t B,
                      int64_t max_pages, const int32_t *cu_new, const int32_t *kv_len, int64_t max_new, int64_t R,
                      int64_t N, int64_t Nkv, int64_t D, float scale, void *o, cp_dtype o_dtype, float *lse,
                      void *workspace, size_t ws_bytes, uint64_t timeout_ns, bool stalled, cudaStream_t stream) {
    if (!q || !k_cache || !v_cache || !table || !cu_new || !kv_len || !o || !lse || (prefix_len > 0 && !prefix_pages))
        return CP_ERR_NULL;
    cp_status st = check_sizes(R, B, max_new, prefix_len, N, Nkv, D, page_size, max_pages);
    if (st == CP_OK) st = check_pages(n_pages, page_size, B, max_pages, Nkv, D);
    if (st != CP_OK) return st;
    if (!dtype_size(o_dtype)) return CP_ERR_DTYPE;
    if (!(std::isfinite(scale) && scale > 0.f)) return CP_ERR_ARGUMENT;
    auto odd = [](const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (odd(q, 16) || odd(k_cache, 16) || odd(v_cache, 16) || odd(o, 16) || odd(lse, 4) || odd(table, 4) ||
        odd(prefix_pages, 4) || odd(cu_new, 4) || odd(kv_len, 4))
        return CP_ERR_ALIGNMENT;
    const Shape s = shape_of(R, B, max_new, prefix_len, N, Nkv, D);
    if (!workspace || ws_bytes < s.bytes) return CP_ERR_WORKSPACE;
    if (odd(workspace, 256)) return CP_ERR_ALIGNMENT;
    if (s.slots[0] * s.lanes > INT32_MAX || s.slots[1] * s.lanes > INT32_MAX) return CP_ERR_SHAPE;
    PrefixArgs a{};
    if ((st = status_word(&a.status)) != CP_OK) return st;
    a.timeout_ns = timeout_ns;
    if (stalled) {
        void *hold = nullptr;
        if ((st = cuda_status(cudaGetSymbolAddress(&hold, g_prefix_hold))) != CP_OK) return st;
        a.hold = static_cast<const int *>(hold);
    }
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k_cache);
    a.v = static_cast<const __nv_bfloat16 *>(v_cache);
    a.own.table = table;
    a.own.B = static_cast<int>(B);
    a.own.max_pages = static_cast<int>(max_pages);
    a.own.n_pages = static_cast<int>(n_pages);
    a.own.shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    a.pre = a.own;
    a.pre.table = prefix_pages;
    a.pre.B = 1;
    a.pre.max_pages = static_cast<int>((prefix_len + page_size - 1) / page_size);
    a.cu = cu_new;
    a.kv_len = kv_len;
    a.R = static_cast<int>(R);
    a.B = static_cast<int>(B);
    a.N = static_cast<int>(N);
    a.Nkv = static_cast<int>(Nkv);
    a.G = static_cast<int>(N / Nkv);
    a.div_g = make_fastdiv(static_cast<uint32_t>(a.G));
    a.lanes = s.lanes;
    a.heads = static_cast<int>(Nkv / s.lanes);
    a.P = prefix_len;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    JoinArgs j{};
    j.cu = cu_new;
    j.kv_len = kv_len;
    j.R = a.R, j.B = a.B, j.N = a.N, j.Nkv = a.Nkv, j.G = a.G;
    j.P = prefix_len;
    j.most = max_pages * page_size;
    j.o = o;
    j.o_bf16 = o_dtype == CP_BF16;
    j.lse = lse;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    return D == 128 ? launch_call<128>(a, s, w, j, stream) : launch_call<64>(a, s, w, j, stream);
}
}  // namespace

extern "C" cp_status cp_prefix_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                        int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                        const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                        const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv,
                                        int64_t D, float scale, void *o, cp_dtype o_dtype, float *lse,
                                        void *workspace, size_t ws_bytes, cudaStream_t stream) {
    return prefix_call(q, k_cache, v_cache, n_pages, page_size, prefix_pages, prefix_len, table, B, max_pages, cu_new,
                       kv_len, max_new, R, N, Nkv, D, scale, o, o_dtype, lse, workspace, ws_bytes, 2000000000ull, false,
                       stream);
}

extern "C" cp_status cp_selftest_stalled_prefix_attn(
    const void *q, const void *k_cache, const void *v_cache, int64_t n_pages, int64_t page_size,
    const int32_t *prefix_pages, int64_t prefix_len, const int32_t *table, int64_t B, int64_t max_pages,
    const int32_t *cu_new, const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv, int64_t D,
    float scale, void *o, cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes, uint64_t timeout_ns,
    cudaStream_t stream) {
    if (timeout_ns < 1000000ull || timeout_ns > 2000000000ull) return CP_ERR_ARGUMENT;
    return prefix_call(q, k_cache, v_cache, n_pages, page_size, prefix_pages, prefix_len, table, B, max_pages, cu_new,
                       kv_len, max_new, R, N, Nkv, D, scale, o, o_dtype, lse, workspace, ws_bytes, timeout_ns, true,
                       stream);
}
