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
// 64-key tiles, and every block takes an equal share of that line, whatever the
// lengths are.  A share that covers part of an item leaves a partial; the k-th
// piece of the line has slot (item + block), which is unique, so the slots need
// no counter.  A second launch joins the pieces of every row in their order:
// the result does not depend on timing.
//
// Inside a block: 4 warps share a double-buffered 64-key stage filled by
// cp.async (page numbers checked, keys past the length zero-filled, so stale
// values in the last page never meet an MMA); each warp owns 16 of the 64 keys,
// so every byte of K and V passes from shared memory to registers once.  Both
// products run on mma.sync m16n8k16: at 16 rows the tensor work is a tenth of
// what the SM can do while it waits for memory.  Running maximum and sum stay in
// fp32 registers; P is rounded to bf16 for the second product (2^-9 of each
// weight at most, as in cp_attn_partial).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "cp_internal.h"
#include "cp_paged.cuh"
#include "cp_ptx.cuh"

namespace cpattn {
namespace {

__device__ int g_prefix_status = 0;

constexpr int kThreads = 128;
constexpr int kKT = 64;  // keys of a stage

struct PrefixArgs {
    const __nv_bfloat16 *q, *k, *v;
    PageTable own, pre;  // the sequences' pages; the prefix as a table of one row
    const int32_t *cu, *kv_len;
    int R, B, N, Nkv, G;
    long long P;
    float scale_log2;
    void *o;
    int o_bf16;
    float *lse;
    // workspace
    long long *head;        // [0]: tiles of a share
    long long *base_tile;   // [B] first tile of each sequence
    int *base_item;         // [B]
    float *slot_ml;         // [slots][TM][2]
    float *slot_o;          // [slots][TM][D]
    int slots;
};

// One problem's shape.
struct Problem {
    int tok0, n;        // rows' tokens
    long long keys;     // keys in all
    int row_tiles;
    long long key_tiles;
};

// Sequence b as the device lists give it; a list that makes no sense is cut to
// what can be read and reported.
__device__ __forceinline__ Problem sequence_problem(const PrefixArgs &a, int b, int tm) {
    Problem p;
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    long long len = __ldg(a.kv_len + b);
    const long long most = static_cast<long long>(a.own.max_pages) << a.own.shift;
    p.tok0 = c0;
    p.n = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > a.R) {
        p.n = 0;
        atomicExch(&g_prefix_status, static_cast<int>(CP_ERR_PAGE));
    }
    if (len < 0 || len > most) {
        len = len < 0 ? 0 : most;
        atomicExch(&g_prefix_status, static_cast<int>(CP_ERR_PAGE));
    }
    p.keys = len;
    p.row_tiles = (p.n * a.G + tm - 1) / tm;
    p.key_tiles = p.n ? (len + kKT - 1) / kKT : 0;
    return p;
}
__device__ __forceinline__ Problem prefix_problem(const PrefixArgs &a, int tm) {
    Problem p;
    p.tok0 = 0;
    p.n = min(max(__ldg(a.cu + a.B), 0), a.R);
    p.keys = a.P;
    p.row_tiles = (p.n * a.G + tm - 1) / tm;
    p.key_tiles = p.n ? (a.P + kKT - 1) / kKT : 0;
    return p;
}

// Where every problem's tiles and items begin on the line: sums over the
// thread's run of sequences, scanned over the block (128 entries in shared
// memory however many sequences there are).
struct Line {
    long long tile[kThreads + 1];
    int item[kThreads + 1];
};

__device__ __forceinline__ void scan_line(const PrefixArgs &a, int tm, Line &line, bool publish) {
    const int tid = threadIdx.x, run = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
    long long tiles = 0;
    int items = 0;
    for (int b = b0; b < b1; ++b) {
        const Problem p = sequence_problem(a, b, tm);
        tiles += static_cast<long long>(a.Nkv) * p.row_tiles * p.key_tiles;
        items += a.Nkv * p.row_tiles;
    }
    line.tile[tid + 1] = tiles;
    line.item[tid + 1] = items;
    if (tid == 0) {
        const Problem p = prefix_problem(a, tm);
        line.tile[0] = static_cast<long long>(a.Nkv) * p.row_tiles * p.key_tiles;
        line.item[0] = a.Nkv * p.row_tiles;
    }
    __syncthreads();
    if (tid < 32) {
        // inclusive scan of 128 entries, 4 to a lane
        long long t[4];
        int n[4];
        for (int i = 0; i < 4; ++i) {
            t[i] = line.tile[1 + 4 * tid + i] + (i ? t[i - 1] : 0);
            n[i] = line.item[1 + 4 * tid + i] + (i ? n[i - 1] : 0);
        }
        long long ts = t[3];
        int ns = n[3];
        for (int o = 1; o < 32; o <<= 1) {
            const long long tv = __shfl_up_sync(0xffffffffu, ts, o);
            const int nv = __shfl_up_sync(0xffffffffu, ns, o);
            if (tid >= o) ts += tv, ns += nv;
        }
        const long long t0 = ts - t[3] + line.tile[0];
        const int n0 = ns - n[3] + line.item[0];
        for (int i = 0; i < 4; ++i) {
            line.tile[1 + 4 * tid + i] = t0 + t[i];
            line.item[1 + 4 * tid + i] = n0 + n[i];
        }
    }
    __syncthreads();
    if (publish) {
        long long t = line.tile[tid];
        int n = line.item[tid];
        for (int b = b0; b < b1; ++b) {
            const Problem p = sequence_problem(a, b, tm);
            a.base_tile[b] = t;
            a.base_item[b] = n;
            t += static_cast<long long>(a.Nkv) * p.row_tiles * p.key_tiles;
            n += a.Nkv * p.row_tiles;
        }
    }
}

// A stretch of one item that a block works on.
struct Piece {
    int b;               // sequence, -1: the prefix
    int item;            // index on the line
    int kvh, tok0, rows; // rows of the problem
    int row0;            // first row of the tile
    long long keys;      // keys of the problem
    long long off;       // rows of token i see keys [0, off + i] (prefix: all)
    long long k0, k1;    // key tiles [k0, k1)
};

// The piece that begins at tile t of the line (t < end), cut at `end`.
__device__ __forceinline__ Piece find_piece(const PrefixArgs &a, int tm, const Line &line, long long t, long long end) {
    Piece x;
    Problem p;
    long long base = 0;
    int item = 0;
    if (t < line.tile[0]) {
        p = prefix_problem(a, tm);
        x.b = -1;
    } else {
        // the thread run that holds t: the last entry with tile <= t
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line.tile[mid] <= t) lo = mid; else hi = mid - 1;
        }
        const int run = (a.B + kThreads - 1) / kThreads;
        base = line.tile[lo];
        item = line.item[lo];
        int b = lo * run;
        for (; b < a.B; ++b) {
            p = sequence_problem(a, b, tm);
            const long long all = static_cast<long long>(a.Nkv) * p.row_tiles * p.key_tiles;
            if (t < base + all) break;
            base += all;
            item += a.Nkv * p.row_tiles;
        }
        x.b = b;
        if (b >= a.B) {
            // only when the lists were changed under the launch: a stretch without rows
            x = Piece{};
            x.k1 = end - t;
            return x;
        }
    }
    const long long at = t - base, which = at / p.key_tiles;
    x.item = item + static_cast<int>(which);
    x.kvh = static_cast<int>(which / p.row_tiles);
    x.row0 = static_cast<int>(which - static_cast<long long>(x.kvh) * p.row_tiles) * tm;
    x.tok0 = p.tok0;
    x.rows = p.n * a.G;
    x.keys = p.keys;
    x.off = x.b < 0 ? a.P : p.keys - p.n;
    x.k0 = at - which * p.key_tiles;
    x.k1 = x.k0 + (end - t) < p.key_tiles ? x.k0 + (end - t) : p.key_tiles;
    return x;
}

// Keys that row i of the problem sees: [0, limit).
__device__ __forceinline__ long long row_limit(const PrefixArgs &a, const Piece &x, int row) {
    if (row >= x.rows) return 0;
    return x.b < 0 ? x.keys : x.off + row / a.G + 1;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
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

template <int D>
struct MmaCfg {
    static constexpr int kTM = 16;
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kKT * kRowBytes;     // K or V of a stage
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kOffOut = kStages * 2 * kTileBytes;  // [4 warps][16 rows][D] fp32
    static constexpr int kOffMl = kOffOut + 4 * 16 * D * 4;   // [4][16][2]
    static constexpr int kOffLine = kOffMl + 4 * 16 * 2 * 4;
    static constexpr int kSmem = kOffLine + static_cast<int>(sizeof(Line));
};

// Byte offset of 16-byte chunk c of row r in a stage tile: chunks are permuted
// by the row's low bits, so the 8 rows of an ldmatrix phase hit 8 bank groups.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) prefix_mma_kernel(const PrefixArgs a) {
    using C = MmaCfg<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    Line &line = *reinterpret_cast<Line *>(smem + C::kOffLine);
    float *out_s = reinterpret_cast<float *>(smem + C::kOffOut);
    float *ml_s = reinterpret_cast<float *>(smem + C::kOffMl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);

    scan_line(a, C::kTM, line, blockIdx.x == 0);
    const long long total = line.tile[kThreads];
    long long share = (total + gridDim.x - 1) / gridDim.x;
    if (share < 1) share = 1;
    if (blockIdx.x == 0 && tid == 0) a.head[0] = share;
    const long long t0 = share * blockIdx.x, t1 = min(t0 + share, total);
    if (t0 >= t1) return;

    // loads run ahead of the products over the tiles of all the block's pieces
    Piece lp = find_piece(a, C::kTM, line, t0, t1);
    long long lt = t0, lk = lp.k0;
    int lstage = 0;
    auto load_next = [&]() {
        if (lt < t1) {
            const PageTable &pt = lp.b < 0 ? a.pre : a.own;
            const int last_row = min(lp.row0 + C::kTM, lp.rows) - 1;
            const long long limit = row_limit(a, lp, last_row);  // keys that any row of the tile sees
            const uint32_t ks = sbase + lstage * 2 * C::kTileBytes, vs = ks + C::kTileBytes;
            constexpr int kChunks = D / 8, kStep = kThreads / kChunks;  // rows between a thread's chunks
            const int c = tid % kChunks;
#pragma unroll
            for (int r = tid / kChunks; r < kKT; r += kStep) {
                const long long key = lk * kKT + r;
                long long slot = -1;
                if (key < limit) {
                    slot = pt.slot(lp.b < 0 ? 0 : lp.b, key);
                    if (slot < 0 && c == 0) atomicExch(&g_prefix_status, static_cast<int>(CP_ERR_PAGE));
                }
                const long long off = slot < 0 ? 0 : (slot * a.Nkv + lp.kvh) * D + c * 8;
                cp_async16(ks + tile_off<D>(r, c), a.k + off, slot >= 0);
                cp_async16(vs + tile_off<D>(r, c), a.v + off, slot >= 0);
            }
            lstage = lstage + 1 == C::kStages ? 0 : lstage + 1;
            ++lt;
            if (++lk == lp.k1 && lt < t1) {
                lp = find_piece(a, C::kTM, line, lt, t1);
                lk = lp.k0;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load_next();

    const int g = lane >> 2, t4 = lane & 3;  // accumulator row (and row + 8), column pair
    int stage = 0;
    for (long long t = t0; t < t1;) {
        const Piece x = find_piece(a, C::kTM, line, t, t1);
        // this warp's copy of the rows as A operands
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = x.row0 + g + 8 * h;
            const bool ok = row < x.rows;
            const int tok = row / a.G;
            const __nv_bfloat16 *qp =
                a.q + (static_cast<long long>(x.tok0 + (ok ? tok : 0)) * a.N + x.kvh * a.G + (ok ? row - tok * a.G : 0)) * D;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[kk][h] = ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + kk * 16 + 2 * t4)) : 0u;
                qf[kk][2 + h] = ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + kk * 16 + 8 + 2 * t4)) : 0u;
            }
        }
        const long long lim0 = row_limit(a, x, x.row0 + g), lim1 = row_limit(a, x, x.row0 + g + 8);
        // tiles from the first that some row does not see whole on are masked
        const long long whole = x.row0 + C::kTM <= x.rows ? row_limit(a, x, x.row0) : 0;
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (long long kt = x.k0; kt < x.k1; ++kt, ++t) {
            load_next();
            cp_async_wait<C::kStages - 1>();
            __syncthreads();
            const uint32_t ks = sbase + stage * 2 * C::kTileBytes, vs = ks + C::kTileBytes;
            const int key0 = warp * 16;
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                // lanes 0-7: keys 0-7, low 8 columns; 8-15: high; 16-31: keys 8-15
                ldsm4(ks + tile_off<D>(key0 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)), b);
                mma16816(s[0], qf[kk], b[0], b[1]);
                mma16816(s[1], qf[kk], b[2], b[3]);
            }
            const long long kb = kt * kKT + key0 + 2 * t4;
            const bool masked = kt * kKT + kKT > whole;
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
                ldsm4t(vs + tile_off<D>(key0 + (lane & 15), 2 * n + (lane >> 4)), b);
                mma16816(o[2 * n], pf, b[0], b[1]);
                mma16816(o[2 * n + 1], pf, b[2], b[3]);
            }
            __syncthreads();  // the stage may be filled again
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }
        // join the four warps' keys and leave the piece's partial
        const int slot = x.item + static_cast<int>(blockIdx.x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (t4 == 0) {
                ml_s[(warp * 16 + g + 8 * h) * 2] = m[h];
                ml_s[(warp * 16 + g + 8 * h) * 2 + 1] = l[h];
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(out_s + (warp * 16 + g + 8 * h) * D + ((8 * n + 2 * t4) ^ ((g & 3) << 3))) =
                    make_float2(o[n][2 * h], o[n][2 * h + 1]);
        }
        __syncthreads();
        if (slot < a.slots) {
            constexpr int kPer = 16 * D / kThreads;  // values of a thread: part of one row
            const int row = tid / (kThreads / 16), c0 = (tid % (kThreads / 16)) * kPer;
            float mw[4], f[4], mx = -INFINITY, ls = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                mw[w] = ml_s[(w * 16 + row) * 2];
                mx = fmaxf(mx, mw[w]);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                f[w] = mw[w] == -INFINITY ? 0.f : fast_exp2(mw[w] - mx);
                ls += f[w] * ml_s[(w * 16 + row) * 2 + 1];
            }
            float *dst = a.slot_o + (static_cast<long long>(slot) * 16 + row) * D;
#pragma unroll
            for (int c = c0; c < c0 + kPer; c += 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 y = *reinterpret_cast<const float4 *>(out_s + (w * 16 + row) * D + (c ^ ((row & 3) << 3)));
                    if (f[w] != 0.f) {  // a warp that saw nothing holds zeros
                        v.x += f[w] * y.x;
                        v.y += f[w] * y.y;
                        v.z += f[w] * y.z;
                        v.w += f[w] * y.w;
                    }
                }
                *reinterpret_cast<float4 *>(dst + c) = v;
            }
            if (c0 == 0) {
                a.slot_ml[(static_cast<long long>(slot) * 16 + row) * 2] = mx;
                a.slot_ml[(static_cast<long long>(slot) * 16 + row) * 2 + 1] = ls;
            }
        } else if (tid == 0) {
            atomicExch(&g_prefix_status, static_cast<int>(CP_ERR_PAGE));
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// One warp joins the pieces of one output row (token, head).
template <int D>
__global__ void __launch_bounds__(128) prefix_join_kernel(const PrefixArgs a) {
    constexpr int TM = MmaCfg<D>::kTM, kV = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.R) * a.N) return;
    const int tok = static_cast<int>(row / a.N), h = static_cast<int>(row - static_cast<long long>(tok) * a.N);
    const int kvh = h / a.G, gh = h - kvh * a.G;
    int begin, count;
    const int b = find_sequence(a.cu, a.B, tok, lane, &begin, &count);
    if (b < 0) return;
    const long long share = a.head[0];
    // the stretch of the line and the slots of the row's two items
    long long first[2], last[2];
    int item[2], r[2];
    {
        const Problem p = prefix_problem(a, TM);
        const int i = tok * a.G + gh;
        const long long at = static_cast<long long>(kvh) * p.row_tiles + i / TM;
        item[0] = static_cast<int>(at);
        first[0] = at * p.key_tiles;
        last[0] = first[0] + p.key_tiles;
        r[0] = i % TM;
    }
    {
        const Problem p = sequence_problem(a, b, TM);
        const int i = (tok - begin) * a.G + gh;
        const long long at = static_cast<long long>(kvh) * p.row_tiles + i / TM;
        item[1] = __ldg(a.base_item + b) + static_cast<int>(at);
        first[1] = __ldg(a.base_tile + b) + at * p.key_tiles;
        last[1] = first[1] + p.key_tiles;
        r[1] = i % TM;
    }
    float mx = -INFINITY, ls = 0.f, acc[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.f;
    for (int part = 0; part < 2; ++part) {
        if (first[part] >= last[part]) continue;
        const int c0 = static_cast<int>(first[part] / share), c1 = static_cast<int>((last[part] - 1) / share);
        for (int cb = c0; cb <= c1; cb += 32) {
            // up to 32 pieces: their (m, l) side by side, then their rows one after another
            const int slot = item[part] + cb + lane;
            float pm = -INFINITY, pl = 0.f;
            if (cb + lane <= c1 && slot < a.slots) {
                const float2 ml = __ldg(reinterpret_cast<const float2 *>(a.slot_ml) + static_cast<long long>(slot) * TM + r[part]);
                pm = ml.x;
                pl = ml.y;
            }
            float top = pm;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top == -INFINITY) continue;
            if (top > mx) {
                const float f = mx == -INFINITY ? 0.f : fast_exp2(mx - top);
                ls *= f;
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[e] *= f;
                mx = top;
            }
            const float w = pm == -INFINITY ? 0.f : fast_exp2(pm - mx);
            float add = w * pl;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
            ls += add;
            const int n = min(32, c1 - cb + 1);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float f = __shfl_sync(0xffffffffu, w, i);
                const float *src = a.slot_o + (static_cast<long long>(item[part] + cb + i) * TM + r[part]) * D + lane * kV;
                if (f != 0.f) {
                    if (kV == 4) {
                        const float4 y = __ldg(reinterpret_cast<const float4 *>(src));
                        acc[0] += f * y.x, acc[1] += f * y.y, acc[2 % kV] += f * y.z, acc[3 % kV] += f * y.w;
                    } else {
                        const float2 y = __ldg(reinterpret_cast<const float2 *>(src));
                        acc[0] += f * y.x, acc[1] += f * y.y;
                    }
                }
            }
        }
    }
    const float inv = mx == -INFINITY ? 0.f : 1.f / ls;
    const long long at = row * D + lane * kV;
    if (a.o_bf16) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.o) + at);
#pragma unroll
        for (int e = 0; e < kV; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    } else {
        float *dst = static_cast<float *>(a.o) + at;
#pragma unroll
        for (int e = 0; e < kV; ++e) dst[e] = acc[e] * inv;
    }
    if (lane == 0)
        a.lse[static_cast<long long>(h) * a.R + tok] =
            mx == -INFINITY ? -INFINITY : (mx + log2f(ls)) * 0.69314718055994530942f;
}

// ---------------------------------------------------------------- host side
int grid_blocks() { return 2 * sm_count(); }

struct Layout {
    size_t base_tile, base_item, slot_ml, slot_o, bytes;
    long long slots;
};
Layout layout_of(int64_t R, int64_t B, int64_t N, int64_t Nkv, int64_t D) {
    const long long G = N / Nkv, tiles = (R * G + 15) / 16;
    Layout l;
    // every row tile of the prefix, of the sequences (each may end a tile early), and a cut for each block
    l.slots = Nkv * (2 * tiles + B) + 2 * 160;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    l.base_tile = 256;
    l.base_item = up(l.base_tile + B * 8);
    l.slot_ml = up(l.base_item + B * 4);
    l.slot_o = up(l.slot_ml + static_cast<size_t>(l.slots) * 16 * 8);
    l.bytes = up(l.slot_o + static_cast<size_t>(l.slots) * 16 * D * 4);
    return l;
}

template <int D>
cp_status launch_typed(const PrefixArgs &a, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(prefix_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaCfg<D>::kSmem);
    });
    if (err != cudaSuccess) return cuda_status(err);
    const int grid = grid_blocks() < 320 ? grid_blocks() : 320;
    prefix_mma_kernel<D><<<grid, kThreads, MmaCfg<D>::kSmem, stream>>>(a);
    cp_status st = last_launch_status();
    if (st != CP_OK) return st;
    const long long rows = static_cast<long long>(a.R) * a.N;
    prefix_join_kernel<D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(a);
    return last_launch_status();
}

cp_status check_sizes(int64_t R, int64_t B, int64_t max_new, int64_t P, int64_t N, int64_t Nkv, int64_t D,
                      int64_t page_size, int64_t max_pages) {
    if (R < 1 || N < 1 || N > 65535 || max_new < 1 || max_new > R || P < 0 || P > INT32_MAX) return CP_ERR_SHAPE;
    const cp_status st = check_pages(1, page_size, B, max_pages, Nkv, D);
    if (st != CP_OK) return st;
    if (N % Nkv) return CP_ERR_DIVISIBILITY;
    if (R * N > INT32_MAX / 4) return CP_ERR_SHAPE;
    return CP_OK;
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
    *bytes = layout_of(R, B, N, Nkv, D).bytes;
    return CP_OK;
}

extern "C" cp_status cp_prefix_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                        int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                        const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                        const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv,
                                        int64_t D, float scale, void *o, cp_dtype o_dtype, float *lse,
                                        void *workspace, size_t ws_bytes, cudaStream_t stream) {
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
    const Layout l = layout_of(R, B, N, Nkv, D);
    if (!workspace || ws_bytes < l.bytes) return CP_ERR_WORKSPACE;
    if (odd(workspace, 256)) return CP_ERR_ALIGNMENT;
    PrefixArgs a{};
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
    a.P = prefix_len;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    a.o = o;
    a.o_bf16 = o_dtype == CP_BF16;
    a.lse = lse;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    a.head = reinterpret_cast<long long *>(w);
    a.base_tile = reinterpret_cast<long long *>(w + l.base_tile);
    a.base_item = reinterpret_cast<int *>(w + l.base_item);
    a.slot_ml = reinterpret_cast<float *>(w + l.slot_ml);
    a.slot_o = reinterpret_cast<float *>(w + l.slot_o);
    a.slots = static_cast<int>(l.slots);
    return D == 128 ? launch_typed<128>(a, stream) : launch_typed<64>(a, stream);
}
