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
#include "cp_prefix.cuh"
#include "cp_ptx.cuh"
#include "prefix_tc.cuh"

namespace cpattn {
namespace {

__device__ int g_prefix_status = 0;

// A problem whose rows for one KV head are more than this runs in tiles of 256
// rows on the tensor memory, else in tiles of 16.
constexpr int kTcRows = 16;

constexpr int kThreads = 128;
constexpr int kTM = 16;  // rows of a tile
constexpr int kKT = 64;  // keys of a stage

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

    scan_line<kTM, kKT>(a, line, blockIdx.x == 0);
    long long t0, t1;
    if (!share_of(a, line, &t0, &t1)) return;

    // loads run ahead of the products over the tiles of all the block's pieces
    Piece lp = find_piece<kTM, kKT>(a, line, t0, t1);
    long long lk = lp.k0;
    int lstage = 0;
    auto load_next = [&]() {
        while (lk == lp.k1 && lp.next < t1) {
            lp = find_piece<kTM, kKT>(a, line, lp.next, t1);
            lk = lp.k0;
        }
        if (lk < lp.k1) {
            const PageTable &pt = lp.b < 0 ? a.pre : a.own;
            // keys that any row of the tile sees
            const long long limit = min(lp.keys, row_limit(a, lp, min(lp.row0 + kTM, lp.rows) - 1));
            const uint32_t ks = sbase + lstage * 2 * C::kTileBytes, vs = ks + C::kTileBytes;
            constexpr int kChunks = D / 8, kStep = kThreads / kChunks;  // rows between a thread's chunks
            const int c = tid % kChunks;
#pragma unroll
            for (int r = tid / kChunks; r < kKT; r += kStep) {
                const long long key = lk * kKT + r;
                long long slot = -1;
                if (key < limit) {
                    slot = pt.slot(lp.b < 0 ? 0 : lp.b, key);
                    if (slot < 0 && c == 0) report(a.status, CP_ERR_PAGE);
                }
                const long long off = slot < 0 ? 0 : (slot * a.Nkv + lp.kvh) * D + c * 8;
                cp_async16(ks + tile_off<D>(r, c), a.k + off, slot >= 0);
                cp_async16(vs + tile_off<D>(r, c), a.v + off, slot >= 0);
            }
            lstage = lstage + 1 == C::kStages ? 0 : lstage + 1;
            ++lk;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load_next();

    const int g = lane >> 2, t4 = lane & 3;  // accumulator row (and row + 8), column pair
    int stage = 0;
    for (long long t = t0; t < t1;) {
        const Piece x = find_piece<kTM, kKT>(a, line, t, t1);
        t = x.next;
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
        const long long lim0 = x.row0 + g < x.rows ? min(x.keys, row_limit(a, x, x.row0 + g)) : 0;
        const long long lim1 = x.row0 + g + 8 < x.rows ? min(x.keys, row_limit(a, x, x.row0 + g + 8)) : 0;
        // tiles from the first that some row does not see whole on are masked
        const long long whole = x.row0 + kTM <= x.rows ? min(x.keys, row_limit(a, x, x.row0)) : 0;
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (long long kt = x.k0; kt < x.k1; ++kt) {
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
            if (c0 == 0) a.slot_ml[static_cast<long long>(slot) * 16 + row] = make_float2(mx, ls);
        } else if (tid == 0) {
            report(a.status, CP_ERR_PAGE);
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// What a launch left, as the join reads it.
struct JoinPart {
    const long long *head, *base_tile;
    const int *base_item;
    const float2 *slot_ml;
    const float *slot_o;
    int slots, tm, kt;
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

// One warp joins the pieces of one output row (token, head).
template <int D>
__global__ void __launch_bounds__(128) prefix_join_kernel(const JoinArgs a) {
    constexpr int kV = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.R) * a.N) return;
    const int tok = static_cast<int>(row / a.N), h = static_cast<int>(row - static_cast<long long>(tok) * a.N);
    const int kvh = h / a.G, gh = h - kvh * a.G;
    int begin, count;
    const int b = find_sequence(a.cu, a.B, tok, lane, &begin, &count);
    if (b < 0) return;
    float mx = -INFINITY, ls = 0.f, acc[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const JoinPart &p = a.part[which];
        // the row's item: its stretch of the line, its pieces' slots and its row in them
        const int n = which ? count : min(max(__ldg(a.cu + a.B), 0), a.R);
        const long long keys = which ? min(max(static_cast<long long>(__ldg(a.kv_len + b)), 0ll), a.most) : a.P;
        const long long key_tiles = (keys + p.kt - 1) / p.kt;
        if (key_tiles == 0) continue;
        const int row_tiles = (n * a.G + p.tm - 1) / p.tm, i = (tok - (which ? begin : 0)) * a.G + gh, r = i % p.tm;
        if (i >= n * a.G) continue;
        const long long at = static_cast<long long>(kvh) * row_tiles + place_of(i / p.tm, row_tiles);
        const int item = (which ? __ldg(p.base_item + b) : 0) + static_cast<int>(at);
        const long long first = (which ? __ldg(p.base_tile + b) : 0) + at * key_tiles;
        const long long share = __ldg(p.head);
        const int c0 = static_cast<int>(first / share), c1 = static_cast<int>((first + key_tiles - 1) / share);
        for (int cb = c0; cb <= c1; cb += 32) {
            // up to 32 pieces: their (m, l) side by side, then their rows one after another
            const int slot = item + cb + lane;
            float pm = -INFINITY, pl = 0.f;
            if (cb + lane <= c1 && slot < p.slots) {
                const float2 ml = __ldg(p.slot_ml + static_cast<long long>(slot) * p.tm + r);
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
            const int m = min(32, c1 - cb + 1);
#pragma unroll 4
            for (int k = 0; k < m; ++k) {
                const float f = __shfl_sync(0xffffffffu, w, k);
                const float *src = p.slot_o + (static_cast<long long>(item + cb + k) * p.tm + r) * D + lane * kV;
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
constexpr int kMaxBlocks = 320;  // of a launch (a slot more for each)

// How a call is cut: which launches it makes and where they leave their pieces.
struct Shape {
    bool tc_prefix, tc_own;  // tensor-memory tiles of 256 rows, else tiles of 16 rows
    long long slots[2];      // of the 16-row launch and the 256-row launch (0: not made)
    size_t head[2], base_tile[2], base_item[2], slot_ml[2], slot_o[2], bytes;
};

Shape shape_of(int64_t R, int64_t B, int64_t max_new, int64_t P, int64_t N, int64_t Nkv, int64_t D) {
    const long long G = N / Nkv;
    Shape s{};
    s.tc_prefix = R * G > kTcRows;
    s.tc_own = max_new * G > kTcRows;
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
        s.slots[k] = Nkv * ((pre ? tiles : 0) + (own ? tiles + (B < R ? B : R) : 0)) + kMaxBlocks;
        s.head[k] = take(8);
        s.base_tile[k] = take(B * 8);
        s.base_item[k] = take(B * 4);
        s.slot_ml[k] = take(static_cast<size_t>(s.slots[k]) * tm * 8);
        s.slot_o[k] = take(static_cast<size_t>(s.slots[k]) * tm * D * 4);
    }
    s.bytes = at;
    return s;
}

template <int D>
cp_status launch_mma(const PrefixArgs &a, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(prefix_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaCfg<D>::kSmem);
    });
    if (err != cudaSuccess) return cuda_status(err);
    const int grid = 2 * sm_count() < kMaxBlocks ? 2 * sm_count() : kMaxBlocks;
    prefix_mma_kernel<D><<<grid, kThreads, MmaCfg<D>::kSmem, stream>>>(a);
    return last_launch_status();
}

template <int D>
cp_status launch_tc(const PrefixArgs &a, int64_t slots, int box_rows, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(prefix_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D>::kSmem);
    });
    if (err != cudaSuccess) return cuda_status(err);
    CUtensorMap mk, mv;
    if (!make_map(&mk, a.k, D, a.Nkv, slots, 1, box_rows) || !make_map(&mv, a.v, D, a.Nkv, slots, 1, box_rows))
        return CP_ERR_CUDA;
    const int grid = sm_count() < kMaxBlocks ? sm_count() : kMaxBlocks;
    prefix_tc_kernel<D><<<grid, kTcThreads, TcCfg<D>::kSmem, stream>>>(mk, mv, a);
    return last_launch_status();
}

template <int D>
cp_status launch_call(PrefixArgs a, const Shape &s, uint8_t *w, JoinArgs j, cudaStream_t stream) {
    const int64_t slots = static_cast<int64_t>(a.own.n_pages) << a.own.shift;
    const int box_rows = a.own.shift < 7 ? 1 << a.own.shift : 128;
    // the wide launch first: it has the prefix, the longer work
    for (int k = 1; k >= 0; --k) {
        if (!s.slots[k]) continue;
        a.with_prefix = a.P > 0 && s.tc_prefix == (k == 1);
        a.with_own = s.tc_own == (k == 1);
        a.head = reinterpret_cast<long long *>(w + s.head[k]);
        a.base_tile = reinterpret_cast<long long *>(w + s.base_tile[k]);
        a.base_item = reinterpret_cast<int *>(w + s.base_item[k]);
        a.slot_ml = reinterpret_cast<float2 *>(w + s.slot_ml[k]);
        a.slot_o = reinterpret_cast<float *>(w + s.slot_o[k]);
        a.slots = static_cast<int>(s.slots[k]);
        const cp_status st = k ? launch_tc<D>(a, slots, box_rows, stream) : launch_mma<D>(a, stream);
        if (st != CP_OK) return st;
        for (int which = 0; which < 2; ++which)
            if (which ? a.with_own : a.with_prefix)
                j.part[which] = JoinPart{a.head, a.base_tile, a.base_item, a.slot_ml, a.slot_o, a.slots,
                                         k ? kTcTM : kTM, k ? kTcKT : kKT};
    }
    if (a.P == 0) j.part[0] = j.part[1];  // not read into a result: no keys
    const long long rows = static_cast<long long>(a.R) * a.N;
    prefix_join_kernel<D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(j);
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
    const Shape s = shape_of(R, B, max_new, prefix_len, N, Nkv, D);
    if (!workspace || ws_bytes < s.bytes) return CP_ERR_WORKSPACE;
    if (odd(workspace, 256)) return CP_ERR_ALIGNMENT;
    if (s.slots[0] > INT32_MAX || s.slots[1] > INT32_MAX) return CP_ERR_SHAPE;
    PrefixArgs a{};
    if ((st = status_word(&a.status)) != CP_OK) return st;
    a.timeout_ns = 2000000000ull;
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
