// cp_prefix.cuh -- how the shared-prefix attention lays its work on a line and
// cuts it into equal shares (prefix.cu, prefix_tc.cuh).
//
// A launch works on problems: the prefix with the rows of all sequences, the
// sequences with their own rows and keys, or both.  For one KV head the rows of
// a problem are its tokens times the G query heads of that KV head (row i =
// token i / G, head i % G), cut into tiles of TM rows; an item is one row tile
// of one KV head of one problem.  The items lie end to end on a line, each
// ceil(keys / KT) + E long (E: what beginning and ending it costs, in tiles), and
// worker c of W works on [c share, (c + 1) share).
//
// The KV heads of a token lie side by side in memory, and their work is the
// same, so blocks that run side by side take the same stretch of the line for
// neighbouring heads: block (x, y) is worker y of lane x, and the line of a lane
// holds heads lane, lane + lanes, ...  (a.heads of them).
//
// The row tiles of a causal problem need fewer keys than its length: a stretch
// [n0, n1) of an item of nominal length T that needs K tiles stands for tiles
// [n0 K / T, n1 K / T).  Row tiles from the beginning and the end take turns on
// the line, so neighbours cost about the average.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_hold.cuh"
#include "cp_paged.cuh"
#include "cp_ptx.cuh"
#include "cp_sched.cuh"

namespace cpattn {

constexpr int kTM = 16, kKT = 64;        // rows and keys of a narrow tile (mma.sync)
constexpr int kTcTM = 256, kTcKT = 128;  // of a wide one (tcgen05)
// What an item costs beside its tiles (queries, first scores, its partial), in
// tiles, for the shares of the line.  A 16-row item costs about 4600 cycles
// against 1200 a tile, a 256-row one of few rows 8 us against 2.  Without (0) a
// block that gets short sequences works on after the others are done: 32768 prefix
// keys and 64 sequences of 32 heads, one own key each, 167 us (71 with 3, 75 with 6);
// 16384 prefix keys and 64 prompts of 20 tokens 495 us (316, 331), 32 of 64 tokens
// 632 (488, 454), 8 of 512 tokens 1046 (886, 898).
constexpr int kExtra = 3;

struct PrefixArgs {
    const __nv_bfloat16 *q, *k, *v;
    PageTable own, pre;  // the sequences' pages; the prefix as a table of one row
    const int32_t *cu, *kv_len;
    int R, B, N, Nkv, G;
    FastDiv div_g;              // by G
    long long P;
    float scale_log2;
    int lanes, heads;           // Nkv = lanes x heads
    int with_prefix, with_own;  // the problems of this launch
    float cost;                 // cycles of a tile, where both kinds of tiles share a launch
    int *status;
    unsigned long long timeout_ns;
    const int *hold;  // self-test: the loads wait for this word (null: they do not)
    // what the launch leaves for the join
    long long *head;      // [0]: tiles of a share
    long long *base_tile; // [B] first tile of each sequence
    int *base_item;       // [B] first item of each sequence
    float2 *slot_ml;      // [slots][TM]: exponent, sum
    float *slot_o;        // [slots][TM][D], not divided by the sum
    int slots;            // of a lane
};

// A bad list never hides that a wait ran out.
__device__ __forceinline__ void report(int *status, cp_status code) {
    if (code == CP_ERR_DEVICE_TIMEOUT)
        atomicExch(status, static_cast<int>(code));
    else
        atomicCAS(status, static_cast<int>(CP_OK), static_cast<int>(code));
}

// The lists, tables and queries are read past L1 (__ldcg): a launch's blocks may
// have started while the kernel that writes them was still running.

// The self-test's wait, by one whole warp: true at once without one.
__device__ __forceinline__ bool released(const PrefixArgs &a, volatile int *abort_flag) {
    return !a.hold || __all_sync(0xffffffffu, hold_wait(a.hold, a.timeout_ns, abort_flag));
}

// One problem's shape.
struct Problem {
    int tok0, n;     // rows' tokens
    long long keys;  // keys in all
    int row_tiles;
    long long key_tiles;  // nominal length of an item
};

// Where every problem's tiles and items begin on the line (entry i + 1: run i of
// the sequences; entry 0: the prefix), in shared memory, and the lists of the
// first `listed` sequences where a kernel has room for them there.
constexpr int kRuns = 128;
struct Line {
    long long tile[kRuns + 1];
    int item[kRuns + 1];
    int worker, workers;  // this block's share, of how many
    int rows_end;         // cu[B]
    int listed;
    int *cu, *len;  // [listed + 1], [listed]
};

// Sequence b as the device lists give it; a list that makes no sense is cut to
// what can be read and reported.
template <int TM, int KT>
__device__ __forceinline__ Problem sequence_problem(const PrefixArgs &a, const Line &line, int b) {
    Problem p;
    const bool listed = b < line.listed;
    const int c0 = listed ? line.cu[b] : __ldcg(a.cu + b), c1 = listed ? line.cu[b + 1] : __ldcg(a.cu + b + 1);
    long long len = listed ? line.len[b] : __ldcg(a.kv_len + b);
    const long long most = static_cast<long long>(a.own.max_pages) << a.own.shift;
    p.tok0 = c0;
    p.n = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > a.R) {
        p.n = 0;
        report(a.status, CP_ERR_PAGE);
    }
    if (len < 0 || len > most) {
        len = len < 0 ? 0 : most;
        report(a.status, CP_ERR_PAGE);
    }
    p.keys = len;
    p.row_tiles = (p.n * a.G + TM - 1) / TM;
    p.key_tiles = p.n && len ? (len + KT - 1) / KT + kExtra : 0;
    return p;
}
template <int TM, int KT>
__device__ __forceinline__ Problem prefix_problem(const PrefixArgs &a, const Line &line) {
    Problem p;
    p.tok0 = 0;
    p.n = min(max(line.rows_end, 0), a.R);
    p.keys = a.P;
    p.row_tiles = (p.n * a.G + TM - 1) / TM;
    p.key_tiles = p.n && a.P ? (a.P + KT - 1) / KT + kExtra : 0;
    return p;
}

// Row tile at place w of a problem's turn order, and back.
__device__ __forceinline__ int tile_at(int w, int tiles) { return w & 1 ? tiles - 1 - (w >> 1) : w >> 1; }
__device__ __forceinline__ int place_of(int j, int tiles) {
    return j < (tiles + 1) / 2 ? 2 * j : 2 * (tiles - 1 - j) + 1;
}

// Fills `line`: the lists of up to `room` sequences (`lists`: 2 room + 1 values),
// sums over runs of sequences, and their scan.
template <int TM, int KT>
__device__ __forceinline__ void scan_line(const PrefixArgs &a, Line &line, int *lists, int room) {
    const int tid = threadIdx.x, run = (a.B + kRuns - 1) / kRuns, listed = a.with_own ? min(a.B, room) : 0;
    if (tid == 0) {
        line.rows_end = __ldcg(a.cu + a.B);
        line.worker = blockIdx.y;
        line.workers = gridDim.y;
        line.listed = listed;
        line.cu = lists;
        line.len = lists + room + 1;
    }
    for (int b = listed ? tid : 1; b <= listed; b += blockDim.x) {
        lists[b] = __ldcg(a.cu + b);
        if (b < listed) lists[room + 1 + b] = __ldcg(a.kv_len + b);
    }
    __syncthreads();
    const int b0 = min(tid * run, a.B), b1 = a.with_own ? min(b0 + run, a.B) : b0;
    if (tid < kRuns) {
        long long tiles = 0;
        int items = 0;
        for (int b = b0; b < b1; ++b) {
            const Problem p = sequence_problem<TM, KT>(a, line, b);
            tiles += static_cast<long long>(a.heads) * p.row_tiles * p.key_tiles;
            items += a.heads * p.row_tiles;
        }
        line.tile[tid + 1] = tiles;
        line.item[tid + 1] = items;
        if (tid == 0) {
            const Problem p = prefix_problem<TM, KT>(a, line);
            line.tile[0] = a.with_prefix ? static_cast<long long>(a.heads) * p.row_tiles * p.key_tiles : 0;
            line.item[0] = a.with_prefix ? a.heads * p.row_tiles : 0;
        }
    }
    __syncthreads();
    if (tid < 32) {
        // inclusive scan of 128 entries, 4 to a lane
        long long t[4];
        int n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = line.tile[1 + 4 * tid + i] + (i ? t[i - 1] : 0);
            n[i] = line.item[1 + 4 * tid + i] + (i ? n[i - 1] : 0);
        }
        long long ts = t[3];
        int ns = n[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long tv = __shfl_up_sync(0xffffffffu, ts, o);
            const int nv = __shfl_up_sync(0xffffffffu, ns, o);
            if (tid >= o) ts += tv, ns += nv;
        }
        const long long t0 = ts - t[3] + line.tile[0];
        const int n0 = ns - n[3] + line.item[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            line.tile[1 + 4 * tid + i] = t0 + t[i];
            line.item[1 + 4 * tid + i] = n0 + n[i];
        }
    }
    __syncthreads();
}

// Leaves the sequences' places for the join; by one block of the launch.
template <int TM, int KT>
__device__ __forceinline__ void leave_places(const PrefixArgs &a, const Line &line) {
    const int tid = threadIdx.x, run = (a.B + kRuns - 1) / kRuns;
    if (a.with_own && tid < kRuns) {
        const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
        long long t = line.tile[tid];
        int n = line.item[tid];
        for (int b = b0; b < b1; ++b) {
            const Problem p = sequence_problem<TM, KT>(a, line, b);
            a.base_tile[b] = t;
            a.base_item[b] = n;
            t += static_cast<long long>(a.heads) * p.row_tiles * p.key_tiles;
            n += a.heads * p.row_tiles;
        }
    }
}

// a / b for 0 <= a, 0 < b, by a 32-bit division where both fit.
__device__ __forceinline__ long long div_floor(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A block's share of its lane's line; false if it has none.
__device__ __forceinline__ bool share_of(const PrefixArgs &a, const Line &line, long long *t0, long long *t1) {
    const long long total = line.tile[kRuns];
    const long long share = max(1ll, div_floor(total + line.workers - 1, line.workers));
    if (blockIdx.x == 0 && line.worker == 0 && threadIdx.x == 0) a.head[0] = share;
    *t0 = share * line.worker;
    *t1 = min(*t0 + share, total);
    return *t0 < *t1;
}

// A row's (exponent, sum) as a piece leaves it.  A row whose scores so far are all
// NaN has no exponent, but must not pass for one that saw no key.
__device__ __forceinline__ float2 left_ml(float m, float l) {
    return make_float2(m == -INFINITY && l != l ? INFINITY : m, l);
}

// A stretch of one item that a block works on.
struct Piece {
    int b;                // sequence, -1: the prefix
    int slot;             // where the piece's partial goes, -1: nowhere
    int kvh, tok0, rows;  // rows of the problem
    int row0;             // first row of the tile
    int keys;             // keys of the problem
    int off;              // rows of token i see keys [0, off + i] (prefix: all)
    int k0, k1;           // key tiles [k0, k1), may be none
};

// Keys that row `row` of the problem sees: [0, limit).
__device__ __forceinline__ int row_limit(const PrefixArgs &a, const Piece &x, int row) {
    return x.b < 0 ? x.keys
                   : min(x.keys, max(0, x.off + static_cast<int>(fdiv(static_cast<uint32_t>(row), a.div_g)) + 1));
}

// Where a block's share begins: the item and the place in it.
struct Start {
    int b, pass, w, item;  // problem, head of the lane, row tile's place, index on the line
    long long n0;
};

// Finds the place t of the line.  By one whole warp; the caller shares `s`.
template <int TM, int KT>
__device__ __forceinline__ void find_start(const PrefixArgs &a, const Line &line, long long t, Start *s) {
    const int lane = threadIdx.x & 31;
    // runs that begin at or before t (their beginnings do not go back)
    int n = 0;
#pragma unroll
    for (int i = 0; i < kRuns / 32; ++i) n += line.tile[lane * (kRuns / 32) + i] <= t;
    const int lo = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n))) - 1;
    if (lane) return;
    Problem p;
    long long base = 0;
    int item = 0, b = -1;
    if (t < line.tile[0]) {
        p = prefix_problem<TM, KT>(a, line);
    } else {
        base = line.tile[lo];
        item = line.item[lo];
        const int run = (a.B + kRuns - 1) / kRuns;
        for (b = lo * run; b < a.B; ++b) {
            p = sequence_problem<TM, KT>(a, line, b);
            const long long all = static_cast<long long>(a.heads) * p.row_tiles * p.key_tiles;
            if (t < base + all) break;
            base += all;
            item += a.heads * p.row_tiles;
        }
    }
    s->b = b;
    if (b >= a.B) return;  // only when the lists were changed under the launch
    const long long at = t - base, which = div_floor(at, p.key_tiles);
    s->pass = static_cast<int>(div_floor(which, p.row_tiles));
    s->w = static_cast<int>(which - static_cast<long long>(s->pass) * p.row_tiles);
    s->item = item + static_cast<int>(which);
    s->n0 = at - which * p.key_tiles;
}

// Walks a block's pieces.  Every warp walks for itself, from the block's Start; a
// step is a few additions.  The walk and the piece it has come to lie in shared
// memory: they are looked at once in many tiles, and the registers of the tile
// loops are scarce.
template <int TM, int KT>
struct Walk {
    Problem p;
    Start s;
    long long left;  // nominal tiles of the share that are left
    Piece x;         // the piece come to
    // Warp-wide.
    __device__ __forceinline__ void begin(const PrefixArgs &a, const Line &line, const Start &start, long long share) {
        if ((threadIdx.x & 31) == 0) {
            s = start;
            left = share;
            if (s.b >= a.B) left = 0;
            else p = s.b < 0 ? prefix_problem<TM, KT>(a, line) : sequence_problem<TM, KT>(a, line, s.b);
        }
        __syncwarp();
    }
    // Comes to the next piece; false if there is none.  Warp-wide.
    __device__ __forceinline__ bool next(const PrefixArgs &a, const Line &line) {
        __syncwarp();
        const bool more = left > 0;
        __syncwarp();
        if (more && (threadIdx.x & 31) == 0) step(a, line);
        __syncwarp();
        return more;
    }
    __device__ __forceinline__ void step(const PrefixArgs &a, const Line &line) {
        const int lane = blockIdx.x, slot = s.item + line.worker;
        x.b = s.b;
        x.kvh = s.pass * a.lanes + lane;
        x.slot = slot < a.slots ? lane * a.slots + slot : -1;
        x.row0 = tile_at(s.w, p.row_tiles) * TM;
        x.tok0 = p.tok0;
        x.rows = p.n * a.G;
        x.keys = static_cast<int>(p.keys);
        x.off = x.keys - p.n;
        const long long n1 = min(s.n0 + left, p.key_tiles);
        const long long need = (static_cast<long long>(row_limit(a, x, min(x.row0 + TM, x.rows) - 1)) + KT - 1) / KT;
        // the part [n0, n1) of the nominal length, scaled to the tiles that the rows need
        x.k0 = static_cast<int>(s.n0 == 0 ? 0 : s.n0 * need / p.key_tiles);
        x.k1 = static_cast<int>(n1 == p.key_tiles ? need : n1 * need / p.key_tiles);
        left -= n1 - s.n0;
        s.n0 = 0;
        ++s.item;
        if (++s.w == p.row_tiles) {
            s.w = 0;
            if (++s.pass == a.heads) {
                s.pass = 0;
                // the next problem with work; the prefix comes before sequence 0
                while (left > 0) {
                    if (++s.b >= a.B) {
                        left = 0;  // only when the lists were changed under the launch
                        break;
                    }
                    p = sequence_problem<TM, KT>(a, line, s.b);
                    if (p.row_tiles > 0 && p.key_tiles > 0) break;
                    s.item += a.heads * p.row_tiles;
                }
            }
        }
    }
};

// The page numbers of a piece, for the warp that starts its copies: 32 entries
// of the page list side by side in the lanes and the next 32 on their way, so no
// tile waits for its page numbers.
struct PageWindow {
    const int32_t *list;
    int n, n_pages, shift;  // entries, pages of the cache
    int base, cur, next;    // first entry of `cur`
    __device__ __forceinline__ int fetch(int first, int lane) const {
        return first + lane < n ? __ldcg(list + first + lane) : -1;
    }
    __device__ __forceinline__ void begin(const PrefixArgs &a, const Piece &x, int first, int lane) {
        const PageTable &t = x.b < 0 ? a.pre : a.own;
        list = t.table + static_cast<long long>(max(x.b, 0)) * t.max_pages;
        n = min(t.max_pages, static_cast<int>((static_cast<long long>(x.keys) + (1 << t.shift) - 1) >> t.shift));
        n_pages = t.n_pages;
        shift = t.shift;
        base = first;
        cur = fetch(base, lane);
        next = fetch(base + 32, lane);
    }
    // Moves on so that entry `first` lies in the window (first never goes back). Warp-wide.
    __device__ __forceinline__ void advance(int first, int lane) {
        while (first >= base + 32) {
            base += 32;
            cur = next;
            next = fetch(base + 32, lane);
        }
    }
    // Cache row of each lane's key `key` (of an entry in the window), -1 for a key
    // past the last or a page number out of range.  Warp-wide.
    __device__ __forceinline__ int rows16(const PrefixArgs &a, int key, int keys) const {
        const int e = key >> shift;
        const int page = __shfl_sync(0xffffffffu, cur, (e - base) & 31);
        if (key >= keys) return -1;
        if (page < 0 || page >= n_pages) {
            report(a.status, CP_ERR_PAGE);
            return -1;
        }
        return (page << shift) + (key & ((1 << shift) - 1));
    }
    // Cache row of key `key` (uniform over the warp, of an entry in the window:
    // 32 is a multiple of a tile's pages, and the window began at a tile's
    // first); the row after the last page for a page number out of range.
    __device__ __forceinline__ int row(const PrefixArgs &a, int key) const {
        const int e = key >> shift;
        const int page = __shfl_sync(0xffffffffu, cur, (e - base) & 31);
        if (page < 0 || page >= n_pages) {
            report(a.status, CP_ERR_PAGE);
            return n_pages << shift;
        }
        return (page << shift) + (key & ((1 << shift) - 1));
    }
};

// Rows kI, kI + kRpi, ... up to 16 of a group, whole (kRpi rows an instruction).
template <int kRpi, int kI>
__device__ __forceinline__ void copy_rows(uint32_t at, uint32_t sw, const char *src, long long step) {
    if constexpr (kI < 16) {
        asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;" ::"r"(at + (sw ^ ((kI & 7) << 4))), "l"(src),
                     "n"(kI * 128)
                     : "memory");
        copy_rows<kRpi, kI + kRpi>(at, sw, src + step, step);
    }
}

// Starts the copies of one tile of KT keys of a piece (K or V) into shared
// memory, 64-column atoms of kAtom bytes, rows of 128 bytes, 128-byte swizzle, by
// one warp with 16-byte cp.async: a warp instruction moves whole head rows of D
// values, the page is looked up once for 16 rows, and keys past the piece's are
// filled with zeros.  TMA tiles of a small page are slower: a copy of 16 rows of
// 128 bytes holds the TMA unit for about 90 cycles, which ends at 3.4 TB/s over
// the GPU with two issuing warps and 4.4 with four, where this reaches 5.9.
// (The loop over 16-row groups is not unrolled: a block copies few tiles, and code
// that is read for the first time costs more than the loop.)
template <int D, int KT, int kAtom>  // KT: a multiple of 16, here also a part of a tile
__device__ __forceinline__ void copy_tile(const PrefixArgs &a, const Piece &x, const PageWindow &win,
                                          const __nv_bfloat16 *cache, uint32_t dst, int key0, int lane) {
    constexpr int kChunks = D / 8, kRpi = 32 / kChunks;  // 16-byte chunks of a row, rows of an instruction
    const int r = lane / kChunks, c = lane % kChunks;
    const long long row_bytes = static_cast<long long>(a.Nkv) * D * 2, step = kRpi * row_bytes;
    const char *lane_src = reinterpret_cast<const char *>(cache) + r * row_bytes + (x.kvh * D + c * 8) * 2;
    uint32_t at = dst + (c >> 3) * kAtom + r * 128;
    const uint32_t sw = ((c & 7) ^ r) << 4;
    // lane g looks up the rows 16 g .. 16 g + 15: where they begin, -1 for none (a bad page or no keys)
    const int mine = win.rows16(a, key0 + 16 * (lane % (KT / 16)), x.keys);
#pragma unroll 2
    for (int g = 0; g < KT / 16; ++g, at += 16 * 128) {
        const int left = x.keys - key0 - 16 * g, row = __shfl_sync(0xffffffffu, mine, g);
        const bool there = row >= 0;
        const char *src = lane_src + (there ? row : 0) * row_bytes;
        if (there && left >= 16) {
            copy_rows<kRpi, 0>(at, sw, src, step);
        } else {
#pragma unroll 1
            for (int i = 0; i < 16; i += kRpi, src += step) {
                const bool in = there && i + r < left;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + i * 128 + (sw ^ ((i & 7) << 4))),
                             "l"(in ? src : reinterpret_cast<const char *>(cache)), "r"(in ? 16 : 0)
                             : "memory");
            }
        }
    }
}
// Arrives on `bar` (count: one for each lane) when the lane's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace cpattn
