// tree.cu -- trees of drafted tokens: their ancestors and positions (cp_tree_plan), and attention over the paged cache by
// them (cp_tree_attn_fwd: a block an item, tree_block.cuh, a cluster an item, tree_cluster.cuh, or the line of
// prefix_call.cuh and prefix_tc.cuh, with a row's mask in the place of its index wherever a key tile reaches into the
// step's new tokens).
//
// Ancestors.  mask_j = {j} + mask_parent(j).  A warp holds 32 tokens in a row, a token a lane, and follows the
// parents among them by doubling (five rounds of shuffles, whatever the tree's shape): each token then knows its branch
// among these 32, one word of its mask, and the earlier token that the branch hangs on.  From there it goes from
// word to word, 16 steps for 512 tokens at most, two reads of shared memory each, all tokens side by side.  300 trees of
// up to 500 tokens take 5.2 us in a graph so; 9.4 where the warps came one after the other and took whole rows over,
// 15.9 by doubling through shared memory over the whole tree.  What bounds it is the latency of the launch and of
// two loads that hang on one another (counts, parents).
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_internal.h"
#include "prefix_call.cuh"
#include "tree_block.cuh"
#include "tree_cluster.cuh"

namespace cpattn {
namespace {

constexpr int kMaxWords = 16;  // of a mask's row: trees of up to 512 tokens

struct TreeArgs {
    const int32_t *parent, *cu, *kv_len;
    int R, words;
    long long pos_base;
    uint32_t *mask;
    int32_t *pos;
    int *status;
};

__global__ void tree_kernel(const TreeArgs a) {
    extern __shared__ uint32_t shared[];
    wait_for_previous();
    launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x, wide = 32 * a.words;
    const int begin = __ldcg(a.cu + b), end = __ldcg(a.cu + b + 1), length = __ldcg(a.kv_len + b), n = end - begin;
    // counts that make no sense, also fewer tokens than new ones, or positions that 32 bits do not hold: nothing is read or
    // written by them
    if (begin < 0 || end < begin || end > a.R || length < n || (n && a.pos_base + length > 1ll << 31)) {
        if (tid == 0) report(a.status, CP_ERR_PAGE);
        return;
    }
    const long long first = a.pos_base + length - n;  // position of a token of depth 0
    if (n > wide) {
        // a prompt: its tokens follow one another
        for (int j = tid; j < n; j += blockDim.x) a.pos[begin + j] = static_cast<int32_t>(first + j);
        return;
    }
    // rows an odd number of words apart, so that neighbouring tokens' are on different banks
    const int stride = a.words | 1;
    uint32_t *bits = shared, *word = bits + wide * stride;  // [32 words][stride], [32 words]
    int *hangs = reinterpret_cast<int *>(word + wide), *depth = hangs + wide;
    const int lane = tid & 31, warp = tid >> 5, at = 32 * warp;
    int up = -1;
    if (tid < n) {
        up = __ldcg(a.parent + begin + tid);
        if (up < -1 || up >= tid) {
            report(a.status, CP_ERR_PAGE);
            up = -1;
        }
    }
    // the branch among these 32 tokens: its bits, its edges, its first token
    uint32_t own = 1u << lane;
    int top = up >= at ? up - at : lane, edges = up >= at;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        own |= __shfl_sync(0xffffffffu, own, top);
        edges += __shfl_sync(0xffffffffu, edges, top);  // (a first token's are none)
        top = __shfl_sync(0xffffffffu, top, top);
    }
    const int before = __shfl_sync(0xffffffffu, up, top);  // the earlier token that it hangs on, or -1
    word[tid] = own;
    hangs[tid] = before;
    depth[tid] = edges;
    for (int w = 0; w < a.words; ++w) bits[tid * stride + w] = 0;
    __syncthreads();
    if (tid < n) {
        // (each token's earlier ones are in an earlier word than it: the walk ends)
        int e = tid, sum = edges;
        for (;;) {
            bits[tid * stride + (e >> 5)] = word[e];
            e = hangs[e];
            if (e < 0) break;
            sum += 1 + depth[e];
        }
        a.pos[begin + tid] = static_cast<int32_t>(first + sum);
    }
    __syncthreads();
    uint32_t *to = a.mask + static_cast<long long>(begin) * a.words;
    if (a.words == 1) {
        if (tid < n) to[tid] = bits[tid];
        return;
    }
    for (int i = tid; i < n * a.words; i += blockDim.x) {
        const int j = i / a.words;
        to[i] = bits[j * stride + i - j * a.words];
    }
}

// ---------------------------------------------------------------- few sequences
template <int D>
cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&at)[2], int items, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(items * blocks));
    c.blockDim = dim3(kClThreads);
    c.dynamicSmemBytes = ClCfg<D>::kSmem;
    c.stream = stream;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(blocks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 2;
    return c;
}

// How many clusters of each size the GPU holds at once (all GPUs of a process are alike); 0 of all if it has none.
struct AtOnce {
    int clusters[kClMost + 1];
};
template <int D>
const AtOnce &clusters_at_once() {
    static AtOnce most{};
    static std::once_flag once;
    std::call_once(once, [] {
        const void *f = reinterpret_cast<const void *>(tree_cluster_kernel<D>);
        if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, ClCfg<D>::kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        for (int i = 2; i <= kClMost; ++i) {
            cudaLaunchAttribute at[2] = {};
            cudaLaunchConfig_t c = cluster_config<D>(at, 1, i, nullptr);
            c.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, f, &c) == cudaSuccess) most.clusters[i] = n;
            else cudaGetLastError();
        }
    });
    return most;
}

// Blocks of a cluster of tree_cluster.cuh, or 0 where it does not take the call: clusters are quick to begin and to
// end, the line of prefix_call.cuh shares the keys of ragged sequences evenly and reads a prefix once, and a block an
// item (tree_block.cuh) needs no join.  As many blocks as let all items run at once, two at least; not where the
// longest sequence that the table can hold would make a block's share more tiles of 128 keys than `tiles`.
// Clusters and line in us (16 tokens, pages of 32; 32 / 8 heads at D = 128, 16 / 4 at 64; all sequences of the figure,
// and up to it; tables as wide as the longest):
//   D = 128   1 of 4096   14.7 18.7               9 of 4096   33.7 48.1, 27.5 36.4
//             1 of 16000  23.0 28.0               9 of 8000   55.4 72.1, 42.8 45.4
//             4 of 8000   31.3 39.8, 27.8 34.6    7 of 6000   39.0 51.9, 33.8 37.2
//             4 of 16000  51.3 60.6, 44.9 47.3 (31 tiles)
//   D = 64    8 of 8000   20.4 28.7, 19.2 23.2    16 of 4000  20.6 29.7, 19.4 23.6
//             8 of 16000  32.3 39.9, 31.5 31.3    16 of 8000  32.9 40.6, 31.0 27.1 (31 tiles)
//             4 of 24000  31.2 34.4, 30.2 26.6    4 of 32000 (beyond the limit) 38.6 39.6, 37.9 30.5
// Near the limit ragged sequences would be better off by the line, by up to 15%, and others worse by as much or more:
// which it is the host does not see.  Up to 16 rows the line has its narrow tiles and the limit is lower: four tokens of
// up to 4000 keys of two sequences 14.2 and 19.0, of four 16.8 and 20.7, at D = 64 of 16 18.2 and 17.9 (all of 4000
// 19.0, 23.0).  A prefix is read once for each sequence, and the limit is lower at D = 128: two of 500 behind 8000 22.0
// and 24.8, four of 4000 behind 4000 26.6 and 37.2, at D = 64 behind 16000 27.1 and 30.0.
// Up to 640 keys a block an item is quicker, as it needs no meeting of blocks.  Blocks and clusters: one sequence of 500
// keys 8.7 and 12.0, of 640 9.8 and 11.5, of 800 11.6 and 11.2, of 1300 16.2 and 11.2; nine of 640 10.8 and 14.7, of
// 800 12.7 and 15.2, of 1300 17.6 and 17.7; at D = 64 two of 500 8.0 and 9.2, of 640 8.9 and 8.7, of 1300 14.9 and 8.5.
template <int D>
int cluster_blocks(const ClusterArgs &c, int64_t rows) {
    const PrefixArgs &a = c.p;
    const long long items = static_cast<long long>(a.B) * c.tiles * a.Nkv;
    const AtOnce &most = clusters_at_once<D>();
    const long long keys = a.P + (static_cast<long long>(a.own.max_pages) << a.own.shift);
    if (keys <= 640) return 0;
    const int tiles = a.P > 0 ? (D == 64 ? 32 : 16) : rows <= kTcRows ? 16 : 32;
    for (int i = kClMost; i >= 2; --i)
        if (items <= most.clusters[i]) return keys <= 128LL * i * tiles ? i : 0;
    return 0;
}

// Whether a block an item (tree_block.cuh), two on an SM, takes the call, rather than the line.  A tile of 64 keys takes
// a block 0.75 us, so the longest sequence that the table holds takes 0.75 k, k its tiles, and all items together, half
// as long on average, items k / 2 x 0.75 / 304 at best (measured 1.3 times that: half of the time memory is what they
// wait for).  The line reads the keys once for 256 rows, a prefix once for all sequences, whatever the lengths, at
// 5 TB/s (6.5 by its narrow tiles), and takes 20 us (13) and 0.05 us (0.03) an item of its own besides.
// Block and line in us (16 tokens, 32 / 8 heads of 128, pages of 16, own keys up to the figure, tables as wide):
//   16 of 4096   47  55    64 of 8000    153 192    300 of 500    83 199    27 tokens, 100 of 1000  77 117
//   32 of 8000  106 122    64 all of it  307 369    300 of 1000  115 236    60 tokens, 60 of 60     39  76
//   1 token, 20 of 500 11 17, 64 of 4000 84 93; prompts of 1000: one 27 46, four 84 111, eight 159 185; 500 tokens of
//   eight prompts of 1000 108 123, 200 of 16 99 118; behind a prefix of 500 64 of 1000 43 110, 200 of 300 82 208, behind
//   one of 2000 64 of 1000 79 126; at D = 64 (16 / 4 heads) 64 of 4000 46 64, 200 of 4000 93 126.
// and where it takes the line: 16 of 8000 83 64 (all of it 95 113), 1 token of 20 of 4000 45 37, 60 tokens, 120 of
//   2000 243 235.
// The estimates know neither the rows' own work nor which tokens are a prompt's, and are wrong in places: the block is
// taken for trees of 500 tokens of eight sequences of 1000 keys (152 138) and for 500 tokens of four prompts of 2000
// (108 94), the line for 200 of 300 behind 2000 (191 264) and 40 of 4000 at D = 64 (42 46).
// Beyond 8192 keys the line is taken as one long sequence among short ones would leave a block alone with it (64 of
// 16000 are quicker by blocks, 324 372).
constexpr int kBlMost = 8192;
template <int D>
bool items_pay(const ClusterArgs &c, int64_t rows) {
    const PrefixArgs &a = c.p;
    const double own = static_cast<double>(static_cast<long long>(a.own.max_pages) << a.own.shift), tile = 0.75;
    const double items = static_cast<double>(a.B) * c.tiles * a.Nkv, shared = static_cast<double>(a.B) * a.Nkv * ((rows + 255) / 256);
    if (a.P + own > kBlMost || items > 1e9) return false;  // (a launch has fewer than 2^31 blocks)
    const double longest = (a.P + own) / kBlKeys * tile, all = items * (a.P + own / 2) / kBlKeys * 1.3 * tile / (2 * sm_count());
    const double bytes = shared * own / 2 * 4 * D;
    const double line = rows <= kTcRows ? 13 + bytes / 6.5e6 + 0.03 * shared : 20 + bytes / 5e6 + 0.05 * shared;
    return longest <= line && all <= line;
}

template <int D>
cp_status launch_clusters(const ClusterArgs &a, int blocks, cudaStream_t stream) {
    cudaLaunchAttribute at[2] = {};
    const cudaLaunchConfig_t c = cluster_config<D>(at, a.p.B * a.tiles * a.p.Nkv, blocks, stream);
    const cudaError_t e = cudaLaunchKernelEx(&c, tree_cluster_kernel<D>, a);
    if (e != cudaSuccess) cudaGetLastError();
    return cuda_status(e);
}

// A block an item, two on an SM; the longest sequences' first where they do not all run at once and the order is
// worth what finding it costs each block, 6 ns a sequence, against a quarter of the longest item's time: 64
// sequences of up to 4096 keys 86 us and 101 without, 32 tokens of 32 of 2000 40 and 50; 150 of 1000 68 and 60.
template <int D>
cp_status launch_items(const ClusterArgs &a, cudaStream_t stream) {
    static cudaError_t err = cudaSuccess;
    static std::once_flag once;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(tree_block_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, BlCfg<D>::kSmem);
    });
    if (err != cudaSuccess) return cuda_status(err);
    const int64_t items = static_cast<int64_t>(a.p.B) * a.tiles * a.p.Nkv, at_once = 2LL * sm_count();
    const double keys = static_cast<double>(a.p.P + (static_cast<long long>(a.p.own.max_pages) << a.p.own.shift));
    const bool order = a.p.B <= kBlThreads && items > at_once && 0.006 * a.p.B * items / at_once < 0.75 / 4 * keys / kBlKeys;
    const BlockArgs x{a, order};
    return launch(tree_block_kernel<D>, dim3(static_cast<unsigned>(items)), kBlThreads, BlCfg<D>::kSmem, stream, x);
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" cp_status cp_tree_plan(const int32_t *parent, const int32_t *cu_new, const int32_t *kv_len, int64_t B,
                                  int64_t R, int64_t words, int64_t pos_base, int32_t *mask, int32_t *pos,
                                  cudaStream_t stream) {
    if (!parent || !cu_new || !kv_len || !mask || !pos) return CP_ERR_NULL;
    if (B < 1 || B > kMaxSequences || R < 1 || R > INT32_MAX / 2 || words < 1 || words > kMaxWords) return CP_ERR_SHAPE;
    if (pos_base < INT32_MIN || pos_base > INT32_MAX) return CP_ERR_ARGUMENT;
    auto odd = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (odd(parent) || odd(cu_new) || odd(kv_len) || odd(mask) || odd(pos)) return CP_ERR_ALIGNMENT;
    const struct {
        const void *p;
        int64_t n;
    } in[] = {{parent, R}, {cu_new, B + 1}, {kv_len, B}, {mask, R * words}};
    // mask apart from the lists, pos from all of them
    auto meet = [](const void *x, int64_t nx, const void *y, int64_t ny) {
        const char *p = static_cast<const char *>(x), *q = static_cast<const char *>(y);
        return p < q + 4 * ny && q < p + 4 * nx;
    };
    for (int i = 0; i < 4; ++i)
        if ((i < 3 && meet(mask, R * words, in[i].p, in[i].n)) || meet(pos, R, in[i].p, in[i].n)) return CP_ERR_ARGUMENT;
    TreeArgs a{parent, cu_new, kv_len, static_cast<int>(R), static_cast<int>(words), pos_base,
               reinterpret_cast<uint32_t *>(mask), pos, nullptr};
    const cp_status st = prefix_status_word(&a.status);
    if (st != CP_OK) return st;
    const int wide = 32 * a.words;
    return launch(tree_kernel, dim3(static_cast<unsigned>(B)), wide, static_cast<size_t>(wide) * (3 + (a.words | 1)) * 4,
                  stream, a);
}

extern "C" cp_status cp_tree_attn_workspace_size(int64_t R, int64_t B, int64_t max_new, int64_t words,
                                                 int64_t prefix_len, int64_t N, int64_t Nkv, int64_t D,
                                                 int64_t page_size, int64_t max_pages, size_t *bytes) {
    if (!bytes) return CP_ERR_NULL;
    if (words < 1 || words > kMaxWords) return CP_ERR_SHAPE;
    const cp_status st = check_sizes(R, B, max_new, prefix_len, N, Nkv, D, page_size, max_pages);
    if (st != CP_OK) return st;
    *bytes = shape_of(R, B, max_new, prefix_len, N, Nkv, D).bytes;
    return CP_OK;
}

namespace {
// cp_tree_attn_fwd, with the limit of its waits; stalled: its loads wait for a word that nothing sets.
cp_status tree_call(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages, int64_t page_size,
                    const int32_t *prefix_pages, int64_t prefix_len, const int32_t *table, int64_t B, int64_t max_pages,
                    const int32_t *cu_new, const int32_t *kv_len, const int32_t *mask, int64_t words, int64_t max_new,
                    int64_t R, int64_t N, int64_t Nkv, int64_t D, float scale, void *o, cp_dtype o_dtype, float *lse,
                    void *workspace, size_t ws_bytes, uint64_t timeout_ns, bool stalled, cudaStream_t stream) {
    if (words < 1 || words > kMaxWords) return CP_ERR_SHAPE;
    Call c;
    const cp_status st = check_call<true>(c, mask, words, q, k_cache, v_cache, n_pages, page_size, prefix_pages,
                                          prefix_len, table, B, max_pages, cu_new, kv_len, max_new, R, N, Nkv, D,
                                          scale, o, o_dtype, lse, workspace, ws_bytes, timeout_ns, stalled);
    if (st != CP_OK) return st;
    const int64_t rows = max_new * c.a.G;  // of an item, about
    auto form = [&](int tile) { return ClusterArgs{c.a, static_cast<int>((rows + tile - 1) / tile), o, o_dtype == CP_BF16, lse}; };
    const ClusterArgs few = form(128), many = form(kBlRows);
    const int blocks = D == 128 ? cluster_blocks<128>(few, rows) : cluster_blocks<64>(few, rows);
    if (blocks) return D == 128 ? launch_clusters<128>(few, blocks, stream) : launch_clusters<64>(few, blocks, stream);
    if (D == 128 ? items_pay<128>(many, rows) : items_pay<64>(many, rows))
        return D == 128 ? launch_items<128>(many, stream) : launch_items<64>(many, stream);
    return launch_line<true>(c, stream);
}
}  // namespace

extern "C" cp_status cp_tree_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                      int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                      const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                      const int32_t *kv_len, const int32_t *mask, int64_t words, int64_t max_new,
                                      int64_t R, int64_t N, int64_t Nkv, int64_t D, float scale, void *o,
                                      cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                                      cudaStream_t stream) {
    return tree_call(q, k_cache, v_cache, n_pages, page_size, prefix_pages, prefix_len, table, B, max_pages, cu_new,
                     kv_len, mask, words, max_new, R, N, Nkv, D, scale, o, o_dtype, lse, workspace, ws_bytes,
                     2000000000ull, false, stream);
}

extern "C" cp_status cp_selftest_stalled_tree_attn(const void *q, const void *k_cache, const void *v_cache,
                                                   int64_t n_pages, int64_t page_size, const int32_t *prefix_pages,
                                                   int64_t prefix_len, const int32_t *table, int64_t B,
                                                   int64_t max_pages, const int32_t *cu_new, const int32_t *kv_len,
                                                   const int32_t *mask, int64_t words, int64_t max_new, int64_t R,
                                                   int64_t N, int64_t Nkv, int64_t D, float scale, void *o,
                                                   cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                                                   uint64_t timeout_ns, cudaStream_t stream) {
    if (timeout_ns < 1000000ull || timeout_ns > 2000000000ull) return CP_ERR_ARGUMENT;
    return tree_call(q, k_cache, v_cache, n_pages, page_size, prefix_pages, prefix_len, table, B, max_pages, cu_new,
                     kv_len, mask, words, max_new, R, N, Nkv, D, scale, o, o_dtype, lse, workspace, ws_bytes,
                     timeout_ns, true, stream);
}
