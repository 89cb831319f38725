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
// end, the line of prefix_call.cuh shares the keys of ragged sequences evenly and reads a prefix once, and a block an item
// (tree_block.cuh) needs no join.  As many blocks as let all items run at once, two at least; not where the longest
// sequence that the table can hold would make a block's share too many tiles of 128 keys.  Clusters and line, us
// (16 tokens, 32 / 8 heads of 128, pages of 32, own keys up to the figure): one sequence of 4096 13.6 and 19.3, of 16000
// 20.6 and 24.3; four of 4096 18.8 and 30, of 8000 31 and 40, ragged 26 and 32, of 16000 (31 tiles) 51 and 62, ragged 45 and 49;
// seven of 6000 (24) 38 and 52, ragged 32 and 29; nine of 4096 (16) 35 and 50, ragged 27 and 34.  At D = 64 (16 / 4 heads) 16 of
// 4000 ragged 19 and 24, of 8000 (31) 31 both, four of 32000 (31) 38 and 32.  Up to 16 rows the line has its narrow tiles:
// four tokens of two sequences of 4000 keys, ragged, 13.1 and 15.9, of four (8) 14.8 and 17.3; at D = 64 of 16 (16) 17.9 and
// 18.6.  A prefix is read once for each sequence: two of 500 behind 8000 20 and 25, four of 4000 behind 4000 (16) 24 and 32,
// at D = 64 behind 16000 (39) 27 and 28.
// Up to 640 keys a block an item is quicker, as it needs no meeting of blocks: one sequence of 16 tokens behind 500 keys
// 9.9 us and 11.5, behind 800 12.8 and 11.4; nine 10.3 and 13.2, 13.2 and 13.8; at D = 64 two of 500 9.1 and 8.7.
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

// Whether a block an item (tree_block.cuh), two on an SM, takes the call, rather than the line.  A tile of 64
// keys takes a block 0.75 us, so the longest sequence that the table holds takes 0.75 k, k its tiles, and all
// items together, half as long on average, items k / 2 x 0.75 / 304 at best (measured 1.3 times that: half of the time
// memory is what they wait for).  The line reads the keys once for 256 rows, a prefix once for all sequences,
// whatever the lengths, at 5 TB/s (6.5 by its narrow tiles), and takes 20 us (13) and 0.05 us (0.03) an item of its own
// besides.  Block and line, us (16 tokens, 32 / 8 heads of 128, pages of 16, own keys up to the figure, ragged): 16 sequences of 4096
// 47 and 50, of 8000 87 and 71 (not ragged 94 and 113), 32 of 8000 109 and 115, 64 of 4096 85 and 126, of 8000 159 and 200; 300 of
// 500 78 and 175, of 1000 117 and 220; 27 tokens of 100 of 1000 58 and 97, 60 tokens of 60 59 and 81, 120 of 60 of 2000
// 163 both, 500 of 8 of 1000 not ragged 152 and 138; a prompt of 1000 tokens 30 and 47, four 92 and 117.  Single tokens of 20 sequences of 500 11.2 and 16.1, of 4000 47 and 38, 64 of 4000 87 and 102.  Behind a prefix
// of 500 64 of 1000 44 and 103, 200 of 300 81 and 162, of 2000 79 and 116, 184 and 192.  At D = 64 (16 / 4 heads) 40 of
// 4000 40 and 36, 64 47 and 58, 200 95 and 118.
// Beyond 8192 keys the line gains by itself (64 of 16000 310 and 349), and one long sequence among short ones would leave
// a block alone with it.
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
