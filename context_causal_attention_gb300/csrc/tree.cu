// tree.cu -- trees of drafted tokens: their ancestors and positions (cp_tree_plan), and attention over the paged cache by
// them (cp_tree_attn_fwd: the kernels of prefix_call.cuh and prefix_tc.cuh, with a row's mask in the place of its
// index wherever a key tile reaches into the step's new tokens).
//
// Ancestors.  mask_j = {j} + mask_parent(j).  A warp holds 32 tokens in a row, a token a lane, and follows the
// parents among them by doubling (five rounds of shuffles, whatever the tree's shape); what is left of a token's
// branch begins at one earlier token, whose row is taken over whole.  So the warps of a block, which works on one
// sequence, come one after the other, and each row is read and written once: 16 short steps for 512 tokens.  Following
// all parents by doubling through shared memory instead took 15.9 us for 300 trees of up to 500 tokens, this 9.4.
// What bounds it is the latency of the launch and of two loads that hang on one another (counts, parents).
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_internal.h"
#include "prefix_call.cuh"

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
    extern __shared__ __align__(16) uint32_t shared[];
    wait_for_previous();
    launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x, wide = 32 * a.words;
    const int begin = __ldcg(a.cu + b), n = __ldcg(a.cu + b + 1) - begin;
    // counts that make no sense: nothing is read or written by them
    if (begin < 0 || n < 0 || n > a.R - begin) {
        if (tid == 0) report(a.status, CP_ERR_PAGE);
        return;
    }
    const long long first = a.pos_base + __ldcg(a.kv_len + b) - n;  // position of a token of depth 0
    if (n > wide) {
        // a prompt: its tokens follow one another
        for (int j = tid; j < n; j += blockDim.x) a.pos[begin + j] = static_cast<int32_t>(first + j);
        return;
    }
    uint32_t *bits = shared;  // [32 words][words]
    int *depth = reinterpret_cast<int *>(bits + wide * a.words);
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
    for (int i = tid; i < wide * a.words; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    const int warps = (n + 31) >> 5;
    for (int k = 0; k < warps; ++k) {
        if (k == warp) {
            if (before >= 0) edges += 1 + depth[before];
            depth[tid] = edges;
            bits[tid * a.words + k] = own;
            // the rows of the earlier tokens, eight at a time, four lanes each
            for (int w0 = 0; w0 < k; w0 += 4) {
                const int w = w0 + (lane & 3);
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = __shfl_sync(0xffffffffu, before, 8 * i + (lane >> 2));
                    v[i] = w < k && from >= 0 ? bits[from * a.words + w] : 0u;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (w < k) bits[(at + 8 * i + (lane >> 2)) * a.words + w] = v[i];
            }
        }
        __syncthreads();
    }
    if (tid < n) a.pos[begin + tid] = static_cast<int32_t>(first + edges);
    uint32_t *to = a.mask + static_cast<long long>(begin) * a.words;
    const int all = n * a.words, fours = (reinterpret_cast<uintptr_t>(to) & 15u) == 0 ? all >> 2 : 0;
    for (int i = tid; i < fours; i += blockDim.x) reinterpret_cast<uint4 *>(to)[i] = reinterpret_cast<uint4 *>(bits)[i];
    for (int i = 4 * fours + tid; i < all; i += blockDim.x) to[i] = bits[i];
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
    return launch(tree_kernel, dim3(static_cast<unsigned>(B)), wide, static_cast<size_t>(wide) * (1 + a.words) * 4,
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

extern "C" cp_status cp_tree_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                      int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                      const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                      const int32_t *kv_len, const int32_t *mask, int64_t words, int64_t max_new,
                                      int64_t R, int64_t N, int64_t Nkv, int64_t D, float scale, void *o,
                                      cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                                      cudaStream_t stream) {
    if (words < 1 || words > kMaxWords) return CP_ERR_SHAPE;
    return prefix_call<true>(mask, words, q, k_cache, v_cache, n_pages, page_size, prefix_pages, prefix_len, table, B,
                             max_pages, cu_new, kv_len, max_new, R, N, Nkv, D, scale, o, o_dtype, lse, workspace,
                             ws_bytes, 2000000000ull, false, stream);
}
