// prefix.cu -- cp_prefix_attn_fwd (its kernels and their reasons: prefix_call.cuh, prefix_tc.cuh), and the
// status word that the tree attention shares with it.
#include <cuda_runtime.h>

#include "cp_internal.h"
#include "prefix_call.cuh"

namespace cpattn {
namespace {
__device__ int g_prefix_status = 0;
__device__ int g_prefix_hold = 0;  // never set
}  // namespace

// Device addresses in the current context (looked up at each call: a new context has others).
cp_status prefix_status_word(int **p) {
    return cuda_status(cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_prefix_status));
}
cp_status prefix_hold_word(int **p) {
    return cuda_status(cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_prefix_hold));
}

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
    Call c;
    const cp_status st = check_call<false>(c, nullptr, 0, q, k_cache, v_cache, n_pages, page_size, prefix_pages,
                                           prefix_len, table, B, max_pages, cu_new, kv_len, max_new, R, N, Nkv, D,
                                           scale, o, o_dtype, lse, workspace, ws_bytes, 2000000000ull, false);
    return st != CP_OK ? st : launch_line<false>(c, stream);
}

extern "C" cp_status cp_selftest_stalled_prefix_attn(
    const void *q, const void *k_cache, const void *v_cache, int64_t n_pages, int64_t page_size,
    const int32_t *prefix_pages, int64_t prefix_len, const int32_t *table, int64_t B, int64_t max_pages,
    const int32_t *cu_new, const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv, int64_t D,
    float scale, void *o, cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes, uint64_t timeout_ns,
    cudaStream_t stream) {
    if (timeout_ns < 1000000ull || timeout_ns > 2000000000ull) return CP_ERR_ARGUMENT;
    Call c;
    const cp_status st = check_call<false>(c, nullptr, 0, q, k_cache, v_cache, n_pages, page_size, prefix_pages,
                                           prefix_len, table, B, max_pages, cu_new, kv_len, max_new, R, N, Nkv, D,
                                           scale, o, o_dtype, lse, workspace, ws_bytes, timeout_ns, true);
    return st != CP_OK ? st : launch_line<false>(c, stream);
}
