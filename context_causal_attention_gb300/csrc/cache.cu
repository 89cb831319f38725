// cache.cu -- appending the keys and values of new tokens to a paged cache,
// with the keys' norm and rotation (and the queries') on the way.
//
// Token j of the n_b new tokens of sequence b gets own index i = kv_len[b] -
// n_b + j, position pos_base + i, and slot i % page_size of page
// table[b][i / page_size].  K: norm, rotation, bf16, into that slot; V: bf16,
// into the same slot of the other cache; Q: norm, rotation, bf16, in place
// order.  Norm and rotation as in rope.cu.  cp_cache_append_at takes slots and positions as
// lists instead (drafted tokens of a tree: siblings share a position): 16 of them for each of 64 sequences, 32 / 8
// heads of 128, normed and rotated, take 6.5 us in a graph, 3.7 at the copy's rate; slot, row and phase follow one another.
//
// Memory-bound where there are many tokens and latency-bound at one token for
// each sequence, so one launch does all three tensors: a warp takes a token
// (or a few of its heads when there are few tokens), finds its sequence with a
// 32-way search over the cumulative counts (one load per lane and level, two
// levels up to 1024 sequences), works out the sines once and streams the rows.
// Every index that comes from device memory is checked before it is used: a
// bad one skips the token and sets the device status word.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cp_internal.h"
#include "cp_paged.cuh"
#include "cp_rope.cuh"

namespace cpattn {
namespace {

__device__ int g_cache_status = 0;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct AppendArgs {
    const void *x[3];  // q, k, v rows
    long long xs[3];   // elements between tokens
    int heads[3];
    __nv_bfloat16 *q_out, *cache[2];
    const void *w[2];
    int w_bf16, norm[2];
    float eps;
    RopeDev rope;
    PageTable pt;
    const int32_t *cu, *kv_len;
    const int32_t *slots, *pos;  // kAt: of each row
    long long tokens, pos_base;
    int group, chunks, hpu;
};

// Sequence b's new token `tok` (the b-th begins at row `begin` and has `count`): its own index, and its slot or -1.
__device__ __forceinline__ long long slot_of(const AppendArgs &a, int b, int tok, int begin, int count, long long *idx) {
    *idx = static_cast<long long>(__ldg(a.kv_len + b)) - count + (tok - begin);
    const long long slot = a.pt.slot(b, *idx);
    if (slot < 0) atomicExch(&g_cache_status, static_cast<int>(CP_ERR_PAGE));
    return slot;
}

// Row tok's slot as its list gives it, or -1 (none, or out of range and reported), and its position.
__device__ __forceinline__ long long slot_in_list(const AppendArgs &a, int tok, long long *pos) {
    *pos = __ldcg(a.pos + tok);
    const long long slot = __ldcg(a.slots + tok), all = static_cast<long long>(a.pt.n_pages) << a.pt.shift;
    if (slot >= -1 && slot < all) return slot;
    atomicExch(&g_cache_status, static_cast<int>(CP_ERR_PAGE));
    return -1;
}

// A unit is `group` tokens in a row with all their heads, or (group 1) `hpu` heads
// of one token.  The rows of q, k and v of a token make one list, so that four rows
// of a lane are in flight whichever tensor they belong to.
template <typename T, int D, int kOrder, bool kAt>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const AppendArgs a) {
    using Map = LaneMap<D, kOrder>;
    constexpr int kU = sizeof(T) == 2 ? 4 : 2;
    const int lane = threadIdx.x & 31, sub = lane / Map::L;
    const Map map(lane, a.rope.half);
    unsigned long long f[Map::kAng];
    if (kAt) {
        // its blocks may have started under the kernel that makes the lists or the rows
        wait_for_previous();
        launch_dependents();
    }
    load_freqs(a.rope, lane, f);
    const int nq = a.heads[0], nk = a.heads[1], all = nq + 2 * nk;
    const long long units = (a.tokens + a.group - 1) / a.group * a.chunks;
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += step) {
        const int tok0 = static_cast<int>(a.chunks == 1 ? u * a.group : u / a.chunks);
        const int first = a.chunks == 1 ? 0 : static_cast<int>(u - static_cast<long long>(tok0) * a.chunks) * a.hpu;
        const int last = min(first + a.hpu, all);
        // lane i looks up token tok0 + i
        long long idx = 0, slot = -1;
        if (kAt) {
            if (lane < a.group && tok0 + lane < a.tokens) slot = slot_in_list(a, tok0 + lane, &idx);
        } else if (a.group == 1) {
            int begin, count;
            const int b = find_sequence(a.cu, a.pt.B, tok0, lane, &begin, &count);
            if (b < 0) continue;  // a row behind the last sequence
            slot = slot_of(a, b, tok0, begin, count, &idx);
        } else if (lane < a.group && tok0 + lane < a.tokens) {
            const int tok = tok0 + lane;
            int lo = 0, hi = a.pt.B - 1;  // the last sequence that begins at or before tok
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(a.cu + mid) <= tok) lo = mid; else hi = mid - 1;
            }
            const int begin = __ldg(a.cu + lo), end = __ldg(a.cu + lo + 1);
            if (tok >= begin && tok < end) slot = slot_of(a, lo, tok, begin, end - begin, &idx);
        }
        for (int i = 0; i < a.group; ++i) {
            const long long to = __shfl_sync(0xffffffffu, slot, i), at = __shfl_sync(0xffffffffu, idx, i);
            const int tok = tok0 + i;
            if (to < 0) continue;  // behind the last sequence, or reported
            float c[8], s[8];
            if (a.rope.half) token_angles<D>(f, a.pos_base + at, a.rope.amp, lane, c, s);
            for (int hb = first; hb < last; hb += kU * Map::kRows) {
                Vec8<T> v0[kU], v1[kU];
#pragma unroll
                for (int k = 0; k < kU; ++k) {
                    const int h = hb + k * Map::kRows + sub;
                    if (h < last) {
                        const int t = h < nq ? 0 : (h < nq + nk ? 1 : 2);
                        const T *x = static_cast<const T *>(a.x[t]) + tok * a.xs[t] + (h - (t == 0 ? 0 : nq + (t - 1) * nk)) * D;
                        v0[k].load(x + map.c0);
                        v1[k].load(x + map.c1);
                    }
                }
#pragma unroll
                for (int k = 0; k < kU; ++k) {
                    if (hb + k * Map::kRows >= last) break;  // uniform over the warp
                    const int h = hb + k * Map::kRows + sub;
                    const int t = h < nq ? 0 : (h < nq + nk ? 1 : 2);
                    float r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0.f;
                    if (h < last) {
                        v0[k].to(r);
                        v1[k].to(r + 8);
                    }
                    const bool norm = t < 2 && a.norm[t];
                    if (__any_sync(0xffffffffu, norm)) {
                        float q = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) q = fmaf(r[e], r[e], q);
                        const float rstd = rsqrtf(row_sum<Map::L>(q) * (1.f / D) + a.eps);
                        if (norm) {
                            float w[16];
                            load_weights(a.w[t], a.w_bf16, map, w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) r[e] = r[e] * rstd * w[e];
                        }
                    }
                    if (a.rope.half) turn_pairs<kOrder, false>(r, c, s, t < 2 ? map.mask : 0u);
                    if (h < last) {
                        __nv_bfloat16 *y = t == 0 ? a.q_out + (static_cast<long long>(tok) * nq + h) * D
                                                  : a.cache[t - 1] + (to * nk + h - nq - (t - 1) * nk) * D;
                        store8(y + map.c0, r);
                        store8(y + map.c1, r + 8);
                    }
                }
            }
        }
    }
}

template <typename T, int D, int kOrder, bool kAt>
cp_status launch_append(AppendArgs &a, cudaStream_t stream) {
    constexpr int rows = LaneMap<D, kOrder>::kRows;
    const int heads = a.heads[0] + a.heads[1] + a.heads[2], most = (heads + rows - 1) / rows;
    // As many tokens to a unit (their lookups go side by side) as leave every SM 16
    // warps, up to 32: 8 prompts' 23377 tokens of 8 KV heads take 37.0 us so (ten to a
    // unit), 40.5 with one.  Where there are fewer tokens than that, fewer heads
    // of one, as in rope.cu: a token each of 64 sequences, 32 + 8 + 8 heads, 3.7 us in a
    // graph in twelve units, 8.7 in one; 1024 tokens 7.3 in two, 9.7 in three.
    const long long warps = static_cast<long long>(sm_count()) * 16;
    const long long group = (a.tokens + warps - 1) / warps;
    a.group = static_cast<int>(group < 32 ? group : 32);
    long long chunks = warps / a.tokens;
    chunks = chunks < 1 ? 1 : (chunks > most ? most : chunks);
    a.hpu = static_cast<int>((most + chunks - 1) / chunks) * rows;
    a.chunks = (heads + a.hpu - 1) / a.hpu;
    const long long blocks = ((a.tokens + a.group - 1) / a.group * a.chunks + kWarps - 1) / kWarps;
    const long long cap = static_cast<long long>(sm_count()) * 4;
    const unsigned grid = static_cast<unsigned>(blocks < cap ? blocks : cap);
    if (kAt) return launch(append_kernel<T, D, kOrder, kAt>, dim3(grid), kThreads, 0, stream, a);
    append_kernel<T, D, kOrder, kAt><<<grid, kThreads, 0, stream>>>(a);
    return last_launch_status();
}

bool misaligned(const void *p) { return p && !aligned16(p); }

}  // namespace

cp_status read_cache_device_status(int *code, bool clear) {
    if (cudaMemcpyFromSymbol(code, g_cache_status, sizeof(int)) != cudaSuccess) return CP_ERR_CUDA;
    if (clear) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_cache_status, &zero, sizeof(int)) != cudaSuccess) return CP_ERR_CUDA;
    }
    return CP_OK;
}

cp_status cache_status_word(int **p) {
    return cuda_status(cudaGetSymbolAddress(reinterpret_cast<void **>(p), g_cache_status));
}

cp_status check_pages(int64_t n_pages, int64_t page_size, int64_t B, int64_t max_pages, int64_t Nkv, int64_t D) {
    if (n_pages < 1 || n_pages > INT32_MAX || B < 1 || B > kMaxSequences || max_pages < 1 || max_pages > INT32_MAX ||
        Nkv < 1 || Nkv > 65535)
        return CP_ERR_SHAPE;
    if (D != 64 && D != 128) return CP_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return CP_ERR_UNSUPPORTED;
    if (n_pages * page_size > kMaxKeys || max_pages * page_size > kMaxKeys) return CP_ERR_SHAPE;
    return CP_OK;
}

}  // namespace cpattn

using namespace cpattn;

namespace {
// cp_cache_append, or with kAt cp_cache_append_at (slots and pos in the place of the lists that the slots follow from).
template <bool kAt>
cp_status append_call(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      cp_dtype dtype, int64_t R, int64_t N, int64_t Nkv, int64_t D, const void *wq, const void *wk,
                      cp_dtype w_dtype, float eps, const cp_rope *rope, int64_t pos_base, void *k_cache, void *v_cache,
                      int64_t n_pages, int64_t page_size, const int32_t *table, int64_t B, int64_t max_pages,
                      const int32_t *cu_new, const int32_t *kv_len, const int32_t *slots, const int32_t *pos, void *q_out,
                      cudaStream_t stream) {
    if (!k || !v || !k_cache || !v_cache || (N > 0 && (!q || !q_out)) ||
        (kAt ? !slots || !pos : !table || !cu_new || !kv_len))
        return CP_ERR_NULL;
    if (R < 1 || R > INT32_MAX / 2 || N < 0 || N > 65535) return CP_ERR_SHAPE;
    cp_status st = check_pages(n_pages, page_size, B, max_pages, Nkv, D);
    if (st != CP_OK) return st;
    const size_t es = dtype_size(dtype);
    if (!es || !dtype_size(w_dtype)) return CP_ERR_DTYPE;
    if ((st = check_rope(rope, D)) != CP_OK) return st;
    if ((N && q_stride < N * D) || k_stride < Nkv * D || v_stride < Nkv * D || q_stride > INT32_MAX ||
        k_stride > INT32_MAX || v_stride > INT32_MAX)
        return CP_ERR_SHAPE;
    if ((wq || wk) && !(std::isfinite(eps) && eps >= 0.f)) return CP_ERR_ARGUMENT;
    if (pos_base < INT32_MIN || pos_base > INT32_MAX) return CP_ERR_ARGUMENT;
    if ((N && q_stride * es % 16) || k_stride * es % 16 || v_stride * es % 16 || misaligned(q) || misaligned(k) ||
        misaligned(v) || misaligned(k_cache) || misaligned(v_cache) || misaligned(q_out) || misaligned(wq) ||
        misaligned(wk) || (reinterpret_cast<uintptr_t>(table) & 3u) || (reinterpret_cast<uintptr_t>(cu_new) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_len) & 3u) || (reinterpret_cast<uintptr_t>(slots) & 3u) ||
        (reinterpret_cast<uintptr_t>(pos) & 3u))
        return CP_ERR_ALIGNMENT;
    const char *kc = static_cast<const char *>(k_cache), *vc = static_cast<const char *>(v_cache);
    const int64_t cache = n_pages * page_size * Nkv * D * 2;
    if (kc < vc + cache && vc < kc + cache) return CP_ERR_ARGUMENT;
    // q_out: dense rows; in place only where the query rows are dense bf16 themselves
    if (N) {
        const char *o0 = static_cast<const char *>(q_out), *o1 = o0 + R * N * D * 2;
        auto meets = [&](const void *p, int64_t stride, int64_t heads) {
            const char *p0 = static_cast<const char *>(p), *p1 = p0 + ((R - 1) * stride + heads * D) * es;
            return o0 < p1 && p0 < o1;
        };
        const bool in_place = q == q_out && dtype == CP_BF16 && q_stride == N * D;
        if ((!in_place && meets(q, q_stride, N)) || meets(k, k_stride, Nkv) || meets(v, v_stride, Nkv))
            return CP_ERR_ARGUMENT;
        if ((o0 < kc + cache && kc < o1) || (o0 < vc + cache && vc < o1)) return CP_ERR_ARGUMENT;
    }
    AppendArgs a{};
    a.x[0] = q, a.x[1] = k, a.x[2] = v;
    a.xs[0] = q_stride, a.xs[1] = k_stride, a.xs[2] = v_stride;
    a.heads[0] = static_cast<int>(N), a.heads[1] = a.heads[2] = static_cast<int>(Nkv);
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.cache[0] = static_cast<__nv_bfloat16 *>(k_cache);
    a.cache[1] = static_cast<__nv_bfloat16 *>(v_cache);
    a.w[0] = wq, a.w[1] = wk;
    a.norm[0] = wq != nullptr, a.norm[1] = wk != nullptr;
    a.w_bf16 = w_dtype == CP_BF16;
    a.eps = eps;
    if (rope) {
        a.rope.freqs = reinterpret_cast<const unsigned long long *>(rope->freqs);
        a.rope.half = static_cast<int>(rope->rot_dim / 2);
        a.rope.amp = rope->amplitude;
    }
    a.pt.table = table;
    a.pt.B = static_cast<int>(B);
    a.pt.max_pages = static_cast<int>(max_pages);
    a.pt.n_pages = static_cast<int>(n_pages);
    a.pt.shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    a.cu = cu_new;
    a.kv_len = kv_len;
    a.slots = slots;
    a.pos = pos;
    a.tokens = R;
    a.pos_base = pos_base;
    const bool inter = rope && rope->order == CP_ROPE_INTERLEAVED;
    if (dtype == CP_BF16) {
        using T = __nv_bfloat16;
        if (D == 128) return inter ? launch_append<T, 128, 1, kAt>(a, stream) : launch_append<T, 128, 0, kAt>(a, stream);
        return inter ? launch_append<T, 64, 1, kAt>(a, stream) : launch_append<T, 64, 0, kAt>(a, stream);
    }
    if (D == 128) return inter ? launch_append<float, 128, 1, kAt>(a, stream) : launch_append<float, 128, 0, kAt>(a, stream);
    return inter ? launch_append<float, 64, 1, kAt>(a, stream) : launch_append<float, 64, 0, kAt>(a, stream);
}
}  // namespace

extern "C" cp_status cp_cache_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, cp_dtype dtype, int64_t R, int64_t N, int64_t Nkv, int64_t D,
                                     const void *wq, const void *wk, cp_dtype w_dtype, float eps, const cp_rope *rope,
                                     int64_t pos_base, void *k_cache, void *v_cache, int64_t n_pages,
                                     int64_t page_size, const int32_t *table, int64_t B, int64_t max_pages,
                                     const int32_t *cu_new, const int32_t *kv_len, void *q_out, cudaStream_t stream) {
    return append_call<false>(q, k, v, q_stride, k_stride, v_stride, dtype, R, N, Nkv, D, wq, wk, w_dtype, eps, rope,
                              pos_base, k_cache, v_cache, n_pages, page_size, table, B, max_pages, cu_new, kv_len,
                              nullptr, nullptr, q_out, stream);
}

extern "C" cp_status cp_cache_append_at(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                                        int64_t v_stride, cp_dtype dtype, int64_t R, int64_t N, int64_t Nkv, int64_t D,
                                        const void *wq, const void *wk, cp_dtype w_dtype, float eps,
                                        const cp_rope *rope, void *k_cache, void *v_cache, int64_t n_pages,
                                        int64_t page_size, const int32_t *slots, const int32_t *pos, void *q_out,
                                        cudaStream_t stream) {
    return append_call<true>(q, k, v, q_stride, k_stride, v_stride, dtype, R, N, Nkv, D, wq, wk, w_dtype, eps, rope, 0,
                             k_cache, v_cache, n_pages, page_size, nullptr, 1, 1, nullptr, nullptr, slots, pos, q_out,
                             stream);
}
