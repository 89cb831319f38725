// pages.cu -- the pages of a step (cp_cache_plan) and the accepted branch of a drafted tree (cp_cache_keep).
//
// cp_cache_plan.  From the lengths alone: which pages a sequence gives back or takes, where its new tokens go, their
// positions.  The free pages are a stack; pages given back are pushed in the order of the sequences, then the
// taken ones popped in the same order, so the result depends on the lists only.  Everything follows from three
// running sums over the sequences (new tokens, pages taken, pages given), which every block of one cluster forms
// for itself (4096 sequences at most: four a thread); then each new row, and each moved page, looks for its
// sequence in the sums in shared memory.  Results may overwrite the lists they come from, so they are written behind a
// barrier of the cluster.  What bounds it is latency: the launch, the lists, the barrier, a page number.  In a graph 64
// sequences of one token take 3.7 us, 1000 of up to 60 tokens 6.4 (8.5 by sums of 64 bits in a cluster of 8).
//
// cp_cache_keep.  Row j of the kept path comes from row path_j >= j of the step, so a thread that takes 16
// bytes of all rows of one sequence in one cache, in rising order, never overwrites what it still has to read, and
// no thread waits for another.  Bound by the latency of scattered rows: up to 6 of 16 tokens of 64 sequences in 32 layers,
// 10.5 MB read and as much written at rows of 2 KB, take 8.7 us in a graph (3.1 at the copy's rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "cp_internal.h"
#include "cp_paged.cuh"
#include "cp_ptx.cuh"

namespace cpattn {
namespace {

// ---------------------------------------------------------------- pages of a step
constexpr int kPlanThreads = 1024;  // of a block, at most
constexpr int kPlanBlocks = 16;     // of the cluster, at most (8 where the GPU has no room for one of 16)
constexpr int kRowsEach = 4;        // neighbouring rows of a thread

struct PlanArgs {
    const int32_t *had, *keep, *n_new;
    int32_t *table, *free_pages;
    const int32_t *n_free;
    int B, max_pages, n_pages, shift, R;
    long long pos_base;
    int32_t *kv_len, *cu, *slots, *pos, *n_free_out;
    int vectors;  // slots and pos lie on 16 bytes
    int *status;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// A barrier of the cluster, behind which its writes so far are seen.
__device__ __forceinline__ void all_read(int blocks) {
    if (blocks == 1) {
        __syncthreads();
    } else {
        cluster_arrive();
        cluster_wait();
    }
}

// The last entry of sums[0 .. n - 1] (non-decreasing, sums[0] = 0) that is at most v.
__device__ __forceinline__ int place_in(const int *sums, int n, int v) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ int sums[];
    // of the B sequences: new tokens before it, pages taken before it, given before it, tokens that stay, pages had
    int *rows = sums, *takes = rows + a.B, *gives = takes + a.B, *stays = gives + a.B, *owned = stays + a.B;
    __shared__ float warp_size[kPlanThreads / 32];
    __shared__ int warp_sum[kPlanThreads / 32][3];
    wait_for_previous();
    launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, each = (a.B + blockDim.x - 1) / blockDim.x;
    const int P1 = (1 << a.shift) - 1, blocks = gridDim.x, rank = cluster_rank();
    const long long most = static_cast<long long>(a.max_pages) << a.shift;
    const int free0 = __ldcg(a.n_free);
    int had[4], keep[4], fresh[4];
    int t[3] = {0, 0, 0};
    float size = 0.f;  // of the three together: whether 32 bits hold them
    bool bad = free0 < 0 || free0 > a.n_pages;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int b = tid * each + k;
        had[k] = keep[k] = fresh[k] = 0;
        if (k < each && b < a.B) {
            had[k] = __ldcg(a.had + b);
            keep[k] = __ldcg(a.keep + b);
            fresh[k] = __ldcg(a.n_new + b);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const long long len = static_cast<long long>(keep[k]) + fresh[k];
        // (the last new position, pos_base + len - 1, has to fit 32 bits)
        const bool far = fresh[k] > 0 && a.pos_base + len > 1ll << 31;
        if (fresh[k] < 0 || keep[k] < 0 || had[k] < keep[k] || len > most || had[k] > most || far) {
            bad = true;
            continue;
        }
        const int move = static_cast<int>((len + P1) >> a.shift) - static_cast<int>((static_cast<long long>(had[k]) + P1) >> a.shift);
        t[0] += fresh[k];
        t[1] += max(move, 0);
        t[2] += max(-move, 0);
        size += static_cast<float>(fresh[k]) + static_cast<float>(abs(move));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) size += __shfl_xor_sync(0xffffffffu, size, o);
    if (lane == 0) warp_size[warp] = size;
    bad = __syncthreads_or(bad);
    int before[3] = {t[0], t[1], t[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int v = __shfl_up_sync(0xffffffffu, before[i], o);
            if (lane >= o) before[i] += v;
        }
    }
    if (lane == 31)
        for (int i = 0; i < 3; ++i) warp_sum[warp][i] = before[i];
    __syncthreads();
    int all[3] = {0, 0, 0};
    {
        // the warps before this one, and all of them
        int v[3], w[3];
        size = lane < blockDim.x / 32 ? warp_size[lane] : 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int mine = lane < blockDim.x / 32 ? warp_sum[lane][i] : 0;
            v[i] = lane < warp ? mine : 0;
            w[i] = mine;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            size += __shfl_xor_sync(0xffffffffu, size, o);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
                w[i] += __shfl_xor_sync(0xffffffffu, w[i], o);
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            before[i] += v[i] - t[i];
            all[i] = w[i];
        }
    }
    // (an fp32 sum of 8192 terms is off by less than its 1000th part: each sum is below 2^31 then; where they are not, R
    // or the stack is too small for them)
    const bool huge = !(size < 0x1.8p30f);
    bad |= huge || all[0] > a.R || all[2] > a.n_pages - free0;
    const int lacking = all[1] - (free0 + all[2]);
    const int gx = rank * blockDim.x + tid, step = blocks * blockDim.x;
    if (bad || lacking > 0) {
        // nothing is handed out: no new rows, the lengths and pages as they were
        all_read(blocks);
        for (int r = gx; r < a.R; r += step) {
            a.slots[r] = -1;
            a.pos[r] = 0;
        }
        if (rank == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = tid * each + k;
                if (k < each && b < a.B) {
                    a.kv_len[b] = had[k];
                    a.cu[b] = 0;
                }
            }
            if (tid == 0) {
                a.cu[a.B] = 0;
                a.n_free_out[0] = free0;
                a.n_free_out[1] = bad ? -1 : lacking;
                if (bad) atomicExch(a.status, static_cast<int>(CP_ERR_PAGE));
            }
        }
        return;
    }
    const int total = all[0], taken = all[1], given = all[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int b = tid * each + k;
        if (k < each && b < a.B) {
            const int pages = (had[k] + P1) >> a.shift, move = ((keep[k] + fresh[k] + P1) >> a.shift) - pages;
            rows[b] = before[0];
            takes[b] = before[1];
            gives[b] = before[2];
            stays[b] = keep[k];
            owned[b] = pages;
            before[0] += fresh[k];
            before[1] += max(move, 0);
            before[2] += max(-move, 0);
        }
    }
    __syncthreads();
    const int top = free0 + given;
    auto last_of = [&](const int *s, int b, int end) { return b + 1 < a.B ? s[b + 1] : end; };
    bool wrong = false;
    // The last given page of a sequence is its last one.  (A page number out of range goes on the stack as it is: told here,
    // by the step that puts it there, and again by the one that pops it.)
    for (int k = gx; k < given; k += step) {
        const int b = place_in(gives, a.B, k);
        const int n = last_of(gives, b, given) - gives[b];
        const int page = __ldcg(a.table + static_cast<long long>(b) * a.max_pages + owned[b] - n + k - gives[b]);
        wrong |= page < 0 || page >= a.n_pages;
        a.free_pages[free0 + k] = page;
    }
    // every block has read the lists, and what was given lies on the stack
    all_read(blocks);
    for (int k = gx; k < taken; k += step) {
        const int b = place_in(takes, a.B, k), page = __ldcg(a.free_pages + top - 1 - k);
        wrong |= page < 0 || page >= a.n_pages;
        a.table[static_cast<long long>(b) * a.max_pages + owned[b] + k - takes[b]] = page;
    }
    for (int r0 = gx * kRowsEach; r0 < a.R; r0 += step * kRowsEach) {
        int slot[kRowsEach], at[kRowsEach], page[kRowsEach];
        int b = r0 < total ? place_in(rows, a.B, r0) : 0;
#pragma unroll
        for (int k = 0; k < kRowsEach; ++k) {
            const int r = r0 + k;
            slot[k] = -1;
            at[k] = 0;
            if (r < total) {
                while (b + 1 < a.B && rows[b + 1] <= r) ++b;
                const int i = stays[b] + r - rows[b], e = i >> a.shift;
                const int32_t *where = e < owned[b] ? a.table + static_cast<long long>(b) * a.max_pages + e
                                                    : a.free_pages + (top - 1 - (takes[b] + e - owned[b]));
                page[k] = __ldcg(where);
                at[k] = static_cast<int>(a.pos_base + i);
                slot[k] = i & P1;
            }
        }
#pragma unroll
        for (int k = 0; k < kRowsEach; ++k)
            if (r0 + k < total) {
                const bool fine = page[k] >= 0 && page[k] < a.n_pages;
                slot[k] = fine ? (page[k] << a.shift) + slot[k] : -1;
                wrong |= !fine;
            }
        if (a.vectors && r0 + kRowsEach <= a.R) {
            *reinterpret_cast<int4 *>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.pos + r0) = make_int4(at[0], at[1], at[2], at[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kRowsEach; ++k)
                if (r0 + k < a.R) {
                    a.slots[r0 + k] = slot[k];
                    a.pos[r0 + k] = at[k];
                }
        }
    }
    if (wrong) atomicExch(a.status, static_cast<int>(CP_ERR_PAGE));
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = tid * each + k;
            if (k < each && b < a.B) {
                a.kv_len[b] = keep[k] + fresh[k];
                a.cu[b] = rows[b];
            }
        }
        if (tid == 0) {
            a.cu[a.B] = total;
            a.n_free_out[0] = top - taken;
            a.n_free_out[1] = 0;
        }
    }
}

// ---------------------------------------------------------------- the accepted branch
constexpr int kKeepThreads = 128;
constexpr int kMaxCaches = 256;  // K and V of 128 layers: their addresses are launch arguments
constexpr int kMaxKept = 512;    // tokens of a path: as many as a mask's row holds
constexpr int kAhead = 4;        // rows in flight of a thread, of each of two columns

struct KeepArgs {
    PageTable pt;
    const int32_t *cu, *kv_len, *kept, *n_kept;
    int32_t *kv_keep;
    int R, most, caches, cols;  // cols: 16-byte pieces of a row
    int units;                  // (cache, piece) pairs of a block
    int *status;
    uint4 *cache[kMaxCaches];
};

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
    __shared__ int from[kMaxKept], to[kMaxKept];
    __shared__ int end;
    wait_for_previous();
    launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int32_t *path = a.kept + static_cast<long long>(b) * a.most;
    // (the beginning of the path is read beside the counts that say how long it is)
    const int at0 = tid < a.most ? __ldcg(path + tid) : 0;
    const int last0 = tid && tid < a.most ? __ldcg(path + tid - 1) : -1;
    const int begin = __ldcg(a.cu + b), n = __ldcg(a.cu + b + 1) - begin, len = __ldcg(a.kv_len + b);
    int count = __ldcg(a.n_kept + b);
    const bool senseless = begin < 0 || n < 0 || n > a.R - begin || len < n;  // the lists
    const bool whole = count < 0 || senseless;                                // all new tokens stay
    bool bad = senseless || count > n || count > a.most;
    if (whole || bad) count = 0;
    const int first = len - n;
    if (tid == 0) end = count;
    __syncthreads();
    // the kept tokens, rising; the first that is not ends the path
    for (int j = tid; j < count; j += kKeepThreads) {
        const int at = j == tid ? at0 : __ldcg(path + j), last = j == tid ? last0 : __ldcg(path + j - 1);
        const bool fine = at > last && last >= -1 && at < n;
        const long long s = fine ? a.pt.slot<true>(b, static_cast<long long>(first) + at) : -1;
        const long long t = fine ? a.pt.slot<true>(b, static_cast<long long>(first) + j) : -1;
        from[j] = static_cast<int>(s);
        to[j] = static_cast<int>(t);
        if (s < 0 || t < 0) {
            atomicMin(&end, j);
            bad = true;
        }
    }
    __syncthreads();
    count = end;
    if (bad) atomicExch(a.status, static_cast<int>(CP_ERR_PAGE));
    if (blockIdx.y == 0 && tid == 0) a.kv_keep[b] = whole ? len : first + count;
    // the tokens that stay where they are come first: the path rises
    int j1 = 0;
    while (j1 < count && from[j1] == to[j1]) ++j1;
    const int u1 = min((static_cast<int>(blockIdx.y) + 1) * a.units, a.caches * a.cols);
    for (int u = blockIdx.y * a.units + tid; u < u1; u += 2 * kKeepThreads) {
        uint4 *column[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = u + i * kKeepThreads, c = v < u1 ? v / a.cols : 0;
            column[i] = v < u1 ? a.cache[c] + (v - c * a.cols) : nullptr;
        }
        for (int j0 = j1; j0 < count; j0 += kAhead) {
            uint4 v[2][kAhead];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (column[i] && j0 + k < count) v[i][k] = __ldcg(column[i] + static_cast<long long>(from[j0 + k]) * a.cols);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (column[i] && j0 + k < count) column[i][static_cast<long long>(to[j0 + k]) * a.cols] = v[i][k];
        }
    }
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

namespace {
// A launch of one cluster (`at`: room for its attributes).
cudaLaunchConfig_t plan_config(cudaLaunchAttribute *at, int blocks, int threads, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return c;
}
bool odd4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
}  // namespace

extern "C" cp_status cp_cache_plan(const int32_t *kv_had, const int32_t *kv_keep, const int32_t *n_new, int64_t B,
                                   int32_t *table, int64_t max_pages, int64_t page_size, int32_t *free_pages,
                                   int64_t n_pages, const int32_t *n_free, int64_t pos_base, int64_t R, int32_t *kv_len,
                                   int32_t *cu_new, int32_t *slots, int32_t *pos, int32_t *n_free_out,
                                   cudaStream_t stream) {
    if (!kv_had || !kv_keep || !n_new || !table || !free_pages || !n_free || !kv_len || !cu_new || !slots || !pos ||
        !n_free_out)
        return CP_ERR_NULL;
    cp_status st = check_pages(n_pages, page_size, B, max_pages, 1, 64);
    if (st != CP_OK) return st;
    if (R < 1 || R > INT32_MAX / 2) return CP_ERR_SHAPE;
    if (pos_base < INT32_MIN || pos_base > INT32_MAX) return CP_ERR_ARGUMENT;
    if (odd4(kv_had) || odd4(kv_keep) || odd4(n_new) || odd4(table) || odd4(free_pages) || odd4(n_free) || odd4(kv_len) ||
        odd4(cu_new) || odd4(slots) || odd4(pos) || odd4(n_free_out))
        return CP_ERR_ALIGNMENT;
    // What is written apart from one another and from what is read; kv_len may be kv_had or kv_keep, n_free_out n_free.
    struct Span {
        const void *p;
        int64_t n;
    };
    const Span out[] = {{table, B * max_pages}, {free_pages, n_pages}, {kv_len, B}, {cu_new, B + 1},
                        {slots, R},             {pos, R},              {n_free_out, 2}};
    const Span in[] = {{kv_had, B}, {kv_keep, B}, {n_new, B}, {n_free, 1}};
    auto meet = [](const Span &x, const Span &y) {
        const char *p = static_cast<const char *>(x.p), *q = static_cast<const char *>(y.p);
        return p < q + 4 * y.n && q < p + 4 * x.n;
    };
    for (int i = 0; i < 7; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return CP_ERR_ARGUMENT;
        for (int j = 0; j < 4; ++j) {
            const bool in_place = out[i].p == in[j].p && ((i == 2 && j < 2) || (i == 6 && j == 3));
            if (!in_place && meet(out[i], in[j])) return CP_ERR_ARGUMENT;
        }
    }
    PlanArgs a{};
    a.had = kv_had, a.keep = kv_keep, a.n_new = n_new;
    a.table = table, a.free_pages = free_pages, a.n_free = n_free;
    a.B = static_cast<int>(B), a.max_pages = static_cast<int>(max_pages), a.n_pages = static_cast<int>(n_pages);
    a.shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    a.R = static_cast<int>(R);
    a.pos_base = pos_base;
    a.kv_len = kv_len, a.cu = cu_new, a.slots = slots, a.pos = pos, a.n_free_out = n_free_out;
    if ((st = cache_status_word(&a.status)) != CP_OK) return st;
    const size_t smem = static_cast<size_t>(B) * 5 * 4;
    static int room = 0;  // blocks of the largest cluster
    static cudaError_t err = cudaSuccess;
    static std::once_flag once;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSequences * 5 * 4);
        if (err == cudaSuccess) err = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        cudaLaunchAttribute at{};
        const cudaLaunchConfig_t c = plan_config(&at, kPlanBlocks, kPlanThreads, kMaxSequences * 5 * 4, nullptr);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, plan_kernel, &c) != cudaSuccess) cudaGetLastError();
        room = n > 0 ? kPlanBlocks : 8;
    });
    if (err != cudaSuccess) return cuda_status(err);
    a.vectors = aligned16(slots) && aligned16(pos);
    // Four sequences a thread at most, and a thread for four rows: up to 2048 rows by a larger block, up to 16384 by more
    // blocks, each of which forms all sums, then by larger ones again.
    int threads = 128, blocks = 1;
    auto rows = [&] { return static_cast<int64_t>(blocks) * threads * kRowsEach; };
    while (threads < kPlanThreads && (threads * 4 < B || (threads < 512 && rows() < R))) threads *= 2;
    while (blocks < room && rows() < R) blocks *= 2;
    while (threads < kPlanThreads && rows() < R) threads *= 2;
    cudaLaunchAttribute at[2] = {};
    cudaLaunchConfig_t c = plan_config(at, blocks, threads, smem, stream);
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&c, plan_kernel, a);
    if (e != cudaSuccess) cudaGetLastError();
    return cuda_status(e);
}

extern "C" cp_status cp_cache_keep(void *const *caches, int64_t n_caches, int64_t n_pages, int64_t page_size, int64_t Nkv,
                                   int64_t D, const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                   const int32_t *kv_len, int64_t R, const int32_t *kept, int64_t max_kept,
                                   const int32_t *n_kept, int32_t *kv_keep, cudaStream_t stream) {
    if (!caches || !table || !cu_new || !kv_len || !kept || !n_kept || !kv_keep) return CP_ERR_NULL;
    cp_status st = check_pages(n_pages, page_size, B, max_pages, Nkv, D);
    if (st != CP_OK) return st;
    if (n_caches < 1 || n_caches > kMaxCaches || max_kept < 1 || max_kept > kMaxKept || R < 1 || R > INT32_MAX / 2)
        return CP_ERR_SHAPE;
    KeepArgs a{};
    const int64_t bytes = n_pages * page_size * Nkv * D * 2;
    for (int64_t i = 0; i < n_caches; ++i) {
        if (!caches[i]) return CP_ERR_NULL;
        if (!aligned16(caches[i])) return CP_ERR_ALIGNMENT;
        a.cache[i] = static_cast<uint4 *>(caches[i]);
    }
    uintptr_t order[kMaxCaches];
    for (int64_t i = 0; i < n_caches; ++i) order[i] = reinterpret_cast<uintptr_t>(caches[i]);
    std::sort(order, order + n_caches);
    for (int64_t i = 1; i < n_caches; ++i)
        if (order[i] - order[i - 1] < static_cast<uintptr_t>(bytes)) return CP_ERR_ARGUMENT;  // two overlap
    if (odd4(table) || odd4(cu_new) || odd4(kv_len) || odd4(kept) || odd4(n_kept) || odd4(kv_keep)) return CP_ERR_ALIGNMENT;
    const char *w = reinterpret_cast<const char *>(kv_keep);
    const struct {
        const void *p;
        int64_t n;
    } in[] = {{table, B * max_pages}, {cu_new, B + 1}, {kv_len, B}, {kept, B * max_kept}, {n_kept, B}};
    for (const auto &x : in) {
        const char *p = static_cast<const char *>(x.p);
        if (w < p + 4 * x.n && p < w + 4 * B) return CP_ERR_ARGUMENT;
    }
    a.pt.table = table;
    a.pt.B = static_cast<int>(B);
    a.pt.max_pages = static_cast<int>(max_pages);
    a.pt.n_pages = static_cast<int>(n_pages);
    a.pt.shift = __builtin_ctzll(static_cast<unsigned long long>(page_size));
    a.cu = cu_new, a.kv_len = kv_len, a.kept = kept, a.n_kept = n_kept, a.kv_keep = kv_keep;
    a.R = static_cast<int>(R), a.most = static_cast<int>(max_kept), a.caches = static_cast<int>(n_caches);
    a.cols = static_cast<int>(Nkv * D / 8);
    if ((st = cache_status_word(&a.status)) != CP_OK) return st;
    const int64_t all = n_caches * a.cols;
    // As many rounds of two columns a thread as leave about eight small blocks an SM: what a block does first costs
    // it three loads in a row, which others' copies have to cover.  A small call needs many blocks, each soon begun.
    // (Up to 6 of 16 tokens of 64 sequences in 32 layers, and of 27 tokens of one in 16, us in a graph: 8 blocks of 128
    // threads 8.7 and 2.9, call after call with other data 9.1; 4 of 256 threads 9.6 and 3.2, 9.5; 2 of 256 10.2, 10.4; 12 of
    // 64 8.5 and 2.8, but 11.1; with six rows in flight 8.6 and 3.1.)
    const int64_t pairs = (all + 2 * kKeepThreads - 1) / (2 * kKeepThreads);
    int64_t most = (8LL * sm_count() + B - 1) / B;
    most = most < pairs ? most : pairs;
    most = most < 4096 ? most : 4096;
    a.units = static_cast<int>((pairs + most - 1) / most * 2 * kKeepThreads);
    const int64_t parts = (all + a.units - 1) / a.units;
    return launch(keep_kernel, dim3(static_cast<unsigned>(B), static_cast<unsigned>(parts)), kKeepThreads, 0, stream, a);
}
