// cp_paged.cuh -- device pieces of the paged cache shared by the append and the
// attention that reads it.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace cpattn {

constexpr int kMaxSequences = 4096;          // sequences of one call
constexpr long long kMaxKeys = 0x7fffff00ll;  // slots of a cache, of a list or of a prefix: the end of the last tile fits 31 bits

// The page lists of B sequences.  Every page number is checked where it is
// read, so a wrong table never leads outside the cache.
struct PageTable {
    const int32_t *table;  // [B][max_pages]
    int B, max_pages, n_pages;
    int shift;  // log2 of the tokens of a page
    // Slot (page * page_size + offset) of own index idx of sequence b, or -1.  kPastL1: see find_sequence().
    template <bool kPastL1 = false>
    __device__ __forceinline__ long long slot(int b, long long idx) const {
        if (idx < 0 || (idx >> shift) >= max_pages) return -1;
        const int32_t *entry = table + static_cast<long long>(b) * max_pages + (idx >> shift);
        const int page = kPastL1 ? __ldcg(entry) : __ldg(entry);
        if (page < 0 || page >= n_pages) return -1;
        return (static_cast<long long>(page) << shift) + (idx & ((1 << shift) - 1));
    }
};

// The sequence that new token `tok` belongs to by the cumulative counts cu[0..B]
// (the last b with cu[b] <= tok; -1 for rows outside all sequences), where it
// begins and how many new tokens it has.  Warp-wide: 32 probes a level.  kPastL1: for a
// kernel that starts under the one before it, when an SM's L1 may still hold what another
// call's list said.
template <bool kPastL1 = false>
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int tok, int lane, int *begin, int *count) {
    auto at = [](const int32_t *p) { return kPastL1 ? __ldcg(p) : __ldg(p); };
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 31) >> 5;
        const int mine = lane * step;
        const bool ok = mine < n && at(cu + lo + mine) <= tok;
        const int k = __popc(__ballot_sync(0xffffffffu, ok));
        if (k == 0) return -1;
        lo += (k - 1) * step;
        if (step == 1) break;
        n = min(step, n - (k - 1) * step);
    }
    const int c0 = at(cu + lo), c1 = at(cu + lo + 1);
    if (tok < c0 || tok >= c1) return -1;
    *begin = c0;
    *count = c1 - c0;
    return lo;
}

}  // namespace cpattn
