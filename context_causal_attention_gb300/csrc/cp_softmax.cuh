// cp_softmax.cuh -- the register arithmetic of a softmax row held by one thread,
// shared by the bf16 tensor-memory kernels (attn.cu, prefix_tc.cuh).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_ptx.cuh"

namespace cpattn {

// p = 2^(s * sl2 - m) for 64 scores, packed to 32 bf16 pairs; returns the
// fp32 sum of p.
__device__ __forceinline__ float exp_pack64(const uint32_t (&h)[64], float sl2, float neg_m, uint32_t (&pk)[32]) {
    const uint64_t sl2x2 = f2_packf(sl2, sl2), nmx2 = f2_packf(neg_m, neg_m);
    uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float x0, x1, x2, x3;
        f2_unpack(f2_fma(f2_pack(h[2 * c], h[2 * c + 1]), sl2x2, nmx2), x0, x1);
        f2_unpack(f2_fma(f2_pack(h[2 * c + 2], h[2 * c + 3]), sl2x2, nmx2), x2, x3);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        const float p2 = fast_exp2(x2), p3 = fast_exp2(x3);
        sum2[(c >> 1) & 1] = f2_add(sum2[(c >> 1) & 1], f2_packf(p0, p1));
        sum2[2 + ((c >> 1) & 1)] = f2_add(sum2[2 + ((c >> 1) & 1)], f2_packf(p2, p3));
        pk[c] = pack_bf16x2(p0, p1);
        pk[c + 1] = pack_bf16x2(p2, p3);
    }
    const uint64_t t = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
    float lo, hi;
    f2_unpack(t, lo, hi);
    return lo + hi;
}

// Row max of the 128 scores of one thread (raw fp32 bits), 8 independent chains.
__device__ __forceinline__ float row_max128(const uint32_t (&sa)[64], const uint32_t (&sb)[64]) {
    float mx[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
#pragma unroll
    for (int c = 0; c < 64; c += 8) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            mx[u] = fmax3(mx[u], __uint_as_float(sa[c + 2 * u]), __uint_as_float(sa[c + 2 * u + 1]));
            mx[4 + u] = fmax3(mx[4 + u], __uint_as_float(sb[c + 2 * u]), __uint_as_float(sb[c + 2 * u + 1]));
        }
    }
    return fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
}

// p = 2^(s * sl2 - m) for the 128 scores of one thread, packed to bf16 pairs
// in pa/pb; returns the sum of the fp32 p in *sum.
__device__ __forceinline__ void exp_pack128(const uint32_t (&sa)[64], const uint32_t (&sb)[64], float sl2,
                                            float neg_m, uint32_t (&pa)[32], uint32_t (&pb)[32], float *sum) {
    const uint64_t sl2x2 = f2_packf(sl2, sl2), nmx2 = f2_packf(neg_m, neg_m);
    uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        float x0, x1, x2, x3;
        f2_unpack(f2_fma(f2_pack(sa[2 * c], sa[2 * c + 1]), sl2x2, nmx2), x0, x1);
        f2_unpack(f2_fma(f2_pack(sb[2 * c], sb[2 * c + 1]), sl2x2, nmx2), x2, x3);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        const float p2 = fast_exp2(x2), p3 = fast_exp2(x3);
        sum2[c & 1] = f2_add(sum2[c & 1], f2_packf(p0, p1));
        sum2[2 + (c & 1)] = f2_add(sum2[2 + (c & 1)], f2_packf(p2, p3));
        pa[c] = pack_bf16x2(p0, p1);
        pb[c] = pack_bf16x2(p2, p3);
    }
    const uint64_t t = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
    float lo, hi;
    f2_unpack(t, lo, hi);
    *sum = lo + hi;
}

}  // namespace cpattn
