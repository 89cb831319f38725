// cp_rope.cuh -- device pieces shared by the kernels that rotate head rows by
// their positions (rope.cu, cache.cu).
//
// A pair (a, b) of a head row at position t becomes
//   a' = A (a cos t theta_i - b sin t theta_i),  b' = A (b cos t theta_i + a sin t theta_i).
// The frequency theta_i is held as a 64-bit fixed-point number of TURNS per
// position, F_i = round(theta_i / (2 pi) 2^64) mod 2^64, so t * F_i mod 2^64 is
// the fraction of a turn at position t: the range reduction is one integer
// multiplication and exact.  What is left of the error that grows with the position is
// that of F, an fp64 quotient: t (theta 2^-52 + 2^-62) radians, 1.3e-7 measured at 2^31
// for base 10000 (an fp32 angle is off by t theta 2^-24, 0.06 at a million).  The top 32 bits
// then go through sincospif.
//
// Work split: a head row of D values is held by L = D/16 lanes, 16 values
// each: the two 16-byte pieces that hold the lane's 8 pairs (half order: the
// same piece of both halves; interleaved order: two neighbouring pieces), so a
// rotation needs no exchange between lanes and an in-place call is safe.  A
// warp holds 32/L rows of one token at a time; the token's sines are computed
// once, one or two per lane, and handed round by shuffles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cp_ptx.cuh"

namespace cpattn {

struct RopeDev {
    const unsigned long long *freqs;  // [half] turns per position, 64-bit fixed point
    int half;                         // rotated pairs (0: no rotation)
    float amp;
};

template <typename T>
struct Vec8;  // 8 values of one 16-byte (bf16) or 32-byte (fp32) piece
template <>
struct Vec8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void load_pieces(const uint4 *p, int) { r = *p; }
    __device__ __forceinline__ void to(float *x) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    // The two 16-byte pieces `apart` places from one another.
    __device__ __forceinline__ void load_pieces(const uint4 *p, int apart) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + apart);
    }
    __device__ __forceinline__ void to(float *x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) {
    uint4 r;
    r.x = pack_bf16x2(x[0], x[1]);
    r.y = pack_bf16x2(x[2], x[3]);
    r.z = pack_bf16x2(x[4], x[5]);
    r.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4 *>(p) = r;
}
__device__ __forceinline__ void store8(float *p, const float *x) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Where this lane's 16 values of a row lie, and which of its 8 pairs turn.
template <int D, int kOrder>
struct LaneMap {
    static constexpr int L = D / 16;       // lanes of a row
    static constexpr int kRows = 32 / L;   // rows of a warp at a time
    static constexpr int kAng = D / 64;    // angles that each lane computes
    int c0, c1;                            // first column of the two pieces
    uint32_t mask;                         // bit e: pair e is rotated
    __device__ __forceinline__ LaneMap(int lane, int half) {
        const int p = lane % L;
        if (kOrder == 0) {
            // half order (half % 8 == 0): piece p of both halves; the lanes past the
            // rotated part hold two neighbouring pieces of the rest
            const int hv = half >> 3;
            const bool turns = p < hv;
            c0 = 8 * (turns ? p : 2 * p);
            c1 = 8 * (turns ? p + hv : 2 * p + 1);
            mask = turns ? 0xffu : 0u;
        } else {
            c0 = 16 * p;
            c1 = c0 + 8;
            const int n = min(8, max(0, half - 8 * p));
            mask = (1u << n) - 1u;
        }
    }
};

// Turns per position of the angles that this lane computes (0 past the end).
template <int kAng>
__device__ __forceinline__ void load_freqs(const RopeDev &r, int lane, unsigned long long (&f)[kAng]) {
#pragma unroll
    for (int i = 0; i < kAng; ++i) {
        const int idx = lane * kAng + i;
        f[i] = idx < r.half ? __ldg(r.freqs + idx) : 0ull;
    }
}

// Amplitude * (cos, sin) of this lane's 8 pairs (pairs 8p .. 8p+7 of the row,
// p = lane % L) at position `pos`.  Warp-wide.
template <int D>
__device__ __forceinline__ void token_angles(const unsigned long long (&f)[D / 64], long long pos, float amp,
                                             int lane, float (&c)[8], float (&s)[8]) {
    constexpr int kAng = D / 64, L = D / 16;
    float cl[kAng], sl[kAng];
#pragma unroll
    for (int i = 0; i < kAng; ++i) {
        const unsigned long long turn = static_cast<unsigned long long>(pos) * f[i];
        // the top 32 bits as a signed fraction of half a turn, in [-1, 1)
        const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
        sincospif(half_turns, &sl[i], &cl[i]);
        cl[i] *= amp;
        sl[i] *= amp;
    }
    const int p = lane % L;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int src = (8 * p + e) / kAng;
        c[e] = __shfl_sync(0xffffffffu, cl[e % kAng], src);
        s[e] = __shfl_sync(0xffffffffu, sl[e % kAng], src);
    }
}

// Column of value v (0..7: piece 0, 8..15: piece 1) in the pair order: pair e
// is (x[ia(e)], x[ib(e)]).
template <int kOrder>
__device__ __forceinline__ constexpr int ia(int e) { return kOrder == 0 ? e : 2 * e; }
template <int kOrder>
__device__ __forceinline__ constexpr int ib(int e) { return kOrder == 0 ? 8 + e : 2 * e + 1; }

// Rotates the lane's 8 pairs in place.  Values outside the rotated part stay
// as they are, bit for bit (kAll: there are none).
template <int kOrder, bool kAll>
__device__ __forceinline__ void turn_pairs(float (&x)[16], const float (&c)[8], const float (&s)[8], uint32_t mask) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = x[ia<kOrder>(e)], b = x[ib<kOrder>(e)];
        const float ra = a * c[e] - b * s[e], rb = b * c[e] + a * s[e];
        const bool t = kAll || ((mask >> e) & 1u);
        x[ia<kOrder>(e)] = t ? ra : a;
        x[ib<kOrder>(e)] = t ? rb : b;
    }
}

// This lane's 16 weights.
template <typename Map>
__device__ __forceinline__ void load_weights(const void *w, int bf16, const Map &m, float (&o)[16]) {
    if (bf16) {
        Vec8<__nv_bfloat16> v;
        v.load(static_cast<const __nv_bfloat16 *>(w) + m.c0);
        v.to(o);
        v.load(static_cast<const __nv_bfloat16 *>(w) + m.c1);
        v.to(o + 8);
    } else {
        Vec8<float> v;
        v.load(static_cast<const float *>(w) + m.c0);
        v.to(o);
        v.load(static_cast<const float *>(w) + m.c1);
        v.to(o + 8);
    }
}

// Sum over the L lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace cpattn
