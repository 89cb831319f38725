// rope.cu -- rotary positions and the per-head norm of q and k with the
// rotation in the same pass, forward and backward.
//
//   rotation      y = A R(t) x                      (cp_rope.cuh)
//   its gradient  dx = A R(-t) dy
//   norm          r = (mean_j x_j^2 + eps)^(-1/2),  y = A R(t) (w . r x)
//   its gradient  g = A R(-t) dy,  xh = r x,  u = w . g,
//                 dx = r (u - xh mean_j(u_j xh_j)),  dw = sum over rows of g . xh
//
// All of it is bound by memory: 2 D (norm backward 3 D) values per head row move
// for a few operations each.  32768 tokens, bf16, heads of 128: the rotation of 32 + 32
// heads 171 us (6.3 TB/s), the norm of 32 + 8 111 us (6.0), its gradient 175 us
// (5.75).  One warp takes a token (or, with few tokens, a
// few of its heads, so that a single token still spreads over the SMs), works
// out its sines once and streams the head rows through registers, several rows
// in flight; everything between the load and the store is in fp32 and rounded
// once.  The weight gradients are kept in registers over all rows of a thread,
// summed over the block in a fixed order and then over the blocks by a second
// small launch, so they are the same from run to run (no atomics).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "cp_internal.h"
#include "cp_rope.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGrid = 608;  // 152 SMs x 4 blocks; also the number of weight-gradient partials

struct RowsArgs {
    const void *x[2], *g[2];  // q and k: the rows (forward: to turn; backward: the norm's input) and the gradients
    void *y[2];
    const void *w[2];
    long long xs[2], gs[2], ys[2];  // elements between tokens
    int heads[2];
    const int32_t *pos;
    RopeDev rope;
    float sgn;        // -1: the rotation is undone
    float eps;
    int w_bf16;
    long long tokens;
    int B, s;         // token ((c B + b) s + i) has position pos[c s + i]
    int chunks, hpu;  // units per token, heads per unit
    int split, kchunks;  // norm backward: blocks of q, units of a token's k rows (chunks: of its q rows)
    float *part;         // norm backward: [grid][D] partial weight gradients
};

__device__ __forceinline__ long long token_position(const RowsArgs &a, long long tok) {
    if (!a.pos) return 0;
    if (a.B == 1) return __ldg(a.pos + tok);
    const uint32_t t = static_cast<uint32_t>(tok), u = t / static_cast<uint32_t>(a.s);
    return __ldg(a.pos + static_cast<long long>(u / static_cast<uint32_t>(a.B)) * a.s + (t - u * a.s));
}

template <typename T, int D, int kOrder, bool kNorm, bool kAll>
__global__ void __launch_bounds__(kThreads, 2) rows_fwd_kernel(const RowsArgs a) {
    using Map = LaneMap<D, kOrder>;
    // rows of a lane in flight (bf16, norm of 32768 tokens: 111 us with four, 151 with two)
    constexpr int kU = sizeof(T) == 2 ? 4 : 2;
    const int lane = threadIdx.x & 31, sub = lane / Map::L;
    const Map map(lane, a.rope.half);
    unsigned long long f[Map::kAng];
    load_freqs(a.rope, lane, f);
    const long long units = a.tokens * a.chunks;
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += step) {
        const long long tok = a.chunks == 1 ? u : u / a.chunks;
        const int first = static_cast<int>(u - tok * a.chunks) * a.hpu;
        const int last = min(first + a.hpu, a.heads[0] + a.heads[1]);
        float c[8], s[8];
        token_angles<D>(f, token_position(a, tok), a.rope.amp, lane, c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] *= a.sgn;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            const int base = t ? a.heads[0] : 0;
            const int h0 = max(first - base, 0), h1 = min(last - base, a.heads[t]);
            if (h0 >= h1) continue;
            const T *x = static_cast<const T *>(a.x[t]) + tok * a.xs[t];
            T *y = static_cast<T *>(a.y[t]) + tok * a.ys[t];
            float w[16];
            if (kNorm) load_weights(a.w[t], a.w_bf16, map, w);
            for (int hb = h0; hb < h1; hb += kU * Map::kRows) {
                Vec8<T> v0[kU], v1[kU];
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    const int h = hb + i * Map::kRows + sub;
                    if (h < h1) {
                        v0[i].load(x + h * D + map.c0);
                        v1[i].load(x + h * D + map.c1);
                    }
                }
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    if (hb + i * Map::kRows >= h1) break;  // uniform over the warp
                    const int h = hb + i * Map::kRows + sub;
                    float r[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0.f;
                    if (h < h1) {
                        v0[i].to(r);
                        v1[i].to(r + 8);
                    }
                    if (kNorm) {
                        float q = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) q = fmaf(r[e], r[e], q);
                        const float rstd = rsqrtf(row_sum<Map::L>(q) * (1.f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[e] = r[e] * rstd * w[e];
                    }
                    turn_pairs<kOrder, kAll>(r, c, s, map.mask);
                    if (h < h1) {
                        store8(y + h * D + map.c0, r);
                        store8(y + h * D + map.c1, r + 8);
                    }
                }
            }
        }
    }
}

// The first `split` blocks take the rows of q, the others those of k, so that a
// thread keeps one set of weights and of weight gradients.  Those and a row's
// values fill the registers, so the rows to come wait in shared memory: a lane
// copies the pieces that it will read itself (cp.async, kAhead rows ahead, over the
// ends of tokens), so no barrier is needed.  S=32768, 32 + 8 heads of 128, bf16, with
// the sums: one row ahead in registers 197 us, two in shared memory 175 us (1.01 GB).
constexpr int kAhead = 2;
template <typename T>
constexpr int kBwdSmem = (kAhead + 1) * kThreads * 4 * 8 * static_cast<int>(sizeof(T));

template <typename T, int D, int kOrder, bool kAll>
__global__ void __launch_bounds__(kThreads, 2) norm_bwd_kernel(const RowsArgs a) {
    using Map = LaneMap<D, kOrder>;
    constexpr int kStages = kAhead + 1;
    constexpr int kPieces = sizeof(T) / 2;  // 16-byte pieces of 8 values
    launch_dependents();
    extern __shared__ __align__(16) uint4 stage_s[];  // [stage][x0, x1, g0, g1: pieces][thread]
    __shared__ float red[kWarps][D];
    const int lane = threadIdx.x & 31, sub = lane / Map::L, warp = threadIdx.x >> 5;
    const Map map(lane, a.rope.half);
    const int t = static_cast<int>(blockIdx.x) >= a.split;
    const int block = blockIdx.x - (t ? a.split : 0), blocks = t ? gridDim.x - a.split : a.split;
    const int heads = a.heads[t], chunks = t ? a.kchunks : a.chunks;
    const long long units = a.tokens * chunks;
    const long long step = static_cast<long long>(blocks) * kWarps;
    // A place in the warp's rows: unit u of token tok, rows hb .. hb + kRows - 1 of its heads up to h1.
    struct At {
        long long u, tok;
        int hb, h1;
    };
    auto open = [&](At &p) {
        p.tok = chunks == 1 ? p.u : p.u / chunks;
        p.hb = static_cast<int>(p.u - p.tok * chunks) * a.hpu;
        p.h1 = min(p.hb + a.hpu, heads);
    };
    auto advance = [&](At &p) {
        p.hb += Map::kRows;
        if (p.hb >= p.h1) {
            p.u += step;
            if (p.u < units) open(p);
        }
    };
    At next;
    next.u = static_cast<long long>(block) * kWarps + warp;
    if (next.u < units) open(next);
    At cur = next;
    int in = 0;
    auto copy_next = [&]() {
        if (next.u < units) {
            const int h = next.hb + sub;
            if (h < next.h1) {
                const T *x = static_cast<const T *>(a.x[t]) + next.tok * a.xs[t] + h * D;
                const T *g = static_cast<const T *>(a.g[t]) + next.tok * a.gs[t] + h * D;
                const T *src[4] = {x + map.c0, x + map.c1, g + map.c0, g + map.c1};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < kPieces; ++k)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         smem_u32(stage_s + ((in * 4 + i) * kPieces + k) * kThreads + threadIdx.x)),
                                     "l"(src[i] + k * (16 / sizeof(T)))
                                     : "memory");
            }
            advance(next);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = in + 1 == kStages ? 0 : in + 1;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) copy_next();
    unsigned long long f[Map::kAng];
    load_freqs(a.rope, lane, f);
    float w[16], dw[16], c[8], s[8];
    load_weights(a.w[t], a.w_bf16, map, w);
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.f;
    long long tok = -1;
    for (int out = 0; cur.u < units; advance(cur), out = out + 1 == kStages ? 0 : out + 1) {
        copy_next();
        if (cur.tok != tok) {
            tok = cur.tok;
            token_angles<D>(f, token_position(a, tok), a.rope.amp, lane, c, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        const int h = cur.hb + sub;
        const bool in_row = h < cur.h1;
        float r[16], d[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = d[e] = 0.f;
        if (in_row) {
            const uint4 *mine = stage_s + out * 4 * kPieces * kThreads + threadIdx.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Vec8<T> v;
                v.load_pieces(mine + i * kPieces * kThreads, kThreads);
                v.to((i < 2 ? r : d) + 8 * (i & 1));
            }
        }
        turn_pairs<kOrder, kAll>(d, c, s, map.mask);
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) q = fmaf(r[e], r[e], q);
        const float rstd = rsqrtf(row_sum<Map::L>(q) * (1.f / D) + a.eps);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            r[e] *= rstd;
            if (in_row) dw[e] = fmaf(d[e], r[e], dw[e]);
            d[e] *= w[e];
            m = fmaf(d[e], r[e], m);
        }
        m = row_sum<Map::L>(m) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) d[e] = rstd * (d[e] - r[e] * m);
        if (in_row) {
            T *y = static_cast<T *>(a.y[t]) + tok * a.ys[t] + h * D;
            store8(y + map.c0, d);
            store8(y + map.c1, d + 8);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // over the rows that the warp held side by side, then over the block's warps
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float v = dw[e];
#pragma unroll
        for (int o = Map::L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0) red[warp][(e < 8 ? map.c0 : map.c1 - 8) + e] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += red[k][i];
        a.part[static_cast<long long>(blockIdx.x) * D + i] = v;
    }
}

// dw[t][j] = sum over the partials of q's blocks (t = 0: the first `split`) or
// k's, in a fixed order; 32 columns to a block.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) dw_sum_kernel(const float *part, int split, int n, int D, float *dwq,
                                                                float *dwk) {
    __shared__ float red[kSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.y, col = blockIdx.x * 32 + lane;
    wait_for_previous();
    float v = 0.f;
#pragma unroll 4
    for (int i = (t ? split : 0) + warp; i < (t ? n : split); i += kSumWarps)
        v += part[static_cast<long long>(i) * D + col];
    red[warp][lane] = v;
    __syncthreads();
    v = red[lane][warp];  // column `warp`: its 32 partial sums across the lanes
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    float *out = t ? dwk : dwq;
    if (out && lane == 0) out[blockIdx.x * 32 + warp] = v;
}

// ---------------------------------------------------------------- host side
bool misaligned(const void *p) { return p && !aligned16(p); }

// One of q and k: `tokens` rows of heads * D values, `stride` elements apart.
struct Rows {
    const char *p;
    long long bytes;  // from the first row to the end of the last
    long long step, row;
    Rows(const void *q, long long tokens, long long stride, long long heads, long long D, size_t es)
        : p(static_cast<const char *>(q)), bytes(q && heads ? ((tokens - 1) * stride + heads * D) * (long long)es : 0),
          step(stride * (long long)es), row(heads * D * (long long)es) {}
    // Whether any value belongs to both (false for slices side by side in the rows of one buffer).
    bool meets(const Rows &o) const {
        if (!bytes || !o.bytes || p >= o.p + o.bytes || o.p >= p + bytes) return false;
        if (step != o.step) return true;
        const long long at = ((o.p - p) % step + step) % step;  // o's rows begin so far behind these
        return at < row || at + o.row > step;
    }
};

cp_status check_sizes(int64_t C, int64_t B, int64_t s, int64_t N, int64_t Nkv, int64_t D) {
    if (C < 1 || B < 1 || s < 1 || N < 0 || Nkv < 0 || N + Nkv < 1) return CP_ERR_SHAPE;
    if (C > INT32_MAX || B > INT32_MAX || s > INT32_MAX || N > 65535 || Nkv > 65535) return CP_ERR_SHAPE;
    if (C * B > INT32_MAX || C * B * s > INT32_MAX) return CP_ERR_SHAPE;
    if (D != 64 && D != 128) return CP_ERR_UNSUPPORTED;
    return CP_OK;
}

}  // namespace

cp_status check_rope(const cp_rope *rope, int64_t D) {
    if (!rope) return CP_OK;
    if (!rope->freqs) return CP_ERR_NULL;
    if (rope->order != CP_ROPE_HALF && rope->order != CP_ROPE_INTERLEAVED) return CP_ERR_ARGUMENT;
    if (rope->rot_dim < 2 || rope->rot_dim > D || rope->rot_dim % 2) return CP_ERR_SHAPE;
    if (rope->order == CP_ROPE_HALF && rope->rot_dim % 16) return CP_ERR_UNSUPPORTED;
    if (!std::isfinite(rope->amplitude)) return CP_ERR_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(rope->freqs) & 7u) return CP_ERR_ALIGNMENT;
    return CP_OK;
}

namespace {

// Checks what every row call shares and fills the common arguments.  x: the
// tensors read with strides qs, ks; y: written, in place of x where the
// pointers are equal, else dense.
cp_status fill_rows(RowsArgs *a, const void *q, const void *k, void *qo, void *ko, const int32_t *pos, int64_t C,
                    int64_t B, int64_t s, int64_t N, int64_t Nkv, int64_t D, int64_t qs, int64_t ks, cp_dtype dtype,
                    const cp_rope *rope) {
    cp_status st = check_sizes(C, B, s, N, Nkv, D);
    if (st != CP_OK) return st;
    if ((N && (!q || !qo)) || (Nkv && (!k || !ko)) || (rope && !pos)) return CP_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if (!es) return CP_ERR_DTYPE;
    if ((st = check_rope(rope, D)) != CP_OK) return st;
    if ((N && qs < N * D) || (Nkv && ks < Nkv * D) || qs > INT32_MAX || ks > INT32_MAX) return CP_ERR_SHAPE;
    if ((N && qs * es % 16) || (Nkv && ks * es % 16) || misaligned(q) || misaligned(k) || misaligned(qo) ||
        misaligned(ko) || (reinterpret_cast<uintptr_t>(pos) & 3u))
        return CP_ERR_ALIGNMENT;
    const long long tokens = C * B * s;
    const bool in_q = N && q == qo, in_k = Nkv && k == ko;
    const Rows rq(q, tokens, qs, N, D, es), rk(k, tokens, ks, Nkv, D, es);
    const Rows oq(qo, tokens, in_q ? qs : N * D, N, D, es), ok(ko, tokens, in_k ? ks : Nkv * D, Nkv, D, es);
    if ((!in_q && oq.meets(rq)) || (!in_k && ok.meets(rk)) || oq.meets(rk) || ok.meets(rq) || oq.meets(ok))
        return CP_ERR_ARGUMENT;
    *a = RowsArgs{};
    a->x[0] = q, a->x[1] = k;
    a->y[0] = qo, a->y[1] = ko;
    a->xs[0] = qs, a->xs[1] = ks;
    a->ys[0] = in_q ? qs : N * D, a->ys[1] = in_k ? ks : Nkv * D;
    a->heads[0] = static_cast<int>(N), a->heads[1] = static_cast<int>(Nkv);
    a->pos = rope ? pos : nullptr;
    if (rope) {
        a->rope.freqs = reinterpret_cast<const unsigned long long *>(rope->freqs);
        a->rope.half = static_cast<int>(rope->rot_dim / 2);
        a->rope.amp = rope->amplitude;
    }
    a->sgn = 1.f;
    a->tokens = tokens;
    a->B = static_cast<int>(B), a->s = static_cast<int>(s);
    return CP_OK;
}

// Heads of a unit: a token's sines are worked out once for a unit, so all of its
// heads, but fewer where that leaves SMs with less than kUnitWarps warps: as many
// units as do not pass that.  Norm of 32 + 8 heads of 128, in a graph: 1 token 2.7 us
// in ten units, 4.7 in one; 256 tokens 3.6 in nine, 5.8 in one, 4.3 in ten;
// 1024 tokens 5.5 in two, 6.1 in one, 6.7 in three; 4096 tokens 14.4 in one, 15.8 in two.
constexpr int kUnitWarps = 16;
int plan_units(RowsArgs *a, int rows) {
    const int heads = a->heads[0] + a->heads[1], most = (heads + rows - 1) / rows;
    long long chunks = static_cast<long long>(sm_count()) * kUnitWarps / a->tokens;
    chunks = chunks < 1 ? 1 : (chunks > most ? most : chunks);
    a->hpu = static_cast<int>((most + chunks - 1) / chunks) * rows;
    a->chunks = (heads + a->hpu - 1) / a->hpu;
    const long long blocks = (a->tokens * a->chunks + kWarps - 1) / kWarps;
    return static_cast<int>(blocks < kMaxGrid ? blocks : kMaxGrid);
}

template <typename T, int D, int kOrder, bool kAll>
cp_status launch_fwd(RowsArgs &a, bool norm, cudaStream_t stream) {
    const int grid = plan_units(&a, LaneMap<D, kOrder>::kRows);
    if (norm)
        rows_fwd_kernel<T, D, kOrder, true, kAll><<<grid, kThreads, 0, stream>>>(a);
    else
        rows_fwd_kernel<T, D, kOrder, false, kAll><<<grid, kThreads, 0, stream>>>(a);
    return last_launch_status();
}

// Calls f<T, D, order, all>() of the call's dtype, head size, order and whether the whole head turns.
template <typename F>
cp_status dispatch(int64_t D, cp_dtype dtype, const cp_rope *rope, F f) {
    const bool inter = rope && rope->order == CP_ROPE_INTERLEAVED, all = rope && rope->rot_dim == D;
    auto with = [&](auto t, auto d) -> cp_status {
        using T = decltype(t);
        constexpr int kD = decltype(d)::value;
        if (inter) return all ? f.template operator()<T, kD, 1, true>() : f.template operator()<T, kD, 1, false>();
        return all ? f.template operator()<T, kD, 0, true>() : f.template operator()<T, kD, 0, false>();
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (dtype == CP_BF16) return D == 128 ? with(__nv_bfloat16{}, D128{}) : with(__nv_bfloat16{}, D64{});
    return D == 128 ? with(float{}, D128{}) : with(float{}, D64{});
}
struct Fwd {
    RowsArgs &a;
    bool norm;
    cudaStream_t stream;
    template <typename T, int D, int kOrder, bool kAll>
    cp_status operator()() const {
        return launch_fwd<T, D, kOrder, kAll>(a, norm, stream);
    }
};
cp_status run_fwd(RowsArgs &a, bool norm, int64_t D, cp_dtype dtype, const cp_rope *rope, cudaStream_t stream) {
    return dispatch(D, dtype, rope, Fwd{a, norm, stream});
}

template <typename T, int D, int kOrder, bool kAll>
cp_status launch_bwd_typed(RowsArgs &a, float *dwq, float *dwk, cudaStream_t stream) {
    constexpr int rows = LaneMap<D, kOrder>::kRows;
    plan_units(&a, rows);
    // the blocks in proportion to the heads, at least one for either tensor
    const long long nq = a.heads[0], nk = a.heads[1];
    a.chunks = static_cast<int>((nq + a.hpu - 1) / a.hpu);
    a.kchunks = static_cast<int>((nk + a.hpu - 1) / a.hpu);
    const long long bq = (a.tokens * a.chunks + kWarps - 1) / kWarps, bk = (a.tokens * a.kchunks + kWarps - 1) / kWarps;
    const long long cap = 2LL * sm_count() < kMaxGrid ? 2LL * sm_count() : kMaxGrid;
    long long gq = bq, gk = bk;
    if (bq + bk > cap) {
        gq = (cap * nq + (nq + nk) / 2) / (nq + nk);
        if (nq && gq < 1) gq = 1;
        if (nk && gq > cap - 1) gq = cap - 1;
        gk = cap - gq;
        if (gq > bq) gq = bq;
        if (gk > bk) gk = bk;
    }
    a.split = static_cast<int>(gq);
    const int grid = static_cast<int>(gq + gk);
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(norm_bwd_kernel<T, D, kOrder, kAll>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kBwdSmem<T>);
    });
    if (err != cudaSuccess) return cuda_status(err);
    norm_bwd_kernel<T, D, kOrder, kAll><<<grid, kThreads, kBwdSmem<T>, stream>>>(a);
    const cp_status st = last_launch_status();
    if (st != CP_OK) return st;
    return launch(dw_sum_kernel, dim3(D / 32, 2), kSumWarps * 32, 0, stream, a.part, a.split, grid, D,
                  nq ? dwq : nullptr, nk ? dwk : nullptr);
}

struct Bwd {
    RowsArgs &a;
    float *dwq, *dwk;
    cudaStream_t stream;
    template <typename T, int D, int kOrder, bool kAll>
    cp_status operator()() const {
        return launch_bwd_typed<T, D, kOrder, kAll>(a, dwq, dwk, stream);
    }
};

cp_status rope_call(const void *q, const void *k, const int32_t *pos, int64_t C, int64_t B, int64_t s, int64_t N,
                    int64_t Nkv, int64_t D, int64_t qs, int64_t ks, cp_dtype dtype, const cp_rope *rope, void *qo,
                    void *ko, float sgn, cudaStream_t stream) {
    if (!rope) return CP_ERR_NULL;
    RowsArgs a;
    const cp_status st = fill_rows(&a, q, k, qo, ko, pos, C, B, s, N, Nkv, D, qs, ks, dtype, rope);
    if (st != CP_OK) return st;
    a.sgn = sgn;
    return run_fwd(a, false, D, dtype, rope, stream);
}

// Checks of the norm's weights and eps, shared by both directions.
cp_status check_norm(const void *wq, const void *wk, int64_t N, int64_t Nkv, cp_dtype w_dtype, float eps) {
    if ((N > 0 && !wq) || (Nkv > 0 && !wk)) return CP_ERR_NULL;
    if (!dtype_size(w_dtype)) return CP_ERR_DTYPE;
    if (!(std::isfinite(eps) && eps >= 0.f)) return CP_ERR_ARGUMENT;
    if (misaligned(wq) || misaligned(wk)) return CP_ERR_ALIGNMENT;
    return CP_OK;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" cp_status cp_rope_phases(const double *inv_freq, int64_t n, uint64_t *freqs) {
    if (!inv_freq || !freqs) return CP_ERR_NULL;
    if (n < 1 || n > 4096) return CP_ERR_SHAPE;
    for (int64_t i = 0; i < n; ++i)
        if (!(std::isfinite(inv_freq[i]) && std::fabs(inv_freq[i]) <= 6.2831853071795864769)) return CP_ERR_ARGUMENT;
    for (int64_t i = 0; i < n; ++i) {
        // turns per position, then its fraction in units of 2^-64 (a double holds 53 bits of
        // it, those of a negative frequency before its complement is taken)
        double t = std::fabs(inv_freq[i]) / 6.2831853071795864769;
        t -= std::floor(t);
        const double hi = std::floor(t * 4294967296.0);  // top 32 bits, exact
        const double lo = (t * 4294967296.0 - hi) * 4294967296.0;
        const uint64_t f = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::llrint(lo));
        freqs[i] = inv_freq[i] < 0.0 ? 0 - f : f;
    }
    return CP_OK;
}

extern "C" cp_status cp_rope_freqs(int64_t rot_dim, double base, cp_rope_scaling scaling, double factor,
                                   double original_len, uint64_t *freqs, float *amplitude) {
    if (!freqs || !amplitude) return CP_ERR_NULL;
    if (rot_dim < 2 || rot_dim > 8192 || rot_dim % 2) return CP_ERR_SHAPE;
    if (!(std::isfinite(base) && base >= 1.0)) return CP_ERR_ARGUMENT;
    if (scaling != CP_ROPE_PLAIN && scaling != CP_ROPE_LINEAR && scaling != CP_ROPE_BASE &&
        scaling != CP_ROPE_BY_PARTS)
        return CP_ERR_ARGUMENT;
    if (scaling != CP_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return CP_ERR_ARGUMENT;
    if (scaling == CP_ROPE_BASE && rot_dim < 4) return CP_ERR_SHAPE;
    if (scaling == CP_ROPE_BY_PARTS && !(std::isfinite(original_len) && original_len >= 1.0)) return CP_ERR_ARGUMENT;
    const double d = static_cast<double>(rot_dim);
    if (scaling == CP_ROPE_BASE) base *= std::pow(factor, d / (d - 2.0));
    if (!std::isfinite(base)) return CP_ERR_ARGUMENT;
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double theta = std::pow(base, -2.0 * static_cast<double>(i) / d);
        if (scaling == CP_ROPE_LINEAR) theta /= factor;
        if (scaling == CP_ROPE_BY_PARTS) {
            // pairs that turn more than 32 times over the original length keep their
            // frequency, those that turn less than once are interpolated, a ramp between
            const double turns = original_len * theta / 6.2831853071795864769;
            const double keep = std::fmin(1.0, std::fmax(0.0, (turns - 1.0) / 31.0));
            theta = theta * keep + theta / factor * (1.0 - keep);
        }
        const cp_status st = cp_rope_phases(&theta, 1, freqs + i);
        if (st != CP_OK) return st;
    }
    *amplitude = scaling == CP_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    return CP_OK;
}

extern "C" cp_status cp_rope_fwd(const void *q, const void *k, const int32_t *pos, int64_t C, int64_t B, int64_t s,
                                 int64_t N, int64_t Nkv, int64_t D, int64_t q_stride, int64_t k_stride,
                                 cp_dtype dtype, const cp_rope *rope, void *q_out, void *k_out, cudaStream_t stream) {
    return rope_call(q, k, pos, C, B, s, N, Nkv, D, q_stride, k_stride, dtype, rope, q_out, k_out, 1.f, stream);
}

extern "C" cp_status cp_rope_bwd(const void *dq_out, const void *dk_out, const int32_t *pos, int64_t C, int64_t B,
                                 int64_t s, int64_t N, int64_t Nkv, int64_t D, int64_t q_stride, int64_t k_stride,
                                 cp_dtype dtype, const cp_rope *rope, void *dq, void *dk, cudaStream_t stream) {
    return rope_call(dq_out, dk_out, pos, C, B, s, N, Nkv, D, q_stride, k_stride, dtype, rope, dq, dk, -1.f, stream);
}

extern "C" cp_status cp_qk_norm_rope_fwd(const void *q, const void *k, const void *wq, const void *wk,
                                         const int32_t *pos, int64_t C, int64_t B, int64_t s, int64_t N, int64_t Nkv,
                                         int64_t D, int64_t q_stride, int64_t k_stride, cp_dtype dtype,
                                         cp_dtype w_dtype, float eps, const cp_rope *rope, void *q_out, void *k_out,
                                         cudaStream_t stream) {
    RowsArgs a;
    cp_status st = fill_rows(&a, q, k, q_out, k_out, pos, C, B, s, N, Nkv, D, q_stride, k_stride, dtype, rope);
    if (st == CP_OK) st = check_norm(wq, wk, N, Nkv, w_dtype, eps);
    if (st != CP_OK) return st;
    a.w[0] = wq, a.w[1] = wk;
    a.w_bf16 = w_dtype == CP_BF16;
    a.eps = eps;
    return run_fwd(a, true, D, dtype, rope, stream);
}

extern "C" cp_status cp_qk_norm_rope_bwd_workspace_size(int64_t C, int64_t B, int64_t s, int64_t N, int64_t Nkv,
                                                        int64_t D, size_t *bytes) {
    if (!bytes) return CP_ERR_NULL;
    const cp_status st = check_sizes(C, B, s, N, Nkv, D);
    if (st != CP_OK) return st;
    *bytes = static_cast<size_t>(kMaxGrid) * static_cast<size_t>(D) * sizeof(float);
    return CP_OK;
}

extern "C" cp_status cp_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                         const void *wq, const void *wk, const int32_t *pos, int64_t C, int64_t B,
                                         int64_t s, int64_t N, int64_t Nkv, int64_t D, int64_t q_stride,
                                         int64_t k_stride, cp_dtype dtype, cp_dtype w_dtype, float eps,
                                         const cp_rope *rope, void *dq, void *dk, float *dwq, float *dwk,
                                         void *workspace, size_t ws_bytes, cudaStream_t stream) {
    RowsArgs a;
    cp_status st = fill_rows(&a, q, k, dq, dk, pos, C, B, s, N, Nkv, D, q_stride, k_stride, dtype, rope);
    if (st == CP_OK) st = check_norm(wq, wk, N, Nkv, w_dtype, eps);
    if (st != CP_OK) return st;
    if ((N && (!dq_out || !dwq)) || (Nkv && (!dk_out || !dwk))) return CP_ERR_NULL;
    if (misaligned(dq_out) || misaligned(dk_out) || (reinterpret_cast<uintptr_t>(dwq) & 3u) ||
        (reinterpret_cast<uintptr_t>(dwk) & 3u))
        return CP_ERR_ALIGNMENT;
    // the gradients come in dense; dq and dk may take their place (each value is
    // read by the thread that writes it) but not lie across them
    const size_t es = dtype_size(dtype);
    const Rows gq(dq_out, a.tokens, N * D, N, D, es), gk(dk_out, a.tokens, Nkv * D, Nkv, D, es);
    const Rows oq(dq, a.tokens, a.ys[0], N, D, es), ok(dk, a.tokens, a.ys[1], Nkv, D, es);
    const bool same_q = dq == dq_out && a.ys[0] == N * D, same_k = dk == dk_out && a.ys[1] == Nkv * D;
    if ((!same_q && oq.meets(gq)) || (!same_k && ok.meets(gk)) || oq.meets(gk) || ok.meets(gq))
        return CP_ERR_ARGUMENT;
    // one buffer for both sums would keep one of them
    const Rows wq_sum(dwq, 1, D, N ? 1 : 0, D, sizeof(float)), wk_sum(dwk, 1, D, Nkv ? 1 : 0, D, sizeof(float));
    if (wq_sum.meets(wk_sum)) return CP_ERR_ARGUMENT;
    size_t need = 0;
    cp_qk_norm_rope_bwd_workspace_size(C, B, s, N, Nkv, D, &need);
    if (!workspace || ws_bytes < need) return CP_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CP_ERR_ALIGNMENT;
    a.g[0] = dq_out, a.g[1] = dk_out;
    a.gs[0] = N * D, a.gs[1] = Nkv * D;
    a.w[0] = wq, a.w[1] = wk;
    a.w_bf16 = w_dtype == CP_BF16;
    a.eps = eps;
    a.part = static_cast<float *>(workspace);
    return dispatch(D, dtype, rope, Bwd{a, dwq, dwk, stream});
}
