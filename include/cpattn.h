/*
 * cpattn.h -- C ABI of libcpattn: blockwise causal attention with
 * log-sum-exp merging for ring / zigzag context parallelism, for C virtual
 * ranks held as buffers on ONE GB300 GPU (sm_103a).
 *
 * Source pages (cited by title and section):
 *   [OCP]   "On Context Parallelism": All-gather, All-to-all, Peer-to-peer
 *   [DAY74] "Context parallelism -- splitting the sequence across GPUs"
 *   [RING]  "Context Parallelism & Ring Attention"
 *   [HB]    "Context parallelism: Ring Attention and Ulysses"
 *   [APPF]  "Appendix F: Context Parallelism and MoE Parallel Folding"
 *
 * General conventions (all entry points):
 *   - Device pointers are raw CUDA device addresses owned by the caller; the
 *     library never allocates device memory on these paths and never frees
 *     caller memory.  Work that needs scratch takes a caller workspace.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream) unless
 *     stated otherwise; they return as soon as the work is enqueued.
 *   - Arguments are validated on the host BEFORE anything is enqueued; on a
 *     validation error nothing is launched and the call returns the status.
 *     No call aborts, throws or prints.
 *   - Tensors are dense, row-major, with the layouts given per call:
 *       sequence-sharded, rank-major: X_sh [C][B][s][N][D], s = S/C
 *       lse: [B][N][Sq] (rank-major shards: [C][B][N][s])
 *     ([OCP] Peer-to-peer / Forward: output [B,S/C,N,D], lse [B,N,S/C].)
 *   - Every device pointer must be 16-byte aligned; rows of N*D elements
 *     must be a multiple of 16 bytes.
 *   - Failures of a launch are reported as CP_ERR_CUDA (cudaGetLastError is
 *     read and cleared).  A kernel that gives up a bounded device-side wait
 *     records CP_ERR_DEVICE_TIMEOUT in a device status word, readable with
 *     cp_device_status().
 */
#ifndef CPATTN_H
#define CPATTN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum cp_status {
    CP_OK = 0,
    CP_ERR_NULL = 1,          /* a required pointer is NULL */
    CP_ERR_SHAPE = 2,         /* a size is <= 0 or out of the supported range */
    CP_ERR_DIVISIBILITY = 3,  /* S % 2C (zigzag), S % C, N % C, Nkv % C or N % Nkv */
    CP_ERR_DTYPE = 4,         /* unknown cp_dtype */
    CP_ERR_ALIGNMENT = 5,     /* pointer or row not 16-byte aligned */
    CP_ERR_WORKSPACE = 6,     /* workspace NULL or smaller than cp_ring_workspace_size */
    CP_ERR_UNSUPPORTED = 7,   /* e.g. D not in {64, 128} for attention */
    CP_ERR_CUDA = 8,          /* a CUDA runtime call or launch failed */
    CP_ERR_DEVICE_TIMEOUT = 9,/* a kernel gave up a bounded wait (see cp_device_status) */
    CP_ERR_ARGUMENT = 10,     /* any other invalid argument (scale, enum, event count) */
    CP_ERR_PAGE = 11          /* a page number, length or count in device memory is out of range
                                 (device status word only, see cp_device_status) */
} cp_status;

typedef enum cp_dtype { CP_BF16 = 0, CP_F32 = 1 } cp_dtype;
typedef enum cp_layout { CP_ZIGZAG = 0, CP_CONTIGUOUS = 1 } cp_layout;
typedef enum cp_dir { CP_SEQ_TO_HEAD = 0, CP_HEAD_TO_SEQ = 1 } cp_dir;
typedef enum cp_seq_order { CP_RANK_ORDER = 0, CP_GLOBAL_ORDER = 1 } cp_seq_order;
typedef enum cp_rope_order { CP_ROPE_HALF = 0, CP_ROPE_INTERLEAVED = 1 } cp_rope_order;
typedef enum cp_rope_scaling {
    CP_ROPE_PLAIN = 0,
    CP_ROPE_LINEAR = 1,
    CP_ROPE_BASE = 2,
    CP_ROPE_BY_PARTS = 3
} cp_rope_scaling;

/* Human-readable name of a status code (static string, never NULL). */
const char *cp_status_string(cp_status status);

/* Library version as "major.minor.patch" (static string). */
const char *cp_version(void);

/* Text of the most recent CUDA runtime error that made a call of this host
 * thread return CP_ERR_CUDA ("no error" if none); static string. */
const char *cp_last_cuda_error(void);

/*
 * cp_zigzag_shard -- split a full sequence into C rank-major shards.
 * [OCP] All-gather: S is cut into 2C chunks of t = S/(2C) tokens and rank r
 * owns [chunk r | chunk 2C-1-r] (layout CP_ZIGZAG; TE's "DualChunkSwap").
 * [RING] "The last remaining axis": rank r owns tokens [r*s, (r+1)*s)
 * (layout CP_CONTIGUOUS).
 *   x     : [B][S][N][D] of `dtype`, read only; memory of the current device, or pinned host
 *           memory mapped at the same address (cudaHostAlloc / cudaMallocHost /
 *           cudaHostRegister under unified addressing), which the kernel then
 *           reads across the host link (the host-to-device copy and the shard
 *           in one pass)
 *   x_sh  : device, [C][B][S/C][N][D] of `dtype`, written (must not overlap x)
 * Requires S % (2C) == 0 (zigzag) or S % C == 0 (contiguous), C >= 1.
 * Any other host memory (pageable, or pinned but not mapped at its host
 * address) is refused with CP_ERR_ARGUMENT before anything is launched.
 * The result is a bit-exact permutation of x.
 */
cp_status cp_zigzag_shard(const void *x, void *x_sh, int64_t B, int64_t S, int64_t N, int64_t D,
                          int C, cp_dtype dtype, cp_layout layout, cudaStream_t stream);

/*
 * cp_zigzag_unshard -- inverse of cp_zigzag_shard: gather the C shards back
 * into global sequence order ([OCP] All-gather: the rank-order result
 * [chunk 0, chunk 7, chunk 1, chunk 6, ...] reordered to sequence order).
 *   x_sh  : device, [C][B][S/C][N][D], read only
 *   x     : [B][S][N][D], written (must not overlap x_sh); current-device memory, or
 *           pinned host memory mapped at the same address (the kernel then
 *           writes across the host link: unshard and device-to-host copy in
 *           one pass); other host memory -> CP_ERR_ARGUMENT
 */
cp_status cp_zigzag_unshard(const void *x_sh, void *x, int64_t B, int64_t S, int64_t N, int64_t D,
                            int C, cp_dtype dtype, cp_layout layout, cudaStream_t stream);

/*
 * cp_zigzag_positions -- global position of every local token, int32 [C][S/C]:
 * zigzag: pos[r] = [r*t .. r*t+t-1] ++ [(2C-1-r)*t .. (2C-1-r)*t+t-1]
 * ([OCP] All-gather ownership; the ring's per-owner positions in
 * Peer-to-peer / Forward); contiguous: pos[r] = [r*s .. r*s+s-1].
 *   pos       : device (on_device != 0, written by a kernel on `stream`) or
 *               host (on_device == 0, written synchronously; stream unused)
 * Requires S <= INT32_MAX.
 */
cp_status cp_zigzag_positions(int32_t *pos, int64_t S, int C, cp_layout layout, int on_device,
                              cudaStream_t stream);

/*
 * cp_ulysses_relayout -- the Ulysses all-to-all as a local permutation of
 * rank-major buffers ([HB] "Ulysses" seq_to_head / head_to_seq; [OCP]
 * All-to-all; [APPF] eq. (96) [B,S/C,H,d_h] -> [B,S,H/C,d_h]).
 *   CP_SEQ_TO_HEAD: in [C][B][S/C][N][D] -> out [C][B][S][N/C][D] with
 *       out[r][b][j*s+u][h'][d] = in[j][b][u][r*N/C + h'][d]
 *     (rank r receives head group r from every shard, shards in rank order).
 *   CP_HEAD_TO_SEQ: the exact inverse (out and in swap roles).
 *   CP_GLOBAL_ORDER additionally puts the gathered sequence in global order
 *     (row j*s+u -> zigzag position of row u of rank j; [OCP] All-to-all:
 *     TE reorders the chunks into global order before attention).  Requires
 *     S % (2C) == 0.  CP_RANK_ORDER is the literal all-to-all.
 * Requires S % C == 0 and N % C == 0 (head divisibility, [OCP] All-to-all;
 * [HB] "Ulysses").  in and out must not overlap.  Bit-exact permutation.
 */
cp_status cp_ulysses_relayout(const void *in, void *out, int64_t B, int64_t S, int64_t N, int64_t D,
                              int C, cp_dtype dtype, cp_dir dir, cp_seq_order order,
                              cudaStream_t stream);

/*
 * cp_attn_partial -- partial causal attention with explicit positions,
 * returning the normalised output and the per-row log-sum-exp.
 * [OCP] Peer-to-peer / Forward (attention(q, k, v, q_positions,
 * kv_positions, scale) -> tile_output, tile_lse); [HB] cp_common.py;
 * [DAY74] the causal softmax formula.  For each (b, h, i):
 *   visible keys V(i) = { j : k_pos[j] <= q_pos[i] }
 *   s_j = scale * <q_i, k_j>,  lse_i = ln sum_{j in V(i)} e^{s_j}
 *   o_i = sum_{j in V(i)} e^{s_j - lse_i} v_j
 *   a row with no visible key gets lse = -inf and o = 0.
 *   q      : device bf16 [B][Sq][N][D]
 *   k, v   : device bf16 [B][Sk][Nkv][D]; query head h reads KV head h/(N/Nkv)
 *   q_pos  : device int32 [Sq];  k_pos : device int32 [Sk] (any values)
 *   o      : device fp32 [B][Sq][N][D], written; 32-byte aligned
 *   lse    : device fp32 [B][N][Sq], written (natural log)
 * Requires D in {64, 128}, N % Nkv == 0, scale finite and > 0.  Runs on the
 * tensor cores (bf16 products, fp32 accumulation and softmax).
 * Work plan: the kernel starts from a plan of its launch (per-tile position
 * ranges, per-block tile counts, the order of work items).  It is built in
 * shared memory when ceil(Sq/128) + ceil(Sk/128) <= 2048 and
 * ceil(Sq/256) <= 1024; beyond that it is built in device memory the caller
 * provides: call cp_attn_partial_ws with a workspace of
 * cp_attn_workspace_size bytes (cp_attn_partial then returns
 * CP_ERR_WORKSPACE).
 */
cp_status cp_attn_partial(const void *q, const void *k, const void *v, const int32_t *q_pos,
                          const int32_t *k_pos, int64_t B, int64_t Sq, int64_t Sk, int64_t N,
                          int64_t Nkv, int64_t D, float scale, float *o, float *lse,
                          cudaStream_t stream);

/*
 * cp_attn_workspace_size / cp_attn_partial_ws -- cp_attn_partial with a
 * caller workspace for the work plan, for any sequence length.
 *   *bytes receives the workspace size for these sizes (0 when the plan fits
 *   in shared memory; then workspace may be NULL).  Host only.
 *   workspace : device, >= cp_attn_workspace_size bytes, 256-byte aligned;
 *               overwritten by the call (stream-ordered), not read back.
 * Everything else as cp_attn_partial.
 */
cp_status cp_attn_workspace_size(int64_t B, int64_t Sq, int64_t Sk, int64_t N, int64_t Nkv, int64_t D,
                                 size_t *bytes);
cp_status cp_attn_partial_ws(const void *q, const void *k, const void *v, const int32_t *q_pos,
                             const int32_t *k_pos, int64_t B, int64_t Sq, int64_t Sk, int64_t N,
                             int64_t Nkv, int64_t D, float scale, float *o, float *lse, void *workspace,
                             size_t ws_bytes, cudaStream_t stream);

/*
 * cp_attn_f32_workspace_size / cp_attn_partial_f32 -- cp_attn_partial for fp32
 * inputs with the tensor cores in tf32 (tcgen05.mma kind::tf32, fp32
 * accumulation).  q, k, v and P are rounded to the nearest tf32 value (10-bit
 * mantissa, ties away from zero) before they enter the tensor cores: q and k
 * by a pass into the workspace, v in its transpose, P in the softmax.
 * Same arguments, result and conventions as cp_attn_partial except:
 *   q : device fp32 [B][Sq][N][D]; k, v : device fp32 [B][Sk][Nkv][D]
 *   workspace : device, >= cp_attn_f32_workspace_size(B, Sq, Sk, N, Nkv, D)
 *               bytes, 256-byte aligned (rounded q and k, v transposed for
 *               the K-major operand and, when ceil(Sk/64) + ceil(Sq/128) >
 *               2048 or ceil(Sq/128) > 1024, the launch's work plan)
 */
cp_status cp_attn_f32_workspace_size(int64_t B, int64_t Sq, int64_t Sk, int64_t N, int64_t Nkv, int64_t D,
                                     size_t *bytes);
cp_status cp_attn_partial_f32(const float *q, const float *k, const float *v, const int32_t *q_pos,
                              const int32_t *k_pos, int64_t B, int64_t Sq, int64_t Sk, int64_t N, int64_t Nkv,
                              int64_t D, float scale, float *o, float *lse, void *workspace, size_t ws_bytes,
                              cudaStream_t stream);

/*
 * cp_lse_merge -- merge a completed partial into an accumulator, in place.
 * [OCP] Peer-to-peer / Forward, the tile merge:
 *   lse = logaddexp(lse_acc, lse_tile)
 *   o   = e^{lse_acc - lse} * o_acc + e^{lse_tile - lse} * o_tile
 * ([HB] "Ring Attention" gives the same two formulas.)  A row whose
 * lse_tile is -inf is left untouched; a row whose lse_acc is -inf takes the
 * tile's values.
 *   o_acc, lse_acc   : device fp32 [B][Sq][N][D] / [B][N][Sq], read+written
 *   o_tile, lse_tile : device fp32, same shapes, read only
 */
cp_status cp_lse_merge(float *o_acc, float *lse_acc, const float *o_tile, const float *lse_tile,
                       int64_t B, int64_t Sq, int64_t N, int64_t D, cudaStream_t stream);

/* Ring options (bit set, argument `flags` of the ring calls). */
#define CP_RING_PREFETCH 1    /* emulate the ring exchange by side-stream K/V copies */
#define CP_RING_FUSED_MERGE 2 /* merge each step's partial in the attention epilogue */
#define CP_RING_TF32 4        /* fp32 q, k, v; tensor cores in tf32 (not with the other two flags) */

/*
 * cp_ring_workspace_size -- bytes of device workspace cp_ring_attention_fwd
 * needs for these sizes and flags: the per-step partial (fp32 o and lse for
 * all C ranks; not with CP_RING_FUSED_MERGE), an fp32 accumulator when o_dtype
 * is CP_BF16, with CP_RING_PREFETCH two K/V rotation buffers, and for long
 * shards (C * (ceil((S/C)/128) * 2) > 2048 position tables, or more than
 * 1024 query blocks in a step) the attention launches' work plan.  Host
 * only; *bytes is written on success.
 */
cp_status cp_ring_workspace_size(int64_t B, int64_t S, int64_t N, int64_t Nkv, int64_t D, int C,
                                 int flags, cp_dtype o_dtype, size_t *bytes);

/*
 * cp_ring_attention_fwd -- ring (P2P) context-parallel attention forward for
 * C virtual ranks resident on this GPU.  [OCP] Peer-to-peer / Forward;
 * [RING] "The ring"; [HB] "Ring Attention".  For step = 0 .. C-1 every rank
 * r attends its queries to the K/V block of owner (r - step) mod C (with
 * both sides' positions) and merges the partial into its running (o, lse);
 * step 0 writes the accumulator directly.  All C ranks of a step run in one
 * launch (zigzag makes their work equal, [RING] "The zigzag fix").
 *   q_sh          : device bf16 [C][B][S/C][N][D]
 *   k_sh, v_sh    : device bf16 [C][B][S/C][Nkv][D]
 *   pos           : device int32 [C][S/C] global positions (cp_zigzag_positions)
 *   layout        : selects the divisibility rule only (S % 2C for zigzag,
 *                   S % C for contiguous); masks come from `pos`
 *   flags         : bit set of
 *                   CP_RING_PREFETCH -- the ring exchange is emulated by
 *                     device copies of the next step's K/V on a second
 *                     stream, overlapped with the current step and ordered
 *                     by events (without it: zero copy, each step reads the
 *                     owner's resident block);
 *                   CP_RING_FUSED_MERGE -- steps >= 1 merge their partial
 *                     into (o, lse) inside the attention epilogue instead of
 *                     writing it and launching cp_lse_merge's kernel
 *   o_sh          : device [C][B][S/C][N][D] of o_dtype (CP_F32 or CP_BF16);
 *                   32-byte aligned when o_dtype is CP_F32
 *   lse_sh        : device fp32 [C][B][N][S/C]
 *   workspace     : device, >= cp_ring_workspace_size(...) bytes, 256-byte
 *                   aligned, caller-owned, contents need not be initialised
 * Same attention restrictions as cp_attn_partial.
 */
cp_status cp_ring_attention_fwd(const void *q_sh, const void *k_sh, const void *v_sh,
                                const int32_t *pos, int64_t B, int64_t S, int64_t N, int64_t Nkv,
                                int64_t D, int C, float scale, cp_layout layout, int flags,
                                void *o_sh, cp_dtype o_dtype, float *lse_sh, void *workspace,
                                size_t ws_bytes, cudaStream_t stream);

/*
 * cp_ring_attention_fwd_traced -- cp_ring_attention_fwd that also records
 * CUDA events on `stream` around every kernel it launches, for timing:
 *   events[4*step + 0], events[4*step + 1] : before / after the attention
 *                                            launch of `step`
 *   events[4*step + 2], events[4*step + 3] : before / after the merge launch
 *                                            of `step` (recorded back to
 *                                            back for step 0 and with
 *                                            CP_RING_FUSED_MERGE)
 * n_events must be >= 4*C; events are caller-created (cudaEventCreate).
 */
cp_status cp_ring_attention_fwd_traced(const void *q_sh, const void *k_sh, const void *v_sh,
                                       const int32_t *pos, int64_t B, int64_t S, int64_t N,
                                       int64_t Nkv, int64_t D, int C, float scale,
                                       cp_layout layout, int flags, void *o_sh,
                                       cp_dtype o_dtype, float *lse_sh, void *workspace,
                                       size_t ws_bytes, cudaStream_t stream,
                                       cudaEvent_t const *events, int n_events);

/*
 * cp_allgather_workspace_size / cp_allgather_attention_fwd -- all-gather
 * context-parallel attention forward for C virtual ranks on this GPU.
 * [OCP] All-gather / Forward: each rank keeps its local queries, K and V are
 * gathered from every rank and reordered to global sequence order, and each
 * rank's queries attend to the full sequence (query positions `pos`, key
 * positions 0..S-1).  Here the gather is cp_zigzag_unshard of the resident
 * shards into the workspace, and all C ranks share one launch.
 *   q_sh, k_sh, v_sh, pos, layout : as for cp_ring_attention_fwd
 *   o_sh   : device fp32 [C][B][S/C][N][D] (32-byte aligned), written
 *   lse_sh : device fp32 [C][B][N][S/C], written
 *   workspace : device, >= cp_allgather_workspace_size bytes (the gathered
 *               K and V, bf16 [B][S][Nkv][D] each, and S int32 positions),
 *               256-byte aligned
 * The result equals cp_ring_attention_fwd's (same partial kernel, one
 * partial instead of C merged ones).
 */
cp_status cp_allgather_workspace_size(int64_t B, int64_t S, int64_t N, int64_t Nkv, int64_t D, int C,
                                      size_t *bytes);
cp_status cp_allgather_attention_fwd(const void *q_sh, const void *k_sh, const void *v_sh,
                                     const int32_t *pos, int64_t B, int64_t S, int64_t N, int64_t Nkv,
                                     int64_t D, int C, float scale, cp_layout layout, float *o_sh,
                                     float *lse_sh, void *workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * cp_ulysses_workspace_size / cp_ulysses_attention_fwd -- all-to-all
 * (Ulysses) context-parallel attention forward for C virtual ranks.
 * [OCP] All-to-all; [HB] "Ulysses": q, k, v are relaid from sequence
 * sharding to head sharding (cp_ulysses_relayout, global sequence order),
 * each head-group rank computes causal attention over the whole sequence for
 * its N/C heads, and the output is relaid back to sequence sharding.
 *   q_sh : device bf16 [C][B][S/C][N][D]; k_sh, v_sh : [C][B][S/C][Nkv][D]
 *          (sharded with `layout`; N % C == 0 and Nkv % C == 0)
 *   o_sh : device fp32 [C][B][S/C][N][D], written
 *   lse_h: device fp32 [C][B][N/C][S], written: the log-sum-exp of head
 *          r*N/C + h' for global query position i is lse_h[r][b][h'][i]
 *          (head-sharded layout, global order, as the attention computes it)
 *   workspace : device, >= cp_ulysses_workspace_size bytes, 256-byte aligned
 */
cp_status cp_ulysses_workspace_size(int64_t B, int64_t S, int64_t N, int64_t Nkv, int64_t D, int C,
                                    size_t *bytes);
cp_status cp_ulysses_attention_fwd(const void *q_sh, const void *k_sh, const void *v_sh, int64_t B,
                                   int64_t S, int64_t N, int64_t Nkv, int64_t D, int C, float scale,
                                   cp_layout layout, float *o_sh, float *lse_h, void *workspace,
                                   size_t ws_bytes, cudaStream_t stream);

/*
 * cp_mesh_workspace_size / cp_mesh_attention_fwd -- A2A x P2P context-parallel
 * attention forward on a two-dimensional mesh of C = A * R virtual ranks.
 * [OCP] "Peer-to-peer + All-to-all": rank c belongs to A2A group c / A (ranks
 * g*A .. g*A+A-1) and to P2P group c % A (ranks a, A+a, 2A+a, ...).  Inside
 * each A2A group q, k, v go from sequence sharding to head sharding (N/A
 * heads; the group's A shards concatenated in rank order, S/R positions), each
 * P2P group runs the ring (as cp_ring_attention_fwd) over its R ranks with
 * those concatenated positions, and the output returns to sequence sharding.
 * A = 1 is the ring; R = 1 is Ulysses in rank order.
 *   q_sh : device bf16 [C][B][S/C][N][D]; k_sh, v_sh : [C][B][S/C][Nkv][D]
 *   pos  : device int32 [C][S/C], the global positions of each shard (for
 *          example cp_zigzag_positions with C and `layout`)
 *   A, R : A2A and P2P group sizes, 1 <= A*R <= 64; N % A == 0, Nkv % A == 0;
 *          S % (2C) == 0 for CP_ZIGZAG, S % C == 0 for CP_CONTIGUOUS
 *   flags: ring options (CP_RING_PREFETCH, CP_RING_FUSED_MERGE)
 *   o_sh : device fp32 [C][B][S/C][N][D], written
 *   lse_h: device fp32 [R][A][B][N/A][S/R], written: P2P rank g, A2A index a,
 *          head a*N/A + h', row a'*S/C + u = query u of shard g*A + a'
 *   workspace : device, >= cp_mesh_workspace_size bytes, 256-byte aligned
 *          (relaid q, k, v, the fp32 head-sharded output and the ring's own
 *          workspace)
 * Everything is validated before anything is enqueued.
 */
cp_status cp_mesh_workspace_size(int64_t B, int64_t S, int64_t N, int64_t Nkv, int64_t D, int A, int R,
                                 int flags, size_t *bytes);
cp_status cp_mesh_attention_fwd(const void *q_sh, const void *k_sh, const void *v_sh, const int32_t *pos,
                                int64_t B, int64_t S, int64_t N, int64_t Nkv, int64_t D, int A, int R,
                                float scale, cp_layout layout, int flags, float *o_sh, float *lse_h,
                                void *workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * cp_attn_bwd_workspace_size / cp_attn_bwd_partial -- backward of one
 * partial attention ("tile backward"): [OCP] Peer-to-peer / Backward,
 * attention_tile_backward(q, k, v, output, grad_output, lse, q_positions,
 * kv_positions, scale) -> (dq, dk, dv).  It takes the FINAL output and lse of
 * the attention the tile belongs to, so p_ij = e^{scale <q_i,k_j> - lse_i}
 * over visible pairs (k_pos[j] <= q_pos[i]), and
 *   dv_j = sum_i p_ij dO_i,  ds_ij = p_ij (<dO_i, v_j> - <dO_i, o_i>),
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
 * (the chain rule of the forward; a KV head's gradients sum over its query
 * heads).  P and dS enter the tensor cores as bf16; accumulation is fp32.
 *   q, dout : device bf16 [B][Sq][N][D]; k, v : device bf16 [B][Sk][Nkv][D]
 *   o       : device fp32 [B][Sq][N][D], the final output
 *   lse     : device fp32 [B][N][Sq], the final natural-log log-sum-exp
 *             (-inf: the row sees nothing and contributes nothing)
 *   q_pos, k_pos : device int32 [Sq], [Sk]
 *   D in {64, 128}; N % Nkv == 0; scale finite and > 0
 *   dq : device fp32 [B][Sq][N][D]; dk, dv : device fp32 [B][Sk][Nkv][D];
 *        32-byte aligned; written, or added to when accumulate != 0
 *   workspace : device, >= cp_attn_bwd_workspace_size(B, Sq, Sk, N) bytes,
 *        256-byte aligned (per-row statistics and, when ceil(Sk/128) +
 *        ceil(Sq/128) > 2048 or either exceeds 1024, the kernels' work plans)
 * Other pointers 16-byte aligned.
 */
cp_status cp_attn_bwd_workspace_size(int64_t B, int64_t Sq, int64_t Sk, int64_t N, size_t *bytes);
cp_status cp_attn_bwd_partial(const void *q, const void *k, const void *v, const float *o, const void *dout,
                              const float *lse, const int32_t *q_pos, const int32_t *k_pos, int64_t B,
                              int64_t Sq, int64_t Sk, int64_t N, int64_t Nkv, int64_t D, float scale, float *dq,
                              float *dk, float *dv, int accumulate, void *workspace, size_t ws_bytes,
                              cudaStream_t stream);

/*
 * cp_ring_bwd_workspace_size / cp_ring_attention_bwd -- ring (P2P)
 * context-parallel attention backward for C virtual ranks.
 * [OCP] Peer-to-peer / Backward: at step = 0 .. C-1 rank r holds the K/V
 * block of owner (r - step) mod C and its travelling dK/dV accumulators; the
 * tile backward of rank r's queries against it (with rank r's final output
 * and lse from the forward) adds to rank r's dq and to the block's dk/dv,
 * which are back on their owner after the full rotation.  On one GPU the
 * travelling accumulators are the owners' own dk_sh / dv_sh; every step is one
 * dK/dV launch and one dQ launch over all C ranks.
 *   q_sh, do_sh : device bf16 [C][B][S/C][N][D]; k_sh, v_sh : [C][B][S/C][Nkv][D]
 *   o_sh  : device fp32 [C][B][S/C][N][D], lse_sh : fp32 [C][B][N][S/C]
 *           (cp_ring_attention_fwd's outputs with o_dtype CP_F32)
 *   pos   : device int32 [C][S/C]
 *   dq_sh : device fp32 [C][B][S/C][N][D]; dk_sh, dv_sh : [C][B][S/C][Nkv][D];
 *           written (32-byte aligned)
 *   workspace : device, >= cp_ring_bwd_workspace_size bytes, 256-byte aligned
 * Everything is validated before anything is enqueued.
 */
cp_status cp_ring_bwd_workspace_size(int64_t B, int64_t S, int64_t N, int C, size_t *bytes);
cp_status cp_ring_attention_bwd(const void *q_sh, const void *k_sh, const void *v_sh, const float *o_sh,
                                const float *lse_sh, const void *do_sh, const int32_t *pos, int64_t B, int64_t S,
                                int64_t N, int64_t Nkv, int64_t D, int C, float scale, cp_layout layout,
                                float *dq_sh, float *dk_sh, float *dv_sh, void *workspace, size_t ws_bytes,
                                cudaStream_t stream);

/*
 * cp_rope -- a rotation of head rows by their token's position.  The first
 * rot_dim values of a row of D form rot_dim/2 pairs, which at position t become
 *   a' = A (a cos t theta_i - b sin t theta_i)
 *   b' = A (b cos t theta_i + a sin t theta_i)
 * and the other D - rot_dim values stay as they are.
 *   freqs     : device uint64 [rot_dim/2], turns per position in 64-bit fixed
 *               point, theta_i / (2 pi) * 2^64 modulo 2^64 (cp_rope_freqs, cp_rope_phases,
 *               copied to the device by the caller and kept as long as calls use
 *               it).  The fraction of a turn of pos * freqs[i] is formed exactly at any
 *               position; freqs[i] comes from an fp64 quotient, so the angle is off by
 *               at most |pos| (theta_i 2^-52 + 2^-62) radians (under 3e-7 measured at 2^31)
 *   order     : CP_ROPE_HALF pairs value i with value i + rot_dim/2,
 *               CP_ROPE_INTERLEAVED pairs 2i with 2i + 1
 *   rot_dim   : even, 2 .. D; a multiple of 16 for CP_ROPE_HALF
 *               (CP_ERR_UNSUPPORTED else)
 *   amplitude : A, finite (1 unless the scaling says otherwise)
 * The struct itself is read on the host during the call.
 */
typedef struct cp_rope {
    const uint64_t *freqs;
    int64_t rot_dim;
    cp_rope_order order;
    float amplitude;
} cp_rope;

/*
 * cp_rope_freqs / cp_rope_phases -- frequencies of a rotation, into host memory.
 * cp_rope_freqs: theta_i = base^(-2i/rot_dim), i < rot_dim/2, and for a context
 * `factor` (>= 1) times longer than the one trained on
 *   CP_ROPE_PLAIN    : as they are (factor and original_len are not read)
 *   CP_ROPE_LINEAR   : theta_i / factor (positions interpolated)
 *   CP_ROPE_BASE     : base * factor^(rot_dim/(rot_dim-2)) in the place of base
 *   CP_ROPE_BY_PARTS : theta_i / factor for pairs that turn less than once over
 *                      original_len positions, theta_i for those that turn more
 *                      than 32 times, a linear ramp over the number of turns
 *                      between; *amplitude = 0.1 ln(factor) + 1
 * *amplitude is 1 for the others.  cp_rope_phases: any other rule, from n
 * angular frequencies in radians per position (each finite, at most 2 pi in
 * size, n <= 4096).  Both compute in fp64.
 */
cp_status cp_rope_freqs(int64_t rot_dim, double base, cp_rope_scaling scaling, double factor, double original_len,
                        uint64_t *freqs, float *amplitude);
cp_status cp_rope_phases(const double *inv_freq, int64_t n, uint64_t *freqs);

/*
 * cp_rope_fwd / cp_rope_bwd -- rotate the rows of q and k by their positions
 * before the attention ([OCP] Introduction: apply_rope(q, k, local_positions)),
 * and rotate gradients back (dx = A R(-t) dy).
 *   q, k  : device, rows of N and Nkv heads of D values (`dtype`), token
 *           ((c*B + b)*s + i) at element offset token * q_stride (k_stride);
 *           dense shards [C][B][s][N][D] have q_stride = N*D, q and k inside
 *           the rows of a fused projection have its row length.  Either may be
 *           left out (NULL with N = 0 or Nkv = 0).
 *   pos   : device int32 [C][s], the position of token (c, b, i) is pos[c][i]
 *           (cp_zigzag_positions for shards; C = B = 1: one per token); any value
 *   q_out, k_out : device, `dtype`; written dense, or in place where the
 *           pointer equals q (k), then with its stride.  Any other overlap with
 *           q, k or one another is refused (CP_ERR_ARGUMENT).
 *   cp_rope_bwd takes the gradients of the rotated rows and writes those of
 *   the unrotated ones; the same arguments.
 * Strides are multiples of 16 bytes; pointers 16-byte aligned (pos 4); D in
 * {64, 128}.  Computed in fp32 and rounded once.
 */
cp_status cp_rope_fwd(const void *q, const void *k, const int32_t *pos, int64_t C, int64_t B, int64_t s, int64_t N,
                      int64_t Nkv, int64_t D, int64_t q_stride, int64_t k_stride, cp_dtype dtype,
                      const cp_rope *rope, void *q_out, void *k_out, cudaStream_t stream);
cp_status cp_rope_bwd(const void *dq_out, const void *dk_out, const int32_t *pos, int64_t C, int64_t B, int64_t s,
                      int64_t N, int64_t Nkv, int64_t D, int64_t q_stride, int64_t k_stride, cp_dtype dtype,
                      const cp_rope *rope, void *dq, void *dk, cudaStream_t stream);

/*
 * cp_qk_norm_rope_fwd -- the root-mean-square norm of every head row of q and
 * k, its weights, and the rotation of cp_rope_fwd in the same pass:
 *   y = A R(t) (w . x r),  r = (mean_j x_j^2 + eps)^(-1/2)
 *   wq, wk  : device [D] of w_dtype, one weight vector for all heads of q (k)
 *   eps     : finite, >= 0
 *   rope    : NULL for the norm alone (pos is not read then)
 * The mean square is formed in fp32: a row of values above 1.6e18 overflows it
 * (its r is 0), and with eps = 0 a row below 1e-19 loses bits of it, below 1e-23 all (its r
 * is infinite).
 * Everything else as for cp_rope_fwd.
 */
cp_status cp_qk_norm_rope_fwd(const void *q, const void *k, const void *wq, const void *wk, const int32_t *pos,
                              int64_t C, int64_t B, int64_t s, int64_t N, int64_t Nkv, int64_t D, int64_t q_stride,
                              int64_t k_stride, cp_dtype dtype, cp_dtype w_dtype, float eps, const cp_rope *rope,
                              void *q_out, void *k_out, cudaStream_t stream);

/*
 * cp_qk_norm_rope_bwd -- gradients of cp_qk_norm_rope_fwd.  With g = A R(-t) dy
 * and xh = x r:
 *   u = w . g,  dx = r (u - xh mean_j(u_j xh_j)),  dw = sum over rows of g . xh
 *   dq_out, dk_out : device, `dtype`, dense: gradients of q_out and k_out
 *   q, k           : the inputs of the forward call, with their strides
 *   dq, dk         : device, `dtype`, written dense, or in place of q (k) with its stride, or in
 *                    place of dq_out (dk_out)
 *   dwq, dwk       : device fp32 [D], written (sums in fp32, in a fixed order: the same
 *                    from run to run); apart from one another (CP_ERR_ARGUMENT else), also where wq
 *                    and wk are one vector, whose gradient is their sum
 *   workspace      : device, >= cp_qk_norm_rope_bwd_workspace_size bytes,
 *                    256-byte aligned; overwritten (stream-ordered), not read back
 */
cp_status cp_qk_norm_rope_bwd_workspace_size(int64_t C, int64_t B, int64_t s, int64_t N, int64_t Nkv, int64_t D,
                                             size_t *bytes);
cp_status cp_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k, const void *wq,
                              const void *wk, const int32_t *pos, int64_t C, int64_t B, int64_t s, int64_t N,
                              int64_t Nkv, int64_t D, int64_t q_stride, int64_t k_stride, cp_dtype dtype,
                              cp_dtype w_dtype, float eps, const cp_rope *rope, void *dq, void *dk, float *dwq,
                              float *dwk, void *workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * cp_cache_append -- put the keys and values of new tokens into a paged cache,
 * with the keys normed and rotated on the way, and the queries of the same
 * tokens in the same launch.
 *   k, v    : device rows of Nkv heads of D values (`dtype`), token r at element offset
 *             r * k_stride (v_stride); q the same with N heads (NULL with N = 0)
 *   cu_new  : device int32 [B+1], non-decreasing from 0: rows cu_new[b] ..
 *             cu_new[b+1]-1 are the n_b new tokens of sequence b (n_b may be 0);
 *             rows from cu_new[B] up to R are padding, and neither they nor
 *             their part of q_out are touched
 *   kv_len  : device int32 [B], tokens of each sequence in the cache AFTER the
 *             call: new token j of sequence b gets index i = kv_len[b] - n_b + j,
 *             goes to slot i % page_size of page table[b][i / page_size], and
 *             has position pos_base + i (pos_base: the length of a shared
 *             prefix that stands before every sequence, 0 without one)
 *   k_cache, v_cache : device bf16 [n_pages][page_size][Nkv][D]
 *   table   : device int32 [B][max_pages]; only the entries that the new tokens fall into are
 *             read.  Two new tokens must not share a slot.
 *   wq, wk  : device [D] of w_dtype, or NULL: no norm of q (k); eps as above
 *   rope    : NULL for no rotation
 *   q_out   : device bf16 [R][N][D], the normed and rotated queries (may be q itself when q is
 *             dense bf16; any other overlap with the rows or the caches, and of the caches
 *             with one another, is refused: CP_ERR_ARGUMENT)
 * The prefix itself is appended as a sequence with its own table.
 * page_size in {16, 32, 64, 128, 256} and D in {64, 128} (else
 * CP_ERR_UNSUPPORTED); R >= 1; B <= 4096; n_pages * page_size and max_pages *
 * page_size at most 2^31 - 256.  cu_new, kv_len and table are read on the device: a token
 * whose index or page number is out of range is skipped and the device status
 * word becomes CP_ERR_PAGE.
 */
cp_status cp_cache_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                          int64_t v_stride, cp_dtype dtype, int64_t R, int64_t N, int64_t Nkv, int64_t D,
                          const void *wq, const void *wk, cp_dtype w_dtype, float eps, const cp_rope *rope,
                          int64_t pos_base, void *k_cache, void *v_cache, int64_t n_pages, int64_t page_size,
                          const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                          const int32_t *kv_len, void *q_out, cudaStream_t stream);

/*
 * cp_prefix_attn_workspace_size / cp_prefix_attn_fwd -- attention of a batch of
 * sequences that share a prefix, over a paged cache filled by cp_cache_append.
 * Query row r (a new token of sequence b with own index i) sees the
 * prefix_len keys of the prefix and its own sequence's keys 0 .. i:
 *   s_j = scale <q_r, k_j>,  lse_r = ln sum_j e^{s_j},  o_r = sum_j e^{s_j - lse_r} v_j
 * The prefix is read once for all rows ([DAY74] How do partial softmax results
 * combine?; the two parts join as in cp_lse_merge).  One call serves single
 * tokens, drafts and prompts, mixed in one batch.
 *   q       : device bf16 [R][N][D], dense; query head h reads KV head h/(N/Nkv)
 *   k_cache, v_cache : device bf16 [n_pages][page_size][Nkv][D]
 *   prefix_pages : device int32 [ceil(prefix_len/page_size)], the prefix's pages
 *             (may be NULL when prefix_len is 0)
 *   table, cu_new, kv_len, B, max_pages : as for cp_cache_append, after it: new token j of
 *             sequence b has own index kv_len[b] - n_b + j (a negative index sees
 *             the prefix alone)
 *   max_new : about the largest n_b, 1 .. R: chooses the tiles only, every n_b is right
 *   o       : device [R][N][D] of o_dtype; a row that sees no key gets o = 0
 *   lse     : device fp32 [N][R] (cp_lse_merge's layout for B = 1), -inf for such a row
 *             Rows from cu_new[B] to R are padding: neither o nor lse is touched there.
 *   workspace : device, >= cp_prefix_attn_workspace_size bytes, 256-byte
 *             aligned; overwritten (stream-ordered), not read back.  Calls that
 *             may overlap need one each.
 * Products are bf16 with fp32 accumulation; the softmax weights are rounded to
 * bf16 before the second product (off by 2^-8 of themselves at most, whatever
 * o_dtype is), lse is not.  Keys that no row of the call sees are not read into
 * a result whatever they hold; a NaN or infinity in a V row that some row sees
 * may reach other rows of its sequence.
 * D in {64, 128}, page_size in {16, 32, 64, 128, 256}; N % Nkv == 0; scale
 * finite and > 0; prefix_len at most 2^31 - 256; R >= 1 (a step without new tokens
 * makes no call).  Its launches overlap one another and the end of the kernel before them on
 * the stream, never one that the caller puts behind.  The lists are read on the
 * device: a page number, length or count out of range sets the device status word to
 * CP_ERR_PAGE, is never followed, and leaves its rows' results unspecified.
 */
cp_status cp_prefix_attn_workspace_size(int64_t R, int64_t B, int64_t max_new, int64_t prefix_len, int64_t N,
                                        int64_t Nkv, int64_t D, int64_t page_size, int64_t max_pages, size_t *bytes);
cp_status cp_prefix_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                             int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                             const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                             const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv, int64_t D,
                             float scale, void *o, cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                             cudaStream_t stream);

/*
 * cp_cache_plan -- the pages and slots of a step, from the sequences' lengths (no counterpart on the
 * pages).  Sequence b has pages for kv_had[b] tokens, of which the first kv_keep[b] stay (all, without
 * rejected drafts; none, when it has ended), and gets n_new[b] new ones:
 *   kv_len[b] = kv_keep[b] + n_new[b], cu_new = running sum of n_new.
 * The pages behind ceil(kv_len / page_size) are pushed on the stack of free pages, in the order of (sequence,
 * index); then the missing ones are popped in the same order and written into the table.  Row r of sequence
 * b (r = cu_new[b] + j) gets own index i = kv_keep[b] + j,
 *   slots[r] = table[b][i / page_size] * page_size + i % page_size,  pos[r] = pos_base + i;
 * rows from cu_new[B] up to R get slot -1 and position 0.  The results feed cp_cache_append(_at) and the
 * attention calls as they are; the next step's kv_had is this step's kv_len.
 *   kv_had, kv_keep, n_new : device int32 [B]
 *   table      : device int32 [B][max_pages]; new pages are written, the others read
 *   free_pages : device int32 [n_pages], the stack; n_free[0] (device int32) of them lie on it.  Entries
 *                behind the new top are unspecified.
 *   R          : rows of slots and pos, at least the sum of n_new
 *   kv_len     : device int32 [B], may be kv_had or kv_keep;  cu_new : device int32 [B+1]
 *   slots, pos : device int32 [R]
 *   n_free_out : device int32 [2], may be n_free: {free pages, 0}; where too few pages are free, {free pages,
 *                pages lacking}, and nothing is handed out or given back: cu_new is 0, every slot -1, kv_len is
 *                kv_had, stack and table stay
 * All lists apart from one another otherwise (CP_ERR_ARGUMENT else).  A count below zero, kv_keep over
 * kv_had, a length past the table, a new position past 32 bits, more than R new tokens or a stack that does not fit
 * n_pages sets the device status word to CP_ERR_PAGE and hands nothing out (n_free_out[1] = -1).  A page number out of
 * range that the step meets, in the table or on the stack, sets the status word too, but the step goes on: its rows
 * get slot -1, a page that is given back or taken moves as it is, and n_free_out[1] stays 0.  Sizes as for
 * cp_cache_append.
 * This call and the four below let a kernel that follows them with programmatic stream serialization start before
 * they end: as behind any such kernel it waits for them itself (cudaGridDependencySynchronize) before it touches what
 * they read or write.  Kernels launched without it are behind them as always.
 */
cp_status cp_cache_plan(const int32_t *kv_had, const int32_t *kv_keep, const int32_t *n_new, int64_t B, int32_t *table,
                        int64_t max_pages, int64_t page_size, int32_t *free_pages, int64_t n_pages,
                        const int32_t *n_free, int64_t pos_base, int64_t R, int32_t *kv_len, int32_t *cu_new,
                        int32_t *slots, int32_t *pos, int32_t *n_free_out, cudaStream_t stream);

/*
 * cp_cache_append_at -- cp_cache_append with the slot and the position of every row given as lists, for
 * tokens whose position is not their index (drafted trees: siblings share one).
 *   slots : device int32 [R], the row's slot (page * page_size + offset), -1: the row is skipped, in
 *           q_out too.  A slot out of range is skipped and sets the device status word to CP_ERR_PAGE.
 *           Two rows must not share a slot.
 *   pos   : device int32 [R], any value (read without a rotation too)
 * Everything else as for cp_cache_append.
 */
cp_status cp_cache_append_at(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, cp_dtype dtype, int64_t R, int64_t N, int64_t Nkv, int64_t D,
                             const void *wq, const void *wk, cp_dtype w_dtype, float eps, const cp_rope *rope,
                             void *k_cache, void *v_cache, int64_t n_pages, int64_t page_size, const int32_t *slots,
                             const int32_t *pos, void *q_out, cudaStream_t stream);

/*
 * cp_cache_keep -- after a drafted tree has been verified: the accepted branch's rows, moved together behind the
 * cached tokens in the caches of all layers.  In each cache the row of own index first + kept[b][j] goes to
 * first + j (j < n_kept[b], first = kv_len[b] - n_b), and
 *   kv_keep[b] = first + n_kept[b], or kv_len[b] where n_kept[b] < 0 (all new tokens stay: a prompt, single tokens).
 *   caches : host array of n_caches (1 .. 256) device pointers, each bf16 [n_pages][page_size][Nkv][D], apart
 *            from one another: K and V of every layer
 *   table, cu_new, kv_len, B, max_pages : of the step, as cp_cache_append and the attention read them
 *   R      : the step's rows (cu_new is checked against it)
 *   kept   : device int32 [B][max_kept] (max_kept 1 .. 512), rising, each below n_b
 *   n_kept : device int32 [B], up to n_b and max_kept
 *   kv_keep: device int32 [B], written, apart from the lists that are read: the next cp_cache_plan's kv_keep,
 *            beside kv_had = kv_len
 * A path ends before its first entry that does not rise, is out of range, or whose page number is; an n_kept out of
 * range keeps nothing; where cu_new or kv_len makes no sense kv_keep is kv_len.  Each sets the device status
 * word to CP_ERR_PAGE.
 */
cp_status cp_cache_keep(void *const *caches, int64_t n_caches, int64_t n_pages, int64_t page_size, int64_t Nkv,
                        int64_t D, const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                        const int32_t *kv_len, int64_t R, const int32_t *kept, int64_t max_kept, const int32_t *n_kept,
                        int32_t *kv_keep, cudaStream_t stream);

/*
 * cp_tree_plan -- ancestors and positions of drafted trees.  The new tokens of sequence b (rows cu_new[b]
 * .. cu_new[b+1]-1) form trees: parent[r] is the place among them of row r's parent, below its own place, or -1
 * for a token that follows the cached ones.
 *   mask[r] : bits of r's ancestors and of r itself, bit i % 32 of word i / 32 for new token i
 *   pos[r]  : pos_base + kv_len[b] - n_b + depth, the depth of a token without a parent being 0
 * A sequence of more than 32 words new tokens is a prompt: its positions count up, its parents are not
 * read and its mask rows not written.
 *   parent : device int32 [R];  cu_new [B+1], kv_len [B] as for cp_cache_append
 *   mask   : device int32 [R][words], words 1 .. 16;  pos : device int32 [R]; rows from cu_new[B] on stay.
 *            Apart from one another and from the lists that are read (CP_ERR_ARGUMENT else)
 * A parent out of range counts as -1 and sets the device status word to CP_ERR_PAGE; so do counts that make no
 * sense, whose rows stay: kv_len[b] below n_b among them, and new tokens behind position 2^31 - 1.
 */
cp_status cp_tree_plan(const int32_t *parent, const int32_t *cu_new, const int32_t *kv_len, int64_t B, int64_t R,
                       int64_t words, int64_t pos_base, int32_t *mask, int32_t *pos, cudaStream_t stream);

/*
 * cp_tree_attn_workspace_size / cp_tree_attn_fwd -- cp_prefix_attn_fwd for drafted trees: a row sees the prefix, the
 * kv_len[b] - n_b cached tokens of its sequence, and those of its sequence's new tokens whose bits its mask
 * has (cp_tree_plan's, or any others; bits from n_b on are not looked at).
 *   mask : device int32 [R][words], words 1 .. 16.  Sequences of more than 32 words new tokens are prompts, causal as
 *          in cp_prefix_attn_fwd, their mask rows not read: trees and prompts mix in one batch.
 * max_pages says how long a sequence may be, which chooses how the work is cut (every length is right): a table no
 * wider than the step needs is worth up to half of the time where it holds a few thousand tokens a sequence.
 * A row that sees one key gets that key's value itself, for scores scale <q, k> up to 2^14 in size.
 * Everything else as for cp_prefix_attn_fwd, but that a NaN or infinity in any V row of a sequence's own keys may
 * reach its other rows (also one that no row's mask has), and that kernels behind it may start early as behind
 * cp_cache_plan.
 */
cp_status cp_tree_attn_workspace_size(int64_t R, int64_t B, int64_t max_new, int64_t words, int64_t prefix_len,
                                      int64_t N, int64_t Nkv, int64_t D, int64_t page_size, int64_t max_pages,
                                      size_t *bytes);
cp_status cp_tree_attn_fwd(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages, int64_t page_size,
                           const int32_t *prefix_pages, int64_t prefix_len, const int32_t *table, int64_t B,
                           int64_t max_pages, const int32_t *cu_new, const int32_t *kv_len, const int32_t *mask,
                           int64_t words, int64_t max_new, int64_t R, int64_t N, int64_t Nkv, int64_t D, float scale,
                           void *o, cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                           cudaStream_t stream);

/*
 * cp_selftest_stalled_producer -- failure-detection self-test of the bounded
 * device-side waits (no counterpart on the pages).  Launches the attention
 * kernel on a [1][128][1][64] problem (q, k, v device bf16 [128][64], pos
 * device int32 [128], o fp32 [128][64] 32-byte aligned, lse fp32 [128]) with
 * its TMA producer held on a device flag that nothing sets and every bounded
 * wait limited to timeout_ns (1 ms .. 2 s, else CP_ERR_ARGUMENT).  The producer
 * gives up after timeout_ns, the other roles see the abort and unwind, TMEM
 * is freed, and the kernel records CP_ERR_DEVICE_TIMEOUT in the device status
 * word; o and lse are left unwritten.  The call itself returns CP_OK when the
 * launch succeeded: read the outcome with cp_device_status().  The context
 * stays usable.
 */
cp_status cp_selftest_stalled_producer(const void *q, const void *k, const void *v, const int32_t *pos, float *o,
                                       float *lse, uint64_t timeout_ns, cudaStream_t stream);

/*
 * cp_selftest_stalled_kernel -- the failure-detection self-test above for any
 * of the attention kernels (no counterpart on the pages): kernel 0 = bf16
 * forward, 1 = tf32 forward, 2 = backward (its dK/dV launch, then its dQ
 * launch).  The call zeroes `scratch` (device, 256-byte aligned, at least
 * CP_SELFTEST_SCRATCH_BYTES bytes), lays a tiny problem (one head, 128 rows,
 * D = 64) and the hold flag out in it, and launches the kernel with its TMA
 * producer held on the flag, which nothing sets, and every bounded wait limited
 * to timeout_ns (1 ms .. 2 s, else CP_ERR_ARGUMENT).  Each launch gives up
 * after timeout_ns and records CP_ERR_DEVICE_TIMEOUT in the device status word
 * (cp_device_status); the call returns CP_OK when the launches succeeded.  The
 * context stays usable.
 */
#define CP_SELFTEST_SCRATCH_BYTES ((size_t)512 << 10)
cp_status cp_selftest_stalled_kernel(int kernel, void *scratch, size_t scratch_bytes, uint64_t timeout_ns,
                                     cudaStream_t stream);

/*
 * cp_selftest_stalled_prefix_attn -- the same self-test of the shared-prefix attention:
 * the arguments of cp_prefix_attn_fwd, which choose the kernels as they do there, with
 * every block's first loads held on a word that nothing sets and every
 * bounded wait limited to timeout_ns (1 ms .. 2 s, else CP_ERR_ARGUMENT).  The
 * blocks give up, unwind and record CP_ERR_DEVICE_TIMEOUT; o and lse are
 * unspecified.
 */
cp_status cp_selftest_stalled_prefix_attn(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                          int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                          const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                          const int32_t *kv_len, int64_t max_new, int64_t R, int64_t N, int64_t Nkv,
                                          int64_t D, float scale, void *o, cp_dtype o_dtype, float *lse,
                                          void *workspace, size_t ws_bytes, uint64_t timeout_ns, cudaStream_t stream);

/*
 * cp_selftest_stalled_tree_attn -- the same self-test of the tree attention: the arguments of cp_tree_attn_fwd, which
 * choose the kernels as they do there (a block an item, a cluster an item, or the shared-prefix attention's).
 */
cp_status cp_selftest_stalled_tree_attn(const void *q, const void *k_cache, const void *v_cache, int64_t n_pages,
                                        int64_t page_size, const int32_t *prefix_pages, int64_t prefix_len,
                                        const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_new,
                                        const int32_t *kv_len, const int32_t *mask, int64_t words, int64_t max_new,
                                        int64_t R, int64_t N, int64_t Nkv, int64_t D, float scale, void *o,
                                        cp_dtype o_dtype, float *lse, void *workspace, size_t ws_bytes,
                                        uint64_t timeout_ns, cudaStream_t stream);

/*
 * cp_ring_attention_fwd_noalloc -- cp_ring_attention_fwd for callers that
 * cannot allocate device memory.  The source pages have no counterpart: this
 * entry point exists for callers that may not call cudaMalloc or cannot hand
 * the library a workspace -- code running inside a custom allocator's
 * callbacks (a cudaMalloc there re-enters the allocator), runtimes that
 * reserve all device memory at start-up and forbid allocation afterwards,
 * processes whose device memory pool belongs to another framework (memory
 * taken outside it escapes its accounting), and code under stream capture in
 * the global mode, where cudaMalloc is refused.
 *   Same arguments and result as cp_ring_attention_fwd with prefetch = 0
 *   (zero-copy owner rotation) and no workspace argument; the caller still
 *   passes all inputs and outputs.
 *   Scratch: the call uses one file-scope device array of
 *   CP_NOALLOC_SCRATCH_BYTES bytes inside the library (every CUDA context
 *   that loads the library's module holds one copy, until that context is
 *   destroyed: at process exit, or at cudaDeviceReset).  The ring's own
 *   argument checks (pointers, enums, shapes, divisibility, alignment) run
 *   first; then sizes whose cp_ring_workspace_size(..., prefetch = 0,
 *   o_dtype, ...) exceeds CP_NOALLOC_SCRATCH_BYTES are rejected with
 *   CP_ERR_WORKSPACE.  Either way nothing is enqueued.  The call never calls
 *   cudaMalloc, cudaFree or any allocating routine.
 *   Set-up: the first call in a CUDA context looks up the array's device
 *   address in that context (cudaGetSymbolAddress, with the caller's device
 *   and context current) and caches it, keyed by the context's id; make that
 *   first call before any stream capture in that context.  A call made in a
 *   new context (after cudaDeviceReset, or under a driver context the caller
 *   made current) looks the address up again, so no stale address is used.
 *   Sharing: all calls on a device share the array, which keeps the last
 *   call's contents (nothing needs clearing: every scratch byte a call reads
 *   it has written itself).  Calls whose executions overlap on the GPU (for
 *   instance on two streams) race on the array and give wrong results:
 *   serialise them.
 */
#define CP_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
cp_status cp_ring_attention_fwd_noalloc(const void *q_sh, const void *k_sh, const void *v_sh,
                                        const int32_t *pos, int64_t B, int64_t S, int64_t N,
                                        int64_t Nkv, int64_t D, int C, float scale, cp_layout layout,
                                        void *o_sh, cp_dtype o_dtype, float *lse_sh,
                                        cudaStream_t stream);

/*
 * cp_device_status -- synchronise `stream`, then read (and, if clear != 0,
 * reset) the library's device status word on the current device.
 * *code receives CP_OK, CP_ERR_DEVICE_TIMEOUT if a kernel of this library
 * gave up a bounded wait since the last reset, or else CP_ERR_PAGE if one met a page
 * number, length or count out of range.  Host-blocking.
 */
cp_status cp_device_status(int *code, int clear, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CPATTN_H */
