/*
 * flint_moe.h -- C ABI of the GB300 (sm_103a) Flint MoE sublayer library.
 *
 * The operation is the MoE sublayer of the Flint model as described in
 * "Day-0 Support for Flint on vLLM" (sections "Model architecture" and
 * "Optimizations"): a 2048-wide token x_hat is scored by a bf16 router over
 * 256 experts, the 6 experts with the largest sigmoid score are selected and
 * their scores renormalised to sum to 1, each selected expert and the
 * always-on shared expert compute down(bf16(silu(gate(x_hat)) * up(x_hat))),
 * and the outputs are combined with the routing weights (shared weight 1) and
 * rounded once to bf16.  Expert weights are NVFP4 (16 E2M1 codes + one E4M3
 * block scale per 16 weights + one fp32 per-tensor scale) used weight-only
 * with bf16 activations ("W4A16", same section), or plain bf16.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers (the current CUDA device) owned
 *     by the caller; every pointer must be 16-byte aligned.  Row-major layouts.
 *   - Arguments are validated on the host before anything is enqueued; an
 *     invalid call returns a negative status and enqueues nothing.  A buffer
 *     the call writes (outputs, workspace) must not share a byte with any
 *     other buffer of the call, weights included (FLINT_MOE_ERR_INVALID_ARG);
 *     buffers that are only read may overlap.
 *   - Work is enqueued asynchronously on `stream` (NULL = legacy default
 *     stream); outputs are valid after the stream is synchronised.
 *   - The library allocates no device memory on the compute path: scratch
 *     space is the caller's workspace `ws` (size from flint_moe_workspace_bytes,
 *     256-byte aligned, no initialisation needed).  Calls that share one
 *     workspace must be ordered on one stream.
 *   - The sublayer calls support only the Flint shapes: hidden 2048, 256
 *     routed experts, 1 shared expert, intermediate 512, top-6.  Anything else
 *     returns FLINT_MOE_ERR_UNSUPPORTED (there is no generic fallback path).
 *     The parts of an FP8 expert layer (flint_moe_route and the calls after
 *     it) and the linear, gated and 8-bit integer products take any shape
 *     within their limits.
 */
#ifndef FLINT_MOE_H
#define FLINT_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (the runtime's stream handle type). */
typedef struct CUstream_st *flint_moe_stream_t;

/* Status codes returned by every int-returning entry point. */
enum {
    FLINT_MOE_OK = 0,
    FLINT_MOE_ERR_INVALID_ARG = -1, /* null, misaligned or overlapping
                                       buffers, bad count                   */
    FLINT_MOE_ERR_UNSUPPORTED = -2, /* shape or batch outside the fast path */
    FLINT_MOE_ERR_WORKSPACE = -3,   /* workspace or output buffer too small */
    FLINT_MOE_ERR_CUDA = -4,        /* a CUDA runtime call failed           */
    FLINT_MOE_ERR_TIMEOUT = -5      /* a bounded device wait gave up        */
};

/* Expert weight formats. */
enum { FLINT_MOE_W_NVFP4 = 0, FLINT_MOE_W_BF16 = 1 };

/* Largest batch of the low-latency decode path ("Optimizations": the
 * low-latency path serves up to 8 requests). */
#define FLINT_MOE_MAX_DECODE_BATCH 8

/* Largest batch of the decode calls.  9..64 tokens (NVFP4 weights only) take
 * the medium-batch kernels: past the low-latency cap of 8 requests, each
 * selected expert's weights are read once per group of up to 16 of the
 * tokens that chose it, instead of once per group of 8 tokens. */
#define FLINT_MOE_MAX_MEDIUM_BATCH 64

/* Decode kernels for NVFP4 weights (flint_moe_set_decode_kernel). */
enum { FLINT_MOE_DECODE_CHAINED = 0, FLINT_MOE_DECODE_PERSISTENT = 1 };

/* Model dimensions.  Must equal {2048, 256, 1, 512, 6, *, eps}. */
typedef struct {
    int hidden;       /* H = 2048                                   */
    int n_experts;    /* E = 256 routed experts                     */
    int n_shared;     /* 1 shared expert (index E in the blobs)     */
    int inter;        /* I = 512 expert intermediate size           */
    int top_k;        /* 6                                          */
    int weight_dtype; /* FLINT_MOE_W_NVFP4 or FLINT_MOE_W_BF16      */
    float rms_eps;    /* RMSNorm epsilon (1e-6 for Flint stacks)    */
} flint_moe_dims;

/* One MoE sublayer's weights (all device pointers, caller-owned). */
typedef struct {
    const void *router_w;       /* bf16 [E][H]                                   */
    const void *experts;        /* packed blob from flint_moe_pack_weights       */
    const float *tensor_scales; /* NVFP4: fp32 [E+1][2] = (gate/up, down) scale
                                   per expert; ignored (may be NULL) for BF16    */
    const void *norm_w;         /* bf16 [H] RMSNorm weight applied to this
                                   sublayer's input, or NULL for no norm         */
} flint_moe_layer;

/* Bytes of one sublayer's packed expert blob (E routed + 1 shared expert):
 * NVFP4 1,769,472 B per expert, BF16 6,291,456 B per expert (the same byte
 * count as the plain layout: the repack is lossless and adds no padding).
 * Returns 0 for unsupported dims. */
size_t flint_moe_packed_bytes(const flint_moe_dims *dims);

/* Workspace bytes for calls with at most `max_tokens` tokens (decode: 1..64,
 * of which 9..64 NVFP4 only; prefill: any T >= 1).  Returns 0 for
 * unsupported dims or token counts. */
size_t flint_moe_workspace_bytes(const flint_moe_dims *dims, int max_tokens);

/*
 * One-time lossless repack of one sublayer's experts from the plain layout
 * into the kernels' interleaved layout ("Model architecture": the NVFP4
 * checkpoint is repacked losslessly at load time).
 *
 * NVFP4 inputs (expert index E is the shared expert):
 *   gate_up        uint8 [E+1][2I][H/2]  rows 0..I-1 gate, I..2I-1 up; byte j
 *                  of a row holds element 2j in its low nibble, 2j+1 high
 *   gate_up_scales uint8 [E+1][2I][H/16] E4M3 scale of each 16-element block
 *   down           uint8 [E+1][H][I/2]
 *   down_scales    uint8 [E+1][H][I/16]
 * BF16 inputs: gate_up bf16 [E+1][2I][H], down bf16 [E+1][H][I]; the scale
 *   pointers must be NULL.
 * packed: output, flint_moe_packed_bytes(dims) bytes.  Runs one device kernel
 * on `stream`; inputs may be freed once the stream has passed it.
 */
int flint_moe_pack_weights(const flint_moe_dims *dims, const void *gate_up,
                           const uint8_t *gate_up_scales, const void *down,
                           const uint8_t *down_scales, void *packed,
                           size_t packed_bytes, flint_moe_stream_t stream);

/*
 * One MoE sublayer for a decode batch of 1..64 independent tokens.
 *   x        bf16 [B][H] input (RMSNorm'd first if layer->norm_w != NULL)
 *   y        bf16 [B][H] output
 *   topk_ids int32 [B][6] selected experts (descending score) or NULL
 *   topk_w   fp32  [B][6] their renormalised weights, or NULL
 * Three steps: the router GEMV with sigmoid top-6; the gate/up GEMV with
 * SiLU*up over the selected experts only; the down GEMV fused with the
 * weighted combine and the shared expert.  By default (and always for BF16
 * weights) they are three kernels chained with programmatic dependent launch;
 * with FLINT_MOE_DECODE_PERSISTENT selected (flint_moe_set_decode_kernel),
 * NVFP4 weights take one cooperative kernel, one thread block per SM (at
 * least 128 SMs, else FLINT_MOE_ERR_UNSUPPORTED), whose blocks exchange
 * logits, h and y through the workspace.  9 <= B <= 64 (NVFP4 only, else
 * FLINT_MOE_ERR_UNSUPPORTED) runs the medium-batch chain: one block per token
 * for the RMSNorm; the router logits over (chunk of 8 tokens, expert) units;
 * one block that selects every token's top-6 and builds the table of
 * slot-chunks (an expert with up to 8 of the tokens that selected it);
 * gate/up and down kernels that stream each selected expert's tiles once per
 * slot-chunk; and one block per token that adds the pairs' down projections
 * in a fixed order (inside a stack it also normalises the next sublayer's
 * input, so that sublayer skips the RMSNorm block).  Its
 * workspace is flint_moe_workspace_bytes(dims, 64) bytes (less returns
 * FLINT_MOE_ERR_WORKSPACE).  B > 64 returns FLINT_MOE_ERR_UNSUPPORTED.  The
 * result is deterministic: the same inputs and kernel choice give the same
 * bits on every call.
 */
int flint_moe_decode_layer(const flint_moe_dims *dims, const flint_moe_layer *layer,
                           const void *x, int B, void *y, int32_t *topk_ids,
                           float *topk_w, void *ws, size_t ws_bytes,
                           flint_moe_stream_t stream);

/*
 * n_layers chained sublayers for one decode batch: sublayer i+1 reads
 * sublayer i's output (through its own RMSNorm when layers[i+1].norm_w is
 * set; no residual is added).
 *   x, y            bf16 [B][H]
 *   ids_per_layer   int32 [n_layers][B][6] or NULL
 *   w_per_layer     fp32  [n_layers][B][6] or NULL
 *   ys_per_layer    bf16  [n_layers][B][H] every sublayer's output, or NULL
 * Chained kernels (the default, BF16 weights, and every 9..64-token batch):
 * the chain of 3 (5 past 8 tokens) kernels per sublayer is captured once
 * into a CUDA graph (cached per argument set; see
 * flint_moe_release) and replayed with one graph launch per call; the graph
 * bakes in every pointer, so buffer contents may change between calls,
 * addresses not.  Persistent kernel (NVFP4, flint_moe_set_decode_kernel): one
 * cooperative launch per 64 sublayers, which prefetches each sublayer's
 * router rows, norm weight, tensor scales and shared-expert tiles while the
 * sublayer before it runs.  A stack call gives the same bits as the chain of
 * flint_moe_decode_layer calls over the same sublayers with the same kernel
 * choice.
 */
int flint_moe_decode_stack(const flint_moe_dims *dims, const flint_moe_layer *layers,
                           int n_layers, const void *x, int B, void *y,
                           int32_t *ids_per_layer, float *w_per_layer,
                           void *ys_per_layer, void *ws, size_t ws_bytes,
                           flint_moe_stream_t stream);

/*
 * One MoE sublayer over T tokens (prefill shape, e.g. T = 8192; "Day-0
 * Support for Flint on vLLM", section "Optimizations": the MoE kernels also
 * serve the 8K prefill).  Same definition as flint_moe_decode_layer, token by
 * token: router logits (approximated on the tensor cores, then recomputed
 * exactly for every expert that can reach the top 6), sigmoid top-6, tokens
 * grouped by expert, grouped gate/up GEMM with SiLU*up and grouped down GEMM
 * on the tensor cores (tcgen05, fp32 accumulation), weighted combine plus the
 * shared expert.
 *   x        bf16 [T][H] (RMSNorm'd first if layer->norm_w != NULL)
 *   y        bf16 [T][H]; must not overlap x (nor either of them the workspace)
 *   topk_ids int32 [T][6] or NULL; topk_w fp32 [T][6] or NULL
 *   ws       flint_moe_workspace_bytes(dims, T) bytes, 256-byte aligned, no
 *            initialisation needed
 * NVFP4 weights only (BF16: FLINT_MOE_ERR_UNSUPPORTED); 1 <= T <= 2^20.
 * The combine adds the experts' fp32 contributions in completion order, so y
 * can differ between runs in its last bits; the routing is exact and
 * repeatable.  Seven kernels on `stream`, asynchronous.
 */
int flint_moe_prefill_layer(const flint_moe_dims *dims, const flint_moe_layer *layer,
                            const void *x, int T, void *y, int32_t *topk_ids,
                            float *topk_w, void *ws, size_t ws_bytes,
                            flint_moe_stream_t stream);

/* Size of the scratch area built into the library for
 * flint_moe_decode_layer_noalloc, and the largest batch it serves. */
#define FLINT_MOE_NOALLOC_SCRATCH_BYTES 1048576
#define FLINT_MOE_NOALLOC_MAX_TOKENS 8

/*
 * flint_moe_decode_layer without a workspace argument, for callers that
 * cannot allocate device memory: code that runs where cudaMalloc is not
 * allowed or not wanted (inside a host callback or another library's
 * allocator hook, under a strict memory budget, or from a runtime that owns
 * every device allocation itself).  The paper has no counterpart; this is a
 * convenience of this library.
 *
 * Scratch lives in one fixed array of FLINT_MOE_NOALLOC_SCRATCH_BYTES in the
 * library's device image: every GPU that loads the library holds it until the
 * process exits, and this call allocates nothing.  Inputs, outputs and
 * weights are as for flint_moe_decode_layer (caller-owned device memory).
 *   B > FLINT_MOE_NOALLOC_MAX_TOKENS returns FLINT_MOE_ERR_WORKSPACE (the
 *   built-in scratch holds at most 8 tokens) and enqueues nothing.
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture (a first
 * call on a capturing stream returns FLINT_MOE_ERR_INVALID_ARG).  Every
 * call on a device shares the one array and it keeps the previous call's
 * contents; each call clears what it must find cleared, and its kernels read
 * no other scratch word before writing it.  Calls whose work overlaps on the GPU
 * (different streams, or other threads) race on the array: order them.
 */
int flint_moe_decode_layer_noalloc(const flint_moe_dims *dims, const flint_moe_layer *layer,
                                   const void *x, int B, void *y, int32_t *topk_ids,
                                   float *topk_w, flint_moe_stream_t stream);

/*
 * Small-batch dense GEMV on NVFP4 weights ("Day-0 Support for Flint on vLLM",
 * section "Optimizations": a small-batch dense GEMV on the same NVFP4 weights
 * serves the attention projections and the dense MLP of the first layers):
 *   y[t][n] = bf16( tensor_scale * sum_k x[t][k] * W[n][k] ),  fp32 accumulation,
 * W[n][k] = e2m1(code) * e4m3(block scale of k / 16).  Shapes: N a multiple
 * of 16 (below 2^24), K a multiple of 256, at most 32768; otherwise
 * FLINT_MOE_ERR_UNSUPPORTED.
 *
 * flint_moe_dense_packed_bytes: bytes of the packed matrix, N * K * 9 / 16
 *   (the plain layout's count: the repack is lossless), or 0 for an
 *   unsupported shape.
 * flint_moe_pack_dense: one-time repack on `stream` of
 *   codes  uint8 [N][K/2] (byte j of a row: element 2j low nibble, 2j+1 high)
 *   scales uint8 [N][K/16] (E4M3 per 16-element block)
 *   into packed (flint_moe_dense_packed_bytes(N, K) bytes).
 * flint_moe_dense_gemv: x bf16 [B][K], y bf16 [B][N]; 1 <= B <= 8 and
 *   B * K <= 32768 (else FLINT_MOE_ERR_UNSUPPORTED).  One kernel on `stream`
 *   (programmatic dependent launch: it requests its first weight tiles before
 *   waiting for the kernel before it), deterministic.  No workspace.
 */
size_t flint_moe_dense_packed_bytes(int N, int K);
int flint_moe_pack_dense(const uint8_t *codes, const uint8_t *scales, int N, int K, void *packed,
                         size_t packed_bytes, flint_moe_stream_t stream);
int flint_moe_dense_gemv(const void *packed, int N, int K, float tensor_scale, const void *x, int B,
                         void *y, flint_moe_stream_t stream);

/*
 * ---- FP8 expert layers of any shape ---------------------------------------
 *
 * The five calls below are the parts of a mixture-of-experts layer whose
 * weights are 8-bit (E4M3) with one fp32 scale per block of 128 x 128, for any
 * number of experts, choices and widths within the limits given.  Used
 * together, for T tokens with k choices each (P = T * k pairs):
 *   flint_moe_route           logits        -> ids, w      [T][k]
 *   flint_moe_group_pairs     ids           -> offsets, order, pos
 *   flint_moe_quantize_rows   x, pos        -> q [P][H], scales (expert order)
 *   flint_moe_block_gemm      gate and up   -> [P][2I]
 *   flint_moe_quantize_rows   silu(g) * u   -> q [P][I], scales
 *   flint_moe_block_gemm      down          -> [P][H]
 *   flint_moe_combine         pos, w        -> y [T][H]
 * "Expert order" is the pairs sorted by expert, those of one expert in
 * ascending order of t * k + j.  The conventions at the top of this file hold,
 * except that buffers may be of any shape within the limits; no workspace is
 * needed.  Every call is deterministic: the same inputs give the same bits.
 * All of them may be captured into a CUDA graph (the first call of a process
 * on a device sets up the library and must come before the capture).
 */

/* Element types of activations. */
enum { FLINT_MOE_T_BF16 = 0, FLINT_MOE_T_F32 = 1 };
/* Score of a logit: 1 / (1 + exp(-x)), or softmax over the row's experts. */
enum { FLINT_MOE_SCORE_SIGMOID = 0, FLINT_MOE_SCORE_SOFTMAX = 1 };
/* Score of a group of experts: its best key, or the sum of its two best. */
enum { FLINT_MOE_GROUP_MAX = 0, FLINT_MOE_GROUP_TOP2 = 1 };

typedef struct {
    int n_experts;   /* E, 1..1024                                            */
    int top_k;       /* 1..16, at most top_groups * E / n_groups              */
    int score;       /* FLINT_MOE_SCORE_*                                     */
    int n_groups;    /* 1..32, divides E: group g is experts g*E/n .. ; 1: none */
    int top_groups;  /* groups a token may choose from, 1..n_groups           */
    int group_score; /* FLINT_MOE_GROUP_*                                     */
    int renormalise; /* non-zero: selected scores are divided by their sum    */
    float scale;     /* factor of every weight (finite)                       */
} flint_moe_routing;

/*
 * Routing of T tokens (1..2^20).
 *   logits  [T][E] of logits_type, rows row_stride elements apart (E to 2^31;
 *           what lies between two rows counts as the buffer's)
 *   bias    fp32 [E] added to the scores for the choice only, or NULL
 *   ids     int32 [T][top_k] in descending order of key, w fp32 [T][top_k]
 * The key of an expert is its logit, or score + bias when a bias is given.  An
 * expert whose logit is -inf or NaN (or whose key is) cannot be chosen and
 * takes no part in the softmax; places that no expert is left for hold id -1
 * and weight 0.  Groups are kept by their score (with GROUP_TOP2 and no bias:
 * the sum of the two best scores; one candidate counts alone).  Keys and group
 * scores are compared as the real numbers that they stand for, as far as fp64
 * tells them apart; ties go to the lower index.  Weights come from the scores
 * without the bias, in fp32; renormalised ones are formed relative to the
 * row's largest, so that very low logits do not underflow together.
 */
int flint_moe_route(const flint_moe_routing *routing, const void *logits, int logits_type,
                    long long row_stride, int T, const float *bias, int32_t *ids, float *w,
                    flint_moe_stream_t stream);

/*
 * Groups n_pairs (1..2^24) pairs by expert.
 *   ids      int32 [n_pairs]; a pair whose id is outside 0..n_experts-1 is dropped
 *   offsets  int32 [n_experts + 1]: expert e owns places offsets[e] ..
 *            offsets[e + 1] - 1; offsets[n_experts] pairs are left
 *   order    int32 [n_pairs]: the pair at each place, -1 behind the last
 *   pos      int32 [n_pairs]: the place of each pair, -1 where dropped
 */
int flint_moe_group_pairs(const int32_t *ids, int n_pairs, int n_experts, int32_t *offsets,
                          int32_t *order, int32_t *pos, flint_moe_stream_t stream);

/*
 * Quantises rows to E4M3 in blocks of 128 elements (the last one shorter where
 * 128 does not divide K).
 *   x       [rows][K] of x_type (silu_mul != 0: [rows][2K], and the row
 *           quantised is silu(first half) * second half, formed in fp32 and not
 *           rounded before; below -87 the activation is 0), rows row_stride elements apart
 *   pos     int32 [rows][top_k]: the places that each row is written to
 *           (places outside 0..places-1 are skipped; two rows must not share
 *           one), or NULL: row i is written to place i, and places == rows
 *   q       E4M3 [places][K]; scales fp32 [ceil(K / 128)][places]
 * With a = max(largest magnitude of the block, 2^-96): scale = a / 448 and
 * code = e4m3(x * (448 / a)), quotient and product in fp32, then to nearest
 * even; a block that holds an infinity or NaN gets a scale that is not finite.
 * Places that no row names are left as they were.  K a multiple of 16, at most
 * 2^17; row_stride a multiple of 16 bytes, at most 2^31 elements; at most 2^24
 * rows and places.  What lies between two rows counts as x's.
 */
int flint_moe_quantize_rows(const void *x, int x_type, long long row_stride, int rows, int K,
                            int silu_mul, const int32_t *pos, int top_k, int places, void *q,
                            float *scales, flint_moe_stream_t stream);

/*
 * Block-scaled FP8 matrix product, dense or grouped by expert:
 *   y[m][n] = sum over K blocks kb of a_scales[kb][m] * b_scales[e][n / 128][kb]
 *             * sum over k in kb of a[m][k] * b[e][n][k]
 * with fp32 sums and one rounding to y's type.
 *   a        E4M3 [M][K], a_scales fp32 [ceil(K / 128)][M]
 *   b        E4M3 [n_experts][N][K] (row-major, as a checkpoint has it),
 *            b_scales fp32 [n_experts][ceil(N / 128)][ceil(K / 128)]
 *   offsets  int32 [n_experts + 1] on the device: rows offsets[e] ..
 *            offsets[e + 1] - 1 of a belong to expert e.  They must start at 0,
 *            not descend and not pass M; rows of y behind the last are left as
 *            they were.  NULL: dense, n_experts == 1.
 *   y        [M][N] of y_type
 * M 1..2^24, N a multiple of 8, K a multiple of 16 (both at most 2^17), up to
 * 1024 experts.
 */
int flint_moe_block_gemm(const void *a, const float *a_scales, int M, const void *b,
                         const float *b_scales, int n_experts, const int32_t *offsets, int N,
                         int K, void *y, int y_type, flint_moe_stream_t stream);

/*
 * y[t] = bf16( sum over j of w[t][j] * rows[pos[t][j]] + shared[t] ), summed in
 * fp32 in the order written.
 *   rows    [n_rows][N] of rows_type; pos int32 [T][top_k] (a place outside
 *           0..n_rows-1 adds nothing), w fp32 [T][top_k]
 *   shared  bf16 [T][N] or NULL; y bf16 [T][N]
 * T 1..2^20, top_k 1..16, N a multiple of 8, at most 2^17.
 */
int flint_moe_combine(const void *rows, int rows_type, int n_rows, const int32_t *pos,
                      const float *w, int T, int top_k, int N, const void *shared, void *y,
                      flint_moe_stream_t stream);

/*
 * ---- Feed-forward blocks of any shape: bf16 with gradients, 8-bit integers ----
 *
 * The two products of a gated feed-forward block in bf16, with their gradients,
 * and in 8-bit integers with one scale for each row (token) and each output
 * (channel); dense, or grouped by expert with the offsets of
 * flint_moe_group_pairs.  A block, for P rows in expert order:
 *   flint_moe_gated_linear     x  [P][K]  -> h [P][I], and gu [P][2I] to train
 *   flint_moe_linear           h  [P][I]  -> y [P][N]
 *   flint_moe_linear_backward  dy [P][N]  -> dh [P][I], dw of the second product
 *   flint_moe_gated_linear_backward  dh   -> dgu [P][2I], dx [P][K], dw of the first
 * and the same block served in 8-bit integers:
 *   flint_moe_integer_quantize_rows  x, pos -> q [P][K], scales
 *   flint_moe_integer_gemm           gated  -> h [P][I] in bf16
 *   flint_moe_integer_quantize_rows  h      -> q [P][I], scales
 *   flint_moe_integer_gemm                  -> y [P][N], for flint_moe_combine
 * Weights are quantised by the same call, their matrices' rows being outputs.
 * Limits of all: M 1..2^24 rows, N a multiple of 8, I (half a gated matrix) a
 * multiple of 16, K a multiple of 16, N, 2 I and K at most 2^17, up to 1024
 * experts; every buffer contiguous.  offsets int32 [n_experts + 1] on the device:
 * rows offsets[e] .. offsets[e + 1] - 1 belong to expert e.  They must start at 0, not
 * descend and not pass M; rows of outputs behind the last are left as they were,
 * and what the inputs hold there is not used.  NULL: dense, n_experts == 1.
 * No workspace is needed, every call is deterministic, and all may be captured
 * into a CUDA graph (the first call of a process on a device sets up the library
 * and must come before the capture).  Sums are fp32 (integer: exact).  The tensor
 * cores cut them, by some n 2^-27 of the magnitudes of n terms; sums of more than
 * 1024 terms (of bf16 outputs: of many more, up to 2^17, where that is a quarter of
 * the output's rounding) are added up from parts with rounding.
 */

/* Activation of a gated product: none (a plain product), x / (1 + exp(-x)), or
 * x / 2 * (1 + tanh(sqrt(2 / pi) * (x + 0.044715 x^3))).  Below -87 the first, and
 * below -9 the second, may be 0. */
enum { FLINT_MOE_ACT_NONE = 0, FLINT_MOE_ACT_SILU = 1, FLINT_MOE_ACT_GELU = 2 };

/*
 * y[m][n] = sum over k of x[m][k] * w[e][n][k], e the expert of row m.
 *   x bf16 [M][K], w bf16 [n_experts][N][K], y [M][N] of y_type (FLINT_MOE_T_*)
 */
int flint_moe_linear(const void *x, int M, const void *w, int n_experts, const int32_t *offsets,
                     int N, int K, void *y, int y_type, flint_moe_stream_t stream);

/*
 * Gradients of flint_moe_linear: dx = dy w, dw[e] = dy^T x over the rows of expert e
 * (zeros for an expert of no rows).
 *   dy bf16 [M][N], x and w as they were; dx bf16 [M][K] or NULL; dw
 *   [n_experts][N][K] of dw_type or NULL; not both NULL
 */
int flint_moe_linear_backward(const void *dy, const void *x, int M, const void *w, int n_experts,
                              const int32_t *offsets, int N, int K, void *dx, void *dw, int dw_type,
                              flint_moe_stream_t stream);

/*
 * Gated projections in one kernel: with g and u the sums of x[m] with rows i and
 * I + i of w[e],  h[m][i] = act(g) * u, formed from the fp32 sums.
 *   x bf16 [M][K], w bf16 [n_experts][2I][K], h bf16 [M][I]
 *   gu bf16 [M][2I] or NULL: the sums, g then u, for the gradient
 */
int flint_moe_gated_linear(const void *x, int M, const void *w, int n_experts, const int32_t *offsets,
                           int I, int K, int act, void *h, void *gu, flint_moe_stream_t stream);

/*
 * Gradients of flint_moe_gated_linear: dg = dh * u * act'(g) and du = dh * act(g),
 * formed in fp32 from gu and rounded to bf16 (dgu), then dx = dgu w and
 * dw[e] = dgu^T x over the rows of expert e.
 *   dh bf16 [M][I], gu bf16 [M][2I], x and w as they were; dgu bf16 [M][2I] is
 *   written; dx and dw as for flint_moe_linear_backward, both may be NULL
 */
int flint_moe_gated_linear_backward(const void *dh, const void *gu, const void *x, int M, const void *w,
                                    int n_experts, const int32_t *offsets, int I, int K, int act,
                                    void *dgu, void *dx, void *dw, int dw_type,
                                    flint_moe_stream_t stream);

/*
 * Rows to 8-bit integers: with a = max(largest magnitude of the row, 2^-96),
 * scale = a * (1 / 127), factor and product in fp32, and code = the whole number next
 * to the real number x / scale, ties to even.  A row that holds an infinity or NaN gets a scale that is
 * not finite, and codes of 0.
 *   x [rows][K] of x_type, rows row_stride elements apart (a multiple of 16 bytes,
 *   at most 2^31; what lies between two rows counts as x's); pos int32 [rows][top_k],
 *   top_k 1..16: the places that each row is written to (places outside
 *   0..places-1 are skipped; two rows must not share one), or NULL: row i is
 *   written to place i, and places == rows
 *   q int8 [places][K], scales fp32 [places]; places that no row names are left
 *   as they were.  At most 2^24 rows and places.
 */
int flint_moe_integer_quantize_rows(const void *x, int x_type, long long row_stride, int rows, int K,
                                    const int32_t *pos, int top_k, int places, int8_t *q, float *scales,
                                    flint_moe_stream_t stream);

/*
 * 8-bit integer product: with s[m][n] = the exact sum over k of a[m][k] * b[e][n][k],
 *   y[m][n] = a_scales[m] * b_scales[e][n] * s[m][n]
 * in fp32 with one rounding to y's type.  act other than FLINT_MOE_ACT_NONE: N is 2I, and
 * y [M][I] = act(value of i) * (value of I + i).
 *   a int8 [M][K], a_scales fp32 [M], b int8 [n_experts][N][K], b_scales fp32
 *   [n_experts][N]; y [M][N] or [M][I] of y_type.  All 256 codes are numbers.
 *   K below 2^17.
 */
int flint_moe_integer_gemm(const int8_t *a, const float *a_scales, int M, const int8_t *b,
                           const float *b_scales, int n_experts, const int32_t *offsets, int N, int K,
                           int act, void *y, int y_type, flint_moe_stream_t stream);

/* Frees cached CUDA graphs of every device the calling thread used.  Call
 * before freeing buffers whose addresses a cached stack graph holds. */
int flint_moe_release(void);

/* Reads (and with reset != 0 clears) the current device's error word.  Bits:
 * 1, 2, 4 = a bounded wait gave up (full / empty barrier / draining copies);
 * 8 = the prefill router's tensor-core logit of some expert was further from
 * the exact value than its assumed error bound allows, and that token's
 * routing was recomputed from all 256 exact logits (results stay correct);
 * 16 = a prefill kernel found its shared memory misaligned and did nothing;
 * 32 = a persistent decode kernel's wait for data of its other thread blocks
 * ran out (flint_moe_set_wait_limit) and the call was abandoned.
 * Synchronises the device.  Returns the word (0 = none) or a negative
 * status. */
int flint_moe_device_error(int reset);

/* The current device's error word as a status: FLINT_MOE_OK (no bit, or only
 * bit 8), FLINT_MOE_ERR_TIMEOUT (bits 1, 2, 4 or 32: a bounded device wait
 * gave up and the outputs of the calls since the last reset are undefined),
 * FLINT_MOE_ERR_CUDA (bit 16, or a CUDA failure).  Synchronises the device;
 * reset != 0 clears the word. */
int flint_moe_device_status(int reset);

/* Selects the decode kernels of later NVFP4 calls (decode layer, stack and
 * the no-allocation call): FLINT_MOE_DECODE_CHAINED (default: router,
 * gate/up and down kernels chained with programmatic dependent launch) or
 * FLINT_MOE_DECODE_PERSISTENT (one cooperative kernel per up to 64
 * sublayers).  Both compute the same sublayer and pass the same parity
 * tests; BF16 weights always use the chained kernels.  Process-wide; returns
 * FLINT_MOE_OK or FLINT_MOE_ERR_INVALID_ARG for an unknown value. */
int flint_moe_set_decode_kernel(int kernel);

/* Cycle limit (SM clock) of every later persistent decode call's device-side waits
 * for data that its other thread blocks write.  A wait that runs out sets bit
 * 32 of the error word and ends the whole call early, with every thread block
 * returning and no copy left in flight.  The default, restored by
 * cycles <= 0, is about one second at the maximum SM clock.  Process-wide;
 * returns FLINT_MOE_OK.  Waits on the library's own bulk copies keep the
 * default limit. */
int flint_moe_set_wait_limit(long long cycles);

/* Static text for a status code. */
const char *flint_moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_MOE_H */
