/*
 * coli_moe.h -- C ABI of libcolimoe, the routed Mixture-of-Experts layer of a
 * GLM-5.2-style decoder on one sm_103a GPU.
 *
 * The layer (colibrì v1.0 README, "What's implemented"; "Colibri (colibrì):
 * GLM-5.2 local inference on 25 GB of RAM", "How it works (validated core
 * mechanics)"):
 *   1. sigmoid noaux_tc router: s = sigmoid(x . Wr^T); experts ranked by
 *      s + correction_bias inside the topk_group best groups; gate weights are
 *      the unbiased s of the selection renormalised, times
 *      routed_scaling_factor;
 *   2. batch-union dispatch: each distinct expert of a call is streamed from
 *      HBM once and applied to every position routed to it;
 *   3. Q8_0-style int8 activations (blocks of 32, one fp32 scale each);
 *   4. packed-int4 (or int8) x int8 SwiGLU expert products with per-row fp32
 *      weight scales; h = silu(g) * u is re-quantised to Q8_0 before the down
 *      product;
 *   5. y = sum_j w_j * expert_j(x) + sum_s shared_s(x).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers, row-major, owned by the caller;
 *     the library allocates nothing and keeps no state between calls.
 *   - Every pointer must be 16-byte aligned (TMA bulk copies read them).
 *   - Work is enqueued on `stream`; no call synchronises except
 *     coli_moe_status().  A call whose return value is not COLI_OK enqueued
 *     nothing.
 *   - Data-dependent failures (non-finite input, an out-of-range expert id,
 *     an expired bounded wait) cannot be returned synchronously: they are OR-ed
 *     into a sticky status word at the start of the workspace and read (and
 *     cleared) with coli_moe_status().
 *   - Calls that share a workspace must be ordered on one stream.
 *   - Kernels of this library may start while the kernel before them on the
 *     stream is finishing (programmatic dependent launch).  Before that
 *     kernel has completed they read only weights (router_w, corr_bias,
 *     expert records and scales), never x, routing or the workspace, so one
 *     call's outputs may be the next call's inputs directly.
 */
#ifndef COLI_MOE_H
#define COLI_MOE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes (synchronous). */
#define COLI_OK            0
#define COLI_EINVAL       -1   /* bad shape, config or null pointer            */
#define COLI_EALIGN       -2   /* a pointer is not 16-byte aligned             */
#define COLI_EWORKSPACE   -3   /* workspace smaller than coli_moe_workspace_size */
#define COLI_ECUDA        -4   /* a CUDA launch or query failed                */
#define COLI_EUNSUPPORTED -5   /* shape outside the kernels' limits            */

/* Device status bits (asynchronous, sticky until read by coli_moe_status). */
#define COLI_STATUS_NONFINITE 1u  /* non-finite router logit, bias or activation */
#define COLI_STATUS_BADIDX    2u  /* forward saw an expert id outside [-1, E)    */
#define COLI_STATUS_TIMEOUT   4u  /* a bounded device wait expired               */

/* Layer shape.  Limits (COLI_EINVAL / COLI_EUNSUPPORTED otherwise):
 * hidden % 128 == 0, inter % 128 == 0, shared_inter % 128 == 0 when
 * n_shared > 0, n_experts <= 1024, n_experts % n_groups == 0,
 * n_groups <= 32, 1 <= topk_group <= n_groups,
 * 1 <= top_k <= topk_group * n_experts / n_groups, top_k <= 32,
 * 0 <= n_shared <= 8, weight_bits in {2, 4, 8}; a gate+up row pair of
 * hidden and four down rows of max(inter, shared_inter) must each fit in
 * 32 KiB (int4: hidden <= 32768, intermediate sizes <= 16384; int8: half;
 * int2: double).  Packed int2 (colibrì v1.0 README, "What's implemented":
 * int8 / packed int4 / packed int2 weights with per-row scales) takes
 * per-row scales only; it runs on the fused single-position kernel for one
 * position per call, on the few-position kernels for 2 to 4 and on the
 * general expert kernel beyond. */
typedef struct coli_moe_cfg {
    int32_t hidden;                 /* H                                    */
    int32_t n_experts;              /* E routed experts                     */
    int32_t n_groups;               /* G expert groups (E/G experts each)   */
    int32_t topk_group;             /* groups kept per token                */
    int32_t top_k;                  /* experts selected per token (k)       */
    int32_t inter;                  /* I, intermediate size of routed experts */
    int32_t n_shared;               /* always-on shared experts             */
    int32_t shared_inter;           /* intermediate size of shared experts  */
    int32_t weight_bits;            /* 4: packed int4, 2: packed int2, 8: int8 */
    float   routed_scaling_factor;  /* multiplies the renormalised weights  */
    int32_t group_size;             /* 0: one scale per output row;
                                       64: one per 64 weights of a row ("gs64",
                                       int4 only: COLI_EUNSUPPORTED with int8
                                       or int2) */
    int32_t ep_rank;                /* expert-parallel shard of this call   */
    int32_t ep_size;                /* shards (0 or 1: no sharding)         */
} coli_moe_cfg;

/* Expert-parallel sharding (colibrì v1.0 README, "Experimental resident CUDA
 * backend": each expert lives whole on one device; JustVugg/colibri README,
 * "Local cluster mode": one batch-union request per layer to each worker).
 * With ep_size = P > 1 a call computes only its shard's part of the layer:
 *   - routed expert e belongs to shard e mod P.  `weights.experts` and
 *     `expert_scales` then hold only this shard's experts, in ascending id
 *     order: expert e (e mod P == ep_rank) is local record e / P;
 *   - the shared experts belong to shard 0 (the other shards pass no shared
 *     weights and compute none);
 *   - the router is not sharded: every shard runs it on the same x and gets
 *     the same topk_idx / topk_w;
 *   - routed slots whose expert belongs to another shard are skipped like
 *     id -1 (no status bit), so the union tables list this shard's experts
 *     only, and y is the shard's partial output
 *         y_r[t] = sum_{j: idx[t][j] mod P == r} w_j o_j + [r == 0] sum_s o_s[t];
 *   - the sum of y_r over the P shards is the layer's output; the caller
 *     forms it (e.g. one all-reduce of y per layer call).
 * Requires 0 <= ep_rank < ep_size <= n_experts (COLI_EINVAL otherwise);
 * ep_size 0 or 1 needs ep_rank 0.  The workspace size depends on the shard
 * (shard 0 holds the shared experts' pairs), so size it with the shard's own
 * cfg. */

/* Expert weights.  One expert "record" is its three matrices stored adjacent
 * (colibrì "JustVugg/colibri" README, "Never wait for the disk twice": an
 * expert's three matrices are read in one go):
 *     gate [Ie][H], up [Ie][H], down [H][Ie]     (Ie = inter or shared_inter)
 * each row-major with K (the reduction dimension) contiguous.
 *   weight_bits 8: one int8 code per weight.
 *   weight_bits 4: two codes per byte; byte j of a row holds element 2j in the
 *                  low nibble and 2j+1 in the high nibble, each stored as
 *                  code + 8 (codes in [-8, 7]).
 *   weight_bits 2: four codes per byte; byte j of a row holds elements
 *                  4j .. 4j+3, element 4j+m in bits 2m and 2m+1, each stored
 *                  as code + 2 (codes in [-2, 1]).
 * Records are consecutive: expert e starts at experts + e * record_bytes,
 * record_bytes = (2*Ie*H + H*Ie) * weight_bits / 8 (with expert-parallel
 * sharding, e is the local record index e / ep_size; see below).
 * Scales are fp32 per output row, consecutive per expert:
 *     expert_scales[e * (2*I + H) + {0..I-1: gate, I..2I-1: up, 2I..: down}]
 * and likewise shared_scales with shared_inter.
 * With group_size 64 (the group-scaled container the colibri GLM-5.2 quick
 * start recommends, "2. Get the model") every run of 64 weights of a row has
 * its own fp32 scale: per expert 3*I*H/64 scales,
 *     gate [I][H/64] | up [I][H/64] | down [H][I/64], each row-major,
 * and an output is sum over Q8_0 blocks b of s[row][b/2] * d_b * (block dot). */
typedef struct coli_moe_weights {
    const void*  experts;        /* [n_experts] records                 */
    const float* expert_scales;  /* [n_experts][2*inter + hidden]       */
    const void*  shared;         /* [n_shared] records (shared_inter)   */
    const float* shared_scales;  /* [n_shared][2*shared_inter + hidden] */
} coli_moe_weights;

/* Bytes of workspace needed for calls with up to max_T positions.  The
 * workspace is caller-owned device memory; it must be prepared once with
 * coli_moe_workspace_init() and may then be reused by any number of calls on
 * one stream.  Returns 0 on an invalid config. */
size_t coli_moe_workspace_size(const coli_moe_cfg* cfg, int32_t max_T);

/* Clears the header of a workspace (enqueued on `stream`): the status word,
 * the device counters and the router's tagged exchange words, i.e. the first
 * min(ws_bytes, 8704) bytes. */
int coli_moe_workspace_init(void* ws, size_t ws_bytes, cudaStream_t stream);

/* Router: "How it works (validated core mechanics)" of the GLM-5.2 write-up
 * ("Colibri (colibrì): GLM-5.2 local inference on 25 GB of RAM")
 * (sigmoid affinities, bias for ranking only, lower id wins ties, unbiased
 * renormalised weights, non-finite input rejected) with DeepSeek-V3 group
 * limiting: group score = sum of the two best biased scores of the group,
 * the topk_group best groups kept (ties to the lower group id), dropped
 * groups never selectable.
 *   x          [T][H]  fp32 activations
 *   router_w   [E][H]  fp32 router weight
 *   corr_bias  [E]     fp32 correction bias (ranking only)
 *   topk_idx   [T][k]  int32 out: expert ids by descending biased score
 *   topk_w     [T][k]  fp32  out: s_sel / sum(s_sel) * routed_scaling_factor
 * Logits are fp32.  A position with a non-finite logit or bias gets ids -1
 * and weights 0, and sets COLI_STATUS_NONFINITE.  T == 0 is a no-op. */
int coli_moe_route(const coli_moe_cfg* cfg, const float* x, int32_t T,
                   const float* router_w, const float* corr_bias,
                   int32_t* topk_idx, float* topk_w,
                   void* ws, size_t ws_bytes, cudaStream_t stream);

/* Q8_0-style activation quantisation (colibrì v1.0 README, "What's
 * implemented", integer-dot kernels): per block of 32 consecutive values,
 * d = amax/127 (IEEE fp32), inv = d > 0 ? 1/d : 0,
 * q = clamp(roundf(x * inv), -127, 127) (half away from zero).
 *   x [T][K] fp32 in, K % 32 == 0;  q [T][K] int8 out;  d [T][K/32] fp32 out.
 * A non-finite value gives code 0 for its element (no status word: this
 * entry point takes no workspace). */
int coli_moe_quantize_act(const float* x, int32_t T, int32_t K,
                          int8_t* q, float* d, cudaStream_t stream);

/* The expert layer for given routing (colibrì v1.0 README, "What's
 * implemented": Q8_0-style int8 activations against packed int4 / int8
 * weights, batch-union MoE, the always-on shared expert; "Experimental Metal
 * backend": the routed-expert SwiGLU; the combine weights are the router's, as
 * "How it works (validated core mechanics)" of the GLM-5.2 write-up gives
 * them): quantise x, build the batch-union
 * tables, run each distinct expert once over its positions (gate/up, SwiGLU,
 * re-quantise h, down) and combine
 *     y[t] = sum_j topk_w[t][j] * o[t,j] + sum_s o_shared_s[t]
 * in fixed j order (deterministic, no floating-point atomics).
 *   x        [T][H] fp32;   topk_idx [T][k] int32 (id -1: slot skipped);
 *   topk_w   [T][k] fp32;   y [T][H] fp32 out.
 * Ids outside [-1, E) are skipped and set COLI_STATUS_BADIDX; non-finite
 * activations set COLI_STATUS_NONFINITE.  T == 0 is a no-op. */
int coli_moe_forward(const coli_moe_cfg* cfg, const coli_moe_weights* weights,
                     const float* x, int32_t T,
                     const int32_t* topk_idx, const float* topk_w, float* y,
                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* The whole layer (the router and the expert layer above, with the passages
 * they cite): coli_moe_route followed by coli_moe_forward, with the
 * same arguments, results and status rules as the two calls (topk_idx and
 * topk_w are outputs here, and the forward part reads them).  For a single
 * position (T == 1, packed int4 or int2) that fits the fused kernel's shared memory,
 * the router runs inside the expert-layer kernel: one launch per call, the
 * shared expert's gate/up rows requested before the routing is known.  The
 * results are bit-identical to the two separate calls. */
int coli_moe_layer(const coli_moe_cfg* cfg, const coli_moe_weights* weights,
                   const float* x, int32_t T,
                   const float* router_w, const float* corr_bias,
                   int32_t* topk_idx, float* topk_w, float* y,
                   void* ws, size_t ws_bytes, cudaStream_t stream);

/* The two launches coli_moe_forward makes, callable separately (e.g. to time
 * the expert kernel alone; the operations and passages of coli_moe_forward).  coli_moe_dispatch quantises x and builds the
 * union tables in ws; coli_moe_experts runs the expert products and the
 * combine from those tables.  Same arguments and rules as coli_moe_forward;
 * coli_moe_experts must follow a coli_moe_dispatch with the same T on the
 * same workspace. */
int coli_moe_dispatch(const coli_moe_cfg* cfg, const float* x, int32_t T,
                      const int32_t* topk_idx, void* ws, size_t ws_bytes,
                      cudaStream_t stream);
int coli_moe_experts(const coli_moe_cfg* cfg, const coli_moe_weights* weights,
                     int32_t T, const float* topk_w, float* y,
                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* Synchronises `stream`, returns the workspace's status bits in *status and
 * clears them. */
int coli_moe_status(void* ws, cudaStream_t stream, uint32_t* status);

/* Static text for a return code. */
const char* coli_moe_strerror(int code);

/* ---- a stack of layers ---------------------------------------------------
 * One decode step through a stack of MoE layers with the hidden state kept
 * on the device between layers (JustVugg/colibri README, "Never wait for the
 * disk twice": the residual stream stays resident on the GPU across layers,
 * COLI_CUDA_PIPE=2).  Layer l runs coli_moe_layer on xs[l]; then a small
 * kernel writes the next layer's input
 *     xs[l+1] = xs[l] + residual[l]            (add_output == 0)
 *     xs[l+1] = (xs[l] + y[l]) + residual[l]   (add_output == 1)
 * in fp32.  Nothing returns to the host between layers; the whole step can
 * be captured once in a CUDA graph and replayed.
 *   layers    [n_layers] per-layer config, weights, router weight and bias;
 *             every layer has the same hidden and top_k (COLI_EINVAL
 *             otherwise); weight formats and the other shapes may differ
 *   xs        [n_layers + 1][T][H] fp32: xs[0] is read, xs[1..] written
 *   residual  [n_layers][T][H] fp32 (NULL: zero)
 *   topk_idx  [n_layers][T][k] int32 out, topk_w [n_layers][T][k] fp32 out
 *   y         [n_layers][T][H] fp32 out: each layer's output
 *   ws        one workspace of at least the largest
 *             coli_moe_workspace_size(layers[l].cfg, T) (COLI_EWORKSPACE
 *             otherwise), prepared with coli_moe_workspace_init
 * Arguments are checked for every layer before anything is enqueued; status
 * bits of all layers accumulate in the workspace's status word. */
typedef struct coli_moe_stack_layer {
    coli_moe_cfg     cfg;
    coli_moe_weights weights;
    const float*     router_w;   /* [E][H] */
    const float*     corr_bias;  /* [E]    */
} coli_moe_stack_layer;

int coli_moe_stack_forward(const coli_moe_stack_layer* layers, int32_t n_layers, int32_t T,
                           float* xs, const float* residual, int32_t add_output,
                           int32_t* topk_idx, float* topk_w, float* y,
                           void* ws, size_t ws_bytes, cudaStream_t stream);

/* ---- inspection (tests) -------------------------------------------------
 * Byte offsets, inside the workspace of coli_moe_workspace_size(cfg, max_T),
 * of the tables and intermediates coli_moe_dispatch / coli_moe_experts leave
 * behind, so that a test can compare them with a reference.  Layouts:
 *   n_entries   int32: routed distinct experts U + n_shared
 *   entry_expert[U+n_shared] int32: ascending routed ids, then E + s
 *   entry_count [U+n_shared] int32: positions per entry
 *   entry_offset[U+n_shared+1] int32: first pair slot of each entry
 *   pair_token  [P] int32, pair_slot_of[T][k] int32 (-1 = skipped)
 *   qx [T][H] int8, dx [T][H/32] fp32  (Q8_0 of x)
 *   qh [P][Imax] int8, dh [P][Imax/32] fp32 (Q8_0 of h per pair slot)
 *   o  [P][H] fp32 (expert output per pair slot)
 * with P = T*k + n_shared*T and Imax = max(inter, shared_inter).  For
 * weight_bits 4, qx and qh hold each group of 8 consecutive codes in the
 * order 0,2,4,6,1,3,5,7 (the order of the low then high nibbles of 4 packed
 * bytes); for weight_bits 2 each group of 16 in the order 0,4,8,12, 1,5,9,13,
 * 2,6,10,14, 3,7,11,15 (the order of the four 2-bit fields of 4 packed bytes);
 * for weight_bits 8 the order is natural. */
typedef struct coli_moe_ws_layout {
    size_t status, n_entries, entry_expert, entry_count, entry_offset,
           pair_token, pair_slot_of, qx, dx, qh, dh, o, total;
} coli_moe_ws_layout;
int coli_moe_workspace_layout(const coli_moe_cfg* cfg, int32_t max_T,
                              coli_moe_ws_layout* out);

/* Test entry point: coli_moe_forward run through the same kernels compiled
 * with a dump of the exact int32 per-32-block dot products:
 *   acc_gu [P][2][Imax][H/32] int32   (gate then up, per pair slot)
 *   acc_d  [P][H][Imax/32]    int32   (down, per pair slot)
 * Either pointer may be NULL.  Slower than coli_moe_forward. */
int coli_moe_forward_dump(const coli_moe_cfg* cfg, const coli_moe_weights* weights,
                          const float* x, int32_t T,
                          const int32_t* topk_idx, const float* topk_w, float* y,
                          void* ws, size_t ws_bytes,
                          int32_t* acc_gu, int32_t* acc_d, cudaStream_t stream);

/* ---- 4-bit microscaled (MX4) experts ---------------------------------------
 * The container of fp4 checkpoints ("JustVugg/colibri" README: MXFP4 expert
 * formats of other families) for activations and weights alike.  A row of K
 * values (K % 32 == 0) is
 *     codes  [K/2]  bytes: element 2j in the low half of byte j, 2j+1 in the
 *                   high half; sign, two exponent bits, one mantissa bit: the
 *                   magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *     scales [K/32] bytes: b stands for 2^(b - 127); 255: the block has no
 *                   value (NaN)
 * and rows of a matrix are consecutive.  Products multiply the values that
 * codes and scales stand for and accumulate in fp32.  Rows have up to
 * COLI_MX4_MAX_K values (COLI_EUNSUPPORTED beyond: the kernels index inside a
 * row, rounded up to their steps, in 32 bits).
 *
 * Value types of the arguments named *_type: */
#define COLI_F32  0
#define COLI_BF16 1
#define COLI_F16  2
#define COLI_MX4  3   /* codes, with their scales in a second argument */

#define COLI_MX4_MAX_K (1 << 30)

/* Quantise rows to MX4: per block of 32 with largest magnitude A,
 * b = max(0, floor(log2 A) + 125) (0 for a block of zeros), every element
 * divided by 2^(b - 127), rounded to the nearest code (ties to the even code)
 * and saturated at 6.  A block holding an infinity or NaN gets b = 255 and
 * codes 0.
 *   x       [T] rows of K values of x_type (COLI_F32, _BF16, _F16), row t at
 *           element t * ldx; any ldx >= K (rows that stay 16-byte aligned are
 *           read in 16-byte pieces, others value by value; x itself is 16-byte
 *           aligned like every pointer here)
 *   codes   [T][K/2] out;  scales [T][K/32] out
 * K % 32 == 0 (COLI_EINVAL otherwise).  T == 0 is a no-op. */
int coli_mx4_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t T, int32_t K,
                      uint8_t* codes, uint8_t* scales, cudaStream_t stream);

/* The values of MX4 rows: out[t][k] (row t at element t * ldo, out_type as
 * x_type above) = code * 2^(b - 127), rounded to out_type once. */
int coli_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t T, int32_t K,
                        void* out, int32_t out_type, int64_t ldo, cudaStream_t stream);

/* Products of MX4 rows, grouped: row p of the activations belongs to group g
 * with offsets[g] <= p < offsets[g+1] and
 *     y[p][n] = sum_k x[p][k] * w[g][n][k].
 *   x_codes [P][K/2], x_scales [P][K/32]
 *   w_codes [G][N][K/2], w_scales [G][N][K/32]
 *   offsets [G+1] int32 on the device, ascending; NULL: one group (G == 1) of
 *           all P rows.  Groups may be empty; values are clamped to [0, P] and
 *           to ascending order; rows of no group are not written.
 *   y       [P] rows of N values of y_type, row p at element p * ldy
 *   ws      a workspace prepared with coli_moe_workspace_init, at least
 *           COLI_MX4_PRODUCT_WS_BYTES (status word: COLI_STATUS_TIMEOUT)
 * K % 32 == 0, any N >= 1, any ldy >= N, 1 <= G <= COLI_MX4_MAX_GROUPS. */
#define COLI_MX4_MAX_GROUPS 1024
#define COLI_MX4_PRODUCT_WS_BYTES 8704u
int coli_mx4_product(const uint8_t* x_codes, const uint8_t* x_scales, int32_t P,
                     const uint8_t* w_codes, const uint8_t* w_scales, int32_t G, int32_t N, int32_t K,
                     const int32_t* offsets, void* y, int32_t y_type, int64_t ldy,
                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* MX4 expert weights: one record per expert, gate [Ie][H], up [Ie][H],
 * down [H][Ie], and the records of their scales in the same order:
 * record bytes 3*Ie*H/2, scale bytes 3*Ie*H/32. */
typedef struct coli_mx4_weights {
    const uint8_t* experts;        /* [n_experts] records (ep shards: as above) */
    const uint8_t* expert_scales;  /* [n_experts][3*inter*hidden/32]            */
    const uint8_t* shared;         /* [n_shared] records (shared_inter)         */
    const uint8_t* shared_scales;
} coli_mx4_weights;

/* Bytes of workspace for coli_mx4_forward with up to max_T positions; the
 * same workspace also serves coli_moe_route with the same cfg.  0 on an
 * invalid config.  Prepared once with coli_moe_workspace_init. */
size_t coli_mx4_workspace_size(const coli_moe_cfg* cfg, int32_t max_T);

/* The expert layer of coli_moe_forward on MX4 weights and activations:
 *     xq = MX4(x[t]);  g = Wg xq, u = Wu xq;  hq = MX4(silu(g) * u);
 *     o = Wd hq;  y[t] = sum_j topk_w[t][j] * o[t,j] + sum_s o_shared_s[t]
 * with fp32 accumulation, fp32 silu and a combine in fixed order.  cfg as for
 * coli_moe_forward with weight_bits 4 and group_size 0 (COLI_EINVAL
 * otherwise) and with its limits (hidden, inter and shared_inter multiples of
 * 128, hidden up to 32768, inter and shared_inter up to 16384, 1024 experts,
 * 32 slots, 8 shared experts); expert-parallel shards as there.
 *   x         [T][H] of x_type, or codes [T][H/2] with x_type COLI_MX4 and
 *             x_scales [T][H/32] (NULL otherwise)
 *   topk_idx  [T][k] int32 (-1: slot skipped);  topk_w [T][k] fp32
 *   y         [T][H] of y_type (COLI_F32, _BF16, _F16)
 * Ids outside [-1, E) are skipped and set COLI_STATUS_BADIDX.  A block of x
 * or h with an infinity or NaN makes its token's outputs NaN and sets
 * COLI_STATUS_NONFINITE.  T == 0 is a no-op. */
int coli_mx4_forward(const coli_moe_cfg* cfg, const coli_mx4_weights* weights,
                     const void* x, int32_t x_type, const uint8_t* x_scales, int32_t T,
                     const int32_t* topk_idx, const float* topk_w, void* y, int32_t y_type,
                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* The norms around a block, with its gate and the scaled residual add:
 *     r  = y * rsqrt(mean(y^2) + eps) * post_w    (post_w NULL: r = y)
 *     x' = x + res_scale * gate * r               (gate NULL: 1; y NULL: x' = x)
 *     n  = x' * rsqrt(mean(x'^2) + eps) * pre_w   (pre_w NULL: no weight)
 * in fp32; x', n and the MX4 codes of n are each rounded once from there.
 *   x, y    [T][H] of `type`, row strides ldx, ldy in elements
 *   gate    `type`; row stride ld_gate, 0: one [H] row for all positions
 *   post_w, pre_w [H] fp32
 *   x_out   [T][H] of `type` (may be x itself), n_out [T][H] of n_type
 *           (`type` or COLI_F32), codes [T][H/2] with scales [T][H/32]
 *           (H % 32 == 0); each may be NULL, not all of them.
 * Any H from 1 to COLI_NORM_MAX_H and any strides; H % 8 == 0 with rows that
 * stay 16-byte aligned is read in 16-byte pieces (the pointers themselves are
 * 16-byte aligned).  T == 0 is a no-op. */
#define COLI_NORM_MAX_H 16384
typedef struct coli_moe_norm_args {
    const void*  x;       int64_t ldx;
    const void*  y;       int64_t ldy;
    const void*  gate;    int64_t ld_gate;
    void*        x_out;   int64_t ld_x_out;
    void*        n_out;   int64_t ld_n_out;
    const float* post_w;
    const float* pre_w;
    uint8_t*     codes;
    uint8_t*     scales;
    float        res_scale;
    float        eps;
    int32_t      type;
    int32_t      n_type;
} coli_moe_norm_args;
int coli_moe_block_norm(const coli_moe_norm_args* args, int32_t T, int32_t H, cudaStream_t stream);

/* ---- 8-bit codes with a scale for each token and each channel --------------
 * The int8 container of the expert records above (int8 codes and one fp32 scale
 * per output row: colibri v1.0 README, "What's implemented") against activations
 * that carry one scale per position, and the steps between a router's logits and
 * the layer's output, each on its own: selection of experts, grouping of the
 * routed pairs, codes of activations, products, weighted sum.  Together they
 * are the expert layer for activations quantised per token. */

/* Selection of experts from scores ("How it works (validated core mechanics)"
 * of the GLM-5.2 write-up, as for coli_moe_route, and the variants of other
 * families):
 *     s = softmax(l) over all experts, or sigmoid(l);   v = s + bias
 *     the topk_group best groups stay: by the sum of their two best v, or by
 *     their best (ties to the lower group)
 *     topk_idx = the top_k best v of them, descending (ties to the lower id)
 *     topk_w = s of these, with renorm divided by their sum, times scaling
 * Without a bias the logits themselves rank the experts and the groups, also
 * where scores saturate or underflow to the same fp32 value (a group by its two
 * best logits; sums of two scores that differ by less than fp32 tells apart,
 * from each other and in their distance from 0, 1 and 2, count as equal).
 *   x          logits [T] rows of n_experts values of `type` (COLI_F32, _BF16,
 *              _F16) with row stride ldx; or, with router_w, the hidden state
 *              [T][hidden] fp32 (ldx == hidden, hidden % 16 == 0), whose logits
 *              x . router_w^T are computed in fp32 first
 *   router_w   [n_experts][hidden] fp32, or NULL
 *   bias       [n_experts] fp32, or NULL
 *   topk_idx   [T][top_k] int32 out; topk_w [T][top_k] fp32 out
 *   ws         a workspace prepared with coli_moe_workspace_init: with router_w
 *              of coli_moe_select_workspace_size bytes; else 256 bytes, or NULL
 *              (status bits are then lost)
 * An expert whose logit or bias is -inf takes no part; it adds nothing to its
 * group's score, and a position with fewer than top_k others gets id -1 and
 * weight 0 in the slots that are left.  Weights whose sum is 0 stay 0.  Any other
 * non-finite logit or bias, and any non-finite logit of a hidden state, gives a
 * position ids -1 and weights 0 and sets COLI_STATUS_NONFINITE.  Limits: n_experts <= 1024, a multiple of n_groups <=
 * 32, top_k <= 32 and <= the experts of topk_group groups; with router_w at most 4194240 positions.  T == 0 is a
 * no-op. */
#define COLI_SCORE_SIGMOID 0
#define COLI_SCORE_SOFTMAX 1
#define COLI_GROUP_TOP2    0
#define COLI_GROUP_MAX     1
typedef struct coli_moe_select_args {
    const void*  x;
    int64_t      ldx;
    const float* router_w;
    const float* bias;
    int32_t*     topk_idx;
    float*       topk_w;
    void*        ws;
    size_t       ws_bytes;
    int32_t      type;
    int32_t      hidden;
    int32_t      n_experts;
    int32_t      n_groups;
    int32_t      topk_group;
    int32_t      top_k;
    int32_t      score;
    int32_t      group_score;
    int32_t      renorm;
    float        scaling;
} coli_moe_select_args;
int coli_moe_select(const coli_moe_select_args* args, int32_t T, cudaStream_t stream);

/* Bytes of workspace for coli_moe_select with router_w and up to max_T
 * positions; 0 for sizes outside its limits. */
size_t coli_moe_select_workspace_size(int32_t max_T, int32_t hidden, int32_t n_experts);

/* The routed pairs in expert order (the batch union of "What's implemented"):
 * pair (t, j) with id e = topk_idx[t][j] joins group e; groups ascend, and inside
 * a group pairs keep the order of t * top_k + j.
 *   topk_idx [T][top_k] int32 (-1: slot skipped)
 *   offsets  [groups + 1] int32 out: first pair of each group, and the end
 *   rows     [T * top_k] int32 out: position t of each pair; entries behind
 *            the last pair are left as they were
 *   slots    [T][top_k] int32 out: place of the pair, -1 for skipped slots
 * With ep_size > 1 the groups are the experts of shard ep_rank (e mod ep_size ==
 * ep_rank) as local records e / ep_size; slots of other shards are skipped.  Ids
 * outside [-1, n_experts) are skipped and set COLI_STATUS_BADIDX.  ws: of
 * coli_moe_group_workspace_size bytes, prepared with coli_moe_workspace_init.
 * T == 0 writes the offsets (all 0). */
int coli_moe_group(const int32_t* topk_idx, int32_t T, int32_t top_k, int32_t n_experts, int32_t ep_rank, int32_t ep_size,
                   int32_t* offsets, int32_t* rows, int32_t* slots, void* ws, size_t ws_bytes, cudaStream_t stream);
size_t coli_moe_group_workspace_size(int32_t max_T, int32_t top_k, int32_t n_experts);

/* y[t] = add[t] + sum_j topk_w[t][j] * o[slots[t][j]], in fp32 and in this
 * order, rounded once.
 *   o      [P] rows of H values of o_type, row stride ldo
 *   slots  [T][top_k] int32; slots outside [0, P) add nothing, whatever their
 *          weight
 *   add    [T] rows of y_type, row stride ld_add, or NULL; may be y itself
 *   y      [T] rows of y_type, row stride ldy
 * Any H, top_k and strides; rows that stay 16-byte aligned with H % 8 == 0 are
 * read in 16-byte pieces.  T == 0 is a no-op. */
int coli_moe_combine(const void* o, int32_t o_type, int64_t ldo, int32_t P, const int32_t* slots, const float* topk_w, int32_t T,
                     int32_t top_k, int32_t H, const void* add, int64_t ld_add, void* y, int32_t y_type, int64_t ldy, cudaStream_t stream);

/* 8-bit codes of rows with one scale a row: with A the row's largest magnitude,
 * scale = A / 127 and code = value * 127 / A rounded to the nearest whole number,
 * ties to even.  A row with A < 2^-100 gets scale 0 and codes 0, a row that
 * holds an infinity or NaN scale NaN and codes 0.
 *   x       [T] rows of x_type, row stride ldx; act COLI_ACT_NONE: K values;
 *           COLI_ACT_SWIGLU: 2 K values, gate then up, and the row quantised is
 *           silu(gate) * up in fp32
 *   codes   [T] rows of K int8 out, row stride ldc (bytes behind K are left);
 *   scales  [T] fp32 out
 * Any K from 1 to COLI_I8_MAX_K.  T == 0 is a no-op. */
#define COLI_ACT_NONE   0
#define COLI_ACT_SWIGLU 1
#define COLI_I8_MAX_K   131071
int coli_i8_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t T, int32_t K, int32_t act, int8_t* codes, int64_t ldc, float* scales,
                     cudaStream_t stream);

/* out[t][k] = codes[t][k] * scales[t], rounded to out_type once from fp32. */
int coli_i8_dequantize(const int8_t* codes, int64_t ldc, const float* scales, int32_t T, int32_t K, void* out, int32_t out_type, int64_t ldo,
                       cudaStream_t stream);

/* Products of 8-bit codes, grouped: row p of y belongs to group g with offsets[g]
 * <= p < offsets[g+1] and, with r = rows[p] (rows NULL: r = p),
 *     y[p][n] = x_scales[r] * w_scales[g][n] * sum_k x_codes[r][k] * w_codes[g][n][k].
 * The sum is exact in 32-bit integers; it is rounded to fp32, scaled by x_scales,
 * then by w_scales.
 *   x_codes [x_rows] rows of K int8, row stride ldx;  x_scales [x_rows] fp32
 *   rows    [P] int32 on the device, or NULL (P <= x_rows).  A row of y whose
 *           activation row is outside [0, x_rows) is NaN and sets
 *           COLI_STATUS_BADIDX
 *   w_codes [G][N] rows of K int8, row stride ldw, group stride w_group (bytes);
 *           w_scales [G][N] fp32, group stride w_scale_group (elements).  The
 *           matrices of int8 expert records are such weights: gate and up of
 *           all experts are [E][2 * inter] rows of hidden codes with w_group
 *           3 * inter * hidden, down [E][hidden] rows of inter codes at
 *           2 * inter * hidden of each record; their scales stand at 0 and at
 *           2 * inter of every 2 * inter + hidden
 *   offsets [G+1] int32 on the device, ascending; NULL: one group (G == 1) of all
 *           P rows.  Groups may be empty; values are clamped to [0, P] and to
 *           ascending order; rows of no group are not written
 *   y       [P] rows of N values of y_type, row stride ldy
 *   ws      prepared with coli_moe_workspace_init, of
 *           coli_i8_product_workspace_size(P, K) bytes (status word)
 * Any N >= 1 and any K from 1 to COLI_I8_MAX_K; ldx, ldw and w_group are multiples of
 * 16 (COLI_EALIGN otherwise), so that every row begins on a 16-byte boundary. */
#define COLI_I8_MAX_GROUPS 1024
typedef struct coli_i8_product_args {
    const int8_t*  x_codes;   int64_t ldx;
    const float*   x_scales;
    const int32_t* rows;
    const int8_t*  w_codes;   int64_t ldw;   int64_t w_group;
    const float*   w_scales;  int64_t w_scale_group;
    const int32_t* offsets;
    void*          y;         int64_t ldy;
    void*          ws;        size_t  ws_bytes;
    int32_t        x_rows;
    int32_t        P;
    int32_t        G;
    int32_t        N;
    int32_t        K;
    int32_t        y_type;
} coli_i8_product_args;
int coli_i8_product(const coli_i8_product_args* args, cudaStream_t stream);
size_t coli_i8_product_workspace_size(int32_t max_P, int32_t K);

/* ---- no-allocation variant ----------------------------------------------
 * The pages have no counterpart to this entry point; it exists for callers
 * that cannot allocate device memory to pass a workspace -- a plain C or FFI
 * host that links only this library and owns no allocator, or a runtime that
 * keeps the whole device-memory budget and forbids stray cudaMalloc calls.
 *
 * coli_moe_forward_static computes exactly what coli_moe_forward computes,
 * with its workspace taken from one static device array of
 * COLI_STATIC_WS_BYTES inside the library (held on every GPU that loads the
 * library until the process exits).  It calls no cudaMalloc, cudaFree or
 * other allocating routine.  The caller still passes x, routing and y.
 *   - Limit: the layer's workspace for T positions must fit in
 *     COLI_STATIC_WS_BYTES (24 MiB: the GLM-5.2-shaped layer up to T = 76);
 *     larger T returns COLI_EWORKSPACE and enqueues nothing.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it per
 *     device ordinal for the life of the process; make that first call before
 *     any stream capture.  The cache assumes the runtime's primary context:
 *     after cudaDeviceReset, or from another driver-API context on the same
 *     device, the cached address is stale and must not be used (this entry
 *     point then gives undefined results).
 *   - Every call on a device shares the one array: calls that overlap on the
 *     GPU (different streams, or host threads without ordering) race and give
 *     wrong results.  Calls ordered on one stream are safe; each call rewrites
 *     every table and counter it reads.
 *   - Device status bits (non-finite input, expert ids outside [-1, E), an
 *     expired bounded wait) are recorded in the array but cannot be read or
 *     cleared by the caller.  In those cases y is undefined: rows of
 *     positions with non-finite x, or with an out-of-range id, and every row
 *     after an expired wait may hold anything.  Callers that need to detect
 *     them use coli_moe_forward with a workspace and coli_moe_status. */
#define COLI_STATIC_WS_BYTES (24u << 20)
int coli_moe_forward_static(const coli_moe_cfg* cfg, const coli_moe_weights* weights,
                            const float* x, int32_t T,
                            const int32_t* topk_idx, const float* topk_w, float* y,
                            cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* COLI_MOE_H */
