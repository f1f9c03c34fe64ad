/*
 * mxmoe.h -- C ABI of libmxmoe.so: a mixture-of-experts layer whose expert
 * weights are MXFP4, for AMD MI355X (gfx950).
 *
 * The layer, as the pages describe it:
 *   - top-k routing over E experts (256 experts / top-6 for the
 *     DeepSeek-V4-Flash shape: ktransformers issue #2172, "Environment";
 *     896 experts / top-16 for Kimi-K3: "Kimi-K3 SM120 FlashInfer MXFP4
 *     MoE", Phase-0 audit table);
 *   - dispatch of the routed tokens to the experts (issue #2172, "Impact");
 *   - expert FC1 (gate and up, twice FC2's inner width for a gated
 *     activation: Kimi-K3 page, on-machine evidence), the gated activation,
 *     expert FC2, with MXFP4 weights against bf16 or MXFP8 activations
 *     (Kimi-K3 page, goal; issue #2172 title);
 *   - the weighted top-k combine that ends a fused MoE (Kimi-K3 page, goal);
 *   - layerwise, double-buffered streaming of expert weights from host
 *     memory during prefill, instead of "load all experts, compute, hard
 *     sync" per layer (issue #2172, "Impact" and "Background / motivation").
 *
 * Number formats (OCP Microscaling Formats v1.0): an MXFP4 matrix [N][K] is
 * stored as packed FP4 E2M1 codes uint8 [N][K/2] (element 2j in the low
 * nibble, 2j+1 in the high nibble) plus E8M0 scales uint8 [N][K/32], one
 * per 32 consecutive elements along K.  MXFP8 activations are E4M3 codes
 * uint8 [rows][K] plus E8M0 scales uint8 [rows][K/32].  bf16 tensors are
 * passed as uint16 bit patterns.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are HIP device memory (or managed memory)
 *     on the current device; "host" pointers are host memory.  The caller
 *     owns every buffer, stream and event; the library never frees or
 *     keeps a pointer past the enqueued work.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Calls only enqueue: none waits for the device.
 *   - All argument checks run before anything is enqueued: a call that
 *     returns an error has enqueued nothing.  The detail of the last error
 *     on the calling thread is in moe_last_error_message().
 *   - Faults inside kernels surface at the caller's next synchronisation
 *     as HIP errors.
 *   - Only gfx950 devices are accepted (MOE_ERR_UNSUPPORTED_DEVICE
 *     otherwise); there is no fallback path.
 *   - The library reads no environment variables.
 */
#ifndef MXMOE_H
#define MXMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MXMOE_ABI_VERSION 3

/* Every enum value is explicit and checked by the binding at load time:
 * a value that means one thing on one side of the boundary and another on
 * the other silently breaks gated activations (Kimi-K3 page, on-machine
 * evidence: the activation enum that disagreed between Python and C++). */
typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,       /* null pointer, bad enum value, negative size */
  MOE_ERR_SHAPE = 2,             /* sizes violate the layout rules stated per call */
  MOE_ERR_UNSUPPORTED_DEVICE = 3,/* current device is not gfx950 */
  MOE_ERR_NOT_PINNED = 4,        /* host weights are not page-locked */
  MOE_ERR_WORKSPACE = 5,         /* workspace missing or smaller than the size query */
  MOE_ERR_HIP = 6,               /* a HIP runtime call or launch failed */
  MOE_ERR_NOT_IMPLEMENTED = 7    /* a valid combination this build does not provide */
} moe_status;

typedef enum moe_act_dtype {     /* the A operand of a grouped GEMM */
  MOE_ACT_BF16 = 0,
  MOE_ACT_MXFP8_E4M3 = 1
} moe_act_dtype;

typedef enum moe_out_dtype {     /* the output of a grouped GEMM / intermediate */
  MOE_OUT_FP32 = 0,
  MOE_OUT_BF16 = 1,
  MOE_OUT_MXFP8_E4M3 = 2,
  MOE_OUT_FP16 = 3               /* rows of moe_combine only (experts with fp16 weights) */
} moe_out_dtype;

typedef enum moe_epilogue {
  MOE_EPI_NONE = 0,              /* C = A * W^T */
  MOE_EPI_SWIGLU_SPLIT = 1,      /* W rows [0,N/2) gate, [N/2,N) up; C[:, i] = silu(g_i) * u_i */
  MOE_EPI_SWIGLU_INTERLEAVED = 2 /* W row 2i gate, 2i+1 up; C[:, i] = silu(g_i) * u_i */
} moe_epilogue;

typedef enum moe_chain {         /* how stacked layers feed each other */
  MOE_CHAIN_RMS = 0,             /* x_{L+1}[t] = bf16(y_L[t] / rms(y_L[t])) */
  MOE_CHAIN_INDEPENDENT = 1      /* every layer reads x_0 */
} moe_chain;

typedef enum moe_weight_format { /* how a weight matrix and its scales sit in memory */
  MOE_W_CANONICAL = 0,           /* packed [E][N][K/2], scales [E][N][K/32] (row-major) */
  MOE_W_TILED = 1                /* the load-time tiling of moe_mxfp4_tile_weights */
} moe_weight_format;

typedef enum moe_expert_copy {   /* which experts the streamed prefill moves to HBM per layer */
  MOE_COPY_ALL = 0,              /* every expert of the layer (one copy-engine transfer) */
  MOE_COPY_ROUTED = 1,           /* only the experts the layer's routing hits (a copy kernel) */
  MOE_COPY_AUTO = 2              /* ROUTED when T <= routed_copy_max_tokens, else ALL */
} moe_expert_copy;

typedef enum moe_float_dtype {   /* tensors of the dense projections */
  MOE_FLOAT_BF16 = 0,
  MOE_FLOAT_FP16 = 1,
  MOE_FLOAT_FP32 = 2
} moe_float_dtype;

typedef enum moe_gate_act {      /* the activation of the dense projections' gated epilogue */
  MOE_GATE_SILU = 0,             /* z / (1 + e^-z) */
  MOE_GATE_GELU = 1              /* tanh form: z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) */
} moe_gate_act;

typedef enum moe_enum_kind {
  MOE_ENUM_STATUS = 0, MOE_ENUM_ACT = 1, MOE_ENUM_OUT = 2, MOE_ENUM_EPI = 3, MOE_ENUM_CHAIN = 4,
  MOE_ENUM_WFORMAT = 5, MOE_ENUM_COPY = 6, MOE_ENUM_FLOAT = 7, MOE_ENUM_GATE = 8
} moe_enum_kind;

/* ------------------------------------------------------------ queries -- */

int         moe_abi_version(void);
/* Static string for a status code; "unknown status" otherwise. */
const char* moe_status_string(int status);
/* Detail of the last failing call on this thread ("" if none).  Valid until
 * the next call on the same thread. */
const char* moe_last_error_message(void);
/* Name of enum value `value` of kind `kind` (e.g. "MOE_EPI_SWIGLU_SPLIT"),
 * or NULL if the value is not defined.  Lets a binding assert that its
 * mirror of every enum agrees with this header. */
const char* moe_enum_name(int kind, int value);
/* 1 if the current HIP device is a gfx950, 0 if not, -1 on a HIP error. */
int         moe_device_supported(void);

/* ------------------------------------------------------------ routing -- */

/* Top-k routing (the router of a top-k MoE: issue #2172 "Environment",
 * Kimi-K3 Phase-0 audit table).
 *   logits   device fp32 [T][E], row-major.
 *   topk_ids device int32 [T][k] out: expert ids, best first.  Order:
 *            logit descending, equal logits -> lower expert id first;
 *            -0.0 equals +0.0; NaN sorts after every number.
 *   topk_w   device fp32 [T][k] out: softmax over the E logits,
 *            renormalised over the k kept = exp(l_j - max) / sum_j'.
 * Sizes: 0 <= T <= 2^26 - 4 (T == 0 enqueues nothing), 1 <= E <= 1024,
 * 1 <= k <= min(E, 64).
 */
moe_status moe_route(const float* logits, int32_t T, int32_t E, int32_t k,
                     int32_t* topk_ids, float* topk_w, void* stream);

/* ------------------------------------------------------- permutation -- */

/* Bytes of device workspace moe_permute needs. */
size_t     moe_permute_workspace_size(int32_t T, int32_t E, int32_t k);

/* Stable counting sort of the T*k (token, slot) pairs by expert: the
 * dispatch of routed tokens to the experts (issue #2172, "Impact").
 *   topk_ids       device int32 [T][k], values in [0, E).
 *   expert_offsets device int32 [E+1] out: exclusive prefix sum of the
 *                  per-expert counts; expert_offsets[E] == T*k.
 *   perm_src       device int32 [T*k] out: permuted row r -> flat index
 *                  f = t*k + j; within an expert, rows are in increasing f.
 *   dest_row       device int32 [T*k] out: f -> permuted row (the inverse).
 *   workspace      device, >= moe_permute_workspace_size(T, E, k) bytes.
 * Sizes: T >= 0, 1 <= E <= 8192, 1 <= k <= E, T*k < 2^31.
 * Ids outside [0, E) are undefined behaviour (not checked on the device).
 */
moe_status moe_permute(const int32_t* topk_ids, int32_t T, int32_t E, int32_t k,
                       int32_t* expert_offsets, int32_t* perm_src, int32_t* dest_row,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------- grouped MXFP4 GEMM -- */

typedef struct moe_gemm_args {
  const void*    a;              /* device: bf16 [a_rows][K] or E4M3 [a_rows][K] */
  const uint8_t* a_scales;       /* device E8M0 [a_rows][K/32] for MXFP8 A; NULL for bf16 */
  const int32_t* a_gather;       /* device int32 [rows] or NULL.  A row of permuted row r is
                                    a_gather[r] / a_gather_div (FC1 gathers token rows of x
                                    with perm_src and div = k); NULL: A row r */
  const uint8_t* w_packed;       /* device [E][N][K/2] packed E2M1 */
  const uint8_t* w_scales;       /* device [E][N][K/32] E8M0 */
  const int32_t* expert_offsets; /* device int32 [E+1] from moe_permute */
  void*          c;              /* device out [rows][N_out]: N_out = N/2 for SWIGLU, else N */
  uint8_t*       c_scales;       /* device out E8M0 [rows][N_out/32] for MXFP8 C; else NULL */
  int32_t        a_dtype;        /* moe_act_dtype */
  int32_t        a_gather_div;   /* >= 1 */
  int32_t        a_rows;         /* rows of A (T when gathering from x, else rows) */
  int32_t        rows;           /* permuted rows = expert_offsets[E] = T*k */
  int32_t        E, N, K;
  int32_t        epilogue;       /* moe_epilogue */
  int32_t        c_dtype;        /* moe_out_dtype (MXFP8 only with a SWIGLU epilogue) */
  int32_t        w_format;       /* moe_weight_format of w_packed / w_scales; MOE_W_TILED
                                    needs K % 512 == 0 and N % 256 == 0 and weights tiled
                                    with this call's epilogue */
} moe_gemm_args;

size_t     moe_grouped_gemm_workspace_size(const moe_gemm_args* args);

/* For every expert e with rows [off[e], off[e+1]):
 *   C[r][:] = epilogue( A[row(r)][:] . dequant(W[e])^T ),  dequant(W)[n][kk] =
 *   E2M1(code[n][kk]) * 2^(scale[n][kk/32] - 127), accumulated in fp32.
 * FC1 of the layer is this call with a SWIGLU epilogue (N = 2*I, K = H);
 * FC2 is this call with MOE_EPI_NONE (N = H, K = I).  bf16 A runs on bf16
 * MFMA with the weights expanded exactly to bf16; MXFP8 A runs on the
 * scaled FP8 x FP4 MFMA with both E8M0 scales applied inside it.
 * MXFP8 C (MOE_OUT_MXFP8_E4M3; SWIGLU epilogue and K % 512 == 0, else
 * MOE_ERR_NOT_IMPLEMENTED): each row's N_out values are cut into 32-element
 * blocks; a block with largest magnitude amax gets the E8M0 exponent X, the
 * smallest integer with amax * 2^-X <= 448 (so no element saturates;
 * clamped to [-127, 127]; amax == 0 gives X = -127), stored as X + 127 in
 * c_scales, and each element v becomes the E4M3 code nearest to v * 2^-X,
 * ties to even.  This is the intermediate of the MXFP8 x MXFP4 layer, which
 * FC2 then reads as MXFP8 A.
 * Shape rules (MOE_ERR_SHAPE): K % 32 == 0, N % 32 == 0, N % 64 == 0 for
 * SWIGLU, N_out % 32 == 0 for MXFP8 C, rows >= 0, 1 <= E; for K % 512 == 0
 * also a gathered A below 4 GiB and one expert's packed weights below 4 GiB.
 */
moe_status moe_mxfp4_grouped_gemm(const moe_gemm_args* args, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * grouped GEMM, with the same arguments, kernels and results as
 * moe_mxfp4_grouped_gemm, but its scratch (the planner's tile lists, tile
 * counts and unit counters) lives in a device array inside the library of
 * MXMOE_STATIC_SCRATCH_BYTES bytes, which each device the library runs on
 * holds until the process ends.  The call allocates and frees nothing.
 * Limit: moe_grouped_gemm_workspace_size(args) <= MXMOE_STATIC_SCRATCH_BYTES
 * (about rows / 32 + E <= 32 700; e.g. rows up to ~1 000 000 at E = 896),
 * MOE_ERR_WORKSPACE above it (nothing enqueued).  Every call on a device
 * shares that device's array: calls that overlap on one device (on different
 * streams, or from different threads) race and must not be issued; calls
 * ordered on one stream are safe.  The array keeps the last call's contents;
 * the planner rewrites every word the GEMM reads, so nothing needs clearing.
 * Errors as for moe_mxfp4_grouped_gemm. */
#define MXMOE_STATIC_SCRATCH_BYTES (1u << 20)
moe_status moe_mxfp4_grouped_gemm_static(const moe_gemm_args* args, void* stream);

/* ----------------------------------------------- load-time weight tiling -- */

/* Load-time repacking of one weight matrix into the order the grouped GEMM
 * streams it: the counterpart of the MXFP4 weight repack and E8M0 scale
 * swizzle that ktransformers issue #2172 (comments on the Marlin MoE path)
 * describes, where raw and repacked copies were both kept; here the caller
 * frees the canonical copy once the tiled one is made.  A 256-column slice of the
 * GEMM ("n-tile") over 128 K elements is one contiguous 16 KB block, already
 * in the slot order the kernels read from LDS, so every weight load is 1 KB
 * of consecutive bytes; an n-tile's E8M0 scales for 512 K elements are one
 * contiguous 4 KB block.  For a SWIGLU epilogue an n-tile holds 128 gate
 * rows and their 128 up rows, in groups of 32 gate then the 32 matching up
 * rows, so the tiling depends on the epilogue the matrix is used with (FC1:
 * its SWIGLU layout; FC2: MOE_EPI_NONE).
 *   w_packed, w_scales  device canonical [E][N][K/2], [E][N][K/32] (input)
 *   t_packed, t_scales  device out, moe_tiled_weight_bytes(E, N, K, 0 / 1)
 *                       bytes (the same byte counts as the canonical arrays)
 * Sizes: E >= 1, K % 512 == 0, N % 256 == 0 (MOE_ERR_SHAPE otherwise);
 * epilogue a moe_epilogue.  Input and output must not overlap.  Enqueued on
 * `stream`; nothing else is written.
 * moe_mxfp4_untile_weights is the exact inverse (tiled -> canonical), with
 * the same arguments in the other direction.
 * moe_tiled_weight_bytes returns 0 for sizes the tiling does not take.
 */
size_t     moe_tiled_weight_bytes(int32_t E, int32_t N, int32_t K, int32_t which);
moe_status moe_mxfp4_tile_weights(const uint8_t* w_packed, const uint8_t* w_scales, int32_t E, int32_t N,
                                  int32_t K, int32_t epilogue, uint8_t* t_packed, uint8_t* t_scales,
                                  void* stream);
moe_status moe_mxfp4_untile_weights(const uint8_t* t_packed, const uint8_t* t_scales, int32_t E, int32_t N,
                                    int32_t K, int32_t epilogue, uint8_t* w_packed, uint8_t* w_scales,
                                    void* stream);

/* ------------------------------------------------------------ combine -- */

/* Weighted top-k combine that ends the fused MoE (Kimi-K3 page, goal):
 *   out[t][h] = sum_{j = 0..k-1, ascending} topk_w[t][j] * y[dest_row[t*k+j]][h]
 * in fp32.  A gather-reduce: no atomics, run-to-run deterministic.
 *   y        device [T*k][H] in permuted row order; y_dtype is a moe_out_dtype
 *            (moe_combine_backward's is a moe_float_dtype, with other numbers):
 *            MOE_OUT_FP32, MOE_OUT_BF16 or MOE_OUT_FP16.
 *   dest_row a row outside [0, T*k) is not there and adds nothing (another
 *            device holds its expert: each device's out is its experts' part
 *            of the sum).
 *   out      device fp32 [T][H].
 *   x_next   device bf16 [T][H] or NULL: if given, also writes
 *            bf16(out[t] / sqrt(mean_h out[t][h]^2)) (the stacked-layer
 *            rule MOE_CHAIN_RMS).
 * Sizes: T >= 0, k >= 1, H >= 1, H % 8 == 0, fewer than 2^32 threads: a token
 * takes H / 8 of them, in whole waves, 1024 at most (fp32 rows: 512), so that
 * T < 2^22 always fits.
 */
moe_status moe_combine(const void* y, int32_t y_dtype, const int32_t* dest_row,
                       const float* topk_w, int32_t T, int32_t k, int32_t H,
                       float* out, uint16_t* x_next, void* stream);

/* ------------------------------------------------ one resident layer -- */

typedef struct moe_layer_args {
  int32_t        T, H, I, E, k;
  int32_t        layout;         /* MOE_EPI_SWIGLU_SPLIT or MOE_EPI_SWIGLU_INTERLEAVED */
  int32_t        act_dtype;      /* moe_act_dtype of x */
  int32_t        inter_dtype;    /* moe_out_dtype of the SwiGLU output fed to FC2:
                                    MOE_OUT_BF16 or MOE_OUT_MXFP8_E4M3 */
  const float*   logits;         /* device fp32 [T][E] */
  const void*    x;              /* device bf16 [T][H] or E4M3 [T][H] */
  const uint8_t* x_scales;       /* device E8M0 [T][H/32] (MXFP8 x only) */
  const uint8_t* w1_packed;      /* device [E][2I][H/2] */
  const uint8_t* w1_scales;      /* device [E][2I][H/32] */
  const uint8_t* w2_packed;      /* device [E][H][I/2] */
  const uint8_t* w2_scales;      /* device [E][H][I/32] */
  float*         out;            /* device fp32 [T][H] */
  uint16_t*      x_next;         /* device bf16 [T][H] or NULL (see moe_combine) */
  void*          workspace;      /* device, >= moe_layer_workspace_size() */
  size_t         workspace_bytes;
  int32_t        w_format;       /* moe_weight_format of both weight matrices (tiled: W1
                                    with `layout`, W2 with MOE_EPI_NONE) */
} moe_layer_args;

/* Bytes of workspace for a layer of these sizes (routing arrays, the
 * intermediate and FC2's output included). */
size_t     moe_layer_workspace_size(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                                    int32_t inter_dtype);

/* Byte offsets, inside the layer workspace, of the routing arrays the layer
 * writes (for inspection after the call): which = 0 topk_ids, 1 topk_w,
 * 2 expert_offsets, 3 perm_src, 4 dest_row.  (size_t)-1 for a bad `which`. */
size_t     moe_layer_workspace_offset(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                                      int32_t inter_dtype, int32_t which);

/* route -> permute -> FC1 + SwiGLU -> FC2 -> combine, all on `stream`. */
moe_status moe_layer_forward(const moe_layer_args* args, void* stream);

/* ------------------------------------------------ captured layer ------ */

/* Graph capture and replay of one resident layer ("Kimi-K3 SM120 FlashInfer
 * MXFP4 MoE" page, Phase-1 gates, item 5: token counts 1/2/8/32 under graph
 * capture/replay).
 *
 * moe_layer_graph_create validates *args exactly as moe_layer_forward does,
 * captures one moe_layer_forward(args) on `stream` into a HIP graph and
 * instantiates it.  Nothing runs during the capture.  The graph keeps every
 * pointer of *args (not the struct itself): a replay reads the inputs'
 * contents at replay time and writes the same outputs and workspace, so
 * replays on one handle must not overlap each other or a moe_layer_forward
 * on the same workspace.  T, the weights and the workspace are fixed per
 * handle.  `stream` must be a created stream (capture on the null stream
 * is MOE_ERR_INVALID_ARG) with no other capture in progress; it is left in
 * normal (non-capturing) mode on every return.  On failure *graph is NULL
 * and the status is forward's (or MOE_ERR_HIP for a capture/instantiate
 * failure).  The handle is host memory owned by the caller until
 * moe_layer_graph_destroy.
 *
 * moe_layer_graph_launch enqueues one replay on `stream` (any stream of the
 * device the graph was captured on; MOE_ERR_INVALID_ARG on another device).
 * Output ordering is that of a kernel launch on `stream`.
 *
 * moe_layer_graph_destroy frees the handle (NULL is accepted); the caller
 * first makes sure no replay is still running.
 */
typedef struct moe_layer_graph moe_layer_graph;
moe_status moe_layer_graph_create(const moe_layer_args* args, void* stream, moe_layer_graph** graph);
moe_status moe_layer_graph_launch(moe_layer_graph* graph, void* stream);
moe_status moe_layer_graph_destroy(moe_layer_graph* graph);

/* ------------------------------------------------ streamed prefill ---- */

typedef struct moe_streamed_args {
  int32_t        num_layers, T, H, I, E, k;
  int32_t        layout;         /* MOE_EPI_SWIGLU_SPLIT or _INTERLEAVED */
  int32_t        chain;          /* moe_chain */
  int32_t        depth;          /* 2: double-buffered (copy of L+1 overlaps compute of L);
                                    1: serialized (copy, compute, copy, ...) for comparison */
  int32_t        num_blobs;      /* distinct host blobs; layer L uses blob L % num_blobs */
  const void* const* host_blobs; /* host array of num_blobs page-locked host pointers; each
                                    blob = W1p | S1 | W2p | S2, each section starting at a
                                    multiple of 256 bytes (moe_blob_section_offset) */
  size_t         blob_bytes;     /* >= moe_blob_bytes(H, I, E) */
  void*          device_slot[2]; /* device, each >= blob_bytes (slot[1] unused at depth 1) */
  const float*   logits;         /* device fp32 [num_layers][T][E] */
  const uint16_t* x;             /* device bf16 [T][H]: the first layer's input */
  float*         out;            /* device fp32 [T][H]: the last layer's output */
  uint16_t*      layer_inputs;   /* device bf16 [num_layers][T][H] or NULL: every layer's
                                    input, recorded for per-layer checks */
  void*          events;         /* host array of num_layers*4 hipEvent_t or NULL: recorded at
                                    copy start, copy end (copy stream), compute start, compute
                                    end (compute stream) of every layer */
  void*          workspace;      /* device, >= moe_streamed_workspace_size() */
  size_t         workspace_bytes;
  int32_t        w_format;       /* moe_weight_format of the blobs' W1/S1 and W2/S2 sections */
  int32_t        expert_copy;    /* moe_expert_copy */
  int32_t        routed_copy_max_tokens; /* MOE_COPY_AUTO: the largest T that copies routed
                                    experts only (the token threshold below which a
                                    layer's batch leaves most experts unused) */
} moe_streamed_args;

/* Bytes of one layer's weight blob, and the byte offset of its sections:
 * which = 0 W1p, 1 S1, 2 W2p, 3 S2. */
size_t     moe_blob_bytes(int32_t H, int32_t I, int32_t E);
size_t     moe_blob_section_offset(int32_t H, int32_t I, int32_t E, int32_t which);
size_t     moe_streamed_workspace_size(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k);

/* Layerwise streamed prefill (issue #2172, "Background / motivation": the
 * double-buffered layerwise pipeline that replaces the serialized
 * per-layer H2D chain).  For L = 0..num_layers-1: the copy stream fills
 * slot (L % 2) with blob (L % num_blobs) once the compute of layer L-2
 * (the slot's previous user) is done; the compute stream waits for that
 * copy and runs the layer.  The copy stream first waits for the compute
 * stream's earlier work.  Nothing waits on the host; on return both
 * streams hold the whole pass and `out` is ordered on `compute`.
 * MOE_ERR_NOT_PINNED if a blob is not page-locked host memory.  At depth 2
 * the two streams must differ (MOE_ERR_INVALID_ARG otherwise: on one
 * stream every copy would wait for the previous layer's compute).
 *
 * Routed expert copy (MOE_COPY_ROUTED, or MOE_COPY_AUTO with
 * T <= routed_copy_max_tokens): the router logits of every layer are inputs
 * of the call, so layer L's routing is known before layer L-1 ends.  The
 * copy stream then routes and permutes layer L itself (into its own
 * double-buffered routing arrays) and moves only the experts with at least
 * one routed row, with a kernel that reads the blob through its
 * device-mapped address (a blob that has none is MOE_ERR_NOT_PINNED); the
 * compute stream runs FC1, FC2 and the combine on that routing.  The
 * experts the layer does not hit keep whatever the slot held before: no
 * kernel reads them.  The GEMMs then leave one CU per XCD free for the copy
 * kernel.  Outputs are bitwise those of MOE_COPY_ALL.  Blob and slot
 * addresses must be 16-byte aligned (MOE_ERR_INVALID_ARG otherwise).
 */
moe_status moe_layer_prefill_streamed(const moe_streamed_args* args, void* compute_stream,
                                      void* copy_stream);

/* ------------------------------- gated feed-forward block, 16-bit weights -- */

/* The dense block that runs beside the routed experts (a shared expert) or in
 * their place (a dense layer), for bf16 or fp16 activations and weights:
 *   gate_up = x * w1^T                          [T][2I], in w1's row order
 *   h[:, i] = act(gate_i) * up_i                [T][I]
 *   out     = (add +) h * w2^T                  [T][H]
 * Products accumulate in fp32, the gate is applied to the fp32 sums; h is
 * rounded once to `dtype` (the matrix cores' operand), out once to out_dtype.
 *
 * Sizes: 0 <= T <= 2^28 (T == 0 enqueues nothing), H and I multiples of 8, both
 * in [8, 262144], T rows of max(H, 2I) fewer than 2^24 tiles of 64 x 64.  Row strides are in elements, multiples of 8, at least the row
 * and at most 2^21; every pointer is 16-byte aligned.  w1, w2 and gate_up are
 * contiguous.  `out` may be `add` itself (same pointer and stride); apart
 * from that no output may overlap an input or another output. */
typedef struct moe_ffn_args {
  int32_t     T, H, I;
  int32_t     layout;            /* MOE_EPI_SWIGLU_SPLIT or _INTERLEAVED: w1's row order */
  int32_t     gate_act;          /* moe_gate_act */
  int32_t     dtype;             /* x, w1, w2: MOE_FLOAT_BF16 or MOE_FLOAT_FP16 */
  int32_t     out_dtype;         /* out and add: `dtype` or MOE_FLOAT_FP32 */
  int32_t     save_dtype;        /* gate_up: `dtype` or MOE_FLOAT_FP32 */
  const void* x;                 /* device [T][H] */
  const void* w1;                /* device [2I][H] */
  const void* w2;                /* device [H][I] */
  const void* add;               /* device [T][H] or NULL */
  void*       out;               /* device out [T][H] */
  void*       gate_up;           /* device out [T][2I], kept for the backward pass, or NULL */
  int64_t     x_stride, add_stride, out_stride;
  void*       workspace;         /* device, >= moe_gated_ffn_workspace_size() */
  size_t      workspace_bytes;
} moe_ffn_args;

/* (0 for sizes outside the limits above, as for the two queries below) */
size_t     moe_gated_ffn_workspace_size(int32_t T, int32_t H, int32_t I);
moe_status moe_gated_ffn_forward(const moe_ffn_args* args, void* stream);
/* forward's checks alone: its status for these arguments, with nothing enqueued
 * (for a caller whose other work must not start before a refusal). */
moe_status moe_gated_ffn_check(const moe_ffn_args* args);

/* The block's gradients from dout and the gate_up that forward kept:
 *   dh = dout * w2;  d_gate = dh * up * act'(gate);  d_up = dh * act(gate)
 *   dx = d_gate_up * w1;  dw1 = d_gate_up^T * x;  dw2 = dout^T * h
 * (the gradient of `add` is dout).  Any of dx, dw1, dw2 may be NULL: it is not
 * computed.  d_gate_up and h are rounded once to `dtype`, the operands of the
 * products that follow: in fp16 a d_gate_up below 2^-25 becomes 0 and one of
 * 65520 or more infinite, so scale dout as fp16 training does.  With accumulate
 * dw1 and dw2 hold earlier gradients and are added to, in fp32, before their
 * rounding.  T == 0 writes zeros to dw1 and dw2 (leaves them with accumulate).
 * Deterministic: no atomics.  Size, stride and overlap rules as above. */
typedef struct moe_ffn_grad_args {
  int32_t     T, H, I;
  int32_t     layout, gate_act;
  int32_t     dtype;             /* dout, x, w1, w2 */
  int32_t     save_dtype;        /* gate_up: `dtype` or MOE_FLOAT_FP32 */
  int32_t     dx_dtype;          /* `dtype` or MOE_FLOAT_FP32 */
  int32_t     dw_dtype;          /* dw1 and dw2: `dtype` or MOE_FLOAT_FP32 */
  int32_t     accumulate;        /* 0 or 1 */
  const void* dout;              /* device [T][H] */
  const void* x;                 /* device [T][H] (read for dw1 only) */
  const void* w1;                /* device [2I][H] (read for dx only) */
  const void* w2;                /* device [H][I] */
  const void* gate_up;           /* device [T][2I] */
  void*       dx;                /* device out [T][H] or NULL */
  void*       dw1;               /* device out [2I][H] or NULL */
  void*       dw2;               /* device out [H][I] or NULL */
  int64_t     dout_stride, x_stride, dx_stride;
  void*       workspace;         /* device, >= moe_gated_ffn_grad_workspace_size() */
  size_t      workspace_bytes;
} moe_ffn_grad_args;

size_t     moe_gated_ffn_grad_workspace_size(int32_t T, int32_t H, int32_t I);
moe_status moe_gated_ffn_backward(const moe_ffn_grad_args* args, void* stream);

/* ------------- low-rank adapters of many requests beside a projection -- */

/* One projection shared by all tokens plus each token's own adapter:
 *   y[t] = (add[t] +) x[t] * w^T + scales[a] * (x[t] * A[a]^T) * B[a]^T,  a = ids[t]
 *   out  = y, or for a SWIGLU epilogue act(gate columns of y) * up columns
 * An id outside [0, num_adapters) means no adapter: that token gets the shared
 * projection alone.  Tokens may come in any order and share adapters.  With
 * ranks, adapter a uses its first ranks[a] (clamped to [0, R]) rows of A and
 * columns of B; what lies behind them is not used.  w may be NULL (MOE_EPI_NONE
 * only): the adapters' part alone, added to what another projection gave
 * (a grouped GEMM with MXFP4 weights, say) through `add`.
 * A token's result depends on its own row and adapter only: infinities or NaN
 * in one adapter or token do not reach the others.
 * The low-rank row scales[a] * x A^T is held in fp32 and enters the second
 * product as it is, or (batches of more than 256 tokens) as a sum of numbers of
 * type `dtype`: three in bf16, which hold all of its 24 bits, two in fp16, which
 * hold 22, of the row times a power of two of its own, so that its range is
 * fp32's there too.
 *
 * Any order of tokens gives the same results; batches of more than 256 tokens
 * are fastest where the tokens of a request stand together, as prompts do.
 *
 * Sizes: 0 <= T <= 2^28 (T == 0 enqueues nothing), K, N multiples of 8 in
 * [8, 262144], T rows of N fewer than 2^24 tiles of 64 x 64;
 * 0 <= num_adapters <= 65536; R a multiple of 8 in [8, 256].  Strides, alignment and overlap as for moe_gated_ffn_forward
 * (ids, scales and ranks: 4-byte aligned; out_stride a multiple of 4 for
 * SWIGLU, whose N/2 columns need not be 8 n).  With a SWIGLU epilogue add has N
 * columns (it is added before the gate) and cannot be `out`. */
typedef struct moe_adapter_args {
  int32_t        T, K, N;
  int32_t        num_adapters, R;
  int32_t        epilogue;       /* moe_epilogue */
  int32_t        gate_act;       /* moe_gate_act (SWIGLU epilogues) */
  int32_t        dtype;          /* x, w, a, b: MOE_FLOAT_BF16 or MOE_FLOAT_FP16 */
  int32_t        out_dtype;      /* out and add: `dtype` or MOE_FLOAT_FP32 */
  const void*    x;              /* device [T][K] */
  const void*    w;              /* device [N][K] or NULL */
  const int32_t* ids;            /* device [T] */
  const void*    a;              /* device [num_adapters][R][K] */
  const void*    b;              /* device [num_adapters][N][R] */
  const float*   scales;         /* device [num_adapters] or NULL: 1 */
  const int32_t* ranks;          /* device [num_adapters] or NULL: R */
  const void*    add;            /* device [T][N] or NULL */
  void*          out;            /* device out [T][N], or [T][N/2] for SWIGLU */
  int64_t        x_stride, add_stride, out_stride;
  void*          workspace;      /* device, >= moe_adapter_workspace_size() */
  size_t         workspace_bytes;
} moe_adapter_args;

size_t     moe_adapter_workspace_size(int32_t T, int32_t K, int32_t N, int32_t num_adapters, int32_t R);
moe_status moe_adapter_linear(const moe_adapter_args* args, void* stream);

/* ------------------------------------- the norm before a layer, with MXFP8 -- */

/* Root-mean-square norm with the residual's addition:
 *   r   = x (+ residual, rounded to residual_dtype and written to residual_out)
 *   out = r / sqrt(mean(r^2) + eps) * weight             over a row of H
 * The norm is taken of r as it is kept, so that the backward pass and a later
 * addition see the number that was normed.  out is written in out_dtype, or as
 * MXFP8 (codes and scales: what the layer and the grouped GEMM take), or both;
 * each is rounded once, from the fp32 value.  An MXFP8 block's scale is the
 * smallest power of two that brings its 32 values to 448 or below, so none
 * saturates; codes are rounded to nearest even; a block that holds an infinity
 * or NaN has scale byte 255 and NaN codes.  Squares are summed in fp32: rows
 * whose sum of squares passes 3.4e38 come out as zeros, and with eps 0 rows whose
 * sum of squares is below 2^-126 lose precision, at 2^-150 all of it.
 *
 * Sizes: 0 <= T < 2^22 (T == 0 enqueues nothing), H a multiple of 8 in
 * [8, 32768], of 32 with codes.  Row strides are in elements, multiples of 8, at
 * least H and at most 2^21; every pointer is 16-byte aligned, `scales` 1-byte;
 * weight, codes and scales are contiguous.  eps is finite and not negative.
 * residual_out may be `residual` or x itself, out may be x itself (same pointer,
 * type and stride); apart from that no output may overlap an input or another
 * output. */
typedef struct moe_norm_args {
  int32_t     T, H;
  int32_t     dtype;             /* the 16-bit type: MOE_FLOAT_BF16 or MOE_FLOAT_FP16 */
  int32_t     x_dtype;           /* each of these `dtype` or MOE_FLOAT_FP32 */
  int32_t     residual_dtype;    /* residual and residual_out */
  int32_t     weight_dtype;
  int32_t     out_dtype;
  float       eps;
  const void* x;                 /* device [T][H] */
  const void* residual;          /* device [T][H] or NULL */
  const void* weight;            /* device [H] */
  void*       residual_out;      /* device out [T][H], with residual (NULL without) */
  void*       out;               /* device out [T][H] or NULL */
  uint8_t*    codes;             /* device out E4M3 [T][H] or NULL */
  uint8_t*    scales;            /* device out E8M0 [T][H/32], with codes */
  int64_t     x_stride, residual_stride, residual_out_stride, out_stride;
} moe_norm_args;

moe_status moe_rms_norm_forward(const moe_norm_args* args, void* stream);

/* The norm's gradients, with x the values that were normed (forward's r):
 *   u = x / sqrt(mean(x^2) + eps);  g = dout * weight
 *   dx = (g - u * mean(g * u)) / sqrt(mean(x^2) + eps) (+ dresidual)
 *   dweight = sum over the rows of dout * u
 * dx is the gradient of forward's x and of its residual alike; dresidual is what
 * reaches residual_out from elsewhere.  For MXFP8 outputs dout is the gradient
 * of the values that the codes stand for (their rounding counts as the
 * identity).  Either of dx and dweight may be NULL.  With accumulate dweight
 * holds an earlier gradient and is added to, in fp32, before its rounding.
 * T == 0 writes zeros to dweight (leaves it with accumulate).  Deterministic: no
 * atomics.  dx may be dout or dresidual itself (same pointer, type and stride).
 * Sizes, strides and alignment as above. */
typedef struct moe_norm_grad_args {
  int32_t     T, H;
  int32_t     dtype;             /* the 16-bit type */
  int32_t     dout_dtype;        /* each of these `dtype` or MOE_FLOAT_FP32 */
  int32_t     x_dtype;
  int32_t     weight_dtype;
  int32_t     dresidual_dtype;
  int32_t     dx_dtype;
  int32_t     dw_dtype;
  int32_t     accumulate;        /* 0 or 1 */
  float       eps;
  const void* dout;              /* device [T][H] */
  const void* x;                 /* device [T][H] */
  const void* weight;            /* device [H] */
  const void* dresidual;         /* device [T][H] or NULL */
  void*       dx;                /* device out [T][H] or NULL */
  void*       dweight;           /* device out [H] or NULL */
  int64_t     dout_stride, x_stride, dresidual_stride, dx_stride;
  void*       workspace;         /* device, >= moe_rms_norm_grad_workspace_size() */
  size_t      workspace_bytes;
} moe_norm_grad_args;

/* (0 for sizes outside the limits above) */
size_t     moe_rms_norm_grad_workspace_size(int32_t T, int32_t H);
moe_status moe_rms_norm_backward(const moe_norm_grad_args* args, void* stream);

/* ------------------------------------ gradients of the combine and the router -- */

/* The combine's gradients (out[t] = sum_j topk_w[t][j] * y[dest_row[t*k + j]]):
 *   dy[dest_row[t*k + j]] = topk_w[t][j] * dout[t]
 *   dtopk_w[t][j]         = sum_h y[dest_row[t*k + j]][h] * dout[t][h]
 * y_dtype and dy_dtype are moe_float_dtypes (moe_combine's y_dtype is a
 * moe_out_dtype, with other numbers).
 * dout is fp32, as the combine's out; dy is rounded once, dtopk_w is fp32.  Either
 * may be NULL; y is read for dtopk_w only.  A dest_row outside [0, T*k) has no
 * row: nothing is written for it and its dtopk_w is 0.  Rows of dy that no
 * dest_row names are left as they were; a row is named once at most (of two
 * gradients one would be kept, either of them).  0 <= T < 2^22, 1 <= k <= 64, H a multiple
 * of 8 in [8, 262144]; y, dout and dy contiguous and 16-byte aligned;
 * no output may overlap an input or the other output. */
moe_status moe_combine_backward(const float* dout, const void* y, int32_t y_dtype /* moe_float_dtype */,
                                const int32_t* dest_row, const float* topk_w, int32_t T, int32_t k, int32_t H,
                                void* dy, int32_t dy_dtype /* moe_float_dtype */, float* dtopk_w, void* stream);

/* The routing's gradient: topk_w is the softmax over a token's k kept logits, so
 *   dlogits[t][topk_ids[t][j]] = w_j * (dtopk_w_j - sum_i w_i * dtopk_w_i)
 * and 0 for the experts that were not kept.  An id outside [0, E) has no logit;
 * an id that a token lists twice gets the sum.  T, E and k as for moe_route. */
moe_status moe_route_backward(const float* dtopk_w, const int32_t* topk_ids, const float* topk_w, int32_t T,
                              int32_t E, int32_t k, float* dlogits, void* stream);

/* -------------------------------- routed experts with 16-bit weights -- */

/* The gated feed-forward block of moe_gated_ffn_forward, one set of weights for
 * each expert: row r with expert_offsets[e] <= r < expert_offsets[e + 1] gets
 *   gate_up[r] = x_r * w1[e]^T;  h = act(gate) * up;  out[r] = h * w2[e]^T
 * where x_r is row r of x, or with `gather` row gather[r] / gather_div of it
 * (moe_permute's perm_src and k, as in the MXFP4 grouped GEMM); a gathered row
 * outside [0, tokens) counts as zeros.  Experts may have any number of rows, none
 * included; rows outside [expert_offsets[0], expert_offsets[E]) are not read and
 * their outputs are left as they were (a part of the experts that one device
 * holds; a padded batch).  moe_combine and moe_combine_backward take every row
 * that dest_row names: give them a dest_row with -1 in the place of rows that are
 * not the experts'.  Offsets ascend; what exceeds [0, rows] is cut.
 * Accumulation and roundings as in moe_gated_ffn_forward.
 *
 * Sizes: 0 <= rows <= 2^28 (0 enqueues nothing), 1 <= E <= 8192, H and I multiples
 * of 8 in [8, 262144], fewer than 2^24 tiles of 64 x 64 in `rows` + 64 * min(E, rows)
 * rows of max(H, 2I) and in the E matrices w1; with gather, tokens * x_stride < 2^30.  Strides, alignment and
 * overlap as for moe_gated_ffn_forward; w1, w2, gate_up are contiguous. */
typedef struct moe_expert_ffn_args {
  int32_t        rows, H, I, E;
  int32_t        layout;         /* MOE_EPI_SWIGLU_SPLIT or _INTERLEAVED: w1's row order */
  int32_t        gate_act;       /* moe_gate_act */
  int32_t        dtype;          /* x, w1, w2: MOE_FLOAT_BF16 or MOE_FLOAT_FP16 */
  int32_t        out_dtype;      /* `dtype` or MOE_FLOAT_FP32 */
  int32_t        save_dtype;     /* gate_up: `dtype` or MOE_FLOAT_FP32 */
  int32_t        tokens;         /* rows of x, with gather */
  int32_t        gather_div;     /* >= 1 with gather, 0 without */
  const void*    x;              /* device [rows][H], with gather [tokens][H] */
  const int32_t* gather;         /* device [rows] or NULL */
  const int32_t* expert_offsets; /* device [E + 1] */
  const void*    w1;             /* device [E][2I][H] */
  const void*    w2;             /* device [E][H][I] */
  void*          out;            /* device out [rows][H] */
  void*          gate_up;        /* device out [rows][2I], kept for the backward pass, or NULL */
  int64_t        x_stride, out_stride;
  void*          workspace;      /* device, >= moe_expert_ffn_workspace_size() */
  size_t         workspace_bytes;
} moe_expert_ffn_args;

/* (0 for sizes outside the limits above, as for the query below) */
size_t     moe_expert_ffn_workspace_size(int32_t rows, int32_t H, int32_t I, int32_t E);
moe_status moe_expert_ffn_forward(const moe_expert_ffn_args* args, void* stream);

/* The experts' gradients from dout and the gate_up that forward kept, row by row
 * as moe_gated_ffn_backward, dw1[e] and dw2[e] summed over expert e's rows (zeros,
 * or with accumulate left as they are, where it has none).
 * dx without gather: [rows][H], rows outside the experts' left as they were.
 * With gather dx is [tokens][H], each token's gradient summed over its rows:
 *   dx[t] = sum_{j < gather_div} dx_row[dest_row[t * gather_div + j]]
 * with moe_permute's dest_row; a dest_row outside the experts' rows counts as
 * none.  The rows' gradients are held in fp32 until they are summed.
 * Any of dx, dw1, dw2 may be NULL.  Deterministic: no atomics.
 * Sizes as for the forward pass, with gather tokens * gather_div < 2^31 for dx and
 * tokens * x_stride < 2^30 for dw1. */
typedef struct moe_expert_ffn_grad_args {
  int32_t        rows, H, I, E;
  int32_t        layout, gate_act;
  int32_t        dtype;          /* dout, x, w1, w2 */
  int32_t        save_dtype;     /* gate_up: `dtype` or MOE_FLOAT_FP32 */
  int32_t        dx_dtype;       /* `dtype` or MOE_FLOAT_FP32 */
  int32_t        dw_dtype;       /* dw1 and dw2: `dtype` or MOE_FLOAT_FP32 */
  int32_t        accumulate;     /* 0 or 1: dw1 and dw2 are added to */
  int32_t        tokens;         /* rows of x and dx, with gather */
  int32_t        gather_div;     /* >= 1 with gather, 0 without */
  const void*    dout;           /* device [rows][H] */
  const void*    x;              /* device [rows][H], with gather [tokens][H] (read for dw1 only) */
  const int32_t* gather;         /* device [rows] or NULL */
  const int32_t* dest_row;       /* device [tokens * gather_div], for dx with gather */
  const int32_t* expert_offsets; /* device [E + 1] */
  const void*    w1;             /* device [E][2I][H] (read for dx only) */
  const void*    w2;             /* device [E][H][I] */
  const void*    gate_up;        /* device [rows][2I] */
  void*          dx;             /* device out or NULL */
  void*          dw1;            /* device out [E][2I][H] or NULL */
  void*          dw2;            /* device out [E][H][I] or NULL */
  int64_t        dout_stride, x_stride, dx_stride;
  void*          workspace;      /* device, >= moe_expert_ffn_grad_workspace_size() */
  size_t         workspace_bytes;
} moe_expert_ffn_grad_args;

/* gathered: 1 for calls with gather, else 0 */
size_t     moe_expert_ffn_grad_workspace_size(int32_t rows, int32_t H, int32_t I, int32_t E, int32_t gathered);
moe_status moe_expert_ffn_backward(const moe_expert_ffn_grad_args* args, void* stream);

#ifdef __cplusplus
} /* extern "C" */
#if __cplusplus >= 201103L

/* moe_combine counts its types by moe_out_dtype, moe_combine_backward by
 * moe_float_dtype: 0 and 1 are valid in both and mean other types.  The other
 * call's names do not compile (C++). */
moe_status moe_combine(const void* y, moe_float_dtype y_dtype, const int32_t* dest_row, const float* topk_w, int32_t T,
                       int32_t k, int32_t H, float* out, uint16_t* x_next, void* stream) = delete;
template <typename Dy>
moe_status moe_combine_backward(const float* dout, const void* y, moe_out_dtype y_dtype, const int32_t* dest_row,
                                const float* topk_w, int32_t T, int32_t k, int32_t H, void* dy, Dy dy_dtype,
                                float* dtopk_w, void* stream) = delete;
template <typename Y>
moe_status moe_combine_backward(const float* dout, const void* y, Y y_dtype, const int32_t* dest_row,
                                const float* topk_w, int32_t T, int32_t k, int32_t H, void* dy, moe_out_dtype dy_dtype,
                                float* dtopk_w, void* stream) = delete;
#endif
#endif
#endif /* MXMOE_H */
