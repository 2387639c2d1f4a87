/*
 * moe.h - C ABI of the GB300 (sm_103a) routed-expert MoE layer library (libmoe.so).
 *
 * The layer is the qwen3_5_moe routed-expert MLP with the routing and combine
 * contract set out on the page "Qwen3.6-35B-A3B (qwen3_5_moe) on the native
 * Metal engine: proposal and gate", section "What I'd build, in slices",
 * slice "The family, plain decode":
 *   1. fp32 router logits over the E experts, and the shared expert's fp32 gate
 *      logit gamma = x . v;
 *   2. top-k experts by logit, ties going to the lower expert id;
 *   3. pick weights exp(l - l_top) over the k picks, normalised over the picks
 *      (the "softmax top-8" of the "Qwen-3.6-35B-A3B-SIQ-K6-K4K3" model card,
 *      section "Reproduction"), rounded to bf16;
 *   4. the shared expert is one more slot with weight bf16(sigmoid(bf16(gamma)));
 *   5. each expert is a SwiGLU MLP, y_e = W_down (silu(W_gate x) * (W_up x))
 *      (the Gate section's "expert gate/up pair, expert down");
 *   6. y = bf16( sum_j p_j y_{e_j} + w_s y_shared ), rounded once.
 * Weights are MLX affine quantised (same slice): experts 4-bit, router 8-bit,
 * groups of 64 consecutive inputs of one output row sharing a bf16 scale s
 * and bias b, w = s * q + b.  The page's slice "8-bit experts" (the same
 * rule with expert codes q in [0, 255]) is supported too: moe_config.bits = 8.
 * Code layout: a row of n inputs holds n * bits / 8 bytes; at 4 bits input j
 * is the low nibble of byte j / 2 for even j and the high nibble for odd j,
 * at 8 bits input j is byte j.
 * Block-scaled experts (moe_config.format = MOE_FORMAT_NVFP4): every expert
 * matrix, shared included, in NVFP4, the checkpoint format named on the model
 * card "Qwen-3.6-35B-A3B-SIQ-K6-K4K3" (served there by a fused FP4 MoE
 * backend); the router stays 8-bit affine.  w_j = e2m1(q_j) * e4m3(s_b) * g
 * with q_j a 4-bit E2M1 code (bit 3 sign, bits 2..1 exponent with bias 1,
 * bit 0 mantissa; packed as the 4-bit affine codes), s_b the E4M3 scale of
 * the block of 16 consecutive inputs holding j, g the matrix's fp32 scale.
 *
 * Conventions shared by every entry point
 *   - Every function returns an int status (enum moe_status).  Argument,
 *     shape and format errors are found on the host, before anything is
 *     enqueued, and leave every buffer untouched.
 *   - Pointers to tensors are caller-owned DEVICE memory unless a parameter
 *     says otherwise.  The library never allocates, frees or synchronises,
 *     except moe_get_device_status, which synchronises the given stream.
 *   - Every tensor pointer must be 16-byte aligned; rows are dense (no
 *     padding between rows).  bf16 tensors are passed as uint16_t bit patterns.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     All work is enqueued asynchronously on it, in order.
 *   - `ws`/`ws_bytes` is caller-owned device scratch of at least
 *     moe_workspace_size() bytes for the call's T; it must not be shared by
 *     calls that may run concurrently.  Its first 512 bytes (the header: the
 *     status word and the grid-wide counters of the fused decode kernel) must
 *     be zero before the workspace's first use: allocate it zero-filled, or
 *     call moe_get_device_status on it once.  The kernels leave the counters
 *     zero when they end; the rest of the workspace carries nothing between
 *     calls.  A header that was not zero-filled is detected as far as the
 *     kernels can (MOE_ERR_WORKSPACE in the status word).
 *   - Device-side failures (a bounded wait that ran out, an index out of
 *     range, a header that was not zero-filled) never trap: the kernel writes
 *     a nonzero code into the workspace status word and returns.  The word
 *     keeps the first such code until moe_get_device_status reads it.
 *   - Values: x and the weights are finite.  Each token's x is scaled by a
 *     power of two before the 16-bit intermediate steps and the scale is
 *     undone after them (exact), so rows far above the fp16 range or entirely
 *     below its normal range keep their precision (within a row, elements
 *     below 2^-17 of its largest are held to fp16's subnormal spacing, an
 *     error of at most 2^-25 of that largest); only an output beyond the
 *     bf16 range overflows.
 *
 * Storage formats (MLX layout, [out, in] with quantisation along `in`)
 *   codes   4-bit: uint8 [rows, in/2], element j of a row in byte j/2, low
 *           nibble for even j.  8-bit: uint8 [rows, in].
 *   scales, biases: bf16 [rows, in/group].
 *   NVFP4 experts: codes as the 4-bit codes; scales holds E4M3 bytes
 *           [rows, in/16] (passed through the scales pointer); biases unused
 *           (may be NULL); gscale fp32, one per matrix ([E] for a stack).
 *           A NaN scale code (0x7F, 0xFF) makes the rows it scales undefined.
 *   Stacked expert matrices add a leading expert dimension:
 *     gate, up   [E, inter, hidden]     down  [E, hidden, inter]
 *     s_gate, s_up [inter, hidden]      s_down [hidden, inter]   (shared expert)
 *     router     [E, hidden] (8-bit)    shared_gate_vec bf16 [hidden]
 */
#ifndef QMOE_GB300_MOE_H
#define QMOE_GB300_MOE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, negative or oversized size */
    MOE_ERR_UNSUPPORTED = 2,  /* a format or shape the kernels do not implement */
    MOE_ERR_WORKSPACE = 3,    /* ws_bytes below moe_workspace_size(); as a device status: a
                                 workspace header that was not zero-filled */
    MOE_ERR_CUDA = 4,         /* a CUDA runtime call failed (launch, attribute query) */
    MOE_ERR_TIMEOUT = 5,      /* device status: a bounded wait inside a kernel ran out */
    MOE_ERR_DEVICE = 6        /* device status: a kernel found an index out of range */
};

enum moe_path {
    MOE_PATH_AUTO = 0,     /* decode for T <= 16, prefill above */
    MOE_PATH_DECODE = 1,   /* weight-streaming dequant-GEMV kernels (any T, meant for small T) */
    MOE_PATH_PREFILL = 2   /* tcgen05 grouped GEMM kernels (any T >= 1) */
};

/* Layer shape and per-call options.  Supported: group == 64, bits == 4 or 8
 * (4 with format == MOE_FORMAT_NVFP4), router_bits == 8, hidden and inter multiples of 64 (hidden <= 8192,
 * inter <= 4096), 1 <= top_k <= min(n_experts, 16), 1 <= n_experts <= 256,
 * has_shared in {0,1}.  Anything else returns MOE_ERR_UNSUPPORTED.
 * wait_polls bounds the in-kernel waits of the call: a wait polls at most
 * that many times (the first poll does not block, later ones sleep briefly),
 * then records MOE_ERR_TIMEOUT and the kernel returns early.  0 (or less)
 * selects the default, 1 << 20 polls (about a second).  A limit of 1 makes
 * any such wait that is not already satisfied run out (fault tests).  In the
 * fused decode kernel (T <= 16) it bounds the waits on other CTAs (published
 * router logits, the grid-wide unit counter); a CTA's waits on its own
 * shared-memory copies keep a fixed bound of the same order, so that a small
 * limit never leaves the copy ring in mid-flight.
 * With bits == 8 the decode path runs the weight-streaming gate/up, down and
 * reduce kernels after the routing kernels (the fused decode kernel and the
 * packed down layout are for 4-bit affine codes), and the prefill path runs
 * every expert on the tensor-memory GEMMs.  NVFP4 experts take the prefill
 * path at every T (MOE_PATH_DECODE and MOE_PATH_AUTO select it too). */
/* Expert storage formats (moe_config.format). */
enum moe_format {
    MOE_FORMAT_AFFINE = 0,  /* MLX affine, bits 4 or 8, groups of 64 */
    MOE_FORMAT_NVFP4 = 1    /* E2M1 codes, E4M3 scale per 16 inputs, fp32 per matrix; bits == 4 */
};

typedef struct moe_config {
    int hidden;       /* H */
    int inter;        /* I, intermediate size of every expert, shared included */
    int n_experts;    /* E routed experts */
    int top_k;        /* k picks per token */
    int group;        /* quantisation group along the input dimension */
    int bits;         /* expert code width */
    int router_bits;  /* router code width */
    int has_shared;   /* 1: the layer has a shared expert slot */
    int wait_polls;   /* bound on the in-kernel waits of the call; 0 = default */
    int format;       /* expert storage format, enum moe_format (0 = affine) */
} moe_config;

/* One quantised matrix (or a stack of them), device pointers, 16-byte aligned
 * (gscale: 4-byte aligned). */
typedef struct moe_qmat {
    const uint8_t *codes;
    const uint16_t *scales;  /* affine: bf16; NVFP4: E4M3 bytes */
    const uint16_t *biases;  /* affine: bf16; NVFP4: unused */
    const float *gscale;     /* NVFP4: fp32 scale per matrix; affine: unused */
} moe_qmat;

/* All weights of one layer, device pointers.  s_* and shared_gate_vec may be
 * NULL when has_shared == 0.
 * down_packed / s_down_packed (optional, NULL for none): the down codes
 * rearranged by moe_pack_down, which the decode kernel streams one contiguous
 * block per (expert, 32 columns of the intermediate dimension) instead of
 * gathering 16-byte pieces of every row.  They are read only by the decode
 * path and give the same results as the MLX layout. */
typedef struct moe_weights {
    moe_qmat router;   /* [E, H], router_bits */
    moe_qmat gate;     /* [E, I, H] */
    moe_qmat up;       /* [E, I, H] */
    moe_qmat down;     /* [E, H, I] */
    moe_qmat s_gate;   /* [I, H] */
    moe_qmat s_up;     /* [I, H] */
    moe_qmat s_down;   /* [H, I] */
    const uint16_t *shared_gate_vec;  /* bf16 [H] */
    const uint8_t *down_packed;       /* [E, I/32, H, 16] bytes, or NULL */
    const uint8_t *s_down_packed;     /* [I/32, H, 16] bytes, or NULL */
} moe_weights;

/* Human-readable name of a status code; never NULL, static storage. */
MOE_API const char *moe_status_string(int status);

/* Checks a configuration against the supported set (see moe_config). */
MOE_API int moe_check_config(const moe_config *cfg);

/* Bytes of workspace every entry point below needs for T tokens (0 <= T <= 65536).
 * *bytes receives the size; the same workspace serves every entry point. */
MOE_API int moe_workspace_size(const moe_config *cfg, int T, size_t *bytes);

/* Steps 1-4: router logits, top-k, pick weights, shared weight.
 *   x           bf16 [T, H]
 *   router_bias fp32 [E] added to every computed logit with one fp32 rounding
 *               (l = fp32(l + bias_e)); NULL for none.  Ignored with logits_in.
 *   logits_in   fp32 [T, E] logits to route on instead of the router GEMV; NULL
 *               to compute them.  Lets a caller with its own router use the layer.
 *   logits_out  fp32 [T, E] or NULL: the logits the top-k ran on.
 *   ids         int32 [T, k] expert ids in rank order (descending logit, ties
 *               to the lower id).
 *   p           bf16 [T, k] pick weights in the same order.
 *   w_shared    bf16 [T] shared-slot weight; NULL allowed; all zero when
 *               has_shared == 0.
 * T == 0 is valid and enqueues nothing. */
MOE_API int moe_route(const moe_config *cfg, const moe_weights *w, const uint16_t *x, int T,
              const float *router_bias, const float *logits_in, float *logits_out,
              int32_t *ids, uint16_t *p, uint16_t *w_shared,
              void *ws, size_t ws_bytes, void *stream);

/* Groups the T*k routed slots by expert: a stable counting sort of the flat
 * slot index f = t*k + j by ids[f] (so slots of one expert are in increasing t).
 *   counts   int32 [E]      slots routed to each expert
 *   offsets  int32 [E + 1]  exclusive prefix sum of counts
 *   perm     int32 [T*k]    perm[offsets[e] + r] = r-th slot routed to e
 *   inv_perm int32 [T*k]    inv_perm[f] = position of slot f in perm
 * ids entries outside [0, E) set MOE_ERR_DEVICE in the status word and the
 * outputs are then unspecified. */
MOE_API int moe_permute(const moe_config *cfg, const int32_t *ids, int T, int32_t *counts,
                int32_t *offsets, int32_t *perm, int32_t *inv_perm,
                void *ws, size_t ws_bytes, void *stream);

/* Step 5 and the weighted sum of step 6 without its rounding:
 *   acc[t, :] += sum_j p[t,j] * y_{ids[t,j]}(x_t) + w_shared[t] * y_shared(x_t)
 * acc is fp32 [T, H], caller-initialised (zero for a plain layer).
 * ids/p/w_shared as produced by moe_route; counts/offsets/perm as produced by
 * moe_permute from the same ids.  w_shared may be NULL when has_shared == 0.
 * path selects the kernels (enum moe_path).  On both paths each slot's expert
 * output is computed once and every acc element receives one fixed-order sum
 * of them, so the result is bit-reproducible for a given batch.  On the decode
 * path it is also independent of the other tokens in the batch; on the
 * prefill path an expert's token count selects the kernels that compute it
 * (exact-code small tiles up to 32 tokens, fp16-dequantised tensor-memory
 * GEMMs above), so a token's last bits can depend on its batch. */
MOE_API int moe_expert_ffn(const moe_config *cfg, const moe_weights *w, const uint16_t *x, int T,
                   const int32_t *ids, const uint16_t *p, const uint16_t *w_shared,
                   const int32_t *counts, const int32_t *offsets, const int32_t *perm,
                   float *acc, int path, void *ws, size_t ws_bytes, void *stream);

/* The single rounding of step 6: y = bf16_rne(acc), acc fp32 [T, H], y bf16 [T, H]. */
MOE_API int moe_combine(const moe_config *cfg, int T, const float *acc, uint16_t *y, void *stream);

/* The whole layer: route, permute, expert FFNs and combine.
 *   y        bf16 [T, H] output.
 *   ids_out  int32 [T, k], p_out bf16 [T, k], w_shared_out bf16 [T]: optional
 *            copies of the routing (NULL to skip).
 * Other arguments as in moe_route / moe_expert_ffn.  With MOE_PATH_DECODE
 * (or AUTO with T <= 16) row t of y, ids_out, p_out and w_shared_out is
 * bit-identical to the result of a T = 1 call on row t alone. */
MOE_API int moe_forward(const moe_config *cfg, const moe_weights *w, const uint16_t *x, int T,
                const float *router_bias, const float *logits_in, uint16_t *y,
                int32_t *ids_out, uint16_t *p_out, uint16_t *w_shared_out, int path,
                void *ws, size_t ws_bytes, void *stream);

/* The decode layer (T <= 16) for callers that cannot allocate device memory.
 * The pages describe nothing like it: it exists for callers such as code that
 * runs inside another engine's enqueue callback (that engine owns all device
 * memory) or a process that must not allocate after start-up.
 * Same arguments and results as moe_forward with MOE_PATH_DECODE, but no
 * workspace: the scratch is a fixed 24 MiB array in the library's own device
 * memory, held on every GPU that loads the library until the process exits
 * (zero at load; the kernels leave its counters zero).  Layers whose decode
 * scratch exceeds 24 MiB are refused with MOE_ERR_WORKSPACE; T outside 0..16
 * with MOE_ERR_INVALID_ARG.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  All calls share the one array, which keeps the last call's
 * contents: calls that overlap on the GPU (other streams, other threads)
 * race and give wrong results, so keep them ordered.  Device-side status is
 * recorded in the array and cannot be read back.  Allocates nothing. */
MOE_API int moe_forward_decode_static(const moe_config *cfg, const moe_weights *w, const uint16_t *x, int T,
                                      const float *router_bias, const float *logits_in, uint16_t *y,
                                      int32_t *ids_out, uint16_t *p_out, uint16_t *w_shared_out, void *stream);

/* Writes the decode layout of the 4-bit down codes (bits == 4 only, else
 * MOE_ERR_UNSUPPORTED): for expert e and column
 * slice c (32 columns of the intermediate dimension, 16 bytes of every row),
 *   down_packed[((e * (I/32) + c) * H + r) * 16 + b] = down.codes[(e * H + r) * I/2 + c * 16 + b]
 * and the same for the shared expert into s_down_packed (skipped when NULL or
 * has_shared == 0).  Each output holds as many bytes as its source; both are
 * caller-owned device memory.  Enqueued on `stream`; run it once after the
 * weights are loaded. */
MOE_API int moe_pack_down(const moe_config *cfg, const moe_weights *w, uint8_t *down_packed,
                          uint8_t *s_down_packed, void *stream);

/* Synchronises `stream`, then reads the device status word of `ws` and zeroes
 * the workspace header (status word and counters).  *device_status receives
 * MOE_OK or the first error code a kernel recorded since the last read. */
MOE_API int moe_get_device_status(void *ws, size_t ws_bytes, void *stream, int *device_status);

/* The intermediate stages of the expert FFNs, for checking each projection on
 * its own (the FP64 check of every projection class in the section "Gate" of
 * the proposal page): for every slot f (routed: f = t k + j, shared:
 * f = T k + t)
 *   h_out     fp32 [T (k + 1), I]  h = silu(W_gate x) * (W_up x) exactly as the
 *             down projection consumes it (after the kernels' own rounding), or NULL;
 *   yslot_out fp32 [T (k + 1), H]  the slot's expert output W_down h before the
 *             pick weight, or NULL.
 * ids/counts/offsets/perm as for moe_expert_ffn (counts/offsets/perm are read
 * on the prefill path only).  The same kernels as moe_expert_ffn compute the
 * stages; nothing is added into an accumulator.  Rows of h_out / yslot_out
 * of slots that do not exist (the
 * shared rows without a shared expert) are not written.  Returns
 * MOE_ERR_UNSUPPORTED for a path whose kernels cannot emit their stages (the
 * decode path of a layer that does not take the fused decode kernel: bits == 8,
 * or a shape outside its shared-memory plan). */
MOE_API int moe_expert_stages(const moe_config *cfg, const moe_weights *w, const uint16_t *x, int T,
                              const int32_t *ids, const int32_t *counts, const int32_t *offsets,
                              const int32_t *perm, float *h_out, float *yslot_out, int path,
                              void *ws, size_t ws_bytes, void *stream);

/* Timeline of the last fused decode launch on `ws` (T <= 16, decode path):
 * synchronises `stream`, then copies per CTA fourteen %globaltimer stamps
 * (ns) to host_stamps [max_ctas, 14]: kernel start, router logits published,
 * every logit seen, x staged for the expert units, top-k done, expert list
 * done, routing done, first gate chunk landed, first down chunk landed, first
 * down chunk computed, expert units done, unit counter reached, combine loads
 * done, combine done (a stamp that was not reached keeps an older value).
 * *n_ctas receives the number of CTAs of the launch. */
MOE_API int moe_decode_timeline(const moe_config *cfg, int T, void *ws, size_t ws_bytes, void *stream,
                                unsigned long long *host_stamps, int max_ctas, int *n_ctas);

/* ------------------------------------------------------------------------
 * Block-scaled operators: rows whose elements are narrow codes with one scale
 * per block of consecutive elements, made by a norm or a quantiser and
 * multiplied on the tensor cores in that form (both operands narrow).  They
 * stand beside the layer above, which keeps its activations in 16 bits: the
 * residual add and norm in front of it, its expert products at the tensor
 * cores' 4-bit rate, and projections of any other kind.
 *
 * Formats (enum moe_scaled_format); v' is the value that is stored for v:
 *   NVFP4  v' = e2m1(q) * e4m3(s) * g, s per 16 elements, g fp32 per row
 *          (activations) or per matrix (weights).  g is given, or for a row
 *          max(amax * (1/2688), 2^-110).  s = e4m3(amax_b * (1/g) * (1/6)),
 *          q = e2m1(v * ((1/g) / s)); q = 0 where s = 0.
 *   MXFP8  v' = e4m3(q) * 2^e, e per 32 elements: the smallest with
 *          amax_b <= 448 * 2^e, -127 <= e <= 127, stored as e + 127 (E8M0).
 *   MXFP4  v' = e2m1(q) * 2^e, e per 32 elements, amax_b <= 6 * 2^e.
 *   Roundings are to nearest, ties to even, saturating.  A block with a
 *   non-finite element gets the NaN scale (0x7F, E8M0 0xFF): every output
 *   computed from that row is then NaN.  NVFP4 scales are unsigned here: the
 *   sign bit of a scale byte must be clear.
 * Codes: rows dense; 4-bit codes two a byte, the lower nibble first.
 * Scales: in tiles of 128 rows x 4 blocks, 512 bytes, the order in which the
 *   tensor core takes them: block b of row r is byte
 *     ((r / 128) * ct + b / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4
 *   with ct = ceil(blocks per row / 4).  Bytes of blocks and rows that do not
 *   exist may hold anything.
 * Groups: rows of a product belong to groups (experts), in order; group g
 *   multiplies matrix g of a stack.
 *   Activations: codes, factors and outputs of R rows are dense; group g's
 *     rows are offsets[g] .. offsets[g + 1] - 1 (the last group's end at
 *     R - 1), and its scale rows start at row tile offsets[g] / 128 + g, so
 *     that they take (R / 128 + G) row tiles in all.
 *   Weights: matrix g's scale rows start at row tile g * ceil(N / 128).
 * Pointers as above (16-byte aligned); MXFP4 weight codes 32-byte aligned.
 * ws is any workspace of at least MOE_SCALED_WS_BYTES bytes whose first 512
 * bytes were zero before its first use; it holds the status word
 * (moe_get_device_status) and may be a workspace of moe_workspace_size too. */
enum moe_scaled_format {
    MOE_SCALED_NVFP4 = 1,
    MOE_SCALED_MXFP8 = 2,   /* activations; their products take MXFP4 weights */
    MOE_SCALED_MXFP4 = 3    /* weights */
};
#define MOE_SCALED_WS_BYTES 512

/* R block-scaled rows (or where to write them). */
typedef struct moe_scaled_rows {
    uint8_t *codes;    /* [R, n] (MXFP8) or [R, n / 2] */
    uint8_t *scales;   /* (R / 128 + G) * ct scale tiles */
    float *row_scale;  /* NVFP4: fp32 [R], or NULL (all ones); other formats: NULL */
} moe_scaled_rows;

/* A stack of G block-scaled weight matrices [N, K]. */
typedef struct moe_scaled_mat {
    const uint8_t *codes;   /* [G, N, K / 2] */
    const uint8_t *scales;  /* G * ceil(N / 128) * ct scale tiles */
    const float *alpha;     /* fp32 [G] factor of each matrix's products, or NULL (ones) */
} moe_scaled_mat;

/* Residual add and root-mean-square norm of T rows of n elements:
 *   s = bf16(x + residual)           (s = x without a residual)
 *   y = s * rsqrt(mean(s^2) + eps) * (weight_offset + weight)   in fp32
 *   residual   bf16 [T, n] or NULL
 *   weight     bf16 [n], or NULL for none
 *   sum_out    bf16 [T, n] s, or NULL; may be x or residual itself
 *   y_out      bf16 [T, n] y rounded once, or NULL
 *   format, q  y as MOE_SCALED_NVFP4 (q->row_scale required) or
 *              MOE_SCALED_MXFP8 rows, one group; format 0 and q NULL for none.
 * The codes are rounded from the fp32 y, not from y_out.  The sum of squares is
 * an fp32 sum: |s| has to stay below about 1e19 / sqrt(n).  n: a multiple of
 * the format's block (8 without one), at most 16384. */
MOE_API int moe_add_rmsnorm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float weight_offset,
                            float eps, int T, int n, uint16_t *sum_out, uint16_t *y_out, int format,
                            const moe_scaled_rows *q, void *stream);

/* Quantises T rows of n elements of x (bf16, or fp32 with x_f32 = 1), T / groups
 * rows to a group, each group's scale rows from a new row tile (so a stack of
 * weight matrices is quantised by one call with groups = G).
 *   gscale  NVFP4: fp32 [groups] given factor g of each group's rows
 *           (q->row_scale is not written), or NULL: a factor per row, written to
 *           q->row_scale.  Other formats: NULL.
 * n: a multiple of the block, at most 2^20, or 16384 for NVFP4 without gscale. */
MOE_API int moe_quantize(int format, const void *x, int x_f32, int T, int n, int groups, const float *gscale,
                         const moe_scaled_rows *q, void *stream);

/* Quantises T rows of bf16 x into the expert-sorted rows of their k picks (ids,
 * inv_perm, offsets as from moe_route and moe_permute) and, with has_shared, into
 * row T*k + t of the shared expert's group E: the rows of a grouped product over
 * E + has_shared groups.  format: NVFP4 (row factors) or MXFP8.  Picks that the
 * arguments place outside the rows are reported (MOE_ERR_DEVICE) and not written.
 * n: a multiple of the block, at most 2^20, or 16384 for NVFP4. */
MOE_API int moe_quantize_routed(int format, const uint16_t *x, int T, int n, int k, int E, int has_shared,
                                const int32_t *ids, const int32_t *inv_perm, const int32_t *offsets,
                                const moe_scaled_rows *q, void *ws, size_t ws_bytes, void *stream);

/* Scales as checkpoints store them (bytes [G, N, n / block], row-major) to scale
 * tiles of a weight stack.  Run once after loading. */
MOE_API int moe_tile_scales(int format, const uint8_t *src, int G, int N, int n, uint8_t *dst, void *stream);

/* Grouped product: y[r, :] = row_scale[r] alpha[g] (a[r, :] . w_g^T), bf16 or
 * (y_f32) fp32 [R, N], accumulated in fp32.
 *   format   of a: MOE_SCALED_NVFP4 (w NVFP4) or MOE_SCALED_MXFP8 (w MXFP4)
 *   offsets  int32 [G] first row of each group, increasing from 0, or NULL
 *            when G == 1 (moe_permute's offsets serve, also with a shared
 *            expert as group E).  With an entry outside [0, R] or below its
 *            predecessor nothing is computed (MOE_ERR_DEVICE is reported).
 * K: a multiple of 64 (NVFP4) or 128 (MXFP8), at most 65536; N: a multiple of 8;
 * G <= 1024; R <= 2^21 rows.  R == 0 enqueues nothing.
 * The same call gives the same bits; sizes select the kernels (few rows run
 * without tiles), so the last bits of a row's sums can depend on R. */
MOE_API int moe_scaled_gemm(int format, const moe_scaled_rows *a, const moe_scaled_mat *w, int R, int N, int K, int G,
                            const int32_t *offsets, void *y, int y_f32, void *ws, size_t ws_bytes, void *stream);

/* Two grouped products and SwiGLU: h = silu(a . gate_g^T) * (a . up_g^T) with both
 * products' factors, quantised to the rows' own format for the next product.
 *   h_scale  NVFP4: fp32 [G] calibrated factor g > 0 of h (fold it into the next
 *            matrices' alpha; h beyond 2688 g saturates); MXFP8: NULL
 *   h        [R, inter] rows, same groups; h->row_scale must be NULL
 * inter: a multiple of 64 (NVFP4) or 128 (MXFP8). */
MOE_API int moe_scaled_swiglu(int format, const moe_scaled_rows *a, const moe_scaled_mat *gate, const moe_scaled_mat *up,
                              int R, int inter, int K, int G, const int32_t *offsets, const float *h_scale,
                              const moe_scaled_rows *h, void *ws, size_t ws_bytes, void *stream);

/* All weights of one layer whose expert products run block-scaled.  gate, up
 * and down are stacks of n_experts + has_shared matrices, the shared expert's
 * last: [G, inter, hidden], [G, inter, hidden], [G, hidden, inter].  With NVFP4
 * a matrix's fp32 scale is its alpha, and down's alpha also carries h_scale. */
typedef struct moe_scaled_weights {
    int format;                       /* MOE_SCALED_NVFP4, or MOE_SCALED_MXFP8 (MXFP4 matrices) */
    moe_qmat router;                  /* as in moe_weights */
    const uint16_t *shared_gate_vec;  /* bf16 [hidden]; may be NULL without a shared expert */
    moe_scaled_mat gate, up, down;
    const float *h_scale;             /* NVFP4: fp32 [G], see moe_scaled_swiglu; MXFP8: NULL */
} moe_scaled_weights;

/* Bytes of workspace moe_scaled_forward needs for T tokens (0 <= T <= 65536); its
 * header as for moe_workspace_size. */
MOE_API int moe_scaled_workspace_size(const moe_config *cfg, int format, int T, size_t *bytes);

/* The whole layer with block-scaled expert products: moe_route, moe_permute,
 * moe_quantize_routed, moe_scaled_swiglu, moe_scaled_gemm (fp32) and the
 * weighted sum of each token's slots, rounded once.  Routing runs on the bf16 x
 * and is that of moe_forward; x and h are quantised, so y differs from
 * moe_forward's by the activations' 4- or 8-bit rounding.  cfg describes the
 * shape and the router (its bits and format fields are not used for the
 * experts); hidden and inter: multiples of 64 (NVFP4) or 128 (MXFP8).  Other
 * arguments as in moe_forward. */
MOE_API int moe_scaled_forward(const moe_config *cfg, const moe_scaled_weights *w, const uint16_t *x, int T,
                               const float *router_bias, const float *logits_in, uint16_t *y, int32_t *ids_out,
                               uint16_t *p_out, uint16_t *w_shared_out, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * 16-bit operators: the layer's products on bf16 matrices (before they are
 * quantised, or to train them), the norms around it, and the backward pass of
 * each.  They stand beside the block-scaled operators and share their groups:
 * rows sorted by group, group g's rows offsets[g] .. offsets[g + 1] - 1 (the
 * last group's end at R - 1); rows before offsets[0] belong to no group and are
 * neither read nor written.  offsets with an entry outside [0, R] or below its
 * predecessor: nothing is computed and MOE_ERR_DEVICE is reported.
 * All rows, matrices and vectors are bf16 and dense unless a parameter says
 * otherwise; products, sums and statistics are fp32 and rounded once, to the
 * type that is written.  Pointers 16-byte aligned (offsets, inv_perm 4-byte).
 * With no rows, pointers to rows may be NULL.  Outputs must not overlap inputs
 * except where that is allowed.  ws as for the block-scaled operators (a
 * header of MOE_SCALED_WS_BYTES), and more where a size function says so.
 * Non-finite values reach the outputs that their formulas use them in, and no
 * other row's.  The same call gives the same bits; sizes select the kernels, so a
 * row's last bits can depend on R. */
enum moe_activation {
    MOE_ACT_NONE = 0,
    MOE_ACT_SILU = 1,     /* v sigmoid(v) */
    MOE_ACT_GELU = 2,     /* tanh form: v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
    MOE_ACT_RELU = 3,
    MOE_ACT_SIGMOID = 4   /* gates of moe_gated_norm only */
};

/* Grouped product with an epilogue:
 *   pre = a w_g^T + a2 w2_g^T + bias_g,  y = act(pre) + residual
 *   a            [R, K]
 *   w            [G, N, K], or with w_transposed = 1 [G, K, N]: the input gradient of a product
 *                with the matrices [G, N', K'] is this with N = K', K = N'
 *   a2, w2       a second pair of the same sizes (both or neither): the input gradient
 *                of a gate/up pair in one sum
 *   bias         [G, N] or NULL
 *   residual     [R, N] or NULL; may be y itself (bf16)
 *   pre_out      [R, N] or NULL: pre, rounded, as moe_act_grad takes it
 *   y            [R, N], fp32 with y_f32 = 1
 * N, K: multiples of 8, K at most 65536, N at most 2^20; G <= 1024; R <= 2^21.
 * offsets may be NULL when G == 1.  R == 0 enqueues nothing. */
MOE_API int moe_gemm(const uint16_t *a, const uint16_t *w, const uint16_t *a2, const uint16_t *w2, int w_transposed, int R,
                     int N, int K, int G, const int32_t *offsets, const uint16_t *bias, int act, const uint16_t *residual,
                     uint16_t *pre_out, void *y, int y_f32, void *ws, size_t ws_bytes, void *stream);

/* Gated pair: g = a gate^T + gate_bias, u = a up^T + up_bias, h = act(g) u, from
 * the unrounded g and u.
 *   gate, up            [G, inter, K]
 *   gate_bias, up_bias  [G, inter] or NULL
 *   gate_out, up_out    [R, inter] or NULL (both or neither): g and u, rounded
 *   h                   [R, inter]
 * Sizes as in moe_gemm. */
MOE_API int moe_gemm_glu(const uint16_t *a, const uint16_t *gate, const uint16_t *up, const uint16_t *gate_bias,
                         const uint16_t *up_bias, int act, int R, int inter, int K, int G, const int32_t *offsets,
                         uint16_t *gate_out, uint16_t *up_out, uint16_t *h, void *ws, size_t ws_bytes, void *stream);

/* Weight gradient of a grouped product: dw_g = dy_g^T x_g and db_g = the column
 * sums of dy_g over the group's rows (zero for a group without rows).
 *   dy [R, N], x [R, K]
 *   dw [G, N, K], db [G, N] or NULL: bf16, or fp32 with f32 = 1
 *   accumulate  1: added to what dw and db hold (f32 only)
 * Sizes as in moe_gemm, N at most 2^20 and K at most 65536. */
MOE_API int moe_gemm_wgrad(const uint16_t *dy, const uint16_t *x, int R, int N, int K, int G, const int32_t *offsets,
                           int accumulate, void *dw, void *db, int f32, void *ws, size_t ws_bytes, void *stream);

/* Gradient through an activation, element by element over R rows of N:
 *   up NULL:  dpre = dy act'(pre)
 *   else      dpre = dy up act'(pre), dup = dy act(pre)     (a gated pair)
 * dpre may be dy or pre itself, dup may be dy, up or pre (but not dpre).
 * N: a multiple of 8. */
MOE_API int moe_act_grad(int act, const uint16_t *dy, const uint16_t *pre, const uint16_t *up, int R, int N, uint16_t *dpre,
                         uint16_t *dup, void *stream);

/* T rows of n elements of x into the expert-sorted rows of their k picks, y[inv_perm[t k + j]] = x[t], and with
 * has_shared into row T k + t (the shared expert's group).  inv_perm as from moe_permute; an entry outside
 * [0, T k) is reported (MOE_ERR_DEVICE) and its row not written.  n: a multiple of 8, at most 2^20.  The backward pass is
 * moe_weighted_sum without weights. */
MOE_API int moe_dispatch(const uint16_t *x, int T, int n, int k, int has_shared, const int32_t *inv_perm, uint16_t *y,
                         void *ws, size_t ws_bytes, void *stream);

/* y[t] = sum_j p[t, j] rows[inv_perm[t k + j]] + w_shared[t] rows[T k + t], picks in
 * order, rounded once.
 *   rows      [T k + T has_shared, n]
 *   p         [T, k], or NULL: ones (then w_shared NULL too)
 *   w_shared  [T]; NULL with has_shared == 0, or without p
 * An inv_perm entry outside [0, T k) is reported and its term left out. */
MOE_API int moe_weighted_sum(const uint16_t *rows, int T, int n, int k, int has_shared, const int32_t *inv_perm,
                             const uint16_t *p, const uint16_t *w_shared, uint16_t *y, void *ws, size_t ws_bytes, void *stream);

/* Its backward pass, from dy [T, n]:
 *   drows      [T k + T has_shared, n]: p[t, j] dy[t] in row inv_perm[t k + j], w_shared[t] dy[t] in row T k + t; may be rows
 *   dp         fp32 [T, k] or NULL: dy[t] . rows[inv_perm[t k + j]] (0 where the entry is out of range)
 *   dw_shared  fp32 [T] or NULL
 * rows may be NULL when dp and dw_shared are.  drows' rows that no entry names are not written. */
MOE_API int moe_weighted_sum_grad(const uint16_t *dy, const uint16_t *rows, int T, int n, int k, int has_shared,
                                  const int32_t *inv_perm, const uint16_t *p, const uint16_t *w_shared, uint16_t *drows,
                                  float *dp, float *dw_shared, void *ws, size_t ws_bytes, void *stream);

/* Shapes of a gate. */
enum moe_gate_shape {
    MOE_GATE_NONE = 0,
    MOE_GATE_ROW = 1,      /* [T], one value a token */
    MOE_GATE_CHANNEL = 2,  /* [n], a scale per channel */
    MOE_GATE_FULL = 3      /* [T, n] */
};

/* The norm after a block, its gate, the residual add and the norm before the next block, of T rows of n elements:
 *   b = x rsqrt(mean(x^2) + eps) (weight_offset + post_weight)     (b = x without post_norm)
 *   s = bf16(residual + scale f(gate) b)
 *   y = s rsqrt(mean(s^2) + eps) (weight_offset + pre_weight)
 *   gate          its shape gate_shape; NULL with MOE_GATE_NONE
 *   gate_act      f: MOE_ACT_NONE, MOE_ACT_SILU or MOE_ACT_SIGMOID (NONE without a gate)
 *   residual      [T, n] or NULL
 *   post_weight, pre_weight  [n] or NULL for none (no offset either); post_weight NULL without post_norm
 *   sum_out       [T, n] s, or NULL; may be x or residual itself
 *   y_out         [T, n] or NULL
 * The sums of squares are fp32 sums: |x| and |s| have to stay below about 1e19 / sqrt(n).
 * n: a multiple of 8, at most 8192. */
MOE_API int moe_gated_norm(const uint16_t *x, const uint16_t *residual, const uint16_t *gate, int gate_shape, int gate_act,
                           float scale, int post_norm, const uint16_t *post_weight, const uint16_t *pre_weight,
                           float weight_offset, float eps, int T, int n, uint16_t *sum_out, uint16_t *y_out, void *stream);

/* Bytes of workspace moe_gated_norm_grad needs (T >= 0, n as there). */
MOE_API int moe_gated_norm_workspace_size(int T, int n, size_t *bytes);

/* Its backward pass.  x, gate, weights and factors as there; sum is the s that it gave.
 *   dy, dsum    [T, n] gradients of y and of s (from the next residual add); either may be NULL (zero), not both
 *   dx          [T, n]; may be x, dy or dsum itself
 *   dresidual   [T, n] or NULL: the gradient of s as a whole; may be sum, dy or dsum itself (but not dx)
 *   dgate       the gate's gradient, or NULL: bf16 [T, n] (FULL), fp32 [T] (ROW), fp32 [n] (CHANNEL)
 *   dpost_weight, dpre_weight  fp32 [n] or NULL; dpost_weight only with post_norm, dpre_weight only with dy
 * Sums over rows are taken in a fixed order that depends on T and n.  With T == 0 the sums over rows are set to zero. */
MOE_API int moe_gated_norm_grad(const uint16_t *x, const uint16_t *sum, const uint16_t *gate, int gate_shape, int gate_act,
                                float scale, int post_norm, const uint16_t *post_weight, const uint16_t *pre_weight,
                                float weight_offset, float eps, int T, int n, const uint16_t *dy, const uint16_t *dsum,
                                uint16_t *dx, uint16_t *dresidual, void *dgate, float *dpost_weight, float *dpre_weight,
                                void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QMOE_GB300_MOE_H */
