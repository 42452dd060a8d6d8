/*
 * gdn.h -- C ABI of the gated delta-rule (GDN) library for NVIDIA GB300 (sm_103a).
 *
 * The library computes the gated delta-rule linear-attention recurrence named
 * in the "Background" section of the "GDN CTE Kernel API Reference" page:
 * for every batch b, value head h (reading query/key head h / (Hv/Hk)) and
 * token t,
 *
 *     S_t = exp(g_t) S_{t-1} + beta_t k_t (v_t - exp(g_t) S_{t-1}^T k_t)^T
 *     o_t = scale * S_t^T q_t
 *
 * with an fp32 state S of shape [Dk, Dv].  Two entry points compute it:
 * a chunk-parallel prefill over a whole sequence (gdn_prefill) and one
 * single-token step (gdn_decode_step).
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers to contiguous row-major memory
 *     owned by the caller; the library never allocates, frees or keeps them.
 *   - Work is enqueued on `stream`; calls return before the GPU finishes.
 *     Host-side argument checks run first: when one fails, nothing is launched
 *     and the error code is returned.  Asynchronous kernel faults surface at
 *     the caller's next synchronisation; kernel-side wait timeouts are recorded
 *     in a per-device status word read by gdn_device_status().
 *   - Preconditions the library does NOT check: q and k are L2-normalised per
 *     token ("GDN CTE Kernel API Reference", Notes), g_log <= 0 (Parameters /
 *     g_log), beta in (0, 1) (Parameters / beta), and the buffers do not overlap
 *     except state_inout with itself.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st* gdn_stream_t;

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,        /* a required pointer is NULL                                  */
    GDN_ERR_DIMS = 2,        /* dims inconsistent with the pages' constraints (see gdn_dims) */
    GDN_ERR_UNSUPPORTED = 3, /* allowed by the pages but not implemented by this build      */
    GDN_ERR_ALIGN = 4,       /* a tensor pointer is not 16-byte aligned                     */
    GDN_ERR_CUDA = 5,        /* a CUDA call (launch, attribute, tensor-map encode) failed    */
    GDN_ERR_TIMEOUT = 6,     /* a kernel wait ran past its bound (device status only)        */
    GDN_ERR_WORKSPACE = 7    /* a caller workspace smaller than the call needs              */
} gdn_status;

/* Compute dtype = dtype of q, k, v and out ("GDN CTE Kernel API Reference",
 * Parameters / query: the query's dtype sets the compute dtype).  g_log, beta
 * and the state are always fp32. */
typedef enum {
    GDN_F32 = 0,
    GDN_BF16 = 1,
    GDN_F8E4M3 = 2  /* 8 bits: sign, 4 exponent and 3 mantissa bits, largest finite value 448, no
                       infinities; of the layer operators only (gdn_rmsnorm_residual, gdn_linear) */
} gdn_dtype;

enum {
    /* The "omitted" recurrent_state form (Parameters / recurrent_state): start
     * from a zero state and emit no load.  state_inout is still required and
     * receives the final state. */
    GDN_ZERO_INITIAL_STATE = 1u << 0,
    /* Run the prefill on the fp32 FFMA kernel even where the tensor-core kernel
     * applies (a cross-check path; same results within fp32 rounding). */
    GDN_FORCE_FFMA = 1u << 1,
    /* Never split a sequence into segments (see gdn_prefill): one pass over
     * every sequence, whatever the SM count, so results do not depend on it. */
    GDN_SINGLE_PASS = 1u << 2,
    /* Linear attention only (gdn_linear_attn_*): g_log is [Hv], one decay a head for all tokens. */
    GDN_HEAD_DECAY = 1u << 3,
    /* gdn_linear_attn_prefill only: rows of out behind a sequence's length are set to zero. */
    GDN_ZERO_PADDING = 1u << 4
};

/*
 * Problem sizes ("GDN CTE Kernel API Reference", Dimensions and Notes):
 *   B  >= 0 batch (0: nothing to do);  Hk >= 1 key/query heads;
 *   Hv >= 1 value heads with Hv % Hk == 0;
 *   S  >= 0 tokens for the prefill (0: no tokens, the state is left as it is,
 *      or zeroed under GDN_ZERO_INITIAL_STATE); the decode step requires S == 1;
 *   Dk, Dv in [1, 128] head dims (Dq == Dk: q and k share Dk).
 * Violations return GDN_ERR_DIMS.  The pages' S % 128 rule belongs to their
 * Trainium algorithm choice; this library accepts any S.  When B == 0 or
 * S == 0, q, k, v, g_log, beta and out may be NULL.
 */
typedef struct {
    int64_t B, Hk, Hv, S, Dk, Dv;
    int32_t dtype;   /* gdn_dtype */
    uint32_t flags;  /* GDN_ZERO_INITIAL_STATE | GDN_FORCE_FFMA | GDN_SINGLE_PASS */
} gdn_dims;

/*
 * gdn_prefill -- chunk-parallel prefill of the recurrence over S tokens.
 * ("GDN CTE Kernel API Reference", API Reference / gdn_cte: Parameters, Returns.)
 *
 *   q           [B, Hk, S, Dk]  compute dtype, token-major, L2-normalised rows
 *   k           [B, Hk, S, Dk]  compute dtype, token-major, L2-normalised rows
 *   v           [B, Hv, S, Dv]  compute dtype
 *   g_log       [B, Hv, S]      fp32 per-token log-decay (negative)
 *   beta        [B, Hv, S]      fp32 per-token update strength in (0, 1)
 *   scale       query scale, applied on the device (typically 1/sqrt(Dk))
 *   state_inout [B, Hv, Dk, Dv] fp32, Dv contiguous.  Read as the initial state
 *               (unless GDN_ZERO_INITIAL_STATE) and overwritten in place with the
 *               final state (the page's aliased in/out recurrent_state).
 *   out         [B, Hv, S, Dv]  compute dtype, head-major, un-normalised
 *
 * Every pointer must be non-NULL and 16-byte aligned.  Returns GDN_OK once the
 * work is enqueued.  Implementation: Dk = Dv = 128 with bf16 runs on the
 * tcgen05 tensor-core kernel; every other supported shape and fp32 compute run
 * on the FFMA kernel.
 *
 * Few long sequences (on the tensor-core path) are split into P >= 2 segments
 * unless GDN_SINGLE_PASS is set, when a host-side model of the launch (one CTA
 * per SM, CTAs dispatched in order) predicts that it saves at least a tenth of
 * one pass; gdn_prefill_segment_starts reports the split.  The recurrence is
 * affine in its start state: a later segment's end state is M S0 + X and its
 * output at token t is out_0[t] + C[t] S0, with X and out_0 its end state and
 * outputs from a zero start and M and C (C[t]: 1 x Dk per token) its end state
 * and outputs from S0 = I with v = 0.  Four kernel launches and a memset: an
 * identity matrix and a zero v tile; one launch of segment 0 from the real
 * start state and both runs of every later
 * segment (out_0 is written to out, C to the scratch); a combine step that
 * chains the maps into every segment's start state and the final state
 * (fp32); a correction that adds C[t] S0 to the later segments' outputs
 * (tcgen05, S0 rounded to bf16; the sum rounded once to bf16).  The scratch
 * (gdn_prefill_workspace_bytes: 3 (P - 1) states per sequence, one identity,
 * and C for every token after segment 0) is allocated with cudaMallocAsync on
 * `stream` and freed there; if that allocation fails, the call runs one pass
 * instead.  The results agree with the one-pass form to within rounding (a
 * similar error against an fp64 reference, from strong decay to none), not bit
 * for bit; segment 0's outputs are those of one pass.
 */
gdn_status gdn_prefill(const void* q, const void* k, const void* v,
                       const float* g_log, const float* beta, float scale,
                       float* state_inout, void* out,
                       const gdn_dims* dims, gdn_stream_t stream);

/*
 * gdn_decode_step -- one token of the recurrence (the prefill at S = 1), the
 * core of the single-token step of the "GDN Block TKG Kernel API Reference"
 * page (its recurrent_state [B, num_v_heads, head_k_dim, head_v_dim] fp32).
 * Same arguments and layouts as gdn_prefill with dims->S == 1 (else
 * GDN_ERR_DIMS).  The state is updated in place: each fp32 state element is
 * read once and written once.
 */
gdn_status gdn_decode_step(const void* q, const void* k, const void* v,
                           const float* g_log, const float* beta, float scale,
                           float* state_inout, void* out,
                           const gdn_dims* dims, gdn_stream_t stream);

/*
 * gdn_decode_gated -- the gated single-token step of the decode block: the
 * decode prologue, one token of the recurrence, and the RMSNormGated output
 * epilogue ("GDN Block TKG Kernel API Reference": gdn_block_tkg Parameters
 * A_log, dt_bias, norm_weight and the z / a / b in_proj outputs; Returns
 * "RMSNormGated decode output").  The page names these inputs but prints no
 * formulas; this library reads them as (eps_l2 = eps_rms = 1e-6):
 *
 *     q^ = q / sqrt(|q|^2 + eps_l2),  k^ likewise (q and k need NOT be normalised)
 *     g  = -exp(A_log[h]) * softplus(a[b, h] + dt_bias[h]),   beta = sigmoid(b[b, h])
 *     (o, S') = the recurrence step of gdn_decode_step on q^, k^, v, g, beta, scale
 *     y  = o / sqrt(mean over Dv of o^2 + eps_rms) * norm_weight * silu(z)
 *
 *   qkv          [B, 2*Hk*Dk + Hv*Dv]  compute dtype: the post-conv q | k | v row
 *                (q [Hk, Dk] head-major, then k [Hk, Dk], then v [Hv, Dv])
 *   z            [B, Hv*Dv]  compute dtype, output gate
 *   a, b         [B, Hv]     compute dtype, raw decay-gate and beta inputs
 *   A_log, dt_bias [Hv] fp32;  norm_weight [Dv] fp32
 *   state_inout  [B, Hv, Dk, Dv] fp32, updated in place (GDN_ZERO_INITIAL_STATE
 *                starts from zeros)
 *   out          [B, Hv*Dv]  compute dtype, y
 * dims as for gdn_decode_step (S == 1, Dk, Dv <= 128, Hv % Hk == 0).  Pointers
 * must be non-NULL and aligned to their element size; the state takes 128-bit
 * accesses when it is 16-byte aligned and Dv % 4 == 0.
 */
#define GDN_L2NORM_EPS 1e-6f
#define GDN_RMSNORM_EPS 1e-6f
gdn_status gdn_decode_gated(const void* qkv, const void* z, const void* a, const void* b,
                            const float* A_log, const float* dt_bias, const float* norm_weight,
                            float scale, float* state_inout, void* out,
                            const gdn_dims* dims, gdn_stream_t stream);

/*
 * Depthwise causal conv1d + SiLU in front of the recurrence, with its conv_state
 * ("GDN Conv1D Kernel API Reference": gdn_conv1d_prefill, gdn_conv1d_decode;
 * Parameters, Returns, Notes).  Every channel is an independent K-tap FIR over
 * the raw (pre-convolution) q|k|v activations:
 *
 *     out[b, c, t] = silu( sum_{m=0}^{K-1} w[c, K-1-m] x[b, c, t-m] ),   silu(z) = z / (1 + e^-z)
 *
 * (weight[c, K-1] multiplies the current token, as in a depthwise Conv1d).
 *
 *   B >= 0 batch (0: nothing to do);  C >= 1 channels;  T >= 0 tokens for the
 *   prefill, T == 1 for the decode step;  K in [1, 8] taps (more returns
 *   GDN_ERR_UNSUPPORTED);  dtype = gdn_dtype of x, out and conv_state; the
 *   weights are fp32.  flags must be 0.
 */
typedef struct {
    int64_t B, C, T, K;
    int32_t dtype;   /* gdn_dtype */
    uint32_t flags;  /* 0 */
} gdn_conv_dims;

/*
 * gdn_conv1d_prefill -- the whole sequence, starting from zeros (the prefill
 * takes no previous window).
 *   mixed           [B, C, T]  dtype, raw input, tokens contiguous per channel
 *   conv_weight     [C, K]     fp32
 *   out             [B, C, T]  dtype, silu(causal conv)
 *   conv_state_out  [B, C, K]  dtype, the last K raw tokens of mixed,
 *                   right-aligned behind zeros when T < K (written when T == 0 too)
 * Pointers must be non-NULL (x and out may be NULL when T == 0 or B == 0) and
 * aligned to their element size (else GDN_ERR_ALIGN).  bf16 rows with T % 8 == 0
 * and 16-byte aligned x / out take the vectorised path.
 */
gdn_status gdn_conv1d_prefill(const void* mixed, const float* conv_weight, void* out, void* conv_state_out,
                              const gdn_conv_dims* dims, gdn_stream_t stream);

/*
 * gdn_conv1d_decode -- one token.
 *   x                 [B, C, 1]  dtype, the current raw token
 *   conv_weight       [C, K]     fp32
 *   conv_state_inout  [B, C, K]  dtype, the previous window; overwritten in place
 *                     with the shifted window (the previous one without its
 *                     oldest token, then x)
 *   out               [B, C, 1]  dtype, silu(sum_k w[c, k] window[k])
 * dims->T must be 1 (else GDN_ERR_DIMS).
 */
gdn_status gdn_conv1d_decode(const void* x, const float* conv_weight, void* conv_state_inout, void* out,
                             const gdn_conv_dims* dims, gdn_stream_t stream);

/*
 * The decode block without its output projection ("GDN Block TKG Kernel API
 * Reference": gdn_block_tkg Parameters, Returns, Notes; the data flow "in_proj
 * matmuls -> gdn_conv1d_decode -> split conv_out + GQA-repeat q,k -> gdn_tkg"):
 * the four input projections of one token's hidden state, the conv1d decode step
 * on the q|k|v channels, and the gated single-token step (gdn_decode_gated, with
 * the query scale 1/sqrt(Dk), the page having no scale argument).
 *
 *   B in [0, 256]; H (hidden size) a multiple of 64; Hk, Hv, Dk, Dv as for
 *   gdn_decode_step; K in [1, 8] conv taps; dtype GDN_BF16 (the page's bf16
 *   weights and activations; others return GDN_ERR_UNSUPPORTED); flags 0.
 *   conv_dim C = 2*Hk*Dk + Hv*Dv; value_dim = Hv*Dv; C, value_dim and Hv must be
 *   multiples of 8 (row pitches of 16 bytes).
 */
typedef struct {
    int64_t B, H, Hk, Hv, Dk, Dv, K;
    int32_t dtype;   /* GDN_BF16 */
    uint32_t flags;  /* 0 */
} gdn_block_dims;

/* Size of the fixed scratch array that gdn_decode_block_noalloc uses (4 MiB). */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)

/* Device workspace bytes gdn_decode_block needs (the inter-stage activations z,
 * a, b in bf16, and a work counter of the gated step); 0 for invalid dims. */
size_t gdn_decode_block_workspace_bytes(const gdn_block_dims* dims);

/*
 * gdn_decode_block -- one token through the block.
 *   hidden            [B, 1, H] bf16
 *   W_qkv             [H, C] bf16, W_z [H, value_dim] bf16, W_a, W_b [H, Hv] bf16
 *                     (each == nn.Linear.weight.T)
 *   conv_weight       [C, K] fp32;  conv_state_inout [B, C, K] bf16, shifted in place
 *   A_log, dt_bias    [Hv] fp32;    norm_weight [Dv] fp32
 *   state_inout       [B, Hv, Dk, Dv] fp32, updated in place
 *   out               [B, 1, value_dim] bf16, the RMSNormGated output
 *   workspace         device memory of at least gdn_decode_block_workspace_bytes,
 *                     16-byte aligned, owned by the caller (else GDN_ERR_DIMS)
 * hidden, the weights and the workspace must be 16-byte aligned, every other
 * pointer aligned to its element (GDN_ERR_ALIGN); all checks run before the
 * first launch.  Launches two kernels on `stream`: the projections (whose
 * q|k|v epilogue shifts the conv windows in place), then the gated step, which
 * takes the conv1d output from the shifted windows and starts loading the state
 * while the projections run (programmatic dependent launch).
 */
gdn_status gdn_decode_block(const void* hidden, const void* W_qkv, const void* W_z, const void* W_a,
                            const void* W_b, const float* conv_weight, void* conv_state_inout,
                            const float* A_log, const float* dt_bias, const float* norm_weight,
                            float* state_inout, void* out, void* workspace, size_t workspace_bytes,
                            const gdn_block_dims* dims, gdn_stream_t stream);

/*
 * gdn_decode_block_noalloc -- gdn_decode_block for callers that cannot allocate
 * device memory: a runtime that owns every byte of the device and hands out no
 * buffers to kernels it does not know, a plugin whose host code must not call the
 * CUDA allocator, or a serving loop that may not risk an allocation (which can
 * synchronise the device or fail under memory pressure) while it runs.  The
 * pages' block kernel has no such variant; it exists for this library's callers.
 *
 * Arguments and results are those of gdn_decode_block without the workspace: the
 * inter-stage scratch (z, a, b in bf16 and the gated step's head counter) lives
 * in a fixed array inside the library, GDN_NOALLOC_SCRATCH_BYTES bytes, of which
 * every CUDA device that loads the library keeps one copy until the process
 * exits.  Dims whose scratch, gdn_decode_block_workspace_bytes, exceeds that size
 * return GDN_ERR_UNSUPPORTED and launch nothing (for the workloads here, B = 64
 * and value_dim = 4096 need 0.5 MiB; B = 256 with value_dim = 4096 about 2 MiB).
 * The call allocates nothing: no cudaMalloc, cudaFree or allocating library
 * routine.
 *
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and caches it; make that first
 * call before any stream capture on the device.  Every call on a device shares
 * the one array, and the array keeps the previous call's contents: each call
 * rewrites z, a and b and clears the counter before reading them, so results do
 * not depend on earlier calls, but two calls whose kernels overlap on the GPU
 * (different streams, or different host threads, without ordering between them)
 * race on the array and give wrong results.  Serialise such calls on one stream.
 */
gdn_status gdn_decode_block_noalloc(const void* hidden, const void* W_qkv, const void* W_z, const void* W_a,
                                    const void* W_b, const float* conv_weight, void* conv_state_inout,
                                    const float* A_log, const float* dt_bias, const float* norm_weight,
                                    float* state_inout, void* out, const gdn_block_dims* dims, gdn_stream_t stream);

/*
 * gdn_rmsnorm_gated -- the RMSNormGated output epilogue ("GDN Block TKG Kernel
 * API Reference": Returns, "RMSNormGated decode output"; norm_weight, the
 * "RMSNormGated weight") over `rows` rows of D elements:
 *     out[r, :] = x[r, :] / sqrt(mean(x[r, :]^2) + GDN_RMSNORM_EPS) * norm_weight * silu(z[r, :])
 *   x, z, out   [rows, D] in `dtype` (GDN_BF16 or GDN_F32), element-aligned;
 *               out may be x (in place)
 *   norm_weight [D] fp32
 * rows >= 0, 1 <= D <= 4096.  One launch on `stream`.
 */
gdn_status gdn_rmsnorm_gated(const void* x, const void* z, const float* norm_weight, void* out, int64_t rows,
                             int64_t D, int32_t dtype, gdn_stream_t stream);

/*
 * gdn_prefill_gated -- gdn_prefill followed by gdn_rmsnorm_gated on its output,
 * per token and value head over Dv (the decode block's RMSNormGated applied to
 * every token of a prefill):
 *   z           [B, Hv, S, Dv] in the compute dtype (head-major, like out)
 *   norm_weight [Dv] fp32
 *   the other arguments as gdn_prefill; out receives the gated output.
 * Every check of both steps runs before the first launch.  Launches the
 * prefill's kernel, then one normalisation pass that reads the output and z
 * and rewrites the output in place.
 */
gdn_status gdn_prefill_gated(const void* q, const void* k, const void* v, const float* g_log, const float* beta,
                             const void* z, const float* norm_weight, float scale, float* state_inout, void* out,
                             const gdn_dims* dims, gdn_stream_t stream);

/*
 * The operators of the layer around the block: the norm in front of it, the
 * output projection behind it, and the feed-forward's products.  (The pages'
 * block kernel leaves them to its caller.)  gdn_rmsnorm_residual's 8-bit rows and
 * scales are gdn_linear's 8-bit x and x_scale.
 */

/*
 * gdn_rmsnorm_residual -- RMS norm behind the residual's addition, over `rows`
 * rows of D elements:
 *     h[r, :] = x[r, :] + residual[r, :]        (fp32; x[r, :] alone where residual is NULL)
 *     y[r, :] = h[r, :] / sqrt(mean(h[r, :]^2) + eps) * norm_weight
 *   x, residual   [rows, D] in `dtype` (GDN_BF16 or GDN_F32)
 *   norm_weight   [D] fp32
 *   residual_out  [rows, D] in `dtype`, receives h rounded once; NULL: not written;
 *                 may be residual (in place) or x
 *   out           [rows, D] in out_dtype: `dtype` (y rounded once; may be x), or GDN_F8E4M3 with one scale a row:
 *                     out_scale[r] = max(max_i |y[r, i]|, GDN_FP8_AMAX_MIN) / 448
 *                     out[r, i]    = e4m3(y[r, i] / out_scale[r])
 *                 so that out[r, i] * out_scale[r] stands for y[r, i]; a row with a NaN
 *                 (or an infinity) in y is NaN whole, its scale too
 *   out_scale     [rows] fp32, read only where out_dtype is GDN_F8E4M3
 *   eps           >= 0
 * The squares are summed in fp32: a row whose sum passes its range (|h| of 1e19 and more) comes out as
 * zeros, and with eps = 0 one whose sum is zero (|h| of 1e-23 and less) as infinities or NaN.
 * rows in [0, 2^31), 1 <= D <= GDN_NORM_MAX_D; pointers aligned to their element;
 * residual_out and out may not share memory, nor with x or residual other than as whole arrays in
 * their place (an 8-bit out not at all): GDN_ERR_UNSUPPORTED.
 * With every pointer 16-byte aligned (and D <= 16384 in bf16, 8192 in fp32; a little less
 * where rows are not whole 16-byte pieces) the accesses are of 128 bits.  One launch on `stream`.
 */
#define GDN_FP8_AMAX_MIN 1e-30f
#define GDN_NORM_MAX_D 32768
gdn_status gdn_rmsnorm_residual(const void* x, const void* residual, const float* norm_weight, void* residual_out,
                                void* out, float* out_scale, int64_t rows, int64_t D, int32_t dtype,
                                int32_t out_dtype, float eps, gdn_stream_t stream);

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_GELU = 2, GDN_ACT_RELU = 3 } gdn_activation;

enum {
    /* The weight is stored [N', K] (nn.Linear.weight) instead of [K, N'] (its transpose, the
     * decode block's layout). */
    GDN_LINEAR_WEIGHT_NK = 1u << 0,
    /* The gated form: the weight, weight_scale and bias have N' = 2 N columns, the gate's N first. */
    GDN_LINEAR_GATED = 1u << 1,
    /* Run on the fp32 FFMA kernel even where the tensor-core kernels apply (a cross-check path). */
    GDN_LINEAR_FORCE_FFMA = 1u << 2
};

/*
 * 0 <= M <= 4194240 rows of x (0: nothing to do), N >= 1 columns of out, K >= 1;
 * N' = N, or 2 N under GDN_LINEAR_GATED; N' and K below 2^31 - 256.
 */
typedef struct {
    int64_t M, N, K;
    int32_t dtype;       /* of x and weight: GDN_BF16, GDN_F32 or GDN_F8E4M3 */
    int32_t out_dtype;   /* of out and residual: GDN_F32, or GDN_BF16 unless dtype is GDN_F32 */
    int32_t activation;  /* gdn_activation */
    uint32_t flags;      /* GDN_LINEAR_* */
} gdn_linear_dims;

/*
 * gdn_linear -- a matrix product with bias, activation and residual in its epilogue:
 *     a[m, n]   = x_scale[m] * weight_scale[n] * sum_k x[m, k] W[k, n] + bias[n]
 *     out[m, n] = act(a[m, n]) + residual[m, n]                              or, gated,
 *     out[m, n] = act(a[m, n]) * a[m, N + n] + residual[m, n]
 * with W[k, n] the weight's element in its layout; sums and the epilogue in fp32, one
 * rounding to out_dtype.  silu(v) = v / (1 + e^-v), gelu(v) = v/2 (1 + erf(v / sqrt 2)),
 * relu(v) = max(v, 0) (NaN stays NaN).  silu's relative error is at most (5 + 1.2 |v|) 2^-23 for v > -87, gelu's of
 * fp32 outputs (v^2 + 5) 2^-22 for v > -13, of bf16 outputs 0.75e-7 |v| before their rounding.
 *   x            [M, K] in dtype
 *   x_scale      [M] fp32 and weight_scale [N'] fp32: GDN_F8E4M3 only (NULL otherwise)
 *   weight       [K, N'] or, under GDN_LINEAR_WEIGHT_NK, [N', K], in dtype;
 *                GDN_F8E4M3 takes GDN_LINEAR_WEIGHT_NK only (else GDN_ERR_UNSUPPORTED)
 *   bias         [N'] fp32, or NULL
 *   residual     [M, N] in out_dtype, or NULL; may be out (in place)
 *   out          [M, N] in out_dtype; may not share memory with x, the weight or, other than in
 *                its place, the residual (GDN_ERR_UNSUPPORTED)
 * Sums of bf16 and e4m3 products are the tensor cores', which truncate a sum at every 16 terms; for
 * fp32 outputs at most 512 (e4m3: 1024) terms are summed so and the blocks added with rounding, so
 * that they are as near as fp32 sums (error about 5e-7 of the norm, and of a sum of one sign, for any K).
 * Pointers aligned to their element.  bf16 and e4m3 run on the tensor cores, in one launch on
 * `stream`, where x and the weight are 16-byte aligned with rows of a multiple of 16 bytes (a
 * gated [K, 2 N] weight: also N).  An operand that is not is copied to such rows first (one more
 * launch) where the product is large enough to pay for it (1e9 operations), and smaller ones run
 * on an FFMA kernel.  fp32 runs on the FFMA kernel, from 3e8 operations, 16 rows and up to
 * K = 4096 on the tensor cores: the operands are split into three bf16 parts each, which add up
 * exactly, and the products of parts down to 2^-16 are summed in fp32 (three launches).  Operands
 * that parts do not fit are found on the device and left to the FFMA kernel: infinities and NaN;
 * operands whose sums could pass fp32's range (K times the product of their largest magnitudes,
 * each rounded up to a power of two, above 2^127); an operand that is below 2^-100 whole, or both
 * where the product of their largest magnitudes is.  In the others, what single elements have below
 * 2^-133, the least bf16 number, is lost.  Copies and parts lie in scratch from cudaMallocAsync on
 * `stream`, freed there (gdn_linear_ws takes it from the caller); calls whose scratch cannot be had,
 * or would pass 4 GiB of parts, run on the FFMA kernel.  Results do not depend on what else runs:
 * every sum has one order for given arguments and device.
 */
gdn_status gdn_linear(const void* x, const float* x_scale, const void* weight, const float* weight_scale,
                      const float* bias, const void* residual, void* out, const gdn_linear_dims* dims,
                      gdn_stream_t stream);

/* Device scratch of a gdn_linear call with these operands (only their alignment matters) and
 * dims: 0 where none is needed, and for invalid dims.  Host only. */
size_t gdn_linear_workspace_bytes(const void* x, const void* weight, const gdn_linear_dims* dims);

/*
 * gdn_linear_ws -- gdn_linear with its scratch supplied by the caller, so that the call
 * allocates nothing: device memory of workspace_bytes >= gdn_linear_workspace_bytes(x, weight,
 * dims) bytes, 16-byte aligned, not touched by anything else until the call's work on `stream`
 * has finished; NULL: the call behaves exactly like gdn_linear.  A workspace that is too small
 * returns GDN_ERR_WORKSPACE (misaligned: GDN_ERR_ALIGN) and launches nothing.
 */
gdn_status gdn_linear_ws(const void* x, const float* x_scale, const void* weight, const float* weight_scale,
                         const float* bias, const void* residual, void* out, const gdn_linear_dims* dims,
                         void* workspace, size_t workspace_bytes, gdn_stream_t stream);

/* How gdn_linear runs a call. */
typedef enum {
    GDN_LINEAR_KERNEL_NONE = 0,   /* M = 0 */
    GDN_LINEAR_KERNEL_FEW = 1,    /* FMA units, few rows */
    GDN_LINEAR_KERNEL_FFMA = 2,   /* FMA units */
    GDN_LINEAR_KERNEL_SMALL = 3,  /* tensor cores, a CTA a tile of 128 weight columns, K over `splits` of them */
    GDN_LINEAR_KERNEL_PAIRS = 4,  /* tensor cores, a CTA pair a tile of 256 weight columns */
    GDN_LINEAR_KERNEL_JOINT = 5   /* the same with K over `splits` pairs */
} gdn_linear_kernel;
enum { GDN_LINEAR_OPERANDS_AS_THEY_LIE = 0, GDN_LINEAR_OPERANDS_COPIED = 1, GDN_LINEAR_OPERANDS_IN_PARTS = 2 };
typedef struct {
    int32_t kernel;    /* gdn_linear_kernel */
    int32_t operands;  /* GDN_LINEAR_OPERANDS_* (in parts: the FFMA kernel where the operands turn out not to fit) */
    int32_t tokens;    /* rows of x in a tile, and the CTAs or pairs that share K; tensor-core kernels only, else 0 */
    int32_t splits;
} gdn_linear_plan_info;

/* gdn_linear_plan -- how a gdn_linear call with these operands (only their alignment matters)
 * and dims runs on a device with sm_count SMs; invalid dims return gdn_linear's code for
 * them, sm_count < 1 GDN_ERR_DIMS.  Host only. */
gdn_status gdn_linear_plan(const void* x, const void* weight, const gdn_linear_dims* dims, int32_t sm_count,
                           gdn_linear_plan_info* info);

/*
 * Linear attention with a decay for each head: the recurrence without the delta rule's correction, of layers
 * that stand beside the gated delta rule's, with the same heads and the same state:
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T,     o_t = scale * S_t^T q_t
 *
 * gdn_linear_attn_prefill -- whole prompts.
 *   q, k        [B, Hk, S, Dk]  compute dtype (need not be normalised)
 *   v           [B, Hv, S, Dv]  compute dtype
 *   g_log       [B, Hv, S] fp32 log-decays, or [Hv] under GDN_HEAD_DECAY; <= 0 (not checked).  Values below -100
 *               count as -100 (e^-100 is 3.7e-44): -infinity drops what came before the token (if that is
 *               finite: an infinity or NaN in the state stays one)
 *   lengths     [B] int32 or NULL: sequence b has lengths[b] tokens (below 0: 0, above S: S).  Rows of q, k, v
 *               and g_log behind them have no influence, whatever they hold, and rows of out are left as they were
 *               (GDN_ZERO_PADDING: set to zero)
 *   state_in    [B, Hv, Dk, Dv] fp32, Dv contiguous, or NULL: zeros
 *   state_out   the same, receives the state behind the last token; may be state_in
 *   out         [B, Hv, S, Dv]  compute dtype
 *   dims        gdn_dims (S < 2^31 - 4096); flags: GDN_HEAD_DECAY, GDN_FORCE_FFMA, GDN_SINGLE_PASS, GDN_ZERO_PADDING.
 *               S = 0 copies the state
 *   workspace   device memory of workspace_bytes >= gdn_linear_attn_workspace_bytes(dims) bytes, 16-byte
 *               aligned, not touched by anything else until the call's work on `stream` has finished; NULL: the call
 *               takes what it needs with cudaMallocAsync on `stream`, and runs one pass where that fails.  Too small:
 *               GDN_ERR_WORKSPACE
 * Pointers aligned to their element; out and state_out may not share memory with an input or one
 * another, but for state_out in state_in's place (GDN_ERR_UNSUPPORTED).
 * bf16 with Dk and Dv multiples of 8 and q, k, v and out on 16 bytes runs on the tensor cores, in chunks of 128
 * tokens: products of bf16 operands with fp32 sums; the decayed scores and the copy of the state that the queries
 * read are rounded to bf16 once (the outputs' own type): outputs are some 0.0023 of their norm off, where their own
 * rounding makes 0.0017 (GDN_FORCE_FFMA: no others).  The state itself is fp32 and is updated with three bf16 parts
 * of exp(.) v, which add up to its 24 bits.  What a chunk's decays leave of the state is taken as e^-64 of it at least
 * in the chunk's outputs (1.6e-28).  An infinity or NaN in v may make NaN of its column's outputs from the beginning
 * of its chunk on (a score of zero in front of it is multiplied too), one in k from its token on, one in q of its
 * token's.  A token's sums over its chunk stand divided by e^c until the end, c >= -64 its log-decays since the chunk's
 * first token: where |q . k|, or the sum of the scores' products with v, passes 3.4e38 e^c (5e10 behind decays of
 * e^-64 and more), its outputs are infinite or NaN, although they may fit bf16.
 * fp32 runs the recurrence itself on the FMA units.  So does bf16 with more than 2^24 heads (B Hv), and with other head
 * dims in small calls (B Hv S Dk Dv up to 3e6) and for heads of a few tokens; other such calls go to the tensor cores by
 * copies of q, k, v and out with padded rows, in the workspace, and round as above.  The FMA units work in fp32
 * throughout.  They sum the log-decays of up to 16 tokens, and those sums' roundings (2^-22 at most) are their largest
 * error: outputs and states are some 1.5e-7 of their norm off behind decays of e^-0.25 a token.  A state is rounded and
 * multiplied by a rounded decay once in 16 tokens, which adds up over those that it remembers: 5e-6 after 8000 tokens at
 * one decay of e^-0.0005 for all (the tensor cores, once in 128: 5e-7 to 1.5e-6).  Products stand
 * multiplied by e^8 at most there: q, k and v, and the state, whose products and sums stay below 1e35 are safe.
 * Few sequences of many tokens are cut into segments that run at once (gdn_linear_attn_segments; GDN_SINGLE_PASS:
 * never): a first launch runs all but the last from zero and keeps their states and decays, a second adds them up to the
 * segments' start states (nothing to do for two segments), and the last runs every segment.  Results of a split agree
 * with one pass's to within rounding.  Many heads that are no whole number of rounds of the SMs: those left over run in
 * parts on several SMs, one handing the state on to the next through state_out (the same bits as one pass's;
 * GDN_SINGLE_PASS: never).  The same call on the same device gives the same bits; a batch's sequences do not influence
 * one another's, unless another batch size changes the split.
 * A wait inside the tensor-core kernel that runs out (some two seconds) ends it with GDN_ERR_TIMEOUT in the device's
 * status word (gdn_device_status) and undefined outputs.
 */
gdn_status gdn_linear_attn_prefill(const void* q, const void* k, const void* v, const float* g_log,
                                   const int32_t* lengths, float scale, const float* state_in, float* state_out,
                                   void* out, const gdn_dims* dims, void* workspace, size_t workspace_bytes,
                                   gdn_stream_t stream);

/* Segments that gdn_linear_attn_prefill cuts each sequence into on a device with sm_count SMs (1: none); 0 for
 * invalid dims or sm_count < 1.  Host only. */
int32_t gdn_linear_attn_segments(const gdn_dims* dims, int32_t sm_count);

/* Device scratch of gdn_linear_attn_prefill on the current device: a state a segment and head; a few KB of flags where
 * heads are handed on; copies of operands whose rows are padded; 0 without any of these, for invalid dims and without a
 * device.  Host only. */
size_t gdn_linear_attn_workspace_bytes(const gdn_dims* dims);

/*
 * gdn_linear_attn_step -- one token of every sequence (dims->S == 1, else GDN_ERR_DIMS): the arguments of
 * gdn_linear_attn_prefill (no lengths, no GDN_ZERO_PADDING), in fp32 throughout.  The state is read once and written once, in one launch.
 */
gdn_status gdn_linear_attn_step(const void* q, const void* k, const void* v, const float* g_log, float scale,
                                const float* state_in, float* state_out, void* out, const gdn_dims* dims,
                                gdn_stream_t stream);

enum {
    /* Channel pairs (2i, 2i + 1) instead of (i, i + R/2). */
    GDN_ROTARY_INTERLEAVED = 1u << 0,
    /* Turns back (by -theta): the transpose, so the gradient too. */
    GDN_ROTARY_INVERSE = 1u << 1,
    /* positions are int32 instead of int64. */
    GDN_ROTARY_POSITIONS_I32 = 1u << 2
};
#define GDN_ROTARY_MAX_D 4096

/*
 * B, S >= 0 (B S D < 2^31 - 4096); Hq, Hk in [0, 65536] heads of q and of k (0: that tensor is not there); head dim
 * 1 <= D <= GDN_ROTARY_MAX_D, of which the first R are turned (even, 2 <= R <= D).  Strides in elements over
 * (batch, head, token), >= 0, a dim's last row at most 2^56 elements from its first; channels are contiguous.
 */
typedef struct {
    int64_t B, Hq, Hk, S, D, R;
    int64_t q_strides[3], k_strides[3], q_out_strides[3], k_out_strides[3];
    int64_t position_stride;  /* of positions over the batch, in elements (0: one row for all) */
    int64_t first_position;   /* where positions is NULL: token s is at first_position + s */
    int32_t dtype;            /* GDN_F32 or GDN_BF16 */
    uint32_t flags;           /* GDN_ROTARY_* */
    float amplitude;          /* what turned channels are multiplied by (1, or a long-context scaling's factor) */
} gdn_rotary_dims;

/*
 * gdn_rotary -- rotary positions of q and k in one launch: with theta = position * inv_freq[i],
 *     y_a = amplitude (x_a cos theta - x_b sin theta),   y_b = amplitude (x_b cos theta + x_a sin theta)
 * for the channel pairs (a, b) = (i, i + R/2), or (2i, 2i + 1), i < R/2; channels from R on are copied.
 *   q, q_out   [B, Hq, S, D] in dtype at their strides (views into packed rows, head-major or token-major);
 *              q_out may be q at the same strides, and otherwise may not share memory with an input or with k_out
 *              (GDN_ERR_UNSUPPORTED; rows that lie among one another are taken where their strides show them apart, as
 *              those of packed rows do); its rows may not lie over one another (GDN_ERR_DIMS).  k, k_out likewise
 *   inv_freq   [R/2] fp64, radians a position (fp32 ones of a model: widened)
 *   positions  int64 (or int32) [B, S], tokens contiguous, or NULL
 * theta is taken mod one turn as a 64-bit fraction, off by at most 1.5 * 2^-64 of a turn a position, times |inv_freq|
 * where that is above 1 (2/pi is kept to 64 bits): frequencies of a model, up to 1, are as accurate at far positions as at
 * near ones.  cos and sin in fp32, one rounding to dtype.  Infinite and NaN frequencies turn nothing.
 * Pointers aligned to their element; accesses are as wide, up to 16 bytes, as every pointer, stride, R/2 (R for
 * GDN_ROTARY_INTERLEAVED) and D - R are multiples of.
 */
gdn_status gdn_rotary(const void* q, const void* k, const double* inv_freq, const void* positions, void* q_out,
                      void* k_out, const gdn_rotary_dims* dims, gdn_stream_t stream);

/* Device scratch a prefill with these dims needs on the current device: the
 * segment states, maps and identity-start outputs of a split (see gdn_prefill;
 * the split depends on the device's SM count), 0 when the call runs one pass.  0 as well for
 * invalid dims or when no CUDA device can be queried.  Host only. */
size_t gdn_prefill_workspace_bytes(const gdn_dims* dims);

/*
 * gdn_prefill_ws -- gdn_prefill with the scratch of a split supplied by the
 * caller.  No counterpart on the pages (their kernels allocate nothing the
 * caller sees); it exists so that a split prefill need not allocate.
 *   workspace        device memory of workspace_bytes >= gdn_prefill_workspace_bytes(dims)
 *                    bytes on the current device, 16-byte aligned, owned by the caller
 *                    and not touched by anything else until the call's work on `stream`
 *                    has finished; NULL: the call behaves exactly like gdn_prefill
 *                    (stream-ordered scratch of its own)
 * A non-NULL workspace that is too small returns GDN_ERR_WORKSPACE (misaligned:
 * GDN_ERR_ALIGN) and launches nothing.  Results are bit-identical to gdn_prefill's.
 */
gdn_status gdn_prefill_ws(const void* q, const void* k, const void* v,
                          const float* g_log, const float* beta, float scale,
                          float* state_inout, void* out, const gdn_dims* dims,
                          void* workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Segments gdn_prefill splits each sequence into for these dims on a device
 * with sm_count SMs (see gdn_prefill): 1 for one pass (every shape off the
 * tensor-core path, GDN_FORCE_FFMA, GDN_SINGLE_PASS, B == 0 or S == 0),
 * otherwise 2 .. 16.  0 for invalid dims or sm_count < 1.  Host only. */
int32_t gdn_prefill_segments(const gdn_dims* dims, int32_t sm_count);

/* gdn_prefill_segments, and where the segments start: with starts != NULL and
 * capacity >= P + 1 (P the return value), starts[j] is the first token of
 * segment j (starts[0] = 0) and starts[P] = S.  Segment 0 may be longer than
 * the others; segments 1 .. P - 2 have the same multiple of 128 tokens and the
 * last one ends at S.  No counterpart on the pages.  Host only. */
int32_t gdn_prefill_segment_starts(const gdn_dims* dims, int32_t sm_count, int64_t* starts, int32_t capacity);

/* Static, NUL-terminated description of a status code. */
const char* gdn_status_string(gdn_status s);

/*
 * gdn_device_status -- read (and, when clear != 0, reset to 0) the kernel-side
 * status word of CUDA device `device`.  0 means no kernel reported a problem;
 * otherwise the value is a gdn_status (GDN_ERR_TIMEOUT).  Synchronises the
 * device.  Returns GDN_ERR_NULL if code is NULL, GDN_ERR_CUDA if the copy fails.
 */
gdn_status gdn_device_status(int device, int clear, int32_t* code);

/*
 * gdn_set_wait_limit_ns -- the time after which a wait inside the tensor-core
 * prefill (gdn_prefill on bf16 with Dk = Dv = 128) gives up, on CUDA device
 * `device`: ns > 0 sets it, 0 restores the default of one second.  A wait that
 * gives up records GDN_ERR_TIMEOUT in the status word (gdn_device_status), the
 * CTA's roles stop, every copy and product already in flight is drained (those
 * drains keep their own one-second bound) and the CTA frees its tensor memory
 * and exits; the outputs of such a call are undefined.  This exists to exercise
 * that path without a GPU fault (a limit of a few microseconds makes ordinary
 * waits run out); it synchronises the device.  The pages define no such knob.
 * gdn_linear_attn_prefill's waits keep a bound of their own, some two seconds,
 * whatever is set here.
 * Returns GDN_ERR_CUDA if the device cannot be selected or the value not set.
 */
gdn_status gdn_set_wait_limit_ns(int device, uint64_t ns);

/*
 * gdn_test_stall_prefill -- test hook for the path above, on CUDA device `device`:
 * while on != 0, every CTA of the tensor-core prefill first waits on a barrier
 * that nothing arrives at, so that the wait runs out after the wait limit (set
 * it low with gdn_set_wait_limit_ns) and the call takes its give-up path:
 * GDN_ERR_TIMEOUT in the status word, nothing computed.  So does every CTA of
 * gdn_linear_attn_prefill's tensor-core kernel, in calls made (or captured) while
 * on != 0; its launches take some two seconds each.  No GPU fault is
 * involved.  Synchronises the device.  Off by default; the pages define no
 * such hook.  Returns GDN_ERR_CUDA if the device cannot be selected or the
 * value not set.
 */
gdn_status gdn_test_stall_prefill(int device, int on);

/* Number of kernels one call of gdn_prefill (in one pass), gdn_decode_step,
 * gdn_decode_gated or the conv1d entry points launches: one.  A split prefill
 * launches four, gdn_decode_block and gdn_prefill_gated two. */
int gdn_kernels_per_call(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
