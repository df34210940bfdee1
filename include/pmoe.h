/*
 * pmoe -- per-token NVFP4 routed-MoE expert path for AMD Instinct MI355X (gfx950).
 *
 * C ABI. Every compute entry point enqueues HIP kernels on the caller's stream
 * (`stream` is a hipStream_t; NULL means the legacy default stream), returns a
 * status code, and never allocates device memory, synchronizes, or aborts.
 * The routed-MoE entry points may also enqueue work on one library-owned
 * stream per device (created on first use, default priority, kept until the
 * process ends), forked from and joined back into the caller's stream with
 * events, so the call stays ordered on the caller's stream and can be captured
 * in a graph.
 * All tensors are caller-owned device buffers (the library keeps no pointer to
 * them after the call returns and caches nothing about them). All checks run on
 * the host before the first launch; when a call returns an error, no kernel was
 * launched and no output was touched (PMOE_ERR_HIP is the one exception: it
 * reports a failed launch after validation passed).
 *
 * Sources of the contract (three public pages):
 *   [Megatron-LM #8262]  per-token NVFP4 squared-ReLU and SwiGLU MoE via FlashInfer
 *                        CuTe DSL (sections: Background, What is added, How to extend,
 *                        What is tested).
 *   [FlashInfer #5019]   CuTe DSL NVFP4 W4A16 MegaMoE (section: Tensor and numerical
 *                        contract).
 *
 * Notation: T tokens, H hidden size, I intermediate size, E local experts,
 * K top-k, N1 = FC1 output width (2*I gated / SwiGLU, I non-gated / squared ReLU),
 * R = number of valid routes (at most T*K).
 *
 * Number formats (NVFP4): E2M1 codes packed two per byte, element 2i in the low
 * nibble; one E4M3 (fn, max 448) block scale per 16 consecutive elements along
 * the reduction dimension; one FP32 scale per token (activations) or per expert
 * (weights, "alpha") [Megatron-LM #8262 . Background; FlashInfer #5019 . Tensor
 * and numerical contract]. BF16 tensors are passed as raw 16-bit storage.
 *
 * Shape limits of this build: H and I multiples of 16 (one block) in
 * [16, 16384]; 1 <= K <= min(32, E); 1 <= E <= 1024; T >= 0 (T == 0 is a
 * successful no-op); T*Hp and T*K*Ip below 2^31, where Hp and Ip are H and I
 * rounded up to a multiple of 64 (the W4A16 recipe: 2*T*Hp and 2*T*K*Ip). The
 * grouped GEMMs reduce over whole chunks of 64 elements: a reduction length
 * that is not a multiple of 64 is padded inside the library with zero codes
 * and zero block scales, which add exactly zero to every sum; the canonical
 * arrays at this interface are never padded.
 */
#ifndef PMOE_H_
#define PMOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- status codes */
#define PMOE_OK 0
#define PMOE_ERR_DEVICE 1    /* current device is not gfx950 (MI355X / MI350X)          */
#define PMOE_ERR_POINTER 2   /* null, host, or misaligned pointer                       */
#define PMOE_ERR_SHAPE 3     /* unsupported sizes, or FC1 width neither I nor 2*I         */
#define PMOE_ERR_ACT 4       /* activation kind disagrees with the FC1 shape             */
#define PMOE_ERR_WORKSPACE 5 /* workspace smaller than the queried size                  */
#define PMOE_ERR_HIP 6       /* a HIP runtime call or kernel launch failed               */
#define PMOE_ERR_ARG 7       /* any other invalid argument (unknown enum value, ...)     */

/* Activation kinds. Squared ReLU is the non-gated expert, SwiGLU the gated one;
 * SwiGLU iff FC1 has twice FC2's input width [Megatron-LM #8262 . What is added]. */
#define PMOE_ACT_RELU2 0
#define PMOE_ACT_SWIGLU 1

/* Element type of topk_ids: signed 32- or 64-bit [FlashInfer #5019 . Tensor and
 * numerical contract, 'Inputs/output']. */
#define PMOE_IDS_INT32 0
#define PMOE_IDS_INT64 1

/* Library version (major*10000 + minor*100 + patch). */
int pmoe_version(void);

/* Message of the last error returned on this host thread: "" after a call
 * that succeeded. The pointer stays valid until the next pmoe call on the
 * same thread. */
const char* pmoe_last_error(void);

/* ============================================================ prepared weights
 *
 * Prepared (kernel-native) layout of one FC matrix with logical shape
 * [E, N, Kd] (N output rows, Kd the reduction length; FC1: N = N1, Kd = H;
 * FC2: N = H, Kd = I). Rows are grouped in blocks of 32 ("col blocks" p,
 * NB = ceil(N/32), or 2*ceil(I/32) for a gated FC1; padded with all-zero
 * blocks to NBp = NB rounded up to a multiple of 8), blocks in column tiles
 * of 8 (ct = p/8, pos = p%8, NT = NBp/8), and the reduction in chunks of 64
 * (c, KC = ceil(Kd/64); the elements in [Kd, 64*KC) are zero). Rows of a block
 * past the matrix (past I in each half of a gated FC1) are zero. Chunk c of a column tile --
 * all 8 of its blocks -- is one contiguous slab, so a GEMM workgroup owning
 * the tile streams a single sequential region:
 *
 *   codes  (uint8, E*NBp*32*Kd/2 bytes): byte offset
 *            (((((e*NT + ct)*KC + c)*8 + pos)*64 + lane)*16 + (2*h + s)*4 + i/2
 *          holds element k = c*64 + 32*s + 8*(lane/16) + i (nibble i%2, low first)
 *          of row n(p, 16*h + lane%16), for h, s in 0..1, i in 0..7 (the operand
 *          order of a 16x16x32 MFMA: lane = column, 8 consecutive k per lane).
 *   scales (uint8, E*NBp*32*Kd/16 bytes): byte offset
 *            ((((e*NT + ct)*KC + c)*8 + pos)*32 + d)*4 + 2*h + s
 *          holds the E4M3 scale of 16-block (c*4 + 2*s + d/16) of row
 *          n(p, 16*h + d%16), for d in 0..31.
 *   alpha  (float32, E values).
 *
 * Row map n(p, col): non-gated FC1 and FC2: n = 32*p + col. Gated FC1 (N1 = 2I)
 * interleaves gate and up blocks so one workgroup holds both halves of a SwiGLU
 * output: p even -> gate row 32*(p/2) + col; p odd -> up row I + 32*(p/2) + col
 * (for 32*(p/2) + col < I)
 * (gate rows are [0, I), up rows [I, 2I) of the canonical FC1 [FlashInfer #5019 .
 * Tensor and numerical contract, 'gate-then-up']).
 *
 * The bytes are the canonical codes/scales of the per-expert NVFP4 recipe
 * (packed [E, N, Kd/2], linear scales [E, N, Kd/16]) permuted by this map
 * (padding is zero); no value is changed and alpha is never folded into the
 * block scales.
 */

/* Sizes in bytes of the four prepared arrays: sizes[0] FC1 codes, sizes[1] FC1
 * scales, sizes[2] FC2 codes, sizes[3] FC2 scales (alphas are E floats each).
 * Host only. Returns PMOE_ERR_SHAPE for unsupported sizes. */
int pmoe_weight_bytes(int E, int N1, int H, int I, size_t sizes[4]);

/* Device workspace needed by pmoe_prepare_weights (bytes). 0 on bad shapes. */
size_t pmoe_prepare_workspace_bytes(int E, int N1, int H, int I);

/*
 * Quantize BF16 expert stacks into the prepared NVFP4 layout
 * [Megatron-LM #8262 . What is added, 'prepare_routed_nvfp4_weights'].
 *   w1 : BF16 [E, N1, H], gate rows then up rows when N1 == 2*I.
 *   w2 : BF16 [E, H, I].
 * Per expert and FC: amax over the whole matrix (gate and up together),
 * w_scale = fp32(2688 / amax), alpha = fp32(1 / w_scale); each 16-block gets the
 * E4M3 scale fp32(fp32(amax_b / 6) / alpha) (round to nearest even, saturating
 * at 448) and E2M1 codes of fp32(w / fp32(dec(scale) * alpha)) (round to nearest,
 * ties to the even code, saturating at 6). An all-zero expert gets alpha = 0 and
 * zero bytes.
 * Outputs are written in place, so their addresses stay valid across refreshes
 * (in-place refit) [Megatron-LM #8262 . What is added]. Gating is detected from
 * the shapes: N1 == 2*I gated, N1 == I non-gated, else PMOE_ERR_SHAPE.
 * ws: at least pmoe_prepare_workspace_bytes(...) bytes of device memory.
 * Alignment: every pointer 16-byte aligned.
 */
int pmoe_prepare_weights(const void* w1, const void* w2, int E, int N1, int H, int I,
                         void* w1_codes, void* w1_scales, float* w1_alpha,
                         void* w2_codes, void* w2_scales, float* w2_alpha,
                         void* ws, size_t ws_bytes, void* stream);

/*
 * Preparation for the per-tensor NVFP4 recipe [Megatron-LM #8262 . How to
 * extend, 'per_tensor']: codes and block scales exactly as pmoe_prepare_weights,
 * with the static FC1 / FC2 input scales folded into the alphas:
 *   w1_alpha[e] = fp32(1 / fp32(w_scale1[e] * a1)),
 *   w2_alpha[e] = fp32(1 / fp32(w_scale2[e] * a2)).
 *   a1_scale, a2_scale : device float32 scalars (4-byte aligned), read by the
 *                        kernels, so the call never waits on the host. They
 *                        use the weights' convention, a = 2688 / calibrated
 *                        amax, and must be positive and finite (not checked:
 *                        they live on the device).
 * Other arguments, layout and errors as pmoe_prepare_weights.
 */
int pmoe_prepare_weights_per_tensor(const void* w1, const void* w2, int E, int N1, int H, int I,
                                    const float* a1_scale, const float* a2_scale,
                                    void* w1_codes, void* w1_scales, float* w1_alpha,
                                    void* w2_codes, void* w2_scales, float* w2_alpha,
                                    void* ws, size_t ws_bytes, void* stream);

/* ============================================================ activations */

/*
 * Per-token NVFP4 quantization of BF16 activations [Megatron-LM #8262 .
 * Background; What is added, 'quantize_routed_nvfp4_input'; How to extend,
 * 'FC1 input' and 'per_token_scale'].
 *   x       : BF16 [T, H] (row-major, contiguous)
 *   xq      : uint8 [T, H/2] packed E2M1 codes (canonical layout)
 *   x_sf    : uint8 [T, H/16] E4M3 block scales
 *   x_scale : float32 [T] per-token scale
 * Per token: g = fp32(amax * fp32(1/2688)) (the recipe constant 1/(448*6));
 * per 16-block: scale = E4M3(fp32(fp32(amax_b / 6) / g)), codes =
 * E2M1(fp32(x / fp32(dec(scale) * g))); g == 0 (all-zero token) gives zero bytes.
 * Bit-exact IEEE binary32 with denormals. Alignment: xq and x 16 bytes,
 * x_sf 4 bytes, x_scale 4 bytes.
 */
int pmoe_quantize_input_per_token(const void* x, int T, int H,
                                  void* xq, void* x_sf, float* x_scale, void* stream);

/*
 * NVFP4 quantization of BF16 activations with a static, calibrated scale
 * (per-tensor recipe) [Megatron-LM #8262 . How to extend, 'per_tensor', row
 * 'FC1 input']: every row uses g = fp32(1 / a1) in the block steps of
 * pmoe_quantize_input_per_token; blocks beyond the scale's range saturate
 * (scale 448, codes +-6). No per-token scale is produced.
 *   a1_scale : device float32 scalar (a1 = 2688 / calibrated amax), positive and finite
 *   xq, x_sf : as pmoe_quantize_input_per_token.
 */
int pmoe_quantize_input_per_tensor(const void* x, int T, int H, const float* a1_scale,
                                   void* xq, void* x_sf, void* stream);

/*
 * The same per-row NVFP4 quantizer applied to FP32 rows: the requantization of
 * the FP32 expert intermediate before FC2 [Megatron-LM #8262 . How to extend,
 * 'fc2_input_scale'; What is tested, 4. Train-gen parity]. routed_moe runs this
 * quantizer on its intermediate; it is exported so it can be checked alone.
 *   h : float32 [R, L], L a multiple of 16 up to 16384;  hq : uint8 [R, L/2];
 *   h_sf : uint8 [R, L/16];  h_scale : float32 [R].
 */
int pmoe_quantize_rows_f32(const float* h, int R, int L,
                           void* hq, void* h_sf, float* h_scale, void* stream);

/* ============================================================ routed MoE */

/* Device workspace needed by pmoe_routed_moe (bytes). 0 on bad shapes. */
size_t pmoe_moe_workspace_bytes(int T, int K, int E, int H, int I, int act);

/* Fields of the routed_moe workspace, for inspection (offsets in bytes). */
#define PMOE_WS_ROW_OF_ROUTE 0   /* int32 [T*K]   expert-sorted row of route t*K+j, -1 if invalid */
#define PMOE_WS_ROUTE_OF_ROW 1   /* int32 [T*K]   route index of each row (first R valid)        */
#define PMOE_WS_EXPERT_OFFSETS 2 /* int32 [E+1]   first row of each local expert; [E] = R          */
#define PMOE_WS_COUNTERS 3       /* int32 [4]     {R, number of M-tiles, first M-tile and first row
                                    of the experts run on the second stream}                    */
#define PMOE_WS_H 4              /* float32 [T*K, I]   activation output (rows < R valid);
                                    BF16 [T*K, Ip] under pmoe_routed_moe_w4a16 (Ip = I rounded
                                    up to 64; columns past I are 0)                             */
#define PMOE_WS_HQ 5             /* uint8 [T*K, Ip/2]  requantized intermediate codes (past I/2: 0) */
#define PMOE_WS_H_SF 6           /* uint8 [T*K, Ip/16] its E4M3 block scales (past I/16: 0)         */
#define PMOE_WS_H_SCALE 7        /* float32 [T*K]      its per-row scales (per-token recipe only)   */
#define PMOE_WS_Z 8              /* BF16 [T*K, H]      per-route FC2 outputs                         */
#define PMOE_WS_NUM_FIELDS 9

/* Offsets (bytes, from the workspace base) of the fields above. Host only. */
int pmoe_moe_workspace_layout(int T, int K, int E, int H, int I, int act,
                              size_t offsets[PMOE_WS_NUM_FIELDS]);

/*
 * Routed-MoE expert path on per-token-quantized activations: routing, FC1
 * grouped GEMM, activation, per-row requantization, FC2 grouped GEMM, and the
 * deterministic finalize [Megatron-LM #8262 . What is added,
 * 'flashinfer_routed_nvfp4_moe'; FlashInfer #5019 . Tensor and numerical
 * contract, 'Compute order'].
 *   xq, x_sf, x_scale : output of pmoe_quantize_input_per_token for [T, H]
 *   topk_ids          : [T, K] int32 or int64 (ids_type); a route is valid iff
 *                       expert_offset <= id < expert_offset + E, others
 *                       (e.g. -1 fill) contribute nothing
 *   topk_w            : float32 [T, K] routing weights, applied in the finalize
 *   N1                : FC1 width the weights were prepared with (I or 2*I, else
 *                       PMOE_ERR_SHAPE)
 *   weights           : the six prepared arrays of pmoe_prepare_weights
 *   act               : PMOE_ACT_RELU2 (needs N1 == I) or PMOE_ACT_SWIGLU (needs
 *                       N1 == 2*I); a disagreement is PMOE_ERR_ACT
 *   ws                : at least pmoe_moe_workspace_bytes(T, K, E, H, I, act) bytes
 *   out               : BF16 [T, H]
 * Per valid route (token t, expert e), row r:
 *   y = fp32(sum_k dec(xq[t,k]) * dec(W1[e,:,k])) * fp32(x_scale[t] * alpha1[e])
 *   h = max(y,0)^2  or  silu(y_gate) * y_up, in FP32
 *   (hq, h_sf, h_scale) = per-row quantization of h (as pmoe_quantize_rows_f32)
 *   z = bf16(fp32(sum_k dec(hq) * dec(W2[e])) * fp32(h_scale[r] * alpha2[e]))
 * and out[t] = bf16(sum over slots j = 0..K-1 in order of fp32(w[t,j] * z)),
 * accumulated in FP32 from +0 without fused multiply-add. A token with no
 * valid route gets +0. The result of a token depends only on its own inputs
 * (batch invariant): the tiling never depends on T and no split-K is used.
 * Alignment: ws 256 bytes (its fields start on 256-byte boundaries); int64
 * topk_ids 8 bytes, int32 topk_ids, x_scale and topk_w 4 bytes; every other
 * pointer 16 bytes. A misaligned pointer is PMOE_ERR_POINTER. The same rules hold
 * for every entry point below that takes these arguments.
 */
int pmoe_routed_moe(const void* xq, const void* x_sf, const float* x_scale,
                    const void* topk_ids, int ids_type, const float* topk_w,
                    int T, int K, int E, int H, int I, int N1, int expert_offset,
                    const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                    const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                    int act, void* ws, size_t ws_bytes, void* out, void* stream);

/*
 * pmoe_routed_moe for callers that cannot allocate device memory (code under
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same arguments without ws / ws_bytes, the same results bit for bit. The
 * workspace is a static device array of PMOE_STATIC_SCRATCH_BYTES that the
 * library holds on every device it runs on until the process ends; the call
 * allocates nothing (no hipMalloc, no library stream or event: everything runs
 * on `stream`). Sizes whose workspace (pmoe_moe_workspace_bytes) exceeds the
 * scratch are PMOE_ERR_WORKSPACE -- at H = 7168, I = 3072 that is about 2300
 * routes (T*K). Every call on one device shares that device's scratch: calls
 * that overlap in time on one device (two streams, two host threads) race and
 * corrupt each other's results; serialize them.
 */
#define PMOE_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
int pmoe_routed_moe_static(const void* xq, const void* x_sf, const float* x_scale,
                           const void* topk_ids, int ids_type, const float* topk_w,
                           int T, int K, int E, int H, int I, int N1, int expert_offset,
                           const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                           const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                           int act, void* out, void* stream);

/* Steps of pmoe_routed_moe, for callers that time or interleave them. */
#define PMOE_STEP_ROUTE 0    /* histogram, scan, tile list, scatter (3 kernels)   */
#define PMOE_STEP_FC1 1      /* FC1 grouped GEMM + activation -> h                */
#define PMOE_STEP_REQUANT 2  /* per-row requantization of h -> hq, h_sf, h_scale  */
#define PMOE_STEP_FC2 3      /* FC2 grouped GEMM -> z                            */
#define PMOE_STEP_FINALIZE 4 /* fixed-order finalize -> out                      */

/*
 * Runs steps first..last (inclusive) of pmoe_routed_moe with the same
 * arguments and workspace; pmoe_routed_moe is steps 0..4. A step reads what the
 * earlier steps left in the workspace, so running the steps one range after
 * another on the same stream gives exactly the result of one full call.
 * PMOE_ERR_ARG unless 0 <= first <= last <= 4.
 */
int pmoe_routed_moe_steps(int first, int last,
                          const void* xq, const void* x_sf, const float* x_scale,
                          const void* topk_ids, int ids_type, const float* topk_w,
                          int T, int K, int E, int H, int I, int N1, int expert_offset,
                          const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                          const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                          int act, void* ws, size_t ws_bytes, void* out, void* stream);

/*
 * The routed path under the per-tensor NVFP4 recipe [Megatron-LM #8262 . How
 * to extend, 'per_tensor']. As pmoe_routed_moe, except:
 *   xq, x_sf   : output of pmoe_quantize_input_per_tensor (no per-token scale)
 *   weights    : output of pmoe_prepare_weights_per_tensor (folded alphas)
 *   a2_scale   : device float32 scalar, the static FC2 input scale
 *   y = fp32(sum_k dec(xq[t,k]) * dec(W1[e,:,k])) * alpha1'[e]
 *   (hq, h_sf) = quantization of h with g = fp32(1 / a2) for every row
 *   z = bf16(fp32(sum_k dec(hq) * dec(W2[e])) * alpha2'[e])
 * The workspace's h_scale field is not written.
 */
int pmoe_routed_moe_per_tensor(const void* xq, const void* x_sf,
                               const void* topk_ids, int ids_type, const float* topk_w,
                               int T, int K, int E, int H, int I, int N1, int expert_offset,
                               const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                               const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                               const float* a2_scale, int act, void* ws, size_t ws_bytes,
                               void* out, void* stream);

/*
 * The routed path with BF16 activations and NVFP4 weights (W4A16, the
 * 'weight_only' recipe) [Megatron-LM #8262 . How to extend, 'weight_only';
 * FlashInfer #5019 . Tensor and numerical contract, 'Compute order'].
 *   x       : BF16 [T, H] activations, not quantized
 *   weights : output of pmoe_prepare_weights (alphas = 1 / w_scale)
 * Per valid route, row r:
 *   y = fp32(sum_k x[t,k] * dec(W1[e,:,k])) * alpha1[e]     (BF16 x BF16 MFMA, FP32 sum)
 *   h = bf16(max(y,0)^2  or  silu(y_gate) * y_up)           (activation in FP32, one rounding)
 *   z = bf16(fp32(sum_k h[r,k] * dec(W2[e,:,k])) * alpha2[e])
 * then the same fixed-order finalize. The workspace's h field holds BF16 h;
 * hq, h_sf and h_scale are not written. Other arguments as pmoe_routed_moe.
 */
int pmoe_routed_moe_w4a16(const void* x, const void* topk_ids, int ids_type, const float* topk_w,
                          int T, int K, int E, int H, int I, int N1, int expert_offset,
                          const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                          const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                          int act, void* ws, size_t ws_bytes, void* out, void* stream);

/* Options of pmoe_routed_moe_ex. */
#define PMOE_RECIPE_PER_TOKEN 0  /* per-token NVFP4 x NVFP4 (x = xq, x_sf, x_scale)        */
#define PMOE_RECIPE_PER_TENSOR 1 /* per-tensor NVFP4 x NVFP4 (x = xq, x_sf; a2_scale)       */
#define PMOE_RECIPE_W4A16 2      /* BF16 x NVFP4 (x = BF16 activations)                     */
#define PMOE_FINALIZE_ORDERED 0  /* fixed slot order, BF16 z per route: batch invariant     */
#define PMOE_FINALIZE_FUSED 1    /* FP32 atomic adds inside FC2: order-free, not invariant  */

typedef struct pmoe_moe_options {
  int recipe;             /* PMOE_RECIPE_*                                                  */
  int finalize;           /* PMOE_FINALIZE_*                                                */
  float swiglu_limit;     /* > 0: SwiGLU clamp, gate <= L and -L <= up <= L; 0: none         */
  const float* a2_scale;  /* per-tensor recipe: device float32 scalar; otherwise NULL       */
  int streams;            /* 0: automatic (two once T*K >= 2048); 1: one stream; 2: the
                             experts are cut at the expert boundary nearest 44 % of the
                             M-tiles and the two parts run FC1 -> requant -> FC2 on the
                             caller's stream and on a second stream, joined before the
                             finalize (same bits either way; needs E >= 2)              */
  const float* a1_scale;  /* pmoe_moe_forward, per-tensor recipe: device float32 scalar
                             (the static FC1 input scale); otherwise NULL               */
  void* const* step_events; /* NULL, or PMOE_STEP_EVENTS caller-created hipEvent_t handles
                             (created with timing enabled, for timing only: not under
                             graph capture), recorded on the stream that runs each
                             grouped GEMM: [0]/[1] before/after FC1 of the first part
                             of the experts, [2]/[3] FC1 of the second part, [4]/[5] FC2
                             of the first part, [6]/[7] FC2 of the second part. With
                             one stream both pairs of a GEMM are recorded around its
                             one launch. A NULL entry is skipped.                     */
} pmoe_moe_options;

#define PMOE_STEP_EVENTS 8

/*
 * The routed path with options; options == NULL means per-token, ordered, no
 * clamp (exactly pmoe_routed_moe).
 *   recipe       : which entry point's contract x / x_sf / x_scale and the
 *                  weights follow (pmoe_routed_moe, pmoe_routed_moe_per_tensor,
 *                  pmoe_routed_moe_w4a16; unused inputs may be NULL).
 *   finalize     : PMOE_FINALIZE_FUSED is the order-free mode the two-stage
 *                  finalize replaces [Megatron-LM #8262 . What is added; Why
 *                  CuTe DSL, 'Controllable determinism']: each route's FC2
 *                  value fp32(acc * scale), times its routing weight, is added
 *                  with FP32 atomics into a per-token FP32 row that is rounded
 *                  to BF16 once. The order of additions is not fixed, so the
 *                  result may differ in the last FP32 bits between runs and is
 *                  not batch invariant; z is not written.
 *   swiglu_limit : the clamp of [FlashInfer #5019 . Tensor and numerical
 *                  contract, 'Compute order']; PMOE_ERR_ARG unless act is
 *                  SwiGLU (or the limit is 0).
 *   streams      : see the struct; automatic means two streams once T*K >= 2048.
 * Other arguments, layout and errors as the recipe's own entry point.
 */
int pmoe_routed_moe_ex(const void* x, const void* x_sf, const float* x_scale,
                       const void* topk_ids, int ids_type, const float* topk_w,
                       int T, int K, int E, int H, int I, int N1, int expert_offset,
                       const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                       const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                       int act, const pmoe_moe_options* options,
                       void* ws, size_t ws_bytes, void* out, void* stream);

/*
 * The whole routed layer from BF16 activations: for the NVFP4 recipes the
 * input is quantized inside the call (per token, or with options->a1_scale for
 * the per-tensor recipe) into the workspace: up to T*K = 8192 routes in the
 * same launch as the routing, on the caller's stream; above that on the
 * library's second stream while the routing runs on the caller's. Then the
 * path of pmoe_routed_moe_ex. For PMOE_RECIPE_W4A16 it is pmoe_routed_moe_ex on x.
 *   x : BF16 [T, H]. Other arguments, options and errors as pmoe_routed_moe_ex
 *   (options == NULL: per-token, ordered, no clamp). The bits of the result
 *   equal quantize + pmoe_routed_moe(_ex) on the same inputs.
 */
int pmoe_moe_forward(const void* x, const void* topk_ids, int ids_type, const float* topk_w,
                     int T, int K, int E, int H, int I, int N1, int expert_offset,
                     const void* w1_codes, const void* w1_scales, const float* w1_alpha,
                     const void* w2_codes, const void* w2_scales, const float* w2_alpha,
                     int act, const pmoe_moe_options* options,
                     void* ws, size_t ws_bytes, void* out, void* stream);

/*
 * Router front: top-k experts and their routing weights from FP32 logits
 * (plain top-k, no group-limited routing [Megatron-LM #8262 . Performance]).
 *   logits    : float32 [T, E], finite, 1 <= E <= 1024
 *   topk_ids  : int32 [T, K] out, 1 <= K <= min(32, E): the K largest logits,
 *               larger first, equal logits ordered by lower expert id (exact:
 *               the choice is made on the logits, and softmax preserves order)
 *   topk_w    : float32 [T, K] out: p = exp(l - max) / sum_e exp(l_e - max) in
 *               FP32 (deterministic order), divided by the sum of the K chosen
 *               p (in slot order) when renormalize == 1
 * Alignment: 4 bytes.
 */
int pmoe_router_topk(const float* logits, int T, int E, int K, int renormalize,
                     int32_t* topk_ids, float* topk_w, void* stream);

/*
 * Deterministic two-stage finalize, standalone [Megatron-LM #8262 . Background,
 * 'two-stage finalize'; FlashInfer #5019 . Tensor and numerical contract]:
 *   out[t, :] = bf16( sum_{j=0..K-1, row(t,j) >= 0} fp32(w[t,j] * z[row(t,j), :]) )
 * in FP32 from +0, slot order, no fused multiply-add, one BF16 rounding.
 *   z : BF16 [R, H];  row_of_route : int32 [T*K] (-1 = skip; values must be < R);
 *   topk_w : float32 [T, K];  out : BF16 [T, H].
 * H must be a multiple of 8. Alignment: z and out 16 bytes, others 4 bytes.
 */
int pmoe_finalize(const void* z, const int32_t* row_of_route, const float* topk_w,
                  int T, int K, int H, void* out, void* stream);

/* ============================================================ router, training side
 *
 * A token is active when one of its ids is in [0, E) and one of its logits is
 * not -inf; a token of padding (all ids -1, say) counts nowhere and has a zero
 * gradient. Sequence s holds the tokens seq_offsets[s] .. seq_offsets[s+1] - 1;
 * seq_offsets is int32 [S+1] on the device, ascending, from >= 0 to <= T, or
 * NULL for one sequence of all tokens (S = 1). Sequences may be empty; tokens
 * before the first or behind the last belong to none. With p = softmax(logits)
 * over all E experts, lse = log sum exp(logits), n_s the active tokens and c_se
 * the routes of sequence s to expert e:
 *   balance_s = E * sum_e c_se / (n_s K) * sum_t p_te / n_s
 *   z_s       = sum_t lse_t^2 / n_s
 * and both are 0 when n_s = 0. balance_s is 1 at an even load of all n_s K slots;
 * slots without an expert are in K but not in c_se.
 */

#define PMOE_MAX_SEQUENCES 65536

/* Device workspace of pmoe_router_balance (bytes). 0 on bad shapes. */
size_t pmoe_router_balance_workspace_bytes(int T, int E, int K, int S);

/*
 * Expert counts, balance loss and z-loss of each sequence.
 *   logits      : float32 [T, E];  topk_ids : [T, K] int32 or int64 (ids_type), as
 *                 pmoe_router_topk gives them; ids outside [0, E) are no routes
 *   counts      : int32 [S, E] out, c_se;   tokens : int32 [S] out, n_s
 *   prob        : float32 [S, E] out, sum_t p_te (not divided by n_s, so that
 *                 counts, tokens and prob of several ranks can be added)
 *   balance, z  : float32 [S] out
 * T = 0 writes zeros. Sums over tokens are taken in a fixed order: the same
 * inputs give the same bits. 1 <= E <= 1024, 1 <= K <= min(32, E), T*K < 2^30,
 * 1 <= S <= PMOE_MAX_SEQUENCES. Alignment: ws 16 bytes, int64 ids 8, others 4.
 * The outputs and ws share no memory with each other or with an input.
 */
int pmoe_router_balance(const float* logits, const void* topk_ids, int ids_type, int T, int K, int E,
                        const int32_t* seq_offsets, int S,
                        int32_t* counts, int32_t* tokens, float* prob, float* balance, float* z,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * Gradient of the logits.
 *   counts, tokens : of pmoe_router_balance, or their sums over ranks (then p of
 *                    this rank's tokens meets the load of all)
 *   d_balance, d_z : float32 [S], gradients of the two losses, or NULL
 *   d_topk_w       : float32 [T, K], gradient of the weights of pmoe_router_topk
 *                    called with the same `renormalize`, or NULL. With
 *                    renormalize = 1 the weights are p over the sum of the slots that have
 *                    an expert in topk_ids. pmoe_router_topk divides by the sum over all K: where
 *                    a slot is dropped after it, keep the slot's id here and give it a
 *                    zero d_topk_w
 *   d_logits       : float32 [T, E] out: the sum of the gradients that are given;
 *                    every row is written. Tokens of no sequence have no part in the
 *                    losses, but may have one in d_topk_w.
 * counts is needed with d_balance, tokens with d_balance or d_z. With
 * renormalize = 1 a token whose chosen experts together have less than 1e-37 of
 * the largest p gets no gradient from d_topk_w. d_logits may be logits itself, but
 * shares no memory with another argument that the call reads. Limits and alignment as above.
 */
int pmoe_router_backward(const float* logits, const void* topk_ids, int ids_type, int T, int K, int E,
                         int renormalize, const int32_t* seq_offsets, int S,
                         const int32_t* counts, const int32_t* tokens,
                         const float* d_balance, const float* d_z, const float* d_topk_w,
                         float* d_logits, void* stream);

/*
 * Gradients of the finalize (pmoe_finalize), for the FP32 sum before its rounding:
 *   d_topk_w[t,j]       = sum_h dout[t,h] * z[row(t,j),h]   in FP32, 0 where row(t,j) < 0
 *   d_z[row(t,j),:]     = bf16(w[t,j] * dout[t,:])
 *   dout : BF16 [T, H];  z, d_z : BF16 [R, H];  row_of_route : int32 [T*K], a value
 *   outside [0, R) is no route and no row is named twice (the routing names none
 *   twice; of a row named twice d_z holds one of the two);  topk_w, d_topk_w : float32 [T, K].
 * Either output may be NULL; z is needed for d_topk_w, topk_w for d_z. Rows of
 * d_z that no route names are left as they were. The outputs share no memory with each
 * other or with an input that the call reads. H must be a multiple of 8, at most 2^30.
 * Alignment: dout, z and d_z 16 bytes, others 4 bytes.
 */
int pmoe_finalize_backward(const void* dout, const void* z, const int32_t* row_of_route,
                           const float* topk_w, int T, int K, int H, int R,
                           float* d_topk_w, void* d_z, void* stream);

/* ============================================================ adapters
 *
 * Low-rank adapters of many requests beside one projection x [T, H] -> [T, N]
 * (with N = H: beside the whole routed layer). Token t uses adapter
 * a = adapter_ids[t]; ids outside [0, n) (-1, say) mean none. Tokens of one
 * adapter need not be neighbours.
 *   down : BF16 [n, R, H];  up : BF16 [n, N, R];  scale : float32 [n].
 * H and N multiples of 16 in [16, 16384], R a multiple of 8 in [8, 128] (an
 * adapter of a smaller rank has zeros in the rest), 1 <= n <= 65535, T <= 2^24;
 * T*H and T*N may pass 2^31. Alignment: ws 256 bytes, ids and scale their own
 * size, everything else 16 bytes. Outputs and ws share no memory with each other
 * or with an argument that the call reads, but out (dx) may be base itself. An
 * infinite entry of x, dy, down or up makes every result that it enters infinite
 * or NaN (FP32 factors enter products as sums of BF16 values, whose products with it
 * may cancel). Runs on the caller's stream alone.
 */

#define PMOE_ADAPTER_MAX 65535
#define PMOE_ADAPTER_MAX_TOKENS (1 << 24)

/* Device workspace of pmoe_adapter_forward (backward = 0) or
 * pmoe_adapter_backward (backward = 1), in bytes. 0 on bad arguments. */
size_t pmoe_adapter_workspace_bytes(int T, int n, int H, int N, int R, int backward);

/*
 *   v[t]   = down[a] x[t]                                (FP32; 0 without an adapter)
 *   out[t] = bf16(base[t] + scale[a] * up[a] v[t])       (base[t] without an adapter)
 *   x : BF16 [T, H];  base : BF16 [T, N] or NULL (zeros);  out : BF16 [T, N], may be
 *   base itself;  v : float32 [T, R] or NULL -- pmoe_adapter_backward wants it.
 * Products and sums are FP32; scale * v enters the second product with 16
 * significant bits. The bits of a token depend on that token, its adapter and
 * the shapes only, not on the other tokens of the call.
 */
int pmoe_adapter_forward(const void* x, const void* adapter_ids, int ids_type, int T, int n, int H, int N,
                         int R, const void* down, const void* up, const float* scale, const void* base,
                         void* out, float* v, void* ws, size_t ws_bytes, void* stream);

/*
 * Gradients for the gradient dy of out, du[t] = scale[a] * up[a]^T dy[t] in FP32:
 *   dx[t]     = bf16(base[t] + down[a]^T du[t])          (base[t] without an adapter)
 *   d_down[a] = sum of du[t] x[t]^T over the tokens of a      float32 [n, R, H]
 *   d_up[a]   = scale[a] * sum of dy[t] v[t]^T                float32 [n, N, R]
 *   dy : BF16 [T, N];  x, v as in the forward call;  base : BF16 [T, H], the gradient
 *   that dx adds to, or NULL (zeros);  dx : BF16 [T, H], may be base itself.
 * dx may be NULL (x has no gradient), or d_down and d_up both (the adapters are
 * not trained; x and v are then not read). down and up are read either way. d_down
 * and d_up are written whole, zeros for adapters without tokens, and their sums over
 * tokens are taken in a fixed order; an infinite v or du makes the entries that it
 * enters NaN. The gradient of base is dy itself.
 */
int pmoe_adapter_backward(const void* dy, const void* x, const float* v, const void* adapter_ids,
                          int ids_type, int T, int n, int H, int N, int R, const void* down,
                          const void* up, const float* scale, const void* base, void* dx,
                          float* d_down, float* d_up, void* ws, size_t ws_bytes, void* stream);

/* ============================================================ tokens sorted by expert
 *
 * The order that pmoe_routed_moe gives its routes inside its workspace, for
 * callers that run the experts' products themselves: the rows of an expert follow
 * ascending route index f = t*K + j. The way back with the weights applied is
 * pmoe_finalize, its gradient pmoe_finalize_backward.
 */

/* Device workspace of pmoe_permute_tokens (bytes). 0 on bad shapes. */
size_t pmoe_permute_workspace_bytes(int T, int K, int E);

/*
 *   topk_ids       : [T, K] int32 or int64 (ids_type); a route is valid iff
 *                    expert_offset <= id < expert_offset + E, others have no row
 *   x              : [T] rows of row_bytes bytes, of any type, or NULL: only the
 *                    order is wanted (rows is NULL too, row_bytes unused)
 *   rows           : [T*K] rows of row_bytes bytes out; row row_of_route[t*K+j] is token
 *                    t's. Rows behind the last valid one are left as they were
 *   row_of_route   : int32 [T*K] out, -1 where the route has no row
 *   route_of_row   : int32 [T*K] out, the valid rows; behind them left as it was
 *   expert_offsets : int32 [E+1] out, first row of each expert; [E] = valid rows
 * T = 0 writes zeros to expert_offsets. 1 <= E <= 1024, 1 <= K <= 32 (K > E where this
 * is a share of few experts), T*K < 2^30, row_bytes a positive multiple of 16, at most
 * 2^20. Outputs and ws share no memory with each other or with an input. Alignment: x
 * and rows 16 bytes, ws 256, int64 ids 8, others 4.
 */
int pmoe_permute_tokens(const void* topk_ids, int ids_type, int T, int K, int E, int expert_offset,
                        const void* x, int row_bytes, void* rows, int32_t* row_of_route,
                        int32_t* route_of_row, int32_t* expert_offsets, void* ws, size_t ws_bytes,
                        void* stream);

/* Element types of the entry points below. */
#define PMOE_BF16 0
#define PMOE_F32 1

/*
 * Gradient of the copy: dx[t] = sum over j of d_rows[row_of_route[t*K+j]], in FP32,
 * slot order, rounded once; +0 for a token without a row. A value of row_of_route
 * outside [0, R) is no row.
 *   d_rows : BF16 or FP32 (type) [R, H];  row_of_route : int32 [T*K];  dx : as d_rows,
 *   [T, H].  1 <= K <= 32, T*K < 2^30, H a multiple of 8 (FP32: 4), at most 2^18.
 * dx shares no memory with the inputs. Alignment: d_rows and dx 16 bytes.
 */
int pmoe_permute_tokens_backward(const void* d_rows, int type, const int32_t* row_of_route, int T, int K,
                                 int R, int H, void* dx, void* stream);

/* ============================================================ microscaled formats
 *
 * Blocks of 32 consecutive elements of a row share one power of two X, stored as
 * its exponent + 127 in a byte (E8M0, 255 = NaN); the conversion is that of the
 * OCP Microscaling Formats specification v1.0, section 6.3:
 *   X = 2^max(floor(log2(amax of the block)) - emax, -127),
 *   element = x / X rounded to nearest, ties to the even code, saturating;
 * emax is 2 and the largest element 6 for E2M1 (codes packed two per byte, element
 * 2i in the low nibble), 8 and 448 for E4M3. A block of zeros has byte 0; a
 * negative value that rounds to 0 keeps its sign. A block with an infinity or a NaN has
 * byte 255 and zero codes, and reads back as NaN. Rows are contiguous, their
 * length n a multiple of 32: codes [rows, n/2] (E4M3: [rows, n]), scales [rows, n/32].
 */
#define PMOE_MX_E2M1 0
#define PMOE_MX_E4M3 1

/* x BF16 or FP32 [rows, n] -> codes, scales. Codes and scales share no memory with
 * each other or x. rows >= 0, n a positive multiple of 32 up to 2^30, rows*n < 2^40.
 * Alignment: x and codes 16 bytes. */
int pmoe_mx_quantize(const void* x, int type, int format, long long rows, int n, void* codes, void* scales,
                     void* stream);

/* The values that codes and scales stand for, rounded once to BF16 or FP32 (exact but where
 * they exceed the type). Sizes and alignment as above; out shares no memory with the inputs. */
int pmoe_mx_dequantize(const void* codes, const void* scales, int format, long long rows, int n, int type,
                       void* out, void* stream);

/*
 * Grouped product of expert-sorted MXFP4 rows with MXFP4 matrices:
 *   out[r] = W[e] a[src(r)],  e the expert of row r:  expert_offsets[e] <= r < expert_offsets[e+1]
 * with src(r) = route_of_row[r] / topk (a holds tokens), or r without route_of_row
 * (a holds the rows). E = 1 is one plain product.
 *   a_codes, a_sf  : E2M1 codes and scales of [a_rows, Kd]; a_rows >= R without route_of_row
 *   route_of_row   : int32 [R] or NULL; a row whose source is outside [0, a_rows) gets zeros
 *   expert_offsets : int32 [E+1] on the device, ascending, within [0, R]; rows of no
 *                    expert (behind the last, say) are left as they were
 *   w_codes, w_sf  : E2M1 codes [E, N, Kd/2] and scales [E, N, Kd/32] (pmoe_mx_quantize of [E*N, Kd])
 *   out            : BF16 or FP32 (out_type) [R, N]
 * Products are exact, sums FP32; each output is one chain of sums whose order
 * depends on Kd alone, so that a row's bits do not depend on the other rows. A
 * block that reads as NaN makes every output that it enters NaN.
 * 1 <= E <= 1024, 0 <= R <= PMOE_MX_MAX_ROWS, N a multiple of 16 up to 32768, Kd a multiple of
 * 32 up to 16384, topk >= 1; with route_of_row a_rows * Kd < 2^32 - 512. out shares no memory
 * with an input. Alignment: codes and out 16 bytes, scales 4 where Kd is a multiple of 128, others 4.
 */
#define PMOE_MX_MAX_ROWS (1 << 23)
int pmoe_mx_grouped_gemm(const void* a_codes, const void* a_sf, int a_rows, const int32_t* route_of_row,
                         int topk, const int32_t* expert_offsets, int R, int E, const void* w_codes,
                         const void* w_sf, int N, int Kd, void* out, int out_type, void* stream);

/*
 * Gradient of the rows of that product, the quantization of the rows passed
 * through: dx[r] = W[e]^T dy[r], dy BF16 [R, N], dx BF16 [R, Kd], FP32 sums rounded once.
 * The matrices are multiplied as BF16, which holds every element at scales up to 252, the largest
 * that pmoe_mx_quantize gives; at scales 253 and 254 (of other origin), elements of 2^128 and
 * above count as infinite here.
 * Other arguments, limits and rows of no expert as above (for the tokens of a
 * gathered product: pmoe_permute_tokens_backward of dx).
 */
int pmoe_mx_grouped_gemm_backward(const void* dy, const int32_t* expert_offsets, int R, int E,
                                  const void* w_codes, const void* w_sf, int N, int Kd, void* dx,
                                  void* stream);

/*
 * The activation between two such products, with an 8-bit checkpoint of its input
 * for the backward pass.
 *   y         : BF16 [R, I] (act PMOE_ACT_RELU2: h = max(y, 0)^2) or [R, 2I], gate then up
 *               (PMOE_ACT_SWIGLU: h = silu(gate) * up; with swiglu_limit L > 0 on
 *               gate <= L and -L <= up <= L)
 *   row_count : int32 on the device, or NULL: only rows below it are read and written
 *               (expert_offsets + E, say)
 *   hq, h_sf  : E2M1 codes [R, I/2] and scales [R, I/32] of h. They are those of the exact h,
 *               not of its FP32 rounding; h beyond FP32's largest counts as infinite
 *   y8, y8_sf : E4M3 codes and scales of y, rows as y's, or both NULL: no checkpoint
 * swiglu_limit is 0 (none) or positive, 0 for squared ReLU. 0 <= R <= PMOE_MX_MAX_ROWS, I a
 * multiple of 32 up to 16384. Outputs share no memory with each other or an input.
 * Alignment: y, hq and y8 16 bytes, row_count 4.
 */
int pmoe_mx_activation(const void* y, int R, int I, int act, float swiglu_limit, const int32_t* row_count,
                       void* hq, void* h_sf, void* y8, void* y8_sf, void* stream);

/*
 * Gradient of y at the values that its checkpoint stands for, the quantization of
 * h passed through: dy from dh BF16 [R, I], in FP32, rounded to BF16 once (d gate starts
 * with dh * up, which is infinite past FP32's largest number). Where the clamp
 * cuts gate or up off, their gradient is 0 (at the limit itself, and of a NaN, it is not).
 */
int pmoe_mx_activation_backward(const void* dh, const void* y8, const void* y8_sf, int R, int I, int act,
                                float swiglu_limit, const int32_t* row_count, void* dy, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PMOE_H_ */
