/*
 * fp4.h -- C ABI of the MI355X (gfx950) block-scaled FP4 library (libfp4.so).
 *
 * Formats.  An FP4 element is E2M1: one sign bit, two exponent bits and one
 * mantissa bit, whose non-negative values are exactly {0, 0.5, 1, 1.5, 2, 3, 4, 6}
 * ("DeepSeek-V4.1-Flash-NVFP4" explainer, section 2, NVFP4 format breakdown).
 *   MXFP4: blocks of 32 consecutive elements along K share one UE8M0 scale byte
 *          b meaning 2^(b-127) (same explainer, section 3, and the "DeepSeek-V4"
 *          architecture article, section 6.3, 1x32 tiles).
 *   NVFP4: groups of 16 consecutive elements along K share one E4M3 (OCP FP8
 *          E4M3FN) scale byte, and the whole tensor shares one fp32 scale s_t
 *          (explainer section 2: group_size 16 plus a tensor-level scale).
 *
 * Memory layout (all tensors row-major, K contiguous, no padding):
 *   codes   uint8 [rows, k/2]: byte j holds element 2j in bits 3:0 and element
 *           2j+1 in bits 7:4; a code is sign*8 + index into the value table.
 *   MX      scales uint8 [rows, k/32] (UE8M0).
 *   NV      scales uint8 [rows, k/16] (E4M3FN), plus one fp32 tensor scale in
 *           device memory.
 *   bf16 inputs/outputs are IEEE bfloat16 bit patterns with a leading dimension
 *   in elements (ld_x, ldc, ld_out >= k or n).
 *
 * Conventions shared by every entry point:
 *   - Pointers are device pointers owned by the caller; the library never
 *     allocates, frees or keeps them.  Every pointer must be 16-byte aligned and
 *     every leading dimension a multiple of 8 elements, else FP4_ERR_ALIGN.
 *   - All work is enqueued on `stream` (a hipStream_t; NULL = the default
 *     stream) and is asynchronous: the return value reports argument and
 *     launch errors only.  Data-dependent results (the remap's inexact count,
 *     computed tensor scales) are written to device memory.
 *   - Arguments are validated before any HIP call; a failing call enqueues
 *     nothing and returns a negative fp4_status.  fp4_last_error() gives the
 *     message of the last failure on the calling thread.
 *   - Zero-sized problems return FP4_OK and enqueue nothing.
 *   - Calls that overlap in time may not share output or workspace buffers.
 */
#ifndef FP4_H
#define FP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP4_OK = 0,
    FP4_ERR_INVALID = -1,      /* null pointer, bad enum, negative size        */
    FP4_ERR_SHAPE = -2,        /* k not a multiple of the block/group size ... */
    FP4_ERR_ALIGN = -3,        /* pointer not 16-B aligned, ld not multiple of 8 */
    FP4_ERR_UNSUPPORTED = -4,  /* no kernel for this combination               */
    FP4_ERR_WORKSPACE = -5,    /* workspace null or smaller than required      */
    FP4_ERR_HIP = -6           /* a HIP runtime call failed                    */
} fp4_status;

typedef enum { FP4_FMT_MX = 0, FP4_FMT_NV = 1 } fp4_format;
typedef enum { FP4_DT_BF16 = 0, FP4_DT_F32 = 1 } fp4_dtype;

/* Version of this ABI (incremented on any incompatible change). */
int fp4_abi_version(void);

/* Static text for a status code. */
const char* fp4_status_string(int status);

/* Message of the last failed call on the calling thread ("" if none). */
const char* fp4_last_error(void);

/*
 * MXFP4 quantization ("DeepSeek-V4.1-Flash-NVFP4" explainer, section 3: one
 * UE8M0 scale per 32 elements; "DeepSeek-V4" article, section 6.3).
 * For each row and each block of 32 elements along k:
 *   amax = max|x|; E = floor(log2 amax) - 2 (E = -127 when amax = 0), clamped to
 *   [-127, 127]; scales = E + 127; code = round-to-nearest-even of x * 2^-E onto
 *   the E2M1 values, saturating at 6, keeping the sign bit of x (so -0.0 gives 0x8).
 * x_bf16: [rows, ld_x] bf16; codes: [rows, k/2]; scales: [rows, k/32].
 * Errors: k % 32 != 0 -> FP4_ERR_SHAPE.  Inputs must be finite.
 */
int fp4_quantize_mx(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                    uint8_t* codes, uint8_t* scales, void* stream);

/*
 * NVFP4 quantization (explainer, section 2: groups of 16 with a per-group scale
 * bringing the group into [-6, 6] and a tensor-level scale; section 4: activation
 * scales are calibrated).
 *   s_t = fp32(amax_tensor / (6 * 448)) unless tensor_scale_is_input != 0, in
 *   which case *tensor_scale (device fp32) is read as the calibrated s_t;
 *   per group: s_g = E4M3 round-to-nearest-even of amax_g / (6 s_t), saturating
 *   at 448; code = E2M1 round-to-nearest-even of x / (s_g s_t), saturating at 6.
 *   Each step is a single correct rounding of the exact real quotient.  When
 *   s_t = 0 or s_g = 0 the group's codes are signed zeros and s_g = 0.
 * codes: [rows, k/2]; scales: [rows, k/16]; tensor_scale: one device float,
 * written when computed.  workspace: device memory of at least
 * fp4_quantize_nv_workspace_bytes() bytes (used for the tensor amax).
 * Errors: k % 16 != 0 -> FP4_ERR_SHAPE; workspace too small -> FP4_ERR_WORKSPACE.
 */
int fp4_quantize_nv(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                    uint8_t* codes, uint8_t* scales, float* tensor_scale,
                    int tensor_scale_is_input,
                    void* workspace, size_t workspace_bytes, void* stream);
size_t fp4_quantize_nv_workspace_bytes(int64_t rows, int64_t k);

/*
 * fp4_quantize_nv for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same operation, arguments and results as fp4_quantize_nv without the
 * workspace.  The tensor-amax partial maxima go to a static device array of
 * the library (4 KiB per GPU, held until the process ends); the call allocates
 * nothing.  Every call on a GPU shares that GPU's array, so calls that overlap
 * in time on one GPU (different streams or threads) race and must be ordered
 * by the caller.  The array's size covers every shape; FP4_ERR_WORKSPACE
 * reports a library built with a smaller one.  A HIP error in looking up the
 * array's address on the current device returns FP4_ERR_HIP.
 * Errors: as fp4_quantize_nv.
 */
int fp4_quantize_nv_noalloc(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                            uint8_t* codes, uint8_t* scales, float* tensor_scale,
                            int tensor_scale_is_input, void* stream);

/*
 * Lossless MXFP4 -> NVFP4 scale remap (explainer, section 1: NVFP4's finer
 * 16-element scale layout can re-express MXFP4 weights block by block without
 * loss; section 6: the conversion script's E2M1 -> E4M3 remap).
 * Codes are reused unchanged (the NVFP4 tensor is (codes, scales_e4m3, s_t)).
 *   E_max = max over blocks of (scale byte - 127); k = E_max - 8;
 *   *tensor_scale = 2^k; both 16-groups of a block with exponent E_b get the
 *   E4M3 value nearest 2^(E_b - k) (exact for E_b - k in [-9, 8]).
 *   *n_inexact_blocks = number of blocks with a nonzero code whose 2^(E_b - k)
 *   is below 2^-9 (those lose precision); 0 means the remap is lossless.
 * codes: [rows, k/2]; scales_e8m0: [rows, k/32]; scales_e4m3: [rows, k/16];
 * tensor_scale: 1 device float; n_inexact_blocks: 1 device int32.
 * workspace: optional device memory of at least
 * fp4_scale_max_workspace_bytes(rows, k) bytes (any alignment, not overlapping
 * the other arguments) for the partial maxima of E_max; the call then takes two
 * kernel launches instead of three.  NULL (with workspace_bytes 0) keeps the
 * maxima in the output array's first bytes until a third launch rewrites them.
 * Results are the same either way.  Calls sharing one workspace must be ordered
 * (one stream).
 * Errors: k % 32 != 0 -> FP4_ERR_SHAPE; workspace too small, or NULL with
 * workspace_bytes != 0 -> FP4_ERR_WORKSPACE.
 */
int fp4_remap_mx_to_nv(const uint8_t* codes, const uint8_t* scales_e8m0,
                       int64_t rows, int64_t k, uint8_t* scales_e4m3,
                       float* tensor_scale, int32_t* n_inexact_blocks,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of the optional workspace of fp4_remap_mx_to_nv and fp4_mx_dequant_fp8
 * for an MX tensor of rows x k (at most 256; 0 for an empty tensor).
 */
size_t fp4_scale_max_workspace_bytes(int64_t rows, int64_t k);

/*
 * Dequantization (explainer, section 2: the block scales multiply back in;
 * "DeepSeek-V4 FP4 QAT" article, section 4.2: FP4 data times the scale).
 *   MX: value = (-1)^s * MAG[i] * 2^(b-127), exact in fp32 and bf16.
 *   NV: fp32 value = round-to-nearest-even(MAG[i] * s_g * s_t); bf16 output is
 *       the bf16 rounding of that fp32 value.
 * out: [rows, ld_out] of out_dtype.  tensor_scale: device float (NV only).
 * Errors: k % 32 (MX) or k % 16 (NV) != 0 -> FP4_ERR_SHAPE.
 */
int fp4_dequant(fp4_format fmt, const uint8_t* codes, const uint8_t* scales,
                const float* tensor_scale, int64_t rows, int64_t k,
                void* out, fp4_dtype out_dtype, int64_t ld_out, void* stream);

/*
 * W4A4 GEMM: C[m, n] = sum_k A_hat[m, k] * B_hat[n, k] with fp32 accumulation
 * (explainer, section 2: activations and weights both 4-bit block-scaled, the
 * accumulator rescaled per block).  A_hat, B_hat are the exact dequantized
 * operands; B is given [n, k] (the nn.Linear weight layout), so C = A . B^T.
 *   MX: scaled MFMA with the UE8M0 block scales applied by the matrix core.
 *   NV: operands expanded exactly to a 16-bit float (code * s_g has at most 6
 *       significant bits: fp16 in the tiled kernels, bf16 in the fallback) and
 *       multiplied on the 16-bit MFMA; the product is scaled by
 *       (*a_tensor_scale) * (*b_tensor_scale).
 * c: [m, ldc] of c_dtype.  Tensor scales are device floats (NV only, else NULL).
 * Errors: k % 32 (MX) or k % 16 (NV) != 0 -> FP4_ERR_SHAPE.
 */
int fp4_gemm(fp4_format fmt,
             const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
             const uint8_t* b_codes, const uint8_t* b_scales, const float* b_tensor_scale,
             int64_t m, int64_t n, int64_t k,
             void* c, fp4_dtype c_dtype, int64_t ldc, void* stream);

/*
 * MXFP4 KV-cache append ("DeepSeek-V4 FP4 QAT" article, section 3.3: the KV
 * cache is kept in MXFP4 and each new token's vector is quantized as it joins
 * the cache; the FP4 QK scores of the attention indexer are then fp4_gemm of
 * the MXFP4 queries against the cache rows, the "DeepSeek-V4" architecture
 * article, section 3, lightning indexer).  Each cache row is one token's vector
 * of d values in the MXFP4 layout above (32-element blocks along d, each with
 * its own UE8M0 byte), so a row's scales never depend on other tokens.
 *   For t in [0, tokens): if 0 <= slots[t] < capacity, row t of x is quantized
 *   exactly as fp4_quantize_mx does and written to cache row slots[t]; tokens
 *   whose slot is outside that range (padding) are skipped.  The in-range slots
 *   must be distinct.
 * x_bf16: [tokens, ld_x] bf16; slots: int32 [tokens] (device); cache_codes:
 * [capacity, d/2]; cache_scales: [capacity, d/32].
 * Errors: d % 32 != 0 -> FP4_ERR_SHAPE.  Inputs must be finite.
 */
int fp4_kv_append_mx(const void* x_bf16, int64_t tokens, int64_t d, int64_t ld_x, const int32_t* slots,
                     uint8_t* cache_codes, uint8_t* cache_scales, int64_t capacity, void* stream);

/*
 * Fake quantization for quantization-aware training ("DeepSeek-V4 FP4 QAT"
 * article, section 2.2: quantize-dequantize nodes on the expert weights in the
 * training forward pass): out = dequant(quantize(x)) in one pass over x, equal
 * element for element to fp4_quantize_mx / fp4_quantize_nv followed by
 * fp4_dequant (same rounding rules, same tensor-scale handling), with no codes
 * or scales materialized.
 *   NV: as fp4_quantize_nv, s_t is computed (and written to *tensor_scale; the
 *   workspace is then required) unless tensor_scale_is_input != 0.  MX:
 *   tensor_scale and the workspace are ignored (may be NULL).
 * x_bf16: [rows, ld_x] bf16; out: [rows, ld_out] of out_dtype.  out may be x
 * itself (in place: same pointer, ld_out == ld_x, bf16 output); any other
 * overlap of x and out is FP4_ERR_INVALID.
 * Errors: k % 32 (MX) or k % 16 (NV) != 0 -> FP4_ERR_SHAPE; NV workspace too
 * small -> FP4_ERR_WORKSPACE.  Inputs must be finite.
 */
int fp4_fake_quant(fp4_format fmt, const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                   void* out, fp4_dtype out_dtype, int64_t ld_out,
                   float* tensor_scale, int tensor_scale_is_input,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Straight-through-estimator backward of the fake-quant node ("DeepSeek-V4"
 * architecture article, section 6.3: the gradient of the quantized weight is
 * handed unchanged to the fp32 master weight):
 *   grad_master[r, c] = (accumulate ? grad_master[r, c] : 0) + grad[r, c],
 * one fp32 addition (round to nearest even) per element.
 * grad: [rows, ld_grad] of grad_dtype (bf16 or fp32); grad_master: fp32
 * [rows, ld_master].  Errors: k % 8 != 0 -> FP4_ERR_SHAPE.
 */
int fp4_ste_backward(const void* grad, fp4_dtype grad_dtype, int64_t rows, int64_t k, int64_t ld_grad,
                     float* grad_master, int64_t ld_master, int accumulate, void* stream);

/*
 * W4A8: FP4 weights with FP8 activations ("DeepSeek-V4 FP4 QAT" article,
 * section 4.3: the recommended deployment pairing; section 4.2: FP4 expands into
 * FP8 without loss).  Activations use MXFP8: E4M3 elements (OCP FP8 E4M3FN,
 * largest value 448) with one UE8M0 scale per 32 elements along k, the same
 * block structure as the MXFP4 weights ("DeepSeek-V4" article, section 6.3;
 * explainer section 3).
 *
 * fp4_quantize_mxfp8: per row and 32-element block, amax = max|x|;
 *   E = floor(log2 amax) - 8 (8 = E4M3's largest exponent; E = -127 when
 *   amax = 0), clamped to [-127, 127]; scales = E + 127; code byte = E4M3
 *   round-to-nearest-even of |x| * 2^-E, saturating at 448 (0x7E), with the
 *   sign bit of x in bit 7 (so -0.0 gives 0x80).
 *   x_bf16: [rows, ld_x] bf16; codes8: [rows, k] bytes; scales: [rows, k/32].
 *   Errors: k % 32 != 0 -> FP4_ERR_SHAPE.  Inputs must be finite.
 */
int fp4_quantize_mxfp8(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                       uint8_t* codes8, uint8_t* scales, void* stream);

/*
 * Lossless MXFP4 -> MXFP8 re-encoding (QAT article, section 4.2; explainer,
 * section 6: E2M1 values are E4M3 values): every E2M1 code becomes the E4M3
 * byte of the same value (sign kept, -0 -> 0x80); the UE8M0 scales are
 * unchanged, so the caller pairs codes8 with the MXFP4 tensor's own scales.
 * codes: [rows, k/2] packed E2M1; codes8: [rows, k] bytes.
 * Errors: k % 32 != 0 -> FP4_ERR_SHAPE.
 */
int fp4_mx_to_mxfp8(const uint8_t* codes, int64_t rows, int64_t k, uint8_t* codes8, void* stream);

/*
 * MXFP4 -> FP8 dequantization through E4M3 block scales ("DeepSeek-V4 FP4 QAT"
 * article, section 4.2: the scale array is re-encoded in E4M3, the 4-bit codes
 * are widened to FP8 and the FP8 scale multiplies the FP8 data; "DeepSeek-V4"
 * architecture article, section 6.3: lossless while the block scale ratio stays
 * under a threshold).  E4M3 spans only 2^-9 .. 448, so the tensor carries one
 * fp32 power of two in front:
 *   E_max = max over blocks of (scale byte - 127); k = E_max - 6;
 *   *tensor_scale = 2^k;  for block b, j = E_b - k (<= 6):
 *   block_scales_e4m3[b] = E4M3 round-to-nearest-even of 2^j (exact for j >= -9;
 *     2^-10 ties to 0);
 *   values_e4m3[r, c] = E4M3 round-to-nearest-even of MAG(code) * block scale,
 *     with the code's sign bit in bit 7 (the largest value is 6 * 2^6 = 384, so
 *     nothing saturates); the dequantized element is that value * 2^k.
 *   *n_inexact_blocks = number of blocks holding an element whose value * 2^k
 *     differs from its MX value.  It is 0 whenever every block exponent is at
 *     least E_max - 14 (a largest-to-smallest block scale ratio of at most 2^14).
 * codes: [rows, k/2]; scales_e8m0: [rows, k/32]; values_e4m3: [rows, k] bytes;
 * block_scales_e4m3: [rows, k/32] or NULL (not written); tensor_scale: 1 device
 * float; n_inexact_blocks: 1 device int32 (cleared, then accumulated, while the
 * call runs).  workspace / workspace_bytes: optional, as for fp4_remap_mx_to_nv
 * (two launches with it, three without; the same results).
 * Errors: k % 32 != 0 -> FP4_ERR_SHAPE; workspace too small, or NULL with
 * workspace_bytes != 0 -> FP4_ERR_WORKSPACE.
 */
int fp4_mx_dequant_fp8(const uint8_t* codes, const uint8_t* scales_e8m0, int64_t rows, int64_t k,
                       uint8_t* values_e4m3, uint8_t* block_scales_e4m3, float* tensor_scale,
                       int32_t* n_inexact_blocks, void* workspace, size_t workspace_bytes, void* stream);

/*
 * W4A8 GEMM: C[m, n] = sum_k A_hat[m, k] * B_hat[n, k] with fp32 accumulation,
 * A_hat the MXFP8 activations (a_codes8 [m, k] E4M3 bytes, a_scales [m, k/32])
 * and B_hat the MXFP4 weights (b_codes [n, k/2], b_scales [n, k/32]), both
 * exactly dequantized.  Mixed-format scaled MFMA (E4M3 x E2M1) with the UE8M0
 * block scales applied by the matrix core.
 * c: [m, ldc] of c_dtype.  Errors: k % 32 != 0 -> FP4_ERR_SHAPE.
 */
int fp4_gemm_w4a8(const uint8_t* a_codes8, const uint8_t* a_scales,
                  const uint8_t* b_codes, const uint8_t* b_scales,
                  int64_t m, int64_t n, int64_t k,
                  void* c, fp4_dtype c_dtype, int64_t ldc, void* stream);

/*
 * Optional intermediate outputs of fp4_moe_grouped_gemm, for staged testing.
 * Every member may be NULL.  Slot s = t * topk + j (token t, choice j).
 *   x_codes   uint8 [tokens, hidden/2], x_scales [tokens, hidden/32|16]  Q(x)
 *   counts    int32 [num_experts]    slots routed to each expert
 *   offsets   int32 [num_experts+1]  exclusive prefix sum of counts
 *   perm      int32 [tokens*topk]    slots grouped by expert, stable
 *   gate_up   fp32  [tokens*topk, 2*inter]  g (first inter) then u, per slot
 *   h_bf16    bf16  [tokens*topk, inter]    SiLU(g)*u rounded to bf16
 *   h_codes   uint8 [tokens*topk, inter/2], h_scales [tokens*topk, inter/32|16]
 *   y         fp32  [tokens*topk, hidden]   down-projection output per slot
 * Stage inputs, for testing each fused stage on given data (NULL = compute):
 *   gate_up_in   fp32 [tokens*topk, 2*inter]: g (first inter) then u per slot,
 *                already including NV tensor scales; replaces the gate/up
 *                product, and SiLU*mul, the bf16 rounding and the quantization
 *                of h run on these values.
 *   h_codes_in, h_scales_in  [tokens*topk, inter/2], [tokens*topk, inter/32|16]:
 *                quantized h per slot (NV: with s_t = act_tensor_scales[1]);
 *                replaces the computed Q(h) as the input of the down stage.
 * Stage timing: stage_events[i], when not NULL, is a hipEvent_t recorded on
 * the call's stream at stage boundary i: 0 entry, 1 after Q(x), 2 after the
 * routing metadata, 3 after gate/up (with SiLU*mul and Q(h)), 4 after down,
 * 5 after the combine.
 */
typedef struct fp4_moe_debug {
    uint8_t* x_codes;
    uint8_t* x_scales;
    int32_t* counts;
    int32_t* offsets;
    int32_t* perm;
    float* gate_up;
    void* h_bf16;
    uint8_t* h_codes;
    uint8_t* h_scales;
    float* y;
    const float* gate_up_in;
    const uint8_t* h_codes_in;
    const uint8_t* h_scales_in;
    void* stage_events[6];
} fp4_moe_debug;

/*
 * Routed-expert MoE layer on block-scaled FP4 weights and activations
 * (explainer, section 3: the routed experts' w1/w2/w3 are the quantized
 * layers; "DeepSeek-V4" article, section 2: 384 routed experts, 6 active;
 * section 6.1: dispatch to experts and combine back).  For each token t and
 * choice j with e = topk_ids[t, j]:
 *   x_hat = dequant(quant(x[t]))  (MX; or NV with s_t = act_tensor_scales[0])
 *   g = x_hat . w1[e]^T, u = x_hat . w3[e]^T   (w13[e] rows 0..inter-1 are w1,
 *                                               rows inter..2*inter-1 are w3)
 *   h = bf16(SiLU(g) * u); h_hat = dequant(quant(h)) (NV: s_t = act_tensor_scales[1])
 *   y = h_hat . w2[e]^T;  out[t] = bf16(sum_j topk_weights[t, j] * y)
 * x_bf16 [tokens, hidden]; topk_ids int32 [tokens, topk] in [0, num_experts);
 * topk_weights fp32 [tokens, topk];
 * w13_codes [E, 2*inter, hidden/2], w13_scales [E, 2*inter, hidden/32|16];
 * w2_codes [E, hidden, inter/2], w2_scales [E, hidden, inter/32|16];
 * NV: w13_tensor_scales, w2_tensor_scales fp32 [E] and act_tensor_scales fp32 [2]
 * (device); MX: all three NULL.  out_bf16 [tokens, hidden].
 * workspace: at least fp4_moe_workspace_bytes(...) bytes of device memory.
 * Errors: hidden or inter not a multiple of 128, or tokens*topk above about
 * 4.1 million -> FP4_ERR_SHAPE; topk outside [1, 16] or num_experts outside
 * [1, 1024] -> FP4_ERR_INVALID; workspace too small -> FP4_ERR_WORKSPACE.
 * A slot whose expert id lies outside [0, num_experts) is routed nowhere and
 * contributes nothing to out.  The combine sums each token's weighted rows in
 * fp32 in order j = 0 .. topk-1 without atomics, so out is deterministic.
 */
int fp4_moe_grouped_gemm(fp4_format fmt, const void* x_bf16, int64_t tokens, int64_t hidden,
                         const int32_t* topk_ids, const float* topk_weights, int topk,
                         int num_experts, int64_t inter,
                         const uint8_t* w13_codes, const uint8_t* w13_scales,
                         const float* w13_tensor_scales,
                         const uint8_t* w2_codes, const uint8_t* w2_scales,
                         const float* w2_tensor_scales,
                         const float* act_tensor_scales,
                         void* out_bf16, void* workspace, size_t workspace_bytes,
                         const fp4_moe_debug* dbg, void* stream);
size_t fp4_moe_workspace_bytes(fp4_format fmt, int64_t tokens, int64_t hidden, int topk,
                               int num_experts, int64_t inter);

/*
 * Attention beside the MXFP4 cache.  The entry points below take a prompt or a
 * step of (drafted) tokens from its projections to its attention: head norms
 * and rotation, attention over the prompt itself, the pages of the cache that
 * fp4_kv_append_mx fills, and attention of drafted tokens over that cache
 * ("DeepSeek-V4 FP4 QAT" article, section 3.3: the KV cache is kept in MXFP4
 * and dequantized where attention reads it).
 *
 * Head layout: a token's heads lie one after another, head h of token t at
 * t * ld + h * head_dim elements, so q, k and v may be columns of one fused
 * projection.  Grouped heads: query head h attends with key/value head
 * h / (q_heads / kv_heads); q_heads is a multiple of kv_heads.
 */

/*
 * Root-mean-square norm of every query and key head and the rotation by the
 * token's position, in one pass:
 *   y = x * rsqrt(mean(x^2) + eps) * weight   (over head_dim, fp32)
 *   the first rot_dim values in pairs (a, b), pair i turned by the position's
 *   angle i: (a cos - b sin, b cos + a sin); pairs are (i, i + rot_dim/2), or
 *   (2i, 2i + 1) with interleaved != 0; the rest unturned; one rounding to bf16.
 * cos_sin: fp32 [max_positions, rot_dim], cos of the rot_dim/2 angles, then sin
 * (a table keeps far positions exact); positions: int32 [tokens].  A token whose
 * position lies outside [0, max_positions) is padding: its output rows are left
 * as they were.  rot_dim 0: norms only, cos_sin and positions ignored (may be NULL).
 * q_weight, k_weight: [head_dim] of weight_dtype, NULL = ones.
 * q [tokens, ld_q], k [tokens, ld_k], q_out [tokens, ld_qo], k_out [tokens,
 * ld_ko]: bf16.  Either output may be its own input (same pointer and leading
 * dimension); any other overlap of an output with an input (weights, cos_sin and
 * positions too) or the other output is FP4_ERR_INVALID.  q_heads or kv_heads may be 0 (its pointers are then
 * ignored).  The squares are summed in fp32: a head whose sum passes 3e38 (values
 * of 1e18 on) or whose values are no numbers comes out as the formula does there, and
 * with an eps below 1e-36 so does one whose squares lose bits below 1e-38 (values
 * under 1e-18).
 * Errors: head_dim not a multiple of 16 in [16, 256], rot_dim not a multiple of
 * 16 in [0, head_dim], 2^24 tokens or more -> FP4_ERR_SHAPE; eps negative or not finite -> FP4_ERR_INVALID.
 */
int fp4_qk_norm_rope(const void* q, const void* k, int64_t tokens, int q_heads, int kv_heads, int head_dim,
                     int64_t ld_q, int64_t ld_k, const void* q_weight, const void* k_weight,
                     fp4_dtype weight_dtype, float eps, const float* cos_sin, int64_t max_positions, int rot_dim,
                     int interleaved, const int32_t* positions, void* q_out, int64_t ld_qo, void* k_out,
                     int64_t ld_ko, void* stream);

/*
 * A paged MXFP4 cache of keys and values in fp4_kv_append_mx's layout: row
 * page * page_size + i is token i of a page, d = kv_heads * head_dim values to
 * a row: codes [num_pages * page_size, d/2], scales [.., d/32].  v_codes and
 * v_scales may both be NULL (a keys-only cache) where no attention reads it.
 * page_size is a multiple of 16 (so every page starts 16-byte aligned), d of 32,
 * and num_pages * page_size is below 2^31 (rows are int32 slots).
 */
typedef struct fp4_kv_cache {
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
    int64_t num_pages;
    int64_t d;
    int64_t page_size;
} fp4_kv_cache;

/*
 * The step from a layer's projections to its cache in one pass: the rotation of
 * fp4_qk_norm_rope on queries and keys, with its head norms where norm != 0 and
 * without any otherwise, and fp4_kv_append_mx of the keys and values to a cache:
 *   q_out[t] = bf16(R(position) n(q[t])),
 *   row slots[t] of the keys = MXFP4(bf16(R(position) n(k[t]))), of the values = MXFP4(v[t]),
 * n the norm or nothing.  With norm != 0 every byte is what fp4_qk_norm_rope and
 * two fp4_kv_append_mx give.  Arguments are as there; without norm, q_weight and
 * k_weight must be NULL and eps is ignored.
 * A token whose position lies outside [0, max_positions) is padding: nothing of it is
 * written.  One whose slot lies outside the cache is not appended, its query row is
 * written.  Slots in range must be distinct.  rot_dim 0: nothing turns, cos_sin and
 * positions ignored (may be NULL).  q_heads may be 0 (q and q_out ignored); a cache
 * without values takes the keys alone (v ignored).  Inputs must be finite.
 * q_out may be q itself (same pointer and leading dimension); any other overlap of
 * q_out or the cache with an input or with one another is FP4_ERR_INVALID.
 * Errors: head_dim not a multiple of 32 in [32, 256], rot_dim not a multiple of 16 in
 * [0, head_dim], cache->d != kv_heads * head_dim, 2^24 tokens or more -> FP4_ERR_SHAPE;
 * eps negative or not finite, weights without norm, kv_heads < 1 -> FP4_ERR_INVALID.
 */
int fp4_kv_append_rope_mx(const void* q, const void* k, const void* v, int64_t tokens, int q_heads, int kv_heads,
                          int head_dim, int64_t ld_q, int64_t ld_k, int64_t ld_v, int norm, const void* q_weight,
                          const void* k_weight, fp4_dtype weight_dtype, float eps, const float* cos_sin,
                          int64_t max_positions, int rot_dim, int interleaved, const int32_t* positions, void* q_out,
                          int64_t ld_qo, const fp4_kv_cache* cache, const int32_t* slots, void* stream);

/*
 * Which pages the sequences of a batch hold (all device memory):
 *   page_table  int32 [batch, max_pages]  page of tokens i*page_size.., -1 = none
 *   page_counts int32 [batch]             entries of the row in use
 *   seq_lens    int32 [batch]             tokens committed to the cache
 *   page_refs   int32 [num_pages]         holders of each page; 0 = free
 * Pages may be shared between sequences (after fp4_kv_fork) up to a sequence's
 * committed length; a sequence writes only rows that fp4_kv_reserve gave it.
 * Page ids outside [0, num_pages), counts outside [0, max_pages] and sequence
 * ids outside [0, batch) are never followed.  Calls on one state are ordered by
 * the caller (one stream).  batch and the lists of ids are shorter than 2^20.
 *
 * One state belongs to one cache: fp4_kv_reserve copies a shared page's rows, and
 * fp4_kv_compact moves accepted rows, in the cache they are given and update the
 * state for it, so a second cache called with the same state would miss both.  A
 * model with a cache for each layer keeps a state for each layer.  What the calls do
 * to a state follows from the state and their arguments alone, so layers that take
 * the same calls have the same tables, lengths and slots at every step.
 */
typedef struct fp4_kv_pages {
    int32_t* page_table;
    int32_t* page_counts;
    int32_t* seq_lens;
    int32_t* page_refs;
    int64_t batch;
    int64_t max_pages;
    int64_t num_pages;
} fp4_kv_pages;

/*
 * Makes room for new_tokens[b] (int32 [batch], negative = 0) more tokens behind
 * the committed ones of every sequence: pages are taken free ones first by
 * index, for the sequences in order, so the result does not depend on timing.
 * A partly filled last page that other sequences hold too is copied first (its
 * committed rows) and the copy takes its place: copy on write.  A reservation starts
 * a step anew: tokens of an earlier one that are not committed yet are to be appended
 * again, to the new slots (where a fork came between, the copy does not have them).
 *   slots: int32 [batch, max_new], the cache row of new token j of sequence b
 *   (position seq_lens[b] + j) for j < new_tokens[b], else -1: the slots of
 *   fp4_kv_append_mx.  May be NULL with max_new 0.
 *   *n_short: int32, 0, or how many pages the pool or the table rows lack; then
 *   nothing is reserved for any sequence and every slot is -1: the new tokens have no
 *   rows, so attention over them and a commit of them have no meaning.
 * workspace: fp4_kv_reserve_workspace_bytes(batch, num_pages) bytes; calls (and
 * replays) that share one are ordered by the caller.
 */
int fp4_kv_reserve(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* new_tokens, int32_t* slots,
                   int64_t max_new, int32_t* n_short, void* workspace, size_t workspace_bytes, void* stream);
size_t fp4_kv_reserve_workspace_bytes(int64_t batch, int64_t num_pages);

/*
 * Forks sequences: for each pair (source, target) of pairs (int32 [n, 2]) the
 * target holds the source's committed tokens, sharing their pages; no row is
 * copied until one of the holders writes (fp4_kv_reserve).  A pair is skipped
 * when an id is outside [0, batch), the target still holds pages, an earlier
 * pair names the same target, or the source is a target of this call.  Drafted
 * tokens that the source has not committed are not shared; it may commit them
 * afterwards, before its next reservation.
 */
int fp4_kv_fork(const fp4_kv_pages* pages, const int32_t* pairs, int64_t n, int64_t page_size, void* stream);

/*
 * Cuts each listed sequence (int32 [n]) back to its first min(keep_lens[i],
 * seq_lens) tokens (keep_lens int32 [n]; NULL = 0: the whole sequence) and lets
 * go of every page behind them, reserved ones included.  A page that nobody
 * holds any more is free.  Ids outside [0, batch) are skipped; of an id listed
 * twice the first entry counts.
 */
int fp4_kv_free(const fp4_kv_pages* pages, const int32_t* seqs, int64_t n, const int32_t* keep_lens,
                int64_t page_size, void* stream);

/*
 * Commits drafted tokens: for every sequence b the rows of its drafted tokens
 * accepted[b, 0 .. accepted_lens[b]) (indices behind the committed length, in
 * any order; reads come before writes, so rows may cross) move to the positions
 * seq_lens[b], seq_lens[b] + 1, ..., and seq_lens[b] grows by that many.
 * accepted: int32 [batch, max_accepted], max_accepted <= 64; accepted_lens:
 * int32 [batch], taken as within [0, max_accepted].  accepted NULL: the first
 * accepted_lens[b] reserved tokens are committed where they are (max_accepted
 * ignored; the end of a prompt's append).  Rows move between pages that the
 * sequence holds, onto rows that no other sequence sees (fp4_kv_reserve saw to
 * that, and a fork since then shares committed rows only), and the length never
 * passes its pages; an accepted index that points elsewhere moves nothing.  Of two
 * sequences that hold one partly filled page, at most one can have reserved rows on
 * it: if accepted_lens names both, rows on that page stay as they are.
 * accepted_lens has to be 0 for a sequence whose reservation gave it no rows, and
 * for all of them where *n_short was not 0: the unused rest of a last page cannot be
 * told from reserved rows, and would be committed as it is.  fp4_kv_compact_reserved
 * sees to that by itself.
 */
int fp4_kv_compact(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* accepted,
                   int64_t max_accepted, const int32_t* accepted_lens, void* stream);
/*
 * The same for the rows of one reservation, whose outcome it follows on the device:
 * slots (int32 [batch, max_new], as that fp4_kv_reserve wrote them, not NULL).
 * A sequence commits its tokens up to the first whose slot is not the row of its
 * position, and an accepted index without such a slot moves nothing.  So nothing is
 * committed for a sequence that the reservation gave no rows, for any sequence
 * where it was refused, or from slots that have been committed before (while the
 * sequence has not been cut back since).
 */
int fp4_kv_compact_reserved(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* accepted,
                            int64_t max_accepted, const int32_t* accepted_lens, const int32_t* slots,
                            int64_t max_new, void* stream);

/*
 * Copies whole pages: for i in [0, n), page src_pages[i] of src to page
 * dst_pages[i] of dst (the same d and page_size; both with values or both
 * without).  Pairs with an id outside its cache are skipped.  The in-range
 * destinations must be distinct, and within one cache no page may be source and
 * destination of the same call.
 */
int fp4_kv_copy_pages(const fp4_kv_cache* src, const fp4_kv_cache* dst, const int32_t* src_pages,
                      const int32_t* dst_pages, int64_t n, void* stream);

/*
 * Attention of drafted tokens over the cache (speculative decoding; drafts = 1
 * is an ordinary decode step).  Query row (b, i) sees the committed tokens
 * [0, seq_lens[b]) of its sequence and drafted token j, whose key and value
 * stand at position seq_lens[b] + j, where bit j of tree_mask[b, i] is set and
 * j < draft_lens[b]:
 *   out = sum_j softmax_j(scale * q . k_j) v_j, softmax statistics and sums in
 *   fp32, keys and values dequantized exactly, weights rounded to bf16.
 * A row that sees nothing gives zeros, and cache rows that nobody sees may hold
 * anything.  A drafted token's block whose scale leaves bf16's range (bytes 253 on)
 * reaches only the rows that see it.
 * q: bf16 [batch * drafts, ld_q]; out: bf16 [batch * drafts, ld_out]; rows
 * i >= draft_lens[b] are left as they were.  draft_lens: int32 [batch], NULL =
 * drafts for all.  tree_mask: uint64 [batch, drafts], NULL = token i sees
 * drafted tokens 0..i.  page_table: int32 [batch, max_pages]; seq_lens: int32
 * [batch].  Positions behind the table's end or on a page id outside
 * [0, num_pages) are not seen.
 * workspace: fp4_attn_tree_workspace_bytes(...) bytes, for the partial results
 * of contexts that are split over workgroups; calls (and replays) that share one
 * are ordered by the caller.  The order of the sums depends on
 * the shapes and lengths alone, so equal calls give equal bits.
 * Errors: head_dim not 64, 128 or 256, or cache->d != kv_heads * head_dim, or
 * q_heads not a multiple of kv_heads -> FP4_ERR_SHAPE; drafts outside [1, 64] ->
 * FP4_ERR_INVALID; scale not finite or above 2^127 in magnitude -> FP4_ERR_INVALID.
 * A magnitude below 7e-38 counts as 7e-38.
 */
int fp4_attn_tree_mx(const void* q, int64_t ld_q, const fp4_kv_cache* cache, const int32_t* page_table,
                     int64_t max_pages, const int32_t* seq_lens, const int32_t* draft_lens,
                     const uint64_t* tree_mask, int64_t batch, int drafts, int q_heads, int kv_heads, int head_dim,
                     float scale, void* out, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);
size_t fp4_attn_tree_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads);

/*
 * fp4_attn_tree_mx for a batch whose sequences share prefixes (forks of a prompt): group
 * g is the neighbouring sequences [groups[g], groups[g + 1]) (int32 [num_groups + 1],
 * ascending; values are taken as within [0, batch]), and their first prefix_lens[g]
 * (int32 [num_groups]) tokens are the same: the cache rows that the table of the group's
 * first sequence names for them are read, once for the whole group (that sequence has to
 * hold them while any of the group has prefix_lens[g] tokens or more).  Sequences outside
 * every group, and those with seq_lens[b] < prefix_lens[g], are attended by their own
 * table alone.  The result is fp4_attn_tree_mx's up to the rounding of the weights (each
 * relative to its row's running reference) and the order of the fp32 sums; the order
 * depends on the shapes, lengths and groups alone, and a sequence's bits on no other
 * sequence's queries, nor on query rows i >= draft_lens[b], which may hold anything.
 * Everything else is as there.  num_groups 0: nothing is shared.  The work is laid out for
 * batch / num_groups sequences to a group, so empty groups and a batch that is mostly
 * outside groups cost time, not correctness.
 * workspace: fp4_attn_shared_workspace_bytes(...) bytes, which serve every smaller batch
 * and num_groups too; calls (and replays) that share one are ordered by the caller.
 * Errors: as there; num_groups negative -> FP4_ERR_INVALID; num_groups of 2^20 or more, or
 * batch * drafts * q_heads / kv_heads of 2^31 or more -> FP4_ERR_SHAPE.
 */
int fp4_attn_shared_mx(const void* q, int64_t ld_q, const fp4_kv_cache* cache, const int32_t* page_table,
                       int64_t max_pages, const int32_t* seq_lens, const int32_t* draft_lens,
                       const uint64_t* tree_mask, const int32_t* groups, const int32_t* prefix_lens,
                       int64_t num_groups, int64_t batch, int drafts, int q_heads, int kv_heads, int head_dim,
                       float scale, void* out, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);
size_t fp4_attn_shared_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads,
                                       int64_t num_groups);

/*
 * Selects cache blocks by a cheap score ("DeepSeek-V4" article, section 3: the
 * lightning indexer scores a query latent against every compressed cache entry at
 * FP4).  A block is a page; the index holds an MXFP4 entry of dim values for every page
 * of the pool and each of `lists` lists: index_codes [num_pages, lists * dim/2],
 * index_scales [num_pages, lists * dim/32], list after list in a row
 * (fp4_kv_append_mx with the page ids as slots fills them).
 * q: bf16 [batch * drafts, ld_q], lists * dim values a token, quantized on the way as
 * fp4_quantize_mx does.  For query token (b, i) and list l, over the complete blocks n
 * of the sequence (n < seq_lens[b] / page_size, within the table's row, whose page id is
 * in [0, num_pages)):
 *   score(n) = sum over dim of q_hat[b, i, l] * entry_hat[page_table[b, n], l],
 * in fp32, exact where the products' block scales of a row lie within 2^7 of one
 * another (and dim <= 128; 2^5 at 512).  A score that is no number counts as -inf.
 * block_ids: int32 [batch, drafts, lists, n_select], the n_select blocks of largest
 * score in ascending order, of equal ones the lowest, then -1 where there are fewer.
 * The first n_first and the last n_recent complete blocks are taken before any other,
 * the lowest first where they are more than n_select.
 * scores: fp32 of the same shape or NULL: the scores of the blocks in block_ids, -inf
 * behind them.  Rows of i >= draft_lens[b] (int32 [batch], NULL = drafts for all) are
 * left as they were.
 * workspace: fp4_kv_select_workspace_bytes(...) bytes; calls (and replays) that share
 * one are ordered by the caller.
 * Errors: dim not a multiple of 32 in [32, 512], page_size not a multiple of 16, batch of
 * 65536 or more, lists above 4096, n_select of 2^20 or more, batch * drafts * lists of
 * 2^23 or more -> FP4_ERR_SHAPE; drafts outside [1, 64], lists < 1, a negative size -> FP4_ERR_INVALID.
 */
int fp4_kv_select_mx(const void* q, int64_t ld_q, const uint8_t* index_codes, const uint8_t* index_scales,
                     int64_t num_pages, int lists, int dim, const int32_t* page_table, int64_t max_pages,
                     const int32_t* seq_lens, const int32_t* draft_lens, int64_t page_size, int64_t batch, int drafts,
                     int n_select, int n_first, int n_recent, int32_t* block_ids, float* scores, void* workspace,
                     size_t workspace_bytes, void* stream);
size_t fp4_kv_select_workspace_bytes(int64_t batch, int drafts, int lists, int64_t max_pages);

/*
 * fp4_attn_tree_mx over selected blocks: query token (b, i) sees, of the committed tokens
 * of its sequence, the blocks (pages) that its list names and those behind the last
 * complete block, and drafted tokens as there.  block_ids: int32 [batch, drafts, lists,
 * n_select], lists 1 (all heads) or kv_heads (a list for each key/value head), as
 * fp4_kv_select_mx writes them; of a list the first min(n_select, seq_lens[b] / page_size)
 * entries are read, in any order; one outside [0, seq_lens[b] / page_size) names nothing,
 * and a block that is named twice counts twice.
 * Everything else is as there.  n_select 0: only what is behind the last complete block.
 * workspace: fp4_attn_blocks_workspace_bytes(...) bytes; calls (and replays) that share
 * one are ordered by the caller.
 * Errors: as there; lists neither 1 nor kv_heads, n_select negative -> FP4_ERR_INVALID;
 * n_select of 2^20 or more, more than 65535 columns of workgroups (drafts * kv_heads for
 * up to 64 query heads each) -> FP4_ERR_SHAPE.
 */
int fp4_attn_blocks_mx(const void* q, int64_t ld_q, const fp4_kv_cache* cache, const int32_t* page_table,
                       int64_t max_pages, const int32_t* seq_lens, const int32_t* draft_lens,
                       const uint64_t* tree_mask, const int32_t* block_ids, int lists, int n_select, int64_t batch,
                       int drafts, int q_heads, int kv_heads, int head_dim, float scale, void* out, int64_t ld_out,
                       void* workspace, size_t workspace_bytes, void* stream);
size_t fp4_attn_blocks_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads);

/*
 * Causal attention over whole prompts, packed one after another:
 *   out_i = sum_{j <= i, j in i's sequence} softmax_j(scale * q_i . k_j) v_j,
 * softmax statistics and sums in fp32, weights rounded to bf16.
 * cu_seqlens: int32 [seqs + 1], ascending: sequence s has the rows
 * [cu_seqlens[s], cu_seqlens[s + 1]); empty sequences are fine, values are taken
 * as within [0, tokens], and rows outside every sequence are left as they were.
 * q [tokens, ld_q], k [tokens, ld_k], v [tokens, ld_v], out [tokens, ld_out]: bf16.
 * out may not overlap q, k or v.  A key or value that is infinite or no number
 * reaches only the rows that see it.
 * Errors: head_dim not 64, 128 or 256, q_heads not a multiple of kv_heads, ld_k
 * or ld_v of 2^24 or more, 2^30 tokens or more, or 2^23 row tiles (of 128 rows, 256
 * at head_dim 256; one more for every sequence) over all query heads ->
 * FP4_ERR_SHAPE; scale not finite or above 2^127 in magnitude -> FP4_ERR_INVALID.  A
 * magnitude below 7e-38 counts as 7e-38.
 */
int fp4_attn_prompt(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int64_t seqs,
                    int64_t tokens, int q_heads, int kv_heads, int head_dim, int64_t ld_q, int64_t ld_k,
                    int64_t ld_v, float scale, void* out, int64_t ld_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4_H */
