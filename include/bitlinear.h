/*
 * bitlinear.h -- C ABI of the MI355X (gfx950) BitNet b1.58 BitLinear library.
 *
 * The BitLinear layer replaces a bias-free nn.Linear ("穿越1比特的奇幻旅程",
 * summary of the BitNet b1.58 2B4T report, section 架构创新). The forward pass
 * computed here is the W1.58A8 product of that report's GPU inference section
 * (推理实现 / GPU端): ternary weights stored four per byte, int8 activations,
 * an int32 product, and a rescale back to fp32.
 *
 * Conventions shared by every call
 *  - Shapes follow nn.Linear: activations x are [m][k] (tokens x in-features),
 *    weights W are [n][k] (out-features x in-features), outputs y are [m][n].
 *    All arrays are dense and row-major.
 *  - Every pointer argument is a DEVICE pointer, except `stream`, which is a
 *    hipStream_t passed as void* (NULL = the null stream). Every call only
 *    enqueues work on `stream` and returns; nothing is synchronised, nothing is
 *    allocated, and the library keeps no mutable global state, so calls on
 *    different streams may run concurrently. The caller owns every buffer.
 *    The one exception is bitlinear_forward_noalloc, which uses a
 *    library-owned scratch array per device (see there).
 *  - Outputs must not alias inputs. Device pointers must be 16-byte aligned.
 *  - Packed weight layout: row-major [n][k/4] bytes; byte j of a row holds the
 *    weights k = 4j+i in bits 2i..2i+1 (i = 0..3) as the code w+1 in {0,1,2};
 *    the code 3 never occurs.
 *  - Argument errors are reported before anything is enqueued. A failed kernel
 *    launch returns BL_ERR_HIP. Faults during execution surface at the
 *    caller's next synchronisation of `stream`. No C++ exception crosses the ABI.
 *  - The library targets gfx950 only.
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BL_OK = 0,
    BL_ERR_NULL = 1,       /* a required pointer is NULL                        */
    BL_ERR_SHAPE = 2,      /* m, n < 1, k < 4, k % 4 != 0, or a size too large   */
    BL_ERR_ALIGN = 3,      /* a device pointer is not 16-byte aligned           */
    BL_ERR_DTYPE = 4,      /* unknown activation dtype                          */
    BL_ERR_WORKSPACE = 5,  /* workspace smaller than bitlinear_workspace_size() */
    BL_ERR_HIP = 6,        /* a kernel launch failed                            */
    BL_ERR_VALUE = 7,      /* a scalar argument is out of range                 */
    /* range sentinels, never returned: every int32 is a value of the type, so
       a caller may pass any int (the library reports unknown values) */
    BL_STATUS_RANGE_MIN_ = -0x7FFFFFFF - 1,
    BL_STATUS_RANGE_MAX_ = 0x7FFFFFFF
} bl_status;

/* Element type of the activation input x (other values: BL_ERR_DTYPE; the
   sentinels make every int32 a value of the type). */
typedef enum {
    BL_F32 = 0,
    BL_BF16 = 1,
    BL_DTYPE_RANGE_MIN_ = -0x7FFFFFFF - 1,
    BL_DTYPE_RANGE_MAX_ = 0x7FFFFFFF
} bl_dtype;

/* Operation selector for bitlinear_workspace_size(): 0 = forward, 1 = FFN, as
 * the two calls a layer makes per batch; the offline pack and the bare integer
 * product follow. */
typedef enum {
    BL_OP_FORWARD = 0,
    BL_OP_FFN = 1,
    BL_OP_PACK = 2,
    BL_OP_GEMM_I32 = 3,
    BL_OP_PACK_THRESHOLD = 4,
    BL_OP_FORWARD_NORM = 5,
    BL_OP_FFN_SPARSE = 6,
    BL_OP_FORWARD_A4 = 7
} bl_op;

/* Largest supported dimension (k, n, hidden, ffn) and token count m. */
#define BL_MAX_DIM ((int64_t)1 << 20)
#define BL_MAX_TOKENS ((int64_t)1 << 22)

/*
 * Bytes of device workspace an operation needs (0 if none), for
 *   BL_OP_FORWARD:   (m, k, n)
 *   BL_OP_FFN:       (m, hidden, ffn)   -- the last two arguments
 *   BL_OP_PACK:      (m ignored, k, n)
 *   BL_OP_GEMM_I32:  (m, k, n)
 *   BL_OP_PACK_THRESHOLD: (m ignored, k, n)
 *   BL_OP_FORWARD_NORM:   (m, k, n)
 *   BL_OP_FFN_SPARSE:     (m, hidden, ffn)
 *   BL_OP_FORWARD_A4:     (m, k, n)
 * Returns 0 for invalid shapes and unknown ops as well; the operation itself
 * then reports the shape error.
 */
size_t bitlinear_workspace_size(int op, int64_t m, int64_t k, int64_t n);

/*
 * Offline weight quantization and packing ("BitNet 1-bit LLM 的混合精度微调技术",
 * BitLinear paragraph and operational-parameter paragraph: absmean scale;
 * "穿越1比特的奇幻旅程", sections 架构创新 and 推理实现 / GPU端: ternary values,
 * four per int8).
 *   w        fp32 [n][k] weights (input)
 *   packed   uint8 [n][k/4] 2-bit codes (output, layout above)
 *   gamma    fp32 [1] per-tensor scale gamma = mean|W| (output). The mean is
 *            accumulated in fp64: each row left to right, rows in order, then
 *            divided by n*k and rounded once to fp32. Weights quantize to
 *            clip(rint(w / gamma), -1, 1) with a correctly rounded fp32
 *            division and ties to even; gamma = 0 quantizes every weight to 0.
 *   workspace  >= bitlinear_workspace_size(BL_OP_PACK, 0, k, n) bytes: the
 *            fp64 row sums of the fixed summation order (one per row), which
 *            the library may not allocate itself.
 * Requires k % 4 == 0.
 */
bl_status bitlinear_pack_weights(const float *w, int64_t n, int64_t k,
                                 uint8_t *packed, float *gamma,
                                 void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Offline weight quantization with a magnitude threshold ("BitNet 三元权重阈值
 * 优化工程实践", section on the core principle of ternary threshold optimization:
 * the threshold is a factor -- 0.7 by default, 0.6-0.75 per layer kind -- times
 * mean|W|; weights above it keep their sign, the rest become 0; the scale is
 * the mean of the kept magnitudes over the whole tensor).
 *   w             fp32 [n][k] weights (input)
 *   delta_factor  finite, >= 0 (else BL_ERR_VALUE)
 *   packed        uint8 [n][k/4] (output): the same 2-bit layout as
 *                 bitlinear_pack_weights, code = w~ + 1 with
 *                 w~ = sign(w) if |w| > delta (strict), else 0
 *   alpha         fp32 [1] (output): sum of |w| over the kept weights divided by
 *                 n*k (all weights), accumulated in fp64 in the fixed order of
 *                 bitlinear_pack_weights, rounded once to fp32. alpha takes
 *                 gamma's place in bitlinear_forward and bitlinear_ffn.
 *   delta_out     optional fp32 [1] (output): delta = delta_factor * mean|W| as
 *                 one fp32 product, mean|W| exactly as gamma above; NULL skips it
 *   workspace     >= bitlinear_workspace_size(BL_OP_PACK_THRESHOLD, 0, k, n) bytes
 * Requires k % 4 == 0.
 */
bl_status bitlinear_pack_weights_threshold(const float *w, int64_t n, int64_t k, float delta_factor,
                                           uint8_t *packed, float *alpha, float *delta_out,
                                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Per-token absmax activation quantization to int8 ("BitNet 1-bit LLM 的混合精度
 * 微调技术", operational-parameter paragraph: absmax with epsilon 1e-5;
 * "BitNet 中使用直通估计器工程化三元权重训练", section 工程化训练流程与参数配置:
 * scale max|X| and factor 127; "穿越1比特的奇幻旅程", section 架构创新: 8-bit, per token).
 *   x        [m][k] activations of type `dtype` (BL_F32 or BL_BF16)
 *   q        int8 [m][k] (output): clamp(rint(x * (127 / s)), -127, 127)
 *   scale    fp32 [m] (output): s = max(max_k |x|, 1e-5)
 * Requires k % 4 == 0.
 */
bl_status bitlinear_quant_act(const void *x, bl_dtype dtype, int64_t m, int64_t k,
                              int8_t *q, float *scale, void *stream);

/*
 * Per-token RMS normalization fused into the absmax quantization: the
 * normalization BitLinear applies to its input before quantizing it ("subln",
 * "穿越1比特的奇幻旅程", section 架构创新: added for the stability of 1-bit
 * training; "BitNet 中使用直通估计器工程化三元权重训练", section
 * 工程化训练流程与参数配置: layer normalization keeping the variance, epsilon 1e-5).
 * The pages give no formula; the form used is RMSNorm without mean subtraction
 * or bias:
 *   S = sum_k x^2 (fp64, each square exact; the sum equals the correctly rounded
 *   fp64 sum except within ~k^2 2^-106 of a rounding boundary),
 *   r = 1 / sqrt(fp32(S / k) + 1e-5) in fp32, x^ = (x * r) * gain[k] in fp32,
 *   then q, scale as bitlinear_quant_act computes them for x^.
 *   gain     optional fp32 [k], 16-byte aligned; NULL = no gain (all ones)
 *   q, scale as in bitlinear_quant_act (scale = max(max_k |x^|, 1e-5))
 */
bl_status bitlinear_quant_act_norm(const void *x, bl_dtype dtype, int64_t m, int64_t k,
                                   const float *gain, int8_t *q, float *scale, void *stream);

/*
 * BitLinear forward of RMS-normalized activations: bitlinear_forward applied to
 * x^ of bitlinear_quant_act_norm, with the normalization fused into the
 * quantization kernel (no x^ in memory).
 *   gain       optional fp32 [k] (NULL = none)
 *   workspace  >= bitlinear_workspace_size(BL_OP_FORWARD_NORM, m, k, n) bytes
 * Other arguments and results as bitlinear_forward.
 */
bl_status bitlinear_forward_norm(const void *x, bl_dtype dtype, int64_t m, int64_t k, const float *gain,
                                 const uint8_t *packed, const float *gamma, int64_t n,
                                 float *y, int32_t *acc_out,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * BitLinear forward: y = (x quantized per token) x (ternary W)^T, rescaled
 * ("穿越1比特的奇幻旅程", section 推理实现 / GPU端: the W1.58A8 matrix product).
 *   x        [m][k] activations of type `dtype`
 *   packed   uint8 [n][k/4], gamma fp32 [1]: output of bitlinear_pack_weights
 *   y        fp32 [m][n] (output): y = (float)acc * ((s / 127) * gamma)
 *   acc_out  optional int32 [m][n] (output): acc = sum_k q[m][k] * w~[n][k];
 *            NULL skips it
 *   workspace  >= bitlinear_workspace_size(BL_OP_FORWARD, m, k, n) bytes
 * Requires k % 4 == 0. No bias (the layer has none: section 架构创新).
 * Cost note: the kernels read weight rows padded to a multiple of 64 inputs.
 * When k % 64 != 0 the workspace also holds such a padded copy of `packed`,
 * rewritten on every call (one extra n*k/4-byte read and write); the same
 * holds for bitlinear_ffn (hidden or ffn not a multiple of 64) and the
 * variants below.
 */
bl_status bitlinear_forward(const void *x, bl_dtype dtype, int64_t m, int64_t k,
                            const uint8_t *packed, const float *gamma, int64_t n,
                            float *y, int32_t *acc_out,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Squared-ReLU gated FFN of three BitLinear layers ("穿越1比特的奇幻旅程", section
 * 架构创新: squared ReLU instead of SwiGLU; "BitNet 1-bit LLM 的混合精度微调技术",
 * operational-parameter paragraph: squared ReLU with GLU gating):
 *   q, s  = quant(x)                         (shared by gate and up)
 *   g, u  = BitLinear_gate(x), BitLinear_up(x)      fp32 [m][ffn]
 *   h     = (max(g,0) * max(g,0)) * u                fp32 [m][ffn]
 *   qh, sh = quant(h)                        (per-token int8 requantization)
 *   y     = BitLinear_down(h)                        fp32 [m][hidden]
 *   x            [m][hidden] of type `dtype`
 *   gate_packed, up_packed  uint8 [ffn][hidden/4];  down_packed uint8 [hidden][ffn/4]
 *   *_gamma      fp32 [1] each
 *   y            fp32 [m][hidden] (output)
 *   hq_out       optional int8 [m][ffn] (output): qh; NULL skips it
 *   hs_out       optional fp32 [m] (output): sh; NULL skips it
 *   workspace    >= bitlinear_workspace_size(BL_OP_FFN, m, hidden, ffn) bytes
 * Requires hidden % 4 == 0 and ffn % 4 == 0.
 */
bl_status bitlinear_ffn(const void *x, bl_dtype dtype, int64_t m, int64_t hidden, int64_t ffn,
                        const uint8_t *gate_packed, const float *gate_gamma,
                        const uint8_t *up_packed, const float *up_gamma,
                        const uint8_t *down_packed, const float *down_gamma,
                        float *y, int8_t *hq_out, float *hs_out,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * bitlinear_forward for callers that cannot allocate device memory: code under
 * HIP graph capture, serving loops and harnesses that forbid hipMalloc. Same
 * arguments and results as bitlinear_forward without the workspace: the
 * scratch space comes from a library-owned device array of
 * BL_NOALLOC_SCRATCH_BYTES per device, which each device the library runs on
 * holds until the process ends. Nothing is allocated, freed or synchronised.
 *   Returns BL_ERR_WORKSPACE when bitlinear_workspace_size(BL_OP_FORWARD, m, k, n)
 *   exceeds BL_NOALLOC_SCRATCH_BYTES (e.g. m * roundup(k, 64) above ~32 M);
 *   BL_ERR_VALUE when `stream` belongs to another device than the current one.
 * Every call on a device shares that device's array, and the array keeps the
 * last call's contents (every call writes what it reads first): calls that
 * overlap on one device race -- serialise them (one stream, or events).
 */
#define BL_NOALLOC_SCRATCH_BYTES ((int64_t)32 << 20)
bl_status bitlinear_forward_noalloc(const void *x, bl_dtype dtype, int64_t m, int64_t k,
                                    const uint8_t *packed, const float *gamma, int64_t n,
                                    float *y, int32_t *acc_out, void *stream);

/*
 * 4-bit activations for the W1.58A4 variant ("BitNet 1-bit LLM 的混合精度微调技术",
 * paragraph on progressive quantization: activations brought to 4 bits in the
 * MinMax FP4 format with E2M1 bits, top-K sparsification of 50 % against
 * outlier channels). The pages give no formula; the form used, per token:
 *   tau  = the keep-th largest |x|; entries with |x| >= tau are kept (ties at
 *          tau all kept), the others become 0
 *   s    = max(max_k |x|, 1e-5); v = x * (6 / s) (one fp32 division per token)
 *   e    = the nearest E2M1 value to v (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 *          negatives), ties to the value whose mantissa bit is 0
 *   q    = 2e, an int8 in [-12, 12], so that x ~ q * s / 12
 *   keep    1..k (BL_ERR_VALUE otherwise); the pages' 50 % is keep = ceil(k / 2)
 *   q, scale  int8 [m][k] and fp32 [m] (output)
 */
bl_status bitlinear_quant_act_a4(const void *x, bl_dtype dtype, int64_t m, int64_t k, int64_t keep,
                                 int8_t *q, float *scale, void *stream);

/*
 * W1.58A4 forward: the 4-bit codes of bitlinear_quant_act_a4 times the ternary
 * weights, y = (float)acc * ((s / 12) * gamma), acc = sum_k q[m][k] * w~[n][k]
 * (exact in int32: the doubled E2M1 codes are small integers).
 *   workspace  >= bitlinear_workspace_size(BL_OP_FORWARD_A4, m, k, n) bytes
 * Other arguments and results as bitlinear_forward.
 */
bl_status bitlinear_forward_a4(const void *x, bl_dtype dtype, int64_t m, int64_t k, int64_t keep,
                               const uint8_t *packed, const float *gamma, int64_t n,
                               float *y, int32_t *acc_out,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * Input-major copy of packed weights (offline, once per weight): the codes of
 * packed [n][k/4] rearranged as packed_t [k][n/4], row c holding the codes of
 * outputs 4j+i of input c in bits 2i..2i+1 of byte j -- the packing of the
 * transposed ternary matrix. Used for the FFN's down projection by
 * bitlinear_ffn_sparse. Requires n % 4 == 0 and k % 4 == 0.
 */
bl_status bitlinear_pack_kmajor(const uint8_t *packed, int64_t n, int64_t k, uint8_t *packed_t, void *stream);

/*
 * bitlinear_ffn for decode (1 <= m <= 4 tokens) with the down projection reading
 * only the weights of the non-zero channels of the requantized h
 * ("BitNet 1-bit LLM 的混合精度微调技术", operational-parameter paragraph: with the
 * squared-ReLU GLU gating, only the non-zero channels are computed). The down
 * weights come input-major (bitlinear_pack_kmajor of the [hidden][ffn/4]
 * matrix), so a channel whose code is 0 for every token skips its whole row.
 * Results are those of bitlinear_ffn: zero codes contribute nothing.
 *   down_packed_t  uint8 [ffn][hidden/4] (input-major)
 *   workspace      >= bitlinear_workspace_size(BL_OP_FFN_SPARSE, m, hidden, ffn)
 * Other arguments as bitlinear_ffn. Requires m <= 4, hidden % 16 == 0 and
 * ffn % 4 == 0 (BL_ERR_SHAPE otherwise).
 */
bl_status bitlinear_ffn_sparse(const void *x, bl_dtype dtype, int64_t m, int64_t hidden, int64_t ffn,
                               const uint8_t *gate_packed, const float *gate_gamma,
                               const uint8_t *up_packed, const float *up_gamma,
                               const uint8_t *down_packed_t, const float *down_gamma,
                               float *y, int8_t *hq_out, float *hs_out,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * The bare ternary x int8 contraction ("穿越1比特的奇幻旅程", section
 * 推理实现 / GPU端), exposed for parity checks of the integer product alone.
 *   q        int8 [m][k] (input, natural layout)
 *   packed   uint8 [n][k/4]
 *   acc      int32 [m][n] (output): sum_k q[m][k] * w~[n][k], exact
 *   workspace  >= bitlinear_workspace_size(BL_OP_GEMM_I32, m, k, n) bytes: the
 *            kernels read q in an internal permuted layout, copied there first
 */
bl_status bitlinear_gemm_i32(const int8_t *q, int64_t m, int64_t k,
                             const uint8_t *packed, int64_t n, int32_t *acc,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Attention between the QKV and the output projection. The projections' fused
 * output is read in place: q, k and v are [m][heads][head_dim] with the heads of
 * a token adjacent and `*_stride` elements from one token to the next (a
 * multiple of 16 bytes, heads * head_dim to 2^24). head_dim is 64 or 128;
 * q_heads is a multiple of kv_heads, and query head h reads kv head
 * h / (q_heads / kv_heads).
 *
 * Packed sequences: `cu_seqlens` int32 [seqs + 1] on the device, sequence s is
 * rows cu_seqlens[s] .. cu_seqlens[s+1]-1 (empty ones are allowed). Offsets are
 * read by the kernels, so a call can be captured and replayed with others;
 * values outside 0..m are taken as the nearest of the two. Offsets do not decrease:
 * where they do, a sequence that ends before it begins is empty, and what a call
 * leaves in the rows (and the cache's pages) that its sequences name is unspecified,
 * but nothing else is read or written. Rows before the first and behind the last
 * sequence are not written and enter nothing.
 */
#define BL_MAX_HEADS ((int64_t)1 << 12)

/* Bytes of workspace of bitlinear_attention (0 if none, or for invalid shapes) */
size_t bitlinear_attention_workspace_size(bl_dtype dtype, int64_t m, int64_t q_heads, int64_t kv_heads,
                                          int64_t head_dim, int64_t seqs);

/*
 * Causal attention over whole prompts: for row i of a sequence and query head h
 *   p_ij = softmax over j <= i of scale * (q_i . k_j),   out_i = sum_j p_ij v_j
 *   out       [m][q_heads * head_dim] of type `dtype` (output)
 *   scale     finite (BL_ERR_VALUE otherwise); usually 1 / sqrt(head_dim)
 * BL_BF16: products of the bf16 inputs summed in fp32, softmax in fp32, p
 * rounded to bf16 for its product with v. BL_F32: sums and softmax in fp32, the
 * factors of the two products held to 2^-22 of their value, but elements of q, k
 * and v no closer than 2^-39 of the largest of their row (one token and head), nor
 * than 2^-137, and the weights no closer than 2^-36 of the row's largest
 * p_ij max |v_j|.
 * A row depends on rows 0..i of its own sequence only: infinities and NaN in
 * later rows or in other sequences do not reach it. Those that a row sees count as
 * the formula has them: a logit of -inf gives its key no weight; one of +inf or NaN
 * makes the row NaN, as -inf in all of them does. An element of v_j that is not
 * finite reaches every row that sees it, whatever its weight: as NaN where the row
 * sees a NaN or infinities of both signs in that dim, otherwise as the infinity
 * (but a row of NaN weights is NaN throughout). Finite values of v beside which
 * 2^8 sum_j |v_j| passes fp32's range may give results that are not (BL_BF16), and so
 * may logits that do.
 * BL_ERR_SHAPE also where m * q_heads / kv_heads, or its 64th part (plus seqs)
 * times kv_heads, passes 2^31 - 1024.
 *   workspace  >= bitlinear_attention_workspace_size() bytes
 */
bl_status bitlinear_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                              const void *v, int64_t v_stride, bl_dtype dtype, int64_t m,
                              int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                              const int32_t *cu_seqlens, int64_t seqs, float scale, void *out,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * The 8-bit key/value cache. Pages hold BL_CACHE_BLOCK tokens; a sequence's
 * block b of 64 tokens lies in page block_table[s][b] (int32 [seqs][max_blocks]).
 * Per page and kv head there are 64 * head_dim int8 codes of K, as many of V, and
 * one fp32 scale for each of the two; the code c stands for c * (scale / 127).
 *   k_codes, v_codes  int8 [pages][kv_heads][64 * head_dim], 16-byte aligned
 *   k_scale, v_scale  fp32 [pages][kv_heads]
 * Inside a page and head the codes lie in 256-byte tiles of 16 rows x 16 bytes,
 * the order in which the matrix instructions take them:
 *   K code of (token, dim): ((token % 4) * (head_dim / 16) + dim / 16) * 256 + (token / 4) * 16 + dim % 16
 *   V code of (token, dim): ((dim / 16) * 4 + token / 16) * 256 + (dim % 16) * 16 + token % 16
 * Table entries outside 0..pages-1 name no page: such a block is not written and
 * holds no tokens. Blocks from max_blocks on do not exist either.
 * `lens` int32 [seqs] counts the tokens that a sequence holds before a call's new
 * ones; a negative entry marks an unused slot, whose rows are skipped.
 * `cu_seqlens` as above, or NULL for one row per sequence (m == seqs).
 */
#define BL_CACHE_BLOCK 64

/*
 * Appends new tokens: row i of sequence s becomes token lens[s] + i. Per block
 * and kv head, for K and V each:
 *   s' = max(s, max |x| over the block's new rows, 1e-30), where s is the stored
 *        scale if the block holds earlier tokens and 0 otherwise
 *   new codes      rint(x * (127 / s'))
 *   earlier codes  rint(c * (s / s')) if the scale grew
 * in fp32, ties to even. Codes of later slots stay as they are. NaN counts as 0
 * and infinities as the largest finite number, beside which the block's other
 * codes become 0 (and c * (scale / 127) may round to an infinity again). `lens` is
 * not changed: the caller adds the new tokens once every layer has appended. Two
 * sequences may share pages that no call writes.
 */
bl_status bitlinear_cache_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                 bl_dtype dtype, int64_t m, int64_t kv_heads, int64_t head_dim,
                                 const int32_t *cu_seqlens, const int32_t *lens, int64_t seqs,
                                 const int32_t *block_table, int64_t max_blocks, int8_t *k_codes,
                                 int8_t *v_codes, float *k_scale, float *v_scale, int64_t pages, void *stream);

/*
 * Reads tokens back: row i of sequence s is token begin[s] + i (begin as `lens`
 * above), as fp32 c * (scale / 127), rounded once more for BL_BF16. Tokens
 * without a page are written as 0.
 *   k_out, v_out  [m][kv_heads][head_dim] of type `dtype` (output), dense
 */
bl_status bitlinear_cache_read(const int8_t *k_codes, const int8_t *v_codes, const float *k_scale,
                               const float *v_scale, int64_t pages, const int32_t *block_table,
                               int64_t max_blocks, const int32_t *cu_seqlens, const int32_t *begin,
                               int64_t seqs, bl_dtype dtype, int64_t m, int64_t kv_heads, int64_t head_dim,
                               void *k_out, void *v_out, void *stream);

/* Bytes of workspace of bitlinear_attention_cached; `weights`: whether block
 * weights are accumulated (0 if none, or for invalid shapes) */
size_t bitlinear_attention_cached_workspace_size(int64_t m, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                 int64_t seqs, int64_t max_blocks, int weights);

/*
 * Attention of new tokens over the cache (decode, and a few tokens at once).
 * Row i of sequence s is the query of token lens[s] + i, already appended, and
 * sees the tokens 0 .. lens[s] + i that have a page; a row that sees none gives 0.
 *   q, out    as in bitlinear_attention
 *   weights   optional fp32 [seqs][max_blocks] (input and output): the attention
 *             weight that each block received, summed over the call's rows and
 *             query heads, is added to it; blocks without one are left alone
 * The codes enter exactly; q is held to 2^-22 of its row's largest (or of 1e-30,
 * where that is larger), the softmax weights to 2^-23 of their block's largest, sums
 * are exact int32 within a block and fp32 across blocks, for either dtype. Logits
 * or sums that pass fp32's range give a row that is not finite. A row of q that is
 * not finite gives NaN and adds nothing to the weights. Results do not depend on
 * the order of execution.
 *   workspace  >= bitlinear_attention_cached_workspace_size() bytes
 */
bl_status bitlinear_attention_cached(const void *q, int64_t q_stride, bl_dtype dtype, int64_t m,
                                     int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                     const int32_t *cu_seqlens, const int32_t *lens, int64_t seqs,
                                     const int32_t *block_table, int64_t max_blocks, const int8_t *k_codes,
                                     const int8_t *v_codes, const float *k_scale, const float *v_scale,
                                     int64_t pages, float scale, void *out, float *weights, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * Chooses the blocks that a sequence keeps, by accumulated attention weight. Of
 * the ceil(lens[s] / 64) blocks (at most max_blocks) the first `first`, the last
 * `recent` and, up to `keep` in all, the ones of the largest weight stay, in
 * their order; of equal weights the lower block stays, and NaN counts as +inf.
 *   keep >= first + recent, first >= 0, recent >= 1 (BL_ERR_VALUE otherwise)
 *   table_out    int32 [seqs][max_blocks]: pages of the kept blocks, then -1
 *   weights_out  fp32 [seqs][max_blocks]: their weights, then 0
 *   lens_out     int32 [seqs]: lens minus 64 per evicted block (unused slots as is)
 *   evicted      int32 [seqs][max_blocks]: pages of the evicted blocks, then -1
 *   evicted_count  int32 [seqs]
 * The outputs lie apart from the inputs. Table entries are passed on as they are: one
 * that names no page may be among the evicted, and a page that other sequences share
 * is theirs still.
 */
bl_status bitlinear_cache_evict(const int32_t *block_table, const int32_t *lens, const float *weights,
                                int64_t seqs, int64_t max_blocks, int64_t keep, int64_t first, int64_t recent,
                                int32_t *table_out, int32_t *lens_out, float *weights_out, int32_t *evicted,
                                int32_t *evicted_count, void *stream);

/*
 * Rotation of queries and keys by their tokens' positions, between the QKV projection
 * and the attention or the cache, with an optional RMS norm of every head before it.
 * Row i of sequence s is position begin[s] + i (begin as `lens` of the cache calls: for
 * a prompt 0, for new tokens the tokens before them, evicted ones included; a negative
 * entry marks an unused slot). Per row and head x, y = x without a gain and otherwise
 *   y = (x * r) * gain[d],  r = 1 / sqrt(mean_d x^2 + eps)
 * in fp32, and for the pairs i < rotary_dim / 2 of y, t = position * inv_freq[i],
 *   (a, b) -> (a * cs - b * sn, b * cs + a * sn),  cs = magnitude * cos t, sn = magnitude * sin t
 * with (a, b) = (y[2i], y[2i + 1]) if `interleaved`, (y[i], y[i + rotary_dim / 2]) if not;
 * elements from rotary_dim on stay y. One rounding to `dtype` at the end. Angles are
 * exact up to rounding of cs and sn to fp32, whatever the position, while |t| < 2^50. A
 * head whose squares pass fp32's range has r = 0.
 *   q, k            as in bitlinear_attention
 *   inv_freq        fp32 [rotary_dim / 2], 4-byte aligned
 *   rotary_dim      16 .. head_dim, a multiple of 16 (BL_ERR_SHAPE otherwise)
 *   interleaved     0 or 1 (BL_ERR_VALUE otherwise)
 *   magnitude       finite, eps finite and >= 0 (BL_ERR_VALUE otherwise)
 *   q_gain, k_gain  optional fp32 [head_dim], 16-byte aligned; NULL = no norm
 *   q_out, k_out    rows like q's and k's (output), `*_stride` elements apart. In place is
 *                   allowed: q_out = q with the same stride, k_out = k likewise. Rows of
 *                   unused slots and outside the sequences are not written.
 */
bl_status bitlinear_rotate(const void *q, int64_t q_stride, const void *k, int64_t k_stride, bl_dtype dtype, int64_t m,
                           int64_t q_heads, int64_t kv_heads, int64_t head_dim, const int32_t *cu_seqlens,
                           const int32_t *begin, int64_t seqs, const float *inv_freq, int64_t rotary_dim, int interleaved,
                           float magnitude, const float *q_gain, const float *k_gain, float eps, void *q_out,
                           int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream);

/* Bytes of workspace of bitlinear_attention_shared (0 for invalid shapes) */
size_t bitlinear_attention_shared_workspace_size(int64_t m, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                 int64_t seqs, int64_t max_blocks, int64_t prefix_blocks);

/*
 * Attention of new tokens over the cache of a batch whose sequences share a prefix: a
 * row sees the prefix's tokens 0 .. prefix_len - 1 that have a page, and its own
 * sequence's as in bitlinear_attention_cached (lens does not count the prefix). The
 * prefix is read once for all rows.
 *   prefix_table  int32 [prefix_blocks] on the device: the prefix's pages, in the caches
 *                 of the sequences' own. Entries that name no page hold no tokens.
 *   prefix_len    int32 [1] on the device; below 1: no prefix, and at most
 *                 64 * prefix_blocks count
 * Over the prefix q is held to 2^-22 of itself (fp32; elements below 2^-17 of their
 * row's largest, or of 1e-30, to 2^-39 of that) or exactly (bf16, to 2^-39 of the
 * largest), and the softmax weights to 2^-22 (fp32) or 2^-11 (bf16) of themselves, or 2^-39
 * of the largest of their block and row; sums are fp32. The rest is as in
 * bitlinear_attention_cached: rows that see nothing, rows of q that are not finite, logits or
 * sums that pass fp32's range, unused slots and rows outside the sequences among it. Results
 * do not depend on the order of execution.
 * BL_ERR_SHAPE also where m * q_heads / kv_heads passes 2^31 - 1024.
 *   workspace  >= bitlinear_attention_shared_workspace_size() bytes
 */
bl_status bitlinear_attention_shared(const void *q, int64_t q_stride, bl_dtype dtype, int64_t m, int64_t q_heads,
                                     int64_t kv_heads, int64_t head_dim, const int32_t *prefix_table, int64_t prefix_blocks,
                                     const int32_t *prefix_len, const int32_t *cu_seqlens, const int32_t *lens,
                                     int64_t seqs, const int32_t *block_table, int64_t max_blocks, const int8_t *k_codes,
                                     const int8_t *v_codes, const float *k_scale, const float *v_scale, int64_t pages,
                                     float scale, void *out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Bounds of the cache's blocks: per page and kv head the largest and the smallest code of
 * K of every dim, over the tokens that the block holds.
 *   bounds  int8 [pages][kv_heads][2][head_dim], 16-byte aligned (output): [0] the largest,
 *           [1] the smallest. Blocks that rows lens[s] .. of a sequence reach are written
 *           (called after bitlinear_cache_append with the same rows: the blocks that
 *           changed), others left as they are.
 * Other arguments as in bitlinear_cache_append; m counts the rows.
 */
bl_status bitlinear_cache_bounds(const int8_t *k_codes, int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t m,
                                 const int32_t *cu_seqlens, const int32_t *lens, int64_t seqs, const int32_t *block_table,
                                 int64_t max_blocks, int8_t *bounds, void *stream);

/* Bytes of workspace of bitlinear_block_select (0 if none, or for invalid shapes) */
size_t bitlinear_block_select_workspace_size(int64_t m, int64_t kv_heads, int64_t max_blocks);

/*
 * Chooses the blocks that a new token attends to, for every row and kv head, by an upper
 * bound of the products of its query heads (summed over the group) with a block's keys. The
 * queries of a row's kv head become integers as activations do,
 *   c = rint(x * (127 / s)),  s = max(max |x| over the group's heads and dims, 1e-30)
 * in fp32, ties to even (NaN counts as 0, infinities as the largest finite number), and
 *   T = sum_d high_d * sum_h max(c_hd, 0) + low_d * sum_h min(c_hd, 0)    (exact)
 *   score = fp32(T) * k_scale of the page
 * Row i of sequence s is token lens[s] + i, already appended and in the bounds, and has
 * (lens[s] + i) / 64 + 1 blocks (at most max_blocks). The first `first`, the last `recent`
 * of these and, up to `keep` in all, the ones of the largest score stay; of equal scores the
 * lower block, NaN counts as +inf, and a block without a page has -inf. The last `recent`
 * blocks' bounds are not needed: with recent >= 1, those of a block that is still filling.
 *   keep      first + recent .. 2^20, first >= 0, recent >= 1 (BL_ERR_VALUE otherwise)
 *   selected  int32 [m][kv_heads][keep] (output): blocks of the sequence, ascending, then
 *             -1; rows of unused slots and outside the sequences are not written
 *   q_heads / kv_heads <= 128 (BL_ERR_SHAPE otherwise)
 *   workspace >= bitlinear_block_select_workspace_size() bytes
 */
bl_status bitlinear_block_select(const void *q, int64_t q_stride, bl_dtype dtype, int64_t m, int64_t q_heads,
                                 int64_t kv_heads, int64_t head_dim, const int32_t *cu_seqlens, const int32_t *lens,
                                 int64_t seqs, const int32_t *block_table, int64_t max_blocks, const int8_t *bounds,
                                 const float *k_scale, int64_t pages, int64_t keep, int64_t first, int64_t recent,
                                 int32_t *selected, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace of bitlinear_attention_selected (0 if none, or for invalid shapes) */
size_t bitlinear_attention_selected_workspace_size(int64_t m, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                                   int64_t keep);

/*
 * Attention of new tokens over chosen blocks of the cache: bitlinear_attention_cached, but
 * a row and kv head sees the tokens 0 .. lens[s] + i of the blocks that
 *   selected  int32 [m][kv_heads][keep], keep 1 .. 2^20
 * lists for it. Entries outside 0 .. max_blocks - 1 name no block, wherever they stand; a
 * block counts as often as it is listed. Precision, rows that see nothing (0) or are not
 * finite, unused slots: as there.
 * BL_ERR_SHAPE also where m * q_heads / kv_heads passes 2^31 - 1024.
 *   workspace  >= bitlinear_attention_selected_workspace_size() bytes
 */
bl_status bitlinear_attention_selected(const void *q, int64_t q_stride, bl_dtype dtype, int64_t m, int64_t q_heads,
                                       int64_t kv_heads, int64_t head_dim, const int32_t *cu_seqlens, const int32_t *lens,
                                       int64_t seqs, const int32_t *block_table, int64_t max_blocks,
                                       const int32_t *selected, int64_t keep, const int8_t *k_codes,
                                       const int8_t *v_codes, const float *k_scale, const float *v_scale, int64_t pages,
                                       float scale, void *out, void *workspace, size_t workspace_bytes, void *stream);

/* Human-readable name of a status code (static string, never NULL). */
const char *bitlinear_status_string(bl_status status);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_H */
