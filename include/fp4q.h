/*
 * fp4q.h -- block-scaled FP4 quantization of bf16 tensors on AMD MI355X
 * (gfx950).  C ABI of libfp4q.so.
 *
 * The method (cited by page title and section):
 *  - NVFP4: FP4 E2M1 values, one FP8 E4M3 scale per 16 consecutive values
 *    and one FP32 tensor scale ("Four Over Six: More Accurate NVFP4
 *    Quantization with Adaptive Block Scaling", sec. 2.1, Eq. 1-3; NVIDIA
 *    NVFP4 pretraining article, sec. 1 and sec. 6).
 *  - Four Over Six: per 16-value block, quantize with the block maximum
 *    scaled to 6 and to 4 and keep the one with the smaller error ("Four
 *    Over Six", sec. 1, Fig. 1 and the worked example).
 *  - Variants for the tensors of a training step (NVIDIA NVFP4 article,
 *    sec. 2 and sec. 7): a 16-point random Hadamard rotation and stochastic
 *    rounding for gradients, 16x16 two-dimensional blocks for weights.
 *  - MXFP4: 32 values per power-of-two (UE8M0) scale (NVIDIA NVFP4 article,
 *    sec. 1 and sec. 5), with a fixed 32-point Hadamard rotation (AMD
 *    MI355X MXFP4 pretraining article, sec. 2) and row- and column-wise
 *    outputs.
 *
 * Conventions shared by every call:
 *  - Every tensor pointer is a DEVICE pointer (HIP device memory of the
 *    current device).  The caller allocates every buffer and owns it; the
 *    library allocates nothing and keeps no state between calls (except the
 *    fixed per-device array of nvfp4_quantize_noalloc).
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *    Work is queued on it asynchronously; the call returns before the GPU
 *    finishes.  Concurrent calls on different streams are safe as long as
 *    they do not share output or workspace buffers.
 *  - Inputs are row-major bf16 bit patterns [rows][cols], 16-byte aligned.
 *  - Packed FP4 codes: two per byte, the even-indexed element in the low
 *    nibble; code = sign << 3 | magnitude index into {0, .5, 1, 1.5, 2, 3,
 *    4, 6}.  Code buffers must be 16-byte aligned.
 *  - Scales are one byte per block in row-major block order; NVFP4 scales
 *    are E4M3 (bias 7, max 448), MXFP4 scales are UE8M0 (2^(code-127)).
 *  - Errors: the return value is an fp4_status.  Argument checks run on the
 *    host before any HIP call, so a rejected call touches no device state.
 *    FP4_E_HIP reports a failed kernel launch (the launch's own return
 *    status; an error left by an earlier, unrelated HIP call is neither
 *    reported nor cleared); faults during execution surface at the caller's
 *    next synchronisation.  A launch of 2^32 threads or more, which HIP would
 *    cut short without an error, is one that fails.
 *  - Tensors holding Inf/NaN, or (NVFP4) whose largest magnitude is below
 *    2^-64 without being zero, are outside the method's domain: the call
 *    succeeds and never faults, but codes and scales are unspecified.
 */
#ifndef FP4Q_H
#define FP4Q_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP4_OK = 0,
  FP4_E_NULL = -1,      /* a required pointer is NULL                     */
  FP4_E_SHAPE = -2,     /* rows/cols negative, not a block multiple, or
                           rows*cols >= 2^40; a size or number out of the
                           range that its call names                      */
  FP4_E_ALIGN = -3,     /* a pointer breaks the alignment rules above     */
  FP4_E_FLAGS = -4,     /* unknown bit or an unsupported combination      */
  FP4_E_WORKSPACE = -5, /* workspace smaller than fp4_workspace_bytes()   */
  FP4_E_HIP = -6        /* kernel launch failed                           */
} fp4_status;

/* Mode flags. */
enum {
  FP4_RTN6 = 0u,               /* NVFP4, block max scaled to 6, nearest-even  */
  FP4_FOUR_OVER_SIX = 1u << 0, /* NVFP4: adaptive choice of 6 or 4 per block  */
  FP4_SR = 1u << 1,            /* NVFP4: stochastic rounding of FP4 values    */
  FP4_RHT16 = 1u << 2,         /* NVFP4: 16-point random Hadamard along rows  */
  FP4_BLOCK2D = 1u << 3,       /* NVFP4: 16x16 tiles instead of 1x16 blocks   */
  FP4_HAD32 = 1u << 4,         /* MXFP4: 32-point Hadamard before quantizing  */
  FP4_ROWWISE = 1u << 5,       /* MXFP4: emit row-wise output                 */
  FP4_COLWISE = 1u << 6,       /* MXFP4: emit column-wise output;
                                  NVFP4 2D: also emit the transpose          */
  FP4_MSEDEN = 1u << 7         /* NVFP4: MS-EDEN -- RTN values, unbiasing
                                  factor, stochastic E4M3 scale (with RHT16) */
};

enum { FP4_FORMAT_NVFP4 = 0, FP4_FORMAT_MXFP4 = 1 };

/* Bytes of device workspace nvfp4_quantize and nvfp4_requantize_t (with
 * amax_in == NULL) and fp4_tensor_amax need for this shape and these
 * flags; 0 if none.  The
 * workspace needs no initialisation and is scratch for the duration of the
 * call (stream order). */
size_t fp4_workspace_bytes(int64_t rows, int64_t cols, uint32_t flags);

/* Largest magnitude of the tensor the NVFP4 quantizer scales by ("Four Over
 * Six" Eq. 1 numerator; NVIDIA NVFP4 article sec. 6 and sec. 9: the extra
 * pass over memory for the global scale).  With FP4_RHT16 it is the
 * largest magnitude after the rotation (seeded by `seed`).  Other NVFP4 flag
 * bits are accepted and ignored; FP4_HAD32 is rejected.
 *   x        [rows][cols] bf16, cols % 16 == 0
 *   amax_out one float (device), written in stream order
 *   ws       fp4_workspace_bytes(rows, cols, flags) bytes (device) */
int fp4_tensor_amax(const uint16_t* x, int64_t rows, int64_t cols,
                    uint32_t flags, uint64_t seed, float* amax_out,
                    void* ws, size_t ws_bytes, void* stream);

/* NVFP4 quantization ("Four Over Six" Eq. 1-3 and sec. 1; NVIDIA NVFP4
 * article sec. 2 and sec. 6).
 *   flags     FP4_RTN6 or any of FOUR_OVER_SIX, SR, RHT16, BLOCK2D
 *             (+ COLWISE with BLOCK2D), or MSEDEN|RHT16.  Rejected:
 *             SR|FOUR_OVER_SIX, BLOCK2D|SR, BLOCK2D|RHT16, HAD32, COLWISE
 *             without BLOCK2D, MSEDEN without RHT16 or with SR,
 *             FOUR_OVER_SIX or BLOCK2D.
 *             MSEDEN (Quartet II / MS-EDEN article, sec. 1: rotation,
 *             round-to-nearest values, randomness only in the 8-bit scale;
 *             the unbiasing factor is EDEN's): per block the values are
 *             rounded to nearest against the unrounded scale Delta_pre,
 *             the scale becomes S * Delta_pre with S = sum t^2 / sum t q
 *             and is rounded stochastically to E4M3 (Philox counter =
 *             (block index lo, hi, 1, 0)); C = 256.
 *   seed      Philox key for SR (counter = row*cols + col) and RHT16 signs.
 *   amax_in   NULL: computed here (one extra read of x, needs `ws`);
 *             else one device float taken as the tensor's largest magnitude.
 *   alpha_out one device float: the FP32 tensor scale amax/(6*C), C = 448,
 *             or 256 with FOUR_OVER_SIX.
 *   codes     [rows][cols/2] bytes.
 *   scales    E4M3, [rows][cols/16] (1D) or [rows/16][cols/16] (BLOCK2D).
 *   choice    NULL or one byte per scale, 1 where the block took M = 4.
 *   codes_t, scales_t  BLOCK2D|COLWISE only (else NULL): the same
 *             quantization laid out for the transpose, [cols][rows/2] and
 *             [cols/16][rows/16].
 *   Shapes: cols % 16 == 0; BLOCK2D also rows % 16 == 0. */
int nvfp4_quantize(const uint16_t* x, int64_t rows, int64_t cols,
                   uint32_t flags, uint64_t seed, const float* amax_in,
                   float* alpha_out, uint8_t* codes, uint8_t* scales,
                   uint8_t* choice, uint8_t* codes_t, uint8_t* scales_t,
                   void* ws, size_t ws_bytes, void* stream);

/* nvfp4_quantize for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same call without a workspace argument.  With amax_in ==
 * NULL the amax pass keeps its per-workgroup partial maxima in a fixed
 * 4 KiB device array of the library (one per device, held until the process
 * ends; its address is looked up once per device on the first call there)
 * instead of caller memory.  The call allocates nothing.
 *   Arguments, results and errors as nvfp4_quantize; FP4_E_WORKSPACE if the
 *   shape and flags would need more than that array (never for the flag
 *   sets nvfp4_quantize accepts).
 *   Every call on one device shares that array: calls that overlap in time
 *   on one device (different streams, or host threads) race and may produce
 *   wrong results; calls in one stream's order are safe.  Nothing in it
 *   needs to start at zero (each call writes every partial it reads). */
int nvfp4_quantize_noalloc(const uint16_t* x, int64_t rows, int64_t cols,
                           uint32_t flags, uint64_t seed, const float* amax_in,
                           float* alpha_out, uint8_t* codes, uint8_t* scales,
                           uint8_t* choice, uint8_t* codes_t, uint8_t* scales_t,
                           void* stream);

/* NVFP4 with one FP32 scale per row, quantized in a single read of x.  The
 * NVIDIA NVFP4 article (sec. 9) names the extra memory pass for the global
 * scale as a cost and proposes finer-grained global scales, per row or per
 * block.  Row r takes alpha_r = amax_r / (6*C) ("Four Over Six" Eq. 1 on
 * the row; C = 448, or 256 with FOUR_OVER_SIX; amax after RHT16 when asked)
 * and is otherwise quantized exactly as nvfp4_quantize would quantize it
 * (Eq. 2-3, 4/6, SR with counter = row*cols + col).  Results differ from
 * nvfp4_quantize wherever rows have different maxima; a consumer decodes
 * row r with alpha_rows[r].
 *   flags      FP4_RTN6 or FOUR_OVER_SIX, SR, RHT16 (SR|FOUR_OVER_SIX
 *              rejected); BLOCK2D, COLWISE, ROWWISE and HAD32 rejected.
 *   alpha_rows [rows] device floats.
 *   codes      [rows][cols/2];  scales [rows][cols/16];  choice NULL or
 *              [rows][cols/16].
 *   Shapes: cols % 16 == 0.  No workspace.
 *   Domain, per row: a row whose largest magnitude (after RHT16) is not
 *   zero but below 2^-64 (e.g. a row of bf16 subnormals) is outside the
 *   method's domain, as a whole tensor with that amax would be: its codes,
 *   scales and choice are unspecified (its alpha_rows entry is still
 *   amax_r / (6*C)).  The other rows are unaffected and the call never
 *   faults. */
int nvfp4_quantize_rows(const uint16_t* x, int64_t rows, int64_t cols,
                        uint32_t flags, uint64_t seed, float* alpha_rows,
                        uint8_t* codes, uint8_t* scales, uint8_t* choice,
                        void* stream);

/* Requantization of a 1D NVFP4 tensor for the transposed operand: the
 * NVFP4 quantization of dequantize(X)^T, with its own tensor scale.  The
 * backward pass quantizes data a second time (Quartet II / MS-EDEN
 * article, sec. 2); the weight gradient contracts over the other
 * dimension, so its operand needs blocks along the other axis (NVIDIA
 * NVFP4 article, sec. 7).  Dequantization is q * (alpha * Delta) in fp32
 * (NVIDIA NVFP4 article, sec. 6); the result equals nvfp4_quantize applied
 * to that fp32 transpose ("Four Over Six" Eq. 1-3), bit for bit.
 *   codes, scales, alpha  the input as a 1D nvfp4_quantize writes it:
 *             codes [rows][cols/2], scales [rows][cols/16] (finite E4M3
 *             codes; the sign bit is ignored, 0x7F is outside the domain),
 *             alpha one device float.
 *   flags     FP4_RTN6 or FOUR_OVER_SIX, SR, RHT16, as for a 1D
 *             nvfp4_quantize (SR|FOUR_OVER_SIX rejected); BLOCK2D, COLWISE,
 *             ROWWISE and HAD32 rejected.
 *   seed      Philox key: SR counter = element index in the output
 *             (out_row * rows + out_col); RHT16 signs as nvfp4_quantize.
 *             The rotation runs along output rows.
 *   amax_in   NULL: the output's largest magnitude (after RHT16 when
 *             asked) is computed here (one extra read of the input, needs
 *             `ws`); else one device float taken as that magnitude.
 *   alpha_out one device float: the output's tensor scale.
 *   codes_t   [cols][rows/2];  scales_t [cols][rows/16];
 *   choice_t  NULL or [cols][rows/16], 1 where the block took M = 4.
 *   ws        fp4_workspace_bytes(rows, cols, flags) bytes (device), or
 *             NULL with amax_in.
 *   Shapes: rows % 16 == 0 and cols % 16 == 0. */
int nvfp4_requantize_t(const uint8_t* codes, const uint8_t* scales, const float* alpha,
                       int64_t rows, int64_t cols, uint32_t flags, uint64_t seed,
                       const float* amax_in, float* alpha_out, uint8_t* codes_t,
                       uint8_t* scales_t, uint8_t* choice_t, void* ws, size_t ws_bytes,
                       void* stream);

/* MXFP4 quantization (NVIDIA NVFP4 article sec. 1 and 5; AMD MI355X MXFP4
 * article sec. 2).  Per 32 values: optional 32-point Hadamard (FP4_HAD32,
 * orthonormal), exponent e = floor(log2(amax)) - 2 (UE8M0 code e + 127,
 * 0 for an all-zero group), values scaled by 2^-e and rounded to nearest
 * even E2M1, saturating at 6.
 *   flags     HAD32 optional; ROWWISE and/or COLWISE (at least one).
 *   codes_r   [rows][cols/2], scales_r [rows][cols/32]   (ROWWISE, cols % 32 == 0)
 *   codes_c   [cols][rows/2], scales_c [cols][rows/32]   (COLWISE, rows % 32 == 0):
 *             the row-wise quantization of the transpose; the rotation and
 *             the 32-value groups run down the columns.
 *   Shapes: cols % 8 == 0 always (16-byte rows), plus the multiples above.
 *   Unused outputs may be NULL. */
int mxfp4_quantize(const uint16_t* x, int64_t rows, int64_t cols,
                   uint32_t flags, uint8_t* codes_r, uint8_t* scales_r,
                   uint8_t* codes_c, uint8_t* scales_c, void* stream);

/* MXFP4 matrix product C = A B, the consumer of the quantized tensors
 * (NVIDIA NVFP4 article sec. 1 and 5: MXFP4, E2M1 values with a UE8M0
 * scale per 32, multiplied directly by block-scaled matrix hardware; AMD
 * MI355X MXFP4 article sec. 2: training with both operands in MXFP4), on
 * gfx950's block-scaled FP4 matrix instructions with fp32 accumulation.
 *   a_codes [M][K/2], a_scales [M][K/32]   A in the row-wise MXFP4 layout
 *                                          (mxfp4_quantize ROWWISE of A)
 *   bt_codes [N][K/2], bt_scales [N][K/32] B^T in the same layout (the
 *                                          COLWISE output of mxfp4_quantize
 *                                          applied to B [K][N])
 *   c  [M][N] fp32, row-major.
 *   With HAD32 on both operands the rotations along K cancel in the product
 *   (the 32-point Hadamard is orthonormal), up to rounding.
 *   Shapes: K % 128 == 0, K < 2^23, N < 2^20, M*N < 2^40; M, N >= 0.  Code
 *   buffers 16-byte aligned, scale buffers and c 4-byte aligned. */
int mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* bt_codes,
               const uint8_t* bt_scales, int64_t M, int64_t N, int64_t K, float* c,
               void* stream);

/* Dequantize to fp32 [rows][cols] (the decode applied by the consumer:
 * NVIDIA NVFP4 article sec. 4 and sec. 6).
 *   format FP4_FORMAT_NVFP4: out = q * (alpha * Delta), alpha = *alpha
 *          (device float); flags FP4_BLOCK2D selects 16x16 tiles.
 *   format FP4_FORMAT_MXFP4: out = q * 2^(code-127); alpha ignored (may be
 *          NULL); pass (cols, rows) of the original to decode COLWISE output.
 *   out    16-byte aligned. */
int fp4_dequantize(int format, const uint8_t* codes, const uint8_t* scales,
                   const float* alpha, int64_t rows, int64_t cols,
                   uint32_t flags, float* out, void* stream);

/* ------------------------------------------------------------------------
 * Attention over a paged FP4 key/value cache, and the norm with rotation
 * that makes its queries and keys.
 *
 * Queries, keys, values, their outputs and gradients are bf16
 * [tokens][heads][head_dim]: a token's heads are contiguous, `*_stride` is
 * the number of elements from one token to the next (a multiple of 8, at
 * least heads * head_dim), so slices of a fused projection need no copy.
 * Pointers are 16-byte aligned.  The structs are read by the call itself and
 * need not outlive it.
 * ------------------------------------------------------------------------ */

/* A paged cache of keys and values in FP4, in the caller's memory.  With
 * page size P, G = 16 (NVFP4) or 32 (MXFP4):
 *   k_codes  [pages][heads][P][head_dim/2]   two codes per byte, even low
 *   k_scales [pages][heads][P][head_dim/G]
 *   v_codes  [pages][heads][head_dim/2][P]   the same bytes, tokens innermost
 *   v_scales [pages][heads][head_dim/G][P]
 * Slot s is token s % P of page s / P.  Every head is quantized along
 * head_dim as nvfp4_quantize (flags FP4_RTN6 or FP4_FOUR_OVER_SIX, the
 * head's largest magnitude given as amax_in) or mxfp4_quantize would;
 * magnitudes past the given one saturate.  The sign bit of an E4M3 scale is
 * ignored.  An infinity is stored as the largest value, a NaN as some finite
 * one, so either reaches only the tokens that see it.  In a program's own bytes
 * the E4M3 code 0x7F and UE8M0 codes above 252 are outside the domain. */
typedef struct {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  const float* k_amax;   /* [heads] device floats, NVFP4 only (else NULL)     */
  const float* v_amax;
  int64_t pages;
  int32_t page_size;     /* a power of two, 16 to 4096                        */
  int32_t heads;
  int32_t head_dim;      /* 64, 128 or 256                                    */
  int32_t format;        /* FP4_FORMAT_NVFP4 or FP4_FORMAT_MXFP4              */
  uint32_t flags;        /* NVFP4: FP4_RTN6 or FP4_FOUR_OVER_SIX; MXFP4: 0    */
} fp4_kv_cache;

/* Quantize the keys and values of `tokens` tokens into the cache at `slots`
 * [tokens] (int64).  A slot outside the cache is skipped; slots of one call
 * are distinct (of equal ones an unspecified mixture is kept). */
int fp4_kv_write(const fp4_kv_cache* cache, const uint16_t* k, int64_t k_stride,
                 const uint16_t* v, int64_t v_stride, const int64_t* slots, int64_t tokens,
                 void* stream);

/* Read the keys and values at `slots` back: q * (alpha * Delta), or
 * q * 2^(code-127), rounded to bf16.  A slot outside the cache reads as 0. */
int fp4_kv_read(const fp4_kv_cache* cache, const int64_t* slots, int64_t tokens, uint16_t* k,
                int64_t k_stride, uint16_t* v, int64_t v_stride, void* stream);

/* New tokens that attend over the cache.  Token i of a sequence's n stands
 * at position kv_len - n + i (its own key is already in the cache) and sees
 * the positions up to its own, with a window W the last W of them.  Position
 * j of sequence b is token j % P of page page_table[b][j / P]. */
typedef struct {
  const uint16_t* q;           /* [tokens][q_heads][head_dim]                 */
  int64_t q_stride;
  int64_t tokens;              /* new tokens of all sequences                 */
  int64_t seqs;
  const int32_t* cu_q;         /* [seqs + 1] first token of each sequence and
                                  the end of the last, none less than the one
                                  before; tokens before cu_q[0] and from
                                  cu_q[seqs] on (a padded batch) belong to no
                                  sequence.  NULL: one token each             */
  int64_t max_q;               /* at least every sequence's number of new
                                  tokens; 0: not known                        */
  const int32_t* kv_lens;      /* [seqs] cached tokens, the new ones included */
  const int32_t* page_table;   /* [seqs][table_width]                         */
  int64_t table_width;
  int32_t q_heads;             /* a multiple of the cache's heads; query head
                                  h reads kv head h / (q_heads / heads)       */
  int32_t window;              /* 0: none                                     */
  float scale;                 /* of the scores, usually head_dim^-1/2        */
  float softcap;               /* c > 0: scores become c tanh(s / c), off by
                                  16 u of themselves and, up to c = 64, 8 u c
                                  (u = 2^-24); 0: none                        */
} fp4_kv_queries;

/* Device workspace of fp4_kv_attention for these sizes (needs no
 * initialisation; may be 0). */
size_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache* cache, const fp4_kv_queries* x);

/* out = softmax(scores) V over the cached tokens that each new token sees,
 * bf16 [tokens][q_heads][head_dim]; lse NULL or [tokens][q_heads] floats,
 * the log of the sum of the scores' exponentials.  A token that sees
 * nothing (kv_len 0, fewer cached tokens than new ones, or no sequence) gets
 * out = 0 and lse = -inf.  Cached bytes past a sequence's length are never looked at,
 * whatever they hold; a page id outside the cache contributes nothing; a
 * length past the table is cut to it.  out may not overlap q; tokens times
 * q_heads, and sequences times q_heads, stay below 2^31.  Equal calls give
 * equal bits. */
int fp4_kv_attention(const fp4_kv_cache* cache, const fp4_kv_queries* x, uint16_t* out,
                     int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream);

enum { FP4_ROPE_INTERLEAVED = 1u << 0 };   /* pairs (2i, 2i+1) instead of (i, i + rot/2) */

/* Queries and keys for the norm with rotation.  Per head of a token at
 * position p:  y = R_p (x / sqrt(mean(x^2) + eps) * weight), R_p rotating
 * pair i of the first rot_dim values by the angle whose cosine and sine are
 * table[p][i]; the other values pass. */
typedef struct {
  const uint16_t* q;           /* [tokens][q_heads][head_dim]; NULL with q_heads 0 */
  const uint16_t* k;           /* [tokens][k_heads][head_dim]; NULL with k_heads 0 */
  int64_t q_stride, k_stride;
  int64_t tokens;
  const uint16_t* q_weight;    /* [head_dim] bf16; NULL: no norm of the queries */
  const uint16_t* k_weight;
  const int64_t* positions;    /* [tokens], in [0, table_rows)                */
  const float* table;          /* [table_rows][rot_dim/2][2]: cosine, sine
                                  (neither is looked at with rot_dim 0)       */
  int64_t table_rows;
  int32_t q_heads, k_heads;
  int32_t head_dim;            /* a multiple of 8, 16 to 256                  */
  int32_t rot_dim;             /* a multiple of 16, at most head_dim          */
  float eps;
  uint32_t flags;              /* FP4_ROPE_INTERLEAVED or 0                   */
} fp4_qk_rope;

/* Forward.  q_out may be q and k_out may be k (with the same strides).
 * Positions outside the table take its nearest row. */
int qk_norm_rope(const fp4_qk_rope* x, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                 int64_t k_out_stride, void* stream);

/* Bytes of device workspace of the backward pass (no initialisation). */
size_t qk_norm_rope_workspace_bytes(int head_dim);

/* Backward: from the gradients of the outputs (dq_out, dk_out) and the
 * forward's inputs, the gradients of q, k (bf16) and of the weights (fp32
 * [head_dim], NULL where not wanted; summed over tokens and heads in an
 * order that depends on the sizes alone).  ws may be NULL without weight
 * gradients.  dq may be dq_out and dk may be dk_out. */
int qk_norm_rope_backward(const fp4_qk_rope* x, const uint16_t* dq_out, int64_t dq_out_stride,
                          const uint16_t* dk_out, int64_t dk_out_stride, uint16_t* dq,
                          int64_t dq_stride, uint16_t* dk, int64_t dk_stride, float* dq_weight,
                          float* dk_weight, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The feed-forward half of a layer: products with FP4 weights, routing to
 * experts, the routed experts, and the norms around a block.
 *
 * Activations are bf16 [tokens][cols]; `*_stride` is the number of elements
 * from one row to the next, at least the row's length and (but for the
 * outputs of fp4_linear) a multiple of 8; that of x in fp4_linear and
 * fp4_experts is below 2^23.  Pointers are 16-byte aligned where
 * nothing else is said.  The structs are read by the call itself and need not
 * outlive it.
 * ------------------------------------------------------------------------ */

enum { FP4_ROW_ALPHA = 1u << 8 };   /* fp4_weights: an alpha for every row */

/* FP4 weights, one matrix [rows][cols] or one for each expert, as
 * nvfp4_quantize (FP4_RTN6, FP4_FOUR_OVER_SIX, also FP4_BLOCK2D),
 * nvfp4_quantize_rows or mxfp4_quantize (FP4_ROWWISE, no FP4_HAD32) lay them
 * out, G = 16 (NVFP4) or 32 (MXFP4):
 *   codes  [experts][rows][cols/2]
 *   scales [experts][rows][cols/G], with FP4_BLOCK2D [experts][rows/16][cols/16]
 *   alpha  NVFP4 only (else NULL): [experts], with FP4_ROW_ALPHA [experts][rows]
 * A weight is q * Delta * alpha, or q * 2^(code-127).  The sign bit of an E4M3
 * scale is ignored; the E4M3 code 0x7F and UE8M0 codes above 252 are outside
 * the domain, and MXFP4 weights below 2^-126 may count as 0. */
typedef struct {
  const uint8_t* codes;
  const uint8_t* scales;       /* 2-byte aligned                              */
  const float* alpha;          /* 4-byte aligned                              */
  int64_t experts;             /* 1 for a plain matrix                        */
  int64_t rows, cols;          /* below 2^24 and 2^22; cols a multiple of 32,
                                  rows of 16 with FP4_BLOCK2D; experts x rows
                                  x cols at most 2^40                         */
  int32_t format;              /* FP4_FORMAT_NVFP4 or FP4_FORMAT_MXFP4        */
  uint32_t flags;              /* NVFP4: FP4_BLOCK2D, FP4_ROW_ALPHA; MXFP4: 0 */
} fp4_weights;

/* Device workspace of fp4_linear (no initialisation; may be 0). */
size_t fp4_linear_workspace_bytes(const fp4_weights* w, int64_t tokens);

/* out[t][n] = sum_k x[t][k] w[n][k] for one matrix (experts 1).  The products
 * of x with q * Delta (or q * 2^k) are exact, their sums fp32, and alpha is
 * applied to the sum.  out is bf16, or fp32 with out_f32, aligned to its
 * elements, out_stride any number from rows on.  out may not overlap x.  Equal
 * calls give equal bits. */
int fp4_linear(const fp4_weights* w, const uint16_t* x, int64_t x_stride, int64_t tokens,
               void* out, int64_t out_stride, int out_f32, void* ws, size_t ws_bytes, void* stream);

/* The experts of each token.  With logits l [tokens][experts] and s = softmax(l)
 * or sigmoid(l) over a token's experts, the candidates' order is by
 *   c = l, or with a bias  c = s + bias  (computed in 64 bits).
 * Experts whose logit or c is -inf or NaN are no candidates.  With groups G > 1
 * (experts / G consecutive experts each) only the candidates of the top_groups
 * groups of largest size stay; a group's size is its largest c, or with
 * group_top 2 the sum of its two largest s (+ bias) among candidates.  The top_k
 * candidates of largest c follow in that order (ties, of groups also: the lower
 * index first), each with
 *   weight = scale s_i, or with renormalize  scale s_i / sum of the chosen s
 * (a quotient in the range of fp32 where the scores leave it; sigmoids of
 * logits that are all below -708 give weights 0).
 * Places without a candidate get expert -1 and weight 0.  A NaN or +inf among
 * softmax's logits makes the weights of its chosen experts NaN; sizes of groups
 * that would be NaN count as equal. */
typedef struct {
  const void* logits;          /* fp32 or bf16, aligned to its elements       */
  int64_t stride;              /* elements between tokens, at least experts   */
  int64_t tokens;
  const float* bias;           /* [experts] or NULL                           */
  int32_t experts, top_k;      /* 1 to 1024; 1 to 64 and at most experts      */
  int32_t groups, top_groups;  /* up to 64 groups, dividing the experts;
                                  top_groups of them hold top_k experts at
                                  least                                       */
  int32_t group_top;           /* 1 or 2                                      */
  int32_t sigmoid;             /* 0: softmax                                  */
  int32_t renormalize;
  int32_t logits_bf16;
  float scale;
} fp4_routing;

/* weights [tokens][top_k] fp32, experts [tokens][top_k]. */
int expert_route(const fp4_routing* r, float* weights, int32_t* experts, void* stream);

/* Gradient of the logits, in their type: from dweights [tokens][top_k] and the
 * experts that the forward chose (numbers outside [0, experts) count as no
 * expert).  The choice and the bias have no gradient: bias, groups, top_groups
 * and group_top are not looked at. */
int expert_route_backward(const fp4_routing* r, const float* dweights, const int32_t* experts,
                          void* dlogits, int64_t dlogits_stride, void* stream);

/* Device workspace of fp4_experts (no initialisation). */
size_t fp4_experts_workspace_bytes(const fp4_weights* gate_up, const fp4_weights* down,
                                   int64_t tokens, int64_t top_k);

/* out[t] = sum_j weights[t][j] D_e (silu(G_e x[t]) * (U_e x[t])), e =
 * experts[t][j]: gate_up holds G_e (rows 0 .. F - 1) and U_e (rows F .. 2F - 1)
 * [experts][2F][cols], down D_e [experts][cols][F].  The hidden values are
 * rounded to bf16 between the products, sums and the rest are fp32.  Numbers
 * outside [0, experts) are skipped; a token without an expert gets 0; an expert
 * named twice counts twice.  Up to 1024 experts, 64 a token.  out may not
 * overlap x.  Equal calls give equal bits. */
int fp4_experts(const fp4_weights* gate_up, const fp4_weights* down, const uint16_t* x,
                int64_t x_stride, int64_t tokens, const float* weights, const int32_t* experts,
                int64_t top_k, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes,
                void* stream);

/* The end of one block and the start of the next:
 *   n = block / sqrt(mean(block^2) + eps) * block_weight  (or block without it)
 *   y = scale x + gate n,   z = y / sqrt(mean(y^2) + eps) * weight
 * with a gate for every channel, one for every token, or none (1). */
typedef struct {
  const uint16_t* x;           /* [tokens][dim] bf16: the residual stream     */
  const uint16_t* block;       /* [tokens][dim] bf16: the block's output      */
  int64_t x_stride, block_stride;
  int64_t tokens;
  const uint16_t* block_weight;/* [dim] bf16 or NULL: no norm of the block    */
  const uint16_t* weight;      /* [dim] bf16                                  */
  const uint16_t* gate;        /* bf16 [dim] or, with token_gate, [tokens]
                                  (2-byte aligned); NULL: none                */
  int32_t token_gate;
  int32_t dim;                 /* a multiple of 8, 8 to 16384                 */
  float scale, eps;
} fp4_residual;

/* Forward: y and z bf16 [tokens][dim].  y may be x and z may be block (with the
 * same strides). */
int residual_norm(const fp4_residual* a, uint16_t* y, int64_t y_stride, uint16_t* z,
                  int64_t z_stride, void* stream);

/* Device workspace of residual_norm_backward (no initialisation). */
size_t residual_norm_workspace_bytes(int64_t tokens, int dim);

/* Backward: from the gradients of y and z and the forward's inputs, those of x
 * and block (bf16), and where wanted (else NULL) of block_weight, weight (fp32
 * [dim]) and gate (fp32, shaped as gate), summed in an order that depends on
 * the sizes alone.  dx may be dy and dblock may be dz. */
int residual_norm_backward(const fp4_residual* a, const uint16_t* dy, int64_t dy_stride,
                           const uint16_t* dz, int64_t dz_stride, uint16_t* dx, int64_t dx_stride,
                           uint16_t* dblock, int64_t dblock_stride, float* dblock_weight,
                           float* dweight, float* dgate, void* ws, size_t ws_bytes, void* stream);

/* Static description of a status code. */
const char* fp4_status_str(int status);

/* Interface version (bumped on any incompatible change). */
int fp4_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FP4Q_H */
