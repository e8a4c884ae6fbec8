/*
 * prism.h -- C ABI of the exact, batch-invariant int8 linear layer for
 * MI355X (gfx950).
 *
 * The operation (StartLux-Prism README): "Why StartLux-Prism" says that the
 * int8 GEMMs sum exactly in int32, so that a request gets the same result
 * whatever it is batched with, and that Q8_0 weights run as int8 (W8A8)
 * while Q4_K_M weights run on their own 4-bit values (W4A8); "How it works"
 * repeats that the int8 tensor-core path sums exactly in int32; "Quick
 * start" says the activations are quantized to int8 with measured ranges.
 * The pages fix neither the activation scale nor the epilogue; the readings
 * taken here are stated at each call below.
 *
 * Conventions shared by every call:
 *   - Every pointer argument is a DEVICE pointer (HBM of the current HIP
 *     device).  The caller allocates and owns all buffers; the library keeps
 *     no pointer after the call returns and allocates nothing (the calls
 *     that need scratch memory take it as an argument).
 *   - Except where a row stride is an argument, matrices are dense and
 *     row-major with no padding: x, q are [M][K],
 *     w is [N][K], w4 is [N][K/2], d is [N][K/32], y and acc are [M][N],
 *     partials is [M][N][K/32].
 *   - x, q, w and w4 must be 16-byte aligned; every other pointer must be
 *     aligned to its element size.
 *   - Work is enqueued on `stream` (a hipStream_t; 0 = the null stream) and
 *     the call returns without synchronizing.  Results are ready when the
 *     stream reaches that point.
 *   - M = 0 is a successful no-op that touches no memory.
 *   - Arguments are validated before any HIP call; an invalid call returns a
 *     negative status, enqueues nothing and writes nothing.
 *   - Results are a pure function of the inputs: they do not depend on M,
 *     on a row's position in the batch, on the stream or on concurrency.
 *     Calls hold no global state except per-device caches of the device's
 *     architecture and compute-unit count, and may be made from several
 *     threads at once.
 */
#ifndef PRISM_H
#define PRISM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Bumped on any change of a signature or of the semantics below. */
#define PRISM_ABI_VERSION 17

/* Largest accepted K.  For K <= 131040 every exact sum of K products of two
 * int8 values (|q|, |w| <= 128) lies strictly inside the int32 range. */
#define PRISM_K_MAX 131040

/* Element types of the fp8 and read-out calls' wider operands. */
#define PRISM_TYPE_F32 0
#define PRISM_TYPE_F16 1  /* IEEE binary16 */
#define PRISM_TYPE_BF16 2 /* bfloat16 */

/* Largest number of top alternatives of prism_token_logprobs. */
#define PRISM_TOP_MAX 32

/* Largest K of the norms, and largest number of experts and of rows of a
 * routed batch. */
#define PRISM_NORM_K_MAX 65536
#define PRISM_EXPERTS_MAX 1024
#define PRISM_ROUTE_M_MAX 16777216

/* What a router's weights are made from (prism_route_experts). */
#define PRISM_SCORE_SOFTMAX 0
#define PRISM_SCORE_SIGMOID 1

/* Status codes. */
#define PRISM_OK 0
#define PRISM_ERR_INVALID_ARG (-1) /* null required pointer, negative size, N or K = 0 with M > 0, K > PRISM_K_MAX or another of the limits, unknown type, row stride below the row, workspace too small, a size whose launch would have 2^32 threads or more */
#define PRISM_ERR_ALIGNMENT (-2)   /* misaligned pointer, or K not a multiple of 16 (32 for block-scale and W4A8, 256 for Q4_K) */
#define PRISM_ERR_UNSUPPORTED (-3) /* the current device is not gfx950, or no device is usable */
#define PRISM_ERR_LAUNCH (-4)      /* the kernel launch reported an error */

/* Returns PRISM_ABI_VERSION of the built library. */
int prism_abi_version(void);

/* Identity of the sources the library was built from: 32 hex digits of the
 * sha256 of its HIP/C++ sources, this header and its compile flags (static
 * string, never NULL).  A binding can compare it with the sources it ships
 * with and refuse a library built from others. */
const char* prism_build_id(void);

/* Static, human-readable text for a status code (never NULL). */
const char* prism_status_string(int status);

/*
 * Per-row int8 activation quantizer (README "Quick start": int8 activation
 * ranges; the per-row absmax form is the reading taken here).
 *   x      [M][K] fp32, input.
 *   q      [M][K] int8, output.
 *   scale  [M] fp32, output.
 * For each row m: a = max_k |x[m][k]|; scale[m] = a / 127 (IEEE division,
 * round to nearest even); q[m][k] = clamp(rint(x[m][k] / scale[m]), -127, 127)
 * with rint rounding half to even.  A row holding a NaN or an infinity gets
 * scale NaN and q = 0; a row whose scale is 0 (all zeros, or a subnormal
 * amax that underflows) gets q = 0.  Rows never influence each other.
 * K must be a multiple of 16.
 */
int prism_quantize_rows(const float* x, int8_t* q, float* scale,
                        int64_t M, int64_t K, void* stream);

/*
 * Int8 activation quantizer with one static, calibrated scale for the whole
 * tensor (README "Quick start": the int8 activation ranges are measured once
 * ahead of time, not per batch).
 *   x      [M][K] fp32, input.
 *   q      [M][K] int8, output.
 *   scale  [M] fp32, output: the row scales to hand to the GEMM calls.
 *   s      the calibrated scale, a host value; must be finite and > 0
 *          (otherwise PRISM_ERR_INVALID_ARG and nothing is enqueued).
 * For each row m without a NaN: scale[m] = s and q[m][k] = clamp(rint(x[m][k]
 * / s), -127, 127) (IEEE division, rint half to even), so values beyond the
 * calibrated range saturate at +-127, an infinite x included.  A row holding
 * a NaN gets scale NaN and q = 0.  Rows never influence each other.
 * K must be a multiple of 16; x and q 16-byte aligned, scale 4-byte aligned.
 */
int prism_quantize_rows_static(const float* x, int8_t* q, float* scale, float s,
                               int64_t M, int64_t K, void* stream);

/*
 * Q8_0 weight blocks -> the (w, d) planes of prism_gemm_w8a8_blockscale
 * (README "Why StartLux-Prism": released Q8_0 files run as int8 W8A8 with no
 * conversion step).  The block layout is the public GGUF one, not given by
 * the pages: 34 bytes per block, a little-endian binary16 scale followed by
 * the 32 int8 codes of k = 32 b .. 32 b + 31 of weight row n; blocks are
 * stored row by row, block n * (K/32) + b.
 *   blocks [N * K/32][34] bytes, input (16-byte aligned).
 *   w      [N][K] int8, output: the codes (16-byte aligned).
 *   d      [N][K/32] binary16 bit patterns, output: the scales (2-byte aligned).
 * Pure byte movement: every output equals an input byte pair or byte.
 * K must be a positive multiple of 32; N = 0 is a no-op.
 */
int prism_repack_q8_0(const uint8_t* blocks, int8_t* w, uint16_t* d,
                      int64_t N, int64_t K, void* stream);

/*
 * Q4_K weight super-blocks -> the planes of prism_gemm_w4a8_q4k (README "Why
 * StartLux-Prism": released Q4_K_M files run on their own 4-bit values).  The
 * super-block layout is the public GGUF one, not given by the pages: 144
 * bytes per 256 consecutive weights of one row: binary16 d and dmin
 * (little-endian), 12 bytes of 6-bit sub-block scales sc_j and mins m_j
 * (j < 4: sc_j = s[j] & 63, m_j = s[j+4] & 63; j >= 4: sc_j = (s[j+4] & 15) |
 * (s[j-4] >> 6) << 4, m_j = (s[j+4] >> 4) | (s[j] >> 6) << 4), then 128 bytes of
 * codes (byte 32 g + l: weight 64 g + l in the low nibble, 64 g + 32 + l in
 * the high one).  Weight = d * sc_j * code - dmin * m_j.
 *   blocks [N * K/256][144] bytes, input (16-byte aligned).
 *   w4     [N][K/2] bytes, output: the 128 code bytes of each super-block, in
 *          the file's own order (super-block t of row n at bytes 128 t ..
 *          128 t + 127 of row n); still 4 bits per weight (16-byte aligned).
 *   hdr    [N][K/256][16] bytes, output: the 16 leading bytes of each
 *          super-block (d, dmin, the 12 scale bytes) (16-byte aligned).
 * Pure byte movement: the two planes hold every byte of the blocks once.
 * K must be a positive multiple of 256; N = 0 is a no-op.
 */
int prism_repack_q4_k(const uint8_t* blocks, uint8_t* w4, uint8_t* hdr,
                      int64_t N, int64_t K, void* stream);

/*
 * W4A8 on Q4_K weights (the planes of prism_repack_q4_k).
 *   q [M][K] int8, s_a [M] fp32, w4 [N][K/2] packed codes, hdr [N][K/256][16].
 *   y [M][N] fp32 output.
 * For sub-block b (32 k) of super-block t = b / 8, j = b % 8: D = d * sc_j and
 * Mn = dmin * m_j from the super-block's header (both exact in fp32);
 * P_b = sum q[m][k] * code[n][k] and S_b = sum q[m][k], both exact integers;
 * f = +0; for b ascending: f = fmaf((float)P_b, D, f); f = fmaf(-(float)S_b,
 * Mn, f); then y[m][n] = f * s_a[m].
 * K must be a multiple of 256; q, w4 and hdr 16-byte aligned.
 */
int prism_gemm_w4a8_q4k(const int8_t* q, const float* s_a, const uint8_t* w4, const uint8_t* hdr,
                        float* y, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * W8A8 GEMM with per-output-channel weight scales (README "Why
 * StartLux-Prism": Q8_0 weights as int8 W8A8, summed exactly in int32).
 *   q    [M][K] int8 activations, s_a [M] fp32 row scales.
 *   w    [N][K] int8 weights (one row per output channel), s_w [N] fp32.
 *   y    [M][N] fp32 output.
 *   acc  [M][N] int32 output, or NULL.
 * acc[m][n] = sum_k q[m][k] * w[n][k], exact in int32;
 * y[m][n]   = ((float)acc[m][n] * s_a[m]) * s_w[n], each product rounded
 * to nearest even on its own, in that order.  K must be a multiple of 16.
 */
int prism_gemm_w8a8(const int8_t* q, const float* s_a, const int8_t* w, const float* s_w,
                    float* y, int32_t* acc, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * W8A8 GEMM with one fp16 weight scale per 32 consecutive k of each weight
 * row (Q8_0-style blocks; README "Why StartLux-Prism", released Q8_0 files).
 *   q [M][K] int8, s_a [M] fp32, w [N][K] int8.
 *   d [N][K/32] binary16 bit patterns: the scale of block b of row n.
 *   y [M][N] fp32 output.
 *   partials [M][N][K/32] int32 output, or NULL (meant for small debug sizes).
 * P_b = sum_{32b <= k < 32b+32} q[m][k] * w[n][k] (exact int32);
 * f = +0; for b = 0, 1, ..., K/32-1 in that order: f = fmaf((float)P_b,
 * (float)d[n][b], f); y[m][n] = f * s_a[m].  K must be a multiple of 32.
 */
int prism_gemm_w8a8_blockscale(const int8_t* q, const float* s_a, const int8_t* w,
                               const uint16_t* d, float* y, int32_t* partials,
                               int64_t M, int64_t N, int64_t K, void* stream);

/*
 * Quantize + W8A8 GEMM in one call (the README's "Quick start" int8
 * activations feeding the exact int32 GEMM of "Why StartLux-Prism").
 *   x     [M][K] fp32 activations (16-byte aligned).
 *   q     [M][K] int8 and scale [M] fp32 outputs: what prism_quantize_rows
 *         writes for x.
 *   w, s_w, y, acc: as for prism_gemm_w8a8 (acc may be NULL).
 * The results are those of prism_quantize_rows(x) followed by
 * prism_gemm_w8a8 on its outputs, bit for bit.  With M = 1 and K <= 16384,
 * and with M = 2, 3 or 4 rows, N <= 16384 and K up to 14336, 10240 or 6144
 * respectively, this is one kernel in which every workgroup quantizes the
 * rows on chip while its first weight rows stream in (decode); otherwise
 * the two steps run as two launches on `stream`.  Either way it allocates
 * nothing.  K must be a multiple of 16.
 */
int prism_quantize_gemm_w8a8(const float* x, int8_t* q, float* scale, const int8_t* w, const float* s_w,
                             float* y, int32_t* acc, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * W4A8 GEMM on packed signed 4-bit weights (README "Why StartLux-Prism":
 * Q4_K_M files run on their own 4-bit weights with int8 activations; the
 * symmetric per-channel form is the reading taken here).
 *   q [M][K] int8, s_a [M] fp32.
 *   w4 [N][K/2] bytes: byte j of row n holds w[n][2j] in its low nibble and
 *      w[n][2j+1] in its high nibble, each a two's-complement value in [-8, 7].
 *   s_w [N] fp32, y [M][N] fp32, acc [M][N] int32 or NULL.
 * acc and y as for prism_gemm_w8a8 with w decoded from the nibbles.
 * K must be a multiple of 32.
 */
int prism_gemm_w4a8(const int8_t* q, const float* s_a, const uint8_t* w4, const float* s_w,
                    float* y, int32_t* acc, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * The shape-dependent kernel choice of prism_gemm_w8a8 / prism_gemm_w4a8,
 * one entry at a time (README "Why StartLux-Prism": kernels are picked per
 * GPU from measured tables; that is safe here because every entry computes
 * the same exact int32 sums and the same per-element epilogue).  These calls
 * exist to verify that claim: the result of every applicable variant is bit
 * for bit the result of PRISM_VARIANT_AUTO, which is what the plain calls run.
 * Same arguments and checks as the plain calls, plus `variant`:
 *   PRISM_VARIANT_AUTO            the plain call's choice;
 *   PRISM_VARIANT_SMALL_<c>x<w>   the small-M kernel with c column blocks of
 *                                 16 (c = 1..4) and w waves per workgroup
 *                                 (M <= 64 only);
 *   PRISM_VARIANT_SMALL_BALANCED  the small-M kernel with one even share of
 *                                 the N columns per CU (M <= 64, N <= 16384);
 *   PRISM_VARIANT_TILE_*          the LDS-tiled kernels: 256x128, 192x128
 *                                 and 128x96 (int8 weights only), 256x192,
 *                                 256x256, 256x320, 128x128 and 64x128, and
 *                                 128x128 or 64x128 with K split over 2, 3 or
 *                                 4 workgroups, 128x96 over 2, whose exact
 *                                 int32 partials are added atomically into y.
 * A variant that does not apply to the call returns PRISM_ERR_INVALID_ARG.
 */
#define PRISM_VARIANT_AUTO 0
#define PRISM_VARIANT_SMALL_1x4 1
#define PRISM_VARIANT_SMALL_1x8 2
#define PRISM_VARIANT_SMALL_1x16 3
#define PRISM_VARIANT_SMALL_2x4 4
#define PRISM_VARIANT_SMALL_2x8 5
#define PRISM_VARIANT_SMALL_2x16 6
#define PRISM_VARIANT_TILE_256x256 7
#define PRISM_VARIANT_TILE_256x128 8
#define PRISM_VARIANT_TILE_128x128 9
#define PRISM_VARIANT_TILE_128x128_SPLIT2 10
#define PRISM_VARIANT_TILE_128x128_SPLIT3 11
#define PRISM_VARIANT_TILE_128x128_SPLIT4 12
#define PRISM_VARIANT_SMALL_3x4 13
#define PRISM_VARIANT_SMALL_3x8 14
#define PRISM_VARIANT_SMALL_4x4 15
#define PRISM_VARIANT_SMALL_4x8 16
#define PRISM_VARIANT_TILE_256x192 17
#define PRISM_VARIANT_TILE_256x320 18
#define PRISM_VARIANT_TILE_64x128 19
#define PRISM_VARIANT_TILE_64x128_SPLIT2 20
#define PRISM_VARIANT_TILE_64x128_SPLIT3 21
#define PRISM_VARIANT_TILE_64x128_SPLIT4 22
#define PRISM_VARIANT_TILE_128x96 23
#define PRISM_VARIANT_TILE_128x96_SPLIT2 24
#define PRISM_VARIANT_SMALL_BALANCED 25
#define PRISM_VARIANT_TILE_192x128 26
#define PRISM_VARIANT_COUNT 27

int prism_gemm_w8a8_variant(const int8_t* q, const float* s_a, const int8_t* w, const float* s_w,
                            float* y, int32_t* acc, int64_t M, int64_t N, int64_t K, int variant,
                            void* stream);
int prism_gemm_w4a8_variant(const int8_t* q, const float* s_a, const uint8_t* w4, const float* s_w,
                            float* y, int32_t* acc, int64_t M, int64_t N, int64_t K, int variant,
                            void* stream);

/*
 * ---- 8-bit floating point: e4m3 codes with one scale per 128 values ----
 *
 * The 8-bit floating point form of the same layer (StartLux-Prism README, "Why
 * StartLux-Prism": quantized weights and activations, a row's result
 * independent of its batch; the pages keep 8-bit floats to the KV cache and
 * give no layout, so the one below is this library's reading).  Codes are OCP
 * e4m3 bytes (largest value 448, no infinities, NaN 0x7f / 0xff).  KB =
 * ceil(K / 128) and NB = ceil(N / 128) count blocks; the last ones may be
 * partial.  x_type is the PRISM_TYPE_* of x.  x may have padded rows: row m
 * starts ld >= K elements after row m - 1, with the rows 16-byte aligned (x
 * 16-byte aligned, ld * element size a multiple of 16).  K must be a multiple
 * of 16 and at most PRISM_K_MAX; q and w are dense and 16-byte aligned.
 *
 * Codes of a group of values with largest magnitude a: s = a / 448 (IEEE
 * fp32 division); code = the e4m3 value nearest (ties to even) to x / s, the
 * correctly rounded fp32 quotient clamped to +-448.  s = 0 gives codes 0.  A
 * group holding a NaN or an infinity gets s = NaN and codes 0.  A zero code
 * may be 0x00 or 0x80.  Groups never influence each other.
 *
 * prism_quantize_blocks_fp8: activations, one group per 128 consecutive k of
 * a row.
 *   x      [M][K] of x_type, rows ld elements apart.
 *   q      [M][K] e4m3, output.
 *   scale  [KB][M] fp32, output: block-major, so that the rows of a tile find
 *          a block's scales in one piece.
 */
int prism_quantize_blocks_fp8(const void* x, int x_type, int64_t ld, uint8_t* q, float* scale,
                              int64_t M, int64_t K, void* stream);

/*
 * Weights (see above), one group per 128 x 128 tile.
 *   x      [N][K] of x_type, rows ld elements apart.
 *   q      [N][K] e4m3, output;  scale [NB][KB] fp32, output.
 * N = 0 is a no-op.
 */
int prism_quantize_tiles_fp8(const void* x, int x_type, int64_t ld, uint8_t* q, float* scale,
                             int64_t N, int64_t K, void* stream);

/*
 * SwiGLU and the activation quantizer behind it, in one pass: what stands
 * between the two products of a gated MLP.
 *   gate, up [M][K] of x_type, rows of both ld elements apart (the halves of
 *            one [M][2 K] product: up = gate + K, ld = 2 K).
 *   q, scale as prism_quantize_blocks_fp8 of h = gate / (1 + exp(-gate)) * up,
 *            computed in fp32.
 */
int prism_swiglu_quantize_fp8(const void* gate, const void* up, int x_type, int64_t ld, uint8_t* q, float* scale,
                              int64_t M, int64_t K, void* stream);

/*
 * GEMM on those codes and scales.
 *   q [M][K] e4m3, s_a [KB][M] fp32; w [N][K] e4m3, s_w [NB][KB] fp32.
 *   y [M][N] of y_type (PRISM_TYPE_*), output, aligned to its element size.
 * P_b = the sum of block b's products; f = +0; for b ascending f =
 * fmaf(P_b, s_a[b][m] * s_w[n / 128][b], f); y[m][n] = f, rounded once to
 * y_type.  With y_type fp32 or fp16 the products are exact and P_b is an fp32
 * sum; an fp16 y is the fp32 y rounded.  With y_type bf16 P_b is the matrix
 * cores' fp8 sum, which aligns each eight products of consecutive k to the
 * largest and cuts what lies 2^-13 below its exponent: products of one sign
 * lose at most 2^-10 of their sum, less than y's rounding; where products
 * cancel, the error can reach 2^-6 of the block's largest product.  Rows have
 * the same bits whatever M is (a bf16 y and the others are two functions).
 */
int prism_gemm_fp8_blockscale(const uint8_t* q, const float* s_a, const uint8_t* w, const float* s_w,
                              void* y, int y_type, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * Token read-out: log probabilities of given tokens, entropy and top
 * alternatives of each row of logits (README "Example": answers are read
 * from the probabilities of given tokens).
 *   logits [M][V] of `type`, rows ld >= V elements apart, aligned to their
 *          element size only (V may be odd).  A masked entry is -inf.
 *   tokens [M][T] int64, or NULL with T = 0.
 *   logprobs [M][T] fp32: z_t - log sum exp z; NaN for a token outside [0, V).
 *   lse, entropy [M] fp32, each may be NULL: log sum exp z, -sum p log p.
 *   top_ids [M][top] int64, top_logprobs [M][top] fp32 (0 <= top <=
 *          PRISM_TOP_MAX; NULL with top = 0): the largest logits, largest
 *          first, the lower index first among equals.  Slots past the last
 *          entry of nonzero probability hold -1 and -inf.
 *   workspace  prism_token_logprobs_workspace bytes (8-byte aligned; may be
 *          NULL if that is 0), free again when the stream passes the call.
 * All sums are fp32 in an order that depends on V and `type` only.  A row with every entry -inf:
 * logprobs and lse -inf, entropy 0.  A row with a NaN or +inf: all NaN, and
 * ids -1.
 */
int prism_token_logprobs_workspace(int64_t M, int64_t V, int top, int64_t* bytes);
int prism_token_logprobs(const void* logits, int type, int64_t ld, const int64_t* tokens, int64_t T, int top,
                         float* logprobs, float* lse, float* entropy, int64_t* top_ids, float* top_logprobs,
                         void* workspace, int64_t workspace_bytes, int64_t M, int64_t V, void* stream);

/*
 * ---- A mixture-of-experts layer on those codes ----
 *
 * The layer of a model whose MLP is a set of experts, in the order of its
 * calls: norm (fp8), the router's product (any GEMM), prism_route_experts,
 * prism_gemm_fp8_grouped on the rows that the routing lists, prism_swiglu_
 * quantize_fp8, prism_gemm_fp8_grouped, prism_combine_experts.  The method's
 * pages name no such model; what they ask of a layer holds for it too: 8-bit
 * products, and a row's result independent of its batch (StartLux-Prism README,
 * "Why StartLux-Prism").
 *
 * Root-mean-square norm with the residual's addition in front of it and an
 * 8-bit quantizer behind it:
 *   h = x + residual, the fp32 sum rounded to res_type (h = x where residual
 *       is NULL);
 *   inv = 1 / sqrt(sum_k h^2 / K + eps), in 64 bits and rounded once to fp32;
 *   y = (h * inv) * gain, each product rounded to fp32;
 *   q, scale: the codes and scales of y.  fp8: as prism_quantize_blocks_fp8
 *       writes them for y in fp32.  Rows (int8): scale[m] = max_k |y| * fp32(1 /
 *       127), one product, so within one step of prism_quantize_rows's quotient;
 *       codes as there, clamp(rint(y / scale[m]), -127, 127).
 *   x        [M][K] of x_type, rows x_ld elements apart.
 *   residual [M][K] of res_type, rows res_ld apart, or NULL.  res_type is
 *            x_type or PRISM_TYPE_F32 (not looked at where residual is NULL).
 *   residual_out [M][K] of res_type, rows out_ld apart, output: h.  May be
 *            NULL, or residual itself with out_ld = res_ld; NULL where residual
 *            is.
 *   gain     [K] of gain_type.
 *   norm     [M][K] of x_type, output: y rounded; may be NULL.
 *   q        [M][K], output; scale [KB][M] (fp8) or [M] (int8), output.
 *   eps      a host value, finite and >= 0.
 * K must be a multiple of 16 and at most PRISM_NORM_K_MAX; every row of x,
 * residual and residual_out, and gain, norm and q, 16-byte aligned.  Outputs
 * overlap no input but as said.  A NaN in a row makes all its y NaN.  Rows
 * never influence each other.
 */
int prism_add_rmsnorm_quantize_fp8(const void* x, int x_type, int64_t x_ld, const void* residual, int64_t res_ld,
                                   void* residual_out, int64_t out_ld, int res_type, const void* gain, int gain_type,
                                   double eps, void* norm, uint8_t* q, float* scale, int64_t M, int64_t K,
                                   void* stream);
int prism_add_rmsnorm_quantize_rows(const void* x, int x_type, int64_t x_ld, const void* residual, int64_t res_ld,
                                    void* residual_out, int64_t out_ld, int res_type, const void* gain, int gain_type,
                                    double eps, void* norm, int8_t* q, float* scale, int64_t M, int64_t K,
                                    void* stream);

/*
 * Routing: each token's experts and their weights, and the rows of each expert.
 *   logits [M][E] of `type`, rows ld >= E elements apart, aligned to their
 *          element size only.  An expert closed to a token is -inf.
 *   bias   [E] fp32, added to the score for the choice only, or NULL.  An expert
 *          whose bias is -inf or NaN is chosen by no token.
 *   score  PRISM_SCORE_SOFTMAX: softmax over the E logits; PRISM_SCORE_SIGMOID.
 *   top    experts of a token, 1 to PRISM_TOP_MAX and at most E.
 *   ids     [M][top] int32, output: the experts of largest key, largest first,
 *           the lower index first among equals.  The key is the logit, with a
 *           bias the score plus the bias, computed in 64 bits.  -1 where no open
 *           expert is left.
 *   weights [M][top] fp32, output: the chosen experts' scores, with
 *           `renormalize` divided by their sum (0 where that is 0), times `scale`;
 *           0 beside -1.
 *   offsets [E + 1] int32, output: expert e has the rows offsets[e] ..
 *           offsets[e + 1] - 1 of a list of all choices, sorted by expert.
 *   rows    [M * top] int32, output: the token of each row of the list, ascending
 *           within an expert; -1 behind the list's end, offsets[E].
 *   slots   [M][top] int32, output: each choice's row in the list, or -1.
 *   workspace  prism_route_experts_workspace bytes (8-byte aligned; may be NULL
 *           if that is 0), free again when the stream passes the call.
 * A token with a NaN or +inf logit: ids and slots -1, weights NaN.  M up to
 * PRISM_ROUTE_M_MAX, E up to PRISM_EXPERTS_MAX, M * top up to 2^31 - 1.
 */
int prism_route_experts_workspace(int64_t M, int64_t E, int64_t* bytes);
int prism_route_experts(const void* logits, int type, int64_t ld, const float* bias, int score, int renormalize,
                        float scale, int top, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                        int32_t* slots, void* workspace, int64_t workspace_bytes, int64_t M, int64_t E, void* stream);

/*
 * GEMM grouped by expert, the groups ragged and known on the device only.
 *   q, s_a  [M][K] e4m3 and [KB][M] fp32, as of prism_quantize_blocks_fp8.
 *   rows    [R] int32 device values: row i of y is made from row rows[i] of q;
 *           or NULL: from row i, with M = R.  A row outside [0, M) counts as zeros.
 *   offsets [E + 1] int32 device values, not descending: rows offsets[e] ..
 *           offsets[e + 1] - 1 of y belong to expert e.
 *   w, s_w  [E][N][K] e4m3 and [E][NB][KB] fp32: each expert's as of
 *           prism_quantize_tiles_fp8.
 *   y       [R][N] of y_type, output, aligned to its element size.  Rows in
 *           front of offsets[0] and from offsets[E] on are left as they are.
 * Row by row the bits of prism_gemm_fp8_blockscale with that expert's weights: with
 * y_type fp32 or fp16 from exact products, with bf16 from the matrix cores' fp8
 * sums, whose error can reach 2^-6 of a block's largest product where products
 * cancel, as said there.
 * Offsets are taken as clamped to 0 .. R; where they descend, what is written
 * of y is not specified (nothing else is).  E up to PRISM_EXPERTS_MAX, R up to
 * 2^31 - 257; with rows, M * K below 2^31.
 */
int prism_gemm_fp8_grouped(const uint8_t* q, const float* s_a, const int32_t* rows, const int32_t* offsets,
                           const uint8_t* w, const float* s_w, void* y, int y_type, int64_t M, int64_t R, int64_t E,
                           int64_t N, int64_t K, void* stream);

/*
 * Which of its kernels such a call runs (all give the same bits), for tests and
 * profiles; a host function, no device is looked at.  Negative status codes for
 * sizes that the call refuses.
 *   PRISM_GROUPED_FEW     16 x 16 tiles, of fp32 and fp16 outputs
 *   PRISM_GROUPED_<r>x<c> LDS tiles of r rows and c columns (64x128: of bf16 only)
 *   PRISM_GROUPED_WIDE    up to 256 rows by 256 columns, of bf16 outputs
 */
#define PRISM_GROUPED_FEW 0
#define PRISM_GROUPED_64x64 1
#define PRISM_GROUPED_64x128 2
#define PRISM_GROUPED_128x128 3
#define PRISM_GROUPED_WIDE 4
int prism_gemm_fp8_grouped_form(int y_type, int64_t R, int64_t E, int64_t N, int64_t K);

/*
 * A token's expert outputs added up with its weights.
 *   x       [R][N] of x_type, aligned to its element size.
 *   weights [M][top] fp32, slots [M][top] int32: as of prism_route_experts; a
 *           slot outside [0, R) counts as a row of zeros.
 *   add     [M][N] of y_type, or NULL: what the sum starts from.
 *   y       [M][N] of y_type, output: x_type or PRISM_TYPE_F32; may be add itself.
 * f = add (or +0); for j ascending f = fmaf(weights[m][j], x[slots[m][j]], f);
 * y = f rounded.  top from 1 to PRISM_TOP_MAX.
 */
int prism_combine_experts(const void* x, int x_type, const float* weights, const int32_t* slots, const void* add,
                          void* y, int y_type, int64_t R, int64_t M, int64_t top, int64_t N, void* stream);

/*
 * Measurement kernels (not part of the GEMM path): what this GPU reaches on
 * the two resources the GEMMs are bound by, for the roofline figures.
 *
 * prism_peak_mfma: 2 x (compute units) workgroups, each of 2 x
 * waves_per_simd waves (waves_per_simd in {1, 2, 4}), every wave running
 * iters x 16 v_mfma_i32_32x32x32_i8 on register operands: iters x 16 x 65536
 * integer ops per wave.  out [2 x CUs x 128 x waves_per_simd] uint32 gets
 * one checksum per thread: the sum modulo 2^32 of the thread's NACC x 16
 * accumulator registers after 16 / NACC steps per iteration on NACC
 * accumulators (NACC = 8, or 4 for waves_per_simd = 4) that alternate the
 * operand pairs (A0, B0) and (A1, B1).  Byte j (0..15) of the fragment of
 * operand s (A0, B0, A1, B1 = 0, 1, 2, 3) in lane l is the top byte of
 * (37 l + 101 j + 7919 s + 13 seed) * 2654435761 modulo 2^32, as int8.
 * iters in [1, 2^24], seed in [0, 2^20]; accumulators wrap past 2^31 for
 * large iters (the checksum is then only a data dependence).
 *
 * prism_peak_read: reads `bytes` (a multiple of 16, at most 2^40) of `buf`
 * (16-byte aligned) once with 16-byte loads and writes the XOR of the
 * 32-bit words each workgroup read to parts[workgroup]; all
 * PRISM_PEAK_READ_PARTS entries of parts are written (unused ones 0), so the
 * XOR of parts is the XOR of every 32-bit word of the buffer.
 *
 * prism_peak_fold: the cost of the block-scale fold (an exact sum per 32-k
 * block of a 32 x 32 output tile, then one fp32 fmaf per output,
 * StartLux-Prism README, "Why StartLux-Prism": Q8_0 weights as W8A8) on
 * registers only.  One workgroup of 8 waves per compute unit; each wave
 * holds 5 tiles and gives each one 32-k block per iteration.  mode 0: int8
 * MFMA from zero, convert, fold; 1: two f16 MFMAs on the same values (the
 * sum exact in fp32, no convert), fold; 2: the int8 MFMAs only
 * (accumulating); 3: the f16 MFMA pairs only (accumulating); 4: the folds
 * only.  out [CUs x 512] float gets one sum per thread.  Modes 0 and 1
 * write the same bits; so do modes 2 and 3 for iters <= 32.  iters in [1,
 * 2^20].
 */
#define PRISM_PEAK_READ_PARTS 4096
int prism_peak_mfma(int64_t iters, int waves_per_simd, int seed, uint32_t* out, void* stream);
int prism_peak_read(const void* buf, int64_t bytes, uint32_t* parts, void* stream);
int prism_peak_fold(int mode, int64_t iters, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PRISM_H */
