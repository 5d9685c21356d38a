/*
 * bsgemm.h -- C ABI of libbsgemm, the MI355X (gfx950) hot path of a
 * row-parallel block-scale fp8 linear layer (DeepSeek-V4-Pro's wo_b):
 *
 *   bsgemm_fp8   block-scale fp8 GEMM, fp32 accumulate, bf16 out, written as
 *                destination-major row bands
 *   band_reduce  fp32 sum of P bf16 partial bands into one bf16 band
 *   rowq_e4m3    per-row e4m3 quantize with one fp32 scale per row
 *   band_rowq_e4m3  band_reduce and rowq_e4m3 fused into one pass (the fused
 *                variant the pages measured and found slower; here it is the
 *                faster path and the one the benchmark's step runs)
 *   rowdq_e4m3   per-row e4m3 dequantize back to bf16
 *   blockq_e4m3  fp32 operand -> e4m3 codes + fp32 block scales (the
 *                activation/weight quantizer that produces bsgemm_fp8's input)
 *   actq_e4m3    bf16 activation -> e4m3 codes + fp32 1x128 scales (the
 *                on-GPU step before bsgemm_fp8 when the layer input is bf16)
 *   bprepack_e4m3  one-time rearrangement of the weight B into the GEMM's
 *                operand order (load-time weight preparation)
 *   bsgemm_fp8_pb  the GEMM reading B in that prepacked form
 *   mxgemm_fp8   the mxfp8 variant of the GEMM: e4m3 operands with E8M0 scales
 *                per 1x32 block on both A and B, applied by the MFMA
 *   mxq_e4m3     bf16 -> e4m3 codes + E8M0 1x32 scales (mxgemm_fp8's operands)
 *
 * and what stands around that layer in a serving stack:
 *
 *   lora_plan    orders a batch's rows by the low-rank adapter each one uses
 *   lora_shrink  H[m] = x[m] A[a]^T, the first low-rank product of every row
 *   lora_expand  out[m] = base[m] + scale[a] (H[m] B[a]^T), the second one added
 *                to a finished row-banded output
 *   bsgemm_fp8_lora  bsgemm_fp8 with the second product added to its fp32
 *                accumulators, so C is written once
 *   resnorm      norm after a block, gate, scaled residual, norm before the
 *                next block and its e4m3 operand, in one pass; takes the
 *                gathered fp8 wire or a bf16 output
 *
 * and the feed-forward block that reads resnorm's operand:
 *
 *   bsgemm_fp8_act  bsgemm_fp8 with bias, activation (gated or not) and residual
 *                in its epilogue
 *   moe_route    each token's experts and their weights, from the router's logits
 *   moe_fp8      the experts of a few tokens: both products, the gated activation
 *                and the weighted sum, in two or three kernels
 *
 * Pages defining the operations (cited by title and section):
 *   [PR40757] sglang PR 40757 "[AMD][gfx950] DSV4: fuse wo_b's GEMM with its
 *             all-reduce via mori cco": "What" (block-scale fp8 GEMM followed
 *             by an all-reduce of [M, hidden]; each destination's row band
 *             written as its own unit), "Numbers" (fused and unfused agree up
 *             to accumulation order).
 *   [PR43480] sglang PR 43480 (DeepSeek-V4.1-Flash wo_b): "What" (an mxfp8
 *             GEMM followed by the all-reduce), "Not in this PR" (V4.1-Flash
 *             quantises at 32-wide ue8m0), "Numerics, measured where the path
 *             engages" (on the aiter route wo_b is handed a plain bf16
 *             activation and quantises it itself); "Worth a reviewer's
 *             attention" (the native gfx950 route rebinds the weight to a
 *             shuffled [N/16, K/128, 2048] layout, and reading one layout as
 *             the other gives an uncorrelated result instead of an error);
 *             the review reply on the duplicated ue8m0 scale rule (exponent
 *             from the IEEE bits, exact at powers of two) and the one on the
 *             lazy second copy of the weight (weight preparation moved to
 *             load time).
 *   [MORI]    "MORI GEMM + All-Reduce Benchmark": "Running the benchmark"
 *             (--quant blockscale: A per 1x128, B per 128x128, fp32 scales;
 *             shape [M,7168], K=2048), "Where the time goes" (reduce /
 *             quantize / dequantize phases), "The fp8 wire" (e4m3 with one
 *             fp32 scale per row; the reduce accumulates in fp32 and outputs
 *             bf16), "Negative results" (the pages keep reduce and quantize
 *             as separate kernels; band_rowq_e4m3 fuses them).
 *
 * Conventions shared by every call:
 *  - All data pointers are DEVICE memory owned by the caller (the library
 *    never allocates, frees or keeps a pointer after returning).  The only
 *    host memory argument is band_reduce's array of part pointers, read
 *    before the call returns.
 *  - bf16 values are passed as their uint16_t bit patterns; e4m3 values as
 *    uint8_t codes of the OCP FP8 E4M3 ("fn") format (max 448, NaN at
 *    S.1111.111, no infinities).  Every matrix is dense row-major.
 *  - stream is a hipStream_t passed as void* (NULL = the null stream).  Calls
 *    only enqueue work: they return before the device finishes and never
 *    synchronize.
 *  - Arguments are validated on the host before anything is enqueued.  On
 *    BS_ERR_INVALID or BS_ERR_UNSUPPORTED nothing is launched and no output
 *    byte is written.  BS_ERR_LAUNCH means the HIP runtime refused the launch
 *    (hipGetLastError after the enqueue); outputs are then unspecified.
 *  - Results are bitwise deterministic for identical inputs and shapes.
 *  - The library holds no global state that calls depend on, reads no
 *    environment variables and is safe to call from several host threads.
 *    Calls whose output ranges overlap another call's input or output on a
 *    concurrently running stream race, as with any kernel.
 */
#ifndef BSGEMM_H
#define BSGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BS_OK = 0,
    BS_ERR_INVALID = 1,     /* null pointer, negative size, aliasing outputs */
    BS_ERR_UNSUPPORTED = 2, /* well-formed but not expressible by the kernels */
    BS_ERR_LAUNCH = 3       /* the HIP runtime rejected the launch */
} bs_status;

/*
 * Block-scale fp8 GEMM with a destination-major band epilogue.
 * [PR40757] "What"; [MORI] "Running the benchmark" (--quant blockscale).
 *
 *   C[m, n] = bf16_rne( acc[m, n] ),  acc accumulated in fp32 over the K
 *   blocks kb = 0 .. K/128-1 in ascending order:
 *     acc += ( sum_{k in block kb} A[m,k] * B[n,k] ) * (a_scale[m,kb] * b_scale[n/128,kb])
 *   the block dot product being one 16x16x128 fp8 MFMA with fp32 result.
 *
 *   A        [M, K]          e4m3 codes (activations)
 *   a_scale  [M, K/128]      fp32, one scale per 1x128 block of A
 *   B        [N, K]          e4m3 codes (the weight as stored, [out, in])
 *   b_scale  [N/128, K/128]  fp32, one scale per 128x128 block of B
 *   C        bf16 output as `bands` row bands of band_rows = M / bands rows:
 *            row m lives in band d = m / band_rows at row r = m % band_rows,
 *            element (m, n) at C[d * band_stride + r * N + n].
 *            band_stride = 0 means band_rows * N (contiguous: identical to a
 *            row-major [M, N] matrix).  Elements between bands are untouched.
 *
 * Requirements: M >= 0 (M = 0 is a no-op); N > 0 and N % 128 == 0;
 * K > 0 and K % 128 == 0; 1 <= bands <= 64 and M % bands == 0;
 * band_stride == 0 or band_stride >= band_rows * N; A, B and C 16-byte
 * aligned, a_scale and b_scale 4-byte aligned; C must not overlap any input;
 * K <= 2^22, M and N below 2^31, and at most 2^23 - 8 tiles of 256 x 256.
 * Violations: null pointers, negative sizes, bands < 1 or overlap ->
 * BS_ERR_INVALID; the rest -> BS_ERR_UNSUPPORTED.  M need not be a multiple
 * of the tile: ragged rows are handled in the kernel.
 */
bs_status bsgemm_fp8(const uint8_t *A, const float *a_scale,
                     const uint8_t *B, const float *b_scale,
                     uint16_t *C,
                     int64_t M, int64_t N, int64_t K,
                     int32_t bands, int64_t band_stride,
                     void *stream);

/*
 * Band reduce: out = bf16_rne( sum_{p=0..P-1} widen(parts[p]) ), the sum in
 * fp32 starting from +0.0 and taken in part-index order.
 * [MORI] "Where the time goes" (reduce), "The fp8 wire" (fp32 accumulate,
 * bf16 output), "Negative results" (one pass streams all P source slices).
 *
 *   parts  HOST array of P device pointers, each a bf16 [rows, N] band
 *   out    bf16 [rows, N]; may not overlap any part
 *
 * Requirements: 1 <= P <= 16; rows >= 0, N > 0, N % 8 == 0; every pointer
 * 16-byte aligned.  Null or out-of-range P -> BS_ERR_INVALID; N % 8 or
 * misalignment -> BS_ERR_UNSUPPORTED.
 */
bs_status band_reduce(const uint16_t *const *parts, int32_t P,
                      uint16_t *out, int64_t rows, int64_t N,
                      void *stream);

/*
 * Per-row e4m3 quantize (the "fp8 wire").  [MORI] "The fp8 wire" (e4m3 with
 * one fp32 scale per row), "What fp8 costs, numerically" (per row chosen).
 *
 *   for each row r:  amax = max_n |x[r,n]|;  scale[r] = amax / 448 (fp32,
 *   round to nearest even);  q[r,n] = e4m3 code nearest to the fp32 quotient
 *   x[r,n] / scale[r] (ties to even, |.| > 448 saturates, sign kept so a
 *   negative value that rounds to zero gives 0x80).  A row whose scale is 0
 *   (all zeros, or amax/448 underflowing) gets scale 0 and codes 0x00.
 *
 *   x      bf16 [rows, N] (finite values; non-finite input is outside the
 *          contract and gives unspecified codes)
 *   q      e4m3 [rows, N]
 *   scale  fp32 [rows]
 *
 * Requirements: rows >= 0, N > 0, N % 8 == 0; x, q 16-byte aligned, scale
 * 4-byte aligned; q and scale must not overlap x or each other.
 */
bs_status rowq_e4m3(const uint16_t *x, uint8_t *q, float *scale,
                    int64_t rows, int64_t N, void *stream);

/*
 * Per-row e4m3 dequantize ("widen" after the gather).  [MORI] "Where the
 * time goes" (dequantize), "Who moves the gather".
 *
 *   y[r,n] = bf16_rne( fp32(decode(q[r,n])) * scale[r] )   (one fp32 multiply)
 *
 *   q      e4m3 [rows, N] (NaN codes 0x7F/0xFF are never produced by
 *          rowq_e4m3 and are outside the contract)
 *   scale  fp32 [rows]
 *   y      bf16 [rows, N]
 *
 * Requirements: rows >= 0, N > 0, N % 8 == 0; q, y 16-byte aligned, scale
 * 4-byte aligned; y must not overlap q or scale.
 */
bs_status rowdq_e4m3(const uint8_t *q, const float *scale, uint16_t *y,
                     int64_t rows, int64_t N, void *stream);

/*
 * Block quantizer for GEMM operands.  [MORI] "Running the benchmark"
 * (--quant blockscale: activations per 1x128 block, weights per 128x128
 * block, fp32 scales).  For each block of block_rows x 128 elements:
 * amax = max |x|; s = amax / 448 (fp32); codes = e4m3 of the fp32 quotient
 * x / s exactly as rowq_e4m3 (zero scale -> codes 0x00).
 *
 *   x      fp32 [rows, cols] (finite)
 *   q      e4m3 [rows, cols]
 *   scale  fp32 [ceil(rows/block_rows), cols/128]
 *
 * Requirements: block_rows is 1 or 128; rows >= 0; cols > 0, cols % 128 ==
 * 0; x, q 16-byte aligned; scale 4-byte aligned; no output overlaps x.
 */
bs_status blockq_e4m3(const float *x, uint8_t *q, float *scale,
                      int64_t rows, int64_t cols, int32_t block_rows,
                      void *stream);

/*
 * Activation quantizer: the bf16 layer input of bsgemm_fp8 quantised on the
 * GPU, as the layer does when it is handed a plain bf16 tensor ([PR43480]
 * "Numerics, measured where the path engages"), at the activation
 * granularity of [MORI] "Running the benchmark" (1x128 blocks, fp32 scales).
 * For each block of 128 consecutive elements of a row: amax = max |x|;
 * s = amax / 448 (fp32); codes = e4m3 of the fp32 quotient x / s exactly as
 * rowq_e4m3 (zero scale -> codes 0x00).  Identical to blockq_e4m3 with
 * block_rows = 1 on the fp32 values of x (every bf16 value is an fp32 value).
 *
 *   x      bf16 [rows, cols] (finite)
 *   q      e4m3 [rows, cols]
 *   scale  fp32 [rows, cols/128]
 *
 * Requirements: rows >= 0; cols > 0, cols % 128 == 0; x, q 16-byte aligned;
 * scale 4-byte aligned; no output overlaps x or the other output.
 */
bs_status actq_e4m3(const uint16_t *x, uint8_t *q, float *scale,
                    int64_t rows, int64_t cols, void *stream);

/*
 * Prepacks the weight B for bsgemm_fp8_pb: a one-time rearrangement done when
 * the weight is loaded ([PR43480], the review reply on the lazy second copy
 * of the weight; [PR40757] "What": the fused path serves only a weight that
 * was preshuffled at load).  Bp holds the same N*K bytes as B in the order
 * the GEMM's MFMA consumes them:
 *
 *   Bp[((nt * (K/128) + kb) * 2 + h) * 1024 + (16 g + r) * 16 + e]
 *       = B[brow(16 nt + r), 128 kb + 16 g + 64 h + e],
 *   brow(64 b + 16 j + r) = 64 b + 32 (j/2) + 8 (r/4) + 4 (j%2) + r%4
 *
 * for 16-row group nt, K block kb, half h in {0,1}, g in [0,4), r in [0,16),
 * e in [0,16): each 2 KiB block is one 16-row x 128 tile of B, laid out as
 * the 64 lanes' operand bytes, its rows taken within each 64-row group in the
 * order the GEMM's epilogue needs (brow).  The layout is a contract between this call and
 * bsgemm_fp8_pb only; nothing infers it from a shape ([PR43480] "Worth a
 * reviewer's attention": one layout read as the other gives garbage, not an
 * error).
 *
 *   B   e4m3 [N, K] row-major (the weight as stored, [out, in])
 *   Bp  e4m3, N*K bytes, prepacked (caller-owned, written here)
 *
 * Requirements: N > 0, N % 128 == 0; K > 0, K % 128 == 0, K <= 2^22; B and Bp
 * 16-byte aligned and not overlapping (no in-place prepack).
 */
bs_status bprepack_e4m3(const uint8_t *B, uint8_t *Bp, int64_t N, int64_t K,
                        void *stream);

/*
 * bsgemm_fp8 with the weight in the prepacked form bprepack_e4m3 writes: the
 * same operation, arguments, requirements, errors and results (bit for bit)
 * as bsgemm_fp8, except that B is replaced by Bp.  The kernel loads each
 * wave's B operands straight from Bp into registers (fully coalesced 1 KiB
 * loads), so B takes no LDS staging; A and the scales are staged as in
 * bsgemm_fp8.  Passing an unpacked B here (or Bp to bsgemm_fp8) is not
 * detected and gives a wrong result.
 */
bs_status bsgemm_fp8_pb(const uint8_t *A, const float *a_scale,
                        const uint8_t *Bp, const float *b_scale,
                        uint16_t *C, int64_t M, int64_t N, int64_t K,
                        int32_t bands, int64_t band_stride, void *stream);

/*
 * mxfp8 GEMM, the variant of [PR43480] "What" / "Not in this PR": C = A * B^T
 * with A [M,K] e4m3 and a_scale [M, K/32] E8M0 bytes (one per 1x32 block of
 * a row; value 2^(byte - 127)), B [N,K] e4m3 and b_scale [N, K/32] E8M0
 * bytes, fp32 accumulation, bf16 output, written in the same destination-major
 * bands as bsgemm_fp8 (bands, band_stride as there).  The block scales are
 * applied by gfx950's scaled MFMA; the sum is accumulated over K in fp32 in
 * the instruction's own order, so results are compared with the exact product
 * at a relL2 tolerance.
 *
 * Requirements: M >= 0; N > 0, N % 128 == 0; K > 0, K % 128 == 0, K <= 2^22;
 * bands in [1, 64] dividing M; band_stride 0 or >= (M/bands)*N and a multiple
 * of 8; A, B, C 16-byte aligned; a_scale, b_scale 4-byte aligned; C must not
 * overlap an input; M and N below 2^31, and at most 2^23 - 8 tiles of 256 x 256.
 */
bs_status mxgemm_fp8(const uint8_t *A, const uint8_t *a_scale,
                     const uint8_t *B, const uint8_t *b_scale,
                     uint16_t *C, int64_t M, int64_t N, int64_t K,
                     int32_t bands, int64_t band_stride, void *stream);

/*
 * mxfp8 operand quantizer ([PR43480] "Not in this PR": 32-wide ue8m0; the
 * review reply on the ue8m0 scale rule: exponent from the IEEE bits, exact at
 * powers of two).  For each block of 32 consecutive elements of a row:
 * amax = max |x|; the scale is 2^k with k the smallest integer such that
 * amax <= 448 * 2^k (clamped below at -127); scale byte = k + 127; codes =
 * e4m3 round-to-nearest-even of x * 2^-k (never saturating).  A zero block
 * gets scale byte 0 and codes 0x00.
 *
 *   x      bf16 [rows, cols] (finite)
 *   q      e4m3 [rows, cols]
 *   scale  E8M0 bytes [rows, cols/32]
 *
 * Requirements: rows >= 0; cols > 0, cols % 32 == 0; x, q 16-byte aligned; no
 * output overlaps x or the other output.
 */
bs_status mxq_e4m3(const uint16_t *x, uint8_t *q, uint8_t *scale,
                   int64_t rows, int64_t cols, void *stream);

/*
 * band_reduce followed by rowq_e4m3, fused into one kernel that never writes
 * the bf16 band: q, scale = rowq_e4m3(band_reduce(parts)), bit for bit (the
 * fp32 part-order sum is rounded to bf16 before the row quantizer sees it).
 * [MORI] "Negative results" reports that fusing the reduce with the quantize
 * was slower than the two separate kernels, because a row's amax needs the
 * whole row before any code can be written.  Here one workgroup takes each
 * row with several parts' loads in flight at once, and the fused pass moves
 * fewer bytes than the two kernels (the bf16 band is neither written nor
 * read back), so it is the faster of the two.
 *
 *   parts  host array of P device pointers, each bf16 [rows, N] (1 <= P <= 16)
 *   q      e4m3 [rows, N];  scale  fp32 [rows]
 *
 * Requirements: 0 <= rows < 2^31 (one workgroup per row); N > 0, N % 8 == 0,
 * N <= 8192; parts and q 16-byte aligned, scale 4-byte aligned; no output
 * overlaps a part or the other output.
 */
bs_status band_rowq_e4m3(const uint16_t *const *parts, int32_t P, uint8_t *q,
                         float *scale, int64_t rows, int64_t N, void *stream);

/*
 * Row order of a batch whose rows use different low-rank adapters.  ids[m] is
 * row m's adapter, in [0, n_adapters); any other value means that the row has
 * none.  With key(m) = ids[m], or n_adapters for a row without an adapter:
 *
 *   plan[a]  for a = 0 .. n_adapters + 1: the number of rows with key < a
 *            (so plan[n_adapters] rows have an adapter, and
 *            plan[n_adapters + 1] = M)
 *   plan[n_adapters + 2 + i], i = 0 .. M - 1: the rows ordered by key, rows of
 *            one key in ascending order
 *
 * One plan serves every layer that the batch passes through.
 *
 * Rows are apart in all of these calls: a value that is not finite, in a row or
 * in the adapter that it uses, makes that row's results non-finite, and no
 * other row's.
 *
 *   ids   int32 [M] (may be null when M = 0)
 *   plan  int32 [n_adapters + 2 + M]
 *
 * Requirements: 0 <= M < 2^30; 1 <= n_adapters <= 4096; 4-byte alignment; plan
 * must not overlap ids.  M = 0 writes n_adapters + 2 zeros.
 */
bs_status lora_plan(const int32_t *ids, int32_t *plan, int64_t M, int64_t n_adapters, void *stream);

/*
 * First low-rank product: H[m, r] = sum_k x[m, k] * A[a, r, k], a = row m's
 * adapter by the plan; H[m] = 0 for a row without one.  bf16 products summed
 * in fp32, and not rounded further: H is fp32.  Under row parallelism x and A
 * hold this GPU's part of K, and H is its partial sum: lora_expand and
 * bsgemm_fp8_lora add it to the same GPU's partial output, whose reduction then
 * completes both.
 *
 *   x     bf16 [M, K]
 *   A     bf16 [n_adapters, R, K] (an adapter of a smaller rank has zero rows)
 *   plan  as lora_plan writes it for these rows and n_adapters.  Entries that
 *         lie outside the batch are ignored, but no check finds that a plan
 *         belongs to another batch
 *   H     fp32 [M, R]
 *
 * Requirements: 0 <= M < 2^30; K > 0, K % 8 == 0, K <= 2^22; 1 <= n_adapters
 * <= 4096; R % 8 == 0, 8 <= R <= 256; x, A, H 16-byte aligned, plan 4-byte; H
 * must not overlap an input.
 */
bs_status lora_shrink(const uint16_t *x, const uint16_t *A, const int32_t *plan, float *H, int64_t M,
                      int64_t K, int64_t n_adapters, int64_t R, void *stream);

/*
 * Second low-rank product, added to a finished output:
 *
 *   out[m, n] = bf16_rne( base[m, n] + scale[a] * sum_r H[m, r] * B[a, n, r] )
 *
 * for a row with adapter a; out[m] = base[m] for one without.  The sum is fp32;
 * scale * H enters the products as two bf16 (17 bits of significand, within bf16's
 * largest value).  base and out are row-banded as bsgemm_fp8's C (bands,
 * band_stride as there); elements between bands are untouched.  out may be base
 * itself.
 *
 *   H      fp32 [M, R] (what rows without an adapter hold does not matter)
 *   B      bf16 [n_adapters, N, R]
 *   scale  fp32 [n_adapters] or null (1)
 *   plan   as for lora_shrink
 *   base   bf16 bands;  out  bf16 bands
 *
 * Requirements: as lora_shrink for M, n_adapters and R; N > 0, N % 8 == 0;
 * 1 <= bands <= 64 and M % bands == 0; band_stride 0 or >= (M / bands) * N and
 * a multiple of 8; H, B, base, out 16-byte aligned, scale and plan 4-byte; out
 * equals base or does not overlap it, and overlaps no other input.
 */
bs_status lora_expand(const float *H, const uint16_t *B, const float *scale, const int32_t *plan,
                      const uint16_t *base, uint16_t *out, int64_t M, int64_t N, int64_t n_adapters,
                      int64_t R, int32_t bands, int64_t band_stride, void *stream);

/*
 * bsgemm_fp8 with its rows' adapters: to the finished fp32 accumulator of row m
 * is added scale[a] * sum_r H[m, r] * lora_B[a, n, r], a = ids[m], before the one
 * rounding to bf16.  A row whose id is outside [0, n_adapters) gets bsgemm_fp8's
 * result, bit for bit, whatever its H holds.  This reads ids directly and needs no
 * plan.
 *
 * Its cost grows with the number of different adapters among 128 consecutive rows.
 * Prefer it to bsgemm_fp8 followed by lora_expand, which writes and reads C once
 * more, for up to a few hundred rows, and for longer batches in runs of rows that
 * share an adapter.  Of a longer batch whose rows mix more than about 8 adapters of
 * rank 16, 4 of rank 64 or 2 of rank 128, either put the rows in adapter order or make
 * the two calls.  N = 7168, K = 2048, us fused / two calls: 16384 rows, R = 64, in runs
 * 255 / 328; strewn over 4 adapters 331 / 336, 8: 413 / 338, 32: 733 / 341, 128: 1329 /
 * 348; R = 16 over 4: 269 / 312, 8: 312 / 315, 32: 412 / 316; R = 128 over 2: 347 / 373,
 * 4: 457 / 373; 1024 rows, R = 64, over 4: 39 / 39, 32: 86 / 57; 200 rows, R = 64, over
 * 4: 16 / 34, 128: 46 / 52.
 *
 *   A, a_scale, B, b_scale, C, bands, band_stride  as for bsgemm_fp8
 *   H           fp32 [M, R], from lora_shrink
 *   lora_B      bf16 [n_adapters, N, R]
 *   lora_scale  fp32 [n_adapters] or null (1)
 *   ids         int32 [M]
 *
 * Requirements: those of bsgemm_fp8, and of lora_expand for M, n_adapters, R and
 * the alignments; C must not overlap an input.
 */
bs_status bsgemm_fp8_lora(const uint8_t *A, const float *a_scale, const uint8_t *B,
                          const float *b_scale, const float *H, const uint16_t *lora_B,
                          const float *lora_scale, const int32_t *ids, uint16_t *C, int64_t M, int64_t N,
                          int64_t K, int64_t n_adapters, int64_t R, int32_t bands, int64_t band_stride,
                          void *stream);

/*
 * The step between two blocks, row by row, with rms(v) = sqrt(mean(v^2) + eps):
 *
 *   y = decode(y) * y_scale[row]        if y_scale is given (the fp8 wire, as
 *                                       rowdq_e4m3 but not rounded to bf16)
 *   p = y / rms(y) * post_w             if post_w is given, else p = y
 *   h = alpha * resid + beta * gate * p      (gate = 1 if null)
 *   resid_out = h, rounded to the residual's type
 *   z = h / rms(h) * pre_w              (pre_w = 1 if null)
 *   q = e4m3(z / s) with s in q_scale   if q_block is 128 (fp32 scale per 1x128
 *                                       block, s = amax / 448) or 32 (E8M0 scale
 *                                       per 1x32 block, as mxq_e4m3)
 *
 * All of it in fp32, each output rounded once: z and q come from the unrounded
 * h, and q from the unrounded z.  An all-zero scale block gets scale 0 (byte 0)
 * and codes 0x00.  A row's results do not depend on the other rows or their number.
 * What is not finite follows the formulas: a NaN or an infinity reaches its own row's
 * z, and a block of z with a NaN gets a NaN scale (byte 0xFF) and NaN codes; one with
 * an infinity gets a scale and codes that decode to NaN (fp32: the scale is infinite;
 * byte 0xFF and NaN codes).  Finite values of any size are normed, those too whose
 * squares are past fp32; only h itself has to lie within it.
 *
 *   y          bf16 [rows, N], or e4m3 [rows, N] with y_scale fp32 [rows]
 *   resid      bf16 [rows, N], or fp32 if resid_f32 is 1; resid_out the same
 *              type, and may be resid itself
 *   post_w, pre_w  bf16 [N] or null
 *   gate       bf16 [N] if gate_row is 0, [rows, N] if gate_row is N; or null
 *   z          bf16 [rows, N] or null
 *   q, q_scale e4m3 [rows, N] with fp32 [rows, N/128] or bytes [rows, N/32];
 *              both null if q_block is 0
 *
 * Requirements: 0 <= rows < 2^31; N > 0, N % 8 == 0 (N % q_block == 0 with
 * q), N <= 16384; eps > 0 and alpha, beta, eps finite; every pointer 16-byte
 * aligned but y_scale and q_scale (4-byte; E8M0 bytes any); outputs overlap
 * neither each other nor an input, except resid_out == resid.
 */
bs_status resnorm(const void *y, const float *y_scale, const void *resid, const uint16_t *post_w,
                  const uint16_t *gate, int64_t gate_row, const uint16_t *pre_w, void *resid_out,
                  uint16_t *z, uint8_t *q, void *q_scale, int64_t rows, int64_t N, int32_t resid_f32,
                  int32_t q_block, float alpha, float beta, float eps, void *stream);

/*
 * bsgemm_fp8 with bias, activation and residual in its epilogue, the products of a
 * feed-forward block.  With acc as in bsgemm_fp8:
 *
 *   t[m, n] = acc[m, n] + bias[n]
 *   v[m, n] = act(t[m, n])                  gated = 0: B [N, K]
 *   v[m, n] = act(t[m, n]) * t[m, N + n]    gated = 1: B [2N, K], the N gate rows first
 *   C[m, n] = bf16_rne( alpha * resid[m, n] + beta * v[m, n] )
 *
 * without the resid term if resid is null, all of it in fp32 and rounded once.  act
 * (bs_act): none, relu, silu t / (1 + e^-t), gelu t/2 erfc(-t / sqrt 2), gelu_tanh
 * t / (1 + e^-2u) with u = sqrt(2/pi) (t + 0.044715 t^3); within 2^-15 of their
 * values, and zero instead of a result below 2^-119.  What is not finite follows these
 * formulas (silu and both gelus of -infinity are NaN).  acc is bit for bit
 * bsgemm_fp8's in every batch, so with no bias, activation or residual and beta = 1 so
 * is C.
 *
 *   A, a_scale  as for bsgemm_fp8
 *   B, b_scale  e4m3 [N or 2N, K], fp32 [N/128 or 2N/128, K/128]
 *   bias        bf16 [N or 2N] or null
 *   resid       bf16, in bands as C (bands, band_stride), or null; may be C itself
 *   C           bf16 bands of M x N
 *
 * Requirements: those of bsgemm_fp8, with 2N for N where B's rows count; alpha and beta
 * finite; bias and resid 16-byte aligned; C must not overlap an input, except resid == C.
 */
typedef enum {
    BS_ACT_NONE = 0,
    BS_ACT_RELU = 1,
    BS_ACT_SILU = 2,
    BS_ACT_GELU = 3,
    BS_ACT_GELU_TANH = 4
} bs_act;

bs_status bsgemm_fp8_act(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale,
                         const uint16_t *bias, const uint16_t *resid, uint16_t *C, int64_t M, int64_t N,
                         int64_t K, int32_t act, int32_t gated, float alpha, float beta, int32_t bands,
                         int64_t band_stride, void *stream);

/*
 * Routing: each row's topk experts and their weights, from the router's logits.
 *
 *   s[e] = softmax(logits)[e] (score = 0) or 1 / (1 + e^-logits[e]) (score = 1)
 *   key[e] = s[e] + bias[e]; without bias and with one group, logits[e] itself
 *   groups > 1: a group is groups-th of the experts, in order; its score is the sum of
 *     its group_top (1 or 2) largest keys; the topk_groups groups of the largest
 *     scores are kept, and the others' experts are not chosen
 *   ids = the topk experts of the largest keys, in descending order
 *   weights[k] = scale * s[ids[k]], or, with renorm, scale * s[ids[k]] / sum of s[ids]
 *
 * The bias so takes part in the choice alone.  Keys, scores and sums are fp64 (which of
 * two close keys is larger does not go by fp32 roundings); weights are rounded
 * once.  Equal keys and scores: the lower number first.  An expert whose logit or bias
 * is -infinity or NaN is not chosen (nor one whose key is NaN); where fewer than
 * topk can be, the last slots get id -1 and weight 0.  (A NaN or +infinity among a row's
 * logits makes its softmax weights NaN.)  Where all chosen scores are 0, renorm leaves
 * 0.
 *
 *   logits   fp32 [rows, E], or bf16 if logits_bf16 is 1
 *   bias     fp32 [E] or null
 *   ids      int32 [rows, topk];  weights  fp32 [rows, topk]
 *
 * Requirements: rows >= 0, rows * E < 2^40; 1 <= E <= 1024; 1 <= topk <= 64, topk <= E;
 * 1 <= groups <= 64 and groups divides E; 1 <= topk_groups <= groups; scale finite;
 * logits, bias, ids, weights aligned to their elements; no output overlaps an input or
 * the other output.
 */
bs_status moe_route(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t rows, int64_t E,
                    int32_t topk, int32_t logits_bf16, int32_t score, int32_t groups, int32_t topk_groups,
                    int32_t group_top, int32_t renorm, float scale, void *stream);

/*
 * The experts of a few tokens.  An expert e has W1 and W3 [I, D], stacked in W13[e]
 * (W1's I rows first), and W2[e] [D, I]:
 *
 *   h[m, e] = act(W1[e] x[m]) * (W3[e] x[m])
 *   out[m] = bf16_rne( base[m] + sum_k weights[m, k] * (W2[e] h[m, e]) ),  e = ids[m, k]
 *
 * without base if it is null.  An id outside [0, E) means that the slot is empty (an
 * expert of another GPU, whose sum is added across GPUs); a row of empty slots is base,
 * or zero.  An expert named twice by a row counts once, with the sum of the two weights.
 * Weights are e4m3 values with 128 x 128 fp32 scales; x is not quantized, and h is
 * carried to 2^-17 (within bf16's largest value).  A row's result does not depend on the
 * other rows or their number, and a value that is not finite, in a row or in an expert
 * that it uses, reaches no other row.
 *
 * Two kernels, three where D is at most 4096 and E more than 2, bound by reading the
 * weights of the experts in use: W13[e] once for each 32 and W2[e] for each 16 of an
 * expert's tokens.
 *
 *   x        bf16 [M, D];  ids  int32 [M, topk];  weights  fp32 [M, topk]
 *   W13      e4m3 [E, 2I, D];  s13  fp32 [E, 2I/128, D/128]
 *   W2       e4m3 [E, D, I];   s2   fp32 [E, D/128, I/128]
 *   base     bf16 [M, D] or null;  out  bf16 [M, D], may be base itself
 *   ws       workspace of the bytes that moe_fp8_workspace gives, written and read by
 *            this call alone: calls that may run at the same time need one each
 *
 * Requirements: 0 <= M <= 128, 1 <= topk <= 64 and M * topk <= 1024; 1 <= E <= 1024; D and
 * I positive multiples of 128, at most 65536; x, W13, W2, base, out, ws 16-byte aligned,
 * the rest 4-byte; out and ws overlap neither each other nor an input, except out ==
 * base.
 */
bs_status moe_fp8(const uint16_t *x, const int32_t *ids, const float *weights, const uint8_t *W13, const float *s13,
                  const uint8_t *W2, const float *s2, const uint16_t *base, uint16_t *out, void *ws, int64_t M,
                  int64_t topk, int64_t E, int64_t D, int64_t I, int32_t act, void *stream);

/* The bytes of moe_fp8's workspace, for its limits on M, topk, E and I. */
bs_status moe_fp8_workspace(int64_t M, int64_t topk, int64_t E, int64_t I, int64_t *bytes);

/* Static, NUL-terminated description of a status code. */
const char *bs_status_str(bs_status status);

#ifdef __cplusplus
}
#endif

#endif /* BSGEMM_H */
