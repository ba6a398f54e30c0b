/*
 * mq.h -- C ABI of the MI355X (gfx950) MosaicQuant library.
 *
 * The library computes the ZipperEngine path of MosaicQuant ("MosaicQuant:
 * Inlier-Outlier Disaggregation for Unified 4-Bit LLM Quantization", technical
 * summary on gist.science): a weight matrix W^ [N][K] (out x in) is decomposed as
 * W^ ~ Q(W^) + R (Methodology 1), a dense 4-bit base plus a 4-bit residual kept
 * only for the top-K (bn x bk) blocks ranked by a Hessian-guided Delta-score
 * (Methodology 2), and Y = Xq Q(W^)^T + Xq R^T is computed by one fused kernel
 * that walks the residual blocks inside the dense 4-bit GEMM (Methodology 3).
 *
 * Conventions shared by every call
 *   - Every pointer argument is a DEVICE pointer (HBM), owned and allocated by the
 *     caller; the library keeps no reference after the call returns.
 *   - `stream` is a hipStream_t (NULL = the default stream). Calls are
 *     asynchronous on it unless stated otherwise.
 *   - Inputs are read-only. Outputs are fully overwritten. Inputs and outputs
 *     must not overlap.
 *   - int4 codes (values in [-7, 7]) are packed eight to a little-endian 32-bit
 *     word, inputs k0..k0+7 with k0 a multiple of 8: nibble e of the word (bits
 *     4e..4e+3) holds |c_e| in its low three bits and, in its high bit, the sign
 *     of code (e - 1) mod 8 (1 = negative; zero has no sign). With this encoding
 *     word & 0x87878787 and rotr(word, 4) & 0x87878787 are the fp8 (e4m3) MFMA
 *     operand bytes of the even and the odd codes (value c * 2^-9, exact).
 *   - Packed layouts (G = K/128 groups, G4 = ceil(G/4)). Each is chosen so that one
 *     64-lane 16-byte load of the GEMM reads 1 KB of contiguous memory:
 *       xq  activations, group-major: the word at byte (g*M + m)*64 + 4i holds
 *           inputs 128g + 8i .. 128g + 8i + 7 of token m.
 *       wq  base codes, tiled by 16 rows x 1 group: row n, group g, byte j (0..63)
 *           of the row's 64-byte group chunk (words in input order) is at
 *             ((n/16)*G + g)*1024 + ((j/16)*16 + n%16)*16 + j%16.
 *       sw  fp16 group scales, four groups per row entry: scale (n, g) is element
 *             (((n/16)*G4 + g/4)*16 + n%16)*4 + g%4   of a u16 array of N*G4*4;
 *           entries of groups g >= G are zero.
 *       rq  residual codes of the chosen blocks, [nnz][bn][bk/2], rows contiguous
 *           (8 words of 8 codes per block row).
 *     Sizes: xq M*K/2 bytes, wq N*K/2 bytes, sw N*G4*4 u16, rq nnz*bn*bk/2 bytes.
 *   - Packed buffers (xq, wq, rq), the activations x and the fp32 w and h must be
 *     16-byte aligned; sw must be 8-byte aligned.
 *   - Argument checks happen before any launch and return MQ_ERR_INVALID_ARG or
 *     MQ_ERR_UNSUPPORTED with nothing written. A failed launch returns
 *     MQ_ERR_HIP; faults inside a kernel surface at the caller's next
 *     synchronisation of `stream`.
 *   - Shapes the GPU path supports: K % 128 == 0, K <= 65536, group == 128, bk == 64,
 *     bn in {64, 128}, N % bn == 0. M may be any value >= 0 (M == 0 is a no-op).
 *   - Inputs must be finite, and max|w| over a group must be below 7 * 65504
 *     (the fp16 scale must be finite); otherwise results are unspecified.
 */
#ifndef MQ_H
#define MQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MQ_OK = 0,
    MQ_ERR_INVALID_ARG = -1,  /* null pointer, bad size, misaligned buffer, k_blocks > NB */
    MQ_ERR_UNSUPPORTED = -2,  /* shape outside the supported set above */
    MQ_ERR_HIP = -3,          /* a HIP runtime call or launch failed */
    MQ_ERR_SCRATCH = -4       /* the shape needs more than the library's static scratch */
} mq_status;

typedef enum { MQ_F32 = 0, MQ_BF16 = 1 } mq_dtype;

/* Human-readable text for a status code (static storage). */
const char* mq_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int mq_version(void);

/*
 * Diagonal-Hessian estimate of the input channels (Methodology 2: the
 * "activation sensitivity" that weights the residual error in the Delta-score).
 *   h[k] = fp32( (sum over m = 0..M-1, in ascending order, of (double)x[m][k]^2) / M )
 * x: [M][K] fp32 or bf16 (x_dtype), h: fp32 [K]. M >= 1, K >= 1.
 */
int mq_hessian_diag(const void* x, int x_dtype, int64_t M, int64_t K, float* h, void* stream);

/*
 * Migration of activation outliers into the weights by an equivalent per-channel
 * transform (Methodology 1: the method starts by moving activation outliers into
 * the weight matrix, SmoothQuant being one such transform; the exponent is not
 * given, alpha = 1/2 here):
 *   a_k = max_m |x[m][k]|, b_k = max_n |w[n][k]|,
 *   s[k] = sqrtf(a_k) / sqrtf(b_k)  (fp32, correctly rounded), 1 when a_k or b_k is 0,
 *   r[k] = 1 / s[k].
 * The migrated layer is W^ = W diag(s) (mq_scale_columns) and X^ = X diag(r), which
 * the *_scaled calls below apply on the fly: X^ W^T = X W^T up to rounding.
 * x: [M][K] fp32 or bf16, w: fp32 [N][K], s and r: fp32 [K]. Asynchronous on `stream`.
 */
int mq_smooth_factors(const void* x, int x_dtype, int64_t M, int64_t K, const float* w, int64_t N,
                      float* s, float* r, void* stream);

/* w_hat[n][k] = fp32(w[n][k] * s[k]) (the migrated weights). K % 4 == 0; w, s and
 * w_hat 16-byte aligned; w_hat may equal w (in place). */
int mq_scale_columns(const float* w, int64_t N, int64_t K, const float* s, float* w_hat, void* stream);

/* mq_hessian_diag of the migrated activations x^[m][k] = fp32(x[m][k] * r[k]). */
int mq_hessian_diag_scaled(const void* x, int x_dtype, int64_t M, int64_t K, const float* r, float* h,
                           void* stream);

/* mq_quantize_act of the migrated activations x^[m][k] = fp32(x[m][k] * r[k]); the
 * per-call path of a migrated layer (r 16-byte aligned). */
int mq_quantize_act_scaled(const void* x, int x_dtype, int64_t M, int64_t K, const float* r, uint8_t* xq,
                           float* sx, void* stream);

/*
 * Per-token symmetric int4 activation quantization (the W4A4 setting of the
 * Experimental Results; "quantization" is the first stage of the ZipperEngine
 * pipeline, Methodology 3).
 *   sx[m] = fp32(max_k |x[m][k]| / 7)
 *   xq[m][k] = sx[m] == 0 ? 0 : clamp(rint(x[m][k] / sx[m]), -7, 7)   (ties to even)
 * x: [M][K] fp32 or bf16 (row-major, 16-byte aligned), xq: M*K/2 bytes in the
 * group-major layout above, sx: fp32 [M]. K % 128 == 0.
 */
int mq_quantize_act(const void* x, int x_dtype, int64_t M, int64_t K, uint8_t* xq, float* sx,
                    void* stream);

/*
 * Hessian-guided Delta-score of every (bn x bk) block and global top-k_blocks
 * selection (Methodology 2 "Block-wise Residual Allocation").
 * For element (n, k) of group g with fp16 base scale s (see mq_pack_weights):
 *   q = base code, E = w - s*q, s_r = fp32(s / 14), r = clamp(rint(E / s_r), -7, 7),
 *   E' = E - s_r*r (single rounding).
 *   Delta_b = sum over rows n of b (ascending) of
 *             [ sum over cols k of b (ascending) of (double)h[k] * (E^2 - E'^2) ]
 * every fp64 operation rounded separately. Blocks are ranked by (Delta descending,
 * id ascending), id = (n / bn) * (K / bk) + k / bk, and the first k_blocks are
 * chosen. Output is CSR over block rows:
 *   row_ptr: int32 [N/bn + 1], col_idx: int32 [k_blocks] (column-block index,
 *   ascending within a row), delta: fp64 [NB] with NB = (N/bn)*(K/bk).
 * w: fp32 [N][K], h: fp32 [K]. 0 <= k_blocks <= NB.
 * delta may be NULL (the scores are then kept in the workspace and not returned).
 * workspace: device scratch of at least mq_select_workspace_bytes(N, K, bn, bk) bytes,
 * 8-byte aligned (the per-block ranks, 4 * NB bytes, and when delta is NULL the
 * scores, 8 * NB more), or NULL: the call then takes a stream-ordered allocation
 * (hipMallocAsync) and releases it on the same stream. Calls sharing one
 * workspace must be ordered on one stream.
 */
int mq_select_blocks(const float* w, const float* h, int64_t N, int64_t K, int group, int bn,
                     int bk, int64_t k_blocks, int32_t* row_ptr, int32_t* col_idx,
                     double* delta, void* workspace, size_t workspace_bytes, void* stream);

/*
 * mq_select_blocks for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc. Same
 * arguments, results and errors as mq_select_blocks without a workspace; its
 * scratch (select ranks, and the scores when delta is NULL) is a static device
 * array of MQ_NOALLOC_SCRATCH_BYTES that the library holds on each GPU it runs
 * on until the process ends. The call makes no allocation of any kind.
 * Limit: 4 * NB bytes (rounded up to 8) plus 8 * NB when delta is NULL must fit,
 * i.e. NB <= 349525 with delta NULL, NB <= 1048576 otherwise; larger shapes
 * return MQ_ERR_SCRATCH with nothing launched. Every call on one GPU shares that
 * GPU's array: calls that overlap on one GPU (different streams, or threads
 * without ordering) race and give wrong results; order them on one stream.
 * The first call on a device looks up the array's address on that device
 * (hipGetSymbolAddress) with the device current.
 */
#define MQ_NOALLOC_SCRATCH_BYTES (4u << 20)
int mq_select_blocks_noalloc(const float* w, const float* h, int64_t N, int64_t K, int group,
                             int bn, int bk, int64_t k_blocks, int32_t* row_ptr,
                             int32_t* col_idx, double* delta, void* stream);

/* Workspace bytes mq_select_blocks needs for this shape with delta == NULL (12 * NB;
   4 * NB suffice when delta is given); 0 for an unsupported shape. */
size_t mq_select_workspace_bytes(int64_t N, int64_t K, int bn, int bk);

/*
 * Packs the dense 4-bit base for every group and the 4-bit residual payload for
 * the chosen blocks (Methodology 1: W^ ~ Q(W^) + R, both parts 4-bit).
 *   sw(n, g) = fp16_rne( fp32(max_{k in g} |w[n][k]|) / 7 )      (fp16 bits)
 *   wq(n, k) = s == 0 ? 0 : clamp(rint(w / s), -7, 7)  with s = fp32(sw(n, g))
 *   rq[p][i][c] = residual code r (see mq_select_blocks) of row (row_block*bn + i),
 *                 column (col_idx[p]*bk + c) for CSR entry p, in CSR order.
 * w: fp32 [N][K] row-major; row_ptr/col_idx as produced by mq_select_blocks (nnz
 * entries); wq, sw, rq in the packed layouts above (rq may be NULL if nnz == 0).
 * Entries with a column-block index outside [0, K/bk) are skipped.
 */
int mq_pack_weights(const float* w, int64_t N, int64_t K, int group, int bn, int bk,
                    const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz,
                    uint8_t* wq, uint16_t* sw, uint8_t* rq, void* stream);

/*
 * The fused ZipperEngine GEMM (Methodology 3): one kernel streams the packed base
 * and, inside the same K-loop, the residual blocks listed for its rows; both
 * products are summed exactly per 128-group (integers; the fp8 MFMA returns them
 * scaled by 2^-18 without rounding), and the group sums are dequantized and
 * summed in fp32:
 *   T[m][n][g] = 14 * P + Pr,  P = sum_{k in g} xq*q,  Pr = sum over chosen blocks in g of xq*r
 *   y[m][n]    = sx[m] * sum_g ( groups with a chosen block in this row: s_r * T,
 *                                otherwise s * P )            (fp32; s_r = fp32(s/14))
 * which equals sx * sum_g (s*P + s_r*Pr) up to fp32 rounding.
 * xq, wq, sw, rq in the packed layouts above (rq NULL if nnz == 0), sx: fp32 [M],
 * row_ptr: int32 [N/bn+1], col_idx: int32 [nnz],
 * y: [M][N] fp32 or bf16 (y_dtype, bf16 rounded to nearest even).
 * acc_dump: NULL, or int32 [M][N][K/group] receiving T (a debug build of the same
 * kernel; production calls pass NULL). Indices outside the CSR ranges are ignored,
 * so a malformed list gives wrong values, never an out-of-bounds access.
 * The call allocates nothing and needs no scratch memory.
 */
int mq_gemm_w4a4_residual(const uint8_t* xq, const float* sx, const uint8_t* wq,
                          const uint16_t* sw, const int32_t* row_ptr, const int32_t* col_idx,
                          const uint8_t* rq, int64_t nnz, int64_t M, int64_t N, int64_t K,
                          int group, int bn, int bk, void* y, int y_dtype, int32_t* acc_dump,
                          void* stream);

/*
 * The dense block map of a selection (Methodology 3: the fused kernel finds each
 * 128-group's residual blocks in step with the K loop; with the map that lookup is
 * one coalesced load per wavefront instead of a walk of the block row's list):
 *   rmap[b][j] = p  if col_idx[p] == j for some p in [row_ptr[b], row_ptr[b+1]),
 *              = -1 otherwise,
 * for block rows b < N/bn and column blocks j < K/bk. rmap: int32 [N/bn][K/bk]
 * (device, 4-byte aligned), fully overwritten. Entries with a column-block index
 * outside [0, K/bk) are skipped; for a block listed twice in one row, one of its
 * positions is kept. Row pointers are clamped to [0, nnz]. Asynchronous.
 */
int mq_block_map(const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz, int64_t N, int64_t K,
                 int bn, int bk, int32_t* rmap, void* stream);

/*
 * mq_gemm_w4a4_residual with the chosen blocks found through a block map
 * (mq_block_map of the CSR lists the payload was packed with) instead of the lists:
 * the same kernels and the same arithmetic, so y and acc_dump are bit-identical to
 * mq_gemm_w4a4_residual's. Map entries outside [0, nnz) mean "no block".
 * Requires nnz * bn * bk / 2 <= 2^31 (else MQ_ERR_UNSUPPORTED).
 */
int mq_gemm_w4a4_residual_mapped(const uint8_t* xq, const float* sx, const uint8_t* wq,
                                 const uint16_t* sw, const int32_t* rmap, const uint8_t* rq,
                                 int64_t nnz, int64_t M, int64_t N, int64_t K, int group, int bn,
                                 int bk, void* y, int y_dtype, int32_t* acc_dump, void* stream);

/*
 * The fused GEMM that also quantizes its activations (Methodology 3 schedules
 * quantization as a stage of the same pipeline as the dense and sparse products):
 * y = mq_gemm_w4a4_residual_mapped applied to mq_quantize_act(x), with xq and sx
 * written as mq_quantize_act writes them (same bits), and y bit-identical to the
 * two calls in sequence.
 * It runs either as one launch (M <= 32): its first M workgroups quantize one
 * token each while the output-column workgroups wait for them (counters in
 * `sync`) before reading any activation; or as two launches on `stream`,
 * mq_quantize_act and then the GEMM. `launch` picks: MQ_ACT_ONE_LAUNCH (M > 32
 * is then an invalid argument), MQ_ACT_TWO_LAUNCHES, or MQ_ACT_AUTO, which takes
 * one launch when mq_act_one_launch(M, N, K) says so and two otherwise. Both give
 * the same bits.
 * x: [M][K] fp32 or bf16 (x_dtype), 16-byte aligned; xq, sx: outputs as in
 * mq_quantize_act; rmap, rq, nnz: as in mq_gemm_w4a4_residual_mapped (rmap required).
 * sync (required when the one-launch form runs, else unused and may be null):
 * int32 [MQ_SYNC_WORDS] device array, all zero before the first call (e.g.
 * zero-filled once); every completed call leaves it zero again, so it needs no
 * clearing between calls and the call can be captured in a HIP graph. It holds the
 * count of quantized tokens, a check-in count and, in one 128-byte line per XCD
 * slot, a ready flag and a count of finished column workgroups. sync[2] becomes 1
 * if a workgroup ever gave up waiting (after well under a few seconds; never
 * expected) and stays 1 until the caller clears it. Calls that share one sync
 * array must not overlap (order them on one stream).
 */
#define MQ_SYNC_WORDS 544
#define MQ_ACT_AUTO 0
#define MQ_ACT_ONE_LAUNCH 1
#define MQ_ACT_TWO_LAUNCHES 2
/*
 * The MQ_ACT_AUTO rule of mq_gemm_w4a4_residual_act, for callers that need to know
 * beforehand whether the counters are required: 1 if the call takes one launch
 * for this shape, else 0 (also for M outside 1..32, and for shapes the GEMM does
 * not accept). Host only; no GPU call.
 * One launch when its per-token quantizing workgroups (the decode plan's waves)
 * are at least as wide as the stand-alone quantizer's, M = 1 and N >= 4096: where
 * it measured faster on MI355X.
 */
int mq_act_one_launch(int64_t M, int64_t N, int64_t K);
int mq_gemm_w4a4_residual_act(const void* x, int x_dtype, const uint8_t* wq, const uint16_t* sw,
                              const int32_t* rmap, const uint8_t* rq, int64_t nnz, int64_t M,
                              int64_t N, int64_t K, int group, int bn, int bk, uint8_t* xq,
                              float* sx, int32_t* sync, int launch, void* y, int y_dtype, void* stream);

/*
 * Measurement aid, not a step of the method: a plain streaming read of `bytes`
 * bytes at p (16-byte aligned, bytes a multiple of 16), the HBM read rate a kernel
 * reaches at that byte count. The decode GEMM streams its weights once, so this
 * is the ceiling its time is compared with (the Experimental Results measure
 * decode overheads against the dense kernel; this measures both against memory).
 * out: uint32 [MQ_READ_PROBE_WORDS] device array; each workgroup writes the XOR of
 * the words it read to one entry (the values mean nothing). Asynchronous.
 */
#define MQ_READ_PROBE_WORDS 8192
int mq_read_probe(const void* p, int64_t bytes, uint32_t* out, void* stream);

/*
 * Dense-only 4-bit GEMM: the same kernel with the residual path compiled out
 * (the "dense 4-bit GEMM kernel" the residual is fused into, Methodology 3).
 * y = sx * sum_g s * P. With nnz == 0 the fused call gives the same bits.
 * acc_dump (optional) receives T = 14 * P.
 */
int mq_gemm_w4a4_dense(const uint8_t* xq, const float* sx, const uint8_t* wq, const uint16_t* sw,
                       int64_t M, int64_t N, int64_t K, int group, void* y, int y_dtype,
                       int32_t* acc_dump, void* stream);

/*
 * The separate-kernel alternative that Methodology 3 argues against: the dense
 * kernel writes fp32 partial outputs to `ws` (fp32 [M][N], caller-allocated),
 * then a second kernel re-reads the activations, computes the residual product
 * block by block, merges it into the partial outputs and writes y.
 * y = sx * sum_g (s*P + s_r*Pr) up to fp32 rounding. Same arguments as the fused
 * call plus ws.
 */
int mq_gemm_residual_separate(const uint8_t* xq, const float* sx, const uint8_t* wq,
                              const uint16_t* sw, const int32_t* row_ptr, const int32_t* col_idx,
                              const uint8_t* rq, int64_t nnz, int64_t M, int64_t N, int64_t K,
                              int group, int bn, int bk, void* y, int y_dtype, float* ws,
                              void* stream);

/*
 * ---------------------------------------------------------------------------------
 * Microscaled 4-bit operands, routing to experts and the experts' products.
 *
 * The format (OCP microscaling, MXFP4): 32 consecutive inputs of a row are a block
 * with one scale X = 2^(byte - 127); a value is code * X, the code one of 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 with a sign (4 bits: sign, then the index). gfx950 multiplies such
 * operands directly, so a product needs no conversion and no scaling of its own.
 *   Device layout of a matrix [R][K] (RT = ceil(R/16), G = ceil(K/128), G4 = ceil(G/4)):
 *     codes   RT * G tiles of 1 KB, 16 rows x 128 inputs: the code of (r, k) is nibble
 *             k % 32 (low nibble first) of the 16 bytes at
 *               (((r/16)*G + k/128)*64 + ((k/32) % 4)*16 + r % 16) * 16
 *     scales  one byte per block: the byte of (r, k) is at
 *               (((r/16)*G4 + k/512)*64 + ((k/32) % 4)*16 + r % 16) * 4 + (k/128) % 4
 *   Rows up to RT * 16 and blocks up to G * 128 (bytes: G4 * 512) inputs exist and hold
 *   codes of zero. A batch [B][R][K] is B such matrices in a row (experts' weights:
 *   B = experts). codes 16-byte aligned, scales 4-byte aligned.
 *   Any R, K >= 1 (K <= 2^20, R <= 2^24).
 *
 * These calls take fp32, bf16 and fp16 (MQ_F16) wherever they take a type. Inputs'
 * last axis is contiguous, other strides are arguments (in elements, >= 0). Outputs are
 * contiguous and 16-byte aligned, except the routing's (4-byte). Sums are held in
 * fp32 and rounded once to the output's type.
 */
#define MQ_F16 2

size_t mq_mx_codes_bytes(int64_t R, int64_t K);   /* 0 outside the supported sizes */
size_t mq_mx_scales_bytes(int64_t R, int64_t K);

/*
 * Quantization: X = 2^(floor(log2(max |x| over the block)) - 2), at least 2^-127;
 * codes are x / X rounded to the nearest, ties to the even index, magnitudes above 6 to
 * 6. A block with a NaN or an infinity gets byte 255 (the format's NaN) and reads back,
 * and multiplies, as NaN.
 * x: [B][R][K] with strides stride_b, stride_r.
 */
int mq_mx_quantize(const void* x, int x_dtype, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r,
                   int64_t K, uint8_t* codes, uint8_t* scales, void* stream);

/* The values back: y [B][R][K], rounded once to y's type (bf16 and fp32 hold every
 * quantized value exactly; fp16 those within its range). */
int mq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t K, void* y,
                     int y_dtype, void* stream);

/* y[m][n] = sum_k xq[m][k] * wq[n][k] (+ bias[n], fp32, may be NULL). xq/xs: an
 * M x K matrix, wq/ws: N x K. */
int mq_mx_gemm(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, int64_t M, int64_t N,
               int64_t K, const float* bias, void* y, int y_dtype, void* stream);

/* The way that such a product takes: 0: K split over a workgroup's waves, 16 rows and 16
 * columns a workgroup; 1, 2, 3: the same with 32 rows and 16, 32, 64 columns; 4 .. 7: tiles of
 * 32, 64, 96, 128 rows and 256 columns. A status below 0 outside the supported sizes. The
 * ways give the same sums in another order of additions. */
int mq_mx_gemm_way(int64_t M, int64_t N, int64_t K);

/* The same from unquantized activations x [M][K] (row stride stride_m): the bits of
 * mq_mx_quantize followed by mq_mx_gemm. workspace: device scratch of at least
 * mq_mx_linear_workspace_bytes, 16-byte aligned (may be NULL where that is 0). */
size_t mq_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mq_mx_linear(const void* x, int x_dtype, int64_t stride_m, const uint8_t* wq, const uint8_t* ws, int64_t M,
                 int64_t N, int64_t K, const float* bias, void* y, int y_dtype, void* workspace,
                 size_t workspace_bytes, void* stream);

/*
 * Routing: the k experts of each token and their weights, from logits [T][E].
 *   score[e] = softmax over e, or sigmoid, of the logits; a logit of -inf masks its expert
 *   key[e] = score[e] + bias[e] (bias fp32 [E]); without a bias the logit itself, in
 *            whose order both scores are. A bias of -inf masks its expert too.
 *   groups > top_groups: experts are `groups` runs of E / groups; a group is worth its
 *            largest key (MQ_GROUP_MAX) or the sum of its two largest (MQ_GROUP_TOP2, of
 *            score + bias); only the top_groups best groups are kept.
 *   ids      the k experts of largest key, in that order
 *   weights  their scores; renormalize: divided by their sum; then times scale
 * Ties go to the lower index, of groups as of experts. Slots that no unmasked expert is
 * left for hold id -1 and weight 0 (a token whose experts are all masked: all of its
 * slots). A token with a NaN key (a NaN logit or bias, or +inf under softmax) has ids -1
 * and weights NaN. Scores and keys are held in 64 bits.
 * ids: int32 [T][k], weights: fp32 [T][k]. E <= MQ_MAX_EXPERTS, k <= 32, groups <= 64,
 * k <= top_groups * E / groups.
 */
#define MQ_MAX_EXPERTS 1024
#define MQ_SCORE_SOFTMAX 0
#define MQ_SCORE_SIGMOID 1
#define MQ_GROUP_MAX 0
#define MQ_GROUP_TOP2 1
int mq_route(const void* logits, int dtype, int64_t T, int64_t stride_t, int64_t E, const float* bias, int score,
             int64_t groups, int64_t top_groups, int group_score, int64_t k, int renormalize, float scale,
             int32_t* ids, float* weights, void* stream);

/*
 * A plan: one row for every (token, slot) whose id is in [0, E), ordered by expert, then
 * by token and slot; each expert's rows start at a multiple of 16.
 *   offsets    int32 [E + 1]: expert e's rows are from offsets[e]; offsets[e + 1] is that
 *              plus its number of rows, rounded up to 16
 *   row_token  int32 [mq_plan_rows(T, k, E)]: the row's token, -1 for rows of none
 *   row_of     int32 [T][k]: the slot's row, -1 for ids outside [0, E)
 * mq_plan_rows is the most rows that any ids can take (-1 outside the supported sizes).
 * T * k <= 2^27.
 */
int64_t mq_plan_rows(int64_t T, int64_t k, int64_t E);
int mq_expert_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets, int32_t* row_token,
                   int32_t* row_of, void* stream);

/*
 * The experts' gate and up products: for row p of expert e with token t = row_token[p]
 *   h[p][i] = silu(g) * u,  g = Q(x[t]) . gate[e][i],  u = Q(x[t]) . up[e][i]
 * with silu(g) = g / (1 + exp(-g)); rows of no token are zero. x: [T][D] (row stride
 * stride_t), gate and up: E matrices I x D, h: [mq_plan_rows][I]. The plan is
 * mq_expert_plan's; entries of row_token and row_of out of range (rows from offsets[E] on
 * among them) are taken as "no row".
 * T * ceil(D / 256) * 128 < 2^32.
 */
size_t mq_mx_experts_up_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t D, int64_t I);
int mq_mx_experts_up(const void* x, int x_dtype, int64_t stride_t, int64_t T, int64_t k, int64_t E, int64_t D,
                     int64_t I, const int32_t* offsets, const int32_t* row_token, const int32_t* row_of,
                     const uint8_t* gate_q, const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s,
                     void* h, int h_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The experts' down products and their weighted sum, added in the order of the slots:
 *   y[t][d] = sum over j of weights[t][j] * (Q(h[row_of[t][j]]) . w[e][d])
 * A slot without a row adds weights[t][j] * 0. h: [mq_plan_rows][I], w: E matrices
 * D x I, y: [T][D].
 */
size_t mq_mx_experts_down_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t D, int64_t I);
int mq_mx_experts_down(const void* h, int h_dtype, int64_t T, int64_t k, int64_t E, int64_t D, int64_t I,
                       const int32_t* offsets, const int32_t* row_of, const float* weights, const uint8_t* wq,
                       const uint8_t* ws, void* y, int y_dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * ---------------------------------------------------------------------------------
 * Group-scaled 4-bit weights and products of unquantized rows with them.
 *
 * The format: `group` (32, 64 or 128) consecutive inputs of a row share a scale s and a
 * zero point z, both 16-bit floats of one type (scale_dtype: MQ_F16 or MQ_BF16); z is 8
 * where there are no zero points. A weight is s * (c - z), its code c = 0 .. 15.
 *   Device layout of a matrix [R][K] (RT = ceil(R/16), G = ceil(K/128), Q = ceil(K/512)):
 *     codes   RT * G tiles of 1 KB, 16 rows x 128 inputs. The codes of row r and the inputs
 *             8j .. 8j + 7 are the word (j/4) % 4 of the 16 bytes at
 *               (((r/16)*G + j/16)*64 + (j % 4)*16 + r % 16) * 16,
 *             input 8j + i in the low half of its byte i (i < 4) or the high half of its
 *             byte i - 4.
 *     scales, zeros   the value of (r, k) is entry
 *               (((r/16)*Q + k/512)*16 + r % 16) * (512/group) + (k % 512)/group
 *   Rows up to RT * 16 and inputs up to G * 128 (scales: Q * 512) exist and hold zeros. A
 *   batch [B][R][K] is B such matrices in a row. codes, scales and zeros 16-byte aligned.
 *   Any R, K >= 1 (K <= 2^20, R <= 2^24).
 */
size_t mq_w4_codes_bytes(int64_t R, int64_t K);   /* 0 outside the supported sizes */
size_t mq_w4_scales_bytes(int64_t R, int64_t K, int group);

/*
 * Quantization, x [B][R][K] with strides stride_b, stride_r; r32 and r16 round to fp32 and
 * to the scales' type, rne to the nearest whole number, ties to even:
 *   zeros NULL:  s = r16(r32(max |x| / 7)),  c = clamp(rne(x / s), -8, 7) + 8
 *   else:        lo = min(0, min x), hi = max(0, max x), s = r16(r32(r32(hi - lo) / 15)),
 *                z = clamp(rne(-lo / s), 0, 15),  c = clamp(rne(x / s) + z, 0, 15)
 * The quotients by s are exact. s is at most the type's largest value; where it is 0,
 * c = z (z = 0 with zero points). A group with a NaN or an infinity gets s = NaN and reads
 * back, and multiplies, as NaN.
 */
int mq_w4_quantize(const void* x, int x_dtype, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r, int64_t K,
                   int group, int scale_dtype, uint8_t* codes, void* scales, void* zeros, void* stream);

/* Weights that are quantized already: c [B][R][K], one code a byte (its low four bits count;
 * strides stride_b, stride_r; a checkpoint that holds several in a word is unpacked first), s and z (or
 * NULL) [B][R][ceil(K/group)], contiguous, of any 16-bit float type, in the library's layout. */
int mq_w4_pack(const uint8_t* c, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r, int64_t K, int group,
               const void* s, const void* z, uint8_t* codes, void* scales, void* zeros, void* stream);

/* The values back: y [B][R][K], in fp32 and rounded to y's type. */
int mq_w4_dequantize(const uint8_t* codes, const void* scales, const void* zeros, int scale_dtype, int64_t B, int64_t R,
                     int64_t K, int group, void* y, int y_dtype, void* stream);

/*
 * y[m][n] = sum_k x[m][k] w[n][k] (+ bias[n], fp32, may be NULL), x [M][K] (row stride
 * stride_m) as it is, w [N][K]: sums of x times codes, which are exact products, are held in
 * fp32, a group's sum is scaled once. A row of x with a NaN or an infinity gives NaN, and so
 * does a group whose sum of |x| times 15 leaves fp32's range. workspace: device scratch of at
 * least mq_w4_linear_workspace_bytes, 16-byte aligned (may be NULL where that is 0). y shares no
 * memory with x, here and by expert.
 */
size_t mq_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, int group);
int mq_w4_linear(const void* x, int x_dtype, int64_t stride_m, const uint8_t* codes, const void* scales,
                 const void* zeros, int scale_dtype, int group, int64_t M, int64_t N, int64_t K, const float* bias,
                 void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* The way that such a product takes, a status below 0 outside the supported sizes. Kernels of
 * few rows, K split over a workgroup's waves: 0: 4 rows and 16 columns a workgroup; 1, 2: 16
 * rows and 16, 32 columns; 4, 5: 32 rows and 32, 64 columns. 8 p + t: tiles with K in p
 * parts, t = 0 .. 4: 32 x 128, 64 x 128, 64 x 256, 96 x 256, 128 x 256
 * (groups of 32: not 2 and 4). Tiles hold sums in
 * units of the present scale of a row of w. Where that leaves fp32's range (32 rows with a result that
 * is not finite), and for rows of w with bf16 scales outside 2^-126 .. 2^126 or more than 2^40 apart, they
 * compute those outputs again group by group, in up to three times a product's time. The ways give
 * the same sums in another order of additions; sums of x times codes below 2^-86 may count as zero
 * in tiles. */
int mq_w4_linear_way(int64_t M, int64_t N, int64_t K, int x_dtype, int group);

/*
 * The same for the rows of a plan (mq_expert_plan), each with its expert's matrix:
 *   y[p][n] = sum_k x[r][k] w[e][n][k], e the expert of row p,
 * r = p, x [mq_plan_rows][K], or by_token r = row_token[p], x [T][K]. Rows of no token are
 * zero. w: E matrices N x K, y: [mq_plan_rows][N]. Entries of the plan out of range are
 * taken as "no row".
 */
size_t mq_w4_experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int by_token, int x_dtype,
                                     int group);
int mq_w4_experts(const void* x, int x_dtype, int64_t stride_r, int by_token, int64_t T, int64_t k, int64_t E, int64_t N,
                  int64_t K, const int32_t* offsets, const int32_t* row_token, const uint8_t* codes, const void* scales,
                  const void* zeros, int scale_dtype, int group, void* y, int y_dtype, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------------
 * Tokens to the rows of their experts and back, over a plan (mq_expert_plan); each is
 * the other's gradient. v[t][j] = weights[t][j] (fp32 [T][k]), or 1 where weights is NULL.
 *   gather   rows[row_of[t][j]] = v[t][j] * x[t]; rows of no token are zero
 *   combine  x[t] = sum over j of v[t][j] * rows[row_of[t][j]], added in the order of the slots;
 *            a slot without a row adds v[t][j] * 0
 * With `other` also the dots, the gradient of the weights, in fp32 [T][k]:
 *   gather   other [mq_plan_rows][D] of rows' type, dots[t][j] = x[t] . other[row_of[t][j]]
 *   combine  other [T][D] of x's type, its rows stride_o apart, dots[t][j] = other[t] .
 *            rows[row_of[t][j]]
 * and 0 for slots without a row. x [T][D] (gather: its rows stride_t apart), rows
 * [mq_plan_rows][D]; each of its own type. Products and sums in fp32, rounded once. Entries of row_of and
 * row_token out of range are taken as "no row". D <= 2^20. What is written shares no memory with what is
 * read.
 */
int mq_experts_gather(const void* x, int x_dtype, int64_t stride_t, int64_t T, int64_t k, int64_t E, int64_t D,
                      const int32_t* row_token, const int32_t* row_of, const float* weights, void* rows, int rows_dtype,
                      const void* other, float* dots, void* stream);
int mq_experts_combine(const void* rows, int rows_dtype, int64_t T, int64_t k, int64_t E, int64_t D,
                       const int32_t* row_of, const float* weights, void* x, int x_dtype, const void* other,
                       int64_t stride_o, float* dots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQ_H */
