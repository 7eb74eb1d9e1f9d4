/*
 * mx.h -- C ABI of libmx: the block-scaled (OCP microscaling, "MX") linear
 * layer y = x . W^T on AMD Instinct MI355X (gfx950).
 *
 * Sources (web pages, cited by title and section):
 *   [weights942]   vllm.models.deepseek_v41.amd.mono.weights942
 *   [rocm_native]  vllm.model_executor.kernels.linear.mxfp8.rocm_native
 *   [a16w4]        vllm.models.minimax_m3.amd.specialized_decode.mono.a16w4
 *   [fused_layout] vllm.models.deepseek_v41.common.ops.fused_layout
 *
 * Number formats.
 *   E4M3   OCP fp8 byte (bias 7, max 448, 0x7F/0xFF NaN)        [weights942]
 *   E2M1   OCP fp4 nibble, two per byte, low nibble = even K       [a16w4] dequant
 *   E8M0   scale code c meaning 2^(c - 127), 255 = NaN            [weights942] ocp_from_dequant
 *   bf16   activations, bias and outputs
 * Every 32 consecutive K values of a weight row share one E8M0 code, laid out
 * either one code per row and block (ROW32, [E*N, K/32]) or one code per
 * 32 rows x 32 K block (BLK32, [E*N/32, K/32]) ([rocm_native]
 * process_weights_after_loading and _as_block32_scale).
 *
 * Conventions for every entry point.
 *   - Pointers marked (device) are device memory of the current HIP device;
 *     (host) are host memory.  The caller allocates and owns every buffer;
 *     the library never allocates device memory in these calls.
 *   - All device work is enqueued on `stream` (0 = the null stream) and the
 *     calls return without synchronizing, except the load-time calls that
 *     read back a validity flag: mx_pack_weights, mx_fold_row_codes,
 *     mx_e4m3_from_dequant and mx_moe_copies.
 *   - Arguments are validated on the host before anything is launched; on an
 *     error nothing is launched and outputs are untouched.
 *   - Each call checks that the current device is gfx950 (MX_ERR_DEVICE).
 *   - Inputs holding NaN or Inf give unspecified outputs.
 */
#ifndef MX_H
#define MX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;
typedef struct ihipStream_t *mx_stream_t; /* same type as hipStream_t */

typedef enum {
    MX_OK = 0,
    MX_ERR_NULL = 1,        /* a required pointer is NULL                      */
    MX_ERR_SHAPE = 2,       /* a size or leading dimension breaks the rules    */
    MX_ERR_ALIGN = 3,       /* a pointer or leading dimension is misaligned    */
    MX_ERR_VALUE = 4,       /* an E8M0 weight code 255 (NaN) was found at pack */
    MX_ERR_UNSUPPORTED = 5, /* a format / layout / mode combination not built  */
    MX_ERR_DEVICE = 6,      /* the current device is not gfx950 (or none)     */
    MX_ERR_WORKSPACE = 7,   /* the workspace is NULL or smaller than required  */
    MX_ERR_LAUNCH = 8       /* a HIP call or kernel launch failed              */
} mx_status;

typedef enum { MX_E4M3 = 0, MX_E2M1 = 1 } mx_elem;
typedef enum { MX_SCALE_ROW32 = 0, MX_SCALE_BLK32 = 1 } mx_scale_layout;
/* Activation scale rules ([rocm_native] _quant_mxfp8_tile and OCP MX v1.0):
 *   MX_RULE_OCP      code = clamp(floor(log2 amax) - 8 + 127, 0, 254); the
 *                    scaled elements are rounded to nearest-even e4m3 and
 *                    saturated to +-448.
 *   MX_RULE_CEIL448  code = clamp(ceil(log2(max(amax, 2^-126) / 448)) + 127,
 *                    0, 254); the scaled elements never exceed 448.
 * Either way a block whose amax is 0 gets code 0, and a zero element keeps
 * its sign (-0 -> 0x80). */
typedef enum { MX_RULE_OCP = 0, MX_RULE_CEIL448 = 1 } mx_quant_rule;
/* MX_ACT_BF16: activations stay bf16 (A16W8 / A16W4).
 * MX_ACT_MXFP8: activations are MXFP8, e4m3 bytes [M, K] with row-major
 * E8M0 codes [M, K/32] ([rocm_native] input_quant_key: row-major, not
 * swizzled), either given pre-quantized or quantized inside the call (W8A8).
 * MX_ACT_MXFP8_T16: MXFP8 activations pre-quantized by mx_quant_act_t16 into
 * the library's 16-token tile layout (below); the same values as
 * MX_ACT_MXFP8, stored the way the matrix cores read them, so a quantized
 * activation can be shared by several linears without re-reading it
 * row-major. */
typedef enum { MX_ACT_BF16 = 0, MX_ACT_MXFP8 = 1, MX_ACT_MXFP8_T16 = 2 } mx_act;

/*
 * T16 activation layout (this library's own; the values are those of
 * mx_quant_act).  S = ceil(K / 128) steps, Q = ceil(S / 4), MB = ceil(M / 16)
 * token tiles, lane l = 16 j + r:
 *   xq     MB * S * 2048 bytes: byte ((mb S + s) 2 + h) 1024 + 16 l + c is
 *          the e4m3 value of token 16 mb + r at K 128 s + 64 h + 16 j + c;
 *   xcodes MB * Q * 256 bytes: byte (mb Q + q) 256 + 4 l + u is the code of
 *          token 16 mb + r, block 4 (4 q + u) + j.
 * Tokens past M and K past the end hold byte 0 and code 127.
 */

/*
 * Packed weight layout ("W-T16", [weights942] dense_copy / fp4_tile_major
 * tile-major idea; [a16w4] module notes for E2M1).
 *   S = ceil(K / 128) steps, T = N / 16 tiles, Q = ceil(S / 4).  Lane
 *   l = 16 j + r.  A tile holds exactly 16 row lengths, TILEB = 16 K (E4M3)
 *   or 8 K (E2M1) bytes: no padding is stored.  When K % 128 != 0 the last
 *   step's chunk holds only its valid bytes, which are the chunk's first
 *   512 (E4M3) or 256 (E2M1) bytes per 32-K block present.
 *   E4M3: chunk (e, t, s) of 2048 bytes at (e T + t) TILEB + 2048 s;
 *         byte 1024 h + 16 l + c = W[e][16 t + r][128 s + 64 h + 16 j + c].
 *   E2M1: chunk (e, t, s) of 1024 bytes at (e T + t) TILEB + 1024 s;
 *         byte 16 l + c = packed byte 64 s + 16 j + c of row 16 t + r.
 *   Codes are padded to 4 Q steps per row (group) with code 128
 *   ([weights942] dense_copy pads its steps).
 * Packed codes:
 *   ROW32: 256 bytes per (e, t, q) at ((e T + t) Q + q) * 256;
 *          byte 4 l + u = code[e N + 16 t + r][4 (4 q + u) + j].
 *   BLK32: 16 bytes per (32-row group R, q) at (R Q + q) * 16, R < E N / 32;
 *          byte 4 j + u = code[R][4 (4 q + u) + j].
 *   Then a 16-byte trailer: byte 0 is the smallest and byte 1 the largest of
 *   the codes given to the pack (padding codes not counted), bytes 2..15
 *   are 0.  The bf16-activation products read it to learn whether every
 *   scaled weight is a normal bf16 number (below).
 * Each lane group j reads one dword per quad of steps, whose byte u is the
 * code of step 4 q + u: the scaled MFMA's byte select picks it directly.
 */

/* Sizes of the packed buffers for a weight of E experts x [N, K].
 * Rules: E >= 1, K >= 32 and K % 32 == 0, N % 16 == 0 (N % 32 == 0 for
 * BLK32).  w_bytes, code_bytes (host) receive the sizes.
 * Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_UNSUPPORTED (unknown enum). */
mx_status mx_packed_sizes(int elem, int layout, int64_t E, int64_t N, int64_t K,
                          size_t *w_bytes, size_t *code_bytes);

/* Load-time repack ([weights942] dense_copy, fp4_tile_major,
 * codes_tile_rounds; [rocm_native] process_weights_after_loading).
 *   w      (device) standard weight bytes: E4M3 [E, N, K], E2M1 [E, N, K/2]
 *   codes  (device) ROW32 [E N, K/32] or BLK32 [E N / 32, K / 32]
 *   w_packed, codes_packed (device) outputs of mx_packed_sizes' sizes
 *   ws     (device) at least 256 bytes of scratch
 * All device pointers 16-byte aligned.  This call synchronizes `stream`: it
 * reads back whether any code is 255 and returns MX_ERR_VALUE if so (the
 * packed outputs are then written but must not be used). */
mx_status mx_pack_weights(int elem, int layout, int64_t E, int64_t N, int64_t K,
                          const void *w, const void *codes, void *w_packed,
                          void *codes_packed, void *ws, size_t ws_bytes,
                          mx_stream_t stream);

/* ---- Ingest of checkpoint forms the packs do not take directly ---- */

/* Fold row-expanded codes back into 32 x 32 block codes ([rocm_native]
 * _as_block32_scale; [weights942] linear_copy): a loader that repeats each
 * 32 x 32 block's E8M0 code over the block's 32 rows hands back [N, K/32]
 * codes; the block codes are then BLK32 codes for mx_pack_weights.
 *   codes_row (device) [N, ldc] bytes, the first K/32 of each row used
 *   codes_blk (device) [N/32, K/32] output: codes_blk[R][b] = codes_row[32 R][b]
 *   ws        (device) at least 256 bytes of scratch, 16-byte aligned
 * Rules: N % 32 == 0, K % 32 == 0, ldc >= K/32.
 * Errors: MX_ERR_VALUE when some block's 32 rows do not all hold the same
 *   code (the output is still written as above but is not the block form;
 *   keep the row codes, ROW32).  Load-time: synchronizes `stream`. */
mx_status mx_fold_row_codes(int64_t N, int64_t K, const void *codes_row, int64_t ldc,
                            void *codes_blk, void *ws, size_t ws_bytes,
                            mx_stream_t stream);

/* The e4m3 bytes behind a weight the loader dequantized to bf16
 * ([weights942] ocp_from_dequant): w[n][k] = dec(byte) * 2^(c - 127), c the
 * code of the weight's block.
 *   layout  MX_SCALE_ROW32 (codes [N, K/32]) or MX_SCALE_BLK32 ([N/32, K/32])
 *   w_bf16  (device) [N, ldw] bf16, 16-byte aligned, ldw % 8 == 0
 *   codes   (device) the codes the weight was dequantized with
 *   w_out   (device) [N, K] e4m3 bytes, 16-byte aligned
 *   ws      (device) at least 256 bytes of scratch, 16-byte aligned
 * A weight is recovered only when some finite e4m3 byte times 2^(c - 127)
 * equals it exactly; a zero keeps its sign (-0 -> 0x80).
 * Errors: MX_ERR_VALUE when some weight is not recovered -- not of that
 *   form, NaN, infinite, or under code 255 (NaN).  Its output byte is then
 *   0xFF (an e4m3 NaN, never a recovered value); every other byte is still
 *   recovered.  Load-time: synchronizes `stream`. */
mx_status mx_e4m3_from_dequant(int layout, int64_t N, int64_t K, const void *w_bf16,
                               int64_t ldw, const void *codes, void *w_out, void *ws,
                               size_t ws_bytes, mx_stream_t stream);

/* Load-time permutations of an MXFP8 linear for an attention kernel's
 * layouts ([fused_layout]: applied once to the weights, so the linear itself
 * produces or consumes the kernel's layout).
 *   kind MX_PERM_Q_ROWS ([fused_layout] permute_wq_b_, q_fused_permutation):
 *     the weight's N = heads * D output rows, cut per head into 16-row chunks,
 *     reordered chunk-major: output row (d / 16) heads 16 + h 16 + d % 16 is
 *     input row h D + d; its ROW32 codes move with their rows (BLK32 codes
 *     cannot: a 32-row block would hold two heads -> MX_ERR_UNSUPPORTED).
 *     Rules: N % heads == 0, D % 16 == 0.
 *   kind MX_PERM_O_COLS ([fused_layout] permute_wo_a_, o_fused_permutation):
 *     the K = heads * D input columns (one group of heads), cut per head into
 *     32-column chunks, reordered chunk-major: output column (c heads + h) 32
 *     + j is input column h D + 32 c + j; each code column (ROW32 or BLK32)
 *     moves with its 32-column chunk.  Rules: K % heads == 0, D % 32 == 0.
 *   w, w_out       (device) E4M3 bytes [N, K], 16-byte aligned, distinct
 *   codes, codes_out (device) ROW32 [N, K/32] or BLK32 [N/32, K/32]
 * Out of place; pack the outputs with mx_pack_weights.  Asynchronous. */
typedef enum { MX_PERM_Q_ROWS = 0, MX_PERM_O_COLS = 1 } mx_perm_kind;
mx_status mx_fused_layout_permute(int kind, int layout, int64_t N, int64_t K, int64_t heads,
                                  const void *w, const void *codes, void *w_out,
                                  void *codes_out, mx_stream_t stream);

/* Per-token MXFP8 activation quantization ([rocm_native] _quant_mxfp8_tile;
 * rule as in mx_quant_rule).
 *   x      (device) bf16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   xq     (device) e4m3 [M, ldq], 16-byte aligned, ldq % 16 == 0, ldq >= K
 *   xcodes (device) E8M0 [M, ldc], ldc >= K / 32
 * Rules: M >= 1, K >= 32, K % 32 == 0.  Bytes and codes are bit-exact with
 * the rule's definition. */
mx_status mx_quant_act(int64_t M, int64_t K, const void *x, int64_t ldx,
                       void *xq, int64_t ldq, void *xcodes, int64_t ldc,
                       int rule, mx_stream_t stream);

/* Sizes (host) of the T16 quantized activation of M tokens x K.
 * Rules: M >= 1, K >= 32, K % 32 == 0. */
mx_status mx_act_t16_sizes(int64_t M, int64_t K, size_t *xq_bytes, size_t *xcodes_bytes);

/* Per-token MXFP8 quantization into the T16 layout: the same bytes and codes
 * as mx_quant_act, rearranged ([rocm_native] _quant_mxfp8_tile).
 *   x      (device) bf16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   xq, xcodes (device) outputs of mx_act_t16_sizes' sizes, 16-byte aligned
 * Every byte of both outputs is written. */
mx_status mx_quant_act_t16(int64_t M, int64_t K, const void *x, int64_t ldx, void *xq,
                           void *xcodes, int rule, mx_stream_t stream);

/* Workspace bytes mx_linear needs for these arguments (0 when none):
 *   act == MX_ACT_MXFP8 quantized inside the call (prequantized = 0): the
 *     T16 activation, round256(MB * S * 2048) + MB * Q * 256;
 *   act == MX_ACT_MXFP8 pre-quantized row-major with M > 64 (prefill GEMM):
 *     the same size: the GEMM reads the T16 layout, so the bytes and codes
 *     are restaged into it (0 in the batch-invariant mode, where the GEMV
 *     reads them as given: see mx_set_batch_invariant);
 *   otherwise 0 (MX_ACT_BF16, MX_ACT_MXFP8_T16, or pre-quantized M <= 64).
 * (K > 8192 with M <= 64 quantized inside the call is the exception: the
 * row-major staging round256(M * Kp) + round256(M * Kp / 32).)
 * E4M3 with M <= 64 quantized inside the call needs none when K % 128 == 0
 * and the decode GEMV's launch plan divides the shape evenly (eight
 * wavefronts of S / 8 steps each, S in {8, 16, 32, 56, 64}, whole tiles per
 * workgroup): the quantization then runs inside the GEMV, with the same bytes
 * and codes as mx_quant_act ([rocm_native] apply_weights fuses it at tiny
 * M).  The environment variable MX_FUSED_QUANT=0, read once per process,
 * turns that off; this function and mx_linear always agree. */
mx_status mx_linear_workspace(int elem, int layout, int64_t N, int64_t K,
                              int64_t M, int act, int prequantized,
                              size_t *bytes);

/* y[M, N] = a . Wf^T (+ bias), bf16 out, fp32 accumulation, one final
 * round to nearest-even bf16 ([rocm_native] apply_weights).
 * Every E8M0 code 0 .. 254 is served exactly on every path: products and
 * partial sums are formed without loss wherever they lie in fp32's normal
 * range.  With bf16 activations the weights are decoded to bf16 with their
 * scale; when a code lies outside 10 .. 246 (E4M3) or 2 .. 252 (E2M1), where
 * a scaled weight would leave bf16's normal range, that work is done on each
 * 32-K block's partial with the scale applied in fp32 instead (slower; such
 * codes mean weights beyond 2^120 or below 2^-117).
 *   Wf[n][k] = dec(W[n][k]) * 2^(code(n, k) - 127) from the packed buffers.
 *   a = x (bf16) when act == MX_ACT_BF16;
 *   a = dec(xq) * 2^(xcode - 127) when act == MX_ACT_MXFP8: if xq and xcodes
 *       are both non-NULL they are used as given (pre-quantized, row-major
 *       codes); otherwise x is quantized first with `rule` into ws;
 *   the same with xq, xcodes in the T16 layout when act == MX_ACT_MXFP8_T16
 *       (ldq, ldc, x and rule unused).
 *   w_packed, codes_packed (device) from mx_pack_weights with the same
 *       elem, layout, E = 1, N, K.
 *   x   (device) bf16 [M, ldx]: 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   xq  (device) e4m3 [M, ldq]: 16-byte aligned, ldq % 16 == 0, ldq >= K
 *   xcodes (device) [M, ldc], ldc >= K / 32
 *   bias (device, nullable) bf16 [N]
 *   y   (device) bf16 [M, ldy]: 16-byte aligned, ldy % 8 == 0, ldy >= N
 *   ws  (device) at least mx_linear_workspace's bytes, 16-byte aligned
 *       (may be NULL when that is 0); its contents on return are unspecified
 * The call is asynchronous on `stream`, allocates nothing and may be
 * captured in a graph.
 * Size limit: every buffer a kernel reads or writes (x, xq, y, the packed
 * weights) must stay below 2 GiB (32-bit buffer offsets), else MX_ERR_SHAPE.
 * Built combinations: E4M3 x {ROW32, BLK32} x {BF16, MXFP8, MXFP8_T16};
 * E2M1 x ROW32 x BF16.  Others: MX_ERR_UNSUPPORTED. */
mx_status mx_linear(int elem, int layout, int64_t N, int64_t K,
                    const void *w_packed, const void *codes_packed, int64_t M,
                    int act, int rule, const void *x, int64_t ldx,
                    const void *xq, int64_t ldq, const void *xcodes,
                    int64_t ldc, const void *bias, void *y, int64_t ldy,
                    void *ws, size_t ws_bytes, mx_stream_t stream);

/* Activations of mx_linear_epilogue: z; max(z, 0); max(z, 0)^2; z / (1 + e^-z);
 * z Phi(z), Phi the normal distribution; z / 2 (1 + tanh(sqrt(2 / pi)
 * (z + 0.044715 z^3))).  At an infinite z they take their limits: +inf, and 0 on the
 * left of all but the first; NaN stays NaN. */
typedef enum {
    MX_FN_NONE = 0,
    MX_FN_RELU = 1,
    MX_FN_RELU2 = 2,
    MX_FN_SILU = 3,
    MX_FN_GELU = 4,
    MX_FN_GELU_TANH = 5
} mx_fn;

/* mx_linear with what follows it in its epilogue:
 *   z[m][n] = the product (+ bias[n])                                    in fp32
 *   gated 0:  y[m][n] = bf16(f(z[m][n]) + residual[m][n])                N columns
 *   gated 1:  y[m][n] = bf16(f(z[m][2 n]) z[m][2 n + 1] + residual[m][n])  N / 2
 *             (gate and up rows interleaved, as mx_moe_copies lays them out; the
 *             bias is of the N rows)
 * f by fn, everything behind the product in fp32 with one rounding at the end: f is
 * within 2^-14 of its value, relative, where that is at least 2^-126.
 *   residual (device, nullable: 0) bf16 [M, ldr], 16-byte aligned, ldr % 8 == 0,
 *            ldr >= the columns; may be y itself (the same pointer and leading
 *            dimension)
 *   y        (device) bf16 [M, ldy], ldy >= the columns
 * Everything else as mx_linear, with the same kernels and workspace
 * (mx_linear_workspace); without activation, gate and residual the results are
 * mx_linear's bit for bit, and z is always summed in its order (the
 * batch-invariant mode included).  Such a call may be the faster one: more than 64 rows
 * over few weight rows take smaller tiles here (M 1001, N 4096, K 1568 12.5 us, mx_linear
 * 22), and a GEMV that quantizes inside larger ones where those save time.
 * Errors: as mx_linear; also MX_ERR_SHAPE when y, the residual or the weights (K
 * rounded up to 128) reach 2 GiB, or when more than 1,048,560 rows would run on a
 * decode kernel (bf16 activations, or the batch-invariant mode);
 * MX_ERR_UNSUPPORTED for an unknown fn or gated, and when y or the workspace
 * overlaps another buffer in any other way than named above. */
mx_status mx_linear_epilogue(int elem, int layout, int64_t N, int64_t K, const void *w_packed,
                             const void *codes_packed, int64_t M, int act, int rule,
                             const void *x, int64_t ldx, const void *xq, int64_t ldq,
                             const void *xcodes, int64_t ldc, const void *bias, int fn, int gated,
                             const void *residual, int64_t ldr, void *y, int64_t ldy, void *ws,
                             size_t ws_bytes, mx_stream_t stream);

/* Workspace bytes mx_moe_linear needs: T * topk * N * 4 when topk_weights is
 * used (combine mode), else 0. */
mx_status mx_moe_workspace(int elem, int64_t E, int64_t N, int64_t K,
                           int64_t T, int64_t topk, int combine,
                           size_t *bytes);

/* Grouped MoE linear over routed experts ([weights942] moe_copies: expert
 * tensors [E, N, K(/2)] with codes [E N, K/32]; [a16w4] module notes):
 *   per slot (topk_weights == NULL): y[t][k][:] = x[t] . Wf[id[t][k]]^T,
 *       y bf16 [T, topk, N] contiguous;
 *   combined (topk_weights != NULL): y[t][:] = sum_k w[t][k] y_slot[t][k][:]
 *       summed in k order in fp32, y bf16 [T, N] contiguous.
 *   w_packed, codes_packed (device) from mx_pack_weights(elem, ROW32, E, N, K)
 *   x (device) bf16 [T, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   topk_ids (device) int32 [T, topk]; an id outside [0, E) gives a zero row
 *   topk_weights (device, nullable) fp32 [T, topk]
 * Rules: T >= 1, 1 <= topk <= E, T * topk <= 4096.  Experts that receive no
 * token read no weight bytes.  Built: E2M1 and E4M3 weights, bf16 x. */
mx_status mx_moe_linear(int elem, int64_t E, int64_t N, int64_t K,
                        const void *w_packed, const void *codes_packed,
                        int64_t T, int64_t topk, const void *x, int64_t ldx,
                        const int32_t *topk_ids, const float *topk_weights,
                        void *y, void *ws, size_t ws_bytes,
                        mx_stream_t stream);

/* mx_moe_linear for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same product with the same kernels and results, but no workspace
 * argument.  The combine's per-slot sums (T * topk * N fp32) go to a device
 * buffer the library holds (4 MiB per GPU, kept until the process ends), so
 * combine mode needs T * topk * N <= 1,048,576; per-slot mode uses no
 * buffer.  The call allocates nothing.  Every call on one GPU shares that
 * buffer: calls that overlap on one GPU (two streams, two threads) race and
 * must be ordered by the caller.  The buffer's contents need no clearing
 * (every value is written before it is read).
 * Errors: as mx_moe_linear; MX_ERR_WORKSPACE when the combine would need
 * more than 4 MiB (checked on the host before any device call). */
mx_status mx_moe_linear_noalloc(int elem, int64_t E, int64_t N, int64_t K,
                                const void *w_packed, const void *codes_packed,
                                int64_t T, int64_t topk, const void *x, int64_t ldx,
                                const int32_t *topk_ids, const float *topk_weights,
                                void *y, mx_stream_t stream);

/* ---- The MoE block around the grouped linear ---- */

/* Load-time expert copies ([weights942] moe_copies).  Input, as a model's
 * checkpoint holds the MoE experts (standard layouts, elem E2M1 or E4M3):
 *   w13 (device) [E, 2 Np, rowb] bytes, rowb = K/2 (E2M1) or K (E4M3): gate
 *       rows 0 .. inter-1, zero rows to Np, up rows Np .. Np+inter-1, zero
 *       rows to 2 Np;  s13 (device) codes [E, 2 Np, K/32];
 *   w2  (device) [E, H, Np values] (Np/2 or Np bytes a row), zero beyond
 *       inter;  s2 (device) codes [E, H, Np/32].
 * Output (device, caller-owned, 16-byte aligned):
 *   w13_out [E, 2 inter, rowb]: gate and up rows interleaved, the even row
 *       2 i holding gate row i and the odd row after it up row i,
 *   s13_out [E, 2 inter, K/32] alike, w2_out [E, H, inter values],
 *   s2_out [E, H, inter/32].
 * Bytes are copied verbatim (-0 nibbles kept).  Then pack them with
 * mx_pack_weights(elem, ROW32, E, 2 inter, K, ...) and
 * mx_pack_weights(elem, ROW32, E, H, inter, ...).
 * Rules: inter % 32 == 0, Np % 32 == 0, inter <= Np, K % 32 == 0, E, H >= 1;
 *   ws (device) at least 256 bytes of scratch.
 * Errors: MX_ERR_VALUE (nothing copied) when a padding byte of w13 or w2 is
 *   not zero, as the page refuses it.  Load-time: the call reads the padding
 *   check back and synchronizes `stream`. */
mx_status mx_moe_copies(int elem, int64_t E, int64_t Np, int64_t inter, int64_t K,
                        int64_t H, const void *w13, const void *s13, const void *w2,
                        const void *s2, void *w13_out, void *s13_out, void *w2_out,
                        void *s2_out, void *ws, size_t ws_bytes, mx_stream_t stream);

/* Up-gate product of the routed experts with the gated activation fused
 * ([weights942] moe_copies pairs each gate row with its up row; the
 * activation is read as SiLU):
 *   h[t k][i] = silu(x[t] . gate_e[i]^T) * (x[t] . up_e[i]^T),  e = id[t][k],
 * fp32 accumulation, silu in fp32, one bf16 rounding.
 *   w13_packed, codes_packed (device): mx_pack_weights(elem, ROW32, E,
 *       2 inter, K) of mx_moe_copies' w13_out / s13_out
 *   x (device) bf16 [T, ldx] as in mx_moe_linear
 *   h (device) bf16 [T topk, ldh], 16-byte aligned, ldh % 8 == 0, ldh >= inter;
 *       a slot whose id is outside [0, E) gets a zero row
 * Rules as mx_moe_linear, with N = 2 inter (inter % 8 == 0). */
mx_status mx_moe_gate_up(int elem, int64_t E, int64_t inter, int64_t K,
                         const void *w13_packed, const void *codes_packed,
                         int64_t T, int64_t topk, const void *x, int64_t ldx,
                         const int32_t *topk_ids, void *h, int64_t ldh,
                         mx_stream_t stream);

/* Down projection of the routed experts on the per-slot hidden rows:
 *   per slot: y[t][k][:] = h[t topk + k] . W2_e^T,  e = id[t][k];
 *   combined (topk_weights != NULL): y[t][:] = sum_k w[t][k] y_slot[t][k][:]
 * (as mx_moe_linear, whose workspace rule applies: mx_moe_workspace(elem, E,
 * H, inter, T, topk, combine)).
 *   w2_packed, codes_packed (device): mx_pack_weights(elem, ROW32, E, H,
 *       inter) of mx_moe_copies' w2_out / s2_out
 *   h (device) bf16 [T topk, ldh] (mx_moe_gate_up's output) */
mx_status mx_moe_down(int elem, int64_t E, int64_t H, int64_t inter,
                      const void *w2_packed, const void *codes_packed,
                      int64_t T, int64_t topk, const void *h, int64_t ldh,
                      const int32_t *topk_ids, const float *topk_weights,
                      void *y, void *ws, size_t ws_bytes, mx_stream_t stream);

/* ---- Around the linear: the norm before it ---- */

/* Residual addition, root-mean-square norm and the quantization of its output
 * in one pass:
 *   s[m][k] = bf16(x[m][k] + residual[m][k])      (residual NULL: s = x)
 *   y[m][k] = bf16(s[m][k] * rsqrt(mean_k(s[m][k]^2) + eps) * weight[k])
 * with the sum of squares and the products in fp32 (each bf16() one rounding to
 * nearest even), and y handed out in the forms that mx_linear and
 * mx_grouped_linear take:
 *   act MX_ACT_BF16       y only
 *   act MX_ACT_MXFP8      xq [M, ldq] and xcodes [M, ldc], as mx_quant_act of y
 *   act MX_ACT_MXFP8_T16  xq and xcodes of mx_act_t16_sizes' sizes, every byte
 *                         written, as mx_quant_act_t16 of y
 * The bytes and codes are exactly those calls' on the bf16 y, also where a value
 * of y is infinite or NaN.  A row's outputs do not depend on M.
 *   x        (device) bf16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   residual (device, nullable) bf16 [M, ldr], the same rules
 *   weight   (device) bf16 [K], 16-byte aligned
 *   eps      >= 0 (0 makes a row of zeros NaN)
 *   sum      (device, nullable) bf16 [M, lds]: receives s; may be x or residual
 *            itself (the same pointer and leading dimension)
 *   y        (device; nullable unless act is MX_ACT_BF16) bf16 [M, ldy]; may be x
 *            or residual itself when sum is not
 *   xq, xcodes (device; unused when act is MX_ACT_BF16): ldq % 16 == 0,
 *            ldq >= K, ldc >= K / 32 (ldq, ldc unused for T16); 16-byte aligned
 *            (xcodes of MX_ACT_MXFP8: any)
 *   rule     as mx_quant_act (checked for every act)
 * Rules: 1 <= M <= 4000000, 32 <= K <= 65536, K % 32 == 0.
 * Errors: MX_ERR_UNSUPPORTED also when an output overlaps another buffer in
 *   any other way than named above. */
mx_status mx_add_rms_norm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *residual,
                          int64_t ldr, const void *weight, float eps, int act, int rule, void *sum,
                          int64_t lds, void *y, int64_t ldy, void *xq, int64_t ldq, void *xcodes,
                          int64_t ldc, mx_stream_t stream);

/* ---- Experts over ragged row ranges (prompts, any number of tokens) ----
 * mx_moe_linear serves decode steps (T * topk <= 4096, bf16 activations).
 * These calls serve any number of tokens on the scaled matrix cores:
 *   mx_moe_sort        the routed pairs in expert order
 *   mx_grouped_linear  one product per expert on its rows, e.g. gate and up
 *                      (MX_EPI_SILU), then down
 *   mx_moe_combine     a token's expert outputs summed with their weights
 * A pair is (token t, choice k), number t * topk + k. */

/* Workspace bytes mx_moe_sort needs (0 for T * topk <= 2048). */
mx_status mx_moe_sort_workspace(int64_t E, int64_t T, int64_t topk, size_t *bytes);

/* The routed pairs in expert order, within an expert by pair number.
 *   topk_ids (device) int32 [T, topk]; an id outside [0, E) takes no expert;
 *            the same id twice in a token is two pairs
 *   offsets  (device) int32 [E + 1]: expert e's pairs have places
 *            offsets[e] .. offsets[e + 1] - 1; offsets[0] = 0
 *   rows     (device) int32 [T topk]: the token of each place, -1 from
 *            offsets[E] on
 *   pos      (device) int32 [T, topk]: the place of each pair, -1 without an
 *            expert
 *   ws       (device) at least mx_moe_sort_workspace's bytes, 16-byte aligned
 *            (may be NULL when that is 0)
 * The result is the same in every run; calls that share a workspace must be
 * ordered.
 * Rules: 1 <= E <= 1024, T >= 1, 1 <= topk <= E, T * topk <= 4000000; the
 * buffers must not overlap (MX_ERR_UNSUPPORTED). */
mx_status mx_moe_sort(int64_t E, int64_t T, int64_t topk, const int32_t *topk_ids,
                      int32_t *offsets, int32_t *rows, int32_t *pos, void *ws, size_t ws_bytes,
                      mx_stream_t stream);

/* Epilogues of mx_grouped_linear. */
typedef enum { MX_EPI_NONE = 0, MX_EPI_SILU = 1 } mx_epi;

/* Workspace bytes mx_grouped_linear needs: the rows' T16 activation
 * (mx_act_t16_sizes of M rows, the first size rounded up to 256) when act is
 * MX_ACT_MXFP8, whether prequantized or not; 0 when act is MX_ACT_MXFP8_T16. */
mx_status mx_grouped_workspace(int elem, int layout, int64_t E, int64_t N, int64_t K, int64_t M,
                               int act, int prequantized, size_t *bytes);

/* Products grouped by expert:
 *   z[i][n] = sum_k a[i][k] Wf[e][n][k]   for offsets[e] <= i < offsets[e + 1]
 *   MX_EPI_NONE  y[i][n] = bf16(z[i][n]),                          N columns
 *   MX_EPI_SILU  y[i][n] = bf16(silu(z[i][2 n]) * z[i][2 n + 1]),  N / 2 columns
 *                (gate and up rows interleaved, as mx_moe_copies lays them out)
 * The scaled matrix cores add the products of eight neighbouring K values at a
 * time, with a last place of 2^-13 of the largest one's binade; these sums, and
 * silu, are in fp32, with one rounding at the end: before it, a product lies
 * within (7 2^-13 + K 2^-23) sum_k |a W| of the exact one, typically within 4e-4
 * of its own size.  Rows of y from offsets[E] on (and before offsets[0]) are left as
 * they were.
 *   w_packed, codes_packed (device) from mx_pack_weights(elem, layout, E, N, K)
 *   M        rows of y, at least offsets[E]
 *   offsets  (device) int32 [E + 1], within 0 .. M and not descending
 *            (mx_moe_sort's); what lies outside 0 .. M is cut off, and with
 *            offsets that descend which rows are written is unspecified
 *   act MX_ACT_MXFP8: row i's activation is source row rows[i] (rows NULL: i,
 *       then xrows >= M); a source row outside [0, xrows) counts as zeros.
 *     x      (device) bf16 [xrows, ldx], 16-byte aligned, ldx % 8 == 0:
 *            quantized with `rule` in the call; or, when xq and xcodes are both
 *            non-NULL, x is unused and
 *     xq     (device) e4m3 [xrows, ldq], 16-byte aligned, ldq % 16 == 0
 *     xcodes (device) E8M0 [xrows, ldc]
 *     rows   (device, nullable) int32 [M]
 *     ws     (device) mx_grouped_workspace's bytes, 16-byte aligned
 *   act MX_ACT_MXFP8_T16: xq, xcodes (device) hold the M rows in the T16 layout
 *       (x, xrows, ldx, ldq, ldc, rule and ws unused, rows must be NULL)
 *   y        (device) bf16 [M, ldy], 16-byte aligned, ldy % 8 == 0
 * Built: E4M3 x {ROW32, BLK32} and E2M1 x ROW32; others, and MX_ACT_BF16, are
 * MX_ERR_UNSUPPORTED, as are outputs that overlap an input.
 * Rules: E <= 65535, 1 <= M <= 4000000; one expert's weights (K rounded up to
 * 128) and 256 rows of y stay below 2 GiB, the staged activation below 256 GiB
 * (MX_ERR_SHAPE).
 * Asynchronous, allocates nothing, may be captured in a graph; calls that share
 * a workspace must be ordered.  The order of summation of an output depends on
 * M, E and N too (two kernels serve the op), unless the batch-invariant mode is
 * on: then it is fixed by K alone, at the decode kernel's speed.
 * The kernel is chosen by M / E, as the host does not see the offsets: its speed
 * assumes that M is close to offsets[E] and the rows are spread over the experts.
 * With few rows an expert on average but most of them on one, that expert's
 * weights are read again for every 16 to 64 of its rows. */
mx_status mx_grouped_linear(int elem, int layout, int64_t E, int64_t N, int64_t K,
                            const void *w_packed, const void *codes_packed, int64_t M,
                            const int32_t *offsets, int act, int rule, int64_t xrows,
                            const void *x, int64_t ldx, const void *xq, int64_t ldq,
                            const void *xcodes, int64_t ldc, const int32_t *rows, int epi, void *y,
                            int64_t ldy, void *ws, size_t ws_bytes, mx_stream_t stream);

/* y[t][:] = sum_k topk_weights[t][k] ys[pos[t][k]][:], in k order in fp32, one
 * rounding to bf16.  A place outside [0, M) adds nothing and its weight is not
 * read; a token without places gets zeros.
 *   ys  (device) bf16 [M, ldys], 16-byte aligned, ldys % 8 == 0, ldys >= N
 *   pos (device) int32 [T, topk] (mx_moe_sort's)
 *   topk_weights (device) fp32 [T, topk]
 *   y   (device) bf16 [T, ldy], 16-byte aligned, ldy % 8 == 0, ldy >= N
 * Rules: T, topk, M >= 1, T * topk and M <= 4000000, N % 8 == 0,
 * N <= 134215680; y overlaps no
 * input (MX_ERR_UNSUPPORTED). */
mx_status mx_moe_combine(int64_t T, int64_t topk, int64_t N, int64_t M, const void *ys,
                         int64_t ldys, const int32_t *pos, const float *topk_weights, void *y,
                         int64_t ldy, mx_stream_t stream);

/* ---- Low-rank adapters beside a projection ---- */

/* Workspace bytes mx_lora_add needs (partial products of x and A in fp32). */
mx_status mx_lora_workspace(int64_t L, int64_t R, int64_t N, int64_t K, int64_t M, size_t *bytes);

/* The adapters of many requests added to a shared projection's output:
 *   y[m][n] = bf16(base[m][n] + scales[g] sum_r (sum_k x[m][k] A[g][r][k]) B[g][n][r])
 * with g = ids[m]; y[m] = base[m] where g is outside [0, L).  Sums in fp32, the
 * inner one kept to 16 significant bits, y rounded once.  Rows in any order.
 * Adapters of smaller rank are padded with zeros to R.
 *   a      (device) bf16 [L, R, K], 16-byte aligned
 *   b      (device) bf16 [L, N, R], 16-byte aligned
 *   scales (device, nullable: 1) fp32 [L]
 *   x      (device) bf16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K: the
 *          projection's input; rows without an adapter are not read
 *   ids    (device) int32 [M]
 *   base   (device) bf16 [M, ldb], 16-byte aligned, ldb % 8 == 0, ldb >= N:
 *          mx_linear's y
 *   y      (device) bf16 [M, ldy], the same rules; may be base itself (the same
 *          pointer and leading dimension)
 *   ws     (device) mx_lora_workspace's bytes, 16-byte aligned
 * Rules: L >= 1, R % 8 == 0, 8 <= R <= 256, K % 32 == 0, N % 16 == 0,
 * 1 <= M <= 4000000; one adapter's A and B and 64 rows of x, base and y stay
 * below 2 GiB; N <= 16776960, K <= 2^26.  Other overlaps of y or ws:
 * MX_ERR_UNSUPPORTED.  Asynchronous, allocates nothing; calls that share a
 * workspace must be ordered.  Below 512 rows the order of summation is fixed by K
 * and R alone; from 512 rows on K is split by M too, so that a row's last bits can
 * change with the number of rows.  In the batch-invariant mode the order below
 * 512 rows serves every M (the workspace's size depends on the mode too). */
mx_status mx_lora_add(int64_t L, int64_t R, int64_t N, int64_t K, const void *a, const void *b,
                      const float *scales, int64_t M, const void *x, int64_t ldx,
                      const int32_t *ids, const void *base, int64_t ldb, void *y, int64_t ldy,
                      void *ws, size_t ws_bytes, mx_stream_t stream);

/* ---- Between the products of a layer ---- */

/* Types of router logits and of a residual stream. */
typedef enum { MX_FLOAT_BF16 = 0, MX_FLOAT_F32 = 1 } mx_float;
/* A router's scores: softmax over all E experts, or a sigmoid of each. */
typedef enum { MX_SCORE_SOFTMAX = 0, MX_SCORE_SIGMOID = 1 } mx_score;

/* The experts of each token, from its router logits x (mx_moe_sort, mx_moe_linear
 * and mx_moe_combine take the result):
 *   s[e] = softmax(x)[e] or sigmoid(x[e]), by score (softmax over all experts whose
 *          logit is not masked, whatever their bias)
 *   c[e] = s[e] + bias[e], a balance that orders but does not weigh; x[e] without a
 *          bias (the same order as the scores', without their rounding)
 *   groups of E / groups neighbouring experts: the topk_groups groups with the
 *          largest sum of their group_best (1 or 2) largest c are kept, equal ones
 *          by lower number (groups 1: all experts)
 *   topk_ids     the topk experts of the kept groups with the largest c, descending,
 *          equal ones by lower number
 *   topk_weights scale * s of the chosen, with renorm 1 divided by their sum (0
 *          where that is 0)
 * With a bias, s is rounded to fp32 from 64 bits, and c and a group's sum in fp32: the
 * choice is a function of the inputs alone.  An expert whose logit or bias is -inf or
 * NaN is masked: its s is 0 and it is not chosen; +inf counts as the largest fp32
 * number.  Choices that find no expert get id -1 and weight 0 (a token whose logits
 * are all masked has none, as a batch's padding); a group with fewer than group_best
 * experts left comes behind all others.  A token's results do not depend on
 * the other tokens or on T.
 *   type     of the logits (mx_float)
 *   logits   (device) [T, ldl], aligned to their elements, ldl >= E
 *   bias     (device, nullable) fp32 [E]
 *   topk_ids (device) int32 [T, topk]
 *   topk_weights (device) fp32 [T, topk]
 * Rules: 1 <= E <= 1024, T >= 1, topk <= 64, T * topk <= 4000000, 1 <= groups <= 64,
 * E % groups == 0, 1 <= topk_groups <= groups, topk <= topk_groups * (E / groups),
 * group_best <= E / groups, a finite scale.
 * Errors: MX_ERR_UNSUPPORTED also for group_best 2 without a bias (zeros will do)
 * and for outputs that overlap another buffer. */
mx_status mx_moe_route(int64_t E, int64_t T, int64_t topk, int type, const void *logits,
                       int64_t ldl, int score, const float *bias, int64_t groups,
                       int64_t topk_groups, int group_best, int renorm, float scale,
                       int32_t *topk_ids, float *topk_weights, mx_stream_t stream);

/* The norms behind a block and ahead of the next one, with the block's gate and the
 * scaled residual stream between them, in one pass:
 *   p[m][k] = x[m][k] * rsqrt(mean_k x[m][k]^2 + eps) * (offset + post_weight[k])
 *             (post_weight NULL: p = x)
 *   s[m][k] = T(alpha * residual[m][k] + gate[g][k] * p[m][k])
 *             (residual NULL: 0; gate NULL: 1)
 *   y[m][k] = bf16(s[m][k] * rsqrt(mean_k s[m][k]^2 + eps) * (offset + weight[k]))
 * in fp32 between the inputs and these roundings (T(), bf16(): to nearest even; p is
 * not rounded), T the residual stream's type; y is handed out as by mx_add_rms_norm:
 *   act MX_ACT_BF16       y only
 *   act MX_ACT_MXFP8      xq [M, ldq] and xcodes [M, ldc], as mx_quant_act of y
 *   act MX_ACT_MXFP8_T16  xq and xcodes of mx_act_t16_sizes' sizes, every byte
 *                         written, as mx_quant_act_t16 of y
 * A row's outputs do not depend on M.
 *   x        (device) bf16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K: the
 *            block's output
 *   post_weight (device, nullable) bf16 [K], 16-byte aligned
 *   gate     (device, nullable) bf16 [gates, ldg], the rules of x; g = gate_ids[m], or
 *            0 without gate_ids; where g is outside [0, gates) the block adds nothing:
 *            s = T(alpha * residual), whatever x, post_weight and the gates hold
 *   gate_ids (device, nullable; unused without a gate) int32 [M]
 *   stream_type  of residual and sum (mx_float)
 *   residual (device, nullable) [M, ldr], 16-byte aligned, rows a multiple of 16 bytes
 *            apart
 *   alpha, offset  finite; offset is 1 where weights are stored around zero
 *   weight   (device, nullable) bf16 [K], 16-byte aligned; without it there is no second
 *            norm: act is MX_ACT_BF16, y NULL, and sum is the only output
 *   eps      >= 0 (0 makes a row of zeros NaN)
 *   sum      (device, nullable with a weight) [M, lds]: receives s; the residual's rules;
 *            may be the residual itself, and, with a bf16 stream, x itself (the same
 *            pointer and leading dimension)
 *   y        (device; nullable unless act is MX_ACT_BF16) bf16 [M, ldy]; may be x itself,
 *            and, with a bf16 stream, the residual itself, when sum is not
 *   xq, xcodes (device; unused when act is MX_ACT_BF16): ldq % 16 == 0,
 *            ldq >= K, ldc >= K / 32 (ldq, ldc unused for T16); 16-byte aligned
 *            (xcodes of MX_ACT_MXFP8: any)
 *   rule     as mx_quant_act (checked for every act)
 * Rules: 1 <= M <= 4000000, 32 <= K <= 65536, K % 32 == 0, gates <= 4000000.
 * Errors: MX_ERR_UNSUPPORTED also when an output overlaps another buffer in any other
 *   way than named above. */
mx_status mx_block_norm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *post_weight,
                        const void *gate, int64_t gates, int64_t ldg, const int32_t *gate_ids,
                        int stream_type, const void *residual, int64_t ldr, float alpha,
                        const void *weight, float offset, float eps, int act, int rule, void *sum,
                        int64_t lds, void *y, int64_t ldy, void *xq, int64_t ldq, void *xcodes,
                        int64_t ldc, mx_stream_t stream);

/* Batch-invariant mode ([rocm_native] process_weights_after_loading: under
 * VLLM_BATCH_INVARIANT the page leaves its block-scaled GEMM, whose split of
 * K varies with M).  Here the decode GEMVs (every A16 call, W8A8 with
 * M <= 64, and the MoE) sum each output in an order fixed by K alone, so a
 * row's result does not depend on the number of rows in the call; W8A8 with
 * M > 64 runs the prefill GEMM, which sums in another order.  With the mode
 * on, W8A8 runs the GEMV for every M: every row's output is then bit-identical
 * to the same row computed in any other call, at the cost of re-reading the
 * weights once per 16 rows.  mx_grouped_linear and mx_lora_add follow the mode
 * too, each as described there.  Process-wide and read once at each call; set it
 * before sizing workspaces (mx_linear_workspace and mx_lora_workspace depend on
 * it).  The environment variable MX_BATCH_INVARIANT=1 turns it on at start-up.
 * Returns the previous setting (0 or 1). */
int mx_set_batch_invariant(int on);

/* Static description of a status code (never NULL).
 * Dispatch trace: with the environment variable MX_LOG=1 (read once per
 * process) mx_linear, the MoE entry points and the operators around the linear
 * write one line to stderr for every kernel they launch, naming the kernel, its launch plan and the
 * shape. */
const char *mx_status_str(mx_status status);

/* Whether an architecture name (e.g. "gfx950:sramecc+:xnack-") is one the
 * kernels are built for; the same test every entry point applies to the
 * current device.  Host only, no device access. */
int mx_arch_supported(const char *gcn_arch_name);

#ifdef __cplusplus
}
#endif
#endif /* MX_H */
