/*
 * qmm.h -- C ABI of the quantized projection matmul library (libqmm.so) for
 * AMD Instinct MI355X (gfx950).
 *
 * The library computes the quantized projection matmul of a decoder LLM:
 *   - an int8 x int8 product with int32 accumulation and the zero-point
 *     correction epilogue, plus optional bias, requantisation or fp32 output;
 *   - per-column int8 weight packing (scale = amax/127) and per-row int8
 *     activation quantisation;
 *   - 4-bit q4_1 block weights (bf16 scale and min per 32 values) decoded
 *     inside the kernels, including the mixture-of-experts form that reads
 *     top-k expert ids through a strided view;
 *   - what a step that verifies drafted tokens needs beside the projections:
 *     4-bit weights with group scales, block tables and slot maps built from
 *     request lengths, a paged key/value cache and the attention of a tree of
 *     drafted tokens over it;
 *   - what many requests with long contexts need beside those: a cache held in 4
 *     bits, attention with a sliding window, low-rank adapters of many requests
 *     at once, and log probabilities of given tokens.
 *
 * Sources (web pages, by title and section):
 *  [P1] "The ONNX pack: weights to Q4NX, matmuls to our kernels, no VitisAI"
 *  [P2] "int8 inference" (onemodel docs), "Product kernel (Int8Gemm)"
 *  [P4] "NPU engine: full ELFs, no xclbin", "Q4NX chunks"
 *  [P5] "Zaya 8B Q4NX on the AMD NPU"
 *
 * Common rules for every entry point:
 *   - Pointers named as device pointers refer to GPU memory owned by the
 *     caller; the library never frees or retains them after the call.
 *   - Matrices are row-major with an explicit leading dimension in elements.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream).  Every
 *     call only enqueues work on it and returns; nothing synchronises unless
 *     stated.
 *   - All arguments are checked on the host before anything is enqueued.  On
 *     an error status nothing is enqueued and no output is written.
 *   - QMM_ERR_UNSUPPORTED means well-formed but not covered (the caller is
 *     expected to fall back, as the pages' execution provider does for a
 *     shape it has no kernel for: [P1] "What the graph gives us").
 *   - Results do not depend on the launch configuration: integer outputs are
 *     exact, and floating-point outputs are bitwise reproducible run to run.
 *   - No call allocates device memory (the one device array the library
 *     owns, q4_1_matmul_id_noalloc's scratch, is part of its code object and
 *     placed by the HIP runtime when it loads the kernels on a GPU).  Results depend
 *     only on the arguments: the only state kept between calls is the
 *     process-wide check-mode flag (qmm_set_check), the per-thread
 *     diagnostics (qmm_last_hip_error, qmm_last_variant) and, for
 *     q4_1_matmul_id_noalloc, one library-owned scratch array per GPU.
 *   - Calls on different streams may run concurrently as long as they do not
 *     share an output or a workspace (and, for q4_1_matmul_id_noalloc, not
 *     on the same GPU).
 *   - Workspaces are scratch: no initial contents are needed, every call
 *     writes what it reads, and a workspace may be reused by any later call
 *     on the same stream.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QMM_OK = 0,
    QMM_ERR_INVALID = 1,     /* null pointer, bad size, ld < width, bad zero point   */
    QMM_ERR_UNSUPPORTED = 2, /* valid but not covered (e.g. q4_1 with K % 32 != 0)   */
    QMM_ERR_WORKSPACE = 3,   /* workspace or packed buffer smaller than required     */
    QMM_ERR_HIP = 4          /* a HIP launch failed; see qmm_last_hip_error()         */
} qmm_status;

typedef enum { QMM_S8 = 0, QMM_U8 = 1 } qmm_i8type;

/* Output selectors for qmm_epilogue.outputs (bitwise OR). */
enum {
    QMM_OUT_I32 = 1, /* corrected int32 accumulator                               */
    QMM_OUT_F32 = 2, /* fp32: Y * row_scale[m] * col_scale[n] * scale + bias_f32[n] */
    QMM_OUT_I8 = 4,  /* requantised int8                                          */
    QMM_OUT_U8 = 8   /* requantised uint8 (exclusive with QMM_OUT_I8)             */
};

/*
 * Epilogue of int8_gemm ([P2] "Product kernel": zero-point correction,
 * optional bias, requantisation or float conversion; [P1] "Why it folds
 * without a new kernel" and "What works today": per-axis scales land in the
 * same epilogue, the output scale folds into one multiply per element, the
 * result rounds half to even and the output zero point is added after
 * rounding).
 *
 * With Y the corrected int32 accumulator (wrapping int32 arithmetic) and
 *   mult = fl32(fl32(rs[m] * cs[n]) * scale)   (rs = row_scale or 1,
 *                                               cs = col_scale or the packed
 *                                               weight's column scales)
 * the outputs are
 *   I32 : y_i32[m*ld_i32 + n] = Y
 *   F32 : y_f32[m*ld_f32 + n] = fl32(Y) * mult + bias_f32[n]      (bias 0 if NULL)
 *   I8/U8: acc = Y + bias_i32[n] (int32);  v = fl32(fl32(acc) * mult);
 *          y_q8[m*ld_q8 + n] = clamp(rne(v) + zp_out, -128..127 or 0..255)
 * Any combination of I32, F32 and one of I8/U8 may be requested at once.
 */
typedef struct {
    uint32_t outputs;
    int32_t *y_i32;          /* device, M x N, used with QMM_OUT_I32          */
    int64_t ld_i32;
    float *y_f32;            /* device, M x N, used with QMM_OUT_F32          */
    int64_t ld_f32;
    void *y_q8;              /* device, M x N int8/uint8, with QMM_OUT_I8/U8  */
    int64_t ld_q8;
    const float *row_scale;  /* device [M] or NULL (= 1)                      */
    const float *col_scale;  /* device [N] or NULL (= packed column scales)   */
    float scale;             /* per-tensor factor (e.g. s_x*s_w/s_y)          */
    const float *bias_f32;   /* device [N] or NULL; F32 output only           */
    const int32_t *bias_i32; /* device [N] or NULL; I8/U8 output only         */
    int32_t zp_out;          /* I8: -128..127, U8: 0..255                     */
} qmm_epilogue;

/* ------------------------------------------------------ int8 weight pack --- */

/* Bytes of a packed int8 weight buffer for a K x N weight. */
size_t qmm_pack_b_int8_bytes(int64_t K, int64_t N);

/*
 * pack_b_int8: [P1] "The three layers of the pack": quantise each weight
 * column to int8 with scale = amax/127 and store the column scales alongside
 * the packed buffer; done once per (tensor, K, N).
 *   W       device fp32 K x N, leading dimension ldw >= N (one column per
 *           output feature n).
 *   packed  device buffer of at least qmm_pack_b_int8_bytes(K, N) bytes,
 *           256-byte aligned.  Receives a 64-byte header, the codes in the
 *           library's tile layout, fp32 scale[N] and int32 colsum[N].
 * Per column: s = fl32(amax/127), q = clamp(rne(fl32(w/s)), -127, 127); an
 * all-zero column gets s = 0 and codes 0; colsum[n] = sum_k q.
 */
qmm_status pack_b_int8(const float *W, int64_t K, int64_t N, int64_t ldw,
                       void *packed, size_t packed_bytes, void *stream);

/*
 * pack_b_int8_raw: pack an already-quantised int8/uint8 weight ([P2]
 * "Product kernel": B is stored as int8 and a uint8 B is shifted by 128).
 * Codes are B (int8) or B - 128 (uint8); scales are 1; colsum is the sum of
 * the shifted codes ([P1] "What works today": the weight column sum is
 * computed once and kept).
 */
qmm_status pack_b_int8_raw(const void *B, qmm_i8type bt, int64_t K, int64_t N, int64_t ldb,
                           void *packed, size_t packed_bytes, void *stream);

/*
 * qmm_packed_b_check: synchronously read the header of a packed buffer and
 * check that it was written by this layout version for this K and N
 * (QMM_ERR_INVALID otherwise).  Optional; int8_gemm does not read the header.
 */
qmm_status qmm_packed_b_check(const void *packed, int64_t K, int64_t N, void *stream);

/*
 * quantize_rows_int8: [P1] "The three layers of the pack", item 2: every
 * matmul input is quantised per row with amax/127.
 *   X  device fp32 M x K (ldx >= K);  Xq device int8 M x K (ldq >= K);
 *   row_scale device fp32 [M].  Same rule as pack_b_int8, along rows.
 */
qmm_status quantize_rows_int8(const float *X, int64_t M, int64_t K, int64_t ldx,
                              int8_t *Xq, int64_t ldq, float *row_scale, void *stream);

/* ----------------------------------------------------------- int8 GEMM --- */

/* Workspace bytes int8_gemm needs for an M x K x N product (may be 0). */
size_t qmm_int8_gemm_workspace_bytes(int64_t M, int64_t K, int64_t N);

/*
 * int8_gemm: [P2] "Product kernel (Int8Gemm)":
 *   S[m,n] = sum_k A'[m,k] * B'[k,n]        (int32; primes = shifted domain,
 *                                            A' = A - 128 for uint8 A)
 *   Y[m,n] = S - zA'*colSum[n] - zB'*(rowSum[m] - K*zA')
 * which equals sum_k (A[m,k]-zA)(B[k,n]-zB) exactly whenever that value fits
 * in int32 (always for K <= 33025), then the epilogue above.
 *   A        device, M x K int8 or uint8 (at), leading dimension lda >= K.
 *   zA       activation zero point in at's range.
 *   packedB  buffer written by pack_b_int8 / pack_b_int8_raw for this K, N.
 *   bt       element type the packed weight was given in (QMM_S8 for
 *            pack_b_int8); zB is in that type's range.
 *   workspace  device scratch of qmm_int8_gemm_workspace_bytes(M,K,N) bytes
 *            (256-byte aligned, any contents); NULL when
 *            that size is 0, which it is for every current kernel variant.
 * K must satisfy K*255*128 < 2^31 ([P2]: the sums cannot overflow below that
 * bound), else QMM_ERR_UNSUPPORTED.  M = 0 or N = 0 is a no-op.
 */
qmm_status int8_gemm(const void *A, qmm_i8type at, int64_t M, int64_t K, int64_t lda, int32_t zA,
                     const void *packedB, qmm_i8type bt, int64_t N, int32_t zB,
                     const qmm_epilogue *ep, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * int8_gemm_per_axis: int8_gemm with a zero point per activation row and one
 * per weight column ([P1] "What works today": asymmetric zero points per
 * axis, on the same axes as the per-axis scales, folded into the epilogue):
 *   Y[m,n] = sum_k (A[m,k] - zA_row[m]) * (B[k,n] - zB_col[n])
 *          = S - zA'[m]*colSum[n] - zB'[n]*(rowSum[m] - K*zA'[m])  (int32)
 * then the same epilogue: per-axis scales come through ep->row_scale (s_x[m])
 * and ep->col_scale (s_w[n]), and the QDQ group "int8 in, int8 out" is the
 * I8/U8 output with ep->scale = 1/s_y and ep->zp_out = zp_y.
 *   zA_row   device int32 [M], each in at's range, or NULL (all 0)
 *   zB_col   device int32 [N], each in bt's range, or NULL (all 0)
 * The ranges are a precondition (device data, not checked on the host).
 * Every other argument, the bound on K and the error codes are int8_gemm's.
 */
qmm_status int8_gemm_per_axis(const void *A, qmm_i8type at, int64_t M, int64_t K, int64_t lda,
                              const int32_t *zA_row, const void *packedB, qmm_i8type bt, int64_t N,
                              const int32_t *zB_col, const qmm_epilogue *ep, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Workspace bytes int8_gemm_dynamic needs (0 when the quantisation is fused,
 * see int8_gemm_dynamic). */
size_t qmm_int8_gemm_dynamic_workspace_bytes(int64_t M, int64_t K, int64_t N);

/*
 * int8_gemm_dynamic: the float MatMul route of [P1] "The three layers of the
 * pack" in one call: fp32 activations X (M x K, ldx >= K) are quantised per
 * row with amax/127 (the quantize_rows_int8 rule) and multiplied with a
 * weight packed by pack_b_int8 (zA = zB = 0); the epilogue uses the computed
 * row scales (ep->row_scale must be NULL).  Results are bit-identical to
 * quantize_rows_int8 followed by int8_gemm.  The quantisation runs inside
 * the product kernel (one launch) when K <= 4096 and the rows, cut into
 * G = 1, 2, 4 or 8 groups of R = ceil(M / G), give R' <= 16 and
 * R' * K <= 16384, R' = R rounded up to a power of 2 (G is the smallest one
 * with R' <= 8 if there is one, else the smallest one with R' <= 16); each
 * group is then a grid row that reads the weight once.  Otherwise the two
 * kernels run in turn.  Xq (M x K int8, ldq >= K) and row_scale ([M] fp32)
 * optionally receive the quantised rows and their scales; pass NULL to skip
 * them (the two-kernel form then keeps them in the workspace).
 */
qmm_status int8_gemm_dynamic(const float *X, int64_t M, int64_t K, int64_t ldx,
                             const void *packedB, int64_t N, const qmm_epilogue *ep,
                             int8_t *Xq, int64_t ldq, float *row_scale,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * int8_gemm_dynamic_grouped: int8_gemm_dynamic over several weights that
 * read the same activations (a decoder layer's q, k and v projections, or
 * its gate and up projections), in one launch: [P1] "What works today, and
 * what does not": a decode-side win needs fewer, longer launches.  X (fp32
 * M x K, ldx >= K) is quantised per row with amax/127 once per row group
 * and multiplied with every item's weight; item i writes
 *   items[i].y_f32[m*ld_f32 + n] = fl32(Y_i) * fl32(fl32(rs[m]*cs_i[n])*scale)
 *                                  + bias_f32[n]          (bias 0 if NULL)
 * with Y_i the int32 product with weight i, rs the computed row scales and
 * cs_i the weight's packed column scales: bit for bit what int8_gemm_dynamic
 * with an F32-only epilogue (row_scale NULL, col_scale NULL, that scale and
 * bias) gives for each weight alone.
 *   items     host array of n_items (1..QMM_MAX_GROUP_ITEMS) descriptors; each
 *             packedB was written by pack_b_int8 for this K and its N; items
 *             with N = 0 are skipped.
 *   workspace device scratch of qmm_int8_gemm_dynamic_grouped_workspace_bytes
 *             (M, K) bytes (0, workspace may be NULL, whenever the rows cut
 *             into the row groups of int8_gemm_dynamic's one-launch form;
 *             otherwise the quantised rows and their scales, the rows
 *             quantised once and each item multiplied in a launch of its own).
 * Errors as int8_gemm_dynamic.
 */
#define QMM_MAX_GROUP_ITEMS 4
typedef struct {
    const void *packedB;     /* device, pack_b_int8 buffer for K x N           */
    int64_t N;
    float *y_f32;            /* device, M x N fp32 output                      */
    int64_t ld_f32;
    const float *bias_f32;   /* device [N] or NULL                             */
} qmm_dynamic_item;
size_t qmm_int8_gemm_dynamic_grouped_workspace_bytes(int64_t M, int64_t K);
qmm_status int8_gemm_dynamic_grouped(const float *X, int64_t M, int64_t K, int64_t ldx,
                                     const qmm_dynamic_item *items, int64_t n_items, float scale,
                                     void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------- q4_1 --- */

/*
 * Canonical q4_1 block ([P4] "Q4NX chunks"; [P5] "Round 26": W = q*scale +
 * min with bf16 scale and min per (row, 32-col) block): 32 consecutive k of
 * one output column n, 20 bytes:
 *   bytes 0-1  d  (bf16, little endian), bytes 2-3  m (bf16),
 *   bytes 4-19 codes: byte j holds element j (low nibble) and j+16 (high).
 * value(k) = q(k) * d + m.  A K x N weight is the array blocks[N][K/32].
 */
#define QMM_Q4_1_BLOCK_BYTES 20

/* Bytes of the device layout of a K x N q4_1 weight. */
size_t qmm_q4_1_packed_bytes(int64_t K, int64_t N);

/*
 * q4_1_repack: copy canonical blocks (device, [N][K/32] x 20 bytes) into the
 * library's tile layout (layout only, no arithmetic; [P5] "Milestones": one
 * raw blob plus a tile-major layout read by the kernel).  K % 32 != 0 gives
 * QMM_ERR_UNSUPPORTED.
 */
qmm_status q4_1_repack(const void *blocks, int64_t K, int64_t N,
                       void *packed, size_t packed_bytes, void *stream);

/* Workspace bytes q4_1_matmul needs for M rows. */
size_t qmm_q4_1_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N);

/*
 * q4_1_matmul: Y[m,n] = sum_k X[m,k] * (q[k,n]*d + m) with X fp32 (M x K,
 * ldx >= K), the weight in the layout written by q4_1_repack, Y fp32 (M x N,
 * ldy >= N).  Codes are decoded inside the kernel and kept exact; the
 * relative Frobenius error against exact arithmetic is below 1e-5.
 * workspace: device, >= qmm_q4_1_matmul_workspace_bytes(M,K,N), 256-byte
 * aligned, any contents (the k-split partial sums).  That size is
 * 0 for M <= 4, and for M <= 16 with K <= 1024 (one launch covers the whole
 * k range: no partial sums); workspace may then be NULL.
 */
qmm_status q4_1_matmul(const float *X, int64_t M, int64_t K, int64_t ldx,
                       const void *Wpacked, int64_t N, float *Y, int64_t ldy,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * q4_1_matmul_q8: q4_1 weights against per-row int8 activations (the codes
 * and scales quantize_rows_int8 writes: [P1] "The three layers of the pack",
 * item 2; [P4] "Q4NX chunks" for W = q*d + m):
 *   Y[m,n] = row_scale[m] * sum_b ( d[n,b] * sum_{k in b} q[n,k]*Xq[m,k]
 *                                 + m[n,b] * sum_{k in b} Xq[m,k] )
 * Each block dot and row sum is exact (int32 MFMA); the combination is fp32.
 * It trades the fp32 activations of q4_1_matmul for int8 ones.
 *   Xq         device int8 M x K (ldq >= K); row_scale device fp32 [M]
 *   Wpacked    written by q4_1_repack for this K, N;  Y device fp32 M x N
 * K % 32 != 0 is QMM_ERR_UNSUPPORTED.  Rows run 16 per launch; no workspace.
 */
qmm_status q4_1_matmul_q8(const int8_t *Xq, const float *row_scale, int64_t M, int64_t K, int64_t ldq,
                          const void *Wpacked, int64_t N, float *Y, int64_t ldy, void *stream);

/* Workspace bytes q4_1_matmul_id needs. */
size_t qmm_q4_1_matmul_id_workspace_bytes(int64_t n_tokens, int64_t n_used, int64_t n_expert,
                                          int64_t K, int64_t N);

/*
 * q4_1_matmul_id: MUL_MAT_ID over stacked q4_1 experts ([P5] "The bugs that
 * were the work": the ids are a strided view and must be read through the
 * stride; "What's next": the shared activation form [k, ntokens]).
 * For t < n_tokens and s < n_used:
 *   e = ids[t*ids_row_stride + s];   Y[t*ldy_token + s*ldy_slot + n] = X[t] . W_e[:, n]
 *   X         device fp32 n_tokens x K (ldx >= K)
 *   Wexperts  device, n_expert weights in the q4_1_repack layout, expert e
 *             at byte offset e*expert_stride (>= qmm_q4_1_packed_bytes(K,N))
 *   ids       device int32, row stride ids_row_stride >= n_used; every used
 *             id must lie in [0, n_expert) (a precondition: pairs with other
 *             ids are skipped, and reported in check mode, qmm_set_check)
 * Tokens routed to each expert are grouped on the device (counting sort) and
 * run in one grouped launch.  workspace: >= qmm_q4_1_matmul_id_workspace_bytes,
 * 256-byte aligned, any contents (routing tables and split activations).
 */
qmm_status q4_1_matmul_id(const float *X, int64_t n_tokens, int64_t K, int64_t ldx,
                          const void *Wexperts, int64_t n_expert, int64_t N, size_t expert_stride,
                          const int32_t *ids, int64_t ids_row_stride, int64_t n_used,
                          float *Y, int64_t ldy_slot, int64_t ldy_token,
                          void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes q4_1_matmul_id_per_slot needs. */
size_t qmm_q4_1_matmul_id_per_slot_workspace_bytes(int64_t n_tokens, int64_t n_used, int64_t n_expert,
                                                   int64_t K, int64_t N);

/*
 * q4_1_matmul_id_per_slot: MUL_MAT_ID whose activations hold a row of their
 * own per (token, slot), the per-expert form [k, n_expert_used, ntokens] the
 * down experts read ([P5] "What's next": reading token t's shared row for
 * every slot made every expert compute with the first slot's activation).
 * For t < n_tokens and s < n_used:
 *   e = ids[t*ids_row_stride + s];
 *   Y[t*ldy_token + s*ldy_slot + n] = X[t*ldx_token + s*ldx_slot + :] . W_e[:, n]
 *   X         device fp32, ldx_slot >= K, ldx_token >= n_used*ldx_slot
 * Every other argument, the error codes and the workspace rule are those of
 * q4_1_matmul_id; the workspace grows with n_tokens*n_used activation rows
 * instead of n_tokens.
 */
qmm_status q4_1_matmul_id_per_slot(const float *X, int64_t n_tokens, int64_t K, int64_t ldx_slot,
                                   int64_t ldx_token, const void *Wexperts, int64_t n_expert, int64_t N,
                                   size_t expert_stride, const int32_t *ids, int64_t ids_row_stride,
                                   int64_t n_used, float *Y, int64_t ldy_slot, int64_t ldy_token,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * q4_1_matmul_id_noalloc: q4_1_matmul_id for callers that cannot allocate
 * device memory or pass a workspace (code under HIP graph capture, serving
 * loops, harnesses that forbid allocation).  Same arguments, results (the
 * same kernels, bit for bit), error codes and check mode as q4_1_matmul_id,
 * without the workspace: the routing tables and split activations live in
 * a library-owned device array of QMM_NOALLOC_SCRATCH_BYTES per GPU, created
 * with the library's code object on each GPU it runs on and held until the
 * process ends.  The call itself allocates nothing and never synchronises
 * (outside check mode).
 *   - A call whose workspace (qmm_q4_1_matmul_id_workspace_bytes) exceeds
 *     QMM_NOALLOC_SCRATCH_BYTES returns QMM_ERR_WORKSPACE before anything
 *     is enqueued (16 MiB covers e.g. 512 tokens x top-8 over 128 experts
 *     at K = 2048, which needs about 4.5 MiB).
 *   - Every call on one GPU shares that GPU's array, and nothing in it needs
 *     to start at any value (each call writes everything it reads): calls
 *     that overlap in time on one GPU (different streams, or different host
 *     threads) race and may return wrong results; serialise them.
 *   - The GPU is the one `stream` belongs to (the current device for NULL).
 */
#define QMM_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
qmm_status q4_1_matmul_id_noalloc(const float *X, int64_t n_tokens, int64_t K, int64_t ldx,
                                  const void *Wexperts, int64_t n_expert, int64_t N, size_t expert_stride,
                                  const int32_t *ids, int64_t ids_row_stride, int64_t n_used,
                                  float *Y, int64_t ldy_slot, int64_t ldy_token, void *stream);

/* ------------------------------------------ 4-bit weights, group scales --- */

/* Element types of the calls below. */
typedef enum { QMM_T_F32 = 0, QMM_T_F16 = 1, QMM_T_BF16 = 2, QMM_T_S8 = 3, QMM_T_Q4 = 4 } qmm_dtype;

/*
 * Group-scaled 4-bit weight: the (q - zero) * scale form ([P5] rounds 27/28),
 * which is another format than q4_1's q * d + m.  A K x N weight has
 *   codes   uint8 [N][ceil(K/2)] (row stride ldc >= ceil(K/2) bytes): byte j of row n
 *           holds k = 2j in its low nibble and k = 2j+1 in its high one;
 *   scales  fp16 or bf16 [N][ceil(K/group)] (row stride lds elements): one per
 *           group of `group` consecutive k (the last group may be shorter);
 *   zeros   uint8 [N][ceil(K/group)], values 0..15 (row stride ldz), or NULL:
 *           8 everywhere (the symmetric form).
 * group is 32, 64 or a multiple of 128 (>= K: one scale per column); other
 * groups are QMM_ERR_UNSUPPORTED.  K and N are any positive sizes of fewer than
 * 2^23 strips of 16 columns and 2^26 records of 128 k x 16 columns (64 GiB of
 * codes), else QMM_ERR_UNSUPPORTED.
 */

/* Bytes of the device layout of such a weight (0 for sizes that are refused). */
size_t qmm_q4_group_packed_bytes(int64_t K, int64_t N, int64_t group);

/*
 * q4_group_repack: copy a group-scaled weight (device) into the library's
 * tile layout (256-byte aligned device buffer).  Codes, scales and zeros are
 * kept exactly (zeros beyond 15 are cut to their low four bits).
 */
qmm_status q4_group_repack(const uint8_t *codes, int64_t ldc, const void *scales, qmm_dtype st, int64_t lds,
                           const uint8_t *zeros, int64_t ldz, int64_t K, int64_t N, int64_t group,
                           void *packed, size_t packed_bytes, void *stream);

/* Workspace bytes that suffice for q4_group_matmul, whatever the alignment of its rows. */
size_t qmm_q4_group_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t group, qmm_dtype xt);

/*
 * q4_group_matmul: Y[m,n] = sum_g s[n,g] * sum_{k in g} (q[n,k] - z[n,g]) * X[m,k]
 *   X        device M x K (ldx >= K) of type xt (fp32, fp16 or bf16)
 *   Wpacked  written by q4_group_repack for this K, N, group
 *   Y        device M x N (ldy >= N) of the same type, rounded once from fp32; it
 *            must not share memory with X (INVALID; columns of one matrix are told
 *            apart), nor with the weight or the workspace
 * Codes and activations enter the products exactly (fp32 activations as three
 * bf16 terms that add up to them); sums are fp32.  Outputs whose sums leave fp32's
 * range are computed again from (q - z) s x, term by term, more slowly: an infinite
 * activation makes them infinite, or NaN where its code is the zero, and very large
 * ones give what the definition gives.  M up to 16 * 65520; few rows
 * (up to 64) are what the kernels are made for.  workspace: device, 256-byte
 * aligned, any contents; none is needed for fp16 or bf16 rows that are 16-byte
 * aligned, up to 16 of them, with K >= 8 (else QMM_ERR_WORKSPACE without it).
 */
qmm_status q4_group_matmul(const void *X, qmm_dtype xt, int64_t M, int64_t K, int64_t ldx,
                           const void *Wpacked, int64_t N, int64_t group, void *Y, int64_t ldy,
                           void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------- paged key/value cache --- */

/*
 * A paged cache: num_pages pages of page_size token rows of n_heads x head_dim
 * values, K and V apart and laid out alike.  Element (page, i, head, d) is at
 *   page*page_stride + i*token_stride + head*head_stride + d
 * elements; `slot` p*page_size + i names token row i of page p.  An int8 cache
 * (QMM_T_S8) has an fp32 scale per (token row, head) in k_scale / v_scale, at
 *   page*scale_page_stride + i*scale_token_stride + head*scale_head_stride,
 * and stands for code * scale.  All offsets are 64-bit.
 *
 * A 4-bit cache (QMM_T_Q4) holds head_dim / 2 bytes in a row, and its strides count
 * bytes.  Each 8 elements are a 4-byte word whose nibbles 0..7, from the low end,
 * hold elements 0, 2, 4, 6, 1, 3, 5, 7.  k_scale / v_scale point at pairs of bf16 (4
 * bytes: the step, then the minimum) per (token row, head), the scale strides count
 * pairs, and a row stands for code * step + minimum.
 *
 * Strides are >= 0; rows are 16-byte aligned (the bases and strides; int8 and 4-bit
 * rows: 8 bytes), head_dim is a multiple of 8 (4-bit rows: 16) up to 256 and
 * page_size is below 2^20, else QMM_ERR_UNSUPPORTED.
 */
typedef struct {
    void *k, *v;               /* device                                       */
    qmm_dtype type;            /* QMM_T_F16, QMM_T_BF16, QMM_T_S8 or QMM_T_Q4  */
    int64_t num_pages, page_size, n_heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
    float *k_scale, *v_scale;  /* device; int8 and 4-bit caches, else NULL     */
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
} qmm_kv_cache;

/* Bits of kv_plan's flags (info[2]). */
enum {
    QMM_PLAN_NEGATIVE = 1,   /* a length below zero (taken as zero)              */
    QMM_PLAN_WIDTH = 2,      /* a request longer than its block table row        */
    QMM_PLAN_NO_PAGES = 4,   /* the free list ran out                            */
    QMM_PLAN_MAX_TOKENS = 8, /* more new tokens than max_tokens                  */
    QMM_PLAN_NO_ENTRY = 16   /* a partly filled page without a block table entry */
};

/*
 * kv_plan: block tables and slot maps on the device from request lengths.
 * Request r has ctx_lens[r] tokens in the cache and brings new_lens[r] new
 * ones; page j of its row of the block table holds its tokens from
 * j*page_size on.  With have = ceil(ctx/P) and need = ceil((ctx+new)/P), both
 * at most table_width, the requests take need - have pages each from the free
 * list, in request order, and
 *   block_table[r*ld_table + j] = the page taken, have <= j < need  (other
 *                                 entries stay as they are)
 *   cu_new[r]     = sum of new_lens before r (R + 1 entries)
 *   slots[t]      = block_table[r][pos/P]*P + pos%P and
 *   positions[t]  = pos = ctx_lens[r] + t - cu_new[r] for new token t of r
 *   info          = {pages taken off the list so far, new tokens, flags,
 *                    longest ctx + new}
 * Tokens without a page (flags above) and slots from the last token up to
 * max_tokens get slot -1 (positions 0 from the last token on); page entries
 * past the free list become -1; of tokens past max_tokens nothing is written.
 * Sums are 64-bit and end at 2^31 - 1 where they are stored in 32 bits.
 *   free_pages   device int32 [n_free] page ids
 *   free_begin   device int32: the first id not yet taken (an earlier call's
 *                info[0]; not this call's info), or NULL for 0
 *   slots, positions  device int64 / int32 [max_tokens];  info device int32 [4]
 * R up to 8192 and table_width*page_size < 2^31, else QMM_ERR_UNSUPPORTED.
 */
qmm_status kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, int64_t R, int32_t *block_table,
                   int64_t ld_table, int64_t table_width, int64_t page_size, const int32_t *free_pages,
                   int64_t n_free, const int32_t *free_begin, int64_t max_tokens, int32_t *cu_new,
                   int64_t *slots, int32_t *positions, int32_t *info, void *stream);

/*
 * kv_append: write T token rows of K and V (device, type xt, element (t, head,
 * d) at t*token_stride + head*head_stride + d) to the slots of a cache.
 * 16-bit caches get each value rounded once (to nearest, ties to even); int8
 * caches each row's codes and scale by the rule of quantize_rows_int8 (a row
 * with an infinity or a NaN gets the scale inf or NaN and codes 0); 4-bit caches
 *   minimum = bf16(min x),  step = bf16(fl32(fl32(max x - minimum) / 15)) or 0 if negative,
 *   code = clamp(rne(fl32(fl32(x - minimum) / step)), 0, 15), 0 where the step is 0
 * (a row with an infinity or a NaN, or whose step or minimum is not finite in bf16,
 * gets the step 0, the minimum NaN and codes 0).
 *   slots  device int64 [T]; rows whose slot lies outside [0, num_pages *
 *          page_size) are skipped; no two rows may share a slot.
 * T * n_heads times head_dim / 8 rounded up to a power of two is below 2^32 - 512
 * (else QMM_ERR_UNSUPPORTED).  K and V must not share memory with the cache.
 */
qmm_status kv_append(const void *K, int64_t k_token_stride, int64_t k_head_stride, const void *V,
                     int64_t v_token_stride, int64_t v_head_stride, qmm_dtype xt, int64_t T,
                     const int64_t *slots, const qmm_kv_cache *cache, void *stream);

/*
 * kv_gather: the rows of K and V at T slots of a cache, as values of type xt
 * (fp32, fp16 or bf16): element (t, head, d) at t*token_stride + head*head_stride
 * + d of K and of V.  16-bit rows are converted, int8 rows become code * scale, 4-bit
 * rows code * step + minimum, each value computed in fp32 with one rounding and then
 * rounded to xt.  For rows that another cache or a check needs as values.
 *   slots  device int64 [T], in any order, any of them twice; rows of slots outside
 *          [0, num_pages * page_size) get zeros.
 * K and V must not share memory with each other, the cache or the slots.  The bound on
 * T * n_heads is kv_append's.
 */
qmm_status kv_gather(const int64_t *slots, int64_t T, const qmm_kv_cache *cache, void *K, int64_t k_token_stride,
                     int64_t k_head_stride, void *V, int64_t v_token_stride, int64_t v_head_stride, qmm_dtype xt,
                     void *stream);

/* Workspace bytes that suffice for tree_attention, whatever the table's width. */
size_t qmm_tree_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t R, int64_t n_heads, int64_t head_dim);

/*
 * tree_attention: attention of drafted tokens over a paged cache that already
 * holds their keys and values.  Request r has ctx_lens[r] context tokens and
 * new = cu_new[r+1] - cu_new[r] drafted ones, query rows t = cu_new[r] ... of Q;
 * its tokens 0 .. ctx+new-1 are at block_table[r*ld_table + j/P], row j%P.
 * Query head h reads cache head h / (Hq / n_heads).  With j visible to t when
 * j < ctx, or j = ctx + i with i < new and mask[t*ld_mask + i] != 0 (without a
 * mask: i <= t - cu_new[r]),
 *   O[t,h,:] = sum_j w_j V[j,:],  w = softmax over the visible j of scale * Q[t,h,:].K[j,:]
 * A row that sees no key (or only keys of score -inf) gets zeros.  Keys that
 * a row does not see never reach it, whatever they hold (NaN included).
 *   Q, O  device, element (t, h, d) at t*token_stride + h*head_stride + d, of type
 *         xt: the cache's type, or bf16 for an int8 or 4-bit cache (else UNSUPPORTED).  O
 *         must not share memory with Q (INVALID; rows that alternate with one
 *         stride, as slices of one tensor do, are told apart), nor with any other
 *         argument
 *   mask  device bytes [T][mask_cols] (row stride ld_mask), or NULL; drafted
 *         tokens from mask_cols on are not visible
 *   cu_new  device int32 [R + 1] (kv_plan's); rows of O past cu_new[R] stay as
 *         they are; tokens past table_width * page_size and on pages outside
 *         [0, num_pages) are not visible
 *   workspace  device, 256-byte aligned, any contents
 * Weights enter the products as two terms of the operand type (16 bits and more);
 * over a 4-bit cache with T * (Hq / n_heads) up to 32 R (16 R for head_dim past 128),
 * weight x step enters as one fp16 number, off by 2^-12 of it, in units of code - 8.
 * Sums, maxima and the output before its one rounding are fp32.  Lengths are read
 * on the device only, so a captured call serves any lengths that its table holds.
 * T * (Hq / n_heads) up to 2^30 and table_width * page_size up to 2^31 - 64,
 * else QMM_ERR_UNSUPPORTED.
 */
qmm_status tree_attention(const void *Q, int64_t q_token_stride, int64_t q_head_stride, qmm_dtype xt, int64_t T,
                          int64_t Hq, const qmm_kv_cache *cache, const int32_t *block_table, int64_t ld_table,
                          int64_t table_width, const int32_t *ctx_lens, const int32_t *cu_new, int64_t R,
                          const uint8_t *mask, int64_t ld_mask, int64_t mask_cols, float scale, void *O,
                          int64_t o_token_stride, int64_t o_head_stride, void *workspace, size_t workspace_bytes,
                          void *stream);

/* Workspace bytes that suffice for window_attention, whatever the table's width. */
size_t qmm_window_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t R, int64_t n_heads, int64_t head_dim);

/*
 * window_attention: causal attention over a paged cache that sees the last `window`
 * tokens and the first `sinks`.  Everything is tree_attention's without a mask, but
 * for what a token sees: new token i of request r stands at position
 * pos = ctx_lens[r] + i and sees
 *   j <= pos with j > pos - window or j < sinks.
 * Blocks of keys that no token of a tile sees are not read, and their block table
 * entries may be anything (pages behind the window may have gone back to the free
 * list).  A window of 2^31 - 1 or more is plain causal attention.
 * window < 1 and sinks < 0 are QMM_ERR_INVALID.
 */
qmm_status window_attention(const void *Q, int64_t q_token_stride, int64_t q_head_stride, qmm_dtype xt, int64_t T,
                            int64_t Hq, const qmm_kv_cache *cache, const int32_t *block_table, int64_t ld_table,
                            int64_t table_width, const int32_t *ctx_lens, const int32_t *cu_new, int64_t R,
                            int64_t window, int64_t sinks, float scale, void *O, int64_t o_token_stride,
                            int64_t o_head_stride, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------- adapters, log probabilities --- */

/* Workspace bytes that suffice for lora_matmul. */
size_t qmm_lora_matmul_workspace_bytes(int64_t T, int64_t K, int64_t rank);

/*
 * lora_matmul: low-rank adapters of many requests at once, beside a projection
 * that they share.  With a = adapters[t],
 *   out[t,n] = base[t,n] + scales[a] * sum_i (sum_k X[t,k] * A[a,i,k]) * B[a,n,i]
 * and out[t,n] = base[t,n] for rows whose a lies outside [0, n_adapters).
 *   X     device T x K (ldx >= K) of type xt (fp32, fp16 or bf16)
 *   A, B  device, adapter a at a*a_stride and a*b_stride elements: rank x K (row stride
 *         lda >= K) and N x rank (ldb >= rank) of type wt: xt, or bf16 for fp32 rows
 *         (else QMM_ERR_UNSUPPORTED)
 *   adapters  device int32 [T]; rows of one adapter need not lie together
 *   scales  device fp32 [n_adapters] (alpha / rank), or NULL: 1
 *   base, out  device T x N (ld >= N) of type xt; base may be NULL (zeros) and may be
 *         out itself with the same stride, else the two must not share memory
 *         (INVALID; columns of one matrix are told apart).  out shares memory with
 *         nothing else.
 *   workspace  device, 256-byte aligned, any contents
 * Ranks up to 128 (smaller adapters are padded with zeros).  The inner sums are
 * fp32 and enter the second product as 16 bits and more (fp32 rows: 24), and the
 * sum with base is rounded once.  NaN and infinities of a row or an adapter reach the
 * rows that use it only.  T * ceil(N / 64) is below 2^24 and sizes below 2^30, else
 * QMM_ERR_UNSUPPORTED.
 */
qmm_status lora_matmul(const void *X, qmm_dtype xt, int64_t T, int64_t K, int64_t ldx, const void *A, int64_t a_stride,
                       int64_t lda, const void *B, int64_t b_stride, int64_t ldb, qmm_dtype wt, int64_t n_adapters,
                       int64_t rank, int64_t N, const int32_t *adapters, const float *scales, const void *base,
                       int64_t ld_base, void *out, int64_t ld_out, void *workspace, size_t workspace_bytes, void *stream);

/* Most alternatives that token_logprobs gives. */
#define QMM_MAX_TOP 32

/* Workspace bytes that suffice for token_logprobs. */
size_t qmm_token_logprobs_workspace_bytes(int64_t T, int64_t V);

/*
 * token_logprobs: log probabilities of given tokens, the entropy and the most likely
 * alternatives, from rows of logits read once.  With z = scale * logits[t,:] and
 * lse = log sum_v exp(z_v),
 *   logprobs[t*n + i]  = z[tokens[t*ld_tokens + i]] - lse,  i < n
 *   entropy[t]         = lse - sum_v p_v z_v,  p = exp(z - lse)
 *   top_ids[t*top + i], top_logprobs[t*top + i] = the i-th largest logit's token and z - lse
 * Equal logits (0 and -0 among them) stand in the order of their tokens; a NaN stands
 * with -inf.  Logits of -inf have probability 0 and add nothing to the entropy.
 * Tokens outside [0, V) get -inf, places of the top past V the token -1 and -inf.  A row
 * of nothing but -inf has the entropy 0 and -inf for every token; a row with a NaN or
 * +inf has the entropy NaN and NaN for every token in [0, V).
 *   logits  device T x V (ld >= V) of type xt (fp32, fp16 or bf16)
 *   tokens  device int64 [T][n] (row stride ld_tokens >= n), or NULL with n = 0
 *   logprobs fp32 [T][n], entropy fp32 [T] or NULL, top_ids int64 and top_logprobs
 *         fp32 [T][top], 0 <= top <= QMM_MAX_TOP (else UNSUPPORTED); outputs share
 *         memory with no other argument
 *   scale   finite and positive (1 / temperature)
 *   workspace  device, 256-byte aligned, any contents
 * Sums are fp32.  V up to 2^28 and T * ceil(V / 2048) below 2^24, else UNSUPPORTED.
 */
qmm_status token_logprobs(const void *logits, qmm_dtype xt, int64_t T, int64_t V, int64_t ld, const int64_t *tokens,
                          int64_t ld_tokens, int64_t n, int64_t top, float scale, float *logprobs, float *entropy,
                          int64_t *top_ids, float *top_logprobs, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------- helpers --- */

const char *qmm_status_string(qmm_status s);
/* hipError_t of the last failed HIP call on this thread (0 if none). */
int qmm_last_hip_error(void);
/* Name of the kernel variant the last call on this thread launched
 * (diagnostics; "" before the first call).  With QMM_TRACE=1 in the
 * environment when the library loads, every call also prints its variant
 * (and the int8 products their launch plan) to stderr. */
const char *qmm_last_variant(void);

/*
 * Check mode, a debug aid (off by default; QMM_CHECK=1 in the environment
 * turns it on when the library loads).  While on, calls that can verify
 * device data do so and synchronise the stream: int8_gemm and
 * int8_gemm_per_axis read the packed weight's header (qmm_packed_b_check)
 * and return QMM_ERR_INVALID before launching if it does not match K and N;
 * q4_1_matmul_id and q4_1_matmul_id_per_slot return QMM_ERR_INVALID after the
 * call if an expert id lay outside [0, n_expert) (those pairs' outputs are
 * left unwritten, every other output is written).  The flag is process-wide.
 */
void qmm_set_check(int on);
int qmm_check_enabled(void);

#ifdef __cplusplus
}
#endif
#endif /* QMM_H */
