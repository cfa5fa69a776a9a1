/*
 * mx_fp4.h -- C ABI of microscaled 4-bit floating point: quantisation of a
 * matrix to E2M1 codes with one 8-bit scale per block of a row, and the product
 * of two such matrices on the block-scaled tensor cores (both operands 4-bit,
 * scales applied by the tensor core, sums in fp32).
 *
 * An E2M1 code is a sign bit and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two formats:
 *   MX_FP4_E4M3_16  blocks of 16 columns, an E4M3 scale s per block and one fp32
 *                   scale g for the whole matrix: value = code * s * g
 *   MX_FP4_E8M0_32  blocks of 32 columns, a power-of-two scale 2^e per block
 *                   (OCP microscaling): value = code * 2^e
 *
 * Quantisation of a block with a = max |x|; fl is one rounding to fp32, e4m3 and
 * e2m1 round to the nearest value of the type, ties to even, and saturate:
 *   MX_FP4_E4M3_16  s = e4m3(fl(a / fl(6 g))), d = fl(s g), code = e2m1(fl(x / d)),
 *                   all codes zero when s is zero
 *   MX_FP4_E8M0_32  e = max(floor(log2 a) - 2, -127), code = e2m1(x / 2^e)
 * A block that holds a NaN or an infinity gets the scale's NaN, so its values are
 * NaN, and so is each output that it takes part in.
 * g is a positive number between 2^-100 and 2^117 (mx_fp4_gscale gives one; values
 * outside are not checked, since g lives on the device).  gA gW may leave fp32's range.
 *
 * Product: Y[m, n] = gA gW sum_k A[m, k] W[n, k] over the codes times their block
 * scales; the products are exact, the sum over k is in fp32 on the tensor cores (K
 * splits, where the path takes them, are added in fp32 in a fixed order), and Y is
 * rounded once to its type.  The same call gives the same bits every time.
 *
 * Conventions as in mx.h: device pointers unless stated, argument errors returned
 * before any launch with the message in mx_last_error(), asynchronous in `stream`.
 * Unlike there, X, Y and dequantised outputs may start at any element and have any
 * row stride of at least a row (16-byte aligned rows are read faster); blobs and
 * workspaces are 16-byte aligned.  The buffers belong to the current device.
 */
#ifndef MX_FP4_H
#define MX_FP4_H

#include "mx.h"
#include "mx_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx_fp4_format { MX_FP4_E4M3_16 = 0, MX_FP4_E8M0_32 = 1 } mx_fp4_format;

#define MX_FP4_KBLOCK 256              /* columns of one stored k-block */
#define MX_FP4_BLOB_MAGIC 0x34465845u  /* first word of a blob */
#define MX_FP4_BLOB_VERSION 1

/*
 * Geometry of `groups` quantised matrices of [rows, K] in one device buffer (one
 * matrix for a linear layer or activations, one per expert for an expert layer):
 *   header   [256 B]  magic, MX_FP4_BLOB_VERSION, rows, K, format, groups
 *   gscale   fp32 [groups]  the matrices' scales g (1 for MX_FP4_E8M0_32)
 *   data     [groups][tiles][kblocks][tile_bytes], a tile being 128 rows and a
 *            k-block 256 columns:
 *     codes  [128 rows][128 B]: two codes a byte, the even column in the low
 *            nibble; the 16-byte chunk holding columns 32c .. 32c+31 of row r
 *            sits at chunk position c XOR (r mod 8)
 *     scales [256 / (4 block)][32][4][4 B]: the scale of row r and block b of
 *            the k-block at byte 512 (b / 4) + 16 (r mod 32) + 4 (r / 32) + b mod 4
 * Columns past K hold zero codes and zero scale bytes.  Rows past `rows` of the
 * last tile are not written and never reach an output.
 */
typedef struct mx_fp4_layout {
    int32_t rows, K, format, groups;
    int32_t block;                 /* columns that share a scale: 16 or 32 */
    int32_t tiles;                 /* ceil(rows / 128), per matrix */
    int32_t kblocks;               /* ceil(K / 256) */
    int32_t tile_bytes;            /* bytes of one (tile, k-block) */
    uint64_t off_gscale, off_data, total_bytes;
} mx_fp4_layout;

/* Options of the products; pass NULL for the defaults (all fields zero). */
typedef struct mx_fp4_opts {
    int32_t path;              /* 0 auto; 1 stream path: one CTA per 128 weight rows and up
                                  to 128 tokens; 2 pair path: 256 weight rows x up to 256
                                  tokens on two SMs */
    int32_t split;             /* stream path: CTAs (one cluster) that share a tile's K range,
                                  0 = auto, 1, 2, 4 or 8 */
    int32_t* status;           /* device int32 or NULL: kernel-side error code */
    int32_t wait_timeout_us;   /* bound on every in-kernel wait (0 = 2 s), in wall time, which also
                                  runs while another process has the GPU; on expiry the kernel writes
                                  MX_ERR_TIMEOUT to *status and returns, parts of Y unwritten */
    int32_t test_stall;        /* testing only: no copies are issued, so the waits run out
                                  (needs status) */
} mx_fp4_opts;

/*
 * mx_fp4_layout_init -- host only.  rows >= 0, K >= 1, groups >= 1.
 * MX_ERR_UNSUPPORTED above 2^31 - 1 rows in all tiles or K above 2^24.
 */
mx_status mx_fp4_layout_init(int rows, int K, int format, int groups, mx_fp4_layout* out);

/* mx_fp4_layout_from_header -- host only; as mx_layout_from_header for these blobs. */
mx_status mx_fp4_layout_from_header(const void* host_header, size_t bytes, mx_fp4_layout* out);

/*
 * mx_fp4_gscale -- a scale for each of the L->groups matrices of X
 * [groups][rows][K] (row stride ldx, matrix stride gsx, in elements):
 * gscale[i] = fl(max |finite x| / 2688), so that the largest block scale is the
 * largest E4M3 number; 1 where the maximum is zero or the quotient is below 2^-100.
 * gscale: device fp32 [groups].
 */
mx_status mx_fp4_gscale(const mx_fp4_layout* L, const void* X, mx_dtype xdtype, int64_t ldx, int64_t gsx,
                        float* gscale, void* stream);

/*
 * mx_fp4_quant -- X [groups][rows][K] (fp32, fp16 or bf16) into blob, whole
 * (L->total_bytes).  gscale: device fp32 [groups], or NULL for g = 1; it must be
 * NULL for MX_FP4_E8M0_32.  rows = 0 writes the header alone.
 */
mx_status mx_fp4_quant(const mx_fp4_layout* L, const void* X, mx_dtype xdtype, int64_t ldx, int64_t gsx,
                       const float* gscale, void* blob, void* stream);

/*
 * mx_fp4_quant_sorted -- activation rows in expert order (mx_experts.h).
 * L has mx_experts_max_rows(P) rows and one group.  The rows of each expert
 * start at a tile of their own (plan section `tiles`), which is what
 * mx_fp4_gemm_sorted reads.
 *   sorted = 0: X is [T][ldx], token rows; sorted row p is token order[p] / k
 *   sorted = 1: X is [n][ldx], rows already in sorted order
 */
mx_status mx_fp4_quant_sorted(const mx_fp4_layout* L, const mx_experts_layout* P, const void* plan, int sorted,
                              const void* X, mx_dtype xdtype, int64_t ldx, const float* gscale, void* blob,
                              void* stream);

/* mx_fp4_dequant -- the values of a blob, out [groups][rows][K] (row stride ldo,
 * matrix stride gso): fl(fl(code * s) * g), then rounded to odtype. */
mx_status mx_fp4_dequant(const mx_fp4_layout* L, const void* blob, void* out, mx_dtype odtype, int64_t ldo,
                         int64_t gso, void* stream);

/*
 * mx_fp4_gemm -- Y [M][ldy] (fp32, fp16 or bf16) = A W^T, with M = LA->rows
 * tokens and N = LW->rows features; both layouts have one group, the same K and
 * format.  M = 0 is a no-op.
 */
mx_status mx_fp4_gemm(const mx_fp4_layout* LW, const void* wblob, const mx_fp4_layout* LA, const void* ablob, void* Y,
                      mx_dtype ydtype, int64_t ldy, const mx_fp4_opts* opts, void* stream);

/*
 * mx_fp4_gemm_sorted -- one product per expert over the sorted rows: for the
 * rows p of expert e, Y[p] = A[p] W[e]^T.  LW has P->E groups; A was written by
 * mx_fp4_quant_sorted with the same plan.  Y: [n][ldy]; rows from offsets[E] on
 * (dropped slots) are left as they were.
 */
mx_status mx_fp4_gemm_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_fp4_layout* LA, const void* ablob,
                             const mx_experts_layout* P, const void* plan, void* Y, mx_dtype ydtype, int64_t ldy,
                             const mx_fp4_opts* opts, void* stream);

/*
 * Bytes of device workspace mx_fp4_linear needs at M tokens: 0 when one kernel
 * quantises and multiplies (up to 4 tokens on the stream path), else room for
 * the quantised activations.
 */
mx_status mx_fp4_linear_workspace_size(const mx_fp4_layout* LW, int M, const mx_fp4_opts* opts, size_t* bytes);

/*
 * mx_fp4_linear -- Y = X W^T in one call, X [M][ldx] quantised with the scale
 * gscale (device fp32 [1] or NULL, as in mx_fp4_quant): one kernel up to 4
 * tokens (stream path; workspace may be NULL), else mx_fp4_quant into the
 * workspace and mx_fp4_gemm, which starts streaming its weights while the
 * quantiser runs.  Y is what mx_fp4_quant and mx_fp4_gemm give, bit for bit.
 */
mx_status mx_fp4_linear(const mx_fp4_layout* LW, const void* wblob, const void* X, mx_dtype xdtype, int M, int64_t ldx,
                        const float* gscale, void* Y, mx_dtype ydtype, int64_t ldy, void* workspace, size_t ws_bytes,
                        const mx_fp4_opts* opts, void* stream);

/* Bytes of device workspace mx_fp4_linear_sorted needs: 0 up to 4 slots on the stream path. */
mx_status mx_fp4_linear_sorted_workspace_size(const mx_fp4_layout* LW, const mx_experts_layout* P,
                                              const mx_fp4_opts* opts, size_t* bytes);

/* mx_fp4_linear_sorted -- mx_fp4_quant_sorted and mx_fp4_gemm_sorted in one call (one kernel up
 * to 4 slots on the stream path). */
mx_status mx_fp4_linear_sorted(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P,
                               const void* plan, int sorted, const void* X, mx_dtype xdtype, int64_t ldx,
                               const float* gscale, void* Y, mx_dtype ydtype, int64_t ldy, void* workspace,
                               size_t ws_bytes, const mx_fp4_opts* opts, void* stream);

/*
 * mx_fp4_experts -- a layer of one projection per expert in one call: mx_experts_sort of ids,
 * mx_fp4_linear_sorted of the token rows X [T][ldx] into fp32 expert outputs, and
 * mx_experts_combine with the routing weights w into Y [T][ldy], which so is
 * rounded once.  The workspace (mx_fp4_experts_workspace_size bytes) holds the
 * plan, at its start, the expert outputs and the quantised activations.
 * T = 0 is a no-op.
 */
mx_status mx_fp4_experts_workspace_size(const mx_fp4_layout* LW, const mx_experts_layout* P, const mx_fp4_opts* opts,
                                        size_t* bytes);
mx_status mx_fp4_experts(const mx_fp4_layout* LW, const void* wblob, const mx_experts_layout* P, const int32_t* ids,
                         const void* X, mx_dtype xdtype, int64_t ldx, const float* gscale, const float* w, void* Y,
                         mx_dtype ydtype, int64_t ldy, void* workspace, size_t ws_bytes, const mx_fp4_opts* opts,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MX_FP4_H */
