/*
 * mx_experts.h -- C ABI of the routing around a layer of experts: the slots of
 * T tokens with k choices each sorted by expert, token rows gathered in that
 * order, expert outputs summed back with the routing weights, and the gradients
 * of both.
 *
 * A slot s = t k + j is choice j of token t; ids[s] is its expert.  A slot whose
 * id lies outside 0 .. E-1 is dropped: it has no row, adds nothing and gets zero
 * gradients.  Several slots of one token may name the same expert; each has its
 * own row.
 *
 * Sums run over a token's slots in the order j = 0 .. k-1, in fp32, and are
 * rounded once; nothing depends on the order in which blocks run.
 *
 * Conventions as in mx.h; row matrices (X, Xs, Ys, Y and their gradients) may
 * start at any element and have any row stride of at least a row.  ids, weights
 * and plans are dense.  Rows have 1 to 2^31 - 1024 columns (MX_ERR_UNSUPPORTED above).
 * T = 0 is a no-op everywhere but in mx_experts_sort, which writes the empty plan.
 */
#ifndef MX_EXPERTS_H
#define MX_EXPERTS_H

#include "mx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX_EXPERTS_MAX 1024        /* largest E */

/*
 * A plan: the sorted order of T k slots over E experts, in one device buffer of
 * total_bytes bytes made of int32 sections (offsets in bytes, 256-byte aligned):
 *   order   [n]      slot of each sorted row: by expert, then by slot; -1 behind
 *                    the last kept row
 *   pos     [n]      sorted row of each slot, -1 where it is dropped
 *   dest    [n]      row of each slot in the tiled activations (each expert's rows
 *                    start at a multiple of 128), -1 where it is dropped
 *   offsets [E + 1]  first sorted row of each expert; the last entry is the number
 *                    of kept rows
 *   tiles   [E + 1]  first 128-row tile of each expert
 */
typedef struct mx_experts_layout {
    int32_t T, k, E, n;            /* n = T k */
    int32_t max_rows;              /* rows that the tiled activations can take (a multiple of 128) */
    int32_t reserved0;
    uint64_t off_order, off_pos, off_dest, off_offsets, off_tiles, total_bytes;
} mx_experts_layout;

/*
 * mx_experts_layout_init -- host only.  T >= 0, k >= 1, 1 <= E <= MX_EXPERTS_MAX;
 * MX_ERR_UNSUPPORTED when T k exceeds 2^24.
 */
mx_status mx_experts_layout_init(int T, int k, int E, mx_experts_layout* out);

/* mx_experts_sort -- ids device int32 [T k] into plan (P->total_bytes bytes, device). */
mx_status mx_experts_sort(const mx_experts_layout* P, const int32_t* ids, void* plan, void* stream);

/*
 * mx_experts_gather -- Xs[p] = X[order[p] / k] for the kept rows; rows behind
 * them are left as they were.  X [T][ldx], Xs [n][lds], H columns, one type.
 */
mx_status mx_experts_gather(const mx_experts_layout* P, const void* plan, const void* X, mx_dtype dtype, int H,
                            int64_t ldx, void* Xs, int64_t lds, void* stream);

/* mx_experts_gather_bwd -- dX[t] = sum over the token's kept slots of dXs[pos[s]]. */
mx_status mx_experts_gather_bwd(const mx_experts_layout* P, const void* plan, const void* dXs, mx_dtype dtype, int H,
                                int64_t lds, void* dX, int64_t ldx, void* stream);

/*
 * mx_experts_combine -- Y[t] = sum over the token's kept slots of w[s] Ys[pos[s]].
 * Ys [n][lds] of type sdtype, w device fp32 [T k], Y [T][ldy] of type ydtype.
 */
mx_status mx_experts_combine(const mx_experts_layout* P, const void* plan, const void* Ys, mx_dtype sdtype, int H,
                             int64_t lds, const float* w, void* Y, mx_dtype ydtype, int64_t ldy, void* stream);

/*
 * mx_experts_combine_bwd -- the gradients of mx_experts_combine:
 *   dYs[pos[s]] = w[s] dY[t]      (rows behind the last are left as they were)
 *   dw[s]       = sum_h dY[t, h] Ys[pos[s], h], 0 where the slot is dropped
 * dY [T][ldy], Ys [n][lds], dYs [n][ldds] of one type; w, dw device fp32 [T k].
 */
mx_status mx_experts_combine_bwd(const mx_experts_layout* P, const void* plan, const void* dY, const void* Ys,
                                 mx_dtype dtype, int H, int64_t ldy, int64_t lds, const float* w, void* dYs,
                                 int64_t ldds, float* dw, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MX_EXPERTS_H */
