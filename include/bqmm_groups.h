/*
 * bqmm_groups.h -- products whose weights differ from row to row, in the same
 * library (libbqmm.so) and under the same conventions as bqmm.h and
 * bqmm_layer.h: device pointers owned by the caller, no allocation, no host
 * synchronization, work enqueued on `stream`, outputs fully overwritten, the
 * same return codes, and every argument check before any HIP call.
 *
 *   - the experts of a sparse layer: a router's choice, the grouping of its
 *     slots, the MXFP4 products with each expert's weights, plain or as a
 *     gated unit, and the weighted sum of each token's slots;
 *   - low-rank adapters of many requests beside a shared projection.
 *
 * Slots.  Token t's j-th choice of `top` is slot t * top + j, and every tensor
 * of slots stands in that order.  Which rows share weights is found on the
 * device: bqm_group_rows sorts slots by their group, and the products gather
 * and scatter their rows through that order.
 *
 * offsets, order: as bqm_group_rows writes them.  An order entry outside the
 * slots is passed over and offsets outside 0..slots are taken as the nearest
 * end, so no contents lead a call outside its tensors; where the entries are
 * not a permutation, what the outputs hold is unspecified.
 */
#ifndef BQMM_GROUPS_H
#define BQMM_GROUPS_H

#include "bqmm_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of groups (experts, adapters). */
#define BQM_MAX_GROUPS 1024
/* Largest count of bqm_group_rows. */
#define BQM_MAX_ROWS 16777216
/* Largest top of bqm_route and bqm_combine. */
#define BQM_MAX_TOP 32
/* Largest slots and k of bqm_mxfp4_expert_gemv. */
#define BQM_EXPERT_GEMV_MAX_SLOTS 256
#define BQM_EXPERT_GEMV_MAX_K 16384
/* Largest rank of bqm_lora_add. */
#define BQM_LORA_MAX_RANK 256

/*
 * The choice of each token's experts from the router's logits l[t][0..e):
 *   ids[t]     = the `top` largest logits' columns, largest first, the lowest
 *                column first among equals (-0 and +0 are equal);
 *   weights[t] = exp(l[t][id] - max) / sum exp(l[t][j] - max), the sum over
 *                all columns, or with renorm over the chosen ones.
 * A logit that is -inf (a masked expert) or NaN is never chosen: where fewer
 * than `top` are left, the last ids are -1 with weight 0.  A row with a NaN or
 * +inf has NaN for the weights of its other slots.
 *
 *   logits, ld : type [m][e], rows ld >= e elements apart, aligned to an
 *                element.
 *   ids        : int32 [m][top] out;  weights : f32 [m][top] out.
 *   m >= 1, 1 <= e <= BQM_MAX_GROUPS, 1 <= top <= min(e, BQM_MAX_TOP) (else
 *   BQM_EINVAL); m <= 2^25 - 4 (else BQM_EUNSUPPORTED).
 */
int bqm_route(const void *logits, int64_t ld, int type, int top, int renorm, int *ids, float *weights, int m, int e,
              void *stream);

/*
 * Rows sorted by group, rows of a group in their own order:
 *   order[0..count)   = the rows 0..count-1, those of group 0 first, then of
 *                       group 1 and so on, and behind the last group those
 *                       whose id is outside 0..groups-1;
 *   offsets[0..groups] = where each group begins, and the last one ends.
 *
 *   ids       : int32 [count].
 *   offsets   : int32 [groups + 1] out;  order : int32 [count] out.
 *   workspace : bqm_group_rows_workspace(count, groups) bytes, 4-byte aligned;
 *               needs no initial contents; NULL if that is 0.
 *   1 <= count <= BQM_MAX_ROWS, 1 <= groups <= BQM_MAX_GROUPS (else
 *   BQM_EINVAL).
 */
int bqm_group_rows(const int *ids, int count, int groups, int *offsets, int *order, void *workspace, void *stream);

/* Bytes of workspace for bqm_group_rows; 0 for none, -1 for sizes it refuses. */
int64_t bqm_group_rows_workspace(int count, int groups);

/*
 * bqm_mxfp4_gemm with weights that depend on the row.  For slot s of group e,
 * on row s / (slots / rows) of x, with bqm_mxfp4_gemm's sums:
 *   p[s][r] = sum_b 2^(xs + ws - 254) sum_{i in b} e2m1(xq) e2m1(w[e][r]);
 *   glu == 0: y[s][r] = p[s][r], r < n;
 *   glu != 0: y[s][j] = p[s][j] / (1 + exp(-p[s][j])) * p[s][n/2 + j],
 *             j < n/2: the gate's weight rows stand before the other half.
 *             A gate of -inf gives NaN, as the formula does.
 * A slot of no group gets zeros.
 *
 *   w, ws   : codes [groups][n][k/2] and scales [groups][n][k/32].
 *   xq, xs  : codes [rows][k/2] and scales [rows][k/32].
 *   offsets, order : as bqm_group_rows(ids, slots, groups) writes them.
 *   y       : y_type [slots][n or n/2] out, dense, aligned to an element; the
 *             f32 result is rounded once.
 *   rows, slots, n >= 1, slots a multiple of rows, 1 <= groups <=
 *   BQM_MAX_GROUPS, k >= 32, n even with glu (else BQM_EINVAL); k % 32 == 0;
 *   w and xq 16-byte aligned; xq less than 4 GiB; k <= 2^22; and
 *   (slots / 256 + min(slots, groups + 1)) * (n / 256, rounded up) < 2^22
 *   (else BQM_EUNSUPPORTED).
 * Scales as in bqm_mxfp4_gemm.  The order of the sums depends on the sizes, on
 * none of the rows: a slot's result does not depend on the other slots.
 */
int bqm_mxfp4_grouped_gemm(const uint8_t *w, const uint8_t *ws, const uint8_t *xq, const uint8_t *xs,
                           const int *offsets, const int *order, void *y, int y_type, int glu, int rows, int slots,
                           int groups, int k, int n, void *stream);

/*
 * The decode / verify form: few slots, f32 activations, experts by their ids
 * as bqm_route writes them, no grouping needed.  With bqm_mxfp4_gemv's sums
 *   p[s][r] = sum_b 2^(ws - 127) sum_{i in b} x[s / (slots / rows)][i] e2m1(w[ids[s]][r]),
 * y as bqm_mxfp4_grouped_gemm, in f32.  A workgroup takes up to five slots of
 * an expert, as many as the sizes let one expect (one where rows == 1, about
 * twice slots / groups otherwise); an expert of more is read by several, the
 * later ones mostly from the caches.  A slot's result does not depend on the
 * others.
 *
 *   x   : f32 [rows][k], 16-byte aligned, dense.
 *   ids : int32 [slots]; a slot whose id is outside 0..groups-1 gets zeros.
 *   y   : f32 [slots][n or n/2] out.
 *   1 <= slots <= BQM_EXPERT_GEMV_MAX_SLOTS, k <= BQM_EXPERT_GEMV_MAX_K (else
 *   BQM_EUNSUPPORTED for k, BQM_EINVAL for slots), any n; the rest as
 *   bqm_mxfp4_grouped_gemm, scales as in bqm_mxfp4_gemv.
 */
int bqm_mxfp4_expert_gemv(const uint8_t *w, const uint8_t *ws, const float *x, const int *ids, float *y, int glu,
                          int rows, int slots, int groups, int k, int n, void *stream);

/*
 * out[t][i] = (res[t][i] +) sum_j weights[t][j] * y[t * top + j][i], j from 0
 * up, in f32, rounded once; the residual is added last.  A slot whose weight
 * is 0 adds nothing, whatever it holds.
 *
 *   y       : y_type [m * top][n], dense.
 *   weights : f32 [m][top].
 *   res     : out_type [m][n], dense; NULL for none.
 *   out     : out_type [m][n] out, dense; may be res.  out_type is BQM_F32 or
 *             y_type (else BQM_EUNSUPPORTED).
 *   m, n >= 1, 1 <= top <= BQM_MAX_TOP (else BQM_EINVAL).  Every pointer is
 *   aligned to its element; with v = 4 for y of f32 and 8 for 16 bits,
 *   m * (n / v, rounded up) < 2^31 - 255 (else BQM_EUNSUPPORTED).
 */
int bqm_combine(const void *y, int y_type, const float *weights, const void *res, void *out, int out_type, int m,
                int top, int n, void *stream);

/*
 * Low-rank adapters beside a projection.  For row t of adapter e:
 *   h = A[e] x[t],  y[t] = (res[t] +) scale[e] * B[e] h;
 * for a row of no adapter: y[t] = res[t], or zeros.  h is held in f32, and no
 * operand is rounded: sums are f32 throughout.
 *
 *   x, ldx  : x_type [m][k], rows ldx >= k elements apart, 16-byte aligned
 *             rows; x_type is BQM_F32 or ab_type.
 *   a       : ab_type [adapters][r][k], 16-byte aligned.
 *   b       : ab_type [adapters][n][r], 16-byte aligned.  ab_type is BQM_F16
 *             or BQM_BF16.  Adapters of lower rank are padded with zeros.
 *   scale   : f32 [adapters]; NULL for ones.
 *   offsets, order : as bqm_group_rows(ids, m, adapters) writes them for the
 *             rows' adapters.
 *   res, ldr: f32 [m][n], the projection's output, any row stride; NULL for
 *             none.
 *   y, ldy  : f32 [m][n] out; may be res itself (same pointer and stride).
 *   workspace : bqm_lora_add_workspace(m, r) bytes, 16-byte aligned; needs no
 *             initial contents.
 *   m, n, k >= 1, 1 <= r <= BQM_LORA_MAX_RANK, 1 <= adapters <=
 *   BQM_MAX_GROUPS (else BQM_EINVAL); k % 8 == 0, r % 8 == 0, k <= 2^21 and,
 *   with t = m / 16 + min(m, adapters + 1), or m / 32 + min(m, adapters + 1)
 *   from 1024 rows and 64 for each adapter on, t <= 65535 and t * (n rounded
 *   up to 512) < 2^31 (else BQM_EUNSUPPORTED).
 * An infinity or NaN in a row of x makes that row infinite or NaN where its
 * adapter reaches.  Bits of x or h below 2^-133 are lost.  A row's result does
 * not depend on the other rows.
 */
int bqm_lora_add(const void *x, int64_t ldx, int x_type, const void *a, const void *b, int ab_type, const float *scale,
                 const int *offsets, const int *order, const float *res, int64_t ldr, float *y, int64_t ldy,
                 void *workspace, int m, int k, int n, int r, int adapters, void *stream);

/* Bytes of workspace for bqm_lora_add; -1 for m < 1 and r outside 1..BQM_LORA_MAX_RANK. */
int64_t bqm_lora_add_workspace(int m, int r);

#ifdef __cplusplus
}
#endif

#endif /* BQMM_GROUPS_H */
