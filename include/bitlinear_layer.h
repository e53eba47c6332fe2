/*
 * bitlinear_layer.h -- operators that stand around the BitLinear product in a
 * decoder layer, in libbitlinear.so next to the entry points of bitlinear.h
 * and under the same conventions (device pointers to contiguous row-major
 * data, 16-byte aligned; caller-owned workspaces; arguments checked on the
 * host before anything is enqueued; nothing allocated, nothing synchronized,
 * no state between calls; every result deterministic).
 *
 *   norm      h = bf16(x + residual), RMSNorm of h, and the per-token int8
 *             codes and scales of its output: the activations that the
 *             ternary products, the 4-bit products and the gradients below
 *             read.  Its gradient.
 *   backward  gradients of a BitLinear from what it keeps: the 8-bit codes
 *             and scales of its input as activation checkpoint, and its
 *             packed ternary weights.  Rounding steps pass gradients straight
 *             through, as in the Falcon-Edge blog's training form
 *             ("A series of powerful, universal and fine-tunable 1.58-bit
 *             language models").
 *   w4        4-bit weights with group scales times the same int8
 *             activations, for the layers a ternary model keeps in more bits
 *             (the output head).
 *
 * Shapes: as in bitlinear.h (M, N, K >= 1; K % 4 == 0; K <= 2^22; N <= 2^30;
 * M <= 2^24; products below 2^40) unless a function says otherwise.  `stream`
 * belongs to the device that is current in the call.  Inputs
 * must be finite, as there; a value that is not spoils the outputs whose
 * formula reads it, and no others.
 * Two launches that overlap in time must not share a workspace.
 */
#ifndef BITLINEAR_LAYER_H
#define BITLINEAR_LAYER_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of a norm's weight. */
#define BL_WEIGHT_NONE 0 /* no weight: all ones */
#define BL_WEIGHT_BF16 1
#define BL_WEIGHT_F32 2

/* --- residual add, RMSNorm, int8 codes --------------------------------- */

/* For every token row m:
 *   h    = bf16(x + residual)             (h = x where residual is NULL)
 *   rstd = fp32(1 / sqrt(mean_k(h^2) + eps))   (sum, mean and root in fp64)
 *   n    = bf16(fp32(h * rstd) * weight)  (two fp32 products; one without a
 *                                          weight)
 *   x_scale = 127 / max(max_k |n|, 1e-5);  q = clamp(round(n * x_scale), -128, 127)
 * that is, q and x_scale are bitlinear_act_quant of n, bit for bit.
 * x, residual: [M][K] bf16.  weight: [K] of weight_type, NULL for
 * BL_WEIGHT_NONE.  eps: 1e-60 to 1e60.  Written, each NULL where it is not
 * wanted: h [M][K] bf16, rstd [M] fp32, n [M][K] bf16; q [M][K] int8 and
 * x_scale [M] fp32 go together (both or neither).  h may be x or residual
 * themselves (the residual stream updated in place); no other output may
 * overlap an input or another output.  One kernel. */
bl_status bitlinear_rms_norm_quant(int64_t m, int64_t k, const uint16_t *x,
                                   const uint16_t *residual, const void *weight,
                                   int32_t weight_type, double eps, uint16_t *h,
                                   float *rstd, uint16_t *n, int8_t *q,
                                   float *x_scale, void *stream);

/* Bytes of workspace bitlinear_rms_norm_quant_backward needs (0: none). */
size_t bitlinear_rms_norm_quant_backward_workspace_bytes(int64_t m, int64_t k,
                                                         int32_t want_dweight);

/* Gradients of the norm, from the gradient dn [M][K] bf16 of n (that of the
 * codes passes straight through) and dh [M][K] bf16 of h (NULL: none), with
 * h and rstd as the forward call wrote them.  With g = dn * weight and
 * z = h * rstd:
 *   dx      = bf16(rstd * (g - z * mean_k(g * z)) + dh)   -- of x and of residual
 *   dweight = sum_m dn * z                                 (fp32 [K])
 * Sums are fp32.  dweight may be NULL; with accumulate != 0 the sum is added
 * to what dweight holds.  dx may be dn or dh themselves, and must not overlap
 * an input otherwise.  One kernel; two with dweight, but for a few short rows. */
bl_status bitlinear_rms_norm_quant_backward(
    int64_t m, int64_t k, const uint16_t *dn, const uint16_t *h, const float *rstd,
    const void *weight, int32_t weight_type, const uint16_t *dh, uint16_t *dx,
    float *dweight, int32_t accumulate, void *workspace, size_t workspace_bytes,
    void *stream);

/* The activations that 8-bit codes stand for: out[m][k] = bf16(q / x_scale),
 * one correctly rounded fp32 division rounded to bf16 (0 < x_scale <= 2^100).
 * One kernel. */
bl_status bitlinear_restore_activations(int64_t m, int64_t k, const int8_t *q,
                                        const float *x_scale, uint16_t *out,
                                        void *stream);

/* --- forward on int8 codes ---------------------------------------------- */

/* Activations of a projection as bitlinear_rms_norm_quant or
 * bitlinear_act_quant write them (device pointers). */
typedef struct {
  const int8_t *q;      /* [M][K] int8 codes, -127..127 */
  const float *x_scale; /* [M] fp32 scales */
} bl_codes;

/* bitlinear_forward_grouped on activations that are int8 codes already:
 * codes: HOST array of `count`; every projs[i].x must be NULL (BL_EINVAL).
 * Outputs and workspace must not overlap an input or each other, but for a
 * projection's residual that is its own output.
 * Results are those of bitlinear_forward_grouped on the bf16 activations
 * that the codes were made of, bit for bit.  Workspace:
 * bitlinear_forward_grouped_workspace_bytes.  The first kernel brings the
 * codes into the contraction's order; then as bitlinear_forward.  (At M <= 4,
 * where bitlinear_forward_grouped quantizes inside the contraction, that call
 * on the norm's bf16 output is one launch less and faster.) */
bl_status bitlinear_forward_grouped_quantized(int32_t count, const bl_projection *projs,
                                              const bl_codes *codes, int64_t m,
                                              void *workspace, size_t workspace_bytes,
                                              void *stream);

/* --- gradients of BitLinear -------------------------------------------- */

/* Bytes of workspace bitlinear_backward needs for dx and/or dw (0: none, or a
 * shape that it refuses).  Shapes: M and N up to 2^21, M*N up to 2^37, M*K and
 * N*K up to 2^36 (2^22 tiles of 128 x 128, the last ones counted whole). */
size_t bitlinear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k,
                                          int32_t want_dx, int32_t want_dw);

/* Gradients of one BitLinear y = x . u^T / w_scale (+ bias), from dy [M][N]
 * bf16, the gradient of y.  Either part is left out where its output is NULL
 * (its inputs are then not read and may be NULL):
 *
 * of the input, dx = bf16(sum_n dy[m][n] * u[n][k] / w_scale) [M][K] bf16
 *   packed: the layer's weights in `layout` (codes 0..2 only, what
 *   bitlinear_pack_weights writes); w_scale: 1 float.  residual: [M][K] bf16
 *   added to the rounded dx (rounded again), or NULL; may be dx itself, so
 *   that layers that share an input add their gradients up.
 *
 * of the latent weights, dw = sum_m dy[m][n] * xhat[m][k] [N][K] fp32, and of
 * the bias, dbias = sum_m dy[m][n] [N] fp32 (NULL: not wanted; only with dw)
 *   xhat = bf16(q / x_scale), what bitlinear_restore_activations gives, from
 *   the codes q [M][K] and scales x_scale [M] of the layer's input: its 8-bit
 *   checkpoint.  accumulate: 0, or 1 to add to what dw and dbias hold.
 *
 * Products are exact and sums fp32.  One kernel for small shapes (no workspace:
 * the size is 0 and `workspace` may be NULL), else two, or three where a
 * product's sum is split across workgroups. */
bl_status bitlinear_backward(int64_t m, int64_t n, int64_t k, const uint16_t *dy,
                             const uint8_t *packed, int32_t layout,
                             const float *w_scale, const uint16_t *residual,
                             uint16_t *dx, const int8_t *q, const float *x_scale,
                             float *dw, float *dbias, int32_t accumulate,
                             void *workspace, size_t workspace_bytes, void *stream);

/* --- 4-bit weights with group scales ------------------------------------ */

/* Storage.  Weight [n][k] stands for scale * v with v in -8..7, one scale
 * (bf16) per row and group of `group` consecutive k (group a power of two,
 * 32 to 1024; K % group == 0; N up to 2^24).  N is padded to whole blocks of 16 rows and K
 * to whole tiles of 128, with zeros.
 *   codes : bytes [ceil(N/16)][ceil(K/128)][4][16][16]; the byte at
 *           [n/16][k/128][(k%32)/8][n%16][4*((k%128)/32) + k%4] holds the v of
 *           the k with (k % 8) < 4 in its high four bits and that of k + 4 in
 *           its low four bits, as 4-bit two's complement.  A block's tile (1 KB)
 *           is one contiguous read of a 64-lane wavefront, 16 bytes a lane, and
 *           a masked dword is four int8 values 16 v.
 *   scales: bf16 [ceil(N/16)][K/group][16]. */
size_t bitlinear_w4_codes_bytes(int64_t n, int64_t k);
size_t bitlinear_w4_scales_bytes(int64_t n, int64_t k, int64_t group);

/* Quantize latent fp32 weights [N][K]: scale = bf16(max|w| / 7) over the
 * group (1 where that is 0), v = clamp(round(w / scale), -8, 7), one
 * correctly rounded fp32 division each.  One kernel. */
bl_status bitlinear_w4_pack(const float *w, int64_t n, int64_t k, int64_t group,
                            uint8_t *codes, uint16_t *scales, void *stream);

/* The weights that the codes stand for: out[n][k] = fp32(scale * v), exact.
 * One kernel. */
bl_status bitlinear_w4_unpack(const uint8_t *codes, const uint16_t *scales, int64_t n,
                              int64_t k, int64_t group, float *out, void *stream);

/* y = bf16(sum_g scale[n][g] * (sum_{k in g} q[m][k] * v[n][k]) / x_scale[m])
 * [M][N] bf16: exact int32 sums within a group (128 of it at a time), fp32
 * over the groups.  q,
 * x_scale: int8 codes [M][K] and scales [M] of the activations.  bias: [N]
 * bf16, added to the rounded output (rounded again), or NULL.  M up to 2^19.
 * One kernel; the weights are read once for every 16 token rows, so that it is
 * a kernel for up to 16 tokens, and right but slow for many more. */
bl_status bitlinear_w4_forward(int64_t m, int64_t n, int64_t k, int64_t group,
                               const int8_t *q, const float *x_scale,
                               const uint8_t *codes, const uint16_t *scales,
                               const uint16_t *bias, uint16_t *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_LAYER_H */
