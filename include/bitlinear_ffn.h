/*
 * bitlinear_ffn.h -- operators of a feed-forward block and of a training step,
 * in libbitlinear.so next to the entry points of bitlinear.h and
 * bitlinear_layer.h and under the same conventions (device pointers to
 * contiguous row-major data, 16-byte aligned unless said otherwise;
 * caller-owned workspaces; arguments checked on the host before anything is
 * enqueued; nothing allocated, nothing synchronized, no state between calls;
 * every result deterministic).
 *
 *   gated     the gate and up projections of a feed-forward block (ternary
 *             weights, int8 activations) with the activation function and the
 *             product of the two, and its gradients
 *   w8        8-bit weights with a scale per output channel times the same
 *             int8 activations, for the layers a ternary model keeps in more
 *             bits, at any number of tokens
 *   clip      the norm of all gradients of a training step together, and the
 *             gradients clipped to it
 *
 * Shapes: as in bitlinear.h (M, N, K >= 1; K % 4 == 0; K <= 2^22; N <= 2^30;
 * M <= 2^24; products below 2^40) unless a function says otherwise; the forward
 * products here take M up to 2^19, N up to 2^24, K up to 2^17 and M * N up to 2^37.
 * `stream` belongs to the device that is current in the call.  Inputs must be
 * finite, as there; a value that is not spoils the outputs whose formula reads
 * it, and no others.  Two launches that overlap in time must not share a workspace.
 */
#ifndef BITLINEAR_FFN_H
#define BITLINEAR_FFN_H

#include "bitlinear_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --- gated feed-forward block ------------------------------------------- */

/* Activation function. */
#define BL_ACT_RELU2 1 /* max(g, 0)^2 */
#define BL_ACT_SILU 2  /* g / (1 + exp(-g)) */

/* Storage of the gate's and the up projection's ternary weights [N][K] each, N
 * padded to whole blocks of 16 rows and K to whole tiles of 256 with zeros: bytes
 * [ceil(N/16)][ceil(K/256)][2][4][16][16], the gate's and the up projection's tile
 * of 16 rows x 256 k in turn, one kilobyte each.  Chunk [g][r] of a tile holds the
 * 64 weights k = 64 g .. 64 g + 63 of row r: weight 16 s + 4 d + j of them in byte
 * 4 s + j at bits 6 - 2 d, as two-bit two's complement (0, 1, -1). */
size_t bitlinear_gated_weights_bytes(int64_t n, int64_t k);

/* Lays packed weights (bitlinear_pack_weights; codes 0..2) out in that storage.
 * Each may be in either layout.  Their scales are not part of it.  One kernel. */
bl_status bitlinear_gated_weights(int64_t n, int64_t k, const uint8_t *gate,
                                  int32_t gate_layout, const uint8_t *up,
                                  int32_t up_layout, uint8_t *codes, void *stream);

/* Bytes of workspace bitlinear_gated_forward needs (0: none, or a shape that it
 * refuses). */
size_t bitlinear_gated_forward_workspace_bytes(int64_t m, int64_t n, int64_t k);

/* From int8 activations q [M][K] with scales x_scale [M], the weights above and
 * their scales (1 float each):
 *   g = acc_gate / (x_scale * gate_scale),  u = acc_up / (x_scale * up_scale)
 *   a = bf16(act(g) * u)                                      [M][N] bf16
 * acc: exact int32 sums; g and u: one correctly rounded fp32 division each; act
 * and the product in fp32 (silu: act(g) first, and exp(-|g|) under 2^-126 is 0).
 * keep_g, keep_u: bf16(g) and bf16(u) [M][N], what the BitLinear projections alone
 * would give and the gradients read; both or neither (NULL).  Outputs and workspace
 * must not overlap an input or each other.  One kernel; one more where K % 16 != 0
 * and the tokens are many (the activations' rows are then aligned first), and one
 * where few tiles' sums are split over K. */
bl_status bitlinear_gated_forward(int64_t m, int64_t n, int64_t k, const int8_t *q,
                                  const float *x_scale, const uint8_t *codes,
                                  const float *gate_scale, const float *up_scale,
                                  int32_t activation, uint16_t *a, uint16_t *keep_g,
                                  uint16_t *keep_u, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Bytes of workspace bitlinear_gated_backward needs for dx and/or dw.  Shapes:
 * those of bitlinear_backward with 2 N outputs. */
size_t bitlinear_gated_backward_workspace_bytes(int64_t m, int64_t n, int64_t k,
                                                int32_t want_dx, int32_t want_dw);

/* Gradients of the block, from da [M][N] bf16, that of a, and the kept g and u
 * [M][N] bf16.  Those of g and u are bf16 values:
 *   dg = bf16(fp32(da * u * act'(g))),  du = bf16(fp32(da * act(g)))
 * (products in fp64 before the rounding to fp32; of relu2 they are exact.)  Either part is
 * left out where its outputs are NULL (its inputs are then not read and may be
 * NULL):
 *   dx = bf16((dg . Ug) / gate_scale + (du . Uu) / up_scale) [M][K]
 *     gate, up: the packed ternary weights [N][K], each in its layout (codes
 *     0..2 only).  residual: [M][K] bf16 added to the rounded dx (rounded
 *     again), or NULL; may be dx itself.
 *   dw_gate = dg^T . xhat,  dw_up = du^T . xhat              [N][K] fp32 each
 *     xhat = bf16(q / x_scale).  Both or neither.  accumulate: 0, or 1 to add to
 *     what they hold.
 * Sums are fp32; dx's gate part is multiplied by up_scale / gate_scale (a normal
 * fp32 value) on the way, and the whole divided by up_scale at the end.  Two
 * kernels, or three where a product's sum is split. */
bl_status bitlinear_gated_backward(
    int64_t m, int64_t n, int64_t k, int32_t activation, const uint16_t *da,
    const uint16_t *g, const uint16_t *u, const uint8_t *gate, int32_t gate_layout,
    const uint8_t *up, int32_t up_layout, const float *gate_scale,
    const float *up_scale, const uint16_t *residual, uint16_t *dx, const int8_t *q,
    const float *x_scale, float *dw_gate, float *dw_up, int32_t accumulate,
    void *workspace, size_t workspace_bytes, void *stream);

/* --- 8-bit weights with a scale per output channel ------------------------ */

/* Storage.  Weight [n][k] stands for scale[n] * v with v in -127..127.  N is
 * padded to whole blocks of 16 rows and K to whole tiles of 64, with zeros:
 *   codes: int8 [ceil(N/16)][ceil(K/64)][4][16][16], [n/16][k/64][(k%64)/16]
 *          [n%16][k%16].
 *   scale: fp32 [N]. */
size_t bitlinear_w8_codes_bytes(int64_t n, int64_t k);

/* Quantize latent fp32 weights [N][K]: scale = max_k|w| / 127 (1 where that is
 * 0), v = clamp(round(w / scale), -127, 127), one correctly rounded fp32
 * division each.  A row with a NaN has the scale NaN, one with an infinity and no NaN
 * an infinite one: none of its outputs is finite.  One kernel. */
bl_status bitlinear_w8_pack(const float *w, int64_t n, int64_t k, int8_t *codes,
                            float *scale, void *stream);

/* The weights that the codes stand for: out[n][k] = fp32(scale * v).  One
 * kernel. */
bl_status bitlinear_w8_unpack(const int8_t *codes, const float *scale, int64_t n,
                              int64_t k, float *out, void *stream);

/* Bytes of workspace bitlinear_w8_forward needs (0: none, or a shape that it
 * refuses). */
size_t bitlinear_w8_forward_workspace_bytes(int64_t m, int64_t n, int64_t k);

/* y = bf16((sum_k q[m][k] * v[n][k]) * scale[n] / x_scale[m]) [M][N] bf16: exact
 * int32 sums, one fp32 product and one division.  q, x_scale: int8 codes [M][K]
 * and scales [M] of the activations.  bias: [N] bf16, added to the rounded output
 * (rounded again), or NULL.  The output and the workspace must not overlap an
 * input or each other.  One kernel; more as bitlinear_gated_forward. */
bl_status bitlinear_w8_forward(int64_t m, int64_t n, int64_t k, const int8_t *q,
                               const float *x_scale, const int8_t *codes,
                               const float *scale, const uint16_t *bias, uint16_t *y,
                               void *workspace, size_t workspace_bytes, void *stream);

/* --- gradient norm and clipping ------------------------------------------ */

#define BL_GRAD_BF16 1
#define BL_GRAD_F32 2

/* One gradient: any number of elements (0 too), contiguous, its pointers aligned
 * to its elements (faster where they are the same modulo 16 bytes). */
typedef struct {
  const void *g;
  void *out;     /* clipped, may be g itself; bitlinear_grad_norm ignores it */
  int64_t numel;
  int32_t type;  /* BL_GRAD_* */
  int32_t reserved; /* must be 0 */
} bl_gradient;

/* Bytes of workspace that the calls below need for these gradients (their numel
 * alone counts; 0: refused).  Up to 2^20 gradients, 2^40 elements in all. */
size_t bitlinear_grad_norm_workspace_bytes(int32_t count, const bl_gradient *grads);

/* norm = fp32(sqrt(sum of g^2 over all elements of all gradients)), 1 float;
 * squares and sums in fp64, in one order whatever the timing.  grads: HOST array
 * of `count`, copied during the call. */
bl_status bitlinear_grad_norm(int32_t count, const bl_gradient *grads, float *norm,
                              void *workspace, size_t workspace_bytes, void *stream);

/* The same norm, and out = g * c rounded to its type, with
 * c = fp32(min(1, max_norm / (norm + 1e-6))), made of the fp64 norm.  A NaN among
 * the gradients makes c and every output NaN, an infinity makes c 0.  max_norm:
 * 0 or more, or infinite (a finite norm is not clipped).  With c = 1, gradients in place
 * are left alone.  Outputs must not overlap a gradient (but their own, exactly),
 * an output or the norm. */
bl_status bitlinear_clip_gradients(int32_t count, const bl_gradient *grads, float max_norm,
                                   float *norm, void *workspace, size_t workspace_bytes,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_FFN_H */
