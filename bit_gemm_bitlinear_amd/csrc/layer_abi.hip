// extern "C" entry points declared in include/bitlinear_layer.h and
// include/bitlinear_ffn.h: host-side argument validation and dispatch.  As in
// abi.hip, no entry point allocates device memory, frees any or synchronizes, and
// every argument is checked before anything is enqueued.
#include "../../include/bitlinear_ffn.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <vector>

#include "internal.hpp"
#include "layer_internal.hpp"

using namespace bl;

namespace {

constexpr int64_t kMaxK = int64_t(1) << 22;
constexpr int64_t kMaxN = int64_t(1) << 30;
constexpr int64_t kMaxM = int64_t(1) << 24;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Grids of the gradients' and the 4-bit kernels: a grid dimension holds 2^32
// threads, the second one 65535 workgroups.
constexpr int64_t kMaxBwdRows = int64_t(1) << 21;
constexpr int64_t kMaxBwdTiles = int64_t(1) << 22;  // 128 x 128 tiles of dx or dw
constexpr int64_t kMaxBwdElems = int64_t(1) << 37;  // of dy or q
constexpr int64_t kMaxW4N = int64_t(1) << 24;
constexpr int64_t kMaxW4M = int64_t(1) << 19;
// 8-bit and gated weights: int32 sums of 128 * 127 (or 128 * 64) a step, the same
// grids, and tiles of 128 x 128 outputs in a grid of 2^32 threads.
constexpr int64_t kMaxSumK = int64_t(1) << 17;
constexpr int64_t kMaxSumOut = int64_t(1) << 37;
constexpr int32_t kMaxGrads = 1 << 20;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bl_status check_ptr(const void* p) {
  if (!p) return BL_EINVAL;
  return aligned16(p) ? BL_OK : BL_EALIGN;
}

bl_status check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps) {
    const bl_status st = check_ptr(p);
    if (st != BL_OK) return st;
  }
  return BL_OK;
}

// Optional pointers: aligned where given.
bl_status check_optional(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return BL_EALIGN;
  return BL_OK;
}

bl_status check_shape(int64_t m, int64_t n, int64_t k) {
  if (m < 1 || n < 1 || k < 1) return BL_ESHAPE;
  if (k % 4 != 0 || k > kMaxK || n > kMaxN || m > kMaxM) return BL_ESHAPE;
  if (m * k >= kMaxElems || n * k >= kMaxElems || m * n >= kMaxElems) return BL_ESHAPE;
  return BL_OK;
}

// Outputs must not overlap inputs or each other.
bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(*o, i)) return false;
    for (const Range* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return false;
  }
  return true;
}

bl_status check_weight(const void* w, int32_t type) {
  if (type == BL_WEIGHT_NONE) return w ? BL_EINVAL : BL_OK;
  if (type != BL_WEIGHT_BF16 && type != BL_WEIGHT_F32) return BL_EINVAL;
  return check_ptr(w);
}

int64_t weight_bytes(int64_t k, int32_t type) {
  return type == BL_WEIGHT_BF16 ? 2 * k : (type == BL_WEIGHT_F32 ? 4 * k : 0);
}

bl_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return need ? BL_EWORKSPACE : BL_OK;
  if (!aligned16(ws)) return BL_EALIGN;
  return have < need ? BL_EWORKSPACE : BL_OK;
}

size_t norm_backward_bytes(int64_t m, int64_t k, bool dweight) {
  const int blocks = norm_backward_blocks(m, k);
  return dweight && blocks > 1 ? align256(sizeof(float) * (size_t)blocks * (size_t)k) : 0;
}

bl_status check_backward_shape(int64_t m, int64_t n, int64_t k) {
  const bl_status st = check_shape(m, n, k);
  if (st != BL_OK) return st;
  if (m > kMaxBwdRows || n > kMaxBwdRows) return BL_ESHAPE;
  if (m * n > kMaxBwdElems || m * k > kMaxBwdElems) return BL_ESHAPE;
  const int64_t ti = (m + 127) / 128, tn = (n + 127) / 128, tk = (k + 127) / 128;
  return ti * tk > kMaxBwdTiles || tn * tk > kMaxBwdTiles ? BL_ESHAPE : BL_OK;
}

bl_status check_w4_shape(int64_t m, int64_t n, int64_t k, int64_t group) {
  const bl_status st = check_shape(m, n, k);
  if (st != BL_OK) return st;
  if (group < 32 || group > 1024 || (group & (group - 1)) != 0) return BL_EINVAL;
  return k % group != 0 || n > kMaxW4N || m > kMaxW4M ? BL_ESHAPE : BL_OK;
}

int64_t w4_codes(int64_t n, int64_t k) { return (n + 15) / 16 * ((k + 127) / 128) * 1024; }
int64_t w4_scales(int64_t n, int64_t k, int64_t group) { return (n + 15) / 16 * (k / group) * 32; }

// Shapes of the 8-bit and the gated products.
bl_status check_sum_shape(int64_t m, int64_t n, int64_t k) {
  const bl_status st = check_shape(m, n, k);
  if (st != BL_OK) return st;
  return k > kMaxSumK || n > kMaxW4N || m > kMaxW4M || m * n > kMaxSumOut ? BL_ESHAPE : BL_OK;
}

int64_t w8_codes(int64_t n, int64_t k) { return (n + 15) / 16 * ((k + 63) / 64) * 1024; }
int64_t gated_codes(int64_t n, int64_t k) { return (n + 15) / 16 * ((k + 255) / 256) * 2048; }

bl_status check_layout(int32_t layout, int64_t n, int64_t k) {
  if (layout == BL_LAYOUT_ROWS) return BL_OK;
  if (layout != BL_LAYOUT_TILED) return BL_EINVAL;
  return n % 16 != 0 || k % 256 != 0 ? BL_ESHAPE : BL_OK;
}

bl_status check_activation(int32_t act) {
  return act == BL_ACT_RELU2 || act == BL_ACT_SILU ? BL_OK : BL_EINVAL;
}

int64_t grad_size(const bl_gradient& g) { return g.type == BL_GRAD_BF16 ? 2 : 4; }

bl_status check_grads(int32_t count, const bl_gradient* g) {
  if (count < 1 || count > kMaxGrads || !g) return BL_EINVAL;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].numel < 0 || g[i].numel > kMaxElems) return BL_ESHAPE;
    if ((total += g[i].numel) > kMaxElems) return BL_ESHAPE;
    if (g[i].type != BL_GRAD_BF16 && g[i].type != BL_GRAD_F32) return BL_EINVAL;
    if (g[i].reserved != 0) return BL_EINVAL;
  }
  return BL_OK;
}

// The gradients' norm, and with `clip` the clipped ones.
bl_status grad_norm(int32_t count, const bl_gradient* grads, bool clip, float max_norm, float* norm,
                    void* workspace, size_t workspace_bytes, void* stream) {
  bl_status st;
  if ((st = check_grads(count, grads)) != BL_OK) return st;
  if ((st = check_ptr(norm)) != BL_OK) return st;
  try {
    std::vector<Gradient> t((size_t)count);
    std::vector<int64_t> numel((size_t)count);
    std::vector<std::pair<Range, bool>> used;  // and whether it is written
    used.reserve(2 * (size_t)count + 2);
    for (int32_t i = 0; i < count; ++i) {
      const bl_gradient& g = grads[i];
      const int64_t size = grad_size(g);
      numel[i] = g.numel;
      t[i] = Gradient{g.g, clip ? g.out : nullptr, g.numel, g.type == BL_GRAD_BF16};
      if (g.numel == 0) continue;
      if (!g.g || (clip && !g.out)) return BL_EINVAL;
      if (reinterpret_cast<uintptr_t>(g.g) % size || (clip && reinterpret_cast<uintptr_t>(g.out) % size))
        return BL_EALIGN;
      const bool in_place = clip && g.out == g.g;
      used.push_back({{g.g, size * g.numel}, in_place});
      if (clip && !in_place) used.push_back({{g.out, size * g.numel}, true});
    }
    const size_t need = grad_norm_bytes(count, numel.data());
    if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
    used.push_back({{norm, 4}, true});
    used.push_back({{workspace, (int64_t)need}, true});
    // In order of their start, a range overlaps an earlier one if it starts before
    // the furthest end so far; of two that are only read that is allowed.
    std::sort(used.begin(), used.end(), [](const auto& a, const auto& b) { return a.first.p < b.first.p; });
    uintptr_t end = 0, written = 0;  // of all, and of those written
    for (const auto& [r, w] : used) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(r.p), e = p + (uintptr_t)r.bytes;
      if (p < (w ? end : written)) return BL_EINVAL;
      end = std::max(end, e);
      if (w) written = std::max(written, e);
    }
    return launch_grad_norm(count, t.data(), clip, max_norm, norm, static_cast<char*>(workspace),
                            static_cast<hipStream_t>(stream)) == hipSuccess
               ? BL_OK
               : BL_EHIP;
  } catch (const std::bad_alloc&) {  // host memory for the lists
    return BL_EHIP;
  }
}

}  // namespace

extern "C" {

bl_status bitlinear_rms_norm_quant(int64_t m, int64_t k, const uint16_t* x,
                                   const uint16_t* residual, const void* weight,
                                   int32_t weight_type, double eps, uint16_t* h, float* rstd,
                                   uint16_t* n, int8_t* q, float* x_scale, void* stream) {
  bl_status st;
  if ((st = check_shape(m, 1, k)) != BL_OK) return st;
  if ((st = check_ptr(x)) != BL_OK || (st = check_weight(weight, weight_type)) != BL_OK) return st;
  if (!(eps >= 1e-60 && eps <= 1e60)) return BL_EINVAL;  // rstd of a zero row fits fp32
  if (!q != !x_scale || (!h && !rstd && !n && !q)) return BL_EINVAL;
  if ((st = check_optional({residual, h, rstd, n, q, x_scale})) != BL_OK) return st;
  const int64_t e = m * k;
  const Range rx = {x, 2 * e}, rr = {residual, 2 * e}, rw = {weight, weight_bytes(k, weight_type)};
  if (!disjoint({{h, 2 * e}, {rstd, 4 * m}, {n, 2 * e}, {q, e}, {x_scale, 4 * m}}, {rw}))
    return BL_EINVAL;
  if (!disjoint({{rstd, 4 * m}, {n, 2 * e}, {q, e}, {x_scale, 4 * m}}, {rx, rr})) return BL_EINVAL;
  if ((h != x && overlap({h, 2 * e}, rx)) || (h != residual && overlap({h, 2 * e}, rr)))
    return BL_EINVAL;
  NormArgs a = {};
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.wtype = weight_type;
  a.k = (int32_t)k;
  a.m = m;
  a.eps = eps;
  a.inv_k = 1.0 / (double)k;
  a.h = h;
  a.rstd = rstd;
  a.n = n;
  a.q = q;
  a.x_scale = x_scale;
  return launch_norm_quant(a, static_cast<hipStream_t>(stream)) == hipSuccess ? BL_OK : BL_EHIP;
}

size_t bitlinear_rms_norm_quant_backward_workspace_bytes(int64_t m, int64_t k,
                                                         int32_t want_dweight) {
  if (check_shape(m, 1, k) != BL_OK) return 0;
  return norm_backward_bytes(m, k, want_dweight != 0);
}

bl_status bitlinear_rms_norm_quant_backward(int64_t m, int64_t k, const uint16_t* dn,
                                            const uint16_t* h, const float* rstd,
                                            const void* weight, int32_t weight_type,
                                            const uint16_t* dh, uint16_t* dx, float* dweight,
                                            int32_t accumulate, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  bl_status st;
  if ((st = check_shape(m, 1, k)) != BL_OK) return st;
  if ((st = check_ptrs({dn, h, rstd, dx})) != BL_OK) return st;
  if ((st = check_weight(weight, weight_type)) != BL_OK) return st;
  if (accumulate != 0 && accumulate != 1) return BL_EINVAL;
  if ((st = check_optional({dh, dweight})) != BL_OK) return st;
  const size_t need = norm_backward_bytes(m, k, dweight != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
  const int64_t e = m * k;
  const Range rdn = {dn, 2 * e}, rh = {h, 2 * e}, rr = {rstd, 4 * m}, rdh = {dh, 2 * e};
  const Range rw = {weight, weight_bytes(k, weight_type)}, rdx = {dx, 2 * e};
  const Range rws = {workspace, (int64_t)need};
  if (!disjoint({rdx, {dweight, 4 * k}, rws}, {rh, rr, rw})) return BL_EINVAL;
  if (!disjoint({{dweight, 4 * k}, rws}, {rdn, rdh})) return BL_EINVAL;
  if ((dx != dn && overlap(rdx, rdn)) || (dx != dh && overlap(rdx, rdh))) return BL_EINVAL;
  NormBwdArgs a = {};
  a.dn = dn;
  a.h = h;
  a.rstd = rstd;
  a.weight = weight;
  a.wtype = weight_type;
  a.k = (int32_t)k;
  a.m = m;
  a.dh = dh;
  a.dx = dx;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.add = 0;
  return launch_norm_backward(a, dweight, accumulate != 0, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? BL_OK
             : BL_EHIP;
}

bl_status bitlinear_restore_activations(int64_t m, int64_t k, const int8_t* q,
                                        const float* x_scale, uint16_t* out, void* stream) {
  bl_status st;
  if ((st = check_shape(m, 1, k)) != BL_OK) return st;
  if ((st = check_ptrs({q, x_scale, out})) != BL_OK) return st;
  if (!disjoint({{out, 2 * m * k}}, {{q, m * k}, {x_scale, 4 * m}})) return BL_EINVAL;
  return launch_restore(q, x_scale, m, k, out, static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t want_dx,
                                          int32_t want_dw) {
  if (check_backward_shape(m, n, k) != BL_OK || (!want_dx && !want_dw)) return 0;
  return backward_bytes(m, n, k, want_dx != 0, want_dw != 0);
}

bl_status bitlinear_backward(int64_t m, int64_t n, int64_t k, const uint16_t* dy,
                             const uint8_t* packed, int32_t layout, const float* w_scale,
                             const uint16_t* residual, uint16_t* dx, const int8_t* q,
                             const float* x_scale, float* dw, float* dbias, int32_t accumulate,
                             void* workspace, size_t workspace_bytes, void* stream) {
  bl_status st;
  if ((st = check_backward_shape(m, n, k)) != BL_OK) return st;
  if (layout != BL_LAYOUT_ROWS && layout != BL_LAYOUT_TILED) return BL_EINVAL;
  if (accumulate != 0 && accumulate != 1) return BL_EINVAL;
  if ((!dx && !dw) || (!dx && residual) || (!dw && dbias)) return BL_EINVAL;
  if ((st = check_ptr(dy)) != BL_OK) return st;
  if (dx) {
    if (layout == BL_LAYOUT_TILED && (n % 16 != 0 || k % 256 != 0)) return BL_ESHAPE;
    if ((st = check_ptrs({packed, w_scale, dx})) != BL_OK) return st;
  }
  if (dw && (st = check_ptrs({q, x_scale, dw})) != BL_OK) return st;
  if ((st = check_optional({residual, dbias})) != BL_OK) return st;
  const size_t need = backward_bytes(m, n, k, dx != nullptr, dw != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
  const Range rdx = {dx, 2 * m * k}, rres = {residual, 2 * m * k}, rws = {workspace, (int64_t)need};
  const Range rdw = {dw, 4 * n * k}, rdb = {dbias, 4 * n}, rdy = {dy, 2 * m * n};
  const Range rp = {dx ? packed : nullptr, n * (k / 4)}, rs = {dx ? w_scale : nullptr, 4};
  const Range rq = {dw ? q : nullptr, m * k}, rx = {dw ? x_scale : nullptr, 4 * m};
  if (!disjoint({rdx, rdw, rdb, rws}, {rdy, rp, rs, rq, rx})) return BL_EINVAL;
  if (overlap(rws, rres) || overlap(rdw, rres) || overlap(rdb, rres)) return BL_EINVAL;
  if (residual != dx && overlap(rdx, rres)) return BL_EINVAL;
  BackwardArgs a = {};
  a.m = m;
  a.n = n;
  a.k = k;
  a.dy = dy;
  a.packed = packed;
  a.tiled = layout == BL_LAYOUT_TILED;
  a.w_scale = w_scale;
  a.residual = residual;
  a.dx = dx;
  a.q = q;
  a.x_scale = x_scale;
  a.dw = dw;
  a.dbias = dbias;
  a.accumulate = accumulate != 0;
  return launch_backward(a, static_cast<char*>(workspace), need, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_w4_codes_bytes(int64_t n, int64_t k) {
  return check_w4_shape(1, n, k, 32) == BL_OK ? (size_t)w4_codes(n, k) : 0;
}

size_t bitlinear_w4_scales_bytes(int64_t n, int64_t k, int64_t group) {
  return check_w4_shape(1, n, k, group) == BL_OK ? (size_t)w4_scales(n, k, group) : 0;
}

bl_status bitlinear_w4_pack(const float* w, int64_t n, int64_t k, int64_t group, uint8_t* codes,
                            uint16_t* scales, void* stream) {
  bl_status st;
  if ((st = check_w4_shape(1, n, k, group)) != BL_OK) return st;
  if ((st = check_ptrs({w, codes, scales})) != BL_OK) return st;
  if (!disjoint({{codes, w4_codes(n, k)}, {scales, w4_scales(n, k, group)}}, {{w, 4 * n * k}}))
    return BL_EINVAL;
  return launch_w4_pack(w, n, k, (int)group, codes, scales, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? BL_OK
             : BL_EHIP;
}

bl_status bitlinear_w4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t n, int64_t k,
                              int64_t group, float* out, void* stream) {
  bl_status st;
  if ((st = check_w4_shape(1, n, k, group)) != BL_OK) return st;
  if ((st = check_ptrs({codes, scales, out})) != BL_OK) return st;
  if (!disjoint({{out, 4 * n * k}}, {{codes, w4_codes(n, k)}, {scales, w4_scales(n, k, group)}}))
    return BL_EINVAL;
  return launch_w4_unpack(codes, scales, n, k, (int)group, out,
                          static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

bl_status bitlinear_w4_forward(int64_t m, int64_t n, int64_t k, int64_t group, const int8_t* q,
                               const float* x_scale, const uint8_t* codes, const uint16_t* scales,
                               const uint16_t* bias, uint16_t* y, void* stream) {
  bl_status st;
  if ((st = check_w4_shape(m, n, k, group)) != BL_OK) return st;
  if ((st = check_ptrs({q, x_scale, codes, scales, y})) != BL_OK) return st;
  if ((st = check_optional({bias})) != BL_OK) return st;
  if (!disjoint({{y, 2 * m * n}}, {{q, m * k}, {x_scale, 4 * m}, {codes, w4_codes(n, k)},
                                   {scales, w4_scales(n, k, group)}, {bias, 2 * n}}))
    return BL_EINVAL;
  return launch_w4_forward(m, n, k, (int)group, q, x_scale, codes, scales, bias, y,
                           static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_gated_weights_bytes(int64_t n, int64_t k) {
  return check_sum_shape(1, n, k) == BL_OK ? (size_t)gated_codes(n, k) : 0;
}

bl_status bitlinear_gated_weights(int64_t n, int64_t k, const uint8_t* gate, int32_t gate_layout,
                                  const uint8_t* up, int32_t up_layout, uint8_t* codes,
                                  void* stream) {
  bl_status st;
  if ((st = check_sum_shape(1, n, k)) != BL_OK) return st;
  if ((st = check_layout(gate_layout, n, k)) != BL_OK) return st;
  if ((st = check_layout(up_layout, n, k)) != BL_OK) return st;
  if ((st = check_ptrs({gate, up, codes})) != BL_OK) return st;
  if (!disjoint({{codes, gated_codes(n, k)}}, {{gate, n * (k / 4)}, {up, n * (k / 4)}})) return BL_EINVAL;
  return launch_gated_weights(gate, gate_layout == BL_LAYOUT_TILED, up, up_layout == BL_LAYOUT_TILED, n,
                              k, codes, static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_gated_forward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return check_sum_shape(m, n, k) == BL_OK ? gated_forward_bytes(m, n, k) : 0;
}

bl_status bitlinear_gated_forward(int64_t m, int64_t n, int64_t k, const int8_t* q,
                                  const float* x_scale, const uint8_t* codes,
                                  const float* gate_scale, const float* up_scale, int32_t activation,
                                  uint16_t* a, uint16_t* keep_g, uint16_t* keep_u, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  bl_status st;
  if ((st = check_sum_shape(m, n, k)) != BL_OK) return st;
  if ((st = check_activation(activation)) != BL_OK) return st;
  if (!keep_g != !keep_u) return BL_EINVAL;
  if ((st = check_ptrs({q, x_scale, codes, gate_scale, up_scale, a})) != BL_OK) return st;
  if ((st = check_optional({keep_g, keep_u})) != BL_OK) return st;
  const size_t need = gated_forward_bytes(m, n, k);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
  const int64_t e = 2 * m * n;
  if (!disjoint({{a, e}, {keep_g, e}, {keep_u, e}, {workspace, (int64_t)need}},
                {{q, m * k}, {x_scale, 4 * m}, {codes, gated_codes(n, k)}, {gate_scale, 4}, {up_scale, 4}}))
    return BL_EINVAL;
  const GatedArgs args = {m, n, k, q, x_scale, codes, gate_scale, up_scale, activation == BL_ACT_SILU,
                          a, keep_g, keep_u};
  return launch_gated_forward(args, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_gated_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t want_dx,
                                                int32_t want_dw) {
  if (n < 1 || n > kMaxN || check_backward_shape(m, 2 * n, k) != BL_OK || (!want_dx && !want_dw)) return 0;
  return gated_backward_bytes(m, n, k, want_dx != 0, want_dw != 0);
}

bl_status bitlinear_gated_backward(int64_t m, int64_t n, int64_t k, int32_t activation,
                                   const uint16_t* da, const uint16_t* g, const uint16_t* u,
                                   const uint8_t* gate, int32_t gate_layout, const uint8_t* up,
                                   int32_t up_layout, const float* gate_scale, const float* up_scale,
                                   const uint16_t* residual, uint16_t* dx, const int8_t* q,
                                   const float* x_scale, float* dw_gate, float* dw_up,
                                   int32_t accumulate, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  bl_status st;
  if (n < 1 || n > kMaxN) return BL_ESHAPE;
  if ((st = check_backward_shape(m, 2 * n, k)) != BL_OK) return st;
  if ((st = check_activation(activation)) != BL_OK) return st;
  if (accumulate != 0 && accumulate != 1) return BL_EINVAL;
  if (!dw_gate != !dw_up || (!dx && !dw_gate) || (!dx && residual)) return BL_EINVAL;
  if ((st = check_ptrs({da, g, u})) != BL_OK) return st;
  if (dx) {
    if ((st = check_layout(gate_layout, n, k)) != BL_OK) return st;
    if ((st = check_layout(up_layout, n, k)) != BL_OK) return st;
    if ((st = check_ptrs({gate, up, gate_scale, up_scale, dx})) != BL_OK) return st;
  }
  if (dw_gate && (st = check_ptrs({q, x_scale, dw_gate, dw_up})) != BL_OK) return st;
  if ((st = check_optional({residual})) != BL_OK) return st;
  const size_t need = gated_backward_bytes(m, n, k, dx != nullptr, dw_gate != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
  const int64_t e = 2 * m * n;
  const Range rdx = {dx, 2 * m * k}, rres = {residual, 2 * m * k}, rws = {workspace, (int64_t)need};
  const Range rwg = {dw_gate, 4 * n * k}, rwu = {dw_up, 4 * n * k};
  const Range rpg = {dx ? gate : nullptr, n * (k / 4)}, rpu = {dx ? up : nullptr, n * (k / 4)};
  const Range rsg = {dx ? gate_scale : nullptr, 4}, rsu = {dx ? up_scale : nullptr, 4};
  const Range rq = {dw_gate ? q : nullptr, m * k}, rx = {dw_gate ? x_scale : nullptr, 4 * m};
  if (!disjoint({rdx, rwg, rwu, rws}, {{da, e}, {g, e}, {u, e}, rpg, rpu, rsg, rsu, rq, rx}))
    return BL_EINVAL;
  if (!disjoint({rwg, rwu, rws}, {rres}) || (residual != dx && overlap(rdx, rres))) return BL_EINVAL;
  GatedBackwardArgs a = {};
  a.m = m;
  a.n = n;
  a.k = k;
  a.silu = activation == BL_ACT_SILU;
  a.da = da;
  a.g = g;
  a.u = u;
  a.gate = gate;
  a.up = up;
  a.gate_tiled = gate_layout == BL_LAYOUT_TILED;
  a.up_tiled = up_layout == BL_LAYOUT_TILED;
  a.gate_scale = gate_scale;
  a.up_scale = up_scale;
  a.residual = residual;
  a.dx = dx;
  a.q = q;
  a.x_scale = x_scale;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  a.accumulate = accumulate != 0;
  return launch_gated_backward(a, static_cast<char*>(workspace), need,
                               static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_w8_codes_bytes(int64_t n, int64_t k) {
  return check_sum_shape(1, n, k) == BL_OK ? (size_t)w8_codes(n, k) : 0;
}

bl_status bitlinear_w8_pack(const float* w, int64_t n, int64_t k, int8_t* codes, float* scale,
                            void* stream) {
  bl_status st;
  if ((st = check_sum_shape(1, n, k)) != BL_OK) return st;
  if ((st = check_ptrs({w, codes, scale})) != BL_OK) return st;
  if (!disjoint({{codes, w8_codes(n, k)}, {scale, 4 * n}}, {{w, 4 * n * k}})) return BL_EINVAL;
  return launch_w8_pack(w, n, k, codes, scale, static_cast<hipStream_t>(stream)) == hipSuccess ? BL_OK
                                                                                              : BL_EHIP;
}

bl_status bitlinear_w8_unpack(const int8_t* codes, const float* scale, int64_t n, int64_t k,
                              float* out, void* stream) {
  bl_status st;
  if ((st = check_sum_shape(1, n, k)) != BL_OK) return st;
  if ((st = check_ptrs({codes, scale, out})) != BL_OK) return st;
  if (!disjoint({{out, 4 * n * k}}, {{codes, w8_codes(n, k)}, {scale, 4 * n}})) return BL_EINVAL;
  return launch_w8_unpack(codes, scale, n, k, out, static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_w8_forward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return check_sum_shape(m, n, k) == BL_OK ? w8_forward_bytes(m, n, k) : 0;
}

bl_status bitlinear_w8_forward(int64_t m, int64_t n, int64_t k, const int8_t* q, const float* x_scale,
                               const int8_t* codes, const float* scale, const uint16_t* bias,
                               uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
  bl_status st;
  if ((st = check_sum_shape(m, n, k)) != BL_OK) return st;
  if ((st = check_ptrs({q, x_scale, codes, scale, y})) != BL_OK) return st;
  if ((st = check_optional({bias})) != BL_OK) return st;
  const size_t need = w8_forward_bytes(m, n, k);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != BL_OK) return st;
  if (!disjoint({{y, 2 * m * n}, {workspace, (int64_t)need}},
                {{q, m * k}, {x_scale, 4 * m}, {codes, w8_codes(n, k)}, {scale, 4 * n}, {bias, 2 * n}}))
    return BL_EINVAL;
  const W8Args a = {m, n, k, q, x_scale, codes, scale, bias, y};
  return launch_w8_forward(a, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)) == hipSuccess
             ? BL_OK
             : BL_EHIP;
}

size_t bitlinear_grad_norm_workspace_bytes(int32_t count, const bl_gradient* grads) {
  if (check_grads(count, grads) != BL_OK) return 0;
  try {
    std::vector<int64_t> numel((size_t)count);
    for (int32_t i = 0; i < count; ++i) numel[i] = grads[i].numel;
    return grad_norm_bytes(count, numel.data());
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

bl_status bitlinear_grad_norm(int32_t count, const bl_gradient* grads, float* norm, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return grad_norm(count, grads, false, 0.0f, norm, workspace, workspace_bytes, stream);
}

bl_status bitlinear_clip_gradients(int32_t count, const bl_gradient* grads, float max_norm, float* norm,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0f)) return BL_EINVAL;
  return grad_norm(count, grads, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
