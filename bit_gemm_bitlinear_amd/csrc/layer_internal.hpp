// Internal interface of the operators of bitlinear_layer.h and bitlinear_ffn.h,
// between their entry points (layer_abi.hip; abi.hip for the forward on codes) and
// the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bl {

// A range of device memory a call reads or writes (nullptr: none),
// for the entry points' checks.
struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// ---- residual add + RMSNorm + int8 codes (norm_quant.hip) ----
struct NormArgs {
  const uint16_t* x;    // [m][k] bf16
  const uint16_t* res;  // [m][k] bf16, or nullptr
  const void* weight;   // [k] bf16 or fp32, or nullptr
  int32_t wtype;        // BL_WEIGHT_*
  int32_t k;
  int64_t m;
  double eps, inv_k;  // inv_k: 1 / k
  uint16_t* h;    // [m][k] bf16, or nullptr
  float* rstd;    // [m], or nullptr
  uint16_t* n;    // [m][k] bf16, or nullptr
  int8_t* q;      // [m][k], or nullptr (with x_scale)
  float* x_scale;
};
hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  const uint16_t* dn;
  const uint16_t* h;
  const float* rstd;
  const void* weight;
  int32_t wtype;
  int32_t k;
  int64_t m;
  const uint16_t* dh;  // or nullptr
  uint16_t* dx;
  float* part;         // [blocks][k] fp32 partial sums of dweight (one block: dweight), or nullptr
  int32_t add;         // one block: dweight is added to
};
// Workgroups of the backward kernel, each with a partial row of dweight.
int norm_backward_blocks(int64_t m, int64_t k);
hipError_t launch_norm_backward(NormBwdArgs a, float* dweight, bool accumulate, hipStream_t s);

hipError_t launch_restore(const int8_t* q, const float* x_scale, int64_t m, int64_t k,
                          uint16_t* out, hipStream_t s);

// ---- gradients of BitLinear (backward.hip) ----
struct BackwardArgs {
  int64_t m, n, k;
  const uint16_t* dy;
  // dx (nullptr: not wanted)
  const uint8_t* packed;
  bool tiled;
  const float* w_scale;
  const uint16_t* residual;
  uint16_t* dx;
  // dw (nullptr: not wanted) and dbias (only with dw)
  const int8_t* q;
  const float* x_scale;
  float* dw;
  float* dbias;
  bool accumulate;
};
size_t backward_bytes(int64_t m, int64_t n, int64_t k, bool dx, bool dw);
hipError_t launch_backward(const BackwardArgs& a, char* ws, size_t ws_bytes, hipStream_t s);

// Those of a gated block's two projections (backward.hip).
struct GatedBackwardArgs {
  int64_t m, n, k;
  bool silu;
  const uint16_t* da;
  const uint16_t* g;
  const uint16_t* u;
  // dx (nullptr: not wanted)
  const uint8_t* gate;
  const uint8_t* up;
  bool gate_tiled, up_tiled;
  const float* gate_scale;
  const float* up_scale;
  const uint16_t* residual;
  uint16_t* dx;
  // both or neither
  const int8_t* q;
  const float* x_scale;
  float* dw_gate;
  float* dw_up;
  bool accumulate;
};
size_t gated_backward_bytes(int64_t m, int64_t n, int64_t k, bool dx, bool dw);
hipError_t launch_gated_backward(const GatedBackwardArgs& a, char* ws, size_t ws_bytes, hipStream_t s);

// ---- gated feed-forward projections (gated.hip) ----
struct GatedArgs {
  int64_t m, n, k;
  const int8_t* q;
  const float* x_scale;
  const uint8_t* codes;  // the storage of bitlinear_ffn.h
  const float* gate_scale;
  const float* up_scale;
  bool silu;
  uint16_t* a;
  uint16_t* g;  // or nullptr
  uint16_t* u;
};
hipError_t launch_gated_weights(const uint8_t* gate, bool gate_tiled, const uint8_t* up, bool up_tiled,
                                int64_t n, int64_t k, uint8_t* codes, hipStream_t s);
size_t gated_forward_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_gated_forward(const GatedArgs& a, char* ws, hipStream_t s);

// ---- 8-bit weights (w8.hip) ----
hipError_t launch_w8_pack(const float* w, int64_t n, int64_t k, int8_t* codes, float* scale, hipStream_t s);
hipError_t launch_w8_unpack(const int8_t* codes, const float* scale, int64_t n, int64_t k, float* out,
                            hipStream_t s);
struct W8Args {
  int64_t m, n, k;
  const int8_t* q;
  const float* x_scale;
  const int8_t* codes;
  const float* scale;
  const uint16_t* bias;  // or nullptr
  uint16_t* y;
};
size_t w8_forward_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_w8_forward(const W8Args& a, char* ws, hipStream_t s);

// ---- gradient norm and clipping (grad_norm.hip) ----
struct Gradient {
  const void* g;
  void* out;
  int64_t numel;
  bool bf16;
};
size_t grad_norm_bytes(int32_t count, const int64_t* numel);
// norm: 1 float.  clip: out = g * min(1, max_norm / (norm + 1e-6)) as well.
hipError_t launch_grad_norm(int32_t count, const Gradient* t, bool clip, float max_norm, float* norm, char* ws,
                            hipStream_t s);

// ---- 4-bit weights (w4.hip) ----
hipError_t launch_w4_pack(const float* w, int64_t n, int64_t k, int group, uint8_t* codes,
                          uint16_t* scales, hipStream_t s);
hipError_t launch_w4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t n, int64_t k,
                            int group, float* out, hipStream_t s);
hipError_t launch_w4_forward(int64_t m, int64_t n, int64_t k, int group, const int8_t* q,
                             const float* x_scale, const uint8_t* codes, const uint16_t* scales,
                             const uint16_t* bias, uint16_t* y, hipStream_t s);

}  // namespace bl
