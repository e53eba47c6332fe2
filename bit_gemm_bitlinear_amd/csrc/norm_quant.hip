// Residual add, RMSNorm and per-token int8 codes in one pass over the rows,
// the norm's gradient, and the activations that the codes stand for.
//
//   h = bf16(x + residual);  rstd = fp32(1 / sqrt(mean(h^2) + eps))
//   n = bf16(fp32(h * rstd) * w);  s = 127 / max(max|n|, 1e-5)
//   q = clamp(round(n * s), -128, 127)
//
// q and s are the Falcon-Edge blog's activation_norm_quant ("A series of
// powerful, universal and fine-tunable 1.58-bit language models", section
// "Falcon-Edge, a series of universal models") of the norm's bf16 output, so
// fusing them changes no bit.  The mean of squares is summed in fp64: squares
// of bf16 values are exact there, and a sum of up to 2^22 of them is off by
// less than 2^-30 of itself whatever the order, so rstd does not depend on
// the split of the row over threads except at a rounding border of fp32, and
// codes next to a rounding border agree with any other evaluation.
#include "../../include/bitlinear_layer.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"
#include "restore.hpp"

namespace bl {

namespace {

constexpr int kT = 256;  // threads of a row's workgroup
constexpr int kWaves = kT / 64;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// VEC (4 or 8) consecutive bf16 values as VEC / 2 dwords.
template <int VEC>
struct Piece {
  uint32_t w[VEC / 2];
};

template <int VEC>
__device__ __forceinline__ Piece<VEC> load_bf16(const uint16_t* p) {
  Piece<VEC> r;
  if constexpr (VEC == 8) {
    const v4i v = *G(reinterpret_cast<const v4i*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)v[i];
  } else {
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    const v2i v = *G(reinterpret_cast<const v2i*>(p));
#pragma unroll
    for (int i = 0; i < 2; ++i) r.w[i] = (uint32_t)v[i];
  }
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Piece<VEC>& r) {
  if constexpr (VEC == 8) {
    *G(reinterpret_cast<v4i*>(p)) =
        v4i{(int32_t)r.w[0], (int32_t)r.w[1], (int32_t)r.w[2], (int32_t)r.w[3]};
  } else {
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    *G(reinterpret_cast<v2i*>(p)) = v2i{(int32_t)r.w[0], (int32_t)r.w[1]};
  }
}

// VEC weights at column e as fp32 (ones without a weight).
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, int wtype, int e, float (&o)[VEC]) {
  if (wtype == BL_WEIGHT_BF16) {
    const Piece<VEC> p = load_bf16<VEC>(static_cast<const uint16_t*>(w) + e);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      o[2 * i] = lo_f(p.w[i]);
      o[2 * i + 1] = hi_f(p.w[i]);
    }
  } else if (wtype == BL_WEIGHT_F32) {
    typedef float v4f __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const v4f v = *G(reinterpret_cast<const v4f*>(static_cast<const float*>(w) + e + i));
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = 1.0f;
  }
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) t += red[i];
  return t;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t t = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) t = max(t, red[i]);
  return t;
}

// h of one piece: x, or the bf16 sum of x and the residual.
template <int VEC>
__device__ __forceinline__ Piece<VEC> load_h(const uint16_t* x, const uint16_t* r, int e) {
  Piece<VEC> p = load_bf16<VEC>(x + e);
  if (r) {
    const Piece<VEC> b = load_bf16<VEC>(r + e);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) p.w[i] = add_bf16x2(p.w[i], b.w[i]);
  }
  return p;
}

template <int VEC>
__device__ __forceinline__ double square_sum(const Piece<VEC>& p) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const double a = (double)lo_f(p.w[i]), b = (double)hi_f(p.w[i]);
    s = __builtin_fma(a, a, s);
    s = __builtin_fma(b, b, s);
  }
  return s;
}

// n = bf16((h * rstd) * w), two fp32 products each rounded (one without a
// weight: multiplying by 1 changes nothing).
template <int VEC>
__device__ __forceinline__ Piece<VEC> normed(const Piece<VEC>& h, float rstd, const float (&w)[VEC]) {
  Piece<VEC> o;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    o.w[i] = pack_bf16x2((lo_f(h.w[i]) * rstd) * w[2 * i], (hi_f(h.w[i]) * rstd) * w[2 * i + 1]);
  return o;
}

template <int VEC>
__device__ __forceinline__ uint32_t absmax_bits(const Piece<VEC>& p) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < VEC / 2; i += 2) a = max(a, absmax_bits4(p.w[i], p.w[i + 1]));
  return a;
}

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* q, const Piece<VEC>& n, float s) {
  uint32_t d[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i)
    d[i] = ((uint32_t)quant_i8(lo_f(n.w[2 * i]), s) & 0xFFu) |
           (((uint32_t)quant_i8(hi_f(n.w[2 * i]), s) & 0xFFu) << 8) |
           (((uint32_t)quant_i8(lo_f(n.w[2 * i + 1]), s) & 0xFFu) << 16) |
           (((uint32_t)quant_i8(hi_f(n.w[2 * i + 1]), s) & 0xFFu) << 24);
  if constexpr (VEC == 8) {
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    *G(reinterpret_cast<v2i*>(q)) = v2i{(int32_t)d[0], (int32_t)d[1]};
  } else {
    *G(reinterpret_cast<uint32_t*>(q)) = d[0];
  }
}

__device__ __forceinline__ float rstd_of(double sum, int k, double eps) {
  return (float)(1.0 / sqrt(sum / (double)k + eps));
}

// Rows go over two grid dimensions: one alone holds 2^32 threads.
constexpr int64_t kGridX = 1 << 20;
__device__ __forceinline__ int64_t row_index() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// One workgroup per row; the row stays in registers (NCH pieces a thread)
// between the sum, the maximum and the codes: x and the residual are read
// once, everything else written once.
template <int VEC, int NCH>
__global__ __launch_bounds__(kT) void norm_quant_kernel(const NormArgs A) {
  __shared__ double red[kWaves];
  __shared__ uint32_t redu[kWaves];
  const int tid = threadIdx.x, k = A.k;
  const int64_t m = row_index();
  if (m >= A.m) return;
  const int64_t row = m * k;
  const uint16_t* x = A.x + row;
  const uint16_t* r = A.res ? A.res + row : nullptr;
  Piece<VEC> h[NCH];
  double ss = 0.0;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
    if (e < k) {
      h[b] = load_h<VEC>(x, r, e);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) h[b].w[i] = 0u;
    }
  }
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
    ss += square_sum(h[b]);
    if (A.h && e < k) store_bf16<VEC>(A.h + row + e, h[b]);
  }
  const float rstd = rstd_of(block_sum(ss, red), k, A.eps);
  if (A.rstd && tid == 0) A.rstd[m] = rstd;
  uint32_t amax = 0;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
    if (e < k) {
      float w[VEC];
      load_weight<VEC>(A.weight, A.wtype, e, w);
      h[b] = normed<VEC>(h[b], rstd, w);
      if (A.n) store_bf16<VEC>(A.n + row + e, h[b]);
      amax = max(amax, absmax_bits<VEC>(h[b]));
    }
  }
  if (!A.q) return;
  const float s = act_scale(bf16_to_f32(block_max(amax, redu)));
  if (tid == 0) A.x_scale[m] = s;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
    if (e < k) store_codes<VEC>(A.q + row + e, h[b], s);
  }
}

// Rows longer than the registers hold: three passes over the row (the later
// ones read h where it was written, else add again).
__global__ __launch_bounds__(kT) void norm_quant_long_kernel(const NormArgs A) {
  __shared__ double red[kWaves];
  __shared__ uint32_t redu[kWaves];
  const int tid = threadIdx.x, k = A.k;
  const int64_t m = row_index();
  if (m >= A.m) return;
  const int64_t row = m * k;
  const uint16_t* x = A.x + row;
  const uint16_t* r = A.res ? A.res + row : nullptr;
  double ss = 0.0;
  for (int e = 4 * tid; e < k; e += 4 * kT) {
    const Piece<4> h = load_h<4>(x, r, e);
    ss += square_sum(h);
    if (A.h) store_bf16<4>(A.h + row + e, h);
  }
  if (A.h) {  // each thread reads back what it wrote itself
    x = A.h + row;
    r = nullptr;
  }
  const float rstd = rstd_of(block_sum(ss, red), k, A.eps);
  if (A.rstd && tid == 0) A.rstd[m] = rstd;
  uint32_t amax = 0;
  for (int e = 4 * tid; e < k; e += 4 * kT) {
    float w[4];
    load_weight<4>(A.weight, A.wtype, e, w);
    const Piece<4> n = normed<4>(load_h<4>(x, r, e), rstd, w);
    if (A.n) store_bf16<4>(A.n + row + e, n);
    amax = max(amax, absmax_bits<4>(n));
  }
  if (!A.q) return;
  const float s = act_scale(bf16_to_f32(block_max(amax, redu)));
  if (tid == 0) A.x_scale[m] = s;
  for (int e = 4 * tid; e < k; e += 4 * kT) {
    float w[4];
    load_weight<4>(A.weight, A.wtype, e, w);
    store_codes<4>(A.q + row + e, normed<4>(load_h<4>(x, r, e), rstd, w), s);
  }
}

// ---- gradient ----

__device__ __forceinline__ float block_sum_f(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) t += red[i];
  return t;
}

// Each workgroup takes every gridDim.x-th row and each thread fixed columns,
// so the thread keeps its columns' sums for dweight in registers over the
// rows; the partial rows of all workgroups are added by a second kernel, in a
// fixed order.
template <int VEC, int NCH>
__global__ __launch_bounds__(kT) void norm_backward_kernel(const NormBwdArgs A) {
  __shared__ float red[2][kWaves];
  const int tid = threadIdx.x, k = A.k;
  const float inv_k = 1.0f / (float)k;
  float dw[NCH][VEC], w[NCH][VEC];
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[b][i] = w[b][i] = 0.0f;
    if (e < k) load_weight<VEC>(A.weight, A.wtype, e, w[b]);
  }
  int it = 0;
  for (int64_t m = blockIdx.x; m < A.m; m += gridDim.x, it ^= 1) {
    const int64_t row = m * k;
    Piece<VEC> dn[NCH], h[NCH], dh[NCH];
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = VEC * (tid + kT * b);
      if (e < k) {
        dn[b] = load_bf16<VEC>(A.dn + row + e);
        h[b] = load_bf16<VEC>(A.h + row + e);
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) dn[b].w[i] = h[b].w[i] = 0u;
      }
    }
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = VEC * (tid + kT * b);
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) dh[b].w[i] = 0u;
      if (A.dh && e < k) dh[b] = load_bf16<VEC>(A.dh + row + e);
    }
    const float rstd = A.rstd[m];
    float dot = 0.0f;
#pragma unroll
    for (int b = 0; b < NCH; ++b)
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float z0 = lo_f(h[b].w[i]) * rstd, z1 = hi_f(h[b].w[i]) * rstd;
        const float d0 = lo_f(dn[b].w[i]), d1 = hi_f(dn[b].w[i]);
        const float t0 = d0 * z0, t1 = d1 * z1;
        dw[b][2 * i] += t0;
        dw[b][2 * i + 1] += t1;
        dot = __builtin_fmaf(t0, w[b][2 * i], dot);
        dot = __builtin_fmaf(t1, w[b][2 * i + 1], dot);
      }
    const float c = block_sum_f(dot, red[it]) * inv_k;
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = VEC * (tid + kT * b);
      if (e >= k) continue;
      Piece<VEC> o;
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float z0 = lo_f(h[b].w[i]) * rstd, z1 = hi_f(h[b].w[i]) * rstd;
        const float g0 = lo_f(dn[b].w[i]) * w[b][2 * i], g1 = hi_f(dn[b].w[i]) * w[b][2 * i + 1];
        o.w[i] = pack_bf16x2(__builtin_fmaf(rstd, g0 - z0 * c, lo_f(dh[b].w[i])),
                             __builtin_fmaf(rstd, g1 - z1 * c, hi_f(dh[b].w[i])));
      }
      store_bf16<VEC>(A.dx + row + e, o);
    }
  }
  if (!A.part) return;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = VEC * (tid + kT * b);
    if (e >= k) continue;
#pragma unroll
    for (int i = 0; i < VEC; ++i) *G(A.part + (int64_t)blockIdx.x * k + e + i) = dw[b][i];
  }
}

// Rows longer than the registers hold: two passes over the row, the sums for
// dweight kept in the workgroup's partial row (each thread its own columns).
__global__ __launch_bounds__(kT) void norm_backward_long_kernel(const NormBwdArgs A) {
  __shared__ float red[2][kWaves];
  const int tid = threadIdx.x, k = A.k;
  const float inv_k = 1.0f / (float)k;
  float* part = A.part ? A.part + (int64_t)blockIdx.x * k : nullptr;
  int it = 0;
  for (int64_t m = blockIdx.x; m < A.m; m += gridDim.x, it ^= 1) {
    const int64_t row = m * k;
    const bool first = m < (int64_t)gridDim.x;
    const float rstd = A.rstd[m];
    float dot = 0.0f;
    for (int e = 4 * tid; e < k; e += 4 * kT) {
      const Piece<4> dn = load_bf16<4>(A.dn + row + e), h = load_bf16<4>(A.h + row + e);
      float w[4];
      load_weight<4>(A.weight, A.wtype, e, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = (i & 1 ? hi_f(h.w[i >> 1]) : lo_f(h.w[i >> 1])) * rstd;
        const float t = (i & 1 ? hi_f(dn.w[i >> 1]) : lo_f(dn.w[i >> 1])) * z;
        if (part) *G(part + e + i) = first ? t : *G(part + e + i) + t;
        dot = __builtin_fmaf(t, w[i], dot);
      }
    }
    const float c = block_sum_f(dot, red[it]) * inv_k;
    for (int e = 4 * tid; e < k; e += 4 * kT) {
      const Piece<4> dn = load_bf16<4>(A.dn + row + e), h = load_bf16<4>(A.h + row + e);
      Piece<4> dh;
      dh.w[0] = dh.w[1] = 0u;
      if (A.dh) dh = load_bf16<4>(A.dh + row + e);
      float w[4];
      load_weight<4>(A.weight, A.wtype, e, w);
      Piece<4> o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float z0 = lo_f(h.w[i]) * rstd, z1 = hi_f(h.w[i]) * rstd;
        const float g0 = lo_f(dn.w[i]) * w[2 * i], g1 = hi_f(dn.w[i]) * w[2 * i + 1];
        o.w[i] = pack_bf16x2(__builtin_fmaf(rstd, g0 - z0 * c, lo_f(dh.w[i])),
                             __builtin_fmaf(rstd, g1 - z1 * c, hi_f(dh.w[i])));
      }
      store_bf16<4>(A.dx + row + e, o);
    }
  }
}

// dweight[k] = sum over the workgroups' partial rows: 32 columns a workgroup,
// 32 slices of the rows, joined in a fixed order.
__global__ __launch_bounds__(1024) void column_join_kernel(const float* __restrict__ part, int rows,
                                                           int k, float* __restrict__ out,
                                                           int accumulate) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int col = 32 * blockIdx.x + c;
  float v = 0.0f;
  if (col < k) {
#pragma unroll 8
    for (int r = s; r < rows; r += 32) v += *G(part + (int64_t)r * k + col);
  }
  red[s][c] = v;
  __syncthreads();
  // transposed: wave w adds columns 2w and 2w + 1, 32 lanes each
  float t = red[threadIdx.x & 31][threadIdx.x >> 5];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor(t, o);
  const int oc = 32 * blockIdx.x + (threadIdx.x >> 5);
  if ((threadIdx.x & 31) == 0 && oc < k) out[oc] = accumulate ? out[oc] + t : t;
}

// ---- restored activations ----

// bf16(q / s) for 16 (WIDE) or 4 codes a thread; blockIdx.y walks the rows.
template <bool WIDE>
__global__ __launch_bounds__(256) void restore_kernel(const int8_t* __restrict__ q,
                                                      const float* __restrict__ x_scale, int64_t m,
                                                      int k, uint16_t* __restrict__ out) {
  constexpr int W = WIDE ? 16 : 4;
  const int e = W * ((int)blockIdx.x * 256 + (int)threadIdx.x);
  if (e >= k) return;
  for (int64_t r = blockIdx.y; r < m; r += gridDim.y) {
    const RestoreRow d = restore_row(*G(x_scale + r));
    uint32_t v[W / 4];
    if constexpr (WIDE) {
      const v4i t = *G(reinterpret_cast<const v4i*>(q + r * k + e));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)t[i];
    } else {
      v[0] = *G(reinterpret_cast<const uint32_t*>(q + r * k + e));
    }
    uint32_t o[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) o[i] = restore2(v[i >> 1], 2 * (i & 1), d);
    uint16_t* dst = out + r * k + e;
    if constexpr (WIDE) {
      *G(reinterpret_cast<v4i*>(dst)) = v4i{(int32_t)o[0], (int32_t)o[1], (int32_t)o[2], (int32_t)o[3]};
      *G(reinterpret_cast<v4i*>(dst + 8)) = v4i{(int32_t)o[4], (int32_t)o[5], (int32_t)o[6], (int32_t)o[7]};
    } else {
      typedef int32_t v2i __attribute__((ext_vector_type(2)));
      *G(reinterpret_cast<v2i*>(dst)) = v2i{(int32_t)o[0], (int32_t)o[1]};
    }
  }
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s) {
  const dim3 g((unsigned)(a.m < kGridX ? a.m : kGridX), (unsigned)((a.m + kGridX - 1) / kGridX));
  if (a.k % 8 == 0 && a.k <= 8 * 8 * kT) {
    const int n = (a.k + 8 * kT - 1) / (8 * kT);
    if (n <= 1) norm_quant_kernel<8, 1><<<g, kT, 0, s>>>(a);
    else if (n <= 2) norm_quant_kernel<8, 2><<<g, kT, 0, s>>>(a);
    else if (n <= 4) norm_quant_kernel<8, 4><<<g, kT, 0, s>>>(a);
    else norm_quant_kernel<8, 8><<<g, kT, 0, s>>>(a);
  } else if (a.k <= 16 * 4 * kT) {
    const int n = (a.k + 4 * kT - 1) / (4 * kT);
    if (n <= 2) norm_quant_kernel<4, 2><<<g, kT, 0, s>>>(a);
    else if (n <= 8) norm_quant_kernel<4, 8><<<g, kT, 0, s>>>(a);
    else norm_quant_kernel<4, 16><<<g, kT, 0, s>>>(a);
  } else {
    norm_quant_long_kernel<<<g, kT, 0, s>>>(a);
  }
  return hipGetLastError();
}

int norm_backward_blocks(int64_t m, int64_t k) {
  (void)k;
  return (int)(m <= 512 ? (m + 1) / 2 : 512);
}

hipError_t launch_norm_backward(const NormBwdArgs& a, float* dweight, bool accumulate,
                                hipStream_t s) {
  const int g = norm_backward_blocks(a.m, a.k);
  if (a.k % 8 == 0 && a.k <= 8 * 8 * kT) {
    const int n = (a.k + 8 * kT - 1) / (8 * kT);
    if (n <= 1) norm_backward_kernel<8, 1><<<g, kT, 0, s>>>(a);
    else if (n <= 2) norm_backward_kernel<8, 2><<<g, kT, 0, s>>>(a);
    else if (n <= 4) norm_backward_kernel<8, 4><<<g, kT, 0, s>>>(a);
    else norm_backward_kernel<8, 8><<<g, kT, 0, s>>>(a);
  } else if (a.k <= 16 * 4 * kT) {
    const int n = (a.k + 4 * kT - 1) / (4 * kT);
    if (n <= 2) norm_backward_kernel<4, 2><<<g, kT, 0, s>>>(a);
    else if (n <= 8) norm_backward_kernel<4, 8><<<g, kT, 0, s>>>(a);
    else norm_backward_kernel<4, 16><<<g, kT, 0, s>>>(a);
  } else {
    norm_backward_long_kernel<<<g, kT, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  column_join_kernel<<<(unsigned)((a.k + 31) / 32), 1024, 0, s>>>(a.part, g, a.k, dweight,
                                                                accumulate ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_restore(const int8_t* q, const float* x_scale, int64_t m, int64_t k,
                          uint16_t* out, hipStream_t s) {
  const int64_t w = k % 16 == 0 ? 16 : 4;
  const unsigned gx = (unsigned)((k / w + 255) / 256);
  const unsigned gy = (unsigned)(m < 65535 ? m : 65535);
  if (w == 16)
    restore_kernel<true><<<dim3(gx, gy), 256, 0, s>>>(q, x_scale, m, (int)k, out);
  else
    restore_kernel<false><<<dim3(gx, gy), 256, 0, s>>>(q, x_scale, m, (int)k, out);
  return hipGetLastError();
}

}  // namespace bl
