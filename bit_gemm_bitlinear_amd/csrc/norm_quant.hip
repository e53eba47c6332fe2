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

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

typedef int32_t v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
// K % 4 == 0: rows start at any multiple of 8 bytes (4 for int8 codes).
typedef v4i v4i_8 __attribute__((aligned(8)));
typedef v2i v2i_4 __attribute__((aligned(4)));
typedef v4i v4i_4 __attribute__((aligned(4)));

// Eight consecutive bf16 values as four dwords.  A row's last piece may hold
// four (`n` values; the others are zeros and are not stored).
struct Piece {
  uint32_t w[4];
};

__device__ __forceinline__ Piece load_bf16(const uint16_t* p, int n) {
  Piece r;
  if (n >= 8) {
    const v4i v = *G(reinterpret_cast<const v4i_8*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)v[i];
  } else {
    const v2i v = n > 0 ? *G(reinterpret_cast<const v2i*>(p)) : v2i{0, 0};
    r.w[0] = (uint32_t)v.x;
    r.w[1] = (uint32_t)v.y;
    r.w[2] = r.w[3] = 0u;
  }
  return r;
}

__device__ __forceinline__ void store_bf16(uint16_t* p, int n, const Piece& r) {
  if (n >= 8)
    *G(reinterpret_cast<v4i_8*>(p)) = v4i{(int32_t)r.w[0], (int32_t)r.w[1], (int32_t)r.w[2], (int32_t)r.w[3]};
  else if (n > 0)
    *G(reinterpret_cast<v2i*>(p)) = v2i{(int32_t)r.w[0], (int32_t)r.w[1]};
}

// Eight weights at column e as fp32 (ones without a weight).
__device__ __forceinline__ void load_weight(const void* w, int wtype, int e, int n, float (&o)[8]) {
  if (wtype == BL_WEIGHT_BF16) {
    const Piece p = load_bf16(static_cast<const uint16_t*>(w) + e, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = lo_f(p.w[i]);
      o[2 * i + 1] = hi_f(p.w[i]);
    }
  } else if (wtype == BL_WEIGHT_F32) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const v4f v = i < n ? *G(reinterpret_cast<const v4f*>(static_cast<const float*>(w) + e + i)) : v4f{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 1.0f;
  }
}

// Reductions over a wave: exchanges within 16 lanes (quad swaps, rotations of
// a row), then the four rows' values by lane reads.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)b) | ((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ float read_lane(float v, int l) { return __uint_as_float(read_lane(__float_as_uint(v), l)); }
__device__ __forceinline__ double read_lane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)read_lane((uint32_t)b, l) | ((uint64_t)read_lane((uint32_t)(b >> 32), l) << 32));
}

template <typename V, typename Op>
__device__ __forceinline__ V wave_reduce(V v, Op op) {
  v = op(v, dpp<0xB1>(v));   // quad: lanes 1 0 3 2
  v = op(v, dpp<0x4E>(v));   // 2 3 0 1
  v = op(v, dpp<0x124>(v));  // row rotated by 4
  v = op(v, dpp<0x128>(v));  // by 8
  return op(op(read_lane(v, 0), read_lane(v, 16)), op(read_lane(v, 32), read_lane(v, 48)));
}

// The same over a workgroup of up to 16 waves.
template <typename V, typename Op>
__device__ __forceinline__ V row_reduce(V v, V* red, Op op) {
  v = wave_reduce(v, op);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < waves; ++i) v = op(v, red[i]);
  return v;
}
template <typename V>
__device__ __forceinline__ V row_sum(V v, V* red) {
  return row_reduce(v, red, [](V a, V b) { return a + b; });
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  return row_reduce(v, red, [](uint32_t a, uint32_t b) { return max(a, b); });
}

__device__ __forceinline__ double square_sum(const Piece& p) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = (double)lo_f(p.w[i]), b = (double)hi_f(p.w[i]);
    s = __builtin_fma(a, a, s);
    s = __builtin_fma(b, b, s);
  }
  return s;
}

// n = bf16((h * rstd) * w), two fp32 products each rounded (one without a
// weight: multiplying by 1 changes nothing).
__device__ __forceinline__ Piece normed(const Piece& h, float rstd, const float (&w)[8]) {
  Piece o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.w[i] = pack_bf16x2((lo_f(h.w[i]) * rstd) * w[2 * i], (hi_f(h.w[i]) * rstd) * w[2 * i + 1]);
  return o;
}

// Largest magnitude pattern of a piece's values and `a`, for each half of a
// dword: the patterns of |bf16| order like the values.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 absmax2(u16x2 a, const Piece& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a = __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, p.w[i] & 0x7FFF7FFFu));
  return a;
}
__device__ __forceinline__ uint32_t absmax_bits(u16x2 a) { return max((uint32_t)a.x, (uint32_t)a.y); }

// Codes of a piece: round(n * s) is at most 127 in magnitude, so that plus 128
// converts to an unsigned byte exactly, into its place, and one xor a dword
// turns the bytes into int8.
__device__ __forceinline__ void store_codes(int8_t* q, int n, const Piece& v, float s) {
  uint32_t d[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = i & 1 ? hi_f(v.w[i >> 1]) : lo_f(v.w[i >> 1]);
    d[i >> 2] = __builtin_amdgcn_cvt_pk_u8_f32(rintf(x * s) + 128.0f, i & 3, d[i >> 2]);
  }
  if (n >= 8)
    *G(reinterpret_cast<v2i_4*>(q)) = v2i{(int32_t)(d[0] ^ 0x80808080u), (int32_t)(d[1] ^ 0x80808080u)};
  else if (n > 0)
    *G(reinterpret_cast<uint32_t*>(q)) = d[0] ^ 0x80808080u;
}

// fp32(1 / sqrt(sum / k + eps)) from the hardware's fp64 estimate y and one
// third-order step: with r = 1 - x y^2, 1 / sqrt(x) = y (1 + r / 2 + 3 r^2 / 8 + O(r^3)),
// exact to fp64 rounding; 0 where the residual add has overflowed to infinity.  (Square root and divisions proper are some 80 fp64
// instructions in every wave: 2.7 us of the 12 us of 2048 rows of 2560.)
__device__ __forceinline__ float rstd_of(double sum, double inv_k, double eps) {
  const double x = __builtin_fma(sum, inv_k, eps);
  const double y = __builtin_amdgcn_rsq(x);
  const double r = __builtin_fma(-x * y, y, 1.0);
  return y == 0.0 ? 0.0f : (float)__builtin_fma(y * r, __builtin_fma(r, 0.375, 0.5), y);
}

// Rows go over two grid dimensions: one alone holds 2^32 threads.
constexpr int64_t kGridX = 1 << 20;
__device__ __forceinline__ int64_t row_index() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// A workgroup a row, of as many threads as it has pieces, NCH a thread.  The
// row stays in registers between the sum, the maximum and the codes: x and
// the residual are read once, everything else written once.  The weights are
// loaded with them where the registers allow (rows of up to two pieces a
// thread): the norm then does not wait for memory again after the sum.
// 2048 rows of 2560 with a residual (36.7 MB): 13.8 us from memory, 10.3 where
// the last-level cache holds the inputs.  A row is five waves, a CU holds six
// such workgroups, 1536 rows in all: a quarter of the rows run in a second
// round, and nothing loads for a workgroup while it reduces and stores.  777
// rows of 14332 (33.4 MB), four pieces a thread and the weight read per row
// after the sum: 16.5 us and 14.6.  One row of 4096: 3.4 us and 3.1.  A wave a
// row took 11.8 us for 2048 x 2560 (next to 10.9 then).
constexpr int kMaxT = 1024;
template <int NCH>
__global__ __launch_bounds__(kMaxT) void norm_quant_kernel(const NormArgs A) {
  __shared__ double red[kMaxT / 64];
  __shared__ uint32_t redu[kMaxT / 64];
  const int tid = threadIdx.x, T = blockDim.x, k = A.k;
  const int64_t m = row_index();
  if (m >= A.m) return;
  const int64_t row = m * k;
  constexpr bool HOLD = NCH <= 2;
  Piece h[NCH];
  float w[HOLD ? NCH : 1][8];
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
    h[b] = load_bf16(A.x + row + e, k - e);
  }
  Piece r[NCH];
  if (A.res) {
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = 8 * (tid + T * b);
      r[b] = load_bf16(A.res + row + e, k - e);
    }
  }
  if constexpr (HOLD) {
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = 8 * (tid + T * b);
      load_weight(A.weight, A.wtype, e, k - e, w[b]);
    }
  }
  if (A.res) {
#pragma unroll
    for (int b = 0; b < NCH; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) h[b].w[i] = add_bf16x2(h[b].w[i], r[b].w[i]);
  }
  double ss = 0.0;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
    ss += square_sum(h[b]);
    if (A.h) store_bf16(A.h + row + e, k - e, h[b]);
  }
  const float rstd = rstd_of(row_sum(ss, red), A.inv_k, A.eps);
  if (A.rstd && tid == 0) A.rstd[m] = rstd;
  u16x2 amax = {0, 0};
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
    if constexpr (HOLD) {
      h[b] = normed(h[b], rstd, w[b]);
    } else {
      load_weight(A.weight, A.wtype, e, k - e, w[0]);
      h[b] = normed(h[b], rstd, w[0]);
    }
    if (A.n) store_bf16(A.n + row + e, k - e, h[b]);
    amax = absmax2(amax, h[b]);
  }
  if (!A.q) return;
  const float s = act_scale(bf16_to_f32(row_max(absmax_bits(amax), redu)));
  if (tid == 0) A.x_scale[m] = s;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
    store_codes(A.q + row + e, k - e, h[b], s);
  }
}

// Rows longer than the registers hold: three passes over the row (the later
// ones read h where it was written, else add again).
constexpr int kLongT = 1024;
__global__ __launch_bounds__(kLongT) void norm_quant_long_kernel(const NormArgs A) {
  __shared__ double red[kLongT / 64];
  __shared__ uint32_t redu[kLongT / 64];
  const int tid = threadIdx.x, k = A.k;
  const int64_t m = row_index();
  if (m >= A.m) return;
  const int64_t row = m * k;
  const uint16_t* x = A.x + row;
  const uint16_t* r = A.res ? A.res + row : nullptr;
  auto load_h = [&](int e) {
    Piece p = load_bf16(x + e, k - e);
    if (r) {
      const Piece b = load_bf16(r + e, k - e);
#pragma unroll
      for (int i = 0; i < 4; ++i) p.w[i] = add_bf16x2(p.w[i], b.w[i]);
    }
    return p;
  };
  double ss = 0.0;
  for (int e = 8 * tid; e < k; e += 8 * kLongT) {
    const Piece h = load_h(e);
    ss += square_sum(h);
    if (A.h) store_bf16(A.h + row + e, k - e, h);
  }
  if (A.h) {  // each thread reads back what it wrote itself
    x = A.h + row;
    r = nullptr;
  }
  const float rstd = rstd_of(row_sum(ss, red), A.inv_k, A.eps);
  if (A.rstd && tid == 0) A.rstd[m] = rstd;
  u16x2 amax = {0, 0};
  for (int e = 8 * tid; e < k; e += 8 * kLongT) {
    float w[8];
    load_weight(A.weight, A.wtype, e, k - e, w);
    const Piece n = normed(load_h(e), rstd, w);
    if (A.n) store_bf16(A.n + row + e, k - e, n);
    amax = absmax2(amax, n);
  }
  if (!A.q) return;
  const float s = act_scale(bf16_to_f32(row_max(absmax_bits(amax), redu)));
  if (tid == 0) A.x_scale[m] = s;
  for (int e = 8 * tid; e < k; e += 8 * kLongT) {
    float w[8];
    load_weight(A.weight, A.wtype, e, k - e, w);
    store_codes(A.q + row + e, k - e, normed(load_h(e), rstd, w), s);
  }
}

// ---- gradient ----
//
//   g = dn * w, z = h * rstd, dx = bf16(rstd * (g - z * mean(g * z)) + dh),
//   dw = sum over the rows of dn * z

__device__ __forceinline__ Piece dx_piece(const Piece& dn, const Piece& h, const Piece& dh,
                                          const float (&w)[8], float rstd, float c) {
  Piece o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z0 = lo_f(h.w[i]) * rstd, z1 = hi_f(h.w[i]) * rstd;
    const float g0 = lo_f(dn.w[i]) * w[2 * i], g1 = hi_f(dn.w[i]) * w[2 * i + 1];
    o.w[i] = pack_bf16x2(__builtin_fmaf(rstd, g0 - z0 * c, lo_f(dh.w[i])),
                         __builtin_fmaf(rstd, g1 - z1 * c, hi_f(dh.w[i])));
  }
  return o;
}

// A row as the kernel holds it.
template <int NCH>
struct BwdRow {
  Piece dn[NCH], h[NCH], dh[NCH];
  float rstd;
};

// Threads and pieces as in the forward kernel; a workgroup takes rows a whole
// grid apart, the next one loading while it works on the current, and each
// thread fixed columns, so that it keeps its columns' sums for dweight in
// registers over the rows.  The partial rows of the workgroups are added by a
// second kernel, in a fixed order.  8191 rows of 2560 (168 MB): 34.2 us from
// memory, 4.9 TB/s of the 5.1 that a large copy reaches, and 27.9 over and over
// on inputs that the last-level cache (256 MB) holds; 512 rows of 4096: 8.0 us
// and 7.2, the latency of two rows one after the other.
constexpr int kBwdT = 512;
template <int NCH>
__global__ __launch_bounds__(kBwdT) void norm_backward_kernel(const NormBwdArgs A) {
  __shared__ float red[2][kBwdT / 64];
  const int tid = threadIdx.x, T = blockDim.x, k = A.k;
  const float inv_k = 1.0f / (float)k;
  float dw[NCH][8], w[NCH][8];
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[b][i] = 0.0f;
    load_weight(A.weight, A.wtype, e, k - e, w[b]);
  }
  auto load = [&](BwdRow<NCH>& r, int64_t m) {
    const int64_t row = m * k;
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = 8 * (tid + T * b);
      r.dn[b] = load_bf16(A.dn + row + e, k - e);
      r.h[b] = load_bf16(A.h + row + e, k - e);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.dh[b].w[i] = 0u;
      if (A.dh) r.dh[b] = load_bf16(A.dh + row + e, k - e);
    }
    r.rstd = *G(A.rstd + m);
  };
  int it = 0;
  auto work = [&](const BwdRow<NCH>& r, int64_t m) {
    float dot = 0.0f;
#pragma unroll
    for (int b = 0; b < NCH; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t0 = lo_f(r.dn[b].w[i]) * (lo_f(r.h[b].w[i]) * r.rstd);
        const float t1 = hi_f(r.dn[b].w[i]) * (hi_f(r.h[b].w[i]) * r.rstd);
        dw[b][2 * i] += t0;
        dw[b][2 * i + 1] += t1;
        dot = __builtin_fmaf(t0, w[b][2 * i], dot);
        dot = __builtin_fmaf(t1, w[b][2 * i + 1], dot);
      }
    const float c = row_sum(dot, red[it]) * inv_k;
    it ^= 1;
#pragma unroll
    for (int b = 0; b < NCH; ++b) {
      const int e = 8 * (tid + T * b);
      store_bf16(A.dx + m * k + e, k - e, dx_piece(r.dn[b], r.h[b], r.dh[b], w[b], r.rstd, c));
    }
  };
  const int64_t step = gridDim.x;
  if constexpr (NCH <= 2) {
    BwdRow<NCH> p, q;
    load(p, blockIdx.x);
    for (int64_t m = blockIdx.x; m < A.m; m += 2 * step) {
      if (m + step < A.m) load(q, m + step);
      work(p, m);
      if (m + step >= A.m) break;
      if (m + 2 * step < A.m) load(p, m + 2 * step);
      work(q, m + step);
    }
  } else {
    BwdRow<NCH> p;
    for (int64_t m = blockIdx.x; m < A.m; m += step) {
      load(p, m);
      work(p, m);
    }
  }
  if (!A.part) return;
  float* part = A.part + (int64_t)blockIdx.x * k;
#pragma unroll
  for (int b = 0; b < NCH; ++b) {
    const int e = 8 * (tid + T * b);
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      if (e + i < k) {
        v4f v = {dw[b][i], dw[b][i + 1], dw[b][i + 2], dw[b][i + 3]};
        if (A.add) v += *G(reinterpret_cast<const v4f*>(part + e + i));
        *G(reinterpret_cast<v4f*>(part + e + i)) = v;
      }
  }
}

// Rows longer than the registers hold: two passes over the row, the sums for
// dweight kept in the workgroup's partial row (each thread its own columns).
__global__ __launch_bounds__(kLongT) void norm_backward_long_kernel(const NormBwdArgs A) {
  __shared__ float red[2][kLongT / 64];
  const int tid = threadIdx.x, k = A.k;
  const float inv_k = 1.0f / (float)k;
  float* part = A.part ? A.part + (int64_t)blockIdx.x * k : nullptr;
  int it = 0;
  for (int64_t m = blockIdx.x; m < A.m; m += gridDim.x, it ^= 1) {
    const int64_t row = m * k;
    const bool first = m < (int64_t)gridDim.x && !A.add;
    const float rstd = *G(A.rstd + m);
    float dot = 0.0f;
    for (int e = 8 * tid; e < k; e += 8 * kLongT) {
      const Piece dn = load_bf16(A.dn + row + e, k - e), h = load_bf16(A.h + row + e, k - e);
      float w[8];
      load_weight(A.weight, A.wtype, e, k - e, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = (i & 1 ? hi_f(h.w[i >> 1]) : lo_f(h.w[i >> 1])) * rstd;
        const float t = (i & 1 ? hi_f(dn.w[i >> 1]) : lo_f(dn.w[i >> 1])) * z;
        if (part && e + i < k) *G(part + e + i) = first ? t : *G(part + e + i) + t;
        dot = __builtin_fmaf(t, w[i], dot);
      }
    }
    const float c = row_sum(dot, red[it]) * inv_k;
    for (int e = 8 * tid; e < k; e += 8 * kLongT) {
      const Piece dn = load_bf16(A.dn + row + e, k - e), h = load_bf16(A.h + row + e, k - e);
      Piece dh = {{0u, 0u, 0u, 0u}};
      if (A.dh) dh = load_bf16(A.dh + row + e, k - e);
      float w[8];
      load_weight(A.weight, A.wtype, e, k - e, w);
      store_bf16(A.dx + row + e, k - e, dx_piece(dn, h, dh, w, rstd, c));
    }
  }
}

// dweight[k] = sum over the workgroups' partial rows: 16 columns a workgroup,
// 64 slices of the rows, joined in a fixed order (512 rows of 2560: 4.7 us).
__global__ __launch_bounds__(1024) void column_join_kernel(const float* __restrict__ part, int rows,
                                                           int k, float* __restrict__ out,
                                                           int accumulate) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 15, s = threadIdx.x >> 4;
  const int col = 16 * blockIdx.x + c;
  float v = 0.0f;
  if (col < k) {
#pragma unroll 8
    for (int r = s; r < rows; r += 64) v += *G(part + (int64_t)r * k + col);
  }
  red[s][c] = v;
  __syncthreads();
  // transposed: wave w adds column w, a slice a lane
  const float t = wave_reduce(red[threadIdx.x & 63][threadIdx.x >> 6], [](float a, float b) { return a + b; });
  const int oc = 16 * blockIdx.x + (threadIdx.x >> 6);
  if ((threadIdx.x & 63) == 0 && oc < k) out[oc] = accumulate ? out[oc] + t : t;
}

// ---- restored activations ----

// bf16(q / s), 16 codes a thread; blockIdx.y walks the rows.  2048 x 2560 (15.7
// MB): 5.1 us; a row is one workgroup's, of whose 256 lanes 160 have codes there.
__global__ __launch_bounds__(256) void restore_kernel(const int8_t* __restrict__ q,
                                                      const float* __restrict__ x_scale, int64_t m,
                                                      int k, uint16_t* __restrict__ out) {
  const int e = 16 * ((int)blockIdx.x * 256 + (int)threadIdx.x);
  if (e >= k) return;
  for (int64_t r = blockIdx.y; r < m; r += gridDim.y) {
    const RestoreRow d = restore_row(*G(x_scale + r));
    const int8_t* src = q + r * k + e;
    uint16_t* dst = out + r * k + e;
    if (e + 16 <= k) {
      const v4i v = *G(reinterpret_cast<const v4i_4*>(src));
#pragma unroll
      for (int i = 0; i < 2; ++i)
        store_bf16(dst + 8 * i, 8, Piece{{restore2((uint32_t)v[2 * i], 0, d), restore2((uint32_t)v[2 * i], 2, d),
                                          restore2((uint32_t)v[2 * i + 1], 0, d), restore2((uint32_t)v[2 * i + 1], 2, d)}});
    } else {
      for (int i = 0; e + i < k; i += 4) {
        const uint32_t v = *G(reinterpret_cast<const uint32_t*>(src + i));
        *G(reinterpret_cast<v2i*>(dst + i)) = v2i{(int32_t)restore2(v, 0, d), (int32_t)restore2(v, 2, d)};
      }
    }
  }
}

}  // namespace

// Threads for `pieces` at n a thread: whole waves.
static int threads_for(int pieces, int n) { return ((pieces + n - 1) / n + 63) / 64 * 64; }

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t s) {
  const int pieces = (a.k + 7) / 8;
  const dim3 g((unsigned)(a.m < kGridX ? a.m : kGridX), (unsigned)((a.m + kGridX - 1) / kGridX));
  // One piece a thread up to 8192 columns where rows are few (their latency
  // counts), else up to 4096.
  if (pieces <= (a.m <= 256 ? 1024 : 512))
    norm_quant_kernel<1><<<g, threads_for(pieces, 1), 0, s>>>(a);
  else if (pieces <= 2 * 512 || (a.m <= 256 && pieces <= 2 * 1024))
    norm_quant_kernel<2><<<g, threads_for(pieces, 2), 0, s>>>(a);
  else if (pieces <= 4 * 1024)
    norm_quant_kernel<4><<<g, threads_for(pieces, 4), 0, s>>>(a);
  else
    norm_quant_long_kernel<<<g, kLongT, 0, s>>>(a);
  return hipGetLastError();
}

// Two rows a workgroup, or more where that would be over 512 partial rows to
// join (8191 x 2560: 512 and 768 alike, 1024 slower).  A few short rows are one
// workgroup's, which writes dweight itself, where the rows one after the other
// cost less than a second launch (8 rows of 512: 5.4 us against 7.8; 6 of 4096:
// 7.2 against 7.9, but 8 of them 8.9; 2 of 14336: 7.1 against 10.5, 4 of them 11.1).
// (Rows over 16384 columns: one a workgroup, their sums go through memory.)
int norm_backward_blocks(int64_t m, int64_t k) {
  if (k > 8 * 4 * kBwdT) return (int)(m <= 512 ? m : 512);
  return (int)(m <= 8 && m * k <= 28672 ? 1 : (m <= 1024 ? (m + 1) / 2 : 512));
}

hipError_t launch_norm_backward(NormBwdArgs a, float* dweight, bool accumulate, hipStream_t s) {
  const int g = norm_backward_blocks(a.m, a.k);
  if (g == 1) {
    a.part = dweight;
    a.add = accumulate ? 1 : 0;
  }
  const int pieces = (a.k + 7) / 8;
  if (pieces <= kBwdT)
    norm_backward_kernel<1><<<g, threads_for(pieces, 1), 0, s>>>(a);
  else if (pieces <= 2 * kBwdT)
    norm_backward_kernel<2><<<g, threads_for(pieces, 2), 0, s>>>(a);
  else if (pieces <= 4 * kBwdT)
    norm_backward_kernel<4><<<g, threads_for(pieces, 4), 0, s>>>(a);
  else
    norm_backward_long_kernel<<<g, kLongT, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dweight || g == 1) return e;
  column_join_kernel<<<(unsigned)((a.k + 15) / 16), 1024, 0, s>>>(a.part, g, a.k, dweight,
                                                                 accumulate ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_restore(const int8_t* q, const float* x_scale, int64_t m, int64_t k,
                          uint16_t* out, hipStream_t s) {
  const dim3 g((unsigned)((k + 4095) / 4096), (unsigned)(m < 65535 ? m : 65535));
  restore_kernel<<<g, 256, 0, s>>>(q, x_scale, m, (int)k, out);
  return hipGetLastError();
}

}  // namespace bl
