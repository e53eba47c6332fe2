// 8-bit weights with a scale per output channel: packing, and the product with
// int8 activations.
//
//   y[m][n] = bf16( (sum_k q[m][k] * v[n][k]) * s[n] / x_scale[m] )
//
// Storage (bitlinear_ffn.h): 16 rows x 64 k are one contiguous kilobyte, 16
// bytes (consecutive k of one row) a lane of a wavefront: an operand of the
// 16x16x64 int8 matrix-core op.  Sums are exact in int32.
//
// Up to 16 tokens the weights' bytes are the cost (codes_rows.hpp), past that tiles
// on the matrix cores (codes_gemm.hpp); codes_plan.hpp chooses, with the figures.
#include "../../include/bitlinear_ffn.h"
#include "codes_gemm.hpp"
#include "codes_plan.hpp"
#include "codes_rows.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"
#include "magnitude.hpp"

namespace bl {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// Offset of weights [row][e .. e + 3] in the storage (e % 4 == 0).
__device__ __forceinline__ int64_t w8_offset(int64_t row, int64_t e, int64_t ktiles) {
  return (((row >> 4) * ktiles + (e >> 6)) * 4 + ((e >> 4) & 3)) * 256 + 16 * (row & 15) + (e & 15);
}

// A workgroup a row: its largest magnitude, its scale, its codes.  Rows past N
// and codes past K are zeros.  The magnitudes are compared as bits: a weight that is not
// a number makes its row's scale, and so the row's outputs, not a number.  (14336 x 4096:
// 105 us; the second reading of a row comes from a cache.)
__global__ __launch_bounds__(256) void w8_pack_kernel(const float* __restrict__ w, int64_t n, int64_t k,
                                                      int64_t rows, int8_t* __restrict__ codes,
                                                      float* __restrict__ scale) {
  __shared__ uint32_t red[4];
  const int64_t ktiles = (k + 63) / 64;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float* src = w + row * k;
    uint32_t a = 0;
    if (row < n)
      for (int64_t e = 4 * threadIdx.x; e < k; e += 1024) {  // K % 4 == 0
        const v4f v = *G(reinterpret_cast<const v4f*>(src + e));
#pragma unroll
        for (int i = 0; i < 4; ++i) a = max(a, magnitude_bits(v[i]));
      }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o));
    __syncthreads();  // the last row's values are read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = max(max(red[0], red[1]), max(red[2], red[3]));
    float s = __uint_as_float(a) / 127.0f;
    if (s == 0.0f) s = 1.0f;
    if (row < n && threadIdx.x == 0) *G(scale + row) = s;
    for (int64_t e = 4 * threadIdx.x; e < ktiles * 64; e += 1024) {
      uint32_t b = 0;
      if (row < n && e < k) {
        const v4f v = *G(reinterpret_cast<const v4f*>(src + e));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b |= ((uint32_t)(int)fminf(fmaxf(rintf(v[i] / s), -127.0f), 127.0f) & 255u) << (8 * i);
      }
      *G(reinterpret_cast<uint32_t*>(codes + w8_offset(row, e, ktiles))) = b;
    }
  }
}

// A workgroup a row, four weights a thread (14336 x 4096: 99 us, by single weights 143).
__global__ __launch_bounds__(256) void w8_unpack_kernel(const int8_t* __restrict__ codes,
                                                        const float* __restrict__ scale, int64_t n, int64_t k,
                                                        float* __restrict__ out) {
  const int64_t ktiles = (k + 63) / 64;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const float s = *G(scale + row);
    for (int64_t e = 4 * threadIdx.x; e < k; e += 1024) {
      const int32_t b = *G(reinterpret_cast<const int32_t*>(codes + w8_offset(row, e, ktiles)));
      *G(reinterpret_cast<v4f*>(out + row * k + e)) =
          v4f{s * (float)(int8_t)b, s * (float)(int8_t)(b >> 8), s * (float)(int8_t)(b >> 16), s * (float)(b >> 24)};
    }
  }
}

// (acc * s) / xs by one product and one division.  With both scales in a middle
// range (xs in 2^-40..2^40, s in 2^-60..2^40) nothing in the division's fast form
// leaves fp32's.
__device__ __forceinline__ bool w8_fast_row(float xs) { return xs >= 9.094947e-13f && xs <= 1.0995116e12f; }
__device__ __forceinline__ bool w8_fast_scale(float s) { return s >= 8.6736174e-19f && s <= 1.0995116e12f; }
__device__ __forceinline__ float w8_value(int32_t acc, float s, float xs, float y, bool fast) {
  const float t = (float)acc * s;
  return fast ? row_div_fast(t, xs, y) : t / xs;
}

// ---------------------------------------------------------------------------
// Up to 16 tokens (codes_rows.hpp).

struct W8RowsArgs {
  RowsJob j;
  const float* x_scale;
  const float* scale;
  const uint16_t* bias;
  uint16_t* y;
};

__global__ __launch_bounds__(64 * kRowsWaves) void w8_rows_kernel(const W8RowsArgs A) {
  extern __shared__ __align__(16) int8_t smem[];
  codes_rows_product<4, false>(A.j, smem, [&](int m, int n, const v4i (&acc)[1]) {
    const float xs = *G(A.x_scale + m);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)acc[0][e] * *G(A.scale + min(n + e, A.j.n - 1)) / xs;
    uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (A.bias) {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = *G(A.bias + min(n + e, A.j.n - 1));
      lo = add_bf16x2(lo, b[0] | (b[1] << 16));
      hi = add_bf16x2(hi, b[2] | (b[3] << 16));
    }
    codes_put4(A.y + (int64_t)m * A.j.n, n, A.j.n, lo, hi);
  });
}

// ---------------------------------------------------------------------------
// More than 16 tokens: tiles on the int8 matrix cores (codes_gemm.hpp).

struct W8GemmArgs {
  CodesJob j;
  const float* x_scale;
  const float* scale;
  const uint16_t* bias;
  uint16_t* y;
};

template <typename T>
__global__ __launch_bounds__(64 * T::NW, 2) void w8_gemm_kernel(const W8GemmArgs A) {
  extern __shared__ __align__(16) int8_t smem[];
  const CodesJob& J = A.j;
  int ti, tj, kp;
  if (!codes_tile_of((int)blockIdx.x, J, &ti, &tj, &kp)) return;
  v16i acc[T::FI][T::FJ];
  T::run(J, ti, tj, kp, smem, acc);
  const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
  const int m0 = ti * T::TI + T::row0() + lr, n0 = tj * T::kCols + T::col0();
  if (J.ksplit > 1) {
#pragma unroll
    for (int i = 0; i < T::FI; ++i) {
      const int m = m0 + 32 * i;
      if (m >= J.m) continue;
      int32_t* row = J.part + ((int64_t)kp * J.m + m) * J.ldp;
#pragma unroll
      for (int j = 0; j < T::FJ; ++j) codes_put_part(row, n0 + 32 * j, J.ldp, acc[i][j]);
    }
    return;
  }
  codes_gemm::barrier();
  typename T::Rows rows(smem + T::wave() * T::Rows::kBytes);
  // scales and bias of the lane's columns
  float s[T::FJ][16];
  uint32_t bias[T::FJ][8];
  bool fast = true;
#pragma unroll
  for (int j = 0; j < T::FJ; ++j)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int n = n0 + 32 * j + 8 * a + 4 * lg;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][4 * a + e] = *G(A.scale + min(n + e, J.n - 1));
        fast = fast && w8_fast_scale(s[j][4 * a + e]);
      }
      if (A.bias)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          bias[j][2 * a + e] = (uint32_t)*G(A.bias + min(n + 2 * e, J.n - 1)) |
                               ((uint32_t)*G(A.bias + min(n + 2 * e + 1, J.n - 1)) << 16);
    }
#pragma unroll
  for (int i = 0; i < T::FI; ++i) {
    const float xs = *G(A.x_scale + min(m0 + 32 * i, J.m - 1)), y = 1.0f / xs;
    auto values = [&](auto fastc) {
#pragma unroll
      for (int j = 0; j < T::FJ; ++j)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          uint32_t w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 4 * a + 2 * e;
            w[e] = pack_bf16x2(w8_value(acc[i][j][r], s[j][r], xs, y, decltype(fastc)::value),
                               w8_value(acc[i][j][r + 1], s[j][r + 1], xs, y, decltype(fastc)::value));
            if (A.bias) w[e] = add_bf16x2(w[e], bias[j][2 * a + e]);
          }
          rows.put(lr, 32 * j + 8 * a + 4 * lg, w[0], w[1]);
        }
    };
    if (__all(fast && w8_fast_row(xs)))
      values(std::true_type{});
    else
      values(std::false_type{});
    rows.store(A.y, m0 - lr + 32 * i, n0, J.m, J.n, J.past_cache);
  }
}

// Adds the parts of a split product: eight outputs of a row a thread.
__global__ __launch_bounds__(256) void w8_finish_kernel(const W8GemmArgs A, int64_t total) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const CodesJob& J = A.j;
  const int cpr = (J.n + 7) >> 3;
  const int64_t m = id / cpr;
  const int n = 8 * (int)(id - m * cpr);
  int32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  codes_add_parts(J.part + m * J.ldp + n, (int64_t)J.m * J.ldp, J.ksplit, v);
  const float xs = *G(A.x_scale + m), y = 1.0f / xs;
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float s = *G(A.scale + min(n + e, J.n - 1));
    t[e] = w8_value(v[e], s, xs, y, w8_fast_row(xs) && w8_fast_scale(s));
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = pack_bf16x2(t[2 * e], t[2 * e + 1]);
    if (A.bias) {
      const uint32_t b0 = *G(A.bias + min(n + 2 * e, J.n - 1)), b1 = *G(A.bias + min(n + 2 * e + 1, J.n - 1));
      w[e] = add_bf16x2(w[e], b0 | (b1 << 16));
    }
  }
  codes_put8(A.y + m * J.n, n, J.n, (J.n & 7) == 0, w);
}

using W8Tile256 = CodesTile<256, 256, 2, 4, 4, false>;
using W8TileWide = CodesTile<128, 256, 2, 4, 5, false>;
template <bool WORDS>
using W8Tile128 = CodesTile<128, 128, 2, 2, 5, false, WORDS>;
template <bool WORDS>
using W8Tile64 = CodesTile<64, 64, 2, 2, 8, false, WORDS>;

template <typename T>
hipError_t w8_gemm(const W8GemmArgs& a, hipStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  const int64_t grid = round_up((int64_t)a.j.tiles_i * a.j.tiles_j * a.j.ksplit, 8);
  return codes_launch(&w8_gemm_kernel<T>, done, dim3((unsigned)grid), 64 * T::NW, T::kLds, T::kLds, s, a);
}

struct W8Layout {
  CodesPlan plan;
  int32_t ldq;
  size_t part, total;
};

W8Layout w8_layout(int64_t m, int64_t n, int64_t k) {
  W8Layout L = {};
  L.plan.cfg = -1;
  if (m > 16) L.plan = plan_codes(m, n, k, false);
  if (L.plan.cfg < 0) return L;
  L.ldq = (int32_t)(L.plan.pad ? round_up(k, 16) : k);
  if (L.plan.pad) L.total = align256((size_t)m * L.ldq);
  L.part = L.total;
  if (L.plan.ksplit > 1) L.total = align256(L.total + 4 * (size_t)L.plan.ksplit * m * part_pitch(n));
  return L;
}

}  // namespace

hipError_t launch_w8_pack(const float* w, int64_t n, int64_t k, int8_t* codes, float* scale, hipStream_t s) {
  const int64_t rows = (n + 15) / 16 * 16;
  w8_pack_kernel<<<(unsigned)(rows < 65536 ? rows : 65536), 256, 0, s>>>(w, n, k, rows, codes, scale);
  return hipGetLastError();
}

hipError_t launch_w8_unpack(const int8_t* codes, const float* scale, int64_t n, int64_t k, float* out,
                            hipStream_t s) {
  w8_unpack_kernel<<<(unsigned)(n < 65536 ? n : 65536), 256, 0, s>>>(codes, scale, n, k, out);
  return hipGetLastError();
}

size_t w8_forward_bytes(int64_t m, int64_t n, int64_t k) { return w8_layout(m, n, k).total; }

hipError_t launch_w8_forward(const W8Args& b, char* ws, hipStream_t s) {
  const W8Layout L = w8_layout(b.m, b.n, b.k);
  if (L.plan.cfg >= 0) {
    W8GemmArgs a = {};
    CodesJob& J = a.j;
    J.q = b.q;
    J.ldq = L.ldq;
    J.m = (int32_t)b.m;
    J.n = (int32_t)b.n;
    J.k = (int32_t)b.k;
    J.w = reinterpret_cast<const uint8_t*>(b.codes);
    J.ktiles = (int32_t)((b.k + 63) / 64);
    J.blocks = (int32_t)((b.n + 15) / 16);
    set_plan(J, L.plan, reinterpret_cast<int32_t*>(ws + L.part));
    a.x_scale = b.x_scale;
    a.scale = b.scale;
    a.bias = b.bias;
    a.y = b.y;
    hipError_t e = hipSuccess;
    if (L.plan.pad) {
      e = codes_pad(b.q, b.m, b.k, L.ldq, reinterpret_cast<int8_t*>(ws), s);
      if (e != hipSuccess) return e;
      J.q = reinterpret_cast<const int8_t*>(ws);
    }
    const bool words = L.ldq % 16 != 0;
    e = L.plan.cfg == 3   ? w8_gemm<W8Tile256>(a, s)
        : L.plan.cfg == 2 ? w8_gemm<W8TileWide>(a, s)
        : L.plan.cfg == 1 ? (words ? w8_gemm<W8Tile128<true>>(a, s) : w8_gemm<W8Tile128<false>>(a, s))
                          : (words ? w8_gemm<W8Tile64<true>>(a, s) : w8_gemm<W8Tile64<false>>(a, s));
    if (e != hipSuccess || J.ksplit == 1) return e;
    const int64_t total = b.m * ((b.n + 7) / 8);
    w8_finish_kernel<<<(unsigned)((total + 255) / 256), 256, 0, s>>>(a, total);
    return hipGetLastError();
  }
  const RowsPlan p = plan_rows(b.m, b.n, b.k, false);
  W8RowsArgs a = {};
  a.j.q = b.q;
  a.j.m = (int32_t)b.m;
  a.j.n = (int32_t)b.n;
  a.j.k = (int32_t)b.k;
  a.j.w = reinterpret_cast<const uint8_t*>(b.codes);
  a.j.ktiles = (int32_t)((b.k + 63) / 64);
  a.j.blocks = (int32_t)((b.n + 15) / 16);
  a.j.wk = p.wk;
  a.j.seg = p.seg;
  a.x_scale = b.x_scale;
  a.scale = b.scale;
  a.bias = b.bias;
  a.y = b.y;
  static std::atomic<bool> done[kMaxDevices];
  return launch_rows(a, p, &w8_rows_kernel, done, s);
}

}  // namespace bl
