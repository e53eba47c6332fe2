// 8-bit weights with a scale per output channel: packing, and the product with
// int8 activations.
//
//   y[m][n] = bf16( (sum_k q[m][k] * v[n][k]) * s[n] / x_scale[m] )
//
// Storage (bitlinear_ffn.h): 16 rows x 64 k are one contiguous kilobyte, 16
// bytes (consecutive k of one row) a lane of a wavefront: an operand of the
// 16x16x64 int8 matrix-core op.  Sums are exact in int32.
#include "../../include/bitlinear_ffn.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"

namespace bl {

namespace {

// A workgroup a row: its largest magnitude, its scale, its codes.  Rows past N
// and codes past K are zeros.
__global__ __launch_bounds__(256) void w8_pack_kernel(const float* __restrict__ w, int64_t n, int64_t k,
                                                      int64_t rows, int8_t* __restrict__ codes,
                                                      float* __restrict__ scale) {
  __shared__ float red[4];
  const int64_t ktiles = (k + 63) / 64;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float* src = w + row * k;
    float a = 0.0f;
    if (row < n)
      for (int64_t e = 4 * threadIdx.x; e < k; e += 1024) {  // K % 4 == 0
        typedef float v4f __attribute__((ext_vector_type(4)));
        const v4f v = *G(reinterpret_cast<const v4f*>(src + e));
        a = fmaxf(fmaxf(a, fmaxf(fabsf(v[0]), fabsf(v[1]))), fmaxf(fabsf(v[2]), fabsf(v[3])));
      }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor(a, o));
    __syncthreads();  // the last row's values are read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float s = a / 127.0f;
    if (s == 0.0f) s = 1.0f;
    if (row < n && threadIdx.x == 0) *G(scale + row) = s;
    for (int64_t e = 4 * threadIdx.x; e < ktiles * 64; e += 1024) {
      uint32_t b = 0;
      if (row < n && e < k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = (int)fminf(fmaxf(rintf(*G(src + e + i) / s), -127.0f), 127.0f);
          b |= ((uint32_t)v & 255u) << (8 * i);
        }
      const int64_t at = (((row >> 4) * ktiles + (e >> 6)) * 4 + ((e >> 4) & 3)) * 256 + 16 * (row & 15) + (e & 15);
      *G(reinterpret_cast<uint32_t*>(codes + at)) = b;
    }
  }
}

__global__ __launch_bounds__(256) void w8_unpack_kernel(const int8_t* __restrict__ codes,
                                                        const float* __restrict__ scale, int64_t n, int64_t k,
                                                        float* __restrict__ out) {
  const int64_t ktiles = (k + 63) / 64, total = n * k;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / k, e = i - row * k;
    const int64_t at = (((row >> 4) * ktiles + (e >> 6)) * 4 + ((e >> 4) & 3)) * 256 + 16 * (row & 15) + (e & 15);
    out[i] = *G(scale + row) * (float)*G(codes + at);
  }
}

struct W8KernelArgs {
  const int8_t* q;
  const float* x_scale;
  const int8_t* codes;
  const float* scale;
  const uint16_t* bias;
  uint16_t* y;
  int32_t m, n, k;
  int32_t ktiles, blocks;
};

// One wave: 16 outputs of 16 tokens.
__global__ __launch_bounds__(64) void w8_kernel(const W8KernelArgs A) {
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const int blk = blockIdx.x, m0 = (int)blockIdx.y * 16;
  const int8_t* cp = A.codes + (int64_t)blk * A.ktiles * 1024 + 16 * lane;
  const int64_t m = min(m0 + lr, A.m - 1);
  const int8_t* qp = A.q + m * A.k;
  v4i acc = {0, 0, 0, 0};
  for (int t = 0; t < A.ktiles; ++t) {
    const v4i w = *G(reinterpret_cast<const v4i*>(cp + (int64_t)t * 1024));
    v4i x;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int k = 64 * t + 16 * lg + 4 * d;
      x[d] = k < A.k ? *G(reinterpret_cast<const int32_t*>(qp + k)) : 0;
    }
    acc = mfma_16x16x64_i8(w, x, acc);
  }
  if (m0 + lr >= A.m) return;
  const float xs = *G(A.x_scale + m);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = 16 * blk + 4 * lg + e;
    if (n >= A.n) continue;
    uint16_t y = f32_to_bf16((float)acc[e] * *G(A.scale + n) / xs);
    if (A.bias) y = add_bf16(y, *G(A.bias + n));
    *G(A.y + m * A.n + n) = y;
  }
}

}  // namespace

hipError_t launch_w8_pack(const float* w, int64_t n, int64_t k, int8_t* codes, float* scale, hipStream_t s) {
  const int64_t rows = (n + 15) / 16 * 16;
  w8_pack_kernel<<<(unsigned)(rows < 65536 ? rows : 65536), 256, 0, s>>>(w, n, k, rows, codes, scale);
  return hipGetLastError();
}

hipError_t launch_w8_unpack(const int8_t* codes, const float* scale, int64_t n, int64_t k, float* out,
                            hipStream_t s) {
  const int64_t grid = (n * k + 255) / 256;
  w8_unpack_kernel<<<(unsigned)(grid < 65536 ? grid : 65536), 256, 0, s>>>(codes, scale, n, k, out);
  return hipGetLastError();
}

size_t w8_forward_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_w8_forward(const W8Args& b, char*, hipStream_t s) {
  W8KernelArgs a = {};
  a.q = b.q;
  a.x_scale = b.x_scale;
  a.codes = b.codes;
  a.scale = b.scale;
  a.bias = b.bias;
  a.y = b.y;
  a.m = (int32_t)b.m;
  a.n = (int32_t)b.n;
  a.k = (int32_t)b.k;
  a.ktiles = (int32_t)((b.k + 63) / 64);
  a.blocks = (int32_t)((b.n + 15) / 16);
  w8_kernel<<<dim3((unsigned)a.blocks, (unsigned)((b.m + 15) / 16)), 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
