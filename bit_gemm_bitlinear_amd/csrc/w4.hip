// 4-bit weights with group scales: packing, and the product with int8
// activations.
//
//   y[m][n] = bf16( sum_g s[n][g] * (sum_{k in g} q[m][k] * v[n][k]) / x_scale[m] )
//
// The activations are the same per-token int8 codes that the ternary products
// read, so the sums within a group are integers on the int8 matrix cores
// (v_mfma_i32_16x16x32_i8), exact; the scales enter once per group in fp32.
//
// Storage (bitlinear_layer.h): 16 rows x 128 k are one contiguous kilobyte, 16
// bytes a lane of a wavefront, ordered so that a dword masked with 0xF0F0F0F0
// (the high nibbles) and the same dword shifted left by 4 and masked (the low
// ones) are the lane's eight int8 values of one matrix-core operand: three
// vector instructions for eight weights, no sign correction.  The values come
// out as 16 v; the factor leaves in the epilogue.
#include "../../include/bitlinear_layer.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"

namespace bl {

namespace {

typedef int32_t v2i __attribute__((ext_vector_type(2)));

// One wave per row and group: the group's largest magnitude, its scale, and
// the bytes of the pairs (k, k + 4).  Rows past N and groups past K are zeros.
__global__ __launch_bounds__(256) void w4_pack_kernel(const float* __restrict__ w, int64_t n,
                                                      int64_t k, int group, int64_t groups_pad,
                                                      int64_t total, uint8_t* __restrict__ codes,
                                                      uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t groups = k / group, ktiles = (k + 127) / 128;
  for (int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); id < total;
       id += (int64_t)gridDim.x * 4) {
    const int64_t row = id / groups_pad, gi = id - row * groups_pad;
    const bool real = row < n && gi < groups;
    const float* src = w + row * k + gi * group;
    float a = 0.0f;
    if (real)
      for (int e = lane; e < group; e += 64) a = fmaxf(a, fabsf(src[e]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor(a, o));
    uint16_t sb = real ? f32_to_bf16(a / 7.0f) : (uint16_t)0;
    if (real && sb == 0) sb = 0x3F80;
    const float s = bf16_to_f32(sb);
    for (int p = lane; p < group / 2; p += 64) {
      const int e = 8 * (p >> 2) + (p & 3);
      uint32_t b = 0;
      if (real) {
        const int hi = (int)fminf(fmaxf(rintf(src[e] / s), -8.0f), 7.0f);
        const int lo = (int)fminf(fmaxf(rintf(src[e + 4] / s), -8.0f), 7.0f);
        b = (((uint32_t)hi & 15u) << 4) | ((uint32_t)lo & 15u);
      }
      const int64_t kk = gi * group + e;
      const int r = (int)(kk & 127);
      codes[((((row >> 4) * ktiles + (kk >> 7)) * 4 + ((r >> 3) & 3)) * 16 + (row & 15)) * 16 +
            4 * (r >> 5) + (r & 3)] = (uint8_t)b;
    }
    if (gi < groups && lane == 0) scales[((row >> 4) * groups + gi) * 16 + (row & 15)] = sb;
  }
}

__global__ __launch_bounds__(256) void w4_unpack_kernel(const uint8_t* __restrict__ codes,
                                                        const uint16_t* __restrict__ scales,
                                                        int64_t n, int64_t k, int group,
                                                        float* __restrict__ out) {
  const int64_t groups = k / group, ktiles = (k + 127) / 128, total = n * k;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / k, kk = i - row * k;
    const int r = (int)(kk & 127);
    const uint32_t b = codes[((((row >> 4) * ktiles + (kk >> 7)) * 4 + ((r >> 3) & 3)) * 16 +
                              (row & 15)) * 16 + 4 * (r >> 5) + (r & 3)];
    const int v = (int)(int8_t)((r & 4) ? (b << 4) : (b & 0xF0u)) >> 4;
    out[i] = bf16_to_f32(scales[((row >> 4) * groups + kk / group) * 16 + (row & 15)]) * (float)v;
  }
}

struct W4Args {
  const int8_t* q;
  const float* x_scale;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* bias;
  uint16_t* y;
  int32_t m, n, k;
  int32_t ktiles, groups;
  int32_t gshift;  // log2(group / 128) where a group spans tiles, else 0
  int32_t blocks;  // blocks of 16 rows
};

// One workgroup: R blocks of 16 weight rows times 16 token rows, the K tiles
// dealt out to its W waves and the waves' sums joined in LDS, in wave order.
// GP: groups per tile (1, 2 or 4; 1 also where a group spans tiles).
template <int W, int R, int GP>
__global__ __launch_bounds__(64 * W) void w4_kernel(const W4Args A) {
  __shared__ float red[W][R * 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int blk0 = (int)blockIdx.x * R;
  const int m0 = (int)blockIdx.y * 16;
  const bool live = m0 + lr < A.m;
  const int8_t* qrow = A.q + (int64_t)min(m0 + lr, A.m - 1) * A.k + 8 * lg;
  const uint8_t* cp[R];
  const uint16_t* sp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = min(blk0 + r, A.blocks - 1);
    cp[r] = A.codes + (int64_t)b * A.ktiles * 1024 + 256 * lg + 16 * lr;
    sp[r] = A.scales + (int64_t)b * A.groups * 16 + 4 * lg;
  }
  float sum[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[r][e] = 0.0f;

  for (int t = wave; t < A.ktiles; t += W) {
    v4i c[R];
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = *G(reinterpret_cast<const v4i*>(cp[r] + (int64_t)t * 1024));
    v2i x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = v2i{0, 0};
      if (live && 128 * t + 32 * i < A.k)
        x[i] = *G(reinterpret_cast<const v2i*>(qrow + 128 * t + 32 * i));
    }
    v2i s[R][GP];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        // a group past K (the padding of the last tile) meets zero codes
        const int gi = GP == 1 ? t >> A.gshift : min(GP * t + g, A.groups - 1);
        s[r][g] = *G(reinterpret_cast<const v2i*>(sp[r] + (int64_t)gi * 16));
      }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        v4i acc = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4 / GP; ++j) {
          const int i = g * (4 / GP) + j;
          const uint32_t d = (uint32_t)c[r][i];
          const v2i w = {(int32_t)(d & 0xF0F0F0F0u), (int32_t)((d << 4) & 0xF0F0F0F0u)};
          acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, w),
                                                      __builtin_bit_cast(long, x[i]), acc, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sw = (uint32_t)s[r][g][e >> 1];
          const float sf = __uint_as_float((e & 1) ? (sw & 0xFFFF0000u) : (sw << 16));
          sum[r][e] = __builtin_fmaf(sf, (float)acc[e], sum[r][e]);
        }
      }
  }

#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][4 * r + e][lane] = sum[r][e];
  __syncthreads();
  // wave w finishes blocks w, w + W, ...: lane = token lr, rows 4 lg .. 4 lg + 3
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r % W != wave) continue;
    const int n = 16 * (blk0 + r) + 4 * lg;
    if (!live || n >= A.n) continue;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = red[0][4 * r + e][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v[e] += red[w][4 * r + e][lane];
    }
    const float xs = *G(A.x_scale + m0 + lr);
    uint16_t* yr = A.y + (int64_t)(m0 + lr) * A.n + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= A.n) continue;
      uint16_t o = f32_to_bf16((v[e] * 0.0625f) / xs);
      if (A.bias) o = add_bf16(o, *G(A.bias + n + e));
      *G(yr + e) = o;
    }
  }
}

}  // namespace

hipError_t launch_w4_pack(const float* w, int64_t n, int64_t k, int group, uint8_t* codes,
                          uint16_t* scales, hipStream_t s) {
  const int64_t gpad = (k + 127) / 128 * 128 / group;  // a group over 128 divides K, and K whole tiles
  const int64_t total = (n + 15) / 16 * 16 * gpad;
  const int64_t grid = (total + 3) / 4;
  w4_pack_kernel<<<(unsigned)(grid < 65536 ? grid : 65536), 256, 0, s>>>(w, n, k, group, gpad,
                                                                        total, codes, scales);
  return hipGetLastError();
}

hipError_t launch_w4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t n, int64_t k,
                            int group, float* out, hipStream_t s) {
  const int64_t grid = (n * k + 255) / 256;
  w4_unpack_kernel<<<(unsigned)(grid < 65536 ? grid : 65536), 256, 0, s>>>(codes, scales, n, k,
                                                                          group, out);
  return hipGetLastError();
}

hipError_t launch_w4_forward(int64_t m, int64_t n, int64_t k, int group, const int8_t* q,
                             const float* x_scale, const uint8_t* codes, const uint16_t* scales,
                             const uint16_t* bias, uint16_t* y, hipStream_t s) {
  W4Args a = {};
  a.q = q;
  a.x_scale = x_scale;
  a.codes = codes;
  a.scales = scales;
  a.bias = bias;
  a.y = y;
  a.m = (int32_t)m;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.ktiles = (int32_t)((k + 127) / 128);
  a.groups = (int32_t)(k / group);
  a.blocks = (int32_t)((n + 15) / 16);
  while ((128 << a.gshift) < group) ++a.gshift;
  const dim3 grid((unsigned)a.blocks, (unsigned)((m + 15) / 16));
  if (group == 32) w4_kernel<4, 1, 4><<<grid, 256, 0, s>>>(a);
  else if (group == 64) w4_kernel<4, 1, 2><<<grid, 256, 0, s>>>(a);
  else w4_kernel<4, 1, 1><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
