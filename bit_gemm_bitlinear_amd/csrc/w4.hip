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

#include <algorithm>

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
  int32_t wk;      // waves sharing a block along K
  int32_t seg;     // K tiles whose activations are in LDS at a time
};

// What a wave holds of U tiles.
template <int GP, int U>
struct W4Chunk {
  v4i c[U];
  v2i s[U][GP];
};

// One workgroup: W / wk blocks of 16 weight rows times up to 16 token rows;
// wk waves share a block along K (contiguous shares of its tiles) and their
// sums are joined in LDS, in wave order.  The token rows' codes are staged in
// LDS first, a segment of K that fits at a time (32 bytes between rows: the 16
// rows of an operand then lie in distinct banks), so a wave's memory loads are
// the weights' alone.  It goes through its tiles U at a time, the next ones
// loading while the current ones multiply.  GP: groups per tile (1, 2 or 4; 1
// also where a group spans tiles).  14336 x 4096 at one token (30 MB): 8.9 us
// from memory, 6.7 where the last-level cache holds the weights; 32768 x 4096 at
// 16 tokens (72 MB): 21.2 us, 3.4 TB/s, and 17.3 (36 us when every wave loaded its
// own activations from memory).  Every further 16 tokens read the weights again:
// 14336 x 4096 at 17 tokens 22.6 us, at 2048 tokens 1353 us (the ternary product of
// that size on the same codes: 119).
template <int W, int GP, int U>
__global__ __launch_bounds__(64 * W) void w4_kernel(const W4Args A) {
  extern __shared__ __align__(16) int8_t xs_lds[];
  __shared__ float red[W][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int blk = (int)blockIdx.x * (W / A.wk) + wave / A.wk;
  const int part = wave % A.wk;
  const int m0 = (int)blockIdx.y * 16, rows = min(16, A.m - m0);
  const int ldx = A.seg * 128 + 32;
  // blocks and token rows past the end read the last one: their sums are not stored
  const int b = min(blk, A.blocks - 1);
  const uint8_t* cp = A.codes + (int64_t)b * A.ktiles * 1024 + 256 * lg + 16 * lr;
  const uint16_t* sp = A.scales + (int64_t)b * A.groups * 16 + 4 * lg;
  const int8_t* xl = xs_lds + min(lr, rows - 1) * ldx + 8 * lg;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  auto load = [&](W4Chunk<GP, U>& h, int tb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u, A.ktiles - 1);
      h.c[u] = *G(reinterpret_cast<const v4i*>(cp + (int64_t)t * 1024));
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const int gi = GP == 1 ? t >> A.gshift : min(GP * t + g, A.groups - 1);
        h.s[u][g] = *G(reinterpret_cast<const v2i*>(sp + (int64_t)gi * 16));
      }
    }
  };

  for (int seg0 = 0; seg0 < A.ktiles; seg0 += A.seg) {
    const int tiles = min(A.seg, A.ktiles - seg0);
    const int per = (tiles + A.wk - 1) / A.wk;
    const int t0 = seg0 + min(part * per, tiles), t1 = min(t0 + per, seg0 + tiles);
    W4Chunk<GP, U> ca, cb;
    if (t0 < t1) load(ca, t0);
    // codes past K are zeros in LDS (they meet the last tile's padding, zeros too)
    if (seg0) __syncthreads();
    const int cpr = tiles * 8;  // 16-byte pieces of a row
    for (int i = threadIdx.x; i < rows * cpr; i += 64 * W) {
      const int r = i / cpr, c = i - r * cpr, k = 128 * seg0 + 16 * c;
      const v4i v = k < A.k ? *G(reinterpret_cast<const v4i*>(A.q + (int64_t)(m0 + r) * A.k + k)) : v4i{0, 0, 0, 0};
      *reinterpret_cast<v4i*>(xs_lds + r * ldx + 16 * c) = v;
    }
    __syncthreads();
    auto multiply = [&](const W4Chunk<GP, U>& h, int tb) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (tb + u >= t1) break;
        v2i x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const v2i*>(xl + 128 * (tb + u - seg0) + 32 * i);
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          v4i acc = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 4 / GP; ++j) {
            const int i = g * (4 / GP) + j;
            const uint32_t d = (uint32_t)h.c[u][i];
            const v2i w = {(int32_t)(d & 0xF0F0F0F0u), (int32_t)((d << 4) & 0xF0F0F0F0u)};
            acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, w),
                                                        __builtin_bit_cast(long, x[i]), acc, 0, 0, 0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t sw = (uint32_t)h.s[u][g][e >> 1];
            const float sf = __uint_as_float((e & 1) ? (sw & 0xFFFF0000u) : (sw << 16));
            sum[e] = __builtin_fmaf(sf, (float)acc[e], sum[e]);
          }
        }
      }
    };
    for (int t = t0; t < t1; t += 2 * U) {
      if (t + U < t1) load(cb, t + U);
      multiply(ca, t);
      if (t + U >= t1) break;
      if (t + 2 * U < t1) load(ca, t + 2 * U);
      multiply(cb, t + U);
    }
  }

#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][e][lane] = sum[e];
  __syncthreads();
  // the first wave of a block finishes it: lane = token lr, rows 4 lg .. 4 lg + 3
  const int n = 16 * blk + 4 * lg;
  if (part != 0 || lr >= rows || n >= A.n) return;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e];
  for (int w = 1; w < A.wk; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += red[wave + w][e][lane];
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

// LDS for activations, with the 1 KB a wave of the join within 64 KB: two
// workgroups a CU.
constexpr int kXBytes8 = 57000, kXBytes16 = 49000;

// Waves per block.  Eight, one block a workgroup, unless
//  * there are few blocks of many tiles (up to one block a CU): sixteen, the
//    memory latency of a wave's share being what counts (4096 x 14336 at one
//    token 8.3 -> 7.8 us, 2048 x 8192 at 16 tokens 13.7 -> 10.6; of few tiles,
//    512 x 1024 at 3 tokens, eight are better: 4.0 -> 3.6); or
//  * there are many blocks and many tokens: as few as leave 16 waves a CU, so
//    that a workgroup stages its activations for several blocks (32768 x 4096
//    at 16 tokens, eight waves a block 29.5 us, two 17.0; at one token, where
//    the activations are small, 12.7 against 13.4; the weights in the last-level
//    cache).
template <int GP>
void launch_w4(W4Args a, hipStream_t s) {
  const int rows = a.m < 16 ? a.m : 16;
  a.wk = 8;
  while (rows > 4 && a.wk > 1 && (int64_t)a.blocks * (a.wk / 2) >= 4096) a.wk /= 2;
  const bool wide = (int64_t)a.blocks <= 256 && a.ktiles >= 64;
  if (wide) a.wk = 16;
  a.seg = std::min(a.ktiles, ((wide ? kXBytes16 : kXBytes8) / rows - 32) / 128);
  const size_t lds = (size_t)rows * (a.seg * 128 + 32);
  const int per = wide ? 1 : 8 / a.wk;
  const dim3 grid((unsigned)((a.blocks + per - 1) / per), (unsigned)((a.m + 15) / 16));
  if (wide)
    w4_kernel<16, GP, 1><<<grid, 1024, lds, s>>>(a);
  else
    w4_kernel<8, GP, 2><<<grid, 512, lds, s>>>(a);
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
  if (group == 32)
    launch_w4<4>(a, s);
  else if (group == 64)
    launch_w4<2>(a, s);
  else
    launch_w4<1>(a, s);
  return hipGetLastError();
}

}  // namespace bl
