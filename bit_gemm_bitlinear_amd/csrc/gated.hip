// The two projections of a gated feed-forward block, its activation function and
// their product, from int8 activations and ternary weights:
//
//   g = (q . Ug) / (xs wsg),  u = (q . Uu) / (xs wsu),  a = bf16(act(g) * u)
//
// Storage (bitlinear_ffn.h): 16 rows x 256 k of the gate are one contiguous
// kilobyte, the up projection's next to it, 16 bytes (64 weights) a lane of a
// wavefront.  A weight is its two-bit two's complement, so that a shift and a mask
// make four int8 values 64 u of a dword, in the activations' own order: no sum of
// codes to subtract, no activations to reorder.  The sums come out 64 times too
// large, exactly; the factor leaves in the epilogue.
#include "../../include/bitlinear_ffn.h"
#include "common.hpp"
#include "internal.hpp"
#include "layer_internal.hpp"

namespace bl {

namespace {

// Two-bit codes u + 1 of 16 weights (four bytes of four) to the storage's order
// and two's complement: weight 4 d + j at byte j, bits 6 - 2 d.
__device__ __forceinline__ uint32_t gated_dword(uint32_t x) {
  const uint32_t lo = x & 0x55555555u, hi = (x >> 1) & 0x55555555u;
  x = (~lo & 0x55555555u) | ((~(hi ^ lo) & 0x55555555u) << 1);  // u mod 4
  uint32_t t = (x ^ (x >> 6)) & 0x00CC00CCu;                    // 4 x 4 transpose
  x ^= t ^ (t << 6);
  t = (x ^ (x >> 12)) & 0x0000F0F0u;
  x ^= t ^ (t << 12);
  x = ((x >> 4) & 0x0F0F0F0Fu) | ((x & 0x0F0F0F0Fu) << 4);  // fields from the top
  return ((x >> 2) & 0x33333333u) | ((x & 0x33333333u) << 2);
}

// A thread makes 16 bytes of the storage.  Rows past N and weights past K are
// zeros (code 1).
__global__ __launch_bounds__(256) void gated_weights_kernel(const uint8_t* __restrict__ gate, int gate_tiled,
                                                            const uint8_t* __restrict__ up, int up_tiled,
                                                            int64_t n, int64_t k, int64_t ktiles, int64_t total,
                                                            uint8_t* __restrict__ codes) {
  const int64_t rb = k >> 2;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
    const int lane = (int)(id & 63), p = (int)(id >> 6) & 1;
    const int64_t bt = id >> 7, b = bt / ktiles, t = bt - b * ktiles;
    const int64_t row = 16 * b + (lane & 15), o = 64 * t + 16 * (lane >> 4);
    const uint8_t* src = p ? up : gate;
    const bool tiled = p ? up_tiled : gate_tiled;
    v4i v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t w = 0x55555555u;
      if (row < n) {
        if (tiled) {
          w = *G(reinterpret_cast<const uint32_t*>(src + tiled_chunk_offset(row, o, rb) + 4 * d));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t at = o + 4 * d + e;
            if (at < rb) w = (w & ~(0xFFu << (8 * e))) | ((uint32_t)*G(src + row * rb + at) << (8 * e));
          }
        }
      }
      v[d] = (int32_t)gated_dword(w);
    }
    *G(reinterpret_cast<v4i*>(codes + 16 * id)) = v;
  }
}

// int8 values 64 u of the 16 weights of a dword, four a dword, in order.
__device__ __forceinline__ v4i expand16(uint32_t p) {
  v4i r;
  r.x = (int32_t)(p & 0xC0C0C0C0u);
  r.y = (int32_t)((p << 2) & 0xC0C0C0C0u);
  r.z = (int32_t)((p << 4) & 0xC0C0C0C0u);
  r.w = (int32_t)((p << 6) & 0xC0C0C0C0u);
  return r;
}

// act(g) * u.  exp(-|g|) is at most 1, so nothing overflows that the result
// does not; exp2 and the reciprocal are the hardware's, a few steps of fp32 off
// where the result keeps eight bits (and 0 for exp(-|g|) under 2^-126).
template <bool SILU>
__device__ __forceinline__ float gate_value(float g, float u) {
  if constexpr (!SILU) {
    const float r = fmaxf(g, 0.0f);
    return (r * u) * r;
  } else {
    const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504f);
    return g * u * ((g >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e));
  }
}

struct GatedKernelArgs {
  const int8_t* q;
  const float* x_scale;
  const uint8_t* codes;
  const float* gate_scale;
  const float* up_scale;
  uint16_t* a;
  uint16_t* g;
  uint16_t* u;
  int32_t m, n, k;
  int32_t ktiles, blocks;
};

// One wave: 16 outputs of 16 tokens.
template <bool SILU>
__global__ __launch_bounds__(64) void gated_kernel(const GatedKernelArgs A) {
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const int blk = blockIdx.x, m0 = (int)blockIdx.y * 16;
  const uint8_t* cp = A.codes + (int64_t)blk * A.ktiles * 2048 + 16 * lane;
  const int64_t m = min(m0 + lr, A.m - 1);
  const int8_t* qp = A.q + m * A.k;
  v4i ag = {0, 0, 0, 0}, au = {0, 0, 0, 0};
  for (int t = 0; t < A.ktiles; ++t) {
    const v4i wg = *G(reinterpret_cast<const v4i*>(cp + (int64_t)t * 2048));
    const v4i wu = *G(reinterpret_cast<const v4i*>(cp + (int64_t)t * 2048 + 1024));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4i x;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int k = 256 * t + 64 * lg + 16 * s + 4 * d;
        x[d] = k < A.k ? *G(reinterpret_cast<const int32_t*>(qp + k)) : 0;
      }
      ag = mfma_16x16x64_i8(expand16((uint32_t)wg[s]), x, ag);
      au = mfma_16x16x64_i8(expand16((uint32_t)wu[s]), x, au);
    }
  }
  if (m0 + lr >= A.m) return;
  const float xs = *G(A.x_scale + m);
  const RowDiv dg = row_div_setup(xs * *G(A.gate_scale)), du = row_div_setup(xs * *G(A.up_scale));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = 16 * blk + 4 * lg + e;
    if (n >= A.n) continue;
    const float g = row_div((float)ag[e] * 0.015625f, dg), u = row_div((float)au[e] * 0.015625f, du);
    const int64_t o = m * A.n + n;
    *G(A.a + o) = f32_to_bf16(gate_value<SILU>(g, u));
    if (A.g) {
      *G(A.g + o) = f32_to_bf16(g);
      *G(A.u + o) = f32_to_bf16(u);
    }
  }
}

}  // namespace

hipError_t launch_gated_weights(const uint8_t* gate, bool gate_tiled, const uint8_t* up, bool up_tiled,
                                int64_t n, int64_t k, uint8_t* codes, hipStream_t s) {
  const int64_t ktiles = (k + 255) / 256, total = (n + 15) / 16 * ktiles * 128;
  const int64_t grid = (total + 255) / 256;
  gated_weights_kernel<<<(unsigned)(grid < 65536 ? grid : 65536), 256, 0, s>>>(gate, gate_tiled, up, up_tiled, n, k,
                                                                              ktiles, total, codes);
  return hipGetLastError();
}

size_t gated_forward_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gated_forward(const GatedArgs& b, char*, hipStream_t s) {
  GatedKernelArgs a = {};
  a.q = b.q;
  a.x_scale = b.x_scale;
  a.codes = b.codes;
  a.gate_scale = b.gate_scale;
  a.up_scale = b.up_scale;
  a.a = b.a;
  a.g = b.g;
  a.u = b.u;
  a.m = (int32_t)b.m;
  a.n = (int32_t)b.n;
  a.k = (int32_t)b.k;
  a.ktiles = (int32_t)((b.k + 255) / 256);
  a.blocks = (int32_t)((b.n + 15) / 16);
  const dim3 grid((unsigned)a.blocks, (unsigned)((b.m + 15) / 16));
  if (b.silu)
    gated_kernel<true><<<grid, 64, 0, s>>>(a);
  else
    gated_kernel<false><<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bl
