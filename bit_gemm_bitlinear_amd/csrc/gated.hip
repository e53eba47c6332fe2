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
// large, exactly; the factor leaves in the epilogue.  Both sums of an output meet in
// one lane, so act(g) * u costs no pass of its own (2048 x 6912 x 2560 with g and u
// kept: 72 us, 2.02 POPS; the plain projections, activation and product as launches
// of their own 118 without keeping them).
#include "../../include/bitlinear_ffn.h"
#include "codes_gemm.hpp"
#include "codes_plan.hpp"
#include "codes_rows.hpp"
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
    v4i v = {0x55555555, 0x55555555, 0x55555555, 0x55555555};
    if (row < n && tiled) {
      v = *G(reinterpret_cast<const v4i*>(src + tiled_chunk_offset(row, o, rb)));
    } else if (row < n && (rb & 15) == 0) {
      if (o < rb) v = *G(reinterpret_cast<const v4i*>(src + row * rb + o));
    } else if (row < n) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (o + e < rb) v[e >> 2] = (v[e >> 2] & ~(0xFF << (8 * (e & 3)))) | ((int)*G(src + row * rb + o + e) << (8 * (e & 3)));
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = (int32_t)gated_dword((uint32_t)v[d]);
    *G(reinterpret_cast<v4i*>(codes + 16 * id)) = v;
  }
}

// act(g) * u.  exp(-|g|) is at most 1 and so is a sigmoid, and act(g) is made before
// it meets u: no step overflows that the result does not (g * u first made NaN of a large
// negative g and a large u, where the result is 0).  exp2 and the reciprocal are the
// hardware's.  exp2's argument is a rounded product, so the error grows with |g|: up to
// (14 + 2 |g|) * 2^-24 of the result (|g| = 80: 1e-5, where it keeps eight bits);
// exp(-|g|) under 2^-126 is 0.
template <bool SILU>
__device__ __forceinline__ float gate_value(float g, float u) {
  if constexpr (!SILU) {
    const float r = g < 0.0f ? 0.0f : g;  // NaN stays NaN
    return (r * u) * r;
  } else {
    const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504f);
    return g * ((g >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e)) * u;
  }
}

// ---------------------------------------------------------------------------
// Up to 16 tokens (codes_rows.hpp).

struct GatedRowsArgs {
  RowsJob j;
  const float* x_scale;
  const float* gate_scale;
  const float* up_scale;
  uint16_t* a;
  uint16_t* g;
  uint16_t* u;
};

template <bool SILU>
__global__ __launch_bounds__(64 * kRowsWaves) void gated_rows_kernel(const GatedRowsArgs A) {
  extern __shared__ __align__(16) int8_t smem[];
  codes_rows_product<1, true>(A.j, smem, [&](int m, int n, const v4i (&acc)[2]) {
    const float xs = *G(A.x_scale + m);
    const RowDiv dg = row_div_setup(xs * *G(A.gate_scale)), du = row_div_setup(xs * *G(A.up_scale));
    float g[4], u[4], a[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g[e] = row_div((float)acc[0][e] * 0.015625f, dg);
      u[e] = row_div((float)acc[1][e] * 0.015625f, du);
      a[e] = gate_value<SILU>(g[e], u[e]);
    }
    const int64_t at = (int64_t)m * A.j.n;
    codes_put4(A.a + at, n, A.j.n, pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    if (A.g) {
      codes_put4(A.g + at, n, A.j.n, pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
      codes_put4(A.u + at, n, A.j.n, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
    }
  });
}

template <bool SILU>
hipError_t launch_gated_rows(const GatedRowsArgs& a, const RowsPlan& p, hipStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  return launch_rows(a, p, &gated_rows_kernel<SILU>, done, s);
}

// ---------------------------------------------------------------------------
// More than 16 tokens: tiles on the int8 matrix cores (codes_gemm.hpp), the
// gate's and the up projection's columns of the same outputs in one wave.

struct GatedGemmArgs {
  CodesJob j;
  const float* x_scale;
  const float* gate_scale;
  const float* up_scale;
  uint16_t* a;
  uint16_t* g;
  uint16_t* u;
};

template <typename T, bool SILU>
__global__ __launch_bounds__(64 * T::NW, 2) void gated_gemm_kernel(const GatedGemmArgs A) {
  extern __shared__ __align__(16) int8_t smem[];
  const CodesJob& J = A.j;
  int ti, tj, kp;
  if (!codes_tile_of((int)blockIdx.x, J, &ti, &tj, &kp)) return;
  v16i acc[T::FI][T::FJ];
  T::run(J, ti, tj, kp, smem, acc);
  constexpr int FO = T::FJ / 2;  // subtiles of outputs
  const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
  const int m0 = ti * T::TI + T::row0() + lr, n0 = tj * T::kCols + T::col0();
  if (J.ksplit > 1) {
#pragma unroll
    for (int i = 0; i < T::FI; ++i) {
      const int m = m0 + 32 * i;
      if (m >= J.m) continue;
#pragma unroll
      for (int j = 0; j < T::FJ; ++j) {
        int32_t* row = J.part + ((int64_t)(2 * kp + (j >= FO)) * J.m + m) * J.ldp;
        codes_put_part(row, n0 + 32 * (j % FO), J.ldp, acc[i][j]);
      }
    }
    return;
  }
  codes_gemm::barrier();
  typename T::Rows rows(smem + T::wave() * T::Rows::kBytes);
  const float gs = load_f32_vmem(A.gate_scale), us = load_f32_vmem(A.up_scale);
#pragma unroll
  for (int i = 0; i < T::FI; ++i) {
    const float xs = *G(A.x_scale + min(m0 + 32 * i, J.m - 1));
    const RowDiv dg = row_div_setup(xs * gs), du = row_div_setup(xs * us);
    auto put = [&](const auto& value) {
#pragma unroll
      for (int j = 0; j < FO; ++j)
#pragma unroll
        for (int a = 0; a < 4; ++a)
          rows.put(lr, 32 * j + 8 * a + 4 * lg, pack_bf16x2(value(j, 4 * a), value(j, 4 * a + 1)),
                   pack_bf16x2(value(j, 4 * a + 2), value(j, 4 * a + 3)));
    };
    // g and u of subtile j's sum r
    auto outputs = [&](auto fastc) {
      auto quotient = [&](int32_t sum, const RowDiv& d) {
        const float v = (float)sum * 0.015625f;
        return decltype(fastc)::value ? row_div_fast(v, d.d, d.y) : v / d.d;
      };
      auto g = [&](int j, int r) { return quotient(acc[i][j][r], dg); };
      auto u = [&](int j, int r) { return quotient(acc[i][j + FO][r], du); };
      put([&](int j, int r) { return gate_value<SILU>(g(j, r), u(j, r)); });
      rows.store(A.a, m0 - lr + 32 * i, n0, J.m, J.n, J.past_cache);
      if (!A.g) return;
      put(g);
      rows.store(A.g, m0 - lr + 32 * i, n0, J.m, J.n, J.past_cache);
      put(u);
      rows.store(A.u, m0 - lr + 32 * i, n0, J.m, J.n, J.past_cache);
    };
    if (__all(dg.fast && du.fast))  // the rows go out together
      outputs(std::true_type{});
    else
      outputs(std::false_type{});
  }
}

// Adds the parts of split sums: eight outputs of a row a thread.
template <bool SILU>
__global__ __launch_bounds__(256) void gated_finish_kernel(const GatedGemmArgs A, int64_t total) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const CodesJob& J = A.j;
  const int cpr = (J.n + 7) >> 3;
  const int64_t m = id / cpr;
  const int n = 8 * (int)(id - m * cpr);
  const int64_t slice = (int64_t)J.m * J.ldp;
  const int32_t* src = J.part + m * J.ldp + n;
  int32_t vg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, vu[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  codes_add_parts(src, 2 * slice, J.ksplit, vg);
  codes_add_parts(src + slice, 2 * slice, J.ksplit, vu);
  const float xs = *G(A.x_scale + m);
  const RowDiv dg = row_div_setup(xs * *G(A.gate_scale)), du = row_div_setup(xs * *G(A.up_scale));
  uint32_t pa[4], pg[4], pu[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float g[2], u[2], a[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      g[e] = row_div((float)vg[2 * h + e] * 0.015625f, dg);
      u[e] = row_div((float)vu[2 * h + e] * 0.015625f, du);
      a[e] = gate_value<SILU>(g[e], u[e]);
    }
    pa[h] = pack_bf16x2(a[0], a[1]);
    pg[h] = pack_bf16x2(g[0], g[1]);
    pu[h] = pack_bf16x2(u[0], u[1]);
  }
  const bool wide = (J.n & 7) == 0;
  codes_put8(A.a + m * J.n, n, J.n, wide, pa);
  if (A.g) {
    codes_put8(A.g + m * J.n, n, J.n, wide, pg);
    codes_put8(A.u + m * J.n, n, J.n, wide, pu);
  }
}

using GatedTile128 = CodesTile<128, 256, 2, 2, 3, true>;
template <bool WORDS>
using GatedTile64 = CodesTile<64, 256, 1, 4, 4, true, WORDS>;
template <bool WORDS>
using GatedTile32 = CodesTile<32, 256, 1, 4, 6, true, WORDS>;

template <typename T, bool SILU>
hipError_t gated_gemm(const GatedGemmArgs& a, hipStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  const int64_t grid = round_up((int64_t)a.j.tiles_i * a.j.tiles_j * a.j.ksplit, 8);
  return codes_launch(&gated_gemm_kernel<T, SILU>, done, dim3((unsigned)grid), 64 * T::NW, T::kLds, T::kLds, s, a);
}

template <bool SILU>
hipError_t launch_gated_gemm(const GatedGemmArgs& a, int cfg, hipStream_t s) {
  const bool words = a.j.ldq % 16 != 0;
  const hipError_t e =
      cfg == 2   ? gated_gemm<GatedTile128, SILU>(a, s)
      : cfg == 1 ? (words ? gated_gemm<GatedTile64<true>, SILU>(a, s) : gated_gemm<GatedTile64<false>, SILU>(a, s))
                 : (words ? gated_gemm<GatedTile32<true>, SILU>(a, s) : gated_gemm<GatedTile32<false>, SILU>(a, s));
  if (e != hipSuccess || a.j.ksplit == 1) return e;
  const int64_t total = (int64_t)a.j.m * ((a.j.n + 7) / 8);
  gated_finish_kernel<SILU><<<(unsigned)((total + 255) / 256), 256, 0, s>>>(a, total);
  return hipGetLastError();
}

struct GatedLayout {
  CodesPlan plan;
  int32_t ldq;
  size_t part, total;
};

GatedLayout gated_layout(int64_t m, int64_t n, int64_t k) {
  GatedLayout L = {};
  L.plan.cfg = -1;
  if (m > 16) L.plan = plan_codes(m, n, k, true);
  if (L.plan.cfg < 0) return L;
  L.ldq = (int32_t)(L.plan.pad ? round_up(k, 16) : k);
  if (L.plan.pad) L.total = align256((size_t)m * L.ldq);
  L.part = L.total;
  if (L.plan.ksplit > 1) L.total = align256(L.total + 8 * (size_t)L.plan.ksplit * m * part_pitch(n));
  return L;
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

size_t gated_forward_bytes(int64_t m, int64_t n, int64_t k) { return gated_layout(m, n, k).total; }

hipError_t launch_gated_forward(const GatedArgs& b, char* ws, hipStream_t s) {
  const GatedLayout L = gated_layout(b.m, b.n, b.k);
  if (L.plan.cfg >= 0) {
    GatedGemmArgs a = {};
    CodesJob& J = a.j;
    J.q = b.q;
    J.ldq = L.ldq;
    J.m = (int32_t)b.m;
    J.n = (int32_t)b.n;
    J.k = (int32_t)b.k;
    J.w = b.codes;
    J.ktiles = (int32_t)((b.k + 255) / 256);
    J.blocks = (int32_t)((b.n + 15) / 16);
    set_plan(J, L.plan, reinterpret_cast<int32_t*>(ws + L.part));
    a.x_scale = b.x_scale;
    a.gate_scale = b.gate_scale;
    a.up_scale = b.up_scale;
    a.a = b.a;
    a.g = b.g;
    a.u = b.u;
    if (L.plan.pad) {
      const hipError_t e = codes_pad(b.q, b.m, b.k, L.ldq, reinterpret_cast<int8_t*>(ws), s);
      if (e != hipSuccess) return e;
      J.q = reinterpret_cast<const int8_t*>(ws);
    }
    return b.silu ? launch_gated_gemm<true>(a, L.plan.cfg, s) : launch_gated_gemm<false>(a, L.plan.cfg, s);
  }
  const RowsPlan p = plan_rows(b.m, b.n, b.k, true);
  GatedRowsArgs a = {};
  a.j.q = b.q;
  a.j.m = (int32_t)b.m;
  a.j.n = (int32_t)b.n;
  a.j.k = (int32_t)b.k;
  a.j.w = b.codes;
  a.j.ktiles = (int32_t)((b.k + 255) / 256);
  a.j.blocks = (int32_t)((b.n + 15) / 16);
  a.j.wk = p.wk;
  a.j.seg = p.seg;
  a.x_scale = b.x_scale;
  a.gate_scale = b.gate_scale;
  a.up_scale = b.up_scale;
  a.a = b.a;
  a.g = b.g;
  a.u = b.u;
  return b.silu ? launch_gated_rows<true>(a, p, s) : launch_gated_rows<false>(a, p, s);
}

}  // namespace bl
