// Products of up to 16 rows of int8 activations a workgroup with 8-bit weights
// (w8.hip) or a gated block's two ternary ones (gated.hip), the weights streamed
// once: what decoding takes, where the weights' bytes are the cost.
//
// A workgroup is 16 waves and takes 16 / wk blocks of 16 weight rows; wk waves share
// a block along K (contiguous shares of its tiles), and their int32 sums are joined
// in LDS.  The token rows are staged in LDS, a segment of K that fits at a time, so
// a wave's memory loads are the weights' alone: whole kilobytes, U tiles ahead.  A
// row of LDS is 16 bytes over a multiple of 256, so that the 16 rows of an operand
// lie in distinct banks.
//
// Bound by memory where the weights are many (8-bit 32768 x 4096 at one token: 24.4
// us, 5.5 TB/s), by a launch, one round of loads and the join where they are few
// (gated 6912 x 2560 at one token 4.9 us, 14336 x 4096 at 16 tokens 9.9 us, 3 TB/s: a
// wave has four tiles of its own there; two tiles a load 10.1).
#pragma once

#include "codes_gemm.hpp"
#include "common.hpp"

#include <algorithm>

namespace bl {

struct RowsJob {
  const int8_t* q;  // [m][k]
  int32_t m, n, k;
  const uint8_t* w;
  int32_t ktiles, blocks;  // of the weights' storage
  int32_t wk;              // waves sharing a block
  int32_t seg;             // tiles of K staged at a time
};

// finish(token, first of four outputs, sums [matrices][4]) is called for what
// exists of tokens and of groups of four outputs.
template <int U, bool TERNARY, typename Finish>
__device__ __forceinline__ void codes_rows_product(const RowsJob& J, int8_t* lds, const Finish& finish) {
  constexpr int W = kRowsWaves, TK = rows_tile_k(TERNARY), MATS = rows_mats(TERNARY);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int blk = (int)blockIdx.x * (W / J.wk) + wave / J.wk;
  const int part = wave % J.wk;
  const int m0 = (int)blockIdx.y * 16, rows = min(16, J.m - m0);
  const int ldx = rows_ldx(J.seg, TERNARY);
  // blocks and token rows past the end read the last one: their sums are not stored
  const uint8_t* wp = J.w + (int64_t)min(blk, J.blocks - 1) * J.ktiles * (1024 * MATS) + 16 * lane;
  const int8_t* xl = lds + min(lr, rows - 1) * ldx + (TERNARY ? 64 : 16) * lg;
  const bool aligned = (J.k & 15) == 0;
  v4i acc[MATS];
#pragma unroll
  for (int p = 0; p < MATS; ++p) acc[p] = v4i{0, 0, 0, 0};
  struct Chunk {
    v4i c[U][MATS];
  };
  auto load = [&](Chunk& h, int tb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u, J.ktiles - 1);
#pragma unroll
      for (int p = 0; p < MATS; ++p)
        h.c[u][p] = *G(reinterpret_cast<const v4i*>(wp + ((int64_t)t * MATS + p) * 1024));
    }
  };
  for (int seg0 = 0; seg0 < J.ktiles; seg0 += J.seg) {
    const int tiles = min(J.seg, J.ktiles - seg0);
    const int per = (tiles + J.wk - 1) / J.wk;
    const int t0 = seg0 + min(part * per, tiles), t1 = min(t0 + per, seg0 + tiles);
    Chunk ca, cb;
    if (t0 < t1) load(ca, t0);
    if (seg0) __syncthreads();
    // what lies past K is zeros (as the weights' padding is)
    const int cpr = tiles * (TK / 16);  // 16-byte pieces of a row
    for (int i = threadIdx.x; i < rows * cpr; i += 64 * W) {
      const int r = i / cpr, c = i - r * cpr, k = TK * seg0 + 16 * c;
      const int8_t* src = J.q + (int64_t)(m0 + r) * J.k + k;
      v4i v = {0, 0, 0, 0};
      if (aligned) {
        if (k < J.k) v = *G(reinterpret_cast<const v4i*>(src));
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          if (k + 4 * d < J.k) v[d] = *G(reinterpret_cast<const int32_t*>(src + 4 * d));
      }
      *reinterpret_cast<v4i*>(lds + r * ldx + 16 * c) = v;
    }
    __syncthreads();
    auto multiply = [&](const Chunk& h, int tb) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (tb + u >= t1) break;
        const int8_t* xt = xl + TK * (tb + u - seg0);
        if constexpr (TERNARY) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const v4i x = *reinterpret_cast<const v4i*>(xt + 16 * s);
#pragma unroll
            for (int p = 0; p < MATS; ++p)
              acc[p] = mfma_16x16x64_i8(expand16((uint32_t)h.c[u][p][s]), x, acc[p]);
          }
        } else {
          acc[0] = mfma_16x16x64_i8(h.c[u][0], *reinterpret_cast<const v4i*>(xt), acc[0]);
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
  __syncthreads();  // the rows are done with: their LDS holds the sums now
  v4i* red = reinterpret_cast<v4i*>(lds);
#pragma unroll
  for (int p = 0; p < MATS; ++p) red[(wave * MATS + p) * 64 + lane] = acc[p];
  __syncthreads();
  // the first wave of a block finishes it: lane = token lr, rows 4 lg .. 4 lg + 3
  const int n = 16 * blk + 4 * lg;
  if (part != 0 || lr >= rows || n >= J.n) return;
  for (int w = 1; w < J.wk; ++w)
#pragma unroll
    for (int p = 0; p < MATS; ++p) acc[p] += red[((wave + w) * MATS + p) * 64 + lane];
  finish(m0 + lr, n, acc);
}

// Four consecutive bf16 outputs of a row, those that exist.
__device__ __forceinline__ void codes_put4(uint16_t* row, int n, int cols, uint32_t lo, uint32_t hi) {
  if ((cols & 3) == 0) {
    typedef int32_t v2i __attribute__((ext_vector_type(2)));
    *G(reinterpret_cast<v2i*>(row + n)) = v2i{(int32_t)lo, (int32_t)hi};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < cols) *G(row + n + e) = (uint16_t)((e & 2 ? hi : lo) >> (16 * (e & 1)));
  }
}

template <typename Args, typename Kernel>
hipError_t launch_rows(const Args& a, const RowsPlan& p, Kernel kernel, std::atomic<bool>* done, hipStream_t s) {
  const int per = kRowsWaves / p.wk;
  const dim3 grid((unsigned)((a.j.blocks + per - 1) / per), (unsigned)((a.j.m + 15) / 16));
  return codes_launch(kernel, done, grid, 64 * kRowsWaves, (size_t)p.lds, kRowsLds, s, a);
}

}  // namespace bl
