// Host-side planning of the products of int8 activations with 8-bit and with a
// gated block's ternary weights: which kernel, which tile, and in how many parts
// the sum is split.  From the shapes alone, so that the workspace queries agree
// with the calls.
//
// Plain C++ (no HIP), so that the host tests can build it on its own.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

constexpr int kCodesCus = 256;  // MI355X

// ---- weights streamed once for 16 token rows (codes_rows.hpp) ----

constexpr int kRowsWaves = 16;
constexpr int kRowsLds = 80000;  // two workgroups a CU

// K of a tile, and matrices (gate and up).
constexpr int rows_tile_k(bool ternary) { return ternary ? 256 : 64; }
constexpr int rows_mats(bool ternary) { return ternary ? 2 : 1; }

// LDS of a token row of a segment.
constexpr int rows_ldx(int seg, bool ternary) { return (seg * rows_tile_k(ternary) + 255) / 256 * 256 + 16; }

// Waves of a block, and the segments of K.  Of ternary weights as many waves as
// leave at most a workgroup a CU (gated 14336 x 4096 at 16 tokens: 224 workgroups
// of four blocks 9.9 us, 448 of two 12.1, 896 of eight waves 15.2; at one token
// 8.7, 10.3 and 9.1), which stage their tokens once.  8-bit weights have four times
// the bytes a tile's tokens: eight waves a block, or 16 where that would leave CUs
// without a workgroup (32768 x 4096 at 16 tokens: eight 29.1, four 32.9; 14336 x
// 4096: eight 12.8, 16 16.3; 4096 x 4096: 16 7.2, eight 8.3).
struct RowsPlan {
  int wk, seg;
  int64_t lds;
};

inline RowsPlan plan_rows(int64_t m, int64_t n, int64_t k, bool ternary) {
  const int tk = rows_tile_k(ternary), rows = (int)std::min<int64_t>(m, 16);
  const int64_t blocks = (n + 15) / 16, ktiles = (k + tk - 1) / tk;
  RowsPlan p = {};
  p.wk = kRowsWaves;
  if (ternary) {
    while (p.wk > 1 && blocks * p.wk > kCodesCus * kRowsWaves) p.wk /= 2;
  } else if (blocks > kCodesCus) {
    p.wk = 8;
  }
  const int64_t most = std::min<int64_t>(ktiles, (kRowsLds / rows - 16) / 256 * 256 / tk);
  const int64_t segs = (ktiles + most - 1) / most;
  p.seg = (int)((ktiles + segs - 1) / segs);  // of about one size
  p.lds = std::max<int64_t>((int64_t)rows * rows_ldx(p.seg, ternary), (int64_t)kRowsWaves * rows_mats(ternary) * 1024);
  return p;
}

// ---- tiles on the matrix cores (codes_gemm.hpp) ----

struct CodesPlan {
  int cfg;  // tile, or -1: codes_rows.hpp, any number of tokens, 16 at a time
  int slabs, tiles_i, tiles_j, ksplit, kspw;
  bool pad;  // the activations' rows are aligned to 16 bytes first
};

// Tile sizes (tokens x outputs), k of a slab, the workgroups a CU holds, and,
// measured on an MI355X (us): the time of a slab where few CUs have a workgroup,
// where each has one, where the first ones have two and where all have; that to
// start a tile and write its outputs.
struct CodesConfig {
  int ti, tj, slab, per_cu;
  float few, one, two, full, put;
};
constexpr CodesConfig kW8Configs[] = {{64, 64, 64, 2, 0.16f, 0.17f, 0.19f, 0.22f, 1.0f},
                                      {128, 128, 64, 2, 0.22f, 0.28f, 0.50f, 0.68f, 2.9f},
                                      {128, 256, 64, 1, 0.32f, 0.52f, 0.0f, 0.0f, 3.0f},
                                      {256, 256, 64, 1, 0.62f, 0.88f, 0.0f, 0.0f, 5.0f}};
constexpr CodesConfig kGatedConfigs[] = {{32, 128, 128, 2, 0.32f, 0.35f, 0.46f, 0.55f, 1.0f},
                                         {64, 128, 128, 2, 0.41f, 0.47f, 0.68f, 0.86f, 1.8f},
                                         {128, 128, 128, 2, 0.71f, 0.87f, 1.24f, 1.55f, 2.5f}};
constexpr float kCodesStartUs = 3.5f;     // a launch
constexpr float kCodesFinishUs = 3.0f;    // one more, that adds the parts
// One before, that aligns the activations' rows, whatever their bytes (2048 x 4100 codes
// 6 us by itself, 4096 x 12604 20, 16384 x 8196 46, where products of 4096 outputs take
// 41, 213 and 540).
constexpr float kCodesPadUs = 3.0f;
// Rows that are no multiple of 16 bytes: the two smaller tiles load them in words, as
// they are, the larger ones, whose loads count for more, from an aligned copy (words
// against the copy, us: 8-bit 64 x 64 401 x 5316 x 356 14.0 and 15.6, 128 x 256 300 x
// 14336 x 4100 41 and 36, 256 x 256 2048 x 14336 x 4100 139 and 128; gated 1348 x 227 x
// 268 6.1 and 8.0, 300 x 6912 x 2564 24.4 and 23.7).
constexpr int kCodesWordTiles = 2;
constexpr float kCodesStageUs = 3e-4f;    // a column of 16 tokens staged four bytes at a time
constexpr float kCodesBytesPerUs = 6e6f;  // of parts
constexpr float kCodesReadPerUs = 5e6f;   // of weights

// Where the last row that a tile of `ti` tokens has begins, from its first one: rows of
// ldq bytes, of which `left` are left of the product.  The tile's own rows are under 2^25
// bytes, those that are left may be past 2^32.
constexpr uint32_t tile_last_row(int32_t ti, int32_t left, int32_t ldq) {
  return (uint32_t)((left < ti ? left : ti) - 1) * (uint32_t)ldq;
}

// The kernel, tile and parts with the smallest estimated time (m > 16).  Measured
// against single choices (us, 8-bit): 17 x 4096 x 4096 rows 6.6, tiles 10; 64 x 14336
// x 4096 rows 35, tiles of 64 x 64 14.6, of 128 x 128 18, of 256 x 256 in four parts 25;
// 2048 x 4096 x 4096 of 128 x 128 43, of 128 x 256 39, of 256 x 256 55; 2048 x 14336 x
// 4096 139, 137 and 122; 300 x 4096 x 14336 of 128 x 256 in five parts, which it takes,
// 38.8, in four 38.1, of 128 x 128 in two 39, of 256 x 256 in seven 46.  Over 240 drawn
// shapes of each product the choice is 1.6% off the best one on average, over 10% in 14,
// a third at most (8-bit 2449 x 1647 x 9396, of 64 x 64: 98; of 128 x 256 74).
inline CodesPlan plan_codes(int64_t m, int64_t n, int64_t k, bool gated) {
  CodesPlan best = {};
  best.cfg = -1;
  const RowsPlan r = plan_rows(16, n, k, gated);
  const int64_t rtk = rows_tile_k(gated), per = kRowsWaves / r.wk, ktiles = (k + rtk - 1) / rtk;
  const int64_t rwgs = ((n + 15) / 16 + per - 1) / per * ((m + 15) / 16);
  const float tiles = ktiles < r.wk ? (float)ktiles / (float)r.wk : (float)((ktiles + r.wk - 1) / r.wk);  // a wave's
  const float load = std::min(1.0f, (float)rwgs / (2 * kCodesCus));
  float least = kCodesStartUs + (float)((rwgs + 2 * kCodesCus - 1) / (2 * kCodesCus)) *
                                    ((gated ? 1.6f + (1.2f + 0.9f * load) * tiles : 1.0f + (0.6f + 0.5f * load) * tiles) +
                                     (k % 16 ? kCodesStageUs * (float)k : 0.0f));
  // reading the weights (more slowly where CUs have two of the smallest tiles: 8-bit 45 x
  // 9299 x 9620 in two parts of those 38 us, of 128 x 128 in three 27; the gated product's
  // smallest tiles take the same factor, which changed none of its 240 choices)
  const float reading = (float)n * (float)k * (gated ? 0.5f : 1.0f) / kCodesReadPerUs;
  for (int cfg = 0; cfg < (gated ? 3 : 4); ++cfg) {
    const CodesConfig& C = gated ? kGatedConfigs[cfg] : kW8Configs[cfg];
    const int64_t ti = (m + C.ti - 1) / C.ti, tj = (n + C.tj - 1) / C.tj, slabs = (k + C.slab - 1) / C.slab;
    const int64_t room = kCodesCus * C.per_cu;
    // the time of a round of up to `room` tiles
    auto round = [&](int64_t wgs, int64_t kspw) {
      const float share = (float)(wgs > kCodesCus ? wgs - kCodesCus : wgs) / kCodesCus;
      const float slab = wgs > kCodesCus ? C.two + (C.full - C.two) * share : C.few + (C.one - C.few) * share;
      return wgs ? (float)kspw * slab + C.put : 0.0f;
    };
    for (int64_t want = 1; want <= 16; ++want) {
      if (want > 1 && (slabs * C.slab < 512 * want || ti * tj * want > 4 * kCodesCus)) break;
      const int64_t kspw = (slabs + want - 1) / want, parts = (slabs + kspw - 1) / kspw, wgs = ti * tj * parts;
      const bool pad = k % 16 != 0 && cfg >= kCodesWordTiles;
      float us = kCodesStartUs + (pad ? kCodesPadUs : 0.0f) +
                 std::max((float)(wgs / room) * round(room, kspw) + round(wgs % room, kspw),
                          cfg == 0 && wgs > kCodesCus ? 1.3f * reading : reading);
      if (parts > 1)
        us += kCodesFinishUs + 8.0f * (float)parts * (float)m * (float)n * (gated ? 2.0f : 1.0f) / kCodesBytesPerUs;
      if (us >= least) continue;
      least = us;
      best = CodesPlan{cfg, (int)slabs, (int)ti, (int)tj, (int)parts, (int)kspw, pad};
    }
  }
  return best;
}

}  // namespace bl
