// Host-side planning of the products of int8 activations with 8-bit and with a
// gated block's ternary weights, past 16 tokens: which tile, and in how many parts
// the sum is split.  From the shapes alone, so that the workspace queries agree
// with the calls.
//
// Plain C++ (no HIP), so that the host tests can build it on its own.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

struct CodesPlan {
  int cfg;
  int slabs, tiles_i, tiles_j, ksplit, kspw;
};

// Tile sizes (tokens x outputs), the workgroups a CU holds of them, and, measured
// on an MI355X: the time of a slab of a workgroup by itself on its CU and with the
// CU full, and the time to start a tile and write its outputs (us).
struct CodesConfig {
  int ti, tj, per_cu;
  float alone, full, put;
};
constexpr CodesConfig kW8Configs[4] = {{32, 128, 2, 0.45f, 0.48f, 2.0f},
                                       {64, 128, 2, 0.50f, 0.70f, 2.0f},
                                       {128, 128, 2, 0.75f, 1.25f, 3.0f},
                                       {256, 256, 1, 1.50f, 2.00f, 4.0f}};
constexpr CodesConfig kGatedConfigs[4] = {{32, 128, 2, 0.30f, 0.40f, 2.0f},
                                          {64, 64, 2, 0.30f, 0.40f, 2.0f},
                                          {128, 128, 2, 0.90f, 1.75f, 4.0f},
                                          {256, 128, 1, 1.10f, 1.75f, 4.0f}};
constexpr int kCodesCus = 256;  // MI355X

// The tile and the parts with the smallest estimated time.
inline CodesPlan plan_codes(int64_t m, int64_t n, int64_t slabs, bool gated) {
  CodesPlan best = {};
  float least = 0.0f;
  for (int cfg = 0; cfg < 4; ++cfg) {
    const CodesConfig& C = gated ? kGatedConfigs[cfg] : kW8Configs[cfg];
    const int64_t ti = (m + C.ti - 1) / C.ti, tj = (n + C.tj - 1) / C.tj, tiles = ti * tj;
    for (int want = 1; want <= 16; ++want) {
      if (want > 1 && (slabs < 4 * want || tiles * want > 4 * kCodesCus)) break;
      const int64_t kspw = (slabs + want - 1) / want, parts = (slabs + kspw - 1) / kspw;
      const int64_t wgs = tiles * parts, room = kCodesCus * C.per_cu;
      const int64_t rounds = (wgs + room - 1) / room;
      const bool full = wgs > kCodesCus;
      float us = (float)rounds * ((float)kspw * (full ? C.full : C.alone) + C.put);
      // one more launch, the sums written and read back
      if (parts > 1) us += 4.0f + 8.0f * (float)parts * (float)m * (float)n * (gated ? 2.0f : 1.0f) / 5e6f;
      if (best.slabs && us >= least) continue;
      least = us;
      best = CodesPlan{cfg, (int)slabs, (int)ti, (int)tj, (int)parts, (int)kspw};
    }
  }
  return best;
}

}  // namespace bl
