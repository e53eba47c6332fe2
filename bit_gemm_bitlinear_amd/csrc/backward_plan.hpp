// Host-side planning of BitLinear's gradients: which kernel takes a shape, with
// which tiles, and in how many parts each product's sum is split.  From the
// shapes alone, so that the workspace queries agree with the calls.
//
// Plain C++ (no HIP), so that the host tests can build it on its own.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

constexpr int kSlab = 64;         // c per slab
constexpr int kStep = 2 * kSlab;  // of a step of the one-launch kernel

struct BackwardPlan {
  int cfg[2], ksplit[2], kspw[2];  // dx, dw
  int order;                       // which of them goes first
  bool direct;                     // the one-launch kernel instead
};

// Tile sizes, with what the plan needs to know of each, measured on an
// MI355X: the time of a slab when the CU's other tiles keep the matrix cores
// busy, that of a slab of a tile by itself (the latency of a step), and the
// time to start a tile and write its outputs, bf16 or fp32 (us).
struct Config {
  int ti, tj;
  float slab, alone, put16, put32;
};
constexpr Config kConfigs[3] = {{64, 64, 0.22f, 0.36f, 0.4f, 1.0f},
                                {128, 128, 0.49f, 0.60f, 1.5f, 3.2f},
                                {256, 256, 1.55f, 1.55f, 4.5f, 11.0f}};
constexpr int kPlanCus = 256;  // MI355X
constexpr int kMinPart = 4;    // slabs of a part
constexpr float kFinishUs = 3.0f;  // one more launch
constexpr float kBytesPerUs = 6e6f;
constexpr float kPrepareUs = 5.0f;  // the operands' launch, empty
// A step of the one-launch kernel as above, alone for dx and dw, and its start.
constexpr float kDirectUs = 1.1f, kDirectAloneUs[2] = {1.3f, 2.8f}, kDirectStartUs = 1.5f;

inline int64_t slabs_of(int64_t c) { return (c + kSlab - 1) / kSlab; }

// When kPlanCus CUs are done with na tiles of time a, dealt out first, and nb
// of time b, each to the CU that is free first.
inline float makespan(int64_t na, float a, int64_t nb, float b) {
  const int64_t q = na / kPlanCus, more = na % kPlanCus;
  const float l1 = q * a, l2 = more ? l1 + a : l1;  // kPlanCus - more CUs, `more` CUs
  if (nb == 0) return l2;
  const float mean = ((kPlanCus - more) * l1 + more * l2 + nb * b) / kPlanCus;
  // tiles of the second kind that the two groups of CUs have room for by `mean`
  // (no schedule ends before it), then one more a CU, whichever group ends it first
  int64_t c1 = (int64_t)std::max(0.0f, (mean - l1) / b), c2 = (int64_t)std::max(0.0f, (mean - l2) / b);
  float t = mean;
  while ((kPlanCus - more) * c1 + more * c2 < nb) {
    const float t1 = l1 + (c1 + 1) * b, t2 = l2 + (c2 + 1) * b;
    t = more && t2 < t1 ? t2 : t1;
    ++(more && t2 < t1 ? c2 : c1);
  }
  return std::max(t, l2);
}

// Per product the tile size and the parts of its sum, with the smallest
// estimated time of all together.  256 x 256 tiles are a kernel of their own.
inline BackwardPlan plan_backward(int64_t m, int64_t n, int64_t k, bool dx, bool dw) {
  const int64_t rows[2] = {m, n}, slabs[2] = {slabs_of(n), slabs_of(m)};
  const bool want[2] = {dx, dw};
  struct Option {
    int cfg, ksplit, kspw;
    int64_t count;
    float us, alone, finish;
  };
  Option opt[2][24];
  int num[2] = {0, 0};
  static const int kParts[] = {1, 2, 3, 4, 6, 8, 12, 16};
  for (int j = 0; j < 2; ++j) {
    if (!want[j]) {  // one option, for each kernel, of no tiles
      opt[j][num[j]++] = Option{0, 1, 1, 0, 0.0f, 0.0f, 0.0f};
      opt[j][num[j]++] = Option{2, 1, 1, 0, 0.0f, 0.0f, 0.0f};
      continue;
    }
    for (int c = 0; c < 3; ++c) {
      const Config& C = kConfigs[c];
      const int64_t tiles = ((rows[j] + C.ti - 1) / C.ti) * ((k + C.tj - 1) / C.tj);
      if ((c == 0 && tiles > 16 * kPlanCus) || (c == 2 && tiles < kPlanCus / 16)) continue;
      for (const int p : kParts) {
        if (p > 1 && (slabs[j] < p * kMinPart || tiles * p > 8 * kPlanCus)) break;
        Option o;
        o.cfg = c;
        o.kspw = (int)((slabs[j] + p - 1) / p);
        o.ksplit = (int)((slabs[j] + o.kspw - 1) / o.kspw);
        o.count = tiles * o.ksplit;
        const float put = j == 1 || o.ksplit > 1 ? C.put32 : C.put16;
        o.us = o.kspw * C.slab + put;
        o.alone = o.kspw * C.alone + put;
        o.finish = o.ksplit > 1 ? 4.0f * rows[j] * k * (o.ksplit + 1) / kBytesPerUs : 0.0f;
        opt[j][num[j]++] = o;
      }
    }
  }
  // The one-launch kernel: its longest sum's steps one after the other, or all
  // its steps where they fill the chip; no other launch, no operands to write.
  const int64_t step[2] = {(n + kStep - 1) / kStep, (m + kStep - 1) / kStep};
  float direct = 0.0f, steps = 0.0f;
  for (int j = 0; j < 2; ++j) {
    if (!want[j]) continue;
    const float tiles = (float)((rows[j] + 63) / 64) * (float)((k + 63) / 64);
    direct = std::max(direct, step[j] * kDirectAloneUs[j]);
    steps += tiles * (step[j] * kDirectUs + (j ? kConfigs[0].put32 : kConfigs[0].put16));
  }
  direct = kDirectStartUs + std::max(direct, steps / kPlanCus);
  const Option *best0 = nullptr, *best1 = nullptr;
  float best = 0.0f;
  for (int x = 0; x < num[0]; ++x)
    for (int y = 0; y < num[1]; ++y) {
      const Option &a = opt[0][x], &b = opt[1][y];
      if ((a.cfg == 2) != (b.cfg == 2)) continue;
      const float finish = a.finish + b.finish > 0.0f ? kFinishUs + a.finish + b.finish : 0.0f;
      // what no order of the tiles can beat
      const float least = std::max(std::max(a.alone, b.alone), (a.count * a.us + b.count * b.us) / kPlanCus);
      if (best0 && least + finish >= best) continue;
      const float us = finish + std::max(least, a.us >= b.us ? makespan(a.count, a.us, b.count, b.us)
                                                             : makespan(b.count, b.us, a.count, a.us));
      if (best0 && us >= best) continue;
      best = us;
      best0 = &a;
      best1 = &b;
    }
  const float operands = (dx ? 2.0f * m * n + 0.25f * n * k : 0.0f) + (dw ? 2.0f * m * n + 2.0f * m * k : 0.0f);
  if (direct <= best + kPrepareUs + 2.0f * operands / kBytesPerUs) return BackwardPlan{{0, 0}, {1, 1}, {1, 1}, 0, true};
  return BackwardPlan{{best0->cfg, best1->cfg}, {best0->ksplit, best1->ksplit}, {best0->kspw, best1->kspw},
                      best0->us >= best1->us ? 0 : 1, false};  // the longer tiles first
}

// dy's own rows are slabs already: whole ones, 16-byte aligned.
inline bool dy_as_is(int64_t n) { return n % kSlab == 0; }

}  // namespace bl
