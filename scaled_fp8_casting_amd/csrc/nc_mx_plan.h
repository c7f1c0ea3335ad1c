// The choice of a product's kernel, from its sizes, formats and the result's type alone.
// Host code without HIP, so that it also compiles by itself.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "narrowcast.h"

namespace nc {

// How a product is cut up.
struct MxPlan {
  int t;             // few-row kernel: t x t strips a workgroup; 0: the many-row kernel,
  int w;             // 64 w x 64 w results a workgroup
  int32_t splits;    // of the columns
};

constexpr int64_t kMostTiles = UINT32_MAX / 256;   // workgroups of 256 threads of a launch
constexpr int64_t kUnits = 256;                  // compute units
constexpr int64_t kMostSplitTiles = 2 * kUnits;  // tiles of 128 that the card holds at once
constexpr int64_t kSplitChunks = 4;              // fewest chunks of a split

// What the kernels take, in us, with operands that come from memory: a fixed part,
// the results on their way out, and for every chunk of 256 columns the larger of a
// part for each workgroup and of what one compute unit takes for its share of them.
// Fitted to 17 sizes of 33 .. 2048 x 256 .. 11008 x 1024 .. 16384 in each class and
// checked at 70 drawn ones (2 .. 8192 x 40 .. 11008 x 70 .. 16384): the choice was
// within 10% of the fastest in all but those where a launch is most of the time and
// one at 16% (253 x 9025 x 9741 E4M3 x E2M1: 47 us against 40.5 in 3 splits).  At 70
// others (profiles/mx_plans.txt) it was within 4% in 67 and 8, 26 and 27% off in three:
// 5411 x 5679 x 1884 E4M3 x E2M1 takes 82 us at 256 a side and 65 at 128, 485 x 614 x
// 9311 E4M3 23 us with 1 strip and 18 with 2.
// Some of them, in us (1 strip, 2 strips, 128 a side, 256 a side, 128 in 4 splits):
//   E2M1 x E2M1    64 x 4096 x 4096    5.6   9.5  12.4          12.0
//                 512 x 4096 x 4096   18.1  13.4  13.6   27.7   26.6
//                2048 x 2048 x 2048   21.3  16.6  10.3   19.4   35.5
//                4096 x 4096 x 4096                46.5   41.7
//   E4M3 x E4M3    32 x 4096 x 4096    6.1   9.0  14.6          11.6
//                  32 x 4096 x 11008  16.2  26.4  46.9          21.4   (8 splits 19.3; the estimate says 14.0)
//                 256 x 4096 x 4096   21.2  13.3  21.9   43.8   19.7
//                1024 x 1024 x 16384  61.9  35.9  75.6  143.8   32.6
//                4096 x 4096 x 4096                75.5   61.9
//   to fp32, E4M3 x E2M1
//                 777 x 1000 x 1357   10.9   9.8  15.2          17.0
//                1024 x 1024 x 16384  63.3  57.3 112.4          43.4
struct MxCost {
  double few1, few1_floor, few2, few2_floor, many2, many2_floor, many4;
};
constexpr MxCost kCost[4] = {
    {0.00038, 0.105, 0.00080, 0.33, 0.0022, 0.53, 1.95},    // 4 x 4 bits
    {0.00056, 0.160, 0.00105, 0.45, 0.0031, 1.0, 2.75},     // 8 x 4
    {0.00105, 0.245, 0.00125, 0.58, 0.0040, 1.05, 3.2},     // 8 x 8
    {0.00098, 0.220, 0.00160, 0.90, 0.0065, 1.7, 1e9},      // through bf16
};
constexpr double kFewFixed = 3.4, kMany2Fixed = 5.0, kMany4Fixed = 6.5, kJoinFixed = 4.0;
constexpr double kFew1Out = 2.5e6, kFew2Out = 1.3e6, kManyOut = 6e6, kJoinBytes = 4e6;   // bytes in a us

inline MxPlan plan_of(int64_t rows_a, int64_t rows_b, int64_t chunks, int32_t fa, int32_t fb, bool f32) {
  if (chunks == 0) return MxPlan{2, 0, 1};
  const int eight = (fa != NC_E2M1) + (fb != NC_E2M1);
  const MxCost& k = kCost[f32 && eight > 0 ? 3 : eight];
  const double c = (double)chunks, units = (double)kUnits;
  const auto tiles = [&](int64_t side) { return (double)((rows_a + side - 1) / side) * (double)((rows_b + side - 1) / side); };
  const auto rounds = [&](double n) { return std::ceil(n / units); };
  MxPlan best = {1, 0, 1};
  const double n1 = tiles(32), n2 = tiles(64), n4 = tiles(128), n8 = tiles(256);
  const double out = (double)rows_a * (double)rows_b * (f32 ? 4 : 2);
  double least = kFewFixed + out / kFew1Out + c * std::max(n1 * k.few1, rounds(n1) * k.few1_floor);
  const auto offer = [&](MxPlan p, double cost) {
    if (cost < least) {
      least = cost;
      best = p;
    }
  };
  offer({2, 0, 1}, kFewFixed + out / kFew2Out + c * std::max(n2 * k.few2, (0.2 + 0.8 * rounds(n2)) * k.few2_floor));
  offer({0, 2, 1}, kMany2Fixed + out / kManyOut + c * std::max(n4 * k.many2, k.many2_floor));
  offer({0, 4, 1}, kMany4Fixed + out / kManyOut + c * rounds(n8) * k.many4);
  for (int64_t s = 2; s <= chunks / kSplitChunks && n4 * (double)s <= (double)kMostSplitTiles; ++s)
    offer({0, 2, (int32_t)s}, kMany2Fixed + kJoinFixed + std::ceil(c / (double)s) * std::max(n4 * (double)s * k.many2, k.many2_floor) +
                                  8.0 * (double)rows_a * (double)rows_b * (double)s / kJoinBytes);
  // more workgroups than a launch of the few-row kernel has
  if (best.t > 0 && tiles(32 * best.t) > (double)(kMostTiles / 2)) best = MxPlan{0, 2, 1};
  return best;
}

}  // namespace nc
