// Host-side checks of the grouped products' grid and tile numbering
// (nvfp4_w4a4_expert_amd/csrc/linear_map.h), built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer: whatever the groups' sizes, the grid holds every tile, the
// numbering meets each tile of each group once, and the entry point's limits keep all
// numbers in 32 bits.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "nvfp4_w4a4_expert_amd/csrc/linear_map.h"

using namespace nvfp4::linear_map;

static void need(bool ok, const char* what, long a = 0, long b = 0) {
  if (!ok) {
    printf("FAILED: %s (%ld, %ld)\n", what, a, b);
    exit(1);
  }
}

// Walks every workgroup of a launch as the kernels do.
static void walk(const std::vector<int32_t>& sizes, int32_t N, bool gated, int kind, int out_type) {
  int64_t M = 0;
  for (int32_t s : sizes) M += s;
  if (M == 0) return;
  const GroupPlan q = group_plan_of((int32_t)M, (int32_t)sizes.size(), N, 2816 * 2, kind, gated, out_type);
  int64_t used = 0;                                            // tile rows of all groups
  for (int32_t s : sizes) used += (s + q.tile - 1) / q.tile;
  const int64_t total = used * q.tiles_n;
  need(used <= q.row_tiles, "the grid holds all row tiles", used, q.row_tiles);
  const int64_t blocks = group_blocks(q.row_tiles, q.tiles_n);
  need(blocks <= 0x7FFFFFFF && blocks >= total, "32-bit numbers", blocks);
  std::vector<char> seen(total, 0);
  std::vector<int64_t> per_xcd(8, 0);
  for (int64_t block = 0; block < blocks; ++block) {
    int32_t row, column;
    group_place((int32_t)block, (int32_t)used, q.tiles_n, row, column);
    if (row < 0) continue;
    need(row < used && column >= 0 && column < q.tiles_n, "a place", row, column);
    const int64_t id = (int64_t)row * q.tiles_n + column;
    need(!seen[id], "each tile once", id);
    seen[id] = 1;
    ++per_xcd[block % 8];
  }
  const auto range = std::minmax_element(per_xcd.begin(), per_xcd.end());
  need(*range.second - *range.first <= 1, "XCDs get equal numbers", *range.first, *range.second);
  for (char c : seen) need(c, "every tile");
}

int main() {
  std::mt19937 rng(1);
  long n = 0;
  for (int round = 0; round < 400; ++round) {
    const int E = 1 + (int)(rng() % (round % 4 == 0 ? 1024 : 20));
    std::vector<int32_t> sizes(E, 0);
    for (auto& s : sizes) {
      const int kind = (int)(rng() % 5);
      s = kind == 0 ? 0 : kind == 1 ? 1 : kind == 2 ? (int)(rng() % 20) : kind == 3 ? (int)(64 * (rng() % 5)) : (int)(rng() % (round % 7 ? 300 : 3000));
    }
    for (int gated = 0; gated < 2; ++gated)
      for (int out : {kOutBf16, kOutBlock8}) {
        const int kinds[] = {kBf16, kF16, kRow8, kBlock8, kRow8Wide, kBlock8Wide};
        walk(sizes, 32 * (1 + (int)(rng() % 40)), gated != 0, kinds[rng() % 6], out);
        ++n;
      }
  }
  printf("grouped ranges ok: %ld launches\n", n);
  return 0;
}
