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
  int64_t used = 0;
  std::vector<int64_t> start;
  for (int32_t s : sizes) {
    start.push_back(used);
    used += (s + q.tile - 1) / q.tile;
  }
  need(used <= q.row_tiles, "the grid holds all row tiles", used, q.row_tiles);
  const int64_t total = used * q.tiles_n;
  need(q.row_tiles * q.tiles_n <= 0x7FFFFFFF, "32-bit numbers", total);
  std::vector<char> seen(total, 0);
  for (int64_t block = 0; block < total; ++block) {
    const int32_t g = xcd_order((int32_t)block, (int32_t)total), at = g / q.tiles_n;
    size_t e = 0;
    while (start[e] + (sizes[e] + q.tile - 1) / q.tile <= at) ++e;
    need(e < sizes.size() && sizes[e] > 0, "a group with rows", e);
    const int32_t tiles = (sizes[e] + q.tile - 1) / q.tile;
    int32_t tm, tn;
    tile_at(tiles, q.tiles_n, (int32_t)(g - start[e] * q.tiles_n), tm, tn);
    need(tm >= 0 && tm < tiles && tn >= 0 && tn < q.tiles_n, "tile of the group", tm, tn);
    const int64_t id = (start[e] + tm) * q.tiles_n + tn;
    need(!seen[id], "each tile once", id);
    seen[id] = 1;
  }
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
