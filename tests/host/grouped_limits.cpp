// Host-side checks of the grouped products' plan at the limits of the entry point
// (nvfp4_w4a4_expert_amd/csrc/linear_map.h), built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer: what the entry point lets through has 32-bit numbers of
// workgroups, threads and places, on both sides of every branch of the plan.  Given lines
// "rows experts N kbytes kind gated" on its input and the argument "plan" it prints the
// rows of their tiles.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <initializer_list>

#include "nvfp4_w4a4_expert_amd/csrc/linear_map.h"

using namespace nvfp4::linear_map;

static void need(bool ok, const char* what, long a = 0, long b = 0) {
  if (!ok) {
    printf("FAILED: %s (%ld, %ld)\n", what, a, b);
    exit(1);
  }
}

static long taken = 0, refused = 0, tiles[257] = {};

static void check(int32_t M, int32_t E, int32_t N, int32_t kbytes, int kind, bool gated) {
  const GroupPlan q = group_plan_of(M, E, N, kbytes, kind, gated, kOutBf16);
  const bool wide = kind >= kRow8;
  need(q.tile == (q.kernel == kTile256 ? 256 : q.kernel == kTile128 ? 128 : 64), "a tile", q.tile);
  need(!(wide && q.tile == 256), "exact 8-bit products have no 256-row tile");
  const int32_t groups = M < E ? M : E;
  need(q.row_tiles >= (M + q.tile - 1) / q.tile && q.row_tiles >= groups, "row tiles", q.row_tiles);
  // one group with all rows and the others empty, or as many as possible with one row
  need((int64_t)(groups - 1) + (M - groups + 1 + q.tile - 1) / q.tile <= q.row_tiles, "the most tiles", q.row_tiles);
  const int64_t blocks = group_blocks(q.row_tiles, q.tiles_n);
  if (blocks > 0x7FFFFFFF / 512) {                             // the entry point refuses these
    ++refused;
    return;
  }
  ++taken;
  ++tiles[q.tile];
  need(blocks * (q.tile == 256 ? 512 : 256) < (int64_t)1 << 32, "threads of a launch", blocks);
  need(q.row_tiles <= 0x7FFFFFFF, "32-bit tile rows", q.row_tiles);
  for (int64_t block : {(int64_t)0, blocks / 3, blocks - 9, blocks - 1}) {
    if (block < 0) continue;
    for (int64_t used : {(int64_t)1, q.row_tiles / 2 + 1, q.row_tiles}) {
      int32_t row, column;
      group_place((int32_t)block, (int32_t)used, q.tiles_n, row, column);
      need(row < used && row >= -1 && column >= 0 && column < q.tiles_n, "a place", row, column);
    }
  }
}

int main(int argc, char** argv) {
  if (argc > 1 && !strcmp(argv[1], "plan")) {
    int32_t M, E, N, kbytes, kind, gated;
    while (scanf("%d %d %d %d %d %d", &M, &E, &N, &kbytes, &kind, &gated) == 6)
      printf("%d\n", group_plan_of(M, E, N, kbytes, kind, gated != 0, kOutBf16).tile);
    return 0;
  }
  const int32_t ms[] = {1, 16, 17, 127, 128, 1000, 4096, 40000, 1 << 20, 1 << 27, (1 << 29) - 1, 1 << 29};
  const int32_t es[] = {1, 2, 63, 64, 65, 128, 1000, 1024};
  const int32_t ns[] = {1, 32, 63, 64, 65, 704, 1411, 8192, 1 << 18, (1 << 24) - 1, 1 << 24};
  const int32_t ks[] = {16, 128, 24 * kStep - 16, 24 * kStep + 16, 5632, 1 << 23};
  for (int32_t M : ms)
    for (int32_t E : es)
      for (int32_t N : ns)
        for (int32_t k : ks)
          for (int kind = kBf16; kind <= kBlock8; ++kind)
            for (int gated = 0; gated < 2; ++gated) check(M, E, N, k, kind, gated != 0);
  need(tiles[64] > 0 && tiles[128] > 0 && tiles[256] > 0 && refused > 0, "every branch", tiles[256], refused);
  printf("grouped limits ok: %ld launches, %ld refused\n", taken, refused);
  return 0;
}
