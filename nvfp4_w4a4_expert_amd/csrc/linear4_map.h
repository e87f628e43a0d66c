// Choice of form, work split and address arithmetic of the linear operator with weights
// in 4 bits (linear4.hip).  The kernels form their tiles' copies and scales through these
// functions, and a host-side test (tests/host/linear4_ranges.cpp) runs the same
// functions over the workgroups of a launch: each tile and each of its steps is computed
// once, and every access lies inside its buffer.  Plain integer arithmetic, no HIP types.
#pragma once

#include <stddef.h>

#include "linear_map.h"

namespace nvfp4 {
namespace linear4_map {

using namespace linear_map;

constexpr int kStep4 = 128;                                    // elements of K per step

// The tile of 16 fm rows of a and 32 rows of w a wavefront: bytes of LDS and copies of
// 1 KiB, four rows of a (256 bytes a step) or sixteen of w (64 bytes of codes).
constexpr int tile4_stages(int fm) { return fm == 1 ? 5 : fm == 2 ? 4 : 3; }
constexpr int tile4_a_bytes(int fm) { return 16 * fm * 256; }
constexpr int tile4_stage(int fm, int waves) { return tile4_a_bytes(fm) + 32 * waves * 64; }
constexpr int tile4_loads_a(int fm, int waves) { return tile4_a_bytes(fm) / (1024 * waves); }

// What a lane copies with copy i of its wavefront: the row of the tile and its 16-byte
// chunk, chunk c of row r at place c ^ (r & 15) (a), c ^ (r >> 1 & 3) (w).
struct Copy4 {
  int32_t row, chunk;
};
NVFP4_LINEAR_HD Copy4 a_copy4(int32_t wave, int32_t lane, int32_t i, int32_t loads) {
  const int32_t row = 4 * (wave * loads + i) + (lane >> 4);
  return {row, (lane & 15) ^ (row & 15)};
}
NVFP4_LINEAR_HD Copy4 w_copy4(int32_t wave, int32_t lane, int32_t i) {
  return {16 * (2 * wave + i) + (lane >> 2), (lane & 3) ^ (lane >> 3 & 3)};
}

// Row of a or w behind a row of the tile; rows past the edge repeat the last one.  The
// tile's rows of w: out_n of them, gated: then their up rows.
NVFP4_LINEAR_HD int64_t a_row4(int64_t m0, int32_t row, int32_t M) { return m0 + row < M ? m0 + row : (int64_t)M - 1; }
NVFP4_LINEAR_HD int64_t w_row4(int32_t n0, int32_t row, int32_t N, int32_t out_n) {
  const int32_t n = n0 + row % out_n;
  return (int64_t)(n < N ? n : N - 1) + (row >= out_n ? N : 0);
}

// Which form: fp16 against UE8M0 scales, whose split costs too much in every workgroup,
// takes the first up to 64 rows and the last beyond.
struct Plan4 {
  enum { kFew, kTile, kWide } form;
  int32_t fm, bm, rows_w, tiles_m, tiles_n, whole, parts, part_steps;
  size_t bytes;
  float cost;
};

// Tiles that fill whole rounds of the CUs are computed whole, those of the last round cut
// along K, as the linear operator's (plan_of).
inline Plan4 tile4_plan(int32_t M, int32_t N, int32_t K, bool gated, int fm, int waves, int32_t slots, float step, float rest) {
  Plan4 q = {};
  q.form = Plan4::kTile;
  q.fm = fm;
  q.bm = 16 * fm;
  q.rows_w = 32 * waves;
  q.tiles_m = (M - 1) / q.bm + 1;
  q.tiles_n = (N - 1) / (gated ? q.rows_w / 2 : q.rows_w) + 1;
  const int32_t steps = (K + kStep4 - 1) / kStep4;
  const int64_t total = (int64_t)q.tiles_m * q.tiles_n;
  if (total > 0x7FFFFFFF / (64 * waves)) {                     // (threads of a launch; the largest tiles always fit)
    q.cost = 3e38f;
    return q;
  }
  const int32_t left = (int32_t)(total % slots);
  const float rounds = (float)(total / slots) * (steps * step + rest);
  for (int32_t parts = 1; parts <= (left ? (slots / left < 16 ? slots / left : 16) : 1); ++parts) {
    const int32_t each = parts == 1 ? steps : ((steps + parts - 1) / parts + 3) / 4 * 4;  // (scales come in fours)
    if ((steps + each - 1) / each != parts) continue;
    float cost = rounds;
    if (left) cost += each * step + rest;
    if (parts > 1) cost += 3.0f + (float)left * parts * q.bm * q.rows_w * 8.0f / 8e6f;
    if (q.cost == 0 || cost < q.cost) {
      q.cost = cost;
      q.parts = parts;
      q.part_steps = each;
      q.whole = (int32_t)(parts > 1 ? total - left : total);
      q.bytes = parts > 1 ? (size_t)left * parts * q.bm * q.rows_w * 4 : 0;
    }
  }
  return q;
}

// Forms' costs in us, by measured rates, and the least of them.  Few rows: w at 3 MB/us,
// and a again for every 16 rows of w at 14 MB/us from L2.  Tiles of 16, 32, 64 and 128 rows:
// a step is bound by widening w (E4M3 to bf16 16 instructions for 8 elements of a lane, to
// fp16 8, UE8M0 4).  Written out: 2.5 bytes an element at 5.3 MB/us, then the linear
// operator.  Forms measured against each other, in us, at 8192 x 8192 with E4M3 scales in
// bf16 (few, tiles of 16, 32, 64, 128, written out): 1 row 17, 19, 22, 29, 47, 71; 16 rows
// 26, 20, 21, 28, 47, 81; 64 rows -, 38, 27, 28, 46, 80; 256 rows -, 119, 66, 58, 51, 118;
// 1024 rows -, 448, 245, 184, 141, 174.  4096 x (2 x 2112) x 2816: 64-row tiles 142, 128-row
// tiles 130, written out 114.
// Sums of parts pass at 8 MB/us (written and read once, mostly in the last-level cache;
// plan_of's choices are measured with half that rate).  With half that rate here as well,
// and 7 us beside the steps of the 16- and 32-row tiles, against 8 and 4:
// 8192 x 8192 in bf16 58.4 and 51.9 for 256 rows, 96.0 and 84.4 for 512; 512 x (2 x 2112) x
// 2816 34.7 and 33.2; 16 rows with UE8M0 16.4 and 15.6; but 256 x 1411 x 2112 with UE8M0
// 12.0 and 14.2, 512 x 1411 x 2112 20.2 and 21.2, 300 x 8192 x 8192 with UE8M0 69.6 and 71.4.
inline Plan4 plan4_of(int32_t M, int32_t N, int32_t K, int kind, bool mx, bool gated) {
  Plan4 few = {}, wide = {};
  few.form = Plan4::kFew;
  wide.form = Plan4::kWide;
  if (mx && kind == kF16) return M <= 64 ? few : wide;
  const float rows = gated ? 2.0f * N : (float)N, weights = rows * K;
  const int c = mx ? 2 : kind == kF16 ? 1 : 0;
  static const float kStepUs[4][3] = {{0.9f, 0.76f, 0.58f}, {0.95f, 0.8f, 0.74f}, {1.38f, 1.27f, 1.08f}, {2.1f, 2.0f, 1.87f}};
  Plan4 best = tile4_plan(M, N, K, gated, 1, 4, 512, kStepUs[0][c], 4.0f);
  auto take = [&](const Plan4& q) {
    if (q.cost < best.cost) best = q;
  };
  if (M > 16) take(tile4_plan(M, N, K, gated, 2, 4, 512, kStepUs[1][c], 4.0f));
  if (M > 32) take(tile4_plan(M, N, K, gated, 4, 4, 512, kStepUs[2][c], 6.0f));
  if (M > 64) take(tile4_plan(M, N, K, gated, 8, 8, 256, kStepUs[3][c], 10.0f));
  if (M <= 16) {
    few.cost = 4.0f + weights * 0.5625f / 3e6f + weights / 16 * M * 2 / 14e6f;
    take(few);
  } else {
    wide.cost = 6.0f + weights * 2.5f / 5.3e6f + plan_of(M, N, 2 * K, kind, gated).cost;
    take(wide);
  }
  return best;
}

}  // namespace linear4_map
}  // namespace nvfp4
