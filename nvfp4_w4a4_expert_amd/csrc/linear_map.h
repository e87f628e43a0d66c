// Kinds, choice of kernel, work split and address arithmetic of the dense linear
// operator (linear.hip).  The kernels form their tiles, parts, copies' offsets and
// places of partial sums through these functions, and a host-side checker
// (tests/host/linear_ranges.cpp) runs the same functions over every workgroup of
// a launch: each tile and each of its K steps is computed once, and every access
// lies inside its buffer.  Plain integer arithmetic, no HIP types.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define NVFP4_LINEAR_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define NVFP4_LINEAR_HD inline
#endif

namespace nvfp4 {
namespace linear_map {

// Operand kinds: 16-bit types, E4M3 with row or block scales, and the wide forms
// of the latter two.
enum { kBf16 = 0, kF16 = 1, kRow8 = 2, kBlock8 = 3, kRow8Wide = 4, kBlock8Wide = 5 };
constexpr bool is_row8(int kind) { return kind == kRow8 || kind == kRow8Wide; }
constexpr bool is_block8(int kind) { return kind == kBlock8 || kind == kBlock8Wide; }
constexpr bool is_wide(int kind) { return kind == kRow8Wide || kind == kBlock8Wide; }
enum { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutBlock8 = 3 };

constexpr int kStep = 128;                                     // bytes of K per step

enum { kFew, kTile64, kTile128, kTile256 };

struct Plan {
  int kernel;
  int32_t tile, tiles_m, tiles_n;
  int32_t whole, parts, part_steps;
  uint64_t bytes;                                              // workspace
  float cost;                                                  // us, by the rates below
};

// What a launch takes, by measured rates in us: `step` per K step of a round (all
// workgroups that the 256 CUs hold at once), `rest` per round (first copies and
// epilogue).
struct Rate { float step, rest; };

inline Rate rate_of(int kind, int kernel) {
  if (kernel == kTile256) return {kind == kBlock8 ? 1.8f : 1.7f, 11.0f};
  if (kernel == kTile128) return {is_wide(kind) ? 1.5f : kind == kBlock8 ? 1.2f : 1.0f, 4.0f};
  return {is_wide(kind) ? 0.8f : 0.42f, 2.0f};
}

// Tiles that fill whole rounds are computed whole.  Those of the last, partly
// filled round may be cut along K into parts that fill it, at the price of a
// second launch that joins the parts and of their sums' way to memory and back
// (about 4 TB/s).  The model's choices against the others, in us, as replays of a
// graph on one set of inputs (in the last-level cache) / on sets of over 800 MB in
// turn (from memory).  8192 x 4224 x 2816 bf16 gated: 128 tiles, the last 64 in 4 parts,
// 191 / 223 (chosen; between calls from Python, outputs in turn, 202); uncut 197 / 244;
// 256 tiles, the last 32 in 4 parts, 193 / 207; uncut 220 / 230: the rates tell the two
// tiles apart by less than the inputs' place does.  4096 x 2816 x 2112 with block scales:
// 256 tiles 40.4 / 46.9 (chosen), 128 tiles 44.8 / 58.5, 64 tiles 69.9 / 86.4.  4096 x 128
// x 2816 bf16: 64 tiles in 4 parts 15.6 / 18.2 (chosen), uncut 17.1 / 18.4; 128 tiles in
// 6 parts 18.9 / 22.0, uncut 27.2 / 51.
inline Plan plan_of(int32_t M, int32_t N, int32_t kbytes, int kind, bool gated) {
  if (M <= 16) return {kFew, 0, 0, 0, 0, 0, 0, 0, 0};
  const int32_t steps = (kbytes + kStep - 1) / kStep;
  Plan best = {};
  float best_cost = 0;
  for (int kernel = kTile64; kernel <= (is_wide(kind) ? kTile128 : kTile256); ++kernel) {
    const int32_t tile = kernel == kTile64 ? 64 : kernel == kTile128 ? 128 : 256;
    const int32_t out_n = gated ? tile / 2 : tile;
    const int32_t slots = kernel == kTile256 ? 256 : 512;
    const int32_t threads = kernel == kTile256 ? 512 : 256;
    Plan q = {kernel, tile, (M - 1) / tile + 1, (N - 1) / out_n + 1, 0, 1, steps, 0, 0};
    // a launch holds at most 2^32 - 1 threads (the callers' limit on sizes leaves
    // room for tiles of 128)
    if ((int64_t)q.tiles_m * q.tiles_n > 0x7FFFFFFF / threads) continue;
    const int32_t total = q.tiles_m * q.tiles_n;
    const Rate r = rate_of(kind, kernel);
    const int32_t left = total % slots;
    const float rounds = (float)(total / slots) * (steps * r.step + r.rest);
    for (int32_t parts = 1; parts <= (left ? (slots / left < 16 ? slots / left : 16) : 1); ++parts) {
      // parts of whole groups of four steps (block scales come in fours)
      int32_t each = parts == 1 ? steps : ((steps + parts - 1) / parts + 3) / 4 * 4;
      const int32_t have = (steps + each - 1) / each;
      if (have != parts) continue;
      float cost = rounds;
      if (left) cost += each * r.step + r.rest;
      if (parts > 1) cost += 3.0f + (float)left * parts * tile * tile * 8.0f / 4e6f;
      if (best_cost == 0 || cost < best_cost) {
        best_cost = cost;
        best = q;
        best.cost = cost;
        best.parts = parts;
        best.part_steps = each;
        best.whole = parts > 1 ? total - left : total;
        best.bytes = parts > 1 ? (uint64_t)left * parts * tile * tile * 4 : 0;
      }
    }
  }
  return best;
}

// 8-bit operands: the exact instructions where fp32's accuracy shows in the output
// (fp32 itself; block scales, which change by a factor of two at a border) and where
// reading w is the bound anyway.
inline int kind_of(int kind, int32_t M, int32_t out_type) {
  if (kind != kRow8 && kind != kBlock8) return kind;
  if (M > 16 && out_type != kOutF32 && out_type != kOutBlock8) return kind;
  return kind == kRow8 ? kRow8Wide : kBlock8Wide;
}

// The tile of a product grouped by expert: M rows over `experts` groups of sizes that only
// the device knows.  row_tiles is the most tiles that M rows can fall into; workgroups
// beyond those in use end at once.
//
// 256-row tiles where the groups fill them on average, 128-row tiles where there are
// enough for the chip, else 64-row tiles; with long rows and few of them 64-row tiles too,
// whose four buffers cover more of the memory's latency.  Measured as 64 / 128 / 256, us,
// a router with likes, 128 experts, hidden 2816, intermediate 704, top-8: gate/up in bf16 of
// 1 token 18 / 32 / -, 4: 28 / 45 / -, 16: 56 / 56 / -, 64: 75 / 86 / -, 256: 113 / 119 / -,
// 512: 150 / 129 / 163, 1024: 219 / 181 / 200, 2048: 359 / 271 / 265, 4096: 615 / 393 / 382;
// with block scales 1: 20 / 30, 16: 49 / 49, 256: 103 / 95, 4096: 546 / 344; down in bf16 of
// 16: 40 / 33 / -, 256: 79 / 67 / -, with block scales 1: 13 / 15, 16: 42 / 33, 4096: 478 / 253.
// 8 experts, top-2, 333 x 1411 x 704 fp16 12.5 / 17 / 36.
//
// 8-bit operands have exact products whatever the result's type and the number of rows, as
// the linear operator's of at most 16 rows: groups often hold a few, and a row would have
// other bits in another batch.  The scaled instruction, which cuts products (linear.hip),
// took 34 us in place of 50 for gate/up of 16 tokens with block scales, 247 in place of 342
// for 4096 and 208 in place of 254 for down of 4096.
struct GroupPlan {
  int kernel;
  int32_t tile, tiles_n;
  int64_t row_tiles;
};

inline GroupPlan group_plan_of(int32_t M, int32_t experts, int32_t N, int32_t kbytes, int kind, bool gated, int out_type) {
  const int32_t groups = M < experts ? M : experts, mean = M / groups;
  // about how many tiles: half a tile's rows of each group are empty
  auto tiles = [&](int32_t tile) {
    const int64_t rows = M / tile + groups / 2;
    return (rows > groups ? rows : groups) * ((N - 1) / (gated ? tile / 2 : tile) + 1);
  };
  GroupPlan q;
  if (mean >= 128 && !is_wide(kind_of(kind, 1, out_type)) && tiles(256) >= 192) {
    q.kernel = kTile256;
    q.tile = 256;
  } else if ((mean > 16 || kbytes <= 24 * kStep) && tiles(128) >= 512) {
    q.kernel = kTile128;
    q.tile = 128;
  } else {
    q.kernel = kTile64;
    q.tile = 64;
  }
  q.tiles_n = (N - 1) / (gated ? q.tile / 2 : q.tile) + 1;
  q.row_tiles = (int64_t)(M - groups) / q.tile + groups;
  return q;
}

// The g-th of `total` workgroups in an order that gives each of the 8 XCDs (which
// receive workgroups in turn) a contiguous range.
NVFP4_LINEAR_HD int32_t xcd_order(int32_t g, int32_t total) {
  const int32_t per = total / 8, rest = total % 8, xcd = g % 8;
  return xcd * per + (xcd < rest ? xcd : rest) + g / 8;
}

// Place of workgroup `block` of a grouped product of row_tiles x tiles_n tiles: the tile
// row among all groups' and the column, row -1 where there is none.  Tiles differ in
// cost (a group's last one has few rows), so runs of kRun tile rows, which mostly share
// their expert's weight, go to the XCDs in turn; of those that are left in the end each
// XCD gets an equal run of tiles.
constexpr int32_t kRun = 2;                                    // (1 to 8 differ by under 3 %)
NVFP4_LINEAR_HD void group_place(int32_t block, int32_t row_tiles, int32_t tiles_n, int32_t& row, int32_t& column) {
  const int32_t turns = row_tiles / (8 * kRun), left = (row_tiles - 8 * kRun * turns) * tiles_n;
  const int32_t xcd = block % 8, i = block / 8;
  if (i < turns * kRun * tiles_n) {
    const int32_t r = i / tiles_n;
    row = (r / kRun * 8 + xcd) * kRun + r % kRun;
    column = i % tiles_n;
    return;
  }
  const int32_t at = (i - turns * kRun * tiles_n) * 8 + xcd;
  const int32_t g = at < left ? xcd_order(at, left) : 0;
  row = at < left ? 8 * kRun * turns + g / tiles_n : -1;
  column = g % tiles_n;
}

// Workgroups that hold every place of at most row_tiles tile rows.
NVFP4_LINEAR_HD int64_t group_blocks(int64_t row_tiles, int32_t tiles_n) { return (row_tiles * tiles_n + 7) / 8 * 8; }

// Tile number -> (tile row, tile column): bands of 8 tile rows, each walked down
// its columns, so that neighbours share rows of a and of w in their L2.
NVFP4_LINEAR_HD void tile_at(int32_t tiles_m, int32_t tiles_n, int32_t t, int32_t& tm, int32_t& tn) {
  constexpr int32_t kBand = 8;
  const int32_t band = t / (kBand * tiles_n);
  const int32_t rows = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  const int32_t in = t - band * kBand * tiles_n;
  tm = band * kBand + in % rows;
  tn = in / rows;
}

// What workgroup `block` computes: a tile, whole (part -1) or one part of its K
// steps.
struct Work {
  int32_t tile, tm, tn, part, step0, steps;
};

NVFP4_LINEAR_HD Work work_at(int32_t block, int32_t tiles_m, int32_t tiles_n, int32_t whole, int32_t parts,
                             int32_t part_steps, int32_t kbytes) {
  const int32_t all = (kbytes + kStep - 1) / kStep;
  Work w;
  if (block < whole) {
    w.tile = xcd_order(block, whole);
    w.part = -1;
    w.step0 = 0;
    w.steps = all;
  } else {
    const int32_t left = tiles_m * tiles_n - whole;
    const int32_t q = xcd_order(block - whole, left * parts);
    w.part = q / left;
    w.tile = whole + q % left;
    w.step0 = w.part * part_steps;
    w.steps = part_steps < all - w.step0 ? part_steps : all - w.step0;
  }
  tile_at(tiles_m, tiles_n, w.tile, w.tm, w.tn);
  return w;
}

// Last row of a tile of `rows` rows from row `from` of a tensor of `have` rows.
NVFP4_LINEAR_HD int32_t last_row_of(int32_t rows, int32_t have, int64_t from) {
  return (int32_t)(have - from < rows ? have - from : rows) - 1;
}

// What a lane of a wavefront copies of each step: from `first` on, 8 * loads rows of
// the operands' tiles (bm rows of a, then out_n rows of w, gated a further out_n),
// all of one operand; the lane's rows are row0, row0 + 8, ... of that part (gate and
// up rows counted apart), its 16 bytes those of `chunk`.
struct Copies {
  bool of_a, of_up;
  int32_t row0, chunk;
};

NVFP4_LINEAR_HD Copies copies_at(int32_t wave, int32_t lane, int32_t loads, int32_t bm, int32_t out_n) {
  const int32_t first = wave * loads * 8;
  Copies c;
  c.of_a = first < bm;
  c.of_up = first >= bm + out_n;
  c.row0 = (c.of_a ? first : (first - bm) % out_n) + (lane >> 3);
  c.chunk = (lane & 7) ^ (lane >> 3);                          // (row & 7) == lane >> 3
  return c;
}

// Offset in its operand of the part's first row, at the first step: tile rows from m0
// (a) or n0 (w, whose up rows follow its N gate rows) on; strides in bytes.
NVFP4_LINEAR_HD int64_t copy_base(const Copies& c, int64_t m0, int32_t n0, int32_t N, int64_t lda, int64_t ldw,
                                  int32_t step0) {
  return (c.of_a ? m0 * lda : (n0 + (c.of_up ? (int64_t)N : 0)) * ldw) + (int64_t)step0 * kStep;
}

// Bytes of a row in the last of `steps` steps from step0 on.
NVFP4_LINEAR_HD int32_t last_bytes(int32_t kbytes, int32_t step0, int32_t steps) {
  const int32_t left = kbytes - (step0 + steps - 1) * kStep;
  return left < kStep ? left : kStep;
}

// Offset of a lane's 16 bytes from its operand's tile at a step: row of the tile
// (at most the last one) and chunk of the step.
NVFP4_LINEAR_HD uint32_t copy_offset(int32_t row, int32_t last_row, uint32_t ld, int32_t chunk) {
  return (uint32_t)(row < last_row ? row : last_row) * ld + (uint32_t)chunk * 16;
}

// Place of a sum among the partial sums: [cut tile][part][row][column].
NVFP4_LINEAR_HD int64_t partial_at(int32_t tile, int32_t part, int32_t parts, int32_t row, int32_t col, int32_t bm,
                                   int32_t bn) {
  return (((int64_t)tile * parts + part) * bm + row) * bn + col;
}

}  // namespace linear_map
}  // namespace nvfp4
