// Host-side checks of the linear operator with 4-bit weights
// (nvfp4_w4a4_expert_amd/csrc/linear4_map.h, through which the kernels form their work and
// addresses), built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer.  For
// each case it plans the launch and walks its workgroups: every tile's steps are computed
// exactly once, every copy and scale of every lane lies inside its row, the copies of a
// step fill their part of LDS once, and partial sums lie inside the workspace.  Given
// lines "M N K kind mx gated" on its input and the argument "plan" it prints their plans.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "nvfp4_w4a4_expert_amd/csrc/linear4_map.h"

using namespace nvfp4::linear4_map;

static void need(bool ok, const char* what, long a = 0, long b = 0) {
  if (!ok) {
    printf("FAILED: %s (%ld, %ld)\n", what, a, b);
    exit(1);
  }
}

// LDS of the tiles, and that a step's copies fill a buffer once, each chunk at its place.
static void check_lds(int fm, int waves, bool mx) {
  const int stage = tile4_stage(fm, waves), scales = 2 * 32 * waves * 4 * (mx ? 4 : 8);
  need(tile4_stages(fm) * stage + scales <= 160 * 1024 / (waves == 4 ? 2 : 1), "LDS of the workgroups of a CU", stage, scales);
  need(16 * fm * (32 * waves + 4) * 4 <= tile4_stages(fm) * stage, "the epilogue's tile");
  need(tile4_a_bytes(fm) % (1024 * waves) == 0 && tile4_loads_a(fm, waves) >= 1, "whole copies of a");
  std::vector<int> seen(stage / 16, 0);
  for (int wave = 0; wave < waves; ++wave)
    for (int lane = 0; lane < 64; ++lane) {
      const int loads = tile4_loads_a(fm, waves);
      for (int i = 0; i < loads; ++i) {
        const Copy4 c = a_copy4(wave, lane, i, loads);
        const int at = (wave * loads + i) * 1024 + lane * 16;
        need(c.row >= 0 && c.row < 16 * fm && c.chunk >= 0 && c.chunk < 16, "a's copy", c.row, c.chunk);
        need(at == c.row * 256 + ((c.chunk ^ (c.row & 15)) << 4), "a's place", c.row, c.chunk);
        ++seen[at / 16];
      }
      for (int i = 0; i < 2; ++i) {
        const Copy4 c = w_copy4(wave, lane, i);
        const int at = tile4_a_bytes(fm) + (2 * wave + i) * 1024 + lane * 16;
        need(c.row >= 0 && c.row < 32 * waves && c.chunk == w_copy4(wave, lane, 0).chunk && c.chunk >= 0 && c.chunk < 4, "w's copy", c.row, c.chunk);
        need(at == tile4_a_bytes(fm) + c.row * 64 + ((c.chunk ^ (c.row >> 1 & 3)) << 4), "w's place", c.row, c.chunk);
        ++seen[at / 16];
      }
    }
  for (int n : seen) need(n == 1, "every chunk of a buffer once", n);
}

static void check_tile(const Work& w, const Plan4& p, int32_t M, int32_t N, int32_t K, bool mx, bool gated) {
  const int waves = p.rows_w / 32, out_n = gated ? p.rows_w / 2 : p.rows_w, loads = tile4_loads_a(p.fm, waves);
  const int64_t m0 = (int64_t)w.tm * p.bm, rows = gated ? 2 * (int64_t)N : N;
  const int32_t n0 = w.tn * out_n;
  need(m0 < M && n0 < N, "tile starts inside", m0, n0);
  for (int wave = 0; wave < waves; ++wave)
    for (int lane = 0; lane < 64; ++lane)
      for (int ks : {0, w.steps - 1}) {
        const int32_t left = K - (w.step0 + ks) * kStep4;
        need(left >= 32, "a step of whole chunks", left);
        for (int i = 0; i < loads; ++i) {
          const Copy4 c = a_copy4(wave, lane, i, loads);
          const int64_t row = a_row4(m0, c.row, M), at = (int64_t)(w.step0 + ks) * 256 + c.chunk * 16;
          if (c.chunk * 8 < left) need(row >= m0 && row < M && at + 16 <= 2 * (int64_t)K, "a's copy inside", row, at);
        }
        for (int i = 0; i < 2; ++i) {
          const Copy4 c = w_copy4(wave, lane, i);
          const int64_t row = w_row4(n0, c.row, N, out_n), at = (int64_t)(w.step0 + ks) * 64 + c.chunk * 16;
          if (c.chunk * 32 < left) need(row >= n0 && row < rows && at + 16 <= K / 2, "w's copy inside", row, at);
          need((c.row >= out_n) == (row >= N), "gate and up rows apart", c.row, row);
        }
      }
  // block scales: four steps at a time, those past the end of the row are left out
  const int32_t nblk = K / (mx ? 32 : 16), blocks = mx ? 4 : 8;
  need(w.step0 % 4 == 0, "scales come in fours", w.step0);
  for (int ks = 0; ks < w.steps; ks += 4) need((int64_t)(w.step0 + ks) * blocks < nblk, "a group of scales", ks);
}

static Plan4 plan(int32_t M, int32_t N, int32_t K, int kind, bool mx, bool gated) { return plan4_of(M, N, K, kind, mx, gated); }

static void check(int32_t M, int32_t N, int32_t K, int kind, bool mx, bool gated) {
  const Plan4 p = plan(M, N, K, kind, mx, gated);
  const bool split = mx && kind == kF16;
  if (p.form == Plan4::kFew) {
    need(M <= (split ? 64 : 16), "few rows", M);
    return;
  }
  if (p.form == Plan4::kWide) {
    need(M > (split ? 64 : 16), "written out", M);
    const Plan q = plan_of(M, N, (split ? 4 : 2) * K, split ? kBf16 : kind, gated);
    need(q.kernel != kFew && (int64_t)q.tiles_m * q.tile >= M, "the linear operator's tiles");
    return;
  }
  need(!split && (p.fm == 1 || p.fm == 2 || p.fm == 4 || p.fm == 8), "tiles", p.fm);
  need(p.bm == 16 * p.fm && p.rows_w == (p.fm == 8 ? 256 : 128), "a tile that is launched", p.bm, p.rows_w);
  const int out_n = gated ? p.rows_w / 2 : p.rows_w;
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n, left = total - p.whole, blocks = p.whole + left * p.parts;
  need((int64_t)p.tiles_m * p.bm >= M && (int64_t)p.tiles_n * out_n >= N, "tiles cover the result");
  need(p.parts >= 1 && p.whole >= 0 && p.whole <= total && (left == 0) == (p.parts == 1), "split", p.whole, p.parts);
  need(blocks * 2 * p.rows_w < (int64_t)1 << 32, "threads of a launch", blocks);
  need(p.bytes == (size_t)(left ? left * p.parts : 0) * p.bm * p.rows_w * 4, "workspace");
  if (total > 100000) return;                                  // the walk below only for launches of a sane length
  const int32_t all = (K + kStep4 - 1) / kStep4;
  std::vector<int32_t> done(total, 0);
  for (int64_t b = 0; b < blocks; ++b) {
    const Work w = work_at((int32_t)b, p.tiles_m, p.tiles_n, p.whole, p.parts, p.part_steps, K);
    need(w.tile >= 0 && w.tile < total && w.tm >= 0 && w.tm < p.tiles_m && w.tn >= 0 && w.tn < p.tiles_n, "tile", w.tile);
    need(w.steps >= 1 && w.step0 >= 0 && w.step0 + w.steps <= all, "steps", w.step0, w.steps);
    need((w.part < 0) == (w.tile < p.whole), "whole tiles first", w.tile);
    done[w.tile] += w.steps;
    if (w.part >= 0) {
      const int64_t lo = partial_at(w.tile - p.whole, w.part, p.parts, 0, 0, p.bm, p.rows_w);
      const int64_t hi = partial_at(w.tile - p.whole, w.part, p.parts, p.bm - 1, p.rows_w - 1, p.bm, p.rows_w);
      need(w.part < p.parts && lo >= 0 && (uint64_t)(hi + 1) * 4 <= p.bytes && hi - lo + 1 == (int64_t)p.bm * p.rows_w, "partial sums", lo, hi);
    }
    if (b < 8 || b + 8 >= blocks || w.tm == p.tiles_m - 1 || w.tn == p.tiles_n - 1) check_tile(w, p, M, N, K, mx, gated);
  }
  for (int64_t t = 0; t < total; ++t) need(done[t] == all, "every step of a tile once", t, done[t]);
}

int main(int argc, char** argv) {
  if (argc > 1 && !strcmp(argv[1], "plan")) {
    int32_t M, N, K, kind, mx, gated;
    while (scanf("%d %d %d %d %d %d", &M, &N, &K, &kind, &mx, &gated) == 6) {
      const Plan4 p = plan(M, N, K, kind, mx != 0, gated != 0);
      if (p.form == Plan4::kTile)
        printf("tile %d %d %d\n", p.fm, p.whole, p.tiles_m * p.tiles_n - p.whole);
      else
        printf("%s 0 0 0\n", p.form == Plan4::kFew ? "few" : "wide");
    }
    return 0;
  }
  for (int mx = 0; mx < 2; ++mx) {
    check_lds(1, 4, mx != 0);
    check_lds(2, 4, mx != 0);
    check_lds(4, 4, mx != 0);
    check_lds(8, 8, mx != 0);
  }
  const int32_t ms[] = {1, 16, 17, 31, 33, 64, 65, 77, 128, 200, 300, 512, 1000, 4096, 8192};
  const int32_t ns[] = {1, 31, 64, 130, 704, 1411, 2112, 8192};
  const int32_t ks[] = {32, 96, 128, 160, 416, 704, 1056, 2112, 2816, 8192};
  long n = 0;
  for (int32_t M : ms)
    for (int32_t N : ns)
      for (int32_t K : ks)
        for (int kind : {kBf16, kF16})
          for (int mx = 0; mx < 2; ++mx)
            for (int gated = 0; gated < 2; ++gated) {
              check(M, N, K, kind, mx != 0, gated != 0);
              ++n;
            }
  // the limits of the entry point: 2^20 tiles of 256, N of 2^24, K of 2^22
  for (int kind : {kBf16, kF16})
    for (int mx = 0; mx < 2; ++mx)
      for (int gated = 0; gated < 2; ++gated) {
        check(1 << 18, (1 << 18) >> gated, 32, kind, mx != 0, gated != 0);
        check(1 << 28, 256 >> gated, 32, kind, mx != 0, gated != 0);
        check(17, 1 << 24, 32, kind, mx != 0, gated != 0);
        check(64, 1 << 24, 1024, kind, mx != 0, gated != 0);
        check(40, 1 << 13, 1 << 21, kind, mx != 0, gated != 0);
        if (!(mx && kind == kF16)) check(70, 1 << 13, 1 << 22, kind, mx != 0, gated != 0);
        n += 6;
      }
  printf("linear4 ranges ok: %ld cases\n", n);
  return 0;
}
