// Host-side checks of the dense linear operator's work split and addresses
// (nvfp4_w4a4_expert_amd/csrc/linear_map.h, through which the kernels form them),
// built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer.  For each
// case it plans the launch and walks its workgroups: every tile's K steps are
// computed exactly once, every copy of every lane lies inside its operand, and
// every partial sum lies inside the workspace and is read back once.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "nvfp4_w4a4_expert_amd/csrc/linear_map.h"

using namespace nvfp4::linear_map;

static void need(bool ok, const char* what, long a = 0, long b = 0) {
  if (!ok) {
    printf("FAILED: %s (%ld, %ld)\n", what, a, b);
    exit(1);
  }
}

// One wavefront's copies of one step, as the tiled kernel forms them.
static void check_copies(const Work& w, int tile, int waves, bool gated, int32_t M, int32_t N, int32_t kbytes,
                         int64_t lda, int64_t ldw) {
  const int loads = 2 * tile / 8 / waves, out_n = gated ? tile / 2 : tile;
  const int64_t m0 = (int64_t)w.tm * tile, n0 = (int64_t)w.tn * out_n;
  need(m0 < M && n0 < N, "tile starts inside", m0, n0);
  const int tail = std::min(kbytes - (w.step0 + w.steps - 1) * kStep, kStep);
  need(tail >= 1 && tail % 16 == 0, "whole chunks", tail);
  for (int wave = 0; wave < waves; ++wave) {
    const int first = wave * loads * 8;
    const bool is_a = first < tile;
    need(is_a ? first + 8 * loads <= tile : first >= tile, "a wavefront copies one operand", first);
    need(is_a || !gated || (first - tile) / out_n == (first + 8 * loads - 1 - tile) / out_n, "gate or up rows", first);
    const int64_t up = gated && !is_a ? (first - tile) / out_n * (int64_t)N : 0;
    const int64_t ld = is_a ? lda : ldw, rows = is_a ? M : (gated ? 2 * (int64_t)N : N);
    const int64_t from = is_a ? m0 : n0 + up;
    const int last = is_a ? last_row_of(tile, M, m0) : last_row_of(out_n, N, n0);
    for (int lane = 0; lane < 64; ++lane) {
      const int chunk = (lane & 7) ^ (lane >> 3);
      const int row0 = (is_a ? first : (first - tile) % out_n) + (lane >> 3);
      for (int i = 0; i < loads; ++i)
        for (int ks : {0, w.steps - 1}) {
          if (chunk * 16 >= (ks == w.steps - 1 ? tail : kStep)) continue;
          const int64_t in_tile = copy_offset(row0 + 8 * i, last, (uint32_t)ld, chunk);
          const int64_t at = from * ld + (int64_t)(w.step0 + ks) * kStep + in_tile;
          const int64_t row = at / ld, col = at % ld;
          need(row >= 0 && row < rows && col + 16 <= kbytes, "copy inside its row", row, col);
          need(row == from + std::min(row0 + 8 * i, last) && col == (w.step0 + ks) * kStep + chunk * 16, "copy's place", row, col);
        }
    }
  }
}

static void check(int32_t M, int32_t N, int32_t kbytes, int kind, bool gated, bool stride) {
  const Plan p = plan_of(M, N, kbytes, kind, gated);
  if (p.kernel == kFew) {
    need(M <= 16, "few rows");
    return;
  }
  const int out_n = gated ? p.tile / 2 : p.tile, waves = p.kernel == kTile256 ? 8 : 4;
  const int64_t lda = kbytes + (stride ? 16 : 0), ldw = kbytes + (stride ? 48 : 0);
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n, left = total - p.whole;
  need(p.kernel >= kTile64 && p.kernel <= (is_wide(kind) ? kTile128 : kTile256), "a kernel is chosen", p.kernel);
  need((int64_t)p.tiles_m * p.tile >= M && (int64_t)p.tiles_n * out_n >= N, "tiles cover the result");
  need(p.whole >= 0 && p.whole <= total && (left == 0) == (p.parts == 1), "split", p.whole, p.parts);
  const int64_t blocks = p.whole + left * p.parts;
  need(blocks * 64 * waves < (int64_t)1 << 32, "threads of a launch", blocks);
  need(p.bytes == (uint64_t)(left * (left ? p.parts : 0)) * p.tile * p.tile * 4, "workspace");
  if (total > 200000) return;                                  // the walk below only for launches of a sane length
  const int32_t all = (kbytes + kStep - 1) / kStep;
  std::vector<int32_t> done(total, 0);
  for (int64_t b = 0; b < blocks; ++b) {
    const Work w = work_at((int32_t)b, p.tiles_m, p.tiles_n, p.whole, p.parts, p.part_steps, kbytes);
    need(w.tile >= 0 && w.tile < total && w.tm >= 0 && w.tm < p.tiles_m && w.tn >= 0 && w.tn < p.tiles_n, "tile", w.tile);
    need(w.steps >= 1 && w.step0 >= 0 && w.step0 + w.steps <= all, "steps", w.step0, w.steps);
    need(w.part < 0 || !is_block8(kind) || w.step0 % 4 == 0, "block scales in fours", w.step0);
    need((w.part < 0) == (w.tile < p.whole), "whole tiles first", w.tile);
    done[w.tile] += w.steps;
    if (w.part >= 0) {
      need(w.part < p.parts, "part", w.part);
      const int64_t lo = partial_at(w.tile - p.whole, w.part, p.parts, 0, 0, p.tile, p.tile);
      const int64_t hi = partial_at(w.tile - p.whole, w.part, p.parts, p.tile - 1, p.tile - 1, p.tile, p.tile);
      need(lo >= 0 && (uint64_t)(hi + 1) * 4 <= p.bytes && hi - lo + 1 == (int64_t)p.tile * p.tile, "partial sums", lo, hi);
      need(lo == ((int64_t)(w.tile - p.whole) * p.parts + w.part) * p.tile * p.tile, "partial sums apart", lo);
    }
    if (b < 40 || b + 40 >= blocks || w.tm == p.tiles_m - 1 || w.tn == p.tiles_n - 1)
      check_copies(w, p.tile, waves, gated, M, N, kbytes, lda, ldw);
  }
  std::vector<char> seen(total, 0);
  for (int64_t t = 0; t < total; ++t) {
    need(done[t] == all, "every K step of a tile once", t, done[t]);
    int32_t tm, tn;
    tile_at(p.tiles_m, p.tiles_n, (int32_t)t, tm, tn);
    const int64_t at = (int64_t)tm * p.tiles_n + tn;
    need(at >= 0 && at < total && !seen[at], "every tile once", t, at);
    seen[at] = 1;
  }
  // the joining launch: whole blocks of 256 threads, 8 outputs each
  need(p.tile * (out_n / 8) % 256 == 0, "joining blocks", p.tile);
}

int main() {
  const int32_t ms[] = {1, 16, 17, 31, 64, 65, 128, 130, 300, 512, 1000, 2100, 4096, 8192};
  const int32_t ns[] = {1, 31, 32, 128, 130, 704, 1411, 2112, 2816, 8192};
  const int32_t ks[] = {16, 128, 144, 704, 1408, 2112, 2832, 5632, 16384};
  long n = 0;
  for (int32_t M : ms)
    for (int32_t N : ns)
      for (int32_t k : ks)
        for (int kind = kBf16; kind <= kBlock8Wide; ++kind)
          for (int gated = 0; gated < 2; ++gated) {
            check(M, N, is_block8(kind) ? (k + 31) / 32 * 32 : k, kind, gated != 0, (n & 1) != 0);
            ++n;
          }
  // the limits of the entry point: 2^20 tiles of 256, N of 2^24, the longest rows
  for (int kind = kBf16; kind <= kBlock8Wide; ++kind)
    for (int gated = 0; gated < 2; ++gated) {
      check(1 << 18, (1 << 18) >> gated, 32, kind, gated != 0, false);
      check(16 * 256, (1 << 24) >> gated, 32, kind, gated != 0, false);
      check(0x7FFFFFFF / 8, 256 >> gated, 64, kind, gated != 0, false);
      check(17, 1 << 14, 1 << 22, kind, gated != 0, false);
      n += 4;
    }
  printf("linear ranges ok: %ld cases\n", n);
  return 0;
}
