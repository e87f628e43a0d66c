// Host-side check of the addresses that the dense linear operator's tiled kernel
// copies from (nvfp4_w4a4_expert_amd/csrc/linear_map.h: the kernel forms them by
// the very same calls), built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer: every lane's 16 bytes lie in the row and the chunk of
// its operand that the tile needs, each row of a tile is copied once, and 32-bit
// offsets hold up to the longest rows that the entry point takes (2^23 bytes).
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>
#include <vector>

#include "nvfp4_w4a4_expert_amd/csrc/linear_map.h"

using namespace nvfp4::linear_map;

static void need(bool ok, const char* what, long a = 0, long b = 0) {
  if (!ok) {
    printf("FAILED: %s (%ld, %ld)\n", what, a, b);
    exit(1);
  }
}

// All copies of a workgroup's first and last step.
static void check_tile(const Work& w, int tile, int waves, bool gated, int32_t M, int32_t N, int32_t kbytes, int64_t lda,
                       int64_t ldw) {
  const int loads = 2 * tile / 8 / waves, out_n = gated ? tile / 2 : tile;
  const int64_t m0 = (int64_t)w.tm * tile;
  const int32_t n0 = w.tn * out_n;
  const int32_t tail = last_bytes(kbytes, w.step0, w.steps);
  need(tail >= 16 && tail <= kStep && tail % 16 == 0, "whole chunks", tail);
  std::vector<int> seen(2 * tile * 8, 0);
  for (int wave = 0; wave < waves; ++wave)
    for (int lane = 0; lane < 64; ++lane) {
      const Copies c = copies_at(wave, lane, loads, tile, out_n);
      const int64_t ld = c.of_a ? lda : ldw;
      const int32_t last = c.of_a ? last_row_of(tile, M, m0) : last_row_of(out_n, N, n0);
      need(c.chunk >= 0 && c.chunk < 8 && last >= 0, "chunk, last row", c.chunk, last);
      need(!c.of_up || (gated && !c.of_a), "up rows of a gated product only", wave);
      const int64_t base = copy_base(c, m0, n0, N, lda, ldw, w.step0);
      const int64_t first_row = c.of_a ? m0 : n0 + (c.of_up ? (int64_t)N : 0);
      for (int i = 0; i < loads; ++i) {
        const int32_t row = c.row0 + 8 * i;                    // of the tile's part
        need(row >= 0 && row < (c.of_a ? tile : out_n), "row of the part", row);
        // its place in LDS: row of a, gate and up rows in turn, chunk exchanged by the row
        const int place = (c.of_a ? 0 : tile + (c.of_up ? out_n : 0)) + row;
        need(place == (wave * loads + i) * 8 + (lane >> 3), "consecutive places", place, lane);
        need(((lane & 7) ^ (place & 7)) == c.chunk, "place of the chunk", lane);
        ++seen[place * 8 + c.chunk];
        for (int32_t ks : {0, w.steps - 1}) {
          if (c.chunk * 16 >= (ks == w.steps - 1 ? tail : kStep)) continue;
          const uint32_t in_tile = copy_offset(row, last, (uint32_t)ld, c.chunk);
          need(in_tile < (1u << 31), "offset in 31 bits", in_tile);
          const int64_t at = base + (int64_t)ks * kStep + in_tile;
          const int64_t want = first_row + (row < last ? row : last);
          need(at / ld == want && want < (c.of_a ? M : (gated ? 2 : 1) * (int64_t)N), "row of the operand", at / ld, want);
          need(at % ld == (w.step0 + ks) * (int64_t)kStep + c.chunk * 16 && at % ld + 16 <= kbytes, "bytes of the row", at % ld);
        }
      }
    }
  for (size_t i = 0; i < seen.size(); ++i) need(seen[i] == 1, "every chunk of the tile once", (long)i, seen[i]);
}

static long check(int32_t M, int32_t N, int32_t kbytes, int64_t lda, int64_t ldw, int kind, bool gated) {
  const Plan p = plan_of(M, N, kbytes, kind, gated);
  if (p.kernel == kFew) return 0;
  const int64_t blocks = p.whole + ((int64_t)p.tiles_m * p.tiles_n - p.whole) * p.parts;
  long n = 0;
  for (int64_t b = 0; b < blocks; b += b < 24 || b + 24 >= blocks ? 1 : (blocks - 48) / 16 + 1) {
    const Work w = work_at((int32_t)b, p.tiles_m, p.tiles_n, p.whole, p.parts, p.part_steps, kbytes);
    check_tile(w, p.tile, p.kernel == kTile256 ? 8 : 4, gated, M, N, kbytes, lda, ldw);
    ++n;
  }
  return n;
}

int main() {
  long n = 0;
  for (int kind = kBf16; kind <= kBlock8Wide; ++kind)
    for (int gated = 0; gated < 2; ++gated) {
      for (int32_t M : {17, 64, 65, 300, 1000, 4096})
        for (int32_t N : {1, 31, 128, 1411, 2816})
          for (int32_t k : {32, 160, 2112, 2848}) n += check(M, N, k, k + 16, k + 48, kind, gated != 0);
      // the longest rows, short ones at the longest strides, the most rows
      const int32_t top = 1 << 23;
      n += check(17, 1 << 14, top, top, top, kind, gated != 0);
      n += check(4096, 2816, top, top, top, kind, gated != 0);
      n += check(4096, 2816, 2112, top, top, kind, gated != 0);
      n += check(0x7FFFFFFF / 8, 256 >> gated, 64, top, top, kind, gated != 0);
      n += check(16 * 256, (1 << 24) >> gated, 32, top, top, kind, gated != 0);
    }
  printf("linear copies ok: %ld workgroups\n", n);
  return 0;
}
