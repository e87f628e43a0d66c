// Linear operator with weights in 4 bits for gfx950:
//
//   v[m, n] = gain * sum_k a[m, k] * E2M1(w[n, k]) * scale[n, k / 16 or 32],
//
// then the linear operator's epilogue (bias, activation or act(gate) * up, residual, one
// rounding).  a is bf16 or fp16; the scales are E4M3 per 16 elements ("nv") or UE8M0 per
// 32 ("mx"), the gain is one fp32 number or 1.
//
// A weight is made exactly in the type that it is multiplied in: E2M1 times E4M3 has six
// significant bits and lies in [2^-10, 2688], a bf16 as well as an fp16 number; times a
// power of two it is a bf16 number in bf16's range.  fp16 activations against the latter
// are split into two bf16 numbers, the upper 8 of their 11 bits and the lower 3, which
// are multiplied apart: every product is exact and the sums are fp32 sums.
//
// Few rows are bound by reading w once and go from memory to registers
// (linear4_few_kernel).  More rows would read a too often so: tiles, with a and w's codes in
// LDS, widen w once for 16 to 128 rows of a (linear4_tile_kernel).  Many rows are bound by
// the matrix units: w is written out in 16 bits once and the linear operator's tiles
// multiply it.
#include "internal.h"
#include "linear4_map.h"
#include "linear_kernels.h"

namespace nvfp4 {
namespace {

using namespace linear4_map;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Eight elements as 16-bit numbers: a word of codes times the block scale in byte kByte
// of `scales`.
template <bool kMx, bool kHalf, int kByte>
__device__ __forceinline__ u32x4 weights8(uint32_t w, uint32_t scales) {
  if constexpr (kMx) {                                         // (bf16 for either a)
    const float s = __uint_as_float(((scales >> (8 * kByte)) & 0xFFu) << 23);
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
  } else if constexpr (kHalf) {
    const half2_t v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, kByte >= 2);
    const half2_t s = kByte % 2 ? half2_t{v.y, v.y} : half2_t{v.x, v.x};
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s)};
  } else {
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)scales, kByte);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    // (the products are bf16 numbers: their upper halves)
    auto pair = [&](const f32x2_t& x) { return __builtin_amdgcn_perm(__float_as_uint(x.y * s), __float_as_uint(x.x * s), 0x07060302u); };
    return u32x4{pair(a), pair(b), pair(c), pair(d)};
  }
}

// 8 fp16 numbers as bf16 numbers hi + lo: the upper 8 significant bits and the rest.
__device__ __forceinline__ void split_f16(const u32x4& a, u32x4& hi, u32x4& lo) {
  float v[8];
  unpack_f16x8(a, v);
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = __float_as_uint(v[i]) & 0xFFFF0000u;
    const float rest = v[i] - __uint_as_float(h[i]);
    l[i] = (h[i] & 0x7F800000u) == 0x7F800000u ? 0u : __float_as_uint(rest);   // (infinities and NaN are whole)
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = __builtin_amdgcn_perm(h[2 * i + 1], h[2 * i], 0x07060302u);
    lo[i] = __builtin_amdgcn_perm(l[2 * i + 1], l[2 * i], 0x07060302u);
  }
}

// bf16 weights without their infinities, which the upper part of an fp16 number has met
// already: 0 for a lower part of 0, infinity times 0 would be NaN.  Elements are infinite
// from scale code 253 on.
constexpr uint32_t kInfiniteFrom = 253;
__device__ __forceinline__ u32x4 finite_bf16(u32x4 w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
    if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
  }
  return w;
}

// acc += w . a over 32 elements of K, w the row operand
template <bool kMx, bool kHalf>
__device__ __forceinline__ f32x4 mma4(const u32x4& w, const u32x4& a, f32x4 acc) {
  if constexpr (!kMx && kHalf)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w), __builtin_bit_cast(half8_t, a), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
}

// The block scales of 128 elements of a row, `blocks` of them inside it (a multiple of 32
// elements): 8 bytes of E4M3 at an even address, or 4 of UE8M0 at any.  Those past the
// end are zeros.
template <bool kMx>
__device__ __forceinline__ void load_scales4(const uint8_t* at, int32_t blocks, uint32_t* s) {
  constexpr int kWords = kMx ? 1 : 2;
  if (blocks >= 4 * kWords) {
    __builtin_memcpy(s, at, 4 * kWords);
    return;
  }
#pragma unroll
  for (int i = 0; i < kWords; ++i) s[i] = 0;
#pragma unroll
  for (int i = 0; i < 4 * kWords; ++i)
    if (i < blocks) s[i / 4] |= (uint32_t)at[i] << (8 * (i % 4));
}

// ---- few rows -------------------------------------------------------------------
// A workgroup owns 16 * kFN rows of w (gated: gate rows, then up rows) and 16 * kRF rows
// of a.  Its wavefronts take groups of 128 elements of K in turn, kBatch groups' loads in
// flight at once and the next ones' w on its way: a lane's 16 bytes of w are 32 elements
// of a row, the next 32 belong to the next group of 16 lanes, and the four matrix
// instructions of a group take 8 elements of each (any order of K that both operands
// share).  The wavefronts' sums are added in order through LDS, 16 rows at a time.
// One row of 2 x 2112 x 2816 takes 6.6 us (6.7 MB: a launch, two rounds of loads and the
// join in LDS), of 8192 x 8192 17 with E4M3 scales and 15 with UE8M0 (37.7 and 35.7 MB, 2.3
// TB/s: with 16 wavefronts a CU their turns of load and widening leave the memory idle).
template <bool kMx, bool kHalf, int kRF, int kFN, bool kGated>
__global__ __launch_bounds__(512) void linear4_few_kernel(const LinParams p) {
  constexpr int kWaves = 8, kRows = 16 * kFN, kCols = kGated ? kRows / 2 : kRows;
  constexpr int kBatch = kRF * kFN <= 2 ? 2 : 1;
  constexpr int kLd = kRows + 4;                               // floats per row of a partial tile
  constexpr bool kSplit = kMx && kHalf;
  constexpr int kBlock = kMx ? 32 : 16;
  __shared__ __align__(16) float part[kWaves][16][kLd];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int32_t n0 = (int32_t)(blockIdx.x % (uint32_t)p.tiles_n) * kCols;
  const int64_t m0 = (int64_t)(blockIdx.x / (uint32_t)p.tiles_n) * (16 * kRF);
  const int32_t K = p.kbytes / 2;                              // (kbytes: of a row of a)

  const char* pw[kFN];
  const uint8_t* sw[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    const int r = j * 16 + i16;
    int32_t n = n0 + r % kCols;
    n = n < p.N ? n : p.N - 1;
    const int64_t row = (int64_t)n + (r >= kCols ? p.N : 0);
    pw[j] = p.w + row * p.ldw;
    sw[j] = static_cast<const uint8_t*>(p.w_scales) + row * (K / kBlock);
  }
  const char* pa[kRF];
#pragma unroll
  for (int i = 0; i < kRF; ++i) pa[i] = p.a + min(m0 + i * 16 + i16, (int64_t)p.M - 1) * p.lda;
  f32x4 acc[kRF][kFN];
#pragma unroll
  for (int i = 0; i < kRF; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  const int groups = (K + 127) / 128;
  struct Weights {
    u32x4 w[kBatch][kFN];
    uint32_t s[kBatch][kFN];                                   // a lane's two E4M3 codes or one UE8M0 code
  };
  // past the end of a row codes, scales and a count as zeros
  auto load_w = [&](int first, Weights& q) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int32_t k = (first + b) * 128 + 32 * g;
#pragma unroll
      for (int j = 0; j < kFN; ++j) {
        q.w[b][j] = u32x4{0, 0, 0, 0};
        q.s[b][j] = 0;
        if (k < K) {
          q.w[b][j] = *reinterpret_cast<const u32x4*>(pw[j] + k / 2);
          if constexpr (kMx) q.s[b][j] = sw[j][k / 32];
          else q.s[b][j] = *reinterpret_cast<const uint16_t*>(sw[j] + k / 16);
        }
      }
    }
  };
  Weights now, next;
  load_w(kBatch * wave, now);
  for (int first = kBatch * wave; first < groups; first += kBatch * kWaves) {
    load_w(first + kBatch * kWaves, next);
    u32x4 a[kBatch][kRF][4];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int32_t k = (first + b) * 128 + 32 * g;
#pragma unroll
      for (int i = 0; i < kRF; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          a[b][i][t] = u32x4{0, 0, 0, 0};
          if (k < K) a[b][i][t] = *reinterpret_cast<const u32x4*>(pa[i] + 2 * k + 16 * t);
        }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      auto part = [&](auto tc, auto infinite) {
        constexpr int t = decltype(tc)::value;
        u32x4 wt[kFN];
#pragma unroll
        for (int j = 0; j < kFN; ++j) wt[j] = weights8<kMx, kHalf, kMx ? 0 : t / 2>(now.w[b][j][t], now.s[b][j]);
#pragma unroll
        for (int i = 0; i < kRF; ++i) {
          if constexpr (kSplit) {
            u32x4 hi, lo;
            split_f16(a[b][i][t], hi, lo);
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], hi, acc[i][j]);
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(infinite.value ? finite_bf16(wt[j]) : wt[j], lo, acc[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], a[b][i][t], acc[i][j]);
          }
        }
      };
      auto group = [&](auto infinite) {
        part(std::integral_constant<int, 0>{}, infinite);
        part(std::integral_constant<int, 1>{}, infinite);
        part(std::integral_constant<int, 2>{}, infinite);
        part(std::integral_constant<int, 3>{}, infinite);
      };
      if constexpr (kSplit) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kFN; ++j) top = max(top, now.s[b][j]);
        if (__any(top >= kInfiniteFrom)) {                     // (for the whole wavefront)
          group(std::true_type{});
          continue;
        }
      }
      group(std::false_type{});
    }
    now = next;
  }

  constexpr int kKind = kHalf ? (int)kF16 : (int)kBf16;
  constexpr int kQuads = kCols / 4;
#pragma unroll
  for (int i = 0; i < kRF; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < kFN; ++j) *reinterpret_cast<f32x4*>(&part[wave][i16][j * 16 + 4 * g]) = acc[i][j];
    __syncthreads();
    // four outputs per thread, consecutive threads consecutive columns: a block of 32
    // columns is 8 neighbouring lanes
    for (int e = threadIdx.x; e < 16 * kQuads; e += 512) {
      const int r = e / kQuads, c = (e % kQuads) * 4;
      f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < kWaves; ++q) {
        v += *reinterpret_cast<const f32x4*>(&part[q][r][c]);
        if constexpr (kGated) u += *reinterpret_cast<const f32x4*>(&part[q][r][kCols + c]);
      }
      const int64_t m = m0 + i * 16 + r;
      const int32_t n = n0 + c;
      const bool in = m < p.M && n < p.N;
      float gv[4] = {v.x, v.y, v.z, v.w}, uv[4] = {u.x, u.y, u.z, u.w};
      const int64_t mr = min(m, (int64_t)p.M - 1);
      Columns<kKind, kGated, 4> cols;
      cols.load(p, n);
      cols.finish(p, mr, gv, uv);
      Residual<4> res;
      res.load(p, mr, n);
      res.add(p, gv);
      if (p.out_type != kOutBlock8) {
        if (in) store_run<4>(p, m, n, gv);
      } else if constexpr (kCols % 32 == 0) {
        store_block<4>(p, m, n, gv, in);
      }
    }
  }
}

// ---- middle numbers of rows -----------------------------------------------------------
// A workgroup of four wavefronts owns kBM = 16 kFM rows of a and 128 rows of w (gated: 64
// gate rows and their up rows), of eight 128 rows of a and 256 of w, each wavefront 32 of
// the latter, and all or a part of K.  The form above reads a again for every few rows of w
// (64 x 8192 x 8192: 268 MB from L2, 41 us for 27 here), so both go to LDS, 128 elements of
// K a step and w as codes; a wavefront widens its own rows of w, once for all rows of a.
// Lane group g holds elements 32 g .. 32 g + 31 of a step, the t-th matrix instruction
// takes eight of them.  16 x 8192 x 8192 takes 11.9 us with UE8M0 scales and 5 for joining
// eight parts (35.7 MB, 3 TB/s while it runs); from 64 rows on the widening bounds it, which
// more rows a tile share.
template <int kFM, int kWaves>
struct TileOf {
  static constexpr int kBM = 16 * kFM, kRowsW = 32 * kWaves, kThreads = 64 * kWaves;
  static constexpr int kABytes = tile4_a_bytes(kFM), kStage = tile4_stage(kFM, kWaves), kStages = tile4_stages(kFM);
  static constexpr int kLoadsA = tile4_loads_a(kFM, kWaves), kLoads = kLoadsA + 2;  // 1 KiB copies of a wavefront and step
};

template <bool kMx, bool kHalf, int kFM, int kWaves, bool kGated>
__global__ __launch_bounds__(64 * kWaves, 2) void linear4_tile_kernel(const LinParams p) {
  typedef TileOf<kFM, kWaves> Tile;
  constexpr int kBM = Tile::kBM, kStages = Tile::kStages, kRowsW = Tile::kRowsW, kThreads = Tile::kThreads;
  constexpr int kOutN = kGated ? kRowsW / 2 : kRowsW;
  constexpr int kBlocks = kMx ? 4 : 8;                         // block scales of a step and row
  constexpr int kKind = kHalf ? (int)kF16 : (int)kBf16;
  __shared__ __align__(1024) char smem[kStages * Tile::kStage];
  // scales of four steps, two buffers
  __shared__ __align__(16) uint8_t s_scale[2][kRowsW][4 * kBlocks];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int32_t K = p.kbytes;                                  // (128 elements a step, as work_at counts)
  const Work work = work_at((int32_t)blockIdx.x, p.tiles_m, p.tiles_n, p.whole, p.parts, p.part_steps, p.kbytes);
  const int step0 = work.step0, steps = work.steps;
  const int64_t m0 = (int64_t)work.tm * kBM;
  const int32_t n0 = work.tn * kOutN;

  // copies into LDS: where each lane's come from
  const char* from_a[Tile::kLoadsA];
  const char* from_w[2];
  const int chunk_w = w_copy4(wave, lane, 0).chunk;            // (the same in both)
#pragma unroll
  for (int i = 0; i < Tile::kLoadsA; ++i) {
    const Copy4 c = a_copy4(wave, lane, i, Tile::kLoadsA);
    from_a[i] = p.a + a_row4(m0, c.row, p.M) * p.lda + c.chunk * 16 + (int64_t)step0 * 256;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    from_w[i] = p.w + w_row4(n0, w_copy4(wave, lane, i).row, p.N, kOutN) * p.ldw + chunk_w * 16 + (int64_t)step0 * 64;
  auto fetch = [&](int ks) {
    char* to = smem + ks % kStages * Tile::kStage;
    const int32_t left = K - (step0 + ks) * 128;               // elements of the rows from this step on
#pragma unroll
    for (int i = 0; i < Tile::kLoadsA; ++i) {
      char* dst = to + (wave * Tile::kLoadsA + i) * 1024;
      if (a_copy4(wave, lane, i, Tile::kLoadsA).chunk * 8 < left) copy_lds16(reinterpret_cast<uint64_t>(from_a[i]), lds_address(dst));
      else *reinterpret_cast<u32x4*>(dst + lane * 16) = u32x4{0, 0, 0, 0};
      from_a[i] += 256;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      char* dst = to + Tile::kABytes + (2 * wave + i) * 1024;
      if (chunk_w * 32 < left) copy_lds16(reinterpret_cast<uint64_t>(from_w[i]), lds_address(dst));
      else *reinterpret_cast<u32x4*>(dst + lane * 16) = u32x4{0, 0, 0, 0};
      from_w[i] += 64;
    }
  };

  // scales: two threads a row, two steps each
  const int scale_of = threadIdx.x >> 1, half = threadIdx.x & 1;
  const int32_t nblk = K / (kMx ? 32 : 16);
  const uint8_t* scale_row = static_cast<const uint8_t*>(p.w_scales) + w_row4(n0, scale_of, p.N, kOutN) * nblk;
  struct Scales {
    uint32_t d[kBlocks / 2];
  };
  auto load = [&](int ks) {
    Scales v;
    const int at = (step0 + ks + 2 * half) * kBlocks;
#pragma unroll
    for (int i = 0; i < kBlocks / 2; i += kBlocks / 4) load_scales4<kMx>(scale_row + min(at + 4 * i, nblk), nblk - at - 4 * i, v.d + i);
    return v;
  };
  auto store = [&](int buf, const Scales& v) {
#pragma unroll
    for (int i = 0; i < kBlocks / 2; ++i) *reinterpret_cast<uint32_t*>(&s_scale[buf][scale_of][half * 2 * kBlocks + 4 * i]) = v.d[i];
  };

  f32x4 acc[kFM][2];
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  // a wavefront's fragments of w: 32 consecutive rows, or 16 gate rows and their up rows
  auto w_first = [&](int j) { return kGated ? j * kOutN + wave * 16 : wave * 32 + j * 16; };

  Scales next;
  auto step = [&](auto tc, int ks) {
    constexpr int T = decltype(tc)::value;
    if (ks + kStages - 1 < steps) fetch(ks + kStages - 1);
    const char* stage = smem + ks % kStages * Tile::kStage;
    u32x4 w[2];
    uint32_t s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = w_first(j) + i16;
      w[j] = *reinterpret_cast<const u32x4*>(stage + Tile::kABytes + r * 64 + ((g ^ (r >> 1 & 3)) << 4));
      const uint8_t* sc = &s_scale[(ks >> 2) & 1][r][T * kBlocks];
      if constexpr (kMx) s[j] = sc[g];
      else s[j] = *reinterpret_cast<const uint16_t*>(sc + 2 * g);
    }
    auto part = [&](auto uc) {
      constexpr int u = decltype(uc)::value;
      u32x4 wt[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) wt[j] = weights8<kMx, kHalf, kMx ? 0 : u / 2>(w[j][u], s[j]);
#pragma unroll
      for (int i = 0; i < kFM; ++i) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(stage + (i * 16 + i16) * 256 + (((4 * g + u) ^ i16) << 4));
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], a, acc[i][j]);
      }
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
    part(std::integral_constant<int, 2>{});
    part(std::integral_constant<int, 3>{});
    // the next four steps' scales: loaded a step before they go to LDS, which is a step
    // before they are read
    if constexpr (T == 1) next = load(ks + 3);
    if constexpr (T == 2) store(1 - ((ks >> 2) & 1), next);
    if (ks + kStages - 1 < steps) step_barrier<(kStages - 2) * Tile::kLoads>();
    else step_barrier<0>();
  };
  store(0, load(0));
#pragma unroll
  for (int ks = 0; ks < kStages - 1; ++ks)
    if (ks < steps) fetch(ks);
  step_barrier<0>();
  for (int ks = 0;;) {
    step(std::integral_constant<int, 0>{}, ks);
    if (++ks == steps) break;
    step(std::integral_constant<int, 1>{}, ks);
    if (++ks == steps) break;
    step(std::integral_constant<int, 2>{}, ks);
    if (++ks == steps) break;
    step(std::integral_constant<int, 3>{}, ks);
    if (++ks == steps) break;
  }

  // a lane's four results are four consecutive columns of one row
  if (work.part >= 0) {
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<f32x4*>(p.partial + partial_at(work.tile - p.whole, work.part, p.parts, i * 16 + i16, w_first(j) + 4 * g, kBM,
                                                         kRowsW)) = acc[i][j];
    return;
  }
  constexpr int kLd = kRowsW + 4;
  static_assert(kBM * kLd * 4 <= kStages * Tile::kStage, "the tile fits the step buffers");
  float* tile = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<f32x4*>(tile + (i * 16 + i16) * kLd + w_first(j) + 4 * g) = acc[i][j];
  __syncthreads();
  constexpr int kPer = kOutN / 8;                              // threads per row
  const int c = (int)(threadIdx.x % kPer) * 8;
  const int32_t n = n0 + c;
  Columns<kKind, kGated, 8> cols;
  cols.load(p, n);
#pragma unroll 1
  for (int r = threadIdx.x / kPer; r < kBM; r += kThreads / kPer) {
    const int64_t m = m0 + r, mr = min(m, (int64_t)p.M - 1);
    const bool in = m < p.M && n < p.N;
    Residual<8> res;
    res.load(p, mr, n);
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = tile[r * kLd + c + e];
      u[e] = tile[r * kLd + c + e + (kGated ? kOutN : 0)];
    }
    cols.finish(p, mr, v, u);
    res.add(p, v);
    if (p.out_type != kOutBlock8) {
      if (in) store_run<8>(p, m, n, v);
    } else {
      store_block<8>(p, m, n, v, in);
    }
  }
}

// ---- many rows ------------------------------------------------------------------------
// w in 16 bits, dense rows of `copies` times K elements, the second copy (for the lower
// parts of a) without its infinities; a thread writes 32 elements.
template <bool kMx, bool kHalf>
__global__ __launch_bounds__(256) void widen4_kernel(const uint8_t* w, int64_t ldw, const uint8_t* scales, int64_t rows, int32_t K,
                                                     int32_t copies, uint16_t* out) {
  const int32_t vecs = K / 32;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= rows * vecs) return;
  const int64_t row = id / vecs;
  const int32_t v = (int32_t)(id - row * vecs);
  const u32x4 c = *reinterpret_cast<const u32x4*>(w + row * ldw + 16 * v);
  u32x4 d[4];
  if constexpr (kMx) {
    const uint32_t s = scales[row * vecs + v];
#pragma unroll
    for (int t = 0; t < 4; ++t) d[t] = weights8<true, kHalf, 0>(c[t], s);
  } else {
    const uint32_t s = *reinterpret_cast<const uint16_t*>(scales + 2 * (row * vecs + v));
    d[0] = weights8<false, kHalf, 0>(c[0], s);
    d[1] = weights8<false, kHalf, 0>(c[1], s);
    d[2] = weights8<false, kHalf, 1>(c[2], s);
    d[3] = weights8<false, kHalf, 1>(c[3], s);
  }
  for (int32_t i = 0; i < copies; ++i) {
    u32x4* dst = reinterpret_cast<u32x4*>(out + (row * copies + i) * K + 32 * v);
#pragma unroll
    for (int t = 0; t < 4; ++t) dst[t] = i ? finite_bf16(d[t]) : d[t];
  }
}

// fp16 rows as bf16 rows of twice the length, upper parts then lower parts.
__global__ __launch_bounds__(256) void split_rows_kernel(const uint16_t* a, int64_t lda, int64_t rows, int32_t K, uint16_t* out) {
  const int32_t vecs = K / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= rows * vecs) return;
  const int64_t row = id / vecs;
  const int32_t v = (int32_t)(id - row * vecs);
  u32x4 hi, lo;
  split_f16(*reinterpret_cast<const u32x4*>(a + row * lda + 8 * v), hi, lo);
  uint16_t* dst = out + row * 2 * K + 8 * v;
  *reinterpret_cast<u32x4*>(dst) = hi;
  *reinterpret_cast<u32x4*>(dst + K) = lo;
}

// ---- launches --------------------------------------------------------------------------
template <bool kMx, bool kHalf, int kRF, int kFN, bool kGated>
hipError_t go_few(LinParams p, hipStream_t stream) {
  const int32_t cols = kGated ? 8 * kFN : 16 * kFN;
  p.tiles_n = (p.N - 1) / cols + 1;
  const int32_t bands = (p.M - 1) / (16 * kRF) + 1;
  hipLaunchKernelGGL((linear4_few_kernel<kMx, kHalf, kRF, kFN, kGated>), dim3((uint32_t)bands * (uint32_t)p.tiles_n), dim3(512), 0, stream, p);
  return hipGetLastError();
}

template <bool kMx, bool kHalf, int kFM, int kWaves, bool kGated>
hipError_t go_tile(LinParams p, const Plan4& q, void* workspace, hipStream_t stream) {
  const int32_t out_n = kGated ? q.rows_w / 2 : q.rows_w;
  const int32_t left = q.tiles_m * q.tiles_n - q.whole;
  p.kbytes /= 2;                                               // elements
  p.tiles_m = q.tiles_m;
  p.tiles_n = q.tiles_n;
  p.whole = q.whole;
  p.parts = q.parts;
  p.part_steps = q.part_steps;
  p.partial = static_cast<float*>(workspace);
  hipLaunchKernelGGL((linear4_tile_kernel<kMx, kHalf, kFM, kWaves, kGated>), dim3((uint32_t)(q.whole + left * q.parts)), dim3(64 * kWaves), 0,
                     stream, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || left == 0) return err;
  hipLaunchKernelGGL((linear_join_kernel<kHalf ? (int)kF16 : (int)kBf16, kGated>), dim3((uint32_t)(((int64_t)left * q.bm * (out_n / 8) + 255) / 256)),
                     dim3(256), 0, stream, p, q.bm, q.rows_w);
  return hipGetLastError();
}

template <bool kMx, bool kHalf, bool kGated>
hipError_t go_rows(const LinParams& p, const Plan4& q, void* workspace, hipStream_t stream) {
  constexpr int kFirst = kGated ? 2 : 1;                       // fragments of w for 16 outputs
  const bool block = p.out_type == kOutBlock8;                 // (32 outputs belong together)
  if (q.form == Plan4::kFew) {
    if (p.M <= 16) return block ? go_few<kMx, kHalf, 1, 2 * kFirst, kGated>(p, stream) : go_few<kMx, kHalf, 1, kFirst, kGated>(p, stream);
    if constexpr (kMx && kHalf) {
      if (p.M <= 32) return go_few<kMx, kHalf, 2, 2 * kFirst, kGated>(p, stream);
      return go_few<kMx, kHalf, 4, 2 * kFirst, kGated>(p, stream);
    }
  }
  if constexpr (!(kMx && kHalf)) {
    if (q.fm == 1) return go_tile<kMx, kHalf, 1, 4, kGated>(p, q, workspace, stream);
    if (q.fm == 2) return go_tile<kMx, kHalf, 2, 4, kGated>(p, q, workspace, stream);
    if (q.fm == 4) return go_tile<kMx, kHalf, 4, 4, kGated>(p, q, workspace, stream);
    return go_tile<kMx, kHalf, 8, 8, kGated>(p, q, workspace, stream);
  }
  return hipErrorInvalidValue;
}

template <bool kMx, bool kHalf>
hipError_t go_gated(const LinParams& p, int32_t gated, const Plan4& q, void* workspace, hipStream_t stream) {
  return gated ? go_rows<kMx, kHalf, true>(p, q, workspace, stream) : go_rows<kMx, kHalf, false>(p, q, workspace, stream);
}

// What the many-row form multiplies: a and w in 16 bits.
struct Wide {
  LinearArgs a;
  size_t w_at, a_at, rest_at;                                  // in the workspace: w, a's parts, the product's own
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

Wide wide_of(const Linear4Args& a) {
  Wide q;
  q.a = a;
  const bool split = a.mx && a.kind == kF16;
  const size_t rows = a.gated ? 2 * (size_t)a.N : (size_t)a.N;
  q.a.kind = split ? kBf16 : a.kind;
  q.a.K = split ? 2 * a.K : a.K;
  q.a.ldw = q.a.K;
  if (split) q.a.lda = q.a.K;
  q.w_at = 0;
  q.a_at = up256(rows * q.a.K * 2);
  q.rest_at = q.a_at + (split ? up256((size_t)a.M * q.a.K * 2) : 0);
  return q;
}

}  // namespace

size_t linear4_workspace_bytes(const Linear4Args& a) {
  if (a.M == 0 || a.N == 0) return 0;
  const Plan4 plan = plan4_of(a.M, a.N, a.K, a.kind, a.mx, a.gated != 0);
  if (plan.form != Plan4::kWide) return plan.bytes;
  const Wide q = wide_of(a);
  return q.rest_at + linear_workspace_bytes(q.a);
}

hipError_t launch_linear4(const Linear4Args& a, void* workspace, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const bool f16 = a.kind == kF16;
  const Plan4 plan = plan4_of(a.M, a.N, a.K, a.kind, a.mx, a.gated != 0);
  if (plan.form != Plan4::kWide) {
    LinParams p = {};
    p.a = static_cast<const char*>(a.a);
    p.w = static_cast<const char*>(a.w);
    p.w_scales = a.w_scales;
    p.bias = a.bias;
    p.residual = a.residual;
    p.out = a.out;
    p.out_scales = a.out_scales;
    p.gain = a.gain;
    p.lda = a.lda * 2;
    p.ldw = a.ldw;
    p.ldr = a.ldr;
    p.ldo = a.ldo;
    p.M = a.M; p.N = a.N; p.kbytes = a.K * 2;
    p.act = a.act; p.bias_type = a.bias_type; p.residual_type = a.residual_type; p.out_type = a.out_type;
    if (a.mx)
      return f16 ? go_gated<true, true>(p, a.gated, plan, workspace, stream) : go_gated<true, false>(p, a.gated, plan, workspace, stream);
    return f16 ? go_gated<false, true>(p, a.gated, plan, workspace, stream) : go_gated<false, false>(p, a.gated, plan, workspace, stream);
  }
  Wide q = wide_of(a);
  char* ws = static_cast<char*>(workspace);
  const int64_t rows = a.gated ? 2 * (int64_t)a.N : a.N;
  const uint8_t* codes = static_cast<const uint8_t*>(a.w);
  const uint8_t* scales = static_cast<const uint8_t*>(a.w_scales);
  uint16_t* w16 = reinterpret_cast<uint16_t*>(ws + q.w_at);
  // (rows * K / 32 and M * K / 8 threads fit a launch: the entry point's limits)
  const dim3 grid((uint32_t)((rows * (a.K / 32) + 255) / 256));
  const int32_t copies = q.a.K / a.K;
  if (a.mx) hipLaunchKernelGGL((widen4_kernel<true, false>), grid, dim3(256), 0, stream, codes, a.ldw, scales, rows, a.K, copies, w16);
  else if (f16) hipLaunchKernelGGL((widen4_kernel<false, true>), grid, dim3(256), 0, stream, codes, a.ldw, scales, rows, a.K, copies, w16);
  else hipLaunchKernelGGL((widen4_kernel<false, false>), grid, dim3(256), 0, stream, codes, a.ldw, scales, rows, a.K, copies, w16);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  q.a.w = w16;
  q.a.w_scales = nullptr;
  if (copies == 2) {
    uint16_t* a16 = reinterpret_cast<uint16_t*>(ws + q.a_at);
    hipLaunchKernelGGL(split_rows_kernel, dim3((uint32_t)(((int64_t)a.M * (a.K / 8) + 255) / 256)), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(a.a), a.lda, (int64_t)a.M, a.K, a16);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    q.a.a = a16;
  }
  return launch_linear(q.a, ws + q.rest_at, stream);
}

}  // namespace nvfp4
