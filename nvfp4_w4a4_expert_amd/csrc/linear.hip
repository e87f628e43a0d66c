// Dense linear operator for gfx950:
//
//   v[m, n]   = sum_k a[m, k] * w[n, k]  (+ bias[n])            fp32 accumulation
//   out[m, n] = residual[m, n] + act(v[m, n])                   or, gated,
//   out[m, n] = residual[m, n] + act(v[m, n]) * v[m, N + n]     (w rows [0, N) gate, [N, 2N) up)
//
// on bf16, fp16 or E4M3 operands (fp32 scale per row of a and w, or UE8M0 scale
// per 32 elements), rounded once to bf16, fp16, fp32 or E4M3 with UE8M0 scales.
//
// Both operands are row-major along K, so a K step is 128 bytes of a row
// whatever the type: 64 elements of 16 bits (two 16x16x32 matrix instructions)
// or 128 of 8 bits (one 16x16x128 scaled instruction, which applies the
// power-of-two block scales itself; row scales are applied in the epilogue and
// the instruction then runs with unit scales).
//
// The scaled instruction adds its products in groups of eight and cuts each to a
// multiple of 2^-13 of the group's largest power of two (found by its results):
// sums of random data are off by about 1.5e-5 of their norm whatever K.  That is
// nothing beside the rounding of a 16-bit or 8-bit output, but a hundred times
// fp32's own error.  fp32 outputs of 8-bit operands therefore run on the bf16
// instruction: an E4M3 value times a power of two is a bf16 number, the products
// are exact and the sums are fp32 sums (the "wide" kinds, at half the rate).
#include <type_traits>

#include "fp8_device.h"
#include "internal.h"

namespace nvfp4 {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Operand kinds: 16-bit types, E4M3 with row or block scales, and the wide forms
// of the latter two.
enum { kBf16 = 0, kF16 = 1, kRow8 = 2, kBlock8 = 3, kRow8Wide = 4, kBlock8Wide = 5 };
constexpr bool is_row8(int kind) { return kind == kRow8 || kind == kRow8Wide; }
constexpr bool is_block8(int kind) { return kind == kBlock8 || kind == kBlock8Wide; }
constexpr bool is_wide(int kind) { return kind == kRow8Wide || kind == kBlock8Wide; }
enum { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutBlock8 = 3 };
enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4 };

constexpr int kStep = 128;                                     // bytes of K per step

struct LinParams {
  const char* a;
  const char* w;
  const void* a_scales;
  const void* w_scales;
  const void* bias;
  const void* residual;
  void* out;
  uint8_t* out_scales;
  int64_t lda, ldw, ldr, ldo;                                  // lda, ldw in bytes
  int32_t M, N, kbytes;
  int32_t act, bias_type, residual_type, out_type;
  int32_t tiles_m, tiles_n;
};

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int32_t type) {
  if (type == kOutF32) return static_cast<const float*>(p)[i];
  const uint16_t u = static_cast<const uint16_t*>(p)[i];
  return type == kOutF16 ? (float)__builtin_bit_cast(_Float16, u) : __uint_as_float((uint32_t)u << 16);
}

// erfc(x) by the Chebyshev fit t * exp(-x^2 + P(t)), t = 1 / (1 + |x| / 2), of
// Press et al., Numerical Recipes (the routine of fractional error below
// 1.2e-7 everywhere), so gelu keeps its relative accuracy where erfc is tiny.
__device__ __forceinline__ float erfc_fit(float x) {
  const float z = fabsf(x), t = 1.0f / (1.0f + 0.5f * z);
  float q = 0.17087277f;
  q = -0.82215223f + t * q;
  q = 1.48851587f + t * q;
  q = -1.13520398f + t * q;
  q = 0.27886807f + t * q;
  q = -0.18628806f + t * q;
  q = 0.09678418f + t * q;
  q = 0.37409196f + t * q;
  q = 1.00002368f + t * q;
  q = -1.26551223f + t * q;
  const float r = t * expf(-z * z + q);
  return x < 0.0f ? 2.0f - r : r;
}

// The activations over a run of values: silu and gelu's tanh form as v *
// sigmoid(z) (z = 2u for the latter: 1 + tanh u would cancel for negative u),
// gelu's erf form as v * erfc(-v / sqrt 2) / 2.
template <int kLen>
__device__ __forceinline__ void activate_run(float* v, int32_t act) {
  if (act == kActNone) return;
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < kLen; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];     // NaN stays NaN
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < kLen; ++i) v[i] = 0.5f * v[i] * erfc_fit(-0.70710678118654752f * v[i]);
  } else {
    const float c1 = act == kActSilu ? 1.0f : 1.5957691216057308f;       // 2 sqrt(2 / pi)
    const float c3 = act == kActSilu ? 0.0f : 0.071354816272600248f;     // 0.044715 c1
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      // c1 + c3 v^2 first: v^3 alone could overflow to inf * 0
      const float z = act == kActSilu ? v[i] : v[i] * (c1 + c3 * (v[i] * v[i]));
      const float e = expf(-fabsf(z));                                   // never overflows
      v[i] = v[i] * (z < 0.0f ? e : 1.0f) / (1.0f + e);
    }
  }
}

// kLen consecutive elements of a tensor of type bf16, fp16 or fp32 from element
// `at` on, the first `have` of them inside the row; wide loads where the address
// allows them.
template <int kLen>
__device__ __forceinline__ void load_run(const void* base, int64_t at, int32_t type, int have, float* v) {
  const char* src = static_cast<const char*>(base) + at * (type == kOutF32 ? 4 : 2);
  if (have >= kLen && (reinterpret_cast<uintptr_t>(src) & 7) == 0) {
    if (type == kOutF32) {
#pragma unroll
      for (int i = 0; i < kLen; i += 2) {
        const float2 d = *reinterpret_cast<const float2*>(src + 4 * i);
        v[i] = d.x;
        v[i + 1] = d.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLen; i += 4) {
        const uint2 d = *reinterpret_cast<const uint2*>(src + 2 * i);
        const uint32_t u[4] = {d.x & 0xFFFFu, d.x >> 16, d.y & 0xFFFFu, d.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i + j] = type == kOutF16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)u[j]) : __uint_as_float(u[j] << 16);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLen; ++i) v[i] = i < have ? load_elem(base, at + i, type) : 0.0f;
  }
}

// The terms of kLen output columns that do not depend on the row: bias, and the
// row scales of w (E4M3 operands with row scales).
template <int kKind, bool kGated, int kLen>
struct Columns {
  float b[kLen], bu[kGated ? kLen : 1];
  float s[is_row8(kKind) ? kLen : 1], su[is_row8(kKind) && kGated ? kLen : 1];

  __device__ __forceinline__ void load(const LinParams& p, int32_t n) {
    const int have = p.N - n;
#pragma unroll
    for (int i = 0; i < kLen; ++i) b[i] = 0.0f;
    if constexpr (kGated) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) bu[i] = 0.0f;
    }
    if (p.bias) {
      load_run<kLen>(p.bias, n, p.bias_type, have, b);
      if constexpr (kGated) load_run<kLen>(p.bias, (int64_t)p.N + n, p.bias_type, have, bu);
    }
    if constexpr (is_row8(kKind)) {
      load_run<kLen>(p.w_scales, n, kOutF32, have, s);
      if constexpr (kGated) load_run<kLen>(p.w_scales, (int64_t)p.N + n, kOutF32, have, su);
    }
  }

  // `gate` (and `up`): the sums of row m; the outputs, before the residual and
  // before rounding, replace `gate`.
  __device__ __forceinline__ void finish(const LinParams& p, int64_t m, float* gate, const float* up) const {
    float am = 1.0f;
    if constexpr (is_row8(kKind)) am = static_cast<const float*>(p.a_scales)[m];
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      if constexpr (is_row8(kKind)) gate[i] *= am * s[i];
      gate[i] += b[i];
    }
    activate_run<kLen>(gate, p.act);
    if constexpr (kGated) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) {
        float u = up[i];
        if constexpr (is_row8(kKind)) u *= am * su[i];
        gate[i] *= u + bu[i];
      }
    }
  }
};

template <int kLen>
__device__ __forceinline__ void add_residual(const LinParams& p, int64_t m, int32_t n, float* v) {
  if (!p.residual) return;
  float r[kLen];
  load_run<kLen>(p.residual, m * p.ldr + n, p.residual_type, p.N - n, r);
#pragma unroll
  for (int i = 0; i < kLen; ++i) v[i] += r[i];
}

// kLen consecutive outputs of row m from column n on, each rounded once; wide
// stores where the row's alignment and the tensor's edge allow them.
template <int kLen>
__device__ __forceinline__ void store_run(const LinParams& p, int64_t m, int32_t n, const float* v) {
  const int64_t at = m * p.ldo + n;
  const int have = p.N - n;
  if (p.out_type == kOutF32) {
    float* dst = static_cast<float*>(p.out) + at;
    if (have >= kLen && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < kLen; i += 4) *reinterpret_cast<f32x4*>(dst + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < kLen; ++i)
        if (i < have) dst[i] = v[i];
    }
    return;
  }
  uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
  uint32_t d[kLen / 2];
#pragma unroll
  for (int i = 0; i < kLen / 2; ++i)
    d[i] = p.out_type == kOutF16 ? pack_f16(v[2 * i], v[2 * i + 1]) : pack_bf16(v[2 * i], v[2 * i + 1]);
  if (have >= kLen && (reinterpret_cast<uintptr_t>(dst) & (kLen >= 8 ? 15 : 7)) == 0) {
    if constexpr (kLen >= 8) {
#pragma unroll
      for (int i = 0; i < kLen / 2; i += 4) *reinterpret_cast<u32x4*>(dst + 2 * i) = u32x4{d[i], d[i + 1], d[i + 2], d[i + 3]};
    } else {
      *reinterpret_cast<uint2*>(dst) = uint2{d[0], d[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLen; ++i)
      if (i < have) dst[i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
  }
}

// kLen consecutive outputs as E4M3 codes; 32 / kLen neighbouring lanes hold a block
// of 32 columns (N is a multiple of 32: a block is stored whole or not at all)
// and agree on its scale.
template <int kLen>
__device__ __forceinline__ void store_block(const LinParams& p, int64_t m, int32_t n, const float* v, bool in) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLen; ++i) top = max(top, finite_mag(v[i]));
#pragma unroll
  for (int off = 1; off < 32 / kLen; off *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  float inv;
  const uint32_t code = block_scale_code(top, inv);
  if (!in) return;
  uint8_t* dst = static_cast<uint8_t*>(p.out) + m * p.ldo + n;
#pragma unroll
  for (int i = 0; i < kLen; i += 4) *reinterpret_cast<uint32_t*>(dst + i) = encode4_e4m3(v + i, inv);
  if (n % 32 == 0) p.out_scales[m * (p.N / 32) + n / 32] = (uint8_t)code;
}

// Workgroup barrier that orders LDS accesses only: stores to memory need not
// have completed, as a full __syncthreads() would demand.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A lane's share of a K step of one row of 16: the 16-byte chunks g and 4 + g of
// the 128 bytes, g its group of 16 lanes.  That is the K order of the
// 16x16x128 instruction, whose lane group g also supplies the scale of the
// step's g-th block of 32; the 16x16x32 instructions take one chunk (wide kinds:
// half a chunk) each, in any K order that both operands share.
struct Frag {
  u32x4 c[2];
};

// 8 E4M3 codes times a power of two, as bf16 (exact).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi, float scale) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// An operand's share as the instruction takes it.  Block scales: a row's UE8M0
// codes of four steps lie in one word per block of a step, step t in byte t; a
// lane holds the word of the g-th block, or (wide kinds) those of the blocks of
// chunks g and 4 + g.
constexpr uint32_t kUnit = 0x7F7F7F7Fu;                           // scale 1 in every byte

template <int kKind, int kByte>
struct Prepared {
  Frag f;
  uint32_t scale;
  __device__ __forceinline__ void set(const Frag& v, const uint32_t* s) { f = v; scale = s[0]; }
};
template <int kByte>
struct PreparedWide {
  bf16x8_t v[4];
  __device__ __forceinline__ void set(const Frag& f, const uint32_t* s) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // 2^(code - 127), code in [1, 254]
      const float scale = __uint_as_float(((s[c] >> (8 * kByte)) & 0xFFu) << 23);
      v[2 * c] = widen8(f.c[c].x, f.c[c].y, scale);
      v[2 * c + 1] = widen8(f.c[c].z, f.c[c].w, scale);
    }
  }
};
template <int kByte>
struct Prepared<kRow8Wide, kByte> : PreparedWide<kByte> {};
template <int kByte>
struct Prepared<kBlock8Wide, kByte> : PreparedWide<kByte> {};

// acc += w . a over a K step; w is the row operand, so a lane's four results are
// four consecutive output columns (instruction rows 4g .. 4g + 3) of one row of a.
template <int kKind, int kByte>
__device__ __forceinline__ f32x4 mma(const Prepared<kKind, kByte>& w, const Prepared<kKind, kByte>& a, f32x4 acc) {
  if constexpr (is_wide(kKind)) {
#pragma unroll
    for (int t = 0; t < 4; ++t) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[t], a.v[t], acc, 0, 0, 0);
  } else if constexpr (kKind == kBf16) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w.f.c[t]),
                                                    __builtin_bit_cast(bf16x8_t, a.f.c[t]), acc, 0, 0, 0);
  } else if constexpr (kKind == kF16) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w.f.c[t]),
                                                   __builtin_bit_cast(half8_t, a.f.c[t]), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8_t, w.f), __builtin_bit_cast(i32x8_t, a.f),
                                                           acc, 0, 0, kByte, (int)w.scale, kByte, (int)a.scale);
  }
  return acc;
}

// 16 scales of a row, of the four steps from block `at` on (past the end of the
// row the data are zeros: any scale does) ...
__device__ __forceinline__ u32x4 load_scales(const uint8_t* row, int at, int nblk) {
  u32x4 d;
  if (at + 16 <= nblk) {
    __builtin_memcpy(&d, row + at, 16);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t w = 0;
#pragma unroll 1                                                  // (once per tile: few registers matter more)
      for (int b = 0; b < 4; ++b) w = (w >> 8) | ((at + 4 * t + b < nblk ? (uint32_t)row[at + 4 * t + b] : 127u) << 24);
      d[t] = w;
    }
  }
  return d;
}

// ... and as four words, one per block of a step (byte t: step t): 4 x 4 bytes
// transposed.
__device__ __forceinline__ u32x4 scale_words(const u32x4& d) {
  const uint32_t lo01 = __builtin_amdgcn_perm(d.y, d.x, 0x05010400u), hi01 = __builtin_amdgcn_perm(d.y, d.x, 0x07030602u);
  const uint32_t lo23 = __builtin_amdgcn_perm(d.w, d.z, 0x05010400u), hi23 = __builtin_amdgcn_perm(d.w, d.z, 0x07030602u);
  return u32x4{__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
               __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
}

// A lane's share from a 128-byte row segment in LDS whose chunk c lies at
// position c ^ (row & 7): eight consecutive rows then start on distinct groups
// of four banks.
__device__ __forceinline__ Frag read_frag(const char* tile, int row, int g) {
  const char* r = tile + row * kStep;
  Frag f;
  f.c[0] = *reinterpret_cast<const u32x4*>(r + ((g ^ (row & 7)) << 4));
  f.c[1] = *reinterpret_cast<const u32x4*>(r + (((4 + g) ^ (row & 7)) << 4));
  return f;
}

__device__ __forceinline__ void load_lds16(const char* src, char* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// Barrier at the turn of a step: this wavefront's copies into LDS have arrived
// and its LDS reads are done before any wavefront passes.  The wait is written
// out because the copies are counted with memory loads, whose completion a
// workgroup barrier by itself does not ask for.
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  lds_barrier();
}

// ---- tiled kernel -------------------------------------------------------------
// A workgroup of kWM x kWN wavefronts owns kBM rows of a and kBN rows of w
// (gated: kBN / 2 output columns, their gate rows, then their up rows).  Each K
// step's rows are copied straight into LDS (two buffers).  The epilogue passes
// the sums through LDS, 32 rows of each wavefront at a time, so that every thread
// finishes 8 consecutive outputs of a row and whole rows are stored.
template <int kKind, int kBM, int kBN, int kWM, int kWN, bool kGated>
__global__ __launch_bounds__(64 * kWM * kWN, 2) void linear_tile_kernel(const LinParams p) {
  constexpr int kWaves = kWM * kWN;
  constexpr int kTM = kBM / kWM, kTN = kBN / kWN;
  constexpr int kFM = kTM / 16, kFN = kTN / 16;
  constexpr int kOutN = kGated ? kBN / 2 : kBN;                // output columns of the tile
  constexpr int kStage = (kBM + kBN) * kStep;
  constexpr int kLoads = (kBM + kBN) / 8 / kWaves;             // 1 KiB copies per wavefront and step
  static_assert((kBM + kBN) / 8 % kWaves == 0 && kBM / 8 % kLoads == 0, "whole copies; a wavefront copies one operand");
  static_assert(!kGated || kOutN % (8 * kLoads) == 0 || 8 * kLoads == kBN, "copies by gate and up rows");
  constexpr bool kScaled = is_block8(kKind);
  static_assert(kBM + kBN == 64 * kWaves || !kScaled, "a thread loads the scales of one row");
  __shared__ __align__(1024) char smem[2 * kStage];
  __shared__ __align__(16) uint32_t s_scale[kScaled ? 2 : 1][kScaled ? kBM + kBN : 1][4];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int wm = wave / kWN, wn = wave % kWN;

  // tiles: each of the 8 XCDs gets a contiguous range of them (workgroups are
  // dealt to the XCDs in turn), walked in groups of 8 tile rows
  int32_t tm, tn;
  {
    const int32_t total = p.tiles_m * p.tiles_n;
    const int32_t per = total / 8, rest = total % 8;
    const int32_t xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const int32_t t = xcd * per + (xcd < rest ? xcd : rest) + at;
    constexpr int32_t kGroup = 8;
    const int32_t band = t / (kGroup * p.tiles_n);
    const int32_t rows = min(kGroup, p.tiles_m - band * kGroup);
    const int32_t in = t - band * kGroup * p.tiles_n;
    tm = band * kGroup + in % rows;
    tn = in / rows;
  }
  const int64_t m0 = (int64_t)tm * kBM;
  const int32_t n0 = tn * kOutN;

  // source of each copy: lane -> (row of the operand's tile, chunk).  Rows past the
  // edge repeat the last row, their results are not stored.  The offset from the
  // tile's first row is formed at each copy (three instructions): kept for all
  // copies, it would cost the registers that the fragments need.
  constexpr int kHalves = kGated && 8 * kLoads > kOutN ? 2 : 1;  // a wavefront's copies hold gate and up rows
  uint64_t base[kHalves];                                      // uniform: the operand's tile at this step
  const int chunk = (lane & 7) ^ (lane >> 3);                  // (row & 7) == lane >> 3
  const int first = wave * kLoads * 8;                         // the wavefront's first row of the tile
  const bool is_a = first < kBM;
  int row0 = (is_a ? first : (first - kBM) % kOutN) + (lane >> 3);
  const int last_row = is_a ? (int)min((int64_t)kBM, p.M - m0) - 1 : min(kOutN, p.N - n0) - 1;
  const uint32_t ld = (uint32_t)(is_a ? p.lda : p.ldw);
  {
    const int64_t up = kGated && !is_a ? (first - kBM) / kOutN * (int64_t)p.N : 0;
    base[0] = reinterpret_cast<uint64_t>(is_a ? p.a + m0 * p.lda : p.w + (n0 + up) * p.ldw);
    if (kHalves == 2) base[kHalves - 1] = is_a ? base[0] : reinterpret_cast<uint64_t>(p.w + ((int64_t)n0 + p.N) * p.ldw);
  }
  const int steps = (p.kbytes + kStep - 1) / kStep;
  const int tail = p.kbytes - (steps - 1) * kStep;             // bytes of the last step
  auto fetch = [&](int ks) {
    char* dst = smem + (ks & 1) * kStage + wave * kLoads * 1024;
    if (chunk * 16 < (ks == steps - 1 ? tail : kStep)) {
      asm volatile("" : "+v"(row0));                           // (formed here, not carried along)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int add = kHalves == 2 && !is_a ? 8 * i % kOutN : 8 * i;
        const uint32_t off = (uint32_t)min(row0 + add, last_row) * ld + chunk * 16;
        load_lds16(reinterpret_cast<const char*>(base[kHalves == 2 ? 8 * i / kOutN : 0]) + off, dst + i * 1024);
      }
    } else {                                                   // past the end of the rows
#pragma unroll
      for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(dst + i * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
      base[i] += kStep;
      asm volatile("" : "+s"(base[i]));
    }
  };

  f32x4 acc[kFN][kFM];
#pragma unroll
  for (int j = 0; j < kFN; ++j)
#pragma unroll
    for (int i = 0; i < kFM; ++i) acc[j][i] = f32x4{0, 0, 0, 0};

  // block scales: every thread loads those of one row of the tile, four steps at
  // a time, and leaves them in LDS
  const int32_t nblk = p.kbytes / 32;
  const uint8_t* scale_row = nullptr;
  u32x4 scale_next;
  if constexpr (kScaled) {
    const int r = threadIdx.x;
    if (r < kBM) {
      scale_row = static_cast<const uint8_t*>(p.a_scales) + min(m0 + r, (int64_t)p.M - 1) * nblk;
    } else {
      const int q = r - kBM;
      scale_row = static_cast<const uint8_t*>(p.w_scales) +
                  ((int64_t)min(n0 + q % kOutN, p.N - 1) + (q >= kOutN ? p.N : 0)) * nblk;
    }
  }

  // Main loop.  A step runs its groups of instructions (one 16-row fragment of a
  // with all of w) in order, the fragments of a being read two groups ahead; the
  // last two groups run fragment of w by fragment of w.  The barrier falls before
  // them: behind it the buffer that the step has read is refilled for the step
  // after next, and each fragment of w is replaced by the next step's as soon as
  // its last instruction is issued, so the matrix unit does not wait for LDS at
  // the turn of a step.  The scheduling barriers keep the compiler from moving
  // the reads back to their uses.  T: the step's number modulo 4 (2 without block
  // scales), for the byte of the scales and the slots of fa when a step has only
  // two groups.
  static_assert(kFM == 2 || kFM % 4 == 0, "fragment slots");
  constexpr int kAhead = kFM == 8 && kKind >= kRow8 ? 1 : 2;   // 8-bit fragments: one group, for want of registers
  constexpr int kWords = kKind == kBlock8Wide ? 2 : 1;         // scale words of a lane and row
  Frag fa[4], fw[kFN];
  uint32_t va[kFM][2], vw[kFN][2];
#pragma unroll
  for (int i = 0; i < kFM; ++i) va[i][0] = va[i][1] = kUnit;
#pragma unroll
  for (int j = 0; j < kFN; ++j) vw[j][0] = vw[j][1] = kUnit;
  auto read_scales = [&](int buf) {
#pragma unroll
    for (int c = 0; c < kWords; ++c) {
      const int word = kKind == kBlock8Wide ? 2 * c + g / 2 : g;
#pragma unroll
      for (int i = 0; i < kFM; ++i) va[i][c] = s_scale[kScaled ? buf : 0][kScaled ? wm * kTM + i * 16 + i16 : 0][word];
#pragma unroll
      for (int j = 0; j < kFN; ++j) vw[j][c] = s_scale[kScaled ? buf : 0][kScaled ? kBM + wn * kTN + j * 16 + i16 : 0][word];
    }
  };
  auto step = [&](auto t, int ks) {
    constexpr int T = decltype(t)::value;
    constexpr int kBase = kFM == 2 ? 2 * (T & 1) : 0;          // slot of group 0
    constexpr int kNext = kFM == 2 ? 2 - 2 * (T & 1) : 0;      // slot of the next step's group 0
    typedef Prepared<kKind, T> Op;
    const char* ta = smem + (ks & 1) * kStage + wm * kTM * kStep;
    const char* na = smem + (1 - (ks & 1)) * kStage + wm * kTM * kStep;
    const char* nw = smem + (1 - (ks & 1)) * kStage + (kBM + wn * kTN) * kStep;
    if constexpr (kScaled && T == 0) read_scales((ks >> 2) & 1);
    Op pw[kFN];
#pragma unroll
    for (int j = 0; j < kFN; ++j) pw[j].set(fw[j], vw[j]);
#pragma unroll
    for (int i = 0; i < kFM - 2; ++i) {
      if (kAhead == 1) fa[(kBase + i + 1) & 3] = read_frag(ta, (i + 1) * 16 + i16, g);
      if (kAhead == 2 || i == kFM - 3) fa[(kBase + i + 2) & 3] = read_frag(ta, (i + 2) * 16 + i16, g);
      __builtin_amdgcn_sched_barrier(0);
      Op pa;
      pa.set(fa[(kBase + i) & 3], va[i]);
#pragma unroll
      for (int j = 0; j < kFN; ++j) acc[j][i] = mma<kKind, T>(pw[j], pa, acc[j][i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kScaled) {
      // the next four steps' scales: loaded a step before they go to LDS, which
      // is a step before they are read
      if constexpr (T == 1) scale_next = load_scales(scale_row, 4 * (ks + 3), nblk);
      if constexpr (T == 2) *reinterpret_cast<u32x4*>(s_scale[1 - ((ks >> 2) & 1)][threadIdx.x]) = scale_words(scale_next);
    }
    step_barrier();                                            // this buffer is read, the other one filled
    if (ks + 2 < steps) fetch(ks + 2);
    Op pa[2];
    pa[0].set(fa[(kBase + kFM - 2) & 3], va[kFM - 2]);
    pa[1].set(fa[(kBase + kFM - 1) & 3], va[kFM - 1]);
    // (after the last step these read an older one, unused)
    fa[kNext] = read_frag(na, i16, g);
    if (kAhead == 2) fa[kNext + 1] = read_frag(na, 16 + i16, g);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[j][kFM - 2 + i] = mma<kKind, T>(pw[j], pa[i], acc[j][kFM - 2 + i]);
      fw[j] = read_frag(nw, j * 16 + i16, g);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  fetch(0);
  if (steps > 1) fetch(1);
  if constexpr (kScaled) *reinterpret_cast<u32x4*>(s_scale[0][threadIdx.x]) = scale_words(load_scales(scale_row, 0, nblk));
  step_barrier();
#pragma unroll
  for (int j = 0; j < kFN; ++j) fw[j] = read_frag(smem + (kBM + wn * kTN) * kStep, j * 16 + i16, g);
  fa[0] = read_frag(smem + wm * kTM * kStep, i16, g);
  if (kAhead == 2) fa[1] = read_frag(smem + wm * kTM * kStep, 16 + i16, g);
  for (int ks = 0;;) {
    step(std::integral_constant<int, 0>{}, ks);
    if (++ks == steps) break;
    step(std::integral_constant<int, 1>{}, ks);
    if (++ks == steps) break;
    if constexpr (kScaled) {
      step(std::integral_constant<int, 2>{}, ks);
      if (++ks == steps) break;
      step(std::integral_constant<int, 3>{}, ks);
      if (++ks == steps) break;
    }
  }

  // Epilogue: groups 2 * pass and 2 * pass + 1 of every wavefront through LDS.
  constexpr int kLd = kBN + 4;                                 // floats per row: 8 rows start on distinct banks
  constexpr int kRows = 32 * kWM;
  constexpr int kPer = kOutN / 8;                              // threads per row
  static_assert(kRows * kLd * 4 <= 2 * kStage, "the pass fits the step buffers");
  float* tile = reinterpret_cast<float*>(smem);
  const int c = (int)(threadIdx.x % kPer) * 8;
  const int32_t n = n0 + c;
  Columns<kKind, kGated, 8> cols;
  cols.load(p, n);
#pragma unroll 1
  for (int pass = 0; pass < kFM / 2; ++pass) {
    lds_barrier();                                             // the steps' (or the last pass's) reads are done
    float* dst = tile + (wm * 32 + i16) * kLd + wn * kTN + 4 * g;
#pragma unroll
    for (int q = 0; q < kFM / 2; ++q)
      if (q == pass) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < kFN; ++j) *reinterpret_cast<f32x4*>(dst + i * 16 * kLd + j * 16) = acc[j][2 * q + i];
      }
    lds_barrier();
#pragma unroll 1
    for (int r = (int)threadIdx.x / kPer; r < kRows; r += 64 * kWaves / kPer) {
      const int64_t m = m0 + (r / 32) * kTM + pass * 32 + r % 32;
      const bool in = m < p.M && n < p.N;
      const int64_t mr = m < p.M ? m : (int64_t)p.M - 1;
      float v[8], u[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(tile + r * kLd + c + 4 * h);
        const f32x4 y = *reinterpret_cast<const f32x4*>(tile + r * kLd + c + 4 * h + (kGated ? kOutN : 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * h + e] = x[e];
          u[4 * h + e] = y[e];
        }
      }
      cols.finish(p, mr, v, u);
      add_residual<8>(p, mr, n, v);
      if (p.out_type != kOutBlock8) {
        if (in) store_run<8>(p, m, n, v);
      } else {
        store_block<8>(p, m, n, v, in);
      }
    }
  }
}

// ---- few rows -------------------------------------------------------------------
// At most 16 * kFM rows of a: bound by reading w once, so w goes straight from
// memory to registers.  A workgroup owns kCols output columns (gated: their gate
// and up rows); its wavefronts take the K steps in turn and their partial sums
// are added in wavefront order through LDS.
template <int kKind, int kFM, int kCols, int kWaves, bool kGated>
__global__ __launch_bounds__(64 * kWaves) void linear_few_kernel(const LinParams p) {
  constexpr int kRows = kGated ? 2 * kCols : kCols;            // rows of w
  constexpr int kFN = kRows / 16;
  constexpr int kLd = kRows + 4;                               // floats per row of a partial tile
  __shared__ __align__(16) float part[kWaves][16 * kFM][kLd];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int32_t n0 = (int32_t)blockIdx.x * kCols;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * kFM);
  const int32_t nblk = p.kbytes / 32;

  const char* pw[kFN];
  const char* pa[kFM];
  const uint8_t* sw[kFN];
  const uint8_t* sa[kFM];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    const int r = j * 16 + i16;
    int32_t n = n0 + r % kCols;
    n = n < p.N ? n : p.N - 1;
    const int64_t row = (int64_t)n + (r >= kCols ? p.N : 0);
    pw[j] = p.w + row * p.ldw;
    sw[j] = static_cast<const uint8_t*>(p.w_scales) + row * nblk;
  }
#pragma unroll
  for (int i = 0; i < kFM; ++i) {
    const int64_t m = m0 + i * 16 + i16;
    const int64_t row = m < p.M ? m : (int64_t)p.M - 1;
    pa[i] = p.a + row * p.lda;
    sa[i] = static_cast<const uint8_t*>(p.a_scales) + row * nblk;
  }
  f32x4 acc[kFN][kFM];
#pragma unroll
  for (int j = 0; j < kFN; ++j)
#pragma unroll
    for (int i = 0; i < kFM; ++i) acc[j][i] = f32x4{0, 0, 0, 0};

  const int steps = (p.kbytes + kStep - 1) / kStep;
  for (int ks = wave; ks < steps; ks += kWaves) {
    // a chunk past the end of the rows counts as zeros
    Frag fw[kFN], fa[kFM];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int at = ks * kStep + (4 * c + g) * 16;
      const bool in = at < p.kbytes;
#pragma unroll
      for (int j = 0; j < kFN; ++j) {
        fw[j].c[c] = u32x4{0, 0, 0, 0};
        if (in) fw[j].c[c] = *reinterpret_cast<const u32x4*>(pw[j] + at);
      }
#pragma unroll
      for (int i = 0; i < kFM; ++i) {
        fa[i].c[c] = u32x4{0, 0, 0, 0};
        if (in) fa[i].c[c] = *reinterpret_cast<const u32x4*>(pa[i] + at);
      }
    }
    // this step's scales of the blocks of chunks g and 4 + g (past the end the
    // data are zeros: any scale does)
    auto scales = [&](const uint8_t* row, uint32_t* d) {
      d[0] = d[1] = kUnit;
      if constexpr (is_block8(kKind)) {
        d[0] = row[min(4 * ks + g / 2, nblk - 1)];
        d[1] = row[min(4 * ks + 2 + g / 2, nblk - 1)];
      }
    };
    Prepared<kKind, 0> qw[kFN], qa[kFM];
    uint32_t sc[2];
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      scales(sw[j], sc);
      qw[j].set(fw[j], sc);
    }
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      scales(sa[i], sc);
      qa[i].set(fa[i], sc);
    }
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int i = 0; i < kFM; ++i) acc[j][i] = mma<kKind, 0>(qw[j], qa[i], acc[j][i]);
  }
#pragma unroll
  for (int j = 0; j < kFN; ++j)
#pragma unroll
    for (int i = 0; i < kFM; ++i)
      *reinterpret_cast<f32x4*>(&part[wave][i * 16 + i16][j * 16 + 4 * g]) = acc[j][i];
  __syncthreads();

  // four outputs per thread: consecutive threads hold consecutive columns, so a
  // block of 32 columns is 8 neighbouring lanes
  constexpr int kQuads = kCols / 4;
  for (int e = threadIdx.x; e < 16 * kFM * kQuads; e += 64 * kWaves) {
    const int r = e / kQuads, c = (e % kQuads) * 4;
    f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      v += *reinterpret_cast<const f32x4*>(&part[w][r][c]);
      if constexpr (kGated) u += *reinterpret_cast<const f32x4*>(&part[w][r][kCols + c]);
    }
    const int64_t m = m0 + r;
    const int32_t n = n0 + c;
    const bool in = m < p.M && n < p.N;
    float gv[4] = {v.x, v.y, v.z, v.w}, uv[4] = {u.x, u.y, u.z, u.w};
    const int64_t mr = m < p.M ? m : (int64_t)p.M - 1;
    Columns<kKind, kGated, 4> cols;
    cols.load(p, n);
    cols.finish(p, mr, gv, uv);
    add_residual<4>(p, mr, n, gv);
    if (p.out_type != kOutBlock8) {
      if (in) store_run<4>(p, m, n, gv);
    } else if constexpr (kCols % 32 == 0) {
      store_block<4>(p, m, n, gv, in);
    }
  }
}

template <int kKind, int kBM, int kBN, int kWM, int kWN, bool kGated>
hipError_t go_tile(LinParams p, hipStream_t stream) {
  p.tiles_m = (p.M + kBM - 1) / kBM;
  constexpr int kOutN = kGated ? kBN / 2 : kBN;
  p.tiles_n = (p.N + kOutN - 1) / kOutN;
  hipLaunchKernelGGL((linear_tile_kernel<kKind, kBM, kBN, kWM, kWN, kGated>), dim3((uint32_t)(p.tiles_m * p.tiles_n)),
                     dim3(64 * kWM * kWN), 0, stream, p);
  return hipGetLastError();
}

template <int kKind, int kFM, int kCols, bool kGated>
hipError_t go_few(LinParams p, hipStream_t stream) {
  constexpr int kWaves = 8;
  hipLaunchKernelGGL((linear_few_kernel<kKind, kFM, kCols, kWaves, kGated>),
                     dim3((uint32_t)((p.N + kCols - 1) / kCols), (uint32_t)((p.M + 16 * kFM - 1) / (16 * kFM))),
                     dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError();
}

template <int kKind, bool kGated>
hipError_t go(const LinParams& p, hipStream_t stream) {
  if (p.M <= 64) {
    // bound by reading w: 8-bit operands take the exact instruction whatever the output
    constexpr int kFew = kKind == kRow8 ? kRow8Wide : kKind == kBlock8 ? kBlock8Wide : kKind;
    if constexpr (kFew == kKind) {
      if (p.M <= 16) return p.out_type == kOutBlock8 ? go_few<kKind, 1, 32, kGated>(p, stream) : go_few<kKind, 1, 16, kGated>(p, stream);
      return p.out_type == kOutBlock8 ? go_few<kKind, 2, 32, kGated>(p, stream) : go_few<kKind, 2, 16, kGated>(p, stream);
    } else {
      return go<kFew, kGated>(p, stream);
    }
  }
  if constexpr (kKind == kRow8 || kKind == kBlock8)
    if (p.out_type == kOutF32 || p.out_type == kOutBlock8) return go<kKind == kRow8 ? kRow8Wide : kBlock8Wide, kGated>(p, stream);
  const int64_t cols = kGated ? 2 * (int64_t)p.N : p.N;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p.M + bm - 1) / bm) * ((cols + bn - 1) / bn); };
  if constexpr (!is_wide(kKind))
    if (tiles(256, 256) >= 192) return go_tile<kKind, 256, 256, 2, 4, kGated>(p, stream);
  if (tiles(128, 128) >= 192) return go_tile<kKind, 128, 128, 2, 2, kGated>(p, stream);
  return go_tile<kKind, 64, 64, 2, 1, kGated>(p, stream);
}

template <int kKind>
hipError_t go_gated(const LinParams& p, int32_t gated, hipStream_t stream) {
  return gated ? go<kKind, true>(p, stream) : go<kKind, false>(p, stream);
}

}  // namespace

size_t linear_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_linear(const LinearArgs& a, void*, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int32_t esz = a.kind <= kF16 ? 2 : 1;
  LinParams p;
  p.a = static_cast<const char*>(a.a);
  p.w = static_cast<const char*>(a.w);
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.out_scales = a.out_scales;
  p.lda = a.lda * esz;
  p.ldw = a.ldw * esz;
  p.ldr = a.ldr;
  p.ldo = a.ldo;
  p.M = a.M; p.N = a.N; p.kbytes = a.K * esz;
  p.act = a.act; p.bias_type = a.bias_type; p.residual_type = a.residual_type; p.out_type = a.out_type;
  switch (a.kind) {
    case kBf16: return go_gated<kBf16>(p, a.gated, stream);
    case kF16: return go_gated<kF16>(p, a.gated, stream);
    case kRow8: return go_gated<kRow8>(p, a.gated, stream);
    case kBlock8: return go_gated<kBlock8>(p, a.gated, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nvfp4
