// The kernels of the dense linear operator (linear.hip) and of the products grouped by
// expert (grouped.hip), for gfx950.
#pragma once

#include <type_traits>

#include "fp8_device.h"
#include "linear_map.h"

namespace nvfp4 {
namespace {

using namespace linear_map;

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4 };

struct LinParams {
  const char* a;
  const char* w;
  const void* a_scales;
  const void* w_scales;
  const void* bias;
  const void* residual;
  void* out;
  uint8_t* out_scales;
  const float* gain;        // 16-bit kinds: a number that multiplies the sums, or null
  int64_t lda, ldw, ldr, ldo;                                  // lda, ldw in bytes
  int32_t M, N, kbytes;
  int32_t act, bias_type, residual_type, out_type;
  int32_t tiles_m, tiles_n;
  // tiles whole .. tiles_m * tiles_n - 1 are computed in `parts` parts of part_steps
  // K steps, whose sums go to partial[tile - whole][part][rows][columns]
  int32_t whole, parts, part_steps;
  float* partial;
};

// Rows grouped by expert (grouped.hip): expert e owns the rows offsets[e] ..
// offsets[e + 1] of the result and its own w, scales of w and bias.
struct GroupParams : LinParams {
  const int32_t* offsets;   // [experts + 1]
  const int32_t* index;     // or null; row m of the result multiplies row index[m] / index_div of a
  int64_t w_each, scales_each, bias_each;                      // between experts: bytes, bytes, elements
  int32_t experts, a_rows, index_div;                          // (M: rows of the result)
};

// The row of a behind row m of the result; with an index, negative where there is none.
__device__ __forceinline__ int64_t a_row_of(const LinParams&, int64_t m) { return m; }
__device__ __forceinline__ int64_t a_row_of(const GroupParams& p, int64_t m) {
  if (!p.index) return m;
  const int32_t i = p.index[m];
  const int32_t r = p.index_div == 1 ? i : (int32_t)((uint32_t)i / (uint32_t)p.index_div);
  return i >= 0 && r < p.a_rows ? r : -1;
}

// Inclusive prefix over a wavefront's lanes of f, whose identity is 0.
template <class F>
__device__ __forceinline__ int32_t wave_prefix(int32_t v, F f) {
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));  // one, two, four and eight lanes up in rows of 16,
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));  // then each row's last lane to the next row
  v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}

// What workgroup `block` computes: the tile's expert and place.  Every wavefront finds
// it by itself, 64 lanes with an equal share of the experts each, from a prefix over
// their row tiles, expert by expert.  (A group's last, partly empty tile is bound by
// reading w and the full ones by the matrix units, so they are better mixed than apart:
// with all full ones first 4096 x 8 rows over 128 experts took 400 us for 375.)
struct GroupTile {
  int32_t expert, first, last;                                 // rows [first, last) of the result; expert -1: nothing to do
  int32_t tm, tn;
};

__device__ __forceinline__ GroupTile group_tile(const GroupParams& p, int32_t block, int32_t bm) {
  constexpr int kPer = 1024 / 64;                              // a lane's experts at most
  const int lane = threadIdx.x & 63;
  const int32_t per = (p.experts + 63) / 64, e0 = lane * per;
  // Offsets count as the largest of those up to them, inside the result: out of order or
  // range they leave groups empty, but neither lead out of it nor share rows.
  int32_t at[kPer + 1];
#pragma unroll
  for (int i = 0; i <= kPer; ++i)
    if (i <= per) at[i] = p.offsets[min(e0 + i, p.experts)];
#pragma unroll
  for (int i = 0; i <= kPer; ++i)
    if (i <= per) {
      at[i] = min(max(at[i], 0), p.M);
      if (i) at[i] = max(at[i], at[i - 1]);
    }
  int32_t last = at[0];
#pragma unroll
  for (int i = 1; i <= kPer; ++i)
    if (i <= per) last = at[i];
  const int32_t upto_last = wave_prefix(last, [](int32_t a, int32_t b) { return max(a, b); });
  const int32_t before = __builtin_amdgcn_update_dpp(0, upto_last, 0x138, 0xF, 0xF, false);  // the lane below's
  int32_t sum = 0;
#pragma unroll
  for (int i = 0; i <= kPer; ++i)
    if (i <= per) {
      at[i] = max(at[i], before);
      if (i) sum += (at[i] - at[i - 1] + bm - 1) / bm;
    }
  const int32_t upto = wave_prefix(sum, [](int32_t a, int32_t b) { return a + b; });
  GroupTile t;
  t.expert = -1;
  t.first = t.last = t.tm = t.tn = 0;
  int32_t q;
  group_place(block, __builtin_amdgcn_readlane(upto, 63), p.tiles_n, q, t.tn);
  if (q < 0) return t;
  const int who = (int)__builtin_ctzll(__ballot(upto > q));     // the first prefix beyond q
  int32_t start = upto - sum, e = -1, first = 0, end = 0, tm = 0;
#pragma unroll
  for (int i = 1; i <= kPer; ++i)
    if (i <= per) {
      const int32_t tiles = (at[i] - at[i - 1] + bm - 1) / bm;
      if (e < 0 && q < start + tiles) {
        e = e0 + i - 1;
        first = at[i - 1];
        end = at[i];
        tm = q - start;
      }
      start += tiles;
    }
  t.expert = __builtin_amdgcn_readlane(e, who);
  t.first = __builtin_amdgcn_readlane(first, who);
  t.last = __builtin_amdgcn_readlane(end, who);
  t.tm = __builtin_amdgcn_readlane(tm, who);
  return t;
}

// The parameters of the tile's expert as those of a product of its own.
__device__ __forceinline__ void take_expert(GroupParams& p, const GroupTile& t) {
  p.M = t.last;
  p.w += t.expert * p.w_each;
  p.w_scales = static_cast<const char*>(p.w_scales) + t.expert * p.scales_each;
  if (p.bias) p.bias = static_cast<const char*>(p.bias) + t.expert * p.bias_each * (p.bias_type == kOutF32 ? 4 : 2);
}

template <bool kGroup>
using ParamsOf = std::conditional_t<kGroup, GroupParams, LinParams>;

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int32_t type) {
  if (type == kOutF32) return static_cast<const float*>(p)[i];
  const uint16_t u = static_cast<const uint16_t*>(p)[i];
  return type == kOutF16 ? (float)__builtin_bit_cast(_Float16, u) : __uint_as_float((uint32_t)u << 16);
}

// exp(x / 2), x in [-256, 88], by the exponential instruction (2^t, off by a step)
// with the rounding of t made up for.  Its square is exp(x) down to fp32's
// smallest numbers, which the instruction alone would flush to zero.
__device__ __forceinline__ float half_exp(float x) {
  const float c = 0.72134752044448170f;                        // log2(e) / 2
  const float t = x * c, rest = __builtin_fmaf(x, c, -t);
  const float h = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(h, rest * 0.69314718055994531f, h);
}

// erfc(x) by the Chebyshev fit t * exp(-x^2 + P(t)), t = 1 / (1 + |x| / 2), of
// Press et al., Numerical Recipes (the routine of fractional error below
// 1.2e-7 everywhere), so gelu does not cancel where erfc is tiny.
__device__ __forceinline__ float erfc_fit(float x) {
  const float z = fabsf(x), t = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
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
  const float h = half_exp(fmaxf(__builtin_fmaf(-z, z, q), -256.0f));
  const float r = t * h * h;
  return x < 0.0f ? 2.0f - r : r;
}

// The activations over a run of values: silu and gelu's tanh form as v *
// sigmoid(z) (z = 2u for the latter: 1 + tanh u would cancel for negative u),
// gelu's erf form as v * erfc(-v / sqrt 2) / 2.  With the exponential and the
// reciprocal instructions (a step each) a value of silu is off by at most 12 + z / 4
// half steps of fp32, of gelu's tanh form by 12 + 3 z and of its erf form by 16 + 4 z,
// where z is the exponent for v < 0 (|v|, |2u|, v^2 / 2; 0 for v >= 0): the
// roundings of z itself are not carried, and count only where the result is exp(-z)
// of v.  It takes about 20 instructions where expf() and a division took 45 (4096 x
// 4224 x 2816 exact, gated, 103 -> 100 us; 8192 x 4224 x 2816 bf16 190 -> 187): the
// epilogue is bound by the instructions it issues.
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
      const float h = half_exp(-fminf(fabsf(z), 256.0f));                // h * h = exp(-|z|)
      const float n = z < 0.0f ? v[i] * h * h : v[i];
      v[i] = n * __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f));
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

// A row scale as mantissa (in [1/2, 1); the scale itself where that is 0, infinite
// or NaN) and exponent.
struct Scale {
  float m;
  int e;
  __device__ __forceinline__ void set(float s) {
    m = __builtin_amdgcn_frexp_mantf(s);
    e = __builtin_amdgcn_frexp_expf(s);
  }
};

// sum * a * w, by mantissas first: the product of two scales alone can leave
// fp32's range where the result does not (1e21 * 1e18 under a sum of 2^-10).  Two
// roundings, as for the plain product, and one more where the result is
// subnormal.  Costs 1 to 2 % (4096 x 2816 x 2112 42.9 -> 43.6 us); with w's scales
// taken apart at each use, which needs no registers for their exponents, 44.1.
__device__ __forceinline__ float times_scales(float sum, const Scale& a, const Scale& w) {
  return __builtin_ldexpf(sum * (a.m * w.m), a.e + w.e);
}

// The terms of kLen output columns that do not depend on the row: bias, and the
// row scales of w (E4M3 operands with row scales).
template <int kKind, bool kGated, int kLen>
struct Columns {
  float b[kLen], bu[kGated ? kLen : 1];
  Scale s[is_row8(kKind) ? kLen : 1], su[is_row8(kKind) && kGated ? kLen : 1];
  float gain;

  __device__ __forceinline__ void load(const LinParams& p, int32_t n) {
    const int have = p.N - n;
    gain = 1.0f;
    if constexpr (kKind == kBf16 || kKind == kF16)
      if (p.gain) gain = *p.gain;
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
      float v[kLen];
      load_run<kLen>(p.w_scales, n, kOutF32, have, v);
#pragma unroll
      for (int i = 0; i < kLen; ++i) s[i].set(v[i]);
      if constexpr (kGated) {
        load_run<kLen>(p.w_scales, (int64_t)p.N + n, kOutF32, have, v);
#pragma unroll
        for (int i = 0; i < kLen; ++i) su[i].set(v[i]);
      }
    }
  }

  // `gate` (and `up`): the sums of row m of a; the outputs, before the residual and
  // before rounding, replace `gate`.
  __device__ __forceinline__ void finish(const LinParams& p, int64_t m, float* gate, const float* up) const {
    Scale am;
    if constexpr (is_row8(kKind)) am.set(static_cast<const float*>(p.a_scales)[m]);
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      if constexpr (is_row8(kKind)) gate[i] = times_scales(gate[i], am, s[i]);
      else if constexpr (kKind == kBf16 || kKind == kF16) gate[i] *= gain;
      gate[i] += b[i];
    }
    activate_run<kLen>(gate, p.act);
    if constexpr (kGated) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) {
        float u = up[i];
        if constexpr (is_row8(kKind)) u = times_scales(u, am, su[i]);
        else if constexpr (kKind == kBf16 || kKind == kF16) u *= gain;
        gate[i] *= u + bu[i];
      }
    }
  }
};

// kLen residual elements of row m, held as they were loaded, so that the loads of
// several rows are in flight together.
template <int kLen>
struct Residual {
  uint32_t d[kLen];                                              // 16-bit types: the first half

  __device__ __forceinline__ void load(const LinParams& p, int64_t m, int32_t n) {
    if (!p.residual || n >= p.N) return;
    const int64_t at = m * p.ldr + n;
    const int have = p.N - n;
    const bool wide = p.residual_type == kOutF32;
    const char* src = static_cast<const char*>(p.residual) + at * (wide ? 4 : 2);
    if (have >= kLen && (reinterpret_cast<uintptr_t>(src) & (kLen >= 8 ? 15 : 7)) == 0) {
      if constexpr (kLen >= 8) {
#pragma unroll
        for (int i = 0; i < kLen / 2; i += 4) *reinterpret_cast<u32x4*>(d + i) = *reinterpret_cast<const u32x4*>(src + 4 * i);
        if (wide) {
#pragma unroll
          for (int i = kLen / 2; i < kLen; i += 4) *reinterpret_cast<u32x4*>(d + i) = *reinterpret_cast<const u32x4*>(src + 4 * i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLen / 2; i += 2) *reinterpret_cast<uint2*>(d + i) = *reinterpret_cast<const uint2*>(src + 4 * i);
        if (wide) {
#pragma unroll
          for (int i = kLen / 2; i < kLen; i += 2) *reinterpret_cast<uint2*>(d + i) = *reinterpret_cast<const uint2*>(src + 4 * i);
        }
      }
    } else if (wide) {
#pragma unroll
      for (int i = 0; i < kLen; ++i)
        if (i < have) d[i] = reinterpret_cast<const uint32_t*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < kLen / 2; ++i) {
        const uint32_t lo = 2 * i < have ? reinterpret_cast<const uint16_t*>(src)[2 * i] : 0;
        const uint32_t hi = 2 * i + 1 < have ? reinterpret_cast<const uint16_t*>(src)[2 * i + 1] : 0;
        d[i] = lo | (hi << 16);
      }
    }
  }

  __device__ __forceinline__ void add(const LinParams& p, float* v) const {
    if (!p.residual) return;
    if (p.residual_type == kOutF32) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) v[i] += __uint_as_float(d[i]);
    } else if (p.residual_type == kOutF16) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) v[i] += (float)__builtin_bit_cast(_Float16, (uint16_t)(d[i / 2] >> (16 * (i & 1))));
    } else {
#pragma unroll
      for (int i = 0; i < kLen; ++i) v[i] += (i & 1) ? bf16_hi(d[i / 2]) : bf16_lo(d[i / 2]);
    }
  }
};

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
  if (p.out_type == kOutF16) {
#pragma unroll
    for (int i = 0; i < kLen / 2; ++i) d[i] = pack_f16(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kLen / 2; ++i) d[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
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
  static_assert(kLen == 4 || kLen == 8, "lanes per block");
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLen; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const bool finite = top < 0x7F800000u;
  if (!finite) {
    top = 0;
#pragma unroll
    for (int i = 0; i < kLen; ++i) top = max(top, finite_mag(v[i]));
  }
  top = quad_max(top);
  if (kLen == 4) top = max(top, (uint32_t)__shfl_xor((int)top, 4, 64));
  float inv;
  const uint32_t code = block_scale_code(top, inv);
  if (!in) return;
  uint8_t* dst = static_cast<uint8_t*>(p.out) + m * p.ldo + n;
#pragma unroll
  for (int i = 0; i < kLen; i += 4) {
    // (finite values over their block's scale are at most 448)
    uint32_t d;
    if (finite) d = encode4_scaled(v + i, inv);
    else d = encode4_e4m3(v + i, inv);
    *reinterpret_cast<uint32_t*>(dst + i) = d;
  }
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
struct WideOp {
  bf16x8_t v[4];
  template <int kByte>
  __device__ __forceinline__ void widen(const Frag& f, const uint32_t* s) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // 2^(code - 127): the conversion reads the exponent alone, so code 0 is 2^-127 and
      // 255 NaN, as for the scaled instruction
      const float scale = __uint_as_float(((s[c] >> (8 * kByte)) & 0xFFu) << 23);
      v[2 * c] = widen8(f.c[c].x, f.c[c].y, scale);
      v[2 * c + 1] = widen8(f.c[c].z, f.c[c].w, scale);
    }
  }
};
template <int kByte>
struct PreparedWide : WideOp {
  __device__ __forceinline__ void set(const Frag& f, const uint32_t* s) { widen<kByte>(f, s); }
};
template <int kByte>
struct Prepared<kRow8Wide, kByte> : PreparedWide<kByte> {};
template <int kByte>
struct Prepared<kBlock8Wide, kByte> : PreparedWide<kByte> {};

// acc += w . a over the s-th of a K step's kSubs parts; w is the row operand, so a
// lane's four results are four consecutive output columns (instruction rows 4g ..
// 4g + 3) of one row of a.
template <int kKind>
constexpr int kSubs = is_wide(kKind) ? 4 : kKind == kRow8 || kKind == kBlock8 ? 1 : 2;

template <int kKind, int kByte>
__device__ __forceinline__ f32x4 mma(const Prepared<kKind, kByte>& w, const Prepared<kKind, kByte>& a, int s, f32x4 acc) {
  if constexpr (is_wide(kKind))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[s], a.v[s], acc, 0, 0, 0);
  else if constexpr (kKind == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w.f.c[s]),
                                                   __builtin_bit_cast(bf16x8_t, a.f.c[s]), acc, 0, 0, 0);
  else if constexpr (kKind == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w.f.c[s]),
                                                  __builtin_bit_cast(half8_t, a.f.c[s]), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8_t, w.f), __builtin_bit_cast(i32x8_t, a.f),
                                                            acc, 0, 0, kByte, (int)w.scale, kByte, (int)a.scale);
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

// Copies 16 bytes per lane from base + off to consecutive places in LDS from `lds`
// on.  Written out because the compiler, where it knows of such a copy, waits for
// all of them before the next LDS read, and the copies of later steps must stay on
// their way.  No register receives the data; step_barrier() waits for it.
__device__ __forceinline__ void copy_lds16(uint64_t base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}

// The same from an address of each lane.
__device__ __forceinline__ void copy_lds16(uint64_t from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)p);
}

// Barrier at the turn of a step: this wavefront's copies into LDS have arrived
// and its LDS reads are done before any wavefront passes.  The wait is written
// out because the copies are counted with memory loads, whose completion a
// workgroup barrier by itself does not ask for.
// kLeft: copies of later steps that may still be on their way.
template <int kLeft>
__device__ __forceinline__ void step_barrier() {
  static_assert(kLeft < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLeft) : "memory");
  lds_barrier();
}

// ---- tiled kernel -------------------------------------------------------------
// A workgroup of kWM x kWN wavefronts owns kBM rows of a and kBN rows of w
// (gated: kBN / 2 output columns, their gate rows, then their up rows).  Each K
// step's rows are copied straight into LDS (kStages buffers).  The epilogue passes
// the sums through LDS, 32 rows of each wavefront at a time, so that every thread
// finishes 8 consecutive outputs of a row and whole rows are stored.
//
// Tiles.  A step of a 256 x 256 tile reads 64 KiB and multiplies 256 x 256 x 128
// bytes: its eight wavefronts of 128 x 64 read 384 LDS rows per 128 matrix
// instructions of 16 cycles, so LDS is busy a quarter of the time and the matrix
// units set the pace.  8192^3, on 256 and on 128 tiles: bf16 833 to 906 us (1.32 to
// 1.21 PFLOP/s, as power holds the clock, 1.5 to 2.0 GHz) and 994 to 1047, row scales 443
// to 500 (2.48 to 2.20 PFLOP/s) and 511 to 536, block scales 446 to 465 and 557 to 581.
// The matrix units are busy 64 % of the cycles in bf16, 61 % with row and 58 % with block
// scales, LDS 25 to 27 % with up to 2 % conflicts; 1.6 GB are read for 268 MB of bf16
// operands.  128 x 128 tiles (two workgroups per CU) take the exact 8-bit products,
// which need the registers for converted operands (8192^3 in 821 to 859 us with row
// scales, the bf16 instruction's rate, 914 to 942 with block scales), and sizes whose
// 256 tiles would leave CUs idle.  64 x 64 tiles with four buffers take middle sizes,
// where latency and not rate counts: 512 x 2816 x 2112 bf16 in 16.1 to 17.6 us on them,
// 24 on 128 tiles; 1000 x 1411 x 704 fp16 10.6 and 16.8.
// The 32x32x16 instructions were 3 % slower (902 against 876 us), copies issued
// between the last instructions of a step 10 % (128 tiles), and four wavefronts of
// 128 x 128 need more accumulators than the compiler keeps in place.
template <int kKind, int kBM, int kBN, int kWM, int kWN, int kStages, bool kGated, bool kGroup>
__global__ __launch_bounds__(64 * kWM * kWN, 2) void linear_tile_kernel(const ParamsOf<kGroup> given) {
  constexpr int kWaves = kWM * kWN;
  constexpr int kTM = kBM / kWM, kTN = kBN / kWN;
  constexpr int kFM = kTM / 16, kFN = kTN / 16;
  constexpr int kOutN = kGated ? kBN / 2 : kBN;                // output columns of the tile
  constexpr int kStage = (kBM + kBN) * kStep;
  constexpr int kLoads = (kBM + kBN) / 8 / kWaves;             // 1 KiB copies per wavefront and step
  static_assert((kBM + kBN) / 8 % kWaves == 0 && kBM / 8 % kLoads == 0, "whole copies; a wavefront copies one operand");
  static_assert(!kGated || kOutN % (8 * kLoads) == 0, "a wavefront copies gate or up rows");
  constexpr bool kScaled = is_block8(kKind);
  static_assert(kBM + kBN <= 64 * kWaves || !kScaled, "a thread loads the scales of one row");
  static_assert((kStages & (kStages - 1)) == 0, "buffer of a step by masking");
  // Grouped: a group's last tile has few rows of a to keep, and w for it comes from memory,
  // so its steps get as many buffers as LDS holds (two workgroups of 128-row tiles a CU).
  constexpr bool kDeep = kGroup && kBM >= 128 && !is_wide(kKind);
  static_assert(!kDeep || !kScaled, "scales would take a part of the LDS");
  constexpr int kSmem = !kDeep ? kStages * kStage : kBM == 256 ? 160 * 1024 : 72 * 1024;
  __shared__ __align__(1024) char smem[kSmem];
  __shared__ __align__(16) uint32_t s_scale[kScaled ? 2 : 1][kScaled ? kBM + kBN : 1][4];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int wm = wave / kWN, wn = wave % kWN;

  // this workgroup's tile and K steps: all of them, or a part's
  ParamsOf<kGroup> p = given;
  Work work;
  int64_t m0;
  if constexpr (kGroup) {
    const GroupTile tile = group_tile(given, (int32_t)blockIdx.x, kBM);
    if (tile.expert < 0) return;
    take_expert(p, tile);
    work = Work{0, tile.tm, tile.tn, -1, 0, (p.kbytes + kStep - 1) / kStep};
    m0 = tile.first + (int64_t)tile.tm * kBM;
  } else {
    work = work_at((int32_t)blockIdx.x, p.tiles_m, p.tiles_n, p.whole, p.parts, p.part_steps, p.kbytes);
    m0 = (int64_t)work.tm * kBM;
  }
  const bool whole = work.part < 0;
  const int step0 = work.step0, steps = work.steps;
  const int32_t n0 = work.tn * kOutN;

  // source of each copy: lane -> (row of the operand's tile, chunk).  Rows past the
  // edge repeat the last row, their results are not stored.  The offset from the
  // tile's first row is formed at each copy (three instructions): kept for all
  // copies, it would cost the registers that the fragments need.
  const Copies from = copies_at(wave, lane, kLoads, kBM, kOutN);
  const int chunk = from.chunk;
  int row0 = from.row0;
  const int last_row = from.of_a ? last_row_of(kBM, p.M, m0) : last_row_of(kOutN, p.N, n0);
  const uint32_t ld = (uint32_t)(from.of_a ? p.lda : p.ldw);
  // (grouped: rows of a may lie anywhere in it, so each copy's row is kept and its
  // address formed in 64 bits)
  uint64_t base = reinterpret_cast<uint64_t>((from.of_a ? p.a : p.w) + copy_base(from, kGroup ? 0 : m0, n0, p.N, p.lda, p.ldw, step0));
  int32_t row_at[kGroup ? kLoads : 1];
  if constexpr (kGroup) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) row_at[i] = min(row0 + 8 * i, last_row);
    if (from.of_a) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) row_at[i] += (int32_t)m0;
      if (p.index) {
        int32_t pair[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) pair[i] = p.index[row_at[i]];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t r = p.index_div == 1 ? (uint32_t)pair[i] : (uint32_t)pair[i] / (uint32_t)p.index_div;
          row_at[i] = pair[i] >= 0 && r < (uint32_t)p.a_rows ? (int32_t)r : 0;
        }
      }
    }
  }
  const int tail = last_bytes(p.kbytes, step0, steps);
  int ring = kStages, stage = kStage, a_bytes = kBM * kStep;
  if constexpr (kDeep) {
    const int rows = last_row_of(kBM, p.M, m0) + 1;
    if (rows <= kBM / 2) {
      const bool quarter = kBM == 256 && rows <= kBM / 4;
      a_bytes = (quarter ? kBM / 4 : kBM / 2) * kStep;
      stage = a_bytes + kBN * kStep;
      ring = quarter ? 4 : 3;
    }
  }
  // (a wavefront copies all rows of its part or, behind the last row, none: step_barrier
  // counts copies)
  const int my_part = wave * kLoads * 1024 - (from.of_a ? 0 : kBM * kStep - a_bytes);
  const bool mine = !kGroup || !from.of_a || __builtin_amdgcn_readfirstlane(row0) <= last_row;
  // step ks's copies, into the buffer at `at`
  auto fetch = [&](int ks, int at) {
    if (!mine) {
      base += kStep;
      return;
    }
    char* dst = smem + at + my_part;
    if (chunk * 16 < (ks == steps - 1 ? tail : kStep)) {
      const uint32_t to = lds_address(dst);
      asm volatile("" : "+v"(row0));                           // (formed here, not carried along)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if constexpr (kGroup) copy_lds16(base + (uint64_t)(uint32_t)row_at[i] * ld + (uint32_t)chunk * 16, to + i * 1024);
        else copy_lds16(base, copy_offset(row0 + 8 * i, last_row, ld, chunk), to + i * 1024);
      }
    } else {                                                   // past the end of the rows
#pragma unroll
      for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(dst + i * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
    }
    base += kStep;
  };

  int slot = 0, slot_next = stage;                              // (kDeep) this step's buffer and the next one's
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
    const int r = min((int)threadIdx.x, kBM + kBN - 1);
    if (r < kBM) {
      scale_row = static_cast<const uint8_t*>(p.a_scales) + max(a_row_of(p, min(m0 + r, (int64_t)p.M - 1)), (int64_t)0) * nblk;
    } else {
      const int q = r - kBM;
      scale_row = static_cast<const uint8_t*>(p.w_scales) +
                  ((int64_t)min(n0 + q % kOutN, p.N - 1) + (q >= kOutN ? p.N : 0)) * nblk;
    }
  }

  // Rows of the operands' tiles that a wavefront multiplies: fragment i of a from row
  // a_first + a_row(i) on, fragment j of w from w_first + w_row(j) on.  Grouped: the
  // wavefronts' fragments take turns, gate before up, so that a tile whose rows or columns
  // end early leaves every wavefront the same fewer of them.
  const int a_first = kGroup ? wm * 16 : wm * kTM, w_first = kGroup ? wn * 16 : wn * kTN;
  auto a_row = [](int i) { return kGroup ? i * 16 * kWM : i * 16; };
  auto w_row = [](int j) {
    if (!kGroup) return j * 16;
    return kGated ? (j & 1) * kOutN + (j >> 1) * 16 * kWN : j * 16 * kWN;
  };
  // Grouped: groups end inside tiles, and empty fragments would cost as much as full ones,
  // so each wavefront leaves out those of a past the tile's last row, and the second half
  // of w's where the tile's columns end before.
  constexpr bool kCut = kGroup && !is_wide(kKind);
  const int have_i = kCut ? (last_row_of(kBM, p.M, m0) + 16 * kWM) / (16 * kWM) : kFM;
  constexpr bool kCutColumns = kCut && kFN >= (kGated ? 4 : 2);  // (gate and up stay together)
  const bool all_j = !kCutColumns || p.N - n0 > kOutN / 2;

  // Main loop.  A step runs its groups of instructions (one 16-row fragment of a
  // with all of w) in order, the fragments of a being read kAhead groups ahead; the
  // last kAhead groups run fragment of w by fragment of w.  The barrier falls before
  // them: behind it the buffer that the step has read is refilled for a later
  // step, and each fragment of w is replaced by the next step's as soon as
  // its last instruction is issued, so the matrix unit does not wait for LDS at
  // the turn of a step.  T: the step's number modulo 4 (2 without block
  // scales), for the byte of the scales and the slots of fa when a step has only
  // two groups.
  static_assert(kFM == 2 || kFM % 4 == 0, "fragment slots");
  constexpr int kAhead = kFM == 8 && kKind >= kRow8 ? 1 : 2;   // 8-bit fragments: one group, for want of registers
  constexpr int kWords = kKind == kBlock8Wide ? 2 : 1;         // scale words of a lane and row
  // copies issued under the first matrix instructions after the barrier rather than
  // right behind it: 8192^3 with block scales on 128-row tiles 650 -> 603 us, but
  // bf16 on them 999 -> 1030
  constexpr bool kLate = kKind >= kRow8 || kFM == 8;
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
      for (int i = 0; i < kFM; ++i) va[i][c] = s_scale[kScaled ? buf : 0][kScaled ? a_first + a_row(i) + i16 : 0][word];
#pragma unroll
      for (int j = 0; j < kFN; ++j) vw[j][c] = s_scale[kScaled ? buf : 0][kScaled ? kBM + w_first + w_row(j) + i16 : 0][word];
    }
  };
  // The compiler would move the reads back to their uses and the matrix
  // instructions to a later block.  The wide kinds are left to it: there it
  // overlaps the conversions with matrix instructions.
  auto hold = [] {
    if constexpr (!is_wide(kKind)) __builtin_amdgcn_sched_barrier(0);
  };
  auto issued = [](f32x4& v) {
    if constexpr (!is_wide(kKind)) asm volatile("" : "+v"(v));
  };
  auto step = [&](auto t, int ks) {
    constexpr int T = decltype(t)::value;
    constexpr int kBase = kFM == 2 ? 2 * (T & 1) : 0;          // slot of group 0
    constexpr int kNext = kFM == 2 ? 2 - 2 * (T & 1) : 0;      // slot of the next step's group 0
    typedef Prepared<kKind, T> Op;
    const int here = kDeep ? slot : (ks & (kStages - 1)) * kStage;
    const int next = kDeep ? slot_next : ((ks + 1) & (kStages - 1)) * kStage;
    const char* ta = smem + here + a_first * kStep;
    const char* na = smem + next + a_first * kStep;
    const char* nw = smem + next + a_bytes + w_first * kStep;
    if constexpr (kScaled && T == 0) read_scales((ks >> 2) & 1);
    Op pw[kFN];
#pragma unroll
    for (int j = 0; j < kFN; ++j) pw[j].set(fw[j], vw[j]);
#pragma unroll
    for (int i = 0; i < kFM - kAhead; ++i) {
      fa[(kBase + i + kAhead) & 3] = read_frag(ta, a_row(i + kAhead) + i16, g);
      hold();
      if (!kCut || i < have_i) {
        Op pa;
        pa.set(fa[(kBase + i) & 3], va[i]);
        // the wavefront that has its fragments goes first: 8192^3 with block scales
        // 501 -> 462 us, nothing lost elsewhere
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int u = 0; u < kSubs<kKind>; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (h == 0 || !kCutColumns || all_j) {
#pragma unroll
              for (int j = h * kFN / 2; j < (h + 1) * kFN / 2; ++j) acc[j][i] = mma<kKind, T>(pw[j], pa, u, acc[j][i]);
            }
#pragma unroll
        for (int j = 0; j < kFN; ++j) issued(acc[j][i]);
        __builtin_amdgcn_s_setprio(0);
      }
      hold();
    }
    if constexpr (kScaled) {
      // the next four steps' scales: loaded a step before they go to LDS, which
      // is a step before they are read
      if constexpr (T == 1) scale_next = load_scales(scale_row, 4 * (step0 + ks + 3), nblk);
      if constexpr (T == 2)
        if (threadIdx.x < kBM + kBN) *reinterpret_cast<u32x4*>(s_scale[1 - ((ks >> 2) & 1)][threadIdx.x]) = scale_words(scale_next);
    }
    // behind the barrier this buffer is read and the next one filled; copies that
    // are on their way then are those of the steps from ks + 2 on
    if (kStages > 2 && ks + kStages <= steps) step_barrier<(kStages - 2) * kLoads>();
    else if (kDeep && kBM == 256 && ring == 4 && ks + 4 <= steps) step_barrier<2 * kLoads>();
    else if (kDeep && ring == 3 && ks + 3 <= steps) step_barrier<kLoads>();
    else step_barrier<0>();
    if (!kLate && ks + ring < steps) fetch(ks + ring, here);
    Op pa[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) pa[i].set(fa[(kBase + kFM - kAhead + i) & 3], va[kFM - kAhead + i]);
    // (after the last step these read an older one, unused)
    fa[kNext] = read_frag(na, i16, g);
    if (kAhead == 2) fa[kNext + 1] = read_frag(na, a_row(1) + i16, g);
    hold();
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      if (!kCut || (kFM - kAhead < have_i && (j < kFN / 2 || !kCutColumns || all_j))) {
#pragma unroll
        for (int u = 0; u < kSubs<kKind>; ++u)
#pragma unroll
          for (int i = kFM - kAhead; i < kFM; ++i) acc[j][i] = mma<kKind, T>(pw[j], pa[i - kFM + kAhead], u, acc[j][i]);
#pragma unroll
        for (int i = kFM - kAhead; i < kFM; ++i) issued(acc[j][i]);
      }
      fw[j] = read_frag(nw, w_row(j) + i16, g);
      hold();
      if (kLate && j == 0 && ks + ring < steps) fetch(ks + ring, here);
    }
    if constexpr (kDeep) {
      slot = slot_next;
      slot_next = slot_next + stage == ring * stage ? 0 : slot_next + stage;
    }
  };
  // The wide kinds' step where a wavefront has four groups: the conversions of each
  // fragment stand among the matrix instructions before its first use (w's for the
  // next step as soon as the last instruction on the old one is issued), two groups
  // at a time, fragment of w by fragment of w.
  constexpr bool kWideStep = is_wide(kKind) && kFM == 4;
  WideOp ww[kWideStep ? kFN : 1], wa[2];
  auto mix = [](auto valu) {                                   // eight matrix instructions, `valu` others after each
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, decltype(valu)::value, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto pair = [&](int j, int i0, const WideOp* a2) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[j][i0 + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[j].v[u], a2[i].v[u], acc[j][i0 + i], 0, 0, 0);
  };
  auto wide_step = [&](auto t, int ks) {
    constexpr int T = decltype(t)::value, N = (T + 1) % 4;
    const char* ta = smem + (ks & (kStages - 1)) * kStage + a_first * kStep;
    const char* na = smem + ((ks + 1) & (kStages - 1)) * kStage + a_first * kStep;
    const char* nw = smem + ((ks + 1) & (kStages - 1)) * kStage + (kBM + w_first) * kStep;
    WideOp wb[2];
    fa[2] = read_frag(ta, a_row(2) + i16, g);
    fa[3] = read_frag(ta, a_row(3) + i16, g);
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      if (j == 0) ww[kFN - 1].template widen<T>(fw[kFN - 1], vw[kFN - 1]);
      if (j == 1) wb[0].template widen<T>(fa[2], va[2]);
      if (j == 2) wb[1].template widen<T>(fa[3], va[3]);
      pair(j, 0, wa);
      mix(std::integral_constant<int, 2>{});
    }
    if constexpr (kScaled) {
      if constexpr (T == 1) scale_next = load_scales(scale_row, 4 * (step0 + ks + 3), nblk);
      if constexpr (T == 2)
        if (threadIdx.x < kBM + kBN) *reinterpret_cast<u32x4*>(s_scale[1 - ((ks >> 2) & 1)][threadIdx.x]) = scale_words(scale_next);
    }
    step_barrier<0>();
    if constexpr (kScaled && T == 3) read_scales(((ks >> 2) + 1) & 1);
    fa[0] = read_frag(na, i16, g);
    fa[1] = read_frag(na, a_row(1) + i16, g);
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      if (j > 0) ww[j - 1].template widen<N>(fw[j - 1], vw[j - 1]);
      if (j >= 2) wa[j - 2].template widen<N>(fa[j - 2], va[j - 2]);
      pair(j, 2, wb);
      fw[j] = read_frag(nw, w_row(j) + i16, g);
      mix(std::integral_constant<int, 3>{});
      if (j == 0 && ks + kStages < steps) fetch(ks + kStages, (ks & (kStages - 1)) * kStage);
    }
  };
  for (int ks = 0; ks < ring && ks < steps; ++ks) fetch(ks, ks * stage);
  if constexpr (kScaled)
    if (threadIdx.x < kBM + kBN) *reinterpret_cast<u32x4*>(s_scale[0][threadIdx.x]) = scale_words(load_scales(scale_row, 4 * step0, nblk));
  // (grouped: short products count every microsecond before the first step)
  if (kDeep && steps >= ring) {
    if (ring == 2) step_barrier<kLoads>();
    else if (ring == 3) step_barrier<2 * kLoads>();
    else step_barrier<3 * kLoads>();
  } else {
    step_barrier<0>();
  }
#pragma unroll
  for (int j = 0; j < kFN; ++j) fw[j] = read_frag(smem + a_bytes + w_first * kStep, w_row(j) + i16, g);
  fa[0] = read_frag(smem + a_first * kStep, i16, g);
  if (kAhead == 2) fa[1] = read_frag(smem + a_first * kStep, a_row(1) + i16, g);
  if constexpr (kWideStep) {
    if constexpr (kScaled) read_scales(0);
#pragma unroll
    for (int j = 0; j < kFN - 1; ++j) ww[j].template widen<0>(fw[j], vw[j]);
#pragma unroll
    for (int i = 0; i < 2; ++i) wa[i].template widen<0>(fa[i], va[i]);
  }
  auto run_step = [&](auto t, int ks) {
    if constexpr (kWideStep) wide_step(t, ks);
    else step(t, ks);
  };
  for (int ks = 0;;) {
    run_step(std::integral_constant<int, 0>{}, ks);
    if (++ks == steps) break;
    run_step(std::integral_constant<int, 1>{}, ks);
    if (++ks == steps) break;
    if constexpr (kScaled) {
      run_step(std::integral_constant<int, 2>{}, ks);
      if (++ks == steps) break;
      run_step(std::integral_constant<int, 3>{}, ks);
      if (++ks == steps) break;
    }
  }

  // Epilogue: groups 2 * pass and 2 * pass + 1 of every wavefront through LDS.
  constexpr int kLd = kBN + 4;                                 // floats per row: 8 rows start on distinct banks
  constexpr int kRows = 32 * kWM;
  constexpr int kPer = kOutN / 8;                              // threads per row
  constexpr int kRowsPerIter = 64 * kWaves / kPer, kIters = kRows / kRowsPerIter;
  static_assert(kRows * kLd * 4 <= kStages * kStage && kRows % kRowsPerIter == 0, "the pass fits the step buffers");
  float* tile = reinterpret_cast<float*>(smem);
  // the tile's row behind row r of a pass (wavefront row, fragment, row)
  auto tile_row = [&](int r, int pass) {
    if (!kGroup) return (r / 32) * kTM + pass * 32 + r % 32;
    return r / 32 * 16 + a_row(2 * pass + (r / 16 & 1)) + (r & 15);
  };
  const int c = (int)(threadIdx.x % kPer) * 8;
  const int32_t n = n0 + c;
  // Gathered: the rows of a once more, all together (they were not worth registers
  // through the loop; loaded row by row here each would be waited for, 0.7 us a pass).
  int32_t* s_rows = reinterpret_cast<int32_t*>(smem + kRows * kLd * 4);
  if constexpr (kGroup) {
    static_assert(kRows * kLd * 4 + kBM * 4 <= kSmem && kBM <= 64 * kWaves, "room for the rows");
    if (p.index && threadIdx.x < kBM) s_rows[threadIdx.x] = m0 + threadIdx.x < p.M ? (int32_t)a_row_of(p, m0 + threadIdx.x) : -1;
  }
  Columns<kKind, kGated, 8> cols;
  cols.load(p, n);
#pragma unroll 1
  for (int pass = 0; pass < (kCut ? (have_i + 1) / 2 : kFM / 2); ++pass) {
    Residual<8> res[kIters];
#pragma unroll
    for (int k = 0; k < kIters; ++k) {
      const int r = (int)threadIdx.x / kPer + k * kRowsPerIter;
      if constexpr (!kGroup)
        if (whole) res[k].load(p, min(m0 + tile_row(r, pass), (int64_t)p.M - 1), n);
    }
    lds_barrier();                                             // the steps' (or the last pass's) reads are done
    float* dst = tile + (wm * 32 + i16) * kLd + w_first + 4 * g;
#pragma unroll
    for (int q = 0; q < kFM / 2; ++q)
      if (q == pass) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < kFN; ++j) *reinterpret_cast<f32x4*>(dst + i * 16 * kLd + w_row(j)) = acc[j][2 * q + i];
      }
    lds_barrier();
#pragma unroll
    for (int k = 0; k < kIters; ++k) {
      const int r = (int)threadIdx.x / kPer + k * kRowsPerIter;
      const int64_t m = m0 + tile_row(r, pass);
      int64_t mr = m < p.M ? m : (int64_t)p.M - 1;
      bool in = m < p.M && n < p.N;
      if constexpr (kGroup) {
        if (p.index) {
          const int32_t ma = s_rows[tile_row(r, pass)];
          in = ma >= 0 && n < p.N;
          mr = max(ma, 0);
        }
      }
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
      if (!whole) {
        float* sum = p.partial + partial_at(work.tile - p.whole, work.part, p.parts, (int)(m - m0), c, kBM, kBN);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<f32x4*>(sum + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
          if constexpr (kGated)
            *reinterpret_cast<f32x4*>(sum + kOutN + 4 * h) = f32x4{u[4 * h], u[4 * h + 1], u[4 * h + 2], u[4 * h + 3]};
        }
        continue;
      }
      cols.finish(p, mr, v, u);
      if constexpr (!kGroup) res[k].add(p, v);
      if (p.out_type != kOutBlock8) {
        if (in) store_run<8>(p, m, n, v);
      } else {
        store_block<8>(p, m, n, v, in);
      }
    }
  }
}

// ---- joining the parts -----------------------------------------------------------
// The sums of a tile's parts, added in order, through the same epilogue; a thread
// finishes 8 consecutive outputs of a row.  Bound by a launch and the sums' way
// back from memory: 4.4 us for 4 parts of 4096 x 128, 6.0 us for the gated last round
// of 8192 x 2112.  With and without the cut (inputs in the last-level cache / from
// memory): 8192 x 4224 x 2816 bf16 gated 191 and 197 us / 223 and 244 (64 of 2112 tiles
// in 4 parts), 4096 x 4224 x 2816 exact 102 and 110 / 110 and 119, 4096 x 128 x 2816 15.6
// and 17.1 / 18.2 and 18.4.
template <int kKind, bool kGated>
__global__ __launch_bounds__(256) void linear_join_kernel(const LinParams p, int32_t bm, int32_t bn) {
  const int32_t out_n = kGated ? bn / 2 : bn, per = out_n / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)(p.tiles_m * p.tiles_n - p.whole) * bm * per) return;  // whole rows of a tile
  const int32_t c = (int32_t)(id % per) * 8;
  const int32_t r = (int32_t)(id / per % bm);
  const int32_t left = (int32_t)(id / ((int64_t)per * bm));
  int32_t tm, tn;
  tile_at(p.tiles_m, p.tiles_n, p.whole + left, tm, tn);
  const int64_t m = (int64_t)tm * bm + r;
  const int32_t n = tn * out_n + c;
  const bool in = m < p.M && n < p.N;
  const int64_t mr = m < p.M ? m : (int64_t)p.M - 1;
  Columns<kKind, kGated, 8> cols;
  cols.load(p, n);
  Residual<8> res;
  res.load(p, mr, n);
  float v[8] = {}, u[8] = {};
  const float* sum = p.partial + partial_at(left, 0, p.parts, r, c, bm, bn);
  // four parts' loads in flight, added in order
  for (int32_t part = 0; part < p.parts; part += 4) {
    f32x4 x[4][2], y[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* from = sum + (int64_t)min(part + q, p.parts - 1) * bm * bn;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[q][h] = *reinterpret_cast<const f32x4*>(from + 4 * h);
        if constexpr (kGated) y[q][h] = *reinterpret_cast<const f32x4*>(from + out_n + 4 * h);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (part + q < p.parts) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] += x[q][i / 4][i % 4];
          if constexpr (kGated) u[i] += y[q][i / 4][i % 4];
        }
      }
  }
  cols.finish(p, mr, v, u);
  res.add(p, v);
  if (p.out_type != kOutBlock8) {
    if (in) store_run<8>(p, m, n, v);
  } else {
    store_block<8>(p, m, n, v, in);
  }
}

// ---- few rows -------------------------------------------------------------------
// At most 16 rows of a: bound by reading w once, so w goes straight from memory to
// registers.  A workgroup owns kCols output columns (gated: their gate and up
// rows); its wavefronts take groups of four K steps in turn (a row's block scales
// of a group are 16 bytes), kBatch steps' loads in flight at once, and their
// partial sums are added in wavefront order through LDS.  With w from memory 1 x 8192 x 8192
// takes 29.0 us in bf16 (134 MB, 4.6 TB/s) and 16.7 with 8 bits and row scales (4.0 TB/s),
// 16 x 8192 x 8192 with block scales 25.3 (2.7 TB/s: scales and conversions of w come on
// top); with w in the last-level cache 25.0, 14.3 and 19.9.  Small products are bound by
// a launch and one round of loads: 5 x 2816 x 2112 in 4.7 us, 16 x 128 x 2816 in 7.2,
// whose eight workgroups each read 180 kB.
template <int kKind, int kCols, int kWaves, bool kGated>
__global__ __launch_bounds__(64 * kWaves) void linear_few_kernel(const LinParams p) {
  constexpr int kRows = kGated ? 2 * kCols : kCols;            // rows of w
  constexpr int kFN = kRows / 16;
  // steps in flight: what 64 (16 wavefronts) or 128 kB of registers hold
  constexpr int kBatch = kFN == 1 ? 4 : kFN == 2 ? (kWaves == 16 ? 2 : 4) : kWaves == 16 ? 1 : 2;
  constexpr int kLd = kRows + 4;                               // floats per row of a partial tile
  __shared__ __align__(16) float part[kWaves][16][kLd];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int32_t n0 = (int32_t)blockIdx.x * kCols;
  const int32_t nblk = p.kbytes / 32;

  const char* pw[kFN];
  const uint8_t* sw[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    const int r = j * 16 + i16;
    int32_t n = n0 + r % kCols;
    n = n < p.N ? n : p.N - 1;
    const int64_t row = (int64_t)n + (r >= kCols ? p.N : 0);
    pw[j] = p.w + row * p.ldw;
    sw[j] = static_cast<const uint8_t*>(p.w_scales) + row * nblk;
  }
  const int64_t row = i16 < p.M ? i16 : p.M - 1;
  const char* pa = p.a + row * p.lda;
  const uint8_t* sa = static_cast<const uint8_t*>(p.a_scales) + row * nblk;
  f32x4 acc[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) acc[j] = f32x4{0, 0, 0, 0};

  const int steps = (p.kbytes + kStep - 1) / kStep;
  for (int first = 4 * wave; first < steps; first += 4 * kWaves) {
    u32x4 da, dw[kFN];                                         // scales: word b, the blocks of step first + b
    if constexpr (is_block8(kKind)) {
      da = load_scales(sa, 4 * first, nblk);
#pragma unroll
      for (int j = 0; j < kFN; ++j) dw[j] = load_scales(sw[j], 4 * first, nblk);
    }
#pragma unroll
    for (int h = 0; h < 4; h += kBatch) {
      // a chunk (or a step) past the end of the rows counts as zeros
      Frag fw[kBatch][kFN], fa[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = (first + h + b) * kStep + (4 * c + g) * 16;
          const bool in = at < p.kbytes;
          fa[b].c[c] = u32x4{0, 0, 0, 0};
          if (in) fa[b].c[c] = *reinterpret_cast<const u32x4*>(pa + at);
#pragma unroll
          for (int j = 0; j < kFN; ++j) {
            fw[b][j].c[c] = u32x4{0, 0, 0, 0};
            if (in) fw[b][j].c[c] = *reinterpret_cast<const u32x4*>(pw[j] + at);
          }
        }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        // the scales of the blocks of chunks g and 4 + g
        auto pair = [&](const u32x4& d, uint32_t* v) {
          v[0] = is_block8(kKind) ? d[h + b] >> (8 * (g / 2)) : kUnit;
          v[1] = is_block8(kKind) ? d[h + b] >> (8 * (2 + g / 2)) : kUnit;
        };
        uint32_t v[2];
        Prepared<kKind, 0> qa, qw[kFN];
        pair(da, v);
        qa.set(fa[b], v);
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          pair(dw[j], v);
          qw[j].set(fw[b][j], v);
        }
#pragma unroll
        for (int u = 0; u < kSubs<kKind>; ++u)
#pragma unroll
          for (int j = 0; j < kFN; ++j) acc[j] = mma<kKind, 0>(qw[j], qa, u, acc[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kFN; ++j) *reinterpret_cast<f32x4*>(&part[wave][i16][j * 16 + 4 * g]) = acc[j];
  __syncthreads();

  // four outputs per thread: consecutive threads hold consecutive columns, so a
  // block of 32 columns is 8 neighbouring lanes
  constexpr int kQuads = kCols / 4;
  for (int e = threadIdx.x; e < 16 * kQuads; e += 64 * kWaves) {
    const int r = e / kQuads, c = (e % kQuads) * 4;
    f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll 4
    for (int w = 0; w < kWaves; ++w) {
      v += *reinterpret_cast<const f32x4*>(&part[w][r][c]);
      if constexpr (kGated) u += *reinterpret_cast<const f32x4*>(&part[w][r][kCols + c]);
    }
    const int64_t m = r;
    const int32_t n = n0 + c;
    const bool in = m < p.M && n < p.N;
    float gv[4] = {v.x, v.y, v.z, v.w}, uv[4] = {u.x, u.y, u.z, u.w};
    const int64_t mr = m < p.M ? m : (int64_t)p.M - 1;
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

}  // namespace
}  // namespace nvfp4
