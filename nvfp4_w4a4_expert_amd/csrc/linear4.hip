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
// Few rows (at most 64) are bound by reading w once and go from memory to registers:
// linear4_few_kernel.  More rows are bound by the matrix units: w is written out in 16
// bits once (4.5 bits read and 16 written an element) and the linear operator's tiles
// multiply it.
#include "internal.h"
#include "linear_kernels.h"

namespace nvfp4 {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// A lane's block scales of 32 elements: E4M3 codes in bytes 0 and 1, or a UE8M0 code in
// byte 0.  Element runs of 8 (t) as 16-bit numbers.
template <bool kMx, bool kHalf>
struct Scale4;
template <>
struct Scale4<false, false> {
  f32x2_t s;
  __device__ __forceinline__ void set(uint32_t c) { s = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false); }
  __device__ __forceinline__ u32x4 weights(uint32_t w, int t) const {
    const float v = t < 2 ? s.x : s.y;
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    // (the products are bf16 numbers: their upper halves)
    auto pair = [&](const f32x2_t& x) { return __builtin_amdgcn_perm(__float_as_uint(x.y * v), __float_as_uint(x.x * v), 0x07060302u); };
    return u32x4{pair(a), pair(b), pair(c), pair(d)};
  }
};
template <>
struct Scale4<false, true> {
  half2_t s;
  __device__ __forceinline__ void set(uint32_t c) { s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false); }
  __device__ __forceinline__ u32x4 weights(uint32_t w, int t) const {
    const half2_t v = t < 2 ? half2_t{s.x, s.x} : half2_t{s.y, s.y};
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * v),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * v),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * v),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * v)};
  }
};
template <bool kHalf>
struct Scale4<true, kHalf> {                                    // (bf16 weights for either a)
  float s;
  __device__ __forceinline__ void set(uint32_t c) { s = __uint_as_float((c & 0xFFu) << 23); }
  __device__ __forceinline__ u32x4 weights(uint32_t w, int) const {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
  }
};

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

// acc += w . a over 32 elements of K, w the row operand
template <bool kMx, bool kHalf>
__device__ __forceinline__ f32x4 mma4(const u32x4& w, const u32x4& a, f32x4 acc) {
  if constexpr (!kMx && kHalf)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w), __builtin_bit_cast(half8_t, a), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
}

// ---- few rows -------------------------------------------------------------------
// A workgroup owns 16 * kFN rows of w (gated: gate rows, then up rows) and 16 * kRF rows
// of a.  Its wavefronts take groups of 128 elements of K in turn, kBatch groups' loads in
// flight at once: a lane's 16 bytes of w are 32 elements of a row, the next 32 belong to
// the next group of 16 lanes, and the four matrix instructions of a group take 8
// elements of each (any order of K that both operands share).  The wavefronts' sums are
// added in order through LDS, 16 rows at a time.
template <bool kMx, bool kHalf, int kRF, int kFN, bool kGated>
__global__ __launch_bounds__(512) void linear4_few_kernel(const LinParams p) {
  constexpr int kWaves = 8, kRows = 16 * kFN, kCols = kGated ? kRows / 2 : kRows;
  constexpr int kBatch = kRF * kFN <= 2 ? 4 : kRF <= 2 ? 2 : 1;
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
  for (int first = kBatch * wave; first < groups; first += kBatch * kWaves) {
    u32x4 w[kBatch][kFN], a[kBatch][kRF][4];
    uint32_t s[kBatch][kFN];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      // past the end of a row codes, scales and a count as zeros
      const int32_t k = (first + b) * 128 + 32 * g;
      const bool in = k < K;
#pragma unroll
      for (int j = 0; j < kFN; ++j) {
        w[b][j] = u32x4{0, 0, 0, 0};
        s[b][j] = 0;
        if (in) {
          w[b][j] = *reinterpret_cast<const u32x4*>(pw[j] + k / 2);
          if constexpr (kMx) s[b][j] = sw[j][k / 32];
          else s[b][j] = *reinterpret_cast<const uint16_t*>(sw[j] + k / 16);
        }
      }
#pragma unroll
      for (int i = 0; i < kRF; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          a[b][i][t] = u32x4{0, 0, 0, 0};
          if (in) a[b][i][t] = *reinterpret_cast<const u32x4*>(pa[i] + 2 * k + 16 * t);
        }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      Scale4<kMx, kHalf> sc[kFN];
#pragma unroll
      for (int j = 0; j < kFN; ++j) sc[j].set(s[b][j]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4 wt[kFN];
#pragma unroll
        for (int j = 0; j < kFN; ++j) wt[j] = sc[j].weights(w[b][j][t], t);
#pragma unroll
        for (int i = 0; i < kRF; ++i) {
          if constexpr (kSplit) {
            u32x4 hi, lo;
            split_f16(a[b][i][t], hi, lo);
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], hi, acc[i][j]);
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], lo, acc[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mma4<kMx, kHalf>(wt[j], a[b][i][t], acc[i][j]);
          }
        }
      }
    }
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

// ---- many rows ------------------------------------------------------------------------
// w in 16 bits, dense rows of `copies` times K elements; a thread writes 32 elements.
template <bool kMx, bool kHalf>
__global__ __launch_bounds__(256) void widen4_kernel(const uint8_t* w, int64_t ldw, const uint8_t* scales, int64_t rows, int32_t K,
                                                     int32_t copies, uint16_t* out) {
  const int32_t vecs = K / 32;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= rows * vecs) return;
  const int64_t row = id / vecs;
  const int32_t v = (int32_t)(id - row * vecs);
  const u32x4 c = *reinterpret_cast<const u32x4*>(w + row * ldw + 16 * v);
  Scale4<kMx, kHalf> s;
  if constexpr (kMx) s.set(scales[row * vecs + v]);
  else s.set(*reinterpret_cast<const uint16_t*>(scales + 2 * (row * vecs + v)));
  u32x4 d[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) d[t] = s.weights(c[t], t);
  for (int32_t i = 0; i < copies; ++i) {
    u32x4* dst = reinterpret_cast<u32x4*>(out + (row * copies + i) * K + 32 * v);
#pragma unroll
    for (int t = 0; t < 4; ++t) dst[t] = d[t];
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
constexpr int32_t kFewRows = 64;

template <bool kMx, bool kHalf, int kRF, int kFN, bool kGated>
hipError_t go_few(LinParams p, hipStream_t stream) {
  const int32_t cols = kGated ? 8 * kFN : 16 * kFN;
  p.tiles_n = (p.N - 1) / cols + 1;
  const int32_t bands = (p.M - 1) / (16 * kRF) + 1;
  hipLaunchKernelGGL((linear4_few_kernel<kMx, kHalf, kRF, kFN, kGated>), dim3((uint32_t)bands * (uint32_t)p.tiles_n), dim3(512), 0, stream, p);
  return hipGetLastError();
}

template <bool kMx, bool kHalf, bool kGated>
hipError_t go_rows(const LinParams& p, hipStream_t stream) {
  constexpr int kFirst = kGated ? 2 : 1;                       // fragments of w for 16 outputs
  const bool block = p.out_type == kOutBlock8;                 // (32 outputs belong together)
  if (p.M <= 16) return block ? go_few<kMx, kHalf, 1, 2 * kFirst, kGated>(p, stream) : go_few<kMx, kHalf, 1, kFirst, kGated>(p, stream);
  if (p.M <= 32) return go_few<kMx, kHalf, 2, 2 * kFirst, kGated>(p, stream);
  return go_few<kMx, kHalf, 4, 2 * kFirst, kGated>(p, stream);
}

template <bool kMx, bool kHalf>
hipError_t go_gated(const LinParams& p, int32_t gated, hipStream_t stream) {
  return gated ? go_rows<kMx, kHalf, true>(p, stream) : go_rows<kMx, kHalf, false>(p, stream);
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
  if (a.M <= kFewRows || a.N == 0) return 0;
  const Wide q = wide_of(a);
  return q.rest_at + linear_workspace_bytes(q.a);
}

hipError_t launch_linear4(const Linear4Args& a, void* workspace, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const bool f16 = a.kind == kF16;
  if (a.M <= kFewRows) {
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
    if (a.mx) return f16 ? go_gated<true, true>(p, a.gated, stream) : go_gated<true, false>(p, a.gated, stream);
    return f16 ? go_gated<false, true>(p, a.gated, stream) : go_gated<false, false>(p, a.gated, stream);
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
