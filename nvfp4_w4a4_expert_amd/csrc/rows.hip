// Row operators of the dense half for gfx950: the RMS norm with the residual's
// addition, written in x's type and/or in 8 bits, and the same 8-bit forms of
// given rows.
//
//   s = rnd(x + r);  y = s * (1 / sqrt(mean(s^2) + eps)) * (offset + weight)
//
// s is rounded to x's type when a residual is given (it is the new residual
// stream, and the norm belongs to what is stored); y and the sums stay in fp32
// and each output is rounded once (the 8-bit codes from the fp32 y, not from a
// rounded one).
//
// One group of kThreads threads owns a row and holds it in registers, 8
// elements per 16-byte load, so every input is read once and every output
// written once whatever combination of outputs is asked for.  Bound by memory:
// 8192 rows of 2816 with residual and all outputs (208 MB) take 37 us on ten sets of
// tensors in turn (5.6 TB/s; a copy of that size, in turn as well, 39 to 42), and 28 to
// 35 on one set, most of which the last-level cache still holds from the call before;
// 16 rows take 4 us, a launch.
#include "fp8_device.h"
#include "internal.h"

namespace nvfp4 {
namespace {

struct RowParams {
  const uint16_t* x;
  const uint16_t* r;        // residual or null
  const uint16_t* w;        // norm weight or null (1)
  uint16_t* sum;            // [rows, lds] or null
  uint16_t* y;              // [rows, ldy] or null
  uint8_t* codes;           // [rows, K] or null
  void* scales;             // fp32 [rows] or uint8 [rows, K/32]
  int64_t ldx, ldr, lds, ldy;
  int32_t first, rows, K;   // the launch's first row; rows of the tensors
  float offset, eps;
};

// Below this sum of squares a row may have lost some to underflow (each is off by at
// most 2^-150), and with an eps below that other bound it shows.
constexpr float kTinySum = 0x1p-100f, kTinyEps = 0x1p-70f;

enum { kFp8None = 0, kFp8Row = 1, kFp8Block = 2 };

template <bool kF16>
__device__ __forceinline__ void unpack8(const u32x4& v, float* f) {
  if constexpr (kF16) unpack_f16x8(v, f);
  else unpack_bf16x8(v, f);
}

template <bool kF16>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = kF16 ? pack_f16(f[2 * i], f[2 * i + 1]) : pack_bf16(f[2 * i], f[2 * i + 1]);
  return v;
}

// Sum / maximum over the kThreads threads of a row's group, in a fixed order.
template <int kThreads, class F, class T>
__device__ __forceinline__ T group_reduce(T v, T* s_part, F f) {
  constexpr int kLanes = kThreads < 64 ? kThreads : 64;
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) v = f(v, (T)__shfl_xor(v, off, 64));
  if constexpr (kThreads > 64) {
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s_part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) v = f(v, s_part[i]);
  }
  return v;
}

// kThreads threads per row, kVec 16-byte vectors per thread (K <= 8 * kThreads
// * kVec); groups of at most a wavefront share a workgroup of 256 threads.
template <bool kF16, bool kNorm, int kFp8, int kThreads, int kVec>
__global__ __launch_bounds__(kThreads > 256 ? kThreads : 256) void rows_kernel(const RowParams p) {
  constexpr int kPer = kThreads <= 64 ? 256 / kThreads : 1;          // rows per workgroup
  __shared__ float s_sum[kThreads / 64 + 1];
  __shared__ uint32_t s_max[kThreads / 64 + 1];
  const int lane = kPer > 1 ? (int)(threadIdx.x % kThreads) : (int)threadIdx.x;
  const int64_t row = p.first + (int64_t)blockIdx.x * kPer + (kPer > 1 ? threadIdx.x / kThreads : 0);
  if (row >= p.rows) return;                                          // whole groups only
  const int nvec = p.K / 8;

  float s[kVec][8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    u32x4 d = {0, 0, 0, 0};
    if (v < nvec) d = *reinterpret_cast<const u32x4*>(p.x + row * p.ldx + 8 * v);
    unpack8<kF16>(d, s[i]);
  }
  if (kNorm && p.r) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = lane + i * kThreads;
      if (v < nvec) {
        float r[8];
        unpack8<kF16>(*reinterpret_cast<const u32x4*>(p.r + row * p.ldr + 8 * v), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] += s[i][j];
        const u32x4 d = pack8<kF16>(r);
        unpack8<kF16>(d, s[i]);
        if (p.sum) *reinterpret_cast<u32x4*>(p.sum + row * p.lds + 8 * v) = d;
      }
    }
  }
  if constexpr (kNorm) {
    float w[kVec][8];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = lane + i * kThreads;
      u32x4 d = {0, 0, 0, 0};
      if (p.w && v < nvec) d = *reinterpret_cast<const u32x4*>(p.w + 8 * v);
      unpack8<kF16>(d, w[i]);
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq += s[i][j] * s[i][j];
    sq = group_reduce<kThreads>(sq, s_sum, [](float a, float b) { return a + b; });
    float eps = p.eps;
    if (!(sq < INFINITY) || (sq < kTinySum && eps < kTinyEps)) {
      // The squares left fp32's range (the same for all threads of the row): once more
      // on s / 2^e, e the exponent of its largest finite element.  e stays above -96,
      // where the squares of the smallest bf16 numbers and eps are both in range.  The
      // test costs ordinary rows under 0.1 us (2 to 3 % from 16384 elements on).
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, finite_mag(s[i][j]));
      top = group_reduce<kThreads>(top, s_max, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const int e = max((int)(top >> 23) - 127, -96);
      sq = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[i][j] = __builtin_ldexpf(s[i][j], -e);
          sq += s[i][j] * s[i][j];
        }
      sq = group_reduce<kThreads>(sq, s_sum, [](float a, float b) { return a + b; });
      eps = __builtin_ldexpf(eps, -2 * e);
    }
    const float inv = 1.0f / sqrtf(sq / (float)p.K + eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = p.w ? p.offset + w[i][j] : 1.0f;
        s[i][j] = (s[i][j] * inv) * g;
      }
    if (p.y) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int v = lane + i * kThreads;
        if (v < nvec) *reinterpret_cast<u32x4*>(p.y + row * p.ldy + 8 * v) = pack8<kF16>(s[i]);
      }
    }
  }
  if constexpr (kFp8 != kFp8None) {
    uint32_t top[kVec], all = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      top[i] = 0;
      const bool in = lane + i * kThreads < nvec;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = in ? finite_mag(s[i][j]) : 0u;
        top[i] = m > top[i] ? m : top[i];
      }
      all = top[i] > all ? top[i] : all;
    }
    float inv = 0.0f;
    if constexpr (kFp8 == kFp8Row) {
      all = group_reduce<kThreads>(all, s_max, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const float scale = row_scale(all, inv);
      if (lane == 0) static_cast<float*>(p.scales)[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = lane + i * kThreads;
      if constexpr (kFp8 == kFp8Block) {
        // K % 32 == 0: the four lanes of a block are inside or outside together
        const uint32_t c = block_scale_code(quad_max(top[i]), inv);
        if (v < nvec && (lane & 3) == 0) static_cast<uint8_t*>(p.scales)[row * (p.K / 32) + v / 4] = (uint8_t)c;
      }
      if (v < nvec) {
        uint2 d;
        d.x = encode4_e4m3(s[i], inv);
        d.y = encode4_e4m3(s[i] + 4, inv);
        *reinterpret_cast<uint2*>(p.codes + row * p.K + 8 * v) = d;
      }
    }
  }
}

template <bool kF16, bool kNorm, int kFp8>
hipError_t launch(const RowParams& p, hipStream_t stream) {
  const int nvec = p.K / 8;
  auto go = [&](auto kernel, int threads) {
    const int per = threads <= 64 ? 256 / threads : 1;
    const int block = threads <= 64 ? 256 : threads;
    // a launch holds at most 2^32 - 1 threads: more rows than that go in parts
    constexpr int32_t kPart = 1 << 21;
    for (int32_t first = 0; first < p.rows; first += kPart) {
      RowParams q = p;
      q.first = first;
      const int32_t rows = p.rows - first < kPart ? p.rows - first : kPart;
      hipLaunchKernelGGL(kernel, dim3((uint32_t)((rows + per - 1) / per)), dim3(block), 0, stream, q);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess || p.rows - first <= kPart) return err;
    }
    return hipSuccess;
  };
  // One 16-byte vector per thread up to 2048 elements: the row's loads are all in
  // flight at once and its reduction crosses the fewest wavefronts.  Measured as
  // threads x vectors (norm with residual, all outputs, about 23 M elements / 16
  // rows, on one set of tensors, partly in the last-level cache), us:       256: 32x1 15.0 / 3.2, 64x1 19.6 / 3.2;   704: 128x1 33.9 / 3.3,
  // 64x2 35.6 / 3.9; 2048: 256x1 30.9 / 3.3, 128x2 31.3 / 3.9; 2816: 256x2 32.2 / 4.0,
  // 512x1 32.9 / 3.6; 8192: 512x2 32.1 / 4.5, 256x4 33.4 / 5.3.
  if (nvec <= 16) return go(rows_kernel<kF16, kNorm, kFp8, 16, 1>, 16);
  if (nvec <= 32) return go(rows_kernel<kF16, kNorm, kFp8, 32, 1>, 32);
  if (nvec <= 64) return go(rows_kernel<kF16, kNorm, kFp8, 64, 1>, 64);
  if (nvec <= 128) return go(rows_kernel<kF16, kNorm, kFp8, 128, 1>, 128);
  if (nvec <= 256) return go(rows_kernel<kF16, kNorm, kFp8, 256, 1>, 256);
  if (nvec <= 512) return go(rows_kernel<kF16, kNorm, kFp8, 256, 2>, 256);
  if (nvec <= 1024) return go(rows_kernel<kF16, kNorm, kFp8, 512, 2>, 512);
  if (nvec <= 2048) return go(rows_kernel<kF16, kNorm, kFp8, 1024, 2>, 1024);
  return go(rows_kernel<kF16, kNorm, kFp8, 1024, 4>, 1024);
}

template <bool kF16, bool kNorm>
hipError_t launch_fp8(const RowParams& p, int fp8, hipStream_t stream) {
  if (fp8 == kFp8Row) return launch<kF16, kNorm, kFp8Row>(p, stream);
  if (fp8 == kFp8Block) return launch<kF16, kNorm, kFp8Block>(p, stream);
  if constexpr (kNorm) return launch<kF16, kNorm, kFp8None>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows(const RowArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.K < 8 || a.K % 8 || a.K > kRowsMaxK) return hipErrorInvalidValue;
  RowParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.r = static_cast<const uint16_t*>(a.residual);
  p.w = static_cast<const uint16_t*>(a.weight);
  p.sum = static_cast<uint16_t*>(a.sum_out);
  p.y = static_cast<uint16_t*>(a.y_out);
  p.codes = a.codes;
  p.scales = a.scales;
  p.ldx = a.ldx; p.ldr = a.ldr; p.lds = a.lds; p.ldy = a.ldy;
  p.first = 0; p.rows = a.rows; p.K = a.K;
  p.offset = a.offset; p.eps = a.eps;
  if (a.fp16) return a.norm ? launch_fp8<true, true>(p, a.fp8, stream) : launch_fp8<true, false>(p, a.fp8, stream);
  return a.norm ? launch_fp8<false, true>(p, a.fp8, stream) : launch_fp8<false, false>(p, a.fp8, stream);
}

}  // namespace nvfp4
