// Device code that the row operators share (rows.hip, block.hip): a row's 16-byte
// vectors, its sums and maxima, its RMS norm and its 8-bit form.  A group of kThreads
// threads holds a row of at most 8 * kThreads * kVec elements in registers.
#pragma once

#include <type_traits>

#include "fp8_device.h"

namespace nvfp4 {
namespace {

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

// 1 / sqrt(mean(s^2) + eps) of a row, for s as it is on return: a row whose squares
// leave fp32's range comes back divided by a power of two, with the inverse of that.
template <int kThreads, int kVec>
__device__ __forceinline__ float row_inverse(float (*s)[8], int32_t K, float eps, float* s_sum, uint32_t* s_max) {
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq += s[i][j] * s[i][j];
  sq = group_reduce<kThreads>(sq, s_sum, [](float a, float b) { return a + b; });
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
  return 1.0f / sqrtf(sq / (float)K + eps);
}

// The row's E4M3 codes and scale or scales, from its fp32 values.
template <int kFp8, int kThreads, int kVec>
__device__ __forceinline__ void store_row_fp8(const float (*s)[8], int64_t row, int32_t K, int lane, uint8_t* codes, void* scales,
                                              uint32_t* s_max) {
  const int nvec = K / 8;
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
    if (lane == 0) static_cast<float*>(scales)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    if constexpr (kFp8 == kFp8Block) {
      // K % 32 == 0: the four lanes of a block are inside or outside together
      const uint32_t c = block_scale_code(quad_max(top[i]), inv);
      if (v < nvec && (lane & 3) == 0) static_cast<uint8_t*>(scales)[row * (K / 32) + v / 4] = (uint8_t)c;
    }
    if (v < nvec) {
      uint2 d;
      d.x = encode4_e4m3(s[i], inv);
      d.y = encode4_e4m3(s[i] + 4, inv);
      *reinterpret_cast<uint2*>(codes + row * K + 8 * v) = d;
    }
  }
}

template <int V>
using Count = std::integral_constant<int, V>;

// Runs go(threads, vectors), integral constants, with the group that a row of nvec
// vectors gets.
template <class Go>
hipError_t with_row_group(int nvec, Go go) {
  // One 16-byte vector per thread up to 2048 elements: the row's loads are all in
  // flight at once and its reduction crosses the fewest wavefronts.  Measured as
  // threads x vectors (norm with residual, all outputs, about 23 M elements / 16
  // rows, on one set of tensors, partly in the last-level cache), us: 256: 32x1 15.0
  // / 3.2, 64x1 19.6 / 3.2; 704: 128x1 33.9 / 3.3, 64x2 35.6 / 3.9; 2048: 256x1 30.9 / 3.3, 128x2 31.3 / 3.9; 2816: 256x2 32.2 / 4.0,
  // 512x1 32.9 / 3.6; 8192: 512x2 32.1 / 4.5, 256x4 33.4 / 5.3.
  if (nvec <= 16) return go(Count<16>{}, Count<1>{});
  if (nvec <= 32) return go(Count<32>{}, Count<1>{});
  if (nvec <= 64) return go(Count<64>{}, Count<1>{});
  if (nvec <= 128) return go(Count<128>{}, Count<1>{});
  if (nvec <= 256) return go(Count<256>{}, Count<1>{});
  if (nvec <= 512) return go(Count<256>{}, Count<2>{});
  if (nvec <= 1024) return go(Count<512>{}, Count<2>{});
  if (nvec <= 2048) return go(Count<1024>{}, Count<2>{});
  return go(Count<1024>{}, Count<4>{});
}

// Launches kernel(p), p.first the first row of each part: a launch holds at most
// 2^32 - 1 threads, so more rows than that go in parts.
template <class P, class Kernel>
hipError_t launch_row_groups(Kernel kernel, int threads, const P& p, hipStream_t stream) {
  const int per = threads <= 64 ? 256 / threads : 1;
  const int block = threads <= 64 ? 256 : threads;
  constexpr int32_t kPart = 1 << 21;
  for (int32_t first = 0; first < p.rows; first += kPart) {
    P q = p;
    q.first = first;
    const int32_t rows = p.rows - first < kPart ? p.rows - first : kPart;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((rows + per - 1) / per)), dim3(block), 0, stream, q);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.rows - first <= kPart) return err;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace nvfp4
