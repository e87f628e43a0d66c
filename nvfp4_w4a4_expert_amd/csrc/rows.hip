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
#include "internal.h"
#include "rows_device.h"

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
    const float inv = row_inverse<kThreads, kVec>(s, p.K, p.eps, s_sum, s_max);
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
    store_row_fp8<kFp8, kThreads, kVec>(s, row, p.K, lane, p.codes, p.scales, s_max);
  }
}

template <bool kF16, bool kNorm, int kFp8>
hipError_t launch(const RowParams& p, hipStream_t stream) {
  return with_row_group(p.K / 8, [&](auto threads, auto vecs) {
    return launch_row_groups(rows_kernel<kF16, kNorm, kFp8, threads.value, vecs.value>, threads.value, p, stream);
  });
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
