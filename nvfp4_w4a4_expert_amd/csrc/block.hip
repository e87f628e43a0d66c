// The end of one block and the start of the next for gfx950: the block's last norm,
// its gate, the residual stream's addition and the next block's first norm, in one
// pass over the rows.
//
//   b = x * (1 / sqrt(mean(x^2) + eps)) * (offset + post_weight), or x
//   t = rnd(residual_scale * residual + gate * b)
//   y = t * (1 / sqrt(mean(t^2) + eps)) * (offset + weight), in x's type and/or 8 bits
//
// b and the gate stay in fp32, t is rounded to x's type (it is the new residual
// stream, and the second norm belongs to what is stored), y is rounded once (the
// 8-bit codes from the fp32 y).  gate is a number times, or not, a tensor of one
// element a row, one a column or one an element, through a sigmoid or a tanh or not.
//
// A group of threads holds its row in registers from the first load to the last
// store, so x and the residual are read once and each output written once, with two
// reductions over the group between them; as separate operators the same rows would
// be read twice more and written once more.  8192 x 2816 with y and 8-bit output (208 MB)
// take 42.3 us on sets of tensors in turn (4.9 TB/s, the rate of a large copy; the norm,
// with half the arithmetic, 37), 16 rows 4.2, a launch.
#include "internal.h"
#include "rows_device.h"

namespace nvfp4 {
namespace {

struct BlockParams {
  const uint16_t* x;
  const uint16_t* r;
  const uint16_t* w_post;   // or null (1)
  const uint16_t* w;        // or null (1)
  const void* gate;         // or null (1): [rows or 1, K or 1] by its strides
  uint16_t* total;
  uint16_t* y;              // or null
  uint8_t* codes;           // or null
  void* scales;
  int64_t ldx, ldr, ldg, ldt, ldy;
  int32_t first, rows, K;
  int32_t post, gate_wide, gate_f32, gate_act;
  float offset, eps, gate_scale, residual_scale;
};

enum { kGatePlain = 0, kGateSigmoid = 1, kGateTanh = 2 };

__device__ __forceinline__ float gate_value(float v, int32_t act) {
  if (act == kGateSigmoid) return 1.0f / (1.0f + expf(-v));
  if (act == kGateTanh) return tanhf(v);
  return v;
}

template <bool kF16>
__device__ __forceinline__ float gate_elem(const BlockParams& p, int64_t at) {
  if (p.gate_f32) return static_cast<const float*>(p.gate)[at];
  const uint16_t u = static_cast<const uint16_t*>(p.gate)[at];
  return kF16 ? (float)__builtin_bit_cast(_Float16, u) : __uint_as_float((uint32_t)u << 16);
}

// v * inv * (offset + w), or without the weight.
template <bool kF16>
__device__ __forceinline__ void normed8(float* v, float inv, const uint16_t* w, const u32x4& d, float offset) {
  if (w) {
    float f[8];
    unpack8<kF16>(d, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (v[j] * inv) * (offset + f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
  }
}

// The row's E4M3 codes and scale or scales, from its fp32 values.  Ordinary rows and
// blocks, all of whose values are finite, need no look at each value: their products with
// the scale's inverse are 448 at most, or a step beyond it, which rounds to 448.
template <int kFp8, int kThreads, int kVec>
__device__ __forceinline__ void store_finite_fp8(const float (*s)[8], int64_t row, int32_t K, int lane, uint8_t* codes, void* scales,
                                              uint32_t* s_max) {
  const int nvec = K / 8;
  auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  auto largest = [&](int i, bool finite_only) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = most(top, finite_only ? finite_mag(s[i][j]) : __float_as_uint(s[i][j]) & 0x7FFFFFFFu);
    return lane + i * kThreads < nvec ? top : 0u;
  };
  float inv = 0.0f;
  bool finite = true;
  if constexpr (kFp8 == kFp8Row) {
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) all = most(all, largest(i, false));
    all = group_reduce<kThreads>(all, s_max, most);
    finite = all < 0x7F800000u;
    if (!finite) {                                               // (for the whole group)
      all = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) all = most(all, largest(i, true));
      if constexpr (kThreads > 64) __syncthreads();              // (the first maxima have been read)
      all = group_reduce<kThreads>(all, s_max, most);
    }
    const float scale = row_scale(all, inv);
    if (lane == 0) static_cast<float*>(scales)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    if constexpr (kFp8 == kFp8Block) {
      // K % 32 == 0: the four lanes of a block are inside or outside together
      uint32_t top = quad_max(largest(i, false));
      finite = __all(top < 0x7F800000u);                         // (one branch for the wavefront)
      if (!finite) top = quad_max(largest(i, true));
      const uint32_t c = block_scale_code(top, inv);
      if (v < nvec && (lane & 3) == 0) static_cast<uint8_t*>(scales)[row * (K / 32) + v / 4] = (uint8_t)c;
    }
    if (v < nvec) {
      uint2 d;
      if (finite) {
        d.x = encode4_scaled(s[i], inv);
        d.y = encode4_scaled(s[i] + 4, inv);
      } else {
        d.x = encode4_e4m3(s[i], inv);
        d.y = encode4_e4m3(s[i] + 4, inv);
      }
      *reinterpret_cast<uint2*>(codes + row * K + 8 * v) = d;
    }
  }
}

template <bool kF16, int kFp8, int kThreads, int kVec>
__global__ __launch_bounds__(kThreads > 256 ? kThreads : 256) void block_kernel(const BlockParams p) {
  constexpr int kPer = kThreads <= 64 ? 256 / kThreads : 1;          // rows per workgroup
  // (a pair for each norm: a wavefront may still read the first while another writes
  // the second)
  __shared__ float s_sum[2][kThreads / 64 + 1];
  __shared__ uint32_t s_max[2][kThreads / 64 + 1];
  const int lane = kPer > 1 ? (int)(threadIdx.x % kThreads) : (int)threadIdx.x;
  const int64_t row = p.first + (int64_t)blockIdx.x * kPer + (kPer > 1 ? threadIdx.x / kThreads : 0);
  if (row >= p.rows) return;                                          // whole groups only
  const int nvec = p.K / 8;

  const u32x4 none = {0, 0, 0, 0};
  u32x4 r[kVec], wp[kVec];
  float s[kVec][8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    u32x4 d = none;
    r[i] = wp[i] = none;
    if (v < nvec) {
      d = *reinterpret_cast<const u32x4*>(p.x + row * p.ldx + 8 * v);
      r[i] = *reinterpret_cast<const u32x4*>(p.r + row * p.ldr + 8 * v);
      if (p.w_post) wp[i] = *reinterpret_cast<const u32x4*>(p.w_post + 8 * v);
    }
    unpack8<kF16>(d, s[i]);
  }
  float one = p.gate_scale;                                           // a gate that the row shares
  if (p.gate && !p.gate_wide) one *= gate_value(gate_elem<kF16>(p, row * p.ldg), p.gate_act);
  if (p.post) {
    const float inv = row_inverse<kThreads, kVec>(s, p.K, p.eps, s_sum[0], s_max[0]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) normed8<kF16>(s[i], inv, p.w_post, wp[i], p.offset);
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    float h[8];
    unpack8<kF16>(r[i], h);
    if (p.gate_wide && v < nvec) {
      float e[8];
      const int64_t at = row * p.ldg + 8 * v;
      if (p.gate_f32) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.gate) + at);
        const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.gate) + at + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = a[j];
          e[4 + j] = b[j];
        }
      } else {
        unpack8<kF16>(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.gate) + at), e);
      }
      if (p.gate_act != kGatePlain) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = gate_value(e[j], p.gate_act);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = __builtin_fmaf(one * e[j], s[i][j], p.residual_scale * h[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = __builtin_fmaf(one, s[i][j], p.residual_scale * h[j]);
    }
    const u32x4 d = pack8<kF16>(h);
    // (past the row's end x and the residual read as zeros, which a gate may make NaN)
    unpack8<kF16>(v < nvec ? d : none, s[i]);
    if (v < nvec && p.total) *reinterpret_cast<u32x4*>(p.total + row * p.ldt + 8 * v) = d;
  }
  if (kFp8 == kFp8None && !p.y) return;
  u32x4 w[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    w[i] = none;
    if (p.w && v < nvec) w[i] = *reinterpret_cast<const u32x4*>(p.w + 8 * v);
  }
  const float inv = row_inverse<kThreads, kVec>(s, p.K, p.eps, s_sum[1], s_max[1]);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = lane + i * kThreads;
    normed8<kF16>(s[i], inv, p.w, w[i], p.offset);
    if (p.y && v < nvec) *reinterpret_cast<u32x4*>(p.y + row * p.ldy + 8 * v) = pack8<kF16>(s[i]);
  }
  if constexpr (kFp8 != kFp8None) store_finite_fp8<kFp8, kThreads, kVec>(s, row, p.K, lane, p.codes, p.scales, s_max[1]);
}

template <bool kF16, int kFp8>
hipError_t launch(const BlockParams& p, hipStream_t stream) {
  const int nvec = p.K / 8;
  auto go = [&](auto threads, auto vecs) {
    return launch_row_groups(block_kernel<kF16, kFp8, threads.value, vecs.value>, threads.value, p, stream);
  };
  // Groups as the norm's but for rows between two groups of the norm: bound by the instructions
  // that it issues, and with two vectors a thread of 256 half a wavefront's are empty at 2816
  // (8192 rows: 256x2 43.9 us, 128x3 42.3, 512x1 54.9; 16 rows 4.8, 5.4, 4.2).
  if (nvec > 256 && nvec <= 512 && p.rows <= 512) return go(Count<512>{}, Count<1>{});
  if (nvec > 256 && nvec <= 384) return go(Count<128>{}, Count<3>{});
  return with_row_group(nvec, go);
}

template <bool kF16>
hipError_t launch_fp8(const BlockParams& p, int fp8, hipStream_t stream) {
  if (fp8 == kFp8Row) return launch<kF16, kFp8Row>(p, stream);
  if (fp8 == kFp8Block) return launch<kF16, kFp8Block>(p, stream);
  return launch<kF16, kFp8None>(p, stream);
}

}  // namespace

hipError_t launch_block(const BlockArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.K < 8 || a.K % 8 || a.K > kRowsMaxK) return hipErrorInvalidValue;
  BlockParams p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.r = static_cast<const uint16_t*>(a.residual);
  p.w_post = static_cast<const uint16_t*>(a.post_weight);
  p.w = static_cast<const uint16_t*>(a.weight);
  p.gate = a.gate;
  p.total = static_cast<uint16_t*>(a.total_out);
  p.y = static_cast<uint16_t*>(a.y_out);
  p.codes = a.codes;
  p.scales = a.scales;
  p.ldx = a.ldx; p.ldr = a.ldr; p.ldg = a.ldg; p.ldt = a.ldt; p.ldy = a.ldy;
  p.rows = a.rows; p.K = a.K;
  p.post = a.post; p.gate_wide = a.gate && a.gate_wide; p.gate_f32 = a.gate_f32; p.gate_act = a.gate_act;
  p.offset = a.offset; p.eps = a.eps; p.gate_scale = a.gate_scale; p.residual_scale = a.residual_scale;
  return a.fp16 ? launch_fp8<true>(p, a.fp8, stream) : launch_fp8<false>(p, a.fp8, stream);
}

}  // namespace nvfp4
