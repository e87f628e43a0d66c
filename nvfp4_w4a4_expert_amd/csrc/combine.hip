// Unpermute + top-k weighted combine (page 3, "矩阵融合" pipeline figure:
// restore token order and sum by routing weight).
//
// out[t, :] = bf16( residual[t, :] + sum_{j<k} w[t, j] * C2[inv[t*k + j], :] )
// with the sum taken in fp32, j ascending, and one rounding to bf16 at the
// end.  A gather (each token reads its k rows), not a scatter-add, so the
// result is deterministic.  One thread produces 4 consecutive outputs: one
// 16-byte load per source row and one 8-byte store (measured at 4096 tokens,
// top-8, hidden 2816 with the routed permutation: 78.3 -> 68.2 us against 8
// outputs per thread).  HBM-bound.
#include "fp8_device.h"
#include "internal.h"

namespace nvfp4 {

__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ c2,
                                                      const float* __restrict__ w,
                                                      const int32_t* __restrict__ inv, int32_t T,
                                                      int32_t k, int32_t H,
                                                      const uint16_t* residual, uint16_t* out) {
  const int32_t h4 = H / 4;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (g >= (int64_t)T * h4) return;
  const int32_t t = (int32_t)(g / h4);
  const int32_t c = (int32_t)(g - (int64_t)t * h4) * 4;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  // Slots in groups of kU: the group's row indices first, then all its row
  // loads, then the sums in slot order (slots past k re-read row k-1 and are
  // not added), so each thread keeps kU loads in flight instead of a chain
  // of index load -> row load per slot.
  constexpr int kU = 8;
  const int64_t q0 = (int64_t)t * k;
  for (int32_t j0 = 0; j0 < k; j0 += kU) {
    int32_t row[kU];
    float wj[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int32_t j = min(j0 + u, k - 1);
      row[u] = inv[q0 + j];
      wj[u] = w[q0 + j];
    }
    f32x4 a[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      a[u] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(c2 + (int64_t)row[u] * H + c));
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (j0 + u < k) {
        acc[0] += wj[u] * a[u].x; acc[1] += wj[u] * a[u].y;
        acc[2] += wj[u] * a[u].z; acc[3] += wj[u] * a[u].w;
      }
    }
  }
  if (residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(residual + (int64_t)t * H + c);
    acc[0] += bf16_lo(r.x); acc[1] += bf16_hi(r.x);
    acc[2] += bf16_lo(r.y); acc[3] += bf16_hi(r.y);
  }
  uint2 o;
  o.x = f32_to_bf16(acc[0]) | (f32_to_bf16(acc[1]) << 16);
  o.y = f32_to_bf16(acc[2]) | (f32_to_bf16(acc[3]) << 16);
  *reinterpret_cast<uint2*>(out + (int64_t)t * H + c) = o;
}

// The same sum as an operator of its own: values, residual and result of any of the
// three float types, rows with strides, pairs without a row left out.  A thread owns 8
// consecutive outputs, so a 16-bit row is read 16 bytes at a time.
namespace {

struct CombineParams {
  const void* v;
  const float* w;
  const int32_t* inv;
  const void* r;            // or null
  void* out;
  int64_t ldv, ldr, ldo;
  int64_t first, last;      // this launch's vectors of 8 outputs
  int32_t rows, k, vecs;    // rows of v; vectors per token
  int32_t r_type, out_type;
};

// 8 consecutive elements of a tensor of type 0 bf16, 1 fp16, 2 fp32, as they were
// loaded (fp32: both halves)
struct Raw8 {
  u32x4 d[2];
};
template <bool kStream>
__device__ __forceinline__ Raw8 load8(const void* base, int64_t at, int32_t type) {
  const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + at * (type == 2 ? 4 : 2));
  Raw8 x;
  x.d[0] = kStream ? __builtin_nontemporal_load(src) : *src;
  x.d[1] = u32x4{0, 0, 0, 0};
  if (type == 2) x.d[1] = kStream ? __builtin_nontemporal_load(src + 1) : src[1];
  return x;
}
__device__ __forceinline__ void floats8(const Raw8& x, int32_t type, float* f) {
  if (type == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(x.d[i / 4][i % 4]);
  } else if (type == 1) {
    unpack_f16x8(x.d[0], f);
  } else {
    unpack_bf16x8(x.d[0], f);
  }
}

template <int kType>
__global__ __launch_bounds__(256) void combine_rows_kernel(const CombineParams p) {
  const int64_t g = p.first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= p.last) return;
  const int64_t t = g <= 0xFFFFFFFFll ? (int64_t)((uint32_t)g / (uint32_t)p.vecs) : g / p.vecs;
  const int64_t c = (g - t * p.vecs) * 8;
  Raw8 res = {};
  if (p.r) res = load8<false>(p.r, t * p.ldr + c, p.r_type);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kU = kType == 2 ? 4 : 8;                        // rows whose loads are in flight together
  const int64_t q0 = t * p.k;
  for (int32_t j0 = 0; j0 < p.k && p.rows > 0; j0 += kU) {
    int32_t row[kU];
    float wj[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int32_t j = min(j0 + u, p.k - 1);
      row[u] = p.inv[q0 + j];
      wj[u] = p.w[q0 + j];
    }
    Raw8 a[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int32_t at = (uint32_t)row[u] < (uint32_t)p.rows ? row[u] : 0;
      a[u] = load8<true>(p.v, at * p.ldv + c, kType);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (j0 + u < p.k && (uint32_t)row[u] < (uint32_t)p.rows) {
        float f[8];
        floats8(a[u], kType, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += wj[u] * f[i];
      }
    }
  }
  if (p.r) {
    float f[8];
    floats8(res, p.r_type, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += f[i];
  }
  if (p.out_type == 2) {
    f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + t * p.ldo + c);
    dst[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    dst[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
  } else {
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = p.out_type == 1 ? pack_f16(acc[2 * i], acc[2 * i + 1]) : pack_bf16(acc[2 * i], acc[2 * i + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + t * p.ldo + c) = d;
  }
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t stream) {
  CombineParams p = {};
  p.v = a.values; p.w = a.weights; p.inv = a.inv; p.r = a.residual; p.out = a.out;
  p.ldv = a.ldv; p.ldr = a.ldr; p.ldo = a.ldo;
  p.rows = a.rows; p.k = a.k; p.vecs = a.H / 8;
  p.r_type = a.residual_type; p.out_type = a.out_type;
  const int64_t total = (int64_t)a.T * p.vecs;
  constexpr int64_t kPart = (int64_t)1 << 31;                   // (a launch holds at most 2^32 - 1 threads)
  for (p.first = 0; p.first < total; p.first += kPart) {
    p.last = total - p.first < kPart ? total : p.first + kPart;
    const dim3 grid((uint32_t)((p.last - p.first + 255) / 256));
    if (a.type == 2) hipLaunchKernelGGL((combine_rows_kernel<2>), grid, dim3(256), 0, stream, p);
    else if (a.type == 1) hipLaunchKernelGGL((combine_rows_kernel<1>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((combine_rows_kernel<0>), grid, dim3(256), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_combine(const float* c2, const float* w, const int32_t* inv, int32_t T,
                          int32_t k, int32_t H, const uint16_t* residual, uint16_t* out,
                          hipStream_t stream) {
  const int64_t total = (int64_t)T * (H / 4);
  if (total == 0) return hipSuccess;
  hipLaunchKernelGGL(combine_kernel, dim3((uint32_t)((total + 255) / 256)), dim3(256), 0, stream,
                     c2, w, inv, T, k, H, residual, out);
  return hipGetLastError();
}

}  // namespace nvfp4
