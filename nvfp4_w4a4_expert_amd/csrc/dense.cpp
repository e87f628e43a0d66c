// C ABI of the dense operators around the routed experts: argument checking of
// nvfp4_rmsnorm, nvfp4_quantize_rows_fp8 and nvfp4_linear.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#define NVFP4_BUILDING_LIBRARY 1
#include "../../include/nvfp4_moe.h"
#include "internal.h"

namespace {

using namespace nvfp4;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

nvfp4_status_t device_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_DEVICE; }

// A row-major 16-bit tensor read and written in 16-byte vectors.
bool bad_rows(const void* p, int64_t ld, int32_t K) { return !aligned(p, 16) || ld < K || ld % 8; }

nvfp4_status_t check_fp8_out(int32_t fp8, int32_t K, const uint8_t* codes, const void* scales) {
  if (!codes || !scales || !aligned(codes, 8)) return NVFP4_ERR_INVALID_ARG;
  if (fp8 == NVFP4_TYPE_FP8_ROW && !aligned(scales, 4)) return NVFP4_ERR_INVALID_ARG;
  return NVFP4_OK;
}

bool is_float_type(int32_t t) { return t == NVFP4_TYPE_BF16 || t == NVFP4_TYPE_FP16 || t == NVFP4_TYPE_FP32; }
size_t float_size(int32_t t) { return t == NVFP4_TYPE_FP32 ? 4 : 2; }
bool is_fp8(int32_t t) { return t == NVFP4_TYPE_FP8_ROW || t == NVFP4_TYPE_FP8_MX; }

int32_t elem_type(int32_t t) {
  return t == NVFP4_TYPE_BF16 ? 0 : t == NVFP4_TYPE_FP16 ? 1 : t == NVFP4_TYPE_FP32 ? 2 : 3;
}

// Sizes and types alone (no pointer of *p is looked at), as nvfp4_linear_workspace_size
// and nvfp4_linear both need them.
nvfp4_status_t check_linear_sizes(const nvfp4_linear_t* p, LinearArgs* a) {
  if (!p || p->M < 0 || p->N < 0 || p->K < 1) return NVFP4_ERR_INVALID_ARG;
  if (p->type != NVFP4_TYPE_BF16 && p->type != NVFP4_TYPE_FP16 && !is_fp8(p->type)) return NVFP4_ERR_INVALID_ARG;
  if (p->K % (p->type == NVFP4_TYPE_FP8_MX ? 32 : is_fp8(p->type) ? 16 : 8)) return NVFP4_ERR_INVALID_ARG;
  if (p->act < NVFP4_ACT_NONE || p->act > NVFP4_ACT_RELU || (p->gated != 0 && p->gated != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (!is_float_type(p->out_type) && p->out_type != NVFP4_TYPE_FP8_MX) return NVFP4_ERR_INVALID_ARG;
  if (p->out_type == NVFP4_TYPE_FP8_MX && p->N % 32) return NVFP4_ERR_INVALID_ARG;
  // 32-bit sizes inside the kernels: a tile's offsets, rows of w, tiles of a launch
  if (p->K > (1 << 22) || p->N > (1 << 24)) return NVFP4_ERR_UNSUPPORTED;
  const int64_t tiles = (((int64_t)p->M + 255) / 256) * (((int64_t)p->N * (p->gated + 1) + 255) / 256);
  if (tiles > (1 << 20)) return NVFP4_ERR_UNSUPPORTED;
  a->M = p->M; a->N = p->N; a->K = p->K;
  a->kind = p->type == NVFP4_TYPE_BF16 ? 0 : p->type == NVFP4_TYPE_FP16 ? 1 : p->type == NVFP4_TYPE_FP8_ROW ? 2 : 3;
  a->act = p->act; a->gated = p->gated;
  a->out_type = elem_type(p->out_type);
  return NVFP4_OK;
}

}  // namespace

extern "C" {

NVFP4_API nvfp4_status_t nvfp4_rmsnorm(int32_t type, const void* x, int64_t ldx, const void* residual,
                                       int64_t ldr, const void* weight, float weight_offset, float eps,
                                       int32_t num_rows, int32_t K, void* sum_out, int64_t lds, void* y_out,
                                       int64_t ldy, int32_t fp8, uint8_t* codes, void* scales,
                                       nvfp4_stream_t stream) {
  if (type != NVFP4_TYPE_BF16 && type != NVFP4_TYPE_FP16) return NVFP4_ERR_INVALID_ARG;
  if (fp8 != NVFP4_FP8_NONE && !is_fp8(fp8)) return NVFP4_ERR_INVALID_ARG;
  if (num_rows < 0 || K < 8 || K % 8 || (fp8 == NVFP4_TYPE_FP8_MX && K % 32)) return NVFP4_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps) || !isfinite(weight_offset)) return NVFP4_ERR_INVALID_ARG;
  if (sum_out && !residual) return NVFP4_ERR_INVALID_ARG;
  if (K > kRowsMaxK) return NVFP4_ERR_UNSUPPORTED;
  if (num_rows == 0) return NVFP4_OK;
  if (!x || bad_rows(x, ldx, K) || (residual && bad_rows(residual, ldr, K)) || (weight && !aligned(weight, 16)) ||
      (sum_out && bad_rows(sum_out, lds, K)) || (y_out && bad_rows(y_out, ldy, K)))
    return NVFP4_ERR_INVALID_ARG;
  if (!sum_out && !y_out && fp8 == NVFP4_FP8_NONE) return NVFP4_ERR_INVALID_ARG;
  if (fp8 != NVFP4_FP8_NONE) {
    const nvfp4_status_t st = check_fp8_out(fp8, K, codes, scales);
    if (st != NVFP4_OK) return st;
  }
  RowArgs a = {};
  a.x = x; a.residual = residual; a.weight = weight; a.sum_out = sum_out; a.y_out = y_out;
  a.codes = codes; a.scales = scales;
  a.ldx = ldx; a.ldr = ldr; a.lds = lds; a.ldy = ldy;
  a.rows = num_rows; a.K = K;
  a.fp8 = fp8 == NVFP4_FP8_NONE ? 0 : fp8 == NVFP4_TYPE_FP8_ROW ? 1 : 2;
  a.offset = weight_offset; a.eps = eps;
  a.fp16 = type == NVFP4_TYPE_FP16; a.norm = true;
  return device_status(launch_rows(a, static_cast<hipStream_t>(stream)));
}

NVFP4_API nvfp4_status_t nvfp4_quantize_rows_fp8(int32_t type, const void* x, int64_t ldx, int32_t num_rows,
                                                 int32_t K, int32_t fp8, uint8_t* codes, void* scales,
                                                 nvfp4_stream_t stream) {
  if (type != NVFP4_TYPE_BF16 && type != NVFP4_TYPE_FP16) return NVFP4_ERR_INVALID_ARG;
  if (!is_fp8(fp8)) return NVFP4_ERR_INVALID_ARG;
  if (num_rows < 0 || K < 8 || K % 8 || (fp8 == NVFP4_TYPE_FP8_MX && K % 32)) return NVFP4_ERR_INVALID_ARG;
  if (K > kRowsMaxK) return NVFP4_ERR_UNSUPPORTED;
  if (num_rows == 0) return NVFP4_OK;
  if (!x || bad_rows(x, ldx, K)) return NVFP4_ERR_INVALID_ARG;
  const nvfp4_status_t st = check_fp8_out(fp8, K, codes, scales);
  if (st != NVFP4_OK) return st;
  RowArgs a = {};
  a.x = x; a.ldx = ldx; a.codes = codes; a.scales = scales;
  a.rows = num_rows; a.K = K;
  a.fp8 = fp8 == NVFP4_TYPE_FP8_ROW ? 1 : 2;
  a.fp16 = type == NVFP4_TYPE_FP16; a.norm = false;
  return device_status(launch_rows(a, static_cast<hipStream_t>(stream)));
}

NVFP4_API nvfp4_status_t nvfp4_linear_workspace_size(const nvfp4_linear_t* p, size_t* bytes) {
  if (!bytes) return NVFP4_ERR_INVALID_ARG;
  LinearArgs a = {};
  const nvfp4_status_t st = check_linear_sizes(p, &a);
  if (st != NVFP4_OK) return st;
  *bytes = linear_workspace_bytes(a);
  return NVFP4_OK;
}

NVFP4_API nvfp4_status_t nvfp4_linear(const nvfp4_linear_t* p, void* workspace, size_t workspace_bytes,
                                      nvfp4_stream_t stream) {
  LinearArgs a = {};
  const nvfp4_status_t st = check_linear_sizes(p, &a);
  if (st != NVFP4_OK) return st;
  if (p->bias && !is_float_type(p->bias_type)) return NVFP4_ERR_INVALID_ARG;
  if (p->residual && !is_float_type(p->residual_type)) return NVFP4_ERR_INVALID_ARG;
  if (p->M == 0 || p->N == 0) return NVFP4_OK;
  const bool f8 = is_fp8(p->type);
  const int64_t esz = f8 ? 1 : 2;
  if (!p->a || !p->w || !p->out || !aligned(p->a, 16) || !aligned(p->w, 16)) return NVFP4_ERR_INVALID_ARG;
  if (p->lda < p->K || p->ldw < p->K || p->lda * esz % 16 || p->ldw * esz % 16) return NVFP4_ERR_INVALID_ARG;
  if (p->lda * esz > (1 << 23) || p->ldw * esz > (1 << 23)) return NVFP4_ERR_UNSUPPORTED;
  if (f8 && (!p->a_scales || !p->w_scales)) return NVFP4_ERR_INVALID_ARG;
  if (p->type == NVFP4_TYPE_FP8_ROW && (!aligned(p->a_scales, 4) || !aligned(p->w_scales, 4)))
    return NVFP4_ERR_INVALID_ARG;
  if (p->bias && !aligned(p->bias, float_size(p->bias_type))) return NVFP4_ERR_INVALID_ARG;
  if (p->residual && (p->ldr < p->N || !aligned(p->residual, float_size(p->residual_type))))
    return NVFP4_ERR_INVALID_ARG;
  if (p->ldo < p->N) return NVFP4_ERR_INVALID_ARG;
  if (p->out_type == NVFP4_TYPE_FP8_MX) {
    if (!p->out_scales || !aligned(p->out, 16) || p->ldo % 16) return NVFP4_ERR_INVALID_ARG;
  } else if (!aligned(p->out, float_size(p->out_type))) {
    return NVFP4_ERR_INVALID_ARG;
  }
  a.a = p->a; a.a_scales = p->a_scales; a.w = p->w; a.w_scales = p->w_scales;
  a.bias = p->bias; a.residual = p->residual; a.out = p->out; a.out_scales = p->out_scales;
  a.lda = p->lda; a.ldw = p->ldw; a.ldr = p->ldr; a.ldo = p->ldo;
  a.bias_type = elem_type(p->bias_type); a.residual_type = elem_type(p->residual_type);
  const size_t need = linear_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return NVFP4_ERR_WORKSPACE;
  return device_status(launch_linear(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
