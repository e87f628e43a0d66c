// C ABI of the dense operators around the routed experts: argument checking of
// nvfp4_rmsnorm, nvfp4_block_norm, nvfp4_quantize_rows_fp8, nvfp4_linear, nvfp4_linear_w4,
// nvfp4_grouped_linear and nvfp4_combine.
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

// Types and sizes that nvfp4_linear and nvfp4_grouped_linear share.
bool bad_product(int32_t type, int32_t out_type, int32_t act, int32_t gated, int32_t N, int32_t K) {
  if (N < 0 || K < 1) return true;
  if (type != NVFP4_TYPE_BF16 && type != NVFP4_TYPE_FP16 && !is_fp8(type)) return true;
  if (K % (type == NVFP4_TYPE_FP8_MX ? 32 : is_fp8(type) ? 16 : 8)) return true;
  if (act < NVFP4_ACT_NONE || act > NVFP4_ACT_RELU || (gated != 0 && gated != 1)) return true;
  if (!is_float_type(out_type) && out_type != NVFP4_TYPE_FP8_MX) return true;
  return out_type == NVFP4_TYPE_FP8_MX && N % 32;
}

int32_t operand_kind(int32_t t) {
  return t == NVFP4_TYPE_BF16 ? 0 : t == NVFP4_TYPE_FP16 ? 1 : t == NVFP4_TYPE_FP8_ROW ? 2 : 3;
}

// Sizes and types alone (no pointer of *p is looked at), as nvfp4_linear_workspace_size
// and nvfp4_linear both need them.
nvfp4_status_t check_linear_sizes(const nvfp4_linear_t* p, LinearArgs* a) {
  if (!p || p->M < 0 || bad_product(p->type, p->out_type, p->act, p->gated, p->N, p->K)) return NVFP4_ERR_INVALID_ARG;
  // 32-bit sizes inside the kernels: a tile's offsets, rows of w, tiles of a launch
  if (p->K > (1 << 22) || p->N > (1 << 24)) return NVFP4_ERR_UNSUPPORTED;
  const int64_t tiles = (((int64_t)p->M + 255) / 256) * (((int64_t)p->N * (p->gated + 1) + 255) / 256);
  if (tiles > (1 << 20)) return NVFP4_ERR_UNSUPPORTED;
  a->M = p->M; a->N = p->N; a->K = p->K;
  a->kind = operand_kind(p->type);
  a->act = p->act; a->gated = p->gated;
  a->out_type = elem_type(p->out_type);
  return NVFP4_OK;
}

// The epilogue's tensors of nvfp4_linear and nvfp4_linear_w4.
nvfp4_status_t check_extra_types(const nvfp4_linear_t* p) {
  if (p->bias && !is_float_type(p->bias_type)) return NVFP4_ERR_INVALID_ARG;
  if (p->residual && !is_float_type(p->residual_type)) return NVFP4_ERR_INVALID_ARG;
  return NVFP4_OK;
}

nvfp4_status_t check_epilogue(const nvfp4_linear_t* p) {
  if (p->bias && !aligned(p->bias, float_size(p->bias_type))) return NVFP4_ERR_INVALID_ARG;
  if (p->residual && (p->ldr < p->N || !aligned(p->residual, float_size(p->residual_type))))
    return NVFP4_ERR_INVALID_ARG;
  if (p->ldo < p->N) return NVFP4_ERR_INVALID_ARG;
  if (p->out_type == NVFP4_TYPE_FP8_MX) {
    if (!p->out_scales || !aligned(p->out, 16) || p->ldo % 16) return NVFP4_ERR_INVALID_ARG;
  } else if (!aligned(p->out, float_size(p->out_type))) {
    return NVFP4_ERR_INVALID_ARG;
  }
  return NVFP4_OK;
}

void take_linear(const nvfp4_linear_t* p, LinearArgs* a) {
  a->a = p->a; a->a_scales = p->a_scales; a->w = p->w; a->w_scales = p->w_scales;
  a->bias = p->bias; a->residual = p->residual; a->out = p->out; a->out_scales = p->out_scales;
  a->lda = p->lda; a->ldw = p->ldw; a->ldr = p->ldr; a->ldo = p->ldo;
  a->bias_type = elem_type(p->bias_type); a->residual_type = elem_type(p->residual_type);
}

nvfp4_status_t check_w4_sizes(const nvfp4_linear_t* p, int32_t w4, Linear4Args* a) {
  if (w4 != NVFP4_W4_NV && w4 != NVFP4_W4_MX) return NVFP4_ERR_INVALID_ARG;
  const nvfp4_status_t st = check_linear_sizes(p, a);
  if (st != NVFP4_OK) return st;
  if (is_fp8(p->type) || p->K % 32) return NVFP4_ERR_INVALID_ARG;
  a->mx = w4 == NVFP4_W4_MX;
  if (a->mx && p->type == NVFP4_TYPE_FP16 && p->K > (1 << 21)) return NVFP4_ERR_UNSUPPORTED;
  if ((int64_t)p->N * (p->gated + 1) > ((int64_t)1 << 36) / p->K || p->M > ((int64_t)1 << 34) / p->K)
    return NVFP4_ERR_UNSUPPORTED;
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

NVFP4_API nvfp4_status_t nvfp4_block_norm(const nvfp4_block_norm_t* p, nvfp4_stream_t stream) {
  if (!p || (p->type != NVFP4_TYPE_BF16 && p->type != NVFP4_TYPE_FP16)) return NVFP4_ERR_INVALID_ARG;
  if (p->fp8 != NVFP4_FP8_NONE && !is_fp8(p->fp8)) return NVFP4_ERR_INVALID_ARG;
  const int32_t K = p->K;
  if (p->num_rows < 0 || K < 8 || K % 8 || (p->fp8 == NVFP4_TYPE_FP8_MX && K % 32)) return NVFP4_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !isfinite(p->eps) || !isfinite(p->weight_offset) || !isfinite(p->gate_scale) ||
      !isfinite(p->residual_scale) || (p->post != 0 && p->post != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (p->gate) {
    if (p->gate_type != p->type && p->gate_type != NVFP4_TYPE_FP32) return NVFP4_ERR_INVALID_ARG;
    if (p->gate_act < NVFP4_GATE_PLAIN || p->gate_act > NVFP4_GATE_TANH) return NVFP4_ERR_INVALID_ARG;
    if ((p->gate_cols != 1 && p->gate_cols != K) || p->ldg < 0) return NVFP4_ERR_INVALID_ARG;
  }
  if (K > kRowsMaxK) return NVFP4_ERR_UNSUPPORTED;
  if (p->num_rows == 0) return NVFP4_OK;
  if (!p->x || !p->residual || bad_rows(p->x, p->ldx, K) || bad_rows(p->residual, p->ldr, K) ||
      (p->post_weight && !aligned(p->post_weight, 16)) || (p->weight && !aligned(p->weight, 16)) ||
      (p->total_out && bad_rows(p->total_out, p->ldt, K)) || (p->y_out && bad_rows(p->y_out, p->ldy, K)))
    return NVFP4_ERR_INVALID_ARG;
  if (p->gate) {
    const int64_t size = float_size(p->gate_type);
    if (!aligned(p->gate, p->gate_cols == 1 ? size : 16)) return NVFP4_ERR_INVALID_ARG;
    if (p->gate_cols != 1 && (p->ldg * size % 16 || (p->ldg != 0 && p->ldg < K))) return NVFP4_ERR_INVALID_ARG;
  }
  if (!p->total_out && !p->y_out && p->fp8 == NVFP4_FP8_NONE) return NVFP4_ERR_INVALID_ARG;
  if (p->fp8 != NVFP4_FP8_NONE) {
    const nvfp4_status_t st = check_fp8_out(p->fp8, K, p->codes, p->scales);
    if (st != NVFP4_OK) return st;
  }
  BlockArgs a = {};
  a.x = p->x; a.residual = p->residual; a.post_weight = p->post_weight; a.weight = p->weight; a.gate = p->gate;
  a.total_out = p->total_out; a.y_out = p->y_out; a.codes = p->codes; a.scales = p->scales;
  a.ldx = p->ldx; a.ldr = p->ldr; a.ldg = p->ldg; a.ldt = p->ldt; a.ldy = p->ldy;
  a.rows = p->num_rows; a.K = K;
  a.fp8 = p->fp8 == NVFP4_FP8_NONE ? 0 : p->fp8 == NVFP4_TYPE_FP8_ROW ? 1 : 2;
  a.gate_act = p->gate ? p->gate_act : 0;
  a.offset = p->weight_offset; a.eps = p->eps; a.gate_scale = p->gate_scale; a.residual_scale = p->residual_scale;
  a.fp16 = p->type == NVFP4_TYPE_FP16; a.post = p->post != 0;
  a.gate_wide = p->gate && p->gate_cols != 1; a.gate_f32 = p->gate && p->gate_type == NVFP4_TYPE_FP32;
  return device_status(launch_block(a, static_cast<hipStream_t>(stream)));
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
  const nvfp4_status_t types = check_extra_types(p);
  if (types != NVFP4_OK) return types;
  if (p->M == 0 || p->N == 0) return NVFP4_OK;
  const bool f8 = is_fp8(p->type);
  const int64_t esz = f8 ? 1 : 2;
  if (!p->a || !p->w || !p->out || !aligned(p->a, 16) || !aligned(p->w, 16)) return NVFP4_ERR_INVALID_ARG;
  if (p->lda < p->K || p->ldw < p->K || p->lda * esz % 16 || p->ldw * esz % 16) return NVFP4_ERR_INVALID_ARG;
  if (p->lda * esz > (1 << 23) || p->ldw * esz > (1 << 23)) return NVFP4_ERR_UNSUPPORTED;
  if (f8 && (!p->a_scales || !p->w_scales)) return NVFP4_ERR_INVALID_ARG;
  if (p->type == NVFP4_TYPE_FP8_ROW && (!aligned(p->a_scales, 4) || !aligned(p->w_scales, 4)))
    return NVFP4_ERR_INVALID_ARG;
  const nvfp4_status_t rest = check_epilogue(p);
  if (rest != NVFP4_OK) return rest;
  take_linear(p, &a);
  const size_t need = linear_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return NVFP4_ERR_WORKSPACE;
  return device_status(launch_linear(a, workspace, static_cast<hipStream_t>(stream)));
}

NVFP4_API nvfp4_status_t nvfp4_linear_w4_workspace_size(const nvfp4_linear_t* p, int32_t w4, size_t* bytes) {
  if (!bytes) return NVFP4_ERR_INVALID_ARG;
  Linear4Args a = {};
  const nvfp4_status_t st = check_w4_sizes(p, w4, &a);
  if (st != NVFP4_OK) return st;
  *bytes = linear4_workspace_bytes(a);
  return NVFP4_OK;
}

NVFP4_API nvfp4_status_t nvfp4_linear_w4(const nvfp4_linear_t* p, int32_t w4, const float* gain, void* workspace,
                                         size_t workspace_bytes, nvfp4_stream_t stream) {
  Linear4Args a = {};
  const nvfp4_status_t st = check_w4_sizes(p, w4, &a);
  if (st != NVFP4_OK) return st;
  const nvfp4_status_t types = check_extra_types(p);
  if (types != NVFP4_OK) return types;
  if (p->M == 0 || p->N == 0) return NVFP4_OK;
  if (!p->a || !p->w || !p->w_scales || !p->out || !aligned(p->a, 16) || !aligned(p->w, 16) || !aligned(gain, 4) ||
      !aligned(p->w_scales, a.mx ? 1 : 2))
    return NVFP4_ERR_INVALID_ARG;
  if (p->lda < p->K || p->ldw < p->K / 2 || p->lda % 8 || p->ldw % 16) return NVFP4_ERR_INVALID_ARG;
  if (p->lda * 2 > (1 << 23) || p->ldw > (1 << 23)) return NVFP4_ERR_UNSUPPORTED;
  const nvfp4_status_t rest = check_epilogue(p);
  if (rest != NVFP4_OK) return rest;
  take_linear(p, &a);
  a.gain = gain;
  const size_t need = linear4_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return NVFP4_ERR_WORKSPACE;
  return device_status(launch_linear4(a, workspace, static_cast<hipStream_t>(stream)));
}

NVFP4_API nvfp4_status_t nvfp4_grouped_linear(const nvfp4_grouped_linear_t* p, nvfp4_stream_t stream) {
  if (!p || p->num_rows < 0 || p->a_rows < 0 || p->num_experts < 1 ||
      bad_product(p->type, p->out_type, p->act, p->gated, p->N, p->K))
    return NVFP4_ERR_INVALID_ARG;
  if (p->index ? p->index_div < 1 : p->a_rows < p->num_rows) return NVFP4_ERR_INVALID_ARG;
  if (p->bias && !is_float_type(p->bias_type)) return NVFP4_ERR_INVALID_ARG;
  if (p->num_experts > 1024 || p->K > (1 << 22) || p->N > (1 << 24) || p->num_rows > (1 << 29)) return NVFP4_ERR_UNSUPPORTED;
  GroupedArgs a = {};
  a.M = p->num_rows; a.a_rows = p->a_rows; a.experts = p->num_experts; a.N = p->N; a.K = p->K; a.index_div = p->index_div;
  a.kind = operand_kind(p->type); a.act = p->act; a.gated = p->gated; a.out_type = elem_type(p->out_type);
  if (!grouped_fits(a)) return NVFP4_ERR_UNSUPPORTED;
  if (p->num_rows == 0 || p->a_rows == 0 || p->N == 0) return NVFP4_OK;
  const bool f8 = is_fp8(p->type);
  const int64_t esz = f8 ? 1 : 2, rows = (int64_t)p->N * (p->gated + 1);
  if (!p->a || !p->w || !p->out || !p->offsets || !aligned(p->a, 16) || !aligned(p->w, 16) || !aligned(p->offsets, 4) ||
      !aligned(p->index, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (p->lda < p->K || p->ldw < p->K || p->lda * esz % 16 || p->ldw * esz % 16) return NVFP4_ERR_INVALID_ARG;
  if (p->lda * esz > (1 << 23) || p->ldw * esz > (1 << 23)) return NVFP4_ERR_UNSUPPORTED;
  if (p->num_experts > 1 && (p->w_each * esz % 16 || p->w_each < (rows - 1) * p->ldw + p->K)) return NVFP4_ERR_INVALID_ARG;
  if (f8 && (!p->a_scales || !p->w_scales)) return NVFP4_ERR_INVALID_ARG;
  if (p->type == NVFP4_TYPE_FP8_ROW && (!aligned(p->a_scales, 4) || !aligned(p->w_scales, 4))) return NVFP4_ERR_INVALID_ARG;
  if (p->bias && !aligned(p->bias, float_size(p->bias_type))) return NVFP4_ERR_INVALID_ARG;
  if (p->ldo < p->N) return NVFP4_ERR_INVALID_ARG;
  if (p->out_type == NVFP4_TYPE_FP8_MX) {
    if (!p->out_scales || !aligned(p->out, 16) || p->ldo % 16) return NVFP4_ERR_INVALID_ARG;
  } else if (!aligned(p->out, float_size(p->out_type))) {
    return NVFP4_ERR_INVALID_ARG;
  }
  a.a = p->a; a.a_scales = p->a_scales; a.w = p->w; a.w_scales = p->w_scales; a.bias = p->bias;
  a.offsets = p->offsets; a.index = p->index; a.out = p->out; a.out_scales = p->out_scales;
  a.lda = p->lda; a.ldw = p->ldw; a.w_each = p->num_experts > 1 ? p->w_each : 0; a.ldo = p->ldo;
  a.bias_type = elem_type(p->bias_type);
  return device_status(launch_grouped(a, static_cast<hipStream_t>(stream)));
}

NVFP4_API nvfp4_status_t nvfp4_combine(int32_t type, const void* values, int64_t ldv, int32_t num_rows,
                                       const float* weights, const int32_t* inv_pair, int32_t num_tokens, int32_t k,
                                       int32_t H, int32_t residual_type, const void* residual, int64_t ldr,
                                       int32_t out_type, void* out, int64_t ldo, nvfp4_stream_t stream) {
  if (!is_float_type(type) || !is_float_type(out_type) || (residual && !is_float_type(residual_type)))
    return NVFP4_ERR_INVALID_ARG;
  if (num_rows < 0 || num_tokens < 0 || k < 1 || H < 8 || H % 8) return NVFP4_ERR_INVALID_ARG;
  if (H > (1 << 24) || k > 1024) return NVFP4_ERR_UNSUPPORTED;
  if (num_tokens == 0) return NVFP4_OK;
  auto bad = [&](const void* p, int64_t ld, int32_t t) {
    return !p || !aligned(p, 16) || ld < H || ld * (int64_t)float_size(t) % 16;
  };
  if ((num_rows > 0 && bad(values, ldv, type)) || bad(out, ldo, out_type) || (residual && bad(residual, ldr, residual_type)) ||
      !weights || !inv_pair || !aligned(weights, 4) || !aligned(inv_pair, 4))
    return NVFP4_ERR_INVALID_ARG;
  CombineArgs a = {};
  a.values = values; a.weights = weights; a.inv = inv_pair; a.residual = residual; a.out = out;
  a.ldv = ldv; a.ldr = ldr; a.ldo = ldo;
  a.rows = num_rows; a.T = num_tokens; a.k = k; a.H = H;
  a.type = elem_type(type); a.residual_type = elem_type(residual_type); a.out_type = elem_type(out_type);
  return device_status(launch_combine_rows(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
