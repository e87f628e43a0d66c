// Products grouped by expert for gfx950: the linear operator's kernels on rows whose
// weight depends on the group that they are in,
//
//   out[m, n] = act(sum_k a[row(m), k] * w[e, n, k] + bias[e, n]),   offsets[e] <= m < offsets[e + 1],
//
// or act(gate) * up.  The groups' sizes stay on the device: the grid covers the most
// tiles that M rows can fall into, each workgroup finds its expert from the offsets (2 us
// with the start of the kernel, by prefixes over the experts in every wavefront), those
// without a tile end.  A tile belongs to one expert, so a group's last tile is partly
// empty: it leaves out the instructions, copies and epilogue of its empty rows and keeps
// more steps on their way (16-bit operands; 8-bit ones are converted to bf16, so that their
// products are exact).  Rows of a are gathered by the copies into LDS themselves.
#include "internal.h"
#include "linear_kernels.h"

namespace nvfp4 {
namespace {

template <int kKind, int kTile, int kWM, int kWN, int kStages, bool kGated>
hipError_t go_tile(const GroupParams& p, uint32_t blocks, hipStream_t stream) {
  hipLaunchKernelGGL((linear_tile_kernel<kKind, kTile, kTile, kWM, kWN, kStages, kGated, true>), dim3(blocks), dim3(64 * kWM * kWN), 0,
                     stream, p);
  return hipGetLastError();
}

template <int kKind, bool kGated>
hipError_t go(GroupParams p, const GroupPlan& plan, hipStream_t stream) {
  const uint32_t blocks = (uint32_t)group_blocks(plan.row_tiles, plan.tiles_n);
  p.tiles_n = plan.tiles_n;
  if constexpr (!is_wide(kKind))
    if (plan.kernel == kTile256) return go_tile<kKind, 256, 2, 4, 2, kGated>(p, blocks, stream);
  if (plan.kernel == kTile128) return go_tile<kKind, 128, 2, 2, 2, kGated>(p, blocks, stream);
  return go_tile<kKind, 64, 2, 2, 4, kGated>(p, blocks, stream);
}

template <int kKind>
hipError_t go_gated(const GroupParams& p, int32_t gated, const GroupPlan& plan, hipStream_t stream) {
  return gated ? go<kKind, true>(p, plan, stream) : go<kKind, false>(p, plan, stream);
}

GroupPlan plan_for(const GroupedArgs& a) {
  return group_plan_of(a.M, a.experts, a.N, a.K * (a.kind <= kF16 ? 2 : 1), a.kind, a.gated != 0, a.out_type);
}

}  // namespace

bool grouped_fits(const GroupedArgs& a) {
  if (a.M == 0 || a.N == 0) return true;
  const GroupPlan q = plan_for(a);
  return group_blocks(q.row_tiles, q.tiles_n) <= 0x7FFFFFFF / 512;  // threads of a launch, with the kernels' 32-bit numbers
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0 || a.a_rows == 0) return hipSuccess;
  const int32_t esz = a.kind <= kF16 ? 2 : 1, rows = a.gated ? 2 * a.N : a.N;
  GroupParams p = {};
  p.a = static_cast<const char*>(a.a);
  p.w = static_cast<const char*>(a.w);
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.out = a.out;
  p.out_scales = a.out_scales;
  p.lda = a.lda * esz;
  p.ldw = a.ldw * esz;
  p.ldo = a.ldo;
  p.M = a.M; p.N = a.N; p.kbytes = a.K * esz;
  p.act = a.act; p.bias_type = a.bias_type; p.out_type = a.out_type;
  p.offsets = a.offsets;
  p.index = a.index;
  p.w_each = a.w_each * esz;
  p.scales_each = a.kind == kRow8 ? (int64_t)rows * 4 : a.kind == kBlock8 ? (int64_t)rows * (a.K / 32) : 0;
  p.bias_each = rows;
  p.experts = a.experts; p.a_rows = a.a_rows; p.index_div = a.index_div;
  const GroupPlan plan = plan_for(a);
  switch (kind_of(a.kind, 1, a.out_type)) {                    // exact products at any number of rows (group_plan_of)
    case kBf16: return go_gated<kBf16>(p, a.gated, plan, stream);
    case kF16: return go_gated<kF16>(p, a.gated, plan, stream);
    case kRow8Wide: return go_gated<kRow8Wide>(p, a.gated, plan, stream);
    case kBlock8Wide: return go_gated<kBlock8Wide>(p, a.gated, plan, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nvfp4
