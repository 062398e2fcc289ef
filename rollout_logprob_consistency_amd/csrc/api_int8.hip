// C-ABI entry points of the 8-bit head (include/liblp_int8.h): argument
// validation and launch arguments. Every check happens before anything is
// enqueued.
#include <math.h>
#include <stdint.h>

#include <limits>

#include "int8_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

constexpr int64_t kI32Max = std::numeric_limits<int32_t>::max();

bool dtype_ok(int32_t dtype) { return dtype == LP_F32 || dtype == LP_BF16 || dtype == LP_F16; }

// (Below 2^-126 the kernels' fp32 scale log2(e) / t would be infinite.)
bool temperature_ok(float t) { return isnormal(t) && t > 0.0f; }

// Rows of a dispatch of one 256-thread workgroup for each, at most 2^32 - 1
// work-items.
constexpr int64_t kRowsMax = 16777215;
static_assert(kRowsMax <= lp::kMaxDispatchItems / 256, "one dispatch");

// A block's rows past V still have 32-bit indices.
constexpr int64_t kVocabMax = kI32Max - 255;

// Checks of the operands that both products share. `go` is set when there is
// work to enqueue.
lp_status product_args(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                       int64_t ldw, const float* w_scale, int64_t T, int64_t H, int64_t V,
                       lp::Int8Args* a, bool* go) {
  *go = false;
  if (T < 0 || H < 1 || V < 1 || ldx < H || ldw < H) return LP_EINVAL;
  if (T == 0) return LP_OK;
  if (!x || !x_scale || !w || !w_scale || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return LP_EINVAL;
  if (H > LP_INT8_MAX_HIDDEN || T > kI32Max || V > kVocabMax || ldw % 16 != 0 ||
      ldw > lp::kInt8StrideMax || !lp::int8_grid_ok(T, V))
    return LP_EUNSUPPORTED;
  if (!aligned(w, 16)) return LP_EINVAL;
  *a = lp::Int8Args{};
  a->x = x;
  a->x_scale = x_scale;
  a->w = w;
  a->w_scale = w_scale;
  a->ldx = ldx;
  a->ldw = ldw;
  a->T = (int32_t)T;
  a->H = (int32_t)H;
  a->V = (int32_t)V;
  *go = true;
  return LP_OK;
}

bool workspace_ok(const void* workspace, size_t bytes, const lp::Int8Workspace& w) {
  return workspace && aligned(workspace, 256) && bytes >= w.total;
}

}  // namespace

extern "C" {

lp_status lp_quantize_int8(const void* x, int64_t ldx, int32_t dtype, int64_t R, int64_t H,
                           int8_t* q, int64_t ldq, float* scale, int32_t* bad_rows,
                           hipStream_t stream) {
  if (R < 0 || H < 1 || ldx < H || ldq < H || ldq % 16 != 0 || !dtype_ok(dtype)) return LP_EINVAL;
  if (R == 0) return LP_OK;
  if (!x || !q || !scale || !aligned(x, (uintptr_t)lp::dtype_bytes(dtype)) || !aligned(q, 16) ||
      !aligned(scale, 4) || !aligned(bad_rows, 4))
    return LP_EINVAL;
  if (R > kRowsMax || H > kI32Max) return LP_EUNSUPPORTED;
  const lp::QuantizeArgs a = {x, ldx, dtype, R, H, q, ldq, scale, bad_rows};
  return lp::launch_quantize_int8(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

size_t lp_logits_int8_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || T > kI32Max || H < 1 || H > LP_INT8_MAX_HIDDEN) return 0;
  const size_t total = lp::int8_workspace_layout(T, H, 0).total;
  return total < 256 ? 256 : total;
}

lp_status lp_logits_int8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                         int64_t ldw, const float* w_scale, int64_t T, int64_t H, int64_t V,
                         void* out, int64_t ld_out, int32_t dtype, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  if (ld_out < V || !dtype_ok(dtype)) return LP_EINVAL;
  lp::Int8Args a;
  bool go;
  const lp_status st = product_args(x, ldx, x_scale, w, ldw, w_scale, T, H, V, &a, &go);
  if (st != LP_OK || !go) return st;
  if (ld_out > lp::kInt8StrideMax) return LP_EUNSUPPORTED;
  const lp::Int8Workspace ws = lp::int8_workspace_layout(T, H, 0);
  if (!out || !aligned(out, (uintptr_t)lp::dtype_bytes(dtype)) ||
      !workspace_ok(workspace, workspace_bytes, ws))
    return LP_EINVAL;
  a.out = out;
  a.ld_out = ld_out;
  a.dtype = dtype;
  a.staged = static_cast<int8_t*>(workspace) + ws.off_staged;
  return lp::launch_int8(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

size_t lp_score_int8_workspace_bytes(int64_t T, int64_t H, int64_t V_true) {
  if (T < 0 || T > kI32Max || H < 1 || H > LP_INT8_MAX_HIDDEN || V_true < 1 || V_true > kVocabMax)
    return 0;
  const size_t total = lp::int8_workspace_layout(T, H, V_true).total;
  return total < 256 ? 256 : total;
}

lp_status lp_score_int8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                        int64_t ldw, const float* w_scale, const int64_t* target_ids, int64_t T,
                        int64_t H, int64_t V_true, float temperature, uint32_t flags,
                        float* out_logprob, float* out_lse, int32_t* bad_rows, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  if (!temperature_ok(temperature) || (flags & ~LP_SCORE_BF16_LOGITS)) return LP_EINVAL;
  lp::Int8Args a;
  bool go;
  const lp_status st = product_args(x, ldx, x_scale, w, ldw, w_scale, T, H, V_true, &a, &go);
  if (st != LP_OK || !go) return st;
  const lp::Int8Workspace ws = lp::int8_workspace_layout(T, H, V_true);
  if (!target_ids || !out_logprob || !aligned(target_ids, 8) || !aligned(out_logprob, 4) ||
      !aligned(out_lse, 4) || !aligned(bad_rows, 4) ||
      !workspace_ok(workspace, workspace_bytes, ws))
    return LP_EINVAL;
  char* base = static_cast<char*>(workspace);
  a.ids = target_ids;
  a.bf16_logits = (flags & LP_SCORE_BF16_LOGITS) != 0;
  a.scale2 = (float)(1.4426950408889634 / (double)temperature);
  a.part_m = reinterpret_cast<float*>(base + ws.off_m);
  a.part_s = reinterpret_cast<float*>(base + ws.off_s);
  a.out_lp = out_logprob;
  a.out_lse = out_lse;
  a.bad_rows = bad_rows;
  a.staged = reinterpret_cast<int8_t*>(base + ws.off_staged);
  return lp::launch_int8(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

}  // extern "C"
