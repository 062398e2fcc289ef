// C-ABI entry points of the operators on rows of logits
// (include/liblp_logits.h): argument validation and launch arguments. Every
// check happens before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <limits>

#include "logits_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

constexpr int64_t kI32Max = std::numeric_limits<int32_t>::max();

bool dtype_ok(int32_t dtype) { return dtype == LP_F32 || dtype == LP_BF16 || dtype == LP_F16; }

// Element size of a valid dtype.
uintptr_t size_of(int32_t dtype) { return (uintptr_t)lp::dtype_bytes(dtype); }

// (Below 2^-126 the kernels' fp32 scale log2(e) / t would be infinite.)
bool temperature_ok(float t) { return isnormal(t) && t > 0.0f; }

// One workgroup of kSelectThreads per row in a dispatch of 2^32 - 1 work-items
// at most (and fewer than 4 194 304 rows, the limit the interface names).
constexpr int64_t kSelectMaxRows = 4194303;
static_assert(kSelectMaxRows <= lp::kMaxDispatchItems / lp::kSelectThreads, "one dispatch");

size_t select_workspace_bytes(int64_t N, int64_t V_true, int32_t dtype) {
  if (N < 0 || N > kSelectMaxRows || V_true < 1 || V_true > LP_SELECT_MAX_VOCAB ||
      !dtype_ok(dtype))
    return 0;
  const size_t most = lp::select_workspace_most(N, V_true, dtype);
  return most < 256 ? 256 : most;
}

bool select_workspace_ok(const void* workspace, size_t bytes, int64_t N, int64_t V_true,
                         int32_t dtype) {
  return aligned(workspace, 256) && bytes >= lp::select_workspace_layout(N, V_true, dtype).total;
}

}  // namespace

extern "C" {

size_t lp_sample_workspace_bytes(int64_t N, int64_t V_true, int32_t dtype) {
  return select_workspace_bytes(N, V_true, dtype);
}

lp_status lp_sample(const void* logits, int64_t ld, int32_t dtype, int64_t N, int64_t V_true,
                    const float* u, const float* temperatures, float temperature,
                    const int32_t* top_ks, int32_t top_k, const float* top_ps, float top_p,
                    const float* min_ps, float min_p, int64_t* out_token, float* out_logprob,
                    float* out_processed, int32_t* out_kept, int32_t* bad_rows, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  if (N < 0 || V_true < 1 || ld < V_true || !dtype_ok(dtype)) return LP_EINVAL;
  if (!temperatures && temperature != 0.0f && !temperature_ok(temperature)) return LP_EINVAL;
  if ((!top_ps && isnan(top_p)) || (!min_ps && isnan(min_p))) return LP_EINVAL;
  if (N == 0) return LP_OK;
  if (!logits || !u || !out_token || !out_logprob || !workspace) return LP_EINVAL;
  if (!aligned(logits, size_of(dtype)) || !aligned(u, 4) || !aligned(temperatures, 4) ||
      !aligned(top_ks, 4) || !aligned(top_ps, 4) || !aligned(min_ps, 4) ||
      !aligned(out_token, 8) || !aligned(out_logprob, 4) || !aligned(out_processed, 4) ||
      !aligned(out_kept, 4) || !aligned(bad_rows, 4))
    return LP_EINVAL;
  if (V_true > LP_SELECT_MAX_VOCAB || N > kSelectMaxRows) return LP_EUNSUPPORTED;
  if (!select_workspace_ok(workspace, workspace_bytes, N, V_true, dtype)) return LP_EINVAL;
  lp::SelectArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.dtype = dtype;
  a.N = N;
  a.V = (int32_t)V_true;
  a.u = u;
  a.temperatures = temperatures;
  a.top_ks = top_ks;
  a.top_ps = top_ps;
  a.min_ps = min_ps;
  a.temperature = temperature;
  a.top_p = top_p;
  a.min_p = min_p;
  a.top_k = top_k;
  a.out_token = out_token;
  a.out_logprob = out_logprob;
  a.out_processed = out_processed;
  a.out_kept = out_kept;
  a.bad_rows = bad_rows;
  return lp::launch_select(a, workspace, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

size_t lp_top_logprobs_workspace_bytes(int64_t N, int64_t V_true, int32_t dtype) {
  return select_workspace_bytes(N, V_true, dtype);
}

lp_status lp_top_logprobs(const void* logits, int64_t ld, int32_t dtype, int64_t N, int64_t V_true,
                          int32_t k, float temperature, int64_t* out_ids, float* out_logits,
                          float* out_logprob, float* out_lse, int32_t* bad_rows, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  if (N < 0 || V_true < 1 || ld < V_true || !dtype_ok(dtype)) return LP_EINVAL;
  if (k < 1 || k > V_true || !temperature_ok(temperature)) return LP_EINVAL;
  if (N == 0) return LP_OK;
  if (!logits || !out_ids || !out_logits || !out_logprob || !workspace) return LP_EINVAL;
  if (!aligned(logits, size_of(dtype)) || !aligned(out_ids, 8) || !aligned(out_logits, 4) ||
      !aligned(out_logprob, 4) || !aligned(out_lse, 4) || !aligned(bad_rows, 4))
    return LP_EINVAL;
  if (k > LP_TOP_MAX || V_true > LP_SELECT_MAX_VOCAB || N > kSelectMaxRows) return LP_EUNSUPPORTED;
  if (!select_workspace_ok(workspace, workspace_bytes, N, V_true, dtype)) return LP_EINVAL;
  lp::SelectArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.dtype = dtype;
  a.N = N;
  a.V = (int32_t)V_true;
  a.temperature = temperature;
  a.top_k = k;
  a.out_ids = out_ids;
  a.out_logits = out_logits;
  a.out_logprob = out_logprob;
  a.out_lse = out_lse;
  a.bad_rows = bad_rows;
  return lp::launch_select(a, workspace, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

size_t lp_distill_workspace_bytes(int64_t T, int64_t V_true, int32_t dtype) {
  if (T < 0 || T > kI32Max || V_true < 1 || V_true > kI32Max || !dtype_ok(dtype)) return 0;
  const size_t total = lp::distill_workspace_layout(T, V_true, dtype).total;
  return total < 256 ? 256 : total;
}

}  // extern "C"

namespace {

// Checks shared by the three distillation calls. `go` is set when there is
// work to enqueue.
lp_status distill_args(const void* logits, int64_t ld, int32_t dtype, int64_t T, int64_t V_true,
                       int64_t V_columns, const int64_t* teacher_ids, const float* teacher,
                       int64_t K, float temperature, uint32_t flags, lp::DistillArgs* a,
                       bool* go) {
  *go = false;
  if (T < 0 || V_true < 1 || ld < V_true || V_columns < V_true || K < 1 || !dtype_ok(dtype))
    return LP_EINVAL;
  if ((flags & ~LP_DISTILL_LOGPROBS) || !temperature_ok(temperature)) return LP_EINVAL;
  if (T == 0) return LP_OK;
  if (!logits || !teacher_ids || !teacher) return LP_EINVAL;
  if (!aligned(logits, size_of(dtype)) || !aligned(teacher_ids, 8) || !aligned(teacher, 4))
    return LP_EINVAL;
  if (K > LP_DISTILL_MAX_K || T > kI32Max || V_columns > kI32Max) return LP_EUNSUPPORTED;
  *a = lp::DistillArgs{};
  a->logits = logits;
  a->ld = ld;
  a->dtype = dtype;
  a->T = T;
  a->V_true = V_true;
  a->V_columns = V_columns;
  a->ids = teacher_ids;
  a->teacher = teacher;
  a->K = (int32_t)K;
  a->logprobs = (flags & LP_DISTILL_LOGPROBS) != 0;
  a->inv_tau = 1.0 / (double)temperature;
  a->scale2 = (float)(1.4426950408889634 / (double)temperature);
  a->slices = lp::distill_slices(V_true, dtype);
  *go = true;
  return LP_OK;
}

// The workspace's parts; false when it is too small or misaligned.
bool distill_workspace(lp::DistillArgs* a, void* workspace, size_t bytes, double** state) {
  const lp::DistillWorkspace w = lp::distill_workspace_layout(a->T, a->V_true, a->dtype);
  if (!workspace || !aligned(workspace, 256) || bytes < w.total) return false;
  char* base = static_cast<char*>(workspace);
  a->part_m = reinterpret_cast<float*>(base + w.off_m);
  a->part_s = reinterpret_cast<double*>(base + w.off_s);
  *state = reinterpret_cast<double*>(base + w.off_state);
  return true;
}

}  // namespace

extern "C" {

lp_status lp_distill_forward(const void* logits, int64_t ld, int32_t dtype, int64_t T,
                             int64_t V_true, const int64_t* teacher_ids, const float* teacher,
                             int64_t K, float temperature, uint32_t flags, float* out_loss,
                             double* row_state, int32_t* bad_rows, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  lp::DistillArgs a;
  bool go;
  const lp_status st = distill_args(logits, ld, dtype, T, V_true, V_true, teacher_ids, teacher, K,
                                    temperature, flags, &a, &go);
  if (st != LP_OK || !go) return st;
  double* unused;
  if (!out_loss || !aligned(out_loss, 4) || !aligned(row_state, 8) || !aligned(bad_rows, 4) ||
      !distill_workspace(&a, workspace, workspace_bytes, &unused))
    return LP_EINVAL;
  a.out_loss = out_loss;
  a.state = row_state;
  a.bad_rows = bad_rows;
  return lp::launch_distill_forward(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

lp_status lp_distill_backward(const void* logits, int64_t ld, int32_t dtype, int64_t T,
                              int64_t V_true, int64_t V_columns, const int64_t* teacher_ids,
                              const float* teacher, int64_t K, float temperature, uint32_t flags,
                              const double* row_state, const float* grad_loss, void* grad_logits,
                              int64_t ld_grad, hipStream_t stream) {
  if (ld_grad < V_columns) return LP_EINVAL;
  lp::DistillArgs a;
  bool go;
  const lp_status st = distill_args(logits, ld, dtype, T, V_true, V_columns, teacher_ids, teacher,
                                    K, temperature, flags, &a, &go);
  if (st != LP_OK || !go) return st;
  if (!row_state || !grad_loss || !grad_logits || !aligned(row_state, 8) ||
      !aligned(grad_loss, 4) || !aligned(grad_logits, size_of(dtype)))
    return LP_EINVAL;
  a.state_in = row_state;
  a.grad = grad_loss;
  a.out_grad = grad_logits;
  a.ld_grad = ld_grad;
  return lp::launch_distill_backward(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

lp_status lp_distill_step(const void* logits, int64_t ld, int32_t dtype, int64_t T, int64_t V_true,
                          int64_t V_columns, const int64_t* teacher_ids, const float* teacher,
                          int64_t K, float temperature, uint32_t flags, const float* weight,
                          float* out_loss, void* grad_logits, int64_t ld_grad, int32_t* bad_rows,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (ld_grad < V_columns) return LP_EINVAL;
  lp::DistillArgs a;
  bool go;
  const lp_status st = distill_args(logits, ld, dtype, T, V_true, V_columns, teacher_ids, teacher,
                                    K, temperature, flags, &a, &go);
  if (st != LP_OK || !go) return st;
  double* state;
  if (!weight || !out_loss || !grad_logits || !aligned(weight, 4) || !aligned(out_loss, 4) ||
      !aligned(grad_logits, size_of(dtype)) || !aligned(bad_rows, 4) ||
      !distill_workspace(&a, workspace, workspace_bytes, &state))
    return LP_EINVAL;
  a.out_loss = out_loss;
  a.state = state;
  a.state_in = state;
  a.grad = weight;
  a.out_grad = grad_logits;
  a.ld_grad = ld_grad;
  a.bad_rows = bad_rows;
  return lp::launch_distill_step(a, stream) == hipSuccess ? LP_OK : LP_EHIP;
}

}  // extern "C"
