// Distillation from a teacher's top logits, forward and backward
// (lp_distill_*): loss = sum_k q_k (ln q_k - ln p[i_k]) with p = softmax(z /
// tau) over the vocabulary, gradient (Q p_v - q_v) / tau.
//
// Forward: one pass over the logits leaves per slice the maximum m and the
// sum of exp((z - m) / tau); a merge, one wave per row, joins the slices in
// order, evaluates the K teacher terms in fp64 and keeps four numbers a row.
// Backward: one pass writes the dense part a exp((z - M) / tau), then the few
// places the teacher names are written again with their full value.
// Both directions are bound by the logits' bytes.
#include <algorithm>

#include "logits_internal.h"

namespace lp {

DistillSlices distill_slices(int64_t V_true, int32_t dtype) {
  const int64_t vec = 16 / dtype_bytes(dtype);
  const int64_t most = (int64_t)kDistillThreads * kDistillGroups * vec;
  DistillSlices s;
  s.n = (int32_t)((V_true + most - 1) / most);
  const int64_t even = (V_true + s.n - 1) / s.n;
  s.len = (even + vec - 1) / vec * vec;
  return s;
}

DistillWorkspace distill_workspace_layout(int64_t T, int64_t V_true, int32_t dtype) {
  const DistillSlices s = distill_slices(V_true, dtype);
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  DistillWorkspace w;
  w.off_m = 0;
  w.off_s = up((size_t)T * (size_t)s.n * sizeof(float));
  w.off_state = w.off_s + up((size_t)T * (size_t)s.n * sizeof(double));
  w.total = w.off_state + up((size_t)T * 4 * sizeof(double));
  return w;
}

namespace {

// Row and slice of a workgroup: slices of a row are neighbours.
struct Place {
  int64_t row;
  int32_t slice;
};
__device__ __forceinline__ Place place_of(int64_t row0, int32_t n) {
  const uint32_t b = blockIdx.x;
  const uint32_t r = b / (uint32_t)n;
  return {row0 + r, (int32_t)(b - r * (uint32_t)n)};
}

// A thread's groups of the slice [begin, end), -inf behind its end.
template <class D>
__device__ __forceinline__ void load_slice(Group<D> (&g)[kDistillGroups],
                                           const typename D::Raw* row, int64_t begin,
                                           int64_t end) {
  const typename D::Raw* p = row + begin + threadIdx.x * D::kVec;
  if (end - begin == (int64_t)kDistillGroups * kDistillThreads * D::kVec) {
#pragma unroll
    for (int j = 0; j < kDistillGroups; ++j) g[j] = load_whole<D>(p + j * kDistillThreads * D::kVec);
  } else {
#pragma unroll
    for (int j = 0; j < kDistillGroups; ++j)
      g[j] = load_group<D>(row, begin + (int64_t)(j * kDistillThreads + threadIdx.x) * D::kVec, end);
  }
}

// One slice's maximum and sum. The slice is held in registers, so its
// exponentials need no running maximum.
template <class D>
__global__ __launch_bounds__(kDistillThreads) void distill_partial_kernel(DistillArgs a,
                                                                          int64_t row0) {
  using Raw = typename D::Raw;
  const Place at = place_of(row0, a.slices.n);
  const Raw* row = static_cast<const Raw*>(a.logits) + at.row * a.ld;
  const int64_t begin = (int64_t)at.slice * a.slices.len;
  const int64_t end = min(begin + a.slices.len, a.V_true);
  const int tid = threadIdx.x;
  Group<D> g[kDistillGroups];
  load_slice<D>(g, row, begin, end);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j)
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) m = fmaxf(m, g[j].get(i));
  __shared__ float sh_m[kDistillThreads / 64];
  __shared__ double sh_s[kDistillThreads / 64];
  const float wm = (float)wave_max((double)m);
  if ((tid & 63) == 0) sh_m[tid >> 6] = wm;
  __syncthreads();
  m = sh_m[0];
#pragma unroll
  for (int i = 1; i < kDistillThreads / 64; ++i) m = fmaxf(m, sh_m[i]);
  // A slice of masked tokens sums to 0 (exp(-inf - 0)); a NaN stays a NaN.
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j) {
    g[j].fresh();
#pragma unroll
    for (int i = 0; i < D::kVec; ++i)
      s += __builtin_amdgcn_exp2f((g[j].get(i) - base) * a.scale2);
  }
  const double ws = wave_sum((double)s);
  if ((tid & 63) == 0) sh_s[tid >> 6] = ws;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int i = 0; i < kDistillThreads / 64; ++i) sum += sh_s[i];
    const int64_t p = at.row * a.slices.n + at.slice;
    a.part_m[p] = m;
    a.part_s[p] = sum;
  }
}

constexpr int kMergeWaves = 4;  // rows per merge workgroup

// One wave per row: slices joined, teacher terms, loss and row state. All in
// fp64: the loss is a small difference of large terms near the teacher.
template <class D>
__global__ __launch_bounds__(kMergeWaves * 64) void distill_merge_kernel(DistillArgs a,
                                                                         int64_t row0,
                                                                         int64_t rows) {
  const int64_t r = (int64_t)blockIdx.x * kMergeWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int64_t row = row0 + r;
  const int lane = threadIdx.x & 63;
  const int32_t n = a.slices.n;
  const float* pm = a.part_m + row * n;
  const double* ps = a.part_s + row * n;
  double M = -INFINITY;
  for (int i = lane; i < n; i += 64) M = fmax(M, (double)pm[i]);
  M = wave_max(M);
  double S = 0.0;
  for (int i = lane; i < n; i += 64) {
    const double m = (double)pm[i];
    // m = -inf: nothing but masked tokens (sum 0) or a NaN among them.
    S += m == -INFINITY ? ps[i] : ps[i] * exp_f64((m - M) * a.inv_tau);
  }
  S = wave_sum(S);

  const int64_t* ids = a.ids + row * a.K;
  const float* x = a.teacher + row * a.K;
  const double scale = a.logprobs ? 1.0 : a.inv_tau;
  double tmax = -INFINITY;
  bool bad = false, nan = false;
  for (int k = lane; k < a.K; k += 64) {
    const int64_t id = ids[k];
    if (id == -1) continue;
    bad |= id < 0 || id >= a.V_true;
    const float xk = x[k];
    nan |= isnan(xk) || xk == INFINITY;
    tmax = fmax(tmax, (double)xk * scale);
  }
  bad = __ballot(bad) != 0;
  nan = __ballot(nan) != 0;
  tmax = wave_max(tmax);
  const bool none = tmax == -INFINITY && !bad && !nan;  // no entry with weight
  double norm = 0.0;  // ln of the teacher's normaliser
  if (!a.logprobs && !none && !bad && !nan) {
    double ts = 0.0;
    for (int k = lane; k < a.K; k += 64)
      if (ids[k] != -1) ts += exp_f64((double)x[k] * scale - tmax);
    norm = tmax + log(wave_sum(ts));
  }
  double Q = 0.0, loss = 0.0;
  if (!none && !bad && !nan) {
    const typename D::Raw* z = static_cast<const typename D::Raw*>(a.logits) + row * a.ld;
    const double lnS = log(S);
    for (int k = lane; k < a.K; k += 64) {
      const int64_t id = ids[k];
      if (id == -1) continue;
      const double lq = (double)x[k] * scale - norm;
      const double q = exp_f64(lq);
      if (q > 0.0) {
        Q += q;
        loss += q * (lq - (((double)D::value(z[id]) - M) * a.inv_tau - lnS));
      }
    }
    Q = wave_sum(Q);
    loss = wave_sum(loss);
    if (Q == 0.0) loss = 0.0;
  }
  if (bad || nan) Q = loss = NAN;
  if (lane == 0) {
    a.out_loss[row] = (float)loss;
    if (a.state) {
      double* s = a.state + row * 4;
      s[0] = M;
      s[1] = S;
      s[2] = norm;
      s[3] = Q;
    }
    if (bad && a.bad_rows) atomicAdd(a.bad_rows, 1);
  }
}

// grad_logits of one slice of one row.
template <class D>
__global__ __launch_bounds__(kDistillThreads) void distill_backward_kernel(DistillArgs a,
                                                                           int64_t row0) {
  using Raw = typename D::Raw;
  const Place at = place_of(row0, a.slices.n);
  const Raw* row = static_cast<const Raw*>(a.logits) + at.row * a.ld;
  Raw* out = static_cast<Raw*>(a.out_grad) + at.row * a.ld_grad;
  const int64_t begin = (int64_t)at.slice * a.slices.len;
  const int64_t end = min(begin + a.slices.len, a.V_true);
  const int tid = threadIdx.x;
  const double* state = a.state_in + at.row * 4;
  const double M = state[0], S = state[1], norm = state[2], Q = state[3];
  const float grad = a.grad[at.row];
  if (at.slice == a.slices.n - 1)  // columns behind the vocabulary
    for (int64_t i = a.V_true + tid; i < a.V_columns; i += kDistillThreads) out[i] = D::round(0.0f);

  Group<D> g[kDistillGroups];
  if (grad == 0.0f || Q == 0.0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) g[0].w[j] = 0;
    for (int j = 0; j < kDistillGroups; ++j)
      store_group<D>(out, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end, g[0]);
    return;
  }
  load_slice<D>(g, row, begin, end);

  // The teacher's entries of this slice, before anything is overwritten (the
  // output may be the logits' own buffer): offset in the slice or -1, and q.
  __shared__ int32_t sh_at[LP_DISTILL_MAX_K];
  __shared__ double sh_q[LP_DISTILL_MAX_K];
  constexpr int kMine = LP_DISTILL_MAX_K / kDistillThreads;
  float z[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int k = j * kDistillThreads + tid;
    if (k < a.K) {
      const int64_t id = a.ids[at.row * a.K + k];
      const bool here = id >= begin && id < end;
      sh_at[k] = here ? (int32_t)(id - begin) : -1;
      if (here) {
        z[j] = D::value(row[id]);
        sh_q[k] = exp_f64((double)a.teacher[at.row * a.K + k] *
                              (a.logprobs ? 1.0 : a.inv_tau) - norm);
      }
    }
  }
  __syncthreads();

  const float m = (float)M;
  const float c = (float)((double)grad * a.inv_tau * Q / S);
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j) {
#pragma unroll
    for (int i = 0; i < D::kVec; ++i)
      g[j].set(i, D::round(c * __builtin_amdgcn_exp2f((g[j].get(i) - m) * a.scale2)));
    store_group<D>(out, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end, g[j]);
  }
  __syncthreads();  // the dense values are in place before any is written again

#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int k = j * kDistillThreads + tid;
    if (k < a.K && sh_at[k] >= 0) {
      // An id that occurs again adds up; its first entry writes the sum.
      const int32_t mine = sh_at[k];
      double q = 0.0;
      bool first = true;
      for (int i = 0; i < a.K; ++i)
        if (sh_at[i] == mine) {
          first &= i >= k;
          q += sh_q[i];
        }
      if (first) {
        const double p = exp_f64(((double)z[j] - M) * a.inv_tau) / S;
        out[begin + mine] = D::round((float)((double)grad * a.inv_tau * (Q * p - q)));
      }
    }
  }
}

// Rows whose workgroups (`n` each of `threads`) fit one dispatch.
int64_t rows_per_dispatch(int64_t n, int64_t threads) {
  return std::max<int64_t>(1, kMaxDispatchItems / (n * threads));
}

template <class D>
hipError_t forward_rows(const DistillArgs& a, int64_t row0, int64_t rows, hipStream_t stream) {
  distill_partial_kernel<D><<<dim3((uint32_t)(rows * a.slices.n)), kDistillThreads, 0, stream>>>(
      a, row0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  distill_merge_kernel<D><<<dim3((uint32_t)((rows + kMergeWaves - 1) / kMergeWaves)),
                            kMergeWaves * 64, 0, stream>>>(a, row0, rows);
  return hipGetLastError();
}

template <class D>
hipError_t backward_rows(const DistillArgs& a, int64_t row0, int64_t rows, hipStream_t stream) {
  distill_backward_kernel<D><<<dim3((uint32_t)(rows * a.slices.n)), kDistillThreads, 0, stream>>>(
      a, row0);
  return hipGetLastError();
}

template <class D>
hipError_t run(const DistillArgs& a, bool forward, bool backward, hipStream_t stream) {
  const int64_t most = rows_per_dispatch(a.slices.n, kDistillThreads);
  for (int64_t r = 0; r < a.T; r += most) {
    const int64_t rows = std::min(most, a.T - r);
    hipError_t e = hipSuccess;
    if (forward) e = forward_rows<D>(a, r, rows, stream);
    if (e == hipSuccess && backward) e = backward_rows<D>(a, r, rows, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t dispatch(const DistillArgs& a, bool forward, bool backward, hipStream_t stream) {
  switch (a.dtype) {
    case LP_F32: return run<F32>(a, forward, backward, stream);
    case LP_BF16: return run<BF16>(a, forward, backward, stream);
    default: return run<F16>(a, forward, backward, stream);
  }
}

}  // namespace

hipError_t launch_distill_forward(const DistillArgs& a, hipStream_t stream) {
  return dispatch(a, true, false, stream);
}

hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t stream) {
  return dispatch(a, false, true, stream);
}

hipError_t launch_distill_step(const DistillArgs& a, hipStream_t stream) {
  return dispatch(a, true, true, stream);
}

}  // namespace lp
