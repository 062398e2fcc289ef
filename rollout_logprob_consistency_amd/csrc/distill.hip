// Distillation from a teacher's top logits, forward and backward
// (lp_distill_*): loss = sum_k q_k (ln q_k - ln p[i_k]) with p = softmax(z /
// tau) over the vocabulary, gradient (Q p_v - q_v) / tau.
//
// Forward: one pass over the logits leaves a maximum m and a sum of exp((z - m)
// / tau) for every wave's part of a slice; a merge, one wave per row, joins the
// parts in order, evaluates the K teacher terms in fp64 and keeps four numbers
// a row. Backward: one pass writes the dense part a exp((z - M) / tau), then
// the few places the teacher names are written again with their full value.
// A step over many rows does all of it in one workgroup per row, whose second
// pass finds the row in the Infinity Cache. Parts, their order and the merge
// are the same in both, so the results are too. All of it is bound by the
// logits' bytes.
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
  const size_t parts = (size_t)T * (size_t)s.n;
  w.off_s = up(parts * sizeof(float));
  w.off_state = w.off_s + up(parts * sizeof(double));
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
                                           int64_t end, int tid) {
  const typename D::Raw* p = row + begin + tid * D::kVec;
  if (end - begin == (int64_t)kDistillGroups * kDistillThreads * D::kVec) {
#pragma unroll
    for (int j = 0; j < kDistillGroups; ++j) g[j] = load_whole<D>(p + j * kDistillThreads * D::kVec);
  } else {
#pragma unroll
    for (int j = 0; j < kDistillGroups; ++j)
      g[j] = load_group<D>(row, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end);
  }
}

// A wave's part of a slice: its maximum and sum. The groups are held in
// registers, so the exponentials need no running maximum.
struct Part {
  float m;
  double s;
};
template <class D>
__device__ __forceinline__ Part part_of(Group<D> (&g)[kDistillGroups], float scale2) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j)
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) m = fmaxf(m, g[j].get(i));
  m = wave_max_f32(m);
  // Masked tokens alone sum to 0 (exp(-inf - 0)); a NaN stays a NaN.
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j) {
    g[j].fresh();
#pragma unroll
    for (int i = 0; i < D::kVec; ++i)
      s += __builtin_amdgcn_exp2f((g[j].get(i) - base) * scale2);
  }
  return {m, wave_sum((double)s)};
}

// The parts of a slice's waves, in order.
__device__ __forceinline__ Part join_waves(const Part* w, double inv_tau) {
  float m = w[0].m;
#pragma unroll
  for (int i = 1; i < kDistillWaves; ++i) m = fmaxf(m, w[i].m);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kDistillWaves; ++i)
    // w.m = -inf: nothing but masked tokens (sum 0) or a NaN among them.
    s += w[i].m == -INFINITY ? w[i].s
                             : w[i].s * exp_f64(((double)w[i].m - (double)m) * inv_tau);
  return {m, s};
}

template <class D>
__global__ __launch_bounds__(kDistillThreads) void distill_partial_kernel(DistillArgs a,
                                                                          int64_t row0) {
  using Raw = typename D::Raw;
  const Place at = place_of(row0, a.slices.n);
  const Raw* row = static_cast<const Raw*>(a.logits) + at.row * a.ld;
  const int64_t begin = (int64_t)at.slice * a.slices.len;
  const int64_t end = min(begin + a.slices.len, a.V_true);
  Group<D> g[kDistillGroups];
  load_slice<D>(g, row, begin, end, threadIdx.x);
  const Part p = part_of<D>(g, a.scale2);
  __shared__ Part sh[kDistillWaves];
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = p;
  __syncthreads();
  if (threadIdx.x == 0) {
    const Part all = join_waves(sh, a.inv_tau);
    const int64_t i = at.row * a.slices.n + at.slice;
    a.part_m[i] = all.m;
    a.part_s[i] = all.s;
  }
}

// What the backward pass needs of a row.
struct RowState {
  double M, S, norm, Q;  // maximum, sum, ln of the teacher's normaliser, sum of q
};

// One wave, one row: n slices' parts joined, teacher terms, loss and row state. All in
// fp64: the loss is a small difference of large terms near the teacher. `z` are
// the row's logits. Lane 0 writes loss, state and the bad-row count.
template <class D>
__device__ __forceinline__ RowState merge_row(const DistillArgs& a, int64_t row,
                                              const float* pm, const double* ps, int n,
                                              const typename D::Raw* z) {
  const int lane = threadIdx.x & 63;
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
  double norm = 0.0;
  if (!a.logprobs && !none && !bad && !nan) {
    double ts = 0.0;
    for (int k = lane; k < a.K; k += 64)
      if (ids[k] != -1) ts += exp_f64((double)x[k] * scale - tmax);
    norm = tmax + log(wave_sum(ts));
  }
  double Q = 0.0, loss = 0.0;
  if (!none && !bad && !nan) {
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
  return {M, S, norm, Q};
}

constexpr int kMergeWaves = 4;  // rows per merge workgroup

template <class D>
__global__ __launch_bounds__(kMergeWaves * 64) void distill_merge_kernel(DistillArgs a,
                                                                         int64_t row0,
                                                                         int64_t rows) {
  const int64_t r = (int64_t)blockIdx.x * kMergeWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int64_t row = row0 + r;
  const int n = a.slices.n;
  merge_row<D>(a, row, a.part_m + row * n, a.part_s + row * n, n,
               static_cast<const typename D::Raw*>(a.logits) + row * a.ld);
}

// The dense part of the gradient: c exp((z - m) / tau) for groups of a slice.
template <class D>
__device__ __forceinline__ void dense_groups(Group<D> (&g)[kDistillGroups], float m, float c,
                                             float scale2) {
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j)
#pragma unroll
    for (int i = 0; i < D::kVec; ++i)
      g[j].set(i, D::round(c * __builtin_amdgcn_exp2f((g[j].get(i) - m) * scale2)));
}

// The teacher's entries of the places [begin, end) of a row, for a workgroup of
// kThreads: taken before anything is overwritten (the output may be the
// logits' own buffer), written after the dense part.
template <class D, int kThreads>
struct Entries {
  static constexpr int kMine = (LP_DISTILL_MAX_K + kThreads - 1) / kThreads;
  float z[kMine];

  // at: place in the slice or -1, and q, of every entry (LDS).
  __device__ __forceinline__ void take(const DistillArgs& a, int64_t row,
                                       const typename D::Raw* logits, int64_t begin, int64_t end,
                                       double norm, int32_t* at, double* q) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int k = j * kThreads + (int)threadIdx.x;
      if (k < a.K) {
        const int64_t id = a.ids[row * a.K + k];
        const bool here = id >= begin && id < end;
        at[k] = here ? (int32_t)(id - begin) : -1;
        if (here) {
          z[j] = D::value(logits[id]);
          q[k] = exp_f64((double)a.teacher[row * a.K + k] * (a.logprobs ? 1.0 : a.inv_tau) - norm);
        }
      } else if (k < LP_DISTILL_MAX_K) {
        at[k] = -1;  // read in fours past K
      }
    }
  }
  __device__ __forceinline__ void write(const DistillArgs& a, const RowState& s, float grad,
                                        typename D::Raw* out, const int32_t* at,
                                        const double* q) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int k = j * kThreads + (int)threadIdx.x;
      if (k < a.K && at[k] >= 0) {
        // An id that occurs again adds up; its first entry writes the sum. Four
        // entries a read tell whether there is one (step, 2 304 bf16 rows of
        // 6 000, K = 256: 55 us, by single entries 57 us).
        const int32_t mine = at[k];
        double sum = q[k];
        bool first = true, again = false;
        for (int i = 0; i < a.K; i += 4) {
          const int4 v = *reinterpret_cast<const int4*>(at + i);
          again |= (v.x == mine && i != k) | (v.y == mine && i + 1 != k) |
                   (v.z == mine && i + 2 != k) | (v.w == mine && i + 3 != k);
        }
        if (again) {
          sum = 0.0;
          for (int i = 0; i < a.K; ++i)
            if (at[i] == mine) {
              first &= i >= k;
              sum += q[i];
            }
        }
        if (first) {
          const double p = exp_f64(((double)z[j] - s.M) * a.inv_tau) / s.S;
          out[mine] = D::round((float)((double)grad * a.inv_tau * (s.Q * p - sum)));
        }
      }
    }
  }
};

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
  const RowState s = {state[0], state[1], state[2], state[3]};
  const float grad = a.grad[at.row];
  if (at.slice == a.slices.n - 1)  // columns behind the vocabulary
    for (int64_t i = a.V_true + tid; i < a.V_columns; i += kDistillThreads) out[i] = D::round(0.0f);

  Group<D> g[kDistillGroups];
  if (grad == 0.0f || s.Q == 0.0) {
    g[0] = {{0, 0, 0, 0}};
    for (int j = 0; j < kDistillGroups; ++j)
      store_group<D>(out, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end, g[0]);
    return;
  }
  load_slice<D>(g, row, begin, end, tid);
  __shared__ __align__(16) int32_t sh_at[LP_DISTILL_MAX_K];
  __shared__ double sh_q[LP_DISTILL_MAX_K];
  Entries<D, kDistillThreads> entries;
  entries.take(a, at.row, row, begin, end, s.norm, sh_at, sh_q);
  __syncthreads();
  dense_groups<D>(g, (float)s.M, (float)((double)grad * a.inv_tau * s.Q / s.S), a.scale2);
#pragma unroll
  for (int j = 0; j < kDistillGroups; ++j)
    store_group<D>(out, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end, g[j]);
  __syncthreads();  // the dense values are in place before any is written again
  entries.write(a, s, grad, out + begin, sh_at, sh_q);
}

// Measured on bf16 rows of 151 936: step over 2 048 rows 316 us (3.9 TB/s of
// the bytes it cannot do without) against 361 us by the three kernels above,
// loss of 4 096 rows 211 us (5.9 TB/s) against 267 us.
//
// Loss (and gradient) of one row: kRowWaves / kDistillWaves slices at a time,
// each by as many threads, in the places and the order of the kernels above.
template <class D, bool kGradient>
__global__ __launch_bounds__(kRowWaves * 64, 8) void distill_row_kernel(DistillArgs a,
                                                                        int64_t row0) {
  using Raw = typename D::Raw;
  constexpr int kThreads = kRowWaves * 64, kTeams = kRowWaves / kDistillWaves;
  __shared__ Part sh_waves[kRowMaxSlices * kDistillWaves];
  __shared__ float sh_m[kRowMaxSlices];
  __shared__ double sh_s[kRowMaxSlices];
  __shared__ RowState sh_state;
  __shared__ __align__(16) int32_t sh_at[LP_DISTILL_MAX_K];
  __shared__ double sh_q[LP_DISTILL_MAX_K];
  const int64_t r = row0 + blockIdx.x;
  const Raw* row = static_cast<const Raw*>(a.logits) + r * a.ld;
  Raw* out = static_cast<Raw*>(a.out_grad) + r * a.ld_grad;
  const int team = threadIdx.x / kDistillThreads, tid = threadIdx.x % kDistillThreads;
  for (int i = team; i < a.slices.n; i += kTeams) {
    const int64_t begin = (int64_t)i * a.slices.len;
    Group<D> g[kDistillGroups];
    load_slice<D>(g, row, begin, min(begin + a.slices.len, a.V_true), tid);
    const Part p = part_of<D>(g, a.scale2);
    if ((tid & 63) == 0) sh_waves[i * kDistillWaves + (tid >> 6)] = p;
  }
  __syncthreads();
  if (threadIdx.x < a.slices.n) {
    const Part p = join_waves(sh_waves + threadIdx.x * kDistillWaves, a.inv_tau);
    sh_m[threadIdx.x] = p.m;
    sh_s[threadIdx.x] = p.s;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const RowState s = merge_row<D>(a, r, sh_m, sh_s, a.slices.n, row);
    if (threadIdx.x == 0) sh_state = s;
  }
  if constexpr (!kGradient) return;
  __syncthreads();
  const RowState s = sh_state;
  const float grad = a.grad[r];
  for (int64_t i = a.V_true + threadIdx.x; i < a.V_columns; i += kThreads) out[i] = D::round(0.0f);
  const bool none = grad == 0.0f || s.Q == 0.0;
  Entries<D, kThreads> entries;
  if (!none) entries.take(a, r, row, 0, a.V_true, s.norm, sh_at, sh_q);
  __syncthreads();
  const float c = (float)((double)grad * a.inv_tau * s.Q / s.S), m = (float)s.M;
  for (int i = team; i < a.slices.n; i += kTeams) {
    const int64_t begin = (int64_t)i * a.slices.len;
    const int64_t end = min(begin + a.slices.len, a.V_true);
    Group<D> g[kDistillGroups];
    if (none) {
#pragma unroll
      for (int j = 0; j < kDistillGroups; ++j) g[j] = {{0, 0, 0, 0}};
    } else {
      load_slice<D>(g, row, begin, end, tid);
      dense_groups<D>(g, m, c, a.scale2);
    }
#pragma unroll
    for (int j = 0; j < kDistillGroups; ++j)
      store_group<D>(out, begin + (int64_t)(j * kDistillThreads + tid) * D::kVec, end, g[j]);
  }
  if (none) return;
  __syncthreads();  // the dense values are in place before any is written again
  entries.write(a, s, grad, out, sh_at, sh_q);
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
  if (forward && a.T >= kRowMinRows && a.slices.n >= kRowMinSlices && a.slices.n <= kRowMaxSlices) {
    const int64_t most = rows_per_dispatch(1, kRowWaves * 64);
    for (int64_t r = 0; r < a.T; r += most) {
      const dim3 rows((uint32_t)std::min(most, a.T - r));
      if (backward) distill_row_kernel<D, true><<<rows, kRowWaves * 64, 0, stream>>>(a, r);
      else distill_row_kernel<D, false><<<rows, kRowWaves * 64, 0, stream>>>(a, r);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
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
