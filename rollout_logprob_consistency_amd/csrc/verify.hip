// Verification of drafted tokens (lp_verify).
//
// With p_j what the target's row j would be drawn from and q_j the draft's, the
// drafted token x_j is accepted where u_j q_j(x_j) < p_j(x_j); the first one that
// is not is replaced by a draw from max(p - q, 0), and behind the last accepted
// one a token is drawn from p. Either is found in index order: the least token
// through which the weights pass u times their sum.
//
// The rows' limits (where the kept tokens end, and what they weigh) come from
// the draw's own kernels. Two more launches end the call: residual_kernel judges
// the drafts (each workgroup for itself: a few loads, against a launch more) and
// sums the weights of the one row, or two, that a sequence's last token is drawn
// from, by stretches of a wave's width; final_kernel finds the stretch and the
// token in it. (One launch whose last workgroup of a sequence ends it took longer:
// 147 us against 91 us for 128 sequences of 151 936, as the fences that it needs
// empty the L2 caches.)
#include <algorithm>

#include "select_row.h"

namespace lp {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / 64;
// Tokens of a stretch: one group a lane.
template <class D>
constexpr int kStretch = 64 * D::kVec;
constexpr int kMostStretches = LP_SELECT_MAX_VOCAB / kStretch<F32>;
constexpr int kSumsPerThread = kMostStretches / kVerifyThreads;
int64_t stretches_of(int64_t V, int32_t dtype) {
  const int64_t n = 64 * (16 / dtype_bytes(dtype));
  return (V + n - 1) / n;
}
// Workgroups that run at once: of residual_kernel six on each of 256 CUs, of
// collect_kernel three.
constexpr int64_t kVerifyPlaces = 1536;
// Slices of all rows. More of them shorten the longest row's way (64 sequences of up
// to 4 drafts, settings of their own: 205 us with 768, 146 with 1 280, 141 with 2 048,
// 142 with 3 000) until joining them takes longer (nucleus rows, 64 sequences of 4:
// 205, 208, 214 and 224 us).
constexpr int64_t kLimitPlaces = 2048;
constexpr int64_t kWholePlaces = 768;
static_assert(LP_VERIFY_MAX_DRAFTS < 64, "a wave holds a sequence's positions");

// The distribution that a row would be drawn from: token v is kept where (z,
// lower index) is no less than the last kept token's.
struct Dist {
  double base, c, log2_kept;  // c = log2(e) / tau
  float z_last;
  int v_last;

  __device__ __forceinline__ bool near(float z) const { return z >= z_last; }
  __device__ __forceinline__ bool keeps(float z, int v) const {
    return z > z_last || (z == z_last && v <= v_last);
  }
  // Whether every token is kept and offset() has its digits: 2^-42 of a weight.
  __device__ __forceinline__ bool plain() const {
    return z_last == -3.4028234663852886e38f && v_last == INT32_MAX && fabs(offset()) < 0x1p11;
  }
  // prob(z) is 2^(z c + offset()).
  __device__ __forceinline__ double offset() const { return -base * c - log2_kept; }
  // Of a finite token that it keeps.
  __device__ __forceinline__ double prob(float z) const {
    return exp2_f64(fma((double)z - base, c, -log2_kept));
  }
};

struct Sequence {
  int64_t b;
  int count;     // drafts
  int accepted;  // of them; -1: a sequence that has no verdict
  double inv_tau;  // 1 where it is greedy
};

// The target's (at <= count) or the draft's (at < count) row of a sequence.
__device__ __forceinline__ int64_t target_row(const VerifyArgs& a, int64_t b, int at) {
  return b * (a.rows.drafts + 1) + at;
}
__device__ __forceinline__ int64_t draft_limit(const VerifyArgs& a, int64_t b, int at) {
  return a.rows.seqs * (a.rows.drafts + 1) + b * a.rows.drafts + at;
}
__device__ __forceinline__ Dist dist_of(const VerifyArgs& a, const Sequence& s, int64_t limit) {
  const SelectLimit l = a.rows.limits[limit];
  // (No limit, and one that is a value alone, hold the lowest place of an index.)
  const bool all = l.last == 0;
  return {l.base, kLog2E * s.inv_tau, l.ln_kept * kLog2E,
          all ? -3.4028234663852886e38f : token_logit(l.last),
          all || (uint32_t)l.last == 0 ? INT32_MAX : token_index(l.last)};
}

template <class D>
__device__ __forceinline__ float logit_at(const void* logits, int64_t ld, int64_t row, int64_t v) {
  return D::value(read_global(static_cast<const typename D::Raw*>(logits), row * ld + v));
}

__device__ __forceinline__ Sequence sequence_of(const VerifyArgs& a, int64_t b) {
  const SelectArgs& r = a.rows;
  const float tau = r.temperatures ? read_global(r.temperatures, b) : r.temperature;
  return {b, r.draft_counts ? read_global(r.draft_counts, b) : r.drafts, -1,
          tau == 0.0f ? 1.0 : 1.0 / (double)tau};
}

// How far a sequence's drafts are accepted: lane j looks at position j. Every
// wave of a workgroup finds the same.
template <class D>
__device__ __forceinline__ Sequence judge(const VerifyArgs& a, int64_t b) {
  const SelectArgs& r = a.rows;
  const int lane = threadIdx.x & 63;
  Sequence s = sequence_of(a, b);
  if (s.count < 0 || s.count > r.drafts) return s;
  const int width = r.drafts + 1;
  bool bad = lane == 63 && isnan(read_global(a.u, b * width + r.drafts)), passed = false;
  if (lane <= s.count) {
    bad |= r.limits[target_row(a, b, lane)].last == kNoLimit;
    if (lane < s.count) {
      const int64_t id = read_global(a.draft_ids, b * r.drafts + lane);
      const float u = read_global(a.u, b * width + lane);
      bad |= isnan(u) || id < 0 || id >= r.V;
      if (r.draft_logits) bad |= r.limits[draft_limit(a, b, lane)].last == kNoLimit;
      if (!bad) {
        const float z = logit_at<D>(r.logits, r.ld, target_row(a, b, lane), id);
        const Dist p = dist_of(a, s, target_row(a, b, lane));
        const double px = p.keeps(z, (int)id) ? p.prob(z) : 0.0;
        double qx = 1.0;
        if (r.draft_logits) {
          const float y = logit_at<D>(r.draft_logits, r.ld_draft, b * r.drafts + lane, id);
          const Dist q = dist_of(a, s, draft_limit(a, b, lane));
          qx = q.keeps(y, (int)id) ? q.prob(y) : 0.0;
        }
        passed = fmin(fmax((double)u, 0.0), 1.0 - 0x1p-24) * qx < px;
      }
    }
  }
  if (__ballot(bad)) return s;
  const uint64_t rejected = ~__ballot(passed);  // (position `count` is one)
  s.accepted = __ffsll((long long)rejected) - 1;
  return s;
}

// The weights that a sequence's last token is drawn from, in its row.
template <class D>
struct Weights {
  Dist p, q;
  const typename D::Raw* target;
  const typename D::Raw* draft;  // null: there is none
  int64_t gone;                  // the token that weighs nothing, -1: none
  int V;
  bool plain;  // all tokens are kept, on both sides; then their offsets for exp2_900
  double p_off, q_off;

  // With `whole`, p itself.
  __device__ __forceinline__ Weights(const VerifyArgs& a, const Sequence& s, bool whole) {
    const SelectArgs& r = a.rows;
    const int64_t t = target_row(a, s.b, s.accepted);
    p = dist_of(a, s, t);
    target = static_cast<const typename D::Raw*>(r.logits) + t * r.ld;
    draft = nullptr;
    gone = -1;
    V = r.V;
    plain = p.plain();
    p_off = p.offset() + kExp2From;
    q_off = 0.0;
    if (whole || s.accepted == s.count) return;
    const int64_t d = s.b * r.drafts + s.accepted;
    if (r.draft_logits) {
      draft = static_cast<const typename D::Raw*>(r.draft_logits) + d * r.ld_draft;
      q = dist_of(a, s, draft_limit(a, s.b, s.accepted));
      plain = plain && q.plain();
      q_off = q.offset() + kExp2From;
    } else {
      gone = read_global(a.draft_ids, d);  // the draft's whole probability
      plain = false;
    }
  }
  // A lane's logits of a stretch, and their weights; 0 behind the row. A wave whose
  // tokens are all below the last kept one forms no exponentials.
  struct Loaded {
    Group<D> z, y;
    int v;
  };
  __device__ __forceinline__ Loaded load(int stretch) const {
    Loaded l;
    l.v = stretch * kStretch<D> + (int)(threadIdx.x & 63) * D::kVec;
    l.z = load_group<D>(target, l.v, V);
    l.y = l.z;
    if (draft) l.y = load_group<D>(draft, l.v, V);
    return l;
  }
  // Where every token is kept there is nothing to compare (128 sequences of 151 936
  // bf16 tokens: 35 us, with the comparisons 60 us).
  __device__ __forceinline__ void weigh(const Loaded& l, double (&w)[D::kVec]) const {
    if (plain) {
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) w[i] = exp2_900(fma((double)l.z.get(i), p.c, p_off));
      if (!draft) return;
#pragma unroll
      for (int i = 0; i < D::kVec; ++i)
        w[i] = fmax(w[i] - exp2_900(fma((double)l.y.get(i), q.c, q_off)), 0.0);
      return;
    }
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) {
      const float a = l.z.get(i), b = l.y.get(i);  // (-inf behind the row)
      w[i] = 0.0;
      if (__ballot(p.near(a)) == 0) continue;
      const bool kept = p.keeps(a, l.v + i) && l.v + i != gone;
      w[i] = kept ? p.prob(a) : 0.0;
      if (!draft || __ballot(kept && q.near(b)) == 0) continue;
      w[i] = kept && q.keeps(b, l.v + i) ? fmax(w[i] - q.prob(b), 0.0) : w[i];
    }
  }
  __device__ __forceinline__ double sum(const Loaded& l) const {
    double x[D::kVec], s = 0.0;
    weigh(l, x);
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) s += x[i];
    return wave_sum(s);
  }
  // The sums of the stretches first, first + step, ..., the next one's logits in
  // flight.
  __device__ __forceinline__ void sums(int first, int step, double* out) const {
    const int n = (V + kStretch<D> - 1) / kStretch<D>;
    if (first >= n) return;
    Loaded now = load(first);
    for (int i = first; i < n; i += step) {
      Loaded next = now;
      if (i + step < n) next = load(i + step);
      const double s = sum(now);
      if ((threadIdx.x & 63) == 0) out[i] = s;
      now = next;
    }
  }
};

template <class D>
__global__ __launch_bounds__(kVerifyThreads) void residual_kernel(VerifyArgs a, int parts) {
  const int64_t b = blockIdx.x / (uint32_t)parts;
  const int part = (int)(blockIdx.x % (uint32_t)parts);
  const Sequence s = judge<D>(a, b);
  if (part == 0 && threadIdx.x == 0) a.verdicts[b] = s.accepted;
  if (s.accepted < 0) return;
  const int64_t n = (a.rows.V + kStretch<D> - 1) / kStretch<D>;
  Weights<D>(a, s, false)
      .sums(part * kVerifyWaves + (threadIdx.x >> 6), parts * kVerifyWaves, a.sums + b * n);
}

// Exclusive prefix sum over the workgroup.
__device__ __forceinline__ double scan(double v, double* words, double* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  double before = __shfl_up(s, 1);
  if (lane == 0) before = 0.0;
  if (lane == 63) words[wave] = s;
  __syncthreads();
  double base = 0.0, sum = 0.0;
#pragma unroll
  for (int w = 0; w < kVerifyWaves; ++w) {
    if (w == wave) base = sum;
    sum += words[w];
  }
  __syncthreads();
  *total = sum;
  return base + before;
}

struct FinalShared {
  double words[kVerifyWaves], before;
  int stretch, last, token;
};

// The least token through which the weights pass u times their sum, from the
// stretches' sums; -1 where all weigh nothing. Where rounding leaves none, the last
// that weighs.
template <class D>
__device__ __forceinline__ int draw(const Weights<D>& w, double u, const double* sums,
                                    FinalShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int n = (w.V + kStretch<D> - 1) / kStretch<D>;
  const int each = (n + kVerifyThreads - 1) / kVerifyThreads;
  double mine[kSumsPerThread], sum = 0.0, total;
  int last = -1;
#pragma unroll
  for (int i = 0; i < kSumsPerThread; ++i) {
    mine[i] = i < each && tid * each + i < n ? sums[tid * each + i] : 0.0;
    sum += mine[i];
    last = mine[i] > 0.0 ? tid * each + i : last;
  }
  if (tid == 0) {
    sh.stretch = INT32_MAX;
    sh.last = -1;
  }
  double before = scan(sum, sh.words, &total);
  if (!(total > 0.0)) return -1;
  const double want = u * total;
  int first = INT32_MAX;
  double at = before;
#pragma unroll
  for (int i = 0; i < kSumsPerThread; ++i) {
    if (first == INT32_MAX && mine[i] > 0.0 && before + mine[i] > want) {
      first = tid * each + i;
      at = before;
    }
    before += mine[i];
  }
  if (first != INT32_MAX) atomicMin(&sh.stretch, first);
  if (last >= 0) atomicMax(&sh.last, last);
  __syncthreads();
  const int stretch = sh.stretch != INT32_MAX ? sh.stretch : sh.last;
  if (first == stretch) sh.before = at;
  else if (sh.stretch == INT32_MAX && tid == 0) sh.before = total;  // rounding: its last token
  __syncthreads();
  if (tid < 64) {
    double x[D::kVec], s = 0.0;
    const auto l = w.load(stretch);
    w.weigh(l, x);
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) s += x[i];
    double c = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(c, d);
      if (lane >= d) c += o;
    }
    c += sh.before - s;
    int hit = -1, some = -1;
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) {
      c += x[i];
      if (x[i] > 0.0) {
        some = l.v + i;
        if (hit < 0 && c > want) hit = l.v + i;
      }
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(some >= 0);
    const int token = hits ? __shfl(hit, __ffsll((long long)hits) - 1)
                           : __shfl(some, any ? 63 - __clzll((long long)any) : 0);
    if (lane == 0) sh.token = token;
  }
  __syncthreads();
  return sh.token;
}

// A sequence's outputs.
template <class D>
__device__ __forceinline__ void finish(const VerifyArgs& a, const Sequence& s, FinalShared& sh) {
  const SelectArgs& r = a.rows;
  const int tid = threadIdx.x, width = r.drafts + 1;
  const double u =
      fmin(fmax((double)read_global(a.u, s.b * width + r.drafts), 0.0), 1.0 - 0x1p-24);
  double* sums = a.sums + s.b * ((r.V + kStretch<D> - 1) / kStretch<D>);
  int token = draw(Weights<D>(a, s, false), u, sums, sh);
  if (token < 0) {
    // The target has nothing beyond the draft: a token of the target's own.
    const Weights<D> w(a, s, true);
    __syncthreads();
    w.sums(tid >> 6, kVerifyWaves, sums);
    __syncthreads();
    token = draw(w, u, sums, sh);
  }
  if (tid < width) {
    float logprob = 0.0f, processed = 0.0f;
    int64_t t = -1;
    if (tid <= s.accepted) {
      t = tid < s.accepted ? read_global(a.draft_ids, s.b * r.drafts + tid) : token;
      const int64_t row = target_row(a, s.b, tid);
      const SelectLimit l = r.limits[row];
      const double gap = ((double)logit_at<D>(r.logits, r.ld, row, t) - l.base) * s.inv_tau;
      // (A token that holds all the weight: the sums' last digits may leave them below it.)
      logprob = (float)fmin(gap - l.ln_all, 0.0);
      processed = (float)fmin(gap - l.ln_kept, 0.0);
    }
    const int64_t out = s.b * width + tid;
    a.out_tokens[out] = t;
    a.out_logprob[out] = logprob;
    if (a.out_processed) a.out_processed[out] = processed;
  }
  if (tid == 0) a.out_accepted[s.b] = s.accepted;
}

template <class D>
__global__ __launch_bounds__(kVerifyThreads) void final_kernel(VerifyArgs a) {
  __shared__ FinalShared sh;
  const SelectArgs& r = a.rows;
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, width = r.drafts + 1;
  const int accepted = read_global(a.verdicts, b);
  if (accepted < 0) {
    if (tid < width) {
      a.out_tokens[b * width + tid] = -1;
      a.out_logprob[b * width + tid] = NAN;
      if (a.out_processed) a.out_processed[b * width + tid] = NAN;
    }
    if (tid == 0) {
      a.out_accepted[b] = -1;
      if (a.bad_rows) atomicAdd(a.bad_rows, 1);
    }
    return;
  }
  Sequence s = sequence_of(a, b);
  s.accepted = accepted;
  finish<D>(a, s, sh);
}

template <class D>
hipError_t launch(const VerifyArgs& a, hipStream_t stream) {
  const SelectArgs& r = a.rows;
  hipError_t e;
  collect_kernel<D, kLimit><<<dim3((uint32_t)(r.whole_blocks + r.N * r.slices)), kThreads, 0,
                              stream>>>(r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  row_kernel<D, kLimit><<<dim3((uint32_t)r.N), kThreads, 0, stream>>>(r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // Four stretches at a time; as many turns for every workgroup as for the others.
  const int64_t turns = (stretches_of(r.V, r.dtype) + kVerifyWaves - 1) / kVerifyWaves;
  const int64_t each = (turns * r.seqs + kVerifyPlaces - 1) / kVerifyPlaces;
  const int64_t parts = (turns + each - 1) / each;
  residual_kernel<D><<<dim3((uint32_t)(r.seqs * parts)), kVerifyThreads, 0, stream>>>(a,
                                                                                    (int)parts);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  final_kernel<D><<<dim3((uint32_t)r.seqs), kVerifyThreads, 0, stream>>>(a);
  return hipGetLastError();
}

size_t up(size_t b) { return (b + 255) / 256 * 256; }

int64_t row_chunks(int64_t V, int32_t dtype) {
  const int64_t chunk = (int64_t)kThreads * kGroups * (16 / dtype_bytes(dtype));
  return (V + chunk - 1) / chunk;
}

}  // namespace

VerifyWorkspace verify_workspace_layout(int64_t seqs, int64_t drafts, int64_t V, int32_t dtype) {
  // (Without a draft model fewer rows have limits; the layout is the same.)
  const int64_t rows = seqs * (2 * drafts + 1);
  VerifyWorkspace w;
  w.off_select = 0;
  w.off_limits = up(select_workspace_most(rows, V, dtype, kLimitPlaces));
  w.off_whole = w.off_limits + up((size_t)rows * sizeof(SelectLimit));
  w.off_sums = w.off_whole + up((size_t)(rows * row_chunks(V, dtype) * kWaves) * sizeof(Part));
  w.off_verdicts =
      w.off_sums + up((size_t)(seqs * stretches_of(V, dtype)) * sizeof(double));
  w.total = w.off_verdicts + up((size_t)seqs * sizeof(int32_t));
  return w;
}

hipError_t launch_verify(VerifyArgs a, void* workspace, hipStream_t stream) {
  SelectArgs& r = a.rows;
  const VerifyWorkspace w = verify_workspace_layout(r.seqs, r.drafts, r.V, r.dtype);
  char* base = static_cast<char*>(workspace);
  r.N = r.seqs * (r.drafts + 1) + (r.draft_logits ? r.seqs * r.drafts : 0);
  r.limits = reinterpret_cast<SelectLimit*>(base + w.off_limits);
  r.whole = reinterpret_cast<SelectPart*>(base + w.off_whole);
  a.verdicts = reinterpret_cast<int32_t*>(base + w.off_verdicts);
  a.sums = reinterpret_cast<double*>(base + w.off_sums);
  place_select(r, base + w.off_select, kLimitPlaces);
  r.whole_blocks = (int32_t)std::min(kWholePlaces, r.N * row_chunks(r.V, r.dtype));
  switch (r.dtype) {
    case LP_F32: return launch<F32>(a, stream);
    case LP_BF16: return launch<BF16>(a, stream);
    default: return launch<F16>(a, stream);
  }
}

}  // namespace lp
