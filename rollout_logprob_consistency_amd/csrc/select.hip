// Token draw (lp_sample) and top logits (lp_top_logprobs): selections in the
// order (logit descending, index ascending) by rank and by probability mass.
//
// Two ways through a row, chosen by its settings alone:
//
// By a short list (top_k in [1, 1024], the greedy draw, min-p without top-p,
// and the top logits): collect_kernel reads the row once, keeps the tokens
// that can still be among the first in a list in LDS, and sums exp(z - m) per
// wave and chunk for the log-sum-exp. The list is sorted; everything else is
// decided in it, with weights and sums in fp64. Where there are few rows, a
// row is cut into slices, each leaves its list, and row_kernel joins them.
//
// By buckets (everything else, and rows whose list overflows): row_kernel
// collects the weights w = exp(s - max s), s = z / tau, in 2 048 buckets of
// 1/32 nat below the maximum: a count and a mass each. Inside bucket b a weight
// is e^{-b/32} P with |ln P| <= 1/64; P is taken in fp64 and summed as an
// integer in units of 2^-43, so a bucket's mass does not depend on the order
// of its terms (LDS integer atomics). Prefix sums over the buckets find the
// bucket in which a rank or a mass is reached; only that bucket's tokens are
// then listed, sorted and summed.
#include <algorithm>

#include "logits_internal.h"

namespace lp {
namespace {

constexpr int kThreads = kSelectThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kBuckets = 2048;        // of 1/32 nat; the last one: weight 0
constexpr double kPerNat = 32.0;
constexpr int kPerThread = kBuckets / kThreads;
constexpr int kList = 4096;           // tokens listed at once
constexpr double kUnit = 8796093022208.0;  // 2^43: the mass unit's inverse
constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer

// Tokens as distinct integers that ascend with (logit, then lower index):
// the order of the selection is their descending order.
__device__ __forceinline__ uint32_t key_of(float z) {
  uint32_t u = __float_as_uint(z);
  if (u == 0x80000000u) u = 0;  // -0 ties with +0
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t token_key(float z, int idx) {
  return ((uint64_t)key_of(z) << 32) | (uint32_t)~(uint32_t)idx;
}
__device__ __forceinline__ int token_index(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float token_logit(uint64_t k) { return key_value((uint32_t)(k >> 32)); }

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // key_of(-inf)

constexpr int kGroups = 4;                     // 16-byte groups per thread and chunk
constexpr int kMaxParts = LP_SELECT_MAX_VOCAB / (kThreads * kGroups * 4) * kWaves;

struct Shared {
  // Buckets: counts and masses while they are collected, then exclusive
  // prefix sums (masses as doubles in units of the maximum's weight).
  union {
    unsigned long long mass[kBuckets];
    double above[kBuckets + 1];
  };
  uint32_t cnt[kBuckets + 1];
  // The listed tokens, or the finer buckets of one that is too full to list.
  union {
    uint64_t list[kList];
    struct {
      unsigned long long fmass[kBuckets];
      uint32_t fcnt[kBuckets];
    };
    SelectPart parts[kMaxParts];
  };
  unsigned long long wave_u64[kWaves];
  double wave_f64[kWaves], shared_f64;
  uint32_t wave_u32[kWaves];
  float wave_f32[kWaves];
  uint32_t flags, n_list, found;
  uint32_t found_cnt;
  unsigned long long found_mass;
  uint32_t bound[2];
};

// A row and its scale. x(z) = 32 (max - z) / tau; the bucket is rint(x).
template <class D>
struct Row {
  const typename D::Raw* p;
  int V;
  double zmax, inv;  // inv = 32 / tau

  __device__ __forceinline__ double x_of(float z) const {
    return fmin((zmax - (double)z) * inv, (double)(kBuckets - 1));
  }
  static __device__ __forceinline__ int bucket(double x) {
    return (int)(uint32_t)__double_as_longlong(x + kMagic);
  }
  // exp((b - x) / 32) in units of 2^-43, by its Taylor series to degree 6
  // (|d| <= 1/64: truncation 5e-17); the last bucket weighs 0.
  static __device__ __forceinline__ unsigned long long mass(double x) {
    const double b = (x + kMagic) - kMagic;
    const double d = (b - x) * (1.0 / kPerNat);
    double p = 1.0 / 720.0;
    p = fma(p, d, 1.0 / 120.0);
    p = fma(p, d, 1.0 / 24.0);
    p = fma(p, d, 1.0 / 6.0);
    p = fma(p, d, 0.5);
    p = fma(p, d, 1.0);
    p = fma(p, d, 1.0);
    const unsigned long long m =
        (unsigned long long)__double_as_longlong(fma(p, kUnit, kMagic)) -
        (unsigned long long)__double_as_longlong(kMagic);
    return b < (double)(kBuckets - 1) ? m : 0ull;
  }

  // f(logit, index) for every token, each thread its 16-byte groups.
  template <class F>
  __device__ __forceinline__ void for_each(F f) const {
    constexpr int kU = 4;
    const int step = kThreads * D::kVec;
    for (int i0 = (int)threadIdx.x * D::kVec; i0 < V; i0 += kU * step) {
      Group<D> g[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) g[j] = load_group<D>(p, (int64_t)i0 + j * step, V);
#pragma unroll
      for (int j = 0; j < kU; ++j)
#pragma unroll
        for (int i = 0; i < D::kVec; ++i) {
          const int idx = i0 + j * step + i;
          if (idx < V) f(g[j].get(i), idx);
        }
    }
  }
};

// Exclusive prefix sum over the workgroup; `total` is the whole sum. Every
// thread gets its result; a barrier on both sides of the shared words.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* words, T* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  T before = __shfl_up(s, 1);
  if (lane == 0) before = T(0);
  if (lane == 63) words[wave] = s;
  __syncthreads();
  T base = T(0), sum = T(0);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) base = sum;
    sum += words[w];
  }
  __syncthreads();
  *total = sum;
  return base + before;
}

__device__ __forceinline__ float block_max(float v, float* words) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  if ((threadIdx.x & 63) == 0) words[threadIdx.x >> 6] = v;
  __syncthreads();
  v = words[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = fmaxf(v, words[w]);
  __syncthreads();
  return v;
}

// The list sorted descending (bitonic, padded with zeros to a power of two).
__device__ __forceinline__ void sort_list(uint64_t* list, uint32_t m) {
  uint32_t n = 1;
  while (n < m) n <<= 1;
  for (uint32_t i = m + threadIdx.x; i < n; i += kThreads) list[i] = 0;
  __syncthreads();
  for (uint32_t k = 2; k <= n; k <<= 1)
    for (uint32_t j = k >> 1; j > 0; j >>= 1) {
      for (uint32_t t = threadIdx.x; t < n / 2; t += kThreads) {
        const uint32_t lo = 2 * t - (t & (j - 1)), hi = lo + j;
        const uint64_t a = list[lo], b = list[hi];
        if ((a < b) == ((lo & k) == 0)) {
          list[lo] = b;
          list[hi] = a;
        }
      }
      __syncthreads();
    }
}

// Tokens with keys in [lo, hi] appended to the list, in any order.
template <class D>
__device__ __forceinline__ uint32_t gather(const Row<D>& row, Shared& sh, uint64_t lo, uint64_t hi) {
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  row.for_each([&](float z, int idx) {
    const uint64_t k = token_key(z, idx);
    if (k >= lo && k <= hi) {
      const uint32_t s = atomicAdd(&sh.n_list, 1u);
      if (s < (uint32_t)kList) sh.list[s] = k;
    }
  });
  __syncthreads();
  return min(sh.n_list, (uint32_t)kList);
}

// Least key whose bucket is at most b (buckets fall as keys rise): a binary
// search by one thread over the finite keys. All threads call it.
template <class D>
__device__ __forceinline__ uint32_t least_key(const Row<D>& row, Shared& sh, int b) {
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t lo = kKeyNegInf + 1, hi = key_of((float)row.zmax);  // bucket(hi) = 0 <= b
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (Row<D>::bucket(row.x_of(key_value(mid))) <= b) hi = mid;
      else lo = mid + 1;
    }
    sh.bound[0] = lo;
  }
  __syncthreads();
  return sh.bound[0];
}

// Where a selection ends inside a bucket: the token, its rank there (from 0)
// and the mass through it, in the bucket's units.
struct Found {
  uint64_t key;
  uint32_t rank;
  unsigned long long mass;
};

enum Mode { kByRank, kByMass, kByMassOver };

// The first token, in order, of bucket b at which
//   kByRank:     `rank` tokens of the bucket are reached (rank >= 1),
//   kByMass:     the mass through it is >= want,
//   kByMassOver: the mass through it is > want.
// count is the bucket's. Where no token's mass gets there (want is rounded),
// the last one.
template <class D>
__device__ Found select_in_bucket(const Row<D>& row, Shared& sh, int b, uint32_t count, Mode mode,
                                  uint32_t rank, double want) {
  uint64_t lo = (uint64_t)least_key(row, sh, b) << 32;
  uint64_t hi = b == 0 ? (((uint64_t)key_of((float)row.zmax) << 32) | 0xFFFFFFFFull)
                       : ((uint64_t)least_key(row, sh, b - 1) << 32) - 1;
  uint32_t base_cnt = 0;
  unsigned long long base_mass = 0;
  auto reached = [&](uint32_t c, unsigned long long m) {
    return mode == kByRank ? c >= rank : (mode == kByMass ? (double)m >= want : (double)m > want);
  };
  while (count > (uint32_t)kList) {
    // Too many to list: 2 048 finer buckets of equal key ranges. The range
    // shrinks 2 048-fold a turn, and keys are distinct, so this ends.
    const uint64_t range = hi - lo;
    const int bits = 64 - __clzll((long long)(range | 1));
    const int shift = bits > 11 ? bits - 11 : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kBuckets; i += kThreads) {
      sh.fmass[i] = 0;
      sh.fcnt[i] = 0;
    }
    __syncthreads();
    row.for_each([&](float z, int idx) {
      const uint64_t k = token_key(z, idx);
      if (k >= lo && k <= hi) {
        const uint32_t f = (uint32_t)((hi - k) >> shift);
        atomicAdd(&sh.fcnt[f], 1u);
        atomicAdd(&sh.fmass[f], Row<D>::mass(row.x_of(z)));
      }
    });
    __syncthreads();
    uint32_t c = 0;
    unsigned long long m = 0;
    for (int i = 0; i < kPerThread; ++i) {
      c += sh.fcnt[threadIdx.x * kPerThread + i];
      m += sh.fmass[threadIdx.x * kPerThread + i];
    }
    uint32_t all_c;
    unsigned long long all_m;
    uint32_t cb = base_cnt + block_scan(c, sh.wave_u32, &all_c);
    unsigned long long mb = base_mass + block_scan(m, sh.wave_u64, &all_m);
    if (threadIdx.x == 0) sh.found = 0xFFFFFFFFu;
    __syncthreads();
    // First finer bucket through which the selection is reached; the last
    // occupied one where rounding of `want` leaves none.
    for (int i = 0; i < kPerThread; ++i) {
      const int f = threadIdx.x * kPerThread + i;
      const uint32_t c1 = cb + sh.fcnt[f];
      const unsigned long long m1 = mb + sh.fmass[f];
      const bool last = c1 == base_cnt + all_c;
      if (sh.fcnt[f] != 0 && (reached(c1, m1) || last) && !(cb != base_cnt && reached(cb, mb))) {
        sh.found = (uint32_t)f;
        sh.found_cnt = cb;
        sh.found_mass = mb;
      }
      cb = c1;
      mb = m1;
    }
    __syncthreads();
    const uint32_t f = sh.found;
    base_cnt = sh.found_cnt;
    base_mass = sh.found_mass;
    count = sh.fcnt[f];
    const uint64_t top = hi - ((uint64_t)f << shift);
    const uint64_t width = (uint64_t)1 << shift;
    lo = top - lo >= width ? top - width + 1 : lo;
    hi = top;
    __syncthreads();
  }

  const uint32_t m = gather(row, sh, lo, hi);
  sort_list(sh.list, m);
  // Masses through every listed token, in order.
  constexpr int kEach = kList / kThreads;
  unsigned long long w[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t t = threadIdx.x * kEach + i;
    w[i] = t < m ? Row<D>::mass(row.x_of(token_logit(sh.list[t]))) : 0ull;
    sum += w[i];
  }
  unsigned long long all;
  unsigned long long mb = base_mass + block_scan(sum, sh.wave_u64, &all);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t t = threadIdx.x * kEach + i;
    const unsigned long long m1 = mb + w[i];
    if (t < m) {
      const uint32_t c1 = base_cnt + t + 1;
      if ((reached(c1, m1) || t == m - 1) && !(t > 0 && reached(c1 - 1, mb))) {
        sh.found = t;
        sh.found_mass = m1;
      }
    }
    mb = m1;
  }
  __syncthreads();
  Found r;
  r.key = sh.list[sh.found];
  r.rank = base_cnt + sh.found;
  r.mass = sh.found_mass;
  __syncthreads();
  return r;
}

// Row statistics: the maximum, then the buckets with their prefix sums.
struct Totals {
  bool bad;
  uint32_t finite;
  double mass;  // of all tokens, in units of the maximum's weight
};

template <class D>
__device__ float row_max(const Row<D>& row, Shared& sh, bool* bad) {
  float m = -INFINITY;
  bool odd = false;
  row.for_each([&](float z, int) {
    m = fmaxf(m, z);
    odd |= !(z < INFINITY);  // NaN or +inf
  });
  if (threadIdx.x == 0) sh.flags = 0;
  m = block_max(m, sh.wave_f32);
  if (odd) sh.flags = 1;
  __syncthreads();
  *bad = sh.flags != 0 || m == -INFINITY;
  return m;
}

template <class D>
__device__ Totals fill_buckets(const Row<D>& row, Shared& sh) {
  for (int i = threadIdx.x; i < kBuckets; i += kThreads) {
    sh.mass[i] = 0;
    sh.cnt[i] = 0;
  }
  __syncthreads();
  row.for_each([&](float z, int) {
    if (z != -INFINITY) {
      const double x = row.x_of(z);
      const int b = Row<D>::bucket(x);
      atomicAdd(&sh.cnt[b], 1u);
      atomicAdd(&sh.mass[b], Row<D>::mass(x));
    }
  });
  __syncthreads();
  uint32_t c[kPerThread], cs = 0;
  double m[kPerThread], ms = 0.0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = threadIdx.x * kPerThread + i;
    c[i] = sh.cnt[b];
    m[i] = (double)sh.mass[b] * (exp_f64(-(double)b / kPerNat) / kUnit);
    cs += c[i];
    ms += m[i];
  }
  Totals t;
  t.bad = false;
  uint32_t cb = block_scan(cs, sh.wave_u32, &t.finite);
  double mb = block_scan(ms, sh.wave_f64, &t.mass);  // (its barriers end the reads above)
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = threadIdx.x * kPerThread + i;
    sh.cnt[b] = cb;
    sh.above[b] = mb;
    cb += c[i];
    mb += m[i];
  }
  if (threadIdx.x == kThreads - 1) {
    sh.cnt[kBuckets] = t.finite;
    sh.above[kBuckets] = mb;
  }
  __syncthreads();
  t.mass = sh.above[kBuckets];
  return t;
}

__device__ __forceinline__ double bucket_weight(int b) { return exp_f64(-(double)b / kPerNat); }

// The bucket that holds the token of rank `k` (from 1).
__device__ __forceinline__ int bucket_of_rank(Shared& sh, uint32_t k) {
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = threadIdx.x * kPerThread + i;
    if (sh.cnt[b] < k && k <= sh.cnt[b + 1]) sh.found = b;
  }
  __syncthreads();
  const int b = (int)sh.found;
  __syncthreads();
  return b;
}

// The first occupied bucket through which the mass is >= want (> want with
// `over`). Prefix sums of neighbouring threads may differ in the last bit, so
// only a bucket's end is looked at; bucket 0 holds the maximum.
__device__ __forceinline__ int bucket_of_mass(Shared& sh, double want, bool over) {
  if (threadIdx.x == 0) sh.found = kBuckets;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = threadIdx.x * kPerThread + i;
    const double end = sh.above[b + 1];
    if (sh.cnt[b + 1] != sh.cnt[b] && (over ? end > want : end >= want)) {
      atomicMin(&sh.found, (uint32_t)b);
      break;
    }
  }
  __syncthreads();
  const int b = sh.found < (uint32_t)kBuckets ? (int)sh.found : 0;
  __syncthreads();
  return b;
}

// ---- The short list ---------------------------------------------------------

constexpr int kListMax = LP_TOP_MAX;           // tokens that a slice leaves
constexpr uint32_t kOverflow = 0xFFFFFFFFu;    // a slice's count: take the buckets
constexpr uint32_t kCrowded = 2048;            // a list is cut down from here on

template <class D>
constexpr int chunk_of() { return kThreads * kGroups * D::kVec; }

using Part = SelectPart;

__device__ __forceinline__ float wave_max_f32(float m) {
  m = fmaxf(m, __int_as_float(xlane<1>(__float_as_int(m))));
  m = fmaxf(m, __int_as_float(xlane<2>(__float_as_int(m))));
  m = fmaxf(m, __int_as_float(xlane<4>(__float_as_int(m))));
  m = fmaxf(m, __int_as_float(xlane<8>(__float_as_int(m))));
  m = fmaxf(m, __int_as_float(xlane<16>(__float_as_int(m))));
  return fmaxf(__int_as_float(lane_value(__float_as_int(m), 0)),
               __int_as_float(lane_value(__float_as_int(m), 32)));
}
__device__ __forceinline__ float wave_sum_f32(float s) {
  s += __int_as_float(xlane<1>(__float_as_int(s)));
  s += __int_as_float(xlane<2>(__float_as_int(s)));
  s += __int_as_float(xlane<4>(__float_as_int(s)));
  s += __int_as_float(xlane<8>(__float_as_int(s)));
  s += __int_as_float(xlane<16>(__float_as_int(s)));
  return __int_as_float(lane_value(__float_as_int(s), 0)) +
         __int_as_float(lane_value(__float_as_int(s), 32));
}

// The part of a wave whose lanes hold these groups: the same terms in the
// same order wherever it is formed. f(z, j, i) sees every logit.
template <class D, class F>
__device__ __forceinline__ Part part_of(Group<D> (&g)[kGroups], float m, float scale2, F f) {
  const float base = m == -INFINITY ? 0.0f : m;  // masked tokens sum to 0, a NaN stays one
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    g[j].fresh();
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) {
      const float z = g[j].get(i);
      s += __builtin_amdgcn_exp2f((z - base) * scale2);
      f(z, j, i);
    }
  }
  return {m, wave_sum_f32(s)};
}

enum Kind { kBuckets_, kTopK, kMinP };

struct Settings {
  float tau, top_p, min_p, u;
  int32_t top_k;
  bool greedy, bad;
  Kind kind;
  uint32_t k;  // kTopK: tokens wanted
};

__device__ __forceinline__ Settings settings_of(const SelectArgs& a, int64_t n) {
  Settings s;
  if (!a.u) {  // the top logits
    s = {a.temperature, 1.0f, 0.0f, 0.0f, a.top_k, false, false, kTopK, (uint32_t)a.top_k};
    return s;
  }
  s.tau = a.temperatures ? a.temperatures[n] : a.temperature;
  s.top_p = a.top_ps ? a.top_ps[n] : a.top_p;
  s.min_p = a.min_ps ? a.min_ps[n] : a.min_p;
  s.top_k = a.top_ks ? a.top_ks[n] : a.top_k;
  s.u = a.u[n];
  s.greedy = s.tau == 0.0f;
  s.bad = !(s.tau >= 0.0f) || isnan(s.u) || isnan(s.top_p) || isnan(s.min_p);
  if (s.greedy) s.tau = 1.0f;
  s.k = s.greedy ? 1u : (uint32_t)max(s.top_k, 0);
  s.kind = kBuckets_;
  if (!s.bad && isfinite(s.tau)) {
    if (s.greedy || (s.top_k > 0 && s.top_k <= kListMax)) s.kind = kTopK;
    else if (s.top_k <= 0 && s.top_p >= 1.0f && s.min_p > 0.0f && s.min_p <= 1.0f) s.kind = kMinP;
  }
  return s;
}

// How far below the maximum a token that min-p keeps can lie, rounded up.
__device__ __forceinline__ float depth_of(const Settings& st) {
  return (float)(-log((double)st.min_p) * (double)st.tau) * 1.000001f;
}
// The least finite logit that `depth` below t reaches.
__device__ __forceinline__ float bound(float t) { return fmaxf(t, -3.4028234663852886e38f); }

__device__ __forceinline__ float scale2_of(float tau) {
  return (float)(1.4426950408889634 / (double)tau);
}

// Slices of a row: every slice leaves at most k (kTopK) or kListMax tokens,
// which have to fit one list together.
__device__ __forceinline__ int slices_of(const SelectArgs& a, const Settings& s) {
  const int most = s.kind == kTopK ? kList / (int)s.k : kList / kListMax;
  return min(a.slices, max(most, 1));
}

__device__ __forceinline__ void write_bad_draw(const SelectArgs& a, int64_t n) {
  a.out_token[n] = -1;
  a.out_logprob[n] = NAN;
  if (a.out_processed) a.out_processed[n] = NAN;
  if (a.out_kept) a.out_kept[n] = 0;
  if (a.bad_rows) atomicAdd(a.bad_rows, 1);
}

// A row without a valid draw or list: -1 and NaN.
__device__ void write_bad_top(const SelectArgs& a, int64_t n) {
  for (int i = threadIdx.x; i < a.top_k; i += kThreads) {
    a.out_ids[n * a.top_k + i] = -1;
    a.out_logits[n * a.top_k + i] = NAN;
    a.out_logprob[n * a.top_k + i] = NAN;
  }
  if (threadIdx.x == 0) {
    if (a.out_lse) a.out_lse[n] = NAN;
    if (a.bad_rows) atomicAdd(a.bad_rows, 1);
  }
}

// The row's maximum and the mass of all its tokens in units of the maximum's
// weight, from its parts: fixed order, each part scaled in fp64. A NaN or
// +inf logit leaves a NaN.
__device__ __forceinline__ double join_parts(const Part* parts, int n, double inv_tau, float* words,
                                             double* words64, float* zmax) {
  float m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += kThreads) m = fmaxf(m, parts[i].m);
  m = block_max(m, words);
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Part p = parts[i];
    // m = -inf: nothing but masked tokens (0), or a NaN among them.
    s += p.m == -INFINITY ? (double)p.s
                          : (double)p.s * exp_f64(((double)p.m - (double)m) * inv_tau);
  }
  double all;
  block_scan(s, words64, &all);
  *zmax = m;
  return all;
}

// First index (of each thread's, then of all) with hit; n where there is none.
// `word` is LDS; a barrier on both sides.
template <class F>
__device__ __forceinline__ uint32_t first_index(uint32_t* word, uint32_t n, uint32_t base, int each,
                                                F hit) {
  if (threadIdx.x == 0) *word = n;
  __syncthreads();
  for (int i = 0; i < each; ++i)
    if (base + i < n && hit(i)) {
      atomicMin(word, base + i);
      break;
    }
  __syncthreads();
  const uint32_t r = *word;
  __syncthreads();
  return r;
}

// The draw from a sorted list that holds every token that can be kept.
template <class Words>
__device__ void finish_draw(const SelectArgs& a, const Settings& st, int64_t n, const uint64_t* list,
                            uint32_t m, float zmax, double all, Words& w) {
  constexpr int kEach = kList / kThreads;
  const double tau = (double)st.tau, top = (double)zmax;
  const uint32_t base = threadIdx.x * kEach;
  double x[kEach], c[kEach], sum = 0.0;  // -ln weight; sums through each token
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    x[i] = base + i < m ? (top - (double)token_logit(list[base + i])) / tau : INFINITY;
    sum += base + i < m ? exp_f64(-x[i]) : 0.0;
    c[i] = sum;
  }
  double total;
  const double before = block_scan(sum, w.wave_f64, &total);
#pragma unroll
  for (int i = 0; i < kEach; ++i) c[i] += before;
  // The sum through token t (from 0) for every thread.
  auto mass_through = [&](uint32_t t) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (base + i == t) w.shared_f64 = c[i];
    __syncthreads();
    const double v = w.shared_f64;
    __syncthreads();
    return v;
  };
  uint32_t kept = st.kind == kTopK ? min(st.k, m) : m;
  if (st.kind == kMinP || (st.min_p > 0.0f && !st.greedy)) {
    const double most = fmax(0.0, -log((double)st.min_p));
    kept = min(kept, st.min_p > 1.0f ? 1u : first_index(&w.found, m, base, kEach, [&](int i) {
                 return x[i] > most;
               }));
  }
  if (st.top_p < 1.0f && !st.greedy) {
    // The nucleus is of what top-k left, whatever min-p drops.
    const double want = (double)st.top_p * mass_through(min(st.k, m) - 1);
    const uint32_t p = want > 0.0 ? first_index(&w.found, m, base, kEach,
                                                [&](int i) { return c[i] >= want; }) + 1
                                  : 1u;
    kept = min(kept, p);
  }
  const double mass = mass_through(kept - 1);
  const double u = st.greedy ? 0.0 : fmin(fmax((double)st.u, 0.0), 1.0 - 0x1p-24);
  const uint32_t rank =
      min(kept - 1, first_index(&w.found, kept, base, kEach, [&](int i) { return c[i] > u * mass; }));
  if (threadIdx.x == 0) {
    const uint64_t t = list[rank];
    const double s = ((double)token_logit(t) - top) / tau;
    a.out_token[n] = token_index(t);
    a.out_logprob[n] = (float)(s - log(all));
    if (a.out_processed) a.out_processed[n] = st.greedy ? 0.0f : (float)(s - log(mass));
    if (a.out_kept) a.out_kept[n] = (int32_t)kept;
  }
}

// The first k tokens from a sorted list of m.
__device__ void finish_top(const SelectArgs& a, int64_t n, const uint64_t* list, uint32_t m,
                           double zmax, double all) {
  const double tau = (double)a.temperature, ln_mass = log(all);
  for (uint32_t i = threadIdx.x; i < (uint32_t)a.top_k; i += kThreads) {
    const bool there = i < m;
    const uint64_t t = there ? list[i] : 0;
    const float z = there ? token_logit(t) : -INFINITY;
    const int64_t o = n * a.top_k + i;
    a.out_ids[o] = there ? token_index(t) : -1;
    a.out_logits[o] = z;
    a.out_logprob[o] = (float)(((double)z - zmax) / tau - ln_mass);
  }
  if (threadIdx.x == 0 && a.out_lse) a.out_lse[n] = (float)(zmax / tau + ln_mass);
}

struct CollectShared {
  uint64_t list[kList];
  Part parts[kMaxParts];
  double wave_f64[kWaves], shared_f64;
  float wave_f32[kWaves];
  uint32_t n_list, found;
};

// One slice of a row (the whole row where a.slices is 1).
template <class D, bool kTop>
__global__ __launch_bounds__(kThreads, 6) void collect_kernel(SelectArgs a) {
  __shared__ CollectShared sh;
  constexpr int kChunk = chunk_of<D>();
  const int64_t n = blockIdx.x / (uint32_t)a.slices;
  const int slice = (int)(blockIdx.x - (uint32_t)n * (uint32_t)a.slices);
  const Settings st = settings_of(a, n);
  uint32_t* count = a.counts + n * a.slices;
  if (st.kind == kBuckets_) {
    if (slice == 0 && threadIdx.x == 0) count[0] = kOverflow;
    return;
  }
  const int slices = slices_of(a, st);
  if (slice >= slices) return;
  const int chunks = (a.V + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * slice / slices);
  const int c1 = (int)((int64_t)chunks * (slice + 1) / slices);
  const typename D::Raw* row = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  const float scale2 = scale2_of(st.tau);
  const float depth = st.kind == kMinP ? depth_of(st) : 0.0f;
  const int tid = threadIdx.x, wave = tid >> 6;

  Group<D> g[kGroups], next[kGroups];
  auto load = [&](Group<D>(&to)[kGroups], int c) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
      to[j] = load_group<D>(row, (int64_t)c * kChunk + (j * kThreads + tid) * D::kVec, a.V);
  };
  // Tokens from theta on enter the list. theta is a logit that `k` tokens
  // reach (kTopK), or the depth below one (kMinP); never below the finite ones.
  float theta = 0.0f;
  // Sorted down to what can still be needed; returns false where the list
  // has lost tokens.
  auto cut = [&](bool always) {
    __syncthreads();
    const uint32_t m = sh.n_list;
    __syncthreads();
    if (m > (uint32_t)kList) return false;
    if (!always && m < kCrowded) return true;
    sort_list(sh.list, m);
    uint32_t keep = m;
    if (st.kind == kTopK) {
      keep = min(m, st.k);
      if (m >= st.k) theta = token_logit(sh.list[st.k - 1]);
    } else if (m > 0) {
      theta = bound(token_logit(sh.list[0]) - depth);
      constexpr int kEach = kList / kThreads;
      keep = first_index(&sh.found, m, tid * kEach, kEach,
                         [&](int i) { return token_logit(sh.list[tid * kEach + i]) < theta; });
    }
    __syncthreads();
    if (tid == 0) sh.n_list = keep;
    __syncthreads();
    return true;
  };

  load(g, c0);
  bool fits = true;
  for (int c = c0; c < c1; ++c) {
    if (c + 1 < c1) load(next, c + 1);
    float tm = -INFINITY, gm[kGroups];
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      gm[j] = -INFINITY;
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) gm[j] = fmaxf(gm[j], g[j].get(i));
      tm = fmaxf(tm, gm[j]);
    }
    const float m = wave_max_f32(tm);
    if (c == c0) {
      // The k-th largest of the threads' (or their groups') maxima: k tokens
      // of this chunk reach it.
      if (st.kind == kTopK) {
        const bool fine = st.k > 256;
        if (fine) {
#pragma unroll
          for (int j = 0; j < kGroups; ++j) sh.list[j * kThreads + tid] = token_key(gm[j], 0);
        } else {
          sh.list[tid] = token_key(tm, 0);
        }
        sort_list(sh.list, fine ? kGroups * kThreads : kThreads);
        theta = bound(token_logit(sh.list[st.k - 1]));
      } else {
        theta = bound(block_max(tm, sh.wave_f32) - depth);
      }
      __syncthreads();
      if (tid == 0) sh.n_list = 0;
      __syncthreads();
    }
    const Part p = part_of<D>(g, m, scale2, [&](float z, int j, int i) {
      if (z >= theta) {
        const uint32_t at = atomicAdd(&sh.n_list, 1u);
        if (at < (uint32_t)kList)
          sh.list[at] = token_key(z, c * kChunk + (j * kThreads + tid) * D::kVec + i);
      }
    });
    if ((tid & 63) == 0) {
      if (a.slices == 1) sh.parts[c * kWaves + wave] = p;
      else a.parts[(n * chunks + c) * kWaves + wave] = p;
    }
    // Cut at the 2nd, 4th, 8th, ... chunk, where a list has about doubled.
    const int done = c - c0 + 1;
    if (c + 1 < c1 && done > 1 && (done & (done - 1)) == 0 && !cut(false)) {
      fits = false;
      break;
    }
#pragma unroll
    for (int j = 0; j < kGroups; ++j) g[j] = next[j];
  }
  fits = fits && cut(true);
  const uint32_t m = fits ? sh.n_list : 0;
  if (!fits || m > (uint32_t)kListMax) {
    if (tid == 0) count[slice] = kOverflow;
    return;
  }
  if (a.slices > 1) {
    uint64_t* keys = a.keys + (n * a.slices + slice) * kListMax;
    for (uint32_t i = tid; i < m; i += kThreads) keys[i] = sh.list[i];
    if (tid == 0) count[slice] = m;
    return;
  }
  float zmax;
  const double all =
      join_parts(sh.parts, chunks * kWaves, 1.0 / (double)st.tau, sh.wave_f32, sh.wave_f64, &zmax);
  if (tid == 0) count[0] = 0;
  if (!(all > 0.0) || zmax == -INFINITY) {
    if (kTop) write_bad_top(a, n);
    else if (tid == 0) write_bad_draw(a, n);
  } else if (kTop) {
    finish_top(a, n, sh.list, m, (double)zmax, all);
  } else {
    finish_draw(a, st, n, sh.list, m, zmax, all, sh);
  }
}

// ---- By buckets -------------------------------------------------------------

template <class D>
__device__ void draw_by_buckets(const SelectArgs& a, const Settings& st, int64_t n, Shared& sh) {
  const bool greedy = st.greedy;
  const double tau = (double)st.tau;
  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  bool bad;
  row.zmax = (double)row_max(row, sh, &bad);
  if (bad || st.bad) {
    if (threadIdx.x == 0) write_bad_draw(a, n);
    return;
  }
  row.inv = kPerNat / tau;
  const Totals all = fill_buckets(row, sh);

  // Lengths of the kept prefix and its mass, filter by filter.
  uint32_t kept = all.finite;
  double mass = all.mass;
  if (greedy) {
    kept = 1;
    mass = 1.0;
  } else {
    if (st.top_k > 0 && (uint32_t)st.top_k < kept) {
      kept = (uint32_t)st.top_k;
      const int b = bucket_of_rank(sh, kept);
      if (b < kBuckets - 1) {
        const Found f = select_in_bucket(row, sh, b, sh.cnt[b + 1] - sh.cnt[b], kByRank,
                                         kept - sh.cnt[b], 0.0);
        mass = sh.above[b] + (double)f.mass * (bucket_weight(b) / kUnit);
      }
    }
    if (st.top_p < 1.0f) {
      const double want = (double)st.top_p * mass;
      if (want > 0.0) {
        const int b = bucket_of_mass(sh, want, false);
        const Found f = select_in_bucket(row, sh, b, sh.cnt[b + 1] - sh.cnt[b], kByMass, 0,
                                         (want - sh.above[b]) * (kUnit / bucket_weight(b)));
        const uint32_t m = sh.cnt[b] + f.rank + 1;
        if (m < kept) {
          kept = m;
          mass = sh.above[b] + (double)f.mass * (bucket_weight(b) / kUnit);
        }
      } else {
        kept = 1;
        mass = 1.0;
      }
    }
    if (st.min_p > 1.0f) {  // no weight reaches it: the first token alone
      kept = 1;
      mass = 1.0;
    } else if (st.min_p > 0.0f) {
      // w >= min_p where x = -32 ln w <= -32 ln min_p.
      const double most = fmax(0.0, -log((double)st.min_p) * kPerNat);
      const int b = Row<D>::bucket(fmin(most, (double)(kBuckets - 1)));
      if (sh.cnt[b] < kept) {
        uint32_t c = 0;
        unsigned long long m = 0;
        row.for_each([&](float z, int) {
          if (z != -INFINITY) {
            const double x = row.x_of(z);
            if ((row.zmax - (double)z) * row.inv <= most && Row<D>::bucket(x) == b) {
              ++c;
              m += Row<D>::mass(x);
            }
          }
        });
        uint32_t call;
        unsigned long long mall;
        block_scan(c, sh.wave_u32, &call);
        block_scan(m, sh.wave_u64, &mall);
        if (sh.cnt[b] + call < kept) {
          kept = sh.cnt[b] + call;
          mass = sh.above[b] + (double)mall * (bucket_weight(b) / kUnit);
        }
      }
    }
  }

  const double u = greedy ? 0.0 : fmin(fmax((double)st.u, 0.0), 1.0 - 0x1p-24);
  const double want = u * mass;
  const int b = bucket_of_mass(sh, want, true);
  const Found f = select_in_bucket(row, sh, b, sh.cnt[b + 1] - sh.cnt[b], kByMassOver, 0,
                                   (want - sh.above[b]) * (kUnit / bucket_weight(b)));
  if (threadIdx.x == 0) {
    const double s = ((double)token_logit(f.key) - row.zmax) / tau;
    a.out_token[n] = token_index(f.key);
    a.out_logprob[n] = (float)(s - log(all.mass));
    if (a.out_processed) a.out_processed[n] = greedy ? 0.0f : (float)(s - log(mass));
    if (a.out_kept) a.out_kept[n] = (int32_t)kept;
  }
}

// The parts of a row as collect_kernel forms them, into sh.parts; returns
// their number.
template <class D>
__device__ int parts_of_row(const Row<D>& row, float tau, Shared& sh) {
  constexpr int kChunk = chunk_of<D>();
  const int tid = threadIdx.x, chunks = (row.V + kChunk - 1) / kChunk;
  const float scale2 = scale2_of(tau);
  for (int c = 0; c < chunks; ++c) {
    Group<D> g[kGroups];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      g[j] = load_group<D>(row.p, (int64_t)c * kChunk + (j * kThreads + tid) * D::kVec, row.V);
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) m = fmaxf(m, g[j].get(i));
    }
    const Part p = part_of<D>(g, wave_max_f32(m), scale2, [](float, int, int) {});
    if ((tid & 63) == 0) sh.parts[c * kWaves + (tid >> 6)] = p;
  }
  __syncthreads();
  return chunks * kWaves;
}

// A row of the short lists whose list overflowed: its tokens by selection,
// then the same ending, so that its results do not depend on how the row was
// cut. A row where min-p leaves more than kListMax goes by buckets for good.
template <class D, bool kTop>
__device__ void list_by_buckets(const SelectArgs& a, const Settings& st, int64_t n, Shared& sh) {
  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  const int parts = parts_of_row(row, st.tau, sh);
  float zmax;
  const double sum =
      join_parts(sh.parts, parts, 1.0 / (double)st.tau, sh.wave_f32, sh.wave_f64, &zmax);
  if (!(sum > 0.0) || zmax == -INFINITY) {
    if constexpr (kTop) write_bad_top(a, n);
    else if (threadIdx.x == 0) write_bad_draw(a, n);
    return;
  }
  row.zmax = (double)zmax;
  row.inv = kPerNat / (double)st.tau;
  if (st.kind == kMinP) {
    gather(row, sh, (uint64_t)key_of(bound(zmax - depth_of(st))) << 32, ~0ull);
    const uint32_t m = sh.n_list;
    __syncthreads();
    if (m > (uint32_t)kListMax) {
      if constexpr (!kTop) draw_by_buckets<D>(a, st, n, sh);
      return;
    }
    sort_list(sh.list, m);
    if constexpr (!kTop) finish_draw(a, st, n, sh.list, m, zmax, sum, sh);
    return;
  }
  const Totals all = fill_buckets(row, sh);
  const uint32_t want = min(st.k, all.finite);
  const int b = bucket_of_rank(sh, want);
  uint64_t lo = b == kBuckets - 1 ? (uint64_t)(kKeyNegInf + 1) << 32
                                  : (uint64_t)least_key(row, sh, b) << 32;
  if (sh.cnt[b + 1] > (uint32_t)kList) {
    // More than the list holds reach that bucket: the last token's own key.
    const uint32_t before = sh.cnt[b];
    lo = select_in_bucket(row, sh, b, sh.cnt[b + 1] - before, kByRank, want - before, 0.0).key;
  }
  sort_list(sh.list, gather(row, sh, lo, ~0ull));
  if constexpr (kTop) finish_top(a, n, sh.list, want, (double)zmax, sum);
  else finish_draw(a, st, n, sh.list, want, zmax, sum, sh);
}

// One row: its slices' lists joined, or the buckets.
template <class D, bool kTop>
__global__ __launch_bounds__(kThreads, 4) void row_kernel(SelectArgs a) {
  __shared__ Shared sh;
  const int64_t n = blockIdx.x;
  const Settings st = settings_of(a, n);
  const int slices = slices_of(a, st);
  const uint32_t* count = a.counts + n * a.slices;
  if constexpr (!kTop)
    if (st.kind == kBuckets_) {
      draw_by_buckets<D>(a, st, n, sh);
      return;
    }
  bool over = false;
  uint32_t m = 0;
  for (int i = 0; i < slices; ++i) {
    const uint32_t c = count[i];
    over |= c == kOverflow;
    m += c;
  }
  if (over) {
    list_by_buckets<D, kTop>(a, st, n, sh);
    return;
  }
  if (a.slices == 1) return;  // collect_kernel has finished the row
  uint32_t at = 0;
  for (int i = 0; i < slices; ++i) {
    const uint32_t c = count[i];
    const uint64_t* keys = a.keys + (n * a.slices + i) * kListMax;
    for (uint32_t j = threadIdx.x; j < c; j += kThreads) sh.list[at + j] = keys[j];
    at += c;
  }
  sort_list(sh.list, m);
  const int chunks = (a.V + chunk_of<D>() - 1) / chunk_of<D>();
  if (st.kind == kTopK) {
    m = min(m, st.k);
  } else {
    constexpr int kEach = kList / kThreads;
    const uint32_t base = threadIdx.x * kEach;
    const float theta = m > 0 ? bound(token_logit(sh.list[0]) - depth_of(st)) : 0.0f;
    m = first_index(&sh.found, m, base, kEach,
                    [&](int i) { return token_logit(sh.list[base + i]) < theta; });
    if (m > (uint32_t)kListMax) {
      list_by_buckets<D, kTop>(a, st, n, sh);
      return;
    }
  }
  float zmax;
  const double all = join_parts(a.parts + n * chunks * kWaves, chunks * kWaves,
                                1.0 / (double)st.tau, sh.wave_f32, sh.wave_f64, &zmax);
  if (!(all > 0.0) || zmax == -INFINITY) {
    if constexpr (kTop) write_bad_top(a, n);
    else if (threadIdx.x == 0) write_bad_draw(a, n);
    return;
  }
  if constexpr (kTop) finish_top(a, n, sh.list, m, (double)zmax, all);
  else finish_draw(a, st, n, sh.list, m, zmax, all, sh);
}

template <class D, bool kTop>
hipError_t launch(const SelectArgs& a, bool lists, hipStream_t stream) {
  if (lists) {
    collect_kernel<D, kTop><<<dim3((uint32_t)(a.N * a.slices)), kThreads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  row_kernel<D, kTop><<<dim3((uint32_t)a.N), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int select_slices(int64_t N, int64_t V, int32_t dtype) {
  const int64_t chunk = (int64_t)kThreads * kGroups * (16 / dtype_bytes(dtype));
  const int64_t chunks = (V + chunk - 1) / chunk;
  // Rows that fill the card by themselves are not cut.
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, 512 / std::max<int64_t>(N, 1)));
}

SelectWorkspace select_workspace_layout(int64_t N, int64_t V, int32_t dtype) {
  const int64_t chunk = (int64_t)kThreads * kGroups * (16 / dtype_bytes(dtype));
  const int64_t chunks = (V + chunk - 1) / chunk;
  const size_t lists = (size_t)N * (size_t)select_slices(N, V, dtype);
  const bool cut = select_slices(N, V, dtype) > 1;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  SelectWorkspace w;
  w.off_counts = 0;
  w.off_parts = up(lists * sizeof(uint32_t));
  w.off_keys = w.off_parts + (cut ? up((size_t)N * chunks * kWaves * sizeof(Part)) : 0);
  w.total = w.off_keys + (cut ? lists * kListMax * sizeof(uint64_t) : 0);
  return w;
}

hipError_t launch_select(SelectArgs a, void* workspace, hipStream_t stream) {
  const SelectWorkspace w = select_workspace_layout(a.N, a.V, a.dtype);
  char* base = static_cast<char*>(workspace);
  a.slices = select_slices(a.N, a.V, a.dtype);
  a.counts = reinterpret_cast<uint32_t*>(base + w.off_counts);
  a.parts = reinterpret_cast<SelectPart*>(base + w.off_parts);
  a.keys = reinterpret_cast<uint64_t*>(base + w.off_keys);
  const bool top = a.u == nullptr;
  // Settings that the host sees and that no row can take by lists.
  const bool lists = top || a.temperatures || a.top_ks || a.top_ps || a.min_ps ||
                     a.temperature == 0.0f || (a.top_k > 0 && a.top_k <= kListMax) ||
                     (a.top_k <= 0 && a.top_p >= 1.0f && a.min_p > 0.0f && a.min_p <= 1.0f);
  switch (a.dtype) {
    case LP_F32: return top ? launch<F32, true>(a, lists, stream) : launch<F32, false>(a, lists, stream);
    case LP_BF16: return top ? launch<BF16, true>(a, lists, stream) : launch<BF16, false>(a, lists, stream);
    default: return top ? launch<F16, true>(a, lists, stream) : launch<F16, false>(a, lists, stream);
  }
}

}  // namespace lp
