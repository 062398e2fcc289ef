// Token draw (lp_sample) and top logits (lp_top_logprobs): selections in the
// order (logit descending, index ascending) by rank and by probability mass.
//
// One workgroup per row. The weights w = exp(s - max s), s = z / tau, are
// collected in 2 048 buckets of 1/32 nat below the maximum: a count and a
// mass each. Inside bucket b a weight is e^{-b/32} P with |ln P| <= 1/64; P is
// taken in fp64 and summed as an integer in units of 2^-43, so a bucket's mass
// does not depend on the order of its terms (LDS integer atomics). Prefix
// sums over the buckets find the bucket in which a rank or a mass is reached;
// only that bucket's tokens are then listed, sorted and summed.
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
  };
  unsigned long long wave_u64[kWaves];
  double wave_f64[kWaves];
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
          if (idx < V) f(D::value(g[j].r[i]), idx);
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
__device__ __forceinline__ void sort_list(Shared& sh, uint32_t m) {
  uint32_t n = 1;
  while (n < m) n <<= 1;
  for (uint32_t i = m + threadIdx.x; i < n; i += kThreads) sh.list[i] = 0;
  __syncthreads();
  for (uint32_t k = 2; k <= n; k <<= 1)
    for (uint32_t j = k >> 1; j > 0; j >>= 1) {
      for (uint32_t t = threadIdx.x; t < n / 2; t += kThreads) {
        const uint32_t lo = 2 * t - (t & (j - 1)), hi = lo + j;
        const uint64_t a = sh.list[lo], b = sh.list[hi];
        if ((a < b) == ((lo & k) == 0)) {
          sh.list[lo] = b;
          sh.list[hi] = a;
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
  sort_list(sh, m);
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

template <class D>
__global__ __launch_bounds__(kThreads) void sample_kernel(SelectArgs a) {
  __shared__ Shared sh;
  const int64_t n = blockIdx.x;
  const float tau0 = a.temperatures ? a.temperatures[n] : a.temperature;
  const float top_p = a.top_ps ? a.top_ps[n] : a.top_p;
  const float min_p = a.min_ps ? a.min_ps[n] : a.min_p;
  const int32_t top_k = a.top_ks ? a.top_ks[n] : a.top_k;
  const float u0 = a.u[n];
  const bool greedy = tau0 == 0.0f;
  const double tau = greedy ? 1.0 : (double)tau0;

  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  bool bad;
  row.zmax = (double)row_max(row, sh, &bad);
  bad |= !(tau0 >= 0.0f) || isnan(u0) || isnan(top_p) || isnan(min_p);
  if (bad) {
    if (threadIdx.x == 0) {
      a.out_token[n] = -1;
      a.out_logprob[n] = NAN;
      if (a.out_processed) a.out_processed[n] = NAN;
      if (a.out_kept) a.out_kept[n] = 0;
      if (a.bad_rows) atomicAdd(a.bad_rows, 1);
    }
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
    if (top_k > 0 && (uint32_t)top_k < kept) {
      kept = (uint32_t)top_k;
      const int b = bucket_of_rank(sh, kept);
      if (b < kBuckets - 1) {
        const Found f = select_in_bucket(row, sh, b, sh.cnt[b + 1] - sh.cnt[b], kByRank,
                                         kept - sh.cnt[b], 0.0);
        mass = sh.above[b] + (double)f.mass * (bucket_weight(b) / kUnit);
      }
    }
    if (top_p < 1.0f) {
      const double want = (double)top_p * mass;
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
    if (min_p > 1.0f) {  // no weight reaches it: the first token alone
      kept = 1;
      mass = 1.0;
    } else if (min_p > 0.0f) {
      // w >= min_p where x = -32 ln w <= -32 ln min_p.
      const double most = fmax(0.0, -log((double)min_p) * kPerNat);
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

  const double u = greedy ? 0.0 : fmin(fmax((double)u0, 0.0), 1.0 - 0x1p-24);
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

template <class D>
__global__ __launch_bounds__(kThreads) void top_kernel(SelectArgs a) {
  __shared__ Shared sh;
  const int64_t n = blockIdx.x;
  const int k = a.top_k;
  const double tau = (double)a.temperature;
  int64_t* ids = a.out_ids + n * k;
  float* zs = a.out_logits + n * k;
  float* lps = a.out_logprob + n * k;

  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  bool bad;
  row.zmax = (double)row_max(row, sh, &bad);
  if (bad) {
    for (int i = threadIdx.x; i < k; i += kThreads) {
      ids[i] = -1;
      zs[i] = NAN;
      lps[i] = NAN;
    }
    if (threadIdx.x == 0) {
      if (a.out_lse) a.out_lse[n] = NAN;
      if (a.bad_rows) atomicAdd(a.bad_rows, 1);
    }
    return;
  }
  row.inv = kPerNat / tau;
  const Totals all = fill_buckets(row, sh);
  const double ln_mass = log(all.mass);
  const uint32_t want = min((uint32_t)k, all.finite);
  const int b = bucket_of_rank(sh, want);
  uint64_t lo = b == kBuckets - 1 ? (uint64_t)(kKeyNegInf + 1) << 32
                                  : (uint64_t)least_key(row, sh, b) << 32;
  if (sh.cnt[b + 1] > (uint32_t)kList) {
    // More than the list holds reach that bucket: the last token's own key.
    const uint32_t before = sh.cnt[b];
    lo = select_in_bucket(row, sh, b, sh.cnt[b + 1] - before, kByRank, want - before, 0.0).key;
  }
  const uint32_t m = gather(row, sh, lo, ~0ull);
  sort_list(sh, m);
  for (uint32_t i = threadIdx.x; i < (uint32_t)k; i += kThreads) {
    const bool there = i < want;
    const uint64_t t = there ? sh.list[i] : 0;
    const float z = there ? token_logit(t) : -INFINITY;
    ids[i] = there ? token_index(t) : -1;
    zs[i] = z;
    lps[i] = (float)(((double)z - row.zmax) / tau - ln_mass);
  }
  if (threadIdx.x == 0 && a.out_lse) a.out_lse[n] = (float)(row.zmax / tau + ln_mass);
}

}  // namespace

hipError_t launch_sample(const SelectArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)a.N);
  switch (a.dtype) {
    case LP_F32: sample_kernel<F32><<<grid, kThreads, 0, stream>>>(a); break;
    case LP_BF16: sample_kernel<BF16><<<grid, kThreads, 0, stream>>>(a); break;
    default: sample_kernel<F16><<<grid, kThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

hipError_t launch_top(const SelectArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)a.N);
  switch (a.dtype) {
    case LP_F32: top_kernel<F32><<<grid, kThreads, 0, stream>>>(a); break;
    case LP_BF16: top_kernel<BF16><<<grid, kThreads, 0, stream>>>(a); break;
    default: top_kernel<F16><<<grid, kThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace lp
