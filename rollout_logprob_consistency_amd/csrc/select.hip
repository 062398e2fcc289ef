// Token draw (lp_sample) and top logits (lp_top_logprobs): selections in the
// order (logit descending, index ascending) by rank and by probability mass.
//
// Two ways through a row, chosen by its settings alone:
//
// By a short list (top_k in [1, 420], the greedy draw, min-p alone, and up to 420
// top logits): collect_kernel reads the row once, keeps the tokens that can still
// be among the first in a list in LDS, and sums exp(z - m) per wave and chunk for
// the log-sum-exp, which log_sum corrects by the listed tokens. The list is
// sorted; everything else is decided in it, with weights and sums in fp64. Where
// there are few rows, a row is cut into slices, each leaves its list, and
// row_kernel joins them.
//
// By buckets (everything else, and rows whose list overflows): the weights are
// collected in 2 048 buckets of 1/32 nat, a count and a mass each, placed so
// that the maximum of the row's first chunk lies 24 nats below the top; a row
// that rises further is collected again from its own maximum. Inside bucket b
// a weight is the bucket's centre times P, |ln P| <= 1/64; P is taken in fp64
// and summed as an integer in units of 2^-43, so a bucket's mass does not
// depend on the order of its terms (integer atomics, in LDS and between
// slices). Prefix sums over the buckets find the bucket in which a rank or a
// mass is reached; only that bucket's tokens are then listed, sorted and
// summed.
#include <algorithm>

#include "logits_internal.h"

// Lambdas here capture by reference; one that is not inlined would put what it
// captures into scratch memory, whose loads wait for the row's.
#define LP_INLINE __attribute__((always_inline))

namespace lp {
namespace {

constexpr int kThreads = kSelectThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kGroups = 4;            // 16-byte groups per thread and chunk
constexpr int kBuckets = 2048;        // of 1/32 nat; the last one: weight 0
constexpr int kSlots = kBuckets + 64; // while they are collected
constexpr double kPerNat = 32.0;
constexpr double kHead = 768.0;       // the anchor's place: 24 nats from the top
constexpr int kPerThread = kBuckets / kThreads;
constexpr int kList = 4096;           // tokens listed at once
constexpr int kShort = 2048;          // ... by a workgroup of collect_kernel
// Largest top_k that goes by short lists. From about 440 on, ordinary rows list
// more than kShort before the first sort, and are gone through twice. Lists
// against buckets, bf16 rows of 151 936. Draws, 512 rows: k = 300 108 us and 116 us,
// 420 119 and 117, 460 211 and 119, 512 262 and 117; 64 rows: 300 65 and 60, 420 84
// and 61, 512 154 and 61 (512 rows of 262 144: 420 146 and 172). Top logits, 512
// rows: 300 101 and 137, 420 112 and 140, 460 282 and 145, 512 778 and 150; 64 rows:
// 420 79 and 81, 460 144 and 82; one row: 420 60 and 77, 512 62 and 80.
constexpr int kShortTop = 420;
constexpr int kListMax = LP_TOP_MAX;  // tokens that a slice leaves
constexpr int kMaxSlices = 512;       // of a row
constexpr uint32_t kOverflow = 0xFFFFFFFFu;    // a slice's count: take the buckets
constexpr double kUnit = 8796093022208.0;      // 2^43: the mass unit's inverse
constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer

template <class D>
constexpr int chunk_of() { return kThreads * kGroups * D::kVec; }
constexpr int kMaxParts = LP_SELECT_MAX_VOCAB / chunk_of<F32>() * kWaves;

using Part = SelectPart;

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
  // prefix sums (masses as doubles in units of the anchor's weight).
  union {
    unsigned long long mass[kSlots];
    double above[kBuckets + 1];
    Part parts[kMaxParts];  // once a row's list is made
  };
  uint32_t cnt[kSlots];
  // The listed tokens, or the finer buckets of one that is too full to list.
  union {
    uint64_t list[kList];
    struct {
      unsigned long long fmass[kBuckets];
      uint32_t fcnt[kBuckets];
    };
  };
  unsigned long long wave_u64[kWaves];
  double wave_f64[kWaves], shared_f64;
  uint32_t wave_u32[kWaves];
  float wave_f32[kWaves];
  uint32_t n_list, found;
  uint32_t found_cnt;
  unsigned long long found_mass;
  float least[4];
  RowFacts facts;
};

// A row and its scale. x(z) = 32 (anchor - z) / tau + 768; the bucket is
// rint(x), the last one from there on.
template <class D>
struct Row {
  const typename D::Raw* p;
  int V;
  double anchor, inv;  // inv = 32 / tau
  float zmax;

  __device__ __forceinline__ double x_of(float z) const {
    return fmin(fma(anchor - (double)z, inv, kHead), (double)(kBuckets - 1));
  }
  static __device__ __forceinline__ uint32_t bucket(double x) {
    return min((uint32_t)__double_as_longlong(x + kMagic), (uint32_t)(kBuckets - 1));
  }
  // Where a lane counts it. The last bucket weighs nothing and takes whole waves
  // (masked tokens, places behind the row), whose adds to one word would go one
  // by one: each lane has a word of its own for it.
  static __device__ __forceinline__ uint32_t slot(double x) {
    const uint32_t b = (uint32_t)__double_as_longlong(x + kMagic);
    return b < (uint32_t)(kBuckets - 1) ? b : kBuckets + (threadIdx.x & 63);
  }
  // exp((b - x) / 32) in units of 2^-43, b = rint(x), by its Taylor series to
  // degree 5 (|b - x| / 32 <= 1/64: truncation 2e-14 relative); the last term
  // rounds to an integer.
  static __device__ __forceinline__ unsigned long long mass(double x) {
    const double y = ((x + kMagic) - kMagic) - x;
    double p = kUnit / (120.0 * 33554432.0);       // 32^5 5!
    p = fma(p, y, kUnit / (24.0 * 1048576.0));
    p = fma(p, y, kUnit / (6.0 * 32768.0));
    p = fma(p, y, kUnit / (2.0 * 1024.0));
    p = fma(p, y, kUnit / 32.0);
    const double m = fma(p, y, kUnit + kMagic);
    return (unsigned long long)__double_as_longlong(m) -
           (unsigned long long)__double_as_longlong(kMagic);
  }
  // A weight of mass m in bucket b, in units of the anchor's weight.
  static __device__ __forceinline__ double unit(int b) {
    return exp_f64((kHead - (double)b) / kPerNat) / kUnit;
  }
  __device__ __forceinline__ double max_weight() const {
    return exp_f64(((double)zmax - anchor) * (inv / kPerNat));
  }

  __device__ __forceinline__ int chunks() const { return (V + chunk_of<D>() - 1) / chunk_of<D>(); }
  __device__ __forceinline__ void load(Group<D> (&g)[kGroups], int c) const {
    const int first = c * chunk_of<D>() + (int)threadIdx.x * D::kVec;
    if ((c + 1) * chunk_of<D>() <= V) {
#pragma unroll
      for (int j = 0; j < kGroups; ++j) g[j] = load_whole<D>(p + first + j * kThreads * D::kVec);
    } else {
#pragma unroll
      for (int j = 0; j < kGroups; ++j) g[j] = load_group<D>(p, first + j * kThreads * D::kVec, V);
    }
  }
  static __device__ __forceinline__ int index(int c, int j, int i) {
    return c * chunk_of<D>() + (j * kThreads + (int)threadIdx.x) * D::kVec + i;
  }
  // f(groups, chunk) for the chunks [c0, c1), the next one's loads in flight.
  template <class F>
  __device__ __forceinline__ void for_chunks(int c0, int c1, F f) const {
    Group<D> g[kGroups], next[kGroups];
    load(g, c0);
    for (int c = c0; c < c1; ++c) {
      if (c + 1 < c1) load(next, c + 1);
      f(g, c);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) g[j] = next[j];
    }
  }
  // f(logit, index) for every token; places behind the row are -inf.
  template <class F>
  __device__ __forceinline__ void for_each(F f) const {
    for_chunks(0, chunks(), [&](Group<D>(&g)[kGroups], int c) LP_INLINE {
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int i = 0; i < D::kVec; ++i) {
          f(g[j].get(i), index(c, j, i));
          if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
        }
    });
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


// ---- Sorting the list -------------------------------------------------------

template <int kJ>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
  if constexpr (kJ == 32) {
    return __shfl_xor((unsigned long long)v, 32);
  } else {
    auto half = [](int x) LP_INLINE {
      if constexpr (kJ <= 2) return xlane<kJ>(x);  // quad permutations are true exchanges
      else return __builtin_amdgcn_ds_swizzle(x, (kJ << 10) | 0x1F);
    };
    const uint32_t lo = (uint32_t)half((int)(uint32_t)v), hi = (uint32_t)half((int)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
  }
}

// Compare and exchange at distance kJ < 64 inside a wave.
template <int kJ>
__device__ __forceinline__ void exchange(uint64_t& e, bool descending, int lane) {
  const uint64_t o = lane_xor<kJ>(e);
  const bool larger = ((lane & kJ) == 0) == descending;
  e = larger == (e < o) ? o : e;
}

// The steps of distance kJ, kJ / 2, ..., 1 on both halves of 128 keys.
template <int kJ>
__device__ __forceinline__ void exchanges(uint64_t& e0, uint64_t& e1, bool d0, bool d1, int lane) {
  exchange<kJ>(e0, d0, lane);
  exchange<kJ>(e1, d1, lane);
  if constexpr (kJ > 1) exchanges<kJ / 2>(e0, e1, d0, d1, lane);
}
__device__ __forceinline__ void exchange_halves(uint64_t& e0, uint64_t& e1, bool descending) {
  const uint64_t hi = e0 > e1 ? e0 : e1, lo = e0 > e1 ? e1 : e0;
  e0 = descending ? hi : lo;
  e1 = descending ? lo : hi;
}
template <int kK>
__device__ __forceinline__ void sort_wave(uint64_t& e0, uint64_t& e1, int lane) {
  if constexpr (kK > 2) sort_wave<kK / 2>(e0, e1, lane);
  const bool d = (lane & kK) == 0;  // (kK = 64: the first half descends, the second ascends)
  exchanges<kK / 2>(e0, e1, kK == 64 ? true : d, kK == 64 ? false : d, lane);
}

// The list sorted descending: a bitonic network over a power of two of keys,
// at least 128, padded with zeros. A wave holds 128 keys in registers for all
// steps of distances up to 64; only longer ones go through LDS with a barrier
// (the plain network's 45 barriers for 512 keys become 6).
__device__ __forceinline__ void sort_list(uint64_t* list, uint32_t m) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t n = 128;
  while (n < m) n <<= 1;
  for (uint32_t i = m + threadIdx.x; i < n; i += kThreads) list[i] = 0;
  __syncthreads();
  for (uint32_t b = wave * 128; b < n; b += kWaves * 128) {
    uint64_t e0 = list[b + lane], e1 = list[b + 64 + lane];
    sort_wave<64>(e0, e1, lane);
    const bool d = (b & 128) == 0;
    exchange_halves(e0, e1, d);
    exchanges<32>(e0, e1, d, d, lane);
    list[b + lane] = e0;
    list[b + 64 + lane] = e1;
  }
  __syncthreads();
  for (uint32_t k = 256; k <= n; k <<= 1) {
    for (uint32_t j = k >> 1; j >= 128; j >>= 1) {
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
    for (uint32_t b = wave * 128; b < n; b += kWaves * 128) {
      uint64_t e0 = list[b + lane], e1 = list[b + 64 + lane];
      const bool d = (b & k) == 0;
      exchange_halves(e0, e1, d);
      exchanges<32>(e0, e1, d, d, lane);
      list[b + lane] = e0;
      list[b + 64 + lane] = e1;
    }
    __syncthreads();
  }
}

// A part of base m counts its exponents z c from the integer next to m c where
// fp32 has one (below 2^22, within 3/4; further out a rounded product is off by
// up to 2^15, and every exponential 0 or infinite), else from m c itself by
// differences of logits. c = log2(e) / tau as a float.
__device__ __forceinline__ bool near_offset(float m, float c) { return fabsf(m * c) < 0x1p22f; }
struct Offset {
  float base, b;  // exponents are (z - base) c - b
};
__device__ __forceinline__ Offset offset_of(float m, float c) {
  const bool near = near_offset(m, c);
  return {near || m == -INFINITY ? 0.0f : m, near ? rintf(m * c) : 0.0f};
}

// The sum of a group's exponentials: fp32, in order.
template <class D>
__device__ __forceinline__ float group_sum(const Group<D>& g, float c, Offset o) {
  float s = __builtin_amdgcn_exp2f(fmaf(g.get(0) - o.base, c, -o.b));
#pragma unroll
  for (int i = 1; i < D::kVec; ++i)
    s += __builtin_amdgcn_exp2f(fmaf(g.get(i) - o.base, c, -o.b));
  return s;
}

// A chunk is gone through in blocks of eight places.
template <class D>
constexpr int kBlocks = kGroups * D::kVec / 8;

// The part of a wave whose lanes hold these groups: the same terms in the same
// order wherever it is formed, fp32 inside a group and fp64 from there on, so
// that join_parts can take a group's sum out again. Its base is the maximum of
// the first groups alone, which spares most of a pass; where the sum gets out
// of 2^32, or is none, it is formed again from the maximum of all. logit(z, e)
// sees the logit of every place e of a block, block(k) the block's end.
template <class D, class F, class B>
__device__ __forceinline__ Part part_of(Group<D> (&g)[kGroups], float c, F logit, B block) {
  float m = g[0].get(0);
#pragma unroll
  for (int i = 1; i < D::kVec; ++i) m = fmaxf(m, g[0].get(i));
  m = wave_max_f32(m);
  const bool near = near_offset(m, c);
  const float b = near ? rintf(m * c) : 0.0f;
  float gs = 0.0f;
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kBlocks<D>; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = (k * 8 + e) / D::kVec, i = (k * 8 + e) % D::kVec;
      if (i == 0) g[j].fresh();
      const float z = g[j].get(i);
      const float t = __builtin_amdgcn_exp2f(fmaf(z, c, -b));
      gs = i == 0 ? t : gs + t;
      if (i == D::kVec - 1) s += (double)gs;
      logit(z, e);
    }
    block(k);
  }
  s = wave_sum(s);
  if (!(s < 0x1p32) || !near) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      g[j].fresh();
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) m = fmaxf(m, g[j].get(i));
    }
    m = wave_max_f32(m);
    const Offset o = offset_of(m, c);  // (masked tokens sum to 0)
    s = 0.0;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      g[j].fresh();
      s += (double)group_sum<D>(g[j], c, o);
    }
    s = wave_sum(s);
  }
  return {m, s};
}

// Which lanes' logits of a block are wanted, place by place. (Masks of a whole
// chunk would not fit the scalar registers.)
struct Hits {
  uint64_t masks[8];
  __device__ __forceinline__ void set(int e, bool hit) { masks[e] = __ballot(hit); }
};

// These tokens appended to the list, in any order. A wave asks for its places
// in the list once a block.
template <class D>
__device__ __forceinline__ void append(const Group<D> (&g)[kGroups], int k, const Hits& hits,
                                       int index0, uint64_t* list, uint32_t size,
                                       uint32_t* n_list) {
  uint64_t any = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) any |= hits.masks[e];
  if (any == 0) return;
  uint32_t total = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) total += (uint32_t)__popcll(hits.masks[e]);
  uint32_t at = 0;
  if ((threadIdx.x & 63) == 0) at = atomicAdd(n_list, total);
  at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint64_t mask = hits.masks[e];
    if (mask == 0) continue;
    const uint32_t to = at + lanes_below(mask);
    if ((mask >> (threadIdx.x & 63) & 1) && to < size) {
      const int j = (k * 8 + e) / D::kVec, i = (k * 8 + e) % D::kVec;
      list[to] = token_key(g[j].get(i), index0 + j * kThreads * D::kVec + i);
    }
    at += (uint32_t)__popcll(mask);
  }
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
  s.tau = a.temperatures ? read_global(a.temperatures, n) : a.temperature;
  s.top_p = a.top_ps ? read_global(a.top_ps, n) : a.top_p;
  s.min_p = a.min_ps ? read_global(a.min_ps, n) : a.min_p;
  s.top_k = a.top_ks ? read_global(a.top_ks, n) : a.top_k;
  s.u = read_global(a.u, n);
  s.greedy = s.tau == 0.0f;
  s.bad = !(s.greedy || (s.tau > 0.0f && isnormal(s.tau))) || isnan(s.u) || isnan(s.top_p) || isnan(s.min_p);
  if (s.greedy) s.tau = 1.0f;
  s.k = s.greedy ? 1u : (uint32_t)max(s.top_k, 0);
  s.kind = kBuckets_;
  if (!s.bad) {
    if (s.greedy || (s.top_k > 0 && s.top_k <= kShortTop)) s.kind = kTopK;
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
// which have to fit one list together; half of it for kTopK, as sorting a
// whole one costs more than the slices gain (draws with top-k 400 over bf16 rows
// of 151 936: 64 rows 83 us with whole lists and 71 us with half, 8 rows 109 us
// and 59 us).
__device__ __forceinline__ int slices_of(const SelectArgs& a, const Settings& s) {
  const int most = s.kind == kTopK ? kList / 2 / (int)s.k : kList / kListMax;
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
__device__ __forceinline__ void write_bad_top(const SelectArgs& a, int64_t n) {
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

// ln of the sum of all exp((z - top) / tau), top the largest logit. NaN where a
// NaN or +inf logit is.
//
// The parts' fp32 exponentials would leave an error of 1e-7 to 1e-6 of the whole
// sum, which is all of a confident row's score. So the groups that hold a listed
// token are taken out of their parts and summed again in fp64 (a group's largest
// token does that; if any of a group is listed, it is). What is left of the
// error is relative to the probability outside the listed groups. c's rounding
// is confined the same way: a part's base goes into the sum with tau itself,
// and differences inside the part alone with c. Products that a sum follows are
// fused here by name, as the same bits are due in every kernel that this is part
// of. (2 304 bf16 rows of 151 936, k =
// 64: 191 us with fp64 sums of groups and this, 183 us with fp32 sums alone; one
// fp32 row 0.5 us more.)
template <class D, class P>  // parts in LDS or in global memory
__device__ __forceinline__ double log_sum(const Row<D>& row, P parts, const uint64_t* list,
                                          uint32_t m, float tau, double* words) {
  const float top = token_logit(list[0]), c = scale2_of(tau);
  const double inv_tau = 1.0 / (double)tau;
  // exp of a part's offset against top's.
  auto scale_of = [&](float base) LP_INLINE {
    double x = ((double)base - (double)top) * inv_tau;
    if (near_offset(base, c))
      x = fma(fma((double)base, -(double)c, (double)rintf(base * c)), 0.69314718055994531, x);
    return exp_f64(x);
  };
  double s = 0.0;
  const int n = row.chunks() * kWaves;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float base = parts[i].m;
    const double t = parts[i].s;
    s = base == -INFINITY ? s + t : fma(t, scale_of(base), s);
  }
  for (uint32_t i = threadIdx.x; i < m; i += kThreads) {
    const int idx = token_index(list[i]), first = idx - idx % D::kVec;
    const Group<D> g = load_group<D>(row.p, first, row.V);
    bool largest = true;
#pragma unroll
    for (int e = 0; e < D::kVec; ++e)
      if (first + e != idx) largest &= token_key(g.get(e), first + e) < list[i];
    if (!largest) continue;
    const int at = idx % chunk_of<D>() / D::kVec % kThreads / 64;
    const float base = parts[idx / chunk_of<D>() * kWaves + at].m;
    double t = 0.0;
#pragma unroll
    for (int e = 0; e < D::kVec; ++e)
      t += exp_f64(((double)g.get(e) - (double)top) * inv_tau);
    s += fma(-(double)group_sum<D>(g, c, offset_of(base, c)), scale_of(base), t);
  }
  double all;
  block_scan(s, words, &all);
  return log(all < 1.0 ? 1.0 : all);  // top's own term is 1, the rest rounds; a NaN stays
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
__device__ __forceinline__ void finish_draw(const SelectArgs& a, const Settings& st, int64_t n, const uint64_t* list,
                            uint32_t m, double ln_all, Words& w) {
  // Lists are no longer than kListMax here.
  constexpr int kEach = kListMax / kThreads;
  const double tau = (double)st.tau, top = (double)token_logit(list[0]);
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
  auto mass_through = [&](uint32_t t) LP_INLINE {
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
    kept = min(kept, st.min_p > 1.0f ? 1u : first_index(&w.found, m, base, kEach, [&](int i) LP_INLINE {
                 return x[i] > most;
               }));
  }
  if (st.top_p < 1.0f && !st.greedy) {
    // The nucleus is of what top-k left, whatever min-p drops.
    const double want = (double)st.top_p * mass_through(min(st.k, m) - 1);
    const uint32_t p = want > 0.0 ? first_index(&w.found, m, base, kEach,
                                                [&](int i) LP_INLINE { return c[i] >= want; }) + 1
                                  : 1u;
    kept = min(kept, p);
  }
  const double mass = mass_through(kept - 1);
  const double u = st.greedy ? 0.0 : fmin(fmax((double)st.u, 0.0), 1.0 - 0x1p-24);
  const uint32_t rank =
      min(kept - 1, first_index(&w.found, kept, base, kEach, [&](int i) LP_INLINE { return c[i] > u * mass; }));
  if (threadIdx.x == 0) {
    const uint64_t t = list[rank];
    const double s = ((double)token_logit(t) - top) / tau;
    a.out_token[n] = token_index(t);
    a.out_logprob[n] = (float)(s - ln_all);
    if (a.out_processed) a.out_processed[n] = st.greedy ? 0.0f : (float)(s - log(mass));
    if (a.out_kept) a.out_kept[n] = (int32_t)kept;
  }
}

// The first k tokens from a sorted list of m.
__device__ __forceinline__ void finish_top(const SelectArgs& a, int64_t n, const uint64_t* list, uint32_t m,
                           double ln_all) {
  const double top = (double)token_logit(list[0]), tau = (double)a.temperature;
  for (uint32_t i = threadIdx.x; i < (uint32_t)a.top_k; i += kThreads) {
    const bool there = i < m;
    const uint64_t t = there ? list[i] : 0;
    const float z = there ? token_logit(t) : -INFINITY;
    const int64_t o = n * a.top_k + i;
    a.out_ids[o] = there ? token_index(t) : -1;
    a.out_logits[o] = z;
    a.out_logprob[o] = (float)(((double)z - top) / tau - ln_all);
  }
  if (threadIdx.x == 0 && a.out_lse) a.out_lse[n] = (float)(top / tau + ln_all);
}

struct CollectShared {
  union {
    uint64_t list[kShort];
    struct {  // a slice's buckets
      unsigned long long mass[kSlots];
      uint32_t cnt[kSlots];
    };
  };
  Part parts[kMaxParts];
  double wave_f64[kWaves], shared_f64;
  float wave_f32[kWaves];
  uint32_t n_list, found;
  RowFacts facts;
};

// ---- Filling the buckets ----------------------------------------------------

// The maximum of the first chunk that has a finite logit (or +inf): the
// anchor of the buckets. -inf where there is none.
template <class D>
__device__ __forceinline__ float anchor_of(const Row<D>& row, float* words) {
  float m = -INFINITY;
  for (int c = 0; c < row.chunks() && m == -INFINITY; ++c) {
    Group<D> g[kGroups];
    row.load(g, c);
    float t = -INFINITY;
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) t = fmaxf(t, g[j].get(i));
    m = block_max(t, words);
  }
  return m;
}

// Counts and masses of the chunks [c0, c1) into LDS (cleared here), and their
// facts. Logits above the first bucket land in the last one: the caller sees
// by the maximum that there are some. -inf goes to the last bucket and is
// counted apart.
template <class D, class S>
__device__ __forceinline__ void collect_buckets(const Row<D>& row, S& sh, int c0, int c1) {
  for (int i = threadIdx.x; i < kSlots; i += kThreads) {
    sh.mass[i] = 0;
    sh.cnt[i] = 0;
  }
  if (threadIdx.x == 0) sh.facts = {0u, 0u, 0u, 0u};
  __syncthreads();
  float top = -INFINITY;
  uint64_t odd = 0;  // by lane
  uint32_t masked = 0;
  row.for_chunks(c0, c1, [&](Group<D>(&g)[kGroups], int) LP_INLINE {
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
      for (int i = 0; i < D::kVec; ++i) {
        const float z = g[j].get(i);
        const double x = row.x_of(z);
        const uint32_t b = Row<D>::slot(x);
        atomicAdd(&sh.cnt[b], 1u);
        atomicAdd(&sh.mass[b], Row<D>::mass(x));
        top = fmaxf(top, z);
        odd |= __ballot(__builtin_amdgcn_classf(z, 0x203));  // NaN, +inf
        masked += (uint32_t)__popcll(__ballot(z == -INFINITY));
        if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
      }
  });
  top = wave_max_f32(top);
  if ((threadIdx.x & 63) == 0) {
    atomicMax(&sh.facts.top, key_of(top));
    if (odd) atomicOr(&sh.facts.odd, 1u);
    atomicAdd(&sh.facts.masked, masked);
  }
  __syncthreads();
  if (threadIdx.x < 64) atomicAdd(&sh.cnt[kBuckets - 1], sh.cnt[kBuckets + threadIdx.x]);
  __syncthreads();
}

// One slice of a row (the whole row where a.slices is 1).
template <class D, bool kTop>
__global__ __launch_bounds__(kThreads, 6) void collect_kernel(SelectArgs a) {
  __shared__ CollectShared sh;
  const int64_t n = blockIdx.x / (uint32_t)a.slices;
  const int slice = (int)(blockIdx.x - (uint32_t)n * (uint32_t)a.slices);
  const Settings st = settings_of(a, n);
  uint32_t* count = a.counts + n * a.slices;
  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  const int chunks = row.chunks(), tid = threadIdx.x, wave = tid >> 6;
  if constexpr (!kTop)
    if (st.kind == kBuckets_) {
      if (a.slices == 1 || st.bad) return;  // row_kernel collects by itself
      const int c0 = chunks * slice / a.slices, c1 = chunks * (slice + 1) / a.slices;
      row.anchor = (double)anchor_of(row, sh.wave_f32);
      row.inv = kPerNat / (double)st.tau;
      collect_buckets(row, sh, c0, c1);
      // Left for row_kernel as they are. (Added up by global atomics they would
      // have to be cleared first, a launch that costs each call 2 to 3 us.)
      const int64_t at = n * a.slices + slice;
      unsigned long long* mass = a.masses + at * kBuckets;
      uint32_t* cnt = a.bucket_counts + at * kBuckets;
      for (int i = tid; i < kBuckets; i += kThreads) {
        mass[i] = sh.mass[i];
        cnt[i] = sh.cnt[i];
      }
      if (tid == 0) a.facts[at] = sh.facts;
      return;
    }
  const int slices = slices_of(a, st);
  if (slice >= slices) return;
  const int c0 = chunks * slice / slices, c1 = chunks * (slice + 1) / slices;
  const float scale2 = scale2_of(st.tau);
  const float depth = st.kind == kMinP ? depth_of(st) : 0.0f;

  // Tokens from theta on enter the list. theta is a logit that k tokens reach
  // (kTopK), or the depth below one (kMinP); never below the finite ones.
  float theta = 0.0f;
  // The r-th largest of a wave's values, by taking the largest away r - 1 times.
  auto rth_largest = [&](float v, uint32_t r) LP_INLINE {
    float m = wave_max_f32(v);
    for (uint32_t i = 1; i < r; ++i) {
      const uint64_t at = __ballot(v == m);
      if ((tid & 63) == __ffsll((long long)at) - 1) v = -INFINITY;
      m = wave_max_f32(v);
    }
    return m;
  };

  // Loads are not taken ahead: with 80 registers three workgroups share a CU,
  // and their loads overlap each other's arithmetic (top 64 of 2 304 bf16 rows
  // of 151 936: 194 us; with the next chunk in registers 206 us, or 223 us with
  // the registers of two workgroups a CU).
  bool fits = true;
  for (int c = c0; c < c1 && fits; ++c) {
    Group<D> g[kGroups];
    row.load(g, c);
    if (c == c0) {
      float tm = -INFINITY, gm[kGroups];
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        gm[j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < D::kVec; ++i) gm[j] = fmaxf(gm[j], g[j].get(i));
        tm = fmaxf(tm, gm[j]);
      }
      if (st.kind == kTopK) {
        // A first theta: with r = ceil(k / 8), the least of the eight waves'
        // r-th largest thread maximum is reached by k tokens of this chunk
        // (with more than 256 wanted, of the four groups' maxima apart: 32 sets
        // of 64). In a chunk that the row ends in, of the sets that have a
        // token in every lane.
        const int groups = (min(row.V - c * chunk_of<D>(), chunk_of<D>())) / D::kVec;
        const int sets = min(groups / 64, st.k > 256 ? kGroups * kWaves : kWaves);
        const uint32_t r = (st.k + max(sets, 1) - 1) / max(sets, 1);
        float least = INFINITY;
        if (sets == 0 || r > 64) {
          least = -INFINITY;  // too few tokens for a bound
        } else if (st.k > 256) {
#pragma unroll
          for (int j = 0; j < kGroups; ++j)
            if (j * kWaves + wave < sets) least = fminf(least, rth_largest(gm[j], r));
        } else if (wave < sets) {
          least = rth_largest(tm, r);
        }
        theta = bound(-block_max(-least, sh.wave_f32));
      } else {
        theta = bound(block_max(tm, sh.wave_f32) - depth);
      }
      if (tid == 0) sh.n_list = 0;
      __syncthreads();
    }
    Hits hits;
    const Part p = part_of<D>(
        g, scale2, [&](float z, int e) LP_INLINE { hits.set(e, z >= theta); },
        [&](int k) LP_INLINE {
          append<D>(g, k, hits, Row<D>::index(c, 0, 0), sh.list, kShort, &sh.n_list);
        });
    if ((tid & 63) == 0) {
      if (a.slices == 1) sh.parts[c * kWaves + wave] = p;
      else a.parts[(n * chunks + c) * kWaves + wave] = p;
    }
    // After the 1st, 2nd, 4th, 8th, ... chunk, where a list has doubled, and
    // the last one: a list that has grown is sorted down to what can still be
    // needed. One that has lost tokens is given up.
    const int done = c - c0 + 1;
    const bool last = c + 1 == c1;
    if (!last && (done & (done - 1)) != 0) continue;
    __syncthreads();
    const uint32_t m = sh.n_list;
    __syncthreads();
    fits = m <= (uint32_t)kShort;
    if (!fits || (!last && m < (st.kind == kTopK ? 2 * st.k + 128 : 1024u))) continue;
    sort_list(sh.list, m);
    uint32_t keep = m;
    if (st.kind == kTopK) {
      keep = min(m, st.k);
      if (m >= st.k) theta = token_logit(sh.list[st.k - 1]);
    } else if (m > 0) {
      theta = bound(token_logit(sh.list[0]) - depth);
      constexpr int kEach = kShort / kThreads;
      keep = first_index(&sh.found, m, tid * kEach, kEach, [&](int i) LP_INLINE {
        return token_logit(sh.list[tid * kEach + i]) < theta;
      });
    }
    __syncthreads();
    if (tid == 0) sh.n_list = keep;
    __syncthreads();
  }
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
  if (tid == 0) count[0] = 0;
  const double ln_all = m == 0 ? NAN : log_sum(row, sh.parts, sh.list, m, st.tau, sh.wave_f64);
  if (isnan(ln_all)) {
    if (kTop) write_bad_top(a, n);
    else if (tid == 0) write_bad_draw(a, n);
  } else if (kTop) {
    finish_top(a, n, sh.list, m, ln_all);
  } else {
    finish_draw(a, st, n, sh.list, m, ln_all, sh);
  }
}

// ---- By buckets -------------------------------------------------------------

// Prefix sums over the collected buckets.
struct Totals {
  uint32_t finite;
  double mass;  // of all tokens, in units of the anchor's weight
};

template <class D>
__device__ __forceinline__ Totals sum_buckets(Shared& sh) {
  uint32_t c[kPerThread], cs = 0;
  double m[kPerThread], ms = 0.0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = threadIdx.x * kPerThread + i;
    const bool last = b == kBuckets - 1;
    c[i] = sh.cnt[b] - (last ? sh.facts.masked : 0u);
    m[i] = last ? 0.0 : (double)sh.mass[b] * Row<D>::unit(b);
    cs += c[i];
    ms += m[i];
  }
  Totals t;
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

// The buckets of a row: `anchor` and zmax set, `ready` where counts, masses
// and facts are collected already. False for a row without a draw.
template <class D>
__device__ __forceinline__ bool fill_buckets(Row<D>& row, Shared& sh, bool ready, Totals* all) {
  if (!ready) collect_buckets(row, sh, 0, row.chunks());
  row.zmax = key_value(sh.facts.top);
  if (sh.facts.odd || row.zmax == -INFINITY) return false;
  if (fma(row.anchor - (double)row.zmax, row.inv, kHead) < -0.5) {
    // The maximum lies above the buckets: once more, from the maximum itself.
    row.anchor = (double)row.zmax;
    __syncthreads();
    collect_buckets(row, sh, 0, row.chunks());
  }
  *all = sum_buckets<D>(sh);
  return true;
}

// Least logit whose bucket is at most b0 .. b3, by wave 0 .. 3 into sh.least
// (+inf where the maximum's bucket is beyond): a search over the finite keys, 64 at a time.
template <class D>
__device__ __forceinline__ void least_logits(const Row<D>& row, Shared& sh, int b0, int b1, int b2, int b3) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  __syncthreads();
  if (wave < 4) {
    const int b = wave == 0 ? b0 : (wave == 1 ? b1 : (wave == 2 ? b2 : b3));
    const bool some = b >= (int)Row<D>::bucket(row.x_of(row.zmax));
    uint32_t lo = kKeyNegInf + 1, hi = key_of(row.zmax);  // hi is in a bucket <= b
    if (some)
      while (lo < hi) {
        const uint32_t step = (hi - lo) / 64 + 1;
        const uint32_t probe = min(hi, lo + (uint32_t)lane * step);  // lo + 63 step may pass hi
        const uint64_t in = __ballot(Row<D>::bucket(row.x_of(key_value(probe))) <= (uint32_t)b);
        const int f = in ? __ffsll((long long)in) - 1 : 64;
        const uint32_t above = f < 64 ? min(hi, lo + (uint32_t)f * step) : hi;
        if (f > 0) lo = min(hi, lo + (uint32_t)(f - 1) * step) + 1;
        hi = above;
      }
    if (lane == 0) sh.least[wave] = some ? key_value(hi) : INFINITY;
  }
  __syncthreads();
}

// The largest finite float below hi (below both zeros where hi is one).
__device__ __forceinline__ float float_before(float hi) {
  return key_value(key_of(hi) - (hi == 0.0f ? 2u : 1u));
}

// Tokens with lo0 <= z < hi0 or lo1 <= z < hi1 appended to the list, in any
// order; returns their number (which may pass the list's size).
template <class D>
__device__ __forceinline__ uint32_t gather(const Row<D>& row, Shared& sh, float lo0, float hi0, float lo1,
                           float hi1) {
  // lo <= z < hi as one comparison: z is its own median with lo and the float
  // before hi.
  const float end0 = float_before(hi0), end1 = float_before(hi1);
  const bool two = lo1 < INFINITY;
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  row.for_chunks(0, row.chunks(), [&](Group<D>(&g)[kGroups], int c) LP_INLINE {
#pragma unroll
    for (int k = 0; k < kBlocks<D>; ++k) {
      Hits hits;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = g[(k * 8 + e) / D::kVec].get((k * 8 + e) % D::kVec);
        hits.set(e, __builtin_amdgcn_fmed3f(z, lo0, end0) == z);
      }
      if (two)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = g[(k * 8 + e) / D::kVec].get((k * 8 + e) % D::kVec);
          hits.masks[e] |= __ballot(__builtin_amdgcn_fmed3f(z, lo1, end1) == z);
        }
      append<D>(g, k, hits, Row<D>::index(c, 0, 0), sh.list, kList, &sh.n_list);
    }
  });
  __syncthreads();
  return sh.n_list;
}

// Where a selection ends inside a bucket: the token, its rank there (from 0)
// and the mass through it, in the bucket's units.
struct Found {
  uint64_t key;
  uint32_t rank;
  unsigned long long mass;
};

enum Mode { kByRank, kByMass, kByMassOver };

// The buckets whose tokens are listed and sorted: up to two ranges, the first
// one nearer the top.
struct Listed {
  int lo0 = 1, hi0 = 0, lo1 = 1, hi1 = 0;
};

// Part of a bucket of more tokens than can be listed: 2 048 finer buckets of
// equal key ranges, turn by turn, until the one in which the selection ends can
// be. Its tokens are listed; returns what lies before them. Out of line: only
// rows of many equal or near logits come here.
struct Refined {
  uint32_t cnt;
  unsigned long long mass;
};
template <class D>
__device__ __noinline__ Refined refine(Row<D> row, Shared& sh, float flo, float fhi,
                                       uint32_t count, Mode mode, uint32_t rank, double want) {
  uint32_t base_cnt = 0;
  unsigned long long base_mass = 0;
  auto reached = [&](uint32_t c, unsigned long long s) LP_INLINE {
    return mode == kByRank ? c >= rank : (mode == kByMass ? (double)s >= want : (double)s > want);
  };
  uint64_t lo = (uint64_t)key_of(flo) << 32;
  uint64_t hi = fhi > row.zmax ? ((uint64_t)key_of(row.zmax) << 32) | 0xFFFFFFFFull
                                         : ((uint64_t)key_of(fhi) << 32) - 1;
  while (count > (uint32_t)kList) {
    // The range shrinks 2 048-fold a turn, and keys are distinct, so this ends.
    const uint64_t range = hi - lo;
    const int bits = 64 - __clzll((long long)(range | 1));
    const int shift = bits > 11 ? bits - 11 : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kBuckets; i += kThreads) {
      sh.fmass[i] = 0;
      sh.fcnt[i] = 0;
    }
    __syncthreads();
    row.for_each([&](float z, int idx) LP_INLINE {
      const uint64_t k = token_key(z, idx);
      if (k >= lo && k <= hi) {
        const uint32_t f = (uint32_t)((hi - k) >> shift);
        atomicAdd(&sh.fcnt[f], 1u);
        atomicAdd(&sh.fmass[f], Row<D>::mass(row.x_of(z)));
      }
    });
    __syncthreads();
    uint32_t c = 0;
    unsigned long long s = 0;
    for (int i = 0; i < kPerThread; ++i) {
      c += sh.fcnt[threadIdx.x * kPerThread + i];
      s += sh.fmass[threadIdx.x * kPerThread + i];
    }
    uint32_t all_c;
    unsigned long long all_m;
    uint32_t cb = base_cnt + block_scan(c, sh.wave_u32, &all_c);
    unsigned long long mb = base_mass + block_scan(s, sh.wave_u64, &all_m);
    // First finer bucket through which the selection is reached; the last
    // occupied one where rounding of `want` leaves none.
    for (int i = 0; i < kPerThread; ++i) {
      const int f = threadIdx.x * kPerThread + i;
      const uint32_t c1 = cb + sh.fcnt[f];
      const unsigned long long m1 = mb + sh.fmass[f];
      const bool last = c1 == base_cnt + all_c;
      if (sh.fcnt[f] != 0 && (reached(c1, m1) || last) &&
          !(cb != base_cnt && reached(cb, mb))) {
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
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  row.for_each([&](float z, int idx) LP_INLINE {
    const uint64_t k = token_key(z, idx);
    if (k >= lo && k <= hi) {
      const uint32_t s = atomicAdd(&sh.n_list, 1u);
      if (s < (uint32_t)kList) sh.list[s] = k;
    }
  });
  __syncthreads();
  return {base_cnt, base_mass};
}

// The first token, in order, of bucket b at which
//   kByRank:     `rank` tokens of the bucket are reached (rank >= 1),
//   kByMass:     the mass through it is >= want,
//   kByMassOver: the mass through it is > want.
// Where no token's mass gets there (want is rounded), the last one.
template <class D>
__device__ __forceinline__ Found select_in_bucket(const Row<D>& row, Shared& sh, Listed& listed, int b, Mode mode,
                                  uint32_t rank, double want) {
  uint32_t count = sh.cnt[b + 1] - sh.cnt[b];
  uint32_t base_cnt = 0, at = 0, m = count;
  unsigned long long base_mass = 0;
  auto reached = [&](uint32_t c, unsigned long long s) LP_INLINE {
    return mode == kByRank ? c >= rank : (mode == kByMass ? (double)s >= want : (double)s > want);
  };
  if (b >= listed.lo0 && b <= listed.hi0) {
    at = sh.cnt[b] - sh.cnt[listed.lo0];
  } else if (b >= listed.lo1 && b <= listed.hi1) {
    at = (listed.lo0 <= listed.hi0 ? sh.cnt[listed.hi0 + 1] - sh.cnt[listed.lo0] : 0) +
         sh.cnt[b] - sh.cnt[listed.lo1];
  } else {
    least_logits(row, sh, b, b - 1, -1, -1);
    float flo = sh.least[0], fhi = sh.least[1];
    if (count > (uint32_t)kList) {
      listed = Listed();
      const Refined r = refine<D>(row, sh, flo, fhi, count, mode, rank, want);
      base_cnt = r.cnt;
      base_mass = r.mass;
    } else {
      gather(row, sh, flo, fhi, INFINITY, INFINITY);
      listed = Listed();
      listed.lo0 = listed.hi0 = b;
    }
    m = min(sh.n_list, (uint32_t)kList);
    __syncthreads();
    sort_list(sh.list, m);
  }

  // Masses through every listed token of the bucket, in order.
  constexpr int kEach = kList / kThreads;
  unsigned long long w[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t t = threadIdx.x * kEach + i;
    w[i] = t < m ? Row<D>::mass(row.x_of(token_logit(sh.list[at + t]))) : 0ull;
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
  r.key = sh.list[at + sh.found];
  r.rank = base_cnt + sh.found;
  r.mass = sh.found_mass;
  __syncthreads();
  return r;
}

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
// only a bucket's end is looked at; where rounding leaves none, the last
// occupied bucket that weighs.
__device__ __forceinline__ int bucket_of_mass(Shared& sh, double want, bool over) {
  int first = kBuckets, last = -1;
#pragma unroll
  for (int i = kPerThread - 1; i >= 0; --i) {
    const int b = threadIdx.x * kPerThread + i;
    const double end = sh.above[b + 1];
    const bool occupied = sh.cnt[b + 1] != sh.cnt[b] && b < kBuckets - 1;
    if (occupied && last < 0) last = b;
    if (occupied && (over ? end > want : end >= want)) first = b;
  }
  // Buckets ascend with lanes: the first lane that has one, the last occupied.
  const uint64_t hit = __ballot(first < kBuckets), some = __ballot(last >= 0);
  const int f = hit ? __builtin_amdgcn_readlane(first, __ffsll((long long)hit) - 1) : kBuckets;
  const int l = some ? __builtin_amdgcn_readlane(last, 63 - __clzll((long long)some)) : 0;
  if ((threadIdx.x & 63) == 0) {
    sh.wave_u32[threadIdx.x >> 6] = (uint32_t)f;
    sh.wave_u64[threadIdx.x >> 6] = (uint64_t)l;
  }
  __syncthreads();
  int b = kBuckets, e = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    b = min(b, (int)sh.wave_u32[w]);
    e = max(e, (int)sh.wave_u64[w]);
  }
  __syncthreads();
  return b < kBuckets ? b : e;
}

// A draw from filled buckets.
template <class D>
__device__ __forceinline__ void draw_from_buckets(const SelectArgs& a, const Settings& st, int64_t n,
                                  const Row<D>& row, const Totals& all, Shared& sh) {
  const double tau = (double)st.tau;
  const double u = fmin(fmax((double)st.u, 0.0), 1.0 - 0x1p-24);
  Listed listed;
  // Length of the kept prefix and its mass, filter by filter.
  uint32_t kept = all.finite;
  double mass = all.mass;
  if (st.top_k > 0 && (uint32_t)st.top_k < kept) {
    kept = (uint32_t)st.top_k;
    const int b = bucket_of_rank(sh, kept);
    if (b < kBuckets - 1) {
      const Found f = select_in_bucket(row, sh, listed, b, kByRank, kept - sh.cnt[b], 0.0);
      mass = sh.above[b] + (double)f.mass * Row<D>::unit(b);
    }
  }
  if (st.top_p < 1.0f) {
    const double want = (double)st.top_p * mass;
    if (want > 0.0) {
      const int b = bucket_of_mass(sh, want, false);
      if (!(st.min_p > 0.0f)) {
        // The kept mass lies between the bucket's ends, so the drawn token's
        // bucket is known to one or a few: list both in one pass.
        const int lo = bucket_of_mass(sh, u * sh.above[b], true);
        const int hi = bucket_of_mass(sh, u * sh.above[b + 1], true);
        Listed both;
        both.lo0 = lo;
        both.hi0 = hi >= b ? b : hi;
        if (hi < b) both.lo1 = both.hi1 = b;
        const uint32_t tokens = sh.cnt[both.hi0 + 1] - sh.cnt[lo] +
                                (hi < b ? sh.cnt[b + 1] - sh.cnt[b] : 0u);
        if (lo <= both.hi0 && tokens <= (uint32_t)kList) {
          least_logits(row, sh, both.hi0, lo - 1, hi < b ? b : -1, hi < b ? b - 1 : -1);
          const float l0 = sh.least[0], h0 = sh.least[1], l1 = sh.least[2], h1 = sh.least[3];
          const uint32_t m = gather(row, sh, l0, h0, l1, h1);
          __syncthreads();
          sort_list(sh.list, m);
          listed = both;
        }
      }
      const Found f = select_in_bucket(row, sh, listed, b, kByMass, 0,
                                       (want - sh.above[b]) / Row<D>::unit(b));
      const uint32_t m = sh.cnt[b] + f.rank + 1;
      if (m < kept) {
        kept = m;
        mass = sh.above[b] + (double)f.mass * Row<D>::unit(b);
      }
    } else {
      kept = 1;
      mass = row.max_weight();
    }
  }
  if (st.min_p > 1.0f) {  // no weight reaches it: the first token alone
    kept = 1;
    mass = row.max_weight();
  } else if (st.min_p > 0.0f) {
    // w >= min_p where 32 (max - z) / tau <= -32 ln min_p. The bucket that
    // this falls in is certain to one, so three are looked through.
    const double most = fmax(0.0, -log((double)st.min_p) * kPerNat);
    const double x0 = fma(row.anchor - (double)row.zmax, row.inv, kHead) + most;
    const int mid = (int)Row<D>::bucket(fmin(fmax(x0, 0.0), (double)(kBuckets - 1)));
    const int b0 = max(mid - 1, 0), b1 = min(mid + 1, kBuckets - 1);
    if (sh.cnt[b0] < kept) {
      uint32_t c[3] = {0, 0, 0};
      unsigned long long w[3] = {0, 0, 0};
      least_logits(row, sh, b1, b0 - 1, -1, -1);
      const float lo = sh.least[0], hi = sh.least[1];
      row.for_each([&](float z, int) LP_INLINE {
        if (z >= lo && z < hi && (row.zmax - (double)z) * row.inv <= most) {
          const double x = row.x_of(z);
          const int d = (int)Row<D>::bucket(x) - b0;
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (d == i) {
              ++c[i];
              w[i] += b0 + i < kBuckets - 1 ? Row<D>::mass(x) : 0ull;
            }
        }
      });
      uint32_t m = sh.cnt[b0];
      double s = sh.above[b0];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        uint32_t call;
        unsigned long long wall;
        block_scan(c[i], sh.wave_u32, &call);
        block_scan(w[i], sh.wave_u64, &wall);
        m += call;
        s += (double)wall * Row<D>::unit(b0 + i);
      }
      if (m < kept) {
        kept = m;
        mass = s;
      }
    }
  }

  const double want = u * mass;
  const int b = bucket_of_mass(sh, want, true);
  const Found f = select_in_bucket(row, sh, listed, b, kByMassOver, 0,
                                   (want - sh.above[b]) / Row<D>::unit(b));
  if (threadIdx.x == 0) {
    const float z = token_logit(f.key);
    // (z - anchor) / tau: the logarithms below are in the anchor's units.
    const double s = ((double)z - row.anchor) / tau;
    a.out_token[n] = token_index(f.key);
    a.out_logprob[n] = (float)(s - log(all.mass));
    if (a.out_processed) a.out_processed[n] = (float)(s - log(mass));
    if (a.out_kept) a.out_kept[n] = (int32_t)kept;
  }
}

// The log-sum of a row with its list, its parts formed (over the buckets' masses)
// as collect_kernel does.
template <class D>
__device__ __forceinline__ double log_sum_of_row(const Row<D>& row, float tau, Shared& sh, uint32_t m) {
  const float scale2 = scale2_of(tau);
  __syncthreads();
  row.for_chunks(0, row.chunks(), [&](Group<D>(&g)[kGroups], int c) LP_INLINE {
    const Part p = part_of<D>(g, scale2, [](float, int) LP_INLINE {}, [](int) LP_INLINE {});
    if ((threadIdx.x & 63) == 0) sh.parts[c * kWaves + (threadIdx.x >> 6)] = p;
  });
  __syncthreads();
  return log_sum(row, (const Part*)sh.parts, sh.list, m, tau, sh.wave_f64);
}

// A row of the short lists whose list overflowed: its tokens by selection,
// then the same ending, so that its results do not depend on how the row was
// cut. A row where min-p leaves more than kListMax goes by buckets for good.
template <class D, bool kTop>
__device__ __noinline__ void list_by_buckets(SelectArgs a, Settings st, int64_t n, Row<D> row,
                                             Shared& sh) {
  row.anchor = (double)anchor_of(row, sh.wave_f32);
  row.inv = kPerNat / (double)st.tau;
  Totals all;
  if (!fill_buckets(row, sh, false, &all)) {
    if constexpr (kTop) write_bad_top(a, n);
    else if (threadIdx.x == 0) write_bad_draw(a, n);
    return;
  }
  if constexpr (!kTop)
    if (st.kind == kMinP) {
      const float lo = bound(row.zmax - depth_of(st));
      // Far more than a short list holds, by the buckets above lo's alone, or
      // by the list itself.
      bool many = sh.cnt[Row<D>::bucket(row.x_of(lo))] > (uint32_t)kListMax;
      if (!many) many = gather(row, sh, lo, INFINITY, INFINITY, INFINITY) > (uint32_t)kListMax;
      if (many) {
        draw_from_buckets(a, st, n, row, all, sh);
        return;
      }
      const uint32_t m = sh.n_list;
      __syncthreads();
      sort_list(sh.list, m);
      finish_draw(a, st, n, sh.list, m, log_sum_of_row(row, st.tau, sh, m), sh);
      return;
    }
  const uint32_t want = min(st.k, all.finite);
  const int b = bucket_of_rank(sh, want);
  uint32_t m = sh.cnt[b + 1];
  if (m <= (uint32_t)kList) {
    least_logits(row, sh, b, -1, -1, -1);
    const float lo = sh.least[0];
    m = gather(row, sh, lo, INFINITY, INFINITY, INFINITY);
  } else {
    // More than the list holds reach that bucket: up to the last token's key.
    Listed none;
    const uint64_t last =
        select_in_bucket(row, sh, none, b, kByRank, want - sh.cnt[b], 0.0).key;
    if (threadIdx.x == 0) sh.n_list = 0;
    __syncthreads();
    row.for_each([&](float z, int idx) LP_INLINE {
      const uint64_t k = token_key(z, idx);
      if (k >= last && z != -INFINITY) {
        const uint32_t s = atomicAdd(&sh.n_list, 1u);
        if (s < (uint32_t)kList) sh.list[s] = k;
      }
    });
    __syncthreads();
    m = sh.n_list;
  }
  __syncthreads();
  sort_list(sh.list, m);
  const double ln_all = log_sum_of_row(row, st.tau, sh, want);
  if constexpr (kTop) finish_top(a, n, sh.list, want, ln_all);
  else finish_draw(a, st, n, sh.list, want, ln_all, sh);
}

// One row: its slices' lists or buckets joined, or the whole of it.
template <class D, bool kTop>
__device__ __forceinline__ void finish_row(const SelectArgs& a, int64_t n, Shared& sh) {
  const Settings st = settings_of(a, n);
  Row<D> row;
  row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
  row.V = a.V;
  if constexpr (!kTop)
    if (st.kind == kBuckets_) {
      if (st.bad) {
        if (threadIdx.x == 0) write_bad_draw(a, n);
        return;
      }
      row.inv = kPerNat / (double)st.tau;
      row.anchor = (double)anchor_of(row, sh.wave_f32);
      const bool ready = a.slices > 1;
      if (ready) {
        const int64_t at = n * a.slices;
        unsigned long long m[kPerThread];
        uint32_t c[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) m[i] = c[i] = 0;
        for (int t = 0; t < a.slices; ++t)
#pragma unroll
          for (int i = 0; i < kPerThread; ++i) {
            const int64_t b = (at + t) * kBuckets + threadIdx.x + i * kThreads;
            m[i] += read_global(a.masses, b);
            c[i] += read_global(a.bucket_counts, b);
          }
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          sh.mass[threadIdx.x + i * kThreads] = m[i];
          sh.cnt[threadIdx.x + i * kThreads] = c[i];
        }
        if (threadIdx.x == 0) sh.facts = {0u, 0u, 0u, 0u};
        __syncthreads();
        if ((int)threadIdx.x < a.slices) {
          const RowFacts f = a.facts[at + threadIdx.x];
          atomicMax(&sh.facts.top, f.top);
          atomicOr(&sh.facts.odd, f.odd);
          atomicAdd(&sh.facts.masked, f.masked);
        }
        __syncthreads();
      }
      Totals all;
      if (fill_buckets(row, sh, ready, &all)) draw_from_buckets(a, st, n, row, all, sh);
      else if (threadIdx.x == 0) write_bad_draw(a, n);
      return;
    }
  if constexpr (kTop)
    if (st.k > (uint32_t)kShortTop) {  // no lists were collected
      list_by_buckets<D, kTop>(a, st, n, row, sh);
      return;
    }
  // The slices' counts, and where each list starts.
  const int slices = slices_of(a, st);
  const uint32_t c = (int)threadIdx.x < slices ? read_global(a.counts, n * a.slices + threadIdx.x) : 0u;
  if (threadIdx.x == 0) sh.found = 0;
  __syncthreads();
  if (c == kOverflow) sh.found = 1;
  uint32_t m;
  const uint32_t at = block_scan(c, sh.wave_u32, &m);
  if (sh.found) {
    __syncthreads();
    list_by_buckets<D, kTop>(a, st, n, row, sh);
    return;
  }
  if (a.slices == 1) return;  // collect_kernel has finished the row
  if ((int)threadIdx.x < slices) {
    sh.cnt[threadIdx.x] = at;
    sh.cnt[kMaxSlices + threadIdx.x] = c;
  }
  __syncthreads();
  for (int i = threadIdx.x >> 6; i < slices; i += kWaves) {
    const uint64_t* keys = a.keys + (n * a.slices + i) * kListMax;
    const uint32_t to = sh.cnt[i], len = sh.cnt[kMaxSlices + i];
    for (uint32_t j = threadIdx.x & 63; j < len; j += 64) sh.list[to + j] = read_global(keys, j);
  }
  __syncthreads();
  sort_list(sh.list, m);
  if (st.kind == kTopK) {
    m = min(m, st.k);
  } else {
    constexpr int kEach = kList / kThreads;
    const uint32_t base = threadIdx.x * kEach;
    const float theta = m > 0 ? bound(token_logit(sh.list[0]) - depth_of(st)) : 0.0f;
    m = first_index(&sh.found, m, base, kEach,
                    [&](int i) LP_INLINE { return token_logit(sh.list[base + i]) < theta; });
    if (m > (uint32_t)kListMax) {
      list_by_buckets<D, kTop>(a, st, n, row, sh);
      return;
    }
  }
  const Global<const Part> parts = (Global<const Part>)(a.parts + n * row.chunks() * kWaves);
  const double ln_all = m == 0 ? NAN : log_sum(row, parts, sh.list, m, st.tau, sh.wave_f64);
  if (isnan(ln_all)) {
    if constexpr (kTop) write_bad_top(a, n);
    else if (threadIdx.x == 0) write_bad_draw(a, n);
    return;
  }
  if constexpr (kTop) finish_top(a, n, sh.list, m, ln_all);
  else finish_draw(a, st, n, sh.list, m, ln_all, sh);
}

template <class D, bool kTop>
__global__ __launch_bounds__(kThreads, 4) void row_kernel(SelectArgs a) {
  __shared__ Shared sh;
  finish_row<D, kTop>(a, blockIdx.x, sh);
}

// The rows of the top logits whose list overflowed, where collect_kernel has
// finished all others (a.slices == 1): kCheckRows rows a workgroup, one after
// the other, so for lists that seldom do (row_kernel takes all rows of longer
// lists: top 1 024 of 300 bf16 rows of 151 936 146 us, by this kernel 751 us).
constexpr int kCheckRows = 8;
template <class D>
__global__ __launch_bounds__(kThreads, 4) void overflow_kernel(SelectArgs a) {
  __shared__ Shared sh;
  const int64_t n0 = (int64_t)blockIdx.x * kCheckRows;
  const int64_t mine = n0 + (threadIdx.x & 63);
  uint64_t over = __ballot((threadIdx.x & 63) < kCheckRows && mine < a.N &&
                           read_global(a.counts, min(mine, a.N - 1)) == kOverflow);
  while (over) {
    const int64_t n = n0 + __ffsll((long long)over) - 1;
    over &= over - 1;
    Row<D> row;
    row.p = static_cast<const typename D::Raw*>(a.logits) + n * a.ld;
    row.V = a.V;
    list_by_buckets<D, true>(a, settings_of(a, n), n, row, sh);
    __syncthreads();
  }
}

template <class D, bool kTop>
hipError_t launch(const SelectArgs& a, bool lists, bool buckets, hipStream_t stream) {
  hipError_t e;
  if (lists || (buckets && a.slices > 1)) {
    collect_kernel<D, kTop><<<dim3((uint32_t)(a.N * a.slices)), kThreads, 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (kTop && lists && a.slices == 1)
    overflow_kernel<D><<<dim3((uint32_t)((a.N + kCheckRows - 1) / kCheckRows)), kThreads, 0,
                         stream>>>(a);
  else
    row_kernel<D, kTop><<<dim3((uint32_t)a.N), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Slices of a row: whole chunks, in all at most two workgroups for each of the
// card's 256 CUs. Times with 256, 512, 768 and 1 024 workgroups at most: top 100 of
// fp16 rows of 50 021, 100 rows 29, 30, 30 and 30 us, 200 rows 33, 34, 34 and 41, 300
// rows 40, 40, 42 and 44, 400 rows 42, 41, 42 and 51; draws over rows of 151 936, 64
// bf16 rows by top-k 20 30, 30, 27 and 27, 300 rows 55, 55, 52 and 53, 512 rows 61, 61,
// 61 and 73; 64 fp32 rows by nucleus 93, 96, 97 and 103.
constexpr int64_t kSelectPlaces = 512;
static_assert(kSelectPlaces <= kMaxSlices, "slices of one row");
static int64_t select_chunks(int64_t V, int32_t dtype) {
  const int64_t chunk = (int64_t)kThreads * kGroups * (16 / dtype_bytes(dtype));
  return (V + chunk - 1) / chunk;
}
static int64_t select_slices(int64_t N, int64_t V, int32_t dtype) {
  return std::max<int64_t>(
      1, std::min(select_chunks(V, dtype), kSelectPlaces / std::max<int64_t>(N, 1)));
}

// A count per row or slice; parts of `cut_rows` rows and the rest of `cut_slices`
// slices, which only cut rows need.
static SelectWorkspace layout_of(size_t counts, size_t cut_rows, size_t cut_slices, size_t chunks) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  SelectWorkspace w;
  w.off_counts = 0;
  w.off_parts = up(counts * sizeof(uint32_t));
  w.off_keys = w.off_parts + up(cut_rows * chunks * kWaves * sizeof(Part));
  w.off_masses = w.off_keys + up(cut_slices * kListMax * sizeof(uint64_t));
  w.off_bucket_counts = w.off_masses + cut_slices * kBuckets * sizeof(unsigned long long);
  w.off_facts = w.off_bucket_counts + cut_slices * kBuckets * sizeof(uint32_t);
  w.total = up(w.off_facts + cut_slices * sizeof(RowFacts));
  return w;
}

SelectWorkspace select_workspace_layout(int64_t N, int64_t V, int32_t dtype) {
  const int64_t slices = select_slices(N, V, dtype);
  const size_t all = (size_t)(N * slices);
  return layout_of(all, slices > 1 ? (size_t)N : 0, slices > 1 ? all : 0, select_chunks(V, dtype));
}

size_t select_workspace_most(int64_t N, int64_t V, int32_t dtype) {
  // Every term of layout_of at its largest over 1 .. N rows.
  const int64_t chunks = select_chunks(V, dtype);
  const int64_t cut_rows = chunks > 1 ? std::min(N, kSelectPlaces / 2) : 0;
  const int64_t cut_slices = std::min(kSelectPlaces, cut_rows * chunks);
  return layout_of((size_t)std::max(N, cut_slices), (size_t)cut_rows, (size_t)cut_slices,
                   (size_t)chunks)
      .total;
}

hipError_t launch_select(SelectArgs a, void* workspace, hipStream_t stream) {
  const SelectWorkspace w = select_workspace_layout(a.N, a.V, a.dtype);
  char* base = static_cast<char*>(workspace);
  a.slices = (int32_t)select_slices(a.N, a.V, a.dtype);
  a.counts = reinterpret_cast<uint32_t*>(base + w.off_counts);
  a.parts = reinterpret_cast<SelectPart*>(base + w.off_parts);
  a.keys = reinterpret_cast<uint64_t*>(base + w.off_keys);
  a.masses = reinterpret_cast<unsigned long long*>(base + w.off_masses);
  a.bucket_counts = reinterpret_cast<uint32_t*>(base + w.off_bucket_counts);
  a.facts = reinterpret_cast<RowFacts*>(base + w.off_facts);
  const bool top = a.u == nullptr;
  // Which ways the rows can take, as far as the host sees the settings.
  const bool seen = !a.temperatures && !a.top_ks && !a.top_ps && !a.min_ps;
  const bool short_list = a.temperature == 0.0f || (a.top_k > 0 && a.top_k <= kShortTop) ||
                          (a.top_k <= 0 && a.top_p >= 1.0f && a.min_p > 0.0f && a.min_p <= 1.0f);
  const bool lists = top ? a.top_k <= kShortTop : !seen || short_list;
  const bool buckets = !top && (!seen || !short_list);
  switch (a.dtype) {
    case LP_F32:
      return top ? launch<F32, true>(a, lists, buckets, stream)
                 : launch<F32, false>(a, lists, buckets, stream);
    case LP_BF16:
      return top ? launch<BF16, true>(a, lists, buckets, stream)
                 : launch<BF16, false>(a, lists, buckets, stream);
    default:
      return top ? launch<F16, true>(a, lists, buckets, stream)
                 : launch<F16, false>(a, lists, buckets, stream);
  }
}

}  // namespace lp
