// Shared by the operators on rows of logits (include/liblp_logits.h):
// element types, row loads, and the launch interface between the C-ABI host
// code and the kernels.
#pragma once

#include <hip/hip_fp16.h>

#include "liblp_logits.h"
#include "lp_internal.h"

namespace lp {

// Element types of a row of logits. kVec elements make one 16-byte load.
struct F32 {
  using Raw = uint32_t;
  static constexpr int kVec = 4;
  static constexpr Raw kNegInf = 0xFF800000u;
  static __device__ __forceinline__ float value(Raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ Raw round(float v) { return __float_as_uint(v); }
};

struct BF16 {
  using Raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr Raw kNegInf = 0xFF80u;
  static __device__ __forceinline__ float value(Raw r) { return __uint_as_float((uint32_t)r << 16); }
  // Nearest, ties to even; a NaN keeps its top bits and stays one.
  static __device__ __forceinline__ Raw round(float v) {
    const __bf16 b = (__bf16)v;
    return __builtin_bit_cast(uint16_t, b);
  }
};

struct F16 {
  using Raw = uint16_t;
  static constexpr int kVec = 8;
  static constexpr Raw kNegInf = 0xFC00u;
  static __device__ __forceinline__ float value(Raw r) {
    return (float)__builtin_bit_cast(_Float16, r);
  }
  static __device__ __forceinline__ Raw round(float v) {
    const _Float16 h = (_Float16)v;
    return __builtin_bit_cast(uint16_t, h);
  }
};

constexpr int64_t dtype_bytes(int32_t dtype) { return dtype == LP_F32 ? 4 : 2; }

// One 16-byte group of a row: elements [i, i + kVec) of p. Groups are counted
// from the row's start, never from an aligned address, so which elements a
// lane holds does not depend on where the row lies (gfx950 takes global loads
// and stores of 16 bytes at any alignment of the element type). A group that
// reaches past `end` is loaded element by element and filled with -inf.
//
// The group stays packed in four registers; elements are taken out where they
// are used. fresh() makes the compiler forget what it has taken out, so that
// two passes over a group do not hold its elements unpacked in between.
template <class D>
struct Group {
  uint32_t w[4];

  __device__ __forceinline__ float get(int i) const {
    if constexpr (D::kVec == 4) return D::value(w[i]);
    else return D::value((typename D::Raw)(w[i >> 1] >> ((i & 1) * 16)));
  }
  __device__ __forceinline__ void set(int i, typename D::Raw r) {
    if constexpr (D::kVec == 4) w[i] = r;
    else if (i & 1) w[i >> 1] = (w[i >> 1] & 0xFFFFu) | ((uint32_t)r << 16);
    else w[i >> 1] = (w[i >> 1] & 0xFFFF0000u) | r;
  }
  __device__ __forceinline__ void fresh() {
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
  }
};

// Four words at any alignment of the element type, and the pointers to global
// memory that rows are read and written through: a pointer whose address space
// is lost in a struct would become flat accesses, which wait for LDS too.
typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
template <class T>
using Global = __attribute__((address_space(1))) T*;

template <class T>
__device__ __forceinline__ T read_global(const T* p, int64_t i) {
  return ((Global<const T>)p)[i];
}

// The group that starts at p, whole.
template <class D>
__device__ __forceinline__ Group<D> load_whole(const typename D::Raw* p) {
  const Words v = *(Global<const Words>)(const Words*)p;
  return {{v.x, v.y, v.z, v.w}};
}

template <class D>
__device__ __forceinline__ Group<D> load_group(const typename D::Raw* p, int64_t i, int64_t end) {
  if (i + D::kVec <= end) return load_whole<D>(p + i);
  constexpr uint32_t kFill = D::kVec == 4 ? (uint32_t)D::kNegInf : D::kNegInf * 0x10001u;
  Group<D> g = {{kFill, kFill, kFill, kFill}};
  if (i >= end) return g;
  const Global<const typename D::Raw> q = (Global<const typename D::Raw>)p;
#pragma unroll
  for (int j = 0; j < D::kVec; ++j) g.set(j, i + j < end ? q[i + j] : D::kNegInf);
  return g;
}

template <class D>
__device__ __forceinline__ void store_whole(typename D::Raw* p, const Group<D>& g) {
  // Streamed past the caches: gradients are not read again soon (bf16 rows of
  // 151 936, backward of 1 100 115 us and step over 2 048 319 us, with plain stores
  // 127 us and 359 us).
  __builtin_nontemporal_store((Words{g.w[0], g.w[1], g.w[2], g.w[3]}), (Global<Words>)(Words*)p);
}

template <class D>
__device__ __forceinline__ void store_group(typename D::Raw* p, int64_t i, int64_t end,
                                            const Group<D>& g) {
  if (i + D::kVec <= end) {
    store_whole<D>(p + i, g);
    return;
  }
  const Global<typename D::Raw> q = (Global<typename D::Raw>)p;
#pragma unroll
  for (int j = 0; j < D::kVec; ++j)
    if (i + j < end) {
      if constexpr (D::kVec == 4) q[i + j] = g.w[j];
      else q[i + j] = (typename D::Raw)(g.w[j >> 1] >> ((j & 1) * 16));
    }
}

// 2^t in fp64: 2^r for |r| <= 1/2 by the polynomial of degree 8 that meets it at
// the Chebyshev nodes (1.1e-12 relative at most, of either sign), then the exact
// scaling, to 0 or infinity far out. An infinite t gives NaN.
__device__ __forceinline__ double exp2_f64(double t) {
  const double n = rint(t), r = t - n;
  double p = 0x1.63d13639e5a95p-20;
  p = fma(p, r, 0x1.00dc4a53498e8p-16);
  p = fma(p, r, 0x1.4308ac85a7188p-13);
  p = fma(p, r, 0x1.5d8745a728180p-10);
  p = fma(p, r, 0x1.3b2ab7181b779p-7);
  p = fma(p, r, 0x1.c6b08dd6fd237p-5);
  p = fma(p, r, 0x1.ebfbdff823cedp-3);
  p = fma(p, r, 0x1.62e42fef84cf0p-1);
  p = fma(p, r, 1.0);
  int k;  // (the instruction saturates, which a conversion in C need not)
  asm("v_cvt_i32_f64 %0, %1" : "=v"(k) : "v"(n));
  return ldexp(p, k);
}

// 2^(t - 900) for t >= 0: two instructions fewer. 2^r by the polynomial of degree 8
// that meets it at the Chebyshev nodes of [0, 1] (1.1e-12 relative at most), times
// 2^-900. (A term fewer is off by 5.5e-11, which a near-certain token's score shows;
// it spares 1 920 rows of 151 936 logits 8 us of 238.)
// For t < 0 a factor of two may be missing, and far below the result is 0. So it is
// for -inf, whose fraction, a NaN, is clamped to 0. A NaN gives 2^-900 as well: the
// caller has to see it by itself.
constexpr double kExp2From = 900.0;
__device__ __forceinline__ double exp2_900(double t) {
  constexpr double kUnit = 0x1p-900;
  double r;
  int k;
  asm("v_fract_f64_e64 %0, %1 clamp" : "=v"(r) : "v"(t));
  asm("v_cvt_i32_f64 %0, %1" : "=v"(k) : "v"(t));  // (saturates)
  double p = 0x1.f733994251afap-20 * kUnit;
  p = fma(p, r, 0x1.dae9136bc3e6dp-17 * kUnit);
  p = fma(p, r, 0x1.456ef35ed7a3dp-13 * kUnit);
  p = fma(p, r, 0x1.5d5a07f99825bp-10 * kUnit);
  p = fma(p, r, 0x1.3b2cb95521505p-7 * kUnit);
  p = fma(p, r, 0x1.c6b074458219dp-5 * kUnit);
  p = fma(p, r, 0x1.ebfbe095b1b52p-3 * kUnit);
  p = fma(p, r, 0x1.62e42fee28c57p-1 * kUnit);
  p = fma(p, r, 0x1.00000000012b7p+0 * kUnit);
  return ldexp(p, k);
}

// Maximum and sum over a wave by the fixed XOR butterfly.
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

// ---- Distillation ---------------------------------------------------------

// A row's vocabulary is cut into slices of equal length (a multiple of the
// 16-byte group), one workgroup each. The cut depends on V_true and the dtype
// only: a row's sums have the same order in every batch.
constexpr int kDistillThreads = 256;
constexpr int kDistillWaves = kDistillThreads / 64;
constexpr int kDistillGroups = 4;  // 16-byte groups per thread and slice, at most
// Forward and step take one workgroup per row from this many rows on, where the
// row has at least three slices (with fewer, most of its 16 waves would idle:
// step over 2 304 bf16 rows of 1 500, 47 us against 27 us by slices; of 12 000,
// 59 us and 49 us; 1 000 rows of 20 000, three slices, 34 us against 37 us) and
// at most kRowMaxSlices. With few rows, cutting them fills the card. Step by rows
// and by slices, bf16 rows of 151 936: 64 rows 32 us and 21 us, 128 33 and 33, 200
// 40 and 45, 256 45 and 53, 300 62 and 59, 400 65 and 74, 2 048 316 and 360; fp32
// rows of 50 021: 64 20 and 21, 255 34 and 41, 500 55 and 64. (Both fill the card
// from 256 rows on; between 128 and 255 whole rows would gain up to a sixth.)
constexpr int kRowWaves = 16;
constexpr int64_t kRowMinRows = 256;
constexpr int kRowMinSlices = 3;
constexpr int kRowMaxSlices = 128;

struct DistillSlices {
  int32_t n;    // slices per row
  int64_t len;  // elements per slice
};
DistillSlices distill_slices(int64_t V_true, int32_t dtype);

struct DistillArgs {
  const void* logits;
  int64_t ld;
  int32_t dtype;
  int64_t T, V_true, V_columns;
  const int64_t* ids;      // [T, K]
  const float* teacher;    // [T, K]
  int32_t K;
  bool logprobs;           // teacher entries are logprobs, taken as they are
  double inv_tau;
  float scale2;            // log2(e) / temperature
  DistillSlices slices;
  float* part_m;           // [T][n] slice maximum of z
  double* part_s;          // [T][n] sum of exp((z - slice maximum) / tau)
  float* out_loss;         // [T]
  double* state;           // [T][4] or null
  const double* state_in;  // [T][4] (backward)
  const float* grad;       // [T] (backward)
  void* out_grad;          // [T, ld_grad] (backward)
  int64_t ld_grad;
  int32_t* bad_rows;       // or null
};

struct DistillWorkspace {
  size_t off_m, off_s, off_state, total;
};
DistillWorkspace distill_workspace_layout(int64_t T, int64_t V_true, int32_t dtype);

hipError_t launch_distill_forward(const DistillArgs& a, hipStream_t stream);
hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t stream);
// out_loss, state, grad and out_grad set; both directions.
hipError_t launch_distill_step(const DistillArgs& a, hipStream_t stream);

// ---- Selection (token draw and top logits) --------------------------------

constexpr int kSelectThreads = 512;

// What the buckets of a row, or of a slice of it, hold besides counts and masses.
struct RowFacts {
  uint32_t top;     // key of the largest logit
  uint32_t odd;     // a NaN or +inf is there
  uint32_t masked;  // -inf logits (in the last bucket's count), fill included
  uint32_t unused;
};

// A base m and the sum of 2^(z c - offset(m)) over a wave's part of a chunk.
struct SelectPart {
  float m;
  double s;
};

// Where the tokens that a draw from a row keeps end, and what they weigh: token v
// has the probability exp((z_v - base) / tau - ln_kept) where its key (the order
// of the selection) is at least `last`, else 0; its raw score is
// (z_v - base) / tau - ln_all.
struct SelectLimit {
  uint64_t last;
  double base, ln_kept, ln_all;
};
constexpr uint64_t kNoLimit = ~0ull;  // `last` of a row without a valid draw

struct SelectArgs {
  const void* logits;
  int64_t ld;
  int32_t dtype;
  int64_t N;
  int32_t V;
  // Token draw. A null array means that the scalar beside it holds.
  const float* u;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  float temperature, top_p, min_p;
  int32_t top_k;           // token draw's scalar; the k of the top logits
  int64_t* out_token;      // [N]
  float* out_logprob;      // [N], or [N, k] for the top logits
  float* out_processed;    // [N] or null
  int32_t* out_kept;       // [N] or null
  // Top logits.
  int64_t* out_ids;        // [N, k]
  float* out_logits;       // [N, k]
  float* out_lse;          // [N] or null
  int32_t* bad_rows;       // or null
  // Set by launch_select.
  int32_t slices;          // per row
  uint32_t* counts;        // [N][slices] listed tokens
  SelectPart* parts;       // [N][chunks][waves], where slices > 1
  uint64_t* keys;          // [N][slices][LP_TOP_MAX], where slices > 1
  // Of a slice that goes by buckets, where slices > 1.
  unsigned long long* masses;  // [N][slices][buckets]
  uint32_t* bucket_counts;     // [N][slices][buckets]
  RowFacts* facts;             // [N][slices]
  // Limits of drafted sequences' rows, settings per sequence: `logits` are the
  // targets' (drafts + 1 rows a sequence), N counts both kinds.
  const void* draft_logits;
  int64_t ld_draft, seqs;
  int32_t drafts;
  const int32_t* draft_counts;  // [seqs] or null: all of them
  SelectLimit* limits;          // [N]
  SelectPart* whole;            // [N][chunks][waves], of rows that are summed whole
  int32_t whole_blocks;         // workgroups that do so
};

struct SelectWorkspace {
  size_t off_counts, off_parts, off_keys, off_masses, off_bucket_counts, off_facts, total;
};
// Rows are cut where there are few: into `places` slices at most, over all rows.
constexpr int64_t kSelectPlaces = 512;  // see select.hip
SelectWorkspace select_workspace_layout(int64_t N, int64_t V, int32_t dtype,
                                        int64_t places = kSelectPlaces);
// Bytes that serve every number of rows up to N (fewer rows are cut into more
// slices, so one layout may be larger than that of more rows).
size_t select_workspace_most(int64_t N, int64_t V, int32_t dtype,
                             int64_t places = kSelectPlaces);

// Sets the slices and the workspace's parts.
void place_select(SelectArgs& a, void* workspace, int64_t places);
// Which ways the draw's rows can take, as far as the host sees the settings.
struct SelectWays {
  bool lists, buckets;
};
SelectWays select_ways(const SelectArgs& a);

// The token draw, or the top logits where u is null.
hipError_t launch_select(SelectArgs a, void* workspace, hipStream_t stream);

// ---- Verification of drafted tokens -----------------------------------------

struct VerifyArgs {
  SelectArgs rows;          // both models' rows and the settings
  const int64_t* draft_ids; // [seqs, drafts]
  const float* u;           // [seqs, drafts + 1]
  int64_t* out_tokens;      // [seqs, drafts + 1]
  int32_t* out_accepted;    // [seqs]
  float* out_logprob;       // [seqs, drafts + 1]
  float* out_processed;     // [seqs, drafts + 1] or null
  int32_t* bad_rows;        // or null
  // Set by launch_verify.
  double* sums;             // [seqs][stretches] of the last token's weights
  int32_t* verdicts;        // [seqs] what out_accepted gets
};

struct VerifyWorkspace {
  size_t off_select, off_limits, off_whole, off_sums, off_verdicts, total;
};
// Where a call's parts lie; `total` serves smaller calls too.
VerifyWorkspace verify_workspace_layout(int64_t seqs, int64_t drafts, int64_t V, int32_t dtype);

hipError_t launch_verify(VerifyArgs a, void* workspace, hipStream_t stream);

}  // namespace lp
