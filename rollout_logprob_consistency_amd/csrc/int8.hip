// The 8-bit LM head on gfx950: rows of logits (lp_logits_int8) and scores of
// given tokens (lp_score_int8).
//
//   z[t, v] = (S x_scale[t]) w_scale[v],  S = sum_k x[t, k] w[v, k]
//
// by v_mfma_i32_16x16x64_i8 with 32-bit integer sums. They are exact, so in
// which order, by which kernel and by how many waves a sum over the hidden
// dimension is formed changes no bit; what has to be fixed for a row's score
// not to depend on its batch is the order of the floating-point operations
// behind it, which block_lse and the merge fix.
//
// Placement. A block is 128 vocabulary rows by 16 tokens of a wave: eight MFMA
// tiles, whose row m of tile i is vocabulary row
//   32 (i / 2) + 8 (m / 4) + 4 (i % 2) + m % 4.
// An MFMA's result has the token l & 15 and the rows 4 (l >> 4) + r, r < 4, in
// lane l; so lane l holds four runs of eight vocabulary rows, run q from
// 32 q + 8 (l >> 4) on: a run of 16-bit logits is one 16-byte store, the four
// lanes of a token store 64 bytes side by side, and the reduction over the
// vocabulary is mostly inside a lane.
#include <math.h>

#include <algorithm>

#include "int8_internal.h"
#include "tile_common.h"

namespace lp {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTiles = 8;            // MFMA tiles of a block along the vocabulary
constexpr int kPerLane = 4 * kTiles; // vocabulary rows of a lane
constexpr double kLn2 = 0.693147180559945309;
static_assert(kInt8BlockV == 16 * kTiles, "a block is one wave's");

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// 16 vocabulary rows x 16 tokens x 64 hidden elements.
__device__ __forceinline__ i32x4 mma(const i32x4& w, const i32x4& x, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
}

// Buffer resource over `bytes` bytes from a wave-uniform base: what lies behind
// it reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return row_rsrc(base, (uint32_t)(bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0ll : bytes));
}

// The row of W that lane l's fragment of tile i holds, from the block's first.
__device__ __forceinline__ int fragment_row(int lane, int i) {
  return 32 * (i >> 1) + 8 * ((lane & 15) >> 2) + 4 * (i & 1) + (lane & 3);
}
// The vocabulary row of a lane's k-th result (tile k / 4, register k % 4), from
// the block's first; rows ascend with k. lg = lane >> 4.
__device__ __forceinline__ int result_row(int lg, int k) {
  return 32 * (k >> 3) + 8 * lg + (k & 7);
}

// ---- Scores -----------------------------------------------------------------

// A logit from its sum, each step rounded to fp32. The empty statement hides the
// product from what follows: the compiler would fuse it with the rounding to
// fp16 (v_fma_mixlo) and skip fp32's.
__device__ __forceinline__ float logit(int sum, float xs, float ws) {
  float z = (float)sum * xs * ws;
  asm("" : "+v"(z));
  return z;
}

// Maximum of z = y f (log2 units) and sum of 2^(z - maximum) of a block for the
// lane's token, y[k] the lane's k-th row's (-inf f behind the vocabulary): over the
// lane's rows in ascending order, then the lanes l ^ 16 and l ^ 32, which end with
// the same bits. A NaN or +inf logit makes the sum NaN.
__device__ __forceinline__ void block_lse(const float (&y)[kPerLane], float f, float& m_out,
                                          float& s_out) {
  float hi = y[0], lo = y[0];
#pragma unroll
  for (int k = 1; k < kPerLane; ++k) {
    hi = fmaxf(hi, y[k]);
    lo = fminf(lo, y[k]);
  }
  float m = (f < 0.0f ? lo : hi) * f;
  m = fmaxf(m, xor_lane<16>(m));
  m = fmaxf(m, xor_lane<32>(m));
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) s += fast_exp2(__builtin_fmaf(y[k], f, -base));
  s += xor_lane<16>(s);
  s += xor_lane<32>(s);
  m_out = m;
  s_out = s;
}

// Joins (m, s) to (M, S). Nothing (-inf, 0) joins without a trace; a NaN stays.
__device__ __forceinline__ void lse_fold(float& M, float& S, float m, float s) {
  const float Mn = fmaxf(M, m), base = Mn == -INFINITY ? 0.0f : Mn;
  S = __builtin_fmaf(s, fast_exp2(m - base), S * fast_exp2(M - base));
  M = Mn;
}

// ---- What a wave does with a block's sums -----------------------------------

// The scales of a lane's rows of the block that starts at v0; rows behind V take
// the last one's.
struct RowScales {
  float s[kPerLane];
};
__device__ __forceinline__ RowScales row_scales(const Int8Args& a, int v0, int lg) {
  RowScales w;
  if (v0 + kInt8BlockV <= a.V) {
    const Global<const Words> p = (Global<const Words>)(const Words*)(a.w_scale + v0 + 8 * lg);
#pragma unroll
    for (int q = 0; q < kTiles; ++q) {
      const Words x = p[8 * (q >> 1) + (q & 1)];
      w.s[4 * q] = __uint_as_float(x.x);
      w.s[4 * q + 1] = __uint_as_float(x.y);
      w.s[4 * q + 2] = __uint_as_float(x.z);
      w.s[4 * q + 3] = __uint_as_float(x.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
      w.s[k] = read_global(a.w_scale, min(v0 + result_row(lg, k), a.V - 1));
  }
  return w;
}

// What a kernel makes of the sums: logits of type D, or scores, of logits in fp32
// or rounded to bf16 first.
template <class D>
struct Logits {
  using Type = D;
};
struct Scores {};
struct RoundedScores {};

// What of the outputs a wave's block reaches, as a buffer: lanes without a token,
// or a token without a place, store behind its end, which drops it. So no lane is
// ever masked while the accumulators are taken out; in a masked region the compiler
// has parked registers in freed accumulators for the lanes at work alone (the build
// looks that no accumulator is written but by an MFMA).
struct Place {
  uint8_t* p;
  uint32_t bytes;
  uint32_t token;  // the lane's token's offset
};

// Of the block that starts at v0, for the 16 tokens from t0 on (or `tokens`, 16 by
// 16); lane: in its row of 16.
template <class D>
__device__ __forceinline__ Place place_of(Logits<D>, const Int8Args& a, int v0, int t0, int tokens,
                                          int lane) {
  constexpr int kSize = sizeof(typename D::Raw);
  const int rows = min(a.T - t0, tokens);
  return {static_cast<uint8_t*>(a.out) + ((int64_t)t0 * a.ld_out + v0) * kSize,
          rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * a.ld_out + a.V - v0) * kSize) : 0u,
          (uint32_t)((lane & 15) * a.ld_out) * kSize};
}
template <class Out>
__device__ __forceinline__ Place place_of(Out, const Int8Args&, int, int, int, int) {
  return {};
}

// The block that starts at v0, for 16 tokens from t on, the j-th 16 of the place's;
// sums[k] is the lane's k-th sum, xs its token's scale.
template <class D>
__device__ __forceinline__ void finish_block(Logits<D>, const Int8Args& a, const Place& at, int j,
                                             const int (&sums)[kPerLane], const RowScales& w,
                                             int v0, int, float xs, int lg) {
  constexpr int kSize = sizeof(typename D::Raw);
  typedef uint32_t Quad __attribute__((ext_vector_type(4)));
  const __amdgpu_buffer_rsrc_t r = row_rsrc(at.p, at.bytes);
  const uint32_t off = at.token + (uint32_t)(16 * j * a.ld_out) * kSize + 8 * lg * kSize;
  if (v0 + kInt8BlockV <= a.V) {
#pragma unroll
    for (int k0 = 0; k0 < kPerLane; k0 += D::kVec) {
      Group<D> g = {};
#pragma unroll
      for (int e = 0; e < D::kVec; ++e) g.set(e, D::round(logit(sums[k0 + e], xs, w.s[k0 + e])));
      __builtin_amdgcn_raw_buffer_store_b128(Quad{g.w[0], g.w[1], g.w[2], g.w[3]}, r,
                                             off + result_row(0, k0) * kSize, 0, 0);
    }
  } else {
    int left = a.V - v0 - 8 * lg;
    asm volatile("" : "+v"(left));  // (or all tokens' comparisons are made, and kept, at once)
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const typename D::Raw z = D::round(logit(sums[k], xs, w.s[k]));
      const uint32_t o = result_row(0, k) < left ? off + result_row(0, k) * kSize : 0xFFFFFFFCu;
      if constexpr (kSize == 4) __builtin_amdgcn_raw_buffer_store_b32(z, r, o, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b16(z, r, o, 0, 0);
    }
  }
}

// A partial of the block; lanes that have none store behind the plane's end.
__device__ __forceinline__ void store_partial(const Int8Args& a, const float (&y)[kPerLane],
                                              float f, int v0, int t, int lg) {
  float m, s;
  block_lse(y, f, m, s);
  const int64_t plane = (int64_t)(v0 / kInt8BlockV) * a.T;
  const uint32_t bytes = (uint32_t)a.T * 4, at = lg == 0 ? (uint32_t)t * 4 : bytes;
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), row_rsrc(a.part_m + plane, bytes), at,
                                        0, 0);
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), row_rsrc(a.part_s + plane, bytes), at,
                                        0, 0);
}

// Rows behind the vocabulary get weight 0. Where the token's factor is 0 (of a scale of
// 0), it is multiplied in here, which leaves 0, or NaN beside an infinite scale of the
// head, and becomes 1: 0 times the infinity that follows would be NaN too.
__device__ __forceinline__ void mask_tail(const Int8Args& a, float (&y)[kPerLane], float& f, int v0,
                                          int lg) {
  if (v0 + kInt8BlockV <= a.V) return;
  const float g = f == 0.0f ? 0.0f : 1.0f;
  f = f == 0.0f ? 1.0f : f;
  const float none = f < 0.0f ? INFINITY : -INFINITY;
  int left = a.V - v0 - 8 * lg;
  asm volatile("" : "+v"(left));  // (or all tokens' comparisons are made, and kept, at once)
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) y[k] = result_row(0, k) < left ? y[k] * g : none;
}

// A token's scale is left to the end (y = S w_scale, z = y x_scale), which spares
// a product a logit.
__device__ __forceinline__ float score_of(Scores, int sum, float, float ws) {
  return (float)sum * ws;
}
__device__ __forceinline__ float factor_of(Scores, float xs, float scale2) { return xs * scale2; }
__device__ __forceinline__ float score_of(RoundedScores, int sum, float xs, float ws) {
  return (float)(__bf16)logit(sum, xs, ws);
}
__device__ __forceinline__ float factor_of(RoundedScores, float, float scale2) { return scale2; }

template <class Out>
__device__ __forceinline__ void finish_block(Out out, const Int8Args& a, const Place&, int,
                                             const int (&sums)[kPerLane], const RowScales& w,
                                             int v0, int t, float xs, int lg) {
  float f = factor_of(out, xs, a.scale2);
  float y[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) y[k] = score_of(out, sums[k], xs, w.s[k]);
  mask_tail(a, y, f, v0, lg);
  store_partial(a, y, f, v0, t, lg);
}

// The stage that a block of vocabulary rows, or a group of tiles, begins with; it
// goes round from there. Rows of a power of two of bytes lie on the same few
// channels at the same place, and workgroups that start together stay together (one
// row of the 151 936 x 4 096 head 138 us from the first stage on, 114 us from a
// KiB further for each block; rows of 4 224 bytes 115 us either way). The sums are
// integers: their order is free.
constexpr int kRotate = 8;
__device__ __forceinline__ int first_stage(int block, int nk) {
  return (int)((uint32_t)block * (uint32_t)kRotate % (uint32_t)nk);
}

// ---- Streaming kernel ---------------------------------------------------------
// A workgroup takes one block of vocabulary rows and all (16 kNT) tokens; its four
// waves take the K stages in turn (the integer sums may be split anyhow), and
// their sums are joined in LDS, each wave finishing a quarter of the token
// tiles. Fragments go from memory straight into registers. What bounds it is reading W:
// one row over 151 936 x 4 096 takes 108 us, 5.75 TB/s.
constexpr int kStreamWaves = 4;

template <int kNT, class Out>
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(Int8Args a) {
  __shared__ int red[kStreamWaves][kNT][kPerLane][64];
  const int lane = threadIdx.x & 63, lcol = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v0 = blockIdx.x * kInt8BlockV;
  const int nk = (a.H + kInt8StageK - 1) / kInt8StageK;
  // Rows are clamped to the matrices; what they give is not stored. Bytes
  // behind H meet zeros of x.
  const int rows = a.V - v0, tokens = a.T;
  const int64_t w_bytes = (int64_t)(rows - 1) * a.ldw + (a.H + 15) / 16 * 16;
  const int64_t x_bytes = (int64_t)(tokens - 1) * a.ldx + (int64_t)nk * kInt8StageK;
  const __amdgpu_buffer_rsrc_t wres = rsrc_of(a.w + (int64_t)v0 * a.ldw, w_bytes);
  const __amdgpu_buffer_rsrc_t xres = rsrc_of(a.x, x_bytes);
  uint32_t woff[kTiles], xoff[kNT];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    woff[i] = (uint32_t)min(fragment_row(lane, i), rows - 1) * (uint32_t)a.ldw + 16 * lg;
#pragma unroll
  for (int j = 0; j < kNT; ++j)
    xoff[j] = (uint32_t)min(16 * j + lcol, tokens - 1) * (uint32_t)a.ldx + 16 * lg;
  auto load = [](__amdgpu_buffer_rsrc_t r, uint32_t off, int k) __attribute__((always_inline)) {
    return __builtin_bit_cast(i32x4,
                              __builtin_amdgcn_raw_buffer_load_b128(r, off, k * kInt8StageK, 0));
  };
  i32x4 acc[kNT][kTiles];
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  // Two stages in registers: one in flight while the other is multiplied. Behind
  // the wave's last stage that one is read again, so that every turn issues the
  // same loads.
  struct Stage {
    i32x4 w[kTiles][2], x[kNT][2];
  };
  const int mine = (nk - wave + kStreamWaves - 1) / kStreamWaves;  // 0: none
  const int first = first_stage(blockIdx.x, nk);
  auto issue = [&](Stage& s, int i) __attribute__((always_inline)) {
    int k = min(wave + kStreamWaves * i, nk - 1) + first;
    k -= k >= nk ? nk : 0;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) s.w[i][c] = load(wres, woff[i] + 64 * c, k);
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) s.x[j][c] = load(xres, xoff[j] + 64 * c, k);
    __builtin_amdgcn_sched_barrier(0);  // (left alone, loads sink down to their first use)
  };
  auto multiply = [&](const Stage& s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[j][i] = mma(s.w[i][c], s.x[j][c], acc[j][i]);
    __builtin_amdgcn_sched_barrier(0);
  };
  Stage even, odd;
  issue(even, 0);
  int i = 0;
  for (; i + 2 <= mine; i += 2) {
    issue(odd, i + 1);
    multiply(even);
    issue(even, i + 2);
    multiply(odd);
  }
  if (i < mine) multiply(even);
  const RowScales scales = row_scales(a, v0, lg);
  const Place place = place_of(Out(), a, v0, 0, 16 * kNT, lane);
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) red[wave][j][k][lane] = acc[j][k / 4][k % 4];
  __syncthreads();
  for (int j = wave; j < kNT; j += kStreamWaves) {
    int sums[kPerLane];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      sums[k] = 0;
#pragma unroll
      for (int w = 0; w < kStreamWaves; ++w) sums[k] += red[w][j][k][lane];
    }
    const int t = 16 * j + lcol;
    finish_block(Out(), a, place, j, sums, scales, v0, t, read_global(a.x_scale, min(t, a.T - 1)),
                 lg);
  }
}

// ---- Tile kernel --------------------------------------------------------------
// Four waves compute 256 vocabulary rows x 32 kJ tokens, 128 x 16 kJ each: with
// kJ = 8, 256 accumulators in the AGPRs. K stages of 128 bytes go from memory
// straight into LDS buffers in turn: three of up to 52 KiB up to kJ = 5, so that a
// stage's copies have a whole stage to land in (heads of 151 936 x 4 096, two buffers
// and three: 320 rows 243 and 219 us, 128 rows 156 and 144, 64 rows 137 and 131), else
// two of up to 64 KiB. The 16-byte chunks of a row are
// permuted (swz_w, swz_x) so that the fragment reads meet no bank conflicts. One
// barrier a stage: the MFMAs of a stage's second half are carried across it, and
// the copies are spread over the whole stage (1 024 rows with one each 6 MFMAs 573 us,
// each 3 606, each 2 635). A workgroup stays on
// its CU and takes tile after tile: during a tile's last stages the next one's
// first are copied, so that the sums' scales, roundings and stores (15 % of a tile
// of 4 096 hidden elements) are all that the MFMAs wait for. Scores of 8 192 rows over
// 151 936 x 4 096 take 3.7 ms: 2.7 POP/s, the matrix units busy for 69 % of the time at
// the 1.9 GHz that the power limit leaves; logits of 320 rows 201 to 208 us (1.9 POP/s), where
// issuing the copies and waiting for a tile's ends weigh more.
constexpr int kTileRows = 256;                      // of W
constexpr int kTileThreads = 256;
constexpr int kUnitB = kTileRows * kInt8StageK;     // 32 KiB of W
constexpr int kUnitCopies = kUnitB / 1024 / 4;      // 1-KiB copies per wave (8)
constexpr int kGroupV = 4;                          // vocabulary tiles per scheduling group
constexpr int kCus = 256;

// Physical chunk of logical chunk c in LDS row `row`; its own inverse. A wave's
// read takes the chunks 4 h + (l >> 4) of sixteen rows: of X consecutive ones, of
// W those of fragment_row, 8 a + b from some multiple of 4 on, a, b < 4.
__device__ __forceinline__ int swz_x(int row, int c) { return c ^ (row & 7); }
__device__ __forceinline__ int swz_w(int row, int c) {
  return c ^ ((row & 3) | ((row >> 1) & 4));
}

// Where a tile lies: its operands' first bytes, and how many there are from there.
struct TileAt {
  const int8_t *w, *x;
  uint32_t w_bytes, x_bytes;
  int v0, t0, first;
};
template <int kTokens>
__device__ __forceinline__ TileAt tile_at(const Int8Args& a, int tile, int n_vt, int n_tt, int nk) {
  int vt, tt;
  tile_of(tile, n_vt, n_tt, kGroupV, vt, tt);
  TileAt t;
  t.v0 = __builtin_amdgcn_readfirstlane(vt) * kTileRows;
  t.t0 = __builtin_amdgcn_readfirstlane(tt) * kTokens;
  t.first = first_stage(t.v0 / (kTileRows * kGroupV), nk);
  t.w = a.w + (int64_t)t.v0 * a.ldw;
  t.x = a.x + (int64_t)t.t0 * a.ldx;
  t.w_bytes = span_bytes((uint64_t)((int64_t)(a.V - t.v0 - 1) * a.ldw + (a.H + 15) / 16 * 16));
  t.x_bytes =
      span_bytes((uint64_t)((int64_t)(a.T - t.t0 - 1) * a.ldx + (int64_t)nk * kInt8StageK));
  return t;
}

template <int kJ, class Out>
__global__ __launch_bounds__(kTileThreads, 1) void tile_kernel(Int8Args a, int n_vt,
                                                                            int n_tt) {
  constexpr int kTokens = 32 * kJ, kCopies = kUnitCopies + kJ;
  constexpr int kBufferB = kUnitB + kTokens * kInt8StageK;
  constexpr int kHalf = kTiles * kJ;                        // MFMAs of a step
  constexpr int kSlotsPerCopy = (2 * kHalf - 2) / kCopies;  // from one copy to the next
  constexpr int kEvery = kSlotsPerCopy < 6 ? kSlotsPerCopy : 6;
  constexpr int kPerGroup = (kJ + 3) / 4;                   // X reads of a group
  constexpr int kBuffers = kJ <= 5 ? 3 : 2, kAhead = kBuffers - 1;
  constexpr int kInFlight = (kAhead - 1) * kCopies;  // copies of the stages after the next
  static_assert(kInFlight < 64, "a counter's width");
  __shared__ __attribute__((aligned(1024))) char ring[kBuffers * kBufferB];
  const int lane = threadIdx.x & 63, lcol = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int nk = (a.H + kInt8StageK - 1) / kInt8StageK;
  const int n_tiles = n_vt * n_tt;

  // Copy j of a unit: wave w fills rows 8 (4 j + w) .. + 7, lane l the physical
  // chunk l & 7 of row l >> 3 of them. Rows behind the matrices read as zeros
  // (the resources end there) and their results are not stored.
  const uint32_t ldw = (uint32_t)a.ldw, ldx = (uint32_t)a.ldx;
  const int row = 8 * wave + (lane >> 3);
  const uint32_t offW = (uint32_t)row * ldw + 16 * swz_w(row, lane & 7);
  const uint32_t offX = (uint32_t)row * ldx + 16 * swz_x(row, lane & 7);
  const uint32_t lds0 =
      __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_char*)ring));
  const uint32_t stepW = 32 * ldw, stepX = 32 * ldx;
  uint32_t voff = offW;
// Copy c (in order, W's first) of the stage at byte off_ of a row into buffer b.
// The offset of the rows goes from copy to copy (one register, by an add that the
// compiler cannot turn into one for each).
#define COPY(c_, wres_, xres_, off_, b_)                                                      \
  do {                                                                                        \
    const bool w_ = (c_) < kUnitCopies;                                                       \
    const uint32_t j_ = (uint32_t)(w_ ? (c_) : (c_) - kUnitCopies);                           \
    if (j_ == 0) voff = w_ ? offW : offX;                                                     \
    else asm volatile("v_add_u32 %0, %1, %0" : "+v"(voff) : "s"(w_ ? stepW : stepX));         \
    copy_lds(w_ ? (wres_) : (xres_),                                                          \
             lds0 + (uint32_t)(b_) * kBufferB + (w_ ? 0u : (uint32_t)kUnitB) + (4 * j_ + wave) * 1024, \
             voff, (off_));                                                                   \
  } while (0)

  // Fragment reads of half h (64 codes) of a stage.
  uint32_t rdW[2], rdX[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int wr = wm * kInt8BlockV + fragment_row(lane, 0), xr = wn * 16 * kJ + lcol;
    // Tile i adds 32 (i / 2) + 4 (i % 2) rows, none of the bits that swz_w sees.
    rdW[h] = (uint32_t)(wr * kInt8StageK + 16 * swz_w(wr, 4 * h + lg));
    rdX[h] = (uint32_t)(kUnitB + xr * kInt8StageK + 16 * swz_x(xr, 4 * h + lg));
  }
#define RD_W(i_, h_, b_)                                                                  \
  *reinterpret_cast<const i32x4*>(ring + (rdW[(h_)] + (uint32_t)(b_) * kBufferB) +        \
                                  (32 * ((i_) >> 1) + 4 * ((i_) & 1)) * kInt8StageK)
#define RD_X(j_, h_, b_) \
  *reinterpret_cast<const i32x4*>(ring + (rdX[(h_)] + (uint32_t)(b_) * kBufferB) + (j_) * 16 * kInt8StageK)
#define FENCE() __builtin_amdgcn_sched_barrier(0)

  // One step: eight groups (W tile g with all X tiles) on fw and mx_, 64 codes
  // (z_: from zero sums), while the next step's fragments are read from half rh_
  // of buffer rb_: X tiles into nx_ during groups 0 .. 3, W tile g into fw[g]
  // behind group g, its last use. A stage (two steps, slots from p0_ on) issues the
  // copies of the stage that follows. The order is fixed.
  i32x4 acc[kTiles][kJ];  // [W tile][X tile]
  i32x4 fw[kTiles], fx0[kJ], fx1[kJ];
#define STEP(do_mma_, z_, do_rd_, mx_, nx_, rh_, rb_, p0_)                                    \
  do {                                                                                        \
    _Pragma("unroll") for (int u = 0; u < kHalf; ++u) {                                       \
      const int g_ = u / kJ, j_ = u % kJ;                                                     \
      if (do_mma_)                                                                            \
        acc[g_][j_] = mma(fw[g_], mx_[j_], (z_) ? i32x4{0, 0, 0, 0} : acc[g_][j_]);           \
      if ((do_rd_) && j_ == kJ / 4 && kPerGroup * g_ < kJ) {                                  \
        const int x_ = kPerGroup * g_ < kJ ? kPerGroup * g_ : 0;                              \
        nx_[x_] = RD_X(x_, (rh_), (rb_));                                                     \
      }                                                                                       \
      if ((do_rd_) && kPerGroup == 2 && j_ == kJ / 4 + 3 && 2 * g_ + 1 < kJ) {                \
        const int x_ = 2 * g_ + 1 < kJ ? 2 * g_ + 1 : 0;                                      \
        nx_[x_] = RD_X(x_, (rh_), (rb_));                                                     \
      }                                                                                       \
      if ((do_rd_) && j_ == kJ - 1) fw[g_] = RD_W(g_, (rh_), (rb_));                          \
      const int pu_ = (p0_) + u;                                                              \
      if (pu_ % kEvery == 1 && pu_ / kEvery < kCopies)                                        \
        COPY(pu_ / kEvery, wres, xres, off, b == 0 ? kAhead : b - 1);                         \
      FENCE();                                                                                \
    }                                                                                         \
  } while (0)
// The beginning of a stage: it has landed, and every wave is done with the buffer
// that the one kAhead stages on goes into. That is the same tile's, or a following
// one's (behind the last tile the first once more, which nothing reads).
#define STAGE()                                                                               \
  __builtin_amdgcn_s_waitcnt(0x0070 | (kInFlight & 15) | (kInFlight >> 4) << 14);             \
  asm volatile("" ::: "memory");                                                              \
  FENCE();                                                                                    \
  __builtin_amdgcn_s_barrier();                                                               \
  asm volatile("" ::: "memory");                                                              \
  FENCE();                                                                                    \
  const int k_ = ahead + at.first;                                                            \
  const uint32_t off = (uint32_t)(k_ >= nk ? k_ - nk : k_) * kInt8StageK;                     \
  const __amdgpu_buffer_rsrc_t wres = make_rsrc(at.w, at.w_bytes);                            \
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(at.x, at.x_bytes);                            \
  NEXT();                                                                                     \
  FENCE()
#define NEXT()                                                                                \
  if (++ahead == nk) {                                                                        \
    ahead = 0;                                                                                \
    after += (int)gridDim.x;                                                                  \
    at = tile_at<kTokens>(a, after < n_tiles ? after : (int)blockIdx.x, n_vt, n_tt, nk);      \
  }

  // The stage that is copied next, and its tile.
  TileAt at = tile_at<kTokens>(a, blockIdx.x, n_vt, n_tt, nk);
  int ahead = 0, after = blockIdx.x;
  int b = 0;
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
    const int k_ = ahead + at.first;
    const uint32_t off = (uint32_t)(k_ >= nk ? k_ - nk : k_) * kInt8StageK;
    const __amdgpu_buffer_rsrc_t wres = make_rsrc(at.w, at.w_bytes);
    const __amdgpu_buffer_rsrc_t xres = make_rsrc(at.x, at.x_bytes);
    FENCE();
#pragma unroll
    for (int c = 0; c < kCopies; ++c) COPY(c, wres, xres, off, s);
    NEXT();
  }
  for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
    int vt, tt;
    tile_of(tile, n_vt, n_tt, kGroupV, vt, tt);
    const int v0 = __builtin_amdgcn_readfirstlane(vt) * kTileRows;
    const int t0 = __builtin_amdgcn_readfirstlane(tt) * kTokens;
    {
      STAGE();
      STEP(false, false, true, fx1, fx0, 0, b, 0);
      STEP(true, true, true, fx0, fx1, 1, b, kHalf);
    }
    for (int k = 1; k < nk; ++k) {
      b = b == kAhead ? 0 : b + 1;
      STAGE();
      STEP(true, false, true, fx1, fx0, 0, b, 0);
      STEP(true, false, true, fx0, fx1, 1, b, kHalf);
    }
    // The epilogue's scales, in flight over the last step. What follows from the
    // lane is formed anew, and a token's part is kept apart from the next one's:
    // next to the accumulators there are no registers for all of it at once.
    const int vb = v0 + wm * kInt8BlockV;
    int lane_e;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane_e));
    const int lg_e = lane_e >> 4, t_e = t0 + wn * 16 * kJ + (lane_e & 15);
    const bool there = vb < a.V;
    RowScales scales = {};
    float xs[kJ];
    if (there) scales = row_scales(a, vb, lg_e);
#pragma unroll
    for (int j = 0; j < kJ; ++j) xs[j] = read_global(a.x_scale, min(t_e + 16 * j, a.T - 1));
    {
      // (Slots behind a stage's copies.)
      const __amdgpu_buffer_rsrc_t wres = make_rsrc(at.w, at.w_bytes), xres = wres;
      const uint32_t off = 0;
      STEP(true, false, false, fx1, fx0, 0, b, 4 * kHalf);
    }
    b = b == kAhead ? 0 : b + 1;
    if (there) {
      const Place place = place_of(Out(), a, vb, t0 + wn * 16 * kJ, 16 * kJ, lane_e);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        int t = t_e + 16 * j;
        asm volatile("" : "+v"(t));
        int sums[kPerLane];
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) sums[k] = acc[k >> 2][j][k & 3];
        finish_block(Out(), a, place, j, sums, scales, vb, t, xs[j], lg_e);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // the last copies land before the LDS is given back
#undef STAGE
#undef NEXT
#undef STEP
#undef COPY
#undef RD_W
#undef RD_X
#undef FENCE
}

// ---- Merge ------------------------------------------------------------------
// A workgroup joins 16 tokens' partials: the blocks are cut into 64 segments, whose
// bounds depend on the vocabulary alone, four for each of 16 waves (lane l: token
// l & 15, segment 4 wave + (l >> 4)). A segment is folded in ascending order, with
// the loads of eight blocks in flight at a time, then a wave's four, then the waves.
constexpr int kMergeTokens = 16;
constexpr int kMergeWaves = 16;
constexpr int kSegments = 4 * kMergeWaves;
constexpr int kMergeLoads = 8;

// The target's logit is formed here, once more: its sum is exact, so it has the
// bits that it has in its block.
__device__ __forceinline__ int row_sum(const Int8Args& a, int64_t t, int64_t id) {
  const Global<const Words> x = (Global<const Words>)(const Words*)(a.x + t * a.ldx);
  const Global<const Words> w = (Global<const Words>)(const Words*)(a.w + id * a.ldw);
  int s = 0;
  for (int i = threadIdx.x & 63; i < (a.H + 15) / 16; i += 64) {
    const Words p = x[i], q = w[i];
    s = __builtin_amdgcn_sdot4((int)p.x, (int)q.x, s, false);
    s = __builtin_amdgcn_sdot4((int)p.y, (int)q.y, s, false);
    s = __builtin_amdgcn_sdot4((int)p.z, (int)q.z, s, false);
    s = __builtin_amdgcn_sdot4((int)p.w, (int)q.w, s, false);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

template <class Out>
__global__ __launch_bounds__(64 * kMergeWaves) void merge_kernel(Int8Args a) {
  __shared__ float wave_m[kMergeWaves][kMergeTokens], wave_s[kMergeWaves][kMergeTokens];
  __shared__ double target[kMergeTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kMergeTokens, t = t0 + (lane & 15);
  static_assert(kMergeTokens == kMergeWaves, "a target for each wave");
  const int64_t mine = t0 + wave;
  if (mine < a.T) {
    const int64_t id = a.ids[mine];
    if (id >= 0 && id < a.V) {
      const float xs = a.x_scale[mine];
      const float z = score_of(Out(), row_sum(a, mine, id), xs, a.w_scale[id]);
      if (lane == 0) target[wave] = (double)z * (double)factor_of(Out(), xs, a.scale2);
    }
  }
  const int blocks = (a.V + kInt8BlockV - 1) / kInt8BlockV;
  const int per = (blocks + kSegments - 1) / kSegments;
  const int lo = min(blocks, (4 * wave + (lane >> 4)) * per), hi = min(blocks, lo + per);
  const int64_t at = min(t, (int64_t)a.T - 1);
  float M = -INFINITY, S = 0.0f;
  for (int b = 0; b < per; b += kMergeLoads) {
    float m[kMergeLoads], s[kMergeLoads];
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) {
      const bool there = lo + b + i < hi;
      const int64_t o = (int64_t)min(lo + b + i, blocks - 1) * a.T + at;
      m[i] = read_global(a.part_m, o);
      s[i] = read_global(a.part_s, o);
      m[i] = there ? m[i] : -INFINITY;
      s[i] = there ? s[i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) lse_fold(M, S, m[i], s[i]);
  }
  // (Either lane of a pair adds the same two products, in its own order.)
  auto pair = [&](float m, float s) __attribute__((always_inline)) {
    const float Mn = fmaxf(M, m), base = Mn == -INFINITY ? 0.0f : Mn;
    const float p = S * fast_exp2(M - base), q = s * fast_exp2(m - base);
    S = p + q;
    M = Mn;
  };
  pair(xor_lane<16>(M), xor_lane<16>(S));
  pair(xor_lane<32>(M), xor_lane<32>(S));
  if (lane < kMergeTokens) {
    wave_m[wave][lane] = M;
    wave_s[wave][lane] = S;
  }
  __syncthreads();
  if (threadIdx.x >= kMergeTokens || t >= a.T) return;
#pragma unroll
  for (int g = 1; g < kMergeWaves; ++g) lse_fold(M, S, wave_m[g][lane], wave_s[g][lane]);
  const int64_t id = a.ids[t];
  const bool ok = id >= 0 && id < a.V;
  // The maximum is a rounded product, the blocks' terms are of the exact one: a token that
  // holds all the weight has S next to 2^(target - M), and no score of its own but
  // what cancels here. (In fp32 its score was off by 2^-24 of its logit, of either sign.)
  const double lse2 = (double)M + log2((double)S), score = (target[lane] - lse2) * kLn2;
  a.out_lp[t] = ok ? (float)(score > 0.0 ? 0.0 : score) : NAN;
  if (a.out_lse) a.out_lse[t] = (float)(lse2 * kLn2);
  if (!ok && a.bad_rows) atomicAdd(a.bad_rows, 1);
}

// ---- Hidden states in whole stages ------------------------------------------

__global__ __launch_bounds__(256) void stage_kernel(Int8Args a, int64_t row) {
  const int64_t words = row / 4, n = (int64_t)a.T * words;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / words, k = (i - t * words) * 4;
    const int8_t* p = a.x + t * a.ldx + k;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e < a.H) w |= (uint32_t)(uint8_t)p[e] << (8 * e);
    reinterpret_cast<uint32_t*>(a.staged)[i] = w;
  }
}

// launch(Out()) for what the call wants.
template <class F>
void with_output(const Int8Args& a, F launch) {
  if (!a.out) {
    if (a.bf16_logits) launch(RoundedScores());
    else launch(Scores());
  } else if (a.dtype == LP_F32) {
    launch(Logits<F32>());
  } else if (a.dtype == LP_BF16) {
    launch(Logits<BF16>());
  } else {
    launch(Logits<F16>());
  }
}

template <int kNT>
void stream(const Int8Args& a, hipStream_t s) {
  const dim3 grid((uint32_t)((a.V + kInt8BlockV - 1) / kInt8BlockV));
  with_output(a, [&](auto out) {
    stream_kernel<kNT, decltype(out)><<<grid, 64 * kStreamWaves, 0, s>>>(a);
  });
}

template <int kJ>
void tiles(const Int8Args& a, hipStream_t s) {
  const int n_vt = (a.V + kTileRows - 1) / kTileRows, n_tt = (a.T + 32 * kJ - 1) / (32 * kJ);
  const dim3 grid((uint32_t)std::min<int64_t>((int64_t)n_vt * n_tt, kCus));
  with_output(a, [&](auto out) {
    tile_kernel<kJ, decltype(out)><<<grid, kTileThreads, 0, s>>>(a, n_vt, n_tt);
  });
}

}  // namespace

Int8Workspace int8_workspace_layout(int64_t T, int64_t H, int64_t V) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t plane = (size_t)((V + kInt8BlockV - 1) / kInt8BlockV) * (size_t)T * sizeof(float);
  Int8Workspace w;
  w.off_staged = 0;
  w.off_m = up((size_t)T * (size_t)int8_staged_row(H));
  w.off_s = w.off_m + up(plane);
  w.total = V > 0 ? w.off_s + up(plane) : w.off_m;
  return w;
}

bool int8_grid_ok(int64_t T, int64_t V) {
  // Streams have a workgroup a block, and the tile kernel counts its tiles, and the
  // grid's stride past them, in 32 bits: ceil(T / 256) tiles along the tokens, or more
  // of them where there are fewer than kCus in all.
  const int64_t blocks = (V + kInt8BlockV - 1) / kInt8BlockV;
  const int64_t tiles = (V + kTileRows - 1) / kTileRows * ((T + 255) / 256);
  return T <= kInt8TokensMax && blocks <= kMaxDispatchItems / (64 * kStreamWaves) &&
         tiles <= INT32_MAX - 2 * kCus &&
         (T + kMergeTokens - 1) / kMergeTokens <= kMaxDispatchItems / (64 * kMergeWaves);
}

hipError_t launch_int8(Int8Args a, hipStream_t stream_) {
  hipError_t e;
  if (!int8_reads_in_place(a.x, a.ldx, a.H)) {
    const int64_t row = int8_staged_row(a.H), words = a.T * (row / 4);
    const uint32_t grid = (uint32_t)std::min<int64_t>((words + 255) / 256, 65536);
    stage_kernel<<<grid, 256, 0, stream_>>>(a, row);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    a.x = a.staged;
    a.ldx = row;
  }
  // Tiles are as few as tokens by 256 make them, and narrower where they would leave
  // CUs idle; and as narrow as their number leaves them. (200 rows over 32 003, H =
  // 4 096, by two tiles of 100 42 us, by one 61; 256 over 16 000 by four 23, by one
  // 44; but 320 over 151 936 by two of 160 210, by three of 107 248.)
  const int64_t n_vt = (a.V + kTileRows - 1) / kTileRows;
  const int64_t n_tt =
      std::max<int64_t>((a.T + 255) / 256, std::min<int64_t>(kCus / n_vt, (a.T + 63) / 64));
  const int64_t width = ((a.T + n_tt - 1) / n_tt + 31) / 32;  // of a tile, by 32 tokens
  // Few tokens by streams, which put twice the workgroups on the rows of W, where
  // there is enough of it for each: up to 16, and up to 32 where all of them run at
  // once. Streams and tiles, H = 4 096: one row over 151 936 108 and 121 us, over
  // 32 003 32 and 38, over 8 000 20 and 18; 32 rows over 151 936 133 and 125, over
  // 32 003 31 and 34, over 8 000 23 and 18; 64 rows over 32 003 36 and 36. H = 1 024,
  // over 50 021: 16 and 12, 20 and 13.
  const int64_t blocks = (a.V + kInt8BlockV - 1) / kInt8BlockV;
  const bool streams = a.H > 15 * kInt8StageK && blocks > kCus / 4;
  if (streams && a.T <= 16) stream<1>(a, stream_);
  else if (streams && a.T <= 32 && blocks <= kCus) stream<2>(a, stream_);
  else if (width <= 2) tiles<2>(a, stream_);
  else if (width <= 4) tiles<4>(a, stream_);
  else if (width <= 5) tiles<5>(a, stream_);
  else if (width <= 6) tiles<6>(a, stream_);
  else tiles<8>(a, stream_);
  if ((e = hipGetLastError()) != hipSuccess || a.out) return e;
  const dim3 grid((uint32_t)((a.T + kMergeTokens - 1) / kMergeTokens));
  if (a.bf16_logits) merge_kernel<RoundedScores><<<grid, 64 * kMergeWaves, 0, stream_>>>(a);
  else merge_kernel<Scores><<<grid, 64 * kMergeWaves, 0, stream_>>>(a);
  return hipGetLastError();
}

}  // namespace lp
