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
// tiles, whose row m of tile i is vocabulary row 32 (m / 4) + 4 i + m % 4. An
// MFMA's result has the token l & 15 and the rows 4 (l >> 4) + r, r < 4, in
// lane l; so lane l holds the 32 vocabulary rows from 32 (l >> 4) on, one after
// the other: logits are stored in whole 16-byte words, and the reduction over
// the vocabulary is mostly inside a lane.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "int8_internal.h"
#include "tile_common.h"

namespace lp {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTiles = 8;            // MFMA tiles of a block along the vocabulary
constexpr int kPerLane = 4 * kTiles; // vocabulary rows of a lane
constexpr float kLn2 = 0.693147180559945309f;
static_assert(kInt8BlockV == 16 * kTiles, "a block is one wave's");

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

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
  return 32 * ((lane & 15) >> 2) + 4 * i + (lane & 3);
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

// Maximum and sum of exp2(z scale2 - maximum) of a block for the lane's token,
// z(k) its logit of the lane's k-th row (-inf behind the vocabulary): over the
// lane's rows in ascending order, then the lanes l ^ 16 and l ^ 32, which end
// with the same bits. A NaN or +inf logit makes the sum NaN.
template <class Z>
__device__ __forceinline__ void block_lse(Z z, float scale2, float& m_out, float& s_out) {
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) m = fmaxf(m, z(k));
  m = fmaxf(m, xor_lane<16>(m));
  m = fmaxf(m, xor_lane<32>(m));
  const float m2 = m * scale2, base = m == -INFINITY ? 0.0f : m2;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) s += fast_exp2(__builtin_fmaf(z(k), scale2, -base));
  s += xor_lane<16>(s);
  s += xor_lane<32>(s);
  m_out = m2;
  s_out = s;
}

// Joins (m, s) to (M, S). Nothing (-inf, 0) joins without a trace; a NaN stays.
__device__ __forceinline__ void lse_fold(float& M, float& S, float m, float s) {
  const float Mn = fmaxf(M, m), base = Mn == -INFINITY ? 0.0f : Mn;
  S = __builtin_fmaf(s, fast_exp2(m - base), S * fast_exp2(M - base));
  M = Mn;
}

// ---- What a wave does with a block's sums -----------------------------------

// acc[i][r]: the sum of the lane's token and vocabulary row v0 + 32 lg + 4 i + r
// of the block that starts at v0.
template <class D>
__device__ __forceinline__ void store_logits(const Int8Args& a, const i32x4 (&acc)[kTiles], int v0,
                                             int t, int lg) {
  if (t >= a.T) return;
  const int v = v0 + 32 * lg;
  const float xs = a.x_scale[t];
  typename D::Raw* p = static_cast<typename D::Raw*>(a.out) + (int64_t)t * a.ld_out;
#pragma unroll
  for (int k0 = 0; k0 < kPerLane; k0 += D::kVec) {
    if (v + k0 >= a.V) break;
    Group<D> g = {};
#pragma unroll
    for (int e = 0; e < D::kVec; ++e) {
      const int k = k0 + e;
      const float ws = read_global(a.w_scale, min(v + k, a.V - 1));
      g.set(e, D::round(logit(acc[k / 4][k % 4], xs, ws)));
    }
    store_group<D>(p, v + k0, a.V, g);
  }
}

__device__ __forceinline__ float rounded(float z, bool bf16) {
  return bf16 ? (float)(__bf16)z : z;
}

__device__ __forceinline__ void store_partial(const Int8Args& a, const i32x4 (&acc)[kTiles], int v0,
                                              int t, int lg) {
  const int v = v0 + 32 * lg;
  const float xs = a.x_scale[min(t, a.T - 1)];
  auto z = [&](int k) __attribute__((always_inline)) {
    const float ws = read_global(a.w_scale, min(v + k, a.V - 1));
    const float x = rounded(logit(acc[k / 4][k % 4], xs, ws), a.bf16_logits);
    return v + k < a.V ? x : -INFINITY;
  };
  float m, s;
  block_lse(z, a.scale2, m, s);
  if (t >= a.T) return;
  const int64_t at = a.ids[t] - v;
  if (at >= 0 && at < kPerLane && v + at < a.V) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) x = k == (int)at ? z(k) : x;
    a.tval[t] = x * a.scale2;
  }
  if (lg == 0) {
    const int64_t o = (int64_t)(v0 / kInt8BlockV) * a.T + t;
    a.part_m[o] = m;
    a.part_s[o] = s;
  }
}

// ---- Streaming kernel ---------------------------------------------------------
// A workgroup takes one block of vocabulary rows and 16 kNT tokens; its four
// waves take the K stages in turn (the integer sums may be split anyhow), and
// their sums are joined in LDS, each wave finishing a quarter of the token
// tiles. Fragments go from memory straight into registers.
constexpr int kStreamWaves = 4;

template <int kNT, class D>  // D: the logits' type, or void for scores
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(Int8Args a) {
  __shared__ int red[kStreamWaves][kNT][kPerLane][64];
  const int lane = threadIdx.x & 63, lcol = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v0 = blockIdx.x * kInt8BlockV, t0 = blockIdx.y * 16 * kNT;
  const int nk = (a.H + kInt8StageK - 1) / kInt8StageK;
  // Rows are clamped to the matrices; what they give is not stored. Bytes
  // behind H meet zeros of x.
  const int rows = a.V - v0, tokens = a.T - t0;
  const int64_t w_bytes = (int64_t)(rows - 1) * a.ldw + (a.H + 15) / 16 * 16;
  const int64_t x_bytes = (int64_t)(tokens - 1) * a.ldx + (int64_t)nk * kInt8StageK;
  const __amdgpu_buffer_rsrc_t wres = rsrc_of(a.w + (int64_t)v0 * a.ldw, w_bytes);
  const __amdgpu_buffer_rsrc_t xres = rsrc_of(a.x + (int64_t)t0 * a.ldx, x_bytes);
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
  auto issue = [&](Stage& s, int i) __attribute__((always_inline)) {
    const int k = min(wave + kStreamWaves * i, nk - 1);
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
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) red[wave][j][k][lane] = acc[j][k / 4][k % 4];
  __syncthreads();
  for (int j = wave; j < kNT; j += kStreamWaves) {
    i32x4 sum[kTiles];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < kStreamWaves; ++w) s += red[w][j][k][lane];
      sum[k / 4][k % 4] = s;
    }
    const int t = t0 + 16 * j + lcol;
    if constexpr (std::is_void_v<D>) store_partial(a, sum, v0, t, lg);
    else store_logits<D>(a, sum, v0, t, lg);
  }
}

// ---- Tile kernel --------------------------------------------------------------
// Four waves compute 256 vocabulary rows x 256 tokens, 128 x 128 each: 256
// accumulators in the AGPRs. K stages of 128 bytes go from memory straight into
// two alternating LDS buffers of 64 KiB; the 16-byte chunks of a row are
// permuted (swz_w, swz_x) so that the fragment reads meet no bank conflicts. One
// barrier a stage: the MFMAs of a stage's second half are carried across it, and
// the next stage's copies are spread over the whole stage.
constexpr int kTileRows = 256;                  // of W, and tokens
constexpr int kTileThreads = 256;
constexpr int kUnitB = kTileRows * kInt8StageK; // 32 KiB of either operand
constexpr int kBufferB = 2 * kUnitB;
constexpr int kUnitCopies = kUnitB / 1024 / 4;  // 1-KiB copies per wave (8)
constexpr int kGroupV = 4;                      // vocabulary tiles per scheduling group
constexpr int kSlotsPerCopy = 6;                // MFMAs from one copy to the next
static_assert(kSlotsPerCopy * 2 * kUnitCopies < 2 * kTiles * kTiles, "copies fit in a stage");

// Physical chunk of logical chunk c in LDS row `row`; its own inverse. A wave's
// read takes the chunks 4 h + (l >> 4) of sixteen rows: of X consecutive ones, of
// W those of fragment_row, 32 a + 4 i + b with a, b < 4.
__device__ __forceinline__ int swz_x(int row, int c) { return c ^ (row & 7); }
__device__ __forceinline__ int swz_w(int row, int c) {
  return c ^ ((row & 3) | ((row >> 3) & 4));
}

template <class D>  // the logits' type, or void for scores
__global__ __launch_bounds__(kTileThreads, 1) void tile_kernel(Int8Args a, int n_vt, int n_tt) {
  __shared__ __attribute__((aligned(1024))) char ring[2 * kBufferB];
  int vt, tt;
  tile_of(blockIdx.x, n_vt, n_tt, kGroupV, vt, tt);
  vt = __builtin_amdgcn_readfirstlane(vt);
  tt = __builtin_amdgcn_readfirstlane(tt);
  const int v0 = vt * kTileRows, t0 = tt * kTileRows;
  const int lane = threadIdx.x & 63, lcol = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;

  // Copy j of a unit: wave w fills rows 8 (4 j + w) .. + 7, lane l the physical
  // chunk l & 7 of row l >> 3 of them. Bit 5 of a row is j's lowest bit, so odd
  // copies of W take the other half of a row. Rows behind the matrices read as
  // zeros (the resources end there) and their results are not stored.
  const int nk = (a.H + kInt8StageK - 1) / kInt8StageK;
  const int64_t w_bytes = (int64_t)(a.V - v0 - 1) * a.ldw + (a.H + 15) / 16 * 16;
  const int64_t x_bytes = (int64_t)(a.T - t0 - 1) * a.ldx + (int64_t)nk * kInt8StageK;
  const __amdgpu_buffer_rsrc_t wres = rsrc_of(a.w + (int64_t)v0 * a.ldw, w_bytes);
  const __amdgpu_buffer_rsrc_t xres = rsrc_of(a.x + (int64_t)t0 * a.ldx, x_bytes);
  const uint32_t ldw = (uint32_t)a.ldw, ldx = (uint32_t)a.ldx;
  const uint32_t row = (uint32_t)(8 * wave + (lane >> 3));
  const uint32_t offW0 = row * ldw + 16 * swz_w(lane >> 3, lane & 7);
  const uint32_t offW1 = row * ldw + 16 * (swz_w(lane >> 3, lane & 7) ^ 4);
  const uint32_t offX = row * ldx + 16 * swz_x(lane >> 3, lane & 7);
  const uint32_t lds0 =
      __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_char*)ring));
// Copy c (0 .. 15, W's first) of stage k into buffer b. A stage behind the last
// one copies that again, into the buffer that nothing reads any more.
#define COPY(c_, k_, b_)                                                                      \
  do {                                                                                        \
    const bool w_ = (c_) < kUnitCopies;                                                       \
    const uint32_t j_ = (uint32_t)((c_) & (kUnitCopies - 1));                                 \
    uint32_t voff_;                                                                           \
    asm volatile("v_add_u32 %0, %1, %2"                                                       \
                 : "=v"(voff_)                                                                \
                 : "s"(j_ * 32 * (w_ ? ldw : ldx)), "v"(w_ ? ((j_ & 1) ? offW1 : offW0) : offX)); \
    copy_lds(w_ ? wres : xres,                                                                \
             lds0 + (uint32_t)(b_) * kBufferB + (w_ ? 0u : (uint32_t)kUnitB) + (4 * j_ + wave) * 1024, \
             voff_, (uint32_t)min((k_), nk - 1) * kInt8StageK);                                \
  } while (0)

  // Fragment reads of half h (64 codes) of a stage.
  uint32_t rdW[2], rdX[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int wr = wm * kInt8BlockV + fragment_row(lane, 0), xr = wn * 128 + lcol;
    // Tile i adds 4 i rows, which swz_w sees in none of its bits.
    rdW[h] = (uint32_t)(wr * kInt8StageK + 16 * swz_w(wr, 4 * h + lg));
    rdX[h] = (uint32_t)(kUnitB + xr * kInt8StageK + 16 * swz_x(xr, 4 * h + lg));
  }
#define RD_W(i_, h_, b_) \
  *reinterpret_cast<const i32x4*>(ring + (rdW[(h_)] + (uint32_t)(b_) * kBufferB) + (i_) * 4 * kInt8StageK)
#define RD_X(j_, h_, b_) \
  *reinterpret_cast<const i32x4*>(ring + (rdX[(h_)] + (uint32_t)(b_) * kBufferB) + (j_) * 16 * kInt8StageK)
#define FENCE() __builtin_amdgcn_sched_barrier(0)

  // One step: eight groups (W tile g with X tiles 0 .. 7) on fw and mx_, 64 codes
  // (z_: from zero sums), while the next step's fragments are read from half rh_
  // of buffer rb_: X tiles 2 g and 2 g + 1 into nx_ during group g < 4, W tile g
  // into fw[g] behind group g, its last use. A stage (two steps, slots from p0_
  // on) issues its copies of stage ck_ into buffer cb_. The order is fixed.
  i32x4 acc[kTiles][kTiles];  // [W tile][X tile]
  i32x4 fw[kTiles], fx0[kTiles], fx1[kTiles];
#define STEP(do_mma_, z_, do_rd_, mx_, nx_, rh_, rb_, p0_, ck_, cb_)                          \
  do {                                                                                        \
    _Pragma("unroll") for (int u = 0; u < kTiles * kTiles; ++u) {                             \
      const int g_ = u >> 3, j_ = u & 7;                                                      \
      if (do_mma_)                                                                            \
        acc[g_][j_] = mma(fw[g_], mx_[j_], (z_) ? i32x4{0, 0, 0, 0} : acc[g_][j_]);           \
      if ((do_rd_) && g_ < 4 && j_ == 2) nx_[2 * (g_ & 3)] = RD_X(2 * (g_ & 3), (rh_), (rb_)); \
      if ((do_rd_) && g_ < 4 && j_ == 5)                                                      \
        nx_[2 * (g_ & 3) + 1] = RD_X(2 * (g_ & 3) + 1, (rh_), (rb_));                         \
      if ((do_rd_) && j_ == 7) fw[g_] = RD_W(g_, (rh_), (rb_));                               \
      const int pu_ = (p0_) + u;                                                              \
      if (pu_ % kSlotsPerCopy == 1 && pu_ / kSlotsPerCopy < 2 * kUnitCopies)                  \
        COPY(pu_ / kSlotsPerCopy, (ck_), (cb_));                                              \
      FENCE();                                                                                \
    }                                                                                         \
  } while (0)

#pragma unroll
  for (int c = 0; c < 2 * kUnitCopies; ++c) COPY(c, 0, 0);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __syncthreads();
  FENCE();
  constexpr int kHalf = kTiles * kTiles;
  STEP(false, false, true, fx1, fx0, 0, 0, 0, 1, 1);
  STEP(true, true, true, fx0, fx1, 1, 0, kHalf, 1, 1);
  for (int k = 1; k < nk; ++k) {
    const int b = k & 1;
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    FENCE();
    STEP(true, false, true, fx1, fx0, 0, b, 0, k + 1, b ^ 1);
    STEP(true, false, true, fx0, fx1, 1, b, kHalf, k + 1, b ^ 1);
  }
  STEP(true, false, false, fx1, fx0, 0, 0, 4 * kHalf, 0, 0);
  __builtin_amdgcn_s_waitcnt(0x0070);  // the last copies land before the LDS is given back
#undef STEP
#undef COPY
#undef RD_W
#undef RD_X
#undef FENCE

  const int vb = v0 + wm * kInt8BlockV;
  if (vb >= a.V) return;
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    const int t = t0 + wn * 128 + 16 * j + lcol;
    i32x4 sum[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) sum[i] = acc[i][j];
    if constexpr (std::is_void_v<D>) store_partial(a, sum, vb, t, lg);
    else store_logits<D>(a, sum, vb, t, lg);
  }
}

// ---- Merge ------------------------------------------------------------------
// A workgroup joins 64 tokens' partials: wave w folds the blocks of segment w
// in ascending order, then the segments are folded in order. The bounds depend
// on the vocabulary alone.
constexpr int kSegs = 16;

__global__ __launch_bounds__(64 * kSegs) void merge_kernel(Int8Args a) {
  __shared__ float seg_m[kSegs][64], seg_s[kSegs][64];
  const int lane = threadIdx.x & 63, seg = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 64 + lane;
  const int blocks = (a.V + kInt8BlockV - 1) / kInt8BlockV;
  const int per = (blocks + kSegs - 1) / kSegs;
  const int lo = min(blocks, seg * per), hi = min(blocks, lo + per);
  float M = -INFINITY, S = 0.0f;
  if (t < a.T)
    for (int b = lo; b < hi; ++b)
      lse_fold(M, S, a.part_m[(int64_t)b * a.T + t], a.part_s[(int64_t)b * a.T + t]);
  seg_m[seg][lane] = M;
  seg_s[seg][lane] = S;
  __syncthreads();
  if (seg != 0 || t >= a.T) return;
#pragma unroll
  for (int g = 1; g < kSegs; ++g) lse_fold(M, S, seg_m[g][lane], seg_s[g][lane]);
  const int64_t id = a.ids[t];
  const bool ok = id >= 0 && id < a.V;
  const float lse2 = M + fast_log2(S);
  a.out_lp[t] = ok ? (a.tval[t] - lse2) * kLn2 : NAN;
  if (a.out_lse) a.out_lse[t] = lse2 * kLn2;
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

template <int kNT>
void stream(const Int8Args& a, hipStream_t s) {
  const dim3 grid((uint32_t)((a.V + kInt8BlockV - 1) / kInt8BlockV),
                  (uint32_t)((a.T + 16 * kNT - 1) / (16 * kNT)));
  const int threads = 64 * kStreamWaves;
  if (!a.out) stream_kernel<kNT, void><<<grid, threads, 0, s>>>(a);
  else if (a.dtype == LP_F32) stream_kernel<kNT, F32><<<grid, threads, 0, s>>>(a);
  else if (a.dtype == LP_BF16) stream_kernel<kNT, BF16><<<grid, threads, 0, s>>>(a);
  else stream_kernel<kNT, F16><<<grid, threads, 0, s>>>(a);
}

void tiles(const Int8Args& a, hipStream_t s) {
  const int n_vt = (a.V + kTileRows - 1) / kTileRows, n_tt = (a.T + kTileRows - 1) / kTileRows;
  const dim3 grid((uint32_t)n_vt * (uint32_t)n_tt);
  if (!a.out) tile_kernel<void><<<grid, kTileThreads, 0, s>>>(a, n_vt, n_tt);
  else if (a.dtype == LP_F32) tile_kernel<F32><<<grid, kTileThreads, 0, s>>>(a, n_vt, n_tt);
  else if (a.dtype == LP_BF16) tile_kernel<BF16><<<grid, kTileThreads, 0, s>>>(a, n_vt, n_tt);
  else tile_kernel<F16><<<grid, kTileThreads, 0, s>>>(a, n_vt, n_tt);
}

}  // namespace

Int8Workspace int8_workspace_layout(int64_t T, int64_t H, int64_t V) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t plane = (size_t)((V + kInt8BlockV - 1) / kInt8BlockV) * (size_t)T * sizeof(float);
  Int8Workspace w;
  w.off_staged = 0;
  w.off_m = up((size_t)T * (size_t)int8_staged_row(H));
  w.off_s = w.off_m + up(plane);
  w.off_t = w.off_s + up(plane);
  w.total = V > 0 ? w.off_t + up((size_t)T * sizeof(float)) : w.off_m;
  return w;
}

bool int8_grid_ok(int64_t T, int64_t V) {
  const int64_t blocks = (V + kInt8BlockV - 1) / kInt8BlockV, tiles = (T + 63) / 64;
  return tiles <= 65535 && blocks * tiles <= kMaxDispatchItems / (64 * kStreamWaves) &&
         tiles <= kMaxDispatchItems / (64 * kSegs);
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
  if (a.T <= 16) stream<1>(a, stream_);
  else if (a.T <= 32) stream<2>(a, stream_);
  else if (a.T <= 64) stream<4>(a, stream_);
  else tiles(a, stream_);
  if ((e = hipGetLastError()) != hipSuccess || a.out) return e;
  merge_kernel<<<dim3((uint32_t)((a.T + 63) / 64)), 64 * kSegs, 0, stream_>>>(a);
  return hipGetLastError();
}

}  // namespace lp
