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

template <int kOff>
__device__ __forceinline__ float xor_lane(float v) {
  const int x = __float_as_int(v), lane = (int)__lane_id();
  if constexpr (kOff == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __int_as_float((lane & 16) ? (int)r[0] : (int)r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __int_as_float((lane & 32) ? (int)r[0] : (int)r[1]);
  }
}

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
  for (int k = wave; k < nk; k += kStreamWaves) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      i32x4 x[kNT];
#pragma unroll
      for (int j = 0; j < kNT; ++j) x[j] = load(xres, xoff[j] + 64 * c, k);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const i32x4 w = load(wres, woff[i] + 64 * c, k);
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[j][i] = mma(w, x[j], acc[j][i]);
      }
    }
  }
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
  else stream<4>(a, stream_);
  if ((e = hipGetLastError()) != hipSuccess || a.out) return e;
  merge_kernel<<<dim3((uint32_t)((a.T + 63) / 64)), 64 * kSegs, 0, stream_>>>(a);
  return hipGetLastError();
}

}  // namespace lp
