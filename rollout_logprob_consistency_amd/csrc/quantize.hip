// Rows in 8-bit integers with a scale each (lp_quantize_int8).
//
//   scale = max |x| (1 / 127),   q = the integer nearest to x / scale
//
// One pass: a wave holds its row in registers between the maximum and the
// codes, so the row is read once (longer rows are read again, from L2).
#include "int8_internal.h"

namespace lp {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The integer nearest to x / s for s > 0, |x| <= 127.5 s: r = rint(x * (1 / s))
// is it or a neighbour, as the product is off by 2^-22 relative. x - r s is
// exact in one fused step (a multiple of s's last place, or of x's below it,
// and smaller than 2 s), so comparing it with s / 2 decides, ties to even.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
  float r = rintf(x * inv);
  const float e = __builtin_fmaf(-r, s, x), h = 0.5f * s;
  const int i = (int)r;
  const bool odd = i & 1;
  const int up = e > h || (e == h && odd), down = e < -h || (e == -h && odd);
  return max(-127, min(127, i + up - down));
}

// Below this the scale's reciprocal or its half leave fp32's normal range:
// such rows are scaled by 2^64 first, which changes no quotient.
constexpr float kTiny = 0x1p-60f;

template <class D>
__device__ __forceinline__ void max_abs(const Group<D>& g, float& m, bool& odd) {
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const float v = fabsf(g.get(i));
    m = fmaxf(m, v);
    odd |= !(v < INFINITY);
  }
}

// The codes of elements [at, at + kVec) of a row; those behind H are zeros, up
// to a multiple of 16 (the row's last group may lie wholly behind H).
template <class D>
__device__ __forceinline__ void put_codes(int8_t* q, int64_t at, int64_t H, const Group<D>& g,
                                          float s, float inv, float lift) {
  uint32_t w[D::kVec / 4];
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const int c = at + i < H && s > 0.0f ? code_of(g.get(i) * lift, s, inv) : 0;
    if (i % 4 == 0) w[i / 4] = 0;
    w[i / 4] |= (uint32_t)(c & 0xFF) << (8 * (i % 4));
  }
  typedef uint32_t Pair __attribute__((ext_vector_type(2)));
  if constexpr (D::kVec == 8) *(Global<Pair>)(Pair*)(q + at) = Pair{w[0], w[1]};
  else *(Global<uint32_t>)(uint32_t*)(q + at) = w[0];
}

template <class D>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a) {
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (row >= a.R) return;
  const int lane = threadIdx.x & 63;
  const typename D::Raw* p = static_cast<const typename D::Raw*>(a.x) + row * a.ldx;
  constexpr int kStep = 64 * D::kVec;
  float m = 0.0f;
  bool odd = false;
  for (int64_t at = lane * D::kVec; at < a.H; at += kStep) {
    const int64_t end = a.H;
    Group<D> g = load_group<D>(p, at, end);
#pragma unroll
    for (int i = 0; i < D::kVec; ++i)
      if (at + i >= end) g.set(i, 0);
    max_abs<D>(g, m, odd);
  }
  m = wave_max_f32(m);
  const bool bad = __ballot(odd) != 0;
  float s = bad ? 0.0f : m * (1.0f / 127.0f);
  if (lane == 0) {
    a.scale[row] = bad ? NAN : s;
    if (bad && a.bad_rows) atomicAdd(a.bad_rows, 1);
  }
  const float lift = s < kTiny ? 0x1p64f : 1.0f;
  s *= lift;
  const float inv = 1.0f / s;
  int8_t* q = a.q + row * a.ldq;
  const int64_t H16 = (a.H + 15) / 16 * 16;
  for (int64_t at = lane * D::kVec; at < H16; at += kStep)
    put_codes<D>(q, at, a.H, load_group<D>(p, at, a.H), s, inv, lift);
}

}  // namespace

hipError_t launch_quantize_int8(const QuantizeArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)((a.R + kWaves - 1) / kWaves));
  switch (a.dtype) {
    case LP_F32: quantize_kernel<F32><<<grid, kThreads, 0, stream>>>(a); break;
    case LP_BF16: quantize_kernel<BF16><<<grid, kThreads, 0, stream>>>(a); break;
    default: quantize_kernel<F16><<<grid, kThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace lp
