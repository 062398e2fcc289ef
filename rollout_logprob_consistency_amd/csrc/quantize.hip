// Rows in 8-bit integers with a scale each (lp_quantize_int8).
//
//   scale = max |x| (1 / 127),   q = the integer nearest to x / scale
//
// One pass: a row's lanes hold it in registers between the maximum and the codes, so
// it is read once (rows of more than 16 KiB are read again, from L2).
#include "int8_internal.h"

#define LP_INLINE __attribute__((always_inline))

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

// A group's largest magnitude; NaN and infinities count as `odd`. Places behind the
// row hold zeros.
template <class D>
__device__ __forceinline__ void max_abs(const Group<D>& g, float& m, bool& odd) {
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const float v = fabsf(g.get(i));
    m = fmaxf(m, v);
    odd |= !(v < INFINITY);
  }
}

template <class D>
__device__ __forceinline__ Group<D> load_zeros(const typename D::Raw* p, int64_t at, int64_t H) {
  if (at + D::kVec <= H) return load_whole<D>(p + at);
  Group<D> g = {{0, 0, 0, 0}};
  const Global<const typename D::Raw> q = (Global<const typename D::Raw>)p;
#pragma unroll
  for (int i = 0; i < D::kVec; ++i)
    if (at + i < H) g.set(i, q[at + i]);
  return g;
}

// A row's scale as stored, and what its elements are divided by.
struct Scale {
  float s, inv, lift;
};
__device__ __forceinline__ Scale scale_of(const QuantizeArgs& a, int64_t row, float m, bool bad,
                                          bool first) {
  float s = bad ? 0.0f : m * (1.0f / 127.0f);
  if (first) {
    a.scale[row] = bad ? NAN : s;
    if (bad && a.bad_rows) atomicAdd(a.bad_rows, 1);
  }
  const float lift = s < kTiny ? 0x1p64f : 1.0f;
  s *= lift;
  return {s, 1.0f / s, lift};
}

// The codes of a group; zeros behind the row give zeros, up to a multiple of 16
// (the row's last group may lie wholly behind its elements).
template <class D>
__device__ __forceinline__ void put_codes(int8_t* q, int64_t at, const Group<D>& g, Scale s) {
  uint32_t w[D::kVec / 4];
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const int c = s.s > 0.0f ? code_of(g.get(i) * s.lift, s.s, s.inv) : 0;
    if (i % 4 == 0) w[i / 4] = 0;
    w[i / 4] |= (uint32_t)(c & 0xFF) << (8 * (i % 4));
  }
  typedef uint32_t Pair __attribute__((ext_vector_type(2)));
  if constexpr (D::kVec == 8) *(Global<Pair>)(Pair*)(q + at) = Pair{w[0], w[1]};
  else *(Global<uint32_t>)(uint32_t*)(q + at) = w[0];
}

// The maximum over each kLanes lanes of a wave, by the fixed XOR butterfly.
template <int kLanes>
__device__ __forceinline__ float lanes_max(float m) {
  auto step = [&](auto of) LP_INLINE { m = fmaxf(m, __int_as_float(of(__float_as_int(m)))); };
  step([](int x) LP_INLINE { return xlane<1>(x); });
  step([](int x) LP_INLINE { return xlane<2>(x); });
  step([](int x) LP_INLINE { return xlane<4>(x); });
  if constexpr (kLanes >= 16) step([](int x) LP_INLINE { return xlane<8>(x); });
  if constexpr (kLanes >= 32) step([](int x) LP_INLINE { return xlane<16>(x); });
  if constexpr (kLanes == 64)
    m = fmaxf(__int_as_float(lane_value(__float_as_int(m), 0)),
              __int_as_float(lane_value(__float_as_int(m), 32)));
  return m;
}

// kLanes lanes hold a row in kG groups each: it is read once.
template <class D, int kLanes, int kG>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a) {
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool there = row < a.R;
  const typename D::Raw* p = static_cast<const typename D::Raw*>(a.x) + (there ? row : 0) * a.ldx;
  Group<D> g[kG];
#pragma unroll
  for (int j = 0; j < kG; ++j) g[j] = load_zeros<D>(p, (j * kLanes + lane) * D::kVec, a.H);
  float m = 0.0f;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kG; ++j) max_abs<D>(g[j], m, odd);
  m = lanes_max<kLanes>(m);
  uint64_t odds = __ballot(odd);
  if constexpr (kLanes < 64) odds &= ((uint64_t(1) << kLanes) - 1) << (threadIdx.x & 63 & ~(kLanes - 1));
  if (!there) return;
  const Scale s = scale_of(a, row, m, odds != 0, lane == 0);
  int8_t* q = a.q + row * a.ldq;
  const int64_t H16 = (a.H + 15) / 16 * 16;
#pragma unroll
  for (int j = 0; j < kG; ++j) {
    const int64_t at = (j * kLanes + lane) * D::kVec;
    if (at < H16) put_codes<D>(q, at, g[j], s);
  }
}

// Longer rows, a wave each, are read again for the codes.
template <class D>
__global__ __launch_bounds__(kThreads) void quantize_long_kernel(QuantizeArgs a) {
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (row >= a.R) return;
  const int lane = threadIdx.x & 63;
  const typename D::Raw* p = static_cast<const typename D::Raw*>(a.x) + row * a.ldx;
  constexpr int kStep = 64 * D::kVec;
  float m = 0.0f;
  bool odd = false;
  for (int64_t at = lane * D::kVec; at < a.H; at += kStep)
    max_abs<D>(load_zeros<D>(p, at, a.H), m, odd);
  const Scale s = scale_of(a, row, lanes_max<64>(m), __ballot(odd) != 0, lane == 0);
  int8_t* q = a.q + row * a.ldq;
  const int64_t H16 = (a.H + 15) / 16 * 16;
  for (int64_t at = lane * D::kVec; at < H16; at += kStep)
    put_codes<D>(q, at, load_zeros<D>(p, at, a.H), s);
}

template <class D, int kLanes, int kG>
void rows(const QuantizeArgs& a, hipStream_t stream) {
  constexpr int kRows = kThreads / kLanes;
  quantize_kernel<D, kLanes, kG>
      <<<dim3((uint32_t)((a.R + kRows - 1) / kRows)), kThreads, 0, stream>>>(a);
}

// As many lanes as a row has groups, up to a wave, then groups a lane.
template <class D>
void launch(const QuantizeArgs& a, hipStream_t stream) {
  const int64_t groups = (a.H + 15) / 16 * 16 / D::kVec;
  if (groups <= 8) rows<D, 8, 1>(a, stream);
  else if (groups <= 16) rows<D, 16, 1>(a, stream);
  else if (groups <= 32) rows<D, 32, 1>(a, stream);
  else if (groups <= 64) rows<D, 64, 1>(a, stream);
  else if (groups <= 128) rows<D, 64, 2>(a, stream);
  else if (groups <= 256) rows<D, 64, 4>(a, stream);
  else if (groups <= 512) rows<D, 64, 8>(a, stream);
  else if (groups <= 1024) rows<D, 64, 16>(a, stream);
  else
    quantize_long_kernel<D>
        <<<dim3((uint32_t)((a.R + kWaves - 1) / kWaves)), kThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_quantize_int8(const QuantizeArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case LP_F32: launch<F32>(a, stream); break;
    case LP_BF16: launch<BF16>(a, stream); break;
    default: launch<F16>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace lp
