// Rows in 8-bit integers with a scale each (lp_quantize_int8).
//
//   scale = max |x| (1 / 127),   q = the integer nearest to x / scale
//
// (The factor is fp32's 1 / 127, which is off by 2^-28: a row's scale is max / 127 to
// 1.07 half steps, and its largest code is 127 as it would be after a division.)
//
// One pass: a row's lanes hold it in registers between the maximum and the codes, so
// it is read once (rows of more than 32 KiB are read again, from L2). Memory bounds it:
// 151 936 rows of 4 096 bf16 take 331 us, 5.6 TB/s read and written.
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

// Magnitudes as the bits of their type: they order as integers, infinities above the
// finite ones and NaN above both. Two 16-bit ones share a word.
typedef uint16_t Halves __attribute__((ext_vector_type(2)));
template <class D>
__device__ __forceinline__ void max_abs(const Group<D>& g, uint32_t& m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (D::kVec == 4) {
      m = max(m, g.w[i] & 0x7FFFFFFFu);
    } else {
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
              __builtin_bit_cast(Halves, m), __builtin_bit_cast(Halves, g.w[i] & 0x7FFF7FFFu)));
    }
  }
}
template <class D>
__device__ __forceinline__ uint32_t larger_half(uint32_t m) {
  return D::kVec == 4 ? m : max(m & 0xFFFFu, m >> 16);
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
template <class D>
__device__ __forceinline__ Scale scale_of(const QuantizeArgs& a, int64_t row, uint32_t bits,
                                          bool first) {
  const float m = D::value((typename D::Raw)bits);
  const bool bad = !(m < INFINITY);
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
// (the row's last group may lie wholly behind its elements). Adding 1.5 2^23 rounds
// x / s to an integer and leaves it in the low byte. Where the rest is below half a
// step for all of a wave's elements that was the nearest one (7 instructions an
// element; 20 by code_of, which bounded the kernel: 151 936 rows of 4 096
// bf16 420 us by code_of, 344 us this way); else, and in rows that are scaled first, code_of decides.
template <class D>
__device__ __forceinline__ void put_codes(int8_t* q, int64_t at, const Group<D>& g, Scale s) {
  constexpr float kMagic = 12582912.0f;
  const float h = 0.5f * s.s;
  uint32_t w[D::kVec / 4], t[D::kVec];
  bool near = s.lift == 1.0f;
#pragma unroll
  for (int i = 0; i < D::kVec; ++i) {
    const float x = g.get(i), r = __builtin_fmaf(x, s.inv, kMagic);
    near &= fabsf(__builtin_fmaf(-(r - kMagic), s.s, x)) < h;
    t[i] = __float_as_uint(r);
  }
#pragma unroll
  for (int i = 0; i < D::kVec; i += 4)
    w[i / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t[i + 3], t[i + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(t[i + 1], t[i], 0x0C0C0400u),
                                     0x05040100u);
  if (__ballot(!near)) {
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) {
      const int c = s.s > 0.0f ? code_of(g.get(i) * s.lift, s.s, s.inv) : 0;
      if (i % 4 == 0) w[i / 4] = 0;
      w[i / 4] |= (uint32_t)(c & 0xFF) << (8 * (i % 4));
    }
  }
  // (Past the caches: the same rows 333 us, 344 us without.)
  typedef uint32_t Pair __attribute__((ext_vector_type(2)));
  if constexpr (D::kVec == 8) __builtin_nontemporal_store(Pair{w[0], w[1]}, (Global<Pair>)(Pair*)(q + at));
  else __builtin_nontemporal_store(w[0], (Global<uint32_t>)(uint32_t*)(q + at));
}

// The maximum over each kLanes lanes of a wave, by the fixed XOR butterfly.
template <int kLanes>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  int m = (int)v;  // (magnitudes have no sign bit)
  m = max(m, xlane<1>(m));
  m = max(m, xlane<2>(m));
  m = max(m, xlane<4>(m));
  if constexpr (kLanes >= 16) m = max(m, xlane<8>(m));
  if constexpr (kLanes >= 32) m = max(m, xlane<16>(m));
  if constexpr (kLanes == 64) m = max(lane_value(m, 0), lane_value(m, 32));
  return (uint32_t)m;
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
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kG; ++j) max_abs<D>(g[j], m);
  m = lanes_max<kLanes>(larger_half<D>(m));
  if (!there) return;
  const Scale s = scale_of<D>(a, row, m, lane == 0);
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
  uint32_t m = 0;
  for (int64_t at = lane * D::kVec; at < a.H; at += kStep)
    max_abs<D>(load_zeros<D>(p, at, a.H), m);
  const Scale s = scale_of<D>(a, row, lanes_max<64>(larger_half<D>(m)), lane == 0);
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
  else if (groups <= 2048) rows<D, 64, 32>(a, stream);
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
