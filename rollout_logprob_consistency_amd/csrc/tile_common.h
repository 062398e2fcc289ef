// Shared by the LM-head products (score.hip, int8.hip): which tile a workgroup
// takes, copies from memory straight into LDS, and lane exchanges.
#pragma once

#include "lp_internal.h"

namespace lp {
namespace {

// Workgroup id -> (vocab tile, token tile). The hardware deals workgroups to
// the 8 XCDs round-robin; give each XCD a contiguous run of logical tiles, and
// order logical tiles in groups of kGroupV vocab tiles with the token tile
// varying fastest, so the workgroups resident on one XCD share W and X slabs
// in that XCD's L2.
__device__ __forceinline__ void tile_of(int b, int n_vt, int n_tt, int group_v, int& vt, int& tt) {
  const int G = n_vt * n_tt;
  const int xcd = b & 7, idx = b >> 3;
  const int per = G >> 3, rem = G & 7;
  const int L = (xcd < rem) ? xcd * (per + 1) + idx
                            : rem * (per + 1) + (xcd - rem) * per + idx;
  const int group = group_v * n_tt;
  const int g = L / group;
  const int first = g * group_v;
  const int gv = min(group_v, n_vt - first);
  const int r = L - g * group;
  vt = first + r % gv;
  tt = r / gv;
}

// Direct buffer -> LDS copies (buffer_load_dwordx4 ... lds): one 16-byte chunk
// per lane, the wave's 64 chunks landing contiguously at the LDS address
// (lane i at byte 16 i); no VGPR round trip.
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
constexpr int kRsrcWord3 = 0x00020000;  // raw buffer, 32-bit data format (gfx9)

// Byte extent of a buffer resource, capped to what num_records can hold.
__device__ __forceinline__ uint32_t span_bytes(uint64_t n) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(n > 0x7FFFFFF0ull ? 0x7FFFFFF0ull : n));
}

// Buffer resource from wave-uniform values, built so the compiler keeps it in
// SGPRs (a resource it cannot prove uniform costs a waterfall loop per load).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  const uint64_t pu = ((uint64_t)hi << 32) | lo;
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(pu), 0,
                                           (int)__builtin_amdgcn_readfirstlane(bytes), kRsrcWord3);
}

// One 1-KiB buffer -> LDS copy (buffer_load_dwordx4 ... lds): lane i moves 16
// bytes from rsrc + voff + soff to LDS byte address lds + 16 i. Written as
// inline assembly so that the compiler does not treat the asynchronous LDS
// write as aliasing every later LDS read (it would wait for every copy in
// flight before each read); the ring's explicit vmcnt waits and barriers order
// copies and reads instead. The LDS address goes in M0 (an operand of the
// statement); an M0 write needs one wait state before an LDS-DMA load.
__device__ __forceinline__ void copy_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, uint32_t voff,
                                         uint32_t soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds)
               : "memory");
}

// The value lane l ^ 16 (kOff = 16) or lane l ^ 32 (kOff = 32) holds, by the
// VALU lane swaps of gfx950 instead of an LDS permute: swapping x with itself
// puts, in the first result, the even rows' (lower half's) values into the
// odd rows (upper half) and, in the second, the odd rows' into the even rows.
template <int kOff>
__device__ __forceinline__ int xor_lane(int x) {
  const int lane = (int)__lane_id();
  if constexpr (kOff == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (lane & 16) ? (int)r[0] : (int)r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return (lane & 32) ? (int)r[0] : (int)r[1];
  }
}

template <int kOff>
__device__ __forceinline__ float xor_lane(float x) {
  return __int_as_float(xor_lane<kOff>(__float_as_int(x)));
}

}  // namespace
}  // namespace lp
