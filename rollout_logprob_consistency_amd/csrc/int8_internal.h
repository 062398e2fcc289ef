// The 8-bit head (include/liblp_int8.h): launch interface between the C-ABI
// host code and the kernels.
#pragma once

#include "liblp_int8.h"
#include "logits_internal.h"

namespace lp {

// Vocabulary rows of a block: one (maximum, sum) partial of the log-sum-exp
// for each block and token, formed by one wave. Never depends on the batch.
constexpr int kInt8BlockV = 128;
// Bytes (codes) of a row per K stage: whole 128-byte lines.
constexpr int kInt8StageK = 128;

struct QuantizeArgs {
  const void* x;
  int64_t ldx;
  int32_t dtype;
  int64_t R, H;
  int8_t* q;
  int64_t ldq;
  float* scale;
  int32_t* bad_rows;  // or null
};
hipError_t launch_quantize_int8(const QuantizeArgs& a, hipStream_t stream);

struct Int8Args {
  const int8_t* x;       // [T, ldx]
  const float* x_scale;  // [T]
  const int8_t* w;       // [V, ldw]
  const float* w_scale;  // [V]
  int64_t ldx, ldw;
  int32_t T, H, V;
  // Rows of logits.
  void* out;             // [T, ld_out] or null: the scores
  int64_t ld_out;
  int32_t dtype;
  // Scores.
  const int64_t* ids;    // [T]
  bool bf16_logits;
  float scale2;          // log2(e) / temperature
  float* part_m;         // [blocks][T] maximum of z, log2 units
  float* part_s;         // [blocks][T] sum of exp2(z - maximum)
  float* out_lp;         // [T]
  float* out_lse;        // [T] or null
  int32_t* bad_rows;     // or null
  int8_t* staged;        // [T, staged row] x laid out in whole stages
};

// Elements of a row of hidden states laid out in whole stages.
constexpr int64_t int8_staged_row(int64_t H) {
  return (H + kInt8StageK - 1) / kInt8StageK * kInt8StageK;
}
// Largest row stride that the kernels read or write: 256 rows of codes, and 128
// of logits, stay inside 32-bit byte offsets.
constexpr int64_t kInt8StrideMax = int64_t(1) << 22;
// Whether the kernels can read x where it lies: whole stages of 16-byte
// aligned rows.
inline bool int8_reads_in_place(const int8_t* x, int64_t ldx, int64_t H) {
  return H % kInt8StageK == 0 && ldx % 16 == 0 && ldx <= kInt8StrideMax &&
         reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

struct Int8Workspace {
  size_t off_staged, off_m, off_s, total;
};
// V = 0: rows of logits, no partials.
Int8Workspace int8_workspace_layout(int64_t T, int64_t H, int64_t V);

// Most tokens of a product, as the interface names it.
constexpr int64_t kInt8TokensMax = 4194240;
// Whether every dispatch of a product of these sizes fits 2^32 - 1 work-items, and
// its tiles 32 bits.
bool int8_grid_ok(int64_t T, int64_t V);

// `a.staged` is used where x is not read in place.
hipError_t launch_int8(Int8Args a, hipStream_t stream);

}  // namespace lp
