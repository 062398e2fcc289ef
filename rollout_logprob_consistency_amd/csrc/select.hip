// Token draw (lp_sample) and top logits (lp_top_logprobs): the kernels of
// select_row.h and their launches.
#include <algorithm>

#include "select_row.h"

namespace lp {
namespace {

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
    list_by_buckets<D, kTopLogits>(a, settings_of<kTopLogits>(a, n), n,
                                   row_at<D, kTopLogits>(a, n), sh);
    __syncthreads();
  }
}

template <class D, Job kJob>
hipError_t launch(const SelectArgs& a, bool lists, bool buckets, hipStream_t stream) {
  hipError_t e;
  if (lists || (buckets && a.slices > 1)) {
    collect_kernel<D, kJob><<<dim3((uint32_t)(a.N * a.slices)), kThreads, 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (kJob == kTopLogits && lists && a.slices == 1)
    overflow_kernel<D><<<dim3((uint32_t)((a.N + kCheckRows - 1) / kCheckRows)), kThreads, 0,
                         stream>>>(a);
  else
    row_kernel<D, kJob><<<dim3((uint32_t)a.N), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Slices of a row: whole chunks, in all at most two workgroups for each of the
// card's 256 CUs. Times with 256, 512, 768 and 1 024 workgroups at most: top 100 of
// fp16 rows of 50 021, 100 rows 29, 30, 30 and 30 us, 200 rows 33, 34, 34 and 41, 300
// rows 40, 40, 42 and 44, 400 rows 42, 41, 42 and 51; draws over rows of 151 936, 64
// bf16 rows by top-k 20 30, 30, 27 and 27, 300 rows 55, 55, 52 and 53, 512 rows 61, 61,
// 61 and 73; 64 fp32 rows by nucleus 93, 96, 97 and 103.
static_assert(LP_SELECT_MAX_VOCAB / chunk_of<F32>() <= kMaxSlices, "slices of one row");
static int64_t select_chunks(int64_t V, int32_t dtype) {
  const int64_t chunk = (int64_t)kThreads * kGroups * (16 / dtype_bytes(dtype));
  return (V + chunk - 1) / chunk;
}
static int64_t select_slices(int64_t N, int64_t V, int32_t dtype, int64_t places) {
  return std::max<int64_t>(1, std::min(select_chunks(V, dtype), places / std::max<int64_t>(N, 1)));
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

SelectWorkspace select_workspace_layout(int64_t N, int64_t V, int32_t dtype, int64_t places) {
  const int64_t slices = select_slices(N, V, dtype, places);
  const size_t all = (size_t)(N * slices);
  return layout_of(all, slices > 1 ? (size_t)N : 0, slices > 1 ? all : 0, select_chunks(V, dtype));
}

size_t select_workspace_most(int64_t N, int64_t V, int32_t dtype, int64_t places) {
  // Every term of layout_of at its largest over 1 .. N rows.
  const int64_t chunks = select_chunks(V, dtype);
  const int64_t cut_rows = chunks > 1 ? std::min(N, places / 2) : 0;
  const int64_t cut_slices = std::min(places, cut_rows * chunks);
  return layout_of((size_t)std::max(N, cut_slices), (size_t)cut_rows, (size_t)cut_slices,
                   (size_t)chunks)
      .total;
}

void place_select(SelectArgs& a, void* workspace, int64_t places) {
  const SelectWorkspace w = select_workspace_layout(a.N, a.V, a.dtype, places);
  char* base = static_cast<char*>(workspace);
  a.slices = (int32_t)select_slices(a.N, a.V, a.dtype, places);
  a.counts = reinterpret_cast<uint32_t*>(base + w.off_counts);
  a.parts = reinterpret_cast<SelectPart*>(base + w.off_parts);
  a.keys = reinterpret_cast<uint64_t*>(base + w.off_keys);
  a.masses = reinterpret_cast<unsigned long long*>(base + w.off_masses);
  a.bucket_counts = reinterpret_cast<uint32_t*>(base + w.off_bucket_counts);
  a.facts = reinterpret_cast<RowFacts*>(base + w.off_facts);
}

SelectWays select_ways(const SelectArgs& a) {
  const bool seen = !a.temperatures && !a.top_ks && !a.top_ps && !a.min_ps;
  const bool short_list = a.temperature == 0.0f || (a.top_k > 0 && a.top_k <= kShortTop) ||
                          (a.top_k <= 0 && a.top_p >= 1.0f && a.min_p > 0.0f && a.min_p <= 1.0f);
  return {!seen || short_list, !seen || !short_list};
}

hipError_t launch_select(SelectArgs a, void* workspace, hipStream_t stream) {
  place_select(a, workspace, kSelectPlaces);
  const bool top = a.u == nullptr;
  const SelectWays ways = select_ways(a);
  const bool lists = top ? a.top_k <= kShortTop : ways.lists, buckets = !top && ways.buckets;
  switch (a.dtype) {
    case LP_F32:
      return top ? launch<F32, kTopLogits>(a, lists, buckets, stream)
                 : launch<F32, kDraw>(a, lists, buckets, stream);
    case LP_BF16:
      return top ? launch<BF16, kTopLogits>(a, lists, buckets, stream)
                 : launch<BF16, kDraw>(a, lists, buckets, stream);
    default:
      return top ? launch<F16, kTopLogits>(a, lists, buckets, stream)
                 : launch<F16, kDraw>(a, lists, buckets, stream);
  }
}

}  // namespace lp
