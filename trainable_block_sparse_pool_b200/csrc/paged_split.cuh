// What the paged decode attention's ranges leave to join, as plain integers (compiled for the host too).
//
// Worker w (a warp; kWarps a CTA) has the costs [share w, share (w + 1)) of the total.  The pieces of a pair that
// begins in worker `first` and ends in another CTA, or in a worker that goes on to another pair, are
//   the second slot of `first` (its run of warps in that CTA),
//   the first slots of the next CTAs' first workers, `ctas` CTAs in all,
//   the first slot of worker `last`, or nothing where last is -1.
//
// Lengths are read on the device by every CTA for itself, so lengths that change while a call runs give CTAs that
// disagree: a pair whose descriptor nobody writes (the workspace holds anything then), or whose end lies past the
// last worker.  Such a call's results mean nothing, but its accesses have to stay in bounds:
// describe_join names existing workers only, and a descriptor is joined only when join_in_bounds says so of it.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define INFLLM2_HD __host__ __device__ __forceinline__
#else
#define INFLLM2_HD inline
#endif

namespace infllm2 {

namespace pattn {

constexpr int kWarps = 8;

struct alignas(16) Join {
  int32_t first, ctas, last, pair;   // ctas = 0: nothing to join
};

INFLLM2_HD int64_t div_pos(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// Of a pair that begins in worker wk, whose range ends at cost x1, with `rest` of the pair behind it.
INFLLM2_HD Join describe_join(int32_t wk, int32_t pair, int64_t x1, int64_t rest, int64_t share, int64_t total,
                              int32_t ctas) {
  const int64_t end = x1 + rest, workers = static_cast<int64_t>(ctas) * kWarps;
  const int64_t w = div_pos(end - 1, share);
  const int32_t wl = static_cast<int32_t>(w < workers ? w : workers - 1), c1 = wl / kWarps;
  Join j{wk, c1 - wk / kWarps + 1, -1, pair};
  // whether the last worker goes on to another pair's tiles
  const int64_t next = (static_cast<int64_t>(wl) + 1) * share;
  const bool on = (total < next ? total : next) - end >= 2;
  if (on && wl > (wk > c1 * kWarps ? wk : c1 * kWarps)) j.last = wl;
  return j;
}

// Whether all slots and rows of the output that j names exist.
INFLLM2_HD bool join_in_bounds(const Join& j, int32_t pairs, int32_t ctas) {
  return j.first >= 0 && j.first < ctas * kWarps && j.ctas > 0 && j.ctas <= ctas - j.first / kWarps && j.last >= -1 &&
         j.last < ctas * kWarps && j.pair >= 0 && j.pair < pairs;
}

INFLLM2_HD int32_t join_pieces(const Join& j) { return j.ctas + (j.last >= 0 ? 1 : 0); }

// Slot of piece i < join_pieces(j).
INFLLM2_HD int32_t join_slot(const Join& j, int32_t i) {
  const int32_t w = i == 0 ? j.first : i < j.ctas ? (j.first / kWarps + i) * kWarps : j.last;
  return 2 * w + (i == 0 ? 1 : 0);
}

}  // namespace pattn

}  // namespace infllm2
