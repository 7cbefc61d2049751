// Packed batches of several new tokens per sequence: tokens of all sequences one behind the
// other, sequence b at [cu[b], cu[b + 1]).  cu is the caller's device array, so every bound read
// from it is clamped to the arrays' extent before it is used as an index: a malformed array
// (decreasing, or past the last token) gives wrong rows and MLA_STATUS_BAD_LENGTH, never an
// access out of range.
#pragma once
#include <cstdint>

#include "mla_status.cuh"

namespace mla {
namespace packed {

struct Span {
  int begin, end;
  __device__ int size() const { return end - begin; }
};

// Sequence b's tokens, clamped to [0, n_tokens).  *bad is set where the clamp changed something.
__device__ __forceinline__ Span span(const int32_t* cu, int b, int n_tokens, bool* bad = nullptr) {
  const int c0 = cu[b], c1 = cu[b + 1];
  const int s0 = min(max(c0, 0), n_tokens), s1 = min(max(c1, s0), n_tokens);
  if (bad && (s0 != c0 || s1 != c1)) *bad = true;
  return {s0, s1};
}

// Reports offsets that decrease or pass n_tokens.  All threads of one block of a grid, which looks at all
// sequences: the others look only as far as their own (right behind that look-up the first of these
// loads are in L1).
__device__ __forceinline__ void check_offsets(const int32_t* cu, int B, int n_tokens,
                                              unsigned int* status) {
  bool bad = false;
  for (int b = threadIdx.x; b < B; b += blockDim.x) (void)span(cu, b, n_tokens, &bad);
  if (bad) atomicOr(status, MLA_STATUS_BAD_LENGTH);
}

// The sequence of token t: the number of entries cu[1 .. B] that are <= t (B if the token lies
// behind the last sequence).  A 32-way search by one warp: ceil(log32 B) dependent reads.
__device__ __forceinline__ int warp_sequence_of(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int last = min((lane + 1) * step, n);  // this lane's slice ends at lo + last
    const bool le = lane * step < n && cu[lo + last] <= t;
    const int full = __popc(__ballot_sync(0xffffffffu, le));  // whole slices of entries <= t
    const int skip = min(full * step, n);
    if (step == 1) return lo + skip;
    lo += skip;
    n = min(step - 1, n - skip);  // the next slice's last entry is > t (or there is no slice)
    if (n < 0) n = 0;
  }
  return lo;
}

// Tile `tile` of the list of all sequences' tiles (ceil(size * rows_per_token / tile_rows) tiles
// each): its sequence and its index there; false behind the last.  One warp, 32 sequences a step.
// Within a sequence the caller may number its tiles in either direction.
__device__ __forceinline__ bool warp_find_tile(const int32_t* cu, int B, int n_tokens,
                                               int tile_rows, int tile, int& seq, int& index,
                                               int& count, Span& s) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < B; b0 += 32) {
    Span mine{0, 0};
    if (b0 + lane < B) mine = span(cu, b0 + lane, n_tokens);
    const int n = (mine.size() + tile_rows - 1) / tile_rows;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, tile < x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      seq = b0 + l;
      count = __shfl_sync(0xffffffffu, n, l);
      index = tile - (__shfl_sync(0xffffffffu, x, l) - count);
      s.begin = __shfl_sync(0xffffffffu, mine.begin, l);
      s.end = __shfl_sync(0xffffffffu, mine.end, l);
      return true;
    }
    tile -= __shfl_sync(0xffffffffu, x, 31);
  }
  return false;
}

}  // namespace packed
}  // namespace mla
