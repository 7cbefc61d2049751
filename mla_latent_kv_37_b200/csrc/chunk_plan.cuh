// Work division of the attention of a chunk of new tokens over the paged latent cache.
//
// The query rows of a sequence, (token, head) pairs with the head running fastest, are cut into
// tiles of 2^tile_shift rows; a tile attends to the keys its last row sees.  The list of all
// tiles' key blocks (2^block_shift keys each) is cut into `parts` ranges of equal cost, one for each
// resident CTA (pair): few rows over long caches spread over the machine (split-KV), many rows
// stay whole.  A range may end inside a tile; the parts of such a tile write normalised partial
// results with their log-sum-exp, which a second kernel merges in the order of the parts, so the
// result does not depend on timing.
//
// Teams.  Where all sequences have the same number w of tiles (a few proposed tokens each, the usual
// case), w parts make a team that takes a range of (sequence, block) pairs together, part k of it
// tile k: the tiles of a sequence then read the same keys at the same time, and the cache comes
// from HBM once.  With ranges of one list of tiles they read them at w different times, and 32 x 4
// tokens over 225 MB of rows read 779 MB.  Not for caches that stay in L2 anyway, nor where the
// parts are not nearly a multiple of w.  One sequence with another number of tiles turns teams off for
// all: 31 x 4 tokens and one of 5 take 207 ... 248 us, 32 x 4 take 193 ... 211.
//
// Every block of the attention kernel finds its own range, a tile a thread and two passes where the
// tiles are more than the threads: a kernel of its own for the plan took 6 us before the first load.
//
// Cost of a tile, in units of the kernel's choice: its start-up (query load, drained pipeline,
// write-back) and its key blocks.
#pragma once
#include "packed.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace chunk {

constexpr int kPage = 64, kRow = 576, kDc = 512;
// What the work is.
struct Shape {
  int n_tokens, batch, n_heads, max_pages;
  int tile_shift, block_shift;  // 2^ rows of a tile, keys of a block
  int cost_shift, seg_cost, least;  // 2^ cost of a block; cost of a segment's start and end; no
                                    // part is worth less than `least` (but for a lone one)
  const int32_t* cu;
  const int32_t* seq_lens;
};

// A sequence's keys, clamped to what its page table can hold.
__device__ __forceinline__ int clamped_len(const Shape& s, int b) {
  return min(max(s.seq_lens[b], 0), s.max_pages * kPage);
}

// One tile: rows [row0, row0 + rows) of its sequence's (token, head) rows; row r sees the first
// `first + r / n_heads + 1` keys (none if that is <= 0).
struct Tile {
  int seq, row0, rows, tok0, first, len;
  __device__ int visible(int r, int n_heads) const {
    return min(max(first + (row0 + r) / n_heads + 1, 0), len);
  }
  __device__ int blocks(const Shape& s) const {  // (the sum may pass 2^31, by less than a block)
    return static_cast<int>(
        (static_cast<unsigned>(visible(rows - 1, s.n_heads)) + (1u << s.block_shift) - 1) >> s.block_shift);
  }
};
// Tiles of a sequence, and its k-th one.
__device__ __forceinline__ int tiles_of(const Shape& s, int tokens) {
  const int64_t rows = static_cast<int64_t>(tokens) * s.n_heads;
  return static_cast<int>((rows + (1 << s.tile_shift) - 1) >> s.tile_shift);
}
__device__ __forceinline__ Tile tile_at(const Shape& s, int seq, int k) {
  Tile t;
  t.seq = seq;
  const packed::Span sp = packed::span(s.cu, seq, s.n_tokens);
  t.row0 = k << s.tile_shift;
  t.rows = min(1 << s.tile_shift, sp.size() * s.n_heads - t.row0);
  t.tok0 = sp.begin;
  t.len = clamped_len(s, seq);
  t.first = t.len - sp.size();
  return t;
}

// A place in the list of blocks: block `block` of tile `k` of sequence `seq`, entry `index` of the
// list of tiles (of teams: of sequences; k is the part's own).
struct Place {
  int seq, k, block, index;
};
// A part's range [from, to), and the parts of its team.
struct Range {
  Place from, to;
  int team;
  bool any;
};
// Where a part begins, for the merge: index < 0 if it has nothing.  row: the first of the tile's
// rows among all (token, head) rows.  The range goes on in part + team.
struct PartStart {
  int32_t index, block, rows, team;
  int64_t row, pad;
};

// Exclusive sum over the block's threads (whole warps, at most 32).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  int64_t before = x - v, sum = 0;
  for (int i = 0; i < warps; ++i) {
    const int64_t y = warp_sums[i];
    if (i < w) before += y;
    sum += y;
  }
  __syncthreads();
  *total = sum;
  return before;
}

constexpr int kMaxPlanThreads = 256;

// Scratch in shared memory of find_part.
struct Scratch {
  int64_t warp_sums[32];
  Place found[2];
  int first[kMaxPlanThreads], size[kMaxPlanThreads], len[kMaxPlanThreads];  // of a round of
                                                                            // sequences
};

// A tile is split into about this many parts at most: the merge reads them one behind the other.
constexpr int kMaxSplit = 24;
// Caches of fewer rows stay in L2 (37 MB of 126) whatever the order.
constexpr int64_t kTeamKeys = 32768;

// The range of part `part` of `parts`.  All threads of the block.
__device__ inline Range find_part(const Shape& s, int parts, int part, Scratch* sc,
                                  unsigned int* status) {
  const int T = blockDim.x, tid = threadIdx.x;
  bool bad = false;
  // this thread's sequence of a round, to the scratch
  const auto load_round = [&](int b0) {
    const int b = b0 + tid;
    int size = 0;
    if (b < s.batch) {
      const int len = s.seq_lens[b];
      size = packed::span(s.cu, b, s.n_tokens, &bad).size();
      sc->len[tid] = min(max(len, 0), s.max_pages * kPage);
      bad |= len < 0 || len > s.max_pages * kPage;
    }
    sc->size[tid] = size;
    __syncthreads();
  };
  load_round(0);
  // the parts of a team: as many as each sequence has tiles, or 1
  int w = tiles_of(s, sc->size[0]);
  if (w < 2 || parts / w * w * 16 < parts * 15) w = 1;
  if (w > 1) {
    int64_t keys = 0, total;
    for (int b0 = 0; w > 1 && b0 < s.batch; b0 += T) {
      if (b0 > 0) load_round(b0);
      const bool in = b0 + tid < s.batch;
      if (in) keys += sc->len[tid];
      if (!__syncthreads_and(!in || tiles_of(s, sc->size[tid]) == w)) w = 1;
    }
    block_scan(keys, sc->warp_sums, &total);
    if (total < kTeamKeys) w = 1;
  }
  const int rank = part / w, ranks = parts / w;
  // f(place of an entry, its cost or 0 without one), a round of T entries at a time; their number
  const auto each_round = [&](auto&& f) {
    int base = 0;
    for (int b0 = 0; b0 < s.batch; b0 += T) {
      if (s.batch > T) {
        __syncthreads();
        load_round(b0);
      }
      const int n = b0 + tid < s.batch ? (w > 1 ? 1 : tiles_of(s, sc->size[tid])) : 0;
      int64_t total;
      sc->first[tid] = static_cast<int>(block_scan(n, sc->warp_sums, &total));
      __syncthreads();
      const int tiles = static_cast<int>(total);
      for (int i0 = 0; i0 < tiles; i0 += T) {
        const int i = i0 + tid;
        Place at{0, 0, 0, base + i};
        int64_t cost = 0;
        if (i < tiles) {
          int lo = 0, hi = T;  // the last sequence that begins at or before tile i is not empty
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sc->first[mid] <= i) lo = mid; else hi = mid;
          }
          at.seq = b0 + lo;
          at.k = i - sc->first[lo];
          Tile t;
          t.row0 = (w > 1 ? w - 1 : at.k) << s.tile_shift;  // a team's last tile has the most keys
          t.rows = min(1 << s.tile_shift, sc->size[lo] * s.n_heads - t.row0);
          t.len = sc->len[lo];
          t.first = t.len - sc->size[lo];
          cost = s.seg_cost + (static_cast<int64_t>(t.blocks(s)) << s.cost_shift);
        }
        f(at, cost);
      }
      __syncthreads();
      base += tiles;
    }
    return base;
  };
  int rounds = 0;
  int64_t V = 0, mine_v = 0, mine_cost = 0;
  Place mine{};
  const int entries = each_round([&](const Place& at, int64_t cost) {
    int64_t total;
    mine = at;
    mine_cost = cost;
    mine_v = block_scan(cost, sc->warp_sums, &total) + V;
    V += total;
    ++rounds;
  });
  if (bad && part == 0) atomicOr(status, MLA_STATUS_BAD_LENGTH);
  // part c begins at place floor(c V / C).  `least` is a block's cost or more, so no two begin at the same block
  // past a tile's first.
  const int most = min(static_cast<int64_t>(ranks), kMaxSplit * static_cast<int64_t>(entries));
  const int C = V >= static_cast<int64_t>(most) * s.least
                    ? most
                    : max(static_cast<int>(V) / s.least, V > 0);
  Range r{};
  r.team = w;
  if (rank >= C) return r;
  const bool small = V <= 0xffffffffll;  // (a 64-bit division takes a few hundred clocks)
  const int64_t q = small ? static_cast<uint32_t>(V) / static_cast<uint32_t>(C) : V / C;
  const uint32_t rest = static_cast<uint32_t>(V - q * C);  // c rest / C: c, rest < C <= 65536
  const auto begin = [&](uint32_t c) { return c * q + c * rest / static_cast<uint32_t>(C); };
  const int64_t u[2] = {begin(rank), rank + 1 == C ? V : begin(rank + 1)};
  const auto locate = [&](const Place& at, int64_t v0, int64_t cost) {  // (cost 0: no tile)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (v0 <= u[e] && u[e] < v0 + cost) {
        sc->found[e] = at;
        if (u[e] - v0 > s.seg_cost)
          sc->found[e].block = static_cast<int>((u[e] - v0 - s.seg_cost) >> s.cost_shift);
      }
  };
  if (tid == 0) sc->found[1] = Place{s.batch, 0, 0, 0x7fffffff};  // behind the last tile
  __syncthreads();
  if (rounds == 1) {
    locate(mine, mine_v, mine_cost);
  } else {
    int64_t before = 0;
    each_round([&](const Place& at, int64_t cost) {
      int64_t total;
      const int64_t v0 = block_scan(cost, sc->warp_sums, &total) + before;
      before += total;
      locate(at, v0, cost);
    });
  }
  __syncthreads();
  r.any = true;
  r.from = sc->found[0];
  r.to = sc->found[1];
  if (w > 1) r.from.k = part % w;
  return r;
}

// The segments of a range: whole tiles, but for a first one that begins and a last one that ends
// inside its tile.  Tiles without a visible key come as segments of no blocks.
struct Segment {
  Tile t;
  int b0, b1;   // blocks (of a team, only those that the tile has)
  bool inside;  // begins inside its tile
  bool split;   // begins or ends inside its tile
};
struct SegIter {
  const Shape* s;
  Place at, to;
  int team;
  __device__ SegIter(const Shape& shape, const Range& r)
      : s(&shape), at(r.from), to(r.any ? r.to : r.from), team(r.team) {}
  __device__ __forceinline__ bool next(Segment& g) {
    if (team > 1) {
      if (at.seq > to.seq || (at.seq == to.seq && at.block >= to.block)) return false;
    } else {
      const auto behind = [&]() {
        return at.seq > to.seq ||
               (at.seq == to.seq && (at.k > to.k || (at.k == to.k && at.block >= to.block)));
      };
      if (behind()) return false;
      while (at.k >= tiles_of(*s, packed::span(s->cu, at.seq, s->n_tokens).size())) {
        if (++at.seq > to.seq || at.seq >= s->batch) return false;  // the next that has tiles
        at.k = 0;
      }
      if (behind()) return false;
    }
    const bool last = at.seq == to.seq && (team > 1 || at.k == to.k);
    g.t = tile_at(*s, at.seq, at.k);
    const int blocks = g.t.blocks(*s);
    g.inside = at.block > 0;
    g.split = g.inside || last;
    g.b0 = min(at.block, blocks);
    g.b1 = last ? min(to.block, blocks) : blocks;
    if (team > 1) ++at.seq; else ++at.k;
    at.block = 0;
    return true;
  }
};

// The merge's record of a part, by one thread.
__device__ __forceinline__ void write_start(const Shape& s, const Range& r, PartStart* out) {
  PartStart p{-1, 0, 0, r.team, 0, 0};
  if (r.any) {
    const Tile t = tile_at(s, r.from.seq, r.from.k);
    p = PartStart{r.from.index, r.from.block, t.rows, r.team,
                  static_cast<int64_t>(t.tok0) * s.n_heads + t.row0, 0};
  }
  *out = p;
}

// Partial results: part c's tile that it enters in the middle goes to slot 2c, the one that it
// begins and does not finish to slot 2c + 1.  part_lse [2 C][tile_rows]; part_o [2 C][tile_rows][512],
// or, where a thread has a row (kByColumn), [2 C][128][tile_rows][4], so that the threads of a warp
// write 512 bytes side by side.
__device__ __forceinline__ int partial_slot(int c, bool inside) { return 2 * c + (inside ? 0 : 1); }

constexpr int kCombineThreads = 256;

template <typename O> __device__ __forceinline__ void store4(O* p, float4 v);
template <> __device__ __forceinline__ void store4<float>(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The parts of a tile that is split, where part c is the first that begins inside it: the slots are
// 2 (c - team) + 1, then 2 k for k = c, c + team ... last.
struct Split {
  PartStart start;
  int c, last, team;
  // One warp: a lane looks at one of the next 32 parts, since one after the other a dozen loads'
  // latencies would add up.
  __device__ bool find(const PartStart* starts, int parts, int part) {
    start = starts[part];
    c = last = part;
    team = start.team;
    if (start.index < 0 || start.block == 0) return false;
    const int lane = threadIdx.x & 31;
    const auto inside = [&](int k) {
      return k < parts && starts[k].index == start.index && starts[k].block > 0;
    };
    if (inside(part - team)) return false;
    for (int n = 32; n == 32; last += n * team) {
      const unsigned no = ~__ballot_sync(0xffffffffu, inside(last + (lane + 1) * team));
      n = no ? __ffs(no) - 1 : 32;
    }
    return true;
  }
  __device__ int count() const { return (last - c) / team + 2; }
  __device__ int slot(int i) const { return i == 0 ? 2 * (c - team) + 1 : 2 * (c + (i - 1) * team); }
};

// Row-major partial results: grid (parts - 1, tile_rows / 8), one warp per row; lane l holds
// columns 4 (l + 32 k) ... + 3.
template <typename O>
__global__ void __launch_bounds__(kCombineThreads)
    combine_rows_kernel(int parts, int tile_rows, const PartStart* starts,
                        const float* part_o, const float* part_lse,
                        O* o, float* lse) {
  griddep_launch_dependents();
  griddep_wait();
  Split sp;
  if (!sp.find(starts, parts, blockIdx.x + 1)) return;
  const PartStart& t = sp.start;
  const int n = sp.count();
  const int r = blockIdx.y * (kCombineThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= t.rows) return;
  const float NEG_INF = -__int_as_float(0x7f800000);
  float m = NEG_INF;
  for (int k = lane; k < n; k += 32)
    m = fmaxf(m, part_lse[static_cast<size_t>(sp.slot(k)) * tile_rows + r]);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  float tot = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const size_t at = static_cast<size_t>(sp.slot(k)) * tile_rows + r;
    const float l = part_lse[at];
    const float w = l == NEG_INF ? 0.f : expf(l - m);
    tot += w;
    const float4* src = reinterpret_cast<const float4*>(part_o + at * kDc);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 x = src[lane + 32 * q];
      acc[q].x += w * x.x;
      acc[q].y += w * x.y;
      acc[q].z += w * x.z;
      acc[q].w += w * x.w;
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;  // (a NaN stays one)
  const int64_t row = t.row + r;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    store4(o + row * kDc + 4 * (lane + 32 * q),
           make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv));
  if (lane == 0 && lse) lse[row] = tot == 0.f ? NEG_INF : m + logf(tot);
}

// Partial results by column groups: grid (parts - 1, tile_rows / 32, 4), lane = row, warp w has the
// columns 128 z + 4 (w + 8 k) ... + 3, k < 4.  The rows go out through shared memory.
template <typename O>
__global__ void __launch_bounds__(kCombineThreads)
    combine_columns_kernel(int parts, int tile_rows, const PartStart* starts,
                           const float* part_o, const float* part_lse,
                           O* o, float* lse) {
  __shared__ float4 turn[32][33];
  griddep_launch_dependents();
  griddep_wait();
  Split sp;
  if (!sp.find(starts, parts, blockIdx.x + 1)) return;
  const PartStart& t = sp.start;
  const int n = sp.count();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.y * 32, r = r0 + lane;
  if (r0 >= t.rows) return;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const auto part_l = [&](int k) {
    return part_lse[static_cast<size_t>(sp.slot(k)) * tile_rows + r];
  };
  float m = NEG_INF;  // (rows past the tile's last hold what the attention left there: -inf and 0)
#pragma unroll 4
  for (int k = 0; k < n; ++k) m = fmaxf(m, part_l(k));
  float tot = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float l = part_l(k), w = l == NEG_INF ? 0.f : expf(l - m);
    tot += w;
    const float4* src =
        reinterpret_cast<const float4*>(part_o) +
        (static_cast<size_t>(sp.slot(k)) * (kDc / 4) + 32 * blockIdx.z + warp) * tile_rows + r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 x = src[static_cast<size_t>(8 * q) * tile_rows];
      acc[q].x += w * x.x;
      acc[q].y += w * x.y;
      acc[q].z += w * x.z;
      acc[q].w += w * x.w;
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;  // (a NaN stays one)
#pragma unroll
  for (int q = 0; q < 4; ++q)
    turn[lane][warp + 8 * q] =
        make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv);
  __syncthreads();
#pragma unroll
  for (int i = warp; i < 32; i += kCombineThreads / 32)
    if (r0 + i < t.rows)
      store4(o + (t.row + r0 + i) * kDc + 128 * blockIdx.z + 4 * lane, turn[i][lane]);
  if (blockIdx.z == 0 && warp == 0 && r < t.rows && lse)
    lse[t.row + r] = tot == 0.f ? NEG_INF : m + logf(tot);
}

}  // namespace chunk
}  // namespace mla
