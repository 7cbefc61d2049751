// Work division of the attention of a chunk of new tokens over the paged latent cache.
//
// The query rows of a sequence, (token, head) pairs with the head running fastest, are cut into
// tiles of `tile_rows` rows; a tile attends to the keys its last row sees.  The list of all
// tiles' key blocks (block_keys keys each) is cut into `parts` ranges of equal cost, one for each
// resident CTA (pair): few rows over long caches spread over the machine (split-KV), many rows
// stay whole.  A range may end inside a tile; the parts of such a tile write normalised partial
// results with their log-sum-exp, which combine_kernel merges in the order of the parts, so the
// result does not depend on timing.
//
// Cost of a tile, in units of the kernel's choice: its start-up (query load, drained pipeline,
// write-back) and its key blocks.
#pragma once
#include "packed.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace chunk {

constexpr int kPage = 64, kRow = 576, kDc = 512;
constexpr int kPlanThreads = 1024;

// Plan in the workspace, written by plan_kernel.
struct Plan {
  int32_t* base;
  int B, max_tiles, max_parts;
  __host__ __device__ static size_t words(int64_t B, int64_t max_tiles, int64_t max_parts) {
    return static_cast<size_t>(4 + 2 * (max_tiles + 1) + (B + 1) + max_tiles + 2 * (max_parts + 1));
  }
  __host__ __device__ int32_t* header() const { return base; }  // tiles, parts
  // virtual start of each tile (int64), then one past the last
  __host__ __device__ int64_t* vstart() const { return reinterpret_cast<int64_t*>(base + 4); }
  __host__ __device__ int32_t* seq_tile() const { return base + 4 + 2 * (max_tiles + 1); }
  __host__ __device__ int32_t* tile_seq() const { return seq_tile() + B + 1; }
  __host__ __device__ int32_t* part_tile() const { return tile_seq() + max_tiles; }
  __host__ __device__ int32_t* part_block() const { return part_tile() + max_parts + 1; }
};

// What a plan is made for.
struct Shape {
  int n_tokens, batch, n_heads, max_pages, tile_rows;
  int block_keys, block_cost, seg_cost;
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
  __device__ int blocks(const Shape& s) const {
    return (visible(rows - 1, s.n_heads) + s.block_keys - 1) / s.block_keys;
  }
};
__device__ __forceinline__ Tile tile_at(const Shape& s, const Plan& plan, int i) {
  Tile t;
  t.seq = plan.tile_seq()[i];
  const packed::Span sp = packed::span(s.cu, t.seq, s.n_tokens);
  t.row0 = (i - plan.seq_tile()[t.seq]) * s.tile_rows;
  t.rows = min(s.tile_rows, sp.size() * s.n_heads - t.row0);
  t.tok0 = sp.begin;
  t.len = clamped_len(s, t.seq);
  t.first = t.len - sp.size();
  return t;
}

__device__ inline int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int64_t before = (w > 0 ? warp_sums[w - 1] : 0) + x - v;
  *total = warp_sums[31];
  __syncthreads();
  return before;
}

// One block.  Tiles per sequence and their prefix, each tile's sequence and virtual start, and
// the place (tile, block) where each part begins.
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const Shape s, Plan plan, int parts_req, unsigned int* status) {
  __shared__ int64_t warp_sums[32];
  griddep_launch_dependents();
  griddep_wait();
  const int T = kPlanThreads, tid = threadIdx.x;
  const int64_t max_tiles = plan.max_tiles, least = s.seg_cost + s.block_cost;
  int64_t total;
  int n_tiles = 0;
  bool bad = false;
  for (int b0 = 0; b0 < s.batch; b0 += T) {
    const int b = b0 + tid;
    int n = 0;
    if (b < s.batch) {
      const int64_t rows =
          static_cast<int64_t>(packed::span(s.cu, b, s.n_tokens, &bad).size()) * s.n_heads;
      n = static_cast<int>((rows + s.tile_rows - 1) / s.tile_rows);
      const int len = s.seq_lens[b];
      bad |= len < 0 || len > s.max_pages * kPage;
    }
    const int64_t at = block_scan(n, warp_sums, &total) + n_tiles;
    if (b < s.batch) plan.seq_tile()[b] = static_cast<int>(min(at, max_tiles));
    // (spans that overlap, which only a malformed cu has, could need more tiles than there are)
    n_tiles = static_cast<int>(min(n_tiles + total, max_tiles));
  }
  if (bad) atomicOr(status, MLA_STATUS_BAD_LENGTH);
  if (tid == 0) plan.seq_tile()[s.batch] = n_tiles;
  __syncthreads();
  // each tile's sequence: the last one that starts at or before it and is not empty
  int64_t v = 0;
  for (int i0 = 0; i0 < n_tiles; i0 += T) {
    const int i = i0 + tid;
    int64_t cost = 0;
    if (i < n_tiles) {
      int lo = 0, hi = s.batch;  // seq_tile[lo] <= i < seq_tile[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (plan.seq_tile()[mid] <= i) lo = mid; else hi = mid;
      }
      plan.tile_seq()[i] = lo;
      cost = s.seg_cost + static_cast<int64_t>(s.block_cost) * tile_at(s, plan, i).blocks(s);
    }
    const int64_t at = block_scan(cost, warp_sums, &total) + v;
    if (i < n_tiles) plan.vstart()[i] = at;
    v += total;
  }
  if (tid == 0) plan.vstart()[n_tiles] = v;
  __syncthreads();
  // part c begins at virtual place floor(c V / C).  No part is worth less than a start-up and a
  // block, so no two of them begin at the same block.
  const int64_t V = v;
  const int64_t most = V / least;
  const int C = most < 1 ? 1 : most < parts_req ? static_cast<int>(most) : parts_req;
  for (int i = tid; i < n_tiles; i += T) {
    const int64_t v0 = plan.vstart()[i], v1 = plan.vstart()[i + 1];
    for (int64_t c = (v0 * C + V - 1) / V; c < C; ++c) {
      const int64_t u = c * V / C;
      if (u >= v1) break;
      if (u < v0) continue;
      plan.part_tile()[c] = i;
      plan.part_block()[c] =
          u - v0 > s.seg_cost ? static_cast<int>((u - v0 - s.seg_cost) / s.block_cost) : 0;
    }
  }
  for (int c = tid; c <= plan.max_parts; c += T)
    if (c >= (n_tiles > 0 ? C : 0)) {
      plan.part_tile()[c] = n_tiles;
      plan.part_block()[c] = 0;
    }
  if (tid == 0) {
    plan.header()[0] = n_tiles;
    plan.header()[1] = n_tiles > 0 ? C : 0;
  }
}

// The segments of part c: whole tiles, but for a first one that begins and a last one that ends
// inside its tile.  Tiles without a visible key come as segments of no blocks.
struct SegIter {
  const Shape* s;
  Plan plan;
  int i, b, i_end, b_end;  // next (tile, block), and where the part ends
  __device__ SegIter(const Shape& shape, const Plan& p, int c) : s(&shape), plan(p) {
    const bool in = c < p.header()[1];
    i = in ? p.part_tile()[c] : 0;
    b = in ? p.part_block()[c] : 0;
    i_end = in ? p.part_tile()[c + 1] : 0;
    b_end = in ? p.part_block()[c + 1] : 0;
  }
  __device__ bool next(Tile& t, int& tile, int& b0, int& b1, int& blocks) {
    if (i > i_end || (i == i_end && b >= b_end)) return false;
    tile = i;
    t = tile_at(*s, plan, i);
    blocks = t.blocks(*s);
    b0 = b;
    b1 = i < i_end ? blocks : b_end;
    ++i;
    b = 0;
    return true;
  }
};

// Partial results: part c's tile that it enters in the middle goes to slot 2c, the one that it
// begins and does not finish to slot 2c + 1.  part_o [2 C][tile_rows][512], part_lse alike.
__device__ __forceinline__ int partial_slot(int c, int b0) { return 2 * c + (b0 == 0 ? 1 : 0); }

constexpr int kCombineWarps = 8;

template <typename O> __device__ __forceinline__ void store4(O* p, float4 v);
template <> __device__ __forceinline__ void store4<float>(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// grid (parts - 1, tile_rows / kCombineWarps): the boundary of parts x and x + 1, if it is the
// first one inside its tile.  One warp per row; lane l holds columns 4 (l + 32 k) ... + 3.
template <typename O>
__global__ void __launch_bounds__(32 * kCombineWarps)
    combine_kernel(const Shape s, Plan plan, const float* __restrict__ part_o,
                   const float* __restrict__ part_lse, O* __restrict__ o, float* __restrict__ lse) {
  griddep_launch_dependents();
  griddep_wait();
  const int C = plan.header()[1], c = blockIdx.x + 1;
  if (c >= C || plan.part_block()[c] == 0) return;
  const int i = plan.part_tile()[c];
  if (plan.part_tile()[c - 1] == i && plan.part_block()[c - 1] > 0) return;  // not the first
  const Tile t = tile_at(s, plan, i);
  const int r = blockIdx.y * kCombineWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= t.rows) return;
  const float NEG_INF = -__int_as_float(0x7f800000);
  // contributors: slot 2 (c - 1) + 1, then 2 k for k = c ... last
  int last = c;
  while (last + 1 < C && plan.part_tile()[last + 1] == i && plan.part_block()[last + 1] > 0) ++last;
  const auto slot = [&](int k) { return k < c ? 2 * k + 1 : 2 * k; };
  float m = NEG_INF;
  for (int k = c - 1 + lane; k <= last; k += 32)
    m = fmaxf(m, part_lse[static_cast<size_t>(slot(k)) * s.tile_rows + r]);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  float tot = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = c - 1; k <= last; ++k) {
    const size_t at = static_cast<size_t>(slot(k)) * s.tile_rows + r;
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
  const int64_t row = static_cast<int64_t>(t.tok0) * s.n_heads + t.row0 + r;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    store4(o + row * kDc + 4 * (lane + 32 * q),
           make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv));
  if (lane == 0 && lse) lse[row] = tot == 0.f ? NEG_INF : m + logf(tot);
}

}  // namespace chunk
}  // namespace mla
