// Attention of several query rows on the SIMT cores with fp32 products (the fp32 configuration:
// the tensor cores have no mode accurate to 1e-5), for whole packed prompts (192-wide keys,
// 128-wide values) and for a chunk of new tokens over the paged latent cache (576 and 512).
//
// A block of 8 warps takes 64 query rows and walks over the keys 64 at a time with an online
// softmax; warp w owns rows 8w ... 8w + 7, so a row's scores, maximum and sum stay inside one
// warp.  Per 64 keys: S = Q K^T in slices of 64 columns (a thread has 8 rows x 2 keys, so 64 FMAs
// follow 16 shared-memory wavefronts of loads), P to shared memory, O += P V in slices of keys
// with O in registers (8 rows x DV / 32 columns a thread).
//
// Bound by the FMA pipe: 2 (DQ + DV) flops per row and key at 128 FMAs a clock and SM.
#pragma once
#include "chunk_plan.cuh"

namespace mla {
namespace simt {

constexpr int kThreads = 256, kRows = 64, kKeys = 64, kSlice = 64;
constexpr int kKPad = kSlice + 4;  // row stride of a key slice: 16-byte loads of 8 rows in a
                                   // phase fall into different banks

template <int DQ, int DV> struct Layout {
  static constexpr int kVKeys = 8192 / DV;  // keys of one value slice: 32 KB
  static constexpr int kQ = 0;                                // [kRows][DQ]
  static constexpr int kK = kQ + kRows * DQ;                  // [kKeys][kKPad]
  static constexpr int kV = kK + kKeys * kKPad;               // [kVKeys][DV]
  static constexpr int kP = kV + kVKeys * DV;                 // [8 warps][kKeys][8 rows]
  static constexpr size_t kBytes = (kP + kKeys * kRows) * sizeof(float);
};

__device__ __forceinline__ float4 load4(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}

// One segment: rows r of the tile against keys [j0, j1).  Src gives, in elements of float:
//   const float* q(r, d): 4 columns from d of row r's query (r < rows);
//   const float* k(j, d), v(j, d): the same of key j (j < j1);  int visible(r): keys row r sees.
// On return m[i], l[i] and o[i][...] hold row 8 warp + i's maximum (log2 units), sum and
// unnormalised output columns 4 (lane + 32 k) + ....
template <int DQ, int DV, class Src>
__device__ __forceinline__ void segment(const Src& src, float* smem, int rows, int j0, int j1,
                                        float scale_log2, float (&m)[8], float (&l)[8],
                                        float (&o)[8][DV / 32]) {
  using L = Layout<DQ, DV>;
  float *sQ = smem + L::kQ, *sK = smem + L::kK, *sV = smem + L::kV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = 8 * warp;
  float* sP = smem + L::kP + warp * kKeys * 8;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();  // the previous segment has read the query
  for (int i = threadIdx.x; i < kRows * DQ / 4; i += kThreads) {
    const int r = i / (DQ / 4), d = 4 * (i % (DQ / 4));
    *reinterpret_cast<float4*>(sQ + r * DQ + d) = r < rows ? load4(src.q(r, d)) : zero;
  }
  int vis[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    vis[i] = r0 + i < rows ? src.visible(r0 + i) : 0;
    m[i] = NEG_INF;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < DV / 32; ++k) o[i][k] = 0.f;
  }
  for (int jb = j0; jb < j1; jb += kKeys) {
    const int nk = min(kKeys, j1 - jb);
    float s[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i][0] = s[i][1] = 0.f;
    for (int d0 = 0; d0 < DQ; d0 += kSlice) {
      __syncthreads();
#pragma unroll
      for (int i = threadIdx.x; i < kKeys * kSlice / 4; i += kThreads) {
        const int j = i / (kSlice / 4), d = 4 * (i % (kSlice / 4));
        *reinterpret_cast<float4*>(sK + j * kKPad + d) =
            j < nk ? load4(src.k(jb + j, d0 + d)) : zero;
      }
      __syncthreads();
#pragma unroll 4
      for (int d = 0; d < kSlice; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(sK + lane * kKPad + d);
        const float4 k1 = *reinterpret_cast<const float4*>(sK + (lane + 32) * kKPad + d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(sQ + (r0 + i) * DQ + d0 + d);
          s[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[i][0]))));
          s[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[i][1]))));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s0 = jb + lane < vis[i] ? s[i][0] * scale_log2 : NEG_INF;
      const float s1 = jb + lane + 32 < vis[i] ? s[i][1] * scale_log2 : NEG_INF;
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      mx = fmaxf(mx, m[i]);
      const float ref = mx == NEG_INF ? 0.f : mx;  // no key seen yet: every weight is 0
      const float alpha = exp2f(m[i] - ref);
      m[i] = mx;
      const float p0 = exp2f(s0 - ref), p1 = exp2f(s1 - ref);
      l[i] = l[i] * alpha + p0 + p1;  // this lane's share of the row's sum
#pragma unroll
      for (int k = 0; k < DV / 32; ++k) o[i][k] *= alpha;
      sP[lane * 8 + i] = p0;
      sP[(lane + 32) * 8 + i] = p1;
    }
    __syncwarp();
    for (int v0 = 0; v0 < nk; v0 += L::kVKeys) {
      __syncthreads();
#pragma unroll 4
      for (int i = threadIdx.x; i < L::kVKeys * DV / 4; i += kThreads) {
        const int j = v0 + i / (DV / 4), d = 4 * (i % (DV / 4));
        *reinterpret_cast<float4*>(sV + 4 * i) = j < nk ? load4(src.v(jb + j, d)) : zero;
      }
      __syncthreads();
      const int jn = min(L::kVKeys, nk - v0);
#pragma unroll 2
      for (int j = 0; j < jn; ++j) {
        const float4 pa = *reinterpret_cast<const float4*>(sP + (v0 + j) * 8);
        const float4 pb = *reinterpret_cast<const float4*>(sP + (v0 + j) * 8 + 4);
        const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int k = 0; k < DV / 128; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(sV + j * DV + 4 * (lane + 32 * k));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][4 * k] = fmaf(pr[i], v.x, o[i][4 * k]);
            o[i][4 * k + 1] = fmaf(pr[i], v.y, o[i][4 * k + 1]);
            o[i][4 * k + 2] = fmaf(pr[i], v.z, o[i][4 * k + 2]);
            o[i][4 * k + 3] = fmaf(pr[i], v.w, o[i][4 * k + 3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
}

constexpr float kLn2 = 0.69314718055994531f;

// ------------------------------------------------------------------------------------------
// whole packed prompts
// ------------------------------------------------------------------------------------------
struct PromptParams {
  int n_tokens, batch, n_heads, n_kv_heads;
  const int32_t* cu;
  const void *q, *k_nope, *k_rope, *v;
  int64_t q_tok, q_head, k_tok, k_head, kr_tok, v_tok, v_head;  // elements
  float scale_log2;
  void* o;
  float* lse;
  unsigned int* status;
};

struct PromptSrc {
  const float *q0, *k0, *kr0, *v0;
  int64_t q_tok, k_tok, kr_tok, v_tok;
  int first;
  __device__ const float* q(int r, int d) const { return q0 + r * q_tok + d; }
  __device__ const float* k(int j, int d) const {
    return d < 128 ? k0 + j * k_tok + d : kr0 + j * kr_tok + (d - 128);
  }
  __device__ const float* v(int j, int d) const { return v0 + j * v_tok + d; }
  __device__ int visible(int r) const { return first + r + 1; }
};

// grid (tiles, heads); a sequence's tiles run from its last rows (the longest) to its first
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PromptParams p) {
  extern __shared__ __align__(16) float smem[];
  griddep_launch_dependents();
  griddep_wait();
  int seq, index, count;
  packed::Span s;
  bool bad = false;
  const bool there = packed::warp_find_tile(p.cu, p.batch, p.n_tokens, kRows, blockIdx.x, seq,
                                            index, count, s, &bad);
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, MLA_STATUS_BAD_LENGTH);
  if (!there) return;
  const int first = (count - 1 - index) * kRows, rows = min(kRows, s.size() - first);
  const int h = blockIdx.y, hk = h / (p.n_heads / p.n_kv_heads);
  const int64_t t0 = s.begin;
  const PromptSrc src{static_cast<const float*>(p.q) + (t0 + first) * p.q_tok + h * p.q_head,
                      static_cast<const float*>(p.k_nope) + t0 * p.k_tok + hk * p.k_head,
                      static_cast<const float*>(p.k_rope) + t0 * p.kr_tok,
                      static_cast<const float*>(p.v) + t0 * p.v_tok + hk * p.v_head,
                      p.q_tok, p.k_tok, p.kr_tok, p.v_tok, first};
  float m[8], l[8], o[8][4];
  segment<192, 128>(src, smem, rows, 0, first + rows, p.scale_log2, m, l, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 8 * warp + i;
    if (r >= rows) break;
    const int64_t row = (t0 + first + r) * p.n_heads + h;
    const float inv = 1.f / l[i];
    chunk::store4(static_cast<float*>(p.o) + row * 128 + 4 * lane,
                  make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv));
    if (lane == 0 && p.lse) p.lse[row] = (m[i] + log2f(l[i])) * kLn2;
  }
}

// ------------------------------------------------------------------------------------------
// a chunk of new tokens over the paged latent cache
// ------------------------------------------------------------------------------------------
struct ChunkParams {
  chunk::Shape shape;  // tile_rows = kRows
  chunk::Plan plan;
  int num_pages;
  const void* q_cat;
  const void* pool;
  const int32_t* page_table;
  float scale_log2;
  void* o;
  float* lse;
  float* part_o;
  float* part_lse;
  unsigned int* status;
};

struct ChunkSrc {
  const float* q0;
  const float* pool;
  const int32_t* pages;
  int num_pages, n_heads;
  chunk::Tile t;
  __device__ const float* q(int r, int d) const { return q0 + static_cast<int64_t>(r) * 576 + d; }
  __device__ const float* k(int j, int d) const {
    const int pg = pages[j / chunk::kPage];
    const int64_t at = pg < 0 || pg >= num_pages ? 0 : pg;
    return pool + (at * chunk::kPage + j % chunk::kPage) * chunk::kRow + d;
  }
  __device__ const float* v(int j, int d) const { return k(j, d); }
  __device__ int visible(int r) const { return t.visible(r, n_heads); }
};

__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) float smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = p.shape.n_heads;
  chunk::SegIter it(p.shape, p.plan, blockIdx.x);
  chunk::Tile t;
  int tile, b0, b1, blocks;
  while (it.next(t, tile, b0, b1, blocks)) {
    const int j0 = b0 * chunk::kBlock;
    const int j1 = min(b1 * chunk::kBlock, t.visible(t.rows - 1, H));
    const int64_t row0 = static_cast<int64_t>(t.tok0) * H + t.row0;
    const ChunkSrc src{static_cast<const float*>(p.q_cat) + row0 * chunk::kRow,
                       static_cast<const float*>(p.pool),
                       p.page_table + static_cast<int64_t>(t.seq) * p.shape.max_pages,
                       p.num_pages, H, t};
    for (int pg = j0 / chunk::kPage + threadIdx.x; pg * chunk::kPage < j1; pg += kThreads)
      if (src.pages[pg] < 0 || src.pages[pg] >= p.num_pages)
        atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    float m[8], l[8], o[8][16];
    segment<576, 512>(src, smem, t.rows, j0, j1, p.scale_log2, m, l, o);
    const bool whole = b0 == 0 && b1 == blocks;
    const int slot = chunk::partial_slot(blockIdx.x, b0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * warp + i;
      if (r >= t.rows) break;
      const int64_t row = whole ? row0 + r : static_cast<int64_t>(slot) * kRows + r;
      float* dst = (whole ? static_cast<float*>(p.o) : p.part_o) + row * chunk::kDc;
      float* dst_lse = whole ? p.lse : p.part_lse;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // (a NaN stays one)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        chunk::store4(dst + 4 * (lane + 32 * k),
                      make_float4(o[i][4 * k] * inv, o[i][4 * k + 1] * inv,
                                  o[i][4 * k + 2] * inv, o[i][4 * k + 3] * inv));
      if (lane == 0 && dst_lse)
        dst_lse[row] = l[i] == 0.f ? -__int_as_float(0x7f800000) : (m[i] + log2f(l[i])) * kLn2;
    }
  }
}

}  // namespace simt
}  // namespace mla
