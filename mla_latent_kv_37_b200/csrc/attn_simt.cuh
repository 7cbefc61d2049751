// Attention of several query rows on the SIMT cores with fp32 products (the fp32 configuration:
// no product of the tensor cores is exact to 1e-5), for whole packed prompts (192-wide keys,
// 128-wide values) and for a chunk of new tokens over the paged latent cache (576 and 512).
//
// A block of W x KS warps takes 8 W query rows and walks over the keys 64 at a time with an online
// softmax; warp w owns rows 8 (w % W) ... + 7, so a row's scores, maximum and sum stay inside one
// warp.  With KS = 2 two warps share the rows: each sums half of the columns of the scores (they
// exchange the halves and then hold the same ones) and adds half of the values, which halves the
// longest chain of a small call.
// Per 64 keys: S = Q K^T in slices of 64 columns (a thread has 4 rows x 4 keys:
// rows lane / 16 + 2 i, keys lane % 16 + 16 j), P to shared memory,
// O += P V in slices of keys with O in registers (8 rows x DV / 32 columns a thread).  The slices,
// 16 KB each, come by cp.async two steps ahead through three stages, with one block barrier a step.
//
// The work is 2 (DQ + DV) flops per row and key at 128 FMAs a clock and SM, and the loads from shared
// memory take twice that: one of 16 bytes costs about four clocks of the SM, whether or not the lanes
// read the same address, so 64 FMAs (16 clocks of the SM) that follow 8 loads (4 rows x 4 keys a
// thread) take 32.  (2 x 8 and 8 x 2 follow 10; a slice of 64 rows x 64 keys measured 4450 clocks with
// them.)  Small calls are bound by neither (FMA and shared memory are both busy for 30 ... 40% of the
// clocks in the two below) but by one tile's chain: a block walks over the tile's keys alone, a barrier
// a slice, with two to four warps a scheduler.  Prompts of 500, 129 and 33 tokens, 16 heads: 98 us (14
// TFLOP/s); 33 and 7 tokens over 700 and 129 rows: 48 us with the merge.
#pragma once
#include "chunk_plan.cuh"

namespace mla {
namespace simt {

constexpr int kKeys = 64, kSlice = 64, kStages = 3;
constexpr int kKPad = kSlice + 4;  // row strides with 16 bytes more than a multiple of 128: the
                                   // 16-byte loads of 4 or 8 rows fall into different banks

template <int DQ, int DV, int W, int KS> struct Layout {
  static constexpr int kThreads = 32 * W * KS, kRows = 8 * W;
  static constexpr int kQPad = DQ + 4;
  static constexpr int kKSteps = DQ / kSlice;
  static constexpr int kVKeys = 4096 / DV;                    // keys of a value slice
  static constexpr int kQ = 0;                                // [kRows][kQPad]
  static constexpr int kStage = kQ + kRows * kQPad;           // [kStages][kKeys][kKPad]
  static constexpr int kP = kStage + kStages * kKeys * kKPad; // [KS][W][kKeys][8 rows]
  static constexpr int kX = kP + KS * W * kKeys * 8;          // KS > 1: [2][W][16][32 lanes]
  static constexpr int kRow = kX + (KS - 1) * 2 * W * 512;    // [2][kKeys] source rows (int32)
  static constexpr size_t kBytes = (kRow + 2 * kKeys) * sizeof(float);
  static_assert(kVKeys * DV <= kKeys * kKPad && kBytes <= 232448, "shared memory");
  static_assert(KS == 1 || (KS == 2 && kVKeys == 32 && kRows * DV <= kStages * kKeys * kKPad),
                "a value slice has 16 keys for each half, and the ring holds a half's results");
};

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D columns of the scores of 4 rows x N keys.  The operands of the next four columns are loaded
// ahead of the products of these: there are two or four warps on a scheduler, too few to hide the
// loads otherwise.
template <int D, int N, int kQPad>
__device__ __forceinline__ void score_slice(const float* q0, const float* sK, float (&s)[4][4]) {
  float4 q[2][4], k[2][N];
  const auto load = [&](int buf, int d) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[buf][i] = *reinterpret_cast<const float4*>(q0 + 2 * i * kQPad + d);
#pragma unroll
    for (int j = 0; j < N; ++j) k[buf][j] = *reinterpret_cast<const float4*>(sK + 16 * j * kKPad + d);
  };
  load(0, 0);
#pragma unroll
  for (int d = 0; d < D; d += 4) {
    const int b = (d >> 2) & 1;
    if (d + 4 < D) load(b ^ 1, d + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[i][j] = fmaf(q[b][i].x, k[b][j].x, s[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[i][j] = fmaf(q[b][i].y, k[b][j].y, s[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[i][j] = fmaf(q[b][i].z, k[b][j].z, s[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[i][j] = fmaf(q[b][i].w, k[b][j].w, s[i][j]);
  }
}

// 8 rows' outputs of 8 keys: weights p[key][8 rows], values v[key][DV].
template <int DV>
__device__ __forceinline__ void value_keys(const float* p, const float* v, float (&o)[8][DV / 32]) {
  float4 w[2][2], x[2][DV / 128];
  const auto load = [&](int buf, int j) {
    w[buf][0] = *reinterpret_cast<const float4*>(p + 8 * j);
    w[buf][1] = *reinterpret_cast<const float4*>(p + 8 * j + 4);
#pragma unroll
    for (int k = 0; k < DV / 128; ++k)
      x[buf][k] = *reinterpret_cast<const float4*>(v + j * DV + 128 * k);
  };
  load(0, 0);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int b = j & 1;
    if (j < 7) load(b ^ 1, j + 1);
    const float pr[8] = {w[b][0].x, w[b][0].y, w[b][0].z, w[b][0].w,
                         w[b][1].x, w[b][1].y, w[b][1].z, w[b][1].w};
#pragma unroll
    for (int k = 0; k < DV / 128; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][4 * k] = fmaf(pr[i], x[b][k].x, o[i][4 * k]);
        o[i][4 * k + 1] = fmaf(pr[i], x[b][k].y, o[i][4 * k + 1]);
        o[i][4 * k + 2] = fmaf(pr[i], x[b][k].z, o[i][4 * k + 2]);
        o[i][4 * k + 3] = fmaf(pr[i], x[b][k].w, o[i][4 * k + 3]);
      }
  }
}

// One segment: rows r of the tile against keys [j0, j1), j0 < j1.  Src gives, in elements of float:
//   const float* q(r, d): 4 columns from d of row r's query (r < rows);
//   int row(j): where key j lies;  const float* k(row, d), v(row, d): 4 of its columns;
//   int visible(r): keys row r sees.
// On return m[i], l[i] and o[i][...] hold row 8 warp + i's maximum (log2 units), sum and
// unnormalised output columns 4 (lane + 32 k) + ..., in the first W warps.
template <int DQ, int DV, int W, int KS, class Src>
__device__ __forceinline__ void segment(const Src& src, float* smem, int rows, int j0, int j1,
                                        float scale_log2, float (&m)[8], float (&l)[8],
                                        float (&o)[8][DV / 32]) {
  using L = Layout<DQ, DV, W, KS>;
  constexpr int kD = kSlice / KS;  // columns of a slice that a warp sums
  float *sQ = smem + L::kQ, *sS = smem + L::kStage;
  int* sRow = reinterpret_cast<int*>(smem + L::kRow);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = 8 * (warp % W), half = warp / W, part = 16 * half;
  const int lr = lane >> 4, lk = lane & 15;
  float* sP = smem + L::kP + warp * kKeys * 8;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const bool idle = r0 >= rows;  // nothing to do but to copy
  __syncthreads();  // the previous segment has read everything
  const auto find_rows = [&](int jb, int buf) {
    for (int i = tid; i < kKeys; i += L::kThreads) sRow[buf * kKeys + i] = jb + i < j1 ? src.row(jb + i) : -1;
  };
  find_rows(j0, 0);
  for (int i = tid; i < L::kRows * DQ / 4; i += L::kThreads) {
    const int r = i / (DQ / 4), d = 4 * (i % (DQ / 4));
    copy16(sQ + r * L::kQPad + d, src.q(r < rows ? r : 0, d), r < rows);
  }
  __syncthreads();
  // the copies' place: two steps ahead of the products
  int cj = j0, cs = 0, cbuf = 0, cstage = 0;
  const auto copy_next = [&]() {
    if (cj < j1) {
      float* dst = sS + cstage * kKeys * kKPad;
      const int* row = sRow + cbuf * kKeys;
      if (cs < L::kKSteps) {
#pragma unroll
        for (int i = tid; i < kKeys * kSlice / 4; i += L::kThreads) {
          const int j = i / (kSlice / 4), d = 4 * (i % (kSlice / 4)), rj = row[j];
          copy16(dst + j * kKPad + d, src.k(max(rj, 0), kSlice * cs + d), rj >= 0);
        }
      } else {
        const int v0 = (cs - L::kKSteps) * L::kVKeys;
#pragma unroll
        for (int i = tid; i < L::kVKeys * DV / 4; i += L::kThreads) {
          const int j = i / (DV / 4), d = 4 * (i % (DV / 4)), rj = row[v0 + j];
          copy16(dst + 4 * i, src.v(max(rj, 0), d), rj >= 0);
        }
      }
      const int n = min(kKeys, j1 - cj);
      if (++cs == L::kKSteps + (n + L::kVKeys - 1) / L::kVKeys) {
        cs = 0;
        cj += kKeys;
        cbuf ^= 1;
      }
      cstage = cstage == kStages - 1 ? 0 : cstage + 1;
    }
    copy_commit();
  };
  copy_next();
  copy_next();
  int vis[4];
  float mr[4], lsum[4];  // rows r0 + lr + 2 i: maximum, and this lane's share of the sum
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + lr + 2 * i;
    vis[i] = r < rows ? min(src.visible(r), j1) : 0;
    mr[i] = NEG_INF;
    lsum[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < DV / 32; ++k) o[i][k] = 0.f;
  int stage = 0, buf = 0;
  // the next step's slice is there, and its place in the ring is free for the copy after it
  const auto step = [&]() -> const float* {
    copy_wait<1>();
    __syncthreads();
    copy_next();
    const float* p = sS + stage * kKeys * kKPad;
    stage = stage == kStages - 1 ? 0 : stage + 1;
    return p;
  };
  for (int jb = j0; jb < j1; jb += kKeys, buf ^= 1) {
    const int nk = min(kKeys, j1 - jb);
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int c = 0; c < L::kKSteps; ++c) {
      const float* sK = step() + lk * kKPad + kD * half;
      if (c == 0 && jb + kKeys < j1) find_rows(jb + kKeys, buf ^ 1);
      if (idle) continue;
      const float* q0 = sQ + (r0 + lr) * L::kQPad + kSlice * c + kD * half;
      if (nk > 48)
        score_slice<kD, 4, L::kQPad>(q0, sK, s);
      else if (nk > 32)
        score_slice<kD, 3, L::kQPad>(q0, sK, s);
      else if (nk > 16)
        score_slice<kD, 2, L::kQPad>(q0, sK, s);
      else
        score_slice<kD, 1, L::kQPad>(q0, sK, s);
    }
    if (!idle) {
      if (KS > 1) {
        float* x = smem + L::kX + (warp % W) * 512 + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[half * W * 512 + 32 * i] = s[i >> 2][i & 3];
        asm volatile("bar.sync %0, 64;" ::"r"(1 + warp % W) : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i >> 2][i & 3] += x[(half ^ 1) * W * 512 + 32 * i];
      }
      float alpha[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = NEG_INF;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = jb + lk + 16 * j < vis[i] ? s[i][j] * scale_log2 : NEG_INF;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        mx = fmaxf(mx, mr[i]);
        const float ref = mx == NEG_INF ? 0.f : mx;  // no key seen yet: every weight is 0
        alpha[i] = exp2f(mr[i] - ref);
        mr[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pr = exp2f(s[i][j] - ref);
          sum += pr;
          sP[(lk + 16 * j) * 8 + lr + 2 * i] = pr;
        }
        lsum[i] = lsum[i] * alpha[i] + sum;
      }
      if (__any_sync(0xffffffffu,
                     alpha[0] != 1.f || alpha[1] != 1.f || alpha[2] != 1.f || alpha[3] != 1.f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = __shfl_sync(0xffffffffu, alpha[i >> 1], 16 * (i & 1));
#pragma unroll
          for (int k = 0; k < DV / 32; ++k) o[i][k] *= a;
        }
      }
      __syncwarp();
    }
    for (int v0 = 0; v0 < nk; v0 += L::kVKeys) {
      const float* sV = step() + part * DV + 4 * lane;
      if (idle) continue;
      // (weights and values past nk are zero)
      const float* p0 = sP + (v0 + part) * 8;
      for (int j = 0; j < min(L::kVKeys / KS, nk - v0 - part); j += 8)
        value_keys<DV>(p0 + 8 * j, sV + j * DV, o);
      __syncwarp();  // P is read before the next keys' is written
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) lsum[i] += __shfl_xor_sync(0xffffffffu, lsum[i], w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = __shfl_sync(0xffffffffu, mr[i >> 1], 16 * (i & 1));
    l[i] = __shfl_sync(0xffffffffu, lsum[i >> 1], 16 * (i & 1));
  }
  if (KS == 1) return;
  // the second half of the values' outputs through the ring, [row][DV]; maxima and sums are the same
  __syncthreads();
  float* sO = sS + r0 * DV + 4 * lane;
  if (half > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < DV / 128; ++k)
        *reinterpret_cast<float4*>(sO + i * DV + 128 * k) =
            make_float4(o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]);
  }
  __syncthreads();
  if (half > 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < DV / 128; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(sO + i * DV + 128 * k);
      o[i][4 * k] += x.x;
      o[i][4 * k + 1] += x.y;
      o[i][4 * k + 2] += x.z;
      o[i][4 * k + 3] += x.w;
    }
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
  __device__ int row(int j) const { return j; }
  __device__ const float* k(int j, int d) const {
    return d < 128 ? k0 + j * k_tok + d : kr0 + j * kr_tok + (d - 128);
  }
  __device__ const float* v(int j, int d) const { return v0 + j * v_tok + d; }
  __device__ int visible(int r) const { return first + r + 1; }
};

// 32 rows a block, two warps for each eight of them, two blocks an SM: of few rows the longest
// tile takes the time.
constexpr int kPromptWarps = 4, kPromptParts = 2;
using PromptLayout = Layout<192, 128, kPromptWarps, kPromptParts>;

// block x: head x % n_heads of tile x / n_heads; a sequence's tiles run from its last rows (the
// longest) to its first
__global__ void __launch_bounds__(PromptLayout::kThreads, 2) prompt_kernel(const PromptParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kRows = PromptLayout::kRows;
  griddep_launch_dependents();
  griddep_wait();
  int seq, index, count;
  packed::Span s;
  const int h = blockIdx.x % p.n_heads, hk = h / (p.n_heads / p.n_kv_heads);
  const bool there = packed::warp_find_tile(p.cu, p.batch, p.n_tokens, kRows,
                                            blockIdx.x / p.n_heads, seq, index, count, s);
  if (blockIdx.x == 0) packed::check_offsets(p.cu, p.batch, p.n_tokens, p.status);
  if (!there) return;
  const int first = (count - 1 - index) * kRows, rows = min(kRows, s.size() - first);
  const int64_t t0 = s.begin;
  const PromptSrc src{static_cast<const float*>(p.q) + (t0 + first) * p.q_tok + h * p.q_head,
                      static_cast<const float*>(p.k_nope) + t0 * p.k_tok + hk * p.k_head,
                      static_cast<const float*>(p.k_rope) + t0 * p.kr_tok,
                      static_cast<const float*>(p.v) + t0 * p.v_tok + hk * p.v_head,
                      p.q_tok, p.k_tok, p.kr_tok, p.v_tok, first};
  float m[8], l[8], o[8][4];
  segment<192, 128, kPromptWarps, kPromptParts>(src, smem, rows, 0, first + rows, p.scale_log2, m, l, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= kPromptWarps) return;
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
  chunk::Shape shape;
  int parts, num_pages;
  chunk::PartStart* starts;
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
  __device__ int row(int j) const {
    const int pg = pages[j / chunk::kPage];
    return (pg < 0 || pg >= num_pages ? 0 : pg) * chunk::kPage + j % chunk::kPage;
  }
  __device__ const float* k(int row, int d) const {
    return pool + static_cast<int64_t>(row) * chunk::kRow + d;
  }
  __device__ const float* v(int row, int d) const { return k(row, d); }
  __device__ int visible(int r) const { return t.visible(r, n_heads); }
};

// 64 rows a block (their queries take 145 KB), and parts that end at any multiple of 16 keys: a
// step of 64 keys takes about 18 us here, too long to be the grain of a small call.
constexpr int kChunkWarps = 8, kChunkTileShift = 6, kChunkBlockShift = 4;
constexpr int kChunkBlock = 1 << kChunkBlockShift;
using ChunkLayout = Layout<576, 512, kChunkWarps, 1>;
static_assert(ChunkLayout::kRows == 1 << kChunkTileShift, "a tile's rows");
// Costs in quarters of a block of 16 keys: a segment's start and write-back take the time of about
// two blocks (40 tokens of 16 heads over 829 rows: 49 ... 58 us; 65 ... 71 us with half a block for them,
// 55 ... 59 us with four; eight single tokens, and one over 4096 rows: the same with each).
constexpr int kChunkCostShift = 2, kChunkSegCost = 8, kChunkLeast = 4;

__global__ void __launch_bounds__(ChunkLayout::kThreads, 1) chunk_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) float smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = p.shape.n_heads;
  const chunk::Range range = chunk::find_part(p.shape, p.parts, blockIdx.x,
                                              reinterpret_cast<chunk::Scratch*>(smem), p.status);
  if (threadIdx.x == 0) chunk::write_start(p.shape, range, p.starts + blockIdx.x);
  __syncthreads();
  chunk::SegIter it(p.shape, range);
  chunk::Segment seg;
  while (it.next(seg)) {
    const chunk::Tile& t = seg.t;
    const int j0 = seg.b0 * kChunkBlock;
    const int j1 = min(seg.b1 * kChunkBlock, t.visible(t.rows - 1, H));
    const int64_t row0 = static_cast<int64_t>(t.tok0) * H + t.row0;
    const ChunkSrc src{static_cast<const float*>(p.q_cat) + row0 * chunk::kRow,
                       static_cast<const float*>(p.pool),
                       p.page_table + static_cast<int64_t>(t.seq) * p.shape.max_pages,
                       p.num_pages, H, t};
    for (int pg = j0 / chunk::kPage + threadIdx.x; pg * chunk::kPage < j1;
         pg += ChunkLayout::kThreads)
      if (src.pages[pg] < 0 || src.pages[pg] >= p.num_pages)
        atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    float m[8], l[8], o[8][16];
    if (j0 < j1) {
      segment<576, 512, kChunkWarps, 1>(src, smem, t.rows, j0, j1, p.scale_log2, m, l, o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = l[i] = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[i][k] = 0.f;
      }
    }
    const bool whole = !seg.split;
    const int slot = chunk::partial_slot(blockIdx.x, seg.inside);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * warp + i;
      if (r >= t.rows) break;
      const int64_t row = whole ? row0 + r : static_cast<int64_t>(slot) * ChunkLayout::kRows + r;
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
