// Rows of several new tokens into the paged latent cache, with the position rotation on the way:
//   pool[page_table[b][p / 64]][p % 64] = [c_KV,t | R(p) k_R,t],   q_out[t][h] = R(p) q[t][h],
// p = seq_lens[b] - n_b + i for token i of sequence b's n_b, R(p) the interleaved-pair rotation.
//
// Bound by HBM: a token's row is read and written once, 2 (576 + 64 H) elements in all, with 6
// flops per rotated pair.  A thread's loads (eight chunks of 16 bytes of the queries) are on their
// way before the block looks up its tokens' places and angles, which takes as long; the frequencies
// come from the host, since a double-precision pow per block took longer than the loads.
#pragma once
#include "packed.cuh"
#include "ptx_sm100.cuh"
#include "rope.cuh"

namespace mla {
namespace rows {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 32;  // a warp finds one token's place and 32 angles
constexpr int kDc = 512, kDr = 64, kRow = 576, kPage = 64;

struct Params {
  int n_tokens, batch, n_heads, max_pages, num_pages, slices;
  const int32_t* cu;
  const int32_t* seq_lens;
  const int32_t* page_table;
  const void* c_kv;
  const void* k_r;
  const void* q;
  void* pool;
  void* k_rope;
  void* q_out;
  int64_t c_stride, kr_stride, q_tok, q_head, qo_tok, qo_head;  // elements
  double inv_freq[32];  // theta^(-2 pair / 64)
  unsigned int* status;
};

// 16 bytes of elements: 8 bf16 or 4 fp32, an even number of them, so pairs never straddle.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  static constexpr int kN = 4, kHeads = kThreads / (kDr / kN);  // heads of a block
  static __device__ __forceinline__ uint4 rotate(uint4 v, const float2* cs) {
    const float a = __uint_as_float(v.x), b = __uint_as_float(v.y);
    const float c = __uint_as_float(v.z), d = __uint_as_float(v.w);
    return make_uint4(__float_as_uint(a * cs[0].x - b * cs[0].y),
                      __float_as_uint(a * cs[0].y + b * cs[0].x),
                      __float_as_uint(c * cs[1].x - d * cs[1].y),
                      __float_as_uint(c * cs[1].y + d * cs[1].x));
  }
};
template <> struct Chunk<__nv_bfloat16> {
  static constexpr int kN = 8, kHeads = kThreads / (kDr / kN);
  // rotated in fp32 and rounded once to the storage type
  static __device__ __forceinline__ uint32_t pair(uint32_t v, float2 cs) {
    const float a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xffff0000u);
    return pack_bf16x2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
  }
  static __device__ __forceinline__ uint4 rotate(uint4 v, const float2* cs) {
    return make_uint4(pair(v.x, cs[0]), pair(v.y, cs[1]), pair(v.z, cs[2]), pair(v.w, cs[3]));
  }
};

// For each kTokens tokens `slices` blocks side by side: the first writes their cache rows, the others
// rotate their queries, kHeads heads each.  (8092 tokens, 128 heads: 55.5 us = 5.1 TB/s; 58 us with
// the tokens side by side; 63 us with six blocks an SM instead of four.)
template <typename T>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const __grid_constant__ Params p) {
  constexpr int kN = Chunk<T>::kN, kPairs = kN / 2, kRotChunks = kDr / kN, kLatChunks = kDc / kN;
  constexpr int kRowChunks = kLatChunks + kRotChunks;
  constexpr int kLoads = (kTokens * kRowChunks + kThreads - 1) / kThreads;  // 3 or 5
  static_assert(kLoads <= kTokens, "both kinds of blocks load into the same registers");
  __shared__ float2 cs[kTokens][kDr / 2];
  __shared__ int64_t slot[kTokens];  // pool row, or -1: the token is skipped
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % p.slices, t0 = blockIdx.x / p.slices * kTokens;
  const int n_here = min(kTokens, p.n_tokens - t0);
  const bool rows = slice == 0;
  griddep_launch_dependents();
  griddep_wait();
  uint4 v[kTokens];
  // queries: thread = (head, chunk), one token a load
  const int h = (slice - 1) * Chunk<T>::kHeads + tid / kRotChunks;
  const int r = tid % kRotChunks;
  if (rows) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = tid + u * kThreads, k = i / kRowChunks, c = i % kRowChunks;
      const int64_t t = t0 + k;
      if (k < n_here)
        v[u] = c < kLatChunks
                   ? reinterpret_cast<const uint4*>(static_cast<const T*>(p.c_kv) + t * p.c_stride)[c]
                   : reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_r) +
                                                    t * p.kr_stride)[c - kLatChunks];
    }
  } else if (h < p.n_heads) {
    const T* src = static_cast<const T*>(p.q) + t0 * p.q_tok + h * p.q_head + r * kN;
#pragma unroll
    for (int u = 0; u < kTokens; ++u)
      if (u < n_here) v[u] = *reinterpret_cast<const uint4*>(src + u * p.q_tok);
  }
  {
    const int t = t0 + warp;
    int64_t s = -1;
    if (t < p.n_tokens) {
      const int b = packed::warp_sequence_of(p.cu, p.batch, t);
      if (b < p.batch) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        unsigned int err = 0;
        if (c0 < 0 || c0 > t || c1 <= t || c1 > p.n_tokens) {
          err = MLA_STATUS_BAD_LENGTH;
        } else {
          const int64_t pos = static_cast<int64_t>(p.seq_lens[b]) - (c1 - t);
          if (pos < 0 || pos >= static_cast<int64_t>(p.max_pages) * kPage) {
            err = MLA_STATUS_BAD_POSITION;
          } else {
            const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pos / kPage];
            if (page < 0 || page >= p.num_pages)
              err = MLA_STATUS_BAD_PAGE;
            else
              s = static_cast<int64_t>(page) * kPage + pos % kPage;
            cs[warp][lane] = rope_cs(p.inv_freq[lane], static_cast<int>(pos));
          }
        }
        if (err && lane == 0) atomicOr(p.status, err);
      }
    }
    if (lane == 0) slot[warp] = s;
    if (blockIdx.x == 0) packed::check_offsets(p.cu, p.batch, p.n_tokens, p.status);
  }
  __syncthreads();
  if (rows) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = tid + u * kThreads, k = i / kRowChunks, c = i % kRowChunks;
      if (k >= n_here || slot[k] < 0) continue;
      uint4 x = v[u];
      if (c >= kLatChunks) {
        const int j = c - kLatChunks;
        x = Chunk<T>::rotate(x, &cs[k][j * kPairs]);
        if (p.k_rope)
          reinterpret_cast<uint4*>(static_cast<T*>(p.k_rope) + static_cast<int64_t>(t0 + k) * kDr)[j] = x;
      }
      reinterpret_cast<uint4*>(static_cast<T*>(p.pool) + slot[k] * kRow)[c] = x;
    }
  } else if (h < p.n_heads) {
    T* dst = static_cast<T*>(p.q_out) + t0 * p.qo_tok + h * p.qo_head + r * kN;
#pragma unroll
    for (int u = 0; u < kTokens; ++u)
      if (u < n_here && slot[u] >= 0)
        *reinterpret_cast<uint4*>(dst + u * p.qo_tok) = Chunk<T>::rotate(v[u], &cs[u][r * kPairs]);
  }
}

}  // namespace rows
}  // namespace mla
