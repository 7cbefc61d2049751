// Rows of several new tokens into the paged latent cache, with the position rotation on the way:
//   pool[page_table[b][p / 64]][p % 64] = [c_KV,t | R(p) k_R,t],   q_out[t][h] = R(p) q[t][h],
// p = seq_lens[b] - n_b + i for token i of sequence b's n_b, R(p) the interleaved-pair rotation.
//
// Bound by HBM: a token's row is read and written once, 2 (576 + 64 H) elements in all, with 6
// flops per rotated pair.
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
  int n_tokens, batch, n_heads, max_pages, num_pages, heads_per_block;
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
  float theta;
  unsigned int* status;
};

// 16 bytes of elements: 8 bf16 or 4 fp32, an even number of them, so pairs never straddle.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  static constexpr int kN = 4;
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
  static constexpr int kN = 8;
  // rotated in fp32 and rounded once to the storage type
  static __device__ __forceinline__ uint32_t pair(uint32_t v, float2 cs) {
    const float a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xffff0000u);
    return pack_bf16x2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
  }
  static __device__ __forceinline__ uint4 rotate(uint4 v, const float2* cs) {
    return make_uint4(pair(v.x, cs[0]), pair(v.y, cs[1]), pair(v.z, cs[2]), pair(v.w, cs[3]));
  }
};

// grid (ceil(n_tokens / kTokens), 1 + head slices): block (x, 0) writes the cache rows of its
// tokens, block (x, 1 + y) rotates their queries of slice y.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const Params p) {
  constexpr int kN = Chunk<T>::kN, kPairs = kN / 2, kRotChunks = kDr / kN, kLatChunks = kDc / kN;
  __shared__ float2 cs[kTokens][kDr / 2];
  __shared__ int64_t slot[kTokens];  // pool row, or -1: the token is skipped
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * kTokens;
  griddep_launch_dependents();
  griddep_wait();
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
            cs[warp][lane] = rope_cs(p.theta, lane, static_cast<int>(pos));
          }
        }
        if (err && lane == 0) atomicOr(p.status, err);
      }
    }
    if (lane == 0) slot[warp] = s;
  }
  __syncthreads();
  const int n_here = min(kTokens, p.n_tokens - t0);
  if (blockIdx.y == 0) {
    for (int i = threadIdx.x; i < n_here * (kLatChunks + kRotChunks); i += kThreads) {
      const int k = i / (kLatChunks + kRotChunks), c = i % (kLatChunks + kRotChunks);
      const int64_t t = t0 + k, s = slot[k];
      if (s < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.pool) + s * kRow) + c;
      if (c < kLatChunks) {
        *dst = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.c_kv) +
                                                    t * p.c_stride) + c);
      } else {
        const int r = c - kLatChunks;
        const uint4 v = Chunk<T>::rotate(
            __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_r) + t * p.kr_stride) +
                  r),
            &cs[k][r * kPairs]);
        *dst = v;
        if (p.k_rope) reinterpret_cast<uint4*>(static_cast<T*>(p.k_rope) + t * kDr)[r] = v;
      }
    }
    return;
  }
  const int h0 = (blockIdx.y - 1) * p.heads_per_block;
  const int per = min(p.heads_per_block, p.n_heads - h0) * kRotChunks;
  for (int i = threadIdx.x; i < n_here * per; i += kThreads) {
    const int k = i / per, c = i % per, h = h0 + c / kRotChunks, r = c % kRotChunks;
    if (slot[k] < 0) continue;
    const int64_t t = t0 + k;
    const uint4 v = *(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + t * p.q_tok +
                                                     h * p.q_head) + r);
    reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + t * p.qo_tok + h * p.qo_head)[r] =
        Chunk<T>::rotate(v, &cs[k][r * kPairs]);
  }
}

}  // namespace rows
}  // namespace mla
