// C ABI of the calls with several new tokens per sequence (see include/mla.h): rows into the
// paged cache, attention over whole packed prompts, attention of a chunk over the paged cache.
// Host side: argument validation before any CUDA call, workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "attn_simt.cuh"
#include "chunk_plan.cuh"
#include "chunk_sm100.cuh"
#include "host_services.h"
#include "prompt_pair_sm100.cuh"
#include "prompt_sm100.cuh"
#include "rows.cuh"

namespace mla {
namespace {

constexpr int kDc = 512, kDr = 64, kDn = 128, kDv = 128, kPageN = 64;
constexpr int kMaxParts = 1 << 16;
// Prompts of this many tokens on average run on pairs of SMs (one of 16384, 32 heads: 2.37 ... 2.41 ms on
// pairs, 2.48 ... 2.51 ms without; 64 heads, 8192 tokens in all: 4096 each 687 ... 737 us and 696 ... 714 us;
// 2048 each 454 ... 463 and 428 us, and one of 2048 alone 134 ... 137 and 129 ... 132 us; 1024 each 333 ...
// 337 and 278 us, 256 each 346 and 178 us, since a pair's 512 rows fill badly).
constexpr int kPairTokens = 4096;
constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t elem_size(const mla_dims* d) { return d->dtype == MLA_BF16 ? 2 : 4; }
// A stride (elements) of 16-byte multiples under which neighbours of `least` elements do not overlap;
// strides of zero or backwards are refused.
bool stride_ok(int64_t stride, int64_t least, size_t elem) {
  return stride >= least && stride < (int64_t{1} << 36) && stride * static_cast<int64_t>(elem) % 16 == 0;
}

float resolve_scale(float softmax_scale) {
  return softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(kDn + kDr));
}

// Kernel attributes, once per device.
int set_attributes() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return host_cuda_error(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return MLA_OK;
  if ((e = cudaFuncSetAttribute(simt::prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(simt::PromptLayout::kBytes))) != cudaSuccess ||
      (e = cudaFuncSetAttribute(simt::chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(simt::ChunkLayout::kBytes))) != cudaSuccess)
    return host_cuda_error(e, "cudaFuncSetAttribute");
  if ((e = cudaFuncSetAttribute(prompt::prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(prompt::kSmemBytes))) != cudaSuccess)
    return host_cuda_error(e, "cudaFuncSetAttribute(prompt_kernel)");
  if ((e = cudaFuncSetAttribute(prompt_pair::pair_kernel,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(prompt_pair::kSmemBytes))) != cudaSuccess)
    return host_cuda_error(e, "cudaFuncSetAttribute(prompt_pair)");
  if ((e = cudaFuncSetAttribute(chunk::pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(chunk::kSmemBytes))) != cudaSuccess)
    return host_cuda_error(e, "cudaFuncSetAttribute(pair_kernel)");
  done[dev] = true;
  return MLA_OK;
}

// Workspace of mla_chunk_attn: where the parts begin, and their partial results.
struct ChunkSpace {
  size_t starts, part_o, part_lse, total;
  int tile_rows, parts;
};
ChunkSpace chunk_space(const mla_dims* d, int num_splits, int sms) {
  ChunkSpace w{};
  const bool bf16 = d->dtype == MLA_BF16;
  w.tile_rows = bf16 ? chunk::kTileRows : simt::ChunkLayout::kRows;
  w.parts = num_splits > 0 ? num_splits : bf16 ? sms / 2 : sms;  // CTA pairs, or CTAs
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  w.starts = take(sizeof(chunk::PartStart) * w.parts);
  w.part_o = take(2ull * w.parts * w.tile_rows * kDc * 4);
  w.part_lse = take(2ull * w.parts * w.tile_rows * 4);
  w.total = off;
  return w;
}

// rows x columns of a call in int32 units on the device, page ids and lengths likewise
bool counts_ok(const mla_dims* d, int32_t n_tokens) {
  return static_cast<int64_t>(n_tokens) * d->n_heads <= INT32_MAX && d->batch < INT32_MAX;
}
bool pages_ok(int32_t num_pages, int32_t max_pages) {
  return num_pages >= 1 && max_pages >= 1 &&
         static_cast<int64_t>(num_pages) * kPageN <= INT32_MAX &&
         static_cast<int64_t>(max_pages) * kPageN <= INT32_MAX;
}
}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_append_rows(const mla_dims* dims, int32_t n_tokens, const int32_t* cu_tokens,
                    const int32_t* seq_lens, const void* c_kv, int64_t c_kv_stride,
                    const void* k_r, int64_t k_r_stride, const int32_t* page_table,
                    int32_t max_pages, void* cache_pool, int32_t num_pages, void* k_rope,
                    const void* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                    void* q_rope_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                    mla_stream_t stream) {
  int rc = host_check_dims(dims);
  if (rc) return rc;
  if (n_tokens < 0 || !pages_ok(num_pages, max_pages)) return MLA_ERR_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!counts_ok(dims, n_tokens)) return MLA_ERR_ARG;
  if (!cu_tokens || !seq_lens || !c_kv || !k_r || !page_table || !cache_pool ||
      !q_rope != !q_rope_out)
    return MLA_ERR_NULL_ARG;
  const size_t e = elem_size(dims);
  if (!stride_ok(c_kv_stride, kDc, e) || !stride_ok(k_r_stride, kDr, e)) return MLA_ERR_ARG;
  if (q_rope && (!stride_ok(q_token_stride, kDr, e) || !stride_ok(q_head_stride, kDr, e) ||
                 !stride_ok(q_out_token_stride, kDr, e) || !stride_ok(q_out_head_stride, kDr, e)))
    return MLA_ERR_ARG;
  if (!aligned(cu_tokens, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) ||
      !aligned(c_kv, 16) || !aligned(k_r, 16) || !aligned(cache_pool, 16) ||
      !aligned(k_rope, 16) || !aligned(q_rope, 16) || !aligned(q_rope_out, 16))
    return MLA_ERR_ALIGN;
  HostDevice dev;
  if ((rc = host_device(&dev))) return rc;
  rows::Params p{};
  p.n_tokens = n_tokens;
  p.batch = dims->batch;
  p.n_heads = dims->n_heads;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.cu = cu_tokens;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.c_kv = c_kv;
  p.k_r = k_r;
  p.q = q_rope;
  p.pool = cache_pool;
  p.k_rope = k_rope;
  p.q_out = q_rope_out;
  p.c_stride = c_kv_stride;
  p.kr_stride = k_r_stride;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.qo_tok = q_out_token_stride;
  p.qo_head = q_out_head_stride;
  rope_frequencies(dims->rope_theta, p.inv_freq);
  p.status = dev.status;
  const unsigned blocks = (static_cast<unsigned>(n_tokens) + rows::kTokens - 1) / rows::kTokens;
  const bool bf16 = dims->dtype == MLA_BF16;
  const int heads = bf16 ? rows::Chunk<__nv_bfloat16>::kHeads : rows::Chunk<float>::kHeads;
  p.slices = 1 + (q_rope ? (dims->n_heads + heads - 1) / heads : 0);
  host_launch(bf16 ? rows::append_rows_kernel<__nv_bfloat16> : rows::append_rows_kernel<float>,
              dim3(blocks * p.slices), dim3(rows::kThreads), 0,
              reinterpret_cast<cudaStream_t>(stream), p);
  return host_launched();
}

int mla_prompt_attn(const mla_dims* dims, int32_t n_tokens, int32_t n_kv_heads,
                    const int32_t* cu_tokens, const void* q, int64_t q_token_stride,
                    int64_t q_head_stride, const void* k_nope, int64_t k_token_stride,
                    int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
                    const void* v, int64_t v_token_stride, int64_t v_head_stride,
                    float softmax_scale, void* o, float* lse, mla_stream_t stream) {
  int rc = host_check_dims(dims);
  if (rc) return rc;
  if (n_tokens < 0 || n_kv_heads < 1 || dims->n_heads % n_kv_heads) return MLA_ERR_ARG;
  if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale)) return MLA_ERR_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!counts_ok(dims, n_tokens)) return MLA_ERR_ARG;
  if (!cu_tokens || !q || !k_nope || !k_rope || !v || !o) return MLA_ERR_NULL_ARG;
  const size_t e = elem_size(dims);
  if (!stride_ok(q_token_stride, kDn + kDr, e) || !stride_ok(q_head_stride, kDn + kDr, e) ||
      !stride_ok(k_token_stride, kDn, e) || !stride_ok(k_head_stride, kDn, e) ||
      !stride_ok(k_rope_stride, kDr, e) || !stride_ok(v_token_stride, kDv, e) ||
      !stride_ok(v_head_stride, kDv, e))
    return MLA_ERR_ARG;
  if (!aligned(cu_tokens, 4) || !aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) ||
      !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return MLA_ERR_ALIGN;
  HostDevice dev;
  if ((rc = host_device(&dev)) || (rc = set_attributes())) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const float scale_log2 = resolve_scale(softmax_scale) * kLog2e;
  // every sequence has at most one tile that is not full, and every tile has a token
  const auto tiles = [&](int rows) {
    return static_cast<unsigned>(std::min<int64_t>(
        n_tokens, int64_t{n_tokens} / rows + std::min(dims->batch, n_tokens)));
  };
  if (dims->dtype == MLA_BF16) {
    const bool pair = static_cast<int64_t>(n_tokens) >= int64_t{kPairTokens} * dims->batch;
    // heads x tokens of 64-column boxes of 128 tokens (a CTA of a pair loads half of the keys); tokens
    // past n_tokens read as zero
    const auto map = [&](CUtensorMap* m, const void* base, int width, int heads, int64_t head_stride,
                         int64_t token_stride, uint32_t tokens) {
      const uint64_t dim[3] = {static_cast<uint64_t>(width), static_cast<uint64_t>(heads),
                               static_cast<uint64_t>(n_tokens)};
      const uint64_t str[2] = {2 * static_cast<uint64_t>(head_stride),
                               2 * static_cast<uint64_t>(token_stride)};
      const uint32_t box[3] = {64, 1, tokens};
      return host_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dim, str, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const uint32_t keys = pair ? prompt::kTile / 2 : prompt::kTile;
    CUtensorMap tq, tk, tkr, tv;
    if ((rc = map(&tq, q, kDn + kDr, dims->n_heads, q_head_stride, q_token_stride, prompt::kTile)) ||
        (rc = map(&tk, k_nope, kDn, n_kv_heads, k_head_stride, k_token_stride, keys)) ||
        (rc = map(&tkr, k_rope, kDr, 1, k_rope_stride, k_rope_stride, keys)) ||
        (rc = map(&tv, v, kDv, n_kv_heads, v_head_stride, v_token_stride, prompt::kTile)))
      return rc;
    const prompt::Params p{n_tokens, dims->batch, dims->n_heads, n_kv_heads, cu_tokens, scale_log2,
                           static_cast<__nv_bfloat16*>(o), lse, dev.status, host_wait_ns(), host_stall()};
    if (pair)
      host_launch(prompt_pair::pair_kernel, dim3(2 * tiles(prompt_pair::kRows), dims->n_heads),
                  dim3(prompt_pair::kThreads), prompt_pair::kSmemBytes, st, tq, tk, tkr, tv, p);
    else
      host_launch(prompt::prompt_kernel, dim3(tiles(prompt::kRows), dims->n_heads),
                  dim3(prompt::kThreads), prompt::kSmemBytes, st, tq, tk, tkr, tv, p);
    return host_launched();
  }
  simt::PromptParams p{};
  p.n_tokens = n_tokens;
  p.batch = dims->batch;
  p.n_heads = dims->n_heads;
  p.n_kv_heads = n_kv_heads;
  p.cu = cu_tokens;
  p.q = q;
  p.k_nope = k_nope;
  p.k_rope = k_rope;
  p.v = v;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.k_tok = k_token_stride;
  p.k_head = k_head_stride;
  p.kr_tok = k_rope_stride;
  p.v_tok = v_token_stride;
  p.v_head = v_head_stride;
  p.scale_log2 = scale_log2;
  p.o = o;
  p.lse = lse;
  p.status = dev.status;
  host_launch(simt::prompt_kernel, dim3(tiles(simt::PromptLayout::kRows) * dims->n_heads),
              dim3(simt::PromptLayout::kThreads), simt::PromptLayout::kBytes, st, p);
  return host_launched();
}

size_t mla_chunk_workspace_size(const mla_dims* dims, int32_t n_tokens, int32_t num_splits) {
  if (host_check_dims(dims) != MLA_OK || n_tokens < 0 || num_splits < 0 ||
      num_splits > kMaxParts || !counts_ok(dims, n_tokens))
    return 0;
  HostDevice dev{148, nullptr};
  (void)host_device(&dev);
  return chunk_space(dims, num_splits, dev.sms).total;
}

int mla_chunk_attn(const mla_dims* dims, int32_t n_tokens, const int32_t* cu_tokens,
                   const void* q_cat, const void* cache_pool, int32_t num_pages,
                   const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                   float softmax_scale, int32_t num_splits, void* workspace,
                   size_t workspace_bytes, void* o_lat, int32_t o_dtype, float* lse,
                   mla_stream_t stream) {
  int rc = host_check_dims(dims);
  if (rc) return rc;
  if (n_tokens < 0 || !pages_ok(num_pages, max_pages) || num_splits < 0 || num_splits > kMaxParts)
    return MLA_ERR_ARG;
  if (o_dtype != MLA_FP32 && o_dtype != dims->dtype) return MLA_ERR_ARG;
  if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale)) return MLA_ERR_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!counts_ok(dims, n_tokens)) return MLA_ERR_ARG;
  if (!cu_tokens || !q_cat || !cache_pool || !page_table || !seq_lens || !o_lat)
    return MLA_ERR_NULL_ARG;
  if (!aligned(cu_tokens, 4) || !aligned(q_cat, 16) || !aligned(cache_pool, 16) ||
      !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(o_lat, 16) || !aligned(lse, 4))
    return MLA_ERR_ALIGN;
  if (!workspace) return MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MLA_ERR_ALIGN;
  HostDevice dev;
  if ((rc = host_device(&dev)) || (rc = set_attributes())) return rc;
  const ChunkSpace w = chunk_space(dims, num_splits, dev.sms);
  if (workspace_bytes < w.total) return MLA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const bool bf16 = dims->dtype == MLA_BF16;
  const chunk::Shape shape{n_tokens, dims->batch, dims->n_heads, max_pages,
                           bf16 ? chunk::kTileShift : simt::kChunkTileShift,
                           bf16 ? chunk::kBlockShift : simt::kChunkBlockShift,
                           bf16 ? chunk::kCostShift : simt::kChunkCostShift,
                           bf16 ? chunk::kSegCost : simt::kChunkSegCost,
                           bf16 ? chunk::kLeast : simt::kChunkLeast, cu_tokens, seq_lens};
  chunk::PartStart* starts = reinterpret_cast<chunk::PartStart*>(ws + w.starts);
  float* part_o = reinterpret_cast<float*>(ws + w.part_o);
  float* part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  const float scale_log2 = resolve_scale(softmax_scale) * kLog2e;
  if (bf16) {
    // rows of 576 in boxes of 64 columns x 64 rows: the queries, and the pool's pages
    const auto map = [&](CUtensorMap* m, const void* base, int64_t rows) {
      const uint64_t dim[2] = {chunk::kRow, static_cast<uint64_t>(rows)};
      const uint64_t str[1] = {2 * chunk::kRow};
      const uint32_t box[2] = {64, 64};
      return host_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dim, str, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    };
    CUtensorMap tq, tc;
    if ((rc = map(&tq, q_cat, static_cast<int64_t>(n_tokens) * dims->n_heads)) ||
        (rc = map(&tc, cache_pool, static_cast<int64_t>(num_pages) * kPageN)))
      return rc;
    const chunk::Params p{shape, w.parts, num_pages, starts, page_table, scale_log2, o_lat,
                          o_dtype == MLA_FP32, lse, part_o, part_lse, dev.status, host_wait_ns(),
                          host_stall()};
    host_launch(chunk::pair_kernel, dim3(2 * w.parts), dim3(chunk::kThreads), chunk::kSmemBytes,
                st, tq, tc, p);
  } else {
    const simt::ChunkParams p{shape, w.parts, num_pages, starts, q_cat, cache_pool, page_table, scale_log2,
                              o_lat, lse, part_o, part_lse, dev.status};
    host_launch(simt::chunk_kernel, dim3(w.parts), dim3(simt::ChunkLayout::kThreads),
                simt::ChunkLayout::kBytes, st, p);
  }
  if ((rc = host_launched())) return rc;
  if (w.parts == 1) return MLA_OK;
  const dim3 block(chunk::kCombineThreads);
  if (!bf16)
    host_launch(chunk::combine_rows_kernel<float>, dim3(w.parts - 1, w.tile_rows / 8), block, 0, st,
                w.parts, w.tile_rows, starts, part_o, part_lse, static_cast<float*>(o_lat), lse);
  else if (o_dtype == MLA_FP32)
    host_launch(chunk::combine_columns_kernel<float>, dim3(w.parts - 1, w.tile_rows / 32, 4), block, 0,
                st, w.parts, w.tile_rows, starts, part_o, part_lse, static_cast<float*>(o_lat), lse);
  else
    host_launch(chunk::combine_columns_kernel<__nv_bfloat16>,
                dim3(w.parts - 1, w.tile_rows / 32, 4), block, 0, st, w.parts, w.tile_rows, starts,
                part_o, part_lse, static_cast<__nv_bfloat16*>(o_lat), lse);
  return host_launched();
}

}  // extern "C"
