// Attention of a chunk of new tokens over the paged latent cache on the tcgen05 tensor cores
// (bf16): S = Q C^T (576 wide), online softmax over the keys a row sees, O += P C_lat (512 wide),
// for tiles of 128 (token, head) rows of a sequence.
//
// A tile's O (128 x 512 fp32) is as large as one SM's tensor memory, so a pair of CTAs shares it:
// every product is one tcgen05.mma over both SMs (cta_group::2, M = 128), of which each SM holds
// 64 rows.  No score and no weight has to cross the pair; each SM's tensor core reads its half of
// the B operand from either SM's shared memory.
//   * TMEM of each CTA: a row's values lie in two lanes, i and i + 64, for the two halves of the
//     product's columns.  O: 2 x 128 columns (values 256 g ... + 127 in lane i, + 128 ... + 255 in
//     lane i + 64, for g = 0, 1).  S: two buffers of 64 columns (the block's first page in lane
//     i, its second in lane i + 64).
//   * A block of 128 keys is two pages.  For S, CTA r loads page r, all 576 columns, in three
//     units of three 8 KB boxes; for O, 64 keys x 128 of its columns make a unit of 16 KB, four a
//     block.  The rows come from L2 twice (62 bytes a clock and SM at the full tensor rate); one
//     copy cannot serve both products, because S wants the same columns at the same place in
//     both CTAs and O wants different ones.  Each ring holds one block and is released unit by
//     unit, and two threads feed the rings, so neither waits for the other.
//   * Shared memory: Q 72 KB | keys 72 KB | values 64 KB | P 16 KB.
//   * The four softmax warps: a thread has half of a row's 128 scores; the two threads of a row
//     exchange their maxima through shared memory.
//   * S and O are issued by two warps, each waiting for its own operands: the tensor core takes what
//     comes, and neither's waits hold up the other.
// Statistics and O are fp32; P is rounded to bf16 for the tensor core (the sum adds the unrounded
// weights).  The running maximum is a reference that moves only when it would grow by more than
// 2^8, so O is hardly ever rescaled.
//
// Bound by the tensor pipe, 2176 flops per visible pair of row and key, and behind it by the power
// limit: 1024 tokens over 16384 rows, 128 heads 3.3 ... 3.7 ms, 1.23 ... 1.37 PFLOP/s (a library
// matrix product runs at 1.37 for seconds on end).  32 x 4 tokens over 4096 ... 8126 rows: 185 ...
// 225 us, the pipe at 60%: a ring holds one block, so that a page that comes from HBM holds the products
// up, and the merge (15 us) follows.  Eight single tokens: 24 us, of which the first copies' latency, the
// partial results and their merge are the most.
#pragma once
#include "chunk_plan.cuh"

namespace mla {
namespace chunk {

constexpr int kTileShift = 7, kTileRows = 1 << kTileShift, kCtaRows = 64;
constexpr int kBlockShift = 7, kBlock = 1 << kBlockShift;  // keys per block: two pages
// Costs in blocks: a segment's start and write-back take the time of about four.  Parts of at least
// four; with parts of two, and of eight and a cost of eight, 128 heads: eight single tokens over 1 ...
// 3000 keys 25.4 us (27.5, 29.7), one over 700 22.4 (19.2, 22.1), one over 16384 36.9 (36.9, 33.9), 32 x 4
// over 4096 ... 8126 186 (186, 189); 16 heads: 64 single tokens over 500 27.5 (27.5, 27.0).
constexpr int kCostShift = 0, kSegCost = 4, kLeast = 4;
constexpr int kThreads = 256;  // 4 softmax warps, key producer, S issuer, value producer, O issuer
constexpr uint32_t kBoxBytes = 64 * 128;  // 64 rows x 64 bf16
constexpr int kKUnits = 3, kVUnits = 4;
constexpr uint32_t kKUnit = 3 * kBoxBytes, kVUnit = 2 * kBoxBytes;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 9 * kBoxBytes;
constexpr uint32_t kOffV = kOffK + kKUnits * kKUnit;
constexpr uint32_t kOffP = kOffV + kVUnits * kVUnit;
constexpr uint32_t kOffBar = kOffP + 2 * kBoxBytes;
constexpr uint32_t kSmemBytes = kOffBar + 1536;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// The reference of a row whose scores so far are all -inf (no key seen, or products beyond fp32): every
// weight is 0 under it, and any score that is finite moves it.
constexpr float kLowest = -3.402823466e38f;
constexpr uint64_t kDrainNs = 200000000ull;

struct Params {
  Shape shape;
  int parts, num_pages;
  PartStart* starts;
  const int32_t* page_table;
  float scale_log2;
  void* o;
  int o_f32;
  float* lse;
  float* part_o;
  float* part_lse;
  unsigned int* status;
  uint64_t wait_ns;
  int stall;  // see host_stall
};

constexpr int kLoadBars = 1 + kKUnits + kVUnits;  // the first barriers: of copies
// Barriers marked L are the leader's (CTA 0): the MMA issuer waits there for both CTAs.  The
// others are each CTA's own; a commit arrives at both CTAs'.
struct ChunkBars {
  uint64_t q_full;            // L: the segment's queries landed (bytes of both CTAs)
  uint64_t k_full[kKUnits];   // L: a key unit landed (bytes of both CTAs)
  uint64_t v_full[kVUnits];   // L: both CTAs' value units landed (2, and bytes)
  uint64_t q_empty;           // the segment's last S is done (commit)
  uint64_t k_empty[kKUnits];  // S has read the unit (commit)
  uint64_t v_empty[kVUnits];  // O has read the unit (commit)
  uint64_t s_full[2];         // S of a block is written (commit)
  uint64_t s_free[2];         // L: the softmax warps of both CTAs have read S (8)
  uint64_t p_full;            // L: the softmax warps of both CTAs have written P (8)
  uint64_t pv_done;           // O of the block is added, P is free (commit)
  uint64_t o_free;            // L: the softmax warps of both CTAs have drained O (8)
  uint64_t v_tail[kVUnits];   // a value unit with rows past the sequence's end landed (bytes)
  uint64_t drain;             // both issuers' products are done (2 commits)
  uint64_t stall;             // nothing ever arrives here (test of a wait that runs out)
  uint32_t tmem_base;
  int abort_flag;
  // what the producers (warps 4 and 6) have issued: blocks begun, segments or ragged blocks begun, and
  // where a wait that ran out left the last of them (0: nowhere)
  int blocks[8], rest[8], left[8];
  int loads[kLoadBars];       // from that, phases of q_full, k_full[], v_full[]
  float xch[2][kTileRows];    // the two halves of a row exchange maxima (block parity) and sums
};
static_assert(sizeof(ChunkBars) <= 1536, "barrier block");

__device__ __forceinline__ void pair_barrier(int id) {  // 64 threads: warps w and w ^ 2
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

// After an abort, by a producer's warp: the phases of its barriers that it has had its part in; and its
// copies that no v_full counts yet, those of a ragged block, have landed.
enum { kLeftQ = 1, kLeftUnit = 16, kLeftRagged = 32, kLeftTail = 48 };
__device__ __forceinline__ void issued_loads(ChunkBars* bars, int warp, int lane, const WaitCtx& w) {
  const bool keys = warp == 4;
  const int units = keys ? kKUnits : kVUnits, n = bars->blocks[warp], rest = bars->rest[warp];
  const int left = bars->left[warp], at = left & ~15, u = left & 15;
  // units issued (of values, announced): all, or up to unit u of the last block
  const int issued = at == 0 ? units * n : units * (n - 1) + (at == kLeftRagged ? 0 : u);
  if (lane < units) bars->loads[(keys ? 1 : 1 + kKUnits) + lane] = (issued + units - 1 - lane) / units;
  if (keys && lane == 0) bars->loads[0] = left == kLeftQ ? rest - 1 : rest;
  if (lane < (at == kLeftTail ? kVUnits : at == kLeftRagged ? u : 0))
    mbar_wait(&bars->v_tail[lane], (rest - 1) & 1, w);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c,
                const __grid_constant__ Params p) {
  // (1024-byte atoms of the swizzle; a base known when compiling makes constants of the descriptors)
  extern __shared__ __align__(1024) uint8_t smem[];
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem + kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int part = blockIdx.x >> 1;
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_c);
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < kKUnits; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < kVUnits; ++i) {
      mbar_init(&bars->v_full[i], 2);
      mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->v_tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 8);
    }
    mbar_init(&bars->p_full, 8);
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->o_free, 8);
    mbar_init(&bars->drain, 2);
    mbar_init(&bars->stall, 1);
    bars->abort_flag = 0;
    bars->left[4] = bars->left[6] = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 5) {
    pair_tmem_alloc(&bars->tmem_base, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort_flag, p.status, p.wait_ns};
  volatile int never = 0;
  const WaitCtx drain_ctx{&never, p.status, kDrainNs};
  griddep_launch_dependents();
  griddep_wait();
  const int H = p.shape.n_heads;
  const Range range =
      find_part(p.shape, p.parts, part, reinterpret_cast<Scratch*>(smem + kOffP), p.status);
  if (rank == 0 && threadIdx.x == 0) write_start(p.shape, range, p.starts + part);
  __syncthreads();  // P's place held the scratch
  if (p.stall != 0 && stall_here(p.stall, warp, rank)) (void)warp_wait(&bars->stall, 0, wc);
  SegIter it(p.shape, range);
  Segment seg;

  if (warp == 4 || warp == 6) {
    // =================== TMA producers: queries and keys (warp 4), values (warp 6) ============
    const bool keys = warp == 4;
    bool ok = true;
    int n = 0, sg = 0, tails = 0;  // blocks, non-empty segments, and ragged blocks so far
    int* note = &bars->left[warp];
    while (ok && it.next(seg)) {
      const Tile t = seg.t;
      const int b0 = seg.b0, b1 = seg.b1;
      if (b0 == b1) continue;
      const int32_t* table = p.page_table + static_cast<int64_t>(t.seq) * p.shape.max_pages;
      const int pages = (t.visible(t.rows - 1, H) + kPage - 1) / kPage;
      if (keys) {
        if (sg > 0) ok = warp_wait_noted(&bars->q_empty, (sg - 1) & 1, wc, note, kLeftQ);
        if (ok && elect_one()) {
          const uint32_t bar = mapa_shared(smem_u32(&bars->q_full), 0);
          if (rank == 0) mbar_arrive_expect_tx(&bars->q_full, 2 * 9 * kBoxBytes);
          const int y = t.tok0 * H + t.row0 + static_cast<int>(rank) * kCtaRows;
          for (int c = 0; c < 9; ++c)
            pair_load_2d(smem + kOffQ + c * kBoxBytes, &tm_q, bar, 64 * c, y);
        }
      }
      for (int b = b0; ok && b < b1; b += 16) {
        // the next 32 page ids; a block's second page may lie past the last one and then is the
        // first again (its keys are masked, and its values cleared like those past the end)
        const int pg = min(2 * b + lane, pages - 1);
        int id = table[pg];
        if (id < 0 || id >= p.num_pages) {
          if (keys) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
          id = 0;
        }
        for (int k = 0; ok && k < min(16, b1 - b); ++k, ++n) {
          const int y0 = __shfl_sync(0xffffffffu, id, 2 * k) * kPage;
          const int y1 = __shfl_sync(0xffffffffu, id, 2 * k + 1) * kPage;
          // keys of this block that the sequence holds
          const int held = t.len - (b + k) * kBlock;
          const bool ragged = held < kBlock;
          if (keys) {
            const int y = rank ? y1 : y0;
#pragma unroll
            for (int u = 0; u < kKUnits; ++u) {
              if (ok && n > 0) ok = warp_wait_noted(&bars->k_empty[u], (n - 1) & 1, wc, note, kLeftUnit + u);
              if (ok && elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(&bars->k_full[u], 2 * kKUnit);
                const uint32_t bar = mapa_shared(smem_u32(&bars->k_full[u]), 0);
#pragma unroll
                for (int c = 0; c < 3; ++c)
                  pair_load_2d(smem + kOffK + u * kKUnit + c * kBoxBytes, &tm_c, bar,
                               64 * (3 * u + c), y);
              }
            }
            continue;
          }
#pragma unroll
          for (int u = 0; u < kVUnits; ++u) {
            if (ok && n > 0)
              ok = warp_wait_noted(&bars->v_empty[u], (n - 1) & 1, wc, note,
                                   (ragged ? kLeftRagged : kLeftUnit) + u);
            if (ok && elect_one()) {
              const uint32_t bar = ragged ? smem_u32(&bars->v_tail[u])
                                          : mapa_shared(smem_u32(&bars->v_full[u]), 0);
              arrive_expect_tx_cluster(bar, kVUnit);
#pragma unroll
              for (int c = 0; c < 2; ++c)
                pair_load_2d(smem + kOffV + u * kVUnit + c * kBoxBytes, &tm_c, bar,
                             256 * (u & 1) + 128 * static_cast<int>(rank) + 64 * c,
                             u >> 1 ? y1 : y0);
            }
          }
          if (!ragged) continue;
          // what the pool holds past the sequence's end must not reach the product: a weight of
          // zero does not silence a NaN
          for (int u = 0; ok && u < kVUnits; ++u) {
            if (!(ok = warp_wait_noted(&bars->v_tail[u], tails & 1, wc, note, kLeftTail + u))) break;
            for (int i = lane; i < 2 * 64 * 8; i += 32) {
              const int key = (i >> 3) & 63;
              if (64 * (u >> 1) + key >= held)
                *reinterpret_cast<uint4*>(smem + kOffV + u * kVUnit + 16 * i) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_cluster(mapa_shared(smem_u32(&bars->v_full[u]), 0));
          }
          ++tails;
        }
      }
      ++sg;
    }
    if (lane == 0) {
      bars->blocks[warp] = n;
      bars->rest[warp] = keys ? sg : tails;
    }
    // the last releases arrive at both CTAs' barriers; a CTA does not exit before it has seen them
    if (ok && n > 0 && lane == 0) {
      if (keys) {
        mbar_wait(&bars->q_empty, (sg - 1) & 1, wc);
        for (int u = 0; u < kKUnits; ++u) mbar_wait(&bars->k_empty[u], (n - 1) & 1, wc);
      } else {
        for (int u = 0; u < kVUnits; ++u) mbar_wait(&bars->v_empty[u], (n - 1) & 1, wc);
      }
    }
  } else if (warp == 5 || warp == 7) {
    // =================== MMA issuers (the leader's): S (warp 5), O (warp 7) ===================
    if (rank == 0) {
      const auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
      bool ok = true;
      int n = 0, sg = 0;  // blocks and non-empty segments so far
      if (warp == 5) {
        const uint32_t id_s = idesc_bf16(kTileRows, kBlock, 0, 0);
        const uint64_t d_q = smem_desc(smem_u32(smem + kOffQ), 16, 1024, kSwizzle128B);
        const uint64_t d_k = smem_desc(smem_u32(smem + kOffK), 16, 1024, kSwizzle128B);
        while (ok && it.next(seg)) {
          const int b0 = seg.b0, b1 = seg.b1;
          if (b0 == b1) continue;
          ok = warp_wait(&bars->q_full, sg & 1, wc);
          for (int b = b0; ok && b < b1; ++b, ++n) {
            if (n >= 2) ok = warp_wait<true>(&bars->s_free[n & 1], ((n >> 1) - 1) & 1, wc);
#pragma unroll
            for (int u = 0; u < kKUnits; ++u) {
              ok = ok && warp_wait(&bars->k_full[u], n & 1, wc);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int c = 0; c < 3; ++c)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    pair_mma_ss(tmem + kTmemS + 64 * (n & 1),
                                at(d_q, (3 * u + c) * kBoxBytes + 32 * k),
                                at(d_k, u * kKUnit + c * kBoxBytes + 32 * k), id_s,
                                u > 0 || c > 0 || k > 0);
                pair_commit(&bars->k_empty[u]);
                if (u == kKUnits - 1) {
                  pair_commit(&bars->s_full[n & 1]);
                  if (b + 1 == b1) pair_commit(&bars->q_empty);
                }
              }
            }
          }
          ++sg;
        }
      } else {
        const uint32_t id_o = idesc_bf16(kTileRows, 256, 0, 1);
        const uint64_t d_p = smem_desc(smem_u32(smem + kOffP), 16, 1024, kSwizzle128B);
        const uint64_t d_v = smem_desc(smem_u32(smem + kOffV), kBoxBytes, 1024, kSwizzle128B);
        while (ok && it.next(seg)) {
          const int b0 = seg.b0, b1 = seg.b1;
          if (b0 == b1) continue;
          if (sg > 0) ok = warp_wait<true>(&bars->o_free, (sg - 1) & 1, wc);
          for (int b = b0; ok && b < b1; ++b, ++n) {
            ok = warp_wait<true>(&bars->p_full, n & 1, wc);
#pragma unroll
            for (int u = 0; u < kVUnits; ++u) {
              ok = ok && warp_wait<true>(&bars->v_full[u], n & 1, wc);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  pair_mma_ss(tmem + kTmemO + 128 * (u & 1), at(d_p, (u >> 1) * kBoxBytes + 32 * k),
                              at(d_v, u * kVUnit + 2048 * k), id_o, u > 1 || k > 0 || b > b0);
                pair_commit(&bars->v_empty[u]);
                if (u == kVUnits - 1) pair_commit(&bars->pv_done);
              }
            }
          }
          ++sg;
        }
      }
      if (elect_one()) pair_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, drain_ctx);
    }
  } else {
    // =================== softmax, O rescale, epilogue ===================
    // lane L = 32 warp + lane of TMEM: row L % 64 of this CTA, keys 64 half ... + 63 of a block
    const int L = 32 * warp + lane, row = L & 63, half = L >> 6, r = static_cast<int>(rank) * kCtaRows + row;
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const uint32_t s_free0 = mapa_shared(smem_u32(&bars->s_free[0]), 0);
    const uint32_t p_full = mapa_shared(smem_u32(&bars->p_full), 0);
    const uint32_t o_free = mapa_shared(smem_u32(&bars->o_free), 0);
    const int pair_id = 1 + (warp & 1);
    const float NEG_INF = -__int_as_float(0x7f800000);
    // After a wait that ran out, a warp goes through the rest without work: its partner must not be
    // left alone at one of their barriers.
    bool ok = true;
    int n = 0;
    while (it.next(seg)) {
      const Tile t = seg.t;
      const int b0 = seg.b0, b1 = seg.b1;
      const int vis = r < t.rows ? t.visible(r, H) : 0;
      float m_ref = NEG_INF, l_sum = 0.f;
      for (int b = b0; b < b1; ++b, ++n) {
        const int pb = n & 1;
        if (!(ok = ok && warp_wait(&bars->s_full[pb], (n >> 1) & 1, wc))) {
          pair_barrier(pair_id);
          continue;
        }
        tc_fence_after();
        uint32_t x[2][32];
        tmem_ld32(tmem + kTmemS + 64 * pb + lanes, x[0]);
        tmem_ld32(tmem + kTmemS + 64 * pb + 32 + lanes, x[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(s_free0 + 8 * pb);
        float s[64];
        const int valid = vis - b * kBlock - 64 * half;
#pragma unroll
        for (int k = 0; k < 64; ++k) s[k] = __uint_as_float(x[k >> 5][k & 31]);
        if (valid < 64) {
#pragma unroll
          for (int k = 0; k < 64; ++k) s[k] = k < valid ? s[k] : NEG_INF;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int k = 4; k < 60; k += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3f(mx[i], s[k + i], s[k + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[60 + i]);
        float m = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
        bars->xch[pb][L] = m;
        pair_barrier(pair_id);
        m = fmaxf(m, bars->xch[pb][L ^ 64]);
        float alpha = 1.f;
        bool move = false;
        if (b == b0) {
          m_ref = fmaxf(m, kLowest);
        } else if (m > m_ref + kRescaleThreshold) {
          alpha = ex2_approx(m_ref - m);
          m_ref = m;
          move = true;
        }
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nb2 = f2_pack(-m_ref, -m_ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[2 * k], s[2 * k + 1]), sc2, nb2), x0, x1);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          acc[k & 3] = f2_add(acc[k & 3], f2_pack(x0, x1));
          pk[k] = pack_bf16x2(x0, x1);
        }
        float a0, a1;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
        l_sum = l_sum * alpha + (a0 + a1);
        // P and O are free once the previous block's O is added
        if (n > 0 && !(ok = warp_wait(&bars->pv_done, (n - 1) & 1, wc))) continue;
        if (__any_sync(0xffffffffu, move)) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            tmem_ld32(tmem + kTmemO + c + lanes, x[0]);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              x[0][k] = __float_as_uint(__uint_as_float(x[0][k]) * alpha);
            tmem_st32(tmem + kTmemO + c + lanes, x[0]);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        uint8_t* dst = smem + kOffP + half * kBoxBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(dst + 16 * (c ^ (row & 7))) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cluster(p_full);
      }
      // ---- O / l -> global ----
      const bool whole = !seg.split;
      const int slot = partial_slot(part, seg.inside);
      const int64_t out = whole ? static_cast<int64_t>(t.tok0) * H + t.row0 + r
                                : static_cast<int64_t>(slot) * kTileRows + r;
      const bool in = r < t.rows || !whole;  // (a partial result has all rows; the rest are zero)
      // the sums of the row's two halves; the block before last used the same places, and its
      // readers have passed a barrier since
      bars->xch[n & 1][L] = l_sum;
      pair_barrier(pair_id);
      l_sum += bars->xch[n & 1][L ^ 64];
      pair_barrier(pair_id);
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;  // (a NaN stays one)
      if (b1 > b0) ok = ok && warp_wait(&bars->pv_done, (n - 1) & 1, wc);
      if (!ok) continue;
      tc_fence_after();
#pragma unroll 2
      for (int c = 0; c < 256; c += 32) {
        uint32_t x[32];
        __syncwarp();
        if (b1 > b0) {
          tmem_ld32(tmem + kTmemO + c + lanes, x);
          tmem_wait_ld();
        }
        if (!in) continue;
        if (l_sum == 0.f) {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0u;
        }
        const int64_t col = 256 * (c >> 7) + 128 * half + (c & 127);
        if (whole && !p.o_f32) {
          __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.o) + out * kDc + col;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(x[8 * k + 2 * i]) * inv,
                                 __uint_as_float(x[8 * k + 2 * i + 1]) * inv);
            reinterpret_cast<uint4*>(d)[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          // a row's columns, or its place among the rows of each group of four
          float4* d = whole ? reinterpret_cast<float4*>(static_cast<float*>(p.o) + out * kDc + col)
                            : reinterpret_cast<float4*>(p.part_o) +
                                  (static_cast<int64_t>(slot) * (kDc / 4) + col / 4) * kTileRows + r;
          const int step = whole ? 1 : kTileRows;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            d[k * step] = make_float4(
                __uint_as_float(x[4 * k]) * inv, __uint_as_float(x[4 * k + 1]) * inv,
                __uint_as_float(x[4 * k + 2]) * inv, __uint_as_float(x[4 * k + 3]) * inv);
        }
      }
      float* lse = whole ? p.lse : p.part_lse;
      if (in && half == 0 && lse)
        lse[out] = l_sum == 0.f ? NEG_INF : (m_ref + log2f(l_sum)) * 0.69314718055994531f;
      if (b1 > b0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(o_free);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5 && lane == 0 && rank == 1) mbar_wait(&bars->drain, 0, drain_ctx);
  __syncwarp();
  cluster_sync();
  // After an abort the leader waits for the copies of both CTAs, whose shared memory nothing may
  // write any more when they exit (a unit's phase is issued only when its last one has been used, so
  // that the last of all is the only one that can be open).  Remote arrivals that nobody waited for may
  // still be on their way too.
  if (bars->abort_flag != 0 || pair_peer_word(&bars->abort_flag, rank) != 0) {
    if (warp == 4 || warp == 6) issued_loads(bars, warp, lane, drain_ctx);
    __syncwarp();
    __syncthreads();
    cluster_sync();
    if (rank == 0 && threadIdx.x < kLoadBars) {
      const int b = threadIdx.x, mine = bars->loads[b], others = pair_peer_word(&bars->loads[b], 0);
      pair_close(&bars->q_full + b, max(mine, others) - 1, mine >= others, others >= mine,
                 b == 0 ? 9 * kBoxBytes : b <= kKUnits ? kKUnit : kVUnit, b > kKUnits, drain_ctx);
    }
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000) {
    }
    __syncwarp();
  }
  cluster_sync();
  if (warp == 5) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace chunk
}  // namespace mla
