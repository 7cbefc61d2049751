// Causal attention over whole packed prompts (prompt_sm100.cuh) on pairs of SMs, for long sequences:
// every product is one tcgen05.mma over both SMs (cta_group::2, M = 256).
//
// A pair takes 512 query rows of one head as two tiles of 256, of which each CTA holds 128 rows with
// their S, P and O.  Each CTA loads half of every key box (64 of its 128 keys) and half of the
// values' columns, and the tensor cores read the other half from the neighbour: a CTA moves 40 KB
// for 128 keys where a CTA of its own moves 80 KB, and its tensor core reads 6 KB instead of 8 KB of
// shared memory for a 128 x 128 x 16 product.  At full load the GPU runs at its power limit, so that
// this is what the rate depends on.
// One prompt of 16384 tokens, 32 query and 4 key heads: 2.36 ... 2.47 ms, 1.11 ... 1.16 PFLOP/s, where
// CTAs of their own take 2.48 ... 2.51 ms on the box of 2.37 ... 2.41.
// Softmax and tensor memory are those of prompt_sm100.cuh; the leader (CTA 0) issues for both, so
// barriers that it waits on collect both CTAs' arrivals.  A tile's products are issued by a warp of
// its own, in the order PV(j) S(j+1): neither tile's waits hold up the other (2.32 ms with one
// warp).  Three stages of keys and values let the tiles drift apart; the single CTA's ring does not
// (8192 tokens in six prompts: 1.05 ms with one issuer, 1.15 ms with two), so it has one.
#pragma once
#include "packed.cuh"
#include "prompt_sm100.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace prompt_pair {

using prompt::kTile;
constexpr int kRows = 4 * kTile;    // query rows of a pair
constexpr int kThreads = 352;       // 8 softmax warps (4 a tile), TMA producer, an MMA issuer a tile
constexpr uint32_t kBox = kTile * 128;   // 128 rows x 64 bf16
constexpr uint32_t kKStage = 3 * kBox / 2, kVStage = kBox;
constexpr int kStages = 3;
constexpr uint32_t kOffQ = 0;                            // [2 tiles][3 boxes]
constexpr uint32_t kOffK = kOffQ + 6 * kBox;             // [kStages][3 boxes of 64 keys]
constexpr uint32_t kOffV = kOffK + kStages * kKStage;    // [kStages][128 keys x 64 columns]
constexpr uint32_t kOffBar = kOffV + kStages * kVStage;
constexpr uint32_t kSmemBytes = kOffBar + 512;
static_assert(kSmemBytes <= 232448, "shared memory budget");
using prompt::kDrainNs;
using prompt::kLowest;
using prompt::kRescaleThreshold;
using prompt::kTmemCols;
using prompt::kTmemO;
using prompt::kTmemS;

// Barriers marked L are the leader's; the others are each CTA's own, a commit arrives at both.
struct Bars {
  uint64_t q_full[2];         // L: a tile's queries landed (bytes of both CTAs)
  uint64_t k_full[kStages];   // L: a key tile landed (bytes of both CTAs)
  uint64_t k_empty[kStages];  // a tile's S has read it (commit, one a tile)
  uint64_t v_full[kStages];   // L: both CTAs' halves of a value tile landed (2, and bytes)
  uint64_t v_empty[kStages];  // a tile's PV has read it (commit, one a tile)
  uint64_t v_tail;            // the sequence's last value tile landed, where it has to be cleared
  uint64_t s_full[2];         // a tile's S is written (commit)
  uint64_t p_half[2];         // L: the tile's softmax warps: P of 64 keys written, O rescaled (8)
  uint64_t p_full[2];         // L: the same: all of P written (8)
  uint64_t o_full[2];         // the tile's last PV is done (commit)
  uint64_t drain[2];          // an issuer's products are done (commit)
  uint64_t stall;             // nothing ever arrives here (test of a wait that runs out)
  uint32_t tmem_base;
  int steps[2], len;          // key tiles of the two query tiles, tokens: for the MMA issuers
  int abort_flag;
  int tiles_begun, left;      // of the producer, and where a wait that ran out left the last (0: nowhere)
  int k_loads, v_loads;       // from that, its key tiles, and its value tiles announced on v_full
};
static_assert(sizeof(Bars) <= 512, "barrier block");
enum { kLeftKeys = 1, kLeftValues, kLeftTail };

__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(168)
    pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v,
                const prompt::Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  griddep_launch_dependents();
  griddep_wait();
  int seq, index, count;
  packed::Span sp;
  const bool there = packed::warp_find_tile(p.cu, p.batch, p.n_tokens, kRows, blockIdx.x >> 1, seq,
                                            index, count, sp);
  if (blockIdx.x == 0 && blockIdx.y == 0) packed::check_offsets(p.cu, p.batch, p.n_tokens, p.status);
  if (!there) return;  // the whole pair
  // the sequence's last rows first: they have the most keys
  const int q0 = (count - 1 - index) * kRows, len = sp.size();
  const int h = blockIdx.y, hk = h / (p.n_heads / p.n_kv_heads);
  // key tiles of the two query tiles (the second may be empty); only the last one of all can hold
  // keys past the sequence
  const int n0 = (min(q0 + 2 * kTile, len) + kTile - 1) / kTile;
  const int n1 = q0 + 2 * kTile < len ? (min(q0 + 4 * kTile, len) + kTile - 1) / kTile : 0;
  const int n_max = max(n0, n1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_half[i], 8);
      mbar_init(&bars->p_full[i], 8);
      mbar_init(&bars->o_full[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);
      mbar_init(&bars->v_full[i], 2);
      mbar_init(&bars->v_empty[i], 2);
    }
    mbar_init(&bars->v_tail, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->drain[i], 1);
    mbar_init(&bars->stall, 1);
    bars->abort_flag = 0;
    bars->left = 0;
    bars->steps[0] = n0;
    bars->steps[1] = n1;
    bars->len = len;
    fence_mbar_init_cluster();
  }
  if (warp == 9) pair_tmem_alloc(&bars->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort_flag, p.status, p.wait_ns};
  volatile int never = 0;
  const WaitCtx drain_ctx{&never, p.status, kDrainNs};
  if (p.stall != 0) {
    if (stall_here(p.stall, warp, rank)) prompt::stall_warp(&bars->stall, wc);
    __syncwarp();
  }

  if (warp == 8) {
    // =================== TMA producer: this CTA's rows, keys and columns ===================
    bool ok = true;
    const auto load_q = [&](int t) {
      if (elect_one()) {
        const uint32_t bar = mapa_shared(smem_u32(&bars->q_full[t]), 0);
        if (rank == 0) mbar_arrive_expect_tx(&bars->q_full[t], 2 * 3 * kBox);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          pair_load_3d(smem + kOffQ + (3 * t + c) * kBox, &tm_q, bar, 64 * c, h,
                       sp.begin + q0 + (2 * t + rank) * kTile);
      }
    };
    load_q(0);
    int j = 0;
    for (; j < n_max; ++j) {
      const int s = j % kStages, y = sp.begin + j * kTile;
      if (j >= kStages)
        ok = warp_wait_noted(&bars->k_empty[s], (j / kStages - 1) & 1, wc, &bars->left, kLeftKeys);
      if (!ok) break;
      if (elect_one()) {
        const uint32_t bar = mapa_shared(smem_u32(&bars->k_full[s]), 0);
        if (rank == 0) mbar_arrive_expect_tx(&bars->k_full[s], 2 * kKStage);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          pair_load_3d(smem + kOffK + s * kKStage + c * (kBox / 2), c < 2 ? &tm_k : &tm_kr, bar,
                       c < 2 ? 64 * c : 0, c < 2 ? hk : 0, y + 64 * rank);
      }
      if (j == 0 && n1 > 0) load_q(1);
      if (j >= kStages)
        ok = warp_wait_noted(&bars->v_empty[s], (j / kStages - 1) & 1, wc, &bars->left, kLeftValues);
      if (!ok) break;
      // values past the sequence's end, among the last 16 keys that PV reads, are cleared first: a
      // weight of zero does not silence a NaN
      const int valid = len - j * kTile;
      const bool ragged = valid < kTile && (valid & 15);
      if (elect_one()) {
        const uint32_t bar = ragged ? smem_u32(&bars->v_tail)
                                    : mapa_shared(smem_u32(&bars->v_full[s]), 0);
        arrive_expect_tx_cluster(bar, kVStage);
        pair_load_3d(smem + kOffV + s * kVStage, &tm_v, bar, 64 * rank, hk, y);
      }
      if (ragged) {
        if (!(ok = warp_wait_noted(&bars->v_tail, 0, wc, &bars->left, kLeftTail))) break;
        const int end = (valid + 15) & ~15;
        for (int i = 8 * valid + lane; i < 8 * end; i += 32)
          *reinterpret_cast<uint4*>(smem + kOffV + s * kVStage + 16 * i) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cluster(mapa_shared(smem_u32(&bars->v_full[s]), 0));
      }
    }
    if (lane == 0) bars->tiles_begun = j;
    // the last releases arrive at both CTAs' barriers; a CTA does not exit before it has seen them
    if (ok)
      for (int i = max(0, n_max - kStages); i < n_max; ++i) {
        mbar_wait(&bars->k_empty[i % kStages], (i / kStages) & 1, wc);
        mbar_wait(&bars->v_empty[i % kStages], (i / kStages) & 1, wc);
      }
  } else if (warp >= 9) {
    // =================== MMA issuers (the leader's), one a tile ===================
    // (the counts are read back from shared memory: see prompt_sm100.cuh)
    if (rank == 0) {
      const int t = warp - 9;
      const volatile Bars* vb = bars;
      const int n = vb->steps[t], len = vb->len, n_max = max(n, vb->steps[t ^ 1]);
      const uint32_t id = idesc_bf16(2 * kTile, kTile, 0, 0), id_o = idesc_bf16(2 * kTile, 128, 0, 1);
      const uint64_t d_q = smem_desc(smem_u32(smem + kOffQ + 3 * t * kBox), 16, 1024, kSwizzle128B);
      const uint64_t d_k = smem_desc(smem_u32(smem + kOffK), 16, 1024, kSwizzle128B);
      const uint64_t d_v = smem_desc(smem_u32(smem + kOffV), kBox, 1024, kSwizzle128B);
      const uint32_t tS = tmem + kTmemS + kTile * t, tO = tmem + kTmemO + 128 * t;
      const auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
      bool ok = n == 0 || warp_wait(&bars->q_full[t], 0, wc);
      for (int j = -1; ok && j < n; ++j) {
        if (j >= 0) {  // O += P V
          const int s = j % kStages, steps = (min(kTile, len - j * kTile) + 15) / 16;
          const uint64_t b = at(d_v, s * kVStage);
          ok = warp_wait(&bars->v_full[s], (j / kStages) & 1, wc);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && warp_wait(half ? &bars->p_full[t] : &bars->p_half[t], j & 1, wc);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              if (steps == kTile / 16) {
#pragma unroll
                for (int k = 4 * half; k < 4 * half + 4; ++k)
                  pair_mma_ts(tO, tS + 8 * k, at(b, 2048 * k), id_o, k > 0 || j > 0);
              } else {
                for (int k = 4 * half; k < min(4 * half + 4, steps); ++k)
                  pair_mma_ts(tO, tS + 8 * k, at(b, 2048 * k), id_o, k > 0 || j > 0);
              }
              if (half) pair_commit(&bars->v_empty[s]);
              if (half && j == n - 1) pair_commit(&bars->o_full[t]);
            }
          }
        }
        if (j + 1 < n) {  // the next S, over P
          const int s = (j + 1) % kStages;
          if (!(ok = ok && warp_wait(&bars->k_full[s], ((j + 1) / kStages) & 1, wc))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              const uint64_t a = at(d_q, c * kBox), b = at(d_k, s * kKStage + c * (kBox / 2));
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pair_mma_ss(tS, at(a, 32 * k), at(b, 32 * k), id, c > 0 || k > 0);
            }
            pair_commit(&bars->k_empty[s]);
            pair_commit(&bars->s_full[t]);
          }
        }
      }
      // the steps of the other tile alone
      for (int j = n; ok && j < n_max; ++j) {
        if (j >= kStages)  // (not before this tile's share of the slot's last release)
          ok = warp_wait(&bars->k_empty[j % kStages], (j / kStages - 1) & 1, wc) &&
               warp_wait(&bars->v_empty[j % kStages], (j / kStages - 1) & 1, wc);
        if (ok && elect_one()) {
          pair_commit(&bars->k_empty[j % kStages]);
          pair_commit(&bars->v_empty[j % kStages]);
        }
      }
      // no MMA may be in flight when TMEM is released
      if (elect_one()) pair_commit(&bars->drain[t]);
      mbar_wait(&bars->drain[t], 0, drain_ctx);
    }
  } else {
    // =================== softmax: warps 4t ... 4t + 3 own tile t, a thread one row ==========
    const int t = warp >> 2, n = t ? n1 : n0;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + kTmemS + kTile * t + lanes, tO = tmem + kTmemO + 128 * t + lanes;
    const uint32_t p_half = mapa_shared(smem_u32(&bars->p_half[t]), 0);
    const uint32_t p_full = mapa_shared(smem_u32(&bars->p_full[t]), 0);
    const int q = q0 + (2 * t + rank) * kTile + 32 * (warp & 3) + lane;  // row of the sequence
    const float NEG_INF = -__int_as_float(0x7f800000);
    float m_ref = NEG_INF, l_sum = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(&bars->s_full[t], j & 1, wc))) break;
      tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, x[c]);
      tmem_wait_ld();
      float s[kTile];
#pragma unroll
      for (int k = 0; k < kTile; ++k) s[k] = __uint_as_float(x[k >> 5][k & 31]);
      const int seen = q + 1 - j * kTile;  // keys of this tile that the row sees
      if (seen - lane < kTile) {           // the warp's first row does not see all
#pragma unroll
        for (int k = 0; k < kTile; ++k) s[k] = k < seen ? s[k] : NEG_INF;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int k = 4; k < kTile; k += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mx[i] = k + 4 + i < kTile ? max3f(mx[i], s[k + i], s[k + 4 + i]) : fmaxf(mx[i], s[k + i]);
      }
      const float m = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
      float alpha = 1.f;
      bool move = false;
      if (j == 0) {
        m_ref = fmaxf(m, kLowest);
      } else if (m > m_ref + kRescaleThreshold) {
        alpha = ex2_approx(m_ref - m);
        m_ref = m;
        move = true;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t y[32];
          tmem_ld32(tO + c, y);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * alpha);
          tmem_st32(tO + c, y);
        }
        l_sum *= alpha;
      }
      const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nb2 = f2_pack(-m_ref, -m_ref);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[64 * c + 2 * k], s[64 * c + 2 * k + 1]), sc2, nb2), x0, x1);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          acc[k & 3] = f2_add(acc[k & 3], f2_pack(x0, x1));
          pk[k] = pack_bf16x2(x0, x1);
        }
        tmem_st32(tS + 32 * c, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(c ? p_full : p_half);
      }
      float a0, a1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
      l_sum += a0 + a1;
    }
    if (ok && n > 0 && warp_wait(&bars->o_full[t], 0, wc)) {
      tc_fence_after();
      const int64_t row = static_cast<int64_t>(sp.begin + q) * p.n_heads + h;
      const float inv = 1.f / l_sum;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t x[32];
        __syncwarp();
        tmem_ld32(tO + c, x);
        tmem_wait_ld();
        if (q < len) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * 128 + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(x[8 * k + 2 * i]) * inv,
                                 __uint_as_float(x[8 * k + 2 * i + 1]) * inv);
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (p.lse && q < len) p.lse[row] = (m_ref + log2f(l_sum)) * 0.69314718055994531f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp >= 9 && lane == 0 && rank == 1) mbar_wait(&bars->drain[warp - 9], 0, drain_ctx);
  __syncwarp();
  cluster_sync();
  // After an abort the leader waits for the copies of both CTAs, whose shared memory nothing may
  // write any more when they exit (a stage's copies are issued only when its last ones have been used,
  // so that only the last kStages of all can be open).  Remote arrivals that nobody waited for may still
  // be on their way too.
  if (bars->abort_flag != 0 || pair_peer_word(&bars->abort_flag, rank) != 0) {
    if (threadIdx.x == 0) {
      const int j = bars->tiles_begun, left = bars->left;
      bars->k_loads = left == kLeftValues || left == kLeftTail ? j + 1 : j;
      bars->v_loads = j;
      if (left == kLeftTail) mbar_wait(&bars->v_tail, 0, drain_ctx);
    }
    __syncwarp();
    __syncthreads();
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
      for (int t = 0; t < 2; ++t)  // (the queries are copied in any case)
        if (bars->steps[t] > 0) mbar_wait(&bars->q_full[t], 0, drain_ctx);
      const int mine_k = bars->k_loads, k = pair_peer_word(&bars->k_loads, 0), nk = max(mine_k, k);
      for (int j = max(0, nk - kStages); j < nk; ++j)
        pair_close(&bars->k_full[j % kStages], j / kStages, mine_k > j, k > j, kKStage, false, drain_ctx);
      const int mine_v = bars->v_loads, v = pair_peer_word(&bars->v_loads, 0), nv = max(mine_v, v);
      for (int j = max(0, nv - kStages); j < nv; ++j)
        pair_close(&bars->v_full[j % kStages], j / kStages, mine_v > j, v > j, kVStage, true, drain_ctx);
    }
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000) {
    }
    __syncwarp();
  }
  cluster_sync();
  if (warp == 9) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace prompt_pair
}  // namespace mla
