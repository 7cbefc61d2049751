// Causal attention over whole packed prompts on the tcgen05 tensor cores (bf16):
//   S = Q K^T (192 wide: 128 of the head's own key, 64 of the shared rotary key), online softmax,
//   O += P V (128 wide), for every sequence of the packed batch and every head.
//
// A CTA takes 256 query rows of one head as two tiles of 128, which share every key and value box
// that is loaded, and walks over the keys 128 at a time.  The two tiles alternate on the tensor
// core: while one tile's softmax runs on its 128 threads (a thread owns a row, so the maximum and
// the sum need no exchange), the other's products do.  Order of the products:
//   PV0(j) S0(j+1) PV1(j) S1(j+1) PV0(j+1) ...
//   * TMEM (512 columns): S0 | S1 | O0 | O1, 128 each.  P (bf16) overwrites the first half of its
//     own S and is the A operand of PV from there, half by half.
//   * Shared memory: the queries 96 KB, a ring of four 16 KB key boxes (128 keys x 64 columns;
//     three make a key tile, released one by one) and two 32 KB value tiles.
//   * The running maximum is a reference that moves only when it would grow by more than 2^8, so O
//     is hardly ever rescaled.  S(j) of a tile completes after PV(j-1) of the same tile, so O may
//     be touched as soon as S(j) is there.
// Statistics and O are fp32; P is rounded to bf16 for the tensor core (the sum adds the unrounded
// weights).
//
// A sequence's last key tile: columns past the row are masked, whatever they hold; PV stops at
// the last 16 keys that hold one of the sequence, and the values of the others among those 16 are
// set to zero first, since a weight of zero does not silence a NaN.
//
// The work is 640 flops per visible pair of rows and head.  8192 tokens in six prompts, 128 heads:
// 1.11 ... 1.15 ms, 0.81 ... 0.83 PFLOP/s, at 1.7 GHz (the power limit, 1 kW).  The tensor pipe is not
// full: 32% of its clocks with prompts of 2048 and 1000 tokens, 64 heads.  A tile's softmax (2100 clocks)
// and its products (1280) follow one another, since S(j+1) is written over all of S after PV(j) has read
// P from its first half; and a block's start and end (search, barriers, tensor memory, first copies,
// write-back) overlap with nothing, one block to an SM.  What was tried against the first: P in
// shared memory, so that S(j+1) need not wait for PV(j) (3.4 ms instead of 2.6 ms for one prompt of
// 16384: the ring shrinks to four boxes, and both operands of PV come from shared memory); an order
// between the two tiles' exponentials (2.64); a part of the exponentials as a polynomial on the FMA
// pipe (2.7 ... 3.0); one ring of eight boxes for keys and values (2.62 against 2.50).  Long prompts
// run on pairs of SMs (prompt_pair_sm100.cuh).
#pragma once
#include "packed.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace prompt {

constexpr int kTile = 128;          // query rows of a tile, keys of a step
constexpr int kRows = 2 * kTile;    // query rows of a CTA
constexpr int kThreads = 320;       // 8 softmax warps (4 a tile), TMA producer, MMA issuer
constexpr uint32_t kBox = kTile * 128;  // 128 rows x 64 bf16
constexpr int kKSlots = 4, kVSlots = 2;
constexpr uint32_t kOffQ = 0;                        // [2 tiles][3 boxes]
constexpr uint32_t kOffK = kOffQ + 6 * kBox;         // [kKSlots]
constexpr uint32_t kOffV = kOffK + kKSlots * kBox;   // [kVSlots][2 boxes]
constexpr uint32_t kOffBar = kOffV + kVSlots * 2 * kBox;
constexpr uint32_t kSmemBytes = kOffBar + 512;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// The reference of a row whose scores so far are all -inf (no key seen, or products beyond fp32): every
// weight is 0 under it, and any score that is finite moves it.
constexpr float kLowest = -3.402823466e38f;
constexpr uint64_t kDrainNs = 200000000ull;

struct Params {
  int n_tokens, batch, n_heads, n_kv_heads;
  const int32_t* cu;
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  unsigned int* status;
  uint64_t wait_ns;
  int stall;  // see host_stall
};

struct Bars {
  uint64_t q_full[2];         // TMA: a tile's queries landed (bytes)
  uint64_t k_full[kKSlots];   // TMA: a key box landed (bytes)
  uint64_t k_empty[kKSlots];  // MMA: both tiles' S have read it (commit)
  uint64_t v_full[kVSlots];   // TMA: a value tile landed (bytes)
  uint64_t v_empty[kVSlots];  // MMA: both tiles' PV have read it (commit)
  uint64_t s_full[2];         // MMA: a tile's S is written (commit)
  uint64_t p_half[2];         // the tile's four softmax warps: P of 64 keys written, O rescaled (4)
  uint64_t p_full[2];         // the same: all of P written (4)
  uint64_t o_full[2];         // MMA: the tile's last PV is done (commit)
  uint64_t drain;
  uint64_t stall;             // nothing ever arrives here (test of a wait that runs out)
  uint32_t tmem_base;
  int steps[2], len;          // key tiles of the two query tiles, tokens: for the MMA issuer
  int abort_flag;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// (a call: inlined, the wait costs six packed prompts of 8192 tokens 1167 instead of 1115 us, and one of
// 16384 on pairs 2.37 instead of 2.36 ms, of 2.35 without any)
static __device__ __noinline__ void stall_warp(uint64_t* bar, const WaitCtx& w) {
  (void)warp_wait(bar, 0, w);
}

// 168 registers: three of the ten warps share a sub-partition's 16384
__global__ void __maxnreg__(168)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v,
                  const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  int seq, index, count;
  packed::Span sp;
  const bool there = packed::warp_find_tile(p.cu, p.batch, p.n_tokens, kRows, blockIdx.x, seq,
                                            index, count, sp);
  if (blockIdx.x == 0 && blockIdx.y == 0) packed::check_offsets(p.cu, p.batch, p.n_tokens, p.status);
  if (!there) return;  // the whole block
  // the sequence's last rows first: they have the most keys
  const int q0 = (count - 1 - index) * kRows, len = sp.size();
  const int h = blockIdx.y, hk = h / (p.n_heads / p.n_kv_heads);
  // key tiles of the two query tiles (the second may be empty); only the last one of all can hold
  // keys past the sequence
  const int n0 = q0 / kTile + 1, n1 = q0 + kTile < len ? n0 + 1 : 0, n_max = max(n0, n1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_half[i], 4);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_full[i], 1);
    }
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->stall, 1);
    bars->abort_flag = 0;
    bars->steps[0] = n0;
    bars->steps[1] = n1;
    bars->len = len;
    fence_mbar_init_cluster();
  }
  if (warp == 9) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort_flag, p.status, p.wait_ns};
  volatile int never = 0;
  const WaitCtx drain_ctx{&never, p.status, kDrainNs};
  if (p.stall != 0 && stall_here(p.stall, warp, 0)) stall_warp(&bars->stall, wc);

  if (warp == 8) {
    // =================== TMA producer ===================
    bool ok = true;
    int kb = 0, vb = 0;
    const auto load_q = [&](int t) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bars->q_full[t], 3 * kBox);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          tma_load_3d(smem + kOffQ + (3 * t + c) * kBox, &tm_q, &bars->q_full[t], 64 * c, h,
                      sp.begin + q0 + t * kTile);
      }
    };
    load_q(0);
    for (int j = 0; ok && j < n_max; ++j) {
      const int y = sp.begin + j * kTile;
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const int s = kb % kKSlots;
        if (kb >= kKSlots) ok = ok && warp_wait(&bars->k_empty[s], (kb / kKSlots - 1) & 1, wc);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->k_full[s], kBox);
          if (c < 2)
            tma_load_3d(smem + kOffK + s * kBox, &tm_k, &bars->k_full[s], 64 * c, hk, y);
          else
            tma_load_3d(smem + kOffK + s * kBox, &tm_kr, &bars->k_full[s], 0, 0, y);
        }
        ++kb;
      }
      if (j == 0 && n1 > 0) load_q(1);
      if (ok) {
        const int s = vb % kVSlots;
        if (vb >= kVSlots) ok = warp_wait(&bars->v_empty[s], (vb / kVSlots - 1) & 1, wc);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->v_full[s], 2 * kBox);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            tma_load_3d(smem + kOffV + (2 * s + c) * kBox, &tm_v, &bars->v_full[s], 64 * c, hk, y);
        }
        ++vb;
      }
    }
    // no copy may still be landing when the CTA exits (after an abort some may be in flight)
    mbar_wait(&bars->q_full[0], 0, drain_ctx);
    if (n1 > 0 && kb > 0) mbar_wait(&bars->q_full[1], 0, drain_ctx);
    for (int i = max(0, kb - kKSlots); i < kb; ++i)
      mbar_wait(&bars->k_full[i % kKSlots], (i / kKSlots) & 1, drain_ctx);
    for (int i = max(0, vb - kVSlots); i < vb; ++i)
      mbar_wait(&bars->v_full[i % kVSlots], (i / kVSlots) & 1, drain_ctx);
  } else if (warp == 9) {
    // =================== MMA issuer ===================
    // (read back from shared memory: the compiler's code for the loop is 3% faster when it knows
    // nothing of where the numbers come from)
    const volatile Bars* vb = bars;
    const int n0 = vb->steps[0], n1 = vb->steps[1], len = vb->len, n_max = max(n0, n1);
    const uint32_t id_s = idesc_bf16(kTile, kTile, 0, 0), id_o = idesc_bf16(kTile, 128, 0, 1);
    const uint64_t d_q = smem_desc(smem_u32(smem + kOffQ), 16, 1024, kSwizzle128B);
    const uint64_t d_k = smem_desc(smem_u32(smem + kOffK), 16, 1024, kSwizzle128B);
    const uint64_t d_v = smem_desc(smem_u32(smem + kOffV), kBox, 1024, kSwizzle128B);
    const auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
    bool ok = true;
    // S_t(j); the first tile to use a key box waits for it, the last one releases it
    const auto issue_s = [&](int t, int j) {
      const bool first = t == 0 || j >= n0, last = t == 1 || j >= n1;
      if (j == 0) ok = ok && warp_wait(&bars->q_full[t], 0, wc);
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const int kb = 3 * j + c, s = kb % kKSlots;
        if (first) ok = ok && warp_wait(&bars->k_full[s], (kb / kKSlots) & 1, wc);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = at(d_q, (3 * t + c) * kBox), b = at(d_k, s * kBox);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + kTmemS + kTile * t, at(a, 32 * k), at(b, 32 * k), id_s, c > 0 || k > 0);
          if (last) mma_commit(&bars->k_empty[s]);
          if (c == 2) mma_commit(&bars->s_full[t]);
        }
      }
    };
    const auto issue_pv = [&](int t, int j) {
      const bool first = t == 0 || j >= n0, last = t == 1 || j >= n1;
      const int s = j % kVSlots;
      if (first) ok = ok && warp_wait(&bars->v_full[s], (j / kVSlots) & 1, wc);
      const int steps = (min(kTile, len - j * kTile) + 15) / 16;
      const uint64_t b = at(d_v, 2 * s * kBox);
      const uint32_t o = tmem + kTmemO + 128 * t, a = tmem + kTmemS + kTile * t;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && warp_wait(half ? &bars->p_full[t] : &bars->p_half[t], j & 1, wc);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          if (steps == kTile / 16) {
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
              mma_ts(o, a + 8 * k, at(b, 2048 * k), id_o, k > 0 || j > 0);
          } else {
            for (int k = 4 * half; k < min(4 * half + 4, steps); ++k)
              mma_ts(o, a + 8 * k, at(b, 2048 * k), id_o, k > 0 || j > 0);
          }
          if (half && last) mma_commit(&bars->v_empty[s]);
          if (half && j == (t ? n1 : n0) - 1) mma_commit(&bars->o_full[t]);
        }
      }
    };
    issue_s(0, 0);
    if (n1 > 0) issue_s(1, 0);
    for (int j = 0; ok && j < n_max; ++j) {
      if (j < n0) {
        issue_pv(0, j);
        if (ok && j + 1 < n0) issue_s(0, j + 1);
      }
      if (ok && j < n1) {
        issue_pv(1, j);
        if (ok && j + 1 < n1) issue_s(1, j + 1);
      }
    }
    // no MMA may be in flight when TMEM is released
    if (elect_one()) mma_commit(&bars->drain);
    mbar_wait(&bars->drain, 0, drain_ctx);
  } else {
    // =================== softmax: warps 4t ... 4t + 3 own tile t, a thread one row ==========
    const int t = warp >> 2, n = t ? n1 : n0;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + kTmemS + kTile * t + lanes, tO = tmem + kTmemO + 128 * t + lanes;
    const int r = 32 * (warp & 3) + lane;
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
      if (j == n - 1) {  // the diagonal tile (n - 1 = the query tile's own place)
#pragma unroll
        for (int k = 0; k < kTile; ++k) s[k] = k <= r ? s[k] : NEG_INF;
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
          uint32_t x[32];
          tmem_ld32(tO + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
          tmem_st32(tO + c, x);
        }
        l_sum *= alpha;
      }
      // values past the sequence's end, among the last 16 keys that PV reads
      const int valid = len - j * kTile;
      if (valid < kTile && (valid & 15)) {
        const int sv = j % kVSlots;
        if (!(ok = warp_wait(&bars->v_full[sv], (j / kVSlots) & 1, wc))) break;
        const int end = (valid + 15) & ~15;
        if (r >= valid && r < end)
          for (int c = 0; c < 2; ++c)
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(smem + kOffV + (2 * sv + c) * kBox + r * 128 + 16 * k) =
                  make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
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
        if (lane == 0) mbar_arrive(c ? &bars->p_full[t] : &bars->p_half[t]);
      }
      float a0, a1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
      l_sum += a0 + a1;
    }
    if (ok && n > 0 && warp_wait(&bars->o_full[t], 0, wc)) {
      tc_fence_after();
      const int q = q0 + t * kTile + r;
      const int64_t row = static_cast<int64_t>(sp.begin + q) * p.n_heads + h;
      const float inv = 1.f / l_sum;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t x[32];
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
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace prompt
}  // namespace mla
