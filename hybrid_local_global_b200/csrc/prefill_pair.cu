// prefill_pair.cu -- prefill attention on CTA pairs: two 128-row query tiles
// of one (batch, q head) on two SMs that share each tcgen05 MMA
// (cta_group::2, M = 256), head_dim 256 and 512; below it k_prefill_stream,
// such pairs for prompts of head_dim 256 with a window plus sinks.
//
// Computes, for every query row i of a (batch, q head) and its KV head
// g = h / (Hq/Hkv) ("Gemma 4: End-to-End Architecture Walkthrough", 3a/3b):
//   out_i = sum_j softmax_j(scale <q~_i, k~_j>) v_j   over visible keys j
// where visible means j <= pos_i and, on a local layer, j > pos_i - window.
//
// Why pairs: in a 2-CTA MMA each SM supplies its own 128 rows of A (Q, or P
// from TMEM) and half of the N rows of B, so every K tile (128 keys) and V
// tile (256 output columns) is loaded and read from shared memory once per
// pair instead of once per query tile. A CTA's tile traffic halves
// (64 KB per key tile at head_dim 256, 96 KB at 512) and the TMA ring looks
// twice as far ahead.
//
// Cluster = 2 CTAs (x-adjacent), rank 0 the MMA leader. Per CTA, 192 threads:
//   warp 0     TMA producer (both CTAs): its own Q tile (D/64 boxes of 128
//              rows x 64 dims), then a ring of 32 KB stages in MMA order:
//              K_0, K_1, V_0, K_2, V_1, ... where its half of K_j is 64 keys
//              x D dims (D/256 stages) and its half of V_j is 128 keys x 128
//              output columns (one stage).
//              Both CTAs' loads of a stage complete on the leader's barrier
//              (cta_group::2 loads, no multicast), which expects both halves.
//   warp 1     TMEM owner (both CTAs); in the leader, the warp issues the
//              MMAs: S_j = Q K_j^T (M=256, N=128, K=D) into one of two
//              128-column TMEM buffers, then O += P_{j-1} V_{j-1} (M=256,
//              N=256, K=128) with P read from both CTAs' TMEM; commits arrive
//              on both CTAs' barriers.
//   warps 2-5  softmax (both CTAs), one query row per thread, as in the
//              single-CTA kernel; P_j is released to the leader's barrier.
// TMEM per CTA: O 0..255 (fp32), S/P buffers 256..383 and 384..511.
// head_dim 512 runs two pairs per query-tile pair (256 output columns
// each; the fp32 O tile of 128 x 512 would fill TMEM), each computing S.
//
// V rows past the sequence end must be finite (their P is 0, but 0 * inf is
// nan): on the one key tile that crosses the end, the MMA warp clears those
// rows in both CTAs' stages before the P.V product.
//
// Every wait is bounded by a %globaltimer deadline. On a timeout the CTA
// raises its abort flag and records GEMMA_ERR_DEVICE_TIMEOUT; the leader
// drains its MMAs, both CTAs wait for their own loads, meet at a cluster
// barrier, free TMEM and exit.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "pair.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace hlg {

namespace {

constexpr int BM = 128, BN = 128, DV = 256;  // rows per CTA, keys per tile, output columns per pair
constexpr int KH = BN / 2;                   // keys of K per CTA
constexpr int VH = DV / 2;                   // V columns per CTA
constexpr int CHUNK_Q = BM * 128;            // Q box: 128 rows x 64 dims (16 KB)
constexpr int CHUNK_K = KH * 128;            // K box: 64 keys x 64 dims (8 KB)
constexpr int CHUNK_V = BN * 128;            // V box: 128 keys x 64 columns (16 KB)
constexpr int STAGE_B = 32768;
constexpr int ALIGN_B = 1024;
constexpr int SMEM_MAX = 232448;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_O = 0, COL_S = 256;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(256, BN, 0, 0);
constexpr uint32_t IDESC_PV = tc::idesc_bf16_f32(256, DV, 0, 1);
constexpr uint16_t BOTH = 0x3;

template <int NSTAGE>
struct Ctl {
  uint64_t q_full;            // leader: both CTAs' Q tiles landed
  uint64_t full[NSTAGE];      // leader: both CTAs' halves of the stage landed
  uint64_t empty[NSTAGE];     // MMAs done with the stage (both CTAs)
  uint64_t s_full[2];
  uint64_t p_ready[2];        // leader: 4 local + 4 peer softmax warps (SK: P_j completes phase j/2 of
                              // p_ready[j % 2]; else phase j of p_ready[0])
  uint64_t o_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued[NSTAGE];
  int consumed[NSTAGE];
  int q_issued, q_consumed;
};

template <int D>
struct PairCfg {
  static constexpr int Q_B = BM * D * 2;           // 64 KB / 128 KB
  static constexpr int K_STAGES = D / 256;          // stages per half K tile
  static constexpr int NV = D / DV;                 // pairs per (query-tile pair, head)
  static constexpr int NSTAGE = (SMEM_MAX - ALIGN_B - Q_B - 1024) / STAGE_B;  // 5 / 3
  static constexpr int SMEM = ALIGN_B + Q_B + NSTAGE * STAGE_B + (int)sizeof(Ctl<NSTAGE>);
  static_assert(NSTAGE >= 3 && SMEM <= SMEM_MAX, "shared memory plan");
};

struct PairArgs {
  int S, window, Hq, Hkv;
  float scale_log2;  // SK: factor of the logits
  int sinks;  // SK instances: positions below it stay visible to every query
  int64_t key_cap;
  const int32_t* seq_lens_before;
  bf16* out;
  float* lse;
  int* status;
  unsigned long long wait_ns;
  int kv_token_major;  // K/V map coordinates: 0 = (d, key, head, b), 1 = (d, head, key, b)
  int key_off_window;  // 1: K/V view row = position - (pos0 - window), else = position
  int n_pairs;         // query-tile pairs per (batch, head); with head_pair: query tiles
  // paged cache (head-major views of the pool): view row = position % page_size,
  // view batch = page_table[b * pages_per_seq + position / page_size]; null: contiguous
  const int32_t* page_table;
  int page_size, pages_per_seq, n_pages;
  int head_pair;       // 1: the CTAs take q heads 2p and 2p+1 of one query tile (same KV head)
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t deadline, int* status, int where, int a = 0,
                                         int b = 0, int c = 0) {
  bool ok = mbar_wait_bounded_at(bar, parity, abort_flag, deadline, status, where, a, b, c);
  return __all_sync(0xffffffffu, ok);
}

// P = 2^(x - mb) over the 128 logits of one row, packed to bf16 pairs, with
// eight independent partial sums (and, if TRACK, partial maxima).
// SCALED: P = 2^(c x - mb).
template <bool TRACK, bool SCALED>
__device__ __forceinline__ void exp_row(const uint32_t (&r)[4][32], float c, float mb, uint32_t (&pk)[2][32],
                                        float (&ls)[8], float (&mx)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    ls[u] = 0.f;
    if (TRACK) mx[u] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const float x0 = __uint_as_float(r[i >> 4][(2 * i) & 31]);
    const float x1 = __uint_as_float(r[i >> 4][(2 * i + 1) & 31]);
    if (TRACK) mx[i & 7] = fmaxf(mx[i & 7], fmaxf(x0, x1));
    const float p0 = tc::ex2(SCALED ? fmaf(x0, c, -mb) : x0 - mb), p1 = tc::ex2(SCALED ? fmaf(x1, c, -mb) : x1 - mb);
    ls[i & 7] += p0 + p1;
    pk[i >> 5][i & 31] = pack_bf16x2(p0, p1);
  }
}

__device__ __forceinline__ float max8(const float (&mx)[8]) {
  return fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
}

__device__ __forceinline__ float max_row(const uint32_t (&r)[4][32]) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int e = 0; e < 32; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(r[c][e]));
  return max8(mx);
}

// Zero V rows [r0, BN) of a stage (the whole warp): both 64-column boxes, in this CTA (local
// stores) and in the peer (distributed shared memory), then make the writes
// visible to the tensor core's reads.
__device__ __forceinline__ void clear_v_tail_pair(uint32_t stage, int r0, int lane) {
  const uint32_t peer = pair::map_to(stage, 1);
  const uint32_t self = pair::map_to(stage, 0);
  for (int i = lane; i < (BN - r0) * 16; i += 32) {
    const uint32_t off = (uint32_t)(((i >> 3) & 1) * CHUNK_V + (r0 + (i >> 4)) * 128 + (i & 7) * 16);
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(self + off), "r"(0) : "memory");
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(peer + off), "r"(0) : "memory");
  }
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

// SK: a window plus sinks (cache views): the key tiles of the sinks, then the
// tiles from the window's first one on.
template <int D, bool SK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(192, 1)
    k_prefill_pair(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                   const PairArgs a) {
  using Cfg = PairCfg<D>;
  constexpr int NSTAGE = Cfg::NSTAGE;
  constexpr int Q_B = Cfg::Q_B;
  extern __shared__ unsigned char sm_raw[];
  const uint32_t raw = smem_u32(sm_raw);
  const uint32_t base = (raw + ALIGN_B - 1) & ~uint32_t(ALIGN_B - 1);
  unsigned char* sm = sm_raw + (base - raw);
  const uint32_t sQ = base;
  const uint32_t sStage = base + Q_B;
  Ctl<NSTAGE>* ctl = reinterpret_cast<Ctl<NSTAGE>*>(sm + Q_B + NSTAGE * STAGE_B);
  volatile int* abort_flag = &ctl->abort;

  const uint32_t rank = pair::cta_rank();
  const bool leader = rank == 0;
  const int vh = blockIdx.y % Cfg::NV, b = blockIdx.z;
  const int pq = a.n_pairs - 1 - (int)(blockIdx.x >> 1);  // heaviest pairs first
  // query-tile pairs: rows pq0 .. pq0 + 255 of one head, rank r takes the
  // r-th 128; head pairs: rows pq0 .. pq0 + 127 of heads 2p and 2p + 1
  const int pq0 = a.head_pair ? pq * BM : pq * 2 * BM;      // first row of the pair
  const int span = a.head_pair ? BM : 2 * BM;               // rows the pair covers
  const int q0 = a.head_pair ? pq0 : pq0 + (int)rank * BM;  // first row of this CTA
  const int h = a.head_pair ? 2 * (int)(blockIdx.y / Cfg::NV) + (int)rank : (int)(blockIdx.y / Cfg::NV);
  const int g = h / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int64_t pos0 = a.seq_lens_before ? (int64_t)a.seq_lens_before[b] : 0;
  const int64_t n_keys = pos0 + a.S;
  // view row of a key = its position - koff (a gathered key window starts at pos0 - window)
  const int64_t koff = a.key_off_window ? pos0 - a.window : 0;
  if (pos0 < 0 || n_keys - koff > a.key_cap) {  // reported by the RoPE kernel; same for both CTAs
    if (SK) after_previous();
    return;
  }
  int64_t lo_first, hi_first, lo_last, hi_last;
  visible_range(pos0 + pq0, a.window, n_keys, &lo_first, &hi_first);
  visible_range(pos0 + min(pq0 + span - 1, a.S - 1), a.window, n_keys, &lo_last, &hi_last);
  const int64_t kt0 = lo_first / BN;
  int n_tiles = (int)(hi_last / BN - kt0 + 1);
  int n_st = 0;  // SK: tiles of the sinks, before tile kt0
  if (SK) {
    const int64_t sink_tiles = ((int64_t)a.sinks + BN - 1) / BN;
    n_st = (int)(sink_tiles < kt0 ? sink_tiles : kt0);
    n_tiles += n_st;
  }
  // first key of the j-th key tile
  const auto tile_key = [&](int j) -> int64_t { return (SK && j < n_st ? j : kt0 + j - n_st) * BN; };

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, 1);
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
      ctl->issued[s] = 0;
      ctl->consumed[s] = 0;
    }
    mbar_init(&ctl->s_full[0], 1);
    mbar_init(&ctl->s_full[1], 1);
    for (int u = 0; u < 2; ++u) mbar_init(&ctl->p_ready[u], 8);  // one arrival per softmax warp of either CTA
    mbar_init(&ctl->o_done[0], 1);
    mbar_init(&ctl->o_done[1], 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ctl->q_issued = 0;
    ctl->q_consumed = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    pair::tmem_alloc2(smem_u32(&ctl->tmem_base), TMEM_COLS);
    pair::tmem_relinquish2();
  }
  if (SK) after_previous();  // the rotation, beside which all of the above ran
  tc::fence_before_sync();
  __syncwarp();
  pair::cluster_sync();  // both CTAs' barriers exist before any remote arrive or commit
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    const uint32_t go = tc::elect_one();
    // both CTAs' halves complete on the leader's barriers, which expect both
    const uint32_t q_bar = pair::map_to(smem_u32(&ctl->q_full), 0);
    if (go) {
      tc::prefetch_tmap(&tm_q);
      tc::prefetch_tmap(&tm_k);
      tc::prefetch_tmap(&tm_v);
      if (leader) mbar_arrive_expect_tx(&ctl->q_full, 2 * Q_B);
      ctl->q_issued = 1;
    }
    __syncwarp();
    for (int c = 0; c < D / 64; ++c) pair::tma_load_4d_pair_if(go, sQ + c * CHUNK_Q, &tm_q, c * 64, h, q0, b, q_bar);
    int item = 0;
    bool ok = true;
    for (int j = 0; j <= n_tiles && ok; ++j) {
      for (int kind = 0; kind < 2 && ok; ++kind) {  // 0: K_j, 1: V_{j-1}
        if ((kind == 0 && j == n_tiles) || (kind == 1 && j == 0)) continue;
        int key0 = (int)(tile_key(j - kind) - koff);  // view row
        int kb = b;                                   // view batch
        if (a.page_table) {
          // tiles never straddle a page (page_size is a multiple of 128); a
          // tile past the sequence's pages holds no visible key: any page
          const int pi = key0 / a.page_size;
          kb = pi < a.pages_per_seq ? a.page_table[(int64_t)b * a.pages_per_seq + pi] : 0;
          if (kb < 0 || kb >= a.n_pages) {
            if (go && (int64_t)key0 < n_keys) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
            kb = 0;
          }
          key0 -= pi * a.page_size;
        }
        const int n_stg = kind == 0 ? Cfg::K_STAGES : 1;
        for (int hs = 0; hs < n_stg; ++hs, ++item) {
          const int s = item % NSTAGE;
          if (item >= NSTAGE &&
              !wait_all(&ctl->empty[s], ((item / NSTAGE) - 1) & 1, abort_flag, deadline, a.status, 31, item, s, j)) {
            ok = false;
            break;
          }
          const uint32_t dst = sStage + s * STAGE_B;
          const uint32_t bar = pair::map_to(smem_u32(&ctl->full[s]), 0);
          if (go) {
            if (leader) mbar_arrive_expect_tx(&ctl->full[s], 2 * STAGE_B);
            ctl->issued[s] += 1;
          }
          __syncwarp();
          if (kind == 0) {
            const int k0 = key0 + (int)rank * KH;  // this CTA's 64 keys
            for (int cc = 0; cc < 4; ++cc) {
              const int d0 = (hs * 4 + cc) * 64;
              if (a.kv_token_major)
                pair::tma_load_4d_pair_if(go, dst + cc * CHUNK_K, &tm_k, d0, g, k0, kb, bar);
              else
                pair::tma_load_4d_pair_if(go, dst + cc * CHUNK_K, &tm_k, d0, k0, g, kb, bar);
            }
          } else {
            const int c0 = vh * DV + (int)rank * VH;  // this CTA's 128 output columns
            for (int c = 0; c < 2; ++c) {
              if (a.kv_token_major)
                pair::tma_load_4d_pair_if(go, dst + c * CHUNK_V, &tm_v, c0 + c * 64, g, key0, kb, bar);
              else
                pair::tma_load_4d_pair_if(go, dst + c * CHUNK_V, &tm_v, c0 + c * 64, key0, g, kb, bar);
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader) {
      const uint32_t go = tc::elect_one();
      bool ok = wait_all(&ctl->q_full, 0, abort_flag, deadline, a.status, 30);
      if (ok && go) ctl->q_consumed = 1;
      const uint64_t dq = tc::smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(sStage, 16, 1024), dv = tc::smem_desc_sw128(sStage, CHUNK_V, 1024);
      int item = 0, taken = 0;
      for (int j = 0; j <= n_tiles && ok; ++j) {
        if (j < n_tiles) {
          const uint32_t d_s = tmem + COL_S + (uint32_t)(j & 1) * 128;
          for (int hs = 0; hs < Cfg::K_STAGES; ++hs, ++item) {
            const int s = item % NSTAGE;
            if (!wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 32, item, s, j)) {
              ok = false;
              break;
            }
            taken = item + 1;
            tc::fence_after_sync();
#pragma unroll
            for (int cc = 0; cc < 4; ++cc)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                pair::mma2_ss_if(go, d_s, dq + (uint64_t)(((hs * 4 + cc) * CHUNK_Q + kk * 32) >> 4),
                                 dk + (uint64_t)((s * STAGE_B + cc * CHUNK_K + kk * 32) >> 4), IDESC_S,
                                 (hs | cc | kk) != 0);
            pair::commit2_mc_if(go, smem_u32(&ctl->empty[s]), BOTH);
          }
          if (!ok) break;
          pair::commit2_mc_if(go, smem_u32(&ctl->s_full[j & 1]), BOTH);
        }
        if (j >= 1) {
          ok = __all_sync(0xffffffffu, pair::wait_bounded_cluster(&ctl->p_ready[SK ? (j - 1) & 1 : 0],
                                                                  (SK ? (j - 1) >> 1 : j - 1) & 1, abort_flag, deadline,
                                                                  a.status, 34, j, 0, 0));
          if (!ok) break;
          const uint32_t p_tm = tmem + COL_S + (uint32_t)((j - 1) & 1) * 128;
          const int s = item % NSTAGE;
          if (!wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 35, item, s, j)) {
            ok = false;
            break;
          }
          taken = item + 1;
          const int64_t rows_valid = n_keys - tile_key(j - 1);
          if (rows_valid < BN) {
            clear_v_tail_pair(sStage + s * STAGE_B, rows_valid > 0 ? (int)rows_valid : 0, lane);
            __syncwarp();
          }
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            pair::mma2_ts_if(go, tmem + COL_O, p_tm + kk * 8, dv + (uint64_t)((s * STAGE_B + kk * 2048) >> 4), IDESC_PV,
                             (j - 1 > 0 || kk) ? 1u : 0u);
          pair::commit2_mc_if(go, smem_u32(&ctl->empty[s]), BOTH);
          pair::commit2_mc_if(go, smem_u32(&ctl->o_done[(j - 1) & 1]), BOTH);
          ++item;
        }
      }
      // no MMA may be in flight when either CTA releases TMEM or shared memory
      pair::commit2_mc_if(go, smem_u32(&ctl->drain), BOTH);
      if (go)
        for (int s = 0; s < NSTAGE; ++s) ctl->consumed[s] = (taken + NSTAGE - 1 - s) / NSTAGE;
    }
    __syncwarp();
    // the leader's MMAs read both CTAs' shared memory and write both TMEMs
    if (lane == 0) {
      volatile int never = 0;
      mbar_wait_bounded_at(&ctl->drain, 0, &never, deadline + 200000000ull, a.status, 37, 0, 0, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax (both CTAs)
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(wq * 32) << 16);
    const bool row_valid = q0 + row < a.S;
    const uint32_t p_ready_addr = pair::map_to(smem_u32(&ctl->p_ready[0]), 0);
    int64_t lo, hi;
    visible_range(pos0 + (row_valid ? q0 + row : a.S - 1), a.window, n_keys, &lo, &hi);
    // SK: the queries carry a power of two of scale * log2(e), which leaves their
    // bits alone, and the rest of it (1 <= c < 2) is applied to the logits
    const float factor = SK ? a.scale_log2 : 1.f;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    int pv_seen = 0;  // P.V products whose completion this thread has consumed
    for (int j = 0; j < n_tiles; ++j) {
      const int64_t kb = tile_key(j);
      if (!wait_all(&ctl->s_full[j & 1], (j >> 1) & 1, abort_flag, deadline, a.status, 45, j)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t s_tm = tm + COL_S + (uint32_t)(j & 1) * 128;
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_tm + c * 32, r[c]);
      tc::tmem_wait_ld();
      // Logits arrive in log2 units (queries carry scale * log2 e). Keys this
      // row cannot see become -inf in place.
      if (!((kb >= lo || (SK && kb + BN <= a.sinks)) && kb + BN - 1 <= hi)) {
        const int64_t dlo = lo - kb, dhi = hi - kb;
        const int c_lo = (int)(dlo < -1 ? -1 : dlo > BN ? BN : dlo);
        const int c_hi = (int)(dhi > BN ? BN : dhi);
        const int c_sink = SK ? (int)(a.sinks - kb > BN ? BN : a.sinks - kb < 0 ? 0 : a.sinks - kb) : 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (SK) {
            // bits, not comparisons per element: three of ten tiles of a window of 1024 are
            // edge tiles, and each took 6000 cycles with chains of predicates, 2000 without
            const uint32_t vis = tc::visible_bits(c * 32, c_lo, c_hi, c_sink);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[c][e] = vis >> e & 1u ? r[c][e] : __float_as_uint(-INFINITY);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int col = c * 32 + e;
              if (col < c_lo || col > c_hi) r[c][e] = __float_as_uint(-INFINITY);
            }
          }
        }
      }
      // One speculative pass against the running max; a row redoes the tile
      // only when its max moved by more than 2^8. Warps with a row that has
      // seen no key yet take the max first.
      float mx[8], ls[8];
      uint32_t pk[2][32];
      bool need;
      float alpha = 1.f;
      if (__any_sync(0xffffffffu, m_used == -INFINITY)) {
        const float m_new = fmaxf(m_used, max_row(r) * factor);
        need = m_new > m_used + RESCALE_LOG2 || (m_used == -INFINITY && m_new != -INFINITY);
        if (need) {
          alpha = (m_used == -INFINITY) ? 0.f : tc::ex2(m_used - m_new);
          l *= alpha;
          m_used = m_new;
        }
        exp_row<false, SK>(r, factor, m_used == -INFINITY ? 0.f : m_used, pk, ls, mx);
      } else {
        exp_row<true, SK>(r, factor, m_used, pk, ls, mx);
        const float m_new = fmaxf(m_used, max8(mx) * factor);
        need = m_new > m_used + RESCALE_LOG2;
        if (need) {
          alpha = tc::ex2(m_used - m_new);
          l *= alpha;
          m_used = m_new;
          exp_row<false, SK>(r, factor, m_used, pk, ls, mx);
        }
      }
      if (j >= 1 && __any_sync(0xffffffffu, need)) {
        // O must be stable: wait for P_{j-1} V_{j-1}
        if (pv_seen < j) {
          if (!wait_all(&ctl->o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 46, j)) {
            ok = false;
            break;
          }
          pv_seen = j;
        }
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tc::tmem_ld32(tm + COL_O + c * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tc::tmem_st32(tm + COL_O + c * 32, o);
        }
        tc::tmem_wait_st();
      }
      l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
      tc::tmem_st32(s_tm, pk[0]);
      tc::tmem_st32(s_tm + 32, pk[1]);
      // consume P_{j-1} V_{j-1} before P_{j+1} V_{j+1} can complete the next
      // phase of the same barrier (parity waits must not fall two behind). Not
      // SK: P_j V_j need not wait for that news to come here and go back. S_j's
      // commit, which this thread waited for, covers P_{j-2} V_{j-2} and all
      // before it, so a wait for P_{j-1} V_{j-1} (above, and after the last tile)
      // has one phase to wait for; and P_{j+2} is not released before S_{j+2},
      // issued after P_j V_j, so a P-ready barrier per buffer of P is enough.
      if (!SK && j >= 1 && pv_seen < j) {
        if (!wait_all(&ctl->o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 46, j)) {
          ok = false;
          break;
        }
        pv_seen = j;
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      // one arrival per warp: a cluster-scope release per thread costs a
      // fence each, and the warp's stores are complete after wait::st
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&ctl->p_ready[SK ? j & 1 : 0]);
        else
          SK ? pair::arrive_remote_tmem(p_ready_addr + (j & 1) * 8) : pair::arrive_remote(p_ready_addr);
      }
    }
    if (ok)
      ok = wait_all(&ctl->o_done[(n_tiles - 1) & 1], ((n_tiles - 1) >> 1) & 1, abort_flag, deadline,
                    a.status, 47, n_tiles);
    // Epilogue: O / l as bf16 into this CTA's Q buffer (free once the last
    // MMA is done), as the 128-byte-swizzled boxes of the output map, then
    // TMA stores of whole rows (rows past the sequence end are clipped).
    unsigned char* sO = sm;  // Q buffer
    if (ok) {
      tc::fence_after_sync();
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[32];
        tc::tmem_ld32(tm + COL_O + c * 32, o);
        tc::tmem_wait_ld();
        unsigned char* box_row = sO + (c >> 1) * CHUNK_Q + row * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 w;
          w.x = pack_bf16x2(__uint_as_float(o[u * 8 + 0]) * inv, __uint_as_float(o[u * 8 + 1]) * inv);
          w.y = pack_bf16x2(__uint_as_float(o[u * 8 + 2]) * inv, __uint_as_float(o[u * 8 + 3]) * inv);
          w.z = pack_bf16x2(__uint_as_float(o[u * 8 + 4]) * inv, __uint_as_float(o[u * 8 + 5]) * inv);
          w.w = pack_bf16x2(__uint_as_float(o[u * 8 + 6]) * inv, __uint_as_float(o[u * 8 + 7]) * inv);
          const int unit = ((c & 1) * 4 + u) ^ (row & 7);
          *reinterpret_cast<uint4*>(box_row + unit * 16) = w;
        }
      }
      if (row_valid && a.lse && vh == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.S + q0 + row] =
            l > 0.f ? (m_used + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
    }
    fence_proxy_async_smem();
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the four softmax warps
    if (warp == 2 && lane == 0 && !*abort_flag && q0 < a.S) {
      for (int c = 0; c < DV / 64; ++c)
        tc::tma_store_4d(&tm_o, smem_u32(sO + c * CHUNK_Q), vh * DV + c * 64, h, q0, b);
      tc::bulk_commit();
      tc::bulk_wait_read0();
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // loads still in flight must land before shared memory is released. Both
    // CTAs' loads complete on the leader's barriers: the leader waits for the
    // phases it has armed; the peer, which has no barrier of its own to
    // watch, gives its loads a bounded 50 us.
    volatile int never = 0;
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    if (leader) {
      if (ctl->q_issued && !ctl->q_consumed) mbar_wait_bounded_at(&ctl->q_full, 0, &never, dl, a.status, 49, 0, 0, 0);
      for (int s = 0; s < NSTAGE; ++s)
        if (ctl->issued[s] > ctl->consumed[s])
          mbar_wait_bounded_at(&ctl->full[s], (ctl->issued[s] - 1) & 1, &never, dl, a.status, 49,
                               ctl->issued[s], s, ctl->consumed[s]);
    } else {
      const uint64_t until = globaltimer_ns() + 50000ull;
      while (globaltimer_ns() < until) {
      }
    }
  }
  __syncwarp();
  // neither CTA leaves while the other may still arrive on its barriers
  pair::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    pair::tmem_dealloc2(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// head_dim 256 with a window plus sinks. A row tile sees few key tiles there, so
// what surrounds them counts: of the 26 us that a CTA of one row tile took for a
// window of 1024, 8 were setup, the first loads and products, and the output.
// Here a pair of CTAs stays and walks row tiles: the key tiles of one follow
// those of the one before through the same ring and TMEM buffers. Its Q is
// loaded once the last S of the one before is done; its first S and softmax run
// beside the last P V, and only then is the output before it taken out of TMEM
// (which its first P V waits for), through 32 KB of shared memory of its own.
//
// Two warps per 32 rows run the softmax, each with half the columns: with one,
// a key tile took 3650 cycles, of which the softmax 2650; with two 2600, of
// which 1024 are its exponentials at the special-function rate and the products
// 2048. B1 S8191 Hq32 Hkv16, window 1024, 16 sinks: 355 us with one CTA per row
// tile, 239 so (1400 TFLOP/s counting the masked parts of edge tiles), the
// rotation before it another 97.
// ---------------------------------------------------------------------------
constexpr int STREAM_Q = BM * 256 * 2;
constexpr int STREAM_WARPS = 8;    // softmax warps
constexpr int STREAM_BOX = 4096;   // output box of a softmax warp: 32 rows x 64 columns
constexpr int STREAM_OUT = STREAM_WARPS * STREAM_BOX;
constexpr int STREAM_T = 64 + 32 * STREAM_WARPS;
constexpr int STREAM_NS = (SMEM_MAX - ALIGN_B - STREAM_Q - STREAM_OUT - 2048) / STAGE_B;  // 4
constexpr int STREAM_SMEM = ALIGN_B + STREAM_Q + STREAM_OUT + STREAM_NS * STAGE_B + 2048;
static_assert(STREAM_NS >= 3 && STREAM_SMEM <= SMEM_MAX, "shared memory plan");

struct StreamCtl {
  Ctl<STREAM_NS> ring;  // q_full and the others' phases run on from row tile to row tile
  uint64_t q_empty;     // the row tile's last S is done
  uint64_t o_free;      // leader: the row tile's output left TMEM (8 local + 8 peer warps)
  float part[2][BM];    // halves of a row: maxima, sums
};
static_assert(sizeof(StreamCtl) <= 2048, "control block");

// A pair's row tile(s) and the key tiles it sees.
struct RowTile {
  int b, h, g, q0;  // this CTA's
  int n_tiles, n_st;
  int64_t pos0, n_keys, kt0;
  __device__ __forceinline__ int64_t key(int j) const { return (j < n_st ? j : kt0 + j - n_st) * BN; }
};

// The i-th of a launch (long ones first within a head); false: its sequence's
// length is out of range, which the rotation reports.
__device__ __forceinline__ bool row_tile(const PairArgs& a, int i, int rank, RowTile* t) {
  const int ny = a.head_pair ? a.Hq / 2 : a.Hq;
  const int pq = a.n_pairs - 1 - i % a.n_pairs, y = i / a.n_pairs % ny;
  t->b = i / a.n_pairs / ny;
  const int first = a.head_pair ? pq * BM : pq * 2 * BM, span = a.head_pair ? BM : 2 * BM;
  t->q0 = a.head_pair ? first : first + rank * BM;
  t->h = a.head_pair ? 2 * y + rank : y;
  t->g = t->h / (a.Hq / a.Hkv);
  t->pos0 = a.seq_lens_before ? (int64_t)a.seq_lens_before[t->b] : 0;
  t->n_keys = t->pos0 + a.S;
  if (t->pos0 < 0 || t->n_keys > a.key_cap) return false;
  int64_t lo_first, hi_first, lo_last, hi_last;
  visible_range(t->pos0 + first, a.window, t->n_keys, &lo_first, &hi_first);
  visible_range(t->pos0 + min(first + span - 1, a.S - 1), a.window, t->n_keys, &lo_last, &hi_last);
  t->kt0 = lo_first / BN;
  const int64_t sink_tiles = ((int64_t)a.sinks + BN - 1) / BN;
  t->n_st = (int)(sink_tiles < t->kt0 ? sink_tiles : t->kt0);
  t->n_tiles = (int)(hi_last / BN - t->kt0 + 1) + t->n_st;
  return true;
}

// AND or OR of a predicate over the 64 threads of two warps.
template <bool AND>
__device__ __forceinline__ bool vote64(int id, bool p) {
  uint32_t r;
  if (AND)
    asm volatile("{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbar.red.and.pred po, %2, 64, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
                 : "=r"(r) : "r"((uint32_t)p), "r"(id) : "memory");
  else
    asm volatile("{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbar.red.or.pred po, %2, 64, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
                 : "=r"(r) : "r"((uint32_t)p), "r"(id) : "memory");
  return r != 0;
}

// exp_row and max_row over half a row.
template <bool TRACK>
__device__ __forceinline__ void exp_half(const uint32_t (&r)[2][32], float c, float mb, uint32_t (&pk)[32], float* sum,
                                         float* top) {
  float ls[8], mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    ls[u] = 0.f;
    mx[u] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float x0 = __uint_as_float(r[i >> 4][(2 * i) & 31]), x1 = __uint_as_float(r[i >> 4][(2 * i + 1) & 31]);
    if (TRACK) mx[i & 7] = fmaxf(mx[i & 7], fmaxf(x0, x1));
    const float p0 = tc::ex2(fmaf(x0, c, -mb)), p1 = tc::ex2(fmaf(x1, c, -mb));
    ls[i & 7] += p0 + p1;
    pk[i] = pack_bf16x2(p0, p1);
  }
  *sum = ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
  if (TRACK) *top = max8(mx);
}
__device__ __forceinline__ float max_half(const uint32_t (&r)[2][32]) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 32; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(r[c][e]));
  return max8(mx);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(STREAM_T, 1)
    k_prefill_stream(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const PairArgs a, const int n_items) {
  constexpr int NSTAGE = STREAM_NS, D = 256;
  extern __shared__ unsigned char sm_raw[];
  const uint32_t raw = smem_u32(sm_raw);
  const uint32_t base = (raw + ALIGN_B - 1) & ~uint32_t(ALIGN_B - 1);
  unsigned char* sm = sm_raw + (base - raw);
  const uint32_t sQ = base, sStage = base + STREAM_Q;
  constexpr int OUT_OFF = STREAM_Q + NSTAGE * STAGE_B;
  StreamCtl* sc = reinterpret_cast<StreamCtl*>(sm + OUT_OFF + STREAM_OUT);
  Ctl<NSTAGE>* ctl = &sc->ring;
  volatile int* abort_flag = &ctl->abort;

  const int rank = (int)pair::cta_rank();
  const bool leader = rank == 0;
  const int step = gridDim.x / 2, item0 = blockIdx.x / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, 1);
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
      ctl->issued[s] = 0;
      ctl->consumed[s] = 0;
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&ctl->s_full[u], 1);
      mbar_init(&ctl->o_done[u], 1);
    }
    for (int u = 0; u < 2; ++u) mbar_init(&ctl->p_ready[u], 2 * STREAM_WARPS);  // one per softmax warp of either CTA
    mbar_init(&ctl->drain, 1);
    mbar_init(&sc->q_empty, 1);
    mbar_init(&sc->o_free, 2 * STREAM_WARPS);
    ctl->abort = 0;
    ctl->q_issued = 0;
    ctl->q_consumed = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    pair::tmem_alloc2(smem_u32(&ctl->tmem_base), TMEM_COLS);
    pair::tmem_relinquish2();
  }
  after_previous();  // the rotation, beside which all of the above ran
  tc::fence_before_sync();
  __syncwarp();
  pair::cluster_sync();  // both CTAs' barriers exist before any remote arrive or commit
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  // Counters that run on over all row tiles: jt key tiles, n row tiles, item
  // ring stages. Deadlines are per row tile: a launch may be long.
  RowTile t;
  int jt = 0, n = 0;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    const uint32_t go = tc::elect_one();
    const uint32_t q_bar = pair::map_to(smem_u32(&ctl->q_full), 0);
    if (go) {
      tc::prefetch_tmap(&tm_q);
      tc::prefetch_tmap(&tm_k);
      tc::prefetch_tmap(&tm_v);
    }
    int item = 0;
    uint64_t deadline = 0;
    // one stage: K rows (this CTA's 64 keys) or V columns (its 128) of a key tile
    const auto load = [&](bool is_v, int b, int g, int64_t key, int64_t n_keys) -> bool {
      // tiles never straddle a page (page_size is a multiple of 128)
      int row = (int)key;
      const int pi = row / a.page_size;
      int kb = pi < a.pages_per_seq ? a.page_table[(int64_t)b * a.pages_per_seq + pi] : 0;
      if (kb < 0 || kb >= a.n_pages) {
        if (go && key < n_keys) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        kb = 0;
      }
      row -= pi * a.page_size;
      const int s = item % NSTAGE;
      if (item >= NSTAGE &&
          !wait_all(&ctl->empty[s], ((item / NSTAGE) - 1) & 1, abort_flag, deadline, a.status, 51, item, s, jt))
        return false;
      ++item;
      const uint32_t dst = sStage + s * STAGE_B, bar = pair::map_to(smem_u32(&ctl->full[s]), 0);
      if (go) {
        if (leader) mbar_arrive_expect_tx(&ctl->full[s], 2 * STAGE_B);
        ctl->issued[s] += 1;
      }
      __syncwarp();
      if (is_v) {
        for (int c = 0; c < 2; ++c)
          pair::tma_load_4d_pair_if(go, dst + c * CHUNK_V, &tm_v, rank * VH + c * 64, row, g, kb, bar);
      } else {
        for (int c = 0; c < 4; ++c)
          pair::tma_load_4d_pair_if(go, dst + c * CHUNK_K, &tm_k, c * 64, row + rank * KH, g, kb, bar);
      }
      return true;
    };
    const auto load_q = [&]() {
      if (go) {
        if (leader) mbar_arrive_expect_tx(&ctl->q_full, 2 * STREAM_Q);
        ctl->q_issued += 1;
      }
      __syncwarp();
      for (int c = 0; c < D / 64; ++c)
        pair::tma_load_4d_pair_if(go, sQ + c * CHUNK_Q, &tm_q, c * 64, t.h, t.q0, t.b, q_bar);
    };
    int vb = 0, vg = 0;  // the key tile before, whose V is loaded next
    int64_t vkey = 0, v_end = 0;
    for (int i = item0; i < n_items && ok; i += step) {
      if (!row_tile(a, i, rank, &t)) continue;
      deadline = globaltimer_ns() + a.wait_ns;
      if (n == 0) load_q();
      for (int j = 0; j < t.n_tiles && ok; ++j, ++jt) {
        ok = load(false, t.b, t.g, t.key(j), t.n_keys);
        if (ok && jt > 0) ok = load(true, vb, vg, vkey, v_end);
        if (ok && j == 0 && n > 0) {
          ok = wait_all(&sc->q_empty, (n - 1) & 1, abort_flag, deadline, a.status, 52, n);
          if (ok) load_q();
        }
        vb = t.b;
        vg = t.g;
        vkey = t.key(j);
        v_end = t.n_keys;
      }
      ++n;
    }
    if (ok && jt > 0) load(true, vb, vg, vkey, v_end);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader) {
      const uint32_t go = tc::elect_one();
      const uint64_t dq = tc::smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(sStage, 16, 1024), dv = tc::smem_desc_sw128(sStage, CHUNK_V, 1024);
      int item = 0, taken = 0;
      uint64_t deadline = 0;
      int64_t v_rows = 0;   // valid rows of the key tile before,
      bool v_first = true;  // the first of its row tile,
      int v_n = 0;          // number v_n
      const auto pv = [&](int k) -> bool {  // O (+)= P_k V_k
        if (v_first && v_n > 0 &&
            !__all_sync(0xffffffffu, pair::wait_bounded_cluster(&sc->o_free, (v_n - 1) & 1, abort_flag, deadline,
                                                                a.status, 56, k, v_n, 0)))
          return false;
        if (!__all_sync(0xffffffffu, pair::wait_bounded_cluster(&ctl->p_ready[k & 1], (k >> 1) & 1, abort_flag, deadline,
                                                                a.status, 54, k, v_n, 0)))
          return false;
        const int s = item % NSTAGE;
        if (!wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 55, item, s, k)) return false;
        taken = ++item;
        if (v_rows < BN) {
          clear_v_tail_pair(sStage + s * STAGE_B, v_rows > 0 ? (int)v_rows : 0, lane);
          __syncwarp();
        }
        tc::fence_after_sync();
        const uint32_t p_tm = tmem + COL_S + (uint32_t)(k & 1) * 128;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          pair::mma2_ts_if(go, tmem + COL_O, p_tm + (kk >> 2) * 64 + (kk & 3) * 8,
                           dv + (uint64_t)((s * STAGE_B + kk * 2048) >> 4), IDESC_PV, (!v_first || kk) ? 1u : 0u);
        pair::commit2_mc_if(go, smem_u32(&ctl->empty[s]), BOTH);
        pair::commit2_mc_if(go, smem_u32(&ctl->o_done[k & 1]), BOTH);
        return true;
      };
      for (int i = item0; i < n_items && ok; i += step) {
        if (!row_tile(a, i, rank, &t)) continue;
        deadline = globaltimer_ns() + a.wait_ns;
        for (int j = 0; j < t.n_tiles && ok; ++j, ++jt) {
          if (j == 0) {
            ok = wait_all(&ctl->q_full, n & 1, abort_flag, deadline, a.status, 50, n);
            if (!ok) break;
            if (go) ctl->q_consumed = n + 1;
          }
          const int s = item % NSTAGE;
          ok = wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 53, item, s, jt);
          if (!ok) break;
          taken = ++item;
          tc::fence_after_sync();
          const uint32_t d_s = tmem + COL_S + (uint32_t)(jt & 1) * 128;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              pair::mma2_ss_if(go, d_s, dq + (uint64_t)((cc * CHUNK_Q + kk * 32) >> 4),
                               dk + (uint64_t)((s * STAGE_B + cc * CHUNK_K + kk * 32) >> 4), IDESC_S, (cc | kk) != 0);
          pair::commit2_mc_if(go, smem_u32(&ctl->empty[s]), BOTH);
          pair::commit2_mc_if(go, smem_u32(&ctl->s_full[jt & 1]), BOTH);
          if (j == t.n_tiles - 1) pair::commit2_mc_if(go, smem_u32(&sc->q_empty), BOTH);
          if (jt > 0) ok = pv(jt - 1);
          v_rows = t.n_keys - t.key(j);
          v_first = j == 0;
          v_n = n;
        }
        ++n;
      }
      if (ok && jt > 0) pv(jt - 1);
      // no MMA may be in flight when either CTA releases TMEM or shared memory
      pair::commit2_mc_if(go, smem_u32(&ctl->drain), BOTH);
      if (go)
        for (int s = 0; s < NSTAGE; ++s) ctl->consumed[s] = (taken + NSTAGE - 1 - s) / NSTAGE;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax (both CTAs)
    // Two warps per 32 rows, each with half the columns of S and of O. A row's two
    // threads keep the same maximum: they vote on whether it has to move.
    const int wq = warp & 3, half = (warp - 2) >> 2;
    const int row = wq * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t p_ready_addr = pair::map_to(smem_u32(&ctl->p_ready[0]), 0);
    const uint32_t o_free_addr = pair::map_to(smem_u32(&sc->o_free), 0);
    unsigned char* box = sm + OUT_OFF + (warp - 2) * STREAM_BOX;
    // the row tile before, whose output still lies in TMEM
    float out_m = 0.f, out_l = 0.f;
    int out_b = 0, out_h = 0, out_q0 = 0;
    const auto put_out = [&]() {
      tc::fence_after_sync();
      const float inv = out_l > 0.f ? 1.f / out_l : 0.f;
#pragma unroll 1
      for (int c = half * 2; c < half * 2 + 2; ++c) {
        uint32_t o[2][32];
        tc::tmem_ld32(tm + COL_O + c * 64, o[0]);
        tc::tmem_ld32(tm + COL_O + c * 64 + 32, o[1]);
        tc::tmem_wait_ld();
        if (c & 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (leader)
              mbar_arrive(&sc->o_free);
            else
              pair::arrive_remote_tmem(o_free_addr);
          }
        }
        if (lane == 0) tc::bulk_wait_read0();  // the store before has read the box
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t* x = &o[u >> 2][(u & 3) * 8];
          uint4 w;
          w.x = pack_bf16x2(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv);
          w.y = pack_bf16x2(__uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
          w.z = pack_bf16x2(__uint_as_float(x[4]) * inv, __uint_as_float(x[5]) * inv);
          w.w = pack_bf16x2(__uint_as_float(x[6]) * inv, __uint_as_float(x[7]) * inv);
          *reinterpret_cast<uint4*>(box + lane * 128 + (u ^ (lane & 7)) * 16) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (out_q0 + wq * 32 < a.S)  // rows past the sequence end are clipped
            tc::tma_store_4d(&tm_o, smem_u32(box), c * 64, out_h, out_q0 + wq * 32, out_b);
          tc::bulk_commit();
        }
        __syncwarp();
      }
      if (half == 0 && out_q0 + row < a.S && a.lse)
        a.lse[((int64_t)out_b * a.Hq + out_h) * a.S + out_q0 + row] =
            out_l > 0.f ? (out_m + __log2f(out_l)) * 0.69314718055994530942f : -INFINITY;
    };
    uint64_t deadline = 0;
    // P V of the key tile before the current one is complete (all earlier ones are
    // since S of the current one is, so there is one phase to wait for)
    const auto pv_done = [&](int k) -> bool {
      return wait_all(&ctl->o_done[k & 1], (k >> 1) & 1, abort_flag, deadline, a.status, 58, k, n);
    };
    const float factor = a.scale_log2;
    // A warp that gave up (ok false) goes on to the next vote, at which both warps leave.
    for (int i = item0; i < n_items && ok; i += step) {
      if (!row_tile(a, i, rank, &t)) continue;
      deadline = globaltimer_ns() + a.wait_ns;
      const bool row_valid = t.q0 + row < a.S;
      int64_t lo, hi;
      visible_range(t.pos0 + (row_valid ? t.q0 + row : a.S - 1), a.window, t.n_keys, &lo, &hi);
      float m_used = -INFINITY, l = 0.f;
      bool left = false;  // both warps, at a vote
      for (int j = 0; j < t.n_tiles; ++j, ++jt) {
        const int64_t kb = t.key(j);
        ok = ok && wait_all(&ctl->s_full[jt & 1], (jt >> 1) & 1, abort_flag, deadline, a.status, 57, jt, n);
        tc::fence_after_sync();
        const uint32_t s_tm = tm + COL_S + (uint32_t)((jt & 1) * 128 + half * 64);
        uint32_t r[2][32];
        tc::tmem_ld32(s_tm, r[0]);
        tc::tmem_ld32(s_tm + 32, r[1]);
        tc::tmem_wait_ld();
        if (!((kb >= lo || kb + BN <= a.sinks) && kb + BN - 1 <= hi)) {
          const int64_t dlo = lo - kb, dhi = hi - kb;
          const int c_lo = (int)(dlo < -1 ? -1 : dlo > BN ? BN : dlo);
          const int c_hi = (int)(dhi > BN ? BN : dhi);
          const int c_sink = (int)(a.sinks - kb > BN ? BN : a.sinks - kb < 0 ? 0 : a.sinks - kb);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t vis = tc::visible_bits(half * 64 + c * 32, c_lo, c_hi, c_sink);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[c][e] = vis >> e & 1u ? r[c][e] : __float_as_uint(-INFINITY);
          }
        }
        // one speculative pass against the running maximum, unless a row has seen no key yet
        float mx, ls;
        uint32_t pk[32];
        const bool fresh = __any_sync(0xffffffffu, m_used == -INFINITY);
        if (fresh)
          mx = max_half(r);
        else
          exp_half<true>(r, factor, m_used, pk, &ls, &mx);
        float alpha = 1.f;
        bool need = false;
        if (vote64<false>(1 + wq, !ok || fresh || mx * factor > m_used + RESCALE_LOG2)) {
          sc->part[half][row] = mx;
          ok = vote64<true>(1 + wq, ok);
          left = !ok;
          if (left) break;
          const float m_new = fmaxf(m_used, fmaxf(mx, sc->part[half ^ 1][row]) * factor);
          need = m_new > m_used + RESCALE_LOG2 || (m_used == -INFINITY && m_new != -INFINITY);
          if (need) {
            alpha = (m_used == -INFINITY) ? 0.f : tc::ex2(m_used - m_new);
            l *= alpha;
            m_used = m_new;
          }
          if (fresh || need) exp_half<false>(r, factor, m_used == -INFINITY ? 0.f : m_used, pk, &ls, &mx);
        }
        if (j >= 1 && __any_sync(0xffffffffu, need)) {
          ok = pv_done(jt - 1);  // O must be stable
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < 4 && ok; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(tm + COL_O + half * 128 + c * 32, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st32(tm + COL_O + half * 128 + c * 32, o);
          }
        }
        l += ls;
        tc::tmem_st32(s_tm, pk);  // each half over its own columns of S
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) {
          if (leader)
            mbar_arrive(&ctl->p_ready[jt & 1]);
          else
            pair::arrive_remote_tmem(p_ready_addr + (jt & 1) * 8);
        }
        if (j == 0 && n > 0) {
          ok = ok && pv_done(jt - 1);
          if (ok) put_out();
        }
      }
      if (left) break;
      ok = vote64<true>(1 + wq, ok);  // the other half's maximum has been read
      sc->part[half][row] = l;
      ok = vote64<true>(1 + wq, ok);
      if (!ok) break;
      out_m = m_used;
      out_l = l + sc->part[half ^ 1][row];
      out_b = t.b;
      out_h = t.h;
      out_q0 = t.q0;
      ++n;
    }
    if (ok && n > 0) {
      ok = pv_done(jt - 1);
      if (ok) put_out();
    }
    if (lane == 0) tc::bulk_wait_read0();
    __syncwarp();
  }

  __syncwarp();
  __syncthreads();
  // the leader's MMAs read both CTAs' shared memory and write both TMEMs
  if (threadIdx.x == 32) {
    volatile int never = 0;
    mbar_wait_bounded_at(&ctl->drain, 0, &never, globaltimer_ns() + a.wait_ns + 200000000ull, a.status, 59, 0, 0, 0);
  }
  if (warp == 0 && lane == 0 && *abort_flag) {
    // loads still in flight must land: see k_prefill_pair
    volatile int never = 0;
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    if (leader) {
      if (ctl->q_issued > ctl->q_consumed)
        mbar_wait_bounded_at(&ctl->q_full, (ctl->q_issued - 1) & 1, &never, dl, a.status, 59, 1, 0, 0);
      for (int s = 0; s < NSTAGE; ++s)
        if (ctl->issued[s] > ctl->consumed[s])
          mbar_wait_bounded_at(&ctl->full[s], (ctl->issued[s] - 1) & 1, &never, dl, a.status, 59, ctl->issued[s], s,
                               ctl->consumed[s]);
    } else {
      const uint64_t until = globaltimer_ns() + 50000ull;
      while (globaltimer_ns() < until) {
      }
    }
  }
  __syncwarp();
  // neither CTA leaves while the other may still arrive on its barriers
  pair::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    pair::tmem_dealloc2(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
template <int D>
cudaError_t launch_pair(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                        const PairArgs& t, int B, cudaStream_t st) {
  using Cfg = PairCfg<D>;
  auto kern = k_prefill_pair<D, false>;
  if constexpr (D == 512)
    if (t.sinks >= 0) kern = k_prefill_pair<D, true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  dim3 grid(2 * t.n_pairs, (t.head_pair ? t.Hq / 2 : t.Hq) * Cfg::NV, B);
  if (t.sinks >= 0) return launch_early(kern, grid, 192, Cfg::SMEM, st, 0, mq, mk, mv, mo, t);
  kern<<<grid, 192, Cfg::SMEM, st>>>(mq, mk, mv, mo, t);
  return cudaGetLastError();
}

cudaError_t launch_stream(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const PrefillAttnArgs& a, const PairArgs& t, int B, cudaStream_t st) {
  CUtensorMap mo;  // boxes of a softmax warp's rows
  const uint64_t D = 256, E = 2;
  const uint64_t dims[4] = {D, (uint64_t)a.Hq, (uint64_t)a.S, (uint64_t)B};
  const uint64_t str[3] = {D * E, a.Hq * D * E, (uint64_t)a.S * a.Hq * D * E};
  const uint32_t box[4] = {64, 1, 32, 1};
  if (!make_map_bf16_4d(&mo, a.out, dims, str, box)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_prefill_stream, cudaFuncAttributeMaxDynamicSharedMemorySize, STREAM_SMEM);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)t.n_pairs * (t.head_pair ? t.Hq / 2 : t.Hq) * B;
  if (items > INT32_MAX - (1 << 20)) return cudaErrorInvalidValue;
  const int pairs = (int)std::min<int64_t>(items, multiprocessors() / 2);
  return launch_early(k_prefill_stream, dim3(2 * pairs), STREAM_T, STREAM_SMEM, st, 0, mq, mk, mv, mo, t, (int)items);
}

}  // namespace

cudaError_t launch_prefill_attn_pair(const PrefillAttnArgs& a, int B, int D, int key_rows_total,
                                     int kv_token_major, int head_pair, cudaStream_t st) {
  if (D != 256 && D != 512) return cudaErrorInvalidValue;
  CUtensorMap mq, mk, mv, mo;
  if (!make_prefill_maps(a, B, D, key_rows_total, kv_token_major, BM, KH, BN, &mq, &mk, &mv, &mo))
    return cudaErrorInvalidValue;
  PairArgs t;
  t.S = a.S;
  t.window = a.window;
  t.sinks = a.sinks;
  t.scale_log2 = a.scale_log2;
  t.Hq = a.Hq;
  t.Hkv = a.Hkv;
  t.key_cap = a.key_cap;
  t.seq_lens_before = a.seq_lens_before;
  t.out = a.out;
  t.lse = a.lse;
  t.status = a.status;
  t.wait_ns = a.wait_ns;
  t.kv_token_major = kv_token_major;
  t.key_off_window = a.key_off_window;
  t.page_table = a.page_table;
  t.page_size = a.page_size;
  t.pages_per_seq = a.pages_per_seq;
  t.n_pages = a.n_pages;
  const int n_qtiles = (a.S + BM - 1) / BM;
  // head pairs need an even number of q heads per KV head (both share its K/V)
  t.head_pair = head_pair && (a.Hq / a.Hkv) % 2 == 0;
  t.n_pairs = t.head_pair ? n_qtiles : (n_qtiles + 1) / 2;
  if (t.sinks >= 0 && D == 256) return launch_stream(mq, mk, mv, a, t, B, st);
  return D == 256 ? launch_pair<256>(mq, mk, mv, mo, t, B, st) : launch_pair<512>(mq, mk, mv, mo, t, B, st);
}

}  // namespace hlg
