// prefill_pair.cu -- prefill attention on CTA pairs: two 128-row query tiles
// of one (batch, q head) on two SMs that share each tcgen05 MMA
// (cta_group::2, M = 256), head_dim 256 and 512.
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
// rows in both CTAs' stages before the P.V product (SK: and those of the edge
// tiles that no row of the pair sees, tc::SeenRows).
//
// Every wait is bounded by a %globaltimer deadline. On a timeout the CTA
// raises its abort flag and records GEMMA_ERR_DEVICE_TIMEOUT; the leader
// drains its MMAs, both CTAs wait for their own loads, meet at a cluster
// barrier, free TMEM and exit.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "launch.h"
#include "prefill_pair.cuh"
#include "tmap.h"

namespace hlg {

namespace {

template <int D>
struct PairCfg {
  static constexpr int Q_B = BM * D * 2;           // 64 KB / 128 KB
  static constexpr int K_STAGES = D / 256;          // stages per half K tile
  static constexpr int NV = D / DV;                 // pairs per (query-tile pair, head)
  static constexpr int NSTAGE = (SMEM_MAX - ALIGN_B - Q_B - 1024) / STAGE_B;  // 5 / 3
  static constexpr int SMEM = ALIGN_B + Q_B + NSTAGE * STAGE_B + (int)sizeof(Ctl<NSTAGE>);
  static_assert(NSTAGE >= 3 && SMEM <= SMEM_MAX, "shared memory plan");
};

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
          const int64_t v_key = tile_key(j - 1);
          const auto product = [&](int kk, bool add) {
            pair::mma2_ts_if(go, tmem + COL_O, p_tm + kk * 8, dv + (uint64_t)((s * STAGE_B + kk * 2048) >> 4), IDESC_PV,
                             add ? 1u : 0u);
          };
          const tc::SeenRows seen =
              SK ? tc::seen_rows(j - 1 < n_st, a.sinks - v_key, lo_first - v_key, hi_last + 1 - v_key)
                 : tc::seen_rows(false, 0, 0, n_keys - v_key);
          if (SK && !seen.all()) {
            if (seen.gap0 < seen.gap1) clear_v_rows_pair(sStage + s * STAGE_B, seen.gap0, seen.gap1, lane);
            if (seen.tail < seen.k1 * 16) clear_v_rows_pair(sStage + s * STAGE_B, seen.tail, seen.k1 * 16, lane);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll 1
            for (int kk = seen.k0; kk < seen.k1; ++kk) product(kk, j - 1 > 0 || kk > seen.k0);
          } else {
            if (!SK && seen.tail < BN) {
              clear_v_rows_pair(sStage + s * STAGE_B, seen.tail, BN, lane);
              __syncwarp();
            }
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk) product(kk, j - 1 > 0 || kk);
          }
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
      const float inv = SK || l > 0.f ? 1.f / l : 0.f;  // SK: as in prefill_stream.cu, 0 and NaN are to show
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
            SK || l > 0.f ? (m_used + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
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

}  // namespace

cudaError_t launch_prefill_attn_pair(const PrefillAttnArgs& a, int B, int D, int key_rows_total,
                                     int kv_token_major, int head_pair, cudaStream_t st) {
  if ((D != 256 && D != 512) || (D == 256 && a.sinks >= 0)) return cudaErrorInvalidValue;
  CUtensorMap mq, mk, mv, mo;
  if (!make_prefill_maps(a, B, D, key_rows_total, kv_token_major, BM, KH, BN, &mq, &mk, &mv, &mo))
    return cudaErrorInvalidValue;
  const PairArgs t = pair_args(a, kv_token_major, head_pair);
  return D == 256 ? launch_pair<256>(mq, mk, mv, mo, t, B, st) : launch_pair<512>(mq, mk, mv, mo, t, B, st);
}

}  // namespace hlg
