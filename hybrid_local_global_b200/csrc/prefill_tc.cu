// prefill_tc.cu -- prefill attention on the 5th-generation tensor cores
// (tcgen05 MMA, TMEM accumulators, TMA-fed shared memory), head_dim 256 and
// 512.
//
// Computes, for every query row i of a (batch, q head) and its KV head
// g = h / (Hq/Hkv) ("Gemma 4: End-to-End Architecture Walkthrough", 3a/3b):
//   out_i = sum_j softmax_j(scale <q~_i, k~_j>) v_j   over visible keys j
// where visible means j <= pos_i and, on a local layer, j > pos_i - window.
//
// CTA = one 128-row query tile of one (batch, q head) and one 256-column
// half of the output (head_dim 512 uses two CTAs: the fp32 O tile of 128 x
// 512 alone would fill the 512 TMEM columns, so each CTA owns 256 output
// columns and computes S over all 512 dims); 192 threads:
//   warp 0     TMA producer: Q once (D/64 boxes of 128 rows x 64 dims), then
//              a ring of 32 KB stages in MMA order: K_0, K_1, V_0, K_2, V_1,
//              ... (a K tile = D/128 stages of 128 keys x 128 dims, a V tile
//              = 2 stages of 64 keys x 256 dims; 128-byte swizzle).
//   warp 1     TMEM owner and MMA issuer: S_j = Q K_j^T into one
//              of two 128-column TMEM buffers (M=128, N=128, K=D), then
//              O += P_{j-1} V_{j-1} (M=128, N=256, K=128) with P read from
//              TMEM; tcgen05.commit frees smem stages and signals S / O.
//   warps 2-5  softmax, one query row per thread (TMEM lane = row): load
//              S_j, mask edge tiles, online softmax in the log2 domain,
//              write P_j (bf16) over S_j's columns, rescale O in TMEM only
//              when the running max grows by more than 2^8; epilogue O / l.
// TMEM columns: O 0..255 (fp32), S/P buffers 256..383 and 384..511.
// The MMA pipe runs P_{j-1} V_{j-1} and S_{j+1} while the softmax works on
// S_j; the softmax waits for P_{j-1} V_{j-1} only before rescaling O (rare)
// and before releasing P_j, by which time it has normally completed.
//
// Tiles: key tiles [lo(first row), hi(last row)] only (window-aware
// skipping); per-element masks only on tiles that cross a row's range.
// Grid order puts the heaviest query tiles first (causal work grows with
// the tile index).
//
// Every wait is bounded by a %globaltimer deadline. On a timeout the CTA
// raises its abort flag, records GEMMA_ERR_DEVICE_TIMEOUT, waits for its
// issued MMAs (commit + bounded wait) and TMA loads, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "pair.cuh"
#include "prefill_row.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace hlg {

namespace {

constexpr int BM = 128, BN = 128, DV = 256;  // DV: output columns per CTA
constexpr int CHUNK_B = 128 * 128;   // [128 rows][64 bf16] swizzled box
constexpr int STAGE_B = 32768;
constexpr int ALIGN_B = 1024;
constexpr int SMEM_MAX = 232448;     // opt-in dynamic shared memory per block
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_O = 0, COL_S = 256;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(128, 128, 0, 0);
constexpr uint32_t IDESC_PV = tc::idesc_bf16_f32(128, 256, 0, 1);

template <int NSTAGE>
struct Ctl {
  uint64_t q_full;
  uint64_t full[NSTAGE];
  uint64_t empty[NSTAGE];
  uint64_t s_full[2];
  uint64_t p_ready[2];  // SK: P_j completes phase j/2 of p_ready[j % 2]; else phase j of p_ready[0]
  uint64_t o_done[2];  // PV_i completes phase i/2 of o_done[i % 2]
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued[NSTAGE];
  int consumed[NSTAGE];
  int q_issued, q_consumed;
};

template <int D>
struct TcCfg {
  static constexpr int Q_B = BM * D * 2;                 // 64 KB / 128 KB
  static constexpr int K_STAGES = D / 128;                // stages per K tile
  static constexpr int NV = D / DV;                       // CTAs per (tile, head)
  static constexpr int NSTAGE = (SMEM_MAX - ALIGN_B - Q_B - 512) / STAGE_B;  // 5 / 3
  static constexpr int SMEM = ALIGN_B + Q_B + NSTAGE * STAGE_B + (int)sizeof(Ctl<NSTAGE>);
  static_assert(NSTAGE >= 3 && SMEM <= SMEM_MAX, "shared memory plan");
};

struct TcArgs {
  int S, window, Hq, Hkv;
  int sinks;  // SK instances: positions below it stay visible to every query
  int64_t key_cap;
  const int32_t* seq_lens_before;
  float scale_log2;
  bf16* out;
  float* lse;
  int* status;
  unsigned long long wait_ns;
  int kv_token_major;  // K/V map coordinates: 0 = (d, key, head, b), 1 = (d, head, key, b)
  int key_off_window;  // 1: K/V view row = position - (pos0 - window), else = position
  int n_qtiles;
  // paged cache (head-major views of the pool): view row = position % page_size,
  // view batch = page_table[b * pages_per_seq + position / page_size]; null: contiguous
  const int32_t* page_table;
  int page_size, pages_per_seq, n_pages;
  // multi-token decode (VF instances): rows (token t, q head g * G + i) = t * G + i
  // of KV head g, keys [split * chunk, +chunk) of the sequence's seq_lens[b]
  const int32_t* seq_lens;
  int tokens, chunk, n_splits;
  float* part_o;
  float* part_lse;
};

// VF: the multi-token decode instance (see launch_verify_attn_rows): a CTA is
// (KV head g and output half, sequence b, key split); its 128-row tile holds
// the G q heads of g for each of the `tokens` new tokens (rows past G *
// tokens see no key), and it writes fp32 partials O / l and log2-sum-exp for
// the combine instead of bf16 rows.
// SK: a window plus sinks (cache views): the key tiles of the sinks, then the
// tiles from the window's first one on.
// VF and SK: a short chunk with a window plus sinks. A CTA's rows are the G q
// heads of one KV head for 128 / G tokens (as VF: the tile is full where a
// chunk of one head would not fill it, and the heads share the keys), and the
// CTAs of a cluster share the key tiles: few rows then still use many SMs. The
// splits merge in distributed shared memory, each CTA for its share of the
// columns, straight into the output.
template <int D, bool VF, bool SK>
__global__ void __launch_bounds__(192, 1)
    k_prefill_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                 const TcArgs a) {
  using Cfg = TcCfg<D>;
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

  constexpr bool ROWS = VF && SK;
  const int G = a.Hq / a.Hkv;
  const int unit = ROWS ? (int)blockIdx.y : (int)blockIdx.x;
  const int vh = unit % Cfg::NV, b = ROWS ? blockIdx.z : blockIdx.y;
  const int h = VF ? 0 : (int)blockIdx.x / Cfg::NV;  // VF: per row, g * G + row % G
  const int g = ROWS ? unit / Cfg::NV % a.Hkv : VF ? unit / Cfg::NV : h / G;
  const int q0 = VF ? 0 : (a.n_qtiles - 1 - (int)blockIdx.z) * BM;
  const int t0 = ROWS ? unit / (Cfg::NV * a.Hkv) * a.tokens : 0;  // first token of the rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int64_t pos0, n_keys, kt0;
  int64_t v_lo = 0, v_end = 0;  // SK: keys that the rows see, sinks apart
  int n_tiles;
  int n_st = 0;  // SK: tiles of the sinks, before tile kt0
  int j0 = 0;    // ROWS: this CTA's first tile
  if (VF && !SK) {
    // token t sits at position seq_lens[b] - tokens + t; this CTA reads keys
    // [split * chunk, min(+chunk, seq_lens[b]))
    n_keys = a.seq_lens[b];
    pos0 = n_keys - a.tokens;
    const int64_t k_begin = (int64_t)blockIdx.z * a.chunk;
    if (pos0 < 0 || n_keys > a.key_cap || k_begin >= n_keys) return;  // range reported by the append kernel
    const int64_t k_end = k_begin + a.chunk < n_keys ? k_begin + a.chunk : n_keys;
    kt0 = k_begin / BN;
    n_tiles = (int)((k_end - 1) / BN - kt0 + 1);
  } else {
    pos0 = a.seq_lens_before ? (int64_t)a.seq_lens_before[b] : 0;
    n_keys = pos0 + a.S;
  }
  // view row of a key = its position - koff (a gathered key window starts at pos0 - window)
  const int64_t koff = (!VF && a.key_off_window) ? pos0 - a.window : 0;
  if (!VF || SK) {
    if (pos0 < 0 || n_keys - koff > a.key_cap) {  // reported by the RoPE kernel
      if (SK) after_previous();
      return;
    }
    const int first = ROWS ? t0 : q0, last = min(ROWS ? t0 + a.tokens - 1 : q0 + BM - 1, a.S - 1);
    int64_t lo_first, hi_first, lo_last, hi_last;
    visible_range(pos0 + first, a.window, n_keys, &lo_first, &hi_first);
    visible_range(pos0 + last, a.window, n_keys, &lo_last, &hi_last);
    kt0 = lo_first / BN;
    n_tiles = (int)(hi_last / BN - kt0 + 1);
    if (SK) {
      v_lo = lo_first;
      v_end = hi_last + 1;
      const int64_t sink_tiles = ((int64_t)a.sinks + BN - 1) / BN;
      n_st = (int)(sink_tiles < kt0 ? sink_tiles : kt0);
      n_tiles += n_st;
    }
    if (ROWS) {
      const int per = (n_tiles + (int)gridDim.x - 1) / (int)gridDim.x;
      j0 = (int)blockIdx.x * per;
      n_tiles = max(0, min(per, n_tiles - j0));
    }
  }
  // first key of the j-th key tile
  const auto tile_key = [&](int j) -> int64_t {
    j += j0;
    return (SK && j < n_st ? j : kt0 + j - n_st) * BN;
  };

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
    mbar_init(&ctl->p_ready[0], 128);
    mbar_init(&ctl->p_ready[1], 128);
    mbar_init(&ctl->o_done[0], 1);
    mbar_init(&ctl->o_done[1], 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ctl->q_issued = 0;
    ctl->q_consumed = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tc::tmem_relinquish();
  }
  if (SK) after_previous();  // the rotation, beside which all of the above ran
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;
  float row_m = -INFINITY, row_l = 0.f;  // ROWS, softmax threads: the row's max and sum over this CTA's keys

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t go = tc::elect_one();
    if (go) {
      tc::prefetch_tmap(&tm_q);
      tc::prefetch_tmap(&tm_k);
      tc::prefetch_tmap(&tm_v);
      // VF: G heads x tokens rows; the tile's other rows are never stored
      mbar_arrive_expect_tx(&ctl->q_full, VF ? (uint32_t)(D * 2 * G * a.tokens) : (uint32_t)Q_B);
      ctl->q_issued = 1;
    }
    __syncwarp();
    for (int c = 0; c < D / 64; ++c) {
      if (VF)
        tc::tma_load_4d_if(go, sQ + c * CHUNK_B, &tm_q, c * 64, g * G, t0, b, smem_u32(&ctl->q_full));
      else
        tc::tma_load_4d_if(go, sQ + c * CHUNK_B, &tm_q, c * 64, h, q0, b, smem_u32(&ctl->q_full));
    }
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
        const int n_stg = kind == 0 ? Cfg::K_STAGES : 2;
        for (int half = 0; half < n_stg; ++half, ++item) {
          const int s = item % NSTAGE;
          if (item >= NSTAGE &&
              !wait_all(&ctl->empty[s], ((item / NSTAGE) - 1) & 1, abort_flag, deadline, a.status, 11, item, s, j)) {
            ok = false;
            break;
          }
          const uint32_t dst = sStage + s * STAGE_B;
          const uint32_t bar = smem_u32(&ctl->full[s]);
          if (go) {
            mbar_arrive_expect_tx(&ctl->full[s], STAGE_B);
            ctl->issued[s] += 1;
          }
          __syncwarp();
          if (kind == 0) {
            for (int cc = 0; cc < 2; ++cc) {
              const int d0 = (half * 2 + cc) * 64;
              if (a.kv_token_major)
                tc::tma_load_4d_if(go, dst + cc * CHUNK_B, &tm_k, d0, g, key0, kb, bar);
              else
                tc::tma_load_4d_if(go, dst + cc * CHUNK_B, &tm_k, d0, key0, g, kb, bar);
            }
          } else {
            const int k0 = key0 + half * 64;
            for (int c = 0; c < 4; ++c) {
              if (a.kv_token_major)
                tc::tma_load_4d_if(go, dst + c * 8192, &tm_v, vh * DV + c * 64, g, k0, kb, bar);
              else
                tc::tma_load_4d_if(go, dst + c * 8192, &tm_v, vh * DV + c * 64, k0, g, kb, bar);
            }
          }
        }
      }
    }
    __syncwarp();  // reconverge before the block barrier below
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t go = tc::elect_one();
    bool ok = wait_all(&ctl->q_full, 0, abort_flag, deadline, a.status, 10);
    if (ok && go) ctl->q_consumed = 1;
    const uint64_t dq = tc::smem_desc_sw128(sQ, 16, 1024);
    const uint64_t dk = tc::smem_desc_sw128(sStage, 16, 1024), dv = tc::smem_desc_sw128(sStage, 8192, 1024);
    int item = 0, taken = 0;
    for (int j = 0; j <= n_tiles && ok; ++j) {
      if (j < n_tiles) {
        const uint32_t d_s = tmem + COL_S + (uint32_t)(j & 1) * 128;
        for (int half = 0; half < Cfg::K_STAGES; ++half, ++item) {
          const int s = item % NSTAGE;
          if (!wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 12, item, s, j)) {
            ok = false;
            break;
          }
          taken = item + 1;
          tc::fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_ss_if(go, d_s, dq + (uint64_t)(((half * 2 + cc) * CHUNK_B + kk * 32) >> 4),
                            dk + (uint64_t)((s * STAGE_B + cc * CHUNK_B + kk * 32) >> 4), IDESC_S,
                            (half | cc | kk) != 0);
          tc::commit_if(go, smem_u32(&ctl->empty[s]));
        }
        if (!ok) break;
        tc::commit_if(go, smem_u32(&ctl->s_full[j & 1]));
      }
      if (j >= 1) {
        if (!wait_all(&ctl->p_ready[SK ? (j - 1) & 1 : 0], (SK ? (j - 1) >> 1 : j - 1) & 1, abort_flag, deadline, a.status,
                      13, j)) {
          ok = false;
          break;
        }
        const int64_t tile_key0 = tile_key(j - 1);
        const tc::SeenRows seen = tc::seen_rows(SK && j - 1 + j0 < n_st, SK ? a.sinks - tile_key0 : 0,
                                                SK ? v_lo - tile_key0 : 0, (SK ? v_end : n_keys) - tile_key0);
        const uint32_t p_tm = tmem + COL_S + (uint32_t)((j - 1) & 1) * 128;
        for (int half = 0; half < 2; ++half, ++item) {
          const int s = item % NSTAGE;
          if (!wait_all(&ctl->full[s], (item / NSTAGE) & 1, abort_flag, deadline, a.status, 14, item, s, j)) {
            ok = false;
            break;
          }
          taken = item + 1;
          const uint32_t st = sStage + s * STAGE_B;
          const auto clear = [&](int from, int to) {  // rows of the tile, of which 64 lie in this stage
            const int r0 = max(from - half * 64, 0), r1 = min(to - half * 64, 64);
            if (r0 >= r1) return;
            for (int idx = lane; idx < (r1 - r0) * 4 * 8; idx += 32) {
              const int r = r0 + idx / 32, c = (idx / 8) % 4, u = idx % 8;
              *reinterpret_cast<uint4*>(sm + (st - base) + c * 8192 + r * 128 + u * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          };
          const auto product = [&](int kk, bool add) {
            tc::mma_ts_if(go, tmem + COL_O, p_tm + half * 32 + kk * 8,
                          dv + (uint64_t)((s * STAGE_B + kk * 2048) >> 4), IDESC_PV, add ? 1u : 0u);
          };
          if (SK && !seen.all()) {
            clear(seen.gap0, seen.gap1);
            clear(seen.tail, seen.k1 * 16);
            tc::fence_after_sync();
#pragma unroll 1
            for (int kk = max(seen.k0 - half * 4, 0); kk < min(seen.k1 - half * 4, 4); ++kk)
              product(kk, j - 1 > 0 || half * 4 + kk > seen.k0);
          } else {
            // keys past the sequence: their P is 0, but their V rows must be finite
            if (!SK) clear(seen.tail, BN);
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) product(kk, j - 1 > 0 || half || kk);
          }
          tc::commit_if(go, smem_u32(&ctl->empty[s]));
        }
        if (!ok) break;
        tc::commit_if(go, smem_u32(&ctl->o_done[(j - 1) & 1]));
      }
    }
    // make sure no MMA is in flight before TMEM can be released
    tc::commit_if(go, smem_u32(&ctl->drain));
    if (go) {
      for (int s = 0; s < NSTAGE; ++s) ctl->consumed[s] = (taken + NSTAGE - 1 - s) / NSTAGE;
      volatile int never = 0;
      mbar_wait_bounded_at(&ctl->drain, 0, &never, globaltimer_ns() + 200000000ull, a.status, 18, 0, 0, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(wq * 32) << 16);
    const bool row_valid = VF ? row < G * a.tokens && t0 + row / G < a.S : q0 + row < a.S;
    int64_t lo, hi;
    if (ROWS) {
      lo = 0;
      hi = -1;  // a row past the tokens sees nothing
      if (row_valid) visible_range(pos0 + t0 + row / G, a.window, n_keys, &lo, &hi);
    } else if (VF) {
      // keys up to the row's token (global layer); a row past the tokens sees none
      lo = row_valid ? 0 : 1;
      hi = row_valid ? pos0 + row / G : 0;
    } else {
      visible_range(pos0 + (row_valid ? q0 + row : a.S - 1), a.window, n_keys, &lo, &hi);
    }
    // SK: the queries carry a power of two of scale * log2(e), which leaves their
    // bits alone, and the rest of it (1 <= c < 2) is applied to the logits
    const float factor = SK ? a.scale_log2 : 1.f;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    int pv_seen = 0;  // P.V products whose completion this thread has consumed
    for (int j = 0; j < n_tiles; ++j) {
      const int64_t kb = tile_key(j);
      if (!wait_all(&ctl->s_full[j & 1], (j >> 1) & 1, abort_flag, deadline, a.status, 15, j)) {
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
      // row cannot see become -inf in place (only tiles that straddle the
      // visible range need it).
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
      // The running max m_used only moves when a tile's max exceeds it by more
      // than 2^8 (or on a row's first visible key), so P = 2^(x - m_used) is
      // computed in one pass that also takes the tile max, and redone in the
      // rare case the max moved. A warp with a row that has seen no key yet
      // takes the max first instead, since its speculation would always fail.
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
          if (!wait_all(&ctl->o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 16, j)) {
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
        if (!wait_all(&ctl->o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 16, j)) {
          ok = false;
          break;
        }
        pv_seen = j;
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&ctl->p_ready[SK ? j & 1 : 0]);
    }
    if (ok && n_tiles > 0)
      ok = wait_all(&ctl->o_done[(n_tiles - 1) & 1], ((n_tiles - 1) >> 1) & 1, abort_flag, deadline,
                    a.status, 17, n_tiles);
    if (ROWS) {
      row_m = m_used;
      row_l = ok ? l : -1.f;
    }
    // Epilogue: O / l as bf16 into the Q buffer (free once the last MMA is
    // done), laid out as the 128-byte-swizzled boxes of the output map, then
    // four TMA stores. A thread owns one row, so direct stores would write
    // 16 bytes per output row per instruction; the staged copy writes whole
    // rows. Rows past the sequence end are clipped by the store.
    unsigned char* sO = sm;  // Q buffer
    if (ROWS) {
      // below, once the cluster is through
    } else if (VF) {
      // fp32 partial O / l of this split and its log2-sum-exp, for the combine
      if (ok) {
        tc::fence_after_sync();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int t = row / G;
        const int64_t pr = (((int64_t)b * a.tokens + t) * a.Hq + g * G + row % G) * a.n_splits + blockIdx.z;
        float* dst = a.part_o + pr * D + vh * DV;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tc::tmem_ld32(tm + COL_O + c * 32, o);  // every lane: the load is warp-wide
          tc::tmem_wait_ld();
          if (row_valid) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<float4*>(dst + c * 32 + u * 4) =
                  make_float4(__uint_as_float(o[u * 4 + 0]) * inv, __uint_as_float(o[u * 4 + 1]) * inv,
                              __uint_as_float(o[u * 4 + 2]) * inv, __uint_as_float(o[u * 4 + 3]) * inv);
          }
        }
        if (row_valid && vh == 0) a.part_lse[pr] = l > 0.f ? m_used + __log2f(l) : -INFINITY;
      }
    } else if (ok) {
      tc::fence_after_sync();
      const float inv = SK || l > 0.f ? 1.f / l : 0.f;  // SK: as in prefill_stream.cu, 0 and NaN are to show
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[32];
        tc::tmem_ld32(tm + COL_O + c * 32, o);
        tc::tmem_wait_ld();
        unsigned char* box_row = sO + (c >> 1) * CHUNK_B + row * 128;
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
    if (!VF && warp == 2 && lane == 0 && !*abort_flag) {
      for (int c = 0; c < DV / 64; ++c)
        tc::tma_store_4d(&tm_o, smem_u32(sO + c * CHUNK_B), vh * DV + c * 64, h, q0, b);
      tc::bulk_commit();
      tc::bulk_wait_read0();
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // loads still in flight must land before shared memory is released
    volatile int never = 0;
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    if (ctl->q_issued && !ctl->q_consumed) mbar_wait_bounded_at(&ctl->q_full, 0, &never, dl, a.status, 19, 0, 0, 0);
    for (int s = 0; s < NSTAGE; ++s)
      if (ctl->issued[s] > ctl->consumed[s])
        mbar_wait_bounded_at(&ctl->full[s], (ctl->issued[s] - 1) & 1, &never, dl, a.status, 19,
                             ctl->issued[s], s, ctl->consumed[s]);
  }
  if constexpr (ROWS) {
    // Merge: each CTA leaves its O (fp32, rows PITCH bytes apart: an odd number
    // of 16-byte words, which spreads them over the banks) and (m, l) in its own
    // Q buffer and ring, and sums every CTA's over its share of the columns.
    // (Remote reads of whole 128-byte runs; remote writes of a row per lane took
    // several times as long.)
    constexpr int PITCH = DV * 4 + 16, ML = BM * PITCH, ALL = ML + BM * 8;
    const int n = gridDim.x, cols = DV / n, own = blockIdx.x;
    if (warp >= 2) {
      const int row = (warp & 3) * 32 + lane;
      const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      if (n_tiles > 0) {
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tc::tmem_ld32(tm + COL_O + c * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(sm + row * PITCH + c * 128 + u * 16) =
                make_uint4(o[u * 4], o[u * 4 + 1], o[u * 4 + 2], o[u * 4 + 3]);
        }
      }
      *reinterpret_cast<float2*>(sm + ML + row * 8) = make_float2(row_m, row_l);
    }
    tc::fence_before_sync();
    __syncwarp();
    pair::cluster_sync();  // every share is in place
    // per row: every split's weight 2^(m - M) / L, then 0 (fine) or 1 (a CTA gave up), M and L
    float* wgt = reinterpret_cast<float*>(sm + ALL);  // [row][12]
    if (threadIdx.x < BM) {
      const int row = threadIdx.x;
      float2 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        v[r] = make_float2(-INFINITY, 0.f);
        if (r < n)
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(v[r].x), "=f"(v[r].y)
                       : "r"(pair::map_to(base + ML + row * 8, r)));
      }
      float M = -INFINITY, L = 0.f, bad = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        M = fmaxf(M, v[r].x);
        if (v[r].y < 0.f) bad = 1.f;  // l < 0: that CTA gave up
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        v[r].x = v[r].x == -INFINITY ? 0.f : tc::ex2(v[r].x - M);  // no visible key there
        L += v[r].x * v[r].y;
      }
      const float inv = 1.f / L;  // NaN stays NaN, and so does 0 / 0 (every logit -inf)
#pragma unroll
      for (int r = 0; r < 8; ++r) wgt[row * 12 + r] = v[r].x * inv;
      wgt[row * 12 + 8] = bad;
      const int t = t0 + row / G;
      if (a.lse && vh == 0 && own == 0 && row < G * a.tokens && t < a.S && bad == 0.f)
        a.lse[((int64_t)b * a.Hq + g * G + row % G) * a.S + t] = (M + __log2f(L)) * 0.69314718055994530942f;
    }
    __syncthreads();
    const int groups = cols / 8;  // 16 bytes of output
    for (int i = threadIdx.x; i < BM * groups; i += 192) {
      const int row = i / groups, c = (i - row * groups) * 8, t = t0 + row / G;
      if (row >= G * a.tokens || t >= a.S || wgt[row * 12 + 8] != 0.f) continue;
      const uint32_t at = base + row * PITCH + (own * cols + c) * 4;
      float o[8][8], x[8];  // all reads on their way before the first sum
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < n) {
          const uint32_t from = pair::map_to(at, r);
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(o[r][0]), "=f"(o[r][1]), "=f"(o[r][2]), "=f"(o[r][3])
                       : "r"(from));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(o[r][4]), "=f"(o[r][5]), "=f"(o[r][6]), "=f"(o[r][7])
                       : "r"(from + 16));
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float w = wgt[row * 12 + r];
        if (r < n && w != 0.f)  // a split without a weight may have left no O
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += w * o[r][e];
      }
      const int64_t hr = ((int64_t)b * a.S + t) * a.Hq + g * G + row % G;
      *reinterpret_cast<uint4*>(a.out + hr * D + vh * DV + own * cols + c) =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    }
    __syncwarp();
    pair::cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

cudaError_t launch_prefill_attn_tc(const PrefillAttnArgs& a, int B, int D, int key_rows_total,
                                   int kv_token_major, cudaStream_t st) {
  if (D != 256 && D != 512) return cudaErrorInvalidValue;
  CUtensorMap mq, mk, mv, mo;
  if (!make_prefill_maps(a, B, D, key_rows_total, kv_token_major, BM, BN, 64, &mq, &mk, &mv, &mo))
    return cudaErrorInvalidValue;
  TcArgs t;
  t.S = a.S;
  t.window = a.window;
  t.sinks = a.sinks;
  t.Hq = a.Hq;
  t.Hkv = a.Hkv;
  t.key_cap = a.key_cap;
  t.seq_lens_before = a.seq_lens_before;
  t.scale_log2 = a.scale_log2;
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
  t.n_qtiles = (a.S + BM - 1) / BM;
  if (D == 256) {
    using Cfg = TcCfg<256>;
    if (a.sinks >= 0) return cudaErrorInvalidValue;  // launch_prefill_attn_stream's
    auto kern = k_prefill_tc<256, false, false>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    dim3 grid(a.Hq * Cfg::NV, B, t.n_qtiles);
    kern<<<grid, 192, Cfg::SMEM, st>>>(mq, mk, mv, mo, t);
  } else {
    using Cfg = TcCfg<512>;
    auto kern = a.sinks >= 0 ? k_prefill_tc<512, false, true> : k_prefill_tc<512, false, false>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    dim3 grid(a.Hq * Cfg::NV, B, t.n_qtiles);
    if (a.sinks >= 0) return launch_early(kern, grid, 192, Cfg::SMEM, st, 0, mq, mk, mv, mo, t);
    kern<<<grid, 192, Cfg::SMEM, st>>>(mq, mk, mv, mo, t);
  }
  return cudaGetLastError();
}

namespace {
// CTAs per unit of rows and columns (the cluster) of the short-chunk form, 0
// where the unsplit kernels are to be used: see launch_prefill_attn_rows.
// Twice the CTAs pay while their clusters run at once (of 148 SMs 74 clusters of
// 2, 33 of 4 and 15 of 8, as none crosses a GPC) and the key tiles that a CTA
// saves (2.8 us each) take longer than the wider merge (4 us with all rows in
// use). Measured (us, n = 1 being the unsplit kernels):
//   8 q heads on 1, dim 512, window  512, 64 tokens: n = 1 21.5, 2 21.6, 4 20.9, 8 22.0
//                                          5 tokens:      22.2,   18.4,   16.3,   16.0
//                                        512 tokens:      26.1,   23.3,   41.9
//   32 on 4,         dim 512, window 4096, 64 tokens:     81.3,   62.5,   46.0,   92.8
//   32 on 16,        dim 256, window 1024, 64 tokens:     33.4,   31.5,   29.9,   50.4
//                                        512 tokens:      41.4,   57.9
template <int D>
int rows_splits(const PrefillAttnArgs& a, int B) {
  using Cfg = TcCfg<D>;
  const int per_tile = BM / (a.Hq / a.Hkv);  // tokens per row tile
  const int tokens = std::min(a.S, per_tile);
  const int64_t units = (int64_t)a.Hkv * Cfg::NV * B * ((a.S + per_tile - 1) / per_tile);
  const int64_t tiles = std::min<int64_t>(((int64_t)a.window + tokens) / BN + 2 + ((int64_t)a.sinks + BN - 1) / BN,
                                          (a.key_cap + BN - 1) / BN);
  const int sms = multiprocessors();
  const auto pays = [&](int n) {  // 2 n CTAs rather than n
    const int64_t room = n == 1 ? sms : n == 2 ? sms * 9 / 10 : sms * 17 / 20;
    const int64_t saved = (tiles + n - 1) / n - (tiles + 2 * n - 1) / (2 * n);
    return units * 2 * n <= room && (double)saved * 2.8 > 4.0 * tokens / per_tile;
  };
  int n = 1;
  while (n < 8 && pays(n)) n *= 2;
  return n > 1 ? n : 0;
}

template <int D>
cudaError_t launch_rows_as(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TcArgs& t,
                           int B, int n, cudaStream_t st) {
  using Cfg = TcCfg<D>;
  auto kern = k_prefill_tc<D, true, true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  const dim3 grid(n, t.Hkv * Cfg::NV * ((t.S + t.tokens - 1) / t.tokens), B);
  return launch_early(kern, grid, 192, Cfg::SMEM, st, n, mq, mk, mv, mq, t);
}
}  // namespace

int prefill_rows_splits(const PrefillAttnArgs& a, int B, int D) {
  return D == 256 ? rows_splits<256>(a, B) : rows_splits<512>(a, B);
}

// A short chunk (window plus sinks, paged cache): see k_prefill_tc.
cudaError_t launch_prefill_attn_rows(const PrefillAttnArgs& a, int B, int D, int n, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  const uint64_t E = 2;
  TcArgs t{};
  t.tokens = BM / G;
  CUtensorMap mq, mk, mv;
  {
    // q_rot [B][S][Hq][D]: a box is the G heads of one KV head for `tokens` tokens
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.S, (uint64_t)B};
    const uint64_t str[3] = {(uint64_t)D * E, (uint64_t)a.Hq * D * E, (uint64_t)a.S * a.Hq * D * E};
    const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)t.tokens, 1};
    if (!make_map_bf16_4d(&mq, a.q_rot, dims, str, box)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.page_size, (uint64_t)a.Hkv, (uint64_t)a.n_pages};
    const uint64_t strk[3] = {(uint64_t)a.k.stride_row * E, (uint64_t)a.k.stride_h * E, (uint64_t)a.k.stride_b * E};
    const uint64_t strv[3] = {(uint64_t)a.v.stride_row * E, (uint64_t)a.v.stride_h * E, (uint64_t)a.v.stride_b * E};
    const uint32_t bk[4] = {64, (uint32_t)BN, 1, 1}, bv[4] = {64, 64, 1, 1};
    if (!make_map_bf16_4d(&mk, a.k.ptr, dims, strk, bk) || !make_map_bf16_4d(&mv, a.v.ptr, dims, strv, bv))
      return cudaErrorInvalidValue;
  }
  t.S = a.S;
  t.window = a.window;
  t.sinks = a.sinks;
  t.Hq = a.Hq;
  t.Hkv = a.Hkv;
  t.key_cap = a.key_cap;
  t.seq_lens_before = a.seq_lens_before;
  t.scale_log2 = a.scale_log2;
  t.out = a.out;
  t.lse = a.lse;
  t.status = a.status;
  t.wait_ns = a.wait_ns;
  t.page_table = a.page_table;
  t.page_size = a.page_size;
  t.pages_per_seq = a.pages_per_seq;
  t.n_pages = a.n_pages;
  return D == 256 ? launch_rows_as<256>(mq, mk, mv, t, B, n, st) : launch_rows_as<512>(mq, mk, mv, t, B, n, st);
}

namespace {
template <int D>
cudaError_t launch_verify_as(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TcArgs& t,
                             int B, cudaStream_t st) {
  using Cfg = TcCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(k_prefill_tc<D, true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  dim3 grid(t.Hkv * Cfg::NV, B, t.n_splits);
  k_prefill_tc<D, true, false><<<grid, 192, Cfg::SMEM, st>>>(mq, mk, mv, mq, t);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_verify_attn_rows(const VerifyAttnArgs& a, int B, int D, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  if ((D != 256 && D != 512) || a.tokens < 1 || G * a.tokens > BM || a.chunk % BN || a.n_splits < 1)
    return cudaErrorInvalidValue;
  const uint64_t E = 2;
  CUtensorMap mq, mk, mv;
  {
    // q_rot [B][tokens][Hq][D]: a box is the G heads of one KV head for every token
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.tokens, (uint64_t)B};
    const uint64_t str[3] = {(uint64_t)D * E, (uint64_t)a.Hq * D * E, (uint64_t)a.tokens * a.Hq * D * E};
    const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)a.tokens, 1};
    if (!make_map_bf16_4d(&mq, a.q_rot, dims, str, box)) return cudaErrorInvalidValue;
  }
  {
    // head-major views (d, row, head, page) of the cache (a page per sequence
    // when contiguous), K boxes of 128 rows, V boxes of 64
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.page_size, (uint64_t)a.Hkv, (uint64_t)a.n_pages};
    const uint64_t strk[3] = {(uint64_t)a.k.stride_row * E, (uint64_t)a.k.stride_h * E, (uint64_t)a.k.stride_b * E};
    const uint64_t strv[3] = {(uint64_t)a.v.stride_row * E, (uint64_t)a.v.stride_h * E, (uint64_t)a.v.stride_b * E};
    const uint32_t bk[4] = {64, (uint32_t)BN, 1, 1}, bv[4] = {64, 64, 1, 1};
    if (!make_map_bf16_4d(&mk, a.k.ptr, dims, strk, bk) || !make_map_bf16_4d(&mv, a.v.ptr, dims, strv, bv))
      return cudaErrorInvalidValue;
  }
  TcArgs t{};
  t.S = a.tokens;
  t.window = 0;
  t.Hq = a.Hq;
  t.Hkv = a.Hkv;
  t.key_cap = a.cache_cap;
  t.seq_lens_before = nullptr;
  t.scale_log2 = 1.f;
  t.out = nullptr;
  t.lse = nullptr;
  t.status = a.status;
  t.wait_ns = a.wait_ns;
  t.kv_token_major = 0;
  t.key_off_window = 0;
  t.n_qtiles = 1;
  t.page_table = a.page_table;
  t.page_size = a.page_size;
  t.pages_per_seq = a.pages_per_seq;
  t.n_pages = a.n_pages;
  t.seq_lens = a.seq_lens;
  t.tokens = a.tokens;
  t.chunk = a.chunk;
  t.n_splits = a.n_splits;
  t.part_o = a.part_o;
  t.part_lse = a.part_lse;
  return D == 256 ? launch_verify_as<256>(mq, mk, mv, t, B, st) : launch_verify_as<512>(mq, mk, mv, t, B, st);
}

}  // namespace hlg
