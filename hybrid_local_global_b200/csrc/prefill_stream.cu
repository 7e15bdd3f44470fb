// prefill_stream.cu -- prefill attention of head_dim 256 under a window plus
// sinks (paged cache), on CTA pairs as in prefill_pair.cu.
//
// A row tile sees few key tiles there, so what surrounds them counts: of the 26
// us that a CTA of one row tile took for a window of 1024, 8 were setup, the
// first loads and products, and the output.
// Here a pair of CTAs stays and walks row tiles: the key tiles of one follow
// those of the one before through the same ring and TMEM buffers. Its Q is
// loaded once the last S of the one before is done; its first S and softmax run
// beside the last P V, and only then is the output before it taken out of TMEM
// (which its first P V waits for), through 32 KB of shared memory of its own.
//
// Two warps per 32 rows run the softmax, each with half the columns: with one,
// a key tile took 3650 cycles, of which the softmax 2650; with two 2600, of
// which 1024 are its exponentials at the special-function rate and the products
// 2048. B1 S8191 Hq32 Hkv16, window 1024, 16 sinks, the whole call in bursts of 20
// ms, which stay below the power limit (1965 MHz): 344 us (445 with one CTA per row
// tile, before this kernel), 380 back to back for seconds (1680 MHz). By itself this
// kernel takes 258 us (1240 TFLOP/s counting the masked parts of edge tiles; 283
// at 1750 MHz) and the rotation 97; its start lies beside the rotation's end.
//
// Waits, timeouts and the clearing of V's unseen rows are k_prefill_pair's.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "launch.h"
#include "prefill_pair.cuh"
#include "tmap.h"

namespace hlg {

namespace {

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

// A pair's row tile(s) and the key tiles it sees. Positions are below 2^31
// (pages_per_seq * page_size is), once row_tile has checked the length.
struct RowTile {
  int b, h, g, q0;  // this CTA's
  int n_tiles, n_st;
  int pos0, n_keys, kt0;
  int lo, end;  // keys that the rows see, sinks apart
  __device__ __forceinline__ int key(int j) const { return (j < n_st ? j : kt0 + j - n_st) * BN; }
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
  const int64_t pos0 = a.seq_lens_before ? (int64_t)a.seq_lens_before[t->b] : 0, n_keys = pos0 + a.S;
  if (pos0 < 0 || n_keys > a.key_cap) return false;
  int64_t lo_first, hi_first, lo_last, hi_last;
  visible_range(pos0 + first, a.window, n_keys, &lo_first, &hi_first);
  visible_range(pos0 + min(first + span - 1, a.S - 1), a.window, n_keys, &lo_last, &hi_last);
  t->pos0 = (int)pos0;
  t->n_keys = (int)n_keys;
  t->kt0 = (int)(lo_first / BN);
  t->lo = (int)lo_first;
  t->end = (int)hi_last + 1;
  t->n_st = (int)min(((int64_t)a.sinks + BN - 1) / BN, (int64_t)t->kt0);
  t->n_tiles = (int)(hi_last / BN) - t->kt0 + 1 + t->n_st;
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
    const auto load = [&](bool is_v, int b, int g, int key, int n_keys) -> bool {
      // tiles never straddle a page (page_size is a multiple of 128)
      const int pi = key / a.page_size, row = key - pi * a.page_size;
      int kb = pi < a.pages_per_seq ? a.page_table[(int64_t)b * a.pages_per_seq + pi] : 0;
      if (kb < 0 || kb >= a.n_pages) {
        if (go && key < n_keys) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        kb = 0;
      }
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
    int vb = 0, vg = 0, vkey = 0, v_end = 0;  // the key tile before, whose V is loaded next
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
      tc::SeenRows seen{};  // rows of the key tile before,
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
        const uint32_t p_tm = tmem + COL_S + (uint32_t)(k & 1) * 128;
        const auto product = [&](int kk, bool add) {
          pair::mma2_ts_if(go, tmem + COL_O, p_tm + (kk >> 2) * 64 + (kk & 3) * 8,
                           dv + (uint64_t)((s * STAGE_B + kk * 2048) >> 4), IDESC_PV, add ? 1u : 0u);
        };
        if (seen.all()) {
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) product(kk, !v_first || kk);
        } else {
          if (seen.gap0 < seen.gap1) clear_v_rows_pair(sStage + s * STAGE_B, seen.gap0, seen.gap1, lane);
          if (seen.tail < seen.k1 * 16) clear_v_rows_pair(sStage + s * STAGE_B, seen.tail, seen.k1 * 16, lane);
          __syncwarp();
          tc::fence_after_sync();
#pragma unroll 1
          for (int kk = seen.k0; kk < seen.k1; ++kk) product(kk, !v_first || kk > seen.k0);
        }
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
          seen = tc::seen_rows(j < t.n_st, (int64_t)a.sinks - t.key(j), t.lo - t.key(j), t.end - t.key(j));
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
      const float inv = 1.f / out_l;  // a row sees a key, itself: 0 (logits of -inf) and NaN are to show
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
            (out_m + __log2f(out_l)) * 0.69314718055994530942f;
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
      int64_t lo64, hi64;
      visible_range((int64_t)t.pos0 + (row_valid ? t.q0 + row : a.S - 1), a.window, t.n_keys, &lo64, &hi64);
      const int lo = (int)lo64, hi = (int)hi64;
      float m_used = -INFINITY, l = 0.f;
      bool left = false;  // both warps, at a vote
      for (int j = 0; j < t.n_tiles; ++j, ++jt) {
        const int kb = t.key(j);
        ok = ok && wait_all(&ctl->s_full[jt & 1], (jt >> 1) & 1, abort_flag, deadline, a.status, 57, jt, n);
        tc::fence_after_sync();
        const uint32_t s_tm = tm + COL_S + (uint32_t)((jt & 1) * 128 + half * 64);
        uint32_t r[2][32];
        tc::tmem_ld32(s_tm, r[0]);
        tc::tmem_ld32(s_tm + 32, r[1]);
        tc::tmem_wait_ld();
        if (!((kb >= lo || kb + BN <= a.sinks) && kb + BN - 1 <= hi)) {
          const int c_lo = lo - kb, c_hi = hi - kb, c_sink = a.sinks - kb;
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

}  // namespace

// head_pair: pairs of heads where the group is even, else of row tiles
cudaError_t launch_prefill_attn_stream(const PrefillAttnArgs& a, int B, int head_pair, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo;
  if (!make_prefill_maps(a, B, 256, a.page_size, 0, BM, KH, BN, &mq, &mk, &mv, &mo)) return cudaErrorInvalidValue;
  const PairArgs t = pair_args(a, 0, head_pair);
  // outputs: boxes of a softmax warp's rows
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

}  // namespace hlg
