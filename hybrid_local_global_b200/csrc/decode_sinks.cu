// decode_sinks.cu -- single-token decode over a paged cache of which a query
// sees a sliding window and the sequence's first tokens ("sinks").
//
// For the new token of sequence b (position p = len - 1) and q head h (KV head
// g = h / G): out = sum_j softmax_j(scale <q~, k~_j>) v_j over the keys j <= p
// with j > p - window or j < sinks ("Gemma 4: End-to-End Architecture
// Walkthrough", 3a: a layer that attends to a fixed recent window).
//
// One launch does the whole step: RoPE of q, RoPE and append of the new key
// and value, the split over the visible keys, and the merge of the splits. The
// visible keys are few by definition, so a (sequence, KV head) needs few
// splits: they are the CTAs of one cluster and merge through distributed
// shared memory, without partial results in HBM or a second kernel.
//
// Visible keys are walked in tiles of 128 aligned positions (each in one page):
// those of the sinks, then those from the one that holds the window's first key
// on (one run when the two meet); of a tile at an edge only the 32-key blocks
// with visible keys are read. The product is taken transposed, as in the
// multi-token kernel, so that the keys fill the MMA's 128 rows and the few q
// heads are its columns:
//   S^T = K Q^T    (M = 128 keys, N = 16, K = head_dim)
//   O^T += V^T P^T (M = 128 value dims per MMA, N = 16, K = 32 keys per block)
// A group has at most 8 heads and N is at least 16: columns 0..7 take the bf16
// values of Q~ (and of the weights P), columns 8..15 what that rounding lost,
// and the two halves are added, so neither rounding shows in the result. The new
// token's logits are 32-bit sums. The angle is formed and reduced in 64 bits and
// then rounded to 32 (off by 9.4e-8 rad, a 40000th of a bf16 half step).
//
// CTA = 224 threads: warp 0 loads 32 KB stages of 128 keys x 128 dims (one TMA
// copy, or boxes of 32 keys where a tile has fewer blocks), warp 1 issues the
// MMAs and owns TMEM, warps 2..5 rotate q and the new key, run the softmax
// (thread = key = TMEM lane) and merge. Warp 6 puts the stages of edge tiles in
// order before their MMAs: the new token's row, which is not read back from the
// cache, and zeros in the rows of V that the query does not see (they are
// masked in S and their weight is 0, but 0 * NaN is not).
//
// HBM-bound: every visible K/V byte is read once per KV head (under K = V
// the second read of a row hits L2).
//
// Every wait is bounded; after a timeout the cluster still meets at its
// barriers and writes no output (GEMMA_ERR_DEVICE_TIMEOUT).
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace hlg {

namespace {

constexpr int BLK = 32;             // keys per block (SinkSpan)
constexpr int BN = 128;             // keys per tile
constexpr int NT = 224;             // threads
constexpr int NQ = 16;              // MMA columns: 8 heads, then 8 remainders
constexpr int CH_B = BN * 128;      // [128 keys][64 dims], swizzled
constexpr int STAGE_B = 2 * CH_B;   // 128 dims of a K or V tile
constexpr int BOX_B = BLK * 128;    // one TMA box: 32 keys x 64 dims
constexpr int P_B = 2 * NQ * 128;   // P^T: two chunks of 64 keys
constexpr int MAX_CLUSTER = 16;     // CTAs per (sequence, KV head); above 8 where the device allows it
constexpr float RESCALE_LOG2 = 8.0f;
constexpr uint32_t IDESC_ST = tc::idesc_bf16_f32(128, NQ, 0, 0);  // K (K-major) x Q (K-major)
constexpr uint32_t IDESC_OT = tc::idesc_bf16_f32(128, NQ, 1, 0);  // V^T (MN-major) x P^T (K-major)

template <int NS>
struct Ctl {
  uint64_t full[NS], empty[NS];
  uint64_t patch_req;             // the issuer has come to the next stages that need warp 6
  uint64_t patched[NS];           // and their rows are in order
  uint64_t q_ready;               // 128 softmax threads: Q and the new rows are staged
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued, taken;              // stages loaded, stages whose load was waited for
  float m[8], f[8], l[8];         // running maxima, rescale factors, sums (this CTA)
  float s_new[4][8];              // the new key's logits, partial sums of each softmax warp
  float red[4][8];
  alignas(16) float wgt[MAX_CLUSTER][8];
  float2 ml[MAX_CLUSTER][8];      // the cluster's (m, l); l < 0: that CTA gave up
};

// CTAS per SM. Two overlap one CTA's prologue and merge with the other's
// stream; one has the whole shared memory for its ring.
template <int D, int CTAS>
struct Cfg {
  static constexpr int MT = D / 128;                 // K stages per tile = O^T blocks = V stages per tile
  static constexpr int Q_B = (D / 64) * NQ * 128;
  static constexpr int NS = CTAS == 2 ? 2 : D == 512 ? 5 : 6;
  static constexpr int Q_OFF = NS * STAGE_B;
  static constexpr int P_OFF = Q_OFF + Q_B;          // two buffers; the angles before the first tile
  static constexpr int NEW_OFF = P_OFF + 2 * P_B;    // the new token's K row, V row
  static constexpr int MERGE_OFF = NEW_OFF + 2 * D * 2;  // [split][column][head]: this CTA's columns of every O^T
  static constexpr int CTL_OFF = MERGE_OFF + 8 * D * 4;
  static constexpr int SMEM = 1024 + CTL_OFF + (int)sizeof(Ctl<NS>);
  static constexpr uint32_t COL_S = MT * NQ;         // after O^T
  static constexpr uint32_t TMEM_COLS = MT * NQ + 2 * NQ <= 64 ? 64 : 128;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "resident CTAs");
  static_assert((D / 2) * 8 <= 2 * P_B, "angles");
};


__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t deadline,
                                         int* status, int where, int a, int b, int c) {
  return __all_sync(0xffffffffu, mbar_wait_bounded_at(bar, parity, abort_flag, deadline, status, where, a, b, c));
}

// OR of a predicate over the 128 softmax threads (named barrier 1).
__device__ __forceinline__ bool any128(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void st_cluster4(uint32_t addr, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w)
               : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// x[c] is this lane's value of column c; returns, in lane l, the max (or sum)
// over the warp of column l % 8. Each of the first steps hands half of the
// remaining columns to the partner lane.
template <bool MAX>
__device__ __forceinline__ float reduce8(const float (&in)[8], int lane) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = in[i];
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, o);
      x[i] = MAX ? fmaxf(keep, recv) : keep + recv;
    }
  }
#pragma unroll
  for (int o = 8; o <= 16; o <<= 1) {
    const float recv = __shfl_xor_sync(0xffffffffu, x[0], o);
    x[0] = MAX ? fmaxf(x[0], recv) : x[0] + recv;
  }
  return x[0];
}

// rotate the four pairs of 16 bytes at dims 8c .. of a vector
__device__ __forceinline__ void turn4(const uint4& x, int c, int n_rot, const float2* trig, float2 (&y)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = unpack_bf16x2(w[j]);
    if (c * 4 + j < n_rot) {
      const float2 t = trig[c * 4 + j];
      y[j] = make_float2(y[j].x * t.x - y[j].y * t.y, y[j].x * t.y + y[j].y * t.x);
    }
  }
}

struct Maps {
  CUtensorMap k, v;            // boxes of 128 keys x 128 dims
  CUtensorMap k_part, v_part;  // boxes of 32 keys x 64 dims
};

template <int D, int CTAS>
__global__ void __launch_bounds__(NT, CTAS)
    k_decode_sinks(const __grid_constant__ Maps maps, const __grid_constant__ SinkDecodeArgs a) {
  using C = Cfg<D, CTAS>;
  constexpr int NS = C::NS, MT = C::MT, CH = D / 8;  // CH: 16-byte chunks of a row
  extern __shared__ unsigned char sm_raw[];
  const uint32_t raw = smem_u32(sm_raw);
  const uint32_t base = (raw + 1023) & ~1023u;
  unsigned char* sm = sm_raw + (base - raw);
  float2* trig = reinterpret_cast<float2*>(sm + C::P_OFF);
  bf16* newrow = reinterpret_cast<bf16*>(sm + C::NEW_OFF);
  Ctl<NS>* ctl = reinterpret_cast<Ctl<NS>*>(sm + C::CTL_OFF);
  volatile int* abort_flag = &ctl->abort;

  const int split = blockIdx.x, n_splits = gridDim.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const int64_t len = a.seq_lens[b];
  const int64_t head0 = (int64_t)b * a.Hq + (int64_t)g * G;  // first q row of the group
  if (len < 1 || len > a.max_len) {  // an idle slot (0) or a bad length: zeros; the whole cluster leaves here
    if (len != 0 && tid == 0 && split == 0 && g == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
    if (split == 0)
      for (int i = tid; i < G * CH; i += NT)
        *reinterpret_cast<uint4*>(a.out + head0 * D + i * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool has_new = a.k_new != nullptr;
  const int len_c = (int)len - (has_new ? 1 : 0);  // rows that are read from the cache
  const SinkSpan sp = sink_span(len, a.window, a.sinks);
  const int per = (sp.tiles + n_splits - 1) / n_splits;
  const int tile0 = min(split * per, sp.tiles);
  const int n_tiles = min(per, sp.tiles - tile0);
  const bool own_new = has_new && n_tiles > 0 && tile0 + n_tiles == sp.tiles;  // the last tile holds the new token
  // position of row 0 and 32-row blocks of this CTA's tile j
  const auto tile = [&](int j, int* nb) { return sp.block0(tile0 + j, (int)len, a.sinks, nb); };
  // whether tile j has rows that the query does not see among the cached ones
  const auto is_edge = [&](int p0, int nb) {
    return !(p0 + nb * BLK <= len_c && (p0 >= sp.lo || p0 + nb * BLK <= a.sinks));
  };

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
      mbar_init(&ctl->patched[s], 1);
    }
    mbar_init(&ctl->q_ready, 128);
    mbar_init(&ctl->patch_req, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_ready[i], 128);
      mbar_init(&ctl->o_done[i], 1);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = ctl->issued = ctl->taken = 0;
    fence_barrier_init();
  }
  if (tid < 8) ctl->m[tid] = -INFINITY;
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  // (producer) the first tile's table entry, ahead of the barriers
  const int32_t* table = a.page_table + (int64_t)b * a.pages_per_seq;
  int nb0 = 0, p0_0 = 0, entry0 = 0;
  if (warp == 0 && n_tiles > 0) {
    p0_0 = tile(0, &nb0);
    entry0 = table[p0_0 / a.page_size];
  }
  __syncwarp();
  __syncthreads();
  pair::cluster_arrive();  // this CTA runs: its shared memory may be written by the others
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;
  float l[8];  // softmax threads: this key lane's sums
#pragma unroll
  for (int n = 0; n < 8; ++n) l[n] = 0.f;
  bool good = true;  // softmax threads

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t go = tc::elect_one();
    if (go) {
      tc::prefetch_tmap(&maps.k);
      tc::prefetch_tmap(&maps.v);
      tc::prefetch_tmap(&maps.k_part);
      tc::prefetch_tmap(&maps.v_part);
    }
    int item = 0;
    bool ok = true;
    const auto load = [&](int p0, int nb, int entry, bool isv) {
      const bool outside = entry < 0 || entry >= a.n_pages;  // report it and read page 0 (finite, wrong)
      if (outside && go) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
      const int page = outside ? 0 : entry, row = p0 % a.page_size;
      // one copy may read rows past the tile's blocks, which nothing uses (past
      // the page they arrive as zeros): worth it for one block in four, or
      // where the call leaves HBM idle
      const bool one = CTAS == 1 || nb >= 3;
      const CUtensorMap* map = one ? (isv ? &maps.v : &maps.k) : (isv ? &maps.v_part : &maps.k_part);
      const uint32_t bytes = one ? STAGE_B : nb * 2 * BOX_B;
      for (int h = 0; h < MT; ++h, ++item) {
        const int s = item % NS;
        if (item >= NS)
          ok = wait_all(&ctl->empty[s], ((item / NS) - 1) & 1, abort_flag, deadline, a.status, 51, item, s, p0);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (a.drop_first_copy && item == 0 && split == 0 && g == 0 && b == 0) continue;
        const uint32_t dst = base + s * STAGE_B, bar = smem_u32(&ctl->full[s]);
        if (go) {
          mbar_arrive_expect_tx(&ctl->full[s], bytes);
          ctl->issued = item + 1;
        }
        __syncwarp();
        tc::tma_load_5d_if(go, dst, map, 0, row, h * 2, g, page, bar);
        if (!one) {
          tc::tma_load_5d_if(go, dst + CH_B, map, 0, row, h * 2 + 1, g, page, bar);
          if (nb > 1) {
            tc::tma_load_5d_if(go, dst + BOX_B, map, 0, row + BLK, h * 2, g, page, bar);
            tc::tma_load_5d_if(go, dst + CH_B + BOX_B, map, 0, row + BLK, h * 2 + 1, g, page, bar);
          }
        }
      }
    };
    // K_0, K_1, V_0, K_2, V_1, ...; a tile's table entry is read a tile ahead
    int nb = nb0, pnb = 0, p0 = p0_0, pp0 = 0, entry = entry0, pentry = 0;
    for (int j = 0; j < n_tiles && ok; ++j) {
      int nnb = 0, np0 = 0, nentry = 0;
      if (j + 1 < n_tiles) {
        np0 = tile(j + 1, &nnb);
        nentry = table[np0 / a.page_size];
      }
      load(p0, nb, entry, false);
      if (j > 0 && ok) load(pp0, pnb, pentry, true);
      pp0 = p0, pnb = nb, pentry = entry;
      p0 = np0, nb = nnb, entry = nentry;
    }
    if (n_tiles > 0 && ok) load(pp0, pnb, pentry, true);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t go = tc::elect_one();
    bool ok = n_tiles == 0 || wait_all(&ctl->q_ready, 0, abort_flag, deadline, a.status, 50, 0, 0, 0);
    const uint64_t dk = tc::smem_desc_sw128(base, 16, 1024), dv = tc::smem_desc_sw128(base, CH_B, 1024);
    const uint64_t dq = tc::smem_desc_sw128(base + C::Q_OFF, 16, 1024), dp = dq + ((C::P_OFF - C::Q_OFF) >> 4);
    int item = 0, taken = 0;
    uint32_t patches = 0;  // parity of each slot's next patch
    // waits for the next stage (and its patch); returns its slot
    const auto take = [&](bool patch) {
      const int s = item % NS;
      const uint32_t parity = patch ? patches >> s & 1u : (uint32_t)(item / NS) & 1u;
      ok = wait_all(patch ? &ctl->patched[s] : &ctl->full[s], parity, abort_flag, deadline, a.status, 52, item, s,
                    patch);
      if (patch) patches ^= 1u << s;
      tc::fence_after_sync();
      ++item;
      if (ok) taken = item;
      return s;
    };
    const auto values = [&](int p0, int nb, int j) {  // O^T += V_j^T P_j^T
      const bool patch = is_edge(p0, nb);
      if (patch && go) mbar_arrive(&ctl->patch_req);
      ok = wait_all(&ctl->p_ready[j & 1], (j >> 1) & 1, abort_flag, deadline, a.status, 53, j, 0, 0);
      const uint64_t pj = dp + (uint64_t)((j & 1) * (P_B >> 4));
      for (int m = 0; m < MT && ok; ++m) {
        const int s = take(patch);
        if (!ok) break;
        // V^T: 128 dims (two 64-dim boxes CH_B apart) x 16 keys; P^T: 16 columns x 16 keys
        const uint64_t v = dv + (uint64_t)(s * (STAGE_B >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk < 2 * nb)
            tc::mma_ss_if(go, tmem + m * NQ, v + kk * (2048 >> 4),
                          pj + (kk >> 2) * (NQ * 128 >> 4) + (kk & 3) * 2, IDESC_OT, (j > 0 || kk) ? 1u : 0u);
        tc::commit_if(go, smem_u32(&ctl->empty[s]));
      }
      if (ok) tc::commit_if(go, smem_u32(&ctl->o_done[j & 1]));
    };
    int pp0 = 0, pnb = 0;
    for (int j = 0; j < n_tiles && ok; ++j) {
      int nb;
      const int p0 = tile(j, &nb);
      for (int h = 0; h < MT; ++h) {  // S_j^T = K_j Q^T
        const int s = take(false);
        if (!ok) break;
        const uint64_t k = dk + (uint64_t)(s * (STAGE_B >> 4)), qh = dq + (uint64_t)(h * (2 * NQ * 128 >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_ss_if(go, tmem + C::COL_S + (j & 1) * NQ, k + (kk >> 2) * (CH_B >> 4) + (kk & 3) * 2,
                        qh + (kk >> 2) * (NQ * 128 >> 4) + (kk & 3) * 2, IDESC_ST, (h | kk) != 0);
        tc::commit_if(go, smem_u32(&ctl->empty[s]));
      }
      if (!ok) break;
      tc::commit_if(go, smem_u32(&ctl->s_full[j & 1]));
      if (j > 0) values(pp0, pnb, j - 1);
      pp0 = p0;
      pnb = nb;
    }
    if (n_tiles > 0 && ok) values(pp0, pnb, n_tiles - 1);
    // no MMA may be in flight when TMEM or shared memory is released
    tc::commit_if(go, smem_u32(&ctl->drain));
    volatile int never = 0;
    mbar_wait_bounded_at(&ctl->drain, 0, &never, globaltimer_ns() + 200000000ull, a.status, 55, 0, 0, 0);
    if (go) ctl->taken = taken;
  } else if (warp == 6) {
    // ------------------------------------------------------------ edge rows
    // The issuer asks for a V tile that needs this warp once it has waited for
    // all stages before it: the parity waits here cannot mistake an older phase
    // for the stage's own. lane: 16-byte unit lane % 16 (of the 128 dims) of
    // every second row.
    bool ok = n_tiles == 0 || wait_all(&ctl->q_ready, 0, abort_flag, deadline, a.status, 61, 0, 0, 0);
    const int cc = (lane >> 3) & 1, u = lane & 7;
    int groups = 0;
    for (int j = 0; j < n_tiles && ok; ++j) {
      int nb;
      const int p0 = tile(j, &nb);
      if (!is_edge(p0, nb)) continue;
      ok = wait_all(&ctl->patch_req, groups++ & 1, abort_flag, deadline, a.status, 63, j, 0, 0);
      uint32_t off[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        off[q] = __ballot_sync(0xffffffffu, q < nb && !sp.sees(p0 + q * BLK + lane, len_c, a.sinks));
      const int new_row = own_new && j == n_tiles - 1 ? len_c - p0 : -1;
      // items: K_0, K_1, V_0, K_2, V_1, ..., V_{n-2}, V_{n-1}
      int item = MT * (j < n_tiles - 1 ? 2 * j + 2 : 2 * n_tiles - 1);
      for (int h = 0; h < MT && ok; ++h, ++item) {
        const int s = item % NS;
        ok = wait_all(&ctl->full[s], (item / NS) & 1, abort_flag, deadline, a.status, 62, item, s, j);
        if (!ok) break;
        unsigned char* st = sm + s * STAGE_B + cc * CH_B;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!(off[q] >> (16 * half) & 0xffffu)) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = half * 16 + 2 * k + (lane >> 4);
              if (off[q] >> r & 1u)
                *reinterpret_cast<uint4*>(st + (q * BLK + r) * 128 + ((u ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
          }
        __syncwarp();
        if (new_row >= 0 && lane < 16)
          *reinterpret_cast<uint4*>(st + new_row * 128 + ((u ^ (new_row & 7)) << 4)) =
              *reinterpret_cast<const uint4*>(newrow + (a.keqv ? 0 : D) + h * 128 + lane * 8);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->patched[s]);
      }
    }
  } else {
    // ------------------------------------------------------------ rotation, softmax
    const int q4 = warp & 3;
    const int kl = q4 * 32 + lane;  // this thread's key of a tile = its TMEM lane
    const int t128 = tid - 64;
    const uint32_t tm = tmem + ((uint32_t)(q4 * 32) << 16);
    if (n_tiles > 0) {
      // Q^T rows 0..7: heads, 8..15: their remainders; 128-byte rows of 64
      // dims, 16-byte units swizzled by the row
      uint4 x[8 * CH / 128];
#pragma unroll
      for (int k = 0; k < 8 * CH / 128; ++k) {
        const int i = t128 + k * 128, r = i / CH, c = i % CH;
        x[k] = r < G ? *reinterpret_cast<const uint4*>(a.q + (head0 + r) * D + c * 8) : make_uint4(0, 0, 0, 0);
      }
      for (int i = t128; i < a.n_rot; i += 128) {
        const double ang = (double)(len - 1) * a.freq[i];
        float s, c;
        sincospif((float)(ang - 2.0 * rint(0.5 * ang)), &s, &c);
        trig[i] = make_float2(c, s);
      }
      sync128();
      // The new key's logits are formed here (its row of S is not used): a
      // thread has 8 dims of some heads and of the key, a warp adds them up.
      const int c = t128 % CH;
      float2 kn[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kn[j] = make_float2(0.f, 0.f);
      if (own_new) {
        turn4(*reinterpret_cast<const uint4*>(a.k_new + ((int64_t)b * a.Hkv + g) * D + c * 8), c, a.n_rot, trig, kn);
#pragma unroll
        for (int j = 0; j < 4; ++j) kn[j] = unpack_bf16x2(pack_bf16x2(kn[j].x, kn[j].y));  // as the cache holds it
      }
#pragma unroll
      for (int k = 0; k < 8 * CH / 128; ++k) {
        const int r = (t128 + k * 128) / CH;
        float2 y[4];
        turn4(x[k], c, a.n_rot, trig, y);
        if (own_new) {
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) dot += y[j].x * kn[j].x + y[j].y * kn[j].y;
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
          if (lane == 0) ctl->s_new[t128 >> 5][r] = dot;
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[j] = pack_bf16x2(y[j].x, y[j].y);
          const float2 h = unpack_bf16x2(hi[j]);
          lo[j] = pack_bf16x2(y[j].x - h.x, y[j].y - h.y);
        }
        unsigned char* dst = sm + C::Q_OFF + (c >> 3) * (NQ * 128) + r * 128 + (((c & 7) ^ r) << 4);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (own_new && t128 < (a.keqv ? 1 : 2) * CH) {
        const int64_t crow = cache_row(a.page_table, a.pages_per_seq, a.page_size, a.n_pages, a.Hkv, b, g, len - 1);
        if (crow < 0 && t128 == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        const bool isv = t128 >= CH;
        uint4 v = make_uint4(pack_bf16x2(kn[0].x, kn[0].y), pack_bf16x2(kn[1].x, kn[1].y),
                             pack_bf16x2(kn[2].x, kn[2].y), pack_bf16x2(kn[3].x, kn[3].y));
        if (isv) v = *reinterpret_cast<const uint4*>(a.v_new + ((int64_t)b * a.Hkv + g) * D + c * 8);
        *reinterpret_cast<uint4*>(newrow + (isv ? D : 0) + c * 8) = v;
        if (crow >= 0) *reinterpret_cast<uint4*>((isv ? a.v_pool : a.k_pool) + crow * D + c * 8) = v;
      }
      fence_proxy_async_smem();
      mbar_arrive(&ctl->q_ready);
    }
    // The running maxima live in shared memory. The four warps pass the same
    // named barriers in the same order whatever their waits return: a failed
    // wait marks the thread bad, and the vote of the next tile ends the loop
    // for all of them.
    bool bad = false;
    int pv_seen = 0;  // PV_0 .. PV_{pv_seen-1} are known complete
    for (int j = 0; j < n_tiles; ++j) {
      int nb;
      const int p0 = tile(j, &nb);
      if (!bad && !wait_all(&ctl->s_full[j & 1], (j >> 1) & 1, abort_flag, deadline, a.status, 56, j, 0, 0)) bad = true;
      tc::fence_after_sync();
      float v[8];
      {
        uint32_t r[16];
        tmem_ld16(tm + C::COL_S + (uint32_t)(j & 1) * NQ, r);
        tc::tmem_wait_ld();
        const bool seen = kl < nb * BLK && sp.sees(p0 + kl, (int)len, a.sinks);
#pragma unroll
        for (int n = 0; n < 8; ++n)
          v[n] = seen ? (__uint_as_float(r[n]) + __uint_as_float(r[n + 8])) * a.scale_log2 : -INFINITY;
        // (its row is in the last tile; an earlier one of few blocks may end less than 128 before it)
        if (own_new && j == n_tiles - 1 && p0 + kl == len_c) {
          // head n's dims lie in the warps with threads of row n: D / 256 of them
#pragma unroll
          for (int n = 0; n < 8; ++n)
            v[n] = (D == 512 ? ctl->s_new[(n & 1) * 2][n] + ctl->s_new[(n & 1) * 2 + 1][n] : ctl->s_new[n & 3][n]) *
                   a.scale_log2;
        }
      }
      bool need = bad;
#pragma unroll
      for (int n = 0; n < 8; ++n) need |= v[n] > ctl->m[n] + RESCALE_LOG2;
      if (j == 0 || any128(need)) {
        // some logit exceeds its head's running max by more than 2^8 (or a
        // wait failed): the tile's maxima, and thread n moves head n's
        if (any128(bad)) break;
        const float mx = reduce8<true>(v, lane);
        if (lane < 8) ctl->red[q4][lane] = mx;
        sync128();
        bool moved = false;
        if (kl < 8) {
          const float mold = ctl->m[kl];
          const float mnew =
              fmaxf(mold, fmaxf(fmaxf(ctl->red[0][kl], ctl->red[1][kl]), fmaxf(ctl->red[2][kl], ctl->red[3][kl])));
          ctl->f[kl] = mold == -INFINITY ? 0.f : tc::ex2(mold - mnew);
          ctl->m[kl] = mnew;
          moved = mold != -INFINITY && mnew != mold;
        }
        moved = any128(moved);  // also publishes m and f
#pragma unroll
        for (int n = 0; n < 8; ++n) l[n] *= ctl->f[n];
        if (moved && j >= 1) {
          // O^T must hold PV_{j-1} before it is rescaled
          if (pv_seen < j) {
            if (wait_all(&ctl->o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 57, j, 0, 0))
              pv_seen = j;
            else
              bad = true;
          }
          if (!bad) {
            tc::fence_after_sync();
#pragma unroll 1
            for (int m = 0; m < MT; ++m) {
              uint32_t o[16];
              tmem_ld16(tm + m * NQ, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ctl->f[e & 7]);
              tmem_st16(tm + m * NQ, o);
            }
            tc::tmem_wait_st();
          }
        }
      }
      // P buffer j & 1 is free once PV_{j-2} is done
      if (!bad && j >= 2 && pv_seen < j - 1) {
        if (wait_all(&ctl->o_done[j & 1], ((j - 2) >> 1) & 1, abort_flag, deadline, a.status, 58, j, 0, 0))
          pv_seen = j - 1;
        else
          bad = true;
      }
      if (bad) continue;  // no arrival: the issuer's bounded wait sees the abort
      unsigned char* prow = sm + C::P_OFF + (j & 1) * P_B + (kl >> 6) * (NQ * 128) + (kl & 7) * 2;
      const int unit = (kl & 63) >> 3;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float mm = ctl->m[n];
        const float p = tc::ex2(v[n] - (mm == -INFINITY ? 0.f : mm));
        l[n] += p;
        const bf16 hi = __float2bfloat16_rn(p);
        *reinterpret_cast<bf16*>(prow + n * 128 + ((unit ^ n) << 4)) = hi;
        *reinterpret_cast<bf16*>(prow + 1024 + n * 128 + ((unit ^ n) << 4)) =
            __float2bfloat16_rn(p - __bfloat162float(hi));
      }
      fence_proxy_async_smem();
      tc::fence_before_sync();
      mbar_arrive(&ctl->p_ready[j & 1]);
    }
    if (!bad && n_tiles > 0)
      bad = !wait_all(&ctl->o_done[(n_tiles - 1) & 1], ((n_tiles - 1) >> 1) & 1, abort_flag, deadline, a.status, 59,
                      n_tiles, 0, 0);
    good = !any128(bad);
    // sums over the tile's 128 key lanes
    const float s = reduce8<false>(l, lane);
    if (lane < 8) ctl->red[q4][lane] = s;
    sync128();
    if (kl < 8) ctl->l[kl] = (ctl->red[0][kl] + ctl->red[1][kl]) + (ctl->red[2][kl] + ctl->red[3][kl]);
    sync128();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // loads still in flight must land before the CTA leaves (a
    // dropped copy, the test hook's, never does: its wait runs out)
    volatile int never = 0;
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    for (int i = ctl->taken; i < ctl->issued; ++i)
      mbar_wait_bounded_at(&ctl->full[i % NS], (i / NS) & 1, &never, dl, a.status, 60, i, i % NS, ctl->taken);
  }
  __syncwarp();
  pair::cluster_wait();  // every CTA has begun
  // Each CTA owns D / n_splits output columns; the others push their share of
  // those into its merge buffer, and their (m, l).
  const int log_n = __ffs(n_splits) - 1, log_cols = (D == 256 ? 8 : 9) - log_n, cols = 1 << log_cols;
  if (warp >= 2 && warp < 6) {
    const int kl = (warp & 3) * 32 + lane;
    if (kl < n_splits * 8)
      st_cluster2(pair::map_to(smem_u32(&ctl->ml[split][kl & 7]), kl >> 3), ctl->m[kl & 7],
                  good ? ctl->l[kl & 7] : -1.f);
    if (n_tiles > 0) {
      tc::fence_after_sync();
      const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      uint32_t o[MT][16];
#pragma unroll
      for (int m = 0; m < MT; ++m) tmem_ld16(tm + m * NQ, o[m]);
      tc::tmem_wait_ld();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float x[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] = __uint_as_float(o[m][n]) + __uint_as_float(o[m][n + 8]);
        const int d = m * 128 + kl;
        const uint32_t to = pair::map_to(base + C::MERGE_OFF, d >> log_cols) + ((split << log_cols) + (d & (cols - 1))) * 32;
        st_cluster4(to, x[0], x[1], x[2], x[3]);
        st_cluster4(to + 16, x[4], x[5], x[6], x[7]);
      }
    }
  }
  tc::fence_before_sync();
  __syncwarp();
  pair::cluster_sync();  // every share has arrived; nothing remote follows
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // Weight of each split's share, 2^(m_s - M) / L (thread: head tid % 8 of split
  // tid / 8). A head's maximum is -inf in a split that saw no number above it: no
  // tile at all (sum 0), logits of -inf (0) or only NaN (a NaN sum, which must reach
  // L: the softmax of NaN is NaN, and so is 0 / 0 where every logit is -inf).
  if (tid < n_splits * 8) {
    const int n = tid & 7;
    float M = -INFINITY, L = 0.f;
    bool ok = true;
    for (int s = 0; s < n_splits; ++s) M = fmaxf(M, ctl->ml[s][n].x);
    for (int s = 0; s < n_splits; ++s) {
      const float2 ml = ctl->ml[s][n];
      ok = ok && !(ml.y < 0.f);
      L += (ml.x == -INFINITY ? 0.f : tc::ex2(ml.x - M)) * ml.y;
    }
    const float m = ctl->ml[tid >> 3][n].x;
    ctl->wgt[tid >> 3][n] = (m == -INFINITY ? 0.f : tc::ex2(m - M)) / L;
    if (!ok) ctl->abort = 1;  // some CTA gave up: no output
  }
  __syncthreads();
  if (*abort_flag) return;
  const int n_full = (sp.tiles + per - 1) / per;  // splits with tiles: the others pushed no share
  for (int i = tid; i < 2 * cols; i += NT) {  // (heads 4 hh .. 4 hh + 3, column d)
    const int hh = i >> log_cols, d = i & (cols - 1);
    if (4 * hh >= G) break;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < n_full; ++s) {
      const float4 w = *reinterpret_cast<const float4*>(&ctl->wgt[s][4 * hh]);
      const float4 v = *reinterpret_cast<const float4*>(sm + C::MERGE_OFF + ((s << log_cols) + d) * 32 + hh * 16);
      x[0] += w.x * v.x;
      x[1] += w.y * v.y;
      x[2] += w.z * v.z;
      x[3] += w.w * v.w;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (4 * hh + n < G)
        a.out[(head0 + 4 * hh + n) * D + (split << log_cols) + d] = __float2bfloat16_rn(x[n]);
  }
}

template <int D, int CTAS>
void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, int n_splits, int Hkv, int B, cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(n_splits, Hkv, B);
  cfg->blockDim = dim3(NT);
  cfg->dynamicSmemBytes = Cfg<D, CTAS>::SMEM;
  cfg->stream = st;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = n_splits;
  at->val.clusterDim.y = 1;
  at->val.clusterDim.z = 1;
  cfg->attrs = at;
  cfg->numAttrs = 1;
}

// Clusters of 2^log_n CTAs that the device holds at once with one CTA per SM
// (0: none): a property of the device, asked once. Sets the attributes of
// both instances.
template <int D>
int resident(int log_n) {
  static std::mutex mu;
  static int known[128][5];  // 1 + the answer
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
  std::lock_guard<std::mutex> lk(mu);
  int& k = known[dev][log_n];
  if (!k) {
    const auto one = k_decode_sinks<D, 1>;
    const auto two = k_decode_sinks<D, 2>;
    const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const auto large = cudaFuncAttributeNonPortableClusterSizeAllowed;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at;
    config<D, 1>(&cfg, &at, 1 << log_n, 1, 1, nullptr);
    int n = 0;
    if (cudaFuncSetAttribute(one, smem, Cfg<D, 1>::SMEM) != cudaSuccess ||
        cudaFuncSetAttribute(two, smem, Cfg<D, 2>::SMEM) != cudaSuccess ||
        (log_n > 3 && (cudaFuncSetAttribute(one, large, 1) != cudaSuccess ||
                       cudaFuncSetAttribute(two, large, 1) != cudaSuccess)) ||
        cudaOccupancyMaxActiveClusters(&n, one, &cfg) != cudaSuccess) {
      n = 0;
      (void)cudaGetLastError();  // this size is not to be had: another one is taken
    }
    k = 1 + n;
  }
  return k - 1;
}

template <int D>
cudaError_t launch(const Maps& maps, const SinkDecodeArgs& a, int B, cudaStream_t st) {
  // The split (a power of two, up to one cluster) and one or two CTAs per SM
  // that look quickest. A tile of 2 x 128 keys takes a CTA that has its SM to
  // itself 2.8 us at head_dim 512 and one that shares it 5.5 us; a wave of
  // clusters costs 8 us besides, and HBM gives 6500 bytes a ns. Measured with
  // every choice: 4096 keys, 4 KV heads, 4 sequences: 32 us (4 CTAs each, alone),
  // 36 (8, shared), 48 (8, alone: the clusters do not fit at once), 96 (1, alone);
  // 64 sequences: 314 us (1, shared), 316 (2), 333 (4), 367 (8).
  const SinkSpan sp = sink_span(a.max_len, a.window, a.sinks);
  const double tile = D / 512.0, pairs = (double)B * a.Hkv;
  const double hbm = pairs * sp.tiles * (a.keqv ? 1 : 2) * (BN * D * 2.0) / 6.5e6;
  double best = 1e300;
  int best_n = 0, best_ctas = 2;
  for (int log_n = 0; log_n < 5; ++log_n)
    for (int ctas = 1; ctas <= 2; ++ctas) {
      const int fit = ctas * resident<D>(log_n);
      if (fit <= 0) continue;
      const int per = (sp.tiles + (1 << log_n) - 1) >> log_n;
      const double waves = std::ceil(pairs / fit);
      const double cost = std::max(waves * per * tile * (ctas == 1 ? 2.8 : 5.5), hbm) + 8.0 * waves;
      if (cost < best) {
        best = cost;
        best_n = 1 << log_n;
        best_ctas = ctas;
      }
    }
  if (!best_n) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute at;
  if (best_ctas == 1) {
    config<D, 1>(&cfg, &at, best_n, a.Hkv, B, st);
    return cudaLaunchKernelEx(&cfg, k_decode_sinks<D, 1>, maps, a);
  }
  config<D, 2>(&cfg, &at, best_n, a.Hkv, B, st);
  return cudaLaunchKernelEx(&cfg, k_decode_sinks<D, 2>, maps, a);
}

}  // namespace

cudaError_t launch_decode_sinks(SinkDecodeArgs& a, int B, int D, double log2_theta, cudaStream_t st) {
  half_turn_ladder(2.0 / D * log2_theta, a.n_rot, a.freq);
  // (64 dims, row, 64-dim chunk, head, page): a box of 2 chunks is a stage
  const uint64_t ps = (uint64_t)a.page_size, H = (uint64_t)a.Hkv, d = (uint64_t)D;
  const uint64_t dims[5] = {64, ps, d / 64, H, (uint64_t)a.n_pages};
  const uint64_t str[4] = {d * 2, 128, ps * d * 2, H * ps * d * 2};
  const uint32_t whole[5] = {64, BN, 2, 1, 1}, part[5] = {64, BLK, 1, 1, 1};
  Maps maps;
  if (!make_map_bf16_5d(&maps.k, a.k_pool, dims, str, whole) || !make_map_bf16_5d(&maps.k_part, a.k_pool, dims, str, part))
    return cudaErrorInvalidValue;
  if (a.keqv) {
    maps.v = maps.k;
    maps.v_part = maps.k_part;
  } else if (!make_map_bf16_5d(&maps.v, a.v_pool, dims, str, whole) ||
             !make_map_bf16_5d(&maps.v_part, a.v_pool, dims, str, part)) {
    return cudaErrorInvalidValue;
  }
  return D == 256 ? launch<256>(maps, a, B, st) : launch<512>(maps, a, B, st);
}

}  // namespace hlg
