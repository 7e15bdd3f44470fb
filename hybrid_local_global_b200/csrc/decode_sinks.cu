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
// Visible keys are walked in a virtual order of whole KT-key tiles: those of
// the sinks, then those from the one that holds the window's first key on (one
// run when the two meet). A tile never straddles a page. Rows of an edge tile
// that the query does not see are masked in S and cleared in V (their weight
// is 0, but 0 * NaN is not). The new token's row is not read back from the
// cache: the CTA that appends it puts it into the tile it belongs to.
//
// CTA = 8 consumer warps and a producer warp, two CTAs per SM. The producer
// streams 32 KB tiles (K_0, V_0, K_1, ...) into a ring of three, as bulk copies
// of row groups (2 KB each, padded by 16 bytes so that ldmatrix is free of
// bank conflicts). For each tile
//   S: warp w takes 16 keys (w % KG) and 128 dims (w / KG) of Q K^T
//      (mma.sync m16n8k16), so its accumulation is 8 steps deep, and leaves its
//      partial sums in shared memory in fragment order;
//   softmax: after one barrier every warp adds up the partials of all KT keys
//      and runs the same online softmax (fp32, log2 domain) in registers;
//   O^T += V^T P^T: warp w takes D / 8 dims of the output for all keys.
// No warp holds more than its own output dims, so nothing is merged inside the
// CTA. (An earlier form, whole dims per warp and 16 keys at a time, took 2 us a
// step on its accumulation chain and 5 us to merge its warps.)
// The query is held to about 16 bits: the MMA's rows 0..7 are the heads'
// bf16 values and rows 8..15, which a group of at most 8 heads leaves free,
// what that rounding lost.
//
// HBM-bound: every visible K/V byte is read once per KV head.
//
// Every barrier wait is bounded; after a timeout the warps keep meeting at
// their barriers with the waits cut short, the cluster meets too, and no output
// is written (GEMMA_ERR_DEVICE_TIMEOUT).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "decode_ring.cuh"
#include "kernels.h"
#include "mma_sync.cuh"
#include "pair.cuh"

namespace hlg {

namespace {

using namespace ms;

constexpr int NCW = 8;          // consumer warps
constexpr int NCT = 32 * NCW;   // consumer threads
constexpr int MAX_CLUSTER = 8;  // CTAs per (sequence, KV head)
constexpr double kInvPi = 0.31830988618379067153776752674503;

template <int D>
struct SinkCfg {
  static constexpr int KT = 16384 / D;            // keys per tile: 32 KB of K (or V)
  static constexpr int KG = KT / 16;              // 16-key groups of a tile
  static constexpr int DQ = NCW / KG;             // parts of the dims in S
  static constexpr int KS = D / DQ / 16;          // MMA steps of a part
  static constexpr int MT = D / NCW / 16;         // 16-dim output tiles per warp
  static constexpr int RPC = 2048 / (D * 2);      // rows per bulk copy
  static constexpr int NGR = KT / RPC;            // row groups per tile
  static constexpr int SLOT_B = NGR * ring_group_bytes(D, RPC);
  static constexpr int NSLOT = 3;
  static constexpr int PART_OFF = NSLOT * SLOT_B;              // [2][NCW][32] float4 partial S
  static constexpr int NEW_OFF = PART_OFF + 2 * NCW * 32 * 16; // the new token's K row, V row
  static constexpr int TRIG_OFF = NEW_OFF + 2 * D * 2;
  static constexpr int BAR_OFF = TRIG_OFF + (D / 2) * 8;
  static constexpr int MISC_OFF = BAR_OFF + 2 * NSLOT * 8;     // ints: abort, issued, consumed
  static constexpr int ML_OFF = MISC_OFF + 32;                 // floats: m, l [MAX_CLUSTER][8], weights, 1 / L
  static constexpr int SMEM = ML_OFF + (3 * MAX_CLUSTER * 8 + 8) * 4;
  static_assert(1 + 2 * NSLOT <= 8, "misc ints");
  static_assert(8 * D * 4 <= PART_OFF, "the merge buffer overlays the drained ring");
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ void st_cluster(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

template <int D>
__global__ void __launch_bounds__(NCT + 32, 2) k_decode_sinks(const __grid_constant__ SinkDecodeArgs a) {
  using C = SinkCfg<D>;
  constexpr int RPC = C::RPC;
  extern __shared__ __align__(128) unsigned char sm[];
  unsigned char* ring = sm;
  float4* part = reinterpret_cast<float4*>(sm + C::PART_OFF);
  bf16* newrow = reinterpret_cast<bf16*>(sm + C::NEW_OFF);
  float2* trig = reinterpret_cast<float2*>(sm + C::TRIG_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  uint64_t* empty = full + C::NSLOT;
  int* misc = reinterpret_cast<int*>(sm + C::MISC_OFF);
  volatile int* abort_flag = misc;
  int* issued = misc + 1;
  int* consumed = issued + C::NSLOT;
  float2* ml = reinterpret_cast<float2*>(sm + C::ML_OFF);       // [splits][8] (m, l); l < 0: that CTA gave up
  float* wgt = reinterpret_cast<float*>(ml + MAX_CLUSTER * 8);  // [splits][8]

  const int split = blockIdx.x, n_splits = gridDim.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const int64_t len = a.seq_lens[b];
  const int64_t head0 = (int64_t)b * a.Hq + (int64_t)g * G;  // first q row of the group
  if (len < 1 || len > a.max_len) {  // an idle slot (0) or a bad length: zeros; the whole cluster leaves here
    if (len != 0 && tid == 0 && split == 0 && g == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
    if (split == 0)
      for (int i = tid; i < G * D / 8; i += NCT + 32)
        *reinterpret_cast<uint4*>(a.out + head0 * D + i * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool has_new = a.k_new != nullptr;
  const int len_c = (int)len - (has_new ? 1 : 0);  // rows that are read from the cache
  const SinkSpan sp = sink_span(len, a.window, a.sinks, C::KT);
  const int tiles = (sp.n + C::KT - 1) / C::KT;
  const int per = (tiles + n_splits - 1) / n_splits;
  const int tile0 = min(split * per, tiles);
  const int n_sub = min(per, tiles - tile0);
  const bool own_new = has_new && n_sub > 0 && tile0 + n_sub == tiles;  // this CTA's last tile holds the new token

  if (tid == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NCW);
      issued[s] = 0;
      consumed[s] = 0;
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;
  const int per_tile = a.keqv ? 1 : 2;  // ring items per tile: K, then V

  const int gq = lane >> 2, tg = lane & 3;
  float o[C::MT][4];
  float m_h = -INFINITY, l_t = 0.f;  // of head gq (the same in every warp); l of this lane's keys
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

  if (warp == NCW) {
    // ---------------- producer ----------------
    int page0 = -1, ent = 0;  // this lane's table entry: of page page0 + lane
    for (int i = 0; i < n_sub * per_tile; ++i) {
      const int slot = i % C::NSLOT;
      bool ok = true;
      if (lane == 0) {
        if (i >= C::NSLOT)
          ok = mbar_wait_bounded_at(&empty[slot], ((i / C::NSLOT) - 1) & 1, abort_flag, deadline, a.status, 51, i,
                                    slot, n_sub);
        if (ok && *abort_flag) ok = false;
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (a.drop_first_copy && i == 0 && split == 0 && g == 0 && b == 0) continue;
      const bool isv = per_tile == 2 && (i & 1);
      const int p0 = sp.position((tile0 + i / per_tile) * C::KT);
      const int nk = max(0, min(C::KT, len_c - p0));
      if (nk == 0) {  // only the new token's row
        if (lane == 0) mbar_arrive(&full[slot]);
        continue;
      }
      const int pi = p0 / a.page_size;
      if (page0 < 0 || pi < page0 || pi >= page0 + 32) {
        page0 = pi;
        ent = pi + lane < a.pages_per_seq ? a.page_table[(int64_t)b * a.pages_per_seq + pi + lane] : 0;
      }
      int page = __shfl_sync(0xffffffffu, ent, pi - page0);
      if (page < 0 || page >= a.n_pages) {  // a page outside the pool: report it and read page 0 (finite, wrong)
        if (lane == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        page = 0;
      }
      const int64_t off = (((int64_t)page * a.Hkv + g) * a.page_size + (p0 - pi * a.page_size)) * D;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[slot], (uint32_t)(nk * D * 2));
        issued[slot] += 1;
      }
      __syncwarp();
      const int left = nk - lane * RPC;
      if (lane < C::NGR && left > 0)
        bulk_g2s(ring + slot * C::SLOT_B + lane * ring_group_bytes(D, RPC),
                 (isv ? a.v_pool : a.k_pool) + off + (int64_t)lane * RPC * D, (left >= RPC ? RPC : left) * D * 2,
                 &full[slot]);
    }
  } else {
    // ---------------- consumers ----------------
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    const int kg = warp % C::KG, dq = warp / C::KG;
    uint32_t qa[C::KS][4];     // A fragments: rows 0..7 q, rows 8..15 what its bf16 rounding lost
    if (n_sub > 0) {
      // this lane's pairs of head gq: elements d0 + 16 ks + 2 tg (+ 8)
      const int d0 = dq * (D / C::DQ) + 2 * tg;
      uint32_t raw[C::KS][2];
      const bf16* qrow = a.q + (head0 + (gq < G ? gq : 0)) * D + d0;
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        raw[ks][0] = *reinterpret_cast<const uint32_t*>(qrow + ks * 16);
        raw[ks][1] = *reinterpret_cast<const uint32_t*>(qrow + ks * 16 + 8);
      }
      for (int i = tid; i < a.n_rot; i += NCT) {
        const double x = (double)(len - 1) * a.freq[i];
        float s, c;
        sincospif((float)(x - 2.0 * rint(0.5 * x)), &s, &c);
        trig[i] = make_float2(c, s);
      }
      named_bar_sync(1, NCT);
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 v = unpack_bf16x2(raw[ks][e]);
          const int pair = (d0 + ks * 16 + e * 8) / 2;
          if (pair < a.n_rot) {
            const float2 t = trig[pair];
            v = make_float2(v.x * t.x - v.y * t.y, v.x * t.y + v.y * t.x);
          }
          if (gq >= G) v = make_float2(0.f, 0.f);
          const uint32_t hi = pack_bf16x2(v.x, v.y);
          const float2 h = unpack_bf16x2(hi);
          qa[ks][2 * e] = hi;
          qa[ks][2 * e + 1] = pack_bf16x2(v.x - h.x, v.y - h.y);
        }
      if (own_new && tid < per_tile * CH) {
        const int64_t crow = cache_row(a.page_table, a.pages_per_seq, a.page_size, a.n_pages, a.Hkv, b, g, len - 1);
        if (crow < 0 && tid == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        const int c = tid % CH;
        const bool isv = tid >= CH;
        const uint4 x =
            *reinterpret_cast<const uint4*>((isv ? a.v_new : a.k_new) + ((int64_t)b * a.Hkv + g) * D + c * 8);
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if (!isv) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c * 4 + j < a.n_rot) {
              const float2 v = unpack_bf16x2(w[j]), t = trig[c * 4 + j];
              w[j] = pack_bf16x2(v.x * t.x - v.y * t.y, v.x * t.y + v.y * t.x);
            }
        }
        const uint4 y = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(newrow + (isv ? D : 0) + c * 8) = y;
        if (crow >= 0) *reinterpret_cast<uint4*>((isv ? a.v_pool : a.k_pool) + crow * D + c * 8) = y;
      }
    }
    const uint32_t frag_off = ring_row_off<D, RPC>(ring_key<RPC>((lane >> 4) * 8 + (lane & 7))) + ((lane >> 3) & 1) * 16;
    constexpr int GROUP16_B = (16 / RPC) * ring_group_bytes(D, RPC);  // 16 rows of a tile

    // waits that fail raise the abort flag: later ones return at once, and the
    // warps go on meeting at the barriers below
    for (int t = 0; t < n_sub; ++t) {
      const int p0 = sp.position((tile0 + t) * C::KT);
      const bool edge = !(p0 + C::KT <= len_c && (p0 >= sp.lo || p0 + C::KT <= a.sinks));
      const bool with_new = own_new && t == n_sub - 1;
      int item = t * per_tile, slot = item % C::NSLOT;
      bool ok = mbar_wait_bounded_at(&full[slot], (item / C::NSLOT) & 1, abort_flag, deadline, a.status, 52, item, slot,
                                     warp);
      if (tid == 0 && ok) consumed[slot] += 1;
      __syncwarp();
      unsigned char* rows = ring + slot * C::SLOT_B;
      if (with_new) {
        if (t == 0) named_bar_sync(1, NCT);  // newrow is written
        if (tid < CH)
          *reinterpret_cast<uint4*>(rows + ring_row_off<D, RPC>(len_c - p0) + tid * 16) =
              *reinterpret_cast<const uint4*>(newrow + tid * 8);
        fence_proxy_async_smem();  // before the slot's next copy
        named_bar_sync(1, NCT);
      }
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t k_addr = smem_u32(rows) + kg * GROUP16_B + frag_off + dq * (D / C::DQ) * 2;
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(k_addr + ks * 32, b0, b1, b2, b3);
        mma_bf16(s0, qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
        mma_bf16(s1, qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
      }
      part[((t & 1) * NCW + warp) * 32 + lane] =
          make_float4(s0[0] + s0[2], s0[1] + s0[3], s1[0] + s1[2], s1[1] + s1[3]);
      if (per_tile == 2) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
      }
      named_bar_sync(1, NCT);  // partials of tile t; those of t - 1 have been read
      float sv[C::KG][4];
      float tmax = -INFINITY;
#pragma unroll
      for (int k = 0; k < C::KG; ++k) {
        float4 x = part[((t & 1) * NCW + k) * 32 + lane];
#pragma unroll
        for (int d = 1; d < C::DQ; ++d) {
          const float4 y = part[((t & 1) * NCW + d * C::KG + k) * 32 + lane];
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        sv[k][0] = x.x * a.scale_log2;
        sv[k][1] = x.y * a.scale_log2;
        sv[k][2] = x.z * a.scale_log2;
        sv[k][3] = x.w * a.scale_log2;
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = p0 + k * 16 + ring_key<RPC>(2 * tg + (i & 1) + (i >> 1) * 8);
            if (!sp.sees(pos, (int)len, a.sinks)) sv[k][i] = -INFINITY;
          }
        }
        tmax = fmaxf(tmax, fmaxf(fmaxf(sv[k][0], sv[k][1]), fmaxf(sv[k][2], sv[k][3])));
      }
      tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
      tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
      const float m_new = fmaxf(m_h, tmax);
      const float base = (m_new == -INFINITY) ? 0.f : m_new;
      const float alpha = exp2f(m_h - base);
      l_t *= alpha;
      m_h = m_new;
      // the weights are rounded to bf16 for the tensor cores; their sum is not
      uint32_t pb[C::KG][2];
#pragma unroll
      for (int k = 0; k < C::KG; ++k) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = exp2f(sv[k][i] - base);
        l_t += (p[0] + p[1]) + (p[2] + p[3]);
        pb[k][0] = pack_bf16x2(p[0], p[1]);
        pb[k][1] = pack_bf16x2(p[2], p[3]);
      }
      const float al0 = __shfl_sync(0xffffffffu, alpha, (2 * tg) * 4);
      const float al1 = __shfl_sync(0xffffffffu, alpha, (2 * tg + 1) * 4);
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        o[mt][0] *= al0;
        o[mt][1] *= al1;
        o[mt][2] *= al0;
        o[mt][3] *= al1;
      }
      if (per_tile == 2) {
        ++item;
        slot = item % C::NSLOT;
        ok = mbar_wait_bounded_at(&full[slot], (item / C::NSLOT) & 1, abort_flag, deadline, a.status, 54, item, slot,
                                  warp);
        if (tid == 0 && ok) consumed[slot] += 1;
        __syncwarp();
        rows = ring + slot * C::SLOT_B;
      }
      if (edge) {
        // (K = V: every warp has read the rows as keys)
        for (int i = tid; i < C::KT * CH; i += NCT) {
          const int r = i / CH, c = i % CH;
          const bool is_new = has_new && p0 + r == len_c;
          if (is_new ? a.keqv : sp.sees(p0 + r, len_c, a.sinks)) continue;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (is_new) v = *reinterpret_cast<const uint4*>(newrow + D + c * 8);
          *reinterpret_cast<uint4*>(rows + ring_row_off<D, RPC>(r) + c * 16) = v;
        }
        fence_proxy_async_smem();
        named_bar_sync(1, NCT);
      }
      const uint32_t v_addr = smem_u32(rows) + frag_off + warp * (D / NCW) * 2;
#pragma unroll
      for (int k = 0; k < C::KG; ++k)
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          uint32_t va0, va1, va2, va3;
          ldsm_x4_t(v_addr + k * GROUP16_B + mt * 32, va0, va1, va2, va3);
          mma_bf16(o[mt], va0, va1, va2, va3, pb[k][0], pb[k][1]);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
  }
  float l_q = l_t + __shfl_xor_sync(0xffffffffu, l_t, 1);
  l_q += __shfl_xor_sync(0xffffffffu, l_q, 2);
  __syncwarp();
  pair::cluster_sync();  // every CTA is done with its ring
  // Each CTA owns D / n_splits output columns; the others push their share of
  // those into its ring: [split][head pair][column] float2, and (m, l).
  const int cols = D / n_splits;
  if (warp < NCW) {
    const bool gave_up = *abort_flag;
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      const int d = warp * (D / NCW) + mt * 16;
      const uint32_t to = pair::map_to(smem_u32(ring), d / cols) + ((split * 4 + tg) * cols + d % cols + gq) * 8;
      st_cluster(to, o[mt][0], o[mt][1]);
      st_cluster(to + 64, o[mt][2], o[mt][3]);
    }
    if (warp < n_splits && tg == 0)
      st_cluster(pair::map_to(smem_u32(ml + split * 8 + gq), warp), m_h, gave_up ? -1.f : l_q);
  } else if (*abort_flag && lane == 0) {
    // drain: wait (bounded) for copies that were issued but never consumed
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    volatile int never = 0;
    for (int s = 0; s < C::NSLOT; ++s)
      if (issued[s] > consumed[s])
        mbar_wait_bounded_at(&full[s], (issued[s] - 1) & 1, &never, dl, a.status, 53, issued[s], s, consumed[s]);
  }
  __syncwarp();
  pair::cluster_sync();  // every share has arrived; nothing remote follows
  if (tid < 8) {
    float M = -INFINITY, L = 0.f;
    bool ok = true;
    for (int s = 0; s < n_splits; ++s) M = fmaxf(M, ml[s * 8 + tid].x);
    for (int s = 0; s < n_splits; ++s) {
      const float2 x = ml[s * 8 + tid];
      const float w = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
      ok = ok && !(x.y < 0.f);
      L += w * x.y;
      wgt[s * 8 + tid] = w;
    }
    wgt[n_splits * 8 + tid] = ok ? 1.f / L : -1.f;  // -1: no output (L is positive, or NaN)
  }
  __syncthreads();
  for (int i = tid; i < 4 * cols; i += NCT + 32) {
    const int hp = i / cols, d = i % cols;
    if (2 * hp >= G) continue;
    float x = 0.f, y = 0.f;
    for (int s = 0; s < n_splits; ++s) {
      const float2 v = *reinterpret_cast<const float2*>(ring + ((s * 4 + hp) * cols + d) * 8);
      x += wgt[s * 8 + 2 * hp] * v.x;
      y += wgt[s * 8 + 2 * hp + 1] * v.y;
    }
    const float ix = wgt[n_splits * 8 + 2 * hp], iy = wgt[n_splits * 8 + 2 * hp + 1];
    bf16* dst = a.out + (head0 + 2 * hp) * D + split * cols + d;
    if (ix != -1.f) dst[0] = __float2bfloat16(x * ix);
    if (iy != -1.f && 2 * hp + 1 < G) dst[D] = __float2bfloat16(y * iy);
  }
}

template <int D>
cudaError_t launch_as(const SinkDecodeArgs& a, int B, int n_splits, cudaStream_t st) {
  using C = SinkCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(k_decode_sinks<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_splits, a.Hkv, B);
  cfg.blockDim = dim3(NCT + 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_decode_sinks<D>, a);
}

}  // namespace

// Splits per (sequence, KV head): the power of two up to MAX_CLUSTER that
// minimises (waves of CTAs) x (keys per CTA + a fixed cost per CTA, in keys).
int decode_sinks_splits(int B, int Hkv, int D, int window, int sinks, int max_len) {
  const SinkSpan sp = sink_span(max_len, window, sinks, 16384 / D);
  const int64_t pairs = (int64_t)B * Hkv, wave = (int64_t)multiprocessors() * 2;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int n = 1; n <= MAX_CLUSTER; n *= 2) {
    const int64_t keys = (sp.n + n - 1) / n;
    const int64_t cost = ((pairs * n + wave - 1) / wave) * (keys + 64);
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

cudaError_t launch_decode_sinks(SinkDecodeArgs& a, int B, int D, double log2_theta, cudaStream_t st) {
  for (int i = 0; i < a.n_rot; ++i) a.freq[i] = std::exp2(-(2.0 * i / D) * log2_theta) * kInvPi;
  const int n = decode_sinks_splits(B, a.Hkv, D, a.window, a.sinks, a.max_len);
  return D == 256 ? launch_as<256>(a, B, n, st) : launch_as<512>(a, B, n, st);
}

}  // namespace hlg
