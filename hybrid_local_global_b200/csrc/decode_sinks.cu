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
// Visible keys are walked in a virtual order of whole 32-key blocks: those of
// the sinks, then those from the one that holds the window's first key on (one
// run when the two meet); a block never straddles a page. Four blocks make a
// tile of 128 keys. The product is taken transposed, as in the multi-token
// kernel, so that the keys fill the MMA's 128 rows and the few q heads are its
// columns:
//   S^T = K Q^T    (M = 128 keys, N = 16, K = head_dim)
//   O^T += V^T P^T (M = 128 value dims per MMA, N = 16, K = 32 keys per block)
// A group has at most 8 heads and N is at least 16: columns 0..7 take the bf16
// values of Q~ (and of the weights P), columns 8..15 what that rounding lost,
// and the two halves are added, so neither rounding shows in the result.
//
// CTA = 192 threads: warp 0 loads (TMA, boxes of 32 keys x 64 dims into 32 KB
// stages of 128 keys x 128 dims), warp 1 issues the MMAs and owns TMEM, warps
// 2..5 rotate q and the new key, run the softmax (thread = key = TMEM lane)
// and merge. The new token's row is not read back from the cache: warp 1 puts
// it into its tile. Rows that the query does not see are masked in S and
// cleared in V (their weight is 0, but 0 * NaN is not).
//
// HBM-bound: every visible K/V byte is read once per KV head (under K = V
// the second read of a row hits L2).
//
// Every wait is bounded; after a timeout the cluster still meets at its
// barriers and writes no output (GEMMA_ERR_DEVICE_TIMEOUT).
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace hlg {

namespace {

constexpr int BLK = 32;             // keys per block of the walk
constexpr int BN = 128;             // keys per tile
constexpr int NQ = 16;              // MMA columns: 8 heads, then 8 remainders
constexpr int CH_B = BN * 128;      // [128 keys][64 dims], swizzled
constexpr int STAGE_B = 2 * CH_B;   // 128 dims of a K or V tile
constexpr int BOX_B = BLK * 128;    // one TMA box: 32 keys x 64 dims
constexpr int P_B = 2 * NQ * 128;   // P^T: two chunks of 64 keys
constexpr int MAX_CLUSTER = 8;      // CTAs per (sequence, KV head)
constexpr float RESCALE_LOG2 = 8.0f;
constexpr double kInvPi = 0.31830988618379067153776752674503;
constexpr uint32_t IDESC_ST = tc::idesc_bf16_f32(128, NQ, 0, 0);  // K (K-major) x Q (K-major)
constexpr uint32_t IDESC_OT = tc::idesc_bf16_f32(128, NQ, 1, 0);  // V^T (MN-major) x P^T (K-major)

template <int NS>
struct Ctl {
  uint64_t full[NS], empty[NS];
  uint64_t q_ready;               // 128 softmax threads: Q and the new rows are staged
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued[NS], consumed[NS];
  float m[8], f[8], l[8];         // running maxima, rescale factors, sums (this CTA)
  float red[4][8];
  float2 ml[MAX_CLUSTER][8];      // the cluster's (m, l); l < 0: that CTA gave up
};

// CTAS per SM. Two overlap one CTA's prologue and merge with the other's
// stream; one has the whole shared memory for its ring.
template <int D, int CTAS>
struct Cfg {
  static constexpr int MT = D / 128;                 // K stages per tile = O^T blocks = V stages per tile
  static constexpr int Q_B = (D / 64) * NQ * 128;
  static constexpr int NS = CTAS == 2 ? 2 : 6;
  static constexpr int Q_OFF = NS * STAGE_B;
  static constexpr int P_OFF = Q_OFF + Q_B;          // two buffers; the angles before the first tile
  static constexpr int NEW_OFF = P_OFF + 2 * P_B;    // the new token's K row, V row
  static constexpr int CTL_OFF = NEW_OFF + 2 * D * 2;
  static constexpr int SMEM = 1024 + CTL_OFF + (int)sizeof(Ctl<NS>);
  static constexpr uint32_t COL_S = MT * NQ;         // after O^T
  static constexpr uint32_t TMEM_COLS = MT * NQ + 2 * NQ <= 64 ? 64 : 128;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "resident CTAs");
  static_assert(8 * D * 4 <= NS * STAGE_B, "the merge buffer overlays the drained ring");
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

template <int D, int CTAS>
__global__ void __launch_bounds__(192, CTAS)
    k_decode_sinks(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ SinkDecodeArgs a) {
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
      for (int i = tid; i < G * CH; i += 192)
        *reinterpret_cast<uint4*>(a.out + head0 * D + i * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool has_new = a.k_new != nullptr;
  const int len_c = (int)len - (has_new ? 1 : 0);  // rows that are read from the cache
  const SinkSpan sp = sink_span(len, a.window, a.sinks, BLK);
  const int blocks = (sp.n + BLK - 1) / BLK;
  const int per = (blocks + n_splits - 1) / n_splits;
  const int blk0 = min(split * per, blocks);
  const int n_blk = min(per, blocks - blk0);       // this CTA's blocks
  const int n_tiles = (n_blk + 3) / 4;
  const bool own_new = has_new && n_blk > 0 && blk0 + n_blk == blocks;  // its last block holds the new token

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
      ctl->issued[s] = ctl->consumed[s] = 0;
    }
    mbar_init(&ctl->q_ready, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_ready[i], 128);
      mbar_init(&ctl->o_done[i], 1);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (tid < 8) ctl->m[tid] = -INFINITY;
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncwarp();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;
  float l[8];  // softmax threads: this key lane's sums
#pragma unroll
  for (int n = 0; n < 8; ++n) l[n] = 0.f;
  bool good = true;  // softmax threads

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int page0 = -1, ent = 0;  // this lane's table entry: of page page0 + lane
    int item = 0;
    bool ok = true;
    for (int j = 0; j <= n_tiles && ok; ++j) {
      for (int kind = 0; kind < 2 && ok; ++kind) {  // 0: K_j, 1: V_{j-1}
        if ((kind == 0 && j == n_tiles) || (kind == 1 && j == 0)) continue;
        const int i0 = (j - kind) * 4, nb = min(4, n_blk - i0);
        // lane's box of every stage: block lane / 2, 64-dim half lane % 2
        int row = 0, page = 0;
        for (int q = 0; q < nb; ++q) {
          const int p0 = sp.position((blk0 + i0 + q) * BLK);
          const int pi = p0 / a.page_size;
          if (page0 < 0 || pi < page0 || pi >= page0 + 32) {
            page0 = pi;
            ent = pi + lane < a.pages_per_seq ? a.page_table[(int64_t)b * a.pages_per_seq + pi + lane] : 0;
          }
          const int e = __shfl_sync(0xffffffffu, ent, pi - page0);
          if (lane >> 1 == q) {
            row = p0 - pi * a.page_size;
            page = e;
          }
        }
        if (page < 0 || page >= a.n_pages) {  // a page outside the pool: report it and read page 0 (finite, wrong)
          set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
          page = 0;
        }
        const CUtensorMap* map = kind == 0 ? &tm_k : &tm_v;
        for (int h = 0; h < MT; ++h, ++item) {
          const int s = item % NS;
          if (lane == 0) {
            if (item >= NS)
              ok = mbar_wait_bounded_at(&ctl->empty[s], ((item / NS) - 1) & 1, abort_flag, deadline, a.status, 51,
                                        item, s, j);
            if (ok && *abort_flag) ok = false;
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (a.drop_first_copy && item == 0 && split == 0 && g == 0 && b == 0) continue;
          if (lane == 0) {
            mbar_arrive_expect_tx(&ctl->full[s], (uint32_t)(nb * 2 * BOX_B));
            ctl->issued[s] += 1;
          }
          __syncwarp();
          if (lane < 2 * nb)
            tc::tma_load_4d(base + s * STAGE_B + (lane & 1) * CH_B + (lane >> 1) * BOX_B, map,
                            h * 128 + (lane & 1) * 64, row, g, page, smem_u32(&ctl->full[s]));
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = n_tiles == 0 || wait_all(&ctl->q_ready, 0, abort_flag, deadline, a.status, 50, 0, 0, 0);
    const int new_row = own_new ? ((n_blk - 1) & 3) * BLK + len_c - sp.position((blk0 + n_blk - 1) * BLK) : -1;
    int item = 0;
    for (int j = 0; j <= n_tiles && ok; ++j) {
      if (j < n_tiles) {
        const uint32_t d_s = tmem + C::COL_S + (uint32_t)(j & 1) * NQ;
        for (int h = 0; h < MT; ++h, ++item) {
          const int s = item % NS;
          if (!wait_all(&ctl->full[s], (item / NS) & 1, abort_flag, deadline, a.status, 52, item, s, j)) {
            ok = false;
            break;
          }
          const uint32_t st = base + s * STAGE_B;
          if (own_new && j == n_tiles - 1) {  // the new key's row
            if (lane < 16) {
              const int cc = lane >> 3, u = lane & 7;
              *reinterpret_cast<uint4*>(sm + s * STAGE_B + cc * CH_B + new_row * 128 + ((u ^ (new_row & 7)) << 4)) =
                  *reinterpret_cast<const uint4*>(newrow + h * 128 + lane * 8);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            ctl->consumed[s] += 1;
            tc::fence_after_sync();
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_ss(d_s, tc::smem_desc_sw128(st + cc * CH_B + kk * 32, 16, 1024),
                           tc::smem_desc_sw128(base + C::Q_OFF + (h * 2 + cc) * (NQ * 128) + kk * 32, 16, 1024),
                           IDESC_ST, (h | cc | kk) != 0);
            tc::commit(smem_u32(&ctl->empty[s]));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) tc::commit(smem_u32(&ctl->s_full[j & 1]));
      }
      if (j >= 1) {
        const int i0 = (j - 1) * 4, nb = min(4, n_blk - i0);
        uint32_t edge = 0;  // blocks with rows to clear or to fill in
        for (int q = 0; q < nb; ++q) {
          const int p0 = sp.position((blk0 + i0 + q) * BLK);
          if (!(p0 + BLK <= len_c && (p0 >= sp.lo || p0 + BLK <= a.sinks))) edge |= 1u << q;
        }
        if (!wait_all(&ctl->p_ready[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, deadline, a.status, 53, j, 0, 0)) {
          ok = false;
          break;
        }
        const uint32_t pb = base + C::P_OFF + (uint32_t)((j - 1) & 1) * P_B;
        for (int m = 0; m < MT; ++m, ++item) {
          const int s = item % NS;
          if (!wait_all(&ctl->full[s], (item / NS) & 1, abort_flag, deadline, a.status, 54, item, s, j)) {
            ok = false;
            break;
          }
          const uint32_t st = base + s * STAGE_B;
          if (edge) {
            for (int q = 0; q < nb; ++q) {
              if (!(edge >> q & 1)) continue;
              const int p0 = sp.position((blk0 + i0 + q) * BLK);
              for (int i = lane; i < BLK * 16; i += 32) {
                const int r = i / 16, cc = (i / 8) & 1, u = i & 7;
                const bool is_new = has_new && p0 + r == len_c;
                if (!is_new && sp.sees(p0 + r, len_c, a.sinks)) continue;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (is_new)
                  v = *reinterpret_cast<const uint4*>(newrow + (a.keqv ? 0 : D) + m * 128 + cc * 64 + u * 8);
                *reinterpret_cast<uint4*>(sm + s * STAGE_B + cc * CH_B + (q * BLK + r) * 128 + ((u ^ (r & 7)) << 4)) = v;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            ctl->consumed[s] += 1;
            tc::fence_after_sync();
            for (int kk = 0; kk < 2 * nb; ++kk)
              // V^T: 128 dims (two 64-dim boxes CH_B apart) x 16 keys; P^T: 16 columns x 16 keys
              tc::mma_ss(tmem + m * NQ, tc::smem_desc_sw128(st + kk * 2048, CH_B, 1024),
                         tc::smem_desc_sw128(pb + (kk >> 2) * (NQ * 128) + (kk & 3) * 32, 16, 1024), IDESC_OT,
                         (j - 1 > 0 || kk) ? 1u : 0u);
            tc::commit(smem_u32(&ctl->empty[s]));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) tc::commit(smem_u32(&ctl->o_done[(j - 1) & 1]));
      }
    }
    // no MMA may be in flight when TMEM or shared memory is released
    if (lane == 0) {
      tc::commit(smem_u32(&ctl->drain));
      volatile int never = 0;
      mbar_wait_bounded_at(&ctl->drain, 0, &never, globaltimer_ns() + 200000000ull, a.status, 55, 0, 0, 0);
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
#pragma unroll
      for (int k = 0; k < 8 * CH / 128; ++k) {
        const int i = t128 + k * 128, r = i / CH, c = i % CH;
        float2 y[4];
        turn4(x[k], c, a.n_rot, trig, y);
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
        const int c = t128 % CH;
        const bool isv = t128 >= CH;
        uint4 v = *reinterpret_cast<const uint4*>((isv ? a.v_new : a.k_new) + ((int64_t)b * a.Hkv + g) * D + c * 8);
        if (!isv) {
          float2 y[4];
          turn4(v, c, a.n_rot, trig, y);
          v = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                         pack_bf16x2(y[3].x, y[3].y));
        }
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
      if (!bad && !wait_all(&ctl->s_full[j & 1], (j >> 1) & 1, abort_flag, deadline, a.status, 56, j, 0, 0)) bad = true;
      tc::fence_after_sync();
      float v[8];
      {
        uint32_t r[16];
        tmem_ld16(tm + C::COL_S + (uint32_t)(j & 1) * NQ, r);
        tc::tmem_wait_ld();
        const int blk = j * 4 + (kl >> 5);
        const bool seen =
            blk < n_blk && sp.sees(sp.position((blk0 + blk) * BLK) + (kl & 31), (int)len, a.sinks);
#pragma unroll
        for (int n = 0; n < 8; ++n)
          v[n] = seen ? (__uint_as_float(r[n]) + __uint_as_float(r[n + 8])) * a.scale_log2 : -INFINITY;
      }
      bool need = bad;
#pragma unroll
      for (int n = 0; n < 8; ++n) need |= v[n] > ctl->m[n] + RESCALE_LOG2;
      if (any128(need)) {
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
    // loads still in flight must land before shared memory is reused
    volatile int never = 0;
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    for (int s = 0; s < NS; ++s)
      if (ctl->issued[s] > ctl->consumed[s])
        mbar_wait_bounded_at(&ctl->full[s], (ctl->issued[s] - 1) & 1, &never, dl, a.status, 60, ctl->issued[s], s,
                             ctl->consumed[s]);
  }
  __syncwarp();
  pair::cluster_sync();  // every CTA is done with its ring
  // Each CTA owns D / n_splits output columns; the others push their share of
  // those into its ring, [split][column][head], and their (m, l).
  const int cols = D / n_splits;
  if (warp >= 2) {
    const int kl = (warp & 3) * 32 + lane;
    if (n_tiles > 0) {
      tc::fence_after_sync();
      const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
      for (int m = 0; m < MT; ++m) {
        uint32_t o[16];
        tmem_ld16(tm + m * NQ, o);
        tc::tmem_wait_ld();
        float x[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] = __uint_as_float(o[n]) + __uint_as_float(o[n + 8]);
        const int d = m * 128 + kl;
        const uint32_t to = pair::map_to(base, d / cols) + (split * cols + d % cols) * 32;
        st_cluster4(to, x[0], x[1], x[2], x[3]);
        st_cluster4(to + 16, x[4], x[5], x[6], x[7]);
      }
    }
    if (kl < n_splits * 8)
      st_cluster2(pair::map_to(smem_u32(&ctl->ml[split][kl & 7]), kl >> 3), ctl->m[kl & 7],
                  good ? ctl->l[kl & 7] : -1.f);
  }
  tc::fence_before_sync();
  __syncwarp();
  pair::cluster_sync();  // every share has arrived; nothing remote follows
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  for (int i = tid; i < 8 * cols; i += 192) {
    const int n = i / cols, d = i % cols;
    if (n >= G) break;
    float M = -INFINITY;
    for (int s = 0; s < n_splits; ++s) M = fmaxf(M, ctl->ml[s][n].x);
    float L = 0.f, x = 0.f;
    bool ok = true;
    for (int s = 0; s < n_splits; ++s) {
      const float2 ml = ctl->ml[s][n];
      ok = ok && !(ml.y < 0.f);
      if (ml.x == -INFINITY) continue;  // no keys there, and no O
      const float w = tc::ex2(ml.x - M);
      L += w * ml.y;
      x += w * *reinterpret_cast<const float*>(sm + ((s * cols + d) * 8 + n) * 4);
    }
    if (ok) a.out[(head0 + n) * D + split * cols + d] = __float2bfloat16_rn(x / L);
  }
}

template <int D, int CTAS>
cudaError_t launch_as(const CUtensorMap& mk, const CUtensorMap& mv, const SinkDecodeArgs& a, int B, int n_splits,
                      cudaStream_t st) {
  using C = Cfg<D, CTAS>;
  cudaError_t e = cudaFuncSetAttribute(k_decode_sinks<D, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_splits, a.Hkv, B);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_decode_sinks<D, CTAS>, mk, mv, a);
}

// Splits per (sequence, KV head): the power of two up to MAX_CLUSTER that
// minimises (waves of CTAs) x (keys per CTA + a fixed cost per CTA, in keys).
int plan_splits(int B, int Hkv, int window, int sinks, int max_len) {
  const SinkSpan sp = sink_span(max_len, window, sinks, BLK);
  const int64_t pairs = (int64_t)B * Hkv, wave = (int64_t)multiprocessors() * 2;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int n = 1; n <= MAX_CLUSTER; n *= 2) {
    const int64_t keys = (sp.n + n - 1) / n;
    const int64_t cost = ((pairs * n + wave - 1) / wave) * (keys + 128);
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_decode_sinks(SinkDecodeArgs& a, int B, int D, double log2_theta, cudaStream_t st) {
  for (int i = 0; i < a.n_rot; ++i) a.freq[i] = std::exp2(-(2.0 * i / D) * log2_theta) * kInvPi;
  const uint64_t ps = (uint64_t)a.page_size, H = (uint64_t)a.Hkv, d = (uint64_t)D;
  const uint64_t dims[4] = {d, ps, H, (uint64_t)a.n_pages}, str[3] = {d * 2, ps * d * 2, H * ps * d * 2};
  const uint32_t box[4] = {64, BLK, 1, 1};
  CUtensorMap mk, mv;
  if (!make_map_bf16_4d(&mk, a.k_pool, dims, str, box) || !make_map_bf16_4d(&mv, a.v_pool, dims, str, box))
    return cudaErrorInvalidValue;
  const int n = plan_splits(B, a.Hkv, a.window, a.sinks, a.max_len);
  const bool deep = (int64_t)B * a.Hkv * n <= multiprocessors();
  if (D == 256) return deep ? launch_as<256, 1>(mk, mv, a, B, n, st) : launch_as<256, 2>(mk, mv, a, B, n, st);
  return deep ? launch_as<512, 1>(mk, mv, a, B, n, st) : launch_as<512, 2>(mk, mv, a, B, n, st);
}

}  // namespace hlg
