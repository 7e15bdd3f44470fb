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
// Visible keys are walked in a virtual order of whole 32-key blocks: the
// blocks of the sinks, then the blocks from the one that holds the window's
// first key on (one run when the two meet). Blocks never straddle a page.
// Rows of an edge block that the query does not see are masked in S and
// cleared in V (their weight is 0, but 0 * NaN is not). The new token's row is
// not read back from the cache: the CTA that appends it puts it into the
// block it belongs to.
//
// CTA (128 threads): warp 3 copies row groups into a ring of padded slots,
// warps 0..2 take every third slot: S = Q K^T and O^T += V^T P^T with
// mma.sync m16n8k16, online softmax in fp32 (log2 domain), as decode.cu.
// HBM-bound: every visible K/V byte is read once per KV head.
//
// Every barrier wait is bounded; after a timeout the cluster still meets at
// its barriers and writes no output (GEMMA_ERR_DEVICE_TIMEOUT).
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

constexpr int NCW = 3;          // consumer warps
constexpr int NCT = 32 * NCW;   // consumer threads
constexpr int MAX_CLUSTER = 8;  // CTAs per (sequence, KV head)
constexpr double kInvPi = 0.31830988618379067153776752674503;

template <int D, int RPC_>
struct SinkCfg {
  static constexpr int KB = 16;
  static constexpr int RPC = RPC_;
  static constexpr int GROUPB = ring_group_bytes(D, RPC);
  static constexpr int GPR = KB / RPC;
  static constexpr int SLOT_B = 2 * GPR * GROUPB;
  static constexpr int NSLOT = 3;
  static_assert(NSLOT % NCW == 0, "each ring slot needs a single consumer warp");
  static constexpr int RING_B = NSLOT * SLOT_B;
  static constexpr int ROW = D + 8;               // padded Q row (elements)
  static constexpr int Q_OFF = RING_B;
  static constexpr int NEW_OFF = Q_OFF + 8 * ROW * 2;  // the new token's K row, V row
  static constexpr int TRIG_OFF = NEW_OFF + 2 * D * 2;
  static constexpr int BAR_OFF = TRIG_OFF + (D / 2) * 8;
  static constexpr int MISC_OFF = BAR_OFF + 2 * NSLOT * 8;
  // ints: abort, issued[NSLOT], consumed[NSLOT]; floats: m, l of each warp
  // [NCW][8] twice, of this CTA [8] twice, of the cluster [MAX_CLUSTER][8] twice
  static constexpr int SMEM = MISC_OFF + (8 + 2 * NCW * 8 + 2 * 8 + 2 * MAX_CLUSTER * 8) * 4;
  static constexpr int OSTR = D + 4;              // merge-buffer row (floats)
  static_assert(NCW * 8 * OSTR * 4 <= RING_B, "the merge buffer overlays the drained ring");
  static_assert(1 + 2 * NSLOT <= 8, "misc ints");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int D, int RPC>
__global__ void __launch_bounds__(128, D == 256 ? 4 : 2) k_decode_sinks(const __grid_constant__ SinkDecodeArgs a) {
  using C = SinkCfg<D, RPC>;
  extern __shared__ __align__(128) unsigned char sm[];
  unsigned char* ring = sm;
  bf16* qs = reinterpret_cast<bf16*>(sm + C::Q_OFF);
  bf16* newrow = reinterpret_cast<bf16*>(sm + C::NEW_OFF);
  float2* trig = reinterpret_cast<float2*>(sm + C::TRIG_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
  uint64_t* empty = full + C::NSLOT;
  int* misc = reinterpret_cast<int*>(sm + C::MISC_OFF);
  volatile int* abort_flag = misc;
  int* issued = misc + 1;
  int* consumed = issued + C::NSLOT;
  float* m_w = reinterpret_cast<float*>(misc + 8);  // [NCW][8]
  float* l_w = m_w + NCW * 8;
  float* m_c = l_w + NCW * 8;                       // [8] this CTA; l < 0: it gave up
  float* l_c = m_c + 8;
  float* m_a = l_c + 8;                             // [splits][8] the cluster's
  float* l_a = m_a + MAX_CLUSTER * 8;

  const int split = blockIdx.x, n_splits = gridDim.x, g = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const int64_t len = a.seq_lens[b];
  const int64_t head0 = (int64_t)b * a.Hq + (int64_t)g * G;  // first q row of the group
  if (len < 1 || len > a.max_len) {  // an idle slot (0) or a bad length: zeros; the whole cluster leaves here
    if (len != 0 && threadIdx.x == 0 && split == 0 && g == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
    if (split == 0)
      for (int i = threadIdx.x; i < G * D / 8; i += 128)
        *reinterpret_cast<uint4*>(a.out + head0 * D + i * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool has_new = a.k_new != nullptr;
  const int len_c = (int)len - (has_new ? 1 : 0);  // rows that are read from the cache
  const SinkSpan sp = sink_span(len, a.window, a.sinks);
  const int kps = a.keqv ? 2 * C::KB : C::KB;      // keys per ring slot
  const int blocks = (sp.n + kps - 1) / kps;
  const int per = (blocks + n_splits - 1) / n_splits;
  const int blk0 = min(split * per, blocks);
  const int n_sub = min(per, blocks - blk0);
  const bool own_new = has_new && n_sub > 0 && blk0 + n_sub == blocks;  // this CTA holds the new token's block

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      issued[s] = 0;
      consumed[s] = 0;
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const uint64_t deadline = globaltimer_ns() + a.wait_ns;

  if (warp == NCW) {
    // ---------------- producer ----------------
    int page0 = -1, ent = 0;  // this lane's table entry: of page page0 + lane
    for (int t = 0; t < n_sub; ++t) {
      const int slot = t % C::NSLOT;
      bool ok = true;
      if (lane == 0) {
        if (t >= C::NSLOT)
          ok = mbar_wait_bounded_at(&empty[slot], ((t / C::NSLOT) - 1) & 1, abort_flag, deadline, a.status, 51, t,
                                    slot, n_sub);
        if (ok && *abort_flag) ok = false;
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (a.drop_first_copy && t == 0 && split == 0 && g == 0 && b == 0) continue;
      const int p0 = sp.position((blk0 + t) * kps);
      const int nk = max(0, min(kps, len_c - p0));
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
        mbar_arrive_expect_tx(&full[slot], (uint32_t)((a.keqv ? 1 : 2) * nk * D * 2));
        issued[slot] += 1;
      }
      __syncwarp();
      if (lane < 2 * C::GPR) {
        const bool isv = !a.keqv && lane >= C::GPR;
        const int grp = a.keqv ? lane : lane % C::GPR;
        const int left = nk - grp * C::RPC;
        if (left > 0)
          bulk_g2s(ring + slot * C::SLOT_B + (isv ? C::GPR * C::GROUPB : 0) + grp * C::GROUPB,
                   (isv ? a.v_pool : a.k_pool) + off + (int64_t)grp * C::RPC * D,
                   (left >= C::RPC ? C::RPC : left) * D * 2, &full[slot]);
      }
    }
  } else {
    // ---------------- consumers ----------------
    const int tid = threadIdx.x;
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    if (n_sub > 0) {
      for (int i = tid; i < a.n_rot; i += NCT) {
        const double x = (double)(len - 1) * a.freq[i];
        float s, c;
        sincospif((float)(x - 2.0 * rint(0.5 * x)), &s, &c);
        trig[i] = make_float2(c, s);
      }
      named_bar_sync(1, NCT);
      const auto turn = [&](uint4 x, int c) {
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c * 4 + j < a.n_rot) {
            const float2 v = unpack_bf16x2(w[j]), t = trig[c * 4 + j];
            w[j] = pack_bf16x2(v.x * t.x - v.y * t.y, v.x * t.y + v.y * t.x);
          }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      for (int i = tid; i < 8 * CH; i += NCT) {
        const int r = i / CH, c = i % CH;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < G) v = turn(*reinterpret_cast<const uint4*>(a.q + (head0 + r) * D + c * 8), c);
        *reinterpret_cast<uint4*>(qs + r * C::ROW + c * 8) = v;
      }
      if (own_new) {
        const int64_t crow = cache_row(a.page_table, a.pages_per_seq, a.page_size, a.n_pages, a.Hkv, b, g, len - 1);
        if (crow < 0 && tid == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
        const int64_t src = ((int64_t)b * a.Hkv + g) * D;
        for (int i = tid; i < (a.keqv ? 1 : 2) * CH; i += NCT) {
          const int c = i % CH;
          const bool isv = i >= CH;
          uint4 v = *reinterpret_cast<const uint4*>((isv ? a.v_new : a.k_new) + src + c * 8);
          if (!isv) v = turn(v, c);
          *reinterpret_cast<uint4*>(newrow + (isv ? D : 0) + c * 8) = v;
          if (crow >= 0) *reinterpret_cast<uint4*>((isv ? a.v_pool : a.k_pool) + crow * D + c * 8) = v;
        }
      }
    }
    named_bar_sync(1, NCT);

    const int gq = lane >> 2, tg = lane & 3;
    float o[D / 16][4];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    float m_h = -INFINITY, l_t = 0.f;
    const uint32_t q_addr = smem_u32(qs) + ((lane & 7) * C::ROW + ((lane >> 3) & 1) * 8) * 2;
    const uint32_t frag_off = ring_row_off<D, RPC>(ring_key<RPC>((lane >> 4) * 8 + (lane & 7))) + ((lane >> 3) & 1) * 16;

    for (int t = warp; t < n_sub; t += NCW) {
      const int slot = t % C::NSLOT;
      const bool ok = mbar_wait_bounded_at(&full[slot], (t / C::NSLOT) & 1, abort_flag, deadline, a.status, 52, t,
                                           slot, warp);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int p0 = sp.position((blk0 + t) * kps);
      const bool edge = !(p0 + kps <= len_c && (p0 >= sp.lo || p0 + kps <= a.sinks));
      unsigned char* rows = ring + slot * C::SLOT_B;
      if (edge) {
        // rows 0..15 of a slot are K and 16..31 V (K = V: 32 K rows)
        for (int i = lane; i < 2 * C::KB * CH; i += 32) {
          const int r = i / CH, c = i % CH;
          const int pos = p0 + (a.keqv ? r : (r & (C::KB - 1)));
          const bool is_new = has_new && pos == len_c;
          if (!is_new && sp.sees(pos, len_c, a.sinks)) continue;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (is_new) v = *reinterpret_cast<const uint4*>(newrow + (!a.keqv && r >= C::KB ? D : 0) + c * 8);
          *reinterpret_cast<uint4*>(rows + ring_row_off<D, RPC>(r) + c * 16) = v;
        }
        fence_proxy_async_smem();  // before the slot's next copy
        __syncwarp();
      }
      for (int half = 0; half < (a.keqv ? 2 : 1); ++half) {
        const int h0 = p0 + half * C::KB;
        if (h0 >= len) break;
        unsigned char* kslot = rows + half * C::GPR * C::GROUPB;
        unsigned char* vslot = a.keqv ? kslot : kslot + C::GPR * C::GROUPB;
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t k_addr = smem_u32(kslot) + frag_off;
#pragma unroll 8
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t qa0, qa2, b0, b1, b2, b3;
          ldsm_x2(q_addr + ks * 32, qa0, qa2);
          ldsm_x4(k_addr + ks * 32, b0, b1, b2, b3);
          mma_bf16(s0, qa0, 0u, qa2, 0u, b0, b1);
          mma_bf16(s1, qa0, 0u, qa2, 0u, b2, b3);
        }
        float sv[4] = {s0[0] * a.scale_log2, s0[1] * a.scale_log2, s1[0] * a.scale_log2, s1[1] * a.scale_log2};
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = h0 + ring_key<RPC>(2 * tg + (i & 1) + (i >> 1) * 8);
            if (!sp.sees(pos, (int)len, a.sinks)) sv[i] = -INFINITY;
          }
        }
        float tmax = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
        tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
        tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
        const float m_new = fmaxf(m_h, tmax);
        const float base = (m_new == -INFINITY) ? 0.f : m_new;
        const float alpha = exp2f(m_h - base);
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = exp2f(sv[i] - base);
        l_t = l_t * alpha + (p[0] + p[1]) + (p[2] + p[3]);
        m_h = m_new;
        const float al0 = __shfl_sync(0xffffffffu, alpha, (2 * tg) * 4);
        const float al1 = __shfl_sync(0xffffffffu, alpha, (2 * tg + 1) * 4);
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[mt][0] *= al0;
            o[mt][1] *= al1;
            o[mt][2] *= al0;
            o[mt][3] *= al1;
          }
        }
        // the weights are rounded to bf16 for the tensor cores; their sum is not
        const uint32_t pb0 = pack_bf16x2(p[0], p[1]);
        const uint32_t pb1 = pack_bf16x2(p[2], p[3]);
        const uint32_t v_addr = smem_u32(vslot) + frag_off;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          uint32_t va0, va1, va2, va3;
          ldsm_x4_t(v_addr + mt * 32, va0, va1, va2, va3);
          mma_bf16(o[mt], va0, va1, va2, va3, pb0, pb1);
        }
      }
      __syncwarp();
      if (lane == 0) {
        consumed[slot] += 1;
        mbar_arrive(&empty[slot]);
      }
    }
    float l_q = l_t + __shfl_xor_sync(0xffffffffu, l_t, 1);
    l_q += __shfl_xor_sync(0xffffffffu, l_q, 2);
    if (tg == 0) {
      m_w[warp * 8 + gq] = m_h;
      l_w[warp * 8 + gq] = l_q;
    }
    __syncwarp();
    named_bar_sync(1, NCT);
    // every consumer warp is done with the ring (on a timeout copies may be in
    // flight: nothing is written over them)
    if (!*abort_flag) {
      float* obuf = reinterpret_cast<float*>(ring);
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int hh = 2 * tg + j;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NCW; ++w) M = fmaxf(M, m_w[w * 8 + hh]);
        const float mw = m_w[warp * 8 + hh];
        f[j] = (mw == -INFINITY) ? 0.f : exp2f(mw - M);
      }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        float* row0 = obuf + (warp * 8 + 2 * tg) * C::OSTR + mt * 16 + gq;
        float* row1 = row0 + C::OSTR;
        row0[0] = o[mt][0] * f[0];
        row1[0] = o[mt][1] * f[1];
        row0[8] = o[mt][2] * f[0];
        row1[8] = o[mt][3] * f[1];
      }
      named_bar_sync(1, NCT);
      // this CTA's O (unnormalised) into the first warp's rows
      for (int i = tid; i < G * D; i += NCT) {
        const int hh = i / D, d = i % D;
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < NCW; ++w) acc += obuf[(w * 8 + hh) * C::OSTR + d];
        obuf[hh * C::OSTR + d] = acc;
      }
      if (tid < 8) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < NCW; ++w) M = fmaxf(M, m_w[w * 8 + tid]);
#pragma unroll
        for (int w = 0; w < NCW; ++w)
          if (m_w[w * 8 + tid] != -INFINITY) L += l_w[w * 8 + tid] * exp2f(m_w[w * 8 + tid] - M);
        m_c[tid] = M;
        l_c[tid] = L;
      }
    } else if (tid < 8) {
      l_c[tid] = -1.f;
    }
  }
  __syncwarp();
  pair::cluster_sync();  // every CTA's m, l and O are in place
  for (int i = threadIdx.x; i < n_splits * 8; i += 128) {
    m_a[i] = ld_cluster_f32(pair::map_to(smem_u32(&m_c[i & 7]), i >> 3));
    l_a[i] = ld_cluster_f32(pair::map_to(smem_u32(&l_c[i & 7]), i >> 3));
  }
  __syncthreads();
  // this CTA's share of the output columns
  const int cols = D / n_splits;
  for (int i = threadIdx.x; i < G * cols; i += 128) {
    const int hh = i / cols, d = split * cols + i % cols;
    float M = -INFINITY;
    bool ok = true;
    for (int s = 0; s < n_splits; ++s) {
      M = fmaxf(M, m_a[s * 8 + hh]);
      ok = ok && !(l_a[s * 8 + hh] < 0.f);
    }
    float L = 0.f, acc = 0.f;
    const uint32_t at = smem_u32(ring) + (hh * C::OSTR + d) * 4;
    for (int s = 0; s < n_splits; ++s) {
      if (m_a[s * 8 + hh] == -INFINITY) continue;  // no keys there, and no O
      const float w = exp2f(m_a[s * 8 + hh] - M);
      L += w * l_a[s * 8 + hh];
      acc += w * ld_cluster_f32(pair::map_to(at, s));
    }
    if (ok) a.out[(head0 + hh) * D + d] = __float2bfloat16(acc / L);
  }
  __syncwarp();
  if (warp == NCW && *abort_flag && lane == 0) {
    // drain: wait (bounded) for copies that were issued but never consumed
    const uint64_t dl = globaltimer_ns() + 200000000ull;
    volatile int never = 0;
    for (int s = 0; s < C::NSLOT; ++s)
      if (issued[s] > consumed[s])
        mbar_wait_bounded_at(&full[s], (issued[s] - 1) & 1, &never, dl, a.status, 53, issued[s], s, consumed[s]);
  }
  __syncwarp();
  pair::cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <int D, int RPC>
cudaError_t launch_as(const SinkDecodeArgs& a, int B, int n_splits, cudaStream_t st) {
  using C = SinkCfg<D, RPC>;
  cudaError_t e =
      cudaFuncSetAttribute(k_decode_sinks<D, RPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_splits, a.Hkv, B);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_decode_sinks<D, RPC>, a);
}

}  // namespace

// Splits per (sequence, KV head): the power of two up to MAX_CLUSTER that
// minimises (waves of CTAs) x (keys per CTA + a fixed cost per CTA, in keys).
int decode_sinks_splits(int B, int Hkv, int D, int window, int sinks, int max_len) {
  const SinkSpan sp = sink_span(max_len, window, sinks);
  const int64_t pairs = (int64_t)B * Hkv, wave = (int64_t)multiprocessors() * (D == 256 ? 4 : 2);
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
  return D == 256 ? launch_as<256, 4>(a, B, n, st) : launch_as<512, 2>(a, B, n, st);
}

}  // namespace hlg
