// prefill_pair.cuh -- what the CTA-pair prefill kernels share (prefill_pair.cu,
// prefill_stream.cu): tile sizes, control block, arguments.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "prefill_row.cuh"
#include "tc.cuh"

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

// Zero V rows [r0, r1) of a stage (the whole warp): both 64-column boxes, in this CTA (local
// stores) and in the peer (distributed shared memory), then make the writes
// visible to the tensor core's reads.
__device__ __forceinline__ void clear_v_rows_pair(uint32_t stage, int r0, int r1, int lane) {
  const uint32_t peer = pair::map_to(stage, 1);
  const uint32_t self = pair::map_to(stage, 0);
  for (int i = lane; i < (r1 - r0) * 16; i += 32) {
    const uint32_t off = (uint32_t)(((i >> 3) & 1) * CHUNK_V + (r0 + (i >> 4)) * 128 + (i & 7) * 16);
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(self + off), "r"(0) : "memory");
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(peer + off), "r"(0) : "memory");
  }
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

// Arguments of a launch, from the API's (head_pair: PairArgs).
inline PairArgs pair_args(const PrefillAttnArgs& a, int kv_token_major, bool head_pair) {
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
  return t;
}

}  // namespace

}  // namespace hlg
