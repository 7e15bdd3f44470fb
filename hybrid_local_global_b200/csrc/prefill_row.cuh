// prefill_row.cuh -- what the prefill kernels (prefill_tc.cu, prefill_pair.cu,
// prefill_stream.cu) share: a warp's bounded wait, and the softmax arithmetic of
// one row of a 128-key logits tile.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace hlg {

namespace {

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t deadline, int* status, int where, int a = 0,
                                         int b = 0, int c = 0) {
  bool ok = mbar_wait_bounded_at(bar, parity, abort_flag, deadline, status, where, a, b, c);
  return __all_sync(0xffffffffu, ok);
}

// P = 2^(x - mb) over the 128 logits of one row, packed to bf16 pairs, with
// eight independent partial sums (and, if TRACK, partial maxima), so that the
// reductions do not run down one dependency chain. The sums take the weights as
// they are before that rounding: what it moves in P V does not move their mean.
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

}  // namespace

}  // namespace hlg
