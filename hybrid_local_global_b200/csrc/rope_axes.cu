// rope_axes.cu -- rotary positions with several axes (time, height, width of
// image and video tokens), and the inverse rotation.
//
// Pair i = (x_2i, x_2i+1) of every head vector of token t turns by the angle
//   pos[axis(i)][t] * freq(i),
// freq(i) = theta^(-2i/D) as the attention calls use, or theta^(-r/n) for the
// r-th of an axis's n pairs (a vision encoder's two-axis form: half of a patch
// embedding turns by x, the other by y; "Gemma 4: End-to-End Architecture
// Walkthrough", 2). A rotation is orthogonal: its gradient and its inverse are
// the rotation by the opposite angle.
//
// Precision: as in rope_kv.cu the angle is formed and reduced in fp64, in
// half-turns (an fp32 product has an ulp of 1/64 rad near position 2.6e5); the
// reduced angle is rounded to fp32 (off by 2^-25 half-turns at most, 9.4e-8 rad, a
// 40000th of a bf16 half step: fp64 sines would cost far more than the HBM traffic
// hides), its sine and cosine and the rotation are fp32, and the result is
// rounded to bf16 once.
//
// Bound by HBM: every vector is read and written once. A thread owns 8 elements
// (4 pairs) of a token's head vectors, so its angles are formed once per token,
// stay in registers and serve all heads, which it loads eight at a time (two
// at a time, and the heads dealt to several CTAs, for a few tokens).
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "kernels.h"

namespace hlg {

namespace {

constexpr int MAX_PAIRS = 256;
constexpr int MAX_AXES = 4;
constexpr int AX_T = 256;

struct AxesArgs {
  double freq[MAX_PAIRS];  // half-turns per position; negated for the inverse
  unsigned char axis[MAX_PAIRS];
  const bf16* q;
  const bf16* k;
  bf16* q_out;
  bf16* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements between tokens
  const int32_t* pos;  // [n_axes][tokens]
  int tokens, Hq, Hkv, D, n_rot;
};

// Thread (c, y): elements 8c .. of token blockIdx.x * R + y; blockIdx.y: one of
// gridDim.y shares of the heads. U: head vectors loaded before the first store
// (8 with three CTAs per SM: 71 us for 8192 tokens of 48 heads of 256, 86 % of the
// copy rate; 4 with four: 72, 12 with two: 81; and for 19881 tokens of 32 heads
// of 64: 30, 34, 37).
template <int U>
__global__ void __launch_bounds__(AX_T, 3) k_rope_axes(const __grid_constant__ AxesArgs a) {
  const int C = a.D / 8, R = AX_T / C;
  const int c = threadIdx.x % C, y = threadIdx.x / C;
  const int64_t t = (int64_t)blockIdx.x * R + y;
  if (y >= R || t >= a.tokens) return;
  const int turning = a.n_rot - c * 4;  // of this thread's four pairs, the first `turning` turn
  float co[4], sn[4];
  bool formed = false;
  const auto stream = [&](const bf16* src, bf16* dst, int heads) {
    if (turning <= 0 && src == dst) return;  // stays as it is
    for (int h0 = 0; h0 < heads; h0 += U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h0 + u < heads) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)(h0 + u) * a.D));
      if (turning <= 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h0 + u < heads) *reinterpret_cast<uint4*>(dst + (int64_t)(h0 + u) * a.D) = v[u];
        continue;
      }
      if (!formed) {  // while the first vectors are on their way
        formed = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = c * 4 + (j < turning ? j : 0);
          const double x = (double)a.pos[(int64_t)a.axis[i] * a.tokens + t] * a.freq[i];
          sincospif((float)(x - 2.0 * rint(0.5 * x)), &sn[j], &co[j]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack_bf16x2(w[j]);
          const uint32_t z = pack_bf16x2(x.x * co[j] - x.y * sn[j], x.x * sn[j] + x.y * co[j]);
          w[j] = j < turning ? z : w[j];
        }
        if (h0 + u < heads) *reinterpret_cast<uint4*>(dst + (int64_t)(h0 + u) * a.D) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  const int64_t share = blockIdx.y, shares = gridDim.y;
  const int q0 = (int)(a.Hq * share / shares), q1 = (int)(a.Hq * (share + 1) / shares);
  const int k0 = (int)(a.Hkv * share / shares), k1 = (int)(a.Hkv * (share + 1) / shares), e = c * 8;
  stream(a.q + t * a.q_stride + q0 * a.D + e, a.q_out + t * a.q_out_stride + q0 * a.D + e, q1 - q0);
  if (k1 > k0) stream(a.k + t * a.k_stride + k0 * a.D + e, a.k_out + t * a.k_out_stride + k0 * a.D + e, k1 - k0);
}

int err(int code, const char* msg) { return record_error(code, msg); }

// Strided vectors [tokens][heads][D]: 16-byte loads need every token to start
// on 16 bytes; a token's heads are dense.
struct Side {
  const void* p;
  long long stride, row;  // elements between tokens, and of a token
};

int check_side(const Side& s, int tokens) {
  if (!s.p) return err(GEMMA_ERR_INVALID_ARG, "null tensor pointer");
  if (reinterpret_cast<uintptr_t>(s.p) & 15u || s.stride % 8)
    return err(GEMMA_ERR_INVALID_ARG, "tensors must be 16-byte aligned with token strides of a multiple of 8 elements");
  if (tokens > 1 && s.stride < s.row)
    return err(GEMMA_ERR_INVALID_ARG, "a token stride is smaller than heads * head_dim");
  if (tokens > 1 && s.stride > (1LL << 60) / tokens) return err(GEMMA_ERR_INVALID_ARG, "token stride out of range");
  return GEMMA_OK;
}

// Whether some token of one tensor shares bytes with some token of the other.
// With one stride: token i of a and token j of b do iff, for t = i - j,
//   d - a.row < t * stride < d + b.row   (d: elements from a to b),
// so head slices of one buffer, interleaved as they are, do not. Tensors of
// different strides are told apart by their extents alone.
bool overlap(const Side& a, const Side& b, int tokens) {
  const long long n = tokens - 1;
  // both 16-byte aligned
  const long long d = (long long)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) / 2;
  if (d >= n * a.stride + a.row || -d >= n * b.stride + b.row) return false;
  if (n == 0 || a.stride != b.stride) return true;
  const auto floor_div = [](long long x, long long y) { return x / y - (x % y < 0); };
  const long long first = floor_div(d - a.row, a.stride) + 1, last = floor_div(d + b.row - 1, a.stride);
  return std::max(first, -n) <= std::min(last, n);
}

// q into q_out and, if any, k into k_out. A thread reads a vector before it
// writes it, so an output may be its input; any other sharing would let one
// token's output go under another's input.
int check_tensors(const Side& q, const Side& q_out, const Side& k, const Side& k_out, int tokens, bool has_k) {
  int rc = check_side(q, tokens);
  if (!rc) rc = check_side(q_out, tokens);
  if (!rc && has_k) rc = check_side(k, tokens);
  if (!rc && has_k) rc = check_side(k_out, tokens);
  if (rc) return rc;
  const auto clash = [tokens](const Side& in, const Side& out) {
    const bool same = in.p == out.p && (tokens == 1 || in.stride == out.stride);
    return !same && overlap(in, out, tokens);
  };
  if (clash(q, q_out) || (has_k && clash(k, k_out)))
    return err(GEMMA_ERR_INVALID_ARG, "an output must be its input (same stride) or must not overlap it");
  if (has_k && (overlap(q_out, k, tokens) || overlap(k_out, q, tokens) || overlap(q_out, k_out, tokens)))
    return err(GEMMA_ERR_INVALID_ARG, "an output overlaps the other input or output");
  return GEMMA_OK;
}

}  // namespace
}  // namespace hlg

using namespace hlg;

extern "C" int gemma_rope_axes(const void* q, long long q_stride, const void* k, long long k_stride,
                               const int32_t* positions, int n_axes, const int* axis_pairs, int tokens, int n_q_heads,
                               int n_kv_heads, int head_dim, float rope_theta, void* q_out, long long q_out_stride,
                               void* k_out, long long k_out_stride, unsigned flags, void* stream) {
  if (flags & ~(GEMMA_ROPE_INTERLEAVED | GEMMA_ROPE_AXIS_LADDERS | GEMMA_ROPE_INVERSE))
    return err(GEMMA_ERR_INVALID_ARG, "unknown flags");
  if (tokens < 0 || n_q_heads <= 0 || n_kv_heads < 0)
    return err(GEMMA_ERR_INVALID_ARG, "tokens, n_q_heads or n_kv_heads out of range");
  if (head_dim <= 0 || head_dim % 8 || head_dim > 2 * MAX_PAIRS)
    return err(GEMMA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 512");
  if ((long long)(n_q_heads + (long long)n_kv_heads) * head_dim > (1 << 30))
    return err(GEMMA_ERR_UNSUPPORTED, "heads * head_dim exceeds 2^30");
  if (n_axes < 1 || n_axes > MAX_AXES || !axis_pairs) return err(GEMMA_ERR_INVALID_ARG, "n_axes must be 1 to 4");
  if (!(rope_theta > 0.f) || !std::isfinite(rope_theta))
    return err(GEMMA_ERR_INVALID_ARG, "rope_theta must be positive and finite");
  long long n_rot = 0;
  for (int x = 0; x < n_axes; ++x) {
    if (axis_pairs[x] < 0) return err(GEMMA_ERR_INVALID_ARG, "axis_pairs must not be negative");
    n_rot += axis_pairs[x];
  }
  if (n_rot > head_dim / 2) return err(GEMMA_ERR_INVALID_ARG, "axis_pairs sum to more than head_dim / 2");
  if (tokens == 0) return record_ok();
  if (!positions || reinterpret_cast<uintptr_t>(positions) & 3u)
    return err(GEMMA_ERR_INVALID_ARG, "positions: null or misaligned pointer");
  const long long q_row = (long long)n_q_heads * head_dim, k_row = (long long)n_kv_heads * head_dim;
  const int rc = check_tensors(Side{q, q_stride, q_row}, Side{q_out, q_out_stride, q_row}, Side{k, k_stride, k_row},
                               Side{k_out, k_out_stride, k_row}, tokens, n_kv_heads > 0);
  if (rc) return rc;

  AxesArgs a;
  const double log2_theta = std::log2((double)rope_theta), sign = (flags & GEMMA_ROPE_INVERSE) ? -1.0 : 1.0;
  double ladder[MAX_AXES][MAX_PAIRS];  // [0]: by the pair's number; with AXIS_LADDERS, of each axis by rank
  if (flags & GEMMA_ROPE_AXIS_LADDERS) {
    for (int x = 0; x < n_axes; ++x)
      if (axis_pairs[x] > 0) half_turn_ladder(log2_theta / axis_pairs[x], axis_pairs[x], ladder[x]);
  } else {
    half_turn_ladder(2.0 / head_dim * log2_theta, (int)n_rot, ladder[0]);
  }
  int i = 0;
  const auto put = [&](int x, int rank) {
    a.freq[i] = sign * ((flags & GEMMA_ROPE_AXIS_LADDERS) ? ladder[x][rank] : ladder[0][i]);
    a.axis[i] = (unsigned char)x;
    ++i;
  };
  if (flags & GEMMA_ROPE_INTERLEAVED) {
    for (int rank = 0; i < n_rot; ++rank)
      for (int x = 0; x < n_axes; ++x)
        if (rank < axis_pairs[x]) put(x, rank);
  } else {
    for (int x = 0; x < n_axes; ++x)
      for (int rank = 0; rank < axis_pairs[x]; ++rank) put(x, rank);
  }
  a.n_rot = (int)n_rot;
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.q_out = static_cast<bf16*>(q_out);
  a.k_out = static_cast<bf16*>(k_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.pos = positions;
  a.tokens = tokens;
  a.Hq = n_q_heads;
  a.Hkv = n_kv_heads;
  a.D = head_dim;
  const int per_cta = AX_T / (head_dim / 8), ctas = (tokens - 1) / per_cta + 1;  // tokens may be the largest int
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (ctas >= multiprocessors()) {
    k_rope_axes<8><<<ctas, AX_T, 0, st>>>(a);
  } else {  // few tokens: two head vectors of a thread, the others in more CTAs
    const int shares = std::min((n_q_heads + n_kv_heads + 1) / 2, 65535);
    k_rope_axes<2><<<dim3(ctas, shares), AX_T, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    char m[256];
    snprintf(m, sizeof m, "multi-axis rotation launch: %s", cudaGetErrorString(e));
    return err(GEMMA_ERR_CUDA, m);
  }
  return record_ok();
}
