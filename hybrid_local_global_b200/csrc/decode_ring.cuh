// decode_ring.cuh -- layout of the decode kernels' shared-memory ring: runs of
// RPC consecutive cached rows, each run (one bulk copy) padded by 16 bytes.
#pragma once

#include <stdint.h>

namespace hlg {

__host__ __device__ constexpr int ring_group_bytes(int D, int RPC) { return RPC * D * 2 + 16; }

// byte offset of row r within a run of row groups
template <int D, int RPC>
__device__ __forceinline__ int ring_row_off(int r) {
  return (r / RPC) * ring_group_bytes(D, RPC) + (r % RPC) * (D * 2);
}

// The key that MMA index n (0..15) of a 16-key sub-block stands for. S and
// P.V only need the same order for the K and V fragments and the mask, so
// the 8 rows each ldmatrix reads are taken from different row groups where
// possible: rows of one group are D*2 bytes apart and share bank groups,
// while consecutive groups are shifted by the 16-byte pad.
template <int RPC>
__device__ __forceinline__ int ring_key(int n) {
  constexpr int NG = 16 / RPC;  // row groups per 16 keys
  return (n % NG) * RPC + n / NG;
}

}  // namespace hlg
