// pages.cu -- upkeep of a paged cache's pages on the device: forking rows of
// the page table, growing them with copy on write, trimming, compacting the
// pool, and copying pages ("Gemma 4: End-to-End Architecture Walkthrough", 3b:
// a global layer caches K/V for the whole context; pages let the pool hold
// only what is still attended to, and let sequences share a prefix).
//
// The book is a page table [n_seqs][pages_per_seq] (entry = page, -1 = none)
// and one reference count per page: the number of table entries that name it.
// A page with count 0 is free; a grant takes the free pages with the lowest
// numbers, in (row, entry) order, so every result is independent of how
// threads interleave (the atomics below are integer sums and maxima).
//
// What bounds these calls: the table work is a few hundred kilobytes at most
// and latency-bound, so each plan is one CTA and one launch; moving page
// contents is bound by HBM (read + write).
#include <algorithm>
#include <cstdio>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "pair.cuh"

namespace hlg {

namespace {

constexpr int MAX_SEQS = 4096;       // rows of a book (row offsets and fork columns live in shared memory)
constexpr int MAX_PAGES = 1 << 20;   // pages of a book (compaction keeps one bit per page in shared memory)
constexpr int MAX_SEGS = 128;        // page segments per copy launch (an int8 pool has two: codes, params)
constexpr int FEW_SEGS = 8;
constexpr int PLAN_T = 1024;
constexpr int SMALL_CTAS = 8;        // CTAs of a one-launch reserve
constexpr int COPY_T = 256;
constexpr int COPY_V = 4;            // 16-byte words per thread and tile
// bytes that T threads copy at a time
constexpr int tile_bytes(int T) { return T * COPY_V * 16; }

struct Book {
  int32_t* table;
  int32_t* ref;
  int n_seqs, pps, n_pages, ps;
};

// Exclusive sum over the CTA's PLAN_T threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  const int ws = warp_sum[lane];
  int s = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  const int before = __shfl_sync(0xffffffffu, s - ws, warp);
  *total = __shfl_sync(0xffffffffu, s, 31);
  __syncthreads();  // warp_sum is reused by the next call
  return before + x - v;
}

// ---------------------------------------------------------------------------
// Fork: row b becomes what row parents[b] was before the call (b itself: as it
// is; -1: empty). A CTA takes FORK_C columns of every row through shared
// memory, so all old entries are read before any is written.
// ---------------------------------------------------------------------------
constexpr int FORK_C = 8;

__global__ void __launch_bounds__(256) k_pages_fork(Book bk, const int32_t* __restrict__ parents, int* status) {
  extern __shared__ int32_t old_s[];  // [n_seqs][FORK_C]
  const int c0 = blockIdx.x * FORK_C;
  const int n = bk.n_seqs * FORK_C;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = i / FORK_C, c = c0 + i % FORK_C;
    old_s[i] = c < bk.pps ? bk.table[(int64_t)b * bk.pps + c] : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = i / FORK_C, c = c0 + i % FORK_C;
    if (c >= bk.pps) continue;
    const int p = parents[b];
    if (p == b) continue;
    if (p < -1 || p >= bk.n_seqs) {  // reported; the row stays as it is
      set_status(status, GEMMA_ERR_DEVICE_RANGE);
      continue;
    }
    const int32_t was = old_s[i], now = p < 0 ? -1 : old_s[p * FORK_C + i % FORK_C];
    if (was == now) continue;
    bk.table[(int64_t)b * bk.pps + c] = now;
    if (now >= 0 && now < bk.n_pages) atomicAdd(&bk.ref[now], 1);
    if (was >= 0 && was < bk.n_pages) atomicSub(&bk.ref[was], 1);
  }
}

// ---------------------------------------------------------------------------
// Trim: drops the entries of pages that hold no position a later token sees.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_pages_trim(Book bk, const int32_t* __restrict__ seq_lens, int window,
                                                    int sinks, int* status) {
  const int b = blockIdx.y;
  const int64_t len = seq_lens[b];
  if (len < 0) return;  // the row stays as it is
  if (len > (int64_t)bk.pps * bk.ps) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(status, GEMMA_ERR_DEVICE_RANGE);
    return;
  }
  for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < bk.pps; c += gridDim.x * blockDim.x) {
    const int32_t e = bk.table[(int64_t)b * bk.pps + c];
    if (e == -1) continue;
    const int64_t begin = (int64_t)c * bk.ps, end = begin + bk.ps < len ? begin + bk.ps : len;
    // the next token sits at position len or later: it sees j < len iff
    // window == 0, j > len - window, or j < sinks
    if (begin < len && (window == 0 || end > len - window + 1 || begin < sinks)) continue;
    bk.table[(int64_t)b * bk.pps + c] = -1;
    if (e >= 0 && e < bk.n_pages)
      atomicSub(&bk.ref[e], 1);
    else
      set_status(status, GEMMA_ERR_DEVICE_RANGE);
  }
}

// ---------------------------------------------------------------------------
// Reserve: makes positions [len, len + new) of every row writable.
// ---------------------------------------------------------------------------
struct ReservePlan {  // workspace
  int32_t* writers;   // [n_pages] entries of this call that write a shared page
  int32_t* last;      // [n_pages] the last of them, in (row, entry) order
  int32_t* fresh;     // [n_pages] free pages granted, in order
  int32_t* slots;     // [n_seqs * pps] per entry to be written: KEEP, GRANT, or the shared page it leaves
  int32_t* copies;    // [n_seqs][3] src, dst, rows
  int32_t* n_copies;
};
constexpr int GRANT = -1, KEEP = -2;

// row whose slots hold slot i: the last b with off[b] <= i
__device__ __forceinline__ int row_of(const int* off, int n_seqs, int i) {
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void reserve_plan(const Book& bk, const int32_t* __restrict__ seq_lens,
                                             const int32_t* __restrict__ new_tokens, int32_t* lacking,
                                             const ReservePlan& ws, int* status) {
  __shared__ int off[MAX_SEQS];  // first slot of each row
  __shared__ int s_copies;
  const int tid = threadIdx.x;
  if (tid == 0) s_copies = 0;
  int n_slots = 0;
  for (int b0 = 0; b0 < bk.n_seqs; b0 += PLAN_T) {
    const int b = b0 + tid;
    int cnt = 0;
    if (b < bk.n_seqs) {
      const int64_t n = new_tokens[b], len = seq_lens[b];
      if (n != 0) {
        if (n < 0 || len < 0 || len + n > (int64_t)bk.pps * bk.ps)
          set_status(status, GEMMA_ERR_DEVICE_RANGE);  // the row is left out
        else
          cnt = (int)((len + n - 1) / bk.ps - len / bk.ps + 1);
      }
    }
    int tot;
    const int ex = block_scan(cnt, &tot);
    if (b < bk.n_seqs) off[b] = n_slots + ex;
    n_slots += tot;
  }
  __syncthreads();
  // what each entry needs
  for (int i = tid; i < n_slots; i += PLAN_T) {
    const int b = row_of(off, bk.n_seqs, i);
    const int c = seq_lens[b] / bk.ps + (i - off[b]);
    const int32_t e = bk.table[(int64_t)b * bk.pps + c];
    int32_t dec = KEEP;
    if (e == -1) {
      dec = GRANT;
    } else if (e < 0 || e >= bk.n_pages || bk.ref[e] < 1) {
      set_status(status, GEMMA_ERR_DEVICE_RANGE);
    } else if (bk.ref[e] > 1) {
      dec = e;
      ws.writers[e] = 0;
      ws.last[e] = -1;
    }
    ws.slots[i] = dec;
  }
  __syncthreads();
  for (int i = tid; i < n_slots; i += PLAN_T) {
    const int32_t e = ws.slots[i];
    if (e < 0) continue;
    atomicAdd(&ws.writers[e], 1);
    atomicMax(&ws.last[e], i);
  }
  __syncthreads();
  // of a page that only entries of this call hold, the last one keeps it
  int mine = 0;
  for (int i = tid; i < n_slots; i += PLAN_T) {
    const int32_t e = ws.slots[i];
    if (e >= 0 && ws.writers[e] >= bk.ref[e] && ws.last[e] == i)
      ws.slots[i] = KEEP;
    else if (e != KEEP)
      ++mine;
  }
  int need;
  block_scan(mine, &need);
  int found = 0;
  for (int p0 = 0; p0 < bk.n_pages && found < need; p0 += PLAN_T * 4) {
    const int p = p0 + tid * 4;
    int cnt = 0;
    bool is_free[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      is_free[u] = p + u < bk.n_pages && bk.ref[p + u] == 0;
      cnt += is_free[u];
    }
    int tot;
    int k = found + block_scan(cnt, &tot);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (is_free[u]) ws.fresh[k++] = p + u;
    found += tot;
  }
  __syncthreads();
  if (found < need) {  // nothing is granted
    if (tid == 0) {
      *lacking = need - found;
      *ws.n_copies = 0;
      set_status(status, GEMMA_ERR_DEVICE_RANGE);
    }
    return;
  }
  int given = 0;
  for (int i0 = 0; i0 < n_slots && given < need; i0 += PLAN_T) {
    const int i = i0 + tid;
    const int32_t dec = i < n_slots ? ws.slots[i] : KEEP;
    int tot;
    const int k = given + block_scan(dec != KEEP, &tot);
    given += tot;
    if (dec == KEEP) continue;
    const int b = row_of(off, bk.n_seqs, i);
    const int len = seq_lens[b];
    const int32_t page = ws.fresh[k];
    bk.table[(int64_t)b * bk.pps + len / bk.ps + (i - off[b])] = page;
    bk.ref[page] = 1;
    if (dec >= 0) {
      atomicSub(&bk.ref[dec], 1);
      if (i == off[b] && len % bk.ps) {  // the entry's page holds rows of the sequence
        const int s = atomicAdd(&s_copies, 1);
        ws.copies[3 * s] = dec;
        ws.copies[3 * s + 1] = page;
        ws.copies[3 * s + 2] = len % bk.ps;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    *lacking = 0;
    *ws.n_copies = s_copies;
  }
}

__global__ void __launch_bounds__(PLAN_T) k_pages_reserve(Book bk, const int32_t* __restrict__ seq_lens,
                                                          const int32_t* __restrict__ new_tokens,
                                                          int32_t* lacking, ReservePlan ws, int* status) {
  let_next_start();  // the copies'
  reserve_plan(bk, seq_lens, new_tokens, lacking, ws, status);
}

// ---------------------------------------------------------------------------
// Compact: with n live pages, the k-th live page numbered n or more moves into
// the k-th free page numbered below n.
// ---------------------------------------------------------------------------
struct CompactPlan {
  int32_t* map;      // [n_pages] new number of each page, -1: free
  int32_t* holes;    // [n_pages]
  int32_t* movers;   // [n_pages]
  int32_t* copies;   // [n_pages][3]
  int32_t* n_copies;
};

__global__ void __launch_bounds__(PLAN_T) k_pages_compact(Book bk, CompactPlan ws, int32_t* n_live) {
  extern __shared__ uint32_t live_s[];  // one bit per page
  let_next_start();  // the copies'
  const int tid = threadIdx.x, lane = tid & 31;
  const int n_words = (bk.n_pages + 31) / 32;
  int cnt = 0;
  for (int p0 = 0; p0 < n_words * 32; p0 += PLAN_T) {
    const int p = p0 + tid;
    const uint32_t bits = __ballot_sync(0xffffffffu, p < bk.n_pages && bk.ref[p] > 0);
    if (lane == 0 && p / 32 < n_words) {
      live_s[p / 32] = bits;
      cnt += __popc(bits);
    }
  }
  int live;
  block_scan(cnt, &live);
  // each thread's run of words: holes below `live`, movers from it on
  const int per = (n_words + PLAN_T - 1) / PLAN_T;
  const int w0 = min(tid * per, n_words), w1 = min(w0 + per, n_words);
  int holes = 0, movers = 0;
  for (int p = w0 * 32; p < w1 * 32 && p < bk.n_pages; ++p) {
    const bool on = live_s[p / 32] >> (p % 32) & 1u;
    holes += !on && p < live;
    movers += on && p >= live;
  }
  int total, moves;
  int h = block_scan(holes, &total), m = block_scan(movers, &moves);
  for (int p = w0 * 32; p < w1 * 32 && p < bk.n_pages; ++p) {
    const bool on = live_s[p / 32] >> (p % 32) & 1u;
    if (!on && p < live) ws.holes[h++] = p;
    if (on && p >= live) ws.movers[m++] = p;
    else ws.map[p] = on ? p : -1;
  }
  __syncthreads();
  for (int k = tid; k < moves; k += PLAN_T) {
    const int32_t src = ws.movers[k], dst = ws.holes[k];
    ws.map[src] = dst;
    bk.ref[dst] = bk.ref[src];
    bk.ref[src] = 0;
    ws.copies[3 * k] = src;
    ws.copies[3 * k + 1] = dst;
    ws.copies[3 * k + 2] = bk.ps;
  }
  if (tid == 0) {
    *n_live = live;
    *ws.n_copies = moves;
  }
}

// ---------------------------------------------------------------------------
// Page contents
// ---------------------------------------------------------------------------
// One run of a page's bytes per head: `rows` of them are copied (row_bytes
// each) from head_bytes apart.
struct Seg {
  unsigned char* base;
  long long page_bytes;
  int head_bytes, row_bytes;
  int tiles_per_head, tile0;  // the segment's first tile of a page
};

struct CopyList {
  int n_segs, tiles;          // tiles per page over all segments
  const int32_t* src;         // pair k: src[k * stride], dst[k * stride], rows[k * stride] (null: whole pages)
  const int32_t* dst;
  const int32_t* rows;
  int stride;
  const int32_t* n_dev;       // pairs: *n_dev, or n_host when null
  int n_host;
  int n_pages, ps;
  int check;                  // 1: the caller's own list: see pair_ok
  int* status;
};
// Two sizes: most calls list a few pools, and a launch copies its parameters.
template <int N>
struct CopyArgs {
  CopyList list;
  Seg seg[N];
};

// A listed pair is carried out iff both pages exist, differ, no other pair
// names the same destination, and no other pair writes its source; the answer
// depends on the list alone. Called by the whole CTA.
__device__ __forceinline__ bool pair_ok(const CopyList& a, int k, int n) {
  const int32_t s = a.src[k], d = a.dst[k];
  if (s == d && s >= 0 && s < a.n_pages) return false;  // nothing to do, unless another pair names it
  bool bad = s < 0 || s >= a.n_pages || d < 0 || d >= a.n_pages;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    if (j == k) continue;
    const int32_t dj = a.dst[j];
    bad |= dj == d || (dj == s && a.src[j] != dj);
  }
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0) set_status(a.status, GEMMA_ERR_DEVICE_RANGE);
  return false;
}

// CTA `cta` of `ctas` copies its share of the list's tiles, T threads of
// COPY_V words each (the list counts tiles of tile_bytes(T)).
template <int T>
__device__ __forceinline__ void copy_tiles(const CopyList& a, const Seg* seg, int cta, int ctas) {
  constexpr int TILE = tile_bytes(T);
  const int n = a.n_dev ? *a.n_dev : a.n_host;
  int checked = -1;
  bool ok = true;
  for (int64_t w = cta; w < (int64_t)n * a.tiles; w += ctas) {
    const int k = (int)(w / a.tiles), t = (int)(w - (int64_t)k * a.tiles);
    if (a.check && checked != k) {
      ok = pair_ok(a, k, n);
      checked = k;
    }
    if (!ok) continue;
    int lo = 0, hi = a.n_segs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (seg[mid].tile0 <= t) lo = mid;
      else hi = mid - 1;
    }
    const Seg& g = seg[lo];
    const int head = (t - g.tile0) / g.tiles_per_head, tile = (t - g.tile0) - head * g.tiles_per_head;
    const int rows = a.rows ? a.rows[(int64_t)k * a.stride] : a.ps;
    const int bytes = min(rows * g.row_bytes - tile * TILE, TILE);
    if (bytes <= 0) continue;
    const int64_t at = (int64_t)head * g.head_bytes + (int64_t)tile * TILE;
    const unsigned char* from = g.base + a.src[(int64_t)k * a.stride] * g.page_bytes + at;
    unsigned char* to = g.base + a.dst[(int64_t)k * a.stride] * g.page_bytes + at;
    uint4 v[COPY_V];
#pragma unroll
    for (int u = 0; u < COPY_V; ++u) {
      const int o = (u * T + threadIdx.x) * 16;
      if (o + 16 <= bytes) v[u] = *reinterpret_cast<const uint4*>(from + o);
    }
#pragma unroll
    for (int u = 0; u < COPY_V; ++u) {
      const int o = (u * T + threadIdx.x) * 16;
      if (o + 16 <= bytes) *reinterpret_cast<uint4*>(to + o) = v[u];
      else if (o < bytes)  // an odd number of 8-byte (min, step) rows
        *reinterpret_cast<uint2*>(to + o) = *reinterpret_cast<const uint2*>(from + o);
    }
  }
}

// The copies of a list; with `map`, first the entries of the book's table by
// their pages' new names.
template <int N>
__global__ void __launch_bounds__(COPY_T) k_pages_copy(const __grid_constant__ CopyArgs<N> a, const Book bk,
                                                       const int32_t* __restrict__ map) {
  after_previous();  // the plan
  if (map) {
    const int64_t n = (int64_t)bk.n_seqs * bk.pps;
    for (int64_t i = (int64_t)blockIdx.x * COPY_T + threadIdx.x; i < n; i += (int64_t)gridDim.x * COPY_T) {
      const int32_t e = bk.table[i];
      if (e == -1) continue;
      const int32_t to = e >= 0 && e < bk.n_pages ? map[e] : -1;
      if (to < 0)
        set_status(a.list.status, GEMMA_ERR_DEVICE_RANGE);  // an entry that names no live page stays as it is
      else if (to != e)
        bk.table[i] = to;
    }
  }
  copy_tiles<COPY_T>(a.list, a.seg, blockIdx.x, gridDim.x);
}

// Reserve in one launch, where few bytes can be copied at most: one cluster,
// whose first CTA makes the plan.
template <int N>
__global__ void __cluster_dims__(SMALL_CTAS, 1, 1) __launch_bounds__(PLAN_T)
    k_pages_reserve_small(Book bk, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ new_tokens,
                          int32_t* lacking, ReservePlan ws, const __grid_constant__ CopyArgs<N> a) {
  if (blockIdx.x == 0) reserve_plan(bk, seq_lens, new_tokens, lacking, ws, a.list.status);
  __syncwarp();
  pair::cluster_sync();  // the plan is visible to the cluster
  copy_tiles<PLAN_T>(a.list, a.seg, blockIdx.x, SMALL_CTAS);
}

// ---------------------------------------------------------------- host side
int err(int code, const char* msg) { return record_error(code, msg); }

int cuda_err(cudaError_t e, const char* what) {
  char m[256];
  snprintf(m, sizeof m, "%s: %s", what, cudaGetErrorString(e));
  return record_error(GEMMA_ERR_CUDA, m);
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool within_limits(int n_seqs, int pages_per_seq, int n_pages) {
  return n_seqs <= MAX_SEQS && n_pages <= MAX_PAGES && (int64_t)n_seqs * pages_per_seq <= (1 << 30);
}

int check_book(const gemma_page_book* b) {
  if (!b || !b->page_table || !b->ref_count) return err(GEMMA_ERR_INVALID_ARG, "page book: null pointer");
  if (b->n_seqs <= 0 || b->pages_per_seq <= 0 || b->n_pages <= 0)
    return err(GEMMA_ERR_INVALID_ARG, "page book: n_seqs, pages_per_seq and n_pages must be positive");
  if (b->page_size <= 0 || b->page_size % 128)
    return err(GEMMA_ERR_INVALID_ARG, "page book: page_size must be a positive multiple of 128");
  if ((int64_t)b->pages_per_seq * b->page_size > INT32_MAX)
    return err(GEMMA_ERR_INVALID_ARG, "page book: pages_per_seq * page_size exceeds 2^31");
  if (!within_limits(b->n_seqs, b->pages_per_seq, b->n_pages))
    return err(GEMMA_ERR_UNSUPPORTED, "page book: more than 4096 rows, 2^20 pages or 2^30 table entries");
  if (misaligned(b->page_table, 4) || misaligned(b->ref_count, 4))
    return err(GEMMA_ERR_INVALID_ARG, "page book: misaligned pointer");
  return GEMMA_OK;
}

int check_pools(const gemma_page_pool* pools, int n_pools, int page_size) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return err(GEMMA_ERR_INVALID_ARG, "bad pool list");
  for (int i = 0; i < n_pools; ++i) {
    const gemma_page_pool& p = pools[i];
    if (!p.pool || misaligned(p.pool, 16)) return err(GEMMA_ERR_INVALID_ARG, "pool pointer null or not 16-byte aligned");
    if (p.n_kv_heads <= 0 || p.head_dim <= 0 || p.head_dim % 16)
      return err(GEMMA_ERR_INVALID_ARG, "pool: n_kv_heads must be positive and head_dim a positive multiple of 16");
    if (p.flags & ~GEMMA_F_KV_INT8) return err(GEMMA_ERR_INVALID_ARG, "pool: unknown flags");
    if ((int64_t)p.n_kv_heads * page_size * p.head_dim * 2 > INT32_MAX)
      return err(GEMMA_ERR_UNSUPPORTED, "pool: a page of 2^31 bytes or more");
  }
  return GEMMA_OK;
}

Book book_of(const gemma_page_book* b) {
  return Book{b->page_table, b->ref_count, b->n_seqs, b->pages_per_seq, b->n_pages, b->page_size};
}

// Segments of pools [i0, i0 + MAX_SEGS / 2) and their tiles of `tile` bytes.
void segments(CopyList& a, Seg* seg, const gemma_page_pool* pools, int n_pools, int i0, int tile) {
  a.n_segs = a.tiles = 0;
  for (int i = i0; i < std::min(n_pools, i0 + MAX_SEGS / 2); ++i) {
    const gemma_page_pool& p = pools[i];
    const bool q8 = p.flags & GEMMA_F_KV_INT8;
    for (int part = 0; part < (q8 ? 2 : 1); ++part) {
      Seg g{};
      const int row = part ? 8 : p.head_dim * (q8 ? 1 : 2);
      g.base = static_cast<unsigned char*>(p.pool) +
               (part ? gemma_kv_codes_bytes(a.n_pages, p.n_kv_heads, a.ps, p.head_dim) : 0);
      g.page_bytes = (long long)p.n_kv_heads * a.ps * row;
      // whole pages are one run; partial ones a run per head
      const int heads = a.rows ? p.n_kv_heads : 1;
      g.row_bytes = a.rows ? row : row * p.n_kv_heads;
      g.head_bytes = a.ps * g.row_bytes;
      g.tiles_per_head = (int)(((int64_t)g.head_bytes + tile - 1) / tile);
      g.tile0 = a.tiles;
      a.tiles += heads * g.tiles_per_head;
      seg[a.n_segs++] = g;
    }
  }
}

template <int N>
cudaError_t launch_copy(const CopyList& list, const Seg* seg, int64_t work, const Book& bk, const int32_t* map,
                        cudaStream_t st) {
  CopyArgs<N> a;
  a.list = list;
  std::copy(seg, seg + list.n_segs, a.seg);
  // 32 CTAs per SM in all (256 MB: 42 us, 92 % of the copy rate; 8 per SM: 45)
  const int64_t grid = std::min<int64_t>(work, (int64_t)multiprocessors() * 32);
  const dim3 ctas((unsigned)std::max<int64_t>(grid, 1));
  if (list.n_dev) return launch_early(k_pages_copy<N>, ctas, COPY_T, 0, st, 0, a, bk, map);
  k_pages_copy<N><<<ctas, COPY_T, 0, st>>>(a, bk, map);
  return cudaGetLastError();
}

// Copies the listed pages of every pool (max_pairs bounds the pairs), and
// renames the book's entries by `map` if given.
cudaError_t copy_pages(CopyList& list, const gemma_page_pool* pools, int n_pools, int64_t max_pairs, const Book& bk,
                       const int32_t* map, cudaStream_t st) {
  Seg seg[MAX_SEGS];
  for (int i0 = 0; i0 == 0 || i0 < n_pools; i0 += MAX_SEGS / 2) {
    segments(list, seg, pools, n_pools, i0, tile_bytes(COPY_T));
    if (i0) map = nullptr;
    const int64_t names = map ? ((int64_t)bk.n_seqs * bk.pps + COPY_T - 1) / COPY_T : 0;
    const int64_t work = std::max(max_pairs * list.tiles, names);
    const cudaError_t e = list.n_segs <= FEW_SEGS ? launch_copy<FEW_SEGS>(list, seg, work, bk, map, st)
                                                  : launch_copy<MAX_SEGS>(list, seg, work, bk, map, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t ints256(int64_t n) { return ((size_t)n * 4 + 255) & ~size_t(255); }

// shared by reserve (writers, last, fresh, slots, copies) and compact (map, holes, movers, copies)
size_t plan_bytes(int64_t n_seqs, int64_t pps, int64_t n_pages) {
  const size_t reserve = 3 * ints256(n_pages) + ints256(n_seqs * pps) + ints256(3 * n_seqs);
  const size_t compact = 3 * ints256(n_pages) + ints256(3 * n_pages);
  return 256 + std::max(reserve, compact);
}

// Lets a kernel have as much dynamic shared memory as its largest book asks for:
// the same on every call, so that no thread with a small book lowers what
// another's launch counts on, and no threshold depends on what the kernel declares.
template <class... P>
cudaError_t allow_shared(void (*kern)(P...), int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

int check_plan_ws(const gemma_page_book* b, const void* ws, size_t bytes) {
  if (!ws || bytes < plan_bytes(b->n_seqs, b->pages_per_seq, b->n_pages))
    return err(GEMMA_ERR_CAPACITY, "workspace smaller than gemma_kv_pages_workspace_size");
  if (misaligned(ws, 16)) return err(GEMMA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return GEMMA_OK;
}

}  // namespace
}  // namespace hlg

using namespace hlg;

extern "C" {

size_t gemma_kv_pages_workspace_size(int n_seqs, int pages_per_seq, int n_pages) {
  if (n_seqs <= 0 || pages_per_seq <= 0 || n_pages <= 0 || !within_limits(n_seqs, pages_per_seq, n_pages)) return 0;
  return plan_bytes(n_seqs, pages_per_seq, n_pages);
}

int gemma_kv_pages_fork(const gemma_page_book* book, const int32_t* parents, void* stream) {
  int rc = check_book(book);
  if (rc) return rc;
  if (!parents || misaligned(parents, 4)) return err(GEMMA_ERR_INVALID_ARG, "parents: null or misaligned pointer");
  int* status = device_status();
  if (!status) return err(GEMMA_ERR_CUDA, "no CUDA device");
  const int smem = book->n_seqs * FORK_C * 4;
  cudaError_t e = allow_shared(k_pages_fork, MAX_SEQS * FORK_C * 4);
  if (e != cudaSuccess) return cuda_err(e, "page fork");
  k_pages_fork<<<(book->pages_per_seq + FORK_C - 1) / FORK_C, 256, smem, static_cast<cudaStream_t>(stream)>>>(
      book_of(book), parents, status);
  e = cudaGetLastError();
  return e != cudaSuccess ? cuda_err(e, "page fork launch") : record_ok();
}

int gemma_kv_pages_trim(const gemma_page_book* book, const int32_t* seq_lens, int window, int sinks, void* stream) {
  int rc = check_book(book);
  if (rc) return rc;
  if (!seq_lens || misaligned(seq_lens, 4)) return err(GEMMA_ERR_INVALID_ARG, "seq_lens: null or misaligned pointer");
  if (window < 0 || sinks < 0) return err(GEMMA_ERR_INVALID_ARG, "window and sinks must not be negative");
  int* status = device_status();
  if (!status) return err(GEMMA_ERR_CUDA, "no CUDA device");
  const dim3 grid(std::min((book->pages_per_seq + 255) / 256, 64), book->n_seqs);
  k_pages_trim<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(book_of(book), seq_lens, window, sinks, status);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? cuda_err(e, "page trim launch") : record_ok();
}

int gemma_kv_pages_reserve(const gemma_page_book* book, const gemma_page_pool* pools, int n_pools,
                           const int32_t* seq_lens, const int32_t* new_tokens, int32_t* lacking, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int rc = check_book(book);
  if (!rc) rc = check_pools(pools, n_pools, book->page_size);
  if (rc) return rc;
  if (!seq_lens || !new_tokens || !lacking || misaligned(seq_lens, 4) || misaligned(new_tokens, 4) ||
      misaligned(lacking, 4))
    return err(GEMMA_ERR_INVALID_ARG, "seq_lens, new_tokens, lacking: null or misaligned pointer");
  rc = check_plan_ws(book, workspace, workspace_bytes);
  if (rc) return rc;
  int* status = device_status();
  if (!status) return err(GEMMA_ERR_CUDA, "no CUDA device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t n_pages = book->n_pages, slots = (int64_t)book->n_seqs * book->pages_per_seq;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  const auto take = [&w](int64_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(w);
    w += ints256(n);
    return p;
  };
  ReservePlan plan;
  plan.n_copies = take(1);
  plan.writers = take(n_pages);
  plan.last = take(n_pages);
  plan.fresh = take(n_pages);
  plan.slots = take(slots);
  plan.copies = take(3 * (int64_t)book->n_seqs);
  CopyList a{};
  a.src = plan.copies;
  a.dst = plan.copies + 1;
  a.rows = plan.copies + 2;
  a.stride = 3;
  a.n_dev = plan.n_copies;
  a.n_pages = book->n_pages;
  a.ps = book->page_size;
  a.status = status;
  // The one-launch form saves a caller 2.4 us of CPU time a call; on the GPU it
  // takes 1 us more with up to 1 MB of tails (all rows splitting full pages;
  // half of it copied: 8.8 us against 7.8), 2.5 us more with 2 MB (10.6 against
  // 8.1) and 10 with 8 MB. So: up to 1 MB.
  double most = 0.0;
  for (int i = 0; i < n_pools; ++i)
    most += (double)book->n_seqs * pools[i].n_kv_heads * book->page_size * pools[i].head_dim * 2;
  if (n_pools > 0 && n_pools <= FEW_SEGS / 2 && most <= 1 << 20) {
    CopyArgs<FEW_SEGS> c;
    segments(a, c.seg, pools, n_pools, 0, tile_bytes(PLAN_T));
    c.list = a;
    k_pages_reserve_small<FEW_SEGS><<<SMALL_CTAS, PLAN_T, 0, st>>>(book_of(book), seq_lens, new_tokens, lacking, plan, c);
    const cudaError_t es = cudaGetLastError();
    return es != cudaSuccess ? cuda_err(es, "page reserve launch") : record_ok();
  }
  k_pages_reserve<<<1, PLAN_T, 0, st>>>(book_of(book), seq_lens, new_tokens, lacking, plan, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_err(e, "page reserve launch");
  if (n_pools > 0) {
    e = copy_pages(a, pools, n_pools, book->n_seqs, book_of(book), nullptr, st);
    if (e != cudaSuccess) return cuda_err(e, "page copy launch");
  }
  return record_ok();
}

int gemma_kv_pages_compact(const gemma_page_book* book, const gemma_page_pool* pools, int n_pools, int32_t* n_live,
                           int32_t* page_map, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_book(book);
  if (!rc) rc = check_pools(pools, n_pools, book->page_size);
  if (rc) return rc;
  if (!n_live || misaligned(n_live, 4) || misaligned(page_map, 4))
    return err(GEMMA_ERR_INVALID_ARG, "n_live null, or n_live or page_map misaligned");
  rc = check_plan_ws(book, workspace, workspace_bytes);
  if (rc) return rc;
  int* status = device_status();
  if (!status) return err(GEMMA_ERR_CUDA, "no CUDA device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t n_pages = book->n_pages;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  const auto take = [&w](int64_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(w);
    w += ints256(n);
    return p;
  };
  CompactPlan plan;
  plan.n_copies = take(1);
  plan.map = take(n_pages);
  plan.holes = take(n_pages);
  plan.movers = take(n_pages);
  plan.copies = take(3 * n_pages);
  if (page_map) plan.map = page_map;
  const int smem = (book->n_pages + 31) / 32 * 4;
  cudaError_t e = allow_shared(k_pages_compact, MAX_PAGES / 8);
  if (e != cudaSuccess) return cuda_err(e, "page compact");
  k_pages_compact<<<1, PLAN_T, smem, st>>>(book_of(book), plan, n_live);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_err(e, "page compact launch");
  CopyList a{};
  a.src = plan.copies;
  a.dst = plan.copies + 1;
  a.stride = 3;
  a.n_dev = plan.n_copies;
  a.n_pages = book->n_pages;
  a.ps = book->page_size;
  a.status = status;
  e = copy_pages(a, pools, n_pools, std::max(1, book->n_pages / 2), book_of(book), plan.map, st);
  return e != cudaSuccess ? cuda_err(e, "page copy launch") : record_ok();
}

int gemma_kv_pages_copy(const gemma_page_pool* pools, int n_pools, int n_pages, int page_size, const int32_t* src,
                        const int32_t* dst, int n_copies, void* stream) {
  if (page_size <= 0 || page_size % 128)
    return err(GEMMA_ERR_INVALID_ARG, "page_size must be a positive multiple of 128");
  if (n_pages <= 0 || n_copies < 0) return err(GEMMA_ERR_INVALID_ARG, "n_pages must be positive, n_copies not negative");
  const int rc = check_pools(pools, n_pools, page_size);
  if (rc) return rc;
  if (n_copies > n_pages) return err(GEMMA_ERR_INVALID_ARG, "more copies than pages: a destination is repeated");
  if (n_copies == 0 || n_pools == 0) return record_ok();
  if (!src || !dst || misaligned(src, 4) || misaligned(dst, 4))
    return err(GEMMA_ERR_INVALID_ARG, "src, dst: null or misaligned pointer");
  int* status = device_status();
  if (!status) return err(GEMMA_ERR_CUDA, "no CUDA device");
  CopyList a{};
  a.src = src;
  a.dst = dst;
  a.stride = 1;
  a.n_host = n_copies;
  a.n_pages = n_pages;
  a.ps = page_size;
  a.check = 1;
  a.status = status;
  const cudaError_t e =
      copy_pages(a, pools, n_pools, n_copies, Book{}, nullptr, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_err(e, "page copy launch") : record_ok();
}

}  // extern "C"
