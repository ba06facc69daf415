// pool_tiles.hpp -- the pool's rows as tiles of a grouped product: which tile a
// workgroup takes, which activation row a pool row reads, and the checks that
// the products' entry points share.
#pragma once
#include "../../include/moelora.h"
#include "checks.hpp"
#include "layer.hpp"

namespace moelora {

struct PoolArgs {
  int E, topk;
  int cap;  // rows of the pool
  uint32_t tok_mul;  // route / topk = route * tok_mul >> tok_shift
  int tok_shift;
  long a_rows;
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* row2r;
};

// Rows of expert e, none past the pool whatever its arrays hold.
__device__ __forceinline__ int rows_of(const PoolArgs& p, int e) {
  const int off = p.offsets[e];
  return off >= 0 && off < p.cap ? max(min(p.counts[e], p.cap - off), 0) : 0;
}
// The activation row of a route, -1: none (a_rows < 2^31).  No branches: loads
// of several routes stay together.
__device__ __forceinline__ int token_of(const PoolArgs& p, int route) {
  const int t = (int)((uint64_t)(uint32_t)route * p.tok_mul >> p.tok_shift);
  return (int)(route >= 0) & (int)(t < (int)p.a_rows) ? t : -1;
}

// Tile b of the pool cut into M tiles of TM rows that never cross experts,
// times nn N tiles: its expert, its index among the expert's M tiles and its
// N tile; false past the last.  Every lane of the wave calls it; the counts
// are summed here (E <= 512: at most eight rounds of a wave scan) rather than
// by a kernel of its own, which costs more than the scan.  Order as in
// group_tile: each XCD a contiguous range of (expert's M chunk, N tile, M
// tile), so that workgroups of one XCD share a weight panel in its L2.
constexpr int MAX_E = 512;
// Rows of a pool, at most: an expert's are rounded up to whole tiles (of 256 rows or
// fewer) in 32 bits.
constexpr int64_t MOST_ROWS = ((int64_t)1 << 31) - 256;
// More tiles than a pool can have: the sums stop there, so that no counts make
// them wrap.
__device__ __forceinline__ int most_tiles(const PoolArgs& p, int TM) { return p.cap / TM + p.E; }
__device__ __forceinline__ bool pool_tile(const PoolArgs& p, int TM, int b, int nn, int gm, int& e, int& m, int& nt) {
  const int lane = threadIdx.x & 63;
  const int most = most_tiles(p, TM);
  int cnt[MAX_E / 64], end[MAX_E / 64], total = 0;
#pragma unroll
  for (int q = 0; q < MAX_E / 64; ++q) {
    cnt[q] = 64 * q + lane < p.E ? (rows_of(p, 64 * q + lane) + TM - 1) / TM : 0;
    if (64 * q < p.E) {
      int x = cnt[q];
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o, 64);
        if (lane >= o) x = min(x + y, most);
      }
      end[q] = min(total + x, most);  // tiles up to and with this lane's expert
      total = __builtin_amdgcn_readlane(end[q], 63);
    }
  }
  if (b >= total * nn) return false;
  const int L = xcd_remap(b, total * nn);
  const int v = L / nn;
  bool found = false;
#pragma unroll
  for (int q = 0; q < MAX_E / 64; ++q) {
    if (64 * q >= p.E || found) continue;
    const unsigned long long past = __ballot(end[q] > v);
    if (past == 0) continue;
    found = true;
    const int l = __ffsll(past) - 1;
    const int n = __builtin_amdgcn_readlane(cnt[q], l), s = __builtin_amdgcn_readlane(end[q], l) - n;
    const int cs = s + gm * ((v - s) / gm);
    const int sz = s + n - cs < gm ? s + n - cs : gm;
    const int r = L - cs * nn;
    e = 64 * q + l;
    m = cs + r % sz - s;
    nt = r / sz;
  }
  return found;
}

// The pool's tiles of TM rows, in LDS: for each expert the number of tiles up
// to and with it, its rows and its first row.
struct PoolTable {
  int *end, *cnt, *off;
  int total;
};
template <int TM>
__device__ __forceinline__ void fill_table(const PoolArgs& p, PoolTable& t, char* at) {
  t.end = (int*)at;
  t.cnt = t.end + p.E;
  t.off = t.cnt + p.E;
  const int lane = threadIdx.x & 63;
  const int most = most_tiles(p, TM);
  int before = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {  // every wave walks all experts; wave 0 writes
    const int e = e0 + lane, c = e < p.E ? rows_of(p, e) : 0;
    int x = (c + TM - 1) / TM;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o, 64);
      if (lane >= o) x = min(x + y, most);
    }
    x = min(before + x, most);
    if (threadIdx.x < 64 && e < p.E) {
      t.end[e] = x;
      t.cnt[e] = c;
      t.off[e] = p.offsets[e];
    }
    before = __shfl(x, 63, 64);
  }
  t.total = __builtin_amdgcn_readfirstlane(before);
  __syncthreads();
}

// One tile of the pool's nn N tiles per M tile (order as in pool_tile).
struct PoolTile {
  int e, nt, nrows;
  long row0;
};
template <int TM>
__device__ __forceinline__ bool find_tile(const PoolTable& t, int E, int b, int nn, PoolTile& out) {
  if (b >= t.total * nn) return false;
  const int lane = threadIdx.x & 63;
  const int L = xcd_remap(b, t.total * nn);
  const int v = L / nn;
  int e = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const unsigned long long past = __ballot(e0 + lane < E && t.end[min(e0 + lane, E - 1)] > v);
    if (past != 0) {
      e = e0 + __ffsll(past) - 1;
      break;
    }
  }
  const int cnt = t.cnt[e], end = t.end[e], off = t.off[e];  // read together
  const int rows = __builtin_amdgcn_readfirstlane(cnt);
  const int n = (rows + TM - 1) / TM, s = __builtin_amdgcn_readfirstlane(end) - n;
  const int cs = s + TILE_GM * ((v - s) / TILE_GM);
  const int sz = s + n - cs < TILE_GM ? s + n - cs : TILE_GM;
  const int r = L - cs * nn, m = cs + r % sz - s;
  out.e = e;
  out.nt = r / sz;
  out.nrows = min(rows - m * TM, TM);
  out.row0 = (long)__builtin_amdgcn_readfirstlane(off) + (long)m * TM;
  return true;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline PoolArgs pool_args(int E, int topk, int64_t a_rows, const moe_pool* pool) {
  // floor(n / k) = floor(n m / 2^(31 + s)) for n < 2^31, with 2^s >= k the
  // smallest and m = ceil(2^(31 + s) / k) < 2^32: n (m k - 2^(31 + s)) < 2^(31 + s)
  const uint64_t k = topk > 0 ? (uint64_t)topk : 1;
  int sh = 31;
  while ((uint64_t)1 << (sh - 31) < k) ++sh;
  const uint32_t mul = (uint32_t)((((uint64_t)1 << sh) + k - 1) / k);
  return PoolArgs{E, topk, (int)pool->capacity, mul, sh, (long)a_rows, pool->counts, pool->offsets, pool->row_to_route};
}
// The routes of a pool of this capacity: build_pool allots BLOCK_M - 1 rows of
// padding to each of min(E, routes) experts.
inline int64_t pool_routes(const moe_pool* pool, int64_t E) {
  const int64_t bm = pool->block_m, cap = pool->capacity;
  return cap >= E * bm ? cap - E * (bm - 1) : (cap + bm - 1) / bm;
}
// Workgroups for at most `tiles` tiles: every kernel of the products walks on
// by its grid until the pool's tiles are done, so the grid is a matter of speed
// alone: as many as are resident, in whole rounds over the XCDs.
inline unsigned grid_of(int64_t tiles, int64_t most) { return (unsigned)(((tiles < most ? tiles : most) + 7) / 8 * 8); }
inline hipError_t device_cus(int& cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  return e;
}

}  // namespace moelora
