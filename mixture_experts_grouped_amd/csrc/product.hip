// product.hip -- expert products in bf16 on the pool's rows and the weight's
// gradient (include/moelora.h states the formulas).
#include "../../include/moelora.h"
#include "checks.hpp"
#include "engine2.hpp"
#include "lanes.hpp"
#include "rows_tile.hpp"

namespace moelora {
namespace {

constexpr int MAX_DIM = 65536;  // N and K: a tile's row offsets stay in 32 bits

struct WgradArgs : PoolArgs {
  int N, K, accumulate;
  const uint16_t* g;
  const uint16_t* a;
  void* out;
};

// dw_e = sum over e's rows of grad^T a on the stage stream: 256 columns n of grad
// (x) by 256 columns k of a (w), both K-outer, a stage 64 of the expert's rows.
// Gathered rows of a: a stage's token ids travel two stages ahead of its loads
// into a ring of LDS; each wave keeps its own copy, so that its own wait covers
// them.  The ids of a tile's first two stages have a place of their own, filled
// when the tile is found.
// 256 x 256 tiles for every size, each tile's rows one chain of stages.  98,304
// rows, 64 x 4096 x 4096 in bf16: 2,984 to 3,137 us by card, 1,050 to 1,100 TFLOP/s
// (matrix cores busy 53 % at 2.0 GHz: both operands come through transposing reads;
// rows of a already in the pool's order 5 % less; ids fetched a stage earlier: no
// change).  One token: 500 us for 2.1 GB of zeros and six experts' tiles, 4.2 TB/s
// (non-temporal stores 630).  40 x 520 x 1000 in fp32, added to: 37.6 us for 166 MB
// read and written, 480 tiles in two rounds over the CUs.  Where there are fewer
// tiles than CUs the others stand idle: 24,576 rows on one expert of 256 x 256 take
// 465 us on one CU (gathered 545), of 64 x 64 as long; 16 experts of 512 x 512 with
// 2,048 rows each 54 us on 64.
struct WgradTile {
  int e, m0, n0, n;  // expert, first column of grad and of a, rows
  long row0;
};
// FAR: an expert's ids may be more than the 2 GB that a descriptor spans, and each
// stage's have one of their own; 0.9 % slower at 98,304 rows (3,017 for 2,992 us),
// so it is a kernel by itself, for pools of 2^29 - 4 rows and more.
template <bool GATHER, bool FAR, class OUT>
struct Wgrad {
  using G = stream::Geo<256, 256, 4, 2, 2>;
  using Tile = WgradTile;
  static constexpr int NI = GATHER ? 1 : 0;
  static constexpr int INSTS = NI + 8, FIRST = NI + 6;
  static constexpr int RING = 4, IDS = G::END;                 // [RING][waves][64]
  static constexpr int HEAD = IDS + RING * G::NW * 256;        // [2][waves][64]
  static constexpr int LDS = HEAD + 2 * G::NW * 256;
  static_assert(LDS <= 160 * 1024, "LDS");

  const WgradArgs& p;
  char* smem;
  int b, nm, nn, lane, wv, wm, wn;
  int sx;  // LDS offset of the wave's half of x
  stream::ColFrags<64> fx, fw;
  // the tile aimed at
  const char *gx, *gw;
  const char* gi;  // FAR: the ids that the next stage's loads fetch
  stream::desc_t da, di;
  int n;
  uint32_t vx[2], vw[2], tok[2];

  __device__ __forceinline__ Wgrad(const WgradArgs& args, char* sm) : p(args), smem(sm) {
    lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wv / G::WN;
    wn = wv % G::WN;
    b = blockIdx.x - gridDim.x;
    nm = (p.N + G::TM - 1) / G::TM;
    nn = (p.K + G::TN - 1) / G::TN;
    fx.init(lane, (wm & 1) * 64);
    fw.init(lane, wn * 64);
    sx = (wm >> 1) * 16384;
  }
  // The following tile.  Tiles of one expert are consecutive, in chunks of
  // TILE_GM of n, all k of a chunk, n fastest; each XCD walks a contiguous range.
  __device__ __forceinline__ bool next(Tile& t) {
    const int per = nm * nn, total = p.E * per;
    while (true) {
      b += gridDim.x;
      if (b >= total) return false;
      const int L = xcd_remap(b, total), e = L / per, r = L % per;
      const int cs = r / (TILE_GM * nn) * TILE_GM, sz = min(nm - cs, TILE_GM), q = r - cs * nn;
      int rows = __builtin_amdgcn_readfirstlane(rows_of(p, e));
      const long row0 = rows > 0 ? __builtin_amdgcn_readfirstlane(p.offsets[e]) : 0;
      if (rows == 0 && p.accumulate) continue;
      if (!GATHER && p.a_rows - row0 < rows) rows = p.a_rows > row0 ? (int)(p.a_rows - row0) : 0;
      t = Tile{e, (cs + q % sz) * G::TM, q / sz * G::TN, rows, row0};
      if constexpr (GATHER) {
        const stream::desc_t d = stream::make_desc(p.row2r + row0, (uint64_t)rows * 4);
#pragma unroll
        for (int s = 0; s < 2; ++s)
          stream::load4(d, smem + HEAD + (s * G::NW + wv) * 256, 4u * (uint32_t)(64 * s + lane), 0);
      }
      return true;
    }
  }
  __device__ __forceinline__ bool first(Tile& t) {
    if (!next(t)) return false;
    v2::wait_vm<0>();
    return true;
  }
  __device__ __forceinline__ int stages(const Tile& t) const { return cmax((t.n + 63) / 64, G::NBUF); }

  __device__ __forceinline__ void aim(const Tile& t, bool any) {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    gx = stream::uniform(p.g + t.row0 * p.N);
    gw = GATHER ? (const char*)p.a : stream::uniform(p.a + t.row0 * p.K);
    n = (int)stream::uniform(any ? (uint32_t)t.n : 0u);
    if constexpr (GATHER) {
      da = stream::make_desc(p.a, any ? (uint64_t)p.a_rows * p.K * 2 : 0);
      if constexpr (FAR)
        gi = stream::uniform(p.row2r + t.row0 + 128);
      else
        di = stream::make_desc(p.row2r + t.row0, (uint64_t)n * 4);
    }
    const int kr = 4 * wv + (l >> 4), c = 8 * ((l & 15) ^ stream::t_swz(kr));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cx = t.m0 + c + 128 * h, cw = t.n0 + c + (c >= 64 ? 64 : 0) + 64 * h;
      vx[h] = cx < p.N ? (uint32_t)kr * (uint32_t)p.N * 2u + 2u * (uint32_t)cx : OFF_NONE;
      vw[h] = cw < p.K ? (GATHER ? 0u : (uint32_t)kr * (uint32_t)p.K * 2u) + 2u * (uint32_t)cw : OFF_NONE;
    }
  }
  __device__ __forceinline__ void fill(int) {}
  __device__ __forceinline__ void begin() {}
  __device__ __forceinline__ void turn() {}

  // rows 64 s .. of an operand, as far as there are any
  __device__ __forceinline__ stream::desc_t rows(const char* base, int s, int ld) const {
    const int left = min(max(n - 64 * s, 0), 64);
    return stream::make_desc(base + (long)(64 * s) * ld * 2, (uint64_t)left * ld * 2);
  }
  __device__ __forceinline__ void issue(int s, int g, int i) {
    char* st = smem + g * G::STAGE;
    if (i < NI) {
      // the ids of stage s + 2, and the tokens of this one
      const int l = threadIdx.x & 63;
      char* to = smem + IDS + ((s & (RING - 1)) * G::NW + wv) * 256;
      if constexpr (FAR) {
        stream::load4(stream::make_desc(gi, 4u * (uint32_t)min(max(n - 64 * s - 128, 0), 64)), to, 4u * (uint32_t)l, 0);
        gi += 256;
      } else {
        stream::load4(di, to, 4u * (uint32_t)(64 * (s + 2) + l), 0);
      }
      const char* from = smem + (s < 2 ? HEAD + (s * G::NW + wv) * 256 : IDS + (((s - 2) & (RING - 1)) * G::NW + wv) * 256);
      const int left = n - 64 * s;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int kr = 4 * wv + (l >> 4) + 32 * q;
        const int t = token_of(p, *(const int*)(from + 4 * kr));
        tok[q] = kr < left && t >= 0 ? (uint32_t)t * (uint32_t)p.K * 2u : OFF_NONE;
      }
      return;
    }
    const int q = (i - NI) & 3, h = q >> 1, r = 32 * (q & 1);
    if (i - NI < 4) {
      stream::load16(rows(gx, s, p.N), st + 16384 * h + 1024 * (wv + 8 * (q & 1)), vx[h], (uint32_t)r * (uint32_t)p.N * 2u);
    } else {
      char* to = st + G::X_BYTES + 16384 * h + 1024 * (wv + 8 * (q & 1));
      if constexpr (GATHER) {
        const uint32_t t = tok[q & 1];
        stream::load16(da, to, (t | vw[h]) & OFF_NONE ? OFF_NONE : t + vw[h], 0);
      } else {
        stream::load16(rows(gw, s, p.K), to, vw[h], (uint32_t)r * (uint32_t)p.K * 2u);
      }
    }
  }
  __device__ __forceinline__ stream::Frag x(const char* buf, int j) const { return fx.get(buf + sx, j); }
  __device__ __forceinline__ stream::Frag w(const char* buf, int i) const { return fw.get(buf + G::X_BYTES, i); }
  template <int H>
  __device__ __forceinline__ void mma(const stream::Frag& w, const stream::Frag& x, f32x4& acc) const {
    acc = mma_bf16(H ? w.hi : w.lo, H ? x.hi : x.lo, acc);
  }

  // A lane holds four neighbouring k of a row n for each block; bf16: of two
  // blocks, rows of 16 lanes trade so that it holds eight of one.
  __device__ __forceinline__ void store(const Tile& t, const f32x4 (&acc)[G::FN][G::FM]) const {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int fr = l & 15, fc = l >> 4;
    const int live = min(p.N - t.m0, G::TM);
    OUT* base = (OUT*)p.out + ((long)t.e * p.N + t.m0) * p.K + t.n0;
    // less what the columns before n0 take: the last row ends there
    const rsrc_t ro = make_rsrc(base, ((uint64_t)live * p.K - t.n0) * sizeof(OUT));
    // what a row of blocks is added to is loaded together: one after another, each
    // waited for before its store, the loads took most of a short tile's time
    constexpr int ADDS = sizeof(OUT) == 4 ? G::FN : G::FN / 2;  // 16-byte pieces of a lane and row of blocks
#pragma unroll
    for (int j = 0; j < G::FM; ++j) {
      const int r = (wm * G::FM + j) * 16 + fr;
      auto place = [&](int q) {
        const int c = sizeof(OUT) == 4 ? (wn * G::FN + q) * 16 + 4 * fc : (wn * G::FN + 2 * q + (fc & 1)) * 16 + 8 * (fc >> 1);
        return r < live && t.n0 + c < p.K ? ((uint32_t)r * (uint32_t)p.K + (uint32_t)c) * (uint32_t)sizeof(OUT) : OFF_NONE;
      };
      u32x4 old[ADDS];
      if (p.accumulate) {
#pragma unroll
        for (int q = 0; q < ADDS; ++q) old[q] = bload(ro, place(q));
      }
#pragma unroll
      for (int q = 0; q < ADDS; ++q) {
        u32x4 w;
        if constexpr (sizeof(OUT) == 4) {
          f32x4 v = acc[q][j];
          if (p.accumulate) v += __builtin_bit_cast(f32x4, old[q]);
          w = __builtin_bit_cast(u32x4, v);
        } else if (p.accumulate) {  // in fp32 before the one rounding
          const int i = 2 * q;
          float o[8];
          widen8(old[q], o);
          f32x4 lo, hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][e]), __float_as_uint(acc[i + 1][j][e]), false, false);
            lo[e] = __uint_as_float(s[0]) + o[e];
            hi[e] = __uint_as_float(s[1]) + o[4 + e];
          }
          w = u32x4{pack2(lo[0], lo[1]), pack2(lo[2], lo[3]), pack2(hi[0], hi[1]), pack2(hi[2], hi[3])};
        } else {
          const int i = 2 * q;
          const auto lo = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][0], acc[i][j][1]),
                                                           pack2(acc[i + 1][j][0], acc[i + 1][j][1]), false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][2], acc[i][j][3]),
                                                           pack2(acc[i + 1][j][2], acc[i + 1][j][3]), false, false);
          w = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
        __builtin_amdgcn_raw_buffer_store_b128(w, ro, (int)place(q), 0, 0);
      }
    }
  }
};

template <bool GATHER, bool FAR, class OUT>
__global__ __launch_bounds__(512) void k_weight_grad(WgradArgs p) {
  extern __shared__ __align__(16) char smem[];
  Wgrad<GATHER, FAR, OUT> t(p, smem);
  WgradTile cur{};
  if (!t.first(cur)) return;
  stream::run(t, cur, smem);
}

template <bool GATHER, bool FAR, class OUT>
hipError_t launch_wgrad(const WgradArgs& p, int64_t tiles, int cus, hipStream_t st) {
  static PerDeviceOnce once;
  using W = Wgrad<GATHER, FAR, OUT>;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_weight_grad<GATHER, FAR, OUT>, W::LDS);
    return ai.err;
  });
  if (e != hipSuccess) return e;
  MOE_LAUNCH_AS("k_weight_grad", (k_weight_grad<GATHER, FAR, OUT>), dim3(grid_of(tiles, cus)), dim3(512), W::LDS, st, p);
  return hipGetLastError();
}
template <class OUT>
hipError_t launch_wgrad(const WgradArgs& p, int64_t tiles, int cus, hipStream_t st) {
  if (p.topk == 0) return launch_wgrad<false, false, OUT>(p, tiles, cus, st);
  return (uint64_t)p.cap * 4 < RSRC_MAX ? launch_wgrad<true, false, OUT>(p, tiles, cus, st)
                                        : launch_wgrad<true, true, OUT>(p, tiles, cus, st);
}

moe_status check_common(const moe_expert_desc* d, const moe_pool* pool) {
  if (d == nullptr || pool == nullptr) return MOE_ERR_INVALID;
  if (d->E < 1 || d->N < 1 || d->K < 1) return MOE_ERR_INVALID;
  if (d->E > MAX_E || d->N % 8 != 0 || d->K % 8 != 0 || d->N > MAX_DIM || d->K > MAX_DIM ||
      (int64_t)d->N * d->K >= (int64_t)1 << 30)
    return MOE_ERR_UNSUPPORTED;
  if (d->topk < 0 || d->a_rows < 1 || pool->capacity < 1 || pool->block_m < 1) return MOE_ERR_INVALID;
  if (pool->capacity > MOST_ROWS || d->a_rows >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  if (d->topk > 0 && d->a_rows * d->K >= (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;  // one buffer descriptor
  if (!aligned(pool->counts, 4) || !aligned(pool->offsets, 4) || !aligned(pool->row_to_route, 4))
    return MOE_ERR_INVALID;
  return MOE_OK;
}
bool overlaps_any(Range out, const Range* in, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(out, in[i])) return true;
  return false;
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

moe_status moe_expert_product(const moe_expert_desc* d, const moe_pool* pool, const void* a, const void* w, void* out,
                              void* stream) {
  const moe_status s = check_common(d, pool);
  if (s != MOE_OK) return s;
  if (d->transposed != 0 && d->transposed != 1) return MOE_ERR_INVALID;
  // tile indices of the smallest tiles are 32 bits
  if ((pool->capacity / FEW_ROWS + d->E) * ((d->N + 15) / 16) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(a) || !aligned16(w) || !aligned16(out)) return MOE_ERR_INVALID;
  const Range in[] = {rng(a, (size_t)d->a_rows * d->K * 2), rng(w, (size_t)d->E * d->N * d->K * 2),
                      rng(pool->counts, (size_t)d->E * 4), rng(pool->offsets, (size_t)d->E * 4 + 4),
                      rng(pool->row_to_route, (size_t)pool->capacity * 4)};
  if (overlaps_any(rng(out, (size_t)pool->capacity * d->N * 2), in, 5)) return MOE_ERR_INVALID;
  int cus = 0;
  hipError_t e = device_cus(cus);
  if (e != hipSuccess) return MOE_ERR_HIP;
  const RowsArgs p{pool_args(d->E, d->topk, d->a_rows, pool), d->N, d->K, (const uint8_t*)a, (const uint8_t*)w,
                   nullptr, nullptr, (uint16_t*)out};
  const int64_t routes = pool_routes(pool, d->E), live = routes < d->E ? routes : d->E;
  auto tiles = [&](int tm) { return routes / tm + live; };
  const hipStream_t st = (hipStream_t)stream;
  if (d->transposed) {
    if (pick(p, Costs{0.0, 4.0, 0.4, 0.9, 9.0, 1.2, 1.65}, routes, cus, 2 * d->K) == Pick::mid)
      e = launch_rows_tile<Kind::bf16_t, GeoM>("k_product_t_tile64", p, tiles(GeoM::TM), 2 * cus, st);
    else
      e = launch_rows_tile<Kind::bf16_t, GeoL>("k_product_t_tile256", p, tiles(GeoL::TM), cus, st);
  } else {
    switch (pick(p, Costs{27000.0, 4.0, 0.31, 0.84, 9.0, 1.0, 1.65}, routes, cus, 2 * d->K)) {
      case Pick::few: e = launch_rows_few<Kind::bf16>("k_product_few", p, tiles(FEW_ROWS), 8 * cus, st); break;
      case Pick::mid: e = launch_rows_tile<Kind::bf16, GeoM>("k_product_tile64", p, tiles(GeoM::TM), 2 * cus, st); break;
      case Pick::large: e = launch_rows_tile<Kind::bf16, GeoL>("k_product_tile256", p, tiles(GeoL::TM), cus, st); break;
    }
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_expert_weight_grad(const moe_expert_desc* d, const moe_pool* pool, const void* grad, const void* a,
                                  void* dw, void* stream) {
  const moe_status s = check_common(d, pool);
  if (s != MOE_OK) return s;
  if (d->out_type != MOE_TYPE_F32 && d->out_type != MOE_TYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (d->accumulate != 0 && d->accumulate != 1) return MOE_ERR_INVALID;
  if (!aligned16(grad) || !aligned16(a) || !aligned16(dw)) return MOE_ERR_INVALID;
  const size_t size = d->out_type == MOE_TYPE_F32 ? 4 : 2;
  const Range in[] = {rng(grad, (size_t)pool->capacity * d->N * 2), rng(a, (size_t)d->a_rows * d->K * 2),
                      rng(pool->counts, (size_t)d->E * 4), rng(pool->offsets, (size_t)d->E * 4 + 4),
                      rng(pool->row_to_route, (size_t)pool->capacity * 4)};
  if (overlaps_any(rng(dw, (size_t)d->E * d->N * d->K * size), in, 5)) return MOE_ERR_INVALID;
  int cus = 0;
  hipError_t e = device_cus(cus);
  if (e != hipSuccess) return MOE_ERR_HIP;
  const WgradArgs p{pool_args(d->E, d->topk, d->a_rows, pool), d->N, d->K, d->accumulate, (const uint16_t*)grad,
                    (const uint16_t*)a, dw};
  const int64_t tiles = (int64_t)d->E * ((d->N + 255) / 256) * ((d->K + 255) / 256);
  const hipStream_t st = (hipStream_t)stream;
  e = d->out_type == MOE_TYPE_F32 ? launch_wgrad<float>(p, tiles, cus, st) : launch_wgrad<uint16_t>(p, tiles, cus, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
