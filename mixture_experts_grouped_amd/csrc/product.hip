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

template <class G>
__device__ __forceinline__ void clear(f32x16 (&acc)[G::NB][G::MB]) {
#pragma unroll
  for (int i = 0; i < G::NB; ++i)
#pragma unroll
    for (int j = 0; j < G::MB; ++j) acc[i][j] = f32x16{};
}

// T tile of the rows of an expert, columns c0 .. of a tensor with ldb bytes a
// row: pool rows (consecutive, the descriptor based at each stage's first row),
// or the tokens of the routes.  Rows past the expert's and columns past the
// tensor's read zero.
template <int R, bool GATHER>
struct RowTile {
  static constexpr int CPR = R / 8, RPI = 64 / CPR, NW = 8, NJ = 64 / (NW * RPI);
  const char* base;
  uint32_t ldb;
  int c0, ncols;
  __device__ __forceinline__ void issue(const PoolArgs& p, long row0, int n, int k0, char* tile) const {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), L = threadIdx.x & 63;
    const int left = n - k0;
    const rsrc_t rs = GATHER ? make_rsrc(base, (uint64_t)p.a_rows * ldb)
                             : make_rsrc(base + (row0 + k0) * (long)ldb, (uint64_t)(left > 0 ? left : 0) * ldb);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int kr = RPI * (w + NW * j) + L / CPR;
      const int c = 8 * ((L % CPR) ^ v2::tswz(kr));
      bool ok = c < ncols && kr < left;
      uint32_t r = (uint32_t)kr;
      if constexpr (GATHER) {
        const int t = ok ? token_of(p, p.row2r[row0 + k0 + kr]) : -1;
        ok = t >= 0;
        r = (uint32_t)t;
      }
      v2::lds_load16(rs, tile + 1024 * (w + NW * j), ok ? r * ldb + 2u * (uint32_t)(c0 + c) : OFF_NONE);
    }
  }
};

template <class G, bool GATHER>
struct WgradLoad {
  using LM = RowTile<G::TM, false>;
  using LN = RowTile<G::TN, GATHER>;
  static constexpr int INSTS = LM::NJ + LN::NJ;
  const PoolArgs* p;
  long row0;
  int n;
  LM m;
  LN a;
  __device__ void issue(int s, char* sM, char* sN) {
    m.issue(*p, row0, n, s * G::KT, sM);
    a.issue(*p, row0, n, s * G::KT, sN);
  }
};

// dw_e: 256 x 256 tiles, both operands K-outer.
template <bool GATHER, class OUT>
__global__ __launch_bounds__(512) void k_weight_grad(WgradArgs p) {
  extern __shared__ __align__(16) char smem[];
  using G = v2::Geo2<4, 2, 2, 4, true, true, 64>;
  const int nn = (p.K + G::TN - 1) / G::TN, per = (p.N + G::TM - 1) / G::TM * nn;
  for (int b = blockIdx.x; b < p.E * per; b += gridDim.x) {
    const int t = xcd_remap(b, p.E * per);
    const int e = t / per, m0 = (t % per) / nn * G::TM, n0 = (t % per) % nn * G::TN;
    const int n = rows_of(p, e);
    if (n == 0 && p.accumulate) continue;
    const long row0 = n > 0 ? p.offsets[e] : 0;
    WgradLoad<G, GATHER> ld;
    ld.p = &p;
    ld.row0 = row0;
    // pool rows past the tensor's: none are read
    const long have = p.a_rows - row0;
    ld.n = GATHER || have >= n ? n : (have > 0 ? (int)have : 0);
    ld.m.base = (const char*)p.g;
    ld.m.ldb = (uint32_t)p.N * 2u;
    ld.m.c0 = m0;
    ld.m.ncols = p.N - m0;
    ld.a.base = (const char*)p.a;
    ld.a.ldb = (uint32_t)p.K * 2u;
    ld.a.c0 = n0;
    ld.a.ncols = p.K - n0;
    f32x16 acc[G::NB][G::MB];
    clear<G>(acc);
    v2::run_stages2<G, 0>(ld, (ld.n + G::KT - 1) / G::KT, acc, smem);
    Epi<G> ep;
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb) {
      const int r = m0 + ep.row(mb);
      if (r >= p.N) continue;
      OUT* o = (OUT*)p.out + ((long)e * p.N + r) * p.K;
#pragma unroll
      for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = n0 + ep.col(nb, g);
          if (c >= p.K) continue;
          f32x4 v = {acc[nb][mb][4 * g], acc[nb][mb][4 * g + 1], acc[nb][mb][4 * g + 2], acc[nb][mb][4 * g + 3]};
          if constexpr (sizeof(OUT) == 4) {
            if (p.accumulate) v += *(const f32x4*)(o + c);
            *(f32x4*)(o + c) = v;
          } else {
            if (p.accumulate) {
              const u32x2 w = *(const u32x2*)(o + c);
              v += f32x4{bf2f(w[0] & 0xffffu), bf2f(w[0] >> 16), bf2f(w[1] & 0xffffu), bf2f(w[1] >> 16)};
            }
            *(u32x2*)(o + c) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
          }
        }
    }
  }
}

constexpr int TILE_LDS = 2 * (256 + 256) * 128;

template <class Kern, class Args>
hipError_t launch(const char* name, Kern kern, PerDeviceOnce& once, int64_t tiles, int cus, const Args& p, hipStream_t st) {
  const hipError_t e = once.run([&] {
    AttrInit ai;
    ai.lds((const void*)kern, TILE_LDS);
    return ai.err;
  });
  if (e != hipSuccess) return e;
  MOE_LAUNCH_AS(name, kern, dim3(grid_of(tiles, cus)), dim3(512), TILE_LDS, st, p);
  return hipGetLastError();
}

moe_status check_common(const moe_expert_desc* d, const moe_pool* pool) {
  if (d == nullptr || pool == nullptr) return MOE_ERR_INVALID;
  if (d->E < 1 || d->N < 1 || d->K < 1) return MOE_ERR_INVALID;
  if (d->E > MAX_E || d->N % 8 != 0 || d->K % 8 != 0 || d->N > MAX_DIM || d->K > MAX_DIM ||
      (int64_t)d->N * d->K >= (int64_t)1 << 30)
    return MOE_ERR_UNSUPPORTED;
  if (d->topk < 0 || d->a_rows < 1 || pool->capacity < 1 || pool->block_m < 1) return MOE_ERR_INVALID;
  if (pool->capacity >= (int64_t)1 << 31 || d->a_rows >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  // tile indices of the smallest tiles are 32 bits
  if ((pool->capacity / 16 + d->E) * ((d->N + 15) / 16) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
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
  constexpr Costs costs{20000.0, 0.84, 0.5, 2.1, 1.35};
  if (d->transposed) {
    if (pick(p, costs, routes, cus, false) == Pick::mid)
      e = launch_rows_tile<Kind::bf16_t, GeoM>("k_product_t_tile64", p, tiles(GeoM::TM), 2 * cus, st);
    else
      e = launch_rows_tile<Kind::bf16_t, GeoL>("k_product_t_tile256", p, tiles(GeoL::TM), cus, st);
  } else {
    switch (pick(p, costs, routes, cus, true)) {
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
  static PerDeviceOnce once[4];
  const bool f32 = d->out_type == MOE_TYPE_F32;
  if (d->topk > 0)
    e = f32 ? launch("k_weight_grad", k_weight_grad<true, float>, once[0], tiles, cus, p, st)
            : launch("k_weight_grad", k_weight_grad<true, uint16_t>, once[1], tiles, cus, p, st);
  else
    e = f32 ? launch("k_weight_grad", k_weight_grad<false, float>, once[2], tiles, cus, p, st)
            : launch("k_weight_grad", k_weight_grad<false, uint16_t>, once[3], tiles, cus, p, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
