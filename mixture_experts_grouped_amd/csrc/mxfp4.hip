// mxfp4.hip -- rows and weights in microscaled 4-bit floating point (e2m1 codes,
// one e8m0 exponent per 32), and the expert products on them
// (include/moelora.h states the formulas).
#include "../../include/moelora.h"
#include "checks.hpp"
#include "engine2.hpp"
#include "lanes.hpp"
#include "rows_tile.hpp"

namespace moelora {
namespace {

constexpr int MAX_DIM = 65536;

// ---------------------------------------------------------------------------
// quantisers
// ---------------------------------------------------------------------------
// The block's held exponent (plus 127) from its largest magnitude's bits, 255 with
// a NaN or an infinity, and the scale that it stands for (2^(e - 127)).
__device__ __forceinline__ uint32_t block_exponent(uint32_t mag_max, float& scale) {
  const int field = (int)(mag_max >> 23);
  const uint32_t e = field == 255 ? 255u : field > 2 ? (uint32_t)(field - 2) : 0u;  // max|x| < 2^-125: the smallest exponent
  scale = e == 255 ? 1.0f : v2::e8m0_value(e);
  return e;
}
// Eight values over the scale to codes of e2m1 (v_cvt_scalef32_pk_fp4: to nearest,
// ties to even, what is beyond 6 to 6; over a million values of all binades and
// scales, ties among them, every code was the formula's but for -0, which becomes
// +0 here: a nibble's magnitude plus 7 carries into bit 3 where it is not zero).
__device__ __forceinline__ uint32_t no_minus_zero(uint32_t w) {
  return w & (0x77777777u | ((w & 0x77777777u) + 0x77777777u));
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return no_minus_zero(w);
}
__device__ __forceinline__ uint32_t codes8(u32x4 v, float scale) {  // bf16 pairs
  auto pair = [](uint32_t x) { return __builtin_bit_cast(bf16x2_t, x); };
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(v[0]), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(v[1]), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(v[2]), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(v[3]), scale, 3);
  return no_minus_zero(w);
}
// The largest of four neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Eight columns a thread, a block of 32 in four lanes.  Bound by memory: 16,384 x
// 4096 in 31.8 us, 5.3 TB/s (two groups of eight a thread: no change); gated 98,304 x
// 2048: SwiGLU 160 us, 5.7 TB/s, GEGLU 184 us (its erf's vector instructions).
template <int ACT>
__global__ __launch_bounds__(256) void k_mxfp4_rows(const uint16_t* __restrict__ src, long n8, int K8,
                                                    uint32_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;  // whole blocks: K % 128 == 0
  uint32_t m = 0;
  float scale;
  if constexpr (ACT < 0) {
    const u32x4 x = ((const u32x4*)src)[i];
#pragma unroll
    for (int q = 0; q < 4; ++q) m = max(m, max((x[q] << 16) & 0x7FFFFFFFu, x[q] & 0x7FFF0000u));
    const uint32_t e = block_exponent(quad_max(m), scale);
    codes[i] = codes8(x, scale);
    if ((threadIdx.x & 3) == 0) exps[i >> 2] = (uint8_t)e;
  } else {
    const long row = i / K8, c = i - row * K8;
    const u32x4* p = (const u32x4*)src + row * 2 * K8 + c;
    float v[8], u[8];
    widen8(p[0], v);
    widen8(p[K8], u);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = (ACT == MOE_ACT_SWIGLU ? v[q] * sigmoidf_(v[q]) : v[q] * norm_cdf_rel(v[q])) * u[q];
      m = max(m, mag(v[q]));
    }
    const uint32_t e = block_exponent(quad_max(m), scale);
    codes[i] = codes8(v, scale);
    if ((threadIdx.x & 3) == 0) exps[i >> 2] = (uint8_t)e;
  }
}

// The transposed weight's codes: a workgroup takes 128 rows n x 32 columns k of
// one expert through LDS; thread t quantises block t / 32 (32 rows n) of column t % 32.
__global__ __launch_bounds__(128) void k_mxfp4_weight_t(const uint16_t* __restrict__ W, int N, int K,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  __shared__ uint16_t tile[128][33];
  const long e = blockIdx.z, n0 = (long)blockIdx.y * 128, k0 = (long)blockIdx.x * 32;
  for (int i = threadIdx.x; i < 128 * 32; i += 128) tile[i >> 5][i & 31] = W[(e * N + n0 + (i >> 5)) * K + k0 + (i & 31)];
  __syncthreads();
  const int k = threadIdx.x & 31, b = threadIdx.x >> 5;
  float v[32];
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    v[q] = bf2f(tile[32 * b + q][k]);
    m = max(m, mag(v[q]));
  }
  float scale;
  const uint32_t x = block_exponent(m, scale);
  u32x4 w;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float(&v8)[8] = *(const float(*)[8])(v + 8 * c);
    w[c] = codes8(v8, scale);
  }
  const long row = e * K + k0 + k;
  *(u32x4*)(codes + row * (N / 2) + (n0 + 32 * b) / 2) = w;
  exps[row * (N / 32) + n0 / 32 + b] = (uint8_t)x;
}

// Eight values a thread; 16,384 x 4096 in 25.2 us, 6.7 TB/s.
__global__ __launch_bounds__(256) void k_mxfp4_values(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                                                      long n8, u32x4* __restrict__ out) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint32_t w = codes[i], e = exps[i >> 2];
  u32x4 o = v2::fp4x8_bf16(w, v2::e8m0_value(e));
  if (e == 255) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  out[i] = o;
}

moe_status check_weight(int32_t E, int32_t N, int32_t K, int32_t nstep) {
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID;
  if (E > MAX_E || N % nstep != 0 || K % 128 != 0 || N > MAX_DIM || K > MAX_DIM || (int64_t)N * K >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
template <int ACT>
hipError_t launch_rows(const void* src, long n8, int K8, void* codes, void* exps, hipStream_t st) {
  MOE_LAUNCH_AS("k_mxfp4_rows", k_mxfp4_rows<ACT>, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, st,
                (const uint16_t*)src, n8, K8, (uint32_t*)codes, (uint8_t*)exps);
  return hipGetLastError();
}
// a launch holds fewer than 2^32 threads, eight columns each, in whole workgroups of 256
constexpr int64_t MOST_VALUES = ((int64_t)1 << 35) - 2048;
bool any_overlap(const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(r[i], r[j])) return true;
  return false;
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

moe_status moe_mxfp4_quantize_rows(const void* src, int64_t rows, int32_t K, int32_t act, void* codes,
                                   void* exponents, void* stream) {
  if (rows < 0 || K < 1) return MOE_ERR_INVALID;
  if (K % 128 != 0 || K > MAX_DIM || rows >= (int64_t)1 << 31 || rows * K > MOST_VALUES) return MOE_ERR_UNSUPPORTED;
  if (act != MOE_FP8_PLAIN && act != MOE_ACT_SWIGLU && act != MOE_ACT_GEGLU) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!aligned16(src) || !aligned16(codes) || !aligned(exponents, 4)) return MOE_ERR_INVALID;
  const size_t n = (size_t)rows * K;
  const Range r[] = {rng(src, n * (act == MOE_FP8_PLAIN ? 2 : 4)), rng(codes, n / 2), rng(exponents, n / 32)};
  if (any_overlap(r, 3)) return MOE_ERR_INVALID;
  const hipStream_t st = (hipStream_t)stream;
  const hipError_t e = act == MOE_FP8_PLAIN    ? launch_rows<MOE_FP8_PLAIN>(src, (long)(n / 8), K / 8, codes, exponents, st)
                       : act == MOE_ACT_SWIGLU ? launch_rows<MOE_ACT_SWIGLU>(src, (long)(n / 8), K / 8, codes, exponents, st)
                                               : launch_rows<MOE_ACT_GEGLU>(src, (long)(n / 8), K / 8, codes, exponents, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_mxfp4_quantize_weight(const void* W, int32_t E, int32_t N, int32_t K, void* codes, void* exponents,
                                     void* codes_t, void* exponents_t, void* stream) {
  const moe_status s = check_weight(E, N, K, 128);
  if (s != MOE_OK) return s;
  const size_t n = (size_t)E * N * K;
  if (n > (size_t)MOST_VALUES) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(W) || !aligned16(codes) || !aligned(exponents, 4)) return MOE_ERR_INVALID;
  if ((codes_t != nullptr) != (exponents_t != nullptr)) return MOE_ERR_INVALID;
  if (codes_t != nullptr && (!aligned16(codes_t) || !aligned(exponents_t, 4))) return MOE_ERR_INVALID;
  const Range r[] = {rng(W, 2 * n), rng(codes, n / 2), rng(exponents, n / 32), rng(codes_t, n / 2), rng(exponents_t, n / 32)};
  if (any_overlap(r, 5)) return MOE_ERR_INVALID;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = launch_rows<MOE_FP8_PLAIN>(W, (long)(n / 8), K / 8, codes, exponents, st);
  if (e == hipSuccess && codes_t != nullptr) {
    MOE_LAUNCH(k_mxfp4_weight_t, dim3(K / 32, N / 128, E), dim3(128), 0, st, (const uint16_t*)W, N, K, (uint8_t*)codes_t,
               (uint8_t*)exponents_t);
    e = hipGetLastError();
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_mxfp4_dequantize(const void* codes, const void* exponents, int64_t rows, int32_t K, void* out,
                                void* stream) {
  if (rows < 0 || K < 1) return MOE_ERR_INVALID;
  if (K % 128 != 0 || K > MAX_DIM || rows >= (int64_t)1 << 31 || rows * K > MOST_VALUES) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!aligned16(codes) || !aligned(exponents, 4) || !aligned16(out)) return MOE_ERR_INVALID;
  const size_t n = (size_t)rows * K;
  const Range o = rng(out, 2 * n);
  if (overlap(o, rng(codes, n / 2)) || overlap(o, rng(exponents, n / 32))) return MOE_ERR_INVALID;
  const long n8 = (long)(n / 8);
  MOE_LAUNCH(k_mxfp4_values, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, (hipStream_t)stream, (const uint32_t*)codes,
             (const uint8_t*)exponents, n8, (u32x4*)out);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_mxfp4_product(const moe_mxfp4_desc* d, const moe_pool* pool, const void* a, const void* a_exponents,
                             const void* w, const void* w_exponents, void* out, void* stream) {
  if (d == nullptr || pool == nullptr) return MOE_ERR_INVALID;
  const moe_status s = check_weight(d->E, d->N, d->K, 32);
  if (s != MOE_OK) return s;
  if (d->topk < 0 || d->a_rows < 1 || pool->capacity < 1 || pool->block_m < 1) return MOE_ERR_INVALID;
  if (pool->capacity > MOST_ROWS || d->a_rows >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  // tile indices of the smallest tiles are 32 bits
  if ((pool->capacity / FEW_ROWS + d->E) * (d->N / 16) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  if (d->topk > 0 && d->a_rows * d->K >= (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;  // one buffer descriptor
  if (!aligned(pool->counts, 4) || !aligned(pool->offsets, 4) || !aligned(pool->row_to_route, 4))
    return MOE_ERR_INVALID;
  if (!aligned16(a) || !aligned(a_exponents, 4) || !aligned16(w) || !aligned(w_exponents, 4) || !aligned16(out))
    return MOE_ERR_INVALID;
  const size_t na = (size_t)d->a_rows * d->K, nw = (size_t)d->E * d->N * d->K;
  const Range ro = rng(out, (size_t)pool->capacity * d->N * 2);
  const Range ins[] = {rng(a, na / 2), rng(a_exponents, na / 32), rng(w, nw / 2), rng(w_exponents, nw / 32),
                       rng(pool->counts, (size_t)d->E * 4), rng(pool->offsets, (size_t)d->E * 4 + 4),
                       rng(pool->row_to_route, (size_t)pool->capacity * 4)};
  for (const Range& r : ins)
    if (overlap(ro, r)) return MOE_ERR_INVALID;
  const RowsArgs p{pool_args(d->E, d->topk, d->a_rows, pool), d->N, d->K, (const uint8_t*)a, (const uint8_t*)w,
                   (const uint8_t*)a_exponents, (const uint8_t*)w_exponents, (uint16_t*)out};
  const int64_t routes = pool_routes(pool, d->E), live = routes < d->E ? routes : d->E;
  auto tiles = [&](int tm) { return routes / tm + live; };
  int cus = 0;
  hipError_t e = device_cus(cus);
  if (e != hipSuccess) return MOE_ERR_HIP;
  const hipStream_t st = (hipStream_t)stream;
  constexpr Kind KIND = Kind::mxfp4;
  switch (pick(p, Costs{21000.0, 4.0, 0.45, 1.15, 8.0, 1.2, 2.2}, routes, cus, d->K / 2)) {
    case Pick::few: e = launch_rows_few<KIND>("k_mxfp4_few", p, tiles(FEW_ROWS), 8 * cus, st); break;
    case Pick::mid: e = launch_rows_tile<KIND, GeoM>("k_mxfp4_tile64", p, tiles(GeoM::TM), 2 * cus, st); break;
    case Pick::large:
      e = d->K % 512 == 0 ? launch_rows_tile<Kind::mxfp4_pairs, GeoL>("k_mxfp4_tile256", p, tiles(GeoL::TM), cus, st)
                          : launch_rows_tile<KIND, GeoL>("k_mxfp4_tile256", p, tiles(GeoL::TM), cus, st);
      break;
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
