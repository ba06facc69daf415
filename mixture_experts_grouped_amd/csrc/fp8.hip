// fp8.hip -- expert products in e4m3 with one fp32 scale per block of 128, and
// the quantisers that make their operands (include/moelora.h states the
// formulas).
//
// One K block of 128 is one LDS stage of a tile row (128 bytes, the pitch of
// a bf16 row of 64 k, so the bf16 engine's direct-to-LDS loaders and their
// swizzle carry it) and one v_mfma_f32_16x16x128_f8f6f4 per 16 x 16 output
// block.  The block's product starts from zero and is added to the fp32
// accumulator times sa * sw: weights are the first operand, so a lane's four
// results belong to one activation row and the scale is one value per lane,
// and a wave's weight rows lie in one block of 128, so sw is one scalar.  The
// instruction's own block scales are powers of two only and stay unused.
#include "../../include/moelora.h"
#include "checks.hpp"
#include "engine2.hpp"
#include "lanes.hpp"
#include "layer.hpp"
#include "trace.hpp"

namespace moelora {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr float E4M3_MAX = 448.0f;
constexpr float TINY = 0x1p-100f;  // a block below it counts as zero (its reciprocal would overflow)

// ---------------------------------------------------------------------------
// quantisers
// ---------------------------------------------------------------------------
struct Block8 {
  float inv, scale;  // codes are e4m3(x * inv), a code stands for code * scale
};
__device__ __forceinline__ Block8 block_scale(uint32_t mag_max) {
  const float amax = __uint_as_float(mag_max);
  if (amax < TINY) return Block8{0.0f, 0.0f};
  return Block8{E4M3_MAX / amax, amax / E4M3_MAX};
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
}
__device__ __forceinline__ void widen8(u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[2 * c] = bf2f(w[c] & 0xffffu);
    v[2 * c + 1] = bf2f(w[c] >> 16);
  }
}

// Eight columns a thread, a block of 128 in one DPP row.  ACT < 0: src is
// [rows, K]; else [rows, 2K] = gate | up.
template <int ACT>
__global__ __launch_bounds__(256) void k_fp8_rows(const uint16_t* __restrict__ src, long n8, int K8,
                                                  uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;  // group of 8 columns
  if (i >= n8) return;                                   // whole blocks: K % 128 == 0
  float v[8];
  if constexpr (ACT < 0) {
    widen8(((const u32x4*)src)[i], v);
  } else {
    const long row = i / K8, c = i - row * K8;
    const u32x4* p = (const u32x4*)src + row * 2 * K8 + c;
    float u[8];
    widen8(p[0], v);
    widen8(p[K8], u);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = (ACT == MOE_ACT_SWIGLU ? v[q] * sigmoidf_(v[q]) : v[q] * norm_cdf(v[q])) * u[q];
  }
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, mag(v[q]));
  const Block8 b = block_scale(row_max(m));
  ((u32x2*)codes)[i] = u32x2{codes4(v[0] * b.inv, v[1] * b.inv, v[2] * b.inv, v[3] * b.inv),
                             codes4(v[4] * b.inv, v[5] * b.inv, v[6] * b.inv, v[7] * b.inv)};
  if ((threadIdx.x & 15) == 0) scales[i >> 4] = b.scale;
}

// One 128 x 128 block of one expert's weight a workgroup: thread t holds 64
// values (row t / 2, half t % 2).  The transposed codes go through LDS.
__global__ __launch_bounds__(256) void k_fp8_weight(const uint16_t* __restrict__ W, int N, int K,
                                                    uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                    uint8_t* __restrict__ codes_t, float* __restrict__ scales_t) {
  constexpr int PITCH = 128 + 4;
  __shared__ uint32_t red[4];
  __shared__ __align__(16) uint8_t tile[128 * PITCH];
  const int tid = threadIdx.x, r = tid >> 1, h = tid & 1;
  const int kb = blockIdx.x, nb = blockIdx.y;
  const long e = blockIdx.z;
  const long at = (e * N + nb * 128 + r) * K + kb * 128 + h * 64;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    widen8(*(const u32x4*)(W + at + 8 * c), v[c]);
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, mag(v[c][q]));
  }
  m = row_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
  const Block8 b = block_scale(max(max(red[0], red[1]), max(red[2], red[3])));
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    u32x4 w;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const float(&x)[8] = v[2 * c + d];
      w[2 * d] = codes4(x[0] * b.inv, x[1] * b.inv, x[2] * b.inv, x[3] * b.inv);
      w[2 * d + 1] = codes4(x[4] * b.inv, x[5] * b.inv, x[6] * b.inv, x[7] * b.inv);
    }
    *(u32x4*)(codes + at + 16 * c) = w;
    if (codes_t != nullptr)
#pragma unroll
      for (int d = 0; d < 4; ++d) *(uint32_t*)(tile + r * PITCH + h * 64 + 16 * c + 4 * d) = w[d];
  }
  if (tid == 0) scales[(e * (N / 128) + nb) * (K / 128) + kb] = b.scale;
  if (codes_t == nullptr) return;
  if (tid == 0) scales_t[(e * (K / 128) + kb) * (N / 128) + nb] = b.scale;
  __syncthreads();
  // thread t writes k-row t / 2, n columns 64 (t % 2) .. + 63
  const long out = (e * K + kb * 128 + r) * N + nb * 128 + h * 64;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    u32x4 w;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t x = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) x |= (uint32_t)tile[(h * 64 + 16 * c + 4 * d + q) * PITCH + r] << (8 * q);
      w[d] = x;
    }
    *(u32x4*)(codes_t + out + 16 * c) = w;
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
struct Fp8Args {
  int E, N, K, topk;
  long a_rows;
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* row2r;
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  uint16_t* out;
};

// Tile b of the pool cut into M tiles of TM rows that never cross experts,
// times nn N tiles: its expert, its index among the expert's M tiles and its
// N tile; false past the last.  Every lane of the wave calls it; the counts
// are summed here (E <= 512: at most eight rounds of a wave scan) rather than
// by a kernel of its own, which costs more than the scan.  Order as in
// group_tile: each XCD a contiguous range of (expert's M chunk, N tile, M
// tile), so that workgroups of one XCD share a weight panel in its L2.
__device__ __forceinline__ bool pool_tile(const Fp8Args& p, int TM, int b, int nn, int gm, int& e, int& m, int& nt) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int x = e0 + lane < p.E ? (p.counts[e0 + lane] + TM - 1) / TM : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    total += x;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  if (b >= total * nn) return false;
  const int L = xcd_remap(b, total * nn);
  const int v = L / nn;
  int before = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int c = e0 + lane < p.E ? (p.counts[e0 + lane] + TM - 1) / TM : 0;
    int x = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    const int end = before + x;  // tiles up to and with this lane's expert
    const unsigned long long past = __ballot(end > v);
    if (past != 0) {
      const int l = __ffsll(past) - 1;
      const int cnt = __shfl(c, l, 64), s = __shfl(end, l, 64) - cnt;
      e = __builtin_amdgcn_readfirstlane(e0 + l);
      const int cs = s + gm * ((v - s) / gm);
      const int sz = s + cnt - cs < gm ? s + cnt - cs : gm;
      const int r = L - cs * nn;
      m = __builtin_amdgcn_readfirstlane(cs + r % sz - s);
      nt = __builtin_amdgcn_readfirstlane(r / sz);
      return true;
    }
    before += __shfl(x, 63, 64);
  }
  return false;
}

__device__ __forceinline__ f32x4 mma8(i32x8 w, i32x8 x, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 pair(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Tile of TM activation rows x TN weight rows, WM x WN waves, NBUF stages in
// LDS (NBUF - 1 in flight).
template <int TM_, int TN_, int WM_, int WN_, int NBUF_>
struct Geo8 {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NBUF = NBUF_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  static constexpr int A_BYTES = TM * 128, W_BYTES = TN * 128, S_BYTES = NW * 256;
  static constexpr int STAGE = A_BYTES + W_BYTES + S_BYTES;
  static constexpr int PITCH = TN * 2 + 16;  // bytes of an output image row
  static constexpr int LDS = cmax(NBUF * STAGE, TM * PITCH);
  static_assert(LDS <= 160 * 1024, "LDS of one workgroup");
  static_assert(128 % (TN / WN) == 0, "a wave's weight rows lie in one block of 128");
  static_assert(NW * 64 >= TM, "one scale a lane");
};

template <class G>
__global__ __launch_bounds__(G::NT) void k_fp8_tile(Fp8Args p) {
  extern __shared__ __align__(16) char smem[];
  using LA = v2::KLoadA<G::TM, 64, G::NW>;
  using LW = v2::KLoadS<G::TN, 64, G::NW>;
  constexpr int INSTS = LA::NJ + LW::NJ + 1;
  int e, m, nt;
  if (!pool_tile(p, G::TM, blockIdx.x, (p.N + G::TN - 1) / G::TN, TILE_GM, e, m, nt)) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / G::WN, wn = w % G::WN;
  const int n0 = nt * G::TN, KB = p.K / 128;
  const long row0 = (long)p.offsets[e] + (long)m * G::TM;
  const int nrows = min(p.counts[e] - m * G::TM, G::TM);
  const int ncols = min(p.N - n0, G::TN);
  // loads: rows of codes as rows of K / 2 16-bit words
  LA la;
  LW lw;
  rsrc_t rs;
  uint32_t soff;
  {
    const int r = 64 * w + lane;  // this lane's activation row for the scales
    if (p.topk > 0) {
      la.rs = make_rsrc(p.a, (uint64_t)p.a_rows * p.K);
#pragma unroll
      for (int j = 0; j < LA::NJ; ++j) {
        const int q = LA::row_of(j);
        const int t = q < nrows ? p.row2r[row0 + q] / p.topk : -1;
        la.set_row(j, t >= 0 && t < p.a_rows ? (uint32_t)t * (uint32_t)p.K : OFF_NONE);
      }
      rs = make_rsrc(p.sa, (uint64_t)p.a_rows * KB * 4);
      const int t = r < nrows ? p.row2r[row0 + r] / p.topk : -1;
      soff = t >= 0 && t < p.a_rows ? (uint32_t)t * (uint32_t)KB * 4u : OFF_NONE;
    } else {
      const long have = p.a_rows - row0;
      const int live = (int)(have < nrows ? (have > 0 ? have : 0) : nrows);
      la.contig((const uint16_t*)p.a, row0, live, p.K / 2);
      rs = make_rsrc(p.sa + row0 * KB, (uint64_t)live * KB * 4);
      soff = r < live ? (uint32_t)r * (uint32_t)KB * 4u : OFF_NONE;
    }
    lw.contig((const uint16_t*)(p.w + (long)e * p.N * p.K), n0, ncols, p.K / 2);
  }
  auto issue = [&](int s) {
    char* st = smem + (s % G::NBUF) * G::STAGE;
    la.issue(64 * s, st);
    lw.issue(64 * s, st + G::A_BYTES);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (v2::lds_void*)(st + G::A_BYTES + G::W_BYTES + 256 * w), 4, soff,
                                             4u * (uint32_t)s, 0, 0);
  };
  // the wave's weight scale of K block s
  const int nb = min((n0 + wn * (G::TN / G::WN)) / 128, p.N / 128 - 1);
  const float* sw = p.sw + ((long)e * (p.N / 128) + nb) * KB;
  f32x4 acc[G::FN][G::FM];
#pragma unroll
  for (int i = 0; i < G::FN; ++i)
#pragma unroll
    for (int j = 0; j < G::FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // fragment row l % 16; chunks l / 16 and l / 16 + 4 of its 128 bytes (both
  // operands alike, so the order of k inside the instruction does not matter)
  const int fr = lane & 15, fc = lane >> 4;
#pragma unroll
  for (int s = 0; s < G::NBUF - 1; ++s)
    if (s < KB) issue(s);
  for (int s = 0; s < KB; ++s) {
    const int left = KB - 1 - s;
    if (G::NBUF >= 4 && left >= 2)
      v2::wait_vm<2 * INSTS>();
    else if (G::NBUF >= 3 && left >= 1)
      v2::wait_vm<INSTS>();
    else
      v2::wait_vm<0>();
    v2::wait_lgkm0();  // this wave is done reading the buffer that is refilled after the barrier
    v2::bar();
    if (s + G::NBUF - 1 < KB) issue(s + G::NBUF - 1);
    const char* st = smem + (s % G::NBUF) * G::STAGE;
    const char* sA = st;
    const char* sW = st + G::A_BYTES;
    const float* sS = (const float*)(st + G::A_BYTES + G::W_BYTES);
    const float ws = sw[s];
    i32x8 x[G::FM];
    float sc[G::FM];
#pragma unroll
    for (int j = 0; j < G::FM; ++j) {
      const int r = (wm * G::FM + j) * 16 + fr;
      x[j] = pair(*(const u32x4*)(sA + v2::koff<64>(r, fc)), *(const u32x4*)(sA + v2::koff<64>(r, fc + 4)));
      sc[j] = sS[r] * ws;
    }
#pragma unroll
    for (int i = 0; i < G::FN; ++i) {
      const int r = (wn * G::FN + i) * 16 + fr;
      const i32x8 a = pair(*(const u32x4*)(sW + v2::koff<64>(r, fc)), *(const u32x4*)(sW + v2::koff<64>(r, fc + 4)));
      f32x4 t[G::FM];
#pragma unroll
      for (int j = 0; j < G::FM; ++j) t[j] = mma8(a, x[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
      for (int j = 0; j < G::FM; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(t[j][q], sc[j], acc[i][j][q]);
    }
  }
  __syncthreads();  // LDS free for the image
#pragma unroll
  for (int i = 0; i < G::FN; ++i)
#pragma unroll
    for (int j = 0; j < G::FM; ++j) {
      const int r = (wm * G::FM + j) * 16 + fr, c = (wn * G::FN + i) * 16 + 4 * fc;
      *(u32x2*)(smem + r * G::PITCH + 2 * c) =
          u32x2{pack2(acc[i][j][0], acc[i][j][1]), pack2(acc[i][j][2], acc[i][j][3])};
    }
  __syncthreads();
  const int cpr = ncols / 8;  // 16-byte chunks per row
  for (int i = tid; i < nrows * cpr; i += G::NT) {
    const int r = i / cpr, c = i - r * cpr;
    *(u32x4*)(p.out + (row0 + r) * p.N + n0 + 8 * c) = *(const u32x4*)(smem + r * G::PITCH + 16 * c);
  }
}

using GL = Geo8<256, 256, 4, 2, 2>;

template <class G>
hipError_t launch_tile(const Fp8Args& p, int64_t mtiles, hipStream_t st) {
  static PerDeviceOnce once;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_fp8_tile<G>, G::LDS);
    return ai.err;
  });
  if (e != hipSuccess) return e;
  const int64_t grid = mtiles * ((p.N + G::TN - 1) / G::TN);
  MOE_LAUNCH_AS("k_fp8_tile", k_fp8_tile<G>, dim3((unsigned)grid), dim3(G::NT), G::LDS, st, p);
  return hipGetLastError();
}

constexpr int MAX_DIM = 65536;  // a tile's row offsets stay in 32 bits

moe_status check_weight(int32_t E, int32_t N, int32_t K) {
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID;
  if (E > 512 || N % 128 != 0 || K % 128 != 0 || N > MAX_DIM || K > MAX_DIM || (int64_t)N * K >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

moe_status moe_fp8_quantize_rows(const void* src, int64_t rows, int32_t K, int32_t act, void* codes, float* scales,
                                 void* stream) {
  if (rows < 0 || K < 1) return MOE_ERR_INVALID;
  if (K % 128 != 0 || K > MAX_DIM || rows >= (int64_t)1 << 31 || rows * (K / 8) >= ((int64_t)1 << 31) * 256)
    return MOE_ERR_UNSUPPORTED;
  if (act != MOE_FP8_PLAIN && act != MOE_ACT_SWIGLU && act != MOE_ACT_GEGLU) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!aligned16(src) || !aligned16(codes) || !aligned(scales, 4)) return MOE_ERR_INVALID;
  const size_t n = (size_t)rows * K;
  const Range ri = rng(src, n * (act == MOE_FP8_PLAIN ? 2 : 4)), rc = rng(codes, n), rs = rng(scales, n / 32);
  if (overlap(ri, rc) || overlap(ri, rs) || overlap(rc, rs)) return MOE_ERR_INVALID;
  const long n8 = (long)(n / 8);
  const dim3 g((unsigned)((n8 + 255) / 256)), b(256);
  const hipStream_t st = (hipStream_t)stream;
  const uint16_t* s = (const uint16_t*)src;
  if (act == MOE_FP8_PLAIN)
    MOE_LAUNCH_AS("k_fp8_rows", k_fp8_rows<MOE_FP8_PLAIN>, g, b, 0, st, s, n8, K / 8, (uint8_t*)codes, scales);
  else if (act == MOE_ACT_SWIGLU)
    MOE_LAUNCH_AS("k_fp8_rows", k_fp8_rows<MOE_ACT_SWIGLU>, g, b, 0, st, s, n8, K / 8, (uint8_t*)codes, scales);
  else
    MOE_LAUNCH_AS("k_fp8_rows", k_fp8_rows<MOE_ACT_GEGLU>, g, b, 0, st, s, n8, K / 8, (uint8_t*)codes, scales);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_fp8_quantize_weight(const void* W, int32_t E, int32_t N, int32_t K, void* codes, float* scales,
                                   void* codes_t, float* scales_t, void* stream) {
  const moe_status st = check_weight(E, N, K);
  if (st != MOE_OK) return st;
  if (!aligned16(W) || !aligned16(codes) || !aligned(scales, 4)) return MOE_ERR_INVALID;
  if ((codes_t != nullptr) != (scales_t != nullptr)) return MOE_ERR_INVALID;
  if (codes_t != nullptr && (!aligned16(codes_t) || !aligned(scales_t, 4))) return MOE_ERR_INVALID;
  const size_t n = (size_t)E * N * K, ns = n / (128 * 128) * 4;
  const Range r[] = {rng(W, 2 * n), rng(codes, n), rng(scales, ns), rng(codes_t, n), rng(scales_t, ns)};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(r[i], r[j])) return MOE_ERR_INVALID;
  MOE_LAUNCH(k_fp8_weight, dim3(K / 128, N / 128, E), dim3(256), 0, (hipStream_t)stream, (const uint16_t*)W, N, K,
             (uint8_t*)codes, scales, (uint8_t*)codes_t, scales_t);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_fp8_product(const moe_fp8_desc* d, const moe_pool* pool, const void* a, const float* a_scales,
                           const void* w, const float* w_scales, void* out, void* stream) {
  if (d == nullptr || pool == nullptr) return MOE_ERR_INVALID;
  const moe_status st = check_weight(d->E, d->N, d->K);
  if (st != MOE_OK) return st;
  if (d->topk < 0 || d->a_rows < 1 || pool->capacity < 1) return MOE_ERR_INVALID;
  if (pool->capacity >= (int64_t)1 << 31 || d->a_rows >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  if (d->topk > 0 && d->a_rows * d->K >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;  // one buffer descriptor
  if (!aligned(pool->counts, 4) || !aligned(pool->offsets, 4) || !aligned(pool->row_to_route, 4))
    return MOE_ERR_INVALID;
  if (!aligned16(a) || !aligned(a_scales, 4) || !aligned16(w) || !aligned(w_scales, 4) || !aligned16(out))
    return MOE_ERR_INVALID;
  const size_t na = (size_t)d->a_rows * d->K, nw = (size_t)d->E * d->N * d->K;
  const Range ro = rng(out, (size_t)pool->capacity * d->N * 2);
  const Range ins[] = {rng(a, na), rng(a_scales, na / 32), rng(w, nw), rng(w_scales, nw / (128 * 128) * 4),
                       rng(pool->counts, (size_t)d->E * 4), rng(pool->offsets, (size_t)d->E * 4 + 4),
                       rng(pool->row_to_route, (size_t)pool->capacity * 4)};
  for (const Range& r : ins)
    if (overlap(ro, r)) return MOE_ERR_INVALID;
  Fp8Args p{d->E, d->N, d->K, d->topk, (long)d->a_rows, pool->counts, pool->offsets, pool->row_to_route,
            (const uint8_t*)a, a_scales, (const uint8_t*)w, w_scales, (uint16_t*)out};
  // M tiles of TM rows any counts of `capacity` rows can make
  auto tiles = [&](int tm) { return pool->capacity / tm + (d->E < pool->capacity ? d->E : pool->capacity); };
  if (tiles(GL::TM) * ((d->N + GL::TN - 1) / GL::TN) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  const hipError_t e = launch_tile<GL>(p, tiles(GL::TM), (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
