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
// Inside the instruction sums are shorter than fp32: of 8 consecutive products
// what lies below 2^-13 of the largest exponent sum is cut, the groups are
// joined in 24 bits (measured with single products beside large ones that
// cancel).  That is up to 2^-10 of the terms' magnitudes, seen up to 2^-16,
// against 2^-4 for each code's own rounding and 2^-8 for the output's; the
// older fp8 instructions, K 32, run at half the rate.
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
constexpr int MAX_DIM = 65536;     // N and K: a tile's row offsets stay in 32 bits
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

// The normal distribution function to fp32's relative precision: a block in its
// lower tail is scaled by its own largest value, which norm_cdf's absolute error
// of 1e-7 would shift (1 % at -8).  Phi(g) = 1/2 exp(-z^2) f(z) at z = -g / sqrt 2
// >= 0, with f(z) = exp(z^2) erfc(z) = t P(t), t = 1 / (1 + 0.46 z): P of degree 7 is
// fitted for the smallest largest relative error over all z, 6.8e-7 (8.7e-7
// evaluated in fp32); here halved.  98,304 x 2048, same inputs: 200 us, 195 with
// norm_cdf, 302 with the math library's erfcf.
__device__ __forceinline__ float norm_cdf_rel(float g) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.46f * 0.70710678118654752f, fabsf(g), 1.0f));
  float q = 0.0338571894f;
  q = fmaf(q, t, -0.113314702f);
  q = fmaf(q, t, 0.084595587f);
  q = fmaf(q, t, 0.0263052463f);
  q = fmaf(q, t, 0.093423918f);
  q = fmaf(q, t, 0.115590938f);
  q = fmaf(q, t, 0.129778633f);
  q = fmaf(q, t, 0.12976353f);
  const float tail = q * t * __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);  // log2(e) / 2
  return g < 0.0f ? tail : 1.0f - tail;
}

// Eight columns a thread, a block of 128 in one DPP row: one pass, bound by
// memory (16,384 x 4096: 34 us, 6.0 TB/s of the 6.5 that plain loads and stores
// reach, 30 us with inputs left in the caches; gated 98,304 x 2048 172 us, 5.9
// TB/s; gated 2,064 x 2048 5.8 us, latency).  GEGLU fills the vector issue slots:
// 98,304 x 2048 200 to 219 us, 2,064 x 2048 6.0 to 7.2.
// ACT < 0: src is [rows, K]; else [rows, 2K] = gate | up.
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
    for (int q = 0; q < 8; ++q) v[q] = (ACT == MOE_ACT_SWIGLU ? v[q] * sigmoidf_(v[q]) : v[q] * norm_cdf_rel(v[q])) * u[q];
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
// values (row t / 2, half t % 2).  The transposed codes go through LDS, four
// bytes from four rows a word (1.7 bank conflicts an instruction).  64 experts of
// 4096 x 4096: 705 us, 4.6 TB/s; with the transposed copy 995 us, 4.3 TB/s.  A
// program does this once for its frozen weights.
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
  int cap;  // rows of the pool
  uint32_t tok_mul;  // route / topk = route * tok_mul >> tok_shift
  int tok_shift;
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

// Rows of expert e, none past the pool whatever its arrays hold.
__device__ __forceinline__ int rows_of(const Fp8Args& p, int e) {
  const int off = p.offsets[e];
  return off >= 0 && off < p.cap ? max(min(p.counts[e], p.cap - off), 0) : 0;
}
// The activation row of a route, -1: none (a_rows < 2^31).  No branches: loads
// of several routes stay together.
__device__ __forceinline__ int token_of(const Fp8Args& p, int route) {
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
// More tiles than a pool can have: the sums stop there, so that no counts make
// them wrap.
__device__ __forceinline__ int most_tiles(const Fp8Args& p, int TM) { return p.cap / TM + p.E; }
__device__ __forceinline__ bool pool_tile(const Fp8Args& p, int TM, int b, int nn, int gm, int& e, int& m, int& nt) {
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

__device__ __forceinline__ f32x4 mma8(i32x8 w, i32x8 x, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 pair(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Tile of TM activation rows x TN weight rows, WM x WN waves, NBUF stages in
// LDS.  SPLIT: a stage's buffer is refilled in two parts (k_fp8_tile).
template <int TM_, int TN_, int WM_, int WN_, int NBUF_>
struct Geo8 {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NBUF = NBUF_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  static constexpr bool SPLIT = NBUF == 2;
  static constexpr int A_BYTES = TM * 128, W_BYTES = TN * 128, S_BYTES = NW * 256;
  static constexpr int STAGE = A_BYTES + W_BYTES + S_BYTES;
  static constexpr int SW_AT = NBUF * STAGE;  // two tiles' weight scales, [2][TN / 128][stages]
  static constexpr int stages(int K) { return cmax(K / 128, NBUF); }
  static constexpr int table_at(int K) { return SW_AT + 2 * (TN / 128) * stages(K) * 4; }  // PoolTable
  static constexpr int lds(int K, int E) { return table_at(K) + 12 * E + 4 * TM; }  // and the next tile's routes
  static_assert(128 % (TN / WN) == 0 && TN % 128 == 0 && TN <= 256, "a wave's weight rows lie in one block of 128");
  static_assert(lds(MAX_DIM, MAX_E) <= 160 * 1024 && NW * 64 >= TM && FN % 2 == 0, "one scale a lane; fragments are stored in pairs");
};

// The pool's tiles of TM rows, in LDS: for each expert the number of tiles up
// to and with it, its rows and its first row.
struct PoolTable {
  int *end, *cnt, *off;
  int total;
};
template <int TM>
__device__ __forceinline__ void fill_table(const Fp8Args& p, PoolTable& t, char* at) {
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
struct Tile8 {
  int e, nt, nrows;
  long row0;
};
template <int TM>
__device__ __forceinline__ bool find_tile(const PoolTable& t, int E, int b, int nn, Tile8& out) {
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

// Lane offsets of the 16-row fragments of a tile of 128-byte rows: lane l
// takes row l % 16 and chunks 2 (l / 16) and 2 (l / 16) + 1, 32 bytes in a
// row.  (The order of k inside the instruction does not matter as long as both
// operands agree; with chunks l / 16 and l / 16 + 4 the 16 lanes that one
// LDS pass serves, 0-3, 12-15 and 20-27 of 32, meet in the same banks under
// this swizzle, which cost 47 % more LDS cycles.)  The chunk swizzle of tile
// row 16 i + r is (r & 7) ^ (r >> 3) ^ 2 (i & 3): four offsets serve every
// fragment, the second chunk in the slot beside.
struct Frag8 {
  uint32_t o[4];
  __device__ __forceinline__ void init(int lane, int first) {  // first: tile index of the wave's fragment 0
    const uint32_t r = lane & 15, c = 2 * (lane >> 4);
    const uint32_t slot = c ^ (r & 7) ^ (r >> 3);
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = 128u * r + ((slot ^ (2u * ((v + first) & 3))) << 4);
  }
  __device__ __forceinline__ i32x8 get(const char* tile, int i) const {  // tile: at the wave's fragment 0
    const u32x4 lo = *(const u32x4*)(tile + o[i & 3] + 2048 * i);
    const u32x4 hi = *(const u32x4*)(tile + (o[i & 3] ^ 16u) + 2048 * i);
    return pair(lo, hi);
  }
};

// A workgroup walks tiles b, b + gridDim.x, ... with one unbroken stream of
// stages: while the last stages of a tile are multiplied the first of the next
// are already loading, and the finished tile is stored from registers.
//
// A stage s in steady state: the products of weight fragment i are issued
// while those before them are scaled and added and fragment i + 1 is read.
// With SPLIT the last two fragments are multiplied in turn, so that an
// activation fragment is done with at every second product and the next
// stage's is read in its place: read at every product, the next stage's five
// fragments took more LDS time than the products above them (1 % slower).  With SPLIT
// a buffer is refilled for stage s + 2 in two parts, each as soon as the
// workgroup has read it: from mid-stage on the activation rows (in registers by
// then) and the weight rows of the first half of the fragments, at the end the
// others, so a load has one and a half stages to arrive from two buffers (one
// with a refill at the end alone).  Without SPLIT whole stages are queued NBUF
// ahead.  The next tile's routes come through LDS, queued a tile ahead: read
// where they are needed, and with the lanes' offsets kept in scratch across the
// K loop, each wait for one waited for all queued loads (2 % slower).
//
// What it measured, 98,304 rows of 4096 x 4096 on 64 experts: 1.55-1.62 ms,
// 2,040-2,130 TFLOP/s (experts of equal size: 1.49; one expert, 8192^3: 2,290; a
// library's product with one scale a tensor 2,660-2,760).  The matrix cores are
// busy 61 % of the cycles at 1.6 GHz, which is the power cap: activations of zeros
// take 1.28 ms.  A tile costs 10 us beyond its 1.6 us a stage, most of it the
// time that its 128 KB take to memory (three quarters of the stores left out:
// 0.10 ms less): waits that leave them out for two stages gained nothing, nor did
// workgroups that start up to 60 us apart.  Loads queued in one burst after the
// barrier instead of spread over the products: 6 % slower; a stage's fragments
// read at its start, each product's result added at once: 2.41 ms.  Touching
// the lines of later stages for L2 cost 0.2 ms: the loads are bound by
// throughput, not by misses.  Rows over an expert's last whole tile as
// 64-row tiles in a launch of their own: no gain, on ragged experts a loss of
// up to 17 %; waves without rows only loading: 2 % slower.  The 64-row tile,
// 689 tokens x 6 with a fifth of the routes dropped, 4096 x 2048: 116 us, 4.9
// TB/s of weights (a kernel that only reads: 7.1); with six buffers instead of three, one workgroup a CU: no
// faster, 0.5 us a K block, which is the chain of barrier, fragment reads and
// products.
//
// Loads past a tile's K (K / 128 < NBUF) or past the last tile go to offsets
// outside every descriptor: zeros, no traffic, and the loop waits by constant
// counts and has no branch.
template <class G>
__global__ __launch_bounds__(G::NT) void k_fp8_tile(Fp8Args p) {
  extern __shared__ __align__(16) char smem[];
  using LA = v2::KLoadA<G::TM, 64, G::NW>;
  using LW = v2::KLoadS<G::TN, 64, G::NW>;
  constexpr int FM = G::FM, FN = G::FN;
  constexpr int INSTS = LA::NJ + LW::NJ + 1;  // direct loads of a wave and stage
  static_assert(!G::SPLIT || (G::TN == 256 && G::NW == 8 && G::WN == 2 && FN == 8),
                "SPLIT: loads 0 and 2 of a stage are the rows of fragments 0-3, 1 and 3 those of 4-7");
  const int KB = p.K / 128, ST = cmax(KB, G::NBUF), nn = (p.N + G::TN - 1) / G::TN;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / G::WN, wn = w % G::WN;
  const int fr = lane & 15;
  PoolTable tab;
  fill_table<G::TM>(p, tab, smem + G::table_at(p.K));
  Tile8 cur;
  int b = blockIdx.x;
  if (!find_tile<G::TM>(tab, p.E, b, nn, cur)) return;

  // queue a tile's routes into LDS, where aim reads them
  char* const routes = smem + G::table_at(p.K) + 12 * p.E;
  auto queue_routes = [&](const Tile8& t) {
    if (p.topk > 0 && 64 * w < G::TM)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(p.row2r + t.row0, (uint64_t)t.nrows * 4),
                                               (v2::lds_void*)(routes + 256 * w), 4, 256u * w + 4u * lane, 0, 0, 0);
  };
  LA la;
  LW lw;
  rsrc_t rs;
  uint32_t soff;
  // aim the loads at a tile, and queue its weight scales into half h.  The
  // lane's number passes through an empty asm so that what is computed from it
  // is computed for each tile: kept across the K loop it went to scratch, and
  // each reload waited for all queued loads.
  auto aim = [&](const Tile8& t, bool any, int h) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int n0 = t.nt * G::TN, ncols = min(p.N - n0, G::TN);
    auto row_of = [&](int j) { return 8 * (w + G::NW * j) + (lane >> 3); };
    auto chunk = [&](int j) { return 16u * (uint32_t)((lane & 7) ^ v2::kswz<64>(row_of(j))); };
    if (p.topk > 0) {
      // tokens of the activation rows that this lane loads: LA::NJ rows of codes, one scale
      int tk[LA::NJ + 1];
#pragma unroll
      for (int j = 0; j <= LA::NJ; ++j)
        tk[j] = ((const int*)routes)[j < LA::NJ ? row_of(j) : min(64 * w + lane, G::TM - 1)];
#pragma unroll
      for (int j = 0; j <= LA::NJ; ++j)
        tk[j] = token_of(p, (j < LA::NJ ? row_of(j) : 64 * w + lane) < t.nrows ? tk[j] : -1);
      la.rs = make_rsrc(p.a, any ? (uint64_t)p.a_rows * p.K : 0);
      rs = make_rsrc(p.sa, any ? (uint64_t)p.a_rows * KB * 4 : 0);
#pragma unroll
      for (int j = 0; j < LA::NJ; ++j) la.voff[j] = tk[j] >= 0 ? (uint32_t)tk[j] * (uint32_t)p.K + chunk(j) : OFF_NONE;
      soff = tk[LA::NJ] >= 0 ? (uint32_t)tk[LA::NJ] * (uint32_t)KB * 4u : OFF_NONE;
    } else {
      const long have = p.a_rows - t.row0;
      const int live = any ? (int)(have < t.nrows ? (have > 0 ? have : 0) : t.nrows) : 0;
      la.rs = make_rsrc(p.a + t.row0 * p.K, (uint64_t)live * p.K);
#pragma unroll
      for (int j = 0; j < LA::NJ; ++j)
        la.voff[j] = row_of(j) < live ? (uint32_t)row_of(j) * (uint32_t)p.K + chunk(j) : OFF_NONE;
      rs = make_rsrc(p.sa + t.row0 * KB, (uint64_t)live * KB * 4);
      soff = 64 * w + lane < live ? (uint32_t)(64 * w + lane) * (uint32_t)KB * 4u : OFF_NONE;
    }
    lw.rs = make_rsrc(p.w + ((long)t.e * p.N + n0) * p.K, any ? (uint64_t)ncols * p.K : 0);
    // scale blocks x stages, 64 values a load; block c of stages past K, and of columns past N, reads zero
    const rsrc_t rw = make_rsrc(p.sw + ((long)t.e * (p.N / 128) + n0 / 128) * KB, any ? (uint64_t)(ncols / 128) * KB * 4 : 0);
    char* to = smem + G::SW_AT + h * (G::TN / 128) * ST * 4;
    for (int c = w; c * 64 < G::TN / 128 * ST; c += G::NW) {
      const int i = 64 * c + lane, blk = i >= ST ? 1 : 0, k = i - blk * ST;  // two blocks at most
      if (i < G::TN / 128 * ST)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (v2::lds_void*)(to + 256 * c), 4,
                                                 k < KB ? (uint32_t)(blk * KB + k) * 4u : OFF_NONE, 0, 0, 0);
    }
  };
  // queue load q of a stage s of the tile aimed at into buffer g: the activation
  // rows, the scales, the weight rows (with SPLIT 0 and 2 first, then 1 and 3)
  auto issue1 = [&](int s, int g, int q) {
    char* st = smem + g * G::STAGE;
    const uint32_t k0 = s < KB ? 128u * (uint32_t)s : (uint32_t)RSRC_MAX;
    if (q < LA::NJ) {
      v2::lds_load16(la.rs, st + 1024 * (w + G::NW * q), la.voff[q], k0);
    } else if (q == LA::NJ) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (v2::lds_void*)(st + G::A_BYTES + G::W_BYTES + 256 * w), 4, soff,
                                               s < KB ? 4u * (uint32_t)s : (uint32_t)RSRC_MAX, 0, 0);
    } else {
      const int i = q - LA::NJ - 1, j = !G::SPLIT ? i : i < 2 ? 2 * i : 2 * i - 3;
      v2::lds_load16(lw.rs, st + G::A_BYTES + 1024 * (w + G::NW * j), (j & 1) ? lw.v1 : lw.v0,
                     k0 + (uint32_t)j * lw.jstep);
    }
  };

  Frag8 fa, fw;
  fa.init(lane, wm * FM);
  fw.init(lane, wn * FN);
  f32x4 acc[FN][FM], t[FM];
  i32x8 x[FM], a;
  float sc[FM], sl[FM];  // this stage's scales, and those of the products in t
  // A tile's first stage adds t * sl for products of none before it: both are
  // zero then, for the scales of the last tile need not be finite.
  auto clear = [&]() {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      t[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      sl[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < FN; ++i) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  // the weight scale of stage s lies at smem + off
  auto read_scales = [&](int g, int off, float (&to)[FM]) {
    const float* sS = (const float*)(smem + g * G::STAGE + G::A_BYTES + G::W_BYTES) + wm * FM * 16 + fr;
    const float ws = *(const float*)(smem + off);
#pragma unroll
    for (int j = 0; j < FM; ++j) to[j] = sS[16 * j] * ws;
  };
  auto sw_at = [&](int h, int s) {
    return G::SW_AT + ((h * (G::TN / 128) + wn * (G::TN / G::WN) / 128) * ST + s) * 4;
  };
  // Products of a stage in order: fragment I(m) of the weight, J(m) of the
  // activations, its result in t[m % FM] until product m + FM has that place.
  constexpr int N = FM * FN;
  auto I = [](int m) constexpr { return G::SPLIT && m >= N - 2 * FM ? FN - 2 + (m & 1) : m / FM; };
  auto J = [](int m) constexpr { return G::SPLIT && m >= N - 2 * FM ? (m - (N - 2 * FM)) / 2 : m % FM; };
  // multiply the stage in buffer g; queue stage q of the tile aimed at into
  // it; read the next stage's first fragments (its weight scale at swn)
  auto stage = [&](int g, int q, int swn) {
    constexpr int LAST = G::SPLIT ? N - 2 * FM : N - FM;  // from here the next stage's fragments are read
    const int gn = g + 1 == G::NBUF ? 0 : g + 1;
    const char* sW = smem + g * G::STAGE + G::A_BYTES + wn * FN * 2048;
    const char* nA = smem + gn * G::STAGE + wm * FM * 2048;
    float sn[FM];
    i32x8 b, c;  // the weight fragments after a
#pragma unroll
    for (int m = 0; m < N; ++m) {
      if (m % FM == 0 && m <= LAST) {
        if (G::SPLIT && m == N / 2 - FM) {
          v2::wait_lgkm0();  // this wave has read the activation rows and the first weight rows
          v2::wait_vm<INSTS>();  // the other weight rows have landed
          v2::bar();
        }
        if (m < LAST) {
          b = fw.get(sW, m / FM + 1);
          if (G::SPLIT && m + FM == LAST) c = fw.get(sW, m / FM + 2);
        } else {
          v2::wait_lgkm0();  // this wave has read all of the stage
          // the next one's first part has landed (SPLIT: one load of the one after is not queued yet)
          v2::wait_vm<G::SPLIT ? INSTS - 1 : (G::NBUF - 2) * INSTS>();
          v2::bar();
          a = fw.get(smem + gn * G::STAGE + G::A_BYTES + wn * FN * 2048, 0);
          read_scales(gn, swn, sn);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const int done = m < FM ? m + N - FM : m - FM, j = J(m);
      const float f = m < FM ? sl[J(done)] : sc[J(done)];
      f32x4& to = acc[I(done)][J(done)];
#pragma unroll
      for (int e = 0; e < 4; ++e) to[e] = fmaf(t[m % FM][e], f, to[e]);
      t[m % FM] = mma8(m < LAST ? a : G::SPLIT && (m & 1) ? c : b, x[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      if constexpr (G::SPLIT) {
        if (m >= LAST && (m & 1)) x[j] = fa.get(nA, j);
        // a load at every other product from mid-stage on
        if ((m & 1) && m > N / 2 - FM && (m - (N / 2 - FM)) / 2 < INSTS) issue1(q, g, (m - (N / 2 - FM)) / 2);
      } else if (m >= LAST) {
        x[j] = fa.get(nA, j);
#pragma unroll
        for (int l = j * INSTS / FM; l < (j + 1) * INSTS / FM; ++l) issue1(q, g, l);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (m % FM == FM - 1 && m + 1 < LAST) a = b;
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      sl[j] = sc[j];
      sc[j] = sn[j];
    }
  };

  lw.contig(nullptr, 0, 0, p.K / 2);  // the lane's offsets in any weight panel
  queue_routes(cur);
  v2::wait_vm<0>();
  v2::bar();
  aim(cur, true, 0);
  int h = 0, g = 0;  // half of the weight scales, buffer of the stage to multiply
#pragma unroll
  for (int s = 0; s < G::NBUF; ++s) {
#pragma unroll
    for (int l = 0; l < INSTS; ++l) issue1(s, s, l);
  }
  v2::wait_vm<(G::NBUF - 1) * INSTS>();
  v2::bar();
  a = fw.get(smem + G::A_BYTES + wn * FN * 2048, 0);
#pragma unroll
  for (int j = 0; j < FM; ++j) x[j] = fa.get(smem + wm * FM * 2048, j);
  read_scales(0, sw_at(0, 0), sc);
  clear();
  while (true) {
    Tile8 nxt = cur;
    b += gridDim.x;
    const bool more = find_tile<G::TM>(tab, p.E, b, nn, nxt);
    if (more) queue_routes(nxt);
    for (int s = 0; s + G::NBUF < ST; ++s) {
      stage(g, s + G::NBUF, sw_at(h, s + 1));
      g = g + 1 == G::NBUF ? 0 : g + 1;
    }
    if (ST < G::NBUF + 2) {  // the routes: the waits of two stages cover them, of fewer not
      v2::wait_vm<0>();
      v2::bar();
    }
    aim(nxt, more, h ^ 1);
    for (int s = 0; s < G::NBUF; ++s) {
      stage(g, s, s + 1 < G::NBUF ? sw_at(h, ST - G::NBUF + s + 1) : sw_at(h ^ 1, 0));
      g = g + 1 == G::NBUF ? 0 : g + 1;
    }
    // A lane holds four columns of a row for each fragment; of two neighbouring
    // fragments, rows of 16 lanes trade so that it holds eight columns of one.
    // Rows past the tile's lie outside the descriptor; a wave's columns are all
    // below N or none.
    int lane2 = lane;
    asm volatile("" : "+v"(lane2));
    const int fr = lane2 & 15, fc = lane2 >> 4;
#pragma unroll
    for (int m = N - FM; m < N; ++m) {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[I(m)][J(m)][c] = fmaf(t[m % FM][c], sl[J(m)], acc[I(m)][J(m)][c]);
    }
    const bool cols = cur.nt * G::TN + wn * FN * 16 < p.N;
    const rsrc_t ro = make_rsrc(p.out + cur.row0 * p.N + cur.nt * G::TN, (uint64_t)cur.nrows * p.N * 2);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = (wm * FM + j) * 16 + fr;
#pragma unroll
      for (int i = 0; i < FN; i += 2) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][0], acc[i][j][1]),
                                                         pack2(acc[i + 1][j][0], acc[i + 1][j][1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][2], acc[i][j][3]),
                                                         pack2(acc[i + 1][j][2], acc[i + 1][j][3]), false, false);
        const int c = (wn * FN + i + (fc & 1)) * 16 + 8 * (fc >> 1);
        const uint32_t off = cols ? (uint32_t)(r * p.N + c) * 2u : OFF_NONE;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, ro, (int)off, 0, 0);
      }
    }
    if (!more) break;
    clear();
    cur = nxt;
    h ^= 1;
  }
  v2::wait_vm<0>();  // the loads queued past the last tile have written their zeros
}

// Few rows per expert (decoding): the weights are read once and bound the
// time, so they go from memory straight into the registers that the matrix
// instruction takes.  A workgroup is one wave (so that the few tiles spread
// evenly over the CUs): 16 activation rows x 16 weight rows, the next FEW_CH K
// blocks in flight while FEW_CH are multiplied.  It walks K in
// order, so a row's sums are those of the tile kernels bit for bit.
// One expert of 4096 x 4096, 1 to 16 rows: 12 us (reading its weights alone: 2.4),
// two of eight 12.6, eight of 128 experts of 1024 x 2048 10.3: each wave's chain
// of K / 128 blocks sets the time, not the bytes.  Split over four waves of a
// workgroup along K instead, with its join, six experts took 44 us, whole
// workgroups of 64 weight rows 27 (384 of them on 256 CUs), single waves 21.
constexpr int FEW_ROWS = 16, FEW_CH = 4;
__global__ __launch_bounds__(64) void k_fp8_few(Fp8Args p) {
  const int lane = threadIdx.x;
  const int fr = lane & 15, fc = lane >> 4;
  const int KB = p.K / 128;
  int e, m, nt;
  for (int b = blockIdx.x; pool_tile(p, FEW_ROWS, b, p.N / 16, TILE_GM, e, m, nt); b += gridDim.x) {
    const int n0 = nt * 16;
    const rsrc_t rw = make_rsrc(p.w + ((long)e * p.N + n0) * p.K, (uint64_t)16 * p.K);
    const uint32_t wo = (uint32_t)fr * (uint32_t)p.K + 32u * (uint32_t)fc;
    const long row0 = (long)p.offsets[e] + (long)m * FEW_ROWS;
    const int nrows = min(rows_of(p, e) - m * FEW_ROWS, FEW_ROWS);
    const float* sw = p.sw + ((long)e * (p.N / 128) + n0 / 128) * KB;
    // this lane's activation row and scale row
    rsrc_t ra, rs;
    long ar = -1;
    if (p.topk > 0) {
      ra = make_rsrc(p.a, (uint64_t)p.a_rows * p.K);
      rs = make_rsrc(p.sa, (uint64_t)p.a_rows * KB * 4);
      if (fr < nrows) ar = token_of(p, p.row2r[row0 + fr]);
    } else {
      const long have = p.a_rows - row0;
      const int live = (int)(have < nrows ? (have > 0 ? have : 0) : nrows);
      ra = make_rsrc(p.a + row0 * p.K, (uint64_t)live * p.K);
      rs = make_rsrc(p.sa + row0 * KB, (uint64_t)live * KB * 4);
      if (fr < live) ar = fr;
    }
    const uint32_t ao = ar >= 0 ? (uint32_t)ar * (uint32_t)p.K + 32u * (uint32_t)fc : OFF_NONE;
    const uint32_t so = ar >= 0 ? (uint32_t)ar * (uint32_t)KB * 4u : OFF_NONE;
    struct Set {
      u32x4 wl[FEW_CH], wh[FEW_CH], al[FEW_CH], ah[FEW_CH];
      float sc[FEW_CH], sb[FEW_CH];
    };
    auto load = [&](Set& q, int c0) {
#pragma unroll
      for (int i = 0; i < FEW_CH; ++i) {
        const int c = c0 + i;
        const bool in = c < KB, has = in && ar >= 0;
        const uint32_t k = 128u * (uint32_t)c;
        q.wl[i] = bload(rw, in ? wo + k : OFF_NONE);
        q.wh[i] = bload(rw, in ? wo + k + 16u : OFF_NONE);
        q.al[i] = bload(ra, has ? ao + k : OFF_NONE);
        q.ah[i] = bload(ra, has ? ao + k + 16u : OFF_NONE);
        q.sc[i] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(has ? so + 4u * (uint32_t)c : OFF_NONE), 0, 0));
        q.sb[i] = in ? sw[c] : 0.0f;
      }
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto mul = [&](const Set& q) {
#pragma unroll
      for (int i = 0; i < FEW_CH; ++i) {
        const f32x4 t = mma8(pair(q.wl[i], q.wh[i]), pair(q.al[i], q.ah[i]), f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        const float sc = q.sc[i] * q.sb[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(t[j], sc, acc[j]);
      }
    };
    Set s0, s1;
    load(s0, 0);
    for (int c = 0; c < KB; c += 2 * FEW_CH) {
      load(s1, c + FEW_CH);
      mul(s0);
      load(s0, c + 2 * FEW_CH);
      mul(s1);
    }
    if (fr < nrows)
      *(u32x2*)(p.out + (row0 + fr) * p.N + n0 + 4 * fc) = u32x2{pack2(acc[0], acc[1]), pack2(acc[2], acc[3])};
  }
}

using GL = Geo8<256, 256, 4, 2, 2>;
using GM = Geo8<64, 128, 1, 4, 3>;

// Which kernel: the routes are known, how they fall on the experts is not, so
// an expert with rows is taken to have the mean, and an M tile more in half
// the cases.  Costs in us per K block, measured at N, K of 1024 to 8192, 1 to
// 64 experts, 1 to 4096 rows each: a 256-row tile a CU takes 1.35 while few
// of them run and 2.1 when all CUs load; two 64-row tiles 0.5 and 0.84.
// E.g. 8 experts, N = K = 4096: 128 rows each 40.6 us on 64-row tiles, 49.9 on
// 256; 1024 rows 211 and 168.  k_fp8_few pays where the 64-row tiles are too
// few for the CUs: its cost goes with the bytes its waves read, 16 weight rows
// and the tile's activation rows, and 20,000 of these rows are where the two
// meet (1 expert, N = K = 4096, 32 rows: 14.6 us and 17.5; 64 rows: 22.8 and
// 18.0).
enum class Pick { few, mid, large };
Pick pick(const Fp8Args& p, int64_t routes, int cus) {
  const double live = (double)(routes < p.E ? routes : p.E), avg = (double)routes / live, fill = cus / 256.0;
  auto mtiles = [&](int tm) { return live * (avg / tm + 0.5 > 1.0 ? avg / tm + 0.5 : 1.0); };
  const double few = mtiles(FEW_ROWS) * (p.N / 16) * (16.0 + (avg < 16.0 ? avg : 16.0));
  if (few <= 20000.0 * fill) return Pick::few;
  const double mid = 0.84 * mtiles(GM::TM) * ((p.N + GM::TN - 1) / GM::TN) / (2 * cus);
  const double large = 2.1 * mtiles(GL::TM) * ((p.N + GL::TN - 1) / GL::TN) / cus;
  return (mid > 0.5 ? mid : 0.5) <= (large > 1.35 ? large : 1.35) ? Pick::mid : Pick::large;
}

// Workgroups for at most `tiles` tiles: every kernel here walks on by its grid
// until the pool's tiles are done, so the grid is a matter of speed alone: as
// many as are resident, in whole rounds over the XCDs.
unsigned grid_of(int64_t tiles, int64_t most) { return (unsigned)(((tiles < most ? tiles : most) + 7) / 8 * 8); }

template <class G>
hipError_t launch_tile(const Fp8Args& p, int64_t mtiles, int resident, hipStream_t st) {
  static PerDeviceOnce once;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_fp8_tile<G>, G::lds(MAX_DIM, MAX_E));
    return ai.err;
  });
  if (e != hipSuccess) return e;
  const unsigned grid = grid_of(mtiles * ((p.N + G::TN - 1) / G::TN), resident);
  MOE_LAUNCH_AS(G::TM == 64 ? "k_fp8_tile64" : "k_fp8_tile256", k_fp8_tile<G>, dim3(grid), dim3(G::NT), G::lds(p.K, p.E), st, p);
  return hipGetLastError();
}

hipError_t launch_few(const Fp8Args& p, int64_t mtiles, int resident, hipStream_t st) {
  const unsigned grid = grid_of(mtiles * (p.N / 16), resident);
  MOE_LAUNCH(k_fp8_few, dim3(grid), dim3(64), 0, st, p);
  return hipGetLastError();
}

moe_status check_weight(int32_t E, int32_t N, int32_t K) {
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID;
  if (E > MAX_E || N % 128 != 0 || K % 128 != 0 || N > MAX_DIM || K > MAX_DIM || (int64_t)N * K >= (int64_t)1 << 31)
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
  // a launch holds fewer than 2^32 threads, eight columns each, in whole workgroups of 256
  if (K % 128 != 0 || K > MAX_DIM || rows >= (int64_t)1 << 31 || rows * K > ((int64_t)1 << 35) - 2048)
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
  if (d->topk < 0 || d->a_rows < 1 || pool->capacity < 1 || pool->block_m < 1)
    return MOE_ERR_INVALID;
  if (pool->capacity >= (int64_t)1 << 31 || d->a_rows >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  // tile indices of the smallest tiles are 32 bits
  if ((pool->capacity / FEW_ROWS + d->E) * (d->N / 16) >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
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
  // floor(n / k) = floor(n m / 2^(31 + s)) for n < 2^31, with 2^s >= k the
  // smallest and m = ceil(2^(31 + s) / k) < 2^32: n (m k - 2^(31 + s)) < 2^(31 + s)
  const uint64_t k = d->topk > 0 ? (uint64_t)d->topk : 1;
  int sh = 31;
  while ((uint64_t)1 << (sh - 31) < k) ++sh;
  const uint32_t mul = (uint32_t)((((uint64_t)1 << sh) + k - 1) / k);
  Fp8Args p{d->E, d->N, d->K, d->topk, (int)pool->capacity, mul, sh, (long)d->a_rows, pool->counts, pool->offsets,
            pool->row_to_route, (const uint8_t*)a, a_scales, (const uint8_t*)w, w_scales, (uint16_t*)out};
  // the routes of a pool of this capacity: build_pool allots BLOCK_M - 1 rows
  // of padding to each of min(E, routes) experts
  const int64_t bm = pool->block_m, cap = pool->capacity, E = d->E;
  const int64_t routes = cap >= E * bm ? cap - E * (bm - 1) : (cap + bm - 1) / bm;
  const int64_t live = routes < E ? routes : E;  // experts with rows, at most
  auto tiles = [&](int tm) { return routes / tm + live; };
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return MOE_ERR_HIP;
  const hipStream_t s = (hipStream_t)stream;
  switch (pick(p, routes, cus)) {
    case Pick::few: e = launch_few(p, tiles(FEW_ROWS), 8 * cus, s); break;
    case Pick::mid: e = launch_tile<GM>(p, tiles(GM::TM), 2 * cus, s); break;
    case Pick::large: e = launch_tile<GL>(p, tiles(GL::TM), cus, s); break;
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
