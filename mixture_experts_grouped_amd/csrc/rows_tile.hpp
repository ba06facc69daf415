// rows_tile.hpp -- tiled products of the pool's rows with their experts' weights
// on the stage stream (tile_stream.hpp): bf16, bf16 with the weight stored
// K-outer, and 4-bit blocks.
#pragma once
#include "pool_tiles.hpp"
#include "tile_stream.hpp"
#include "trace.hpp"

namespace moelora {

struct RowsArgs : PoolArgs {
  int N, K;
  const uint8_t* a;
  const uint8_t* w;
  const uint8_t* ea;  // 4-bit: exponents
  const uint8_t* ew;
  uint16_t* out;
};

enum class Kind { bf16, bf16_t, mxfp4, mxfp4_pairs };

typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x4 mma_bf16(u32x4 w, u32x4 x, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}
// 128 k of 4-bit codes, the exponent in byte H of each scale
template <int H>
__device__ __forceinline__ f32x4 mma_mxfp4(u32x4 w, u32x4 x, f32x4 c, int ew, int ex) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0},
                                                          i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0}, c,
                                                          4, 4, H, ew, H, ex);
}

template <Kind KIND, class G_>
struct RowsTile {
  using G = G_;
  using Tile = PoolTile;
  static constexpr bool PAIRS = KIND == Kind::mxfp4_pairs, MX = KIND == Kind::mxfp4 || PAIRS, TR = KIND == Kind::bf16_t;
  static constexpr int NX = G::X_BYTES / (1024 * G::NW), NWT = G::W_BYTES / (1024 * G::NW);
  // Exponents: 8 bytes of each row a stage, by one load a wave and operand; or
  // (PAIRS, whole pairs of stages) 16 bytes for two stages, by one load a wave at
  // even stages and none at odd ones, which halves the lines of memory touched: a
  // stage's 512 pieces of 8 bytes cost as many as its codes (98,304 rows of 4096 x
  // 4096: 110 of 930 us).
  static constexpr int NS = PAIRS ? 1 : MX ? 2 : 0;
  static constexpr int INSTS = NX + NWT + NS, FIRST = NX + NS + NWT / 2;
  static constexpr int SLOT = PAIRS ? (G::TM + G::TN) * 16 : 2 * G::NW * 256;  // bytes of a stage's (a pair's) exponents: x, then w
  static constexpr int SLOTS = PAIRS ? 2 : 3, COUNT = PAIRS ? 4 : 3;  // sl and fl count stages modulo COUNT
  static constexpr int SCALES = G::END;
  static constexpr int TABLE = SCALES + (MX ? SLOTS * SLOT : 0) + (PAIRS ? 1024 : 0);  // and where the loads of odd stages go
  static constexpr int lds(int E) { return TABLE + 12 * E + 4 * G::TM; }
  static_assert(!MX || PAIRS || (G::TM * 8 <= G::NW * 256 && G::TN * 8 == G::NW * 256), "one load of exponents a wave and operand");
  static_assert(!PAIRS || (G::SPLIT && G::TM == 64 * 4 && G::TN == 64 * 4), "waves 0-3 load x's exponents, 4-7 w's");
  static_assert(lds(MAX_E) <= 160 * 1024, "LDS");
  using Desc = typename std::conditional<TR, stream::desc_t, rsrc_t>::type;
  __device__ static __forceinline__ Desc desc(const void* base, uint64_t bytes) {
    if constexpr (TR)
      return stream::make_desc(base, bytes);
    else
      return make_rsrc(base, bytes);
  }
  static_assert(!G::SPLIT || (G::TN == 256 && G::NW == 8 && G::WN == 2 && G::FN == 8), "the halves of w");
  static_assert(G::SPLIT || (G::TN == 128 && G::NW == 4 && G::WN == 4), "");

  const RowsArgs& p;
  char* smem;
  PoolTable tab;
  int b, nn, RB, RE, lane, wv, wm, wn;
  stream::RowFrags fx, fw;
  stream::ColFrags<G::SPLIT ? 64 : 32> ft;
  Desc rx, rw, rsx, rsw;
  uint32_t vx[NX], vw[2], vsx, vsw;
  int sl, fl;  // slots of exponents: of the stage that x() and w() read, and that issue() fills

  __device__ __forceinline__ RowsTile(const RowsArgs& args, char* sm) : p(args), smem(sm) {
    lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wv / G::WN;
    wn = wv % G::WN;
    b = blockIdx.x;
    nn = (p.N + G::TN - 1) / G::TN;
    RB = MX ? p.K / 2 : 2 * p.K;  // bytes of a row
    RE = p.K / 32;
    fx.init(lane, wm * G::FM);
    if constexpr (TR)
      ft.init(lane, wn * (G::SPLIT ? 64 : 32));
    else
      fw.init(lane, wn * G::FN);
    sl = COUNT - 1;
  }
  __device__ __forceinline__ bool first(Tile& t) {
    fill_table<G::TM>(p, tab, smem + TABLE);
    if (!find_tile<G::TM>(tab, p.E, b, nn, t)) return false;
    queue_routes(t);
    v2::wait_vm<0>();
    v2::bar();
    return true;
  }
  __device__ __forceinline__ void queue_routes(const Tile& t) {
    if (p.topk > 0 && 64 * wv < G::TM)
      stream::load4(desc(p.row2r + t.row0, (uint64_t)t.nrows * 4), smem + TABLE + 12 * p.E + 256 * wv, 256u * wv + 4u * lane, 0);
  }
  __device__ __forceinline__ bool next(Tile& t) {
    b += gridDim.x;
    if (!find_tile<G::TM>(tab, p.E, b, nn, t)) return false;
    queue_routes(t);
    return true;
  }
  __device__ __forceinline__ int stages(const Tile&) const { return cmax((RB + 127) / 128, G::NBUF); }

  // The lane's number passes through an empty asm so that what is computed from
  // it is computed for each tile instead of being kept across the K loop.
  __device__ __forceinline__ void aim(const Tile& t, bool any) {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    const int n0 = t.nt * G::TN, ncols = min(p.N - n0, G::TN);
    auto row_of = [&](int j) { return 8 * (wv + G::NW * j) + (l >> 3); };
    auto chunk = [&](int j) { return 16u * (uint32_t)((l & 7) ^ v2::kswz<64>(row_of(j))); };
    // the row whose exponents this lane loads, of either operand, and its bytes in them
    const int erow = PAIRS ? 64 * (wv & 3) + l : 32 * wv + (l >> 1);
    const uint32_t ebyte = PAIRS ? 0u : 4u * (l & 1);
    if (p.topk > 0) {
      int tk[NX + 1];
      const int* routes = (const int*)(smem + TABLE + 12 * p.E);
#pragma unroll
      for (int j = 0; j <= NX; ++j) {
        const int r = j < NX ? row_of(j) : erow;
        tk[j] = j < NX || MX ? routes[min(r, G::TM - 1)] : -1;
        tk[j] = token_of(p, r < t.nrows ? tk[j] : -1);
      }
      rx = desc(p.a, any ? (uint64_t)p.a_rows * RB : 0);
#pragma unroll
      for (int j = 0; j < NX; ++j) vx[j] = tk[j] >= 0 ? (uint32_t)tk[j] * (uint32_t)RB + chunk(j) : OFF_NONE;
      if constexpr (MX) {
        rsx = desc(p.ea, any ? (uint64_t)p.a_rows * RE : 0);
        vsx = tk[NX] >= 0 ? (uint32_t)tk[NX] * (uint32_t)RE + ebyte : OFF_NONE;
      }
    } else {
      const long have = p.a_rows - t.row0;
      const int live = any ? (int)(have < t.nrows ? (have > 0 ? have : 0) : t.nrows) : 0;
      rx = desc(p.a + t.row0 * RB, (uint64_t)live * RB);
#pragma unroll
      for (int j = 0; j < NX; ++j) vx[j] = row_of(j) < live ? (uint32_t)row_of(j) * (uint32_t)RB + chunk(j) : OFF_NONE;
      if constexpr (MX) {
        rsx = desc(p.ea + t.row0 * RE, (uint64_t)live * RE);
        vsx = erow < live ? (uint32_t)erow * (uint32_t)RE + ebyte : OFF_NONE;
      }
    }
    if constexpr (TR) {
      rw = desc(p.w + (long)t.e * p.N * RB, any ? (uint64_t)p.K * p.N * 2 : 0);
      const int kr = 4 * wv + (l >> 4);
      // vw[h]: half h of the columns, or (one tile of 128) even and odd instructions, 16 rows apart
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 8 * ((l & 15) ^ stream::t_swz(kr + (G::SPLIT ? 0 : 16 * h)));
        const int col = n0 + (G::SPLIT ? c + (c >= 64 ? 64 : 0) + 64 * h : c);
        vw[h] = col < p.N ? (uint32_t)kr * (uint32_t)p.N * 2u + 2u * (uint32_t)col : OFF_NONE;
      }
    } else {
      rw = desc(p.w + ((long)t.e * p.N + n0) * RB, any ? (uint64_t)ncols * RB : 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) vw[j] = (uint32_t)(8 * wv + (l >> 3)) * (uint32_t)RB + chunk(j);
      if constexpr (MX) {
        rsw = desc(p.ew + ((long)t.e * p.N + n0) * RE, any ? (uint64_t)ncols * RE : 0);
        vsw = (uint32_t)erow * (uint32_t)RE + ebyte;
        if (PAIRS && wv >= 4) vsx = vsw;
      }
    }
  }

  __device__ __forceinline__ void fill(int s) { fl = s; }
  __device__ __forceinline__ void begin() { fl = !G::SPLIT ? sl : PAIRS ? (sl + 2) & 3 : sl == 0 ? 2 : sl - 1; }
  __device__ __forceinline__ void turn() { sl = sl == COUNT - 1 ? 0 : sl + 1; }
  // exponents of the stage that x() and w() read: where row r's begin
  __device__ __forceinline__ const char* scales(int r) const {
    return PAIRS ? smem + SCALES + (sl >> 1) * SLOT + 16 * r + 8 * (sl & 1) : smem + SCALES + sl * SLOT + 8 * r;
  }

  // Load i of stage s into buffer g.  What lies past the row's end reads zero.
  __device__ __forceinline__ void issue(int s, int g, int i) const {
    char* st = smem + g * G::STAGE;
    const int l = threadIdx.x & 63;
    auto in_row = [&](int j) {  // chunk j's (even or odd) place in the row
      const uint32_t c = 16u * (uint32_t)((l & 7) ^ v2::kswz<64>(8 * (wv + G::NW * (j & 1)) + (l >> 3)));
      return (int)c < RB - 128 * s;
    };
    if (i < NX) {
      stream::load16(rx, st + 1024 * (wv + G::NW * i), in_row(i) ? vx[i] : OFF_NONE, 128u * (uint32_t)s);
    } else if (i < NX + NS) {
      if constexpr (PAIRS) {
        // waves 0-3: 64 rows of x each, 4-7 of w
        const bool even = (s & 1) == 0;
        char* to = even ? smem + SCALES + (fl >> 1) * SLOT + 1024 * wv : smem + SCALES + 2 * SLOT;
        stream::load16(wv < 4 ? rsx : rsw, to, even && 8 * s < RE ? vsx : OFF_NONE, 8u * (uint32_t)s);
        return;
      }
      const bool in = 8 * s + 4 * (l & 1) < RE;
      char* to = smem + SCALES + fl * SLOT + (i > NX ? G::NW * 256 : 0) + 256 * wv;
      stream::load4(i > NX ? rsw : rsx, to, in ? (i > NX ? vsw : vsx) : OFF_NONE, 8u * (uint32_t)s);
    } else {
      const int q = i - NX - NS;
      if constexpr (TR) {
        // instruction q: half q / 2 (one half: all four), K-rows 4 (wave + ..)
        const int h = G::SPLIT ? q >> 1 : 0, r = G::SPLIT ? 32 * (q & 1) : 16 * q;
        char* to = st + G::X_BYTES + 16384 * h + 1024 * (wv + (G::SPLIT ? 8 * (q & 1) : 4 * q));
        stream::load16(rw, to, vw[G::SPLIT ? h : q & 1], (uint32_t)(64 * s + r) * (uint32_t)p.N * 2u);
      } else {
        const int j = !G::SPLIT ? q : q < 2 ? 2 * q : 2 * q - 3;  // the first halves of the waves' rows first
        stream::load16(rw, st + G::X_BYTES + 1024 * (wv + G::NW * j), in_row(j) ? vw[j & 1] : OFF_NONE,
                       128u * (uint32_t)s + (uint32_t)j * (8u * G::NW) * (uint32_t)RB);
      }
    }
  }

  __device__ __forceinline__ stream::Frag x(const char* buf, int j) const {
    stream::Frag f = fx.get(buf + wm * G::FM * 2048, j);
    if constexpr (MX)
      f.scale = *(const uint16_t*)(scales((wm * G::FM + j) * 16 + (lane & 15)) + 2 * (lane >> 4));
    return f;
  }
  __device__ __forceinline__ stream::Frag w(const char* buf, int i) const {
    if constexpr (TR) {
      return ft.get(buf + G::X_BYTES, i);
    } else {
      stream::Frag f = fw.get(buf + G::X_BYTES + wn * G::FN * 2048, i);
      if constexpr (MX)
        f.scale = *(const uint16_t*)(scales((PAIRS ? G::TM : G::NW * 32) + (wn * G::FN + i) * 16 + (lane & 15)) + 2 * (lane >> 4));
      return f;
    }
  }
  template <int H>
  __device__ __forceinline__ void mma(const stream::Frag& w, const stream::Frag& x, f32x4& acc) const {
    if constexpr (MX)
      acc = mma_mxfp4<H>(H ? w.hi : w.lo, H ? x.hi : x.lo, acc, w.scale, x.scale);
    else
      acc = mma_bf16(H ? w.hi : w.lo, H ? x.hi : x.lo, acc);
  }

  // A lane holds four columns of a row for each block; of two neighbouring
  // blocks, rows of 16 lanes trade so that it holds eight columns of one.  Rows
  // past the tile's lie outside the descriptor.
  __device__ __forceinline__ void store(const Tile& t, const f32x4 (&acc)[G::FN][G::FM]) const {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int fr = l & 15, fc = l >> 4;
    const rsrc_t ro = make_rsrc(p.out + t.row0 * p.N + t.nt * G::TN, (uint64_t)t.nrows * p.N * 2);
#pragma unroll
    for (int j = 0; j < G::FM; ++j) {
      const int r = (wm * G::FM + j) * 16 + fr;
#pragma unroll
      for (int i = 0; i < G::FN; i += 2) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][0], acc[i][j][1]),
                                                         pack2(acc[i + 1][j][0], acc[i + 1][j][1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][2], acc[i][j][3]),
                                                         pack2(acc[i + 1][j][2], acc[i + 1][j][3]), false, false);
        const int c = (wn * G::FN + i + (fc & 1)) * 16 + 8 * (fc >> 1);
        const uint32_t off = t.nt * G::TN + c < p.N ? (uint32_t)(r * p.N + c) * 2u : OFF_NONE;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, ro, (int)off, 0, 0);
      }
    }
  }
};

// 256 x 256 tiles, eight waves of 128 x 64, two buffers refilled in halves: many
// rows an expert, where an operand's read must feed as many products as the
// registers hold sums for.  bf16, 98,304 rows of 4096 x 4096: 2,550 us, 1,295
// TFLOP/s, the rate that the library's 8192^3 product reaches (matrix cores busy 76 %
// at the power cap's 1.73 GHz; without the results' stores 2,448 us; on other cards
// up to 2,680, and the next two by as much).  Weight stored
// K-outer (4096 x 2048): 1,390 us, 1,185 TFLOP/s, 65 % at 1.91 GHz: the transposing
// reads carry half as much an instruction.  4 bits: 900 us, 3,660 TFLOP/s; a block
// product takes 19 clocks of a SIMD, its operands' reads and refills together 83 % of
// the same time in LDS; without the exponents' loads 819 us, without the stores 830,
// without both 744.
// 64 x 128 tiles, four waves, three buffers, two workgroups a CU: in between, bound
// by reading the weights (689 tokens, a fifth of the routes dropped, 4096 x 2048: 208
// us, 5.2 TB/s; 4-bit weights for one token: 12.4 us).
template <Kind KIND, class G>
__global__ __launch_bounds__(G::NT) void k_rows_tile(RowsArgs p) {
  extern __shared__ __align__(16) char smem[];
  RowsTile<KIND, G> t(p, smem);
  PoolTile cur;
  if (!t.first(cur)) return;
  stream::run(t, cur, smem);
}

// Few rows per expert (decoding): the weights are read once and bound the
// time, so they go from memory straight into the registers that the matrix
// instruction takes.  A workgroup is one wave: 16 activation rows x 16 weight
// rows, the next FEW_CH stages of 128 bytes in flight while FEW_CH are
// multiplied.  bf16: an instruction takes 64 bytes of each row in one piece (the
// order of k inside a stage is free; 16 bytes at a distance of 32: 2 % slower; eight
// stages in flight: 25 %); 4 bits: 32 bytes a lane, whose two blocks' exponents lie
// side by side.  One token, six experts of 4096 x 4096 in bf16: 36.5 us, 5.5 TB/s
// (non-temporal loads 39); 64-row tiles 41.
constexpr int FEW_ROWS = 16, FEW_CH = 4;
template <Kind KIND>
__global__ __launch_bounds__(64) void k_rows_few(RowsArgs p) {
  constexpr bool MX = KIND == Kind::mxfp4;
  const int lane = threadIdx.x, fr = lane & 15, fc = lane >> 4;
  const int RB = MX ? p.K / 2 : 2 * p.K, RE = p.K / 32, KB = (RB + 127) / 128;
  int e, m, nt;
  for (int b = blockIdx.x; pool_tile(p, FEW_ROWS, b, (p.N + 15) / 16, TILE_GM, e, m, nt); b += gridDim.x) {
    const int n0 = nt * 16, ncols = min(p.N - n0, 16);
    const long row0 = (long)p.offsets[e] + (long)m * FEW_ROWS;
    const int nrows = min(rows_of(p, e) - m * FEW_ROWS, FEW_ROWS);
    const rsrc_t rw = make_rsrc(p.w + ((long)e * p.N + n0) * RB, (uint64_t)ncols * RB);
    constexpr uint32_t CB = MX ? 32u : 16u, HB = MX ? 16u : 64u;
    const uint32_t wo = (uint32_t)fr * (uint32_t)RB + CB * (uint32_t)fc;
    // this lane's activation row
    rsrc_t ra, rea, rew;
    long ar = -1;
    if (p.topk > 0) {
      ra = make_rsrc(p.a, (uint64_t)p.a_rows * RB);
      if constexpr (MX) rea = make_rsrc(p.ea, (uint64_t)p.a_rows * RE);
      if (fr < nrows) ar = token_of(p, p.row2r[row0 + fr]);
    } else {
      const long have = p.a_rows - row0;
      const int live = (int)(have < nrows ? (have > 0 ? have : 0) : nrows);
      ra = make_rsrc(p.a + row0 * RB, (uint64_t)live * RB);
      if constexpr (MX) rea = make_rsrc(p.ea + row0 * RE, (uint64_t)live * RE);
      if (fr < live) ar = fr;
    }
    if constexpr (MX) rew = make_rsrc(p.ew + ((long)e * p.N + n0) * RE, (uint64_t)ncols * RE);
    const uint32_t ao = (uint32_t)ar * (uint32_t)RB + CB * (uint32_t)fc;
    const uint32_t eo = (uint32_t)ar * (uint32_t)RE + 2u * (uint32_t)fc, eow = (uint32_t)fr * (uint32_t)RE + 2u * (uint32_t)fc;
    struct Set {
      stream::Frag w[FEW_CH], x[FEW_CH];
    };
    auto load = [&](Set& q, int c0) {
#pragma unroll
      for (int i = 0; i < FEW_CH; ++i) {
        const uint32_t k = 128u * (uint32_t)(c0 + i);
        const int left = RB - (int)k - (int)CB * fc;  // bytes of the row from this lane's on
        const bool lo = left > 0, hi = left > (int)HB, has = ar >= 0;
        q.w[i].lo = bload(rw, lo ? wo + k : OFF_NONE);
        q.w[i].hi = bload(rw, hi ? wo + k + HB : OFF_NONE);
        q.x[i].lo = bload(ra, lo && has ? ao + k : OFF_NONE);
        q.x[i].hi = bload(ra, hi && has ? ao + k + HB : OFF_NONE);
        if constexpr (MX) {  // K % 128 == 0: both halves or none
          const uint32_t x = 8u * (uint32_t)(c0 + i);
          q.w[i].scale = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rew, (int)(lo ? eow + x : OFF_NONE), 0, 0);
          q.x[i].scale = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rea, (int)(lo && has ? eo + x : OFF_NONE), 0, 0);
        }
      }
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto mul = [&](const Set& q) {
#pragma unroll
      for (int i = 0; i < FEW_CH; ++i) {
        if constexpr (MX) {
          acc = mma_mxfp4<0>(q.w[i].lo, q.x[i].lo, acc, q.w[i].scale, q.x[i].scale);
          acc = mma_mxfp4<1>(q.w[i].hi, q.x[i].hi, acc, q.w[i].scale, q.x[i].scale);
        } else {
          acc = mma_bf16(q.w[i].lo, q.x[i].lo, acc);
          acc = mma_bf16(q.w[i].hi, q.x[i].hi, acc);
        }
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
    if (fr < nrows && 4 * fc < ncols)
      *(u32x2*)(p.out + (row0 + fr) * p.N + n0 + 4 * fc) = u32x2{pack2(acc[0], acc[1]), pack2(acc[2], acc[3])};
  }
}

template <Kind KIND>
hipError_t launch_rows_few(const char* name, const RowsArgs& p, int64_t mtiles, int resident, hipStream_t st) {
  MOE_LAUNCH_AS(name, k_rows_few<KIND>, dim3(grid_of(mtiles * ((p.N + 15) / 16), resident)), dim3(64), 0, st, p);
  return hipGetLastError();
}

using GeoL = stream::Geo<256, 256, 4, 2, 2>;
using GeoM = stream::Geo<64, 128, 1, 4, 3>;

template <Kind KIND, class G>
hipError_t launch_rows_tile(const char* name, const RowsArgs& p, int64_t mtiles, int resident, hipStream_t st) {
  static PerDeviceOnce once;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_rows_tile<KIND, G>, RowsTile<KIND, G>::lds(MAX_E));
    return ai.err;
  });
  if (e != hipSuccess) return e;
  const unsigned grid = grid_of(mtiles * ((p.N + G::TN - 1) / G::TN), resident);
  MOE_LAUNCH_AS(name, (k_rows_tile<KIND, G>), dim3(grid), dim3(G::NT), (RowsTile<KIND, G>::lds(p.E)), st, p);
  return hipGetLastError();
}

// Which kernel: the routes are known, how they fall on the experts is not, so
// an expert with rows is taken to have the mean, and an M tile more in half the
// cases.  Costs in us, fitted to a sweep of 1 to 64 experts of 512 x 512 to 4096 x
// 4096 with 1 to 512 rows each: a start, and for each stage of 128 bytes of K
// what the rounds of tiles over the CUs take, or the least that one tile does.
enum class Pick { few, mid, large };
struct Costs {
  double few;  // weight and activation rows read by all tiles of 16 rows, up to which single waves are faster
  double mid_start, mid_least, mid;  // two 64-row tiles on a CU
  double large_start, large_least, large;
};
inline Pick pick(const RowsArgs& p, const Costs& c, int64_t routes, int cus, int row_bytes) {
  const double live = (double)(routes < p.E ? routes : p.E), avg = (double)routes / live, fill = cus / 256.0;
  const double stages = (row_bytes + 127) / 128;
  auto mtiles = [&](int tm) { return live * (avg / tm + 0.5 > 1.0 ? avg / tm + 0.5 : 1.0); };
  if (mtiles(FEW_ROWS) * ((p.N + 15) / 16) * (16.0 + (avg < 16.0 ? avg : 16.0)) <= c.few * fill) return Pick::few;
  const double mid = c.mid * mtiles(GeoM::TM) * ((p.N + GeoM::TN - 1) / GeoM::TN) / (2 * cus);
  const double large = c.large * mtiles(GeoL::TM) * ((p.N + GeoL::TN - 1) / GeoL::TN) / cus;
  return c.mid_start + stages * (mid > c.mid_least ? mid : c.mid_least) <=
                 c.large_start + stages * (large > c.large_least ? large : c.large_least)
             ? Pick::mid
             : Pick::large;
}

}  // namespace moelora
