// tile_stream.hpp -- the stage stream of the tiled expert products: one
// workgroup walks tiles, and while the last stages of a tile are multiplied the
// first of the next are already loading.
//
// A stage is 128 bytes of K of a tile's rows (64 bf16, 256 4-bit codes), or 64
// K-rows of its columns, in one of NBUF LDS buffers, filled by direct loads.
// Waves hold FM x FN blocks of 16 x 16.  The first matrix operand (w) gives four
// neighbouring results of a lane, the second (x) the lane's row.
//
// A policy P provides:
//   G                     the geometry (below)
//   INSTS, FIRST          direct loads of a wave and stage; those that a stage's
//                         start needs (the rest: the second half of its w blocks)
//   aim(tile, any)        point the loads at a tile (any: there is one)
//   issue(s, g, i)        queue load i of stage s of the tile aimed at into buffer g
//   x(buf, j), w(buf, i)  block j / i of the wave from a buffer's tiles
//   next(tile)            the following tile, and queue what aim() reads of it
//   stages(tile)          its number of stages, at least NBUF
//   mma<H>(w, x, acc)     half H of a block product
//   store(tile, acc)
//   fill(s), begin(), turn()  the stage that the next issue() calls fill first, the
//                         start of a stage, and the step of x() and w() to the next
//
// SPLIT (two buffers): a buffer is refilled for stage s + 2 in two parts, each
// as soon as the workgroup has read it: from the middle of the stage on x (in
// registers by then) and the first half of w's blocks, at the end the others,
// so a load has one and a half stages to arrive.  The last two w blocks are
// multiplied in turn, so that an x block is done with every four instructions and
// the next stage's is read in its place.  Otherwise whole stages are queued
// NBUF ahead.
#pragma once
#include "engine2.hpp"

namespace moelora {
namespace stream {

template <int TM_, int TN_, int WM_, int WN_, int NBUF_, int EXTRA_ = 0>
struct Geo {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NBUF = NBUF_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  static constexpr bool SPLIT = NBUF == 2;
  static constexpr int X_BYTES = TM * 128, W_BYTES = TN * 128;
  static constexpr int STAGE = X_BYTES + W_BYTES;
  static constexpr int END = NBUF * STAGE;  // LDS behind the buffers is the policy's
};

// Direct loads for kernels that read LDS by transposing reads: before each of
// those the compiler waits for every direct load that it knows of, the stages
// ahead included, so here the load is one that it does not see.  It has no
// register results; the caller waits for it by count.  The descriptor is the
// four words of a raw buffer (make_rsrc).  A vector instruction may have written
// the scalar operands just before (v_readfirstlane), after which a buffer
// instruction needs five wait states, and M0 needs one: the compiler counts
// neither for inline assembly.
typedef u32x4 desc_t;
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const void* p) {
  const uint64_t b = (uint64_t)p;
  return (const char*)((uint64_t)uniform((uint32_t)(b >> 32)) << 32 | uniform((uint32_t)b));
}
__device__ __forceinline__ desc_t make_desc(const void* base, uint64_t bytes) {
  const uint64_t b = (uint64_t)base;
  const uint32_t n = (uint32_t)(bytes < RSRC_MAX ? bytes : RSRC_MAX);
  return desc_t{uniform((uint32_t)b), uniform((uint32_t)(b >> 32) & 0xffffu), uniform(n), 0x00020000u};
}
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return uniform((uint32_t)(uintptr_t)(v2::lds_void*)p);
}
__device__ __forceinline__ void load16(desc_t d, char* lds_wave_base, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds_address(lds_wave_base)), "v"(off), "s"(d), "s"(uniform(soff)) : "memory", "m0");
}
__device__ __forceinline__ void load4(desc_t d, char* lds_wave_base, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds_address(lds_wave_base)), "v"(off), "s"(d), "s"(uniform(soff)) : "memory", "m0");
}
// The same through the compiler.
__device__ __forceinline__ void load16(rsrc_t d, char* lds_wave_base, uint32_t off, uint32_t soff) {
  v2::lds_load16(d, lds_wave_base, off, soff);
}
__device__ __forceinline__ void load4(rsrc_t d, char* lds_wave_base, uint32_t off, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(d, (v2::lds_void*)lds_wave_base, 4, off, soff, 0, 0);
}

struct Frag {
  u32x4 lo, hi;  // 16 bytes each: the two halves of a block's K
  int scale;     // 4-bit blocks: the two halves' exponents
};

// Lane offsets of the 16-row blocks of a K tile of 128-byte rows: lane l takes
// row l % 16 and chunks 2 (l / 16) and 2 (l / 16) + 1.  (The order of k inside an
// instruction does not matter as long as both operands agree; with chunks l / 16
// and l / 16 + 4 the 16 lanes that one LDS pass serves meet in the same banks
// under this swizzle.)  The chunk swizzle of tile row 16 i + r is
// (r & 7) ^ (r >> 3) ^ 2 (i & 3): four offsets serve every block, the second
// chunk in the slot beside.
struct RowFrags {
  uint32_t o[4];
  __device__ __forceinline__ void init(int lane, int first) {  // first: tile index of the wave's block 0
    const uint32_t r = lane & 15, c = 2 * (lane >> 4);
    const uint32_t slot = c ^ (r & 7) ^ (r >> 3);
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = 128u * r + ((slot ^ (2u * ((v + first) & 3))) << 4);
  }
  __device__ __forceinline__ Frag get(const char* tile, int i) const {  // tile: at the wave's block 0
    return Frag{*(const u32x4*)(tile + o[i & 3] + 2048 * i), *(const u32x4*)(tile + (o[i & 3] ^ 16u) + 2048 * i), 0};
  }
};

// T tiles (K-outer): [64 k][128 columns] of bf16, pitch 256 bytes, 16-byte chunk j
// of row k in slot j ^ swz(k); a tile of 256 columns is two of them, the first
// holding columns 0 .. 63 and 128 .. 191.  A transposing read touches, for each 16
// lanes, two chunks of four rows k0 .. k0 + 3, and two such groups of lanes, 16 rows
// apart, are served together: with the last two bits of k in the slot's upper bits
// and bit 4 in bit 1 the two cover all banks once (without the latter half of the
// LDS cycles of the weight gradient were conflicts).
__device__ __forceinline__ int t_swz(int k) { return ((k & 3) << 2) ^ (((k >> 4) & 1) << 1); }

// Lane offsets of its 16-column blocks.  A lane takes k 16 (l / 16) .. + 15 of a
// column by four reads.  PER: columns of a wave in one tile.
template <int PER>
struct ColFrags {
  uint32_t o[4];
  __device__ __forceinline__ void init(int lane, int first) {  // first: the wave's first column in the tile
    const int g = lane >> 4, i = lane & 15, k = 16 * g + (i >> 2);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int chunk = (first >> 3) + 2 * v + ((i & 3) >> 1);
      o[v] = (uint32_t)(k * 256 + ((chunk ^ t_swz(k)) << 4) + (i & 1) * 8);
    }
  }
  __device__ __forceinline__ Frag get(const char* tile, int i) const {
    constexpr int N = PER / 16;  // blocks of the wave in a tile
    const char* p = tile + (i / N) * 16384 + o[i % N];
    auto rd = [&](int t) {
      return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v2::s16x4*)(p + 1024 * t)));
    };
    const u32x2 a = rd(0), b = rd(1), c = rd(2), d = rd(3);
    return Frag{u32x4{a[0], a[1], b[0], b[1]}, u32x4{c[0], c[1], d[0], d[1]}, 0};
  }
};

template <class P>
__device__ __forceinline__ void run(P& p, typename P::Tile cur, char* smem) {
  using G = typename P::G;
  constexpr int FM = G::FM, FN = G::FN, NBUF = G::NBUF, INSTS = P::INSTS, FIRST = P::FIRST;
  constexpr int EVERY = 4;                    // matrix instructions between two loads (SPLIT)
  constexpr int MID = FN / 2 - 1;             // w block before which x and the first half of w have been read
  constexpr int BEFORE = (FN - 2 - MID) * 2 * FM / EVERY;  // loads issued between the two barriers
  static_assert(!G::SPLIT || (FN >= 4 && BEFORE <= FIRST && INSTS * EVERY <= (FN - 2 - MID) * 2 * FM + 4 * FM), "");
  f32x4 acc[FN][FM];
  Frag x[FM], a;
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // multiply the stage in buffer g, queue stage q of the tile aimed at into it,
  // and read the next stage's first blocks
  auto stage = [&](int g, int q) {
    const int gn = g + 1 == NBUF ? 0 : g + 1;
    const char* B = smem + g * G::STAGE;
    const char* Bn = smem + gn * G::STAGE;
    p.begin();
    if constexpr (G::SPLIT) {
      Frag b, c;
#pragma unroll
      for (int i = 0; i < FN - 2; ++i) {
        if (i == MID) {
          v2::wait_lgkm0();      // this wave has read x and the first half of w
          v2::wait_vm<INSTS>();  // the other half has landed
          v2::bar();
        }
        b = p.w(B, i + 1);
        if (i == FN - 3) c = p.w(B, FN - 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 2 * FM; ++m) {
          const int j = m % FM;
          if (m < FM)
            p.template mma<0>(a, x[j], acc[i][j]);
          else
            p.template mma<1>(a, x[j], acc[i][j]);
          const int t = (i - MID) * 2 * FM + m;
          if (i >= MID && t % EVERY == EVERY - 1 && t / EVERY < INSTS) p.issue(q, g, t / EVERY);
          if (m & 1) __builtin_amdgcn_sched_barrier(0);
        }
        a = b;
      }
      v2::wait_lgkm0();  // this wave has read all of the stage
      // the next one's first part has landed
      v2::wait_vm<INSTS - FIRST + BEFORE>();
      v2::bar();
      b = c;
      p.turn();
      Frag n = p.w(Bn, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        p.template mma<0>(a, x[j], acc[FN - 2][j]);
        p.template mma<0>(b, x[j], acc[FN - 1][j]);
        __builtin_amdgcn_sched_barrier(0);
        p.template mma<1>(a, x[j], acc[FN - 2][j]);
        p.template mma<1>(b, x[j], acc[FN - 1][j]);
        x[j] = p.x(Bn, j);
        const int t = (FN - 2 - MID) * 2 * FM + 4 * j + 3;
        if (t / EVERY < INSTS) p.issue(q, g, t / EVERY);
        __builtin_amdgcn_sched_barrier(0);
      }
      a = n;
    } else {
      Frag b;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        if (i + 1 < FN) {
          b = p.w(B, i + 1);
        } else {
          v2::wait_lgkm0();                   // this wave has read all of the stage
          v2::wait_vm<(NBUF - 2) * INSTS>();  // the next one has landed
          v2::bar();
          p.turn();
          b = p.w(Bn, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < FN) {
#pragma unroll
          for (int m = 0; m < 2 * FM; ++m) {
            const int j = m % FM;
            if (m < FM)
              p.template mma<0>(a, x[j], acc[i][j]);
            else
              p.template mma<1>(a, x[j], acc[i][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < FM; ++j) {
            p.template mma<0>(a, x[j], acc[i][j]);
            p.template mma<1>(a, x[j], acc[i][j]);
            x[j] = p.x(Bn, j);
#pragma unroll
            for (int l = j * INSTS / FM; l < (j + 1) * INSTS / FM; ++l) p.issue(q, g, l);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        a = b;
      }
    }
  };

  p.aim(cur, true);
  int g = 0, ST = p.stages(cur);
#pragma unroll
  for (int s = 0; s < NBUF; ++s) {
    p.fill(s);
#pragma unroll
    for (int l = 0; l < INSTS; ++l) p.issue(s, s, l);
  }
  v2::wait_vm<(NBUF - 1) * INSTS>();
  v2::bar();
  p.turn();
  a = p.w(smem, 0);
#pragma unroll
  for (int j = 0; j < FM; ++j) x[j] = p.x(smem, j);
  clear();
  while (true) {
    typename P::Tile nxt = cur;
    const bool more = p.next(nxt);
    for (int s = 0; s + NBUF < ST; ++s) {
      stage(g, s + NBUF);
      g = g + 1 == NBUF ? 0 : g + 1;
    }
    if (ST < NBUF + 2) {  // what next() queued: the waits of two stages cover it, of fewer not
      v2::wait_vm<0>();
      v2::bar();
    }
    p.aim(nxt, more);
    for (int s = 0; s < NBUF; ++s) {
      stage(g, s);
      g = g + 1 == NBUF ? 0 : g + 1;
    }
    p.store(cur, acc);
    if (!more) break;
    clear();
    cur = nxt;
    ST = p.stages(cur);
  }
  v2::wait_vm<0>();  // the loads queued past the last tile have written their zeros
}

}  // namespace stream
}  // namespace moelora
