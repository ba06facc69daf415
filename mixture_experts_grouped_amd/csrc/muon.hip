// muon.hip -- one optimiser step whose update is orthogonalised by rounds of a
// quintic polynomial (include/moelora.h states the formulas).
//
// With r = min(m, n) the short and L = max(m, n) the long side and U as r rows:
// every round multiplies X by a polynomial of S = X X^T, and all these
// polynomials are polynomials of S0 = U U^T, which commute and are symmetric.
// So the rounds run on r x r matrices,
//   P_k = a I + b S_k + c S_k^2,  S_k+1 = S_k P_k^2,  Q = P_last ... P_0,
// and X_last = Q X_0: U is read twice instead of three times a round.  A
// rounding of S_k in a direction of small singular value is amplified by about
// a^2 = 12 in each later round, since S_k is not formed anew from X: in fp32 the
// result is 1e-4 off where the singular values decay over five decades (rounds
// on X in fp32: 1e-5), in fp64 1e-7, so S and Q are fp64 (the matrix cores'
// fp64 rate is half their fp32 rate).
//
// Three kernels: the momentum and S0 (columns of U split over workgroups, partial
// sums added in a fixed order), the rounds (a workgroup a matrix), Q U and the
// parameters.
#include <cmath>

#include "../../include/moelora.h"
#include "checks.hpp"
#include "engine.hpp"
#include "pool_tiles.hpp"
#include "trace.hpp"

namespace moelora {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
constexpr int MAX_SHORT = 256;
constexpr int TENSORS = 40;   // a launch: their table travels in the kernel's arguments
// Entries of the long side in LDS at a time: a thread holds its share of the next
// ones in registers, of which two workgroups on a CU leave it 128.
__device__ __host__ constexpr int gram_chunk(int RB) { return RB <= 128 ? 64 : 32; }
__device__ __host__ constexpr int apply_chunk(int RB) { return RB <= 64 ? 64 : 32; }
constexpr int NT = 512, NW = 8;

struct MuonTensor {
  void* param;
  float* master;
  const void* grad;
  float* momentum;
  long first;        // this tensor's first workgroup in a launch over splits
  long matrix0;      // index of its first matrix
  double* part;      // a matrix: partial sums of S0 [splits][lower tiles], then (long short sides) the rounds' matrices
  float* q;          // [matrices][R][R]
  int r, L, tall;    // tall: stored [L, r]
  int R;             // r in whole tiles of 16
  int splits, span;  // workgroups along L, entries each
  int vec;           // groups of four neighbours in memory are whole and aligned
};
struct MuonArgs {
  MuonTensor t[TENSORS];
  int count, nesterov, rounds;
  long groups;    // workgroups of a launch over splits
  long matrices;
  float lr, momentum, weight_decay, grad_scale, rms;
  double a, b, c, eps;
  const moe_muon_control* control;
};
static_assert(sizeof(MuonArgs) <= 4096, "kernel arguments");

// A workgroup's tensor, matrix and part of the long side.
__device__ __forceinline__ void find(const MuonArgs& p, long b, int& t, long& mat, int& s) {
  t = 0;
  while (t + 1 < p.count && b >= p.t[t + 1].first) ++t;
  const long i = b - p.t[t].first;
  mat = i / p.t[t].splits;
  s = (int)(i - mat * p.t[t].splits);
}

// U (a chunk of the long side) lies in LDS as in memory: [l][c] of a tall
// tensor, [c][l] of a wide one, at a pitch of 20 of 64 banks: 16 rows of four
// neighbours meet in no bank.
__device__ __host__ constexpr int pitch_of(int n) { return (n + 43) / 64 * 64 + 20; }

template <class T>
__device__ __forceinline__ f32x4 load4(const T* p, bool vec, int live) {  // the first `live` of four
  if (vec) {
    if (live <= 0) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (sizeof(T) == 4) return *(const f32x4*)p;
    else {
      const u32x2 w = *(const u32x2*)p;
      return f32x4{bf2f(w[0] & 0xffffu), bf2f(w[0] >> 16), bf2f(w[1] & 0xffffu), bf2f(w[1] >> 16)};
    }
  }
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) {
      if constexpr (sizeof(T) == 4) v[e] = p[e];
      else v[e] = bf2f(p[e]);
    }
  return v;
}
template <class T>
__device__ __forceinline__ void store4(T* p, bool vec, int live, f32x4 v) {
  if (vec) {
    if (live <= 0) return;
    if constexpr (sizeof(T) == 4) *(f32x4*)p = v;
    else *(u32x2*)p = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) {
      if constexpr (sizeof(T) == 4) p[e] = v[e];
      else p[e] = (T)f2bf(v[e]);
    }
}

// What a thread moves of each chunk: groups of four neighbours in memory.
template <int RB, bool TALL, int CHUNK_>
struct Share {
  static constexpr int CHUNK = CHUNK_, N = RB * CHUNK / (4 * NT);
  static constexpr int PITCH = pitch_of(TALL ? RB : CHUNK);
  // LDS steps along the short and the long side
  static constexpr int KS = TALL ? 1 : PITCH, LS = TALL ? PITCH : 1;
  int at[N], lds[N];  // element in the chunk; LDS place, -1: none
  int live[N];        // tall: entries of the short side from here on, and 2^16 times the long side's; wide: of the chunk from here on
  int step;           // elements from one chunk to the next
  __device__ __forceinline__ void init(const MuonTensor& t) {
    const int B = TALL ? t.R : CHUNK, A = TALL ? CHUNK : t.R;
    step = TALL ? CHUNK * t.r : CHUNK;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int g = threadIdx.x + i * NT, a = g / (B / 4), b = 4 * (g - a * (B / 4));
      lds[i] = a < A ? a * PITCH + b : -1;
      at[i] = a * (TALL ? t.r : t.L) + b;
      if (TALL)
        live[i] = a < A && b < t.r ? (t.r - b) + (a << 16) : 0;
      else
        live[i] = a < A && a < t.r ? CHUNK - b : 0;
    }
  }
  // of group i, the elements there are in the chunk with `left` entries
  __device__ __forceinline__ int have(int i, int left) const {
    if (TALL) return (live[i] >> 16) < left ? live[i] & 0xffff : 0;
    return live[i] > 0 ? left - (CHUNK - live[i]) : 0;
  }
};

// Tile t of the lower triangle of tiles.
__device__ __forceinline__ void tri(int t, int& i, int& j) {
  i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  j = t - i * (i + 1) / 2;
}
__device__ __host__ constexpr int tri_tiles(int n) { return n * (n + 1) / 2; }

// Where a matrix's part of the workspace begins.
constexpr int SHORT_R = 128;   // up to here the rounds run in LDS
constexpr int LONG_SLOTS = 6;  // beyond, they have matrices behind the partial sums
__device__ __host__ constexpr long part_size(int R, int splits) {
  return (long)splits * tri_tiles(R / 16) * 256 + (R > SHORT_R ? (long)LONG_SLOTS * R * R : 0);
}
__device__ __forceinline__ long part_at(const MuonTensor& t, long mat) { return mat * part_size(t.R, t.splits); }

// The new momentum, and S0 of a part of the long side as lower tiles of 16 x 16.
// The next chunk's loads are in flight while this one is multiplied.
template <class GT, int RB, bool TALL, int N>
__device__ __forceinline__ void gram(const MuonArgs& p, const MuonTensor& t, long mat, int s, float* S) {
  using Sh = Share<RB, TALL, gram_chunk(RB)>;
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tiles = tri_tiles(t.R / 16);
  Sh sh;
  sh.init(t);
  const int l_begin = s * t.span;
  int left = min(t.L - l_begin, t.span);
  const bool vec = t.vec != 0;
  const long at = mat * (long)t.r * t.L + (TALL ? (long)l_begin * t.r : l_begin);
  const GT* g = (const GT*)t.grad + at;
  float* mo = t.momentum + at;
  f32x4 gv[Sh::N], mv[Sh::N];
  auto fetch = [&](int have) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      gv[i] = load4(g + sh.at[i], vec, sh.have(i, have));
      mv[i] = load4(mo + sh.at[i], vec, sh.have(i, have));
    }
  };
  f64x4 acc[cmax(N, 1)];
  int xi[cmax(N, 1)], yj[cmax(N, 1)];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    int i = 0, j = 0;
    if (w + NW * q < tiles) tri(w + NW * q, i, j);
    const int lo = (lane >> 4) * Sh::LS + (lane & 15) * Sh::KS;
    xi[q] = lo + 16 * i * Sh::KS;
    yj[q] = lo + 16 * j * Sh::KS;
    acc[q] = f64x4{0.0, 0.0, 0.0, 0.0};
  }
  fetch(left);
  for (; left > 0; left -= Sh::CHUNK) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      f32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = gv[i][e] * gs;
        mv[i][e] = fmaf(p.momentum, mv[i][e], x);
        u[e] = p.nesterov ? fmaf(p.momentum, mv[i][e], x) : mv[i][e];
      }
      store4(mo + sh.at[i], vec, sh.have(i, left), mv[i]);
      if (sh.lds[i] >= 0) *(f32x4*)(S + sh.lds[i]) = u;  // zeros where there is nothing
    }
    __syncthreads();
    g += sh.step;
    mo += sh.step;
    if (left > Sh::CHUNK) fetch(left - Sh::CHUNK);
    if constexpr (N > 0) {
      // operands of the next step are read while this one is multiplied
      float x[2][N], y[2][N];
      auto load = [&](int to, int k4) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
          x[to][q] = S[xi[q] + k4 * Sh::LS];
          y[to][q] = S[yj[q] + k4 * Sh::LS];
        }
      };
      load(0, 0);
#pragma unroll
      for (int k4 = 0; k4 < Sh::CHUNK; k4 += 4) {
        const int b = (k4 >> 2) & 1;
        if (k4 + 4 < Sh::CHUNK) load(b ^ 1, k4 + 4);
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[b][q], (double)y[b][q], acc[q], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
  }
  double* out = t.part + part_at(t, mat) + s * (long)(tiles * 256);
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (w + NW * q < tiles)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[(w + NW * q) * 256 + v * 64 + lane] = acc[q][v];  // row 4 v + lane / 16 of the tile
}
// Waves of at most N tiles; what a wave has less is multiplied and not stored.
template <class GT, int RB, bool TALL>
__device__ __forceinline__ void gram_of(const MuonArgs& p, const MuonTensor& t, long mat, int s, float* S) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = (tri_tiles(t.R / 16) - w + NW - 1) / NW;
  if constexpr (RB <= 64) {
    if (n >= 2) gram<GT, RB, TALL, 2>(p, t, mat, s, S);
    else if (n == 1) gram<GT, RB, TALL, 1>(p, t, mat, s, S);
    else gram<GT, RB, TALL, 0>(p, t, mat, s, S);
  } else if constexpr (RB <= 128) {
    if (n >= 5) gram<GT, RB, TALL, 5>(p, t, mat, s, S);
    else if (n == 4) gram<GT, RB, TALL, 4>(p, t, mat, s, S);
    else gram<GT, RB, TALL, 3>(p, t, mat, s, S);
  } else {
    if (n > 12) gram<GT, RB, TALL, 17>(p, t, mat, s, S);
    else if (n > 7) gram<GT, RB, TALL, 12>(p, t, mat, s, S);
    else gram<GT, RB, TALL, 7>(p, t, mat, s, S);
  }
}

template <class GT, int RB>
__global__ __launch_bounds__(NT, RB <= 128 ? 4 : 2) void k_muon_gram(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  int ti, s;
  long mat;
  find(p, blockIdx.x, ti, mat, s);
  const MuonTensor& t = p.t[ti];
  if (t.tall)
    gram_of<GT, RB, true>(p, t, mat, s, (float*)smem);
  else
    gram_of<GT, RB, false>(p, t, mat, s, (float*)smem);
}

// The rounds of a matrix of at most RB rows in LDS: two matrices as lower tiles
// of 16 x 16 at a pitch of 17, at which a column and a row of 16 lie in 16
// different pairs of banks.
template <int RB>
struct Rounds {
  static constexpr int MT = (tri_tiles(RB / 16) + NW - 1) / NW;
  static constexpr int PITCH = 17 * 8, TILE = 16 * PITCH;
  int nt, tiles, w, lane, mine;  // mine: tiles of the wave
  int ti[MT], tj[MT];
  int oc, orow;  // lane offsets of a column block and of a row block

  __device__ __forceinline__ void init(int R) {
    nt = R / 16;
    tiles = tri_tiles(nt);
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    mine = max(0, (tiles - w + NW - 1) / NW);
    oc = (lane & 15) * PITCH + (lane >> 4) * 8;
    orow = (lane >> 4) * PITCH + (lane & 15) * 8;
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      int i = 0, j = 0;
      if (live(q)) tri(w + NW * q, i, j);
      ti[q] = __builtin_amdgcn_readfirstlane(i);
      tj[q] = __builtin_amdgcn_readfirstlane(j);
    }
  }
  __device__ __forceinline__ bool live(int q) const { return w + NW * q < tiles; }
  // z = X Y for the wave's first N tiles.  Operands of a k-step (k = 16 kt + 4 s +
  // lane / 16) are read while the one before is multiplied: 16 rows of block i come
  // from a column of tile (i, kt), or above the diagonal from a row of (kt, i).
  template <int N>
  __device__ __forceinline__ void mul_n(const char* X, const char* Y, f64x4 (&z)[MT]) const {
    double v[2][2 * N];
    const char* at[2 * N];
    int step[2 * N];
    auto aim = [&](int kt) {
#pragma unroll
      for (int o = 0; o < 2 * N; ++o) {
        const int i = o < N ? ti[o] : tj[o - N];
        const bool low = i >= kt;
        const int base = (low ? tri_tiles(i) + kt : tri_tiles(kt) + i) * TILE;
        at[o] = (o < N ? X : Y) + base + (low ? oc : orow);
        step[o] = low ? 32 : 4 * PITCH;
      }
    };
    auto load = [&](int to) {
#pragma unroll
      for (int o = 0; o < 2 * N; ++o) {
        v[to][o] = *(const double*)at[o];
        at[o] += step[o];
      }
    };
#pragma unroll
    for (int q = 0; q < N; ++q) z[q] = f64x4{0.0, 0.0, 0.0, 0.0};
    aim(0);
    load(0);
    for (int kt = 0; kt < nt; ++kt)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s == 3) aim(min(kt + 1, nt - 1));  // after the last step: read again, not used
        load((s + 1) & 1);
#pragma unroll
        for (int q = 0; q < N; ++q) z[q] = __builtin_amdgcn_mfma_f64_16x16x4f64(v[s & 1][q], v[s & 1][N + q], z[q], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
  template <int N = MT>
  __device__ __forceinline__ void mul(const char* X, const char* Y, f64x4 (&z)[MT]) const {
    if constexpr (N > 0) {
      if (mine == N)
        mul_n<N>(X, Y, z);
      else
        mul<N - 1>(X, Y, z);
    }
  }
  __device__ __forceinline__ void put(char* X, const f64x4 (&z)[MT]) const {
#pragma unroll
    for (int q = 0; q < MT; ++q)
      if (live(q))
#pragma unroll
        for (int v = 0; v < 4; ++v) *(double*)(X + (w + NW * q) * TILE + orow + 4 * v * PITCH) = z[q][v];
  }
  __device__ __forceinline__ bool diagonal(int q, int v) const { return ti[q] == tj[q] && 4 * v + (lane >> 4) == (lane & 15); }
};

template <int RB>
__global__ __launch_bounds__(NT) void k_muon_rounds(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ double red[NW];
  int ti = 0;
  while (ti + 1 < p.count && (long)blockIdx.x >= p.t[ti + 1].matrix0) ++ti;
  const MuonTensor& t = p.t[ti];
  const long mat = blockIdx.x - t.matrix0;
  Rounds<RB> k;
  constexpr int MT = Rounds<RB>::MT;
  k.init(t.R);
  const int size = k.tiles * 256;
  char *A = smem, *B = smem + k.tiles * Rounds<RB>::TILE;
  f64x4 S[MT], Q[MT], z[MT];
  // the parts in order, and the trace: the sum of U's squares
  const double* part = t.part + part_at(t, mat);
  double tr = 0.0;
#pragma unroll
  for (int q = 0; q < MT; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      double x = 0.0;
      if (k.live(q)) {
        const double* at = part + (k.w + NW * q) * 256 + v * 64 + k.lane;
#pragma unroll 4
        for (int s = 0; s < t.splits; ++s) x += at[s * (long)size];
        if (k.diagonal(q, v)) tr += x;
      }
      S[q][v] = x;
    }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  if (k.lane == 0) red[k.w] = tr;
  __syncthreads();
  tr = 0.0;
#pragma unroll
  for (int i = 0; i < NW; ++i) tr += red[i];
  const double inv = 1.0 / (sqrt(tr) + p.eps), inv2 = inv * inv;
#pragma unroll
  for (int q = 0; q < MT; ++q) S[q] *= inv2;
  k.put(A, S);
  __syncthreads();
  for (int n = 0; n < p.rounds; ++n) {
    const bool last = n + 1 == p.rounds;
    k.mul(A, A, z);  // A = S
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v) z[q][v] = fma(p.c, z[q][v], fma(p.b, S[q][v], k.diagonal(q, v) ? p.a : 0.0));
    k.put(B, z);  // P
    if (n == 0) {
#pragma unroll
      for (int q = 0; q < MT; ++q) Q[q] = z[q];
    }
    __syncthreads();
    if (!last) {
      k.mul(A, B, z);
      __syncthreads();
      k.put(A, z);  // S P
      __syncthreads();
      k.mul(A, B, S);  // S P P: the next S
      __syncthreads();
    }
    if (n > 0) {
      if (last) __syncthreads();
      k.put(A, Q);
      __syncthreads();
      k.mul(B, A, Q);
      __syncthreads();
    }
    if (!last) {
      k.put(A, S);
      __syncthreads();
    }
  }
  float* out = t.q + mat * (long)t.R * t.R;
#pragma unroll
  for (int q = 0; q < MT; ++q)
    if (k.live(q))
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * k.ti[q] + 4 * v + (k.lane >> 4), c = 16 * k.tj[q] + (k.lane & 15);
        const float x = (float)(Q[q][v] * inv);
        out[(long)r * t.R + c] = x;
        out[(long)c * t.R + r] = x;
      }
}

// Longer short sides: the rounds' matrices in memory, whole, a launch a product,
// a wave a tile of 16 x 16.
__device__ __forceinline__ const MuonTensor& long_matrix(const MuonArgs& p, long& mat, int& tile, int per) {
  const long m = blockIdx.x / per;
  tile = (int)(blockIdx.x - m * per) * NW + (threadIdx.x >> 6);
  int ti = 0;
  while (ti + 1 < p.count && m >= p.t[ti + 1].matrix0) ++ti;
  mat = m - p.t[ti].matrix0;
  return p.t[ti];
}
__device__ __forceinline__ double* long_slot(const MuonTensor& t, long mat, int slot) {
  return t.part + part_at(t, mat) + t.splits * (long)(tri_tiles(t.R / 16) * 256) + slot * (long)t.R * t.R;
}
__device__ __forceinline__ double long_inv(const MuonArgs& p, const MuonTensor& t, long mat) {  // 1 / (|U| + eps), by every wave
  const long tiles = (long)tri_tiles(t.R / 16) * 256;
  const double* part = long_slot(t, mat, 0) - t.splits * tiles;
  double tr = 0.0;
  for (int c = threadIdx.x & 63; c < t.R; c += 64)
    for (int s = 0; s < t.splits; ++s) {
      const int i = c >> 4;
      tr += part[s * tiles + (tri_tiles(i) + i) * 256 + (c & 15) * 17];
    }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  return 1.0 / (sqrt(tr) + p.eps);
}
__global__ __launch_bounds__(NT) void k_muon_long_sum(MuonArgs p, int per) {
  long mat;
  int tile, i, j;
  const MuonTensor& t = long_matrix(p, mat, tile, per);
  if (tile >= tri_tiles(t.R / 16)) return;
  tri(tile, i, j);
  const double inv = long_inv(p, t, mat), inv2 = inv * inv;
  const long tiles = (long)tri_tiles(t.R / 16) * 256;
  double* S = long_slot(t, mat, 0);
  const double* part = S - t.splits * tiles + tile * 256;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    double x = 0.0;
    for (int s = 0; s < t.splits; ++s) x += part[s * tiles + v * 64 + lane];
    const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
    S[(long)r * t.R + c] = x * inv2;
    S[(long)c * t.R + r] = x * inv2;
  }
}
// z = fc x y + fb x + fa I (all symmetric); out: to q, over the norm, in fp32
__global__ __launch_bounds__(NT) void k_muon_long_mul(MuonArgs p, int per, int x, int y, int z, double fc, double fb, double fa, int out) {
  long mat;
  int tile, i, j;
  const MuonTensor& t = long_matrix(p, mat, tile, per);
  if (tile >= tri_tiles(t.R / 16)) return;
  tri(tile, i, j);
  const int lane = threadIdx.x & 63;
  const double *X = long_slot(t, mat, x), *Y = long_slot(t, mat, y);
  // symmetric: a row block is read as a column block, 16 neighbours
  const double* a = X + (long)(lane >> 4) * t.R + 16 * i + (lane & 15);
  const double* b = Y + (long)(lane >> 4) * t.R + 16 * j + (lane & 15);
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int k4 = 0; k4 < t.R; k4 += 4)
    acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a[(long)k4 * t.R], b[(long)k4 * t.R], acc, 0, 0, 0);
  double* Z = long_slot(t, mat, z);
  const double inv = out ? long_inv(p, t, mat) : 0.0;
  float* q = t.q + mat * (long)t.R * t.R;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
    const double d = fma(fc, acc[v], fb != 0.0 ? fma(fb, X[(long)r * t.R + c], r == c ? fa : 0.0) : 0.0);
    if (out) {
      q[(long)r * t.R + c] = (float)(d * inv);
      q[(long)c * t.R + r] = (float)(d * inv);
    } else {
      Z[(long)r * t.R + c] = d;
      Z[(long)c * t.R + r] = d;
    }
  }
}

// Q U for a part of the long side, and the parameters.  A wave keeps its columns
// of Q in registers; the results go back to where U was in LDS, so that the
// parameters are read and written in the order of memory.
template <class PT, class GT, int RB, bool TALL>
__device__ __forceinline__ void apply(const MuonArgs& p, const MuonTensor& t, long mat, int s, float* S) {
  using Sh = Share<RB, TALL, apply_chunk(RB)>;
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const float lr = p.control != nullptr ? p.control->lr : p.lr;
  const float step = lr * (p.rms * sqrtf((float)t.L)), decay = lr * p.weight_decay;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int KT = RB / 16;                        // blocks of Q's rows
  constexpr int WI = RB <= 64 ? RB / 16 : NW;        // waves along the short side
  constexpr int IW = RB / 16 / WI;                   // blocks of it a wave
  constexpr int JW = (Sh::CHUNK / 16) * WI / NW;     // blocks of the chunk a wave
  const int nt = t.R / 16, wi = w % WI, wj = w / WI * JW;
  Sh sh;
  sh.init(t);
  const int l_begin = s * t.span;
  int left = min(t.L - l_begin, t.span);
  const bool vec = t.vec != 0;
  const long at = mat * (long)t.r * t.L + (TALL ? (long)l_begin * t.r : l_begin);
  const GT* g = (const GT*)t.grad + at;
  const float* mo = t.momentum + at;
  float* ma = t.master != nullptr ? t.master + at : nullptr;
  PT* pa = (PT*)t.param + at;
  f32x4 gv[Sh::N], mv[Sh::N], pv[Sh::N];
  auto fetch = [&](int have) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      gv[i] = load4(g + sh.at[i], vec, sh.have(i, have));
      mv[i] = load4(mo + sh.at[i], vec, sh.have(i, have));
    }
  };
  fetch(left);
  float q[IW][KT][4];
#pragma unroll
  for (int i = 0; i < IW; ++i)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * kt + 4 * e + (lane >> 4), col = 16 * (wi + WI * i) + (lane & 15);
        q[i][kt][e] = kt < nt && wi + WI * i < nt ? t.q[mat * (long)t.R * t.R + (long)row * t.R + col] : 0.0f;
      }
  const float* Sf = S + (lane >> 4) * Sh::KS + (lane & 15) * Sh::LS + 16 * wj * Sh::LS;
  for (; left > 0; left -= Sh::CHUNK) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      f32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = p.nesterov ? fmaf(p.momentum, mv[i][e], gv[i][e] * gs) : mv[i][e];
      if (sh.lds[i] >= 0) *(f32x4*)(S + sh.lds[i]) = u;
      const int have = sh.have(i, left);
      pv[i] = ma != nullptr ? load4(ma + sh.at[i], vec, have) : load4(pa + sh.at[i], vec, have);
    }
    __syncthreads();
    g += sh.step;
    mo += sh.step;
    if (left > Sh::CHUNK) fetch(left - Sh::CHUNK);
    f32x4 acc[IW][JW];
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < JW; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      if (kt < nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[JW];
#pragma unroll
          for (int j = 0; j < JW; ++j) y[j] = Sf[(16 * kt + 4 * e) * Sh::KS + 16 * j * Sh::LS];
          // a lane's four results are neighbours in memory: along the short side where the tensor is tall
#pragma unroll
          for (int i = 0; i < IW; ++i)
#pragma unroll
            for (int j = 0; j < JW; ++j)
              acc[i][j] = TALL ? __builtin_amdgcn_mfma_f32_16x16x4f32(q[i][kt][e], y[j], acc[i][j], 0, 0, 0)
                               : __builtin_amdgcn_mfma_f32_16x16x4f32(y[j], q[i][kt][e], acc[i][j], 0, 0, 0);
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < JW; ++j)
        if (wi + WI * i < nt) {
          const int c = 16 * (wi + WI * i), l = 16 * (wj + j);
          const int a = TALL ? l : c, b = TALL ? c : l;
          *(f32x4*)(S + (a + (lane & 15)) * Sh::PITCH + b + 4 * (lane >> 4)) = acc[i][j];
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      if (sh.lds[i] < 0) continue;
      const int have = sh.have(i, left);
      const f32x4 o = *(const f32x4*)(S + sh.lds[i]);
      f32x4 x = pv[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] -= fmaf(step, o[e], decay * x[e]);
      if (ma != nullptr) store4(ma + sh.at[i], vec, have, x);
      store4(pa + sh.at[i], vec, have, x);
    }
    __syncthreads();
    pa += sh.step;
    if (ma != nullptr) ma += sh.step;
  }
}

template <class PT, class GT, int RB>
__global__ __launch_bounds__(NT, RB <= 128 ? 4 : 2) void k_muon_apply(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  int ti, s;
  long mat;
  find(p, blockIdx.x, ti, mat, s);
  const MuonTensor& t = p.t[ti];
  if (t.tall)
    apply<PT, GT, RB, true>(p, t, mat, s, (float*)smem);
  else
    apply<PT, GT, RB, false>(p, t, mat, s, (float*)smem);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int round16(int r) { return (r + 15) / 16 * 16; }

// Entries of the long side that a workgroup takes: enough workgroups for the
// chip over all tensors of the call, in whole chunks.
int span_of(const moe_muon_tensor* t, int32_t count, int cus) {
  double total = 0;
  for (int32_t i = 0; i < count; ++i)
    if (t[i].batch > 0) total += (double)t[i].batch * (t[i].m > t[i].n ? t[i].m : t[i].n);
  const double span = total / (4.0 * cus);
  return span < 64 ? 64 : span > 0x1p30 ? 1 << 30 : (int)((span + 63) / 64) * 64;
}

moe_status check_desc(const moe_muon_desc* d, const moe_muon_tensor* t, int32_t count) {
  if (d == nullptr || count < 0 || (count > 0 && t == nullptr)) return MOE_ERR_INVALID;
  for (int32_t ty : {d->param_type, d->grad_type})
    if (ty != MOE_TYPE_F32 && ty != MOE_TYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if ((d->nesterov != 0 && d->nesterov != 1) || d->rounds < 1) return MOE_ERR_INVALID;
  if (d->rounds > 16) return MOE_ERR_UNSUPPORTED;
  auto ok = [](double v) { return std::isfinite((float)v); };
  if (!ok(d->lr) || !ok(d->momentum) || !ok(d->weight_decay) || !ok(d->rms) || !ok(d->eps) || !ok(d->grad_scale) ||
      !ok(d->a) || !ok(d->b) || !ok(d->c))
    return MOE_ERR_INVALID;
  if (d->lr < 0 || d->weight_decay < 0 || d->rms < 0 || d->momentum < 0 || !((float)d->momentum < 1.0f) ||
      !((float)d->eps > 0.0f))
    return MOE_ERR_INVALID;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].batch < 0) return MOE_ERR_INVALID;
    if (t[i].batch == 0) continue;
    if (t[i].m < 1 || t[i].n < 1) return MOE_ERR_INVALID;
    const int64_t mn = (int64_t)t[i].m * t[i].n;
    if ((t[i].m < t[i].n ? t[i].m : t[i].n) > MAX_SHORT || mn >= (int64_t)1 << 31 || t[i].batch > (int64_t)1 << 18 ||
        t[i].batch * mn >= (int64_t)1 << 40)
      return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

struct Plan {
  int r, L, R, splits, span;
  size_t part, q;  // bytes
};
Plan plan_of(const moe_muon_tensor& t, int span) {
  Plan p;
  p.r = t.m < t.n ? t.m : t.n;
  p.L = t.m < t.n ? t.n : t.m;
  p.R = round16(p.r);
  p.span = span;
  p.splits = (p.L + span - 1) / span;
  p.part = (size_t)t.batch * part_size(p.R, p.splits) * 8;
  p.q = ((size_t)t.batch * p.R * p.R * 4 + 15) / 16 * 16;
  return p;
}

// LDS of a chunk of U for short sides up to RB, either way round
constexpr int lds_of(int RB, int chunk) { return cmax(pitch_of(RB) * chunk, pitch_of(chunk) * RB) * 4; }

template <class GT, int RB>
hipError_t launch_gram(const MuonArgs& p, hipStream_t st) {
  MOE_LAUNCH_AS("k_muon_gram", (k_muon_gram<GT, RB>), dim3((unsigned)p.groups), dim3(NT), lds_of(RB, gram_chunk(RB)), st, p);
  return hipGetLastError();
}
template <class PT, class GT, int RB>
hipError_t launch_apply(const MuonArgs& p, hipStream_t st) {
  MOE_LAUNCH_AS("k_muon_apply", (k_muon_apply<PT, GT, RB>), dim3((unsigned)p.groups), dim3(NT), lds_of(RB, apply_chunk(RB)), st, p);
  return hipGetLastError();
}
hipError_t launch_long_rounds(const MuonArgs& p, int R, hipStream_t st) {
  const int per = (tri_tiles(R / 16) + NW - 1) / NW;
  const dim3 g((unsigned)(p.matrices * per)), b(NT);
  MOE_LAUNCH(k_muon_long_sum, g, b, 0, st, p, per);
  auto mul = [&](int x, int y, int z, double c, double fb, double a, int out) {
    MOE_LAUNCH(k_muon_long_mul, g, b, 0, st, p, per, x, y, z, c, fb, a, out);
  };
  int S = 0, T = 1, Q = 2, spare[3] = {3, 4, 5};
  for (int n = 0; n < p.rounds; ++n) {
    const bool last = n + 1 == p.rounds;
    const int P = spare[0], next = spare[1];
    if (n == 0) {
      mul(S, S, Q, p.c, p.b, p.a, last);  // P is Q
      if (!last) {
        mul(S, Q, T, 1.0, 0.0, 0.0, 0);
        mul(T, Q, S, 1.0, 0.0, 0.0, 0);
      }
      continue;
    }
    mul(S, S, P, p.c, p.b, p.a, 0);
    mul(P, Q, next, 1.0, 0.0, 0.0, last);
    spare[1] = Q;
    Q = next;
    if (!last) {
      mul(S, P, T, 1.0, 0.0, 0.0, 0);
      mul(T, P, S, 1.0, 0.0, 0.0, 0);
    }
  }
  return hipGetLastError();
}

template <int RB>
hipError_t prepare_kernels() {
  static PerDeviceOnce once;
  return once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_muon_gram<uint16_t, RB>, lds_of(RB, gram_chunk(RB)));
    ai.lds((const void*)k_muon_gram<float, RB>, lds_of(RB, gram_chunk(RB)));
    if constexpr (RB <= SHORT_R) ai.lds((const void*)k_muon_rounds<RB>, 2 * tri_tiles(RB / 16) * Rounds<RB>::TILE);
    ai.lds((const void*)k_muon_apply<uint16_t, uint16_t, RB>, lds_of(RB, apply_chunk(RB)));
    ai.lds((const void*)k_muon_apply<uint16_t, float, RB>, lds_of(RB, apply_chunk(RB)));
    ai.lds((const void*)k_muon_apply<float, uint16_t, RB>, lds_of(RB, apply_chunk(RB)));
    ai.lds((const void*)k_muon_apply<float, float, RB>, lds_of(RB, apply_chunk(RB)));
    return ai.err;
  });
}

// R: the longest short side of the tensors
template <int RB>
hipError_t launch_step(const MuonArgs& p, int R, bool pbf, bool gbf, hipStream_t st) {
  hipError_t e = prepare_kernels<RB>();
  if (e == hipSuccess) e = gbf ? launch_gram<uint16_t, RB>(p, st) : launch_gram<float, RB>(p, st);
  if (e != hipSuccess) return e;
  if constexpr (RB <= SHORT_R) {
    MOE_LAUNCH_AS("k_muon_rounds", k_muon_rounds<RB>, dim3((unsigned)p.matrices), dim3(NT), 2 * tri_tiles(R / 16) * Rounds<RB>::TILE, st, p);
    e = hipGetLastError();
  } else {
    e = launch_long_rounds(p, R, st);
  }
  if (e != hipSuccess) return e;
  if (pbf) return gbf ? launch_apply<uint16_t, uint16_t, RB>(p, st) : launch_apply<uint16_t, float, RB>(p, st);
  return gbf ? launch_apply<float, uint16_t, RB>(p, st) : launch_apply<float, float, RB>(p, st);
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

moe_status moe_muon_workspace_size(const moe_muon_desc* d, const moe_muon_tensor* t, int32_t count, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID;
  const moe_status s = check_desc(d, t, count);
  if (s != MOE_OK) return s;
  int cus = 0;
  if (device_cus(cus) != hipSuccess) return MOE_ERR_HIP;
  const int span = span_of(t, count, cus);
  size_t n = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].batch == 0) continue;
    const Plan p = plan_of(t[i], span);
    n += p.part + p.q;
  }
  *bytes = n;
  return MOE_OK;
}

moe_status moe_muon_step(const moe_muon_desc* d, const moe_muon_tensor* t, int32_t count, void* workspace,
                         size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const moe_status s = moe_muon_workspace_size(d, t, count, &need);
  if (s != MOE_OK) return s;
  if (d->control != nullptr && !aligned(d->control, 4)) return MOE_ERR_INVALID;
  const size_t ps = d->param_type == MOE_TYPE_F32 ? 4 : 2, gs = d->grad_type == MOE_TYPE_F32 ? 4 : 2;
  bool any = false, masters = false;
  for (int32_t i = 0; i < count; ++i) {
    const moe_muon_tensor& x = t[i];
    if (x.batch == 0) continue;
    if (!aligned16(x.param) || !aligned16(x.grad) || !aligned16(x.momentum)) return MOE_ERR_INVALID;
    if (x.master != nullptr && (!aligned16(x.master) || d->param_type != MOE_TYPE_BF16)) return MOE_ERR_INVALID;
    if (any && masters != (x.master != nullptr)) return MOE_ERR_INVALID;
    any = true;
    masters = x.master != nullptr;
    const size_t n = (size_t)x.batch * x.m * x.n;
    const Range r[] = {rng(x.param, n * ps), rng(x.master, n * 4), rng(x.momentum, n * 4), rng(x.grad, n * gs),
                       rng(workspace, need)};
    for (int a = 0; a < 5; ++a)
      for (int b = 0; b < a; ++b)
        if (overlap(r[a], r[b])) return MOE_ERR_INVALID;
  }
  if (!any) return MOE_OK;
  if (!aligned16(workspace)) return MOE_ERR_INVALID;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int cus = 0;
  if (device_cus(cus) != hipSuccess) return MOE_ERR_HIP;
  const int span = span_of(t, count, cus);
  MuonArgs p{};
  p.nesterov = d->nesterov;
  p.rounds = d->rounds;
  p.lr = (float)d->lr;
  p.momentum = (float)d->momentum;
  p.weight_decay = (float)d->weight_decay;
  p.grad_scale = (float)d->grad_scale;
  p.rms = (float)d->rms;
  p.a = d->a;
  p.b = d->b;
  p.c = d->c;
  p.eps = d->eps;
  p.control = d->control;
  // short sides up to SHORT_R, then longer ones: the launches of a group take one
  // kernel each
  char* at = (char*)workspace;
  int R = 0;
  const bool pbf = d->param_type == MOE_TYPE_BF16, gbf = d->grad_type == MOE_TYPE_BF16;
  const hipStream_t st = (hipStream_t)stream;
  auto flush = [&]() {
    if (p.count == 0) return hipSuccess;
    const hipError_t e = R <= 64        ? launch_step<64>(p, R, pbf, gbf, st)
                         : R <= SHORT_R ? launch_step<SHORT_R>(p, R, pbf, gbf, st)
                                        : launch_step<MAX_SHORT>(p, R, pbf, gbf, st);
    p.count = R = 0;
    p.groups = p.matrices = 0;
    return e;
  };
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t i = 0; i < count; ++i) {
      const moe_muon_tensor& x = t[i];
      if (x.batch == 0) continue;
      const Plan pl = plan_of(x, span);
      if ((pl.R > SHORT_R) != (pass == 1)) continue;
      // a launch holds fewer than 2^32 threads; long rounds take 17 workgroups a matrix
      if (p.count == TENSORS || p.groups + x.batch * pl.splits >= (int64_t)1 << 23 ||
          (pass == 1 && p.matrices + x.batch >= (int64_t)1 << 18))
        if (flush() != hipSuccess) return MOE_ERR_HIP;
      MuonTensor& m = p.t[p.count++];
      const bool tall = x.m > x.n;
      m = MuonTensor{x.param, x.master, x.grad, x.momentum, p.groups, p.matrices, (double*)at, (float*)(at + pl.part),
                     pl.r, pl.L, tall, pl.R, pl.splits, pl.span, (tall ? pl.r : pl.L) % 4 == 0};
      at += pl.part + pl.q;
      p.groups += x.batch * pl.splits;
      p.matrices += x.batch;
      if (pl.R > R) R = pl.R;
    }
    if (flush() != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}

}  // extern "C"
