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
// sums added in a fixed order), the rounds (a workgroup a matrix; beyond 128 rows a
// launch for each product), Q U and the parameters.  Production factors (50.8 M
// parameters): 551 us; the bytes alone 160-200 us, fp64 products 98 + 112, fp32 85.
#include <cmath>
#include <type_traits>

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
constexpr int NT = 512, NW = 8;

struct MuonTensor {
  void* param;
  float* master;
  const void* grad;
  float* momentum;
  long first;        // this tensor's first workgroup in a launch over splits
  long matrix0;      // index of its first matrix
  double* part;      // a matrix: partial sums of S0 [splits][lower tiles], then (long short sides) the rounds' matrices
  float* q;          // a matrix: Q over U's norm [R][R], and what U is multiplied by (see Norm)
  int r, L, tall;    // tall: stored [L, r]
  int R;             // r in whole tiles of 16
  int splits, span;  // workgroups along L, entries each
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

// Four neighbours in memory as they are loaded (converted where they are used, so
// that nothing waits for a load before that).
template <class T>
struct Four {
  typename std::conditional<sizeof(T) == 4, f32x4, u32x2>::type v;
  __device__ __forceinline__ f32x4 get() const {
    if constexpr (sizeof(T) == 4)
      return v;
    else
      return f32x4{bf2f(v[0] & 0xffffu), bf2f(v[0] >> 16), bf2f(v[1] & 0xffffu), bf2f(v[1] >> 16)};
  }
  __device__ __forceinline__ void set(f32x4 x) {
    if constexpr (sizeof(T) == 4)
      v = x;
    else
      v = u32x2{pack2(x[0], x[1]), pack2(x[2], x[3])};
  }
};
// A tensor's part of the long side, a chunk at a time.  VEC: groups of four are
// whole and a matrix is within 2 GB (fewer than 2^29 elements): they go through a
// buffer descriptor, which reads zeros for and does not write what is not there,
// so that nothing branches and the loads in flight stay countable.  Else element
// by element: what is not there is read from the tensor's start, without a branch,
// and masked by the caller.
template <bool VEC, class T>
struct Part {
  T* base;
  const T* safe;
  long left;  // elements from base to the matrix's end
  rsrc_t r;
  __device__ __forceinline__ void init(const T* tensor, long matrix, long size, long at) {
    base = const_cast<T*>(tensor) + matrix + at;
    safe = tensor;
    left = size - at;
    next(0);
  }
  __device__ __forceinline__ void next(long step) {
    base += step;
    left -= step;
    if constexpr (VEC) r = make_rsrc(base, left > 0 ? (uint64_t)left * sizeof(T) : 0);
  }
  // (none: past the extent of either type, 2^30 bytes for two a piece)
  __device__ __forceinline__ static int place(int at, int have) {
    return have > 0 ? at * (int)sizeof(T) : (int)(OFF_NONE / (4 / sizeof(T)));
  }
  __device__ __forceinline__ void load(Four<T>& f, int at, int have) const {
    if constexpr (VEC) {
      if constexpr (sizeof(T) == 4)
        f.v = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, place(at, have), 0, 0));
      else
        f.v = __builtin_amdgcn_raw_buffer_load_b64(r, place(at, have), 0, 0);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f.v[e] = *(e < have ? base + at + e : safe);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        f.v[e] = (uint32_t)*(2 * e < have ? base + at + 2 * e : safe) |
                 (uint32_t)*(2 * e + 1 < have ? base + at + 2 * e + 1 : safe) << 16;
    }
  }
  __device__ __forceinline__ void store(int at, int have, f32x4 x) const {
    Four<T> f;
    f.set(x);
    if constexpr (VEC) {
      if constexpr (sizeof(T) == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f.v), r, place(at, have), 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(f.v, r, place(at, have), 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < have) {
          if constexpr (sizeof(T) == 4)
            base[at + e] = f.v[e];
          else
            base[at + e] = (T)(f.v[e >> 1] >> (16 * (e & 1)));
        }
    }
  }
};

// What a thread moves of each chunk (CHUNK entries of the long side): groups of
// four neighbours in memory.  A chunk lies in LDS as in memory: [l][c] of a tall
// tensor, [c][l] of a wide one.
template <int RB, bool TALL, int CHUNK_, int PITCH_>
struct Share {
  static constexpr int CHUNK = CHUNK_, PITCH = PITCH_, N = cmax(RB * CHUNK / (4 * NT), 1);
  // LDS steps along the short and the long side
  static constexpr int KS = TALL ? 1 : PITCH, LS = TALL ? PITCH : 1;
  static constexpr int SIZE = (TALL ? CHUNK : RB) * PITCH;  // elements in LDS; a lane's four more behind them for what is nowhere
  int lds[N];    // LDS place
  int first[N];  // the group's first entry of the chunk's long side (2^30: it is not there)
  int live[N];   // tall: entries of the short side from here on
  int at[N];     // element in the chunk (a matrix has fewer than 2^31)
  __device__ __forceinline__ void init(const MuonTensor& t) {
    const int B = TALL ? t.R : CHUNK, A = TALL ? CHUNK : t.R;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int g = threadIdx.x + i * NT, a = g / (B / 4), b = 4 * (g - a * (B / 4));
      const bool there = a < A && (TALL ? b < t.r : a < t.r);
      lds[i] = a < A ? a * PITCH + b : SIZE + 4 * (threadIdx.x & 63);
      at[i] = there ? a * (TALL ? t.r : t.L) + b : 0;
      first[i] = there ? (TALL ? a : b) : 1 << 30;
      live[i] = t.r - b;
    }
  }
  // elements from one chunk to the next
  __device__ __forceinline__ static long step(const MuonTensor& t) { return TALL ? (long)CHUNK * t.r : CHUNK; }
  // of group i, the elements there are in a chunk with `left` entries
  __device__ __forceinline__ int have(int i, int left) const {
    return TALL ? (first[i] < left ? live[i] : 0) : left - first[i];
  }
  template <bool VEC>
  __device__ __forceinline__ static f32x4 only(f32x4 x, int have) {
    if constexpr (VEC) return x;  // zeros were read
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < have ? x[e] : 0.0f;
    return x;
  }
};
// Entries of the long side in LDS at a time, and pitches that keep the operands'
// reads free of bank conflicts: S0 reads doubles, 16 of the short side by 4 of the
// long side; Q U reads floats, 16 of the long side by 4 of the short side.
__device__ __host__ constexpr int gram_chunk(int RB) { return RB <= 16 ? 128 : RB <= 128 ? 64 : 32; }
__device__ __host__ constexpr int gram_pitch(int RB, bool tall) { return tall ? (RB + 15) / 32 * 32 + 16 : gram_chunk(RB) + 2; }
__device__ __host__ constexpr int apply_chunk(int RB) { return RB <= 16 ? 128 : RB <= 64 ? 64 : 32; }
__device__ __host__ constexpr int apply_pitch(int RB, bool tall) { return tall ? (RB + 43) / 64 * 64 + 20 : apply_chunk(RB) + 16; }

// Tile t of the lower triangle of tiles.
__device__ __forceinline__ void tri(int t, int& i, int& j) {
  i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  j = t - i * (i + 1) / 2;
}
__device__ __host__ constexpr int tri_tiles(int n) { return n * (n + 1) / 2; }

// 1 / (|U| + eps) in two factors: a power of two for U, in fp32, and the rest for
// Q before its rounding to fp32.  As one factor of Q it leaves fp32's range where
// |U| is within a^rounds of either end (a matrix of zeros beside a small eps:
// infinities times zero).  Powers of two change no result inside the range.
struct Norm {
  double all, of_q;  // of_q: 0 for a matrix of zeros, whatever the polynomial's value there
  float of_u;
  __device__ __forceinline__ Norm(double squares, double eps) {
    const double n = sqrt(squares) + eps;
    all = 1.0 / n;
    const int e = min(max((int)(__builtin_bit_cast(uint64_t, n) >> 52) - 1023, -126), 126);  // NaN, infinity: 126
    of_u = __uint_as_float((uint32_t)(127 - e) << 23);
    const double up = __builtin_bit_cast(double, (uint64_t)(1023 + e) << 52);
    // infinite squares: S is NaN, and Q has to stay so
    of_q = squares == 0.0 ? 0.0 : (squares < __builtin_inf() ? all : 1.0) * up;
  }
};
__device__ __forceinline__ float over_norm(double q, double of_q) { return of_q != 0.0 ? (float)(q * of_q) : 0.0f; }
// A matrix's part of q, in floats.
__device__ __host__ constexpr long q_size(int R) { return (long)R * R + 4; }

// Where a matrix's part of the workspace begins.
constexpr int SHORT_R = 128;   // up to here the rounds run in LDS
constexpr int LONG_SLOTS = 6;  // beyond, they have matrices behind the partial sums
__device__ __host__ constexpr long part_size(int R, int splits) {
  return (long)splits * tri_tiles(R / 16) * 256 + (R > SHORT_R ? (long)LONG_SLOTS * R * R + 2 : 0);
}
__device__ __forceinline__ long part_at(const MuonTensor& t, long mat) { return mat * part_size(t.R, t.splits); }

// The new momentum, and S0 of a part of the long side as lower tiles of 16 x 16.
// The next chunk's loads are in flight while this one is multiplied.  U goes to
// LDS as doubles, so that no instruction stands between the reads and the matrix
// instructions: on the fp64 matrix path vector instructions take their time from
// it (each about 4 clocks of the 72 that a product takes).
// N: tiles of the waves, at most; what a wave has less is multiplied and not stored.
// 195 matrices of 128 rows (50.8 M elements): 171 us; without the loads and stores
// 150, without the products 110, the lower tiles at the fp64 rate 98.
template <class GT, int RB, bool TALL, bool VEC, int N>
__device__ __forceinline__ void gram(const MuonArgs& p, const MuonTensor& t, long mat, int s, double* S) {
  using Sh = Share<RB, TALL, gram_chunk(RB), gram_pitch(RB, TALL)>;
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tiles = tri_tiles(t.R / 16);
  constexpr bool ALONG = RB <= 16;                         // one tile: the waves share its chunk
  constexpr int PART = ALONG ? Sh::CHUNK / NW : Sh::CHUNK;  // entries of a chunk that a wave multiplies
  Sh sh;
  sh.init(t);
  const int l_begin = s * t.span;
  int left = min(t.L - l_begin, t.span);
  const long size = (long)t.r * t.L, at = TALL ? (long)l_begin * t.r : l_begin;
  Part<VEC, GT> g;
  Part<VEC, float> mo;
  g.init((const GT*)t.grad, mat * size, size, at);
  mo.init(t.momentum, mat * size, size, at);
  Four<GT> gv[Sh::N];
  Four<float> mv[Sh::N];
  auto fetch = [&](int have) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      g.load(gv[i], sh.at[i], sh.have(i, have));
      mo.load(mv[i], sh.at[i], sh.have(i, have));
    }
  };
  f64x4 acc[cmax(N, 1)];
  int xi[cmax(N, 1)], yj[cmax(N, 1)];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    int i = 0, j = 0;
    if (!ALONG && w + NW * q < tiles) tri(w + NW * q, i, j);
    const int lo = (lane >> 4) * Sh::LS + (lane & 15) * Sh::KS + (ALONG ? w * PART * Sh::LS : 0);
    xi[q] = lo + 16 * i * Sh::KS;
    yj[q] = lo + 16 * j * Sh::KS;
    acc[q] = f64x4{0.0, 0.0, 0.0, 0.0};
  }
  fetch(left);
  for (; left > 0; left -= Sh::CHUNK) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      const f32x4 x = gv[i].get();
      f32x4 m = mv[i].get(), u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = x[e] * gs;
        m[e] = fmaf(p.momentum, m[e], y);
        u[e] = p.nesterov ? fmaf(p.momentum, m[e], y) : m[e];
      }
      mo.store(sh.at[i], sh.have(i, left), m);
      u = Sh::template only<VEC>(u, sh.have(i, left));
      typedef double f64x2 __attribute__((ext_vector_type(2)));
      *(f64x2*)(S + sh.lds[i]) = f64x2{u[0], u[1]};
      *(f64x2*)(S + sh.lds[i] + 2) = f64x2{u[2], u[3]};
    }
    __syncthreads();
    g.next(Sh::step(t));
    mo.next(Sh::step(t));
    fetch(left - Sh::CHUNK);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (N > 0) {
      // operands are read D products ahead
      constexpr int D = N < 4 ? 4 : N < 6 ? N : 6, STEPS = PART / 4 * N;
      double x[D], y[D];
#pragma unroll
      for (int n = -D; n < STEPS; ++n) {
        const int b = (n + D) % D;
        if (n >= 0) acc[n % N] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[b], y[b], acc[n % N], 0, 0, 0);
        if (n + D < STEPS) {
          x[b] = S[xi[(n + D) % N] + (n + D) / N * 4 * Sh::LS];
          y[b] = S[yj[(n + D) % N] + (n + D) / N * 4 * Sh::LS];
        }
        if (n >= 0) __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
  }
  double* out = t.part + part_at(t, mat) + s * (long)(tiles * 256);
  if constexpr (ALONG) {
#pragma unroll
    for (int v = 0; v < 4; ++v) S[w * 256 + v * 64 + lane] = acc[0][v];
    __syncthreads();
    if (threadIdx.x < 256) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) sum += S[i * 256 + threadIdx.x];
      out[threadIdx.x] = sum;
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (w + NW * q < tiles)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[(w + NW * q) * 256 + v * 64 + lane] = acc[q][v];  // row 4 v + lane / 16 of the tile
}
template <class GT, int RB, bool TALL, bool VEC>
__device__ __forceinline__ void gram_of(const MuonArgs& p, const MuonTensor& t, long mat, int s, double* S) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = (tri_tiles(t.R / 16) - w + NW - 1) / NW;
  if constexpr (RB <= 16) {
    gram<GT, RB, TALL, VEC, 1>(p, t, mat, s, S);
  } else if constexpr (RB <= 64) {
    if (n >= 2) gram<GT, RB, TALL, VEC, 2>(p, t, mat, s, S);
    else if (n == 1) gram<GT, RB, TALL, VEC, 1>(p, t, mat, s, S);
    else gram<GT, RB, TALL, VEC, 0>(p, t, mat, s, S);
  } else if constexpr (RB <= 128) {
    if (n >= 5) gram<GT, RB, TALL, VEC, 5>(p, t, mat, s, S);
    else if (n == 4) gram<GT, RB, TALL, VEC, 4>(p, t, mat, s, S);
    else gram<GT, RB, TALL, VEC, 3>(p, t, mat, s, S);
  } else {
    if (n > 12) gram<GT, RB, TALL, VEC, 17>(p, t, mat, s, S);
    else if (n > 7) gram<GT, RB, TALL, VEC, 12>(p, t, mat, s, S);
    else gram<GT, RB, TALL, VEC, 7>(p, t, mat, s, S);
  }
}

template <class GT, int RB, bool VEC>
__global__ __launch_bounds__(NT, RB <= 128 ? 4 : 2) void k_muon_gram(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  int ti, s;
  long mat;
  find(p, blockIdx.x, ti, mat, s);
  const MuonTensor& t = p.t[ti];
  if (t.tall)
    gram_of<GT, RB, true, VEC>(p, t, mat, s, (double*)smem);
  else
    gram_of<GT, RB, false, VEC>(p, t, mat, s, (double*)smem);
}

// ---------------------------------------------------------------------------
// rounds
// ---------------------------------------------------------------------------
__device__ __forceinline__ const MuonTensor& find_matrix(const MuonArgs& p, long m, long& mat) {
  int ti = 0;
  while (ti + 1 < p.count && m >= p.t[ti + 1].matrix0) ++ti;
  mat = m - p.t[ti].matrix0;
  return p.t[ti];
}

// Up to 16 rows: one wave, all in registers.  Element v of a lane's result is row
// 4 v + lane / 16, column lane % 16, which is the operand of k-step v on either
// side, the matrices being symmetric.
__device__ __forceinline__ f64x4 mul16(f64x4 x, f64x4 y) {
  f64x4 z = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f64_16x16x4f64(x[s], y[s], z, 0, 0, 0);
  return z;
}
__global__ __launch_bounds__(64) void k_muon_rounds16(MuonArgs p) {
  long mat;
  const MuonTensor& t = find_matrix(p, blockIdx.x, mat);
  const int lane = threadIdx.x;
  const double* part = t.part + part_at(t, mat) + lane;
  f64x4 S = {0.0, 0.0, 0.0, 0.0}, Q = S, one = S;
#pragma unroll 4
  for (int s = 0; s < t.splits; ++s)
#pragma unroll
    for (int v = 0; v < 4; ++v) S[v] += part[s * 256 + v * 64];
  double tr = 0.0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    one[v] = 4 * v + (lane >> 4) == (lane & 15) ? 1.0 : 0.0;
    tr += one[v] != 0.0 ? S[v] : 0.0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  const Norm norm(tr, p.eps);
  S *= norm.all * norm.all;
  for (int n = 0; n < p.rounds; ++n) {
    f64x4 P = mul16(S, S);
#pragma unroll
    for (int v = 0; v < 4; ++v) P[v] = fma(p.c, P[v], fma(p.b, S[v], p.a * one[v]));
    Q = n == 0 ? P : mul16(P, Q);
    if (n + 1 < p.rounds) S = mul16(mul16(S, P), P);
  }
  float* out = t.q + mat * q_size(16);
#pragma unroll
  for (int v = 0; v < 4; ++v) out[v * 64 + lane] = over_norm(Q[v], norm.of_q);
  if (lane == 0) out[256] = norm.of_u;
}

// 16 B rows, B from 2 to 8: two matrices as lower tiles of 16 x 16 in LDS, at a
// pitch of 17, at which a column and a row of 16 lie in 16 different pairs of
// banks.  A wave's tiles are w, w + 8, ... of the lower triangle, known when this
// is compiled for each wave, so that every operand is one LDS read at a fixed
// offset: on the fp64 matrix path each vector instruction takes its time from the
// products (addresses formed for each read: 250 us for 195 matrices of 128 rows).
// 17 products of lower tiles for five rounds: 210 us for the 195 matrices on as many
// of the 256 CUs; at the fp64 rate a matrix alone takes 147 us of a CU.
template <int B>
struct Rounds {
  static constexpr int TILES = tri_tiles(B), MT = (TILES + NW - 1) / NW;
  static constexpr int PITCH = 17 * 8, TILE = 16 * PITCH, HIGH = 18;  // offsets from tile HIGH on have a base of their own
  static constexpr int LDS = 2 * TILES * TILE;
  struct Bases {
    const char *c[2], *r[2];  // of columns and of rows of a tile
  };
  __device__ static constexpr int row_of(int t) {
    int i = 0;
    while (tri_tiles(i + 1) <= t) ++i;
    return i;
  }
  // 16 rows of block I at k = 16 KT + 4 s + lane / 16: from a column of tile (I, KT),
  // or above the diagonal from a row of (KT, I)
  template <int I, int KT, int SS>
  __device__ static __forceinline__ double get(const Bases& m) {
    constexpr int t = I >= KT ? tri_tiles(I) + KT : tri_tiles(KT) + I, h = t >= HIGH ? 1 : 0;
    return *(const double*)((I >= KT ? m.c[h] : m.r[h]) + (t - h * HIGH) * TILE + SS * (I >= KT ? 32 : 4 * PITCH));
  }
  template <int W, int STEP, int Q>
  __device__ static __forceinline__ void read(const Bases& X, const Bases& Y, double (&v)[2 * MT]) {
    constexpr int t = W + NW * Q;
    if constexpr (Q < MT) {
      if constexpr (t < TILES && STEP < 4 * B) {
        constexpr int i = row_of(t), j = t - tri_tiles(i);
        v[Q] = get<i, STEP / 4, STEP % 4>(X);
        v[MT + Q] = get<j, STEP / 4, STEP % 4>(Y);
      }
    }
  }
  template <int W, int Q>
  __device__ static __forceinline__ void first(const Bases& X, const Bases& Y, double (&v)[2 * MT]) {
    if constexpr (Q < MT) {
      read<W, 0, Q>(X, Y, v);
      first<W, Q + 1>(X, Y, v);
    }
  }
  // a pair's operands of the next step are read behind its product
  template <int W, int STEP, int Q>
  __device__ static __forceinline__ void steps(const Bases& X, const Bases& Y, double (&cur)[2 * MT], double (&nxt)[2 * MT], f64x4 (&z)[MT]) {
    if constexpr (STEP < 4 * B) {
      if constexpr (Q < MT && W + NW * Q < TILES) {
        z[Q] = __builtin_amdgcn_mfma_f64_16x16x4f64(cur[Q], cur[MT + Q], z[Q], 0, 0, 0);
        read<W, STEP + 1, Q>(X, Y, nxt);
        __builtin_amdgcn_sched_barrier(0);
        steps<W, STEP, Q + 1>(X, Y, cur, nxt, z);
      } else {
        steps<W, STEP + 1, 0>(X, Y, nxt, cur, z);
      }
    }
  }
  template <int W>
  __device__ static __forceinline__ void mul_of(int w, const Bases& X, const Bases& Y, f64x4 (&z)[MT]) {
    if constexpr (W < NW && W < TILES) {
      if (w == W) {
        double a[2 * MT], b[2 * MT];
        first<W, 0>(X, Y, a);
        steps<W, 0, 0>(X, Y, a, b, z);
      } else {
        mul_of<W + 1>(w, X, Y, z);
      }
    }
  }
  __device__ static __forceinline__ Bases bases(const char* m, int lane) {
    const char* c = m + (lane & 15) * PITCH + (lane >> 4) * 8;
    const char* r = m + (lane >> 4) * PITCH + (lane & 15) * 8;
    return Bases{{c, c + HIGH * TILE}, {r, r + HIGH * TILE}};
  }
};

template <int B>
__global__ __launch_bounds__(NT) void k_muon_rounds(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ double red[NW];
  using K = Rounds<B>;
  constexpr int MT = K::MT, R = 16 * B;
  long mat;
  const MuonTensor& t = find_matrix(p, blockIdx.x, mat);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  char *const A = smem, *const Bm = smem + K::TILES * K::TILE;
  auto live = [&](int q) { return w + NW * q < K::TILES; };
  int ti[MT], tj[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    int i = 0, j = 0;
    if (live(q)) tri(w + NW * q, i, j);
    ti[q] = __builtin_amdgcn_readfirstlane(i);
    tj[q] = __builtin_amdgcn_readfirstlane(j);
  }
  auto diagonal = [&](int q, int v) { return ti[q] == tj[q] && 4 * v + (lane >> 4) == (lane & 15); };
  // element v of the wave's tile q: row 4 v + lane / 16, column lane % 16
  auto place = [&](char* m, int q, int v) { return (double*)(m + (w + NW * q) * K::TILE + (lane >> 4) * K::PITCH + (lane & 15) * 8 + 4 * v * K::PITCH); };
  auto put = [&](char* m, const f64x4 (&z)[MT]) {
#pragma unroll
    for (int q = 0; q < MT; ++q)
      if (live(q))
#pragma unroll
        for (int v = 0; v < 4; ++v) *place(m, q, v) = z[q][v];
  };
  // Q waits in memory between its products, where the first part was: each thread
  // its own elements
  double* const Qm = t.part + part_at(t, mat) + w * 256 + lane;
  auto save_q = [&](const f64x4 (&z)[MT]) {
#pragma unroll
    for (int q = 0; q < MT; ++q)
      if (live(q))
#pragma unroll
        for (int v = 0; v < 4; ++v) Qm[NW * q * 256 + v * 64] = z[q][v];
  };
  auto put_q = [&](char* m) {
#pragma unroll
    for (int q = 0; q < MT; ++q)
      if (live(q))
#pragma unroll
        for (int v = 0; v < 4; ++v) *place(m, q, v) = Qm[NW * q * 256 + v * 64];
  };
  f64x4 next[MT], z[MT];
  // the parts in order, all of one part's loads together, and the trace: the sum
  // of U's squares
  const double* part = t.part + part_at(t, mat) + w * 256 + lane;
#pragma unroll
  for (int q = 0; q < MT; ++q) z[q] = f64x4{0.0, 0.0, 0.0, 0.0};
  for (int s = 0; s < t.splits; ++s, part += K::TILES * 256)
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v) z[q][v] += live(q) ? part[NW * q * 256 + v * 64] : 0.0;
  double tr = 0.0;
#pragma unroll
  for (int q = 0; q < MT; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) tr += live(q) && diagonal(q, v) ? z[q][v] : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  if (lane == 0) red[w] = tr;
  __syncthreads();
  tr = 0.0;
#pragma unroll
  for (int i = 0; i < NW; ++i) tr += red[i];
  const Norm norm(tr, p.eps);
  const double inv2 = norm.all * norm.all;
#pragma unroll
  for (int q = 0; q < MT; ++q) z[q] *= inv2;
  put(A, z);
  __syncthreads();
  // The products of round n in turn: S S (to P), S P, (S P) P (the next S), P Q.
  // A holds S, then S P, then Q; Bm holds P.
  enum { SS, SP, SPP, PQ } what = SS;
  const char *X = A, *Y = A;
  for (int n = 0;;) {
    const bool last = n + 1 == p.rounds;
#pragma unroll
    for (int q = 0; q < MT; ++q) z[q] = f64x4{0.0, 0.0, 0.0, 0.0};
    K::template mul_of<0>(w, K::bases(X, lane), K::bases(Y, lane), z);
    if (what == SS) {
#pragma unroll
      for (int q = 0; q < MT; ++q)
        if (live(q))
#pragma unroll
          for (int v = 0; v < 4; ++v) z[q][v] = fma(p.c, z[q][v], fma(p.b, *place(A, q, v), diagonal(q, v) ? p.a : 0.0));
      put(Bm, z);
      if (n == 0) {
        if (last) break;  // z is Q
        save_q(z);
      }
      __syncthreads();
      if (last) {
        put_q(A);
        __syncthreads();
        what = PQ, X = Bm, Y = A;
      } else {
        what = SP, X = A, Y = Bm;
      }
    } else if (what == SP) {
      __syncthreads();
      put(A, z);
      __syncthreads();
      what = SPP;
    } else if (what == SPP) {
      __syncthreads();
      if (n == 0) {
        put(A, z);
        what = SS, X = A, Y = A, ++n;
      } else {
#pragma unroll
        for (int q = 0; q < MT; ++q) next[q] = z[q];
        put_q(A);
        what = PQ, X = Bm, Y = A;
      }
      __syncthreads();
    } else {
      if (last) break;  // z is Q
      save_q(z);
      __syncthreads();
      put(A, next);
      __syncthreads();
      what = SS, X = A, Y = A, ++n;
    }
  }
  float* out = t.q + mat * q_size(R);
  if (threadIdx.x == 0) out[R * R] = norm.of_u;
#pragma unroll
  for (int q = 0; q < MT; ++q)
    if (live(q))
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * ti[q] + 4 * v + (lane >> 4), c = 16 * tj[q] + (lane & 15);
        const float x = over_norm(z[q][v], norm.of_q);
        out[(long)r * R + c] = x;
        out[(long)c * R + r] = x;
      }
}

// Longer short sides: the rounds' matrices in memory, whole, a launch a product,
// a wave a tile of 16 x 16.
__device__ __forceinline__ const MuonTensor& long_matrix(const MuonArgs& p, long& mat, int& tile, int per) {
  const long m = blockIdx.x / per;
  tile = (int)(blockIdx.x - m * per) * NW + (threadIdx.x >> 6);
  return find_matrix(p, m, mat);
}
__device__ __forceinline__ double* long_slot(const MuonTensor& t, long mat, int slot) {
  return t.part + part_at(t, mat) + t.splits * (long)(tri_tiles(t.R / 16) * 256) + slot * (long)t.R * t.R;
}
// the norm's factor of Q, behind a matrix's slots
__device__ __forceinline__ double* long_norm(const MuonTensor& t, long mat) { return long_slot(t, mat, LONG_SLOTS); }

__global__ __launch_bounds__(NT) void k_muon_long_sum(MuonArgs p, int per) {
  __shared__ double sums[NW];
  long mat;
  int tile, i, j;
  const MuonTensor& t = long_matrix(p, mat, tile, per);
  const int lane = threadIdx.x & 63;
  const long tiles = (long)tri_tiles(t.R / 16) * 256;
  double* S = long_slot(t, mat, 0);
  const double* part = S - t.splits * tiles;
  // every workgroup adds up the diagonals by itself, in the same order: no launch before this one
  double tr = 0.0;
#pragma unroll 8
  for (int n = threadIdx.x; n < t.splits * t.R; n += NT) {
    const int s = n / t.R, c = n - s * t.R, d = c >> 4;
    tr += part[s * tiles + (tri_tiles(d) + d) * 256 + (c & 15) * 17];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  if (lane == 0) sums[threadIdx.x >> 6] = tr;
  __syncthreads();
  tr = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) tr += sums[w];
  const Norm norm(tr, p.eps);
  const double inv2 = norm.all * norm.all;
  if (tile >= tri_tiles(t.R / 16)) return;
  if (tile == 0) {
    *long_norm(t, mat) = norm.of_q;
    t.q[mat * q_size(t.R) + (long)t.R * t.R] = norm.of_u;
  }
  tri(tile, i, j);
  part += tile * 256;
  double x[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int s = 0; s < t.splits; ++s)
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] += part[s * tiles + v * 64 + lane];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
    S[(long)r * t.R + c] = x[v] * inv2;
    S[(long)c * t.R + r] = x[v] * inv2;
  }
}
// z = fc x y + fb x + fa I (all symmetric; a plain product has fb = fa = 0, a
// polynomial may have either alone); out: to q, over the norm, in fp32
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
  // the loads of 64 rows at a time in flight (one at a time, a product of 256 x 256 waited 64 times for memory)
  for (int k0 = 0; k0 < t.R; k0 += 64) {
    double av[16], bv[16];
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const long k = k0 + 4 * s < t.R ? k0 + 4 * s : 0;
      av[s] = a[k * t.R];
      bv[s] = b[k * t.R];
    }
#pragma unroll
    for (int s = 0; s < 16; ++s)
      if (k0 + s / 4 * 16 < t.R) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(av[s], bv[s], acc, 0, 0, 0);
  }
  double* Z = long_slot(t, mat, z);
  const double of_q = out ? *long_norm(t, mat) : 0.0;
  float* q = t.q + mat * q_size(t.R);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
    const double one = r == c ? fa : 0.0;
    const double d = fma(fc, acc[v], fb != 0.0 ? fma(fb, X[(long)r * t.R + c], one) : one);
    if (out) {
      q[(long)r * t.R + c] = over_norm(d, of_q);
      q[(long)c * t.R + r] = over_norm(d, of_q);
    } else {
      Z[(long)r * t.R + c] = d;
      Z[(long)c * t.R + r] = d;
    }
  }
}

// Q U for a part of the long side, and the parameters.  A wave keeps its columns
// of Q in registers; the results go through LDS, so that the parameters are read
// and written in the order of memory.  The next chunk's gradient and momentum and
// this one's parameters are in flight behind the products.  50.8 M elements in 195
// matrices of 128 rows: 183 us, 4.4 TB/s of 813 MB read and written (without the
// products the same, without memory 136; the fp32 rate's share 85).
// XT: what is updated, the master copy (then `param`, bf16, gets its rounding) or
// the parameter itself.
template <class XT, bool COPY, class GT, int RB, bool TALL, bool VEC>
__device__ __forceinline__ void apply(const MuonArgs& p, const MuonTensor& t, long mat, int s, float* S) {
  using Sh = Share<RB, TALL, apply_chunk(RB), apply_pitch(RB, TALL)>;
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const float lr = p.control != nullptr ? p.control->lr : p.lr;
  const float step = lr * (p.rms * sqrtf((float)t.L)), decay = lr * p.weight_decay;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int KT = RB / 16;                        // blocks of Q's rows
  constexpr int JT = Sh::CHUNK / 16;                 // blocks of the chunk
  constexpr int WI = cmax(KT <= 4 ? KT : NW, NW / JT);  // waves along the short side
  constexpr int IW = cmax(KT / WI, 1);               // blocks of it a wave
  constexpr int JW = cmax(JT * WI / NW, 1);          // blocks of the chunk a wave
  const int nt = t.R / 16, wi = w % WI, wj = w / WI * JW;
  Sh sh;
  sh.init(t);
  const int l_begin = s * t.span;
  int left = min(t.L - l_begin, t.span);
  const long size = (long)t.r * t.L, at = TALL ? (long)l_begin * t.r : l_begin;
  Part<VEC, GT> g;
  Part<VEC, float> mo;
  Part<VEC, XT> xs;
  Part<VEC, uint16_t> copy;
  g.init((const GT*)t.grad, mat * size, size, at);
  mo.init(t.momentum, mat * size, size, at);
  xs.init(COPY ? (const XT*)t.master : (const XT*)t.param, mat * size, size, at);
  if (COPY) copy.init((const uint16_t*)t.param, mat * size, size, at);
  Four<GT> gv[Sh::N];
  Four<float> mv[Sh::N];
  auto fetch = [&](int have) {
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      g.load(gv[i], sh.at[i], sh.have(i, have));
      mo.load(mv[i], sh.at[i], sh.have(i, have));
    }
  };
  fetch(left);
  const float* Q = t.q + mat * q_size(t.R);
  float q[IW][KT][4];
#pragma unroll
  for (int i = 0; i < IW; ++i)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * kt + 4 * e + (lane >> 4), col = 16 * (wi + WI * i) + (lane & 15);
        q[i][kt][e] = kt < nt && wi + WI * i < nt ? Q[(long)row * t.R + col] : 0.0f;
      }
  const float of_u = Q[(long)t.R * t.R];
  // rows past the short side are multiplied by zeros of Q and must be finite
  float* O = S + Sh::SIZE + 256;
  for (int i = threadIdx.x; i < Sh::SIZE; i += NT) S[i] = 0.0f;
  __syncthreads();
  const float* Sf = S + (lane >> 4) * Sh::KS + (lane & 15) * Sh::LS + 16 * wj * Sh::LS;
  for (; left > 0; left -= Sh::CHUNK) {
    Four<XT> xv[Sh::N];
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      const f32x4 x = gv[i].get(), m = mv[i].get();
      f32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = (p.nesterov ? fmaf(p.momentum, m[e], x[e] * gs) : m[e]) * of_u;
      *(f32x4*)(S + sh.lds[i]) = Sh::template only<VEC>(u, sh.have(i, left));
    }
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) xs.load(xv[i], sh.at[i], sh.have(i, left));
    __syncthreads();
    g.next(Sh::step(t));
    mo.next(Sh::step(t));
    fetch(left - Sh::CHUNK);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 acc[IW][JW];
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < JW; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // a lane's four results are neighbours in memory: along the short side where the tensor is tall
    // operands are read two steps ahead
    auto blocks = [&](auto lo, auto hi) {
      constexpr int FROM = 4 * lo.value, TO = 4 * hi.value;
      float y[4][JW];
#pragma unroll
      for (int k = FROM - 2; k < TO; ++k) {
        if (k + 2 < TO)
#pragma unroll
          for (int j = 0; j < JW; ++j) y[(k + 2) & 3][j] = Sf[4 * (k + 2) * Sh::KS + 16 * j * Sh::LS];
        if (k < FROM) continue;
#pragma unroll
        for (int i = 0; i < IW; ++i)
#pragma unroll
          for (int j = 0; j < JW; ++j)
            acc[i][j] = TALL ? __builtin_amdgcn_mfma_f32_16x16x4f32(q[i][k / 4][k % 4], y[k & 3][j], acc[i][j], 0, 0, 0)
                             : __builtin_amdgcn_mfma_f32_16x16x4f32(y[k & 3][j], q[i][k / 4][k % 4], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // short sides that come here have more than half of RB: few branches, for long runs between them
    constexpr int K1 = KT / 2 + KT % 2 + (KT > 2 ? 1 : 0), K2 = cmax(K1, KT * 3 / 4);
    blocks(std::integral_constant<int, 0>{}, std::integral_constant<int, K1>{});
    if (K2 > K1 && nt > K1) blocks(std::integral_constant<int, K1>{}, std::integral_constant<int, K2>{});
    if (KT > K2 && nt > K2) blocks(std::integral_constant<int, K2>{}, std::integral_constant<int, KT>{});
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int j = 0; j < JW; ++j) {
        const int c = 16 * (wi + WI * i), l = 16 * (wj + j);
        const int a = TALL ? l : c, b = TALL ? c : l;
        if (KT >= WI || wi < KT) *(f32x4*)(O + (a + (lane & 15)) * Sh::PITCH + b + 4 * (lane >> 4)) = acc[i][j];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Sh::N; ++i) {
      const int have = sh.have(i, left);
      const f32x4 o = *(const f32x4*)(O + sh.lds[i]);
      f32x4 x = xv[i].get();
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] -= fmaf(step, o[e], decay * x[e]);
      xs.store(sh.at[i], have, x);
      if (COPY) copy.store(sh.at[i], have, x);
    }
    xs.next(Sh::step(t));
    if (COPY) copy.next(Sh::step(t));
  }
}

template <class XT, bool COPY, class GT, int RB, bool VEC>
__global__ __launch_bounds__(NT, RB <= 128 ? 4 : 2) void k_muon_apply(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  int ti, s;
  long mat;
  // backwards: what the first pass read last may still be in the memory-side cache (wide: 208 -> 190 us)
  find(p, p.groups - 1 - blockIdx.x, ti, mat, s);
  const MuonTensor& t = p.t[ti];
  if (t.tall)
    apply<XT, COPY, GT, RB, true, VEC>(p, t, mat, s, (float*)smem);
  else
    apply<XT, COPY, GT, RB, false, VEC>(p, t, mat, s, (float*)smem);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int round16(int r) { return (r + 15) / 16 * 16; }

// The long sides of all matrices of the call, a CU.
double share_of(const moe_muon_tensor* t, int32_t count, int cus) {
  double total = 0;
  for (int32_t i = 0; i < count; ++i)
    if (t[i].batch > 0) total += (double)t[i].batch * (t[i].m > t[i].n ? t[i].m : t[i].n);
  return total / cus;
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
Plan plan_of(const moe_muon_tensor& t, double share) {
  Plan p;
  p.r = t.m < t.n ? t.m : t.n;
  p.L = t.m < t.n ? t.n : t.m;
  p.R = round16(p.r);
  // Entries of the long side that a workgroup takes, in whole chunks: two rounds of two workgroups a CU; beyond
  // SHORT_R one workgroup a CU, since a part's tiles of S0 weigh more than its U (16 matrices of 256 x 4096: 64 parts
  // of each 811 us, 16 of each 637)
  const double span = p.R > SHORT_R ? share : share / 4;
  p.span = span < 64 ? 64 : span > 0x1p30 ? 1 << 30 : (int)((span + 63) / 64) * 64;
  p.splits = 1 + (p.L - 1) / p.span;  // a long side just below 2^31 leaves no room for another span
  p.part = (size_t)t.batch * part_size(p.R, p.splits) * 8;
  p.q = (size_t)t.batch * q_size(p.R) * 4;  // a multiple of 16
  return p;
}

// LDS for short sides up to RB, either way round: a chunk of U (and of Q U), with what is nowhere behind it
constexpr int gram_lds(int RB) { return (cmax(gram_pitch(RB, true) * gram_chunk(RB), gram_pitch(RB, false) * RB) + 256) * 8; }
constexpr int apply_lds(int RB) {
  return (cmax(apply_pitch(RB, true) * apply_chunk(RB), apply_pitch(RB, false) * RB) + 256) * 2 * 4;
}

template <class GT, int RB, bool VEC>
hipError_t launch_gram(const MuonArgs& p, hipStream_t st) {
  static PerDeviceOnce once;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_muon_gram<GT, RB, VEC>, gram_lds(RB));
    return ai.err;
  });
  if (e != hipSuccess) return e;
  MOE_LAUNCH_AS("k_muon_gram", (k_muon_gram<GT, RB, VEC>), dim3((unsigned)p.groups), dim3(NT), gram_lds(RB), st, p);
  return hipGetLastError();
}
template <class XT, bool COPY, class GT, int RB, bool VEC>
hipError_t launch_apply(const MuonArgs& p, hipStream_t st) {
  static PerDeviceOnce once;
  const hipError_t e = once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_muon_apply<XT, COPY, GT, RB, VEC>, apply_lds(RB));
    return ai.err;
  });
  if (e != hipSuccess) return e;
  MOE_LAUNCH_AS("k_muon_apply", (k_muon_apply<XT, COPY, GT, RB, VEC>), dim3((unsigned)p.groups), dim3(NT), apply_lds(RB),
                st, p);
  return hipGetLastError();
}
template <int B>
hipError_t launch_rounds(const MuonArgs& p, int R, hipStream_t st) {
  if (R < 16 * B) return launch_rounds<B - 1>(p, R, st);
  if constexpr (B == 1) {
    MOE_LAUNCH_AS("k_muon_rounds", k_muon_rounds16, dim3((unsigned)p.matrices), dim3(64), 0, st, p);
  } else {
    static PerDeviceOnce once;
    const hipError_t e = once.run([] {
      AttrInit ai;
      ai.lds((const void*)k_muon_rounds<B>, Rounds<B>::LDS);
      return ai.err;
    });
    if (e != hipSuccess) return e;
    MOE_LAUNCH_AS("k_muon_rounds", k_muon_rounds<B>, dim3((unsigned)p.matrices), dim3(NT), Rounds<B>::LDS, st, p);
  }
  return hipGetLastError();
}
template <>
hipError_t launch_rounds<0>(const MuonArgs&, int, hipStream_t) { return hipErrorInvalidValue; }
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

// All tensors of p have short sides of R (in whole tiles) and are VEC or not.
template <class GT, int RB, bool VEC>
hipError_t launch_step(const MuonArgs& p, int R, bool pbf, hipStream_t st) {
  hipError_t e = launch_gram<GT, RB, VEC>(p, st);
  if (e != hipSuccess) return e;
  e = R <= SHORT_R ? launch_rounds<SHORT_R / 16>(p, R, st) : launch_long_rounds(p, R, st);
  if (e != hipSuccess) return e;
  if (!pbf) return launch_apply<float, false, GT, RB, VEC>(p, st);
  return p.t[0].master != nullptr ? launch_apply<float, true, GT, RB, VEC>(p, st)
                                  : launch_apply<uint16_t, false, GT, RB, VEC>(p, st);
}
template <int RB, bool VEC>
hipError_t launch_step(const MuonArgs& p, int R, bool pbf, bool gbf, hipStream_t st) {
  return gbf ? launch_step<uint16_t, RB, VEC>(p, R, pbf, st) : launch_step<float, RB, VEC>(p, R, pbf, st);
}
template <bool VEC>
hipError_t launch_step(const MuonArgs& p, int R, bool pbf, bool gbf, hipStream_t st) {
  if (R <= 16) return launch_step<16, VEC>(p, R, pbf, gbf, st);
  if (R <= 64) return launch_step<64, VEC>(p, R, pbf, gbf, st);
  if (R <= SHORT_R) return launch_step<SHORT_R, VEC>(p, R, pbf, gbf, st);
  return launch_step<MAX_SHORT, VEC>(p, R, pbf, gbf, st);
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
  const double share = share_of(t, count, cus);
  size_t n = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].batch == 0) continue;
    const Plan p = plan_of(t[i], share);
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
  const double share = share_of(t, count, cus);
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
  // One launch of each kernel for the tensors that take the same ones: equal short
  // sides in whole tiles, and groups of four in memory whole or not.
  char* at = (char*)workspace;
  const bool pbf = d->param_type == MOE_TYPE_BF16, gbf = d->grad_type == MOE_TYPE_BF16;
  const hipStream_t st = (hipStream_t)stream;
  for (int R = 16; R <= MAX_SHORT; R += 16)
    for (int vec = 0; vec < 2; ++vec) {
      auto flush = [&]() {
        if (p.count == 0) return hipSuccess;
        const hipError_t e = vec ? launch_step<true>(p, R, pbf, gbf, st) : launch_step<false>(p, R, pbf, gbf, st);
        p.count = 0;
        p.groups = p.matrices = 0;
        return e;
      };
      for (int32_t i = 0; i < count; ++i) {
        const moe_muon_tensor& x = t[i];
        if (x.batch == 0) continue;
        const bool tall = x.m > x.n;
        const bool whole = x.n % 4 == 0 && (int64_t)x.m * x.n < (int64_t)1 << 29;  // see Part
        if (round16(tall ? x.n : x.m) != R || whole != (vec != 0)) continue;
        const Plan pl = plan_of(x, share);
        // a launch holds fewer than 2^32 threads; long rounds take 17 workgroups a matrix
        if (p.count == TENSORS || p.groups + x.batch * pl.splits >= (int64_t)1 << 23 ||
            (R > SHORT_R && p.matrices + x.batch >= (int64_t)1 << 18))
          if (flush() != hipSuccess) return MOE_ERR_HIP;
        p.t[p.count++] = MuonTensor{x.param, x.master, x.grad, x.momentum, p.groups, p.matrices, (double*)at,
                                    (float*)(at + pl.part), pl.r, pl.L, tall, pl.R, pl.splits, pl.span};
        at += pl.part + pl.q;
        p.groups += x.batch * pl.splits;
        p.matrices += x.batch;
      }
      if (flush() != hipSuccess) return MOE_ERR_HIP;
    }
  return MOE_OK;
}

}  // extern "C"
