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
constexpr int CHUNK = 64;     // entries of the long side in LDS at a time
constexpr int NT = 512, NW = 8;

struct MuonTensor {
  void* param;
  float* master;
  const void* grad;
  float* momentum;
  long first;        // this tensor's first workgroup in a launch over splits
  long matrix0;      // index of its first matrix
  double* part;      // [matrices][slots][R][R]: partial sums of S0, then the rounds' matrices
  float* q;          // [matrices][R][R]
  int r, L, tall;    // tall: stored [L, r]
  int R;             // r in whole tiles of 16
  int splits, span;  // workgroups along L, entries each
  int slots;         // at least four
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

template <class T>
__device__ __forceinline__ float value(const T* p, long i) {
  if constexpr (sizeof(T) == 2)
    return bf2f(p[i]);
  else
    return p[i];
}

// A workgroup's tensor, matrix and part of the long side.
__device__ __forceinline__ bool find(const MuonArgs& p, long b, int& t, long& mat, int& s) {
  t = 0;
  while (t + 1 < p.count && b >= p.t[t + 1].first) ++t;
  const long i = b - p.t[t].first;
  mat = i / p.t[t].splits;
  s = (int)(i - mat * p.t[t].splits);
  return b < p.groups;
}

// LDS pitch of U held by long entries, [CHUNK][R]: 18 of 64 banks on, so that
// neither four entries side by side nor four rows of 16 meet in a bank.
__device__ __host__ constexpr int pitch_long(int R) { return (R + 63 - 18) / 64 * 64 + 18; }

// U of entries l0 .. l0 + CHUNK - 1 into LDS as S[l][c]; zeros past L and r.
// WRITE: forms the new momentum and stores it, else reads it.
template <class GT, bool WRITE>
__device__ __forceinline__ void load_u(const MuonArgs& p, const MuonTensor& t, long mat, int l0, int lend, float gs, float* S) {
  const int pitch = pitch_long(t.R);
  const long at = mat * (long)t.r * t.L;
  const GT* g = (const GT*)t.grad + at;
  float* mo = t.momentum + at;
  for (int i = threadIdx.x; i < CHUNK * t.R; i += NT) {
    int l, c;
    if (t.tall) {
      l = i / t.R;
      c = i - l * t.R;
    } else {
      c = i / CHUNK;
      l = i - c * CHUNK;
    }
    float u = 0.0f;
    if (l0 + l < lend && c < t.r) {
      const long k = t.tall ? (long)(l0 + l) * t.r + c : (long)c * t.L + l0 + l;
      const float x = value(g, k) * gs;
      float m = mo[k];
      if (WRITE) {
        m = fmaf(p.momentum, m, x);
        mo[k] = m;
      }
      u = p.nesterov ? fmaf(p.momentum, m, x) : m;
    }
    S[l * pitch + c] = u;
  }
}

// Tile t of the lower triangle of tiles.
__device__ __forceinline__ void tri(int t, int& i, int& j) {
  i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  j = t - i * (i + 1) / 2;
}

// Partial S0 of a part of the long side.
template <class GT, int RB>
__global__ __launch_bounds__(NT) void k_muon_gram(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  float* S = (float*)smem;
  constexpr int MT = ((RB / 16) * (RB / 16 + 1) / 2 + NW - 1) / NW;  // tiles a wave
  int ti, s;
  long mat;
  if (!find(p, blockIdx.x, ti, mat, s)) return;
  const MuonTensor& t = p.t[ti];
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int nt = t.R / 16, pitch = pitch_long(t.R);
  const int tiles = nt * (nt + 1) / 2;
  f64x4 acc[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) acc[q] = f64x4{0.0, 0.0, 0.0, 0.0};
  const int l_end = min(t.L, (s + 1) * t.span);
  for (int l0 = s * t.span; l0 < l_end; l0 += CHUNK) {
    load_u<GT, true>(p, t, mat, l0, l_end, gs, S);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < MT; ++q) {
      const int k = w + NW * q;
      if (k >= tiles) continue;
      int i, j;
      tri(k, i, j);
      const float* x = S + (lane >> 4) * pitch + 16 * i + (lane & 15);
      const float* y = S + (lane >> 4) * pitch + 16 * j + (lane & 15);
#pragma unroll
      for (int k4 = 0; k4 < CHUNK; k4 += 4)
        acc[q] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[k4 * pitch], (double)y[k4 * pitch], acc[q], 0, 0, 0);
    }
    __syncthreads();
  }
  double* out = t.part + (mat * t.slots + s) * (long)t.R * t.R;
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int k = w + NW * q;
    if (k >= tiles) continue;
    int i, j;
    tri(k, i, j);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * i + 4 * v + (lane >> 4), col = 16 * j + (lane & 15);
      out[(long)row * t.R + col] = acc[q][v];
      out[(long)col * t.R + row] = acc[q][v];
    }
  }
}

// The rounds on one matrix of R x R in memory: z = x y, lower tiles and their
// mirror images; f(row, col, xy) is what is stored.
template <class F>
__device__ __forceinline__ void product(const double* x, const double* y, double* z, int R, F&& f) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int nt = R / 16, tiles = nt * (nt + 1) / 2;
  for (int k = w; k < tiles; k += NW) {
    int i, j;
    tri(k, i, j);
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
    const double* a = x + (long)(lane >> 4) * R + 16 * i + (lane & 15);  // symmetric: rows read as columns
    const double* b = y + (long)(lane >> 4) * R + 16 * j + (lane & 15);
    for (int k4 = 0; k4 < R; k4 += 4)
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a[(long)k4 * R], b[(long)k4 * R], acc, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * i + 4 * v + (lane >> 4), col = 16 * j + (lane & 15);
      const double d = f(row, col, acc[v]);
      z[(long)row * R + col] = d;
      z[(long)col * R + row] = d;
    }
  }
}

// The rounds' matrices S, P, T and Q lie where the partial sums were: the sum at
// an element goes to T's, by the thread that has read all parts there.
__global__ __launch_bounds__(NT) void k_muon_rounds(MuonArgs p) {
  __shared__ double red[NW];
  int ti = 0;
  while (ti + 1 < p.count && (long)blockIdx.x >= p.t[ti + 1].matrix0) ++ti;
  const MuonTensor& t = p.t[ti];
  const long mat = blockIdx.x - t.matrix0;
  const int R = t.R;
  const long RR = (long)R * R;
  double* S = t.part + mat * t.slots * RR;  // the sum of the parts, in place of the first
  double* P = S + RR;
  double* T = P + RR;
  double* Q = T + RR;
  double tr = 0.0;
  for (long i = threadIdx.x; i < RR; i += NT) {
    double v = S[i];
    for (int s = 1; s < t.splits; ++s) v += S[s * RR + i];
    T[i] = v;
    if (i / R == i % R) tr += v;
  }
  // fixed order: lanes, then waves
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) tr += __shfl_xor(tr, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = tr;
  __syncthreads();
  tr = 0.0;
#pragma unroll
  for (int i = 0; i < NW; ++i) tr += red[i];
  const double inv = 1.0 / (sqrt(tr) + p.eps), inv2 = inv * inv;
  for (long i = threadIdx.x; i < RR; i += NT) S[i] = T[i] * inv2;
  __syncthreads();
  for (int k = 0; k < p.rounds; ++k) {
    const bool last = k + 1 == p.rounds;
    product(S, S, P, R, [&](int row, int col, double v) {
      return fma(p.c, v, fma(p.b, S[(long)row * R + col], row == col ? p.a : 0.0));
    });
    __syncthreads();
    if (k == 0) {
      for (long i = threadIdx.x; i < RR; i += NT) Q[i] = P[i];
    } else {
      product(P, Q, T, R, [](int, int, double v) { return v; });
      __syncthreads();
      for (long i = threadIdx.x; i < RR; i += NT) Q[i] = T[i];
    }
    __syncthreads();
    if (last) break;
    product(S, P, T, R, [](int, int, double v) { return v; });
    __syncthreads();
    product(T, P, S, R, [](int, int, double v) { return v; });
    __syncthreads();
  }
  float* q = t.q + mat * RR;
  for (long i = threadIdx.x; i < RR; i += NT) q[i] = (float)(Q[i] * inv);
}

// Q U for a part of the long side, and the parameters.
template <class PT, class GT>
__global__ __launch_bounds__(NT) void k_muon_apply(MuonArgs p) {
  extern __shared__ __align__(16) char smem[];
  float* S = (float*)smem;
  int ti, s;
  long mat;
  if (!find(p, blockIdx.x, ti, mat, s)) return;
  const MuonTensor& t = p.t[ti];
  const float gs = p.control != nullptr ? p.control->grad_scale : p.grad_scale;
  const float lr = p.control != nullptr ? p.control->lr : p.lr;
  const float step = lr * (p.rms * sqrtf((float)t.L)), decay = lr * p.weight_decay;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int nt = t.R / 16, pitch = pitch_long(t.R);
  const float* q = t.q + mat * (long)t.R * t.R;
  const long at = mat * (long)t.r * t.L;
  const int l_end = min(t.L, (s + 1) * t.span);
  for (int l0 = s * t.span; l0 < l_end; l0 += CHUNK) {
    load_u<GT, false>(p, t, mat, l0, l_end, gs, S);
    __syncthreads();
    for (int k = w; k < nt * (CHUNK / 16); k += NW) {
      const int i = k % nt, j = k / nt;  // 16 of the short side, 16 of the long
      const float* x = q + (long)(lane >> 4) * t.R + 16 * i + (lane & 15);
      const float* y = S + (16 * j + (lane & 15)) * pitch + (lane >> 4);
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      // a lane's four results are neighbours in memory: along the short side where the tensor is tall
      if (t.tall)
        for (int k4 = 0; k4 < t.R; k4 += 4) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[(long)k4 * t.R], y[k4], acc, 0, 0, 0);
      else
        for (int k4 = 0; k4 < t.R; k4 += 4) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(y[k4], x[(long)k4 * t.R], acc, 0, 0, 0);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int c = 16 * i + (t.tall ? 4 * (lane >> 4) + v : lane & 15);
        const int l = l0 + 16 * j + (t.tall ? lane & 15 : 4 * (lane >> 4) + v);
        if (c >= t.r || l >= l_end) continue;
        const long n = at + (t.tall ? (long)l * t.r + c : (long)c * t.L + l);
        float x0 = t.master != nullptr ? t.master[n] : value((const PT*)t.param, n);
        x0 -= fmaf(step, acc[v], decay * x0);
        if (t.master != nullptr) t.master[n] = x0;
        if constexpr (sizeof(PT) == 2)
          ((PT*)t.param)[n] = (PT)f2bf(x0);
        else
          ((PT*)t.param)[n] = x0;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int round16(int r) { return (r + 15) / 16 * 16; }

// The split of the long side: enough workgroups for the chip, none with less
// than 256 entries.
void split(int64_t matrices, int L, int cus, int& splits, int& span) {
  int64_t want = (4 * (int64_t)cus + matrices - 1) / matrices;
  const int64_t most = (L + 255) / 256;
  if (want > most) want = most;
  span = (int)(((L + want - 1) / want + CHUNK - 1) / CHUNK * CHUNK);
  splits = (L + span - 1) / span;
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
    if ((t[i].m < t[i].n ? t[i].m : t[i].n) > MAX_SHORT || mn >= (int64_t)1 << 31 || t[i].batch > (int64_t)1 << 20 ||
        t[i].batch * mn >= (int64_t)1 << 40)
      return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

struct Plan {
  int r, L, R, splits, span, slots;
  size_t part, q;  // bytes
};
Plan plan_of(const moe_muon_tensor& t, int cus) {
  Plan p;
  p.r = t.m < t.n ? t.m : t.n;
  p.L = t.m < t.n ? t.n : t.m;
  p.R = round16(p.r);
  split(t.batch, p.L, cus, p.splits, p.span);
  const size_t RR = (size_t)p.R * p.R;
  p.slots = p.splits > 4 ? p.splits : 4;
  p.part = (size_t)t.batch * p.slots * RR * 8;
  p.q = ((size_t)t.batch * RR * 4 + 15) / 16 * 16;
  return p;
}

constexpr int lds_of(int RB) { return pitch_long(RB) * CHUNK * 4; }

template <class GT>
hipError_t launch_gram(const MuonArgs& p, int R, hipStream_t st) {
  const dim3 g((unsigned)p.groups), b(NT);
  if (R <= 64)
    MOE_LAUNCH_AS("k_muon_gram", (k_muon_gram<GT, 64>), g, b, lds_of(64), st, p);
  else if (R <= 128)
    MOE_LAUNCH_AS("k_muon_gram", (k_muon_gram<GT, 128>), g, b, lds_of(128), st, p);
  else
    MOE_LAUNCH_AS("k_muon_gram", (k_muon_gram<GT, 256>), g, b, lds_of(256), st, p);
  return hipGetLastError();
}
template <class PT, class GT>
hipError_t launch_apply(const MuonArgs& p, int R, hipStream_t st) {
  MOE_LAUNCH_AS("k_muon_apply", (k_muon_apply<PT, GT>), dim3((unsigned)p.groups), dim3(NT),
                lds_of(R <= 64 ? 64 : R <= 128 ? 128 : 256), st, p);
  return hipGetLastError();
}

hipError_t prepare_kernels() {
  static PerDeviceOnce once;
  return once.run([] {
    AttrInit ai;
    ai.lds((const void*)k_muon_gram<uint16_t, 64>, lds_of(64));
    ai.lds((const void*)k_muon_gram<uint16_t, 128>, lds_of(128));
    ai.lds((const void*)k_muon_gram<uint16_t, 256>, lds_of(256));
    ai.lds((const void*)k_muon_gram<float, 64>, lds_of(64));
    ai.lds((const void*)k_muon_gram<float, 128>, lds_of(128));
    ai.lds((const void*)k_muon_gram<float, 256>, lds_of(256));
    ai.lds((const void*)k_muon_apply<uint16_t, uint16_t>, lds_of(256));
    ai.lds((const void*)k_muon_apply<uint16_t, float>, lds_of(256));
    ai.lds((const void*)k_muon_apply<float, uint16_t>, lds_of(256));
    ai.lds((const void*)k_muon_apply<float, float>, lds_of(256));
    return ai.err;
  });
}

hipError_t launch_step(const MuonArgs& p, int R, bool pbf, bool gbf, hipStream_t st) {
  hipError_t e = gbf ? launch_gram<uint16_t>(p, R, st) : launch_gram<float>(p, R, st);
  if (e != hipSuccess) return e;
  MOE_LAUNCH(k_muon_rounds, dim3((unsigned)p.matrices), dim3(NT), 0, st, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pbf) return gbf ? launch_apply<uint16_t, uint16_t>(p, R, st) : launch_apply<uint16_t, float>(p, R, st);
  return gbf ? launch_apply<float, uint16_t>(p, R, st) : launch_apply<float, float>(p, R, st);
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
  size_t n = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].batch == 0) continue;
    const Plan p = plan_of(t[i], cus);
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
  if (device_cus(cus) != hipSuccess || prepare_kernels() != hipSuccess) return MOE_ERR_HIP;
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
  char* at = (char*)workspace;
  int R = 0;
  auto flush = [&]() {
    if (p.count == 0) return hipSuccess;
    const hipError_t e =
        launch_step(p, R, d->param_type == MOE_TYPE_BF16, d->grad_type == MOE_TYPE_BF16, (hipStream_t)stream);
    p.count = R = 0;
    p.groups = p.matrices = 0;
    return e;
  };
  for (int32_t i = 0; i < count; ++i) {
    const moe_muon_tensor& x = t[i];
    if (x.batch == 0) continue;
    const Plan pl = plan_of(x, cus);
    // a launch holds fewer than 2^32 threads
    if (p.count == TENSORS || p.groups + x.batch * pl.splits >= (int64_t)1 << 23)
      if (flush() != hipSuccess) return MOE_ERR_HIP;
    MuonTensor& m = p.t[p.count++];
    m = MuonTensor{x.param, x.master, x.grad, x.momentum, p.groups, p.matrices, (double*)at, (float*)(at + pl.part),
                   pl.r, pl.L, x.m > x.n, pl.R, pl.splits, pl.span, pl.slots};
    at += pl.part + pl.q;
    p.groups += x.batch * pl.splits;
    p.matrices += x.batch;
    if (pl.R > R) R = pl.R;
  }
  return flush() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
