// router.hip -- top-k routing with expert loads and balance loss, and its
// gradient (include/moelora.h states the formulas).
//
// Sixteen lanes (one DPP row) hold one token's logits, lane j the experts
// j, j + 16, ...: maxima, sums and index minima over a token are four DPP
// instructions without LDS, a wave works on four tokens, and a lane's
// experts are the same for every token, so the probability mass per expert
// adds up in registers.  A pass reads each logit once.  The top-k takes the
// largest key k times; a key is the logit's bits mapped to an unsigned
// integer of the same order, so the choice is exact and equals go to the
// lowest expert.
//
// At 16,384 x 64 fp32 the logits are 4 MB, 0.7 us of memory time, so latency
// bounds all three kernels: k_route 6.4 us (bf16 logits the same; each workgroup
// one round of 64 tokens; four rounds of 16 took 9.7; the choice of six experts is
// about half of it), k_route_sum 4.8 us (one workgroup reads 131 KB of sums that
// other XCDs wrote, all loads in flight together; chunks of 128 tokens halve them
// and cost k_route more: 1.2 us in sum), k_route_bwd 5.1 us (16 tokens a workgroup;
// 8.6 with four rounds; its tokens' LDS rows padded apart: no bank conflicts
// instead of 2.8 an instruction, and the same time).  One token: k_route alone,
// 3.8 us.
#include <cmath>

#include "../../include/moelora.h"
#include "checks.hpp"
#include "lanes.hpp"
#include "layer.hpp"
#include "trace.hpp"

namespace moelora {
namespace {

// A workgroup's threads by V, the experts a lane holds (more registers: fewer
// waves); 16 of them work on one token.
template <int V>
constexpr int THREADS = V <= 8 ? 1024 : V == 16 ? 512 : 256;
constexpr int BWD_THREADS = 256;  // 16 tokens: nothing is summed over tokens there
constexpr int RT_TOKENS = 64;     // tokens of one workgroup's chunk, times the multiple that keeps
constexpr int RT_CHUNKS = 512;    // the chunks (whose sums one workgroup adds) to about this many,
constexpr int RT_MOST = 64;       // but this at most: a lane adds its tokens' probabilities in fp32
constexpr int BWD_CHUNKS = 1 << 20;  // workgroups of the gradient (a launch holds fewer than 2^32 threads)
constexpr uint32_t KEY_NINF = 0x007FFFFFu;  // the key of -inf: nothing at or below it is chosen

struct RouterArgs {
  int T, E, k, renorm, na;
  int chunk;  // tokens of a workgroup, a multiple of RT_TOKENS
  int roots[MAX_ADAPTERS + 1];
  const void* logits;
  const uint8_t* valid;
  int32_t* idx;
  float* w;
  int32_t* counts;
  int32_t* active;
  float* loss;
  int32_t* err;
  // per chunk E + 1 pairs: each expert's probability mass (fp32 bits) and
  // routes, then the active and the bad tokens
  uint2* sums;
  // backward
  const float* gw;
  const float* gloss;
  void* glogits;
};

// chunk b of at most n tokens, never crossing roots: its tokens and root
__device__ __forceinline__ bool chunk_of(const RouterArgs& a, int b, int n, int& t0, int& nt, int& root) {
  for (int q = 0; q < a.na; ++q) {
    const int r0 = a.roots[q], r1 = a.roots[q + 1];
    const int c = (r1 - r0 + n - 1) / n;
    if (b < c) {
      t0 = r0 + b * n;
      nt = min(n, r1 - t0);
      root = q;
      return true;
    }
    b -= c;
  }
  return false;
}

__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((uint32_t)((int32_t)~key >> 31) | 0x80000000u));
}

// The logits of token t held by this lane (experts j + 16 i; -inf past E and
// for a token that is not `in` the chunk or not valid).  Returns whether it is
// both.  Every lane loads, at t and an expert below E, and the mask is loaded
// beside the logits: a load in a branch would be waited for at its end, one
// after another.  t: a token of the batch.
template <bool BF, int V>
__device__ __forceinline__ bool load_logits(const RouterArgs& a, long t, int j, bool in, float (&l)[V]) {
  uint32_t raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const long at = t * a.E + min(j + 16 * i, a.E - 1);
    raw[i] = BF ? (uint32_t)((const uint16_t*)a.logits)[at] : ((const uint32_t*)a.logits)[at];
  }
  const bool on = in && (a.valid == nullptr || a.valid[t] != 0);
#pragma unroll
  for (int i = 0; i < V; ++i)  // -0 to +0: equal logits have equal keys
    l[i] = on && j + 16 * i < a.E ? (BF ? bf2f(raw[i]) : __uint_as_float(raw[i])) + 0.0f : -INFINITY;
  return on;
}

// whether any of the row's 16 lanes holds `c`
__device__ __forceinline__ bool row_any(bool c) {
  return ((__ballot(c) >> (threadIdx.x & 48)) & 0xFFFFull) != 0;
}

__device__ __forceinline__ float loss_of(const RouterArgs& a, double mass_hits, int active) {
  const double n = (double)(active > 0 ? active : 1);
  return (float)(mass_hits * (double)a.E / ((double)a.k * n * n));
}

// ONE: at most ONE_TOKENS tokens of a single root, whose sums are the results.
constexpr int ONE_THREADS = 256, ONE_TOKENS = ONE_THREADS / 16;
template <bool BF, int V, bool ONE>
__global__ __launch_bounds__(ONE ? ONE_THREADS : THREADS<V>) void k_route(RouterArgs a) {
  constexpr int NT = ONE ? ONE_THREADS : THREADS<V>, ROWS = NT / 16, WAVES = NT / 64;
  __shared__ float smass[WAVES][16 * V];
  __shared__ int shits[16 * V];
  __shared__ int stally[2];
  __shared__ double part[WAVES];
  int t0, nt, root;
  if (!chunk_of(a, blockIdx.x, a.chunk, t0, nt, root)) return;
  const int tid = threadIdx.x, j = tid & 15, row = tid >> 4;
  for (int e = tid; e < 16 * V; e += NT) shits[e] = 0;
  if (tid < 2) stally[tid] = 0;
  __syncthreads();
  float mass[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mass[i] = 0.0f;
  for (int o = 0; o < nt; o += ROWS) {
    const bool in = o + row < nt;
    const long t = (long)t0 + min(o + row, nt - 1);
    float l[V];
    load_logits<BF, V>(a, t, j, in, l);
    bool strange = false;
#pragma unroll
    for (int i = 0; i < V; ++i) strange |= !(l[i] < INFINITY);
    const bool bad = row_any(strange);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = bad ? 0u : key_of(l[i]);
    int my_idx = -1;
    uint32_t my_key = 0, top = 0;
    for (int it = 0; it < a.k; ++it) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      best = row_max(best);
      if (it == 0) top = best;
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(j + 16 * i) : at;
      at = row_min(at);
      const bool take = best > KEY_NINF;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = (uint32_t)(j + 16 * i) == at ? 0u : key[i];
      if (j == it) {
        my_idx = take ? (int)at : -1;
        my_key = best;
      }
    }
    const bool act = top > KEY_NINF;
    const float mx = logit_of(top);
    float p[V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = act ? __expf(l[i] - mx) : 0.0f;
      sum += p[i];
    }
    sum = row_sum(sum);
    const float inv = act ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) mass[i] += p[i] * inv;
    float wt = my_idx >= 0 ? __expf(logit_of(my_key) - mx) : 0.0f;
    if (a.renorm) {
      const float ws = row_sum(wt);
      wt = act ? wt / ws : 0.0f;
    } else {
      wt *= inv;
    }
    if (in && j < a.k) {
      a.idx[t * a.k + j] = my_idx;
      a.w[t * a.k + j] = wt;
      if (my_idx >= 0) atomicAdd(&shits[my_idx], 1);
    }
    if (in && j == 0) {
      if (act) atomicAdd(&stally[0], 1);
      if (bad) atomicAdd(&stally[1], 1);
    }
  }
  // the four tokens of a wave, then the waves in order
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float m = mass[i];
    m += __shfl_xor(m, 16, 64);
    m += __shfl_xor(m, 32, 64);
    if ((tid & 48) == 0) smass[tid >> 6][j + 16 * i] = m;
  }
  __syncthreads();
  uint2* sums = a.sums + (long)blockIdx.x * (a.E + 1);
  double v = 0.0;
  for (int e = tid; e < a.E; e += NT) {
    float m = 0.0f;
#pragma unroll
    for (int wv = 0; wv < WAVES; ++wv) m += smass[wv][e];
    if constexpr (ONE) {
      a.counts[e] = shits[e];
      v += (double)m * (double)shits[e];
    } else {
      sums[e] = make_uint2(__float_as_uint(m), (uint32_t)shits[e]);
    }
  }
  if constexpr (ONE) {
    v = wave_sum(v);
    if ((tid & 63) == 0) part[tid >> 6] = v;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int q = 0; q < WAVES; ++q) s += part[q];
      a.active[0] = stally[0];
      a.loss[0] = loss_of(a, s, stally[0]);
      if (a.err != nullptr) *a.err = stally[1];
    }
  } else if (tid == 0) {
    sums[a.E] = make_uint2((uint32_t)stally[0], (uint32_t)stally[1]);
  }
}

// Loads and loss of root blockIdx.x from its chunks' sums: thread (slice,
// expert) adds every slices-th chunk, the slices are added in order, so the
// result does not depend on timing.  Workgroup 0 also counts the bad tokens.
constexpr int RS_THREADS = 1024;
__global__ __launch_bounds__(RS_THREADS) void k_route_sum(RouterArgs a) {
  __shared__ double sm[RS_THREADS];
  __shared__ int sh[RS_THREADS];
  __shared__ double part[RS_THREADS / 64];
  __shared__ int2 tally[RS_THREADS / 64];
  const int tid = threadIdx.x, root = blockIdx.x;
  int first = 0, nc = 0, all = 0;
  for (int q = 0; q < a.na; ++q) {
    const int c = (a.roots[q + 1] - a.roots[q] + a.chunk - 1) / a.chunk;
    if (q == root) {
      first = all;
      nc = c;
    }
    all += c;
  }
  const uint2* from = a.sums + (long)first * (a.E + 1);
  // one chunk's tokens a thread (below two million tokens), in flight with the sums below
  int act = 0, bad = 0;
  for (int c = tid; c < nc; c += RS_THREADS) act += (int)from[(long)c * (a.E + 1) + a.E].x;
  if (root == 0)
    for (int c = tid; c < all; c += RS_THREADS) bad += (int)a.sums[(long)c * (a.E + 1) + a.E].y;
  // EP experts side by side, the smallest power of two that covers E
  const int lg = a.E <= 1 ? 0 : 32 - __clz(a.E - 1), EP = 1 << lg;
  const int e = tid & (EP - 1), slice = tid >> lg, slices = RS_THREADS >> lg, W = a.E + 1;  // chunks * W: below 2^21
  double m = 0.0;
  int h = 0;
  if (e < a.E) {
    for (int c = slice; c < nc; c += 16 * slices) {
      uint2 r[16];  // in flight together
#pragma unroll
      for (int u = 0; u < 16; ++u) r[u] = from[min(c + u * slices, nc - 1) * W + e];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const bool in = c + u * slices < nc;
        m += (double)(in ? __uint_as_float(r[u].x) : 0.0f);
        h += in ? (int)r[u].y : 0;
      }
    }
  }
  sm[tid] = m;
  sh[tid] = h;
  act = wave_sum(act);
  bad = wave_sum(bad);
  if ((tid & 63) == 0) tally[tid >> 6] = make_int2(act, bad);
  __syncthreads();
  double v = 0.0;
  if (tid < a.E) {  // slice 0
    double mass = 0.0;
    int hits = 0;
#pragma unroll 8
    for (int q = 0; q < slices; ++q) {
      mass += sm[(q << lg) + tid];
      hits += sh[(q << lg) + tid];
    }
    a.counts[(long)root * a.E + tid] = hits;
    v = mass * (double)hits;
  }
  v = wave_sum(v);
  if ((tid & 63) == 0) part[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    act = bad = 0;
#pragma unroll
    for (int q = 0; q < RS_THREADS / 64; ++q) {
      s += part[q];
      act += tally[q].x;
      bad += tally[q].y;
    }
    a.active[root] = act;
    a.loss[root] = loss_of(a, s, act);
    if (root == 0 && a.err != nullptr) *a.err = bad;
  }
}

// The gradient: the token's softmax again from its logits, the chosen
// experts' terms placed through a row of LDS per token.
template <bool BF, int V>
__global__ __launch_bounds__(BWD_THREADS) void k_route_bwd(RouterArgs a) {
  constexpr int ROWS = BWD_THREADS / 16;
  __shared__ float place[ROWS][16 * V];
  int t0, nt, root;
  if (!chunk_of(a, blockIdx.x, a.chunk, t0, nt, root)) return;
  const int tid = threadIdx.x, j = tid & 15, row = tid >> 4;
  float* mine = place[row];
  float u[V], c = 0.0f;
  if (a.gloss != nullptr) {
    const float n = (float)max(a.active[root], 1);
    c = a.gloss[root] * (float)a.E / ((float)a.k * n * n);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) u[i] = 0.0f;
  if (a.gloss != nullptr) {
    int n[V];
#pragma unroll
    for (int i = 0; i < V; ++i) n[i] = a.counts[(long)root * a.E + min(j + 16 * i, a.E - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = j + 16 * i < a.E ? c * (float)n[i] : 0.0f;
  }
  for (int o = 0; o < nt; o += ROWS) {
    const bool in = o + row < nt;
    const long t = (long)t0 + min(o + row, nt - 1);
    int idx = -1;
    float g = 0.0f, lsel = 0.0f;
    if (a.gw != nullptr) {
      idx = a.idx[t * a.k + min(j, a.k - 1)];
      g = a.gw[t * a.k + min(j, a.k - 1)];
    }
    float l[V];
    const bool on = load_logits<BF, V>(a, t, j, in, l);
    if (!on || j >= a.k || idx < 0 || idx >= a.E) idx = -1;
    // the chosen logits, through the token's row of LDS
#pragma unroll
    for (int i = 0; i < V; ++i) mine[j + 16 * i] = l[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (idx >= 0) lsel = mine[idx];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bool strange = false;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      strange |= !(l[i] < INFINITY);
      top = max(top, key_of(l[i]));
    }
    top = row_max(top);
    const bool act = !row_any(strange) && top > KEY_NINF;
    const float mx = logit_of(top);
    float p[V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = act ? __expf(l[i] - mx) : 0.0f;
      sum += p[i];
    }
    const float inv = act ? 1.0f / row_sum(sum) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= inv;
      s += p[i] * u[i];
    }
    if (!act) idx = -1;
    if (idx < 0) g = 0.0f;  // whatever the buffer holds where there is no route
    float psel = idx >= 0 ? __expf(lsel - mx) : 0.0f;
    float term;
    if (a.renorm) {
      const float ws = row_sum(psel);
      const float wt = psel > 0.0f ? psel / ws : 0.0f;
      term = wt * (g - row_sum(wt * g));
    } else {
      term = psel * inv * g;
      s += term;
    }
    s = row_sum(s);
#pragma unroll
    for (int i = 0; i < V; ++i) mine[j + 16 * i] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (idx >= 0) mine[idx] = term;  // a row's ids are distinct
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (in) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = j + 16 * i;
        if (e < a.E) {
          const float d = act ? p[i] * (u[i] - s) + mine[e] : 0.0f;
          if (BF)
            ((uint16_t*)a.glogits)[t * a.E + e] = (uint16_t)f2bf(d);
          else
            ((float*)a.glogits)[t * a.E + e] = d;
        }
      }
    }
  }
}

int chunks_of(const RouterArgs& a) {
  int n = 0;
  for (int q = 0; q < a.na; ++q) n += (a.roots[q + 1] - a.roots[q] + a.chunk - 1) / a.chunk;
  return n;
}

// Few tokens: one launch, 3.8 us at one token (two: 3.7 and 2.9).  Beyond one
// round of its workgroup a round costs about 1.5 us and the sums lose their
// parallel chunks.
bool one_launch(const RouterArgs& a) { return a.na == 1 && a.T <= ONE_TOKENS; }

// experts a lane holds: the smallest of 4, 8, 16, 32 that covers E
template <template <bool, int> class F, class... A>
void by_shape(bool bf, int E, A&&... args) {
  if (E <= 64)
    bf ? F<true, 4>::go(args...) : F<false, 4>::go(args...);
  else if (E <= 128)
    bf ? F<true, 8>::go(args...) : F<false, 8>::go(args...);
  else if (E <= 256)
    bf ? F<true, 16>::go(args...) : F<false, 16>::go(args...);
  else
    bf ? F<true, 32>::go(args...) : F<false, 32>::go(args...);
}
template <bool BF, int V>
struct GoRoute {
  static void go(const RouterArgs& a, int n, hipStream_t st) {
    if (one_launch(a))
      MOE_LAUNCH_AS("k_route", (k_route<BF, V, true>), dim3(1), dim3(ONE_THREADS), 0, st, a);
    else
      MOE_LAUNCH_AS("k_route", (k_route<BF, V, false>), dim3(n), dim3(THREADS<V>), 0, st, a);
  }
};
template <bool BF, int V>
struct GoRouteBwd {
  static void go(const RouterArgs& a, int n, hipStream_t st) {
    MOE_LAUNCH_AS("k_route_bwd", (k_route_bwd<BF, V>), dim3(n), dim3(BWD_THREADS), 0, st, a);
  }
};

moe_status check_router(const moe_router_desc* d, const moe_adapters* ad, RouterArgs& a) {
  if (d == nullptr || d->T < 1 || d->E < 1 || d->topk < 1 || d->topk > d->E) return MOE_ERR_INVALID;
  if (d->renorm != 0 && d->renorm != 1) return MOE_ERR_INVALID;
  if (d->E > 512 || d->topk > 16) return MOE_ERR_UNSUPPORTED;
  if (d->logits_type != MOE_TYPE_F32 && d->logits_type != MOE_TYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (d->T > 1 << 30 || (int64_t)d->T * d->E >= (int64_t)1 << 31 || (int64_t)d->T * d->topk >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  a = RouterArgs{};
  a.T = d->T;
  a.E = d->E;
  a.k = d->topk;
  a.renorm = d->renorm;
  a.na = 1;
  a.roots[1] = d->T;
  const int mult = (d->T + RT_TOKENS * RT_CHUNKS - 1) / (RT_TOKENS * RT_CHUNKS);
  a.chunk = RT_TOKENS * (mult < RT_MOST ? mult : RT_MOST);
  if (ad == nullptr) return MOE_OK;
  if (ad->offsets == nullptr || ad->count < 1) return MOE_ERR_INVALID;
  if (ad->count > MAX_ADAPTERS) return MOE_ERR_UNSUPPORTED;
  if (ad->offsets[0] != 0 || ad->offsets[ad->count] != d->T) return MOE_ERR_INVALID;
  for (int q = 0; q < ad->count; ++q)
    if (ad->offsets[q + 1] < ad->offsets[q]) return MOE_ERR_INVALID;
  a.na = ad->count;
  for (int q = 0; q <= ad->count; ++q) a.roots[q] = ad->offsets[q];
  return MOE_OK;
}

size_t workspace_of(const RouterArgs& a) { return (size_t)chunks_of(a) * (a.E + 1) * sizeof(uint2); }

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

moe_status moe_router_workspace_size(const moe_router_desc* d, const moe_adapters* ad, size_t* bytes) {
  RouterArgs a;
  const moe_status st = check_router(d, ad, a);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID;
  *bytes = workspace_of(a);
  return MOE_OK;
}

moe_status moe_router_forward(const moe_router_desc* d, const moe_adapters* ad, const void* logits,
                              const uint8_t* valid, int32_t* topk_idx, float* topk_w, int32_t* counts,
                              int32_t* active, float* loss, int32_t* device_error, void* workspace,
                              size_t workspace_bytes, void* stream) {
  RouterArgs a;
  const moe_status st = check_router(d, ad, a);
  if (st != MOE_OK) return st;
  if (!aligned16(logits) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(counts, 4) ||
      !aligned(active, 4) || !aligned(loss, 4) || (device_error != nullptr && !aligned(device_error, 4)) ||
      !aligned16(workspace))
    return MOE_ERR_INVALID;
  const size_t need = workspace_of(a);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  const size_t le = d->logits_type == MOE_TYPE_BF16 ? 2 : 4, routes = (size_t)a.T * a.k;
  const Range ins[] = {rng(logits, (size_t)a.T * a.E * le), rng(valid, (size_t)a.T)};
  const Range outs[] = {rng(topk_idx, routes * 4), rng(topk_w, routes * 4), rng(counts, (size_t)a.na * a.E * 4),
                        rng(active, (size_t)a.na * 4), rng(loss, (size_t)a.na * 4), rng(device_error, 4),
                        rng(workspace, need)};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return MOE_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_ERR_INVALID;
  }
  a.logits = logits;
  a.valid = valid;
  a.idx = topk_idx;
  a.w = topk_w;
  a.counts = counts;
  a.active = active;
  a.loss = loss;
  a.err = device_error;
  a.sums = (uint2*)workspace;
  const int n = chunks_of(a);
  const hipStream_t s = (hipStream_t)stream;
  by_shape<GoRoute>(d->logits_type == MOE_TYPE_BF16, a.E, a, n, s);
  if (!one_launch(a)) MOE_LAUNCH(k_route_sum, dim3(a.na), dim3(RS_THREADS), 0, s, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_router_backward(const moe_router_desc* d, const moe_adapters* ad, const void* logits,
                               const uint8_t* valid, const int32_t* topk_idx, const int32_t* counts,
                               const int32_t* active, const float* grad_topk_w, const float* grad_loss,
                               void* grad_logits, void* stream) {
  RouterArgs a;
  const moe_status st = check_router(d, ad, a);
  if (st != MOE_OK) return st;
  if (!aligned16(logits) || !aligned16(grad_logits) || !aligned(topk_idx, 4) || !aligned(counts, 4) ||
      !aligned(active, 4) || (grad_topk_w != nullptr && !aligned(grad_topk_w, 4)) ||
      (grad_loss != nullptr && !aligned(grad_loss, 4)))
    return MOE_ERR_INVALID;
  const size_t le = d->logits_type == MOE_TYPE_BF16 ? 2 : 4, routes = (size_t)a.T * a.k;
  const Range ro = rng(grad_logits, (size_t)a.T * a.E * le), rl = rng(logits, (size_t)a.T * a.E * le);
  const Range ins[] = {rng(valid, (size_t)a.T), rng(topk_idx, routes * 4), rng(counts, (size_t)a.na * a.E * 4),
                       rng(active, (size_t)a.na * 4), rng(grad_topk_w, routes * 4),
                       rng(grad_loss, (size_t)a.na * 4)};
  if (grad_logits != logits && overlap(ro, rl)) return MOE_ERR_INVALID;
  for (const Range& r : ins)
    if (overlap(ro, r)) return MOE_ERR_INVALID;
  a.logits = logits;
  a.valid = valid;
  a.idx = const_cast<int32_t*>(topk_idx);
  a.counts = const_cast<int32_t*>(counts);
  a.active = const_cast<int32_t*>(active);
  a.gw = grad_topk_w;
  a.gloss = grad_loss;
  a.glogits = grad_logits;
  a.chunk = BWD_THREADS / 16;
  a.chunk *= (a.T + a.chunk * BWD_CHUNKS - 1) / (a.chunk * BWD_CHUNKS);
  by_shape<GoRouteBwd>(d->logits_type == MOE_TYPE_BF16, a.E, a, chunks_of(a), (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
