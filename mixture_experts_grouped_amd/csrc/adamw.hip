// adamw.hip -- one AdamW step over many tensors, moments in fp32 or in 8 bits
// per 128 elements (include/moelora.h states the formulas).
//
// One pass over memory: a thread takes eight consecutive elements, so bf16
// operands move 16 bytes a lane and codes 8; the sixteen lanes of a DPP row
// hold one run of 128 elements, whose largest moments are four DPP maxima.
// The tensors' pointers travel in the kernel argument (as many per launch as
// 4 KB hold: 100 with fp32 moments, 63 with masters and 8-bit ones); a workgroup
// finds its tensor by ballots over the tensors' first chunks.
//
// Memory bounds it, and vector instructions not far behind: the production
// factors (52 M elements, bf16 parameters and gradients, fp32 masters, 8-bit
// moments: 16 bytes an element) take 157 us, 5.4 TB/s of the 6.5 that a plain
// copy kernel reaches, with 79 vector instructions an element in 73 % of their
// issue slots; 96 tensors of 14,080 fp32 elements on average, one launch, 9.7 us
// (8.6 with inputs left in the caches; two launches of 48 took 12.5 where one
// took 9.2); 110 K elements in six tensors 4.2 us, latency.
#include <cmath>

#include "../../include/moelora.h"
#include "checks.hpp"
#include "lanes.hpp"
#include "trace.hpp"

namespace moelora {
namespace {

constexpr int AW_THREADS = 256;
constexpr int AW_CHUNK = AW_THREADS * 8;  // elements of a workgroup's chunk
constexpr size_t AW_ARGS = 4096;          // bytes of kernel arguments
constexpr int64_t AW_GRID = 1 << 23;      // chunks of a launch (it holds fewer than 2^32 threads)
constexpr float E4M3_MAX = 448.0f, E5M2_MAX = 57344.0f;
constexpr float TINY = 0x1p-100f;  // below it a run's moments count as zero (its reciprocal would overflow)

struct AdamwHead {
  int count, chunks;
  float b1, omb1, b2, omb2, eps, wd;
  float lr, bias1, bias2, gscale;
  uint32_t seed;
  const moe_adamw_control* control;
};
// One tensor's buffers; only those that the call's kinds have, so that as
// many tensors as possible go into one launch.
struct AwBase {
  void* param;
  const void* grad;
  void *m, *v;
  int first;      // the tensor's first chunk; its chunks end where the next one's begin
  uint32_t tail;  // elements missing from its last chunk
};
template <bool MASTER>
struct AwMaster {
  float* master;
};
template <>
struct AwMaster<false> {};
template <bool S8>
struct AwScales {
  float *m_scale, *v_scale;
};
template <>
struct AwScales<false> {};
template <bool MASTER, bool S8>
struct AwTensor : AwBase, AwMaster<MASTER>, AwScales<S8> {};
template <bool MASTER, bool S8>
struct AdamwArgs : AdamwHead {
  static constexpr int FIT = (AW_ARGS - sizeof(AdamwHead)) / sizeof(AwTensor<MASTER, S8>), MAX = FIT < 128 ? FIT : 128;
  AwTensor<MASTER, S8> t[MAX];
};

__device__ __forceinline__ uint32_t noise_of(uint32_t i, uint32_t seed) {
  uint32_t x = i * 0x9E3779B9u + seed;
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// one rounding each, never fused with another operation
__device__ __forceinline__ float mul1(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}
__device__ __forceinline__ float add1(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// eight values of a T tensor at p + i; those past n read zero
template <class T>
__device__ __forceinline__ void load8(const T* p, long i, long n, float (&v)[8]) {
  constexpr bool BF = sizeof(T) == 2;
  if (i + 8 <= n) {
    if constexpr (BF) {
      const u32x4 w = *(const u32x4*)(p + i);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[2 * c] = bf2f(w[c] & 0xffffu);
        v[2 * c + 1] = bf2f(w[c] >> 16);
      }
    } else {
      const f32x4 a = *(const f32x4*)(p + i), b = *(const f32x4*)(p + i + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = a[c];
        v[4 + c] = b[c];
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[c] = 0.0f;
      if (i + c < n) v[c] = BF ? bf2f(((const uint16_t*)p)[i + c]) : ((const float*)p)[i + c];
    }
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, long i, long n, const float (&v)[8]) {
  constexpr bool BF = sizeof(T) == 2;
  if (i + 8 <= n) {
    if constexpr (BF) {
      *(u32x4*)(p + i) = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    } else {
      *(f32x4*)(p + i) = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4*)(p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (i + c < n) {
        if constexpr (BF)
          p[i + c] = (uint16_t)f2bf(v[c]);
        else
          p[i + c] = v[c];
      }
  }
}
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, long i, long n) {
  if (i + 8 <= n) return *(const u32x2*)(p + i);
  uint64_t w = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (i + c < n) w |= (uint64_t)p[i + c] << (8 * c);
  return u32x2{(uint32_t)w, (uint32_t)(w >> 32)};
}
__device__ __forceinline__ void store_codes(uint8_t* p, long i, long n, u32x2 w) {
  if (i + 8 <= n) {
    *(u32x2*)(p + i) = w;
    return;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (i + c < n) p[i + c] = (uint8_t)(w[c >> 2] >> (8 * (c & 3)));
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
template <bool E5M2>
__device__ __forceinline__ void decode(u32x2 w, float s, float (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    f32x2 lo, hi;
    if constexpr (E5M2) {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[c], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[c], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[c], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[c], true);
    }
    v[4 * c] = lo[0] * s;
    v[4 * c + 1] = lo[1] * s;
    v[4 * c + 2] = hi[0] * s;
    v[4 * c + 3] = hi[1] * s;
  }
}

// Codes of a run's eight values in this lane.  `noise`: random bits, of which
// the conversion takes the upper ones as u, adds u times the format's step at y
// below the last kept place and cuts: floor(|y| / step + u) * step, the step
// 2^-9 (e4m3) or 2^-16 (e5m2) below the normal range.  Only 16 bits are set, so
// y's own bits below 2^-16 of a step do not matter.  Adding the noise to y's fp32
// mantissa and rounding to nearest instead puts it below the place that the
// format keeps once y is subnormal: such moments were rounded to nearest, so
// that small ones neither grew nor decayed.
// Returns the run's scale.  A maximum that is not finite makes the scale so.
template <bool E5M2>
__device__ __forceinline__ float encode(const float (&x)[8], const uint32_t (&noise)[8], u32x2& w) {
  constexpr float TOP = E5M2 ? E5M2_MAX : E4M3_MAX;
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) m = max(m, mag(x[c]));
  const float amax = __uint_as_float(row_max(m));
  const bool zero = amax < TINY;
  const float inv = zero ? 0.0f : mul1(1.0f / amax, TOP);
  float y[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    y[c] = fminf(fmaxf(x[c] * inv, E5M2 ? 0.0f : -TOP), TOP);
    if (E5M2 && x[c] > 0.0f) y[c] = fmaxf(y[c], 0x1p-16f);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int p = 0;
    if constexpr (E5M2) {
      p = __builtin_amdgcn_cvt_sr_bf8_f32(y[4 * h], (int)noise[4 * h], p, 0);
      p = __builtin_amdgcn_cvt_sr_bf8_f32(y[4 * h + 1], (int)noise[4 * h + 1], p, 1);
      p = __builtin_amdgcn_cvt_sr_bf8_f32(y[4 * h + 2], (int)noise[4 * h + 2], p, 2);
      p = __builtin_amdgcn_cvt_sr_bf8_f32(y[4 * h + 3], (int)noise[4 * h + 3], p, 3);
    } else {
      p = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * h], (int)noise[4 * h], p, 0);
      p = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * h + 1], (int)noise[4 * h + 1], p, 1);
      p = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * h + 2], (int)noise[4 * h + 2], p, 2);
      p = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * h + 3], (int)noise[4 * h + 3], p, 3);
    }
    w[h] = (uint32_t)p;
  }
  return zero ? 0.0f : amax * (1.0f / TOP);
}

template <class P, class G, bool MASTER, bool S8>
__global__ __launch_bounds__(AW_THREADS) void k_adamw(AdamwArgs<MASTER, S8> a) {
  const int lane = threadIdx.x & 63;
  // the last tensor whose first chunk is not past this one (none is empty)
  int q = -1;
#pragma unroll
  for (int h = 0; h < a.MAX; h += 64) {
    const int i = h + lane;
    q += __popcll(__ballot(i < a.count && a.t[i < a.count ? i : 0].first <= (int)blockIdx.x));
  }
  const AwTensor<MASTER, S8>& t = a.t[q];
  const int end = q + 1 < a.count ? a.t[q + 1 < a.MAX ? q + 1 : q].first : a.chunks;
  const long n = (long)(end - t.first) * AW_CHUNK - t.tail;
  const long i = (long)((int)blockIdx.x - t.first) * AW_CHUNK + 8 * threadIdx.x;
  float lr = a.lr, c1 = a.bias1, c2 = a.bias2, gs = a.gscale;
  uint32_t seed = a.seed;
  if (a.control != nullptr) {
    lr = a.control->lr;
    c1 = a.control->bias1;
    c2 = a.control->bias2;
    gs = a.control->grad_scale;
    seed = a.control->seed;
  }
  const float step = lr / c1, ic2 = 1.0f / c2, decay = lr * a.wd;
  float p[8], g[8], m[8], v[8];
  load8((const G*)t.grad, i, n, g);
  if constexpr (MASTER)
    load8(t.master, i, n, p);
  else
    load8((const P*)t.param, i, n, p);
  const long run = i >> 7;
  if constexpr (S8) {
    const float ms = i < n ? t.m_scale[run] : 0.0f, vs = i < n ? t.v_scale[run] : 0.0f;
    decode<false>(load_codes((const uint8_t*)t.m, i, n), ms, m);
    decode<true>(load_codes((const uint8_t*)t.v, i, n), vs, v);
  } else {
    load8((const float*)t.m, i, n, m);
    load8((const float*)t.v, i, n, v);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float gc = mul1(g[c], gs);
    // one rounding an operation, none fused: which code a moment is rounded to
    // then follows from the inputs alone, for anyone who computes it again
    m[c] = add1(mul1(m[c], a.b1), mul1(gc, a.omb1));
    v[c] = add1(mul1(v[c], a.b2), mul1(mul1(gc, gc), a.omb2));
    // the whole change first, then one subtraction: 1 - decay in fp32 would be
    // off by up to 2^-25 in every step alike (all of a decay below that)
    p[c] -= fmaf(decay, p[c], step * m[c] / (sqrtf(v[c] * ic2) + a.eps));
  }
  store8((P*)t.param, i, n, p);
  if constexpr (MASTER) store8(t.master, i, n, p);
  if constexpr (S8) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t r = noise_of((uint32_t)(i + c), seed);
      lo[c] = r << 16;
      hi[c] = r & 0xFFFF0000u;
    }
    u32x2 w;
    const float ms = encode<false>(m, lo, w);
    store_codes((uint8_t*)t.m, i, n, w);
    const float vs = encode<true>(v, hi, w);
    store_codes((uint8_t*)t.v, i, n, w);
    if ((lane & 15) == 0 && i < n) {
      t.m_scale[run] = ms;
      t.v_scale[run] = vs;
    }
  } else {
    store8((float*)t.m, i, n, m);
    store8((float*)t.v, i, n, v);
  }
}

template <class P, class G, bool MASTER, bool S8>
void launch_all(const AdamwHead& head, const moe_adamw_tensor* tensors, int count, hipStream_t st) {
  AdamwArgs<MASTER, S8> a;
  (AdamwHead&)a = head;
  a.count = a.chunks = 0;
  auto flush = [&]() {
    if (a.count != 0)
      MOE_LAUNCH_AS("k_adamw", (k_adamw<P, G, MASTER, S8>), dim3(a.chunks), dim3(AW_THREADS), 0, st, a);
    a.count = a.chunks = 0;
  };
  for (int q = 0; q < count; ++q) {
    const moe_adamw_tensor& s = tensors[q];
    if (s.n == 0) continue;
    const int64_t chunks = (s.n + AW_CHUNK - 1) / AW_CHUNK;  // at most AW_GRID
    if (a.count == a.MAX || a.chunks + chunks > AW_GRID) flush();
    AwTensor<MASTER, S8>& t = a.t[a.count++];
    t.param = s.param;
    t.grad = s.grad;
    t.m = s.m;
    t.v = s.v;
    t.first = a.chunks;
    t.tail = (uint32_t)(chunks * AW_CHUNK - s.n);
    if constexpr (MASTER) t.master = s.master;
    if constexpr (S8) {
      t.m_scale = s.m_scale;
      t.v_scale = s.v_scale;
    }
    a.chunks += (int)chunks;
  }
  flush();
}
template <class P, class G, bool MASTER>
void launch_states(const AdamwHead& h, bool s8, const moe_adamw_tensor* t, int count, hipStream_t st) {
  s8 ? launch_all<P, G, MASTER, true>(h, t, count, st) : launch_all<P, G, MASTER, false>(h, t, count, st);
}
template <class G>
void launch_params(const AdamwHead& h, const moe_adamw_desc* d, bool master, const moe_adamw_tensor* t, int count,
                   hipStream_t st) {
  const bool s8 = d->state_bits == 8;
  if (d->param_type == MOE_TYPE_F32)
    launch_states<float, G, false>(h, s8, t, count, st);
  else if (master)
    launch_states<uint16_t, G, true>(h, s8, t, count, st);
  else
    launch_states<uint16_t, G, false>(h, s8, t, count, st);
}

bool unit(double b) { return b >= 0.0 && b < 1.0; }  // false for NaN
bool finite(double v) { return std::isfinite((float)v); }  // as the kernel takes it
bool positive(double v) { return finite(v) && v >= 0.0; }

moe_status check_adamw(const moe_adamw_desc* d) {
  if (d == nullptr) return MOE_ERR_INVALID;
  for (const int32_t t : {d->param_type, d->grad_type})
    if (t != MOE_TYPE_F32 && t != MOE_TYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (d->state_bits != 32 && d->state_bits != 8) return MOE_ERR_UNSUPPORTED;
  if (!unit(d->beta1) || !unit(d->beta2) || !positive(d->weight_decay) || !finite(d->eps) || !((float)d->eps > 0.0f))
    return MOE_ERR_INVALID;
  if (d->control != nullptr) return aligned(d->control, 4) ? MOE_OK : MOE_ERR_INVALID;
  if (!positive(d->lr) || !finite(d->grad_scale) || d->step < 1) return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_tensor(const moe_adamw_desc* d, const moe_adamw_tensor& t, bool master) {
  const size_t pb = d->param_type == MOE_TYPE_BF16 ? 2 : 4, gb = d->grad_type == MOE_TYPE_BF16 ? 2 : 4;
  const size_t sb = d->state_bits / 8, n = (size_t)t.n, runs = (n + 127) / 128;
  if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v)) return MOE_ERR_INVALID;
  if (master ? !aligned16(t.master) : t.master != nullptr) return MOE_ERR_INVALID;
  const bool s8 = d->state_bits == 8;
  if (s8 ? !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4) : t.m_scale != nullptr || t.v_scale != nullptr)
    return MOE_ERR_INVALID;
  const Range r[] = {rng(t.grad, n * gb), rng(t.param, n * pb), rng(t.master, n * 4), rng(t.m, n * sb),
                     rng(t.v, n * sb), rng(t.m_scale, runs * 4), rng(t.v_scale, runs * 4)};
  for (int i = 0; i < 7; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(r[i], r[j])) return MOE_ERR_INVALID;
  return MOE_OK;
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" moe_status moe_adamw_step(const moe_adamw_desc* d, const moe_adamw_tensor* tensors, int32_t count,
                                     void* stream) {
  const moe_status st = check_adamw(d);
  if (st != MOE_OK) return st;
  if (count < 0 || (count > 0 && tensors == nullptr)) return MOE_ERR_INVALID;
  bool master = false, any = false;
  for (int q = 0; q < count; ++q) {
    if (tensors[q].n < 0) return MOE_ERR_INVALID;
    if (tensors[q].n == 0) continue;
    if (tensors[q].n > AW_GRID * AW_CHUNK) return MOE_ERR_UNSUPPORTED;
    if (!any) master = tensors[q].master != nullptr;
    any = true;
    if (master && d->param_type != MOE_TYPE_BF16) return MOE_ERR_INVALID;
    const moe_status s = check_tensor(d, tensors[q], master);
    if (s != MOE_OK) return s;
  }
  if (!any) return MOE_OK;
  AdamwHead a{};
  a.b1 = (float)d->beta1;
  a.omb1 = (float)(1.0 - d->beta1);
  a.b2 = (float)d->beta2;
  a.omb2 = (float)(1.0 - d->beta2);
  a.eps = (float)d->eps;
  a.wd = (float)d->weight_decay;
  a.lr = (float)d->lr;
  a.bias1 = (float)(1.0 - std::pow(d->beta1, (double)d->step));
  a.bias2 = (float)(1.0 - std::pow(d->beta2, (double)d->step));
  a.gscale = (float)d->grad_scale;
  a.seed = d->seed;
  a.control = d->control;
  const hipStream_t s = (hipStream_t)stream;
  if (d->grad_type == MOE_TYPE_BF16)
    launch_params<uint16_t>(a, d, master, tensors, count, s);
  else
    launch_params<float>(a, d, master, tensors, count, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
