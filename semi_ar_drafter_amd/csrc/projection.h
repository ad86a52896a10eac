// Shared parts of the projection kernels (linear.hip, gated.hip,
// markov_loss.hip): the operand and tile descriptions and the epilogues.
//
// Every product is written as C(a, b) = sum_k A(a, k) * B(b, k).  The a axis
// is always the one that is contiguous in the output, because an MFMA
// accumulator holds four consecutive a of one b per lane: outputs are stored
// four values at a time, and a softmax over a needs only an in-lane reduction
// and two lane exchanges.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "device_util.h"

namespace dspark {

typedef uint16_t bf16_t;   // storage of a bfloat16

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16_t x) { return bf16_to_f32(x); }

// fp32 -> bf16, round to nearest even (NaN stays NaN): the only rounding of
// an output, after all sums have been made in fp32.
__device__ __forceinline__ bf16_t f32_to_bf16(float f) {
  const __bf16 h = (__bf16)f;
  return __builtin_bit_cast(bf16_t, h);
}
template <typename T> __device__ __forceinline__ T from_f32(float f);
template <> __device__ __forceinline__ float from_f32<float>(float f) { return f; }
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float f) { return f32_to_bf16(f); }

// Four consecutive values at p; `vec` (uniform): p is aligned for one wide access.
__device__ __forceinline__ f32x4_t load4(const float* p, int n, bool vec) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (vec && n >= 4) return *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] = p[i];
  return v;
}
__device__ __forceinline__ f32x4_t load4(const bf16_t* p, int n, bool vec) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (vec && n >= 4) {
    const u32x2_t u = *reinterpret_cast<const u32x2_t*>(p);
    v[0] = bf16_lo(u[0]);
    v[1] = bf16_hi(u[0]);
    v[2] = bf16_lo(u[1]);
    v[3] = bf16_hi(u[1]);
    return v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] = bf16_to_f32(p[i]);
  return v;
}
__device__ __forceinline__ void store4(float* p, f32x4_t v, int n, bool vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<f32x4_t*>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = v[i];
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4_t v, int n, bool vec) {
  if (vec && n >= 4) {
    typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
    const bf16x4_t h = __builtin_convertvector(v, bf16x4_t);   // two packed conversions, nearest even
    *reinterpret_cast<bf16x4_t*>(p) = h;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = f32_to_bf16(v[i]);
}

// Four stored values as they lie in memory, and widened: a tile's loads are
// all sent off before the first is used.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  f32x4_t v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const f32x4_t*>(p); }
  __device__ __forceinline__ f32x4_t wide() const { return v; }
};
template <> struct Raw4<bf16_t> {
  u32x2_t v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const u32x2_t*>(p); }
  __device__ __forceinline__ f32x4_t wide() const { return f32x4_t{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])}; }
};

// exp(x), x <= 0, of one logit: for fp32 storage to the last bit or two; for
// bf16 storage by the hardware's base-2 exponential, whose argument rounding
// costs |x| 2^-23 relative, far below the half step 2^-8 that dz is rounded by.
// In lse and nll, which are fp32, a term of share p = e^x / sum errs by p |x|
// 2^-23 of the sum: the mean of |x| over the softmax, below ln V, in units of
// 2^-23, as much as rounding a sum of lse's size to fp32 (measured against 64
// bits: 2e-7 of nll for 8 rows of V = 151936, 5e-7 for 1024 rows of 129280, the
// plain fp32 form 2e-7 and 1e-6).
// The partial sums of tiles are joined with __expf for both types: |x| 2^-23
// relative again, of a share of at most e^x, and |x| e^x <= 1 / e: below 2^-24
// of the sum.
template <typename T> __device__ __forceinline__ float exp_of(float x);
template <> __device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ float exp_of<bf16_t>(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// Lets a kernel use `bytes` of LDS on the current device: once per kernel and
// device (the attribute belongs to both).
inline hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& devices) {
  int d = 0;
  hipError_t e = hipGetDevice(&d);
  if (e != hipSuccess) return e;
  const uint64_t bit = d < 64 ? uint64_t(1) << d : 0;
  if (bit && (devices.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// One operand: element (a, k) at p[a * sa + k * sk], one of the strides 1;
// a in [0, n).
template <typename T>
struct Operand {
  const T* p;
  long sa, sk;
  int n;
};

// A product whose contraction has up to two parts (the output projection and
// the Markov factor share one accumulator).
template <typename T>
struct Product {
  Operand<T> A[2], B[2];
  int K[2];
  // Device-side sizes, where a host does not know them (rows that have a
  // label): the number of b in use, and the length of the first contraction.
  const int* nb = nullptr;
  const int* k0 = nullptr;
};

// Where a wave's accumulators lie: acc[i][j][e] is C(a0 + 16 i + 4 (lane / 16)
// + e, b0 + 16 j + lane % 16).  tile_a: index of the workgroup's tile along a;
// wave_a of waves_a: the wave's place along a inside it.
struct TileAt {
  int a0, b0, nb, tile_a, wave_a, wave_b;
};

// ---------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------
// The normal distribution's integral P(z) and density times sqrt(2 pi),
// exp(-z^2 / 2).  P by way of erfc(-z / sqrt 2), which keeps its relative
// accuracy for negative z, where 1 + erf loses it (10 % at z = -5 in fp32).
// fp32 storage takes the library's function.  For bf16 storage erfc(x) =
// t q(t) exp(-x^2), t = 1 / (1 + p x), x = |z| / sqrt 2, whose exponential is
// the density's: q of degree 6, p and q fitted to exp(x^2) erfc(x) on [0, 9.6]
// for the least relative error, 6e-7 (about 17 instructions instead of 60).
template <typename T> __device__ __forceinline__ float normal_cdf(float z, float* e);
template <> __device__ __forceinline__ float normal_cdf<float>(float z, float* e) {
  *e = expf(-0.5f * z * z);
  return 0.5f * erfcf(z * -0.70710678118654752f);
}
template <> __device__ __forceinline__ float normal_cdf<bf16_t>(float z, float* e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(1.f + 0.3725f * x);
  *e = __expf(-x * x);
  float q = -0.1394701151540878f;
  q = q * t + 0.41369502739896746f;
  q = q * t - 0.16042987722460397f;
  q = q * t + 0.3019267804465362f;
  q = q * t + 0.15901532659798573f;
  q = q * t + 0.21541323049746136f;
  q = q * t + 0.20984971869445848f;
  const float tail = 0.5f * q * t * *e;   // P(-|z|)
  return z < 0.f ? tail : 1.f - tail;
}
template <typename T> __device__ __forceinline__ float sigmoid(float z);
template <> __device__ __forceinline__ float sigmoid<float>(float z) { return 1.f / (1.f + expf(-z)); }
template <> __device__ __forceinline__ float sigmoid<bf16_t>(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}

template <typename T>
__device__ __forceinline__ float act_value(int act, float z) {
  float e;
  if (act == 1) return z < 0.f ? 0.f : z;   // NaN stays NaN
  if (act == 2) return z * normal_cdf<T>(z, &e);
  if (act == 3) return z * sigmoid<T>(z);
  return z;
}
// d act / dz (relu: 0 at 0, NaN at NaN)
template <typename T>
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == 1) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
  if (act == 2) {
    float e;
    const float c = normal_cdf<T>(z, &e);
    return c + z * 0.39894228040143268f * e;
  }
  if (act == 3) {
    const float s = sigmoid<T>(z);
    return s + z * s * (1.f - s);
  }
  return 1.f;
}

// ---------------------------------------------------------------------------
// Epilogues.  init() fills the accumulators before the product, done() takes
// them after it; lds is the workgroup's shared memory, free by then.
// ---------------------------------------------------------------------------
template <int FM, int FN>
__device__ __forceinline__ void acc_zero(f32x4_t (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// y[b][a] = act(C + bias[a]) + residual[b][a]; pre[b][a] = C + bias[a] if asked for.
template <typename T>
struct LinearEpi {
  const T* bias;
  const T* residual;
  T* y;
  float* pre;
  int act, na;
  bool vec;   // rows of na values keep four-value alignment, and so does bias
  // of the rows from b on (a multiple of four)
  LinearEpi from(int b) const {
    LinearEpi r = *this;
    const size_t at = size_t(b) * na;
    r.y += at;
    if (r.residual) r.residual += at;
    if (r.pre) r.pre += at;
    return r;
  }
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt&) const {
    acc_zero(acc);
  }
  // four values from (b, a) on, n of them inside the row; bias and residual
  // already widened
  __device__ __forceinline__ void finish(f32x4_t v, f32x4_t bv, f32x4_t rv, int b, int a, int n) const {
    v += bv;
    const size_t at = size_t(b) * na + a;
    if (pre) store4(pre + at, v, n, vec);
    if (act) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value<T>(act, v[e]);
    }
    if (residual) v += rv;
    store4(y + at, v, n, vec);
  }
  __device__ __forceinline__ void join(f32x4_t v, int b, int a, int n) const {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    finish(v, bias ? load4(bias + a, n, vec) : zero, residual ? load4(residual + size_t(b) * na + a, n, vec) : zero, b, a, n);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
    const int a_lane = t.a0 + 4 * (lane >> 4), b_lane = t.b0 + (lane & 15);
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (vec && t.a0 + 16 * FM <= na && t.b0 + 16 * FN <= t.nb) {   // the wave's part lies inside
      Raw4<T> bv[FM];
      if (bias) {
#pragma unroll
        for (int i = 0; i < FM; ++i) bv[i].load(bias + a_lane + 16 * i);
      }
      // two columns of tiles at a time: their residuals are on the way together
      constexpr int G = FN % 2 ? 1 : 2;
#pragma unroll
      for (int j0 = 0; j0 < FN; j0 += G) {
        Raw4<T> rv[G][FM];
        if (residual) {
#pragma unroll
          for (int j = 0; j < G; ++j)
#pragma unroll
            for (int i = 0; i < FM; ++i)
              rv[j][i].load(residual + size_t(b_lane + 16 * (j0 + j)) * na + a_lane + 16 * i);
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int i = 0; i < FM; ++i)
            finish(acc[i][j0 + j], bias ? bv[i].wide() : zero, residual ? rv[j][i].wide() : zero,
                   b_lane + 16 * (j0 + j), a_lane + 16 * i, 4);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int a = a_lane + 16 * i;
      if (a >= na) continue;
      const f32x4_t bv = bias ? load4(bias + a, na - a, false) : zero;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = b_lane + 16 * j;
        if (b >= t.nb) continue;
        const f32x4_t rv = residual ? load4(residual + size_t(b) * na + a, na - a, vec) : zero;
        finish(acc[i][j], bv, rv, b, a, na - a);
      }
    }
  }
};

// out[b][a] = C as T (row stride ld): a weight gradient.
template <typename T>
struct StoreEpi {
  T* out;
  long ld;
  int na;
  bool vec;
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt&) const {
    acc_zero(acc);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int a = t.a0 + 16 * i + 4 * (lane >> 4);
      if (a >= na) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15);
        if (b < t.nb) store4(out + size_t(b) * ld + a, acc[i][j], na - a, vec);
      }
    }
  }
};

// sum[b][a] (+)= C in fp32 (row stride ld, a multiple of 4): a row gradient
// gathered over the pieces of the vocabulary, in piece order.
struct AddEpi {
  float* sum;
  long ld;
  int na;
  bool first;
  long split = 0;   // split s of the contraction sums into sum + s * split
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt& t) const {
    acc_zero(acc);
    if (first) return;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int a = t.a0 + 16 * i + 4 * (lane >> 4);
      if (a >= na) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15);
        if (b < t.nb) acc[i][j] = load4(sum + blockIdx.y * split + size_t(b) * ld + a, na - a, true);
      }
    }
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int a = t.a0 + 16 * i + 4 * (lane >> 4);
      if (a >= na) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15);
        if (b < t.nb) store4(sum + blockIdx.y * split + size_t(b) * ld + a, acc[i][j], na - a, true);
      }
    }
  }
};

// The logits' share of the loss kernels: a is a token id (from v0 on), b a
// compact row; U[row[b]][v0 + a] starts the accumulator if base logits are
// given.
template <typename T>
struct BaseLogits {
  const T* U;
  const int* row;
  long V;
  int v0, na;
  bool vec;   // v0 and V keep four-value alignment
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt& t) const {
    acc_zero(acc);
    if (!U) return;
    const int lane = threadIdx.x & 63, a0 = t.a0 + 4 * (lane >> 4);
    const T* u[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)   // rows behind the last one read it again
      u[j] = U + size_t(row[min(t.b0 + 16 * j + (lane & 15), t.nb - 1)]) * V + v0 + a0;
    if (vec && t.a0 + 16 * FM <= na) {
      Raw4<T> raw[FM][FN];
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) raw[i][j].load(u[j] + 16 * i);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j] = raw[i][j].wide();
      return;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        if (a0 + 16 * i < na) acc[i][j] = load4(u[j] + 16 * i, na - a0 - 16 * i, vec);
  }
};

// Softmax statistics of one tile of the vocabulary: stat[tile_a][b] = (max,
// sum of exp(z - max)) in fp32; zlab[b] = the logit of the row's label, by
// the tile that holds it.  A tile whose logits are all -inf (masked base
// logits) has max -inf and sum 0.
template <typename T, int WAVES_A, int BN>
struct StatsEpi {
  BaseLogits<T> base;
  const int* label;   // by compact row, as lse and g below
  float2* stat;       // [tiles][stat_ld]
  long stat_ld;
  float* zlab;
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt& t) const {
    base.init(acc, t);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void* lds) const {
    const int lane = threadIdx.x & 63;
    float2* part = static_cast<float2*>(lds);   // [WAVES_A][BN]
    const float ninf = -__builtin_huge_valf();
    int labels[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) labels[j] = label[min(t.b0 + 16 * j + (lane & 15), t.nb - 1)] - base.v0;
    if (t.a0 + 16 * FM > base.na) {   // tokens behind the vocabulary's end
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t.a0 + 16 * i + 4 * (lane >> 4) + e >= base.na) {
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j][e] = ninf;
          }
    }
    // few waves hold the label of any of their rows
    bool mine = false;
#pragma unroll
    for (int j = 0; j < FN; ++j) mine |= unsigned(labels[j] - t.a0) < unsigned(16 * FM);
    if (__any(mine)) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15), y = b < t.nb ? labels[j] : -1;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t.a0 + 16 * i + 4 * (lane >> 4) + e == y) zlab[b] = acc[i][j][e];
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      float m = ninf;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, acc[i][j][e]);
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const float ref = m == ninf ? 0.f : m;
      // four sums: the additions do not wait for one another
      f32x4_t part4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) part4[e] += exp_of<T>(acc[i][j][e] - ref);
      float s = (part4[0] + part4[1]) + (part4[2] + part4[3]);
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (lane < 16) part[t.wave_a * BN + t.wave_b * 16 * FN + 16 * j + lane] = make_float2(m, s);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < BN; c += blockDim.x) {
      const int b = t.b0 - t.wave_b * 16 * FN + c;
      if (b >= t.nb) continue;
      float2 q = part[c];
      for (int w = 1; w < WAVES_A; ++w) {
        const float2 o = part[w * BN + c];
        const float m = fmaxf(q.x, o.x);
        const float ref = m == ninf ? 0.f : m;
        q.y = q.y * __expf(q.x - ref) + o.y * __expf(o.x - ref);
        q.x = m;
      }
      stat[size_t(t.tile_a) * stat_ld + b] = q;
    }
  }
};

// Gradient of the loss by the logits, of one piece of the vocabulary:
// dz[b][a] = g (exp(z - lse) - [a is the label]), rounded to T because the
// next products take it in T: the matrix unit multiplies bf16 by bf16, and
// keeping the rounded-off part as a second operand would double two of the
// four products.  With the rounding of the result, which errs as much, that
// gives 1.4 times the result's rounding alone (2.3e-3 against 1.7e-3 of the
// norm; up to twice it below 16 rows, where one dz makes most of a gradient).
// fp32 storage rounds nothing here.  Rows of dz behind the last one in use are left
// alone; dU, if asked for, gets the same values.
template <typename T>
struct GradEpi {
  BaseLogits<T> base;
  const int* label;
  const float* lse;
  const float* g;
  T* dz;
  long dz_ld;
  T* dU;
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt& t) const {
    base.init(acc, t);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
    int labels[FN];
    float lses[FN], gs[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int b = min(t.b0 + 16 * j + (lane & 15), t.nb - 1);
      labels[j] = label[b] - base.v0;
      lses[j] = lse[b];
      gs[j] = g[b];
    }
    const bool edge = t.a0 + 16 * FM > base.na;
    bool mine = edge;
#pragma unroll
    for (int j = 0; j < FN; ++j) mine |= unsigned(labels[j] - t.a0) < unsigned(16 * FM);
    mine = __any(mine);   // few waves hold the label of any of their rows, or the vocabulary's end
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int b = t.b0 + 16 * j + (lane & 15);
      if (b >= t.nb) continue;
      T* u = dU ? dU + size_t(base.row[b]) * base.V + base.v0 : nullptr;
      T* out = dz + size_t(b) * dz_ld;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int a = t.a0 + 16 * i + 4 * (lane >> 4);
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = exp_of<T>(acc[i][j][e] - lses[j]);
        if (mine) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = a + e >= base.na ? 0.f : a + e == labels[j] ? v[e] - 1.f : v[e];
        }
        v *= gs[j];
        // the piece's width dz_ld is a multiple of the tile: every a of the tile is inside it
        store4(out + a, v, 4, true);
        if (dU && a < base.na) store4(u + a, v, base.na - a, base.vec);
      }
    }
  }
};

}  // namespace dspark
