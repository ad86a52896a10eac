// Gated linear recurrence over packed sequences, and its gradients.
//
//   sigmoid   a_t = 1 / (1 + exp(-g_t)),  b_t = (1 - a_t) x_t
//   decay     a_t = gate[c],              b_t = x_t
//   h_t = a_t h_{t-1} + b_t                    (h before a sequence's first row: h0)
//   d_t = dh_t + a_{t+1} d_{t+1}               (last row: dh_t + dlast)
//   sigmoid   dx = d (1 - a),  dg = d a (1 - a) (h_{t-1} - x)
//   decay     dx = d,          dgate[c] = sum_t d_t h_{t-1}
//   dh0 = a d at the first row
//
// The state is fp32 throughout; the rounding of h to the storage type is of
// the output alone.  The gradient makes h_{t-1} again from the inputs, block
// by block of 32 rows, from the fp32 states that the forward pass kept.
#include "launch.h"
#include "projection.h"

namespace dspark {

namespace {

constexpr int kBlock = 32;   // rows from one kept state to the next

// Two neighbouring channels of a row, as stored, at element alignment.
template <typename T> struct Pair;
template <> struct Pair<bf16_t> {
  uint32_t raw;
  __device__ __forceinline__ void load(const bf16_t* p, bool both) {
    if (both)
      __builtin_memcpy(&raw, p, 4);
    else
      raw = *p;
  }
  __device__ __forceinline__ float get(int i) const { return i ? bf16_hi(raw) : bf16_lo(raw); }
};
template <> struct Pair<float> {
  u32x2_t raw;
  __device__ __forceinline__ void load(const float* p, bool both) {
    if (both) {
      __builtin_memcpy(&raw, p, 8);
    } else {
      raw[0] = __float_as_uint(*p);
      raw[1] = 0;
    }
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(raw[i]); }
};
template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b, bool both) {
  if (both) {
    T v[2] = {from_f32<T>(a), from_f32<T>(b)};
    __builtin_memcpy(p, v, 2 * sizeof(T));
  } else {
    *p = from_f32<T>(a);
  }
}

// a = 1 / (1 + exp(-g)) and 1 - a, each to its own relative accuracy: by
// exp(-|g|), so that nothing cancels for gates near 1.  An error of a is
// multiplied by the number of rows that a state lives, and states are fp32
// for both types: the reciprocal gets a Newton step.
template <typename T>
__device__ __forceinline__ void gate_of(float g, float* a, float* rest) {
  float e, r;
  if constexpr (sizeof(T) == 4) {
    e = expf(-fabsf(g));
    r = 1.f / (1.f + e);
  } else {
    e = __expf(-fabsf(g));
    const float d = 1.f + e;
    r = __builtin_amdgcn_rcpf(d);
    r = fmaf(r, fmaf(-d, r, 1.f), r);
  }
  const float small = e * r;
  *a = g >= 0.f ? r : small;
  *rest = g >= 0.f ? small : r;
  if (g != g) *a = *rest = g;
}

// First and last row (exclusive) of sequence s.
struct Sequences {
  const int32_t* offsets;   // null: `each` rows in every sequence
  int T, each;
  __device__ __forceinline__ int begin(int s) const { return offsets ? min(max(offsets[s], 0), T) : s * each; }
  __device__ __forceinline__ int end(int s) const { return offsets ? min(max(offsets[s + 1], 0), T) : (s + 1) * each; }
};

// One wave goes through its sequences row after row, R rows of loads at a
// time, two channels a lane.
template <typename T, bool SIGMOID, int R>
__global__ __launch_bounds__(256) void rows_kernel(Sequences seq, int S, int C, const T* __restrict__ x,
                                                   const void* __restrict__ gate, const float* h0, T* __restrict__ h,
                                                   float* last, float* __restrict__ states) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.x * 128 + 2 * lane;
  if (c >= C) return;
  const bool both = c + 1 < C;
  const T* gates = static_cast<const T*>(gate);
  float a0 = 0.f, a1 = 0.f;
  if (!SIGMOID) {
    a0 = static_cast<const float*>(gate)[c];
    a1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
  }
  for (int s = blockIdx.y * 4 + wave; s < S; s += gridDim.y * 4) {
    const int begin = seq.begin(s), end = seq.end(s);
    float s0 = 0.f, s1 = 0.f;
    if (h0) {
      s0 = h0[size_t(s) * C + c];
      if (both) s1 = h0[size_t(s) * C + c + 1];
    }
    for (int t0 = begin; t0 < end; t0 += R) {
      const int n = end - t0;
      Pair<T> px[R], pg[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          const size_t at = size_t(t0 + i) * C + c;
          px[i].load(x + at, both);
          if (SIGMOID) pg[i].load(gates + at, both);
        }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          const int t = t0 + i;
          if (states && t % kBlock == 0) store2(states + size_t(t / kBlock) * C + c, s0, s1, both);
          float b0 = px[i].get(0), b1 = px[i].get(1);
          if (SIGMOID) {
            float r0, r1;
            gate_of<T>(pg[i].get(0), &a0, &r0);
            gate_of<T>(pg[i].get(1), &a1, &r1);
            b0 *= r0;
            b1 *= r1;
          }
          s0 = fmaf(a0, s0, b0);
          s1 = fmaf(a1, s1, b1);
          store2(h + size_t(t) * C + c, s0, s1, both);
        }
    }
    if (last) store2(last + size_t(s) * C + c, s0, s1, both);
  }
}

// The same backwards, block by block of the kept states.  part[unit][C]: a
// wave's share of dgate (decay).
template <typename T, bool SIGMOID>
__global__ __launch_bounds__(256) void rows_backward_kernel(Sequences seq, int S, int C, const T* __restrict__ dh,
                                                            const T* __restrict__ x, const void* __restrict__ gate,
                                                            const float* __restrict__ h0, const float* dlast,
                                                            const float* __restrict__ states, T* __restrict__ dx,
                                                            T* __restrict__ dg, float* dh0, float* __restrict__ part) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.x * 128 + 2 * lane;
  if (c >= C) return;
  const bool both = c + 1 < C;
  const T* gates = static_cast<const T*>(gate);
  float decay0 = 0.f, decay1 = 0.f, sum0 = 0.f, sum1 = 0.f;
  if (!SIGMOID) {
    decay0 = static_cast<const float*>(gate)[c];
    decay1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
  }
  const int unit = blockIdx.y * 4 + wave;
  for (int s = unit; s < S; s += gridDim.y * 4) {
    const int begin = seq.begin(s), end = seq.end(s);
    float e0 = 0.f, e1 = 0.f;   // a d of the row behind
    if (dlast) {
      e0 = dlast[size_t(s) * C + c];
      if (both) e1 = dlast[size_t(s) * C + c + 1];
    }
    for (int k = end > begin ? (end - 1) / kBlock : -1; k >= 0 && k * kBlock + kBlock > begin; --k) {
      const int t0 = k * kBlock, lo = max(begin - t0, 0), hi = min(end - t0, kBlock);
      Pair<T> px[kBlock], pg[kBlock], pd[kBlock];
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (i >= lo && i < hi) {
          const size_t at = size_t(t0 + i) * C + c;
          px[i].load(x + at, both);
          if (SIGMOID) pg[i].load(gates + at, both);
          pd[i].load(dh + at, both);
        }
      const float* from = lo == 0 && t0 > begin ? states + size_t(k) * C + c : h0 ? h0 + size_t(s) * C + c : nullptr;
      float s0 = from ? from[0] : 0.f, s1 = from && both ? from[1] : 0.f;
      float before0[kBlock], before1[kBlock];
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (i >= lo && i < hi) {
          before0[i] = s0;
          before1[i] = s1;
          float a0 = decay0, a1 = decay1, b0 = px[i].get(0), b1 = px[i].get(1);
          if (SIGMOID) {
            float r0, r1;
            gate_of<T>(pg[i].get(0), &a0, &r0);
            gate_of<T>(pg[i].get(1), &a1, &r1);
            b0 *= r0;
            b1 *= r1;
          }
          s0 = fmaf(a0, s0, b0);
          s1 = fmaf(a1, s1, b1);
        }
      float here0 = 0.f, here1 = 0.f;
#pragma unroll
      for (int i = kBlock - 1; i >= 0; --i)
        if (i >= lo && i < hi) {
          const size_t at = size_t(t0 + i) * C + c;
          const float d0 = pd[i].get(0) + e0, d1 = pd[i].get(1) + e1;
          if (SIGMOID) {
            float a0, a1, r0, r1;
            gate_of<T>(pg[i].get(0), &a0, &r0);
            gate_of<T>(pg[i].get(1), &a1, &r1);
            if (dx) store2(dx + at, d0 * r0, d1 * r1, both);
            if (dg)
              store2(dg + at, d0 * r0 * (a0 * (before0[i] - px[i].get(0))), d1 * r1 * (a1 * (before1[i] - px[i].get(1))),
                     both);
            e0 = a0 * d0;
            e1 = a1 * d1;
          } else {
            if (dx) store2(dx + at, d0, d1, both);
            here0 = fmaf(d0, before0[i], here0);
            here1 = fmaf(d1, before1[i], here1);
            e0 = decay0 * d0;
            e1 = decay1 * d1;
          }
        }
      sum0 += here0;
      sum1 += here1;
    }
    if (dh0) store2(dh0 + size_t(s) * C + c, e0, e1, both);
  }
  if (part) store2(part + size_t(unit) * C + c, sum0, sum1, both);
}

// dgate[c] = sum over the units, eight threads per channel, joined in order.
__global__ __launch_bounds__(256) void gate_join_kernel(int C, int units, const float* __restrict__ part,
                                                        float* __restrict__ out) {
  __shared__ float sums[8][32];
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int u = q; u < units; u += 8) s += part[size_t(u) * C + c];
  }
  sums[q][l] = s;
  __syncthreads();
  if (q == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][l];
    out[c] = s;
  }
}

Sequences sequences(const RecurrenceArgs& a) { return {a.offsets, a.T, a.S > 0 ? a.T / a.S : 0}; }

// Workgroups of four waves along the sequences.
int groups(int S, bool backward) {
  const int g = (S + 3) / 4, most = backward ? 256 : 16384;
  return g < most ? g : most;
}

template <typename T, bool SIGMOID>
hipError_t forward_t(const RecurrenceArgs& a, hipStream_t stream) {
  if (a.S == 0) return hipSuccess;
  const dim3 grid((a.C + 127) / 128, groups(a.S, false));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, sequences(a), a.S, a.C, static_cast<const T*>(a.x), a.gate,
                       a.h0, static_cast<T*>(a.h), a.last, a.states);
    return hipGetLastError();
  };
  return a.T == a.S ? go(rows_kernel<T, SIGMOID, 1>) : go(rows_kernel<T, SIGMOID, 16>);
}

template <typename T, bool SIGMOID>
hipError_t backward_t(const RecurrenceArgs& a, hipStream_t stream) {
  const int g = groups(a.S, true);
  float* part = !SIGMOID && a.dgate ? static_cast<float*>(a.ws) : nullptr;
  hipError_t e = hipSuccess;
  if (a.S > 0) {
    hipLaunchKernelGGL((rows_backward_kernel<T, SIGMOID>), dim3((a.C + 127) / 128, g), dim3(256), 0, stream,
                       sequences(a), a.S, a.C, static_cast<const T*>(a.dh), static_cast<const T*>(a.x), a.gate, a.h0,
                       a.dlast, a.states_in, static_cast<T*>(a.dx), SIGMOID ? static_cast<T*>(a.dgate) : nullptr,
                       a.dh0, part);
    e = hipGetLastError();
  }
  if (SIGMOID || !a.dgate || e != hipSuccess) return e;
  hipLaunchKernelGGL(gate_join_kernel, dim3((a.C + 31) / 32), dim3(256), 0, stream, a.C, a.S > 0 ? 4 * g : 0, part,
                     static_cast<float*>(a.dgate));
  return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) { return 0; }
size_t recurrence_backward_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) {
  if (sigmoid) return 0;
  return (size_t(groups(S, true)) * 4 * C * 4 + 255) & ~size_t(255);
}

hipError_t launch_recurrence(const RecurrenceArgs& a, hipStream_t stream) {
  if (a.bf16) return a.sigmoid ? forward_t<bf16_t, true>(a, stream) : forward_t<bf16_t, false>(a, stream);
  return a.sigmoid ? forward_t<float, true>(a, stream) : forward_t<float, false>(a, stream);
}

hipError_t launch_recurrence_backward(const RecurrenceArgs& a, hipStream_t stream) {
  if (a.bf16) return a.sigmoid ? backward_t<bf16_t, true>(a, stream) : backward_t<bf16_t, false>(a, stream);
  return a.sigmoid ? backward_t<float, true>(a, stream) : backward_t<float, false>(a, stream);
}

}  // namespace dspark
