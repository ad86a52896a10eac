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

// ---------------------------------------------------------------------------
// Long sequences: the rows are split into tiles as well
// ---------------------------------------------------------------------------
// A tile is W waves of 32 rows by 128 channels, read once and kept in
// registers.  What rows do to the state before them is h -> A h + B; a wave
// makes its (A, B), LDS joins the waves', and the tile's is published.  The
// state before the tile is then the fold, in order, of the published pairs
// since the last kept state; every kGroup-th tile publishes the state behind
// it, so that no fold is longer than kGroup and the tiles wait for one another
// once in kGroup only.  The order of all sums is fixed: results do not depend
// on which tile comes first.
//
// A tile takes its number (rows first, then channels) from a counter, so
// that every tile it waits for belongs to a workgroup that is already running
// and itself waits for lower numbers only.
//
// Where a sequence begins, A = 0 and B holds what its h0 gives: join() then
// ignores the state before, whatever it is.
constexpr int kGroup = 16;
constexpr int kSpin = 1 << 22;   // polls of a few hundred nanoseconds; a state not seen by then is NaN
constexpr uint64_t kEmpty = ~uint64_t(0);

__device__ __forceinline__ float join(float a, float b, float before) {
  return a == 0.f || before == 0.f ? b : fmaf(a, before, b);
}
__device__ __forceinline__ float join_factor(float a, float before) { return a == 0.f ? 0.f : a * before; }

// A published pair in one 64-bit word, written and read whole: no order between
// memory accesses is needed.  All ones mean that it is not there yet.
__device__ __forceinline__ void publish(uint64_t* at, float a, float b) {
  uint32_t lo = __float_as_uint(b);
  if (lo == 0xFFFFFFFFu) lo = 0x7FC00000u;   // one NaN for another
  __hip_atomic_store(at, uint64_t(__float_as_uint(a)) << 32 | lo, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* at) {
  return __hip_atomic_load(const_cast<uint64_t*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What the tiles share in the workspace.
struct TileSpace {
  uint32_t* ctrl;    // the counter, and the first row and the row behind the last one of any sequence
  uint2* marks;      // per 32 rows: which begin, and which end, a sequence
  int32_t* owner;    // of the marked rows: their sequence
  uint64_t* pairs;   // [tiles along the rows][C]
  uint64_t* kept;    // [groups][C]: the state before the group, as B
};

// Before the tiles: counter, marks, empty words, and the ends of sequences
// without rows (to = from, or 0).
__global__ __launch_bounds__(256) void tile_setup_kernel(Sequences seq, int S, int C, TileSpace ws, size_t words,
                                                         const float* from, float* to) {
  const int tid = blockIdx.x * 256 + threadIdx.x, all = gridDim.x * 256;
  if (tid == 0) {
    ws.ctrl[0] = 0;
    ws.ctrl[1] = seq.begin(0);
    ws.ctrl[2] = seq.end(S - 1);
  }
  for (size_t i = tid; i < words; i += all) ws.pairs[i] = kEmpty;   // kept lies behind pairs
  for (int k = tid; k < (seq.T + kBlock - 1) / kBlock; k += all) {
    const int t0 = k * kBlock;
    uint2 m = {0u, 0u};
    // the first sequence that ends behind t0 and those that begin or end in the block
    int lo = 0, hi = S;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (seq.end(mid) <= t0)
        lo = mid + 1;
      else
        hi = mid;
    }
    for (int s = lo; s < S; ++s) {
      const int b = seq.begin(s), e = seq.end(s);
      if (b >= t0 + kBlock) break;
      if (b >= e) continue;
      if (b >= t0) {
        m.x |= 1u << (b - t0);
        ws.owner[b] = s;
      }
      if (e > t0 && e <= t0 + kBlock) {
        m.y |= 1u << (e - 1 - t0);
        ws.owner[e - 1] = s;
      }
    }
    ws.marks[k] = m;
  }
  if (!to) return;
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    if (seq.begin(s) >= seq.end(s))
      for (int c = threadIdx.x; c < C; c += 256) to[size_t(s) * C + c] = from ? from[size_t(s) * C + c] : 0.f;
}

// The state before tile number k (in the order of the recurrence): what the
// words of two channels from `at` on fold to.
__device__ __forceinline__ void fold_before(const TileSpace& ws, int k, int C, int c, bool live, bool both, float* v0,
                                            float* v1) {
  const int group = k / kGroup, first = group * kGroup, n = k - first;
  uint64_t kept0 = 0, kept1 = 0, w0[kGroup], w1[kGroup];
  *v0 = *v1 = 0.f;
  if (k == 0) return;
  const uint64_t* pk = ws.kept + size_t(group) * C + c;
  const uint64_t* pw = ws.pairs + size_t(first) * C + c;
  bool ready = false;
  for (int spin = 0; spin < kSpin; ++spin) {
    ready = true;
    if (live) {
      if (group > 0) {
        kept0 = peek(pk);
        kept1 = both ? peek(pk + 1) : 0;
      }
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (j < n) {
          w0[j] = peek(pw + size_t(j) * C);
          w1[j] = both ? peek(pw + size_t(j) * C + 1) : 0;
        }
      ready = kept0 != kEmpty && kept1 != kEmpty;
#pragma unroll
      for (int j = 0; j < kGroup - 1; ++j)
        if (j < n) ready = ready && w0[j] != kEmpty && w1[j] != kEmpty;
    }
    if (__all(ready)) break;
    __builtin_amdgcn_s_sleep(1);
  }
  if (!live) return;
  if (!ready) {
    *v0 = *v1 = __uint_as_float(0x7FC00000u);
    return;
  }
  *v0 = __uint_as_float(uint32_t(kept0));
  *v1 = __uint_as_float(uint32_t(kept1));
#pragma unroll
  for (int j = 0; j < kGroup - 1; ++j)
    if (j < n) {
      *v0 = join(__uint_as_float(uint32_t(w0[j] >> 32)), __uint_as_float(uint32_t(w0[j])), *v0);
      *v1 = join(__uint_as_float(uint32_t(w1[j] >> 32)), __uint_as_float(uint32_t(w1[j])), *v1);
    }
}

// The waves' pairs, in the order of the recurrence, to the state before each
// of them: wave 0 of the workgroup publishes the tile's pair, waits for the
// state before the tile, and publishes the state behind it where a group ends.
template <int W>
__device__ __forceinline__ void waves_before(const TileSpace& ws, const float4 (&pairs)[W][64], float2 (&before)[W][64],
                                             int k, int tiles, int C, int c, bool live, bool both, int lane) {
  float a0 = 1.f, a1 = 1.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float4 p = pairs[w][lane];
    b0 = join(p.x, p.y, b0);
    a0 = join_factor(p.x, a0);
    b1 = join(p.z, p.w, b1);
    a1 = join_factor(p.z, a1);
  }
  if (live) {
    uint64_t* at = ws.pairs + size_t(k) * C + c;
    publish(at, a0, b0);
    if (both) publish(at + 1, a1, b1);
  }
  float v0, v1;
  fold_before(ws, k, C, c, live, both, &v0, &v1);
  if (k % kGroup == kGroup - 1 && k + 1 < tiles && live) {
    uint64_t* at = ws.kept + size_t(k / kGroup + 1) * C + c;
    publish(at, 0.f, join(a0, b0, v0));
    if (both) publish(at + 1, 0.f, join(a1, b1, v1));
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    before[w][lane] = make_float2(v0, v1);
    const float4 p = pairs[w][lane];
    v0 = join(p.x, p.y, v0);
    v1 = join(p.z, p.w, v1);
  }
}

// The tile that this workgroup takes next: its number along the rows, and its
// first channel.
__device__ __forceinline__ void take_tile(const TileSpace& ws, int blocks, int* k, int* c0) {
  __shared__ uint32_t ticket;
  if (threadIdx.x == 0)
    ticket = __hip_atomic_fetch_add(ws.ctrl, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const uint32_t t = __builtin_amdgcn_readfirstlane(ticket);
  *k = int(t / blocks);
  *c0 = int(t % blocks) * 128;
}

template <typename T, bool SIGMOID, int W>
__global__ __launch_bounds__(64 * W) void tile_kernel(TileSpace ws, int tiles, int C, const T* __restrict__ x,
                                                      const void* __restrict__ gate, const float* h0, T* __restrict__ h,
                                                      float* last, float* __restrict__ states) {
  __shared__ float4 pairs[W][64];
  __shared__ float2 before[W][64];
  int k, c0;
  take_tile(ws, (C + 127) / 128, &k, &c0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = c0 + 2 * lane, block = k * W + wave, t0 = block * kBlock;
  const bool live = c < C, both = c + 1 < C;
  const int lo = max(int(ws.ctrl[1]) - t0, 0), hi = min(int(ws.ctrl[2]) - t0, kBlock);   // this wave's rows
  const T* gates = static_cast<const T*>(gate);
  Pair<T> px[kBlock], pg[kBlock];
  uint2 marks = {0u, 0u};
  float a0 = 0.f, a1 = 0.f, A0 = 1.f, A1 = 1.f, s0 = 0.f, s1 = 0.f;
  if (hi > lo) {
    marks = ws.marks[block];
    if (live) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (i >= lo && i < hi) {
          const size_t at = size_t(t0 + i) * C + c;
          px[i].load(x + at, both);
          if (SIGMOID) pg[i].load(gates + at, both);
        }
      if (!SIGMOID) {
        a0 = static_cast<const float*>(gate)[c];
        a1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
      }
    }
  }
  // one row: the state behind it from the one before it
  auto step = [&](int i) {
    float b0 = px[i].get(0), b1 = px[i].get(1);
    if (SIGMOID) {
      float r0, r1;
      gate_of<T>(pg[i].get(0), &a0, &r0);
      gate_of<T>(pg[i].get(1), &a1, &r1);
      b0 *= r0;
      b1 *= r1;
    }
    if (marks.x >> i & 1) {
      const float* p = h0 ? h0 + size_t(ws.owner[t0 + i]) * C + c : nullptr;
      s0 = p ? p[0] : 0.f;
      s1 = p && both ? p[1] : 0.f;
      A0 = A1 = 0.f;
    }
    s0 = fmaf(a0, s0, b0);
    s1 = fmaf(a1, s1, b1);
    A0 = join_factor(A0, a0);
    A1 = join_factor(A1, a1);
  };
  if (live) {
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
      if (i >= lo && i < hi) step(i);
  }
  pairs[wave][lane] = make_float4(A0, s0, A1, s1);
  __syncthreads();
  if (wave == 0) waves_before<W>(ws, pairs, before, k, tiles, C, c, live, both, lane);
  __syncthreads();
  if (!live || hi <= lo) return;
  s0 = before[wave][lane].x;
  s1 = before[wave][lane].y;
  if (states) store2(states + size_t(block) * C + c, s0, s1, both);
#pragma unroll
  for (int i = 0; i < kBlock; ++i)
    if (i >= lo && i < hi) {
      step(i);
      store2(h + size_t(t0 + i) * C + c, s0, s1, both);
      if (last && (marks.y >> i & 1)) store2(last + size_t(ws.owner[t0 + i]) * C + c, s0, s1, both);
    }
}

// Backwards: tiles, waves and rows in the other order; what passes from row to
// row is e = a d.
template <typename T, bool SIGMOID, int W>
__global__ __launch_bounds__(64 * W) void tile_backward_kernel(
    TileSpace ws, int tiles, int C, const T* __restrict__ dh, const T* __restrict__ x, const void* __restrict__ gate,
    const float* __restrict__ h0, const float* dlast, const float* __restrict__ states, T* __restrict__ dx,
    T* __restrict__ dg, float* dh0, float* __restrict__ part) {
  __shared__ float4 pairs[W][64];
  __shared__ float2 before[W][64];
  int k, c0;
  take_tile(ws, (C + 127) / 128, &k, &c0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = c0 + 2 * lane, block = (tiles - 1 - k) * W + W - 1 - wave, t0 = block * kBlock;
  const bool live = c < C, both = c + 1 < C;
  const int lo = max(int(ws.ctrl[1]) - t0, 0), hi = min(int(ws.ctrl[2]) - t0, kBlock);   // this wave's rows
  const T* gates = static_cast<const T*>(gate);
  Pair<T> px[kBlock], pg[kBlock], pd[kBlock];
  float h_0[kBlock], h_1[kBlock];   // the state before each row
  uint2 marks = {0u, 0u};
  float a0 = 0.f, a1 = 0.f, r0 = 0.f, r1 = 0.f, A0 = 1.f, A1 = 1.f, e0 = 0.f, e1 = 0.f, d0 = 0.f, d1 = 0.f;
  auto gates_of = [&](int i) {
    if (SIGMOID) {
      gate_of<T>(pg[i].get(0), &a0, &r0);
      gate_of<T>(pg[i].get(1), &a1, &r1);
    }
  };
  if (hi > lo) {
    marks = ws.marks[block];
    if (live) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (i >= lo && i < hi) {
          const size_t at = size_t(t0 + i) * C + c;
          px[i].load(x + at, both);
          if (SIGMOID) pg[i].load(gates + at, both);
          pd[i].load(dh + at, both);
        }
      if (!SIGMOID) {
        a0 = static_cast<const float*>(gate)[c];
        a1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
      }
      float s0 = states[size_t(block) * C + c], s1 = both ? states[size_t(block) * C + c + 1] : 0.f;
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (i >= lo && i < hi) {
          if (marks.x >> i & 1) {
            const float* p = h0 ? h0 + size_t(ws.owner[t0 + i]) * C + c : nullptr;
            s0 = p ? p[0] : 0.f;
            s1 = p && both ? p[1] : 0.f;
          }
          h_0[i] = s0;
          h_1[i] = s1;
          gates_of(i);
          s0 = fmaf(a0, s0, SIGMOID ? r0 * px[i].get(0) : px[i].get(0));
          s1 = fmaf(a1, s1, SIGMOID ? r1 * px[i].get(1) : px[i].get(1));
        }
    }
  }
  auto step = [&](int i) {
    if (marks.y >> i & 1) {
      const float* p = dlast ? dlast + size_t(ws.owner[t0 + i]) * C + c : nullptr;
      e0 = p ? p[0] : 0.f;
      e1 = p && both ? p[1] : 0.f;
      A0 = A1 = 0.f;
    }
    gates_of(i);
    d0 = pd[i].get(0) + e0;
    d1 = pd[i].get(1) + e1;
    e0 = a0 * d0;
    e1 = a1 * d1;
    A0 = join_factor(A0, a0);
    A1 = join_factor(A1, a1);
  };
  if (live) {
#pragma unroll
    for (int i = kBlock - 1; i >= 0; --i)
      if (i >= lo && i < hi) step(i);
  }
  pairs[wave][lane] = make_float4(A0, e0, A1, e1);
  __syncthreads();
  if (wave == 0) waves_before<W>(ws, pairs, before, k, tiles, C, c, live, both, lane);
  __syncthreads();
  e0 = before[wave][lane].x;
  e1 = before[wave][lane].y;
  float sum0 = 0.f, sum1 = 0.f;
  if (live) {
#pragma unroll
    for (int i = kBlock - 1; i >= 0; --i)
      if (i >= lo && i < hi) {
        step(i);
        const size_t at = size_t(t0 + i) * C + c;
        if (SIGMOID) {
          if (dx) store2(dx + at, d0 * r0, d1 * r1, both);
          if (dg) store2(dg + at, d0 * r0 * (a0 * (h_0[i] - px[i].get(0))), d1 * r1 * (a1 * (h_1[i] - px[i].get(1))), both);
        } else {
          if (dx) store2(dx + at, d0, d1, both);
          sum0 = fmaf(d0, h_0[i], sum0);
          sum1 = fmaf(d1, h_1[i], sum1);
        }
        if (dh0 && (marks.x >> i & 1)) store2(dh0 + size_t(ws.owner[t0 + i]) * C + c, e0, e1, both);
      }
  }
  if (SIGMOID || !part) return;
  before[wave][lane] = make_float2(sum0, sum1);   // each lane overwrites what it alone has read
  __syncthreads();
  if (wave == 0 && live) {
#pragma unroll
    for (int w = 1; w < W; ++w) {
      sum0 += before[w][lane].x;
      sum1 += before[w][lane].y;
    }
    store2(part + size_t(k) * C + c, sum0, sum1, both);
  }
}

// Waves of a tile: eight, or (backwards, where a wave holds three rows' worth
// of registers) four, so that two workgroups share a compute unit.
constexpr int kWaves = 8, kWavesBackward = 4;

// Whether the rows are split into tiles.
bool tiled(int T, int S) { return T >= 128 * long(S); }

// Offsets of TileSpace's parts, and of dgate's shares behind them.
struct TileLayout {
  int tiles;
  size_t marks, owner, pairs, kept, part, total, words;
};
TileLayout tile_layout(int T, int C, int waves, bool shares) {
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  TileLayout l;
  l.tiles = (T + kBlock * waves - 1) / (kBlock * waves);
  const size_t row = size_t(C) * 8, groups = size_t((l.tiles + kGroup - 1) / kGroup);
  l.marks = 256;
  l.owner = l.marks + up(size_t((T + kBlock - 1) / kBlock) * 8);
  l.pairs = l.owner + up(size_t(T) * 4);
  l.kept = l.pairs + l.tiles * row;
  l.words = (l.tiles + groups) * size_t(C);
  l.part = up(l.kept + groups * row);
  l.total = l.part + (shares ? up(size_t(l.tiles) * C * 4) : 0);
  return l;
}
TileSpace tile_space(void* ws, const TileLayout& l) {
  unsigned char* p = static_cast<unsigned char*>(ws);
  return {reinterpret_cast<uint32_t*>(p), reinterpret_cast<uint2*>(p + l.marks), reinterpret_cast<int32_t*>(p + l.owner),
          reinterpret_cast<uint64_t*>(p + l.pairs), reinterpret_cast<uint64_t*>(p + l.kept)};
}
hipError_t tile_setup(const Sequences& seq, int S, int C, const TileSpace& ws, const TileLayout& l, const float* from,
                      float* to, hipStream_t stream) {
  const size_t blocks = (l.words + 1023) / 1024;
  hipLaunchKernelGGL(tile_setup_kernel, dim3(unsigned(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, seq, S, C,
                     ws, l.words, from, to);
  return hipGetLastError();
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
  if (tiled(a.T, a.S)) {
    const TileLayout l = tile_layout(a.T, a.C, kWaves, false);
    const TileSpace ws = tile_space(a.ws, l);
    const hipError_t e = tile_setup(sequences(a), a.S, a.C, ws, l, a.h0, a.last, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((tile_kernel<T, SIGMOID, kWaves>), dim3(unsigned(l.tiles) * ((a.C + 127) / 128)),
                       dim3(64 * kWaves), 0, stream, ws, l.tiles, a.C, static_cast<const T*>(a.x), a.gate, a.h0,
                       static_cast<T*>(a.h), a.last, a.states);
    return hipGetLastError();
  }
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
  int units = a.S > 0 ? 4 * g : 0;
  hipError_t e = hipSuccess;
  if (a.S > 0 && tiled(a.T, a.S)) {
    const TileLayout l = tile_layout(a.T, a.C, kWavesBackward, !SIGMOID);
    const TileSpace ws = tile_space(a.ws, l);
    if (part) part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + l.part);
    units = l.tiles;
    e = tile_setup(sequences(a), a.S, a.C, ws, l, a.dlast, a.dh0, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((tile_backward_kernel<T, SIGMOID, kWavesBackward>),
                       dim3(unsigned(l.tiles) * ((a.C + 127) / 128)), dim3(64 * kWavesBackward), 0, stream, ws, l.tiles,
                       a.C, static_cast<const T*>(a.dh), static_cast<const T*>(a.x), a.gate, a.h0, a.dlast,
                       a.states_in, static_cast<T*>(a.dx), SIGMOID ? static_cast<T*>(a.dgate) : nullptr, a.dh0, part);
    e = hipGetLastError();
  } else if (a.S > 0) {
    hipLaunchKernelGGL((rows_backward_kernel<T, SIGMOID>), dim3((a.C + 127) / 128, g), dim3(256), 0, stream,
                       sequences(a), a.S, a.C, static_cast<const T*>(a.dh), static_cast<const T*>(a.x), a.gate, a.h0,
                       a.dlast, a.states_in, static_cast<T*>(a.dx), SIGMOID ? static_cast<T*>(a.dgate) : nullptr,
                       a.dh0, part);
    e = hipGetLastError();
  }
  if (SIGMOID || !a.dgate || e != hipSuccess) return e;
  hipLaunchKernelGGL(gate_join_kernel, dim3((a.C + 31) / 32), dim3(256), 0, stream, a.C, units, part,
                     static_cast<float*>(a.dgate));
  return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) {
  return tiled(T, S) ? tile_layout(T, C, kWaves, false).total : 0;
}
size_t recurrence_backward_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) {
  if (tiled(T, S)) return tile_layout(T, C, kWavesBackward, !sigmoid).total;
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
