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
// by block of 16 rows, from the fp32 states that the forward pass kept.
//
// Bound by memory, and with long sequences by the words that tiles pass on:
// 65536 rows of 2560 take 268 us forward for 1.0 GB, 438 backward for 1.7 GB, in
// training 717 together with their setup (the same loads and stores without the
// words: 212 and 358, with cheaper gates); a step of 256 sequences 3.9 us.
#include "launch.h"
#include "projection.h"

namespace dspark {

namespace {

constexpr int kBlock = 16;   // rows from one kept state to the next

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
// past: by the caches, which need not keep it: so tiles write h and the gradients
// (forward, and in training with what reads them next, us with and without, bf16: 65536 x
// 2560 283 against 298 and 1110 against 1143, 16384 x 512 42 and 43, 145 and 144,
// 1024 x 1024 14.3 and 14.4, 42 and 42; fp32: 65536 x 1600 273 and 292, 1244 and
// 1297, 1024 x 1024 16.5 and 17.3, 48 and 52).
template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b, bool both, bool past = false) {
  if (both && past) {
    typedef uint32_t pair_t __attribute__((ext_vector_type(sizeof(T) / 2), aligned(sizeof(T))));
    T v[2] = {from_f32<T>(a), from_f32<T>(b)};
    pair_t w;
    __builtin_memcpy(&w, v, 2 * sizeof(T));
    __builtin_nontemporal_store(w, reinterpret_cast<pair_t*>(p));
  } else if (both) {
    T v[2] = {from_f32<T>(a), from_f32<T>(b)};
    __builtin_memcpy(p, v, 2 * sizeof(T));
  } else {
    *p = from_f32<T>(a);
  }
}

// a = 1 / (1 + exp(-g)) and 1 - a = exp(-g) a, each to its own relative accuracy:
// nothing cancels for gates near 1.  From g = -87 on, where a falls below 2^-125,
// it is 0 and 1 - a is 1; minimum() passes NaN on.  For bf16 logits the
// exponential is the hardware's of base 2, with log2(e) = HI + the rest: g HI is
// exact, as HI has 16 bits, and the rest enters as exp(-g REST) to first order
// (off by 2^-23 at |g| = 87); the reciprocal is the hardware's, off by one unit in
// the last place.  (Without that product and the 0 for far logits 65536 rows of
// 2560 in training take 709 us instead of 725, and 1 - a is off by |g| 2^-24.)
template <typename T>
__device__ __forceinline__ void gate_of(float g, float* a, float* rest) {
  const float m = __builtin_elementwise_minimum(-g, 87.f);
  float e, r;
  if constexpr (sizeof(T) == 4) {
    e = expf(m);
    r = 1.f / (1.f + e);
  } else {
    constexpr float HI = 1.44268798828125f, REST = 4.888495152e-06f;   // REST = 1 - HI ln 2
    e = __builtin_amdgcn_exp2f(m * HI);
    e = fmaf(e, __builtin_elementwise_maximum(m, -200.f) * REST, e);   // (not 0 times infinity)
    r = __builtin_amdgcn_rcpf(1.f + e);
  }
  *a = m >= 87.f ? 0.f : r;
  *rest = e * r;
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
// A tile is W waves of 16 rows by 128 channels, read once and kept in
// registers.  What rows do to the state before them is h -> A h + B; a wave
// makes its (A, B), LDS joins the waves', and the tile's pair is published.
// Every kSub-th tile publishes the pair of the last kSub, and every kGroup-th
// the state behind it; a tile folds, in order, the last such state, the pairs
// of kSub tiles since then and the single ones since then: 15 words at most,
// and the tiles wait for one another in a row once in kGroup only.  The order
// of all sums is fixed: results do not depend on which tile comes first.
//
// A tile takes its number along the rows from a counter of its channels, so
// that every tile it waits for belongs to a workgroup that is already running
// and itself waits for lower numbers only.  (One counter for all channels
// hands out a number every 56 ns: 10240 tiles then took 577 us.)
//
// Where a sequence begins, A is NaN, which all products keep, and B holds what
// its h0 gives: join() then ignores the state before, whatever it is.  (A gate
// that is NaN makes B NaN as well.)  A product of gates that has become 0 (300
// rows of ordinary gates are enough) is published as the smallest value that is
// not, so that an infinity or NaN before it goes on to the sequence's end, as it
// does row after row.  To a finite state that adds 2^-149 of itself, less than
// 2^-21.
constexpr int kSub = 8, kGroup = 64;
constexpr int kSpin = 1 << 22;   // polls of a few hundred nanoseconds; a state not seen by then is NaN
constexpr uint64_t kEmpty = ~uint64_t(0);
constexpr int kLine = 32;   // 32-bit words

constexpr float kBegins = __builtin_nanf("");   // A where a sequence begins
__device__ __forceinline__ float join(float a, float b, float before) {
  return a != a || before == 0.f ? b : fmaf(a, before, b);
}
// A of rows with the product a of gates and marks.
__device__ __forceinline__ float factor(float a) { return a == 0.f ? copysignf(__uint_as_float(1u), a) : a; }

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
  uint32_t* ctrl;    // the first row of any sequence, and the row behind the last one
  uint32_t* tickets; // a counter per 128 channels, each in a line of its own
  uint32_t* marks;   // per 16 rows: which begin (low half), and which end (high half), a sequence
  int32_t* owner;    // of the marked rows: their sequence
  uint64_t* pairs;   // [tiles along the rows][C]
  uint64_t* subs;    // [kSub tiles][C]
  uint64_t* kept;    // [kGroup tiles][C]: the state before the group, as B
};

// Before the tiles: counter, marks, empty words, and the ends of sequences
// without rows (to = from, or 0).
__global__ __launch_bounds__(256) void tile_setup_kernel(Sequences seq, int S, int C, TileSpace ws, size_t words,
                                                         const float* from, float* to) {
  const int tid = blockIdx.x * 256 + threadIdx.x, all = gridDim.x * 256;
  if (tid == 0) {
    ws.ctrl[0] = seq.begin(0);
    ws.ctrl[1] = seq.end(S - 1);
  }
  for (int i = tid; i < (C + 127) / 128; i += all) ws.tickets[i * kLine] = 0;
  for (size_t i = tid; i < words; i += all) ws.pairs[i] = kEmpty;   // subs and kept lie behind pairs
  for (int k = tid; k < (seq.T + kBlock - 1) / kBlock; k += all) {
    const int t0 = k * kBlock;
    uint32_t m = 0u;
    // the first sequence that ends behind t0, and those from it on that begin or end in the block
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
        m |= 1u << (b - t0);
        ws.owner[b] = s;
      }
      if (e > t0 && e <= t0 + kBlock) {
        m |= 0x10000u << (e - 1 - t0);
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

// One lane's two channels of a word in LDS: (A, B) of both.
__device__ __forceinline__ float4 wide(uint64_t w0, uint64_t w1) {
  return make_float4(__uint_as_float(uint32_t(w0 >> 32)), __uint_as_float(uint32_t(w0)),
                     __uint_as_float(uint32_t(w1 >> 32)), __uint_as_float(uint32_t(w1)));
}
struct State2 {
  float v0, v1;
  __device__ __forceinline__ void behind(const float4& p) {
    v0 = join(p.x, p.y, v0);
    v1 = join(p.z, p.w, v1);
  }
};
struct Pair2 {
  float a0 = 1.f, b0 = 0.f, a1 = 1.f, b1 = 0.f;
  __device__ __forceinline__ void behind(const float4& p) {
    b0 = join(p.x, p.y, b0);
    a0 *= p.x;
    b1 = join(p.z, p.w, b1);
    a1 *= p.z;
  }
  __device__ __forceinline__ void to(uint64_t* at, bool both) const {
    publish(at, factor(a0), b0);
    if (both) publish(at + 1, factor(a1), b1);
  }
};

// A tile's shared memory: its waves' pairs, and the words of the tiles before.
template <int W>
struct TileLds {
  float4 pairs[W][64];
  float4 words[2 * kSub - 1][64];   // of kSub tiles each, of single tiles, and the kept state
};

// The state before this wave's rows.  k: the tile's number, waves and tiles
// counted in the order of the recurrence; the waves' pairs are in lds.
template <int W>
__device__ __forceinline__ State2 state_before(TileLds<W>& lds, const TileSpace& ws, int k, int tiles, int C, int c,
                                               bool live, bool both, int wave, int lane) {
  __syncthreads();
  const int singles = k % kSub, subs = k % kGroup / kSub, group = k / kGroup;
  if (wave == 0 && live) {
    Pair2 p;
#pragma unroll
    for (int w = 0; w < W; ++w) p.behind(lds.pairs[w][lane]);
    p.to(ws.pairs + size_t(k) * C + c, both);
  }
  // the waves share the words between them
  constexpr int N = 2 * kSub - 1, per = (N + W - 1) / W;
  const uint64_t* at[per];   // row of words, or null
  uint64_t w0[per], w1[per];
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int j = wave + i * W;
    at[i] = nullptr;
    if (j < kSub - 1) {
      if (j < subs) at[i] = ws.subs + size_t(group * (kGroup / kSub) + j) * C;
    } else if (j < N - 1) {
      if (j - (kSub - 1) < singles) at[i] = ws.pairs + size_t(k - singles + j - (kSub - 1)) * C;
    } else if (j == N - 1) {
      if (group > 0) at[i] = ws.kept + size_t(group) * C;
    }
  }
  bool ready = false;
  for (int spin = 0; spin < kSpin; ++spin) {
    // all lanes look at one word: a thousand waves that read all of theirs over
    // and over would take the memory's whole bandwidth
    bool some = true;
#pragma unroll
    for (int i = 0; i < per; ++i)
      if (at[i]) some = some && peek(at[i] + (c - 2 * lane)) != kEmpty;
    if (__all(some)) {
      ready = true;
      if (live) {
#pragma unroll
        for (int i = 0; i < per; ++i)
          if (at[i]) {
            w0[i] = peek(at[i] + c);
            w1[i] = both ? peek(at[i] + c + 1) : 0;
          }
#pragma unroll
        for (int i = 0; i < per; ++i)
          if (at[i]) ready = ready && w0[i] != kEmpty && w1[i] != kEmpty;
      }
      if (__all(ready)) break;
    }
    __builtin_amdgcn_s_sleep(2);
  }
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int j = wave + i * W;
    // what never came is NaN
    if (at[i]) lds.words[j][lane] = ready ? wide(w0[i], w1[i]) : wide(0x7FC000007FC00000ull, 0x7FC000007FC00000ull);
  }
  __syncthreads();
  if (wave == 0 && live && singles == kSub - 1) {
    Pair2 p;
    for (int j = 0; j < kSub - 1; ++j) p.behind(lds.words[kSub - 1 + j][lane]);
#pragma unroll
    for (int w = 0; w < W; ++w) p.behind(lds.pairs[w][lane]);
    p.to(ws.subs + size_t(k / kSub) * C + c, both);
  }
  State2 v = {0.f, 0.f};
  if (group > 0) {
    const float4 p = lds.words[N - 1][lane];
    v = {p.y, p.w};
  }
  for (int j = 0; j < subs; ++j) v.behind(lds.words[j][lane]);
  for (int j = 0; j < singles; ++j) v.behind(lds.words[kSub - 1 + j][lane]);
  for (int w = 0; w < wave; ++w) v.behind(lds.pairs[w][lane]);
  if (wave == W - 1 && live && k % kGroup == kGroup - 1 && k + 1 < tiles) {
    State2 end = v;
    end.behind(lds.pairs[W - 1][lane]);
    uint64_t* to = ws.kept + size_t(group + 1) * C + c;
    publish(to, 0.f, end.v0);
    if (both) publish(to + 1, 0.f, end.v1);
  }
  return v;
}

// The tile that this workgroup takes: its number along the rows, and its first channel.
__device__ __forceinline__ void take_tile(const TileSpace& ws, int C, int* k, int* c0) {
  __shared__ uint32_t ticket;
  const int block = blockIdx.x % ((C + 127) / 128);
  if (threadIdx.x == 0)
    ticket = __hip_atomic_fetch_add(ws.tickets + block * kLine, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  *k = int(__builtin_amdgcn_readfirstlane(ticket));
  *c0 = block * 128;
}

// A wave's rows of a tile: those from lo to hi - 1 of 16 belong to a sequence.
struct Rows {
  int block, t0, lo, hi;
  uint32_t marks;
  bool whole;   // all 16, none of them the first or last of a sequence
  __device__ __forceinline__ void init(const TileSpace& ws, int b) {
    block = b;
    t0 = b * kBlock;
    lo = __builtin_amdgcn_readfirstlane(max(int(ws.ctrl[0]) - t0, 0));
    hi = __builtin_amdgcn_readfirstlane(min(int(ws.ctrl[1]) - t0, kBlock));
    marks = hi > lo ? __builtin_amdgcn_readfirstlane(ws.marks[b]) : 0u;
    whole = lo == 0 && hi == kBlock && marks == 0u;
  }
  __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
  __device__ __forceinline__ bool begins(int i) const { return marks >> i & 1; }
  __device__ __forceinline__ bool ends(int i) const { return marks >> (16 + i) & 1; }
};

// Two values by sequence (of the marked row i): v[owner][c] and its neighbour, or 0.
__device__ __forceinline__ State2 of_sequence(const float* v, const TileSpace& ws, const Rows& r, int i, int C, int c,
                                              bool both) {
  if (!v) return {0.f, 0.f};
  const float* p = v + size_t(ws.owner[r.t0 + i]) * C + c;
  return {p[0], both ? p[1] : 0.f};
}

template <typename T, bool SIGMOID, int W>
__global__ __launch_bounds__(64 * W, 4) void tile_kernel(TileSpace ws, int tiles, int C, const T* __restrict__ x,
                                                      const void* __restrict__ gate, const float* h0, T* __restrict__ h,
                                                      float* last, float* __restrict__ states) {
  __shared__ TileLds<W> lds;
  int k, c0;
  take_tile(ws, C, &k, &c0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = c0 + 2 * lane;
  const bool live = c < C, both = c + 1 < C;
  Rows r;
  r.init(ws, k * W + wave);
  const T* gates = static_cast<const T*>(gate);
  float decay0 = 0.f, decay1 = 0.f;
  if (!SIGMOID && live) {
    decay0 = static_cast<const float*>(gate)[c];
    decay1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
  }
  // a row: state -> a state + b; one that is not there changes nothing, and the
  // first of a sequence (a marked, b from its h0) forgets what was before
  float a0[kBlock], a1[kBlock], b0[kBlock], b1[kBlock];
  Pair2 p;
  if (live) {
    Pair<T> px[kBlock], pg[kBlock];
    auto load = [&](int i) {
      const size_t at = size_t(r.t0 + i) * C + c;
      px[i].load(x + at, both);
      if (SIGMOID) pg[i].load(gates + at, both);
    };
    auto make = [&](int i) {
      b0[i] = px[i].get(0);
      b1[i] = px[i].get(1);
      a0[i] = decay0;
      a1[i] = decay1;
      if (SIGMOID) {
        float r0, r1;
        gate_of<T>(pg[i].get(0), &a0[i], &r0);
        gate_of<T>(pg[i].get(1), &a1[i], &r1);
        b0[i] *= r0;
        b1[i] *= r1;
      }
    };
    if (r.whole) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i) load(i);
#pragma unroll
      for (int i = 0; i < kBlock; ++i) {
        make(i);
        p.b0 = fmaf(a0[i], p.b0, b0[i]);
        p.b1 = fmaf(a1[i], p.b1, b1[i]);
        p.a0 *= a0[i];
        p.a1 *= a1[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (r.has(i)) load(i);
#pragma unroll
      for (int i = 0; i < kBlock; ++i) {
        a0[i] = a1[i] = 1.f;
        b0[i] = b1[i] = 0.f;
        if (r.has(i)) {
          make(i);
          if (r.begins(i)) {
            const State2 v = of_sequence(h0, ws, r, i, C, c, both);
            b0[i] = fmaf(a0[i], v.v0, b0[i]);
            b1[i] = fmaf(a1[i], v.v1, b1[i]);
            a0[i] = a1[i] = kBegins;
          }
        }
        p.behind(make_float4(a0[i], b0[i], a1[i], b1[i]));
      }
    }
    p.a0 = factor(p.a0);
    p.a1 = factor(p.a1);
  }
  lds.pairs[wave][lane] = make_float4(p.a0, p.b0, p.a1, p.b1);
  State2 v = state_before<W>(lds, ws, k, tiles, C, c, live, both, wave, lane);
  if (!live || r.hi <= r.lo) return;
  if (states) store2(states + size_t(r.block) * C + c, v.v0, v.v1, both);
  T* out = h + size_t(r.t0) * C + c;
  if (r.whole) {
#pragma unroll
    for (int i = 0; i < kBlock; ++i) {
      v.v0 = fmaf(a0[i], v.v0, b0[i]);
      v.v1 = fmaf(a1[i], v.v1, b1[i]);
      store2(out + size_t(i) * C, v.v0, v.v1, both, true);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
      if (r.has(i)) {
        v.behind(make_float4(a0[i], b0[i], a1[i], b1[i]));
        store2(out + size_t(i) * C, v.v0, v.v1, both, true);
        if (last && r.ends(i)) store2(last + size_t(ws.owner[r.t0 + i]) * C + c, v.v0, v.v1, both);
      }
  }
}

// Backwards: tiles, waves and rows in the other order; what passes from row to
// row is e = a d, e -> a (dh + e).  dlast is read before the pair is published
// and not again: behind that, the wave of the sequence's first row may have
// written dh0, which may be dlast itself.  LDS keeps it (65536 rows of 2560 in
// training 702 us; in registers 745, which leave two workgroups of bf16 to a
// compute unit instead of three).
template <typename T, bool SIGMOID, int W>
__global__ __launch_bounds__(64 * W) void tile_backward_kernel(
    TileSpace ws, int tiles, int C, const T* __restrict__ dh, const T* __restrict__ x, const void* __restrict__ gate,
    const float* __restrict__ h0, const float* dlast, const float* __restrict__ states, T* __restrict__ dx,
    T* __restrict__ dg, float* dh0, float* __restrict__ part) {
  __shared__ TileLds<W> lds;
  __shared__ float2 ends[W][kBlock][64];   // dlast where a sequence ends
  int k, c0;
  take_tile(ws, C, &k, &c0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = c0 + 2 * lane;
  const bool live = c < C, both = c + 1 < C;
  Rows r;
  r.init(ws, (tiles - 1 - k) * W + W - 1 - wave);
  const T* gates = static_cast<const T*>(gate);
  float decay0 = 0.f, decay1 = 0.f;
  if (!SIGMOID && live) {
    decay0 = static_cast<const float*>(gate)[c];
    decay1 = both ? static_cast<const float*>(gate)[c + 1] : 0.f;
  }
  // a row's gate, what dx is of d (1 - a) and what dgate is of it (SIGMOID:
  // a (1 - a) (h before - x), DECAY: h before)
  float a0[kBlock], a1[kBlock], r0[kBlock], r1[kBlock], w0[kBlock], w1[kBlock];
  Pair<T> pd[kBlock];
  Pair2 p;
  auto gate0 = [&](int i) { return SIGMOID ? a0[i] : decay0; };
  auto gate1 = [&](int i) { return SIGMOID ? a1[i] : decay1; };
  if (live && r.hi > r.lo) {
    Pair<T> px[kBlock], pg[kBlock];
    auto load = [&](int i) {
      const size_t at = size_t(r.t0 + i) * C + c;
      px[i].load(x + at, both);
      if (SIGMOID) pg[i].load(gates + at, both);
      pd[i].load(dh + at, both);
    };
    const float* from = states + size_t(r.block) * C + c;
    State2 v = {from[0], both ? from[1] : 0.f};
    auto make = [&](int i) {   // v: the state before the row, then behind it
      const float x0 = px[i].get(0), x1 = px[i].get(1);
      if (SIGMOID) {
        gate_of<T>(pg[i].get(0), &a0[i], &r0[i]);
        gate_of<T>(pg[i].get(1), &a1[i], &r1[i]);
        w0[i] = a0[i] * (v.v0 - x0);
        w1[i] = a1[i] * (v.v1 - x1);
        v = {fmaf(a0[i], v.v0, r0[i] * x0), fmaf(a1[i], v.v1, r1[i] * x1)};
      } else {
        w0[i] = v.v0;
        w1[i] = v.v1;
        v = {fmaf(decay0, v.v0, x0), fmaf(decay1, v.v1, x1)};
      }
    };
    if (r.whole) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i) load(i);
#pragma unroll
      for (int i = 0; i < kBlock; ++i) make(i);
#pragma unroll
      for (int i = kBlock - 1; i >= 0; --i) {
        p.b0 = gate0(i) * (pd[i].get(0) + p.b0);
        p.b1 = gate1(i) * (pd[i].get(1) + p.b1);
        p.a0 *= gate0(i);
        p.a1 *= gate1(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (r.has(i)) load(i);
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (r.has(i)) {
          if (r.begins(i)) v = of_sequence(h0, ws, r, i, C, c, both);
          make(i);
        }
#pragma unroll
      for (int i = kBlock - 1; i >= 0; --i)
        if (r.has(i)) {
          if (r.ends(i)) {
            const State2 e = of_sequence(dlast, ws, r, i, C, c, both);
            ends[wave][i][lane] = make_float2(e.v0, e.v1);
            p.a0 = p.a1 = kBegins;
            p.b0 = e.v0;
            p.b1 = e.v1;
          }
          p.b0 = gate0(i) * (pd[i].get(0) + p.b0);
          p.b1 = gate1(i) * (pd[i].get(1) + p.b1);
          p.a0 *= gate0(i);
          p.a1 *= gate1(i);
        }
    }
    p.a0 = factor(p.a0);
    p.a1 = factor(p.a1);
  }
  lds.pairs[wave][lane] = make_float4(p.a0, p.b0, p.a1, p.b1);
  State2 e = state_before<W>(lds, ws, k, tiles, C, c, live, both, wave, lane);
  float sum0 = 0.f, sum1 = 0.f;
  if (live) {
    auto row = [&](int i) {
      const float d0 = pd[i].get(0) + e.v0, d1 = pd[i].get(1) + e.v1;
      const size_t at = size_t(r.t0 + i) * C + c;
      if (SIGMOID) {
        const float u0 = d0 * r0[i], u1 = d1 * r1[i];
        if (dx) store2(dx + at, u0, u1, both, true);
        if (dg) store2(dg + at, u0 * w0[i], u1 * w1[i], both, true);
      } else {
        if (dx) store2(dx + at, d0, d1, both, true);
        sum0 = fmaf(d0, w0[i], sum0);
        sum1 = fmaf(d1, w1[i], sum1);
      }
      e = {gate0(i) * d0, gate1(i) * d1};
    };
    if (r.whole) {
#pragma unroll
      for (int i = kBlock - 1; i >= 0; --i) row(i);
    } else {
#pragma unroll
      for (int i = kBlock - 1; i >= 0; --i)
        if (r.has(i)) {
          if (r.ends(i)) e = {ends[wave][i][lane].x, ends[wave][i][lane].y};
          row(i);
          if (dh0 && r.begins(i)) store2(dh0 + size_t(ws.owner[r.t0 + i]) * C + c, e.v0, e.v1, both);
        }
    }
  }
  if (SIGMOID || !part) return;
  __syncthreads();   // the waves' pairs have been read
  lds.pairs[wave][lane] = make_float4(sum0, sum1, 0.f, 0.f);
  __syncthreads();
  if (wave == 0 && live) {
#pragma unroll
    for (int w = 1; w < W; ++w) {
      sum0 += lds.pairs[w][lane].x;
      sum1 += lds.pairs[w][lane].y;
    }
    store2(part + size_t(k) * C + c, sum0, sum1, both);
  }
}

// Waves of a tile: eight, or (backwards, where a wave holds three rows' worth
// of registers) four, so that two workgroups share a compute unit, of bf16 three.
constexpr int kWaves = 8, kWavesBackward = 4;

// Whether the rows are split into tiles.  In training, us: a wave takes 4 + 0.5
// a row of the longest sequence (decay 0.3); tiles take 24, for three launches
// and words that go round, and 0.006 a row of all sequences, as they wait for
// one another (bf16, 256 channels: 1 sequence of 32 rows 20 against 26, of 64 38
// and 26; 16 of 64 39 and 33, of 512 278 and 71; 128 of 64 41 and 75, of 512 293
// and 398; with 2560 channels 16 of 512 296 and 106, 128 of 64 72 and 116).  Of
// sequences that differ the longest is taken to be three times the mean, or all
// rows of one or two (one of 20 rows 17 us against 25, of 32 22 and 25, of 48 25
// by tiles).  The host does not see the lengths: where one of hundreds of
// sequences has nearly all rows, it is gone through row by row all the same (511
// of 3 rows and one of 64000, 2560 channels: 38 ms, with 12 sequences 0.68).
bool tiled(int T, int S, bool packed) { return 250l * (packed ? S < 3 ? S : 3 : 1) * T >= S * (10000l + 3l * T); }

// Offsets of TileSpace's parts, and of dgate's shares behind them.
struct TileLayout {
  int tiles;
  size_t tickets, marks, owner, pairs, subs, kept, part, total, words;
};
TileLayout tile_layout(int T, int C, int waves, bool shares) {
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  TileLayout l;
  l.tiles = (T + kBlock * waves - 1) / (kBlock * waves);
  const size_t row = size_t(C) * 8, subs = size_t((l.tiles + kSub - 1) / kSub),
               groups = size_t((l.tiles + kGroup - 1) / kGroup);
  l.tickets = 256;
  l.marks = l.tickets + up(size_t((C + 127) / 128) * kLine * 4);
  l.owner = l.marks + up(size_t(l.tiles) * waves * 4);
  l.pairs = l.owner + up(size_t(T) * 4);
  l.subs = l.pairs + l.tiles * row;
  l.kept = l.subs + subs * row;
  l.words = (l.tiles + subs + groups) * size_t(C);
  l.part = up(l.kept + groups * row);
  l.total = l.part + (shares ? up(size_t(l.tiles) * C * 4) : 0);
  return l;
}
TileSpace tile_space(void* ws, const TileLayout& l) {
  unsigned char* p = static_cast<unsigned char*>(ws);
  return {reinterpret_cast<uint32_t*>(p),          reinterpret_cast<uint32_t*>(p + l.tickets),
          reinterpret_cast<uint32_t*>(p + l.marks), reinterpret_cast<int32_t*>(p + l.owner),
          reinterpret_cast<uint64_t*>(p + l.pairs), reinterpret_cast<uint64_t*>(p + l.subs),
          reinterpret_cast<uint64_t*>(p + l.kept)};
}
hipError_t tile_setup(const Sequences& seq, int S, int C, const TileSpace& ws, const TileLayout& l, const float* from,
                      float* to, hipStream_t stream) {
  const size_t fill = (l.words + 1023) / 1024, marks = (size_t(seq.T) / kBlock + 255) / 256;
  const size_t blocks = fill > marks ? fill : marks > 0 ? marks : 1;
  hipLaunchKernelGGL(tile_setup_kernel, dim3(unsigned(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, seq, S, C,
                     ws, l.words, from, to);
  return hipGetLastError();
}

Sequences sequences(const RecurrenceArgs& a) { return {a.offsets, a.T, a.S > 0 ? a.T / a.S : 0}; }

// Workgroups of four waves along the sequences; fewer where each wave leaves a
// share of dgate.
int groups(int S, bool shares) {
  const int g = (S + 3) / 4, most = shares ? 256 : 16384;
  return g < most ? g : most;
}

template <typename T, bool SIGMOID>
hipError_t forward_t(const RecurrenceArgs& a, hipStream_t stream) {
  if (a.S == 0) return hipSuccess;
  if (tiled(a.T, a.S, a.offsets != nullptr)) {
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
  const int g = groups(a.S, !SIGMOID);
  float* part = !SIGMOID && a.dgate ? static_cast<float*>(a.ws) : nullptr;
  int units = a.S > 0 ? 4 * g : 0;
  hipError_t e = hipSuccess;
  if (a.S > 0 && tiled(a.T, a.S, a.offsets != nullptr)) {
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

// (what packed sequences take is enough for those of equal length)
size_t recurrence_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) {
  return tiled(T, S, true) ? tile_layout(T, C, kWaves, false).total : 0;
}
size_t recurrence_backward_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid) {
  const size_t tiles = tiled(T, S, true) ? tile_layout(T, C, kWavesBackward, !sigmoid).total : 0;
  const size_t rows = sigmoid ? 0 : (size_t(groups(S, true)) * 4 * C * 4 + 255) & ~size_t(255);
  return tiles > rows ? tiles : rows;
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
