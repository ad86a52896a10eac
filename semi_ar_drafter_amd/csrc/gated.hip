// Gated feed-forward projection: y = act(x wg^T + bg) * (x wu^T + bu), and its
// gradients.
//
//   forward    C(a = feature of wg and of wu, b = row): one product whose a
//              operand is both matrices, 64 (or 32, 16) features of the one and
//              the same of the other in a wave's share of a tile, so that a lane
//              holds a feature's gate and value: the activation and the product
//              are the epilogue
//   dz         dzg = dy zu act'(zg),  dzu = dy act(zg), once, side by side:
//              [row][dzg, padded to 64 | dzu, padded to 64]
//   dx         C(a = input, b = row) = sum_n wg[n][a] dzg[b][n] + wu[n][a] dzu[b][n]:
//              one contraction of two parts
//   dwg, dwu   C(a = input, b = column of dz) = sum_m x[m][a] dz[m][b]: one product
// dz is rounded to the storage type, which the products take (see linear.hip):
// bf16 gradients are off by 2.35e-3 of their norm, where their own rounding alone
// is 1.66e-3; keeping the rounded-off part as a second operand would double both
// products (1.4 ms more of 2.3 at 4096 x 10240 x 5120).  The pre-activations that
// the gradient reads are fp32: rounded to bf16 they would add half a bf16 step of
// zu to every dzg.
//
// Bound by reading the weights with few rows (16384 x 4096, one row: 45.8 us, 5.9
// TB/s), by the main loop of the matrix unit's tiles with many (2048 rows: 428 to
// 476 us from card to card, 1.15 to 1.28 PFLOP/s; 4096 x 10240 x 5120 in training
// 2.29 to 2.33 ms, under the profiler: 709 us forward with its 420 MB of
// pre-activations and outputs, gradients 683 and 760 us, dz 112).
#include "launch.h"
#include "product.h"

namespace dspark {

namespace {

// As store4(); without alignment one store instead of four (weights' gradients of
// one row, 4480 x 4002: 141 us for the training pass before, 106 so).
template <typename T>
__device__ __forceinline__ void store4_any(T* p, f32x4_t v, int n, bool vec) {
  if (!vec && n >= 4) {
    const T e[4] = {from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])};
    __builtin_memcpy(p, e, sizeof e);
  } else {
    store4(p, v, n, vec);
  }
}

template <typename T>
struct GatedEpi {
  const T *bg, *bu;
  T* y;
  float *zg, *zu;   // pre-activations, or null
  int act, na;
  bool vec;         // rows of na values keep four-value alignment, and so do the biases
  // of the rows from b on (a multiple of four)
  GatedEpi from(int b) const {
    GatedEpi r = *this;
    const size_t at = size_t(b) * na;
    r.y += at;
    if (r.zg) r.zg += at;
    if (r.zu) r.zu += at;
    return r;
  }
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt&) const {
    acc_zero(acc);
  }
  __device__ __forceinline__ void finish(f32x4_t g, f32x4_t u, int b, int a, int n) const {
    const size_t at = size_t(b) * na + a;
    if (bg) g += load4(bg + a, n, vec);
    if (bu) u += load4(bu + a, n, vec);
    if (zg) {
      store4_any(zg + at, g, n, vec);
      store4_any(zu + at, u, n, vec);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] *= act_value<T>(act, g[e]);
    store4_any(y + at, u, n, vec);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) {
      const int a = t.a0 + 16 * i + 4 * (lane >> 4);
      if (a >= na) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15);
        if (b < t.nb) finish(acc[i][j], acc[i + FM / 2][j], b, a, na - a);
      }
    }
  }
};

// A split's sums: part[split][b][zg, ld values | zu, ld values].
struct GatedAddEpi {
  float* part;
  long ld, split;
  int na;
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt&) const {
    acc_zero(acc);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void done(f32x4_t (&acc)[FM][FN], const TileAt& t, void*) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int a = t.a0 + 16 * (i % (FM / 2)) + 4 * (lane >> 4);
      if (a >= na) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int b = t.b0 + 16 * j + (lane & 15);
        if (b < t.nb)
          store4(part + blockIdx.y * split + size_t(b) * 2 * ld + (i < FM / 2 ? 0 : ld) + a, acc[i][j], na - a, true);
      }
    }
  }
};

template <typename T>
__global__ __launch_bounds__(256) void join_gated_kernel(int M, int splits, const float* __restrict__ part, long ld,
                                                         GatedEpi<T> epi) {
  const int quads = (epi.na + 3) / 4;
  const long at = long(blockIdx.x) * 256 + threadIdx.x;
  if (at >= long(M) * quads) return;
  const int b = int(at / quads), a = int(at % quads) * 4;
  f32x4_t g = {0.f, 0.f, 0.f, 0.f}, u = g;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float* p = part + (size_t(s) * M + b) * 2 * ld + a;
    g += *reinterpret_cast<const f32x4_t*>(p);
    u += *reinterpret_cast<const f32x4_t*>(p + ld);
  }
  epi.finish(g, u, b, a, epi.na - a);
}

// 16 bytes of a row.  ODD: rows of an odd number of values, of which every
// second begins between two words: loads that do so take twice as long, so the
// words are loaded and shifted (one row, 4480 x 3999: 47 us before, 34 so).  A value behind the
// last of the eight has to exist, and one before a row that begins between words.
template <bool ODD>
__device__ __forceinline__ u32x4_t load_row(const bf16_t* p) {
  u32x4_t v;
  if (!ODD) {
    __builtin_memcpy(&v, p, 16);
    return v;
  }
#if defined(__HIP_DEVICE_COMPILE__)
  const bool between = reinterpret_cast<uintptr_t>(p) & 2;
  typedef uint32_t words_t __attribute__((ext_vector_type(4), aligned(4)));
  const words_t w = *reinterpret_cast<const words_t*>(p - between);
  const uint32_t next = *reinterpret_cast<const uint32_t*>(between ? p + 7 : p), shift = between ? 16 : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbit(i < 3 ? w[i + 1] : next, w[i], shift);
#endif
  return v;
}

// A few rows (M <= 16): both weights are read once, straight into the matrix
// instruction's operand registers; each of eight waves takes a share of the
// contraction, and LDS joins them (16384 x 4096, one row: 45.8 us, 5.9 TB/s, with
// four waves 57).  16 features per workgroup.  Any K: rows need element alignment
// only, and what is left of the contraction is masked.
//
// A load takes 128 bytes of each of 8 features, whole lines (with 64 bytes of
// 16 features, as the instruction's operand wants them, 10240 x 5120 takes 55 us
// for one row instead of 43): its operand rows l < 8 hold feature l and the
// first 32 of 64 of the contraction, l >= 8 feature l - 8 and the other 32.  Two
// instructions multiply it by both halves of x; of each result the half that
// belongs together is used.
template <bool ODD>
__global__ __launch_bounds__(512) void few_rows_gated_kernel(int M, int N, int K, const bf16_t* __restrict__ x,
                                                            const bf16_t* __restrict__ wg,
                                                            const bf16_t* __restrict__ wu, GatedEpi<bf16_t> epi) {
  constexpr int WAVES = 8;
  __shared__ f32x4_t part[WAVES][2][64];
#if defined(__HIP_DEVICE_COMPILE__)
  // uniform: matrix instructions ignore the lane mask, so nothing around them may diverge
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int a0 = blockIdx.x * 16;
  const int full = K / 64;   // whole steps of 64
  const int s0 = full * wave / WAVES, s1 = full * (wave + 1) / WAVES;
  const int chunk = (q + (l >> 3) * 4) * 8;   // this lane's place in a step, of the weights
  const long row0 = long(min(a0 + (l & 7), N - 1)) * K + chunk, row1 = long(min(a0 + 8 + (l & 7), N - 1)) * K + chunk;
  const bf16_t* px = x + long(min(l, M - 1)) * K + q * 8;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[2][2][2] = {{{zero, zero}, {zero, zero}}, {{zero, zero}, {zero, zero}}};   // matrix, features, half
  struct Step {
    u32x4_t w[2][2], b[2];
  };
  auto multiply = [&](const Step& t) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[m][f][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, t.w[m][f]),
                                                                 __builtin_bit_cast(bf16x8_t, t.b[h]), acc[m][f][h], 0, 0, 0);
  };
  constexpr int U = 2;   // steps in flight: 8 KiB of weights per wave
  for (int s = s0; s < s1; s += U) {
    Step t[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1) {
        const long at = long(s + i) * 64;
        t[i].w[0][0] = load_row<ODD>(wg + row0 + at);
        t[i].w[0][1] = load_row<ODD>(wg + row1 + at);
        t[i].w[1][0] = load_row<ODD>(wu + row0 + at);
        t[i].w[1][1] = load_row<ODD>(wu + row1 + at);
        t[i].b[0] = load_row<ODD>(px + at);
        t[i].b[1] = load_row<ODD>(px + at + 32);
      }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1) multiply(t[i]);
  }
  if (wave == WAVES - 1 && full * 64 < K) {   // the rest, zero behind the row's end
    const long at = long(full) * 64;
    const int left = K - full * 64;
    auto some = [&](const bf16_t* p, int n) {
      uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) v[e >> 1] |= uint32_t(p[e]) << (16 * (e & 1));
      return u32x4_t{v[0], v[1], v[2], v[3]};
    };
    Step t;
    t.w[0][0] = some(wg + row0 + at, left - chunk);
    t.w[0][1] = some(wg + row1 + at, left - chunk);
    t.w[1][0] = some(wu + row0 + at, left - chunk);
    t.w[1][1] = some(wu + row1 + at, left - chunk);
    t.b[0] = some(px + at, left - q * 8);
    t.b[1] = some(px + at + 32, left - q * 8 - 32);
    multiply(t);
  }
  // features 4 q + e: of the first eight in lanes q < 2, of the others in q >= 2;
  // the other half of the contraction's sum is two quarters away
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    f32x4_t v = q < 2 ? acc[m][0][0] : acc[m][1][1];
    const f32x4_t o = q < 2 ? acc[m][1][0] : acc[m][0][1];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(o[e], 32, 64);
    part[wave][m][lane] = v;
  }
  __syncthreads();
  if (wave == 0) {
    f32x4_t g = part[0][0][lane], u = part[0][1][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) {
      g += part[v][0][lane];
      u += part[v][1][lane];
    }
    const int a = a0 + 4 * q;
    if (l < M && a < N) epi.finish(g, u, l, a, N - a);
  }
#endif
}

// Four values at element alignment, n of them inside the row.
template <typename T>
__device__ __forceinline__ f32x4_t load4_any(const T* p, int n) {
  T v[4] = {};
  if (n >= 4) {
    __builtin_memcpy(v, p, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = p[i];
  }
  return f32x4_t{to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3])};
}

// Pre-activations, which are read this once: by the caches (4096 x 10240: 106 us
// for the kernel, 127 without).
__device__ __forceinline__ f32x4_t load4_once(const float* p, int n) {
  typedef float quad_t __attribute__((ext_vector_type(4), aligned(4)));
  if (n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const quad_t*>(p));
  return load4_any(p, n);
}

// dz[m][0][n] and dz[m][1][n] into rows of 2 ld values (columns N..ld of each
// half and rows M..rows zero), and the sums of both over a chunk of `per` rows,
// in fp32, before the rounding to T: part[chunk][2][n], or (one chunk) dbg and
// dbu themselves.  64 x 4 threads: four columns and every fourth row each.
template <typename T>
__global__ __launch_bounds__(256) void gated_dz_kernel(int M, int rows, int N, int act, const T* __restrict__ dy,
                                                       const float* __restrict__ zg, const float* __restrict__ zu,
                                                       T* __restrict__ dz, long ld, float* __restrict__ part, int per,
                                                       T* dbg, T* dbu) {
  __shared__ f32x4_t sums[3][2][64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6, n = (blockIdx.x * 64 + l) * 4;
  const int m1 = min(rows, (int(blockIdx.y) + 1) * per), left = N - n;
  f32x4_t sg = {0.f, 0.f, 0.f, 0.f}, su = sg;
  if (n < ld) {
#pragma unroll 4
    for (int m = blockIdx.y * per + q; m < m1; m += 4) {
      f32x4_t dg = {0.f, 0.f, 0.f, 0.f}, du = dg;
      if (m < M && left > 0) {
        const size_t at = size_t(m) * N + n;
        const f32x4_t d = load4_any(dy + at, left), g = load4_once(zg + at, left), u = load4_once(zu + at, left);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dg[e] = d[e] * u[e] * act_slope<T>(act, g[e]);
          du[e] = d[e] * act_value<T>(act, g[e]);
        }
      }
      if (dz) {
        store4(dz + size_t(m) * 2 * ld + n, dg, 4, true);
        store4(dz + size_t(m) * 2 * ld + ld + n, du, 4, true);
      }
      sg += dg;
      su += du;
    }
  }
  if (!part && !dbg && !dbu) return;
  if (q > 0) {
    sums[q - 1][0][l] = sg;
    sums[q - 1][1][l] = su;
  }
  __syncthreads();
  if (q > 0) return;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    sg += sums[i][0][l];
    su += sums[i][1][l];
  }
  float* p = part + size_t(blockIdx.y) * 2 * N + n;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) {
      if (part) {
        p[e] = sg[e];
        p[N + e] = su[e];
      } else {
        if (dbg) dbg[n + e] = from_f32<T>(sg[e]);
        if (dbu) dbu[n + e] = from_f32<T>(su[e]);
      }
    }
}

// dbg and dbu: sums over the chunks of the columns of both, 8 threads each,
// joined in order.  32 columns per workgroup.
template <typename T>
__global__ __launch_bounds__(256) void gated_dbias_kernel(int N, int chunks, const float* __restrict__ part, T* dbg,
                                                          T* dbu) {
  __shared__ float sums[8][32];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5, n = blockIdx.x * 32 + c;
  float s = 0.f;
  if (n < 2 * N) {
#pragma unroll 8
    for (int i = q; i < chunks; i += 8) s += part[size_t(i) * 2 * N + n];
  }
  sums[q][c] = s;
  __syncthreads();
  if (q == 0 && n < 2 * N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][c];
    T* out = n < N ? dbg : dbu;
    if (out) out[n < N ? n : n - N] = from_f32<T>(s);
  }
}

// The weights' gradients: row b of the product is a row of dwg (b < half) or of dwu.
template <typename T>
struct TwoOutEpi {
  T *g, *u;
  int half, N, na;
  bool vec;
  int first = 0;
  TwoOutEpi from(int b) const {
    TwoOutEpi r = *this;
    r.first = first + b;
    return r;
  }
  template <int FM, int FN>
  __device__ __forceinline__ void init(f32x4_t (&acc)[FM][FN], const TileAt&) const {
    acc_zero(acc);
  }
  __device__ __forceinline__ void join(f32x4_t v, int b, int a, int n) const {
    b += first;
    T* out = b < half ? g : u;
    const int row = b < half ? b : b - half;
    if (out && row < N) store4_any(out + size_t(row) * na + a, v, n, vec);
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
        if (b < t.nb) join(acc[i][j], b, a, na - a);
      }
    }
  }
};

template <typename T>
GatedEpi<T> gated_epi(const GatedArgs& a) {
  GatedEpi<T> epi;
  epi.bg = static_cast<const T*>(a.bg);
  epi.bu = static_cast<const T*>(a.bu);
  epi.y = static_cast<T*>(a.y);
  epi.zg = a.pre;
  epi.zu = a.pre ? a.pre + size_t(a.M) * a.N : nullptr;
  epi.act = a.act;
  epi.na = a.N;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.bg) | reinterpret_cast<uintptr_t>(a.bu);
  epi.vec = a.N % 4 == 0 && at % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.pre) % 16 == 0;
  return epi;
}

// Where the rows are few enough for few_rows_gated_kernel (weights from memory,
// us, against the tiles: one row of 8192 x 2560 17.3 and 20.3, of 16384 x 4096
// 45.8 and 60.7; sixteen 20.6 and 21.7, 50.9 and 60.3), whose rows of x come in
// 64-byte pieces: a long contraction of more than four is the tiles' (10240 x
// 5120, four rows 43.9 and 42.5, sixteen 50.8 and 44.2), unless they had to copy
// unaligned weights first.
bool few_gated_rows(int M, int K) { return M <= 4 || (M <= 16 && (K <= 4096 || K % 8 != 0)); }

Plan gated_plan(int M, int N, int K, bool bf16) {
  return bf16 ? plan_for(2 * N, M, K, false, false, true) : Plan{0, f32_splits(2 * N, M, K)};
}
// The rows of the first launch, and its or the second's split sums.
int gated_first(int M, int N, int K, bool bf16) { return bf16 ? second_part(2 * N, M, K, false) : M; }
size_t gated_split_bytes(int M, int N, int K, bool bf16) {
  const int first = gated_first(M, N, K, bf16);
  size_t most = 0;
  for (const int rows : {first, M - first}) {
    const int s = rows > 0 ? gated_plan(rows, N, K, bf16).splits : 1;
    const size_t n = s > 1 ? up256(size_t(s) * rows * 2 * up64(N) * 4) : 0;
    most = n > most ? n : most;
  }
  return most;
}
// Bytes of a copy of `rows` rows of K values to rows of whole steps.
size_t padded_bytes(long rows, int K) { return up256(size_t(rows) * up64(K) * 2); }

// Up to three matrices of K columns, copied to rows of ld values, zeros behind:
// one launch (y: which), eight values per thread.
struct Padded {
  const bf16_t* src[3];
  bf16_t* dst[3];
  long rows[3];
};
__global__ __launch_bounds__(256) void pad_matrices_kernel(Padded p, long n, long ld) {
  const bf16_t* src = blockIdx.y == 0 ? p.src[0] : blockIdx.y == 1 ? p.src[1] : p.src[2];
  bf16_t* dst = blockIdx.y == 0 ? p.dst[0] : blockIdx.y == 1 ? p.dst[1] : p.dst[2];
  const long rows = blockIdx.y == 0 ? p.rows[0] : blockIdx.y == 1 ? p.rows[1] : p.rows[2];
  const uint32_t per = uint32_t(ld / 8);
  const long at = long(blockIdx.x) * 256 + threadIdx.x;
  if (at >= rows * per) return;
  const long r = at / per, c = (at - r * per) * 8;
  const bf16_t* s = src + r * n;
  *reinterpret_cast<u32x4_t*>(dst + at * 8) = load_any(s + c, s + (c < n ? n : c));
}

// Copies to be made; add() gives one its place in the workspace, which *ws is
// moved on behind, and puts *p there.
struct Copies {
  Padded pad = {};
  int count = 0;
  void add(long rows, int K, const bf16_t** p, unsigned char** ws) {
    bf16_t* copy = reinterpret_cast<bf16_t*>(*ws);
    *ws += padded_bytes(rows, K);
    pad.src[count] = *p;
    pad.dst[count] = copy;
    pad.rows[count++] = rows;
    *p = copy;
  }
  hipError_t run(int K, hipStream_t stream) const {
    long most = 0;
    for (int i = 0; i < count; ++i) most = pad.rows[i] > most ? pad.rows[i] : most;
    if (most == 0) return hipSuccess;
    const long ld = up64(K), threads = most * (ld / 8);
    if (threads > 1l << 30) {   // more than a grid of three holds: one by one, in pieces
      for (int i = 0; i < count; ++i) {
        const hipError_t e = pad_rows(pad.rows[i], K, ld, pad.src[i], pad.dst[i], stream);
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    }
    hipLaunchKernelGGL(pad_matrices_kernel, dim3(unsigned((threads + 255) / 256), count), dim3(256), 0, stream, pad,
                       long(K), ld);
    return hipGetLastError();
  }
};

template <typename T>
hipError_t gated_rows(const Product<T>& g, const GatedEpi<T>& epi, int M, int N, int K, float* part, hipStream_t stream) {
  const Plan plan = gated_plan(M, N, K, sizeof(T) == 2);
  auto run = [&](auto&& make) {
    if constexpr (sizeof(T) == 2)
      return launch_bf16_dual(g, make, N, M, plan, stream);
    else
      return launch_f32_dual(g, make, N, M, plan.splits, stream);
  };
  if (plan.splits == 1) return run([&](auto) { return epi; });
  const long ld = up64(N);
  const hipError_t e = run([&](auto) { return GatedAddEpi{part, ld, long(M) * 2 * ld, N}; });
  if (e != hipSuccess) return e;
  const long quads = long(M) * ((N + 3) / 4);
  hipLaunchKernelGGL((join_gated_kernel<T>), dim3(unsigned((quads + 255) / 256)), dim3(256), 0, stream, M, plan.splits,
                     part, ld, epi);
  return hipGetLastError();
}

template <typename T>
hipError_t gated_product(const GatedArgs& a, const Product<T>& g, float* part, hipStream_t stream) {
  const GatedEpi<T> epi = gated_epi<T>(a);
  const int first = gated_first(a.M, a.N, a.K, sizeof(T) == 2);
  Product<T> p = g;
  p.B[0].n = first;
  const hipError_t e = gated_rows(p, epi, first, a.N, a.K, part, stream);
  if (e != hipSuccess || first == a.M) return e;
  p.B[0].n = a.M - first;
  p.B[0].p = g.B[0].p + long(first) * g.B[0].sa;
  return gated_rows(p, epi.from(first), a.M - first, a.N, a.K, part, stream);
}

hipError_t gated_bf16(const GatedArgs& a, hipStream_t stream) {
  const bf16_t *x = static_cast<const bf16_t*>(a.x), *wg = static_cast<const bf16_t*>(a.wg),
               *wu = static_cast<const bf16_t*>(a.wu);
  if (few_gated_rows(a.M, a.K)) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned((a.N + 15) / 16)), dim3(512), 0, stream, a.M, a.N, a.K, x, wg, wu,
                         gated_epi<bf16_t>(a));
      return hipGetLastError();
    };
    return a.K % 2 ? go(few_rows_gated_kernel<true>) : go(few_rows_gated_kernel<false>);
  }
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  // the b operand has to end in zeros, and the a operand's rows to be aligned
  const long ldx = a.K % kStep ? up64(a.K) : a.K, ldw = a.K % 8 ? up64(a.K) : a.K;
  Copies copies;
  if (a.K % kStep) copies.add(a.M, a.K, &x, &ws);
  if (a.K % 8) {
    copies.add(a.N, a.K, &wg, &ws);
    copies.add(a.N, a.K, &wu, &ws);
  }
  const hipError_t e = copies.run(a.K, stream);
  if (e != hipSuccess) return e;
  Product<bf16_t> g = {};
  g.A[0] = {wg, ldw, 1, a.N};
  g.A[1] = {wu, ldw, 1, a.N};
  g.B[0] = {x, ldx, 1, a.M};
  g.K[0] = a.K;
  return gated_product(a, g, reinterpret_cast<float*>(ws), stream);
}

hipError_t gated_f32(const GatedArgs& a, hipStream_t stream) {
  Product<float> g = {};
  g.A[0] = {static_cast<const float*>(a.wg), a.K, 1, a.N};
  g.A[1] = {static_cast<const float*>(a.wu), a.K, 1, a.N};
  g.B[0] = {static_cast<const float*>(a.x), a.K, 1, a.M};
  g.K[0] = a.K;
  return gated_product(a, g, static_cast<float*>(a.ws), stream);
}

long dz_rows(int M, bool bf16) { return bf16 ? up64(M) : M; }
// Rows whose sums one workgroup of gated_dz_kernel makes: all of few, whose
// bias gradients then need no second launch (8 x 256: 42 us against 38 for a
// training pass), else 16; the grid's second axis holds 65535 chunks.
int chunk_rows(long rows) { return rows <= 64 ? 64 : rows > 65535l * 16 ? 32 : 16; }
size_t part_bytes(int M, int N) {
  const long rows = up64(M), per = chunk_rows(rows);
  return rows <= per ? 0 : up256(size_t((rows + per - 1) / per) * 2 * N * 4);
}

template <typename T>
hipError_t gated_backward_t(const GatedBackwardArgs& a, hipStream_t stream) {
  constexpr bool bf16 = sizeof(T) == 2;
  const long ld = up64(a.N), rows = dz_rows(a.M, bf16);
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  const bool sums = a.dbg || a.dbu, products = (a.dx || a.dwg || a.dwu) && a.K > 0;
  const int per = chunk_rows(up64(a.M)), chunks = int((rows + per - 1) / per);
  float* part = up64(a.M) > per ? reinterpret_cast<float*>(ws) : nullptr;   // one chunk: the sums are the gradients
  ws += part_bytes(a.M, a.N);
  T* dz = reinterpret_cast<T*>(ws);
  ws += up256(size_t(rows) * 2 * ld * sizeof(T));
  hipError_t e = hipSuccess;
  if (rows > 0 && a.N > 0) {
    const float* zu = a.pre + size_t(a.M) * a.N;
    hipLaunchKernelGGL((gated_dz_kernel<T>), dim3(unsigned((ld + 255) / 256), unsigned(chunks)), dim3(256), 0, stream,
                       a.M, int(rows), a.N, a.act, static_cast<const T*>(a.dy), a.pre, zu, products ? dz : nullptr, ld,
                       sums ? part : nullptr, per, part ? nullptr : static_cast<T*>(a.dbg),
                       part ? nullptr : static_cast<T*>(a.dbu));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (sums && a.N > 0 && (part || rows == 0)) {
    hipLaunchKernelGGL((gated_dbias_kernel<T>), dim3(unsigned((2l * a.N + 31) / 32)), dim3(256), 0, stream, a.N, chunks,
                       part, static_cast<T*>(a.dbg), static_cast<T*>(a.dbu));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const T *wg = static_cast<const T*>(a.wg), *wu = static_cast<const T*>(a.wu), *x = static_cast<const T*>(a.x);
  long ldw = a.K;
  if constexpr (bf16) {
    if (a.K % 8) {   // the products' a operands need aligned rows
      ldw = up64(a.K);
      Copies copies;
      if (a.dx && a.M > 0) {
        copies.add(a.N, a.K, &wg, &ws);
        copies.add(a.N, a.K, &wu, &ws);
      }
      if ((a.dwg || a.dwu) && a.N > 0) copies.add(a.M, a.K, &x, &ws);
      if ((e = copies.run(a.K, stream)) != hipSuccess) return e;
    }
  }
  if (a.dx && a.K > 0 && a.M > 0) {
    Product<T> g = {};
    g.A[0] = {wg, 1, ldw, a.K};
    g.A[1] = {wu, 1, ldw, a.K};
    g.B[0] = {dz, 2 * ld, 1, a.M};
    g.B[1] = {dz + ld, 2 * ld, 1, a.M};
    g.K[0] = g.K[1] = a.N;
    LinearEpi<T> epi = {};
    epi.y = static_cast<T*>(a.dx);
    epi.na = a.K;
    epi.vec = aligned4<T>(a.dx, a.K);
    e = product_in_parts<kCols, kRows>(g, epi, a.K, a.M, reinterpret_cast<float*>(ws), stream);
    if (e != hipSuccess) return e;
  }
  if ((a.dwg || a.dwu) && a.K > 0 && a.N > 0) {
    Product<T> g = {};
    g.A[0] = {x, 1, ldw, a.K};
    g.B[0] = {dz, 1, 2 * ld, int(2 * ld)};
    g.K[0] = a.M;
    TwoOutEpi<T> epi;
    epi.g = static_cast<T*>(a.dwg);
    epi.u = static_cast<T*>(a.dwu);
    epi.half = int(ld);
    epi.N = a.N;
    epi.na = a.K;
    epi.vec = (!a.dwg || aligned4<T>(a.dwg, a.K)) && (!a.dwu || aligned4<T>(a.dwu, a.K));
    return product_in_parts<kCols, kCols>(g, epi, a.K, int(2 * ld), reinterpret_cast<float*>(ws), stream);
  }
  return hipSuccess;
}

}  // namespace

size_t gated_workspace_bytes(int M, int N, int K, bool bf16) {
  if (!bf16) return gated_split_bytes(M, N, K, false);
  if (few_gated_rows(M, K)) return 0;
  return (K % kStep ? padded_bytes(M, K) : 0) + (K % 8 ? 2 * padded_bytes(N, K) : 0) + gated_split_bytes(M, N, K, true);
}

size_t gated_backward_workspace_bytes(int M, int N, int K, bool bf16) {
  const long ld = up64(N);
  const size_t dz = part_bytes(M, N) + up256(size_t(dz_rows(M, bf16)) * 2 * ld * (bf16 ? 2 : 4));
  const size_t copies = bf16 && K % 8 != 0 ? 2 * padded_bytes(N, K) + padded_bytes(M, K) : 0;
  // the products come one after the other
  const size_t dx = parts_bytes(K, M, 2l * N, bf16, true), dw = parts_bytes(K, int(2 * ld), M, bf16, true);
  return dz + copies + (dx > dw ? dx : dw);
}

hipError_t launch_gated(const GatedArgs& a, hipStream_t stream) {
  return a.bf16 ? gated_bf16(a, stream) : gated_f32(a, stream);
}

hipError_t launch_gated_backward(const GatedBackwardArgs& a, hipStream_t stream) {
  return a.bf16 ? gated_backward_t<bf16_t>(a, stream) : gated_backward_t<float>(a, stream);
}

}  // namespace dspark
