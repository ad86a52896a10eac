// Matrix product of fp32 operands on v_mfma_f32_16x16x4_f32, for any layout,
// size and alignment.
//
// A step covers 32 of the contraction.  Each operand's step goes through
// registers (16-byte loads at element alignment, sent off a step ahead) into
// one of two LDS buffers, as it is stored:
//   kRows  [a][32 k], 128 bytes a row; one ds_read_b128 gives a lane four
//          consecutive k, the operands of four MFMAs (the contraction's order
//          is free as long as both operands agree: MFMA e takes k = 16 half +
//          4 (lane / 16) + e).  16-byte chunk c of row a lies at c ^ (a & 7).
//   kCols  [32 k][a]; four ds_read_b32, each 16 neighbouring a of four k that
//          are four rows apart: rows are padded by 4 so that these fall on
//          different banks.
#pragma once
#include "projection.h"

namespace dspark {

constexpr int kStepF32 = 32;

// Tile: BM along a, BN along b, WA x WB waves.
template <int BM_, int BN_, int WA_, int WB_>
struct TileF32 {
  static constexpr int BM = BM_, BN = BN_, WA = WA_, WB = WB_;
  static constexpr int threads = 64 * WA * WB, FM = BM / WA / 16, FN = BN / WB / 16;
  // bytes of one operand's step, in either layout
  static constexpr int bytes(int rows) { return (rows + 4) * kStepF32 * 4; }
  static constexpr int stage = bytes(BM) + bytes(BN), lds = 2 * stage;
};

// One operand's step: `ROWS` rows of a by 32 of k, LOADS 16-byte chunks per thread.
// PAIR > 0: PAIR rows of o and PAIR of `other` in turn, both by rows.
template <int ROWS, int THREADS, int PAIR = 0>
struct StepF32 {
  static constexpr int chunks = ROWS * kStepF32 / 4, loads = (chunks + THREADS - 1) / THREADS;
  f32x4_t v[loads];

  __device__ __forceinline__ void load(const Operand<float>& o, int first, int k0, int K, int tid,
                                       const float* other = nullptr) {
#pragma unroll
    for (int i = 0; i < loads; ++i) {
      const int at = tid + i * THREADS;
      if (chunks % THREADS && at >= chunks) break;
      f32x4_t r = {0.f, 0.f, 0.f, 0.f};
      int n;           // values of the chunk that exist
      const float* p;
      if (PAIR || o.sk == 1) {
        const int row = at / 8, k = k0 + at % 8 * 4;
        const int a = first + (PAIR ? row / (2 * PAIR + !PAIR) * PAIR + row % (PAIR + !PAIR) : row);
        n = a < o.n ? K - k : 0;
        p = (PAIR && row / (PAIR + !PAIR) % 2 ? other : o.p) + long(a) * o.sa + k;
      } else {
        const int k = k0 + at / (ROWS / 4), a = first + at % (ROWS / 4) * 4;
        n = k < K ? o.n - a : 0;
        p = o.p + long(k) * o.sk + a;
      }
      if (n >= 4) {
        __builtin_memcpy(&r, p, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) r[e] = p[e];
      }
      v[i] = r;
    }
  }
  __device__ __forceinline__ void put(float* lds, bool rows, int tid) const {
#pragma unroll
    for (int i = 0; i < loads; ++i) {
      const int at = tid + i * THREADS;
      if (chunks % THREADS && at >= chunks) break;
      float* d;
      if (rows) {
        const int a = at / 8;
        d = lds + a * 32 + ((at % 8) ^ (a & 7)) * 4;
      } else {
        d = lds + at / (ROWS / 4) * (ROWS + 4) + at % (ROWS / 4) * 4;
      }
      *reinterpret_cast<f32x4_t*>(d) = v[i];
    }
  }
};

// One fragment: a lane's values for the four MFMAs of 16 of k.
template <int ROWS>
__device__ __forceinline__ f32x4_t frag_f32(const float* lds, bool rows, int a, int half, int lane) {
  const int l = lane & 15, q = lane >> 4;
  if (rows) return *reinterpret_cast<const f32x4_t*>(lds + (a + l) * 32 + (((half * 4 + q) ^ (l & 7)) * 4));
  f32x4_t r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = lds[(half * 16 + q * 4 + e) * (ROWS + 4) + a + l];
  return r;
}

// grid: x tiles (of b fastest), y splits of the contraction.  DUAL: the a
// operand is two matrices of na rows, A[0] and A[1], multiplied by the same b
// over one contraction; a wave's accumulators i < FM / 2 belong to the first.
template <class Sh, class Epi, bool DUAL = false>
__global__ __launch_bounds__(Sh::threads) void tile_f32_kernel(Product<float> g, Epi epi, int na, int nb) {
  extern __shared__ __align__(128) float smem_f32[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles_b = (nb + Sh::BN - 1) / Sh::BN;
  if (g.nb) nb = *g.nb;
  const int tile_a = blockIdx.x / tiles_b, tile_b = blockIdx.x % tiles_b;
  constexpr int BM = DUAL ? Sh::BM / 2 : Sh::BM;
  static_assert(!DUAL || Sh::FM % 2 == 0, "two matrices by rows");
  const int a_first = tile_a * BM, b_first = tile_b * Sh::BN;
  if (b_first >= nb) return;   // all its rows are behind the last one in use
  const int K0 = g.k0 ? *g.k0 : g.K[0], K1 = g.K[1];
  const int T0 = (K0 + kStepF32 - 1) / kStepF32, T = T0 + (K1 + kStepF32 - 1) / kStepF32;
  const int t_begin = int(long(T) * blockIdx.y / gridDim.y), t_end = int(long(T) * (blockIdx.y + 1) / gridDim.y);
  TileAt t;
  t.wave_a = wave / Sh::WB;
  t.wave_b = wave % Sh::WB;
  t.a0 = a_first + t.wave_a * (BM / Sh::WA);
  t.b0 = b_first + t.wave_b * (Sh::BN / Sh::WB);
  t.nb = nb;
  t.tile_a = tile_a;

  StepF32<Sh::BM, Sh::threads, DUAL ? BM / Sh::WA : 0> sa;
  StepF32<Sh::BN, Sh::threads> sb;
  auto load = [&](int s) {
    const int part = s >= T0;
    const int k = (part ? s - T0 : s) * kStepF32, K = part ? K1 : K0;
    sa.load(g.A[part], a_first, k, K, tid, DUAL ? g.A[1].p : nullptr);
    sb.load(g.B[part], b_first, k, K, tid);
  };
  if (t_begin < t_end) load(t_begin);
  f32x4_t acc[Sh::FM][Sh::FN];
  epi.init(acc, t);
  for (int s = t_begin; s < t_end; ++s) {
    const int part = s >= T0;
    const bool rows_a = g.A[part].sk == 1, rows_b = g.B[part].sk == 1;
    float* A = smem_f32 + (s & 1) * (Sh::stage / 4);
    float* B = A + Sh::bytes(Sh::BM) / 4;
    sa.put(A, rows_a, tid);
    sb.put(B, rows_b, tid);
    // one barrier a step: the buffer written next was read before this one
    __syncthreads();
    if (s + 1 < t_end) load(s + 1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f32x4_t a[Sh::FM], b[Sh::FN];
#pragma unroll
      for (int i = 0; i < Sh::FM; ++i)
        a[i] = frag_f32<Sh::BM>(A, rows_a, t.wave_a * (Sh::BM / Sh::WA) + 16 * i, half, lane);
#pragma unroll
      for (int j = 0; j < Sh::FN; ++j)
        b[j] = frag_f32<Sh::BN>(B, rows_b, t.wave_b * (Sh::BN / Sh::WB) + 16 * j, half, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < Sh::FM; ++i)
#pragma unroll
          for (int j = 0; j < Sh::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();
  epi.done(acc, t, smem_f32);
}

using WideF32 = TileF32<128, 128, 2, 2>;
using MidF32 = TileF32<64, 64, 2, 2>;
using SlimF32 = TileF32<64, 16, 4, 1>;
using SlimDualF32 = TileF32<128, 16, 4, 1>;   // two matrices take an even number of fragments

// 0: few rows; 1: too few wide tiles for the compute units; 2: wide.  With a
// contraction of 1024, wide against narrow, us: 128 tiles 63 against 67, 192
// 101 against 86 (its splits leave a quarter of the last round empty), 256 105
// against 109, 512 (2048 long) 348 against 404, 1024 351 against 400.
inline int f32_choice(int na, int nb) {
  if (nb <= 16) return 0;
  const long wide = long((na + 127) / 128) * ((nb + 127) / 128);
  return wide >= 192 ? 2 : 1;
}
// Splits of a contraction into fp32 sums, for about two workgroups per
// compute unit, each with at least two steps (for one, two and four, us: 256 x
// 1024 x 2048 30.6, 24.9 and 25.5; 128 x 4096 x 2560 62, 47 and 44.5; 8 x 4096
// x 1024 13.1, 9.9 and 10.1).
inline int f32_splits(int na, int nb, long K) {
  const int c = f32_choice(na, nb), bm = c == 2 ? 128 : 64, bn = c == 2 ? 128 : c == 1 ? 64 : 16;
  const long tiles = long((na + bm - 1) / bm) * ((nb + bn - 1) / bn), steps = (K + kStepF32 - 1) / kStepF32;
  long s = 512 / tiles;
  if (s > steps / 2) s = steps / 2;
  return s < 1 ? 1 : s > 64 ? 64 : int(s);
}

template <class Sh, bool DUAL = false, class Epi>
hipError_t launch_tile_f32(const Product<float>& g, const Epi& epi, int na, int nb, int splits, hipStream_t stream) {
  constexpr int BM = DUAL ? Sh::BM / 2 : Sh::BM;
  const unsigned tiles = unsigned((na + BM - 1) / BM) * unsigned((nb + Sh::BN - 1) / Sh::BN);
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(&tile_f32_kernel<Sh, Epi, DUAL>), Sh::lds, allowed);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_f32_kernel<Sh, Epi, DUAL>), dim3(tiles, unsigned(splits)), dim3(Sh::threads), Sh::lds, stream, g,
                     epi, na, nb);
  return hipGetLastError();
}

// make(shape) gives the epilogue.
template <class Make>
hipError_t launch_f32(const Product<float>& g, const Make& make, int na, int nb, int splits, hipStream_t stream) {
  if (na <= 0 || nb <= 0) return hipSuccess;
  switch (f32_choice(na, nb)) {
    case 0: return launch_tile_f32<SlimF32>(g, make(SlimF32()), na, nb, splits, stream);
    case 1: return launch_tile_f32<MidF32>(g, make(MidF32()), na, nb, splits, stream);
    default: return launch_tile_f32<WideF32>(g, make(WideF32()), na, nb, splits, stream);
  }
}

// The same for two matrices of na rows each, chosen and split as 2 na.
template <class Make>
hipError_t launch_f32_dual(const Product<float>& g, const Make& make, int na, int nb, int splits, hipStream_t stream) {
  if (na <= 0 || nb <= 0) return hipSuccess;
  switch (f32_choice(2 * na, nb)) {
    case 0: return launch_tile_f32<SlimDualF32, true>(g, make(SlimDualF32()), na, nb, splits, stream);
    case 1: return launch_tile_f32<MidF32, true>(g, make(MidF32()), na, nb, splits, stream);
    default: return launch_tile_f32<WideF32, true>(g, make(WideF32()), na, nb, splits, stream);
  }
}

}  // namespace dspark
