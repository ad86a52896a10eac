// Matrix product on the fp32 matrix instruction (v_mfma_f32_16x16x4_f32) for
// any type, layout, size and alignment: operands are read element by element
// with bounds checks and widened to fp32 on the way into LDS.
#pragma once
#include "projection.h"

namespace dspark {

constexpr int kTileF32 = 128;   // tile along a and along b
constexpr int kTileF32K = 16;   // contraction per step
constexpr int kTileF32Pad = kTileF32 + 4;
constexpr int kTileF32Lds = 2 * kTileF32K * kTileF32Pad;   // floats

// 256 threads = 2 x 2 waves, 64 x 64 of C each.  One workgroup per tile,
// tiles of b fastest.
template <typename T, class Epi>
__global__ __launch_bounds__(256) void tile_f32_kernel(Product<T> g, Epi epi, int na, int nb) {
  __shared__ float lds[kTileF32Lds];
  float* As = lds;
  float* Bs = lds + kTileF32K * kTileF32Pad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles_b = (nb + kTileF32 - 1) / kTileF32;
  if (g.nb) nb = *g.nb;
  const int tile_a = blockIdx.x / tiles_b, tile_b = blockIdx.x % tiles_b;
  const int a_first = tile_a * kTileF32, b_first = tile_b * kTileF32;
  if (b_first >= nb) return;   // all its rows are behind the last one in use
  TileAt t;
  t.wave_a = wave >> 1;
  t.wave_b = wave & 1;
  t.a0 = a_first + 64 * t.wave_a;
  t.b0 = b_first + 64 * t.wave_b;
  t.nb = nb;
  t.tile_a = tile_a;
  f32x4_t acc[4][4];
  epi.init(acc, t);
  for (int part = 0; part < 2; ++part) {
    const int K = part == 0 && g.k0 ? *g.k0 : g.K[part];
    const Operand<T>&A = g.A[part], &B = g.B[part];
    for (int k0 = 0; k0 < K; k0 += kTileF32K) {
      __syncthreads();
#pragma unroll
      for (int op = 0; op < 2; ++op) {
        const Operand<T>& O = op ? B : A;
        float* S = op ? Bs : As;
        const int first = op ? b_first : a_first;
#pragma unroll
        for (int i = 0; i < kTileF32 * kTileF32K / 256; ++i) {
          const int e = tid + 256 * i;
          const int c = O.sk == 1 ? e / kTileF32K : e % kTileF32;
          const int k = O.sk == 1 ? e % kTileF32K : e / kTileF32;
          float v = 0.f;
          if (first + c < O.n && k0 + k < K) v = to_f32(O.p[long(first + c) * O.sa + long(k0 + k) * O.sk]);
          S[k * kTileF32Pad + c] = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kTileF32K; kk += 4) {
        const int row = (kk + (lane >> 4)) * kTileF32Pad + (lane & 15);
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = As[row + 64 * t.wave_a + 16 * i];
          b[i] = Bs[row + 64 * t.wave_b + 16 * i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    }
  }
  __syncthreads();
  epi.done(acc, t, lds);
}

template <typename T, class Epi>
hipError_t launch_tile_f32(const Product<T>& g, const Epi& epi, int na, int nb, hipStream_t stream) {
  if (na <= 0 || nb <= 0) return hipSuccess;
  const unsigned tiles = unsigned((na + kTileF32 - 1) / kTileF32) * unsigned((nb + kTileF32 - 1) / kTileF32);
  hipLaunchKernelGGL((tile_f32_kernel<T, Epi>), dim3(tiles), dim3(256), 0, stream, g, epi, na, nb);
  return hipGetLastError();
}

}  // namespace dspark
