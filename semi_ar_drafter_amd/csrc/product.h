// A product of either storage type into an epilogue, its contraction split
// into fp32 sums where there are too few tiles for the compute units.
#pragma once
#include "projection.h"
#include "tile_bf16.h"
#include "tile_f32.h"

namespace dspark {

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
inline long up64(long x) { return (x + 63) / 64 * 64; }

// Splits of a product's contraction into partial sums [split][rows][up64(na)].
inline size_t split_bytes(int na, int nb, long K, bool bf16, bool any, bool cols) {
  if (na == 0 || nb == 0) return 0;
  const int s = bf16 ? plan_for(na, nb, K, any, cols, true).splits : f32_splits(na, nb, K);
  return s > 1 ? up256(size_t(s) * nb * up64(na) * 4) : 0;
}

// The first of nb rows that a bf16 product makes in a second launch, or nb.
// Where the last round of 256 x 256 tiles fills a small part of the compute
// units, the rows of whole rounds come first, and the rest, split, takes a
// fraction of a round (4096 x 10240 x 5120, the input's gradient: 496 + 176 + 13
// us, in three splits 708 + 52; the weights': 688 + 53 + 13 us, in 6.25 rounds
// 789).
inline int second_part(int na, int nb, long K, bool cols) {
  const Plan whole = plan_for(na, nb, K, false, cols, true);
  if (whole.cost < 100) return nb;   // 160 us, of which another launch is a few
  const long tiles_a = (na + 255) / 256, tiles_b = (nb + 255) / 256, rounds = tiles_a * tiles_b / kComputeUnits;
  const long first = rounds * kComputeUnits / tiles_a * 256;   // rows of whole rounds
  if (first <= 0 || first >= nb) return nb;
  const Plan a = plan_for(na, int(first), K, false, cols, true), b = plan_for(na, int(nb - first), K, false, cols, true);
  return a.tile == 4 && a.splits == 1 && a.cost + b.cost + 3 < 0.97 * whole.cost ? int(first) : nb;
}

template <typename T>
bool aligned4(const void* p, int n) {
  return n % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

namespace {

// The epilogue of the sum over splits, in order: four values per thread.
template <class Epi>
__global__ __launch_bounds__(256) void join_splits_kernel(int M, int N, int splits, const float* __restrict__ part,
                                                          long ld, Epi epi) {
  const int quads = (N + 3) / 4;
  const long at = long(blockIdx.x) * 256 + threadIdx.x;
  if (at >= long(M) * quads) return;
  const int b = int(at / quads), a = int(at % quads) * 4, n = N - a;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(part + (size_t(s) * M + b) * ld + a);
  epi.join(v, b, a, n);
}

// A product into epi, or by way of split partial sums in `part`; LA, LB and
// any are for bf16 (fp32 kernels read any layout).
template <int LA, int LB, typename T, class Epi>
hipError_t product(const Product<T>& g, bool any, const Epi& epi, int na, int nb, float* part, hipStream_t stream) {
  if (na == 0 || nb == 0) return hipSuccess;
  constexpr bool bf16 = sizeof(T) == 2;
  const long K = long(g.K[0]) + g.K[1];
  const Plan plan = bf16 ? plan_for(na, nb, K, any, LA == kCols, true) : Plan{0, f32_splits(na, nb, K)};
  const int splits = plan.splits;
  auto run = [&](auto&& make) {
    if constexpr (bf16)
      return any ? launch_bf16<LA, LA, LB, true>(g, make, na, nb, plan, stream)
                 : launch_bf16<LA, LA, LB, false>(g, make, na, nb, plan, stream);
    else
      return launch_f32(g, make, na, nb, splits, stream);
  };
  if (splits == 1) return run([&](auto) { return epi; });
  const long ld = up64(na);
  const hipError_t e = run([&](auto) { return AddEpi{part, ld, na, true, long(nb) * ld}; });
  if (e != hipSuccess) return e;
  const long quads = long(nb) * ((na + 3) / 4);
  hipLaunchKernelGGL((join_splits_kernel<Epi>), dim3(unsigned((quads + 255) / 256)), dim3(256), 0, stream, nb, na,
                     splits, part, ld, epi);
  return hipGetLastError();
}

// The same in up to two launches; epi.from(b) is the epilogue of the rows from
// b on.  fp32 has one.
template <int LA, int LB, typename T, class Epi>
hipError_t product_in_parts(const Product<T>& g, const Epi& epi, int na, int nb, float* part, hipStream_t stream) {
  const int first = sizeof(T) == 2 && na > 0 && nb > 0 ? second_part(na, nb, long(g.K[0]) + g.K[1], LA == kCols) : nb;
  Product<T> p = g;
  for (int i = 0; i < 2; ++i) p.B[i].n = first;
  const hipError_t e = product<LA, LB>(p, false, epi, na, first, part, stream);
  if (e != hipSuccess || first == nb) return e;
  for (int i = 0; i < 2; ++i) {
    p.B[i].n = nb - first;
    if (g.B[i].p) p.B[i].p = g.B[i].p + long(first) * g.B[i].sa;
  }
  return product<LA, LB>(p, false, epi.from(first), na, nb - first, part, stream);
}
inline size_t parts_bytes(int na, int nb, long K, bool bf16, bool cols) {
  if (na == 0 || nb == 0 || !bf16) return split_bytes(na, nb, K, bf16, false, cols);
  const int first = second_part(na, nb, K, cols);
  const size_t a = split_bytes(na, first, K, true, false, cols), b = split_bytes(na, nb - first, K, true, false, cols);
  return a > b ? a : b;
}

}  // namespace

}  // namespace dspark
