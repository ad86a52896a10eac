// Linear layer: y = act(x w^T + bias) + residual, and its gradients.
//
//   forward    C(a = output feature, b = row) = w[a] . x[b]
//   dx         C(a = input feature, b = row)  = sum_n w[n][a] dz[b][n]
//   dw         C(a = input feature, b = output feature) = sum_m x[m][a] dz[m][b]
// with dz = dy act'(pre), made once by dz_kernel together with the sums over
// rows that give the bias gradient.
#include "launch.h"
#include "projection.h"
#include "tile_f32.h"

namespace dspark {

namespace {

constexpr int kDzRows = 64;   // rows per workgroup of dz_kernel

// dz[m][n] = T(dy act'(pre)) into rows of ld values (columns N..ld zero), and
// part[chunk][n] = the chunk's sum of dz over its rows, in fp32, before the
// rounding to T.  256 threads, one column each.
template <typename T>
__global__ __launch_bounds__(256) void dz_kernel(int M, int N, int act, const T* __restrict__ dy,
                                                 const float* __restrict__ pre, T* __restrict__ dz, long ld,
                                                 float* __restrict__ part) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int m0 = blockIdx.y * kDzRows, m1 = min(M, m0 + kDzRows);
  if (n >= N) {
    if (dz && n < ld)
      for (int m = m0; m < m1; ++m) dz[size_t(m) * ld + n] = from_f32<T>(0.f);
    return;
  }
  float s = 0.f;
  for (int m = m0; m < m1; ++m) {
    float v = to_f32(dy[size_t(m) * N + n]);
    if (act) v *= act_slope(act, pre[size_t(m) * N + n]);
    if (dz) dz[size_t(m) * ld + n] = from_f32<T>(v);
    s += v;
  }
  if (part) part[size_t(blockIdx.y) * N + n] = s;
}

// dbias[n] = sum over chunks, in chunk order.
template <typename T>
__global__ __launch_bounds__(256) void dbias_kernel(int N, int chunks, const float* __restrict__ part,
                                                    T* __restrict__ dbias) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  for (int c = 0; c < chunks; ++c) s += part[size_t(c) * N + n];
  dbias[n] = from_f32<T>(s);
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
inline long dz_stride(int N) { return (long(N) + 63) / 64 * 64; }
inline int dz_chunks(int M) { return (M + kDzRows - 1) / kDzRows; }

template <typename T>
hipError_t linear_t(const LinearArgs& a, hipStream_t stream) {
  Product<T> g = {};
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  g.A[0] = {w, a.K, 1, a.N};
  g.B[0] = {x, a.K, 1, a.M};
  g.K[0] = a.K;
  LinearEpi<T> epi;
  epi.bias = static_cast<const T*>(a.bias);
  epi.residual = static_cast<const T*>(a.residual);
  epi.y = static_cast<T*>(a.y);
  epi.pre = a.pre;
  epi.act = a.act;
  epi.na = a.N;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.residual);
  epi.vec = a.N % 4 == 0 && at % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.pre) % 16 == 0;
  return launch_tile_f32(g, epi, a.N, a.M, stream);
}

template <typename T>
hipError_t linear_backward_t(const LinearBackwardArgs& a, hipStream_t stream) {
  const T* dz = static_cast<const T*>(a.dy);
  long ld = a.N;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  float* part = reinterpret_cast<float*>(ws);
  hipError_t e;
  if (a.N > 0 && (a.act || a.dbias)) {
    T* out = nullptr;
    if (a.act) {
      ld = dz_stride(a.N);
      out = reinterpret_cast<T*>(ws + up256(size_t(dz_chunks(a.M)) * a.N * 4));
      dz = out;
    }
    if (a.M > 0)
      hipLaunchKernelGGL((dz_kernel<T>), dim3(unsigned((ld + 255) / 256), unsigned(dz_chunks(a.M))), dim3(256), 0,
                         stream, a.M, a.N, a.act, static_cast<const T*>(a.dy), a.pre, out, ld,
                         a.dbias ? part : nullptr);
    if (a.dbias)
      hipLaunchKernelGGL((dbias_kernel<T>), dim3(unsigned((a.N + 255) / 256)), dim3(256), 0, stream, a.N,
                         dz_chunks(a.M), part, static_cast<T*>(a.dbias));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dx && a.M > 0 && a.K > 0) {
    Product<T> g = {};
    g.A[0] = {static_cast<const T*>(a.w), 1, a.K, a.K};
    g.B[0] = {dz, ld, 1, a.M};
    g.K[0] = a.N;
    StoreEpi<T> epi{static_cast<T*>(a.dx), a.K, a.K,
                    a.K % 4 == 0 && reinterpret_cast<uintptr_t>(a.dx) % (4 * sizeof(T)) == 0};
    if ((e = launch_tile_f32(g, epi, a.K, a.M, stream)) != hipSuccess) return e;
  }
  if (a.dw && a.N > 0 && a.K > 0) {
    Product<T> g = {};
    g.A[0] = {static_cast<const T*>(a.x), 1, a.K, a.K};
    g.B[0] = {dz, 1, ld, a.N};
    g.K[0] = a.M;
    StoreEpi<T> epi{static_cast<T*>(a.dw), a.K, a.K,
                    a.K % 4 == 0 && reinterpret_cast<uintptr_t>(a.dw) % (4 * sizeof(T)) == 0};
    if ((e = launch_tile_f32(g, epi, a.K, a.N, stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t linear_workspace_bytes(int, int, int, bool) { return 0; }

size_t linear_backward_workspace_bytes(int M, int N, int, bool bf16) {
  return up256(size_t(dz_chunks(M)) * N * 4) + up256(size_t(M) * dz_stride(N) * (bf16 ? 2 : 4));
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  return a.bf16 ? linear_t<bf16_t>(a, stream) : linear_t<float>(a, stream);
}

hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t stream) {
  return a.bf16 ? linear_backward_t<bf16_t>(a, stream) : linear_backward_t<float>(a, stream);
}

}  // namespace dspark
