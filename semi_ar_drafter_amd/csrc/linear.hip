// Linear layer: y = act(x w^T + bias) + residual, and its gradients.
//
//   forward    C(a = output feature, b = row) = w[a] . x[b]
//   dx         C(a = input feature, b = row)  = sum_n w[n][a] dz[b][n]
//   dw         C(a = input feature, b = output feature) = sum_m x[m][a] dz[m][b]
// with dz = dy act'(pre), made once by dz_kernel together with the sums over
// rows that give the bias gradient.  dz is rounded to the storage type, which
// the products take: dx and dw then err 1.4 times as much as by their own
// rounding (2.3e-3 against 1.7e-3 of the norm in bf16); without an activation
// dz is dy and nothing is rounded.
//
// Bound by reading w with few rows (8 rows, 151936 x 2560: 134 us, 5.8 TB/s), by
// the main loop of the matrix unit's tiles with many (1024 rows, 151936 x 4096:
// 1.07 ms, 1.19 PFLOP/s; 4096 x 5120 x 5120 with its gradients: 242 + 246 + 212
// us, whose last rounds of tiles fill a part of the compute units, dz_kernel 37
// us for 168 MB).
#include "launch.h"
#include "product.h"

namespace dspark {

namespace {

constexpr int kDzRows = 16;   // rows per workgroup of dz_kernel where it sums, 4 where it does not

// dz[m][n] = T(dy act'(pre)) into rows of ld values (columns N..ld and rows
// M..rows zero), and part[chunk][n] = the chunk's sum of dz over its rows, in
// fp32, before the rounding to T.  256 threads, four columns each; vec: rows
// of N values keep four-value alignment.
template <typename T>
__global__ __launch_bounds__(256) void dz_kernel(int M, int rows, int N, int act, const T* __restrict__ dy,
                                                 const float* __restrict__ pre, T* __restrict__ dz, long ld,
                                                 float* __restrict__ part, bool vec, int per) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int m0 = blockIdx.y * per, m1 = min(rows, m0 + per);
  if (n >= ld) return;
  const int left = N - n;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int m = m0; m < m1; ++m) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (m < M && left > 0) {
      v = load4(dy + size_t(m) * N + n, left, vec);
      if (act) {
        const f32x4_t z = load4(pre + size_t(m) * N + n, left, vec);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= act_slope<T>(act, z[e]);
      }
    }
    // a row of dz is dy's own (no copy) or ld long, a multiple of 64
    if (dz) store4(dz + size_t(m) * ld + n, v, 4, true);
    s += v;
  }
  if (part) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) part[size_t(blockIdx.y) * N + n + e] = s[e];
  }
}

// dbias[n] = sum over chunks: 8 threads per column take every eighth chunk
// each, then join in order.  32 columns per workgroup.
template <typename T>
__global__ __launch_bounds__(256) void dbias_kernel(int N, int chunks, const float* __restrict__ part,
                                                    T* __restrict__ dbias) {
  __shared__ float sums[8][32];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5, n = blockIdx.x * 32 + c;
  float s = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int i = q; i < chunks; i += 8) s += part[size_t(i) * N + n];
  }
  sums[q][c] = s;
  __syncthreads();
  if (q == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][c];
    dbias[n] = from_f32<T>(s);
  }
}

// A few rows (M <= 16): the weights are read once, straight into the matrix
// instruction's operand registers (a lane takes 16 bytes of one of 16 rows of
// w), and the rows of x come the same way out of the caches.  Each of WAVES
// waves takes a share of the contraction; LDS joins them.  16 output features
// per workgroup.  Any K: rows need element alignment only, and the last 32 of
// the contraction are masked.
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void few_rows_kernel(int M, int N, int K, const bf16_t* __restrict__ x,
                                                              const bf16_t* __restrict__ w, LinearEpi<bf16_t> epi) {
  __shared__ f32x4_t part[WAVES][64];
#if defined(__HIP_DEVICE_COMPILE__)
  // uniform: matrix instructions ignore the lane mask, so nothing around them may diverge
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
  const int a0 = blockIdx.x * 16;
  const int full = K / 32;   // whole steps of 32
  const int s0 = full * wave / WAVES, s1 = full * (wave + 1) / WAVES;
  const bf16_t* pw = w + long(min(a0 + l, N - 1)) * K + q * 8;
  const bf16_t* px = x + long(min(l, M - 1)) * K + q * 8;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto step = [&](u32x4_t a, u32x4_t b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc,
                                                  0, 0, 0);
  };
  int s = s0;
  constexpr int U = 8;   // steps in flight: 8 KiB of weights per wave
  for (; s + U <= s1; s += U) {
    u32x4_t a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) __builtin_memcpy(&a[u], pw + (s + u) * 32, 16);
#pragma unroll
    for (int u = 0; u < U; ++u) __builtin_memcpy(&b[u], px + (s + u) * 32, 16);
#pragma unroll
    for (int u = 0; u < U; ++u) step(a[u], b[u]);
  }
  if (s < s1) {
    u32x4_t a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) {
        __builtin_memcpy(&a[u], pw + (s + u) * 32, 16);
        __builtin_memcpy(&b[u], px + (s + u) * 32, 16);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) step(a[u], b[u]);
  }
  if (wave == WAVES - 1 && full * 32 < K) {   // the rest, zero behind the row's end
    const int n = K - full * 32 - q * 8;
    uint32_t a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) {
        a[e >> 1] |= uint32_t(pw[full * 32 + e]) << (16 * (e & 1));
        b[e >> 1] |= uint32_t(px[full * 32 + e]) << (16 * (e & 1));
      }
    step(u32x4_t{a[0], a[1], a[2], a[3]}, u32x4_t{b[0], b[1], b[2], b[3]});
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int v = 1; v < WAVES; ++v) acc += part[v][lane];
    const int a = a0 + 4 * q, n = N - a;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (l < M && n > 0)
      epi.finish(acc, epi.bias ? load4(epi.bias + a, n, epi.vec) : zero,
                 epi.residual ? load4(epi.residual + size_t(l) * N + a, n, epi.vec) : zero, l, a, n);
  }
#endif
}

inline long dz_stride(int N) { return up64(N); }
inline int dz_chunks(int M) { return int((up64(M) + kDzRows - 1) / kDzRows); }

template <typename T>
LinearEpi<T> linear_epi(const LinearArgs& a) {
  LinearEpi<T> epi;
  epi.bias = static_cast<const T*>(a.bias);
  epi.residual = static_cast<const T*>(a.residual);
  epi.y = static_cast<T*>(a.y);
  epi.pre = a.pre;
  epi.act = a.act;
  epi.na = a.N;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.residual) |
                       reinterpret_cast<uintptr_t>(a.bias);
  epi.vec = a.N % 4 == 0 && at % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.pre) % 16 == 0;
  return epi;
}

// Where few_rows_kernel beats the tiles (per call, in a graph): for one row
// always (4096 x 2560: 6.0 us against 10.0, 65536 x 4096: 92 against 107); for
// sixteen, whose rows of x come in 64-byte pieces at the same rate as the
// weights, up to 8192 features (11.7 us against 13.3; at 16384 20.7 against
// 19.1).  Rows that are not 16-byte aligned halve both: 8192 x 2561, one row
// 19 us against 20, sixteen 33 against 21.
bool few_rows(int M, int N, int K) {
  return K % 8 == 0 ? M <= 4 || (M <= 16 && N <= 8192) : M <= 16 && N * M <= 32768;
}

// Whether a product's a operand of `rows` rows (none: nothing to copy) of K
// values is copied to aligned rows: only for many b (77 x 1027 x 1001, split:
// 17.1 us without, 19.8 with the copy).
bool copies(int rows, int K, int nb) {
  return rows > 0 && K % 8 != 0 && nb >= 256 && size_t(rows) * up64(K) * 2 <= kCopyBytes;
}
// Bytes of the copy, and whether the product still sees unaligned rows.
size_t copy_bytes(int rows, int K, int nb) { return copies(rows, K, nb) ? up256(size_t(rows) * up64(K) * 2) : 0; }
bool stays_any(int rows, int K, int nb) { return K % 8 != 0 && !copies(rows, K, nb); }

hipError_t linear_bf16(const LinearArgs& a, hipStream_t stream) {
  if (few_rows(a.M, a.N, a.K)) {
    const bf16_t *x = static_cast<const bf16_t*>(a.x), *w = static_cast<const bf16_t*>(a.w);
    const dim3 grid(unsigned((a.N + 15) / 16));
    // more waves share the contraction where there are too few workgroups to
    // fill the compute units (one row, 8 waves against 4, us: 4096 x 4096 7.4
    // against 8.0, 8192 x 4096 13.2 against 14.5, 16384 x 4096 23.2 both,
    // 151936 x 512 26.0 against 24.4)
    if (a.N <= 16 * 2 * kComputeUnits)
      hipLaunchKernelGGL((few_rows_kernel<8>), grid, dim3(512), 0, stream, a.M, a.N, a.K, x, w, linear_epi<bf16_t>(a));
    else
      hipLaunchKernelGGL((few_rows_kernel<4>), grid, dim3(256), 0, stream, a.M, a.N, a.K, x, w, linear_epi<bf16_t>(a));
    return hipGetLastError();
  }
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  const bf16_t* x = static_cast<const bf16_t*>(a.x);
  long ldx = a.K;
  if (a.K % kStep) {   // the b operand has to end in zeros
    ldx = up64(a.K);
    bf16_t* xp = reinterpret_cast<bf16_t*>(ws);
    ws += up256(size_t(a.M) * ldx * 2);
    const hipError_t e = pad_rows(a.M, a.K, ldx, x, xp, stream);
    if (e != hipSuccess) return e;
    x = xp;
  }
  const bf16_t* w = static_cast<const bf16_t*>(a.w);
  long ldw = a.K;
  if (copies(a.N, a.K, a.M)) {
    ldw = up64(a.K);
    bf16_t* wp = reinterpret_cast<bf16_t*>(ws);
    ws += up256(size_t(a.N) * ldw * 2);
    const hipError_t e = pad_rows(a.N, a.K, ldw, w, wp, stream);
    if (e != hipSuccess) return e;
    w = wp;
  }
  Product<bf16_t> g = {};
  g.A[0] = {w, ldw, 1, a.N};
  g.B[0] = {x, ldx, 1, a.M};
  g.K[0] = a.K;
  return product<kRows, kRows>(g, ldw % 8 != 0, linear_epi<bf16_t>(a), a.N, a.M, reinterpret_cast<float*>(ws), stream);
}

hipError_t linear_f32(const LinearArgs& a, hipStream_t stream) {
  Product<float> g = {};
  g.A[0] = {static_cast<const float*>(a.w), a.K, 1, a.N};
  g.B[0] = {static_cast<const float*>(a.x), a.K, 1, a.M};
  g.K[0] = a.K;
  return product<kRows, kRows>(g, false, linear_epi<float>(a), a.N, a.M, static_cast<float*>(a.ws), stream);
}

// dz and its chunk sums; `dz` (with its row length) is dy itself where no
// copy is needed.
template <typename T>
hipError_t make_dz(const LinearBackwardArgs& a, bool copy, long rows, const T** dz, long* ld, unsigned char** ws,
                   hipStream_t stream) {
  *dz = static_cast<const T*>(a.dy);
  *ld = a.N;
  float* part = reinterpret_cast<float*>(*ws);
  *ws += up256(size_t(dz_chunks(a.M)) * a.N * 4);
  T* out = nullptr;
  if (copy) {
    *ld = dz_stride(a.N);
    out = reinterpret_cast<T*>(*ws);
    *ws += up256(size_t(rows) * *ld * sizeof(T));
    *dz = out;
  }
  if (a.N == 0) return hipSuccess;
  // the grid's second axis holds 65535 chunks
  const int per = rows > 65535l * kDzRows ? 2 * kDzRows : a.dbias || rows > 65535l * 4 ? kDzRows : 4;
  if (rows > 0 && (copy || a.dbias))
    hipLaunchKernelGGL((dz_kernel<T>), dim3(unsigned((*ld + 1023) / 1024), unsigned((rows + per - 1) / per)),
                       dim3(256), 0, stream, a.M, int(rows), a.N, a.act, static_cast<const T*>(a.dy), a.pre, out, *ld,
                       a.dbias ? part : nullptr,
                       a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.pre) % 16 == 0, per);
  if (a.dbias)
    hipLaunchKernelGGL((dbias_kernel<T>), dim3(unsigned((a.N + 31) / 32)), dim3(256), 0, stream, a.N,
                       rows > 0 ? int((rows + per - 1) / per) : 0, part, static_cast<T*>(a.dbias));
  return hipGetLastError();
}

// The gradient's products through the same epilogue as the forward one,
// without bias, activation and residual.
template <typename T>
LinearEpi<T> plain_epi(void* out, int na) {
  LinearEpi<T> epi = {};
  epi.y = static_cast<T*>(out);
  epi.na = na;
  epi.vec = aligned4<T>(out, na);
  return epi;
}

// Whether dz is an array of its own: with an activation, or as bf16 b operand,
// which ends in zeros along both axes.  Otherwise it is dy itself.
bool copies_dz(int M, int N, bool act, bool bf16) { return act || (bf16 && (N % kStep != 0 || M % kStep != 0)); }

template <typename T>
hipError_t linear_backward_t(const LinearBackwardArgs& a, hipStream_t stream) {
  const T* dz;
  long ld;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  hipError_t e = make_dz(a, copies_dz(a.M, a.N, a.act != 0, a.bf16), a.bf16 ? up64(a.M) : long(a.M), &dz, &ld, &ws, stream);
  if (e != hipSuccess) return e;
  // the a operand, its rows copied where they are not aligned
  auto operand = [&](const void* p, int rows, int nb, const T** out, long* ld_out, float** part) {
    *out = static_cast<const T*>(p);
    *ld_out = a.K;
    *part = reinterpret_cast<float*>(ws);
    if constexpr (sizeof(T) == 2) {
      if (copies(rows, a.K, nb)) {
        bf16_t* copy = reinterpret_cast<bf16_t*>(ws);
        *out = copy;
        *ld_out = up64(a.K);
        *part = reinterpret_cast<float*>(ws + copy_bytes(rows, a.K, nb));
        return pad_rows(rows, a.K, *ld_out, static_cast<const bf16_t*>(p), copy, stream);
      }
    }
    return hipSuccess;
  };
  const T* A;
  long lda;
  float* part;
  if (a.dx && a.K > 0 && a.M > 0) {
    if ((e = operand(a.w, a.N, a.M, &A, &lda, &part)) != hipSuccess) return e;
    Product<T> g = {};
    g.A[0] = {A, 1, lda, a.K};
    g.B[0] = {dz, ld, 1, a.M};
    g.K[0] = a.N;
    if ((e = product<kCols, kRows>(g, lda % 8 != 0, plain_epi<T>(a.dx, a.K), a.K, a.M, part, stream)) != hipSuccess)
      return e;
  }
  if (a.dw && a.K > 0 && a.N > 0) {
    if ((e = operand(a.x, a.M, a.N, &A, &lda, &part)) != hipSuccess) return e;
    Product<T> g = {};
    g.A[0] = {A, 1, lda, a.K};
    g.B[0] = {dz, 1, ld, a.N};
    g.K[0] = a.M;
    if ((e = product<kCols, kCols>(g, lda % 8 != 0, plain_epi<T>(a.dw, a.K), a.K, a.N, part, stream)) != hipSuccess)
      return e;
  }
  return hipSuccess;
}

}  // namespace

size_t linear_workspace_bytes(int M, int N, int K, bool bf16) {
  if (bf16 && few_rows(M, N, K)) return 0;
  if (!bf16) return split_bytes(N, M, K, false, false, false);
  return (K % kStep ? up256(size_t(M) * up64(K) * 2) : 0) + copy_bytes(N, K, M) +
         split_bytes(N, M, K, true, stays_any(N, K, M), false);
}

size_t linear_backward_workspace_bytes(int M, int N, int K, bool bf16, bool act) {
  const size_t dz = up256(size_t(dz_chunks(M)) * N * 4) +
                    (copies_dz(M, N, act, bf16) ? up256(size_t(up64(M)) * dz_stride(N) * (bf16 ? 2 : 4)) : 0);
  // dx reads w, dw reads x, one after the other
  const size_t dx = (bf16 ? copy_bytes(N, K, M) : 0) + split_bytes(K, M, N, bf16, stays_any(N, K, M), true);
  const size_t dw = (bf16 ? copy_bytes(M, K, N) : 0) + split_bytes(K, N, M, bf16, stays_any(M, K, N), true);
  return dz + (dx > dw ? dx : dw);
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  return a.bf16 ? linear_bf16(a, stream) : linear_f32(a, stream);
}

hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t stream) {
  return a.bf16 ? linear_backward_t<bf16_t>(a, stream) : linear_backward_t<float>(a, stream);
}

}  // namespace dspark
