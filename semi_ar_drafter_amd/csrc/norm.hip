// Layer and root-mean-square normalisation of rows with the residual stream's
// sum, and its gradients.
//
//   s = x + residual,  y = (s - mu) rstd w + b            (rms: mu = 0)
//   with q = dy w and n = (s - mu) rstd:
//   ds = rstd (q - mean q - n mean(q n)) + dsum           (rms: without mean q)
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// Bound by memory (16384 x 5120 with a residual, in training: 271 us for 1.34 GB
// and 21 MB of shares, 5.0 TB/s; under the profiler 140 forward, 160 and 7
// backward; one row: 3.6 us, latency).  A row is read once and kept in registers
// as it is stored, 16 bytes a lane and load; its mean and the sum of squares around it are made
// wave by wave and joined in LDS (n_a, m_a, M_a with n_b, m_b, M_b: the squares
// around the joint mean are M_a + M_b + (m_a - m_b)^2 n_a n_b / (n_a + n_b)),
// so that no precision is lost to a mean that is large against the spread.
#include "launch.h"
#include "projection.h"

namespace dspark {

namespace {

// 16 bytes of a row, at element alignment.
template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  u32x4_t raw;
  __device__ __forceinline__ void load(const T* p, int n) {   // n values exist, zeros behind
    if (n >= N) {
      __builtin_memcpy(&raw, p, 16);
      return;
    }
    T e[N] = {};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) e[i] = p[i];
    __builtin_memcpy(&raw, e, 16);
  }
  // past: by the caches, which need not keep it
  __device__ __forceinline__ void store(T* p, int n, bool past) const {
    if (n >= N && past) {
      typedef uint32_t chunk_t __attribute__((ext_vector_type(4), aligned(2)));   // element alignment
      __builtin_nontemporal_store(chunk_t(raw), reinterpret_cast<chunk_t*>(p));
    } else if (n >= N) {
      __builtin_memcpy(p, &raw, 16);
    } else {
      T e[N];
      __builtin_memcpy(e, &raw, 16);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) p[i] = e[i];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(raw[i]);
    else return i & 1 ? bf16_hi(raw[i >> 1]) : bf16_lo(raw[i >> 1]);
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
    T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = from_f32<T>(v[i]);
    __builtin_memcpy(&raw, e, 16);
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

constexpr int kMaxWaves = 16;

// A barrier for what lies in LDS alone: loads on their way from memory stay there.
__device__ __forceinline__ void meet_lds() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#endif
}

// Where a thread works: `waves` waves to a row (whole workgroup) or one (ONE:
// every wave has rows of its own).
struct Place {
  int t, threads, wave, waves, unit, units;
};
template <bool ONE>
__device__ __forceinline__ Place place(int grid) {
  Place p;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = blockDim.x >> 6;
  p.t = ONE ? threadIdx.x & 63 : threadIdx.x;
  p.threads = ONE ? 64 : blockDim.x;
  p.wave = ONE ? 0 : w;
  p.waves = ONE ? 1 : n;
  p.unit = ONE ? blockIdx.x * n + w : blockIdx.x;
  p.units = ONE ? grid * n : grid;
  return p;
}

// NV chunks per thread, of at most MOST, cover a row.  sum: where x + residual goes (with a
// residual); stat: (mu, rstd) by row or null.
template <typename T, int NV, int MOST, bool ONE, bool CENTER>
__global__ __launch_bounds__(MOST) void norm_kernel(int M, int C, const T* x, const T* residual,
                                                    const T* __restrict__ w, const T* __restrict__ b, float eps, T* sum,
                                                    T* __restrict__ y, float2* __restrict__ stat, bool past) {
  constexpr int N = Chunk<T>::N;
  __shared__ float2 parts[2][kMaxWaves];
  const Place p = place<ONE>(gridDim.x);
  const float each = 1.f / float(C);
  int turn = 0;
  for (int row = p.unit; row < M; row += p.units, turn ^= 1) {
    Chunk<T> v[NV], r[NV];
    const size_t at = size_t(row) * C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.threads + p.t) * N;
      v[i].load(x + at + c, C - c);
    }
    if (residual) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * p.threads + p.t) * N;
        r[i].load(residual + at + c, C - c);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * p.threads + p.t) * N;
        float s[N];
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = v[i].get(e) + r[i].get(e);
        v[i].set(s);   // what is stored is what is normalised: the gradient reads it again
        if (c < C) v[i].store(sum + at + c, C - c, past);
      }
    }
    // this wave's values: their number, mean and squares around it
    float mean = 0.f, sq = 0.f;
    if (CENTER) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) mean += v[i].get(e);
      int mine = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) mine += min(max(C - (i * p.threads + p.wave * 64) * N, 0), 64 * N);
      mean = wave_sum(mean);
      mean = mine ? mean / float(mine) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = C - (i * p.threads + p.t) * N;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = v[i].get(e) - mean;
        sq += e < left ? d * d : 0.f;
      }
    }
    sq = wave_sum(sq);
    if (!ONE) {
      if (p.t % 64 == 0) parts[turn][p.wave] = make_float2(mean, sq);
      __syncthreads();
      float n = 0.f;
      mean = sq = 0.f;
      for (int k = 0; k < p.waves; ++k) {
        const float2 o = parts[turn][k];
        if (CENTER) {
          int has = 0;
#pragma unroll
          for (int i = 0; i < NV; ++i) has += min(max(C - (i * p.threads + k * 64) * N, 0), 64 * N);
          const float m = float(has), both = n + m;
          if (has) {
            const float d = o.x - mean;
            sq += o.y + d * d * (n * m / both);
            mean += d * (m / both);
            n = both;
          }
        } else {
          sq += o.y;
        }
      }
    }
    const float rstd = 1.f / sqrtf(sq * each + eps);
    if (stat && p.t == 0) stat[row] = make_float2(mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.threads + p.t) * N;
      if (c >= C) continue;
      Chunk<T> cw, cb, o;
      if (w) cw.load(w + c, C - c);
      if (b) cb.load(b + c, C - c);
      float s[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s[e] = (v[i].get(e) - mean) * rstd;
        if (w) s[e] *= cw.get(e);
        if (b) s[e] += cb.get(e);
      }
      o.set(s);
      o.store(y + at + c, C - c, past);
    }
  }
}

// dw and db of 32 channels from all rows, by one workgroup: its threads take
// every (threads / 32)-th row of a channel, in four sums in turn (one sum of 42
// rows was off by 1.4e-7 of the gradient's norm in fp32, with four it is 0.9e-7),
// joined in order.
template <typename T>
__device__ __forceinline__ void columns(int first, int M, int C, const T* __restrict__ dy, const T* __restrict__ x,
                                        const float2* __restrict__ stat, T* dw, T* db) {
  __shared__ float2 sums[32][33];
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5, parts = blockDim.x >> 5, c = first + l;
  float fw[4] = {}, fb[4] = {};
  if (c < C) {
    auto add = [&](int i, int row) {
      const size_t at = size_t(row) * C + c;
      const float2 st = stat[row];
      const float g = to_f32(dy[at]);
      fw[i] = fmaf(g, (to_f32(x[at]) - st.x) * st.y, fw[i]);
      fb[i] += g;
    };
    int row = q;
    for (; row + 7 * parts < M; row += 8 * parts) {
#pragma unroll
      for (int i = 0; i < 8; ++i) add(i & 3, row + i * parts);
    }
    for (; row < M; row += 4 * parts) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i * parts < M) add(i, row + i * parts);
    }
  }
  float sw = (fw[0] + fw[1]) + (fw[2] + fw[3]), sb = (fb[0] + fb[1]) + (fb[2] + fb[3]);
  sums[q][l] = make_float2(sw, sb);
  __syncthreads();
  if (q == 0 && c < C) {
    for (int i = 1; i < parts; ++i) {
      sw += sums[i][l].x;
      sb += sums[i][l].y;
    }
    if (dw) dw[c] = from_f32<T>(sw);
    if (db) db[c] = from_f32<T>(sb);
  }
}

// Each unit (a workgroup, or ONE: a wave) goes through its rows and keeps its
// share of dw and db in registers: part[unit][0 and 1][C].  The next row's
// loads are sent off before this one's sums, and nothing else is loaded in
// between (loads come back in order): the weights stay in registers.  With
// few rows dw and db are made beside dx, by workgroups of their own.
template <typename T, int NV, int MOST, bool ONE, bool CENTER>
__global__ __launch_bounds__(MOST) void norm_backward_kernel(
    int M, int C, const T* __restrict__ dy, const T* __restrict__ x, const float2* __restrict__ stat,
    const T* __restrict__ w, const T* dsum, T* dx, float* __restrict__ part, int rows_grid, T* dw_out, T* db_out,
    bool past) {
  constexpr int N = Chunk<T>::N;
  if (int(blockIdx.x) >= rows_grid) {   // the workgroups behind those of the rows, if any, take channels
    columns((int(blockIdx.x) - rows_grid) * 32, M, C, dy, x, stat, dw_out, db_out);
    return;
  }
  // 1024 threads have 128 registers each, which hold no second row of bf16
  constexpr bool AHEAD = NV <= 2 && (MOST <= 512 || sizeof(T) == 4);
  __shared__ float2 parts[2][kMaxWaves];
  const Place p = place<ONE>(rows_grid);
  const float each = 1.f / float(C);
  float dw[NV][N] = {}, db[NV][N] = {};
  Chunk<T> cw[NV], v[NV], g[NV], d[NV];
  float2 st;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * p.threads + p.t) * N;
    if (w) {
      cw[i].load(w + c, C - c);
    } else {
      float one[N];
#pragma unroll
      for (int e = 0; e < N; ++e) one[e] = 1.f;
      cw[i].set(one);
    }
  }
  auto load = [&](int row) {
    const size_t at = size_t(row) * C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.threads + p.t) * N;
      v[i].load(x + at + c, C - c);
      g[i].load(dy + at + c, C - c);
      if (dsum && dx) d[i].load(dsum + at + c, C - c);
    }
    st = stat[row];
  };
  int turn = 0;
  if (AHEAD && p.unit < M) load(p.unit);
  for (int row = p.unit; row < M; row += p.units, turn ^= 1) {
    if (!AHEAD) load(row);
    float sq = 0.f, sn = 0.f;   // sums of q and of q n
    float n[AHEAD ? NV : 1][N], q[AHEAD ? NV : 1][N];   // (else made again)
    Chunk<T> ds[NV];
    const float mean = st.x, rstd = st.y;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.threads + p.t) * N;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float gy = g[i].get(e), ni = (v[i].get(e) - mean) * rstd, qi = gy * cw[i].get(e);
        if (AHEAD) {
          n[i][e] = ni;
          q[i][e] = qi;
        }
        sq += qi;
        if (c + e < C) sn += qi * ni;   // behind the end n is not 0
        dw[i][e] += gy * ni;
        db[i][e] += gy;
      }
      ds[i] = d[i];
    }
    if (AHEAD && row + p.units < M) load(row + p.units);
    if (!dx) continue;   // for all threads alike
    if (CENTER) sq = wave_sum(sq);
    sn = wave_sum(sn);
    if (!ONE) {
      if (p.t % 64 == 0) parts[turn][p.wave] = make_float2(sq, sn);
      meet_lds();
      sq = sn = 0.f;
      for (int k = 0; k < p.waves; ++k) {
        const float2 o = parts[turn][k];
        sq += o.x;
        sn += o.y;
      }
    }
    sq = CENTER ? sq * each : 0.f;
    sn *= each;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * p.threads + p.t) * N;
      if (c >= C) continue;
      Chunk<T> o;
      float s[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float ni = AHEAD ? n[i][e] : (v[i].get(e) - mean) * rstd;
        const float qi = AHEAD ? q[i][e] : g[i].get(e) * cw[i].get(e);
        s[e] = rstd * (qi - sq - ni * sn);
        if (dsum) s[e] += ds[i].get(e);
      }
      o.set(s);
      o.store(dx + size_t(row) * C + c, C - c, past);
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * p.threads + p.t) * N;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < C) {
        part[(size_t(p.unit) * 2) * C + c + e] = dw[i][e];
        part[(size_t(p.unit) * 2 + 1) * C + c + e] = db[i][e];
      }
  }
}

// dw and db (grid y: which): the units' shares, eight threads per column,
// joined in order.
template <typename T>
__global__ __launch_bounds__(256) void norm_join_kernel(int C, int units, const float* __restrict__ part, T* dw, T* db) {
  __shared__ float sums[8][32];
  T* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int u = q; u < units; u += 8) s += part[(size_t(u) * 2 + blockIdx.y) * C + c];
  }
  sums[q][l] = s;
  __syncthreads();
  if (q == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][l];
    out[c] = from_f32<T>(s);
  }
}

// Launch shape: threads per workgroup, chunks per thread, whether a wave has
// rows of its own, workgroups.  Where these leave shares of dw and db (shares),
// two workgroups stay on each compute unit and go through the rows (16384 x
// 5120: 152 us so and 7 us for joining, with 1024 workgroups 167 and 13, with
// 768 160 and 10), and fewer with fewer rows, whose shares would be as long as
// the rows themselves (1024 x 5120, forward and backward: 39 us with 128, 46
// with 512).
struct Shape {
  int threads, nv;
  bool one;
  int grid, units;
};
Shape shape_for(int M, int C, bool bf16, bool shares) {
  const int chunks = (C + (bf16 ? 8 : 4) - 1) / (bf16 ? 8 : 4);
  Shape s;
  s.one = chunks <= 64;
  s.nv = chunks <= 512 ? 1 : chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
  s.threads = s.one ? 256 : (chunks + s.nv - 1) / s.nv;
  s.threads = (s.threads + 63) / 64 * 64;
  const int rows = s.one ? 4 : 1, groups = (M + rows - 1) / rows;
  const int most = !shares ? 8192 : groups >= 4096 ? 512 : groups >= 1024 ? groups / 8 : 128;
  s.grid = groups < most ? groups : most;
  s.units = s.grid * rows;
  return s;
}

// Whether the rows written go by the caches: many of them would only drive out
// what is in there (forward, us with and without: 16384 x 4096 104 against 129,
// 1024 x 4096 9.1 and 10.9, and 14.9 and 15.8 with a kernel that reads them next;
// 256 x 4096 with one 7.7 and 7.5).
bool past_caches(int M, int C, size_t elem) { return size_t(M) * C * elem >= size_t(4) << 20; }

// go(the kernel of this shape)
#define DSPARK_NORM_SHAPES(kernel, T, CENTER, s, go)                                 \
  (s.one              ? go(kernel<T, 1, 512, true, CENTER>)                          \
   : s.nv == 1        ? go(kernel<T, 1, 512, false, CENTER>)                         \
   : s.nv == 2 && s.threads <= 512 ? go(kernel<T, 2, 512, false, CENTER>)            \
   : s.nv == 2        ? go(kernel<T, 2, 1024, false, CENTER>)                        \
   : s.nv == 4        ? go(kernel<T, 4, 1024, false, CENTER>)                        \
                      : go(kernel<T, sizeof(T) == 4 ? 8 : 4, 1024, false, CENTER>))

template <typename T, bool CENTER>
hipError_t norm_t(const NormArgs& a, hipStream_t stream) {
  const Shape s = shape_for(a.M, a.C, sizeof(T) == 2, false);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(s.grid), dim3(s.threads), 0, stream, a.M, a.C, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.residual), static_cast<const T*>(a.w), static_cast<const T*>(a.b), a.eps,
                       static_cast<T*>(a.sum), static_cast<T*>(a.y), reinterpret_cast<float2*>(a.stat),
                       past_caches(a.M, a.C, sizeof(T)));
    return hipGetLastError();
  };
  return DSPARK_NORM_SHAPES(norm_kernel, T, CENTER, s, go);
}

// Whether dw and db are made beside dx in one launch, from the inputs again,
// instead of from shares in a second one (forward and backward, us, bf16: 64 x
// 64 6.7 against 9.0, 128 x 2560 7.8 and 13.1, 512 x 1001 12.8 and 14.9, 512 x
// 5120 18.6 and 24.2, 512 x 32768 181 and 190, 1024 x 256 14.9 and 14.0, 1024 x
// 32768 390 and 374; fp32: 512 x 1001 10.4 and 14.2, 512 x 5120 20.9 and 23.5, 1024
// x 2560 28.1 and 23.7; only fp32 rows of 16384 channels and more lose at 512, 74
// and 70).
bool beside(int M) { return M <= 512; }

template <typename T, bool CENTER>
hipError_t norm_backward_t(const NormBackwardArgs& a, hipStream_t stream) {
  const bool sums = a.dw || a.db, one = sums && a.M > 0 && beside(a.M);
  const Shape s = shape_for(a.M, a.C, sizeof(T) == 2, sums && !one);
  float* part = sums && !one ? static_cast<float*>(a.ws) : nullptr;
  const int rows_grid = one && !a.dx ? 0 : s.grid, grid = rows_grid + (one ? (a.C + 31) / 32 : 0);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(s.threads), 0, stream, a.M, a.C, static_cast<const T*>(a.dy),
                       static_cast<const T*>(a.x), reinterpret_cast<const float2*>(a.stat), static_cast<const T*>(a.w),
                       static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), part, rows_grid, static_cast<T*>(a.dw),
                       static_cast<T*>(a.db), past_caches(a.M, a.C, sizeof(T)));
    return hipGetLastError();
  };
  hipError_t e = hipSuccess;
  if (a.M > 0) e = DSPARK_NORM_SHAPES(norm_backward_kernel, T, CENTER, s, go);
  if (e != hipSuccess || !sums || one) return e;
  hipLaunchKernelGGL((norm_join_kernel<T>), dim3((a.C + 31) / 32, 2), dim3(256), 0, stream, a.C, a.M > 0 ? s.units : 0,
                     part, static_cast<T*>(a.dw), static_cast<T*>(a.db));
  return hipGetLastError();
}

}  // namespace

size_t norm_backward_workspace_bytes(int M, int C, bool bf16) {
  if (beside(M)) return 0;
  const size_t n = size_t(shape_for(M, C, bf16, true).units) * 2 * C * 4;
  return (n + 255) & ~size_t(255);
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.bf16) return a.center ? norm_t<bf16_t, true>(a, stream) : norm_t<bf16_t, false>(a, stream);
  return a.center ? norm_t<float, true>(a, stream) : norm_t<float, false>(a, stream);
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
  if (a.bf16) return a.center ? norm_backward_t<bf16_t, true>(a, stream) : norm_backward_t<bf16_t, false>(a, stream);
  return a.center ? norm_backward_t<float, true>(a, stream) : norm_backward_t<float, false>(a, stream);
}

}  // namespace dspark
