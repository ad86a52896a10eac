// Softmax cross entropy over the drafting heads' logits, without keeping the
// logits, and its gradient.
//
//   z_n(v) = U[n][v] + h_n . Wo[v] + W1[prev_n] . W2[:, v]
//   lse_n  = ln sum_v exp z_n(v),  nll_n = lse_n - z_n(label_n)
//   dz_n(v) = g_n (exp(z_n(v) - lse_n) - [v = label_n])
//
// Rows without a label are left out at the start: the rows that have one are
// gathered into X = [h | W1[prev]] (both parts zero-padded to a multiple of
// 64), so that ignored rows cost no product and whatever they hold touches
// nothing.  Their number stays on the device.
//
// Forward: the product of X with [Wo | W2^T] tile by tile; each tile leaves
// (max, sum of exponentials) per row, which one small kernel joins.
// Backward, piece by piece of the vocabulary (the piece's dz is the only
// array of its width that is kept): logits again, dz, then
//   dX += dz [Wo | W2^T]     (fp32, over the pieces in order)
//   dWo = dz^T h,  dW2 = e^T dz    (final: rows are not split)
// and at the end dX is rounded into dh and summed into dW1, rows with the
// same previous token in four interleaved sums, each in row order.  Nothing is
// added by atomics: results do not depend on any order of execution.
//
// Bound by: the matrix unit with many rows (4096 rows, V = 151936, d = 5120, r
// = 256: four products of 4.9 to 5.4 ms, 1.2 PFLOP/s), reading Wo and W2 with
// few (8 rows, d = 2560: 143 us, 6.0 TB/s), the tiles' ends where the
// contraction is short (rank 256 alone: 770 us for the statistics of 4096 rows,
// of which four steps' MFMAs are 150).
#include "launch.h"
#include "projection.h"
#include "tile_bf16.h"
#include "tile_f32.h"

namespace dspark {

namespace {

inline size_t up(size_t x, size_t m) { return (x + m - 1) / m * m; }

// Most bytes of a piece's dz array.  Larger pieces mean fewer, fuller rounds of
// tiles and fewer passes over dX (4096 rows, V = 151936, rank 256 alone / with d
// = 5120: 128 MB 3.57 / 22.6 ms, 256 MB 3.28 / 22.2, 512 MB 3.14 / 21.8); the
// logits themselves would be 1.2 GB in bf16.
constexpr size_t kPieceBytes = size_t(512) << 20;
constexpr int kPieceAlign = 256;
constexpr int kLeastTile = 64;   // along the vocabulary

// Lists the rows that have a label, in order: row[i] = n, place[n] = i or -1.
// One workgroup; each thread takes a run of rows.
__global__ __launch_bounds__(1024) void compact_kernel(int N, int V, const int* __restrict__ label,
                                                       int* __restrict__ count, int* __restrict__ row,
                                                       int* __restrict__ place) {
  __shared__ int sums[1024];
  const int tid = threadIdx.x;
  const int per = (N + 1023) / 1024;
  const int lo = min(N, tid * per), hi = min(N, lo + per);
  int c = 0;
  for (int n = lo; n < hi; ++n) c += unsigned(label[n]) < unsigned(V);
  sums[tid] = c;
  __syncthreads();
  for (int s = 1; s < 1024; s *= 2) {
    const int o = tid >= s ? sums[tid - s] : 0;
    __syncthreads();
    sums[tid] += o;
    __syncthreads();
  }
  int at = sums[tid] - c;
  for (int n = lo; n < hi; ++n) {
    const bool used = unsigned(label[n]) < unsigned(V);
    place[n] = used ? at : -1;
    if (used) row[at++] = n;
  }
  if (tid == 1023) *count = sums[1023];
}

// What the products' epilogues need of every row in use, by compact row.
struct RowData {
  const int* label_in;
  const float *lse_in, *g_in;   // of the gradient only
  int *label, *token;
  float *lse, *g;
};

constexpr int kCountRows = 8192;   // up to so many rows, prepare_kernel counts for itself
constexpr int kFillBytes = 256 * 16 * 8;   // zeros per workgroup of prepare_kernel

template <typename T>
struct PrepareArgs {
  int N, V, d, dp, r, rp;
  int *count, *row, *place;
  const int* prev;
  const T *h, *W1;
  T* X;
  RowData rows;
  T* dU;          // rows without a label get zeros (nullptr: no dU)
  T* dz;          // rows from count to the next multiple of 64 get zeros (nullptr: none)
  long width;     // of dz
  T* dW1;         // cleared (nullptr: none)
  size_t dW1_n;
  bool counted;   // compact_kernel has filled count, row and place
};

__device__ __forceinline__ int labels_in(const int* label, int n, int V, int* sums) {
  int c = 0;
  for (int i = threadIdx.x; i < n; i += 256) c += unsigned(label[i]) < unsigned(V);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) c += __shfl_xor(c, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = c;
  __syncthreads();
  return sums[0] + sums[1] + sums[2] + sums[3];
}

// A workgroup's share of zeros from p on, n values: 16 bytes at a time where
// they are aligned.
template <typename T>
__device__ __forceinline__ void fill_share(T* p, size_t n, int part, int parts) {
  const size_t per = (n + parts - 1) / parts, at = ((per + 15) & ~size_t(15)) * part;
  const size_t end = min(n, at + ((per + 15) & ~size_t(15)));
  if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    constexpr int V = 16 / sizeof(T);
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    for (size_t i = at + size_t(threadIdx.x) * V; i + V <= end; i += 256 * V) *reinterpret_cast<u32x4_t*>(p + i) = zero;
    for (size_t i = (end > at ? at + (end - at) / V * V : end) + threadIdx.x; i < end; i += 256) p[i] = from_f32<T>(0.f);
  } else {
    for (size_t i = at + threadIdx.x; i < end; i += 256) p[i] = from_f32<T>(0.f);
  }
}

// All that comes before the products, in one launch.  Workgroup n < N: row n
// takes its place i among the rows in use (their number before it) and writes
// X[i] = [h[n] | 0 | W1[prev[n]] | 0] and the row's label, token, lse and g;
// the next 64: rows of X from count up to the next multiple of 64 are zero;
// the rest: zeros elsewhere.
template <typename T>
__global__ __launch_bounds__(256) void prepare_kernel(PrepareArgs<T> p) {
  __shared__ int sums[4];
  const int n = blockIdx.x, tid = threadIdx.x;
  const T zero = from_f32<T>(0.f);
  if (n < p.N) {
    const int y = p.rows.label_in[n];
    const bool used = unsigned(y) < unsigned(p.V);
    int i;
    if (p.counted) {
      i = p.place[n];
    } else {
      i = labels_in(p.rows.label_in, n, p.V, sums);
      if (tid == 0) {
        p.place[n] = used ? i : -1;
        if (used) p.row[i] = n;
        if (n == p.N - 1) *p.count = i + used;
      }
    }
    if (!used) {
      if (p.dU) {
        T* u = p.dU + size_t(n) * p.V;
        for (int v = tid; v < p.V; v += 256) u[v] = zero;
      }
      return;
    }
    if (tid == 0) {
      p.rows.label[i] = y;
      if (p.rows.lse_in) {
        p.rows.lse[i] = p.rows.lse_in[n];
        p.rows.g[i] = p.rows.g_in[n];
      }
    }
    T* x = p.X + size_t(i) * (p.dp + p.rp);
    const T* hr = p.h + size_t(n) * p.d;
    for (int c = tid; c < p.dp; c += 256) x[c] = c < p.d ? hr[c] : zero;
    if (p.rp) {
      const int t = min(max(p.prev[n], 0), p.V - 1);
      if (tid == 0) p.rows.token[i] = t;
      const T* wr = p.W1 + size_t(t) * p.r;
      for (int c = tid; c < p.rp; c += 256) x[p.dp + c] = c < p.r ? wr[c] : zero;
    }
    return;
  }
  const int total = p.counted ? *p.count : labels_in(p.rows.label_in, p.N, p.V, sums);
  const int end = (total + 63) & ~63;
  if (n < p.N + 64) {
    const int i = total + n - p.N;
    if (i >= end) return;
    T* x = p.X + size_t(i) * (p.dp + p.rp);
    for (int c = tid; c < p.dp + p.rp; c += 256) x[c] = zero;
    return;
  }
  const int part = n - p.N - 64, parts = gridDim.x - p.N - 64;
  if (p.dz) fill_share(p.dz + size_t(total) * p.width, size_t(end - total) * p.width, part, parts);
  if (p.dW1) fill_share(p.dW1, p.dW1_n, part, parts);
}

// lse and nll of every row from the tiles' statistics, in a fixed order: LANES
// threads per row, each taking every LANES-th tile, then joined pairwise.
template <int LANES>
__global__ __launch_bounds__(256) void join_kernel(int N, int tiles, const int* __restrict__ place,
                                                   const float2* __restrict__ stat, long stat_ld,
                                                   const float* __restrict__ zlab, float* __restrict__ nll,
                                                   float* __restrict__ lse) {
  constexpr int ROWS = 256 / LANES;   // neighbouring threads take neighbouring rows
  __shared__ float2 part[256];
  const int n = blockIdx.x * ROWS + threadIdx.x % ROWS, first = threadIdx.x / ROWS;
  const int i = n < N ? place[n] : -1;
  const float ninf = -__builtin_huge_valf();
  float m = ninf, s = 0.f;
  if (i >= 0) {
#pragma unroll 4
    for (int t = first; t < tiles; t += LANES) {
      const float2 q = stat[size_t(t) * stat_ld + i];
      const float top = fmaxf(m, q.x), ref = top == ninf ? 0.f : top;
      s = s * __expf(m - ref) + q.y * __expf(q.x - ref);
      m = top;
    }
  }
  part[threadIdx.x] = make_float2(m, s);
  for (int x = LANES / 2; x >= 1; x /= 2) {
    __syncthreads();
    if (first < x) {
      const float2 o = part[threadIdx.x + x * ROWS];
      const float top = fmaxf(m, o.x), ref = top == ninf ? 0.f : top;
      s = s * __expf(m - ref) + o.y * __expf(o.x - ref);
      m = top;
      part[threadIdx.x] = make_float2(m, s);
    }
  }
  if (n < N && first == 0) {
    // nll from the maximum, not from the rounded lse: where the label has
    // the maximum, what is left is log(s) to its own accuracy
    const float l = logf(s);
    lse[n] = i >= 0 ? m + l : 0.f;
    nll[n] = i >= 0 ? (m - zlab[i]) + l : 0.f;
  }
}

// dh[n] = the row's sum over splits, in order; zero for rows without a label.
template <typename T>
__device__ __forceinline__ void dh_row(int n, int d, long ld, int splits, long split, const int* place,
                                       const float* dX, T* dh) {
  const int i = place[n];
  // the grid's second axis takes turns at the columns
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < d; c += blockDim.x * gridDim.y) {
    float v = 0.f;
    if (i >= 0) {
#pragma unroll 8
      for (int s = 0; s < splits; ++s) v += dX[size_t(s) * split + size_t(i) * ld + c];
    }
    dh[size_t(n) * d + c] = from_f32<T>(v);
  }
}

// Workgroup n < N: dh[n] (if asked for); the others: dE of every row in use,
// its splits, in order, into the first one's place.
template <typename T>
__global__ __launch_bounds__(256) void join_rows_kernel(int N, int d, long ld_h, int splits_h, long split_h,
                                                        const int* __restrict__ place, const float* __restrict__ dX,
                                                        T* __restrict__ dh, long ld, int splits, long split,
                                                        const int* __restrict__ count, float* __restrict__ dE) {
  if (int(blockIdx.x) < N) {
    if (dh) dh_row(blockIdx.x, d, ld_h, splits_h, split_h, place, dX, dh);
    return;
  }
  const int i = blockIdx.x - N;
  if (i >= *count) return;
  for (int c = blockIdx.y * 256 + threadIdx.x; c < ld; c += 256 * gridDim.y) {
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += dE[size_t(s) * split + size_t(i) * ld + c];
    dE[size_t(i) * ld + c] = v;
  }
}

// dW1[t] = sum of dE over the rows whose previous token is t.  One workgroup
// per row; the token's first row does the sum (the table was zeroed before).
// Its rows are listed in LDS, kSegment rows at a time, and added in four
// interleaved sums (a frequent token has hundreds of rows: their loads are
// all independent), joined in order.  A second run of N workgroups does dh.
constexpr int kSegment = 2048;
template <typename T>
__global__ __launch_bounds__(1024) void dw1_kernel(int N, int r, long ld, const int* __restrict__ count,
                                                   const int* __restrict__ token, const float* __restrict__ dE,
                                                   T* __restrict__ dW1, int d, long ld_h, int splits_h, long split_h,
                                                   const int* __restrict__ place, const float* __restrict__ dX,
                                                   T* __restrict__ dh) {
  if (int(blockIdx.x) >= N) {
    dh_row(blockIdx.x - N, d, ld_h, splits_h, split_h, place, dX, dh);
    return;
  }
  __shared__ int list[kSegment];
  __shared__ int found, waves[16];
  __shared__ float sums[1024];
  const int i = blockIdx.x, n = *count, tid = threadIdx.x, lane = tid & 63;
  if (i >= n) return;
  const int t = token[i];
  if (tid == 0) found = 0;
  __syncthreads();
  bool earlier = false;
  for (int j = tid; j < i; j += 1024) earlier |= token[j] == t;
  if (earlier) found = 1;
  __syncthreads();
  if (found) return;
  const int c = tid & 255, phase = tid >> 8;
  for (int c0 = 0; c0 < r; c0 += 256) {
    float s = 0.f;
    for (int j0 = i; j0 < n; j0 += kSegment) {
      int len = 0;   // the segment's rows with this token, in order
      for (int half = 0; half < kSegment / 1024; ++half) {
        const int j = j0 + half * 1024 + tid;
        const bool same = j < n && token[j] == t;
        const uint64_t mask = __ballot(same);
        __syncthreads();
        if (lane == 0) waves[tid >> 6] = __builtin_popcountll(mask);
        __syncthreads();
        int before = len;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          if (w < (tid >> 6)) before += waves[w];
          len += waves[w];
        }
        if (same) list[before + __builtin_popcountll(mask & ((1ull << lane) - 1))] = j;
      }
      __syncthreads();
      if (c0 + c < r) {
#pragma unroll 4
        for (int q = phase; q < len; q += 4) s += dE[size_t(list[q]) * ld + c0 + c];
      }
    }
    __syncthreads();
    sums[tid] = s;
    __syncthreads();
    if (tid < 256 && c0 + c < r)
      dW1[size_t(t) * r + c0 + c] = from_f32<T>((sums[c] + sums[256 + c]) + (sums[512 + c] + sums[768 + c]));
  }
}

// What the forward and the backward call carve out of the workspace.
struct Layout {
  size_t row, place, token, label, lse, g, X, W2, Wo, stat, zlab, dz, dXh, dXe, total;
  int dp, rp, rows, width;   // padded parts of X, padded rows, width of a piece
  long w2_ld, wo_ld;         // row lengths of W2 and Wo as the products read them
  bool any;                  // rows of Wo are not 16-byte aligned
  Plan h, e;                 // of the contractions over a piece's tokens
};

Layout layout(int N, int V, int d, int r, bool bf16, bool backward) {
  const size_t elem = bf16 ? 2 : 4;
  Layout L = {};
  L.dp = int(up(d, 64));
  L.rp = int(up(r, 64));
  L.rows = int(up(N > 0 ? N : 1, 256));
  size_t at = 256;   // count
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += up(bytes, 256);
    return p;
  };
  L.row = take(size_t(N) * 4);
  L.place = take(size_t(N) * 4);
  L.token = take(size_t(N) * 4);
  L.label = take(size_t(N) * 4);
  if (backward) {
    L.lse = take(size_t(N) * 4);
    L.g = take(size_t(N) * 4);
  }
  L.X = take(size_t(L.rows) * (L.dp + L.rp) * elem);
  L.w2_ld = V;
  if (bf16 && r && V % 8) {
    L.w2_ld = long(up(V, 64));
    L.W2 = take(size_t(r) * L.w2_ld * 2);
  }
  L.wo_ld = d;
  // The copy reads and writes what the product reads once more: worth it where
  // that product has few tiles, each with many steps, or many rows (forward /
  // with all gradients, us, copied against not: 24 rows, V = 1088, d = 3535 40
  // against 60 / 72 against 90; 1024 rows, V = 50021, d = 601 126 against 133 /
  // 424 against 444; but 24 rows, V = 50021, d = 601 45 against 29 / 134 against
  // 124, and 333 rows 72 against 66 / 244 against 234).
  if (bf16 && d % 8 && d >= 256 && (V <= 8192 || N > 512) && size_t(V) * L.dp * 2 <= kCopyBytes) {
    L.wo_ld = L.dp;
    L.Wo = take(size_t(V) * L.dp * 2);
  }
  L.any = bf16 && L.wo_ld % 8 != 0;
  if (!backward) {
    L.stat = take((size_t(V) + kLeastTile - 1) / kLeastTile * N * sizeof(float2));
    L.zlab = take(size_t(N) * 4);
  } else {
    const size_t full = up(V, kPieceAlign);
    const size_t most = kPieceBytes / (size_t(L.rows) * elem);
    const size_t pieces = most >= full ? 1 : (full + (most ? most : 1) - 1) / (most ? most : 1);
    L.width = int(up((full + pieces - 1) / pieces, kPieceAlign));
    auto plan = [&](int na, bool any, bool cols) {
      if (!na || !N) return Plan{0, 1};
      return bf16 ? plan_for(na, N, L.width, any, cols, true) : Plan{0, f32_splits(na, N, L.width)};
    };
    L.h = plan(d, L.any, true);
    L.e = plan(r, false, false);
    L.dz = take(size_t(L.rows) * L.width * elem);
    L.dXh = take(size_t(L.h.splits) * L.rows * L.dp * 4);
    L.dXe = take(size_t(L.e.splits) * L.rows * L.rp * 4);
  }
  L.total = at;
  return L;
}

template <typename T>
struct Parts {
  Layout L;
  int *count, *row, *place;
  RowData rows;
  T* X;
  const T *W2, *Wo;
  int kx;
};

template <typename T>
hipError_t start(const LossArgs& a, const Layout& L, Parts<T>& p, PrepareArgs<T> pre, hipStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  p.L = L;
  p.count = reinterpret_cast<int*>(ws);
  p.row = reinterpret_cast<int*>(ws + L.row);
  p.place = reinterpret_cast<int*>(ws + L.place);
  p.rows.label_in = a.label;
  p.rows.lse_in = a.lse_in;
  p.rows.g_in = a.g;
  p.rows.label = reinterpret_cast<int*>(ws + L.label);
  p.rows.token = reinterpret_cast<int*>(ws + L.token);
  p.rows.lse = reinterpret_cast<float*>(ws + L.lse);
  p.rows.g = reinterpret_cast<float*>(ws + L.g);
  p.X = reinterpret_cast<T*>(ws + L.X);
  p.W2 = static_cast<const T*>(a.W2);
  p.kx = L.dp + L.rp;
  const size_t fills = (pre.dW1 ? pre.dW1_n * sizeof(T) : 0) + (pre.dz ? size_t(64) * pre.width * sizeof(T) : 0);
  size_t parts = (fills + kFillBytes - 1) / kFillBytes;
  if (parts > 2048) parts = 2048;
  pre.N = a.N;
  pre.V = a.V;
  pre.d = a.d;
  pre.dp = L.dp;
  pre.r = a.r;
  pre.rp = L.rp;
  pre.count = p.count;
  pre.row = p.row;
  pre.place = p.place;
  pre.prev = a.prev;
  pre.h = static_cast<const T*>(a.h);
  pre.W1 = static_cast<const T*>(a.W1);
  pre.X = p.X;
  pre.rows = p.rows;
  pre.counted = a.N > kCountRows || a.N == 0;
  if (pre.counted)
    hipLaunchKernelGGL(compact_kernel, dim3(1), dim3(1024), 0, stream, a.N, a.V, a.label, p.count, p.row, p.place);
  hipLaunchKernelGGL((prepare_kernel<T>), dim3(unsigned(a.N + 64 + parts)), dim3(256), 0, stream, pre);
  p.Wo = static_cast<const T*>(a.Wo);
  hipError_t e = hipGetLastError();
  if constexpr (sizeof(T) == 2) {
    if (e == hipSuccess && L.W2) {
      bf16_t* copy = reinterpret_cast<bf16_t*>(ws + L.W2);
      p.W2 = copy;
      e = pad_rows(a.r, a.V, L.w2_ld, static_cast<const bf16_t*>(a.W2), copy, stream);
    }
    if (e == hipSuccess && L.Wo) {
      bf16_t* copy = reinterpret_cast<bf16_t*>(ws + L.Wo);
      p.Wo = copy;
      e = pad_rows(a.V, a.d, L.wo_ld, static_cast<const bf16_t*>(a.Wo), copy, stream);
    }
  }
  return e;
}

// The logits of tokens [v0, v0 + nv) as a product.
template <typename T>
Product<T> logits(const LossArgs& a, const Parts<T>& p, int v0, int nv) {
  Product<T> g = {};
  g.B[0] = g.B[1] = {p.X, p.kx, 1, p.L.rows};
  if (a.d) {
    g.A[0] = {p.Wo + size_t(v0) * p.L.wo_ld, p.L.wo_ld, 1, nv};
    g.K[0] = a.d;
  }
  if (a.r) {
    g.A[1] = {p.W2 + v0, 1, p.L.w2_ld, nv};
    g.B[1].p = p.X + p.L.dp;
    g.K[1] = a.r;
  }
  g.nb = p.count;
  return g;
}

template <typename T>
BaseLogits<T> base_logits(const LossArgs& a, const Parts<T>& p, int v0, int nv, const void* dU) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.U) | reinterpret_cast<uintptr_t>(dU);
  return {static_cast<const T*>(a.U), p.row, a.V, v0, nv, a.V % 4 == 0 && at % (4 * sizeof(T)) == 0};
}

// One product by the storage type: bf16 on the bf16 matrix instruction
// (layouts of the operands given), fp32 on the fp32 one.  make(shape) gives
// the epilogue; any: rows of the a operand are not 16-byte aligned.
template <int LA0, int LA1, int LB, class Make>
hipError_t multiply(const Product<bf16_t>& g, bool any, const Make& make, int na, int nb, Plan plan,
                    hipStream_t stream) {
  return any ? launch_bf16<LA0, LA1, LB, true>(g, make, na, nb, plan, stream)
             : launch_bf16<LA0, LA1, LB, false>(g, make, na, nb, plan, stream);
}
template <int LA0, int LA1, int LB, class Make>
hipError_t multiply(const Product<float>& g, bool, const Make& make, int na, int nb, Plan plan,
                    hipStream_t stream) {
  return launch_f32(g, make, na, nb, plan.splits, stream);
}

template <typename T>
hipError_t loss_t(const LossArgs& a, hipStream_t stream) {
  const Layout L = layout(a.N, a.V, a.d, a.r, a.bf16, false);
  Parts<T> p;
  hipError_t e = start(a, L, p, PrepareArgs<T>{}, stream);
  if (e != hipSuccess) return e;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  float2* stat = reinterpret_cast<float2*>(ws + L.stat);
  float* zlab = reinterpret_cast<float*>(ws + L.zlab);
  int bm = 0;
  auto make = [&](auto shape) {
    bm = shape.BM;
    return StatsEpi<T, shape.WA, shape.BN>{base_logits(a, p, 0, a.V, nullptr), p.rows.label, stat, a.N, zlab};
  };
  if ((e = multiply<kRows, kCols, kRows>(logits(a, p, 0, a.V), L.any, make, a.V, a.N,
                                         plan_for(a.V, a.N, a.d + a.r, L.any, a.d == 0, false), stream)) != hipSuccess)
    return e;
  // few rows: all threads of a workgroup on one row's tiles; many: neighbours
  // in a wave read neighbouring rows (whole call, V = 151936, rank 16, us: 256
  // rows 36 against 39, 512 rows 62 against 61, 2048 rows 209 against 186)
  const int tiles = (a.V + bm - 1) / bm;
  if (a.N <= 512)
    hipLaunchKernelGGL((join_kernel<256>), dim3(unsigned(a.N)), dim3(256), 0, stream, a.N, tiles, p.place, stat,
                       long(a.N), zlab, a.nll, a.lse);
  else
    hipLaunchKernelGGL((join_kernel<16>), dim3(unsigned((a.N + 15) / 16)), dim3(256), 0, stream, a.N, tiles, p.place,
                       stat, long(a.N), zlab, a.nll, a.lse);
  return hipGetLastError();
}

template <typename T>
hipError_t loss_backward_t(const LossArgs& a, hipStream_t stream) {
  const Layout L = layout(a.N, a.V, a.d, a.r, a.bf16, true);
  Parts<T> p;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  T* dz = reinterpret_cast<T*>(ws + L.dz);
  float *dXh = reinterpret_cast<float*>(ws + L.dXh), *dXe = reinterpret_cast<float*>(ws + L.dXe);
  const long split_h = long(L.rows) * L.dp, split_e = long(L.rows) * L.rp;
  T *dU = static_cast<T*>(a.dU), *dh = static_cast<T*>(a.dh), *dWo = static_cast<T*>(a.dWo);
  T *dW1 = static_cast<T*>(a.dW1), *dW2 = static_cast<T*>(a.dW2);
  const bool any = L.any;
  PrepareArgs<T> pre = {};
  pre.dU = dU;
  if (a.bf16 && (dWo || dW2)) {   // the bf16 products take whole steps of rows
    pre.dz = dz;
    pre.width = L.width;
  }
  pre.dW1 = dW1;
  pre.dW1_n = size_t(a.V) * a.r;
  hipError_t e = start(a, L, p, pre, stream);
  if (e != hipSuccess) return e;
  for (int v0 = 0; v0 < a.V; v0 += L.width) {
    const int nv = a.V - v0 < L.width ? a.V - v0 : L.width;
    auto grad = [&](auto) {
      return GradEpi<T>{base_logits(a, p, v0, nv, dU), p.rows.label, p.rows.lse, p.rows.g, dz, L.width, dU};
    };
    if ((e = multiply<kRows, kCols, kRows>(logits(a, p, v0, nv), any, grad, nv, a.N,
                                           plan_for(nv, a.N, a.d + a.r, any, a.d == 0, false), stream)) != hipSuccess) return e;
    const Operand<T> dz_rows = {dz, L.width, 1, L.rows}, dz_tokens = {dz, 1, L.width, nv};
    if (dh) {
      Product<T> g = {};
      g.A[0] = {p.Wo + size_t(v0) * L.wo_ld, 1, L.wo_ld, a.d};
      g.B[0] = dz_rows;
      g.K[0] = nv;
      g.nb = p.count;
      auto add = [&](auto) { return AddEpi{dXh, L.dp, a.d, v0 == 0, split_h}; };
      if ((e = multiply<kCols, kCols, kRows>(g, any, add, a.d, a.N, L.h, stream)) != hipSuccess) return e;
    }
    if (dW1) {
      Product<T> g = {};
      g.A[0] = {p.W2 + v0, L.w2_ld, 1, a.r};
      g.B[0] = dz_rows;
      g.K[0] = nv;
      g.nb = p.count;
      auto add = [&](auto) { return AddEpi{dXe, L.rp, a.r, v0 == 0, split_e}; };
      if ((e = multiply<kRows, kRows, kRows>(g, false, add, a.r, a.N, L.e, stream)) != hipSuccess) return e;
    }
    if (dWo) {
      Product<T> g = {};
      g.A[0] = {p.X, 1, p.kx, a.d};
      g.B[0] = dz_tokens;
      g.k0 = p.count;
      const bool vec = a.d % 4 == 0 && reinterpret_cast<uintptr_t>(dWo) % (4 * sizeof(T)) == 0;
      auto store = [&](auto) { return StoreEpi<T>{dWo + size_t(v0) * a.d, a.d, a.d, vec}; };
      if ((e = multiply<kCols, kCols, kCols>(g, false, store, a.d, nv,
                                             plan_for(a.d, nv, a.N, false, true, false), stream)) != hipSuccess) return e;
    }
    if (dW2) {
      Product<T> g = {};
      g.A[0] = dz_tokens;
      g.B[0] = {p.X + L.dp, 1, p.kx, a.r};
      g.k0 = p.count;
      const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(dW2) % (4 * sizeof(T)) == 0;
      auto store = [&](auto) { return StoreEpi<T>{dW2 + v0, a.V, nv, vec}; };
      if ((e = multiply<kCols, kCols, kCols>(g, false, store, nv, a.r,
                                             plan_for(nv, a.r, a.N, false, true, false), stream)) != hipSuccess) return e;
    }
  }
  if (a.N == 0) return hipSuccess;
  const unsigned rows = unsigned(a.N);
  // split sums are many values for few rows: a launch of their own, spread over
  // the columns below 1024 rows (whole call for dh and dW1, V = 30000, d = 2560,
  // spread against not, us: 128 rows 110 against 117, 512 220 against 231, 1024
  // 379 against 376, 4096 1351 against 1331)
  const bool join_e = dW1 && L.e.splits > 1, join_h = dh && (!dW1 || join_e || L.h.splits > 1);
  const unsigned wide = unsigned(((a.d > a.r ? a.d : a.r) + 255) / 256);
  if (join_e || join_h)
    hipLaunchKernelGGL((join_rows_kernel<T>), dim3(join_e ? 2 * rows : rows, rows >= 1024 ? 1 : wide), dim3(256), 0, stream, a.N, a.d,
                       long(L.dp), L.h.splits, split_h, p.place, dXh, dh, long(L.rp), L.e.splits, split_e, p.count,
                       dXe);
  if (dW1)
    hipLaunchKernelGGL((dw1_kernel<T>), dim3(dh && !join_h ? 2 * rows : rows), dim3(1024), 0, stream, a.N, a.r,
                       long(L.rp), p.count, p.rows.token, dXe, dW1, a.d, long(L.dp), L.h.splits, split_h, p.place, dXh,
                       dh);
  return hipGetLastError();
}

}  // namespace

size_t loss_workspace_bytes(int N, int V, int d, int r, bool bf16, bool backward) {
  return layout(N, V, d, r, bf16, backward).total;
}

hipError_t launch_markov_loss(const LossArgs& a, hipStream_t stream) {
  return a.bf16 ? loss_t<bf16_t>(a, stream) : loss_t<float>(a, stream);
}

hipError_t launch_markov_loss_backward(const LossArgs& a, hipStream_t stream) {
  return a.bf16 ? loss_backward_t<bf16_t>(a, stream) : loss_backward_t<float>(a, stream);
}

}  // namespace dspark
