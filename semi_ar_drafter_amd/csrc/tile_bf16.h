// Matrix product of bf16 operands on v_mfma_f32_16x16x32_bf16, tiles staged
// through LDS by direct-to-LDS loads.
//
// A step covers 64 of the contraction.  Each operand is stored with either the
// contraction contiguous (kRows: one row per a) or the a axis contiguous
// (kCols: one row per k), and is staged as it is stored:
//   kRows  LDS [a][64 k], 128 bytes a row; a fragment is one ds_read_b128.
//          16-byte chunk c of row a lies at place c ^ (a & 7), so that any 16
//          rows of one chunk fall on all 64 banks.
//   kCols  LDS [64 k][a]; a fragment is two ds_read_b64_tr_b16, which transpose
//          4 k x 16 a on the way out.  32-byte pair p of row k lies at p ^
//          pair_turn(k), so that the eight rows that half a wave reads (k to
//          k + 3 and k + 8 to k + 11) fall on all banks.
// The exchange is made on the global side (each lane picks which chunk it
// loads), because a direct-to-LDS load always writes lane after lane.
//
// Byte offsets inside a step are 32 bits: of a row length up to 2^24 values,
// 127 rows fit.
//
// Requirements, all met by the callers: bases 16-byte aligned; the b operand
// rows of a multiple of 8 values, zero from K to the next multiple of 64
// (kRows: the columns, kCols: the rows); the a operand, whatever its memory
// holds there, is loaded as zeros behind K, so that no infinity meets a zero.
// Its rows either have a multiple of 8 values (direct loads; up to 7 values
// behind K, in the row's own padding, have to be finite), or any number (ANY:
// loads to registers at element alignment, then LDS).
#pragma once
#include "projection.h"

namespace dspark {

enum Layout2 { kRows = 0, kCols = 1 };
constexpr int kStep = 64;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) unsigned char lds_u8_t;

// A load from kNowhere on, where the buffer ends, gives zeros.  It lies behind
// every offset of a step (127 rows of 2^25 bytes and a chunk: below 0xFE000100).
constexpr uint32_t kNowhere = 0xFF000000u;

#if defined(__HIP_DEVICE_COMPILE__)
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(kNowhere), 0x00020000);
}
// lane j: 16 bytes from base + off (per lane) to lds + 16 j
__device__ __forceinline__ void buffer_to_lds16(rsrc_t r, unsigned char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
#endif

template <int N> __device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Tile shape: BM along a, BN along b, WA x WB waves, S steps in LDS.
template <int BM_, int BN_, int WA_, int WB_, int S_>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WA = WA_, WB = WB_, S = S_;
  static constexpr int waves = WA * WB, threads = 64 * waves;
  static constexpr int FM = BM / WA / 16, FN = BN / WB / 16;
  static constexpr int a_bytes = BM * kStep * 2, b_bytes = BN * kStep * 2;
  static constexpr int stage = a_bytes + b_bytes, lds = S * stage;
  static constexpr int la = a_bytes / 1024, lb = b_bytes / 1024;   // 1 KiB wave loads per step
};

// Where the pairs of row k of a kCols tile of `rows` values are turned: bank
// = (32-byte pair of the row + rows / 16 * k) mod 8, and k, k + 1, k + 2,
// k + 3, k + 8, .. k + 11 have to differ (as far as the row has pairs).
__device__ __forceinline__ constexpr int pair_turn(int rows, int k) {
  return rows >= 128 ? (k & 3) | ((k >> 3 & 1) << 2) : rows == 64 ? (k >> 1 & 1) | ((k >> 3 & 1) << 1)
         : rows == 32 ? k >> 3 & 1 : 0;
}
// Turn of the chunks of row a of a kRows tile.
__device__ __forceinline__ constexpr int chunk_turn(int a) { return a & 7; }

// Number of wave loads of `n` that wave w of `waves` issues: a fixed count per
// wave, so that waits can count them (surplus waves repeat the last one).
constexpr int loads_per_wave(int n, int waves) { return (n + waves - 1) / waves; }

// One operand's staging by one wave: per-lane byte offsets from the tile's
// base, fixed over the steps.
// PAIR > 0 (kRows): the tile's rows are those of two matrices, PAIR of the one
// and PAIR of the other in turn (a wave's share of the tile is 2 PAIR rows, so
// that its accumulators of both lie in the same lanes).
template <int LAYOUT, int ROWS, int LOADS, int PAIR = 0>
struct Stager {
  static constexpr int units = ROWS * kStep / 512;   // 1 KiB each
  static constexpr int chunks = LAYOUT == kRows ? kStep / 8 : ROWS / 8;   // in a row of LDS
  uint32_t off[LOADS];

  __device__ __forceinline__ static int unit_of(int w, int i) { return min(w * LOADS + i, units - 1); }
  // the chunk of its row that a lane loads in any unit (kRows)
  __device__ __forceinline__ static int chunk_of(int lane) {
    return (lane % chunks) ^ chunk_turn(lane / chunks);
  }

  // first: the tile's first row along the operand's axis; n: its size; ld: row
  // length in values; w: wave.
  __device__ __forceinline__ void init(int first, int n, long ld, int w, int lane) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int row = (unit_of(w, i) * 64 + lane) / chunks;
      if (LAYOUT == kRows) {
        // rows behind the last one repeat it: their results are not stored
        const int r = PAIR ? row / (2 * PAIR + !PAIR) * PAIR + row % (PAIR + !PAIR) : row;
        off[i] = uint32_t(min(r, n - 1 - first)) * uint32_t(ld * 2) + uint32_t(chunk_of(lane)) * 16;
      } else {
        const int c = (unit_of(w, i) * 64 + lane) % chunks ^ (pair_turn(ROWS, row) << 1);
        // chunks behind the last one repeat it
        off[i] = uint32_t(row) * uint32_t(ld * 2) + uint32_t(min(c, (n - first + 7) / 8 - 1)) * 16;
      }
    }
  }

  // Whether load i of wave w is of the second matrix.
  __device__ __forceinline__ static bool other(int w, int i) { return PAIR && unit_of(w, i) * 8 / (PAIR + !PAIR) % 2; }

  // The last step of a contraction that ends inside it: whether the chunk
  // (kRows) or row (kCols) of a load lies behind its end.  left: what is left of it.
  __device__ __forceinline__ static bool behind(int i, int w, int lane, int left) {
    return LAYOUT == kRows ? chunk_of(lane) * 8 >= left : (unit_of(w, i) * 64 + lane) / chunks >= left;
  }
  // Offset of a direct load of that step: zeros behind the end.
  __device__ __forceinline__ uint32_t tail(int i, int w, int lane, int left) const {
    return behind(i, w, lane, left) ? kNowhere : off[i];
  }
};

// What every wave has waited for is visible to all behind it.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// 16 bytes at element alignment, not past `end`.
__device__ __forceinline__ u32x4_t load_any(const bf16_t* p, const bf16_t* end) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (p + 8 <= end) {
    __builtin_memcpy(&v, p, 16);
  } else {
    bf16_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p + i < end) e[i] = p[i];
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// Fragments of 32 of a step's 64, from `half` * 32 on.
template <int LAYOUT, int ROWS, int F>
__device__ __forceinline__ void read_frags(bf16x8_t (&f)[F], const unsigned char* lds, int first, int half, int lane) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int q = lane >> 4, l = lane & 15;
  if (LAYOUT == kRows) {
    const unsigned char* p = lds + (first + l) * (kStep * 2) + (((half * 4 + q) ^ chunk_turn(l)) * 16);
#pragma unroll
    for (int i = 0; i < F; ++i) f[i] = *reinterpret_cast<const bf16x8_t*>(p + i * 32 * kStep);
  } else {
    const int k = half * 32 + q * 8 + (l >> 2);   // and k + 4, which turns the same way
    const unsigned char* row = lds + k * (ROWS * 2) + (l & 3) * 8;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int pair = (first / 16 + i) ^ pair_turn(ROWS, k);
      const unsigned char* p = row + pair * 32;
      s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
      s16x4_t hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(p + 4 * ROWS * 2));
      const s16x8_t both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      f[i] = __builtin_bit_cast(bf16x8_t, both);
    }
  }
#endif
}

// Place of tile `id` of a grid of tiles_a x tiles_b: workgroups go round the
// eight XCDs, so each XCD takes a contiguous run of tiles; inside a run, up to
// eight tiles of b share their tile of a in the XCD's L2.
__device__ __forceinline__ void tile_place(int id, int tiles_a, int tiles_b, int* ta, int* tb) {
  const int n = tiles_a * tiles_b, q = n >> 3, r = n & 7, x = id & 7, at = id >> 3;
  const int t = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + at;
  const int group = 8 * tiles_a, g = t / group, in = t - g * group;
  const int wide = min(8, tiles_b - 8 * g);
  *ta = in / wide;
  *tb = 8 * g + in - *ta * wide;
}

// grid: x tiles, y splits of the contraction.  LA0, LA1: layout of the a
// operand in the two parts of the contraction; LB of b.  DUAL: the a operand
// is two matrices of na rows, A[0] and A[1], multiplied by the same b over one
// contraction; a wave's accumulators i < FM / 2 belong to the first, the others
// to the same rows of the second.
template <class Sh, int LA0, int LA1, int LB, bool ANY, class Epi, bool DUAL = false>
__global__ __launch_bounds__(Sh::threads) void tile_bf16_kernel(Product<bf16_t> g, Epi epi, int na, int nb) {
  extern __shared__ __align__(1024) unsigned char smem[];
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NA = loads_per_wave(Sh::la, Sh::waves), NB = loads_per_wave(Sh::lb, Sh::waves);
  constexpr bool two = LA0 != LA1;
  constexpr int halves = DUAL ? 2 : 1, BM = Sh::BM / halves, pair = DUAL ? BM / Sh::WA : 0;
  static_assert(!DUAL || (LA0 == kRows && LA1 == kRows && !ANY && Sh::FM % 2 == 0 && pair % 8 == 0), "two matrices by rows");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tile_a, tile_b;
  tile_place(blockIdx.x, (na + BM - 1) / BM, (nb + Sh::BN - 1) / Sh::BN, &tile_a, &tile_b);
  const int a_first = tile_a * BM, b_first = tile_b * Sh::BN;
  if (g.nb) nb = *g.nb;
  if (b_first >= nb) return;   // all its rows are behind the last one in use
  const int K0 = g.k0 ? *g.k0 : g.K[0], K1 = g.K[1];
  const int T0 = (K0 + kStep - 1) / kStep, T = T0 + (K1 + kStep - 1) / kStep;
  const int t_begin = int(long(T) * blockIdx.y / gridDim.y), t_end = int(long(T) * (blockIdx.y + 1) / gridDim.y);

  TileAt at;
  at.wave_a = wave / Sh::WB;
  at.wave_b = wave % Sh::WB;
  at.a0 = a_first + at.wave_a * (BM / Sh::WA);
  at.b0 = b_first + at.wave_b * (Sh::BN / Sh::WB);
  at.nb = nb;
  at.tile_a = tile_a;

  Stager<LA0, Sh::BM, NA, pair> sa0;
  Stager<LA1, Sh::BM, NA> sa1;
  Stager<LB, Sh::BN, NB> sb;
  const long lda0 = LA0 == kRows ? g.A[0].sa : g.A[0].sk, lda1 = LA1 == kRows ? g.A[1].sa : g.A[1].sk;
  const long ldb0 = LB == kRows ? g.B[0].sa : g.B[0].sk;
  sa0.init(a_first, g.A[0].n, lda0, wave, lane);
  sa1.init(a_first, g.A[1].n, lda1, wave, lane);
  sb.init(b_first, g.B[0].n, ldb0, wave, lane);
  const bf16_t* a0 = g.A[0].p + (LA0 == kRows ? long(a_first) * lda0 : long(a_first));
  const bf16_t* a1 = g.A[1].p + (LA1 == kRows ? long(a_first) * lda1 : long(a_first));
  const bf16_t* b0 = g.B[0].p + (LB == kRows ? long(b_first) * ldb0 : long(b_first));
  const bf16_t* b1 = g.B[1].p + (LB == kRows ? long(b_first) * ldb0 : long(b_first));   // both parts of b share ldb
  u32x4_t held[ANY ? NA : 1];

  // sends off the loads of step t
  auto issue = [&](int t) {
    unsigned char* st = smem + (t % Sh::S) * Sh::stage;
    const bool second = t >= T0;
    const int k = (second ? t - T0 : t) * kStep;
    {
      const rsrc_t rb = make_rsrc((second ? b1 : b0) + (LB == kRows ? long(k) : long(k) * ldb0));
#pragma unroll
      for (int i = 0; i < NB; ++i)
        buffer_to_lds16(rb, st + Sh::a_bytes + sb.unit_of(wave, i) * 1024, sb.off[i]);
    }
    const int left = (second ? K1 : K0) - k;
    if (ANY) {
      if (!second) {
        const bf16_t* p = a0 + (LA0 == kRows ? long(k) : long(k) * lda0);
        const bf16_t* end = g.A[0].p + (LA0 == kRows ? long(g.A[0].n - 1) * lda0 + K0 : long(K0 - 1) * lda0 + g.A[0].n);
#pragma unroll
        for (int i = 0; i < NA; ++i) {
          if (left < kStep && sa0.behind(i, wave, lane, left)) {
            held[i] = u32x4_t{0u, 0u, 0u, 0u};
            continue;
          }
          held[i] = load_any(reinterpret_cast<const bf16_t*>(reinterpret_cast<const char*>(p) + sa0.off[i]), end);
          if (LA0 == kRows && left < kStep) {   // values behind K belong to the next row
            const int keep = left - sa0.chunk_of(lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e >= keep) held[i][e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
        return;
      }
    }
    if (DUAL) {
      const rsrc_t r0 = make_rsrc(a0 + k), r1 = make_rsrc(a1 + k);
#pragma unroll
      for (int i = 0; i < NA; ++i)
        buffer_to_lds16(sa0.other(wave, i) ? r1 : r0, st + sa0.unit_of(wave, i) * 1024,
                        left < kStep ? sa0.tail(i, wave, lane, left) : sa0.off[i]);
    } else if (!two || !second) {
      const rsrc_t ra = make_rsrc((second ? a1 : a0) + (LA0 == kRows ? long(k) : long(k) * (second ? lda1 : lda0)));
      if (left < kStep) {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          buffer_to_lds16(ra, st + sa0.unit_of(wave, i) * 1024,
                          second ? sa1.tail(i, wave, lane, left) : sa0.tail(i, wave, lane, left));
      } else {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          buffer_to_lds16(ra, st + sa0.unit_of(wave, i) * 1024, second ? sa1.off[i] : sa0.off[i]);
      }
    } else {
      const rsrc_t ra = make_rsrc(a1 + (LA1 == kRows ? long(k) : long(k) * lda1));
      if (left < kStep) {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          buffer_to_lds16(ra, st + sa1.unit_of(wave, i) * 1024, sa1.tail(i, wave, lane, left));
      } else {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          buffer_to_lds16(ra, st + sa1.unit_of(wave, i) * 1024, sa1.off[i]);
      }
    }
  };
  // ANY: what issue() holds in registers goes to LDS
  auto put = [&](int t) {
    if (!ANY || t >= T0) return;
    unsigned char* st = smem + (t % Sh::S) * Sh::stage;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      *reinterpret_cast<u32x4_t*>(st + sa0.unit_of(wave, i) * 1024 + lane * 16) = held[i];
  };

  const int wa = at.wave_a * (Sh::BM / Sh::WA), wb = at.wave_b * (Sh::BN / Sh::WB);
  bf16x8_t fa[2][Sh::FM], fb[2][Sh::FN];   // a step's fragments
  f32x4_t acc[Sh::FM][Sh::FN];
  auto read = [&](int t) {
    const unsigned char* st = smem + (t % Sh::S) * Sh::stage;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      read_frags<LB, Sh::BN>(fb[half], st + Sh::a_bytes, wb, half, lane);
      if (two && t >= T0)
        read_frags<LA1, Sh::BM>(fa[half], st, wa, half, lane);
      else
        read_frags<LA0, Sh::BM>(fa[half], st, wa, half, lane);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < Sh::FM; ++i)
#pragma unroll
        for (int j = 0; j < Sh::FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[half][i], fb[half][j], acc[i][j], 0, 0, 0);
  };
  // A ring of S stages, one barrier a step; other workgroups of the compute
  // unit multiply while this one waits.  Loads go before the fragment reads
  // (after them: 800 us against 780 for a 5120 x 5120 layer's training pass).
  constexpr int per_step = NA + NB;
#pragma unroll
  for (int s = 0; s < Sh::S - 1; ++s)
    if (t_begin + s < t_end) {
      issue(t_begin + s);
      put(t_begin + s);
    }
  epi.init(acc, at);
  for (int t = t_begin; t < t_end; ++t) {
    // this wave's loads of step t have landed; later steps' may be on their way
    if (ANY || Sh::S == 2 || t_end - t - 1 < Sh::S - 2)
      wait_vm<0>();
    else
      wait_vm<per_step*(Sh::S - 2)>();
    lds_wait();
    meet();
    if (t + Sh::S - 1 < t_end) issue(t + Sh::S - 1);
    read(t);
    multiply();
    if (ANY && t + 1 < t_end) put(t + 1);
  }
  __syncthreads();
  epi.done(acc, at, smem);
#endif
}

// The 256 x 256 tile: 8 waves of 128 x 64, two per SIMD, one workgroup per
// compute unit, steps of 64.  Waves 0 to 3 ("lead") hold the first 128 of a,
// waves 4 to 7 the others; every SIMD has one of each.
//
// The two halves take turns: while one multiplies (64 MFMAs, 1024 cycles),
// the other reads its fragments from LDS.  In phase p the lead half reads step
// p / 2 (p even) or multiplies it (p odd); the other is one phase behind.
//
// Loads run at all times, because a step's 64 KiB take most of a step to
// arrive: rows of 128 bytes come at 35 to 50 bytes a cycle into a compute unit
// (64-byte rows at 18, measured), and a step at the full MFMA rate is 2048
// cycles.  A wave sends off one load after every eighth MFMA; sent off in one
// burst they hold up the reads and MFMAs behind them.  LDS holds two steps of
// each half's rows of a (a half overwrites its own as soon as it has read
// them) and three steps of b: 64 + 96 KiB.  In its MFMAs of step t a wave loads
// its half's a of step t + 2, and half of b: the lead of step t + 2, the other
// half (by then step t has been read by all) of step t + 3.  At their end it
// waits for what it sent off one step before.
struct Tile256 {
  static constexpr int BM = 256, BN = 256, WA = 2, WB = 4;
  static constexpr int a_half = 128 * kStep * 2, b_step = 256 * kStep * 2;
  static constexpr int lds = 4 * a_half + 3 * b_step;
};

// Byte offset of what `lane` loads in unit `unit` (1 KiB) of a tile of ROWS
// rows (of a, or values of one k), not held in registers.  n: the operand's
// size along its axis, from the tile's first on; what lies behind repeats the
// last.  left: what is left of the contraction; zeros behind it.
template <int LAYOUT, int ROWS>
__device__ __forceinline__ uint32_t unit_offset(int unit, int lane, uint32_t ld2, int n, int left) {
  constexpr int chunks = LAYOUT == kRows ? kStep / 8 : ROWS / 8;
  const int at = unit * 64 + lane, row = at / chunks;
  const int c = (at % chunks) ^ (LAYOUT == kRows ? chunk_turn(row) : pair_turn(ROWS, row) << 1);
  const bool behind = LAYOUT == kRows ? c * 8 >= left : row >= left;
  const uint32_t off = LAYOUT == kRows ? uint32_t(min(row, n - 1)) * ld2 + uint32_t(c) * 16
                                       : uint32_t(row) * ld2 + uint32_t(min(c, (n - 1) / 8)) * 16;
  return behind ? kNowhere : off;
}

// x, so that what is made from it is made here: held over the loop, read
// addresses and the last steps' offsets would spill what the MFMAs need.
__device__ __forceinline__ int here(int x) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(x));
#endif
  return x;
}

template <int LA0, int LA1, int LB, class Epi, bool DUAL = false>
__global__ __launch_bounds__(512) void tile256_kernel(Product<bf16_t> g, Epi epi, int na, int nb) {
  extern __shared__ __align__(1024) unsigned char smem[];
#if defined(__HIP_DEVICE_COMPILE__)
  typedef Tile256 Sh;
  constexpr bool two = LA0 != LA1;
  constexpr int BM = DUAL ? 128 : 256;
  static_assert(!DUAL || (LA0 == kRows && LA1 == kRows), "two matrices by rows");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tile_a, tile_b;
  tile_place(blockIdx.x, (na + BM - 1) / BM, (nb + 255) / 256, &tile_a, &tile_b);
  const int a_first = tile_a * BM, b_first = tile_b * 256;
  if (g.nb) nb = *g.nb;
  if (b_first >= nb) return;   // all its rows are behind the last one in use
  const int K0 = g.k0 ? *g.k0 : g.K[0], K1 = g.K[1];
  const int T0 = (K0 + kStep - 1) / kStep, T = T0 + (K1 + kStep - 1) / kStep;
  const int t_begin = int(long(T) * blockIdx.y / gridDim.y), t_end = int(long(T) * (blockIdx.y + 1) / gridDim.y);

  TileAt at;
  at.wave_a = wave >> 2;
  at.wave_b = wave & 3;
  at.a0 = a_first + at.wave_a * (BM / 2);
  at.b0 = b_first + at.wave_b * 64;
  at.nb = nb;
  at.tile_a = tile_a;
  const bool lead = wave < 4;
  const int w4 = wave & 3;

  const long lda0 = LA0 == kRows ? g.A[0].sa : g.A[0].sk, lda1 = LA1 == kRows ? g.A[1].sa : g.A[1].sk;
  const long ldb = LB == kRows ? g.B[0].sa : g.B[0].sk;   // of both parts of b
  // a half that lies wholly behind the operand's end repeats its last row
  const int n0 = g.A[0].n, n1 = g.A[1].n, nbo = g.B[0].n;
  const int f0 = min(at.a0, LA0 == kRows ? n0 - 1 : (n0 - 1) & ~7), f1 = min(at.a0, LA1 == kRows ? n1 - 1 : (n1 - 1) & ~7);
  // DUAL: of a half's 128 rows the first 64, which waves 0 and 1 load, are of A[0]
  const bf16_t* a0 = (DUAL && w4 >= 2 ? g.A[1].p : g.A[0].p) + (LA0 == kRows ? long(f0) * lda0 : long(f0));
  const bf16_t* a1 = g.A[1].p + (LA1 == kRows ? long(f1) * lda1 : long(f1));
  // kRows: from the wave's own 32 rows on, since 256 rows can be longer than a 32-bit offset reaches
  const int bf = LB == kRows ? min(b_first + wave * 32, nbo - 1) : b_first;
  const bf16_t* b0 = g.B[0].p + (LB == kRows ? long(bf) * ldb : long(bf));
  const bf16_t* b1 = g.B[1].p + (LB == kRows ? long(bf) * ldb : long(bf));

  // What a step's loads need besides the lane offsets: made while fragments
  // are on their way, so that little but the loads stands between the MFMAs.
  uint32_t off_a[4], off_b[4];
  rsrc_t rsrc_a, rsrc_b;
  unsigned char *lds_a, *lds_b;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    off_b[i] = unit_offset<LB, 256>(LB == kRows ? i : wave * 4 + i, lane, uint32_t(ldb * 2), nbo - bf, kStep);
  auto prepare_a = [&](int t, bool fresh) {   // this wave's four of its half's 16 units
    const bool second = t >= T0;
    const int k = (second ? t - T0 : t) * kStep, left = (second ? K1 : K0) - k;
    lds_a = smem + ((t & 1) * 2 + at.wave_a) * Sh::a_half + w4 * 4096;
    if (!two || !second) {
      const long ld = second ? lda1 : lda0;
      rsrc_a = make_rsrc((second ? a1 : a0) + (LA0 == kRows ? long(k) : long(k) * ld));
      if (fresh || t == T0 || left < kStep) {
        const int n = second ? n1 - f1 : n0 - f0, vlane = here(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          off_a[i] = unit_offset<LA0, 128>((DUAL ? w4 & 1 : w4) * 4 + i, vlane, uint32_t(ld * 2), n, left);
      }
    } else {
      rsrc_a = make_rsrc(a1 + (LA1 == kRows ? long(k) : long(k) * lda1));
      if (fresh || t == T0 || left < kStep) {
        const int vlane = here(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          off_a[i] = unit_offset<LA1, 128>(w4 * 4 + i, vlane, uint32_t(lda1 * 2), n1 - f1, left);
      }
    }
  };
  auto prepare_b = [&](int t) {   // this wave's four of all 32 units
    const bool second = t >= T0;
    const int k = (second ? t - T0 : t) * kStep;
    rsrc_b = make_rsrc((second ? b1 : b0) + (LB == kRows ? long(k) : long(k) * ldb));
    lds_b = smem + 4 * Sh::a_half + (t % 3) * Sh::b_step + wave * 4096;
  };
  auto load_a = [&](int i) { buffer_to_lds16(rsrc_a, lds_a + i * 1024, off_a[i]); };
  auto load_b = [&](int i) { buffer_to_lds16(rsrc_b, lds_b + i * 1024, off_b[i]); };

  bf16x8_t fa[2][8], fb[2][4];   // a step's fragments
  f32x4_t acc[8][4];
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int t = t_begin + s;
    if (t >= t_end) break;
    if (s < 2) {
      prepare_a(t, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_a(i);
    }
    if (s < 2 || !lead) {
      prepare_b(t);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_b(i);
    }
  }
  epi.init(acc, at);
  if (t_begin < t_end) {
    // the first step has landed: 8 of the loads sent off, in order
    if (t_end - t_begin == 1)
      wait_vm<0>();
    else if (lead || t_end - t_begin == 2)
      wait_vm<8>();
    else
      wait_vm<12>();
    meet();
    if (!lead) meet();   // phase 0 of the second half
    for (int t = t_begin; t < t_end; ++t) {
      const unsigned char* sa = smem + ((t & 1) * 2 + at.wave_a) * Sh::a_half;
      const unsigned char* sb = smem + 4 * Sh::a_half + (t % 3) * Sh::b_step;
      const int vlane = here(lane);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        read_frags<LB, 256>(fb[half], sb, at.wave_b * 64, half, vlane);
        if (two && t >= T0)
          read_frags<LA1, 128>(fa[half], sa, 0, half, vlane);
        else
          read_frags<LA0, 128>(fa[half], sa, 0, half, vlane);
      }
      const int next_a = t + 2, next_b = lead ? t + 2 : t + 3;
      if (next_a < t_end) prepare_a(next_a, false);
      if (next_b < t_end) prepare_b(next_b);
      lds_wait();
      // the second half's share of the second step's b, which the lead reads next
      if (!lead && t == t_begin) {
        if (t_end - t_begin > 2)
          wait_vm<4>();
        else
          wait_vm<0>();
      }
      meet();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int half = n >> 3, i = n & 7;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[half][i], fb[half][j], acc[i][j], 0, 0, 0);
        if (n % 2 == 0) {
          __builtin_amdgcn_sched_barrier(0);
          if (n < 8) {
            if (next_a < t_end) load_a(n / 2);
          } else {
            if (next_b < t_end) load_b(n / 2 - 4);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      if (next_b < t_end)
        wait_vm<8>();   // all but what this step sent off
      else
        wait_vm<0>();
      meet();
    }
    if (lead) meet();
  }
  __syncthreads();
  epi.done(acc, at, smem);
#endif
}

template <int LA0, int LA1, int LB, bool DUAL = false, class Epi>
hipError_t launch_tile256(const Product<bf16_t>& g, const Epi& epi, int na, int nb, int splits, hipStream_t stream) {
  if (na <= 0 || nb <= 0) return hipSuccess;
  constexpr int BM = DUAL ? 128 : 256;
  const unsigned tiles = unsigned((na + BM - 1) / BM) * unsigned((nb + 255) / 256);
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e =
      allow_lds(reinterpret_cast<const void*>(&tile256_kernel<LA0, LA1, LB, Epi, DUAL>), Tile256::lds, allowed);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile256_kernel<LA0, LA1, LB, Epi, DUAL>), dim3(tiles, unsigned(splits)), dim3(512), Tile256::lds,
                     stream, g, epi, na, nb);
  return hipGetLastError();
}

template <class Sh, int LA0, int LA1, int LB, bool ANY, bool DUAL = false, class Epi>
hipError_t launch_tile_bf16(const Product<bf16_t>& g, const Epi& epi, int na, int nb, int splits, hipStream_t stream) {
  static_assert(!ANY || Sh::S == 2, "register staging is double buffered");
  if (na <= 0 || nb <= 0) return hipSuccess;
  constexpr int BM = DUAL ? Sh::BM / 2 : Sh::BM;
  const unsigned tiles = unsigned((na + BM - 1) / BM) * unsigned((nb + Sh::BN - 1) / Sh::BN);
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e =
      allow_lds(reinterpret_cast<const void*>(&tile_bf16_kernel<Sh, LA0, LA1, LB, ANY, Epi, DUAL>), Sh::lds, allowed);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_bf16_kernel<Sh, LA0, LA1, LB, ANY, Epi, DUAL>), dim3(tiles, unsigned(splits)), dim3(Sh::threads),
                     Sh::lds, stream, g, epi, na, nb);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Choice of the tile
// ---------------------------------------------------------------------------
// Few rows: bound by reading the a operand once, so narrow tiles with a deep
// ring, several workgroups per compute unit.  Many rows: 256 x 256, where one
// step's 128 MFMAs per SIMD cover the loads of the next.
using Tile16 = TileShape<128, 16, 4, 1, 4>;
using Tile32 = TileShape<128, 32, 4, 1, 3>;
using Tile64 = TileShape<128, 64, 2, 2, 3>;
using Tile128 = TileShape<128, 128, 2, 2, 2>;
// Where there is at most one workgroup per compute unit anyhow: two steps more
// in flight.  It pays where nearly all units have one and the contraction is
// long (loss of 100 rows, V = 30000, d = 2048: 37.3 us against 42.4), and costs
// a few per cent otherwise (1000 rows, V = 4000, d = 2048: 41.8 against 39.9;
// 250 rows, V = 8192, d = 512: 18.4 against 18.1).
using Tile128Deep = TileShape<128, 128, 2, 2, 4>;
using Tile16Any = TileShape<128, 16, 4, 1, 2>;
using Tile32Any = TileShape<128, 32, 4, 1, 2>;
using Tile64Any = TileShape<128, 64, 2, 2, 2>;

constexpr int kComputeUnits = 256;

// dst[r][0..ld) = src[r][0..n), zeros behind: rows that are not 16-byte
// aligned, or no whole number of steps, copied.  Eight values per thread.
static __global__ __launch_bounds__(256) void pad_rows_kernel(long rows, long n, long ld, const bf16_t* __restrict__ src,
                                                              bf16_t* __restrict__ dst) {
  const uint32_t per = uint32_t(ld / 8);   // ld is a multiple of 8
  const long at = long(blockIdx.x) * 256 + threadIdx.x;
  if (at >= rows * per) return;
  const long r = at / per, c = (at - r * per) * 8;
  const bf16_t* s = src + r * n;
  const u32x4_t v = load_any(s + c, s + (c < n ? n : c));
  *reinterpret_cast<u32x4_t*>(dst + at * 8) = v;
}
// At most 2^31 threads a launch, where a grid holds less than 2^32.
inline hipError_t pad_rows(long rows, long n, long ld, const bf16_t* src, bf16_t* dst, hipStream_t stream) {
  const long most = (1l << 31) / (ld / 8);
  for (long r0 = 0; r0 < rows; r0 += most) {
    const long some = rows - r0 < most ? rows - r0 : most;
    hipLaunchKernelGGL(pad_rows_kernel, dim3(unsigned((some * (ld / 8) + 255) / 256)), dim3(256), 0, stream, some, n, ld,
                       src + r0 * n, dst + r0 * ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// Weights whose rows are not 16-byte aligned are copied up to this size, where
// their product is long: the copy takes a few microseconds, and direct loads
// then take less than half of a step by register staging (24 rows, 1088 x
// 3535: 52 us for the logits before, 27 with the copy), or allow the large
// tile.
constexpr size_t kCopyBytes = size_t(64) << 20;

// Which tile a product takes (0 .. 4: Tile16 .. Tile256) and into how many
// fp32 sums its contraction is split.
struct Plan {
  int tile, splits;
  double cost = 0;   // in steps of the 256 x 256 tile, as below
};

// any: register staging, which the large tile has no registers left for.
// split: the caller can join split sums.
//
// A compute unit works through its tiles one after the other (two of the
// smaller ones side by side), so the time goes with the number of rounds.
// In units of a step of the 256 x 256 tile (1.64 us at 8192^3), a round of
// that tile takes its steps and 7 for its ends; two 128 x 128 tiles side by
// side take 3 and, a step, 0.6 or (cols: the a operand is kCols) 0.72.
// (8192^3: 840 us against 1000 and 1230; 4096 x 5120 x 5120, 320 large tiles
// on 256 units: 267 against 248 and 285; 1000 x 50021 outputs of five steps:
// 76 against 70.)  A split costs the writing and
// reading of its tile in fp32: 12 and 4.
inline Plan plan_for(int na, int nb, long K, bool any, bool cols, bool split) {
  const long steps = (K + kStep - 1) / kStep;
  const int first = nb <= 16 ? 0 : nb <= 32 ? 1 : nb <= 64 ? 2 : 3, last = first < 3 || any ? first : 4;
  Plan best = {first, 1};
  double least = 1e300;
  for (int c = last; c >= first; --c) {
    const bool large = c == 4;
    const long bm = large ? 256 : 128, bn = large ? 256 : 16l << c, slots = (large ? 1 : 2) * kComputeUnits;
    const long tiles = ((na + bm - 1) / bm) * ((nb + bn - 1) / bn);
    for (int s = 1; s <= 64 && (s == 1 || (split && s * 4 <= steps)); ++s) {
      const double rounds = double((tiles * s + slots - 1) / slots);
      const double steps_s = double((steps + s - 1) / s);
      const double cost = rounds * (large ? steps_s + 7 + (s > 1 ? 12 : 0) : (cols ? 0.72 : 0.6) * steps_s + 3 + (s > 1 ? 4 : 0));
      if (cost < least * 0.97) {
        least = cost;
        best = {c, s, cost};
      }
    }
  }
  return best;
}

// make(shape) gives the epilogue for a tile shape (its statistics depend on
// the shape).
template <int LA0, int LA1, int LB, bool ANY, class Make>
hipError_t launch_bf16(const Product<bf16_t>& g, const Make& make, int na, int nb, Plan plan, hipStream_t stream) {
  const int s = plan.splits;
  if constexpr (ANY) {
    switch (plan.tile) {
      case 0: return launch_tile_bf16<Tile16Any, LA0, LA1, LB, true>(g, make(Tile16Any()), na, nb, s, stream);
      case 1: return launch_tile_bf16<Tile32Any, LA0, LA1, LB, true>(g, make(Tile32Any()), na, nb, s, stream);
      case 2: return launch_tile_bf16<Tile64Any, LA0, LA1, LB, true>(g, make(Tile64Any()), na, nb, s, stream);
      default: return launch_tile_bf16<Tile128, LA0, LA1, LB, true>(g, make(Tile128()), na, nb, s, stream);
    }
  } else {
    switch (plan.tile) {
      case 0: return launch_tile_bf16<Tile16, LA0, LA1, LB, false>(g, make(Tile16()), na, nb, s, stream);
      case 1: return launch_tile_bf16<Tile32, LA0, LA1, LB, false>(g, make(Tile32()), na, nb, s, stream);
      case 2: return launch_tile_bf16<Tile64, LA0, LA1, LB, false>(g, make(Tile64()), na, nb, s, stream);
      case 3:
        if (long((na + 127) / 128) * ((nb + 127) / 128) * s <= kComputeUnits)
          return launch_tile_bf16<Tile128Deep, LA0, LA1, LB, false>(g, make(Tile128Deep()), na, nb, s, stream);
        return launch_tile_bf16<Tile128, LA0, LA1, LB, false>(g, make(Tile128()), na, nb, s, stream);
      default: return launch_tile256<LA0, LA1, LB>(g, make(Tile256()), na, nb, s, stream);
    }
  }
}

// The same for two matrices of na rows each, whose plan is that of 2 na.
template <class Make>
hipError_t launch_bf16_dual(const Product<bf16_t>& g, const Make& make, int na, int nb, Plan plan, hipStream_t stream) {
  const int s = plan.splits;
  switch (plan.tile) {
    case 0: return launch_tile_bf16<Tile16, kRows, kRows, kRows, false, true>(g, make(Tile16()), na, nb, s, stream);
    case 1: return launch_tile_bf16<Tile32, kRows, kRows, kRows, false, true>(g, make(Tile32()), na, nb, s, stream);
    case 2: return launch_tile_bf16<Tile64, kRows, kRows, kRows, false, true>(g, make(Tile64()), na, nb, s, stream);
    case 3: return launch_tile_bf16<Tile128, kRows, kRows, kRows, false, true>(g, make(Tile128()), na, nb, s, stream);
    default: return launch_tile256<kRows, kRows, kRows, true>(g, make(Tile256()), na, nb, s, stream);
  }
}

}  // namespace dspark
