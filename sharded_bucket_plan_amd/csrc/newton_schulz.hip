// Newton-Schulz orthogonalisation of weight-matrix updates on CDNA4 (gfx950).
//
// Per matrix U (rows x cols), with X on its short side (m <= n; X = U, or U'
// where rows > cols):
//   X_0 = U / max(|U|_F, eps)
//   A = X X',  B = b A + c A^2,  X <- a X + B X      (steps times)
//   out = bf16(out_scale * X)
//
// The iterate stays in its matrix's own orientation, S (rows x cols): S = X
// where rows <= cols (wide), S = X' otherwise (tall).  Three products per step,
// one kernel core:
//   gram   A  = X X'          lower-triangle tiles only, mirrored on the way out
//   poly   B  = b A + c A A'  (A is symmetric) likewise
//   apply  S' = a S + B S  (wide)  or  a S + S B  (tall)
// C = P Q' wants rows of P and Q with the contracted index along the row.  A,
// B, wide gram and tall apply have that; wide apply's and tall gram's S runs
// across, and is read from LDS with the transposing reads of gfx950.  (Keeping
// X in both orientations instead, written twice by every apply, took 45% of
// apply's time in its epilogue at 14336 x 4096.)
//
// Numbers.  The products run on fp16 MFMA with binary32 accumulation: fp16
// keeps 11 significand bits where bf16 keeps 8, at the same rate, and every
// operand has a known range that a power of two places inside fp16's:
//   X_0     U * 2^k with the Frobenius norm in [2^13, 2^14): exact for bf16
//           U down to 2^-28 of the norm; the rest of the normalisation, rho =
//           1 / (max(norm, eps) 2^k), multiplies the accumulators of step 1
//   X       * 2^12 (entries up to 16); a matrix whose norm lies below eps
//           gets a further power of two that its iterates cannot outgrow
//   A       * 2^12,  B * 2^10
// Two roundings would stand out, and their remainders are kept:
//   - A and B end near multiples of the identity, so the rounding of their
//     diagonals dominates theirs; the diagonals' remainders (binary32, m of
//     each) enter B's epilogue as (A + D)^2 and apply's as (a + D) X;
//   - the step's amplification of small singular values (a^steps ~ 485)
//     amplifies X's rounding noise as well.  It reaches them only through the
//     term a X, since B's share of it is multiplied by B, small on exactly
//     those directions; so while at least three steps remain, X's remainder
//     is kept (fp16, * 2^11) and a X is formed from both parts.
// Relative error against the iteration in 64 bits, 5 steps, before the
// output's rounding (1.7e-3 by itself), on spectra from flat to rank 16 plus
// 0.03 of noise: 4e-4 .. 1.0e-3 (rank 16 plus 0.003: 2.3e-3); without the
// diagonals' remainders up to 2.2e-3, without either up to 2.6e-2, with bf16
// products 7e-3 .. 2e-1.
// The squared norm is summed in float64 in a fixed order, so results are the
// same from run to run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>
#include <vector>

#include "bf16.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256;
constexpr int kXcds = 8;
constexpr int kPad = 64;        // both padded sides are multiples of this
constexpr int kMaxGroups = 16;  // groups of equal matrices per launch
constexpr int kMaxNormBlocks = 256;
constexpr float kScaleX = 4096.0f, kScaleA = 4096.0f, kScaleB = 1024.0f, kScaleLo = 2048.0f;

// Per-matrix scalars, written by the prologue.
// Stored X_0 = X_0 / rho, stored X_k = X_k * sx for k >= 1.
struct Scal {
  float gram_first, gram;  // accumulator -> stored A: rho^2 * 2^12, 2^12 / sx^2
  float apply_first;       // step 1's accumulator -> stored X_1: rho * sx
  float inv_sx;
};

// One group: `count` matrices of one shape, at equal distances.
struct Group {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_ld, out_ld, in_stride, out_stride;
  _Float16* base;    // S, S2, L (count*m*n each), A, B (count*m*m each)
  double* partial;   // count * norm_blocks
  Scal* scal;        // count
  float* diag;       // m each: count for A, count for B (rounding remainders)
  int32_t rows, cols, count;
  int32_t rp, cp;    // rows and cols padded
  int32_t m, n;      // the smaller and the larger of rp and cp
  int32_t norm_blocks;
  float out_scale;
  int32_t in_vec, out_vec;  // 16-byte rows
  uint32_t t_norm, t_pro, t_gram, t_apply;  // first block of the group in each launch

  __host__ __device__ bool tall() const { return rows > cols; }
  __device__ int64_t mn() const { return static_cast<int64_t>(m) * n; }
  __device__ _Float16* S(int which, int item) const {
    return base + (static_cast<int64_t>(which) * count + item) * mn();
  }
  __device__ _Float16* L(int item) const {
    return base + (static_cast<int64_t>(2) * count + item) * mn();
  }
  __device__ float* D(int which, int item) const {
    return diag + (static_cast<int64_t>(which) * count + item) * m;
  }
  __device__ _Float16* A(int which, int item) const {
    return base + static_cast<int64_t>(3) * count * mn() +
           (static_cast<int64_t>(which) * count + item) * m * m;
  }
};

struct Groups {
  Group g[kMaxGroups];
  int32_t n;
};

struct Step {
  float a, b, c, eps;
  int32_t grow;   // the iterates of a matrix grow by less than 2^grow in all
  int32_t first, last, lo_in, lo_out;
  int32_t in;     // which of the two copies of S this step reads
};

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = x + __shfl_xor(x, off, 64);
  return x;
}

// Sum over the block in a fixed order, in every thread.
__device__ __forceinline__ double block_sum_all(double x) {
  __shared__ double per_wave[kBlock / 64];
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) per_wave[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kBlock / 64; ++w) t = t + per_wave[w];
  return t;
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x[q] = lo[q];
    x[4 + q] = hi[q];
  }
}

// Up to 8 consecutive bf16 values of a row, zeros from `left` on.
__device__ __forceinline__ u32x4 load_row8(const uint16_t* p, int left, bool vec) {
  if (vec && left >= 8) return *reinterpret_cast<const u32x4*>(p);
  u32x4 w{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
  return w;
}

// ---- squared norms: one float64 partial per block ----------------------------
// A wave takes one row's 512 columns at a time; block b of a matrix's
// norm_blocks takes units b*4 + wave, then every norm_blocks*4 further on.
__global__ void __launch_bounds__(kBlock) ns_norm_kernel(Groups gs) {
  int gi = 0;
  while (gi + 1 < gs.n && blockIdx.x >= gs.g[gi + 1].t_norm) ++gi;
  const Group& g = gs.g[gi];
  const int local = blockIdx.x - g.t_norm;
  const int item = local / g.norm_blocks, nb = local % g.norm_blocks;
  const uint16_t* in = g.in + item * g.in_stride;
  const int segs = (g.cols + 511) / 512;
  const int64_t units = static_cast<int64_t>(g.rows) * segs;
  const int lane = threadIdx.x & 63;
  double sum = 0.0;
  for (int64_t u = nb * 4 + (threadIdx.x >> 6); u < units; u += g.norm_blocks * 4) {
    const int64_t row = u / segs;
    const int col = static_cast<int>(u % segs) * 512 + lane * 8;
    if (col < g.cols) {
      const u32x4 w = load_row8(in + row * g.in_ld + col, g.cols - col, g.in_vec);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double x = sbp::bf16_lo(w[q]), y = sbp::bf16_hi(w[q]);
        sum = sum + x * x;
        sum = sum + y * y;
      }
    }
  }
  sum = block_sum_all(sum);
  if (threadIdx.x == 0) g.partial[local] = sum;
}

// ---- prologue: S_0 in fp16, zero-padded ----------------------------------------
// A block takes 32 rows of 64 columns of the padded matrix.
__global__ void __launch_bounds__(kBlock) ns_prologue_kernel(Groups gs, float eps, int grow) {
  int gi = 0;
  while (gi + 1 < gs.n && blockIdx.x >= gs.g[gi + 1].t_pro) ++gi;
  const Group& g = gs.g[gi];
  const int tc = g.cp / 64, per = (g.rp / 32) * tc;
  const int local = blockIdx.x - g.t_pro;
  const int item = local / per, t = local % per;
  const int row = t / tc * 32 + (threadIdx.x >> 3), col = t % tc * 64 + (threadIdx.x & 7) * 8;
  u32x4 w{0, 0, 0, 0};
  if (row < g.rows && col < g.cols)
    w = load_row8(g.in + item * g.in_stride + row * g.in_ld + col, g.cols - col, g.in_vec);

  double sq = 0.0;
  for (int i = threadIdx.x; i < g.norm_blocks; i += kBlock)
    sq = sq + g.partial[item * g.norm_blocks + i];
  const double norm = sqrt(block_sum_all(sq));
  // norm * 2^k in [2^13, 2^14); 0 for a zero, infinite or NaN norm
  const bool plain = norm > 0.0 && norm < __builtin_huge_val();
  const int k = plain ? 13 - ilogb(norm) : 0;
  if (t == 0 && threadIdx.x == 0) {
    const double floor_norm = norm < eps ? static_cast<double>(eps) : norm;  // NaN stays
    int below = plain && norm < eps ? ilogb(static_cast<double>(eps)) - ilogb(norm) : 0;
    below = below > grow + 2 ? below - grow - 2 : 0;
    below = below < 100 ? below : 100;
    const double rho = 1.0 / (floor_norm * ldexp(1.0, k));
    const double sx = ldexp(static_cast<double>(kScaleX), below);
    g.scal[item] = Scal{static_cast<float>(rho * rho * kScaleA),
                        static_cast<float>(kScaleA / (sx * sx)), static_cast<float>(rho * sx),
                        static_cast<float>(1.0 / sx)};
  }
  f16x8 h;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h[2 * q] = static_cast<_Float16>(ldexpf(sbp::bf16_lo(w[q]), k));
    h[2 * q + 1] = static_cast<_Float16>(ldexpf(sbp::bf16_hi(w[q]), k));
  }
  *reinterpret_cast<f16x8*>(g.S(0, item) + static_cast<int64_t>(row) * g.cp + col) = h;
}

// ---- the product ------------------------------------------------------------------

enum Mode { kGram, kPoly, kApply, kLast };  // kLast: apply, to the caller's matrices

// One T x T tile of C = P Q' per block of 4 waves (2 x 2, each T/2 square, in
// 32 x 32 MFMA tiles).  Slices of BK k elements go straight from memory to one
// of four LDS buffers, three slices ahead of the one being multiplied.
template <int T, int BK>
struct Tile {
  static constexpr int kHalf = T * BK * 2;  // one operand's slice, bytes
  static constexpr int kBuf = 2 * kHalf;
  static constexpr int kSub = T / 64;                // 32 x 32 tiles per wave and side
  static constexpr int kLoads = kHalf / (4 * 1024);  // per operand, slice and lane
  static constexpr int kPhases = BK / 16;
};

// This wave's share of one operand's slice, `bytes` from `from`.
template <int T, int BK>
__device__ __forceinline__ void stage(char* buf, const char* from, int bytes, int wave, int voff,
                                      int round_bytes) {
  const __amdgpu_buffer_rsrc_t rows =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0, bytes, 0x00027000);
#pragma unroll
  for (int r = 0; r < Tile<T, BK>::kLoads; ++r)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rows, (__attribute__((address_space(3))) void*)(buf + (r * 4 + wave) * 1024), 16, voff,
        r * round_bytes, 0, 0);
}

// One operand of a tile.  Along: the matrix's rows r0 .. are the operand's
// rows, and a slice is BK consecutive elements of each; LDS keeps a row's
// 16-byte pieces rotated by row.  Across: the matrix's columns r0 .. are the
// operand's rows, and a slice is BK rows of T elements; LDS keeps a row's
// 64-byte pieces rotated by row, and the reads transpose.  Both rotations come
// from the lanes' global addresses and spread the reads over the banks.
// Rows past the matrix read as zero or as a neighbour: they only reach
// results that are not stored.
template <int T, int BK, bool ACROSS>
struct Operand {
  using TL = Tile<T, BK>;
  const char* from;  // next slice to load
  int64_t step;
  int bytes, voff, round_bytes;
  int at;                            // LDS offset of this lane's first fragment
  int off[ACROSS ? TL::kSub : TL::kPhases];  // further offset by sub-tile or phase

  __device__ __forceinline__ void init(const _Float16* mat, int rows, int ld, int r0, int wave,
                                       int lane, int wrow) {
    if constexpr (ACROSS) {
      constexpr int kLanes = T / 8;  // lanes per row
      from = reinterpret_cast<const char*>(mat + r0);
      step = static_cast<int64_t>(BK) * ld * 2;
      bytes = (BK * ld - r0) * 2;
      const int row = wave * (64 / kLanes) + lane / kLanes;
      const int piece = lane % kLanes;
      voff = row * ld * 2 + ((((piece >> 2) ^ turn(row)) << 2) | (piece & 3)) * 16;
      round_bytes = 4 * (64 / kLanes) * ld * 2;
      const int k = (lane >> 5) * 8 + ((lane >> 2) & 3);  // of this lane's address
      at = k * (T * 2) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < TL::kSub; ++i) off[i] = ((wrow / 32 + i) ^ turn(k)) * 64;
    } else {
      constexpr int kLanes = BK / 8;
      from = reinterpret_cast<const char*>(mat + static_cast<int64_t>(r0) * ld);
      step = BK * 2;
      const int have = rows - r0 < T ? rows - r0 : T;
      bytes = have * ld * 2;
      const int row = wave * (64 / kLanes) + lane / kLanes;
      voff = row * ld * 2 + ((lane % kLanes) ^ turn(row)) * 16;
      round_bytes = 4 * (64 / kLanes) * ld * 2;
      at = (wrow + (lane & 31)) * (BK * 2);
#pragma unroll
      for (int p = 0; p < TL::kPhases; ++p) off[p] = ((p * 2 + (lane >> 5)) ^ turn(lane)) * 16;
    }
  }
  // The rotation of a row; rows that differ by 32 (along) or 4 (across) agree.
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (ACROSS) return T >= 128 ? row & 3 : (row >> 1) & 1;
    else return BK == 32 ? (row >> 2) & 3 : row & 7;
  }
  // Along, the last rows' slices end before `bytes` does by what is consumed.
  __device__ __forceinline__ void load(char* buf, int wave) {
    stage<T, BK>(buf, from, bytes, wave, voff, round_bytes);
    from += step;
    if constexpr (!ACROSS) bytes -= BK * 2;
  }
  __device__ __forceinline__ f16x8 read(const char* buf, int phase, int i) const {
    if constexpr (ACROSS) {
      typedef __fp16 h4 __attribute__((__vector_size__(8)));
      typedef __attribute__((address_space(3))) h4* lds_h4;
      const char* p = buf + at + off[i] + phase * 16 * (T * 2);
      const h4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)p);
      const h4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)(p + 4 * (T * 2)));
      return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const f16x8*>(buf + at + off[phase] + i * 32 * (BK * 2));
    }
  }
};

template <int T>
struct Frags {
  f16x8 p[T / 64], q[T / 64];
};

template <int T>
using Acc = f32x16[T / 64][T / 64];

template <int T>
__device__ __forceinline__ void multiply(const Frags<T>& f, Acc<T>& acc) {
#pragma unroll
  for (int i = 0; i < T / 64; ++i)
#pragma unroll
    for (int j = 0; j < T / 64; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.p[i], f.q[j], acc[i][j], 0, 0, 0);
}

// Order of a phase's instructions: MFMAs, LDS reads and loads to LDS in turn,
// so that both kinds of memory work run under the MFMAs.
template <int T, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
  constexpr int mfmas = (T / 64) * (T / 64);
  constexpr int r1 = (READS + mfmas - 1) / mfmas, l1 = (LOADS + mfmas - 1) / mfmas;
#pragma unroll
  for (int i = 0; i < mfmas; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i * r1 < READS) __builtin_amdgcn_sched_group_barrier(0x100, r1, 0);
    if (i * l1 < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, l1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// All of this wave's loads but the newest LEFT are done, and its LDS reads;
// then everyone's.
template <int LEFT>
__device__ __forceinline__ void slice_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// This wave's LDS work is done, then everyone's; loads and stores run on.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// acc = P Q' over `slices` slices.
template <int T, int BK, bool PX, bool QX>
__device__ __forceinline__ void product(char* buf0, char* buf1, char* buf2, char* buf3,
                                        Operand<T, BK, PX>& P, Operand<T, BK, QX>& Q, int slices,
                                        int wave, Acc<T>& acc) {
  using TL = Tile<T, BK>;
  constexpr int L = TL::kLoads, H = TL::kHalf, N = TL::kPhases;
  constexpr int kReads = TL::kSub * ((PX ? 2 : 1) + (QX ? 2 : 1));
  Frags<T> f[2];
  auto load = [&](char* to) {
    P.load(to, wave);
    Q.load(to + H, wave);
  };
  auto read = [&](const char* buf, int phase, Frags<T>& to) {
#pragma unroll
    for (int i = 0; i < TL::kSub; ++i) {
      to.p[i] = P.read(buf, phase, i);
      to.q[i] = Q.read(buf + H, phase, i);
    }
  };
  // One slice: it is in `cur`, its first fragments in f[0].  The barrier sits
  // before the last multiply, so that each multiply hides the next one's reads.
  // LOAD: the slice three further on is loaded into `to`; LEFT: loads that may
  // still be under way when the next slice has to be there (-1: no next one).
  auto slice = [&](const char* cur, const char* nxt, char* to, auto load_c, auto left_c) {
    constexpr bool kLoad = decltype(load_c)::value;
    constexpr int kLeft = decltype(left_c)::value;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ph = 0; ph < N - 1; ++ph) {
      if (kLoad && ph == 0) P.load(to, wave);
      read(cur, ph + 1, f[(ph + 1) & 1]);
      multiply<T>(f[ph & 1], acc);
      if (kLoad && ph == 0) interleave<T, kReads, L>();
      else interleave<T, kReads, 0>();
    }
    if constexpr (kLeft >= 0) {
      slice_barrier<kLeft>();
      if constexpr (kLoad) Q.load(to + H, wave);
      read(nxt, 0, f[0]);
    }
    multiply<T>(f[1], acc);
    interleave<T, kLeft >= 0 ? kReads : 0, kLoad ? L : 0>();
  };
  constexpr std::true_type kYes{};
  constexpr std::false_type kNo{};
  // two slices under way, and the first half of a third
  constexpr std::integral_constant<int, 3 * L> kSteady{};
  constexpr std::integral_constant<int, 2 * L> kOne{};
  constexpr std::integral_constant<int, 0> kNone{};
  constexpr std::integral_constant<int, -1> kEnd{};
  // The last slice is in buf3, so that there is one way into the loop's rounds
  // of four and one way out; a number that is no multiple of four starts
  // further on, and drains its loads once (known to the compiler, whose own
  // waits in the loop would else provide for the other way in).  With BK = 32
  // the number is even.
  constexpr bool kOdd = BK != 32;
  const int rest = slices & 3;
  if (slices < 4) {
    if (kOdd && rest == 3) load(buf1);
    if (!kOdd || rest >= 2) load(buf2);
    load(buf3);
    slice_barrier<0>();
    read(kOdd && rest == 3 ? buf1 : !kOdd || rest == 2 ? buf2 : buf3, 0, f[0]);
    if (kOdd && rest == 3) slice(buf1, buf2, nullptr, kNo, kNone);
    if (!kOdd || rest >= 2) slice(buf2, buf3, nullptr, kNo, kNone);
  } else {
    if (rest == 0) {
      load(buf0);
      load(buf1);
      load(buf2);
      slice_barrier<4 * L>();
      read(buf0, 0, f[0]);
    } else {
      if (kOdd && rest == 3) {
        load(buf1);
        load(buf2);
        load(buf3);
        slice_barrier<4 * L>();
        read(buf1, 0, f[0]);
        slice(buf1, buf2, buf0, kYes, kSteady);
      }
      if (rest >= 2) {
        if (!kOdd || rest == 2) {
          load(buf2);
          load(buf3);
          load(buf0);
          slice_barrier<4 * L>();
          read(buf2, 0, f[0]);
        }
        slice(buf2, buf3, buf1, kYes, kSteady);
      }
      if (kOdd && rest == 1) {
        load(buf3);
        load(buf0);
        load(buf1);
        slice_barrier<4 * L>();
        read(buf3, 0, f[0]);
      }
      slice(buf3, buf0, buf2, kYes, kSteady);
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    }
    for (int s = slices >> 2; s > 1; --s) {
      slice(buf0, buf1, buf3, kYes, kSteady);
      slice(buf1, buf2, buf0, kYes, kSteady);
      slice(buf2, buf3, buf1, kYes, kSteady);
      slice(buf3, buf0, buf2, kYes, kSteady);
    }
    slice(buf0, buf1, buf3, kYes, kSteady);
    slice(buf1, buf2, nullptr, kNo, kOne);
    slice(buf2, buf3, nullptr, kNo, kNone);
  }
  slice(buf3, nullptr, nullptr, kNo, kEnd);
}

// Up to 8 consecutive bf16 values of a row of the caller's output.
__device__ __forceinline__ void store_out8(uint16_t* p, int left, bool vec, const float (&v)[8]) {
  uint32_t b[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) b[q] = sbp::bf16_rne(v[q]);
  if (vec && left >= 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{b[0] | (b[1] << 16), b[2] | (b[3] << 16),
                                         b[4] | (b[5] << 16), b[6] | (b[7] << 16)};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left) p[q] = static_cast<uint16_t>(b[q]);
  }
}

// Where (row, col) of the epilogue's binary32 slab is kept: 32 rows in each of
// two buffers; groups of 8 columns are rotated by the row's 8-row group, so
// that both a row's 8 columns and a column's 8 rows are read without bank
// conflicts.
template <int T>
__device__ __forceinline__ float* slab_at(char* lo, char* hi, int row, int col) {
  float* half = reinterpret_cast<float*>(row & 32 ? hi : lo);
  return half + (row & 31) * T + (col ^ (((row >> 3) & 7) << 3));
}

template <int T, int BK, Mode M>
__global__ void __launch_bounds__(kBlock, T == 256 ? 1 : 2)
ns_product_kernel(Groups gs, Step st, unsigned total) {
  using TL = Tile<T, BK>;
  // separate arrays: reads of one do not wait for loads into another
  __shared__ __align__(16) char buf0[TL::kBuf];
  __shared__ __align__(16) char buf1[TL::kBuf];
  __shared__ __align__(16) char buf2[TL::kBuf];
  __shared__ __align__(16) char buf3[TL::kBuf];
  constexpr int W = T / 2;  // a wave's side
  constexpr bool kApplies = M == kApply || M == kLast;

  // neighbouring tiles to one XCD: its L2 then holds the rows they share
  unsigned b = blockIdx.x;
  const unsigned per_xcd = total / kXcds;
  if (b < per_xcd * kXcds) b = (b % kXcds) * per_xcd + b / kXcds;
  int gi = 0;
  while (gi + 1 < gs.n && b >= (kApplies ? gs.g[gi + 1].t_apply : gs.g[gi + 1].t_gram)) ++gi;
  const Group& g = gs.g[gi];
  const bool tall = g.tall();
  const int m = g.m;
  const int crows = kApplies ? g.rp : m, ccols = kApplies ? g.cp : m;  // of C
  int item, ti, tj;
  if constexpr (kApplies) {
    const int tr = (crows + T - 1) / T, tc = (ccols + T - 1) / T;
    const int local = b - g.t_apply;
    item = local / (tr * tc);
    const int t = local % (tr * tc);
    // strips of 8 tile rows, column by column
    constexpr int kStrip = 8;
    const int strip = t / (kStrip * tc), left = tr - strip * kStrip;
    const int high = left < kStrip ? left : kStrip;
    const int s = t - strip * kStrip * tc;
    ti = strip * kStrip + s % high;
    tj = s / high;
  } else {
    const int tm = (m + T - 1) / T, per = tm * (tm + 1) / 2;
    const int local = b - g.t_gram;
    item = local / per;
    const int t = local % per;
    ti = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
  }
  const int r0 = ti * T, c0 = tj * T;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wr = wave >> 1, wc = wave & 1;

  Acc<T> acc = {};
  auto along = [&](const _Float16* Pm, const _Float16* Qm, int k) {
    Operand<T, BK, false> P, Q;
    P.init(Pm, crows, k, r0, wave, lane, wr * W);
    Q.init(Qm, ccols, k, c0, wave, lane, wc * W);
    product<T, BK>(buf0, buf1, buf2, buf3, P, Q, k / BK, wave, acc);
  };
  const _Float16* S = g.S(st.in, item);
  if constexpr (M == kPoly) {
    along(g.A(0, item), g.A(0, item), m);
  } else if constexpr (M == kGram) {
    if (tall) {
      Operand<T, BK, true> P, Q;
      P.init(S, m, m, r0, wave, lane, wr * W);
      Q.init(S, m, m, c0, wave, lane, wc * W);
      product<T, BK>(buf0, buf1, buf2, buf3, P, Q, g.n / BK, wave, acc);
    } else {
      along(S, S, g.n);
    }
  } else {
    if (tall) {
      along(S, g.A(1, item), m);
    } else {
      Operand<T, BK, false> P;
      Operand<T, BK, true> Q;
      P.init(g.A(1, item), m, m, r0, wave, lane, wr * W);
      Q.init(S, ccols, ccols, c0, wave, lane, wc * W);
      product<T, BK>(buf0, buf1, buf2, buf3, P, Q, m / BK, wave, acc);
    }
  }

  // Epilogue, 64 rows at a time: accumulators to LDS as binary32, then row by
  // row (8 columns a thread) the additions and the store; gram and poly store
  // the mirrored tile as well.  What the additions read is asked for ahead of
  // the barriers, which wait for LDS alone: nothing else would hide that
  // latency where a block has one wave per SIMD.
  static_assert(32 * T * 4 <= TL::kBuf, "half the slab fits one buffer");
  const Scal sc = g.scal[item];
  const bool cross = !kApplies && ti != tj;
  constexpr int kPerRow = T / 8, kRowsAtOnce = kBlock / kPerRow, kPasses = 64 / kRowsAtOnce;
  const int prow = threadIdx.x / kPerRow, pcol = (threadIdx.x % kPerRow) * 8;
  const int gc = c0 + pcol;
  const bool col_in = gc < ccols;
  // the matrix added and the remainders of the product's diagonal
  const _Float16* add = M == kPoly ? g.A(0, item) : S;
  const _Float16* rem = kApplies && st.lo_in ? g.L(item) : nullptr;
  const float* diag = M == kPoly ? g.D(0, item) : g.D(1, item);
  const float alpha = st.first ? sc.gram_first : sc.gram;
  const float fb = st.b * (kScaleB / kScaleA), fc = st.c * (kScaleB / (kScaleA * kScaleA));
  const float fx = (st.first ? sc.apply_first : 1.0f) * (M == kLast ? g.out_scale * sc.inv_sx : 1.0f);
  float dc[8] = {};
  if (M != kGram && col_in && (M == kPoly || tall)) load8(diag + gc, dc);
  lds_barrier();  // the last slice is read
#pragma unroll 1
  for (int sl = 0; sl < T / 64; ++sl) {
    f16x8 ad[kPasses], re[kPasses];
    float dr[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int gr = r0 + sl * 64 + p * kRowsAtOnce + prow;
      const int64_t idx = static_cast<int64_t>(gr) * ccols + gc;
      ad[p] = re[p] = f16x8{};
      dr[p] = 0.0f;
      if (gr < crows && col_in) {
        if constexpr (M != kGram) ad[p] = *reinterpret_cast<const f16x8*>(add + idx);
        if (M == kPoly || (kApplies && !tall)) dr[p] = diag[gr];
        if (kApplies && rem != nullptr) re[p] = *reinterpret_cast<const f16x8*>(rem + idx);
      }
    }
#pragma unroll
    for (int part = 0; part < T / 64; ++part) {
      if (part != sl) continue;
#pragma unroll
      for (int i = 0; i < TL::kSub; ++i) {
        const int rb = wr * TL::kSub + i;  // 32-row block of the tile
        if (rb / 2 == part) {
#pragma unroll
          for (int j = 0; j < TL::kSub; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int row = (rb & 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
              const int col = wc * W + j * 32 + (lane & 31);
              *slab_at<T>(buf0, buf1, row, col) = acc[i][j][e];
            }
        }
      }
    }
    lds_barrier();
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = p * kRowsAtOnce + prow;
      const int gr = r0 + sl * 64 + row;
      if (gr >= crows || !col_in) continue;
      float* at = slab_at<T>(buf0, buf1, row, pcol);
      const int64_t idx = static_cast<int64_t>(gr) * ccols + gc;
      float v[8];
      load8(at, v);
      f16x8 h;
      if constexpr (M == kGram) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = v[q] * alpha;
          h[q] = static_cast<_Float16>(v[q]);
          if (gr == gc + q) g.D(0, item)[gr] = v[q] - static_cast<float>(h[q]);
        }
        *reinterpret_cast<f16x8*>(g.A(0, item) + idx) = h;
      } else if constexpr (M == kPoly) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          // (A + D)^2 = A^2 + D A + A D + D^2 for the diagonal remainder D
          const float x = static_cast<float>(ad[p][q]);
          v[q] = fb * x + fc * (v[q] + (dr[p] + dc[q]) * x);
          if (gr == gc + q) v[q] = v[q] + (fb * dr[p] + fc * (dr[p] * dr[p]));
          h[q] = static_cast<_Float16>(v[q]);
          if (gr == gc + q) g.D(1, item)[gr] = v[q] - static_cast<float>(h[q]);
        }
        *reinterpret_cast<f16x8*>(g.A(1, item) + idx) = h;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          // the diagonal's remainder multiplies S's row (wide) or column (tall)
          const float a = st.a + (dr[p] + dc[q]) * (1.0f / kScaleB);
          const float x =
              static_cast<float>(ad[p][q]) + static_cast<float>(re[p][q]) * (1.0f / kScaleLo);
          v[q] = (a * x + v[q] * (1.0f / kScaleB)) * fx;
        }
        if constexpr (M == kApply) {
#pragma unroll
          for (int q = 0; q < 8; ++q) h[q] = static_cast<_Float16>(v[q]);
          *reinterpret_cast<f16x8*>(g.S(st.in ^ 1, item) + idx) = h;
          if (st.lo_out) {
            f16x8 l;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              l[q] = static_cast<_Float16>((v[q] - static_cast<float>(h[q])) * kScaleLo);
            *reinterpret_cast<f16x8*>(g.L(item) + idx) = l;
          }
        } else if (gr < g.rows) {
          store_out8(g.out + item * g.out_stride + gr * g.out_ld + gc, g.cols - gc, g.out_vec, v);
        }
      }
      if (cross) {
        *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
    lds_barrier();
    if (cross) {
      // 8 threads take the 64 rows of one column, 8 rows each
#pragma unroll
      for (int p = 0; p < T / 32; ++p) {
        const int col = p * 32 + (threadIdx.x >> 3), row = (threadIdx.x & 7) * 8;
        const int gr = r0 + sl * 64 + row, xr = c0 + col;
        if (gr >= m || xr >= m) continue;
        f16x8 h;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          h[q] = static_cast<_Float16>(*slab_at<T>(buf0, buf1, row + q, col));
        *reinterpret_cast<f16x8*>(g.A(M == kGram ? 0 : 1, item) + static_cast<int64_t>(xr) * m +
                                  gr) = h;
      }
      lds_barrier();
    }
  }
}

// ---- host ---------------------------------------------------------------------------

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Matrices run in chunks that share one workspace: at most this many padded
// elements (and kMaxGroups groups), or a single matrix.
constexpr int64_t kChunkElems = int64_t{1} << 28;

struct Piece {
  int32_t group;  // caller's group
  int64_t first, count;
};

struct Chunk {
  std::vector<Piece> pieces;
  int64_t bytes = 0;
};

struct Shape {
  int64_t m, n;  // padded short and long side
  int64_t norm_blocks;
};

Shape shape_of(const sbp_matrices& g) {
  Shape s;
  s.m = up(std::min(g.rows, g.cols), kPad);
  s.n = up(std::max(g.rows, g.cols), kPad);
  const int64_t units = g.rows * ((g.cols + 511) / 512);
  s.norm_blocks = std::max<int64_t>(1, std::min<int64_t>(kMaxNormBlocks, (units + 31) / 32));
  return s;
}

// Bytes one piece takes: fp16 arrays, norm partials, scalars (each 256-B aligned).
int64_t half_bytes(const Shape& s, int64_t count) {
  return up(2 * count * (3 * s.m * s.n + 2 * s.m * s.m), 256);
}
int64_t partial_bytes(const Shape& s, int64_t count) { return up(8 * count * s.norm_blocks, 256); }
int64_t diag_bytes(const Shape& s, int64_t count) { return up(8 * count * s.m, 256); }
int64_t scal_bytes(int64_t count) { return up(static_cast<int64_t>(sizeof(Scal)) * count, 256); }

std::vector<Chunk> chunks_of(const sbp_matrices* groups, int32_t n_groups) {
  std::vector<Chunk> out;
  int64_t room = 0;
  for (int32_t i = 0; i < n_groups; ++i) {
    const sbp_matrices& g = groups[i];
    if (g.rows == 0 || g.cols == 0) continue;
    const Shape s = shape_of(g);
    const int64_t elems = s.m * s.n;
    for (int64_t first = 0; first < g.count;) {
      if (out.empty() || room < elems ||
          static_cast<int>(out.back().pieces.size()) == kMaxGroups) {
        out.emplace_back();
        room = std::max(kChunkElems, elems);
      }
      const int64_t take = std::min(g.count - first, room / elems);
      out.back().pieces.push_back(Piece{i, first, take});
      out.back().bytes += half_bytes(s, take) + partial_bytes(s, take) +
                          diag_bytes(s, take) + scal_bytes(take);
      room -= take * elems;
      first += take;
    }
  }
  return out;
}

// Argument checks of the groups alone (no pointers): shared with the size query.
sbp_status check_shapes(const std::string& w, const sbp_matrices* groups, int32_t n_groups) {
  if (n_groups < 0) return sbp::fail(SBP_EINVAL, w + ": n_groups < 0");
  if (n_groups > 0 && groups == nullptr) return sbp::fail(SBP_EINVAL, w + ": groups is null");
  for (int32_t i = 0; i < n_groups; ++i) {
    const sbp_matrices& g = groups[i];
    if (g.rows < 0 || g.cols < 0 || g.count < 0)
      return sbp::fail(SBP_EINVAL, w + ": negative rows, cols or count");
    if (g.rows > SBP_NS_MAX_DIM || g.cols > SBP_NS_MAX_DIM || g.count > SBP_NS_MAX_DIM)
      return sbp::fail(SBP_ERANGE, w + ": rows, cols or count above SBP_NS_MAX_DIM");
    if (g.rows * g.cols > SBP_NS_MAX_NUMEL)
      return sbp::fail(SBP_ERANGE, w + ": a matrix above SBP_NS_MAX_NUMEL elements");
  }
  return SBP_OK;
}

// A group's elements as a byte range, and the lattice they lie on.
struct Span {
  uintptr_t lo, hi;  // bytes
  int64_t ld, stride, cols, count;
  int32_t group;
  bool out;
  // columns a row of `ld` holds, and whether every matrix starts in the same one
  int64_t width;
  bool aligned_rows;
};

Span span_of(const void* p, const sbp_matrices& g, int64_t ld, int64_t stride, int32_t group,
             bool out) {
  const int64_t between = g.count > 1 ? stride : 0;
  const int64_t all = (g.rows - 1) * ld + g.cols + (g.count - 1) * between;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  Span s{lo, lo + 2 * static_cast<uintptr_t>(all), ld, between, g.cols, g.count, group, out,
         g.cols, between % ld == 0};
  const int64_t beside = (g.count - 1) * between + g.cols;  // matrices next to each other
  if (beside <= ld) {
    s.width = beside;
    s.aligned_rows = true;
  }
  return s;
}

// Whether two groups' elements are disjoint although their ranges overlap:
// column blocks of one buffer with a common row distance.
bool disjoint_columns(const Span& a, const Span& b) {
  if (a.ld != b.ld || !a.aligned_rows || !b.aligned_rows) return false;
  const int64_t ld = a.ld;
  const int64_t bytes = static_cast<int64_t>(b.lo - a.lo);  // a.lo <= b.lo
  if (bytes % 2) return false;
  const int64_t d = (bytes / 2) % ld;  // b's first column relative to a's
  return a.width <= d && d + b.width <= ld;
}

bool same_place(const Span& a, const Span& b) {
  return a.lo == b.lo && a.ld == b.ld && a.stride == b.stride;
}

sbp_status check_overlap(const std::string& w, std::vector<Span>& spans) {
  std::sort(spans.begin(), spans.end(),
            [](const Span& a, const Span& b) { return a.lo < b.lo; });
  std::vector<const Span*> open;
  for (const Span& s : spans) {
    open.erase(std::remove_if(open.begin(), open.end(),
                              [&](const Span* o) { return o->hi <= s.lo; }),
               open.end());
    for (const Span* o : open) {
      if (!o->out && !s.out) continue;  // two inputs may share memory
      if (o->group == s.group && o->out != s.out && same_place(*o, s)) continue;  // in place
      if (disjoint_columns(*o, s)) continue;
      return sbp::fail(SBP_EINVAL, w + ": an output overlaps another matrix");
    }
    open.push_back(&s);
  }
  return SBP_OK;
}

sbp_status launched(const char* who) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return sbp::fail(SBP_EHIP, std::string(who) + ": launch failed: " + hipGetErrorString(e));
  return SBP_OK;
}

struct Tiles {
  uint32_t gram = 0, apply = 0;
};

// First blocks of every group for tiles of side T; the launches' sizes.
Tiles lay_tiles(Groups& gs, int T) {
  Tiles t;
  for (int i = 0; i < gs.n; ++i) {
    Group& g = gs.g[i];
    const uint32_t tm = (g.m + T - 1) / T, tn = (g.n + T - 1) / T;
    g.t_gram = t.gram;
    g.t_apply = t.apply;
    t.gram += g.count * (tm * (tm + 1) / 2);
    t.apply += g.count * tm * tn;
  }
  return t;
}

template <int T, int BK>
sbp_status run_step(const char* who, const Groups& gs, const Tiles& t, const Step& st,
                    hipStream_t stream) {
  hipLaunchKernelGGL((ns_product_kernel<T, BK, kGram>), dim3(t.gram), dim3(kBlock), 0, stream, gs, st,
                     t.gram);
  hipLaunchKernelGGL((ns_product_kernel<T, BK, kPoly>), dim3(t.gram), dim3(kBlock), 0, stream, gs, st,
                     t.gram);
  if (st.last)
    hipLaunchKernelGGL((ns_product_kernel<T, BK, kLast>), dim3(t.apply), dim3(kBlock), 0, stream, gs,
                       st, t.apply);
  else
    hipLaunchKernelGGL((ns_product_kernel<T, BK, kApply>), dim3(t.apply), dim3(kBlock), 0, stream, gs,
                       st, t.apply);
  return launched(who);
}

sbp_status run_chunk(const char* who, const sbp_matrices* groups, const Chunk& c,
                     const sbp_ns_hparams& hp, char* ws, hipStream_t stream) {
  Groups gs{};
  gs.n = static_cast<int32_t>(c.pieces.size());
  uint32_t norm = 0, pro = 0;
  for (int i = 0; i < gs.n; ++i) {
    const Piece& p = c.pieces[i];
    const sbp_matrices& src = groups[p.group];
    const Shape s = shape_of(src);
    Group& g = gs.g[i];
    g.in = static_cast<const uint16_t*>(src.in) + p.first * src.in_stride;
    g.out = static_cast<uint16_t*>(src.out) + p.first * src.out_stride;
    g.in_ld = src.in_ld;
    g.out_ld = src.out_ld;
    g.in_stride = src.in_stride;
    g.out_stride = src.out_stride;
    g.rows = static_cast<int32_t>(src.rows);
    g.cols = static_cast<int32_t>(src.cols);
    g.count = static_cast<int32_t>(p.count);
    g.rp = static_cast<int32_t>(up(src.rows, kPad));
    g.cp = static_cast<int32_t>(up(src.cols, kPad));
    g.m = static_cast<int32_t>(s.m);
    g.n = static_cast<int32_t>(s.n);
    g.norm_blocks = static_cast<int32_t>(s.norm_blocks);
    g.out_scale = src.out_scale;
    const bool many = p.count > 1;
    g.in_vec = sbp::aligned(g.in, 16) && src.in_ld % 8 == 0 && (!many || src.in_stride % 8 == 0);
    g.out_vec =
        sbp::aligned(g.out, 16) && src.out_ld % 8 == 0 && (!many || src.out_stride % 8 == 0);
    g.base = reinterpret_cast<_Float16*>(ws);
    ws += half_bytes(s, p.count);
    g.partial = reinterpret_cast<double*>(ws);
    ws += partial_bytes(s, p.count);
    g.diag = reinterpret_cast<float*>(ws);
    ws += diag_bytes(s, p.count);
    g.scal = reinterpret_cast<Scal*>(ws);
    ws += scal_bytes(p.count);
    g.t_norm = norm;
    g.t_pro = pro;
    norm += g.count * g.norm_blocks;
    pro += g.count * (g.rp / 32) * (g.cp / 64);
  }
  // |x| grows by at most a factor sum |coefficients| per step while small
  double grow = 0.0;
  for (int s = 0; s < hp.steps; ++s)
    grow += std::log2(std::max(1.0, std::fabs(static_cast<double>(hp.coefs[3 * s]))));
  const int igrow = static_cast<int>(std::min(200.0, std::ceil(grow)));

  hipLaunchKernelGGL(ns_norm_kernel, dim3(norm), dim3(kBlock), 0, stream, gs);
  hipLaunchKernelGGL(ns_prologue_kernel, dim3(pro), dim3(kBlock), 0, stream, gs, hp.eps, igrow);
  sbp_status rc = launched(who);
  if (rc != SBP_OK) return rc;

  // the largest tile that still gives every CU one: fewer bytes read per flop
  int T = 256;
  Tiles t = lay_tiles(gs, T);
  while (T > 64 && t.apply < 256) {
    T /= 2;
    t = lay_tiles(gs, T);
  }
  for (int s = 0; s < hp.steps; ++s) {
    Step st{};
    st.a = hp.coefs[3 * s];
    st.b = hp.coefs[3 * s + 1];
    st.c = hp.coefs[3 * s + 2];
    st.first = s == 0;
    st.last = s == hp.steps - 1;
    st.lo_out = hp.steps - 1 - s >= 3;
    st.lo_in = s > 0 && hp.steps - s >= 3;
    st.in = s & 1;
    rc = T == 256   ? run_step<256, 32>(who, gs, t, st, stream)
         : T == 128 ? run_step<128, 32>(who, gs, t, st, stream)
                    : run_step<64, 64>(who, gs, t, st, stream);
    if (rc != SBP_OK) return rc;
  }
  return SBP_OK;
}

}  // namespace

extern "C" {

int64_t sbp_newton_schulz_workspace(const sbp_matrices* groups, int32_t n_groups) {
  if (check_shapes("sbp_newton_schulz_workspace", groups, n_groups) != SBP_OK) return -1;
  (void)sbp::ok();
  int64_t most = 0;
  for (const Chunk& c : chunks_of(groups, n_groups)) most = std::max(most, c.bytes);
  return most;
}

sbp_status sbp_newton_schulz(const sbp_matrices* groups, int32_t n_groups,
                             const sbp_ns_hparams* hp, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
  const char* who = "sbp_newton_schulz";
  const std::string w(who);
  sbp_status st = check_shapes(w, groups, n_groups);
  if (st != SBP_OK) return st;
  if (hp == nullptr) return sbp::fail(SBP_EINVAL, w + ": hp is null");
  if (hp->steps < 1 || hp->steps > SBP_NS_MAX_STEPS)
    return sbp::fail(SBP_EINVAL, w + ": steps must be in 1..SBP_NS_MAX_STEPS");
  if (!(hp->eps >= 0.0f) || !std::isfinite(hp->eps))
    return sbp::fail(SBP_EINVAL, w + ": eps must be finite and >= 0");
  for (int i = 0; i < 3 * hp->steps; ++i)
    if (!(std::fabs(hp->coefs[i]) <= SBP_NS_MAX_COEF))
      return sbp::fail(SBP_EINVAL, w + ": a coefficient beyond SBP_NS_MAX_COEF");
  std::vector<Span> spans;
  for (int32_t i = 0; i < n_groups; ++i) {
    const sbp_matrices& g = groups[i];
    if (!std::isfinite(g.out_scale))
      return sbp::fail(SBP_EINVAL, w + ": out_scale must be finite");
    if (g.rows == 0 || g.cols == 0 || g.count == 0) continue;
    if (g.in == nullptr || g.out == nullptr)
      return sbp::fail(SBP_EINVAL, w + ": null matrix pointer");
    if (!sbp::aligned(g.in, 2) || !sbp::aligned(g.out, 2))
      return sbp::fail(SBP_EALIGN, w + ": matrices must be 2-byte aligned");
    if (g.in_ld < g.cols || g.out_ld < g.cols)
      return sbp::fail(SBP_EINVAL, w + ": a row distance below cols");
    if (g.in_ld > SBP_NS_MAX_LD || g.out_ld > SBP_NS_MAX_LD)
      return sbp::fail(SBP_ERANGE, w + ": a row distance above SBP_NS_MAX_LD");
    const int64_t out_one = (g.rows - 1) * g.out_ld + g.cols;
    if (g.count > 1) {
      const int64_t most = INT64_MAX / 8 / g.count;
      if (g.in_stride < 0 || g.out_stride < 0)
        return sbp::fail(SBP_EINVAL, w + ": a negative matrix distance");
      if (g.in_stride > most || g.out_stride > most)
        return sbp::fail(SBP_ERANGE, w + ": a matrix distance too large");
      // a group's outputs: one after the other, or side by side in the rows
      const bool apart = g.out_stride >= out_one;
      const bool beside = g.out_stride >= g.cols &&
                          (g.count - 1) * g.out_stride + g.cols <= g.out_ld;
      if (!apart && !beside)
        return sbp::fail(SBP_EINVAL, w + ": a group's outputs overlap each other");
    }
    spans.push_back(span_of(g.in, g, g.in_ld, g.in_stride, i, false));
    spans.push_back(span_of(g.out, g, g.out_ld, g.out_stride, i, true));
  }
  if (spans.empty()) return sbp::ok();  // nothing is read or written
  st = check_overlap(w, spans);
  if (st != SBP_OK) return st;
  const std::vector<Chunk> chunks = chunks_of(groups, n_groups);
  int64_t need = 0;
  for (const Chunk& c : chunks) need = std::max(need, c.bytes);
  if (workspace == nullptr) return sbp::fail(SBP_EINVAL, w + ": workspace is null");
  if (!sbp::aligned(workspace, 256))
    return sbp::fail(SBP_EALIGN, w + ": workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return sbp::fail(SBP_EINVAL, w + ": workspace too small (see sbp_newton_schulz_workspace)");
  const uintptr_t wlo = reinterpret_cast<uintptr_t>(workspace);
  for (const Span& s : spans)
    if (s.lo < wlo + static_cast<uintptr_t>(need) && wlo < s.hi)
      return sbp::fail(SBP_EINVAL, w + ": the workspace overlaps a matrix");
  (void)hipGetLastError();
  for (const Chunk& c : chunks) {
    st = run_chunk(who, groups, c, *hp, static_cast<char*>(workspace), stream);
    if (st != SBP_OK) return st;
  }
  return sbp::ok();
}

}  // extern "C"
