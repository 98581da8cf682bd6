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
// across, and is read from LDS with the transposing reads of gfx950, so that X
// is kept, and written by apply, in one orientation only.
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
// output's rounding (1.7e-3 by itself): 4e-4 .. 1.0e-3 for noise, and for strong
// directions over noise of their size; up to 2.5e-3 where the noise is weaker
// and its directions come up from next to nothing within the steps (rank 16
// plus 0.03: 1.7e-3, plus 0.003: 2.4e-3).  Without the diagonals' remainders up
// to 2.2e-3 for noise, without either up to 2.6e-2, with bf16 products 7e-3 ..
// 2e-1.
// Where all entries are alike their roundings are too, and do not average out:
// up to 1e-2.
// The squared norm: above a short side of 128 in float64; up to it the trace of
// the first Gram matrix, whose sums are binary32 (at the longest sides 1024 in a
// row a block, then 64 blocks': within 7e-5).  Both in a fixed order, so results
// are the same from run to run.
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
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256;
constexpr int kXcds = 8;
constexpr int kPad = 64;        // both padded sides are multiples of this
constexpr int kMaxGroups = 16;  // groups of equal matrices per launch
constexpr int kMaxNormBlocks = 256;
constexpr int kLogX = 12;       // X is stored times 2^12
constexpr float kScaleA = 4096.0f, kScaleB = 1024.0f, kScaleLo = 2048.0f;

// Per-matrix scalars, written by the prologue.
// Stored X_0 = X_0 / rho, stored X_k = X_k * sx for k >= 1.
struct Scal {
  float gram_first, gram;  // accumulator -> stored A: rho^2 * 2^12, 2^12 / sx^2
  float apply_first;       // step 1's accumulator -> stored X_1: rho * sx
  int32_t log_sx;
};

// One group: `count` matrices of one shape, at equal distances.
struct Group {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_ld, out_ld, in_stride, out_stride;
  _Float16* base;    // S, S2, L (count*m*n each), A, B (count*m*m each);
                     // short side of at most 128: S, L
  double* partial;   // count * norm_blocks
  Scal* scal;        // count
  float* diag;       // m each: count for A, count for B (rounding remainders)
  int32_t rows, cols, count;
  int32_t rp, cp;    // rows and cols padded
  int32_t m, n;      // the smaller and the larger of rp and cp
  int32_t norm_blocks;
  // out_scale = out_frac * 2^out_exp, the former in [1/2, 1) or 0: the power of
  // two is applied last, with X's, so that no factor leaves binary32's range
  float out_frac;
  int32_t out_exp;
  int32_t in_vec, out_vec;  // 16-byte rows
  uint32_t t_norm, t_pro, t_gram, t_apply;  // first block of the group in each launch
  // short side of at most 128 only: blocks per matrix; their partial Gram
  // matrices (twice, for steps in turn) and the powers of two of the first;
  // whether a kernel sums those, into the first of them, between the steps
  int32_t splits;
  int32_t summed;
  float* parts;
  int32_t* part_ks;

  __host__ __device__ bool tall() const { return rows > cols; }
  __device__ int64_t mn() const { return static_cast<int64_t>(m) * n; }
  __device__ _Float16* S(int which, int item) const {
    return base + (static_cast<int64_t>(which) * count + item) * mn();
  }
  __device__ _Float16* L(int item) const {
    return base + (static_cast<int64_t>(splits > 0 ? 1 : 2) * count + item) * mn();
  }
  __device__ float* D(int which, int item) const {
    return diag + (static_cast<int64_t>(which) * count + item) * m;
  }
  __device__ float* part(int which, int item, int split) const {
    return parts + ((static_cast<int64_t>(which) * count + item) * splits + split) * m * m;
  }
  __device__ int32_t* part_k(int item, int split) const {  // [splits]: the sum's
    return part_ks + static_cast<int64_t>(item) * (splits + 1) + split;
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
  float a, b, c;
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
  auto one = [&](int j) -> uint32_t {  // element 0 exists: no branches
    const uint32_t x = p[j < left ? j : 0];
    return j < left ? x : 0u;
  };
  return u32x4{one(0) | one(1) << 16, one(2) | one(3) << 16, one(4) | one(5) << 16,
               one(6) | one(7) << 16};
}

// 8 bf16 values times 2^k in fp16.
__device__ __forceinline__ f16x8 half8(u32x4 w, int k) {
  auto lo = [&](uint32_t x) { return static_cast<_Float16>(ldexpf(sbp::bf16_lo(x), k)); };
  auto hi = [&](uint32_t x) { return static_cast<_Float16>(ldexpf(sbp::bf16_hi(x), k)); };
  return f16x8{lo(w.x), hi(w.x), lo(w.y), hi(w.y), lo(w.z), hi(w.z), lo(w.w), hi(w.w)};
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

// How a matrix of this norm is stored: X_0 = U * 2^k with the norm in [2^13,
// 2^14) (k = 0 for a zero, infinite or NaN norm), X_0 = stored * rho, later
// X = stored / sx.
struct Norm {
  int k, log_sx;
  double floor_norm, rho, sx;
};
__device__ __forceinline__ Norm norm_of(double norm, float eps, int grow) {
  Norm r;
  const bool plain = norm > 0.0 && norm < __builtin_huge_val();
  r.k = plain ? 13 - ilogb(norm) : 0;
  r.floor_norm = norm < eps ? static_cast<double>(eps) : norm;  // NaN stays
  int below = plain && norm < eps ? ilogb(static_cast<double>(eps)) - ilogb(norm) : 0;
  below = below > grow + 2 ? below - grow - 2 : 0;
  r.rho = 1.0 / (r.floor_norm * ldexp(1.0, r.k));
  r.log_sx = kLogX + below;  // below 300: from bf16's least to binary32's largest
  r.sx = ldexp(1.0, r.log_sx);
  return r;
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
  const Norm nm = norm_of(sqrt(block_sum_all(sq)), eps, grow);
  if (t == 0 && threadIdx.x == 0)
    g.scal[item] = Scal{static_cast<float>(nm.rho * nm.rho * kScaleA),
                        static_cast<float>(kScaleA / (nm.sx * nm.sx)),
                        static_cast<float>(nm.rho * nm.sx), nm.log_sx};
  const f16x8 h = half8(w, nm.k);
  *reinterpret_cast<f16x8*>(g.S(0, item) + static_cast<int64_t>(row) * g.cp + col) = h;
}

// ---- the product ------------------------------------------------------------------

// Tiles of side T of the lower triangle of an m x m matrix.
__host__ __device__ __forceinline__ int lower_tiles(int m, int T) {
  const int side = (m + T - 1) / T;
  return side * (side + 1) / 2;
}

// kApplyLo: apply where S's remainder is read or stored; kLast: to the caller's
// matrices, after the steps that keep one.
enum Mode { kGram, kPoly, kApplyLo, kApply, kLast };

// One T x T tile of C = P Q' per block of 4 waves (2 x 2, each a quarter, in
// 16 x 16 MFMA tiles, so that 32 k are one round of products).  Slices of BK k
// elements go straight from memory to one of NB LDS buffers, NB slices ahead.
// Rows along k come by lines of 128 bytes, which 64 elements use whole; with 32
// each line passes the CU's cache twice (tile 128, half a round of 256-tiles of
// k = 4096: 106 us, with 64 80 us).  At the largest tile two slices of 64 are all
// of LDS, and their loads come in bursts that are not hidden where k is long
// (three of 14336 x 4096: gram 707 us, with four slices of 32 613; apply 1200
// and 1225), so it takes 32.
// What bounds it: at 256 the main loop keeps the matrix units 78 to 84% busy, at
// the clock of 1.85 GHz that full load leaves; a tile's epilogue adds about 20 us
// to the 90 of k = 4096, as all CUs reach it together and read and write their
// tiles of S at once.  Three of 14336 x 4096: gram 1.25 PFLOP/s of what it
// computes, apply 1.15; of 4096 x 14336: 1.13 and 1.25.
template <int T_>
struct Tile {
  static constexpr int T = T_, BK = T == 256 ? 32 : 64;
  static constexpr int NB = T == 128 ? 2 : 4;  // slices in LDS
  static constexpr int kHalf = T * BK * 2;  // one operand's slice, bytes
  static constexpr int kBuf = 2 * kHalf;    // P, then Q
  static constexpr int kSub = T / 32;       // 16 x 16 tiles per wave and side
  static constexpr int kPhases = BK / 32;
  static constexpr int kLoads = kHalf / 4096;  // per operand, slice and lane
  static_assert(32 * T * 4 <= kBuf, "half the epilogue's slab fits one buffer");
};

// `bytes` from p on as a buffer; loads from beyond them give zeros, stores do
// nothing.  An access is held to `bytes - scalar offset`, unsigned, so a scalar
// offset past the end would lift the bound: whole offsets go into the vector
// one, and the scalar one stays 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
template <typename V>
__device__ __forceinline__ V load16(__amdgpu_buffer_rsrc_t from, int off) {
  return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(from, off, 0, 0));
}
template <typename V>
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t to, V v, int off) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), to, off, 0, 0);
}

// One operand of a tile.  Along: the matrix's rows r0 .. are the operand's
// rows, and a slice is BK consecutive elements of each; LDS keeps a row's
// 16-byte pieces rotated by row.  Across: the matrix's columns r0 .. are the
// operand's rows, and a slice is BK rows of T elements; LDS keeps a row's
// 32-byte pieces rotated by row, and the reads transpose.  Both rotations come
// from the lanes' global addresses and spread the reads over the banks.
// Rows past the matrix read as zero or as a neighbour: they only reach
// results that are not stored.
template <int T, int BK, bool ACROSS>
struct Operand {
  static constexpr int kSub = T / 32, kPhases = BK / 32;
  const char* from;  // next slice to load
  int64_t step;
  int bytes, round_bytes;
  int voff[2];                       // of even and odd rounds
  int at;                            // LDS offset of this lane's first fragment
  int off[ACROSS ? kSub : kPhases];  // further offset by sub-tile or phase

  __device__ __forceinline__ void init(const _Float16* mat, int rows, int ld, int r0, int wave,
                                       int lane, int wrow) {
    if constexpr (ACROSS) {
      constexpr int kLanes = T / 8;  // lanes per row
      from = reinterpret_cast<const char*>(mat + r0);
      step = static_cast<int64_t>(BK) * ld * 2;
      bytes = (BK * ld - r0) * 2;
      constexpr int kRows = 64 / kLanes;  // per wave and round
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = (r * 4 + wave) * kRows + lane / kLanes;
        voff[r] = row * ld * 2 + (((lane % kLanes) * 16) ^ (turn(row) * 32)) - r * 4 * kRows * ld * 2;
      }
      round_bytes = 4 * (64 / kLanes) * ld * 2;
      const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);  // of this lane's address
      at = k * (T * 2) + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < kSub; ++i) off[i] = ((wrow / 16 + i) ^ turn(k)) * 32;
    } else {
      constexpr int kLanes = BK / 8;
      from = reinterpret_cast<const char*>(mat + static_cast<int64_t>(r0) * ld);
      step = BK * 2;
      const int have = rows - r0 < T ? rows - r0 : T;
      bytes = have * ld * 2;
      const int row = wave * (64 / kLanes) + lane / kLanes;
      voff[0] = voff[1] = row * ld * 2 + ((lane % kLanes) ^ turn(row)) * 16;
      round_bytes = 4 * (64 / kLanes) * ld * 2;
      at = (wrow + (lane & 15)) * (BK * 2);
#pragma unroll
      for (int p = 0; p < kPhases; ++p) off[p] = ((p * 4 + (lane >> 4)) ^ turn(lane & 15)) * 16;
    }
  }
  // The rotation of a row.  Along, rows that differ by 16 agree; across, those
  // that differ by 4 (of a group of 8) and by 16.
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (ACROSS)
      return T >= 128 ? (row & 3) | ((row >> 3) & 1) << 2 : ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
    else
      return BK == 32 ? ((row >> 1) ^ (row >> 2)) & 2 | ((row >> 3) ^ (row >> 1)) & 1 : row & 7;
  }
  __device__ __forceinline__ void load_round(char* buf, int wave, int r) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        buffer(from, bytes),
        (__attribute__((address_space(3))) void*)(buf + (r * 4 + wave) * 1024), 16,
        voff[r & 1] + r * round_bytes, 0, 0, 0);
  }
  // Along, the last rows' slices end before `bytes` does by what is consumed.
  __device__ __forceinline__ void advance() {
    from += step;
    if constexpr (!ACROSS) bytes -= BK * 2;
  }
  __device__ __forceinline__ void load(char* buf, int wave) {
#pragma unroll
    for (int r = 0; r < T * BK * 2 / 4096; ++r) load_round(buf, wave, r);
    advance();
  }
  __device__ __forceinline__ f16x8 read(const char* buf, int phase, int i) const {
    if constexpr (ACROSS) {
      typedef __fp16 h4 __attribute__((__vector_size__(8)));
      typedef __attribute__((address_space(3))) h4* lds_h4;
      const char* p = buf + at + off[i] + phase * 32 * (T * 2);
      const h4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)p);
      const h4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)(p + 4 * (T * 2)));
      return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const f16x8*>(buf + at + off[phase] + i * 16 * (BK * 2));
    }
  }
};

template <typename TL>
struct Frags {
  f16x8 p[TL::kSub], q[TL::kSub];
};

template <typename TL>
using Acc = f32x4[TL::kSub][TL::kSub];

template <typename TL>
__device__ __forceinline__ void multiply(const Frags<TL>& f, Acc<TL>& acc) {
#pragma unroll
  for (int i = 0; i < TL::kSub; ++i)
#pragma unroll
    for (int j = 0; j < TL::kSub; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.p[i], f.q[j], acc[i][j], 0, 0, 0);
}

// The same for one accumulator, in its registers: at the large tile all 256 are
// taken, and the compiler, free to give a product another place than its
// summand, moved them about between the products (13% of apply).  It does not
// see these as matrix instructions, so the wait states that it would fill in are
// kept by hand:
// - an accumulator is read or written by anything else 19 or more wait states
//   after its last product (18 is the longest any needs): settle() ends every
//   run of products, before the first way out of it, since moves may stand
//   wherever two ways meet;
// - a fragment or accumulator is written by a vector instruction 5 or more before
//   a product reads it (2 are needed): fragments come from LDS, whose reads the
//   compiler waits for, and the accumulators' zeros are settled too;
// - a product's own accumulator is used again 64 products later.
// That a build keeps both distances, on every path, is what
// tests/test_matrix_unit_hazards.py reads from its disassembly.
template <bool FIRST>
__device__ __forceinline__ void multiply_in_place(f32x4& c, f16x8 p, f16x8 q) {
  if constexpr (FIRST)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "=a"(c) : "v"(p), "v"(q));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(p), "v"(q));
}
template <typename TL>
__device__ __forceinline__ void settle(Acc<TL>& acc) {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < TL::kSub; ++i)
#pragma unroll
    for (int j = 0; j < TL::kSub; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
}

// Order of a phase's instructions: MFMAs, LDS reads and loads to LDS in turn,
// so that both kinds of memory work run under the MFMAs.
template <typename TL, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
  constexpr int mfmas = TL::kSub * TL::kSub;
#pragma unroll
  for (int i = 0; i < mfmas; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int kOver = mfmas > 8 ? mfmas * 3 / 4 : mfmas;
    const int a = i < kOver ? i : kOver, z = i + 1 < kOver ? i + 1 : kOver;
    const int r = z * READS / kOver - a * READS / kOver, l = z * LOADS / kOver - a * LOADS / kOver;
    if (r == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (r == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    if (r == 3) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
    if (r == 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
    if (l == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if (l == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// All of this wave's loads but the newest LEFT are done, and its LDS reads;
// then everyone's.
template <int LEFT>
__device__ __forceinline__ void slice_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | ((LEFT >> 4) << 14) | 0x70);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// This wave's LDS reads are done.
__device__ __forceinline__ void lds_wait() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}

// This wave's LDS work is done, then everyone's; loads and stores run on.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// acc = P Q' over `slices` slices.  early() issues EARLY loads of the
// epilogue's, once all slices are loaded or under way.
template <typename TL, int EARLY, bool PX, bool QX, typename F>
__device__ __forceinline__ void product(char* (&buf)[TL::NB],
                                        Operand<TL::T, TL::BK, PX>& P,
                                        Operand<TL::T, TL::BK, QX>& Q, int slices, int wave,
                                        Acc<TL>& acc, F&& early) {
  constexpr int T = TL::T, NB = TL::NB, N = TL::kPhases, L = TL::kLoads, kSub = TL::kSub;
  constexpr int kReads = kSub * ((PX ? 2 : 1) + (QX ? 2 : 1));
  constexpr std::true_type kYes{};
  constexpr std::false_type kNo{};
  Frags<TL> f[2];
  auto load = [&](char* to) {
    P.load(to, wave);
    Q.load(to + TL::kHalf, wave);
  };
  auto read = [&](const char* from, int phase, Frags<TL>& to) {
#pragma unroll
    for (int i = 0; i < kSub; ++i) to.p[i] = P.read(from, phase, i);
#pragma unroll
    for (int j = 0; j < kSub; ++j) to.q[j] = Q.read(from + TL::kHalf, phase, j);
  };
  // Products of f[h], under which the other half's fragments are read (READ:
  // phase `phase` of `from`) and a slice is loaded into `to` (LOAD).  The first
  // ones (FIRST) start the sums.
  auto multiplies = [&](int h, const char* from, int phase, char* to, auto read_c, auto load_c,
                        auto first_c) {
    constexpr bool kRead = decltype(read_c)::value, kLoad = decltype(load_c)::value;
    if constexpr (T == 256) {
#pragma unroll
      for (int t = 0; t < kSub * kSub; ++t) {
        multiply_in_place<decltype(first_c)::value>(acc[t / kSub][t % kSub], f[h].p[t / kSub],
                                                    f[h].q[t % kSub]);
        if (kRead && t % 3 == 0 && t / 3 < 2 * kSub) {
          const int c = t / 3;
          if (c < kSub) f[h ^ 1].p[c] = P.read(from, phase, c);
          else f[h ^ 1].q[c - kSub] = Q.read(from + TL::kHalf, phase, c - kSub);
        }
        if (kLoad && t % 6 == 2 && t / 6 < 2 * L) {
          const int r = t / 6;
          if (r < L) P.load_round(to, wave, r);
          else Q.load_round(to + TL::kHalf, wave, r - L);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (kLoad) {
        P.advance();
        Q.advance();
      }
    } else {
      if constexpr (kLoad) load(to);
      if constexpr (kRead) read(from, phase, f[h ^ 1]);
      multiply<TL>(f[h], acc);
      interleave<TL, kRead ? kReads : 0, kLoad ? 2 * L : 0>();
    }
  };
  // One slice, in buf[i], its first fragments in f[0] (of slices of one phase:
  // of odd ones in f[1]).  Before its last phase all of it is in registers and
  // the next slice has to be there (but for LEFT newer loads; -1: no next one),
  // so its buffer is loaded anew (LOAD) with the slice NB further on.
  auto slice = [&](int i, auto load_c, auto left_c, auto first_c) {
    constexpr int kLeft = decltype(left_c)::value;
    const int h = N == 1 ? i & 1 : 1;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (N == 2) multiplies(0, buf[i], 1, nullptr, kYes, kNo, first_c);
    std::conditional_t<N == 1, decltype(first_c), std::false_type> starts;
    if constexpr (kLeft >= 0) {
      slice_barrier<kLeft>();
      multiplies(h, buf[(i + 1) % NB], 0, buf[i], kYes, load_c, starts);
    } else {
      lds_wait();
      multiplies(h, nullptr, 0, nullptr, kNo, kNo, starts);
    }
  };
  // the last slices, of which the last is in the last buffer
  auto tail = [&](auto self, auto i_c) {
    constexpr int i = decltype(i_c)::value;
    if constexpr (i < NB) {
      constexpr int kLeft = i == NB - 1 ? -1 : (NB - 2 - i) * 2 * L + EARLY;
      slice(i, kNo, std::integral_constant<int, kLeft>{}, kNo);
      self(self, std::integral_constant<int, i + 1>{});
    }
  };
  constexpr std::integral_constant<int, (NB - 2) * 2 * L> kSteady{};
  constexpr std::integral_constant<int, (NB - 1) * 2 * L> kStart{};
  static_assert(NB * 2 * L + EARLY < 64, "what vmcnt can count");
  // There is one way into the loop's rounds of NB slices and one way out; a
  // number that is no multiple of NB starts further on, and drains its loads
  // once (known to the compiler, whose own waits in the loop would else provide
  // for the other way in).  At least 3 slices: both padded sides are multiples
  // of 64 and more than 128.
  const int rest = static_cast<unsigned>(slices) % NB;
  if (NB > 192 / TL::BK && slices < NB) {
#pragma unroll
    for (int i = NB - 3; i < NB; ++i) load(buf[i]);
    slice_barrier<0>();
    read(buf[NB - 3], 0, f[0]);
    early();
    tail(tail, std::integral_constant<int, NB - 3>{});
  } else {
    if (rest == 0) {
#pragma unroll
      for (int i = 0; i < NB; ++i) load(buf[i]);
      if constexpr (T == 256) settle<TL>(acc);
      slice_barrier<kStart>();
      read(buf[0], 0, f[0]);
    } else {
#pragma unroll
      for (int r = 1; r < NB; ++r) {  // r slices before the rounds
        // slices of 32 come in pairs: both padded sides are multiples of 64
        if (rest != r || (TL::BK == 32 && r % 2 == 1)) continue;
#pragma unroll
        for (int i = 0; i < NB; ++i) load(buf[(NB - r + i) % NB]);
        slice_barrier<kStart>();
        read(buf[NB - r], 0, f[N == 1 ? r & 1 : 0]);
#pragma unroll
        for (int i = NB - r; i < NB; ++i) {
          if (i == NB - r) slice(i, kYes, kSteady, kYes);
          else slice(i, kYes, kSteady, kNo);
        }
        // the compiler places moves where the ways in join
        if constexpr (T == 256) settle<TL>(acc);
      }
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    }
    for (int s = slices / NB; s > 1; --s) {
#pragma unroll
      for (int i = 0; i < NB; ++i) slice(i, kYes, kSteady, kNo);
    }
    early();
    tail(tail, std::integral_constant<int, 0>{});
  }
  if constexpr (T == 256) settle<TL>(acc);
}

// Up to 8 consecutive bf16 values of a row of the caller's output.
__device__ __forceinline__ void store_bits8(uint16_t* p, int left, bool vec, u32x4 w) {
  if (vec && left >= 8) {
    *reinterpret_cast<u32x4*>(p) = w;
  } else {
    auto one = [&](int j, uint32_t x) {
      if (j < left) p[j] = static_cast<uint16_t>(x);
    };
    one(0, w.x), one(1, w.x >> 16), one(2, w.y), one(3, w.y >> 16);
    one(4, w.z), one(5, w.z >> 16), one(6, w.w), one(7, w.w >> 16);
  }
}
__device__ __forceinline__ void store_out8(uint16_t* p, int left, bool vec, const float (&v)[8],
                                           int exp) {
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  bf16x8 b;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    b[q] = static_cast<__bf16>(ldexpf(v[q], exp));  // nearest, ties to even
  store_bits8(p, left, vec, __builtin_bit_cast(u32x4, b));
}

// Where (row, col) of the epilogue's binary32 slab is kept: 32 rows in
// each of two buffers; groups of 8 columns are rotated by the row's 8-row
// group, so that both a row's 8 columns and a column's 8 rows are read without
// bank conflicts, and halves of 64 by its 4-row group, whose rows one
// instruction writes two of.
template <typename TL>
__device__ __forceinline__ float* slab_at(char* lo, char* hi, int row, int col) {
  float* half = reinterpret_cast<float*>(row & 32 ? hi : lo);
  const int turned =
      col ^ (((row >> 3) & 1) << 4) ^ (((row >> 4) & 1) << 3) ^ ((((row >> 5) ^ (row >> 2)) & 1) << 5);
  return half + (row & 31) * TL::T + turned;
}

// SUB: the blocks' tiles are the quarters of tiles of twice the side, from tile
// `from` on.
template <typename TL, Mode M, bool SUB>
__global__ void __launch_bounds__(kBlock, TL::T == 256 ? 1 : 2)
ns_product_kernel(Groups gs, Step st, unsigned total, unsigned from) {
  constexpr int T = TL::T, BK = TL::BK, PT = SUB ? 2 * T : T;
  // separate arrays: reads of one do not wait for loads into another
  __shared__ __align__(16) char buf0[TL::kBuf];
  __shared__ __align__(16) char buf1[TL::kBuf];
  char* buf[TL::NB];
  buf[0] = buf0;
  buf[1] = buf1;
  if constexpr (TL::NB == 4) {
    __shared__ __align__(16) char buf2[TL::kBuf];
    __shared__ __align__(16) char buf3[TL::kBuf];
    buf[2] = buf2;
    buf[3] = buf3;
  }
  constexpr bool kApplies = M == kApplyLo || M == kApply || M == kLast;

  // neighbouring tiles to one XCD: its L2 then holds the rows they share
  unsigned b = blockIdx.x;
  const unsigned per_xcd = total / kXcds;
  if (b < per_xcd * kXcds) b = (b % kXcds) * per_xcd + b / kXcds;
  const unsigned quarter = b & 3;
  if constexpr (SUB) b = from + b / 4;
  int gi = 0;
  while (gi + 1 < gs.n && b >= (kApplies ? gs.g[gi + 1].t_apply : gs.g[gi + 1].t_gram)) ++gi;
  const Group& g = gs.g[gi];
  const bool tall = g.tall();
  const int m = g.m;
  const int crows = kApplies ? g.rp : m, ccols = kApplies ? g.cp : m;  // of C
  int item, ti, tj;
  if constexpr (kApplies) {
    const int tr = (crows + PT - 1) / PT, tc = (ccols + PT - 1) / PT;
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
    const int per = lower_tiles(m, PT);
    const int local = b - g.t_gram;
    item = local / per;
    const int t = local % per;
    ti = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
  }
  if constexpr (SUB) {
    ti = 2 * ti + (quarter >> 1);
    tj = 2 * tj + (quarter & 1);
    if (ti * T >= crows || tj * T >= ccols || (!kApplies && tj > ti)) return;
  }
  const int r0 = ti * T, c0 = tj * T;  // inside C
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wr = wave >> 1, wc = wave & 1;

  // The epilogue goes by a slab of rows at a time: accumulators to LDS as
  // binary32, then row by row (8 columns a thread) the additions and the store;
  // gram and poly store the mirrored tile as well.  Its barriers wait for LDS
  // alone, what the additions read is asked for a slab ahead, and for the first
  // slab under the last products: a block has one wave per SIMD at the large
  // tile, so nothing else would hide that latency.
  constexpr int kSlab = 64;
  constexpr int kPerRow = T / 8, kRowsAtOnce = kBlock / kPerRow, kPasses = kSlab / kRowsAtOnce;
  const int prow = threadIdx.x / kPerRow, pcol = (threadIdx.x % kPerRow) * 8;
  const int gc = c0 + pcol;
  const bool cross = !kApplies && ti != tj;
  const _Float16* S = g.S(st.in, item);
  // C's rows r0 .. as buffers: rows and columns past the matrix are not
  // touched (columns by an offset of the buffers' end)
  const int have = crows - r0 < T ? crows - r0 : T;  // 1 .. T
  const int64_t tile_at = static_cast<int64_t>(r0) * ccols;
  const int tile_bytes = have * ccols * 2;
  const int row_off = gc < ccols ? (prow * ccols + gc) * 2 : tile_bytes;
  const auto add = buffer(M == kPoly ? g.A(0, item) + tile_at : S + tile_at, tile_bytes);
  const auto rem = buffer(g.L(item) + tile_at, st.lo_in ? tile_bytes : 0);  // else zeros
  const auto rem_out = buffer(g.L(item) + tile_at, st.lo_out ? tile_bytes : 0);
  const auto out = buffer((M == kGram   ? g.A(0, item)
                           : M == kPoly ? g.A(1, item)
                                        : g.S(st.in ^ 1, item)) + tile_at, tile_bytes);
  // the remainders of the product's diagonal: by row, by column, or (poly) both
  const float* diag = M == kPoly ? g.D(0, item) : g.D(1, item);
  const bool by_row = M == kPoly || !tall, by_col = M == kPoly || tall;
  const auto diag_row = buffer(diag + r0, by_row ? have * 4 : 0);
  const auto diag_col = buffer(diag, by_col ? m * 4 : 0);
  f16x8 ad[kPasses], re[kPasses];
  float dr[kPasses], dc[8];
  auto ask = [&](int sl, int p) {
    const int row = sl * kSlab + p * kRowsAtOnce;
    if constexpr (M != kGram) {
      ad[p] = load16<f16x8>(add, row_off + row * ccols * 2);
      dr[p] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(diag_row, (prow + row) * 4, 0, 0));
    }
  };
  auto ask_rem = [&](int sl, int p) {
    if constexpr (M == kApplyLo)
      re[p] = load16<f16x8>(rem, row_off + (sl * kSlab + p * kRowsAtOnce) * ccols * 2);
  };
  // (the large tile has no registers left for it)
  constexpr bool kAhead = M != kGram && T < 256;
  constexpr int kEarly = kAhead ? 2 + kPasses * 2 : 0;
  auto ask_first = [&] {
    if constexpr (M != kGram) {
      const int at = gc < ccols ? gc * 4 : m * 4;
      const f32x4 lo = load16<f32x4>(diag_col, at), hi = load16<f32x4>(diag_col, at + 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        dc[q] = lo[q];
        dc[4 + q] = hi[q];
      }
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) ask(0, p);
  };
  auto early = [&] {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kAhead) ask_first();
    __builtin_amdgcn_sched_barrier(0);
  };

  Acc<TL> acc = {};
  auto along = [&](const _Float16* Pm, const _Float16* Qm, int k) {
    Operand<T, BK, false> P;
    Operand<T, BK, false> Q;
    P.init(Pm, crows, k, r0, wave, lane, wr * (T / 2));
    Q.init(Qm, ccols, k, c0, wave, lane, wc * (T / 2));
    product<TL, kEarly>(buf, P, Q, k / BK, wave, acc, early);
  };
  if constexpr (M == kPoly) {
    along(g.A(0, item), g.A(0, item), m);
  } else if constexpr (M == kGram) {
    if (tall) {
      Operand<T, BK, true> P;
      Operand<T, BK, true> Q;
      P.init(S, m, m, r0, wave, lane, wr * (T / 2));
      Q.init(S, m, m, c0, wave, lane, wc * (T / 2));
      product<TL, kEarly>(buf, P, Q, g.n / BK, wave, acc, early);
    } else {
      along(S, S, g.n);
    }
  } else {
    if (tall) {
      along(S, g.A(1, item), m);
    } else {
      Operand<T, BK, false> P;
      Operand<T, BK, true> Q;
      P.init(g.A(1, item), m, m, r0, wave, lane, wr * (T / 2));
      Q.init(S, ccols, ccols, c0, wave, lane, wc * (T / 2));
      product<TL, kEarly>(buf, P, Q, m / BK, wave, acc, early);
    }
  }

  const Scal sc = g.scal[item];
  const float alpha = st.first ? sc.gram_first : sc.gram;
  const float fb = st.b * (kScaleB / kScaleA), fc = st.c * (kScaleB / (kScaleA * kScaleA));
  // apply: a x + acc / 2^10, scaled; the factors carry the scale
  const float fx = (st.first ? sc.apply_first : 1.0f) * (M == kLast ? g.out_frac : 1.0f);
  const int out_exp = g.out_exp - sc.log_sx;
  const float fd = fx * (1.0f / kScaleB), fa = fx * st.a;
  if constexpr (!kAhead) ask_first();
#pragma unroll
  for (int p = 0; p < kPasses; ++p) ask_rem(0, p);
  lds_barrier();  // the last slice is read
  if constexpr (kApplies) {
#pragma unroll
    for (int q = 0; q < 8; ++q) dc[q] = fmaf(dc[q], fd, fa);
  }
#pragma unroll 1
  for (int sl = 0; sl < T / kSlab; ++sl) {
#pragma unroll
    for (int part = 0; part < T / kSlab; ++part) {
      if (part != sl) continue;
#pragma unroll
      for (int i = 0; i < TL::kSub; ++i) {
        const int rb = wr * TL::kSub + i;  // 16-row block of the tile
        if (rb / (kSlab / 16) == part) {
#pragma unroll
          for (int j = 0; j < TL::kSub; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = rb * 16 % kSlab + 4 * (lane >> 4) + e;
              const int col = wc * (T / 2) + j * 16 + (lane & 15);
              *slab_at<TL>(buf0, buf1, row, col) = acc[i][j][e];
            }
        }
      }
    }
    lds_barrier();
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = p * kRowsAtOnce + prow;
      const int gr = r0 + sl * kSlab + row;
      const int off = (sl * kSlab + p * kRowsAtOnce) * ccols * 2;
      float* at = slab_at<TL>(buf0, buf1, row, pcol);
      float v[8];
      load8(at, v);
      f16x8 h;
      if constexpr (M == kGram) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = v[q] * alpha;
      } else if constexpr (M == kPoly) {
        // (A + D)^2 = A^2 + D A + A D + D^2 for the diagonal remainder D
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float x = static_cast<float>(ad[p][q]);
          v[q] = fmaf(fc, fmaf(dr[p] + dc[q], x, v[q]), fb * x);
        }
        if (!cross) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (gr == gc + q) v[q] = v[q] + (fb * dr[p] + fc * (dr[p] * dr[p]));
        }
      } else {
        // the diagonal's remainder multiplies S's row (wide) or column (tall)
        const float d = fmaf(dr[p], fd, fa);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float x = static_cast<float>(ad[p][q]);
          if constexpr (M == kApplyLo)
            x = fmaf(static_cast<float>(re[p][q]), 1.0f / kScaleLo, x);
          v[q] = fmaf(tall ? dc[q] : d, x, v[q] * fd);
        }
      }
      if (sl + 1 < T / kSlab) {
        ask(sl + 1, p);
        ask_rem(sl + 1, p);
      }
      if constexpr (M == kLast) {
        if (gr < g.rows && gc < g.cols)
          store_out8(g.out + item * g.out_stride + gr * g.out_ld + gc, g.cols - gc, g.out_vec, v,
                     out_exp);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) h[q] = static_cast<_Float16>(v[q]);
        store16(out, h, row_off + off);
        if constexpr (M == kApplyLo) {
          f16x8 l;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            l[q] = static_cast<_Float16>((v[q] - static_cast<float>(h[q])) * kScaleLo);
          store16(rem_out, l, row_off + off);
        }
        if (!kApplies && !cross && gr < m) {
          float* d = g.D(M == kGram ? 0 : 1, item);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (gr == gc + q) d[gr] = v[q] - static_cast<float>(h[q]);
        }
      }
      if (cross) {
        *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
    lds_barrier();
    if (cross) {
      // kSlab / 8 threads take the rows of one column, 8 rows each
      constexpr int kPerCol = kSlab / 8, kColsAtOnce = kBlock / kPerCol;
#pragma unroll
      for (int p = 0; p < T / kColsAtOnce; ++p) {
        const int col = p * kColsAtOnce + threadIdx.x / kPerCol;
        const int row = threadIdx.x % kPerCol * 8;
        const int gr = r0 + sl * kSlab + row, xr = c0 + col;
        if (gr >= m || xr >= m) continue;
        f16x8 h;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          h[q] = static_cast<_Float16>(*slab_at<TL>(buf0, buf1, row + q, col));
        *reinterpret_cast<f16x8*>(g.A(M == kGram ? 0 : 1, item) + static_cast<int64_t>(xr) * m +
                                  gr) = h;
      }
      lds_barrier();
    }
  }
}

// ---- matrices with a short side of at most 128 ----------------------------------
// Here A and B fit a block's LDS, and a launch per product would be all latency.
// One kernel per step instead: every block of a matrix sums the partial Gram
// matrices of the step before, forms B from them for itself, multiplies its own
// columns of X (of 64 at a time) by it, and adds their products into its partial
// of the next Gram matrix while they are in LDS.  A matrix that one block
// handles alone goes through all its steps in one launch, with the Gram matrix
// staying in registers.  The first Gram matrix comes from the input as it is,
// by a power of two that each block keeps for itself, and its trace is the
// squared norm, so there is no prologue.
//   MP    the padded short side, 64 or 128
//   LDS   B (A before it); 64 columns of X and their remainder
// 16-byte pieces of LDS rows are rotated by row against bank conflicts.

// Chunks of 64 columns that fit LDS together: such matrices never leave it.
constexpr int kStay64 = 4, kStay128 = 3;

template <int MP>
struct Flat {
  static constexpr int kSub = MP / 64;          // 32 x 32 tiles per wave and side of MP
  static constexpr int kPasses = MP / 32;       // 16-byte pieces of 64 columns per thread
  static constexpr int kB = MP * MP * 2, kX = MP * 64 * 2;
};

// Byte of piece `piece` (8 elements) of a row of COLS elements.
template <int COLS>
__device__ __forceinline__ int flat_at(int row, int piece) {
  constexpr int kMask = (COLS / 8 < 16 ? COLS / 8 : 16) - 1;
  return row * (COLS * 2) + ((piece * 16) ^ ((row & kMask) * 16));
}

// A lane's part of an MFMA operand: 32 rows of a matrix of COLS columns, k along
// them, or 32 columns, k running over the rows.
template <int COLS>
struct Along {
  const char* at;
  int turn;
  __device__ __forceinline__ Along(const char* mat, int row, int lane) {
    at = mat + (row + (lane & 31)) * (COLS * 2);
    turn = flat_at<COLS>(lane & 31, lane >> 5) - (lane & 31) * (COLS * 2);
  }
  // phase ph (16 k), 32 rows further on for each i
  __device__ __forceinline__ f16x8 read(int ph, int i) const {
    return *reinterpret_cast<const f16x8*>(at + ((ph * 32) ^ turn) + i * 32 * (COLS * 2));
  }
};
template <int COLS>
struct Across {
  const char* lo;
  const char* hi;
  int turn_lo, turn_hi;
  __device__ __forceinline__ Across(const char* mat, int col, int lane) {
    const int k = (lane >> 5) * 8 + ((lane >> 2) & 3);
    const int piece = (col >> 3) + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    lo = mat + (lane & 1) * 8 + k * (COLS * 2);
    hi = lo + 4 * (COLS * 2);
    turn_lo = flat_at<COLS>(k, piece) - k * (COLS * 2);
    turn_hi = flat_at<COLS>(k + 4, piece) - (k + 4) * (COLS * 2);
  }
  // phase ph: 16 rows further on, whose rotation is the same; i: 32 columns
  __device__ __forceinline__ f16x8 read(int ph, int i) const {
    typedef __fp16 h4 __attribute__((__vector_size__(8)));
    typedef __attribute__((address_space(3))) h4* lds_h4;
    const int step = ph * 16 * (COLS * 2);
    const h4 a = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)(lo + (turn_lo ^ (i * 64)) + step));
    const h4 b = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_h4)(hi + (turn_hi ^ (i * 64)) + step));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

struct FlatStep {
  float a, b, c;
  int32_t last, lo_in, lo_out;
};
struct FlatSteps {
  FlatStep s[SBP_NS_MAX_STEPS];
  float eps;
  int32_t grow;
};

// A Gram matrix of values times 2^-by, brought back (by <= 0; what lies 2^70
// below counts for nothing).
__device__ __forceinline__ float gram_scale(int by) { return ldexpf(1.0f, 2 * (by < -70 ? -70 : by)); }

// What a stage does with a block's columns: the input's Gram matrix; a step from
// the input or from the stored X, with X's remainder kept, without it, or to the
// caller's matrix.
enum Kind { kInputGram, kInput, kInputLast, kKept, kPlain, kStoredLast };

struct Columns {
  int lo, hi;     // chunks of 64
  int k;          // the input times 2^k
  float fa, fd;   // X' = fa X + fd * accumulators, with the diagonal's remainder * fd
  int out_exp;    // the caller's matrix: X' * 2^out_exp
  bool keep;      // store the remainder
};

template <int MP>
struct Buffers {
  char *B, *X, *L;
  float *dA, *dB, *red;
};

// TALL: X lies across, a row of the chunk holds MP elements.  G: the products
// of this block's columns of the result (of the input * 2^kx).  STAYS: all of the
// matrix's chunks have places of their own in LDS and stay there between stages.
template <int MP, bool TALL, bool STAYS, Kind K>
__device__ __forceinline__ void flat_columns(const Group& g, const Buffers<MP>& all, int item,
                                             const Columns& cs, int wave, int lane,
                                             f32x16 (&G)[MP / 64][MP / 64], int& kx) {
  using F = Flat<MP>;
  constexpr int kSub = F::kSub, H = MP / 2;
  constexpr int XC = TALL ? MP : 64;
  constexpr bool kFromInput = K == kInputGram || K == kInput || K == kInputLast;
  constexpr bool kStep = K != kInputGram, kLast = K == kInputLast || K == kStoredLast;
  constexpr bool kLoIn = K == kKept, kLo = K == kKept || K == kInput;
  constexpr bool kFetch = kFromInput || !STAYS;
  Buffers<MP> lds = all;
  const int wr = wave >> 1, wc = wave & 1;
  const uint16_t* in = g.in + item * g.in_stride;
  uint16_t* out = g.out + item * g.out_stride;
  _Float16* S = g.S(0, item);
  _Float16* L = g.L(item);
  const int ld = g.cp;
  // this thread's pieces of a chunk
  auto row_of = [&](int p) { return (p * kBlock + wave * 64 + lane) / (XC / 8); };
  const int piece = lane % (XC / 8);
  u32x4 next[F::kPasses], next_lo[F::kPasses];
  auto fetch = [&](int c) {
#pragma unroll
    for (int p = 0; p < F::kPasses; ++p) {
      const int gr = TALL ? c * 64 + row_of(p) : row_of(p), gc = TALL ? piece * 8 : c * 64 + piece * 8;
      if constexpr (kFromInput) {
        u32x4 v{0, 0, 0, 0};
        if (gr < g.rows && gc < g.cols) v = load_row8(in + gr * g.in_ld + gc, g.cols - gc, g.in_vec);
        next[p] = v;
      } else {
        const int64_t idx = static_cast<int64_t>(gr) * ld + gc;
        next[p] = *reinterpret_cast<const u32x4*>(S + idx);
        if constexpr (kLoIn) next_lo[p] = *reinterpret_cast<const u32x4*>(L + idx);
      }
    }
  };
  // where a lane's accumulators lie in X: 4 neighbours of a row for each u and q
  const int x_row = TALL ? wc * 32 + (lane & 31) : wc * H + (lane & 31);
  auto x_at = [&](int u, int q) {
    return TALL ? flat_at<XC>(x_row, (wr * H + u * 32) / 8 + q) + (lane >> 5) * 8
                : flat_at<XC>(x_row, wr * 4 + q) + (lane >> 5) * 8 + u * 32 * (XC * 2);
  };
  if constexpr (kFetch) fetch(cs.lo);
#pragma unroll 1
  for (int c = cs.lo; c < cs.hi; ++c) {
    if constexpr (STAYS) {
      lds.X = all.X + c * F::kX;
      lds.L = all.L + c * F::kX;
    }
    if constexpr (K == kInputGram) {  // the chunk's largest magnitude sets its power of two
      float big = 0.0f;
      auto two = [&](uint32_t x) {
        big = fmaxf(big, fmaxf(fabsf(sbp::bf16_lo(x)), fabsf(sbp::bf16_hi(x))));
      };
#pragma unroll
      for (int p = 0; p < F::kPasses; ++p)
        two(next[p].x), two(next[p].y), two(next[p].z), two(next[p].w);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor(big, off, 64));
      if (lane == 0) lds.red[wave] = big;
      lds_barrier();
      big = fmaxf(fmaxf(lds.red[0], lds.red[1]), fmaxf(lds.red[2], lds.red[3]));
      // 2^7 <= big * 2^k < 2^8; an infinity needs no room
      const int k = big > 0.0f && big < __builtin_huge_valf() ? 7 - ilogbf(big) : 200;
      if (k < kx) {
        const float by = kx == 200 ? 1.0f : gram_scale(k - kx);
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int j = 0; j < kSub; ++j) G[i][j] = G[i][j] * by;
        kx = k;
      }
    }
    if constexpr (kFetch) {
      const int k = K == kInputGram ? kx : cs.k;
#pragma unroll
      for (int p = 0; p < F::kPasses; ++p) {
        const int at = flat_at<XC>(row_of(p), piece);
        *reinterpret_cast<u32x4*>(lds.X + at) =
            kFromInput ? __builtin_bit_cast(u32x4, half8(next[p], k)) : next[p];
        if constexpr (kLoIn) *reinterpret_cast<u32x4*>(lds.L + at) = next_lo[p];
      }
      lds_barrier();
      if (c + 1 < cs.hi) fetch(c + 1);
    }
    if constexpr (kStep) {
      // D = 64 columns x MP (wide) or MP x 64 columns (tall): a lane's 4 rows of D
      // are 4 neighbours of one row of X
      constexpr int DI = TALL ? kSub : 1, DJ = TALL ? 1 : kSub;
      f32x16 D[DI][DJ] = {};
      const Along<MP> b(lds.B, (TALL ? wr : wc) * H, lane);
      const Along<XC> xa(lds.X, wc * 32, lane);
      const Across<XC> xt(lds.X, wr * 32, lane);
#pragma unroll 4
      for (int ph = 0; ph < MP / 16; ++ph) {
        const f16x8 x = TALL ? xa.read(ph, 0) : xt.read(ph, 0);
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          if constexpr (TALL) D[u][0] = mfma(b.read(ph, u), x, D[u][0]);
          else D[0][u] = mfma(x, b.read(ph, u), D[0][u]);
        }
      }
      f16x4 hi[kSub][4], rest[kSub][4];
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f16x4 x = *reinterpret_cast<const f16x4*>(lds.X + x_at(u, q));
          f16x4 l{};
          if constexpr (kLoIn) l = *reinterpret_cast<const f16x4*>(lds.L + x_at(u, q));
          f32x4 d;
          if constexpr (TALL)
            d = *reinterpret_cast<const f32x4*>(lds.dB + wr * H + u * 32 + q * 8 + 4 * (lane >> 5));
          else
            d = f32x4{} + lds.dB[wc * H + u * 32 + (lane & 31)];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = static_cast<float>(x[e]);
            if constexpr (kLoIn) y = fmaf(static_cast<float>(l[e]), 1.0f / kScaleLo, y);
            const float acc = TALL ? D[u % DI][0][q * 4 + e] : D[0][u % DJ][q * 4 + e];
            const float v = fmaf(fmaf(d[e], cs.fd, cs.fa), y, acc * cs.fd);
            if constexpr (kLast) {
              hi[u][q][e] = __builtin_bit_cast(_Float16, static_cast<__bf16>(ldexpf(v, cs.out_exp)));
            } else {
              hi[u][q][e] = static_cast<_Float16>(v);
              if constexpr (kLo)
                rest[u][q][e] =
                    static_cast<_Float16>((v - static_cast<float>(hi[u][q][e])) * kScaleLo);
            }
          }
        }
      lds_barrier();  // X is read
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *reinterpret_cast<f16x4*>(lds.X + x_at(u, q)) = hi[u][q];
          if constexpr (kLo) *reinterpret_cast<f16x4*>(lds.L + x_at(u, q)) = rest[u][q];
        }
      lds_barrier();
#pragma unroll
      for (int p = 0; p < F::kPasses; ++p) {
        if constexpr (STAYS && !kLast) continue;
        const int gr = TALL ? c * 64 + row_of(p) : row_of(p);
        const int gc = TALL ? piece * 8 : c * 64 + piece * 8;
        const int at = flat_at<XC>(row_of(p), piece);
        const u32x4 w = *reinterpret_cast<const u32x4*>(lds.X + at);
        if constexpr (kLast) {
          if (gr < g.rows && gc < g.cols)
            store_bits8(out + gr * g.out_ld + gc, g.cols - gc, g.out_vec, w);
        } else {
          const int64_t idx = static_cast<int64_t>(gr) * ld + gc;
          *reinterpret_cast<u32x4*>(S + idx) = w;
          if (kLo && cs.keep)
            *reinterpret_cast<u32x4*>(L + idx) = *reinterpret_cast<const u32x4*>(lds.L + at);
        }
      }
    }
    if constexpr (!kLast) {
      const Along<XC> pa(lds.X, wr * H, lane), qa(lds.X, wc * H, lane);
      const Across<XC> pt(lds.X, wr * H, lane), qt(lds.X, wc * H, lane);
#pragma unroll
      for (int ph = 0; ph < 4; ++ph) {
        f16x8 p[kSub], q[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
          p[i] = TALL ? pt.read(ph, i) : pa.read(ph, i);
          q[i] = TALL ? qt.read(ph, i) : qa.read(ph, i);
        }
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int j = 0; j < kSub; ++j) G[i][j] = mfma(p[i], q[j], G[i][j]);
      }
    }
    if constexpr (!STAYS) lds_barrier();  // X and L are free
  }
}

__device__ __forceinline__ int least(const int32_t* k, int count) {
  int r = k[0];
  for (int i = 1; i < count; ++i) r = k[i] < r ? k[i] : r;
  return r;
}

// Sums a matrix's partial Gram matrices into the first: 1024 elements a block.
__global__ void __launch_bounds__(kBlock) ns_flat_sum_kernel(Groups gs, int which, int scaled) {
  int gi = 0;
  while (gi + 1 < gs.n && blockIdx.x >= gs.g[gi + 1].t_gram) ++gi;
  const Group& g = gs.g[gi];
  const int per = g.m * g.m / 1024;
  const int local = blockIdx.x - g.t_gram, item = local / per;
  const int64_t at = static_cast<int64_t>(local % per) * 1024 + threadIdx.x * 4;
  const int32_t* pk = g.part_k(item, 0);
  const int kx = scaled ? least(pk, g.splits) : 0;
  f32x4 sum{};
#pragma unroll 8
  for (int s = 0; s < g.splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(g.part(which, item, s) + at);
    const float by = scaled ? gram_scale(kx - pk[s]) : 1.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(v[e], by, sum[e]);
  }
  *reinterpret_cast<f32x4*>(g.part(which, item, 0) + at) = sum;
  if (local % per == 0 && threadIdx.x == 0) *g.part_k(item, g.splits) = kx;
}

// Stages first .. end-1: stage 0 is the input's Gram matrix, stage s step s.
template <int MP, bool TALL, bool STAYS>
__device__ __forceinline__ void flat_stages(const Group& g, const FlatSteps& fs, int item,
                                            int split, int first, int end,
                                            const Buffers<MP>& lds) {
  constexpr int kSub = MP / 64, H = MP / 2;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lane = threadIdx.x & 63;
  const int wr = wave >> 1, wc = wave & 1;
  const int chunks = g.n / 64;
  Columns cs{};
  cs.lo = static_cast<int>(static_cast<int64_t>(chunks) * split / g.splits);
  cs.hi = static_cast<int>(static_cast<int64_t>(chunks) * (split + 1) / g.splits);
  f32x16 G[kSub][kSub];
  int kx = 0;
  int log_sx = 0;
  float gram = 0.0f, apply_first = 0.0f;
  if (first > 1) {
    const Scal sc = g.scal[item];
    log_sx = sc.log_sx;
    gram = sc.gram;
  }
#pragma unroll 1
  for (int stage = first; stage < end; ++stage) {
    // offsets are worked out again each stage: kept, they would not fit the registers
    asm volatile("" : "+v"(lane));
    if (stage > 0) {
      const FlatStep st = fs.s[stage - 1];
      // -- the Gram matrix of the stage before
      if (g.splits > 1) {
        const float* part = g.part(stage & 1, item, 0) + wave * (H * H) + lane * 4;
        const int parts = g.summed ? 1 : g.splits;
        const int32_t* pk = g.part_k(item, g.summed ? g.splits : 0);
        kx = stage == 1 ? least(pk, parts) : 0;
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int j = 0; j < kSub; ++j) G[i][j] = f32x16{};
#pragma unroll 2
        for (int s = 0; s < parts; ++s) {
          const float by = stage == 1 ? gram_scale(kx - pk[s]) : 1.0f;
          const float* p = part + static_cast<int64_t>(s) * (MP * MP);
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int j = 0; j < kSub; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(p + ((i * kSub + j) * 4 + q) * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e) G[i][j][q * 4 + e] = fmaf(v[e], by, G[i][j][q * 4 + e]);
              }
        }
      }
      if (stage == 1) {
        double tr = 0.0;
        if (wr == wc) {
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              tr = tr + (8 * (e >> 2) + 4 * (lane >> 5) + (e & 3) == (lane & 31) ? G[i][i][e] : 0.0f);
        }
        const double norm = sqrt(block_sum_all(tr)) * ldexp(1.0, -kx);
        const Norm nm = norm_of(norm, fs.eps, fs.grow);
        cs.k = nm.k;
        log_sx = nm.log_sx;
        apply_first = static_cast<float>(nm.rho * nm.sx);
        gram = static_cast<float>(kScaleA * ldexp(1.0, -2 * kx) / (nm.floor_norm * nm.floor_norm));
        if (split == 0 && threadIdx.x == 0)
          g.scal[item] = Scal{0.0f, static_cast<float>(kScaleA / (nm.sx * nm.sx)), 0.0f, log_sx};
      }
      // -- A, then B, into LDS (symmetric: a lane's 4 rows of a column go into the
      // column's row), their diagonals' remainders next to them
      auto put = [&](const f32x16 (&v)[kSub][kSub], float* d) {
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            const int col = wc * H + j * 32 + (lane & 31);
            float rest = 0.0f;  // of this lane's diagonal element, if it has one
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              f16x4 h;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                h[e] = static_cast<_Float16>(v[i][j][q * 4 + e]);
                if (i == j)
                  rest = q * 8 + 4 * (lane >> 5) + e == (lane & 31)
                             ? v[i][j][q * 4 + e] - static_cast<float>(h[e])
                             : rest;
              }
              *reinterpret_cast<f16x4*>(lds.B + flat_at<MP>(col, (wr * H + i * 32) / 8 + q) +
                                        (lane >> 5) * 8) = h;
            }
            if (i == j && wr == wc && ((lane >> 2) & 1) == lane >> 5) d[col] = rest;
          }
      };
#pragma unroll
      for (int i = 0; i < kSub; ++i)
#pragma unroll
        for (int j = 0; j < kSub; ++j) G[i][j] = G[i][j] * gram;
      put(G, lds.dA);
      lds_barrier();
      f32x16 sq[kSub][kSub] = {};
      {
        const Along<MP> pa(lds.B, wr * H, lane), qa(lds.B, wc * H, lane);
#pragma unroll 2
        for (int ph = 0; ph < MP / 16; ++ph) {
          f16x8 p[kSub], q[kSub];
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            p[i] = pa.read(ph, i);
            q[i] = qa.read(ph, i);
          }
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int j = 0; j < kSub; ++j) sq[i][j] = mfma(p[i], q[j], sq[i][j]);
        }
      }
      const float fb = st.b * (kScaleB / kScaleA), fc = st.c * (kScaleB / (kScaleA * kScaleA));
#pragma unroll
      for (int i = 0; i < kSub; ++i)
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          const float dc = lds.dA[wc * H + j * 32 + (lane & 31)];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 dr = *reinterpret_cast<const f32x4*>(lds.dA + wr * H + i * 32 + q * 8 +
                                                             4 * (lane >> 5));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // (A + D)^2 = A^2 + D A + A D + D^2 for the diagonal remainder D
              const float a = G[i][j][q * 4 + e], x = static_cast<float>(static_cast<_Float16>(a));
              float s = fmaf(dr[e] + dc, x, sq[i][j][q * 4 + e]);
              if (i == j)
                s = wr == wc && q * 8 + 4 * (lane >> 5) + e == (lane & 31) ? fmaf(dc, dc, s) : s;
              sq[i][j][q * 4 + e] = fmaf(fc, s, fb * a);
            }
          }
        }
      lds_barrier();  // A is read
      put(sq, lds.dB);
      lds_barrier();
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int j = 0; j < kSub; ++j) G[i][j] = f32x16{};

    // -- this block's columns
    if (stage == 0) {
      kx = 200;  // nothing yet
      flat_columns<MP, TALL, STAYS, kInputGram>(g, lds, item, cs, wave, lane, G, kx);
    } else {
      const FlatStep st = fs.s[stage - 1];
      const float fx = (stage == 1 ? apply_first : 1.0f) * (st.last ? g.out_frac : 1.0f);
      cs.fd = fx * (1.0f / kScaleB);
      cs.fa = fx * st.a;
      cs.out_exp = g.out_exp - log_sx;
      cs.keep = st.lo_out;
      if (stage == 1 && st.last)
        flat_columns<MP, TALL, STAYS, kInputLast>(g, lds, item, cs, wave, lane, G, kx);
      else if (stage == 1)
        flat_columns<MP, TALL, STAYS, kInput>(g, lds, item, cs, wave, lane, G, kx);
      else if (st.last)
        flat_columns<MP, TALL, STAYS, kStoredLast>(g, lds, item, cs, wave, lane, G, kx);
      else if (st.lo_in)
        flat_columns<MP, TALL, STAYS, kKept>(g, lds, item, cs, wave, lane, G, kx);
      else
        flat_columns<MP, TALL, STAYS, kPlain>(g, lds, item, cs, wave, lane, G, kx);
      if (stage == 1) gram = ldexpf(kScaleA, -2 * log_sx);
      if (st.last) return;
    }
    if (g.splits > 1) {
      float* p = g.part((stage + 1) & 1, item, split) + wave * (H * H) + lane * 4;
#pragma unroll
      for (int i = 0; i < kSub; ++i)
#pragma unroll
        for (int j = 0; j < kSub; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(p + ((i * kSub + j) * 4 + q) * 256) =
                f32x4{G[i][j][q * 4], G[i][j][q * 4 + 1], G[i][j][q * 4 + 2], G[i][j][q * 4 + 3]};
      if (stage == 0 && threadIdx.x == 0) *g.part_k(item, split) = kx;
    }
    __syncthreads();  // a block that goes on by itself reads what it stored
  }
}

// CHUNKS: places in LDS for the chunks of a matrix that one block handles alone;
// 0: one place, the chunks come and go.
template <int MP, int CHUNKS>
__global__ void __launch_bounds__(kBlock, MP == 128 && CHUNKS > 0 ? 1 : 2)
ns_flat_kernel(Groups gs, FlatSteps fs, int first, int end) {
  constexpr int kPlaces = CHUNKS > 0 ? CHUNKS : 1;
  __shared__ __align__(16) char LB[Flat<MP>::kB];
  __shared__ __align__(16) char LX[kPlaces * Flat<MP>::kX];
  __shared__ __align__(16) char LL[kPlaces * Flat<MP>::kX];
  __shared__ __align__(16) float dA[MP], dB[MP], red[4];
  const Buffers<MP> lds{LB, LX, LL, dA, dB, red};
  int gi = 0;
  while (gi + 1 < gs.n && blockIdx.x >= gs.g[gi + 1].t_apply) ++gi;
  const Group& g = gs.g[gi];
  // a matrix's blocks go to one XCD (blocks are handed to the XCDs in turn),
  // whose L2 then serves the partial sums that all of them read
  const unsigned local = blockIdx.x - g.t_apply, round = local / (kXcds * g.splits);
  const unsigned in = local % (kXcds * g.splits);
  const unsigned items = g.count - round * kXcds < kXcds ? g.count - round * kXcds : kXcds;
  const int item = round * kXcds + in % items, split = in / items;
  if (g.tall())
    flat_stages<MP, true, (CHUNKS > 0)>(g, fs, item, split, first, end, lds);
  else
    flat_stages<MP, false, (CHUNKS > 0)>(g, fs, item, split, first, end, lds);
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

struct Shape {
  int64_t m, n;  // padded short and long side
  int64_t norm_blocks;
  int64_t splits;  // blocks per matrix of the flat kernel, 0 for the products
  bool summed;     // their partial sums added by a kernel of its own
};

// What a matrix's results depend on (the flat kernel or the products, and its
// splits) goes by its shape alone, so that ranks that hold different parts of a
// model get the same bits for the same matrix.
//
// Splits, measured: a block takes about 2.5 us for 64 columns, as long as for
// reading another block's 128 x 128 partial Gram matrix (a quarter of it at 64 x
// 64), and a launch of its own for each step costs about as much as 4 chunks,
// so what fits one block's LDS (kStay64, kStay128) stays in it; beyond, reading and working balance at the
// square root.  Where 128-wide matrices have 32 chunks and more a kernel of their
// own sums the partials (5 us), and blocks take 4 chunks.
Shape shape_of(const sbp_matrices& g) {
  Shape s;
  s.m = up(std::min(g.rows, g.cols), kPad);
  s.n = up(std::max(g.rows, g.cols), kPad);
  const int64_t units = g.rows * ((g.cols + 511) / 512);
  s.norm_blocks = std::max<int64_t>(1, std::min<int64_t>(kMaxNormBlocks, (units + 7) / 8));
  s.splits = 0;
  s.summed = false;
  if (s.m <= 128) {
    const int64_t chunks = s.n / 64;
    s.splits = 1;
    if (chunks > (s.m == 64 ? kStay64 : kStay128))
      while ((s.splits + 1) * (s.splits + 1) <= chunks && s.splits < 64) ++s.splits;
    s.summed = s.m == 128 && chunks >= 32;
    if (s.summed) s.splits = std::min<int64_t>(64, chunks / 4);
  }
  return s;
}

// Which launches a shape takes part in.
enum Class {
  kProducts, kFlat64, kFlat64Steps, kFlat128, kFlat128Steps, kFlat128Summed, kClasses
};
Class class_of(const Shape& s) {
  if (s.splits == 0) return kProducts;
  if (s.m == 64) return s.splits == 1 ? kFlat64 : kFlat64Steps;
  return s.summed ? kFlat128Summed : s.splits == 1 ? kFlat128 : kFlat128Steps;
}

struct Chunk {
  Class cls;
  std::vector<Piece> pieces;
  int64_t bytes = 0;
};

// Bytes one piece takes, array by array (each 256-B aligned).
int64_t half_bytes(const Shape& s, int64_t count) {
  if (s.splits == 1) return 0;  // all in LDS
  return up(2 * count * (s.splits ? 2 * s.m * s.n : 3 * s.m * s.n + 2 * s.m * s.m), 256);
}
int64_t partial_bytes(const Shape& s, int64_t count) {
  return s.splits ? 0 : up(8 * count * s.norm_blocks, 256);
}
int64_t diag_bytes(const Shape& s, int64_t count) {
  return s.splits ? 0 : up(8 * count * s.m, 256);
}
int64_t scal_bytes(int64_t count) { return up(static_cast<int64_t>(sizeof(Scal)) * count, 256); }
int64_t parts_bytes(const Shape& s, int64_t count) {
  return s.splits > 1 ? up(2 * 4 * count * s.splits * s.m * s.m, 256) : 0;
}
int64_t part_k_bytes(const Shape& s, int64_t count) { return up(4 * count * (s.splits + 1), 256); }

std::vector<Chunk> chunks_of(const sbp_matrices* groups, int32_t n_groups) {
  std::vector<Chunk> out;
  for (int cls = 0; cls < kClasses; ++cls) {
    int64_t room = 0;
    bool open = false;
    for (int32_t i = 0; i < n_groups; ++i) {
      const sbp_matrices& g = groups[i];
      if (g.rows == 0 || g.cols == 0) continue;
      const Shape s = shape_of(g);
      if (class_of(s) != cls) continue;
      const int64_t elems = s.m * s.n;
      for (int64_t first = 0; first < g.count;) {
        if (!open || room < elems || static_cast<int>(out.back().pieces.size()) == kMaxGroups) {
          out.emplace_back();
          out.back().cls = static_cast<Class>(cls);
          open = true;
          room = std::max(kChunkElems, elems);
        }
        const int64_t take = std::min(g.count - first, room / elems);
        out.back().pieces.push_back(Piece{i, first, take});
        out.back().bytes += half_bytes(s, take) + partial_bytes(s, take) + diag_bytes(s, take) +
                            scal_bytes(take) + parts_bytes(s, take) + part_k_bytes(s, take);
        room -= take * elems;
        first += take;
      }
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

static_assert(sizeof(Groups) + sizeof(FlatSteps) + 8 <= 4096, "kernel arguments");

// How a product's tiles are launched: `tiles` of side T, then those of side 256
// from `tiles` on as quarters.
struct Launches {
  int T;
  uint32_t tiles, quarters;
};

// Measured, at k = 4096: a round of 256 tiles of side 256, one a CU, takes 112
// us, 1024 of side 128, two a CU, 125 us.  So side 256 takes whole rounds, and
// what is left over where that is more than half a round; less goes by quarters
// of side 128 (half a round in 80 us).  Short sums leave more of a large tile's
// time to its first loads and its epilogue, which side 128 hides behind a second
// block: between one and a half and two rounds of side 256 it is faster while it
// makes at most 3.5 rounds of its own 512.  The five steps' applies, side 256
// against side 128:
//   k      tiles 256  128     us
//   1024         400  1600   414   376
//   1024         448  1792   429   419
//   1024         496  1984   453   468  (so these take side 256)
//    960         400  1600   380   360
//    960         496  1984   409   440
//    768         387  1548   365   345
//    768         432  1728   380   363
//    768         504  2016   410   416
//    640         504  1400   323   248  (a third of the large tiles hangs over)
//    512         388  1552   312   260
//    512         508  2032   364   357
// At k = 2048 side 256 is ahead again (448 tiles: 120 to 129 us against 126 to
// 136).  Under one round, side 128 where it gives most CUs a tile (252 and 432
// tiles at k = 768: 17 and 18 us against 40 and 28 of side 256), else side 64
// (216 tiles of side 128: 13.2 us, 864 of side 64 14.7; 126: 14.3 against 9.6;
// 30: 15.1 against 7.4).
Launches launches_of(uint32_t at256, uint32_t at128, uint32_t at64, int k) {
  const uint32_t left = at256 % 256;
  const bool few_short = at256 < 512 && left > 128 && at128 <= 1792 && k <= 1024;
  if (at256 >= 256 && !few_short) {
    if (left > 0 && left <= 128) return Launches{256, at256 - left, 4 * left};
    return Launches{256, at256, 0};
  }
  if (at128 >= 192) return Launches{128, at128, 0};
  return Launches{64, at64, 0};
}

uint32_t gram_tiles(const Group& g, int T) {
  return static_cast<uint32_t>(g.count) * lower_tiles(g.m, T);
}
uint32_t apply_tiles(const Group& g, int T) {
  return static_cast<uint32_t>(g.count) * ((g.rp + T - 1) / T) * ((g.cp + T - 1) / T);
}

// Launches of one kind of product for all groups, whose first tiles are set.
template <uint32_t (*TILES)(const Group&, int), int32_t Group::*K>
Launches lay_out(Groups& gs, uint32_t Group::*first) {
  uint32_t at[3] = {0, 0, 0};
  int k = 0;  // the longest sum
  constexpr int kSides[3] = {256, 128, 64};
  for (int i = 0; i < gs.n; ++i) {
    for (int t = 0; t < 3; ++t) at[t] += TILES(gs.g[i], kSides[t]);
    k = std::max(k, gs.g[i].*K);
  }
  const Launches l = launches_of(at[0], at[1], at[2], k);
  uint32_t next = 0;
  for (int i = 0; i < gs.n; ++i) {
    gs.g[i].*first = next;
    next += TILES(gs.g[i], l.T);
  }
  return l;
}

template <Mode M>
void launch_product(const Launches& l, const Groups& gs, const Step& st, hipStream_t stream) {
  const dim3 block(kBlock);
  if (l.T == 256)
    hipLaunchKernelGGL((ns_product_kernel<Tile<256>, M, false>), dim3(l.tiles), block, 0,
                       stream, gs, st, l.tiles, 0u);
  else if (l.T == 128)
    hipLaunchKernelGGL((ns_product_kernel<Tile<128>, M, false>), dim3(l.tiles), block, 0,
                       stream, gs, st, l.tiles, 0u);
  else
    hipLaunchKernelGGL((ns_product_kernel<Tile<64>, M, false>), dim3(l.tiles), block, 0,
                       stream, gs, st, l.tiles, 0u);
  if (l.quarters > 0)
    hipLaunchKernelGGL((ns_product_kernel<Tile<128>, M, true>), dim3(l.quarters), block, 0,
                       stream, gs, st, l.quarters, l.tiles);
}

sbp_status run_steps(const char* who, Groups& gs, const sbp_ns_hparams& hp, hipStream_t stream) {
  const Launches gram = lay_out<gram_tiles, &Group::n>(gs, &Group::t_gram);
  const Launches apply = lay_out<apply_tiles, &Group::m>(gs, &Group::t_apply);
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
    launch_product<kGram>(gram, gs, st, stream);
    launch_product<kPoly>(gram, gs, st, stream);
    if (st.last) launch_product<kLast>(apply, gs, st, stream);
    else if (st.lo_in || st.lo_out) launch_product<kApplyLo>(apply, gs, st, stream);
    else launch_product<kApply>(apply, gs, st, stream);
    const sbp_status rc = launched(who);
    if (rc != SBP_OK) return rc;
  }
  return SBP_OK;
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
    int out_exp;
    g.out_frac = std::frexp(src.out_scale, &out_exp);
    g.out_exp = out_exp;
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
    g.splits = static_cast<int32_t>(s.splits);
    g.summed = s.summed;
    g.parts = reinterpret_cast<float*>(ws);
    ws += parts_bytes(s, p.count);
    g.part_ks = reinterpret_cast<int32_t*>(ws);
    ws += part_k_bytes(s, p.count);
    g.t_norm = norm;
    g.t_pro = pro;
    norm += g.count * g.norm_blocks;
    pro += g.count * (g.rp / 32) * (g.cp / 64);
  }
  // While X is far below 1 a step multiplies it by a: b and c come in with its
  // square.  What they add on the last steps before X gets near 1 has a factor
  // 64 of room, between 2^10, where this bound puts X, and fp16's end.
  double grow = 0.0;
  for (int s = 0; s < hp.steps; ++s)
    grow += std::log2(std::max(1.0, std::fabs(static_cast<double>(hp.coefs[3 * s]))));
  const int igrow = static_cast<int>(std::min(200.0, std::ceil(grow)));

  if (c.cls != kProducts) {
    FlatSteps fs{};
    fs.eps = hp.eps;
    fs.grow = igrow;
    for (int s = 0; s < hp.steps; ++s)
      fs.s[s] = FlatStep{hp.coefs[3 * s], hp.coefs[3 * s + 1], hp.coefs[3 * s + 2],
                         s == hp.steps - 1, s > 0 && hp.steps - s >= 3, hp.steps - 1 - s >= 3};
    uint32_t blocks = 0, sums = 0;
    for (int i = 0; i < gs.n; ++i) {
      gs.g[i].t_apply = blocks;
      gs.g[i].t_gram = sums;
      blocks += gs.g[i].count * gs.g[i].splits;
      sums += gs.g[i].count * (gs.g[i].m * gs.g[i].m / 1024);
    }
    const bool at_once = c.cls == kFlat64 || c.cls == kFlat128;
    const bool wide = c.cls == kFlat128 || c.cls == kFlat128Steps || c.cls == kFlat128Summed;
    auto kernel = at_once ? (wide ? ns_flat_kernel<128, kStay128> : ns_flat_kernel<64, kStay64>)
                          : (wide ? ns_flat_kernel<128, 0> : ns_flat_kernel<64, 0>);
    for (int stage = 0; stage <= hp.steps; stage += at_once ? hp.steps + 1 : 1) {
      hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBlock), 0, stream, gs, fs, stage,
                         at_once ? hp.steps + 1 : stage + 1);
      if (c.cls == kFlat128Summed && stage < hp.steps)
        hipLaunchKernelGGL(ns_flat_sum_kernel, dim3(sums), dim3(kBlock), 0, stream, gs,
                           (stage + 1) & 1, stage == 0 ? 1 : 0);
      const sbp_status rc = launched(who);
      if (rc != SBP_OK) return rc;
    }
    return SBP_OK;
  }

  hipLaunchKernelGGL(ns_norm_kernel, dim3(norm), dim3(kBlock), 0, stream, gs);
  hipLaunchKernelGGL(ns_prologue_kernel, dim3(pro), dim3(kBlock), 0, stream, gs, hp.eps, igrow);
  sbp_status rc = launched(who);
  if (rc != SBP_OK) return rc;

  return run_steps(who, gs, hp, stream);
}

sbp_status newton_schulz(const char* who, const sbp_matrices* groups, int32_t n_groups,
                         const sbp_ns_hparams* hp, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream) {
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

}  // namespace

extern "C" {

int64_t sbp_newton_schulz_workspace(const sbp_matrices* groups, int32_t n_groups) {
  const char* who = "sbp_newton_schulz_workspace";
  try {
    if (check_shapes(who, groups, n_groups) != SBP_OK) return -1;
    int64_t most = 0;
    for (const Chunk& c : chunks_of(groups, n_groups)) most = std::max(most, c.bytes);
    (void)sbp::ok();
    return most;
  } catch (...) {
    (void)sbp::fail(SBP_ENOMEM, std::string(who) + ": out of host memory");
    return -1;
  }
}

// The lists are made before anything is launched.
sbp_status sbp_newton_schulz(const sbp_matrices* groups, int32_t n_groups,
                             const sbp_ns_hparams* hp, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
  const char* who = "sbp_newton_schulz";
  try {
    return newton_schulz(who, groups, n_groups, hp, workspace, workspace_bytes, stream);
  } catch (...) {
    return sbp::fail(SBP_ENOMEM, std::string(who) + ": out of host memory");
  }
}

}  // extern "C"
