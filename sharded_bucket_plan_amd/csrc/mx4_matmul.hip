// C = A B' of two microscaled 4-bit operands (mx4.h) on CDNA4's scaled matrix
// instructions.  Exact semantics are in include/sbp.h.
//
// v_mfma_scale_f32_16x16x128 takes 16 rows of each operand and 128 contracted
// values: lane l holds row l % 16's block l / 16 of 32 values (16 bytes) and its
// scale byte.  B's rows go in as the first operand, A's as the second, so that a
// lane's four results are neighbours in a row of C.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "bf16.h"
#include "internal.h"
#include "mx4.h"

#pragma clang fp contract(off)

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kFp4 = 4;  // the instruction's operand format

struct Problem {
  const char* a;  // codes
  const char* b;
  const uint8_t* sa;
  const uint8_t* sb;
  int64_t m, n, kb;  // kb: blocks of a row
  void* out;
  int64_t ld;
  int32_t f32, accumulate;
  int32_t vec;  // out's rows are 16-byte aligned
};

__device__ __forceinline__ f32x4 product(u32x4 b, uint32_t sb, u32x4 a, uint32_t sa, f32x4 c) {
  const i32x8 x{static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z),
                static_cast<int>(b.w), 0, 0, 0, 0};
  const i32x8 y{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                static_cast<int>(a.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, kFp4, kFp4, 0,
                                                          static_cast<int>(sb), 0,
                                                          static_cast<int>(sa));
}

// Four neighbours of a row of C, from column c on.
__device__ __forceinline__ void store4(const Problem& p, int64_t row, int64_t c, f32x4 v) {
  const int64_t at = row * p.ld + c;
  if (p.f32) {
    float* o = static_cast<float*>(p.out) + at;
    if (p.vec && c + 4 <= p.n) {
      if (p.accumulate) v = *reinterpret_cast<const f32x4*>(o) + v;
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.n) o[i] = p.accumulate ? o[i] + v[i] : v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    const uint32_t w[4] = {sbp::bf16_rne(v.x), sbp::bf16_rne(v.y), sbp::bf16_rne(v.z),
                           sbp::bf16_rne(v.w)};
    if (p.vec && c + 4 <= p.n) {
      *reinterpret_cast<u32x2*>(o) = u32x2{w[0] | w[1] << 16, w[2] | w[3] << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.n) o[i] = static_cast<uint16_t>(w[i]);
    }
  }
}

// ---- few rows: 16 columns and 16 * MT rows of C a block ---------------------------
// Its W waves share the contracted axis in runs of steps (128 values), each with
// operands straight from memory; their sums meet in LDS, in the waves' order.
template <int MT, int W>
__global__ void __launch_bounds__(W * 64) mx4_few_kernel(Problem p) {
  __shared__ f32x4 sums[W][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const unsigned across = static_cast<unsigned>((p.n + 15) / 16);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % across) * 16;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / across) * (16 * MT);
  // rows past the matrix read the last one; their results are not stored
  auto row = [](int64_t x, int64_t rows) { return x < rows ? x : rows - 1; };
  const int64_t br = row(n0 + r, p.n) * p.kb;
  int64_t ar[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ar[i] = row(m0 + i * 16 + r, p.m) * p.kb;
  const int64_t steps = (p.kb + 3) / 4, per = (steps + W - 1) / W;
  const int64_t last = (wave + 1) * per < steps ? (wave + 1) * per : steps;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
  for (int64_t s = wave * per; s < last; ++s) {
    const int64_t block = s * 4 + g;
    const bool in = block < p.kb;
    const int64_t at = in ? block : p.kb - 1;
    auto codes = [&](const char* base, int64_t row_at) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(base + (row_at + at) * 16);
      return in ? w : u32x4{0, 0, 0, 0};
    };
    auto scale = [&](const uint8_t* base, int64_t row_at) -> uint32_t {
      return in ? base[row_at + at] : 0u;
    };
    const u32x4 b = codes(p.b, br);
    const uint32_t sb = scale(p.sb, br);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      acc[i] = product(b, sb, codes(p.a, ar[i]), scale(p.sa, ar[i]), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += W) {
    f32x4 v = sums[0][i][lane];
    for (int w = 1; w < W; ++w) v = v + sums[w][i][lane];
    const int64_t at = m0 + i * 16 + r;
    if (at < p.m) store4(p, at, n0 + g * 4, v);
  }
}

// ---- tiles --------------------------------------------------------------------------
// One T x T tile of C per block of 4 waves (2 x 2, each a quarter in 16 x 16 MFMA
// tiles).  Slices of 128 contracted values (64 bytes of codes a row) go straight
// from memory to one of four LDS buffers, four slices ahead; the scales, packed
// beforehand as the instruction takes them, a chunk of four slices at a time.
template <int T_>
struct Tile {
  static constexpr int T = T_, NB = 4;
  static constexpr int kHalf = T * 64;       // one operand's slice, bytes
  static constexpr int kBuf = 2 * kHalf;     // A, then B
  static constexpr int kSub = T / 32;        // 16 x 16 tiles per wave and side
  static constexpr int kLoads = T * 64 / 4096;  // per operand, slice and lane
  static constexpr int kScales = T * 16;     // one operand's scales of a chunk, bytes
  // bytes a lane loads of the two operands' scales at once, and how often
  static constexpr int kScaleBytes = T >= 128 ? 16 : 4;
  static constexpr int kScaleLoads = 2 * kScales / (256 * kScaleBytes);
};

// Row of B (inside a wave's columns) that row i of MFMA tile j holds.  With bf16
// results a lane's values of two tiles are 8 neighbours, 16 bytes; with fp32 the
// 4 of one tile are.
template <bool PAIRS>
__host__ __device__ __forceinline__ int row_of(int j, int i) {
  return PAIRS ? (j >> 1) * 32 + (i >> 2) * 8 + (j & 1) * 4 + (i & 3) : j * 16 + i;
}

// Scales of 16 rows and a chunk of 16 blocks as a wave takes them: lane (r, g)'s
// word holds those of row r, blocks 4s + g of its slices s = 0 .. 3.  Zeros past
// the matrix.  packed: [chunk][tile of 16 rows][lane].
struct Pack {
  const uint8_t* scales;
  uint32_t* packed;
  int64_t rows;
  int32_t tiles, pairs, sub;  // 16-row tiles, padded; B's order for bf16; tiles per wave
};
__global__ void __launch_bounds__(256)
mx4_pack_kernel(Pack a, Pack b, int64_t kb, unsigned blocks_a) {
  const bool second = blockIdx.x >= blocks_a;
  const Pack p = second ? b : a;
  const int64_t w = static_cast<int64_t>(second ? blockIdx.x - blocks_a : blockIdx.x) * 4 +
                    (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t chunks = (kb + 15) / 16;
  if (w >= chunks * p.tiles) return;
  const int64_t c = w / p.tiles;
  const int t = static_cast<int>(w - c * p.tiles);
  const int j = t % p.sub;
  const int64_t row = static_cast<int64_t>(t - j) * 16 + (p.pairs ? row_of<true>(j, r) : j * 16 + r);
  uint32_t word = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t block = c * 16 + s * 4 + g;
    if (row < p.rows && block < kb) word |= static_cast<uint32_t>(p.scales[row * kb + block]) << (8 * s);
  }
  p.packed[w * 64 + lane] = word;
}

// `bytes` from p on as a buffer; loads from beyond them give zeros.  Whole offsets
// go into the vector one: a scalar offset past the end would lift the bound.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
typedef __attribute__((address_space(3))) void* lds_ptr;

// One operand of a tile.  LDS keeps a row's four 16-byte pieces (the blocks of a
// slice) rotated by row, which spreads the reads over the banks; the rotation
// comes from the lanes' global addresses.
template <typename TL, bool PAIRS>
struct Operand {
  static constexpr int kSub = TL::kSub;
  static constexpr int kOut = 0x7FFFFFF0;  // an offset beyond every buffer
  const char* from;                        // next slice to load
  int bytes, round_bytes, voff, piece;
  int at[PAIRS ? 2 : 1];                   // LDS offsets of this lane's first fragments
  // of the packed scales
  const char* scales;
  int scale_voff;
  int64_t scale_step;

  static __device__ __forceinline__ int turn(int i) {  // of row i of an MFMA tile
    return (((i >> 1) ^ (i >> 2)) & 2) | (((i >> 3) ^ (i >> 1)) & 1);
  }
  static __device__ __forceinline__ int index(int row) {  // its row in its MFMA tile
    return PAIRS ? ((row >> 3) & 3) * 4 + (row & 3) : row & 15;
  }
  // wrow: the wave's first row in the tile
  __device__ __forceinline__ void init(const char* codes, int64_t rows, int64_t kb, int64_t r0,
                                       int wave, int lane, int wrow) {
    from = codes + r0 * kb * 16;
    // a 64-bit comparison is a vector instruction: the descriptor has to be scalar
    const int have = __builtin_amdgcn_readfirstlane(
        rows - r0 < TL::T ? static_cast<int>(rows - r0) : TL::T);
    bytes = have * static_cast<int>(kb) * 16;
    const int row = wave * 16 + lane / 4;
    piece = (lane & 3) ^ turn(index(row));
    voff = row * static_cast<int>(kb) * 16 + piece * 16;
    round_bytes = 64 * static_cast<int>(kb) * 16;
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < (PAIRS ? 2 : 1); ++h)
      at[h] = (wrow + row_of<PAIRS>(h, i)) * 64 + (g ^ turn(i)) * 16;
  }
  __device__ __forceinline__ void load_round(char* buf, int wave, int r) const {
    // a length below 0 would count as a huge one
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(from, bytes > 0 ? bytes : 0),
                                             (lds_ptr)(buf + (r * 4 + wave) * 1024), 16,
                                             voff + r * round_bytes, 0, 0, 0);
  }
  // To the next slice; `bytes` may go below 0.
  __device__ __forceinline__ void advance() {
    from += 64;
    bytes -= 64;
  }
  // `left` blocks of the rows remain for the next slice: the rest reads as zeros.
  __device__ __forceinline__ void cut(int left) {
    if (left < 4) voff = piece < left ? voff : kOut;
  }
  __device__ __forceinline__ u32x4 read(const char* buf, int i) const {
    const int off = PAIRS ? at[i & 1] + (i >> 1) * 32 * 64 : at[0] + i * 16 * 64;
    return *reinterpret_cast<const u32x4*>(buf + off);
  }
};

template <typename TL>
struct Frags {
  u32x4 a[TL::kSub], b[TL::kSub];
};
template <typename TL>
struct Scales {
  uint32_t a[TL::kSub], b[TL::kSub];
};
template <typename TL>
using Acc = f32x4[TL::kSub][TL::kSub];

template <int S>
__device__ __forceinline__ f32x4 product_of(u32x4 b, uint32_t sb, u32x4 a, uint32_t sa, f32x4 c) {
  const i32x8 x{static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z),
                static_cast<int>(b.w), 0, 0, 0, 0};
  const i32x8 y{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                static_cast<int>(a.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, kFp4, kFp4, S,
                                                          static_cast<int>(sb), S,
                                                          static_cast<int>(sa));
}

// The same for one accumulator, in its registers: at the large tile all 256 are
// taken, and the compiler, free to give a product another place than its summand,
// moves them about between the products.  It does not see these as matrix
// instructions, so the wait states that it would fill in are kept by hand:
// - an accumulator is read or written by anything else 19 or more wait states
//   after its last product (18 is the longest any needs): settle() ends every run
//   of products, before any two ways through the code join;
// - a fragment, scale or accumulator is written by a vector instruction 5 or more
//   before a product reads it (2 are needed): fragments and scales come from LDS,
//   whose reads the compiler waits for, and the accumulators' zeros are settled;
// - a product's own accumulator is used again 64 products later.
// tests/test_matrix_unit_distances.py reads from a build's disassembly that both
// distances hold on every path.
template <int S>
__device__ __forceinline__ void multiply_in_place(f32x4& c, u32x4 b, uint32_t sb, u32x4 a,
                                                  uint32_t sa) {
#define SBP_MX_PRODUCT(LO, HI)                                                       \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" LO \
               "," LO ",0] op_sel_hi:[" HI "," HI ",0] cbsz:4 blgp:4"                 \
               : "+a"(c)                                                              \
               : "v"(b), "v"(a), "v"(sb), "v"(sa))
  if constexpr (S == 0) SBP_MX_PRODUCT("0", "0");
  if constexpr (S == 1) SBP_MX_PRODUCT("1", "0");
  if constexpr (S == 2) SBP_MX_PRODUCT("0", "1");
  if constexpr (S == 3) SBP_MX_PRODUCT("1", "1");
#undef SBP_MX_PRODUCT
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

// This wave's loads but the newest LEFT and its LDS reads are done; then everyone's.
template <int LEFT>
__device__ __forceinline__ void slice_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | ((LEFT >> 4) << 14) | 0x70);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

struct Packed {
  const char* a;
  const char* b;
  int64_t step_a, step_b;  // bytes from chunk to chunk
};

// kSplit: fp32 partial sums of a part of the contracted axis, to the workspace.
enum Out { kBf16, kF32, kSplit };

template <typename TL, Out O>
__global__ void __launch_bounds__(256, TL::T == 256 ? 1 : 2)
mx4_tile_kernel(Problem p, Packed packed, unsigned total) {
  constexpr int T = TL::T, kSub = TL::kSub;
  constexpr bool kPairs = O == kBf16;
  // separate arrays: reads of one do not wait for loads into another
  __shared__ __align__(16) char buf0[TL::kBuf];
  __shared__ __align__(16) char buf1[TL::kBuf];
  __shared__ __align__(16) char buf2[TL::kBuf];
  __shared__ __align__(16) char buf3[TL::kBuf];
  __shared__ __align__(16) char scl0[2 * TL::kScales];
  __shared__ __align__(16) char scl1[2 * TL::kScales];
  char* buf[4] = {buf0, buf1, buf2, buf3};
  char* scl[2] = {scl0, scl1};
  const unsigned tr = static_cast<unsigned>((p.m + T - 1) / T);
  const unsigned tc = static_cast<unsigned>((p.n + T - 1) / T);
  // neighbouring tiles to one XCD, in strips of 8 tile rows, column by column
  unsigned t = blockIdx.x;
  const unsigned per = total / 8;
  if (t < per * 8) t = (t % 8) * per + t / 8;
  constexpr unsigned kStrip = 8;
  const unsigned strip = t / (kStrip * tc), left = tr - strip * kStrip;
  const unsigned high = left < kStrip ? left : kStrip, s = t - strip * kStrip * tc;
  // the divisions go by vector instructions: back to scalars
  const unsigned ti = __builtin_amdgcn_readfirstlane(strip * kStrip + s % high);
  const unsigned tj = __builtin_amdgcn_readfirstlane(s / high);
  const int64_t r0 = static_cast<int64_t>(ti) * T, c0 = static_cast<int64_t>(tj) * T;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wr = (wave >> 1) * (T / 2), wc = (wave & 1) * (T / 2);

  Operand<TL, false> A;
  Operand<TL, kPairs> B;
  A.init(p.a, p.m, p.kb, r0, wave, lane, wr);
  B.init(p.b, p.n, p.kb, c0, wave, lane, wc);
  const char* pa = packed.a + static_cast<int64_t>(ti) * TL::kScales;
  const char* pb = packed.b + static_cast<int64_t>(tj) * TL::kScales;
  int ahead = static_cast<int>(p.kb);  // blocks from the next slice to load on
  auto begin_load = [&]() {
    A.cut(ahead);
    B.cut(ahead);
  };
  auto end_load = [&]() {
    ahead -= 4;
    A.advance();
    B.advance();
  };
  auto load = [&](char* to) {
    begin_load();
#pragma unroll
    for (int r = 0; r < TL::kLoads; ++r) A.load_round(to, wave, r);
#pragma unroll
    for (int r = 0; r < TL::kLoads; ++r) B.load_round(to + TL::kHalf, wave, r);
    end_load();
  };
  int scales_left = static_cast<int>((p.kb + 15) / 16);  // the last chunk's are loaded twice
  auto load_scales = [&](char* to) {
    constexpr int kWave = 64 * TL::kScaleBytes;
#pragma unroll
    for (int r = 0; r < TL::kScaleLoads; ++r) {
      const int off = (r * 4 + wave) * kWave;  // in A's scales, then B's
      const char* src = off < TL::kScales ? pa + off : pb + (off - TL::kScales);
      if constexpr (TL::kScaleBytes == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(src, kWave), (lds_ptr)(to + off), 16,
                                                 lane * 16, 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(src, kWave), (lds_ptr)(to + off), 4,
                                                 lane * 4, 0, 0, 0);
    }
    if (--scales_left > 0) {
      pa += packed.step_a;
      pb += packed.step_b;
    }
  };
  Frags<TL> f[2];
  Scales<TL> sc[2];
  auto read = [&](const char* from, Frags<TL>& to) {
#pragma unroll
    for (int i = 0; i < kSub; ++i) to.a[i] = A.read(from, i);
#pragma unroll
    for (int j = 0; j < kSub; ++j) to.b[j] = B.read(from + TL::kHalf, j);
  };
  auto read_scales = [&](const char* from, Scales<TL>& to) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(from) + lane;
#pragma unroll
    for (int i = 0; i < kSub; ++i) to.a[i] = w[(wr / 16 + i) * 64];
#pragma unroll
    for (int j = 0; j < kSub; ++j) to.b[j] = w[TL::kScales / 4 + (wc / 16 + j) * 64];
  };
  Acc<TL> acc;
#pragma unroll
  for (int i = 0; i < kSub; ++i)
#pragma unroll
    for (int j = 0; j < kSub; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  constexpr int L = 2 * TL::kLoads, K = TL::kScaleLoads;
  // Slice I of a chunk of scales in sc[C], its fragments in f[I & 1]: once all waves
  // have read it and the next one is there, its buffer is loaded anew.
  auto slice = [&](auto i_c, auto chunk_c) {
    constexpr int I = decltype(i_c)::value, C = decltype(chunk_c)::value;
    constexpr int now = I & 1, next = now ^ 1;
    // newer than the next slice: two slices, and scales asked for in their time
    slice_barrier<2 * L + (I == 1 || I == 2 ? K : 0)>();
    if constexpr (I == 0) load_scales(scl[C ^ 1]);
    const char* from = buf[(I + 1) & 3];
    if constexpr (T == 256) {
      begin_load();
      const uint32_t* words = reinterpret_cast<const uint32_t*>(scl[C ^ 1]) + lane;
#pragma unroll
      for (int t = 0; t < kSub * kSub; ++t) {
        const int i = t / kSub, j = t % kSub;
        multiply_in_place<I>(acc[i][j], f[now].b[j], sc[C].b[j], f[now].a[i], sc[C].a[i]);
        if (t % 3 == 0 && t / 3 < 2 * kSub) {
          const int c = t / 3;
          if (c < kSub) f[next].a[c] = A.read(from, c);
          else f[next].b[c - kSub] = B.read(from + TL::kHalf, c - kSub);
        }
        if (t % 6 == 2 && t / 6 < L) {
          const int r = t / 6;
          if (r < TL::kLoads) A.load_round(buf[I], wave, r);
          else B.load_round(buf[I] + TL::kHalf, wave, r - TL::kLoads);
        }
        if (I == 3 && t % 3 == 1 && t / 3 < 2 * kSub) {
          const int c = t / 3;
          if (c < kSub) sc[C ^ 1].a[c] = words[(wr / 16 + c) * 64];
          else sc[C ^ 1].b[c - kSub] = words[TL::kScales / 4 + (wc / 16 + c - kSub) * 64];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      end_load();
    } else {
      load(buf[I]);
      if constexpr (I == 3) read_scales(scl[C ^ 1], sc[C ^ 1]);
      read(from, f[next]);
#pragma unroll
      for (int i = 0; i < kSub; ++i)
#pragma unroll
        for (int j = 0; j < kSub; ++j)
          acc[i][j] = product_of<I>(f[now].b[j], sc[C].b[j], f[now].a[i], sc[C].a[i], acc[i][j]);
    }
  };
  auto round = [&](auto chunk_c) {
    slice(std::integral_constant<int, 0>{}, chunk_c);
    slice(std::integral_constant<int, 1>{}, chunk_c);
    slice(std::integral_constant<int, 2>{}, chunk_c);
    slice(std::integral_constant<int, 3>{}, chunk_c);
  };
  const int chunks = static_cast<int>((p.kb + 15) / 16);
  auto start = [&](auto chunk_c) {  // with its scales in place C
    constexpr int C = decltype(chunk_c)::value;
    load_scales(scl[C]);
#pragma unroll
    for (int i = 0; i < 4; ++i) load(buf[i]);
    if constexpr (T == 256) settle<TL>(acc);
    slice_barrier<3 * L>();
    read_scales(scl[C], sc[C]);
    read(buf[0], f[0]);
  };
  // pairs of chunks; an odd one goes before them
  if (chunks & 1) {
    start(std::integral_constant<int, 1>{});
    round(std::integral_constant<int, 1>{});
    // the compiler places moves where the ways in join
    if constexpr (T == 256) settle<TL>(acc);
  } else {
    start(std::integral_constant<int, 0>{});
  }
  for (int c = chunks / 2; c > 0; --c) {
    round(std::integral_constant<int, 0>{});
    round(std::integral_constant<int, 1>{});
  }
  if constexpr (T == 256) settle<TL>(acc);
  // nothing is left under way into LDS when the block ends
  __builtin_amdgcn_s_waitcnt(0x0F70);

  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int64_t row = r0 + wr + i * 16 + r;
    if (row < p.m) {
#pragma unroll
      for (int j = 0; j < kSub; ++j)
        store4(p, row, c0 + wc + row_of<kPairs>(j, g * 4), acc[i][j]);
    }
  }
}

// k == 0
__global__ void __launch_bounds__(256) mx4_zero_kernel(Problem p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  for (int64_t row = blockIdx.y; row < p.m; row += gridDim.y)
    if (c < p.n) store4(p, row, c, f32x4{0, 0, 0, 0});
}

// ---- host ---------------------------------------------------------------------------

using Text = std::string;

sbp_status check_sizes(const Text& w, int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0) return sbp::fail(SBP_EINVAL, w + ": m, n or k < 0");
  if (m > SBP_MX_MAX_DIM || n > SBP_MX_MAX_DIM || k > SBP_MX_MAX_K)
    return sbp::fail(SBP_ERANGE, w + ": a size above SBP_MX_MAX_DIM or SBP_MX_MAX_K");
  return SBP_OK;
}

constexpr int64_t kFewRows = 64;

// Side of the tiles.
int tile_of(int64_t m, int64_t n) {
  auto tiles = [&](int64_t T) { return ((m + T - 1) / T) * ((n + T - 1) / T); };
  if (tiles(256) >= 128) return 256;
  return tiles(128) >= 192 ? 128 : 64;
}

struct Layout {
  int64_t step_a, step_b, bytes;  // of a chunk's packed scales
};
Layout layout_of(int64_t m, int64_t n, int64_t kb, int T) {
  const int64_t a = (m + T - 1) / T * T * 16, b = (n + T - 1) / T * T * 16;
  return {a, b, (kb + 15) / 16 * (a + b)};
}

int64_t workspace_of(int64_t m, int64_t n, int64_t k) {
  if (m <= kFewRows || n == 0 || k == 0) return 0;
  return layout_of(m, n, sbp::mx4_blocks(k), tile_of(m, n)).bytes;
}

template <int T>
sbp_status run_tiles(const char* who, const Problem& p, char* ws, hipStream_t stream);

sbp_status launched(const char* who) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return sbp::fail(SBP_EHIP, Text(who) + ": launch failed: " + hipGetErrorString(e));
  return sbp::ok();
}

template <int T>
sbp_status run_tiles(const char* who, const Problem& p, char* ws, hipStream_t stream) {
  using TL = Tile<T>;
  const Layout l = layout_of(p.m, p.n, p.kb, T);
  const int64_t chunks = (p.kb + 15) / 16, words_a = l.step_a / 256 * chunks,
                words_b = l.step_b / 256 * chunks;
  const Pack a{p.sa, reinterpret_cast<uint32_t*>(ws), p.m, static_cast<int32_t>(l.step_a / 256), 0,
               TL::kSub};
  const Pack b{p.sb, reinterpret_cast<uint32_t*>(ws + chunks * l.step_a), p.n,
               static_cast<int32_t>(l.step_b / 256), p.f32 ? 0 : 1, TL::kSub};
  const unsigned blocks_a = static_cast<unsigned>((words_a + 3) / 4);
  const unsigned blocks_b = static_cast<unsigned>((words_b + 3) / 4);
  hipLaunchKernelGGL(mx4_pack_kernel, dim3(blocks_a + blocks_b), dim3(256), 0, stream, a, b, p.kb,
                     blocks_a);
  sbp_status st = launched(who);
  if (st != SBP_OK) return st;
  const unsigned total =
      static_cast<unsigned>(((p.m + T - 1) / T) * ((p.n + T - 1) / T));
  const Packed packed{ws, ws + chunks * l.step_a, l.step_a, l.step_b};
  if (p.f32)
    hipLaunchKernelGGL((mx4_tile_kernel<TL, kF32>), dim3(total), dim3(256), 0, stream, p, packed, total);
  else
    hipLaunchKernelGGL((mx4_tile_kernel<TL, kBf16>), dim3(total), dim3(256), 0, stream, p, packed, total);
  return launched(who);
}

sbp_status matmul_call(const char* who, const void* codes_a, const void* scales_a,
                       const void* codes_b, const void* scales_b, int64_t m, int64_t n, int64_t k,
                       void* out, int32_t type, int64_t ld, int32_t accumulate, void* workspace,
                       int64_t workspace_bytes, hipStream_t stream) {
  const Text w(who);
  sbp_status st = check_sizes(w, m, n, k);
  if (st != SBP_OK) return st;
  if (type != SBP_BF16 && type != SBP_F32)
    return sbp::fail(SBP_EINVAL, w + ": the type must be SBP_BF16 or SBP_F32");
  if (accumulate != 0 && type != SBP_F32)
    return sbp::fail(SBP_EINVAL, w + ": only SBP_F32 accumulates");
  if (m == 0 || n == 0 || (k == 0 && accumulate != 0)) return sbp::ok();
  if (out == nullptr) return sbp::fail(SBP_EINVAL, w + ": out is null");
  const int size = type == SBP_F32 ? 4 : 2;
  if (!sbp::aligned(out, size)) return sbp::fail(SBP_EALIGN, w + ": out is not aligned to its type");
  if (m > 1 && ld < n) return sbp::fail(SBP_EINVAL, w + ": a row distance below n");
  if (m > 1 && ld > int64_t{1} << 32) return sbp::fail(SBP_ERANGE, w + ": ld above 2^32");
  const int64_t kb = sbp::mx4_blocks(k), span = ((m > 1 ? (m - 1) * ld : 0) + n) * size;
  const int64_t need = workspace_of(m, n, k);
  if (k > 0) {
    if (codes_a == nullptr || scales_a == nullptr || codes_b == nullptr || scales_b == nullptr)
      return sbp::fail(SBP_EINVAL, w + ": null operand pointer");
    if (!sbp::aligned(codes_a, 16) || !sbp::aligned(codes_b, 16))
      return sbp::fail(SBP_EALIGN, w + ": codes must be 16-byte aligned");
    if (need > 0) {
      if (workspace == nullptr) return sbp::fail(SBP_EINVAL, w + ": workspace is null");
      if (!sbp::aligned(workspace, 256))
        return sbp::fail(SBP_EALIGN, w + ": workspace must be 256-byte aligned");
      if (workspace_bytes < need)
        return sbp::fail(SBP_EINVAL, w + ": workspace too small (see sbp_mx_matmul_workspace)");
    }
    const struct { const void* p; int64_t n; } in[] = {
        {codes_a, m * kb * 16}, {scales_a, m * kb}, {codes_b, n * kb * 16}, {scales_b, n * kb}};
    for (const auto& x : in) {
      if (sbp::overlaps(out, span, x.p, x.n))
        return sbp::fail(SBP_EINVAL, w + ": out overlaps an operand");
      if (need > 0 && sbp::overlaps(workspace, need, x.p, x.n))
        return sbp::fail(SBP_EINVAL, w + ": the workspace overlaps an operand");
    }
    if (need > 0 && sbp::overlaps(workspace, need, out, span))
      return sbp::fail(SBP_EINVAL, w + ": the workspace overlaps out");
  }
  Problem p{static_cast<const char*>(codes_a), static_cast<const char*>(codes_b),
            static_cast<const uint8_t*>(scales_a), static_cast<const uint8_t*>(scales_b),
            m, n, kb, out, ld, type == SBP_F32, accumulate != 0,
            sbp::aligned(out, 16) && (m == 1 || ld * size % 16 == 0)};
  (void)hipGetLastError();
  if (k == 0) {
    const dim3 grid(static_cast<unsigned>((n + 1023) / 1024),
                    static_cast<unsigned>(std::min<int64_t>(m, 1024)));
    hipLaunchKernelGGL(mx4_zero_kernel, grid, dim3(256), 0, stream, p);
    return launched(who);
  }
  if (m > kFewRows) {
    char* ws = static_cast<char*>(workspace);
    const int T = tile_of(m, n);
    return T == 256   ? run_tiles<256>(who, p, ws, stream)
           : T == 128 ? run_tiles<128>(who, p, ws, stream)
                      : run_tiles<64>(who, p, ws, stream);
  }
  const int64_t tiles = ((n + 15) / 16) * ((m + 15) / 16);
  if (tiles >= int64_t{1} << 24) return sbp::fail(SBP_ERANGE, w + ": too many results");
  const dim3 grid(static_cast<unsigned>(tiles));
  hipLaunchKernelGGL((mx4_few_kernel<1, 4>), grid, dim3(256), 0, stream, p);
  return launched(who);
}

}  // namespace

extern "C" {

int64_t sbp_mx_matmul_workspace(int64_t m, int64_t n, int64_t k) {
  try {
    if (check_sizes("sbp_mx_matmul_workspace", m, n, k) != SBP_OK) return -1;
    (void)sbp::ok();
    return workspace_of(m, n, k);
  } catch (...) {
    return -1;
  }
}

sbp_status sbp_mx_matmul(const void* codes_a, const void* scales_a, const void* codes_b,
                          const void* scales_b, int64_t m, int64_t n, int64_t k, void* out,
                          int32_t type, int64_t ld, int32_t accumulate, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream) {
  try {
    return matmul_call("sbp_mx_matmul", codes_a, scales_a, codes_b, scales_b, m, n, k, out, type,
                       ld, accumulate, workspace, workspace_bytes, stream);
  } catch (...) {
    return sbp::fail(SBP_ENOMEM, "sbp_mx_matmul: out of host memory");
  }
}

}  // extern "C"
