// C = A B' of two microscaled 4-bit operands (mx4.h) on CDNA4's scaled matrix
// instructions.  Exact semantics are in include/sbp.h.
//
//   C[i][j] = sum over blocks b of 2^(sa[i][b] - 127) * 2^(sb[j][b] - 127)
//             * sum over the block's 32 values of a * b
//
// v_mfma_scale_f32_16x16x128 takes 16 rows of each operand and 128 contracted
// values: lane l holds row l % 16's block l / 16 of 32 values (16 bytes) and its
// scale byte; 32x32x64 takes 32 rows and two blocks of each.  Both apply the scales
// and sum in binary32.  B's rows go in as the first operand, A's as the second, so
// that a lane's results are neighbours in a row of C.
//
// What bounds it.  A few rows: B's codes and scales, once from memory (16 x 28672 x
// 4096, 62 MB, 12.6 us: 5.0 TB/s), and below some 10 MB the launch and one
// memory latency after another (1 x 4096 x 4096 4 us).  Many rows: the matrix units, of
// which large tiles keep 62% busy at 1.66 GHz, where the card's power holds them:
// the large tile's loop sustains 4.65 PFLOP/s on random data and 7.2 on zeros, and other
// orders of its loads, reads and products change nothing.  On two sets of operands in
// turn 8192 x 14336 x 4096 takes 237 to 249 us a call (3.9 to 4.1 PFLOP/s; 224 to 227
// repeated on one set), 4096 x 4096 x 8192 added to fp32 sums 85 to 87 (3.2; 78 repeated);
// 5 of them are the packing of the scales.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "bf16.h"
#include "internal.h"
#include "mx4.h"
#include "mx4_index.h"

#pragma clang fp contract(off)

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
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
  // small tiles: parts of the contracted axis, each of so many chunks of 512 values
  // and with sums of its own, this many elements further on
  int32_t parts, part_chunks;
  int64_t part_step;
  int64_t cols;  // of a row of out that may be written: n, padded for parts' sums
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

// An operand's scales as a lane takes them: 4 * W of a row at a time, `skip` blocks on.
// load() asks for them, at any address, and only fix() waits for them.  Past a row's end
// there are zeros; its last ones may end the array (of at least 4 * W), where the bytes
// before that are read.  No branch around the load, behind which the compiler would
// wait for all loads on the way.  WIDE: rows of whole chunks.
template <bool WIDE, int W>
struct RowScales {
  using Words = uint32_t __attribute__((ext_vector_type(W)));
  const uint8_t* row;
  const uint8_t* end;  // of all rows'
  int skip;
  __device__ __forceinline__ RowScales(const uint8_t* scales, int64_t r, int64_t rows, int64_t kb,
                                       int skip_)
      : row(scales + r * kb + skip_), end(scales + rows * kb), skip(skip_) {}
  RowScales() = default;
  __device__ __forceinline__ Words load(int64_t block) const {
    Words w;
    const uint8_t* from = row + block;
    if constexpr (!WIDE) from = from + 4 * W > end ? end - 4 * W : from;
    __builtin_memcpy(&w, from, 4 * W);
    return w;
  }
  __device__ __forceinline__ Words fix(Words w, int64_t block, int64_t kb) const {
    if (WIDE || block + 16 <= kb) return w;
    const int64_t over = row + block + 4 * W - end;
    const int shift = over > 0 ? static_cast<int>(over) : 0;  // bytes
    const int have = static_cast<int>(kb - block) - skip;
    Words out;
#pragma unroll
    for (int d = 0; d < W; ++d) {
      uint32_t lo = 0, hi = 0;  // words d + shift / 4 and the next
#pragma unroll
      for (int e = 0; e < W; ++e) {
        lo = e == d + (shift >> 2) ? w[e] : lo;
        hi = e == d + (shift >> 2) + 1 ? w[e] : hi;
      }
      const uint32_t x = __builtin_amdgcn_alignbyte(hi, lo, shift & 3);
      const int n = have - 4 * d;
      out[d] = n >= 4 ? x : n > 0 ? x & ((1u << (8 * n)) - 1) : 0u;
    }
    return out;
  }
};

// Of the 8 scales that a lane has of a row's 16, the lower half of the lanes the first
// and the upper half the others: to each half its own, the even or the odd ones, of both.
__device__ __forceinline__ u32x2 every_other(u32x2 w) {
  const uint32_t even = __builtin_amdgcn_perm(w.y, w.x, 0x06040200u);
  const uint32_t odd = __builtin_amdgcn_perm(w.y, w.x, 0x07050301u);
  const auto r = __builtin_amdgcn_permlane32_swap(even, odd, false, false);
  return u32x2{r[0], r[1]};
}
// Four neighbours of a row of C, from column c on.
__device__ __forceinline__ void store4(const Problem& p, int64_t row, int64_t c, f32x4 v) {
  const int64_t at = row * p.ld + c;
  if (p.f32) {
    float* o = static_cast<float*>(p.out) + at;
    if (c + 4 <= p.n) {
      if (p.accumulate) {
        f32x4 old;
        __builtin_memcpy(&old, o, 16);
        v = old + v;
      }
      __builtin_memcpy(o, &v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.n) o[i] = p.accumulate ? o[i] + v[i] : v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    const uint32_t w[4] = {sbp::bf16_rne(v.x), sbp::bf16_rne(v.y), sbp::bf16_rne(v.z),
                           sbp::bf16_rne(v.w)};
    if (c + 4 <= p.n) {
      const u32x2 x{w[0] | w[1] << 16, w[2] | w[3] << 16};
      __builtin_memcpy(o, &x, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.n) o[i] = static_cast<uint16_t>(w[i]);
    }
  }
}

// ---- few rows: 16 columns and 16 * MT rows of C a block ------------------------------
// Its W waves share the contracted axis: a wave takes every W-th chunk of 512 values
// (16 blocks, four products), with operands straight from memory, 4 KB of B's codes
// under way a wave.  The waves' sums meet in LDS, in the waves' order.  Also for an
// operand of fewer than 16 blocks in all, of any rows of A.
template <bool WIDE>
struct FewOperand {
  const char* codes;  // of this lane's row and its first block
  RowScales<WIDE, 4> scales;
  bool tiny;  // fewer than 16 blocks in all
};
template <bool WIDE>
struct Chunk {
  u32x4 codes[4];
  u32x4 scales;
  __device__ __forceinline__ void load(const FewOperand<WIDE>& o, int64_t c, int g, int64_t kb) {
    const bool whole = WIDE || c * 16 + 16 <= kb;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      codes[s] = u32x4{0, 0, 0, 0};
      if (whole || c * 16 + s * 4 + g < kb)
        codes[s] = *reinterpret_cast<const u32x4*>(o.codes + c * 256 + s * 64);
    }
    if (!WIDE && o.tiny) {  // then there is one chunk
      scales = u32x4{0, 0, 0, 0};
      for (int i = 0; i < kb; ++i)
        scales[i >> 2] |= static_cast<uint32_t>(o.scales.row[i]) << (8 * (i & 3));
    } else {
      scales = o.scales.load(c * 16);
    }
  }
  __device__ __forceinline__ void fix(const FewOperand<WIDE>& o, int64_t c, int64_t kb) {
    if (WIDE || !o.tiny) scales = o.scales.fix(scales, c * 16, kb);
  }
  // The lane's scale in the lowest byte.
  __device__ __forceinline__ uint32_t of(int s, int g) const { return scales[s] >> (8 * g); }
};

template <int MT, int W, bool WIDE>
__global__ void __launch_bounds__(W * 64) mx4_few_kernel(Problem p) {
  __shared__ f32x4 sums[W][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const unsigned across = static_cast<unsigned>((p.n + 15) / 16);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / across) * (16 * MT);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % across) * 16;
  // rows past the matrix read the last one; their results are not stored
  auto operand = [&](const char* codes, const uint8_t* scales, int64_t row, int64_t rows) {
    const int64_t at = row < rows ? row : rows - 1;
    return FewOperand<WIDE>{codes + (at * p.kb + g) * 16,
                            RowScales<WIDE, 4>(scales, at, rows, p.kb, 0), rows * p.kb < 16};
  };
  const FewOperand<WIDE> B = operand(p.b, p.sb, n0 + r, p.n);
  FewOperand<WIDE> A[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) A[i] = operand(p.a, p.sa, m0 + i * 16 + r, p.m);
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const int64_t chunks = (p.kb + 15) / 16;
  for (int64_t c = wave; c < chunks; c += W) {
    Chunk<WIDE> a[MT], b;
    b.load(B, c, g, p.kb);
#pragma unroll
    for (int i = 0; i < MT; ++i) a[i].load(A[i], c, g, p.kb);
    b.fix(B, c, p.kb);
#pragma unroll
    for (int i = 0; i < MT; ++i) a[i].fix(A[i], c, p.kb);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = product(b.codes[s], b.of(s, g), a[i].codes[s], a[i].of(s, g), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < MT) {
    f32x4 v = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v = v + sums[w][wave][lane];
    const int64_t row = m0 + wave * 16 + r;
    if (row < p.m) store4(p, row, n0 + g * 4, v);
  }
}

// ---- tiles --------------------------------------------------------------------------
// One T x T tile of C per block of 4 waves (2 x 2, each a quarter in 32 x 32 MFMA
// tiles, 64 contracted values at a time: lane l holds row l % 32's block l / 32).
// Slices of 128 contracted values (64 bytes of codes a row; 256 at the small tile) go
// straight from memory to one of four LDS buffers, four slices ahead.  The scales go
// by chunks of 512 values: at the large tile packed beforehand as the instruction
// takes them, and through LDS; else each lane takes its rows' from memory.
template <int T_, int BYTES>
struct Tile {
  static constexpr int T = T_, NB = 4;
  static constexpr bool kLarge = T == 256;
  static constexpr int kRow = BYTES;               // a row's part of a slice
  static constexpr int kSteps = kRow / 32;         // of 64 values
  static constexpr int kChunk = 256 / kRow;        // slices
  static constexpr int kHalf = T * kRow;           // one operand's slice, bytes
  static constexpr int kBuf = 2 * kHalf;           // A, then B
  static constexpr int kSub = T / 64;              // 32 x 32 tiles per wave and side
  static constexpr int kLoads = kHalf / 4096;      // per operand, slice and lane
  static constexpr int kScales = T * 16;           // one operand's scales of a chunk, bytes
  static constexpr int kScaleLoads = kLarge ? 2 * kScales / 4096 : 0;  // a lane's
};
using Large = Tile<256, 64>;
using Middle = Tile<128, 64>;
using Small = Tile<64, 128>;

// Row of B that row i of an MFMA tile holds.  A lane's results are rows 8q + 4h + t
// of B for its half h: with fp32 results four neighbours are 16 bytes; with bf16
// bits 2 and 3 change places, which makes 8 neighbours of two of the fours.
template <bool PAIRS>
__host__ __device__ __forceinline__ int row_of(int i) {
  return PAIRS ? (i & ~12) | ((i >> 1) & 4) | ((i << 1) & 8) : i;
}

// Scales of 32 rows and a chunk of 16 blocks as a wave takes them: lane (r, h) has
// two words, byte s % 4 of word s / 4 the scale of row r, block 2s + h, for its
// steps s = 0 .. 7 of 64 values.  Zeros past the matrix.
// packed: [chunk][tile of 32 rows][word][lane].
struct Pack {
  const uint8_t* scales;
  uint32_t* packed;
  int64_t rows;
  int32_t tiles, pairs;  // 32-row tiles, padded; B's order for bf16
};
__global__ void __launch_bounds__(256)
mx4_pack_kernel(Pack a, Pack b, int64_t kb, unsigned blocks_a) {
  const bool second = blockIdx.x >= blocks_a;
  const Pack p = second ? b : a;
  const unsigned w = second ? blockIdx.x - blocks_a : blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles = p.tiles, t = w % p.tiles, c0 = static_cast<int64_t>(w / p.tiles) * 8;
  const int64_t row = t * 32 + (p.pairs ? row_of<true>(lane & 31) : lane & 31);
  const RowScales<false, 2> from(p.scales, row < p.rows ? row : p.rows - 1, p.rows, kb,
                                 lane >> 5 << 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t c = c0 + wave + i * 4;
    if (c * 16 >= kb) break;
    u32x2 v = every_other(from.fix(from.load(c * 16), c * 16, kb));
    if (row >= p.rows) v = u32x2{0, 0};
    uint32_t* to = p.packed + (c * tiles + t) * 128 + lane;
    to[0] = v.x;
    to[64] = v.y;
  }
}

// `bytes` from p on as a buffer; loads from beyond them give zeros.  Whole offsets
// go into the vector one: a scalar offset past the end would lift the bound.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
typedef __attribute__((address_space(3))) void* lds_ptr;

// One operand of a tile.  LDS keeps a row's 16-byte pieces (the blocks of a slice)
// rotated by row, which spreads the reads over the banks; the rotation
// comes from the lanes' global addresses.
template <typename TL, bool PAIRS>
struct Operand {
  using Loads = sbp::Mx4Loads<TL::kRow>;
  static constexpr int kLanes = Loads::kLanes;  // that load a row
  const char* from;                             // next slice to load
  int bytes, piece;
  sbp::Mx4Offset round_bytes, all, voff;  // voff: `all`, or kMx4Past past the rows' end
  int at[TL::kSteps];                     // LDS offsets of this lane's first fragments

  static __device__ __forceinline__ int turn(int i) {  // of row i of an MFMA tile
    if constexpr (kLanes == 8) return (i >> 1) & 7;
    else return (((i >> 1) ^ (i >> 2)) & 2) | (((i >> 3) ^ (i >> 1)) & 1);
  }
  // wrow: the wave's first row in the tile
  __device__ __forceinline__ void init(int kb, int wave, int lane, int wrow) {
    const int row = Loads::row(wave, lane);
    piece = lane % kLanes ^ turn(row_of<PAIRS>(row & 31));  // row_of undoes itself
    all = Loads::first(row, kb, piece);
    round_bytes = Loads::round_bytes(kb);
    const int i = lane & 31, h = lane >> 5;
#pragma unroll
    for (int k = 0; k < TL::kSteps; ++k)
      at[k] = (wrow + row_of<PAIRS>(i)) * TL::kRow + ((2 * k + h) ^ turn(i)) * 16;
  }
  // At the first slice of the tile of rows r0 ..
  // and the chunk c0.
  __device__ __forceinline__ void aim(const char* codes, int64_t rows, int64_t kb, int64_t r0,
                                      int c0) {
    from = codes + r0 * kb * 16 + c0 * 256;
    // a 64-bit comparison is a vector instruction: the descriptor has to be scalar
    const int have = __builtin_amdgcn_readfirstlane(
        rows - r0 < TL::T ? static_cast<int>(rows - r0) : TL::T);
    bytes = have * static_cast<int>(kb) * 16 - c0 * 256;
    voff = all;
  }
  __device__ __forceinline__ void load_round(char* buf, int wave, int r) const {
    // a length below 0 would count as a huge one
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(from, bytes > 0 ? bytes : 0),
                                             (lds_ptr)(buf + (r * 4 + wave) * 1024), 16,
                                             static_cast<int>(Loads::at(voff, round_bytes, r)), 0,
                                             0, 0);
  }
  // To the next slice; `bytes` may go below 0.
  __device__ __forceinline__ void advance() {
    from += TL::kRow;
    bytes -= TL::kRow;
  }
  // `left` blocks of the rows remain for the next slice: the rest reads as zeros.
  __device__ __forceinline__ void cut(int left) {
    if (left < kLanes) voff = piece < left ? voff : sbp::kMx4Past;
  }
  // Step k of a slice, MFMA tile i.
  __device__ __forceinline__ u32x4 read(const char* buf, int k, int i) const {
    return *reinterpret_cast<const u32x4*>(buf + at[k] + i * 32 * TL::kRow);
  }
};

template <typename TL>
struct Frags {  // of a slice
  u32x4 a[TL::kSteps][TL::kSub], b[TL::kSteps][TL::kSub];
};
template <typename TL>
struct Scales {  // of a chunk: byte s % 4 of word s / 4 for its steps s of 64 values
  u32x2 a[TL::kSub], b[TL::kSub];
};
template <typename TL>
using Acc = f32x16[TL::kSub][TL::kSub];

// Step S of a chunk.
template <int S>
__device__ __forceinline__ f32x16 product_of(u32x4 b, u32x2 sb, u32x4 a, u32x2 sa, f32x16 c) {
  const i32x8 x{static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z),
                static_cast<int>(b.w), 0, 0, 0, 0};
  const i32x8 y{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                static_cast<int>(a.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, kFp4, kFp4, S & 3,
                                                         static_cast<int>(sb[S >> 2]), S & 3,
                                                         static_cast<int>(sa[S >> 2]));
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
//   whose reads the compiler waits for;
// - a product's own accumulator is used again 16 products later.
// tests/test_matrix_unit_distances.py reads from a build's disassembly that both
// distances hold on every path.
// FIRST: in place of a sum with what was there.
template <int S, bool FIRST>
__device__ __forceinline__ void multiply_in_place(f32x16& c, u32x4 b, u32x2 sb, u32x4 a,
                                                  u32x2 sa) {
  const uint32_t wb = sb[S >> 2], wa = sa[S >> 2];
#define SBP_MX_FORM(SUM, LO, HI)                                                           \
  "v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, " SUM ", %3, %4 op_sel:[" LO "," LO        \
  ",0] op_sel_hi:[" HI "," HI ",0] cbsz:4 blgp:4"
#define SBP_MX_PRODUCT(LO, HI)                                                             \
  if constexpr (FIRST)                                                                     \
    asm volatile(SBP_MX_FORM("0", LO, HI) : "=a"(c) : "v"(b), "v"(a), "v"(wb), "v"(wa));   \
  else                                                                                     \
    asm volatile(SBP_MX_FORM("%0", LO, HI) : "+a"(c) : "v"(b), "v"(a), "v"(wb), "v"(wa))
  if constexpr ((S & 3) == 0) { SBP_MX_PRODUCT("0", "0"); }
  if constexpr ((S & 3) == 1) { SBP_MX_PRODUCT("1", "0"); }
  if constexpr ((S & 3) == 2) { SBP_MX_PRODUCT("0", "1"); }
  if constexpr ((S & 3) == 3) { SBP_MX_PRODUCT("1", "1"); }
#undef SBP_MX_PRODUCT
#undef SBP_MX_FORM
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

enum Out { kBf16, kF32, kAdd };

// The first `left` values of 16 bytes of results.
template <Out O>
__device__ __forceinline__ void store_piece(char* to, int left, u32x4 w) {
  if constexpr (O == kBf16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(to);
    if (left >= 8) {
      __builtin_memcpy(o, &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* o = reinterpret_cast<float*>(to);
    f32x4 v = __builtin_bit_cast(f32x4, w);
    if (left >= 4) {
      if constexpr (O == kAdd) {
        f32x4 old;
        __builtin_memcpy(&old, o, 16);
        v = old + v;
      }
      __builtin_memcpy(o, &v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) o[i] = O == kAdd ? o[i] + v[i] : v[i];
    }
  }
}

// DIRECT: C's rows are made of whole 16-byte pieces on such addresses, a tile's within
// 2^31 bytes.
// WIDE: rows of whole chunks (small and middle tiles).
template <typename TL, Out O, bool DIRECT, bool WIDE>
__global__ void __launch_bounds__(256, TL::kLarge ? 1 : 2)
mx4_tile_kernel(Problem p, Packed packed, unsigned total) {
  constexpr int T = TL::T, kSub = TL::kSub;
  constexpr bool kPairs = O == kBf16, kLarge = TL::kLarge;
  // separate arrays: reads of one do not wait for loads into another
  __shared__ __align__(16) char buf0[TL::kBuf];
  __shared__ __align__(16) char buf1[TL::kBuf];
  __shared__ __align__(16) char buf2[TL::kBuf];
  __shared__ __align__(16) char buf3[TL::kBuf];
  __shared__ __align__(16) char scl[kLarge ? 2 * TL::kScales : 16];
  // for the results: the large tile's buffers hold the next tile meanwhile
  constexpr int kSlab = T == 64 && O == kBf16 ? 2048 : 4096;  // a wave's
  constexpr bool kOwnSlabs = kLarge || 4 * kSlab > TL::kBuf;
  __shared__ __align__(16) char slabs[kOwnSlabs ? 4 * kSlab : 16];
  constexpr int NB = TL::NB, kChunk = TL::kChunk, kSteps = TL::kSteps;
  char* buf[NB] = {buf0, buf1, buf2, buf3};
  const unsigned tr = static_cast<unsigned>((p.m + T - 1) / T);
  const unsigned tc = static_cast<unsigned>((p.n + T - 1) / T);
  // Neighbouring tiles to one XCD: an eighth of them to each.  Of the large ones a
  // block takes every (blocks / 8)-th of its XCD's.
  const unsigned per = (total + 7) / 8, step = gridDim.x / 8;
  unsigned index = blockIdx.x / 8;  // in the XCD's eighth
  const unsigned base = blockIdx.x % 8 * per;
  auto exists = [&](unsigned i) { return i < per && base + i < total; };
  if (!exists(index)) return;
  struct Place {
    unsigned ti, tj;
  };
  // Strips of 4 tile rows, column by column (4096 x 4096 x 4096 40.2 us, then, of 8 41.1; at
  // larger sizes within 0.5%, of 16 up to 2% behind).
  auto place_of = [&](unsigned i) {
    constexpr unsigned kStrip = 4;
    const unsigned t = (base + i) % (tr * tc);
    const unsigned strip = t / (kStrip * tc), left = tr - strip * kStrip;
    const unsigned high = left < kStrip ? left : kStrip, s = t - strip * kStrip * tc;
    // the divisions go by vector instructions: back to scalars
    return Place{static_cast<unsigned>(__builtin_amdgcn_readfirstlane(strip * kStrip + s % high)),
                 static_cast<unsigned>(__builtin_amdgcn_readfirstlane(s / high))};
  };
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wr = (wave >> 1) * (T / 2), wc = (wave & 1) * (T / 2);

  // The loads run four slices ahead of the products, on into the next tile.
  Operand<TL, false> A;
  Operand<TL, kPairs> B;
  A.init(static_cast<int>(p.kb), wave, lane, wr);
  B.init(static_cast<int>(p.kb), wave, lane, wc);
  const char *pa, *pb;
  int ahead;  // blocks from the next slice to load on
  const int part = kLarge ? 0 : __builtin_amdgcn_readfirstlane((base + index) / (tr * tc));
  const int first_chunk = part * p.part_chunks;
  auto aim = [&](Place t) {
    A.aim(p.a, p.m, p.kb, static_cast<int64_t>(t.ti) * T, first_chunk);
    B.aim(p.b, p.n, p.kb, static_cast<int64_t>(t.tj) * T, first_chunk);
    if constexpr (kLarge) {
      pa = packed.a + static_cast<int64_t>(t.ti) * TL::kScales;
      pb = packed.b + static_cast<int64_t>(t.tj) * TL::kScales;
    }
    // up to a part's end: the rest reads as zeros
    const int64_t end = kLarge ? p.kb : static_cast<int64_t>(first_chunk + p.part_chunks) * 16;
    ahead = __builtin_amdgcn_readfirstlane(static_cast<int>(end < p.kb ? end : p.kb)) -
            first_chunk * 16;
  };
  auto begin_load = [&]() {
    A.cut(ahead);
    B.cut(ahead);
  };
  auto end_load = [&]() {
    ahead -= TL::kRow / 16;
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
  auto load_scales = [&]() {
#pragma unroll
    for (int r = 0; r < TL::kScaleLoads; ++r) {
      const int off = (r * 4 + wave) * 1024;  // in A's scales, then B's
      const char* src = off < TL::kScales ? pa + off : pb + (off - TL::kScales);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(src, 1024), (lds_ptr)(scl + off), 16,
                                               lane * 16, 0, 0, 0);
    }
    pa += packed.step_a;
    pb += packed.step_b;
  };
  // small tiles: the lane's rows' scales; past the matrix the last row's
  RowScales<WIDE, 2> row_a[kSub], row_b[kSub];
  int64_t scale_block = static_cast<int64_t>(first_chunk) * 16;
  Frags<TL> f[2];
  Scales<TL> sc;
  u32x2 raw_a[kLarge ? 1 : kSub], raw_b[kLarge ? 1 : kSub];  // the next chunk's
  auto ask_scales = [&]() {
    // a chunk past the end repeats the last one's blocks; it is not used
    const int64_t last = (p.kb - 1) / 16 * 16;
    if (scale_block > last) scale_block = last;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      raw_a[i] = row_a[i].load(scale_block);
      raw_b[i] = row_b[i].load(scale_block);
    }
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      sc.a[i] = every_other(row_a[i].fix(raw_a[i], scale_block, p.kb));
      sc.b[i] = every_other(row_b[i].fix(raw_b[i], scale_block, p.kb));
    }
    scale_block += 16;
  };
  constexpr int kReads = 2 * kSteps * kSub;
  auto read_one = [&](const char* from, Frags<TL>& to, int c) {  // c: 0 .. kReads - 1
    const int k = c / (2 * kSub), i = c % (2 * kSub);
    if (i < kSub) to.a[k][i] = A.read(from, k, i);
    else to.b[k][i - kSub] = B.read(from + TL::kHalf, k, i - kSub);
  };
  auto read_scale = [&](int word, int c) {  // c: 0 .. 2 * kSub - 1
    const uint32_t* w = reinterpret_cast<const uint32_t*>(scl) + word * 64 + lane;
    if (c < kSub) sc.a[c][word] = w[(wr / 32 + c) * 128];
    else sc.b[c - kSub][word] = w[TL::kScales / 4 + (wc / 32 + c - kSub) * 128];
  };
  Acc<TL> acc;

  constexpr int L = 2 * TL::kLoads, K = TL::kScaleLoads;
  // Stores of a whole tile's results, a wave; 63 is what vmcnt can count.
  constexpr int kStores = kLarge && DIRECT ? (T / 2) * (T / 2) * (O == kBf16 ? 2 : 4) / 1024 : 0;
  // Slice I of a chunk, its fragments in f[I & 1]: once all waves have read it and
  // the next one is there, its buffer is loaded anew.  Slices 0 and 1 use the first
  // word of a chunk's scales, 2 and 3 the second: that one is read in slice 0, the
  // next chunk's first in slice 3, and the next chunk's are asked for in slice 1, when
  // all waves have read this one's.  FIRST: of a tile.
  auto slice = [&](auto i_c, auto first_c) {
    constexpr int I = decltype(i_c)::value;
    constexpr bool kFirst = decltype(first_c)::value;
    constexpr int now = I & 1, next = now ^ 1;
    // newer than the next slice: all other slices, scales asked for in their time, and
    // the last tile's stores where the next slice was asked for before them
    constexpr int kNewer = (NB - 2) * L + (I == 2 ? K : 0) + (kFirst && I < 3 ? kStores : 0);
    slice_barrier<(kNewer < 63 ? kNewer : 63)>();
    if constexpr (I == 1 && kLarge) load_scales();
    if constexpr (I % kChunk == 0 && !kLarge) ask_scales();
    const char* from = buf[(I + 1) % NB];
    if constexpr (kLarge) {
      begin_load();
      constexpr int kAll = kSub * kSub;
#pragma unroll
      for (int t = 0; t < 2 * kAll; ++t) {
        // to and fro along B: each product shares an operand with the one before (0.4%)
        const int i = t % kAll / kSub, j = i % 2 ? kSub - 1 - t % kSub : t % kSub;
        if (t < kAll)
          multiply_in_place<2 * I, kFirst && I == 0>(acc[i][j], f[now].b[0][j], sc.b[j],
                                                     f[now].a[0][i], sc.a[i]);
        else
          multiply_in_place<2 * I + 1, false>(acc[i][j], f[now].b[1][j], sc.b[j], f[now].a[1][i],
                                              sc.a[i]);
        // two reads, then a load, under each three products
        if (t % 3 < 2 && t / 3 * 2 + t % 3 < kReads) read_one(from, f[next], t / 3 * 2 + t % 3);
        if (t % 3 == 2 && t / 3 < L) {
          const int r = t / 3;
          if (r < TL::kLoads) A.load_round(buf[I], wave, r);
          else B.load_round(buf[I] + TL::kHalf, wave, r - TL::kLoads);
          if (I == 3) read_scale(0, r);
          if (I == 0) read_scale(1, r);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      end_load();
    } else {
      load(buf[I]);
#pragma unroll
      for (int c = 0; c < kReads; ++c) read_one(from, f[next], c);
      auto step = [&](auto k_c) {
        constexpr int k = decltype(k_c)::value;
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int j = 0; j < kSub; ++j)
            acc[i][j] = product_of<I % kChunk * kSteps + k>(f[now].b[k][j], sc.b[j],
                                                            f[now].a[k][i], sc.a[i], acc[i][j]);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      if constexpr (kSteps == 4) {
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
      }
      if constexpr (I % kChunk == kChunk - 1) take_scales();
    }
  };
  auto round = [&](auto first_c) {
    slice(std::integral_constant<int, 0>{}, first_c);
    slice(std::integral_constant<int, 1>{}, first_c);
    slice(std::integral_constant<int, 2>{}, first_c);
    slice(std::integral_constant<int, 3>{}, first_c);
  };

  constexpr int kPiece = O == kBf16 ? 8 : 4;                   // values
  constexpr int kSpan = T == 64 ? 32 : 16 * kPiece / 2;        // columns at a time
  constexpr int kPieces = kSpan / kPiece;                      // of a row: 8 or 4
  constexpr int kAtOnce = kSpan / 32;                          // MFMA tiles
  constexpr int kRows = 64 / kPieces;                          // a store covers
  static_assert(32 * kPieces * 16 == kSlab, "a wave's slab");
  // Results pass through LDS, 32 rows of 128 bytes at a time, for stores of whole
  // lines; 16-byte pieces are rotated by row against bank conflicts.  DIRECT: the rows
  // of C are a buffer, and what lies past C's end is dropped by its bound: always the
  // same number of stores.
  auto results = [&](Place t) {
    // addresses are worked out here, not kept in registers through the products
    unsigned lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const unsigned r = lane & 31, h = lane >> 5;
    char* slab = (kOwnSlabs ? slabs : buf0) + wave * kSlab;
    char* to = slab + r * (kPieces * 16);
    const unsigned key = (r / (16 / kPieces) % kPieces) ^ h;
    const unsigned row0 = lane / kPieces, piece = lane % kPieces;
    const unsigned turned = row0 * (kPieces * 16) + (piece ^ (row0 / (16 / kPieces))) * 16;
    constexpr int kSize = O == kBf16 ? 2 : 4;
    const int64_t r0 = static_cast<int64_t>(t.ti) * T + wr;
    const int64_t c0 = static_cast<int64_t>(t.tj) * T + wc;
    // as scalars: 64-bit comparisons are vector instructions
    const int have = __builtin_amdgcn_readfirstlane(
        static_cast<int>(p.m - r0 < T / 2 ? (p.m > r0 ? p.m - r0 : 0) : T / 2));
    const int wide = __builtin_amdgcn_readfirstlane(
        static_cast<int>(p.cols - c0 < T / 2 ? (p.cols > c0 ? p.cols - c0 : 0) : T / 2));
    char* corner = static_cast<char*>(p.out) + (r0 * p.ld + c0 + part * p.part_step) * kSize;
    const int line = static_cast<int>(p.ld) * kSize;  // DIRECT: below 2^23
    // the last row ends with its last column
    const auto rows = buffer(corner, have > 0 && wide > 0 ? (have - 1) * line + wide * kSize : 0);
    constexpr int kTimes = 32 / kRows, kParts = kSub / kAtOnce;  // of 32 rows
    auto offset = [&](int i, int j0) {
      const int c = j0 * 32 + piece * kPiece;
      return c < wide ? (i * 32 + row0) * line + c * kSize : 0x7FFFFFF0u;
    };
    // what the results are added to is asked for this many parts ahead (4096 x 4096 x
    // 8192 88.5 us with 1, 84.3 with 4)
    constexpr int kAhead = kSub * kParts < 4 ? kSub * kParts : 4;
    f32x4 old[O == kAdd ? kAhead : 1][kTimes];
    auto ask = [&](int part) {
      const unsigned off = offset(part / kParts, part % kParts * kAtOnce);
#pragma unroll
      for (int q = 0; q < kTimes; ++q)
        old[part % kAhead][q] = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, off + q * kRows * line, 0, 0));
    };
    if constexpr (DIRECT && O == kAdd) {
#pragma unroll
      for (int part = 0; part < kAhead; ++part) ask(part);
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
#pragma unroll
      for (int j0 = 0; j0 < kSub; j0 += kAtOnce) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          // one after the other: registers are short
          __builtin_amdgcn_sched_barrier(0);
          // and not read before their turn
          if constexpr (kLarge) asm volatile("" : "+a"(acc[i][j0 + j]));
          const f32x16 v = acc[i][j0 + j];
          if constexpr (O == kBf16) {
            typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              bf16x8 w;
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = static_cast<__bf16>(v[q * 8 + e]);
              *reinterpret_cast<u32x4*>(to + ((j * 4 + q * 2) ^ key) * 16) =
                  __builtin_bit_cast(u32x4, w);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<f32x4*>(to + ((j * 8 + q * 2) ^ key) * 16) =
                  f32x4{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
          }
        }
        auto from = [&](int q) {  // rows q * kRows ..
          return reinterpret_cast<const u32x4*>(
              slab + (q * 1024 + (kPieces == 8 ? turned ^ ((q & 1) * 64u) : turned)));
        };
        if constexpr (DIRECT) {
          const unsigned off = offset(i, j0);
          u32x4 w[kTimes];
          if constexpr (O == kAdd) {
            const int part = i * kParts + j0 / kAtOnce;
#pragma unroll
            for (int q = 0; q < kTimes; ++q)
              w[q] = __builtin_bit_cast(u32x4, old[part % kAhead][q] +
                                                   *reinterpret_cast<const f32x4*>(from(q)));
            if (part + kAhead < kSub * kParts) ask(part + kAhead);
          } else {
#pragma unroll
            for (int q = 0; q < kTimes; ++q) w[q] = *from(q);
          }
#pragma unroll
          for (int q = 0; q < kTimes; ++q)
            __builtin_amdgcn_raw_buffer_store_b128(w[q], rows, off + q * kRows * line, 0, 0);
        } else {
#pragma unroll 1
          for (int q = 0; q < kTimes; ++q) {
            const int row = i * 32 + q * kRows + row0, c = j0 * 32 + piece * kPiece;
            if (row < have && c < wide)
              store_piece<O>(corner + (row * p.ld + c) * kSize, wide - c, *from(q));
          }
        }
      }
    }
  };

  Place now = place_of(index);
  aim(now);
  if constexpr (kLarge) {
    load_scales();
  } else {
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      const int64_t ra = static_cast<int64_t>(now.ti) * T + wr + i * 32 + (lane & 31);
      const int64_t rb =
          static_cast<int64_t>(now.tj) * T + wc + i * 32 + row_of<kPairs>(lane & 31);
      const int half = lane >> 5 << 3;
      row_a[i] = RowScales<WIDE, 2>(p.sa, ra < p.m ? ra : p.m - 1, p.m, p.kb, half);
      row_b[i] = RowScales<WIDE, 2>(p.sb, rb < p.n ? rb : p.n - 1, p.n, p.kb, half);
    }
    ask_scales();
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) load(buf[i]);
  slice_barrier<kLarge ? 0 : (NB - 1) * L>();
  if constexpr (kLarge) {
#pragma unroll
    for (int c = 0; c < 2 * kSub; ++c) read_scale(0, c);
  } else {
    take_scales();
  }
#pragma unroll
  for (int c = 0; c < kReads; ++c) read_one(buf[0], f[0], c);
  const int all_chunks = static_cast<int>((p.kb + 15) / 16) - first_chunk;
  const int own = kLarge || all_chunks < p.part_chunks ? all_chunks : p.part_chunks;
  const int rounds = (own + NB / kChunk - 1) / (NB / kChunk);
  for (;;) {
    const bool more = kLarge && exists(index + step);
    const Place then = more ? place_of(index + step) : now;
    // from the last chunk on the loads are the next tile's, or none (a length of 0,
    // and scales that are not used)
    auto turn_to_next = [&]() {
      aim(then);
      if (!more) A.bytes = B.bytes = 0;
    };
    if constexpr (!kLarge) {
#pragma unroll
      for (int i = 0; i < kSub; ++i)
#pragma unroll
        for (int j = 0; j < kSub; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    }
    if (rounds == 1) turn_to_next();
    round(std::true_type{});
    // the compiler places moves where the ways join
    if constexpr (kLarge) settle<TL>(acc);
    for (int c = 1; c < rounds; ++c) {
      if (c + 1 == rounds) turn_to_next();
      round(std::false_type{});
    }
    if constexpr (kLarge) settle<TL>(acc);
    else slice_barrier<0>();  // the buffers are free
    results(now);
    if constexpr (!DIRECT) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): any number of them
    if (!more) break;
    index += step;
    now = then;
  }
  // nothing is left under way into LDS when the block ends
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// The parts' sums, in their order.
__global__ void __launch_bounds__(256)
mx4_join_kernel(Problem p, const float* parts, int32_t count, int64_t quads, int64_t step) {
  const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = q / quads;
  if (row >= p.m) return;
  const float* from = parts + q * 4;
  f32x4 v = *reinterpret_cast<const f32x4*>(from);
  for (int s = 1; s < count; ++s) v = v + *reinterpret_cast<const f32x4*>(from + s * step);
  store4(p, row, (q - row * quads) * 4, v);
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
  // 2^32 blocks of an operand are 64 GiB of codes; 2^36 results of 4 bytes 256 GiB
  const int64_t kb = sbp::mx4_blocks(k);
  if (m * kb > int64_t{1} << 32 || n * kb > int64_t{1} << 32 || m * n > int64_t{1} << 36)
    return sbp::fail(SBP_ERANGE, w + ": an operand above 2^32 blocks or a result above 2^36 values");
  return SBP_OK;
}

// How a product goes about it: the tiles' side, the parts of the contracted axis
// (chunks of 512 values each), and what the workspace holds.
struct Form {
  int T;  // 0: few rows
  int parts, part_chunks;
  int64_t step_a, step_b;  // large tile: bytes of a chunk's packed scales
  int64_t part_ld;         // parts: a row of their sums, elements
  int64_t bytes;
};
Form form_of(int64_t m, int64_t n, int64_t kb) {
  auto tiles = [&](int64_t T) { return ((m + T - 1) / T) * ((n + T - 1) / T); };
  const int64_t chunks = (kb + 15) / 16;
  Form f{};
  f.part_chunks = static_cast<int>(chunks);
  f.parts = 1;
  // Few rows: 16 x 8192 x 4096 6.3 us, with small tiles 6.8; 32 x 4096 x 4096 5.4 and
  // 7.0; but 32 x 8192 x 4096 8.6 and 7.0, 16 x 16384 x 4096 10.8 and 8.5, since each 16
  // columns read all of A.  (All at k = 4096; k is not looked at.)
  if (m == 1 || (m <= 32 && n <= 4096) || (m <= 16 && n <= 8192) || std::min(m, n) * kb < 16)
    return f;
  // Microseconds as measured (bf16 results), by the chunks c; 512 of the small and the
  // middle tiles run at once, 256 of the large.  fp32 and added results go by the same
  // costs, which do not know of their larger C.
  //                            small   middle   large
  //   1024 x 1024, c = 8 / 28    7 / 19  13 / 42  25 / 69
  //   1024 x 2048, c = 8           12      13       25
  //   2048 x 2048, c = 4 / 8     12 / 23  10 / 16  17 / 26
  //   4096 x 2048, c = 8           42      28       29
  //   4224 x 4224, c = 8           91      62       57
  //   4096 x 4096, c = 8 / 16    82 / 147 54 / 104 41 / 69
  //   4096 x 8192, c = 1 / 2     59 / 58  24 / 34  30 / 41
  //                c = 4 / 8     88 / 161 55 / 107 47 / 71
  //   8192 x 8192, c = 1           113      44       54 (taken: the fit is off here)
  const double c = static_cast<double>(chunks);
  const double t64 = tiles(64) / 512.0, t128 = tiles(128) / 512.0, t256 = tiles(256) / 256.0;
  const double rounds = std::floor(t256), rest = t256 - rounds;
  double cost64 = t64 < 1 ? 3 + c * std::max(0.6, 1.15 * t64) : t64 * (2.5 + 0.95 * c);
  double cost128 = t128 < 1 ? 3 + c * std::max(1.3, 3.1 * t128) : t128 * (3 + 3.1 * c);
  const double cost256 = 8 + rounds * (7 + 3 * c) + (rest > 0 ? c * (2.05 + 0.8 * rest) : 0);
  if (kb % 16) {
    // The small tile's scales at odd addresses and its cut last chunk: 64 x 4096 x 11008
    // 11.5, x 11264 11.0; 1440 x 1440 x 2304 13.9, x 2560 11.8; 2880 x 2880 x 2080 37.7,
    // with large tiles 23.9.  The middle tile has no registers for them: with spills 44.
    cost64 *= 1.2;
    cost128 = HUGE_VAL;
  }
  f.T = cost64 <= std::min(cost128, cost256) ? 64 : cost128 <= cost256 ? 128 : 256;
  // Few tiles and long sums: parts of at least four chunks, up to a tile a compute
  // unit.  256 x 256 x 14336 17.0, in 7 parts 9.6; 512 x 512 17.0, in 4 parts 11.9; but
  // 16 tiles c = 8 7.5, in 2 parts 8.3: the joining takes 3 to 4.
  int64_t parts = 1;
  if (f.T == 64 && chunks >= 12)
    parts = std::max<int64_t>(1, std::min(256 / tiles(64), chunks / 4));
  f.part_chunks = static_cast<int>((chunks + parts - 1) / parts);
  f.parts = static_cast<int>((chunks + f.part_chunks - 1) / f.part_chunks);
  if (f.T == 256) {
    f.step_a = (m + 255) / 256 * 4096;
    f.step_b = (n + 255) / 256 * 4096;
    f.bytes = chunks * (f.step_a + f.step_b);
  } else if (f.parts > 1) {
    f.part_ld = (n + 3) / 4 * 4;
    f.bytes = f.parts * m * f.part_ld * 4;
  }
  return f;
}

int64_t workspace_of(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0 || k == 0) return 0;
  return form_of(m, n, sbp::mx4_blocks(k)).bytes;
}

sbp_status launched(const char* who) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return sbp::fail(SBP_EHIP, Text(who) + ": launch failed: " + hipGetErrorString(e));
  return sbp::ok();
}

template <typename K>
sbp_status launch_tiles(const char* who, K kernel, const Problem& p, const Packed& packed, int T,
                        hipStream_t stream) {
  const unsigned total =
      static_cast<unsigned>(((p.m + T - 1) / T) * ((p.n + T - 1) / T) * p.parts);
  const unsigned per = (total + 7) / 8;
  const unsigned blocks = 8 * (T == 256 && per > 32 ? 32 : per);  // large: one a CU, 32 an XCD
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, stream, p, packed, total);
  return launched(who);
}

// C's rows as whole 16-byte pieces on such addresses, those of a tile within 2^31 bytes.
bool direct_of(const Problem& p) {
  const int64_t size = p.f32 ? 4 : 2;
  return p.m > 1 && sbp::aligned(p.out, 16) && p.ld * size % 16 == 0 && p.cols * size % 16 == 0 &&
         p.ld * size < int64_t{1} << 23;
}

sbp_status run_large(const char* who, const Problem& p, const Form& f, char* ws,
                     hipStream_t stream) {
  using TL = Large;
  const int64_t chunks = (p.kb + 15) / 16;
  const int32_t tiles_a = static_cast<int32_t>(f.step_a / 512);
  const int32_t tiles_b = static_cast<int32_t>(f.step_b / 512);
  const Pack a{p.sa, reinterpret_cast<uint32_t*>(ws), p.m, tiles_a, 0};
  const Pack b{p.sb, reinterpret_cast<uint32_t*>(ws + chunks * f.step_a), p.n, tiles_b, !p.f32};
  const unsigned blocks_a = static_cast<unsigned>((chunks + 7) / 8 * tiles_a);
  const unsigned blocks_b = static_cast<unsigned>((chunks + 7) / 8 * tiles_b);
  hipLaunchKernelGGL(mx4_pack_kernel, dim3(blocks_a + blocks_b), dim3(256), 0, stream, a, b, p.kb,
                     blocks_a);
  sbp_status st = launched(who);
  if (st != SBP_OK) return st;
  const Packed packed{ws, ws + chunks * f.step_a, f.step_a, f.step_b};
  auto of = [&](auto direct_c) -> sbp_status {
    constexpr bool kDirect = decltype(direct_c)::value;
    auto go = [&](auto kernel) { return launch_tiles(who, kernel, p, packed, 256, stream); };
    if (!p.f32) return go(mx4_tile_kernel<TL, kBf16, kDirect, true>);
    if (p.accumulate) return go(mx4_tile_kernel<TL, kAdd, kDirect, true>);
    return go(mx4_tile_kernel<TL, kF32, kDirect, true>);
  };
  return direct_of(p) ? of(std::true_type{}) : of(std::false_type{});
}

template <typename TL>
sbp_status run_small(const char* who, Problem p, const Form& f, char* ws, hipStream_t stream) {
  const Problem whole = p;
  p.parts = f.parts;
  p.part_chunks = f.part_chunks;
  if (f.parts > 1) {
    p.out = ws;
    p.ld = f.part_ld;
    p.f32 = 1;
    p.accumulate = 0;
    p.part_step = p.m * f.part_ld;
    p.cols = f.part_ld;
  }
  auto of = [&](auto direct_c, auto wide_c) -> sbp_status {
    constexpr bool kDirect = decltype(direct_c)::value, kWide = decltype(wide_c)::value;
    auto go = [&](auto kernel) { return launch_tiles(who, kernel, p, Packed{}, TL::T, stream); };
    if (!p.f32) return go(mx4_tile_kernel<TL, kBf16, kDirect, kWide>);
    if (p.accumulate) return go(mx4_tile_kernel<TL, kAdd, kDirect, kWide>);
    return go(mx4_tile_kernel<TL, kF32, kDirect, kWide>);
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  auto wide_of = [&](auto direct_c) {
    if constexpr (TL::T == 128) return of(direct_c, yes);
    else return p.kb % 16 == 0 ? of(direct_c, yes) : of(direct_c, no);
  };
  sbp_status st = direct_of(p) ? wide_of(yes) : wide_of(no);
  if (st != SBP_OK || f.parts == 1) return st;
  const int64_t quads = f.part_ld / 4;
  const dim3 grid(static_cast<unsigned>((quads * p.m + 255) / 256));
  hipLaunchKernelGGL(mx4_join_kernel, grid, dim3(256), 0, stream, whole,
                     reinterpret_cast<const float*>(ws), f.parts, quads, p.part_step);
  return launched(who);
}

sbp_status run_few(const char* who, const Problem& p, hipStream_t stream) {
  constexpr int kWaves = 4;
  auto go = [&](auto kernel) -> sbp_status {
    const int64_t rows = p.m <= 16 ? 16 : 32;
    const unsigned blocks = static_cast<unsigned>((p.n + 15) / 16 * ((p.m + rows - 1) / rows));
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kWaves * 64), 0, stream, p);
    return launched(who);
  };
  if (p.kb % 16)
    return p.m <= 16 ? go(mx4_few_kernel<1, kWaves, false>) : go(mx4_few_kernel<2, kWaves, false>);
  return p.m <= 16 ? go(mx4_few_kernel<1, kWaves, true>) : go(mx4_few_kernel<2, kWaves, true>);
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
            m, n, kb, out, ld, type == SBP_F32, accumulate != 0, 1,
            static_cast<int32_t>((kb + 15) / 16), 0, n};
  (void)hipGetLastError();
  if (k == 0) {
    const dim3 grid(static_cast<unsigned>((n + 1023) / 1024),
                    static_cast<unsigned>(std::min<int64_t>(m, 1024)));
    hipLaunchKernelGGL(mx4_zero_kernel, grid, dim3(256), 0, stream, p);
    return launched(who);
  }
  const Form f = form_of(m, n, kb);
  char* ws = static_cast<char*>(workspace);
  return f.T == 0     ? run_few(who, p, stream)
         : f.T == 256 ? run_large(who, p, f, ws, stream)
         : f.T == 128 ? run_small<Middle>(who, p, f, ws, stream)
                      : run_small<Small>(who, p, f, ws, stream);
}

}  // namespace

extern "C" {

int64_t sbp_mx_matmul_workspace(int64_t m, int64_t n, int64_t k) {
  try {
    if (check_sizes("sbp_mx_matmul_workspace", m, n, k) != SBP_OK) return -1;
    (void)sbp::ok();
    return workspace_of(m, n, k);
  } catch (...) {
    (void)sbp::fail(SBP_ENOMEM, "sbp_mx_matmul_workspace: out of host memory");
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
