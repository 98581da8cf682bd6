// The 4-bit exchange on CDNA4 (gfx950): values to microscaled 4-bit floats
// (mx4.h), back, and R peers' 4-bit chunks summed.  Exact semantics are in
// include/sbp.h.
//
// Per block of 32 values, with a = max |x| and E(a) its biased exponent:
//   nearest   s = max(E(a) - 2, 0): a lies in [4, 8) of 2^(s - 127); codes
//             round to nearest, ties to even, and above 6 saturate
//   random    s is one more where a > 6 * 2^(s - 127), so that nothing
//             saturates; with Y = floor(|x| * 2^(127 - s) * 2^17) a code's step
//             is 2^(16 + h), h = 0, 1, 2 for Y below 2^18, 2^19 and above, and
//             code = (((Y >> h) + r) >> 16) + 2h
//             for 16 random bits r: up with the probability of what is cut off
//             (its 16 highest bits), so the mean is x but for less than 2^-16
//             of a step
//   a NaN or an infinity in the block: s = 255 (all its values NaN), codes 0
// Random bits: Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy
// as 1, 2, 3", 2011), key = seed, counter = (block * 4 + octet, offset); eight
// half words for eight values.  They are never stored.
//
// Every kernel is one pass over memory.  A lane works on octets of 8 values,
// four neighbouring lanes on a block, so that loads and stores of a wave are
// contiguous and the block's maximum takes two lane exchanges.  Whole octets are 16
// bytes of bf16 (32 of fp32) at any address that fits their type: the hardware's
// vector loads and stores take those.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <type_traits>
#include <utility>

#include "bf16.h"
#include "internal.h"
#include "mx4.h"

#pragma clang fp contract(off)

namespace {

constexpr int kBlock = 256;
constexpr int kXcds = 8;
constexpr int kTile = 128;  // side of a tile of the matrix kernel

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Random {
  uint32_t key0, key1, off0, off1;
};

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Philox4x32-10 of the counter (index, its highest bit set where `upper`; offset).
__device__ __forceinline__ u32x4 philox(uint64_t index, bool upper, const Random& rnd) {
  uint32_t c0 = static_cast<uint32_t>(index);
  uint32_t c1 = static_cast<uint32_t>(index >> 32) | (upper ? 0x80000000u : 0u);
  uint32_t c2 = rnd.off0, c3 = rnd.off1, k0 = rnd.key0, k1 = rnd.key1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
    c1 = static_cast<uint32_t>(p1);
    c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// ---- eight values -------------------------------------------------------------

template <typename T>
struct Octet;

template <>
struct Octet<uint16_t> {  // bf16 bits, two a word
  u32x4 w;
  __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const uint16_t* p) { __builtin_memcpy(&w, p, 16); }
  __device__ __forceinline__ void load_some(const uint16_t* p, int64_t left) {
    auto one = [&](int j) -> uint32_t { return j < left ? p[j] : 0u; };
    w = u32x4{one(0) | one(1) << 16, one(2) | one(3) << 16, one(4) | one(5) << 16,
              one(6) | one(7) << 16};
  }
  // Largest magnitude, as binary32 bits (NaN above infinity above all else).
  __device__ __forceinline__ uint32_t top() const {
    u16x2 m = __builtin_bit_cast(u16x2, w.x & 0x7FFF7FFFu);
#pragma unroll
    for (int q = 1; q < 4; ++q)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[q] & 0x7FFF7FFFu));
    return static_cast<uint32_t>(m.x > m.y ? m.x : m.y) << 16;
  }
  __device__ __forceinline__ float value(int j) const {
    return j & 1 ? sbp::bf16_hi(w[j >> 1]) : sbp::bf16_lo(w[j >> 1]);
  }
  __device__ __forceinline__ uint32_t nearest(float scale) const {
    // through a copy: a bit cast of a vector's element takes the vector's first
    auto pair = [&](int q) {
      const uint32_t x = w[q];
      return __builtin_bit_cast(bf16x2, x);
    };
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, pair(0), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(1), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(2), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(3), scale, 3);
  }
};

template <>
struct Octet<float> {
  alignas(16) float v[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p) {
    f32x4 a, b;
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
  __device__ __forceinline__ void load_some(const float* p, int64_t left) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.0f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    return m;
  }
  __device__ __forceinline__ float value(int j) const { return v[j]; }
  __device__ __forceinline__ uint32_t nearest(float scale) const {
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
  }
};

// The larger of the four lanes' of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t a = __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  x = a > x ? a : x;
  const uint32_t b = __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return b > x ? b : x;
}

// Scale byte of a block whose largest magnitude has these binary32 bits.
template <bool RANDOM>
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  const uint32_t e = top >> 23;
  int s = static_cast<int>(e) - 2;
  if constexpr (RANDOM) s += (top & 0x7FFFFFu) > 0x400000u ? 1 : 0;
  s = s > 0 ? s : 0;
  return e == 255 ? 255u : static_cast<uint32_t>(s);
}

template <typename T>
__device__ __forceinline__ uint32_t random8(const Octet<T>& x, uint32_t s, u32x4 words) {
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = x.value(j);
    const uint32_t r = j & 1 ? words[j >> 1] >> 16 : words[j >> 1] & 0xFFFFu;
    const uint32_t Y =
        static_cast<uint32_t>(__builtin_ldexpf(fabsf(v), 144 - static_cast<int>(s)));
    const uint32_t top = Y >> 18, h = top < 2 ? top : 2;
    const uint32_t code = ((Y >> h) + r + (h << 17)) >> 16;
    out |= (code | ((__float_as_uint(v) >> 28) & 8u)) << (4 * j);
  }
  return out;
}

// Codes of an octet in a block of scale s; `index` is the octet's number.
template <bool RANDOM, typename T>
__device__ __forceinline__ uint32_t codes_of(const Octet<T>& x, uint32_t s, uint64_t index,
                                             bool upper, const Random& rnd) {
  uint32_t c;
  if constexpr (RANDOM) c = random8(x, s, philox(index, upper, rnd));
  else c = x.nearest(sbp::mx4_scale(s));
  return s == 255 ? 0u : c;
}

// ---- quantize: consecutive values ------------------------------------------------
// n values, zeros up to the last block's end.  An octet a lane: with four (64 lanes
// apart) 103.9M values in fp32 at random take 93 us, with one 79; in bf16 to nearest
// 47 and 45.
template <typename T, bool RANDOM>
__global__ void __launch_bounds__(kBlock)
quantize_flat_kernel(const T* __restrict__ x, int64_t n, int64_t blocks,
                     uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, Random rnd) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x, at = o * 8;
  Octet<T> v;
  if (at + 8 <= n) v.load(x + at);
  else if (at < n) v.load_some(x + at, n - at);
  else v.zero();
  const uint32_t s = scale_of<RANDOM>(quad_max(v.top()));
  const uint32_t c = codes_of<RANDOM>(v, s, static_cast<uint64_t>(o), false, rnd);
  if (o < blocks * 4) {
    codes[o] = c;
    if ((o & 3) == 0) scales[o >> 2] = static_cast<uint8_t>(s);
  }
}

// ---- quantize: a matrix's rows, columns, or both ------------------------------------
// A tile of 128 x 128: 16 lanes to a row for the rows' blocks; for the columns'
// the tile goes through LDS, a wave to 32 rows and a lane to two columns.
struct MatrixOut {
  uint32_t* codes;
  uint8_t* scales;
  int64_t blocks;  // of a row
};

template <typename T, bool RANDOM, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kBlock)
quantize_matrix_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                       MatrixOut along, MatrixOut across, Random rnd, unsigned total) {
  __shared__ __align__(16) T tile[COLS ? kTile * kTile : 1];
  // neighbouring tiles to one XCD, down strips of four: lines that several tiles write
  // parts of (a column's codes and scales, a row's codes) meet in its L2.  8192 x 4096 in
  // bf16, columns alone: along strips of two rows 26.2 us, this way 23.9
  unsigned t = blockIdx.x;
  const unsigned per = total / kXcds;
  if (t < per * kXcds) t = (t % kXcds) * per + t / kXcds;
  const unsigned tr = static_cast<unsigned>((rows + kTile - 1) / kTile);
  const unsigned tc = static_cast<unsigned>((cols + kTile - 1) / kTile);
  const unsigned strip = t / (4 * tr), left = t - strip * 4 * tr;
  const unsigned wide = tc - 4 * strip < 4 ? tc - 4 * strip : 4;
  const int64_t c0 = static_cast<int64_t>(4 * strip + left % wide) * kTile;
  const int64_t r0 = static_cast<int64_t>(left / wide) * kTile;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int oct = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t c = c0 + oct * 8;
  constexpr int kPasses = kTile / (kBlock / 16);
  Octet<T> v[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * 16 + row;
    const T* from = x + r * ld + c;
    if (r < rows && c + 8 <= cols) v[p].load(from);
    else if (r < rows && c < cols) v[p].load_some(from, cols - c);
    else v[p].zero();
  }
  if constexpr (COLS) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      *reinterpret_cast<Octet<T>*>(tile + (p * 16 + row) * kTile + oct * 8) = v[p];
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int64_t r = r0 + p * 16 + row, b = c0 / 32 + oct / 4;
      const int64_t o = (r * along.blocks + b) * 4 + (oct & 3);
      const uint32_t s = scale_of<RANDOM>(quad_max(v[p].top()));
      const uint32_t w = codes_of<RANDOM>(v[p], s, static_cast<uint64_t>(o), false, rnd);
      if (r < rows && b < along.blocks) {
        along.codes[o] = w;
        if ((oct & 3) == 0) along.scales[r * along.blocks + b] = static_cast<uint8_t>(s);
      }
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int64_t rb = r0 / 32 + wave;
    if (rb >= across.blocks) return;
    // two neighbouring columns of 32 rows stay in registers, each as four octets
    Octet<T> q[2][4];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const T* p = tile + (wave * 32 + i) * kTile + lane * 2;
      if constexpr (std::is_same_v<T, float>) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          q[k][i / 8].v[i % 8] = p[k];
          q[k][i / 8].v[i % 8 + 1] = p[kTile + k];
        }
      } else {
        const uint32_t lo = *reinterpret_cast<const uint32_t*>(p);
        const uint32_t hi = *reinterpret_cast<const uint32_t*>(p + kTile);
        q[0][i / 8].w[i % 8 / 2] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        q[1][i / 8].w[i % 8 / 2] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t col = c0 + lane * 2 + k;
      uint32_t top = 0;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const uint32_t m = q[k][o].top();
        top = m > top ? m : top;
      }
      const uint32_t s = scale_of<RANDOM>(top);
      const int64_t b = col * across.blocks + rb;
      u32x4 w;
#pragma unroll
      for (int o = 0; o < 4; ++o)
        w[o] = codes_of<RANDOM>(q[k][o], s, static_cast<uint64_t>(b * 4 + o), true, rnd);
      if (col < cols) {
        reinterpret_cast<u32x4*>(across.codes)[b] = w;
        across.scales[b] = static_cast<uint8_t>(s);
      }
    }
  }
}

// ---- dequantize ---------------------------------------------------------------------

__device__ __forceinline__ void store_octet(uint16_t* p, uint32_t w, float scale,
                                            int64_t left) {
  const u32x4 v{sbp::mx4_pair_bf16<0>(w, scale), sbp::mx4_pair_bf16<1>(w, scale),
                sbp::mx4_pair_bf16<2>(w, scale), sbp::mx4_pair_bf16<3>(w, scale)};
  if (left >= 8) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void store_octet(float* p, uint32_t w, float scale,
                                            int64_t left) {
  float v[8];
  sbp::mx4_octet(w, scale, v);
  if (left >= 8) {
    const f32x4 a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
    __builtin_memcpy(p, &a, 16);
    __builtin_memcpy(p + 4, &b, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = v[j];
  }
}

// FLAT: the rows' blocks and values lie one after the other.  An octet a lane, as
// above: 103.9M values to bf16 52 us, with four 56.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kBlock)
dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                  int64_t octets, int64_t row_octets, int64_t cols, int64_t ld,
                  T* __restrict__ out) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (o >= octets) return;
  const uint32_t w = codes[o], s = scales[o >> 2];
  int64_t at = o * 8, left = cols - at;
  if constexpr (!FLAT) {
    const int64_t row = octets <= UINT32_MAX
                            ? static_cast<uint32_t>(o) / static_cast<uint32_t>(row_octets)
                            : o / row_octets;
    const int64_t c = (o - row * row_octets) * 8;
    at = row * ld + c;
    left = cols - c;
  }
  if (left > 0) store_octet(out + at, w, sbp::mx4_scale(s), left);
}

// ---- reduce: out = fl((acc + S) * scale) ------------------------------------------------
struct Mx4Peers {
  const uint32_t* codes[SBP_MAX_PEERS];
  const uint8_t* scales[SBP_MAX_PEERS];
};

// An octet a lane: more of them fall behind as the peers grow (R = 8 with an
// accumulator, 103.9M values 237 us, with two 250; R = 2 without 116, with four 127).
template <int R, bool ACC>
__global__ void __launch_bounds__(kBlock)
reduce_mx4_kernel(Mx4Peers P, const float* acc, float scale, float* out, int64_t n) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x, left = n - o * 8;
  if (left <= 0) return;
  uint32_t w[R], s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    w[r] = P.codes[r][o];
    s[r] = P.scales[r][o >> 2];
  }
  Octet<float> a;
  if constexpr (ACC) {
    if (left >= 8) a.load(acc + o * 8);
    else a.load_some(acc + o * 8, left);
  }
  float S[8], v[8];
  sbp::mx4_octet(w[0], sbp::mx4_scale(s[0]), S);
#pragma unroll
  for (int r = 1; r < R; ++r) {
    sbp::mx4_octet(w[r], sbp::mx4_scale(s[r]), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) S[j] = S[j] + v[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (ACC) S[j] = a.v[j] + S[j];
    S[j] = S[j] * scale;
  }
  if (left >= 8) {
    f32x4* p = reinterpret_cast<f32x4*>(out + o * 8);
    p[0] = f32x4{S[0], S[1], S[2], S[3]};
    p[1] = f32x4{S[4], S[5], S[6], S[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) out[o * 8 + j] = S[j];
  }
}

// ---- host ------------------------------------------------------------------------------

using Text = std::string;

sbp_status launched(const char* who) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return sbp::fail(SBP_EHIP, Text(who) + ": launch failed: " + hipGetErrorString(e));
  return sbp::ok();
}

constexpr int64_t kMaxLd = int64_t{1} << 40;    // elements from row to row
constexpr int64_t kMaxSpan = int64_t{1} << 60;  // rows * ld: the bytes of a span fit 63 bits

int type_bytes(int32_t type) { return type == SBP_F32 ? 4 : 2; }

// Sizes of a matrix and its row distance; down: its columns are cut into blocks too, or
// its tiles of 128 x 128 are counted.
sbp_status check_matrix(const Text& w, int64_t rows, int64_t cols, int64_t ld, int32_t type,
                        bool down) {
  if (type != SBP_BF16 && type != SBP_F32)
    return sbp::fail(SBP_EINVAL, w + ": the type must be SBP_BF16 or SBP_F32");
  if (rows < 0 || cols < 0) return sbp::fail(SBP_EINVAL, w + ": rows or cols < 0");
  if (rows == 0 || cols == 0) return SBP_OK;
  if (rows > 1 && ld < cols) return sbp::fail(SBP_EINVAL, w + ": a row distance below cols");
  if (rows > 1 && ld > kMaxLd) return sbp::fail(SBP_ERANGE, w + ": a row distance above 2^40");
  const int64_t most = SBP_MAX_SHARD_NUMEL;
  if (rows > most || cols > most || sbp::mx4_blocks(cols) * 32 > most / rows ||
      (down && sbp::mx4_blocks(rows) * 32 > most / cols))
    return sbp::fail(SBP_ERANGE, w + ": more than SBP_MAX_SHARD_NUMEL values in whole blocks");
  if (rows > 1 && ld > kMaxSpan / rows)
    return sbp::fail(SBP_ERANGE, w + ": rows * ld above 2^60");
  return SBP_OK;
}

struct Bytes {
  const void* p;
  int64_t n;
};

// Whether any of the first `outs` ranges overlaps another one.
bool any_overlap(const Bytes* r, int n, int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (sbp::overlaps(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
  return false;
}

unsigned grid_of(int64_t octets) {
  return static_cast<unsigned>((octets + kBlock - 1) / kBlock);
}

// Calls f(std::integral_constant<int, R>) for R in 1..16.
template <typename F, int... I>
sbp_status with_peers(int32_t R, F&& f, std::integer_sequence<int, I...>) {
  sbp_status st = SBP_EINVAL;
  (void)((R == I + 1 ? (st = f(std::integral_constant<int, I + 1>{}), true) : false) || ...);
  return st;
}

template <typename T>
sbp_status quantize(const char* who, const T* x, int64_t rows, int64_t cols, int64_t ld,
                    MatrixOut along, MatrixOut across, bool random, Random rnd,
                    hipStream_t stream) {
  auto go = [&](auto random_c) -> sbp_status {
    constexpr bool kRandom = decltype(random_c)::value;
    if (across.codes == nullptr && (rows == 1 || (ld == cols && cols % 32 == 0))) {
      const int64_t n = rows * cols, blocks = sbp::mx4_blocks(n);
      auto flat = [&](auto kernel) -> sbp_status {
        hipLaunchKernelGGL(kernel, dim3(grid_of(blocks * 4)), dim3(kBlock), 0, stream, x, n, blocks,
                           along.codes, along.scales, rnd);
        return launched(who);
      };
      return flat(quantize_flat_kernel<T, kRandom>);
    }
    const int64_t tiles = ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
    auto matrix = [&](auto kernel) -> sbp_status {
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tiles)), dim3(kBlock), 0, stream, x,
                         rows, cols, ld, along, across, rnd, static_cast<unsigned>(tiles));
      return launched(who);
    };
    if (across.codes == nullptr) return matrix(quantize_matrix_kernel<T, kRandom, true, false>);
    if (along.codes == nullptr) return matrix(quantize_matrix_kernel<T, kRandom, false, true>);
    return matrix(quantize_matrix_kernel<T, kRandom, true, true>);
  };
  return random ? go(std::true_type{}) : go(std::false_type{});
}

sbp_status quantize_call(const char* who, const void* x, int32_t type, int64_t rows, int64_t cols,
                         int64_t ld, void* codes, void* scales, void* codes_t, void* scales_t,
                         const sbp_mx_random* random, hipStream_t stream) {
  const Text w(who);
  sbp_status st = check_matrix(w, rows, cols, ld, type, rows > 1 || codes_t != nullptr);
  if (st != SBP_OK) return st;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return sbp::fail(SBP_EINVAL, w + ": codes without scales, or scales without codes");
  if (rows == 0 || cols == 0) return sbp::ok();  // nothing is read or written
  if (codes == nullptr && codes_t == nullptr) return sbp::fail(SBP_EINVAL, w + ": no output");
  if (x == nullptr) return sbp::fail(SBP_EINVAL, w + ": x is null");
  const int size = type_bytes(type);
  if (!sbp::aligned(x, size)) return sbp::fail(SBP_EALIGN, w + ": x is not aligned to its type");
  if (!sbp::aligned(codes, 16) || !sbp::aligned(codes_t, 16))
    return sbp::fail(SBP_EALIGN, w + ": codes must be 16-byte aligned");
  const int64_t kb = sbp::mx4_blocks(cols), kt = sbp::mx4_blocks(rows);
  const int64_t span = ((rows > 1 ? (rows - 1) * ld : 0) + cols) * size;
  const Bytes ranges[] = {{codes, codes ? rows * kb * 16 : 0},
                          {scales, scales ? rows * kb : 0},
                          {codes_t, codes_t ? cols * kt * 16 : 0},
                          {scales_t, scales_t ? cols * kt : 0},
                          {x, span}};
  if (any_overlap(ranges, 5, 4)) return sbp::fail(SBP_EINVAL, w + ": buffers overlap");
  Random rnd{0, 0, 0, 0};
  if (random != nullptr)
    rnd = Random{static_cast<uint32_t>(random->seed), static_cast<uint32_t>(random->seed >> 32),
                 static_cast<uint32_t>(random->offset),
                 static_cast<uint32_t>(random->offset >> 32)};
  const MatrixOut along{static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales), kb};
  const MatrixOut across{static_cast<uint32_t*>(codes_t), static_cast<uint8_t*>(scales_t), kt};
  (void)hipGetLastError();
  if (type == SBP_F32)
    return quantize(who, static_cast<const float*>(x), rows, cols, ld, along, across,
                    random != nullptr, rnd, stream);
  return quantize(who, static_cast<const uint16_t*>(x), rows, cols, ld, along, across,
                  random != nullptr, rnd, stream);
}

template <typename T>
sbp_status dequantize(const char* who, const void* codes, const void* scales, int64_t rows,
                      int64_t cols, T* out, int64_t ld, hipStream_t stream) {
  const int64_t row_octets = sbp::mx4_blocks(cols) * 4, octets = rows * row_octets;
  const bool flat = rows == 1 || (ld == cols && cols % 32 == 0);
  const int64_t width = flat ? rows * cols : cols;
  auto go = [&](auto kernel) -> sbp_status {
    hipLaunchKernelGGL(kernel, dim3(grid_of(octets)), dim3(kBlock), 0, stream,
                       static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales),
                       octets, row_octets, width, ld, out);
    return launched(who);
  };
  return flat ? go(dequantize_kernel<T, true>) : go(dequantize_kernel<T, false>);
}

sbp_status dequantize_call(const char* who, const void* codes, const void* scales, int64_t rows,
                           int64_t cols, void* out, int32_t type, int64_t ld, hipStream_t stream) {
  const Text w(who);
  sbp_status st = check_matrix(w, rows, cols, ld, type, false);
  if (st != SBP_OK) return st;
  if (rows == 0 || cols == 0) return sbp::ok();  // nothing is read or written
  if (codes == nullptr || scales == nullptr || out == nullptr)
    return sbp::fail(SBP_EINVAL, w + ": null pointer");
  const int size = type_bytes(type);
  if (!sbp::aligned(codes, 16)) return sbp::fail(SBP_EALIGN, w + ": codes must be 16-byte aligned");
  if (!sbp::aligned(out, size)) return sbp::fail(SBP_EALIGN, w + ": out is not aligned to its type");
  const int64_t kb = sbp::mx4_blocks(cols);
  const Bytes ranges[] = {{out, ((rows > 1 ? (rows - 1) * ld : 0) + cols) * size},
                          {codes, rows * kb * 16},
                          {scales, rows * kb}};
  if (any_overlap(ranges, 3, 1)) return sbp::fail(SBP_EINVAL, w + ": out overlaps an input");
  (void)hipGetLastError();
  if (type == SBP_F32)
    return dequantize(who, codes, scales, rows, cols, static_cast<float*>(out), ld, stream);
  return dequantize(who, codes, scales, rows, cols, static_cast<uint16_t*>(out), ld, stream);
}

sbp_status reduce_call(const char* who, const void* const* codes, const void* const* scales,
                       int32_t R, int64_t n, const float* acc, float scale, float* out,
                       hipStream_t stream) {
  const Text w(who);
  if (R < 1 || R > SBP_MAX_PEERS) return sbp::fail(SBP_EINVAL, w + ": R must be in 1..16");
  if (n < 0) return sbp::fail(SBP_EINVAL, w + ": n < 0");
  if (n == 0) return sbp::ok();  // nothing is read or written
  if (codes == nullptr || scales == nullptr)
    return sbp::fail(SBP_EINVAL, w + ": codes or scales is null");
  if (out == nullptr) return sbp::fail(SBP_EINVAL, w + ": out is null");
  if (!sbp::aligned(out, 16) || !sbp::aligned(acc, 16))
    return sbp::fail(SBP_EALIGN, w + ": acc and out must be 16-byte aligned");
  if (n > SBP_MAX_SHARD_NUMEL) return sbp::fail(SBP_ERANGE, w + ": n above SBP_MAX_SHARD_NUMEL");
  const int64_t blocks = sbp::mx4_blocks(n);
  Mx4Peers P{};
  for (int32_t r = 0; r < R; ++r) {
    if (codes[r] == nullptr || scales[r] == nullptr)
      return sbp::fail(SBP_EINVAL, w + ": a peer pointer is null");
    if (!sbp::aligned(codes[r], 16))
      return sbp::fail(SBP_EALIGN, w + ": peers' codes must be 16-byte aligned");
    if (sbp::overlaps(out, 4 * n, codes[r], 16 * blocks) || sbp::overlaps(out, 4 * n, scales[r], blocks))
      return sbp::fail(SBP_EINVAL, w + ": out overlaps a peer");
    P.codes[r] = static_cast<const uint32_t*>(codes[r]);
    P.scales[r] = static_cast<const uint8_t*>(scales[r]);
  }
  if (acc != nullptr && acc != out && sbp::overlaps(out, 4 * n, acc, 4 * n))
    return sbp::fail(SBP_EINVAL, w + ": out overlaps acc without being it");
  (void)hipGetLastError();
  return with_peers(R, [&](auto rc) -> sbp_status {
    constexpr int RR = decltype(rc)::value;
    auto go = [&](auto kernel) -> sbp_status {
      hipLaunchKernelGGL(kernel, dim3(grid_of(blocks * 4)), dim3(kBlock), 0, stream, P, acc,
                         scale, out, n);
      return launched(who);
    };
    return acc ? go(reduce_mx4_kernel<RR, true>) : go(reduce_mx4_kernel<RR, false>);
  }, std::make_integer_sequence<int, SBP_MAX_PEERS>{});
}

}  // namespace

extern "C" {

sbp_status sbp_mx_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld,
                            void* codes, void* scales, void* codes_t, void* scales_t,
                            const sbp_mx_random* random, hipStream_t stream) {
  const char* who = "sbp_mx_quantize";
  try {
    return quantize_call(who, x, type, rows, cols, ld, codes, scales, codes_t, scales_t, random,
                         stream);
  } catch (...) {
    return sbp::fail(SBP_ENOMEM, "sbp_mx_quantize: out of host memory");
  }
}

sbp_status sbp_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols,
                              void* out, int32_t type, int64_t ld, hipStream_t stream) {
  const char* who = "sbp_mx_dequantize";
  try {
    return dequantize_call(who, codes, scales, rows, cols, out, type, ld, stream);
  } catch (...) {
    return sbp::fail(SBP_ENOMEM, "sbp_mx_dequantize: out of host memory");
  }
}

sbp_status sbp_mx_reduce_shard(const void* const* codes, const void* const* scales, int32_t R,
                                int64_t n, const float* acc, float scale, float* out,
                                hipStream_t stream) {
  const char* who = "sbp_mx_reduce_shard";
  try {
    return reduce_call(who, codes, scales, R, n, acc, scale, out, stream);
  } catch (...) {
    return sbp::fail(SBP_ENOMEM, "sbp_mx_reduce_shard: out of host memory");
  }
}

}  // extern "C"
