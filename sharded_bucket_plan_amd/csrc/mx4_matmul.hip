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

int64_t workspace_of(int64_t, int64_t, int64_t) { return 0; }

sbp_status launched(const char* who) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return sbp::fail(SBP_EHIP, Text(who) + ": launch failed: " + hipGetErrorString(e));
  return sbp::ok();
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
