// Rows of K and V between bf16 and the 8-bit caches (E4M3 codes with one fp32 scale per
// token and KV head): quantised as they are written, and read back.
//
// Writing a row x of 128 bf16 values: a = the largest finite |x_d|, scale = a / 448 rounded
// to fp32 (1 for a row of zeros), code_d = the E4M3 value nearest to the exact quotient
// 448 x_d / a, ties to even.  E4M3 has no infinities: an infinite or NaN x_d becomes the NaN
// code, so a broken element stays visible in the cache and spoils no other.
//
// Rounding the exact quotient without a division per element: with inv = fl(448 / a) the
// product y = fl(x_d inv) is within 2^-22 of the quotient.  A tie of the E4M3 grid has at most
// five significant bits, and a quotient 7 X 2^m / A of integers X, A < 2^8 that is not a tie T
// differs from it by at least 1 / (31 * 255) > 2^-13 of it (the integers 7 X 2^m and T A
// differ by one at least).  So y rounded to 17 fraction bits (18 significant ones) is the tie
// itself when the quotient is one, and on the quotient's side of it when not: the conversion of
// that gives the correctly rounded code.
//
// Eight lanes take a row, 16 values each (32 bytes of bf16, 16 of codes), so a warp moves 1 KB and
// 512 bytes in one piece; K and V are the grid's y.  Bound by HBM, 388 bytes per row either way:
// 8 x 32,768 tokens of 2 KV heads written in 62.0 us (6.57 TB/s, 0.97 of a copy's rate), 131,072
// rows of 4 KV heads read back in 58.8 us (6.9 TB/s; 65 us before each lane stored its 32 bytes at
// once).  A single token per sequence: 1.6 us, the launch.
#include "kv_codes.h"
#include "ptx_blocks.cuh"

namespace embla {
namespace {

constexpr int kCodeThreads = 256;
constexpr int kLanesPerRow = 8;
constexpr int kRowsPerBlock = kCodeThreads / kLanesPerRow;
constexpr uint32_t kBf16Inf = 0x7F80u;
// below 2^-109 the reciprocal 448 / a could overflow: such rows divide
constexpr uint32_t kBf16Tiny = 0x0900u;

// y rounded to 17 fraction bits (to nearest; y is finite).
__device__ __forceinline__ float snap17(float y) {
  return __uint_as_float((__float_as_uint(y) + 0x20u) & ~0x3Fu);
}

// The two bf16 halves of w as magnitudes, infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_abs2(uint32_t w) {
  uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  if (lo >= kBf16Inf) lo = 0u;
  if (hi >= kBf16Inf) hi = 0u;
  return lo | (hi << 16);
}

// The largest of a row's packed magnitudes, over the lane's words and the row's lanes.
__device__ __forceinline__ uint32_t row_max(const uint32_t (&m)[8]) {
  uint32_t x = m[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) x = __vmaxs2(x, m[i]);
#pragma unroll
  for (int o = 1; o < kLanesPerRow; o <<= 1) x = __vmaxs2(x, __shfl_xor_sync(0xffffffffu, x, o));
  return max(x & 0xFFFFu, x >> 16);
}

// One element by division (rows holding an infinity or NaN, tiny rows, rows of zeros).  The
// quotient's terms are scaled down together where 448 x could overflow.
__device__ __forceinline__ float quotient(uint32_t bits, float a) {
  if ((bits & 0x7FFFu) >= kBf16Inf) return __uint_as_float(0x7FC00000u);
  const float f = a >= 1.0f ? 0x1p-20f : 1.0f;
  return a > 0.0f ? __fdiv_rn(__uint_as_float(bits << 16) * f * 448.0f, a * f) : 0.0f;
}

__global__ void __launch_bounds__(kCodeThreads) quantize_rows_kernel(const QuantizeParams p) {
  pdl_wait_primary();  // the rows are written; whoever read the cache's old rows is done
  pdl_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const uint16_t *rows = is_v ? p.job[1].src : p.job[0].src;
  uint8_t *codes = is_v ? p.job[1].codes : p.job[0].codes;
  float *scales = is_v ? p.job[1].scales : p.job[0].scales;
  const uint32_t part = threadIdx.x % kLanesPerRow;
  const uint32_t r = blockIdx.x * kRowsPerBlock + threadIdx.x / kLanesPerRow;
  const bool live = r < p.rows;
  uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
  if (live) {
    const uint4 *src = reinterpret_cast<const uint4 *>(rows + static_cast<int64_t>(r) * kHeadDim) + 2 * part;
    x0 = __ldcs(src);
    x1 = __ldcs(src + 1);
  }
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = w[i] & 0x7FFF7FFFu;
  uint32_t top = row_max(m);
  const bool plain = top < kBf16Inf && top >= kBf16Tiny;
  if (__any_sync(0xffffffffu, top >= kBf16Inf)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = finite_abs2(w[i]);
    top = row_max(m);
  }
  const float a = __uint_as_float(top << 16);
  uint32_t code[4];
  if (plain) {
    const float inv = __fdiv_rn(448.0f, a);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      code[i] = f32x4_to_e4m3x4(snap17(bf16lo(w[2 * i]) * inv), snap17(bf16hi(w[2 * i]) * inv),
                                snap17(bf16lo(w[2 * i + 1]) * inv), snap17(bf16hi(w[2 * i + 1]) * inv));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      code[i] = f32x4_to_e4m3x4(quotient(w[2 * i] & 0xFFFFu, a), quotient(w[2 * i] >> 16, a),
                                quotient(w[2 * i + 1] & 0xFFFFu, a), quotient(w[2 * i + 1] >> 16, a));
  }
  if (!live) return;
  const uint32_t u = r / static_cast<uint32_t>(p.tokens);
  const int64_t row = u * p.cache_stride + p.pos + (r - u * static_cast<uint32_t>(p.tokens));
  reinterpret_cast<uint4 *>(codes + row * kHeadDim)[part] = make_uint4(code[0], code[1], code[2], code[3]);
  if (part == 0) scales[row] = a > 0.0f ? __fdiv_rn(a, 448.0f) : 1.0f;
}

// The four codes of c times s as bf16 (product in fp32, then rounded to nearest even).
__device__ __forceinline__ uint2 scaled_bf16x4(uint32_t c, float s) {
  float v0, v1, v2, v3;
  e4m3x4_to_f32(c, v0, v1, v2, v3);
  return make_uint2(pack_bf16x2(v0 * s, v1 * s), pack_bf16x2(v2 * s, v3 * s));
}

__global__ void __launch_bounds__(kCodeThreads) dequantize_rows_kernel(const DequantizeParams p) {
  pdl_wait_primary();  // the cache's rows are written
  pdl_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const uint8_t *codes = is_v ? p.job[1].codes : p.job[0].codes;
  const float *scales = is_v ? p.job[1].scales : p.job[0].scales;
  uint16_t *rows = is_v ? p.job[1].dst : p.job[0].dst;
  const uint32_t part = threadIdx.x % kLanesPerRow;
  const uint32_t r = blockIdx.x * kRowsPerBlock + threadIdx.x / kLanesPerRow;
  if (r >= p.rows) return;
  const uint32_t u = r / static_cast<uint32_t>(p.tokens);
  const uint32_t t = r - u * static_cast<uint32_t>(p.tokens);
  const int64_t row = u * p.cache_stride + p.pos + t;
  const uint4 c = __ldcs(reinterpret_cast<const uint4 *>(codes + row * kHeadDim) + part);
  const float s = __ldcs(scales + row);
  const uint2 e0 = scaled_bf16x4(c.x, s), e1 = scaled_bf16x4(c.y, s);
  const uint2 e2 = scaled_bf16x4(c.z, s), e3 = scaled_bf16x4(c.w, s);
  uint4 *dst = reinterpret_cast<uint4 *>(rows + (u * p.dst_stride + t) * kHeadDim) + 2 * part;
  const uint4 lo = make_uint4(e0.x, e0.y, e1.x, e1.y), hi = make_uint4(e2.x, e2.y, e3.x, e3.y);
  if (p.dst32) {  // whole sectors
    st_global_v8(dst, lo, hi);
  } else {
    dst[0] = lo;
    dst[1] = hi;
  }
}

// Blocks for `rows` rows of each of two arrays: one row per eight lanes.
unsigned row_blocks(int64_t rows) { return static_cast<unsigned>((rows + kRowsPerBlock - 1) / kRowsPerBlock); }

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeParams &p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  return launch_pdl(quantize_rows_kernel, dim3(row_blocks(p.rows), 2), dim3(kCodeThreads), 0, stream, 0u, p);
}

cudaError_t launch_dequantize_rows(DequantizeParams p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  p.dst32 = ((reinterpret_cast<uintptr_t>(p.job[0].dst) | reinterpret_cast<uintptr_t>(p.job[1].dst)) & 31u) == 0;
  return launch_pdl(dequantize_rows_kernel, dim3(row_blocks(p.rows), 2), dim3(kCodeThreads), 0, stream, 0u, p);
}

}  // namespace embla
