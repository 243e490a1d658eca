// Queries and keys of packed tokens normed per head and rotated at their positions in one pass,
// the newest rows of every sequence written into its window rings ("The Architecture of Embla 1",
// "Three kinds of attention": the window layers are the positional ones, and a ring holds keys
// that were rotated when they were written).
//
//   y = x                                    or  x / sqrt(mean(x^2) + eps) * gain   (fp32)
//   (y_2i, y_2i+1) turned by p base^(-2i/D)                                         (fp32)
//   rounded once to bf16.
//
// The angle.  A pair turns by f_i = base^(-2i/D) / (2 pi) of a circle per position, and only the
// fraction of p f_i counts.  The host gives F_i = f_i 2^64 rounded to an integer: p F_i modulo 2^64 is that
// fraction with no error but F_i's own (p 2^-54 of a circle from the double it came from, 2^-34 at
// a position of 2^20), by one integer product and no 64-bit floats.  Its top 32 bits, as a signed part
// of half a circle, go to sincospif.
//
// Sixteen lanes take the G query heads and the key head of one KV group of one token, 16 bytes of
// each row per lane, so a lane works out its four angles once for G + 1 rows and has all of their
// loads in flight together; nothing waits on another lane but the norms' sums.  Bound by HBM: 4 x 32,768
// tokens of 16 + 4 heads, normed, in 209 us (6.4 TB/s, 0.95 of a copy's rate); a step of 8 tokens 2.3 us, the
// launch.  Blocks of tokens that shared their angles through shared memory took 242 us (a barrier and
// fewer loads in flight).  Small blocks start and leave sooner: 64 threads 209, 128 210, 256 214, 512 235 us.
// Each query is stored as it is done (all of them at the end: 210 to 217 us by how the stores are ordered).
// Rows whose squares leave the floats' range are not looked for: times a power of two first, in a branch
// that no other row takes, they cost every call with norms 1.5 to 6 % (213 to 222 us; 5,072 ragged tokens 11.2 to 11.7).
// Registers: 56 (36 warps to an SM) 204 us, but 2,000 tokens 6.6 against 5.9 and the step 2.6.
#include "ptx_blocks.cuh"
#include "ragged.h"

namespace embla {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeLanes = 16;  // lanes per (token, KV group)
constexpr int kRopePerBlock = kRopeThreads / kRopeLanes;

// How many sequences end at or before token t (cu[b + 1] <= t), found by the sixteen lanes of a
// half warp 16 ways at a time: the sequence that t lies in, or `batch` past the last one.
__device__ __forceinline__ int sequence_of(const PackedTokens &s, int64_t t, int sl, uint32_t half) {
  int lo = 0, hi = s.batch;  // the answer lies in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 15) / 16;
    const int at = lo + (sl + 1) * step;  // sequences lo .. at - 1 end by t if number at - 1 does
    const bool past = at <= hi && s.cu[at] <= t;
    const int n = __popc(__ballot_sync(half, past) & half);
    const int from = lo + n * step;
    hi = min(hi, from + step - 1);
    lo = from;
  }
  return lo;
}

template <int G, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, G == 4 ? 16 : 12) rope_kernel(const __grid_constant__ RopeParams p) {
  pdl_wait_primary();  // the rows are written; whoever read the old outputs and rings is done
  pdl_launch_dependents();
  const int sl = threadIdx.x % kRopeLanes;
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopePerBlock + threadIdx.x / kRopeLanes;
  const int64_t t = w / p.Hkv;
  const int g = static_cast<int>(w - t * p.Hkv);
  if (t >= p.seqs.tokens) return;  // (half warps leave whole)
  const int d = sl * 8;            // this lane's dims d .. d + 7: pairs 4 sl .. 4 sl + 3
  uint4 x[G + 1], v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int h = 0; h < G; ++h)
    x[h] = __ldcs(reinterpret_cast<const uint4 *>(p.q.base + t * p.q.stride + (g * G + h) * kHeadDim + d));
  x[G] = __ldcs(reinterpret_cast<const uint4 *>(p.k.base + t * p.k.stride + g * kHeadDim + d));
  const int b = sequence_of(p.seqs, t, sl, half);
  if (b >= p.seqs.batch) return;  // behind the last sequence
  const int64_t first = p.seqs.cu[b], end = p.seqs.cu[b + 1];
  if (t < first) return;
  const uint32_t pos = (p.pos0 ? static_cast<uint32_t>(p.pos0[b]) : 0u) + static_cast<uint32_t>(t - first);
  const bool ring = p.k_win != nullptr && t >= end - p.window;  // among the newest
  if (ring) v = __ldcs(reinterpret_cast<const uint4 *>(p.v.base + t * p.v.stride + g * kHeadDim + d));
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t half_turns = static_cast<int32_t>((pos * p.turn[4 * sl + i]) >> 32);
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s[i], &c[i]);
  }
  float rs[G + 1];
  if constexpr (NORM) {
#pragma unroll
    for (int h = 0; h <= G; ++h) {
      float a = 0.0f, e = 0.0f;
      sq_acc_bf16x2(x[h].x, a, e);
      sq_acc_bf16x2(x[h].y, a, e);
      sq_acc_bf16x2(x[h].z, a, e);
      sq_acc_bf16x2(x[h].w, a, e);
      rs[h] = a + e;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int h = 0; h <= G; ++h) rs[h] += __shfl_xor_sync(half, rs[h], o);
#pragma unroll
    for (int h = 0; h <= G; ++h) rs[h] = rsqrtf(rs[h] * (1.0f / kHeadDim) + p.eps);
  }
  float gain[8];
  uint16_t *to = p.q_out + (t * p.Hkv + g) * G * kHeadDim + d;
#pragma unroll
  for (int h = 0; h <= G; ++h) {
    if constexpr (NORM) {
      if (h == 0 || h == G) {  // the queries' gains, then the key's
        const float *from = h == 0 ? p.q_gain : p.k_gain;
        const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        const float4 g0 = from ? *reinterpret_cast<const float4 *>(from + d) : one;
        const float4 g1 = from ? *reinterpret_cast<const float4 *>(from + d + 4) : one;
        gain[0] = g0.x, gain[1] = g0.y, gain[2] = g0.z, gain[3] = g0.w;
        gain[4] = g1.x, gain[5] = g1.y, gain[6] = g1.z, gain[7] = g1.w;
      }
    }
    const uint32_t r[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float e = bf16lo(r[i]), f = bf16hi(r[i]);
      if constexpr (NORM) {
        mul_f32x2(e, f, e, f, gain[2 * i], gain[2 * i + 1]);
        mul_f32x2(e, f, e, f, rs[h], rs[h]);
      }
      // (e, f) c + (-f, e) s
      float u, v2;
      mul_f32x2(u, v2, -f, e, s[i], s[i]);
      fma_f32x2(u, v2, e, f, c[i], c[i], u, v2);
      y[i] = pack_bf16x2(u, v2);
    }
    x[h] = make_uint4(y[0], y[1], y[2], y[3]);
    if (h < G) *reinterpret_cast<uint4 *>(to + h * kHeadDim) = x[h];
  }
  if (ring) {
    const int64_t row = (static_cast<int64_t>(b) * p.Hkv + g) * p.window + pos % static_cast<uint32_t>(p.window);
    *reinterpret_cast<uint4 *>(p.k_win + row * kHeadDim + d) = x[G];
    *reinterpret_cast<uint4 *>(p.v_win + row * kHeadDim + d) = v;
  }
  if (p.k_out) *reinterpret_cast<uint4 *>(p.k_out + (t * p.Hkv + g) * kHeadDim + d) = x[G];
}

template <int G>
cudaError_t launch_rope_g(const RopeParams &p, cudaStream_t stream) {
  const int64_t blocks = (p.seqs.tokens * p.Hkv + kRopePerBlock - 1) / kRopePerBlock;
  return launch_pdl(p.norm ? rope_kernel<G, true> : rope_kernel<G, false>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kRopeThreads), 0, stream, 0u, p);
}

}  // namespace

cudaError_t launch_rope_qkv(int G, const RopeParams &p, cudaStream_t stream) {
  if (p.seqs.tokens == 0) return cudaSuccess;
  if (G == 4) return launch_rope_g<4>(p, stream);
  if (G == 8) return launch_rope_g<8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace embla
