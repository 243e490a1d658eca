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
// fraction with no error but F_i's own (p 2^-54 of a circle from the double it came from, 2^-33 at
// a position of 2^20), by one integer product and no 64-bit floats.  Its top 32 bits, as a signed part
// of half a circle, go to sincospif.
//
// A block takes a few tokens with all their heads.  Half a warp per token finds its sequence (16 ways at
// a time) and the block works out the tokens' 64 sines and cosines once, into shared memory; then
// eight lanes take a row, 32 bytes each, so that a warp moves 1 KB in one piece.  The first rows are
// requested before the angles are worked out.  Bound by HBM.
#include "ptx_blocks.cuh"
#include "ragged.h"

namespace embla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = kRopeThreads / 8;  // rows that a block works on at a time
constexpr int kRopeMaxTokens = 16;           // per block: half a warp each

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

struct RopeToken {
  uint32_t pos;
  int32_t slot;  // ring row b * Hkv * window + position % window; -1: not among the newest; -2: no sequence
};

// 16 values of a row to fp32 (normed and scaled), turned, and back to bf16.  Lane l of eight holds dims
// 16 l .. 16 l + 15, pairs 8 l .. 8 l + 7: cs[k], k < 2: cosines of pairs 8 l + 4 k .. + 3, k - 2: sines.
template <bool NORM>
__device__ __forceinline__ void turn_row(uint4 &x0, uint4 &x1, const float4 (&cs)[4], const float4 *gain, float eps,
                                         uint32_t mine) {
  const uint32_t r[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float rs = 1.0f;
  if constexpr (NORM) {
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) sq_acc_bf16x2(r[i], a[2 * (i & 1)], a[2 * (i & 1) + 1]);
    float ss = (a[0] + a[1]) + (a[2] + a[3]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(mine, ss, o);
    rs = 1.0f / sqrtf(ss * (1.0f / kHeadDim) + eps);
  }
  const float c[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
  const float s[8] = {cs[2].x, cs[2].y, cs[2].z, cs[2].w, cs[3].x, cs[3].y, cs[3].z, cs[3].w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float e = bf16lo(r[i]), f = bf16hi(r[i]);
    if constexpr (NORM) {
      // gains lie as the cosines do: pieces of four dims, lane by lane
      const float4 g = gain[(i >> 1) * 8];
      mul_f32x2(e, f, e, f, i & 1 ? g.z : g.x, i & 1 ? g.w : g.y);
      mul_f32x2(e, f, e, f, rs, rs);
    }
    // (e, f) c + (-f, e) s
    float u, v;
    mul_f32x2(u, v, -f, e, s[i], s[i]);
    fma_f32x2(u, v, e, f, c[i], c[i], u, v);
    y[i] = pack_bf16x2(u, v);
  }
  x0 = make_uint4(y[0], y[1], y[2], y[3]);
  x1 = make_uint4(y[4], y[5], y[6], y[7]);
}

template <bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ RopeToken tok[kRopeMaxTokens];
  __shared__ float4 angles[kRopeMaxTokens][4][8];  // [token][cos, cos, sin, sin][lane]
  __shared__ float4 gains[2][4][8];                // of queries and keys, pieces of four dims by lane
  pdl_wait_primary();  // the rows are written; whoever read the old outputs and rings is done
  pdl_launch_dependents();
  const int part = threadIdx.x % 8;
  const uint32_t mine = 0xFFu << (threadIdx.x & 24);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.block_tokens;
  const int ntok = static_cast<int>(p.seqs.tokens - t0 < p.block_tokens ? p.seqs.tokens - t0 : p.block_tokens);
  const int per = p.Hq + p.Hkv + (p.k_win ? p.Hkv : 0);  // rows of a token: queries, keys, values for the ring
  const int rows = ntok * per;

  // row r of the block: its token, head and kind, and its 32 bytes of this lane
  auto locate = [&](int r, int &t, int &h) {
    t = r / per;
    h = r - t * per;
  };
  auto request = [&](int r, uint4 &a, uint4 &b) {
    int t, h;
    locate(r, t, h);
    const uint16_t *src = h < p.Hq            ? p.q.base + (t0 + t) * p.q.stride + h * kHeadDim
                          : h < p.Hq + p.Hkv ? p.k.base + (t0 + t) * p.k.stride + (h - p.Hq) * kHeadDim
                                             : p.v.base + (t0 + t) * p.v.stride + (h - p.Hq - p.Hkv) * kHeadDim;
    const uint4 *at = reinterpret_cast<const uint4 *>(src) + 2 * part;
    a = __ldcs(at);
    b = __ldcs(at + 1);
  };
  // the first two rows of these lanes (values are asked for when it is known that they are needed)
  uint4 x[2][2];
  const int r0 = threadIdx.x / 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + i * kRopeRows;
    x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && r % per < p.Hq + p.Hkv) request(r, x[i][0], x[i][1]);
  }

  {
    const int i = threadIdx.x / 16, sl = threadIdx.x % 16;
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
    if (i < ntok) {
      const int64_t t = t0 + i;
      const int b = sequence_of(p.seqs, t, sl, half);
      RopeToken k = {0u, -2};
      if (b < p.seqs.batch && t >= p.seqs.cu[b]) {
        k.pos = (p.pos0 ? static_cast<uint32_t>(p.pos0[b]) : 0u) + static_cast<uint32_t>(t - p.seqs.cu[b]);
        k.slot = -1;
        if (p.k_win && t >= static_cast<int64_t>(p.seqs.cu[b + 1]) - p.window)
          k.slot = b * p.Hkv * p.window + static_cast<int32_t>(k.pos % static_cast<uint32_t>(p.window));
      }
      if (sl == 0) tok[i] = k;
      // this token's 64 angles, four to a lane
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pair = 4 * sl + e;  // lane pair / 8, value pair % 8
        const int32_t half_turns = static_cast<int32_t>((k.pos * p.turn[pair]) >> 32);
        float c, s;
        sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
        reinterpret_cast<float *>(&angles[i][(pair & 4) >> 2][pair >> 3])[pair & 3] = c;
        reinterpret_cast<float *>(&angles[i][2 + ((pair & 4) >> 2)][pair >> 3])[pair & 3] = s;
      }
    }
    if (NORM && threadIdx.x < 64) {
      const int which = threadIdx.x >> 5, d = threadIdx.x & 31;  // dims 4 d .. 4 d + 3
      const float *g = which ? p.k_gain : p.q_gain;
      gains[which][d & 3][d >> 2] =
          g ? *reinterpret_cast<const float4 *>(g + 4 * d) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    }
  }
  __syncthreads();

  for (int r = r0; r < rows; r += 2 * kRopeRows) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ri = r + i * kRopeRows;
      if (ri >= rows) break;
      int t, h;
      locate(ri, t, h);
      const RopeToken k = tok[t];
      uint4 a = x[i][0], b = x[i][1];
      // the row after next of these lanes
      const int rn = ri + 2 * kRopeRows;
      if (rn < rows && rn % per < p.Hq + p.Hkv) request(rn, x[i][0], x[i][1]);
      if (k.slot == -2) continue;  // behind the last sequence
      const bool value = h >= p.Hq + p.Hkv;
      uint16_t *to = nullptr;
      if (value) {
        if (k.slot < 0) continue;
        request(ri, a, b);
      } else {
        float4 cs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = angles[t][e][part];
        turn_row<NORM>(a, b, cs, &gains[h < p.Hq ? 0 : 1][0][part], p.eps, mine);
        if (h < p.Hq)
          to = p.q_out + ((t0 + t) * p.Hq + h) * kHeadDim;
        else if (p.k_out)
          to = p.k_out + ((t0 + t) * p.Hkv + h - p.Hq) * kHeadDim;
      }
      if (to) {
        uint4 *at = reinterpret_cast<uint4 *>(to) + 2 * part;
        if (p.out32) {  // whole sectors
          st_global_v8(at, a, b);
        } else {
          at[0] = a;
          at[1] = b;
        }
      }
      if (h >= p.Hq && k.slot >= 0) {
        uint16_t *ring = value ? p.v_win : p.k_win;
        const int64_t head = value ? h - p.Hq - p.Hkv : h - p.Hq;
        uint4 *at = reinterpret_cast<uint4 *>(ring + (k.slot + head * p.window) * kHeadDim) + 2 * part;
        at[0] = a;
        at[1] = b;
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_qkv(RopeParams p, int sm_count, cudaStream_t stream) {
  if (p.seqs.tokens == 0) return cudaSuccess;
  // As many tokens per block as leave two blocks to an SM, a power of two: the search and the angles are
  // then shared by more rows.
  p.block_tokens = 1;
  while (p.block_tokens < kRopeMaxTokens && p.seqs.tokens >= 4ll * sm_count * p.block_tokens) p.block_tokens *= 2;
  p.out32 = ((reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out)) & 31u) == 0;
  const int64_t blocks = (p.seqs.tokens + p.block_tokens - 1) / p.block_tokens;
  return launch_pdl(p.norm ? rope_kernel<true> : rope_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kRopeThreads), 0, stream, 0u, p);
}

}  // namespace embla
