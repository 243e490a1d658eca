// Window-layer decode of sequences at positions of their own ("The Architecture of Embla 1",
// "Three kinds of attention", Sliding window): softmax of tau q . k over the keys in a ring, then the
// weighted sum of their values.  Query and keys were rotated when they were written, and a softmax does
// not ask for the order of its keys: the valid ones are the ring's rows 0 .. min(pos + 1, window) - 1.
//
// Two kernels: where the units' rows fit the SMs at once, 128 to a CTA, each CTA takes its share in one
// step (window_step_kernel); else warps go through longer shares by themselves (window_stream_kernel).
// Either way a cluster of CTAs may share a unit: each finishes a share of its outputs, and every one
// writes its part of them, its maxima and its sums into the others' shared memory (writes do not wait;
// reading each other's took a third of the kernel's time).  P is fp32 in three bf16 parts (hi + mid +
// lo, all 24 bits), because the output is fp32.
//
// 96 sequences of 2 KV heads over rings of 1,024 keys (84 MB): 18.7 to 20.6 us (boards differ), 4.5 to 4.1 TB/s; of
// 4 heads (200 MB) 33.2 us, 6.0 TB/s, 0.89 of a copy's rate: the first microseconds, until rows arrive,
// and the merge do not shrink with the rings.  96 of 4 over rings of 128 (26 MB) 5.2 us; 8 of 4, 2.9 us, the launch and a trip to
// memory (3.0 where the rows are asked for after the position).
#include <cooperative_groups.h>

#include "ptx_blocks.cuh"
#include "ragged.h"

namespace cg = cooperative_groups;

namespace embla {
namespace {

constexpr int kRwWarps = 8;
constexpr int kRwThreads = kRwWarps * 32;
constexpr int kRwRows = 128;  // ring rows per CTA, 16 to a warp
constexpr int kRwRowBytes = kHeadDim * 2;
constexpr int kRwBuffer = kRwRows * kRwRowBytes;  // 32 KB of K rows, as much of V

struct RwShared {
  // parts of P, [part][head][row], padded so that heads start in different banks (those past G are zeros)
  uint16_t p[3][8][kRwRows + 8];
  float wm[kRwWarps][8];  // each warp's maximum per head
  float wl[kRwWarps][8];  // and sum
  float l[8];             // the CTA's
};

// What a CTA of a cluster is sent, over its K rows once it is done with them: every CTA's maxima and
// sums, and their sums of the outputs that this one finishes.
template <int G, int CL>
struct RwReceived {
  float m[CL][8], l[CL][8];
  float o[CL][G * kHeadDim / CL];
};

// An output that came out infinite or NaN though its sum of weights did not: a value is, or the products' sum
// passed the largest float before it was divided.  P's three parts make NaN of an infinite value (its second
// part may be zero or negative), so the output is computed once more.  (Nothing else pays for it: rings without
// such values take what they took.  One infinite value to a ring: 8 sequences of 4 KV heads 69 us instead of 2.9 over
// 128 keys, 141 instead of 6.5 over 1,024; 96 of 2 over 1,024 536 instead of 16.)
__device__ __forceinline__ bool is_broken(float y, float l) { return !(fabsf(y) <= 3.402823466e38f) && l == l; }

// Dim `dim` of a head (each lane's own) over the first `nv` rows of its unit's ring, from memory, by one warp: a key
// weighs nothing only where its score is minus infinity, weights are divided before the sum, and an infinite or NaN
// value enters as it is.
__device__ __noinline__ float output_again(const uint16_t *q, const uint8_t *K, const uint8_t *V, int nv, float tau2,
                                           int dim) {
  const int lane = threadIdx.x & 31;
  auto score = [&](int j) {
    if (j >= nv) return -INFINITY;
    const uint4 *k = reinterpret_cast<const uint4 *>(K + static_cast<int64_t>(j) * kRwRowBytes);
    const uint4 *x = reinterpret_cast<const uint4 *>(q);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int c = 0; c < kRwRowBytes / 16; ++c) {
      const uint4 a = k[c], b = x[c];
      s[0] = fmaf(bf16lo(a.x), bf16lo(b.x), fmaf(bf16hi(a.x), bf16hi(b.x), s[0]));
      s[1] = fmaf(bf16lo(a.y), bf16lo(b.y), fmaf(bf16hi(a.y), bf16hi(b.y), s[1]));
      s[2] = fmaf(bf16lo(a.z), bf16lo(b.z), fmaf(bf16hi(a.z), bf16hi(b.z), s[2]));
      s[3] = fmaf(bf16lo(a.w), bf16lo(b.w), fmaf(bf16hi(a.w), bf16hi(b.w), s[3]));
    }
    return tau2 * ((s[0] + s[1]) + (s[2] + s[3]));
  };
  float m = -INFINITY, l = 0.0f;
  auto join = [&](float m2, float l2) {
    const float mn = fmaxf(m, m2);
    l = l * (m == mn ? 1.0f : exp2f(m - mn)) + l2 * (m2 == mn ? 1.0f : exp2f(m2 - mn));
    m = mn;
  };
#pragma unroll 1
  for (int j = lane; j < nv; j += 32) {
    const float z = score(j);
    if (z != -INFINITY) join(z, 1.0f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
  if (l == 0.0f) return 0.0f;
  float y = 0.0f;
#pragma unroll 1
  for (int j0 = 0; j0 < nv; j0 += 32) {
    const float z = score(j0 + lane);
    const float mine = z == -INFINITY ? -1.0f : exp2f(z - m) / l;
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 16) {
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = reinterpret_cast<const uint16_t *>(V + static_cast<int64_t>(min(j0 + i0 + i, nv - 1)) * kRwRowBytes)[dim];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = __shfl_sync(0xffffffffu, mine, i0 + i), v = __uint_as_float(x[i] << 16);
        if (w != -1.0f) y = (x[i] & 0x7F80u) == 0x7F80u ? y + v : fmaf(w, v, y);
      }
    }
  }
  return y;
}

// This CTA's share of a unit's outputs (nv keys) from what every CTA of the cluster sent.
template <int G, int CL>
__device__ __forceinline__ void finish_outputs(const RwReceived<G, CL> &in, int rank, int64_t u, int nv,
                                               const RaggedWindowParams &p, int threads) {
  constexpr int per = G * kHeadDim / CL;
  static_assert(per % 32 == 0, "a warp's outputs are one head's");
  for (int li = threadIdx.x; li < per; li += threads) {
    const int at = rank * per + li, h = at / kHeadDim;
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < CL; ++c) M = fmaxf(M, in.m[c][h]);
    float L = 0.0f, A = 0.0f;
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      // (a CTA without keys has nothing to add, which its sum tells: NaN scores leave the maximum at minus infinity)
      if (in.l[c][h] != 0.0f) {
        const float f = exp2f(in.m[c][h] - M);
        L = fmaf(in.l[c][h], f, L);
        A = fmaf(in.o[c][li], f, A);
      }
    }
    float y = L > 0.0f || L != L ? A / L : 0.0f;
    if (__any_sync(0xffffffffu, is_broken(y, L))) {
      const int64_t ring = u * p.window * kRwRowBytes;
      const float z = output_again(p.q + (u * G + h) * kHeadDim, p.K + ring, p.V + ring, nv, p.tau2, at % kHeadDim);
      if (is_broken(y, L)) y = z;
    }
    p.out[u * G * kHeadDim + at] = y;
  }
}

// byte offset of 16-byte piece c of staged row r: eight rows of an ldmatrix read eight bank groups
__device__ __forceinline__ uint32_t rw_piece(int r, int c) {
  return static_cast<uint32_t>(r * kRwRowBytes + ((c ^ (r & 7)) << 4));
}

// ----------------------------------------------------------------------------- one step
//
// Eight warps copy 16 rows each, all of them in flight at once, and compute S = Q K^T of them as m16n8k16
// MMAs (M: the G query heads) as soon as the K rows are there; the maxima are exchanged and P goes to shared
// memory; each warp then computes 16 of the 128 output dims over all the rows, O^T = V^T P^T, so no
// warp's sums have to be added to another's.  Three CTAs fit an SM, so that one's arithmetic has the
// others' copies beside it.
//
// AHEAD: the CTA asks for every ring row that could be its own before it knows the position, which saves a
// trip to memory and reads up to 64 KB of rows that hold nothing yet.
template <int G, int CL, bool AHEAD>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kRwThreads, 3)
    window_step_kernel(const RaggedWindowParams p) {
  pdl_wait_primary();  // the query, the rings and the positions are complete
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];  // K rows, V rows, RwShared
  RwShared &sh = *reinterpret_cast<RwShared *>(smem + 2 * kRwBuffer);
  const int rank = CL > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int64_t u = blockIdx.x / CL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int last = p.pos[static_cast<uint32_t>(u) / static_cast<uint32_t>(p.Hkv)];
  // This warp's rows of the CTA's `count` from row `first` on: an instruction moves two whole ones; rows past
  // them are zeros (they read nothing, from an address inside the ring).
  const int wrow = warp * 16, piece = lane & 15;
  auto copy = [&](const uint8_t *ring, uint8_t *to, int first, int count) {
    const uint8_t *from = ring + u * p.window * kRwRowBytes;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = wrow + 2 * k + (lane >> 4);
      const bool live = r < count;
      cp_async16_zfill(to + rw_piece(r, piece),
                       from + (live ? static_cast<int64_t>(first + r) * kRwRowBytes : 0) + piece * 16, live ? 16u : 0u);
    }
    cp_async_commit();
  };
  int r0 = rank * kRwRows;
  if constexpr (AHEAD) {
    copy(p.K, smem, r0, p.window - r0);
    copy(p.V, smem + kRwBuffer, r0, p.window - r0);
  }
  const int nv = last < 0 ? 0 : (last >= p.window ? p.window : last + 1);  // valid rows of the ring
  const int share = AHEAD ? kRwRows : (nv + CL - 1) / CL;
  r0 = min(nv, rank * share);
  const int rows = min(nv, r0 + share) - r0;  // of this CTA
  if constexpr (!AHEAD) {
    copy(p.K, smem, r0, rows);
    copy(p.V, smem + kRwBuffer, r0, rows);
  }
  // query as the A operand of S: row g (head g), dims 16ks + 2t, +1 and +8, +9
  uint32_t qa0[8], qa2[8];
  {
    const uint32_t *qrow = reinterpret_cast<const uint32_t *>(p.q + (u * G + (g < G ? g : 0)) * kHeadDim);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qa0[ks] = g < G ? qrow[8 * ks + t] : 0u;
      qa2[ks] = g < G ? qrow[8 * ks + 4 + t] : 0u;
    }
  }
  cp_async_wait<1>();  // the K rows
  __syncwarp();

  // S of the warp's rows, eight to a tile: head g, rows 2t and 2t + 1 of each
  const int mat = lane >> 3, mr = lane & 7;
  float z[4], mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int row = wrow + 8 * j;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t bk[4];
      ldmatrix_x4(bk, smem_u32(smem) + rw_piece(row + mr, 4 * kk + mat));
      mma_16816_bf16(s, qa0[2 * kk], 0u, qa2[2 * kk], 0u, bk[0], bk[1]);
      mma_16816_bf16(s, qa0[2 * kk + 1], 0u, qa2[2 * kk + 1], 0u, bk[2], bk[3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) z[2 * j + i] = row + 2 * t + i < rows ? p.tau2 * s[i] : -INFINITY;
    mx = fmaxf(mx, fmaxf(z[2 * j], z[2 * j + 1]));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if (t == 0) sh.wm[warp][g] = mx;
  __syncthreads();
  if constexpr (CL > 1) cluster_arrive();  // this CTA's K rows are read: the others may write over them
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kRwWarps; ++w) m = fmaxf(m, sh.wm[w][g]);
  float l = 0.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float a = z[2 * j] == -INFINITY ? 0.0f : exp2f(z[2 * j] - m);
    float b = z[2 * j + 1] == -INFINITY ? 0.0f : exp2f(z[2 * j + 1] - m);
    l += a + b;
    uint32_t *to = reinterpret_cast<uint32_t *>(&sh.p[0][g][wrow + 8 * j + 2 * t]);
    constexpr int kPart = 8 * (kRwRows + 8) / 2;  // words from one part to the next
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const uint32_t h = g < G ? pack_bf16x2(a, b) : 0u;  // (the operand's heads past G are zeros)
      to[part * kPart] = h;
      a -= bf16lo(h);
      b -= bf16hi(h);
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) sh.wl[warp][g] = l;
  cp_async_wait<0>();  // the V rows
  if constexpr (AHEAD) {
    // rows that hold nothing yet may hold anything: a weight of zero needs a value
    if (rows < wrow + 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = wrow + 2 * k + (lane >> 4);
        if (r >= rows) *reinterpret_cast<uint4 *>(smem + kRwBuffer + rw_piece(r, piece)) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __syncthreads();  // everyone's, P and the sums

  // O^T of dims 16 warp .. + 15: A = V^T (16 dims x 16 rows per step), B = P^T
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // dims g (o[0], o[1]) and g + 8, heads 2t and 2t + 1
#pragma unroll
  for (int k = 0; k < kRwRows / 16; ++k) {
    if (16 * k >= rows) break;
    uint32_t av[4];
    ldmatrix_x4_trans(av, smem_u32(smem + kRwBuffer) + rw_piece(16 * k + (mat >> 1) * 8 + mr, 2 * warp + (mat & 1)));
#pragma unroll
    for (int part = 2; part >= 0; --part) {  // the small parts first
      const uint32_t *b = reinterpret_cast<const uint32_t *>(&sh.p[part][g][16 * k + 2 * t]);
      mma_16816_bf16(o, av[0], av[1], av[2], av[3], b[0], b[4]);
    }
  }
  if constexpr (CL == 1) {
    if (warp == 0 && lane < 8) {
      float ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kRwWarps; ++w) ls += sh.wl[w][lane];
      sh.l[lane] = ls;
    }
    __syncthreads();
    bool broken = false;
    float *out = p.out + u * G * kHeadDim + 16 * warp;
    if (2 * t < G) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = 2 * t + (i & 1);
        const float lh = sh.l[h], y = lh > 0.0f || lh != lh ? o[i] / lh : 0.0f;
        out[h * kHeadDim + g + 8 * (i >> 1)] = y;
        broken |= is_broken(y, lh);
      }
    }
    if (__any_sync(0xffffffffu, broken)) {
      __syncwarp();  // the warp's outputs are written
      const int64_t ring = u * p.window * kRwRowBytes;
      const int d = lane & 15;
#pragma unroll 1
      for (int h = 0; h < G; ++h) {
        const bool mine = is_broken(out[h * kHeadDim + d], sh.l[h]);
        if (!__any_sync(0xffffffffu, mine)) continue;
        const float y = output_again(p.q + (u * G + h) * kHeadDim, p.K + ring, p.V + ring, nv, p.tau2, 16 * warp + d);
        if (mine && lane < 16) out[h * kHeadDim + d] = y;
      }
    }
  } else {
    constexpr int per = G * kHeadDim / CL;  // outputs that a CTA finishes: parts of one head, or whole heads
    cg::cluster_group cluster = cg::this_cluster();
    using Received = RwReceived<G, CL>;
    Received *mine = reinterpret_cast<Received *>(smem);
    static_assert(sizeof(Received) <= kRwBuffer, "over the K rows");
    cluster_wait();  // every CTA of the cluster has read its K rows
    if (2 * t < G) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (2 * t + (i & 1)) * kHeadDim + 16 * warp + g + 8 * (i >> 1);
        cluster.map_shared_rank(mine, at / per)->o[rank][at % per] = o[i];
      }
    }
    // maximum and sum of head g (the same in every warp), from warp w to CTA w
    if (warp < CL && t == 0) {
      float ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kRwWarps; ++w) ls += sh.wl[w][g];
      Received *to = cluster.map_shared_rank(mine, warp);
      to->m[rank][g] = m;
      to->l[rank][g] = ls;
    }
    cluster_arrive();
    cluster_wait();  // everything is here, and nobody reads or writes another's shared memory any more
    finish_outputs<G, CL>(*mine, rank, u, nv, p, kRwThreads);
  }
}

// ----------------------------------------------------------------------------- many units
//
// Where the units' steps do not fit the SMs at once, warps go through the rows by themselves: each takes
// every so many blocks of 16 rows of its unit, one block on its way while it works on another, with a
// running maximum, sum and O (all 128 dims of every head) in registers.  S's accumulators are the operand
// of the next product as they lie, so P stays in registers too.  Warps and CTAs merge at the end.
constexpr int kWsWarps = 4;
constexpr int kWsThreads = kWsWarps * 32;
constexpr int kWsRows = 16;
constexpr int kWsBlock = 2 * kWsRows * kRwRowBytes;  // K and V rows of a block: 8 KB
constexpr int kWsStages = 2;

template <int G>
struct WsMerge {  // over the rows
  float m[kWsWarps][8], l[kWsWarps][8];
  float o[kWsWarps][G][kHeadDim];
};

template <int G, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kWsThreads, 3)
    window_stream_kernel(const RaggedWindowParams p) {
  if constexpr (CL > 1) cluster_arrive();  // (waited for before anything is sent: every CTA has started)
  pdl_wait_primary();  // the query, the rings and the positions are complete
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];  // rows, then WsMerge; behind them what is received
  const int rank = CL > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int64_t u = blockIdx.x / CL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int last = p.pos[static_cast<uint32_t>(u) / static_cast<uint32_t>(p.Hkv)];
  const int nv = last < 0 ? 0 : (last >= p.window ? p.window : last + 1);  // valid rows of the ring
  const int blocks = (nv + kWsRows - 1) / kWsRows;
  uint8_t *rows = smem + warp * kWsStages * kWsBlock;
  // Block n's rows into a stage: an instruction moves two whole rows; rows past the valid ones are zeros
  // (they read nothing, from an address inside the ring).  A group ends with each call.
  auto copy = [&](int n, int stage) {
    if (n < blocks) {
      uint8_t *to = rows + stage * kWsBlock;
      const int piece = lane & 15;
      const int64_t unit = u * p.window * kRwRowBytes + piece * 16;
#pragma unroll
      for (int k = 0; k < kWsRows / 2; ++k) {
        const int r = 2 * k + (lane >> 4);
        const bool live = n * kWsRows + r < nv;
        const int64_t off = unit + (live ? static_cast<int64_t>(n * kWsRows + r) * kRwRowBytes : 0);
        cp_async16_zfill(to + rw_piece(r, piece), p.K + off, live ? 16u : 0u);
        cp_async16_zfill(to + kWsRows * kRwRowBytes + rw_piece(r, piece), p.V + off, live ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  constexpr int kStep = CL * kWsWarps;
  const int first = rank * kWsWarps + warp;
  copy(first, 0);
  copy(first + kStep, 1);
  // query as the A operand of S: row g (head g), dims 16ks + 2t, +1 and +8, +9
  uint32_t qa0[8], qa2[8];
  {
    const uint32_t *qrow = reinterpret_cast<const uint32_t *>(p.q + (u * G + (g < G ? g : 0)) * kHeadDim);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qa0[ks] = g < G ? qrow[8 * ks + t] : 0u;
      qa2[ks] = g < G ? qrow[8 * ks + 4 + t] : 0u;
    }
  }
  float m = -INFINITY, l = 0.0f;  // head g: running maximum (base 2) and sum
  float o[8][4];                  // O^T tile i: dims 16i + g (+8), heads 2t and 2t + 1
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  const int mat = lane >> 3, row = (mat >> 1) * 8 + (lane & 7);
  int stage = 0;
  for (int n = first; n < blocks; n += kStep, stage ^= 1) {
    cp_async_wait<1>();
    __syncwarp();
    const uint32_t sK = smem_u32(rows + stage * kWsBlock), sV = sK + kWsRows * kRwRowBytes;
    float s0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t bk[4];
      ldmatrix_x4(bk, sK + rw_piece(row, 2 * ks + (mat & 1)));
      mma_16816_bf16(s0, qa0[ks], 0u, qa2[ks], 0u, bk[0], bk[1]);
      mma_16816_bf16(s1, qa0[ks], 0u, qa2[ks], 0u, bk[2], bk[3]);
    }
    // head g, rows 2t, 2t + 1 (s0) and 8 + 2t, 9 + 2t (s1)
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[i] = n * kWsRows + 8 * (i >> 1) + 2 * t + (i & 1) < nv ? p.tau2 * (i < 2 ? s0[i] : s1[i - 2]) : -INFINITY;
    float mn = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
    mn = fmaxf(m, fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2)));
    const float sc = m == mn ? 1.0f : exp2f(m - mn);
    m = mn;
    float ps = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = z[i] == -INFINITY ? 0.0f : exp2f(z[i] - m);
      ps += z[i];
    }
    ps += __shfl_xor_sync(0xffffffffu, ps, 1);
    ps += __shfl_xor_sync(0xffffffffu, ps, 2);
    l = fmaf(l, sc, ps);
    uint32_t part[3][2];  // P in three bf16 parts
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        part[k][i] = pack_bf16x2(z[2 * i], z[2 * i + 1]);
        z[2 * i] -= bf16lo(part[k][i]);
        z[2 * i + 1] -= bf16hi(part[k][i]);
      }
    const float sca = __shfl_sync(0xffffffffu, sc, 8 * t), scb = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t av[4];
      ldmatrix_x4_trans(av, sV + rw_piece(row, 2 * i + (mat & 1)));
      // (the tensor cores cut off what does not fit their sum, so a block has one of its own)
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 2; k >= 0; --k) mma_16816_bf16(d, av[0], av[1], av[2], av[3], part[k][0], part[k][1]);
      o[i][0] = fmaf(o[i][0], sca, d[0]);
      o[i][1] = fmaf(o[i][1], scb, d[1]);
      o[i][2] = fmaf(o[i][2], sca, d[2]);
      o[i][3] = fmaf(o[i][3], scb, d[3]);
    }
    __syncwarp();  // the stage is read before the next copies land in it
    copy(n + 2 * kStep, stage);
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its rows
  WsMerge<G> &mg = *reinterpret_cast<WsMerge<G> *>(smem);
  static_assert(sizeof(WsMerge<G>) <= kWsWarps * kWsStages * kWsBlock, "over the rows");
  if (t == 0) {
    mg.m[warp][g] = m;
    mg.l[warp][g] = l;
  }
  if (2 * t < G) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) mg.o[warp][2 * t + (e & 1)][16 * i + g + 8 * (e >> 1)] = o[i][e];
  }
  __syncthreads();
  using Received = RwReceived<G, CL>;
  Received *mine = reinterpret_cast<Received *>(smem + kWsWarps * kWsStages * kWsBlock);
  constexpr int per = G * kHeadDim / CL;  // outputs that a CTA finishes: parts of one head, or whole heads
  if constexpr (CL > 1) cluster_wait();
#pragma unroll
  for (int h = 0; h < G; ++h) {
    // thread: dim threadIdx.x of head h
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWsWarps; ++w) M = fmaxf(M, mg.m[w][h]);
    float L = 0.0f, A = 0.0f;
#pragma unroll
    for (int w = 0; w < kWsWarps; ++w) {
      // (a warp without rows has nothing to add, which its sum tells: as in finish_outputs)
      if (mg.l[w][h] != 0.0f) {
        const float f = exp2f(mg.m[w][h] - M);
        L = fmaf(mg.l[w][h], f, L);
        A = fmaf(mg.o[w][h][threadIdx.x], f, A);
      }
    }
    if constexpr (CL == 1) {
      float y = L > 0.0f || L != L ? A / L : 0.0f;
      if (__any_sync(0xffffffffu, is_broken(y, L))) {
        const int64_t ring = u * p.window * kRwRowBytes;
        const float z = output_again(p.q + (u * G + h) * kHeadDim, p.K + ring, p.V + ring, nv, p.tau2, threadIdx.x);
        if (is_broken(y, L)) y = z;
      }
      p.out[(u * G + h) * kHeadDim + threadIdx.x] = y;
    } else {
      const int at = h * kHeadDim + threadIdx.x;
      Received *to = cg::this_cluster().map_shared_rank(mine, at / per);
      to->o[rank][at % per] = A;
      if (at % per == 0 || (at & (kHeadDim - 1)) == 0) {
        // the first of this CTA's, or of a head: maximum and sum beside it
        to->m[rank][h] = M;
        to->l[rank][h] = L;
      }
    }
  }
  if constexpr (CL > 1) {
    cluster_arrive();
    cluster_wait();  // everything is here, and nobody writes another's shared memory any more
    finish_outputs<G, CL>(*mine, rank, u, nv, p, kWsThreads);
  }
}

template <int G, int CL, bool AHEAD>
cudaError_t launch_step(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  constexpr int bytes = 2 * kRwBuffer + static_cast<int>(sizeof(RwShared));
  static_assert(3 * (bytes + 1024) <= 228 * 1024, "three CTAs per SM");
  constexpr auto kernel = window_step_kernel<G, CL, AHEAD>;
  const cudaError_t e = allow_smem_once<kernel>(dev, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(units * CL)), dim3(kRwThreads), bytes, stream, 0u, p);
}

// Rows are asked for ahead where each CTA has an SM to itself: what that reads in vain is then at most 10 MB
// (8 sequences of 4 KV heads 2.85 us against 3.05, rings of 1,024 of 2 5.2 and 5.5; 32 with 7 rows each 2.75
// and 2.62).
template <int G, int CL>
cudaError_t launch_rw(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  return units * CL <= dev.sms ? launch_step<G, CL, true>(units, p, dev, stream)
                               : launch_step<G, CL, false>(units, p, dev, stream);
}

template <int G, int CL>
cudaError_t launch_ws(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  constexpr int bytes = kWsWarps * kWsStages * kWsBlock + static_cast<int>(sizeof(RwReceived<G, CL>));
  static_assert(3 * (bytes + 1024) <= 228 * 1024, "three CTAs per SM");
  constexpr auto kernel = window_stream_kernel<G, CL>;
  const cudaError_t e = allow_smem_once<kernel>(dev, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(units * CL)), dim3(kWsThreads), bytes, stream, 0u, p);
}

// One step of up to 128 rows per CTA where all CTAs are resident at once, or a ring has no more; else as
// many CTAs of four warps to a unit as are resident at once.  (64 sequences of 4 KV heads with rings of 512
// keys: 19.0 us in steps, 14.6 streamed; 96 of 2 with 1,024: 27.9 and 18.7; 8 of 4 with 1,024, which fit: 6.3.)
template <int G>
cudaError_t launch_rw_g(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  const int64_t resident = 3ll * dev.sms;
  int cl = 1;
  while (cl * 128 < p.window) cl *= 2;
  if (cl == 1) return launch_rw<G, 1>(units, p, dev, stream);
  if (units * cl <= resident) {
    if (cl == 2) return launch_rw<G, 2>(units, p, dev, stream);
    if (cl == 4) return launch_rw<G, 4>(units, p, dev, stream);
    return launch_rw<G, 8>(units, p, dev, stream);
  }
  while (cl > 1 && units * cl > resident) cl /= 2;
  if (cl == 1) return launch_ws<G, 1>(units, p, dev, stream);
  if (cl == 2) return launch_ws<G, 2>(units, p, dev, stream);
  return launch_ws<G, 4>(units, p, dev, stream);
}

}  // namespace

cudaError_t launch_window_decode_ragged(int G, int64_t units, const RaggedWindowParams &p,
                                        const LaunchDevice &dev, cudaStream_t stream) {
  if (units == 0) return cudaSuccess;
  if (G == 4) return launch_rw_g<4>(units, p, dev, stream);
  if (G == 8) return launch_rw_g<8>(units, p, dev, stream);
  return cudaErrorInvalidValue;
}

}  // namespace embla
