// Window-layer decode of sequences at positions of their own ("The Architecture of Embla 1",
// "Three kinds of attention", Sliding window): softmax of tau q . k over the keys in a ring, then the
// weighted sum of their values.  Query and keys were rotated when they were written, and a softmax does
// not ask for the order of its keys: the valid ones are the ring's rows 0 .. min(pos + 1, window) - 1.
//
// A cluster of CTAs takes a (sequence, KV head) unit, an equal share of its valid rows to a CTA.  Where all
// units' shares of up to 128 rows fit the SMs at once, a CTA takes its share in one step; else it goes
// through a longer one in steps of 64 rows, the next 64 on their way meanwhile.  In a step
//   - eight warps take 8 or 16 rows each, copied by themselves, and compute S = Q K^T as m16n8k16 MMAs (M:
//     the G query heads);
//   - the rows' maximum per head is exchanged, and P = exp2(z - m) for the running maximum m written as
//     three bf16 parts (hi + mid + lo, all 24 bits: the output is fp32);
//   - each warp adds P V to its 16 of the 128 output dims over all the rows, O^T += V^T P^T, so no warp's
//     sums have to be added to another's.
// The CTAs of a unit each finish a share of its outputs: every one writes its part of them, its maxima
// and its sums into the others' shared memory, over K rows that are no longer needed (writes do not
// wait; reading each other's took a third of the kernel's time).  Three CTAs fit an SM, so that
// one's arithmetic has the others' copies beside it.
#include <cooperative_groups.h>

#include "ptx_blocks.cuh"
#include "ragged.h"

namespace cg = cooperative_groups;

namespace embla {
namespace {

constexpr int kRwWarps = 8;
constexpr int kRwThreads = kRwWarps * 32;
constexpr int kRwRowBytes = kHeadDim * 2;
constexpr int kRwBuffer = 128 * kRwRowBytes;  // 32 KB of K rows, as much of V

// ROWS: ring rows per step, 128 (one step) or 64 (the buffers hold two steps).
template <int ROWS>
struct RwShared {
  // parts of P, [part][head][row], padded so that heads start in different banks (those past G are zeros)
  uint16_t p[3][8][ROWS + 8];
  float wm[2][kRwWarps][8];  // each warp's maximum per head, of one step and the next
  float wl[kRwWarps][8];     // each warp's sum
  float l[8];                // the CTA's
};

// What a CTA of a cluster is sent, over its K rows once it is done with them: every CTA's maxima and
// sums, and their sums of the outputs that this one finishes.
template <int G, int CL>
struct RwReceived {
  float m[CL][8], l[CL][8];
  float o[CL][G * kHeadDim / CL];
};

// byte offset of 16-byte piece c of staged row r: eight rows of an ldmatrix read eight bank groups
__device__ __forceinline__ uint32_t rw_piece(int r, int c) {
  return static_cast<uint32_t>(r * kRwRowBytes + ((c ^ (r & 7)) << 4));
}

template <int G, int CL, int ROWS>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kRwThreads, 3)
    window_ragged_kernel(const RaggedWindowParams p) {
  constexpr bool kOnce = ROWS == 128;
  constexpr int kTiles = ROWS / 64;             // n8 tiles of a warp's rows
  constexpr int kStage = ROWS * kRwRowBytes;
  pdl_wait_primary();  // the query, the rings and the positions are complete
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];  // K rows, V rows, RwShared
  RwShared<ROWS> &sh = *reinterpret_cast<RwShared<ROWS> *>(smem + 2 * kRwBuffer);
  const int rank = CL > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int64_t u = blockIdx.x / CL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int last = p.pos[u / p.Hkv];
  const int nv = last < 0 ? 0 : (last >= p.window ? p.window : last + 1);  // valid rows of the ring
  const int share = (nv + CL - 1) / CL;
  const int r0 = min(nv, rank * share), rows = min(nv, r0 + share) - r0;  // of this CTA
  const int steps = kOnce ? min(rows, 1) : (rows + ROWS - 1) / ROWS;

  // Copies of step c's rows of this warp: an instruction moves two whole rows; rows past the share are
  // zeros (they read nothing, from an address inside the ring).  A group ends with each call.
  auto copy = [&](const uint8_t *ring, int c, uint8_t *to) {
    if (c < steps) {
      const uint8_t *from = ring + u * p.window * kRwRowBytes;
      const int piece = lane & 15;
#pragma unroll
      for (int k = 0; k < 4 * kTiles; ++k) {
        const int r = warp * 8 * kTiles + 2 * k + (lane >> 4);
        const bool live = c * ROWS + r < rows;
        cp_async16_zfill(to + rw_piece(r, piece),
                         from + (live ? static_cast<int64_t>(r0 + c * ROWS + r) * kRwRowBytes : 0) + piece * 16,
                         live ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  uint8_t *const bufK = smem, *const bufV = smem + kRwBuffer;
  copy(p.K, 0, bufK);
  copy(p.V, 0, bufV);
  if constexpr (!kOnce) {
    copy(p.K, 1, bufK + kStage);
    copy(p.V, 1, bufV + kStage);
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
  const int mat = lane >> 3, mr = lane & 7;
  float m = -INFINITY, l = 0.0f;           // head g: running maximum (base 2), sum over this warp's rows
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // dims 16 warp + g (o[0], o[1]) and + 8, heads 2t and 2t + 1
  if (CL > 1 && steps == 0) cluster_arrive();
  for (int c = 0; c < steps; ++c) {
    const int at = kOnce ? 0 : (c & 1) * kStage;
    if (kOnce)
      cp_async_wait<1>();  // this warp's K rows (behind them V)
    else if (c == 0)
      cp_async_wait<3>();  // (V, K and V)
    else
      cp_async_wait<2>();  // (V and K)
    __syncwarp();
    // S of the warp's rows, eight to a tile
    float z[2 * kTiles];  // head g, rows 2t and 2t + 1 of each tile
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int row = (warp * kTiles + j) * 8;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t bk[4];
        ldmatrix_x4(bk, smem_u32(bufK + at) + rw_piece(row + mr, 4 * kk + mat));
        mma_16816_bf16(s, qa0[2 * kk], 0u, qa2[2 * kk], 0u, bk[0], bk[1]);
        mma_16816_bf16(s, qa0[2 * kk + 1], 0u, qa2[2 * kk + 1], 0u, bk[2], bk[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        z[2 * j + i] = c * ROWS + row + 2 * t + i < rows ? p.tau2 * s[i] : -INFINITY;
      mx = fmaxf(mx, fmaxf(z[2 * j], z[2 * j + 1]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (t == 0) sh.wm[c & 1][warp][g] = mx;
    __syncthreads();  // the maxima are there; the K rows of this step and the V rows and P of the last are read
    if (CL > 1 && c == steps - 1) cluster_arrive();  // the others may write over this CTA's K rows
    if constexpr (!kOnce) {
      if (c > 0) copy(p.V, c + 1, bufV + (kStage - at));
      copy(p.K, c + 2, bufK + at);
    }
    float mn = m;
#pragma unroll
    for (int w = 0; w < kRwWarps; ++w) mn = fmaxf(mn, sh.wm[c & 1][w][g]);
    const float sc = m == mn ? 1.0f : exp2f(m - mn);
    m = mn;
    float ps = 0.0f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      float a = z[2 * j] == -INFINITY ? 0.0f : exp2f(z[2 * j] - m);
      float b = z[2 * j + 1] == -INFINITY ? 0.0f : exp2f(z[2 * j + 1] - m);
      ps += a + b;
      uint32_t *to = reinterpret_cast<uint32_t *>(&sh.p[0][g][(warp * kTiles + j) * 8 + 2 * t]);
      constexpr int kPart = 8 * (ROWS + 8) / 2;  // words from one part to the next
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint32_t h = g < G ? pack_bf16x2(a, b) : 0u;  // (the operand's heads past G are zeros)
        to[part * kPart] = h;
        a -= bf16lo(h);
        b -= bf16hi(h);
      }
    }
    ps += __shfl_xor_sync(0xffffffffu, ps, 1);
    ps += __shfl_xor_sync(0xffffffffu, ps, 2);
    l = fmaf(l, sc, ps);
    // O follows the maximum; heads 2t and 2t + 1 have their factors in lanes 8t and 8t + 4
    const float sca = __shfl_sync(0xffffffffu, sc, 8 * t), scb = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
    cp_async_wait<kOnce ? 0 : 3>();  // this warp's V rows (behind them K, V and K)
    __syncthreads();                 // everyone's, and P
    // O^T of dims 16 warp .. + 15: A = V^T (16 dims x 16 rows per step), B = P^T.  The tensor cores cut off
    // what does not fit their sum, so a step has one of its own.
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < ROWS / 16; ++k) {
      if (c * ROWS + 16 * k >= rows) break;
      uint32_t av[4];
      ldmatrix_x4_trans(av, smem_u32(bufV + at) + rw_piece(16 * k + (mat >> 1) * 8 + mr, 2 * warp + (mat & 1)));
#pragma unroll
      for (int part = 2; part >= 0; --part) {  // the small parts first
        const uint32_t *b = reinterpret_cast<const uint32_t *>(&sh.p[part][g][16 * k + 2 * t]);
        mma_16816_bf16(d, av[0], av[1], av[2], av[3], b[0], b[4]);
      }
    }
    o[0] = fmaf(o[0], sca, d[0]);
    o[1] = fmaf(o[1], scb, d[1]);
    o[2] = fmaf(o[2], sca, d[2]);
    o[3] = fmaf(o[3], scb, d[3]);
  }
  cp_async_wait<0>();  // (empty groups)
  if (t == 0) sh.wl[warp][g] = l;
  __syncthreads();
  if constexpr (CL == 1) {
    if (warp == 0 && lane < 8) {
      float ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kRwWarps; ++w) ls += sh.wl[w][lane];
      sh.l[lane] = ls;
    }
    __syncthreads();
    if (2 * t < G) {
      float *out = p.out + u * G * kHeadDim + 16 * warp + g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = 2 * t + (i & 1);
        const float lh = sh.l[h];
        out[h * kHeadDim + 8 * (i >> 1)] = lh > 0.0f || lh != lh ? o[i] / lh : 0.0f;
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
    for (int li = threadIdx.x; li < per; li += kRwThreads) {
      const int h = (rank * per + li) / kHeadDim;
      float M = -INFINITY;
#pragma unroll
      for (int c = 0; c < CL; ++c) M = fmaxf(M, mine->m[c][h]);
      float L = 0.0f, A = 0.0f;
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        // (a CTA without keys has nothing to add)
        const float f = mine->m[c][h] == -INFINITY ? 0.0f : exp2f(mine->m[c][h] - M);
        if (f != 0.0f) {
          L = fmaf(mine->l[c][h], f, L);
          A = fmaf(mine->o[c][li], f, A);
        }
      }
      p.out[u * G * kHeadDim + rank * per + li] = L > 0.0f || L != L ? A / L : 0.0f;
    }
  }
}

template <int G, int CL, int ROWS>
cudaError_t launch_rw(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  constexpr int bytes = 2 * kRwBuffer + static_cast<int>(sizeof(RwShared<ROWS>));
  static_assert(3 * (bytes + 1024) <= 228 * 1024, "three CTAs per SM");
  constexpr auto kernel = window_ragged_kernel<G, CL, ROWS>;
  const cudaError_t e = allow_smem_once<kernel>(dev, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(units * CL)), dim3(kRwThreads), bytes, stream, 0u, p);
}

// One step of up to 128 rows per CTA where all CTAs are resident at once, or a ring has no more; else
// longer shares in steps of 64, as many CTAs to a unit as are resident at once.  (8 sequences of 4 KV heads
// with rings of 1,024 keys: 6.3 us in one step, 7.7 in two of 64; 96 of 2: 27.9 and 23.3; rings of 128: 5.4
// and 6.4.)
template <int G>
cudaError_t launch_rw_g(int64_t units, const RaggedWindowParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  const int64_t resident = 3ll * dev.sms;
  int cl = 1;
  while (cl * 128 < p.window) cl *= 2;
  if (cl == 1) return launch_rw<G, 1, 128>(units, p, dev, stream);
  if (units * cl <= resident) {
    if (cl == 2) return launch_rw<G, 2, 128>(units, p, dev, stream);
    if (cl == 4) return launch_rw<G, 4, 128>(units, p, dev, stream);
    return launch_rw<G, 8, 128>(units, p, dev, stream);
  }
  while (cl > 1 && units * cl > resident) cl /= 2;
  if (cl == 1) return launch_rw<G, 1, 64>(units, p, dev, stream);
  if (cl == 2) return launch_rw<G, 2, 64>(units, p, dev, stream);
  return launch_rw<G, 4, 64>(units, p, dev, stream);
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
