// Window-layer decode of sequences at positions of their own ("The Architecture of Embla 1",
// "Three kinds of attention", Sliding window): softmax of tau q . k over the keys in a ring, then the
// weighted sum of their values.  Query and keys were rotated when they were written, and a softmax does
// not ask for the order of its keys: the valid ones are the ring's rows 0 .. min(pos + 1, window) - 1.
//
// A cluster of CTAs takes a (sequence, KV head) unit, 128 ring rows to a CTA.  In a CTA
//   - each of eight warps copies 16 K rows and the same V rows into shared memory, all of them in
//     flight at once, and as soon as its K rows are there computes S = Q K^T of them as m16n8k16 MMAs
//     (M: the G query heads);
//   - the rows' maximum per head is exchanged, and P = exp2(z - max) written as three bf16 parts
//     (hi + mid + lo, all 24 bits: the output is fp32);
//   - each warp computes 16 of the 128 output dims over all 128 rows, O^T = V^T P^T, so no warp's
//     sums have to be added to another's.
// One pass, no running rescale.  CTAs of a unit exchange maximum, sum and O through distributed
// shared memory at the end.  Three CTAs fit an SM, so that one's arithmetic has the others' copies
// beside it.
#include <cooperative_groups.h>

#include "ptx_blocks.cuh"
#include "ragged.h"

namespace cg = cooperative_groups;

namespace embla {
namespace {

constexpr int kRwWarps = 8;
constexpr int kRwThreads = kRwWarps * 32;
constexpr int kRwRows = 128;  // ring rows per CTA
constexpr int kRwRowBytes = kHeadDim * 2;
constexpr int kRwStage = kRwRows * kRwRowBytes;  // 32 KB of K, as much of V
// the parts of P in one row per head, padded so that heads start in different banks
constexpr int kRwPRow = kRwRows + 8;

template <int G>
struct RwShared {
  uint16_t p[3][8][kRwPRow];  // parts of P, [part][head][row] (heads past G stay zero)
  float wm[kRwWarps][8];      // each warp's maximum per head
  float wl[kRwWarps][8];      // and sum
  float m[8], l[8];           // the CTA's
};

// byte offset of 16-byte piece c of staged row r: eight rows of an ldmatrix read eight bank groups
__device__ __forceinline__ uint32_t rw_piece(int r, int c) {
  return static_cast<uint32_t>(r * kRwRowBytes + ((c ^ (r & 7)) << 4));
}

template <int G, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kRwThreads, 3)
    window_ragged_kernel(const RaggedWindowParams p) {
  pdl_wait_primary();  // the query, the rings and the positions are complete
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];  // K rows, V rows, RwShared
  RwShared<G> &sh = *reinterpret_cast<RwShared<G> *>(smem + 2 * kRwStage);
  float(*so)[kHeadDim] = reinterpret_cast<float(*)[kHeadDim]>(smem);  // the CTA's sums for the cluster, over K
  const int rank = CL > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int64_t u = blockIdx.x / CL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int last = p.pos[u / p.Hkv];
  const int nv = last < 0 ? 0 : (last >= p.window ? p.window : last + 1);  // valid rows of the ring
  const int r0 = rank * kRwRows;
  const int rows = max(0, min(kRwRows, nv - r0));  // of this CTA

  // copies: one instruction moves two whole rows; rows past the valid ones are zeros
  {
    const uint8_t *Ku = p.K + (u * p.window + r0) * kRwRowBytes;
    const uint8_t *Vu = p.V + (u * p.window + r0) * kRwRowBytes;
    const int piece = lane & 15;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = warp * 16 + 2 * k + (lane >> 4);
      const uint32_t n = r < rows ? 16u : 0u;
      // (absent rows read nothing; their address stays inside the ring)
      const int64_t off = (r < rows ? r * kRwRowBytes : -static_cast<int64_t>(r0) * kRwRowBytes) + piece * 16;
      cp_async16_zfill(smem + rw_piece(r, piece), Ku + off, n);
    }
    cp_async_commit();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = warp * 16 + 2 * k + (lane >> 4);
      const uint32_t n = r < rows ? 16u : 0u;
      const int64_t off = (r < rows ? r * kRwRowBytes : -static_cast<int64_t>(r0) * kRwRowBytes) + piece * 16;
      cp_async16_zfill(smem + kRwStage + rw_piece(r, piece), Vu + off, n);
    }
    cp_async_commit();
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

  // S of rows 0-7 (s0) and 8-15 (s1) of this warp's 16
  const int mat = lane >> 3, mr = lane & 7;
  const int wrow = warp * 16;
  float s0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  {
    const uint32_t sK = smem_u32(smem);
    const int row = wrow + (mat >> 1) * 8 + mr;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t bk[4];
      ldmatrix_x4(bk, sK + rw_piece(row, 2 * ks + (mat & 1)));
      mma_16816_bf16(s0, qa0[ks], 0u, qa2[ks], 0u, bk[0], bk[1]);
      mma_16816_bf16(s1, qa0[ks], 0u, qa2[ks], 0u, bk[2], bk[3]);
    }
  }
  // head g, rows 2t, 2t + 1 (z[0], z[1]) and 8 + 2t, 9 + 2t (z[2], z[3]) of the warp's
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = wrow + 8 * (i >> 1) + 2 * t + (i & 1);
    z[i] = r < rows ? p.tau2 * (i < 2 ? s0[i] : s1[i - 2]) : -INFINITY;
  }
  float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if (t == 0) sh.wm[warp][g] = mx;
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kRwWarps; ++w) m = fmaxf(m, sh.wm[w][g]);
  float pz[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pz[i] = z[i] == -INFINITY ? 0.0f : exp2f(z[i] - m);
  float l = (pz[0] + pz[1]) + (pz[2] + pz[3]);
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) sh.wl[warp][g] = l;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    uint32_t *to = reinterpret_cast<uint32_t *>(&sh.p[0][g][wrow + 4 * i + 2 * t]);
    constexpr int kPart = 8 * kRwPRow / 2;  // words from one part to the next
    float a = pz[i], b = pz[i + 1];
    const bool head = g < G;  // the operand's heads past G are zeros
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const uint32_t h = head ? pack_bf16x2(a, b) : 0u;
      to[part * kPart] = h;
      a -= bf16lo(h);
      b -= bf16hi(h);
    }
  }
  cp_async_wait<0>();  // the V rows
  __syncthreads();

  // O^T of dims 16 warp .. + 15: A = V^T (16 dims x 16 rows per step), B = P^T
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // dims g (o[0], o[1]) and g + 8, heads 2t and 2t + 1
  {
    const uint32_t sV = smem_u32(smem + kRwStage);
    const int steps = (rows + 15) / 16;
    for (int k = 0; k < steps; ++k) {
      uint32_t av[4];
      const int row = 16 * k + (mat >> 1) * 8 + mr;
      ldmatrix_x4_trans(av, sV + rw_piece(row, 2 * warp + (mat & 1)));
#pragma unroll
      for (int part = 2; part >= 0; --part) {  // the small parts first
        const uint32_t *b = reinterpret_cast<const uint32_t *>(&sh.p[part][g][16 * k + 2 * t]);
        mma_16816_bf16(o, av[0], av[1], av[2], av[3], b[0], b[4]);
      }
    }
  }
  float ls = 0.0f;  // the CTA's sum for head `lane`
  if (warp == 0 && lane < 8) {
#pragma unroll
    for (int w = 0; w < kRwWarps; ++w) ls += sh.wl[w][lane];
  }
  if constexpr (CL == 1) {
    if (warp == 0 && lane < 8) sh.l[lane] = ls;
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
    cg::cluster_group cluster = cg::this_cluster();
    if (warp == 0 && lane < 8) {
      sh.l[lane] = ls;
    }
    if (warp == 1 && lane < 8) {
      float c = -INFINITY;
#pragma unroll
      for (int w = 0; w < kRwWarps; ++w) c = fmaxf(c, sh.wm[w][lane]);
      sh.m[lane] = c;
    }
    if (2 * t < G) {
#pragma unroll
      for (int i = 0; i < 4; ++i) so[2 * t + (i & 1)][16 * warp + g + 8 * (i >> 1)] = o[i];
    }
    cluster.sync();
    // each CTA finishes its share of the outputs from all the CTAs' states
    constexpr int per = G * kHeadDim / CL;
    for (int li = threadIdx.x; li < per; li += kRwThreads) {
      const int i = rank * per + li;
      const int h = i / kHeadDim, d = i % kHeadDim;
      float cm[CL], M = -INFINITY;
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        cm[c] = cluster.map_shared_rank(&sh, c)->m[h];
        M = fmaxf(M, cm[c]);
      }
      float L = 0.0f, A = 0.0f;
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        const RwShared<G> *other = cluster.map_shared_rank(&sh, c);
        // (a CTA without keys has nothing to add)
        const float f = cm[c] == -INFINITY ? 0.0f : exp2f(cm[c] - M);
        if (f != 0.0f) {
          L = fmaf(other->l[h], f, L);
          A = fmaf(cluster.map_shared_rank(&so[0][0], c)[h * kHeadDim + d], f, A);
        }
      }
      p.out[u * G * kHeadDim + i] = L > 0.0f || L != L ? A / L : 0.0f;
    }
    cluster_arrive();  // done reading the other CTAs' shared memory
    cluster_wait();    // and they are done reading this one's
  }
}

template <int G, int CL>
cudaError_t launch_rw(int64_t units, const RaggedWindowParams &p, cudaStream_t stream) {
  constexpr int bytes = 2 * kRwStage + static_cast<int>(sizeof(RwShared<G>));
  static_assert(3 * (bytes + 1024) <= 228 * 1024, "three CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(window_ragged_kernel<G, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(window_ragged_kernel<G, CL>, dim3(static_cast<unsigned>(units * CL)), dim3(kRwThreads), bytes,
                    stream, 0u, p);
}

// As many CTAs to a unit as its ring has blocks of 128 rows, rounded up to a power of two.
template <int G>
cudaError_t launch_rw_g(int64_t units, const RaggedWindowParams &p, cudaStream_t stream) {
  if (p.window <= kRwRows) return launch_rw<G, 1>(units, p, stream);
  if (p.window <= 2 * kRwRows) return launch_rw<G, 2>(units, p, stream);
  if (p.window <= 4 * kRwRows) return launch_rw<G, 4>(units, p, stream);
  return launch_rw<G, 8>(units, p, stream);
}

}  // namespace

cudaError_t launch_window_decode_ragged(int G, int64_t units, const RaggedWindowParams &p, cudaStream_t stream) {
  if (units == 0) return cudaSuccess;
  if (p.window < 1 || p.window > 8 * kRwRows) return cudaErrorInvalidValue;
  if (G == 4) return launch_rw_g<4>(units, p, stream);
  if (G == 8) return launch_rw_g<8>(units, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace embla
