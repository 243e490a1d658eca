// Causal attention over packed prompts of different lengths: the window layers' softmax over the
// newest `window` keys, and the full layers' ReLU^2 weights over all keys ("The Architecture of
// Embla 1", "Three kinds of attention" and "KV bridge, KV reuse, and prefill").
//
// Rows are packed token-major, [tokens][heads][128] bf16 with a stride between tokens, as a projection
// leaves them.  Sequence b has the queries cu_q[b] .. cu_q[b+1]-1 and the keys cu_k[b] .. cu_k[b+1]-1,
// and its queries are the last of its keys: query t sees the keys 0 .. p, p = Lk - Lq + t, of them the
// newest `window` only.
//
// packed_knorm_kernel (ReLU^2): rk[g][j] = 1 / sqrt(mean(k_j^2) + eps) for every key row.
//
// packed_prefill_kernel: a block is 128 / G tokens with the G query heads of one KV head, 128 rows
// of a matrix product that read the same keys; its key tiles of N rows start at the first key that
// some row of it sees.  Persistent CTAs, one per SM, take blocks in turn.  Warp roles:
//   warp 0     finds each block's sequence (below), hands the block's description to the others and
//              loads by TMA: the 128 query rows once, per tile the K and V rows, in rings of 3.
//   warp 1     tcgen05 issuer of S = Q K^T (M 128 rows x N keys) into one of three tensor-memory
//              buffers; S of tile t takes the buffer of tile t - 3 once its P V is done.
//   last warp  tcgen05 issuer of O += P V, P from tensor memory (over its S), V as it lies.
//   warps 2..9 the weights: a warp takes 16 rows, a row lies in the four lanes of a quad (the
//              fragment layout of 16x256b loads), so a row's maximum is two shuffles and no
//              other warp's business, and P, packed in pairs, goes back in 16x128b stores to the
//              columns of its own rows.
//
// Softmax.  With z = tau log2(e) s, P = exp2(z - m) for a running reference m per row and l = sum P.
// m follows the maximum only when that has grown by more than 2^8 (kSlack): O, in tensor memory, is then
// multiplied by exp2(m_old - m) once its last product is done; O / l does not depend on m.  m, l and
// O are fp32; P enters the product as bf16 (2^-9 of each weight, as much as the output's own
// rounding to bf16).
// ReLU^2.  w' = max(dot rk_j, 0)^2, a2 = alpha^2 / (mean(q^2) + eps): out = a2 O' / (c + a2 sum w').
//
// A weight of zero times an infinite or NaN value would be NaN, and a tile holds rows that a query
// must not see (later ones, older ones, other sequences').  An output that comes out infinite or NaN
// is therefore computed again by its warp, key by key over the visible ones (slow_row); nothing
// else pays for it.
//
// A block's sequence.  The host knows no lengths, so block numbers are spread with room to spare: sequence
// b owns the numbers from floor(cu_q[b] / R) + b (R tokens to a block), which is enough for its blocks,
// and a number past them is skipped.  The owner is found by a 32-way search.
#include "ptx_blocks.cuh"
#include "ragged.h"

namespace embla {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kWarpPV = 2 + kEpiWarps;
constexpr int kThreads = (3 + kEpiWarps) * 32;
constexpr int kRing = 3;           // K and V stages, S/P buffers
constexpr int kBoxQ = 128 * 128;   // [128 rows][64 bf16]
constexpr float kSlack = 8.0f;     // P stays below 2^kSlack
constexpr uint64_t kLimitNs = 10000000000ull;  // 10 s: a row computed key by key holds the others up
constexpr int kColO = kRing * 128, kTmemCols = 512;
static_assert(kColO + 128 <= kTmemCols, "tensor memory");
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128) | (1u << 16);  // B (V) MN-major

// What a block is, relative to its first key row k0: row i / G's newest key is p0 + i, its oldest
// max(seq0, p0 + i - window + 1).
struct Block {
  int32_t tiles;  // key tiles; -1: no more blocks
  int32_t q0;     // first token
  int32_t nq;     // tokens
  int32_t g;      // KV head
  int32_t k0;     // first key row of tile 0
  int32_t p0;     // the first token's newest key, less k0
  int32_t seq0;   // the sequence's first key, less k0
  int32_t pad;
};

template <int N>
struct Layout {
  static constexpr int kBoxKV = N * 128;  // [N rows][64 bf16]
  static constexpr int kStage = 2 * kBoxKV;
  static constexpr int kOffK = 2 * kBoxQ;
  static constexpr int kOffV = kOffK + kRing * kStage;
  static constexpr int kOffSum = kOffV + kRing * kStage;  // [2][128] row sums
  static constexpr int kOffBlock = kOffSum + 2 * 128 * 4;
  static constexpr int kOffBar = kOffBlock + 2 * static_cast<int>(sizeof(Block));
  static constexpr int kNBars = 5 * kRing + 4;
  static constexpr int kOffMisc = kOffBar + kNBars * 8;
  static constexpr int kBytes = kOffMisc + 16 + 1024;  // + room to align the base to 1024
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, kLimitNs); }

__device__ __forceinline__ void set_abort(volatile int *abort_flag, uint32_t *flags) {
  *abort_flag = 1;
  atomicOr(flags, kFlagWaitTimeout);
}

// The k-th block number of CTA c among P: a round of P at a time, alternate rounds in reverse
// order, so the CTAs' sums of key tiles stay close.  -1 past the end.
__device__ __forceinline__ int64_t block_of(const PackedPrefillParams &p, int k, int c, int P) {
  const int64_t idx = static_cast<int64_t>(k) * P + ((k & 1) ? P - 1 - c : c);
  return idx < p.blocks ? idx : -1;
}

// Entries that do not ascend or lie outside the rows.
__device__ __forceinline__ bool bad_sequence(const PackedPrefillParams &p, int64_t q_lo, int64_t q_hi, int64_t k_lo,
                                             int64_t k_hi) {
  return q_lo < 0 || q_hi < q_lo || q_hi > p.tokens || k_lo < 0 || k_hi < k_lo || k_hi > p.keys;
}

// Block number idx (the whole warp calls); tiles < 0 where there is none.
template <int MODE, int N, int G>
__device__ __forceinline__ Block find_block(const PackedPrefillParams &p, int64_t idx, int lane) {
  constexpr int R = 128 / G;
  Block r = {};
  r.tiles = -1;
  r.g = static_cast<int32_t>(idx % p.Hkv);
  const int64_t v = p.blocks / p.Hkv - 1 - idx / p.Hkv;  // the last ones, with the most keys, first
  // sequences whose successor's numbers begin at or before v
  int lo = 0, hi = p.batch;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool past = at <= hi && p.cu_q[at] / R + at <= v;
    const int n = __popc(__ballot_sync(0xffffffffu, past));
    const int from = lo + n * step;
    hi = min(hi, from + step - 1);
    lo = from;
  }
  if (lo >= p.batch) return r;
  const int64_t q_lo = p.cu_q[lo], q_hi = p.cu_q[lo + 1], k_lo = p.cu_k[lo], k_hi = p.cu_k[lo + 1];
  if (bad_sequence(p, q_lo, q_hi, k_lo, k_hi)) return r;
  const int64_t t0 = (v - (q_lo / R + lo)) * R, lq = q_hi - q_lo, lk = k_hi - k_lo;
  if (t0 < 0 || t0 >= lq) return r;
  r.q0 = static_cast<int32_t>(q_lo + t0);
  r.nq = static_cast<int32_t>(lq - t0 < R ? lq - t0 : R);
  const int64_t first = lk - lq + t0, last = first + r.nq - 1;  // newest keys of the first and last token
  const int64_t oldest = first - p.window + 1 > 0 ? first - p.window + 1 : 0;
  int64_t k0 = k_lo + oldest;
  if (MODE == kPackedRelu2) k0 &= ~static_cast<int64_t>(3);  // (the key norms are read in pairs)
  r.tiles = last < 0 ? 0 : static_cast<int32_t>((k_lo + last - k0) / N) + 1;
  r.k0 = static_cast<int32_t>(k0);
  r.p0 = static_cast<int32_t>(k_lo + first - k0);
  r.seq0 = static_cast<int32_t>(k_lo - k0);
  return r;
}

// Row r of a block (token r / G, head r % G) computed key by key: columns 64 half .. + 63 of its
// output, by one warp.  In two passes, so that no partial sum is larger than the result needs:
// maximum and sum (ReLU^2: the sum), then the values by their normalised weights.
template <int MODE, int G>
__device__ __noinline__ void slow_row(const PackedPrefillParams &p, const Block &b, int r, int half, int lane) {
  const int i = r / G, h = b.g * G + r % G;
  const uint16_t *q = p.q.base + static_cast<int64_t>(b.q0 + i) * p.q.stride + h * kHeadDim;
  const uint2 qw = *reinterpret_cast<const uint2 *>(q + 4 * lane);
  const float qf[4] = {bf16lo(qw.x), bf16hi(qw.x), bf16lo(qw.y), bf16hi(qw.y)};
  float scale = p.tau2;
  if (MODE == kPackedRelu2) {
    float ss = (qf[0] * qf[0] + qf[1] * qf[1]) + (qf[2] * qf[2] + qf[3] * qf[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    scale = p.alpha / sqrtf(ss * (1.0f / kHeadDim) + p.eps);
  }
  const int64_t newest = b.p0 + i;
  const int64_t oldest = newest - p.window + 1 > b.seq0 ? newest - p.window + 1 : b.seq0;
  // the score of key j for lane (j - first key of the step)
  auto score = [&](int64_t j) {
    const bool live = j <= newest;
    const uint16_t *k = p.k.base + (b.k0 + (live ? j : newest)) * p.k.stride + b.g * kHeadDim;
    float s = 0.0f;
    for (int d = 0; d < kHeadDim; d += 8) {
      const uint4 x = *reinterpret_cast<const uint4 *>(k + d);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(__shfl_sync(0xffffffffu, qf[(2 * e) & 3], (d + 2 * e) / 4), bf16lo(w[e]), s);
        s = fmaf(__shfl_sync(0xffffffffu, qf[(2 * e + 1) & 3], (d + 2 * e) / 4), bf16hi(w[e]), s);
      }
    }
    s *= scale;
    if (MODE == kPackedRelu2) {
      const float w = live ? fmaxf(s * p.rk[b.g * p.rk_stride + b.k0 + j], 0.0f) : 0.0f;
      return w * w;
    }
    return live ? s : -INFINITY;
  };
  float m = -INFINITY, l = 0.0f;
  for (int64_t j0 = oldest; j0 <= newest; j0 += 32) {
    const float s = score(j0 + lane);
    if (MODE == kPackedRelu2) {
      l += s;
    } else {
      const float mn = fmaxf(m, s);
      l = l * (m == mn ? 1.0f : exp2f(m - mn)) + (s == -INFINITY ? 0.0f : exp2f(s - mn));
      m = mn;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    if (MODE == kPackedRelu2) {
      l += l2;
    } else {
      const float mn = fmaxf(m, m2);
      l = l * (m == mn ? 1.0f : exp2f(m - mn)) + l2 * (m2 == mn ? 1.0f : exp2f(m2 - mn));
      m = mn;
    }
  }
  const float z = MODE == kPackedRelu2 ? p.c + l : l;
  const float f = z == 0.0f ? 0.0f : 1.0f / z;
  float a0 = 0.0f, a1 = 0.0f;
  for (int64_t j0 = oldest; j0 <= newest; j0 += 32) {
    const float s = score(j0 + lane);
    const float w = MODE == kPackedRelu2 ? s * f : (s == -INFINITY ? 0.0f : exp2f(s - m) * f);
    const int n = static_cast<int>(newest - j0 + 1 < 32 ? newest - j0 + 1 : 32);
    for (int c = 0; c < n; ++c) {
      const float wc = __shfl_sync(0xffffffffu, w, c);
      if (MODE == kPackedRelu2 && wc == 0.0f) continue;  // weighs nothing, whatever its value holds
      const uint32_t x = *reinterpret_cast<const uint32_t *>(p.v.base + (b.k0 + j0 + c) * p.v.stride + b.g * kHeadDim +
                                                             64 * half + 2 * lane);
      a0 = fmaf(wc, bf16lo(x), a0);
      a1 = fmaf(wc, bf16hi(x), a1);
    }
  }
  *reinterpret_cast<uint32_t *>(p.out + (static_cast<int64_t>(b.q0 + i) * p.Hkv * G + h) * kHeadDim + 64 * half +
                                2 * lane) = pack_bf16x2(a0, a1);
}

template <int MODE, int N, int G>
__global__ void __launch_bounds__(kThreads, 1)
    packed_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PackedPrefillParams p) {
  using L = Layout<N>;
  static_assert(N % 16 == 0 && N <= 128, "key tile");
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, N);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem, *sK = smem + L::kOffK, *sV = smem + L::kOffV;
  float *sSum = reinterpret_cast<float *>(smem + L::kOffSum);
  Block *sBlock = reinterpret_cast<Block *>(smem + L::kOffBlock);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  // A K stage is free once its tile's S is done (sfull), a V stage once its P V is done
  // (pvdone).  Block k's barriers take phase k & 1, tile g's phase (g / kRing) & 1.
  uint64_t *kfull = bars, *vfull = kfull + kRing;
  uint64_t *sfull = vfull + kRing;   // S of a tile in tensor memory; its K stage free
  uint64_t *pfull = sfull + kRing;   // its P written over it
  uint64_t *pvdone = pfull + kRing;  // its P V done: the S/P buffer and the V stage are free
  uint64_t *qfull = pvdone + kRing;  // a block's description and query rows are there
  uint64_t *qempty = qfull + 1;      // the description read by everyone, the query rows used
  uint64_t *ofull = qempty + 1;      // a block's P V all done
  uint64_t *ofree = ofull + 1;       // its O read out of tensor memory
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  uint32_t *s_tmem = misc;
  volatile int *s_abort = reinterpret_cast<volatile int *>(misc + 1);
  volatile int *s_issued = reinterpret_cast<volatile int *>(misc + 2);   // loads issued: 2 per tile
  volatile int *s_qissued = reinterpret_cast<volatile int *>(misc + 3);  // query loads issued

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x), P = static_cast<int>(gridDim.x);

  if (warp == 0) {
    if (lane < kRing) {
      mbar_init(&kfull[lane], 1);
      mbar_init(&vfull[lane], 1);
      mbar_init(&sfull[lane], 1);
      mbar_init(&pfull[lane], kEpiWarps);
      mbar_init(&pvdone[lane], 1);
    }
    if (lane == 0) {
      mbar_init(qfull, 1);
      mbar_init(qempty, 2 + kEpiWarps);  // the S issuer's commit, the P V issuer, the weights' warps
      mbar_init(ofull, 1);
      mbar_init(ofree, kEpiWarps);
      *s_abort = 0;
      *s_issued = 0;
      *s_qissued = 0;
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);
  pdl_wait_primary();  // the rows, the lengths and the key norms are complete
  pdl_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------------ blocks and loads
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int g = 0, k = 0;
    bool ok = true, more = true;
    for (int n = 0; ok && more; ++n) {
      const int64_t idx = block_of(p, n, cta, P);
      more = idx >= 0;
      Block b = {};
      b.tiles = -1;
      if (more) {
        b = find_block<MODE, N, G>(p, idx, lane);
        if (b.tiles < 0) continue;
      }
      if (lane == 0) {
        // the query buffer and the description are free once the block before is done with them
        ok = k == 0 || wait_bar(qempty, (k - 1) & 1);
        if (ok) {
          sBlock[k & 1] = b;
          if (b.tiles > 0) {
            mbar_arrive_expect_tx(qfull, 2 * kBoxQ);
            tma_load_4d(sQ, &tm_q, qfull, 0, 0, b.g, b.q0);
            tma_load_4d(sQ + kBoxQ, &tm_q, qfull, 64, 0, b.g, b.q0);
          } else {
            mbar_arrive(qfull);
          }
          *s_qissued = k + 1;
          for (int t = 0; t < b.tiles; ++t, ++g) {
            const int s = g % kRing;
            const uint32_t ph = ((g / kRing) - 1) & 1;
            if (g >= kRing && !wait_bar(&sfull[s], ph)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&kfull[s], L::kStage);
            tma_load_3d(sK + s * L::kStage, &tm_k, &kfull[s], 0, b.g, b.k0 + t * N);
            tma_load_3d(sK + s * L::kStage + L::kBoxKV, &tm_k, &kfull[s], 64, b.g, b.k0 + t * N);
            if (g >= kRing && !wait_bar(&pvdone[s], ph)) {
              *s_issued = 2 * g + 1;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&vfull[s], L::kStage);
            tma_load_3d(sV + s * L::kStage, &tm_v, &vfull[s], 0, b.g, b.k0 + t * N);
            tma_load_3d(sV + s * L::kStage + L::kBoxKV, &tm_v, &vfull[s], 64, b.g, b.k0 + t * N);
            *s_issued = 2 * g + 2;
          }
        }
        if (!ok) set_abort(s_abort, p.flags);
      }
      ++k;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    // entries that no block could use are reported
    for (int64_t b = static_cast<int64_t>(cta) * 32 + lane; b < p.batch; b += static_cast<int64_t>(P) * 32)
      if (bad_sequence(p, p.cu_q[b], p.cu_q[b + 1], p.cu_k[b], p.cu_k[b + 1])) atomicOr(p.flags, kFlagIndexRange);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S issuer
    if (lane == 0) {
      const uint64_t qdesc = smem_desc_sw128(smem_u32(sQ));
      const uint64_t kdesc = smem_desc_sw128(smem_u32(sK));
      int g = 0, blocks = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = !*s_abort && wait_bar(qfull, k & 1);
        if (!ok) break;
        const int tiles = sBlock[k & 1].tiles;
        if (tiles < 0) break;
        for (int t = 0; ok && t < tiles; ++t, ++g) {
          const int sb = g % kRing;
          ok = wait_bar(&kfull[sb], (g / kRing) & 1) &&
               (g < kRing || wait_bar(&pvdone[sb], ((g / kRing) - 1) & 1));
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // dims 16kk .. 16kk + 15: 32 bytes into a 128-byte row; dims 64.. start the second box
            const uint64_t qo = static_cast<uint64_t>(((kk >> 2) * kBoxQ + (kk & 3) * 32) >> 4);
            const uint64_t ko = static_cast<uint64_t>((sb * L::kStage + (kk >> 2) * L::kBoxKV + (kk & 3) * 32) >> 4);
            tc_mma_bf16(tmem + sb * 128, qdesc + qo, kdesc + ko, kIdescS, kk > 0 ? 1u : 0u);
          }
          tc_commit(&sfull[sb]);
        }
        if (ok) {
          tc_commit(qempty);
          blocks = k + 1;
        }
      }
      if (!ok) set_abort(s_abort, p.flags);
      // every MMA of this thread has completed, and its last commit arrived, before the tensor
      // memory is released and the CTA leaves (also when another role has given up)
      if (g > 0) wait_bar(&sfull[(g - 1) % kRing], ((g - 1) / kRing) & 1);
      if (blocks > 0) wait_bar(qempty, (blocks - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------------------ P V issuer
    if (lane == 0) {
      int g = 0, blocks = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = !*s_abort && wait_bar(qfull, k & 1);
        if (!ok) break;
        const int tiles = sBlock[k & 1].tiles;
        mbar_arrive(qempty);
        if (tiles < 0) break;
        ok = k == 0 || wait_bar(ofree, (k - 1) & 1);  // the block before's O has been read
        for (int t = 0; ok && t < tiles; ++t, ++g) {
          const int pb = g % kRing;
          ok = wait_bar(&pfull[pb], (g / kRing) & 1) && wait_bar(&vfull[pb], (g / kRing) & 1);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < N / 16; ++kk) {
            // keys 16kk .. 16kk + 15: eight columns of P, V rows 16kk .. (2 KB apart)
            const uint64_t vd = smem_desc_sw128_mn(smem_u32(sV + pb * L::kStage + kk * 2048), L::kBoxKV);
            tc_mma_bf16_tmem_a(tmem + kColO, tmem + pb * 128 + 8 * kk, vd, kIdescPV, (t > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&pvdone[pb]);
        }
        if (ok) {
          tc_commit(ofull);
          blocks = k + 1;
        }
      }
      if (!ok) set_abort(s_abort, p.flags);
      // every MMA of this thread has completed before the tensor memory is released
      if (g > 0) wait_bar(&pvdone[(g - 1) % kRing], ((g - 1) / kRing) & 1);
      if (blocks > 0) wait_bar(ofull, (blocks - 1) & 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ weights and outputs
    const int quarter = warp & 3;      // the tensor-memory lanes this warp may reach
    const int half = (warp - 2) >> 2;  // rows 16 half .. of them; at the end columns 64 half .. of O
    const int row0 = quarter * 32 + half * 16 + (lane >> 2);  // this lane's rows: row0 and row0 + 8
    const int q2 = 2 * (lane & 3);                            // its columns: 8j + q2 and the next
    const uint32_t lanes32 = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t lanes16 = lanes32 + (static_cast<uint32_t>(half * 16) << 16);
    const bool flip = MODE == kPackedSoftmax && p.tau2 < 0.0f;
    const float tau2 = fabsf(p.tau2);
    int g = 0;
    bool ok = true;
    for (int k = 0;; ++k) {
      // (every decision to go on is the group's: what follows is warp-wide and has barriers)
      ok = __all_sync(0xffffffffu, ok && !*s_abort && wait_bar(qfull, k & 1));
      ok = named_bar_and(1, kEpiWarps * 32, ok);
      if (!ok) break;
      const Block b = sBlock[k & 1];
      if (b.tiles < 0) break;
      float a2 = 0.0f;  // ReLU^2, row quarter * 32 + lane: alpha^2 / (mean(q^2) + eps)
      if (MODE == kPackedRelu2 && b.tiles > 0) {
        const int r = quarter * 32 + lane;
        a2 = (p.alpha * p.alpha) / (row_square_sum(sQ, kBoxQ, r, r & 7) * (1.0f / kHeadDim) + p.eps);
        // the query rows are read: every lane's sum depends on them
        const float used = __shfl_sync(0xffffffffu, a2, 0) + __shfl_sync(0xffffffffu, a2, 31);
        __syncwarp();
        if (lane == 0) mbar_arrive_after(qempty, used);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty);
      }
      // the keys that a row sees lie between these two, relative to k0
      int newest[2], oldest[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        newest[i] = b.p0 + (row0 + 8 * i) / G;
        oldest[i] = max(b.seq0, newest[i] - p.window + 1);
      }
      // tiles between these two are seen whole by every row of the block
      const int whole0 = max(b.seq0, b.p0 + b.nq - p.window), whole1 = b.p0;
      float m[2] = {-INFINITY, -INFINITY};  // reference of each row (base 2)
      float l[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // sums of its weights in this lane, two chains per row
      for (int t = 0; t < b.tiles; ++t, ++g) {
        const int sb = g % kRing;
        const int j0 = t * N;
        float2 rk[MODE == kPackedRelu2 ? N / 8 : 1];
        if constexpr (MODE == kPackedRelu2) {
          const float *from = p.rk + b.g * p.rk_stride + b.k0 + j0 + q2;
#pragma unroll
          for (int j = 0; j < N / 8; ++j) rk[j] = *reinterpret_cast<const float2 *>(from + 8 * j);
        }
        ok = __all_sync(0xffffffffu, wait_bar(&sfull[sb], (g / kRing) & 1));
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t cols = tmem + lanes16 + sb * 128;
        uint32_t acc[N / 2];  // element 4j + 2i + e: row row0 + 8i, key j0 + 8j + q2 + e
        if constexpr (N == 128) {
          tmem_load_16x256b_x16(cols, acc);
          tmem_wait_ld(acc);
        } else {
          static_assert(N == 128 || N == 80, "tile loads");
          uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&acc[0]);
          uint32_t(&hi)[8] = *reinterpret_cast<uint32_t(*)[8]>(&acc[32]);
          tmem_load_16x256b_x8(cols, lo);
          tmem_load_16x256b_x2(cols + 64, hi);
          tmem_wait_ld(acc);
        }
        const bool masked = j0 < whole0 || j0 + N - 1 > whole1;
        uint32_t hi[N / 4];
        if constexpr (MODE == kPackedSoftmax) {
          if (flip) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) acc[e] ^= 0x80000000u;
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t span = static_cast<uint32_t>(newest[i] - oldest[i]);
              const int off = j0 + q2 - oldest[i];
              const bool none = newest[i] < oldest[i];
#pragma unroll
              for (int j = 0; j < N / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (none || static_cast<uint32_t>(off + 8 * j + e) > span) acc[4 * j + 2 * i + e] = 0xFF800000u;
            }
          }
          float neg[2];
          bool grown = false;
          float sc[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < N / 8; ++j)
              x[j & 3] = max3(x[j & 3], __uint_as_float(acc[4 * j + 2 * i]), __uint_as_float(acc[4 * j + 2 * i + 1]));
            float mx = max3(fmaxf(x[0], x[1]), x[2], x[3]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx *= tau2;
            sc[i] = 1.0f;
            if (mx > m[i] + kSlack) {  // (from -infinity: the row's first keys, with nothing to rescale)
              if (m[i] != -INFINITY) {
                grown = true;
                sc[i] = exp2_approx(m[i] - mx);
              }
              m[i] = mx;
            }
            neg[i] = m[i] == -INFINITY ? 0.0f : -m[i];
          }
          if (t > 0 && __any_sync(0xffffffffu, grown)) {
            // O of these rows, once the products before this tile are done
            ok = __all_sync(0xffffffffu, wait_bar(&pvdone[(g - 1) % kRing], ((g - 1) / kRing) & 1));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] *= sc[i >> 1];
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
              uint32_t o[32];
              tmem_load_16x256b_x8(tmem + lanes16 + kColO + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sc[(e >> 1) & 1]);
              tmem_store_16x256b_x8(tmem + lanes16 + kColO + c, o);
            }
          }
#pragma unroll
          for (int j = 0; j < N / 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float e0, e1;
              fma_f32x2(e0, e1, __uint_as_float(acc[4 * j + 2 * i]), __uint_as_float(acc[4 * j + 2 * i + 1]), tau2,
                        tau2, neg[i], neg[i]);
              e0 = exp2_approx(e0);
              e1 = exp2_approx(e1);
              fma_f32x2(l[2 * i], l[2 * i + 1], e0, e1, 1.0f, 1.0f, l[2 * i], l[2 * i + 1]);
              hi[2 * j + i] = pack_bf16x2(e0, e1);
            }
        } else {
#pragma unroll
          for (int j = 0; j < N / 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // (a NaN score weighs nothing: the maximum of NaN and 0 is 0)
              float e0, e1;
              fma_f32x2(e0, e1, __uint_as_float(acc[4 * j + 2 * i]), __uint_as_float(acc[4 * j + 2 * i + 1]), rk[j].x,
                        rk[j].y, 0.0f, 0.0f);
              e0 = fmaxf(e0, 0.0f);
              e1 = fmaxf(e1, 0.0f);
              if (masked) {
                const int c = j0 + 8 * j + q2;
                if (c < oldest[i] || c > newest[i]) e0 = 0.0f;
                if (c + 1 < oldest[i] || c + 1 > newest[i]) e1 = 0.0f;
              }
              fma_f32x2(e0, e1, e0, e1, e0, e1, 0.0f, 0.0f);
              const uint32_t h = pack_bf16x2(e0, e1);
              hi[2 * j + i] = h;
              // the denominator sums the weights the numerator multiplies
              fma_f32x2(l[2 * i], l[2 * i + 1], bf16lo(h), bf16hi(h), 1.0f, 1.0f, l[2 * i], l[2 * i + 1]);
            }
        }
        if constexpr (N == 128) {
          tmem_store_16x128b_x16(cols, hi);
        } else {
          tmem_store_16x128b_x8(cols, *reinterpret_cast<const uint32_t(*)[16]>(&hi[0]));
          tmem_store_16x128b_x2(cols + 32, *reinterpret_cast<const uint32_t(*)[4]>(&hi[16]));
        }
        tmem_wait_st();
        tc_fence_before_sync();  // P is read by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[sb]);
      }
      // the row sums, for the lanes that finish the rows
      float *sum = sSum + (k & 1) * 128;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[2 * i] + l[2 * i + 1];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (q2 == 0) sum[row0 + 8 * i] = x;
      }
      ok = __all_sync(0xffffffffu, ok && !*s_abort && wait_bar(ofull, k & 1));
      ok = named_bar_and(1, kEpiWarps * 32, ok);
      if (!ok) break;
      tc_fence_after_sync();
      // row quarter * 32 + lane, columns 64 half .. + 63
      const int r = quarter * 32 + lane;
      uint32_t o[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32)
        tmem_load_x32(tmem + lanes32 + kColO + half * 64 + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c]));
      tmem_wait_ld(o);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);  // the next block's P V may overwrite O
      const float s = sum[r];
      float f;  // 0 where no key weighs anything
      if (MODE == kPackedRelu2) {
        const float z = p.c + a2 * s;
        f = s != 0.0f && z != 0.0f ? a2 / z : 0.0f;
      } else {
        f = s != 0.0f ? 1.0f / s : 0.0f;
      }
      const bool live = r / G < b.nq;
      const bool empty = f == 0.0f;
      float chk = 0.0f;  // NaN if an output is infinite or NaN
      uint32_t y[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float y0 = __uint_as_float(o[2 * c]) * f, y1 = __uint_as_float(o[2 * c + 1]) * f;
        chk = fmaf(y0, 0.0f, fmaf(y1, 0.0f, chk));
        y[c] = empty ? 0u : pack_bf16x2(y0, y1);
      }
      if (live) {
        uint16_t *dst = p.out + (static_cast<int64_t>(b.q0 + r / G) * p.Hkv * G + b.g * G + r % G) * kHeadDim + half * 64;
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
          const uint4 w0 = make_uint4(y[c], y[c + 1], y[c + 2], y[c + 3]);
          const uint4 w1 = make_uint4(y[c + 4], y[c + 5], y[c + 6], y[c + 7]);
          if (p.out32) {  // whole sectors
            st_global_v8(dst + 2 * c, w0, w1);
          } else {
            *reinterpret_cast<uint4 *>(dst + 2 * c) = w0;
            *reinterpret_cast<uint4 *>(dst + 2 * c + 8) = w1;
          }
        }
      }
      uint32_t bad = __ballot_sync(0xffffffffu, live && !empty && chk != 0.0f);
      while (bad) {
        const int at = __ffs(bad) - 1;
        bad &= bad - 1;
        __syncwarp();
        slow_row<MODE, G>(p, b, quarter * 32 + at, half, lane);
      }
    }
    if (!ok) set_abort(s_abort, p.flags);
  }

  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) {
    // No copy may still be landing in shared memory when the CTA leaves.  Without an abort
    // every copy issued was waited for by the role that used it; after one, wait (bounded)
    // for the last armed phase of every barrier that a copy completes.
    const int qi = *s_qissued;
    if (qi > 0) wait_bar(qfull, (qi - 1) & 1);
    const int issued = *s_issued;  // 2 per key tile: K, V
    const int nk = (issued + 1) / 2, nv = issued / 2;
    for (int s = 0; s < kRing; ++s) {
      int uses = nk > s ? (nk - 1 - s) / kRing + 1 : 0;
      if (uses) wait_bar(&kfull[s], (uses - 1) & 1);
      uses = nv > s ? (nv - 1 - s) / kRing + 1 : 0;
      if (uses) wait_bar(&vfull[s], (uses - 1) & 1);
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// rk[g][j] = 1 / sqrt(mean(k_j^2) + eps): eight lanes per (key, KV head) row, 32 bytes each.
__global__ void __launch_bounds__(256) packed_knorm_kernel(const PackedPrefillParams p, float *rk) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x / 8;
  const int part = threadIdx.x % 8;
  const int64_t j = row / p.Hkv;
  const int g = static_cast<int>(row - j * p.Hkv);
  if (j >= p.keys) return;  // (eight lanes leave together)
  const uint4 *src = reinterpret_cast<const uint4 *>(p.k.base + j * p.k.stride + g * kHeadDim) + 2 * part;
  const uint4 x = src[0], y = src[1];
  float a = 0.0f, b = 0.0f;
  sq_acc_bf16x2(x.x, a, b);
  sq_acc_bf16x2(x.y, a, b);
  sq_acc_bf16x2(x.z, a, b);
  sq_acc_bf16x2(x.w, a, b);
  sq_acc_bf16x2(y.x, a, b);
  sq_acc_bf16x2(y.y, a, b);
  sq_acc_bf16x2(y.z, a, b);
  sq_acc_bf16x2(y.w, a, b);
  a += b;
  const uint32_t mine = 0xFFu << (threadIdx.x & 24);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(mine, a, o);
  if (part == 0) rk[g * p.rk_stride + j] = 1.0f / sqrtf(a * (1.0f / kHeadDim) + p.eps);
}

template <int MODE, int N, int G>
cudaError_t launch_packed(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                          const PackedPrefillParams &p, int ctas, cudaStream_t stream) {
  auto kernel = packed_prefill_kernel<MODE, N, G>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), static_cast<size_t>(Layout<N>::kBytes),
                    stream, 0u, tm_q, tm_k, tm_v, p);
}

}  // namespace

// Keys per tile: a block of 128 / G tokens sees window + 128 / G - 1 keys at most.
int packed_tile_keys(int mode, int G, int64_t window) {
  (void)mode;
  (void)G;
  (void)window;
  return 128;
}

int64_t packed_rk_stride(int64_t keys) { return (keys + 3) & ~static_cast<int64_t>(3); }

// The last tile's norms may be read up to a tile past the last row's.
size_t packed_workspace_bytes(int64_t keys, int Hkv) {
  return (static_cast<size_t>(Hkv) * static_cast<size_t>(packed_rk_stride(keys)) * 4 + 128 * 4 + 255) &
         ~static_cast<size_t>(255);
}

int64_t packed_blocks(int64_t tokens, int batch, int G, int Hkv) { return (tokens / (128 / G) + batch) * Hkv; }

cudaError_t launch_packed_prefill(int mode, int G, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                  const CUtensorMap &tm_v, const PackedPrefillParams &p, float *rk, int sm_count,
                                  cudaStream_t stream) {
  if (p.blocks == 0) return cudaSuccess;
  if (mode == kPackedRelu2 && p.keys > 0) {
    const int64_t rows = p.keys * p.Hkv;
    cudaError_t e = launch_pdl(packed_knorm_kernel, dim3(static_cast<unsigned>((rows + 31) / 32)), dim3(256), 0, stream,
                               0u, p, rk);
    if (e != cudaSuccess) return e;
  }
  const int ctas = static_cast<int>(p.blocks < sm_count ? p.blocks : sm_count);
  if (mode == kPackedRelu2) {
    if (G == 4) return launch_packed<kPackedRelu2, 128, 4>(tm_q, tm_k, tm_v, p, ctas, stream);
    if (G == 8) return launch_packed<kPackedRelu2, 128, 8>(tm_q, tm_k, tm_v, p, ctas, stream);
    return cudaErrorInvalidValue;
  }
  if (G == 4) return launch_packed<kPackedSoftmax, 128, 4>(tm_q, tm_k, tm_v, p, ctas, stream);
  if (G == 8) return launch_packed<kPackedSoftmax, 128, 8>(tm_q, tm_k, tm_v, p, ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace embla
