// Full-layer (ReLU^2) decode of a batch whose sequences share one prefix: the prefix's keys
// are held once and read once for the whole batch, each sequence's own keys follow them.
//
// Source: "The Architecture of Embla 1", "Sevren Sparse Attention learns to be sparse" and
// "Three kinds of attention" (the weights, the normaliser and the score the selection ranks
// are those of the full-layer decode).  With q^, k^ the RMS-normalised rows and
// s' = q^ . k^, a query head's weights are w' = max(s', 0)^2 and
//   out = sum_j w'_j v_j / (c / alpha^2 + sum_j w'_j)
// over the prefix's keys and the sequence's own: sums over keys add, so pieces of the key
// axis give partial sums (records) that a second kernel adds in a fixed order.
//
// One KV head's queries of 128 / G sequences make one 128-row operand, so every key tile is
// a dense product for all of them:
//   S  = Q K^T   (M 128 query rows x N 128 keys, fp32 in tensor memory)
//   O += P V     (P = w' as two bf16 matrices hi + lo, about 17 bits of weight, in tensor
//                memory over S; V as the cached rows lie)
// A tile of a sequence's own keys runs through the same operands with every other sequence's
// weights zero.  Value tiles are read whole: a prefix key is dead for all of 128 rows far too
// rarely to skip (0.95^128), and fetching an own tile's live rows alone would put another trip to
// memory between its scores and its products.
//
// Weights reach the value product as hi + lo, two bf16 roundings: 2.5e-6 of the output against
// 64 bits (4.9e-6 at 40 tiles per CTA, see kMaxTiles).  A third part would cost half as many products
// again and 64 more tensor-memory columns per tile than there are.  Denominators, scores and the
// sums over records are fp32.
//
// Work split: one CTA per SM, each one piece of a row block's tile list; the CTAs of different row
// blocks walk the same prefix tiles at the same time, so the prefix comes from HBM once.
//
// Warp roles: 0 TMA producer of K (two tiles); 1 issuer of S; 2 issuer of P V; 3 TMA producer of
// the query rows and of V (two tiles; its waits do not hold up K); 4-7 key norms, one thread per key; 8-23 epilogue, two groups of eight warps on alternate tiles, each warp a
// quarter of the query rows and half of the tile's keys.  The epilogue reads S in the fragment
// layout of the warp MMAs, where a thread holds rows l, l + 8, l + 16 and l + 24 of its quarter,
// and the query rows lie in the block so that those are heads of one sequence: the group maximum
// that the selection ranks is taken within a thread (by shuffles it cost two and a half
// instructions per score on the pipe that bound the epilogue).
//
// What bounds it (clock stamps): up to 128 query rows HBM, 64 KB of K and V per tile in about
// 2,800 cycles against 2,250 for the epilogue and 1,536 for the products; with more row blocks HBM
// and the epilogue (sixteen warps, about 1,400 instructions per tile and scheduler) together: at
// B 64 the CTAs leave 52 to 58 us after the first load, 336 MB read and written.  The fixed
// part of a call is about 9 us: 2 until the first tile lands, 2.5 from a tile's landing to its
// products, 1.5 for writing the records (10 MB at once), 2 to 3 for the finishing kernel.  Measured,
// a call in a graph of calls: B 32, GQA 4, 32k prefix, 300 own keys 29.1 us (97 MB needed, 3.3
// TB/s); B 8, GQA 8, 32k 16.2 us; B 64, 64k, 1,024 own 75.6 us (285 MB, 3.8 TB/s; 11 us of it the
// histogram's reading of 68 MB of scores, most of which L2 no longer holds, stored evict_last or
// not).  Without scores and histogram: 25.0, 15.6 and 61.0 us.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "ptx_blocks.cuh"
#include "shared_prefix.h"

namespace embla {
namespace {

constexpr int kRows = 128;               // query rows of a row block
constexpr int kRing = 3;                 // key norms and S/P buffers
constexpr int kStages = 2;               // K stages, V stages (three of each: within 3 % either way)
constexpr int kWarpPV = 2;
constexpr int kWarpV = 3;
constexpr int kWarpNorm = 4;             // first of the key-norm warps
constexpr int kNormWarps = 4;
constexpr int kWarpEpi = kWarpNorm + kNormWarps;
constexpr int kEpiWarps = 16;
constexpr int kParts = kEpiWarps / 4;    // epilogue warps of a quarter of the rows
constexpr int kPartCols = 128 / kParts;  // columns of O that each of them takes at the end
// The epilogue's two groups of eight warps take alternate tiles, so that one group's waits and
// memory accesses overlap the other's arithmetic (one group of sixteen on every tile: 79.3 us
// against 75.5 at B 64 with a 64k prefix, the same at shorter ones).
constexpr int kGroups = 2;
constexpr int kSThreads = (kWarpEpi + kEpiWarps) * 32;
constexpr int kBox = 128 * 128;          // one [128 rows][64 bf16] box, 16 KB
constexpr int kTileB = 2 * kBox;         // a 128 x 128 bf16 tile
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kTileB;
constexpr int kOffV = kOffK + kStages * kTileB;
constexpr int kOffRK = kOffV + kStages * kTileB;
constexpr int kOffBar = kOffRK + kRing * kRows * 4;
constexpr int kNBars = 1 + 2 * kStages + 3 * kRing + 3;
constexpr int kOffMisc = kOffBar + kNBars * 8;
constexpr int kSSmem = kOffMisc + 32 + 1024;  // + room to align the base to 1024
static_assert(kSSmem <= 227 * 1024, "shared memory per CTA");
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128) | (1u << 16);  // B (V) MN-major
constexpr int kColO = kRing * 128, kTmemCols = 512;

// A record, the sums of one KV head's tiles in one piece: the numerators of 128 rows, each row's
// denominator and each sequence's survivor count for each quarter of the tiles' keys.
constexpr int kRecNum = kRows * kHeadDim;
constexpr int kRecDen = kParts * kRows;
constexpr int kRecCnt = kParts * 32;
constexpr int kRecWords = kRecNum + kRecDen + kRecCnt;
static_assert(kRecWords % 8 == 0, "records keep 32-byte alignment");

struct SharedParams {
  SharedSplit sp;
  float *rec;
  uint32_t *flags;
  float *sel;              // [B, Hkv, score_stride] or null
  uint32_t *hist;          // [B, Hkv, 2048] and n_surv [B, Hkv]: zeroed here when there are scores
  int32_t *n_surv;
  int64_t score_stride;
  int32_t pair_prefix, pair_own;  // score rows of prefix / own tiles start on 8 bytes
  float alpha, eps;
};

// Two fp32 lanes at once, each rounded as the scalar operation would be: half the instructions.
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// The largest of three; NaN counts as absent.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The tensor cores add to an fp32 accumulator by cutting the sum off, not rounding it: values of one
// sign lose 4.5e-7 of their sum per tile (measured: 1.3e-5 after 32 tiles, 1.15e-3 after 2,048).  So the
// sum in tensor memory ends after kMaxTiles tiles and goes to the record, where the next one is
// added with a rounding of its own: at most 2.9e-5 for a prefix of any length, at 5 us every 64
// tiles (2,048 tiles per CTA: 2.32 ms, in one sum 2.16; B 64 with a 64k prefix has 40 and ends
// nowhere: 75.5 us, with 32 tiles at most 79.7).
constexpr int kMaxTiles = 64;

// A CTA's part of the work: a piece of row block rb's tile list, taken in stretches of at most
// kMaxTiles tiles of one KV head's list.
struct Walk {
  int rb, nb;        // the row block, its sequences
  uint32_t gt;       // tiles per KV head
  uint32_t t, end;   // the next tile, the piece's end
  int piece;
  int g, t0, t1;     // stretch: KV head, tiles [t0, t1) of its list
  int s0;            // the first tile of the head's list in this piece
  __device__ Walk(const SharedSplit &sp, int cta) {
    g = -1;
    rb = sp.block_of_cta(cta);
    piece = cta - rb * sp.ctas_full;
    nb = sp.sequences(rb);
    gt = static_cast<uint32_t>(sp.group_tiles(rb));
    const uint32_t T = gt * sp.Hkv, Q = static_cast<uint32_t>(sp.pieces(rb));
    t = sp.piece_start(piece, T, Q);
    end = sp.piece_start(piece + 1, T, Q);
  }
  __device__ bool next() {
    if (t >= end) return false;
    const int head = static_cast<int>(t / gt);
    t0 = static_cast<int>(t - head * gt);
    if (head != g) g = head, s0 = t0;
    uint32_t m = gt - t0 < end - t ? gt - t0 : end - t;
    if (m > kMaxTiles) m = kMaxTiles;
    t1 = t0 + static_cast<int>(m);
    t += m;
    return true;
  }
};

__device__ __forceinline__ void give_up(volatile int *abort_flag, uint32_t *flags) {
  *abort_flag = 1;
  atomicOr(flags, kFlagWaitTimeout);
}

// Row of the block that holds head h of sequence seq: a quarter of 32 rows holds 32 / G
// sequences; head h lies in the quarter's eight rows number h / (G / 4), where a sequence has
// G / 4 rows.
template <int G>
__host__ __device__ constexpr int block_row(int seq, int h) {
  constexpr int kSeqsQ = 32 / G, kHeads8 = G / 4;
  return seq / kSeqsQ * 32 + h / kHeads8 * 8 + seq % kSeqsQ * kHeads8 + h % kHeads8;
}

// Weights are carried as (s' / 128)^2: |s'| <= 128 (two rows of mean square 1), so the clamp of
// a saturating product is the maximum with 0.
constexpr float kWeightScale = 128.0f * 128.0f;

// SCORES: every key's group maximum is written out (and the survivors are counted from those by
// the next kernel, as the histogram is); without, the survivors are counted here.
template <int G, bool SCORES>
__global__ void __launch_bounds__(kSThreads, 1)
    shared_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kp,
                         const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_ko,
                         const __grid_constant__ CUtensorMap tm_vo, const SharedParams p) {
  constexpr int kSeqs = kRows / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem + kOffQ;
  uint8_t *sK = smem + kOffK;
  uint8_t *sV = smem + kOffV;
  float *sRK = reinterpret_cast<float *>(smem + kOffRK);
  uint64_t *qfull = reinterpret_cast<uint64_t *>(smem + kOffBar);
  uint64_t *kfull = qfull + 1;
  uint64_t *vfull = kfull + kStages;
  uint64_t *sfull = vfull + kStages;   // S done and the key norms taken: the K stage is free
  uint64_t *pfull = sfull + kRing;
  uint64_t *pvdone = pfull + kRing;  // P V done: the V stage, S/P buffer and norms are free
  uint64_t *ofull = pvdone + kRing;  // a stretch's P V all done
  uint64_t *qempty = ofull + 1;      // its query rows no longer needed
  uint64_t *ofree = qempty + 1;      // its O read out of tensor memory
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + kOffMisc);
  uint32_t *s_tmem = misc;
  volatile int *s_abort = reinterpret_cast<volatile int *>(misc + 1);
  volatile int *s_kissued = reinterpret_cast<volatile int *>(misc + 2);  // K tile loads issued
  volatile int *s_vissued = reinterpret_cast<volatile int *>(misc + 3);  // V tile loads issued
  volatile int *s_qissued = reinterpret_cast<volatile int *>(misc + 4);  // query loads issued

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SharedSplit &sp = p.sp;
  const int tp = static_cast<int>(sp.tp), ts = static_cast<int>(sp.ts);  // prefix, own tiles

  if (warp == 0) {
    if (lane < kStages) {
      mbar_init(&kfull[lane], 1);
      mbar_init(&vfull[lane], 1);
    }
    if (lane < kRing) {
      mbar_init(&sfull[lane], 1 + kNormWarps);  // the S issuer's commit and the norms
      mbar_init(&pfull[lane], kEpiWarps / kGroups);
      mbar_init(&pvdone[lane], 1);
    }
    if (lane == 0) {
      mbar_init(qfull, 1);
      mbar_init(ofull, 1);
      mbar_init(qempty, 1 + kEpiWarps);  // the S issuer's commit + every epilogue warp
      mbar_init(ofree, kEpiWarps);
      *s_abort = 0;
      *s_kissued = 0;
      *s_vissued = 0;
      *s_qissued = 0;
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kWarpV * 32) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_ko);
    tma_prefetch_desc(&tm_vo);
  }
  Walk w(sp, static_cast<int>(blockIdx.x));
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);

  // Every role waits for the kernels before this one (pdl_wait_primary) by itself, with its first
  // addresses at hand, and before any wait that has a time limit: a kernel that runs long ahead
  // of this one is not a timeout here.  Every role walks the CTA's stretches in the
  // same order, and their tiles through the rings by a running tile count i: K and V stage
  // i % kStages, S/P buffer i % kRing, each in its ring's phase.  Stretch k's query and output
  // barriers take phase k & 1.

  // where tile t of the walk's stretch lies (own keys or the prefix's): the plane and the row
  auto place = [&](int t, int &plane, int &row) {
    const bool own = t >= tp;
    const int x = t - tp;
    row = (own ? x % ts : t) * kTileKeys;
    plane = own ? (w.rb * kSeqs + x / ts) * sp.Hkv + w.g : w.g;
    return own;
  };
  // L2: rows that one CTA reads go first; the prefix's stay for the other row blocks, if any
  const uint64_t once = policy_evict_first(), shared = sp.blocks > 1 ? policy_evict_normal() : once;
  if (warp == 0) {
    // ------------------------------------------------------------------ K producer
    if (lane == 0) {
      int i = 0;
      bool ok = true;
      while (ok && w.next()) {
#pragma unroll 1
        for (int t = w.t0; t < w.t1; ++t, ++i) {
          const int s = i % kStages;
          int plane, row;
          const bool own = place(t, plane, row);
          const CUtensorMap *map = own ? &tm_ko : &tm_kp;
          if (i == 0) pdl_wait_primary();
          if (i >= kStages && !mbar_wait(&sfull[(i - kStages) % kRing], ((i - kStages) / kRing) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&kfull[s], kTileB);
          tma_load_3d_hint(sK + s * kTileB, map, &kfull[s], 0, row, plane, own ? once : shared);
          tma_load_3d_hint(sK + s * kTileB + kBox, map, &kfull[s], 64, row, plane, own ? once : shared);
          *s_kissued = i + 1;
        }
      }
      if (!ok) give_up(s_abort, p.flags);
    }
    __syncwarp();
  } else if (warp == kWarpV) {
    // ------------------------------------------------------------------ query and V producer
    if (lane == 0) {
      int i = 0;
      bool ok = true;
      for (int k = 0; ok && w.next(); ++k) {
        if (k > 0 && !mbar_wait(qempty, (k - 1) & 1)) {
          ok = false;
          break;
        }
        if (k == 0) pdl_wait_primary();
        mbar_arrive_expect_tx(qfull, kTileB);
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {  // a quarter of the rows at a time (block_row)
          const int seq = w.rb * kSeqs + e * (32 / G);
          tma_load_5d(sQ + e * 4096, &tm_q, qfull, 0, 0, seq, 0, w.g);
          tma_load_5d(sQ + kBox + e * 4096, &tm_q, qfull, 64, 0, seq, 0, w.g);
        }
        *s_qissued = k + 1;
#pragma unroll 1
        for (int t = w.t0; t < w.t1; ++t, ++i) {
          const int s = i % kStages;
          int plane, row;
          const bool own = place(t, plane, row);
          const CUtensorMap *map = own ? &tm_vo : &tm_vp;
          if (i >= kStages && !mbar_wait(&pvdone[(i - kStages) % kRing], ((i - kStages) / kRing) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&vfull[s], kTileB);
          tma_load_3d_hint(sV + s * kTileB, map, &vfull[s], 0, row, plane, own ? once : shared);
          tma_load_3d_hint(sV + s * kTileB + kBox, map, &vfull[s], 64, row, plane, own ? once : shared);
          *s_vissued = i + 1;
        }
      }
      if (!ok) give_up(s_abort, p.flags);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S issuer
    // The warp walks together and one lane issues (elect_one).
    const uint64_t qdesc = smem_desc_sw128(smem_u32(sQ));
    const uint64_t kdesc = smem_desc_sw128(smem_u32(sK));
    int i = 0, done = 0;
    bool ok = true;
    pdl_wait_primary();
    for (int k = 0; ok && w.next(); ++k) {
      ok = __all_sync(0xffffffffu, !*s_abort && mbar_wait(qfull, k & 1));
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++i) {
        const int s = i % kRing;
        ok = mbar_wait(&kfull[i % kStages], (i / kStages) & 1) &&
             (i < kRing || mbar_wait(&pvdone[s], ((i / kRing) - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // dims 16kk..16kk+15: 32 bytes into a 128-byte row; dims 64.. start the second box
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kBox + (kk & 3) * 32) >> 4);
            tc_mma_bf16(tmem + s * 128, qdesc + off, kdesc + static_cast<uint64_t>((i % kStages * kTileB) >> 4) + off,
                        kIdescS, kk > 0 ? 1u : 0u);
          }
          tc_commit(&sfull[s]);
        }
        __syncwarp();
      }
      if (ok) {
        if (elect_one()) tc_commit(qempty);
        __syncwarp();
        done = k + 1;
      }
    }
    if (!ok && lane == 0) give_up(s_abort, p.flags);
    // every MMA of this warp has completed, and its last commit arrived, before the tensor memory
    // is released and the CTA leaves (also when another role has given up)
    if (i > 0) mbar_wait(&sfull[(i - 1) % kRing], ((i - 1) / kRing) & 1);
    if (done > 0) mbar_wait(qempty, (done - 1) & 1);
    __syncwarp();
  } else if (warp == kWarpPV) {
    // ------------------------------------------------------------------ P V issuer
    const uint64_t vdesc = smem_desc_sw128_mn(smem_u32(sV), kBox);
    int i = 0, done = 0;
    bool ok = true;
    pdl_wait_primary();
    for (int k = 0; ok && w.next(); ++k) {
      ok = __all_sync(0xffffffffu, !*s_abort && (k == 0 || mbar_wait(ofree, (k - 1) & 1)));
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++i) {
        const int s = i % kRing;
        ok = mbar_wait(&pfull[s], (i / kRing) & 1) && mbar_wait(&vfull[i % kStages], (i / kStages) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // keys 16kk..16kk+15: in their group of 16 columns hi takes the first 8, lo the rest
            const uint32_t a_hi = tmem + s * 128 + kk * 16;
            const uint64_t vd = vdesc + static_cast<uint64_t>((i % kStages * kTileB + kk * 2048) >> 4);
            tc_mma_bf16_tmem_a(tmem + kColO, a_hi, vd, kIdescPV, (t > w.t0 || kk > 0) ? 1u : 0u);
            tc_mma_bf16_tmem_a(tmem + kColO, a_hi + 8, vd, kIdescPV, 1u);
          }
          tc_commit(&pvdone[s]);
        }
        __syncwarp();
      }
      if (ok) {
        if (elect_one()) tc_commit(ofull);
        __syncwarp();
        done = k + 1;
      }
    }
    if (!ok && lane == 0) give_up(s_abort, p.flags);
    // every MMA of this warp has completed before the tensor memory is released
    if (done > 0) mbar_wait(ofull, (done - 1) & 1);
    __syncwarp();
  } else if (warp < kWarpEpi) {
    // ------------------------------------------------------------------ key norms
    const int r = (warp - kWarpNorm) * 32 + lane;  // this thread's key of every tile
    int i = 0;
    bool ok = true;
    pdl_wait_primary();
    while (ok && w.next()) {
#pragma unroll 1
      for (int t = w.t0; ok && t < w.t1; ++t, ++i) {
        const int s = i % kRing;
        ok = mbar_wait(&kfull[i % kStages], (i / kStages) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float rk = rsqrtf(row_square_sum(sK + i % kStages * kTileB, kBox, r, r & 7) * (1.0f / kHeadDim) + p.eps);
        ok = i < kRing || mbar_wait(&pvdone[s], ((i / kRing) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        sRK[s * kRows + r] = rk;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[s]);
      }
    }
    if (!ok && lane == 0) give_up(s_abort, p.flags);
    // the counts that the next kernel adds up start at zero
    if constexpr (SCORES) {
      uint4 *h = reinterpret_cast<uint4 *>(p.hist);
      const int64_t n4 = static_cast<int64_t>(sp.B) * sp.Hkv * (kHistBins / 4);
#pragma unroll 1
      for (int64_t e = static_cast<int64_t>(blockIdx.x) * kRows + r; e < n4; e += static_cast<int64_t>(gridDim.x) * kRows)
        h[e] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
      for (int64_t e = static_cast<int64_t>(blockIdx.x) * kRows + r; e < static_cast<int64_t>(sp.B) * sp.Hkv;
           e += static_cast<int64_t>(gridDim.x) * kRows)
        p.n_surv[e] = 0;
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3;            // the tensor-memory lanes this warp may read
    const int part = (warp - kWarpEpi) >> 2;
    const int group = part >> 1;
    const int first_key = (part & 1) * 64;   // of the group's tiles this warp takes 64 keys
    const int q4 = lane & 3;                 // columns 8j + 2 q4, + 1 of those
    constexpr int kSeqsQ = 32 / G;           // sequences of a quarter
    const int seq = quarter * kSeqsQ + (lane >> 2) / (G / 4);  // this thread's sequence
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t part_col = static_cast<uint32_t>(part * kPartCols);
    // this lane's key of each pair of scores (groups of 8 end up split over two lanes)
    const int odd = G == 8 ? (lane >> 2) & 1 : 0;
    int i = 0;
    bool ok = true;
    pdl_wait_primary();
    pdl_launch_dependents();
    for (int k = 0; ok && w.next(); ++k) {
      ok = !*s_abort && mbar_wait(qfull, k & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float rq[4], den[4][2];
      int live = 0;  // keys of this thread's share with a group maximum above zero
#pragma unroll
      for (int m = 0; m < 4; ++m) den[m][0] = den[m][1] = 0.0f;
      // 1 / rms of the thread's four rows: each lane takes one of its four lanes' rows
      {
        const float ss = row_square_sum(sQ, kBox, quarter * 32 + (lane >> 2) + 8 * q4, (lane & 3) * 2 + ((lane >> 2) & 1));
        const float mine = rsqrtf(ss * (1.0f / kHeadDim) + p.eps);
#pragma unroll
        for (int m = 0; m < 4; ++m) rq[m] = __shfl_sync(0xffffffffu, mine, (lane & ~3) | m);
        // the query rows are read: every lane's sum depends on them
        const float used = __shfl_sync(0xffffffffu, ss, 0) + __shfl_sync(0xffffffffu, ss, 31);
        __syncwarp();
        if (lane == 0) mbar_arrive_after(qempty, used);
      }
      const bool valid = seq < w.nb;
      const bool some = quarter * kSeqsQ < w.nb;  // this warp has valid rows
      // this thread's (sequence, KV head)'s scores, at its first key
      float *scores = SCORES && valid ? p.sel + (static_cast<int64_t>(w.rb * kSeqs + seq) * sp.Hkv + w.g) *
                                                    p.score_stride + 2 * q4 + odd
                                      : nullptr;
      // this group's tiles: every other one of the running count
      const int skip = (group - i) & 1;
      for (int t = w.t0 + skip, it = i + skip; t < w.t1; t += kGroups, it += kGroups) {
        const int s = it % kRing;
        ok = mbar_wait(&sfull[s], (it / kRing) & 1);
        ok = __all_sync(0xffffffffu, ok);  // the warp works on the tile together or not at all
        if (!ok) break;
        const bool own = t >= tp;
        const int x = t - tp;
        const int owner = own ? x / ts : seq;
        if (!own ? some : owner / kSeqsQ == quarter) {
          tc_fence_after_sync();
          // another sequence's keys weigh nothing here
          const float f = seq == owner ? 1.0f / 128.0f : 0.0f;
          // the tile's first key in the score row, and how many keys it has
          const int kt = own ? x - owner * ts : t;
          const int rest = static_cast<int>(own ? sp.n : sp.P) - kt * kTileKeys;
          const bool reads = valid && seq == owner;
          const bool pairs = rest >= kTileKeys && (G == 8 || (own ? p.pair_own : p.pair_prefix));
          float *dst = scores + (own ? sp.P : 0) + static_cast<int64_t>(kt) * kTileKeys;
          const uint32_t stage = tmem + lane_base + s * 128;
          const float *rkp = sRK + s * kRows + 2 * q4;
          float top[4];  // the maximum over this thread's four heads for its four of 16 keys
          // Sixteen keys of rows l / 4 + 16 side and + 8: weights, P, the maximum so far.
          auto rows16 = [&](const uint32_t (&acc)[8], const float2 (&rks)[2], int col, auto which) {
            constexpr int side = decltype(which)::value;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 rk = rks[j];
              float s0 = 0.0f, s1 = 0.0f;  // the first of the two rows' scores
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                float v0 = __uint_as_float(acc[4 * j + 2 * m]), v1 = __uint_as_float(acc[4 * j + 2 * m + 1]);
                mul2(v0, v1, rk.x, rk.y);
                mul2(v0, v1, rq[2 * side + m], rq[2 * side + m]);
                if (m == 0) {
                  s0 = v0, s1 = v1;
                } else {
                  // from minus infinity: a key whose score is NaN for every head ranks last
                  top[2 * j] = max3(side == 0 ? -INFINITY : top[2 * j], s0, v0);
                  top[2 * j + 1] = max3(side == 0 ? -INFINITY : top[2 * j + 1], s1, v1);
                }
                float w0 = __saturatef(v0 * f), w1 = __saturatef(v1 * f);
                mul2(w0, w1, w0, w1);
                add2(den[2 * side + m][0], den[2 * side + m][1], w0, w1);
                // the weights over the scores' columns: 8 columns of hi, then 8 of lo
                const uint32_t b = pack_bf16x2(w0, w1);
                sub_bf16x2(b, w0, w1);
                hi[2 * j + m] = b;
                lo[2 * j + m] = pack_bf16x2(w0, w1);
              }
            }
            tmem_store_16x128b_x2(stage + col + (side * 16u << 16), hi);
            tmem_store_16x128b_x2(stage + col + (side * 16u << 16) + 8, lo);
          };
          // Those keys' maxima over the whole group: counted and written out.
          auto group_scores = [&](int col) {
            if constexpr (G == 8) {
              // the other four heads are the lane's across: each keeps one key of every pair
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float give = odd ? top[2 * j] : top[2 * j + 1];
                const float keep = odd ? top[2 * j + 1] : top[2 * j];
                top[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 4));
              }
            }
            constexpr int kEach = G == 8 ? 1 : 2;  // keys of every 8 that this thread keeps
            if constexpr (!SCORES) {
#pragma unroll
              for (int e = 0; e < 2 * kEach; ++e) live += reads && top[e] > 0.0f ? 1 : 0;
            } else if (pairs) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if constexpr (G == 8)
                  st_global_if(reads, dst + col + 8 * j, p.alpha * top[j]);
                else
                  st_global_v2_if(reads, dst + col + 8 * j, p.alpha * top[2 * j], p.alpha * top[2 * j + 1]);
              }
            } else {
              const int room = rest - col - 2 * q4 - odd;
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                  st_global_if(reads && 8 * j + e < room, dst + col + 8 * j + e, p.alpha * top[kEach * j + e]);
            }
          };
          // each load is on its way while the rows before it are worked on
          uint32_t a[8], b[8];
          const int col0 = first_key, col1 = col0 + 64;
          tmem_load_16x256b_x2(stage + col0, a);
          float2 rks[2] = {*reinterpret_cast<const float2 *>(rkp + col0),
                           *reinterpret_cast<const float2 *>(rkp + col0 + 8)};
#pragma unroll 1
          for (int col = col0; col < col1; col += 16) {
            tmem_wait_ld(a);
            tmem_load_16x256b_x2(stage + col + (16u << 16), b);
            rows16(a, rks, col, std::integral_constant<int, 0>{});
            tmem_wait_ld(b);
            const int next = col + 16 < col1 ? col + 16 : col0;  // past the last: read, not used
            tmem_load_16x256b_x2(stage + next, a);
            rows16(b, rks, col, std::integral_constant<int, 1>{});
            rks[0] = *reinterpret_cast<const float2 *>(rkp + next);
            rks[1] = *reinterpret_cast<const float2 *>(rkp + next + 8);
            group_scores(col);
          }
          tmem_wait_ld(a);
          tmem_wait_st();
          tc_fence_before_sync();  // P is read by the tensor cores
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[s]);
        } else {
          // no row of this warp reads the tile: zero weights for rows that other tiles count
          // for (rows past the batch hold anything, no other row sees them)
          if (some) {
            tc_fence_after_sync();
            const uint32_t zero[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            for (int c = 0; c < 64; c += 16) tmem_store_x16(tmem + lane_base + s * 128 + first_key + c, zero);
            tmem_wait_st();
            tc_fence_before_sync();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[s]);
        }
      }
      i += w.t1 - w.t0;
      if (!ok) break;
      ok = mbar_wait(ofull, k & 1) && !*s_abort;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t o[kPartCols];
      tmem_load_x32(tmem + lane_base + kColO + part_col, o);
      tmem_wait_ld(o);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);  // the next stretch's P V may overwrite O
      // The record: every row when the stretch holds prefix tiles, else the rows of the
      // sequences whose tiles it holds.
      const int first_seq = w.t0 < tp ? 0 : (w.t0 - tp) / ts;
      const int last_seq = w.t0 < tp ? w.nb - 1 : (w.t1 - 1 - tp) / ts;
      // its four rows' weight sums and (without scores) its sequence's count, over the lanes that
      // share them
      if constexpr (!SCORES) {
        live += __shfl_xor_sync(0xffffffffu, live, 1);
        live += __shfl_xor_sync(0xffffffffu, live, 2);
        if constexpr (G == 8) live += __shfl_xor_sync(0xffffffffu, live, 4);
      }
      float dsum = 0.0f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float d = den[m][0] + den[m][1];
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        if (m == q4) dsum = d;
      }
      float *rec = p.rec + sp.slot(w.rb, w.piece, w.g) * kRecWords;
      float *rec_den = rec + kRecNum + part * kRows + quarter * 32 + (lane >> 2) + 8 * q4;
      int32_t *rec_cnt = reinterpret_cast<int32_t *>(rec) + kRecNum + kRecDen + part * 32 + seq;
      const bool counts = !SCORES && q4 == 0 && odd == 0;
      // the numerators: lane l holds row l of the quarter, of sequence
      const int row_seq = quarter * kSeqsQ + (lane & 7) / (G / 4);
      float *dst = rec + (quarter * 32 + lane) * kHeadDim + part_col;
      const bool den_here = seq >= first_seq && seq <= last_seq, num_here = row_seq >= first_seq && row_seq <= last_seq;
      // the last sequence that earlier stretches of the head's list wrote rows for (-1: none)
      int written = -1;
      if (__builtin_expect(w.t0 != w.s0, 0)) {
        written = w.s0 < tp ? w.nb - 1 : (w.t0 - 1 - tp) / ts;
        // added to those by the same threads, in their order
        if (den_here && seq <= written) {
          atomicAdd(rec_den, dsum);
          if (counts) atomicAdd(rec_cnt, live);
        }
        if (num_here && row_seq <= written)
#pragma unroll
          for (int c = 0; c < kPartCols; c += 4)
            red_global_add_v4(dst + c, __uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]),
                              __uint_as_float(o[c + 3]));
      }
      if (den_here && seq > written) {
        *rec_den = dsum;
        if (counts) *rec_cnt = live;
      }
      if (num_here && row_seq > written) {
#pragma unroll
        for (int c = 0; c < kPartCols; c += 8)
          st_global_v8(dst + c, __uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]),
                       __uint_as_float(o[c + 3]), __uint_as_float(o[c + 4]), __uint_as_float(o[c + 5]),
                       __uint_as_float(o[c + 6]), __uint_as_float(o[c + 7]));
      }
    }
    if (!ok && lane == 0) give_up(s_abort, p.flags);
  }

  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) {
    // No copy may still be landing in shared memory when the CTA leaves.  Without an abort
    // every copy issued was waited for by the role that used it; after one, wait (bounded)
    // for the last armed phase of every barrier that a copy completes.
    const int qi = *s_qissued;
    if (qi > 0) mbar_wait(qfull, (qi - 1) & 1);
    const int nk = *s_kissued, nv = *s_vissued;
#pragma unroll 1
    for (int s = 0; s < kStages; ++s) {
      int uses = nk > s ? (nk - 1 - s) / kStages + 1 : 0;
      if (uses) mbar_wait(&kfull[s], (uses - 1) & 1);
      uses = nv > s ? (nv - 1 - s) / kStages + 1 : 0;
      if (uses) mbar_wait(&vfull[s], (uses - 1) & 1);
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ----------------------------------------------------------------------------- finish

constexpr int kFThreads = 256;
constexpr int kFWarps = kFThreads / 32;
constexpr int kFCtasPerSm = 3;   // registers for ten records in flight per warp
constexpr int kHistStep = 1024;  // a CTA's share of the scores starts at a multiple of this
constexpr int kItemSteps = 12;   // an item's time in steps (with 6, B 32 took 1 us more)

struct FinishParams {
  SharedSplit sp;
  const float *rec;
  const uint16_t *q;
  const uint16_t *kp, *vp, *ko, *vo;
  int64_t prefix_stride, cache_stride;
  const float *sel;
  uint32_t *hist;
  int64_t score_stride;
  // padded scores per CTA: hist_few for the first hist_few_first by rank, hist_many for the others
  int64_t hist_few, hist_many, hist_few_first;
  int32_t hist_vec;                // score rows start on 16 bytes
  int32_t rows;                    // query heads per item: 1 or 2
  float *out;
  int32_t *n_surv;
  float alpha, c, eps;
};

// A row whose sums are not finite, term by term: the products of a whole value tile give NaN
// where a weight of zero meets a value that is infinite or NaN, and a key of weight zero (or
// another sequence's key) contributes nothing here.  One pass of a CTA over all keys per row, for
// every row whose block met such a value: slow (one NaN row in the prefix: 0.26 ms at B 4 behind 2k keys,
// 5 ms at B 32 behind 32k, 33 ms at B 64 behind 64k), and only for inputs that hold such values.
__device__ __noinline__ void row_term_by_term(const FinishParams &p, int b, int hq, float *s_q, float *s_w,
                                              float *s_sum) {
  const SharedSplit &sp = p.sp;
  const int g = hq / sp.G, tid = threadIdx.x;
  if (tid < kHeadDim)
    s_q[tid] = __uint_as_float(static_cast<uint32_t>(p.q[(static_cast<int64_t>(b) * sp.G * sp.Hkv + hq) * kHeadDim + tid]) << 16);
  __syncthreads();
  float qs = 0.0f;
#pragma unroll 1
  for (int d = 0; d < kHeadDim; ++d) qs = fmaf(s_q[d], s_q[d], qs);
  const float rq = rsqrtf(qs * (1.0f / kHeadDim) + p.eps);
  const int64_t N = sp.P + sp.n;
  const int64_t unit = static_cast<int64_t>(b) * sp.Hkv + g;
  float num = 0.0f, den = 0.0f;  // thread d < 128: dimension d
  for (int64_t j0 = 0; j0 < N; j0 += kFThreads) {
    const int64_t j = j0 + tid;
    float w = 0.0f;
    if (j < N) {
      const uint16_t *kr = j < sp.P ? p.kp + (g * p.prefix_stride + j) * kHeadDim
                                    : p.ko + (unit * p.cache_stride + j - sp.P) * kHeadDim;
      float dot = 0.0f, k0 = 0.0f, k1 = 0.0f;
#pragma unroll 2
      for (int d = 0; d < kHeadDim; d += 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(kr + d);
        dot = fmaf(s_q[d], bf16lo(x), dot);
        dot = fmaf(s_q[d + 1], bf16hi(x), dot);
        sq_acc_bf16x2(x, k0, k1);
      }
      w = fmaxf(dot * rsqrtf((k0 + k1) * (1.0f / kHeadDim) + p.eps) * rq, 0.0f);
      w *= w;
    }
    s_w[tid] = w;
    __syncthreads();
    if (tid < kHeadDim) {
      float a = 0.0f, z = 0.0f;
      const int m = N - j0 < kFThreads ? static_cast<int>(N - j0) : kFThreads;
#pragma unroll 1
      for (int i = 0; i < m; ++i) {
        const float wi = s_w[i];
        if (wi == 0.0f) continue;
        const int64_t ji = j0 + i;
        const uint16_t *vr = ji < sp.P ? p.vp + (g * p.prefix_stride + ji) * kHeadDim
                                       : p.vo + (unit * p.cache_stride + ji - sp.P) * kHeadDim;
        a = fmaf(wi, __uint_as_float(static_cast<uint32_t>(vr[tid]) << 16), a);
        z += wi;
      }
      num += a;
      den += z;
    }
    __syncthreads();
  }
  if (tid < kHeadDim) {
    s_sum[tid] = num;
    if (tid == 0) s_sum[kHeadDim] = den;
  }
  __syncthreads();
}

// The batch's outputs from the records, then the survivors' counts and the selection's histograms
// from the scores: one wave of CTAs, each with its share of both.
template <bool SCORES>
__global__ void __launch_bounds__(kFThreads, kFCtasPerSm) shared_finish_kernel(const FinishParams p) {
  __shared__ __align__(16) uint32_t s_mem[kHistBins];
  const SharedSplit &sp = p.sp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = sp.G * sp.Hkv;
  // An item: one or two query heads' outputs, rows row0 (and row0 + 1, of the same KV head), each
  // by `slices` of the CTA's warps.  The first round has no records and writes nothing: it
  // fetches the code while the decode's last CTAs run.
  const int rows = p.rows, slices = kFWarps / rows, items = sp.B * Hq / rows;
  // Consecutive CTAs share an SM, so the CTA's rank spreads the items over the SMs.
  const int rank = static_cast<int>(blockIdx.x % kFCtasPerSm * (gridDim.x / kFCtasPerSm) + blockIdx.x / kFCtasPerSm);
  int item = rank;
  bool real = false;
#pragma unroll 1
  while (true) {
    const int row0 = (item < items ? item : 0) * rows, row = row0 + warp % rows;
    const int b = row / Hq, hq = row - b * Hq, g = hq / sp.G;
    const int seqs = kRows / sp.G;
    const int rb = b / seqs, seq = b - rb * seqs, h = hq - g * sp.G;
    const int r = sp.G == 4 ? block_row<4>(seq, h) : block_row<8>(seq, h);
    const SharedSplit::RowPieces pc = sp.row_pieces(rb, seq, g);
    const int n1 = pc.prefix, all = n1 + pc.rest;
    const float *first = p.rec + sp.slot(rb, pc.first, g) * kRecWords;
    const int64_t gap = static_cast<int64_t>(pc.own - pc.first - n1) * kRecWords;  // past the prefix's records
    // (twice for the first item: the round without records, then the item)
#pragma unroll 1
    while (true) {
      const int nrec = real ? all : 0;
      // each warp adds every slices-th record, lane l dims 4l .. 4l + 3; then the warps in order
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float den = 0.0f;
      // without scores, the survivors that the decode counted: eight of the warp's records at a time,
      // four lanes (a count each) to a record, the first eight on their way with the sums
      auto counted = [&](int i) {
        const float *rec = first + static_cast<int64_t>(i) * kRecWords + (i < n1 ? 0 : gap);
        return reinterpret_cast<const int32_t *>(rec)[kRecNum + kRecDen + lane % kParts * 32 + seq];
      };
      const int i1 = warp / rows + lane / kParts * slices;
      int live = 0;
      if (!SCORES && i1 < nrec) live = counted(i1);
      constexpr int kBatch = 10;  // records in flight per warp (past the last: read again, not used)
      const int part = lane & (kParts - 1);
#pragma unroll 1
      for (int i0 = warp / rows; i0 < nrec; i0 += kBatch * slices) {
        float4 x[kBatch];
        float xd[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = i0 + e * slices < nrec ? i0 + e * slices : nrec - 1;
          const float *rec = first + static_cast<int64_t>(i) * kRecWords + (i < n1 ? 0 : gap);
          x[e] = *reinterpret_cast<const float4 *>(rec + r * kHeadDim + 4 * lane);
          xd[e] = rec[kRecNum + part * kRows + r];
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          if (i0 + e * slices < nrec) {
            acc.x += x[e].x;
            acc.y += x[e].y;
            acc.z += x[e].z;
            acc.w += x[e].w;
            den += xd[e];
          }
        }
      }
      if constexpr (!SCORES) {
        for (int i = i1 + 32 / kParts * slices; i < nrec; i += 32 / kParts * slices) live += counted(i);
        live = __reduce_add_sync(0xffffffffu, live);
      }
      float *s_acc = reinterpret_cast<float *>(s_mem);                 // [8 warps][128]
      float *s_den = s_acc + kFWarps * kHeadDim;                       // [8][kParts]
      int *s_live = reinterpret_cast<int *>(s_den + kParts * kFWarps);  // [8]
      *reinterpret_cast<float4 *>(s_acc + warp * kHeadDim + 4 * lane) = acc;
      if (lane < kParts) s_den[warp * kParts + lane] = den;
      if (!SCORES && lane == 0) s_live[warp] = live;
      __syncthreads();
      // thread: dimension tid % 128 of the first (tid < 128) or the second row
      const int mine = threadIdx.x / kHeadDim, d = threadIdx.x % kHeadDim;
      float num = 0.0f, dsum = 0.0f;
      int nlive = 0;
      if (mine < rows) {
#pragma unroll 4
        for (int k = mine; k < kFWarps; k += rows) {
          num += s_acc[k * kHeadDim + d];
          const float4 z4 = *reinterpret_cast<const float4 *>(s_den + k * kParts);
          dsum += (z4.x + z4.y) + (z4.z + z4.w);
          if constexpr (!SCORES) nlive += s_live[k];
        }
      }
      static_assert(kParts == 4, "a warp's sums are one vector");
      num *= kWeightScale;
      dsum *= kWeightScale;
      const bool bad = !(fabsf(num) <= 3.402823466e38f);
      if (__syncthreads_or(bad)) {
        float *s_sum = reinterpret_cast<float *>(s_mem);  // [129]
#pragma unroll 1
        for (int k = 0; k < rows; ++k) {
          row_term_by_term(p, b, row0 + k - b * Hq, s_sum + 256, s_sum + 512, s_sum);
          if (mine == k) {
            num = s_sum[d];
            dsum = s_sum[kHeadDim];
          }
          __syncthreads();
        }
      }
      const float z = p.c / p.alpha / p.alpha + dsum;
      if (real && mine < rows) {
        p.out[static_cast<int64_t>(row0 + mine) * kHeadDim + d] = z != 0.0f ? num / z : 0.0f;
        if (!SCORES && threadIdx.x == 0 && h == 0) p.n_surv[static_cast<int64_t>(b) * sp.Hkv + g] = nlive;
      }
      if (real) break;
      pdl_wait_primary();  // the records and scores are complete
      pdl_launch_dependents();
      real = true;
      if (item >= items) break;
    }
    item += static_cast<int>(gridDim.x);
    if (item >= items) break;
  }
  if constexpr (!SCORES) return;

  // The scores of all units one after another, each padded to N4 keys: this CTA's share of them,
  // counted unit by unit in shared memory.
  __syncthreads();
#pragma unroll 1
  for (int e = threadIdx.x; e < kHistBins; e += kFThreads) s_mem[e] = 0u;
  const int64_t N = sp.P + sp.n, N4 = (N + kHistStep - 1) / kHistStep * kHistStep;
  // (CTAs with one more item than others take less of the scores)
  const int64_t more = p.hist_few_first;
  int64_t at = rank < more ? rank * p.hist_few : more * p.hist_few + (rank - more) * p.hist_many;
  const int64_t stop_all = static_cast<int64_t>(sp.B) * sp.Hkv * N4;
  const int64_t share = rank < more ? p.hist_few : p.hist_many;
  const int64_t stop = at + share < stop_all ? at + share : stop_all;
#pragma unroll 1
  while (at < stop) {
    const int64_t u = at / N4, j0 = at - u * N4;
    const int64_t len = N4 - j0 < stop - at ? N4 - j0 : stop - at;
    const int m = static_cast<int>(len < N - j0 ? len : N - j0);  // keys there are
    at += len;
    const float *su = p.sel + u * p.score_stride + j0;
    __syncthreads();  // the bins are zero
    int live = 0;
    auto count = [&](float x) {
      live += x > 0.0f ? 1 : 0;
      // order_key(x) >> 21: the top bits of a positive score, the inverted ones of a negative
      const int t = __float_as_int(x + 0.0f) >> 21;  // (-0 counts as 0)
      atomicAdd(&s_mem[t ^ (t >> 31 | kHistBins / 2)], 1u);
    };
    if (p.hist_vec) {
      const float4 *s4 = reinterpret_cast<const float4 *>(su);
      constexpr int kLoads = 8;  // in flight per thread (B 64, 64k: 75.5 us; 4: 77.4, 12 and a second batch ahead: no faster)
      const int m4 = m / 4;
#pragma unroll 1
      for (int e = threadIdx.x; e < m4; e += kLoads * kFThreads) {
        float4 x[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
          if (e + k * kFThreads < m4) x[k] = s4[e + k * kFThreads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
          if (e + k * kFThreads < m4) count(x[k].x), count(x[k].y), count(x[k].z), count(x[k].w);
      }
      if (static_cast<int>(threadIdx.x) < m % 4) count(su[m4 * 4 + threadIdx.x]);
    } else {
#pragma unroll 4
      for (int e = threadIdx.x; e < m; e += kFThreads) count(su[e]);
    }
    live = __reduce_add_sync(0xffffffffu, live);
    if (lane == 0 && live != 0) atomicAdd(&p.n_surv[u], live);
    __syncthreads();
#pragma unroll 2
    for (int k = threadIdx.x; k < kHistBins; k += kFThreads)
      if (s_mem[k] != 0u) {
        atomicAdd(&p.hist[u * kHistBins + k], s_mem[k]);
        s_mem[k] = 0u;
      }
  }
}

}  // namespace

SharedSplit shared_split(int B, int Hkv, int G, int64_t P, int64_t n, int sm_count) {
  SharedSplit sp = {};
  sp.P = P;
  sp.n = n;
  sp.B = B;
  sp.Hkv = Hkv;
  sp.G = G;
  sp.tp = (P + kTileKeys - 1) / kTileKeys;
  sp.ts = (n + kTileKeys - 1) / kTileKeys;
  const int seqs = kRows / G;
  sp.blocks = (B + seqs - 1) / seqs;
  if (sp.blocks == 0 || sp.tp + sp.ts == 0) return sp;
  // CTAs per row block in proportion to its tiles: as many as fit the SMs, one at least
  const int64_t full = sp.group_tiles(0) * Hkv, last = sp.group_tiles(sp.blocks - 1) * Hkv;
  int64_t cf = sm_count / (sp.blocks > 1 ? sp.blocks - 1 : 1);
  if (cf > full) cf = full;
  int64_t cl = 1;
  for (; cf >= 1; --cf) {
    cl = (cf * last + full - 1) / full;
    if (cl > last) cl = last;
    if ((sp.blocks - 1) * cf + cl <= sm_count) break;
  }
  if (cf < 1) {
    cf = 1;
    cl = 1;
  }
  sp.ctas_full = static_cast<int32_t>(cf);
  sp.ctas_last = static_cast<int32_t>(cl);
  return sp;
}

size_t shared_workspace_bytes(const SharedSplit &sp) {
  if (sp.ctas() == 0) return 0;
  // + room to align the records to 32 bytes
  return static_cast<size_t>(sp.slot(sp.blocks, 0, 0)) * kRecWords * 4 + 16;
}

// The kernel's shared-memory limit is a setting of the device's context: made by the first call
// on a device (or by several at once, to the same value).
template <class Kernel>
cudaError_t allow_smem_once(const SharedCall &a, Kernel kernel) {
  static std::atomic<uint64_t> done[4];  // by kernel: head groups x scores; a bit per device
  const int which = (a.group == 8 ? 2 : 0) + (a.sel_scores != nullptr ? 1 : 0);
  const uint64_t bit = uint64_t{1} << a.device;
  if (done[which].load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSSmem);
  if (e == cudaSuccess) done[which].fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_shared_decode(const SharedCall &a, const SharedSplit &sp, cudaStream_t stream) {
  SharedParams p;
  p.sp = sp;
  p.rec = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(a.workspace) + 31u) & ~uintptr_t{31});
  p.flags = a.flags;
  p.sel = a.sel_scores;
  p.hist = a.sel_hist;
  p.score_stride = a.score_stride;
  p.pair_prefix = a.score_stride % 2 == 0;
  p.pair_own = p.pair_prefix && sp.P % 2 == 0;
  p.alpha = a.alpha;
  p.eps = a.eps;
  p.n_surv = a.n_surv;
  auto kernel = a.sel_scores != nullptr ? (sp.G == 4 ? shared_decode_kernel<4, true> : shared_decode_kernel<8, true>)
                                        : (sp.G == 4 ? shared_decode_kernel<4, false> : shared_decode_kernel<8, false>);
  cudaError_t e = allow_smem_once(a, kernel);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(sp.ctas())), dim3(kSThreads), static_cast<size_t>(kSSmem),
                 stream, 0u, *a.tm_q, *a.tm_kp, *a.tm_vp, *a.tm_ko, *a.tm_vo, p);
  if (e != cudaSuccess) return e;
  FinishParams f;
  f.sp = sp;
  f.rec = p.rec;
  f.q = static_cast<const uint16_t *>(a.q);
  f.kp = static_cast<const uint16_t *>(a.k_prefix);
  f.vp = static_cast<const uint16_t *>(a.v_prefix);
  f.ko = static_cast<const uint16_t *>(a.k_cache);
  f.vo = static_cast<const uint16_t *>(a.v_cache);
  f.prefix_stride = a.prefix_stride;
  f.cache_stride = a.cache_stride;
  f.sel = a.sel_scores;
  f.hist = a.sel_hist;
  f.score_stride = a.score_stride;
  const int64_t units = static_cast<int64_t>(sp.B) * sp.Hkv;
  // two rows per item, a row's records over four warps, where that still gives every SM a few
  // items; eight warps a row for smaller batches (more records in flight)
  f.rows = units * sp.G >= 4 * static_cast<int64_t>(a.sm_count) ? 2 : 1;
  // one wave of CTAs at most: a second one would find the first's caches cold again
  const int64_t N4 = (sp.P + sp.n + kHistStep - 1) / kHistStep * kHistStep;
  const int64_t items = units * sp.G / f.rows, steps = a.sel_hist != nullptr ? units * (N4 / kHistStep) : 0;
  const int64_t most = static_cast<int64_t>(kFCtasPerSm) * a.sm_count, want = items > steps ? items : steps;
  const int64_t ctas = ((want < most ? want : most) + kFCtasPerSm - 1) / kFCtasPerSm * kFCtasPerSm;
  // an item takes about as long as kItemSteps steps of scores: the CTAs that have one more item
  // than the others have that much less to count
  f.hist_few_first = items % ctas;
  const int64_t even = (steps + f.hist_few_first * kItemSteps + ctas - 1) / ctas;
  const int64_t few = even > kItemSteps ? even - kItemSteps : 0;
  f.hist_few = few * kHistStep;
  f.hist_many = (steps - f.hist_few_first * few + ctas - f.hist_few_first - 1) / (ctas - f.hist_few_first) * kHistStep;
  f.hist_vec = a.score_stride % 4 == 0;
  f.out = a.out;
  f.n_surv = a.n_surv;
  f.alpha = a.alpha;
  f.c = a.c;
  f.eps = a.eps;
  return launch_pdl(a.sel_scores != nullptr ? shared_finish_kernel<true> : shared_finish_kernel<false>,
                    dim3(static_cast<unsigned>(ctas)), dim3(kFThreads), 0, stream, 0u, f);
}

}  // namespace embla
