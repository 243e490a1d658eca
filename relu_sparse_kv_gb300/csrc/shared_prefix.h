// Launchers of the decode behind a shared prefix (shared_decode.cu and the sparse layers'
// kernels), and its work split; not part of the ABI.
#pragma once

#include "internal.h"

namespace embla {

// Full-layer decode over a shared prefix of P keys and n own keys per sequence.  The queries
// of one KV head of 128 / G sequences make a row block; its work per KV head is a list of
// 128-key tiles, the prefix's tp tiles and then each of its sequences' ts own tiles, and the
// lists of the KV heads follow one another.  Each row block's list is cut into as many equal
// pieces as it gets CTAs; the record of KV head g's tiles inside piece q lives in
// slot(rb, q, g).  Tiles times pieces of a row block stay below 2^31 (fits()), so the device
// splits in 32 bits.
struct SharedSplit {
  int64_t P, n;
  int64_t tp, ts;
  int32_t B, Hkv, G;
  int32_t blocks;                // row blocks; all but the last hold 128 / G sequences
  int32_t ctas_full, ctas_last;  // CTAs (pieces) of each full row block, of the last one
  __host__ __device__ int sequences(int rb) const {
    const int seqs = 128 / G, left = B - rb * seqs;
    return left < seqs ? left : seqs;
  }
  __host__ __device__ int64_t group_tiles(int rb) const { return tp + sequences(rb) * ts; }
  __host__ __device__ int64_t pieces(int rb) const { return rb < blocks - 1 ? ctas_full : ctas_last; }
  __host__ __device__ int64_t ctas() const {
    return blocks > 0 ? static_cast<int64_t>(blocks - 1) * ctas_full + ctas_last : 0;
  }
  __host__ __device__ int block_of_cta(int cta) const {
    const int rb = ctas_full > 0 ? cta / ctas_full : 0;
    return rb < blocks - 1 ? rb : blocks - 1;
  }
  __host__ __device__ bool fits() const {
    return blocks == 0 || group_tiles(0) * Hkv * (ctas_full > ctas_last ? ctas_full : ctas_last) <= INT32_MAX;
  }
  __host__ __device__ uint32_t piece_start(uint32_t q, uint32_t T, uint32_t Q) const { return q * T / Q; }
  __host__ __device__ uint32_t piece_of_tile(uint32_t t, uint32_t T, uint32_t Q) const {
    return ((t + 1) * Q - 1) / T;
  }
  // The pieces whose records hold the rows of a row block's sequence seq for KV head g: those with
  // prefix tiles of g, [first, first + prefix), then those with own tiles of seq only,
  // [own, own + rest).
  struct RowPieces {
    int first, prefix, own, rest;
  };
  __host__ __device__ RowPieces row_pieces(int rb, int seq, int g) const {
    const uint32_t gt = static_cast<uint32_t>(group_tiles(rb)), T = gt * Hkv;
    const uint32_t Q = static_cast<uint32_t>(pieces(rb)), base = g * gt;
    int qa = 0, qb = -1, qc = 0, qd = -1;
    if (tp > 0) {
      qa = static_cast<int>(piece_of_tile(base, T, Q));
      qb = static_cast<int>(piece_of_tile(base + static_cast<uint32_t>(tp) - 1, T, Q));
    }
    if (ts > 0) {
      const uint32_t first_own = base + static_cast<uint32_t>(tp + seq * ts);
      qc = static_cast<int>(piece_of_tile(first_own, T, Q));
      qd = static_cast<int>(piece_of_tile(first_own + static_cast<uint32_t>(ts) - 1, T, Q));
      if (qc <= qb) qc = qb + 1;
    }
    return {qa, qb - qa + 1, qc, qd >= qc ? qd - qc + 1 : 0};
  }
  __host__ __device__ int64_t slot(int rb, int64_t piece, int g) const {
    return static_cast<int64_t>(rb) * (ctas_full + Hkv) + piece + g;
  }
};
SharedSplit shared_split(int B, int Hkv, int G, int64_t P, int64_t n, int sm_count);
size_t shared_workspace_bytes(const SharedSplit &sp);
struct SharedCall {
  const CUtensorMap *tm_q, *tm_kp, *tm_vp, *tm_ko, *tm_vo;
  const void *q, *k_prefix, *v_prefix, *k_cache, *v_cache;
  int64_t prefix_stride, cache_stride;
  float *sel_scores;
  uint32_t *sel_hist;
  int64_t score_stride;
  void *workspace;
  float *out;
  int32_t *n_surv;
  uint32_t *flags;
  float alpha, c, eps;
  int group;             // query heads per KV head
  int device, sm_count;  // the current device (below 64)
};
cudaError_t launch_shared_decode(const SharedCall &a, const SharedSplit &sp, cudaStream_t stream);

// Sparse-layer decode (bf16 caches) with the prefix's rows: key indices below prefix.len are rows of
// the prefix's planes [Hkv, stride, D], the others rows idx - len of the unit's own cache; n counts
// both.  The other arguments as for launch_sparse_decode.
struct SharedRows {
  const void *k, *v;
  int64_t len, stride;
};
cudaError_t launch_sparse_decode_shared(int G, int Hq, const void *q, const SharedRows &prefix,
                                        const void *k_cache, const void *v_cache, const int32_t *idx,
                                        int idx_stride, const int32_t *count, int64_t units, int Hkv,
                                        int64_t n, int64_t ncap, float tau, float *out,
                                        uint32_t *flags, int sm_count, cudaStream_t stream);

}  // namespace embla
