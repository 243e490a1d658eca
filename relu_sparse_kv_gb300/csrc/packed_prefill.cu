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
//              loads by TMA the 128 query rows (two blocks' worth fit) and the tiles' K rows.
//   warp 1     tcgen05 issuer of S = Q K^T (M 128 rows x N keys) into one of three tensor-memory
//              buffers, S of tile t into that of tile t - 3 once its P V is done; full layers: of two
//              buffers, once tile t - 2's is read.
//   warps 2..  one team or two of eight warps: the weights.  A warp takes 16 rows, a row lies in the four
//              lanes of a quad (the fragment layout of 16x256b loads), so a row's maximum is two
//              shuffles and no other warp's business, and P, packed in pairs, goes back in 16x128b stores
//              over its S; full layers: into one of two buffers of its own.  At the end of a block they
//              divide O and store it.
//   then       the tcgen05 issuer of O += P V, P from tensor memory, V as it lies;
//   and last   the loads of the tiles' V rows.
//
// Softmax.  With z = tau log2(e) s, P = exp2(z - m) for a running reference m per row and l = sum P.
// m follows the maximum only when that has grown by more than 2^8 (kSlack): O, in tensor memory, is then
// multiplied by exp2(m_old - m) once its last product is done; O / l does not depend on m.  m, l and
// O are fp32; P enters the product as bf16 (2^-8 of each weight at most, as much as the output's own
// rounding to bf16).
// ReLU^2.  w' = max(dot rk_j, 0)^2, a2 = alpha^2 / (mean(q^2) + eps): out = a2 O' / (c + a2 sum w').
//
// A weight of zero times an infinite or NaN value would be NaN, and a tile holds rows that a query
// must not see.  Value rows of other sequences, or behind the last (which nothing may have written), are
// cleared in shared memory before the product.  Against its own later and older rows, an output that
// comes out infinite or NaN is computed again by its warp over the visible keys (slow_rows); nothing else
// pays for it.  Measured: 16,300 tokens of a full layer with NaN behind them 0.60 ms (80 ms when a sequence's
// neighbours were left to a slow path too), with NaN in all of them 133 ms; 8 x 16,384 tokens of a window layer
// 18 ms.  (Cleared by the weights' warps, or by the one that loads V, 4 to 20 % more on every call.)
//
// A block's sequence.  The host knows no lengths, so block numbers are spread with room to spare: sequence
// b owns the numbers from floor(cu_q[b] / R) + b (R tokens to a block), which is enough for its blocks,
// and a number past them is skipped.  The owner is found by a 32-way search, whose first step needs no memory
// (one of 32 sequences; reading each block's own took the warp that also loads Q and K 1,500 cycles more).
//
// What bounds it, and what was measured (16 query heads):
//   - long prompts: the tensor cores.  One prompt of 16,384 tokens through a full layer 564 to 630 us from a graph,
//     1,950 to 1,745 TFLOP/s of visible products (boards differ; 0.92 to 1.03 of the burst rate), 660 us in a loop
//     of calls under the power cap (1,670, 0.97 of the sustained rate); softmax over all keys 1,520 (8,192
//     tokens), there the exponentials and the maximum add what the tensor cores cannot hide.
//   - a window of 128 keys: memory.  8 x 16,384 tokens 213 us from a graph, 6.3 TB/s (0.93 of a copy's rate),
//     230 in a loop of calls; a block is
//     two tiles of 80 keys, so most of a warp's time is a chain of short waits.  Two teams hide each other's:
//     one team of eight warps on tiles of 128 took 480 us, two on tiles of 80 with a barrier per block 315.
//     The issuers walk their loops as whole warps with places and phases counted on, so that a product's
//     descriptor is two additions (one lane of each, with divisions: 247); every wait polls without a
//     suspend hint (with one of 20 us 8 ragged prompts of 6,164 tokens took 20.6 against 19.4, a window of
//     1,024 218 against 215).  What a block's end needs of its description is read then (in registers all
//     along, the weights spilled: 237).
//     With four warps of their own for the outputs beside one team 320 us (they take longer for a
//     block than its weights do; the long prompt gained, 604 us).
//   - short prompts: what a block costs beside its tiles, about 4,000 cycles.  Describing blocks earlier, a
//     second O, teams on alternate tiles of two blocks, and outputs read while the next block's
//     first weights are worked out each measured the same or slower.
#include <type_traits>

#include "ptx_blocks.cuh"
#include "ragged.h"

namespace embla {
namespace {

constexpr int kTeamWarps = 8;      // warps that turn a block's scores into weights
constexpr int kRing = 3;           // V stages
constexpr int kBoxQ = 128 * 128;   // [128 rows][64 bf16]
constexpr float kSlack = 8.0f;     // P stays below 2^kSlack
constexpr uint32_t kSumExp = 27, kSumExps = 200;  // a sum of weights, 2^-100 .. 2^100, has lost none of them (biased)
constexpr uint64_t kLimitNs = 10000000000ull;  // 10 s: rows computed again (slow_rows) hold the others up
constexpr int kBlocksAhead = 4;    // descriptions of blocks in flight
constexpr int kTmemCols = 512;
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
  int32_t seqn;   // its last key, less k0
  int32_t tile0;  // tiles of the blocks before
};

// TEAMS sets of kTeamWarps warps take blocks in turn; each has an O of its own.  P is written over its S, and
// three such buffers go round.  For ReLU^2 and one team it has two buffers apart, and S two that are free once
// they are read: the tensor cores wait less for a tile's weights (16,384 tokens 622 us over S, 589 apart), but
// a weights warp waits for P's buffer, and softmax, the longer work, does not gain (window 128, when it was
// tried, 220 us over S, 245 apart).  Sixteen warps on half rows each: 148 us for 14,496 tokens in four sequences, eight 140.
template <int MODE, int N, int TEAMS>
struct Layout {
  static constexpr bool kApart = MODE == kPackedRelu2 && TEAMS == 1;
  static constexpr int kBuffers = kApart ? 2 : kRing;
  static constexpr int kThreads = (4 + TEAMS * kTeamWarps) * 32;
  static constexpr int kWarpPV = 2 + TEAMS * kTeamWarps, kWarpV = kWarpPV + 1;
  static constexpr int kRingK = N < 128 ? 4 : 2;  // K stages
  static constexpr int kQ = 2;                    // blocks whose query rows are there
  static_assert(kQ % TEAMS == 0, "a team's blocks have the same places");
  static constexpr int kColP = kApart ? kBuffers * N : 0, kStepP = kApart ? N / 2 : N;  // columns
  static constexpr int kColO = 3 * N;  // TEAMS times 128
  static_assert(kColO + TEAMS * 128 <= kTmemCols, "tensor memory");
  static constexpr int kBoxKV = N * 128;  // [N rows][64 bf16]
  static constexpr int kStage = 2 * kBoxKV;
  static constexpr int kSlowCols = TEAMS == 1 ? 64 : (MODE == kPackedRelu2 ? 16 : 32);
  static constexpr int kOffK = kQ * 2 * kBoxQ;
  static constexpr int kOffV = kOffK + kRingK * kStage;
  static constexpr int kOffBlock = kOffV + kRing * kStage;
  static constexpr int kOffBar = kOffBlock + kBlocksAhead * static_cast<int>(sizeof(Block));
  static constexpr int kNBars = 2 * kRingK + 2 * kRing + (1 + TEAMS + kApart) * kBuffers + 2 * kBlocksAhead + 2 * kQ +
                                2 * TEAMS;
  static constexpr int kOffMisc = kOffBar + kNBars * 8;
  static constexpr int kBytes = kOffMisc + 32 + 1024;  // + room to align the base to 1024
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, kLimitNs); }

// A place in a ring of R barriers and the parity of its phase.
template <int R>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == R) {
      at = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ Ring before() const { return at > 0 ? Ring{at - 1, phase} : Ring{R - 1, phase ^ 1u}; }
};
// The place before was completed (at once where there was none).
template <int R>
__device__ __forceinline__ bool wait_before(uint64_t *bars, Ring<R> r) {
  const Ring<R> b = r.before();
  return mbar_wait(&bars[b.at], b.phase, kLimitNs);
}

__device__ __forceinline__ void set_abort(volatile int *abort_flag, uint32_t *flags) {
  *abort_flag = 1;
  atomicOr(flags, kFlagWaitTimeout);
}

// Entries that do not ascend or lie outside the rows.
__device__ __forceinline__ bool bad_sequence(const PackedPrefillParams &p, int q_lo, int q_hi, int k_lo, int k_hi) {
  return q_lo < 0 || q_hi < q_lo || q_hi > p.tokens || k_lo < 0 || k_hi < k_lo || k_hi > p.keys;
}

// The blocks of a CTA, one after the other (the whole warp calls).  Tokens, keys and block numbers lie
// below 2^31.
template <int MODE, int N, int G>
struct BlockFinder {
  static constexpr int R = 128 / G;
  uint32_t at, step, numbers;  // this CTA's place in the next round of numbers, and numbers per KV head
  bool draw = false;
  // The first step of the search, kept in registers: the first number past lane's group of sequences; and
  // where a group is one sequence, its queries and keys.
  int past = INT32_MAX;
  int seq_q0 = 0, seq_q1 = 0, seq_k0 = 0, seq_k1 = 0;
  // the sequence found last: its block numbers, queries and keys
  int first = 0, end = 0, q_lo = 0, q_hi = 0, k_lo = 0, k_hi = 0;
  __device__ BlockFinder(const PackedPrefillParams &p, uint32_t cta, uint32_t ctas, int lane)
      : at(cta), step(ctas), numbers(static_cast<uint32_t>(p.blocks) / static_cast<uint32_t>(p.Hkv)) {
    const int w = (p.batch + 31) / 32, i = (lane + 1) * w;
    if (i <= p.batch) past = p.cu_q[i] / R + i;
    if (p.batch <= 32 && lane < p.batch) {
      seq_q0 = p.cu_q[lane], seq_q1 = p.cu_q[lane + 1];
      seq_k0 = p.cu_k[lane], seq_k1 = p.cu_k[lane + 1];
    }
  }

  // The sequence that owns block number v becomes the one found last; false where there is none.
  __device__ __forceinline__ bool find(const PackedPrefillParams &p, int v, int lane) {
    if (v >= first && v < end) return true;
    // sequences whose successor's numbers begin at or before v
    int w = (p.batch + 31) / 32;
    int lo = __popc(__ballot_sync(0xffffffffu, past <= v)) * w, hi = min(p.batch, lo + w - 1);
    while (hi > lo) {
      w = (hi - lo + 31) / 32;
      const int i = lo + (lane + 1) * w;
      const int n = __popc(__ballot_sync(0xffffffffu, i <= hi && p.cu_q[i] / R + i <= v));
      lo += n * w;
      hi = min(hi, lo + w - 1);
    }
    if (lo >= p.batch) return false;
    if (p.batch <= 32) {
      q_lo = __shfl_sync(0xffffffffu, seq_q0, lo), q_hi = __shfl_sync(0xffffffffu, seq_q1, lo);
      k_lo = __shfl_sync(0xffffffffu, seq_k0, lo), k_hi = __shfl_sync(0xffffffffu, seq_k1, lo);
    } else {
      q_lo = p.cu_q[lo], q_hi = p.cu_q[lo + 1], k_lo = p.cu_k[lo], k_hi = p.cu_k[lo + 1];
    }
    first = end = q_lo / R + lo;
    if (bad_sequence(p, q_lo, q_hi, k_lo, k_hi)) return false;
    end = first + (q_hi - q_lo + R - 1) / R;
    return v >= first && v < end;
  }

  // The next block; tiles < 0 after the last.  A round of numbers is dealt at a time, alternate rounds in
  // reverse order, so the CTAs' sums of key tiles stay close.  With a ticket counter that holds for two
  // rounds, and then each CTA draws its next number when it has asked for the last rows of a block.
  __device__ __forceinline__ Block next(const PackedPrefillParams &p, int lane) {
    Block r = {};
    r.tiles = -1;
    for (;;) {
      if (draw) {
        uint32_t ticket = 0;
        if (lane == 0) ticket = atomicAdd(p.ticket, 1u);
        at = 2 * step + __shfl_sync(0xffffffffu, ticket, 0);
      }
      const uint32_t idx = at;
      const uint32_t base = idx - idx % step;
      if (base >= static_cast<uint32_t>(p.blocks)) return r;
      at = base + step + (step - 1 - (idx - base));
      draw = p.ticket != nullptr && at >= 2 * step;
      if (idx >= static_cast<uint32_t>(p.blocks)) continue;
      const uint32_t up = idx / static_cast<uint32_t>(p.Hkv);
      const int v = static_cast<int>(numbers - 1 - up);  // the last ones, with the most keys, first
      if (!find(p, v, lane)) continue;
      const int t0 = (v - first) * R, lq = q_hi - q_lo, lk = k_hi - k_lo;
      r.g = static_cast<int>(idx - up * static_cast<uint32_t>(p.Hkv));
      r.q0 = q_lo + t0;
      r.nq = min(lq - t0, R);
      const int newest = lk - lq + t0, last = newest + r.nq - 1;  // of the first and last token
      const int oldest = max(newest - p.window + 1, 0);
      r.k0 = k_lo + oldest;
      if (MODE == kPackedRelu2) r.k0 &= ~3;  // (the key norms are read in pairs)
      r.tiles = last < 0 ? 0 : (k_lo + last - r.k0) / N + 1;
      r.p0 = k_lo + newest - r.k0;
      r.seq0 = k_lo - r.k0;
      r.seqn = k_hi - 1 - r.k0;
      return r;
    }
  }
};

// The 16 rows of a warp from rowa on once more, from memory and by warp products, those of `bad` (bit r: row
// rowa + r) stored.  In two passes, so that no partial sum is larger than the result needs: maximum and sum
// (ReLU^2: the sum), then the values by their normalised weights, in two bf16 parts.  Infinite and NaN values are
// zeros to the products, and are added to the rows that see them.  (COLS columns at a time, nothing kept that can
// be read again: what does not fit beside the caller's registers makes those spill, 5 to 30 % on every call.)
template <int MODE, int G, int COLS>
__device__ __noinline__ void slow_rows(const PackedPrefillParams &p, const Block &b, int rowa, uint32_t bad, int lane) {
  const int g = lane >> 2, t = lane & 3;  // this lane's rows: g and g + 8; its keys of eight: 2t and 2t + 1
  const int tokens = b.nq - 1;
  const int low = max(b.seq0, b.p0 + min(rowa / G, tokens) - p.window + 1), high = b.p0 + min((rowa + 15) / G, tokens);
  const int newest0 = b.p0 + min((rowa + g) / G, tokens), newest1 = b.p0 + min((rowa + g + 8) / G, tokens);
  auto row = [&](int i) {  // of the query, [token][head]
    const int r = rowa + g + 8 * i;
    return p.q.base + static_cast<int64_t>(b.q0 + min(r / G, tokens)) * p.q.stride + (b.g * G + r % G) * kHeadDim;
  };
  float scale0 = p.tau2, scale1 = p.tau2;
  if (MODE == kPackedRelu2) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const uint32_t *q = reinterpret_cast<const uint32_t *>(row(i)) + t;
      float ss = 0.0f;
#pragma unroll 4
      for (int k = 0; k < 16; ++k) {
        const float x = bf16lo(q[4 * k]), y = bf16hi(q[4 * k]);
        ss = fmaf(x, x, fmaf(y, y, ss));
      }
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      (i ? scale1 : scale0) = p.alpha / sqrtf(ss * (1.0f / kHeadDim) + p.eps);
    }
  }
  // keys j0 .. j0 + 7: elements 2i + e are row g + 8i, key j0 + 2t + e; ReLU^2: their weights
  auto scores = [&](int j0, float (&s)[4]) {
    const uint32_t *k = reinterpret_cast<const uint32_t *>(
        p.k.base + static_cast<int64_t>(b.k0 + min(j0 + g, high)) * p.k.stride + b.g * kHeadDim) + t;
    const uint32_t *q0 = reinterpret_cast<const uint32_t *>(row(0)) + t;
    const uint32_t *q1 = reinterpret_cast<const uint32_t *>(row(1)) + t;
    s[0] = s[1] = s[2] = s[3] = 0.0f;
#pragma unroll (COLS > 32 ? 4 : 2)
    for (int ks = 0; ks < 64; ks += 8) mma_16816_bf16(s, q0[ks], q1[ks], q0[ks + 4], q1[ks + 4], k[ks], k[ks + 4]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + 2 * t + (e & 1), newest = e < 2 ? newest0 : newest1;
      const bool live = j >= b.seq0 && j > newest - p.window && j <= newest;
      s[e] *= e < 2 ? scale0 : scale1;
      if (MODE == kPackedRelu2) {
        const float w = live ? fmaxf(s[e] * p.rk[b.g * p.rk_stride + b.k0 + j], 0.0f) : 0.0f;
        s[e] = w * w;
      } else if (!live) {
        s[e] = -INFINITY;
      }
    }
  };
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  auto join = [&](int i, float m2, float l2) {
    const float mn = fmaxf(m[i], m2);
    l[i] = l[i] * (m[i] == mn ? 1.0f : exp2f(m[i] - mn)) + l2 * (m2 == mn ? 1.0f : exp2f(m2 - mn));
    m[i] = mn;
  };
#pragma unroll 1
  for (int j0 = low; j0 <= high; j0 += 8) {
    float s[4];
    scores(j0, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (MODE == kPackedRelu2)
        l[e >> 1] += s[e];
      else if (s[e] != -INFINITY)
        join(e >> 1, s[e], 1.0f);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[i], o), l2 = __shfl_xor_sync(0xffffffffu, l[i], o);
      if (MODE == kPackedRelu2)
        l[i] += l2;
      else
        join(i, m2, l2);
    }
    const float z = MODE == kPackedRelu2 ? p.c + l[i] : l[i];
    l[i] = z == 0.0f ? 0.0f : 1.0f / z;
  }
#pragma unroll 1
  for (int c = 0; c < kHeadDim; c += COLS) {
    float o[COLS / 8][4];  // columns c + 8n + 2t and the next of rows g and g + 8
#pragma unroll
    for (int n = 0; n < COLS / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll 1
    for (int j0 = low; j0 <= high; j0 += 16) {
      uint32_t a[3][4];  // the weights' two parts, and ones where the row sees the key
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s[4];
        scores(j0 + 8 * h, s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float w[2];
          uint32_t seen = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[2 * i + e];
            w[e] = MODE == kPackedRelu2 ? x * l[i] : (x == -INFINITY ? 0.0f : exp2f(x - m[i]) * l[i]);
            if (MODE == kPackedRelu2 ? x > 0.0f : x != -INFINITY) seen |= 0x3F80u << (16 * e);
          }
          const uint32_t hi = pack_bf16x2(w[0], w[1]);
          a[0][2 * h + i] = hi;
          a[1][2 * h + i] = pack_bf16x2(w[0] - bf16lo(hi), w[1] - bf16hi(hi));
          a[2][2 * h + i] = seen;
        }
      }
#pragma unroll
      for (int n = 0; n < COLS / 8; ++n) {
        uint32_t x[4], clean[4];  // keys 2t, 2t + 1, 2t + 8 and 2t + 9
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = min(j0 + 2 * t + (e & 1) + 8 * (e >> 1), high);
          x[e] = p.v.base[static_cast<int64_t>(b.k0 + j) * p.v.stride + b.g * kHeadDim + c + 8 * n + g];
          const bool broken = (x[e] & 0x7F80u) == 0x7F80u;
          odd |= broken;
          clean[e] = broken ? 0u : x[e];
        }
#pragma unroll
        for (int part = 1; part >= 0; --part)
          mma_16816_bf16(o[n], a[part][0], a[part][1], a[part][2], a[part][3], clean[0] | clean[1] << 16,
                         clean[2] | clean[3] << 16);
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
          for (int kind = 0; kind < 3; ++kind) {  // NaN, +infinity, -infinity: how many of them each row sees
            uint32_t is[4];
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              is[e] = (kind == 0 ? (x[e] & 0x7FFFu) > 0x7F80u : x[e] == (kind == 1 ? 0x7F80u : 0xFF80u)) ? 0x3F80u : 0u;
            mma_16816_bf16(d, a[2][0], a[2][1], a[2][2], a[2][3], is[0] | is[1] << 16, is[2] | is[3] << 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (d[e] > 0.0f) o[n][e] += kind == 0 ? NAN : (kind == 1 ? INFINITY : -INFINITY);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rowa + g + 8 * i;
      if (bad >> (g + 8 * i) & 1u) {
        uint16_t *to = p.out + (static_cast<int64_t>(b.q0 + r / G) * p.Hkv * G + b.g * G + r % G) * kHeadDim + c + 2 * t;
#pragma unroll
        for (int n = 0; n < COLS / 8; ++n)
          *reinterpret_cast<uint32_t *>(to + 8 * n) = pack_bf16x2(o[n][2 * i], o[n][2 * i + 1]);
      }
    }
  }
}

// Scores of 16 rows x N keys to registers: element 4j + 2i + e is row l / 4 + 8i, key 8j + 2(l % 4) + e; and
// their weights back over them, packed in pairs: word 2j + i.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&acc)[N / 2]) {
  static_assert(N == 128 || N == 80, "key tile");
  if constexpr (N == 128) {
    tmem_load_16x256b_x16(taddr, acc);
  } else {
    tmem_load_16x256b_x8(taddr, *reinterpret_cast<uint32_t(*)[32]>(&acc[0]));
    tmem_load_16x256b_x2(taddr + 64, *reinterpret_cast<uint32_t(*)[8]>(&acc[32]));
  }
  tmem_wait_ld(acc);
}
template <int N>
__device__ __forceinline__ void store_weights(uint32_t taddr, const uint32_t (&w)[N / 4]) {
  if constexpr (N == 128) {
    tmem_store_16x128b_x16(taddr, w);
  } else {
    tmem_store_16x128b_x8(taddr, *reinterpret_cast<const uint32_t(*)[16]>(&w[0]));
    tmem_store_16x128b_x2(taddr + 32, *reinterpret_cast<const uint32_t(*)[4]>(&w[16]));
  }
}

// Eight words of each lane of a quad, word j the lane's part (l % 4) of group j, become the lane's two whole
// groups 2 (l % 4) and 2 (l % 4) + 1, four words each.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[8], int lane) {
  // exchange halves with the lane two away, then quarters with the next lane
  const bool b1 = lane & 2, b0 = lane & 1;
  uint32_t h[2][4];  // [part of the sender: own half's lane pair bit][group of the lane's half]
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t keep = b1 ? w[4 + j] : w[j], send = b1 ? w[j] : w[4 + j];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 2);
    h[0][j] = b1 ? got : keep;  // parts of the lanes 0, 1
    h[1][j] = b1 ? keep : got;  // parts of the lanes 2, 3
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint32_t keep = b0 ? h[part][2 + j] : h[part][j], send = b0 ? h[part][j] : h[part][2 + j];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 1);
      w[4 * j + 2 * part] = b0 ? got : keep;
      w[4 * j + 2 * part + 1] = b0 ? keep : got;
    }
}

template <int MODE, int N, int G, int TEAMS>
__global__ void __launch_bounds__(Layout<MODE, N, TEAMS>::kThreads, 1)
    packed_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PackedPrefillParams p) {
  using L = Layout<MODE, N, TEAMS>;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, N);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem, *sK = smem + L::kOffK, *sV = smem + L::kOffV;
  Block *sBlock = reinterpret_cast<Block *>(smem + L::kOffBlock);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  // Tile g has V stage g % kRing in phase (g / kRing) & 1, K stage g % kRingK in phase (g / kRingK) & 1, and
  // S and P buffers g % kBuffers in phase (g / kBuffers) & 1.  Block k has the description k % kBlocksAhead, the
  // query rows k % kQ
  // and the O of team k % TEAMS.
  constexpr int kRingK = L::kRingK, kBuffers = L::kBuffers;
  uint64_t *kfull = bars, *kempty = kfull + kRingK, *vfull = kempty + kRingK;
  // S of a tile in tensor memory: a team's tiles by its own count, so that it sees every phase
  uint64_t *sfull = vfull + kRing;
  uint64_t *pfull = sfull + TEAMS * kBuffers;  // its P there
  uint64_t *pvdone = pfull + kBuffers;         // its P V done: the P buffer and the V stage are free
  uint64_t *bfull = pvdone + kRing;  // a block's description is there
  uint64_t *bempty = bfull + kBlocksAhead;  // and has been read by everyone
  uint64_t *qfull = bempty + kBlocksAhead, *qempty = qfull + L::kQ;  // its query rows are there, and used
  uint64_t *ofull = qempty + L::kQ;  // a block's P V all done
  uint64_t *ofree = ofull + TEAMS;   // its O read out of tensor memory
  uint64_t *sempty = ofree + TEAMS;  // apart: an S has been read out of it
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  uint32_t *s_tmem = misc;
  volatile int *s_abort = reinterpret_cast<volatile int *>(misc + 1);
  volatile int *s_issued = reinterpret_cast<volatile int *>(misc + 2);   // K tiles, V tiles and query blocks
                                                                         // whose loads were issued

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x), P = static_cast<int>(gridDim.x);

  if (warp == 0) {
    if (lane < kRing) {
      mbar_init(&vfull[lane], 1);
      mbar_init(&pvdone[lane], 1);
    }
    if (lane < kBuffers) {
      for (int i = 0; i < TEAMS; ++i) mbar_init(&sfull[i * kBuffers + lane], 1);
      if (L::kApart) mbar_init(&sempty[lane], kTeamWarps);
      mbar_init(&pfull[lane], kTeamWarps);
    }
    if (lane < kRingK) {
      mbar_init(&kfull[lane], 1);
      mbar_init(&kempty[lane], 1);
    }
    if (lane < L::kQ) {
      mbar_init(&qfull[lane], 1);
      mbar_init(&qempty[lane], 1 + (MODE == kPackedRelu2 ? kTeamWarps : 0));  // S done, and the rows' norms
    }
    if (lane < TEAMS) {
      mbar_init(&ofull[lane], 1);
      mbar_init(&ofree[lane], kTeamWarps);
    }
    if (lane < kBlocksAhead) {
      mbar_init(&bfull[lane], 1);
      mbar_init(&bempty[lane], 3 + kTeamWarps);  // the two issuers, the V loads, the team
    }
    if (lane == 0) {
      *s_abort = 0;
      s_issued[0] = s_issued[1] = s_issued[2] = 0;
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
    // ------------------------------------------------------------------ blocks, Q and K loads
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
    }
    BlockFinder<MODE, N, G> finder(p, cta, P, lane);
    Block b = finder.next(p, lane);
    Ring<kBlocksAhead> d;
    Ring<L::kQ> q;
    Ring<kRingK> r;
    int issued = 0;
    bool ok = true;
    for (int k = 0, ends = 0; ok && ends < TEAMS; ++k) {  // (each team is told of the end)
      // (a barrier's first wait, for the phase before its first, ends at once)
      b.tile0 = issued;
      ok = __all_sync(0xffffffffu, wait_bar(&bempty[d.at], d.phase ^ 1u));
      if (!ok) break;
      if (lane == 0) {
        sBlock[d.at] = b;
        mbar_arrive(&bfull[d.at]);
      }
      d.next();
      if (b.tiles < 0) {
        ++ends;
        continue;
      }
      // (blocks without tiles take their turn with the query rows, but load none)
      ok = __all_sync(0xffffffffu, wait_bar(&qempty[q.at], q.phase ^ 1u));
      if (!ok) break;
      if (elect_one()) {
        if (b.tiles > 0) {
          uint8_t *to = sQ + q.at * 2 * kBoxQ;
          mbar_arrive_expect_tx(&qfull[q.at], 2 * kBoxQ);
          tma_load_4d(to, &tm_q, &qfull[q.at], 0, 0, b.g, b.q0);
          tma_load_4d(to + kBoxQ, &tm_q, &qfull[q.at], 64, 0, b.g, b.q0);
        } else {
          mbar_arrive(&qfull[q.at]);
        }
        s_issued[2] = k + 1;
      }
      __syncwarp();
      q.next();
      for (int t = 0, row = b.k0; t < b.tiles; ++t, row += N) {
        ok = __all_sync(0xffffffffu, wait_bar(&kempty[r.at], r.phase ^ 1u));
        if (!ok) break;
        ++issued;
        if (elect_one()) {
          uint8_t *to = sK + r.at * L::kStage;
          mbar_arrive_expect_tx(&kfull[r.at], L::kStage);
          tma_load_3d(to, &tm_k, &kfull[r.at], 0, b.g, row);
          tma_load_3d(to + L::kBoxKV, &tm_k, &kfull[r.at], 64, b.g, row);
          s_issued[0] = issued;
        }
        __syncwarp();
        r.next();
      }
      if (ok) b = finder.next(p, lane);
    }
    if (!ok && lane == 0) set_abort(s_abort, p.flags);
    // entries that no block could use are reported
    for (int64_t b = static_cast<int64_t>(cta) * 32 + lane; b < p.batch; b += static_cast<int64_t>(P) * 32)
      if (bad_sequence(p, p.cu_q[b], p.cu_q[b + 1], p.cu_k[b], p.cu_k[b + 1])) atomicOr(p.flags, kFlagIndexRange);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S issuer
    // (the warp walks its loop together and one lane issues: descriptors stay in uniform registers)
    const uint64_t qdesc = smem_desc_sw128(smem_u32(sQ));
    const uint64_t kdesc = smem_desc_sw128(smem_u32(sK));
    Ring<kBlocksAhead> d;
    Ring<L::kQ> q;
    Ring<kBuffers> sb, mine[TEAMS];  // mine: the tiles of the team whose turn it is, then the other's
    Ring<kRingK> kb;
    bool ok = true;
    while (ok) {
      ok = !*s_abort && wait_bar(&bfull[d.at], d.phase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int tiles = sBlock[d.at].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bempty[d.at]);
      d.next();
      if (tiles < 0) break;
      ok = __all_sync(0xffffffffu, wait_bar(&qfull[q.at], q.phase));
      const int s = TEAMS > 1 ? q.at % TEAMS : 0;
      for (int t = 0; ok && t < tiles; ++t) {
        ok = wait_bar(&kfull[kb.at], kb.phase) && wait_bar(&(L::kApart ? sempty : pvdone)[sb.at], sb.phase ^ 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint64_t qd = qdesc + static_cast<uint64_t>(q.at * (2 * kBoxQ >> 4));
          const uint64_t kd = kdesc + static_cast<uint64_t>(kb.at * (L::kStage >> 4));
          const uint32_t to = tmem + sb.at * N;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            // dims 16kk .. 16kk + 15: 32 bytes into a 128-byte row; dims 64.. start the second box
            tc_mma_bf16(to, qd + (((kk >> 2) * kBoxQ + (kk & 3) * 32) >> 4),
                        kd + (((kk >> 2) * L::kBoxKV + (kk & 3) * 32) >> 4), kIdescS, kk > 0 ? 1u : 0u);
          tc_commit(&sfull[s * kBuffers + mine[0].at]);
          tc_commit(&kempty[kb.at]);
          if (t + 1 == tiles) tc_commit(&qempty[q.at]);
        }
        __syncwarp();
        sb.next();
        kb.next();
        mine[0].next();
      }
      if (ok && tiles == 0 && lane == 0) mbar_arrive(&qempty[q.at]);
      if (ok) q.next();
      if (TEAMS > 1 && ok) {
        const Ring<kBuffers> m = mine[0];
        mine[0] = mine[TEAMS - 1];
        mine[TEAMS - 1] = m;
      }
    }
    if (!ok && lane == 0) set_abort(s_abort, p.flags);
    // every MMA of this warp has completed, and its last commits arrived, before the tensor memory is
    // released and the CTA leaves (also when another role has given up)
    const int s = TEAMS > 1 ? q.at % TEAMS : 0;  // the team of mine[0]
    wait_before(sfull + s * kBuffers, mine[0]);
    if (TEAMS > 1) wait_before(sfull + (s ^ 1) * kBuffers, mine[TEAMS - 1]);
    wait_before(kempty, kb);
    wait_before(qempty, q);
    wait_before(qempty, q.before());
    __syncwarp();
  } else if (warp == L::kWarpPV) {
    // ------------------------------------------------------------------ P V issuer
    const uint64_t vdesc = smem_desc_sw128_mn(smem_u32(sV), L::kBoxKV);
    Ring<kBlocksAhead> d;
    Ring<TEAMS> o;
    Ring<kRing> vb;
    Ring<2> pair;  // apart: the P buffers
    bool ok = true;
    while (ok) {
      ok = !*s_abort && wait_bar(&bfull[d.at], d.phase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int tiles = sBlock[d.at].tiles, seq0 = sBlock[d.at].seq0, seqn = sBlock[d.at].seqn;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bempty[d.at]);
      d.next();
      if (tiles < 0) break;
      // the O of the team's block before has been read
      ok = __all_sync(0xffffffffu, wait_bar(&ofree[o.at], o.phase ^ 1u));
      for (int t = 0; ok && t < tiles; ++t) {
        ok = __all_sync(0xffffffffu, wait_bar(&vfull[vb.at], vb.phase));
        if (!ok) break;
        if (t * N < seq0 || t * N + N - 1 > seqn) {  // value rows of other sequences, or behind the last
          uint8_t *v = sV + vb.at * L::kStage;
          for (int x = lane; x < 16 * N; x += 32) {
            const int j = t * N + (x >> 3) % N;  // (a row's 128 bytes of a box stay together)
            if (j < seq0 || j > seqn) *reinterpret_cast<uint4 *>(v + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // read by the tensor cores
          __syncwarp();
        }
        const int pb = L::kApart ? pair.at : vb.at;
        ok = __all_sync(0xffffffffu, wait_bar(&pfull[pb], L::kApart ? pair.phase : vb.phase));
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint64_t vd = vdesc + static_cast<uint64_t>(vb.at * (L::kStage >> 4));
          const uint32_t to = tmem + L::kColO + o.at * 128, from = tmem + L::kColP + pb * L::kStepP;
#pragma unroll
          for (int kk = 0; kk < N / 16; ++kk)
            // keys 16kk .. 16kk + 15: eight columns of P, V rows 16kk .. (2 KB apart)
            tc_mma_bf16_tmem_a(to, from + 8 * kk, vd + (kk * 2048 >> 4), kIdescPV, (t > 0 || kk > 0) ? 1u : 0u);
          tc_commit(&pvdone[vb.at]);
          if (t + 1 == tiles) tc_commit(&ofull[o.at]);
        }
        __syncwarp();
        vb.next();
        pair.next();
      }
      if (ok && tiles == 0 && lane == 0) mbar_arrive(&ofull[o.at]);
      if (ok) o.next();
    }
    if (!ok && lane == 0) set_abort(s_abort, p.flags);
    // every MMA of this warp has completed before the tensor memory is released
    wait_before(pvdone, vb);
    wait_before(ofull, o);
    if (TEAMS > 1) wait_before(ofull, o.before());
    __syncwarp();
  } else if (warp == L::kWarpV) {
    // ------------------------------------------------------------------ V loads
    if (lane == 0) {
      tma_prefetch_desc(&tm_v);
      Ring<kBlocksAhead> d;
      Ring<kRing> r;
      int issued = 0;
      bool ok = true;
      while (ok) {
        ok = !*s_abort && wait_bar(&bfull[d.at], d.phase);
        if (!ok) break;
        const int tiles = sBlock[d.at].tiles, head = sBlock[d.at].g, k0 = sBlock[d.at].k0;
        mbar_arrive(&bempty[d.at]);
        d.next();
        if (tiles < 0) break;
        for (int t = 0, row = k0; t < tiles; ++t, row += N) {
          ok = wait_bar(&pvdone[r.at], r.phase ^ 1u);
          if (!ok) break;
          uint8_t *to = sV + r.at * L::kStage;
          mbar_arrive_expect_tx(&vfull[r.at], L::kStage);
          tma_load_3d(to, &tm_v, &vfull[r.at], 0, head, row);
          tma_load_3d(to + L::kBoxKV, &tm_v, &vfull[r.at], 64, head, row);
          s_issued[1] = ++issued;
          r.next();
        }
      }
      if (!ok) set_abort(s_abort, p.flags);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ weights and outputs
    const int team = (warp - 2) / kTeamWarps;
    const int quarter = warp & 3;           // the tensor-memory lanes this warp may reach
    const int half = ((warp - 2) >> 2) & 1;     // rows 16 half .. of them
    const int rowa = quarter * 32 + half * 16;  // the warp's first row
    const int row0 = rowa + (lane >> 2);        // this lane's rows: row0 and row0 + 8
    const int q2 = 2 * (lane & 3);              // its columns: 8j + q2 and the next
    const uint32_t lanes16 = static_cast<uint32_t>(rowa) << 16;
    const uint32_t colo = tmem + L::kColO + team * 128 + lanes16;
    const bool flip = MODE == kPackedSoftmax && p.tau2 < 0.0f;
    const float tau2 = fabsf(p.tau2);
    bool ok = true;
    Ring<kBuffers> mine;  // the team's tiles
    for (int k = team, n = 0; ok; k += TEAMS, ++n) {  // the team's n-th block
      // (every decision to go on is the warp's: what follows is warp-wide)
      const int d = k % kBlocksAhead;
      ok = __all_sync(0xffffffffu, !*s_abort && wait_bar(&bfull[d], (k / kBlocksAhead) & 1));
      if (!ok) break;
      // (the description stays until the block is done: what its end needs is read then)
      const Block &b = sBlock[d];
      const int tiles = b.tiles, window = p.window;
      if (tiles < 0) break;
      Ring<kRing> tile{b.tile0 % kRing, static_cast<uint32_t>(b.tile0 / kRing) & 1u};
      int pair = b.tile0 & 1;  // apart: the tile's buffers
      // a row sees the keys oldest .. oldest + span, relative to k0 (none: from far behind the last)
      int oldest[2];
      uint32_t span[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int newest = b.p0 + (row0 + 8 * i) / G;
        oldest[i] = max(b.seq0, newest - window + 1);
        span[i] = static_cast<uint32_t>(newest - oldest[i]);
        if (newest < oldest[i]) {
          oldest[i] = 1 << 30;
          span[i] = 0;
        }
      }
      // every row of the warp sees the keys between these two
      const int whole0 = max(b.seq0, b.p0 + (rowa + 15) / G - window + 1), whole1 = b.p0 + rowa / G;
      float m[2] = {-INFINITY, -INFINITY};    // reference of each row (base 2)
      float l[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // sums of its weights in this lane, two chains per row
      // ReLU^2: the norms of this lane's keys, each read again for the next tile once it is used
      float2 rk[MODE == kPackedRelu2 ? N / 8 : 1];
      const float *rkp = nullptr;
      if constexpr (MODE == kPackedRelu2) {
        rkp = p.rk + b.g * p.rk_stride + b.k0 + q2;
        if (tiles > 0) {
#pragma unroll
          for (int j = 0; j < N / 8; ++j) rk[j] = *reinterpret_cast<const float2 *>(rkp + 8 * j);
        }
      }
      float a2[2] = {0.0f, 0.0f};  // ReLU^2: alpha^2 / (mean(q^2) + eps) of this lane's rows
      auto query_norms = [&]() {
        if constexpr (MODE == kPackedRelu2) {
          const int q = k % L::kQ;
          ok = __all_sync(0xffffffffu, wait_bar(&qfull[q], (k / L::kQ) & 1));
          if (!ok) return false;
          // two lanes to a row, a box each
          const int r = rowa + (lane >> 1);
          float ss = box_square_sum(sQ + (2 * q + (lane & 1)) * kBoxQ, r, (r & 7) ^ (4 * (lane & 1)));
          ss += __shfl_xor_sync(0xffffffffu, ss, 1);
          const float a = (p.alpha * p.alpha) / (ss * (1.0f / kHeadDim) + p.eps);
          a2[0] = __shfl_sync(0xffffffffu, a, 2 * (lane >> 2));
          a2[1] = __shfl_sync(0xffffffffu, a, 2 * (lane >> 2) + 16);
          // the query rows are read: these depend on every lane's sum
          const float used = __shfl_sync(0xffffffffu, a2[0], 0) + a2[1];
          __syncwarp();
          if (lane == 0) mbar_arrive_after(&qempty[q], used);
        }
        return true;
      };
      if constexpr (TEAMS > 1) {  // (early, so that the rows of the team's next block may come)
        if (!query_norms()) break;
      }
      for (int t = 0; t < tiles; ++t) {
        const int j0 = t * N;
        ok = __all_sync(0xffffffffu, wait_bar(&sfull[team * kBuffers + mine.at], mine.phase));
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t acc[N / 2];
        const int buffer = L::kApart ? pair : tile.at;
        load_scores<N>(tmem + lanes16 + buffer * N, acc);
        if constexpr (L::kApart) {
          tc_fence_before_sync();  // the buffer is free for another S
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[buffer]);
        }
        uint32_t hi[N / 4];
        if constexpr (MODE == kPackedSoftmax) {
          if (flip) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) acc[e] ^= 0x80000000u;
          }
          // keys that some row of the warp does not see, sixteen at a time
          if (j0 < whole0 || j0 + N - 1 > whole1) {
            const int lo[2] = {oldest[0] - j0 - q2, oldest[1] - j0 - q2};
#pragma unroll
            for (int c = 0; c < N; c += 16) {
              if (j0 + c < whole0 || j0 + c + 15 > whole1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (static_cast<uint32_t>(c + 8 * (e >> 2) + (e & 1) - lo[(e >> 1) & 1]) > span[(e >> 1) & 1])
                    acc[c / 2 + e] = 0xFF800000u;
              }
            }
          }
          float neg[2], sc[2];
          bool grown = false;
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
            ok = __all_sync(0xffffffffu, wait_before(pvdone, tile));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] *= sc[i >> 1];
#pragma unroll
            for (int c = 0; c < 128; c += 16) {
              uint32_t o[8];
              tmem_load_16x256b_x2(colo + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sc[(e >> 1) & 1]);
              tmem_store_16x256b_x2(colo + c, o);
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
              add_f32x2(l[2 * i], l[2 * i + 1], e0, e1);
              hi[2 * j + i] = pack_bf16x2(e0, e1);
            }
        } else {
          const bool next = t + 1 < tiles;
          rkp += N;
          auto weights = [&](auto with_mask) {
            const int lo[2] = {oldest[0] - j0 - q2, oldest[1] - j0 - q2};
#pragma unroll
            for (int j = 0; j < N / 8; ++j) {
              float e[4];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                mul_f32x2(e[2 * i], e[2 * i + 1], __uint_as_float(acc[4 * j + 2 * i]),
                          __uint_as_float(acc[4 * j + 2 * i + 1]), rk[j].x, rk[j].y);
              if (next) rk[j] = *reinterpret_cast<const float2 *>(rkp + 8 * j);
              if constexpr (decltype(with_mask)::value) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (static_cast<uint32_t>(8 * j + (i & 1) - lo[i >> 1]) > span[i >> 1]) e[i] = 0.0f;
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // max(x, 0)^2 = max(x |x|, 0); the denominator sums the weights the numerator multiplies.
                // (A NaN score makes the row NaN here, and slow_rows gives the key no weight.)
                const uint32_t h = pack_relu_bf16x2(e[2 * i] * fabsf(e[2 * i]), e[2 * i + 1] * fabsf(e[2 * i + 1]));
                hi[2 * j + i] = h;
                add_bf16x2(h, l[2 * i], l[2 * i + 1]);
              }
            }
          };
          // one code path per case, so that the common one has no mask
          if (j0 < whole0 || j0 + N - 1 > whole1)
            weights(std::true_type{});
          else
            weights(std::false_type{});
        }
        if constexpr (L::kApart) {
          // the product that read the P buffer's last weights is done
          ok = __all_sync(0xffffffffu, wait_before(pvdone, tile.before()));
          if (!ok) break;
          tc_fence_after_sync();
        }
        store_weights<N>(tmem + lanes16 + L::kColP + buffer * L::kStepP, hi);
        tmem_wait_st();
        tc_fence_before_sync();  // P is read by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[buffer]);
        mine.next();
        tile.next();
        pair ^= 1;
      }
      if (!ok) break;
      if constexpr (TEAMS == 1) {  // (late, so that it has the last products' time)
        if (!query_norms()) break;
      }
      // What O is multiplied with; NaN sends the row to slow_rows.  ReLU^2: 0 where no key weighs anything, NaN where the
      // sum is too large for a float, as the squares of scores that wait for their query's norm may be.  Softmax:
      // the largest weight is about 1 but where the reference is so far from zero (2^30) that its rounding
      // moves the exponents out of the floats' range; rows without keys come along, which costs them little.
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[2 * i] + l[2 * i + 1];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if constexpr (MODE == kPackedRelu2) {
          const float z = p.c + a2[i] * x;
          f[i] = x != 0.0f && z != 0.0f ? a2[i] / z + (z - z) : 0.0f;
        } else {
          f[i] = __float_as_uint(x) - (kSumExp << 23) <= kSumExps << 23 ? 1.0f / x : NAN;
        }
      }
      ok = __all_sync(0xffffffffu, !*s_abort && wait_bar(&ofull[team], n & 1));
      if (!ok) break;
      tc_fence_after_sync();
      float chk[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // NaN if an output of the row is infinite or NaN
      uint16_t *dst[2];
      bool live[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + 8 * i;
        live[i] = r / G < b.nq;
        dst[i] = p.out + (static_cast<int64_t>(b.q0 + r / G) * p.Hkv * G + b.g * G + r % G) * kHeadDim + 8 * q2;
      }
#pragma unroll
      for (int c = 0; c < 128; c += 64) {
        uint32_t o[32], y[2][8];
        tmem_load_16x256b_x8(colo + c, o);
        tmem_wait_ld(o);
        if (c == 64) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ofree[team]);  // the team's next P V may overwrite O
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y0, y1;
            mul_f32x2(y0, y1, __uint_as_float(o[4 * j + 2 * i]), __uint_as_float(o[4 * j + 2 * i + 1]), f[i], f[i]);
            fma_f32x2(chk[2 * i], chk[2 * i + 1], y0, y1, 0.0f, 0.0f, chk[2 * i], chk[2 * i + 1]);
            y[i][j] = pack_bf16x2(y0, y1);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // the quad's lanes hold columns 2l, 2l + 1 of eight groups of eight; lane l takes the groups
          // 2l and 2l + 1, 32 bytes, so that the quad stores 128 bytes at once
          quad_transpose(y[i], lane);
          if (MODE == kPackedRelu2 && f[i] == 0.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = 0u;
          }
          if (live[i]) {
            const uint4 w0 = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
            const uint4 w1 = make_uint4(y[i][4], y[i][5], y[i][6], y[i][7]);
            if (p.out32) {  // whole sectors
              st_global_v8(dst[i] + c, w0, w1);
            } else {
              *reinterpret_cast<uint4 *>(dst[i] + c) = w0;
              *reinterpret_cast<uint4 *>(dst[i] + c + 8) = w1;
            }
          }
        }
        __syncwarp();
      }
      uint32_t bad = 0u;  // bit r: row rowa + r
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool weighs = MODE == kPackedSoftmax || f[i] != 0.0f;
        const uint32_t lanes = __ballot_sync(0xffffffffu, live[i] && weighs && chk[2 * i] + chk[2 * i + 1] != 0.0f);
        if (lanes == 0u) continue;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (lanes >> (4 * r) & 15u) bad |= 1u << (r + 8 * i);
      }
      if (bad != 0u) {
        __syncwarp();
        slow_rows<MODE, G, L::kSlowCols>(p, b, rowa, bad, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bempty[d]);
    }
    if (!ok) set_abort(s_abort, p.flags);
  }

  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) {
    // No copy may still be landing in shared memory when the CTA leaves.  Without an abort
    // every copy issued was waited for by the role that used it; after one, wait (bounded)
    // for the last armed phase of every barrier that a copy completes.
    const int nk = s_issued[0], nv = s_issued[1], nq = s_issued[2];
    for (int g = nk - 1; g >= 0 && g >= nk - kRingK; --g) wait_bar(&kfull[g % kRingK], (g / kRingK) & 1);
    for (int g = nv - 1; g >= 0 && g >= nv - kRing; --g) wait_bar(&vfull[g % kRing], (g / kRing) & 1);
    for (int k = nq - 1; k >= 0 && k >= nq - L::kQ; --k) wait_bar(&qfull[k % L::kQ], (k / L::kQ) & 1);
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// rk[g][j] = 1 / sqrt(mean(k_j^2) + eps): eight lanes per (key, KV head) row, 32 bytes each.  Also sets
// the attention kernel's ticket counter.
__global__ void __launch_bounds__(256) packed_knorm_kernel(const PackedPrefillParams p, float *rk) {
  pdl_wait_primary();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0u;
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
  // (a row of zeros with eps = 0 has no direction: it weighs nothing)
  const float z = a * (1.0f / kHeadDim) + p.eps;
  if (part == 0) rk[g * p.rk_stride + j] = z == 0.0f ? 0.0f : 1.0f / sqrtf(z);
}

template <int MODE, int N, int G, int TEAMS>
cudaError_t launch_packed(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                          const PackedPrefillParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  using L = Layout<MODE, N, TEAMS>;
  constexpr auto kernel = packed_prefill_kernel<MODE, N, G, TEAMS>;
  const cudaError_t e = allow_smem_once<kernel>(dev, L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t ctas = p.blocks < dev.sms ? p.blocks : dev.sms;  // one per SM
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(L::kThreads), static_cast<size_t>(L::kBytes),
                    stream, 0u, tm_q, tm_k, tm_v, p);
}

template <int G, int N, int TEAMS>
cudaError_t launch_kind(int mode, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                        const PackedPrefillParams &p, const LaunchDevice &dev, cudaStream_t stream) {
  if (mode == kPackedRelu2) return launch_packed<kPackedRelu2, N, G, TEAMS>(tm_q, tm_k, tm_v, p, dev, stream);
  return launch_packed<kPackedSoftmax, N, G, TEAMS>(tm_q, tm_k, tm_v, p, dev, stream);
}

}  // namespace

// Two teams on tiles of 80 are faster than one on tiles of 128, which waits at each block's ends, where blocks
// have few keys.  A block of 128 / G tokens sees window + 128 / G - 1 at most: up to about a thousand (2 x 16,384
// tokens, 4 KV heads, us: window 128 61 against 105, 256 87 and 125, 512 133 and 165, 1,024 240 and 238; 2 KV
// heads, 1,024 220 and 237; 2,048 393 against 380).  In a full layer it sees half of its sequence's on average:
// up to 1,500 keys to a sequence (8,192 tokens in sequences of 256 28.2 against 31.0, 512 31.8 and 35.2, 1,024
// 40.7 and 42.6, 2,048 58.9 and 58.6, 4,096 98.0 and 90.0).
constexpr int64_t kShortSpan = 1100, kShortContext = 1500;
int packed_tile_keys(int mode, int G, int64_t window, int64_t keys, int batch) {
  return (mode == kPackedSoftmax ? window + 128 / G - 1 <= kShortSpan : keys <= kShortContext * batch) ? 80 : 128;
}

int64_t packed_rk_stride(int64_t keys) { return (keys + 3) & ~static_cast<int64_t>(3); }

// The last tile's norms may be read up to a tile past the last row's; then the ticket counter.
static size_t packed_norm_bytes(int64_t keys, int Hkv) {
  return (static_cast<size_t>(Hkv) * static_cast<size_t>(packed_rk_stride(keys)) * 4 + 128 * 4 + 255) &
         ~static_cast<size_t>(255);
}
size_t packed_workspace_bytes(int64_t keys, int Hkv) { return packed_norm_bytes(keys, Hkv) + 256; }

int64_t packed_blocks(int64_t tokens, int batch, int G, int Hkv) { return (tokens / (128 / G) + batch) * Hkv; }

cudaError_t launch_packed_prefill(int mode, int G, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                  const CUtensorMap &tm_v, PackedPrefillParams p, float *rk,
                                  const LaunchDevice &dev, cudaStream_t stream) {
  if (p.blocks == 0) return cudaSuccess;
  p.ticket = nullptr;
  if (mode == kPackedRelu2 && p.keys > 0) {
    p.ticket = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(rk) + packed_norm_bytes(p.keys, p.Hkv));
    const int64_t rows = p.keys * p.Hkv;
    cudaError_t e = launch_pdl(packed_knorm_kernel, dim3(static_cast<unsigned>((rows + 31) / 32)), dim3(256), 0, stream,
                               0u, p, rk);
    if (e != cudaSuccess) return e;
  }
  const bool shorter = packed_tile_keys(mode, G, p.window, p.keys, p.batch) == 80;
  if (G == 4)
    return shorter ? launch_kind<4, 80, 2>(mode, tm_q, tm_k, tm_v, p, dev, stream)
                   : launch_kind<4, 128, 1>(mode, tm_q, tm_k, tm_v, p, dev, stream);
  if (G == 8)
    return shorter ? launch_kind<8, 80, 2>(mode, tm_q, tm_k, tm_v, p, dev, stream)
                   : launch_kind<8, 128, 1>(mode, tm_q, tm_k, tm_v, p, dev, stream);
  return cudaErrorInvalidValue;
}

}  // namespace embla
