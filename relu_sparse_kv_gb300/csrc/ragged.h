// Launchers of the calls on batches whose sequences have different lengths (rope.cu,
// window_ragged.cu, packed_prefill.cu), not part of the ABI.
#pragma once

#include <atomic>

#include "internal.h"

namespace embla {

// The device that a call launches on (its index below 64), and its number of SMs.
struct LaunchDevice {
  int index, sms;
};

// Raises a kernel's limit of dynamic shared memory, once per device.
template <auto Kernel>
cudaError_t allow_smem_once(const LaunchDevice &dev, int bytes) {
  static std::atomic<uint64_t> done;  // a bit per device
  const uint64_t bit = uint64_t{1} << dev.index;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Packed tokens: sequence b of `batch` is tokens cu[b] .. cu[b + 1] - 1 of `tokens`.
struct PackedTokens {
  const int32_t *cu;
  int64_t tokens;
  int batch;
};

// Rows of packed tokens in memory: head h of token t at base + t * stride + h * kHeadDim elements.
struct TokenRows {
  const uint16_t *base;
  int64_t stride;
};

struct RopeParams {
  PackedTokens seqs;
  const int32_t *pos0;  // position of each sequence's first token; null: 0
  TokenRows q, k, v;
  uint16_t *q_out, *k_out;  // k_out null: not written
  uint16_t *k_win, *v_win;  // both null: no rings
  const float *q_gain, *k_gain;
  float eps;
  int norm, window, Hkv;
  uint64_t turn[kHeadDim / 2];  // pair i turns by turn[i] * 2^-64 of a circle per position
};
cudaError_t launch_rope_qkv(int G, const RopeParams &p, cudaStream_t stream);

// Rows 0 .. min(pos[b] + 1, window) - 1 of every ring of sequence b.
struct RaggedWindowParams {
  const uint16_t *q;
  const uint8_t *K, *V;
  const int32_t *pos;
  float *out;
  int32_t Hkv, window;
  float tau2;  // tau * log2(e)
};
cudaError_t launch_window_decode_ragged(int G, int64_t units, const RaggedWindowParams &p,
                                        const LaunchDevice &dev, cudaStream_t stream);

// Causal attention over packed prompts (kinds of weights).
constexpr int kPackedSoftmax = 0, kPackedRelu2 = 1;
struct PackedPrefillParams {
  const int32_t *cu_q, *cu_k;  // queries and keys of each sequence
  TokenRows q, k, v;
  const float *rk;             // ReLU^2: 1 / norm of every key row, [Hkv, rk_stride]
  uint32_t *ticket;            // ReLU^2: block numbers drawn past each CTA's first (set by the launcher)
  uint16_t *out;               // [tokens, Hq, 128] bf16
  uint32_t *flags;
  int64_t tokens, keys, rk_stride;
  int64_t blocks;              // packed_blocks
  int32_t batch, Hkv, window;  // window: keys a query sees at most
  int32_t out32;               // out starts on 32 bytes
  float tau2;                  // softmax: tau * log2(e), not 0
  float alpha, c, eps;         // ReLU^2
};
// Keys per tile (the rows of the K and V maps' boxes) and block numbers to walk.
int packed_tile_keys(int mode, int G, int64_t window, int64_t keys, int batch);
int64_t packed_blocks(int64_t tokens, int batch, int G, int Hkv);
int64_t packed_rk_stride(int64_t keys);
size_t packed_workspace_bytes(int64_t keys, int Hkv);
cudaError_t launch_packed_prefill(int mode, int G, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                  const CUtensorMap &tm_v, PackedPrefillParams p, float *rk,
                                  const LaunchDevice &dev, cudaStream_t stream);

}  // namespace embla
