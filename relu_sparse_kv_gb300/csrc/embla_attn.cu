// C ABI of the library: host-side argument checks, workspace sizing, TMA descriptor
// encoding and the launches of the kernels in this directory.  Declarations and the
// meaning of every argument are in include/embla_attn.h.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "embla_attn.h"
#include "internal.h"
#include "kv_codes.h"
#include "ptx.cuh"
#include "ragged.h"
#include "shared_prefix.h"

using namespace embla;

// Scratch of embla_full_decode_static_scratch: one fixed array per device, so that
// call needs no workspace from its caller and allocates nothing itself.
static __device__ __align__(256) unsigned char g_full_scratch[EMBLA_FULL_DECODE_SCRATCH_BYTES];

namespace {

// Device-side check word (flag bits, see embla_device_check).
__device__ uint32_t g_check_flags;

constexpr int kMaxDevices = 64;

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev;
}

// Per-device values looked up once and kept.  Every slot is an atomic, filled at most
// once per device (a look-up that fails leaves the slot empty, so the next call retries);
// two host threads making their first call on a device at the same time may both look the
// value up, and both store the same value.
std::atomic<int> g_sm_count[kMaxDevices];
std::atomic<void *> g_flags_addr[kMaxDevices];
std::atomic<void *> g_scratch_addr[kMaxDevices];

int sm_count_of(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int v = g_sm_count[dev].load(std::memory_order_acquire);
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    g_sm_count[dev].store(v, std::memory_order_release);
  }
  return v;
}

// Device address of a __device__ symbol on the current device, cached in `slot`.
template <typename T>
void *symbol_address(std::atomic<void *> (&slot)[kMaxDevices], const T &symbol) {
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  void *p = slot[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    if (cudaGetSymbolAddress(&p, symbol) != cudaSuccess) return nullptr;
    slot[dev].store(p, std::memory_order_release);
  }
  return p;
}

uint32_t *flags_ptr() { return static_cast<uint32_t *>(symbol_address(g_flags_addr, g_check_flags)); }

// One thread waits, through the kernels' bounded wait, on a shared-memory barrier that
// nothing arrives at; when the limit runs out it records a timed-out wait in the check
// word, as a kernel's pipeline wait does, and returns.  If `arrive` is set the thread
// arrives first, so the wait succeeds at once and nothing is recorded.
__global__ void wait_limit_kernel(uint32_t *flags, uint64_t limit_ns, int arrive) {
  __shared__ uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  fence_barrier_init();
  if (arrive) mbar_arrive(&bar);
  if (!mbar_wait(&bar, 0u, limit_ns)) atomicOr(flags, kFlagWaitTimeout);
}

// Device address of g_full_scratch on the current device, looked up on the first
// call for that device and kept; nullptr if the look-up fails.
void *full_scratch_ptr() { return symbol_address(g_scratch_addr, g_full_scratch); }

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D bf16 tensor [rows, 128] with 256-byte rows, boxes of {64 columns, box_rows}, 128B swizzle.
bool encode_rows(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows,
                 CUtensorMapL2promotion promo) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kHeadDim), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kHeadDim * 2)};
  const cuuint32_t box[2] = {64u, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promo,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D uint8 tensor [rows, 128] of E4M3 codes (128-byte rows), boxes of {128 columns,
// box_rows}, 128B swizzle.
bool encode_rows_e4m3(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kHeadDim), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kHeadDim)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kHeadDim), box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D fp32 tensor [units, ncap] of per-token scales, boxes of {128 tokens, 1 unit}; tokens
// past ncap read as 0.
bool encode_scales(CUtensorMap *map, const float *base, uint64_t units, uint64_t ncap) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {ncap, units};
  const cuuint64_t strides[1] = {ncap * 4};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kTileKeys), 1u};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D bf16 tensor [planes][rows][128] (256-byte rows, planes `plane_rows` rows apart),
// boxes of {64 columns, 128 rows, 1 plane}, 128B swizzle; rows past `rows` read as zeros.
bool encode_planes(CUtensorMap *map, const void *base, uint64_t rows, uint64_t plane_rows,
                   uint64_t planes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), rows, planes};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim * 2), plane_rows * kHeadDim * 2};
  const cuuint32_t box[3] = {64u, 128u, 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 5-D bf16 map of q [batch][Hkv][4][G / 4][128] with the batch inside the groups of G / 4 heads,
// boxes of {64 columns, G / 4 heads, 32 / G sequences, 4 groups, 1 KV head}: 32 query rows of one
// KV head, in the order of the decode's row blocks; sequences past the batch read as zeros.
bool encode_query_block(CUtensorMap *map, const void *q, int batch, int Hq, int Hkv) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = kHeadDim * 2, G = static_cast<cuuint64_t>(Hq / Hkv);
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(kHeadDim), G / 4, static_cast<cuuint64_t>(batch), 4u,
                              static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[4] = {row, row * static_cast<cuuint64_t>(Hq), row * (G / 4), row * G};
  const cuuint32_t box[5] = {64u, static_cast<cuuint32_t>(G / 4), static_cast<cuuint32_t>(32 / G), 4u, 1u};
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed token rows [tokens][heads][128] bf16, `stride` elements between tokens, 128B swizzle.
// Queries: 4-D, boxes of {64 columns, G heads of one group, 128 / G tokens}, 128 rows token by token.
bool encode_packed_queries(CUtensorMap *map, const void *q, uint64_t tokens, uint64_t stride, int Hkv, int G) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = kHeadDim * 2, g = static_cast<cuuint64_t>(G);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim), g, static_cast<cuuint64_t>(Hkv), tokens};
  const cuuint64_t strides[3] = {row, row * g, stride * 2};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(G), 1u, static_cast<cuuint32_t>(128 / G)};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Keys or values: 3-D, boxes of {64 columns, 1 head, box_rows tokens}; rows past the last are zeros.
bool encode_packed_keys(CUtensorMap *map, const void *base, uint64_t rows, uint64_t stride, int Hkv,
                        uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(Hkv), rows};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim * 2), stride * 2};
  const cuuint32_t box[3] = {64u, 1u, box_rows};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool finite(float x) { return x == x && x - x == 0.0f; }

// Common shape checks; sets *G.  ctx_checks: also validate ctx_len / cache_stride.
embla_status check_shape(const embla_shape *s, int *G, bool ctx_checks) {
  if (!s) return EMBLA_ERR_INVALID_ARG;
  if (s->batch < 0 || s->n_q_heads < 1 || s->n_kv_heads < 1) return EMBLA_ERR_INVALID_ARG;
  if (s->n_q_heads % s->n_kv_heads) return EMBLA_ERR_INVALID_ARG;
  if (s->head_dim < 1) return EMBLA_ERR_INVALID_ARG;
  if (ctx_checks) {
    if (s->ctx_len < 0 || s->ctx_len > INT32_MAX) return EMBLA_ERR_INVALID_ARG;
    if (s->cache_stride < s->ctx_len) return EMBLA_ERR_INVALID_ARG;
  }
  *G = s->n_q_heads / s->n_kv_heads;
  if (s->head_dim != kHeadDim) return EMBLA_ERR_UNSUPPORTED;
  if (*G != 4 && *G != 8) return EMBLA_ERR_UNSUPPORTED;
  return EMBLA_OK;
}

// A shared prefix of `len` keys and the shape's own keys make a context of fewer than 2^31 keys
// (with room for a tile past its end).
bool prefix_fits(const embla_shape *s, int64_t len) {
  return len >= 0 && len <= INT32_MAX - 256 - s->ctx_len;
}

// Rows pos .. pos + count - 1 lie in the cache's planes.
bool rows_in_cache(const embla_shape *s, int64_t pos, int64_t count) {
  return s->cache_stride >= 0 && pos >= 0 && count >= 0 && pos <= s->cache_stride &&
         count <= s->cache_stride - pos;
}

// Packed rows of `heads` heads may lie `stride` elements apart: whole rows, 16-byte steps.
bool token_stride_ok(int64_t stride, int32_t heads) {
  return stride >= static_cast<int64_t>(heads) * kHeadDim && stride % 8 == 0;
}
constexpr int64_t kMaxPackedTokens = static_cast<int64_t>(1) << 30;  // and sequences
constexpr int64_t kMaxPackedStride = static_cast<int64_t>(1) << 38;  // TMA strides stay below 2^40 bytes

embla_status cuda_status(cudaError_t e) { return e == cudaSuccess ? EMBLA_OK : EMBLA_ERR_CUDA; }

}  // namespace

extern "C" {

const char *embla_status_string(embla_status status) {
  switch (status) {
    case EMBLA_OK: return "ok";
    case EMBLA_ERR_INVALID_ARG: return "invalid argument";
    case EMBLA_ERR_UNSUPPORTED: return "unsupported shape (head_dim must be 128, G in {4, 8})";
    case EMBLA_ERR_WORKSPACE: return "workspace too small";
    case EMBLA_ERR_CUDA: return "CUDA error";
    case EMBLA_ERR_DEVICE_CHECK: return "device-side check failed";
  }
  return "unknown status";
}

int embla_device_sm_count(void) { return sm_count_of(current_device()); }

size_t embla_full_decode_workspace_size(const embla_shape *shape) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK) return 0;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return 0;
  return full_workspace_bytes(
      full_split(static_cast<int64_t>(shape->batch) * shape->n_kv_heads, shape->ctx_len, sms), G);
}

}  // extern "C"

namespace {

// The selection requested together with a full-layer decode.
struct SelectArgs {
  int32_t topk, recent;
  int32_t *idx;
  int32_t idx_stride;
  int32_t *count;
};

// The full-layer decode for bf16 caches (k_scales and v_scales null) or 8-bit E4M3 caches
// with per-token scales; with sa, followed by the selection over its scores (the workspace
// then holds the decode's records, then the selection's workspace).
embla_status full_decode_impl(const embla_shape *shape, const void *q, const void *k_cache,
                              const float *k_scales, const void *v_cache, const float *v_scales,
                              bool kv8, float alpha, float c, float eps, float *out,
                              int32_t *n_surv, float *sel_scores, uint32_t *sel_hist,
                              void *workspace, size_t workspace_bytes, void *stream,
                              float *head_scores = nullptr, uint32_t *head_hist = nullptr,
                              int max_pieces = kMaxPiecesPerCta,
                              const SelectArgs *sa = nullptr) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (!(finite(alpha) && alpha > 0.0f) || !(finite(c) && c >= 0.0f) ||
      !(finite(eps) && eps >= 0.0f))
    return EMBLA_ERR_INVALID_ARG;
  // the scale arrays are read as [units, cache_stride] with 16-byte aligned rows
  if (kv8 && shape->cache_stride % 4 != 0) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!q || !k_cache || !v_cache || !out || !n_surv || !workspace) return EMBLA_ERR_INVALID_ARG;
  if (kv8 && (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)))
    return EMBLA_ERR_INVALID_ARG;
  if ((sel_scores == nullptr) != (sel_hist == nullptr)) return EMBLA_ERR_INVALID_ARG;
  if (sa && (!sel_scores || sa->topk < 0 || sa->recent < 0 ||
             static_cast<int64_t>(sa->topk) + sa->recent > INT32_MAX ||
             sa->idx_stride < sa->topk + sa->recent || !sa->idx || !sa->count ||
             !aligned16(sa->idx) || !aligned16(sa->count)))
    return EMBLA_ERR_INVALID_ARG;
  if ((head_scores == nullptr) != (head_hist == nullptr)) return EMBLA_ERR_INVALID_ARG;
  if (head_scores && (!aligned16(head_scores) || !aligned16(head_hist)))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace) || (sel_scores && (!aligned16(sel_scores) || !aligned16(sel_hist))))
    return EMBLA_ERR_INVALID_ARG;
  // TMA row coordinates are 32-bit
  if (units * shape->cache_stride + kTileKeys > INT32_MAX) return EMBLA_ERR_UNSUPPORTED;
  const int dev = current_device();
  const int sms = sm_count_of(dev);
  if (sms <= 0) return EMBLA_ERR_CUDA;
  const FullSplit sp = full_split(units, shape->ctx_len, sms, max_pieces);
  const size_t rec_bytes = full_workspace_bytes(sp, G);
  const size_t sel_bytes = sa ? select_workspace_bytes(units, shape->ctx_len) : 0;
  if (workspace_bytes < rec_bytes + sel_bytes) return EMBLA_ERR_WORKSPACE;
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  if (sp.tiles == 0) {
    // no keys: every output is 0, nothing survives, the histogram is empty
    if (sel_scores)
      st = cuda_status(cudaMemsetAsync(sel_hist, 0, static_cast<size_t>(units) * kHistBins * 4, s));
    if (st == EMBLA_OK && head_scores)
      st = cuda_status(cudaMemsetAsync(head_hist, 0,
                                       static_cast<size_t>(shape->batch) * shape->n_q_heads * kHistBins * 4, s));
    if (st == EMBLA_OK)
      st = cuda_status(cudaMemsetAsync(out, 0, static_cast<size_t>(units) * G * kHeadDim * 4, s));
    if (st == EMBLA_OK) st = cuda_status(cudaMemsetAsync(n_surv, 0, static_cast<size_t>(units) * 4, s));
    if (st == EMBLA_OK && sa)  // no keys to select
      st = cuda_status(cudaMemsetAsync(sa->count, 0, static_cast<size_t>(units) * 4, s));
    return st;
  }
  // the launch zeroes the histogram and the survivor counts itself
  const uint64_t rows = static_cast<uint64_t>(units * shape->cache_stride);
  CUtensorMap tm_k, tm_q, tm_ks, tm_vs;
  const bool kmap = kv8 ? encode_rows_e4m3(&tm_k, k_cache, rows, kTileKeys)
                        : encode_rows(&tm_k, k_cache, rows, kTileKeys,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (!kmap ||
      !encode_rows(&tm_q, q, static_cast<uint64_t>(shape->batch) * shape->n_q_heads,
                   static_cast<uint32_t>(G), CU_TENSOR_MAP_L2_PROMOTION_NONE))
    return EMBLA_ERR_CUDA;
  if (kv8 && (!encode_scales(&tm_ks, k_scales, static_cast<uint64_t>(units),
                             static_cast<uint64_t>(shape->cache_stride)) ||
              !encode_scales(&tm_vs, v_scales, static_cast<uint64_t>(units),
                             static_cast<uint64_t>(shape->cache_stride))))
    return EMBLA_ERR_CUDA;
  SelectJob sj = {};
  if (sa) {
    sj.topk = sa->topk;
    sj.recent = sa->recent;
    sj.idx = sa->idx;
    sj.idx_stride = sa->idx_stride;
    sj.count = sa->count;
    sj.workspace = sel_bytes ? static_cast<uint8_t *>(workspace) + rec_bytes : nullptr;
    sj.sm_count = sms;
  }
  st = cuda_status(launch_full_decode(G, kv8, tm_k, tm_q, kv8 ? &tm_ks : nullptr,
                                      kv8 ? &tm_vs : nullptr, v_cache, sel_scores, head_scores,
                                      sel_hist, workspace, out, n_surv, c, flags, sp,
                                      shape->ctx_len, shape->cache_stride, shape->n_q_heads,
                                      shape->n_kv_heads, alpha, eps, s, sa ? &sj : nullptr));
  if (st == EMBLA_OK && head_scores)
    st = cuda_status(launch_score_hist(head_scores,
                                       static_cast<int64_t>(shape->batch) * shape->n_q_heads,
                                       shape->ctx_len, shape->cache_stride, head_hist, s));
  return st;
}

}  // namespace

extern "C" {

embla_status embla_full_decode(const embla_shape *shape, const void *q, const void *k_cache,
                               const void *v_cache, float alpha, float c, float eps, float *out,
                               int32_t *n_surv, float *sel_scores, uint32_t *sel_hist,
                               void *workspace, size_t workspace_bytes, void *stream) {
  return full_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, alpha, c, eps,
                          out, n_surv, sel_scores, sel_hist, workspace, workspace_bytes, stream);
}

embla_status embla_full_decode_head_scores(const embla_shape *shape, const void *q,
                                           const void *k_cache, const void *v_cache, float alpha,
                                           float c, float eps, float *out, int32_t *n_surv,
                                           float *head_scores, uint32_t *head_hist,
                                           void *workspace, size_t workspace_bytes, void *stream) {
  if (!head_scores || !head_hist) return EMBLA_ERR_INVALID_ARG;
  return full_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, alpha, c, eps,
                          out, n_surv, nullptr, nullptr, workspace, workspace_bytes, stream,
                          head_scores, head_hist);
}

embla_status embla_full_decode_e4m3(const embla_shape *shape, const void *q,
                                    const uint8_t *k_codes, const float *k_scales,
                                    const uint8_t *v_codes, const float *v_scales, float alpha,
                                    float c, float eps, float *out, int32_t *n_surv,
                                    float *sel_scores, uint32_t *sel_hist, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  return full_decode_impl(shape, q, k_codes, k_scales, v_codes, v_scales, true, alpha, c, eps,
                          out, n_surv, sel_scores, sel_hist, workspace, workspace_bytes, stream);
}

size_t embla_full_decode_select_workspace_size(const embla_shape *shape, int32_t topk,
                                               int32_t recent) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK || topk < 0 || recent < 0) return 0;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return 0;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  return full_workspace_bytes(full_split(units, shape->ctx_len, sms), G) +
         select_workspace_bytes(units, shape->ctx_len);
}

embla_status embla_full_decode_select(const embla_shape *shape, const void *q, const void *k_cache,
                                      const void *v_cache, float alpha, float c, float eps,
                                      float *out, int32_t *n_surv, float *sel_scores,
                                      uint32_t *sel_hist, int32_t topk, int32_t recent,
                                      int32_t *idx, int32_t idx_stride, int32_t *count,
                                      void *workspace, size_t workspace_bytes, void *stream) {
  const SelectArgs sa = {topk, recent, idx, idx_stride, count};
  return full_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, alpha, c, eps, out,
                          n_surv, sel_scores, sel_hist, workspace, workspace_bytes, stream, nullptr,
                          nullptr, kMaxPiecesPerCta, &sa);
}

embla_status embla_full_decode_e4m3_select(const embla_shape *shape, const void *q,
                                           const uint8_t *k_codes, const float *k_scales,
                                           const uint8_t *v_codes, const float *v_scales,
                                           float alpha, float c, float eps, float *out,
                                           int32_t *n_surv, float *sel_scores, uint32_t *sel_hist,
                                           int32_t topk, int32_t recent, int32_t *idx,
                                           int32_t idx_stride, int32_t *count, void *workspace,
                                           size_t workspace_bytes, void *stream) {
  const SelectArgs sa = {topk, recent, idx, idx_stride, count};
  return full_decode_impl(shape, q, k_codes, k_scales, v_codes, v_scales, true, alpha, c, eps, out,
                          n_surv, sel_scores, sel_hist, workspace, workspace_bytes, stream, nullptr,
                          nullptr, kMaxPiecesPerCta, &sa);
}

embla_status embla_full_decode_static_scratch(const embla_shape *shape, const void *q,
                                              const void *k_cache, const void *v_cache,
                                              float alpha, float c, float eps, float *out,
                                              int32_t *n_surv, float *sel_scores,
                                              uint32_t *sel_hist, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  // fewer pieces per CTA (fewer records) where the usual split's records do not fit
  int max_pieces = kMaxPiecesPerCta;
  size_t need = full_workspace_bytes(full_split(units, shape->ctx_len, sms, max_pieces), G);
  while (need > EMBLA_FULL_DECODE_SCRATCH_BYTES && max_pieces > 1) {
    max_pieces -= 2;
    need = full_workspace_bytes(full_split(units, shape->ctx_len, sms, max_pieces), G);
  }
  if (need > EMBLA_FULL_DECODE_SCRATCH_BYTES) return EMBLA_ERR_WORKSPACE;
  void *scratch = full_scratch_ptr();
  if (!scratch) return EMBLA_ERR_CUDA;
  return full_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, alpha, c, eps, out,
                          n_surv, sel_scores, sel_hist, scratch, need, stream, nullptr, nullptr,
                          max_pieces);
}

size_t embla_select_topk_workspace_size(const embla_shape *shape, int32_t topk, int32_t recent) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK || topk < 0 || recent < 0) return 0;
  return select_workspace_bytes(static_cast<int64_t>(shape->batch) * shape->n_kv_heads,
                                shape->ctx_len);
}

embla_status embla_select_topk(const embla_shape *shape, const float *sel_scores,
                               const uint32_t *sel_hist, int32_t topk, int32_t recent,
                               int32_t *idx, int32_t idx_stride, int32_t *count, void *workspace,
                               size_t workspace_bytes, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (topk < 0 || recent < 0 || static_cast<int64_t>(topk) + recent > INT32_MAX ||
      idx_stride < topk + recent)
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  const size_t ws_need = select_workspace_bytes(units, shape->ctx_len);
  if (!sel_scores || !sel_hist || !idx || !count || (ws_need && !workspace))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(sel_scores) || !aligned16(sel_hist) || !aligned16(idx) || !aligned16(count) ||
      (workspace && !aligned16(workspace)))
    return EMBLA_ERR_INVALID_ARG;
  if (workspace_bytes < ws_need) return EMBLA_ERR_WORKSPACE;
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  return cuda_status(launch_select(sel_scores, sel_hist, units, shape->ctx_len,
                                   shape->cache_stride, topk, recent, idx, idx_stride, count,
                                   workspace, flags, sms, static_cast<cudaStream_t>(stream)));
}

size_t embla_select_topk_per_head_workspace_size(const embla_shape *shape, int32_t topk,
                                                  int32_t recent) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK || topk < 0 || recent < 0) return 0;
  return select_workspace_bytes(static_cast<int64_t>(shape->batch) * shape->n_q_heads,
                                shape->ctx_len);
}

embla_status embla_select_topk_per_head(const embla_shape *shape, const float *head_scores,
                                        const uint32_t *head_hist, int32_t topk, int32_t recent,
                                        int32_t *idx, int32_t idx_stride, int32_t *count,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (topk < 0 || recent < 0 || static_cast<int64_t>(topk) + recent > INT32_MAX ||
      idx_stride < topk + recent)
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_q_heads;
  if (units == 0) return EMBLA_OK;
  const size_t ws_need = select_workspace_bytes(units, shape->ctx_len);
  if (!head_scores || !head_hist || !idx || !count || (ws_need && !workspace))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(head_scores) || !aligned16(head_hist) || !aligned16(idx) || !aligned16(count) ||
      (workspace && !aligned16(workspace)))
    return EMBLA_ERR_INVALID_ARG;
  if (workspace_bytes < ws_need) return EMBLA_ERR_WORKSPACE;
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  return cuda_status(launch_select(head_scores, head_hist, units, shape->ctx_len,
                                   shape->cache_stride, topk, recent, idx, idx_stride, count,
                                   workspace, flags, sms, static_cast<cudaStream_t>(stream)));
}

size_t embla_sparse_decode_workspace_size(const embla_shape *shape, int32_t idx_stride) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK || idx_stride < 0) return 0;
  return sparse_workspace_bytes(static_cast<int64_t>(shape->batch) * shape->n_kv_heads, G,
                                idx_stride);
}

}  // extern "C"

namespace {

embla_status sparse_decode_impl(const embla_shape *shape, const void *q, const void *k_cache,
                                const float *k_scales, const void *v_cache,
                                const float *v_scales, bool kv8, const int32_t *idx,
                                int32_t idx_stride, const int32_t *count, float tau, float *out,
                                void *workspace, size_t workspace_bytes, void *stream,
                                bool per_head = false) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (!finite(tau) || idx_stride < 0) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) *
                       (per_head ? shape->n_q_heads : shape->n_kv_heads);
  if (units == 0) return EMBLA_OK;
  if (!q || !k_cache || !v_cache || !idx || !count || !out || !workspace)
    return EMBLA_ERR_INVALID_ARG;
  if (kv8 && (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace) || !aligned16(idx) || !aligned16(count))
    return EMBLA_ERR_INVALID_ARG;
  if (workspace_bytes < sparse_workspace_bytes(units, G, idx_stride)) return EMBLA_ERR_WORKSPACE;
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  return cuda_status(launch_sparse_decode(G, per_head, shape->n_q_heads, q, k_cache, v_cache,
                                          kv8 ? k_scales : nullptr,
                                          kv8 ? v_scales : nullptr, idx, idx_stride, count,
                                          units, shape->n_kv_heads, shape->ctx_len,
                                          shape->cache_stride, tau, out, workspace, flags, sms,
                                          static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

embla_status embla_sparse_decode(const embla_shape *shape, const void *q, const void *k_cache,
                                 const void *v_cache, const int32_t *idx, int32_t idx_stride,
                                 const int32_t *count, float tau, float *out, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  return sparse_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, idx, idx_stride,
                            count, tau, out, workspace, workspace_bytes, stream);
}

embla_status embla_sparse_decode_per_head(const embla_shape *shape, const void *q,
                                          const void *k_cache, const void *v_cache,
                                          const int32_t *idx, int32_t idx_stride,
                                          const int32_t *count, float tau, float *out,
                                          void *workspace, size_t workspace_bytes, void *stream) {
  return sparse_decode_impl(shape, q, k_cache, nullptr, v_cache, nullptr, false, idx, idx_stride,
                            count, tau, out, workspace, workspace_bytes, stream, true);
}

embla_status embla_sparse_decode_e4m3(const embla_shape *shape, const void *q,
                                      const uint8_t *k_codes, const float *k_scales,
                                      const uint8_t *v_codes, const float *v_scales,
                                      const int32_t *idx, int32_t idx_stride,
                                      const int32_t *count, float tau, float *out,
                                      void *workspace, size_t workspace_bytes, void *stream) {
  return sparse_decode_impl(shape, q, k_codes, k_scales, v_codes, v_scales, true, idx,
                            idx_stride, count, tau, out, workspace, workspace_bytes, stream);
}

size_t embla_prefill_workspace_size(const embla_shape *shape) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK) return 0;
  return prefill_workspace_bytes(static_cast<int64_t>(shape->batch) * shape->n_kv_heads,
                                 shape->ctx_len);
}

embla_status embla_prefill(const embla_shape *shape, int64_t n_new, const void *q,
                           const void *k_cache, const void *v_cache, float alpha, float c,
                           float eps, float *out, void *workspace, size_t workspace_bytes,
                           void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (n_new < 0 || n_new > shape->ctx_len) return EMBLA_ERR_INVALID_ARG;
  if (!(finite(alpha) && alpha > 0.0f) || !(finite(c) && c >= 0.0f) ||
      !(finite(eps) && eps >= 0.0f))
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0 || n_new == 0) return EMBLA_OK;
  if (!q || !k_cache || !v_cache || !out || !workspace) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return EMBLA_ERR_INVALID_ARG;
  // TMA coordinates are 32-bit; one CTA per (sequence, head, 128 prompt tokens)
  const int64_t bh = static_cast<int64_t>(shape->batch) * shape->n_q_heads;
  if (shape->ctx_len > INT32_MAX - 256 || bh > INT32_MAX || bh * ((n_new + 127) / 128) > INT32_MAX)
    return EMBLA_ERR_UNSUPPORTED;
  if (workspace_bytes < prefill_workspace_bytes(units, shape->ctx_len)) return EMBLA_ERR_WORKSPACE;
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  float *rk = static_cast<float *>(workspace);
  CUtensorMap tm_q, tm_k, tm_v, tm_rk;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return EMBLA_ERR_CUDA;
  const cuuint64_t rdims[2] = {static_cast<cuuint64_t>(shape->ctx_len), static_cast<cuuint64_t>(units)};
  const cuuint64_t rstrides[1] = {static_cast<cuuint64_t>(prefill_rk_stride(shape->ctx_len)) * 4};
  const cuuint32_t rbox[2] = {128u, 1u};
  const cuuint32_t restr[2] = {1u, 1u};
  if (!encode_planes(&tm_q, q, static_cast<uint64_t>(n_new), static_cast<uint64_t>(n_new),
                     static_cast<uint64_t>(bh)) ||
      !encode_planes(&tm_k, k_cache, static_cast<uint64_t>(shape->ctx_len),
                     static_cast<uint64_t>(shape->cache_stride), static_cast<uint64_t>(units)) ||
      !encode_planes(&tm_v, v_cache, static_cast<uint64_t>(shape->ctx_len),
                     static_cast<uint64_t>(shape->cache_stride), static_cast<uint64_t>(units)) ||
      fn(&tm_rk, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, rk, rdims, rstrides, rbox, restr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return EMBLA_ERR_CUDA;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  return cuda_status(launch_prefill(tm_q, tm_k, tm_v, tm_rk, k_cache, rk, out, flags, shape->batch,
                                    shape->n_q_heads, shape->n_kv_heads, shape->ctx_len, n_new,
                                    shape->cache_stride, alpha, c, eps, sms,
                                    static_cast<cudaStream_t>(stream)));
}

size_t embla_full_decode_shared_workspace_size(const embla_shape *shape, int64_t prefix_len) {
  int G = 0;
  if (check_shape(shape, &G, true) != EMBLA_OK || !prefix_fits(shape, prefix_len)) return 0;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return 0;
  return shared_workspace_bytes(
      shared_split(shape->batch, shape->n_kv_heads, G, prefix_len, shape->ctx_len, sms));
}

embla_status embla_full_decode_shared(const embla_shape *shape, int64_t prefix_len,
                                      int64_t prefix_stride, const void *q, const void *k_prefix,
                                      const void *v_prefix, const void *k_cache,
                                      const void *v_cache, float alpha, float c, float eps,
                                      float *out, int32_t *n_surv, float *sel_scores,
                                      int64_t score_stride, uint32_t *sel_hist, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (!prefix_fits(shape, prefix_len) || prefix_stride < prefix_len) return EMBLA_ERR_INVALID_ARG;
  if (!(finite(alpha) && alpha > 0.0f) || !(finite(c) && c >= 0.0f) ||
      !(finite(eps) && eps >= 0.0f))
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  const int64_t n = shape->ctx_len;
  if (units == 0) return EMBLA_OK;
  if (!q || !out || !n_surv || (prefix_len > 0 && (!k_prefix || !v_prefix)) ||
      (n > 0 && (!k_cache || !v_cache)) || (prefix_len + n > 0 && !workspace))
    return EMBLA_ERR_INVALID_ARG;
  if ((sel_scores == nullptr) != (sel_hist == nullptr)) return EMBLA_ERR_INVALID_ARG;
  if (sel_scores && score_stride < prefix_len + n) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out) || !aligned16(n_surv) || !aligned16(sel_scores) ||
      !aligned16(sel_hist) || !aligned16(workspace))
    return EMBLA_ERR_INVALID_ARG;
  // TMA plane coordinates and the second kernel's grid are 32-bit
  if (units * G > INT32_MAX / 2) return EMBLA_ERR_UNSUPPORTED;
  // TMA strides stay below 2^40 bytes
  if (prefix_stride > UINT32_MAX || shape->cache_stride > UINT32_MAX) return EMBLA_ERR_UNSUPPORTED;
  const int dev = current_device();
  const int sms = sm_count_of(dev);  // 0 past kMaxDevices
  if (sms <= 0) return EMBLA_ERR_CUDA;
  const SharedSplit sp = shared_split(shape->batch, shape->n_kv_heads, G, prefix_len, n, sms);
  if (!sp.fits()) return EMBLA_ERR_UNSUPPORTED;
  if (workspace_bytes < shared_workspace_bytes(sp)) return EMBLA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sp.ctas() == 0) {
    // no keys: every output is 0, nothing survives, the histogram is empty
    if (sel_hist)
      st = cuda_status(cudaMemsetAsync(sel_hist, 0, static_cast<size_t>(units) * kHistBins * 4, s));
    if (st == EMBLA_OK)
      st = cuda_status(cudaMemsetAsync(out, 0, static_cast<size_t>(units) * G * kHeadDim * 4, s));
    if (st == EMBLA_OK) st = cuda_status(cudaMemsetAsync(n_surv, 0, static_cast<size_t>(units) * 4, s));
    return st;
  }
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  // Planes of the prefix and of the own caches; a side without keys has no tiles, and its maps
  // stand in for nothing.
  CUtensorMap tm_q, tm_kp, tm_vp, tm_ko, tm_vo;
  const uint64_t planes = static_cast<uint64_t>(shape->n_kv_heads);
  if (prefix_len > 0 &&
      (!encode_planes(&tm_kp, k_prefix, static_cast<uint64_t>(prefix_len),
                      static_cast<uint64_t>(prefix_stride), planes) ||
       !encode_planes(&tm_vp, v_prefix, static_cast<uint64_t>(prefix_len),
                      static_cast<uint64_t>(prefix_stride), planes)))
    return EMBLA_ERR_CUDA;
  if (n > 0 && (!encode_planes(&tm_ko, k_cache, static_cast<uint64_t>(n),
                               static_cast<uint64_t>(shape->cache_stride), static_cast<uint64_t>(units)) ||
                !encode_planes(&tm_vo, v_cache, static_cast<uint64_t>(n),
                               static_cast<uint64_t>(shape->cache_stride), static_cast<uint64_t>(units))))
    return EMBLA_ERR_CUDA;
  if (n == 0) tm_ko = tm_kp, tm_vo = tm_vp;
  if (prefix_len == 0) tm_kp = tm_ko, tm_vp = tm_vo;
  if (!encode_query_block(&tm_q, q, shape->batch, shape->n_q_heads, shape->n_kv_heads)) return EMBLA_ERR_CUDA;
  SharedCall a = {};
  a.tm_q = &tm_q;
  a.tm_kp = &tm_kp;
  a.tm_vp = &tm_vp;
  a.tm_ko = &tm_ko;
  a.tm_vo = &tm_vo;
  a.q = q;
  a.k_prefix = k_prefix;
  a.v_prefix = v_prefix;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.prefix_stride = prefix_stride;
  a.cache_stride = shape->cache_stride;
  a.sel_scores = sel_scores;
  a.sel_hist = sel_hist;
  a.score_stride = score_stride;
  a.workspace = workspace;
  a.out = out;
  a.n_surv = n_surv;
  a.flags = flags;
  a.alpha = alpha;
  a.c = c;
  a.eps = eps;
  a.group = G;
  a.device = dev;
  a.sm_count = sms;
  return cuda_status(launch_shared_decode(a, sp, s));
}

embla_status embla_sparse_decode_shared(const embla_shape *shape, int64_t prefix_len,
                                        int64_t prefix_stride, const void *q, const void *k_prefix,
                                        const void *v_prefix, const void *k_cache,
                                        const void *v_cache, const int32_t *idx,
                                        int32_t idx_stride, const int32_t *count, float tau,
                                        float *out, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (!prefix_fits(shape, prefix_len) || prefix_stride < prefix_len) return EMBLA_ERR_INVALID_ARG;
  if (!finite(tau) || idx_stride < 0) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!q || !idx || !count || !out || (prefix_len > 0 && (!k_prefix || !v_prefix)) ||
      (shape->ctx_len > 0 && (!k_cache || !v_cache)))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(idx) || !aligned16(count) || !aligned16(out))
    return EMBLA_ERR_INVALID_ARG;
  if (units > INT32_MAX / 8) return EMBLA_ERR_UNSUPPORTED;  // the grid, in clusters of 8
  uint32_t *flags = flags_ptr();
  if (!flags) return EMBLA_ERR_CUDA;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  const SharedRows prefix = {k_prefix, v_prefix, prefix_len, prefix_stride};
  return cuda_status(launch_sparse_decode_shared(
      G, shape->n_q_heads, q, prefix, k_cache, v_cache, idx, idx_stride, count, units, shape->n_kv_heads,
      prefix_len + shape->ctx_len, shape->cache_stride, tau, out, flags, sms, static_cast<cudaStream_t>(stream)));
}

size_t embla_relu2_mlp_workspace_size(int64_t d, int64_t f) {
  const int sms = sm_count_of(current_device());
  if (sms <= 0 || d < 1 || f < 1) return 0;
  return mlp_workspace_bytes(d, f, sms);
}

embla_status embla_relu2_mlp(int64_t d, int64_t f, const void *x, const void *w_up,
                             const void *w_down, float *y, int32_t *n_live, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (d != 512 && d != 1024 && d != 2048) return d < 1 ? EMBLA_ERR_INVALID_ARG : EMBLA_ERR_UNSUPPORTED;
  if (f < 1 || f > (static_cast<int64_t>(1) << 30)) return EMBLA_ERR_INVALID_ARG;
  if (!x || !w_up || !w_down || !y || !n_live || !workspace) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_up) || !aligned16(w_down) || !aligned16(y) ||
      !aligned16(n_live) || !aligned16(workspace))
    return EMBLA_ERR_INVALID_ARG;
  const int sms = sm_count_of(current_device());
  if (sms <= 0) return EMBLA_ERR_CUDA;
  if (workspace_bytes < mlp_workspace_bytes(d, f, sms)) return EMBLA_ERR_WORKSPACE;
  return cuda_status(launch_relu2_mlp(x, w_up, w_down, d, f, y, n_live, workspace, sms,
                                      static_cast<cudaStream_t>(stream)));
}

size_t embla_window_decode_workspace_size(const embla_shape *shape, int32_t window) {
  (void)shape;
  (void)window;
  return 0;
}

embla_status embla_window_decode(const embla_shape *shape, const void *q, const void *k_win,
                                 const void *v_win, int32_t window, int64_t pos, float rope_base,
                                 float tau, float *out, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  (void)workspace;
  (void)workspace_bytes;
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (window < 1 || window > 1024 || pos < 0 || !(finite(rope_base) && rope_base > 0.0f) ||
      !finite(tau))
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!q || !k_win || !v_win || !out) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_win) || !aligned16(v_win) || !aligned16(out))
    return EMBLA_ERR_INVALID_ARG;
  return cuda_status(launch_window_decode(G, q, k_win, v_win, units, window, pos, rope_base, tau,
                                          out, static_cast<cudaStream_t>(stream)));
}

embla_status embla_rope_qkv(const embla_shape *shape, int64_t n_tokens, const int32_t *cu_tokens,
                            const int32_t *pos0, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, float rope_base,
                            int norm, float eps, const float *q_gain, const float *k_gain,
                            void *q_out, void *k_out, int32_t window, void *k_win, void *v_win,
                            void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (n_tokens < 0 || !(finite(rope_base) && rope_base > 0.0f)) return EMBLA_ERR_INVALID_ARG;
  if (norm ? !(finite(eps) && eps >= 0.0f) : (q_gain || k_gain)) return EMBLA_ERR_INVALID_ARG;
  const bool ring = k_win || v_win;
  if (ring && (!k_win || !v_win || window < 1 || window > 1024)) return EMBLA_ERR_INVALID_ARG;
  if (n_tokens == 0 || shape->batch == 0) return EMBLA_OK;
  if (!cu_tokens || !q || !k || !q_out || (ring && !v)) return EMBLA_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, shape->n_q_heads) || !token_stride_ok(k_stride, shape->n_kv_heads) ||
      (ring && !token_stride_ok(v_stride, shape->n_kv_heads)))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(cu_tokens) || !aligned16(pos0) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(q_gain) || !aligned16(k_gain) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(k_win) || !aligned16(v_win))
    return EMBLA_ERR_INVALID_ARG;
  if (n_tokens > kMaxPackedTokens || shape->batch > kMaxPackedTokens || n_tokens * shape->n_kv_heads > INT32_MAX)
    return EMBLA_ERR_UNSUPPORTED;
  if (q_stride > kMaxPackedStride || k_stride > kMaxPackedStride || (ring && v_stride > kMaxPackedStride))
    return EMBLA_ERR_UNSUPPORTED;
  RopeParams p = {};
  p.seqs = {cu_tokens, n_tokens, shape->batch};
  p.pos0 = pos0;
  p.q = {static_cast<const uint16_t *>(q), q_stride};
  p.k = {static_cast<const uint16_t *>(k), k_stride};
  p.v = {static_cast<const uint16_t *>(v), v_stride};
  p.q_out = static_cast<uint16_t *>(q_out);
  p.k_out = static_cast<uint16_t *>(k_out);
  p.k_win = static_cast<uint16_t *>(k_win);
  p.v_win = static_cast<uint16_t *>(v_win);
  p.q_gain = q_gain;
  p.k_gain = k_gain;
  p.eps = eps;
  p.norm = norm ? 1 : 0;
  p.window = window;
  p.Hkv = shape->n_kv_heads;
  // the fraction of a circle that each pair turns by per position (whole circles do not count): one power,
  // and 63 products (a relative error of i 2^-53 where f has fallen to base^(-i/64))
  const double step = std::pow(static_cast<double>(rope_base), -2.0 / kHeadDim);
  double f = 1.0 / 6.283185307179586476925286766559;
  for (int i = 0; i < kHeadDim / 2; ++i, f *= step)
    p.turn[i] = static_cast<uint64_t>((f - std::floor(f)) * 0x1p64);
  return cuda_status(launch_rope_qkv(G, p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Causal attention over packed prompts; the caller fills in what belongs to the kind of weights.
embla_status packed_prefill_impl(int mode, const embla_shape *shape, int G, int64_t n_tokens,
                                 const int32_t *cu_tokens, int64_t n_keys, const int32_t *cu_keys,
                                 const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                 const void *v, int64_t v_stride, int64_t window, PackedPrefillParams p,
                                 void *out, void *workspace, size_t workspace_bytes, void *stream) {
  if (n_tokens < 0 || n_keys < 0 || (!cu_keys && n_keys != n_tokens)) return EMBLA_ERR_INVALID_ARG;
  if (n_tokens == 0 || shape->batch == 0) return EMBLA_OK;
  const bool norms = mode == kPackedRelu2 && n_keys > 0;
  if (!cu_tokens || !q || !out || (n_keys > 0 && (!k || !v)) || (norms && !workspace)) return EMBLA_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, shape->n_q_heads) ||
      (n_keys > 0 && (!token_stride_ok(k_stride, shape->n_kv_heads) || !token_stride_ok(v_stride, shape->n_kv_heads))))
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(cu_tokens) || !aligned16(cu_keys) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(out) || !aligned16(workspace))
    return EMBLA_ERR_INVALID_ARG;
  if (n_tokens > kMaxPackedTokens || n_keys > kMaxPackedTokens || shape->batch > kMaxPackedTokens ||
      n_keys * shape->n_kv_heads > INT32_MAX)
    return EMBLA_ERR_UNSUPPORTED;
  if (q_stride > kMaxPackedStride || (n_keys > 0 && (k_stride > kMaxPackedStride || v_stride > kMaxPackedStride)))
    return EMBLA_ERR_UNSUPPORTED;
  p.blocks = packed_blocks(n_tokens, shape->batch, G, shape->n_kv_heads);
  if (p.blocks > INT32_MAX) return EMBLA_ERR_UNSUPPORTED;
  if (norms && workspace_bytes < packed_workspace_bytes(n_keys, shape->n_kv_heads)) return EMBLA_ERR_WORKSPACE;
  LaunchDevice dev = {current_device(), 0};
  dev.sms = sm_count_of(dev.index);  // 0 past kMaxDevices
  p.flags = flags_ptr();
  if (dev.sms <= 0 || !p.flags) return EMBLA_ERR_CUDA;
  if (window > kMaxPackedTokens) window = kMaxPackedTokens;  // more than any sequence has
  const uint32_t rows = static_cast<uint32_t>(packed_tile_keys(mode, G, window, n_keys, shape->batch));
  CUtensorMap tm_q, tm_k, tm_v;
  // (without keys no tile is loaded, and the maps of K and V stand in for nothing)
  if (n_keys == 0) {
    k = v = q;
    k_stride = v_stride = q_stride;
  }
  const uint64_t map_rows = static_cast<uint64_t>(n_keys > 0 ? n_keys : 1);
  if (!encode_packed_queries(&tm_q, q, static_cast<uint64_t>(n_tokens), static_cast<uint64_t>(q_stride),
                             shape->n_kv_heads, G) ||
      !encode_packed_keys(&tm_k, k, map_rows, static_cast<uint64_t>(k_stride), shape->n_kv_heads, rows) ||
      !encode_packed_keys(&tm_v, v, map_rows, static_cast<uint64_t>(v_stride), shape->n_kv_heads, rows))
    return EMBLA_ERR_CUDA;
  p.cu_q = cu_tokens;
  p.cu_k = cu_keys ? cu_keys : cu_tokens;
  p.q = {static_cast<const uint16_t *>(q), q_stride};
  p.k = {static_cast<const uint16_t *>(k), k_stride};
  p.v = {static_cast<const uint16_t *>(v), v_stride};
  p.rk = static_cast<const float *>(workspace);
  p.out = static_cast<uint16_t *>(out);
  p.tokens = n_tokens;
  p.keys = n_keys;
  p.rk_stride = packed_rk_stride(n_keys);
  p.batch = shape->batch;
  p.Hkv = shape->n_kv_heads;
  p.window = static_cast<int32_t>(window);
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 ? 1 : 0;
  return cuda_status(launch_packed_prefill(mode, G, tm_q, tm_k, tm_v, p, static_cast<float *>(workspace), dev,
                                           static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

embla_status embla_window_prefill(const embla_shape *shape, int64_t n_tokens, const int32_t *cu_tokens,
                                  int64_t n_keys, const int32_t *cu_keys, const void *q,
                                  int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                  int64_t v_stride, int64_t window, float tau, void *out,
                                  void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (window < 1 || !finite(tau)) return EMBLA_ERR_INVALID_ARG;
  PackedPrefillParams p = {};
  // scores are kept in base 2; a scale of zero stays above it, so that unseen keys at minus infinity do
  p.tau2 = tau == 0.0f ? 0x1p-100f : tau * 1.4426950408889634f;
  return packed_prefill_impl(kPackedSoftmax, shape, G, n_tokens, cu_tokens, n_keys, cu_keys, q, q_stride, k, k_stride,
                             v, v_stride, window, p, out, nullptr, 0, stream);
}

size_t embla_prefill_packed_workspace_size(const embla_shape *shape, int64_t n_keys) {
  int G = 0;
  if (check_shape(shape, &G, false) != EMBLA_OK || n_keys < 1 || n_keys > kMaxPackedTokens) return 0;
  return packed_workspace_bytes(n_keys, shape->n_kv_heads);
}

embla_status embla_prefill_packed(const embla_shape *shape, int64_t n_tokens, const int32_t *cu_tokens,
                                  int64_t n_keys, const int32_t *cu_keys, const void *q,
                                  int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                  int64_t v_stride, float alpha, float c, float eps, void *out,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (!(finite(alpha) && alpha > 0.0f) || !(finite(c) && c >= 0.0f) || !(finite(eps) && eps >= 0.0f))
    return EMBLA_ERR_INVALID_ARG;
  PackedPrefillParams p = {};
  p.alpha = alpha;
  p.c = c;
  p.eps = eps;
  return packed_prefill_impl(kPackedRelu2, shape, G, n_tokens, cu_tokens, n_keys, cu_keys, q, q_stride, k, k_stride, v,
                             v_stride, kMaxPackedTokens, p, out, workspace, workspace_bytes, stream);
}

embla_status embla_window_decode_ragged(const embla_shape *shape, const void *q, const void *k_win,
                                        const void *v_win, int32_t window, const int32_t *pos,
                                        float tau, float *out, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (window < 1 || window > 1024 || !finite(tau)) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!q || !k_win || !v_win || !pos || !out) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_win) || !aligned16(v_win) || !aligned16(pos) || !aligned16(out))
    return EMBLA_ERR_INVALID_ARG;
  if (units > INT32_MAX / 8) return EMBLA_ERR_UNSUPPORTED;
  const RaggedWindowParams p = {static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(k_win),
                                static_cast<const uint8_t *>(v_win), pos, out, shape->n_kv_heads, window,
                                tau * 1.4426950408889634f};
  LaunchDevice dev = {current_device(), 0};
  dev.sms = sm_count_of(dev.index);  // 0 past kMaxDevices
  if (dev.sms <= 0) return EMBLA_ERR_CUDA;
  return cuda_status(launch_window_decode_ragged(G, units, p, dev, static_cast<cudaStream_t>(stream)));
}

embla_status embla_skip_stats(const embla_shape *shape, const float *sel_scores, int32_t chunk,
                              int32_t *keys_needed, int32_t *chunks_needed, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, true);
  if (st != EMBLA_OK) return st;
  if (chunk < 1 || chunk > 1024 || (chunk & (chunk - 1)) != 0) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!sel_scores || !keys_needed || !chunks_needed) return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(sel_scores) || !aligned16(keys_needed) || !aligned16(chunks_needed))
    return EMBLA_ERR_INVALID_ARG;
  return cuda_status(launch_skip_stats(sel_scores, units, shape->ctx_len, shape->cache_stride,
                                       chunk, keys_needed, chunks_needed,
                                       static_cast<cudaStream_t>(stream)));
}

embla_status embla_append_kv(const embla_shape *shape, int64_t pos, const void *k_rows,
                             const void *v_rows, void *k_cache, void *v_cache, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (shape->cache_stride < 1 || pos < 0 || pos >= shape->cache_stride)
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!k_rows || !v_rows || !k_cache || !v_cache) return EMBLA_ERR_INVALID_ARG;
  const int64_t rb = 2 * kHeadDim;
  const AppendJob jobs[2] = {
      {static_cast<const uint8_t *>(k_rows), static_cast<uint8_t *>(k_cache), rb, shape->cache_stride, 0},
      {static_cast<const uint8_t *>(v_rows), static_cast<uint8_t *>(v_cache), rb, shape->cache_stride, 0}};
  return cuda_status(launch_append_rows(jobs, 2, units, pos, static_cast<cudaStream_t>(stream)));
}

embla_status embla_append_kv_e4m3(const embla_shape *shape, int64_t pos, const uint8_t *k_code_rows,
                                  const float *k_scale_rows, const uint8_t *v_code_rows,
                                  const float *v_scale_rows, uint8_t *k_codes, float *k_scales,
                                  uint8_t *v_codes, float *v_scales, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (shape->cache_stride < 1 || pos < 0 || pos >= shape->cache_stride)
    return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0) return EMBLA_OK;
  if (!k_code_rows || !k_scale_rows || !v_code_rows || !v_scale_rows || !k_codes || !k_scales ||
      !v_codes || !v_scales)
    return EMBLA_ERR_INVALID_ARG;
  const int64_t ncap = shape->cache_stride;
  const AppendJob jobs[4] = {
      {k_code_rows, k_codes, kHeadDim, ncap, 0},
      {v_code_rows, v_codes, kHeadDim, ncap, 0},
      {reinterpret_cast<const uint8_t *>(k_scale_rows), reinterpret_cast<uint8_t *>(k_scales), 4, ncap, 0},
      {reinterpret_cast<const uint8_t *>(v_scale_rows), reinterpret_cast<uint8_t *>(v_scales), 4, ncap, 0}};
  return cuda_status(launch_append_rows(jobs, 4, units, pos, static_cast<cudaStream_t>(stream)));
}

embla_status embla_quantize_kv_e4m3(const embla_shape *shape, int64_t pos, int64_t n_new,
                                    const void *k_rows, const void *v_rows, uint8_t *k_codes,
                                    float *k_scales, uint8_t *v_codes, float *v_scales,
                                    void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (!rows_in_cache(shape, pos, n_new)) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0 || n_new == 0) return EMBLA_OK;
  if (!k_rows || !v_rows || !k_codes || !k_scales || !v_codes || !v_scales)
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_codes) || !aligned16(v_codes) ||
      !aligned16(k_scales) || !aligned16(v_scales))
    return EMBLA_ERR_INVALID_ARG;
  if (n_new > INT32_MAX / units) return EMBLA_ERR_UNSUPPORTED;
  const QuantizeParams p = {
      {{static_cast<const uint16_t *>(k_rows), k_codes, k_scales},
       {static_cast<const uint16_t *>(v_rows), v_codes, v_scales}},
      units * n_new, n_new, shape->cache_stride, pos};
  return cuda_status(launch_quantize_rows(p, static_cast<cudaStream_t>(stream)));
}

embla_status embla_dequantize_kv_e4m3(const embla_shape *shape, int64_t pos, int64_t n_rows,
                                      const uint8_t *k_codes, const float *k_scales,
                                      const uint8_t *v_codes, const float *v_scales, void *k_rows,
                                      void *v_rows, int64_t rows_stride, void *stream) {
  int G = 0;
  embla_status st = check_shape(shape, &G, false);
  if (st != EMBLA_OK) return st;
  if (!rows_in_cache(shape, pos, n_rows) || rows_stride < n_rows) return EMBLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(shape->batch) * shape->n_kv_heads;
  if (units == 0 || n_rows == 0) return EMBLA_OK;
  if (!k_rows || !v_rows || !k_codes || !k_scales || !v_codes || !v_scales)
    return EMBLA_ERR_INVALID_ARG;
  if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_codes) || !aligned16(v_codes) ||
      !aligned16(k_scales) || !aligned16(v_scales))
    return EMBLA_ERR_INVALID_ARG;
  if (n_rows > INT32_MAX / units) return EMBLA_ERR_UNSUPPORTED;
  const DequantizeParams p = {
      {{k_codes, k_scales, static_cast<uint16_t *>(k_rows)},
       {v_codes, v_scales, static_cast<uint16_t *>(v_rows)}},
      units * n_rows, n_rows, shape->cache_stride, pos, rows_stride, 0};
  return cuda_status(launch_dequantize_rows(p, static_cast<cudaStream_t>(stream)));
}

embla_status embla_self_test_wait_limit(uint32_t limit_us, int arrive, void *stream) {
  if (limit_us == 0 || limit_us > 1000000u) return EMBLA_ERR_INVALID_ARG;
  uint32_t *d = flags_ptr();
  if (!d) return EMBLA_ERR_CUDA;
  wait_limit_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      d, static_cast<uint64_t>(limit_us) * 1000ull, arrive);
  return cuda_status(cudaGetLastError());
}

embla_status embla_device_check(uint32_t *flags, int clear, void *stream) {
  uint32_t *d = flags_ptr();
  if (!d || !flags) return d ? EMBLA_ERR_INVALID_ARG : EMBLA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, d, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return EMBLA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return EMBLA_ERR_CUDA;
  if (clear && v) {
    if (cudaMemsetAsync(d, 0, sizeof(uint32_t), s) != cudaSuccess) return EMBLA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return EMBLA_ERR_CUDA;
  }
  *flags = v;
  return v ? EMBLA_ERR_DEVICE_CHECK : EMBLA_OK;
}

}  // extern "C"
