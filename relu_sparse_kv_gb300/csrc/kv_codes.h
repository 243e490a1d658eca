// Launchers of the 8-bit caches' rows (kv_codes.cu), not part of the ABI.
#pragma once

#include "internal.h"

namespace embla {

// Rows of the 8-bit caches: `rows` = units * tokens packed bf16 rows (unit-major) quantised
// into rows pos .. pos + tokens - 1 of every plane of the K ([0]) and V ([1]) codes and
// scales, or those rows read back as bf16 into planes dst_stride rows apart.  rows < 2^31.
struct QuantizeJob {
  const uint16_t *src;
  uint8_t *codes;
  float *scales;
};
struct QuantizeParams {
  QuantizeJob job[2];
  int64_t rows, tokens, cache_stride, pos;
};
cudaError_t launch_quantize_rows(const QuantizeParams &p, cudaStream_t stream);
struct DequantizeJob {
  const uint8_t *codes;
  const float *scales;
  uint16_t *dst;
};
struct DequantizeParams {
  DequantizeJob job[2];
  int64_t rows, tokens, cache_stride, pos, dst_stride;
  int dst32;  // set by the launcher: both destinations start on 32 bytes
};
cudaError_t launch_dequantize_rows(DequantizeParams p, cudaStream_t stream);

}  // namespace embla
