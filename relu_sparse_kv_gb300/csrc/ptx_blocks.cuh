// More inline-PTX building blocks (beside ptx.cuh): tiled copies of five dimensions and with cache
// hints, an elected issuing lane, tensor memory in the fragment layout of the warp MMAs, stores
// of whole sectors and predicated stores.
#pragma once

#include "ptx.cuh"

namespace embla {

// True in one lane of a converged warp (the same one each time): a warp that walks its loop
// together and issues from the elected lane keeps loop values and descriptors in uniform
// registers, which the tensor-core instructions take.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// 5-D tiled TMA load.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// tma_load_3d with an L2 cache policy (createpolicy result).
__device__ __forceinline__ void tma_load_3d_hint(void *dst, const CUtensorMap *map, uint64_t *bar,
                                                 int32_t x, int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 16 lanes x 16 consecutive 32-bit columns in the fragment layout of the warp MMAs: register
// 4j + 2i + e of lane l holds lane l / 4 + 8i of the 16, column 8j + 2(l % 4) + e.
__device__ __forceinline__ void tmem_load_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// 16 lanes x 8 consecutive 32-bit columns from registers: register 2j + i of lane l goes to
// lane l / 4 + 8i of the 16, column 4j + l % 4.
__device__ __forceinline__ void tmem_store_16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// 32 bytes to global memory in one store (dst 32-byte aligned).
__device__ __forceinline__ void st_global_v8(void *dst, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Two floats (dst 8-byte aligned) or one to global memory where `on` holds: a predicated store, no
// branch.
__device__ __forceinline__ void st_global_v2_if(bool on, float *dst, float a0, float a1) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "@p st.global.v2.f32 [%0], {%1, %2};\n\t}" ::"l"(dst),
      "f"(a0), "f"(a1), "r"(static_cast<uint32_t>(on))
      : "memory");
}
__device__ __forceinline__ void st_global_if(bool on, float *dst, float a) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p st.global.f32 [%0], %1;\n\t}" ::"l"(dst),
      "f"(a), "r"(static_cast<uint32_t>(on))
      : "memory");
}

// Four floats added to global memory (dst 16-byte aligned): the additions of one thread to one
// address happen in its order.
__device__ __forceinline__ void red_global_add_v4(float *dst, float a0, float a1, float a2, float a3) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "f"(a0), "f"(a1),
               "f"(a2), "f"(a3)
               : "memory");
}

// a - lo(w), b - hi(w) for the two bf16 values packed in w (each one rounding in fp32).
__device__ __forceinline__ void sub_bf16x2(uint32_t w, float &a, float &b) {
  asm("{\n\t.reg .b16 lo, hi, m;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "mov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, lo, m, %0;\n\t"
      "fma.rn.f32.bf16 %1, hi, m, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(w));
}

// Sum of squares of row r of a 128 x 128 bf16 tile in shared memory (two 64-column boxes of
// 128-byte rows).  Pieces are taken in an order that `turn` (0 .. 7) rotates, so lanes with
// different turns read different banks; the sum does not care which columns a piece holds.
__device__ __forceinline__ float row_square_sum(const uint8_t *tile, int box_bytes, int r, int turn) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 0.0f;
#pragma unroll 2
  for (int c = 0; c < 8; ++c) {
    const int pc = (c ^ turn) * 16;
    const uint4 x0 = *reinterpret_cast<const uint4 *>(tile + r * 128 + pc);
    const uint4 x1 = *reinterpret_cast<const uint4 *>(tile + box_bytes + r * 128 + pc);
    sq_acc_bf16x2(x0.x, a[0], a[1]);
    sq_acc_bf16x2(x0.y, a[2], a[3]);
    sq_acc_bf16x2(x0.z, a[4], a[5]);
    sq_acc_bf16x2(x0.w, a[6], a[7]);
    sq_acc_bf16x2(x1.x, a[0], a[1]);
    sq_acc_bf16x2(x1.y, a[2], a[3]);
    sq_acc_bf16x2(x1.z, a[4], a[5]);
    sq_acc_bf16x2(x1.w, a[6], a[7]);
  }
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

}  // namespace embla
