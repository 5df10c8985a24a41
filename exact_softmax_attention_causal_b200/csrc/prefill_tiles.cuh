// What the prefill kernels share: the 128 x 128 tile's MMA steps, the output
// row's rescaling in TMEM, and the tensor map of a paged pool.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;  // query rows per tile (= TMEM lanes)
constexpr int kBN = 128;  // keys per tile

// Instruction descriptor for kind::f16: fp32 accumulate, bf16 A and B, A
// K-major, B K-major (0) or MN-major (1), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  if (status != nullptr) atomicOr(status, ATTN_STATUS_BIT_TIMEOUT);
}

// One MMA step of S = Q K^T: descriptors are the operand bases plus a fixed
// offset (16-byte units) added inside the asm, so the compiler cannot hoist a
// descriptor per step into registers.
template <uint32_t OFF, uint32_t IDESC>
__device__ __forceinline__ void mma_ss_step(uint32_t d_tmem, uint64_t a_base, uint64_t b_base, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %3, 0;\n add.s64 da, %1, %4;\n add.s64 db, %2, %4;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d_tmem),
      "l"(a_base), "l"(b_base), "r"(accumulate), "n"(OFF), "n"(IDESC)
      : "memory");
}
// One MMA step of O += P V with P in TMEM at column offset ACOL and V at OFF.
template <uint32_t ACOL, uint32_t OFF, uint32_t IDESC>
__device__ __forceinline__ void mma_ts_step(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_base, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 ta;\n .reg .b64 db;\n setp.ne.b32 p, %3, 0;\n add.u32 ta, %1, %4;\n"
      " add.s64 db, %2, %5;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %6, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_base), "r"(accumulate), "n"(ACOL), "n"(OFF), "n"(IDESC)
      : "memory");
}
// All D/16 steps of one score MMA (K dimension = head dim; 64-column boxes of
// 16 KB hold 4 steps of 32 bytes each).
template <int D, int KK = 0>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  constexpr uint32_t off = static_cast<uint32_t>(((KK >> 2) * (128 * 128) + (KK & 3) * 32) >> 4);
  mma_ss_step<off, idesc_bf16(kBM, kBN, 0)>(d_tmem, dq, dk, KK > 0 ? 1u : 0u);
  if constexpr (KK + 1 < D / 16) mma_scores<D, KK + 1>(d_tmem, dq, dk);
}
// Steps [KK, END) of one P.V MMA (16 keys per step: 8 TMEM columns of P, 2 KB of V).
template <int D, int KK, int END>
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t dv, bool first) {
  constexpr uint32_t voff = static_cast<uint32_t>((KK * 2048) >> 4);
  mma_ts_step<KK * 8, voff, idesc_bf16(kBM, D, 1)>(d_tmem, p_tmem, dv, (!first || KK > 0) ? 1u : 0u);
  if constexpr (KK + 1 < END) mma_pv<D, KK + 1, END>(d_tmem, p_tmem, dv, first);
}

// Warp-collective forms: every lane of a converged warp executes them and the
// lane that elect.sync picks issues four steps at a time. A branch on one lane
// leaves the compiler to find the lane for every instruction: a step then took
// about 100 cycles to issue, more than it takes to run at d = 64.
// d (+)= A B over four steps of 16 along the head dimension, operands from their bases.
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss4_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " setp.ne.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %4, t;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(accumulate), "n"(IDESC)
      : "memory");
}
// The same with A in TMEM, 8 columns a step, and B 2 KB a step (16 keys of V).
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts4_w(uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b32 a1, a2, a3;\n .reg .b64 b1, b2, b3;\n"
      " setp.ne.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
      " add.s64 b1, %2, 128;\n add.s64 b2, %2, 256;\n add.s64 b3, %2, 384;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, t;\n}\n" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(accumulate), "n"(IDESC)
      : "memory");
}
template <int D>
__device__ __forceinline__ void mma_scores_w(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  mma_ss4_w<idesc_bf16(kBM, kBN, 0)>(d_tmem, dq, dk, 0u);
  if constexpr (D == 128) mma_ss4_w<idesc_bf16(kBM, kBN, 0)>(d_tmem, dq + 1024, dk + 1024, 1u);
}
// Half of one P V: keys 0-63 (half 0) or 64-127 of a tile.
template <int D>
__device__ __forceinline__ void mma_pv_w(uint32_t d_tmem, uint32_t p_tmem, uint64_t dv, int half, bool first) {
  mma_ts4_w<idesc_bf16(kBM, D, 1)>(d_tmem, p_tmem + 32u * half, dv + 512ull * half, first && half == 0 ? 0u : 1u);
}

// Multiply this thread's TMEM output row by f (warp-collective).
template <int D>
__device__ __forceinline__ void rescale_row_t(uint32_t colO, float f) {
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t ov[16];
    tmem_ld_32x32b_x16(colO + c * 16, ov);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
    tmem_st_32x32b_x16(colO + c * 16, ov);
  }
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The paged pool [num_blocks][block_size][Hkv][d] bf16 as a rank-4 tensor
// (d, Hkv, slot, block); box = 64 columns x 1 head x box_slots slots x 1
// block, 128-byte swizzle: box_slots = block_size loads one block of one head,
// box_slots = 1 one token row.
bool encode_pool(CUtensorMap* map, const void* base, int d, int hkv, int block_size, int num_blocks,
                 int box_slots) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(hkv),
                              static_cast<cuuint64_t>(block_size), static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(hkv) * d * 2,
                                 static_cast<cuuint64_t>(block_size) * hkv * d * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_slots), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace
}  // namespace attn
