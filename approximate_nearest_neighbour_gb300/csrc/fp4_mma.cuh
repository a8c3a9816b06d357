// Block-scaled 4-bit tensor-core products: operand copies, scale tiles, the
// instruction and the arguments shared by the narrow and the wide kernel.
#pragma once

#include "fp4.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ivfpq {

constexpr int BN = 128;            // columns of out (rows of b) per CTA

// Bytes of K per stage and row: 128, or 64 where all of K fits. A row is one
// request of the copy engine however much of it lies inside the matrix, and what
// lies outside costs more than what is read (77 x 100096 took 15.8 us at K = 128
// in boxes of 128 bytes, half of each outside, and 10.9 us at K = 256).
constexpr int kShortK = 128;  // columns

struct ProdArgs {
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  const float* a_ts;
  const float* b_ts;
  void* out;
  int64_t ldo;
  int64_t m, n;
  int kp;       // padded K
  int ntile;    // scale tiles along K
  int dtype;
  int overlap;  // launched to start while the kernel that writes a runs
  int* err;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Operand tile in shared memory: K-major rows of KB bytes, swizzled over KB bytes,
// 8-row groups 8 KB bytes apart.
template <int KB>
__device__ __forceinline__ uint64_t code_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(8 * KB >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(KB == 128 ? 2 : 4) << 61);
}
// Scale tile in shared memory: 32 rows of 16 bytes, no swizzle, 8-row groups
// 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}
// The issuing warp runs its loops converged, so that descriptors and addresses
// stay uniform, and one lane (el != 0) issues: a lane branching off alone made
// each scale copy cost 61 clocks and an empty step 800 (the operands move from
// vector registers one by one).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(e));
  return e;
}
// One scale tile to four TMEM columns of all four lane groups.
template <int CG>
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t desc, uint32_t el) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
        " @q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}" ::"r"(tmem),
        "l"(desc), "r"(el)
        : "memory");
  else
    asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}" ::"r"(tmem),
      "l"(desc), "r"(el)
      : "memory");
}
#define IVFPQ_MMA_FP4(GROUP, KIND)                                                               \
  asm volatile(                                                                                  \
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 q, %7, 0;\n"                    \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::" KIND                                         \
      " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),                                           \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(el)                            \
      : "memory")
template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sa, uint32_t sb, uint32_t acc, uint32_t el) {
  if (FMT == IVFPQ_MXFP4 && CG == 1) IVFPQ_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
  if (FMT == IVFPQ_NVFP4 && CG == 1) IVFPQ_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
  if (FMT == IVFPQ_MXFP4 && CG == 2) IVFPQ_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
  if (FMT == IVFPQ_NVFP4 && CG == 2) IVFPQ_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
}
#undef IVFPQ_MMA_FP4
__device__ __forceinline__ void mma_commit_el(uint32_t bar, uint32_t el) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          bar),
      "r"(el)
      : "memory");
}
// Instruction descriptor: E2M1 operands, K-major, M = 128 per CTA, N = T, the scale
// type, and (MXFP4) which half of a TMEM column's four scales this product
// uses.
template <int FMT, int T, int CG>
__device__ __forceinline__ uint32_t fp4_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(T >> 3) << 17) |
         (uint32_t(FMT == IVFPQ_MXFP4 ? 1 : 0) << 23) | (uint32_t(CG * BN >> 7) << 27) |
         (sf_id << 29);
}
__device__ __forceinline__ void store_out(void* out, int64_t at, int dtype, float v) {
  if (dtype == IVFPQ_F32)
    static_cast<float*>(out)[at] = v;
  else if (dtype == IVFPQ_BF16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(out)[at] = __float2half_rn(v);
}
// Tensor map over packed code rows; a box is kb bytes of K by box_rows rows.
int fp4_code_map(CUtensorMap* m, const uint8_t* p, int64_t rows, int64_t pitch, int kb,
                 int box_rows);

// The wide kernel (fp4_wide.cu).
int fp4_product_wide(const uint8_t* a, const uint8_t* b, const ProdArgs& p, int fmt,
                     cudaStream_t s);

}  // namespace ivfpq
