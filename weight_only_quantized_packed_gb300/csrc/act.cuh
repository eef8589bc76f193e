// Primitives and formats of the quantised-activation GEMMs (gemm_act_rows.cu,
// gemm_act_cols.cu): tcgen05 with 8-bit operands, and with 4-bit operands
// whose scales the tensor core applies itself.
#pragma once
#include "decode.cuh"
#include "tc.cuh"

namespace wqp {
namespace act {

using namespace tc;

// ---------------------------------------------------------------- MMA
// D[tmem] (+)= A * B^T, both operands from shared memory, E4M3, K = 32.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with E2M1 operands, K = 64, and an unsigned E4M3 scale per row and
// 16 K of each operand from tensor memory (sa, sb).
__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes from shared memory into 4 columns of tensor memory,
// repeated in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// mma_commit, arriving at the same barrier of every CTA of the cluster in mask.
__device__ __forceinline__ void mma_commit_multicast(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
// tma_load_2d into the same place of every CTA of the cluster in mask, each
// completing on its own barrier at that place.
__device__ __forceinline__ void tma_load_2d_multicast(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                                      uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "h"(mask)
      : "memory");
}

// Instruction descriptors: N >> 3 at bits 17..22, M >> 4 at bits 24..28; FP32
// accumulation. E4M3 operands are format 0; E2M1 with block scales is format
// 1 of both operands, the scale type (bit 23) 0 for E4M3.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x NC columns from tensor memory without waiting; the registers are
// valid after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- 4-bit scales
// A raw stage holds a row's 16 scales (256 K) as 16 bytes. The tensor core
// wants, per 64-K step, lane l of column i to hold the 4 scales of row
// 32 i + l, and copy_scales takes that column group as 32 rows of 16 bytes:
// step j of a 128-row block is the 512 bytes at dst + 512 j. `half` (0, 1)
// does the steps 2 half and 2 half + 1; only the first `rows` rows exist. The
// tensor core reads the scales as unsigned: a code with its sign bit set
// becomes NaN, so that it cannot pass for a positive one.
constexpr int kScaleBlock = 2048;      // bytes of a 128-row block, raw or rearranged

__device__ __forceinline__ uint32_t scales_no_sign(uint32_t w) { return w | (((w & 0x80808080u) >> 7) * 0x7Fu); }

__device__ __forceinline__ void rearrange_scales(const uint8_t* raw, uint8_t* dst, int half, int lane, int rows) {
  uint2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = make_uint2(0, 0);
    if (32 * i + lane < rows) v[i] = *reinterpret_cast<const uint2*>(raw + (32 * i + lane) * 16 + 8 * half);
    v[i].x = scales_no_sign(v[i].x);
    v[i].y = scales_no_sign(v[i].y);
  }
  uint8_t* d = dst + half * 1024 + lane * 16;
  *reinterpret_cast<uint4*>(d) = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
  *reinterpret_cast<uint4*>(d + 512) = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
}
// Copy one rearranged 64-K step (at saddr) into 4 columns.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) { return sdesc(saddr, 16, 128, 0); }

// Row-major operand tile of 128-byte rows, 128-byte swizzle, 8-row atoms.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) { return sdesc(saddr, 16, 1024, 2); }

// ---------------------------------------------------------------- formats
// A stage is 128 bytes of every operand row: 256 4-bit or 128 8-bit elements,
// four MMA steps of 32 bytes either way.
struct F4 {
  static constexpr bool kScaled = true;     // the tensor core applies the scales
  static constexpr int kStageK = 256;
};
struct F8 {
  static constexpr bool kScaled = false;    // the epilogue folds them per 128 K
  static constexpr int kStageK = 128;
};

}  // namespace act
}  // namespace wqp
