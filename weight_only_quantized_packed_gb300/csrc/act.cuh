// Primitives and formats of the quantised-activation GEMMs (gemm_act_few.cu,
// gemm_act_many.cu): tcgen05 with 8-bit operands, and with 4-bit operands
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

// The pair forms: two CTAs of a cluster (ranks 2i and 2i + 1) work on one
// 256-row tile. The even CTA issues for both: the same shared and tensor
// memory addresses are meant in each. Each CTA holds its 128 rows of A and of
// D, and half the rows of B.
__device__ __forceinline__ void pair_mma_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_mma_f4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sa,
                                            uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrives at this barrier of both CTAs when this thread's earlier pair
// operations are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// The same, at a barrier of this CTA alone.
__device__ __forceinline__ void pair_commit_own(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// A tile into this CTA's shared memory, completing on a barrier of either CTA
// of the pair (bar is a shared::cluster address).
__device__ __forceinline__ void pair_tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// mbar_arrive and mbar_arrive_expect_tx at a shared::cluster address. They
// order this CTA's own accesses only (a release at cluster scope costs about
// a microsecond, a stage's whole time): what the arrival announces is in this
// CTA's shared or tensor memory, complete behind a proxy or tcgen05 fence,
// and only tcgen05 operations of the pair use it.
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One float into a CTA's shared memory through a shared::cluster address,
// completing as 4 bytes on that CTA's mbarrier.
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v), "r"(bar)
               : "memory");
}

// A tile of this CTA's shared memory to global memory; rows and columns
// outside the map are dropped. One thread stores, closes a group after each
// place where a store may have been, and waits until all but the last N groups
// have been read before their shared memory is written again, or the CTA ends.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_store_close() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Whether a barrier's phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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

// 32 lanes x 32 or 16 columns from tensor memory without waiting; the
// registers are valid after tmem_ld_wait.
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
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor-memory loads; r stands for what they wrote,
// so that no use of it moves above the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// The same for further loads that a wait has covered.
__device__ __forceinline__ void tmem_ld_after(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two FP32 values in one register pair, (x, y) = (x, y) * f + (x, y)' and (x, y) * f.
__device__ __forceinline__ uint64_t pair_f32(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32);
}
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint64_t v, uint64_t f) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(f));
}
__device__ __forceinline__ void mul_f32x2(uint64_t& v, uint64_t f) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(f));
}

// ---------------------------------------------------------------- 4-bit scales
// A stage takes 16 scales (256 K) of every row: 16 bytes. The tensor core
// wants, per 64-K step, lane l of column i to hold the 4 scales of row
// 32 i + l of a 128-row block, and copy_scales takes that column group as 32
// rows of 16 bytes: step j of a block is the 512 bytes at 512 j. The tensor
// core reads the scales as unsigned: a code with its sign bit set becomes NaN,
// so that it cannot pass for a positive one.
constexpr int kScaleBlock = 2048;      // bytes of a 128-row block

__device__ __forceinline__ uint32_t scales_no_sign(uint32_t w) { return w | (((w & 0x80808080u) >> 7) * 0x7Fu); }

// A block of two stages that a tensor copy brought as rows of 32 bytes, made
// into the blocks of the two (2048 bytes each) in place by one warp. Only the
// first `rows` rows of the block exist. (Copied a stage at a time, as rows of 16
// bytes, the scales take twice the copies' time.)
__device__ __forceinline__ void rearrange_scales(uint8_t* block, int lane, int rows) {
  uint4 v[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4* p = reinterpret_cast<const uint4*>(block + (32 * i + lane) * 32);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[e][i] = 32 * i + lane < rows ? p[e] : make_uint4(0, 0, 0, 0);
      v[e][i].x = scales_no_sign(v[e][i].x);
      v[e][i].y = scales_no_sign(v[e][i].y);
      v[e][i].z = scales_no_sign(v[e][i].z);
      v[e][i].w = scales_no_sign(v[e][i].w);
    }
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint8_t* d = block + e * kScaleBlock + lane * 16;
    *reinterpret_cast<uint4*>(d) = make_uint4(v[e][0].x, v[e][1].x, v[e][2].x, v[e][3].x);
    *reinterpret_cast<uint4*>(d + 512) = make_uint4(v[e][0].y, v[e][1].y, v[e][2].y, v[e][3].y);
    *reinterpret_cast<uint4*>(d + 1024) = make_uint4(v[e][0].z, v[e][1].z, v[e][2].z, v[e][3].z);
    *reinterpret_cast<uint4*>(d + 1536) = make_uint4(v[e][0].w, v[e][1].w, v[e][2].w, v[e][3].w);
  }
}

// The same straight from global memory, through registers: warp `half` has
// the columns 2 half and 2 half + 1, so two rows of a block per thread. Rows
// that do not exist read the last one that does (their operand rows are
// zero). Where the weights stream from HBM this beats the tensor copies, whose
// 16-byte rows cost about as much time as 128-byte ones (1x34816x5120: 22.4 ->
// 19.3 us); in the kernel for many rows its latency is in the way (258 -> 374
// us at 4096x34816x5120).
struct ScaleRows {
  const uint8_t* p[2];
  __device__ __forceinline__ void at(const uint8_t* scales, int row0, int rows, int pitch, int half, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      p[e] = scales + static_cast<long long>(min(row0 + 64 * half + 32 * e + lane, rows - 1)) * pitch;
  }
  // kWeights: through the read-only path. The activations' scales may have been
  // written while this grid was already there (PDL), which that path does not
  // allow for.
  template <bool kWeights>
  __device__ __forceinline__ void load(int stage, uint4 (&v)[2]) const {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint4* q = reinterpret_cast<const uint4*>(p[e] + static_cast<long long>(stage) * 16);
      v[e] = kWeights ? __ldg(q) : *q;
    }
  }
};
__device__ __forceinline__ void put_scale_rows(uint8_t* block, int half, int lane, const uint4 (&v)[2]) {
  const uint32_t a[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, b[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint2*>(block + 512 * j + lane * 16 + half * 8) = make_uint2(scales_no_sign(a[j]), scales_no_sign(b[j]));
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
