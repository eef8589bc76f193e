// Products of quantised activations with packed weights, many rows: 4-bit by
// 4-bit with E4M3 scales per 16 K, and 8-bit by 8-bit with FP32 scales per
// 128 K.
//
// Bound by the tensor core, so a tile is as wide as the MMA allows: 128
// activation rows (the MMA's M side, one tensor-memory lane each) by BN weight
// rows. Persistent CTAs, one per SM, walk over the tiles; with CL = 2 a
// cluster of two takes two row tiles of the same weights, and each CTA loads
// half of the weight tile for both.
//  * 4 bits: the tensor core applies the scales (act.cuh: rearranged by two
//    warps, copied to tensor memory by the MMA warp). One accumulator, drained
//    into registers as BF16 before the next tile's first MMA.
//  * 8 bits: two accumulators that take turns per 128 K; the epilogue adds each,
//    times its activation row's and weight block's scale, to FP32 sums in
//    registers while the tensor core fills the other.
//
// Warps: 0 copies, 1 MMA (and tensor memory), 2..3 scales (4 bits), 4..11
// epilogue: lane quarter = warp % 4, column half = (warp - 4) / 4.
#include "act.cuh"

namespace wqp {
namespace act {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4;

constexpr uint32_t kScaleCol = 256;    // 4 bits: two sets of a stage's scales

struct ManyParams {
  const float* SA;
  const float* SW;
  float gscale;
  uint16_t* C;
  int M, N, K, ldc;
  int mt, nt;           // row tiles in units of CL, weight tiles
  int stages;           // per tile
  int vec;              // C rows are 16-byte aligned
  unsigned* err;
};

template <class F, int BN, int CL>
struct ManyLayout {
  static constexpr int kAux = F::kScaled ? 2 * kScaleBlock * (1 + BN / 128) : 0;
  static constexpr int kStageBytes = 16384 + BN * 128 + kAux;
  static constexpr int kS = (220 * 1024) / kStageBytes;
  static constexpr int kA = 0;
  static constexpr int kB = kA + kS * 16384;
  static constexpr int kRawA = kB + kS * BN * 128;
  static constexpr int kRawB = kRawA + (F::kScaled ? kS * kScaleBlock : 0);
  static constexpr int kSclA = kRawB + (F::kScaled ? kS * kScaleBlock * (BN / 128) : 0);
  static constexpr int kSclB = kSclA + (F::kScaled ? kS * kScaleBlock : 0);
  static constexpr int kBytes = kSclB + (F::kScaled ? kS * kScaleBlock * (BN / 128) : 0);
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr int kLoad = 16384 + BN * 128 + kAux / 2;     // bytes that arrive per stage
  static constexpr int kAcc = F::kScaled ? 1 : 2;
  static_assert(kAlloc <= 227 * 1024 - 1024, "shared memory");
};

// Tile i of the walk: groups of 8 row tiles go through all weight tiles, row
// tiles first, so that the tiles in flight share both operands in L2.
__device__ __forceinline__ void tile_at(int i, int mt, int nt, int& m, int& n) {
  constexpr int G = 8;
  const int per = G * nt;
  const int g = i / per, rows = min(G, mt - g * G);
  const int j = i - g * per;
  n = j / rows;
  m = g * G + (j - n * rows);
}

template <class F, int BN, int CL>
__global__ void __launch_bounds__(kThreads, 1)
    many_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, ManyParams p) {
  using L = ManyLayout<F, BN, CL>;
  constexpr int S = L::kS, NACC = L::kAcc, COLS = BN / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_sh[S], empty_sh[S], scaled_sh[S], acc_full_sh[NACC], acc_free_sh[NACC], drained_sh;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CL > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / CL, step = gridDim.x / CL, total = p.mt * p.nt;
  const uint32_t full = smem_u32(full_sh), empty = smem_u32(empty_sh), scaled = smem_u32(scaled_sh);
  const uint32_t acc_full = smem_u32(acc_full_sh), acc_free = smem_u32(acc_free_sh);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, CL);
      mbar_init(scaled + 8 * i, 2);
    }
    for (int i = 0; i < NACC; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_free + 8 * i, 8);
    }
    mbar_init(smem_u32(&drained_sh), 1);
    abort_sh = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  if (CL > 1) cluster_sync();                  // every barrier exists before a peer's copy or arrive
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_launch_dependents();

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      int it = 0;
      if (lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        pdl_wait();
        bool live = true;
        for (int i = first; i < total && live; i += step) {
          int mi, ni;
          tile_at(i, p.mt, p.nt, mi, ni);
          const int m0 = (mi * CL + rank) * 128, n0 = ni * BN;
          for (int k = 0; k < p.stages; ++k, ++it) {
            const int s = it % S;
            if (it >= S && !wait_or_abort(empty + 8 * s, ((it / S) - 1) & 1, p.err, abort_flag)) {
              live = false;
              break;
            }
            const uint32_t bar = full + 8 * s;
            mbar_arrive_expect_tx(bar, L::kLoad);
            tma_load_2d(sb + L::kA + s * 16384, &tmA, k * 128, m0, bar);
            const uint32_t db = sb + L::kB + s * BN * 128;
            if (F::kScaled) tma_load_2d(sb + L::kRawA + s * kScaleBlock, &tmSA, k * 16, m0, bar);
            const uint32_t ds = sb + L::kRawB + s * kScaleBlock * (BN / 128);
            if (CL == 1) {
              tma_load_2d(db, &tmB, k * 128, n0, bar);
              if (F::kScaled) tma_load_2d(ds, &tmSB, k * 16, n0, bar);
            } else {
              constexpr int R = BN / CL;
              tma_load_2d_multicast(db + rank * R * 128, &tmB, k * 128, n0 + rank * R, bar, (1 << CL) - 1);
              if (F::kScaled) tma_load_2d_multicast(ds + rank * R * 16, &tmSB, k * 16, n0 + rank * R, bar, (1 << CL) - 1);
            }
          }
        }
        // Every stage has been consumed here and by the peer, and the peer's
        // arrivals have come, before the CTA may exit.
        for (int t = it > S ? it - S : 0; t < it; ++t)
          if (!wait_or_abort(empty + 8 * (t % S), (t / S) & 1, p.err, abort_flag))
            mbar_wait(full + 8 * (t % S), (t / S) & 1, p.err);
      }
      __syncwarp();
    } else if (warp == 1) {
      constexpr uint32_t idesc = F::kScaled ? idesc_f4(128, BN) : idesc_f8(128, BN);
      int it = 0, blk = 0;                     // stages, and accumulators handed over
      bool live = true;
      for (int i = first; i < total && live; i += step) {
        for (int k = 0; k < p.stages; ++k, ++it) {
          const int s = it % S, slot = blk % NACC;
          bool ok = wait_or_abort(full + 8 * s, (it / S) & 1, p.err, abort_flag);
          if (F::kScaled) ok = ok && wait_or_abort(scaled + 8 * s, (it / S) & 1, p.err, abort_flag);
          if ((!F::kScaled || k == 0) && blk >= NACC)
            ok = ok && wait_or_abort(acc_free + 8 * slot, ((blk / NACC) - 1) & 1, p.err, abort_flag);
          live = __all_sync(0xFFFFFFFFu, ok);
          if (!live) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = tile_desc(sb + L::kA + s * 16384), bd = tile_desc(sb + L::kB + s * BN * 128);
            if constexpr (F::kScaled) {
              constexpr int NB = BN / 128;
              const uint32_t sa = tmem + kScaleCol + (it & 1) * 64, sw = sa + 16;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                copy_scales(sa + 4 * j, scale_desc(sb + L::kSclA + s * kScaleBlock + 512 * j));
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  copy_scales(sw + (j * NB + b) * 4,
                              scale_desc(sb + L::kSclB + (s * NB + b) * kScaleBlock + 512 * j));
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f4(tmem, ad + 2 * j, bd + 2 * j, idesc, sa + 4 * j, sw + j * NB * 4, (k | j) ? 1u : 0u);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_f8(tmem + slot * 256, ad + 2 * j, bd + 2 * j, idesc, j ? 1u : 0u);
            }
            if (CL == 1) mma_commit(empty + 8 * s);
            else mma_commit_multicast(empty + 8 * s, (1 << CL) - 1);
            if (!F::kScaled || k == p.stages - 1) mma_commit(acc_full + 8 * slot);
          }
          __syncwarp();
          if (!F::kScaled || k == p.stages - 1) ++blk;
        }
      }
      // This warp's MMAs are done before tensor memory is freed.
      if (elect_one()) mma_commit(smem_u32(&drained_sh));
      __syncwarp();
      mbar_wait(smem_u32(&drained_sh), 0, p.err);
    } else if constexpr (F::kScaled) {
      int it = 0;
      bool live = true;
      for (int i = first; i < total && live; i += step) {
        for (int k = 0; k < p.stages; ++k, ++it) {
          const int s = it % S;
          live = __all_sync(0xFFFFFFFFu, wait_or_abort(full + 8 * s, (it / S) & 1, p.err, abort_flag));
          if (!live) break;
          rearrange_scales(smem + L::kRawA + s * kScaleBlock, smem + L::kSclA + s * kScaleBlock, warp - 2, lane, 128);
#pragma unroll
          for (int b = 0; b < BN / 128; ++b) {
            const int at = (s * (BN / 128) + b) * kScaleBlock;
            rearrange_scales(smem + L::kRawB + at, smem + L::kSclB + at, warp - 2, lane, 128);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(scaled + 8 * s);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q = warp & 3, h = (warp - kEpiWarp0) >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * COLS;
    const int kb = p.K >> 7;
    pdl_wait();                                // 8 bits: the activations' scales
    int blk = 0;
    bool live = true;
    for (int i = first; i < total && live; i += step) {
      int mi, ni;
      tile_at(i, p.mt, p.nt, mi, ni);
      const int m = (mi * CL + rank) * 128 + q * 32 + lane, n0 = ni * BN + h * COLS;
      uint32_t packed[COLS / 2];
      if constexpr (F::kScaled) {
        live = __all_sync(0xFFFFFFFFu, wait_or_abort(acc_full, blk & 1, p.err, abort_flag));
        if (!live) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t v[32];
          tmem_ld32_start(tl + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            packed[c / 2 + j] = pack_bf16(__uint_as_float(v[2 * j]) * p.gscale, __uint_as_float(v[2 * j + 1]) * p.gscale);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free);
        ++blk;
      } else {
        const float* sa = p.SA + static_cast<long long>(min(m, p.M - 1)) * kb;
        const float* sw = p.SW + static_cast<long long>(min(n0, p.N - 1) >> 7) * kb;
        float acc[COLS];
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] = 0.0f;
        float next = sa[0] * __ldg(sw);
        for (int k = 0; k < kb; ++k, ++blk) {
          const int slot = blk & 1;
          const float f = next;
          if (k + 1 < kb) next = sa[k + 1] * __ldg(sw + k + 1);
          live = __all_sync(0xFFFFFFFFu, wait_or_abort(acc_full + 8 * slot, (blk >> 1) & 1, p.err, abort_flag));
          if (!live) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            uint32_t v[32];
            tmem_ld32_start(tl + slot * 256 + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(v[j]), f, acc[c + j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_free + 8 * slot);
        }
        if (!live) break;
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) packed[j] = pack_bf16(acc[2 * j], acc[2 * j + 1]);
      }
      if (m < p.M) {
        uint16_t* c = p.C + static_cast<long long>(m) * p.ldc + n0;
        if (p.vec && n0 + COLS <= p.N) {
#pragma unroll
          for (int j = 0; j < COLS / 8; ++j)
            reinterpret_cast<uint4*>(c)[j] = make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < COLS / 2; ++j) {
            if (n0 + 2 * j < p.N) c[2 * j] = static_cast<uint16_t>(packed[j] & 0xFFFFu);
            if (n0 + 2 * j + 1 < p.N) c[2 * j + 1] = static_cast<uint16_t>(packed[j] >> 16);
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (CL > 1) cluster_sync();
}

template <class F, int BN, int CL>
cudaError_t launch_many_t(const ActGemmArgs& a, cudaStream_t s) {
  using L = ManyLayout<F, BN, CL>;
  const uint64_t row = F::kScaled ? static_cast<uint64_t>(a.K) / 2 : static_cast<uint64_t>(a.K);
  const uint64_t srow = static_cast<uint64_t>(a.K) / 16;
  const uint64_t M = static_cast<uint64_t>(a.M), N = static_cast<uint64_t>(a.N);
  CUtensorMap ma, mb, msa, msb;
  constexpr auto kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cudaError_t e = make_map_2d(&ma, kU8, a.A, row, M, row, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess) e = cached_map_2d(&mb, kU8, a.W, row, N, row, 128, BN / CL, CU_TENSOR_MAP_SWIZZLE_128B);
  msa = ma;
  msb = mb;
  if (F::kScaled) {
    if (e == cudaSuccess) e = make_map_2d(&msa, kU8, a.SA, srow, M, srow, 16, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess) e = cached_map_2d(&msb, kU8, a.SW, srow, N, srow, 16, BN / CL, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  static AttrLatch latch;
  if (e == cudaSuccess) e = set_smem_attrs(many_kernel<F, BN, CL>, latch, L::kAlloc, true);
  if (e != cudaSuccess) return e;
  ManyParams p = {};
  if (!F::kScaled) {
    p.SA = static_cast<const float*>(a.SA);
    p.SW = static_cast<const float*>(a.SW);
  }
  p.gscale = a.gscale;
  p.C = static_cast<uint16_t*>(a.C);
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.ldc = a.ldc;
  p.mt = (a.M + 128 * CL - 1) / (128 * CL);
  p.nt = (a.N + BN - 1) / BN;
  p.stages = a.K / F::kStageK;
  p.vec = a.ldc % 8 == 0 && reinterpret_cast<uintptr_t>(a.C) % 16 == 0;
  p.err = a.err;
  const long long total = static_cast<long long>(p.mt) * p.nt;
  const int clusters = static_cast<int>(total < a.num_sms / CL ? total : a.num_sms / CL);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * CL);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, many_kernel<F, BN, CL>, ma, mb, msa, msb, p);
}

template <class F>
cudaError_t launch_many(const ActGemmArgs& a, cudaStream_t s) {
  if (a.M <= 128) return launch_many_t<F, 256, 1>(a, s);
  return launch_many_t<F, 256, 2>(a, s);
}

}  // namespace
}  // namespace act

cudaError_t launch_w4a4_many(const ActGemmArgs& a, cudaStream_t s) { return act::launch_many<act::F4>(a, s); }
cudaError_t launch_w8a8_many(const ActGemmArgs& a, cudaStream_t s) { return act::launch_many<act::F8>(a, s); }

}  // namespace wqp
