// Products of quantised activations with packed weights, few rows: 4-bit by
// 4-bit with E4M3 scales per 16 K, and 8-bit by 8-bit with FP32 scales per
// 128 K.
//
// Bound by the weights' bytes. Swap-AB: the 128 weight rows of a tile are the
// MMA's M side and the call's activation rows, zero-padded to NT by the
// copies, its N side, so one pass over the weights serves NT of them:
//   D[n, m] = sum_k W[n, k] A[m, k]      (tcgen05.mma, FP32 accumulators)
// Both operands go from global to shared memory as they lie (128-byte rows,
// 128-byte swizzle) and into the tensor core undecoded.
//  * 4 bits: the tensor core multiplies each 16-K product sum by both scales;
//    two warps bring a stage's scales, in the order it reads them in, and the
//    MMA warp copies them to tensor memory. One accumulator for all of K.
//  * 8 bits: one MMA group per 128 K; the epilogue reads it and adds it, times
//    its two scales, to FP32 accumulators in registers.
// With few tiles, K is split over a cluster of up to 8 CTAs. Rank q owns the
// tile's activation rows q, q + splits, ...; the others push their partial sums of
// those into its shared memory (asynchronous stores that complete on its
// barrier), and it adds them in rank order, so the result does not depend on
// timing.
//
// Warps: 0 copies, 1 MMA (and tensor memory), 2..3 scales (4 bits), the rest
// epilogue (lane quarter = warp % 4).
#include "act.cuh"

namespace wqp {
namespace act {
namespace {

constexpr int kEpiWarp0 = 4;
// CTAs of a tile, at most: a portable cluster.
constexpr int kMaxSplits = 8;

struct FewParams {
  const void* SA;
  const void* SW;
  float gpow, gscale;
  uint16_t* C;
  int M, N, K, ldc;
  int splits, stages;
  unsigned* err;
};

// kShared: two CTAs of an SM share its memory; otherwise a CTA has it to itself.
// NT = 16, and 8 bits NT = 32, share it always. Wider tiles share it where there
// are more tiles than SMs, and then have no room to receive parts of a split K
// in: 64x34816x5120, 8 bits, 32.3 us against 39.5; 32x34816x5120, 4 bits, 17.2
// against 24.8.
template <class F, int NT, bool kShared>
struct FewLayout {
  // Epilogue warps: one to four per lane quarter, with NT, NT / 2 or NT / 4 columns
  // each: as many as registers allow, for a shorter time per 128 K (8 bits) and
  // at the end (with two at NT = 64, 128: 61x5120x17408, 8 bits, 20.8 us against
  // 20.0, 800x640x5120 12.6 against 11.4; 128x640x5120, 4 bits, 8.8 against 7.9).
  static constexpr int kEpi = NT >= 64 ? (kShared ? 8 : 16) : (NT == 32 && !(F::kScaled && kShared) ? 8 : 4);
  static constexpr int kCols = NT * 4 / kEpi;
  static constexpr int kThreads = (kEpiWarp0 + kEpi) * 32;
  static constexpr bool kWhole = kShared && NT >= (F::kScaled ? 32 : 64);  // a tile's K is not split
  static constexpr int kS = kShared ? (NT == 64 ? 3 : 4) : (NT == 128 ? 4 : 6);   // stages
  static constexpr int kAcc = F::kScaled ? 1 : (NT <= 64 ? 4 : 2);        // accumulator slots
  // Stages of a hand-over between copies, MMAs and epilogue: a hand-over takes the
  // MMA warp about as long as 64 columns of MMAs (64x10240x5120, 8 bits, one stage
  // | two: 16.9 | 15.7 us). With 128 columns and two: 28.2 | 28.9 at 128x5120x17408.
  static constexpr int kB = !F::kScaled && NT == 64 && !kShared ? 2 : 1;
  static constexpr int kW = 0;
  static constexpr int kA = kW + kS * 16384;
  static constexpr int kSclW = kA + kS * NT * 128;
  static constexpr int kSclA = kSclW + (F::kScaled ? kS * kScaleBlock : 0);
  static constexpr int kFac = kSclA + (F::kScaled ? kS * kScaleBlock : 0);
  static constexpr int kRecv = kFac + (F::kScaled ? 0 : 4 * NT * 4);
  static constexpr int kBytes = kRecv + (kWhole ? 0 : (NT + 7) * 128 * 4);
  static constexpr int kAlloc = kBytes + 1024;                            // slack for 1024-byte alignment
  static constexpr int kStageBytes = 16384 + NT * 128;
  // Tensor memory: the accumulators, then (4 bits) two sets of a stage's
  // scales, 4 columns per step and operand.
  static constexpr int kTmem = F::kScaled ? (NT + 64 <= 128 ? 128 : 256) : (kAcc * NT <= 64 ? 64 : (kAcc * NT <= 128 ? 128 : 256));
  static constexpr int kCtas = kShared ? 2 : 1;                           // per SM
  static_assert(!kShared || (kAlloc + 2048 <= 114 * 1024 && kTmem <= 256), "two CTAs of an SM");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

template <class F, int NT, bool kShared>
__global__ void __launch_bounds__(FewLayout<F, NT, kShared>::kThreads, FewLayout<F, NT, kShared>::kCtas)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, FewParams p) {
  using L = FewLayout<F, NT, kShared>;
  constexpr int B = L::kB, S = L::kS / B, NACC = L::kAcc / B;   // ring and accumulators, in hand-overs
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_sh[S], empty_sh[S], scaled_sh[S], acc_full_sh[NACC], acc_free_sh[NACC],
      recv_sh;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = L::kWhole ? 1 : p.splits;
  const int tile = blockIdx.x / splits, rank = blockIdx.x - tile * splits;
  const int n0 = tile * 128, m0 = blockIdx.y * NT, rows = min(NT, p.M - m0);   // activation rows m0..
  const int st0 = static_cast<int>(static_cast<long long>(rank) * p.stages / splits);
  const int nst = static_cast<int>(static_cast<long long>(rank + 1) * p.stages / splits) - st0;
  const uint32_t full = smem_u32(full_sh), empty = smem_u32(empty_sh), scaled = smem_u32(scaled_sh);
  const uint32_t acc_full = smem_u32(acc_full_sh), acc_free = smem_u32(acc_free_sh), recv_bar = smem_u32(&recv_sh);
  const int own = (rows - rank + splits - 1) / splits;     // of them: rank, rank + splits, ...
  volatile int* abort_flag = &abort_sh;
  // A whole sum to C: the global scales come last, as parts of a sum could pass
  // FP32's range with them where the sum does not.
  const auto rounded = [&](float v) { return f32_to_bf16_rn(F::kScaled ? (v * p.gpow) * p.gscale : v); };

  // The thread that copies: sets up the barriers and starts the first stages'
  // weights, which do not depend on the previous grid, before the CTA meets.
  // (Prefetching later stages into L2 on top: 17.1 -> 18.3..20.1 us at
  // 1x17408x5120.) Copies and MMAs are issued under elect.sync (see
  // gemm_act_many.cu).
  const int ahead = min(L::kS, nst), nu = (nst + B - 1) / B;   // nu: hand-overs
  int issued = 0;                                // stages whose copies this thread started
  const uint64_t pol = policy_evict_first();
  const auto load_w = [&](int t) {
    const int i = t % L::kS;
    const uint32_t bar = full + 8 * (i / B);
    if (t % B == 0) mbar_arrive_expect_tx(bar, min(B, nst - t) * L::kStageBytes);
    tma_load_2d_hint(sb + L::kW + i * 16384, &tmW, (st0 + t) * 128, n0, bar, pol);
  };
  const auto load_a = [&](int t) {
    const int i = t % L::kS;
    tma_load_2d(sb + L::kA + i * NT * 128, &tmA, (st0 + t) * 128, m0, full + 8 * (i / B));
  };
  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&tmW);
      prefetch_tmap(&tmA);
      for (int i = 0; i < S; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
        mbar_init(scaled + 8 * i, 2);
      }
      for (int i = 0; i < NACC; ++i) {
        mbar_init(acc_full + 8 * i, 1);
        mbar_init(acc_free + 8 * i, L::kEpi);
      }
      mbar_init(recv_bar, 1);
      abort_sh = 0;
      mbar_fence_init();
      // Every rank's share of this rank's rows, its own among them.
      if (splits > 1) mbar_arrive_expect_tx(recv_bar, static_cast<uint32_t>(own) * 512u * splits);
      for (int t = 0; t < ahead; ++t) load_w(t);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_sh), L::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_launch_dependents();
  if (splits > 1) cluster_arrive_relaxed();      // matched before the first push

  if (warp == 0) {
    if (elect_one()) {
      pdl_wait();
      for (int t = 0; t < ahead; ++t) load_a(t);
      issued = ahead;
      for (int t = ahead; t < nst; ++t) {
        const int u = t / B;
        if (t % B == 0 && !wait_or_abort(empty + 8 * (u % S), ((u / S) - 1) & 1, p.err, abort_flag)) break;
        load_w(t);
        load_a(t);
        issued = t + 1;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = F::kScaled ? idesc_f4(128, NT) : idesc_f8(128, NT);
    // 8 bits: what the next stage needs is looked up before this stage's MMAs are
    // issued (see gemm_act_many.cu; 61x5120x17408: 23.3 -> 21.1 us). With 4 bits
    // the scales of the next stage are hardly ever there yet, and it costs 2 %.
    int last = -1, s = 0, slot = 0;
    uint32_t ph = 0, acc_ph = 1;
    bool loaded = false, freed = true;
    for (int t = 0; t < nu; ++t) {
      bool ok = true;
      if (!loaded) {
        ok = wait_or_abort(full + 8 * s, ph, p.err, abort_flag);
        if (F::kScaled) ok = ok && wait_or_abort(scaled + 8 * s, ph, p.err, abort_flag);
      }
      if (!F::kScaled && !freed) ok = ok && wait_or_abort(acc_free + 8 * slot, acc_ph, p.err, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const int s1 = s + 1 == S ? 0 : s + 1, slot1 = slot + 1 == NACC ? 0 : slot + 1;
      const uint32_t ph1 = s1 ? ph : ph ^ 1, acc_ph1 = slot1 ? acc_ph : acc_ph ^ 1;
      const bool l1 = !F::kScaled && mbar_test(full + 8 * s1, ph1);
      // Parity 1 of a barrier that has completed no phase counts as complete.
      const bool f1 = F::kScaled || mbar_test(acc_free + 8 * slot1, acc_ph1);
      if (elect_one()) {
        const uint64_t wd = tile_desc(sb + L::kW + s * B * 16384), ad = tile_desc(sb + L::kA + s * B * NT * 128);
        if constexpr (F::kScaled) {
          const uint32_t sw = tmem + NT + (t & 1) * 32, sa = sw + 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            copy_scales(sw + 4 * j, scale_desc(sb + L::kSclW + s * kScaleBlock + 512 * j));
            copy_scales(sa + 4 * j, scale_desc(sb + L::kSclA + s * kScaleBlock + 512 * j));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f4(tmem, wd + 2 * j, ad + 2 * j, idesc, sw + 4 * j, sa + 4 * j, (t | j) ? 1u : 0u);
        } else {
#pragma unroll
          for (int b = 0; b < B; ++b) {
            if (b && t * B + b >= nst) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f8(tmem + (slot * B + b) * NT, wd + b * 1024 + 2 * j, ad + b * NT * 8 + 2 * j, idesc, j ? 1u : 0u);
          }
        }
        mma_commit(empty + 8 * s);
        if (!F::kScaled || t == nst - 1) mma_commit(acc_full + 8 * (F::kScaled ? 0 : slot));
      }
      __syncwarp();
      last = t;
      loaded = __all_sync(0xFFFFFFFFu, l1);
      freed = __all_sync(0xFFFFFFFFu, f1);
      s = s1, ph = ph1;
      if (!F::kScaled) slot = slot1, acc_ph = acc_ph1;
    }
    // This warp's MMAs are done before tensor memory is freed.
    if (last >= 0) mbar_wait(empty + 8 * (last % S), (last / S) & 1, p.err);
  } else if (warp < kEpiWarp0) {
    if constexpr (F::kScaled) {
      // Four stages' scales are on their way at a time.
      constexpr int D = 4;
      const int half = warp - 2, pitch = p.K >> 4;
      ScaleRows rw, ra;
      rw.at(static_cast<const uint8_t*>(p.SW), n0, p.N, pitch, half, lane);
      ra.at(static_cast<const uint8_t*>(p.SA), m0, p.M, pitch, half, lane);
      const bool any = 64 * half < NT;           // this warp's activation columns exist
      uint4 vw[D][2], va[D][2];
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (d < nst) rw.load<true>(st0 + d, vw[d]);
      pdl_wait();
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (d < nst && any) ra.load<false>(st0 + d, va[d]);
      for (int t0 = 0; t0 < nst; t0 += D) {        // after an abort: to the end, without waiting
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int t = t0 + d, s = t % S;
          if (t < nst) {
            if (t >= S) wait_or_abort(empty + 8 * s, ((t / S) - 1) & 1, p.err, abort_flag);
            put_scale_rows(smem + L::kSclW + s * kScaleBlock, half, lane, vw[d]);
            if (any) put_scale_rows(smem + L::kSclA + s * kScaleBlock, half, lane, va[d]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(scaled + 8 * s);
            if (t + D < nst) {
              rw.load<true>(st0 + t + D, vw[d]);
              if (any) ra.load<false>(st0 + t + D, va[d]);
            }
          }
        }
      }
    }
  } else {
    constexpr int COLS = L::kCols;
    const int q = warp & 3, r = q * 32 + lane, c0 = (warp - kEpiWarp0) / 4 * COLS;   // its first activation row
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + c0;
    float acc[COLS];
#pragma unroll
    for (int m = 0; m < COLS; ++m) acc[m] = 0.0f;
    bool live = true;
    if constexpr (F::kScaled) {
      live = __all_sync(0xFFFFFFFFu, wait_or_abort(acc_full, 0, p.err, abort_flag));
      if (live) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
          uint32_t v[16];
          tmem_ld16_start(tl + c, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] = __uint_as_float(v[i]);
        }
      }
    } else {
      // Lane l brings the scales of activation rows l, l + 32, ..., D groups
      // ahead of their use: a fetch takes longer than a group.
      constexpr int kPer = (COLS + 31) / 32, D = 4;
      const int kb = p.K >> 7;
      const float* sw = static_cast<const float*>(p.SW) + static_cast<long long>(tile) * kb + st0;
      const float* sa[kPer];
      float fa[D][kPer], fw[D];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        sa[i] = static_cast<const float*>(p.SA) + static_cast<long long>(min(m0 + c0 + 32 * i + lane, p.M - 1)) * kb + st0;
      float* fac = reinterpret_cast<float*>(smem + L::kFac) + (warp - kEpiWarp0) * COLS;
#pragma unroll
      for (int d = 0; d < D; ++d) fw[d] = d < nst ? __ldg(sw + d) : 0.0f;
      pdl_wait();
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < kPer; ++i) fa[d][i] = d < nst ? sa[i][d] : 0.0f;
      for (int t0 = 0; t0 < nst && live; t0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int t = t0 + d, u = t / B, slot = u % NACC;
          if (t < nst && live) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              if (32 * i + lane < COLS) fac[32 * i + lane] = fa[d][i] * fw[d];
              if (t + D < nst) fa[d][i] = sa[i][t + D];
            }
            if (t + D < nst) fw[d] = __ldg(sw + t + D);
            __syncwarp();
            if (t % B == 0)
              live = __all_sync(0xFFFFFFFFu, wait_or_abort(acc_full + 8 * slot, (u / NACC) & 1, p.err, abort_flag));
            if (live) {
              tc_fence_after();
              // The next 16 columns are on their way while these are added; the
              // accumulator is free once the last have arrived.
              uint32_t v[2][16];
              const uint32_t ta = tl + (slot * B + t % B) * NT;
              tmem_ld16_start(ta, v[0]);
#pragma unroll
              for (int c = 0; c < COLS; c += 16) {
                uint32_t(&x)[16] = v[(c / 16) & 1];
                tmem_ld_wait(x);
                if (c + 16 < COLS) {
                  tmem_ld16_start(ta + c + 16, v[(c / 16 + 1) & 1]);
                } else {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0 && (t % B == B - 1 || t == nst - 1)) mbar_arrive(acc_free + 8 * slot);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(__uint_as_float(x[i]), fac[c + i], acc[c + i]);
              }
            }
          }
        }
      }
    }
    if (splits > 1) {
      cluster_wait();
      // Row m goes to rank m % splits, into [source rank][m / splits][weight row].
      // After an abort too: the owner counts on it.
      const int per = (NT + splits - 1) / splits;
      const uint32_t dst = sb + L::kRecv + 4 * (rank * per * 128 + r);
      uint32_t at = c0 / splits * 512;
      int owner = c0 % splits;
#pragma unroll
      for (int m = 0; m < COLS; ++m) {
        if (c0 + m < rows) st_async_f32(mapa_shared(dst + at, owner), acc[m], mapa_shared(recv_bar, owner));
        if (++owner == splits) owner = 0, at += 512;
      }
    } else if (live && n0 + r < p.N) {
      uint16_t* c = p.C + static_cast<long long>(m0 + c0) * p.ldc + n0 + r;
#pragma unroll
      for (int m = 0; m < COLS; ++m)
        if (c0 + m < rows) c[static_cast<long long>(m) * p.ldc] = rounded(acc[m]);
    }
  }
  if (splits > 1 && warp < kEpiWarp0) cluster_wait();

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
  const bool failed = *abort_flag != 0;
  if (failed)                                    // no copy may still be in flight when the CTA exits
    for (int n = (issued + B - 1) / B, u = max(0, n - S); u < n; ++u) mbar_wait(full + 8 * (u % S), (u / S) & 1, p.err);
  if (splits > 1 && own > 0) {
    // No one writes into this CTA once its rows' sums are complete. A peer may
    // use up two waits of its own before it sends them.
    const bool complete = mbar_wait_ns(recv_bar, 0, p.err, 3 * kWaitLimitNs);
    const int per = (NT + splits - 1) / splits;
    const float* recv = reinterpret_cast<const float*>(smem + L::kRecv);
    const int r = threadIdx.x & 127;
    if (complete && !failed && n0 + r < p.N) {
      for (int i = threadIdx.x >> 7; i < own; i += L::kThreads / 128) {
        float v = recv[i * 128 + r];
        for (int src = 1; src < splits; ++src) v += recv[(src * per + i) * 128 + r];
        p.C[static_cast<long long>(m0 + i * splits + rank) * p.ldc + n0 + r] = rounded(v);
      }
    }
  }
}

// How many clusters of 2, 3, ... CTAs, each with an SM to itself, are resident
// at once, as (*found)[size]. It depends on how the device's SMs are spread over
// its GPCs, so it is asked for, once per device.
cudaError_t resident_clusters(const std::atomic<int>** found) {
  using L = FewLayout<F8, 128, false>;
  static_assert(L::kAlloc > 114 * 1024, "one CTA an SM");
  static std::atomic<int> table[kMaxDevices][kMaxSplits + 1];
  static AttrLatch latch, attrs;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  *found = table[dev];
  if (latch.done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const auto kern = few_kernel<F8, 128, false>;
  if (cudaError_t e = set_smem_attrs(kern, attrs, L::kAlloc, true); e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  for (int size = 2; size <= kMaxSplits; ++size) {
    int n = 0;
    attr.val.clusterDim.x = size;
    cfg.gridDim = dim3(size);
    if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg); e != cudaSuccess) return e;
    table[dev][size].store(n, std::memory_order_relaxed);
  }
  latch.done[dev].store(1, std::memory_order_release);
  return cudaSuccess;
}

// CTAs of a tile: as many as leave every cluster resident, with `ctas` CTAs an
// SM (of 2..8 CTAs with an SM each, 76, 46, 36, 28, 23, 15 and 15 clusters are; one
// wave too many costs most: 600x1280x5120, 8 bits, 50 tiles of 3 | 2 CTAs 26.0 |
// 17.1 us, 1000x256x5120, 16 of 7 | 6 18.4 | 10.5). More than 4 only with two
// stages each, and CTAs with an SM each only from 4 stages on, as less work saved
// does not pay for the sums (1x2560x2560, 4 bits, by 7 | 5: 4.7 | 4.3 us;
// 64x2560x256, 8 bits, by 2 | not: 6.2 | 4.7).
cudaError_t few_splits(long long tiles, int stages, int ctas, int* splits) {
  *splits = 1;
  if (stages < 2 || (ctas == 1 && stages < 4)) return cudaSuccess;
  const std::atomic<int>* resident;
  if (cudaError_t e = resident_clusters(&resident); e != cudaSuccess) return e;
  for (int sp = 2; sp <= kMaxSplits && sp <= (sp <= 4 ? stages : stages / 2); ++sp)
    if (tiles <= static_cast<long long>(resident[sp].load(std::memory_order_relaxed)) * ctas) *splits = sp;
  return cudaSuccess;
}

template <class F, int NT, bool kShared>
cudaError_t launch_few_nt(const ActGemmArgs& a, cudaStream_t s) {
  using L = FewLayout<F, NT, kShared>;
  const uint64_t row = F::kScaled ? static_cast<uint64_t>(a.K) / 2 : static_cast<uint64_t>(a.K);
  CUtensorMap mw, ma;
  cudaError_t e = cached_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.W, row, static_cast<uint64_t>(a.N), row, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, row, static_cast<uint64_t>(a.M), row, 128, NT,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  static AttrLatch latch;
  if (e = set_smem_attrs(few_kernel<F, NT, kShared>, latch, L::kAlloc, true); e != cudaSuccess) return e;
  FewParams p = {};
  p.SA = a.SA;
  p.SW = a.SW;
  p.gpow = a.gpow;
  p.gscale = a.gscale;
  p.C = static_cast<uint16_t*>(a.C);
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.ldc = a.ldc;
  p.stages = a.K / F::kStageK;
  p.err = a.err;
  const int tiles = (a.N + 127) / 128, mt = (a.M + NT - 1) / NT;
  p.splits = 1;
  if (!L::kWhole) e = few_splits(static_cast<long long>(tiles) * mt, p.stages, L::kCtas, &p.splits);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * p.splits, mt);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<F, NT, kShared>, mw, ma, p);
}

// Whether a call is this kernel's: always up to 64 rows (with 4 bits a fixed
// choice that costs a tenth where nearly every SM has one tile whose K is not
// split: 64x10240x5120 below), and where K can be split over the SMs that few
// tiles leave idle and that saves more time than the sums of the parts cost;
// else gemm_act_many.cu's wide tiles win. Measured, here | there, us:
//  * 4 bits: 40x10240x5120 12.1 | 12.9, 49x17408x5120 13.7 | 18.5, 64x10240x5120
//    12.7 | 11.3, 64x17408x2560 8.8 | 11.5, 64x34816x5120 19.7 | 25.0,
//    64x2560x10240 8.7 | 15.7; 100x640x5120 7.5 | 10.1, 100x5120x5120 10.3 | 10.4,
//    128x7168x5120 12.6 | 10.6, 200x1280x2560 7.6 | 7.4, 300x640x10240 9.7 | 15.7,
//    300x256x1024 7.1 | 5.8, 1000x256x5120 8.7 | 10.2;
//  * 8 bits: 64x10240x5120 15.3 | 18.3, 64x34816x5120 32.3 | 40.4, 64x2560x10240
//    9.8 | 25.4; 128x5120x17408 26.9 | 41.0, 128x7168x5120 16.1 | 14.9,
//    100x1280x1280 6.9 | 6.5, 300x640x2560 7.8 | 9.1, 800x640x5120 11.4 | 14.6,
//    1146x21x14336 13.3 | 34.0.
template <class F>
cudaError_t few_fits(const ActGemmArgs& a, bool* fits) {
  *fits = a.M <= 64;
  if (*fits) return cudaSuccess;
  const int stages = a.K / F::kStageK;
  const long long tiles = static_cast<long long>((a.N + 127) / 128) * ((a.M + 127) / 128);
  if (2 * tiles > a.num_sms) return cudaSuccess;
  int splits;
  const cudaError_t e = few_splits(tiles, stages, 1, &splits);
  // In eighths of a microsecond: a stage here 4 and there 9 / 4, and what a call
  // costs more here.
  const int here = (stages + splits - 1) / splits * 4 + (F::kScaled ? 17 : 26);
  *fits = splits > 1 && 4 * here < 9 * stages;
  return e;
}

template <class F>
cudaError_t launch_few(const ActGemmArgs& a, cudaStream_t s) {
  const bool wide = (a.N + 127) / 128 > a.num_sms;
  if (a.M <= 16) return launch_few_nt<F, 16, true>(a, s);
  if (a.M <= 32) return wide || !F::kScaled ? launch_few_nt<F, 32, true>(a, s) : launch_few_nt<F, 32, false>(a, s);
  if (a.M <= 64) return wide ? launch_few_nt<F, 64, true>(a, s) : launch_few_nt<F, 64, false>(a, s);
  return launch_few_nt<F, 128, false>(a, s);
}

}  // namespace
}  // namespace act

// Calls of more than 2^20 rows go in pieces, so that tile counts stay within
// an int.
template <class F>
static cudaError_t launch_act_gemm(const ActGemmArgs& a, cudaStream_t s) {
  constexpr int kPiece = 1 << 20;
  cudaError_t e = cudaSuccess;
  for (int r0 = 0; r0 < a.M && e == cudaSuccess; r0 += kPiece) {
    ActGemmArgs b = a;
    b.M = a.M - r0 < kPiece ? a.M - r0 : kPiece;
    const size_t r = static_cast<size_t>(r0), K = static_cast<size_t>(a.K);
    b.A = static_cast<const char*>(a.A) + r * (F::kScaled ? K / 2 : K);
    b.SA = static_cast<const char*>(a.SA) + r * (F::kScaled ? K / 16 : K / 128 * 4);
    b.C = static_cast<char*>(a.C) + r * a.ldc * 2;
    bool few = false;
    e = act::few_fits<F>(b, &few);
    if (e != cudaSuccess) return e;
    if (few) e = act::launch_few<F>(b, s);
    else e = F::kScaled ? launch_w4a4_many(b, s) : launch_w8a8_many(b, s);
    if (a.M - r0 <= kPiece) break;
  }
  return e;
}

cudaError_t launch_w4a4_gemm(const ActGemmArgs& a, cudaStream_t s) { return launch_act_gemm<act::F4>(a, s); }
cudaError_t launch_w8a8_gemm(const ActGemmArgs& a, cudaStream_t s) { return launch_act_gemm<act::F8>(a, s); }

}  // namespace wqp
