// Products of quantised activations with packed weights, many rows: 4-bit by
// 4-bit with E4M3 scales per 16 K, and 8-bit by 8-bit with FP32 scales per
// 128 K.
//
// Bound by the tensor core and, at its 8- and 4-bit rates, by the shared
// memory that feeds it: a tile is 256 activation rows by BN weight rows, held
// by a pair of CTAs on two SMs (act.cuh), so that each SM reads half of the
// weight tile for all of its MMA's work. Persistent pairs walk over the tiles.
//  * 4 bits: the tensor core applies the scales, rearranged by warps of each CTA
//    (its 128 activation rows, all BN weight rows) and copied to tensor memory
//    by the MMA warp. One or two accumulators, drained into registers as BF16.
//    4096x34816x5120: 236 us, 6.2 PFLOP/s until the power cap slows the clock,
//    264 to 272 us, 5.4 PFLOP/s, in steady use.
//    The tensor pipe is busy for two thirds of it; next are the bytes into an
//    SM (38 KB a stage, at 64 a clock nine tenths of a stage's time) and the
//    drains between tiles.
//  * 8 bits: two to four accumulators that take turns per 128 K; the epilogue
//    adds each, times its activation row's and weight block's scale, to FP32
//    sums in registers while the tensor core fills the others.
//    4096x5120x17408: 277 to 290 us, 2.5 PFLOP/s, until the power cap slows the
//    clock, 315 to 324 us in steady use. Bound by that reading and adding: 773
//    clocks per 128 K of a 256-column tile, of which the MMAs are 544; without
//    the additions 238 us.
// With 4 bits the operands may change places (kSwap): 256 weight rows by BN
// activation rows, where that leaves less of the tiles empty.
// Output goes through shared memory, 32 rows by 32 columns a warp at a time,
// and leaves as bulk tensor stores (rows of C that are not 16-byte aligned: as
// stores of 8, 4 or 2 bytes a lane from there).
//
// Warps: 0 copies, 1 MMA (even CTA; tensor memory in both), 4 bits: 2..7
// scales; then 8 epilogue warps, one per lane quarter (warp % 4) and half of the
// columns (16 with a quarter each read tensor memory no faster and have too few
// registers: 348 us at 4096x5120x17408).
#include "act.cuh"

namespace wqp {
namespace act {
namespace {

struct ManyParams {
  const float* SA;
  const float* SW;
  float gpow, gscale;
  uint16_t* C;
  int M, N, K, ldc;
  int mt, nt;           // tiles of 256 rows of the first operand, of BN rows of the second
  int stages;           // per tile
  int align;            // of C's rows, bytes: 16, 8, 4 or 2
  unsigned* err;
};

template <class F, int BN>
struct ManyLayout {
  // Warps before the epilogue's: copies and MMA, then 4 bits: two sets of three
  // that rearrange scales, 8 bits: two idle ones (register shares are set by
  // four warps at a time).
  static constexpr int kRoles = F::kScaled ? 8 : 4;
  static constexpr int kCols = BN / 2;                          // columns of an epilogue warp
  static constexpr int kEpi = 8;                                // epilogue warps
  static constexpr int kThreads = (kRoles + kEpi) * 32;
  static constexpr int kNB = (BN + 127) / 128;                  // 128-row blocks of the weights' scales
  static constexpr int kStageBytes = 16384 + BN * 64;
  // 4 bits: the scales of two stages at a time, in a ring of their own (three
  // slots: 236 us at 4096x34816x5120, four 233; a stage at a time 245).
  static constexpr int kR = 4;
  static constexpr int kSclBytes = F::kScaled ? kR * 2 * kScaleBlock * (1 + kNB) : 0;
  static constexpr int kOutBufs = F::kScaled && BN == 256 ? 1 : 2;   // two there would cost a stage
  static constexpr int kOutBytes = 32 * 64;                     // what an epilogue warp stores at a time
  static constexpr int kS = (225 * 1024 - kOutBufs * kEpi * kOutBytes - kSclBytes) / kStageBytes;
  static constexpr int kA = 0;
  static constexpr int kB = kA + kS * 16384;
  static constexpr int kOut = kB + kS * BN * 64;                // [epilogue warp][buffer][32 rows][32 columns]
  static constexpr int kSclA = kOut + kOutBufs * kEpi * kOutBytes;   // [kR][2 stages]
  static constexpr int kSclB = kSclA + (F::kScaled ? kR * 2 * kScaleBlock : 0);   // [kR][block][2 stages]
  static constexpr int kBytes = kSclA + kSclBytes;
  static constexpr int kAlloc = kBytes + 1024;
  // Accumulators of BN columns in tensor memory, and (4 bits) behind them two
  // sets of a stage's scales.
  static constexpr int kAcc = F::kScaled ? (BN <= 192 ? 2 : 1) : 512 / BN;
  static constexpr uint32_t kScaleCol = kAcc * BN;
  static_assert(kScaleCol + (F::kScaled ? 64 + 16 + 16 * kNB : 0) <= 512, "tensor memory");
  static_assert(kAlloc <= 227 * 1024 - 1024, "shared memory");
};

// Tile i of the walk: groups of G row tiles go through all weight tiles, row
// tiles first, so that the tiles in flight share both operands in L2. A group
// is as many bytes in either format (4096x34816x5120, 4 bits: 261 us at G = 8,
// 254 at 16; 4096x5120x17408, 8 bits: 305 us at 8, 310 at 16).
template <class F>
__device__ __forceinline__ void tile_at(int i, int mt, int nt, int& m, int& n) {
  constexpr int G = F::kScaled ? 16 : 8;
  const int per = G * nt;
  const int g = i / per, rows = min(G, mt - g * G);
  const int j = i - g * per;
  n = j / rows;
  m = g * G + (j - n * rows);
}

// A 32 x 32 chunk at columns n.. of rows m0.. of C, whose rows are 2 E-byte
// aligned, E elements a lane: chunk_at(r, j) is 16-byte piece j of row r.
template <int E, class At>
__device__ __forceinline__ void store_rows(const At& chunk_at, const ManyParams& p, int m0, int n, int lane) {
  constexpr int kLanes = 32 / E, kRows = 32 / kLanes;        // lanes of a row, rows at a time
  const int r0 = lane / kLanes, col = lane % kLanes * E, left = p.N - n - col;
  const int rows = min(32, p.M - m0) - r0;
  uint16_t* c = p.C + static_cast<long long>(m0 + r0) * p.ldc + n + col;
#pragma unroll 8
  for (int r = 0; r < 32; r += kRows, c += static_cast<long long>(kRows) * p.ldc) {
    if (r >= rows) break;
    const uint8_t* v = chunk_at(r0 + r, col >> 3) + (col & 7) * 2;
    if (E == 4 && left >= 4) {
      *reinterpret_cast<uint2*>(c) = *reinterpret_cast<const uint2*>(v);
    } else if (E == 2 && left >= 2) {
      *reinterpret_cast<uint32_t*>(c) = *reinterpret_cast<const uint32_t*>(v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < left) c[e] = reinterpret_cast<const uint16_t*>(v)[e];
    }
  }
}

// kSwap: the weights are the first operand, and a tile is stored transposed.
template <class F, int BN, bool kSwap>
__global__ void __launch_bounds__(ManyLayout<F, BN>::kThreads, 1)
    many_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmC, ManyParams p) {
  using L = ManyLayout<F, BN>;
  constexpr int S = L::kS, R = L::kR, NACC = L::kAcc, COLS = L::kCols, NB = L::kNB;
  extern __shared__ uint8_t smem_raw[];
  // full, scaled and acc_free count both CTAs' work and are used in the even
  // CTA; raw_full is each CTA's own; empty, scl_empty and acc_full are told to
  // both.
  __shared__ __align__(8) uint64_t full_sh[S], empty_sh[S], raw_full_sh[R], scaled_sh[R], scl_empty_sh[R], acc_full_sh[NACC],
      acc_free_sh[NACC], drained_sh;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, total = p.mt * p.nt;
  const uint32_t full = smem_u32(full_sh), raw_full = smem_u32(raw_full_sh), empty = smem_u32(empty_sh);
  const uint32_t scaled = smem_u32(scaled_sh), scl_empty = smem_u32(scl_empty_sh), acc_full = smem_u32(acc_full_sh), acc_free = smem_u32(acc_free_sh);
  const uint32_t drained = smem_u32(&drained_sh);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + 8 * i, 2);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < R; ++i) {
      mbar_init(raw_full + 8 * i, 1);
      mbar_init(scaled + 8 * i, 2 * (1 + NB));
      mbar_init(scl_empty + 8 * i, 1);
    }
    for (int i = 0; i < NACC; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_free + 8 * i, 2 * L::kEpi);
    }
    mbar_init(drained, 1);
    abort_sh = 0;
    mbar_fence_init();
  }
  // The copying warp goes on as soon as every barrier of the pair exists (no
  // peer's copy or arrive may come before); the others meet for the tensor
  // memory's address first. The cluster barriers only order execution: the
  // barriers' set-up is published by its own fence, and a release here costs
  // half a microsecond.
  __syncwarp();
  cluster_arrive_relaxed();
  if (warp == 1) {
    pair_tmem_alloc(smem_u32(&tmem_sh), 512);
    tc_fence_before();
  }
  if (warp != 0) {
    asm volatile("bar.sync 1, %0;" ::"n"(L::kThreads - 32) : "memory");
    tc_fence_after();
  }
  cluster_wait();
  const uint32_t tmem = warp != 0 ? tmem_sh : 0u;
  pdl_launch_dependents();

  // The loops below keep their place in a ring as an index and a parity: their
  // instructions are on the path from one stage to the next. Copies, MMAs and
  // stores are issued under elect.sync, whose one thread the compiler knows to
  // be one: behind a test of the lane number the same instructions took twice
  // the kernel's time (4096x34816x5120, 4 bits: 494 us against 261). A wait that
  // runs out ends its warp's loop (the epilogue's: at the end of the tile, with
  // nothing stored), and the others' with it.
  if (warp < L::kRoles) {
    if (!F::kScaled) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && elect_one()) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      pdl_wait();
      const uint32_t full0 = mapa_shared(full, 0);
      int s = 0, used = 0, r = 0, rused = 0;   // stages and scale slots used, up to S and R
      uint32_t ph = 1, rph = 1;                // parity of the stage's (slot's) last consumption
      for (int i = first; i < total && !*abort_flag; i += step) {
        int mi, ni;
        tile_at<F>(i, p.mt, p.nt, mi, ni);
        const int m0 = mi * 256 + rank * 128, n0 = ni * BN;
        for (int k = 0; k < p.stages; ++k) {
          if (F::kScaled && k % 2 == 0) {
            if (rused == R) {
              if (!wait_or_abort(scl_empty + 8 * r, rph, p.err, abort_flag)) break;
            } else {
              ++rused;
            }
            mbar_arrive_expect_tx(raw_full + 8 * r, (128 + BN) * 32);
            tma_load_2d(sb + L::kSclA + r * 2 * kScaleBlock, &tmSA, k * 16, m0, raw_full + 8 * r);
            tma_load_2d(sb + L::kSclB + r * 2 * kScaleBlock * NB, &tmSB, k * 16, n0, raw_full + 8 * r);
            if (++r == R) r = 0, rph ^= 1;
          }
          if (used == S) {
            if (!wait_or_abort(empty + 8 * s, ph, p.err, abort_flag)) break;
          } else {
            ++used;
          }
          // The even CTA's barrier takes both CTAs' bytes; each announces its own.
          pair_arrive_expect_tx(full0 + 8 * s, 16384 + BN * 64);
          pair_tma_load_2d(sb + L::kA + s * 16384, &tmA, k * 128, m0, full0 + 8 * s);
          pair_tma_load_2d(sb + L::kB + s * BN * 64, &tmB, k * 128, n0 + rank * (BN / 2), full0 + 8 * s);
          if (++s == S) s = 0, ph ^= 1;
        }
      }
      // Every stage has been consumed, or (after an abort) has at least
      // arrived, before the CTA may exit: the oldest first.
      for (int t = 0; t < used; ++t) {
        const int at = used < S ? t : s;
        const uint32_t par = used < S ? 0u : ph;
        if (!wait_or_abort(empty + 8 * at, par, p.err, abort_flag) && rank == 0) mbar_wait(full + 8 * at, par, p.err);
        if (used == S && ++s == S) s = 0, ph ^= 1;
      }
      for (int t = 0; t < rused; ++t) {
        const int at = rused < R ? t : r;
        const uint32_t par = rused < R ? 0u : rph;
        if (!wait_or_abort(scl_empty + 8 * at, par, p.err, abort_flag)) mbar_wait(raw_full + 8 * at, par, p.err);
        if (rused == R && ++r == R) r = 0, rph ^= 1;
      }
    } else if (warp == 1 && rank == 0) {
      constexpr uint32_t idesc = F::kScaled ? idesc_f4(256, BN) : idesc_f8(256, BN);
      const uint64_t ad0 = tile_desc(sb + L::kA), bd0 = tile_desc(sb + L::kB);
      const uint64_t sad0 = scale_desc(sb + L::kSclA), sbd0 = scale_desc(sb + L::kSclB);
      // A wait that follows MMAs costs the tensor core a pause (the warp comes
      // back from it only when the MMAs have been taken), so what the next
      // stage needs is looked up before this stage's are issued, and waited for
      // only if it was not there yet.
      int s = 0, slot = 0, k = 0, r = 0;
      uint32_t ph = 0, acc_ph = 1, rph = 0, set = 0;
      bool loaded = false, freed = true;       // of the next stage; accumulators start free
      const long long stages = static_cast<long long>((total - first + step - 1) / step) * p.stages;
      for (long long it = 0; it < stages; ++it) {
        bool ok = true;
        if (!freed) ok = wait_or_abort(acc_free + 8 * slot, acc_ph, p.err, abort_flag);
        if (!loaded) {
          ok = ok && wait_or_abort(full + 8 * s, ph, p.err, abort_flag);
          if (F::kScaled && k % 2 == 0) ok = ok && wait_or_abort(scaled + 8 * r, rph, p.err, abort_flag);
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const int s1 = s + 1 == S ? 0 : s + 1, k1 = k + 1 == p.stages ? 0 : k + 1;
        const uint32_t ph1 = s1 ? ph : ph ^ 1;
        const bool hand = !F::kScaled || k1 == 0;                    // this stage completes an accumulator
        const int slot1 = !hand ? slot : (slot + 1 == NACC ? 0 : slot + 1);
        const uint32_t acc_ph1 = hand && slot1 == 0 ? acc_ph ^ 1 : acc_ph;
        const bool next = k1 % 2 == 0;                               // it is the last that uses its scale slot
        const int r1 = !next ? r : (r + 1 == R ? 0 : r + 1);
        const uint32_t rph1 = next && r1 == 0 ? rph ^ 1 : rph;
        bool l1 = mbar_test(full + 8 * s1, ph1);
        if (F::kScaled && next) l1 = l1 && mbar_test(scaled + 8 * r1, rph1);
        // Parity 1 of a barrier that has completed no phase counts as complete.
        const bool f1 = !hand || mbar_test(acc_free + 8 * slot1, acc_ph1);
        if (elect_one()) {
          // Addresses in a descriptor are in units of 16 bytes.
          const uint64_t ad = ad0 + s * (16384 >> 4), bd = bd0 + s * ((BN * 64) >> 4);
          if constexpr (F::kScaled) {
            const uint64_t sad = sad0 + (r * 2 + k % 2) * (kScaleBlock >> 4);
            const uint64_t sbd = sbd0 + (r * 2 * NB + k % 2) * (kScaleBlock >> 4);
            const uint32_t sa = tmem + L::kScaleCol + set * 64, sw = sa + 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              pair_copy_scales(sa + 4 * j, sad + 32 * j);
#pragma unroll
              for (int b = 0; b < NB; ++b) pair_copy_scales(sw + (j * NB + b) * 4, sbd + 2 * b * (kScaleBlock >> 4) + 32 * j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              pair_mma_f4(tmem + slot * BN, ad + 2 * j, bd + 2 * j, idesc, sa + 4 * j, sw + j * NB * 4, (k | j) ? 1u : 0u);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) pair_mma_f8(tmem + slot * BN, ad + 2 * j, bd + 2 * j, idesc, j ? 1u : 0u);
          }
          if (hand) pair_commit(acc_full + 8 * slot);
          if (F::kScaled && next) pair_commit(scl_empty + 8 * r);
          pair_commit(empty + 8 * s);
        }
        __syncwarp();
        loaded = __all_sync(0xFFFFFFFFu, l1);
        freed = __all_sync(0xFFFFFFFFu, f1);
        set ^= 1;
        s = s1, ph = ph1, k = k1, slot = slot1, acc_ph = acc_ph1, r = r1, rph = rph1;
      }
      // The pair's MMAs are done before the cluster barrier below, and tensor
      // memory is freed after it.
      if (elect_one()) pair_commit_own(drained);
      __syncwarp();
      mbar_wait(drained, 0, p.err);
    } else if (F::kScaled && warp >= 2) {
      // Two sets of warps take the scale slots in turn, one 128-row block a warp.
      const int set = (warp - 2) / 3, b = (warp - 2) % 3;
      if (b < 1 + NB) {
        const uint32_t scaled0 = mapa_shared(scaled, 0);
        const long long slots = static_cast<long long>((total - first + step - 1) / step) * ((p.stages + 1) / 2);
        int r = set;
        uint32_t rph = 0;
        for (long long it = set; it < slots; it += 2) {
          if (!__all_sync(0xFFFFFFFFu, wait_or_abort(raw_full + 8 * r, rph, p.err, abort_flag))) break;
          if (b == 0) rearrange_scales(smem + L::kSclA + r * 2 * kScaleBlock, lane, 128);
          else rearrange_scales(smem + L::kSclB + (r * NB + b - 1) * 2 * kScaleBlock, lane, min(128, BN - 128 * (b - 1)));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) pair_arrive(scaled0 + 8 * r);
          r += 2;
          if (r >= R) r -= R, rph ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    if (!F::kScaled) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3, ew = warp - L::kRoles, h = ew >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * COLS;
    const uint32_t acc_free0 = mapa_shared(acc_free, 0);
    uint8_t* const outs = smem + L::kOut + ew * L::kOutBufs * L::kOutBytes;   // one, or two in turn
    uint8_t* out = outs;
    const int kb = p.K >> 7;
    if (!F::kScaled) pdl_wait();               // the activations' scales
    int slot = 0;
    uint32_t ph = 0;
    for (int i = first; i < total; i += step) {
      int mi, ni;
      tile_at<F>(i, p.mt, p.nt, mi, ni);
      const int a0 = mi * 256 + rank * 128 + q * 32, b0 = ni * BN + h * COLS;   // the warp's rows of either operand
      uint32_t packed[COLS / 2];
      if constexpr (F::kScaled) {
        // Both factors always, two values an instruction: a branch on the power (1
        // but for extreme global scales) costs registers that there are not.
        const uint64_t gp = pair_f32(__float_as_uint(p.gpow), __float_as_uint(p.gpow));
        const uint64_t gs = pair_f32(__float_as_uint(p.gscale), __float_as_uint(p.gscale));
        wait_or_abort(acc_full + 8 * slot, ph, p.err, abort_flag);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t v[32];
          tmem_ld32_start(tl + slot * BN + c, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint64_t x = pair_f32(v[2 * j], v[2 * j + 1]);
            mul_f32x2(x, gp);
            mul_f32x2(x, gs);
            packed[c / 2 + j] = pack_bf16(__uint_as_float(static_cast<uint32_t>(x)), __uint_as_float(static_cast<uint32_t>(x >> 32)));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && i + NACC * step < total) pair_arrive(acc_free0 + 8 * slot);
        if (++slot == NACC) slot = 0, ph ^= 1;
      } else {
        // Tiles after this one, as far as it matters: a use of an accumulator is
        // announced as over where NACC uses later another one follows, as only that
        // one waits for it. (An arrive at the other CTA that nobody waits for could
        // come after that CTA's end. With K = 128 there are fewer uses a tile than
        // accumulators, so that a following tile alone does not mean one.)
        const int left = min((total - 1 - i) / step, NACC);
        const float* sa = p.SA + static_cast<long long>(min(a0 + lane, p.M - 1)) * kb;
        // The warp's columns lie in one or two weight blocks; `cross` is the
        // first column of the second.
        const int cross = 128 - (b0 & 127);
        const float* sw0 = p.SW + static_cast<long long>(min(b0, p.N - 1) >> 7) * kb;
        const float* sw1 = p.SW + static_cast<long long>(min(b0 + COLS - 1, p.N - 1) >> 7) * kb;
        uint64_t acc[COLS / 2];
#pragma unroll
        for (int c = 0; c < COLS / 2; ++c) acc[c] = 0;
        // Scales are fetched D blocks ahead of their use: a fetch may take longer
        // than a block.
        constexpr int D = 4;
        constexpr bool kTwo = BN % 256 != 0;
        float fa[D], fw0[D], fw1[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
          fa[d] = d < kb ? sa[d] : 0.0f;
          fw0[d] = d < kb ? __ldg(sw0 + d) : 0.0f;
          fw1[d] = kTwo && d < kb ? __ldg(sw1 + d) : 0.0f;
        }
        for (int k0 = 0; k0 < kb; k0 += D) {
#pragma unroll
          for (int d = 0; d < D; ++d) {
            const int k = k0 + d;
            if (k >= kb) break;
            const float s0 = fa[d] * fw0[d], s1 = kTwo ? fa[d] * fw1[d] : s0;
            const uint64_t f0 = pair_f32(__float_as_uint(s0), __float_as_uint(s0));
            const uint64_t f1 = pair_f32(__float_as_uint(s1), __float_as_uint(s1));
            if (k + D < kb) {
              fa[d] = sa[k + D];
              fw0[d] = __ldg(sw0 + k + D);
              if (kTwo) fw1[d] = __ldg(sw1 + k + D);
            }
            wait_or_abort(acc_full + 8 * slot, ph, p.err, abort_flag);
            __syncwarp();
            tc_fence_after();
            // The next 32 columns are on their way while these are added; the
            // accumulator is free once the last have arrived.
            const uint32_t at = tl + slot * BN;
            uint32_t v[2][2][16];
            tmem_ld16_start(at, v[0][0]);
            tmem_ld16_start(at + 16, v[0][1]);
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += 32) {
              uint32_t(&x)[2][16] = v[(c0 / 32) & 1];
              uint32_t(&y)[2][16] = v[(c0 / 32 + 1) & 1];
              tmem_ld_wait(x[0]);
              if (c0 + 16 < COLS) tmem_ld_after(x[1]);
              if (c0 + 32 < COLS) tmem_ld16_start(at + c0 + 32, y[0]);
              if (c0 + 48 < COLS) tmem_ld16_start(at + c0 + 48, y[1]);
              if (c0 + 32 >= COLS) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && k + NACC < (left + 1) * kb) pair_arrive(acc_free0 + 8 * slot);
              }
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int c = c0 + 16 * u;
                if (c < COLS) {
                  const uint64_t f = (!kTwo || c < cross) ? f0 : f1;
#pragma unroll
                  for (int j = 0; j < 8; ++j) fma_f32x2(acc[c / 2 + j], pair_f32(x[u][2 * j], x[u][2 * j + 1]), f);
                }
              }
            }
            if (++slot == NACC) slot = 0, ph ^= 1;
          }
        }
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j)
          packed[j] = pack_bf16(__uint_as_float(static_cast<uint32_t>(acc[j])), __uint_as_float(static_cast<uint32_t>(acc[j] >> 32)));
      }
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
      // 32 rows of 64 bytes in the 64-byte swizzle (16-byte chunk j of row r at
      // j ^ (r / 2 mod 4)): free of bank conflicts here, and the store map's own.
      const auto chunk_at = [&](int r, int j) { return out + r * 64 + ((j ^ ((r >> 1) & 3)) << 4); };
#pragma unroll
      for (int c = 0; c < COLS; c += 32) {
        if (L::kOutBufs == 2) out = out == outs ? outs + L::kOutBytes : outs;
        if (elect_one()) tma_store_wait_read<L::kOutBufs - 1>();
        __syncwarp();
        if constexpr (kSwap) {                 // the lane has a column of the chunk
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint16_t* v = reinterpret_cast<uint16_t*>(chunk_at(2 * j, lane >> 3)) + (lane & 7);
            v[0] = static_cast<uint16_t>(packed[c / 2 + j]);
            v[32] = static_cast<uint16_t>(packed[c / 2 + j] >> 16);   // row 2j + 1, in the same swizzle
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(chunk_at(lane, j)) =
                make_uint4(packed[c / 2 + 4 * j], packed[c / 2 + 4 * j + 1], packed[c / 2 + 4 * j + 2], packed[c / 2 + 4 * j + 3]);
        }
        const int m0 = kSwap ? b0 + c : a0, n0 = kSwap ? a0 : b0 + c;   // the chunk's place in C
        // A tensor store writes whole 16-byte units, past the end of the row too:
        // its map ends at the last whole unit, and the few columns after that are
        // stored by themselves.
        if (p.align == 16 && n0 < p.N) {
          fence_proxy_async_smem();
          __syncwarp();
          const int whole = p.N & ~7;
          if (elect_one() && m0 < p.M && n0 < whole) tma_store_2d(&tmC, n0, m0, smem_u32(out));
          const int rest = whole - (n0);   // column of the chunk where they begin
          if (rest >= 0 && rest < 32 && m0 + lane < p.M)
            for (int e = 0; whole + e < p.N; ++e)
              p.C[static_cast<long long>(m0 + lane) * p.ldc + whole + e] =
                  *reinterpret_cast<const uint16_t*>(chunk_at(lane, rest >> 3) + e * 2);
          __syncwarp();
        } else if (n0 < p.N) {
          __syncwarp();
          if (p.align >= 8) store_rows<4>(chunk_at, p, m0, n0, lane);
          else if (p.align >= 4) store_rows<2>(chunk_at, p, m0, n0, lane);
          else store_rows<1>(chunk_at, p, m0, n0, lane);
          __syncwarp();
        }
        if (elect_one()) tma_store_close();
      }
    }
    if (elect_one()) tma_store_wait_read<0>();  // the grid ends with the writes
  }
  // Both CTAs are done with the pair's tensor memory. Nothing of the pair is on
  // its way any more: every copy and commit has been waited for, and no arrive
  // was sent that nobody waits for.
  __syncwarp();
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 512);
  }
}

template <class F, int BN, bool kSwap>
cudaError_t launch_many_t(const ActGemmArgs& a, cudaStream_t s) {
  using L = ManyLayout<F, BN>;
  const uint64_t row = F::kScaled ? static_cast<uint64_t>(a.K) / 2 : static_cast<uint64_t>(a.K);
  const uint64_t srow = static_cast<uint64_t>(a.K) / 16;
  const uint64_t M = static_cast<uint64_t>(a.M), N = static_cast<uint64_t>(a.N);
  CUtensorMap ma = {}, mb = {}, msa = {}, msb = {}, mc = {};
  CUtensorMap &mx = kSwap ? mb : ma, &mw = kSwap ? ma : mb, &msx = kSwap ? msb : msa, &msw = kSwap ? msa : msb;
  constexpr auto kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  // Rows of a copy: a CTA's own 128 of the first operand and half the tile's of
  // the second, but the scales of all of those.
  constexpr int kX = kSwap ? BN : 128, kXHalf = kSwap ? BN / 2 : 128;
  constexpr int kW = kSwap ? 128 : BN, kWHalf = kSwap ? 128 : BN / 2;
  cudaError_t e = make_map_2d(&mx, kU8, a.A, row, M, row, 128, kXHalf, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess) e = cached_map_2d(&mw, kU8, a.W, row, N, row, 128, kWHalf, CU_TENSOR_MAP_SWIZZLE_128B);
  if (F::kScaled) {
    if (e == cudaSuccess) e = make_map_2d(&msx, kU8, a.SA, srow, M, srow, 32, kX, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess) e = cached_map_2d(&msw, kU8, a.SW, srow, N, srow, 32, kW, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.C) | static_cast<uintptr_t>(a.ldc) * 2;
  const int align = at % 16 == 0 && a.N >= 8 ? 16 : (at % 8 == 0 ? 8 : (at % 4 == 0 ? 4 : 2));
  if (e == cudaSuccess && align == 16)
    e = make_map_2d(&mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.C, N & ~uint64_t(7), M, static_cast<uint64_t>(a.ldc) * 2, 32, 32,
                    CU_TENSOR_MAP_SWIZZLE_64B);
  static AttrLatch latch;
  if (e == cudaSuccess) e = set_smem_attrs(many_kernel<F, BN, kSwap>, latch, L::kAlloc, true);
  if (e != cudaSuccess) return e;
  ManyParams p = {};
  if (!F::kScaled) {
    p.SA = static_cast<const float*>(a.SA);
    p.SW = static_cast<const float*>(a.SW);
  }
  p.gpow = a.gpow;
  p.gscale = a.gscale;
  p.C = static_cast<uint16_t*>(a.C);
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.ldc = a.ldc;
  p.mt = ((kSwap ? a.N : a.M) + 255) / 256;
  p.nt = ((kSwap ? a.M : a.N) + BN - 1) / BN;
  p.stages = a.K / F::kStageK;
  p.align = align;
  p.err = a.err;
  const long long total = static_cast<long long>(p.mt) * p.nt;
  const int pairs = static_cast<int>(total < a.num_sms / 2 ? total : a.num_sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs * 2);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, many_kernel<F, BN, kSwap>, ma, mb, msa, msb, mc, p);
}

// Width of the weight tiles: the pairs take whole rounds of tiles, and a round
// takes a time proportional to BN + 140 (4 bits) or BN + 100 (8 bits). Measured,
// BN = 256 | 192 | 128, us: 4 bits 333x7168x5120 13.3 | 12.2 | 16.9, 2048x5120x5120
// 30.2 | 25.9 | 34.2, 4096x34816x5120 248 | 274 | 336; 8 bits 333x7168x5120 20.2 |
// 18.3 | 24.4, 2048x7168x5120 55.8 | 63.0 | 68.3, 4096x5120x17408 277 | 284 | 310.
// With 4 bits the operands change places where the activation rows then leave
// less of a tile empty: 128x34816x5120 26.1 us as they are | 22.4 changed,
// 192x34816x5120 26.4 | 25.1, 384x17408x5120 22.8 | 21.0. (256 columns changed do
// not fit the registers: 33.5 us at 256x34816x5120 against 26.7. With 8 bits every
// column would have a factor of its own: 128x34816x5120 41.1 | 43.2.)
template <class F>
cudaError_t launch_many(const ActGemmArgs& a, cudaStream_t s) {
  const long long M = a.M, N = a.N, pairs = a.num_sms / 2;
  const auto cost = [&](long long first, long long second, int bn) {
    return ((first + 255) / 256 * ((second + bn - 1) / bn) + pairs - 1) / pairs * (bn + (F::kScaled ? 140 : 100));
  };
  const long long c256 = cost(M, N, 256), c192 = cost(M, N, 192), c128 = cost(M, N, 128);
  const long long best = c256 < c192 ? (c256 < c128 ? c256 : c128) : (c192 < c128 ? c192 : c128);
  if constexpr (F::kScaled) {
    const long long s192 = cost(N, M, 192), s128 = cost(N, M, 128);
    if (s192 < best && s192 < s128) return launch_many_t<F, 192, true>(a, s);
    if (s128 < best) return launch_many_t<F, 128, true>(a, s);
  }
  if (c256 == best) return launch_many_t<F, 256, false>(a, s);
  return c192 == best ? launch_many_t<F, 192, false>(a, s) : launch_many_t<F, 128, false>(a, s);
}

}  // namespace
}  // namespace act

cudaError_t launch_w4a4_many(const ActGemmArgs& a, cudaStream_t s) { return act::launch_many<act::F4>(a, s); }
cudaError_t launch_w8a8_many(const ActGemmArgs& a, cudaStream_t s) { return act::launch_many<act::F8>(a, s); }

}  // namespace wqp
