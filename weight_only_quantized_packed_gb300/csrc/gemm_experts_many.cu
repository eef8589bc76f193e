// Products of rows with their experts' packed W4A16 matrices on the 5th-
// generation tensor core, for any number of rows an expert.
//
// The weights are the first operand: a tile is 256 weight rows by up to 192 of
// an expert's pairs (its pairs are split evenly, in whole 32s), on a pair of CTAs
// (act.cuh) that hold 128 weight rows and half of the pairs' activations each. One
// CTA an SM, which takes every 76th tile of the walk; a tile's steps are stages of
// 128 K, five of them in tensor memory and shared memory at a time.
//
//  * Rows first go to FP16 in the order of the pairs (half_rows_kernel below), so
//    that both operands are FP16: the hardware converts E2M1 to FP16 at 2.5 clocks
//    a pair and scheduler with its product, to BF16 at 6 to 8, and a tile's rows are
//    consecutive. e2m1 * e4m3 is exact in FP16.
//  * Packed weights, one warp for the codes (tensor copies) and one for the scales
//    (asynchronous copies): a ring of four double stages of 128 rows.
//  * Decoding, three sets of four warps that take the double stages in turn: a
//    thread owns a weight row (a lane of tensor memory), and its FP16 weights go
//    straight to tensor memory, from where the MMAs take them.
//  * Activations, one thread: tensor copies of kBox rows.
//  * MMA, one thread of the even CTA: M = 256, N = the tile's pairs rounded up to
//    32, so that a short expert costs no more than its rows.
//  * Output, eight warps: a lane has a weight row and, column by column, the
//    pairs. Gated: gate and up rows take turns as lanes, and lanes exchange
//    halves of their columns.
//
// Measured (128 experts, rows' conversion included): 333x8, gated 4096x5120 347
// us, 4.4 TB/s of packed weights; 4096x8, gated 4096x5120 950 us, 1.4 PFLOP/s, and
// 4096x8, 5120x2048 563 us (925 to 965 and 525 to 610, process by process; with rows
// of C off 16 bytes, element by element: 1338 and 975, 333x8 368). The plain kernel
// spills 56 bytes a thread of its copying and MMA warps, at 32 registers. No
// unit is full: at 333x8 DRAM is 56 % busy, issue slots and the ALU 58 %, the tensor
// core 21 %. What a stage costs is its hand-overs: copies and barriers alone, without
// decoding, stores to tensor memory and seven of eight MMAs, take 290, 700 and 403
// us; one MMA of eight instead of all saves 7 of 350 and 125 of 960. At a tile's end
// the MMAs wait some 3300 clocks for the accumulator. Did not help: 256 pairs a tile
// and four stages (410, 966, 522 us), as many activations as fit (362, 975, 573), a
// longer ring of weights for narrow tiles (363), two accumulators in turn (362, 924,
// 546), looks at barriers by another warp (356, 946, 515), 256 K a stage (348, 1051,
// 625).
#include "act.cuh"
#include "experts.cuh"
#include "mma_f16.cuh"

namespace wqp {
namespace act {
namespace {

constexpr int kMaxN = 192;                     // pairs of a tile
constexpr int kBox = 32;                       // rows of activations a copy
constexpr int kS = 5;                          // stages of 128 K
constexpr int kHalfB = kMaxN * 64;             // activations of half a stage: kMaxN / 2 rows of 64 K
constexpr int kStageB = 2 * kHalfB;
constexpr int kSets = 3;                       // decoding sets
constexpr int kRing = 4;                       // double stages of packed weights: 128 rows x 256 K
constexpr int kCodes = 128 * 128, kScales = 128 * 16;   // bytes of one
constexpr int kEpi = 8;                        // output warps
constexpr int kOut = 32 * 64;                  // 32 pairs by 32 outputs of an output warp
constexpr int kCodesAt = kS * kStageB, kScalesAt = kCodesAt + kRing * kCodes, kOutAt = kScalesAt + kRing * kScales;
constexpr int kFactorsAt = kOutAt + kEpi * kOut, kFactors = kMaxN / 2 * 4;   // an output warp's pairs' factors
constexpr int kTableAt = kFactorsAt + kEpi * kFactors;
constexpr int kWarpEpi = 4 * kSets, kWarpMma = kWarpEpi + kEpi, kWarpRows = kWarpMma + 1, kWarpCodes = kWarpMma + 2, kWarpScales = kWarpMma + 3;
constexpr int kThreads = (kWarpMma + 4) * 32;  // registers are shared out by four warps at a time
// Registers a thread: at launch (and decoding), of the output's and of the rest.
// A plain output holds more at a time; 104 and 32 for both took 929 us instead of 921
// at 4096x8, gated 4096x5120, 96 and 40 for both 537 instead of 529 at 5120x2048.
constexpr int kRegsLaunch = 80;
__host__ __device__ constexpr int regs_out(bool gated) { return gated ? 96 : 104; }
__host__ __device__ constexpr int regs_rest(bool gated) { return gated ? 40 : 32; }
constexpr bool regs_fit(bool gated) {
  return kSets * kRegsLaunch + kEpi / 4 * regs_out(gated) + regs_rest(gated) <= kThreads / 128 * kRegsLaunch;
}
static_assert(regs_fit(true) && regs_fit(false), "registers");
// Tensor memory: the accumulator, then kS stages of 64 columns.
constexpr uint32_t kColA = kMaxN;
static_assert(kColA + kS * 64 <= 512 && kSets <= kRing && kS > 2 * (kSets - 1), "stages");

constexpr int many_bytes(int E) { return 1024 + kTableAt + experts::Table::bytes(E); }
static_assert(many_bytes(kMaxExperts) <= 226 * 1024, "shared memory");

// idesc_bf16 with FP16 operands.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D (+)= A * B^T, A from tensor memory, 16-bit operands, K = 16, by a pair.
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// One arrival at the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_land(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// An arrival that waits for nothing of this thread: what it announces is in
// tensor memory, behind the store's own wait and fence. (A release would wait for
// the copies of later chunks.)
__device__ __forceinline__ void pair_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// wait_or_abort with a long time limit of the wait itself: the polls of the warps
// that wait take issue slots from those that decode.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, unsigned* err, volatile int* abort_flag) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (int i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000)
        : "memory");
    if (ok) return true;
    if ((i & 15) == 15) {
      if (*abort_flag) return false;
      const uint64_t t = global_ns();
      if (!t0) t0 = t;
      else if (t - t0 > kWaitLimitNs) break;
    }
  }
  set_error(err, WQP_DEV_ERR_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// A tile of the walk: token tiles of each expert in turn, all its weight tiles
// one after the other.
struct Tile {
  int expert, nt, p0, pairs, n;                // pairs p0 .. p0 + pairs - 1 of the order; n: rounded up
  __device__ __forceinline__ void at(const experts::Table& table, int id, int weight_tiles) {
    const int t = id / weight_tiles;
    nt = id - t * weight_tiles;
    expert = table.expert_of(t);
    const int begin = table.begin[expert], count = table.begin[expert + 1] - begin;
    const int tiles = (count + kMaxN - 1) / kMaxN;
    // Even shares of whole 32s, at most kMaxN, none empty.
    const int whole = (count + 31) >> 5, share = t - table.tiles[expert];
    const int from = static_cast<int>(static_cast<long long>(whole) * share / tiles) * 32;
    const int to = static_cast<int>(static_cast<long long>(whole) * (share + 1) / tiles) * 32;
    p0 = begin + from;
    pairs = min(count, to) - from;
    n = (pairs + 31) & ~31;
  }
};

// Eight E2M1 codes of a word with their group's scale (f16x2), exactly.
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t s, uint32_t* r) {
  r[0] = f16op::mul_f16x2(f16op::e2m1x2_byte<0>(w), s);
  r[1] = f16op::mul_f16x2(f16op::e2m1x2_byte<1>(w), s);
  r[2] = f16op::mul_f16x2(f16op::e2m1x2_byte<2>(w), s);
  r[3] = f16op::mul_f16x2(f16op::e2m1x2_byte<3>(w), s);
}

// How C's rows are aligned, in bytes: 16 or 2.
__device__ __forceinline__ int out_align(const ExpertsArgs& a) {
  return (reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && a.ldc % 8 == 0) ? 16 : 2;
}
// Up to 8 outputs of a row, of which `left` are inside it.
__device__ __forceinline__ void store_piece(uint16_t* c, const uint8_t* from, int left, int align) {
  const uint4 v = *reinterpret_cast<const uint4*>(from);
  if (align == 16 && left >= 8) {
    *reinterpret_cast<uint4*>(c) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) c[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
  }
}

// The row of a stage's packed weights that lane `row` of tensor memory takes.
// Gated: a warp's lanes 0..15 have gates (rows 0..63), 16..31 the ups of the same
// outputs (rows 64..127).
template <bool kGated>
__device__ __forceinline__ int smem_row(int row) {
  return kGated ? (row & 16) * 4 + (row >> 5) * 16 + (row & 15) : row;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // full (a stage's activations and decoded weights) and acc_free count both CTAs'
  // work and are used in the even CTA; done (a stage's MMAs) and acc_full are told
  // to both; raw_full and raw_empty are each CTA's own.
  __shared__ __align__(8) uint64_t full_sh[kS], done_sh[kS], raw_full_sh[kRing], raw_empty_sh[kRing], acc_full_sh, acc_free_sh, drained_sh;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const uint32_t full = smem_u32(full_sh), done = smem_u32(done_sh), raw_full = smem_u32(raw_full_sh), raw_empty = smem_u32(raw_empty_sh);
  const uint32_t acc_full = smem_u32(&acc_full_sh), acc_free = smem_u32(&acc_free_sh), drained = smem_u32(&drained_sh);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(full + 8 * i, 2 * (1 + 4));
      mbar_init(done + 8 * i, 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(raw_full + 8 * i, 1 + 32);
      mbar_init(raw_empty + 8 * i, 4);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 2 * kEpi);
    mbar_init(drained, 1);
    abort_sh = 0;
    mbar_fence_init();
  }
  __syncwarp();
  cluster_arrive_relaxed();
  if (warp == kWarpMma) {
    pair_tmem_alloc(smem_u32(&tmem_sh), 512);
    tc_fence_before();
  }
  pdl_launch_dependents();
  pdl_wait();
  const int R = a.T * a.slots;
  experts::Table table;                        // its barriers publish tmem_sh too
  table.make(smem + kTableAt, a.offsets, a.E, R, [](int n) { return (n + kMaxN - 1) / kMaxN; });
  tc_fence_after();
  cluster_wait();
  const uint32_t tmem = tmem_sh;

  const int outs = kGated ? a.N / 2 : a.N;
  constexpr int kOuts = kGated ? 128 : 256;    // outputs of a tile
  const int weight_tiles = (outs + kOuts - 1) / kOuts, total = table.total() * weight_tiles;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int mine = first < total ? (total - first + step - 1) / step : 0;   // tiles of this pair
  const int stages = a.K >> 7;                                              // of a tile
  const uint32_t full0 = mapa_shared(full, 0);

  if (warp < kWarpEpi) {
    // Weights. A thread has a lane of tensor memory; a set of four warps takes every
    // kSets-th stage.
    const int set = warp >> 2, row = (warp & 3) * 32 + lane;
    // Rows of 128 bytes in the 128-byte swizzle: piece j of row r at j ^ (r mod 8).
    const int from = smem_row<kGated>(row);
    const uint8_t* const codes = smem + kCodesAt + from * 128;
    const uint8_t* const scales_at = smem + kScalesAt + from * 16;
    const uint32_t at = tmem + kColA + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // Double stage u of tile i, number `get` of all, is for this set; its stages go
    // to places s and s + 1.
    const int doubles = (stages + 1) >> 1;
    int i = 0, u = 0, get = 0, s = 0;
    uint32_t raw_ph = 0, ph = 1;
    const auto skip = [&](int n) {             // the next n double stages
      for (; n > 0 && i < mine; --n) {
        s += 2 * u + 1 < stages ? 2 : 1;
        if (s >= kS) s -= kS, ph ^= 1;
        if (++get == kRing) get = 0, raw_ph ^= 1;
        if (++u == doubles) u = 0, ++i;
      }
    };
    skip(set);
    while (i < mine) {
      // A set sees only every kSets-th use of the ring, and a barrier tells its phases
      // apart by parity alone: that the place's last contents have been used shows that
      // the phase waited for is the next one.
      if (!__all_sync(0xFFFFFFFFu, wait_long(raw_empty + 8 * get, raw_ph ^ 1, a.err, abort_flag) &&
                                       wait_long(raw_full + 8 * get, raw_ph, a.err, abort_flag)))
        break;
      const int x = from & 7;
      int place = s;
      uint32_t place_ph = ph;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (2 * u + d >= stages) break;
        uint4 packed[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) packed[j] = *reinterpret_cast<const uint4*>(codes + get * kCodes + (((4 * d + j) ^ x) << 4));
        const uint2 scales = *reinterpret_cast<const uint2*>(scales_at + get * kScales + 8 * d);
        if (d == 1 || 2 * u + 1 >= stages) {
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_empty + 8 * get);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 w0 = packed[2 * h], w1 = packed[2 * h + 1];
          const uint32_t s4 = h ? scales.y : scales.x;
          const uint32_t f01 = e4m3x2_to_f16x2(s4 & 0xFFFFu), f23 = e4m3x2_to_f16x2(s4 >> 16);
          const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          uint32_t r[32];
#pragma unroll
          for (int gr = 0; gr < 4; ++gr) {
            const uint32_t f = gr < 2 ? f01 : f23;
            const uint32_t sf = __byte_perm(f, f, gr & 1 ? 0x3232 : 0x1010);
            decode_word(ww[2 * gr], sf, r + 8 * gr);
            decode_word(ww[2 * gr + 1], sf, r + 8 * gr + 4);
          }
          // Parity 1 of a barrier that has completed no phase counts as complete. The set's
          // stage before was kS stages back or later, so it has seen the phase before.
          if (h == 0 && !__all_sync(0xFFFFFFFFu, wait_long(done + 8 * place, place_ph, a.err, abort_flag))) goto decoding_over;
          if (h == 0) tc_fence_after();
          tmem_st32(at + place * 64 + h * 32, r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_arrive_relaxed(full0 + 8 * place);
        if (++place == kS) place = 0, place_ph ^= 1;
      }
      skip(kSets);
    }
  decoding_over:;
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(regs_out(kGated)));
    // Output: this warp's 32 lanes, all columns. First into registers as BF16, so
    // that the accumulator is free for the next tile; then, while that is
    // computed, 32 pairs at a time through shared memory to rows of C.
    const int q = warp & 3, ew = warp - kWarpEpi, h = ew >> 2;   // every second 32 columns
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t acc_free0 = mapa_shared(acc_free, 0);
    uint8_t* const out = smem + kOutAt + ew * kOut;
    float* const factors = reinterpret_cast<float*>(smem + kFactorsAt + ew * kFactors);   // the inverses of their rows' scaling
    const int align = out_align(a);
    uint32_t ph = 0;
    constexpr int kChunks = kMaxN / 32 / 2;
    for (int i = 0; i < mine; ++i) {
      Tile tile;
      tile.at(table, first + i * step, weight_tiles);
      const float gs = a.globals ? a.globals[tile.expert] : 1.0f;
      int pl[kChunks];                         // the pair of column 32 (2 ch + h) + lane, and
      __syncwarp();
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        const int c = 32 * (2 * ch + h) + lane, p = c < tile.pairs ? a.rows[tile.p0 + c] : -1;
        pl[ch] = static_cast<unsigned>(p) < static_cast<unsigned>(R) ? p : -1;
        factors[32 * ch + lane] = pl[ch] >= 0 ? a.row_scales[tile.p0 + c] : 1.0f;
      }
      wait_long(acc_full, ph, a.err, abort_flag);
      ph ^= 1;
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
      tc_fence_after();
      // The inverse power of two first: FP32 may not hold its product with gs where it
      // holds the output.
      uint32_t packed[kChunks][kGated ? 8 : 16];
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        if (32 * (2 * ch + h) >= tile.n) break;
        uint32_t v[32];
        tmem_ld32_start(tl + 32 * (2 * ch + h), v);
        tmem_ld_wait(v);
        if constexpr (kGated) {
          // Lanes 0..15 have gates and take columns 0..15, the others the same outputs'
          // ups and columns 16..31.
          const bool odd = lane & 16;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f2 = *reinterpret_cast<const float2*>(factors + 32 * ch + (lane & 16) + 2 * j);
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 2 * j + e;
              const float keep = __uint_as_float(odd ? v[16 + c] : v[c]), give = __uint_as_float(odd ? v[c] : v[16 + c]);
              const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 16);
              const float f = e ? f2.y : f2.x;
              y[e] = experts::silu((odd ? got : keep) * f * gs) * ((odd ? keep : got) * f * gs);
            }
            packed[ch][j] = pack_bf16(y[0], y[1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 f = *reinterpret_cast<const float2*>(factors + 32 * ch + 2 * j);
            packed[ch][j] = pack_bf16(__uint_as_float(v[2 * j]) * f.x * gs, __uint_as_float(v[2 * j + 1]) * f.y * gs);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && i + 1 < mine) pair_arrive(acc_free0);

      // Outputs o0 .. of this warp: 32, or (gated) 16.
      const int o0 = kGated ? tile.nt * 128 + rank * 64 + q * 16 : tile.nt * 256 + rank * 128 + q * 32;
      const int left = outs - o0;
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        if (32 * (2 * ch + h) >= tile.n) break;
        __syncwarp();
        if constexpr (kGated) {                // 32 pairs of 32 bytes, piece h of pair c at h ^ (c / 4 mod 2)
          const int n = lane & 15;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 2 * j + (lane & 16);
            *reinterpret_cast<uint16_t*>(out + c * 32 + (((n >> 3) ^ ((c >> 2) & 1)) << 4) + (n & 7) * 2) = static_cast<uint16_t>(packed[ch][j]);
            *reinterpret_cast<uint16_t*>(out + (c + 1) * 32 + (((n >> 3) ^ ((c >> 2) & 1)) << 4) + (n & 7) * 2) =
                static_cast<uint16_t>(packed[ch][j] >> 16);
          }
          __syncwarp();
          const int p = pl[ch];
          if (p >= 0) {
            uint16_t* const c = static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc + o0;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              store_piece(c + 8 * e, out + lane * 32 + ((e ^ ((lane >> 2) & 1)) << 4), left - 8 * e, align);
          }
        } else {                               // 32 pairs of 64 bytes, piece h of pair c at h ^ (c / 2 mod 4)
          const int n = lane;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint8_t* const d = out + 2 * j * 64 + (((n >> 3) ^ (j & 3)) << 4) + (n & 7) * 2;
            *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(packed[ch][j]);
            *reinterpret_cast<uint16_t*>(d + 64) = static_cast<uint16_t>(packed[ch][j] >> 16);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = 8 * k + (lane >> 2), e = lane & 3;
            const int p = __shfl_sync(0xFFFFFFFFu, pl[ch], c);
            if (p >= 0)
              store_piece(static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc + o0 + 8 * e,
                          out + c * 64 + ((e ^ ((c >> 1) & 3)) << 4), left - 8 * e, align);
          }
        }
      }
    }
  } else if (warp < kWarpMma + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(regs_rest(kGated)));
  }
  if (warp == kWarpRows && elect_one()) {
    // Activations: this CTA's half of the tile's rows, kBox at a time (more of them
    // than the tile has: their columns go nowhere), in two tiles of 64 K.
    int s = 0;
    uint32_t ph = 1;
    long long c = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      Tile tile;
      tile.at(table, first + i * step, weight_tiles);
      const int half = tile.n >> 1, row0 = tile.p0 + rank * half, boxes = (half + kBox - 1) / kBox;
      for (int k = 0; k < stages; ++k, ++c) {
        if (c >= kS && !(ok = wait_long(done + 8 * s, ph, a.err, abort_flag))) break;
        // The even CTA's barrier takes both CTAs' bytes; each announces its own.
        pair_arrive_expect_tx(full0 + 8 * s, boxes * kBox * 256);
        const uint32_t dst = sb + s * kStageB;
        for (int b = 0; b < boxes; ++b) {
          pair_tma_load_2d(dst + b * kBox * 128, &tmA, k * 128, row0 + b * kBox, full0 + 8 * s);
          pair_tma_load_2d(dst + kHalfB + b * kBox * 128, &tmA, k * 128 + 64, row0 + b * kBox, full0 + 8 * s);
        }
        if (++s == kS) s = 0, ph ^= 1;
      }
    }
    // Every stage's MMAs are done, and told to both CTAs, before this one ends; or
    // (after an abort) its copies have at least arrived.
    for (int t = 0; t < kS; ++t) {
      if (c >= kS - t && !wait_long(done + 8 * s, ph, a.err, abort_flag) && rank == 0) mbar_wait(full + 8 * s, ph, a.err);
      if (++s == kS) s = 0, ph ^= 1;
    }
  } else if (warp == kWarpCodes && elect_one()) {
    // Packed weights: 128 rows of a tile, 128 bytes each (gated: 64 gate rows, then
    // the 64 up rows of the same outputs; behind the end of a row: zeros).
    int s = 0;
    uint32_t ph = 1;
    long long c = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      const int id = first + i * step, t = id / weight_tiles, nt = id - t * weight_tiles, e = table.expert_of(t);
      const int n0 = kGated ? nt * 128 + rank * 64 : nt * 256 + rank * 128;
      for (int k = 0; k < stages; k += 2, ++c) {
        if (c >= kRing && !(ok = wait_long(raw_empty + 8 * s, ph, a.err, abort_flag))) break;
        mbar_arrive_expect_tx(raw_full + 8 * s, kCodes);
        const uint32_t dst = sb + kCodesAt + s * kCodes;
        tma_load_3d(dst, &tmW, k * 64, n0, e, raw_full + 8 * s);
        if (kGated) tma_load_3d(dst + kCodes / 2, &tmW, k * 64, outs + n0, e, raw_full + 8 * s);
        if (++s == kRing) s = 0, ph ^= 1;
      }
    }
    // Every copy has been used, or (after an abort) has at least arrived.
    for (int t = 0; t < kRing; ++t) {
      if (c >= kRing - t && !wait_long(raw_empty + 8 * s, ph, a.err, abort_flag)) mbar_wait(raw_full + 8 * s, ph, a.err);
      if (++s == kRing) s = 0, ph ^= 1;
    }
  } else if (warp == kWarpScales) {
    // Their scales: 16 bytes of a row (8 behind an odd stage), four rows a lane; rows
    // past the last read that one.
    int s = 0;
    uint32_t ph = 1;
    long long c = 0;
    bool ok = true;
    const bool odd = stages & 1;               // rows are not multiples of 16 bytes
    const uint32_t dst = sb + kScalesAt + lane * 16;
    for (int i = 0; i < mine && ok; ++i) {
      const int id = first + i * step, t = id / weight_tiles, nt = id - t * weight_tiles;
      const long long base = static_cast<long long>(table.expert_of(t)) * a.N;
      const uint8_t* src[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 32 * j + lane;
        const long long n = kGated ? min(nt * 128 + rank * 64 + (r & 63), outs - 1) + (r >> 6) * static_cast<long long>(outs)
                                   : min(nt * 256 + rank * 128 + r, outs - 1);
        src[j] = a.scales + (base + n) * (a.K >> 4);
      }
      for (int k = 0; k < stages; k += 2, ++c) {
        if (c >= kRing && !(ok = __all_sync(0xFFFFFFFFu, wait_long(raw_empty + 8 * s, ph, a.err, abort_flag)))) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t d = dst + s * kScales + j * 512;
          if (!odd) {
            copy16(d, src[j]);
          } else {
            copy8(d, src[j]);
            if (k + 1 < stages) copy8(d + 8, src[j] + 8);
          }
          src[j] += 16;
        }
        copies_land(raw_full + 8 * s);
        if (++s == kRing) s = 0, ph ^= 1;
      }
    }
    copies_close();
    copies_wait<0>();
  } else if (warp == kWarpMma && rank == 0) {
    // All by one thread: the warp's own steps between stages took longer than a
    // narrow stage's MMAs. A look at a barrier costs it some 120 clocks, as much as
    // those MMAs, so it looks at two at a time.
    if (elect_one()) {
      const uint64_t bd0 = tile_desc(sb);
      int s = 0;
      uint32_t ph = 0, acc_ph = 1;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        Tile tile;
        tile.at(table, first + i * step, weight_tiles);
        const uint32_t idesc = idesc_f16(256, tile.n);
        if (i > 0) ok = wait_long(acc_free, acc_ph, a.err, abort_flag);
        acc_ph ^= 1;
        int ready = 0;                         // stages from this one on that are known to be full
        for (int k = 0; k < stages && ok; ++k) {
          if (!ready) {
            const int s1 = s + 1 == kS ? 0 : s + 1;
            const bool l0 = mbar_test(full + 8 * s, ph), l1 = mbar_test(full + 8 * s1, s1 ? ph : ph ^ 1);
            ready = l0 && l1 ? 2 : 1;
            if (!l0) ok = wait_long(full + 8 * s, ph, a.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
          }
          --ready;
          const uint64_t bd = bd0 + s * (kStageB >> 4);
          const uint32_t at = tmem + kColA + s * 64;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            pair_mma_ts(tmem, at + 8 * j, bd + (j >> 2) * (kHalfB >> 4) + 2 * (j & 3), idesc, (k | j) ? 1u : 0u);
          pair_commit(done + 8 * s);
          if (k + 1 == stages) pair_commit(acc_full);
          if (++s == kS) s = 0, ph ^= 1;
        }
      }
      pair_commit_own(drained);
      mbar_wait(drained, 0, a.err);
    }
  }
  // Nothing of the pair is on its way any more, and both are done with the
  // pair's tensor memory.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == kWarpMma) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 512);
  }
}

// The rows of X (BF16) in the order of the pairs, as FP16 [R, K], each times a
// power of two (f16_shift): exact for what is at least 2^-31 of its largest
// magnitude; what is smaller is off by 2^-39 of that at most. inv [R] receives
// the inverse powers. In that order a tile's rows are consecutive, and
// few threads copy them (gathered by the kernel itself, through asynchronous
// copies, they took four warps, and their latency every third stage).
constexpr int kHalfThreads = 128, kHalfHeld = 8;   // chunks of 8 elements a thread keeps between the passes
// kWarps warps a row: one for rows that its registers hold (a block's latency per
// row of 4 KB took 58 us at 32768x2048).
template <int kWarps>
__global__ void __launch_bounds__(kHalfThreads)
    half_rows_kernel(const uint16_t* X, const int* rows, uint16_t* Y, float* inv, int R, int slots, int K, int ldx) {
  constexpr int kThreads = kWarps * 32, kRows = kHalfThreads / kThreads;
  __shared__ uint32_t most_sh[kHalfThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int at = static_cast<int>(threadIdx.x) % kThreads, r = blockIdx.x * kRows + static_cast<int>(threadIdx.x) / kThreads;
  const int p = r < R ? rows[r] : -1;
  if (static_cast<unsigned>(p) >= static_cast<unsigned>(R)) return;   // all threads of the row
  const uint16_t* x = X + static_cast<long long>(p / slots) * ldx;
  uint16_t* y = Y + static_cast<long long>(r) * K;
  const int chunks = K >> 3;
  uint4 held[kHalfHeld];
  uint32_t mx = 0;
  const auto most = [&](const uint4& v) {          // BF16 magnitudes order like their bits
    mx = __vmaxu2(__vmaxu2(mx, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  };
#pragma unroll
  for (int i = 0; i < kHalfHeld; ++i) {
    const int c = at + i * kThreads;
    held[i] = c < chunks ? *reinterpret_cast<const uint4*>(x + 8 * c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kHalfHeld; ++i) most(held[i]);
  for (int c = at + kHalfHeld * kThreads; c < chunks; c += kThreads) most(*reinterpret_cast<const uint4*>(x + 8 * c));
  mx = __reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFFFu, mx >> 16));
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) most_sh[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHalfThreads / 32; ++i) mx = max(mx, most_sh[i]);
  }
  const int sh = f16op::f16_shift(mx);
  const float scale = f16op::pow2(sh);
  if (at == 0) inv[r] = f16op::pow2(-sh);
  const auto put = [&](int c, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = f16op::f32x2_to_f16x2(bf16hi(w[i]) * scale, bf16lo(w[i]) * scale);
    *reinterpret_cast<uint4*>(y + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
  };
#pragma unroll
  for (int i = 0; i < kHalfHeld; ++i) {
    const int c = at + i * kThreads;
    if (c < chunks) put(c, held[i]);
  }
  for (int c = at + kHalfHeld * kThreads; c < chunks; c += kThreads) put(c, *reinterpret_cast<const uint4*>(x + 8 * c));
}

cudaError_t launch_half_rows(const ExpertsArgs& a, uint16_t* rows, float* inv, cudaStream_t s) {
  const int R = a.T * a.slots;
  const auto* X = static_cast<const uint16_t*>(a.A);
  if (a.K <= 32 * 8 * kHalfHeld)
    return launch(half_rows_kernel<1>, dim3((R + 3) / 4), dim3(kHalfThreads), 0, s, a.pdl, X, a.rows, rows, inv, R, a.slots, a.K, a.lda);
  return launch(half_rows_kernel<4>, dim3(R), dim3(kHalfThreads), 0, s, a.pdl, X, a.rows, rows, inv, R, a.slots, a.K, a.lda);
}

template <bool kGated>
cudaError_t launch_experts_many_t(const ExpertsArgs& a, bool pdl, cudaStream_t s) {
  static AttrLatch latch;
  cudaError_t e = set_smem_attrs(experts_kernel<kGated>, latch, many_bytes(kMaxExperts), true);
  CUtensorMap ma = {}, mw = {};
  const uint64_t row = static_cast<uint64_t>(a.K) / 2, N = static_cast<uint64_t>(a.N);
  if (e == cudaSuccess)
    e = make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.A, a.K, static_cast<uint64_t>(a.T) * a.slots, static_cast<uint64_t>(a.K) * 2, 64,
                    kBox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess)
    e = make_map_3d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.W, {row, N, static_cast<uint64_t>(a.E)}, {row, row * N},
                      {128, kGated ? 64 : 128, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_sms / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = many_bytes(a.E);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, experts_kernel<kGated>, ma, mw, a);
}

}  // namespace
}  // namespace act

// Two launches: the rows to FP16, in the workspace (decoding to BF16 took more
// than twice the time), and the products. The second may always overlap the first,
// for which it waits before it reads anything.
cudaError_t launch_w4a16_experts_many(const ExpertsArgs& a, cudaStream_t s) {
  ExpertsArgs h = a;
  const int R = a.T * a.slots;
  uint16_t* rows = static_cast<uint16_t*>(a.workspace);
  float* inv = reinterpret_cast<float*>(rows + static_cast<size_t>(R) * a.K);
  const cudaError_t e = act::launch_half_rows(a, rows, inv, s);
  if (e != cudaSuccess) return e;
  h.A = rows;
  h.row_scales = inv;
  return a.gated ? act::launch_experts_many_t<true>(h, true, s) : act::launch_experts_many_t<false>(h, true, s);
}

}  // namespace wqp
