// Products of rows with their experts' packed W4A16 matrices on the 5th-
// generation tensor core, for any number of rows an expert.
//
// The weights are the first operand: a tile is 256 weight rows by up to 256 of
// an expert's pairs, on a pair of CTAs (act.cuh) that hold 128 weight rows and
// half of the pairs' activations each. Decoding them is what has to be fed
// (128 * 128 weights a CTA and stage), and it has the same cost however few
// pairs there are: from about 100 pairs a tile the tensor core is the limit,
// below that the decoding or the bytes.
//
//  * Decoding, two sets of four warps that take the stages in turn: a
//    thread owns a weight row (a lane of tensor memory). Its codes and scales
//    come by asynchronous copies into a ring that only its warp uses, so no
//    barrier is in between; e2m1 * e4m3 is exact in BF16, and goes straight to
//    tensor memory, from where the MMAs take it.
//  * Activations, four warps: rows of BF16 gathered by pair, 16 bytes a copy,
//    into 128-byte-swizzled tiles of 64 K, two a stage.
//  * MMA, one warp of the even CTA: M = 256, N = the tile's pairs rounded up to
//    32, so that a short expert costs no more than its rows.
//  * Output, four warps: a lane has a weight row and, column by column, the
//    pairs. Gated: gate and up rows take turns as lanes, and lanes exchange
//    halves of their columns.
#include "act.cuh"
#include "experts.cuh"
#include "mma_f16.cuh"

namespace wqp {
namespace act {
namespace {

constexpr int kS = 4;                          // stages of 128 K
constexpr int kHalfB = 128 * 128;              // activations of half a stage: 128 rows of 64 K
constexpr int kStageB = 2 * kHalfB;
constexpr int kSets = 2, kSlots = 4;           // decoding sets, and stages in a set's ring
constexpr int kSlot = 128 * 72;                // codes and scales of 128 rows x 128 K
constexpr int kRaw = kS * kStageB, kOutAt = kRaw + kSets * kSlots * kSlot;
constexpr int kOut = 32 * 64;                  // 32 pairs by 32 outputs of an output warp
constexpr int kTableAt = kOutAt + 4 * kOut;
constexpr int kFeeders = 4, kDecoders = 4 * kSets, kEpi = 4;
constexpr int kWarpDec = kFeeders, kWarpEpi = kWarpDec + kDecoders, kWarpMma = kWarpEpi + kEpi,
              kWarpRelay = kWarpMma + 1;
constexpr int kThreads = (kWarpMma + 4) * 32;  // registers are shared out by four warps at a time
// Registers: launched with 96 a thread, 480 to the five threads of one index.
constexpr int kRegsLaunch = 96, kRegsFeed = 80, kRegsOut = 168, kRegsRest = 40;
static_assert(kThreads == 640 && kRegsFeed + 2 * kRegsLaunch + kRegsOut + kRegsRest <= 5 * kRegsLaunch, "registers");
constexpr int kMaxN = 256;                     // pairs of a tile
constexpr uint32_t kColA = 256;                // tensor memory: accumulator, then kS stages of 64 columns
static_assert(kColA + kS * 64 <= 512, "tensor memory");

constexpr int many_bytes(int E) { return 1024 + kTableAt + experts::Table::bytes(E); }
static_assert(many_bytes(kMaxExperts) <= 226 * 1024, "shared memory");

// D (+)= A * B^T, A from tensor memory, BF16, K = 16, by a pair.
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
    const int each = ((count + tiles - 1) / tiles + 31) & ~31;   // even shares: at most kMaxN, none empty
    const int from = (t - table.tiles[expert]) * each;
    p0 = begin + from;
    pairs = min(count - from, each);
    n = (pairs + 31) & ~31;
  }
};

// Eight E2M1 codes of a word to BF16 pairs with their group's scale (f16x2),
// exactly: the product is exact in FP16, and widened to FP32 it has nothing in
// its lower half.
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t s, uint32_t* r) {
  r[0] = f16x2_to_bf16x2_exact(f16op::mul_f16x2(f16op::e2m1x2_byte<0>(w), s));
  r[1] = f16x2_to_bf16x2_exact(f16op::mul_f16x2(f16op::e2m1x2_byte<1>(w), s));
  r[2] = f16x2_to_bf16x2_exact(f16op::mul_f16x2(f16op::e2m1x2_byte<2>(w), s));
  r[3] = f16x2_to_bf16x2_exact(f16op::mul_f16x2(f16op::e2m1x2_byte<3>(w), s));
}

// g * sigmoid(g), through e^-|g|, which cannot overflow: 4 roundings and two
// approximations of 2 ulp.
__device__ __forceinline__ float silu(float g) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g * (g < 0.0f ? t : 1.0f), 1.0f + t);
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

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // full and acc_free count both CTAs' work and are used in the even CTA; empty
  // and acc_full are told to both; landed is each CTA's own.
  __shared__ __align__(8) uint64_t full_sh[kS], empty_sh[kS], landed_sh[kS], acc_full_sh, acc_free_sh, drained_sh;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const uint32_t full = smem_u32(full_sh), empty = smem_u32(empty_sh), landed = smem_u32(landed_sh);
  const uint32_t acc_full = smem_u32(&acc_full_sh), acc_free = smem_u32(&acc_free_sh), drained = smem_u32(&drained_sh);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(full + 8 * i, 2 * (1 + 4));
      mbar_init(landed + 8 * i, kFeeders * 32);
      mbar_init(empty + 8 * i, 1);
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

  if (warp < kWarpDec) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFeed));
    // Activations. Thread t copies 16-byte piece t % 16 of rows t / 16 + 8 i.
    const int piece = threadIdx.x & 15, row0 = threadIdx.x >> 4;
    const uint32_t dst0 = sb + (piece >> 3) * kHalfB + row0 * 128 + (((piece & 7) ^ row0) << 4);
    int s = 0;
    uint32_t ph = 1;
    long long issued = 0;
    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
      Tile tile;
      tile.at(table, first + i * step, weight_tiles);
      const int half = tile.n >> 1;            // of this CTA, a multiple of 16
      const uint8_t* src[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {           // rows without a pair: any row, their columns go nowhere
        const int r = row0 + 8 * j, c = rank * half + r;
        const int p = r < half && c < tile.pairs ? a.rows[tile.p0 + c] : 0;
        const int t = static_cast<unsigned>(p) < static_cast<unsigned>(R) ? p / a.slots : 0;
        src[j] = static_cast<const uint8_t*>(a.A) + static_cast<long long>(t) * a.lda * 2 + piece * 16;
      }
      for (int k = 0; k < stages; ++k) {
        if (issued >= kS) ok = __all_sync(0xFFFFFFFFu, wait_or_abort(empty + 8 * s, ph, a.err, abort_flag));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          if (8 * j >= half) break;
          copy16(dst0 + s * kStageB + j * 1024, src[j]);
          copy16(dst0 + s * kStageB + j * 1024 + 1024, src[j + 1]);
          src[j] += 256;
          src[j + 1] += 256;
        }
        copies_land(landed + 8 * s);
        ++issued;
        if (++s == kS) s = 0, ph ^= 1;
      }
    }
    copies_close();
    copies_wait<0>();
    // Every stage's MMAs are done, and told to both CTAs, before this one ends.
    if (warp == 0) {
      const int used = issued < kS ? static_cast<int>(issued) : kS;
      for (int t = 0; t < used && ok; ++t) {
        const int at = used < kS ? t : s;
        ok = __all_sync(0xFFFFFFFFu, wait_or_abort(empty + 8 * at, used < kS ? 0u : ph, a.err, abort_flag));
        if (used == kS && ++s == kS) s = 0, ph ^= 1;
      }
    }
  } else if (warp < kWarpEpi) {
    // Weights. Thread: lane `row` of tensor memory.
    const int set = (warp - kWarpDec) >> 2, row = (warp & 3) * 32 + lane;
    // A warp's rows in a slot: 32 rows of 64 bytes, piece j of row r at j ^ (r / 2
    // mod 4), then 32 of 8. A copy takes whole rows of 64 bytes (as 16 bytes of 32
    // rows the copies took most of a stage's time).
    const uint32_t raw = sb + kRaw + set * kSlots * kSlot + (warp & 3) * kSlot / 4;
    const uint8_t* const raw_ptr = smem + kRaw + set * kSlots * kSlot + (warp & 3) * kSlot / 4;
    const uint32_t dst_w = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    const uint32_t at = tmem + kColA + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // The next stage of this set to copy: the stages of all tiles are numbered
    // through, and the sets take them in turn.
    int ai = 0, ac = set;                      // tile of the pair, stage in it
    while (ai < mine && ac >= stages) ac -= stages, ++ai;
    int loaded = -1, put = 0;
    const uint8_t *w[4] = {}, *sc = nullptr;
    const auto copy_next = [&] {
      if (ai < mine) {
        if (loaded != ai) {
          loaded = ai;
          const int id = first + ai * step, t = id / weight_tiles, nt = id - t * weight_tiles;
          const long long base = static_cast<long long>(table.expert_of(t)) * a.N;
          const auto row_at = [&](int r) {     // the weight row of lane r of the tile; rows past the last read that one
            return kGated ? base + min(nt * 128 + rank * 64 + (r >> 1), outs - 1) + (r & 1) * static_cast<long long>(outs)
                          : base + min(nt * 256 + rank * 128 + r, outs - 1);
          };
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = a.W + row_at((warp & 3) * 32 + 8 * j + (lane >> 2)) * (a.K >> 1) + ac * 64 + (lane & 3) * 16;
          sc = a.scales + row_at(row) * (a.K >> 4) + ac * 8;
        }
        const uint32_t dst = raw + put * kSlot;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          copy16(dst + j * 512 + dst_w, w[j]);
          w[j] += kSets * 64;
        }
        copy8(dst + 2048 + lane * 8, sc);
        sc += kSets * 8;
        ac += kSets;
        while (ai < mine && ac >= stages) ac -= stages, ++ai;
      }
      copies_close();
      if (++put == kSlots) put = 0;
    };
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) copy_next();
    const long long all = static_cast<long long>(mine) * stages;
    int get = 0, s = set;
    uint32_t ph = 1;
    for (long long c = set; c < all; c += kSets) {
      __syncwarp();                            // the slot that the next copies fill has been read
      copy_next();
      copies_wait<kSlots - 1>();
      __syncwarp();
      const uint8_t* q = raw_ptr + get * kSlot;
      const uint2 scales = *reinterpret_cast<const uint2*>(q + 2048 + lane * 8);
      q += lane * 64;
      if (++get == kSlots) get = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int x = (lane >> 1) & 3;
        const uint4 w0 = *reinterpret_cast<const uint4*>(q + ((2 * h ^ x) << 4));
        const uint4 w1 = *reinterpret_cast<const uint4*>(q + (((2 * h + 1) ^ x) << 4));
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
        if (h == 0 && c >= kS && !__all_sync(0xFFFFFFFFu, wait_or_abort(empty + 8 * s, ph, a.err, abort_flag))) goto decoded;
        if (h == 0) tc_fence_after();
        tmem_st32(at + s * 64 + h * 32, r);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive_relaxed(full0 + 8 * s);
      s += kSets;
      if (s >= kS) s -= kS, ph ^= 1;
    }
  decoded:
    copies_wait<0>();
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    // Output: this warp's 32 lanes, all columns. First into registers as BF16, so
    // that the accumulator is free for the next tile; then, while that is
    // computed, 32 pairs at a time through shared memory to rows of C.
    const int q = warp & 3;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t acc_free0 = mapa_shared(acc_free, 0);
    uint8_t* const out = smem + kOutAt + q * kOut;
    const int align = out_align(a);
    uint32_t ph = 0;
    for (int i = 0; i < mine; ++i) {
      Tile tile;
      tile.at(table, first + i * step, weight_tiles);
      const float gs = a.globals ? a.globals[tile.expert] : 1.0f;
      wait_or_abort(acc_full, ph, a.err, abort_flag);
      ph ^= 1;
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
      tc_fence_after();
      uint32_t packed[kMaxN / 32][kGated ? 8 : 16], next[32];
      tmem_ld32_start(tl, next);
#pragma unroll
      for (int ch = 0; ch < kMaxN / 32; ++ch) {
        if (32 * ch >= tile.n) break;
        uint32_t v[32];
        tmem_ld_wait(next);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = next[j];
        if (kGated && ch + 1 < kMaxN / 32 && 32 * ch + 32 < tile.n) tmem_ld32_start(tl + 32 * ch + 32, next);
        if constexpr (kGated) {
          // Even lanes have gates and take columns 0..15, odd ones ups and 16..31.
          const bool odd = lane & 1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 2 * j + e;
              const float keep = __uint_as_float(odd ? v[16 + c] : v[c]), give = __uint_as_float(odd ? v[c] : v[16 + c]);
              const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
              y[e] = silu((odd ? got : keep) * gs) * ((odd ? keep : got) * gs);
            }
            packed[ch][j] = pack_bf16(y[0], y[1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) packed[ch][j] = pack_bf16(__uint_as_float(v[2 * j]) * gs, __uint_as_float(v[2 * j + 1]) * gs);
          if (ch + 1 < kMaxN / 32 && 32 * ch + 32 < tile.n) tmem_ld32_start(tl + 32 * ch + 32, next);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && i + 1 < mine) pair_arrive(acc_free0);

      // Outputs o0 .. of this warp: 32, or (gated) 16.
      const int o0 = kGated ? tile.nt * 128 + rank * 64 + q * 16 : tile.nt * 256 + rank * 128 + q * 32;
      const int left = outs - o0;
#pragma unroll
      for (int ch = 0; ch < kMaxN / 32; ++ch) {
        if (32 * ch >= tile.n) break;
        const int pl = 32 * ch + lane < tile.pairs ? a.rows[tile.p0 + 32 * ch + lane] : -1;   // the pair of column 32 ch + lane
        __syncwarp();
        if constexpr (kGated) {                // 32 pairs of 32 bytes, piece h of pair c at h ^ (c / 4 mod 2)
          const int n = lane >> 1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 2 * j + (lane & 1) * 16;
            *reinterpret_cast<uint16_t*>(out + c * 32 + (((n >> 3) ^ ((c >> 2) & 1)) << 4) + (n & 7) * 2) = static_cast<uint16_t>(packed[ch][j]);
            *reinterpret_cast<uint16_t*>(out + (c + 1) * 32 + (((n >> 3) ^ ((c >> 2) & 1)) << 4) + (n & 7) * 2) =
                static_cast<uint16_t>(packed[ch][j] >> 16);
          }
          __syncwarp();
          const int p = pl;
          if (static_cast<unsigned>(p) < static_cast<unsigned>(R)) {
            uint16_t* const c = static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc + o0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              store_piece(c + 8 * h, out + lane * 32 + ((h ^ ((lane >> 2) & 1)) << 4), left - 8 * h, align);
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
            const int c = 8 * k + (lane >> 2), h = lane & 3;
            const int p = __shfl_sync(0xFFFFFFFFu, pl, c);
            if (static_cast<unsigned>(p) < static_cast<unsigned>(R))
              store_piece(static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc + o0 + 8 * h,
                          out + c * 64 + ((h ^ ((c >> 1) & 3)) << 4), left - 8 * h, align);
          }
        }
      }
    }
  } else if (warp < kWarpMma + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  }
  if (warp == kWarpRelay) {
    // Announces the stages whose activations have landed. The fence that makes
    // them visible to the MMAs waits for all copies of the thread that makes it,
    // so a feeder would wait for those of later stages.
    const long long all = static_cast<long long>(mine) * stages;
    int s = 0;
    uint32_t ph = 0;
    for (long long c = 0; c < all; ++c) {
      if (!__all_sync(0xFFFFFFFFu, wait_or_abort(landed + 8 * s, ph, a.err, abort_flag))) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) pair_arrive(full0 + 8 * s);
      if (++s == kS) s = 0, ph ^= 1;
    }
  } else if (warp == kWarpMma && rank == 0) {
    // A wait that follows MMAs costs the tensor core a pause, so the next stage is
    // looked up before this one's MMAs are issued.
    const uint64_t bd0 = tile_desc(sb);
    int s = 0;
    uint32_t ph = 0, acc_ph = 0;
    bool ok = true, loaded = false;
    for (int i = 0; i < mine && ok; ++i) {
      Tile tile;
      tile.at(table, first + i * step, weight_tiles);
      const uint32_t idesc = idesc_bf16(256, tile.n);
      if (i > 0) {
        ok = __all_sync(0xFFFFFFFFu, wait_or_abort(acc_free, acc_ph, a.err, abort_flag));
        acc_ph ^= 1;
      }
      for (int k = 0; k < stages && ok; ++k) {
        if (!loaded) ok = __all_sync(0xFFFFFFFFu, wait_or_abort(full + 8 * s, ph, a.err, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int s1 = s + 1 == kS ? 0 : s + 1;
        const uint32_t ph1 = s1 ? ph : ph ^ 1;
        const bool l1 = mbar_test(full + 8 * s1, ph1);
        if (elect_one()) {
          const uint64_t bd = bd0 + s * (kStageB >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            pair_mma_ts(tmem, tmem + kColA + s * 64 + 8 * j, bd + (j >> 2) * (kHalfB >> 4) + 2 * (j & 3), idesc, (k | j) ? 1u : 0u);
          pair_commit(empty + 8 * s);
          if (k + 1 == stages) pair_commit(acc_full);
        }
        __syncwarp();
        loaded = __all_sync(0xFFFFFFFFu, l1);
        s = s1, ph = ph1;
      }
    }
    if (elect_one()) pair_commit_own(drained);
    __syncwarp();
    mbar_wait(drained, 0, a.err);
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

template <bool kGated>
cudaError_t launch_experts_many_t(const ExpertsArgs& a, cudaStream_t s) {
  static AttrLatch latch;
  const cudaError_t e = set_smem_attrs(experts_kernel<kGated>, latch, many_bytes(kMaxExperts), true);
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
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, experts_kernel<kGated>, a);
}

}  // namespace
}  // namespace act

cudaError_t launch_w4a16_experts_many(const ExpertsArgs& a, cudaStream_t s) {
  return a.gated ? act::launch_experts_many_t<true>(a, s) : act::launch_experts_many_t<false>(a, s);
}

}  // namespace wqp
