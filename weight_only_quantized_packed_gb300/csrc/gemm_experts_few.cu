// Products of rows with their experts' packed W4A16 matrices, few rows an
// expert: C[p] = A[p / slots] @ dequant(W[e])^T * g[e] for the pairs p of each
// expert e, or silu(gate) * up of the two halves of that.
//
// Bound by the experts' packed weights, which are read once for up to 8 pairs: a
// token's few rows share nothing across experts, so the bytes are those of the
// experts that were chosen.
//
//  * Work: a unit is 16 weight rows (plain: 16 outputs; gated: 8 gate rows and
//    the 8 up rows of the same outputs, so that a lane of the MMA has both) by
//    one tile of 8 pairs. Units are numbered through all experts, and each CTA
//    takes an equal run of them: of 2048 units on 304 CTAs none takes more than
//    7, where tiles of 64 rows would leave every sixth CTA idle.
//  * A CTA takes up to eight units of one tile at a time. Its eight warps split
//    K: a warp turns its part of the pairs' activations into MMA fragments once
//    for them all, and the warps' sums meet in shared memory.
//  * Weights arrive by 16-byte asynchronous copies, each lane's own into a
//    ring of its warp, which runs on through the ends of units: a warp waits
//    for its copies alone, and there is no barrier between CTAs or warps but
//    the two around the sums.
//  * Operands are FP16 (mma_f16.cuh): e2m1 * e4m3 is exact there, and the
//    activations of a step (256 K, or 128 at the end of a warp's part) are
//    scaled by a power of two per pair.
//
// 16x8 of 128, 5120x2048: 112 us, 4.3 TB/s of the experts' weights; 1x8, gated
// 4096x5120: 25.0 us (25.5 with the output rows and global scales loaded after the
// sums). The instructions around the MMAs set the pace, not the bytes: in steps of
// 128 K 120 us (191 instructions a unit and 128 K, 72 of them MMAs, conversions and
// products), with four units at a time 139 us; 24 warps of 80 registers instead of
// 16 148 us; sums in shared memory, so that the loop over the units need not be
// unrolled, 123 us; the next run's pairs loaded during this one 127 us.
#include "experts.cuh"
#include "mma_f16.cuh"
#include "decode.cuh"

namespace wqp {
namespace {

using namespace f16op;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kUnits = 8;                      // units at a time
constexpr int kPairs = 8;                      // of a tile
constexpr int kStage = 16 * 128 + 16 * 16;     // codes and scales of 16 rows x 256 K
constexpr int kStages = 3;                     // of a warp's ring
constexpr int kRow = 16 * kUnits + 4;          // floats of a pair's sums (+ 4: free of bank conflicts)

constexpr int few_bytes(int E) { return kWarps * kStages * kStage + kWarps * kPairs * kRow * 4 + experts::Table::bytes(E); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Units [first, last) of a CTA, in runs of at most kUnits within one tile.
struct Run {
  long long at, last;
  int per;                                     // units of a tile
  int expert, tile, unit, units;               // the run: tile within the expert, first unit, units
  __device__ __forceinline__ bool next(const experts::Table& table) {
    if (at >= last) return false;
    const int t = static_cast<int>(at / per);
    unit = static_cast<int>(at - static_cast<long long>(t) * per);
    units = static_cast<int>(min(static_cast<long long>(min(kUnits, per - unit)), last - at));
    expert = table.expert_of(t);
    tile = t - table.tiles[expert];
    at += units;
    return true;
  }
};

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(ExpertsArgs a) {
  extern __shared__ __align__(16) uint8_t few_sh[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  uint8_t* const ring = few_sh + warp * kStages * kStage;
  float* const sums = reinterpret_cast<float*>(few_sh + kWarps * kStages * kStage);
  pdl_launch_dependents();
  pdl_wait();
  const int R = a.T * a.slots;
  experts::Table table;
  table.make(few_sh + kWarps * kStages * kStage + kWarps * kPairs * kRow * 4, a.offsets, a.E, R,
             [](int n) { return (n + kPairs - 1) / kPairs; });

  const int outs = kGated ? a.N / 2 : a.N;     // outputs of a pair
  constexpr int kOuts = kGated ? 8 : 16;       // of a unit
  const int per = (outs + kOuts - 1) / kOuts;
  const long long units = static_cast<long long>(table.total()) * per;
  const long long first = units * blockIdx.x / gridDim.x, last = units * (blockIdx.x + 1) / gridDim.x;
  const int blocks = a.K >> 7;                 // of 128 K; this warp's: [b0, b1), two a step
  const int b0 = blocks * warp / kWarps, b1 = blocks * (warp + 1) / kWarps;

  // The copies run kStages - 1 stages ahead of their use, in the same order:
  // per run its steps, per step its units. A lane copies its own 16 bytes a
  // 128 K of rows g and g + 8 of a unit (gated: gate row g and up row
  // g), and lanes 0..15 the scales of rows 0..15; rows past the last read that one.
  const uint32_t wpitch = static_cast<uint32_t>(a.K) >> 1, spitch = static_cast<uint32_t>(a.K) >> 4;
  const long long half = kGated ? static_cast<long long>(outs) : 0;
  const int r_lo = g, r_hi = kGated ? g : g + 8, r_s = kGated ? lane & 7 : lane & 15;
  const uint32_t ring_at = smem_u32(ring) + lane * 16, ring_sc = smem_u32(ring) + 2048 + lane * 16;
  Run ahead = {first, last, per, 0, 0, 0, 0};
  const uint8_t *w_lo = nullptr, *w_hi = nullptr, *w_s = nullptr;   // of row 0 of the expert's halves, at block ab
  int ab = b1, au = 0, put = 0;
  bool more = b0 < b1;
  const auto copy_next = [&] {
    if (ab >= b1) {
      more = more && ahead.next(table);
      ab = b0;
      au = ahead.unit;
      if (more) {
        const long long row = static_cast<long long>(ahead.expert) * a.N;
        w_lo = a.W + row * wpitch + b0 * 64;
        w_hi = w_lo + half * wpitch;
        w_s = a.scales + (row + (kGated && lane >= 8 ? half : 0)) * spitch + b0 * 8;
      }
    }
    if (more) {
      const bool two = ab + 1 < b1;
      const int o = au * kOuts, top = outs - 1;
      const uint64_t lo = static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_lo, top))) * wpitch + 16 * t4;
      const uint64_t hi = static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_hi, top))) * wpitch + 16 * t4;
      copy16(ring_at + put, w_lo + lo);
      copy16(ring_at + put + 512, w_hi + hi);
      if (two) {
        copy16(ring_at + put + 1024, w_lo + lo + 64);
        copy16(ring_at + put + 1536, w_hi + hi + 64);
      }
      if (lane < 16) {
        const uint8_t* s = w_s + static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_s, top))) * spitch;
        copy8(ring_sc + put, s);
        if (two) copy8(ring_sc + put + 8, s + 8);
      }
      if (++au == ahead.unit + ahead.units) {
        au = ahead.unit;
        ab += 2;
        w_lo += 128;
        w_hi += 128;
        w_s += 16;
      }
    }
    copies_close();
    put = put == (kStages - 1) * kStage ? 0 : put + kStage;
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_next();

  int get = 0;
  Run run = {first, last, per, 0, 0, 0, 0};
  while (run.next(table)) {
    const int p0 = table.begin[run.expert] + run.tile * kPairs;
    const int pairs = min(table.begin[run.expert + 1] - p0, kPairs);
    const auto pair_at = [&](int i) {          // pair i of the tile, or -1
      const int p = i < pairs ? a.rows[p0 + i] : -1;
      return static_cast<unsigned>(p) < static_cast<unsigned>(R) ? p : -1;
    };
    // Without a pair: any row, the sums go nowhere.
    const uint16_t* act = static_cast<const uint16_t*>(a.A) + static_cast<long long>(max(pair_at(g), 0) / a.slots) * a.lda + b0 * 128;
    const int p = pair_at(warp);               // the sums' part: a warp to a pair
    const float gs = a.globals ? a.globals[run.expert] : 1.0f;
    float tot[kUnits][4];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[u][i] = 0.0f;

#pragma unroll 1
    for (int b = b0; b < b1; b += 2, act += 256) {
      // Lane t of a pair has activations 32 t .. 32 t + 31 of each 128 K, as it has
      // the weights' codes.
      const bool two = b + 1 < b1;
      uint32_t bf[32];
      float inv0, inv1;
      {
        const uint16_t* src = act + 32 * t4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * q);
          bf[4 * q] = v.x, bf[4 * q + 1] = v.y, bf[4 * q + 2] = v.z, bf[4 * q + 3] = v.w;
        }
        if (two) {
#pragma unroll
          for (int q = 4; q < 8; ++q) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 96 + 8 * q);
            bf[4 * q] = v.x, bf[4 * q + 1] = v.y, bf[4 * q + 2] = v.z, bf[4 * q + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int q = 16; q < 32; ++q) bf[q] = 0;
        }
        // BF16 magnitudes order like their bits.
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = __vmaxu2(mx, bf[i] & 0x7FFF7FFFu);
        mx = max(mx & 0xFFFFu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const int sh = f16_shift(mx);
        const float scale = pow2(sh), own = pow2(-sh);
#pragma unroll
        for (int i = 0; i < 32; ++i) bf[i] = f32x2_to_f16x2(bf16hi(bf[i]) * scale, bf16lo(bf[i]) * scale);
        inv0 = __shfl_sync(0xFFFFFFFFu, own, 8 * t4);
        inv1 = __shfl_sync(0xFFFFFFFFu, own, 8 * t4 + 4);
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (u < run.units) {
          __syncwarp();                        // the slot that the next copies fill has been read
          copy_next();
          copies_wait<kStages - 1>();
          __syncwarp();
          const uint8_t* st = ring + get;
          get = get == (kStages - 1) * kStage ? 0 : get + kStage;
          // Of a lane's 32 codes a row and 128 K, the first two words are one group of
          // 16, the others the next.
          const uint8_t* sc = st + 2048 + g * 16 + 2 * t4;
          float d[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !two) break;
            const uint4 lo = lds128(st + 1024 * h + lane * 16), hi = lds128(st + 1024 * h + 512 + lane * 16);
            const uint32_t slo = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc + 8 * h));
            const uint32_t shi = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc + 8 * h + 128));
            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t sl = __byte_perm(slo, slo, q < 2 ? 0x1010 : 0x3232), sh = __byte_perm(shi, shi, q < 2 ? 0x1010 : 0x3232);
              const uint32_t a00 = mul_f16x2(e2m1x2_byte<0>(wl[q]), sl), a01 = mul_f16x2(e2m1x2_byte<0>(wh[q]), sh);
              const uint32_t a02 = mul_f16x2(e2m1x2_byte<1>(wl[q]), sl), a03 = mul_f16x2(e2m1x2_byte<1>(wh[q]), sh);
              const uint32_t a10 = mul_f16x2(e2m1x2_byte<2>(wl[q]), sl), a11 = mul_f16x2(e2m1x2_byte<2>(wh[q]), sh);
              const uint32_t a12 = mul_f16x2(e2m1x2_byte<3>(wl[q]), sl), a13 = mul_f16x2(e2m1x2_byte<3>(wh[q]), sh);
              if (q == 0) mma_f16_16816_z(d[h], a00, a01, a02, a03, bf[16 * h], bf[16 * h + 1]);
              else mma_f16_16816(d[h], a00, a01, a02, a03, bf[16 * h + 4 * q], bf[16 * h + 4 * q + 1]);
              mma_f16_16816(d[h], a10, a11, a12, a13, bf[16 * h + 4 * q + 2], bf[16 * h + 4 * q + 3]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[u][i] += (i & 1 ? inv1 : inv0) * (two ? d[0][i] + d[1][i] : d[0][i]);
        }
      }
    }

    // The warps' sums, in the warps' order. The first barrier: the sums before
    // have been read.
    __syncthreads();
    float* const mine = sums + warp * kPairs * kRow;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(2 * t4 + (i & 1)) * kRow + 16 * u + g + 8 * (i >> 1)] = tot[u][i];
    __syncthreads();
    if (p < 0) continue;
    uint16_t* const c = static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc;
    const float* s = sums + warp * kRow;
    const auto sum_at = [&](int r) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s[w * kPairs * kRow + r];
      return v * gs;
    };
    if (kGated) {
#pragma unroll
      for (int h = 0; h < kUnits / 4; ++h) {
        const int i8 = 32 * h + lane, o = run.unit * 8 + i8;
        if (i8 < run.units * 8 && o < outs) {
          const int r = (i8 >> 3) * 16 + (i8 & 7);
          const float gate = sum_at(r), up = sum_at(r + 8);
          c[o] = f32_to_bf16_rn(experts::silu(gate) * up);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < kUnits / 2; ++h) {
        const int r = 32 * h + lane, o = run.unit * 16 + r;
        if (r < run.units * 16 && o < outs) c[o] = f32_to_bf16_rn(sum_at(r));
      }
    }
  }
  copies_wait<0>();
}

template <bool kGated>
cudaError_t launch_few_t(const ExpertsArgs& a, cudaStream_t s) {
  static AttrLatch latch;
  const cudaError_t e = set_smem_attrs(few_kernel<kGated>, latch, few_bytes(kMaxExperts), false);
  if (e != cudaSuccess) return e;
  return launch(few_kernel<kGated>, dim3(2 * a.num_sms), dim3(kThreads), few_bytes(a.E), s, a.pdl, a);
}

// Whether the kernel above is taken, from the sizes alone: pairs without an expert
// count as well. Mostly it is the faster one then; small products of more pairs it
// would have sooner too (the other's two launches). The other takes some 8 us for its two
// launches and has the weights' bytes through in the same time for any number of
// rows; this one takes longer per expert the longer its rows are, and again for
// every 8 pairs. Measured, this | the other, us: 128 experts of 4096x5120 (gated),
// pairs an expert 1/16: 30.1 | 34.0, 1/4: 88.9 | 81.8, 1: 237 | 212; 128 of
// 5120x2048, 1: 115 | 127, 4: 183 | 196, 6: 212 | 199; 8 of 4096x4096, 1/4: 11.2 |
// 17.0, 4: 23.5 | 29.0, 8: 32.4 | 29.1; 32 of 2048x1024, 1/4: 6.5 | 9.4, 3: 20.7 |
// 22.6, 4: 25.3 | 22.7.
bool experts_few(int T, int slots, int E, int N, int K) {
  const long long pairs = static_cast<long long>(T) * slots, used = pairs < E ? pairs : E;
  return pairs <= 4ll * E && (K <= 2048 || used * N * K <= 1ll << 28);
}

}  // namespace

size_t experts_workspace(int T, int slots, int E, int N, int K) {
  return experts_few(T, slots, E, N, K) ? 0 : static_cast<size_t>(T) * slots * (static_cast<size_t>(K) * 2 + 4);
}

cudaError_t launch_w4a16_experts(const ExpertsArgs& a, cudaStream_t s) {
  if (!experts_few(a.T, a.slots, a.E, a.N, a.K)) return launch_w4a16_experts_many(a, s);
  return a.gated ? launch_few_t<true>(a, s) : launch_few_t<false>(a, s);
}

}  // namespace wqp
