// Products of rows with their experts' packed W4A16 matrices, few rows an
// expert: C[p] = A[p / slots] @ dequant(W[e])^T * g[e] for the pairs p of each
// expert e, or silu(gate) * up of the two halves of that.
//
// Bound by the experts' packed weights, which are read once for up to
// 8 * kTiles pairs: a token's few rows share nothing across experts, so the
// bytes are those of the experts that were chosen.
//
//  * Work: a unit is 16 weight rows (plain: 16 outputs; gated: 8 gate rows and
//    the 8 up rows of the same outputs, so that a lane of the MMA has both) by
//    one tile of pairs. Units are numbered through all experts, and each CTA
//    takes an equal run of them: of 2048 units on 304 CTAs none takes more than
//    7, where tiles of 64 rows would leave every sixth CTA idle.
//  * A CTA takes up to eight units of one tile at a time. Its eight warps split
//    K: a warp turns its part of the pairs' activations into MMA fragments once
//    for them all, and the warps' sums meet in shared memory.
//  * Weights arrive by 16-byte asynchronous copies, each lane's own into a
//    ring of its warp, which runs on through the ends of units: a warp waits
//    for its copies alone, and there is no barrier between CTAs or warps but
//    the two around the sums.
//  * Operands are FP16 (mma_f16.cuh): e2m1 * e4m3 is exact there, and each
//    (pair, 128 K) block of activations is scaled by a power of two.
#include "experts.cuh"
#include "mma_f16.cuh"
#include "decode.cuh"

namespace wqp {
namespace {

using namespace f16op;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kUnits = 8;                      // units at a time
constexpr int kStage = 16 * 64 + 16 * 8;       // codes and scales of 16 rows x 128 K
constexpr int kStages = 7;                     // of a warp's ring
constexpr int kRow = 16 * kUnits + 4;          // floats of a pair's sums (+ 4: free of bank conflicts)

template <int kTiles>
constexpr int few_bytes(int E) {
  return kWarps * kStages * kStage + kWarps * 8 * kTiles * kRow * 4 + experts::Table::bytes(E);
}

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

template <int kTiles, bool kGated>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(ExpertsArgs a) {
  extern __shared__ __align__(16) uint8_t few_sh[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  uint8_t* const ring = few_sh + warp * kStages * kStage;
  float* const sums = reinterpret_cast<float*>(few_sh + kWarps * kStages * kStage);
  pdl_launch_dependents();
  pdl_wait();
  const int R = a.T * a.slots;
  experts::Table table;
  table.make(few_sh + kWarps * kStages * kStage + kWarps * 8 * kTiles * kRow * 4, a.offsets, a.E, R,
             [](int n) { return (n + 8 * kTiles - 1) / (8 * kTiles); });

  const int outs = kGated ? a.N / 2 : a.N;     // outputs of a pair
  constexpr int kOuts = kGated ? 8 : 16;       // of a unit
  const int per = (outs + kOuts - 1) / kOuts;
  const long long units = static_cast<long long>(table.total()) * per;
  const long long first = units * blockIdx.x / gridDim.x, last = units * (blockIdx.x + 1) / gridDim.x;
  const int blocks = a.K >> 7;                 // of 128 K; this warp's: [b0, b1)
  const int b0 = blocks * warp / kWarps, b1 = blocks * (warp + 1) / kWarps;

  // The copies run kStages - 1 stages ahead of their use, in the same order:
  // per run its blocks, per block its units. A lane copies its own 16 bytes of
  // rows g and g + 8 of a unit (gated: gate row g and up row g), and lanes 0..15
  // the scales of rows 0..15; rows past the last read that one.
  const uint32_t wpitch = static_cast<uint32_t>(a.K) >> 1, spitch = static_cast<uint32_t>(a.K) >> 4;
  const long long half = kGated ? static_cast<long long>(outs) : 0;
  const int r_lo = g, r_hi = kGated ? g : g + 8, r_s = kGated ? lane & 7 : lane & 15;
  const uint32_t ring_at = smem_u32(ring) + lane * 16, ring_sc = smem_u32(ring) + 1024 + lane * 8;
  Run ahead = {first, last, per, 0, 0, 0, 0};
  const uint8_t *w_lo = nullptr, *w_hi = nullptr, *w_s = nullptr;   // of row 0 of the expert's halves, at block ab
  int ab = b1, au = 0, put = 0;
  bool more = b0 < b1;
  const auto copy_next = [&] {
    if (ab == b1) {
      more = more && ahead.next(table);
      ab = b0;
      au = ahead.unit;
      if (more) {
        const long long row = static_cast<long long>(ahead.expert) * a.N;
        w_lo = a.W + row * wpitch + b0 * 64 + t4 * 16;
        w_hi = w_lo + half * wpitch;
        w_s = a.scales + (row + (kGated && lane >= 8 ? half : 0)) * spitch + b0 * 8;
      }
    }
    if (more) {
      const int o = au * kOuts, top = outs - 1;
      copy16(ring_at + put, w_lo + static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_lo, top))) * wpitch);
      copy16(ring_at + put + 512, w_hi + static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_hi, top))) * wpitch);
      if (lane < 16) copy8(ring_sc + put, w_s + static_cast<uint64_t>(static_cast<uint32_t>(min(o + r_s, top))) * spitch);
      if (++au == ahead.unit + ahead.units) {
        au = ahead.unit;
        ++ab;
        w_lo += 64;
        w_hi += 64;
        w_s += 8;
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
    const int p0 = table.begin[run.expert] + run.tile * 8 * kTiles;
    const int pairs = min(table.begin[run.expert + 1] - p0, 8 * kTiles);
    const auto pair_at = [&](int i) {          // pair i of the tile, or -1
      const int p = i < pairs ? a.rows[p0 + i] : -1;
      return static_cast<unsigned>(p) < static_cast<unsigned>(R) ? p : -1;
    };
    const uint16_t* act[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int p = pair_at(8 * n + g);        // without a pair: any row, the sums go nowhere
      act[n] = static_cast<const uint16_t*>(a.A) + static_cast<long long>(max(p, 0) / a.slots) * a.lda + b0 * 128 + 32 * t4;
    }
    float tot[kUnits][kTiles][4];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[u][n][i] = 0.0f;

#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      uint32_t bf[kTiles][16];
      float inv[kTiles][2];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        uint32_t r[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v = *reinterpret_cast<const uint4*>(act[n] + 8 * q);
          r[4 * q] = v.x, r[4 * q + 1] = v.y, r[4 * q + 2] = v.z, r[4 * q + 3] = v.w;
        }
        act[n] += 128;
        float own;
        build_bfrag_regs(r, bf[n], own);
        inv[n][0] = __shfl_sync(0xFFFFFFFFu, own, 8 * t4);
        inv[n][1] = __shfl_sync(0xFFFFFFFFu, own, 8 * t4 + 4);
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
          const uint4 lo = lds128(st + lane * 16), hi = lds128(st + 512 + lane * 16);
          const uint32_t slo = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(st + 1024 + g * 8 + 2 * t4));
          const uint32_t shi = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(st + 1024 + (g + 8) * 8 + 2 * t4));
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
          float d[kTiles][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // Words 0 and 1 are the first 16 K of the lane, 2 and 3 the second.
            const uint32_t sl = __byte_perm(slo, slo, q < 2 ? 0x1010 : 0x3232), sh = __byte_perm(shi, shi, q < 2 ? 0x1010 : 0x3232);
            const uint32_t a00 = mul_f16x2(e2m1x2_byte<0>(wl[q]), sl), a01 = mul_f16x2(e2m1x2_byte<0>(wh[q]), sh);
            const uint32_t a02 = mul_f16x2(e2m1x2_byte<1>(wl[q]), sl), a03 = mul_f16x2(e2m1x2_byte<1>(wh[q]), sh);
            const uint32_t a10 = mul_f16x2(e2m1x2_byte<2>(wl[q]), sl), a11 = mul_f16x2(e2m1x2_byte<2>(wh[q]), sh);
            const uint32_t a12 = mul_f16x2(e2m1x2_byte<3>(wl[q]), sl), a13 = mul_f16x2(e2m1x2_byte<3>(wh[q]), sh);
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
              if (q == 0) mma_f16_16816_z(d[n], a00, a01, a02, a03, bf[n][0], bf[n][1]);
              else mma_f16_16816(d[n], a00, a01, a02, a03, bf[n][4 * q], bf[n][4 * q + 1]);
              mma_f16_16816(d[n], a10, a11, a12, a13, bf[n][4 * q + 2], bf[n][4 * q + 3]);
            }
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[u][n][i] += inv[n][i & 1] * d[n][i];
        }
      }
    }

    // The warps' sums, in the warps' order. The first barrier: the sums before
    // have been read.
    __syncthreads();
    float* const mine = sums + warp * 8 * kTiles * kRow;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(8 * n + 2 * t4 + (i & 1)) * kRow + 16 * u + g + 8 * (i >> 1)] = tot[u][n][i];
    __syncthreads();
    const float gs = a.globals ? a.globals[run.expert] : 1.0f;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int i = 8 * n + warp, p = pair_at(i);
      if (p < 0) continue;
      uint16_t* const c = static_cast<uint16_t*>(a.C) + static_cast<long long>(p) * a.ldc;
      const float* s = sums + i * kRow;
      const auto sum_at = [&](int r) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s[w * 8 * kTiles * kRow + r];
        return v * gs;
      };
      if (kGated) {
#pragma unroll
        for (int h = 0; h < kUnits / 4; ++h) {
          const int i8 = 32 * h + lane, o = run.unit * 8 + i8;
          if (i8 < run.units * 8 && o < outs) {
            const int r = (i8 >> 3) * 16 + (i8 & 7);
            const float gate = sum_at(r), up = sum_at(r + 8);
            c[o] = f32_to_bf16_rn(gate / (1.0f + expf(-gate)) * up);
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
  }
  copies_wait<0>();
}

template <int kTiles, bool kGated>
cudaError_t launch_few_t(const ExpertsArgs& a, cudaStream_t s) {
  static AttrLatch latch;
  const cudaError_t e = set_smem_attrs(few_kernel<kTiles, kGated>, latch, few_bytes<kTiles>(kMaxExperts), false);
  if (e != cudaSuccess) return e;
  return launch(few_kernel<kTiles, kGated>, dim3(2 * a.num_sms), dim3(kThreads), few_bytes<kTiles>(a.E), s, a.pdl, a);
}

}  // namespace

#ifndef RF
#define RF 4
#endif
size_t experts_workspace(int T, int slots, int E, int K) {
  const long long pairs = static_cast<long long>(T) * slots;
  return pairs > RF * E ? static_cast<size_t>(pairs) * (static_cast<size_t>(K) * 2 + 4) : 0;
}

cudaError_t launch_w4a16_experts(const ExpertsArgs& a, cudaStream_t s) {
  const long long pairs = static_cast<long long>(a.T) * a.slots;
  if (pairs > RF * a.E) return launch_w4a16_experts_many(a, s);
  return a.gated ? launch_few_t<1, true>(a, s) : launch_few_t<1, false>(a, s);
}

}  // namespace wqp
