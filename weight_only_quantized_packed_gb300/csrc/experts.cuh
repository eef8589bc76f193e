// What the kernels of the experts' products share: silu, and the table of tiles
// that each CTA makes from the experts' offsets.
#pragma once
#include "common.cuh"

namespace wqp {
namespace experts {

// g * sigmoid(g), through e^-|g|, which cannot overflow. expf is 2 ulp off at any
// argument, where __expf's error grows with it (25 ulp at 20); it costs 1 % at
// 4096x8, gated 4096x5120 (955 -> 965 us). The quotient is 2 ulp off: an IEEE
// division took 1060 us there.
__device__ __forceinline__ float silu(float g) {
  const float t = expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * t : g, 1.0f + t);
}

// Per expert its first position and, summed up, how many tiles of pairs it and
// the experts before it have. Offsets are taken as expert_order writes them;
// whatever else they hold, no position outside 0..R is used.
struct Table {
  int* begin;           // [E + 1]
  int* tiles;           // [E + 1], tiles[0] = 0
  int E;

  __host__ __device__ static constexpr int bytes(int E) { return 2 * (E + 1) * static_cast<int>(sizeof(int)); }

  // By all threads of a block (a multiple of 32 that is at least 32); tile_of(count)
  // gives an expert's tiles. Ends with the block's barrier.
  template <class TileOf>
  __device__ __forceinline__ void make(uint8_t* smem, const int* offsets, int experts, int R, const TileOf& tile_of) {
    E = experts;
    begin = reinterpret_cast<int*>(smem);
    tiles = begin + E + 1;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) begin[e] = min(max(offsets[e], 0), R);
    __syncthreads();
    if (threadIdx.x < 32) {                                // one warp: at most 1024 experts
      const int lane = threadIdx.x;
      int at = begin[0], sum = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int end = max(e < E ? begin[e + 1] : 0, at);       // positions do not go back
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, end, o);
          if (lane >= o) end = max(end, u);
        }
        const int before = __shfl_up_sync(0xFFFFFFFFu, end, 1);
        int v = e < E ? tile_of(end - (lane ? before : at)) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += u;
        }
        if (e < E) {
          begin[e + 1] = end;
          tiles[e + 1] = sum + v;
        }
        sum += __shfl_sync(0xFFFFFFFFu, v, 31);
        at = __shfl_sync(0xFFFFFFFFu, end, 31);
      }
      if (lane == 0) tiles[0] = 0;
    }
    __syncthreads();
  }
  __device__ __forceinline__ int total() const { return tiles[E]; }
  // The expert of a tile below total().
  __device__ __forceinline__ int expert_of(int tile) const {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tiles[mid + 1] > tile) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  }
};

}  // namespace experts
}  // namespace wqp
