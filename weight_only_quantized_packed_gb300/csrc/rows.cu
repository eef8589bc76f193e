// Row kernels of the quantised-activation path: 4-bit and 8-bit quantisation
// and the root-mean-square norm with the residual's addition.
//
// All three are bound by memory: each element is read once and written once,
// and the arithmetic between (a maximum, a quotient, a conversion) has to fit
// under the time of its bytes.
//
// w4_quantize, per group of 16 (amax = largest magnitude, g = global scale):
//   s = e4m3(amax / (6 g)), d = s * g, code = e2m1(x / d), or 0 where d is 0
// a8_quantize, per group of 128 (amax floored at 2^-100):
//   s = amax / 448, code = e4m3(x * (448 / amax))
// rms_norm: h = x + r, y = (h * rsqrt(mean h^2 + eps)) * w, in FP32 from the
// unrounded sum; y is rounded once, to its own type or by a8_quantize's rule.
// A lane always holds 8 consecutive elements, so a group of 16 is a lane pair
// and a group of 128 is half a warp; the maxima keep NaNs.
#include <cuda_fp16.h>

#include "decode.cuh"
#include "tc.cuh"

namespace wqp {
namespace {

constexpr float kA8Floor = 0x1p-100f;

// 8 consecutive elements as FP32.
template <class T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
};
template <>
struct Vec8<__half> {
  uint4 r;
  __device__ __forceinline__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f16x2_to_float2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Largest magnitude; NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float absmax(const float (&v)[8]) {
  return max3_abs(max3_abs(v[0], v[1], v[2]), max3_abs(v[3], v[4], v[5]), max3_abs(v[6], v[7], v[7]));
}
__device__ __forceinline__ bool finite(float amax) { return amax < __uint_as_float(0x7F800000u); }

// Two products, and two sums of products, in one instruction each.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(x)) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }

// Two FP32 -> two E4M3 (first in the low byte), and two E2M1 (first in the
// low nibble); both round to nearest even and saturate.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

// This lane's 8 elements of a 16-group (the neighbour lane holds the others):
// their codes, and the group's scale code in both lanes.
__device__ __forceinline__ uint32_t quantise4(const float (&v)[8], float g, float six_g, uint32_t& scale) {
  float m = absmax(v);
  m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const float t = m / six_g;
  const uint32_t s = f32x2_to_e4m3x2(t, 0.0f) & 0xFFu;
  const float d = e4m3_to_f32(s) * g;
  const bool fin = finite(m);
  const float inv = (d > 0.0f && fin) ? 1.0f / d : 0.0f;
  // x / d, correctly rounded, from the correctly rounded reciprocal by one
  // residual step (P. Markstein, "Computation of elementary functions on the
  // IBM RISC System/6000 processor", 1990): a quotient that falls on the
  // middle between two codes has to be recognised as such, which x * inv
  // alone misses for 3 of the 8 scale mantissas. A quotient may overflow where
  // the scale saturates by far; elements beyond 8 d, which end at +-6, are
  // brought to 8 d there.
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v[i];
  const bool far = t > 0x1p100f;
  if (__any_sync(0xFFFFFFFFu, far)) {
    const float lim = far ? 8.0f * d : __uint_as_float(0x7F7FFFFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -lim), lim);
  }
  float q[8];
  const uint64_t inv2 = pack2(inv, inv), nd2 = pack2(-d, -d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x2 = pack2(x[2 * i], x[2 * i + 1]);
    uint64_t q2 = mul2(x2, inv2);
    q2 = fma2(fma2(q2, nd2, x2), inv2, q2);
    q[2 * i] = lo2(q2);
    q[2 * i + 1] = hi2(q2);
  }
  scale = fin ? s : 0x7Fu;
  return inv > 0.0f ? f32x8_to_e2m1(q) : 0u;     // not the sign of x where d is 0
}

// This lane's 8 elements of a 128-group (16 lanes): their codes, and the
// group's scale in all lanes. A group with a NaN or an infinity gets a NaN
// scale. The floor keeps 448 / amax finite.
__device__ __forceinline__ uint2 quantise8(const float (&v)[8], float& scale) {
  float m = absmax(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float amax = finite(m) ? fmaxf(m, kA8Floor) : __uint_as_float(0x7FFFFFFFu);
  scale = amax / 448.0f;
  const float inv = 448.0f / amax;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ------------------------------------------------------------ quantisation
// One block = kThreads * U chunks of 8 elements. Contiguous rows are one long
// row; rows with a pitch find theirs by one division per thread and, from
// there, a multiplication by the reciprocal of the row's chunks: `recip` =
// ceil(2^40 / cpr), exact for numerators below 2^18 + 2^11 and cpr <= 2^17.
// Codes and scales are contiguous either way.
constexpr int kThreads = 256;

template <class T, bool kA8, bool kPitched, int U>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const T* X, uint8_t* codes, void* scales, float g,
                                                            float six_g, long long chunks, int cpr, int ldx,
                                                            unsigned long long recip) {
  pdl_launch_dependents();
  pdl_wait();
  const long long b0 = static_cast<long long>(blockIdx.x) * (kThreads * U), c0 = b0 + threadIdx.x;
  const long long row0 = kPitched ? b0 / cpr : 0;
  const unsigned col0 = kPitched ? static_cast<unsigned>(b0 - row0 * cpr) + threadIdx.x : 0;
  Vec8<T> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * kThreads;
    x[u] = Vec8<T>{};
    if (c < chunks) {
      long long at = c * 8;
      if (kPitched) {
        const unsigned n = col0 + u * kThreads;
        const unsigned r = static_cast<unsigned>((n * recip) >> 40);
        at = (row0 + r) * ldx + static_cast<long long>(n - r * cpr) * 8;
      }
      x[u].load(X + at);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * kThreads;
    float v[8];
    x[u].get(v);
    if (kA8) {
      float s;
      const uint2 q = quantise8(v, s);
      if (c < chunks) {
        *reinterpret_cast<uint2*>(codes + c * 8) = q;
        if ((threadIdx.x & 15) == 0) static_cast<float*>(scales)[c >> 4] = s;
      }
    } else {
      uint32_t s;
      const uint32_t q = quantise4(v, g, six_g, s);
      if (c < chunks) {
        *reinterpret_cast<uint32_t*>(codes + c * 4) = q;
        if ((threadIdx.x & 1) == 0) static_cast<uint8_t*>(scales)[c >> 1] = static_cast<uint8_t>(s);
      }
    }
  }
}

template <class T, bool kA8>
cudaError_t launch_quantise_t(const QuantArgs& a, cudaStream_t s) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  const int cpr = a.K / 8;
  const long long chunks = static_cast<long long>(a.M) * cpr;
  const long long blocks = (chunks + kThreads * U - 1) / (kThreads * U);
  const float six_g = 6.0f * a.gscale;
  const dim3 grid(static_cast<unsigned>(blocks));
  const unsigned long long recip = ((1ull << 40) + cpr - 1) / cpr;
  if (a.ldx == a.K || a.M == 1)
    return launch(quantise_kernel<T, kA8, false, U>, grid, dim3(kThreads), 0, s, a.pdl, static_cast<const T*>(a.X),
                  a.codes, a.scales, a.gscale, six_g, chunks, cpr, a.ldx, recip);
  return launch(quantise_kernel<T, kA8, true, U>, grid, dim3(kThreads), 0, s, a.pdl, static_cast<const T*>(a.X),
                a.codes, a.scales, a.gscale, six_g, chunks, cpr, a.ldx, recip);
}

// ------------------------------------------------------------ norm
struct NormParams {
  const void* X;
  const void* R;
  const void* W;
  void* H;
  void* Y;
  float* S;
  float eps;
  int M, K;
  int ldx, ldr, ldh, ldy;
};

// Sum over the threads of a row: half a warp (kHalf), or `warps` whole warps
// that share a slice of `part`. Every row of a block takes part.
template <bool kHalf>
__device__ __forceinline__ float row_sum(float v, float* part, int warps, int w) {
  if (kHalf) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
  v = warp_sum(v);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[w] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = threadIdx.x & 31; i < warps; i += 32) t += part[i];
  return warp_sum(t);
}

// blockDim = (threads per row, rows per block). V > 0: a thread holds its V
// chunks of the row (chunk i of thread t is t + i * threads) in registers
// between the sum and the output, so the row is read once; V == 0 (rows too
// long for that) reads it again. kHalf: rows of one group, 16 threads each.
template <class T, bool kA8, int V, bool kHalf>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p) {
  __shared__ float part[32];
  pdl_launch_dependents();
  const int tpr = blockDim.x, warps = tpr >> 5;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.M;
  const int chunks = p.K >> 3;
  const T* x = static_cast<const T*>(p.X) + static_cast<long long>(row) * p.ldx;
  const T* r = p.R ? static_cast<const T*>(p.R) + static_cast<long long>(row) * p.ldr : nullptr;
  T* h = p.H ? static_cast<T*>(p.H) + static_cast<long long>(row) * p.ldh : nullptr;
  const T* w = static_cast<const T*>(p.W);

  auto sum_of = [&](int c, float (&v)[8]) {
    Vec8<T> a;
    a.load(x + 8 * c);
    a.get(v);
    if (r) {
      Vec8<T> b;
      float u[8];
      b.load(r + 8 * c);
      b.get(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
  };
  // Every lane of a warp comes here for the same chunk row (quantise8
  // shuffles); `in` marks the lanes that have one.
  auto out_of = [&](int c, bool in, const float (&v)[8], Vec8<T> wv, bool have, float rstd) {
    float y[8] = {};
    if (in) {
      if (h) store8(h + 8 * c, v);
      if (!have) wv.load(w + 8 * c);
      wv.get(y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (v[i] * rstd) * y[i];
    }
    if constexpr (kA8) {
      float s;
      const uint2 q = quantise8(y, s);
      if (in) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Y) + static_cast<long long>(row) * p.K + 8 * c) = q;
        if ((threadIdx.x & 15) == 0) p.S[static_cast<long long>(row) * (p.K >> 7) + (c >> 4)] = s;
      }
    } else if (in) {
      store8(static_cast<T*>(p.Y) + static_cast<long long>(row) * p.ldy + 8 * c, y);
    }
  };

  pdl_wait();
  if constexpr (V > 0) {
    float v[V][8];
    // One chunk a thread (few rows): the weights are on their way during the
    // sum. With more, their registers cost more rows in flight than it gains.
    constexpr bool kEarly = V == 1;
    Vec8<T> wv[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * tpr;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
      wv[i] = Vec8<T>{};
      if (live && c < chunks) {
        sum_of(c, v[i]);
        if (kEarly) wv[i].load(w + 8 * c);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    }
    ss = row_sum<kHalf>(ss, part + threadIdx.y * warps, warps, threadIdx.x >> 5);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * tpr;
      out_of(c, live && c < chunks, v[i], wv[i], kEarly, rstd);
    }
  } else {
    float ss = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += tpr) {
      float v[8];
      sum_of(c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
    }
    ss = row_sum<false>(ss, part, warps, threadIdx.x >> 5);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.K) + p.eps);
    for (int c0 = 0; c0 < chunks; c0 += tpr) {
      const int c = c0 + threadIdx.x;
      float v[8] = {};
      if (c < chunks) sum_of(c, v);
      out_of(c, c < chunks, v, Vec8<T>{}, false, rstd);
    }
  }
}

// Many rows: a block takes rows blockIdx.x, + gridDim.x, ..., and the copies
// of its next rows (bulk copies into a ring of `stages` rows of X and R) run
// while it sums and writes the current one, so that loads are always in
// flight; the weights are copied once. One barrier a row: after it every
// thread has the row in registers, its slot is refilled, and the partial sums
// (two sets, by the row's parity) are complete.
constexpr int kMaxStages = 4;

template <class T, bool kA8, int V>
__global__ void __launch_bounds__(1024) norm_stream_kernel(NormParams p, int stages, unsigned* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_sh[kMaxStages + 1];
  __shared__ float part[2][32];
  __shared__ int abort_sh;
  volatile int* abort_flag = &abort_sh;
  const int chunks = p.K >> 3, row_bytes = p.K * static_cast<int>(sizeof(T));
  const int slot_bytes = p.R ? 2 * row_bytes : row_bytes;
  const uint32_t full = smem_u32(full_sh), base = smem_u32(smem);
  const int n = (p.M - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  int issued = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i <= stages; ++i) mbar_init(full + 8 * i, 1);
    abort_sh = 0;
    mbar_fence_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const auto issue = [&](int i) {
    const int s = i % stages;
    const long long row = blockIdx.x + static_cast<long long>(i) * gridDim.x;
    const uint32_t dst = base + row_bytes + s * slot_bytes;
    mbar_arrive_expect_tx(full + 8 * s, slot_bytes);
    bulk_g2s(dst, static_cast<const T*>(p.X) + row * p.ldx, row_bytes, full + 8 * s);
    if (p.R) bulk_g2s(dst + row_bytes, static_cast<const T*>(p.R) + row * p.ldr, row_bytes, full + 8 * s);
    issued = i + 1;
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < min(stages, n); ++i) issue(i);
    mbar_arrive_expect_tx(full + 8 * stages, row_bytes);
    bulk_g2s(base, p.W, row_bytes, full + 8 * stages);
  }
  const T* w = reinterpret_cast<const T*>(smem);
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = 0; i < n; ++i) {
    const int s = i % stages;
    const T* x = reinterpret_cast<const T*>(smem + row_bytes + s * slot_bytes);
    const T* r = x + p.K;
    tc::wait_or_abort(full + 8 * s, (i / stages) & 1, err, abort_flag);
    float v[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
      if (c < chunks) {
        Vec8<T> a;
        a.load(x + 8 * c);
        a.get(v[k]);
        if (p.R) {
          float u[8];
          a.load(r + 8 * c);
          a.get(u);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] += u[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) part[i & 1][warp] = ss;
    __syncthreads();
    if (threadIdx.x == 0 && i + stages < n && !*abort_flag) issue(i + stages);
    const float t = warp_sum(lane < warps ? part[i & 1][lane] : 0.0f);
    const float rstd = __frsqrt_rn(t / static_cast<float>(p.K) + p.eps);
    if (i == 0) tc::wait_or_abort(full + 8 * stages, 0, err, abort_flag);
    const long long row = blockIdx.x + static_cast<long long>(i) * gridDim.x;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      const bool in = c < chunks;
      float y[8] = {};
      if (in) {
        if (p.H) store8(static_cast<T*>(p.H) + row * p.ldh + 8 * c, v[k]);
        Vec8<T> wv;
        wv.load(w + 8 * c);
        wv.get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (v[k][e] * rstd) * y[e];
      }
      if constexpr (kA8) {
        __syncwarp();
        float sc;
        const uint2 q = quantise8(y, sc);
        if (in) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Y) + row * p.K + 8 * c) = q;
          if ((threadIdx.x & 15) == 0) p.S[row * (p.K >> 7) + (c >> 4)] = sc;
        }
      } else if (in) {
        store8(static_cast<T*>(p.Y) + row * p.ldy + 8 * c, y);
      }
    }
  }
  // After an abort no copy may still be in flight when the block ends.
  if (threadIdx.x == 0 && *abort_flag) {
    for (int i = max(0, issued - stages); i < issued; ++i) mbar_wait(full + 8 * (i % stages), (i / stages) & 1, err);
    mbar_wait(full + 8 * stages, 0, err);
  }
}

template <class T, bool kA8, int V>
cudaError_t launch_norm_stream(const NormParams& p, const NormArgs& a, int threads, int stages, int per_sm, size_t smem,
                               cudaStream_t s) {
  static AttrLatch latch;
  if (cudaError_t e = set_smem_attrs(norm_stream_kernel<T, kA8, V>, latch, 226 * 1024 - 2048, true); e != cudaSuccess)
    return e;
  const int grid = a.M < per_sm * a.num_sms ? a.M : per_sm * a.num_sms;
  return launch(norm_stream_kernel<T, kA8, V>, dim3(grid), dim3(threads), smem, s, a.pdl, p, stages, a.err);
}

template <class T, bool kA8>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s) {
  const NormParams p = {a.X, a.R, a.W, a.H, a.Y, a.S, a.eps, a.M, a.K, a.ldx, a.ldr, a.ldh, a.ldy};
  const int chunks = a.K / 8;
  if (chunks == 16)
    return launch(norm_kernel<T, kA8, 1, true>, dim3((a.M + 15) / 16), dim3(16, 16), 0, s, a.pdl, p);
  // Many long rows with the 8-bit output, whose group maxima make the time
  // between a row's loads long: the ring, four chunks a thread and as many
  // blocks as fit an SM with 2 to 4 rows each in flight (8192x5120 with
  // residual: 58.6 us in the kernel above, 52.0 with two chunks a thread, 47.9
  // with four; 4096x17408: 158 -> 84). The other output is as fast or faster
  // above (51.5 against 56.0), and so are short rows (8192x1024: 9.9 against 17.9).
  const int row_bytes = a.K * static_cast<int>(sizeof(T));
  const int slot = a.R ? 2 * row_bytes : row_bytes;
  constexpr int kRoom = 222 * 1024;
  if constexpr (kA8) {
    const int threads = ((chunks + 3) / 4 + 31) / 32 * 32;
    if (a.M > 4 * a.num_sms && chunks >= 512 && threads <= 1024 && row_bytes + 2 * slot + 2048 <= kRoom) {
      int per_sm = kRoom / (row_bytes + 2 * slot + 2048), stages = 2;
      if (per_sm > 2048 / threads) per_sm = 2048 / threads;
      while (stages < kMaxStages && per_sm * (row_bytes + (stages + 1) * slot + 2048) <= kRoom) ++stages;
      const size_t smem = static_cast<size_t>(row_bytes) + static_cast<size_t>(stages) * slot;
      return launch_norm_stream<T, kA8, 4>(p, a, threads, stages, per_sm, smem, s);
    }
  }
  // Few rows: as many threads to a row as it has chunks, for latency.
  int v = a.M <= a.num_sms ? 1 : 2;
  while (v < 4 && (chunks + v - 1) / v > 1024) v *= 2;
  if ((chunks + v - 1) / v > 1024) v = 0;
  const int tpr = v ? ((chunks + v - 1) / v + 31) / 32 * 32 : 1024;
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const dim3 grid((a.M + rows - 1) / rows), block(tpr, rows);
  if (v == 1) return launch(norm_kernel<T, kA8, 1, false>, grid, block, 0, s, a.pdl, p);
  if (v == 2) return launch(norm_kernel<T, kA8, 2, false>, grid, block, 0, s, a.pdl, p);
  if (v == 4) return launch(norm_kernel<T, kA8, 4, false>, grid, block, 0, s, a.pdl, p);
  return launch(norm_kernel<T, kA8, 0, false>, grid, dim3(1024, 1), 0, s, a.pdl, p);
}

}  // namespace

cudaError_t launch_w4_quantize(const QuantArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_quantise_t<__nv_bfloat16, false>(a, s);
  if (a.dtype == 1) return launch_quantise_t<__half, false>(a, s);
  return launch_quantise_t<float, false>(a, s);
}
cudaError_t launch_a8_quantize(const QuantArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_quantise_t<__nv_bfloat16, true>(a, s);
  if (a.dtype == 1) return launch_quantise_t<__half, true>(a, s);
  return launch_quantise_t<float, true>(a, s);
}
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_norm_t<__nv_bfloat16, false>(a, s);
  if (a.dtype == 1) return launch_norm_t<__half, false>(a, s);
  return launch_norm_t<float, false>(a, s);
}
cudaError_t launch_rms_norm_a8(const NormArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_norm_t<__nv_bfloat16, true>(a, s);
  if (a.dtype == 1) return launch_norm_t<__half, true>(a, s);
  return launch_norm_t<float, true>(a, s);
}

}  // namespace wqp
