// Row kernels of the quantised-activation path: 4-bit and 8-bit quantisation
// and the root-mean-square norm with the residual's addition.
//
// All three are bound by memory: each element is read once and written once,
// and the arithmetic between (a maximum, a quotient, a conversion) has to fit
// under the time of its bytes.
//
// w4_quantize, per group of 16 (amax = largest magnitude, g = global scale):
//   s = e4m3(amax / (6 g)), d = s * g, code = e2m1(x / d)
// a8_quantize, per group of 128 (amax floored at 2^-100):
//   s = amax / 448, code = e4m3(x * (448 / amax))
// rms_norm: h = x + r, y = (h * rsqrt(mean h^2 + eps)) * w, in FP32 from the
// unrounded sum; y is rounded once, to its own type or by a8_quantize's rule.
// A lane always holds 8 consecutive elements, so a group of 16 is a lane pair
// and a group of 128 is half a warp; the maxima are taken on the bits of the
// magnitudes, where a NaN is above infinity and infinity above every number.
#include <cuda_fp16.h>

#include "decode.cuh"

namespace wqp {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;
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

__device__ __forceinline__ uint32_t absmax_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

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
  uint32_t m = absmax_bits(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const float t = __uint_as_float(m) / six_g;
  const uint32_t s = f32x2_to_e4m3x2(t, 0.0f) & 0xFFu;
  const float d = e4m3_to_f32(s) * g;
  const bool finite = m < kInfBits;
  const float inv = (d > 0.0f && finite) ? 1.0f / d : 0.0f;
  float q[8];
  // x / d, correctly rounded, from the correctly rounded reciprocal by one
  // residual step (P. Markstein, "Computation of elementary functions on the
  // IBM RISC System/6000 processor", 1990): a quotient that falls on the
  // middle between two codes has to be recognised as such, which x * inv
  // alone misses for 3 of the 8 scale mantissas. Groups whose scale saturates
  // may overflow there and take the product as it is: they end at +-6.
  if (t <= 448.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = v[i] * inv;
      q[i] = fmaf(fmaf(-q0, d, v[i]), inv, q0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
  }
  scale = finite ? s : 0x7Fu;
  return finite ? f32x8_to_e2m1(q) : 0u;
}

// This lane's 8 elements of a 128-group (16 lanes): their codes, and the
// group's scale in all lanes. A group with a NaN or an infinity gets a NaN
// scale. The floor keeps 448 / amax finite.
__device__ __forceinline__ uint2 quantise8(const float (&v)[8], float& scale) {
  uint32_t m = absmax_bits(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  m = max(m, __float_as_uint(kA8Floor));
  const float amax = __uint_as_float(m < kInfBits ? m : 0x7FFFFFFFu);
  scale = amax / 448.0f;
  const float inv = 448.0f / amax;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ------------------------------------------------------------ quantisation
// One block = kThreads * U chunks of 8 elements. Contiguous rows are one long
// row; rows with a pitch find theirs by one division per chunk. Codes and
// scales are contiguous either way.
constexpr int kThreads = 256;

template <class T, bool kA8, bool kPitched, int U>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const T* X, uint8_t* codes, void* scales, float g,
                                                            float six_g, long long chunks, int cpr, int ldx) {
  pdl_launch_dependents();
  pdl_wait();
  const long long c0 = static_cast<long long>(blockIdx.x) * (kThreads * U) + threadIdx.x;
  Vec8<T> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long c = c0 + u * kThreads;
    x[u] = Vec8<T>{};
    if (c < chunks) {
      long long at = c * 8;
      if (kPitched) {
        const long long row = c / cpr;
        at = row * ldx + (c - row * cpr) * 8;
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
  if (a.ldx == a.K || a.M == 1)
    return launch(quantise_kernel<T, kA8, false, U>, grid, dim3(kThreads), 0, s, a.pdl, static_cast<const T*>(a.X),
                  a.codes, a.scales, a.gscale, six_g, chunks, cpr, a.ldx);
  return launch(quantise_kernel<T, kA8, true, U>, grid, dim3(kThreads), 0, s, a.pdl, static_cast<const T*>(a.X),
                a.codes, a.scales, a.gscale, six_g, chunks, cpr, a.ldx);
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

// Sum over the threads of a row: `warps` whole warps that share a slice of
// `part`. Every row of a block takes part.
__device__ __forceinline__ float row_sum(float v, float* part, int warps, int w) {
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
// long for that) reads it again.
template <class T, bool kA8, int V>
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
  auto out_of = [&](int c, bool in, const float (&v)[8], float rstd) {
    float y[8] = {};
    if (in) {
      if (h) store8(h + 8 * c, v);
      Vec8<T> wv;
      wv.load(w + 8 * c);
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
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * tpr;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
      if (live && c < chunks) sum_of(c, v[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    }
    ss = row_sum(ss, part + threadIdx.y * warps, warps, threadIdx.x >> 5);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * tpr;
      out_of(c, live && c < chunks, v[i], rstd);
    }
  } else {
    float ss = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += tpr) {
      float v[8];
      sum_of(c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
    }
    ss = row_sum(ss, part, warps, threadIdx.x >> 5);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.K) + p.eps);
    for (int c0 = 0; c0 < chunks; c0 += tpr) {
      const int c = c0 + threadIdx.x;
      float v[8] = {};
      if (c < chunks) sum_of(c, v);
      out_of(c, c < chunks, v, rstd);
    }
  }
}

template <class T, bool kA8>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s) {
  const NormParams p = {a.X, a.R, a.W, a.H, a.Y, a.S, a.eps, a.M, a.K, a.ldx, a.ldr, a.ldh, a.ldy};
  const int chunks = a.K / 8;
  // Few rows: as many threads to a row as it has chunks, for latency.
  int v = a.M <= a.num_sms ? 1 : 2;
  while (v < 4 && (chunks + v - 1) / v > 1024) v *= 2;
  if ((chunks + v - 1) / v > 1024) v = 0;
  const int tpr = v ? ((chunks + v - 1) / v + 31) / 32 * 32 : 1024;
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const dim3 grid((a.M + rows - 1) / rows), block(tpr, rows);
  if (v == 1) return launch(norm_kernel<T, kA8, 1>, grid, block, 0, s, a.pdl, p);
  if (v == 2) return launch(norm_kernel<T, kA8, 2>, grid, block, 0, s, a.pdl, p);
  if (v == 4) return launch(norm_kernel<T, kA8, 4>, grid, block, 0, s, a.pdl, p);
  return launch(norm_kernel<T, kA8, 0>, grid, dim3(1024, 1), 0, s, a.pdl, p);
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
