// C-ABI layer of libwqp.so: argument validation, per-device set-up, row
// chunking and dispatch to the kernel translation units. Declarations and the
// contract of every entry point are in include/wqp.h.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/wqp.h"
#include "common.cuh"
#include "internal.h"

using namespace wqp;

namespace {

// Device error word (one per device image of this module).
__device__ unsigned g_device_error = 0;

thread_local char t_last_error[256] = "";

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_last_error, sizeof(t_last_error), fmt, ap);
  va_end(ap);
  return status;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(WQP_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

std::atomic<int> g_pdl{0};

struct DeviceInfo {
  std::once_flag once;
  int status = WQP_OK;
  int num_sms = 0;
  unsigned* err = nullptr;
  char msg[160] = "";
};
DeviceInfo g_dev[kMaxDevices];

// Per-device set-up, run once with that device current: checks for sm_103
// and resolves the device error word's address.
int device_setup(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(WQP_ERR_UNSUPPORTED, "device %d", dev);
  DeviceInfo& d = g_dev[dev];
  std::call_once(d.once, [&] {
    int major = 0, minor = 0;
    cudaError_t e1 = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaError_t e2 = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaError_t e3 = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e1 != cudaSuccess || e2 != cudaSuccess || e3 != cudaSuccess) {
      d.status = WQP_ERR_CUDA;
      snprintf(d.msg, sizeof(d.msg), "device attribute query failed");
      return;
    }
    if (major != 10 || minor != 3) {
      d.status = WQP_ERR_UNSUPPORTED;
      snprintf(d.msg, sizeof(d.msg), "device %d is sm_%d%d; libwqp is built for sm_103a", dev,
               major, minor);
      return;
    }
    cudaError_t e4 = cudaGetSymbolAddress(reinterpret_cast<void**>(&d.err), g_device_error);
    if (e4 != cudaSuccess) {
      d.status = WQP_ERR_CUDA;
      snprintf(d.msg, sizeof(d.msg), "cudaGetSymbolAddress: %s", cudaGetErrorString(e4));
    }
  });
  if (d.status != WQP_OK) return fail(d.status, "%s", d.msg);
  *out = &d;
  return WQP_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

enum class Fmt { Q2, W4, W8, W8TC, Q2TC, W4TC, Q2MMA, W8MMA, W4MMA };

const char* fmt_name(Fmt f) {
  switch (f) {
    case Fmt::Q2: return "q2_gemv";
    case Fmt::W4: return "w4a16_gemv";
    case Fmt::W8: return "w8a16_gemm";
    case Fmt::W8TC: return "w8a16_gemm_tc";
    case Fmt::Q2TC: return "q2_gemm_tc";
    case Fmt::W4TC: return "w4a16_gemm_tc";
    case Fmt::Q2MMA: return "q2_gemm_mma";
    case Fmt::W8MMA: return "w8a16_gemm_mma";
    case Fmt::W4MMA: return "w4a16_gemm_mma";
  }
  return "?";
}

int validate(Fmt f, const void* A, int lda, const void* W, const void* scales, void* C, int ldc,
             int M, int N, int K) {
  const char* nm = fmt_name(f);
  if (M < 0) return fail(WQP_ERR_INVALID_ARG, "%s: M=%d < 0", nm, M);
  const bool w4 = (f == Fmt::W4 || f == Fmt::W4TC || f == Fmt::W4MMA);
  const bool q2 = (f == Fmt::Q2 || f == Fmt::Q2TC || f == Fmt::Q2MMA);
  if (N < 1 || N > (1 << 24)) return fail(WQP_ERR_INVALID_ARG, "%s: N=%d outside 1..2^24", nm, N);
  if (K < 128 || K > (1 << 20) || K % 128 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 128 in [128, 2^20]", nm, K);
  if (!A || !W || !C) return fail(WQP_ERR_INVALID_ARG, "%s: NULL A, W or C", nm);
  if ((f == Fmt::Q2TC || f == Fmt::Q2MMA || f == Fmt::W8MMA || f == Fmt::W4MMA) && K % 1024 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 1024", nm, K);
  if (f == Fmt::W4TC && K % 256 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 256", nm, K);
  if (q2 && scales)
    return fail(WQP_ERR_INVALID_ARG, "%s: Q2_0 scales are inline; scales must be NULL", nm);
  if (!q2 && !scales) return fail(WQP_ERR_INVALID_ARG, "%s: NULL scales", nm);
  if (!aligned(A, 16) || !aligned(W, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: A and W must be 16-byte aligned", nm);
  if (w4 && !aligned(scales, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be 16-byte aligned", nm);
  if ((f == Fmt::W8 || f == Fmt::W8TC) && !aligned(scales, 4))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", nm);
  if (f == Fmt::W8MMA && !aligned(scales, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be 16-byte aligned", nm);
  if (!aligned(C, 2)) return fail(WQP_ERR_INVALID_ARG, "%s: C must be 2-byte aligned", nm);
  if (lda < K || lda % 8 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: lda=%d must be >= K=%d and a multiple of 8", nm, lda, K);
  if (ldc < N) return fail(WQP_ERR_INVALID_ARG, "%s: ldc=%d must be >= N=%d", nm, ldc, N);
  return WQP_OK;
}

int run_gemm(Fmt f, const void* A, int lda, const void* W, const void* scales, float gscale,
             void* C, int ldc, int M, int N, int K, void* stream) {
  int st = validate(f, A, lda, W, scales, C, ldc, M, N, K);
  if (st != WQP_OK) return st;
  if ((f == Fmt::W4 || f == Fmt::W4TC || f == Fmt::W4MMA) && !(gscale == gscale))
    return fail(WQP_ERR_INVALID_ARG, "%s: global_scale is NaN", fmt_name(f));
  if (M == 0) return WQP_OK;
  DeviceInfo* dev = nullptr;
  if ((st = device_setup(&dev)) != WQP_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GemvArgs a = {};
  a.W = W;
  a.scales = scales;
  a.N = N;
  a.K = K;
  a.lda = lda;
  a.ldc = ldc;
  a.gscale = gscale;
  a.err = dev->err;
  a.num_sms = dev->num_sms;
  a.pdl = g_pdl.load(std::memory_order_relaxed) != 0;
  const int step = WQP_MAX_M_PER_LAUNCH;
  for (int r0 = 0; r0 < M; r0 += step) {
    a.M = (M - r0) < step ? (M - r0) : step;
    a.A = static_cast<const char*>(A) + static_cast<size_t>(r0) * lda * 2;
    a.C = static_cast<char*>(C) + static_cast<size_t>(r0) * ldc * 2;
    cudaError_t e = cudaSuccess;
    switch (f) {
      case Fmt::Q2: e = launch_q2_gemv(a, s); break;
      case Fmt::W4: e = launch_w4a16_gemv(a, s); break;
      case Fmt::W8: e = launch_w8a16_gemm(a, s); break;
      case Fmt::W8TC: e = launch_w8a16_gemm_tc(a, s); break;
      case Fmt::Q2TC: e = launch_q2_gemm_tc(a, s); break;
      case Fmt::W4TC: e = launch_w4a16_gemm_tc(a, s); break;
      case Fmt::Q2MMA: e = launch_q2_gemm_mma(a, s); break;
      case Fmt::W8MMA: e = launch_w8a16_gemm_mma(a, s); break;
      case Fmt::W4MMA: e = launch_w4a16_gemm_mma(a, s); break;
    }
    if (e != cudaSuccess) return cuda_fail(e, fmt_name(f));
  }
  return WQP_OK;
}

int run_dequant(int fmt, const void* W, const void* scales, float gscale, float* out, int N, int K,
                void* stream) {
  static const char* names[] = {"q2_dequant", "w4a16_dequant", "w8a16_dequant"};
  const char* nm = names[fmt];
  if (N < 1 || N > (1 << 24)) return fail(WQP_ERR_INVALID_ARG, "%s: N=%d outside 1..2^24", nm, N);
  if (K < 128 || K > (1 << 20) || K % 128 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 128 in [128, 2^20]", nm, K);
  if (!W || !out) return fail(WQP_ERR_INVALID_ARG, "%s: NULL W or out", nm);
  if (fmt == 0 && scales) return fail(WQP_ERR_INVALID_ARG, "%s: scales must be NULL", nm);
  if (fmt != 0 && !scales) return fail(WQP_ERR_INVALID_ARG, "%s: NULL scales", nm);
  if (!aligned(W, 16) || !aligned(out, 4))
    return fail(WQP_ERR_INVALID_ARG, "%s: W must be 16-byte and out 4-byte aligned", nm);
  if (fmt == 1 && !aligned(scales, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be 16-byte aligned", nm);
  if (fmt == 2 && !aligned(scales, 4))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", nm);
  DeviceInfo* dev = nullptr;
  int st = device_setup(&dev);
  if (st != WQP_OK) return st;
  DequantArgs a = {W, scales, out, N, K, gscale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fmt == 0   ? launch_q2_dequant(a, s)
                  : fmt == 1 ? launch_w4a16_dequant(a, s)
                             : launch_w8a16_dequant(a, s);
  if (e != cudaSuccess) return cuda_fail(e, nm);
  return WQP_OK;
}

// Shape of the quantised-activation entries: M, K, and one operand with rows.
int check_rows(const char* nm, int M, int K, int dtype) {
  if (M < 0) return fail(WQP_ERR_INVALID_ARG, "%s: M=%d < 0", nm, M);
  if (K < 128 || K > (1 << 20) || K % 128 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 128 in [128, 2^20]", nm, K);
  if (dtype < WQP_BF16 || dtype > WQP_F32)
    return fail(WQP_ERR_INVALID_ARG, "%s: dtype=%d is not a wqp_dtype", nm, dtype);
  return WQP_OK;
}

int check_pitched(const char* nm, const char* what, const void* p, int ld, int K) {
  if (!p) return fail(WQP_ERR_INVALID_ARG, "%s: NULL %s", nm, what);
  if (!aligned(p, 16)) return fail(WQP_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", nm, what);
  if (ld < K || ld % 8 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: pitch %d of %s must be >= K=%d and a multiple of 8", nm, ld, what, K);
  return WQP_OK;
}

int check_codes(const char* nm, const void* codes, const void* scales, uintptr_t scale_align) {
  if (!codes || !scales) return fail(WQP_ERR_INVALID_ARG, "%s: NULL codes or scales", nm);
  if (!aligned(codes, 8)) return fail(WQP_ERR_INVALID_ARG, "%s: codes must be 8-byte aligned", nm);
  if (!aligned(scales, scale_align))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be %d-byte aligned", nm, static_cast<int>(scale_align));
  return WQP_OK;
}

int run_quantize(bool a8, const void* X, int ldx, int dtype, float gscale, void* codes, void* scales, int M, int K,
                 void* stream) {
  const char* nm = a8 ? "a8_quantize" : "w4_quantize";
  int st = check_rows(nm, M, K, dtype);
  if (st == WQP_OK && !(gscale >= 0x1p-100f && gscale <= 0x1p100f))
    st = fail(WQP_ERR_INVALID_ARG, "%s: global_scale=%g outside 2^-100..2^100", nm, gscale);
  if (st == WQP_OK && M == 0) return WQP_OK;
  if (st == WQP_OK) st = check_pitched(nm, "X", X, ldx, K);
  if (st == WQP_OK) st = check_codes(nm, codes, scales, a8 ? 4 : 1);
  DeviceInfo* dev = nullptr;
  if (st != WQP_OK || (st = device_setup(&dev)) != WQP_OK) return st;
  const QuantArgs a = {X,     static_cast<uint8_t*>(codes), scales, gscale, dtype, M, K, ldx,
                       g_pdl.load(std::memory_order_relaxed) != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a8 ? launch_a8_quantize(a, s) : launch_w4_quantize(a, s);
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

int run_norm(bool a8, const void* X, int ldx, const void* R, int ldr, const void* W, float eps, void* H, int ldh,
             void* Y, int ldy, float* S, int dtype, int M, int K, void* stream) {
  const char* nm = a8 ? "rms_norm_a8" : "rms_norm";
  int st = check_rows(nm, M, K, dtype);
  if (st == WQP_OK && !(eps >= 0.0f && eps <= 3.4e38f))
    st = fail(WQP_ERR_INVALID_ARG, "%s: eps=%g must be finite and not negative", nm, eps);
  if (st == WQP_OK && M == 0) return WQP_OK;
  if (st == WQP_OK) st = check_pitched(nm, "X", X, ldx, K);
  if (st == WQP_OK && R) st = check_pitched(nm, "residual", R, ldr, K);
  if (st == WQP_OK && H) st = check_pitched(nm, "residual_out", H, ldh, K);
  if (st == WQP_OK) st = check_pitched(nm, "weight", W, K, K);
  if (st == WQP_OK) st = a8 ? check_codes(nm, Y, S, 4) : check_pitched(nm, "Y", Y, ldy, K);
  DeviceInfo* dev = nullptr;
  if (st != WQP_OK || (st = device_setup(&dev)) != WQP_OK) return st;
  const NormArgs a = {X,   R,   W,   H,   Y,   S, eps, dtype, M, K, ldx, ldr, ldh, ldy, dev->err, dev->num_sms,
                      g_pdl.load(std::memory_order_relaxed) != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a8 ? launch_rms_norm_a8(a, s) : launch_rms_norm(a, s);
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

// a * b as a power of two times a factor. The power is 1 unless FP32 has the
// product as infinity, as 0 or with fewer bits, though a sum times it may be in
// BF16's range: the 4-bit sums are 0 or between 2^-20 and 2^43 in magnitude, so
// their product with the power is in FP32's normal range, and the factor takes
// it out of that only where the result is.
void split_scale(float a, float b, float* pow, float* factor) {
  const double p = static_cast<double>(a) * b, m = p < 0.0 ? -p : p;     // exact
  *pow = 1.0f;
  *factor = a * b;
  if (m > 0.0 && m < 0x1p-126) {
    *pow = 0x1p-84f;
    *factor = static_cast<float>(p * 0x1p84);
  } else if (m >= 0x1p128 && m < 0x1p256) {      // from 2^148 on only zeros stay finite
    *pow = 0x1p60f;
    *factor = m < 0x1p187 ? static_cast<float>(p * 0x1p-60) : (p < 0.0 ? -0x1p127f : 0x1p127f);
  }
}

int run_act_gemm(bool w4, const void* A, const void* SA, float ga, const void* W, const void* SW, float gw, void* C,
                 int ldc, int M, int N, int K, void* stream) {
  const char* nm = w4 ? "w4a4_gemm" : "w8a8_gemm";
  const int unit = w4 ? 256 : 128;
  if (M < 0) return fail(WQP_ERR_INVALID_ARG, "%s: M=%d < 0", nm, M);
  if (N < 1 || N > (1 << 24)) return fail(WQP_ERR_INVALID_ARG, "%s: N=%d outside 1..2^24", nm, N);
  if (K < unit || K > (1 << 20) || K % unit != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of %d in [%d, 2^20]", nm, K, unit, unit);
  if (!(ga == ga) || !(gw == gw)) return fail(WQP_ERR_INVALID_ARG, "%s: a global scale is NaN", nm);
  if (M == 0) return WQP_OK;
  if (!A || !SA || !W || !SW || !C) return fail(WQP_ERR_INVALID_ARG, "%s: NULL A, W, C or scales", nm);
  if (!aligned(A, 16) || !aligned(W, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: A and W must be 16-byte aligned", nm);
  const uintptr_t sal = w4 ? 16 : 4;
  if (!aligned(SA, sal) || !aligned(SW, sal))
    return fail(WQP_ERR_INVALID_ARG, "%s: scales must be %d-byte aligned", nm, static_cast<int>(sal));
  if (!aligned(C, 2)) return fail(WQP_ERR_INVALID_ARG, "%s: C must be 2-byte aligned", nm);
  if (ldc < N) return fail(WQP_ERR_INVALID_ARG, "%s: ldc=%d must be >= N=%d", nm, ldc, N);
  DeviceInfo* dev = nullptr;
  const int st = device_setup(&dev);
  if (st != WQP_OK) return st;
  float gpow, gscale;
  split_scale(ga, gw, &gpow, &gscale);
  const ActGemmArgs a = {A, SA, W, SW, C, gpow, gscale, M, N, K, ldc, dev->err, dev->num_sms,
                         g_pdl.load(std::memory_order_relaxed) != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = w4 ? launch_w4a4_gemm(a, s) : launch_w8a8_gemm(a, s);
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

// Experts, the slots of a token, and their pairs.
int check_pairs(const char* nm, int T, int slots, int E) {
  if (T < 0) return fail(WQP_ERR_INVALID_ARG, "%s: T=%d < 0", nm, T);
  if (slots < 1 || slots > kMaxTopK) return fail(WQP_ERR_INVALID_ARG, "%s: %d slots outside 1..%d", nm, slots, kMaxTopK);
  if (E < 1 || E > kMaxExperts) return fail(WQP_ERR_INVALID_ARG, "%s: E=%d outside 1..%d", nm, E, kMaxExperts);
  if (static_cast<long long>(T) * slots > (1 << 30))
    return fail(WQP_ERR_INVALID_ARG, "%s: %d tokens of %d slots are more than 2^30 pairs", nm, T, slots);
  return WQP_OK;
}

int check_words(const char* nm, const char* what, const void* p) {
  if (!p) return fail(WQP_ERR_INVALID_ARG, "%s: NULL %s", nm, what);
  if (!aligned(p, 4)) return fail(WQP_ERR_INVALID_ARG, "%s: %s must be 4-byte aligned", nm, what);
  return WQP_OK;
}

int run_route(const void* X, int ldl, int dtype, const float* bias, int* ids, float* weights, int T, int E, int top_k,
              int scoring, int groups, int top_groups, int group_best, int renormalise, float scale, void* stream) {
  const char* nm = "expert_route";
  int st = check_pairs(nm, T, top_k, E);
  if (st != WQP_OK) return st;
  if (dtype < WQP_BF16 || dtype > WQP_F32) return fail(WQP_ERR_INVALID_ARG, "%s: dtype=%d is not a wqp_dtype", nm, dtype);
  if (scoring != WQP_SOFTMAX && scoring != WQP_SIGMOID)
    return fail(WQP_ERR_INVALID_ARG, "%s: scoring=%d is not a wqp_scoring", nm, scoring);
  if (groups < 1 || groups > kMaxGroups || E % groups != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: groups=%d must divide E=%d and be at most %d", nm, groups, E, kMaxGroups);
  if (top_groups < 1 || top_groups > groups)
    return fail(WQP_ERR_INVALID_ARG, "%s: top_groups=%d outside 1..%d", nm, top_groups, groups);
  if (group_best != 1 && group_best != 2) return fail(WQP_ERR_INVALID_ARG, "%s: group_best=%d is not 1 or 2", nm, group_best);
  if (top_k > E / groups * top_groups)
    return fail(WQP_ERR_INVALID_ARG, "%s: top_k=%d of %d experts", nm, top_k, E / groups * top_groups);
  if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return fail(WQP_ERR_INVALID_ARG, "%s: scale=%g must be finite", nm, scale);
  if (T == 0) return WQP_OK;
  if (!X) return fail(WQP_ERR_INVALID_ARG, "%s: NULL logits", nm);
  if (!aligned(X, dtype == WQP_F32 ? 4 : 2)) return fail(WQP_ERR_INVALID_ARG, "%s: logits must be aligned to their type", nm);
  if (ldl < E) return fail(WQP_ERR_INVALID_ARG, "%s: pitch %d of logits must be >= E=%d", nm, ldl, E);
  if (bias && !aligned(bias, 4)) return fail(WQP_ERR_INVALID_ARG, "%s: bias must be 4-byte aligned", nm);
  if ((st = check_words(nm, "ids", ids)) != WQP_OK || (st = check_words(nm, "weights", weights)) != WQP_OK) return st;
  DeviceInfo* dev = nullptr;
  if ((st = device_setup(&dev)) != WQP_OK) return st;
  const RouteArgs a = {X, bias, ids, weights, dtype, T, E, ldl, top_k, scoring == WQP_SIGMOID, renormalise != 0,
                       groups, top_groups, group_best, scale, g_pdl.load(std::memory_order_relaxed) != 0};
  const cudaError_t e = launch_expert_route(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

int run_order(const int* ids, int* rows, int* offsets, int R, int E, void* stream) {
  const char* nm = "expert_order";
  if (R < 0 || R > (1 << 30)) return fail(WQP_ERR_INVALID_ARG, "%s: R=%d outside 0..2^30", nm, R);
  if (E < 1 || E > kMaxExperts) return fail(WQP_ERR_INVALID_ARG, "%s: E=%d outside 1..%d", nm, E, kMaxExperts);
  int st = check_words(nm, "offsets", offsets);
  if (st == WQP_OK && R > 0) st = check_words(nm, "ids", ids);
  if (st == WQP_OK && R > 0) st = check_words(nm, "rows", rows);
  DeviceInfo* dev = nullptr;
  if (st != WQP_OK || (st = device_setup(&dev)) != WQP_OK) return st;
  const OrderArgs a = {ids, rows, offsets, R, E, g_pdl.load(std::memory_order_relaxed) != 0};
  const cudaError_t e = launch_expert_order(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

int run_experts(const void* A, int lda, const void* W, const void* scales, const float* globals, const int* rows,
                const int* offsets, void* C, int ldc, int T, int slots, int E, int N, int K, int gated, void* workspace,
                void* stream) {
  const char* nm = "w4a16_experts";
  int st = check_pairs(nm, T, slots, E);
  if (st != WQP_OK) return st;
  if (N < 1 || N > (1 << 24)) return fail(WQP_ERR_INVALID_ARG, "%s: N=%d outside 1..2^24", nm, N);
  if (gated && N % 2 != 0) return fail(WQP_ERR_INVALID_ARG, "%s: N=%d must be even, gate and up", nm, N);
  if (K < 128 || K > (1 << 20) || K % 128 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: K=%d must be a multiple of 128 in [128, 2^20]", nm, K);
  if (T == 0) return WQP_OK;
  if ((st = check_pitched(nm, "A", A, lda, K)) != WQP_OK) return st;
  if (!W || !scales || !C) return fail(WQP_ERR_INVALID_ARG, "%s: NULL W, scales or C", nm);
  if (!aligned(W, 16) || !aligned(scales, 16))
    return fail(WQP_ERR_INVALID_ARG, "%s: W and scales must be 16-byte aligned", nm);
  if (globals && !aligned(globals, 4)) return fail(WQP_ERR_INVALID_ARG, "%s: global_scales must be 4-byte aligned", nm);
  if ((st = check_words(nm, "rows", rows)) != WQP_OK || (st = check_words(nm, "offsets", offsets)) != WQP_OK) return st;
  const int outs = gated ? N / 2 : N;
  if (!workspace && experts_workspace(T, slots, E, N, K)) return fail(WQP_ERR_INVALID_ARG, "%s: NULL workspace", nm);
  if (workspace && !aligned(workspace, 16)) return fail(WQP_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", nm);
  if (static_cast<long long>(T) * slots * outs > (1ll << 38))
    return fail(WQP_ERR_INVALID_ARG, "%s: %lld rows of %d outputs are too many", nm, static_cast<long long>(T) * slots, outs);
  if (!aligned(C, 2)) return fail(WQP_ERR_INVALID_ARG, "%s: C must be 2-byte aligned", nm);
  if (ldc < outs) return fail(WQP_ERR_INVALID_ARG, "%s: ldc=%d must be >= %d", nm, ldc, outs);
  DeviceInfo* dev = nullptr;
  if ((st = device_setup(&dev)) != WQP_OK) return st;
  const ExpertsArgs a = {A, static_cast<const uint8_t*>(W), static_cast<const uint8_t*>(scales), globals, rows, offsets, C,
                         lda, ldc, T, slots, E, N, K, gated != 0, workspace, nullptr, dev->err, dev->num_sms,
                         g_pdl.load(std::memory_order_relaxed) != 0};
  const cudaError_t e = launch_w4a16_experts(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

int run_combine(const void* Y, int ldy, const float* weights, const int* ids, int E, const void* R, int ldr, void* out,
                int ldo, int dtype, int T, int slots, int H, void* stream) {
  const char* nm = "expert_combine";
  int st = check_pairs(nm, T, slots, E);
  if (st != WQP_OK) return st;
  if (dtype < WQP_BF16 || dtype > WQP_F32) return fail(WQP_ERR_INVALID_ARG, "%s: dtype=%d is not a wqp_dtype", nm, dtype);
  if (H < 8 || H > (1 << 20) || H % 8 != 0)
    return fail(WQP_ERR_INVALID_ARG, "%s: H=%d must be a multiple of 8 in [8, 2^20]", nm, H);
  if (static_cast<long long>(T) * H > (1ll << 38)) return fail(WQP_ERR_INVALID_ARG, "%s: T=%d rows of %d are too many", nm, T, H);
  if (T == 0) return WQP_OK;
  st = check_pitched(nm, "Y", Y, ldy, H);
  if (st == WQP_OK && R) st = check_pitched(nm, "residual", R, ldr, H);
  if (st == WQP_OK) st = check_pitched(nm, "out", out, ldo, H);
  if (st == WQP_OK) st = check_words(nm, "weights", weights);
  if (st == WQP_OK) st = check_words(nm, "ids", ids);
  DeviceInfo* dev = nullptr;
  if (st != WQP_OK || (st = device_setup(&dev)) != WQP_OK) return st;
  const CombineArgs a = {Y, weights, ids, R, out, ldy, ldr, ldo, dtype, T, slots, E, H,
                         g_pdl.load(std::memory_order_relaxed) != 0};
  const cudaError_t e = launch_expert_combine(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WQP_OK : cuda_fail(e, nm);
}

}  // namespace

namespace wqp {
// A bounded wait that nothing completes: one CTA waits, through the same
// helper the GEMM kernels use, on an mbarrier no thread arrives on. The wait
// gives up after limit_ns of wall time, records the timeout in the device
// error word and the kernel returns (no trap, no fault, no hang).
__global__ void wait_timeout_selftest_kernel(unsigned* err, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t never;
  const uint32_t bar = smem_u32(&never);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_ns(bar, 0, err, limit_ns);
}
}  // namespace wqp

extern "C" {

int q2_gemv(const void* A, const void* W, const void* scales, void* C, int M, int N, int K,
            void* stream) {
  if (scales) return fail(WQP_ERR_INVALID_ARG, "q2_gemv: Q2_0 scales are inline; must be NULL");
  return run_gemm(Fmt::Q2, A, K, W, nullptr, 1.0f, C, N, M, N, K, stream);
}

int q2_gemv_strided(const void* A, int lda, const void* W, void* C, int ldc, int M, int N, int K,
                    void* stream) {
  return run_gemm(Fmt::Q2, A, lda, W, nullptr, 1.0f, C, ldc, M, N, K, stream);
}

int q2_gemm_tc(const void* A, const void* W, void* C, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::Q2TC, A, K, W, nullptr, 1.0f, C, N, M, N, K, stream);
}

int q2_gemm_tc_strided(const void* A, int lda, const void* W, void* C, int ldc, int M, int N, int K,
                       void* stream) {
  return run_gemm(Fmt::Q2TC, A, lda, W, nullptr, 1.0f, C, ldc, M, N, K, stream);
}

int q2_gemm_mma(const void* A, const void* W, void* C, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::Q2MMA, A, K, W, nullptr, 1.0f, C, N, M, N, K, stream);
}

int q2_gemm_mma_strided(const void* A, int lda, const void* W, void* C, int ldc, int M, int N, int K,
                        void* stream) {
  return run_gemm(Fmt::Q2MMA, A, lda, W, nullptr, 1.0f, C, ldc, M, N, K, stream);
}

int w4a16_gemv(const void* A, const void* W, const void* scales, void* C, int M, int N, int K,
               void* stream) {
  return run_gemm(Fmt::W4, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w4a16_gemv_ex(const void* A, int lda, const void* W, const void* scales, float global_scale,
                  void* C, int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W4, A, lda, W, scales, global_scale, C, ldc, M, N, K, stream);
}

int w4a16_gemm_tc(const void* A, const void* W, const void* scales, void* C, int M, int N, int K,
                  void* stream) {
  return run_gemm(Fmt::W4TC, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w4a16_gemm_tc_ex(const void* A, int lda, const void* W, const void* scales, float global_scale,
                     void* C, int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W4TC, A, lda, W, scales, global_scale, C, ldc, M, N, K, stream);
}

int w4a16_gemm_mma(const void* A, const void* W, const void* scales, void* C, int M, int N, int K,
                   void* stream) {
  return run_gemm(Fmt::W4MMA, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w4a16_gemm_mma_ex(const void* A, int lda, const void* W, const void* scales, float global_scale,
                      void* C, int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W4MMA, A, lda, W, scales, global_scale, C, ldc, M, N, K, stream);
}

int w8a16_gemm_mma(const void* A, const void* W, const float* scales, void* C, int M, int N, int K,
                   void* stream) {
  return run_gemm(Fmt::W8MMA, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w8a16_gemm_mma_strided(const void* A, int lda, const void* W, const float* scales, void* C,
                           int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W8MMA, A, lda, W, scales, 1.0f, C, ldc, M, N, K, stream);
}

int w8a16_gemm(const void* A, const void* W, const float* scales, void* C, int M, int N, int K,
               void* stream) {
  return run_gemm(Fmt::W8, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w8a16_gemm_strided(const void* A, int lda, const void* W, const float* scales, void* C,
                       int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W8, A, lda, W, scales, 1.0f, C, ldc, M, N, K, stream);
}

int w8a16_gemm_tc(const void* A, const void* W, const float* scales, void* C, int M, int N, int K,
                  void* stream) {
  return run_gemm(Fmt::W8TC, A, K, W, scales, 1.0f, C, N, M, N, K, stream);
}

int w8a16_gemm_tc_strided(const void* A, int lda, const void* W, const float* scales, void* C,
                          int ldc, int M, int N, int K, void* stream) {
  return run_gemm(Fmt::W8TC, A, lda, W, scales, 1.0f, C, ldc, M, N, K, stream);
}

int w4_quantize(const void* X, int ldx, int dtype, float global_scale, void* codes, void* scales, int M, int K,
                void* stream) {
  return run_quantize(false, X, ldx, dtype, global_scale, codes, scales, M, K, stream);
}

int a8_quantize(const void* X, int ldx, int dtype, void* codes, float* scales, int M, int K, void* stream) {
  return run_quantize(true, X, ldx, dtype, 1.0f, codes, scales, M, K, stream);
}

int rms_norm(const void* X, int ldx, const void* residual, int ldr, const void* weight, float eps, void* residual_out,
             int ldro, void* Y, int ldy, int dtype, int M, int K, void* stream) {
  return run_norm(false, X, ldx, residual, ldr, weight, eps, residual_out, ldro, Y, ldy, nullptr, dtype, M, K, stream);
}

int rms_norm_a8(const void* X, int ldx, const void* residual, int ldr, const void* weight, float eps,
                void* residual_out, int ldro, void* codes, float* scales, int dtype, int M, int K, void* stream) {
  return run_norm(true, X, ldx, residual, ldr, weight, eps, residual_out, ldro, codes, K, scales, dtype, M, K, stream);
}

int w4a4_gemm(const void* A, const void* a_scales, float a_global, const void* W, const void* w_scales,
              float w_global, void* C, int ldc, int M, int N, int K, void* stream) {
  return run_act_gemm(true, A, a_scales, a_global, W, w_scales, w_global, C, ldc, M, N, K, stream);
}

int w8a8_gemm(const void* A, const float* a_scales, const void* W, const float* w_scales, void* C, int ldc, int M,
              int N, int K, void* stream) {
  return run_act_gemm(false, A, a_scales, 1.0f, W, w_scales, 1.0f, C, ldc, M, N, K, stream);
}

int expert_route(const void* logits, int ldl, int dtype, const float* bias, int* ids, float* weights, int T, int E,
                 int top_k, int scoring, int groups, int top_groups, int group_best, int renormalise, float scale,
                 void* stream) {
  return run_route(logits, ldl, dtype, bias, ids, weights, T, E, top_k, scoring, groups, top_groups, group_best, renormalise,
                   scale, stream);
}

int expert_order(const int* ids, int* rows, int* offsets, int R, int E, void* stream) {
  return run_order(ids, rows, offsets, R, E, stream);
}

int w4a16_experts(const void* A, int lda, const void* W, const void* scales, const float* global_scales, const int* rows,
                  const int* offsets, void* C, int ldc, int T, int slots, int E, int N, int K, int gated, void* workspace,
                  void* stream) {
  return run_experts(A, lda, W, scales, global_scales, rows, offsets, C, ldc, T, slots, E, N, K, gated, workspace, stream);
}

size_t w4a16_experts_workspace(int T, int slots, int E, int N, int K) {
  if (check_pairs("w4a16_experts_workspace", T, slots, E) != WQP_OK) return 0;
  if (N < 1 || N > (1 << 24) || K < 128 || K > (1 << 20) || K % 128 != 0) return 0;
  return experts_workspace(T, slots, E, N, K);
}

int expert_combine(const void* Y, int ldy, const float* weights, const int* ids, int E, const void* residual, int ldr,
                   void* out, int ldo, int dtype, int T, int slots, int H, void* stream) {
  return run_combine(Y, ldy, weights, ids, E, residual, ldr, out, ldo, dtype, T, slots, H, stream);
}

int q2_dequant(const void* W, float* out, int N, int K, void* stream) {
  return run_dequant(0, W, nullptr, 1.0f, out, N, K, stream);
}

int w4a16_dequant(const void* W, const void* scales, float global_scale, float* out, int N, int K,
                  void* stream) {
  return run_dequant(1, W, scales, global_scale, out, N, K, stream);
}

int w8a16_dequant(const void* W, const float* scales, float* out, int N, int K, void* stream) {
  return run_dequant(2, W, scales, 1.0f, out, N, K, stream);
}

int wqp_row_chunks(int M, int K, int N, int max_rows, long long* out, int cap) {
  if (M < 0 || K < 0 || N < 0 || max_rows < 1 || cap < 0) return -1;
  int n = 0;
  for (int r0 = 0; r0 < M; r0 += max_rows) {
    if (n >= cap || !out) return -1;
    int rows = (M - r0) < max_rows ? (M - r0) : max_rows;
    out[3 * n + 0] = static_cast<long long>(r0) * K * 2;
    out[3 * n + 1] = static_cast<long long>(r0) * N * 2;
    out[3 * n + 2] = rows;
    ++n;
  }
  return n;
}

int wqp_set_pdl(int enable) { return g_pdl.exchange(enable ? 1 : 0); }

int wqp_selftest_wait_timeout(int limit_us, void* stream) {
  if (limit_us < 1 || limit_us > 1000000)
    return fail(WQP_ERR_INVALID_ARG, "wqp_selftest_wait_timeout: limit_us=%d outside 1..10^6", limit_us);
  DeviceInfo* dev = nullptr;
  int st = device_setup(&dev);
  if (st != WQP_OK) return st;
  wait_timeout_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      dev->err, static_cast<uint64_t>(limit_us) * 1000u);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "wqp_selftest_wait_timeout");
  return WQP_OK;
}

int wqp_get_device_error(void) {
  DeviceInfo* dev = nullptr;
  int st = device_setup(&dev);
  if (st != WQP_OK) return st;
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v));
  if (e != cudaSuccess) return cuda_fail(e, "wqp_get_device_error");
  if (v) {
    unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_fail(e, "wqp_get_device_error");
    return fail(WQP_ERR_DEVICE_TIMEOUT, "a kernel's bounded wait expired (word 0x%x)", v);
  }
  return WQP_OK;
}

const char* wqp_status_string(int status) {
  switch (status) {
    case WQP_OK: return "WQP_OK";
    case WQP_ERR_INVALID_ARG: return "WQP_ERR_INVALID_ARG";
    case WQP_ERR_UNSUPPORTED: return "WQP_ERR_UNSUPPORTED";
    case WQP_ERR_CUDA: return "WQP_ERR_CUDA";
    case WQP_ERR_DEVICE_TIMEOUT: return "WQP_ERR_DEVICE_TIMEOUT";
  }
  return "WQP_ERR_UNKNOWN";
}

const char* wqp_last_error(void) { return t_last_error; }

int wqp_abi_version(void) { return WQP_ABI_VERSION; }

}  // extern "C"
