// The steps around the experts' products: routing, ordering the pairs by
// expert, and combining a token's rows.
//
// expert_route, per token, with logits l: s = softmax(l) or sigmoid(l),
// choice c = s + bias (l itself without a bias: the same order). Of groups of
// experts the ones with the largest sums of their best choices stay; of their
// experts the top_k largest choices are taken, equal ones by the lower index.
// weight = s, divided by the sum of those taken, times scale.
#include <cuda_fp16.h>

#include "decode.cuh"
#include "tc.cuh"

namespace wqp {
namespace {

using tc::cluster_rank;
using tc::cluster_sync;
using tc::mapa_shared;

constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// ------------------------------------------------------------ routing
struct RouteParams {
  const void* X;
  const float* bias;
  int* ids;
  float* weights;
  int T, E, ldl, top_k;
  int sigmoid, renormalise;
  int groups, top_groups, group_best;
  float scale;
};

// Keys that order as the numbers do; 0 is below every number's but -inf's and
// NaN's, which are not candidates.
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);            // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double c) {
  const unsigned long long b = __double_as_longlong(c + 0.0);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ double value_of(unsigned long long k) {
  return __longlong_as_double(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(kAll, v, o);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Whether the experts' order needs scores, and their groups' the choices.
__device__ __forceinline__ bool by_scores(const RouteParams& p) { return p.bias || (p.groups > 1 && p.group_best == 2); }
__device__ __forceinline__ bool group_by_choice(const RouteParams& p) { return p.bias || p.group_best == 1; }

// One token in one warp, in FP64: its experts, slot `lane`'s in the result, or -1.
// For tokens without NaN whose order needs scores and is too close for FP32; loops
// over shared memory (key [E]).
template <class T>
__device__ __noinline__ int route_exact(const RouteParams& p, const T* x, int lane, unsigned long long* key) {
  const double none = __longlong_as_double(0xFFF0000000000000ll);
  double top = none, inv = 1.0;
  if (!p.sigmoid) {
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32) top = fmax(top, static_cast<double>(to_f32(x[i])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
  }
  const auto power = [&](int i) {              // of a sigmoid e^-l, of a softmax e^(l - top): -inf gives inf and 0
    const double l = to_f32(x[i]);
    return exp(p.sigmoid ? -l : l - top);
  };
  const auto score = [&](int i) {
    const double e = power(i);
    return p.sigmoid ? 1.0 / (1.0 + e) : e * inv;
  };
  if (!p.sigmoid) {
    double sum = 0.0;
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32) sum += power(i);
    inv = 1.0 / warp_add(sum);
  }
  __syncwarp();
  const int size = p.E / p.groups;
  const bool from_choice = group_by_choice(p);
#pragma unroll 4
  for (int i = lane; i < p.E; i += 32) {
    const double l = to_f32(x[i]), s = score(i), c = p.bias ? s + p.bias[i] : l;
    key[i] = l > none && c > none ? key_of(from_choice ? c : s) : 0;
  }
  __syncwarp();
  unsigned long long mine = 0;                 // of group `lane`: its score's key
#pragma unroll 1
  for (int g = 0; g < p.groups; ++g) {
    unsigned long long k1 = 0, k2 = 0;
#pragma unroll 1
    for (int j = lane; j < size; j += 32) {
      const unsigned long long k = key[g * size + j];
      k2 = max(k2, min(k, k1));
      k1 = max(k1, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long u1 = __shfl_xor_sync(kAll, k1, o), u2 = __shfl_xor_sync(kAll, k2, o);
      k2 = max(max(k2, u2), min(k1, u1));
      k1 = max(k1, u1);
    }
    if (lane == g) mine = k2 && p.group_best == 2 ? key_of(value_of(k1) + value_of(k2)) : k1;
  }
  int better = 0;
#pragma unroll 1
  for (int h = 0; h < p.groups; ++h) {
    const unsigned long long k = __shfl_sync(kAll, mine, h);
    better += k > mine || (k == mine && h < lane);
  }
  const unsigned keep = __ballot_sync(kAll, better < p.top_groups);
  if (!from_choice)                            // the choices are the logits
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32)
      if (key[i]) key[i] = key_of(static_cast<double>(to_f32(x[i])));
  __syncwarp();
  int id = -1;
#pragma unroll 1
  for (int k = 0; k < p.top_k; ++k) {
    unsigned long long best = 0;
    int at = 0x7FFFFFFF;
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32)
      if (key[i] > best && (keep >> (i / size) & 1)) best = key[i], at = i;
    const unsigned long long m = warp_max(best);
    if (!m) break;
    const int i = __reduce_min_sync(kAll, best == m ? at : 0x7FFFFFFF);
    if (lane == k) id = i;
    if (at == i) key[i] = 0;
    __syncwarp();
  }
  return id;
}

constexpr float kNone = -INFINITY;

// A token's logits; expert i is element i / 32 of lane i % 32.
template <int NV>
struct Logits {
  float l[NV];                                             // -inf behind the last
  float top;
  bool odd;                                                // NaN, or an infinite exponential
};

// One token in one warp, in FP32; `part` is the warp's [E] scratch. Returns
// false where two choices that matter lie closer than the arithmetic's error and
// it takes more than the experts found to tell: route_exact's is then the answer. (One
// token in thousands with sigmoids and a bias; never without a bias and without
// groups, where the logits themselves are the keys.) id: as route_exact's.
template <class T, int NV>
__device__ __forceinline__ bool route_token(const RouteParams& p, const T* x, int lane, float* part, Logits<NV>& logits, int& id) {
  float (&l)[NV] = logits.l;
  bool odd = false;
  float top = kNone;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 32 * j;
    l[j] = i < p.E ? to_f32(x[i]) : kNone;
    odd |= l[j] != l[j] || (!p.sigmoid && l[j] == __int_as_float(0x7F800000));
    top = fmaxf(top, l[j]);
  }
  logits.odd = odd = __any_sync(kAll, odd);
  logits.top = top = value_of(warp_max(key_of(top)));

  // Scores where the order needs them.
  const bool by_score = !odd && by_scores(p);
  float inv = 1.0f;                                           // of the exponentials' sum
  if (!p.sigmoid && by_score) {
    float e = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) e += __expf(l[j] - top);   // -inf gives 0
    inv = 1.0f / warp_sum(e);
  }
  const auto score = [&](float v) {
    if (p.sigmoid) return __fdividef(1.0f, 1.0f + __expf(-v));
    return __expf(v - top) * inv;
  };
  uint32_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 32 * j;
    float c = l[j];
    if (by_score && p.bias && i < p.E) c = score(l[j]) + p.bias[i];
    key[j] = l[j] > kNone && c > kNone ? key_of(c) : 0u;
  }
  // The error of a choice c is at most 2^-24 (64 s_max + |c|): of a sigmoid s,
  // whose exponential is off by 4 + 3 |l| of these units, s (1 - s) times that and
  // 3 s more, under 8; of a softmax, whose sum has up to 37 roundings on any path,
  // at most 64 of its largest score. Two that are closer than twice that may
  // have changed places.
  const float s_max = p.sigmoid ? 0.125f : inv;
  const auto close = [&](float a, float b, float terms, float most) {
    return a - b <= 0x1p-23f * (64.0f * terms * s_max + most);
  };

  if (p.groups > 1 && !odd) {
    const int size = p.E / p.groups;
    const bool from_choice = group_by_choice(p);
    // Group g's two best, in the lanes from g << shift on.
    int shift = 0;
    float a = kNone, b = kNone;
    if (size == 32) {                                      // group j is element j of every lane
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j < p.groups) {
          const uint32_t k = from_choice || !key[j] ? key[j] : key_of(score(l[j]));
          const uint32_t k1 = warp_max(k);
          const int owner = __ffs(__ballot_sync(kAll, k == k1)) - 1;
          const uint32_t k2 = warp_max(lane == owner ? 0u : k);
          if (lane == j) {
            if (k1) a = value_of(k1);
            if (k2) b = value_of(k2);
          }
        }
    } else {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = lane + 32 * j;
        if (i < p.E) part[i] = !key[j] ? kNone : (from_choice ? value_of(key[j]) : score(l[j]));
      }
      __syncwarp();
      int log = 0;
      while ((1 << log) < p.groups) ++log;
      shift = 5 - log;
      const int lanes = 32 >> log, own = lane >> shift;
      if (own < p.groups)
        for (int i = lane & (lanes - 1); i < size; i += lanes) {
          const float v = part[own * size + i];
          const float lo = v < a ? v : a;
          a = v < a ? a : v;
          b = b < lo ? lo : b;
        }
      for (int o = 1; o < lanes; o <<= 1) {
        const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        const float lo = a < a2 ? a : a2, hi = b > b2 ? b : b2;
        a = a > a2 ? a : a2;
        b = lo > hi ? lo : hi;
      }
    }
    const int g = lane >> shift;
    const bool pair = p.group_best == 2 && b > kNone;
    const float mine = pair ? a + b : a;
    // A group stays where fewer than top_groups are better.
    int better = 0;
    for (int h = 0; h < p.groups; ++h) {
      const float v = __shfl_sync(kAll, mine, h << shift);
      better += v > mine || (v == mine && h < g);
    }
    const bool stays = g < p.groups && better < p.top_groups;
    unsigned keep = __ballot_sync(kAll, stays);
    if (p.top_groups < p.groups && by_score) {
      const auto magnitude = [](float v) { return v > -3e38f && v < 3e38f ? fabs(v) : 0.0f; };
      const uint32_t least = ~warp_max(static_cast<uint32_t>(stays ? ~key_of(mine) : 0u));
      const uint32_t above = warp_max(!stays && g < p.groups ? key_of(mine) : 0u);
      const float most = value_of(warp_max(key_of(magnitude(a) + (pair ? magnitude(b) : 0.0f))));
      if (above && close(value_of(least), value_of(above), 2.0f, 2 * most)) {
        // Sigmoids: the groups again in FP64, from the experts that can be among a
        // group's best, a lane each (of a softmax that needs the whole sum).
        if (!p.sigmoid) return false;
        const float last = pair ? b : a, low = fabsf(last) < INFINITY ? last - 0x1p-23f * (64.0f * s_max + fabsf(last)) : last;
        int* const cand = reinterpret_cast<int*>(part);
        int n = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int i = lane + 32 * j, of = min(i, p.E - 1) / size;
          const float least_in = __shfl_sync(kAll, low, of << shift);
          const bool in = key[j] && (from_choice ? value_of(key[j]) : score(l[j])) >= least_in;
          const unsigned who = __ballot_sync(kAll, in);
          const int to = n + __popc(who & ((1u << lane) - 1));
          if (in && to < 32) cand[to] = i;
          n += __popc(who);
        }
        __syncwarp();
        if (n > 32) return false;
        unsigned long long mine64 = 0;
        int of = -1;
        if (lane < n) {
          const int i = cand[lane];
          const double v = 1.0 / (1.0 + exp(-static_cast<double>(to_f32(x[i])))) + (from_choice ? p.bias[i] : 0.0f);
          mine64 = key_of(v);
          of = i / size;
        }
        __syncwarp();
        unsigned long long k1 = 0, k2 = 0;     // the two best of group `lane`
        for (int j = 0; j < n; ++j) {
          const unsigned long long k = __shfl_sync(kAll, mine64, j);
          if (__shfl_sync(kAll, of, j) != lane) continue;
          k2 = max(k2, min(k, k1));
          k1 = max(k1, k);
        }
        if (k2 && p.group_best == 2) k1 = key_of(value_of(k1) + value_of(k2));
        int above64 = 0;
        for (int h = 0; h < p.groups; ++h) {
          const unsigned long long k = __shfl_sync(kAll, k1, h);
          above64 += k > k1 || (k == k1 && h < lane);
        }
        const unsigned stay64 = __ballot_sync(kAll, lane < p.groups && above64 < p.top_groups);
        keep = __ballot_sync(kAll, stay64 >> g & 1);
      }
    }
    if (size == 32) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (!(keep >> j & 1)) key[j] = 0;
    } else {
      const float per = 1.0f / static_cast<float>(size);   // i / size, for i < 1024, from (i + 1/2) / size
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = lane + 32 * j, of = static_cast<int>((static_cast<float>(i) + 0.5f) * per);
        if (!(keep >> (of << shift & 31) & 1)) key[j] = 0;
      }
    }
  }

  // The best key of a lane's own, of equal ones the lowest index.
  uint32_t best;
  int at;                                                  // its index
  const auto own_best = [&] {
    best = key[0];
    at = lane;
#pragma unroll
    for (int j = 1; j < NV; ++j)
      if (key[j] > best) best = key[j], at = 32 * j + lane;
  };
  own_best();
  id = -1;                                                 // of slot `lane`
  const bool check = p.bias && !odd;
  bool sorted = false;
  if (p.top_k < 32) {
    // Only keys of at least the (top_k + 1)-th largest of the lanes' best can be
    // among the top_k + 1: a few more than that, mostly. They are collected and
    // ranked, a lane each.
    uint32_t v = best;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
      for (int o = size >> 1; o > 0; o >>= 1) {
        const uint32_t u = __shfl_xor_sync(kAll, v, o);
        const bool up = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
        v = up == (u > v) ? u : v;
      }
    const uint32_t least = max(__shfl_sync(kAll, v, p.top_k), 1u);
    uint32_t* const cand = reinterpret_cast<uint32_t*>(part);   // keys, indexes, and again in order
    int n = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = key[j] >= least;
      const unsigned who = __ballot_sync(kAll, in);
      const int to = n + __popc(who & ((1u << lane) - 1));
      if (in && to < 32) {
        cand[to] = static_cast<uint32_t>(key[j]);
        cand[32 + to] = 32 * j + lane;
      }
      n += __popc(who);
    }
    __syncwarp();
    if (n <= 32) {
      const uint32_t k = lane < n ? cand[lane] : 0;
      int place = 0;                                       // in rising order of the index
      for (int j = 0; j < n; ++j) {
        const uint32_t u = __shfl_sync(kAll, k, j);
        place += u > k || (u == k && j < lane);
      }
      if (lane < n) {
        cand[64 + place] = k;
        cand[96 + place] = cand[32 + lane];
      }
      __syncwarp();
      const int last = min(n, p.top_k);
      bool near = false;
      if (check && lane < last && lane + 1 < n) {
        const float a = value_of(static_cast<uint32_t>(cand[64 + lane])), b = value_of(static_cast<uint32_t>(cand[64 + lane + 1]));
        near = close(a, b, 1.0f, fabs(a));
      }
      sorted = !__any_sync(kAll, near);
      if (sorted && lane < last) id = cand[96 + lane];
    }
  }
  // One after the other, where there are too many of equal keys, or some too
  // close to each other: the best of the lanes', top_k times; with choices that
  // FP32 rounds, on to the first that is clearly less.
  uint32_t prev = 0;
  int found = 0;
  bool unsure = false;
  for (; !sorted; ++found) {
    const uint32_t m = warp_max(best);
    if (!m || (!check && found == p.top_k)) break;
    if (check && found > 0) {
      const float a = value_of(prev), b = value_of(m);
      const bool near = close(a, b, 1.0f, fabs(a));
      if (!near && found >= p.top_k) break;
      unsure |= near;
    }
    if (found == 32) {
      if (unsure) return false;
      break;
    }
    const int i = __reduce_min_sync(kAll, best == m ? at : 0x7FFFFFFF);
    prev = m;
    if (lane == found) id = i;
    if (at == i) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (i == 32 * j + lane) key[j] = 0;
      own_best();
    }
  }
  if (unsure) {
    // The experts found so far hold the top_k for sure: their order by FP64
    // choices, a lane each (of a softmax those need the whole sum).
    if (!p.sigmoid) return false;
    double c = id >= 0 ? 1.0 / (1.0 + exp(-static_cast<double>(to_f32(x[id])))) + p.bias[id] : 0.0;
    int place = 0;
    for (int j = 0; j < found; ++j) {
      const double u = __shfl_sync(kAll, c, j);
      const int v = __shfl_sync(kAll, id, j);
      place += u > c || (u == c && v < id);
    }
    int at_place = -1;
    for (int j = 0; j < found; ++j) {
      const int u = __shfl_sync(kAll, place, j), v = __shfl_sync(kAll, id, j);
      if (u == lane) at_place = v;
    }
    id = at_place;
  }
  if (lane >= p.top_k) id = -1;
  return true;
}

// The weights of a token's experts, and both to memory.
template <class T, int NV>
__device__ __forceinline__ void route_write(const RouteParams& p, const T* x, int t, int lane, const Logits<NV>& logits, int id) {
  const bool live = id >= 0;
  const float lg = live ? to_f32(x[id]) : kNone;
  float w = 0.0f;
  if (p.renormalise || p.sigmoid) {
    // Renormalised: scores relative to the largest taken, so that they cannot all
    // vanish. A sigmoid is e^min(l, 0) / (1 + e^-|l|), where nothing overflows.
    const float most = p.renormalise ? value_of(warp_max(live ? key_of(lg) : 0u)) : 0.0f;
    if (live) w = p.sigmoid ? expf(fminf(lg, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(lg))) : expf(lg - most);
    if (p.renormalise) {
      const float total = warp_sum(w);
      w = total > 0.0f ? w / total : 0.0f;
    }
  } else {
    float e = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) e += logits.l[j] > kNone ? expf(logits.l[j] - logits.top) : 0.0f;
    e = warp_sum(e);
    if (live) w = expf(lg - logits.top) / e;
  }
  w *= p.scale;
  if (logits.odd) w = __int_as_float(0x7FFFFFFF);
  if (lane < p.top_k) {
    const long long o = static_cast<long long>(t) * p.top_k + lane;
    p.ids[o] = id;
    p.weights[o] = w;
  }
}

constexpr int kRouteWarps = 4;
// Doubles of a warp's scratch: the choices, or four times 32 words.
__host__ __device__ constexpr int route_scratch(int E) { return E > 64 ? E : 64; }

// Bound by the latency of one token's chain of steps, which warps overlap: its
// logits' loads, their maximum, an exponential an expert where the order needs
// scores, the groups' maxima and ranks, a sort of the lanes' best and the ranking of
// the candidates above it, the weights (issue slots 58 %, ALU 50 % at 8191x256). One
// expert after the other only where choices are equal or close, or top_k is 32.
// 8191x256, 8 groups: 16.4 us; 25 us where close groups send the whole token to
// route_exact, 8 of them for the last such token's FP64 steps. 8192x128, softmax: 7.5 us.
template <class T, int NV>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p) {
  extern __shared__ double route_part[];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= p.T) return;
  double* part = route_part + static_cast<size_t>(warp) * route_scratch(p.E);
  const T* x = static_cast<const T*>(p.X) + static_cast<long long>(t) * p.ldl;
  Logits<NV> logits;
  int id;
  if (!route_token<T, NV>(p, x, lane, reinterpret_cast<float*>(part), logits, id))
    id = route_exact(p, x, lane, reinterpret_cast<unsigned long long*>(part));
  route_write(p, x, t, lane, logits, id);
}

template <class T>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s) {
  const RouteParams p = {a.X, a.bias, a.ids, a.weights, a.T, a.E, a.ldl, a.top_k, a.sigmoid, a.renormalise,
                         a.groups, a.top_groups, a.group_best, a.scale};
  const dim3 grid((a.T + kRouteWarps - 1) / kRouteWarps), block(kRouteWarps * 32);
  const size_t smem = sizeof(double) * kRouteWarps * route_scratch(a.E);   // 32 KB at most: no opt-in
  if (a.E <= 64) return launch(route_kernel<T, 2>, grid, block, smem, s, a.pdl, p);
  if (a.E <= 128) return launch(route_kernel<T, 4>, grid, block, smem, s, a.pdl, p);
  if (a.E <= 256) return launch(route_kernel<T, 8>, grid, block, smem, s, a.pdl, p);
  if (a.E <= 512) return launch(route_kernel<T, 16>, grid, block, smem, s, a.pdl, p);
  return launch(route_kernel<T, 32>, grid, block, smem, s, a.pdl, p);
}

// ------------------------------------------------------------ ordering
// A counting sort that keeps the pairs' order: every warp counts the ids of
// its run of pairs, the counts of earlier warps (of earlier CTAs, through the
// cluster's shared memory) give each warp its place in each expert's list, and
// a second pass over the run puts the pairs there. One launch; the order of the
// counts' atomics does not show, so the result is the same every time.
constexpr int kOrderWarps = 32;

__global__ void __launch_bounds__(kOrderWarps * 32) order_kernel(const int* ids, int* rows, int* offsets, int R, int E, int run) {
  extern __shared__ int order_sh[];
  __shared__ int scan_sh[33];
  int* const count = order_sh;                             // [warps][E]: counts, then places
  int* const total = order_sh + kOrderWarps * E;           // [E]: this CTA's counts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ranks = gridDim.x, rank = ranks > 1 ? static_cast<int>(cluster_rank()) : 0;
  pdl_launch_dependents();
  pdl_wait();
  const long long first = static_cast<long long>(rank * kOrderWarps + warp) * run;
  const int begin = static_cast<int>(first < R ? first : R), end = static_cast<int>(first + run < R ? first + run : R);
  int* const mine = count + warp * E;
  const auto id_at = [&](int i) {
    const int e = i < end ? ids[i] : -1;
    return static_cast<unsigned>(e) < static_cast<unsigned>(E) ? e : -1;
  };
  // The first eight batches of a run stay in registers for the second pass.
  constexpr int kKept = 8;
  int kept[kKept];
#pragma unroll
  for (int b = 0; b < kKept; ++b) kept[b] = id_at(begin + 32 * b + lane);
  for (int i = lane; i < E; i += 32) mine[i] = 0;
  __syncwarp();
#pragma unroll
  for (int b = 0; b < kKept; ++b)
    if (kept[b] >= 0) atomicAdd(mine + kept[b], 1);
  for (int i = begin + 32 * kKept; i < end; i += 32) {
    const int e = id_at(i + lane);
    if (e >= 0) atomicAdd(mine + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kOrderWarps; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  // Thread e: expert e's counts of every CTA, and where its list starts.
  const int e = threadIdx.x;
  int all = 0, before = 0;
  if (e < E) {
    if (ranks > 1) {
      const uint32_t at = smem_u32(total + e);
      for (int r = 0; r < ranks; ++r) {
        int c;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(mapa_shared(at, r)) : "memory");
        before += r < rank ? c : 0;
        all += c;
      }
    } else {
      all = total[e];
    }
  }
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) scan_sh[warp] = incl;
  // No CTA reads another's shared memory after this, nor ends before it.
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  if (warp == 0) {
    int v = scan_sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += u;
    }
    scan_sh[lane] = v;
  }
  __syncthreads();
  const int start = incl - all + (warp ? scan_sh[warp - 1] : 0);
  const int live = scan_sh[31];
  if (e < E) {
    total[e] = start + before;
    if (rank == 0) {
      offsets[e] = start;
      if (e == E - 1) offsets[E] = live;
    }
  }
  __syncthreads();
  // Lanes of one id from a vote on each of its bits (a match of whole values
  // took 32 of the kernel's first 39 thousand clocks at 65536 pairs of 256).
  const int bits = 32 - __clz(E);
  const auto place_batch = [&](int i, int e) {
    unsigned same = kAll;
    for (int b = 0; b < bits; ++b) {
      const bool on = (e + 1) >> b & 1;
      const unsigned vote = __ballot_sync(kAll, on);
      same &= on ? vote : ~vote;
    }
    int at = 0;
    if (e >= 0) at = mine[e];
    __syncwarp();
    if (e >= 0) {
      rows[total[e] + at + __popc(same & ((1u << lane) - 1))] = i;
      if (lane == __ffs(same) - 1) mine[e] = at + __popc(same);
    }
    __syncwarp();
  };
#pragma unroll
  for (int b = 0; b < kKept; ++b)
    if (begin + 32 * b < end) place_batch(begin + 32 * b + lane, kept[b]);
  for (int i = begin + 32 * kKept; i < end; i += 32) place_batch(i + lane, id_at(i + lane));
  for (long long i = live + static_cast<long long>(rank) * blockDim.x + threadIdx.x; i < R; i += static_cast<long long>(ranks) * blockDim.x)
    rows[i] = -1;
}

// ------------------------------------------------------------ combining
// Bound by memory: every row of Y is read once. A thread has one piece of a
// token, the loads of eight slots in flight at a time, and adds in FP32 in the
// slots' order, the residual last. A piece is 32 bytes where the rows allow it
// (8192x8x5120 with the residual, BF16: 128 us, 6.6 TB/s), else 16 (145 us; 156 with
// outputs stored to stay in L2).
template <int W>
struct Piece {                                             // W words
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (W == 8) {
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p));
    } else {
      const uint4 v = ld_act_v4(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (W == 8) {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                   "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {
      __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
};
// A word's elements, and back.
__device__ __forceinline__ void add_word(float* v, uint32_t x, float w, __nv_bfloat16) {
  v[0] += w * bf16lo(x);
  v[1] += w * bf16hi(x);
}
__device__ __forceinline__ void add_word(float* v, uint32_t x, float w, __half) {
  const float2 f = f16x2_to_float2(x);
  v[0] += w * f.x;
  v[1] += w * f.y;
}
__device__ __forceinline__ void add_word(float* v, uint32_t x, float w, float) { v[0] += w * __uint_as_float(x); }
__device__ __forceinline__ uint32_t to_word(const float* v, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t to_word(const float* v, __half) {
  const __half2 h = __floats2half2_rn(v[0], v[1]);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t to_word(const float* v, float) { return __float_as_uint(v[0]); }

constexpr int kCombineThreads = 64;

template <class T, int W>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineArgs a, int pieces) {
  constexpr int E = 4 / sizeof(T), N = W * E;              // elements of a word and of a piece
  pdl_launch_dependents();
  pdl_wait();
  const long long c = static_cast<long long>(blockIdx.x) * kCombineThreads + threadIdx.x;
  const long long t = c / pieces;
  if (t >= a.T) return;
  const int col = static_cast<int>(c - t * pieces) * N;
  const T* y = static_cast<const T*>(a.Y) + t * a.slots * a.ldy + col;
  const int* ids = a.ids + t * a.slots;
  const float* weights = a.weights + t * a.slots;
  Piece<W> r;
  if (a.R) r.load(static_cast<const T*>(a.R) + t * a.ldr + col);
  float v[N] = {};
  const auto add = [&](const Piece<W>& x, float w) {
#pragma unroll
    for (int i = 0; i < W; ++i) add_word(v + E * i, x.w[i], w, T());
  };
  constexpr int U = 8;
  for (int s0 = 0; s0 < a.slots; s0 += U) {
    Piece<W> x[U];
    float w[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      on[u] = s0 + u < a.slots && static_cast<unsigned>(ids[s0 + u]) < static_cast<unsigned>(a.E);
      if (on[u]) {
        x[u].load(y + static_cast<long long>(s0 + u) * a.ldy);
        w[u] = weights[s0 + u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on[u]) add(x[u], w[u]);
  }
  if (a.R) add(r, 1.0f);
#pragma unroll
  for (int i = 0; i < W; ++i) r.w[i] = to_word(v + E * i, T());
  r.store(static_cast<T*>(a.out) + t * a.ldo + col);
}

template <class T, int W>
cudaError_t launch_combine_tw(const CombineArgs& a, cudaStream_t s) {
  const int pieces = a.H / (W * 4 / static_cast<int>(sizeof(T)));
  const long long blocks = (static_cast<long long>(a.T) * pieces + kCombineThreads - 1) / kCombineThreads;
  return launch(combine_kernel<T, W>, dim3(static_cast<unsigned>(blocks)), dim3(kCombineThreads), 0, s, a.pdl, a, pieces);
}
template <class T>
cudaError_t launch_combine_t(const CombineArgs& a, cudaStream_t s) {
  const auto wide = [](const void* p, int ld) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && static_cast<size_t>(ld) * sizeof(T) % 32 == 0;
  };
  const bool all = wide(a.Y, a.ldy) && wide(a.out, a.ldo) && (!a.R || wide(a.R, a.ldr)) && wide(nullptr, a.H);
  return all ? launch_combine_tw<T, 8>(a, s) : launch_combine_tw<T, 4>(a, s);
}

}  // namespace

cudaError_t launch_expert_route(const RouteArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_route_t<__nv_bfloat16>(a, s);
  if (a.dtype == 1) return launch_route_t<__half>(a, s);
  return launch_route_t<float>(a, s);
}

// One CTA up to 2048 pairs, else a cluster of eight.
cudaError_t launch_expert_order(const OrderArgs& a, cudaStream_t s) {
  constexpr int kOne = 2048, kCluster = 8;
  const int ranks = a.R <= kOne ? 1 : kCluster;
  const long long warps = static_cast<long long>(ranks) * kOrderWarps;
  const int run = static_cast<int>((a.R + warps * 32 - 1) / (warps * 32) * 32);
  const size_t smem = sizeof(int) * (kOrderWarps + 1) * a.E;
  static AttrLatch latch;
  const cudaError_t e = set_smem_attrs(order_kernel, latch, static_cast<int>(sizeof(int)) * (kOrderWarps + 1) * kMaxExperts, false);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kOrderWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, order_kernel, a.ids, a.rows, a.offsets, a.R, a.E, run);
}

cudaError_t launch_expert_combine(const CombineArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_combine_t<__nv_bfloat16>(a, s);
  if (a.dtype == 1) return launch_combine_t<__half>(a, s);
  return launch_combine_t<float>(a, s);
}

}  // namespace wqp
