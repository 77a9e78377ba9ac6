// The choice of experts from router logits, and the gradient of the logits from the weights':
//
//   score s_e = softmax(l)_e or sigmoid(l_e);  value v_e = s_e + b_e
//   groups of E / G neighbouring experts: the top_groups groups with the largest sums of their `best` largest values
//   the k experts of these groups with the largest values (without b by the logits, which have the
//   scores' order), ties to the lower number;  w_i = scale s_i, or scale s_i / sum_j s_j
//
// An expert whose logit or bias is -inf or NaN is off: it has no score and is never chosen.  Places that no expert
// is left for get expert -1 and weight 0.
//
// The order has to be that of the values themselves, which fp32 scores do not always tell apart: a wave that finds
// two values it has to order (or two groups at the border) closer than fp32's errors takes its token again in 64
// bits.  Weights need no such care.  They are computed relative to the largest chosen score, so that
// scores too small for fp32 still share their token.
#include <cmath>

#include "block.h"
#include "moe_vq_device.h"

namespace mvq {

namespace {

constexpr int CHOOSE_THREADS = 256;  // a token per wave

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_total(float v) { return wave_sum(v); }
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// A token's scores over a wave: expert e = lane + 64 i in entry i.
template <typename T, int NPL>
__device__ __forceinline__ void scores(const ChooseArgs& a, const float* l, T* s, T& total, float top) {
  T sum = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (a.sigmoid) {
      s[i] = T(1) / (T(1) + exp_of(-T(l[i])));
    } else {
      // (an infinite logit takes everything, several share it)
      s[i] = l[i] == -INFINITY ? T(0) : (l[i] == top ? T(1) : exp_of(T(l[i]) - T(top)));
      sum += s[i];
    }
  }
  if (!a.sigmoid) {
    total = wave_total(sum);
    const T inv = total > 0 ? T(1) / total : T(0);
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = sizeof(T) == 8 ? (total > 0 ? s[i] / total : T(0)) : s[i] * inv;
  }
}

// The expert with the largest of v over the wave (the lowest of equal ones), or -1 if all are -inf; its entry is
// set to -inf, and its logit goes to *at.
template <typename T, int NPL>
__device__ __forceinline__ int take_best(T* v, const float* l, int lane, T& best, float* at = nullptr) {
  best = v[0];
#pragma unroll
  for (int i = 1; i < NPL; ++i) best = v[i] > best ? v[i] : best;
  best = wave_max(best);
  if (best == T(-INFINITY)) return -1;
  int id = -1;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const uint64_t m = __ballot(v[i] == best);
    if (id < 0 && m) {
      const int from = __builtin_ctzll(m);
      id = 64 * i + from;
      if (at) *at = lane_f32(l[i], from);
      if (lane == from) v[i] = T(-INFINITY);
    }
  }
  return id;
}

// The k experts in order: place j's in lane j (-1: none) with its logit.  Returns whether T tells them apart.
template <typename T, int NPL>
__device__ __forceinline__ bool choose(const ChooseArgs& a, const float* l, const float* b, int lane, float top, float b_most,
                                       int& my_id, float& my_l, T& total) {
  constexpr bool SINGLE = sizeof(T) == 4;
  const T NONE = T(-INFINITY);
  T rank[NPL];
  T near = 0;  // how close two values may be for T to order them
  const bool groups = a.top_groups < a.groups;
  if (a.bias || groups || !(a.renorm || a.sigmoid)) {
    scores<T, NPL>(a, l, rank, total, top);
    if (SINGLE) {
      // fp32: a score is within 2^-21 of the largest, its sum with b within 2^-24 of itself
      float most = rank[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) most = fmaxf(most, rank[i]);
      near = ldexpf(wave_max(most) + b_most, -19);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const T v = a.bias ? rank[i] + T(b[i]) : rank[i];
      rank[i] = l[i] == -INFINITY ? NONE : v;
    }
  }
  bool sure = true;
  uint64_t taken = ~0ull;  // groups, 64 of them at most
  if (groups) {
    const int size = a.E / a.groups;
    T mine = NONE;  // lane g: the value of group g
    for (int g = 0; g < a.groups; ++g) {
      T v[NPL], sum = 0, best;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 64 * i;
        v[i] = e >= g * size && e < (g + 1) * size ? rank[i] : NONE;
      }
      bool any = false;
      for (int j = 0; j < a.best; ++j) {
        if (take_best<T, NPL>(v, l, lane, best) < 0) break;
        sum += best;
        any = true;
      }
      if (lane == g) mine = any ? sum : NONE;
    }
    taken = 0;
    T v[1] = {mine}, last = 0, best;
    for (int j = 0; j <= a.top_groups; ++j) {
      const int g = take_best<T, 1>(v, l, lane, best);
      if (g < 0) break;
      if (j == a.top_groups) sure = sure && !(SINGLE && last - best <= 2 * near);  // (groups' values are sums of two)
      else taken |= 1ull << g;
      last = best;
    }
  }
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) rank[i] = T(l[i]);
  }
  if (groups) {
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < NPL; ++i) rank[i] = (taken >> ((lane + 64 * i) / size)) & 1 ? rank[i] : NONE;
  }
  my_id = -1;
  my_l = -INFINITY;
  T last = 0;
  for (int j = 0; j < a.k + (SINGLE && a.bias ? 1 : 0); ++j) {
    T best;
    float at = 0.f;
    const int id = take_best<T, NPL>(rank, l, lane, best, &at);
    if (id < 0) break;
    if (SINGLE && a.bias && j > 0 && last - best <= near) sure = false;
    last = best;
    if (lane == j && j < a.k) { my_id = id; my_l = at; }
  }
  return sure;
}

// log sigmoid(l)
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// The weights of the chosen experts, place j's in lane j: score (of the sums' share, or alone).
__device__ __forceinline__ float weight_of(const ChooseArgs& a, bool chosen, float l, float top, float total) {
  if (!a.renorm) {
    if (!chosen) return 0.f;
    if (a.sigmoid) return 1.0f / (1.0f + expf(-l));
    return (l == top ? 1.f : expf(l - top)) / total;
  }
  const float s = !chosen ? -INFINITY : (a.sigmoid ? log_sigmoid(l) : l);
  const float most = wave_max(s);
  const float p = !chosen ? 0.f : (s == most ? 1.f : expf(s - most));
  const float sum = wave_sum(p);
  return chosen ? p / sum : 0.f;
}

// The token's logits (-inf where an expert is off), the biases and the largest of both.
template <int NPL>
__device__ __forceinline__ float load_logits(const ChooseArgs& a, int t, int lane, float* l, float* b, float& b_most) {
  float top = -INFINITY;
  b_most = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < a.E ? a.logits[(size_t)t * a.E + e] : -INFINITY;
    b[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (!(l[i] > -INFINITY) || !(b[i] > -INFINITY)) l[i] = -INFINITY;  // off (NaN too)
    top = fmaxf(top, l[i]);
    b_most = fmaxf(b_most, fabsf(b[i]));
  }
  if (a.bias) b_most = wave_max(b_most);
  return wave_max(top);
}

template <int NPL>
__global__ __launch_bounds__(CHOOSE_THREADS) void choose_kernel(ChooseArgs a) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * (CHOOSE_THREADS / 64) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  float l[NPL], b[NPL], b_most;
  const float top = load_logits<NPL>(a, t, lane, l, b, b_most);
  int id;
  float at, total = 1.f;
  if (!choose<float, NPL>(a, l, b, lane, top, b_most, id, at, total)) {
    double wide;
    choose<double, NPL>(a, l, b, lane, top, b_most, id, at, wide);
  }
  const float w = weight_of(a, id >= 0, at, top, total);
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = id;
    a.w[(size_t)t * a.k + lane] = id >= 0 ? a.scale * w : 0.f;
  }
}

// With p_i the chosen experts' shares (renormalised: w_i / scale) or scores:
//   d log p_i = p_i (dw_i - sum_j p_j dw_j) scale, or p_i dw_i scale;   sigmoid: d l_i = d log p_i (1 - s_i);
//   softmax: d l_e = sum of e's places, without renormalisation less s_e sum_j d log p_j.
// An expert that occurs twice gets both places' parts.
template <int NPL>
__global__ __launch_bounds__(CHOOSE_THREADS) void choose_back_kernel(ChooseArgs a) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * (CHOOSE_THREADS / 64) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const bool spread = !a.sigmoid && !a.renorm;  // every logit has a part
  const size_t at = (size_t)t * a.k + lane;
  int id = lane < a.k ? a.ids[at] : -1;
  float dw = lane < a.k ? a.w[at] * a.scale : 0.f;
  float l = (uint32_t)id < (uint32_t)a.E ? a.logits[(size_t)t * a.E + id] : -INFINITY;
  const bool chosen = l > -INFINITY;
  if (!chosen) { id = -1; dw = 0.f; }
  float s[NPL], top = 0.f, total = 1.f, b_most;
  if (spread) {
    float row[NPL], b[NPL];
    top = load_logits<NPL>(a, t, lane, row, b, b_most);
    scores<float, NPL>(a, row, s, total, top);
  }
  const float p = weight_of(a, chosen, l, top, total);
  float part = a.renorm ? p * (dw - wave_sum(p * dw)) : p * dw;
  if (a.sigmoid) part *= 1.0f / (1.0f + expf(l));
  if (!chosen) part = 0.f;
  const float pull = spread ? wave_sum(part) : 0.f;
  float out[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) out[i] = spread ? -s[i] * pull : 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float v = lane_f32(part, j);
#pragma unroll
    for (int i = 0; i < NPL; ++i) out[i] += e == lane + 64 * i ? v : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (lane + 64 * i < a.E) a.dlogits[(size_t)t * a.E + lane + 64 * i] = out[i];
}

template <typename F>
void by_width(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_choose(const ChooseArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.T + CHOOSE_THREADS / 64 - 1) / (CHOOSE_THREADS / 64));
  by_width(a.E, [&](auto n) { choose_kernel<decltype(n)::value><<<grid, CHOOSE_THREADS, 0, st>>>(a); });
  return hipGetLastError();
}

hipError_t launch_choose_back(const ChooseArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.T + CHOOSE_THREADS / 64 - 1) / (CHOOSE_THREADS / 64));
  by_width(a.E, [&](auto n) { choose_back_kernel<decltype(n)::value><<<grid, CHOOSE_THREADS, 0, st>>>(a); });
  return hipGetLastError();
}

}  // namespace mvq
