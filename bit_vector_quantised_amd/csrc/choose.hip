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
// The order has to be that of the values themselves, which fp32 scores do not always tell apart: a token with two values
// to be ordered (or two groups at the border) closer than fp32's errors is taken again in 64 bits.
// Weights need no such care.  They are computed relative to the largest chosen score, so that
// scores too small for fp32 still share their token.
#include <cmath>

#include "block.h"
#include "moe_vq_device.h"

namespace mvq {

namespace {

constexpr int CHOOSE_THREADS = 256, CHOOSE_WAVES = CHOOSE_THREADS / 64;

// ---------------------------------------------------------------------------------------
// A token by L lanes (16, or the wave)
// ---------------------------------------------------------------------------------------

template <int L>
__device__ __forceinline__ float max_of(float v) {
  v = fmaxf(v, dpp_f32<dpp::QUAD_XOR1>(v));
  v = fmaxf(v, dpp_f32<dpp::QUAD_XOR2>(v));
  v = fmaxf(v, dpp_f32<dpp::ROW_HALF_MIRROR>(v));
  v = fmaxf(v, dpp_f32<dpp::ROW_MIRROR>(v));
  if (L == 64) v = fmaxf(fmaxf(lane_f32(v, 0), lane_f32(v, 16)), fmaxf(lane_f32(v, 32), lane_f32(v, 48)));
  return v;
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
  const uint32_t o = (uint32_t)dpp_i32<CTRL>((int)v);
  return o > v ? o : v;
}
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  v = max_with<dpp::QUAD_XOR1>(v);
  v = max_with<dpp::QUAD_XOR2>(v);
  v = max_with<dpp::ROW_HALF_MIRROR>(v);
  v = max_with<dpp::ROW_MIRROR>(v);
  if (L == 64) {
    const uint32_t r0 = __builtin_amdgcn_readlane((int)v, 0), r1 = __builtin_amdgcn_readlane((int)v, 16),
                   r2 = __builtin_amdgcn_readlane((int)v, 32), r3 = __builtin_amdgcn_readlane((int)v, 48);
    const uint32_t a = r0 > r1 ? r0 : r1, b = r2 > r3 ? r2 : r3;
    v = a > b ? a : b;
  }
  return v;
}

// The weights of the chosen experts, place j's in lane j of L: score (of the sums' share, or alone).
template <int L>
__device__ __forceinline__ float weight_of(const ChooseArgs& a, bool chosen, float l, float top, float total) {
  if (!a.renorm) {
    if (!chosen) return 0.f;
    if (a.sigmoid) return 1.0f / (1.0f + expf(-l));
    return (l == top ? 1.f : expf(l - top)) / total;
  }
  // relative to the largest chosen score: exp(l - most), for sigmoid over 1 + exp(l) if that is at most 2
  const float first = max_of<L>(chosen ? l : -INFINITY), most = a.sigmoid ? fminf(first, 0.f) : first;
  float p = l == most ? 1.f : __expf(l - most);
  if (a.sigmoid) p = (l < 0.f ? p : 1.f) * __builtin_amdgcn_rcpf(1.0f + __expf(-fabsf(l)));
  if (!chosen) p = 0.f;
  const float sum = group_sum<L>(p);
  return chosen ? p / sum : 0.f;
}

// The expert of entry i of lane j: four neighbours per lane and 16-byte load.
template <int L>
__device__ __forceinline__ int expert_of(int i, int j) { return (i >> 2) * (L * 4) + j * 4 + (i & 3); }

// (no branch around a load, so that all of them go out at once: entries without an expert repeat the first)
template <int L, int N>
__device__ __forceinline__ void load_row(const float* row, int E, int j, float* v) {
  if (E % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int e = expert_of<L>(i, j);
      const f32x4_any u = *reinterpret_cast<const f32x4_any*>(row + (e < E ? e : 0));
      v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert_of<L>(i, j);
      v[i] = row[e < E ? e : 0];
    }
  }
}
// A token's logits (-inf where an expert is off) and the biases.
template <int L, int N>
__device__ __forceinline__ void load_token(const ChooseArgs& a, int t, int j, float* l, float* b) {
  load_row<L, N>(a.logits + (size_t)t * a.E, a.E, j, l);
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = 0.f;
  if (a.bias) load_row<L, N>(a.bias, a.E, j, b);
#pragma unroll
  for (int i = 0; i < N; ++i)
    l[i] = expert_of<L>(i, j) < a.E && l[i] > -INFINITY && b[i] > -INFINITY ? l[i] : -INFINITY;  // (NaN too)
}
// Scores, for softmax also the sum of exp(l - top).  exp and 1/x by the hardware: an error of |x| 2^-24 of
// the exponential beside a few roundings.
template <int L, int N>
__device__ __forceinline__ void scores(const ChooseArgs& a, const float* l, float top, float* s, float& total) {
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
    return;
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // (an infinite logit takes everything, several share it)
    s[i] = l[i] == -INFINITY ? 0.f : (l[i] == top ? 1.f : __expf(l[i] - top));
    sum += s[i];
  }
  total = group_sum<L>(sum);
  const float inv = total > 0.f ? 1.0f / total : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] *= inv;
}

constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// LDS as the wave's own: its accesses complete in order, the fences keep the compiler to it.
__device__ __forceinline__ void lds_turn() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The two largest of this lane's two and another lane's.
template <int CTRL>
__device__ __forceinline__ void two_best(float& m1, float& m2) {
  const float o1 = dpp_f32<CTRL>(m1), o2 = dpp_f32<CTRL>(m2);
  m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
  m1 = fmaxf(m1, o1);
}

template <int I, int J>
__device__ __forceinline__ void order_two(uint32_t* k) {  // the larger first
  const uint32_t x = k[I], y = k[J];
  k[I] = x > y ? x : y;
  k[J] = x > y ? y : x;
}
// N words, the largest first (Batcher's merge exchange network over powers of two).
template <int N>
__device__ __forceinline__ void order_all(uint32_t* k) {
  static_for<0, log2_of(N)>([&](auto pp) {
    constexpr int P = 1 << decltype(pp)::value;
    static_for<0, decltype(pp)::value + 1>([&](auto qq) {
      constexpr int K = P >> decltype(qq)::value;
      static_for<0, N>([&](auto ii) {
        constexpr int I = decltype(ii)::value, J0 = K % P;
        if constexpr (I >= J0 && (I - J0) % (2 * K) < K && I + K < N && I / (2 * P) == (I + K) / (2 * P)) order_two<I, I + K>(k);
      });
    });
  });
}

// ---- A token by the whole wave in 64 bits: experts N lane .. N lane + N - 1 in a lane.  Hardly any token comes here, but
// a wave that does is the last of its launch (of 16384 tokens among 256 experts some 40 do; 5 us with an entry's exponential
// after another's and groups by a scan of LDS, this way 4).  Ties all come: 16384 tokens by softmax 10 us, from bf16 logits 21,
// with all logits equal 26; sigmoid with biases and groups 15, with one bias of -1e9 41.

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp_i32<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp_i32<CTRL>((int)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_max64(double v) {
  v = fmax(v, dpp_f64<dpp::QUAD_XOR1>(v));
  v = fmax(v, dpp_f64<dpp::QUAD_XOR2>(v));
  v = fmax(v, dpp_f64<dpp::ROW_HALF_MIRROR>(v));
  v = fmax(v, dpp_f64<dpp::ROW_MIRROR>(v));
  return fmax(fmax(lane_f64(v, 0), lane_f64(v, 16)), fmax(lane_f64(v, 32), lane_f64(v, 48)));
}
// The larger two of both pairs (m1 >= m2).
__device__ __forceinline__ void two_of(double& m1, double& m2, double o1, double o2) {
  m2 = fmax(fmin(m1, o1), fmax(m2, o2));
  m1 = fmax(m1, o1);
}
template <int CTRL>
__device__ __forceinline__ void two_best(double& m1, double& m2) { two_of(m1, m2, dpp_f64<CTRL>(m1), dpp_f64<CTRL>(m2)); }

// The entry with the largest of v over the wave (of equal ones the lowest expert), which is set to -inf; -1 if all are.
template <int N>
__device__ __forceinline__ int take_best(double* v, int lane) {
  double most = v[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < N; ++i) {
    at = v[i] > most ? i : at;
    most = fmax(most, v[i]);
  }
  const double best = wave_max64(most);
  if (!(best > -INFINITY)) return -1;
  const int first = __builtin_ctzll(__ballot(most == best));
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane == first && at == i ? -INFINITY : v[i];
  return first * N + __builtin_amdgcn_readlane(at, first);
}

// Place j's expert in lane j (-1: none).  room: the wave's LDS, 64 N values.
template <int N>
__device__ __forceinline__ int choose64(const ChooseArgs& a, int t, int lane, float top, double* room) {
  const double NONE = -INFINITY;
  float l[N], b[N];
  double v[N], sum = 0;
  const bool groups = a.top_groups < a.groups;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane * N + i, at = e < a.E ? e : 0;
    const float x = a.logits[(size_t)t * a.E + at];
    b[i] = a.bias ? a.bias[at] : 0.f;
    l[i] = e < a.E && x > -INFINITY && b[i] > -INFINITY ? x : -INFINITY;
    v[i] = l[i];
  }
  if (a.bias || groups) {
    // (both scores by the same exponentials, so that the entries' chains of steps run side by side)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = exp(a.sigmoid ? -(double)l[i] : (l[i] == top ? 0.0 : (double)l[i] - top));
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 1.0 / (1.0 + v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) sum += l[i] == -INFINITY ? 0.0 : v[i];
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = l[i] == -INFINITY ? NONE : v[i] + (double)b[i];
  }
  if (groups) {
    const int size = a.E / a.groups, w = size / N;  // w: lanes of a group
    double m1 = NONE, m2 = NONE;
    // lane g: the two best of group g
    if (size % N == 0 && w <= 16 && (w & (w - 1)) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) two_of(m1, m2, v[i], NONE);
      if (w >= 2) two_best<dpp::QUAD_XOR1>(m1, m2);
      if (w >= 4) two_best<dpp::QUAD_XOR2>(m1, m2);
      if (w >= 8) two_best<dpp::ROW_HALF_MIRROR>(m1, m2);
      if (w >= 16) two_best<dpp::ROW_MIRROR>(m1, m2);
      m1 = __shfl(m1, lane * w & 63);
      m2 = __shfl(m2, lane * w & 63);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) room[lane * N + i] = v[i];
      lds_turn();
      if (lane < a.groups) {
#pragma unroll 4
        for (int c = 0; c < size; ++c) two_of(m1, m2, room[lane * size + c], NONE);
      }
      lds_turn();
    }
    const double of = a.best > 1 && m2 > NONE ? m1 + m2 : m1;
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const double o = lane_f64(of, g);
      rank += o > of || (o == of && g < lane) ? 1 : 0;
    }
    const uint64_t taken = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool on = l[i] > -INFINITY && ((taken >> ((lane * N + i) / size)) & 1);
      v[i] = !on ? NONE : (a.bias ? v[i] : (double)l[i]);
    }
  }
  int mine = -1;
#pragma unroll 1
  for (int r = 0; r < a.k; ++r) {
    const int id = take_best<N>(v, lane);
    mine = lane == r ? id : mine;
  }
  return mine;
}

// The choice: 64 / L tokens of a wave side by side, N experts in a lane: what goes over a token's lanes is shared by
// four tokens (a token to a wave with its rounds over 64-bit words: 92 us for 16384 tokens among 256 experts in 8 groups
// with biases, this way 16, of which the last 4 are waves with a token for 64 bits; 65536 tokens 36 us, some 350
// instructions a token, where their logits alone take 14; one token 5.1).  Values become whole numbers of
// BITS bits over their range with the expert's number below them, so that a round of the choice is a maximum of 32-bit
// words that are all different, and ties fall to the lower expert.
// KEEP of a lane's words in order are enough for k + 1 rounds.
template <int L, int N, int KEEP>
__global__ __launch_bounds__(CHOOSE_THREADS) void choose_kernel(ChooseArgs a) {
  constexpr int TOK = 64 / L, ID_BITS = L == 16 ? 8 : 10, BITS = 32 - ID_BITS;
  constexpr uint32_t ID_MASK = (1u << ID_BITS) - 1;
  static_assert(L * N <= 1 << ID_BITS, "an expert's number fits");
  constexpr float UNITS = (float)(1 << BITS);
  constexpr int ROW = L * N + L * N / 32;  // values of a token in LDS, one more place behind each 32
  constexpr int ROOM = TOK * ROW > 2 * L * N ? TOK * ROW : 2 * L * N;  // (fp32 values of all tokens, or 64-bit ones of one)
  __shared__ __align__(8) float lds[CHOOSE_WAVES][ROOM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L, slot = lane / L;
  const int t0 = (blockIdx.x * CHOOSE_WAVES + wave) * TOK;
  if (t0 >= a.T) return;
  const bool there = t0 + slot < a.T;
  const int t = there ? t0 + slot : a.T - 1;
  float l[N], b[N], v[N], top = -INFINITY, b_most = 0.f, total = 1.f;
  load_token<L, N>(a, t, j, l, b);
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, l[i]);
  top = max_of<L>(top);
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i) b_most = fmaxf(b_most, l[i] > -INFINITY ? fabsf(b[i]) : 0.f);
    b_most = max_of<L>(b_most);
  }
  const bool groups = a.top_groups < a.groups;
  bool sure = top < INFINITY;
  float near = 0.f, most = 0.f;  // how close two values may be for fp32 to order them; the largest score
  const bool scored = a.bias || groups || !(a.renorm || a.sigmoid);
  if (scored) {
    scores<L, N>(a, l, top, v, total);
    most = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-top)) : (total > 0.f ? __builtin_amdgcn_rcpf(total) : 0.f);
    // In units of 2^-23: exp(-l) is off by 0.75 |l| + 1 of itself (the exponent's rounding, v_exp_f32), 1 + exp(-l) by
    // 1/2, its reciprocal by 1, and s (1 - s) |l| is at most 0.23, or for l <= top < 0 (|top| + 1) exp(top): a sigmoid is off
    // by 4 + 0.75 |top| of the largest, |top| if below 0.  A softmax score is off by 2 of the largest, and all of a
    // token's by one factor, its sum's 20 additions: 10 of the difference.  The sum with b is off by 1/2 of both.
    // All of it twice, for two values.
    near = ldexpf(most * (a.sigmoid ? 9.f + fmaxf(-top, 0.f) * 1.5f : 16.f) + b_most, -23);
    if (!(top > -INFINITY)) near = 0.f;
    else if (a.sigmoid && top < -60.f) sure = false;  // (scores near and below fp32's smallest have no such errors)
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += b[i];
    }
    if (groups) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = l[i] == -INFINITY ? -INFINITY : v[i];
    }
  }
  uint64_t taken = ~0ull;
  const int size = a.E / a.groups;
  const uint32_t per = (1u << 20) / size + 1;  // e / size = e * per >> 20 (e, size <= 1024)
  if (groups) {
    float* part = &lds[wave][slot * ROW];
    const int w = size >> 2;  // lanes of a group
    if (size % 4 == 0 && w <= 16 && (w & (w - 1)) == 0) {
      // a group's two best by exchanges between the lanes that hold it
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        float m1 = fmaxf(v[i], v[i + 1]), m2 = fminf(v[i], v[i + 1]);
        const float n1 = fmaxf(v[i + 2], v[i + 3]), n2 = fminf(v[i + 2], v[i + 3]);
        m2 = fmaxf(fminf(m1, n1), fmaxf(m2, n2));
        m1 = fmaxf(m1, n1);
        if (w >= 2) two_best<dpp::QUAD_XOR1>(m1, m2);
        if (w >= 4) two_best<dpp::QUAD_XOR2>(m1, m2);
        if (w >= 8) two_best<dpp::ROW_HALF_MIRROR>(m1, m2);
        if (w >= 16) two_best<dpp::ROW_MIRROR>(m1, m2);
        const int e = expert_of<L>(i, j);
        if (e < a.E && (j & (w - 1)) == 0) part[(e * per) >> 20] = a.best > 1 && m2 > -INFINITY ? m1 + m2 : m1;
      }
    } else {
      // Lane p of the wave, then p + 64 ..: group p % groups of token p / groups, by a scan.
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = expert_of<L>(i, j);
        part[e + (e >> 5)] = v[i];
      }
      lds_turn();
      float of[TOK];
#pragma unroll
      for (int q = 0; q < TOK; ++q) {
        const int p = lane + 64 * q, s = p / a.groups, g = p - s * a.groups;
        float m1 = -INFINITY, m2 = -INFINITY;
        if (s < TOK) {
          const float* from = &lds[wave][s * ROW];
#pragma unroll 4
          for (int c = 0; c < size; ++c) {
            const int e = g * size + c;
            const float x = from[e + (e >> 5)];
            m2 = fmaxf(m2, fminf(m1, x));
            m1 = fmaxf(m1, x);
          }
        }
        of[q] = a.best > 1 && m2 > -INFINITY ? m1 + m2 : m1;
      }
      lds_turn();
#pragma unroll
      for (int q = 0; q < TOK; ++q) {
        const int p = lane + 64 * q, s = p / a.groups;
        if (s < TOK) lds[wave][s * ROW + p - s * a.groups] = of[q];
      }
    }
    lds_turn();
    // Lane j of a token ranks group j, then j + L ..
    taken = 0;
    float in = INFINITY, out = -INFINITY;
#pragma unroll 1
    for (int g0 = 0; g0 < a.groups; g0 += L) {
      const int g = g0 + j;
      const float mine = part[g < a.groups ? g : 0];
      int rank = 0;
#pragma unroll 8
      for (int h = 0; h < a.groups; ++h) {
        const float o = part[h];
        rank += o > mine || (o == mine && h < g) ? 1 : 0;
      }
      const bool real = g < a.groups, stays = real && rank < a.top_groups;
      if (stays) in = fminf(in, mine);
      else if (real) out = fmaxf(out, mine);
      const uint64_t all = __ballot(stays) >> (lane - j);
      taken |= (L == 64 ? all : all & 0xFFFFull) << g0;
    }
    in = -max_of<L>(-in);
    out = max_of<L>(out);
    // (both values are sums of two, each rounded once more, by 2^-24 of at most twice the largest; nothing hangs on groups
    // without experts)
    if (out > -INFINITY && !(in - out > 2.f * near + ldexpf(most + b_most, -22))) sure = false;
  }
  // ---- whole numbers, 1 and more
  uint32_t key[N], tol = 0;
  {
    float low, unit;
    if (a.bias) {
      const float span = most + 2.f * b_most;  // (values lie in -b_most .. most + b_most)
      low = -b_most;
      unit = UNITS / span;
      tol = (uint32_t)fminf(near * unit, 1.0e6f) + 4;  // (and the roundings on the way here)
      if (!(span < INFINITY)) sure = false;
    } else {
      low = top - 16.f;  // (what lies below is told apart in 64 bits)
      unit = UNITS / 16.f;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = l[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert_of<L>(i, j);
      const float x = fmaf(v[i] - low, unit, 1.f);
      const uint32_t n = (uint32_t)__builtin_amdgcn_fmed3f(x, 1.f, UNITS - 1.f);
      key[i] = l[i] > -INFINITY ? (n << ID_BITS) | (ID_MASK - e) : 0u;
    }
  }
  auto stay = [&](int i) -> uint32_t {  // all bits if entry i's group is taken
    return 0u - (uint32_t)((taken >> ((expert_of<L>(i, j) * per) >> 20)) & 1);
  };
  if (groups && size % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint32_t m = stay(i);
#pragma unroll
      for (int c = 0; c < 4; ++c) key[i + c] &= m;
    }
  } else if (groups) {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] &= stay(i);
  }
  // ---- the rounds, one more than k for the border: every lane's words in order, the largest first one is taken
  order_all<N>(key);
  uint32_t mine = 0, last = 0, gap = ~0u;  // gap: the smallest between two words in order
#pragma unroll 1
  for (int r = 0; r <= a.k; ++r) {
    const uint32_t best = max_of<L>(key[0]), less = last - best;  // (the first round's wraps: it is no gap)
    gap = best && r > 0 && less < gap ? less : gap;
    last = best;
    mine = j == r ? best : mine;
    const uint32_t out = key[0] == best ? ~0u : 0u;  // (by masks: a choice between two places becomes a search for the index)
#pragma unroll
    for (int i = 0; i + 1 < KEEP; ++i) key[i] = (out & key[i + 1]) | (~out & key[i]);
    key[KEEP - 1] &= ~out;
  }
  // (words of values tol apart differ by less than this)
  if (gap < (tol + 1) << ID_BITS) sure = false;
  int id = mine ? (int)(ID_MASK - (mine & ID_MASK)) : -1;
  for (uint64_t again = __ballot(there && !sure && j == 0); __builtin_expect(again != 0, 0); again &= again - 1) {
    const int first = __builtin_ctzll(again);  // of the token's lanes
    const int exact = choose64<L * N / 64>(a, t0 + first / L, lane, lane_f32(top, first), reinterpret_cast<double*>(&lds[wave][0]));
    // (from lanes 0 .. k - 1 to the token's)
    const int moved = __shfl(exact, j);
    id = lane / L == first / L ? moved : id;
  }
  if (j >= a.k) id = -1;
  const float at = id >= 0 ? a.logits[(size_t)t * a.E + id] : -INFINITY;
  const float w = weight_of<L>(a, id >= 0, at, top, total);
  if (there && j < a.k) {
    a.ids[(size_t)t * a.k + j] = id;
    a.w[(size_t)t * a.k + j] = id >= 0 ? a.scale * w : 0.f;
  }
}

// With p_i the chosen experts' shares (renormalised: w_i / scale) or scores:
//   d log p_i = p_i (dw_i - sum_j p_j dw_j) scale, or p_i dw_i scale;   sigmoid: d l_i = d log p_i (1 - s_i);
//   softmax: d l_e = sum of e's places, without renormalisation less s_e sum_j d log p_j.
// An expert that occurs twice gets both places' parts.
template <int L, int N>
__global__ __launch_bounds__(CHOOSE_THREADS) void choose_back_kernel(ChooseArgs a) {
  constexpr int TOK = 64 / L;
  __shared__ __align__(16) float lds[CHOOSE_WAVES][TOK][L * N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L, slot = lane / L;
  const int t0 = (blockIdx.x * CHOOSE_WAVES + wave) * TOK;
  if (t0 >= a.T) return;
  const bool there = t0 + slot < a.T;
  const int t = there ? t0 + slot : a.T - 1;
  const bool spread = !a.sigmoid && !a.renorm;  // every logit has a part
  const size_t at = (size_t)t * a.k + j;
  int id = j < a.k ? a.ids[at] : -1;
  float dw = j < a.k ? a.w[at] * a.scale : 0.f;
  const bool named = (uint32_t)id < (uint32_t)a.E;
  float l = named ? a.logits[(size_t)t * a.E + id] : -INFINITY;
  const bool chosen = l > -INFINITY && !(a.bias && !(a.bias[named ? id : 0] > -INFINITY));  // (an expert that is off has no part)
  if (!chosen) { id = -1; dw = 0.f; }
  float s[N], top = -INFINITY, total = 1.f;
  if (spread) {
    float row[N], b[N];
    load_token<L, N>(a, t, j, row, b);
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, row[i]);
    top = max_of<L>(top);
    scores<L, N>(a, row, top, s, total);
  }
  const float p = weight_of<L>(a, chosen, l, top, total);
  float part = a.renorm ? p * (dw - group_sum<L>(p * dw)) : p * dw;
  if (a.sigmoid) part *= 1.0f / (1.0f + expf(l));
  if (!chosen) part = 0.f;
  const float pull = spread ? group_sum<L>(part) : 0.f;
  // The chosen experts' parts in LDS, each in its expert's place: one after the other, should an expert occur twice.
  float* parts = &lds[wave][slot][0];
  float out[N];
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(parts + expert_of<L>(i, j)) = make_float4(0.f, 0.f, 0.f, 0.f);
  lds_turn();
  if (chosen) parts[id] = __builtin_bit_cast(float, j);
  lds_turn();
  const bool twice = chosen && __builtin_bit_cast(int, parts[id]) != j;
  lds_turn();
  if (__ballot(twice) == 0) {
    if (chosen) parts[id] = part;
  } else {
    if (chosen) parts[id] = 0.f;
    lds_turn();
    for (int r = 0; r < a.k; ++r) {
      if (chosen && j == r) parts[id] += part;
      lds_turn();
    }
  }
  lds_turn();
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 u = *reinterpret_cast<const float4*>(parts + expert_of<L>(i, j));
    out[i] = u.x; out[i + 1] = u.y; out[i + 2] = u.z; out[i + 3] = u.w;
  }
  if (spread) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = fmaf(-s[i], pull, out[i]);
  }
  if (!there) return;
  float* row = a.dlogits + (size_t)t * a.E;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const int e = expert_of<L>(i, j);
    if (e + 4 <= a.E) {
      *reinterpret_cast<f32x4_any*>(row + e) = f32x4_any{out[i], out[i + 1], out[i + 2], out[i + 3]};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < a.E) row[e + c] = out[i + c];
    }
  }
}

// f(lanes of a token, experts of a lane, words that a lane keeps)
template <typename F>
void by_width(const ChooseArgs& a, F&& f) {
  using std::integral_constant;
  auto wave = [&](auto n) { f(integral_constant<int, 64>{}, n, n); };
  auto rows = [&](auto n) { f(integral_constant<int, 16>{}, n, n); };
  if (a.E <= 256 && a.k <= 16) {
    if (a.E <= 64) rows(integral_constant<int, 4>{});
    else if (a.E <= 128) rows(integral_constant<int, 8>{});
    else if (a.k > 8) rows(integral_constant<int, 16>{});
    else f(integral_constant<int, 16>{}, integral_constant<int, 16>{}, integral_constant<int, 9>{});
  } else if (a.E <= 256) {
    wave(integral_constant<int, 4>{});
  } else if (a.E <= 512) {
    wave(integral_constant<int, 8>{});
  } else {
    wave(integral_constant<int, 16>{});
  }
}
unsigned choose_grid(const ChooseArgs& a, int lanes) {
  const int tokens = CHOOSE_WAVES * (64 / lanes);
  return (unsigned)((a.T + tokens - 1) / tokens);
}

}  // namespace

hipError_t launch_choose(const ChooseArgs& a, hipStream_t st) {
  by_width(a, [&](auto l, auto n, auto keep) {
    choose_kernel<decltype(l)::value, decltype(n)::value, decltype(keep)::value><<<choose_grid(a, decltype(l)::value), CHOOSE_THREADS, 0, st>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_choose_back(const ChooseArgs& a, hipStream_t st) {
  by_width(a, [&](auto l, auto n, auto) {
    choose_back_kernel<decltype(l)::value, decltype(n)::value><<<choose_grid(a, decltype(l)::value), CHOOSE_THREADS, 0, st>>>(a);
  });
  return hipGetLastError();
}

}  // namespace mvq
