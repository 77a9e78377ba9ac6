// Device helpers of the dense operators: activations and their derivatives, and accesses of eight
// consecutive values of a row in either element type.
#pragma once

#include "moe_vq_device.h"

namespace mvq {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------------------

// Phi(-a) for a >= 0 from e = exp(-a^2 / 2): e q(a), with q(a) = erfc(a / sqrt(2)) exp(a^2 / 2) / 2, a smooth function
// between 1/2 and 0.4 / a, as a polynomial in s = 1 / (1 + 0.23 a) fitted to its relative error over 0..14 (5e-8;
// evaluated in fp32 4.2e-7).  The usual 1 + erf(z / sqrt(2)) loses what is left of Phi below z = -4, and is 0 from
// -5.5 on; the library's erfcf keeps it (column sums of dz, 8192 x 8192 values in bf16: 52 us this way, 76 by
// erff, 104 by erfcf).
__device__ __forceinline__ float normal_tail(float a, float e) {
  const float s = __builtin_amdgcn_rcpf(fmaf(0.23f, a, 1.0f));
  constexpr float C[] = {-2.7751521e-05f, 0.09237833f, 0.08576334f, 0.119514026f, -0.032923725f,
                         0.3014828f, -0.27813974f, 0.29042214f, -0.078469455f};
  float q = C[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) q = fmaf(q, s, C[i]);
  return e * q;
}
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float p = normal_tail(fabsf(z), e);
  return z < 0.f ? p : 1.0f - p;
}
__device__ __forceinline__ float gelu(float z) { return z * normal_cdf(z, __expf(-0.5f * z * z)); }
// (v_rcp_f32: within one unit in the last place)
__device__ __forceinline__ float sigmoid_fast(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// d silu(z) / dz = s + z s (1 - s), s = sigmoid(z)
__device__ __forceinline__ float silu_grad(float z, float s) { return s * (1.0f + z * (1.0f - s)); }
// d gelu(z) / dz = Phi(z) + z phi(z)
__device__ __forceinline__ float gelu_grad(float z) {
  const float e = __expf(-0.5f * z * z);
  return normal_cdf(z, e) + z * 0.39894228f * e;
}

// ---------------------------------------------------------------------------------------
// Accesses
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ float load_as_f32(const void* p, size_t i, int dtype) {
  return dtype == MOE_VQ_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_as(void* p, size_t i, int dtype, float v) {
  if (dtype == MOE_VQ_BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
  else static_cast<float*>(p)[i] = v;
}
// Eight consecutive values from index i, the first `n` of them valid: as one or two accesses where all are.
__device__ __forceinline__ void load8(const void* p, size_t i, int dtype, int n, float* v) {
  if (n >= 8 && dtype == MOE_VQ_BF16) {
    const u32x4_any u = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_bits_to_f32(w[q] & 0xFFFFu);
      v[2 * q + 1] = __builtin_bit_cast(float, w[q] & 0xFFFF0000u);
    }
  } else if (n >= 8) {
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4_any u = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i + q);
      v[q] = u.x; v[q + 1] = u.y; v[q + 2] = u.z; v[q + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? load_as_f32(p, i + j, dtype) : 0.f;
  }
}
// The same in two steps, loads now and values later: the bits of eight values as they lie in memory.
template <int DTYPE>
struct Bits8 {
  uint32_t w[DTYPE == MOE_VQ_BF16 ? 4 : 8];
};
template <int DTYPE, bool STREAM = false>
__device__ __forceinline__ void load_bits8(const void* p, size_t i, int n, Bits8<DTYPE>& b) {
  if constexpr (DTYPE == MOE_VQ_BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (n >= 8) {
      const u32x4_any u = load_vec<STREAM>(reinterpret_cast<const u32x4_any*>(q));
      b.w[0] = u.x; b.w[1] = u.y; b.w[2] = u.z; b.w[3] = u.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b.w[j] = (2 * j < n ? q[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)q[2 * j + 1] << 16 : 0u);
    }
  } else {
    const uint32_t* q = static_cast<const uint32_t*>(p) + i;
    if (n >= 8) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const u32x4_any u = load_vec<STREAM>(reinterpret_cast<const u32x4_any*>(q + j));
        b.w[j] = u.x; b.w[j + 1] = u.y; b.w[j + 2] = u.z; b.w[j + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b.w[j] = j < n ? q[j] : 0u;
    }
  }
}
template <int DTYPE>
__device__ __forceinline__ float value_of(const Bits8<DTYPE>& b, int j) {
  if constexpr (DTYPE == MOE_VQ_BF16) return j & 1 ? __builtin_bit_cast(float, b.w[j >> 1] & 0xFFFF0000u) : bf16_bits_to_f32(b.w[j >> 1] & 0xFFFFu);
  else return __builtin_bit_cast(float, b.w[j]);
}

// STREAM: nontemporal stores, which leave the L2 to the operands that other tiles share.
template <bool STREAM = false>
__device__ __forceinline__ void store8(void* p, size_t i, int dtype, int n, const float* v) {
  if (n >= 8 && dtype == MOE_VQ_BF16) {
    store_vec<STREAM>(reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i),
                      u32x4_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
  } else if (n >= 8) {
#pragma unroll
    for (int q = 0; q < 8; q += 4)
      store_vec<STREAM>(reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i + q), f32x4_any{v[q], v[q + 1], v[q + 2], v[q + 3]});
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) store_as(p, i + j, dtype, v[j]);
  }
}

}  // namespace mvq
