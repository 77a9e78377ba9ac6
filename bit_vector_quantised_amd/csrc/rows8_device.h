// Rows in 8 bits on the device: blocks of 32 columns as e4m3 values times a power of two.
#pragma once

#include "block.h"
#include "dense_device.h"

namespace mvq {

typedef uint32_t u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));

// The exponent + 127 of a block's scale from the bits of its largest magnitude: the smallest power of two, 2^-110 or
// more, that brings it to 448 = 1.75 * 2^8 or less.  Scales no smaller than that keep every value a normal number
// in bf16 and fp32 (the smallest magnitude is 2^-9 scales).  255, which stands for NaN, if a value is not finite.
__device__ __forceinline__ uint32_t scale8(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return top >= 0x7F800000u ? 255u : (uint32_t)(e < 17 ? 17 : e);
}
__device__ __forceinline__ uint32_t top_bits8(const float* v) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  return top;
}
// Eight values in units of the scale, rounded to nearest even (v_cvt_pk_fp8_f32; none is above 448).  Zeros stay zeros in a
// block of NaN too: those behind the row's last column are zeros always.
__device__ __forceinline__ u32x2_t to_e4m3(const float* v, uint32_t scale) {
  const float inv = __builtin_bit_cast(float, (scale < 254u ? 254u - scale : 0u) << 23);
  int w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w[h], true);
  }
  return u32x2_t{(uint32_t)w[0], (uint32_t)w[1]};
}
// Eight neighbouring columns per lane, blocks of four lanes: the lane's bytes and its block's scale.
__device__ __forceinline__ u32x2_t block8(const float* v, uint32_t& scale) {
  uint32_t top = top_bits8(v);
  uint32_t o = (uint32_t)dpp_i32<dpp::QUAD_XOR1>((int)top);
  top = o > top ? o : top;
  o = (uint32_t)dpp_i32<dpp::QUAD_XOR2>((int)top);
  top = o > top ? o : top;
  scale = scale8(top);
  return to_e4m3(v, scale);
}

// Four e4m3 values times a scale.
__device__ __forceinline__ void from_e4m3(uint32_t w, float scale, float* v) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0] * scale;
  v[1] = lo[1] * scale;
  v[2] = hi[0] * scale;
  v[3] = hi[1] * scale;
}
// Eight consecutive values from column c of a row, the first `n` of them valid.  ALIGNED: c is a multiple of 8;
// otherwise they may lie in two blocks.
template <bool ALIGNED>
__device__ __forceinline__ void load8_q(const uint8_t* q, const uint8_t* e, int c, int n, float* v) {
  if (ALIGNED || n >= 8) {
    const u32x2_byte w = *reinterpret_cast<const u32x2_byte*>(q + c);
    const int b = c >> 5;
    const float scale = e8m0_to_f32(e[b]);
    if (ALIGNED) {
      from_e4m3(w.x, scale, v);
      from_e4m3(w.y, scale, v + 4);
    } else {
      const float next = e8m0_to_f32(e[(c + 7) >> 5]);
      from_e4m3(w.x, 1.f, v);
      from_e4m3(w.y, 1.f, v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= (c + j) >> 5 == b ? scale : next;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      if (j < n) from_e4m3(q[c + j], e8m0_to_f32(e[(c + j) >> 5]), t);
      v[j] = t[0];
    }
  }
}

}  // namespace mvq
