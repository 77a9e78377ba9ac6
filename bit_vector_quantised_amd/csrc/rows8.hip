// Rows kept in 8 bits for the backward pass, and what reads them there:
//
//   pack      each block of 32 columns to e4m3 values in units of a power of two (rows8_device.h)
//   unpack    the values again, exact in bf16 and fp32; with the pairs' rows, each token's row to its k
//             experts' places
//   act_back  from z in 8 bits and dy, the gradient of the weighted sum's input rows, of each routed pair p with
//             row r:  y_r = w_p act(z_r),  dz_r = w_p dy_r act'(z_r),  dw_p = <dy_r, act(z_r)>
//
// All of them move each byte once and are bound by memory.
#include "rows8_device.h"

namespace mvq {

namespace {

constexpr int PACK_THREADS = 256;

// Eight columns per thread, four threads to a block.  The columns behind the row's last are zeros.
template <int DTYPE>
__global__ __launch_bounds__(PACK_THREADS) void rows8_pack_kernel(Rows8Args a, uint32_t units) {
  const uint32_t id = blockIdx.x * PACK_THREADS + threadIdx.x, row = id / units;
  const int c = (int)(id - row * units) * 8;
  bool there = row < (uint32_t)a.M;
  if (a.start) there = there && (int)row >= a.start[0] && (int)row < a.start[a.G];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (there && c < a.C) load8(a.x, (size_t)row * a.C + c, DTYPE, a.C - c, v);
  uint32_t scale;
  const u32x2_t w = block8(v, scale);  // (a block's four threads hold or miss a row together)
  if (!there) return;
  const size_t pitch = rows8_pitch(a.C);
  *reinterpret_cast<u32x2_t*>(a.q + row * pitch + c) = w;
  if ((threadIdx.x & 3) == 0) a.e[row * (pitch / 32) + (c >> 5)] = (uint8_t)scale;
}

// Sixteen columns per thread, to each of the token's k rows (GATHER) or to its own.
template <int DTYPE, bool GATHER>
__global__ __launch_bounds__(PACK_THREADS) void rows8_unpack_kernel(Rows8Args a, uint32_t units) {
  const uint32_t id = blockIdx.x * PACK_THREADS + threadIdx.x, row = id / units;
  const int c = (int)(id - row * units) * 16, left = (int)a.pitch - c;
  if (row >= (uint32_t)a.M) return;
  if (a.start && ((int)row < a.start[0] || (int)row >= a.start[a.G])) return;
  const size_t pitch = rows8_pitch(a.C);
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(a.q + row * pitch + c);
  const float scale = e8m0_to_f32(a.e[row * (pitch / 32) + (c >> 5)]);
  float v[16];
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) from_e4m3(words[i], scale, v + 4 * i);
  const int n = GATHER ? a.k : 1;
  for (int i = 0; i < n; ++i) {
    const int to = GATHER ? a.pair_row[(size_t)row * n + i] : (int)row;
    if (GATHER && (uint32_t)to >= (uint32_t)(a.M * n)) continue;
    const size_t at = (size_t)to * a.pitch + c;
    store8(a.y, at, DTYPE, left, v);
    if (left > 8) store8(a.y, at + 8, DTYPE, left - 8, v + 8);
  }
}

// The activation and its derivatives (SWIGLU: by gate and by up) at eight columns.
template <int ACT>
__device__ __forceinline__ void act_values(float lim, const float* zg, const float* zu, float* y, float* dg, float* du) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (ACT == MOE_VQ_ACT_NONE) {
      y[j] = zg[j];
      dg[j] = 1.f;
    } else if (ACT == MOE_VQ_ACT_SILU) {
      const float s = sigmoid_fast(zg[j]);
      y[j] = zg[j] * s;
      dg[j] = silu_grad(zg[j], s);
    } else if (ACT == MOE_VQ_ACT_GELU) {
      const float e = __expf(-0.5f * zg[j] * zg[j]), p = normal_cdf(zg[j], e);
      y[j] = zg[j] * p;
      dg[j] = p + zg[j] * 0.39894228f * e;
    } else {
      // no gradient through a value that was clamped
      float g = zg[j], u = zu[j];
      bool gin = true, uin = true;
      if (lim > 0.f) {
        gin = !(g > lim);
        uin = !(u > lim) && !(u < -lim);
        g = gin ? g : lim;
        u = u > lim ? lim : (u < -lim ? -lim : u);
      }
      const float s = sigmoid_fast(g), gs = g * s;
      y[j] = gs * u;
      dg[j] = gin ? u * silu_grad(g, s) : 0.f;
      du[j] = uin ? gs : 0.f;
    }
  }
}

constexpr int ACT_THREADS = 256;

// A pair by TX threads (a wave, or the workgroup), eight columns of a thread at a time.  ALIGNED: N is a
// multiple of 8, and so are the up values' places.
template <int DTYPE, int DY_DTYPE, int ACT, int TX, bool ALIGNED>
__global__ __launch_bounds__(ACT_THREADS) void act_back_kernel(ActBackArgs a) {
  __shared__ float red[ACT_THREADS / 64];
  constexpr bool two = ACT == MOE_VQ_ACT_SWIGLU;
  const int tx = threadIdx.x % TX, p = blockIdx.x * (ACT_THREADS / TX) + threadIdx.x / TX;
  const int r = p < a.P ? a.pair_row[p] : -1;
  const bool there = (uint32_t)r < (uint32_t)a.P;
  float sum = 0.f;
  if (there) {
    const float w = a.w ? a.w[p] : 1.f;
    const size_t row = r, pitch = rows8_pitch(a.R);
    const uint8_t *q = a.q + row * pitch, *e = a.e + row * (pitch / 32);
    for (int n = tx * 8; n < a.N; n += TX * 8) {
      const int left = a.N - n;
      float zg[8], zu[8], dy[8], y[8], dg[8], du[8];
      load8(a.dy, row * a.N + n, DY_DTYPE, left, dy);
      load8_q<true>(q, e, n, left, zg);  // (the pitch holds whole eights)
      if (two) load8_q<ALIGNED>(q, e, a.N + n, left, zu);
      act_values<ACT>(a.lim, zg, zu, y, dg, du);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (ALIGNED || j < left) sum = fmaf(dy[j], y[j], sum);
        const float d = w * dy[j];
        y[j] *= w;
        dg[j] *= d;
        if (two) du[j] *= d;
      }
      if (a.y) store8(a.y, row * a.N + n, DTYPE, left, y);
      if (a.dz) {
        store8(a.dz, row * a.R + n, DTYPE, left, dg);
        if (two) store8(a.dz, row * a.R + a.N + n, DTYPE, left, du);
      }
    }
  }
  if (!a.dw) return;
  sum = wave_sum(sum);
  if (TX > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < ACT_THREADS / 64; ++i) sum += red[i];
  }
  if (tx == 0 && p < a.P) a.dw[p] = there ? sum : 0.f;  // (a dropped pair's weight moved nothing)
}

}  // namespace

static unsigned rows8_grid(int M, uint32_t units) { return (unsigned)(((size_t)M * units + PACK_THREADS - 1) / PACK_THREADS); }

hipError_t launch_rows8_pack(const Rows8Args& a, int dtype, hipStream_t st) {
  const uint32_t units = (uint32_t)(rows8_pitch(a.C) / 8);
  const unsigned grid = rows8_grid(a.M, units);
  if (dtype == MOE_VQ_BF16) rows8_pack_kernel<MOE_VQ_BF16><<<grid, PACK_THREADS, 0, st>>>(a, units);
  else rows8_pack_kernel<MOE_VQ_F32><<<grid, PACK_THREADS, 0, st>>>(a, units);
  return hipGetLastError();
}

hipError_t launch_rows8_unpack(const Rows8Args& a, int dtype, hipStream_t st) {
  const uint32_t units = (uint32_t)((a.pitch + 15) / 16);
  const unsigned grid = rows8_grid(a.M, units);
  auto go = [&](auto t, auto gather) {
    rows8_unpack_kernel<decltype(t)::value, decltype(gather)::value><<<grid, PACK_THREADS, 0, st>>>(a, units);
  };
  auto typed = [&](auto t) {
    if (a.pair_row) go(t, std::true_type{});
    else go(t, std::false_type{});
  };
  if (dtype == MOE_VQ_BF16) typed(std::integral_constant<int, MOE_VQ_BF16>{});
  else typed(std::integral_constant<int, MOE_VQ_F32>{});
  return hipGetLastError();
}

template <int DTYPE, int DY_DTYPE, int ACT>
static void act_back_go(const ActBackArgs& a, hipStream_t st) {
  auto go = [&](auto tx, auto aligned) {
    constexpr int TX = decltype(tx)::value, rows = ACT_THREADS / TX;
    act_back_kernel<DTYPE, DY_DTYPE, ACT, TX, decltype(aligned)::value><<<(a.P + rows - 1) / rows, ACT_THREADS, 0, st>>>(a);
  };
  auto wide = [&](auto aligned) {
    if (a.N <= 1024) go(std::integral_constant<int, 64>{}, aligned);
    else go(std::integral_constant<int, ACT_THREADS>{}, aligned);
  };
  if (a.N % 8 == 0) wide(std::true_type{});
  else wide(std::false_type{});
}

template <int DTYPE, int DY_DTYPE>
static void act_back_act(const ActBackArgs& a, hipStream_t st) {
  if (a.act == MOE_VQ_ACT_NONE) act_back_go<DTYPE, DY_DTYPE, MOE_VQ_ACT_NONE>(a, st);
  else if (a.act == MOE_VQ_ACT_SILU) act_back_go<DTYPE, DY_DTYPE, MOE_VQ_ACT_SILU>(a, st);
  else if (a.act == MOE_VQ_ACT_GELU) act_back_go<DTYPE, DY_DTYPE, MOE_VQ_ACT_GELU>(a, st);
  else act_back_go<DTYPE, DY_DTYPE, MOE_VQ_ACT_SWIGLU>(a, st);
}

hipError_t launch_act_back(const ActBackArgs& a, int dtype, int dy_dtype, hipStream_t st) {
  if (dtype == MOE_VQ_BF16) {
    if (dy_dtype == MOE_VQ_BF16) act_back_act<MOE_VQ_BF16, MOE_VQ_BF16>(a, st);
    else act_back_act<MOE_VQ_BF16, MOE_VQ_F32>(a, st);
  } else {
    if (dy_dtype == MOE_VQ_BF16) act_back_act<MOE_VQ_F32, MOE_VQ_BF16>(a, st);
    else act_back_act<MOE_VQ_F32, MOE_VQ_F32>(a, st);
  }
  return hipGetLastError();
}

}  // namespace mvq
