// Rows kept in 8 bits for the backward pass, and what reads them there:
//
//   pack      each block of 32 columns to e4m3 values in units of a power of two (rows8_device.h)
//   unpack    the values again, exact in bf16 and fp32; with the pairs' rows, each token's row to its k
//             experts' places
//   act_back  from z in 8 bits and dy, the gradient of the weighted sum's input rows, of each routed pair p with
//             row r:  y_r = w_p act(z_r),  dz_r = w_p dy_r act'(z_r),  dw_p = <dy_r, act(z_r)>
//
// All of them move each byte once and are bound by memory (a large copy: 5.0 TB/s).  In bf16: 32768 rows of 4096 columns
// into 8 bits 80 us (406 MB), out of them 69; 4096 tokens of 7168 columns to 8 rows each 91 us (500 MB); the way back
// through swiglu of 32768 rows of 2048 columns 140 us (674 MB).
#include "rows8_device.h"

namespace mvq {

namespace {

constexpr int PACK_THREADS = 256;
constexpr size_t STREAM_BYTES = (size_t)256 << 20;  // outputs that the memory-side cache does not hold are streamed

// Eight columns per thread, four threads to a block; rows from `first` on.  The columns behind the row's last are zeros.
template <int DTYPE>
__global__ __launch_bounds__(PACK_THREADS) void rows8_pack_kernel(Rows8Args a, uint32_t units, int first) {
  const uint32_t id = blockIdx.x * PACK_THREADS + threadIdx.x, at_row = id / units;
  const int row = first + (int)at_row, c = (int)(id - at_row * units) * 8;
  bool there = row < a.M;
  if (a.start) there = there && row >= a.start[0] && row < a.start[a.G];
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

// 16 bytes of each output row per thread, to each of the token's k rows (GATHER) or to its own; rows from `first` on.
// Neighbouring threads' stores join: with 32 bytes to a thread, in two stores, streamed ones take 256 us
// instead of 92 for 4096 tokens of 7168 bf16 columns to 8 rows each (not streamed 108 either way).
template <int DTYPE, bool GATHER, bool STREAM>
__global__ __launch_bounds__(PACK_THREADS) void rows8_unpack_kernel(Rows8Args a, uint32_t units, int first) {
  constexpr int N = DTYPE == MOE_VQ_BF16 ? 8 : 4;
  const uint32_t id = blockIdx.x * PACK_THREADS + threadIdx.x, at_row = id / units;
  const int row = first + (int)at_row, c = (int)(id - at_row * units) * N, left = (int)a.pitch - c;
  if (row >= a.M) return;
  if (a.start && (row < a.start[0] || row >= a.start[a.G])) return;
  const size_t pitch = rows8_pitch(a.C);
  const uint8_t* q = a.q + row * pitch + c;
  const float scale = e8m0_to_f32(a.e[row * (pitch / 32) + (c >> 5)]);
  float v[8];
  if constexpr (N == 8) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(q);
    from_e4m3(w.x, scale, v);
    from_e4m3(w.y, scale, v + 4);
  } else {
    from_e4m3(*reinterpret_cast<const uint32_t*>(q), scale, v);
  }
  const int n = GATHER ? a.k : 1;
  for (int i = 0; i < n; ++i) {
    const int to = GATHER ? a.pair_row[(size_t)row * n + i] : row;
    if (GATHER && (uint32_t)to >= (uint32_t)(a.M * n)) continue;
    const size_t at = (size_t)to * a.pitch + c;
    if constexpr (N == 8) {
      store8<STREAM>(a.y, at, DTYPE, left, v);
    } else {
      float* y = static_cast<float*>(a.y) + at;
      if (left >= 4) {
        store_vec<STREAM>(reinterpret_cast<f32x4_any*>(y), f32x4_any{v[0], v[1], v[2], v[3]});
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < left) y[j] = v[j];
      }
    }
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

// A pair by TX threads (16, a wave, or the workgroup), eight columns of a thread at a time.  ALIGNED: N is a
// multiple of 8, and so are the up values' places.
template <int DTYPE, int DY_DTYPE, int ACT, int TX, bool ALIGNED, bool STREAM>
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
      if (a.y) store8<STREAM>(a.y, row * a.N + n, DTYPE, left, y);
      if (a.dz) {
        store8<STREAM>(a.dz, row * a.R + n, DTYPE, left, dg);
        if (two) store8<STREAM>(a.dz, row * a.R + a.N + n, DTYPE, left, du);
      }
    }
  }
  if (!a.dw) return;
  sum = group_sum<TX < 64 ? TX : 64>(sum);
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

// f(workgroups, first row): threads count their units, `units` to a row, in 32 bits, so many rows take several launches.
template <typename F>
static void rows8_go(int M, uint32_t units, F&& f) {
  const int most = (int)((1u << 30) / units);  // (units: 1 to 8192)
  for (int first = 0, n; first < M; first += n) {
    n = M - first < most ? M - first : most;
    f((unsigned)(((size_t)n * units + PACK_THREADS - 1) / PACK_THREADS), first);
  }
}

hipError_t launch_rows8_pack(const Rows8Args& a, int dtype, hipStream_t st) {
  const uint32_t units = (uint32_t)(rows8_pitch(a.C) / 8);
  rows8_go(a.M, units, [&](unsigned grid, int first) {
    if (dtype == MOE_VQ_BF16) rows8_pack_kernel<MOE_VQ_BF16><<<grid, PACK_THREADS, 0, st>>>(a, units, first);
    else rows8_pack_kernel<MOE_VQ_F32><<<grid, PACK_THREADS, 0, st>>>(a, units, first);
  });
  return hipGetLastError();
}

hipError_t launch_rows8_unpack(const Rows8Args& a, int dtype, hipStream_t st) {
  const int size = dtype == MOE_VQ_BF16 ? 2 : 4, per = 16 / size;
  const uint32_t units = (uint32_t)((a.pitch + per - 1) / per);
  const bool stream = (size_t)a.M * (a.pair_row ? a.k : 1) * a.pitch * size > STREAM_BYTES;
  rows8_go(a.M, units, [&](unsigned grid, int first) {
    auto go = [&](auto t, auto gather) {
      constexpr int T = decltype(t)::value;
      constexpr bool G = decltype(gather)::value;
      if (stream) rows8_unpack_kernel<T, G, true><<<grid, PACK_THREADS, 0, st>>>(a, units, first);
      else rows8_unpack_kernel<T, G, false><<<grid, PACK_THREADS, 0, st>>>(a, units, first);
    };
    auto typed = [&](auto t) {
      if (a.pair_row) go(t, std::true_type{});
      else go(t, std::false_type{});
    };
    if (dtype == MOE_VQ_BF16) typed(std::integral_constant<int, MOE_VQ_BF16>{});
    else typed(std::integral_constant<int, MOE_VQ_F32>{});
  });
  return hipGetLastError();
}

template <int DTYPE, int DY_DTYPE, int ACT>
static void act_back_go(const ActBackArgs& a, hipStream_t st) {
  auto go = [&](auto tx, auto aligned) {
    constexpr int TX = decltype(tx)::value, rows = ACT_THREADS / TX;
    constexpr bool A = decltype(aligned)::value;
    // (32768 rows of 2048 columns, swiglu: 144 us, streamed 140; of fp32 rows a thread's 32 bytes are two stores, see above)
    if constexpr (TX == ACT_THREADS && DTYPE == MOE_VQ_BF16 && A) {
      if ((size_t)a.P * (a.R + a.N) * 2 > STREAM_BYTES) {
        act_back_kernel<DTYPE, DY_DTYPE, ACT, TX, A, true><<<(a.P + rows - 1) / rows, ACT_THREADS, 0, st>>>(a);
        return;
      }
    }
    act_back_kernel<DTYPE, DY_DTYPE, ACT, TX, A, false><<<(a.P + rows - 1) / rows, ACT_THREADS, 0, st>>>(a);
  };
  auto wide = [&](auto aligned) {
    // (129312 rows of 128 fp32 columns, swiglu: 115 us by a wave to a row, 68 by 16 lanes)
    if (a.N <= 256) go(std::integral_constant<int, 16>{}, aligned);
    else if (a.N <= 1024) go(std::integral_constant<int, 64>{}, aligned);
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
