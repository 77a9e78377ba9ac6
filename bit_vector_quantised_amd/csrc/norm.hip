// Root-mean-square norm with the residual's addition before it, and its gradients:
//
//   forward   s = x + r,  y = s rho g,  rho = (mean(s^2) + eps)^(-1/2);  y in bf16 or fp32, and (or) in 8 bits
//   gradients with t = g (dy + dy2):
//             dx = ds + rho t - s rho^3 mean(t s)        (of x and of r alike)
//             dg = sum over the rows of (dy + dy2) s rho
//
// Every value is moved once and the sums are over the row that a workgroup holds in registers, so both are bound
// by memory: 4096 rows of 7168 columns in bf16 take 55 us forward with s, y and 8 bits (265 MB: 4.8 TB/s; a large copy
// reaches 5.0) and 59 us back with two gradients of y and one of s (294 MB), the gain's parts 5 us more; one row 3.3 us.
// Sums are fp32 in a fixed order, without atomics.
#include "rows8_device.h"

namespace mvq {

namespace {

constexpr int V = 8;  // columns per thread and chunk

// Sums over the threads of a row: LPR lanes of a wave, or (0) the workgroup, whose waves' sums meet in red[].
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float* v, float (*red)[N]) {
  if constexpr (LPR > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<LPR>(v[i]);
  } else {
    const int waves = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < waves; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[w][i];
    }
  }
}

// A row by LPR lanes, or (0) by a workgroup of as many threads as it has eights of columns (up to 8192 columns in one
// chunk: one load of each operand per thread, and as many waves on their way as a CU takes), NCH chunks of eight
// columns per thread.
template <int XT, int ST, int YT, int NCH, int LPR>
__global__ __launch_bounds__(LPR ? 256 : 1024) void norm_kernel(NormArgs a) {
  __shared__ float red[16][1];
  const int width = LPR ? LPR : blockDim.x, tx = LPR ? threadIdx.x % LPR : threadIdx.x;
  int row = LPR ? blockIdx.x * (256 / (LPR ? LPR : 1)) + threadIdx.x / (LPR ? LPR : 1) : blockIdx.x;
  const bool there = row < a.M;
  if (!there) row = a.M - 1;  // (every lane takes part in the sums)
  const size_t at = (size_t)row * a.C;
  float v[NCH][V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * width + tx) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] = 0.f;
    if (c < a.C) {
      load8(a.x, at + c, XT, a.C - c, v[i]);
      if (a.res) {
        float r[V];
        load8(a.res, at + c, ST, a.C - c, r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += r[j];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sum = fmaf(v[i][j], v[i][j], sum);
  }
  row_sums<LPR, 1>(&sum, red);
  // (s goes out rounded, y is made from the unrounded sum)
  const float rho = 1.0f / sqrtf(sum / (float)a.C + a.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * width + tx) * V, left = a.C - c;
    if (a.s && there && c < a.C) store8(a.s, at + c, ST, left, v[i]);
    float g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = 0.f;
    if (c < a.C) load8(a.gain, c, MOE_VQ_F32, left, g);
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] = c + j < a.C ? v[i][j] * rho * g[j] : 0.f;
    if (a.y && there && c < a.C) store8(a.y, at + c, YT, left, v[i]);
    if (a.q) {
      uint32_t scale;
      const u32x2_t w = block8(v[i], scale);
      const size_t pitch = rows8_pitch(a.C);
      if (there && c < (int)pitch) {
        *reinterpret_cast<u32x2_t*>(a.q + row * pitch + c) = w;
        if ((threadIdx.x & 3) == 0) a.e[row * (pitch / 32) + (c >> 5)] = (uint8_t)scale;
      }
    }
  }
}

// Both sums of a row at once, then its gradient; a workgroup walks rows and adds up its part of dg in registers.  The
// next row's loads go out before this one's sums.
template <int DYT, int ST, int DXT, int NCH, int LPR>
__global__ __launch_bounds__(LPR ? 256 : 1024) void norm_back_kernel(NormBackArgs a) {
  constexpr int RP = LPR ? 256 / LPR : 1;  // rows of a workgroup at a time
  __shared__ float red[2][16][2];
  __shared__ float meet[LPR ? 256 * V : 1];
  const int width = LPR ? LPR : blockDim.x, tx = LPR ? threadIdx.x % LPR : threadIdx.x;
  struct Row {
    Bits8<ST> s[NCH];
    Bits8<DYT> dy[NCH], dy2[NCH];
    Bits8<DXT> ds[NCH];
  } row[2];
  const int mine = LPR ? threadIdx.x / (LPR ? LPR : 1) : 0;
  auto load = [&](Row& to, int r0) {
    const int r = r0 + mine < a.M ? r0 + mine : a.M - 1;
    const size_t at = (size_t)r * a.C;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * width + tx) * V, left = c < a.C ? a.C - c : 0;
      load_bits8<ST>(a.s, at + c, left, to.s[i]);
      load_bits8<DYT>(a.dy, at + c, left, to.dy[i]);
      if (a.dy2) load_bits8<DYT>(a.dy2, at + c, left, to.dy2[i]);
      if (a.ds) load_bits8<DXT>(a.ds, at + c, left, to.ds[i]);
    }
  };
  constexpr bool AHEAD = NCH == 1;  // (two chunks of two rows, or of a row and the gain, would not fit the registers)
  float g[NCH][V], acc[NCH][V];
  auto load_gain = [&](int i) {
    const int c = (i * width + tx) * V;
    load8(a.gain, c, MOE_VQ_F32, c < a.C ? a.C - c : 0, g[i]);
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if (AHEAD) load_gain(i);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = 0.f;
  }
  const int step = gridDim.x * RP;
  auto turn = [&](Row& now, Row& then, float (*part)[2], int r0) {
    if (!AHEAD) load(now, r0);
    else if (r0 + step < a.M) load(then, r0 + step);
    const bool there = r0 + mine < a.M;
    const size_t at = (size_t)(there ? r0 + mine : a.M - 1) * a.C;
    float sum[2] = {0.f, 0.f};
    auto dy_of = [&](int i, int j) { return a.dy2 ? value_of(now.dy[i], j) + value_of(now.dy2[i], j) : value_of(now.dy[i], j); };
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!AHEAD) load_gain(i);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float s = value_of(now.s[i], j);
        sum[0] = fmaf(s, s, sum[0]);
        sum[1] = fmaf(dy_of(i, j) * g[i][j], s, sum[1]);
      }
    }
    row_sums<LPR, 2>(sum, part);
    const float rho = 1.0f / sqrtf(sum[0] / (float)a.C + a.eps);
    const float pull = rho * (rho * (sum[1] / (float)a.C));  // (rho^2 alone is infinite for eps below 2^-128 and zeros)
    if (!there) return;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * width + tx) * V, left = a.C - c;
      if (!AHEAD) load_gain(i);
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float s = value_of(now.s[i], j), d = dy_of(i, j);
        acc[i][j] = fmaf(d, s * rho, acc[i][j]);
        o[j] = rho * (d * g[i][j] - s * pull);
        if (a.ds) o[j] += value_of(now.ds[i], j);
      }
      if (a.dx && c < a.C) store8(a.dx, at + c, DXT, left, o);
    }
  };
  // (two turns' sums lie apart: a wave may be a row ahead)
  int r0 = blockIdx.x * RP;
  if constexpr (AHEAD) {
    if (r0 < a.M) load(row[0], r0);
    for (; r0 < a.M; r0 += 2 * step) {
      turn(row[0], row[1], red[0], r0);
      if (r0 + step < a.M) turn(row[1], row[0], red[1], r0 + step);
    }
  } else {
    for (int k = 0; r0 < a.M; r0 += step, k ^= 1) turn(row[0], row[0], red[k], r0);
  }
  if (!a.dgain) return;
  if constexpr (LPR > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) meet[threadIdx.x * V + j] = acc[0][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.C; c += 256) {
      float t = 0.f;
#pragma unroll
      for (int r = 0; r < RP; ++r) t += meet[r * LPR * V + c];
      a.part[(size_t)blockIdx.x * a.C + c] = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * width + tx) * V;
      if (c < a.C) store8(a.part, (size_t)blockIdx.x * a.C + c, MOE_VQ_F32, a.C - c, acc[i]);
    }
  }
}

// dg from the workgroups' parts: 32 columns by 32 shares of the parts, the shares in order.
__global__ __launch_bounds__(1024) void norm_gain_kernel(const float* part, float* out, int n, int parts) {
  __shared__ float red[32][32];
  const int c = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  const int per = (parts + 31) / 32, q0 = share * per, q1 = q0 + per < parts ? q0 + per : parts;
  float s = 0.f;
  if (i < n) {
#pragma unroll 8
    for (int q = q0; q < q1; ++q) s += part[(size_t)q * n + i];
  }
  red[share][c] = s;
  __syncthreads();
  if (share == 0 && i < n) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += red[q][c];
    out[i] = t;
  }
}

// How a row lies over threads.
struct NormShape {
  int lpr, nch, threads;
};
NormShape norm_shape(int C) {
  if (C <= 16 * V) return {16, 1, 256};
  if (C <= 64 * V) return {64, 1, 256};
  const int nch = C <= 1024 * V ? 1 : 2;
  return {0, nch, ((C + V * nch - 1) / (V * nch) + 63) / 64 * 64};
}

// f(integral constants of two element types ..., chunks, lanes per row)
template <typename F>
void norm_types(int a, int b, int c, const NormShape& s, F&& f) {
  auto shape = [&](auto ta, auto tb, auto tc) {
    using std::integral_constant;
    if (s.lpr == 16) f(ta, tb, tc, integral_constant<int, 1>{}, integral_constant<int, 16>{});
    else if (s.lpr == 64) f(ta, tb, tc, integral_constant<int, 1>{}, integral_constant<int, 64>{});
    else if (s.nch == 1) f(ta, tb, tc, integral_constant<int, 1>{}, integral_constant<int, 0>{});
    else f(ta, tb, tc, integral_constant<int, 2>{}, integral_constant<int, 0>{});
  };
  using B = std::integral_constant<int, MOE_VQ_BF16>;
  using F32 = std::integral_constant<int, MOE_VQ_F32>;
  auto third = [&](auto ta, auto tb) {
    if (c == MOE_VQ_BF16) shape(ta, tb, B{});
    else shape(ta, tb, F32{});
  };
  auto second = [&](auto ta) {
    if (b == MOE_VQ_BF16) third(ta, B{});
    else third(ta, F32{});
  };
  if (a == MOE_VQ_BF16) second(B{});
  else second(F32{});
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, int s_dtype, int y_dtype, hipStream_t st) {
  const NormShape s = norm_shape(a.C);
  const int rows = s.lpr ? 256 / s.lpr : 1;
  norm_types(dtype, s_dtype, y_dtype, s, [&](auto x, auto t, auto y, auto nch, auto lpr) {
    norm_kernel<decltype(x)::value, decltype(t)::value, decltype(y)::value, decltype(nch)::value, decltype(lpr)::value>
        <<<(a.M + rows - 1) / rows, s.threads, 0, st>>>(a);
  });
  return hipGetLastError();
}

// As many workgroups as make 16 waves of a CU, whose loads run a row ahead (4096 x 7168 in bf16, all five tensors: 59 us
// by one workgroup of 14; two that wait for each row's loads 72).
int norm_back_blocks(int M, int C) {
  const NormShape s = norm_shape(C);
  const int rows = s.lpr ? 256 / s.lpr : 1, need = (M + rows - 1) / rows, waves = s.threads / 64;
  const int most = 256 * (waves < 16 ? 16 / waves : 1);
  return need < most ? need : most;
}

hipError_t launch_norm_back(const NormBackArgs& a, int dy_dtype, int s_dtype, int dx_dtype, hipStream_t st) {
  const NormShape s = norm_shape(a.C);
  const int blocks = norm_back_blocks(a.M, a.C);
  if (blocks > 0)
    norm_types(dy_dtype, s_dtype, dx_dtype, s, [&](auto dy, auto t, auto dx, auto nch, auto lpr) {
      norm_back_kernel<decltype(dy)::value, decltype(t)::value, decltype(dx)::value, decltype(nch)::value, decltype(lpr)::value>
          <<<blocks, s.threads, 0, st>>>(a);
    });
  if (a.dgain) norm_gain_kernel<<<(a.C + 31) / 32, 1024, 0, st>>>(a.part, a.dgain, a.C, blocks);
  return hipGetLastError();
}

}  // namespace mvq
