// Tokens sorted by expert and back: the routed pairs p = t*k + i sorted stably by expert
// id, the tokens' rows copied into that order, the experts' rows added up per token with
// the routing weights, and the gradients of both.
//
//   sort      start[e] = #{valid p : id_p < e};  row of p = start[id_p] + #{q < p : id_q = id_p}
//   gather    xs[row(p)] = x[p / k]
//   combine   y[t] = r[t] + sum_i w[t,i] rows[row(t,i)]
//   gradients dx[t] = sum_i dxs[row(t,i)]          (combine without weights)
//             drows[row(p)] = w_p dy[t],  dw_p = <dy[t], rows[row(p)]>
//
// Everything here moves rows through HBM once and computes next to nothing, so each
// kernel is laid out to touch a row's bytes once: gather and the weighted gradient read a
// token's row once for its k copies, combine holds a token's sums in registers while its
// k rows stream by.  Sums run over i in order and in fp32, without atomics: repeated
// calls give the same bits.
#include "dense.h"
#include "moe_vq_device.h"

namespace mvq {

// ---------------------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------------------

// Lanes of the wave that hold the same id as this one (among the valid lanes), from one
// ballot per id bit.
__device__ __forceinline__ uint64_t match_lanes(int id, bool ok, int bits) {
  uint64_t m = __ballot(ok);
  for (int b = 0; b < bits; ++b) {
    const bool set = (id >> b) & 1;
    const uint64_t with = __ballot(set);
    m &= set ? with : ~with;
  }
  return m;
}

// A counting sort.  Each wave takes 64 * STEPS consecutive pairs, 64 at a time in order,
// and counts them per expert in its own row of LDS: a pair's place among the wave's equal
// ids is the count so far plus the equal lanes below it, so no atomics are needed and
// the order is stable.  Prefix sums over waves, experts and workgroups then give the rows.
// ALL: one workgroup does everything.  Otherwise the first launch (COUNT) writes each
// workgroup's counts and the second adds them up (every workgroup for itself) and places
// its pairs.
enum SortMode { SORT_ALL = 0, SORT_COUNT = 1, SORT_PLACE = 2 };

template <int STEPS, int MODE>
__global__ __launch_bounds__(SORT_THREADS) void sort_kernel(SortArgs a) {
  __shared__ volatile uint16_t cnt[SORT_WAVES][MAX_E];  // (at most 16 * 1024 pairs: 16 bits hold any count)
  __shared__ int base[MAX_E];
  __shared__ int wave_tot[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, P = a.P;
  for (int i = lane; i < E; i += 64) cnt[wave][i] = 0;
  __builtin_amdgcn_wave_barrier();
  const int bits = 32 - __clz(E > 1 ? E - 1 : 1);
  const int p0 = (blockIdx.x * SORT_WAVES + wave) * (64 * STEPS) + lane;
  int id[STEPS], place[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int p = p0 + s * 64;
    id[s] = p < P ? a.ids[p] : -1;
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const bool ok = (uint32_t)id[s] < (uint32_t)E;
    const int e = ok ? id[s] : 0;
    const uint64_t same = match_lanes(e, ok, bits);
    const int below = __popcll(same & ((1ull << lane) - 1));
    // (the wave's LDS accesses complete in order: every lane reads the count before the
    // lowest of its equals writes the new one, and the next step reads that)
    const int c = cnt[wave][e];
    place[s] = ok ? c + below : -1;
    if (ok && below == 0) cnt[wave][e] = (uint16_t)(c + __popcll(same));
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // this workgroup's count of expert tid, and the waves' offsets in it
  int mine = 0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int c = cnt[w][tid];
      cnt[w][tid] = (uint16_t)mine;
      mine += c;
    }
  }
  if (MODE == SORT_COUNT) {
    if (tid < E) a.hist[(size_t)blockIdx.x * E + tid] = mine;
    return;
  }
  int before = 0, all = mine;
  if (MODE == SORT_PLACE && tid < E) {
    all = 0;
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int c = a.hist[(size_t)b * E + tid];
      if (b < (int)blockIdx.x) before += c;
      all += c;
    }
  }
  const int inc = wave_incl_scan(all);
  if (lane == 63) wave_tot[wave] = inc;
  __syncthreads();
  int below_waves = 0, total = 0;
#pragma unroll
  for (int w = 0; w < SORT_WAVES; ++w) {
    const int c = wave_tot[w];
    if (w < wave) below_waves += c;
    total += c;
  }
  const int first = below_waves + inc - all;
  if (tid < E) {
    base[tid] = first + before;
    if (blockIdx.x == 0) a.start[tid] = first;
  }
  if (blockIdx.x == 0 && tid == 0) a.start[E] = total;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int p = p0 + s * 64;
    if (p >= P) continue;
    int row = -1;
    if (place[s] >= 0) {
      row = base[id[s]] + cnt[wave][id[s]] + place[s];
      a.row_pair[row] = p;
    }
    a.pair_row[p] = row;
    if (p >= total) a.row_pair[p] = -1;  // rows behind the last expert's (written by no pair)
  }
}

hipError_t launch_sort(const SortArgs& a, hipStream_t st) {
  const int nb = sort_blocks(a.P);
  const bool few = sort_steps(a.P) == 4;
  if (nb <= 1) {
    if (few) sort_kernel<4, SORT_ALL><<<1, SORT_THREADS, 0, st>>>(a);
    else sort_kernel<16, SORT_ALL><<<1, SORT_THREADS, 0, st>>>(a);
    return hipGetLastError();
  }
  if (few) {
    sort_kernel<4, SORT_COUNT><<<nb, SORT_THREADS, 0, st>>>(a);
    sort_kernel<4, SORT_PLACE><<<nb, SORT_THREADS, 0, st>>>(a);
  } else {
    sort_kernel<16, SORT_COUNT><<<nb, SORT_THREADS, 0, st>>>(a);
    sort_kernel<16, SORT_PLACE><<<nb, SORT_THREADS, 0, st>>>(a);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------------------

// N consecutive elements of a bf16 (uint16_t) or fp32 row, as fp32.  N > 1: the address is
// a multiple of N elements' bytes, at most 16.
template <int N>
__device__ __forceinline__ void load_n(const uint16_t* p, float* v) {
  if constexpr (N == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) { v[2 * q] = bf16_bits_to_f32(w[q] & 0xFFFFu); v[2 * q + 1] = __builtin_bit_cast(float, w[q] & 0xFFFF0000u); }
  } else if constexpr (N == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16_bits_to_f32(u.x & 0xFFFFu); v[1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
    v[2] = bf16_bits_to_f32(u.y & 0xFFFFu); v[3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
  } else {
    static_assert(N == 1, "elements per load");
    v[0] = bf16_bits_to_f32(*p);
  }
}
template <int N>
__device__ __forceinline__ void load_n(const float* p, float* v) {
  if constexpr (N == 1) {
    v[0] = *p;
  } else {
    static_assert(N % 4 == 0, "elements per load");
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 u = reinterpret_cast<const float4*>(p)[q];
      v[4 * q] = u.x; v[4 * q + 1] = u.y; v[4 * q + 2] = u.z; v[4 * q + 3] = u.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t* p, const float* v) {
  if constexpr (N == 1) {
    *p = f32_to_bf16_rne(v[0]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int q = 0; q < N / 2; ++q)
      w[q] = (uint32_t)f32_to_bf16_rne(v[2 * q]) | ((uint32_t)f32_to_bf16_rne(v[2 * q + 1]) << 16);
    if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float* v) {
  if constexpr (N == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  }
}

constexpr int ROW_THREADS = 256;

// Units of a row over a workgroup's threads: TX of them side by side on one token (a power
// of two, so a narrow row does not leave lanes idle), 256 / TX tokens.
struct RowGrid {
  int tx_log, nbx;
  unsigned grid;
};
static RowGrid row_grid(int units, int T) {
  RowGrid g{};
  while (g.tx_log < 8 && (1 << g.tx_log) < units) ++g.tx_log;
  g.nbx = (units + (1 << g.tx_log) - 1) >> g.tx_log;
  const int ty = ROW_THREADS >> g.tx_log;
  g.grid = (unsigned)g.nbx * (unsigned)((T + ty - 1) / ty);
  return g;
}
__device__ __forceinline__ void row_pos(int tx_log, int nbx, int& t, int& u) {
  const int bx = blockIdx.x % nbx, bt = blockIdx.x / nbx;
  t = bt * (ROW_THREADS >> tx_log) + ((int)threadIdx.x >> tx_log);
  u = (bx << tx_log) + ((int)threadIdx.x & ((1 << tx_log) - 1));
}

// xs[row(t,i)] = x[t] for the token's k pairs, in units of type U.  Bound by the k row
// writes; the token's row is read once.
template <typename U>
__global__ __launch_bounds__(ROW_THREADS) void gather_kernel(RowsArgs a, int units, int tx_log, int nbx) {
  int t, u;
  row_pos(tx_log, nbx, t, u);
  if (t >= a.T || u >= units) return;
  const U v = static_cast<const U*>(a.x)[(size_t)t * units + u];
  const int32_t* at = a.pair_row + (size_t)t * a.k;
  const int P = a.T * a.k;
  for (int i = 0; i < a.k; ++i) {
    const int r = at[i];
    if ((uint32_t)r < (uint32_t)P) static_cast<U*>(a.y)[(size_t)r * units + u] = v;
  }
}

hipError_t launch_gather(const RowsArgs& a, int dtype, hipStream_t st) {
  const size_t bytes = (size_t)a.C * (dtype == MOE_VQ_BF16 ? 2 : 4);
  auto go = [&](auto unit) {
    using U = decltype(unit);
    const int units = (int)(bytes / sizeof(U));
    const RowGrid g = row_grid(units, a.T);
    gather_kernel<U><<<g.grid, ROW_THREADS, 0, st>>>(a, units, g.tx_log, g.nbx);
  };
  // (a row of an odd width starts anywhere: the widest unit that divides its bytes)
  if (bytes % 16 == 0) go(uint4{});
  else if (bytes % 4 == 0) go(uint32_t{});
  else go(uint16_t{});
  return hipGetLastError();
}

// y[t] = add[t] + sum_i w_i rows[row_i], N columns per thread, fp32 sums in the order of i.
// Eight rows' loads are issued before the first is used; a dropped pair's load is
// redirected to row 0 and its value dropped (selected, not multiplied: it may hold NaN).
template <typename TR, typename TY, int N>
__global__ __launch_bounds__(ROW_THREADS) void combine_rows_kernel(RowsArgs a, int units, int tx_log, int nbx) {
  int t, u;
  row_pos(tx_log, nbx, t, u);
  if (t >= a.T || u >= units) return;
  const int k = a.k, P = a.T * k;
  const size_t C = (size_t)a.C, col = (size_t)u * N;
  const TR* rows = static_cast<const TR*>(a.x);
  const int32_t* at = a.pair_row + (size_t)t * k;
  const float* wt = a.pair_w ? a.pair_w + (size_t)t * k : nullptr;
  float acc[N];
  if (a.add) {
    load_n<N>(static_cast<const TY*>(a.add) + (size_t)t * C + col, acc);
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q) acc[q] = 0.f;
  }
  for (int i0 = 0; i0 < k; i0 += 8) {
    float v[8][N], w[8];
    bool ok[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = i0 + i < k ? i0 + i : k - 1;
      const int r = at[j];
      ok[i] = i0 + i < k && (uint32_t)r < (uint32_t)P;
      w[i] = wt ? wt[j] : 1.f;
      load_n<N>(rows + (ok[i] ? (size_t)r : 0) * C + col, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < N; ++q) acc[q] = ok[i] ? fmaf(w[i], v[i][q], acc[q]) : acc[q];
  }
  store_n<N>(static_cast<TY*>(a.y) + (size_t)t * C + col, acc);
}

template <typename TR, typename TY>
static void combine_go(const RowsArgs& a, hipStream_t st) {
  constexpr int N = 16 / sizeof(TR);
  const bool vec = a.C % N == 0;
  const int units = vec ? a.C / N : a.C;
  const RowGrid g = row_grid(units, a.T);
  if (vec) combine_rows_kernel<TR, TY, N><<<g.grid, ROW_THREADS, 0, st>>>(a, units, g.tx_log, g.nbx);
  else combine_rows_kernel<TR, TY, 1><<<g.grid, ROW_THREADS, 0, st>>>(a, units, g.tx_log, g.nbx);
}

hipError_t launch_combine_rows(const RowsArgs& a, int dtype, int y_dtype, hipStream_t st) {
  if (dtype == MOE_VQ_BF16) {
    if (y_dtype == MOE_VQ_BF16) combine_go<uint16_t, uint16_t>(a, st);
    else combine_go<uint16_t, float>(a, st);
  } else {
    if (y_dtype == MOE_VQ_BF16) combine_go<float, uint16_t>(a, st);
    else combine_go<float, float>(a, st);
  }
  return hipGetLastError();
}

// Gradients of combine for PG pairs of one token: drows[row_i] = w_i dy[t] and
// dw_i = <dy[t], rows[row_i]>, so dy[t] is read once for PG rows.  One workgroup walks the
// columns; the PG sums of each thread meet in LDS at the end.
template <typename TR, typename TY, int N, int PG>
__global__ __launch_bounds__(ROW_THREADS) void combine_rows_bwd_kernel(RowsArgs a) {
  __shared__ float red[ROW_THREADS / 64][PG];
  const int ng = (a.k + PG - 1) / PG;
  const int t = blockIdx.x / ng, i0 = (blockIdx.x % ng) * PG;
  const int k = a.k, P = a.T * k;
  const size_t C = (size_t)a.C;
  const TR* rows = static_cast<const TR*>(a.x);
  const TY* dy = static_cast<const TY*>(a.add) + (size_t)t * C;
  TR* drows = static_cast<TR*>(a.y);
  size_t off[PG];
  float w[PG], sum[PG];
  bool ok[PG];
#pragma unroll
  for (int i = 0; i < PG; ++i) {
    const int j = i0 + i < k ? i0 + i : k - 1;
    const int r = a.pair_row[(size_t)t * k + j];
    ok[i] = i0 + i < k && (uint32_t)r < (uint32_t)P;
    off[i] = (ok[i] ? (size_t)r : 0) * C;
    w[i] = a.pair_w ? a.pair_w[(size_t)t * k + j] : 1.f;
    sum[i] = 0.f;
  }
  for (int c = threadIdx.x * N; c < a.C; c += ROW_THREADS * N) {
    float g[N];
    load_n<N>(dy + c, g);
    if (a.dw) {
      float v[PG][N];
#pragma unroll
      for (int i = 0; i < PG; ++i) load_n<N>(rows + off[i] + c, v[i]);
#pragma unroll
      for (int i = 0; i < PG; ++i)
#pragma unroll
        for (int q = 0; q < N; ++q) sum[i] = fmaf(g[q], v[i][q], sum[i]);
    }
    if (drows) {
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        float v[N];
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = w[i] * g[q];
        if (ok[i]) store_n<N>(drows + off[i] + c, v);
      }
    }
  }
  if (!a.dw) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < PG; ++i) {
    const float s = wave_sum(sum[i]);
    if (lane == 0) red[wave][i] = s;
  }
  __syncthreads();
  if (threadIdx.x < PG && i0 + (int)threadIdx.x < k) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < ROW_THREADS / 64; ++v) s += red[v][threadIdx.x];
    const size_t p = (size_t)t * k + i0 + threadIdx.x;
    a.dw[p] = (uint32_t)a.pair_row[p] < (uint32_t)P ? s : 0.f;  // (a dropped pair's weight moved nothing)
  }
}

template <typename TR, typename TY>
static void combine_bwd_go(const RowsArgs& a, hipStream_t st) {
  constexpr int N = 16 / sizeof(TR);
  const bool vec = a.C % N == 0;
  // Eight pairs share one read of dy; a small batch takes one pair per workgroup instead,
  // so that it still fills the device.
  const bool wide = (long)a.T * ((a.k + 7) / 8) >= 512;
  const int ng = wide ? (a.k + 7) / 8 : a.k;
  const unsigned grid = (unsigned)a.T * (unsigned)ng;
  if (vec && wide) combine_rows_bwd_kernel<TR, TY, N, 8><<<grid, ROW_THREADS, 0, st>>>(a);
  else if (vec) combine_rows_bwd_kernel<TR, TY, N, 1><<<grid, ROW_THREADS, 0, st>>>(a);
  else if (wide) combine_rows_bwd_kernel<TR, TY, 1, 8><<<grid, ROW_THREADS, 0, st>>>(a);
  else combine_rows_bwd_kernel<TR, TY, 1, 1><<<grid, ROW_THREADS, 0, st>>>(a);
}

hipError_t launch_combine_rows_backward(const RowsArgs& a, int dtype, int dy_dtype, hipStream_t st) {
  if (dtype == MOE_VQ_BF16) {
    if (dy_dtype == MOE_VQ_BF16) combine_bwd_go<uint16_t, uint16_t>(a, st);
    else combine_bwd_go<uint16_t, float>(a, st);
  } else {
    if (dy_dtype == MOE_VQ_BF16) combine_bwd_go<float, uint16_t>(a, st);
    else combine_bwd_go<float, float>(a, st);
  }
  return hipGetLastError();
}

}  // namespace mvq
