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
    for (int b0 = 0; b0 < (int)gridDim.x; b0 += 8) {  // (eight loads at once; behind the last, its count again)
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = b0 + i < (int)gridDim.x ? b0 + i : (int)gridDim.x - 1;
        c[i] = a.hist[(size_t)b * E + tid];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (b0 + i < (int)blockIdx.x) before += c[i];
        if (b0 + i < (int)gridDim.x) all += c[i];
      }
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

// At most 64 pairs: every lane holds one and counts the pairs before it (smaller expert, or the same and an
// earlier pair); the rest of the work, the experts' first rows, is counted the same way.
// Measured 3.8 us for one token's eight pairs, where the counting sort takes 5.0.
constexpr int SORT_FEW = 64;

__global__ __launch_bounds__(256) void sort_few_kernel(SortArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, E = a.E, P = a.P;
  const int id = lane < P ? a.ids[lane] : -1;
  const bool ok = (uint32_t)id < (uint32_t)E;
  const int key = ok ? id : E;
  const int total = __popcll(__ballot(ok));
  if (tid < 64) {
    int row = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const int k = __builtin_amdgcn_readlane(key, j);
      row += (k < key || (k == key && j < lane)) ? 1 : 0;
    }
    if (lane < P) {
      a.pair_row[lane] = ok ? row : -1;
      if (ok) a.row_pair[row] = lane;
      if (lane >= total) a.row_pair[lane] = -1;
    }
  }
  for (int e0 = 0; e0 <= E; e0 += 256) {
    int first = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j) first += __builtin_amdgcn_readlane(key, j) < e0 + tid ? 1 : 0;
    if (e0 + tid <= E) a.start[e0 + tid] = first;
  }
}

hipError_t launch_sort(const SortArgs& a, hipStream_t st) {
  if (a.P <= SORT_FEW) {
    sort_few_kernel<<<1, 256, 0, st>>>(a);
    return hipGetLastError();
  }
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

// N consecutive elements of a bf16 (uint16_t) or fp32 row, as fp32.  STREAM: for rows that no cache would
// hold until they are read again.
template <int N, bool STREAM>
__device__ __forceinline__ void load_n(const uint16_t* p, float* v) {
  if constexpr (N == 1) {
    v[0] = bf16_bits_to_f32(*p);
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const u32x4_any u = load_vec<STREAM>(reinterpret_cast<const u32x4_any*>(p));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
      const u32x2_any u = load_vec<STREAM>(reinterpret_cast<const u32x2_any*>(p));
      w[0] = u.x; w[1] = u.y;
    }
#pragma unroll
    for (int q = 0; q < N / 2; ++q) {
      v[2 * q] = bf16_bits_to_f32(w[q] & 0xFFFFu);
      v[2 * q + 1] = __builtin_bit_cast(float, w[q] & 0xFFFF0000u);
    }
  }
}
template <int N, bool STREAM>
__device__ __forceinline__ void load_n(const float* p, float* v) {
  if constexpr (N == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const f32x4_any u = load_vec<STREAM>(reinterpret_cast<const f32x4_any*>(p + q));
      v[q] = u.x; v[q + 1] = u.y; v[q + 2] = u.z; v[q + 3] = u.w;
    }
  }
}
template <int N, bool STREAM>
__device__ __forceinline__ void store_n(uint16_t* p, const float* v) {
  if constexpr (N == 1) {
    *p = f32_to_bf16_rne(v[0]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int q = 0; q < N / 2; ++q) w[q] = pack_bf16(v[2 * q], v[2 * q + 1]);
    if constexpr (N == 8) store_vec<STREAM>(reinterpret_cast<u32x4_any*>(p), u32x4_any{w[0], w[1], w[2], w[3]});
    else store_vec<STREAM>(reinterpret_cast<u32x2_any*>(p), u32x2_any{w[0], w[1]});
  }
}
template <int N, bool STREAM>
__device__ __forceinline__ void store_n(float* p, const float* v) {
  if constexpr (N == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int q = 0; q < N; q += 4)
      store_vec<STREAM>(reinterpret_cast<f32x4_any*>(p + q), f32x4_any{v[q], v[q + 1], v[q + 2], v[q + 3]});
  }
}

// Rows of more bytes than the memory-side cache holds are streamed: gather 90 us instead of 114,
// combine 123 instead of 141 with an fp32 residual, 96 instead of 130 in bf16 alone (470 MB of rows); smaller ones
// stay where the next kernel finds them.  Streamed rows are fastest with workgroups of 128 threads (gather
// 90 us, 256 threads 98; combine 123, 131), rows that a cache holds a little faster with 256 (combine of 32 tokens
// of 7168 fp32 columns, top-8: 4.0 us, 4.3 with 128; of 1021 tokens of 2047 columns, top-6: 17 either way).
constexpr int row_threads_log(bool stream) { return stream ? 7 : 8; }
static bool streamed(const RowsArgs& a, size_t size) { return (size_t)a.T * a.k * a.C * size > ((size_t)256 << 20); }

// Units of a row over a workgroup's threads: TX of them side by side on one token (a power
// of two, so a narrow row does not leave lanes idle), and the other threads on other tokens.
struct RowGrid {
  int tx_log, nbx;
  unsigned grid;
};
static RowGrid row_grid(int units, int T, bool stream) {
  RowGrid g{};
  while (g.tx_log < row_threads_log(stream) && (1 << g.tx_log) < units) ++g.tx_log;
  g.nbx = (units + (1 << g.tx_log) - 1) >> g.tx_log;
  const int ty = 1 << (row_threads_log(stream) - g.tx_log);
  g.grid = (unsigned)g.nbx * (unsigned)((T + ty - 1) / ty);
  return g;
}
__device__ __forceinline__ void row_pos(int tx_log, int nbx, int& t, int& u) {
  const int bx = blockIdx.x % nbx, bt = blockIdx.x / nbx;
  t = bt * ((int)blockDim.x >> tx_log) + ((int)threadIdx.x >> tx_log);
  u = (bx << tx_log) + ((int)threadIdx.x & ((1 << tx_log) - 1));
}

// xs[row(t,i)] = x[t] for the token's k pairs, 16 bytes per thread (the row's last ones by element).  Bound by
// the k row writes; the token's row is read once.
template <bool STREAM>
__global__ __launch_bounds__(1 << row_threads_log(STREAM)) void gather_kernel(RowsArgs a, size_t bytes, int units, int tx_log, int nbx) {
  int t, u;
  row_pos(tx_log, nbx, t, u);
  if (t >= a.T || u >= units) return;
  const size_t at = (size_t)u * 16;
  const char* from = static_cast<const char*>(a.x) + (size_t)t * bytes + at;
  char* to = static_cast<char*>(a.y) + at;
  const int32_t* row = a.pair_row + (size_t)t * a.k;
  const int P = a.T * a.k;
  if (at + 16 <= bytes) {
    const u32x4_any v = *reinterpret_cast<const u32x4_any*>(from);  // (streaming the loads too: 101 us)
    for (int i = 0; i < a.k; ++i) {
      const int r = row[i];
      if ((uint32_t)r < (uint32_t)P) store_vec<STREAM>(reinterpret_cast<u32x4_any*>(to + (size_t)r * bytes), v);
    }
  } else {
    const int n = (int)(bytes - at) / 2;  // (an element is two bytes, or four)
    for (int i = 0; i < a.k; ++i) {
      const int r = row[i];
      if ((uint32_t)r >= (uint32_t)P) continue;
      for (int j = 0; j < n; ++j)
        reinterpret_cast<uint16_t*>(to + (size_t)r * bytes)[j] = reinterpret_cast<const uint16_t*>(from)[j];
    }
  }
}

hipError_t launch_gather(const RowsArgs& a, int dtype, hipStream_t st) {
  const size_t bytes = (size_t)a.C * (dtype == MOE_VQ_BF16 ? 2 : 4);
  const int units = (int)((bytes + 15) / 16);
  auto go = [&](auto stream) {
    constexpr bool S = decltype(stream)::value;
    const RowGrid g = row_grid(units, a.T, S);
    gather_kernel<S><<<g.grid, 1 << row_threads_log(S), 0, st>>>(a, bytes, units, g.tx_log, g.nbx);
  };
  if (streamed(a, bytes / a.C)) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

// y[t] = add[t] + sum_i w_i rows[row_i], N columns per thread, fp32 sums in the order of i.
// Eight rows' loads are issued before the first is used; a dropped pair's load is
// redirected to row 0 and its value dropped (selected, not multiplied: it may hold NaN).
template <typename TR, typename TY, int N, bool STREAM>
__device__ __forceinline__ void combine_columns(const RowsArgs& a, int t, size_t col) {
  const int k = a.k, P = a.T * k;
  const size_t C = (size_t)a.C;
  const TR* rows = static_cast<const TR*>(a.x);
  const int32_t* at = a.pair_row + (size_t)t * k;
  const float* wt = a.pair_w ? a.pair_w + (size_t)t * k : nullptr;
  float acc[N];
  if (a.add) {
    load_n<N, STREAM>(static_cast<const TY*>(a.add) + (size_t)t * C + col, acc);
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
      load_n<N, STREAM>(rows + (ok[i] ? (size_t)r : 0) * C + col, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < N; ++q) acc[q] = ok[i] ? fmaf(w[i], v[i][q], acc[q]) : acc[q];
  }
  store_n<N, STREAM>(static_cast<TY*>(a.y) + (size_t)t * C + col, acc);
}

template <typename TR, typename TY, int N, bool STREAM>
__global__ __launch_bounds__(1 << row_threads_log(STREAM)) void combine_rows_kernel(RowsArgs a, int units, int tx_log, int nbx) {
  int t, u;
  row_pos(tx_log, nbx, t, u);
  if (t >= a.T || u >= units) return;
  const int whole = a.C / N;  // units of N columns; the first threads take one more column each behind them
  if (u < whole) combine_columns<TR, TY, N, STREAM>(a, t, (size_t)u * N);
  if (u < a.C - whole * N) combine_columns<TR, TY, 1, STREAM>(a, t, (size_t)whole * N + u);
}

template <typename TR, typename TY>
static void combine_go(const RowsArgs& a, hipStream_t st) {
  constexpr int N = 16 / sizeof(TR);
  const int units = a.C / N > a.C % N ? a.C / N : a.C % N;
  auto go = [&](auto stream) {
    constexpr bool S = decltype(stream)::value;
    const RowGrid g = row_grid(units, a.T, S);
    combine_rows_kernel<TR, TY, N, S><<<g.grid, 1 << row_threads_log(S), 0, st>>>(a, units, g.tx_log, g.nbx);
  };
  if (streamed(a, sizeof(TR))) go(std::true_type{});
  else go(std::false_type{});
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
constexpr int BWD_THREADS = 256;

template <typename TR, typename TY, int N, int PG, bool STREAM>
__global__ __launch_bounds__(BWD_THREADS) void combine_rows_bwd_kernel(RowsArgs a) {
  __shared__ float red[BWD_THREADS / 64][PG];
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
  // W columns from c on: all loads first, then the sums, then the stores
  auto columns = [&](auto width, auto with_dw, int c) {
    constexpr int W = decltype(width)::value;
    constexpr bool DW = decltype(with_dw)::value;
    float g[W], v[PG][W];
    load_n<W, STREAM>(dy + c, g);
    if constexpr (DW) {
#pragma unroll
      for (int i = 0; i < PG; ++i) load_n<W, STREAM>(rows + off[i] + c, v[i]);
      __builtin_amdgcn_sched_group_barrier(0x020, 2 * PG + 2, 0);
#pragma unroll
      for (int i = 0; i < PG; ++i)
#pragma unroll
        for (int q = 0; q < W; ++q) sum[i] = fmaf(g[q], v[i][q], sum[i]);
    }
    if (drows) {
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        float d[W];
#pragma unroll
        for (int q = 0; q < W; ++q) d[q] = w[i] * g[q];
        if (ok[i]) store_n<W, STREAM>(drows + off[i] + c, d);
      }
    }
  };
  auto all = [&](auto with_dw) {
    for (int c = threadIdx.x * N; c + N <= a.C; c += BWD_THREADS * N) columns(std::integral_constant<int, N>{}, with_dw, c);
    const int last = a.C / N * N + threadIdx.x;  // the columns behind the last N, one per thread
    if (last < a.C) columns(std::integral_constant<int, 1>{}, with_dw, last);
  };
  if (a.dw) all(std::true_type{});
  else all(std::false_type{});
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
    for (int v = 0; v < BWD_THREADS / 64; ++v) s += red[v][threadIdx.x];
    const size_t p = (size_t)t * k + i0 + threadIdx.x;
    a.dw[p] = (uint32_t)a.pair_row[p] < (uint32_t)P ? s : 0.f;  // (a dropped pair's weight moved nothing)
  }
}

template <typename TR, typename TY>
static void combine_bwd_go(const RowsArgs& a, hipStream_t st) {
  constexpr int N = 16 / sizeof(TR);
  // Eight pairs share one read of dy; a small batch takes one pair per workgroup instead,
  // so that it still fills the device.
  const bool wide = (long)a.T * ((a.k + 7) / 8) >= 512;
  const int ng = wide ? (a.k + 7) / 8 : a.k;
  const unsigned grid = (unsigned)a.T * (unsigned)ng;
  if (wide && streamed(a, sizeof(TR))) combine_rows_bwd_kernel<TR, TY, N, 8, true><<<grid, BWD_THREADS, 0, st>>>(a);
  else if (wide) combine_rows_bwd_kernel<TR, TY, N, 8, false><<<grid, BWD_THREADS, 0, st>>>(a);
  else combine_rows_bwd_kernel<TR, TY, N, 1, false><<<grid, BWD_THREADS, 0, st>>>(a);
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
