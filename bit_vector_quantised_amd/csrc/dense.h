// Arguments and launches of the row operators (rows.hip) and of the dense product
// (linear.hip); the entry points that check and call them are in dense_api.hip.
#pragma once

#include "block.h"

namespace mvq {

// A failed HIP call recorded for moe_vq_last_hip_error() and mapped to MOE_VQ_EHIP (api.hip).
int hip_status(hipError_t e);

constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;

// Pairs one workgroup of the sort takes: few enough that a large sort fills some CUs, so
// many that every workgroup can add up all workgroups' counts by itself (at most 128 of them).
__host__ __device__ constexpr int sort_steps(int P) { return P <= 4096 ? 4 : (P <= 16384 ? 16 : (P <= 131072 ? 4 : 16)); }
__host__ __device__ constexpr int sort_blocks(int P) {
  const int per = sort_steps(P) * SORT_THREADS;
  return (P + per - 1) / per;
}

struct SortArgs {
  const int32_t* ids;  // [P]
  int P, E;
  int32_t* start;      // [E + 1]
  int32_t* pair_row;   // [P]
  int32_t* row_pair;   // [P]
  int32_t* hist;       // [blocks][E], more than one block only
};
hipError_t launch_sort(const SortArgs& a, hipStream_t st);

struct RowsArgs {
  const int32_t* pair_row;  // [T*k]
  const float* pair_w;      // [T*k] or null
  const void* x;            // gather: x [T][C]; combine, backward: the experts' rows [T*k][C]
  const void* add;          // combine: residual [T][C] or null; backward: dy [T][C]
  void* y;                  // gather, backward: rows [T*k][C]; combine: y [T][C]
  float* dw;                // backward: [T*k] or null
  int T, k, C;
};
hipError_t launch_gather(const RowsArgs& a, int dtype, hipStream_t st);
hipError_t launch_combine_rows(const RowsArgs& a, int dtype, int y_dtype, hipStream_t st);
hipError_t launch_combine_rows_backward(const RowsArgs& a, int dtype, int dy_dtype, hipStream_t st);

// One dense product, forward or backward, with its workspace offsets.
struct LinearPlan {
  int M, K, N, R, G;         // rows, n_in, n_out, weight rows (2 n_out for SWIGLU), groups
  int dtype, size;           // element type of x, w, z, dx, dw and its bytes
  int Kp, Rp;                // pitches (elements) of packed x / w and of dz: multiples of 16 bytes
  bool pack_k;               // x and w need repacking (K is no multiple of 16 bytes)
  struct Cut {
    int tile, splits;  // side of the square output tiles; parts of the contraction
  } fwd, dx, dw;
  bool few;                  // forward by the few-rows kernel, unless rows are in a table
  int split_bias;            // parts of a group's rows in the sums of dbias
  size_t xp, wp, dz, bias_part, part, dw_part, total;
};
// kept8: with room for x from 8 bits
LinearPlan linear_plan(const moe_vq_linear* L, int n_rows, bool backward, bool kept8 = false);
size_t linear_max_bytes(const moe_vq_linear* L, int n_rows, bool backward, bool kept8 = false);  // of every call with up to n_rows rows

struct LinearCall {
  const moe_vq_linear* L;
  const void* x;
  const int32_t* group_start;
  const void* residual;
  void* y;
  int y_dtype;
  void* z;            // forward: written if not null; backward: read
  const void* dy;
  void *dx, *dw;
  float* dbias;
  moe_vq_rows8 x8, z8;  // backward: x and z in 8 bits (q not null), instead of x and z
  void* ws;
};
hipError_t launch_linear_forward(const LinearPlan& p, const LinearCall& c, hipStream_t st);
hipError_t launch_linear_backward(const LinearPlan& p, const LinearCall& c, hipStream_t st);

}  // namespace mvq
