// Arguments and launches of the operators around the experts: the norm (norm.hip), the choice of experts
// (choose.hip) and rows kept in 8 bits (rows8.hip); the entry points that check and call them are
// in block_api.hip.
#pragma once

#include "moe_vq_internal.h"

namespace mvq {

struct NormArgs {
  const void* x;
  const void* res;    // [M][C] or null
  void* s;            // x + res, or null
  const float* gain;  // [C]
  void* y;            // or null
  uint8_t *q, *e;     // y in 8 bits (pitch rows8_pitch(C)), or null
  float eps;
  int M, C;
};
hipError_t launch_norm(const NormArgs& a, int dtype, int s_dtype, int y_dtype, hipStream_t st);

struct NormBackArgs {
  const void* s;
  const void *dy, *dy2;  // dy2 or null
  const void* ds;        // or null
  void* dx;              // or null
  const float* gain;
  float* dgain;          // or null
  float* part;           // [norm_back_blocks][C]
  float eps;
  int M, C;
};
int norm_back_blocks(int M, int C);
hipError_t launch_norm_back(const NormBackArgs& a, int dy_dtype, int s_dtype, int dx_dtype, hipStream_t st);

struct ChooseArgs {
  const float* logits;  // [T][E]
  const float* bias;    // [E] or null
  int32_t* ids;         // [T][k] (the gradient reads it)
  float* w;             // [T][k]; gradient: dw
  float* dlogits;       // gradient only
  int T, E, k, groups, top_groups, best;
  bool sigmoid, renorm;
  float scale;
};
hipError_t launch_choose(const ChooseArgs& a, hipStream_t st);
hipError_t launch_choose_back(const ChooseArgs& a, hipStream_t st);

// Bytes of a row in 8 bits (its scales: a 32nd of that).
__host__ __device__ constexpr size_t rows8_pitch(int cols) { return ((size_t)cols + 31) / 32 * 32; }

struct Rows8Args {
  const void* x;  // rows [M][C], packing
  void* y;        // rows [M][C] (gather: [M*k][C]), unpacking
  uint8_t *q, *e;
  const int32_t* start;     // rows outside start[0] .. start[G] are left alone; or null
  const int32_t* pair_row;  // gather: [M*k]; or null
  int M, C, k, G;
  size_t pitch;             // elements between rows of y (unpacking)
};
hipError_t launch_rows8_pack(const Rows8Args& a, int dtype, hipStream_t st);
hipError_t launch_rows8_unpack(const Rows8Args& a, int dtype, hipStream_t st);

struct ActBackArgs {
  const uint8_t *q, *e;     // z [rows][R]
  const int32_t* pair_row;  // [T*k]
  const float* w;           // [T*k] or null
  const void* dy;           // [rows][N]
  void *dz, *y;             // [rows][R], [rows][N]; each may be null
  float* dw;                // [T*k] or null
  int P, N, R, act;
  float lim;
};
hipError_t launch_act_back(const ActBackArgs& a, int dtype, int dy_dtype, hipStream_t st);

}  // namespace mvq
