// The dense product with bias, activation and residual in its epilogue, for one weight
// matrix or one per group of rows (the experts' products over sorted tokens), and its
// gradients:
//
//   forward   z = x W^T + b,  y = act(z) + r          contraction over n_in
//   dz        dz = dy * act'(z)                        element by element, and db = column sums
//   dx        dx = dz W                                contraction over the weight rows R
//   dw        dW_g = dz_g^T x_g                        contraction over the group's rows
//
// One kernel does the three products.  It is bound by the matrix cores once a tile's
// operands come from LDS often enough: a BM x BN tile moves (BM + BN) * 128 bytes through
// LDS for BM * BN * 128 / size products.  What differs is how an operand lies in memory:
//   "along"   the contraction runs along its rows (x and W forward, dz for dx)
//   "across"  the contraction runs across its rows (W for dx, dz and x for dw)
// A contraction step takes 128 bytes of an along operand's row (64 bf16 or 32 fp32 values) and
// as many rows of an across operand.  Both go from memory to LDS without passing through
// registers (16 bytes per lane).  The buffer descriptor ends at the last valid row, so what
// lies behind reads as zero: rows of the next group never enter a sum.
//
// Matrix instructions: bf16 v_mfma_f32_16x16x32_bf16; fp32 four v_mfma_f32_16x16x4_f32 per
// 16-byte chunk, chunk element j feeding the j-th, which permutes the contraction index
// the same way in both operands.  The weight rows take the instruction's row side, so that
// a lane ends with four consecutive output columns of one row.
#include <type_traits>

#include "dense.h"
#include "moe_vq_device.h"

namespace mvq {

namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

constexpr int STEP_BYTES = 128;  // an along operand's bytes per contraction step

// GATED: forward with SWIGLU, whose tile takes blocks of 16 gate rows and the matching 16 up rows.
enum GemmMode { GEMM_FWD = 0, GEMM_GATED = 1, GEMM_DX = 2, GEMM_DW = 3 };

struct GemmArgs {
  const char* a;  // FWD x, DX dz, DW dz
  const char* b;  // FWD w, DX w, DW x
  uint32_t a_pitch, b_pitch;  // bytes between rows
  uint64_t w_group;           // bytes between the groups' weights (FWD, DX)
  const int32_t* group_start;
  int G, M;   // groups; rows of x
  int kc;     // contraction length (FWD n_in, DX R; DW: the group's rows)
  int out_m, out_n;  // DW: rows and columns of dW; FWD, DX: out_n columns of the tile space
  int splits;
  float* part;  // splits > 1: fp32 partial sums [splits][rows][columns]
  // epilogue
  const float* bias;
  const void* res;
  void* out;
  void* z;
  int ldo;    // output columns
  int out_dtype, z_dtype, act;
  float lim;
};

// ---------------------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ float gelu(float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678f)); }
__device__ __forceinline__ float sigmoid_fast(float z) { return 1.0f / (1.0f + __expf(-z)); }

// d silu(z) / dz = s + z s (1 - s)
__device__ __forceinline__ float silu_grad(float z) {
  const float s = sigmoid_fast(z);
  return s * (1.0f + z * (1.0f - s));
}
// d gelu(z) / dz = Phi(z) + z phi(z)
__device__ __forceinline__ float gelu_grad(float z) {
  return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
}

// ---------------------------------------------------------------------------------------
// Element types
// ---------------------------------------------------------------------------------------

struct Bf16 {
  using T = uint16_t;
  static constexpr int SIZE = 2, UNIT = 32;  // UNIT: bytes of 16 values
  static __device__ __forceinline__ void mma(const u32x4_t& a, const u32x4_t& b, f32x4_t& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
};
struct F32 {
  using T = float;
  static constexpr int SIZE = 4, UNIT = 64;
  static __device__ __forceinline__ void mma(const u32x4_t& a, const u32x4_t& b, f32x4_t& c) {
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, av[j]), __builtin_bit_cast(float, bv[j]), c, 0, 0, 0);
  }
};

__device__ __forceinline__ float load_as_f32(const void* p, size_t i, int dtype) {
  return dtype == MOE_VQ_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_as(void* p, size_t i, int dtype, float v) {
  if (dtype == MOE_VQ_BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
  else static_cast<float*>(p)[i] = v;
}
// Up to four consecutive values from index i (n of them valid); as one access where wide.
__device__ __forceinline__ void load4(const void* p, size_t i, int dtype, int n, bool wide, float* v) {
  if (wide) {
    if (dtype == MOE_VQ_BF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      v[0] = bf16_bits_to_f32(u.x & 0xFFFFu); v[1] = bf16_bits_to_f32(u.x >> 16);
      v[2] = bf16_bits_to_f32(u.y & 0xFFFFu); v[3] = bf16_bits_to_f32(u.y >> 16);
    } else {
      const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? load_as_f32(p, i + j, dtype) : 0.f;
  }
}
__device__ __forceinline__ void store4(void* p, size_t i, int dtype, int n, bool wide, const float* v) {
  if (wide) {
    if (dtype == MOE_VQ_BF16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          make_uint2((uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16),
                     (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) store_as(p, i + j, dtype, v[j]);
  }
}

// Epilogue of four consecutive output columns n.. of output row m: bias, z, activation,
// residual, one rounding to the output's type.  v: the sums (SWIGLU: the gate's), u: the up
// sums.  z keeps the values before the activation, rounded once to its type.
template <bool GATED>
__device__ __forceinline__ void epilogue4(const GemmArgs& g, int grp, size_t m, int n, float* v, float* u) {
  const int left = g.ldo - n;
  const bool wide = (g.ldo & 3) == 0;  // (then left >= 4, and every row starts on a multiple of four)
  const size_t wrows = GATED ? 2 * (size_t)g.ldo : (size_t)g.ldo;
  if (g.bias) {
    const float* b = g.bias + grp * wrows;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < left) {
        v[j] += b[n + j];
        if (GATED) u[j] += b[(size_t)g.ldo + n + j];
      }
    }
  }
  if (g.z) {
    store4(g.z, m * wrows + n, g.z_dtype, left, wide, v);
    if (GATED) store4(g.z, m * wrows + g.ldo + n, g.z_dtype, left, wide, u);
  }
  if (GATED) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = swiglu(v[j], u[j], g.lim);
  } else if (g.act == MOE_VQ_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = silu_fast(v[j]);
  } else if (g.act == MOE_VQ_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = gelu(v[j]);
  }
  const size_t at = m * (size_t)g.ldo + n;
  if (g.res) {
    float r[4];
    load4(g.res, at, g.out_dtype, left, wide, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += r[j];
  }
  store4(g.out, at, g.out_dtype, left, wide, v);
}

// ---------------------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------------------

// Rows of group grp, clamped to the rows there are (the table is device data).
__device__ __forceinline__ void group_rows(const GemmArgs& g, int grp, int& r0, int& r1) {
  if (!g.group_start) { r0 = 0; r1 = g.M; return; }
  r0 = g.group_start[grp]; r1 = g.group_start[grp + 1];
  r0 = r0 < 0 ? 0 : (r0 > g.M ? g.M : r0);
  r1 = r1 < r0 ? r0 : (r1 > g.M ? g.M : r1);
}

// The workgroups of one XCD (every eighth) take neighbouring tiles, so that its L2 serves
// the operands they share.
__device__ __forceinline__ int xcd_order(int bid, int n) {
  const int x = bid & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (bid >> 3);
}

// Tile id -> (row tile, column tile): bands of eight row tiles, column by column within a band,
// so that 32 neighbouring tiles share eight row tiles and four column tiles.
__device__ __forceinline__ void band_order(int id, int mt, int nt, int& im, int& in) {
  constexpr int BAND = 8;
  const int band = id / (BAND * nt), rem = id - band * BAND * nt;
  const int h = mt - band * BAND < BAND ? mt - band * BAND : BAND;
  in = rem / h;
  im = band * BAND + (rem - in * h);
}

// LDS position of 16-byte chunk c (0..7) of an along operand's row: the chunks of a row are
// exchanged by its number so that the 16 rows a matrix operand reads at one chunk column lie
// in 16 different groups of four banks.
__device__ __forceinline__ int along_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// The same for an across operand's row, in units of 16 values (32 bytes of bf16, 64 of fp32):
// the rows that one read touches spread over the units of a 256-byte bank window.
template <typename E, int B>
__device__ __forceinline__ int across_swizzle(int row) {
  if (E::SIZE == 4) return (row >> 2) & 3;
  constexpr int UNITS = B * E::SIZE / E::UNIT;
  return UNITS >= 8 ? (row & 3) | ((row >> 1) & 4) : (row & 3) ^ ((row >> 3) & 1);
}

// This wave's loads into LDS have landed (vmcnt 0; the barrier after it then covers every wave's).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// One operand of a tile: B rows of output space (ALONG) or B columns (across), loaded by NW waves.
template <typename E, int B, bool ALONG, int NW>
struct Operand {
  static constexpr int BYTES = B * STEP_BYTES;
  static constexpr int LOADS = BYTES / 1024 / NW;     // 1 KiB per wave and load
  static constexpr int ROWB = B * E::SIZE;            // bytes of an across row
  static constexpr int KT = STEP_BYTES / E::SIZE;     // contraction values per step
  static_assert(LOADS >= 1 && LOADS * NW * 1024 == BYTES, "loads divide evenly over the waves");
  uint64_t base;    // address of this step's first byte
  uint32_t left;    // bytes from base to the end of what may be read
  uint32_t step, cut;  // bytes base advances per step; across: bytes of one row
  uint32_t off[LOADS];
  uint32_t tail[LOADS];  // along: first contraction value of the lane's chunk

  // along: the rows start at p, `bytes` of them may be read; row r of the tile is row
  // r, or with half > 0 the r-th of blocks of 16 gate rows and 16 up rows (half rows apart).
  __device__ __forceinline__ void init_along(const char* p, uint64_t bytes, uint32_t pitch, int half, int lane, int wave) {
    base = (uint64_t)p;
    left = (uint32_t)bytes;
    step = STEP_BYTES;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int q = wave * LOADS + j, row = q * 8 + (lane >> 3);
      const int c = (lane & 7) ^ along_swizzle(row);
      const int src = half ? ((row >> 4) & 1) * half + (row >> 5) * 16 + (row & 15) : row;
      off[j] = (uint32_t)src * pitch + c * 16;
      tail[j] = c * (16 / E::SIZE);
    }
  }
  // across: contraction rows from p on, `rows` of them; col: byte offset of the tile's first column.
  __device__ __forceinline__ void init_across(const char* p, uint32_t pitch, int col, int lane, int wave) {
    base = (uint64_t)p + col;
    step = (uint32_t)KT * pitch;
    cut = pitch;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int at = (wave * LOADS + j) * 1024 + lane * 16;
      const int row = at / ROWB, b = at % ROWB;
      const int unit = (b / E::UNIT) ^ across_swizzle<E, B>(row);
      off[j] = (uint32_t)row * pitch + unit * E::UNIT + b % E::UNIT;
    }
  }
  __device__ __forceinline__ void issue(lds_char* lds, uint32_t avail, int rest, int wave) const {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)avail, 0x00020000);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      // (a chunk behind the end of an along row is sent out of range, which reads as zero)
      const uint32_t o = ALONG && (int)tail[j] >= rest ? 0x80000000u : off[j];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * LOADS + j) * 1024), 16, o, 0, 0, 0);
    }
  }
  // Load the step that has `rest` contraction values left (across: rows), and move on.
  __device__ __forceinline__ void load(lds_char* lds, int rest, int wave) {
    if (ALONG) {
      issue(lds, left, rest, wave);
      base += step;
      left -= left < step ? left : step;
    } else {
      const uint32_t rows = rest < KT ? rest : KT;
      // (the descriptor starts at the tile's first column and ends with the last row)
      issue(lds, rows * cut - left, rest, wave);
      base += step;
    }
  }
  // Matrix operand f (16 rows or columns of output space) of half-step s.
  static __device__ __forceinline__ u32x4_t frag(const lds_char* lds, int f, int s, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if (ALONG) {
      const int row = f * 16 + i;
      const int c = (s * 4 + g) ^ along_swizzle(row);
      return *(const __attribute__((address_space(3))) u32x4_t*)(lds + row * STEP_BYTES + c * 16);
    } else if (E::SIZE == 2) {
      u32x2_t v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = s * 32 + g * 8 + h * 4 + (i >> 2);
        const int at = row * ROWB + (f ^ across_swizzle<E, B>(row)) * E::UNIT + (i & 3) * 8;
        v[h] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at)));
      }
      return u32x4_t{v[0].x, v[0].y, v[1].x, v[1].y};
    } else {
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = s * 16 + g * 4 + j;
        v[j] = *(const __attribute__((address_space(3))) uint32_t*)(lds + row * ROWB + (f ^ across_swizzle<E, B>(row)) * E::UNIT + i * 4);
      }
      return u32x4_t{v[0], v[1], v[2], v[3]};
    }
  }
};

template <typename E, int BM, int BN, int WM, int WN, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void gemm_kernel(GemmArgs g) {
  constexpr int NW = WM * WN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  using OpA = Operand<E, BM, MODE != GEMM_DW, NW>;
  constexpr bool GATED = MODE == GEMM_GATED, FORWARD = MODE == GEMM_FWD || GATED;
  static_assert(!GATED || FN % 2 == 0, "a wave holds gate and up of its columns");
  using OpB = Operand<E, BN, FORWARD, NW>;
  constexpr int KT = OpA::KT;
  __shared__ __align__(1024) char lds_mem[2 * (BM + BN) * STEP_BYTES];
  lds_char* lds = (lds_char*)lds_mem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // ---- which tile
  constexpr int per_n = GATED ? BN / 2 : BN;  // output columns of a tile
  const int nt = (g.out_n + per_n - 1) / per_n;
  int grp = 0, im, in, split, r0, r1, m0;
  if (MODE == GEMM_DW) {
    const int mt = (g.out_m + BM - 1) / BM;
    const int tiles = mt * nt * g.G;
    const int bid = xcd_order(blockIdx.x, tiles * g.splits);
    split = bid / tiles;
    const int id = bid - split * tiles;
    grp = id / (mt * nt);
    band_order(id - grp * mt * nt, mt, nt, im, in);
    group_rows(g, grp, r0, r1);
    m0 = im * BM;
  } else {
    // every lane counts the row tiles of its share of the groups
    const int q = (g.G + 63) / 64;
    int cnt = 0;
    for (int i = 0; i < q; ++i) {
      const int e = lane * q + i;
      if (e < g.G) {
        int a, b;
        group_rows(g, e, a, b);
        cnt += (b - a + BM - 1) / BM;
      }
    }
    const int inc = wave_incl_scan(cnt);
    const int mt = __builtin_amdgcn_readlane(inc, 63);
    const int tiles = mt * nt;
    if ((int)blockIdx.x >= tiles * g.splits) return;
    const int bid = xcd_order(blockIdx.x, tiles * g.splits);
    split = bid / tiles;
    band_order(bid - split * tiles, mt, nt, im, in);
    const int l = __popcll(__ballot(inc <= im));  // the lane whose groups hold row tile im
    int rel = im - (__builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(cnt, l));
    grp = l * q;
    for (;;) {
      group_rows(g, grp, r0, r1);
      const int n = (r1 - r0 + BM - 1) / BM;
      if (rel < n || grp + 1 >= g.G) break;
      rel -= n;
      ++grp;
    }
    m0 = r0 + rel * BM;
  }
  const int n0 = in * per_n;

  // ---- this split's part of the contraction
  const int kc = MODE == GEMM_DW ? r1 - r0 : g.kc;
  const int all_steps = (kc + KT - 1) / KT;
  const int per = (all_steps + g.splits - 1) / g.splits;
  const int s0 = split * per;
  const int steps = s0 >= all_steps ? 0 : (all_steps - s0 < per ? all_steps - s0 : per);
  const int k0 = s0 * KT;
  int rest = kc - k0;

  OpA a;
  OpB b;
  if (MODE != GEMM_DW) {
    const int rows = r1 - m0 < BM ? r1 - m0 : BM;
    a.init_along(g.a + (size_t)m0 * g.a_pitch, (uint64_t)rows * g.a_pitch, g.a_pitch, 0, lane, wave);
    a.base += (size_t)k0 * E::SIZE;
    a.left -= k0 * E::SIZE;
    const char* w = g.b + (size_t)grp * g.w_group;
    if (FORWARD) {
      const int wrows = GATED ? 2 * g.out_n : g.out_n;
      b.init_along(w + (size_t)n0 * g.b_pitch, (uint64_t)(wrows - n0) * g.b_pitch, g.b_pitch, GATED ? g.out_n : 0, lane, wave);
      b.base += (size_t)k0 * E::SIZE;
      b.left -= k0 * E::SIZE;
    } else {
      b.init_across(w + (size_t)k0 * g.b_pitch, g.b_pitch, n0 * E::SIZE, lane, wave);
      b.left = n0 * E::SIZE;
    }
  } else {
    a.init_across(g.a + (size_t)(r0 + k0) * g.a_pitch, g.a_pitch, m0 * E::SIZE, lane, wave);
    a.left = m0 * E::SIZE;
    b.init_across(g.b + (size_t)(r0 + k0) * g.b_pitch, g.b_pitch, n0 * E::SIZE, lane, wave);
    b.left = n0 * E::SIZE;
  }

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // ---- the contraction: the next step's operands arrive while this step is multiplied
  constexpr int STAGE = (BM + BN) * STEP_BYTES;
  if (steps > 0) {
    a.load(lds, rest, wave);
    b.load(lds + OpA::BYTES, rest, wave);
    rest -= KT;
  }
  wait_loads();
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    lds_char* cur = lds + (s & 1) * STAGE;
    lds_char* nxt = lds + ((s + 1) & 1) * STAGE;
    if (s + 1 < steps) {
      a.load(nxt, rest, wave);
      b.load(nxt + OpA::BYTES, rest, wave);
      rest -= KT;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = OpA::frag(cur, wm * FM + i, h, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = OpB::frag(cur + OpA::BYTES, wn * FN + j, h, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) E::mma(fb[j], fa[i], acc[i][j]);
    }
    wait_loads();
    __syncthreads();
  }

  // ---- outputs, 16 rows at a time: lane (i, g) of matrix (fm, fn) holds row 16 fm + i, columns
  // 16 fn + 4 g ..; through the wave's own part of LDS neighbouring lanes get neighbouring columns
  // of one row, so that rows leave in long runs
  constexpr int PITCH = FN * 16 + 4;
  constexpr int COLS = GATED ? FN * 8 : FN * 16;  // output columns of the wave
  constexpr int QUADS = COLS / 4;
  static_assert(NW * 16 * PITCH * 4 <= (int)sizeof(lds_mem), "output staging");
  float* stage = reinterpret_cast<float*>(lds_mem) + wave * 16 * PITCH;
  const int m_end = MODE == GEMM_DW ? g.out_m : r1;
  const size_t out_rows = MODE == GEMM_DW ? (size_t)g.G * g.out_m : (size_t)g.M;
  static_for<0, FM>([&](auto fi) {
    constexpr int i = decltype(fi)::value;
    static_for<0, FN>([&](auto fj) {
      constexpr int j = decltype(fj)::value;
      *reinterpret_cast<f32x4_t*>(stage + (lane & 15) * PITCH + j * 16 + (lane >> 4) * 4) = acc[i][j];
    });
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
    for (int t = lane; t < 16 * QUADS; t += 64) {
      const int rr = t / QUADS, c = (t % QUADS) * 4;
      const int m = m0 + (wm * FM + i) * 16 + rr, n = n0 + wn * COLS + c;
      if (m >= m_end || n >= g.out_n) continue;
      const size_t row = MODE == GEMM_DW ? (size_t)grp * g.out_m + m : (size_t)m;
      float v[4], u[4];
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(stage + rr * PITCH + (GATED ? (c >> 4) * 32 + (c & 15) : c));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = lo[q];
      if (GATED) {
        const f32x4_t up = *reinterpret_cast<const f32x4_t*>(stage + rr * PITCH + (c >> 4) * 32 + 16 + (c & 15));
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] = up[q];
      }
      if (g.splits > 1) {
        const size_t cols = GATED ? 2 * (size_t)g.out_n : (size_t)g.out_n;
        float* p = g.part + ((size_t)split * out_rows + row) * cols;
        store4(p, n, MOE_VQ_F32, g.out_n - n, (g.out_n & 3) == 0, v);
        if (GATED) store4(p, (size_t)g.out_n + n, MOE_VQ_F32, g.out_n - n, (g.out_n & 3) == 0, u);
      } else {
        epilogue4<GATED>(g, grp, row, n, v, u);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  });
}

// The sum of the splits' parts in order, then the epilogue: four columns per thread.
template <bool GATED>
__global__ __launch_bounds__(256) void split_sum_kernel(GemmArgs g, int rows) {
  const int units = (g.ldo + 3) / 4;
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (size_t)rows * units) return;
  const size_t m = at / units;
  const int n = (int)(at - m * units) * 4, left = g.ldo - n;
  const size_t cols = GATED ? 2 * (size_t)g.ldo : (size_t)g.ldo;
  const bool wide = (g.ldo & 3) == 0;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.splits; ++s) {
    const float* p = g.part + ((size_t)s * rows + m) * cols;
    float t[4];
    load4(p, n, MOE_VQ_F32, left, wide, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += t[j];
    if (GATED) {
      load4(p, (size_t)g.ldo + n, MOE_VQ_F32, left, wide, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] += t[j];
    }
  }
  epilogue4<GATED>(g, 0, m, n, v, u);
}

// ---------------------------------------------------------------------------------------
// Repacking rows whose width is no multiple of 16 bytes (dst pitch: the next one, zero-filled)
// ---------------------------------------------------------------------------------------

template <typename T>
__global__ __launch_bounds__(256) void pack_rows_kernel(const T* src, T* dst, size_t rows, int cols, int pitch) {
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= rows * (size_t)pitch) return;
  const size_t r = at / pitch;
  const int c = (int)(at - r * pitch);
  dst[at] = c < cols ? src[r * cols + c] : T(0);
}

// ---------------------------------------------------------------------------------------
// dz = dy * act'(z), and the column sums of dz per group
// ---------------------------------------------------------------------------------------

struct DzArgs {
  const void* dy;
  const void* z;
  void* dz;        // [M][pitch], or null (column sums only)
  float* bias;     // [splits][G][R] column sums, or null
  const int32_t* group_start;
  int M, N, R, G, pitch, splits;
  int dtype, dy_dtype, act;
  float lim;
};

constexpr int DZ_TX = 64, DZ_TY = 4;  // threads over columns, over rows

// One workgroup: DZ_TX * V columns of one split of one group's rows.  Bound by reading dy and z and
// writing dz, each once.  dz is rounded to the element type for the matrix products; the
// column sums add the unrounded values in fp32, rows in a fixed order.
template <int V>
__global__ __launch_bounds__(DZ_TX* DZ_TY) void dz_kernel(DzArgs a) {
  __shared__ float red[DZ_TY][2][DZ_TX * V];
  const int tx = threadIdx.x % DZ_TX, ty = threadIdx.x / DZ_TX;
  const int n = (blockIdx.x * DZ_TX + tx) * V;
  const int grp = blockIdx.y, split = blockIdx.z;
  int r0 = 0, r1 = a.M;
  if (a.group_start) {
    r0 = a.group_start[grp]; r1 = a.group_start[grp + 1];
    r0 = r0 < 0 ? 0 : (r0 > a.M ? a.M : r0);
    r1 = r1 < r0 ? r0 : (r1 > a.M ? a.M : r1);
  }
  const int per = (r1 - r0 + a.splits - 1) / a.splits;
  const int m0 = r0 + split * per, m1 = m0 + per < r1 ? m0 + per : r1;
  const bool two = a.act == MOE_VQ_ACT_SWIGLU;
  float sum[2][V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[0][j] = sum[1][j] = 0.f;
  if (n < a.N) {
    for (int m = m0 + ty; m < m1; m += DZ_TY) {
      float dy[V], zg[V], zu[V], dg[V], du[V];
      const size_t zrow = (size_t)m * a.R + n;
      if constexpr (V == 4) {
        load4(a.dy, (size_t)m * a.N + n, a.dy_dtype, 4, true, dy);
        if (a.act != MOE_VQ_ACT_NONE) load4(a.z, zrow, a.dtype, 4, true, zg);
        if (two) load4(a.z, zrow + a.N, a.dtype, 4, true, zu);
      } else {
        dy[0] = load_as_f32(a.dy, (size_t)m * a.N + n, a.dy_dtype);
        if (a.act != MOE_VQ_ACT_NONE) zg[0] = load_as_f32(a.z, zrow, a.dtype);
        if (two) zu[0] = load_as_f32(a.z, zrow + a.N, a.dtype);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (a.act == MOE_VQ_ACT_NONE) {
          dg[j] = dy[j];
        } else if (a.act == MOE_VQ_ACT_SILU) {
          dg[j] = dy[j] * silu_grad(zg[j]);
        } else if (a.act == MOE_VQ_ACT_GELU) {
          dg[j] = dy[j] * gelu_grad(zg[j]);
        } else {
          // h = silu(min(g, L)) * clamp(u, -L, L): no gradient through a value that was clamped
          float gv = zg[j], uv = zu[j];
          bool gin = true, uin = true;
          if (a.lim > 0.f) {
            gin = !(gv > a.lim);
            uin = !(uv > a.lim) && !(uv < -a.lim);
            gv = gin ? gv : a.lim;
            uv = uv > a.lim ? a.lim : (uv < -a.lim ? -a.lim : uv);
          }
          dg[j] = gin ? dy[j] * uv * silu_grad(gv) : 0.f;
          du[j] = uin ? dy[j] * silu_fast(gv) : 0.f;
          sum[1][j] += du[j];
        }
        sum[0][j] += dg[j];
      }
      if (a.dz) {
        const size_t row = (size_t)m * a.pitch;
        if constexpr (V == 4) {
          store4(a.dz, row + n, a.dtype, 4, true, dg);
          if (two) store4(a.dz, row + a.N + n, a.dtype, 4, true, du);
        } else {
          store_as(a.dz, row + n, a.dtype, dg[0]);
          if (two) store_as(a.dz, row + a.N + n, a.dtype, du[0]);
        }
        // (the pitch's last columns take part in dx's contraction as zeros)
        if (n == 0)
          for (int c = a.R; c < a.pitch; ++c) store_as(a.dz, row + c, a.dtype, 0.f);
      }
    }
  }
  if (!a.bias) return;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    red[ty][0][tx * V + j] = sum[0][j];
    red[ty][1][tx * V + j] = sum[1][j];
  }
  __syncthreads();
  if (ty < (two ? 2 : 1) && n < a.N) {
    float* out = a.bias + ((size_t)split * a.G + grp) * a.R + (size_t)ty * a.N + n;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float s = 0.f;
#pragma unroll
      for (int y = 0; y < DZ_TY; ++y) s += red[y][ty][tx * V + j];
      out[j] = s;
    }
  }
}

__global__ __launch_bounds__(256) void bias_sum_kernel(const float* part, float* out, int n, int splits) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int q = 0; q < splits; ++q) s += part[(size_t)q * n + i];
  out[i] = s;
}

constexpr int TARGET_TILES = 256;  // one workgroup per compute unit

// Splits of a contraction of `steps` steps when `tiles` tiles leave compute units idle: enough to fill
// the device, with at least eight steps each (a split's partial tile costs a write and a read).
int pick_splits(long tiles, int steps) {
  if (tiles <= 0 || tiles * 2 > TARGET_TILES) return 1;
  long s = TARGET_TILES / tiles;
  if (s > steps / 8) s = steps / 8;
  return (int)(s < 1 ? 1 : (s > 32 ? 32 : s));
}

constexpr int TILE = 128;
int div_up(long a, long b) { return (int)((a + b - 1) / b); }

template <typename E, int MODE>
void gemm_go(const GemmArgs& g, int grid, hipStream_t st) {
  gemm_kernel<E, TILE, TILE, 2, 2, MODE><<<grid, 256, 0, st>>>(g);
}

template <int MODE>
hipError_t launch_gemm(const LinearPlan& p, GemmArgs& g, hipStream_t st) {
  const int per_n = MODE == GEMM_GATED ? TILE / 2 : TILE;
  const long nt = div_up(g.out_n, per_n);
  // (each group of rows adds at most one partial row tile)
  const long mt = MODE == GEMM_DW ? (long)div_up(g.out_m, TILE) * g.G
                                  : (g.group_start ? (long)g.M / TILE + (g.G < g.M ? g.G : g.M) : div_up(g.M, TILE));
  const long grid = nt * mt * g.splits;
  if (grid <= 0) return hipSuccess;
  if (p.dtype == MOE_VQ_BF16) gemm_go<Bf16, MODE>(g, (int)grid, st);
  else gemm_go<F32, MODE>(g, (int)grid, st);
  if (g.splits > 1) {
    const int rows = MODE == GEMM_DW ? g.G * g.out_m : g.M;
    const size_t n = (size_t)rows * ((g.ldo + 3) / 4);
    split_sum_kernel<MODE == GEMM_GATED><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g, rows);
  }
  return hipGetLastError();
}

void pack_rows(const LinearPlan& p, const void* src, void* dst, size_t rows, hipStream_t st) {
  const size_t n = rows * p.Kp;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (n == 0) return;
  if (p.size == 2)
    pack_rows_kernel<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), rows, p.K, p.Kp);
  else
    pack_rows_kernel<uint32_t><<<grid, 256, 0, st>>>(static_cast<const uint32_t*>(src), static_cast<uint32_t*>(dst), rows, p.K, p.Kp);
}

template <typename T>
T* at(void* base, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(base) + off); }

}  // namespace

// bound: the workspace of every call with at most n_rows rows (fewer rows may take more splits).
static LinearPlan plan_of(const moe_vq_linear* L, int n_rows, bool backward, bool bound) {
  LinearPlan p{};
  p.M = n_rows; p.K = L->n_in; p.N = L->n_out; p.G = L->n_groups;
  p.R = L->act == MOE_VQ_ACT_SWIGLU ? 2 * p.N : p.N;
  p.dtype = L->dtype;
  p.size = p.dtype == MOE_VQ_BF16 ? 2 : 4;
  const int e16 = 16 / p.size, kt = STEP_BYTES / p.size;
  p.Kp = (p.K + e16 - 1) / e16 * e16;
  p.Rp = (p.R + e16 - 1) / e16 * e16;
  p.pack_k = p.Kp != p.K;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
  p.xp = take(p.pack_k ? (size_t)p.M * p.Kp * p.size : 0);
  p.wp = take(p.pack_k ? (size_t)p.G * p.R * p.Kp * p.size : 0);
  p.split_fwd = p.split_dx = p.split_dw = p.split_bias = 1;
  size_t part = 0;
  // (splits * tiles <= TARGET_TILES, at most 32 splits)
  auto most = [&](int cols) {
    const size_t a = (size_t)TARGET_TILES * TILE * TILE * 4, b = (size_t)32 * p.M * cols * 4;
    return a < b ? a : b;
  };
  if (!backward) {
    if (p.G == 1) p.split_fwd = pick_splits((long)div_up(p.M, TILE) * div_up(p.R, TILE), div_up(p.K, kt));
    if (bound && p.G == 1) part = most(p.R);
    else if (p.split_fwd > 1) part = (size_t)p.split_fwd * p.M * p.R * 4;
  } else {
    p.dz = take((size_t)p.M * p.Rp * p.size);
    const long strips = (long)div_up(p.N, DZ_TX * 4) * p.G;
    const long want = 2048 / (strips < 1 ? 1 : strips), can = div_up(p.M, 16 * p.G);
    p.split_bias = (int)(want < 1 || can < 1 ? 1 : (want < can ? want : can));
    p.bias_part = take(p.split_bias > 1 ? (size_t)p.split_bias * p.G * p.R * 4 : 0);
    if (p.G == 1) p.split_dx = pick_splits((long)div_up(p.M, TILE) * div_up(p.K, TILE), div_up(p.R, kt));
    p.split_dw = pick_splits((long)p.G * div_up(p.R, TILE) * div_up(p.K, TILE), div_up(p.M, (long)kt * p.G));
    if (bound && p.G == 1) part = most(p.K);
    else if (p.split_dx > 1) part = (size_t)p.split_dx * p.M * p.K * 4;
    const size_t dw = p.split_dw > 1 ? (size_t)p.split_dw * p.G * p.R * p.K * 4 : 0;
    part = part > dw ? part : dw;
  }
  p.part = take(part);
  p.total = off < 256 ? 256 : off;
  return p;
}

LinearPlan linear_plan(const moe_vq_linear* L, int n_rows, bool backward) { return plan_of(L, n_rows, backward, false); }
size_t linear_max_bytes(const moe_vq_linear* L, int n_rows, bool backward) { return plan_of(L, n_rows, backward, true).total; }

hipError_t launch_linear_forward(const LinearPlan& p, const LinearCall& c, hipStream_t st) {
  if (p.M == 0) return hipSuccess;
  GemmArgs g{};
  g.a = static_cast<const char*>(c.x);
  g.b = static_cast<const char*>(c.L->w);
  if (p.pack_k) {
    pack_rows(p, c.x, at<char>(c.ws, p.xp), p.M, st);
    pack_rows(p, c.L->w, at<char>(c.ws, p.wp), (size_t)p.G * p.R, st);
    g.a = at<char>(c.ws, p.xp);
    g.b = at<char>(c.ws, p.wp);
  }
  g.a_pitch = g.b_pitch = (uint32_t)p.Kp * p.size;
  g.w_group = (uint64_t)p.R * g.b_pitch;
  g.group_start = c.group_start;
  g.G = p.G; g.M = p.M;
  g.kc = p.K;
  g.out_n = p.N;
  // (a table of one group may leave rows out, which the sum over splits would not know)
  g.splits = c.group_start ? 1 : p.split_fwd;
  g.part = at<float>(c.ws, p.part);
  g.bias = c.L->bias;
  g.res = c.residual;
  g.out = c.y;
  g.z = c.z;
  g.ldo = p.N;
  g.out_dtype = c.y_dtype;
  g.z_dtype = p.dtype;
  g.act = c.L->act;
  g.lim = c.L->swiglu_limit;
  return c.L->act == MOE_VQ_ACT_SWIGLU ? launch_gemm<GEMM_GATED>(p, g, st) : launch_gemm<GEMM_FWD>(p, g, st);
}

hipError_t launch_linear_backward(const LinearPlan& p, const LinearCall& c, hipStream_t st) {
  // dz: dy itself where nothing changes it
  const bool same = c.L->act == MOE_VQ_ACT_NONE && c.y_dtype == p.dtype && p.Rp == p.R;
  const bool need_dz = (c.dx || c.dw) && !same;
  const void* dz = same ? c.dy : at<void>(c.ws, p.dz);
  if (need_dz || c.dbias) {
    DzArgs d{};
    d.dy = c.dy; d.z = c.z;
    d.dz = need_dz ? at<void>(c.ws, p.dz) : nullptr;
    d.splits = p.split_bias;
    d.bias = !c.dbias ? nullptr : (d.splits > 1 ? at<float>(c.ws, p.bias_part) : c.dbias);
    d.group_start = c.group_start;
    d.M = p.M; d.N = p.N; d.R = p.R; d.G = p.G; d.pitch = p.Rp;
    d.dtype = p.dtype; d.dy_dtype = c.y_dtype; d.act = c.L->act; d.lim = c.L->swiglu_limit;
    const bool vec = p.N % 4 == 0;
    const dim3 grid(div_up(p.N, DZ_TX * (vec ? 4 : 1)), p.G, d.splits);
    if (vec) dz_kernel<4><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
    else dz_kernel<1><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
    if (c.dbias && d.splits > 1)
      bias_sum_kernel<<<div_up((long)p.G * p.R, 256), 256, 0, st>>>(d.bias, c.dbias, p.G * p.R, d.splits);
  }
  const void* x = c.x;
  const void* w = c.L->w;
  if (p.pack_k) {
    if (c.dw) { pack_rows(p, c.x, at<char>(c.ws, p.xp), p.M, st); x = at<char>(c.ws, p.xp); }
    if (c.dx) { pack_rows(p, c.L->w, at<char>(c.ws, p.wp), (size_t)p.G * p.R, st); w = at<char>(c.ws, p.wp); }
  }
  GemmArgs g{};
  g.a = static_cast<const char*>(dz);
  g.a_pitch = (uint32_t)p.Rp * p.size;
  g.b_pitch = (uint32_t)p.Kp * p.size;
  g.w_group = (uint64_t)p.R * g.b_pitch;
  g.group_start = c.group_start;
  g.G = p.G; g.M = p.M;
  g.part = at<float>(c.ws, p.part);
  g.out_n = g.ldo = p.K;
  g.out_dtype = p.dtype;
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && c.dx && p.M > 0) {
    g.b = static_cast<const char*>(w);
    g.kc = p.R;
    g.out = c.dx;
    g.splits = c.group_start ? 1 : p.split_dx;
    e = launch_gemm<GEMM_DX>(p, g, st);
  }
  if (e == hipSuccess && c.dw) {
    g.b = static_cast<const char*>(x);
    g.out_m = p.R;
    g.out = c.dw;
    g.splits = p.split_dw;
    e = launch_gemm<GEMM_DW>(p, g, st);
  }
  return e;
}

}  // namespace mvq
