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
// A contraction step takes 128 bytes of an along operand's row (a cache line: 64 bf16 or 32 fp32
// values, two matrix instructions deep; 64 bytes measured 10 % slower) and as many rows of an across
// operand.  Both go from memory to LDS without passing through registers (16 bytes per lane).  The
// buffer descriptor ends at the last valid row, so what lies behind reads as zero: rows of the next
// group never enter a sum.
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
// Element types
// ---------------------------------------------------------------------------------------

struct Bf16 {
  // UNIT: bytes of 16 values; MMAS: instructions of one mma
  static constexpr int SIZE = 2, DTYPE = MOE_VQ_BF16, UNIT = 32, MMAS = 1;
  static __device__ __forceinline__ void mma(const u32x4_t& a, const u32x4_t& b, f32x4_t& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
};
struct F32 {
  static constexpr int SIZE = 4, DTYPE = MOE_VQ_F32, UNIT = 64, MMAS = 4;
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

// Epilogue of eight consecutive output columns n.. of output row m: bias, z, activation, residual, one
// rounding to the output's type.  v: the sums (SWIGLU: the gate's), u: the up sums.  z keeps the
// values before the activation, rounded once to its type.
template <bool GATED, bool STREAM = false>
__device__ __forceinline__ void epilogue8(const GemmArgs& g, int grp, size_t m, int n, float* v, float* u) {
  const int left = g.ldo - n;
  const size_t wrows = GATED ? 2 * (size_t)g.ldo : (size_t)g.ldo;
  if (g.bias) {
    const float* b = g.bias + grp * wrows;
    float t[8];
    load8(b, n, MOE_VQ_F32, left, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += t[j];
    if (GATED) {
      load8(b, (size_t)g.ldo + n, MOE_VQ_F32, left, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += t[j];
    }
  }
  if (g.z) {
    store8<STREAM>(g.z, m * wrows + n, g.z_dtype, left, v);
    if (GATED) store8<STREAM>(g.z, m * wrows + g.ldo + n, g.z_dtype, left, u);
  }
  if (GATED) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = swiglu(v[j], u[j], g.lim);
  } else if (g.act == MOE_VQ_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_fast(v[j]);
  } else if (g.act == MOE_VQ_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = gelu(v[j]);
  }
  const size_t at = m * (size_t)g.ldo + n;
  if (g.res) {
    float r[8];
    load8(g.res, at, g.out_dtype, left, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  store8<STREAM>(g.out, at, g.out_dtype, left, v);
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

// The workgroups of one XCD (every eighth) take neighbouring ones of n tiles, so that its L2 serves the
// operands they share.
__device__ __forceinline__ int xcd_order(int bid, int n) {
  const int x = bid & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (bid >> 3);
}

// Tile id -> (row tile, column tile): bands of BAND row tiles, column by column within a band, so that
// 32 neighbouring tiles (one XCD's at a time) share eight row tiles and four column tiles, or four and
// eight where the column operand is the smaller.
template <int BAND>
__device__ __forceinline__ void band_order(int id, int mt, int nt, int& im, int& in) {
  const int band = id / (BAND * nt), rem = id - band * BAND * nt;
  const int h = mt - band * BAND < BAND ? mt - band * BAND : BAND;
  in = rem / h;
  im = band * BAND + (rem - in * h);
}

// LDS position of 16-byte chunk c (0..7) of an along operand's row: the chunks of a row are
// exchanged by its number, so that the lanes of each of a 16-byte read's four phases (lanes 0-3,
// 12-15, 20-27 in the first) lie in 16 different groups of four banks.  Measured without
// conflicts; exchanging rows 8 to 15 once more, which would suit phases of 16 consecutive lanes,
// doubles the reads' time.
__device__ __forceinline__ int along_swizzle(int row) { return row & 7; }

// The same for an across operand's row, in units of 16 values (32 bytes of bf16, 64 of fp32):
// the rows that one read touches spread over the units of a 256-byte bank window.
template <typename E, int B>
__device__ __forceinline__ int across_swizzle(int row) {
  if (E::SIZE == 4) return (row >> 2) & 3;
  constexpr int UNITS = B * E::SIZE / E::UNIT;
  return UNITS >= 8 ? (row & 3) | ((row >> 1) & 4) : (row & 3) ^ ((row >> 3) & 1);
}

// A barrier behind which, for every wave, all but the last N of its loads into LDS have landed
// (vmcnt N) and every read of LDS before it is done (lgkmcnt 0).  The empty asm keeps the
// compiler from moving memory accesses over it.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One operand of a tile: B rows of output space (ALONG) or B columns (across), loaded by NW waves.
template <typename E, int B, bool ALONG, int NW>
struct Operand {
  static constexpr int BYTES = B * STEP_BYTES;
  static constexpr int LOADS = BYTES / 1024 / NW;     // 1 KiB per wave and load
  static constexpr int ROWB = B * E::SIZE;            // bytes of an across row
  static constexpr int KT = STEP_BYTES / E::SIZE;     // contraction values per step
  static constexpr int READS = ALONG ? 1 : E::SIZE;   // LDS reads of a matrix operand (2 of bf16, 4 of fp32 across)
  static_assert(LOADS >= 1 && LOADS * NW * 1024 == BYTES, "loads divide evenly over the waves");
  uint64_t base;    // address of this step's first byte
  uint32_t left;    // along: bytes from base to the end of what may be read; across: byte offset of the
                    // tile's first column
  uint32_t step, cut;  // across: bytes of a step's rows, of one row
  uint32_t off[LOADS];
  int first;        // along: first contraction value of the lane's chunk

  // along: the rows start at p, `bytes` of them may be read; row r of the tile is row
  // r, or with half > 0 the r-th of blocks of 16 gate rows and 16 up rows (half rows apart).
  __device__ __forceinline__ void init_along(const char* p, uint64_t bytes, uint32_t pitch, int half, int lane, int wave) {
    base = (uint64_t)p;
    left = (uint32_t)bytes;
    const int c = (lane & 7) ^ along_swizzle(lane >> 3);
    first = c * (16 / E::SIZE);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int row = (wave * LOADS + j) * 8 + (lane >> 3);
      const int src = half ? ((row >> 4) & 1) * half + (row >> 5) * 16 + (row & 15) : row;
      off[j] = (uint32_t)src * pitch + c * 16;
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
  // One of the LOADS loads (1 KiB per wave) of the step that has `rest` contraction values (across: rows)
  // left, or of none with rest <= 0: what is out of range reads as zero.  WHOLE: a whole step is left.
  template <bool WHOLE>
  __device__ __forceinline__ void load(lds_char* lds, int rest, int wave, int j) const {
    // (an across descriptor starts at the tile's first column and ends with the last row)
    const uint32_t bytes = WHOLE || rest >= KT ? step : (uint32_t)rest * cut;
    const uint32_t avail = !WHOLE && rest <= 0 ? 0u : (ALONG ? left : bytes - left);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)avail, 0x00020000);
    // (a chunk behind the end of an along row is sent out of range)
    const uint32_t o = ALONG && !WHOLE && first >= rest ? 0x80000000u : off[j];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * LOADS + j) * 1024), 16, o, 0, 0, 0);
  }
  __device__ __forceinline__ void next() {
    base += ALONG ? STEP_BYTES : step;
    if (ALONG) left -= STEP_BYTES;
  }
  // Matrix operand f (16 rows or columns of output space) of half-step s.
  static __device__ __forceinline__ u32x4_t frag(const lds_char* lds, int f, int s, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if (ALONG) {
      return *(const __attribute__((address_space(3))) u32x4_t*)(lds + (f * 16 + i) * STEP_BYTES + ((s * 4 + g) ^ along_swizzle(i)) * 16);
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

template <typename E, int BM, int BN, int WM, int WN, int NS, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void gemm_kernel(GemmArgs g) {
  constexpr int NW = WM * WN;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  using OpA = Operand<E, BM, MODE != GEMM_DW, NW>;
  constexpr bool GATED = MODE == GEMM_GATED, FORWARD = MODE == GEMM_FWD || GATED;
  static_assert(!GATED || FN % 2 == 0, "a wave holds gate and up of its columns");
  using OpB = Operand<E, BN, FORWARD, NW>;
  constexpr int KT = OpA::KT;
  constexpr int STAGE = (BM + BN) * STEP_BYTES;
  __shared__ __align__(1024) char lds_mem[NS * STAGE];
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
    band_order<4>(id - grp * mt * nt, mt, nt, im, in);
    group_rows(g, grp, r0, r1);
    m0 = im * BM;
  } else {
    // Every lane counts the row tiles of its share of the groups.  A group's tiles are neighbours, so
    // that its weights are read from memory once: its short last tile among them (run after all
    // others instead, to even out the end, those tiles read the weights again and took longer).
    const int q = (g.G + 63) / 64;
    int cnt = 0;
    for (int i = 0; i < q; ++i) {
      const int e = lane * q + i;
      if (e < g.G) {
        int lo, hi;
        group_rows(g, e, lo, hi);
        cnt += (hi - lo + BM - 1) / BM;
      }
    }
    const int inc = wave_incl_scan(cnt);
    const int tiles = __builtin_amdgcn_readlane(inc, 63) * nt;
    if ((int)blockIdx.x >= tiles * g.splits) return;  // (the grid is an upper bound)
    const int bid = xcd_order(blockIdx.x, tiles * g.splits);
    split = bid / tiles;
    const int id = bid - split * tiles, row_tile = id / nt;
    const int l = __popcll(__ballot(inc <= row_tile));  // the lane whose groups hold it
    int before = __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(cnt, l), n;
    grp = l * q;
    for (;;) {
      group_rows(g, grp, r0, r1);
      n = (r1 - r0 + BM - 1) / BM;
      if (row_tile < before + n || grp + 1 >= g.G) break;
      before += n;
      ++grp;
    }
    band_order<8>(id - before * nt, n, nt, im, in);
    m0 = r0 + im * BM;
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

  // ---- the contraction: NS stages of LDS, so NS - 1 steps' operands are on their way while one is
  // multiplied.  One barrier per step: behind it the step's operands are there for every wave, and
  // every wave has done with the step before, whose stage takes the next load.
  constexpr int LOADS = OpA::LOADS + OpB::LOADS;
  auto load = [&](lds_char* to, auto piece, auto whole) {  // load `piece` of the step's, A's first
    constexpr int P = decltype(piece)::value;
    constexpr bool W = decltype(whole)::value;
    if constexpr (P < OpA::LOADS) a.template load<W>(to, rest, wave, P);
    else b.template load<W>(to + OpA::BYTES, rest, wave, P - OpA::LOADS);
  };
  auto load_all = [&](lds_char* to) {
    if (rest >= KT) static_for<0, LOADS>([&](auto p) { load(to, p, std::true_type{}); });
    else static_for<0, LOADS>([&](auto p) { load(to, p, std::false_type{}); });
  };
  auto next = [&]() {
    a.next();
    b.next();
    rest -= KT;
  };
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (s < steps) {
      load_all(lds + s * STAGE);
      next();
    }
  }
  // Row block i of the wave is block i * WM + wm of the tile: the waves share the rows of a short tile
  // (a group's last), and skip what lies behind them in pairs of blocks.
  constexpr int Q = FM >= 2 ? 2 : 1, UNITS = FM / Q;
  const int m_end = MODE == GEMM_DW ? g.out_m : r1;
  const int blocks = (m_end - m0 + 15) / 16;
  const int live = blocks >= BM / 16 ? FM : (blocks - wm + WM - 1) / WM;
  const int units = blocks >= BM / 16 ? UNITS : ((blocks + WM - 1) / WM + Q - 1) / Q;

  // One step on `units` units of Q row operands, as a software pipeline: the next unit's reads of LDS go
  // out before this unit's matrix instructions (8192^3 forward 836 us, all reads of a half first 862).
  // The loads of a later step go out over the first SPREAD units, or (0) before them.  Measured at
  // 8192^3, before / over 1 / 2 / 3 / 4 / 6 units: forward 863 / 877 / 872 / 839 / 848 / 886 us, dx 936 / 853 /
  // 850 / 854 / 827 / 832, dw 965 / 925 / 932 / 942 / 953 / 1022.  The smaller tiles, two workgroups on a CU,
  // lose by it (2000 x 7168 -> 2048 gated 121 / 129 / 133 / 135 / 139 us).
  constexpr int SPREAD = BM * BN < 256 * 256 ? 0 : (FORWARD ? 3 : (MODE == GEMM_DX ? 4 : 1));
  auto multiply = [&](auto live_units, const lds_char* at, lds_char* to) {
    constexpr int U = decltype(live_units)::value, HALVES = STEP_BYTES / 64;  // (a matrix instruction takes 64 bytes of a row)
    u32x4_t fa[2][Q], fb[2][FN];
    static_for<0, FN>([&](auto j) { fb[0][j] = OpB::frag(at + OpA::BYTES, wn * FN + j, 0, lane); });
    static_for<0, Q>([&](auto i) { fa[0][i] = OpA::frag(at, i * WM + wm, 0, lane); });
    __builtin_amdgcn_sched_group_barrier(0x100, FN * OpB::READS + Q * OpA::READS, 0);
    static_for<0, HALVES * U>([&](auto uu) {
      constexpr int u = decltype(uu)::value, h = u / U, q = u % U, n = u + 1, nh = n / U, nq = n % U;
      if constexpr (n < HALVES * U) {
        if constexpr (nq == 0) static_for<0, FN>([&](auto j) { fb[nh][j] = OpB::frag(at + OpA::BYTES, wn * FN + j, nh, lane); });
        static_for<0, Q>([&](auto i) { fa[n & 1][i] = OpA::frag(at, (nq * Q + i) * WM + wm, nh, lane); });
        __builtin_amdgcn_sched_group_barrier(0x100, (nq == 0 ? FN * OpB::READS : 0) + Q * OpA::READS, 0);
      }
      if constexpr (SPREAD > 0) {
        constexpr int OVER = HALVES * U < SPREAD ? HALVES * U : SPREAD;
        constexpr int FIRST = u < OVER ? LOADS * u / OVER : LOADS, LAST = u < OVER ? LOADS * (u + 1) / OVER : LOADS;
        static_for<FIRST, LAST>([&](auto p) { load(to, p, std::false_type{}); });
        __builtin_amdgcn_sched_group_barrier(0x020, LAST - FIRST, 0);
      }
      static_for<0, Q>([&](auto i) {
        static_for<0, FN>([&](auto j) { E::mma(fb[h][j], fa[u & 1][i], acc[q * Q + i][j]); });
      });
      __builtin_amdgcn_sched_group_barrier(0x008, Q * FN * E::MMAS, 0);
    });
  };
  auto contract = [&](auto live_units) {
    int cur = 0, fill = NS - 1;
    for (int s = 0; s < steps; ++s) {
      if (s + NS - 1 <= steps) step_barrier<(NS - 2) * LOADS>();
      else step_barrier<0>();  // (the last steps: fewer younger ones are on their way)
      if (SPREAD == 0 && s + NS - 1 < steps) load_all(lds + fill * STAGE);
      multiply(live_units, lds + cur * STAGE, lds + fill * STAGE);
      next();
      cur = cur + 1 == NS ? 0 : cur + 1;
      fill = fill + 1 == NS ? 0 : fill + 1;
    }
  };
  if (units > UNITS / 2) contract(std::integral_constant<int, UNITS>{});
  else contract(std::integral_constant<int, UNITS >= 2 ? UNITS / 2 : 1>{});
  step_barrier<0>();  // (the outputs are staged where the operands were, and where the last, empty loads go)

  // ---- outputs, 16 rows at a time: lane (i, g) of a matrix operand holds row i, columns 4 g .. of its
  // 16; through the wave's own part of LDS a lane gets eight neighbouring columns of one row, so that
  // rows leave in long runs.  Two parts take turns, so one can fill while the other is read.
  constexpr int PITCH = FN * 16 + 4;
  constexpr int COLS = GATED ? FN * 8 : FN * 16;  // output columns of the wave
  static_assert(NW * 2 * 16 * PITCH * 4 <= (int)sizeof(lds_mem), "output staging");
  // The largest tiles' outputs exceed the L2s many times over: streamed, dw of 16 experts' 512 rows each
  // takes 779 us instead of 924, and at 8192^3 dx gains 9 % and dw 9 %.
  constexpr bool STREAM = BM * BN >= 256 * 256;
  float* stage = reinterpret_cast<float*>(lds_mem) + wave * 2 * 16 * PITCH;
  const size_t out_rows = MODE == GEMM_DW ? (size_t)g.G * g.out_m : (size_t)g.M;
  const size_t out_cols = GATED ? 2 * (size_t)g.out_n : (size_t)g.out_n;
  // eight columns of the 16 rows: unit t of row block i
  auto put = [&](const float* part, int i, int t) __attribute__((always_inline)) {
    constexpr int PER = COLS / 8;
    const int rr = t / PER, c = (t % PER) * 8;
    const int m = m0 + (i * WM + wm) * 16 + rr, n = n0 + wn * COLS + c;
    if (m >= m_end || n >= g.out_n) return;
    const size_t row = MODE == GEMM_DW ? (size_t)grp * g.out_m + m : (size_t)m;
    const float* from = part + rr * PITCH + (GATED ? (c >> 4) * 32 + (c & 15) : c);
    float v[8], u[8];
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(from + q);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q + j] = lo[j];
      if (GATED) {
        const f32x4_t up = *reinterpret_cast<const f32x4_t*>(from + 16 + q);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[q + j] = up[j];
      }
    }
    if (g.splits > 1) {
      float* p = g.part + ((size_t)split * out_rows + row) * out_cols;
      store8(p, n, MOE_VQ_F32, g.out_n - n, v);
      if (GATED) store8(p, (size_t)g.out_n + n, MOE_VQ_F32, g.out_n - n, u);
    } else if (FORWARD) {
      epilogue8<GATED, STREAM>(g, grp, row, n, v, u);
    } else {
      store8<STREAM>(g.out, row * (size_t)g.ldo + n, E::DTYPE, g.out_n - n, v);
    }
  };
  static_for<0, FM>([&](auto fi) __attribute__((always_inline)) {
    constexpr int i = decltype(fi)::value;
    if (i >= live) return;
    float* part = stage + (i & 1) * 16 * PITCH;
    static_for<0, FN>([&](auto fj) {
      constexpr int j = decltype(fj)::value;
      *reinterpret_cast<f32x4_t*>(part + (lane & 15) * PITCH + j * 16 + (lane >> 4) * 4) = acc[i][j];
    });
    // (the wave's LDS accesses complete in order; the fences keep the compiler to it)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int t = 0; t < 16 * COLS / 8; t += 64)
      if (16 * COLS / 8 >= 64 || lane < 16 * COLS / 8) put(part, i, t + lane);
  });
}

// ---------------------------------------------------------------------------------------
// Few rows: the weights' bytes are what counts
// ---------------------------------------------------------------------------------------

// The part of a dword to keep whose first `drop` bytes go (a multiple of 2; all of it if 0 or less).
__device__ __forceinline__ uint32_t few_keep(int drop) { return drop <= 0 ? 0xFFFFFFFFu : (drop >= 4 ? 0u : 0xFFFF0000u); }

// Forward product of at most 16 rows.  Bound by streaming W from HBM once; a 64 x 64 tile spends as much on
// the parts of its split contraction and their sum (one row, 7168 -> 2048 gated, weights not in
// any cache: 19 us) as on the weights (12 us here, of which the 59 MB take 10).  A workgroup
// takes 16 weight rows (gated: eight gate rows and their up rows), its eight waves split the
// contraction among them, and their sums meet in LDS in a fixed order: one launch.  W goes from
// memory to the registers of the matrix operand, 16 rows of 64 bytes per load; the rows of x, which
// every workgroup reads, come from L2.  Of 2, 4, 8 and 14 loads ahead two
// and four measured best (12.3, 12.3, 13.7, 13.5 us), of 4, 8 and 16 waves eight (14.8, 12.3, 14.7).
constexpr int FEW_ROWS = 16, FEW_WAVES = 8, FEW_STREAM = 4;

//
// ODD: rows of any width of at least 16 bytes, where they lie (repacked to 16-byte rows, W would move three
// times: one row, 7071 -> 4096 bf16, 23 us instead of 38; eight in fp32 37 instead of 74).  A row's last chunk is then its last 16 bytes; what the chunk before has counted is
// replaced by zeros, in both operands: an infinity times zero would be NaN.
template <typename E, bool GATED, bool ODD>
__global__ __launch_bounds__(64 * FEW_WAVES) void few_rows_kernel(GemmArgs g) {
  constexpr int STEP = 64;   // bytes of a row per load of its 16 rows
  constexpr int PITCH = 20;  // floats between the staged rows
  __shared__ __align__(16) float red[FEW_WAVES][FEW_ROWS][PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  constexpr int PER = GATED ? 8 : 16;  // output columns
  const int n0 = (int)blockIdx.x * PER;
  // this lane's weight row (rows behind the last repeat it; their sums are dropped)
  int col = GATED ? n0 + (i & 7) : n0 + i;
  col = col < g.out_n ? col : g.out_n - 1;
  const int wrow = GATED && i >= 8 ? g.out_n + col : col;
  const char* w = g.b + (size_t)wrow * g.b_pitch + q * 16;
  const char* x = g.a + (size_t)(i < g.M ? i : g.M - 1) * g.a_pitch + q * 16;
  const int bytes = g.kc * E::SIZE;  // of a row; chunks behind it count as zeros
  const int steps = (bytes + STEP - 1) / STEP, per = (steps + FEW_WAVES - 1) / FEW_WAVES;
  const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; s += FEW_STREAM) {
    u32x4_t wv[FEW_STREAM], xv[FEW_STREAM];
#pragma unroll
    for (int j = 0; j < FEW_STREAM; ++j) {
      // (a load behind this wave's share repeats its last one, a chunk behind the row's end its first one;
      // both are replaced by zeros below)
      const int at = (s + j < s1 ? s + j : s1 - 1) * STEP;
      int off = at + q * 16 < bytes ? at : -q * 16;
      if (ODD) {
        off = off + q * 16 + 16 > bytes ? bytes - 16 - q * 16 : off;
        const u32x4_any a = *reinterpret_cast<const u32x4_any*>(w + off), b = *reinterpret_cast<const u32x4_any*>(x + off);
        wv[j] = u32x4_t{a.x, a.y, a.z, a.w};
        xv[j] = u32x4_t{b.x, b.y, b.z, b.w};
      } else {
        wv[j] = *reinterpret_cast<const u32x4_t*>(w + off);
        xv[j] = *reinterpret_cast<const u32x4_t*>(x + off);
      }
    }
#pragma unroll
    for (int j = 0; j < FEW_STREAM; ++j) {
      const bool ok = s + j < s1 && (s + j) * STEP + q * 16 < bytes;
      const u32x4_t none = {0, 0, 0, 0};
      if (ODD) {
        const int drop = (s + j) * STEP + q * 16 + 16 - bytes;  // bytes of the chunk that the one before holds
        const u32x4_t keep = {few_keep(drop), few_keep(drop - 4), few_keep(drop - 8), few_keep(drop - 12)};
        wv[j] &= keep;
        xv[j] &= keep;
      }
      E::mma(ok ? wv[j] : none, ok ? xv[j] : none, acc);
    }
  }
  // lane (i, q) holds row i of x, weight rows 4 q .. of the 16
  *reinterpret_cast<f32x4_t*>(&red[wave][i][q * 4]) = acc;
  __syncthreads();
  const int m = threadIdx.x / (PER / 8), c = (threadIdx.x % (PER / 8)) * 8;
  if (m < g.M && n0 + c < g.out_n) {
    float v[8], up[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = up[j] = 0.f;
#pragma unroll
    for (int k = 0; k < FEW_WAVES; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] += red[k][m][c + j];
        if (GATED) up[j] += red[k][m][8 + c + j];
      }
    }
    epilogue8<GATED>(g, 0, m, n0 + c, v, up);
  }
}

// The group whose rows hold row m, or -1: the last one that starts at or before it, if it reaches that far.
__device__ __forceinline__ int group_of(const GemmArgs& g, int m) {
  if (!g.group_start) return 0;
  int lo = 0, hi = g.G;  // (group_start[lo] <= m < group_start[hi] inside the table)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.group_start[mid] <= m) lo = mid;
    else hi = mid;
  }
  return g.group_start[lo] <= m && m < g.group_start[lo + 1] ? lo : -1;
}

// The sum of the splits' parts in order, then the epilogue: eight columns per thread.  ROWS: of forward or dx,
// whose rows in no group have no sums and are left as they were.
template <bool GATED, bool ROWS>
__global__ __launch_bounds__(256) void split_sum_kernel(GemmArgs g, int rows) {
  const int units = (g.ldo + 7) / 8;
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= (size_t)rows * units) return;
  const size_t m = at / units;
  const int n = (int)(at - m * units) * 8, left = g.ldo - n;
  const int grp = ROWS ? group_of(g, (int)m) : 0;
  if (grp < 0) return;
  const size_t cols = GATED ? 2 * (size_t)g.ldo : (size_t)g.ldo;
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
#pragma unroll 2
  for (int s = 0; s < g.splits; ++s) {
    const float* p = g.part + ((size_t)s * rows + m) * cols;
    float t[8];
    load8(p, n, MOE_VQ_F32, left, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += t[j];
    if (GATED) {
      load8(p, (size_t)g.ldo + n, MOE_VQ_F32, left, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += t[j];
    }
  }
  epilogue8<GATED>(g, grp, m, n, v, u);
}

// ---------------------------------------------------------------------------------------
// Repacking rows whose width is no multiple of 16 bytes (dst pitch: the next one, zero-filled)
// ---------------------------------------------------------------------------------------

// 16 bytes of dst per thread and turn; the turns cover any number of rows with a bounded grid.  With a row table of
// G groups, only what the groups use: of x (wrows 0) the rows of groups, of the weights those of groups
// that have rows, `wrows` of each group blockIdx.y.
template <typename T>
__global__ __launch_bounds__(256) void pack_rows_kernel(const T* src, T* dst, size_t rows, int cols, int pitch,
                                                        const int32_t* group_start, int G, int wrows) {
  constexpr int N = 16 / sizeof(T);
  const size_t per = pitch / N;
  size_t begin = 0, end = rows;
  if (group_start && wrows) {
    const int g = blockIdx.y;
    if (group_start[g] >= group_start[g + 1]) return;
    begin = (size_t)g * wrows;
    end = begin + wrows;
  } else if (group_start) {
    const int lo = group_start[0], hi = group_start[G];
    begin = lo < 0 ? 0 : lo;
    end = hi < 0 ? 0 : ((size_t)hi < rows ? hi : rows);
  }
  end *= per;
  for (size_t at = begin * per + (size_t)blockIdx.x * 256 + threadIdx.x; at < end; at += (size_t)gridDim.x * 256) {
    const size_t r = at / per;
    const int c = (int)(at - r * per) * N;
    const T* from = src + r * cols + c;
    if (c + N <= cols) {
      const u32x4_any v = *reinterpret_cast<const u32x4_any*>(from);
      *reinterpret_cast<u32x4_t*>(dst + at * N) = u32x4_t{v.x, v.y, v.z, v.w};
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) dst[at * N + j] = c + j < cols ? from[j] : T(0);
    }
  }
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
  float lim;
};

constexpr int DZ_TX = 32, DZ_TY = 8;  // threads over columns, over rows

// dz of eight columns of one row: the gate's (or the only) factor in d[0], the up's in d[1].
template <int ACT>
__device__ __forceinline__ void dz_values(const DzArgs& a, const float* dy, const float* zg, const float* zu, float (*d)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    d[1][j] = 0.f;
    if (ACT == MOE_VQ_ACT_NONE) {
      d[0][j] = dy[j];
    } else if (ACT == MOE_VQ_ACT_SILU) {
      d[0][j] = dy[j] * silu_grad(zg[j], sigmoid_fast(zg[j]));
    } else if (ACT == MOE_VQ_ACT_GELU) {
      d[0][j] = dy[j] * gelu_grad(zg[j]);
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
      const float sg = sigmoid_fast(gv);
      d[0][j] = gin ? dy[j] * uv * silu_grad(gv, sg) : 0.f;
      d[1][j] = uin ? dy[j] * gv * sg : 0.f;
    }
  }
}

// One workgroup: 8 DZ_TX columns of one split of one group's rows, two rows of a thread at a time (their loads
// are issued together).  Bound by reading dy and z and writing dz, each once (8192 rows of 16 groups, 2 x 2048
// columns: 168 MB in 46 us; 64 with types and activation chosen per value at run time, which keeps loads from
// overlapping; rows of 1024 bytes, streamed loads or stores and half or twice the workgroups change
// nothing or cost 2 to 3 us).  dz is rounded to the element type for the matrix products; the column
// sums add the unrounded values in fp32, rows in a fixed order.
template <int DTYPE, int DY_DTYPE, int ACT>
__global__ __launch_bounds__(DZ_TX* DZ_TY) void dz_kernel(DzArgs a) {
  __shared__ float red[DZ_TY][2][DZ_TX * 8];
  const int tx = threadIdx.x % DZ_TX, ty = threadIdx.x / DZ_TX;
  // (a row's last eight columns may overlap the eight before them: both threads write the same values)
  int n = (blockIdx.x * DZ_TX + tx) * 8;
  if (n < a.N && n > a.N - 8 && a.N >= 8) n = a.N - 8;
  const int grp = blockIdx.y, split = blockIdx.z;
  int r0 = 0, r1 = a.M;
  if (a.group_start) {
    r0 = a.group_start[grp]; r1 = a.group_start[grp + 1];
    r0 = r0 < 0 ? 0 : (r0 > a.M ? a.M : r0);
    r1 = r1 < r0 ? r0 : (r1 > a.M ? a.M : r1);
  }
  const int per = (r1 - r0 + a.splits - 1) / a.splits;
  const int m0 = r0 + split * per, m1 = m0 + per < r1 ? m0 + per : r1;
  constexpr bool two = ACT == MOE_VQ_ACT_SWIGLU, any = ACT != MOE_VQ_ACT_NONE;
  constexpr int V = 8;
  const int left = a.N - n;
  float sum[2][V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[0][j] = sum[1][j] = 0.f;
  auto put = [&](int m, float (*d)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) { sum[0][j] += d[0][j]; sum[1][j] += d[1][j]; }
    if (!a.dz) return;
    const size_t row = (size_t)m * a.pitch;
    store8(a.dz, row + n, DTYPE, left, d[0]);
    if (two) store8(a.dz, row + a.N + n, DTYPE, left, d[1]);
    // (the pitch's last columns take part in dx's contraction as zeros)
    if (n == 0)
      for (int c = a.R; c < a.pitch; ++c) store_as(a.dz, row + c, DTYPE, 0.f);
  };
  if (n < a.N) {
    for (int m = m0 + ty; m < m1; m += 2 * DZ_TY) {
      float dy[2][V], zg[2][V], zu[2][V], d[2][2][V];
      const int next = m + DZ_TY < m1 ? m + DZ_TY : m;  // (a thread without a second row loads the first again)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t r = i ? next : m;
        load8(a.dy, r * a.N + n, DY_DTYPE, left, dy[i]);
        if (any) load8(a.z, r * a.R + n, DTYPE, left, zg[i]);
        if (two) load8(a.z, r * a.R + a.N + n, DTYPE, left, zu[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) dz_values<ACT>(a, dy[i], zg[i], zu[i], d[i]);
      put(m, d[0]);
      if (m + DZ_TY < m1) put(next, d[1]);
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
      if (j < left) out[j] = s;
    }
  }
}

// The splits' column sums added up: 32 columns by 8 shares of the splits per workgroup, the shares in order.
__global__ __launch_bounds__(256) void bias_sum_kernel(const float* part, float* out, int n, int splits) {
  __shared__ float red[8][32];
  const int c = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  const int per = (splits + 7) / 8, q0 = share * per, q1 = q0 + per < splits ? q0 + per : splits;
  float s = 0.f;
  if (i < n) {
#pragma unroll 4
    for (int q = q0; q < q1; ++q) s += part[(size_t)q * n + i];
  }
  red[share][c] = s;
  __syncthreads();
  if (share == 0 && i < n) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += red[q][c];
    out[i] = t;
  }
}

using Cut = LinearPlan::Cut;
constexpr int CUS = 256;

// A kind of tile: its side, how many workgroups of it a CU holds, and what a workgroup takes (microseconds,
// measured): per contraction step with its CU full, per step if it has the CU to itself, and before
// and after them.
struct TileKind {
  int side, per_cu;
  float step, step_alone, rest;
};
constexpr TileKind BF16_TILES[] = {{256, 1, 1.95f, 1.95f, 8.f}, {128, 2, 1.2f, 0.8f, 6.f}, {64, 2, 0.6f, 0.45f, 5.f}};
constexpr TileKind F32_TILES[] = {{128, 2, 3.9f, 2.1f, 6.f}, {64, 2, 1.0f, 0.75f, 5.f}};

// How a product is cut.  rows: output rows in all, of `groups` groups; cols: output columns (weight rows forward);
// steps: contraction steps.  The cut with the smallest estimate is taken: rounds of workgroups over the
// device, times a workgroup's time, and for a split contraction the write and read of its parts (from
// the caches: 10 TB/s) and one more launch.  Large products so take 256 x 256 tiles (at 8192^3, on a card where they reach 1400 TFLOP/s, 128 x 128
// tiles, which read LDS twice as often for their products, reach 1150) unless the last round would be nearly empty; small outputs with
// long contractions are split, and outputs too small for that take small tiles.
Cut pick_cut(int dtype, long rows, long groups, long cols, int steps, bool forward) {
  const long per = (rows + groups - 1) / groups;
  Cut best{64, 1};
  float least = 3.0e38f;
  auto consider = [&](const TileKind& k) {
    // (few rows wait for weights: forward, where those lie along, small tiles have more loads on their way: 64
    // rows of 32 groups, 2048 -> 7168, 126 us by 64 x 64 tiles, 151 by 128 x 128.  For dx they lie across,
    // where wide tiles read longer runs: 358 rows of 21 groups, 3328 -> 5376, 148 us by 128 x 128, 200 by 64 x 64)
    if (forward && k.side > 64 && k.side >= 2 * per) return;
    const long tiles = (per + k.side - 1) / k.side * groups * ((cols + k.side - 1) / k.side);
    for (int parts = 1; parts <= 32; parts *= 2) {
      // (at most two workgroups per CU are split ones, of at least eight steps)
      if (parts > 1 && (k.side > 128 || tiles * parts > 2 * CUS || steps < 8 * parts)) break;
      const long n = tiles * parts, slots = (long)k.per_cu * CUS;
      const float rounds = n <= slots ? 1.f : (n < 3 * slots ? (float)((n + slots - 1) / slots) : (float)n / slots + 0.5f);
      const int each = (steps + parts - 1) / parts;
      float t = rounds * (each * (n <= CUS ? k.step_alone : k.step) + k.rest);
      if (parts > 1) t += 4.f + 0.5f * parts + 8.f * parts * rows * cols / 10.0e6f;
      if (t < least) { least = t; best = {k.side, parts}; }
    }
  };
  if (dtype == MOE_VQ_BF16) for (const TileKind& k : BF16_TILES) consider(k);
  else for (const TileKind& k : F32_TILES) consider(k);
  return best;
}

int div_up(long a, long b) { return (int)((a + b - 1) / b); }

template <typename E, int MODE, int BM, int BN, int WM, int WN, int NS>
void gemm_go(const GemmArgs& g, hipStream_t st) {
  const int per_n = MODE == GEMM_GATED ? BN / 2 : BN;
  const long nt = div_up(g.out_n, per_n);
  // (each group of rows adds at most one partial row tile)
  const long mt = MODE == GEMM_DW ? (long)div_up(g.out_m, BM) * g.G
                                  : (g.group_start ? (long)g.M / BM + (g.G < g.M ? g.G : g.M) : div_up(g.M, BM));
  const long grid = nt * mt * g.splits;
  if (grid > 0) gemm_kernel<E, BM, BN, WM, WN, NS, MODE><<<(unsigned)grid, 64 * WM * WN, 0, st>>>(g);
}

template <int MODE>
hipError_t launch_gemm(const LinearPlan& p, GemmArgs& g, int tile, hipStream_t st) {
  if (p.dtype == MOE_VQ_BF16) {
    if (tile == 256) gemm_go<Bf16, MODE, 256, 256, 2, 4, 2>(g, st);
    else if (tile == 128) gemm_go<Bf16, MODE, 128, 128, 2, 2, 2>(g, st);
    else gemm_go<Bf16, MODE, 64, 64, 2, 2, 4>(g, st);
  } else {
    if (tile == 128) gemm_go<F32, MODE, 128, 128, 2, 2, 2>(g, st);
    else gemm_go<F32, MODE, 64, 64, 2, 2, 4>(g, st);
  }
  if (g.splits > 1) {
    const int rows = MODE == GEMM_DW ? g.G * g.out_m : g.M;
    const size_t n = (size_t)rows * ((g.ldo + 7) / 8);
    split_sum_kernel<MODE == GEMM_GATED, MODE != GEMM_DW><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g, rows);
  }
  return hipGetLastError();
}

template <typename E>
void few_go(const GemmArgs& g, bool gated, hipStream_t st) {
  const unsigned grid = (unsigned)div_up(g.out_n, gated ? 8 : 16);
  const bool odd = g.b_pitch % 16 != 0;
  if (gated && odd) few_rows_kernel<E, true, true><<<grid, 64 * FEW_WAVES, 0, st>>>(g);
  else if (gated) few_rows_kernel<E, true, false><<<grid, 64 * FEW_WAVES, 0, st>>>(g);
  else if (odd) few_rows_kernel<E, false, true><<<grid, 64 * FEW_WAVES, 0, st>>>(g);
  else few_rows_kernel<E, false, false><<<grid, 64 * FEW_WAVES, 0, st>>>(g);
}

template <int DTYPE, int DY_DTYPE>
void dz_go(const LinearPlan& p, const DzArgs& d, int act, hipStream_t st) {
  const dim3 grid(div_up(p.N, DZ_TX * 8), p.G, d.splits);
  if (act == MOE_VQ_ACT_NONE) dz_kernel<DTYPE, DY_DTYPE, MOE_VQ_ACT_NONE><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
  else if (act == MOE_VQ_ACT_SILU) dz_kernel<DTYPE, DY_DTYPE, MOE_VQ_ACT_SILU><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
  else if (act == MOE_VQ_ACT_GELU) dz_kernel<DTYPE, DY_DTYPE, MOE_VQ_ACT_GELU><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
  else dz_kernel<DTYPE, DY_DTYPE, MOE_VQ_ACT_SWIGLU><<<grid, DZ_TX * DZ_TY, 0, st>>>(d);
}

void launch_dz(const LinearPlan& p, const DzArgs& d, int dy_dtype, int act, hipStream_t st) {
  if (p.dtype == MOE_VQ_BF16) {
    if (dy_dtype == MOE_VQ_BF16) dz_go<MOE_VQ_BF16, MOE_VQ_BF16>(p, d, act, st);
    else dz_go<MOE_VQ_BF16, MOE_VQ_F32>(p, d, act, st);
  } else {
    if (dy_dtype == MOE_VQ_BF16) dz_go<MOE_VQ_F32, MOE_VQ_BF16>(p, d, act, st);
    else dz_go<MOE_VQ_F32, MOE_VQ_F32>(p, d, act, st);
  }
}

void pack_rows(const LinearPlan& p, const void* src, void* dst, size_t rows, const int32_t* group_start, int wrows,
               hipStream_t st) {
  // (groups side by side; enough workgroups for each that a few of them that have rows fill the device)
  const unsigned groups = group_start && wrows ? p.G : 1, most = 64 * CUS / groups > 64 ? 64 * CUS / groups : 64;
  const size_t blocks = (rows / groups * p.Kp * p.size / 16 + 255) / 256;
  if (blocks == 0) return;
  const dim3 grid((unsigned)(blocks < most ? blocks : most), groups);
  auto go = [&](auto t) {
    using T = decltype(t);
    pack_rows_kernel<T><<<grid, 256, 0, st>>>(static_cast<const T*>(src), static_cast<T*>(dst), rows, p.K, p.Kp, group_start, p.G, wrows);
  };
  if (p.size == 2) go(uint16_t{});
  else go(uint32_t{});
}
// x's rows and the weights, to where the plan has them in the workspace.
const char* pack_x(const LinearPlan& p, const LinearCall& c, hipStream_t st) {
  pack_rows(p, c.x, static_cast<char*>(c.ws) + p.xp, p.M, c.group_start, 0, st);
  return static_cast<char*>(c.ws) + p.xp;
}
const char* pack_w(const LinearPlan& p, const LinearCall& c, hipStream_t st) {
  pack_rows(p, c.L->w, static_cast<char*>(c.ws) + p.wp, (size_t)p.G * p.R, c.group_start, p.R, st);
  return static_cast<char*>(c.ws) + p.wp;
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
  p.fwd = pick_cut(p.dtype, p.M, p.G, p.R, div_up(p.K, kt), true);
  p.few = p.G == 1 && p.M <= FEW_ROWS;
  p.dx = pick_cut(p.dtype, p.M, p.G, p.K, div_up(p.R, kt), false);
  p.dw = pick_cut(p.dtype, (long)p.G * p.R, p.G, p.K, div_up(p.M, (long)kt * p.G), false);
  size_t part = 0;
  // (parts * tiles <= 2 CUS of at most 128 x 128 sums, and at most 32 parts)
  auto most = [&](size_t rows, int cols) {
    const size_t a = (size_t)2 * CUS * 128 * 128 * 4, b = 32 * rows * cols * 4;
    return a < b ? a : b;
  };
  if (!backward) {
    if (bound) part = most(p.M, p.R);
    else if (p.fwd.splits > 1) part = (size_t)p.fwd.splits * p.M * p.R * 4;
  } else {
    p.dz = take((size_t)p.M * p.Rp * p.size);
    // (as many workgroups as keep the device busy, each with a row per thread at least)
    const long strips = (long)div_up(p.N, DZ_TX * 8) * p.G, want = 2048 / strips, can = div_up(p.M, DZ_TY * p.G);
    p.split_bias = (int)(want < 1 || can < 1 ? 1 : (want < can ? want : can));
    p.bias_part = take(p.split_bias > 1 ? (size_t)p.split_bias * p.G * p.R * 4 : 0);
    if (bound) {
      part = most(p.M, p.K);
      const size_t dw = most((size_t)p.G * p.R, p.K);
      part = part > dw ? part : dw;
    } else {
      part = p.dx.splits > 1 ? (size_t)p.dx.splits * p.M * p.K * 4 : 0;
      const size_t dw = p.dw.splits > 1 ? (size_t)p.dw.splits * p.G * p.R * p.K * 4 : 0;
      part = part > dw ? part : dw;
    }
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
  const bool few = p.few && !c.group_start, as_is = few && p.K * p.size >= 16;
  if (p.pack_k && !as_is) {
    g.a = pack_x(p, c, st);
    g.b = pack_w(p, c, st);
  }
  g.a_pitch = g.b_pitch = (uint32_t)(as_is ? p.K : p.Kp) * p.size;
  g.w_group = (uint64_t)p.R * g.b_pitch;
  g.group_start = c.group_start;
  g.G = p.G; g.M = p.M;
  g.kc = p.K;
  g.out_n = p.N;
  g.splits = p.fwd.splits;
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
  if (few) {
    if (p.dtype == MOE_VQ_BF16) few_go<Bf16>(g, c.L->act == MOE_VQ_ACT_SWIGLU, st);
    else few_go<F32>(g, c.L->act == MOE_VQ_ACT_SWIGLU, st);
    return hipGetLastError();
  }
  return c.L->act == MOE_VQ_ACT_SWIGLU ? launch_gemm<GEMM_GATED>(p, g, p.fwd.tile, st)
                                       : launch_gemm<GEMM_FWD>(p, g, p.fwd.tile, st);
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
    d.lim = c.L->swiglu_limit;
    launch_dz(p, d, c.y_dtype, c.L->act, st);
    if (c.dbias && d.splits > 1)
      bias_sum_kernel<<<div_up((long)p.G * p.R, 32), 256, 0, st>>>(d.bias, c.dbias, p.G * p.R, d.splits);
  }
  const void* x = c.x;
  const void* w = c.L->w;
  if (p.pack_k) {
    if (c.dw) x = pack_x(p, c, st);
    if (c.dx) w = pack_w(p, c, st);
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
    g.splits = p.dx.splits;
    e = launch_gemm<GEMM_DX>(p, g, p.dx.tile, st);
  }
  if (e == hipSuccess && c.dw) {
    g.b = static_cast<const char*>(x);
    g.out_m = p.R;
    g.out = c.dw;
    g.splits = p.dw.splits;
    e = launch_gemm<GEMM_DW>(p, g, p.dw.tile, st);
  }
  return e;
}

}  // namespace mvq
