// Argument checks that the entry points of the dense operators share.
#pragma once

#include <initializer_list>

#include "block.h"

namespace mvq {

constexpr int MAX_COLS = 65536;
constexpr int MAX_ROWS = MAX_T * MAX_K;

inline bool dtype_ok(int d) { return d == MOE_VQ_F32 || d == MOE_VQ_BF16; }
inline bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }
inline bool off4(const void* p) { return ((uintptr_t)p & 3) != 0; }

// A buffer of n bytes (p null: not there).
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
  return a.p && b.p && a.n && b.n && (uintptr_t)a.p < (uintptr_t)b.p + b.n && (uintptr_t)b.p < (uintptr_t)a.p + a.n;
}
// A buffer that is written shares a byte with another one, or with one that is read: a workgroup would write
// it while another still reads, or writes, the same byte.
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}
inline size_t size_of(int d) { return d == MOE_VQ_BF16 ? 2 : 4; }

// The bytes and the scales of rows in 8 bits (none: r null).
inline Span bytes8(const moe_vq_rows8* r, int rows, int cols) { return {r ? r->q : nullptr, rows * rows8_pitch(cols)}; }
inline Span scales8(const moe_vq_rows8* r, int rows, int cols) { return {r ? r->e : nullptr, rows * (rows8_pitch(cols) / 32)}; }

}  // namespace mvq
