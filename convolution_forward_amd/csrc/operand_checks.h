// Host checks of strided operands shared by the row operators (layer norm, dropout,
// rows to 8 bits) and the 8-bit linear layer: strides, offsets, alignment, overlap.
// Plain C++ with no HIP include.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "conv.h"
#include "plan.h"

namespace convfwd {

constexpr int64_t kRowsMax = 2147483647LL;   // rows of an operand
constexpr int64_t kExtentMax = 1LL << 20;    // contiguous extents and strides

// A matrix in memory: rows of cols elements of es bytes, ld elements apart.
struct Operand {
  uintptr_t base;  // of its first element
  int64_t rows, cols, ld;
  int es;
};

// ld of a matrix with rows of `cols` elements: 0 = dense; -1 if out of range
inline int64_t row_stride(int64_t ld, int64_t cols) {
  if (ld == 0) return cols;
  return ld >= cols && ld <= kExtentMax ? ld : -1;
}

// the last element's byte offset stays in int64, and an operand below 2^40
// elements (beyond the card's memory)
inline bool offset_fits(int64_t off, int64_t rows, int64_t ld, int es) {
  int64_t e, b;
  if (off < 0) return false;
  if (__builtin_mul_overflow(rows < 1 ? 1 : rows, ld, &e) || e > (1LL << 40)) return false;
  return !__builtin_add_overflow(e, off, &e) && !__builtin_mul_overflow(e, (int64_t)es, &b);
}

inline Operand operand(const void* p, int64_t off, int64_t rows, int64_t cols, int64_t ld, int es) {
  return {(uintptr_t)p + (uintptr_t)off * (uintptr_t)es, rows, cols, ld, es};
}

inline uintptr_t operand_end(const Operand& a) {
  return a.base + (uintptr_t)((a.rows - 1) * a.ld + a.cols) * (uintptr_t)a.es;
}

inline bool on_elements(const Operand& a) { return a.base % (uintptr_t)a.es == 0; }

// Whether two matrices share a byte.  Matrices of one stride in bytes whose columns do
// not meet (two halves of the rows of one buffer) do not.
inline bool operands_meet(const Operand& a, const Operand& b) {
  if (a.rows < 1 || b.rows < 1) return false;
  if (a.base >= operand_end(b) || b.base >= operand_end(a)) return false;
  const int64_t stride = a.ld * a.es;
  if (stride == b.ld * b.es) {
    const Operand &lo = a.base < b.base ? a : b, &hi = a.base < b.base ? b : a;
    const int64_t d = (int64_t)((hi.base - lo.base) % (uintptr_t)stride);
    if (d >= lo.cols * lo.es && d + hi.cols * hi.es <= stride) return false;
  }
  return true;
}

inline bool same_operand(const Operand& a, const Operand& b) {
  return a.base == b.base && a.es == b.es && a.rows == b.rows && a.cols == b.cols &&
         (a.ld == b.ld || a.rows <= 1);
}

// The operands of a call as they are gathered: inputs, outputs, and which inputs an
// output may equal exactly.
struct Operands {
  static constexpr int N = 8;
  Operand in[N], out[N];
  int allowed[N];  // bit j: out[i] may equal in[j]
  int ni = 0, no = 0;

  int read(const Operand& o) {
    in[ni] = o;
    return 1 << ni++;
  }
  void write(const Operand& o, int may_equal = 0) {
    out[no] = o;
    allowed[no++] = may_equal;
  }
  // CONV_ERR_ARG for an operand off its elements, then CONV_ERR_OVERLAP for an output
  // that meets an input, another output or the scratch, or an input that meets it.
  int check(const void* scratch, int64_t scratch_bytes) const {
    for (int i = 0; i < ni; ++i)
      if (!on_elements(in[i])) return CONV_ERR_ARG;
    for (int i = 0; i < no; ++i)
      if (!on_elements(out[i])) return CONV_ERR_ARG;
    const Operand s = {(uintptr_t)scratch, scratch_bytes > 0 ? 1 : 0, scratch_bytes, scratch_bytes, 1};
    for (int i = 0; i < no; ++i) {
      for (int j = 0; j < ni; ++j) {
        if ((allowed[i] >> j & 1) && same_operand(out[i], in[j])) continue;
        if (operands_meet(out[i], in[j])) return CONV_ERR_OVERLAP;
      }
      for (int j = i + 1; j < no; ++j)
        if (operands_meet(out[i], out[j])) return CONV_ERR_OVERLAP;
      if (operands_meet(out[i], s)) return CONV_ERR_OVERLAP;
    }
    for (int j = 0; j < ni; ++j)
      if (operands_meet(in[j], s)) return CONV_ERR_OVERLAP;
    return CONV_OK;
  }
};

inline int scratch_fits(const void* scratch, uint64_t bytes, int64_t need) {
  if (need == 0) return CONV_OK;
  if (bytes < (uint64_t)need) return CONV_ERR_SCRATCH;
  if (!scratch || (uintptr_t)scratch % 256 != 0) return CONV_ERR_ARG;
  return CONV_OK;
}

inline bool float_dtype(int dtype) {
  return dtype == CONV_F32 || dtype == CONV_F16 || dtype == CONV_BF16;
}

inline const char* float_dtype_name(int dtype) {
  return dtype == CONV_F16 ? "f16" : dtype == CONV_BF16 ? "bf16" : "f32";
}

inline int put_name(const char* text, char* buf, uint64_t len) {
  const size_t need = strlen(text) + 1;
  if (!buf || len < need) return CONV_ERR_ARG;
  memcpy(buf, text, need);
  return CONV_OK;
}

}  // namespace convfwd
