// From a plan to a launch's arguments, for the products of the linear, gated and 8-bit
// linear calls.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "linear_args.h"
#include "linear_plan.h"

namespace convfwd {

template <typename T>
inline T* at(T* p, int64_t off, int es) {
  typedef std::conditional_t<std::is_const_v<T>, const char, char> C;
  return p ? static_cast<T*>(static_cast<C*>(p) + off * es) : nullptr;
}

// Rows that start on multiples of 4 bytes.
inline bool rows4(const void* p, int64_t ld, int es) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld * es % 4 == 0;
}

// Whether the operands can go to LDS directly: rows from multiples of 4 bytes, of
// whole 16-byte pieces or padded to that with zeros.
inline bool direct(const ProductShape& s, const ProductArgs& a, int es, bool p_padded, bool q_padded) {
  for (int i = 0; i < 2; ++i) {
    if (a.P[i] && !rows4(a.P[i], a.ldp, es)) return false;
    if (a.Q[i] && !rows4(a.Q[i], a.ldq, es)) return false;
  }
  if (!p_padded && (s.pt ? s.R : s.K) * es % 16 != 0) return false;
  return q_padded || (s.qt ? s.C : s.K) * es % 16 == 0;
}

// The plan into a product's arguments; its operands and epilogue are set.
inline void set_plan(const ProductShape& s, const ProductPlan& pl, void* planes, ProductArgs* a) {
  a->R = (int)s.R; a->C = (int)s.C; a->K = (int)s.K;
  a->nseg = s.nseg; a->nz = s.nz;
  a->ktiles = (int)pl.ktiles; a->splits = pl.splits; a->per_split = (int)pl.per_split;
  a->planes = static_cast<float*>(planes);
  a->plane_ld = pl.plane_ld;
  a->e.R = a->R;
}

inline JoinArgs join_of(const ProductShape& s, const ProductArgs& a) {
  JoinArgs j{};
  j.planes = a.planes;
  j.plane_ld = a.plane_ld;
  j.plane_stride = a.plane_ld * s.C * s.nz * (s.gated ? 2 : 1);
  j.splits = a.splits;
  j.C = a.C;
  j.nz = s.nz;
  j.e = a.e;
  return j;
}

// The copies of the operands that the plan packs; points src[i] and ld[i], the i-th item's
// operand (null: not wanted by this call), to them.  False: there are none.
inline bool fill_pack(const Packing& k, int es, const void** src, int64_t* ld, void* scratch,
                      PackArgs* out) {
  PackArgs a{};
  for (int i = 0; i < k.n; ++i) {
    const PackItem& q = k.item[i];
    if (!k.on || !q.need || !src[i] || q.rows == 0) continue;
    a.src[a.n] = src[i];
    a.dst[a.n] = static_cast<char*>(scratch) + q.off;
    a.ld[a.n] = ld[i];
    a.packed_ld[a.n] = q.packed_ld;
    a.pieces[a.n] = q.rows * (q.packed_ld * es / 16);
    a.cols[a.n] = (int)q.cols;
    a.first[a.n + 1] = a.first[a.n] + (int)ceil_div(a.pieces[a.n], 1024);
    src[i] = a.dst[a.n];
    ld[i] = q.packed_ld;
    ++a.n;
  }
  *out = a;
  return a.n > 0;
}

}  // namespace convfwd
