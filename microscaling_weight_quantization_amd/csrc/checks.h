// Host-side argument checks of the FP8 group quantizer, the FP8 products and the
// expert routing (group_quant.hip, product.hip, experts.hip): byte ranges of the
// operands, overlap, alignment, launch status.  mxq.hip has the same rules in
// its own words, for its own list-of-weights calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <initializer_list>

#include "mxq.h"

namespace mxq_host {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Bytes [lo, hi) of an operand.  ok is false where the span cannot be a real
// allocation: 2^56 bytes or more, or past the end of the address space.
struct Range {
  uintptr_t lo, hi;
  bool ok;
};

// A [rows, cols] matrix with row stride ld; an empty one is an empty range.
inline Range matrix_range(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esize) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (rows <= 0 || cols <= 0) return Range{lo, lo, true};
  const __int128 span = ((__int128)(rows - 1) * ld + cols) * (__int128)esize;
  const bool ok = span > 0 && span < ((__int128)1 << 56) && (unsigned __int128)lo + span <= UINTPTR_MAX;
  return Range{lo, ok ? lo + (uintptr_t)span : lo, ok};
}

// `count` such matrices, `stride` elements apart.
inline Range stack_range(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                         size_t esize) {
  const Range one = matrix_range(p, rows, cols, ld, esize);
  if (!one.ok || one.lo == one.hi || count <= 1) return one;
  const __int128 span = (__int128)(count - 1) * stride * (__int128)esize + (__int128)(one.hi - one.lo);
  const bool ok = span > 0 && span < ((__int128)1 << 56) && (unsigned __int128)one.lo + span <= UINTPTR_MAX;
  return Range{one.lo, ok ? one.lo + (uintptr_t)span : one.lo, ok};
}

inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

// No output shares a byte with an input or with another output.
inline bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(*o, i)) return false;
    for (auto p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return false;
  }
  return true;
}

inline bool all_ok(std::initializer_list<Range> rs) {
  for (const Range& r : rs)
    if (!r.ok) return false;
  return true;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

// A launch has fewer than 2^32 lanes in a dimension.  Calls that need more go out as
// launches of up to 2^31: this many rows each, of `lanes` lanes (at most 2^31) a row.
inline int64_t rows_per_launch(int64_t lanes) { return ((int64_t)1 << 31) / lanes; }

inline bool is_float(mxq_dtype dt) { return dt == MXQ_BF16 || dt == MXQ_FP32; }
inline size_t size_of(mxq_dtype dt) { return dt == MXQ_BF16 ? 2 : 4; }
inline int64_t groups_of(int64_t n) { return (n + 127) / 128; }

// Rows, columns and slots are counted in 32 bits on the device.
constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxExperts = 512;

}  // namespace mxq_host
