// Which kernel a product of FP8 operands takes.  All compute the same sums; the
// choice is made on sizes and alignment alone, from sweeps over 1 to 3000 rows,
// 1024 to 28672 columns and 8 to 128 experts.
//
// Plain C++ (no HIP types): product.hip uses it, and so does a host test that pins
// which sizes reach which kernel.
#pragma once

#include <stdint.h>

namespace mxq_host {

constexpr int64_t kCUs = 256;

enum Mode { kForward, kDgrad, kWgrad };

enum ProductKernel {
  kFewRows16,       // few rows, 16, 32 or 64 of them a workgroup
  kFewRows32,
  kFewRows64,
  kTiles128,        // FP8 sums, tiles of 128 x 128 or 256 x 256 results
  kTiles256,
  kCarried,         // FP8 sums, rows of any alignment
  kExact,           // sums in fp32
  kExactCarried,    // sums in fp32, rows of any alignment
};

// Tiles of B x B of the I x J outputs that have rows, as far as the host can tell: it does not
// read the offsets, and takes every expert to have its share.  experts is 0 for one weight.
inline int64_t tiles_of(int64_t I, int64_t J, int64_t experts, int64_t B) {
  const int64_t ti = experts ? I / B + (I < experts ? I : experts) : (I + B - 1) / B;
  return ti * ((J + B - 1) / B);
}

// fast: the FP8 instructions' sums; fed: rows that can be fed straight to LDS.
inline ProductKernel choose_kernel(Mode mode, bool fast, bool fed, int64_t I, int64_t J, int64_t experts) {
  if (mode != kWgrad) {
    // Rows that meet one weight: all of them, or an expert's share.
    const int64_t rows = experts ? (I + experts - 1) / experts : I;
    // The few-rows kernels read V anew for every 64 columns and U for every 64
    // rows, so they are the faster ones while they make about one workgroup for
    // each CU (192 rows x 4096 x 4096: 25.7 us against 29.3 in tiles; 192 x 8192 x
    // 8192: 83.7 against 53.0), and beyond for the fewest rows.  Where 128 x 128 tiles
    // fill the card, those are up to 8 rows (y with FP8 sums: 5 rows each for 48 experts
    // 19.4 against 21.5, 12 rows 26.1 against 23.6), none (dx: 1 row 18.9 against
    // 13.7) or 32 (sums in fp32: 25 rows 39 against 45, 40 rows 69 against 45).  Where
    // they do not, as when fewer rows than experts come, up to 8, none or 16 (18 rows
    // for 48 experts of 1024 x 2048: 11.1 against 16.2, sums in fp32 12.2 against 22.0; 8
    // rows x 20480 x 4096: 26.4 against 35.2; 32 rows of dx in fp32: 50 against 40).
    // Unaligned rows reach the tiles through registers, so the few-rows kernels
    // hold out for twice as many.
    const int64_t step = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    const int64_t groups = ((J + 63) / 64) * (experts ? experts * ((rows + step - 1) / step) : (rows + step - 1) / step);
    const bool full = tiles_of(I, J, experts, 128) >= kCUs * 3 / 4;
    const int64_t most = !fast ? 32 : mode == kForward ? 8 : 0;
    const bool few = !fed ? rows <= 16 || groups <= 2 * kCUs
                   : full ? rows <= most
                          : rows <= (most < 16 ? most : 16) || groups <= kCUs;
    if (few)
      return step == 16 ? kFewRows16 : step == 32 ? kFewRows32 : kFewRows64;
  }
  if (!fast) return fed ? kExact : kExactCarried;
  if (!fed) return kCarried;
  // A CU has one 256 x 256 tile or two of 128 x 128 at a time.  A round of the
  // former takes 1.8 us for each reduction block, one of the latter 1.1 us.
  const int64_t big = (tiles_of(I, J, experts, 256) + kCUs - 1) / kCUs,
                small = (tiles_of(I, J, experts, 128) + 2 * kCUs - 1) / (2 * kCUs);
  return 18 * big <= 11 * small ? kTiles256 : kTiles128;
}

}  // namespace mxq_host
