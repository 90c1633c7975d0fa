// group_quant.hip -- FP8 (E4M3) quantization of activations and gradients with
// one E8M0 code for each group of 128, on gfx950.
//
// How a group gets its code and payload stands in group128.h.
//
// Everything is bound by the bytes moved: x is read once, whether the groups
// run along the rows, along the columns or both ways.
// Both ways over 270 MB take 50.5 us (5.3 TB/s; a plain copy reaches 6.6); a single
// token takes 9.1 us, nearly all of it the launch and the call on the host.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "fastdiv.h"
#include "group128.h"

namespace {

using namespace mxq_host;
using namespace mxq_dev;

struct Source {
  const void* x;
  int64_t ld;
  int x_rows;
  const int32_t* slots;   // null: row r reads row r of x
  MxqDivisor top_k;
};

// The row of x that row r of the result reads; -1: none (a dropped slot, or one out of range).
__device__ __forceinline__ int source_row(const Source& s, int r) {
  if (!s.slots) return r;
  const int slot = s.slots[r];
  if (slot < 0) return -1;
  const int row = (int)mxq_quot((uint32_t)slot, s.top_k);
  return row < s.x_rows ? row : -1;
}

// ---- groups along the rows ------------------------------------------------------------
// 16 lanes per group, 16 groups per workgroup, one group a lane.
constexpr int kRowThreads = 256;

template <typename T, bool kVec>
__global__ __launch_bounds__(kRowThreads) void row_groups_kernel(Source src, int K, MxqDivisor groups, uint32_t total,
                                                                 uint8_t* data, int64_t ld_data, uint8_t* scale,
                                                                 int64_t scale_ld) {
  keep_denormals();
  const uint32_t g = blockIdx.x * (kRowThreads / 16) + threadIdx.x / 16;
  if (g >= total) return;   // whole groups of 16 lanes leave together
  const uint32_t r = mxq_quot(g, groups), b = g - r * groups.d;
  const int c = (int)b * kGroup + (threadIdx.x & 15) * kEPL;
  const int from = source_row(src, (int)r);
  Chunk<T> v = load_chunk<T, kVec>((const T*)src.x + (from < 0 ? 0 : from) * src.ld, from < 0 ? K : c, K);
  const uint32_t code = code_of<T>(max16(v.amax()));
  store_chunk<kVec, false>(data + (int64_t)r * ld_data, c, K, payload_of(v, code));
  if ((threadIdx.x & 15) == 0) scale[(int64_t)r * scale_ld + b] = (uint8_t)code;
}

// ---- groups along the columns, and along both -------------------------------------------
template <typename T, bool kVec, bool kRow, bool kStream>
__global__ __launch_bounds__(kTileThreads) void tile_groups_kernel(Source src, int first_id, int rows,
                                                                   const int32_t* offsets, int experts, TileOut out) {
  keep_denormals();
  __shared__ TileShared<kTileRows> shared;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup + (threadIdx.x & 15) * kEPL;
  const TileRows t = tile_rows(offsets, experts, rows, id, shared);
  if (!t.owned) clear_codes(out, id, blockIdx.x);
  if (t.first >= t.hi) return;   // the same for the whole workgroup
  Chunk<T> v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = t.first + threadIdx.x / 16 + 16 * i;
    const int from = r < t.hi ? source_row(src, (int)r) : -1;
    v[i] = load_chunk<T, kVec>((const T*)src.x + (from < 0 ? 0 : from) * src.ld, from < 0 ? out.K : c, out.K);
  }
  if (kVec && whole_tile(t, blockIdx.x, out.K)) store_tile<T, kVec, kRow, kStream, kVec>(v, out, t, id, blockIdx.x, shared);
  else store_tile<T, kVec, kRow, kStream, false>(v, out, t, id, blockIdx.x, shared);
}

struct Checked {
  Source src;
  Range rx, rslots, roff;
};

// The checks that all forms share.  For a call with nothing to do *empty is set.
int check_source(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
                 const int32_t* slots, int64_t top_k, const int32_t* offsets, int64_t experts, Checked* out,
                 bool* empty) {
  *empty = false;
  if (!is_float(dt)) return MXQ_ERR_DTYPE;
  if (rows < 0 || K < 0 || x_rows < 0 || rows > kMaxDim || K > kMaxDim || x_rows > kMaxDim) return MXQ_ERR_SHAPE;
  if (slots ? top_k < 1 || top_k > kMaxDim : rows > x_rows) return MXQ_ERR_SHAPE;
  if (offsets && (experts < 1 || experts > kMaxExperts)) return MXQ_ERR_SHAPE;
  if (rows == 0 || K == 0) {
    *empty = true;
    return MXQ_OK;
  }
  if (!x && x_rows > 0) return MXQ_ERR_NULL;
  if (ld_x < K) return MXQ_ERR_SHAPE;
  out->rx = matrix_range(x, x_rows, K, ld_x, size_of(dt));
  out->rslots = matrix_range(slots, 1, slots ? rows : 0, rows, 4);
  out->roff = matrix_range(offsets, 1, offsets ? experts + 1 : 0, experts + 1, 4);
  if (!all_ok({out->rx, out->rslots, out->roff}) || !aligned(slots, 4) || !aligned(offsets, 4) ||
      !aligned(x, size_of(dt)))
    return MXQ_ERR_SHAPE;
  out->src = Source{x, ld_x, (int)x_rows, slots, mxq_divisor(slots ? (uint32_t)top_k : 1u)};
  return MXQ_OK;
}

bool vector_input(const void* x, int64_t ld_x, int64_t K, mxq_dtype dt) {
  return aligned(x, 16) && ld_x % (16 / (int64_t)size_of(dt)) == 0 && K % kEPL == 0;
}
bool vector_payload(const uint8_t* p, int64_t ld) { return aligned(p, 8) && ld % 8 == 0; }

template <typename T>
int launch_rows(const Checked& c, int64_t rows, int64_t K, bool vec, uint8_t* data, int64_t ld_data, uint8_t* scale,
                int64_t scale_ld, hipStream_t stream) {
  const int64_t groups = groups_of(K), step = rows_per_launch(groups * 16);
  const MxqDivisor d = mxq_divisor((uint32_t)groups);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t total = std::min(step, rows - r) * groups;
    const dim3 grid((uint32_t)((total + kRowThreads / 16 - 1) / (kRowThreads / 16)));
    Source src = c.src;   // from row r of the result on
    if (src.slots) src.slots += r;
    else src.x = (const T*)src.x + r * src.ld;
    if (vec)
      hipLaunchKernelGGL((row_groups_kernel<T, true>), grid, dim3(kRowThreads), 0, stream, src, (int)K, d,
                         (uint32_t)total, data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    else
      hipLaunchKernelGGL((row_groups_kernel<T, false>), grid, dim3(kRowThreads), 0, stream, src, (int)K, d,
                         (uint32_t)total, data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
  return MXQ_OK;
}

template <typename T>
int launch_tiles(const Checked& c, int64_t rows, int64_t K, bool vec, const int32_t* offsets, int64_t experts,
                 int64_t code_rows, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale, int64_t row_scale_ld,
                 uint8_t* col_data, int64_t ld_col, uint8_t* col_scale, int64_t col_scale_ld, hipStream_t stream) {
  const int64_t tiles = code_rows + (offsets ? 2 : 0);   // the rows of no expert, behind and before the others, may take two more
  constexpr int64_t kStep = 65535;   // of a grid's second dimension
  const dim3 block(kTileThreads);
  const TileOut out{(int)K, (int)code_rows, row_data, ld_row, row_scale, row_scale_ld, col_data, ld_col, col_scale,
                    col_scale_ld};
#define MXQ_TILE_LAUNCH(V, R, S)                                                                                       \
  hipLaunchKernelGGL((tile_groups_kernel<T, V, R, S>), grid, block, 0, stream, c.src, (int)t, (int)rows, offsets,      \
                     (int)experts, out)
  const bool big = rows * K > kStreamBytes;
  for (int64_t t = 0; t < tiles; t += kStep) {
    const dim3 grid((uint32_t)groups_of(K), (uint32_t)std::min(kStep, tiles - t));
    if (row_data) {
      if (!vec) MXQ_TILE_LAUNCH(false, true, false);
      else if (big) MXQ_TILE_LAUNCH(true, true, true);
      else MXQ_TILE_LAUNCH(true, true, false);
    } else {
      if (!vec) MXQ_TILE_LAUNCH(false, false, false);
      else if (big) MXQ_TILE_LAUNCH(true, false, true);
      else MXQ_TILE_LAUNCH(true, false, false);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_TILE_LAUNCH
  return MXQ_OK;
}

int tile_entry(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
               const int32_t* slots, int64_t top_k, const int32_t* offsets, int64_t experts, bool row,
               uint8_t* row_data, int64_t ld_row, uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data,
               int64_t ld_col, uint8_t* col_scale, int64_t col_scale_ld, hipStream_t stream) {
  Checked c;
  bool empty;
  const int st = check_source(x, ld_x, x_rows, rows, K, dt, slots, top_k, offsets, experts, &c, &empty);
  if (st != MXQ_OK) return st;
  if (empty) return offsets && rows == 0 ? clear_code_rows(col_scale, col_scale_ld, experts, K, offsets, stream) : MXQ_OK;
  if (!col_data || !col_scale || (row && (!row_data || !row_scale))) return MXQ_ERR_NULL;
  if (ld_col < K || col_scale_ld < K || (row && (ld_row < K || row_scale_ld < groups_of(K)))) return MXQ_ERR_SHAPE;
  const int64_t code_rows = offsets ? rows / kGroup + experts : groups_of(rows);
  const Range cd = matrix_range(col_data, rows, K, ld_col, 1), cs = matrix_range(col_scale, code_rows, K, col_scale_ld, 1);
  const Range rd = matrix_range(row_data, row ? rows : 0, K, ld_row, 1),
              rs = matrix_range(row_scale, row ? rows : 0, groups_of(K), row_scale_ld, 1);
  if (!all_ok({cd, cs, rd, rs})) return MXQ_ERR_SHAPE;
  if (!disjoint({cd, cs, rd, rs}, {c.rx, c.rslots, c.roff})) return MXQ_ERR_ALIAS;
  const bool vec = vector_input(x, ld_x, K, dt) && vector_payload(col_data, ld_col) &&
                   (!row || vector_payload(row_data, ld_row));
  if (!row) row_data = row_scale = nullptr;
  return dt == MXQ_BF16
             ? launch_tiles<uint16_t>(c, rows, K, vec, offsets, experts, code_rows, row_data, ld_row, row_scale,
                                      row_scale_ld, col_data, ld_col, col_scale, col_scale_ld, stream)
             : launch_tiles<uint32_t>(c, rows, K, vec, offsets, experts, code_rows, row_data, ld_row, row_scale,
                                      row_scale_ld, col_data, ld_col, col_scale, col_scale_ld, stream);
}

}  // namespace

extern "C" {

int mxq_quantize_fp8_group128(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
                              const int32_t* slots, int64_t top_k, uint8_t* data, int64_t ld_data, uint8_t* scale,
                              int64_t scale_ld, hipStream_t stream) {
  Checked c;
  bool empty;
  const int st = check_source(x, ld_x, x_rows, rows, K, dt, slots, top_k, nullptr, 0, &c, &empty);
  if (st != MXQ_OK || empty) return st;
  if (!data || !scale) return MXQ_ERR_NULL;
  if (ld_data < K || scale_ld < groups_of(K)) return MXQ_ERR_SHAPE;
  const Range rd = matrix_range(data, rows, K, ld_data, 1), rs = matrix_range(scale, rows, groups_of(K), scale_ld, 1);
  if (!all_ok({rd, rs})) return MXQ_ERR_SHAPE;
  if (!disjoint({rd, rs}, {c.rx, c.rslots})) return MXQ_ERR_ALIAS;
  const bool vec = vector_input(x, ld_x, K, dt) && vector_payload(data, ld_data);
  return dt == MXQ_BF16 ? launch_rows<uint16_t>(c, rows, K, vec, data, ld_data, scale, scale_ld, stream)
                        : launch_rows<uint32_t>(c, rows, K, vec, data, ld_data, scale, scale_ld, stream);
}

int mxq_quantize_fp8_group128_col(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K, mxq_dtype dt,
                                  const int32_t* slots, int64_t top_k, const int32_t* offsets, int64_t n_experts,
                                  uint8_t* data, int64_t ld_data, uint8_t* scale, int64_t scale_ld,
                                  hipStream_t stream) {
  return tile_entry(x, ld_x, x_rows, rows, K, dt, slots, top_k, offsets, n_experts, false, nullptr, 0, nullptr, 0,
                    data, ld_data, scale, scale_ld, stream);
}

int mxq_quantize_fp8_group128_row_col(const void* x, int64_t ld_x, int64_t x_rows, int64_t rows, int64_t K,
                                      mxq_dtype dt, const int32_t* slots, int64_t top_k, const int32_t* offsets,
                                      int64_t n_experts, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, hipStream_t stream) {
  return tile_entry(x, ld_x, x_rows, rows, K, dt, slots, top_k, offsets, n_experts, true, row_data, ld_row, row_scale,
                    row_scale_ld, col_data, ld_col, col_scale, col_scale_ld, stream);
}

}  // extern "C"
