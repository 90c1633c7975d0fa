// group_quant.hip -- FP8 (E4M3) quantization of activations and gradients with
// one E8M0 code for each group of 128, on gfx950.
//
// A group's largest magnitude is reduced as an integer on the bit patterns
// (sign cleared, bf16 and fp32 patterns order as their values do).  With A that
// pattern and E its exponent field, amax <= 448 * 2^S first holds at S = E - 127
// - 8 when the mantissa is at most 1.75 and one above otherwise, so the code is
// max(((A + 1/4 - 1 ulp) >> mantissa bits) - 8, 0).  The payload is rounded once,
// by the scaled conversion of the hardware (RTNE of x / 2^S onto E4M3 with
// subnormals; the scale is a power of two, so the division is exact).  An Inf or
// NaN pattern compares above every finite one and poisons its group: code 255,
// payload 0x7F.
//
// Everything is bound by the bytes moved: x is read once, whether the groups
// run along the rows, along the columns or both ways.
// Both ways over 270 MB take 52.7 us (5.1 TB/s; a plain copy reaches 6.6); a single
// token takes 9.5 us, nearly all of it the launch and the call on the host.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "fastdiv.h"
#include "segments.h"

namespace {

using namespace mxq_host;
using mxq_dev::Segment;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

constexpr int kGroup = 128;
constexpr int kEPL = 8;                  // elements per lane: 16 lanes hold a group of a row
constexpr uint32_t kPoison4 = 0x7F7F7F7Fu;

// FP_DENORM field of the MODE register: keep denormals, whatever the build's flags.
constexpr int kModeFpDenorm = 1 | (4 << 6) | (3 << 11);
__device__ __forceinline__ void keep_denormals() { __builtin_amdgcn_s_setreg(kModeFpDenorm, 0xF); }

// Eight elements of a row as their bit patterns.
template <typename T>
struct Chunk {
  static constexpr int kWords = sizeof(T) * kEPL / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ uint32_t mag(int i) const {
    if constexpr (sizeof(T) == 2) return (w[i / 2] >> (16 * (i & 1))) & 0x7FFFu;
    else return w[i] & 0x7FFFFFFFu;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = mag(0);
#pragma unroll
    for (int i = 1; i < kEPL; i++) m = max(m, mag(i));
    return m;
  }
  // Four payload bytes of elements 4 h .. 4 h + 3 at scale 2^(code - 127).
  __device__ __forceinline__ uint32_t e4m3x4(int h, uint32_t code) const {
    const float s = __builtin_bit_cast(float, code << 23);   // code 0 stands for 2^-127 here
    s16x2 r{0, 0};
    if constexpr (sizeof(T) == 2) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[2 * h]), s, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w[2 * h + 1]), s, true);
    } else {
      const float* f = reinterpret_cast<const float*>(w) + 4 * h;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, f[0], f[1], s, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, f[2], f[3], s, true);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
};

// Code of a group whose largest magnitude has this bit pattern; 255 where it holds an Inf or NaN.
template <typename T>
__device__ __forceinline__ uint32_t code_of(uint32_t amax) {
  constexpr int MB = sizeof(T) == 2 ? 7 : 23;
  constexpr uint32_t kInf = 0xFFu << MB;
  const int code = (int)((amax + ((1u << (MB - 2)) - 1u)) >> MB) - 8;
  return amax >= kInf ? 255u : (uint32_t)max(code, 0);
}

// Elements [c, c + 8) of a row of K; those from K on are 0.
template <typename T, bool kVec>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c, int K) {
  Chunk<T> v;
  if (kVec) {
    if (c < K) {
      const u32x4* p = reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
      for (int i = 0; i < Chunk<T>::kWords / 4; i++) reinterpret_cast<u32x4*>(v.w)[i] = p[i];
      return v;
    }
#pragma unroll
    for (int i = 0; i < Chunk<T>::kWords; i++) v.w[i] = 0;
  } else {
#pragma unroll
    for (int i = 0; i < Chunk<T>::kWords; i++) v.w[i] = 0;
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < K) {
        if constexpr (sizeof(T) == 2) v.w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        else v.w[i] = row[c + i];
      }
  }
  return v;
}

template <bool kVec, bool kStream>
__device__ __forceinline__ void store_chunk(uint8_t* row, int c, int K, u32x2 v) {
  if (kVec) {
    if (c < K) {
      if (kStream) __builtin_nontemporal_store(v, reinterpret_cast<u32x2*>(row + c));
      else *reinterpret_cast<u32x2*>(row + c) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < K) row[c + i] = (uint8_t)(v[i / 4] >> (8 * (i & 3)));
  }
}

// Largest value over the 16 lanes that hold one group of a row (a DPP row).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
  v = max(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  v = max(v, dpp<0x141>(v));   // row_half_mirror
  return max(v, dpp<0x140>(v));   // row_mirror
}

template <typename T>
__device__ __forceinline__ u32x2 payload_of(const Chunk<T>& v, uint32_t code) {
  if (code == 255u) return u32x2{kPoison4, kPoison4};
  return u32x2{v.e4m3x4(0, code), v.e4m3x4(1, code)};
}

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
// A workgroup takes a tile of 128 rows x 128 columns, which holds whole groups
// both ways: 16 lanes across a row, 16 rows at a time, 8 rows a lane, all of it
// in registers.  A column's largest magnitude is reduced over a lane's rows, over
// the wave's four lane rows and, through LDS, over the four waves.
constexpr int kTileThreads = 256, kTileRows = kGroup / (kTileThreads / 16);
// Payloads of more than the L2s hold (32 MiB) leave with the non-temporal hint:
// 5000 x 8192 bf16 both ways 36.2 -> 30.6 us, 8192 x 8192 fp32 76 -> 72 us, bf16
// 53.0 -> 54.0 us.  The row kernel was 3% slower with it.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

template <typename T, bool kVec, bool kRow, bool kStream>
__global__ __launch_bounds__(kTileThreads) void tile_groups_kernel(
    Source src, int first_id, int rows, int K, const int32_t* offsets, int experts, int code_rows, uint8_t* row_data,
    int64_t ld_row, uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
    int64_t col_scale_ld) {
  keep_denormals();
  __shared__ uint32_t part[kTileThreads / 64][kGroup];
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x / 16, wave = threadIdx.x / 64;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup + lane16 * kEPL;
  Segment s{0, id, 0, rows, 0};
  if (offsets) s = mxq_dev::find_tile<kGroup>(offsets, experts, rows, id);
  const bool owned = !offsets || s.expert < experts;
  // a code row that no group of an expert fills
  if (!owned && id < code_rows && row16 == 0) {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < K) col_scale[(int64_t)id * col_scale_ld + c + i] = 0;
  }
  const int64_t first = (int64_t)s.lo + (int64_t)s.tile * kGroup;
  if (first >= s.hi) return;   // the same for the whole workgroup
  Chunk<T> v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = first + row16 + 16 * i;
    const int from = r < s.hi ? source_row(src, (int)r) : -1;
    v[i] = load_chunk<T, kVec>((const T*)src.x + (from < 0 ? 0 : from) * src.ld, from < 0 ? K : c, K);
  }
  if constexpr (kRow) {
#pragma unroll
    for (int i = 0; i < kTileRows; i++) {
      const int64_t r = first + row16 + 16 * i;
      const uint32_t code = code_of<T>(max16(v[i].amax()));
      if (r < s.hi) {
        store_chunk<kVec, kStream>(row_data + r * ld_row, c, K, payload_of(v[i], code));
        if (lane16 == 0) row_scale[r * row_scale_ld + blockIdx.x] = (uint8_t)code;
      }
    }
  }
  uint32_t code[kEPL];
  if (owned) {   // the same for the whole workgroup
    uint32_t m[kEPL];
#pragma unroll
    for (int j = 0; j < kEPL; j++) {
      m[j] = v[0].mag(j);
#pragma unroll
      for (int i = 1; i < kTileRows; i++) m[j] = max(m[j], v[i].mag(j));
      m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
      m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32));
    }
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
      for (int j = 0; j < kEPL; j++) part[wave][lane16 * kEPL + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEPL; j++) {
      const int at = lane16 * kEPL + j;
      code[j] = code_of<T>(max(max(part[0][at], part[1][at]), max(part[2][at], part[3][at])));
    }
    if (row16 == 0 && id < code_rows) {
#pragma unroll
      for (int j = 0; j < kEPL; j++)
        if (c + j < K) col_scale[(int64_t)id * col_scale_ld + c + j] = (uint8_t)code[j];
    }
  }
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = first + row16 + 16 * i;
    if (r >= s.hi) continue;
    u32x2 q{0, 0};
    if (owned) {
#pragma unroll
      for (int j = 0; j < kEPL; j++) {
        uint32_t byte = 0x7F;
        if (code[j] != 255u) {
          const float sc = __builtin_bit_cast(float, code[j] << 23);
          s16x2 p{0, 0};
          if constexpr (sizeof(T) == 2) {
            const uint32_t one = (v[i].w[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
            p = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(p, __builtin_bit_cast(bf16x2, one), sc, false);
          } else {
            p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, __builtin_bit_cast(float, v[i].w[j]), 0.0f, sc, false);
          }
          byte = __builtin_bit_cast(uint32_t, p) & 0xFFu;
        }
        q[j / 4] |= byte << (8 * (j & 3));
      }
    }
    store_chunk<kVec, kStream>(col_data + r * ld_col, c, K, q);
  }
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
#define MXQ_TILE_LAUNCH(V, R, S)                                                                                      \
  hipLaunchKernelGGL((tile_groups_kernel<T, V, R, S>), grid, block, 0, stream, c.src, (int)t, (int)rows, (int)K, offsets, \
                     (int)experts, (int)code_rows, row_data, ld_row, row_scale, row_scale_ld, col_data, ld_col,    \
                     col_scale, col_scale_ld)
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
  if (st != MXQ_OK || empty) return st;
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
