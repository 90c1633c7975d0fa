// Groups of 128 in FP8 (E4M3) with one E8M0 code each, as the kernels that write them share it: eight elements a
// lane, sixteen lanes a group of a row, a workgroup of 256 lanes a tile of 128 x 128 for groups along the columns.
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
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checks.h"
#include "segments.h"

namespace mxq_dev {

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

// The larger magnitude of two fp32 values, a NaN if one of them is: one instruction for three values.
__device__ __forceinline__ float larger(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}
__device__ __forceinline__ uint32_t magnitude_bits(float m) { return __builtin_bit_cast(uint32_t, m) & 0x7FFFFFFFu; }

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
    if constexpr (sizeof(T) == 4) {
      float m = value(0);
#pragma unroll
      for (int i = 1; i < kEPL; i++) m = larger(m, value(i));
      return magnitude_bits(m);
    }
    uint32_t m = mag(0);
#pragma unroll
    for (int i = 1; i < kEPL; i++) m = max(m, mag(i));
    return m;
  }
  __device__ __forceinline__ float value(int i) const { return __builtin_bit_cast(float, w[i]); }   // of fp32
  // Four payload bytes of elements 4 h .. 4 h + 3 at scale 2^(code - 127).
  __device__ __forceinline__ uint32_t e4m3x4(int h, uint32_t code) const {
    const float s = __builtin_bit_cast(float, code << 23);   // code 0 stands for 2^-127 here
    s16x2 r = __builtin_nondeterministic_value(r);           // both halves are written
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

// The same 16 and 8 bytes at any address: the hardware's loads and stores take them.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// Elements [c, c + 8) of a row of K; those from K on are 0.  kVec: rows lie at multiples of 16 bytes and K is a multiple of 8.
// kOnce: with the non-temporal hint, for rows that nothing reads again soon.
template <typename T, bool kVec, bool kOnce = false>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c, int K) {
  Chunk<T> v;
  if (kVec ? c < K : c + kEPL <= K) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::kWords / 4; i++) {
      if constexpr (kVec) {
        const u32x4* p = reinterpret_cast<const u32x4*>(row + c) + i;
        reinterpret_cast<u32x4*>(v.w)[i] = kOnce ? __builtin_nontemporal_load(p) : *p;
      } else {
        reinterpret_cast<u32x4*>(v.w)[i] = reinterpret_cast<const u32x4_any*>(row + c)[i];
      }
    }
    return v;
  }
#pragma unroll
  for (int i = 0; i < Chunk<T>::kWords; i++) v.w[i] = 0;
  if (!kVec && c < K) {   // the end of the row
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
  } else if (c + kEPL <= K) {
    *reinterpret_cast<u32x2_any*>(row + c) = v;
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

// Lane rows (16 lanes) 1 and 3 of a change places with rows 0 and 2 of b; the upper half of a with the lower of b.
__device__ __forceinline__ u32x2 swap16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
}
__device__ __forceinline__ u32x2 swap32(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
}

template <typename T>
__device__ __forceinline__ u32x2 payload_of(const Chunk<T>& v, uint32_t code) {
  if (code == 255u) return u32x2{kPoison4, kPoison4};
  return u32x2{v.e4m3x4(0, code), v.e4m3x4(1, code)};
}

// ---- groups along the columns, and along both -------------------------------------------
// A workgroup takes a tile of 128 rows x 128 columns, which holds whole groups
// both ways: 16 lanes across a row, 16 or 32 rows at a time, 8 or 4 rows a lane, all of it
// in registers.  A column's largest magnitude is reduced over a lane's rows, over
// the wave's four lane rows and, through LDS, over the waves.
constexpr int kTileThreads = 256, kTileRows = kGroup / (kTileThreads / 16);
// Payloads of more than the L2s hold (32 MiB) leave with the non-temporal hint:
// 5000 x 8192 bf16 both ways 34.9 -> 26.2 us, 8192 x 8192 fp32 74.0 -> 70.8 us, bf16
// 52.4 -> 50.5 us.  The row kernel was 3% slower with it.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

struct TileOut {
  int K, code_rows;
  uint8_t* row_data;
  int64_t ld_row;
  uint8_t* row_scale;
  int64_t row_scale_ld;
  uint8_t* col_data;
  int64_t ld_col;
  uint8_t* col_scale;
  int64_t col_scale_ld;
};
// Rows of a tile: `first` to `hi`; owned: they are an expert's (or there are no experts).
struct TileRows {
  int64_t first, hi;
  bool owned;
  __device__ __forceinline__ int have() const { return (int)min(hi - first, (int64_t)kGroup); }
};

// In LDS, for a workgroup whose lanes hold kRows rows each: 256 lanes with eight or 512 with four.
template <int kRows>
struct TileShared {
  static constexpr int kThreads = 16 * kGroup / kRows;
  uint32_t amax[kThreads / 64][kGroup];
  float scale[kGroup];
  int poisoned[2];   // of the first and of the second matrix that the workgroup stores
  TileRows rows;
};

// The rows of tile `id`, found by the first wave for all.  Every lane calls it, before store_tile.
template <int kRows>
__device__ __forceinline__ TileRows tile_rows(const int32_t* offsets, int experts, int rows, int id,
                                              TileShared<kRows>& sh) {
  if (threadIdx.x < 2) sh.poisoned[threadIdx.x] = 0;   // seen by all behind store_tile's first barrier
  if (!offsets) return TileRows{(int64_t)id * kGroup, rows, true};
  if (threadIdx.x < 64) {
    const Segment s = find_tile<kGroup>(offsets, experts, rows, id);
    if (threadIdx.x == 0) sh.rows = TileRows{(int64_t)s.lo + (int64_t)s.tile * kGroup, s.hi, s.expert < experts};
  }
  __syncthreads();
  // the same for all lanes, and known to be
  const auto uniform = [](int64_t v) {
    return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
           (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
  };
  return TileRows{uniform(sh.rows.first), uniform(sh.rows.hi), __builtin_amdgcn_readfirstlane((int)sh.rows.owned) != 0};
}

// The code row of a tile that no expert owns is one that no group needs: zeros in the columns of tile column `at`.
__device__ __forceinline__ void clear_codes(const TileOut& o, int id, int at) {
  const int c = at * kGroup + (int)threadIdx.x;
  if (id < o.code_rows && threadIdx.x < kGroup && c < o.K) o.col_scale[(int64_t)id * o.col_scale_ld + c] = 0;
}

// Payloads and codes of the tile in tile column `at` of which this lane holds every kStep-th row from row16 on (zeros
// where there is no such row).  All lanes of the workgroup call it, once, or a second time with kSecond.  kWhole: the tile
// has 128 rows and 128 columns.
template <typename T, bool kVec, bool kRow, bool kStream, bool kWhole, bool kSecond = false, int kRows>
__device__ __forceinline__ void store_tile(const Chunk<T> (&v)[kRows], const TileOut& o, const TileRows& t, int id,
                                           int at, TileShared<kRows>& sh) {
  constexpr int kStep = kGroup / kRows;
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x / 16, wave = threadIdx.x / 64;
  const int c = at * kGroup + lane16 * kEPL;
  const int have = kWhole ? kGroup : t.have();
  if constexpr (kRow) {
    uint8_t* p = o.row_data + t.first * o.ld_row + row16 * o.ld_row;
    uint32_t mine = 0;   // lane i of the 16 stores the code of their i-th row
#pragma unroll
    for (int i = 0; i < kRows; i++) {
      if (kWhole || kStep * i < have) {   // the same for the whole workgroup
        const uint32_t code = code_of<T>(max16(v[i].amax()));
        if (kWhole || row16 + kStep * i < have) store_chunk<kVec, kStream>(p, c, kWhole ? c + 1 : o.K, payload_of(v[i], code));
        mine = lane16 == i ? code : mine;
      }
      p += kStep * o.ld_row;
    }
    const int r = row16 + kStep * lane16;
    if (lane16 < kRows && (kWhole || r < have)) o.row_scale[t.first * o.row_scale_ld + r * o.row_scale_ld + at] = (uint8_t)mine;
  }
  uint8_t* p = o.col_data + t.first * o.ld_col + row16 * o.ld_col;
  if (!t.owned) {   // the same for the whole workgroup
#pragma unroll
    for (int i = 0; i < kRows; i++) {
      if (kWhole || row16 + kStep * i < have) store_chunk<kVec, kStream>(p, c, kWhole ? c + 1 : o.K, u32x2{0, 0});
      p += kStep * o.ld_col;
    }
    return;
  }
  uint32_t m[kEPL];
#pragma unroll
  for (int j = 0; j < kEPL; j++) {
    if constexpr (sizeof(T) == 4) {
      float f = v[0].value(j);
#pragma unroll
      for (int i = 1; i < kRows; i++) f = larger(f, v[i].value(j));
      m[j] = magnitude_bits(f);
    } else {
      m[j] = v[0].mag(j);
#pragma unroll
      for (int i = 1; i < kRows; i++) m[j] = max(m[j], v[i].mag(j));
    }
  }
  // The wave's four lane rows: swaps leave lane row q with the whole wave's columns q and 4 + q.
#pragma unroll
  for (int j = 0; j < kEPL; j += 2) {
    const u32x2 s = swap16(m[j], m[j + 1]);
    m[j / 2] = max(s[0], s[1]);
  }
#pragma unroll
  for (int j = 0; j < kEPL / 2; j += 2) {
    const u32x2 s = swap32(m[j], m[j + 1]);
    sh.amax[wave][lane16 * kEPL + (threadIdx.x & 63) / 16 + 2 * j] = max(s[0], s[1]);
  }
  __syncthreads();
  if (threadIdx.x < kGroup) {   // a column a lane
    const int k = threadIdx.x;
    uint32_t amax = sh.amax[0][k];
#pragma unroll
    for (int w = 1; w < TileShared<kRows>::kThreads / 64; w++) amax = max(amax, sh.amax[w][k]);
    const uint32_t code = code_of<T>(amax);
    sh.scale[k] = __builtin_bit_cast(float, code << 23);   // code 0 stands for 2^-127 here
    if (code == 255u) sh.poisoned[kSecond] = 1;
    if (id < o.code_rows && (kWhole || at * kGroup + k < o.K))
      o.col_scale[(int64_t)id * o.col_scale_ld + at * kGroup + k] = (uint8_t)code;
  }
  __syncthreads();
  float scale[kEPL];
#pragma unroll
  for (int j = 0; j < kEPL; j++) scale[j] = sh.scale[lane16 * kEPL + j];
  u32x2 poison{0, 0};
  if (sh.poisoned[kSecond]) {   // the same for the whole workgroup
#pragma unroll
    for (int j = 0; j < kEPL; j++)
      if (__builtin_bit_cast(uint32_t, scale[j]) == 255u << 23) poison[j / 4] |= 0xFFu << (8 * (j & 3));
  }
  // Two rows at a time: a conversion takes two values of one scale, so a column's pair of rows.
#pragma unroll
  for (int i = 0; i < kRows; i += 2) {
    if (!kWhole && kStep * i >= have) break;   // the same for the whole workgroup
    uint32_t pair[kEPL / 2];   // bytes: row i, row i + 1 of column 2 j, then of column 2 j + 1
#pragma unroll
    for (int j = 0; j < kEPL / 2; j++) {
      s16x2 b = __builtin_nondeterministic_value(b);   // both halves are written
      if constexpr (sizeof(T) == 2) {
        const uint32_t lo = __builtin_amdgcn_perm(v[i + 1].w[j], v[i].w[j], 0x05040100u);
        const uint32_t hi = __builtin_amdgcn_perm(v[i + 1].w[j], v[i].w[j], 0x07060302u);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(bf16x2, lo), scale[2 * j], false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(bf16x2, hi), scale[2 * j + 1], true);
      } else {
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[i].value(2 * j), v[i + 1].value(2 * j), scale[2 * j], false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[i].value(2 * j + 1), v[i + 1].value(2 * j + 1),
                                                     scale[2 * j + 1], true);
      }
      pair[j] = __builtin_bit_cast(uint32_t, b);
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const uint32_t pick = k ? 0x07050301u : 0x06040200u;
      u32x2 q{__builtin_amdgcn_perm(pair[1], pair[0], pick), __builtin_amdgcn_perm(pair[3], pair[2], pick)};
      q = (q & ~poison) | (poison & kPoison4);
      if (kWhole || row16 + kStep * (i + k) < have) store_chunk<kVec, kStream>(p, c, kWhole ? c + 1 : o.K, q);
      p += kStep * o.ld_col;
    }
  }
}

// Whether the tile in tile column `at` has 128 rows and 128 columns.
__device__ __forceinline__ bool whole_tile(const TileRows& t, int at, int K) {
  return t.hi - t.first >= kGroup && (at + 1) * kGroup <= K;
}

// A column a lane, a code row a workgroup's row.
template <int kThreads>
__global__ __launch_bounds__(kThreads) void clear_code_rows_kernel(uint8_t* scale, int64_t ld, int K) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c < K) scale[blockIdx.y * ld + c] = 0;
}

}  // namespace mxq_dev

namespace mxq_host {

// A call by expert on no rows: its code rows, one an expert, are all ones that no group needs.  Without a place for them
// there is nothing to do.
template <int kThreads = 256>
int clear_code_rows(uint8_t* scale, int64_t ld, int64_t experts, int64_t K, const int32_t* offsets, hipStream_t stream) {
  if (!scale || K == 0) return MXQ_OK;
  const Range rs = matrix_range(scale, experts, K, ld, 1), ro = matrix_range(offsets, 1, experts + 1, experts + 1, 4);
  if (ld < K || !all_ok({rs, ro}) || !aligned(offsets, 4)) return MXQ_ERR_SHAPE;
  if (overlap(rs, ro)) return MXQ_ERR_ALIAS;
  const dim3 grid((uint32_t)((K + kThreads - 1) / kThreads), (uint32_t)experts);
  hipLaunchKernelGGL((mxq_dev::clear_code_rows_kernel<kThreads>), grid, dim3(kThreads), 0, stream, scale, ld, (int)K);
  return launch_status();
}

}  // namespace mxq_host
