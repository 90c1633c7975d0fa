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
typedef uint32_t TilePart[kTileThreads / 64][kGroup];   // in LDS

// Rows of a tile: `first` to `hi`; owned: they are an expert's (or there are no experts).
struct TileRows {
  int64_t first, hi;
  bool owned;
};
__device__ __forceinline__ TileRows tile_rows(const int32_t* offsets, int experts, int rows, int id) {
  Segment s{0, id, 0, rows, 0};
  if (offsets) s = find_tile<kGroup>(offsets, experts, rows, id);
  return TileRows{(int64_t)s.lo + (int64_t)s.tile * kGroup, s.hi, !offsets || s.expert < experts};
}

// The code row of a tile that no expert owns is one that no group needs: zeros in the columns of tile column `at`.
__device__ __forceinline__ void clear_codes(const TileOut& o, int id, int at) {
  const int c = at * kGroup + (threadIdx.x & 15) * kEPL;
  if (id < o.code_rows && threadIdx.x / 16 == 0) {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < o.K) o.col_scale[(int64_t)id * o.col_scale_ld + c + i] = 0;
  }
}

// Payloads and codes of the tile in tile column `at` whose rows row16, row16 + 16, ... this lane holds (zeros
// where there is no such row).  All lanes of the workgroup call it; `part` is free again behind a barrier.
template <typename T, bool kVec, bool kRow, bool kStream>
__device__ __forceinline__ void store_tile(const Chunk<T> (&v)[kTileRows], const TileOut& o, const TileRows& t, int id,
                                           int at, TilePart& part) {
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x / 16, wave = threadIdx.x / 64;
  const int c = at * kGroup + lane16 * kEPL;
  if constexpr (kRow) {
#pragma unroll
    for (int i = 0; i < kTileRows; i++) {
      const int64_t r = t.first + row16 + 16 * i;
      const uint32_t code = code_of<T>(max16(v[i].amax()));
      if (r < t.hi) {
        store_chunk<kVec, kStream>(o.row_data + r * o.ld_row, c, o.K, payload_of(v[i], code));
        if (lane16 == 0) o.row_scale[r * o.row_scale_ld + at] = (uint8_t)code;
      }
    }
  }
  uint32_t code[kEPL];
  if (t.owned) {   // the same for the whole workgroup
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
      const int k = lane16 * kEPL + j;
      code[j] = code_of<T>(max(max(part[0][k], part[1][k]), max(part[2][k], part[3][k])));
    }
    if (row16 == 0 && id < o.code_rows) {
#pragma unroll
      for (int j = 0; j < kEPL; j++)
        if (c + j < o.K) o.col_scale[(int64_t)id * o.col_scale_ld + c + j] = (uint8_t)code[j];
    }
  }
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = t.first + row16 + 16 * i;
    if (r >= t.hi) continue;
    u32x2 q{0, 0};
    if (t.owned) {
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
    store_chunk<kVec, kStream>(o.col_data + r * o.ld_col, c, o.K, q);
  }
}

}  // namespace mxq_dev
