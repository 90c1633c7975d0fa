// Eight elements of a row as floats, rounded once on their way out, and sums over a
// row's lanes (norm.hip, activate.hip, route.hip).
#pragma once

#include "group128.h"

namespace mxq_dev {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The types as the kernels name them: uint16_t for bf16, uint32_t for fp32 bit patterns.
template <typename T>
__device__ __forceinline__ f32x8 widen(const Chunk<T>& v) {
  f32x8 f;
#pragma unroll
  for (int i = 0; i < kEPL; i++) {
    if constexpr (sizeof(T) == 2)
      f[i] = __builtin_bit_cast(float, i & 1 ? v.w[i / 2] & 0xFFFF0000u : v.w[i / 2] << 16);
    else
      f[i] = __builtin_bit_cast(float, v.w[i]);
  }
  return f;
}

template <typename T>
__device__ __forceinline__ Chunk<T> narrow(f32x8 f) {
  Chunk<T> v;
  if constexpr (sizeof(T) == 2) {
    const bf16x8 b = __builtin_convertvector(f, bf16x8);   // to nearest, ties to even
#pragma unroll
    for (int i = 0; i < 4; i++) v.w[i] = __builtin_bit_cast(u32x4, b)[i];
  } else {
    const u32x8 b = __builtin_bit_cast(u32x8, f);   // as a whole: of one element the cast takes the vector's first
#pragma unroll
    for (int i = 0; i < kEPL; i++) v.w[i] = b[i];
  }
  return v;
}

template <typename T, bool kVec, bool kOnce = false>
__device__ __forceinline__ f32x8 load_floats(const void* row, int c, int K) {
  return widen<T>(load_chunk<T, kVec, kOnce>((const T*)row, c, K));
}

template <typename T, bool kVec, bool kStream = false>
__device__ __forceinline__ void store_floats(void* row, int c, int K, f32x8 f) {
  const Chunk<T> v = narrow<T>(f);
  T* const p = (T*)row + c;
  if (kVec) {
    if (c < K) {
#pragma unroll
      for (int i = 0; i < Chunk<T>::kWords / 4; i++) {
        const u32x4 q{v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]};
        if (kStream) __builtin_nontemporal_store(q, (u32x4*)p + i);
        else ((u32x4*)p)[i] = q;
      }
    }
  } else if (c + kEPL <= K) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::kWords / 4; i++)
      reinterpret_cast<u32x4_any*>(p)[i] = u32x4{v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < K) {
        if constexpr (sizeof(T) == 2) p[i] = (T)(v.w[i / 2] >> (16 * (i & 1)));
        else p[i] = v.w[i];
      }
  }
}

// Payload and code of the group of a row that 16 lanes hold, eight values each.
template <bool kVec, bool kStream>
__device__ __forceinline__ void store_group(uint8_t* data, uint8_t* scale, int c, int K, f32x8 f) {
  const Chunk<uint32_t> v = narrow<uint32_t>(f);
  const uint32_t code = code_of<uint32_t>(max16(v.amax()));
  store_chunk<kVec, kStream>(data, c, K, payload_of(v, code));
  if ((threadIdx.x & 15) == 0 && c < K) scale[c / kGroup] = (uint8_t)code;
}

// The same with four elements a lane, so that 16 bytes of fp32 a lane cover whole lines; rows lie at multiples of 16 bytes and
// K is a multiple of 4.
__device__ __forceinline__ f32x4 widen4(u32x2 w) {
  return __builtin_bit_cast(f32x4, u32x4{w[0] << 16, w[0] & 0xFFFF0000u, w[1] << 16, w[1] & 0xFFFF0000u});
}
__device__ __forceinline__ u32x2 narrow4(f32x4 f) { return __builtin_bit_cast(u32x2, __builtin_convertvector(f, bf16x4)); }

template <typename T, bool kOnce = false>
__device__ __forceinline__ f32x4 load_four(const void* row, int c, int K) {
  if (c >= K) return f32x4{};
  if constexpr (sizeof(T) == 4) {
    const f32x4* const p = (const f32x4*)((const float*)row + c);
    return kOnce ? __builtin_nontemporal_load(p) : *p;
  } else {
    const u32x2* const p = (const u32x2*)((const uint16_t*)row + c);
    return widen4(kOnce ? __builtin_nontemporal_load(p) : *p);
  }
}

template <typename T, bool kStream = false>
__device__ __forceinline__ void store_four(void* row, int c, int K, f32x4 f) {
  if (c >= K) return;
  if constexpr (sizeof(T) == 4) {
    f32x4* const p = (f32x4*)((float*)row + c);
    if (kStream) __builtin_nontemporal_store(f, p);
    else *p = f;
  } else {
    u32x2* const p = (u32x2*)((uint16_t*)row + c);
    if (kStream) __builtin_nontemporal_store(narrow4(f), p);
    else *p = narrow4(f);
  }
}

// 32 lanes hold the group.
template <bool kStream>
__device__ __forceinline__ void store_group_four(uint8_t* data, uint8_t* scale, int c, int K, f32x4 f) {
  const uint32_t m = max16(magnitude_bits(larger(larger(f[0], f[1]), larger(f[2], f[3]))));
  const u32x2 rows = swap16(m, m);
  const uint32_t code = code_of<uint32_t>(max(rows[0], rows[1]));
  const float s = __builtin_bit_cast(float, code << 23);   // code 0 stands for 2^-127 here
  s16x2 q = __builtin_nondeterministic_value(q);           // both halves are written
  q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, f[0], f[1], s, false);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, f[2], f[3], s, true);
  const uint32_t bytes = code == 255u ? kPoison4 : __builtin_bit_cast(uint32_t, q);
  if (c >= K) return;
  uint32_t* const p = (uint32_t*)(data + c);
  if (kStream) __builtin_nontemporal_store(bytes, p);
  else *p = bytes;
  if ((threadIdx.x & 31) == 0) scale[c / kGroup] = (uint8_t)code;
}

__device__ __forceinline__ float add8(f32x8 v) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// Sum over the aligned groups of kLanes lanes of a wave, the same in each of them.
template <int kLanes>
__device__ __forceinline__ float lane_sum(float v) {
  const auto with = [](float v, uint32_t o) { return v + __builtin_bit_cast(float, o); };
  const auto bits = [](float v) { return __builtin_bit_cast(uint32_t, v); };
  v = with(v, dpp<0xB1>(bits(v)));    // quad_perm [1,0,3,2]
  v = with(v, dpp<0x4E>(bits(v)));    // quad_perm [2,3,0,1]
  v = with(v, dpp<0x141>(bits(v)));   // row_half_mirror: quads hold one value each by now
  v = with(v, dpp<0x140>(bits(v)));   // row_mirror
  static_assert(kLanes == 16 || kLanes == 64, "a row of lanes or a wave");
  if constexpr (kLanes == 64) {
    u32x2 s = swap16(bits(v), bits(v));
    v = __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
    s = swap32(bits(v), bits(v));
    v = __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
  }
  return v;
}

}  // namespace mxq_dev
