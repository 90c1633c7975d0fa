// product.hip -- matrix products of FP8 (E4M3) operands whose E8M0 codes stand
// for groups of 128 and for 128 x 128 tiles, on gfx950: y = x w^T, dx = dy w and
// dw = dy^T x, for one weight or for the weights of experts.
//
// One kernel computes out[i][j] = sum over r of V[i][r] * U[j][r].  The
// reduction runs in blocks of 128, the length of a group, so that within a block
// each row of V has one code and each row of U has one code.  U is the product
// instructions' first operand, which leaves each lane with four neighbouring
// columns j of one row i.
//
// Two ways to sum:
//   kFast   one v_mfma_scale_f32_16x16x128_f8f6f4 a block.  It multiplies by the
//           two power-of-two scales itself and adds to fp32 accumulators, so the
//           codes cost no arithmetic.  But the FP8 instructions of this card
//           (the unscaled ones too) line up each 8 products to the largest of
//           them and drop what falls below 2^-13 of it (a subnormal payload counts
//           as 2^-6 there): up to 2^-10 of the sum of magnitudes, 2^-11.7 seen on
//           random bytes, where bf16 output rounds by 2^-9.  The caller asks for
//           it, and only for activations and their gradients: weight gradients
//           feed an optimizer, and their segments may be a few rows long.
//   else    the payloads become bf16, which holds every E4M3 value, and sum in fp32
//           at half the instruction rate.  With many rows the codes go into the
//           conversion to bf16 (exact: they are powers of two) and the sums run
//           through v_mfma_f32_32x32x16_bf16; with few rows a block is four
//           v_mfma_f32_16x16x32_bf16, whose sum is scaled and added in fp32.
//
// Reached on one MI355X: 8192^3 with kFast 477 us (2304 TFLOP/s; a large library
// product in FP8 reaches 2659), bound by the clock the card holds under this load (2.0
// GHz of 2.4); dx of 1.9 TFLOP 832 us; dw of 103 GFLOP over experts with 403 MB of
// results 239 us, bound by one workgroup a CU (294 registers a lane), which hides
// neither a tile's start nor its stores; one token through 235 MB of weights 47.7 us
// (4.9 TB/s where a plain read reaches 6.7): 448 workgroups on 256 CUs.
//
//   product   i   j   r    V                     U                     U's code
//   y         m   n   k    x, r contiguous       w, r contiguous       (j / 128, r / 128)
//   dx        m   k   n    dy, r contiguous      w, r strided          (r / 128, j / 128)
//   dw        n   k   m    dy, r strided         x, r strided          (r / 128, j)
//
// Where r is the strided axis, tiles stay in LDS as they are in memory and
// ds_read_b64_tr_b8 transposes 8 x 16 bytes on the way to the registers.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <type_traits>

#include "checks.h"
#include "product_choice.h"
#include "segments.h"

namespace {

using namespace mxq_host;
using mxq_dev::Segment;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4_w __attribute__((ext_vector_type(4), aligned(4)));   // 16 bytes at a word's address
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define MXQ_LDS_AT(T, a) ((__attribute__((address_space(3))) T*)(uintptr_t)(uint32_t)(a))
#define MXQ_LDS(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kR = 128;   // the reduction block: one group, one product instruction

struct Operand {
  const uint8_t* data;
  int64_t ld;
  int64_t expert_stride;     // elements from one expert's matrix to the next (a weight)
  const uint8_t* code;
  int64_t code_x, code_r;    // strides of the code along i (or j) and along reduction blocks
  int64_t code_expert_stride;
  int x_shift;               // 7: one code for 128 rows of U, 0: one for each
};

struct Args {
  Operand v, u;
  void* out;
  int64_t ld_out, out_expert_stride;
  const int32_t* offsets;    // null: one segment
  int experts, I, J, R;
  bool vec_out, out_bf16;
};

// 16 bytes on their way from p, of which the first `avail` are wanted and the
// others are 0.  The memory pipeline is slow at addresses that are no multiple of 4
// (odd row strides took 4 times as long), so such bytes come as the aligned words
// around them and are shifted into place by done(), when they are needed.  Every
// word that is read holds at least one wanted byte.
__device__ __forceinline__ i32x4 first_bytes(i32x4 w, int n) {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const int m = n - 4 * k;
    w[k] &= m >= 4 ? -1 : m > 0 ? (1 << (8 * m)) - 1 : 0;
  }
  return w;
}
template <bool kAligned>
struct Bytes16;
template <>
struct Bytes16<true> {   // p is a multiple of 16
  i32x4 w;
  __device__ __forceinline__ Bytes16() {}
  __device__ __forceinline__ Bytes16(const uint8_t* p, int avail) {
    if (avail >= 16) {
      w = *reinterpret_cast<const i32x4*>(p);
      return;
    }
    const int last = (avail - 1) / 4;
    i32x4 v{0, 0, 0, 0};
    if (avail > 0) {
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] = reinterpret_cast<const int*>(p)[min(k, last)];
    }
    w = first_bytes(v, avail);
  }
  __device__ __forceinline__ i32x4 done() const { return w; }
};
template <>
struct Bytes16<false> {
  i32x4 w;
  int more, shift, wanted;
  __device__ __forceinline__ Bytes16() {}
  __device__ __forceinline__ Bytes16(const uint8_t* p, int avail) {
    shift = (int)((uintptr_t)p & 3);
    wanted = avail;
    const int* const q = reinterpret_cast<const int*>(p - shift);
    if (avail >= 16) {
      w = *reinterpret_cast<const i32x4_w*>(q);
      more = q[shift ? 4 : 3];
      return;
    }
    w = i32x4{0, 0, 0, 0};
    more = 0;
    if (avail > 0) {
      const int last = (shift + avail - 1) / 4;
#pragma unroll
      for (int k = 0; k < 4; k++) w[k] = q[min(k, last)];
      more = q[last];
    }
  }
  __device__ __forceinline__ i32x4 done() const {
    const i32x4 v{(int)__builtin_amdgcn_alignbyte(w[1], w[0], shift), (int)__builtin_amdgcn_alignbyte(w[2], w[1], shift),
                  (int)__builtin_amdgcn_alignbyte(w[3], w[2], shift), (int)__builtin_amdgcn_alignbyte(more, w[3], shift)};
    return __all(wanted >= 16) ? v : first_bytes(v, wanted);
  }
};

// Which reduction indexes of a block a lane holds: chunks g and g + 4 of 16, g =
// lane / 16.  V and U agree on it, and it is all that the products ask for.
__device__ __forceinline__ int chunk_of(int g, int half) { return g + 4 * half; }

// A tile of X rows (of V or U) by kR of the reduction in LDS, in 16-byte chunks,
// each row's chunks in an order of its own so that what lanes read at once falls
// on different banks of the 64 (no bank conflict is counted):
// kContig: [X][kR], chunk c of row x at place c ^ (x / 2 % 8).  A read takes one
// chunk of 16 rows in each of the four lane groups.
// Else [kR][X], chunk c of row r at place c ^ turn(r).  A read takes one chunk of
// 8 rows in each lane group, whose rows are 16 apart.
template <bool kContig, int X>
struct Tile {
  static constexpr int kBytes = X * kR;

  // LDS offset of chunk pos of row x (kContig) or r.
  static __device__ __forceinline__ int at(int row, int pos) {
    return row * (kContig ? kR : X) + ((pos ^ turn(row)) << 4);
  }
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (kContig) return (row >> 1) & 7;
    else if constexpr (X == 64) return ((row >> 2) & 1) | ((row >> 3) & 2);
    else if constexpr (X == 128) return (row & 6) | ((row >> 4) & 1);
    else return (row & 7) | ((row >> 1) & 8);
  }
  // Operand registers of rows x .. x + 15: lane l holds row x + l % 16.
  static __device__ __forceinline__ i32x8 fragment(const uint8_t* lds, int x) {
    const int lane = threadIdx.x & 63, g = lane / 16, i = lane % 16;
    i32x8 f;
    if constexpr (kContig) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + at(x + i, chunk_of(g, 0)));
      const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + at(x + i, chunk_of(g, 1)));
      f = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    } else {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const int r = 16 * chunk_of(g, t / 2) + t % 2 * 8 + i / 2;
        const uint8_t* p = lds + at(r, x >> 4) + (i & 1) * 8;
        const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(MXQ_LDS(i32x2, p));
        f[2 * t] = w[0];
        f[2 * t + 1] = w[1];
      }
    }
    return f;
  }
};

__device__ __forceinline__ void store4(float* p, f32x4 v, int n, bool vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<f32x4*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(__bf16* p, f32x4 v, int n, bool vec) {
  const bf16x4 b = __builtin_convertvector(v, bf16x4);   // the only rounding to fewer bits, at the very end
  if (vec && n >= 4) {
    *reinterpret_cast<bf16x4*>(p) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < n) p[i] = b[i];
  }
}

// The 32 payload bytes of a lane as bf16, exactly.
struct Wide {
  bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(i32x8 f) {
  Wide w;
#pragma unroll
  for (int q = 0; q < 4; q++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int word = f[2 * q + h];
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.0f, true);
      w.v[q][4 * h] = lo[0], w.v[q][4 * h + 1] = lo[1], w.v[q][4 * h + 2] = hi[0], w.v[q][4 * h + 3] = hi[1];
    }
  return w;
}

// Fragments of V as the products take them.
template <bool kFast, int N>
struct Prepared;
template <int N>
struct Prepared<true, N> {
  i32x8 v[N];
  __device__ __forceinline__ explicit Prepared(const i32x8 (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = f[i];
  }
};
template <int N>
struct Prepared<false, N> {
  Wide v[N];
  __device__ __forceinline__ explicit Prepared(const i32x8 (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = widen(f[i]);
  }
};

// Codes of U that one lane needs for rows col .. col + 15: that of its own row
// (lane % 16) for the scaled product, or those of its four results' rows.
template <bool kFast>
struct Codes {
  int c[kFast ? 1 : 4];
};
// One reduction block of 16 rows of U times 16 N rows of V, added to acc.
template <bool kFast, int N>
__device__ __forceinline__ void multiply(f32x4 (&acc)[N], const Prepared<kFast, N>& v, const int (&cv)[N], i32x8 u,
                                         const Codes<kFast>& cu) {
  if constexpr (kFast) {
#pragma unroll
    for (int i = 0; i < N; i++)
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v.v[i], acc[i], 0, 0, 0, cu.c[0], 0, cv[i]);
  } else {
    const Wide w = widen(u);
#pragma unroll
    for (int i = 0; i < N; i++) {
      f32x4 sum{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; q++) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[q], v.v[i].v[q], sum, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const float scaled = __builtin_ldexpf(sum[t], cu.c[t] + cv[i] - 254);
        acc[i][t] += cu.c[t] == 255 || cv[i] == 255 ? __builtin_nanf("") : scaled;
      }
    }
  }
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)v) | (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32);
}
template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
  return (const T*)uniform((int64_t)p);
}

// Which tile and segment a workgroup has.
struct Work {
  int i0, i_end, j0, r_begin, r_end, expert, weight;   // weight: the expert whose weight to read (0 where none is)
  int64_t code_block;                                  // first reduction block's place among the codes
  bool none;
};
template <Mode kMode, int BI, int BJ>
__device__ __forceinline__ Work work_of(const Args& a, int bi, int bj) {
  Work w{bi * BI, a.I, bj * BJ, 0, a.R, 0, 0, 0, false};
  if (a.offsets) {
    if constexpr (kMode == kWgrad) {
      w.expert = blockIdx.z;
      const Segment s = mxq_dev::find_expert<kR>(a.offsets, a.experts, a.R, w.expert);
      w.r_begin = uniform(s.lo), w.r_end = uniform(s.hi), w.code_block = uniform(s.first);
    } else {
      const Segment s = mxq_dev::find_tile<BI>(a.offsets, a.experts, a.I, bi);
      w.expert = uniform(s.expert);
      w.i0 = uniform((int)min((int64_t)s.lo + (int64_t)s.tile * BI, (int64_t)s.hi)), w.i_end = uniform(s.hi);
      w.none = w.i0 >= w.i_end;
      if (w.expert == a.experts) w.r_end = w.r_begin;   // rows of no expert: zeros
    }
  }
  w.weight = kMode == kWgrad || w.expert == a.experts ? 0 : w.expert;
  return w;
}

// A wave's WI x WJ results, rows i and columns j on, of 16 x 16 products.
template <typename TO, int WI, int WJ>
__device__ __forceinline__ void store_tile(const Args& a, const Work& w, int i0, int j0, const f32x4 (&acc)[WJ / 16][WI / 16]) {
  const int lane = threadIdx.x & 63;
  TO* const out = reinterpret_cast<TO*>(a.out);
#pragma unroll
  for (int i = 0; i < WI / 16; i++) {
    const int row = i0 + 16 * i + lane % 16;
    if (row >= w.i_end) continue;
#pragma unroll
    for (int j = 0; j < WJ / 16; j++) {
      const int col = j0 + 16 * j + lane / 16 * 4;
      if (col < a.J) store4(out + row * a.ld_out + col, acc[j][i], a.J - col, a.vec_out);
    }
  }
}

// A tile of X rows by kR of the reduction on its way to LDS through registers,
// for rows of any alignment; P says where its chunks go.
template <typename P, bool kContig, int X, int kThreads>
struct Carry {
  static constexpr int kChunks = X * kR / 16 / kThreads, kPer = kContig ? kR / 16 : X / 16;
  Bytes16<false> c[kChunks];
  // rows x0 .. of at most x_end, reduction r0 .. of at most r_end
  __device__ __forceinline__ void fetch(const uint8_t* base, int64_t ld, int x0, int x_end, int r0, int r_end) {
#pragma unroll
    for (int q = 0; q < kChunks; q++) {
      const int at = threadIdx.x + q * kThreads;
      if constexpr (kContig) {
        const int x = min(x0 + at / kPer, x_end - 1), r = r0 + at % kPer * 16;   // what rows past the end add is not stored
        c[q] = Bytes16<false>(base + x * ld + r, r_end - r);
      } else {
        const int r = r0 + at / kPer, x = x0 + at % kPer * 16;
        c[q] = Bytes16<false>(base + r * ld + x, r < r_end ? x_end - x : 0);
      }
    }
  }
  __device__ __forceinline__ void store(uint8_t* lds) const {
#pragma unroll
    for (int q = 0; q < kChunks; q++) {
      const int at = threadIdx.x + q * kThreads;
      *reinterpret_cast<i32x4*>(lds + P::at(at / kPer, at % kPer)) = c[q].done();
    }
  }
};

template <Mode kMode, typename TO, int BI, int BJ, int WI, int WJ>
__global__ __launch_bounds__(BI / WI * (BJ / WJ) * 64) void carried_kernel(Args a, int tj) {
  constexpr int kThreads = BI / WI * (BJ / WJ) * 64;
  constexpr bool kUContig = kMode == kForward;
  using TV = Tile<true, BI>;
  using TU = Tile<kUContig, BJ>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TV::kBytes + TU::kBytes];
  uint8_t* const lv = lds;
  uint8_t* const lu = lds + TV::kBytes;

  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int wi = wave / (BJ / WJ) * WI, wj = wave % (BJ / WJ) * WJ;
  const Work w = work_of<kMode, BI, BJ>(a, blockIdx.x / tj, blockIdx.x % tj);
  if (w.none) return;
  const uint8_t* const ud = a.u.data + w.weight * a.u.expert_stride;
  const uint8_t* const uc = a.u.code + w.weight * a.u.code_expert_stride;

  f32x4 acc[WJ / 16][WI / 16];
#pragma unroll
  for (int j = 0; j < WJ / 16; j++)
#pragma unroll
    for (int i = 0; i < WI / 16; i++) acc[j][i] = f32x4{0, 0, 0, 0};

  Carry<TV, true, BI, kThreads> sv;   // a block ahead of the products
  Carry<TU, kUContig, BJ, kThreads> su;
  auto fetch = [&](int r0) {
    sv.fetch(a.v.data, a.v.ld, w.i0, w.i_end, r0, w.r_end);
    su.fetch(ud, a.u.ld, w.j0, a.J, r0, w.r_end);
  };
  if (w.r_end) fetch(0);
  for (int b = 0; b * kR < w.r_end; b++) {
    __syncthreads();
    sv.store(lv);
    su.store(lu);
    __syncthreads();
    if ((b + 1) * kR < w.r_end) fetch((b + 1) * kR);
    int cv[WI / 16];
    i32x8 fv[WI / 16];
#pragma unroll
    for (int i = 0; i < WI / 16; i++) {
      const int row = min(w.i0 + wi + 16 * i + lane % 16, w.i_end - 1);
      cv[i] = a.v.code[row * a.v.code_x + b * a.v.code_r];
      fv[i] = TV::fragment(lv, wi + 16 * i);
    }
    const Prepared<true, WI / 16> pv(fv);
#pragma unroll
    for (int j = 0; j < WJ / 16; j++) {
      const int col = min(w.j0 + wj + 16 * j, a.J - 1);   // 16 neighbouring columns lie in one tile
      const Codes<true> cu{{uc[(col >> 7) * a.u.code_x + b * a.u.code_r]}};
      multiply<true>(acc[j], pv, cv, TU::fragment(lu, wj + 16 * j), cu);
    }
  }
  store_tile<TO, WI, WJ>(a, w, w.i0 + wi, w.j0 + wj, acc);
}

template <Mode kMode, typename TO, int BI, int BJ, int WI, int WJ>
int launch_carried(const Args& a, hipStream_t stream) {
  const int64_t tj = ((int64_t)a.J + BJ - 1) / BJ, ti = a.offsets ? a.I / BI + a.experts + 2 : ((int64_t)a.I + BI - 1) / BI;
  hipLaunchKernelGGL((carried_kernel<kMode, TO, BI, BJ, WI, WJ>), dim3((uint32_t)(ti * tj)),
                     dim3(BI / WI * (BJ / WJ) * 64), 0, stream, a, (int)tj);
  return launch_status();
}

// ---- many rows ------------------------------------------------------------------------------
// Tiles of V and U go from memory to LDS without passing through registers
// (buffer loads to LDS), one block ahead of the products; one barrier a block.
// The LDS places of a wave's 64 chunks are consecutive, so the swizzle is applied
// to the addresses that its lanes read.  A buffer's bound turns reads past the
// operand's end into zeros.
//
// Needs 16-byte aligned rows (and a contiguous axis that ends on a whole chunk).


// Loads from a buffer to LDS.  A buffer is bytes [base, base + left), at most
// 2^31 - 1 of them; offsets at or past its end read zeros.  A wave's lanes write
// consecutive words (or 16 bytes each) from the LDS address `to` on.  These are
// instructions and not the compiler's builtins, which would wait for them before
// every later LDS read; they have no output register.  They say that m0 is written
// (a reserved register, which the compiler remarks on), so that no value of the
// compiler's own is taken to live on in it.  arrive() waits for this wave's and then
// for the workgroup's.
constexpr int kPastEnd = 0x7FFFFFFF;
__device__ __forceinline__ i32x4 buffer(const uint8_t* base, int64_t left) {
  const uint64_t p = (uint64_t)base;
  return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), (int)min(max(left, (int64_t)0), (int64_t)kPastEnd), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
#define MXQ_LOAD_TO_LDS(name, instruction)                                                             \
  __device__ __forceinline__ void name(i32x4 from, uint32_t to, int off) {                             \
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\t" instruction " %0, %1, 0 offen lds" ::"v"(off), "s"(from), "s"(to) \
                 : "m0", "memory");                                                                    \
  }
MXQ_LOAD_TO_LDS(load_to_lds_16, "buffer_load_dwordx4")
MXQ_LOAD_TO_LDS(load_to_lds_4, "buffer_load_dword")
MXQ_LOAD_TO_LDS(load_to_lds_1, "buffer_load_ubyte")
#undef MXQ_LOAD_TO_LDS
#pragma clang diagnostic pop
// Waits for this wave's loads to LDS but the last kLeft, then for the workgroup.
template <int kLeft>
__device__ __forceinline__ void arrive_but() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void arrive() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <typename P, bool kContig, int X, int kThreads>
struct Feed {
  static constexpr int kChunks = X * kR / 16 / kThreads;
  const uint8_t* base;   // row x0, block 0
  int64_t step;          // bytes from one block to the next
  int64_t left;          // bytes from base to the operand's end
  int32_t off[kChunks];
  int32_t r_of_chunk;    // kContig: reduction index within the block, the same for all of this lane's chunks

  // rows x0 .. x_end - 1 (of the axis that the output keeps), reduction r0 .. r_end - 1
  __device__ __forceinline__ Feed(const uint8_t* data, int64_t ld, int x0, int x_end, int r0, int r_end) {
    if constexpr (kContig) {
      base = uniform(data + x0 * ld + r0);
      step = kR;
      left = (int64_t)(x_end - x0 - 1) * ld + (r_end - r0);
    } else {
      base = uniform(data + r0 * ld + x0);
      step = kR * ld;
      left = (int64_t)(r_end - r0 - 1) * ld + (x_end - x0);
    }
    left = uniform(left);
    r_of_chunk = 0;
#pragma unroll
    for (int q = 0; q < kChunks; q++) {
      const int c = threadIdx.x + q * kThreads;
      if constexpr (kContig) {
        const int x = c / 8, pos = (c % 8) ^ P::turn(x);   // x advances by multiples of 16 with q
        off[q] = (int32_t)(x * ld + pos * 16);
        r_of_chunk = pos * 16;
      } else {
        const int r = c / (X / 16), pos = (c % (X / 16)) ^ P::turn(r);
        off[q] = (int32_t)(r * ld + pos * 16);
      }
    }
  }
  // Block b, of whose reduction `valid` indexes exist, to the tile at lds.
  __device__ __forceinline__ void load(uint8_t* lds, int b, int valid) const {
    const i32x4 from = buffer(base + b * step, left - b * step);
    const bool none = kContig && r_of_chunk >= valid;
    const uint32_t to = lds_address(lds) + uniform((int)threadIdx.x / 64) * 1024;
#pragma unroll
    for (int q = 0; q < kChunks; q++) load_to_lds_16(from, to + q * kThreads * 16, none ? kPastEnd : off[q]);
  }
};

// This lane's LDS offsets of the fragments of rows x, x + 16, ... of a tile, x a multiple of 16 (kContig) or 64.
template <bool kContig, int X, int N>
struct Reader {
  int at[kContig ? 2 : N];
  __device__ __forceinline__ explicit Reader(int x) {
    const int lane = threadIdx.x & 63, g = lane / 16, i = lane % 16;
    using T = Tile<kContig, X>;
    if constexpr (kContig) {
      at[0] = T::at(i, chunk_of(g, 0)) + x * kR;
      at[1] = T::at(i, chunk_of(g, 1)) + x * kR;
    } else {
#pragma unroll
      for (int n = 0; n < N; n++) at[n] = T::at(16 * chunk_of(g, 0) + i / 2, x / 16 + n) + (i & 1) * 8;
    }
  }
  __device__ __forceinline__ i32x8 fragment(const uint8_t* lds, int n) const {
    i32x8 f;
    if constexpr (kContig) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + at[0] + 16 * n * kR);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + at[1] + 16 * n * kR);
      f = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    } else {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(MXQ_LDS(i32x2, lds + at[n] + (t / 2 * 64 + t % 2 * 8) * X));
        f[2 * t] = w[0];
        f[2 * t + 1] = w[1];
      }
    }
    return f;
  }
};

// Codes of a tile's rows, one 32-bit word a row in LDS.  With two stages, where
// four blocks' codes of a row are an aligned word in memory, they come in one load
// every four blocks (a code is in a cache line of its own in every row: byte by
// byte 8192^3 took 25 us more).  Else byte by byte, every block, so that a wave's
// loads of a block are always as many.
template <int X, int kStages>
struct CodeFeed {
  const uint8_t* base;
  int64_t step, left;
  int32_t off;
  bool words;

  __device__ __forceinline__ CodeFeed(const uint8_t* code, const Operand& o, int x0, int x_end, int blocks, int first_wave) {
    const int64_t start = (int64_t)(x0 >> o.x_shift) * o.code_x;
    base = uniform(code + start);
    step = o.code_r;
    left = uniform((int64_t)((x_end - 1) >> o.x_shift) * o.code_x + (blocks - 1) * step + 1 - start);
    words = kStages == 2 && step == 1 && blocks % 4 == 0 && o.code_x % 4 == 0 && ((uintptr_t)base & 3) == 0;
    const int x = min(x0 + ((int)threadIdx.x - first_wave * 64), x_end - 1);
    off = (int32_t)(((x >> o.x_shift) - (x0 >> o.x_shift)) * o.code_x);
  }
  // Called by X / 64 waves from first_wave on.
  __device__ __forceinline__ void load(uint32_t* lds, int b, int stage, int first_wave) const {
    const i32x4 from = buffer(base + b * step, left - b * step);
    const uint32_t to = lds_address(place(lds, b, stage)) + (uniform((int)threadIdx.x / 64) - first_wave) * 256;
    if (!words) load_to_lds_1(from, to, off);
    else if (b % 4 == 0) load_to_lds_4(from, to, off);
  }
  // Where block b's words are, and by how many bits they are shifted.
  __device__ __forceinline__ uint32_t* place(uint32_t* lds, int b, int stage) const {
    return lds + (words ? b / 4 & 1 : stage) * X;
  }
  __device__ __forceinline__ int shift(int b) const { return words ? 8 * (b & 3) : 0; }
};

template <Mode kMode, typename TO, int BI, int BJ, int WI, int WJ, int kStages>
__global__ __launch_bounds__(BI / WI * (BJ / WJ) * 64) void tile_kernel(Args a, int ti, int tj) {
  constexpr int kWaves = BI / WI * (BJ / WJ), kThreads = kWaves * 64;
  constexpr bool kUContig = kMode == kForward;
  using TV = Tile<true, BI>;
  using TU = Tile<kUContig, BJ>;
  constexpr int kStage = TV::kBytes + TU::kBytes;
  static_assert(BI / 64 + BJ / 64 == kWaves, "one load of codes a wave");
  constexpr int kLoads = (BI + BJ) * kR / 16 / kThreads + 1;   // a wave's loads to LDS of one block
  static_assert(kLoads * (kStages - 2) < 64, "the count of loads that a wave can wait for");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * kStage];
  __shared__ __attribute__((aligned(16))) uint32_t codes_v[kStages * BI], codes_u[kStages * BJ];

  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x / 64);
  const int wi = wave / (BJ / WJ) * WI, wj = wave % (BJ / WJ) * WJ;
  const Work w = work_of<kMode, BI, BJ>(a, blockIdx.x / tj, blockIdx.x % tj);
  if (w.none) return;
  const int blocks = (w.r_end + kR - 1) / kR;

  f32x4 acc[WJ / 16][WI / 16];
#pragma unroll
  for (int j = 0; j < WJ / 16; j++)
#pragma unroll
    for (int i = 0; i < WI / 16; i++) acc[j][i] = f32x4{0, 0, 0, 0};

  const Feed<TV, true, BI, kThreads> v(a.v.data, a.v.ld, w.i0, w.i_end, 0, w.r_end);
  const Feed<TU, kUContig, BJ, kThreads> u(a.u.data + w.weight * a.u.expert_stride, a.u.ld, w.j0, a.J, 0, w.r_end);
  const CodeFeed<BI, kStages> vc(a.v.code, a.v, w.i0, w.i_end, blocks, 0);
  const CodeFeed<BJ, kStages> uc(a.u.code + w.weight * a.u.code_expert_stride, a.u, w.j0, a.J, blocks, BI / 64);
  const Reader<true, BI, WI / 16> rv(wi);
  const Reader<kUContig, BJ, WJ / 16> ru(wj);
  auto load = [&](int b, int stage) {   // past the last block: zeros that nobody reads
    uint8_t* const to = lds + stage * kStage;
    if (wave < BI / 64) vc.load(codes_v, b, stage, 0);
    else uc.load(codes_u, b, stage, BI / 64);
    v.load(to, b, w.r_end - b * kR);
    u.load(to + TV::kBytes, b, w.r_end - b * kR);
  };
  if (blocks) {
#pragma unroll
    for (int s = 0; s < kStages - 1; s++) load(s, s);
  }
  for (int b = 0, stage = 0; b < blocks; b++) {
    arrive_but<kLoads * (kStages - 2)>();   // block b is in LDS, and no wave reads block b - 1 any more
    load(b + kStages - 1, stage ? stage - 1 : kStages - 1);
    const uint8_t* const lv = lds + stage * kStage;
    const uint8_t* const lu = lv + TV::kBytes;
    const uint32_t* const wv = vc.place(codes_v, b, stage) + wi;
    const uint32_t* const wu = uc.place(codes_u, b, stage) + wj;
    i32x8 fv[WI / 16];
    int cv[WI / 16];
#pragma unroll
    for (int i = 0; i < WI / 16; i++) {
      cv[i] = wv[16 * i + lane % 16] >> vc.shift(b) & 255;
      fv[i] = rv.fragment(lv, i);
    }
    const Prepared<true, WI / 16> pv(fv);
#pragma unroll
    for (int j = 0; j < WJ / 16; j++) {
      const Codes<true> cu{{(int)(wu[16 * j + lane % 16] >> uc.shift(b) & 255)}};
      multiply<true>(acc[j], pv, cv, ru.fragment(lu, j), cu);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load is on its way to LDS when the workgroup gives it back
  store_tile<TO, WI, WJ>(a, w, w.i0 + wi, w.j0 + wj, acc);
}

template <Mode kMode, typename TO, int BI, int BJ, int WI, int WJ, int kStages>
int launch_tiles(const Args& a, hipStream_t stream) {
  const int64_t tj = ((int64_t)a.J + BJ - 1) / BJ;
  const int64_t ti = a.offsets ? a.I / BI + a.experts + 2 : ((int64_t)a.I + BI - 1) / BI;
  hipLaunchKernelGGL((tile_kernel<kMode, TO, BI, BJ, WI, WJ, kStages>), dim3((uint32_t)(ti * tj)),
                     dim3(BI / WI * (BJ / WJ) * 64), 0, stream, a, (int)ti, (int)tj);
  return launch_status();
}

// ---- many rows, sums in fp32 ------------------------------------------------------------------
// Places of a tile's 16-byte chunks in LDS for fragments of 32 rows and 64
// reduction indexes: a lane holds row lane % 32 and, with p = lane / 32, chunks
// p, p + 2 (first half of the block) and p + 4, p + 6 (second half).
// kContig: [X][kR], chunk c of row x at place c ^ (x / 2 % 8).  Else [kR][X], chunk
// c of row r at place c ^ turn(r): the transposing read takes two neighbouring
// chunks of 8 rows at once, which then fall on all 64 banks.
template <bool kContig, int X>
struct Places {
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (kContig) return (row >> 1) & 7;
    else if constexpr (X == 128) return row & 6;
    else return (row & 7) << 1;
  }
  static __device__ __forceinline__ int at(int row, int c) { return row * (kContig ? kR : X) + ((c ^ turn(row)) << 4); }
};

// The codes of 64 of a tile's rows, one 32-bit word each in LDS; each wave brings
// those of other rows, of V or of U.
struct ByteCodeFeed {
  const uint8_t* base;
  int64_t step, left;
  int32_t off;

  // codes of rows x0 .. x_end - 1, lane by lane, `blocks` blocks from `code` on
  __device__ __forceinline__ ByteCodeFeed(const uint8_t* code, int64_t code_x, int64_t code_r, int shift, int x0, int x_end,
                                      int blocks) {
    const int64_t first = min(x0, x_end - 1) >> shift;
    base = uniform(code + first * code_x);
    step = code_r;
    left = uniform((((x_end - 1) >> shift) - first) * code_x + (blocks - 1) * code_r + 1);
    off = (int32_t)(((min(x0 + ((int)threadIdx.x & 63), x_end - 1) >> shift) - first) * code_x);
  }
  __device__ __forceinline__ void load(uint32_t to, int b) const {
    load_to_lds_1(buffer(base + b * step, left - b * step), to, off);
  }
};

// The same through a register, for code rows so far apart that 64 of them pass a
// buffer's 32-bit offsets.
struct ByteCodeCarry {
  const uint8_t* row;
  int64_t step;
  uint32_t next;

  __device__ __forceinline__ ByteCodeCarry(const uint8_t* code, int64_t code_x, int64_t code_r, int shift, int x0, int x_end,
                                       int)
      : row(code + (int64_t)(min(x0 + ((int)threadIdx.x & 63), x_end - 1) >> shift) * code_x), step(code_r), next(0) {}
  __device__ __forceinline__ void fetch(int b) { next = row[b * step]; }
  __device__ __forceinline__ void store(uint32_t* to) const { to[threadIdx.x & 63] = next; }
};

// 32 rows' payloads of one block: two halves of 64 reduction indexes.
struct Rows32 {
  i32x8 h[2];
};

__device__ __forceinline__ bool all_zero(const Rows32& f) {   // of either sign
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < 16; k++) any |= (uint32_t)f.h[k / 8][k % 8];
  return (any & 0x7F7F7F7Fu) == 0;
}

// This lane's LDS addresses of the fragments of rows x, x + 32, ... of a tile, x a multiple of 32.
template <bool kContig, int X, int N>
struct Reader32 {
  static constexpr int kCount = kContig ? 4 : N;
  uint32_t at[kCount];
  __device__ __forceinline__ Reader32(const uint8_t* tile, int x) {
    const int lane = threadIdx.x & 63, p = lane / 32;
    using P = Places<kContig, X>;
    const uint32_t base = lds_address(tile);
    if constexpr (kContig) {
#pragma unroll
      for (int q = 0; q < 4; q++) at[q] = base + P::at(lane % 32, p + 2 * q) + x * kR;
    } else {
      const int i = lane % 16;
#pragma unroll
      for (int n = 0; n < N; n++) at[n] = base + P::at(16 * p + i / 2, x / 16 + 2 * n + lane / 16 % 2) + (i & 1) * 8;
    }
  }
  __device__ __forceinline__ Rows32 rows(uint32_t stage, int n) const {
    Rows32 f;
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int q = 0; q < 2; q++) {
        if constexpr (kContig) {
          const i32x4 w = *MXQ_LDS_AT(i32x4, at[2 * h + q] + stage + 32 * n * kR);
#pragma unroll
          for (int t = 0; t < 4; t++) f.h[h][4 * q + t] = w[t];
        } else {
#pragma unroll
          for (int t = 0; t < 2; t++) {
            const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                MXQ_LDS_AT(i32x2, at[n] + stage + (64 * h + 32 * q + 8 * t) * X));
            f.h[h][4 * q + 2 * t] = w[0];
            f.h[h][4 * q + 2 * t + 1] = w[1];
          }
        }
      }
    return f;
  }
  // Reads after this stay after it.
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int n = 0; n < kCount; n++) asm volatile("" : "+v"(at[n]));
  }
};

// 64 payloads of a row as bf16 times 2^(code - 127).
struct Wide64 {
  bf16x8 v[8];
};
__device__ __forceinline__ Wide64 widen(const Rows32& f, float scale) {
  Wide64 w;
#pragma unroll
  for (int k = 0; k < 16; k++) {
    const int word = f.h[k / 8][k % 8];
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, scale, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, scale, true);
    bf16x8& to = w.v[k / 2];
    to[4 * (k % 2)] = lo[0], to[4 * (k % 2) + 1] = lo[1], to[4 * (k % 2) + 2] = hi[0], to[4 * (k % 2) + 3] = hi[1];
  }
  return w;
}

// Sums in fp32 take the codes into the conversion to bf16 where no value can leave
// bf16's normal range by it and no product or sum fp32's: codes from 77 to 167
// (group maxima from about 4e-13 to 4.9e14).  The smallest product is then 2^(-18 -
// 2 * 50), and 2^30 of the largest, 448^2 * 2^(2 * 40), add up to less than 2^128:
// a sum overflows only if the true one does, and products that cancel do so in
// fp32.  A block with any other code, 255 among them, is summed unscaled, then scaled
// exactly, as the few-rows kernels always do.  A group of zeros has code 0, but any
// scale does for it: it counts as plain, lest one such group (a masked token's row, a
// column that an activation left at 0) send the rest of a wave's sums through the
// second way, which takes 4 times as long.
constexpr uint32_t kPlainFirst = 77, kPlainLast = 167;
__device__ __forceinline__ bool plain_code(uint32_t code) { return code - kPlainFirst <= kPlainLast - kPlainFirst; }
__device__ __forceinline__ float two_to(uint32_t code) { return __builtin_bit_cast(float, code << 23); }


template <Mode kMode, bool kFed, typename TO, int BI, int BJ, int WI, int WJ, int kStages>
__global__ __launch_bounds__(BI / WI * (BJ / WJ) * 64) void exact_kernel(Args a, int ti, int tj) {
  constexpr int kWaves = BI / WI * (BJ / WJ), kThreads = kWaves * 64, NI = WI / 32, NJ = WJ / 32;
  constexpr bool kVContig = kMode != kWgrad, kUContig = kMode == kForward;
  constexpr int kVBytes = BI * kR, kStage = kVBytes + BJ * kR;
  using FV = Feed<Places<kVContig, BI>, kVContig, BI, kThreads>;
  using FU = Feed<Places<kUContig, BJ>, kUContig, BJ, kThreads>;
  constexpr int kLoads = FV::kChunks + FU::kChunks + 1;   // a wave's loads to LDS of one block
  static_assert(BI / 64 + BJ / 64 == kWaves, "64 rows' codes a wave");
  static_assert(kLoads * (kStages - 2) < 64, "the count of loads that a wave can wait for");
  __shared__ __attribute__((aligned(128))) uint8_t lds[kStages * kStage];
  __shared__ __attribute__((aligned(16))) uint32_t codes[kStages][BI + BJ];

  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x / 64);
  const int wi = wave / (BJ / WJ) * WI, wj = wave % (BJ / WJ) * WJ;
  const Work w = work_of<kMode, BI, BJ>(a, blockIdx.x / tj, blockIdx.x % tj);
  if (w.none) return;
  const int blocks = (w.r_end - w.r_begin + kR - 1) / kR;

  f32x16 acc[NJ][NI];
#pragma unroll
  for (int j = 0; j < NJ; j++)
#pragma unroll
    for (int i = 0; i < NI; i++) acc[j][i] = f32x16{};

  const uint8_t* const ud = a.u.data + w.weight * a.u.expert_stride;
  const FV v(a.v.data, a.v.ld, w.i0, w.i_end, w.r_begin, w.r_end);
  const FU u(ud, a.u.ld, w.j0, a.J, w.r_begin, w.r_end);
  using FC = std::conditional_t<kFed, ByteCodeFeed, ByteCodeCarry>;
  FC c = wave < BI / 64 ? FC(a.v.code + w.code_block * a.v.code_r, a.v.code_x, a.v.code_r, a.v.x_shift, w.i0 + wave * 64,
                             w.i_end, blocks)
                        : FC(a.u.code + w.weight * a.u.code_expert_stride + w.code_block * a.u.code_r, a.u.code_x,
                             a.u.code_r, a.u.x_shift, w.j0 + (wave - BI / 64) * 64, a.J, blocks);
  Carry<Places<kVContig, BI>, kVContig, BI, kThreads> sv;   // unless kFed
  Carry<Places<kUContig, BJ>, kUContig, BJ, kThreads> su;
  auto fetch = [&](int b) {
    sv.fetch(a.v.data, a.v.ld, w.i0, w.i_end, w.r_begin + b * kR, w.r_end);
    su.fetch(ud, a.u.ld, w.j0, a.J, w.r_begin + b * kR, w.r_end);
    if constexpr (!kFed) c.fetch(b);
  };
  const Reader32<kVContig, BI, NI> rv(lds, wi);
  const Reader32<kUContig, BJ, NJ> ru(lds + kVBytes, wj);
  auto load = [&](int b, int stage) {   // past the last block: zeros that nobody reads
    uint8_t* const to = lds + stage * kStage;
    if constexpr (kFed) c.load(lds_address(codes[stage]) + wave * 256, b);
    v.load(to, b, w.r_end - w.r_begin - b * kR);
    u.load(to + kVBytes, b, w.r_end - w.r_begin - b * kR);
  };
  if (blocks) {
    if constexpr (kFed) {
#pragma unroll
      for (int s = 0; s < kStages - 1; s++) load(s, s);
    } else {
      fetch(0);
    }
  }
  Rows32 fu[NJ];
  uint32_t cu[NJ], cv[NI];
  int b = 0, stage = 0;
  auto begin = [&] {
    if constexpr (kFed) {
      arrive_but<kLoads * (kStages - 2)>();   // block b is in LDS, and no wave reads block b - 1 any more
      load(b + kStages - 1, stage ? stage - 1 : kStages - 1);
    } else {
      // no wave reads block b - 2, whose place this is, since all came here for block b - 1
      c.store(codes[stage] + wave * 64);
      sv.store(lds + stage * kStage);
      su.store(lds + stage * kStage + kVBytes);
      arrive();
      if (b + 1 < blocks) fetch(b + 1);
    }
  };
  auto next = [&] {
    b++;
    stage = stage + 1 == kStages ? 0 : stage + 1;
  };
  auto read = [&] {
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      cu[j] = codes[stage][BI + wj + 32 * j + lane % 32];
      fu[j] = ru.rows(stage * kStage, j);
    }
#pragma unroll
    for (int i = 0; i < NI; i++) cv[i] = codes[stage][wi + 32 * i + lane % 32];
  };
  // Whether all codes of the block are plain; with `zeros`, groups of zeros count as such.
  auto plain = [&](auto zeros) {
    bool all = true;
#pragma unroll
    for (int j = 0; j < NJ; j++) all = all && (plain_code(cu[j]) || (zeros && cu[j] == 0 && all_zero(fu[j])));
#pragma unroll
    for (int i = 0; i < NI; i++)
      all = all && (plain_code(cv[i]) || (zeros && cv[i] == 0 && all_zero(rv.rows(stage * kStage, i))));
    return (bool)__all(all);
  };
  auto add_plain = [&] {
    Wide64 wu[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j++) wu[j] = widen(fu[j], two_to(cu[j]));
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const Wide64 wv = widen(rv.rows(stage * kStage, i), two_to(cv[i]));
#pragma unroll
      for (int k = 0; k < 8; k++)
#pragma unroll
        for (int j = 0; j < NJ; j++)
          acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wu[j].v[k], wv.v[k], acc[j][i], 0, 0, 0);
    }
  };
  // Up to the first block with a code that is not plain, from there on up to the
  // first that is so for another reason than a group of zeros, and the rest: three
  // loops, so that each one's registers know nothing of the others.  With the second
  // loop's look at the zeros in the first, all sums take 3% longer.
  while (b < blocks) {
    begin();
    read();
    if (!plain(std::false_type())) break;
    add_plain();
    next();
  }
  bool begun = true;
  while (b < blocks) {
    if (!begun) {
      begin();
      read();
    }
    begun = true;
    if (!plain(std::false_type()) && !plain(std::true_type())) break;
    add_plain();
    next();
    begun = false;
  }
  while (b < blocks) {
    if (!begun) {
      begin();
      read();
    }
    begun = false;
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const Wide64 wv = widen(rv.rows(stage * kStage, i), 1.0f);
#pragma unroll
      for (int j = 0; j < NJ; j++) {
        const Wide64 wu = widen(fu[j], 1.0f);
        f32x16 sum{};
#pragma unroll
        for (int k = 0; k < 8; k++) sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wu.v[k], wv.v[k], sum, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < 16; t++) {
          const int code = __shfl((int)cu[j], t / 4 * 8 + lane / 32 * 4 + t % 4);
          const float scaled = __builtin_ldexpf(sum[t], code + (int)cv[i] - 254);
          acc[j][i][t] += code == 255 || cv[i] == 255 ? __builtin_nanf("") : scaled;
        }
      }
    }
    next();
  }
  // Results leave through LDS, a wave's own part of it, so that a store writes
  // whole rows of WJ columns and not 32 bytes of each of 32 rows.
  static_assert(WJ == 64 && kWaves * WI * WJ * 4 <= kStages * kStage, "a wave's results");
  arrive();   // no wave reads LDS any more, and no load is on its way there
  float* const own = reinterpret_cast<float*>(lds) + wave * WI * WJ;
  auto place = [](int row, int chunk) { return row * WJ + ((chunk ^ (row & 15)) << 2); };
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
      for (int q = 0; q < 4; q++)
        *reinterpret_cast<f32x4*>(own + place(32 * i + lane % 32, 8 * j + 2 * q + lane / 32)) =
            f32x4{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  TO* const out = reinterpret_cast<TO*>(a.out) + (kMode == kWgrad ? w.expert * a.out_expert_stride : 0);
  const int col = w.j0 + wj + lane % 16 * 4;
#pragma unroll 4
  for (int r = lane / 16; r < WI; r += 4) {
    const int row = w.i0 + wi + r;
    const f32x4 y = *reinterpret_cast<const f32x4*>(own + place(r, lane % 16));
    if (row < w.i_end && col < a.J) store4(out + row * a.ld_out + col, y, a.J - col, a.vec_out);
  }
}

template <Mode kMode, bool kFed, typename TO, int BI, int BJ, int WI, int WJ, int kStages>
int launch_exact(const Args& a, hipStream_t stream) {
  const int64_t tj = ((int64_t)a.J + BJ - 1) / BJ;
  int64_t ti = ((int64_t)a.I + BI - 1) / BI, tz = 1;
  if (a.offsets) {
    if (kMode == kWgrad) tz = a.experts;
    else ti = a.I / BI + a.experts + 2;
  }
  hipLaunchKernelGGL((exact_kernel<kMode, kFed, TO, BI, BJ, WI, WJ, kStages>), dim3((uint32_t)(ti * tj), 1, (uint32_t)tz),
                     dim3(BI / WI * (BJ / WJ) * 64), 0, stream, a, (int)ti, (int)tj);
  return launch_status();
}

// Whether all rows of an operand begin at multiples of 16 bytes.
bool chunked(const Operand& o, int64_t experts) {
  return aligned(o.data, 16) && o.ld % 16 == 0 && (experts <= 1 || o.expert_stride % 16 == 0);
}

// Whether an operand's tiles can be fed straight to LDS: rows at multiples of 16
// bytes, whole chunks along the contiguous axis, 32-bit offsets within a tile.
bool feedable(const Operand& o, int contiguous, int64_t experts) {
  return chunked(o, experts) && contiguous % 16 == 0 && o.ld < ((int64_t)1 << 22) && o.code_x < ((int64_t)1 << 22);
}

// ---- few rows -------------------------------------------------------------------------------
// With few rows i a product is bound by reading U once, so nothing is shared
// between waves on the way: each of a workgroup's waves takes every kWaves-th
// reduction block of the same 16 kNJ rows of U, straight from memory to the
// product instructions, one block ahead of them, and the waves' sums are added
// through LDS in a fixed order at the end.  Where U's reduction axis is strided
// (dx), a wave turns its block around in an LDS tile of its own.  The forms of eight
// waves spill registers: 32 of y with 64 rows and sums in fp32, of dx with 64 rows 51 (FP8
// sums, unaligned: none) and 78, of dx with 16 rows 21 and 22.

// This lane's part of reduction r .. r + 127 of a row, which ends at r_end.
template <bool kAligned>
struct RowPart {
  Bytes16<kAligned> half[2];
  __device__ __forceinline__ RowPart() {}
  __device__ __forceinline__ RowPart(const uint8_t* row, int r, int r_end) {
    const int g = (threadIdx.x & 63) / 16;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int at = r + 16 * chunk_of(g, h);
      half[h] = Bytes16<kAligned>(row + at, r_end - at);
    }
  }
  __device__ __forceinline__ i32x8 done() const {
    const i32x4 lo = half[0].done(), hi = half[1].done();
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
};

template <Mode kMode, bool kFast, bool kAligned, int kNI, int kNJ, int kFewWaves>
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(Args a) {
  static_assert(kMode != kWgrad, "a weight gradient reduces over the rows");
  constexpr bool kTurn = kMode == kDgrad;
  constexpr int BJ = 16 * kNJ, kChunks = BJ * kR / 16 / 64;
  using T = Tile<false, BJ>;
  constexpr int kSum = kNI * kNJ * 64 * 4;                       // floats of one wave's sums
  constexpr int kShared = kFewWaves / 2 * kSum * 4;
  constexpr int kTurned = kTurn ? kFewWaves * BJ * kR : 0;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTurned > kShared ? kTurned : kShared];

  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int j0 = blockIdx.x * BJ;
  int i0 = blockIdx.y * 16 * kNI, i_end = a.I, blocks = (a.R + kR - 1) / kR, expert = 0;
  if (a.offsets) {
    const Segment s = mxq_dev::find_tile<16 * kNI>(a.offsets, a.experts, a.I, blockIdx.y);
    i0 = min((int64_t)s.lo + (int64_t)s.tile * 16 * kNI, (int64_t)s.hi), i_end = s.hi;
    if (i0 >= i_end) return;
    if (s.expert == a.experts) blocks = 0;
    else expert = s.expert;
  }
  const uint8_t* const ud = a.u.data + expert * a.u.expert_stride;
  const uint8_t* const uc = a.u.code + expert * a.u.code_expert_stride;
  uint8_t* const tile = lds + wave * BJ * kR;

  // rows past the end read the last one's bytes: what they add is not stored
  const uint8_t* vrow[kNI];
  const uint8_t* vcode[kNI];
#pragma unroll
  for (int i = 0; i < kNI; i++) {
    const int row = min(i0 + 16 * i + lane % 16, i_end - 1);
    vrow[i] = a.v.data + row * a.v.ld;
    vcode[i] = a.v.code + row * a.v.code_x;
  }
  const uint8_t* urow[kNJ];
  if constexpr (!kTurn) {
#pragma unroll
    for (int j = 0; j < kNJ; j++) urow[j] = ud + min(j0 + 16 * j + lane % 16, a.J - 1) * a.u.ld;
  }
  const uint8_t* ucode[kNJ];
#pragma unroll
  for (int j = 0; j < kNJ; j++) ucode[j] = uc + (min(j0 + 16 * j, a.J - 1) >> 7) * a.u.code_x;

  struct Block {
    RowPart<kAligned> v[kNI];
    int cv[kNI], cu[kNJ];
    RowPart<kAligned> u[kTurn ? 1 : kNJ];
    Bytes16<kAligned> raw[kTurn ? kChunks : 1];
  };
  auto load = [&](Block& k, int b) {
    const int r = b * kR;
    if constexpr (kTurn) {
#pragma unroll
      for (int q = 0; q < kChunks; q++) {
        const int c = lane + 64 * q, ur = b * kR + c / kNJ, uj = j0 + c % kNJ * 16;
        k.raw[q] = Bytes16<kAligned>(ud + ur * a.u.ld + uj, ur < a.R ? a.J - uj : 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kNJ; j++) k.u[j] = RowPart<kAligned>(urow[j], r, a.R);
    }
#pragma unroll
    for (int i = 0; i < kNI; i++) {
      k.v[i] = RowPart<kAligned>(vrow[i], r, a.R);
      k.cv[i] = vcode[i][b];
    }
#pragma unroll
    for (int j = 0; j < kNJ; j++) k.cu[j] = ucode[j][b * a.u.code_r];
  };

  f32x4 acc[kNJ][kNI];
#pragma unroll
  for (int j = 0; j < kNJ; j++)
#pragma unroll
    for (int i = 0; i < kNI; i++) acc[j][i] = f32x4{0, 0, 0, 0};

  // Aligned blocks are loaded one ahead of the products; the words around
  // unaligned ones take half as many registers again, which leaves no room for that.
  Block now, next;
  if (kAligned && wave < blocks) load(now, wave);
  for (int b = wave; b < blocks; b += kFewWaves) {
    if constexpr (kAligned) {
      if (b + kFewWaves < blocks) load(next, b + kFewWaves);
    } else {
      load(now, b);
    }
    if constexpr (kTurn) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int q = 0; q < kChunks; q++) {
        const int c = lane + 64 * q;
        *reinterpret_cast<i32x4*>(tile + T::at(c / kNJ, c % kNJ)) = now.raw[q].done();
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    i32x8 fv[kNI];
#pragma unroll
    for (int i = 0; i < kNI; i++) fv[i] = now.v[i].done();
    const Prepared<kFast, kNI> pv(fv);
#pragma unroll
    for (int j = 0; j < kNJ; j++) {
      Codes<kFast> cu;   // 16 neighbouring columns lie in one tile
#pragma unroll
      for (int t = 0; t < (kFast ? 1 : 4); t++) cu.c[t] = now.cu[j];
      i32x8 u;
      if constexpr (kTurn) u = T::fragment(tile, 16 * j);
      else u = now.u[j].done();
      multiply<kFast>(acc[j], pv, now.cv, u, cu);
    }
    if constexpr (kAligned) now = next;
  }

  float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int half = kFewWaves / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < kNI * kNJ; t++)
        *reinterpret_cast<f32x4*>(sums + (wave - half) * kSum + (t * 64 + lane) * 4) = acc[t / kNI][t % kNI];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < kNI * kNJ; t++)
        acc[t / kNI][t % kNI] += *reinterpret_cast<const f32x4*>(sums + wave * kSum + (t * 64 + lane) * 4);
    }
  }
  if (wave) return;
#pragma unroll
  for (int i = 0; i < kNI; i++) {
    const int row = i0 + 16 * i + lane % 16;
    if (row >= i_end) continue;
#pragma unroll
    for (int j = 0; j < kNJ; j++) {
      const int col = j0 + 16 * j + lane / 16 * 4;
      if (col >= a.J) continue;
      if (a.out_bf16) store4(reinterpret_cast<__bf16*>(a.out) + row * a.ld_out + col, acc[j][i], a.J - col, a.vec_out);
      else store4(reinterpret_cast<float*>(a.out) + row * a.ld_out + col, acc[j][i], a.J - col, a.vec_out);
    }
  }
}

template <Mode kMode, bool kFast, int kNI, int kNJ>
int launch_few(const Args& a, hipStream_t stream) {
  const int64_t tj = ((int64_t)a.J + 16 * kNJ - 1) / (16 * kNJ);
  const int64_t ti = a.offsets ? a.I / (16 * kNI) + a.experts + 2 : ((int64_t)a.I + 16 * kNI - 1) / (16 * kNI);
  if (ti > 65535) return MXQ_ERR_SHAPE;   // launch() sends so many rows elsewhere
  const dim3 grid((uint32_t)tj, (uint32_t)ti);
  // Eight waves a workgroup where the workgroups do not fill the card (one row x
  // 8192 x 8192: 20.9 us, with four 26.7), else four, which leave less of a wave's
  // time to joining sums (9 tokens through 6 of 48 experts: 14.8 us, with eight 16.5).
  const bool wide = tj * ti <= kCUs;
  const bool by_chunks = chunked(a.v, 0) && chunked(a.u, a.experts);
#define MXQ_FEW(ALIGNED, WAVES)                                                                                       \
  hipLaunchKernelGGL((few_rows_kernel<kMode, kFast, ALIGNED, kNI, kNJ, WAVES>), grid, dim3(WAVES * 64), 0, stream, a)
  if (!by_chunks) MXQ_FEW(false, 8);   // not a block ahead, so the more waves the better
  else if (wide) MXQ_FEW(true, 8);
  else MXQ_FEW(true, 4);
#undef MXQ_FEW
  return launch_status();
}

template <Mode kMode, bool kFast, typename TO>
int launch(const Args& a, hipStream_t stream) {
  const bool fed = feedable(a.v, kMode == kWgrad ? a.I : a.R, 0) && feedable(a.u, kMode == kForward ? a.R : a.J, a.experts);
  const ProductKernel kernel = choose_kernel(kMode, kFast, fed, a.I, a.J, a.offsets ? a.experts : 0);
  if constexpr (kMode != kWgrad) {
    if (kernel == kFewRows16) return launch_few<kMode, kFast, 1, kMode == kDgrad ? 8 : 4>(a, stream);
    if (kernel == kFewRows32) return launch_few<kMode, kFast, 2, 4>(a, stream);
    if (kernel == kFewRows64) return launch_few<kMode, kFast, 4, 4>(a, stream);
  }
  if constexpr (kFast) {
    if (kernel == kCarried) return launch_carried<kMode, TO, 128, 128, 64, 64>(a, stream);
    if (kernel == kTiles256) return launch_tiles<kMode, TO, 256, 256, 128, 64, 2>(a, stream);
    return launch_tiles<kMode, TO, 128, 128, 64, 64, 2>(a, stream);
  } else {
    if (kernel == kExactCarried) return launch_exact<kMode, false, TO, 128, 128, 64, 64, 2>(a, stream);
    return launch_exact<kMode, true, TO, 128, 128, 64, 64, 2>(a, stream);
  }
}

// One operand as the caller gives it: a [rows, cols] payload and its codes.
struct Given {
  const uint8_t* data;
  int64_t ld, rows, cols;
  const uint8_t* code;
  int64_t code_ld, code_rows, code_cols;
  int64_t experts, stride, code_stride;   // experts > 0: that many of them, so far apart

  bool null() const { return rows > 0 && cols > 0 && (!data || !code); }
  bool shape_ok() const {
    if (rows == 0 || cols == 0) return true;
    if (ld < cols || code_ld < code_cols) return false;
    return experts <= 1 || (stride >= (rows - 1) * ld + cols && code_stride >= (code_rows - 1) * code_ld + code_cols);
  }
  Range data_range() const { return stack_range(data, experts ? experts : 1, stride, rows, cols, ld, 1); }
  Range code_range() const {
    return stack_range(code, experts ? experts : 1, code_stride, rows > 0 && cols > 0 ? code_rows : 0, code_cols,
                       code_ld, 1);
  }
};

int check(const Given& v, const Given& u, int64_t M, int64_t N, int64_t K, const int32_t* offsets, int64_t experts,
          void* out, int64_t ld_out, int64_t out_stride, int64_t out_count, int64_t out_rows, int64_t out_cols,
          mxq_dtype out_dt, bool* empty) {
  *empty = false;
  if (!is_float(out_dt)) return MXQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return MXQ_ERR_SHAPE;
  if (offsets && (experts < 1 || experts > kMaxExperts)) return MXQ_ERR_SHAPE;
  if (out_rows == 0 || out_cols == 0) {
    *empty = true;
    return MXQ_OK;
  }
  if (!out || v.null() || u.null()) return MXQ_ERR_NULL;
  if (!v.shape_ok() || !u.shape_ok() || ld_out < out_cols) return MXQ_ERR_SHAPE;
  if (out_count > 1 && out_stride < (out_rows - 1) * ld_out + out_cols) return MXQ_ERR_SHAPE;
  const Range ro = stack_range(out, out_count, out_stride, out_rows, out_cols, ld_out, size_of(out_dt));
  const Range r[4] = {v.data_range(), v.code_range(), u.data_range(), u.code_range()};
  const Range roff = matrix_range(offsets, 1, offsets ? experts + 1 : 0, experts + 1, 4);
  if (!all_ok({ro, r[0], r[1], r[2], r[3], roff}) || !aligned(out, size_of(out_dt)) || !aligned(offsets, 4))
    return MXQ_ERR_SHAPE;
  if (!disjoint({ro}, {r[0], r[1], r[2], r[3], roff})) return MXQ_ERR_ALIAS;
  return MXQ_OK;
}

// Four neighbouring outputs of a row go out in one store.
bool vector_out(const void* out, int64_t ld, int64_t stride, mxq_dtype dt) {
  return aligned(out, 4 * size_of(dt)) && ld % 4 == 0 && stride % 4 == 0;
}

template <Mode kMode>
int dispatch_columns(const Args& a, bool fast, hipStream_t stream) {
  if constexpr (kMode != kWgrad) {
    if (fast) return a.out_bf16 ? launch<kMode, true, __bf16>(a, stream) : launch<kMode, true, float>(a, stream);
  }
  return a.out_bf16 ? launch<kMode, false, __bf16>(a, stream) : launch<kMode, false, float>(a, stream);
}

// A launch has fewer than 2^32 lanes in a dimension: outputs of more than 2^22
// tiles of 128 x 128, or of more than 2^28 columns, are made some columns at a time.
template <Mode kMode>
int dispatch(const Args& a, bool fast, hipStream_t stream) {
  const int64_t ti = a.offsets && kMode != kWgrad ? a.I / 128 + a.experts + 2 : ((int64_t)a.I + 127) / 128;
  const int64_t tj = std::min(std::max((int64_t)1, ((int64_t)1 << 22) / ti), (int64_t)1 << 21), step = tj * 128;
  if (a.J <= step) return dispatch_columns<kMode>(a, fast, stream);
  for (int64_t j = 0; j < a.J; j += step) {
    Args part = a;
    part.J = (int)std::min(step, a.J - j);
    part.u.data += kMode == kForward ? j * a.u.ld : j;
    part.u.code += (j >> a.u.x_shift) * a.u.code_x;
    part.out = (uint8_t*)a.out + j * (a.out_bf16 ? 2 : 4);
    const int st = dispatch_columns<kMode>(part, fast, stream);
    if (st != MXQ_OK) return st;
  }
  return MXQ_OK;
}

}  // namespace

extern "C" {

int mxq_matmul_fp8_block128(const uint8_t* x, int64_t ld_x, const uint8_t* x_scale, int64_t x_scale_ld,
                            const uint8_t* w, int64_t ld_w, int64_t w_stride, const uint8_t* tile_code,
                            int64_t tile_ld, int64_t tile_stride, int64_t M, int64_t N, int64_t K,
                            const int32_t* offsets, int64_t n_experts, void* out, int64_t ld_out, mxq_dtype out_dt,
                            int fast_accum, hipStream_t stream) {
  const int64_t n = offsets ? n_experts : 0;
  const Given v{x, ld_x, M, K, x_scale, x_scale_ld, M, groups_of(K), 0, 0, 0};
  const Given u{w, ld_w, N, K, tile_code, tile_ld, groups_of(N), groups_of(K), n, w_stride, tile_stride};
  bool empty;
  const int st = check(v, u, M, N, K, offsets, n_experts, out, ld_out, 0, 1, M, N, out_dt, &empty);
  if (st != MXQ_OK || empty) return st;
  const Args a{Operand{x, ld_x, 0, x_scale, x_scale_ld, 1, 0, 0},
               Operand{w, ld_w, w_stride, tile_code, tile_ld, 1, tile_stride, 7},
               out, ld_out, 0, offsets, (int)n, (int)M, (int)N, (int)K, vector_out(out, ld_out, 0, out_dt), out_dt == MXQ_BF16};
  return dispatch<kForward>(a, fast_accum != 0, stream);
}

int mxq_matmul_fp8_block128_dgrad(const uint8_t* dy, int64_t ld_dy, const uint8_t* dy_scale, int64_t dy_scale_ld,
                                  const uint8_t* w, int64_t ld_w, int64_t w_stride, const uint8_t* tile_code,
                                  int64_t tile_ld, int64_t tile_stride, int64_t M, int64_t N, int64_t K,
                                  const int32_t* offsets, int64_t n_experts, void* dx, int64_t ld_dx,
                                  mxq_dtype out_dt, int fast_accum, hipStream_t stream) {
  const int64_t n = offsets ? n_experts : 0;
  const Given v{dy, ld_dy, M, N, dy_scale, dy_scale_ld, M, groups_of(N), 0, 0, 0};
  const Given u{w, ld_w, N, K, tile_code, tile_ld, groups_of(N), groups_of(K), n, w_stride, tile_stride};
  bool empty;
  const int st = check(v, u, M, N, K, offsets, n_experts, dx, ld_dx, 0, 1, M, K, out_dt, &empty);
  if (st != MXQ_OK || empty) return st;
  const Args a{Operand{dy, ld_dy, 0, dy_scale, dy_scale_ld, 1, 0, 0},
               Operand{w, ld_w, w_stride, tile_code, 1, tile_ld, tile_stride, 7},
               dx, ld_dx, 0, offsets, (int)n, (int)M, (int)K, (int)N, vector_out(dx, ld_dx, 0, out_dt), out_dt == MXQ_BF16};
  return dispatch<kDgrad>(a, fast_accum != 0, stream);
}

int mxq_matmul_fp8_group128_wgrad(const uint8_t* dy, int64_t ld_dy, const uint8_t* dy_scale, int64_t dy_scale_ld,
                                  const uint8_t* x, int64_t ld_x, const uint8_t* x_scale, int64_t x_scale_ld,
                                  int64_t M, int64_t N, int64_t K, const int32_t* offsets, int64_t n_experts,
                                  void* dw, int64_t ld_dw, int64_t dw_stride, mxq_dtype out_dt, hipStream_t stream) {
  const int64_t n = offsets ? n_experts : 0, code_rows = offsets ? M / kR + n : groups_of(M);
  const Given v{dy, ld_dy, M, N, dy_scale, dy_scale_ld, code_rows, N, 0, 0, 0};
  const Given u{x, ld_x, M, K, x_scale, x_scale_ld, code_rows, K, 0, 0, 0};
  bool empty;
  const int st = check(v, u, M, N, K, offsets, n_experts, dw, ld_dw, dw_stride, n ? n : 1, N, K, out_dt, &empty);
  if (st != MXQ_OK || empty) return st;
  const Args a{Operand{dy, ld_dy, 0, dy_scale, 1, dy_scale_ld, 0, 0},
               Operand{x, ld_x, 0, x_scale, 1, x_scale_ld, 0, 0},
               dw, ld_dw, dw_stride, offsets, (int)n, (int)N, (int)K, (int)M,
               vector_out(dw, ld_dw, n > 1 ? dw_stride : 0, out_dt), out_dt == MXQ_BF16};
  return dispatch<kWgrad>(a, false, stream);
}

}  // extern "C"
