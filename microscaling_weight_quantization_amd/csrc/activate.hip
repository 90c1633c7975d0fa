// activate.hip -- the activation between the two products of a feed-forward layer,
// with FP8 output in groups of 128, and its backward pass, on gfx950.
//
//   a = act(gate) up, or act(gate) where there is no up
//   silu(g) = g p(g), gelu(g) = g p(2 sqrt(2/pi) (g + 0.044715 g^3)) (its tanh form), relu2(g) = max(g, 0)^2
//   p(z) = 1 / (1 + exp(-z)), which is (1 + tanh(z / 2)) / 2
//   dgate = da up act'(gate), dup = da act(gate)
//
// Everything is computed in fp32 and rounded once, to E4M3.
//
// Memory bounds it; every element is read once.  2048 x 28672 bf16 by rows 47.6 us (294 MB, 6.2 TB/s, a plain copy's rate
// being 6.6); both ways 128 rows x 128 columns a workgroup, of whose rows it touches 256 bytes each: 49152 x 1024 54.4 us
// (303 MB, 5.6 TB/s), its gradients 99 (505 MB, 5.1), of which two workgroups fit a CU.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "fastdiv.h"
#include "floats.h"

namespace {

using namespace mxq_host;
using namespace mxq_dev;

struct ActArgs {
  const void *gate, *up, *da;   // up null: not gated; da null: forward
  int64_t ld_gate, ld_up, ld_da;
  int F;
  int act;
};

// p(z) and, with kRest, q = 1 - p(z), without overflow and without cancellation in either tail: with u = 2^-64 exp(-z) they
// are 2^-64 / (2^-64 + u) and u / (2^-64 + u), off by 6.4 half steps of fp32 at most.  exp(-z) is 2^n 2^f with n whole and |f| at
// most 1/2, log2(e) taken in two parts, so that f is exact to 2^-25 whatever z is.  Beyond the bounds of x p is what it
// is there, and so is q, 0.  With exp2(64 - |z| log2(e)) instead, whose argument is rounded by up to 2^-18, p was off by up to 24
// half steps; 2048 x 28672 bf16 by rows took 47.3 us for 47.6, 49152 x 1024 both ways 53.9 for 54.4, its gradients 98.5 for 99.4.
struct Logistic {
  float p, q;
};
template <bool kRest>
__device__ __forceinline__ Logistic logistic(float z) {
  constexpr float kLog2e = 1.44269504088896341f, kLess = (float)(1.44269504088896341 - (double)kLog2e);
  constexpr float kWhole = 0x1.8p23f - 64.0f;   // a sum with it is whole, n - 64 in its lowest bits
  const float x = __builtin_amdgcn_fmed3f(z, -128.0f, kRest ? 128.0f : 42.0f);   // a number for a NaN, which p then meets
  const float m = fmaf(-x, kLog2e, kWhole), n = m - kWhole;
  const float e = __builtin_amdgcn_exp2f(fmaf(-x, kLess, fmaf(-x, kLog2e, -n)));
  const uint32_t bits = __builtin_bit_cast(uint32_t, m);
  // up to z = 42 u is a normal number, so n may be added to its exponent
  const float u = kRest ? __builtin_amdgcn_ldexpf(e, (int)(bits - __builtin_bit_cast(uint32_t, 0x1.8p23f)))
                        : __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, e) + (bits << 23));
  const float r = __builtin_amdgcn_rcpf(0x1p-64f + u);
  return Logistic{r * 0x1p-64f, u * r};
}

constexpr float kGelu = 1.59576912160573071f;   // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

// max(g, 0), a NaN if g is one.
__device__ __forceinline__ float positive(float g) { return __builtin_elementwise_maximum(g, 0.0f); }

template <int kAct>
__device__ __forceinline__ float act_of(float g) {
  if constexpr (kAct == MXQ_SILU) return g * logistic<false>(g).p;
  if constexpr (kAct == MXQ_GELU_TANH) return g * logistic<false>(kGelu * (g + kCube * g * g * g)).p;
  return positive(g) * positive(g);
}

// act(g) into *a, act'(g) as the result.
template <int kAct>
__device__ __forceinline__ float slope_of(float g, float* a) {
  if constexpr (kAct == MXQ_SILU) {
    const Logistic l = logistic<true>(g);
    *a = g * l.p;
    return l.p + *a * l.q;
  }
  if constexpr (kAct == MXQ_GELU_TANH) {
    const float g2 = g * g;
    const Logistic l = logistic<true>(kGelu * g * (1.0f + kCube * g2));
    *a = g * l.p;
    // far out p q is 0 and g may be anything: the product is then 0, not 0 * Inf
    const float t = *a * l.q;
    return l.p + (t == 0.0f ? 0.0f : t * kGelu * (1.0f + 3.0f * kCube * g2));
  }
  const float r = positive(g);
  *a = r * r;
  return 2.0f * r;
}

// What a lane reads for eight elements of a row; da in the backward pass only.
template <typename T, bool kBack>
struct Raw {
  Chunk<T> gate, up, da;
};
// kOnce: each line is read by one instruction and by no other workgroup, and leaves with the non-temporal hint.  That holds
// for bf16 (a lane's 32 bytes of fp32 are two loads, each of half of every line): 49152 x 1024 bf16 both ways 61.8 -> 53.9
// us, 2048 x 28672 by rows 51.0 -> 46.5; 16000 x 1024 fp32 29.9 -> 34.2, so not there, nor for 16000 x 1000 bf16 backward,
// where two workgroups read each line (53.5 -> 60.5).
template <typename T, bool kVec, bool kOnce, bool kBack>
__device__ __forceinline__ void load_raw(Raw<T, kBack>& v, const ActArgs& s, int64_t r, int c) {
  v.gate = load_chunk<T, kVec, kOnce>((const T*)s.gate + r * s.ld_gate, c, s.F);
  if (s.up) v.up = load_chunk<T, kVec, kOnce>((const T*)s.up + r * s.ld_up, c, s.F);
  if constexpr (kBack) v.da = load_chunk<T, kVec, kOnce>((const T*)s.da + r * s.ld_da, c, s.F);
}

// The rows of a tile of which this lane holds every kStep-th, one after the other.
template <typename T, bool kVec, bool kOnce, bool kBack, bool kWhole, int kStep>
struct Walk {
  const ActArgs& s;
  const T *gate, *up, *da;
  int row, have, c;
  int64_t first;
  __device__ __forceinline__ Walk(const ActArgs& a, const TileRows& t, int column)
      : s(a), row(threadIdx.x / 16), have(t.have()), c(column + (threadIdx.x & 15) * kEPL), first(t.first) {
    if constexpr (kWhole) {
      gate = (const T*)s.gate + first * s.ld_gate + row * s.ld_gate + c;
      up = s.up ? (const T*)s.up + first * s.ld_up + row * s.ld_up + c : nullptr;
      if constexpr (kBack) da = (const T*)s.da + first * s.ld_da + row * s.ld_da + c;
    }
  }
  __device__ __forceinline__ void next(Raw<T, kBack>& v) {
    if constexpr (kWhole) {
      v.gate = load_chunk<T, kVec, kOnce>(gate, 0, 1);
      gate += kStep * s.ld_gate;
      if (s.up) v.up = load_chunk<T, kVec, kOnce>(up, 0, 1), up += kStep * s.ld_up;
      if constexpr (kBack) v.da = load_chunk<T, kVec, kOnce>(da, 0, 1), da += kStep * s.ld_da;
    } else {
      load_raw<T, kVec, kOnce>(v, s, first + min(row, have - 1), row < have ? c : s.F);
      row += kStep;
    }
  }
};

template <typename T, int kAct>
__device__ __forceinline__ f32x8 value_of(const Raw<T, false>& v, bool gated) {
  const f32x8 g = widen<T>(v.gate);
  f32x8 a;
#pragma unroll
  for (int i = 0; i < kEPL; i++) a[i] = act_of<kAct>(g[i]);
  return gated ? a * widen<T>(v.up) : a;
}

// ---- groups along the rows ------------------------------------------------------------
// 16 lanes per group, 16 groups per workgroup, one group a lane.
constexpr int kRowThreads = 256;

template <typename T, int kAct, bool kVec>
__global__ __launch_bounds__(kRowThreads) void act_rows_kernel(ActArgs s, MxqDivisor groups, uint32_t total,
                                                               uint8_t* data, int64_t ld_data, uint8_t* scale,
                                                               int64_t scale_ld) {
  keep_denormals();
  const uint32_t g = blockIdx.x * (kRowThreads / 16) + threadIdx.x / 16;
  if (g >= total) return;   // whole groups of 16 lanes leave together
  const uint32_t r = mxq_quot(g, groups), b = g - r * groups.d;
  const int c = (int)b * kGroup + (threadIdx.x & 15) * kEPL;
  Raw<T, false> v;
  load_raw<T, kVec, kVec && sizeof(T) == 2>(v, s, r, c);
  store_group<kVec, false>(data + (int64_t)r * ld_data, scale + (int64_t)r * scale_ld, c, s.F,
                           value_of<T, kAct>(v, s.up != nullptr));
}

// ---- groups along both -----------------------------------------------------------------
template <typename T, int kAct, bool kVec, bool kStream, bool kWhole, int kRows>
__device__ __forceinline__ void act_tile(const ActArgs& s, const TileRows& t, int id, const TileOut& out,
                                         TileShared<kRows>& shared) {
  Chunk<uint32_t> v[kRows];
  const int have = t.have();
  constexpr int kAtOnce = sizeof(T) == 2 ? kRows : kRows / 2;   // rows whose operands are on their way at once
  Walk<T, kVec, kVec && sizeof(T) == 2, false, kWhole, kGroup / kRows> walk(s, t, blockIdx.x * kGroup);
#pragma unroll
  for (int i0 = 0; i0 < kRows; i0 += kAtOnce) {
    Raw<T, false> raw[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; i++) walk.next(raw[i]);
#pragma unroll
    for (int i = 0; i < kAtOnce; i++) {   // rows that there are not are not computed: 130 x 11904 of 56 experts 34.3 -> 18.8 us
      v[i0 + i] = Chunk<uint32_t>{};
      if (kWhole || kGroup / kRows * (i0 + i) < have) v[i0 + i] = narrow<uint32_t>(value_of<T, kAct>(raw[i], s.up != nullptr));
    }
  }
  store_tile<uint32_t, kVec, true, kStream, kWhole>(v, out, t, id, blockIdx.x, shared);
}

template <typename T, int kAct, bool kVec, bool kStream, int kRows>
__global__ __launch_bounds__(16 * kGroup / kRows) void act_tiles_kernel(ActArgs s, int first_id, int rows,
                                                                        const int32_t* offsets, int experts,
                                                                        TileOut out) {
  keep_denormals();
  __shared__ TileShared<kRows> shared;
  const int id = first_id + (int)blockIdx.y;
  const TileRows t = tile_rows(offsets, experts, rows, id, shared);
  if (!t.owned) clear_codes(out, id, blockIdx.x);
  if (t.first >= t.hi) return;   // the same for the whole workgroup
  if (kVec && whole_tile(t, blockIdx.x, s.F)) act_tile<T, kAct, kVec, kStream, kVec, kRows>(s, t, id, out, shared);
  else act_tile<T, kAct, kVec, kStream, false, kRows>(s, t, id, out, shared);
}

// ---- backward ----------------------------------------------------------------------------
// Eight elements of dgate and of dup; what is not used is not computed.
struct Both {
  f32x8 gate, up;
};
template <typename T, int kAct>
__device__ __forceinline__ Both gradients_of(const Raw<T, true>& v, bool gated) {
  const f32x8 g = widen<T>(v.gate), da = widen<T>(v.da);
  f32x8 a, d;
#pragma unroll
  for (int i = 0; i < kEPL; i++) {
    float one;
    d[i] = slope_of<kAct>(g[i], &one);
    a[i] = one;
  }
  return Both{gated ? da * widen<T>(v.up) * d : da * d, da * a};
}

// Elements [c, c + 8) of a row [dgate, dup], wherever they lie.
template <typename T, int kAct, bool kVec>
__device__ __forceinline__ f32x8 gradient_at(const ActArgs& s, int64_t r, int c) {
  Raw<T, true> v;
  if (c + kEPL <= s.F || c >= s.F) {
    load_raw<T, kVec, false>(v, s, r, c < s.F ? c : c - s.F);
    const Both b = gradients_of<T, kAct>(v, true);
    return c < s.F ? b.gate : b.up;
  }
  // across the end of the first half: elements from F on are the first of the second
  load_raw<T, false, false>(v, s, r, c);
  f32x8 out = gradients_of<T, kAct>(v, true).gate;
  load_raw<T, false, false>(v, s, r, 0);
  const f32x8 u = gradients_of<T, kAct>(v, true).up;
  const int n = s.F - c;
#pragma unroll
  for (int i = 0; i < kEPL; i++) {
#pragma unroll
    for (int j = 0; j < kEPL; j++)
      if (i == n + j) out[i] = u[j];
  }
  return out;
}

// What a workgroup takes: the same 128 columns of both halves, which reads them once; or 128 columns of the result, which
// lie in one of the halves or across their border.  The latter, where F is no multiple of 128, reads gate and da twice and
// takes the exponentials twice: 16000 x 1000 bf16 53.0 us, of 1024 columns 35.1.
enum Part { kBothHalves, kGateHalf, kUpHalf, kBorder };

template <typename T, int kAct, bool kVec, bool kStream, Part kPart, bool kWhole, int kRows>
__device__ __forceinline__ void act_backward_tile(const ActArgs& s, const TileRows& t, int id, const TileOut& out,
                                                  TileShared<kRows>& shared) {
  constexpr int kStep = kGroup / kRows;
  const int have = t.have();
  Chunk<uint32_t> v[kRows], u[kPart == kBothHalves ? kRows : 1];
  if constexpr (kPart != kBorder) {
    constexpr int kAtOnce = sizeof(T) == 2 ? kRows : kRows / 2;   // rows whose operands are on their way at once
    Walk<T, kVec, kVec && sizeof(T) == 2 && kPart == kBothHalves, true, kWhole, kStep> walk(s, t, blockIdx.x * kGroup - (kPart == kUpHalf ? s.F : 0));
#pragma unroll
    for (int i0 = 0; i0 < kRows; i0 += kAtOnce) {
      Raw<T, true> raw[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) walk.next(raw[i]);
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) {
        if (!kWhole && kStep * (i0 + i) >= have) {   // no such row
          v[i0 + i] = Chunk<uint32_t>{};
          if constexpr (kPart == kBothHalves) u[i0 + i] = Chunk<uint32_t>{};
          continue;
        }
        const Both b = gradients_of<T, kAct>(raw[i], s.up != nullptr);
        v[i0 + i] = narrow<uint32_t>(kPart == kUpHalf ? b.up : b.gate);
        if constexpr (kPart == kBothHalves) u[i0 + i] = narrow<uint32_t>(b.up);
      }
    }
  } else {
    const int c = blockIdx.x * kGroup + (threadIdx.x & 15) * kEPL;
#pragma unroll 1
    for (int i = 0; i < kRows; i++) {
      const int64_t r = t.first + threadIdx.x / 16 + kStep * i;
      const Chunk<uint32_t> one = narrow<uint32_t>(r < t.hi && c < out.K ? gradient_at<T, kAct, kVec>(s, r, c) : f32x8{});
#pragma unroll
      for (int j = 0; j < kRows; j++)
        if (i == j) v[j] = one;
    }
  }
  store_tile<uint32_t, kVec, true, kStream, kWhole>(v, out, t, id, blockIdx.x, shared);
  if constexpr (kPart == kBothHalves)
    store_tile<uint32_t, kVec, true, kStream, kWhole, true>(u, out, t, id, blockIdx.x + s.F / kGroup, shared);
}

template <typename T, int kAct, bool kVec, bool kStream, bool kBoth, int kRows>
__global__ __launch_bounds__(16 * kGroup / kRows) void act_backward_kernel(ActArgs s, int first_id, int rows,
                                                                           const int32_t* offsets, int experts,
                                                                           TileOut out) {
  keep_denormals();
  __shared__ TileShared<kRows> shared;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup;
  const TileRows t = tile_rows(offsets, experts, rows, id, shared);
  if (!t.owned) {
    clear_codes(out, id, blockIdx.x);
    if (kBoth) clear_codes(out, id, blockIdx.x + s.F / kGroup);
  }
  if (t.first >= t.hi) return;   // all of this is the same for the whole workgroup
  const bool whole = kVec && whole_tile(t, blockIdx.x, kBoth ? s.F : out.K);
  if constexpr (kBoth) {
    if (whole) act_backward_tile<T, kAct, kVec, kStream, kBothHalves, kVec, kRows>(s, t, id, out, shared);
    else act_backward_tile<T, kAct, kVec, kStream, kBothHalves, false, kRows>(s, t, id, out, shared);
  } else if (c + kGroup <= s.F || !s.up) {
    if (whole) act_backward_tile<T, kAct, kVec, kStream, kGateHalf, kVec, kRows>(s, t, id, out, shared);
    else act_backward_tile<T, kAct, kVec, kStream, kGateHalf, false, kRows>(s, t, id, out, shared);
  } else if (c >= s.F) {
    if (whole) act_backward_tile<T, kAct, kVec, kStream, kUpHalf, kVec, kRows>(s, t, id, out, shared);
    else act_backward_tile<T, kAct, kVec, kStream, kUpHalf, false, kRows>(s, t, id, out, shared);
  } else {
    act_backward_tile<T, kAct, kVec, kStream, kBorder, false, kRows>(s, t, id, out, shared);
  }
}

// ---- host --------------------------------------------------------------------------------

bool known(int act) { return act == MXQ_SILU || act == MXQ_GELU_TANH || act == MXQ_RELU2; }

struct Operands {
  Range gate, up, da;
};

// The checks that all forms share.  For a call with nothing to do *empty is set.
int check_operands(const ActArgs& a, int64_t rows, int64_t F, mxq_dtype dt, bool backward, Operands* out, bool* empty) {
  *empty = false;
  if (!is_float(dt) || !known(a.act)) return MXQ_ERR_DTYPE;
  if (rows < 0 || F < 0 || rows > kMaxDim || F > kMaxDim / 2) return MXQ_ERR_SHAPE;
  if (rows == 0 || F == 0) {
    *empty = true;
    return MXQ_OK;
  }
  if (!a.gate || (backward && !a.da)) return MXQ_ERR_NULL;
  if (a.ld_gate < F || (a.up && a.ld_up < F) || (backward && a.ld_da < F)) return MXQ_ERR_SHAPE;
  const size_t es = size_of(dt);
  *out = Operands{matrix_range(a.gate, rows, F, a.ld_gate, es), matrix_range(a.up, a.up ? rows : 0, F, a.ld_up, es),
                  matrix_range(a.da, backward ? rows : 0, F, a.ld_da, es)};
  if (!all_ok({out->gate, out->up, out->da}) || !aligned(a.gate, es) || !aligned(a.up, es) || !aligned(a.da, es))
    return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

template <typename T, int kAct>
int launch_rows(const ActArgs& a, int64_t rows, bool vec, uint8_t* data, int64_t ld_data, uint8_t* scale,
                int64_t scale_ld, hipStream_t stream) {
  const int64_t groups = groups_of(a.F), step = rows_per_launch(groups * 16);
  const MxqDivisor d = mxq_divisor((uint32_t)groups);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t total = std::min(step, rows - r) * groups;
    const dim3 grid((uint32_t)((total + kRowThreads / 16 - 1) / (kRowThreads / 16)));
    ActArgs s = a;   // from row r on
    s.gate = (const T*)a.gate + r * a.ld_gate;
    if (a.up) s.up = (const T*)a.up + r * a.ld_up;
    if (vec)
      hipLaunchKernelGGL((act_rows_kernel<T, kAct, true>), grid, dim3(kRowThreads), 0, stream, s, d, (uint32_t)total,
                         data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    else
      hipLaunchKernelGGL((act_rows_kernel<T, kAct, false>), grid, dim3(kRowThreads), 0, stream, s, d, (uint32_t)total,
                         data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
  return MXQ_OK;
}

// Rows a lane: four, in workgroups of 512, forward; eight, in workgroups of 256, backward, where four take 131 registers
// and so leave one workgroup a CU.  49152 x 1024 forward 53.6 us (eight: 54.6), backward 97 (four: 119).
constexpr int kForwardRows = 4, kBackwardRows = 8;

template <typename T, int kAct>
int launch_tiles(const ActArgs& a, int64_t rows, bool vec, const int32_t* offsets, int64_t experts, const TileOut& out,
                 hipStream_t stream) {
  const int64_t tiles = out.code_rows + (offsets ? 2 : 0);   // the rows of no expert, behind and before the others, may take two more
  constexpr int64_t kStep = 65535;   // of a grid's second dimension
  const bool both = a.da && a.up && a.F % kGroup == 0;
  // Payloads that fill half of the last-level cache leave with the non-temporal hint: forward 8192 x 14336 130.8 -> 125.4 us,
  // 49152 x 1024 53.9 -> 56.3; backward 49152 x 1024 103.6 -> 98.1.
  const bool big = rows * out.K > (int64_t)64 << 20;
  const int64_t columns = both ? a.F / kGroup : groups_of(out.K);
#define MXQ_ACT_LAUNCH(kRows, ...)                                                                                     \
  hipLaunchKernelGGL((__VA_ARGS__, kRows>), grid, dim3(16 * kGroup / kRows), 0, stream, a, (int)t, (int)rows, offsets, \
                     (int)experts, out)
  for (int64_t t = 0; t < tiles; t += kStep) {
    const dim3 grid((uint32_t)columns, (uint32_t)std::min(kStep, tiles - t));
    if (!a.da) {
      if (!vec) MXQ_ACT_LAUNCH(kForwardRows, act_tiles_kernel<T, kAct, false, false);
      else if (big) MXQ_ACT_LAUNCH(kForwardRows, act_tiles_kernel<T, kAct, true, true);
      else MXQ_ACT_LAUNCH(kForwardRows, act_tiles_kernel<T, kAct, true, false);
    } else if (both) {
      if (!vec) MXQ_ACT_LAUNCH(kBackwardRows, act_backward_kernel<T, kAct, false, false, true);
      else if (big) MXQ_ACT_LAUNCH(kBackwardRows, act_backward_kernel<T, kAct, true, true, true);
      else MXQ_ACT_LAUNCH(kBackwardRows, act_backward_kernel<T, kAct, true, false, true);
    } else {
      if (vec) MXQ_ACT_LAUNCH(kBackwardRows, act_backward_kernel<T, kAct, true, false, false);
      else MXQ_ACT_LAUNCH(kBackwardRows, act_backward_kernel<T, kAct, false, false, false);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_ACT_LAUNCH
  return MXQ_OK;
}

// The call for the activation and the type at hand.
#define MXQ_ACT_DISPATCH(fn, ...)                                                                        \
  switch (a.act * 2 + (dt == MXQ_FP32)) {                                                                \
    case MXQ_SILU * 2: return fn<uint16_t, MXQ_SILU>(__VA_ARGS__);                                       \
    case MXQ_SILU * 2 + 1: return fn<uint32_t, MXQ_SILU>(__VA_ARGS__);                                   \
    case MXQ_GELU_TANH * 2: return fn<uint16_t, MXQ_GELU_TANH>(__VA_ARGS__);                             \
    case MXQ_GELU_TANH * 2 + 1: return fn<uint32_t, MXQ_GELU_TANH>(__VA_ARGS__);                         \
    case MXQ_RELU2 * 2: return fn<uint16_t, MXQ_RELU2>(__VA_ARGS__);                                     \
    default: return fn<uint32_t, MXQ_RELU2>(__VA_ARGS__);                                                \
  }

int tile_entry(const ActArgs& a, int64_t rows, int64_t F, mxq_dtype dt, const int32_t* offsets, int64_t experts,
               uint8_t* row_data, int64_t ld_row, uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data,
               int64_t ld_col, uint8_t* col_scale, int64_t col_scale_ld, bool backward, hipStream_t stream) {
  if (offsets && (experts < 1 || experts > kMaxExperts)) return MXQ_ERR_SHAPE;
  Operands in;
  bool empty;
  const int st = check_operands(a, rows, F, dt, backward, &in, &empty);
  if (st != MXQ_OK) return st;
  const int64_t K = backward && a.up ? 2 * F : F;
  if (empty) return offsets && rows == 0 ? clear_code_rows(col_scale, col_scale_ld, experts, K, offsets, stream) : MXQ_OK;
  if (!row_data || !row_scale || !col_data || !col_scale) return MXQ_ERR_NULL;
  if (ld_row < K || row_scale_ld < groups_of(K) || ld_col < K || col_scale_ld < K) return MXQ_ERR_SHAPE;
  const int64_t code_rows = offsets ? rows / kGroup + experts : groups_of(rows);
  const Range rd = matrix_range(row_data, rows, K, ld_row, 1), rs = matrix_range(row_scale, rows, groups_of(K), row_scale_ld, 1),
              cd = matrix_range(col_data, rows, K, ld_col, 1), cs = matrix_range(col_scale, code_rows, K, col_scale_ld, 1),
              ro = matrix_range(offsets, 1, offsets ? experts + 1 : 0, experts + 1, 4);
  if (!all_ok({rd, rs, cd, cs, ro}) || !aligned(offsets, 4)) return MXQ_ERR_SHAPE;
  if (!disjoint({rd, rs, cd, cs}, {in.gate, in.up, in.da, ro})) return MXQ_ERR_ALIAS;
  const bool vec = F % kEPL == 0 && wide_rows(a.gate, a.ld_gate, dt) && wide_rows(a.up, a.ld_up, dt) && wide_rows(a.da, a.ld_da, dt) &&
                   wide_payload(row_data, ld_row) && wide_payload(col_data, ld_col);
  const TileOut out{(int)K, (int)code_rows, row_data, ld_row, row_scale, row_scale_ld, col_data, ld_col, col_scale, col_scale_ld};
  MXQ_ACT_DISPATCH(launch_tiles, a, rows, vec, offsets, experts, out, stream)
}

}  // namespace

extern "C" {

int mxq_activate_fp8_group128(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t rows, int64_t F,
                              mxq_dtype dt, mxq_activation act, uint8_t* data, int64_t ld_data, uint8_t* scale,
                              int64_t scale_ld, hipStream_t stream) {
  const ActArgs a{gate, up, nullptr, ld_gate, ld_up, 0, (int)std::min(F, kMaxDim), (int)act};
  Operands in;
  bool empty;
  const int st = check_operands(a, rows, F, dt, false, &in, &empty);
  if (st != MXQ_OK || empty) return st;
  if (!data || !scale) return MXQ_ERR_NULL;
  if (ld_data < F || scale_ld < groups_of(F)) return MXQ_ERR_SHAPE;
  const Range rd = matrix_range(data, rows, F, ld_data, 1), rs = matrix_range(scale, rows, groups_of(F), scale_ld, 1);
  if (!all_ok({rd, rs})) return MXQ_ERR_SHAPE;
  if (!disjoint({rd, rs}, {in.gate, in.up})) return MXQ_ERR_ALIAS;
  const bool vec = F % kEPL == 0 && wide_rows(gate, ld_gate, dt) && wide_rows(up, ld_up, dt) && wide_payload(data, ld_data);
  MXQ_ACT_DISPATCH(launch_rows, a, rows, vec, data, ld_data, scale, scale_ld, stream)
}

int mxq_activate_fp8_group128_row_col(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t rows,
                                      int64_t F, mxq_dtype dt, mxq_activation act, const int32_t* offsets,
                                      int64_t n_experts, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, hipStream_t stream) {
  const ActArgs a{gate, up, nullptr, ld_gate, ld_up, 0, (int)std::min(F, kMaxDim), (int)act};
  return tile_entry(a, rows, F, dt, offsets, n_experts, row_data, ld_row, row_scale, row_scale_ld, col_data, ld_col,
                    col_scale, col_scale_ld, false, stream);
}

int mxq_activate_fp8_group128_backward(const void* da, int64_t ld_da, const void* gate, int64_t ld_gate, const void* up,
                                       int64_t ld_up, int64_t rows, int64_t F, mxq_dtype dt, mxq_activation act,
                                       const int32_t* offsets, int64_t n_experts, uint8_t* row_data, int64_t ld_row,
                                       uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col,
                                       uint8_t* col_scale, int64_t col_scale_ld, hipStream_t stream) {
  const ActArgs a{gate, up, da, ld_gate, ld_up, ld_da, (int)std::min(F, kMaxDim), (int)act};
  return tile_entry(a, rows, F, dt, offsets, n_experts, row_data, ld_row, row_scale, row_scale_ld, col_data, ld_col,
                    col_scale, col_scale_ld, true, stream);
}

}  // extern "C"
