// activate.hip -- the activation between the two products of a feed-forward layer,
// with FP8 output in groups of 128, and its backward pass, on gfx950.
//
//   a = act(gate) up, or act(gate) where there is no up
//   silu(g) = g p(g), gelu(g) = g p(2 sqrt(2/pi) (g + 0.044715 g^3)) (its tanh form), relu2(g) = max(g, 0)^2
//   p(z) = 1 / (1 + exp(-z)), which is (1 + tanh(z / 2)) / 2
//   dgate = da up act'(gate), dup = da act(gate)
//
// Everything is computed in fp32 and rounded once, to E4M3.
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

// p(z), and 1 - p(z), without overflow and without cancellation in either tail.
struct Logistic {
  float p, q;
};
__device__ __forceinline__ Logistic logistic(float z) {
  const float e = exp2f(-fabsf(z) * 1.44269504088896341f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return z < 0 ? Logistic{e * r, r} : Logistic{r, e * r};
}

constexpr float kGelu = 1.59576912160573071f;   // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

__device__ __forceinline__ f32x8 act_of(int act, f32x8 g) {
  f32x8 a;
  if (act == MXQ_SILU) {
#pragma unroll
    for (int i = 0; i < kEPL; i++) a[i] = g[i] * logistic(g[i]).p;
  } else if (act == MXQ_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < kEPL; i++) a[i] = g[i] * logistic(kGelu * (g[i] + kCube * g[i] * g[i] * g[i])).p;
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++) a[i] = g[i] > 0 ? g[i] * g[i] : (g[i] <= 0 ? 0.0f : g[i]);   // a NaN stays one
  }
  return a;
}

// act(g) into *a, act'(g) as the result.
__device__ __forceinline__ f32x8 slope_of(int act, f32x8 g, f32x8* a) {
  f32x8 d;
  if (act == MXQ_SILU) {
#pragma unroll
    for (int i = 0; i < kEPL; i++) {
      const Logistic l = logistic(g[i]);
      (*a)[i] = g[i] * l.p;
      d[i] = l.p * (1.0f + g[i] * l.q);
    }
  } else if (act == MXQ_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < kEPL; i++) {
      const float g2 = g[i] * g[i];
      const Logistic l = logistic(kGelu * g[i] * (1.0f + kCube * g2));
      (*a)[i] = g[i] * l.p;
      // far out q is 0 and g may be anything: the product is then 0, not 0 * Inf
      const float t = l.p * l.q;
      d[i] = l.p + (t == 0.0f ? 0.0f : g[i] * t * kGelu * (1.0f + 3.0f * kCube * g2));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++) {
      const float r = g[i] > 0 ? g[i] : (g[i] <= 0 ? 0.0f : g[i]);
      (*a)[i] = r * r;
      d[i] = 2.0f * r;
    }
  }
  return d;
}

template <typename T, bool kVec>
__device__ __forceinline__ f32x8 value_at(const ActArgs& s, int64_t r, int c) {
  const f32x8 g = load_floats<T, kVec>((const T*)s.gate + r * s.ld_gate, c, s.F);
  f32x8 a = act_of(s.act, g);
  if (s.up) a *= load_floats<T, kVec>((const T*)s.up + r * s.ld_up, c, s.F);
  return a;
}

// ---- groups along the rows ------------------------------------------------------------
// 16 lanes per group, 16 groups per workgroup, one group a lane.
constexpr int kRowThreads = 256;

template <typename T, bool kVec>
__global__ __launch_bounds__(kRowThreads) void act_rows_kernel(ActArgs s, MxqDivisor groups, uint32_t total,
                                                               uint8_t* data, int64_t ld_data, uint8_t* scale,
                                                               int64_t scale_ld) {
  keep_denormals();
  const uint32_t g = blockIdx.x * (kRowThreads / 16) + threadIdx.x / 16;
  if (g >= total) return;   // whole groups of 16 lanes leave together
  const uint32_t r = mxq_quot(g, groups), b = g - r * groups.d;
  const int c = (int)b * kGroup + (threadIdx.x & 15) * kEPL;
  const f32x8 a = value_at<T, kVec>(s, r, c);
  store_group<kVec, false>(data + (int64_t)r * ld_data, scale + (int64_t)r * scale_ld, c, s.F, a);
}

// ---- groups along both -----------------------------------------------------------------
template <typename T, bool kVec, bool kStream>
__global__ __launch_bounds__(kTileThreads) void act_tiles_kernel(ActArgs s, int first_id, int rows,
                                                                 const int32_t* offsets, int experts, TileOut out) {
  keep_denormals();
  __shared__ TilePart part;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup + (threadIdx.x & 15) * kEPL;
  const TileRows t = tile_rows(offsets, experts, rows, id);
  if (!t.owned) clear_codes(out, id, blockIdx.x);
  if (t.first >= t.hi) return;   // the same for the whole workgroup
  Chunk<uint32_t> v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = t.first + threadIdx.x / 16 + 16 * i;
    v[i] = narrow<uint32_t>(r < t.hi ? value_at<T, kVec>(s, r, c) : f32x8{});
  }
  store_tile<uint32_t, kVec, true, kStream>(v, out, t, id, blockIdx.x, part);
}

// ---- backward ----------------------------------------------------------------------------
// Eight elements of dgate, and of dup, from column c of the halves.
struct Both {
  f32x8 gate, up;
};
template <typename T, bool kVec>
__device__ __forceinline__ Both gradients_at(const ActArgs& s, int64_t r, int c) {
  const f32x8 g = load_floats<T, kVec>((const T*)s.gate + r * s.ld_gate, c, s.F);
  const f32x8 da = load_floats<T, kVec>((const T*)s.da + r * s.ld_da, c, s.F);
  f32x8 a;
  const f32x8 d = slope_of(s.act, g, &a);
  if (!s.up) return Both{da * d, f32x8{}};
  const f32x8 u = load_floats<T, kVec>((const T*)s.up + r * s.ld_up, c, s.F);
  return Both{da * u * d, da * a};
}

// Elements [c, c + 8) of a row [dgate, dup].
template <typename T, bool kVec>
__device__ __forceinline__ f32x8 gradient_at(const ActArgs& s, int64_t r, int c) {
  if (!s.up || c + kEPL <= s.F) return gradients_at<T, kVec>(s, r, c).gate;
  if (c >= s.F) return gradients_at<T, kVec>(s, r, c - s.F).up;
  // across the end of the first half: elements from F on are the first of the second
  f32x8 v = gradients_at<T, false>(s, r, c).gate;
  const f32x8 u = gradients_at<T, false>(s, r, 0).up;
  const int n = s.F - c;
#pragma unroll
  for (int i = 0; i < kEPL; i++) {
#pragma unroll
    for (int j = 0; j < kEPL; j++)
      if (i == n + j) v[i] = u[j];
  }
  return v;
}

// kBoth: a workgroup takes the same 128 columns of both halves (F is a multiple of 128), which reads them once;
// otherwise 128 columns of the result, wherever they lie.
template <typename T, bool kVec, bool kBoth, bool kStream>
__global__ __launch_bounds__(kTileThreads) void act_backward_kernel(ActArgs s, int first_id, int rows,
                                                                    const int32_t* offsets, int experts, TileOut out) {
  keep_denormals();
  __shared__ TilePart part;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup + (threadIdx.x & 15) * kEPL;
  const TileRows t = tile_rows(offsets, experts, rows, id);
  if (!t.owned) {
    clear_codes(out, id, blockIdx.x);
    if (kBoth) clear_codes(out, id, blockIdx.x + s.F / kGroup);
  }
  if (t.first >= t.hi) return;   // the same for the whole workgroup
  Chunk<uint32_t> v[kTileRows], u[kBoth ? kTileRows : 1];
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = t.first + threadIdx.x / 16 + 16 * i;
    if constexpr (kBoth) {
      const Both b = r < t.hi ? gradients_at<T, kVec>(s, r, c) : Both{};
      v[i] = narrow<uint32_t>(b.gate);
      u[i] = narrow<uint32_t>(b.up);
    } else {
      v[i] = narrow<uint32_t>(r < t.hi && c < out.K ? gradient_at<T, kVec>(s, r, c) : f32x8{});
    }
  }
  store_tile<uint32_t, kVec, true, kStream>(v, out, t, id, blockIdx.x, part);
  if constexpr (kBoth) {
    __syncthreads();
    store_tile<uint32_t, kVec, true, kStream>(u, out, t, id, blockIdx.x + s.F / kGroup, part);
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

template <typename T>
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
      hipLaunchKernelGGL((act_rows_kernel<T, true>), grid, dim3(kRowThreads), 0, stream, s, d, (uint32_t)total,
                         data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    else
      hipLaunchKernelGGL((act_rows_kernel<T, false>), grid, dim3(kRowThreads), 0, stream, s, d, (uint32_t)total,
                         data + r * ld_data, ld_data, scale + r * scale_ld, scale_ld);
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
  return MXQ_OK;
}

template <typename T>
int launch_tiles(const ActArgs& a, int64_t rows, bool vec, const int32_t* offsets, int64_t experts, const TileOut& out,
                 hipStream_t stream) {
  const int64_t tiles = out.code_rows + (offsets ? 2 : 0);   // the rows of no expert, behind and before the others, may take two more
  constexpr int64_t kStep = 65535;   // of a grid's second dimension
  const bool both = a.da && a.up && a.F % kGroup == 0;
  const bool big = rows * out.K > kStreamBytes;
  const int64_t columns = both ? a.F / kGroup : groups_of(out.K);
  const dim3 block(kTileThreads);
#define MXQ_ACT_LAUNCH(...)                                                                                       \
  hipLaunchKernelGGL((__VA_ARGS__), grid, block, 0, stream, a, (int)t, (int)rows, offsets, (int)experts, out)
  for (int64_t t = 0; t < tiles; t += kStep) {
    const dim3 grid((uint32_t)columns, (uint32_t)std::min(kStep, tiles - t));
    if (!a.da) {
      if (!vec) MXQ_ACT_LAUNCH(act_tiles_kernel<T, false, false>);
      else if (big) MXQ_ACT_LAUNCH(act_tiles_kernel<T, true, true>);
      else MXQ_ACT_LAUNCH(act_tiles_kernel<T, true, false>);
    } else if (both) {
      if (!vec) MXQ_ACT_LAUNCH(act_backward_kernel<T, false, true, false>);
      else if (big) MXQ_ACT_LAUNCH(act_backward_kernel<T, true, true, true>);
      else MXQ_ACT_LAUNCH(act_backward_kernel<T, true, true, false>);
    } else {
      if (!vec) MXQ_ACT_LAUNCH(act_backward_kernel<T, false, false, false>);
      else if (big) MXQ_ACT_LAUNCH(act_backward_kernel<T, true, false, true>);
      else MXQ_ACT_LAUNCH(act_backward_kernel<T, true, false, false>);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_ACT_LAUNCH
  return MXQ_OK;
}

int tile_entry(const ActArgs& a, int64_t rows, int64_t F, mxq_dtype dt, const int32_t* offsets, int64_t experts,
               uint8_t* row_data, int64_t ld_row, uint8_t* row_scale, int64_t row_scale_ld, uint8_t* col_data,
               int64_t ld_col, uint8_t* col_scale, int64_t col_scale_ld, bool backward, hipStream_t stream) {
  if (offsets && (experts < 1 || experts > kMaxExperts)) return MXQ_ERR_SHAPE;
  Operands in;
  bool empty;
  const int st = check_operands(a, rows, F, dt, backward, &in, &empty);
  if (st != MXQ_OK || empty) return st;
  if (!row_data || !row_scale || !col_data || !col_scale) return MXQ_ERR_NULL;
  const int64_t K = backward && a.up ? 2 * F : F;
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
  return dt == MXQ_BF16 ? launch_tiles<uint16_t>(a, rows, vec, offsets, experts, out, stream)
                        : launch_tiles<uint32_t>(a, rows, vec, offsets, experts, out, stream);
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
  return dt == MXQ_BF16 ? launch_rows<uint16_t>(a, rows, vec, data, ld_data, scale, scale_ld, stream)
                        : launch_rows<uint32_t>(a, rows, vec, data, ld_data, scale, scale_ld, stream);
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
