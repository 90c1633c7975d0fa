// norm.hip -- root-mean-square norm of rows with the residual's addition and FP8
// output in groups of 128, and its backward pass, on gfx950.
//
//   s = x + residual, rounded to the residual's type; y = s r w, r = 1 / sqrt(mean(s^2) + eps)
//
// The norm is that of s as it is stored, so that a backward pass, or a forward pass that is
// run again from the stored s, works on the same values.  Sums are in fp32.  A
// row whose sum of squares passes 2^128 is summed again with its values times 2^-80.
//
//   u = s r, g = dy w:  dx = r (g - u mean(g u)) + dresidual,  dw = sum over rows of dy u
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "floats.h"

namespace {

using namespace mxq_host;
using namespace mxq_dev;

// What a row's values are multiplied by: s * r, then * f (the other way round small values of a row of huge ones
// would vanish on the way).  f is 1 but for rows whose squares overflow.
struct Stats {
  float f, r;
};

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t ld_x, ld_res;
  bool w_bf16;
  float eps;
  int rows, K;
  void *sum, *y;
  int64_t ld_sum, ld_y;
  uint8_t *data, *scale;
  int64_t ld_data, scale_ld;
  Stats* stats;
};

constexpr float kDown = 0x1p-80f;

template <bool kVec>
__device__ __forceinline__ f32x8 weight_at(const void* w, bool bf16, int c, int K) {
  if (!w) return f32x8{1, 1, 1, 1, 1, 1, 1, 1};
  return bf16 ? load_floats<uint16_t, kVec>(w, c, K) : load_floats<uint32_t, kVec>(w, c, K);
}

// Elements [c, c + 8) of s of a row.
template <typename TX, typename TS, bool kVec>
__device__ __forceinline__ f32x8 stream_at(const NormArgs& a, int64_t row, int c) {
  const f32x8 x = load_floats<TX, kVec>((const TX*)a.x + row * a.ld_x, c, a.K);
  if (!a.residual) return x;
  const f32x8 r = load_floats<TS, kVec>((const TS*)a.residual + row * a.ld_res, c, a.K);
  return widen<TS>(narrow<TS>(x + r));
}

// Sum over the kLanes lanes of a row, the same in each of them; several waves of a row meet in LDS.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* part) {
  if constexpr (kLanes <= 64) return lane_sum<kLanes>(v);
  v = lane_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  float s = part[0];
#pragma unroll
  for (int i = 1; i < kLanes / 64; i++) s += part[i];
  return s;
}

__device__ __forceinline__ float inverse_root(float sum, float f, const NormArgs& a) {
  return 1.0f / sqrtf(sum / (float)a.K + a.eps * f * f);
}

constexpr int kThreads = 256;

// A row in the registers of kLanes lanes, kChunks pieces of eight elements each.
template <typename TX, typename TS, int kLanes, int kChunks, bool kVec>
__global__ __launch_bounds__(kLanes > kThreads ? kLanes : kThreads) void norm_kernel(NormArgs a) {
  keep_denormals();
  constexpr int kRows = kLanes < kThreads ? kThreads / kLanes : 1;
  __shared__ float part[16];
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (row >= a.rows) return;   // a workgroup that meets at barriers has one row
  f32x8 s[kChunks];
  float sum = 0;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * kEPL;
    s[i] = stream_at<TX, TS, kVec>(a, row, c);
  }
#pragma unroll
  for (int i = 0; i < kChunks; i++) sum += add8(s[i] * s[i]);
  Stats t{1.0f, 0.0f};
  sum = row_sum<kLanes>(sum, part);
  if (!(sum < __builtin_inff())) {   // the same for the whole row
    t.f = kDown;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kChunks; i++) sum += add8((s[i] * kDown) * (s[i] * kDown));
    sum = row_sum<kLanes>(sum, part);
  }
  t.r = inverse_root(sum, t.f, a);
  if (a.stats && lane == 0) a.stats[row] = t;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * kEPL;
    const f32x8 y = s[i] * t.r * t.f * weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
    if (a.sum) store_floats<TS, kVec>((TS*)a.sum + row * a.ld_sum, c, a.K, s[i]);
    if (a.y) store_floats<TX, kVec>((TX*)a.y + row * a.ld_y, c, a.K, y);
    if (a.data) store_group<kVec, false>(a.data + row * a.ld_data, a.scale + row * a.scale_ld, c, a.K, y);
  }
}

// Rows that the registers do not hold: a workgroup walks the row, s is read again for the results.
constexpr int kLong = 1024;

template <typename TX, typename TS, bool kVec>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormArgs a) {
  keep_denormals();
  __shared__ float part[16];
  const int64_t row = blockIdx.x;
  TS* const stored = a.sum ? (TS*)a.sum + row * a.ld_sum : nullptr;
  float sum = 0;
  for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kLong * kEPL) {
    const f32x8 s = stream_at<TX, TS, kVec>(a, row, (int)c);
    if (stored) store_floats<TS, kVec>(stored, (int)c, a.K, s);   // the residual may be stored in its own place
    sum += add8(s * s);
  }
  const auto again = [&](int c) {
    return stored ? load_floats<TS, kVec>(stored, c, a.K) : stream_at<TX, TS, kVec>(a, row, c);
  };
  Stats t{1.0f, 0.0f};
  sum = row_sum<kLong>(sum, part);
  if (!(sum < __builtin_inff())) {
    t.f = kDown;
    sum = 0;
    for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kLong * kEPL) {
      const f32x8 s = again((int)c) * kDown;
      sum += add8(s * s);
    }
    sum = row_sum<kLong>(sum, part);
  }
  t.r = inverse_root(sum, t.f, a);
  if (a.stats && threadIdx.x == 0) a.stats[row] = t;
  // all lanes of a group of 16 walk as far
  for (int64_t c0 = (threadIdx.x & ~15) * kEPL; c0 < a.K; c0 += kLong * kEPL) {
    const int c = (int)c0 + (threadIdx.x & 15) * kEPL;
    const f32x8 y = again(c) * t.r * t.f * weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
    if (a.y) store_floats<TX, kVec>((TX*)a.y + row * a.ld_y, c, a.K, y);
    if (a.data) store_group<kVec, false>(a.data + row * a.ld_data, a.scale + row * a.scale_ld, c, a.K, y);
  }
}

// Groups along the columns, from s and each row's statistics.
template <typename TX, typename TS, bool kVec, bool kStream>
__global__ __launch_bounds__(kTileThreads) void norm_columns_kernel(NormArgs a, int first_id, TileOut out) {
  keep_denormals();
  __shared__ TileShared<kTileRows> shared;
  const int id = first_id + (int)blockIdx.y, c = blockIdx.x * kGroup + (threadIdx.x & 15) * kEPL;
  const TileRows t = tile_rows(nullptr, 0, a.rows, id, shared);
  const f32x8 w = weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
  Chunk<uint32_t> v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; i++) {
    const int64_t r = t.first + threadIdx.x / 16 + 16 * i;
    f32x8 s{};
    Stats st{};
    if (r < a.rows) {
      s = a.sum ? load_floats<TS, kVec>((const TS*)a.sum + r * a.ld_sum, c, a.K) : stream_at<TX, TS, kVec>(a, r, c);
      st = a.stats[r];
    }
    v[i] = narrow<uint32_t>(s * st.r * st.f * w);
  }
  if (kVec && whole_tile(t, blockIdx.x, a.K)) store_tile<uint32_t, kVec, false, kStream, kVec>(v, out, t, id, blockIdx.x, shared);
  else store_tile<uint32_t, kVec, false, kStream, false>(v, out, t, id, blockIdx.x, shared);
}

// ---- backward ----------------------------------------------------------------------------
struct BackArgs {
  const void *dy, *s, *weight, *dres;
  int64_t ld_dy, ld_s, ld_dres;
  bool w_bf16;
  float eps;
  int rows, K, per_block;   // rows of a block of the second kernel
  void* dx;
  int64_t ld_dx;
  float4* stats;            // f, r, mean(g u) of each row
  float* part;              // [blocks, K] sums of dw; null: not wanted
};

template <typename TY, typename TS, bool kVec>
__global__ __launch_bounds__(kThreads) void back_stats_kernel(BackArgs a) {
  keep_denormals();
  __shared__ float part[16];
  const int64_t row = blockIdx.x;
  const TS* const s = (const TS*)a.s + row * a.ld_s;
  const TY* const dy = (const TY*)a.dy + row * a.ld_dy;
  float f = 1.0f, sum, dot;
  for (;;) {
    sum = dot = 0;
    for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kThreads * kEPL) {
      const f32x8 v = load_floats<TS, kVec>(s, (int)c, a.K) * f;
      const f32x8 g = load_floats<TY, kVec>(dy, (int)c, a.K) * weight_at<kVec>(a.weight, a.w_bf16, (int)c, a.K);
      sum += add8(v * v);
      dot += add8(g * v);
    }
    sum = row_sum<kThreads>(sum, part);
    dot = row_sum<kThreads>(dot, part);
    if (sum < __builtin_inff() || f != 1.0f) break;
    f = kDown;
  }
  const float r = 1.0f / sqrtf(sum / (float)a.K + a.eps * f * f);
  if (threadIdx.x == 0) a.stats[row] = float4{f, r, dot * r / (float)a.K, 0.0f};
}

// dx of a block of rows and 2048 columns, and its part of dw.
template <typename TY, typename TS, bool kVec>
__global__ __launch_bounds__(kThreads) void back_rows_kernel(BackArgs a) {
  keep_denormals();
  const int64_t c64 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kEPL;
  if (c64 >= a.K) return;
  const int c = (int)c64;
  const int64_t lo = (int64_t)blockIdx.y * a.per_block;
  const int64_t hi = min(lo + a.per_block, (int64_t)a.rows);
  const f32x8 w = weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
  f32x8 dw{};
  for (int64_t row = lo; row < hi; row++) {
    const float4 t = a.stats[row];
    const f32x8 u = load_floats<TS, kVec>((const TS*)a.s + row * a.ld_s, c, a.K) * t.y * t.x;
    const f32x8 dy = load_floats<TY, kVec>((const TY*)a.dy + row * a.ld_dy, c, a.K);
    f32x8 dx = (dy * w - u * t.z) * t.y * t.x;
    if (a.dres) dx += load_floats<TS, kVec>((const TS*)a.dres + row * a.ld_dres, c, a.K);
    store_floats<TS, kVec>((TS*)a.dx + row * a.ld_dx, c, a.K, dx);
    dw += dy * u;
  }
  if (a.part) {
    float* const p = a.part + (int64_t)blockIdx.y * a.K;
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < a.K) p[c + i] = dw[i];
  }
}

// dw: the blocks' parts added up in their order, 64 columns a workgroup, its 16 waves taking turns.
constexpr int kFoldThreads = 1024;
__global__ __launch_bounds__(kFoldThreads) void back_weight_kernel(const float* part, int blocks, int K, float* dw) {
  __shared__ float sums[kFoldThreads / 64][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int c = blockIdx.x * 64 + lane;
  float sum = 0;
  if (c < K)
    for (int b = wave; b < blocks; b += kFoldThreads / 64) sum += part[(int64_t)b * K + c];
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && c < K) {
#pragma unroll
    for (int i = 1; i < kFoldThreads / 64; i++) sum += sums[i][lane];
    dw[c] = sum;
  }
}

// ---- host --------------------------------------------------------------------------------

#define MXQ_TRY(call)              \
  do {                             \
    const int st_ = (call);        \
    if (st_ != MXQ_OK) return st_; \
  } while (0)

// The same arguments from row r on, `n` of them.
template <typename TX, typename TS>
NormArgs from_row(NormArgs a, int64_t r, int64_t n) {
  a.x = (const TX*)a.x + r * a.ld_x;
  if (a.residual) a.residual = (const TS*)a.residual + r * a.ld_res;
  if (a.sum) a.sum = (TS*)a.sum + r * a.ld_sum;
  if (a.y) a.y = (TX*)a.y + r * a.ld_y;
  if (a.data) a.data += r * a.ld_data, a.scale += r * a.scale_ld;
  if (a.stats) a.stats += r;
  a.rows = (int)n;
  return a;
}

template <typename TX, typename TS, int kLanes, int kChunks, bool kVec>
int launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int threads = std::max(kLanes, kThreads), per = threads / kLanes;
  const int64_t step = rows_per_launch(kLanes);
  for (int64_t r = 0; r < a.rows; r += step) {
    const int64_t n = std::min<int64_t>(step, a.rows - r);
    hipLaunchKernelGGL((norm_kernel<TX, TS, kLanes, kChunks, kVec>), dim3((uint32_t)((n + per - 1) / per)), dim3(threads),
                       0, stream, from_row<TX, TS>(a, r, n));
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

// A row takes as many lanes as hold it in up to eight pieces each.
template <typename TX, typename TS, bool kVec>
int norm_rows(const NormArgs& a, hipStream_t stream) {
  const int K = a.K;
  if (K <= 16 * 8) return launch_norm<TX, TS, 16, 1, kVec>(a, stream);
  if (K <= 64 * 8) return launch_norm<TX, TS, 64, 1, kVec>(a, stream);
  if (K <= 256 * 8) return launch_norm<TX, TS, 256, 1, kVec>(a, stream);
  if (K <= 256 * 16) return launch_norm<TX, TS, 256, 2, kVec>(a, stream);
  if (K <= 256 * 32) return launch_norm<TX, TS, 256, 4, kVec>(a, stream);
  if (K <= 1024 * 16) return launch_norm<TX, TS, 1024, 2, kVec>(a, stream);
  const int64_t step = rows_per_launch(kLong);
  for (int64_t r = 0; r < a.rows; r += step) {
    const int64_t n = std::min<int64_t>(step, a.rows - r);
    hipLaunchKernelGGL((norm_long_kernel<TX, TS, kVec>), dim3((uint32_t)n), dim3(kLong), 0, stream,
                       from_row<TX, TS>(a, r, n));
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

template <typename TX, typename TS>
int norm_columns(const NormArgs& a, const TileOut& out, bool vec, hipStream_t stream) {
  const int64_t tiles = groups_of(a.rows);
  const bool big = (int64_t)a.rows * a.K > kStreamBytes;
  constexpr int64_t kStep = 65535;   // of a grid's second dimension
  for (int64_t t = 0; t < tiles; t += kStep) {
    const dim3 grid((uint32_t)groups_of(a.K), (uint32_t)std::min(kStep, tiles - t)), block(kTileThreads);
    if (!vec) hipLaunchKernelGGL((norm_columns_kernel<TX, TS, false, false>), grid, block, 0, stream, a, (int)t, out);
    else if (big) hipLaunchKernelGGL((norm_columns_kernel<TX, TS, true, true>), grid, block, 0, stream, a, (int)t, out);
    else hipLaunchKernelGGL((norm_columns_kernel<TX, TS, true, false>), grid, block, 0, stream, a, (int)t, out);
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

template <typename TX, typename TS>
int norm_launch(const NormArgs& a, const TileOut* columns, bool vec, hipStream_t stream) {
  MXQ_TRY(vec ? (norm_rows<TX, TS, true>(a, stream)) : (norm_rows<TX, TS, false>(a, stream)));
  return columns ? norm_columns<TX, TS>(a, *columns, vec, stream) : MXQ_OK;
}

struct Columns {
  uint8_t *data, *scale;
  int64_t ld, scale_ld;
  void* workspace;
  int64_t bytes;
};

int norm_entry(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, mxq_dtype res_dt, const void* weight,
               mxq_dtype w_dt, float eps, int64_t rows, int64_t K, mxq_dtype dt, void* sum, int64_t ld_sum, void* y,
               int64_t ld_y, bool fp8, uint8_t* data, int64_t ld_data, uint8_t* scale, int64_t scale_ld,
               const Columns* col, hipStream_t stream) {
  if (!residual) res_dt = dt;
  if (!is_float(dt) || !is_float(res_dt) || (weight && !is_float(w_dt))) return MXQ_ERR_DTYPE;
  if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim || !(eps > 0) || !(eps < __builtin_inff())) return MXQ_ERR_SHAPE;
  if (rows == 0 || K == 0) return MXQ_OK;
  if (!x || (sum && !residual) || (fp8 ? !data || !scale : !y)) return MXQ_ERR_NULL;
  const int64_t need = col ? mxq_rms_norm_fp8_group128_row_col_workspace(rows) : 0;
  if (col && (!col->data || !col->scale || !col->workspace)) return MXQ_ERR_NULL;
  if (ld_x < K || (residual && ld_res < K) || (sum && ld_sum < K) || (y && ld_y < K) ||
      (fp8 && (ld_data < K || scale_ld < groups_of(K))) ||
      (col && (col->ld < K || col->scale_ld < K || col->bytes < need)))
    return MXQ_ERR_SHAPE;
  const size_t es = size_of(dt), rs = size_of(res_dt);
  const Range rx = matrix_range(x, rows, K, ld_x, es), rr = matrix_range(residual, residual ? rows : 0, K, ld_res, rs),
              rw = matrix_range(weight, weight ? 1 : 0, K, K, weight ? size_of(w_dt) : 4),
              ru = matrix_range(sum, sum ? rows : 0, K, ld_sum, rs), ry = matrix_range(y, y ? rows : 0, K, ld_y, es),
              rd = matrix_range(data, fp8 ? rows : 0, K, ld_data, 1),
              rc = matrix_range(scale, fp8 ? rows : 0, groups_of(K), scale_ld, 1),
              cd = matrix_range(col ? col->data : nullptr, col ? rows : 0, K, col ? col->ld : 0, 1),
              cc = matrix_range(col ? col->scale : nullptr, col ? groups_of(rows) : 0, K, col ? col->scale_ld : 0, 1),
              wk = matrix_range(col ? col->workspace : nullptr, 1, need, need, 1);
  if (!all_ok({rx, rr, rw, ru, ry, rd, rc, cd, cc, wk}) || !aligned(x, es) || !aligned(y, es) || !aligned(residual, rs) ||
      !aligned(sum, rs) || (weight && !aligned(weight, size_of(w_dt))) || (col && !aligned(col->workspace, 8)))
    return MXQ_ERR_SHAPE;
  // the sum may be stored in the residual's own place: each element is read before it is written, by the same lane
  const bool in_place = sum && sum == residual && ld_sum == ld_res;
  if (!disjoint({ru, ry, rd, rc, cd, cc, wk}, {rx, in_place ? Range{0, 0, true} : rr, rw})) return MXQ_ERR_ALIAS;
  const bool vec = K % kEPL == 0 && wide_rows(x, ld_x, dt) && wide_rows(residual, ld_res, res_dt) && wide_rows(sum, ld_sum, res_dt) &&
                   wide_rows(y, ld_y, dt) && (!weight || aligned(weight, 16)) && wide_payload(fp8 ? data : nullptr, ld_data) &&
                   (!col || wide_payload(col->data, col->ld));
  const NormArgs a{x,   residual, weight, ld_x, ld_res, w_dt == MXQ_BF16,     eps,   (int)rows, (int)K,
                   sum, y,        ld_sum, ld_y, fp8 ? data : nullptr, scale, ld_data, scale_ld,
                   col ? (Stats*)col->workspace : nullptr};
  TileOut out{};
  if (col)
    out = TileOut{(int)K, (int)groups_of(rows), nullptr, 0, nullptr, 0, col->data, col->ld, col->scale, col->scale_ld};
  const TileOut* const o = col ? &out : nullptr;
  if (dt == MXQ_BF16)
    return res_dt == MXQ_BF16 ? norm_launch<uint16_t, uint16_t>(a, o, vec, stream)
                              : norm_launch<uint16_t, uint32_t>(a, o, vec, stream);
  return res_dt == MXQ_BF16 ? norm_launch<uint32_t, uint16_t>(a, o, vec, stream)
                            : norm_launch<uint32_t, uint32_t>(a, o, vec, stream);
}

// Rows of a block of the backward pass: enough blocks to fill the card, few enough that their parts stay small.
int64_t back_rows_per_block(int64_t rows) { return std::max<int64_t>(4, (rows + 255) / 256); }
int64_t back_blocks(int64_t rows) {
  const int64_t per = back_rows_per_block(rows);
  return (rows + per - 1) / per;
}

template <typename TY, typename TS, bool kVec>
int back_launch(BackArgs a, float* dw, hipStream_t stream) {
  const int64_t step = rows_per_launch(kThreads), blocks = back_blocks(a.rows);
  for (int64_t r = 0; r < a.rows; r += step) {
    BackArgs b = a;
    b.s = (const TS*)a.s + r * a.ld_s;
    b.dy = (const TY*)a.dy + r * a.ld_dy;
    b.stats = a.stats + r;
    hipLaunchKernelGGL((back_stats_kernel<TY, TS, kVec>), dim3((uint32_t)std::min<int64_t>(step, a.rows - r)),
                       dim3(kThreads), 0, stream, b);
    MXQ_TRY(launch_status());
  }
  const uint32_t strips = (uint32_t)((a.K + kThreads * kEPL - 1) / (kThreads * kEPL));
  hipLaunchKernelGGL((back_rows_kernel<TY, TS, kVec>), dim3(strips, (uint32_t)blocks), dim3(kThreads), 0, stream, a);
  MXQ_TRY(launch_status());
  if (!dw) return MXQ_OK;
  hipLaunchKernelGGL(back_weight_kernel, dim3((uint32_t)((a.K + 63) / 64)), dim3(kFoldThreads), 0, stream, a.part,
                     (int)blocks, a.K, dw);
  return launch_status();
}

template <typename TY, typename TS>
int back_launch(const BackArgs& a, bool vec, float* dw, hipStream_t stream) {
  return vec ? back_launch<TY, TS, true>(a, dw, stream) : back_launch<TY, TS, false>(a, dw, stream);
}

}  // namespace

extern "C" {

int mxq_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, mxq_dtype residual_dt,
                 const void* weight, mxq_dtype weight_dt, float eps, int64_t rows, int64_t K, mxq_dtype dt, void* sum,
                 int64_t ld_sum, void* y, int64_t ld_y, hipStream_t stream) {
  return norm_entry(x, ld_x, residual, ld_residual, residual_dt, weight, weight_dt, eps, rows, K, dt, sum, ld_sum, y,
                    ld_y, false, nullptr, 0, nullptr, 0, nullptr, stream);
}

int mxq_rms_norm_fp8_group128(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                              mxq_dtype residual_dt, const void* weight, mxq_dtype weight_dt, float eps, int64_t rows,
                              int64_t K, mxq_dtype dt, void* sum, int64_t ld_sum, void* y, int64_t ld_y, uint8_t* data,
                              int64_t ld_data, uint8_t* scale, int64_t scale_ld, hipStream_t stream) {
  return norm_entry(x, ld_x, residual, ld_residual, residual_dt, weight, weight_dt, eps, rows, K, dt, sum, ld_sum, y,
                    ld_y, true, data, ld_data, scale, scale_ld, nullptr, stream);
}

int64_t mxq_rms_norm_fp8_group128_row_col_workspace(int64_t rows) {
  return rows < 1 || rows > kMaxDim ? 0 : rows * (int64_t)sizeof(Stats);
}

int mxq_rms_norm_fp8_group128_row_col(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                                      mxq_dtype residual_dt, const void* weight, mxq_dtype weight_dt, float eps,
                                      int64_t rows, int64_t K, mxq_dtype dt, void* sum, int64_t ld_sum, void* y,
                                      int64_t ld_y, uint8_t* row_data, int64_t ld_row, uint8_t* row_scale,
                                      int64_t row_scale_ld, uint8_t* col_data, int64_t ld_col, uint8_t* col_scale,
                                      int64_t col_scale_ld, void* workspace, int64_t workspace_bytes,
                                      hipStream_t stream) {
  const Columns col{col_data, col_scale, ld_col, col_scale_ld, workspace, workspace_bytes};
  return norm_entry(x, ld_x, residual, ld_residual, residual_dt, weight, weight_dt, eps, rows, K, dt, sum, ld_sum, y,
                    ld_y, true, row_data, ld_row, row_scale, row_scale_ld, &col, stream);
}

int64_t mxq_rms_norm_backward_workspace(int64_t rows, int64_t K) {
  if (rows < 1 || K < 1 || rows > kMaxDim || K > kMaxDim) return 0;
  return rows * 16 + back_blocks(rows) * K * 4;
}

int mxq_rms_norm_backward(const void* dy, int64_t ld_dy, mxq_dtype dt, const void* x, int64_t ld_x, mxq_dtype x_dt,
                          const void* weight, mxq_dtype weight_dt, float eps, const void* dresidual,
                          int64_t ld_dresidual, int64_t rows, int64_t K, void* dx, int64_t ld_dx, float* dweight,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!is_float(dt) || !is_float(x_dt) || (weight && !is_float(weight_dt))) return MXQ_ERR_DTYPE;
  if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim || !(eps > 0) || !(eps < __builtin_inff())) return MXQ_ERR_SHAPE;
  if (K == 0) return MXQ_OK;
  const size_t ys = size_of(dt), xs = size_of(x_dt);
  if (rows > 0 && (!dy || !x || !dx || !workspace)) return MXQ_ERR_NULL;
  if (rows > 0 && (ld_dy < K || ld_x < K || ld_dx < K || (dresidual && ld_dresidual < K))) return MXQ_ERR_SHAPE;
  const int64_t need = mxq_rms_norm_backward_workspace(rows, K);
  if (workspace_bytes < need) return MXQ_ERR_SHAPE;
  const Range rg = matrix_range(dy, rows, K, ld_dy, ys), rx = matrix_range(x, rows, K, ld_x, xs),
              rw = matrix_range(weight, weight ? 1 : 0, K, K, weight ? size_of(weight_dt) : 4),
              rr = matrix_range(dresidual, dresidual ? rows : 0, K, ld_dresidual, xs),
              rd = matrix_range(dx, rows, K, ld_dx, xs), rv = matrix_range(dweight, dweight ? 1 : 0, K, K, 4),
              wk = matrix_range(workspace, 1, need, need, 1);
  if (!all_ok({rg, rx, rw, rr, rd, rv, wk}) || !aligned(dy, ys) || !aligned(x, xs) || !aligned(dresidual, xs) ||
      !aligned(dx, xs) || !aligned(dweight, 4) || !aligned(workspace, 16) ||
      (weight && !aligned(weight, size_of(weight_dt))))
    return MXQ_ERR_SHAPE;
  if (!disjoint({rd, rv, wk}, {rg, rx, rw, rr})) return MXQ_ERR_ALIAS;
  if (rows == 0) {   // the gradient of a weight that met no row
    if (!dweight) return MXQ_OK;
    hipLaunchKernelGGL(back_weight_kernel, dim3((uint32_t)((K + 63) / 64)), dim3(kFoldThreads), 0, stream,
                       (const float*)nullptr, 0, (int)K, dweight);
    return launch_status();
  }
  const bool vec = K % kEPL == 0 && wide_rows(dy, ld_dy, dt) && wide_rows(x, ld_x, x_dt) && wide_rows(dresidual, ld_dresidual, x_dt) &&
                   wide_rows(dx, ld_dx, x_dt) && (!weight || aligned(weight, 16));
  const BackArgs a{dy,  x,          weight, dresidual, ld_dy, ld_x, ld_dresidual, weight_dt == MXQ_BF16,
                   eps, (int)rows,  (int)K, (int)back_rows_per_block(rows),       dx,   ld_dx, (float4*)workspace,
                   dweight ? (float*)workspace + rows * 4 : nullptr};
  if (dt == MXQ_BF16)
    return x_dt == MXQ_BF16 ? back_launch<uint16_t, uint16_t>(a, vec, dweight, stream)
                            : back_launch<uint16_t, uint32_t>(a, vec, dweight, stream);
  return x_dt == MXQ_BF16 ? back_launch<uint32_t, uint16_t>(a, vec, dweight, stream)
                          : back_launch<uint32_t, uint32_t>(a, vec, dweight, stream);
}

}  // extern "C"
