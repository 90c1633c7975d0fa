// norm.hip -- root-mean-square norm of rows with the residual's addition and FP8
// output in groups of 128, and its backward pass, on gfx950.
//
//   s = x + residual, rounded to the residual's type; y = s r w, r = 1 / sqrt(mean(s^2) + eps)
//
// The norm is that of s as it is stored, so that a backward pass, or a forward pass that is
// run again from the stored s, works on the same values.  Sums are in fp32.  A
// row whose sum of squares (or of g s) passes 2^128 is summed again with its values times 2^-80.
//
//   u = s r, g = dy w:  dx = r (g - u mean(g u)) + dresidual,  dw = sum over rows of dy u
//
// Memory bounds all of it: a row is read once, into as many lanes as hold it, and stays in registers between the sum and the
// results.  8192 x 8192 bf16 with a residual and y 101 us (605 MB, 6.0 TB/s, a plain copy's rate being 6.6); its gradients
// with the residual's 94 (537 MB, 5.7); 4096 x 8192 of an fp32 stream to groups along both 96, of which the second
// pass over the sum, for the columns, is 26.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "floats.h"

namespace {

using namespace mxq_host;
using namespace mxq_dev;

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
  float* stats;   // 1 / sqrt(mean(s^2) + eps) of each row
};

constexpr float kDown = 0x1p-80f;

template <bool kVec>
__device__ __forceinline__ f32x8 weight_at(const void* w, bool bf16, int c, int K) {
  if (!w) return f32x8{1, 1, 1, 1, 1, 1, 1, 1};
  return bf16 ? load_floats<uint16_t, kVec>(w, c, K) : load_floats<uint32_t, kVec>(w, c, K);
}

// Elements [c, c + 8) of s of a row.  kOnce: loads carry the non-temporal hint.
template <typename TX, typename TS, bool kVec, bool kOnce = false>
__device__ __forceinline__ f32x8 stream_at(const NormArgs& a, int64_t row, int c) {
  const f32x8 x = load_floats<TX, kVec, kOnce>((const TX*)a.x + row * a.ld_x, c, a.K);
  if (!a.residual) return x;
  const f32x8 r = load_floats<TS, kVec, kOnce>((const TS*)a.residual + row * a.ld_res, c, a.K);
  return widen<TS>(narrow<TS>(x + r));
}

// Sum over the kLanes lanes of a row, the same in each of them; several waves of a row meet in `part`, which one sum uses.
struct Meeting {
  float part[16];
};
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, Meeting& m) {
  if constexpr (kLanes <= 64) return lane_sum<kLanes>(v);
  constexpr int kWaves = kLanes / 64;
  v = lane_sum<64>(v);
  if ((threadIdx.x & 63) == 0) m.part[threadIdx.x / 64] = v;
  __syncthreads();
  const int lane16 = threadIdx.x & 15;
  return lane_sum<16>(lane16 < kWaves ? m.part[lane16] : 0.0f);
}

template <typename V>
__device__ __forceinline__ float add_squares(V s, float sum) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); i++) sum = fmaf(s[i], s[i], sum);
  return sum;
}

// r of a row from its sum of squares, or with f from that of its values times f.  f is a power of two, so r f is as exact as
// r, but for rows beyond 2^126, whose r f has 21 places or more.
__device__ __forceinline__ float inverse_root(float sum, float f, float eps, int K) {
  return f / sqrtf(sum / (float)K + eps * f * f);
}

constexpr int kThreads = 256;
// A workgroup: one row, or 256 lanes of those that are a wave's or less.
template <int kLanes>
constexpr int kNormThreads = kLanes > 64 ? kLanes : kThreads;

// A row in the registers of kLanes lanes, kChunks pieces of eight elements each.  kStream: outputs leave with the
// non-temporal hint; otherwise the inputs come with it, so that the caches keep the sum for the columns.
template <typename TX, typename TS, int kLanes, int kChunks, bool kVec, bool kStream>
__global__ __launch_bounds__(kNormThreads<kLanes>) void norm_kernel(NormArgs a) {
  keep_denormals();
  __shared__ Meeting meet[2];
  const int64_t row = (int64_t)blockIdx.x * (kNormThreads<kLanes> / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (row >= a.rows) return;   // a workgroup that meets at barriers has one row
  f32x8 s[kChunks];
  float sum = 0;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * kEPL;
    s[i] = stream_at<TX, TS, kVec, kVec && !kStream>(a, row, c);
  }
#pragma unroll
  for (int i = 0; i < kChunks; i++) sum = add_squares(s[i], sum);
  sum = row_sum<kLanes>(sum, meet[0]);
  float f = 1.0f;
  if (!(sum < __builtin_inff())) {   // the same for the whole row
    f = kDown;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kChunks; i++) sum = add_squares(s[i] * kDown, sum);
    sum = row_sum<kLanes>(sum, meet[1]);
  }
  const float r = inverse_root(sum, f, a.eps, a.K);
  if (a.stats && lane == 0) a.stats[row] = r;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * kEPL;
    const f32x8 y = s[i] * r * weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
    // two stores of fp32 each fill half of a line, and the hint sends the halves out one by one: 8192 x 8192 fp32
    // of such pieces 210 -> 256 us
    if (a.sum) store_floats<TS, kVec, kStream && sizeof(TS) == 2>((TS*)a.sum + row * a.ld_sum, c, a.K, s[i]);
    if (a.y) store_floats<TX, kVec, kStream && sizeof(TX) == 2>((TX*)a.y + row * a.ld_y, c, a.K, y);
    if (a.data) store_group<kVec, kStream>(a.data + row * a.ld_data, a.scale + row * a.scale_ld, c, a.K, y);
  }
}

// As norm_kernel, for fp32 rows at multiples of 16 bytes, with pieces of four elements: an instruction covers whole lines, and
// the hint sends out whole ones.  8192 x 8192 fp32 with a residual and y 194 us, in pieces of eight 208; groups along both
// of 4096 x 8192 99 for 111.  With a bf16 x beside an fp32 residual it is as fast either way.
template <typename TS, int kLanes, int kChunks, bool kStream>
__global__ __launch_bounds__(kNormThreads<kLanes>) void norm_four_kernel(NormArgs a) {
  keep_denormals();
  __shared__ Meeting meet[2];
  static_assert(kLanes >= 64, "32 lanes hold a group");
  const int64_t row = (int64_t)blockIdx.x * (kNormThreads<kLanes> / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (row >= a.rows) return;   // a workgroup that meets at barriers has one row
  f32x4 s[kChunks];
  float sum = 0;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * 4;
    s[i] = load_four<uint32_t, !kStream>((const float*)a.x + row * a.ld_x, c, a.K);
    if (a.residual) s[i] += load_four<TS, !kStream>((const TS*)a.residual + row * a.ld_res, c, a.K);
    if (a.residual && sizeof(TS) == 2) s[i] = widen4(narrow4(s[i]));
  }
#pragma unroll
  for (int i = 0; i < kChunks; i++) sum = add_squares(s[i], sum);
  sum = row_sum<kLanes>(sum, meet[0]);
  float f = 1.0f;
  if (!(sum < __builtin_inff())) {   // the same for the whole row
    f = kDown;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kChunks; i++) sum = add_squares(s[i] * kDown, sum);
    sum = row_sum<kLanes>(sum, meet[1]);
  }
  const float r = inverse_root(sum, f, a.eps, a.K);
  if (a.stats && lane == 0) a.stats[row] = r;
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    const int c = (i * kLanes + lane) * 4;
    f32x4 w{1, 1, 1, 1};
    if (a.weight) w = a.w_bf16 ? load_four<uint16_t>(a.weight, c, a.K) : load_four<uint32_t>(a.weight, c, a.K);
    const f32x4 y = s[i] * r * w;
    if (a.sum) store_four<TS, kStream>((TS*)a.sum + row * a.ld_sum, c, a.K, s[i]);
    if (a.y) store_four<uint32_t, kStream>((float*)a.y + row * a.ld_y, c, a.K, y);
    if (a.data) store_group_four<kStream>(a.data + row * a.ld_data, a.scale + row * a.scale_ld, c, a.K, y);
  }
}

// Rows that the registers do not hold: a workgroup walks the row, s is read again for the results.  2048 x 32768 bf16 with a
// residual and y 132 us (740 MB at 5.6 TB/s, of which 135 are s again); to groups along both of an fp32 stream 220, of which
// the columns are 63.
constexpr int kLong = 1024;

template <typename TX, typename TS, bool kVec>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormArgs a) {
  keep_denormals();
  __shared__ Meeting meet[2];
  const int64_t row = blockIdx.x;
  TS* const stored = a.sum ? (TS*)a.sum + row * a.ld_sum : nullptr;
  float sum = 0;
  for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kLong * kEPL) {
    const f32x8 s = stream_at<TX, TS, kVec>(a, row, (int)c);
    if (stored) store_floats<TS, kVec>(stored, (int)c, a.K, s);   // the residual may be stored in its own place
    sum = add_squares(s, sum);
  }
  const auto again = [&](int c) {
    return stored ? load_floats<TS, kVec>(stored, c, a.K) : stream_at<TX, TS, kVec>(a, row, c);
  };
  sum = row_sum<kLong>(sum, meet[0]);
  float f = 1.0f;
  if (!(sum < __builtin_inff())) {
    f = kDown;
    sum = 0;
    for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kLong * kEPL) sum = add_squares(again((int)c) * kDown, sum);
    sum = row_sum<kLong>(sum, meet[1]);
  }
  const float r = inverse_root(sum, f, a.eps, a.K);
  if (a.stats && threadIdx.x == 0) a.stats[row] = r;
  // all lanes of a group of 16 walk as far
  for (int64_t c0 = (threadIdx.x & ~15) * kEPL; c0 < a.K; c0 += kLong * kEPL) {
    const int c = (int)c0 + (threadIdx.x & 15) * kEPL;
    const f32x8 y = again(c) * r * weight_at<kVec>(a.weight, a.w_bf16, c, a.K);
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
    float root = 0;
    if (r < a.rows) {
      s = a.sum ? load_floats<TS, kVec, kVec && sizeof(TS) == 2>((const TS*)a.sum + r * a.ld_sum, c, a.K) : stream_at<TX, TS, kVec>(a, r, c);
      root = a.stats[r];
    }
    v[i] = narrow<uint32_t>(s * root * w);
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
  int rows, K, per_block;   // rows of a block, where rows are long
  void* dx;
  int64_t ld_dx;
  float2* stats;            // r and mean(g u) of each row, where rows are long
  float* part;              // [blocks, K] sums of dw; null: not wanted
};

// mean(g u) from the sum of g s, or with up = 2^80 from that of (g 2^-80) (s 2^-80).
__device__ __forceinline__ float mean_dot(float sum, float r, float up, int K) { return sum / (float)K * (r * up) * up; }

// What a lane reads of a row.
template <typename TY, typename TS, int kChunks>
struct BackRow {
  Chunk<TS> s[kChunks], dres[kChunks];
  Chunk<TY> dy[kChunks];
};

// A workgroup takes a row (as many as it has lanes for), and then every one as many rows further as the card works on at
// once, the next row on its way while this one is worked out; it keeps its part of dw in registers.  8192 x 8192 bf16 96.5
// us; 102.0 where each takes a run of neighbouring rows.  Loads with the non-temporal hint, stores without: so 99.9, plain
// loads 113, stores with it as well 102.5, loads without and stores with it 109, all in such runs.  Of fp32 a load takes half
// of each line and goes without it: 8192 x 8192 fp32 206.9 -> 197.9 us, bf16 beside an fp32 stream 178.9 -> 167.7.
template <typename TY, typename TS, int kLanes, int kChunks, bool kVec>
__global__ __launch_bounds__(kNormThreads<kLanes>) void back_kernel(BackArgs a) {
  keep_denormals();
  constexpr int kSlots = kNormThreads<kLanes> / kLanes, kWaves = kLanes / 64;
  __shared__ float2 meet[2][16];
  __shared__ float fold[kSlots > 1 ? kSlots : 1][kSlots > 1 ? kLanes * kEPL : 1];
  const int slot = kSlots > 1 ? threadIdx.x / kLanes : 0, lane = threadIdx.x % kLanes;
  const int64_t lo = (int64_t)blockIdx.x * kSlots, hi = a.rows, step = (int64_t)gridDim.x * kSlots;
  f32x8 w[kChunks], dw[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; i++) {
    w[i] = weight_at<kVec>(a.weight, a.w_bf16, (i * kLanes + lane) * kEPL, a.K);
    dw[i] = f32x8{};
  }
  using Row = BackRow<TY, TS, kChunks>;
  const auto load = [&](Row& v, int64_t row) {
    const int64_t r = min(row, (int64_t)a.rows - 1);
#pragma unroll
    for (int i = 0; i < kChunks; i++) {
      const int c = row < hi ? (i * kLanes + lane) * kEPL : a.K;
      v.s[i] = load_chunk<TS, kVec, sizeof(TS) == 2>((const TS*)a.s + r * a.ld_s, c, a.K);
      v.dy[i] = load_chunk<TY, kVec, sizeof(TY) == 2>((const TY*)a.dy + r * a.ld_dy, c, a.K);
      if (a.dres) v.dres[i] = load_chunk<TS, kVec, sizeof(TS) == 2>((const TS*)a.dres + r * a.ld_dres, c, a.K);
    }
  };
  int turn = 0;
  // (sum of squares, sum of g s) of a row from its lanes' parts, the same in all of them
  const auto meeting = [&](float2 v) {
    v = float2{lane_sum<kLanes == 16 ? 16 : 64>(v.x), lane_sum<kLanes == 16 ? 16 : 64>(v.y)};
    if constexpr (kLanes > 64) {   // the waves meet in one of two places in turn, so that one barrier is enough
      if ((threadIdx.x & 63) == 0) meet[turn][threadIdx.x / 64] = v;
      __syncthreads();
      const int lane16 = threadIdx.x & 15;
      v = lane16 < kWaves ? meet[turn][lane16] : float2{0, 0};
      v = float2{lane_sum<16>(v.x), lane_sum<16>(v.y)};
      turn ^= 1;
    }
    return v;
  };
  const auto work = [&](const Row& v, int64_t row) {
    float2 sum{0, 0};
#pragma unroll
    for (int i = 0; i < kChunks; i++) {
      const f32x8 s = widen<TS>(v.s[i]), g = widen<TY>(v.dy[i]) * w[i];
#pragma unroll
      for (int j = 0; j < kEPL; j++) sum.x = fmaf(s[j], s[j], sum.x), sum.y = fmaf(g[j], s[j], sum.y);
    }
    sum = meeting(sum);
    float f = 1.0f, up = 1.0f;
    if (!(sum.x < __builtin_inff()) || !(fabsf(sum.y) < __builtin_inff())) {   // the same for the whole row
      float2 low{0, 0};
#pragma unroll
      for (int i = 0; i < kChunks; i++) {
        const f32x8 s = widen<TS>(v.s[i]) * kDown, g = widen<TY>(v.dy[i]) * w[i] * kDown;
        low.x = add_squares(s, low.x);
        low.y += add8(g * s);
      }
      low = meeting(low);
      if (!(sum.x < __builtin_inff())) f = kDown, sum.x = low.x;
      if (!(fabsf(sum.y) < __builtin_inff())) up = 1.0f / kDown, sum.y = low.y;
    }
    const float r = inverse_root(sum.x, f, a.eps, a.K), m = mean_dot(sum.y, r, up, a.K);
#pragma unroll
    for (int i = 0; i < kChunks; i++) {
      const int c = row < hi ? (i * kLanes + lane) * kEPL : a.K;
      const f32x8 u = widen<TS>(v.s[i]) * r, dy = widen<TY>(v.dy[i]);
      f32x8 dx = a.dres ? widen<TS>(v.dres[i]) : f32x8{};
#pragma unroll
      for (int j = 0; j < kEPL; j++) {
        dx[j] = fmaf(fmaf(-u[j], m, dy[j] * w[i][j]), r, dx[j]);
        dw[i][j] = fmaf(dy[j], u[j], dw[i][j]);
      }
      store_floats<TS, kVec>((TS*)a.dx + row * a.ld_dx, c, a.K, dx);
    }
  };
  Row even;
  if constexpr (kChunks > 1) {   // two rows of these would not fit into the registers
    for (int64_t row = lo + slot; row - slot < hi; row += step) {
      load(even, row);
      work(even, row);
    }
  } else {
    Row odd;
    load(even, lo + slot);
    for (int64_t row = lo + slot; row - slot < hi; row += 2 * step) {
      load(odd, row + step);
      work(even, row);
      if (row - slot + step >= hi) break;
      load(even, row + 2 * step);
      work(odd, row + step);
    }
  }
  if (!a.part) return;   // the same for all
  float* const p = a.part + (int64_t)blockIdx.x * a.K;
  if constexpr (kSlots > 1) {
#pragma unroll
    for (int i = 0; i < kEPL; i++) fold[slot][lane * kEPL + i] = dw[0][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.K; c += kNormThreads<kLanes>) {   // K is at most kLanes * 8
      float sum = fold[0][c];
#pragma unroll
      for (int i = 1; i < kSlots; i++) sum += fold[i][c];
      p[c] = sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; i++) {
      const int c = (i * kLanes + lane) * kEPL;
#pragma unroll
      for (int j = 0; j < kEPL; j++)
        if (c + j < a.K) p[c + j] = dw[i][j];
    }
  }
}

// Rows that the registers do not hold: their statistics first, then dx and the parts of dw, a column a lane.  Both passes read
// dy and s: 2048 x 32768 bf16 185 us, 66 for the statistics, 112 for dx and 8 for dw.

template <typename TY, typename TS, bool kVec>
__global__ __launch_bounds__(kThreads) void back_stats_kernel(BackArgs a) {
  keep_denormals();
  __shared__ Meeting meet[4];
  const int64_t row = blockIdx.x;
  const TS* const s = (const TS*)a.s + row * a.ld_s;
  const TY* const dy = (const TY*)a.dy + row * a.ld_dy;
  float f = 1.0f, up = 1.0f, squares = 0, dots = 0;
  for (int k = 0; k < 4; k += 2) {   // in the second round with s and g times 2^-80
    const float down = k ? kDown : 1.0f;
    float sum = 0, dot = 0;
    for (int64_t c = threadIdx.x * kEPL; c < a.K; c += kThreads * kEPL) {
      const f32x8 v = load_floats<TS, kVec>(s, (int)c, a.K) * down;
      const f32x8 g = load_floats<TY, kVec>(dy, (int)c, a.K) * weight_at<kVec>(a.weight, a.w_bf16, (int)c, a.K) * down;
      sum = add_squares(v, sum);
      dot += add8(g * v);
    }
    sum = row_sum<kThreads>(sum, meet[k]);
    dot = row_sum<kThreads>(dot, meet[k + 1]);
    if (!k) {
      squares = sum, dots = dot;
      if (sum < __builtin_inff() && fabsf(dot) < __builtin_inff()) break;   // the same for all
    } else {
      if (!(squares < __builtin_inff())) f = kDown, squares = sum;
      if (!(fabsf(dots) < __builtin_inff())) up = 1.0f / kDown, dots = dot;
    }
  }
  const float r = inverse_root(squares, f, a.eps, a.K);
  if (threadIdx.x == 0) a.stats[row] = float2{r, mean_dot(dots, r, up, a.K)};
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
    const float2 t = a.stats[row];
    const f32x8 u = load_floats<TS, kVec>((const TS*)a.s + row * a.ld_s, c, a.K) * t.x;
    const f32x8 dy = load_floats<TY, kVec>((const TY*)a.dy + row * a.ld_dy, c, a.K);
    f32x8 dx = (dy * w - u * t.y) * t.x;
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

// dw: the blocks' parts added up in an order that their number fixes, 32 columns a workgroup, 32 of its lanes a column.
constexpr int kFoldThreads = 1024, kFoldColumns = 32, kFoldSlots = kFoldThreads / kFoldColumns;
__global__ __launch_bounds__(kFoldThreads) void back_weight_kernel(const float* part, int blocks, int K, int first,
                                                                   float* dw) {
  __shared__ float sums[kFoldSlots][kFoldColumns + 1];
  const int lane = threadIdx.x % kFoldColumns, slot = threadIdx.x / kFoldColumns;
  const int64_t c = first + (int64_t)blockIdx.x * kFoldColumns + lane;
  float sum = 0;
  if (c < K) {
#pragma unroll 4
    for (int b = slot; b < blocks; b += kFoldSlots) sum += part[(int64_t)b * K + c];
  }
  sums[slot][lane] = sum;
  __syncthreads();
  if (slot == 0 && c < K) {
#pragma unroll
    for (int i = 1; i < kFoldSlots; i++) sum += sums[i][lane];
    dw[c] = sum;
  }
}

// ---- host --------------------------------------------------------------------------------

// Squares below 2^-149 vanish; against this they are rounding.
constexpr float kLeastEps = 0x1p-126f;

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

template <typename TX, typename TS, int kLanes, int kChunks, bool kVec, bool kStream>
int launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int threads = kNormThreads<kLanes>, per = threads / kLanes;
  const auto kernel = [] {
    if constexpr (sizeof(TX) == 4 && kVec && kLanes >= 64) return norm_four_kernel<TS, kLanes, 2 * kChunks, kStream>;
    else return norm_kernel<TX, TS, kLanes, kChunks, kVec, kStream>;
  }();
  const int64_t step = rows_per_launch(kLanes);
  for (int64_t r = 0; r < a.rows; r += step) {
    const int64_t n = std::min<int64_t>(step, a.rows - r);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((n + per - 1) / per)), dim3(threads), 0, stream, from_row<TX, TS>(a, r, n));
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

// A row takes as many lanes as hold it in one piece each, up to a workgroup of 1024 with two: 8192 x 8192 bf16 with a
// residual and y 102 us, with 512 lanes and two pieces 105, with 256 and four 112.
template <typename TX, typename TS, bool kVec, bool kStream>
int norm_rows(const NormArgs& a, hipStream_t stream) {
  const int K = a.K;
  if (K <= 16 * 8) return launch_norm<TX, TS, 16, 1, kVec, kStream>(a, stream);
  if (K <= 64 * 8) return launch_norm<TX, TS, 64, 1, kVec, kStream>(a, stream);
  if (K <= 128 * 8) return launch_norm<TX, TS, 128, 1, kVec, kStream>(a, stream);
  if (K <= 256 * 8) return launch_norm<TX, TS, 256, 1, kVec, kStream>(a, stream);
  if (K <= 512 * 8) return launch_norm<TX, TS, 512, 1, kVec, kStream>(a, stream);
  if (K <= 640 * 8) return launch_norm<TX, TS, 640, 1, kVec, kStream>(a, stream);
  if (K <= 768 * 8) return launch_norm<TX, TS, 768, 1, kVec, kStream>(a, stream);
  if (K <= 1024 * 8) return launch_norm<TX, TS, 1024, 1, kVec, kStream>(a, stream);
  if (K <= 1024 * 16) return launch_norm<TX, TS, 1024, 2, kVec, kStream>(a, stream);
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
  // The hint for outputs that nothing reads at once: not for a sum that the columns come from.  8192 x 8192 bf16 106 ->
  // 102 us, 2048 x 8192 27.4 -> 22.9; rows and columns of 4096 x 8192 with the hint 92.8 -> 99.0.  There the inputs have it:
  // 99.3 -> 95.9, 8192 x 8192 bf16 122.9 -> 114.2.
  MXQ_TRY(!vec      ? (norm_rows<TX, TS, false, false>(a, stream))
          : columns ? (norm_rows<TX, TS, true, false>(a, stream))
                    : (norm_rows<TX, TS, true, true>(a, stream)));
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
  if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim || !(eps >= kLeastEps) || !(eps < __builtin_inff())) return MXQ_ERR_SHAPE;
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
                   col ? (float*)col->workspace : nullptr};
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

constexpr int kHeld = 1024 * 16;   // elements of a row that registers hold
// Lanes of a workgroup of the backward pass.
int back_threads(int64_t K) {
  for (int lanes : {64, 128, 256, 512, 640, 768})
    if (K <= lanes * 8) return lanes > 64 ? lanes : kThreads;
  return 1024;
}
// Rows of a workgroup: as many workgroups as have 1024 lanes for each CU (8192 x 8192 bf16 95.7 us; twice as many 104.8).  A
// workgroup of rows of up to 512 elements takes 4 or 16 at a time, so with few rows some have none and add zeros to dw.
int64_t back_rows_per_block(int64_t rows, int64_t K) {
  const int64_t fill = K > kHeld ? 256 : 256 * (1024 / back_threads(K));
  return std::max<int64_t>(K > kHeld ? 4 : 1, (rows + fill - 1) / fill);
}
int64_t back_blocks(int64_t rows, int64_t K) {
  const int64_t per = back_rows_per_block(rows, K);
  return (rows + per - 1) / per;
}

template <typename TY, typename TS, int kLanes, int kChunks, bool kVec>
int launch_back(const BackArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((back_kernel<TY, TS, kLanes, kChunks, kVec>), dim3((uint32_t)back_blocks(a.rows, a.K)),
                     dim3(kNormThreads<kLanes>), 0, stream, a);
  return launch_status();
}

template <typename TY, typename TS, bool kVec>
int back_rows(const BackArgs& a, hipStream_t stream) {
  const int K = a.K;
  if (K <= 16 * 8) return launch_back<TY, TS, 16, 1, kVec>(a, stream);
  if (K <= 64 * 8) return launch_back<TY, TS, 64, 1, kVec>(a, stream);
  if (K <= 128 * 8) return launch_back<TY, TS, 128, 1, kVec>(a, stream);
  if (K <= 256 * 8) return launch_back<TY, TS, 256, 1, kVec>(a, stream);
  if (K <= 512 * 8) return launch_back<TY, TS, 512, 1, kVec>(a, stream);
  if (K <= 640 * 8) return launch_back<TY, TS, 640, 1, kVec>(a, stream);
  if (K <= 768 * 8) return launch_back<TY, TS, 768, 1, kVec>(a, stream);
  if (K <= 1024 * 8) return launch_back<TY, TS, 1024, 1, kVec>(a, stream);
  if (K <= kHeld) return launch_back<TY, TS, 1024, 2, kVec>(a, stream);
  const int64_t step = rows_per_launch(kThreads);
  for (int64_t r = 0; r < a.rows; r += step) {
    BackArgs b = a;
    b.s = (const TS*)a.s + r * a.ld_s;
    b.dy = (const TY*)a.dy + r * a.ld_dy;
    b.stats = a.stats + r;
    hipLaunchKernelGGL((back_stats_kernel<TY, TS, kVec>), dim3((uint32_t)std::min<int64_t>(step, a.rows - r)),
                       dim3(kThreads), 0, stream, b);
    MXQ_TRY(launch_status());
  }
  const uint32_t strips = (uint32_t)((a.K + (int64_t)kThreads * kEPL - 1) / (kThreads * kEPL));
  hipLaunchKernelGGL((back_rows_kernel<TY, TS, kVec>), dim3(strips, (uint32_t)back_blocks(a.rows, a.K)), dim3(kThreads), 0,
                     stream, a);
  return launch_status();
}

int fold_weight(const float* part, int64_t blocks, int64_t K, float* dw, hipStream_t stream) {
  const int64_t step = rows_per_launch(kFoldThreads) * kFoldColumns;
  for (int64_t c = 0; c < K; c += step) {
    const int64_t n = std::min(step, K - c);
    hipLaunchKernelGGL(back_weight_kernel, dim3((uint32_t)((n + kFoldColumns - 1) / kFoldColumns)), dim3(kFoldThreads), 0,
                       stream, part, (int)blocks, (int)K, (int)c, dw);
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

template <typename TY, typename TS>
int back_launch(const BackArgs& a, bool vec, hipStream_t stream) {
  return vec ? back_rows<TY, TS, true>(a, stream) : back_rows<TY, TS, false>(a, stream);
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

// A float a row is in use; callers are told eight bytes.
int64_t mxq_rms_norm_fp8_group128_row_col_workspace(int64_t rows) {
  return rows < 1 || rows > kMaxDim ? 0 : rows * 8;
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
  return (K > kHeld ? rows * (int64_t)sizeof(float2) : 0) + back_blocks(rows, K) * K * 4;
}

int mxq_rms_norm_backward(const void* dy, int64_t ld_dy, mxq_dtype dt, const void* x, int64_t ld_x, mxq_dtype x_dt,
                          const void* weight, mxq_dtype weight_dt, float eps, const void* dresidual,
                          int64_t ld_dresidual, int64_t rows, int64_t K, void* dx, int64_t ld_dx, float* dweight,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!is_float(dt) || !is_float(x_dt) || (weight && !is_float(weight_dt))) return MXQ_ERR_DTYPE;
  if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim || !(eps >= kLeastEps) || !(eps < __builtin_inff())) return MXQ_ERR_SHAPE;
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
    return fold_weight(nullptr, 0, K, dweight, stream);
  }
  const bool vec = K % kEPL == 0 && wide_rows(dy, ld_dy, dt) && wide_rows(x, ld_x, x_dt) && wide_rows(dresidual, ld_dresidual, x_dt) &&
                   wide_rows(dx, ld_dx, x_dt) && (!weight || aligned(weight, 16));
  float2* const stats = K > kHeld ? (float2*)workspace : nullptr;
  float* const part = (float*)workspace + (K > kHeld ? rows * 2 : 0);
  const BackArgs a{dy,  x,         weight, dresidual, ld_dy, ld_x, ld_dresidual, weight_dt == MXQ_BF16,
                   eps, (int)rows, (int)K, (int)back_rows_per_block(rows, K),    dx,   ld_dx, stats,
                   dweight ? part : nullptr};
  MXQ_TRY(dt == MXQ_BF16 ? (x_dt == MXQ_BF16 ? back_launch<uint16_t, uint16_t>(a, vec, stream)
                                             : back_launch<uint16_t, uint32_t>(a, vec, stream))
                         : (x_dt == MXQ_BF16 ? back_launch<uint32_t, uint16_t>(a, vec, stream)
                                             : back_launch<uint32_t, uint32_t>(a, vec, stream)));
  return dweight ? fold_weight(part, back_blocks(rows, K), K, dweight, stream) : MXQ_OK;
}

}  // extern "C"
