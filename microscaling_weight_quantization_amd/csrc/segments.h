// Rows sorted by expert, as the kernels see them: expert e owns rows
// [offsets[e], offsets[e + 1]); the rows from offsets[n] on, and those before
// offsets[0], belong to no expert.  offsets is device memory that the host does not read, so each
// workgroup finds its own segment: a wave takes 64 experts at a time, turns
// their row counts into tile counts and adds them up across its lanes.
//
// offsets are clamped to [0, rows] as they are read, and where they fall they
// count as the largest so far.  So segments never overlap, their tiles number at
// most rows / tile + n, and no value of theirs takes an access out of a matrix.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq_dev {

struct Segment {
  int expert;   // n: the rows of no expert
  int tile;     // index of the tile within the segment
  int lo, hi;   // the segment's rows
  int first;    // tiles of all earlier segments
};

// Inclusive sum, and largest value so far, over the lanes of a wave.
__device__ __forceinline__ int wave_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int wave_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v = max(v, o);
  }
  return v;
}

// Rows [lo, hi) of expert base + lane (of none from n on: empty).  `end` is
// where the experts before `base` end, and is moved past these 64.
struct Rows {
  int lo, hi;
};
__device__ __forceinline__ Rows rows_of(const int32_t* offsets, int n, int rows, int base, int& end) {
  const int e = base + (int)(threadIdx.x & 63);
  const int first = min(max(offsets[min(e, n)], 0), rows), last = min(max(offsets[min(e + 1, n)], 0), rows);
  Rows r{first, last};
  if (__any(last < first || first < end)) {   // they do not rise everywhere
    const int top = max(end, wave_max(max(first, last)));
    const int before = __shfl_up(top, 1);
    r = Rows{max(first, (threadIdx.x & 63) ? before : end), top};
  }
  end = __shfl(r.hi, 63);
  return r;
}

// Segment of tile number `id` when every segment is cut into tiles of kTile
// rows; ids past the experts' tiles count through the rows of no expert, those
// behind the experts' rows first.  There are at most rows / kTile + n + 2 tiles.
// All lanes of a wave call it with the same id and get the same answer.
template <int kTile>
__device__ __forceinline__ Segment find_tile(const int32_t* offsets, int n, int rows, int id) {
  int first = 0, end = 0;
  for (int base = 0; base < n; base += 64) {
    const Rows r = rows_of(offsets, n, rows, base, end);
    const int tiles = (r.hi - r.lo + kTile - 1) / kTile;
    const int sum = wave_sum(tiles);
    const unsigned long long found = __ballot(id < first + sum);
    if (found) {
      const int at = __builtin_ctzll(found);
      const int before = first + __shfl(sum - tiles, at);
      return Segment{base + at, id - before, __shfl(r.lo, at), __shfl(r.hi, at), before};
    }
    first += __shfl(sum, 63);
  }
  const int behind = (rows - end + kTile - 1) / kTile;
  if (id < first + behind) return Segment{n, id - first, end, rows, first};
  return Segment{n, id - first - behind, 0, min(max(offsets[0], 0), rows), first};
}

// Segment `expert` < n and the number of tiles before it.
template <int kTile>
__device__ __forceinline__ Segment find_expert(const int32_t* offsets, int n, int rows, int expert) {
  int first = 0, end = 0;
  for (int base = 0;; base += 64) {
    const Rows r = rows_of(offsets, n, rows, base, end);
    const int tiles = (r.hi - r.lo + kTile - 1) / kTile;
    const int sum = wave_sum(tiles), at = expert - base;
    if (at < 64) return Segment{expert, 0, __shfl(r.lo, at), __shfl(r.hi, at), first + __shfl(sum - tiles, at)};
    first += __shfl(sum, 63);
  }
}

}  // namespace mxq_dev
