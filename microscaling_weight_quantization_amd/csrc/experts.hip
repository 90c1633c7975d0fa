// experts.hip -- token slots sorted by expert, rows brought into that order and
// back, on gfx950.
//
// A slot is one (token, choice) pair, slot = token * top_k + choice.  Sorting is
// a stable counting sort: slots of one expert keep their order, so the result is
// the same on every run.  Slots whose expert id is out of range are dropped: they
// sort behind all others and are marked by the bitwise complement, which is
// negative, in both directions (slots[] and position[]).
//
// The row kernels are bound by the bytes moved: sort and rows into order, 605 MB
// with each row of x read once, take 155 us (a token's row passes the L2s for nearly
// each of its 8 places: 510 MB read, largely from the last-level cache, and 537
// written), 672 MB of rows back and their gradients 120 us (the second kernel finds
// rows of the first in the last-level cache).  A few tokens' routing is two launches
// and their calls on the host, 19.6 us.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "checks.h"
#include "fastdiv.h"

namespace {

using namespace mxq_host;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---- the sort ----------------------------------------------------------------------------
// A workgroup of 16 waves takes kSlots slots, each wave a run of consecutive
// ones.  Every wave counts its run's experts in LDS; the counts are summed over
// waves (and, where there are several workgroups, over the counts that a first
// launch left in the workspace: a few of those each workgroup adds up itself, many a
// launch in between, so that the work stays in proportion to the slots); then
// each wave walks its run 64 slots at a time: the lanes that hold the same expert
// find each other with one ballot for each bit of the id, and a lane's place is the
// expert's next free one plus the number of such lanes below it.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortSlots = 2048;          // slots per workgroup where there are several
constexpr int kSortAlone = 8192;          // as many as one workgroup takes without a second launch
// Counts that each workgroup adds up itself.  All of them together read their number
// times the workgroups, so more are added up once: 2^17 slots for 128 experts (8256
// counts) take 15 us against 18, 2^18 (16512) 18 against 18, 2^20 for 512 experts
// (262656) 101 against 29, 2^22 1390 against 81.
constexpr int64_t kSortDirect = 16384;

__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t ld, MxqDivisor top_k, int slot, int n) {
  const uint32_t t = mxq_quot((uint32_t)slot, top_k);
  const int e = ids[(int64_t)t * ld + (slot - (int)t * (int)top_k.d)];
  return (uint32_t)e < (uint32_t)n ? e : n;
}

struct SortArgs {
  const int32_t* ids;
  int64_t ld;
  MxqDivisor top_k, per_group;   // per_group: n + 1
  int total, n, per_wave;        // slots in all, experts, slots per wave
  int32_t* offsets;
  int32_t* slots;
  int32_t* position;
  int32_t* counts;          // [workgroups][n + 1]; null: one workgroup
  const int32_t* totals;    // [n + 1]: counts are summed over the workgroups before; null: they are not
};

__global__ __launch_bounds__(kSortThreads) void count_kernel(SortArgs a) {
  extern __shared__ int hist[];
  for (int e = threadIdx.x; e <= a.n; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int begin = blockIdx.x * kSortSlots, end = min(begin + kSortSlots, a.total);
  for (int s = begin + (int)threadIdx.x; s < end; s += kSortThreads)
    atomicAdd(&hist[expert_of(a.ids, a.ld, a.top_k, s, a.n)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.n; e += kSortThreads) a.counts[(int64_t)blockIdx.x * (a.n + 1) + e] = hist[e];
}

// Turns each workgroup's counts into the sums over those before it, and leaves the
// sums over all behind them.  One expert a lane; each wave has a run of workgroups,
// read twice.
__global__ __launch_bounds__(kSortThreads) void sums_kernel(int32_t* counts, int groups, int n1) {
  __shared__ int part[kSortWaves][64];
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64, e = blockIdx.x * 64 + lane;
  const int per = (groups + kSortWaves - 1) / kSortWaves;
  const int begin = min(wave * per, groups), end = min(begin + per, groups);
  int32_t* const column = counts + min(e, n1 - 1);
  int sum = 0;
#pragma unroll 8
  for (int g = begin; g < end; g++) sum += column[(int64_t)g * n1];
  part[wave][lane] = sum;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSortWaves; w++) {
    before += w < wave ? part[w][lane] : 0;
    all += part[w][lane];
  }
  if (e >= n1) return;
  if (wave == 0) column[(int64_t)groups * n1] = all;
  for (int g0 = begin; g0 < end; g0 += kAhead) {
    int c[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) c[i] = column[(int64_t)min(g0 + i, end - 1) * n1];
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      if (g0 + i < end) column[(int64_t)(g0 + i) * n1] = before;
      before += c[i];
    }
  }
}

// Exclusive sum over the workgroup of one value a lane.
__device__ __forceinline__ int block_exclusive(int v, int* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) scratch[wave] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; w++) before += scratch[w];
  __syncthreads();
  return before + s - v;
}

__global__ __launch_bounds__(kSortThreads) void sort_kernel(SortArgs a) {
  extern __shared__ int lds[];              // [waves][n + 1] counts, then next free places; two more rows of sums
  __shared__ int scratch[kSortWaves];
  const int n1 = a.n + 1, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  for (int i = threadIdx.x; i < kSortWaves * n1; i += kSortThreads) lds[i] = 0;
  __syncthreads();
  int* const mine = lds + wave * n1;
  const int begin = min((blockIdx.x * kSortWaves + wave) * a.per_wave, a.total);
  const int end = min(begin + a.per_wave, a.total);
  for (int s = begin + lane; s < end; s += 64) atomicAdd(&mine[expert_of(a.ids, a.ld, a.top_k, s, a.n)], 1);
  __syncthreads();
  // the sums over all workgroups, and over those before this one, from the counts
  // that the first launch left: all lanes at once, added up in LDS
  int* const all = lds + kSortWaves * n1;
  int* const before = all + n1;
  if (a.totals) {
    for (int e = threadIdx.x; e < n1; e += kSortThreads) {
      all[e] = a.totals[e];
      before[e] = a.counts[(int64_t)blockIdx.x * n1 + e];
    }
    __syncthreads();
  } else if (a.counts) {
    for (int e = threadIdx.x; e < 2 * n1; e += kSortThreads) all[e] = 0;
    __syncthreads();
    const int n = (int)gridDim.x * n1, mark = (int)blockIdx.x * n1;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
      const int c = a.counts[i], e = i - (int)mxq_quot((uint32_t)i, a.per_group) * n1;
      if (c) {
        atomicAdd(&all[e], c);
        if (i < mark) atomicAdd(&before[e], c);
      }
    }
    __syncthreads();
  }
  // one expert a lane
  {
    static_assert(kMaxExperts < kSortThreads, "a lane for each expert and one for the dropped slots");
    const int e = threadIdx.x;
    int total = 0;
    if (e < n1) {
      if (a.counts) {
        total = all[e];
      } else {
        for (int w = 0; w < kSortWaves; w++) total += lds[w * n1 + e];
      }
    }
    const int start = block_exclusive(total, scratch);
    if (e < n1) {
      if (blockIdx.x == 0) a.offsets[e] = start;   // offsets[n]: where the dropped ones begin
      int next = start + (a.counts ? before[e] : 0);
      for (int w = 0; w < kSortWaves; w++) {
        const int c = lds[w * n1 + e];
        lds[w * n1 + e] = next;
        next += c;
      }
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.n | 1);
  for (int s0 = begin; s0 < end; s0 += 64) {
    const int s = s0 + lane;
    const bool in = s < end;
    const int e = in ? expert_of(a.ids, a.ld, a.top_k, s, a.n) : 0;
    unsigned long long same = __ballot(in);
    for (int b = 0; b < bits; b++) {
      const unsigned long long one = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? one : ~one;
    }
    if (in) {
      const unsigned long long below = same & ((1ull << lane) - 1);
      const int place = mine[e] + __popcll(below);
      const bool dropped = e == a.n;
      a.slots[place] = dropped ? ~s : s;
      a.position[s] = dropped ? ~place : place;
      // the first lane of each expert takes the places after all have read the old count
      __builtin_amdgcn_wave_barrier();
      if (below == 0) mine[e] = place + __popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Results of more than this leave with the non-temporal hint: the L2s together
// hold 32 MiB, and without it lines that nobody reads again push others out.
// Sorting 131072 slots and bringing their rows of 2048 bf16
// into order takes 183 us without and 156 with it; 8192 tokens of 6 such rows back
// and their gradients 139 and 121.  Smaller results are left where the
// next kernel finds them.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

// ---- rows into sorted order and back ----------------------------------------------------------
constexpr int kRowThreads = 256, kEPL = 8;

template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  typedef u32x4 Raw;
  static __device__ __forceinline__ f32x8 widen(Raw r) {
    return __builtin_convertvector(__builtin_bit_cast(bf16x8, r), f32x8);
  }
  static __device__ __forceinline__ Raw narrow(f32x8 v) {
    return __builtin_bit_cast(Raw, __builtin_convertvector(v, bf16x8));
  }
};
template <>
struct Eight<float> {
  typedef f32x8 Raw;
  static __device__ __forceinline__ f32x8 widen(Raw r) { return r; }
  static __device__ __forceinline__ Raw narrow(f32x8 v) { return v; }
};

// Elements [c, c + 8) of a row of H; those from H on are 0 and are not written.
template <typename T, bool kVec>
__device__ __forceinline__ typename Eight<T>::Raw load8(const T* row, int c, int H) {
  typename Eight<T>::Raw v{};
  if (kVec) {
    if (c < H) {
      typedef u32x4 A __attribute__((may_alias));
      if constexpr (sizeof(T) == 2) {
        v = *reinterpret_cast<const A*>(row + c);
      } else {
        const u32x4 lo = *reinterpret_cast<const A*>(row + c), hi = *reinterpret_cast<const A*>(row + c + 4);
        v = __builtin_bit_cast(f32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < H) {
        if constexpr (sizeof(T) == 2) v[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        else v[i] = row[c + i];
      }
  }
  return v;
}
template <typename T, bool kVec, bool kStream = false>
__device__ __forceinline__ void store8(T* row, int c, int H, typename Eight<T>::Raw v) {
  if (kVec) {
    if (c < H) {
      typedef u32x4 A __attribute__((may_alias));
      auto put = [](T* p, u32x4 w) {
        if constexpr (kStream) __builtin_nontemporal_store(w, reinterpret_cast<A*>(p));
        else *reinterpret_cast<A*>(p) = w;
      };
      if constexpr (sizeof(T) == 2) {
        put(row + c, v);
      } else {
        put(row + c, __builtin_bit_cast(u32x4, __builtin_shufflevector(v, v, 0, 1, 2, 3)));
        put(row + c + 4, __builtin_bit_cast(u32x4, __builtin_shufflevector(v, v, 4, 5, 6, 7)));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEPL; i++)
      if (c + i < H) {
        if constexpr (sizeof(T) == 2) row[c + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        else row[c + i] = v[i];
      }
  }
}

template <typename T, bool kVec, bool kStream>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const T* x, int64_t ld_x, int x_rows,
                                                               const int32_t* slots, MxqDivisor top_k, int H,
                                                               T* out, int64_t ld_out, MxqDivisor chunks,
                                                               uint32_t total) {
  const uint32_t g = blockIdx.x * kRowThreads + threadIdx.x;
  if (g >= total) return;
  const uint32_t r = mxq_quot(g, chunks);
  const int c = (int)(g - r * chunks.d) * kEPL;
  const int slot = slots[r];
  const int from = slot < 0 ? -1 : (int)mxq_quot((uint32_t)slot, top_k);
  const bool some = from >= 0 && from < x_rows;
  store8<T, kVec, kStream>(out + (int64_t)r * ld_out, c, H, load8<T, kVec>(x + (some ? from : 0) * ld_x, some ? c : H, H));
}

// y[t] = sum over the token's slots of weight * row.  One lane per 8 columns of a token.
constexpr int kAhead = 4;   // rows in flight per lane

template <typename T, bool kVec, bool kStream>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const T* rows, int64_t ld_rows, int n_rows,
                                                              const int32_t* position, const float* weights, int top_k,
                                                              int H, T* y, int64_t ld_y, MxqDivisor chunks,
                                                              uint32_t total) {
  const uint32_t g = blockIdx.x * kRowThreads + threadIdx.x;
  if (g >= total) return;
  const uint32_t t = mxq_quot(g, chunks);
  const int c = (int)(g - t * chunks.d) * kEPL;
  const int64_t slot0 = (int64_t)t * top_k;
  f32x8 sum{};
  for (int j0 = 0; j0 < top_k; j0 += kAhead) {
    typename Eight<T>::Raw v[kAhead];
    float w[kAhead];
    bool some[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const bool in = j0 + j < top_k;
      const int p = in ? position[slot0 + j0 + j] : -1;
      some[j] = p >= 0 && p < n_rows;
      w[j] = some[j] ? (weights ? weights[slot0 + j0 + j] : 1.0f) : 0.0f;
      v[j] = load8<T, kVec>(rows + (some[j] ? p : 0) * ld_rows, some[j] ? c : H, H);
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      if (some[j]) sum += Eight<T>::widen(v[j]) * w[j];
  }
  store8<T, kVec, kStream>(y + (int64_t)t * ld_y, c, H, Eight<T>::narrow(sum));
}

// Gradients of combine: drows[p] = weight * dy[t], dweights[slot] = <dy[t], rows[p]>.
// One workgroup per token, so dy comes from memory once for all of the token's
// slots (from the caches for those after the first) and the dot products are summed
// in a fixed order.  Its 256 lanes take 2048 columns at a time; of narrower rows some
// lanes have none.
template <typename T, bool kVec, bool kStream>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(const T* dy, int64_t ld_dy, const T* rows,
                                                                       int64_t ld_rows, int n_rows,
                                                                       const int32_t* position, const float* weights,
                                                                       int top_k, int H, T* drows, int64_t ld_drows,
                                                                       float* dweights) {
  __shared__ float part[kRowThreads / 64];
  const int64_t slot0 = (int64_t)blockIdx.x * top_k;
  const T* const g = dy + (int64_t)blockIdx.x * ld_dy;
  for (int j = 0; j < top_k; j++) {
    const int p = position[slot0 + j];
    const bool kept = p >= 0;
    const int at = kept ? p : ~p;
    const bool some = at < n_rows;
    const float w = kept ? (weights ? weights[slot0 + j] : 1.0f) : 0.0f;
    float dot = 0.0f;
    if (some) {
      for (int c = threadIdx.x * kEPL; c < H; c += kRowThreads * kEPL) {
        f32x8 d{};
        if (kept) {
          d = Eight<T>::widen(load8<T, kVec>(g, c, H));
          const f32x8 v = Eight<T>::widen(load8<T, kVec>(rows + at * ld_rows, c, H));
#pragma unroll
          for (int i = 0; i < kEPL; i++) dot += d[i] * v[i];
          d *= w;
        }
        store8<T, kVec, kStream>(drows + at * ld_drows, c, H, Eight<T>::narrow(d));
      }
    }
    if (dweights) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) dot += __shfl_xor(dot, m);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = dot;
      __syncthreads();
      if (threadIdx.x == 0) dweights[slot0 + j] = (part[0] + part[1]) + (part[2] + part[3]);
      __syncthreads();
    }
  }
}

bool vector_rows(const void* p, int64_t ld, mxq_dtype dt) {
  return aligned(p, 16) && ld % (16 / (int64_t)size_of(dt)) == 0;
}

// Lanes of a row, 8 columns each.
int64_t lanes_of(int64_t H) { return (H + kEPL - 1) / kEPL; }
dim3 grid_for(int64_t rows, int64_t H) { return dim3((uint32_t)((rows * lanes_of(H) + kRowThreads - 1) / kRowThreads)); }

}  // namespace

extern "C" {

int64_t mxq_sort_experts_workspace(int64_t n_tokens, int64_t top_k, int64_t n_experts) {
  if (n_tokens < 1 || top_k < 1 || n_experts < 1 || top_k > kMaxDim || n_tokens > kMaxDim / top_k) return 0;
  const int64_t total = n_tokens * top_k;
  if (total <= kSortAlone) return 0;
  const int64_t counts = (total + kSortSlots - 1) / kSortSlots * (n_experts + 1);
  return (counts + (counts > kSortDirect ? n_experts + 1 : 0)) * 4;
}

int mxq_sort_experts(const int32_t* ids, int64_t ld_ids, int64_t n_tokens, int64_t top_k, int64_t n_experts,
                     int32_t* offsets, int32_t* slots, int32_t* position, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  if (n_tokens < 0 || top_k < 1 || n_experts < 1 || n_experts > kMaxExperts || top_k > kMaxDim ||
      n_tokens > kMaxDim / top_k || ld_ids < top_k)
    return MXQ_ERR_SHAPE;
  const int64_t total = n_tokens * top_k, need = mxq_sort_experts_workspace(n_tokens, top_k, n_experts);
  if (!offsets || (total && (!ids || !slots || !position)) || (need && !workspace)) return MXQ_ERR_NULL;
  if (workspace_bytes < need) return MXQ_ERR_SHAPE;
  const Range ri = matrix_range(ids, n_tokens, top_k, ld_ids, 4), ro = matrix_range(offsets, 1, n_experts + 1, n_experts + 1, 4),
              rs = matrix_range(slots, 1, total, total, 4), rp = matrix_range(position, 1, total, total, 4),
              rw = matrix_range(workspace, 1, need, need, 1);
  if (!all_ok({ri, ro, rs, rp, rw}) || !aligned(ids, 4) || !aligned(offsets, 4) || !aligned(slots, 4) ||
      !aligned(position, 4) || !aligned(workspace, 4))
    return MXQ_ERR_SHAPE;
  if (!disjoint({ro, rs, rp, rw}, {ri})) return MXQ_ERR_ALIAS;
  const bool alone = need == 0;
  const int blocks = alone ? 1 : (int)((total + kSortSlots - 1) / kSortSlots);
  const int64_t counts = blocks * (n_experts + 1);
  const int per_wave = alone ? (int)((total + kSortThreads - 1) / kSortThreads * 64) : kSortSlots / kSortWaves;
  const SortArgs a{ids,      ld_ids, mxq_divisor((uint32_t)top_k), mxq_divisor((uint32_t)n_experts + 1), (int)total,
                   (int)n_experts, per_wave, offsets, slots, position, alone ? nullptr : (int32_t*)workspace,
                   !alone && counts > kSortDirect ? (int32_t*)workspace + counts : nullptr};
  const uint32_t hist = (uint32_t)(n_experts + 1) * 4;
  if (!alone) {
    hipLaunchKernelGGL(count_kernel, dim3(blocks), dim3(kSortThreads), hist, stream, a);
    int st = launch_status();
    if (st != MXQ_OK) return st;
    if (a.totals) {
      hipLaunchKernelGGL(sums_kernel, dim3((uint32_t)(n_experts + 64) / 64), dim3(kSortThreads), 0, stream, a.counts, blocks,
                         (int)n_experts + 1);
      st = launch_status();
      if (st != MXQ_OK) return st;
    }
  }
  hipLaunchKernelGGL(sort_kernel, dim3(blocks), dim3(kSortThreads), hist * (kSortWaves + 2), stream, a);
  return launch_status();
}

int mxq_dispatch_rows(const void* x, int64_t ld_x, int64_t x_rows, const int32_t* slots, int64_t rows, int64_t top_k,
                      int64_t H, mxq_dtype dt, void* out, int64_t ld_out, hipStream_t stream) {
  if (!is_float(dt)) return MXQ_ERR_DTYPE;
  if (rows < 0 || H < 0 || x_rows < 0 || top_k < 1 || rows > kMaxDim || H > kMaxDim || x_rows > kMaxDim || top_k > kMaxDim)
    return MXQ_ERR_SHAPE;
  if (rows == 0 || H == 0) return MXQ_OK;
  if ((!x && x_rows > 0) || !slots || !out) return MXQ_ERR_NULL;
  if (ld_x < H || ld_out < H) return MXQ_ERR_SHAPE;
  const Range rx = matrix_range(x, x_rows, H, ld_x, size_of(dt)), rs = matrix_range(slots, 1, rows, rows, 4),
              ro = matrix_range(out, rows, H, ld_out, size_of(dt));
  if (!all_ok({rx, rs, ro}) || !aligned(slots, 4) || !aligned(x, size_of(dt)) || !aligned(out, size_of(dt)))
    return MXQ_ERR_SHAPE;
  if (!disjoint({ro}, {rx, rs})) return MXQ_ERR_ALIAS;
  const bool vec = vector_rows(x, ld_x, dt) && vector_rows(out, ld_out, dt) && H % kEPL == 0;
  const dim3 block(kRowThreads);
  const MxqDivisor k = mxq_divisor((uint32_t)top_k), chunks = mxq_divisor((uint32_t)lanes_of(H));
  const bool stream_out = rows * H * (int64_t)size_of(dt) > kStreamBytes;
#define MXQ_DISPATCH(T, V, S)                                                                                          \
  hipLaunchKernelGGL((dispatch_kernel<T, V, S>), grid, block, 0, stream, (const T*)x, ld_x, (int)x_rows, slots + r, k, \
                     (int)H, (T*)out + r * ld_out, ld_out, chunks, (uint32_t)(n * lanes_of(H)))
  const int64_t step = rows_per_launch(lanes_of(H));
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = std::min(step, rows - r);
    const dim3 grid = grid_for(n, H);
    if (dt == MXQ_BF16) {
      if (!vec) MXQ_DISPATCH(uint16_t, false, false);
      else if (stream_out) MXQ_DISPATCH(uint16_t, true, true);
      else MXQ_DISPATCH(uint16_t, true, false);
    } else {
      if (!vec) MXQ_DISPATCH(float, false, false);
      else if (stream_out) MXQ_DISPATCH(float, true, true);
      else MXQ_DISPATCH(float, true, false);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_DISPATCH
  return MXQ_OK;
}

int mxq_combine_rows(const void* rows, int64_t ld_rows, int64_t n_rows, const int32_t* position, const float* weights,
                     int64_t n_tokens, int64_t top_k, int64_t H, mxq_dtype dt, void* y, int64_t ld_y,
                     hipStream_t stream) {
  if (!is_float(dt)) return MXQ_ERR_DTYPE;
  if (n_rows < 0 || n_tokens < 0 || H < 0 || top_k < 1 || n_rows > kMaxDim || H > kMaxDim || top_k > kMaxDim ||
      n_tokens > kMaxDim / top_k)
    return MXQ_ERR_SHAPE;
  if (n_tokens == 0 || H == 0) return MXQ_OK;
  if ((!rows && n_rows > 0) || !position || !y) return MXQ_ERR_NULL;
  if (ld_rows < H || ld_y < H) return MXQ_ERR_SHAPE;
  const int64_t slots = n_tokens * top_k;
  const Range rr = matrix_range(rows, n_rows, H, ld_rows, size_of(dt)), rp = matrix_range(position, 1, slots, slots, 4),
              rw = matrix_range(weights, 1, weights ? slots : 0, slots, 4),
              ry = matrix_range(y, n_tokens, H, ld_y, size_of(dt));
  if (!all_ok({rr, rp, rw, ry}) || !aligned(position, 4) || !aligned(weights, 4) || !aligned(rows, size_of(dt)) ||
      !aligned(y, size_of(dt)))
    return MXQ_ERR_SHAPE;
  if (!disjoint({ry}, {rr, rp, rw})) return MXQ_ERR_ALIAS;
  const bool vec = vector_rows(rows, ld_rows, dt) && vector_rows(y, ld_y, dt) && H % kEPL == 0;
  const dim3 block(kRowThreads);
  const MxqDivisor chunks = mxq_divisor((uint32_t)lanes_of(H));
  const bool stream_out = n_tokens * H * (int64_t)size_of(dt) > kStreamBytes;
#define MXQ_COMBINE(T, V, S)                                                                                          \
  hipLaunchKernelGGL((combine_kernel<T, V, S>), grid, block, 0, stream, (const T*)rows, ld_rows, (int)n_rows,         \
                     position + t * top_k, weights ? weights + t * top_k : weights, (int)top_k, (int)H,               \
                     (T*)y + t * ld_y, ld_y, chunks, (uint32_t)(n * lanes_of(H)))
  const int64_t step = rows_per_launch(lanes_of(H));
  for (int64_t t = 0; t < n_tokens; t += step) {
    const int64_t n = std::min(step, n_tokens - t);
    const dim3 grid = grid_for(n, H);
    if (dt == MXQ_BF16) {
      if (!vec) MXQ_COMBINE(uint16_t, false, false);
      else if (stream_out) MXQ_COMBINE(uint16_t, true, true);
      else MXQ_COMBINE(uint16_t, true, false);
    } else {
      if (!vec) MXQ_COMBINE(float, false, false);
      else if (stream_out) MXQ_COMBINE(float, true, true);
      else MXQ_COMBINE(float, true, false);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_COMBINE
  return MXQ_OK;
}

int mxq_combine_rows_backward(const void* dy, int64_t ld_dy, const void* rows, int64_t ld_rows, int64_t n_rows,
                              const int32_t* position, const float* weights, int64_t n_tokens, int64_t top_k,
                              int64_t H, mxq_dtype dt, void* drows, int64_t ld_drows, float* dweights,
                              hipStream_t stream) {
  if (!is_float(dt)) return MXQ_ERR_DTYPE;
  if (n_rows < 0 || n_tokens < 0 || H < 0 || top_k < 1 || n_rows > kMaxDim || H > kMaxDim || top_k > kMaxDim ||
      n_tokens > kMaxDim / top_k)
    return MXQ_ERR_SHAPE;
  if (n_tokens == 0) return MXQ_OK;
  if (!position || (H > 0 && (!dy || (n_rows > 0 && (!rows || !drows))))) return MXQ_ERR_NULL;
  if (ld_dy < H || ld_rows < H || ld_drows < H) return MXQ_ERR_SHAPE;
  const int64_t slots = n_tokens * top_k;
  const size_t es = size_of(dt);
  const Range rg = matrix_range(dy, n_tokens, H, ld_dy, es), rr = matrix_range(rows, n_rows, H, ld_rows, es),
              rp = matrix_range(position, 1, slots, slots, 4), rw = matrix_range(weights, 1, weights ? slots : 0, slots, 4),
              rd = matrix_range(drows, n_rows, H, ld_drows, es),
              rv = matrix_range(dweights, 1, dweights ? slots : 0, slots, 4);
  if (!all_ok({rg, rr, rp, rw, rd, rv}) || !aligned(position, 4) || !aligned(weights, 4) || !aligned(dweights, 4) ||
      !aligned(dy, es) || !aligned(rows, es) || !aligned(drows, es))
    return MXQ_ERR_SHAPE;
  if (!disjoint({rd, rv}, {rg, rr, rp, rw})) return MXQ_ERR_ALIAS;
  const bool vec = vector_rows(dy, ld_dy, dt) && vector_rows(rows, ld_rows, dt) && vector_rows(drows, ld_drows, dt) &&
                   H % kEPL == 0;
  const dim3 block(kRowThreads);
  const bool stream_out = n_rows * H * (int64_t)size_of(dt) > kStreamBytes;
#define MXQ_BACKWARD(T, V, S)                                                                                        \
  hipLaunchKernelGGL((combine_backward_kernel<T, V, S>), grid, block, 0, stream, (const T*)dy + t * ld_dy, ld_dy,     \
                     (const T*)rows, ld_rows, (int)n_rows, position + t * top_k, weights ? weights + t * top_k : weights, \
                     (int)top_k, (int)H, (T*)drows, ld_drows, dweights ? dweights + t * top_k : dweights)
  const int64_t step = rows_per_launch(kRowThreads);
  for (int64_t t = 0; t < n_tokens; t += step) {
    const dim3 grid((uint32_t)std::min(step, n_tokens - t));
    if (dt == MXQ_BF16) {
      if (!vec) MXQ_BACKWARD(uint16_t, false, false);
      else if (stream_out) MXQ_BACKWARD(uint16_t, true, true);
      else MXQ_BACKWARD(uint16_t, true, false);
    } else {
      if (!vec) MXQ_BACKWARD(float, false, false);
      else if (stream_out) MXQ_BACKWARD(float, true, true);
      else MXQ_BACKWARD(float, true, false);
    }
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
#undef MXQ_BACKWARD
  return MXQ_OK;
}

}  // extern "C"
