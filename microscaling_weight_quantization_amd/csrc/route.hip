// route.hip -- each token's experts and their weights from a router's logits, and the
// gradient of the logits, on gfx950.
//
// A token's experts are the top_k largest keys: the logits themselves, or with a bias score
// + bias, in 64 bits, so that a choice does not turn on the last places of an exp.  An expert
// whose key is -inf is closed.  With groups only the experts of the best groups take part.  Equal
// keys, and equal groups, go by the lower index.
//   weights    w_j = scale p_j, or scale p_j / sum over the chosen p
//   gradients  softmax:  dl_e = p_e (h_e - sum h p) with h the gradient of p
//              sigmoid:  dl_e = p_e (1 - p_e) h_e
//              where the weights sum to scale, p_j h_j = w_j (g_j - sum g w / scale), for both,
//              and sum h p = 0
//
// Choices need 64 bits, weights and gradients do not: where sixteen lanes share a token they are computed in fp32, the weights
// off by 6e-8 of themselves in the root mean square and by up to 4e-7; where a wave has it in 64 bits (2.5e-8, 6e-8).
//
// Instructions bound the choice, 1259 a wave of four fp32 tokens of 256 experts with a bias and 8 groups, most of them
// comparisons in pairs: 131072 tokens take 64 us (2.2 TB/s) with 94% of the issue slots taken; 16384 are one round of waves,
// 14.0 us and 39%.  131072 bf16 tokens of 128 experts take 26.3 us (596 instructions a wave, 94%).  A wave that has a token
// to itself takes 1235: 65536 fp32 tokens of 128 experts, 20 of them chosen, 115 us, all slots taken.  Gradients of 131072
// tokens of 128 experts take 23.5 us in fp32 (6.1 TB/s) and 15.8 in bf16 (4.8); for 65536 fp32 tokens of 20 choices, a wave
// each in 64 bits, 65.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <type_traits>

#include "checks.h"
#include "fastdiv.h"
#include "floats.h"

namespace {

using namespace mxq_host;
using namespace mxq_dev;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int tokens, experts;
  const float* bias;
  const uint8_t* mask;
  int sigmoid, renormalize;
  float scale;
  int groups, top_groups, group_top, top_k;
  MxqDivisor group_size;
  int group_lanes_log, per;   // lanes of a group (2 to this power) and experts of a lane, where 16 lanes share a token
  bool wide, wide_bias;       // whose experts fill the lanes and can be read 16 bytes at a time
  int32_t* ids;
  float* weights;
};

constexpr int kThreads = 256;
constexpr int kMost = 512;            // experts
constexpr int kPer = kMost / 64;      // of a lane where a wave has a token to itself
constexpr double kClosed = -__builtin_inf();
constexpr double kNaN = -0x1p990;     // a NaN's place among the keys: open, below all others
constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504088896341f;

template <bool kBf16>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  return kBf16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t*)row)[e] << 16) : ((const float*)row)[e];
}
template <bool kBf16>
__device__ __forceinline__ const char* logit_row(const void* logits, int64_t ld, int64_t token) {
  return (const char*)logits + token * ld * (kBf16 ? 2 : 4);
}

// ---- a wave to a token, in 64 bits -------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ double row_dpp(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{dpp<CTRL>(b[0]), dpp<CTRL>(b[1])});
}
// Lane exchanges between pairs, quads and halves of a row of 16: the last two of values that are equal in the lanes below.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor4 = 0x141, kXor8 = 0x140;

// What two neighbouring rows hold, and the two halves of the wave, in both of them.
struct Two {
  double a, b;
};
__device__ __forceinline__ Two rows_of_two(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v), lo = swap16(b[0], b[0]), hi = swap16(b[1], b[1]);
  return Two{__builtin_bit_cast(double, u32x2{lo[0], hi[0]}), __builtin_bit_cast(double, u32x2{lo[1], hi[1]})};
}
__device__ __forceinline__ Two halves_of(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v), lo = swap32(b[0], b[0]), hi = swap32(b[1], b[1]);
  return Two{__builtin_bit_cast(double, u32x2{lo[0], hi[0]}), __builtin_bit_cast(double, u32x2{lo[1], hi[1]})};
}
template <typename F>
__device__ __forceinline__ double wave_fold(double v, F f) {
  v = f(v, row_dpp<kXor1>(v));
  v = f(v, row_dpp<kXor2>(v));
  v = f(v, row_dpp<kXor4>(v));
  v = f(v, row_dpp<kXor8>(v));
  Two t = rows_of_two(v);
  t = halves_of(f(t.a, t.b));
  return f(t.a, t.b);
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_fold(v, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_add(double v) {
  return wave_fold(v, [](double a, double b) { return a + b; });
}
// LDS that the lanes of one wave hand each other.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The larger and the smaller of two numbers (neither of these is a NaN, so nothing needs to be made quiet first).
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// What a wave needs in LDS: the experts' values and logits, the groups' values and which of them are kept, the choice.
struct WaveLds {
  double *value, *rank;
  float* logit;
  int32_t* chosen;
  uint8_t* kept;
  __host__ __device__ static size_t bytes(int experts, int top_k, int groups) {
    return ((size_t)experts * 12 + (size_t)top_k * 4 + (size_t)groups * 9 + 15) / 16 * 16;
  }
  __device__ __forceinline__ WaveLds(char* lds, const RouteArgs& a) {
    value = (double*)(lds + threadIdx.x / 64 * bytes(a.experts, a.top_k, a.groups));
    rank = value + a.experts;
    logit = (float*)(rank + a.groups);
    chosen = (int32_t*)(logit + a.experts);
    kept = (uint8_t*)(chosen + a.top_k);
  }
};

// Which groups are kept, from the experts' values.  A group is shared by as many lanes as there are for it, a power of two;
// its place is the number of groups before it.
__device__ __forceinline__ void keep_groups(const RouteArgs& a, const WaveLds& sh) {
  const int lane = threadIdx.x & 63, size = a.group_size.d;
  const int share_log = a.groups > 32 ? 0 : 31 - __builtin_clz(64 / a.groups), share = 1 << share_log;
  for (int g = lane >> share_log; g < a.groups; g += 64 >> share_log) {   // a group's lanes walk together
    double first = kClosed, second = kClosed;
    const auto fold = [&](double f, double o) {
      second = max64(max64(second, o), min64(first, f));
      first = max64(first, f);
    };
    for (int j = lane & (share - 1); j < size; j += share) fold(sh.value[g * size + j], kClosed);
    if (share > 1) fold(row_dpp<kXor1>(first), row_dpp<kXor1>(second));
    if (share > 2) fold(row_dpp<kXor2>(first), row_dpp<kXor2>(second));
    if (share > 4) fold(row_dpp<kXor4>(first), row_dpp<kXor4>(second));
    if (share > 8) fold(row_dpp<kXor8>(first), row_dpp<kXor8>(second));
    if (share > 16) {   // two groups: all lanes are here
      const Two f = rows_of_two(first), s = rows_of_two(second);
      first = f.a, second = s.a;
      fold(f.b, s.b);
    }
    double rank = first;
    if (a.group_top == 2 && second != kClosed) rank = !a.bias && second == kNaN ? kNaN : first + second;
    if (!(lane & (share - 1))) sh.rank[g] = rank;
  }
  wave_sync();
  for (int g = lane; g < a.groups; g += 64) {
    const double mine = sh.rank[g];
    int before = 0;
    for (int o = 0; o < a.groups; o++) before += sh.rank[o] > mine || (sh.rank[o] == mine && o < g);
    sh.kept[g] = before < a.top_groups;
  }
  wave_sync();
}

// kOwn experts a lane: lane + 64 i.  4096 fp32 tokens of 128 experts, 20 of them chosen: 11.4 us.  Each choice is a fold of the
// whole wave, one after the other.
template <bool kBf16, int kOwn>
__device__ void route_exact(const RouteArgs& a, int64_t token, char* lds) {
  const WaveLds sh(lds, a);
  const int lane = threadIdx.x & 63;
  const bool open = !a.mask || a.mask[token];
  const bool sums = a.groups > 1 && a.group_top == 2;   // groups rank by scores
  const bool scores = a.bias || sums;
  const char* const row = logit_row<kBf16>(a.logits, a.ld, token);
  double key[kOwn];
  double top = kClosed, sum = 0;
  {
    double l[kOwn], p[kOwn], bias[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      const int e = lane + 64 * i;
      const float v = e < a.experts ? logit_at<kBf16>(row, e) : -kInf;
      bias[i] = a.bias && e < a.experts ? a.bias[e] : 0.0f;
      l[i] = open ? (double)v : kClosed;
      if (e < a.experts) sh.logit[e] = v;
    }
    if (!a.sigmoid && (scores || !a.renormalize)) {
#pragma unroll
      for (int i = 0; i < kOwn; i++) top = fmax(top, l[i]);
      top = wave_max(top);
      if (top == kClosed) top = 0;
#pragma unroll
      for (int i = 0; i < kOwn; i++) {
        p[i] = exp(l[i] - top);
        sum += p[i];
      }
      sum = wave_add(sum);
    }
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      const int e = lane + 64 * i;
      if (scores) p[i] = a.sigmoid ? 1 / (1 + exp(-l[i])) : p[i] / sum;
      key[i] = a.bias && l[i] != kClosed ? p[i] + bias[i] : l[i];
      if (key[i] != key[i]) key[i] = kNaN;
      double v = key[i];
      if (sums && !a.bias && v != kClosed) v = p[i] == p[i] ? p[i] : kNaN;
      if (e < a.experts) sh.value[e] = v;
    }
  }
  wave_sync();
  if (a.groups > 1) {
    keep_groups(a, sh);
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      const int e = lane + 64 * i;
      if (e < a.experts && !sh.kept[mxq_quot((uint32_t)e, a.group_size)]) key[i] = kClosed;
    }
  }
  for (int j = 0; j < a.top_k; j++) {   // the largest, the lowest index where several are equal
    double most = key[0];
#pragma unroll
    for (int i = 1; i < kOwn; i++) most = max64(most, key[i]);
    most = wave_fold(most, [](double a, double b) { return max64(a, b); });
    int at = -1;
#pragma unroll
    for (int i = kOwn - 1; i >= 0; i--) {
      const uint64_t equal = __ballot(key[i] == most && most != kClosed);
      if (equal) at = 64 * i + __builtin_ctzll(equal);
    }
#pragma unroll
    for (int i = 0; i < kOwn; i++)
      if (lane + 64 * i == at) key[i] = kClosed;
    if (lane == 0) sh.chosen[j] = at;
  }
  wave_sync();
  // weights: relative to the largest of the chosen logits where they are made to sum to scale
  double largest = kClosed, total = 0;
  if (a.renormalize) {
    for (int j = lane; j < a.top_k; j += 64)
      if (sh.chosen[j] >= 0) largest = fmax(largest, (double)sh.logit[sh.chosen[j]]);
    largest = wave_max(largest);
  }
  for (int j = lane; j < a.top_k; j += 64) {
    const int e = sh.chosen[j];
    const double v = e < 0 ? kClosed : (double)sh.logit[e];
    double w;
    if (!a.sigmoid) {
      w = a.renormalize ? exp(v - largest) : exp(v - top) / sum;
    } else {
      const double m = a.renormalize ? fmin(largest, 0.0) : 0.0;
      w = v > 0 ? exp(-m) / (1 + exp(-v)) : exp(v - m) / (1 + exp(v));
    }
    if (e < 0) w = 0;
    sh.value[j] = w;   // the values have been used
    total += w;
  }
  const double scale = a.scale / (a.renormalize ? [](double t) { return t != 0 ? t : 1.0; }(wave_add(total)) : 1.0);
  for (int j = lane; j < a.top_k; j += 64) {
    a.ids[token * a.top_k + j] = sh.chosen[j];
    a.weights[token * a.top_k + j] = (float)(sh.value[j] * scale);
  }
  wave_sync();   // the LDS may take another token
}

template <bool kBf16, int kOwn>
__global__ __launch_bounds__(kThreads) void route_wave_kernel(RouteArgs a) {
  extern __shared__ __align__(16) char lds[];
  const int64_t token = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
  if (token < a.tokens) route_exact<kBf16, kOwn>(a, token, lds);
}

// ---- sixteen lanes to a token ------------------------------------------------------------
// Keys are taken in fp32 first, which without a bias is what they are.  A biased score, or the sum of two scores that ranks
// a group, is known to within a bound.  Where two chosen experts, or the last of them and one that is left out, or two
// groups lie nearer than that, the few in question are put in order by their keys in 64 bits, a lane each; where they are
// not few, or a key is not finite, the wave takes the token as above.  All of the wave's tokens again in 64 bits took 16.0 us
// where this takes 14.0, and that has about one token in a thousand in question.
//
// A key and its expert are one double: the key with the expert's index in the lowest nine bits, so that equal keys fall
// by index and a comparison moves both.  Each lane sorts its own, and four exchanges between lanes leave the token's
// largest kList in each of them.

template <int CTRL>
__device__ __forceinline__ float row_dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <typename F>
__device__ __forceinline__ float row_fold(float v, F f) {
  v = f(v, row_dpp<kXor1>(v));
  v = f(v, row_dpp<kXor2>(v));
  v = f(v, row_dpp<kXor4>(v));
  return f(v, row_dpp<kXor8>(v));
}
template <typename F>
__device__ __forceinline__ double row_fold(double v, F f) {
  v = f(v, row_dpp<kXor1>(v));
  v = f(v, row_dpp<kXor2>(v));
  v = f(v, row_dpp<kXor4>(v));
  return f(v, row_dpp<kXor8>(v));
}
// A NaN stays.
__device__ __forceinline__ float high(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float low(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float row_max(float v) { return row_fold(v, high); }
__device__ __forceinline__ float row_min(float v) { return row_fold(v, low); }
template <typename F>
__device__ __forceinline__ F row_add(F v) {
  return row_fold(v, [](F a, F b) { return a + b; });
}
__device__ __forceinline__ bool row_any(bool v) { return row_max(v ? 1.0f : 0.0f) != 0; }

__device__ __forceinline__ void order(double& a, double& b) {
  const double x = max64(a, b);
  b = min64(a, b);
  a = x;
}

// Falling order of n values that first rise and then fall, or the other way round.
template <int n>
__device__ __forceinline__ void merge_bitonic(double* v) {
#pragma unroll
  for (int d = n / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < n; i++)
      if (!(i & d)) order(v[i], v[i + d]);
}
// Falling order of n values: Batcher's merging of odd and even places.
template <int n>
__device__ __forceinline__ void sort_falling(double* v) {
#pragma unroll
  for (int p = 1; p < n; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < n; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; i++)
          if (j + i + k < n && (j + i) / (2 * p) == (j + i + k) / (2 * p)) order(v[j + i], v[j + i + k]);
}

constexpr double kOpen = -0x1p995, kShut = -0x1p1000;   // open keys lie above kOpen

// The key is an fp32 value, its lowest nine bits are 0.  An infinite key makes a NaN, whose token is in doubt anyway.
__device__ __forceinline__ double with_index(double key, int e) {
  u32x2 b = __builtin_bit_cast(u32x2, max64(key, kShut));
  const uint32_t at = (uint32_t)(kMost - 1 - e) ^ ((uint32_t)((int)b[1] >> 31) & (kMost - 1));   // e itself below 0
  b[0] |= at;
  return __builtin_bit_cast(double, b);
}
__device__ __forceinline__ int index_of(double v) {
  return (int)(__builtin_bit_cast(u32x2, v)[0] & (kMost - 1)) ^ (v < 0 ? 0 : kMost - 1);
}

// Steps that the list of a token takes through the row's other lanes.
template <int CTRL, int kList>
__device__ __forceinline__ void merge_lanes(double (&v)[kList]) {
  double o[kList];
#pragma unroll
  for (int i = 0; i < kList; i++) o[i] = row_dpp<CTRL>(v[i]);
#pragma unroll
  for (int i = 0; i < kList; i++) v[i] = max64(v[i], o[kList - 1 - i]);
  merge_bitonic<kList>(v);
}

// The largest kList of n values, falling.
template <int n, int kList>
__device__ __forceinline__ void largest_of(const double (&d)[n], double (&v)[kList]) {
  constexpr int kFirst = n < kList ? n : kList;
#pragma unroll
  for (int i = 0; i < kList; i++) v[i] = i < kFirst ? d[i < n ? i : 0] : kShut;
  sort_falling<kFirst>(v);
#pragma unroll
  for (int at = kList; at < n; at += kList) {
    double o[kList];
#pragma unroll
    for (int i = 0; i < kList; i++) o[i] = d[at + i < n ? at + i : 0];
    sort_falling<kList>(o);
#pragma unroll
    for (int i = 0; i < kList; i++) v[i] = max64(v[i], o[kList - 1 - i]);
    merge_bitonic<kList>(v);
  }
}

// How many groups go before this lane's: those of a larger value, or of an equal one and a lower index.
template <int N, typename F>
__device__ __forceinline__ int groups_before(F v, int g, int group_lanes) {
  int before = 0;
  if constexpr (N < 16) {
    before = groups_before<N + 1>(v, g, group_lanes);
    if ((N & (group_lanes - 1)) == 0) {
      const F o = row_dpp<0x120 + N>(v);   // rotated by N lanes
      const int og = (int)dpp<0x120 + N>((uint32_t)g);
      before += o > v || (o == v && og < g);
    }
  }
  return before;
}

// How far two scores in fp32 may be off together.  A sigmoid is off by 2^-23 for each of exp2 and the reciprocal, half of
// that for the sum and, with p (1 - p) |x| < 0.23, by a fifth of it for the exponent: less than 2^-22 each.  A softmax is off
// in parts of the largest score: the sum by 36 roundings and by its terms, 2.5 |z| + 2 of 2^-24 each with a weighted mean of
// |z| < log 512, and the scores' own places: 62 of 2^-24 at most.  A key adds its own rounding, in parts of itself, and so does
// a sum of two keys, which is no larger than their magnitudes: 2^-24 of these for the keys and as much for the sum.
constexpr float kSigmoidOff = 0x1p-21f, kSoftmaxOff = 0x1p-18f, kKeyOff = 0x1p-22f;
__device__ __forceinline__ float exponential(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }

// A lane's experts: base, base + 1, ...; x their logits, -inf where there is none or it is closed; bias theirs.
template <int kEach>
struct Mine {
  int lane16, group, base;
  float x[kEach], bias[kEach];
};

// What lane j knows of its token's j-th expert.
struct Pick {
  int expert;
  bool has;
};

// The experts for which near(i) holds, i of this lane's, into the token's place in LDS, up to 16 of them.  Returns how many.
template <int kEach, typename F>
__device__ __forceinline__ int list_near(const Mine<kEach>& m, int* list, F near) {
  int count = 0;
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    const bool it = near(i);
    const uint32_t all = (uint32_t)(__ballot(it) >> (threadIdx.x & 48)) & 0xFFFFu;   // of the token's lanes
    const int at = count + __builtin_popcount(all & ((1u << m.lane16) - 1));
    if (it && at < 16) list[at] = m.base + i;
    count += __builtin_popcount(all);
  }
  wave_sync();
  return count;
}

// In 64 bits: what divides a token's scores, and an expert's key (or score, where there is no bias).
template <bool kBf16>
__device__ __forceinline__ double sum_of_scores(const RouteArgs& a, const char* row, float top) {
  if (a.sigmoid) return 1;
  double sum = 0;
#pragma unroll 1
  for (int e = threadIdx.x & 15; e < a.experts; e += 16) sum += exp((double)logit_at<kBf16>(row, e) - (double)top);
  return row_add(sum);
}
template <bool kBf16>
__device__ __forceinline__ double key_of(const RouteArgs& a, const char* row, float top, double sum, int e) {
  const double l = logit_at<kBf16>(row, e), t = exp(a.sigmoid ? -l : l - (double)top);
  return (a.sigmoid ? 1 / (1 + t) : t / sum) + (a.bias ? (double)a.bias[e] : 0.0);
}

// f for the other lanes of the row, each N lanes away.
template <int N = 1, typename F>
__device__ __forceinline__ void for_others(F f) {
  if constexpr (N < 16) {
    f(std::integral_constant<int, 0x120 + N>{});
    for_others<N + 1>(f);
  }
}

// The groups in question (asked), put in order by values in 64 bits: the best of them are kept, as many as there is room
// for.  Of a group's experts those whose values lie at `floor` or above can be its first two.  Returns whether these are
// more than 16 for the token.
template <bool kBf16, int kEach>
__device__ __forceinline__ bool settle_groups(const RouteArgs& a, const Mine<kEach>& m, const char* row, float top,
                                              const float (&value)[kEach], float floor, bool asked, int room, int* list,
                                              bool* kept) {
  const int count = list_near(m, list, [&](int i) { return asked && value[i] >= floor && value[i] > -kInf; });
  const double sum = sum_of_scores<kBf16>(a, row, top);
  const bool mine = m.lane16 < count;
  const int e = mine ? list[m.lane16] : kMost, g = mine ? (int)mxq_quot((uint32_t)e, a.group_size) : -1 - m.lane16;
  const double key = mine ? key_of<kBf16>(a, row, top, sum, e) : kClosed;
  double first = key, second = kClosed;
  bool leads = mine;   // one lane speaks for its group
  for_others([&](auto ctrl) {
    const double o = row_dpp<ctrl.value>(key);
    const int og = (int)dpp<ctrl.value>((uint32_t)g), oe = (int)dpp<ctrl.value>((uint32_t)e);
    if (og == g) {
      second = fmax(second, fmin(first, o));
      first = fmax(first, o);
      leads &= !(o > key || (o == key && oe < e));
    }
  });
  const double rank = a.group_top == 2 && second != kClosed ? first + second : first;
  int before = 0;
  for_others([&](auto ctrl) {
    const double o = row_dpp<ctrl.value>(rank);
    const int og = (int)dpp<ctrl.value>((uint32_t)g);
    before += dpp<ctrl.value>((uint32_t)leads) && (o > rank || (o == rank && og < g));
  });
  wave_sync();
  list[m.lane16] = 0;
  wave_sync();
  if (leads) list[g] = before < room;
  wave_sync();
  *kept = list[m.group] != 0;
  wave_sync();
  return count > 16;
}

// The experts whose keys lie at `edge` or above, put in order by their keys in 64 bits, a lane each.  Returns whether they
// are more than that.
template <bool kBf16, int kEach>
__device__ __forceinline__ bool settle(const RouteArgs& a, const Mine<kEach>& m, const char* row, float top, bool kept,
                                       const float (&key)[kEach], float edge, int* list, Pick* pick) {
  // the edge itself may lie beyond the largest number
  const int count = list_near(m, list, [&](int i) { return kept && key[i] >= edge && key[i] > -kInf; });
  const double sum = sum_of_scores<kBf16>(a, row, top);
  const bool mine = m.lane16 < count;
  const int e = mine ? list[m.lane16] : kMost + m.lane16;
  const int place = groups_before<1>(mine ? key_of<kBf16>(a, row, top, sum, e) : kClosed, e, 1);
  wave_sync();
  list[place] = e;
  wave_sync();
  *pick = Pick{list[m.lane16], mine && m.lane16 < a.top_k};
  wave_sync();
  return count > 16;
}

// Lane j's pick, the token's j-th expert, into *pick.  Returns whether the choice is in doubt.
template <bool kBf16, int kList, int kEach>
__device__ __forceinline__ bool choose(const RouteArgs& a, const Mine<kEach>& m, const char* row, float top, int* list,
                                       Pick* pick) {
  const bool sums = a.groups > 1 && a.group_top == 2;      // groups rank by scores
  bool doubt = false;
  float s[kEach], bound = kSigmoidOff;
  if (a.bias || sums) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < kEach; i++) s[i] = __builtin_amdgcn_rcpf(1 + exponential(-m.x[i]));
    } else {
      float sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; i++) {
        s[i] = exponential(m.x[i] - top);
        sum += s[i];
      }
      sum = row_add(sum);
      const float r = sum > 0 ? 1 / sum : 0.0f;
      bound = kSoftmaxOff * r;
#pragma unroll
      for (int i = 0; i < kEach; i++) s[i] *= r;
    }
  }
  float key[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    key[i] = m.x[i];
    if (a.bias) {
      key[i] = m.x[i] == -kInf ? -kInf : s[i] + m.bias[i];
      doubt |= !(key[i] < kInf);
    }
  }
  bool kept = true;
  if (a.groups > 1) {
    const int lanes = 1 << a.group_lanes_log;
    float value[kEach], first = -kInf, second = first;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      value[i] = sums && !a.bias ? (m.x[i] == -kInf ? -kInf : s[i]) : key[i];
      second = fmaxf(second, fminf(first, value[i]));
      first = fmaxf(first, value[i]);
    }
    const auto fold = [&](float f, float o) {
      second = fmaxf(fmaxf(second, o), fminf(first, f));
      first = fmaxf(first, f);
    };
    if (lanes > 1) fold(row_dpp<kXor1>(first), row_dpp<kXor1>(second));
    if (lanes > 2) fold(row_dpp<kXor2>(first), row_dpp<kXor2>(second));
    if (lanes > 4) fold(row_dpp<kXor4>(first), row_dpp<kXor4>(second));
    const bool two = sums && second != -kInf;
    const float rank = two ? first + second : first;
    kept = groups_before<1>(rank, m.group, lanes) < a.top_groups;
    if (a.bias || sums) {
      doubt |= fabsf(rank) == kInf && fabsf(first) != kInf;   // a sum beyond the largest number
      // as far as the rank may be off: keys of opposite signs are rounded each in parts of itself, however small their sum is
      const float off = first == -kInf ? 0.0f : bound + (fabsf(first) + (two ? fabsf(second) : 0.0f)) * kKeyOff;
      const float least = row_min(kept ? rank - off : kInf), most = row_max(kept ? -kInf : rank + off);
      const bool asked = most > -kInf && !(kept ? rank - off > most : rank + off < least);
      const bool near = row_any(asked);
      if (__any(near)) {
        const float last = a.group_top == 2 ? second : first;
        const int sure = (int)row_add(kept && !asked ? 1.0f : 0.0f) >> a.group_lanes_log;
        bool settled;
        const bool many = settle_groups<kBf16>(a, m, row, top, value, last - bound - fabsf(last) * kKeyOff, asked,
                                               a.top_groups - sure, list, &settled);
        if (asked) kept = settled;
        doubt |= near && many;
      }
    }
  }
  double d[kEach], v[kList];
#pragma unroll
  for (int i = 0; i < kEach; i++)   // + 0: of the zeros one is as good as the other
    d[i] = with_index(kept ? (double)(key[i] + 0) : kClosed, min(m.base + i, kMost - 1));
  largest_of<kEach, kList>(d, v);
  merge_lanes<kXor1>(v);
  merge_lanes<kXor2>(v);
  merge_lanes<kXor4>(v);
  merge_lanes<kXor8>(v);
  double mine = v[0];
#pragma unroll
  for (int j = 1; j < kList; j++) mine = m.lane16 == j ? v[j] : mine;
  *pick = Pick{index_of(mine), m.lane16 < a.top_k && mine > kOpen};
  doubt = row_any(doubt);
  if (a.bias) {
    const float k = (float)mine, next = (float)row_dpp<0x101>(mine);   // of the next lane
    const float step = bound + fabsf(k) * kKeyOff;
    bool near = pick->has && m.lane16 + 1 < a.top_k && next > (float)kOpen && k - next < step;
    // and the last of them against those that are left out: how many keys lie above it less the step
    const float edge = row_min(pick->has ? k - step : kInf);
    int above = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) above += kept && key[i] >= edge;
    near |= row_add((float)above) > (float)a.top_k;
    near = row_any(near) && !doubt;
    if (__any(near)) {
      Pick settled;
      const bool many = settle<kBf16>(a, m, row, top, kept, key, edge, list, &settled);
      if (near) *pick = settled, doubt = many;
    }
  }
  return doubt;
}

// A lane's row of experts, kAt of them in 16 bytes; those from `count` on -inf.
template <int kEach, bool kBf16>
__device__ __forceinline__ void load_wide(float (&x)[kEach], const char* p, int count) {
  constexpr int kAt = kBf16 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < kEach; i += kAt) {
    const u32x4 w = i < count ? *(const u32x4*)(p + i * (kBf16 ? 2 : 4)) : u32x4{};
#pragma unroll
    for (int j = 0; j < kAt && i + j < kEach; j++) {
      const uint32_t bits = kBf16 ? (j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16) : w[j % 4];
      x[i + j] = i < count ? __builtin_bit_cast(float, bits) : -kInf;
    }
  }
}

template <int kEach, int kList, bool kBf16>
__global__ __launch_bounds__(kThreads) void route_row_kernel(RouteArgs a) {
  keep_denormals();
  extern __shared__ __align__(16) char lds[];
  __shared__ int lists[kThreads / 16][16];
  Mine<kEach> m;
  m.lane16 = threadIdx.x & 15;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
  const bool live = token < a.tokens, open = live && (!a.mask || a.mask[token]);
  const char* const row = logit_row<kBf16>(a.logits, a.ld, live ? token : 0);
  m.group = m.lane16 >> a.group_lanes_log;
  const int in_group = (m.lane16 & ((1 << a.group_lanes_log) - 1)) * a.per;
  m.base = m.group * (int)a.group_size.d + in_group;
  const int here = min(a.per, (int)a.group_size.d - in_group), count = open ? here : 0;
  if (a.wide) {
    load_wide<kEach, kBf16>(m.x, row + m.base * (kBf16 ? 2 : 4), count);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; i++) m.x[i] = i < count ? logit_at<kBf16>(row, m.base + i) : -kInf;
  }
  if (a.bias && a.wide_bias) {
    load_wide<kEach, false>(m.bias, (const char*)(a.bias + m.base), here);
  } else if (a.bias) {
#pragma unroll
    for (int i = 0; i < kEach; i++) m.bias[i] = i < here ? a.bias[m.base + i] : 0.0f;
  }
  float top = m.x[0];
#pragma unroll
  for (int i = 1; i < kEach; i++) top = high(top, m.x[i]);
  top = row_max(top);
  const bool odd = !(top < kInf);   // a NaN or +Inf among the logits
  if (top == -kInf) top = 0;
  Pick pick;
  const bool again = (choose<kBf16, kList>(a, m, row, top, lists[threadIdx.x / 16], &pick) || odd) && open;
  const bool has = pick.has;
  const int e = pick.expert;
  const float l = has ? logit_at<kBf16>(row, min(e, a.experts - 1)) : -kInf;
  float w = 0;
  if (a.renormalize) {
    const float largest = row_max(l);
    if (has) {
      if (a.sigmoid) {
        const float t = expf(-fabsf(l));
        w = (l > 0 ? 1.0f : expf(l - fminf(largest, 0.0f))) / (1.0f + t);
      } else {
        w = expf(l - largest);
      }
    }
    const float total = row_add(w);
    w = total > 0 ? w / total : w;
  } else if (a.sigmoid) {
    const float t = expf(-fabsf(l));
    w = has ? (l > 0 ? 1.0f : t) / (1.0f + t) : 0.0f;
  } else {
    float sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) sum += exponential(m.x[i] - top);
    sum = row_add(sum);
    w = has ? expf(l - top) / sum : 0.0f;
  }
  if (live && !again && m.lane16 < a.top_k) {
    a.ids[token * a.top_k + m.lane16] = has ? e : -1;
    a.weights[token * a.top_k + m.lane16] = w * a.scale;
  }
  // the tokens that are still in doubt, one after the other
  for (uint64_t left = __ballot(again && m.lane16 == 0); left; left &= left - 1) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 64 * 4;
    route_exact<kBf16, kEach / 4>(a, first + __builtin_ctzll(left) / 16, lds);
  }
}

// ---- backward ----------------------------------------------------------------------------
struct BackArgs {
  const float* dweights;
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int tokens, experts, top_k;
  int sigmoid, renormalize;
  float scale;
  void* out;
  int64_t ld_out;
};

// A wave to a token, in 64 bits, for any number of choices.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void route_backward_wave_kernel(BackArgs a) {
  __shared__ float shared[kThreads / 64][kMost];
  float* const d = shared[threadIdx.x / 64];
  const int lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
  if (token >= a.tokens) return;
  const char* const row = logit_row<kBf16>(a.logits, a.ld, token);
  const int32_t* const ids = a.ids + token * a.top_k;
  const float* const grads = a.dweights + token * a.top_k;
  const bool dense = !a.sigmoid && !a.renormalize;
  double l[kPer];
  double top = kClosed, sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int e = lane + 64 * i;
    l[i] = e < a.experts ? (double)logit_at<kBf16>(row, e) : kClosed;
    top = fmax(top, l[i]);
    d[e] = 0;
  }
  top = wave_max(top);
  if (top == kClosed) top = 0;
  if (dense) {
#pragma unroll
    for (int i = 0; i < kPer; i++) sum += exp(l[i] - top);
    sum = wave_add(sum);
    if (sum == 0) sum = 1;   // every expert is closed
  }
  wave_sync();
  const auto chosen = [&](int j) { return ids[j] < a.experts ? ids[j] : -1; };
  double largest = kClosed;
  for (int j = lane; j < a.top_k; j += 64)
    if (chosen(j) >= 0) largest = fmax(largest, (double)logit_at<kBf16>(row, chosen(j)));
  largest = wave_max(largest);
  if (largest == kClosed) largest = 0;   // no choice, or closed ones
  const auto weight = [&](int e) -> double {   // p, times a factor that is the same for the token where they are renormalized
    const double v = logit_at<kBf16>(row, e);
    if (!a.sigmoid) return a.renormalize ? exp(v - largest) : exp(v - top) / sum;
    const double m = a.renormalize ? fmin(largest, 0.0) : 0.0;
    return v > 0 ? exp(-m) / (1 + exp(-v)) : exp(v - m) / (1 + exp(v));
  };
  double total = 0, dot = 0;
  bool some = false;
  for (int j = lane; j < a.top_k; j += 64)
    if (chosen(j) >= 0) {
      some = true;
      const double p = weight(chosen(j));
      total += p;
      dot += p * grads[j];
    }
  const bool spread = dense && __any(some);   // of a token without a choice the gradient is 0, whatever the logits hold
  total = wave_add(total);
  dot = wave_add(dot);
  for (int j = lane; j < a.top_k; j += 64) {
    const int e = chosen(j);
    if (e < 0) continue;
    const double p = weight(e), v = logit_at<kBf16>(row, e);
    double h = a.renormalize ? (total != 0 ? p / total * (grads[j] - dot / total) : 0.0) : p * grads[j];
    if (a.sigmoid) h *= v > 0 ? exp(-v) / (1 + exp(-v)) : 1 / (1 + exp(v));
    atomicAdd(d + e, (float)(h * a.scale));   // one addition for each expert, unless ids names one twice
  }
  wave_sync();
  char* const out = (char*)a.out + token * a.ld_out * (kBf16 ? 2 : 4);
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int e = lane + 64 * i;
    if (e >= a.experts) continue;
    double v = d[e];
    if (spread) v -= exp(l[i] - top) / sum * dot * a.scale;
    if constexpr (kBf16) ((__bf16*)out)[e] = (__bf16)(float)v;
    else ((float*)out)[e] = (float)v;
  }
}

// Sixteen lanes to a token, lane j with its j-th choice; the choices' gradients meet the experts' places in LDS.
// kAt: experts that a lane reads and writes at once.
template <int kEach, int kAt, bool kBf16>
__global__ __launch_bounds__(kThreads) void route_backward_row_kernel(BackArgs a) {
  keep_denormals();
  constexpr int kRow = kEach * 16 + 4;   // the tokens' rows begin in other banks
  __shared__ __align__(16) float shared[kThreads / 16][kRow];
  float* const d = shared[threadIdx.x / 16];
  const int lane16 = threadIdx.x & 15;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
  const bool live = token < a.tokens;
  const char* const row = logit_row<kBf16>(a.logits, a.ld, live ? token : 0);
  const bool dense = !a.sigmoid && !a.renormalize;
  const int32_t id = live && lane16 < a.top_k ? a.ids[token * a.top_k + lane16] : -1;
  const bool has = id >= 0 && id < a.experts;
  const uint64_t chosen = __ballot(has);   // of the wave's four tokens
  const float grad = has ? a.dweights[token * a.top_k + lane16] : 0.0f;
  const float l = has ? logit_at<kBf16>(row, id) : -kInf;
  float x[kEach], top = -kInf, sum = 1.0f;
#pragma unroll
  for (int i = 0; i < kEach; i++) d[i * 16 + lane16] = 0;
  if (dense) {
#pragma unroll
    for (int i = 0; i < kEach; i += kAt) {
      const int e = i * 16 + lane16 * kAt;
      if constexpr (kAt == 1) {
        x[i] = e < a.experts ? logit_at<kBf16>(row, e) : -kInf;
      } else {
        const u32x4 w = e < a.experts ? *(const u32x4*)(row + e * (kBf16 ? 2 : 4)) : u32x4{};
#pragma unroll
        for (int j = 0; j < kAt; j++) {
          const uint32_t bits = kBf16 ? (j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16) : w[j % 4];
          x[i + j] = e < a.experts ? __builtin_bit_cast(float, bits) : -kInf;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; i++) top = __builtin_elementwise_maximum(top, x[i]);
    top = row_max(top);
    if (top == -kInf) top = 0;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      x[i] = __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
      sum += x[i];
    }
    sum = row_add(sum);
    if (sum == 0) sum = 1;   // every expert is closed
  }
  float largest = row_max(l), p = 0, h = 0;
  if (largest == -kInf) largest = 0;   // no choice, or closed ones
  const float t = expf(-fabsf(l));
  if (has) {   // p, times a factor that is the same for the token where they are renormalized
    if (!a.sigmoid) p = a.renormalize ? expf(l - largest) : expf(l - top) / sum;
    else p = (l > 0 ? 1.0f : expf(l - (a.renormalize ? fminf(largest, 0.0f) : 0.0f))) / (1.0f + t);
  }
  const float total = row_add(p), dot = row_add(p * grad);
  if (has) {
    h = a.renormalize ? (total != 0 ? p / total * (grad - dot / total) : 0.0f) : p * grad;
    if (a.sigmoid) h *= (l > 0 ? t : 1.0f) / (1.0f + t);
  }
  wave_sync();   // a token's lanes are of one wave
  if (has) atomicAdd(d + id, h * a.scale);   // one addition for each expert, unless ids names one twice
  wave_sync();
  if (!live) return;
  // of a token without a choice the gradient is 0, whatever the logits hold
  const bool spread = dense && (uint16_t)(chosen >> (threadIdx.x & 48)) != 0;
  const float less = spread ? dot * a.scale / sum : 0.0f;
  char* const out = (char*)a.out + token * a.ld_out * (kBf16 ? 2 : 4);
#pragma unroll
  for (int i = 0; i < kEach; i += kAt) {
    const int e = i * 16 + lane16 * kAt;
    if (e >= a.experts) continue;
    if constexpr (kAt == 1) {
      const float v = spread ? d[e] - x[i] * less : d[e];
      if constexpr (kBf16) ((__bf16*)out)[e] = (__bf16)v;
      else ((float*)out)[e] = v;
    } else {
      f32x8 v{};
#pragma unroll
      for (int j = 0; j < kAt; j++) v[j] = spread ? d[e + j] - x[i + j] * less : d[e + j];
      const Chunk<uint16_t> b = narrow<uint16_t>(v);
      const u32x4 half{b.w[0], b.w[1], b.w[2], b.w[3]};
      const u32x8 full = __builtin_bit_cast(u32x8, v);
      *(u32x4*)(out + e * (kBf16 ? 2 : 4)) = kBf16 ? half : u32x4{full[0], full[1], full[2], full[3]};
    }
  }
}

// ---- host --------------------------------------------------------------------------------

// Up to 2^31 lanes a launch; `from` gives the arguments from a token on.
template <typename Args, typename From, typename Kernel>
int launch_tokens(const Args& a, int lanes, From from, Kernel kernel, size_t lds, hipStream_t stream) {
  const int64_t step = rows_per_launch(lanes), per = kThreads / lanes;
  for (int64_t t = 0; t < a.tokens; t += step) {
    Args b = from(t);
    b.tokens = (int)std::min<int64_t>(step, a.tokens - t);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((b.tokens + per - 1) / per)), dim3(kThreads), lds, stream, b);
    const int st = launch_status();
    if (st != MXQ_OK) return st;
  }
  return MXQ_OK;
}

constexpr int kListMost = 16;   // choices of a token that sixteen lanes share

template <bool kBf16>
int launch_route(RouteArgs a, hipStream_t stream) {
  const auto from = [&a](int64_t t) {
    RouteArgs b = a;
    b.logits = (const char*)a.logits + t * a.ld * (kBf16 ? 2 : 4);
    if (a.mask) b.mask += t;
    b.ids += t * a.top_k;
    b.weights += t * a.top_k;
    return b;
  };
  const size_t lds = kThreads / 64 * WaveLds::bytes(a.experts, a.top_k, a.groups);
  // groups of whole lanes: 1, 2, 4, 8 or 16 of them
  if (a.groups > 16 || (a.groups & (a.groups - 1)) || a.top_k > kListMost)
    return a.experts <= 128   ? launch_tokens(a, 64, from, route_wave_kernel<kBf16, 2>, lds, stream)
           : a.experts <= 256 ? launch_tokens(a, 64, from, route_wave_kernel<kBf16, 4>, lds, stream)
                              : launch_tokens(a, 64, from, route_wave_kernel<kBf16, 8>, lds, stream);
  const int size = a.experts / a.groups, lanes = 16 / a.groups;
  a.group_lanes_log = __builtin_ctz(lanes);
  a.per = (size + lanes - 1) / lanes;
  constexpr int kAt = kBf16 ? 8 : 4;
  a.wide = a.per * lanes == size && a.per % kAt == 0 && aligned(a.logits, 16) && a.ld % kAt == 0;
  a.wide_bias = a.per * lanes == size && a.per % 4 == 0 && aligned(a.bias, 16);
  const bool few = a.top_k <= 8;
#define MXQ_ROUTE(kEach) \
  return few ? launch_tokens(a, 16, from, route_row_kernel<kEach, 8, kBf16>, lds, stream) \
             : launch_tokens(a, 16, from, route_row_kernel<kEach, 16, kBf16>, lds, stream)
  if (a.per <= 4) MXQ_ROUTE(4);
  if (a.per <= 8) MXQ_ROUTE(8);
  if (a.per <= 16) MXQ_ROUTE(16);
  MXQ_ROUTE(32);
#undef MXQ_ROUTE
}

template <bool kBf16>
int launch_backward(const BackArgs& a, hipStream_t stream) {
  const auto from = [&a](int64_t t) {
    BackArgs b = a;
    b.dweights += t * a.top_k;
    b.ids += t * a.top_k;
    b.logits = (const char*)a.logits + t * a.ld * (kBf16 ? 2 : 4);
    b.out = (char*)a.out + t * a.ld_out * (kBf16 ? 2 : 4);
    return b;
  };
  if (a.top_k > kListMost) return launch_tokens(a, 64, from, route_backward_wave_kernel<kBf16>, 0, stream);
  constexpr int kAt = kBf16 ? 8 : 4;
  const bool wide = a.experts % kAt == 0 && aligned(a.logits, 16) && aligned(a.out, 16) && a.ld % kAt == 0 && a.ld_out % kAt == 0;
#define MXQ_BACK(kEach) \
  return wide ? launch_tokens(a, 16, from, route_backward_row_kernel<kEach, kAt, kBf16>, 0, stream) \
              : launch_tokens(a, 16, from, route_backward_row_kernel<kEach, 1, kBf16>, 0, stream)
  if (a.experts <= 128) MXQ_BACK(8);
  if (a.experts <= 256) MXQ_BACK(16);
  MXQ_BACK(32);
#undef MXQ_BACK
}

int check(int64_t tokens, int64_t experts, int64_t top_k, mxq_dtype dt, int score, float scale) {
  if (!is_float(dt) || (score != MXQ_SOFTMAX && score != MXQ_SIGMOID)) return MXQ_ERR_DTYPE;
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > experts || tokens > kMaxDim / top_k ||
      !(scale - scale == 0))
    return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

}  // namespace

extern "C" {

int mxq_route_experts(const void* logits, int64_t ld_logits, int64_t n_tokens, int64_t n_experts, mxq_dtype dt,
                      const float* bias, const uint8_t* mask, mxq_score score, int renormalize, float scale,
                      int64_t n_groups, int64_t top_groups, int64_t group_top, int64_t top_k, int32_t* ids,
                      float* weights, hipStream_t stream) {
  const int st = check(n_tokens, n_experts, top_k, dt, (int)score, scale);
  if (st != MXQ_OK) return st;
  if (n_groups < 1 || n_groups > n_experts || n_experts % n_groups || top_groups < 1 || top_groups > n_groups ||
      group_top < 1 || group_top > 2 || top_k > n_experts / n_groups * top_groups)
    return MXQ_ERR_SHAPE;
  if (n_tokens == 0) return MXQ_OK;
  if (!logits || !ids || !weights) return MXQ_ERR_NULL;
  if (ld_logits < n_experts) return MXQ_ERR_SHAPE;
  const size_t es = size_of(dt);
  const int64_t slots = n_tokens * top_k;
  const Range rl = matrix_range(logits, n_tokens, n_experts, ld_logits, es),
              rb = matrix_range(bias, bias ? 1 : 0, n_experts, n_experts, 4),
              rm = matrix_range(mask, mask ? 1 : 0, n_tokens, n_tokens, 1), ri = matrix_range(ids, 1, slots, slots, 4),
              rw = matrix_range(weights, 1, slots, slots, 4);
  if (!all_ok({rl, rb, rm, ri, rw}) || !aligned(logits, es) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return MXQ_ERR_SHAPE;
  if (!disjoint({ri, rw}, {rl, rb, rm})) return MXQ_ERR_ALIAS;
  const RouteArgs a{logits, ld_logits, (int)n_tokens, (int)n_experts, bias, mask, score == MXQ_SIGMOID, renormalize != 0,
                    scale, (int)n_groups, (int)top_groups, (int)group_top, (int)top_k,
                    mxq_divisor((uint32_t)(n_experts / n_groups)), 0, 0, false, false, ids, weights};
  return dt == MXQ_BF16 ? launch_route<true>(a, stream) : launch_route<false>(a, stream);
}

int mxq_route_experts_backward(const float* dweights, const void* logits, int64_t ld_logits, const int32_t* ids,
                               int64_t n_tokens, int64_t n_experts, int64_t top_k, mxq_dtype dt, mxq_score score,
                               int renormalize, float scale, void* dlogits, int64_t ld_dlogits, hipStream_t stream) {
  const int st = check(n_tokens, n_experts, top_k, dt, (int)score, scale);
  if (st != MXQ_OK) return st;
  if (n_tokens == 0) return MXQ_OK;
  if (!dweights || !logits || !ids || !dlogits) return MXQ_ERR_NULL;
  if (ld_logits < n_experts || ld_dlogits < n_experts) return MXQ_ERR_SHAPE;
  const size_t es = size_of(dt);
  const int64_t slots = n_tokens * top_k;
  const Range rg = matrix_range(dweights, 1, slots, slots, 4), rl = matrix_range(logits, n_tokens, n_experts, ld_logits, es),
              ri = matrix_range(ids, 1, slots, slots, 4), rd = matrix_range(dlogits, n_tokens, n_experts, ld_dlogits, es);
  if (!all_ok({rg, rl, ri, rd}) || !aligned(dweights, 4) || !aligned(logits, es) || !aligned(ids, 4) || !aligned(dlogits, es))
    return MXQ_ERR_SHAPE;
  if (!disjoint({rd}, {rg, rl, ri})) return MXQ_ERR_ALIAS;
  const BackArgs a{dweights, logits, ld_logits, ids, (int)n_tokens, (int)n_experts, (int)top_k, score == MXQ_SIGMOID,
                   renormalize != 0, scale, dlogits, ld_dlogits};
  return dt == MXQ_BF16 ? launch_backward<true>(a, stream) : launch_backward<false>(a, stream);
}

}  // extern "C"
