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
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

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
  int32_t* ids;
  float* weights;
};

constexpr int kMost = 512;            // experts
constexpr int kPer = kMost / 64;      // a lane
constexpr int kTokens = 4;            // of a workgroup, a wave each
constexpr double kClosed = -__builtin_inf();
constexpr double kNaN = -1e300;       // a NaN's place among the keys: open, below all others

__device__ __forceinline__ float logit_at(const void* row, int e, bool bf16) {
  return bf16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t*)row)[e] << 16) : ((const float*)row)[e];
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmax(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The largest of the wave's keys, the lowest index where several are equal; element lane + 64 i is key[i].
struct Best {
  double key;
  int at;
};
__device__ __forceinline__ Best best_of(const double (&key)[kPer]) {
  const int lane = threadIdx.x & 63;
  Best b{key[0], lane};
#pragma unroll
  for (int i = 1; i < kPer; i++)
    if (key[i] > b.key) b = Best{key[i], lane + 64 * i};
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const Best o{__shfl_xor(b.key, m), __shfl_xor(b.at, m)};
    if (o.key > b.key || (o.key == b.key && o.at < b.at)) b = o;
  }
  return b;
}
__device__ __forceinline__ void take(double (&key)[kPer], int at) {
#pragma unroll
  for (int i = 0; i < kPer; i++)
    if (at == (int)(threadIdx.x & 63) + 64 * i) key[i] = kClosed;
}

struct RouteShared {
  double key[kMost], value[kMost];
  int32_t chosen[kMost];
  uint8_t kept[kMost];
};

template <bool kBf16>
__global__ __launch_bounds__(64 * kTokens) void route_kernel(RouteArgs a) {
  __shared__ RouteShared shared[kTokens];
  RouteShared& sh = shared[threadIdx.x / 64];
  const int lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * kTokens + threadIdx.x / 64;
  const bool live = token < a.tokens;
  const bool open = live && (!a.mask || a.mask[token]);
  const char* const row = (const char*)a.logits + (live ? token : 0) * a.ld * (kBf16 ? 2 : 4);
  double l[kPer], key[kPer];
  double top = kClosed;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int e = lane + 64 * i;
    l[i] = open && e < a.experts ? (double)logit_at(row, e, kBf16) : kClosed;
    top = fmax(top, l[i]);
  }
  top = wave_max(top);
  if (top == kClosed) top = 0;
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) sum += exp(l[i] - top);
  sum = a.sigmoid ? 1.0 : wave_add(sum);
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int e = lane + 64 * i;
    const double p = a.sigmoid ? 1 / (1 + exp(-l[i])) : exp(l[i] - top) / sum;
    key[i] = l[i];
    if (a.bias && l[i] != kClosed) key[i] = p + (double)a.bias[e];
    if (key[i] != key[i]) key[i] = kNaN;
    if (e < a.experts) {
      sh.key[e] = key[i];
      sh.value[e] = a.bias ? key[i] : p;
    }
  }
  __syncthreads();
  if (a.groups > 1) {
    const int size = a.group_size.d;
    double rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int g = lane + 64 * i;
      rank[i] = kClosed;
      if (g < a.groups) {
        double first = kClosed, second = kClosed, v1 = 0, v2 = 0;
        for (int j = 0; j < size; j++) {
          const double k = sh.key[g * size + j], v = sh.value[g * size + j];
          if (k > first) second = first, v2 = v1, first = k, v1 = v;
          else if (k > second) second = k, v2 = v;
        }
        rank[i] = a.group_top == 1 || first == kClosed ? first : v1 + (second == kClosed ? 0.0 : v2);
        if (rank[i] != rank[i]) rank[i] = kNaN;
        sh.kept[g] = 0;
      }
    }
    for (int j = 0; j < a.top_groups; j++) {
      const Best b = best_of(rank);
      if (b.key == kClosed) break;
      take(rank, b.at);
      if (lane == 0) sh.kept[b.at] = 1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int e = lane + 64 * i;
      if (e < a.experts && !sh.kept[mxq_quot((uint32_t)e, a.group_size)]) key[i] = kClosed;
    }
  }
  for (int j = 0; j < a.top_k; j++) {
    const Best b = best_of(key);
    take(key, b.at);
    if (lane == 0) sh.chosen[j] = b.key == kClosed ? -1 : b.at;
  }
  __syncthreads();
  // weights: relative to the largest of the chosen logits where they are made to sum to scale
  double largest = kClosed;
  for (int j = lane; j < a.top_k; j += 64) {
    const int e = sh.chosen[j];
    if (e >= 0) largest = fmax(largest, (double)logit_at(row, e, kBf16));
  }
  largest = wave_max(largest);
  const auto weight = [&](int e) -> double {
    if (e < 0) return 0.0;
    const double v = logit_at(row, e, kBf16);
    if (!a.sigmoid) return a.renormalize ? exp(v - largest) : exp(v - top) / sum;
    const double m = a.renormalize ? fmin(largest, 0.0) : 0.0;
    return v > 0 ? exp(-m) / (1 + exp(-v)) : exp(v - m) / (1 + exp(v));
  };
  double total = 0;
  for (int j = lane; j < a.top_k; j += 64) total += weight(sh.chosen[j]);
  total = wave_add(total);
  const double scale = a.scale / (a.renormalize && total != 0 ? total : 1.0);
  if (live)
    for (int j = lane; j < a.top_k; j += 64) {
      a.ids[token * a.top_k + j] = sh.chosen[j];
      a.weights[token * a.top_k + j] = (float)(weight(sh.chosen[j]) * scale);
    }
}

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

template <bool kBf16>
__global__ __launch_bounds__(64 * kTokens) void route_backward_kernel(BackArgs a) {
  __shared__ float shared[kTokens][kMost];
  float* const d = shared[threadIdx.x / 64];
  const int lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * kTokens + threadIdx.x / 64;
  const bool live = token < a.tokens;
  const char* const row = (const char*)a.logits + (live ? token : 0) * a.ld * (kBf16 ? 2 : 4);
  const int32_t* const ids = a.ids + (live ? token : 0) * a.top_k;
  const float* const grads = a.dweights + (live ? token : 0) * a.top_k;
  const bool dense = !a.sigmoid && !a.renormalize;
  double l[kPer];
  double top = kClosed, sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int e = lane + 64 * i;
    l[i] = live && e < a.experts ? (double)logit_at(row, e, kBf16) : kClosed;
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
  __syncthreads();
  const auto chosen = [&](int j) {
    const int e = live ? ids[j] : -1;
    return e < a.experts ? e : -1;
  };
  double largest = kClosed;
  for (int j = lane; j < a.top_k; j += 64)
    if (chosen(j) >= 0) largest = fmax(largest, (double)logit_at(row, chosen(j), kBf16));
  largest = wave_max(largest);
  const auto weight = [&](int e) -> double {   // p, times a factor that is the same for the token where they are renormalized
    const double v = logit_at(row, e, kBf16);
    if (!a.sigmoid) return a.renormalize ? exp(v - largest) : exp(v - top) / sum;
    const double m = a.renormalize ? fmin(largest, 0.0) : 0.0;
    return v > 0 ? exp(-m) / (1 + exp(-v)) : exp(v - m) / (1 + exp(v));
  };
  double total = 0, dot = 0;
  for (int j = lane; j < a.top_k; j += 64)
    if (chosen(j) >= 0) {
      const double p = weight(chosen(j));
      total += p;
      dot += p * grads[j];
    }
  total = wave_add(total);
  dot = wave_add(dot);
  for (int j = lane; j < a.top_k; j += 64) {
    const int e = chosen(j);
    if (e < 0) continue;
    const double p = weight(e), v = logit_at(row, e, kBf16);
    double h = a.renormalize ? (total != 0 ? p / total * (grads[j] - dot / total) : 0.0) : p * grads[j];
    if (a.sigmoid) h *= v > 0 ? exp(-v) / (1 + exp(-v)) : 1 / (1 + exp(v));
    atomicAdd(d + e, (float)(h * a.scale));   // one addition for each expert, unless ids names one twice
  }
  __syncthreads();
  if (live) {
    char* const out = (char*)a.out + token * a.ld_out * (kBf16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int e = lane + 64 * i;
      if (e >= a.experts) continue;
      double v = d[e];
      if (dense) v -= exp(l[i] - top) / sum * dot * a.scale;
      if constexpr (kBf16) ((__bf16*)out)[e] = (__bf16)(float)v;
      else ((float*)out)[e] = (float)v;
    }
  }
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
  const int64_t step = rows_per_launch(64);
  for (int64_t t = 0; t < n_tokens; t += step) {
    const int64_t n = std::min(step, n_tokens - t);
    const RouteArgs a{(const char*)logits + t * ld_logits * (int64_t)es, ld_logits, (int)n, (int)n_experts, bias,
                      mask ? mask + t : mask, score == MXQ_SIGMOID, renormalize != 0, scale, (int)n_groups, (int)top_groups,
                      (int)group_top, (int)top_k, mxq_divisor((uint32_t)(n_experts / n_groups)), ids + t * top_k,
                      weights + t * top_k};
    const dim3 grid((uint32_t)((n + kTokens - 1) / kTokens)), block(64 * kTokens);
    if (dt == MXQ_BF16) hipLaunchKernelGGL((route_kernel<true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_kernel<false>), grid, block, 0, stream, a);
    const int rc = launch_status();
    if (rc != MXQ_OK) return rc;
  }
  return MXQ_OK;
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
  const int64_t step = rows_per_launch(64);
  for (int64_t t = 0; t < n_tokens; t += step) {
    const int64_t n = std::min(step, n_tokens - t);
    const BackArgs a{dweights + t * top_k, (const char*)logits + t * ld_logits * (int64_t)es, ld_logits, ids + t * top_k,
                     (int)n, (int)n_experts, (int)top_k, score == MXQ_SIGMOID, renormalize != 0, scale,
                     (char*)dlogits + t * ld_dlogits * (int64_t)es, ld_dlogits};
    const dim3 grid((uint32_t)((n + kTokens - 1) / kTokens)), block(64 * kTokens);
    if (dt == MXQ_BF16) hipLaunchKernelGGL((route_backward_kernel<true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_backward_kernel<false>), grid, block, 0, stream, a);
    const int rc = launch_status();
    if (rc != MXQ_OK) return rc;
  }
  return MXQ_OK;
}

}  // extern "C"
