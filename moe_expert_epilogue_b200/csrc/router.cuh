// router.cuh -- the choice of a token's experts and their weights by one warp,
// shared by the router and the few-token expert layer.
#pragma once

#include <math.h>

#include "common.cuh"
#include "moe_epilogue.h"

namespace moe {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kInf = INFINITY;

// Image of a logit whose unsigned order is the selection's: 0 for -inf (never
// chosen), all ones for NaN; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v == -kInf ? 0u : b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The logits of experts [lane * V, lane * V + V) of one row; -inf past E.
template <class D, int V>
__device__ __forceinline__ void load_logits(const typename D::T* row, int E, int lane,
                                            float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    v[i] = e < E ? load1<D>(row + e) : -kInf;
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// The number of live tokens: *valid clamped to [0, tokens].
__device__ __forceinline__ int64_t live_tokens(const int32_t* valid, int64_t tokens,
                                               int32_t* err) {
  if (!valid) return tokens;
  const int64_t n = *valid;
  if (n < 0 || n > tokens) {
    flag_error(err, MOE_DEVERR_COUNT);
    return n < 0 ? 0 : tokens;
  }
  return n;
}

// Score of one chosen expert relative to the others of its token, up to a
// common factor: e^{l - max}, or sig(l); far below 0, where sig(l) = e^l to
// the last bit, the common factor e^{max} keeps it from underflowing.
__device__ __forceinline__ float chosen_score(bool softmax, float v, float top) {
  if (softmax || top < -40.0f) return expf(v - top);
  return 1.0f / (1.0f + expf(-v));
}

// The K choices of M tokens from their logits, side by side (lane i holds experts
// i * V .. i * V + V - 1 in v[m], -inf past the last).  Lane k gets the weight of
// the k-th choice and its expert (-1 and 0 where nothing is left, or k >= K).
template <int V, int M>
__device__ __forceinline__ void route_tokens(const float (&v)[M][V], int K, int lane,
                                             bool softmax, bool normalise, float scale,
                                             int (&id)[M], float (&w)[M]) {
  uint32_t key[M][V];
  float mine[M];           // lane k: logit of the k-th choice
#pragma unroll
  for (int m = 0; m < M; ++m) {
    mine[m] = -kInf;
    id[m] = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) key[m][i] = order_key(v[m][i]);
  }
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) best = max(best, key[m][i]);
      const uint32_t top = __reduce_max_sync(kAll, best);
      if (M == 1 && top == 0) { k = K; break; }
      // the lowest lane, and in it the lowest expert, that holds the largest key
      const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
      int at = 0;
      if (lane == src) {
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[m][i] == top) at = i;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == at) key[m][i] = 0;
      }
      at = __shfl_sync(kAll, at, src);
      if (lane == k && top != 0) {
        mine[m] = key_value(top);
        id[m] = src * V + at;
      }
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float top = __shfl_sync(kAll, mine[m], 0);   // the row's largest logit
    float x = id[m] >= 0 ? chosen_score(softmax, mine[m], top) : 0.0f;
    if (softmax && !normalise) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[m][i] == -kInf ? 0.0f : expf(v[m][i] - top);
      x = x / warp_sum(s);
    } else if (normalise) {
      x = x / warp_sum(x);
    } else if (id[m] >= 0) {
      x = 1.0f / (1.0f + expf(-mine[m]));
    }
    w[m] = id[m] >= 0 ? x * scale : 0.0f;
  }
}

}  // namespace moe
