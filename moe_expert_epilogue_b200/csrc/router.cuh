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

// The K choices of one token from its logits (lane i holds experts i * V ..
// i * V + V - 1 in v, -inf past the last).  Lane k returns the weight of the
// k-th choice and its expert in *id (0 and -1 where nothing is left, or k >= K).
// A choice waits for the one before: the chain of a round is the lanes' maximum,
// the vote on who holds it, and the removal, without branches.
template <int V>
__device__ __forceinline__ float route_token(const float (&v)[V], int K, int lane, bool softmax,
                                             bool normalise, float scale, int* id_out) {
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
  float mine = -kInf;      // lane k: logit and expert of the k-th choice
  int id = -1;
  for (int k = 0; k < K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    if (top == 0) break;
    // the lowest lane, and in it the lowest expert, that holds the largest key
    const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
    bool here = lane == src;
    int expert = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool hit = here && key[i] == top;
      key[i] = hit ? 0u : key[i];
      expert = hit ? lane * V + i : expert;
      here = here && !hit;
    }
    expert = __shfl_sync(kAll, expert, src);
    mine = lane == k ? key_value(top) : mine;
    id = lane == k ? expert : id;
  }
  const float top = __shfl_sync(kAll, mine, 0);   // the row's largest logit
  float w = id >= 0 ? chosen_score(softmax, mine, top) : 0.0f;
  if (softmax && !normalise) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += v[i] == -kInf ? 0.0f : expf(v[i] - top);
    w = w / warp_sum(s);
  } else if (normalise) {
    w = w / warp_sum(w);
  } else if (id >= 0) {
    w = 1.0f / (1.0f + expf(-mine));
  }
  *id_out = id;
  return id >= 0 ? w * scale : 0.0f;
}

}  // namespace moe
