// router.cuh -- the choice of a token's experts and their weights by one warp,
// shared by the router and the few-token expert layer.
#pragma once

#include <math.h>

#include "common.cuh"
#include "moe_epilogue.h"

namespace moe {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kInf = INFINITY;

// Image of a logit whose unsigned order is the selection's.  Adding +0 makes -0
// and +0 one and any NaN the positive one, which then lies above +inf; -inf and
// what is never a logit (0) do not lie above kDeadKey.
constexpr uint32_t kDeadKey = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float v) {
  const int32_t b = __float_as_int(__fadd_rn(v, 0.0f));
  return (uint32_t)(b ^ (b >> 31 | (int32_t)0x80000000));
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The logits of experts lane, lane + 32, ... of one row; -inf past E.
template <class D, int V>
__device__ __forceinline__ void load_logits(const typename D::T* row, int E, int lane,
                                            float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    v[i] = e < E ? load1<D>(row + e) : -kInf;
  }
}

// Sum over all experts of e^{l - top}, experts in the order of load_logits.
template <int V>
__device__ __forceinline__ float exp_sum(const float (&v)[V], float top) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += v[i] == -kInf ? 0.0f : expf(v[i] - top);
  return warp_sum(s);
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

// Routing weights of the choices in a warp: `lanes` neighbouring lanes (a power of
// two) hold a token's, in their order; value -inf and id -1 where there is none.
// all: softmax over all experts, the sum of e^{l - the token's largest l}.
__device__ __forceinline__ float choice_weight(float value, int id, int lanes, int lane,
                                               bool softmax, bool normalise, float scale,
                                               float all) {
  const float top = __shfl_sync(kAll, value, lane & ~(lanes - 1));   // the row's largest logit
  float w = id >= 0 ? chosen_score(softmax, value, top) : 0.0f;
  if (normalise) {
    float s = w;
    for (int o = lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    w = w / s;
  } else if (softmax) {
    w = w / all;
  } else if (id >= 0) {
    w = 1.0f / (1.0f + expf(-value));
  }
  return id >= 0 ? w * scale : 0.0f;
}

// The K choices of one token from its logits (as load_logits leaves them).  Lane k
// returns the weight of the k-th choice and its expert in *id (0 and -1 where
// nothing is left, or k >= K).  A choice waits for the one before: the chain of a
// round is the lanes' maximum, the lowest expert that has it, and its removal,
// without branches.
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
    if (top <= kDeadKey) break;
    unsigned first = ~0u;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) first = key[i] == top ? i * 32 + lane : first;
    const unsigned expert = __reduce_min_sync(kAll, first);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i * 32 + lane == (int)expert ? 0u : key[i];
    mine = lane == k ? key_value(top) : mine;
    id = lane == k ? (int)expert : id;
  }
  float all = 0.f;
  if (softmax && !normalise) all = exp_sum<V>(v, __shfl_sync(kAll, mine, 0));
  *id_out = id;
  return choice_weight(mine, id, 32, lane, softmax, normalise, scale, all);
}

}  // namespace moe
