// router_topk.cu -- the experts of each token: the K largest logits, their
// routing weights, and the gradient of the logits.
//
// Selection compares the logits themselves (softmax and sigmoid keep their
// order): the K largest, ties to the lowest expert, NaN above everything,
// -inf never (a slot that finds nothing else is id -1 with weight 0).
// With s the scale and C the chosen experts of a token:
//   softmax           w_i = s e^{l_i} / sum_j e^{l_j}       (all experts)
//   softmax, normal.  w_i = s e^{l_i} / sum_{j in C} e^{l_j}
//   sigmoid           w_i = s sig(l_i)
//   sigmoid, normal.  w_i = s sig(l_i) / sum_{j in C} sig(l_j)
// Backward, with g_i the gradient of w_i and v_i = w_i / s:
//   softmax           dl_j = v_j (s g_j [j in C] - sum_{i in C} s g_i v_i)
//   normalised        dl_i = v_i (s g_i - sum_{j in C} s g_j v_j) [times
//                            1 - sig(l_i) for the sigmoid],  0 outside C
//   sigmoid           dl_i = s g_i sig(l_i) (1 - sig(l_i)),  0 outside C
//
// The logits are read once and little is written: for many tokens the instructions
// bound the forward, not HBM.  router_fwd: one warp per token; lane i holds the
// experts i, i + 32, ...  Each lane sorts its logits once, so that a choice costs
// one maximum over the lanes and a shift in one of them, and the weights of as many
// tokens as fit a warp are computed together.  router_fwd_many: below.
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "router.cuh"

namespace moe {

namespace {

// A logit of a 16-bit type and its expert in one number whose order is the
// selection's: the upper half as order_key, the lower half falling with the
// expert, so that no two are equal.
template <class D>
__device__ __forceinline__ uint32_t pair_key(uint16_t raw, uint32_t low) {
  int32_t b;
  if (std::is_same<D, BF16>::value) {
    b = __float_as_int(__fadd_rn(__uint_as_float((uint32_t)raw << 16), 0.0f));
  } else {
    asm("add.rn.f16 %0, %0, %1;" : "+h"(raw) : "h"((uint16_t)0));
    b = (int32_t)((uint32_t)raw << 16);
  }
  return ((uint32_t)(b ^ (b >> 31 | (int32_t)0x80000000)) & 0xffff0000u) | low;
}

template <class D>
__device__ __forceinline__ float pair_value(uint32_t key) {
  const uint32_t m = key >> 16;
  const uint32_t bits = m & 0x8000u ? m ^ 0x8000u : m ^ 0xffffu;
  if (std::is_same<D, BF16>::value) return __uint_as_float(bits << 16);
  return f16_to_f32((uint16_t)bits);
}

// The logits of a lane, largest first.  take() removes the largest left in the
// warp and leaves it in `mine` of the lane asked; false if there is none.
struct Choice {
  uint32_t key = 0, at = 0;                                            // 0: none
};
template <class D, int V> struct Sorted {                              // 16-bit types
  uint32_t key[V];
  // -inf, as order_key leaves it
  static constexpr uint32_t kDead = std::is_same<D, BF16>::value ? 0x007fffffu : 0x03ffffffu;
  __device__ __forceinline__ void set(const uint16_t (&raw)[V], int E, int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < E ? pair_key<D>(raw[i], 0xffffu - e) : 0u;
    }
    if constexpr (V > 1) merge<0, 0>();
  }
  // Batcher's odd-even merge sort: steps of 2^Q within sorted runs of 2^P.
  template <int P, int Q> __device__ __forceinline__ void merge() {
    constexpr int kStep = 1 << Q, kSkip = Q == P ? 0 : kStep;
#pragma unroll
    for (int i = kSkip; i + kStep < V; ++i) {
      if (((i - kSkip) & (2 * kStep - 1)) < kStep && i >> (P + 1) == (i + kStep) >> (P + 1)) {
        const uint32_t lo = min(key[i], key[i + kStep]);
        key[i] = max(key[i], key[i + kStep]);
        key[i + kStep] = lo;
      }
    }
    if constexpr (Q > 0) merge<P, Q - 1>();
    else if constexpr (2 << P < V) merge<P + 1, P + 1>();
  }
  __device__ __forceinline__ bool take(Choice& mine, bool asked) {
    const uint32_t top = __reduce_max_sync(kAll, key[0]);
    if (top <= kDead) return false;
    if (key[0] == top) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0;
    }
    if (asked) mine.key = top;
    return true;
  }
  static __device__ __forceinline__ float value(const Choice& c) { return pair_value<D>(c.key); }
  static __device__ __forceinline__ int expert(const Choice& c) {
    return 0xffff - (int)(c.key & 0xffffu);
  }
};
template <int V> struct Sorted<F32, V> {
  uint32_t key[V];
  uint32_t at[V];                                                      // experts
  static constexpr uint32_t kDead = kDeadKey;
  static constexpr bool kSort = V <= 8;     // beyond, sorting costs more than looking
  __device__ __forceinline__ void set(const float (&raw)[V], int E, int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      at[i] = i * 32 + lane;
      key[i] = (int)at[i] < E ? order_key(raw[i]) : 0u;
    }
    if (kSort) {
      // neighbours are exchanged only when out of order: equal ones keep theirs
#pragma unroll
      for (int n = 0; n < V; ++n)
#pragma unroll
        for (int i = n & 1; i + 1 < V; i += 2) {
          const bool swap = key[i] < key[i + 1];
          const uint32_t k0 = key[i], a0 = at[i];
          key[i] = swap ? key[i + 1] : k0;
          key[i + 1] = swap ? k0 : key[i + 1];
          at[i] = swap ? at[i + 1] : a0;
          at[i + 1] = swap ? a0 : at[i + 1];
        }
    }
  }
  __device__ __forceinline__ bool take(Choice& mine, bool asked) {
    uint32_t best = key[0], first = ~0u;
    if (!kSort) {
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
    }
    const uint32_t top = __reduce_max_sync(kAll, best);
    if (top <= kDead) return false;
    if (kSort) {
      first = key[0] == top ? at[0] : ~0u;
    } else {
#pragma unroll
      for (int i = V - 1; i >= 0; --i) first = key[i] == top ? at[i] : first;
    }
    const uint32_t e = __reduce_min_sync(kAll, first);
    if (kSort) {
      if (first == e) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) {
          key[i] = key[i + 1];
          at[i] = at[i + 1];
        }
        key[V - 1] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = at[i] == e ? 0u : key[i];
    }
    if (asked) {
      mine.key = top;
      mine.at = e;
    }
    return true;
  }
  static __device__ __forceinline__ float value(const Choice& c) { return key_value(c.key); }
  static __device__ __forceinline__ int expert(const Choice& c) { return (int)c.at; }
};

// `lanes`: K up to a power of two; `group` (a power of two, up to 32 / lanes)
// neighbouring tokens per warp.
template <class D, int V>
__global__ void __launch_bounds__(kThreads)
router_fwd(const typename D::T* __restrict__ logits, float* __restrict__ weights,
           int32_t* __restrict__ ids, const int32_t* __restrict__ valid, int64_t tokens, int E,
           int K, int lanes, int group, int64_t ld, bool softmax, bool normalise, float scale,
           int32_t* err) {
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const int64_t n = live_tokens(valid, tokens, err);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * group;
  for (int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * group; t0 < n;
       t0 += step) {
    Choice mine;                        // lane g * lanes + k: the k-th choice of token t0 + g
    float all = 0.f;
    for (int g = 0; g < group && t0 + g < n; ++g) {
      const typename D::T* row = logits + (t0 + g) * ld;
      typename D::T raw[V];
#pragma unroll
      for (int i = 0; i < V; ++i) raw[i] = i * 32 + lane < E ? __ldg(row + i * 32 + lane) : 0;
      Sorted<D, V> left;
      left.set(raw, E, lane);
      for (int k = 0; k < K; ++k)
        if (!left.take(mine, lane == g * lanes + k)) break;
      if (softmax && !normalise) {
        float v[V];
        load_logits<D, V>(row, E, lane, v);
        const float first = __shfl_sync(kAll, Sorted<D, V>::value(mine), g * lanes);
        const float s = exp_sum<V>(v, first);
        all = lane / lanes == g ? s : all;
      }
    }
    const int id = mine.key ? Sorted<D, V>::expert(mine) : -1;
    const float value = mine.key ? Sorted<D, V>::value(mine) : -kInf;
    const float w = choice_weight(value, id, lanes, lane, softmax, normalise, scale, all);
    const int64_t t = t0 + lane / lanes;
    const int k = lane & (lanes - 1);
    if (k < K && lane / lanes < group && t < n) {
      weights[t * K + k] = w;
      ids[t * K + k] = id;
    }
  }
}

// Many tokens: four or eight lanes to a token.  A lane takes eight experts at a
// time, sorts them and keeps the eight largest of these and of those it has (the
// larger of one list's i-th and the other's i-th from the end, then the end of a
// bitonic sort); two or three such steps between the lanes leave every lane the
// token's eight.  K <= 8.  About half of the instructions of the rounds above: 32768
// x 256, K = 8, bf16 16.6 us there and 10.8 here, fp32 24.2 and 18.0.
// A key is a logit and its expert in one number: pair_key, and of fp32 the upper 22
// bits of order_key with 0x3ff - expert (E <= 1024).  These order all but logits
// that agree in 22 bits; so of fp32 the eight are ordered once more by their whole
// logits, and a token whose ninth largest key shares the eighth's upper part is
// chosen again, expert by expert.  (Keys of 64 bits: 32768 x 256 26.1 us.)
template <bool NINTH>
struct Eight {
  uint32_t key[8];                                                     // largest first
  uint32_t ninth = 0;                                                  // largest left out
  __device__ __forceinline__ void order(int i, int j) {
    const uint32_t lo = min(key[i], key[j]);
    key[i] = max(key[i], key[j]);
    key[j] = lo;
  }
  __device__ __forceinline__ void sort() {                             // Batcher's, 19 steps
#pragma unroll
    for (int p = 1; p < 8; p *= 2)
#pragma unroll
      for (int q = p; q > 0; q /= 2)
#pragma unroll
        for (int i = q == p ? 0 : q; i + q < 8; ++i)
          if (((i - (q == p ? 0 : q)) & (2 * q - 1)) < q && i / (2 * p) == (i + q) / (2 * p))
            order(i, i + q);
  }
  __device__ __forceinline__ void keep(const uint32_t (&other)[8]) {   // also largest first
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (NINTH) ninth = max(ninth, min(key[i], other[7 - i]));
      key[i] = max(key[i], other[7 - i]);
    }
#pragma unroll
    for (int o = 4; o > 0; o /= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & o)) order(i, i + o);
  }
};

// pair_key of two logits at once.
template <class D>
__device__ __forceinline__ void pair_keys(uint32_t raw, uint32_t low, uint32_t& k0, uint32_t& k1) {
  if (std::is_same<D, BF16>::value) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(raw) : "r"(0u));
  else asm("add.rn.f16x2 %0, %0, %1;" : "+r"(raw) : "r"(0u));
  const uint32_t m = raw ^ ((raw >> 15 & 0x00010001u) * 0xffffu | 0x80008000u);
  k0 = __byte_perm(m, low, 0x1054);
  k1 = __byte_perm(m, low, 0x3276);
}

// Whether a logit of the token has one of the bits that the keys leave out.  Only asked of tokens
// whose keys do not decide: asked of all of them, 32768 x 256 random logits take 18.3 us instead
// of 18.0 (17.7 where it is not asked; logits from bf16 17.0, 17.2 and 27.7).
__device__ __forceinline__ bool lower_bits(const float* row, int E, int lane) {
  uint32_t bits = 0;
  for (int e = lane; e < E; e += 32) bits |= __float_as_uint(__ldg(row + e));
  return __any_sync(kAll, bits & 0x3ffu);
}

// The eight choices of one fp32 token by the whole warp, in the order of (logit, expert).
__device__ __forceinline__ void choose_again(const float* row, int E, int lane, uint32_t* key,
                                             uint16_t* who) {
  uint32_t last = ~0u, last_at = ~0u;
  for (int k = 0; k < 8; ++k) {
    uint32_t best = 0, at = ~0u;
    for (int e = lane; e < E; e += 32) {
      const uint32_t v = order_key(__ldg(row + e));
      const bool left = v < last || (v == last && (k == 0 || (uint32_t)e > last_at));
      if (left && v > best) {
        best = v;
        at = e;
      }
    }
    last = __reduce_max_sync(kAll, best);
    last_at = __reduce_min_sync(kAll, best == last ? at : ~0u);
    if (lane == 0) {
      key[k] = last;
      who[k] = (uint16_t)last_at;
    }
  }
}

// LANES to a token; WIDE: rows of whole 16-byte words.
template <class D, bool WIDE, int LANES>
__global__ void __launch_bounds__(kThreads)
router_fwd_many(const typename D::T* __restrict__ logits, float* __restrict__ weights,
                int32_t* __restrict__ ids, const int32_t* __restrict__ valid, int64_t tokens,
                int E, int K, int lanes, int64_t ld, bool softmax, bool normalise, float scale,
                int32_t* err) {
  constexpr bool kHalf = D::kBytes == 2;
  constexpr int kWords = 2 * D::kBytes;                                // of eight logits
  constexpr uint32_t kClosed =                                         // a word of -inf
      std::is_same<D, BF16>::value ? 0xff80ff80u : kHalf ? 0xfc00fc00u : 0xff800000u;
  constexpr uint32_t kDead = Sorted<D, 1>::kDead;
  constexpr int kWarpTokens = 32 / LANES;
  __shared__ uint32_t chosen[kThreads / 32][kWarpTokens][8];
  __shared__ uint16_t who[kThreads / 32][kWarpTokens][kHalf ? 1 : 8];  // of fp32: the experts
  __shared__ float sums[kThreads / 32][kWarpTokens];
  pdl_prologue();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = live_tokens(valid, tokens, err);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32) * kWarpTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + warp) * kWarpTokens; t0 < n;
       t0 += step) {
    const int64_t t = t0 + lane / LANES;
    const typename D::T* row = logits + t * ld;
    const auto load = [&](int e, uint32_t (&raw)[kWords]) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) raw[i] = kClosed;
      if (t >= n) return;
      if constexpr (WIDE) {
        if (e < E) {
#pragma unroll
          for (int i = 0; i < kWords; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e) + i / 4);
            raw[i] = v.x; raw[i + 1] = v.y; raw[i + 2] = v.z; raw[i + 3] = v.w;
          }
        }
      } else if constexpr (kHalf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = e + 2 * i < E ? __ldg(row + e + 2 * i) : kClosed & 0xffffu;
          const uint32_t b = e + 2 * i + 1 < E ? __ldg(row + e + 2 * i + 1) : kClosed & 0xffffu;
          raw[i] = a | b << 16;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < E) raw[i] = __float_as_uint(__ldg(row + e + i));
      }
    };
    Eight<!kHalf> top;
    int e = (lane & (LANES - 1)) * 8;
    uint32_t next[kWords];
    load(e, next);
    for (int e0 = 0; e0 < E; e0 += 8 * LANES, e += 8 * LANES) {
      Eight<!kHalf> some;
      if constexpr (kHalf) {
        // the lower half of a key: 0xffff - expert
        const uint32_t low = (0xffffu - e) | (0xfffeu - e) << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pair_keys<D>(next[i], low - i * 0x00020002u, some.key[2 * i], some.key[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          some.key[i] = (order_key(__uint_as_float(next[i])) & ~0x3ffu) | (~(e + i) & 0x3ff);
        }
      }
      if (e0 + 8 * LANES < E) load(e + 8 * LANES, next);
      some.sort();
      if (e0 == 0) top = some;
      else top.keep(some.key);
    }
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) {
      uint32_t other[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, top.key[i], o);
      if (!kHalf) top.ninth = max(top.ninth, __shfl_xor_sync(kAll, top.ninth, o));
      top.keep(other);
    }
    if ((lane & (LANES - 1)) == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) chosen[warp][lane / LANES][i] = top.key[i];
    }
    __syncwarp();
    if constexpr (!kHalf) {
#pragma unroll
      for (int at = lane; at < 8 * kWarpTokens; at += 32) {
        const int g = at / 8, k = at & 7;
        const uint32_t key = chosen[warp][g][k], expert = ~key & 0x3ffu;
        const uint32_t whole =
            key > kDead ? order_key(__ldg(logits + (t0 + g) * ld + expert)) : 0u;
        int place = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t v = __shfl_sync(kAll, whole, j, 8);
          place += v > whole || (v == whole && j < k);       // equal ones are in order already
        }
        __syncwarp();
        chosen[warp][g][place] = whole;
        who[warp][g][place] = (uint16_t)expert;
      }
      const bool unsure = top.key[7] > kDead && top.ninth >> 10 == top.key[7] >> 10;
      uint32_t tokens_left = __ballot_sync(kAll, unsure && (lane & (LANES - 1)) == 0);
      __syncwarp();
      for (; tokens_left; tokens_left &= tokens_left - 1) {
        const int g = (__ffs(tokens_left) - 1) / LANES;
        const typename D::T* unsure_row = logits + (t0 + g) * ld;
        // (of logits without lower bits, say from a 16-bit type, the keys hold all)
        if (lower_bits(unsure_row, E, lane))
          choose_again(unsure_row, E, lane, chosen[warp][g], who[warp][g]);
      }
      __syncwarp();
    }
    const auto value = [&](uint32_t key) {
      if constexpr (kHalf) return pair_value<D>(key);
      else return key_value(key);
    };
    if (softmax && !normalise) {
      // as exp_sum, four tokens at a time; a token past the last repeats it
      for (int g0 = 0; g0 < kWarpTokens && t0 + g0 < n; g0 += 4) {
        const typename D::T* from[4];
        float first[4], s[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int g = t0 + g0 + j < n ? g0 + j : g0;
          from[j] = logits + (t0 + g) * ld;
          first[j] = value(chosen[warp][g][0]);
        }
        for (int i = lane; i < E; i += 32) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v = load1<D>(from[j] + i);
            s[j] += v == -kInf ? 0.0f : expf(v - first[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = warp_sum(s[j]);
        if (lane < 4)
          sums[warp][g0 + lane] = lane & 2 ? lane & 1 ? s[3] : s[2] : lane & 1 ? s[1] : s[0];
      }
      __syncwarp();
    }
    for (int at = lane; at - lane < kWarpTokens * lanes; at += 32) {
      const int g = at / lanes, k = at & (lanes - 1);
      const bool mine = g < kWarpTokens && k < K && t0 + g < n;
      const uint32_t key = mine ? chosen[warp][g][k] : 0u;
      const bool some = key > kDead;
      int id = -1;
      if (some) id = kHalf ? 0xffff - (int)(key & 0xffffu) : who[warp][g][kHalf ? 0 : k];
      const float all = softmax && !normalise && mine ? sums[warp][g] : 1.0f;
      const float w = choice_weight(some ? value(key) : -kInf, id, lanes, lane, softmax, normalise,
                                    scale, all);
      if (mine) {
        weights[(t0 + g) * K + k] = w;
        ids[(t0 + g) * K + k] = id;
      }
    }
    __syncwarp();
  }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// LANES to a token: lane i of them holds the experts i, i + LANES, ... (V at most)
// and the i-th choice.
template <class D, int V, int LANES>
__global__ void __launch_bounds__(kThreads)
router_bwd(const typename D::T* __restrict__ logits, const int32_t* __restrict__ ids,
           const float* __restrict__ gw, typename D::T* __restrict__ gl,
           const int32_t* __restrict__ valid, int64_t tokens, int E, int K, int64_t ld,
           int64_t ld_g, bool softmax, bool normalise, float scale, int32_t* err) {
  constexpr int kTokens = 32 / LANES;
  pdl_prologue();
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t n = live_tokens(valid, tokens, err);
  const int64_t step = (int64_t)gridDim.x * (kThreads / LANES);
  for (int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kTokens; t0 < n;
       t0 += step) {
    const int64_t t = t0 + (threadIdx.x & 31) / LANES;
    const int open = t < n ? E : 0;           // experts of this token to read and write
    const typename D::T* row = logits + t * ld;
    int id = open > 0 && lane < K ? __ldg(ids + t * K + lane) : -1;
    if (id >= E) {
      flag_error(err, MOE_DEVERR_MAP);
      id = -1;
    }
    const bool live = id >= 0;
    const float l = live ? load1<D>(row + id) : -kInf;
    const float g = live ? __ldg(gw + t * K + lane) * scale : 0.0f;
    typename D::T* out = gl + t * ld_g;
    float d;                  // gradient of the lane's own choice, beside that of every expert:
    float rest = 0.0f;
    if (softmax && !normalise) {
      float v[V], top = -kInf, s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * LANES + lane;
        v[i] = e < open ? load1<D>(row + e) : -kInf;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
      top = lanes_max<LANES>(top);
      if (top == -kInf) top = 0.f;               // every expert closed: all terms are 0
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i * LANES >= E) break;
        v[i] = expf(v[i] - top);
        s += v[i];
      }
      s = lanes_sum<LANES>(s);
      const float inv = s == 0.0f ? 1.0f : 1.0f / s;
      const float p = live ? expf(l - top) * inv : 0.0f;
      d = p * g;
      const float dot = lanes_sum<LANES>(d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * LANES + lane;
        if (e < open) store1<D>(out + e, -(v[i] * inv) * dot);
      }
      rest = -p * dot;
    } else {
      const float z = 1.0f / (1.0f + expf(-l));
      if (normalise) {
        const float top = lanes_max<LANES>(l);
        float w = live && l != -kInf ? chosen_score(softmax, l, top) : 0.0f;
        const float s = lanes_sum<LANES>(w);
        if (w != 0.0f) w = w / s;
        d = w * (g - lanes_sum<LANES>(w * g));
        if (!softmax) d *= 1.0f / (1.0f + expf(l));
      } else {
        d = live ? g * z * (1.0f / (1.0f + expf(l))) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * LANES + lane;
        if (e < open) store1<D>(out + e, 0.0f);
      }
    }
    // The choices' own entries, once the row is written: an expert named twice has both
    // gradients (each of its lanes stores the same sum).
    float sum = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int e = __shfl_sync(kAll, id, k, LANES);
      const float dk = __shfl_sync(kAll, d, k, LANES);
      if (e == id) sum += dk;
    }
    __syncwarp();
    if (live) store1<D>(out + id, rest + sum);
  }
}

template <class D, int V>
int launch_fwd(const void* logits, float* weights, int32_t* ids, const int32_t* valid,
               int64_t tokens, int E, int K, int64_t ld, bool softmax, bool normalise,
               float scale, int32_t* err, cudaStream_t stream) {
  int lanes = 1, grid = 0;
  while (lanes < K) lanes *= 2;
  // Fewer tokens leave its warps waiting for themselves (2048 x 256 bf16: 2.8 us a token a
  // warp, 3.1 with eight lanes to a token; 4096: 4.0 and 3.2; fp32 4096: 5.0 and 5.9, 8192: 8.2 and
  // 7.5).  Four lanes need fewer steps between lanes, eight more of them at once (16384 x 256:
  // 6.6 us both, 32768: 10.7 with four, 11.9 with eight), and the sums over all experts wait less
  // with fewer tokens a warp (32768: 19.0 and 18.0), as do the second looks of fp32 (19.0 and
  // 17.9; of 512 experts 31.9 and 32.4).
  constexpr bool kHalf = D::kBytes == 2;
  if (K <= 8 && tokens >= (kHalf ? 4096 : 8192)) {
    const bool wide =
        ((reinterpret_cast<uintptr_t>(logits) & 15) | (ld * D::kBytes & 15) | (E & 7)) == 0;
    const bool four = kHalf && tokens > 16384 && !(softmax && !normalise);
    constexpr int kFour = kHalf ? 4 : 8;
    const auto k = four ? wide ? router_fwd_many<D, true, kFour> : router_fwd_many<D, false, kFour>
                        : wide ? router_fwd_many<D, true, 8> : router_fwd_many<D, false, 8>;
    const int64_t per = kThreads / (four ? 4 : 8);
    if (int rc = persistent_grid((const void*)k, 0, (tokens + per - 1) / per, &grid)) return rc;
    launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(logits), weights, ids,
                  valid, tokens, E, K, lanes, ld, softmax, normalise, scale, err);
    return check_launch();
  }
  auto k = router_fwd<D, V>;
  // one token a warp as long as there are warps for them, which is quicker for each token (K > 8)
  const int group = tokens > 16384 ? 32 / lanes : 1;
  const int64_t per = (int64_t)(kThreads / 32) * group;
  if (int rc = persistent_grid((const void*)k, 0, (tokens + per - 1) / per, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(logits), weights, ids,
                valid, tokens, E, K, lanes, group, ld, softmax, normalise, scale, err);
  return check_launch();
}

template <class D, int V, int LANES>
int launch_bwd_lanes(const void* logits, const int32_t* ids, const float* gw, void* gl,
                     const int32_t* valid, int64_t tokens, int E, int K, int64_t ld, int64_t ld_g,
                     bool softmax, bool normalise, float scale, int32_t* err,
                     cudaStream_t stream) {
  auto k = router_bwd<D, V, LANES>;
  int grid = 0;
  const int64_t per = kThreads / LANES;
  if (int rc = persistent_grid((const void*)k, 0, (tokens + per - 1) / per, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(logits), ids, gw,
                static_cast<typename D::T*>(gl), valid, tokens, E, K, ld, ld_g, softmax,
                normalise, scale, err);
  return check_launch();
}

// Eight lanes to a token, above 128 experts sixteen, where the choices fit them: the steps that
// do not grow with the experts serve four or two tokens at once (32768 tokens, all experts'
// softmax, bf16: of 64 experts 11.7 us with 32 lanes, 7.3 with 16, 5.6 with 8; of 256 16.6, 14.2
// and 15.4).  Not by the number of tokens: a token's sums have the same order in every batch.
template <class D, int V, typename... Args>
int launch_bwd(const void* logits, const int32_t* ids, const float* gw, void* gl,
               const int32_t* valid, int64_t tokens, int E, int K, Args... args) {
  constexpr int kLanes = V <= 4 ? 8 : V <= 16 ? 16 : 32;
  if (K <= kLanes)
    return launch_bwd_lanes<D, V * 32 / kLanes, kLanes>(logits, ids, gw, gl, valid, tokens, E, K,
                                                        args...);
  return launch_bwd_lanes<D, V, 32>(logits, ids, gw, gl, valid, tokens, E, K, args...);
}

#define MOE_ROUTER_WIDTHS(F, D, ...)                    \
  (E <= 32    ? F<D, 1>(__VA_ARGS__)                    \
   : E <= 64  ? F<D, 2>(__VA_ARGS__)                    \
   : E <= 128 ? F<D, 4>(__VA_ARGS__)                    \
   : E <= 256 ? F<D, 8>(__VA_ARGS__)                    \
   : E <= 512 ? F<D, 16>(__VA_ARGS__)                   \
              : F<D, 32>(__VA_ARGS__))
#define MOE_ROUTER_DISPATCH(F, ...)                               \
  switch (dt) {                                                   \
    case MOE_BF16: return MOE_ROUTER_WIDTHS(F, BF16, __VA_ARGS__); \
    case MOE_FP16: return MOE_ROUTER_WIDTHS(F, F16, __VA_ARGS__);  \
    default: return MOE_ROUTER_WIDTHS(F, F32, __VA_ARGS__);        \
  }

}  // namespace

int launch_router_topk_fwd(const void* logits, moe_dtype dt, float* weights, int32_t* ids,
                           const int32_t* valid, int64_t tokens, int E, int K, int64_t ld,
                           bool softmax, bool normalise, float scale, int32_t* err,
                           cudaStream_t stream) {
  MOE_ROUTER_DISPATCH(launch_fwd, logits, weights, ids, valid, tokens, E, K, ld, softmax,
                      normalise, scale, err, stream)
}

int launch_router_topk_bwd(const void* logits, moe_dtype dt, const int32_t* ids, const float* gw,
                           void* gl, const int32_t* valid, int64_t tokens, int E, int K,
                           int64_t ld, int64_t ld_g, bool softmax, bool normalise, float scale,
                           int32_t* err, cudaStream_t stream) {
  MOE_ROUTER_DISPATCH(launch_bwd, logits, ids, gw, gl, valid, tokens, E, K, ld, ld_g, softmax,
                      normalise, scale, err, stream)
}

}  // namespace moe
