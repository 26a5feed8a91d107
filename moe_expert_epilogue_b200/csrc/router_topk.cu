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
// One warp per token; lane i holds the V consecutive experts from i * V (V a
// power of two, 32 V >= E).
#include "common.cuh"
#include "launch.cuh"
#include "router.cuh"

namespace moe {

namespace {

template <class D, int V>
__global__ void __launch_bounds__(kThreads)
router_fwd(const typename D::T* __restrict__ logits, float* __restrict__ weights,
           int32_t* __restrict__ ids, const int32_t* __restrict__ valid, int64_t tokens, int E,
           int K, int64_t ld, bool softmax, bool normalise, float scale, int32_t* err) {
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const int64_t n = live_tokens(valid, tokens, err);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < n; t += step) {
    float v[V];
    int id;
    load_logits<D, V>(logits + t * ld, E, lane, v);
    const float w = route_token<V>(v, K, lane, softmax, normalise, scale, &id);
    if (lane < K) {
      weights[t * K + lane] = w;
      ids[t * K + lane] = id;
    }
  }
}

template <class D, int V>
__global__ void __launch_bounds__(kThreads)
router_bwd(const typename D::T* __restrict__ logits, const int32_t* __restrict__ ids,
           const float* __restrict__ gw, typename D::T* __restrict__ gl,
           const int32_t* __restrict__ valid, int64_t tokens, int E, int K, int64_t ld,
           int64_t ld_g, bool softmax, bool normalise, float scale, int32_t* err) {
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const int64_t n = live_tokens(valid, tokens, err);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < n; t += step) {
    const typename D::T* row = logits + t * ld;
    int id = lane < K ? __ldg(ids + t * K + lane) : -1;
    if (id >= E) {
      flag_error(err, MOE_DEVERR_MAP);
      id = -1;
    }
    const bool live = id >= 0;
    const float l = live ? load1<D>(row + id) : -kInf;
    const float g = live ? __ldg(gw + t * K + lane) * scale : 0.0f;
    float grad[V];
#pragma unroll
    for (int i = 0; i < V; ++i) grad[i] = 0.f;
    float d;
    if (softmax && !normalise) {
      float v[V], top = -kInf, s = 0.f;
      load_logits<D, V>(row, E, lane, v);
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
      top = warp_max(top);
      if (top == -kInf) top = 0.f;               // every expert closed: all terms are 0
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = expf(v[i] - top);
        s += v[i];
      }
      s = warp_sum(s);
      if (s == 0.0f) s = 1.0f;
      d = live ? expf(l - top) / s * g : 0.0f;
      const float dot = warp_sum(d);
#pragma unroll
      for (int i = 0; i < V; ++i) grad[i] = -(v[i] / s) * dot;
    } else {
      const float z = 1.0f / (1.0f + expf(-l));
      if (normalise) {
        const float top = warp_max(l);
        float w = live && l != -kInf ? chosen_score(softmax, l, top) : 0.0f;
        const float s = warp_sum(w);
        if (w != 0.0f) w = w / s;
        d = w * (g - warp_sum(w * g));
        if (!softmax) d *= 1.0f / (1.0f + expf(l));
      } else {
        d = live ? g * z * (1.0f / (1.0f + expf(l))) : 0.0f;
      }
    }
    if (!live) d = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int e = __shfl_sync(kAll, id, k);
      const float dk = __shfl_sync(kAll, d, k);
      if (e >= 0 && e / V == lane) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == e % V) grad[i] += dk;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < E) store1<D>(gl + t * ld_g + e, grad[i]);
    }
  }
}

template <class D, int V>
int launch_fwd(const void* logits, float* weights, int32_t* ids, const int32_t* valid,
               int64_t tokens, int E, int K, int64_t ld, bool softmax, bool normalise,
               float scale, int32_t* err, cudaStream_t stream) {
  auto k = router_fwd<D, V>;
  int grid = 0;
  const int64_t per = kThreads / 32;
  if (int rc = persistent_grid((const void*)k, 0, (tokens + per - 1) / per, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(logits), weights, ids,
                valid, tokens, E, K, ld, softmax, normalise, scale, err);
  return check_launch();
}

template <class D, int V>
int launch_bwd(const void* logits, const int32_t* ids, const float* gw, void* gl,
               const int32_t* valid, int64_t tokens, int E, int K, int64_t ld, int64_t ld_g,
               bool softmax, bool normalise, float scale, int32_t* err, cudaStream_t stream) {
  auto k = router_bwd<D, V>;
  int grid = 0;
  const int64_t per = kThreads / 32;
  if (int rc = persistent_grid((const void*)k, 0, (tokens + per - 1) / per, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(logits), ids, gw,
                static_cast<typename D::T*>(gl), valid, tokens, E, K, ld, ld_g, softmax,
                normalise, scale, err);
  return check_launch();
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
