// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens.
//
//   logits = x router_weight^T                     (64-bit sums, rounded to fp32)
//   choice and weights of each token's experts     (router.cuh)
//   z = w1[e] x,  h = p silu(min(z_gate, L)) clamp(z_up, -L, L)
//   out = residual + (sum over the chosen experts, ascending, of w2[e] h + shared)
//
// A decode step reads every chosen expert's 3 * inter * hidden weights once and
// computes almost nothing with them: HBM bandwidth bounds it.  Two kernels: the
// logits (which also clears the second kernel's counters), then one cooperative
// kernel with one CTA per SM for everything else, its phases separated by grid
// barriers: choice (every CTA makes the same tables for itself), first product
// and activation, second product, combine.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "router.cuh"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int kMaxTokens = 128, kMaxSlots = 1024, kMaxLayerExperts = 512;
constexpr int kUnitTokens = 32;                        // tokens of one unit at most
constexpr int kMaxUnits = kMaxLayerExperts + kMaxSlots / kUnitTokens;
constexpr int kBarriers = 2;

// One expert and up to kUnitTokens of its tokens: a row of the product's work.
struct Unit { uint16_t expert, first, count; };

// The choice, as every CTA holds it: slots are (token, k) pairs, token-major;
// `order` lists the live ones by ascending expert (then by slot), and the
// intermediate rows in the workspace are indexed by position in `order`.
struct Tables {
  float weight[kMaxSlots];       // by slot
  int16_t expert[kMaxSlots];     // by slot; -1: none
  uint16_t order[kMaxSlots];     // position -> slot
  uint16_t position[kMaxSlots];  // slot -> position
  uint8_t rank[kMaxSlots];       // by slot: k-th place -> k of the token's place-th lowest expert
  uint8_t live[kMaxTokens];      // live slots of a token
  uint16_t count[kMaxLayerExperts], first[kMaxLayerExperts];
  Unit unit[kMaxUnits];
  int units;
  int tokens;
};

// Everything a call works on.
struct Layer {
  const void *x, *router_w, *logits, *w1, *w2, *shared, *residual;
  void* out;
  float* topk_weights;
  int32_t* topk_ids;
  const int32_t* valid;
  int tokens, hidden, inter, E, K;
  int64_t ld_x, ld_logits, ld_shared, ld_residual, ld_out;
  int logits_dt;
  bool router_f32, softmax, normalise;
  float scale, limit;
  int32_t* err;
  // workspace
  unsigned* barrier;     // [kBarriers]
  float* own_logits;     // [tokens, E]
  uint16_t* h;           // [slots, 2, inter]: the activation's high and low halves
  float* y;              // [slots, hidden]
};

// ------------------------------------------------------------ logits

constexpr int kLogitTokens = 4;   // tokens per CTA of the logits kernel

// One expert and kLogitTokens tokens per CTA.  The products and their sum are
// in 64 bits, so that the summation order cannot decide between two experts:
// a choice depends on the inputs alone.
template <class D, class R>
__global__ void __launch_bounds__(kThreads)
layer_logits(Layer a) {
  pdl_prologue();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kBarriers) a.barrier[threadIdx.x] = 0;
  if (!a.router_w) return;
  __shared__ double red[kThreads / 32][kLogitTokens];
  const int e = blockIdx.x, t0 = blockIdx.y * kLogitTokens;
  const auto* w = static_cast<const typename R::T*>(a.router_w) + (int64_t)e * a.hidden;
  const auto* x = static_cast<const typename D::T*>(a.x);
  double acc[kLogitTokens] = {};
  for (int h = threadIdx.x; h < a.hidden; h += kThreads) {
    const double wv = load1<R>(w + h);
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i)
      if (t0 + i < a.tokens) acc[i] += wv * (double)load1<D>(x + (t0 + i) * a.ld_x + h);
  }
#pragma unroll
  for (int i = 0; i < kLogitTokens; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(kAll, acc[i], o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][i] = acc[i];
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i < kLogitTokens && t0 + i < a.tokens) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) s += red[k][i];
    a.own_logits[(int64_t)(t0 + i) * a.E + e] = (float)s;
  }
}

// ------------------------------------------------------------ choice

template <int V>
__device__ void choose_token(const Layer& a, Tables& tb, int t, int lane) {
  float v[V];
  const int64_t row = (int64_t)t * a.ld_logits;
  if (a.logits_dt == MOE_FP32)
    load_logits<F32, V>(static_cast<const float*>(a.logits) + row, a.E, lane, v);
  else if (a.logits_dt == MOE_BF16)
    load_logits<BF16, V>(static_cast<const uint16_t*>(a.logits) + row, a.E, lane, v);
  else
    load_logits<F16, V>(static_cast<const uint16_t*>(a.logits) + row, a.E, lane, v);
  int id;
  const float w = route_token<V>(v, a.K, lane, a.softmax, a.normalise, a.scale, &id);
  int place = 0;             // how many of the token's live experts are lower
  for (int k = 0; k < a.K; ++k) {
    const int other = __shfl_sync(kAll, id, k);
    place += other >= 0 && other < id;
  }
  const unsigned live = __ballot_sync(kAll, id >= 0);
  if (lane < a.K) {
    const int slot = t * a.K + lane;
    tb.expert[slot] = (int16_t)id;
    tb.weight[slot] = w;
    if (id >= 0) tb.rank[t * a.K + place] = (uint8_t)lane;
    if (blockIdx.x == 0) {
      if (a.topk_weights) a.topk_weights[slot] = w;
      if (a.topk_ids) a.topk_ids[slot] = id;
    }
  }
  if (lane == 0) tb.live[t] = (uint8_t)__popc(live);
}

// Fills the tables; all `threads` threads of the CTA take part.
__device__ void make_tables(const Layer& a, Tables& tb, int threads) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int live = (int)live_tokens(a.valid, a.tokens, a.err);
  for (int e = threadIdx.x; e < a.E; e += threads) tb.count[e] = 0;
  if (threadIdx.x == 0) tb.tokens = live;
  for (int t = warp; t < live; t += threads / 32) {
    if (a.E <= 64) choose_token<2>(a, tb, t, lane);
    else if (a.E <= 256) choose_token<8>(a, tb, t, lane);
    else choose_token<16>(a, tb, t, lane);
  }
  __syncthreads();
  if (warp == 0) {
    // each slot's place among its expert's, in slot order
    const int slots = live * a.K;
    for (int s0 = 0; s0 < slots; s0 += 32) {
      const int e = s0 + lane < slots ? tb.expert[s0 + lane] : -1;
      const unsigned peers = __match_any_sync(kAll, e);
      const int before = e >= 0 ? tb.count[e] : 0;
      __syncwarp();
      if (e >= 0) {
        tb.position[s0 + lane] = (uint16_t)(before + __popc(peers & ((1u << lane) - 1u)));
        if (lane == 31 - __clz(peers)) tb.count[e] = (uint16_t)(before + __popc(peers));
      }
      __syncwarp();
    }
    // the experts' first positions and units
    int base = 0, units = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane, n = e < a.E ? tb.count[e] : 0;
      const int u = (n + kUnitTokens - 1) / kUnitTokens;
      int sn = n, su = u;                                   // inclusive prefix sums
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int pn = __shfl_up_sync(kAll, sn, o), pu = __shfl_up_sync(kAll, su, o);
        if (lane >= o) { sn += pn; su += pu; }
      }
      if (e < a.E) {
        const int first = base + sn - n;
        tb.first[e] = (uint16_t)first;
        for (int i = 0; i < u; ++i)
          tb.unit[units + su - u + i] = {(uint16_t)e, (uint16_t)(first + i * kUnitTokens),
                                         (uint16_t)min(kUnitTokens, n - i * kUnitTokens)};
      }
      base += __shfl_sync(kAll, sn, 31);
      units += __shfl_sync(kAll, su, 31);
    }
    if (lane == 0) tb.units = units;
    __syncwarp();
    for (int s = lane; s < slots; s += 32) {
      const int e = tb.expert[s];
      if (e >= 0) {
        const int p = tb.first[e] + tb.position[s];
        tb.position[s] = (uint16_t)p;
        tb.order[p] = (uint16_t)s;
      }
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------ grid barrier

// All CTAs' writes before are visible to all CTAs after.  The launch is
// cooperative, so every CTA is resident; the wait is bounded all the same.
// Called by one thread between two CTA barriers; false: gave up.
__device__ __forceinline__ bool grid_arrive_and_wait(unsigned* word, int32_t* err) {
  __threadfence();
  atomicAdd(word, 1u);
  const long long t0 = clock64();
  while (true) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (v >= gridDim.x) return true;
    if (clock64() - t0 > tma::kWaitCycles) {
      flag_error(err, MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// ------------------------------------------------------------ products

__device__ __forceinline__ float activation(float g, float u, float p, float L) {
  const float gc = clamp_max(g, L);
  return gc * sigmoid(gc) * clamp_sym(u, L) * p;
}

// v as the sum of two values of D: v rounded (no further than the largest
// finite value), and what that left, rounded.
template <class D>
__device__ __forceinline__ void split(float v, uint16_t* hi, uint16_t* lo) {
  constexpr float kMax = std::is_same<D, F16>::value ? 65504.0f : 0x1.fep127f;
  const bool inf = fabsf(v) == kInf;
  const float h = round_to<D>(inf ? v : clamp_sym(v, kMax));
  store1<D>(hi, h);
  store1<D>(lo, inf ? 0.0f : v - h);
}

// The coherent load of a value that another CTA wrote before a grid barrier.
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_cg(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}

template <class D>
__device__ __forceinline__ float widen1(uint16_t v);
template <> __device__ __forceinline__ float widen1<BF16>(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}
template <> __device__ __forceinline__ float widen1<F16>(uint16_t v) { return f16_to_f32(v); }

template <class D>
__global__ void __launch_bounds__(kThreads, 1)
layer_experts(Layer a) {
  __shared__ Tables tb;
  __shared__ int gave_up;
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32);
  const int warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const auto* x = static_cast<const uint16_t*>(a.x);
  const auto* w1 = static_cast<const uint16_t*>(a.w1);
  const auto* w2 = static_cast<const uint16_t*>(a.w2);
  if (threadIdx.x == 0) gave_up = 0;
  make_tables(a, tb, kThreads);
  // first product: one warp per (unit, column of the activation)
  const int64_t n1 = (int64_t)tb.units * a.inter;
  for (int64_t i = warp; i < n1; i += warps) {
    const Unit u = tb.unit[i / a.inter];
    const int j = (int)(i % a.inter);
    const uint16_t* wg = w1 + ((int64_t)u.expert * 2 * a.inter + j) * a.hidden;
    const uint16_t* wu = wg + (int64_t)a.inter * a.hidden;
    for (int n = 0; n < u.count; ++n) {
      const int slot = tb.order[u.first + n];
      const uint16_t* xr = x + (slot / a.K) * a.ld_x;
      float g = 0.f, v = 0.f;
      for (int h = lane; h < a.hidden; h += 32) {
        const float xv = load1<D>(xr + h);
        g = fmaf(load1<D>(wg + h), xv, g);
        v = fmaf(load1<D>(wu + h), xv, v);
      }
      g = warp_sum(g);
      v = warp_sum(v);
      if (lane == 0) {
        const float act = activation(g, v, tb.weight[slot], a.limit);
        uint16_t* hr = a.h + (int64_t)(u.first + n) * 2 * a.inter + j;
        split<D>(act, hr, hr + a.inter);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && !grid_arrive_and_wait(&a.barrier[0], a.err)) gave_up = 1;
  __syncthreads();
  if (gave_up) return;
  // second product: one warp per (unit, hidden column)
  const int64_t n2 = (int64_t)tb.units * a.hidden;
  for (int64_t i = warp; i < n2; i += warps) {
    const Unit u = tb.unit[i / a.hidden];
    const int c = (int)(i % a.hidden);
    const uint16_t* w = w2 + ((int64_t)u.expert * a.hidden + c) * a.inter;
    for (int n = 0; n < u.count; ++n) {
      const uint16_t* hr = a.h + (int64_t)(u.first + n) * 2 * a.inter;
      float s = 0.f;
      for (int j = lane; j < a.inter; j += 32)
        s = fmaf(load1<D>(w + j), widen1<D>(ld_cg(hr + j)) + widen1<D>(ld_cg(hr + a.inter + j)), s);
      s = warp_sum(s);
      if (lane == 0) a.y[(int64_t)(u.first + n) * a.hidden + c] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && !grid_arrive_and_wait(&a.barrier[1], a.err)) gave_up = 1;
  __syncthreads();
  if (gave_up) return;
  // combine: the chosen experts of a token in ascending order
  const int64_t total = (int64_t)tb.tokens * a.hidden;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int t = (int)(i / a.hidden), c = (int)(i % a.hidden);
    float s = 0.f;
    for (int k = 0; k < tb.live[t]; ++k) {
      const int slot = t * a.K + tb.rank[t * a.K + k];
      s += ld_cg(a.y + (int64_t)tb.position[slot] * a.hidden + c);
    }
    if (a.shared)
      s += load1<D>(static_cast<const uint16_t*>(a.shared) + t * a.ld_shared + c);
    // (read before written: out may be residual)
    if (a.residual)
      s = load1c<D>(static_cast<const uint16_t*>(a.residual) + t * a.ld_residual + c) + s;
    store1<D>(static_cast<uint16_t*>(a.out) + t * a.ld_out + c, s);
  }
}

// ------------------------------------------------------------ workspace

inline int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Byte offsets of the workspace's parts, and its size.
struct Space { int64_t logits, h, y, bytes; };

Space layer_space(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  Space s;
  s.logits = 256;                                        // the barrier words come first
  s.h = s.logits + up256(tokens * E * 4);
  s.y = s.h + up256(tokens * K * 2 * inter * 2);
  s.bytes = s.y + up256(tokens * K * hidden * 4);
  return s;
}

template <class D>
int launch(Layer& a, cudaStream_t stream) {
  const dim3 grid = a.router_w ? dim3((unsigned)a.E, (unsigned)((a.tokens + kLogitTokens - 1) /
                                                                kLogitTokens))
                               : dim3(1);
  launch_kernel_grid(a.router_f32 ? layer_logits<D, F32> : layer_logits<D, D>, grid, kThreads, 0,
                     stream, a);
  if (int rc = check_launch()) return rc;
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  (void)cudaLaunchKernelEx(&cfg, layer_experts<D>, a);
  return check_launch();
}

}  // namespace

bool moe_layer_shape_ok(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  return tokens >= 0 && tokens <= kMaxTokens && E >= 1 && E <= kMaxLayerExperts && K >= 1 &&
         K <= 32 && K <= E && tokens * K <= kMaxSlots && hidden >= 0 && inter >= 0 &&
         hidden <= (1 << 20) && inter <= (1 << 20);
}

int64_t moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  return layer_space(tokens, hidden, inter, E, K).bytes;
}

int launch_moe_layer(const MoeLayerArgs& m, cudaStream_t stream) {
  Layer a = {};
  a.x = m.x; a.router_w = m.router_w; a.w1 = m.w1; a.w2 = m.w2;
  a.shared = m.shared; a.residual = m.residual; a.out = m.out;
  a.topk_weights = m.topk_weights; a.topk_ids = m.topk_ids; a.valid = m.valid;
  a.tokens = m.tokens; a.hidden = m.hidden; a.inter = m.inter; a.E = m.E; a.K = m.K;
  a.ld_x = m.ld_x; a.ld_shared = m.ld_shared; a.ld_residual = m.ld_residual; a.ld_out = m.ld_out;
  a.router_f32 = m.router_dt == MOE_FP32;
  a.softmax = m.softmax; a.normalise = m.normalise; a.scale = m.scale; a.limit = m.limit;
  a.err = m.err;
  const Space s = layer_space(m.tokens, m.hidden, m.inter, m.E, m.K);
  auto* ws = static_cast<uint8_t*>(m.workspace);
  a.barrier = reinterpret_cast<unsigned*>(ws);
  a.own_logits = reinterpret_cast<float*>(ws + s.logits);
  a.h = reinterpret_cast<uint16_t*>(ws + s.h);
  a.y = reinterpret_cast<float*>(ws + s.y);
  a.logits = m.router_w ? a.own_logits : m.logits;
  a.logits_dt = m.router_w ? MOE_FP32 : m.logits_dt;
  a.ld_logits = m.router_w ? m.E : m.ld_logits;
  return m.dt == MOE_BF16 ? launch<BF16>(a, stream) : launch<F16>(a, stream);
}

}  // namespace moe
