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
//
// The products.  A work item is a tile of weight rows of one unit (an expert and
// up to 32 of its tokens); the weights are the 16-row operand of
// mma.m16n8k16 and the tokens its 8 columns, so one pass over the weights serves
// all of the unit's tokens.  One producer warp brings 32 KB of weights at a time
// into a ring of shared-memory stages by bulk copies, three others the tokens'
// matching columns (cp.async); eight consumer warps multiply.  The weight
// producer waits for nothing but free stages: while the slowest CTA finishes the
// first product, the others' rings fill with the second's weights.
//
// The summation order is the same however a product is tiled: a block of 256
// columns of the axis is cut into eight slices of 32, one to a consumer warp,
// which adds its slices up block after block; the eight sums are added in a fixed
// tree.  No two warps read the same columns of the tokens.
//   kWide   tiles of 64 rows by 256 columns: 3-D tensor copies of 64 columns
//           (128-byte swizzle)
//   kNarrow tiles of 16 rows by 1024 columns, up to 8 tokens a unit: one bulk copy
//           of 2 KB a row
//   kAny    as kNarrow (up to 16 tokens) where rows start off 16-byte boundaries:
//           the copies take the 16-byte words around a weight row, and the
//           consumers shift; the first kernel lays the tokens out anew
// Row copies of 512 bytes instead of kWide's boxes were bound by their number:
// halving their bytes changed nothing.  Four warps to a slice of 128 columns, each
// with a quarter of the rows, were bound by shared memory in the second product.
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "router.cuh"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int kMaxTokens = 128, kMaxSlots = 1024, kMaxLayerExperts = 512;
constexpr int kUnitTokens = 32;                        // tokens of one unit at most,
constexpr int kNarrowTokens = 8;                       // or in tiles of 16 rows (kAny: 16)
constexpr int kMaxUnits = kMaxLayerExperts + kMaxSlots / kNarrowTokens;
constexpr int kBarriers = 3;      // after the choice, between the products, before the combine

// Error bits of waits that gave up in calls without an error word of their own
// (read by moe_device_errors).
__device__ int32_t g_layer_errors;

// One expert and up to kUnitTokens (kNarrowTokens) of its tokens.
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
  uint8_t token[kMaxSlots];      // by position
  uint16_t first[kMaxLayerExperts];
  Unit unit[kMaxUnits];
  int units;
  int most;                      // tokens of the largest unit
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
  bool eights;           // shared, residual and out in 16-byte pieces
  float scale, limit;
  int32_t* err;
  int stall;             // tests of the waits (STALLED kernels): what is withheld, and the limit
  long long wait_cycles;
  // workspace
  unsigned* barrier;     // [kBarriers]
  uint16_t* padded_x;    // kAny: [tokens, hidden up to a multiple of 8], else null
  float* own_logits;     // [tokens, E]
  uint16_t* h;           // [slots, 2, ld_h]: the activation's high and low halves
  int ld_h;              // inter, up to a multiple of 8
  float* y;              // [slots, hidden]
  float* choice_weight;  // [slots], and
  int32_t* choice_id;    // of a choice that the CTAs share
};

// ------------------------------------------------------------ logits

constexpr int kLogitTokens = 4;   // tokens per CTA of the logits kernel

// Sums of N values over the warp with shared butterflies: each step leaves half
// of the values to a lane while there are several.  Value i ends up in every lane
// whose highest bits are i's (from lane 16's bit down), in v[0].
template <int N>
__device__ __forceinline__ void warp_sums(double (&v)[N], int lane) {
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= n) break;
        const double keep = lane & o ? v[i + n] : v[i], give = lane & o ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(kAll, give, o);
      }
    } else {
      v[0] += __shfl_xor_sync(kAll, v[0], o);
    }
  }
}

// EXPERTS experts and kLogitTokens tokens per CTA, VEC elements a thread at a
// time.  The products and their sums are in 64 bits, so that the summation order
// cannot decide between two experts: a choice depends on the inputs alone.  What
// bounds it is the conversion to 64 bits (16 a clock and SM), of which a tile of
// 4 x 4 needs half a conversion a product.
template <class D, class R, int VEC, int EXPERTS>
__global__ void __launch_bounds__(kThreads)
layer_logits(Layer a) {
  pdl_prologue();
  const int cta = blockIdx.y * gridDim.x + blockIdx.x, ctas = gridDim.x * gridDim.y;
  if (cta == 0 && threadIdx.x < kBarriers) a.barrier[threadIdx.x] = 0;
  if (a.padded_x) {      // the tokens in rows of a multiple of 8 columns, the surplus zero
    const int ld = (a.hidden + 7) / 8 * 8;
    for (int i = cta * kThreads + threadIdx.x; i < a.tokens * ld; i += ctas * kThreads) {
      const int t = i / ld, h = i - t * ld;
      a.padded_x[i] = h < a.hidden ? __ldg(static_cast<const uint16_t*>(a.x) + t * a.ld_x + h)
                                   : (uint16_t)0;
    }
  }
  if (!a.router_w) return;
  constexpr int N = EXPERTS * kLogitTokens;
  __shared__ double red[kThreads / 32][N];
  const int e0 = blockIdx.x * EXPERTS, t0 = blockIdx.y * kLogitTokens, lane = threadIdx.x & 31;
  const auto* w = static_cast<const typename R::T*>(a.router_w);
  const auto* x = static_cast<const typename D::T*>(a.x);
  double acc[N] = {};
#pragma unroll 2
  for (int h = threadIdx.x * VEC; h < a.hidden; h += kThreads * VEC) {
    // (past the last expert or token: the last one again, whose sums nothing reads)
    float wv[EXPERTS][VEC], xv[kLogitTokens][VEC];
#pragma unroll
    for (int i = 0; i < EXPERTS; ++i) {
      const auto* p = w + (int64_t)min(e0 + i, a.E - 1) * a.hidden + h;
      if constexpr (VEC == 8) widen8<R>(load8<R>(p), wv[i]);
      else wv[i][0] = load1<R>(p);
    }
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
      const auto* p = x + min(t0 + i, a.tokens - 1) * a.ld_x + h;
      if constexpr (VEC == 8) widen8<D>(load8<D>(p), xv[i]);
      else xv[i][0] = load1<D>(p);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      double wd[EXPERTS];
#pragma unroll
      for (int i = 0; i < EXPERTS; ++i) wd[i] = wv[i][j];
#pragma unroll
      for (int i = 0; i < kLogitTokens; ++i) {
        if (EXPERTS == 1 && t0 + i >= a.tokens) break;
        const double xd = xv[i][j];
#pragma unroll
        for (int k = 0; k < EXPERTS; ++k)
          acc[i * EXPERTS + k] = fma(wd[k], xd, acc[i * EXPERTS + k]);
      }
    }
  }
  warp_sums<N>(acc, lane);
  constexpr int kSpread = 32 / N;
  if (lane % kSpread == 0) red[threadIdx.x >> 5][lane / kSpread] = acc[0];
  __syncthreads();
  const int i = threadIdx.x / EXPERTS, k = threadIdx.x % EXPERTS;
  if (i < kLogitTokens && t0 + i < a.tokens && e0 + k < a.E) {
    double s = 0.0;
#pragma unroll
    for (int r = 0; r < kThreads / 32; ++r) s += red[r][threadIdx.x];
    a.own_logits[(int64_t)(t0 + i) * a.E + e0 + k] = (float)s;
  }
}

template <class D, class R>
void launch_logits(const Layer& a, cudaStream_t stream) {
  const bool vec = a.hidden % kVec == 0 && a.ld_x % kVec == 0 && aligned16(a.x) &&
                   aligned16(a.router_w);
  // four experts a CTA where that leaves a CTA to most of the SMs
  const int64_t tiles = (int64_t)((a.E + 3) / 4) * ((a.tokens + kLogitTokens - 1) / kLogitTokens);
  const int experts = tiles >= 128 ? 4 : 1;
  const dim3 grid = a.router_w ? dim3((unsigned)((a.E + experts - 1) / experts),
                                      (unsigned)((a.tokens + kLogitTokens - 1) / kLogitTokens))
                               : dim3(a.padded_x ? 64 : 1);
  const auto k = vec ? (experts == 4 ? layer_logits<D, R, 8, 4> : layer_logits<D, R, 8, 1>)
                     : (experts == 4 ? layer_logits<D, R, 1, 4> : layer_logits<D, R, 1, 1>);
  launch_kernel_grid(k, grid, kThreads, 0, stream, a);
}

// ------------------------------------------------------------ waits

// Every wait gives up after `limit` cycles (kWaitCycles): the waiter reports it
// and sets the CTA's flag.  From then on nobody in the CTA waits, so that the
// kernel runs to its end (its results are void) with every CTA barrier met; the
// producers end at the next stage that they cannot have (Slot).

struct GiveUp {
  volatile int* flag;   // shared memory
  int32_t* err;
  long long limit;
  __device__ __forceinline__ bool now(long long t0) const {
    if (*flag) return true;
    if (clock64() - t0 <= limit) return false;
    *flag = 1;
    flag_error(err, MOE_DEVERR_TIMEOUT);
    return true;
  }
};

// What a STALLED kernel (tests of the waits) withholds in its first CTA: the third
// fill of a producer, or an arrival at the grid barrier kStallBarrier + i.
enum Stall { kStallWeights1 = 0, kStallWeights2, kStallTokens, kStallBarrier };
constexpr int kStalls = kStallBarrier + kBarriers;

template <bool STALLED>
__device__ __forceinline__ bool withheld(const Layer& a, int what) {
  return STALLED && blockIdx.x == 0 && a.stall == what;
}

// Whether the phase was seen complete.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const GiveUp& g) {
  if (tma::mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!tma::mbar_try(bar, parity))
    if (g.now(t0)) return false;
  return true;
}

// Grid barrier, in two parts.  The launch is cooperative: all CTAs are resident.
__device__ __forceinline__ void grid_arrive(unsigned* word) {
  __threadfence();
  atomicAdd(word, 1u);
}
__device__ __forceinline__ void grid_wait(unsigned* word, const GiveUp& g) {
  const long long t0 = clock64();
  while (true) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (v >= gridDim.x || g.now(t0)) return;
  }
}

// Orders this thread's generic accesses against bulk copies.
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// The load of a value that another CTA wrote before a grid barrier.
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int32_t ld_cg(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// ------------------------------------------------------------ choice

// The logits of token t (as load_logits).
template <int V>
__device__ __forceinline__ void token_logits(const Layer& a, int t, int lane, float (&v)[V]) {
  const int64_t row = (int64_t)t * a.ld_logits;
  if (a.logits_dt == MOE_FP32)
    load_logits<F32, V>(static_cast<const float*>(a.logits) + row, a.E, lane, v);
  else if (a.logits_dt == MOE_BF16)
    load_logits<BF16, V>(static_cast<const uint16_t*>(a.logits) + row, a.E, lane, v);
  else
    load_logits<F16, V>(static_cast<const uint16_t*>(a.logits) + row, a.E, lane, v);
}

// The choices of the tokens t, t + step, ... below `live` by one warp, the next
// one's logits loaded ahead; take(slot, expert, weight) in lane k for the k-th.
// (Several tokens side by side took longer: much of the time here is the first
// fetch of the instructions.)
template <int V, class F>
__device__ __forceinline__ void choose(const Layer& a, int t, int step, int live, F take) {
  const int lane = threadIdx.x & 31;
  float next[V];
  if (t < live) token_logits<V>(a, t, lane, next);
  for (; t < live; t += step) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    if (t + step < live) token_logits<V>(a, t + step, lane, next);
    int id;
    const float w = route_token<V>(v, a.K, lane, a.softmax, a.normalise, a.scale, &id);
    if (lane < a.K) take(t * a.K + lane, id, w);
  }
}

template <class F>
__device__ __forceinline__ void choose(const Layer& a, int t, int step, int live, F take) {
  if (a.E <= 64) choose<2>(a, t, step, live, take);
  else if (a.E <= 256) choose<8>(a, t, step, live, take);
  else choose<16>(a, t, step, live, take);
}

// Fills the tables, units of at most `unit_tokens`; all `threads` threads of the
// CTA take part.  chosen [E][kMaxTokens / 32] (scratch): the tokens of each expert
// as bits, from which counts and places follow without an order of writing.
//   A choice takes a warp about 2 us.  Up to two tokens a warp every CTA makes
// them all; more are shared among the CTAs, at the price of a grid barrier (64
// tokens of 64 experts: 12 us down to 5).
template <bool STALLED>
__device__ void make_tables(const Layer& a, Tables& tb, uint32_t* chosen, int unit_tokens,
                            int threads, const GiveUp& g) {
  constexpr int kWords = kMaxTokens / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = threads / 32;
  const int live = (int)live_tokens(a.valid, a.tokens, a.err);
  for (int i = threadIdx.x; i < a.E * kWords; i += threads) chosen[i] = 0;
  if (threadIdx.x == 0) tb.tokens = live;
  __syncthreads();
  const auto enter = [&](int slot, int id, float w) {
    const int t = slot / a.K;
    tb.expert[slot] = (int16_t)id;
    tb.weight[slot] = w;
    if (id >= 0) atomicOr(&chosen[id * kWords + (t >> 5)], 1u << (t & 31));
  };
  const auto report = [&](int slot, int id, float w) {
    if (a.topk_weights) a.topk_weights[slot] = w;
    if (a.topk_ids) a.topk_ids[slot] = id;
  };
  if (live <= 2 * warps) {
    choose(a, warp, warps, live, [&](int slot, int id, float w) {
      enter(slot, id, w);
      if (blockIdx.x == 0) report(slot, id, w);
    });
  } else {
    if (warp == 0) {
      choose(a, blockIdx.x, gridDim.x, live, [&](int slot, int id, float w) {
        a.choice_weight[slot] = w;
        a.choice_id[slot] = id;
        report(slot, id, w);
      });
      __syncwarp();
      if (lane == 0) {
        if (!withheld<STALLED>(a, kStallBarrier)) grid_arrive(&a.barrier[0]);
        grid_wait(&a.barrier[0], g);
      }
    }
    __syncthreads();
    const bool none = *g.flag;           // after a wait that gave up they may be anything
    for (int s = threadIdx.x; s < live * a.K; s += threads)
      enter(s, none ? -1 : ld_cg(a.choice_id + s), ld_cg(a.choice_weight + s));
  }
  __syncthreads();
  if (warp == 0) {
    // the experts' first positions and units
    int base = 0, units = 0, most = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < a.E) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) n += __popc(chosen[e * kWords + i]);
      }
      const int u = (n + unit_tokens - 1) / unit_tokens;
      most = max(most, min(n, unit_tokens));
      int sum = n | u << 16;                                // inclusive prefix sums
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int before = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += before;
      }
      if (e < a.E) {
        const int first = base + (sum & 0xffff) - n;
        tb.first[e] = (uint16_t)first;
        for (int i = 0; i < u; ++i)
          tb.unit[units + (sum >> 16) - u + i] = {(uint16_t)e, (uint16_t)(first + i * unit_tokens),
                                                  (uint16_t)min(unit_tokens, n - i * unit_tokens)};
      }
      const int total = __shfl_sync(kAll, sum, 31);
      base += total & 0xffff;
      units += total >> 16;
    }
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) {
      tb.units = units;
      tb.most = most;
    }
  }
  __syncthreads();
  for (int t = threadIdx.x; t < live; t += threads) {
    int n = 0;
    for (int k = 0; k < a.K; ++k) n += tb.expert[t * a.K + k] >= 0;
    tb.live[t] = (uint8_t)n;
  }
  for (int s = threadIdx.x; s < live * a.K; s += threads) {
    const int e = tb.expert[s], t = s / a.K;
    if (e < 0) continue;
    int place = 0;             // how many of the token's live experts are lower
    for (int k = 0; k < a.K; ++k) {
      const int other = tb.expert[t * a.K + k];
      place += other >= 0 && other < e;
    }
    tb.rank[t * a.K + place] = (uint8_t)(s - t * a.K);
    int p = tb.first[e] + __popc(chosen[e * kWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
    for (int i = 0; i < t >> 5; ++i) p += __popc(chosen[e * kWords + i]);
    tb.position[s] = (uint16_t)p;
    tb.order[p] = (uint16_t)s;
    tb.token[p] = (uint8_t)t;
  }
  __syncthreads();
}

// ------------------------------------------------------------ products

__device__ __forceinline__ float activation(float g, float u, float p, float L) {
  const float gc = clamp_max(g, L);
  return gc * sigmoid(gc) * clamp_sym(u, L) * p;
}

// v as the sum of two values of D: v rounded (no further than the largest
// finite value), and what that left, rounded.  One rounding alone (2^-9 of
// each term on average) would cost as much accuracy as the output's.
template <class D>
__device__ __forceinline__ void split(float v, uint16_t* hi, uint16_t* lo) {
  constexpr float kMax = std::is_same<D, F16>::value ? 65504.0f : 0x1.fep127f;
  const bool inf = fabsf(v) == kInf;
  const float h = round_to<D>(inf ? v : clamp_sym(v, kMax));
  store1<D>(hi, h);
  store1<D>(lo, inf ? 0.0f : v - h);
}

__device__ __forceinline__ void ld_cg4(const float* p, float* v) {
  asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "l"(p)
               : "memory");
}

constexpr int kConsumers = 8, kTokenWarps = 3;                   // and one weight warp
constexpr int kLayerThreads = (kConsumers + 1 + kTokenWarps) * 32;
constexpr int kSplitCols = 256;                                  // a block of the axis
constexpr int kSlice = kSplitCols / kConsumers;                  // and a warp's part of it
static_assert(kSlice == 32, "two k-steps");
constexpr int kMaxStages = 8;

enum Tiling { kWide, kNarrow, kAny };

template <Tiling T>
struct Tile {
  static constexpr int kRows = T == kWide ? 64 : 16;
  static constexpr int kCols = T == kWide ? kSplitCols : 4 * kSplitCols;
  // Rows of an odd multiple of 16 bytes: ldmatrix without bank conflicts.  A row of kAny
  // fills its pitch; what is read past its end is not used.
  static constexpr int kTokenPitch = kCols * 2 + 16;
  static constexpr int kPitch = kCols * 2 + 16;                    // not of kWide
  static constexpr int kWeightBytes = T == kWide ? kRows * kCols * 2 : kRows * kPitch;
  static constexpr int kTokens = T == kWide ? kUnitTokens : T == kAny ? 2 * kNarrowTokens
                                                                      : kNarrowTokens;
  // one buffer of the warps' sums (of kWide there is one, and a barrier more: its place holds
  // a third stage of units of 25 and more tokens); the ring: stages of weights, then up to
  // 2 * most token rows
  static constexpr int kRed = kConsumers * (kRows / 16) * 32 * 16, kReds = T == kWide ? 1 : 2;
  static constexpr int kRing =
      (232448 - (int)sizeof(Tables) - 512 - kReds * kRed - 1024) / 1024 * 1024;
};

static_assert(Tile<kWide>::kRing >= 2 * (Tile<kWide>::kWeightBytes +
                                         2 * kUnitTokens * Tile<kWide>::kTokenPitch + 1023) &&
                  Tile<kAny>::kRing >= 2 * (Tile<kAny>::kWeightBytes +
                                            4 * kNarrowTokens * Tile<kAny>::kTokenPitch + 1023),
              "two stages at least");
static_assert(Tile<kWide>::kRing >= kMaxLayerExperts * (kMaxTokens / 32) * 4,
              "room for make_tables' scratch");

struct Ring {
  uint8_t* base;         // 1024-byte aligned
  uint64_t *full, *empty;
  volatile int* filled;  // the stages of weights, once their producer has ended; before: -1
  int stage_bytes, stages;
};

__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Whose slots: of the tokens' producers, of the weights' (kWide: the first lane issues all
// copies; else every lane its row's).
enum Producer { kTokens, kBoxes, kRows };

// A place in the ring: the slot and the parity of its current use.
struct Slot {
  int at = 0;
  uint32_t parity = 0;   // bit 1, of a consumer: a wait gave up
  int uses = 0;          // of the ring before this one
  __device__ __forceinline__ void next(const Ring& r) {
    ++uses;
    if (++at == r.stages) { at = 0; parity ^= 1u; }
  }
  // Consumers: waits until the slot has been filled.  One that gave up releases no slot any more.
  __device__ __forceinline__ void wait(const Ring& r, const GiveUp& g) {
    if (!wait_phase(&r.full[at], parity & 1u, g)) parity |= 2u;
  }
  __device__ __forceinline__ bool dead() const { return parity > 1u; }

  // How the producers end, in order or where a wait has given up.  As consumers that gave up
  // release nothing, a slot is only had if the fill before it has landed: the barriers' phases
  // follow the fills, and their counts of bytes stay small.  A producer that does not get its
  // slot ends there (of the tokens', each lane for itself).  The weights' first lane says how
  // many stages have been filled, and waits until they have landed, as a CTA does not end before
  // its copies; a lane of the tokens' that stopped earlier makes up for its arrivals at these.
  __device__ __forceinline__ void end_weights(const Ring& r, const GiveUp& g) const {
    *r.filled = uses;
    for (int i = 0; i < min(uses, r.stages); ++i)
      if (!tma::mbar_wait(&r.full[i], i < at ? parity : parity ^ 1u, g.limit))
        flag_error(g.err, MOE_DEVERR_TIMEOUT);
  }
  __device__ __forceinline__ void end_tokens(const Ring& r) {
    const long long t0 = clock64();
    // (said as soon as the weights' producer meets a slot that it has to wait for)
    while (*r.filled < 0 && clock64() - t0 <= tma::kWaitCycles) {}
    for (; uses < *r.filled; next(r)) tma::mbar_arrive(&r.full[at]);
    cp_async_wait();
  }
  // Producers: waits until the slot may be overwritten.  (One token of 4096 x 2048 experts 75.8
  // us, 128 tokens 712; where it returns that the slot may not be had, and the callers' loops are
  // left by a branch, 77 to 83 and 730 to 767.)
  template <Producer P>
  __device__ __forceinline__ void claim(const Ring& r, const GiveUp& g, int lane) {
    const bool had = uses < r.stages || wait_phase(&r.empty[at], parity ^ 1u, g);
    if (P == kRows ? __all_sync(kAll, had) : had) return;
    if (P == kTokens) end_tokens(r);
    else if (lane == 0) end_weights(r, g);
    asm volatile("exit;");
    __builtin_unreachable();
  }
};

struct Product {
  int axis;      // columns of the weights
  int tiles;     // row tiles of an expert
  int items;     // units x tiles
  int chunks;    // stages per item; an empty axis has one empty stage
};

template <Tiling T, bool SECOND>
__device__ __forceinline__ Product make_product(const Layer& a, const Tables& tb) {
  using S = Tile<T>;
  Product p;
  p.axis = SECOND ? a.inter : a.hidden;
  p.tiles = ((SECOND ? a.hidden : 2 * a.inter) + S::kRows - 1) / S::kRows;
  if (!SECOND) p.tiles = (a.inter + S::kRows / 2 - 1) / (S::kRows / 2);
  p.items = tb.units * p.tiles;
  p.chunks = max(1, (p.axis + S::kCols - 1) / S::kCols);
  return p;
}

// Calls f(unit, tile, first column, columns) for each stage of this CTA's items,
// in order.
template <Tiling T, class F>
__device__ __forceinline__ void for_stages(const Tables& tb, const Product& p, F f) {
  for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
    const Unit u = tb.unit[item / p.tiles];
    const int tile = item % p.tiles;
    for (int c = 0; c < p.chunks; ++c) {
      const int k0 = c * Tile<T>::kCols;
      f(u, tile, k0, min(Tile<T>::kCols, p.axis - k0));
    }
  }
}

// ---- producers

struct WeightMaps {
  CUtensorMap w1, w2;    // kWide
};

// Box of 64 columns of a 3-D tensor into shared memory (128-byte swizzle).
__device__ __forceinline__ void tensor_load(void* dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tma::smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(tma::smem_addr(bar))
      : "memory");
}

// Weight row r of a 16-row tile, or null past the last.  First product: 8 gate
// rows, then the 8 up rows of the same columns of the activation.
template <bool SECOND>
__device__ __forceinline__ const uint16_t* weight_row(const Layer& a, int expert, int tile,
                                                      int r) {
  if (SECOND) {
    const int col = tile * 16 + r;
    if (col >= a.hidden) return nullptr;
    return static_cast<const uint16_t*>(a.w2) + ((int64_t)expert * a.hidden + col) * a.inter;
  }
  const int j = tile * 8 + (r & 7);
  if (j >= a.inter) return nullptr;
  return static_cast<const uint16_t*>(a.w1) +
         (((int64_t)expert * 2 + (r >> 3)) * a.inter + j) * a.hidden;
}

template <Tiling T, bool SECOND, bool STALLED>
__device__ __forceinline__ void produce_weights(const Layer& a, const WeightMaps& maps,
                                                const Tables& tb, const Ring& ring, Slot& slot,
                                                const GiveUp& g, int lane) {
  using S = Tile<T>;
  int fills = 0;
  for_stages<T>(tb, make_product<T, SECOND>(a, tb), [&](Unit u, int tile, int k0, int len) {
    const bool hold = STALLED && fills++ == 2 &&
                      withheld<STALLED>(a, SECOND ? kStallWeights2 : kStallWeights1);
    // (what does not need the slot comes before the wait for it)
    uint8_t* stage = ring.base + (size_t)slot.at * ring.stage_bytes;
    uint64_t* full = &ring.full[slot.at];
    if (T == kWide) {
      // 64-column boxes of 64 rows (first product: 32 gate rows, 32 up rows)
      const int boxes = (len + 63) / 64;
      slot.claim<kBoxes>(ring, g, lane);
      if (lane == 0 && !hold) {
        tma::mbar_arrive_expect_tx(full, boxes * 8192);
        for (int b = 0; b < boxes; ++b) {
          if (SECOND) {
            tensor_load(stage + b * 8192, &maps.w2, k0 + b * 64, tile * 64, u.expert, full);
          } else {
            tensor_load(stage + b * 8192, &maps.w1, k0 + b * 64, tile * 32, u.expert * 2, full);
            tensor_load(stage + b * 8192 + 4096, &maps.w1, k0 + b * 64, tile * 32,
                        u.expert * 2 + 1, full);
          }
        }
      }
    } else {
      const uint16_t* src = lane < 16 ? weight_row<SECOND>(a, u.expert, tile, lane) : nullptr;
      uint8_t* dst = stage + lane * S::kPitch;
      uint32_t bytes = src && !hold ? len * 2 : 0;
      if (src) src += k0;
      slot.claim<kRows>(ring, g, lane);
      if (T == kAny) {
        // the 16-byte words that hold the row, unless they reach past the tensor
        // (its first and its last row): those are put together element by element
        const uintptr_t lo = reinterpret_cast<uintptr_t>(SECOND ? a.w2 : a.w1);
        const uintptr_t hi = lo + (uintptr_t)2 * a.E * (SECOND ? 1 : 2) * a.hidden * a.inter;
        const uintptr_t from = reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15;
        const uintptr_t to = (reinterpret_cast<uintptr_t>(src) + bytes + 15) & ~(uintptr_t)15;
        unsigned edge = __ballot_sync(kAll, bytes > 0 && (from < lo || to > hi));
        const int shift = (int)(reinterpret_cast<uintptr_t>(src) - from);
        for (unsigned rows = edge; rows; rows &= rows - 1) {
          const int r = __ffs(rows) - 1;
          const auto* row = reinterpret_cast<const uint16_t*>(
              __shfl_sync(kAll, reinterpret_cast<uint64_t>(src), r));
          auto* to_row = reinterpret_cast<uint16_t*>(stage + r * S::kPitch +
                                                     __shfl_sync(kAll, shift, r));
          for (int c = lane; c < len; c += 32) to_row[c] = __ldg(row + c);
        }
        if (edge) fence_async_proxy();   // later bulk copies into the stage come after
        __syncwarp();
        if (edge >> lane & 1) bytes = 0;
        if (bytes > 0) {
          src = reinterpret_cast<const uint16_t*>(from);
          bytes = (uint32_t)(to - from);
        }
      }
      uint32_t total = (SECOND ? min(16, a.hidden - tile * 16) : 2 * min(8, a.inter - tile * 8)) *
                       len * 2;
      if (T == kAny) total = __reduce_add_sync(kAll, bytes);
      if (lane == 0 && !hold) tma::mbar_arrive_expect_tx(full, total);
      __syncwarp();
      if (bytes > 0) tma::bulk_load(dst, src, bytes, full);
    }
    slot.next(ring);
  });
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival of this thread once all of its cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tma::smem_addr(bar))
               : "memory");
}

// The stages' columns of the unit's tokens (second product: of both halves of
// their activations).  Both lie in rows that end with zeros up to a multiple of 8.
template <Tiling T, bool SECOND, bool STALLED>
__device__ __forceinline__ void produce_tokens(const Layer& a, const Tables& tb, const Ring& ring,
                                               Slot& slot, const GiveUp& g, int warp, int lane) {
  using S = Tile<T>;
  int fills = 0;
  for_stages<T>(tb, make_product<T, SECOND>(a, tb), [&](Unit u, int, int k0, int len) {
    const uint32_t dst = tma::smem_addr(ring.base + (size_t)slot.at * ring.stage_bytes) +
                         S::kWeightBytes;
    const int rows = SECOND ? 2 * u.count : u.count, pieces = (len + 7) / 8;
    slot.claim<kTokens>(ring, g, lane);
    if (STALLED && fills++ == 2 && warp == 0 && withheld<STALLED>(a, kStallTokens)) {
      slot.next(ring);
      return;
    }
    for (int r = warp; r < rows; r += kTokenWarps) {
      const uint16_t* src;
      if (SECOND) {
        const int n = r < u.count ? r : r - u.count;
        src = a.h + ((int64_t)(u.first + n) * 2 + (r < u.count ? 0 : 1)) * a.ld_h + k0;
      } else {
        src = static_cast<const uint16_t*>(a.x) + tb.token[u.first + r] * a.ld_x + k0;
      }
#pragma unroll 4
      for (int c = lane; c < pieces; c += 32)
        cp_async16(dst + r * S::kTokenPitch + c * 16, src + c * 8);
    }
    cp_async_arrive(&ring.full[slot.at]);
    slot.next(ring);
  });
}

// ---- consumers

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <class D>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<D, BF16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two neighbouring 16-bit elements at any even address of shared memory, the
// second (both) cleared where fewer than two (one) are left.
__device__ __forceinline__ uint32_t lds_pair(uint32_t addr, int left) {
  uint32_t w0, w1;
  const uint32_t at = addr & ~3u;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(at));
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w1) : "r"(at + 4));
  const uint32_t v = __funnelshift_r(w0, w1, (addr & 2u) * 8);
  return left >= 2 ? v : left == 1 ? v & 0xffffu : 0u;
}

// Where 16 rows of weights lie in a stage, for this lane.
template <Tiling T>
struct WeightAddr {
  uint32_t row;           // kWide, kNarrow: this lane's ldmatrix row; kAny: row g
  uint32_t row8;          // kAny: row g + 8
};

// The fragments of 16 rows and the 16 columns from `col` on (of which `left` are
// there) of a stage.
template <Tiling T>
__device__ __forceinline__ void load_weights(uint32_t (&r)[4], const WeightAddr<T>& w, int col,
                                             int lane, int left) {
  if constexpr (T == kWide) {
    const int piece = (col >> 3 & 7) + (lane >> 4);
    ldsm4(r, w.row + (col >> 6) * 8192 + ((piece ^ (lane & 7)) * 16));
  } else if constexpr (T == kNarrow) {
    ldsm4(r, w.row + col * 2);
  } else {
    const int c = (lane & 3) * 2;
    const uint32_t at = (col + c) * 2;
    r[0] = lds_pair(w.row + at, left - c);
    r[1] = lds_pair(w.row8 + at, left - c);
    r[2] = lds_pair(w.row + at + 16, left - c - 8);
    r[3] = lds_pair(w.row8 + at + 16, left - c - 8);
  }
}

// A slice of a stage: the 32 columns from `col` on, of which `left` are there:
// acc[m][j] += weights (16-row group m) x tokens 8 j .. 8 j + 7, for the first CNT
// groups of tokens.  Columns past the unit's last token repeat it; nothing reads
// their sums.
//   FULL: all 32, without branches.  Else: shared memory is filled to a multiple
// of 8 columns; of a last k-step of 16 with 8, the upper half of the fragments is
// cleared, since what lies there may be anything.
template <class D, Tiling T, bool SECOND, bool FULL, int CNT, int M, int NT>
__device__ __forceinline__ void multiply(float (&acc)[M][NT][4], const WeightAddr<T> (&w)[M],
                                         uint32_t tokens, const uint32_t (&boff)[NT],
                                         uint32_t lo_off, int col, int left, int lane) {
  if (!FULL && left <= 0) return;
  const bool both = FULL || left > 16;
  const bool cut0 = !FULL && left <= 8, cut1 = !FULL && left <= 24;
  uint32_t b[CNT][SECOND ? 2 : 1][4];
#pragma unroll
  for (int j = 0; j < CNT; ++j) {
#pragma unroll
    for (int h = 0; h < (SECOND ? 2 : 1); ++h) {
      ldsm4(b[j][h], tokens + boff[j] + h * lo_off + col * 2);
      if (cut0) b[j][h][1] = 0;
      if (cut1) b[j][h][3] = 0;
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    uint32_t a0[4], a1[4];
    load_weights<T>(a0, w[m], col, lane, left);
    if (both) load_weights<T>(a1, w[m], col + 16, lane, left - 16);
    if (cut0) a0[2] = a0[3] = 0;
    if (cut1) a1[2] = a1[3] = 0;
#pragma unroll
    for (int h = 0; h < (SECOND ? 2 : 1); ++h)
#pragma unroll
      for (int j = 0; j < CNT; ++j) mma16816<D>(acc[m][j], a0, b[j][h][0], b[j][h][1]);
    if (both) {
#pragma unroll
      for (int h = 0; h < (SECOND ? 2 : 1); ++h)
#pragma unroll
        for (int j = 0; j < CNT; ++j) mma16816<D>(acc[m][j], a1, b[j][h][2], b[j][h][3]);
    }
  }
}

// This warp's slices of a stage of `len` columns.
template <class D, Tiling T, bool SECOND, int CNT, int M, int NT>
__device__ __forceinline__ void multiply_stage(float (&acc)[M][NT][4], const WeightAddr<T> (&w)[M],
                                               uint32_t tokens, const uint32_t (&boff)[NT],
                                               uint32_t lo_off, int len, int warp, int lane) {
  const int col = warp * kSlice;
  if (len == Tile<T>::kCols) {
#pragma unroll
    for (int c = 0; c < Tile<T>::kCols; c += kSplitCols)
      multiply<D, T, SECOND, true, CNT>(acc, w, tokens, boff, lo_off, c + col, kSlice, lane);
  } else {
    for (int c = 0; c < len; c += kSplitCols)
      multiply<D, T, SECOND, false, CNT>(acc, w, tokens, boff, lo_off, c + col, len - c - col,
                                         lane);
  }
}

// Lane (g, q) of a 16 x 8 block of sums: rows g, g + 8, tokens 2 q, 2 q + 1.
// `row0`: hidden column (second product) or activation column of row 0.
template <class D, bool SECOND>
__device__ __forceinline__ void finish(const Layer& a, const Tables& tb, const Unit& u, int row0,
                                       int tok0, int lane, const float (&c)[4]) {
  const int g = lane >> 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = tok0 + (lane & 3) * 2 + i;
    if (tok >= u.count) continue;
    const int pos = u.first + tok;
    if (SECOND) {
      float* y = a.y + (int64_t)pos * a.hidden;
      if (row0 + g < a.hidden) y[row0 + g] = c[i];
      if (row0 + g + 8 < a.hidden) y[row0 + g + 8] = c[i + 2];
    } else {
      const int j = row0 + g;
      uint16_t* h = a.h + (int64_t)pos * 2 * a.ld_h + j;
      if (j < a.inter)
        split<D>(activation(c[i], c[i + 2], tb.weight[tb.order[pos]], a.limit), h, h + a.ld_h);
      else if (j < a.ld_h)
        h[0] = h[a.ld_h] = 0;
    }
  }
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

template <class D, Tiling T, bool SECOND>
__device__ __forceinline__ void consume(const Layer& a, const Tables& tb, const Ring& ring,
                                        Slot& slot, float4* red, int& buffer, const GiveUp& g) {
  using S = Tile<T>;
  constexpr int M = S::kRows / 16, NT = S::kTokens / 8;      // groups of rows, of tokens
  const Product p = make_product<T, SECOND>(a, tb);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring_base = tma::smem_addr(ring.base);
  for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
    const Unit u = tb.unit[item / p.tiles];
    const int tile = item % p.tiles;
    const int nt = (u.count + 7) / 8;
    uint32_t boff[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) boff[j] = min(j * 8 + (lane & 7), u.count - 1) * S::kTokenPitch;
    const uint32_t lo_off = u.count * S::kTokenPitch;
    WeightAddr<T> rel[M];                                     // within the stage
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (T == kWide) {
        // gate rows 0 .. 31 and up rows 32 .. 63 of the first product's boxes
        rel[m].row = (SECOND ? m * 16 + (lane & 15) : m * 8 + (lane & 7) + (lane & 8) * 4) * 128;
      } else if (T == kNarrow) {
        rel[m].row = (lane & 15) * S::kPitch + (lane >> 4) * 16;
      } else {
        const int r = lane >> 2;
        const auto lo = reinterpret_cast<uintptr_t>(weight_row<SECOND>(a, u.expert, tile, r));
        const auto hi = reinterpret_cast<uintptr_t>(weight_row<SECOND>(a, u.expert, tile, r + 8));
        rel[m].row = r * S::kPitch + (uint32_t)(lo & 15);
        rel[m].row8 = (r + 8) * S::kPitch + (uint32_t)(hi & 15);
      }
    }
    float acc[M][NT][4] = {};
    for (int c = 0; c < p.chunks; ++c) {
      const int len = min(S::kCols, p.axis - c * S::kCols);
      const uint32_t stage = ring_base + slot.at * ring.stage_bytes;
      slot.wait(ring, g);
      __syncwarp();
      WeightAddr<T> w[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        w[m].row = rel[m].row + stage;
        w[m].row8 = rel[m].row8 + stage;
      }
      const uint32_t tokens = stage + S::kWeightBytes + (lane >> 3) * 16;
      if (NT == 1 || nt == 1)
        multiply_stage<D, T, SECOND, 1>(acc, w, tokens, boff, lo_off, len, warp, lane);
      else if (nt == 2)
        multiply_stage<D, T, SECOND, NT < 2 ? 1 : 2>(acc, w, tokens, boff, lo_off, len, warp, lane);
      else if (nt == 3)
        multiply_stage<D, T, SECOND, NT < 3 ? 1 : 3>(acc, w, tokens, boff, lo_off, len, warp, lane);
      else
        multiply_stage<D, T, SECOND, NT>(acc, w, tokens, boff, lo_off, len, warp, lane);
      __syncwarp();
      if (lane == 0 && !slot.dead()) tma::mbar_arrive(&ring.empty[slot.at]);
      slot.next(ring);
    }
    // The warps' sums, in one tree, a group of tokens at a time; half of the warps finish a
    // group, the others the next.
    const int row0 = SECOND ? tile * S::kRows : tile * (S::kRows / 2);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j >= nt) break;
      float4* r = red + (S::kReds == 1 ? 0 : buffer) * (S::kRed / 16);
      if (S::kReds == 1) consumers_sync();             // the last sums have been read
#pragma unroll
      for (int m = 0; m < M; ++m)
        r[(warp * M + m) * 32 + lane] =
            make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
      consumers_sync();
      const int m = M == 1 ? 0 : warp & 3;
      if (M == 1 ? warp == item % kConsumers : warp >> 2 == buffer) {
        float4 v[kConsumers];
#pragma unroll
        for (int i = 0; i < kConsumers; ++i) v[i] = r[(i * M + m) * 32 + lane];
#pragma unroll
        for (int o = 1; o < kConsumers; o *= 2)
#pragma unroll
          for (int i = 0; i < kConsumers; i += 2 * o) {
            v[i].x += v[i + o].x;
            v[i].y += v[i + o].y;
            v[i].z += v[i + o].z;
            v[i].w += v[i + o].w;
          }
        const float c[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        finish<D, SECOND>(a, tb, u, row0 + m * (SECOND ? 16 : 8), j * 8, lane, c);
      }
      buffer ^= 1;      // the next sums must not meet readers of these
    }
  }
}

// out = residual + (the rows of a token's experts, ascending, + shared), VEC
// columns a thread at a time; the loads of four experts' rows are in flight together.
template <class D, int VEC>
__device__ __forceinline__ void combine(const Layer& a, const Tables& tb) {
  const int per_row = a.hidden / VEC, total = tb.tokens * per_row;
  for (int i = blockIdx.x * (kConsumers * 32) + threadIdx.x; i < total;
       i += gridDim.x * (kConsumers * 32)) {
    const int t = i / per_row, c = (i - t * per_row) * VEC;
    const int live = tb.live[t];
    float s[VEC] = {};
    for (int k0 = 0; k0 < live; k0 += 4) {
      float v[4][VEC];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k0 + k >= live) break;
        const int slot = t * a.K + tb.rank[t * a.K + k0 + k];
        const float* y = a.y + (int64_t)tb.position[slot] * a.hidden + c;
        if constexpr (VEC == 8) {
          ld_cg4(y, v[k]);
          ld_cg4(y + 4, v[k] + 4);
        } else {
          v[k][0] = ld_cg(y);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k0 + k >= live) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[j] += v[k][j];
      }
    }
    const auto add = [&](const void* base, int64_t ld) {
      const uint16_t* p = static_cast<const uint16_t*>(base) + t * ld + c;
      if constexpr (VEC == 8) {
        float o[8];
        widen8<D>(load8<D, false>(p), o);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = o[j] + s[j];
      } else {
        s[0] = load1c<D>(p) + s[0];
      }
    };
    if (a.shared) add(a.shared, a.ld_shared);
    if (a.residual) add(a.residual, a.ld_residual);      // (before the store: out may be it)
    uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.ld_out + c;
    if constexpr (VEC == 8) store8<D>(out, s);
    else store1<D>(out, s[0]);
  }
}

template <class D, Tiling T, bool STALLED>
__global__ void __launch_bounds__(kLayerThreads, 1)
layer_experts(const __grid_constant__ Layer a, const __grid_constant__ WeightMaps maps) {
  using S = Tile<T>;
  __shared__ Tables tb;
  __shared__ uint64_t bars[2 * kMaxStages];
  __shared__ int gave_up, filled;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    gave_up = 0;
    filled = -1;
    for (int i = 0; i < kMaxStages; ++i) {
      tma::mbar_init(&bars[i], 1 + kTokenWarps * 32);
      tma::mbar_init(&bars[kMaxStages + i], kConsumers);
    }
    tma::mbar_init_fence();
  }
  pdl_prologue();
  // (the ring serves as scratch before its first copies)
  const GiveUp g{&gave_up, a.err ? a.err : &g_layer_errors,
                 STALLED ? a.wait_cycles : tma::kWaitCycles};
  make_tables<STALLED>(a, tb, reinterpret_cast<uint32_t*>(ring_mem), S::kTokens, kLayerThreads, g);
  fence_async_proxy();                   // ... by bulk copies
  __syncthreads();
  Ring ring;
  ring.base = ring_mem + ((1024u - (tma::smem_addr(ring_mem) & 1023u)) & 1023u);
  ring.full = bars;
  ring.empty = bars + kMaxStages;
  ring.filled = &filled;
  ring.stage_bytes = (S::kWeightBytes + 2 * tb.most * S::kTokenPitch + 1023) / 1024 * 1024;
  ring.stages = min(kMaxStages, S::kRing / ring.stage_bytes);
  float4* red = reinterpret_cast<float4*>(ring.base + S::kRing);
  Slot slot;
  if (warp == kConsumers) {
    produce_weights<T, false, STALLED>(a, maps, tb, ring, slot, g, lane);
    produce_weights<T, true, STALLED>(a, maps, tb, ring, slot, g, lane);
    if (lane == 0) slot.end_weights(ring, g);
    return;
  }
  if (warp > kConsumers) {
    const int w = warp - kConsumers - 1;
    produce_tokens<T, false, STALLED>(a, tb, ring, slot, g, w, lane);
    if (lane == 0) grid_wait(&a.barrier[1], g);
    __syncwarp();
    produce_tokens<T, true, STALLED>(a, tb, ring, slot, g, w, lane);
    cp_async_wait();
    return;
  }
  int buffer = 0;
  consume<D, T, false>(a, tb, ring, slot, red, buffer, g);
  consumers_sync();
  if (threadIdx.x == 0 && !withheld<STALLED>(a, kStallBarrier + 1)) grid_arrive(&a.barrier[1]);
  consume<D, T, true>(a, tb, ring, slot, red, buffer, g);
  consumers_sync();
  if (threadIdx.x == 0) {
    if (!withheld<STALLED>(a, kStallBarrier + 2)) grid_arrive(&a.barrier[2]);
    grid_wait(&a.barrier[2], g);
  }
  consumers_sync();
  if (a.eights) combine<D, 8>(a, tb);
  else combine<D, 1>(a, tb);
}

// ------------------------------------------------------------ workspace

inline int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Byte offsets of the workspace's parts, and its size.
struct Space { int64_t logits, weight, id, x, h, y, bytes; };

Space layer_space(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  Space s;
  s.logits = 256;                                        // the barrier words come first
  s.weight = s.logits + up256(tokens * E * 4);
  s.id = s.weight + up256(tokens * K * 4);
  s.x = s.id + up256(tokens * K * 4);
  s.h = s.x + up256(tokens * ((hidden + 7) / 8 * 8) * 2);
  s.y = s.h + up256(tokens * K * 2 * ((inter + 7) / 8 * 8) * 2);
  s.bytes = s.y + up256(tokens * K * hidden * 4);
  return s;
}

// The driver's tensor-map encoder, looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                           cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiled>(p) : nullptr;
  }();
  return fn;
}

// Boxes of 64 columns and `box` rows of a [depth, rows, cols] tensor of 16-bit
// elements (only their bits are moved); outside of it they read zeros.
int weight_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t depth,
               int box) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return cuda_fail(cudaErrorNotSupported);
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1}, steps[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims,
                            strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : cuda_fail(cudaErrorInvalidValue);
}

template <class D, Tiling T, bool STALLED>
int launch_experts(const Layer& a, const WeightMaps& maps, int sms, cudaStream_t stream) {
  constexpr size_t smem = Tile<T>::kRing + Tile<T>::kReds * Tile<T>::kRed + 1024;
  if (int rc = ensure_smem_limit((const void*)layer_experts<D, T, STALLED>, smem)) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kLayerThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = MOE_PDL;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  (void)cudaLaunchKernelEx(&cfg, layer_experts<D, T, STALLED>, a, maps);
  return check_launch();
}

// Time (us) of both products in tiles of `rows` rows: the rounds of items over the
// SMs, an item by the bytes that an SM's share of HBM brings (44 KB a us), but at
// least the 0.75 us that a CTA needs from one item to the next.
double tiles_time(const Layer& a, int rows, int sms) {
  const int64_t experts = a.E < (int64_t)a.tokens * a.K ? a.E : a.tokens * a.K;
  const auto product = [&](int64_t row_count, int64_t axis) {
    const int64_t items = experts * ((row_count + rows - 1) / rows);
    const double one = (double)rows * axis * 2 / 44e3;
    return (double)((items + sms - 1) / sms) * (one > 0.75 ? one : 0.75);
  };
  return product(2 * (int64_t)a.inter, a.hidden) + product(a.hidden, a.inter);
}

template <class D, bool STALLED>
int launch(const Layer& given, cudaStream_t stream) {
  if (given.router_f32) launch_logits<D, F32>(given, stream);
  else launch_logits<D, D>(given, stream);
  if (int rc = check_launch()) return rc;
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  WeightMaps maps = {};
  Layer a = given;
  if (a.padded_x) {
    a.x = a.padded_x;
    a.ld_x = (a.hidden + 7) / 8 * 8;
    return launch_experts<D, kAny, STALLED>(a, maps, sms, stream);
  }
  // The narrow tiles' units hold 8 tokens: more tokens may need the weights again.  One token
  // of eight 4096 x 2048 experts: 75 us in narrow tiles, 78 in wide ones; eight tokens of 64
  // experts of 2048 x 512: 78 and 60.
  if ((a.tokens <= kNarrowTokens && tiles_time(a, 16, sms) <= tiles_time(a, 64, sms)) ||
      a.inter == 0)
    return launch_experts<D, kNarrow, STALLED>(a, maps, sms, stream);
  if (int rc = weight_map(&maps.w1, a.w1, a.hidden, a.inter, 2 * (int64_t)a.E, 32)) return rc;
  if (int rc = weight_map(&maps.w2, a.w2, a.inter, a.hidden, a.E, 64)) return rc;
  return launch_experts<D, kWide, STALLED>(a, maps, sms, stream);
}

}  // namespace

bool moe_layer_shape_ok(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  return tokens >= 0 && tokens <= kMaxTokens && E >= 1 && E <= kMaxLayerExperts && K >= 1 &&
         K <= 32 && K <= E && tokens * K <= kMaxSlots && hidden >= 0 && inter >= 0 &&
         hidden <= (1 << 20) && inter <= (1 << 20);
}

bool moe_layer_stall_ok(int stall) { return stall >= 0 && stall < kStalls; }

int moe_layer_device_errors(int32_t* bits, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_layer_errors, sizeof(int32_t));
  if (e != cudaSuccess) return cuda_fail(e);
  if (clear) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_layer_errors, &zero, sizeof(int32_t));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MOE_OK;
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
  a.choice_weight = reinterpret_cast<float*>(ws + s.weight);
  a.choice_id = reinterpret_cast<int32_t*>(ws + s.id);
  a.ld_h = (m.inter + 7) / 8 * 8;
  if (m.hidden % 8 != 0 || m.ld_x % 8 != 0 || m.inter % 8 != 0 || !aligned16(m.x) ||
      !aligned16(m.w1) || !aligned16(m.w2))
    a.padded_x = reinterpret_cast<uint16_t*>(ws + s.x);
  a.eights = m.hidden % kVec == 0 && m.ld_out % kVec == 0 && aligned16(m.out) &&
             (!m.shared || (m.ld_shared % kVec == 0 && aligned16(m.shared))) &&
             (!m.residual || (m.ld_residual % kVec == 0 && aligned16(m.residual)));
  a.logits = m.router_w ? a.own_logits : m.logits;
  a.logits_dt = m.router_w ? MOE_FP32 : m.logits_dt;
  a.ld_logits = m.router_w ? m.E : m.ld_logits;
  if (m.wait_cycles > 0) {
    a.stall = m.stall;
    a.wait_cycles = m.wait_cycles;
    return launch<BF16, true>(a, stream);
  }
  return m.dt == MOE_BF16 ? launch<BF16, false>(a, stream) : launch<F16, false>(a, stream);
}

}  // namespace moe
