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
// The summation order is the same however a product is tiled: the axis is cut
// into blocks of 256, block c's halves of 128 are accumulated in order into the
// partial sums (c mod 4, half), and these eight are added in a fixed tree.
//   kWide   tiles of 64 rows by 256 columns: 2-D tensor copies of 64 columns
//           (128-byte swizzle); four warps share a block half, each keeping the
//           four block classes of its 16 rows in registers
//   kNarrow tiles of 16 rows by 1024 columns, up to 8 tokens a unit: one bulk copy
//           of 2 KB a row; each warp has one of the eight partial sums
//   kAny    as kNarrow where rows start off 16-byte boundaries: the copies take
//           the 16-byte words around a row, and the consumers shift
// Row copies of 512 bytes instead of kWide's boxes were bound by their number:
// halving their bytes changed nothing.
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
constexpr int kNarrowTokens = 8;                       // or in tiles of 16 rows
constexpr int kMaxUnits = kMaxLayerExperts + kMaxSlots / kNarrowTokens;
constexpr int kBarriers = 2;

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
  // workspace
  unsigned* barrier;     // [kBarriers]
  float* own_logits;     // [tokens, E]
  uint16_t* h;           // [slots, 2, ld_h]: the activation's high and low halves
  int ld_h;              // inter, up to a multiple of 8
  float* y;              // [slots, hidden]
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
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kBarriers) a.barrier[threadIdx.x] = 0;
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
                               : dim3(1);
  const auto k = vec ? (experts == 4 ? layer_logits<D, R, 8, 4> : layer_logits<D, R, 8, 1>)
                     : (experts == 4 ? layer_logits<D, R, 1, 4> : layer_logits<D, R, 1, 1>);
  launch_kernel_grid(k, grid, kThreads, 0, stream, a);
}

// ------------------------------------------------------------ choice

// The logits of token t, experts [lane * V, lane * V + V).
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

// The choices of all live tokens, a warp per token, the next one's logits loaded
// ahead.  (Several tokens side by side took longer: most of a call's time here is
// the first fetch of the instructions.)
template <int V>
__device__ __forceinline__ void choose(const Layer& a, Tables& tb, uint32_t* chosen, int live,
                                       int threads) {
  const int warps = threads / 32, lane = threadIdx.x & 31;
  int t = threadIdx.x >> 5;
  float next[V];
  if (t < live) token_logits<V>(a, t, lane, next);
  for (; t < live; t += warps) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    if (t + warps < live) token_logits<V>(a, t + warps, lane, next);
    int id;
    const float w = route_token<V>(v, a.K, lane, a.softmax, a.normalise, a.scale, &id);
    int place = 0;             // how many of the token's live experts are lower
    for (int k = 0; k < a.K; ++k) {
      const int other = __shfl_sync(kAll, id, k);
      place += other >= 0 && other < id;
    }
    const unsigned alive = __ballot_sync(kAll, id >= 0);
    if (lane < a.K) {
      const int slot = t * a.K + lane;
      tb.expert[slot] = (int16_t)id;
      tb.weight[slot] = w;
      if (id >= 0) {
        tb.rank[t * a.K + place] = (uint8_t)lane;
        atomicOr(&chosen[id * (kMaxTokens / 32) + (t >> 5)], 1u << (t & 31));
      }
      if (blockIdx.x == 0) {
        if (a.topk_weights) a.topk_weights[slot] = w;
        if (a.topk_ids) a.topk_ids[slot] = id;
      }
    }
    if (lane == 0) tb.live[t] = (uint8_t)__popc(alive);
  }
}

// Fills the tables, units of at most `unit_tokens`; all `threads` threads of the
// CTA take part.  chosen [E][kMaxTokens / 32] (scratch): the tokens of each expert
// as bits, from which counts and places follow without an order of writing.
__device__ void make_tables(const Layer& a, Tables& tb, uint32_t* chosen, int unit_tokens,
                            int threads) {
  constexpr int kWords = kMaxTokens / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int live = (int)live_tokens(a.valid, a.tokens, a.err);
  for (int i = threadIdx.x; i < a.E * kWords; i += threads) chosen[i] = 0;
  if (threadIdx.x == 0) tb.tokens = live;
  __syncthreads();
  if (a.E <= 64) choose<2>(a, tb, chosen, live, threads);
  else if (a.E <= 256) choose<8>(a, tb, chosen, live, threads);
  else choose<16>(a, tb, chosen, live, threads);
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
  for (int s = threadIdx.x; s < live * a.K; s += threads) {
    const int e = tb.expert[s], t = s / a.K;
    if (e < 0) continue;
    int p = tb.first[e] + __popc(chosen[e * kWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
    for (int i = 0; i < t >> 5; ++i) p += __popc(chosen[e * kWords + i]);
    tb.position[s] = (uint16_t)p;
    tb.order[p] = (uint16_t)s;
    tb.token[p] = (uint8_t)t;
  }
  __syncthreads();
}

// ------------------------------------------------------------ waits

// Every wait gives up after kWaitCycles: the waiter reports it and sets the
// CTA's flag, and from then on nobody in the CTA waits, so that the kernel runs
// to its end (its results are void) with every CTA barrier met.

struct GiveUp {
  volatile int* flag;   // shared memory
  int32_t* err;
  __device__ __forceinline__ bool now(long long t0) const {
    if (*flag) return true;
    if (clock64() - t0 <= tma::kWaitCycles) return false;
    *flag = 1;
    flag_error(err, MOE_DEVERR_TIMEOUT);
    return true;
  }
};

__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, const GiveUp& g) {
  if (tma::mbar_try(bar, parity)) return;
  const long long t0 = clock64();
  while (!tma::mbar_try(bar, parity) && !g.now(t0)) {}
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

// The load of a value that another CTA wrote before a grid barrier.
__device__ __forceinline__ float ld_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
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
constexpr int kMaxStages = 8;
constexpr int kRedBytes = 4 * 4 * 32 * 16;                       // one buffer of partial sums

enum Tiling { kWide, kNarrow, kAny };

template <Tiling T>
struct Tile {
  static constexpr int kRows = T == kWide ? 64 : 16;
  static constexpr int kCols = T == kWide ? kSplitCols : 4 * kSplitCols;
  // rows of an odd multiple of 16 bytes: ldmatrix without bank conflicts
  static constexpr int kTokenPitch = kCols * 2 + 16;
  static constexpr int kPitch = T == kAny ? kCols * 2 + 32 : kCols * 2 + 16;   // not of kWide
  static constexpr int kWeightBytes = T == kWide ? kRows * kCols * 2 : kRows * kPitch;
  static constexpr int kTokens = T == kWide ? kUnitTokens : kNarrowTokens;
};

// The ring: stages of weights, then up to 2 * most token rows.
constexpr int kRingBytes = (232448 - (int)sizeof(Tables) - 2 * kRedBytes - 256) / 1024 * 1024 - 1024;
static_assert(kRingBytes / 1024 >= 2 * (32 + 2 * kUnitTokens * (kSplitCols * 2 + 16) / 1024 + 1),
              "two stages at least");
static_assert(kRingBytes >= kMaxLayerExperts * (kMaxTokens / 32) * 4, "room for make_tables");

struct Ring {
  uint8_t* base;         // 1024-byte aligned
  uint64_t *full, *empty;
  int stage_bytes, stages;
};

// A place in the ring: the slot and the parity of its current use.
struct Slot {
  int at = 0;
  uint32_t parity = 0;
  int fresh;             // slots not used yet
  __device__ explicit Slot(const Ring& r) : fresh(r.stages) {}
  __device__ __forceinline__ void next(const Ring& r) {
    if (++at == r.stages) { at = 0; parity ^= 1u; }
  }
  // Waits until the slot may be overwritten.
  __device__ __forceinline__ void claim(const Ring& r, const GiveUp& g) {
    if (fresh > 0) --fresh;
    else wait_phase(&r.empty[at], parity ^ 1u, g);
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

template <Tiling T, bool SECOND>
__device__ __forceinline__ void produce_weights(const Layer& a, const WeightMaps& maps,
                                                const Tables& tb, const Ring& ring, Slot& slot,
                                                const GiveUp& g, int lane) {
  using S = Tile<T>;
  for_stages<T>(tb, make_product<T, SECOND>(a, tb), [&](Unit u, int tile, int k0, int len) {
    slot.claim(ring, g);
    uint8_t* stage = ring.base + (size_t)slot.at * ring.stage_bytes;
    uint64_t* full = &ring.full[slot.at];
    if (T == kWide) {
      // 64-column boxes of 64 rows (first product: 32 gate rows, 32 up rows)
      const int boxes = (len + 63) / 64;
      if (lane == 0) {
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
      uint32_t bytes = src ? len * 2 : 0;
      if (src) src += k0;
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
      const uint32_t total = __reduce_add_sync(kAll, bytes);
      if (lane == 0) tma::mbar_arrive_expect_tx(full, total);
      __syncwarp();
      if (bytes > 0) tma::bulk_load(dst, src, bytes, full);
    }
    slot.next(ring);
  });
}

// Waits until every stage filled has landed: a CTA does not end before its copies.
__device__ __forceinline__ void drain(const Ring& ring, const Slot& slot, const GiveUp& g) {
  for (int i = 0; i < ring.stages - slot.fresh; ++i) {
    const uint32_t parity = i < slot.at ? slot.parity : slot.parity ^ 1u;
    if (!tma::mbar_wait(&ring.full[i], parity)) flag_error(g.err, MOE_DEVERR_TIMEOUT);
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival of this thread once all of its cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tma::smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Columns [col, col + 8) of a row of `len` columns into shared memory, zeros
// past the end, element by element.
__device__ __forceinline__ void copy8(uint32_t dst, const uint16_t* row, int col, int len) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = col + 2 * i;
    const uint32_t lo = c < len ? __ldg(row + c) : 0u;
    const uint32_t hi = c + 1 < len ? __ldg(row + c + 1) : 0u;
    w[i] = lo | hi << 16;
  }
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3])
               : "memory");
}

// The stages' columns of the unit's tokens (second product: of both halves of
// their activations), zeros up to a multiple of 8.
template <Tiling T, bool SECOND>
__device__ __forceinline__ void produce_tokens(const Layer& a, const Tables& tb, const Ring& ring,
                                               Slot& slot, const GiveUp& g, int warp, int lane) {
  using S = Tile<T>;
  for_stages<T>(tb, make_product<T, SECOND>(a, tb), [&](Unit u, int, int k0, int len) {
    slot.claim(ring, g);
    const uint32_t dst = tma::smem_addr(ring.base + (size_t)slot.at * ring.stage_bytes) +
                         S::kWeightBytes;
    const int rows = SECOND ? 2 * u.count : u.count, pieces = (len + 7) / 8;
    for (int r = warp; r < rows; r += kTokenWarps) {
      const uint16_t* src;
      if (SECOND) {
        const int n = r < u.count ? r : r - u.count;
        src = a.h + ((int64_t)(u.first + n) * 2 + (r < u.count ? 0 : 1)) * a.ld_h + k0;
      } else {
        src = static_cast<const uint16_t*>(a.x) + tb.token[u.first + r] * a.ld_x + k0;
      }
#pragma unroll 4
      for (int c = lane; c < pieces; c += 32) {
        // (the activation's rows end with zeros up to a multiple of 8)
        if (SECOND || T != kAny) cp_async16(dst + r * S::kTokenPitch + c * 16, src + c * 8);
        else copy8(dst + r * S::kTokenPitch + c * 16, src, c * 8, len);
      }
    }
    if (SECOND || T != kAny) cp_async_arrive(&ring.full[slot.at]);
    else tma::mbar_arrive(&ring.full[slot.at]);
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

// Where a warp's 16 rows of weights lie in a stage.
template <Tiling T>
struct WeightAddr {
  uint32_t row;           // kWide, kNarrow: this lane's ldmatrix row; kAny: row g
  uint32_t row8;          // kAny: row g + 8
};

// The fragment of k-step ks (16 columns) of this warp's 128.
template <Tiling T>
__device__ __forceinline__ void load_weights(uint32_t (&r)[4], const WeightAddr<T>& w, int half,
                                             int ks, int lane, int len) {
  if constexpr (T == kWide) {
    const int piece = (ks & 3) * 2 + (lane >> 4);
    ldsm4(r, w.row + (half * 2 + (ks >> 2)) * 8192 + ((piece ^ (lane & 7)) * 16));
  } else if constexpr (T == kNarrow) {
    ldsm4(r, w.row + ks * 32);
  } else {
    const int c = ks * 16 + (lane & 3) * 2;
    r[0] = lds_pair(w.row + c * 2, len - c);
    r[1] = lds_pair(w.row8 + c * 2, len - c);
    r[2] = lds_pair(w.row + c * 2 + 16, len - c - 8);
    r[3] = lds_pair(w.row8 + c * 2 + 16, len - c - 8);
  }
}

// This warp's `len` (up to 128) columns of one stage: acc[j] += weights (16
// rows) x tokens 8 j .. 8 j + 7, for the first CNT of the NT groups of tokens.
// Columns past the unit's last token repeat it; nothing reads their sums.  The
// second product's low halves have sums of their own for the stage, so that half
// as many products wait for one another.
//   FULL: all 128 columns, without branches.  Else: shared memory is filled to a
// multiple of 8 columns; of a last k-step of 16 with 8, the upper half of the
// fragments is cleared, since what lies there may be anything.
template <class D, Tiling T, bool SECOND, bool FULL, int CNT, int NT>
__device__ __forceinline__ void multiply(float (&acc)[NT][4], const WeightAddr<T>& w,
                                         uint32_t tokens, const uint32_t (&boff)[NT],
                                         uint32_t lo_off, int len, int half, int lane) {
  float low[SECOND ? CNT : 1][4] = {};
#pragma unroll
  for (int kp = 0; kp < 4; ++kp) {
    if (!FULL && kp * 32 >= len) break;
    uint32_t a0[4], a1[4];
    const bool both = FULL || kp * 32 + 16 < len;
    const bool cut0 = !FULL && kp * 32 + 8 >= len, cut1 = !FULL && kp * 32 + 24 >= len;
    load_weights<T>(a0, w, half, 2 * kp, lane, len);
    if (both) load_weights<T>(a1, w, half, 2 * kp + 1, lane, len);
    if (cut0) a0[2] = a0[3] = 0;
    if (cut1) a1[2] = a1[3] = 0;
#pragma unroll
    for (int j = 0; j < CNT; ++j) {
      uint32_t b[4];
      ldsm4(b, tokens + boff[j] + kp * 64);
      if (cut0) b[1] = 0;
      if (cut1) b[3] = 0;
      mma16816<D>(acc[j], a0, b[0], b[1]);
      if (both) mma16816<D>(acc[j], a1, b[2], b[3]);
      if constexpr (SECOND) {
        ldsm4(b, tokens + boff[j] + lo_off + kp * 64);
        if (cut0) b[1] = 0;
        if (cut1) b[3] = 0;
        mma16816<D>(low[j], a0, b[0], b[1]);
        if (both) mma16816<D>(low[j], a1, b[2], b[3]);
      }
    }
  }
  if constexpr (SECOND) {
#pragma unroll
    for (int j = 0; j < CNT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] += low[j][i];
  }
}

// The same for nt groups of tokens.
template <class D, Tiling T, bool SECOND, int NT, class... Args>
__device__ __forceinline__ void multiply_groups(int nt, int len, float (&acc)[NT][4],
                                                const Args&... args) {
  if constexpr (NT == 1) {
    if (len == kSplitCols / 2) multiply<D, T, SECOND, true, 1, NT>(acc, args...);
    else multiply<D, T, SECOND, false, 1, NT>(acc, args...);
  } else {
    const bool full = len == kSplitCols / 2;
    if (nt == 1) {
      if (full) multiply<D, T, SECOND, true, 1, NT>(acc, args...);
      else multiply<D, T, SECOND, false, 1, NT>(acc, args...);
    } else if (nt == 2) {
      if (full) multiply<D, T, SECOND, true, 2, NT>(acc, args...);
      else multiply<D, T, SECOND, false, 2, NT>(acc, args...);
    } else {
      // (a fourth group that the unit does not have repeats its last token)
      if (full) multiply<D, T, SECOND, true, 4, NT>(acc, args...);
      else multiply<D, T, SECOND, false, 4, NT>(acc, args...);
    }
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
  constexpr bool WIDE = T == kWide;
  constexpr int NS = WIDE ? 4 : 1, NT = WIDE ? 4 : 1;
  const Product p = make_product<T, SECOND>(a, tb);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = warp >> 2, quarter = warp & 3;
  const int group = WIDE ? quarter : 0;                       // 16-row group of the tile
  const int off = (WIDE ? 0 : quarter * kSplitCols) + half * (kSplitCols / 2);
  const uint32_t ring_base = tma::smem_addr(ring.base);
  for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
    const Unit u = tb.unit[item / p.tiles];
    const int tile = item % p.tiles;
    const int nt = (u.count + 7) / 8;
    uint32_t boff[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) boff[j] = min(j * 8 + (lane & 7), u.count - 1) * S::kTokenPitch;
    const uint32_t lo_off = u.count * S::kTokenPitch;
    WeightAddr<T> rel;                                        // within the stage
    if (T == kWide) {
      // gate rows 0 .. 31 and up rows 32 .. 63 of the first product's boxes
      rel.row = (SECOND ? group * 16 + (lane & 15)
                        : group * 8 + (lane & 7) + (lane & 8) * 4) * 128;
    } else if (T == kNarrow) {
      rel.row = (lane & 15) * S::kPitch + (off + (lane >> 4) * 8) * 2;
    } else {
      const int r = lane >> 2;
      const auto lo = reinterpret_cast<uintptr_t>(weight_row<SECOND>(a, u.expert, tile, r));
      const auto hi = reinterpret_cast<uintptr_t>(weight_row<SECOND>(a, u.expert, tile, r + 8));
      rel.row = r * S::kPitch + off * 2 + (uint32_t)(lo & 15);
      rel.row8 = (r + 8) * S::kPitch + off * 2 + (uint32_t)(hi & 15);
    }
    float acc[NS][NT][4] = {};
    for (int c0 = 0; c0 < p.chunks; c0 += NS) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (c0 + s >= p.chunks) break;
        const int len = min(S::kCols, p.axis - (c0 + s) * S::kCols) - off;
        const uint32_t stage = ring_base + slot.at * ring.stage_bytes;
        wait_phase(&ring.full[slot.at], slot.parity, g);
        __syncwarp();
        WeightAddr<T> w = rel;
        w.row += stage;
        w.row8 += stage;
        const int cols = min(kSplitCols / 2, len);
        multiply_groups<D, T, SECOND, NT>(nt, cols, acc[s], w,
                                          stage + S::kWeightBytes + (off + (lane >> 3) * 8) * 2,
                                          boff, lo_off, cols, half, lane);
        __syncwarp();
        if (lane == 0) tma::mbar_arrive(&ring.empty[slot.at]);
        slot.next(ring);
      }
    }
    // the eight partial sums, in one order: ((0 + 1) + (2 + 3)) of each half, then the halves
    float4* r = red + buffer * (kRedBytes / 16);
    if constexpr (WIDE) {
      float sum[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum[j][i] = (acc[0][j][i] + acc[1][j][i]) + (acc[2][j][i] + acc[3][j][i]);
        if (half == 1 && j < nt)
          r[(group * 4 + j) * 32 + lane] = make_float4(sum[j][0], sum[j][1], sum[j][2], sum[j][3]);
      }
      consumers_sync();
      if (half == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= nt) break;
          const float4 o = r[(group * 4 + j) * 32 + lane];
          const float c[4] = {sum[j][0] + o.x, sum[j][1] + o.y, sum[j][2] + o.z, sum[j][3] + o.w};
          finish<D, SECOND>(a, tb, u, SECOND ? tile * 64 + group * 16 : tile * 32 + group * 8,
                            j * 8, lane, c);
        }
      }
    } else {
      r[warp * 32 + lane] = make_float4(acc[0][0][0], acc[0][0][1], acc[0][0][2], acc[0][0][3]);
      consumers_sync();
      // one warp finishes an item, another the next
      if (warp == (item / (int)gridDim.x) % kConsumers) {
        float c[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v0 = r[(h * 4 + 0) * 32 + lane], v1 = r[(h * 4 + 1) * 32 + lane];
          const float4 v2 = r[(h * 4 + 2) * 32 + lane], v3 = r[(h * 4 + 3) * 32 + lane];
          c[h][0] = (v0.x + v1.x) + (v2.x + v3.x);
          c[h][1] = (v0.y + v1.y) + (v2.y + v3.y);
          c[h][2] = (v0.z + v1.z) + (v2.z + v3.z);
          c[h][3] = (v0.w + v1.w) + (v2.w + v3.w);
        }
        const float s[4] = {c[0][0] + c[1][0], c[0][1] + c[1][1], c[0][2] + c[1][2],
                            c[0][3] + c[1][3]};
        finish<D, SECOND>(a, tb, u, SECOND ? tile * 16 : tile * 8, 0, lane, s);
      }
    }
    buffer ^= 1;      // the next item's sums must not meet readers of these
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

template <class D, Tiling T>
__global__ void __launch_bounds__(kLayerThreads, 1)
layer_experts(const __grid_constant__ Layer a, const __grid_constant__ WeightMaps maps) {
  using S = Tile<T>;
  __shared__ Tables tb;
  __shared__ float4 red[2 * kRedBytes / 16];
  __shared__ uint64_t bars[2 * kMaxStages];
  __shared__ int gave_up;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      tma::mbar_init(&bars[i], 1 + kTokenWarps * 32);
      tma::mbar_init(&bars[kMaxStages + i], kConsumers);
    }
    tma::mbar_init_fence();
  }
  pdl_prologue();
  // (the ring serves as scratch before its first copies)
  make_tables(a, tb, reinterpret_cast<uint32_t*>(ring_mem), S::kTokens, kLayerThreads);
  fence_async_proxy();                   // ... by bulk copies
  __syncthreads();
  const GiveUp g{&gave_up, a.err};
  Ring ring;
  ring.base = ring_mem + ((1024u - (tma::smem_addr(ring_mem) & 1023u)) & 1023u);
  ring.full = bars;
  ring.empty = bars + kMaxStages;
  ring.stage_bytes = (S::kWeightBytes + 2 * tb.most * S::kTokenPitch + 1023) / 1024 * 1024;
  ring.stages = min(kMaxStages, kRingBytes / ring.stage_bytes);
  Slot slot(ring);
  if (warp == kConsumers) {
    produce_weights<T, false>(a, maps, tb, ring, slot, g, lane);
    produce_weights<T, true>(a, maps, tb, ring, slot, g, lane);
    if (lane == 0) drain(ring, slot, g);
    return;
  }
  if (warp > kConsumers) {
    const int w = warp - kConsumers - 1;
    produce_tokens<T, false>(a, tb, ring, slot, g, w, lane);
    if (lane == 0) grid_wait(&a.barrier[0], g);
    __syncwarp();
    produce_tokens<T, true>(a, tb, ring, slot, g, w, lane);
    cp_async_wait();
    return;
  }
  int buffer = 0;
  consume<D, T, false>(a, tb, ring, slot, red, buffer, g);
  consumers_sync();
  if (threadIdx.x == 0) grid_arrive(&a.barrier[0]);
  consume<D, T, true>(a, tb, ring, slot, red, buffer, g);
  consumers_sync();
  if (threadIdx.x == 0) {
    grid_arrive(&a.barrier[1]);
    grid_wait(&a.barrier[1], g);
  }
  consumers_sync();
  if (a.eights) combine<D, 8>(a, tb);
  else combine<D, 1>(a, tb);
}

// ------------------------------------------------------------ workspace

inline int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Byte offsets of the workspace's parts, and its size.
struct Space { int64_t logits, h, y, bytes; };

Space layer_space(int64_t tokens, int64_t hidden, int64_t inter, int64_t E, int64_t K) {
  Space s;
  s.logits = 256;                                        // the barrier words come first
  s.h = s.logits + up256(tokens * E * 4);
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

template <class D, Tiling T>
int launch_experts(const Layer& a, const WeightMaps& maps, int sms, cudaStream_t stream) {
  constexpr size_t smem = kRingBytes + 1024;
  if (int rc = ensure_smem_limit((const void*)layer_experts<D, T>, smem)) return rc;
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
  (void)cudaLaunchKernelEx(&cfg, layer_experts<D, T>, a, maps);
  return check_launch();
}

template <class D>
int launch(const Layer& a, cudaStream_t stream) {
  if (a.router_f32) launch_logits<D, F32>(a, stream);
  else launch_logits<D, D>(a, stream);
  if (int rc = check_launch()) return rc;
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  WeightMaps maps = {};
  if (a.hidden % 8 != 0 || a.ld_x % 8 != 0 || a.inter % 8 != 0 || !aligned16(a.x) ||
      !aligned16(a.w1) || !aligned16(a.w2))
    return launch_experts<D, kAny>(a, maps, sms, stream);
  // tiles of 16 rows for a few tokens whose experts make few tiles of 64: with fewer than 8 of
  // these a CTA, the last round would leave up to an eighth of the time of some CTAs idle
  const int64_t experts = a.E < (int64_t)a.tokens * a.K ? a.E : a.tokens * a.K;
  if ((a.tokens <= kNarrowTokens && experts * ((a.inter + 31) / 32) < 8 * (int64_t)sms) ||
      a.inter == 0)
    return launch_experts<D, kNarrow>(a, maps, sms, stream);
  if (int rc = weight_map(&maps.w1, a.w1, a.hidden, a.inter, 2 * (int64_t)a.E, 32)) return rc;
  if (int rc = weight_map(&maps.w2, a.w2, a.inter, a.hidden, a.E, 64)) return rc;
  return launch_experts<D, kWide>(a, maps, sms, stream);
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
  a.ld_h = (m.inter + 7) / 8 * 8;
  a.eights = m.hidden % kVec == 0 && m.ld_out % kVec == 0 && aligned16(m.out) &&
             (!m.shared || (m.ld_shared % kVec == 0 && aligned16(m.shared))) &&
             (!m.residual || (m.ld_residual % kVec == 0 && aligned16(m.residual)));
  a.logits = m.router_w ? a.own_logits : m.logits;
  a.logits_dt = m.router_w ? MOE_FP32 : m.logits_dt;
  a.ld_logits = m.router_w ? m.E : m.ld_logits;
  return m.dt == MOE_BF16 ? launch<BF16>(a, stream) : launch<F16>(a, stream);
}

}  // namespace moe
