// layer_norm.cu -- layer norm over the hidden axis, forward and backward.
//
//   mean = 1/H sum_h x,  var = 1/H sum_h (x - mean)^2,  rstd = (var + eps)^-1/2
//   y    = (x - mean) * rstd * w + b
// and, with xhat = (x - mean) * rstd and a = dy * w,
//   dx = rstd * (a - mean_h(a) - xhat * mean_h(a * xhat))
//   dw = sum_r dy * xhat,   db = sum_r dy
//
// All sums are fp32.  The variance is taken around the mean in a second pass
// (E[x^2] - mean^2 loses every digit of rows whose mean is large).  The
// parameter gradients are summed in two fixed steps: up to kNormGroups groups of
// rows, each in row order, then the groups' partial sums in group order.  The
// groups follow from the sizes, the types and the alignment of the data, so the
// bits depend neither on the launch nor on the device.
//
// HBM bandwidth bounds both passes: the rows are read once, held in registers,
// and written once.  A warp holds a short row, a CTA a long one; a thread loads
// 8 consecutive elements at a time, or single ones where the rows do not start
// on 16-byte boundaries or the width is no multiple of 8.  Rows beyond 8192
// (16384: forward, in eights) elements take the *_any kernels, which read them
// again for each pass.
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int kNormGroups = 148;   // row groups of the parameter gradients (one per SM)

// Groups of `rows` rows that are taken `at_once` at a time.
inline int norm_groups(int64_t rows, int at_once = 1) {
  const int64_t n = (rows + at_once - 1) / at_once;
  return (int)(n < kNormGroups ? n : kNormGroups);
}

// Error bits of waits that gave up (read by moe_device_errors).
__device__ int32_t g_norm_errors;

// Sum over the CTA's threads, the same on every thread; `red` is one slot of
// a double buffer (a caller alternates two of them between barriers).
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  return s;
}

// ------------------------------------------------------------ any width

// One CTA per row; three passes over the row (the second and third read it
// from L1 / L2).  Any width, stride and alignment.
template <class D, class W>
__global__ void __launch_bounds__(kThreads)
norm_fwd_any(const typename D::T* __restrict__ x, const typename W::T* __restrict__ w,
             const typename W::T* __restrict__ b, typename D::T* __restrict__ y,
             float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t rows,
             int64_t hidden, int64_t ld_x, int64_t ld_y, float eps) {
  pdl_prologue();
  __shared__ float red[2][kThreads / 32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const typename D::T* xr = x + r * ld_x;
    float s = 0.f;
    for (int64_t h = threadIdx.x; h < hidden; h += kThreads) s += load1<D>(xr + h);
    const float mean = cta_sum(s, red[0]) / (float)hidden;
    s = 0.f;
    for (int64_t h = threadIdx.x; h < hidden; h += kThreads) {
      const float d = load1<D>(xr + h) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = __frsqrt_rn(cta_sum(s, red[1]) / (float)hidden + eps);
    for (int64_t h = threadIdx.x; h < hidden; h += kThreads) {
      const float v = (load1<D>(xr + h) - mean) * rstd * load1<W>(w + h);
      store1<D>(y + r * ld_y + h, b ? v + load1<W>(b + h) : v);
    }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

template <class D, class W>
__global__ void __launch_bounds__(kThreads)
norm_bwd_rows_any(const typename D::T* __restrict__ gy, const typename D::T* __restrict__ x,
                  const typename W::T* __restrict__ w, const float* __restrict__ mean,
                  const float* __restrict__ rstd, typename D::T* __restrict__ gx, int64_t rows,
                  int64_t hidden, int64_t ld_gy, int64_t ld_x, int64_t ld_gx) {
  pdl_prologue();
  __shared__ float red[2][kThreads / 32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const typename D::T *xr = x + r * ld_x, *gr = gy + r * ld_gy;
    const float m = __ldg(mean + r), rs = __ldg(rstd + r);
    float s1 = 0.f, s2 = 0.f;
    for (int64_t h = threadIdx.x; h < hidden; h += kThreads) {
      const float a = load1<D>(gr + h) * load1<W>(w + h);
      s1 += a;
      s2 = fmaf(a, (load1<D>(xr + h) - m) * rs, s2);
    }
    s1 = cta_sum(s1, red[0]) / (float)hidden;
    s2 = cta_sum(s2, red[1]) / (float)hidden;
    for (int64_t h = threadIdx.x; h < hidden; h += kThreads) {
      const float a = load1<D>(gr + h) * load1<W>(w + h);
      const float xh = (load1<D>(xr + h) - m) * rs;
      store1<D>(gx + r * ld_gx + h, rs * (a - s1 - xh * s2));
    }
  }
}

// Partial parameter gradients of row group blockIdx.y: one thread per column.
template <class D>
__global__ void __launch_bounds__(kThreads)
norm_bwd_cols_any(const typename D::T* __restrict__ gy, const typename D::T* __restrict__ x,
                  const float* __restrict__ mean, const float* __restrict__ rstd,
                  float* __restrict__ pw, float* __restrict__ pb, int64_t rows, int64_t hidden,
                  int64_t ld_gy, int64_t ld_x) {
  pdl_prologue();
  const int64_t h = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (h >= hidden) return;
  float dw = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const float g = load1<D>(gy + r * ld_gy + h);
    dw = fmaf(g, (load1<D>(x + r * ld_x + h) - __ldg(mean + r)) * __ldg(rstd + r), dw);
    db += g;
  }
  pw[(int64_t)blockIdx.y * hidden + h] = dw;
  pb[(int64_t)blockIdx.y * hidden + h] = db;
}

// ------------------------------------------------------------ rows in registers

// VEC consecutive elements: raw bits as loaded, and widened.
template <class D, int VEC> struct Unit;
template <class D> struct Unit<D, 8> {
  Raw8<D> raw;
  __device__ __forceinline__ void load(const typename D::T* p) { raw = load8<D>(p); }
  __device__ __forceinline__ void load_shared(const typename D::T* p) { raw = tma::lds8<D>(p); }
  // a parameter: read by every row, so kept in L1
  __device__ __forceinline__ void load_param(const typename D::T* p) {
#pragma unroll
    for (int i = 0; i < D::kBytes / 2; ++i) raw.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const { widen8<D>(raw, v); }
  static __device__ __forceinline__ void store(typename D::T* p, const float (&v)[8]) {
    store8<D>(p, v);
  }
};
template <class D> struct Unit<D, 1> {
  // (as loaded: widening here would wait for each element before the next is asked for)
  typename D::T raw;
  __device__ __forceinline__ void load(const typename D::T* p) { raw = __ldg(p); }
  __device__ __forceinline__ void load_param(const typename D::T* p) { raw = __ldg(p); }
  __device__ __forceinline__ void widen(float (&v)[1]) const {
    if constexpr (std::is_same<D, BF16>::value) v[0] = __uint_as_float((uint32_t)raw << 16);
    else if constexpr (std::is_same<D, F16>::value) v[0] = f16_to_f32(raw);
    else v[0] = raw;
  }
  static __device__ __forceinline__ void store(typename D::T* p, const float (&v)[1]) {
    store1<D>(p, v[0]);
  }
};

// Sum over a team of TPR threads (a power of two of warps), the same on each of
// them; `red` as for cta_sum.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* red) {
  if constexpr (TPR == 32) return warp_sum(v);
  if constexpr (TPR == kThreads) return cta_sum(v, red);
  const int team = threadIdx.x / TPR;
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TPR) : "memory");
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < TPR / 32; ++i) s += red[team * (TPR / 32) + i];
  return s;
}

// TPR threads per row, C units of VEC elements per thread; the next row is loaded
// while this one is reduced.  Four units a thread and as few threads as that
// needs: a row's sums then meet few barriers, and several rows share a CTA (16384
// x 2048 bf16: 38 us with a CTA to a row).
template <class D, class W, int VEC, int C, int TPR>
__global__ void __launch_bounds__(kThreads)
norm_fwd_rows(const typename D::T* __restrict__ x, const typename W::T* __restrict__ w,
              const typename W::T* __restrict__ b, typename D::T* __restrict__ y,
              float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t rows,
              int hidden, int64_t ld_x, int64_t ld_y, float eps) {
  pdl_prologue();
  __shared__ float red[2][kThreads / 32];
  const int t = threadIdx.x % TPR;
  constexpr int kRows = kThreads / TPR;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  Unit<D, VEC> next[C];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + t) * VEC;
      if (h < hidden) next[c].load(x + row * ld_x + h);
    }
  };
  if (r < rows) load(r);
  // Single elements: the thread's parameters in registers for all its rows (a load for each
  // element of each row took as long as the rest).  Eights: from L1 as they are needed.
  constexpr bool kKeep = VEC == 1;
  float keep_w[kKeep ? C : 1], keep_b[kKeep ? C : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = c * TPR + t;
      keep_w[c] = h < hidden ? load1<W>(w + h) : 0.f;
      keep_b[c] = b && h < hidden ? load1<W>(b + h) : 0.f;
    }
  }
  for (; r < rows; r += step) {
    float v[C][VEC];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if ((c * TPR + t) * VEC < hidden) {
        next[c].widen(v[c]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += v[c][i];
      }
    }
    if (r + step < rows) load(r + step);
    const float mean = team_sum<TPR>(s, red[0]) / (float)hidden;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if ((c * TPR + t) * VEC < hidden) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          v[c][i] -= mean;
          s = fmaf(v[c][i], v[c][i], s);
        }
      }
    }
    const float rstd = __frsqrt_rn(team_sum<TPR>(s, red[1]) / (float)hidden + eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + t) * VEC;
      if (h < hidden) {
        if constexpr (kKeep) {
          v[c][0] = v[c][0] * rstd * keep_w[c];
          if (b) v[c][0] += keep_b[c];
        } else {
          Unit<W, VEC> u;
          float p[VEC];
          u.load_param(w + h);
          u.widen(p);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[c][i] = v[c][i] * rstd * p[i];
          if (b) {
            u.load_param(b + h);
            u.widen(p);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[c][i] += p[i];
          }
        }
        Unit<D, VEC>::store(y + r * ld_y + h, v[c]);
      }
    }
    if (t == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

// Packed pairs of fp32 (one instruction for both on sm_100), or single values.
struct Two { unsigned long long v; };
__device__ __forceinline__ Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split2(const Two& a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ Two add(Two a, Two b) {
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
  return a;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
  return a;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(c.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return c;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }

// The VEC elements of a unit as pairs (VEC 8) or as they are (VEC 1).
template <int VEC> struct Lanes;
template <> struct Lanes<8> {
  using T = Two;
  static constexpr int N = 4;
  static __device__ __forceinline__ Two all(float v) { return two(v, v); }
  static __device__ __forceinline__ void pack(const float (&v)[8], Two (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = two(v[2 * i], v[2 * i + 1]);
  }
  static __device__ __forceinline__ void unpack(const Two (&v)[4], float (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(v[i], o[2 * i], o[2 * i + 1]);
  }
  static __device__ __forceinline__ float total(const Two& a) {
    float lo, hi;
    split2(a, lo, hi);
    return lo + hi;
  }
};
template <> struct Lanes<1> {
  using T = float;
  static constexpr int N = 1;
  static __device__ __forceinline__ float all(float v) { return v; }
  static __device__ __forceinline__ void pack(const float (&v)[1], float (&o)[1]) { o[0] = v[0]; }
  static __device__ __forceinline__ void unpack(const float (&v)[1], float (&o)[1]) { o[0] = v[0]; }
  static __device__ __forceinline__ float total(float a) { return a; }
};

// Backward.  One CTA of 16 warps per row group; a team of WPR warps takes a row,
// so that 16 / WPR rows are in work at once, each thread with C units of VEC
// columns and their shares of the parameter gradients in registers for all its
// rows.
//   gather(k)  row k's terms of the parameter gradients, and the two sums over
//              this warp's columns
//   finish(k)  the sums over the team, grad_x
// With VEC = 8 the rows of x and grad_y come through a ring of `stages` stages in
// shared memory (bulk copies) and finish reads them there again: registers go to
// the gradients' shares, so that few warps hold a row and several rows' chains of
// dependent steps (about 1 us each) overlap.  Single elements are loaded a row
// ahead and kept in registers.  The arithmetic is packed in pairs (one
// instruction for two elements).  At 16384 x 7168 bf16: one row at a time over 16
// warps 229 us, over 32 warps 167, with the next row gathered first 169.
constexpr int kBwdSmem = 222 * 1024;      // the ring, then the weights in fp32

// Sums a and b over the warp with shared butterflies (the first step leaves each
// half of the warp with one of them): lanes 0 .. 15 return a's, the others b's.
__device__ __forceinline__ float warp_sum2(float a, float b) {
  constexpr unsigned kAll = 0xffffffffu;
  const bool up = threadIdx.x & 16;
  float v = (up ? b : a) + __shfl_xor_sync(kAll, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

constexpr int kBwdThreads = 512;

// STALLED (tests of the bounded waits): row `stall`'s copies are withheld, and waits
// give up after `limit` cycles.
template <class D, class W, int VEC, int C, int WPR, bool STALLED = false>
__global__ void __launch_bounds__(kBwdThreads, 1)
norm_bwd_rows(const typename D::T* __restrict__ gy, const typename D::T* __restrict__ x,
              const typename W::T* __restrict__ w, const float* __restrict__ mean,
              const float* __restrict__ rstd, typename D::T* __restrict__ gx,
              float* __restrict__ pw, float* __restrict__ pb, int64_t rows, int hidden,
              int64_t ld_gy, int64_t ld_x, int64_t ld_gx, int stages, int64_t stall,
              long long limit) {
  using T = typename D::T;
  using L = Lanes<VEC>;
  using P = typename L::T;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kWarps = kBwdThreads / 32, kTeams = kWarps / WPR, TPR = WPR * 32, N = L::N;
  constexpr bool kRing = VEC == 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 slots[2][kWarps];     // the warps' sums, in turn by row
  __shared__ uint64_t bars[kTeams * 8];
  __shared__ float2 stats[kTeams * 8];    // mean and rstd of the stages' rows
  const int team = threadIdx.x / TPR, t = threadIdx.x % TPR, lane = threadIdx.x & 31;
  if (kRing && threadIdx.x == 0) {
    for (int i = 0; i < kTeams * 8; ++i) tma::mbar_init(&bars[i], 1);
    tma::mbar_init_fence();
  }
  pdl_prologue();
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kTeams + team, step = (int64_t)gridDim.x * kTeams;
  const int n = rows > first ? (int)((rows - 1 - first) / step + 1) : 0;
  const uint32_t row_bytes = (uint32_t)hidden * sizeof(T);
  uint8_t* ring = smem + (size_t)team * stages * 2 * row_bytes;
  uint64_t* full = bars + team * 8;
  // A thread whose wait gave up waits no more; the team's first thread then fetches nothing more
  // (as long as it waits itself, it refills a stage only when the copies before have landed), and
  // waits at the end for what it asked for.
  bool dead = false;
  const long long cycles = STALLED ? limit : tma::kWaitCycles;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (tma::mbar_try(bar, parity) || dead) return;
    if (!tma::mbar_wait(bar, parity, cycles)) {
      atomicOr(&g_norm_errors, MOE_DEVERR_TIMEOUT);
      dead = true;
    }
  };
  // The stages are used in turn: `put` and `get` walk through them.
  int put = 0, get = 0, issued = 0;
  uint32_t parity = 0;
  float next_m = 0.f, next_rs = 0.f;      // the statistics of the row to be loaded next
  auto load_stats = [&](int k) {
    if (k < n) {
      next_m = __ldg(mean + first + k * step);
      next_rs = __ldg(rstd + first + k * step);
    }
  };
  load_stats(0);
  auto issue = [&] {                      // the next row's copies; by the team's first thread
    const int64_t r = first + issued * step;
    uint8_t* dst = ring + (size_t)put * 2 * row_bytes;
    stats[team * 8 + put] = make_float2(next_m, next_rs);
    if (!STALLED || r != stall) {
      tma::mbar_arrive_expect_tx(&full[put], 2 * row_bytes);
      tma::bulk_load(dst, x + r * ld_x, row_bytes, &full[put]);
      tma::bulk_load(dst + row_bytes, gy + r * ld_gy, row_bytes, &full[put]);
    }
    load_stats(++issued);
    if (++put == stages) put = 0;
  };
  Unit<D, VEC> nx[kRing ? 1 : C], ng[kRing ? 1 : C];
  auto load = [&](int k) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + t) * VEC;
      if (h < hidden) {
        nx[c].load(x + (first + k * step) * ld_x + h);
        ng[c].load(gy + (first + k * step) * ld_gy + h);
      }
    }
  };
  if constexpr (kRing) {
    if (t == 0)
      while (issued < stages && issued < n) issue();
  } else {
    if (n > 0) load(0);
  }
  // With VEC = 8 the weights lie in shared memory (a unit's halves in two planes,
  // free of bank conflicts), else in registers.
  float4* const weights = reinterpret_cast<float4*>(smem + (size_t)kTeams * stages * 2 * row_bytes);
  const int units = hidden / 8;
  P kept[kRing ? 1 : C][N];
  if constexpr (kRing) {
    for (int c = threadIdx.x; c < units; c += blockDim.x) {
      Unit<W, VEC> u;
      float v[VEC];
      u.load_param(w + c * 8);
      u.widen(v);
      weights[c] = make_float4(v[0], v[1], v[2], v[3]);
      weights[units + c] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
  }
  P dw[C][N], db[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * TPR + t) * VEC;
    if constexpr (!kRing) {
      if (h < hidden) {
        Unit<W, VEC> u;
        float v[VEC];
        u.load_param(w + h);
        u.widen(v);
        L::pack(v, kept[c]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) dw[c][i] = db[c][i] = L::all(0.f);
  }
  auto param = [&](int c, P (&p)[N]) {
    if constexpr (kRing) {
      const float4 lo = weights[c * TPR + t], hi = weights[units + c * TPR + t];
      const float v[VEC] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      L::pack(v, p);
    } else {
      p[0] = kept[c][0];
    }
  };
  const float inv = 1.0f / (float)hidden;

  P xh[kRing ? 1 : C][N], av[kRing ? 1 : C][N];      // the row's xhat and grad_y * weight
  float m, rs, sum;                       // sum: this lane's of the two (warp_sum2)
  // xhat, grad_y and a of unit c, from the stage `src` or the registers loaded.
  auto unit = [&](const T* src, int c, P (&xv)[N], P (&gv)[N], P (&a)[N]) {
    const int h = (c * TPR + t) * VEC;
    if constexpr (kRing) {
      nx[0].load_shared(src + h);
      ng[0].load_shared(src + hidden + h);
    }
    P p[N];
    float v[VEC];
    param(c, p);
    nx[kRing ? 0 : c].widen(v);
    L::pack(v, xv);
    ng[kRing ? 0 : c].widen(v);
    L::pack(v, gv);
    const P sub = L::all(-m), scale = L::all(rs);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      xv[i] = mul(add(xv[i], sub), scale);
      a[i] = mul(gv[i], p[i]);
    }
  };
  auto stage = [&](int at) { return reinterpret_cast<const T*>(ring + (size_t)at * 2 * row_bytes); };
  for (int k = 0; k < n; ++k) {
    // ---- gather
    const int at = get;
    if constexpr (kRing) {
      wait(&full[get], parity);
      const float2 st = stats[team * 8 + get];
      m = st.x;
      rs = st.y;
      if (++get == stages) { get = 0; parity ^= 1u; }
    } else {
      m = next_m;
      rs = next_rs;
      load_stats(k + 1);
    }
    P t1 = L::all(0.f), t2 = L::all(0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if ((c * TPR + t) * VEC < hidden) {
        P xv[N], gv[N], a[N];
        unit(stage(at), c, xv, gv, a);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dw[c][i] = fma(gv[i], xv[i], dw[c][i]);
          db[c][i] = add(db[c][i], gv[i]);
          t1 = add(t1, a[i]);
          t2 = fma(a[i], xv[i], t2);
          if constexpr (!kRing) {
            xh[c][i] = xv[i];
            av[c][i] = a[i];
          }
        }
      }
    }
    if constexpr (!kRing) {
      if (k + 1 < n) load(k + 1);
    }
    sum = warp_sum2(L::total(t1), L::total(t2));
    float v = sum;
    if constexpr (WPR > 1) {
      if ((lane & 15) == 0)
        reinterpret_cast<float*>(&slots[k & 1][threadIdx.x >> 5])[lane >> 4] = sum;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TPR) : "memory");
      // ---- finish: lanes 0 .. 15 the first sum of the team's warps, the others the second
      v = reinterpret_cast<const float*>(slots[k & 1] + team * WPR)[(lane & (WPR - 1)) * 2 +
                                                                   (lane >> 4)];
#pragma unroll
      for (int o = WPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    }
    const float s1 = __shfl_sync(kAll, v, 0) * inv, s2 = __shfl_sync(kAll, v, 16) * inv;
    // The team has met (a warp alone: met itself), so it has finished the row before: that
    // row's stage can be refilled.
    if constexpr (kRing) {
      if (WPR == 1) __syncwarp();
      if (t == 0 && !dead && k > 0 && issued < n) issue();
    }
    // rstd (a - mean(a) - xhat mean(a xhat))
    const P scale = L::all(rs), a1 = L::all(-rs * s1), a2 = L::all(-rs * s2);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = (c * TPR + t) * VEC;
      if (h < hidden) {
        P xv[N], gv[N], a[N];
        float out[VEC];
        if constexpr (kRing) {
          unit(stage(at), c, xv, gv, a);
        } else {
          xv[0] = xh[c][0];
          a[0] = av[c][0];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = fma(xv[i], a2, fma(a[i], scale, a1));
        L::unpack(a, out);
        Unit<D, VEC>::store(gx + (first + k * step) * ld_gx + h, out);
      }
    }
  }
  if (kRing && dead && t == 0)            // before the CTA ends, its copies land
    for (int k = issued > stages ? issued - stages : 0; k < issued; ++k)
      tma::mbar_wait(&full[k % stages], (uint32_t)(k / stages) & 1, cycles);
  pw += (int64_t)blockIdx.x * hidden;
  pb += (int64_t)blockIdx.x * hidden;
  if constexpr (kTeams > 1) __syncthreads();   // every team is done with its ring
  float* all = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * TPR + t) * VEC;
    if (h < hidden) {
      float vw[VEC], vb[VEC];
      L::unpack(dw[c], vw);
      L::unpack(db[c], vb);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        (kTeams == 1 ? pw : all + team * hidden)[h + i] = vw[i];
        (kTeams == 1 ? pb : all + (kTeams + team) * hidden)[h + i] = vb[i];
      }
    }
  }
  if constexpr (kTeams > 1) {             // the teams' shares, in their order
    __syncthreads();
    for (int h = threadIdx.x; h < 2 * hidden; h += blockDim.x) {
      const bool bias = h >= hidden;
      const float* v = all + (bias ? kTeams * hidden + h - hidden : h);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kTeams; ++i) s += v[i * hidden];
      (bias ? pb + h - hidden : pw + h)[0] = s;
    }
  }
}

// Sums the groups' partials of 32 columns per CTA: warps 0 .. 15 the weight's,
// the others the bias's; warp i takes the groups i, i + 16, ..., in order, and
// the sixteen sums are added in warp order.
constexpr int kSumThreads = 1024, kSumWarps = kSumThreads / 64;

template <class W>
__global__ void __launch_bounds__(kSumThreads)
norm_bwd_groups(const float* __restrict__ pw, const float* __restrict__ pb,
                typename W::T* __restrict__ gw, typename W::T* __restrict__ gb, int groups,
                int64_t hidden) {
  pdl_prologue();
  __shared__ float sums[2][kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool bias = warp >= kSumWarps;
  const int64_t h = (int64_t)blockIdx.x * 32 + lane;
  const float* src = bias ? pb : pw;
  typename W::T* dst = bias ? gb : gw;
  float s = 0.f;
  if (h < hidden && dst) {
#pragma unroll
    for (int i = 0; i < (kNormGroups + kSumWarps - 1) / kSumWarps; ++i) {
      const int g = i * kSumWarps + (warp & (kSumWarps - 1));
      if (g < groups) s += __ldg(src + g * hidden + h);
    }
  }
  sums[bias][warp & (kSumWarps - 1)][lane] = s;
  __syncthreads();
  if ((warp & (kSumWarps - 1)) == 0 && h < hidden && dst) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) s += sums[bias][i][lane];
    store1<W>(dst + h, s);
  }
}

// ------------------------------------------------------------ launchers

// In eights where every row and parameter starts on a 16-byte boundary.
inline bool eights(int64_t hidden, std::initializer_list<const void*> ps,
                   std::initializer_list<int64_t> lds) {
  bool ok = hidden % kVec == 0;
  for (const void* p : ps) ok = ok && aligned16(p);
  for (int64_t ld : lds) ok = ok && ld % kVec == 0;
  return ok;
}

template <class D, class W>
int fwd(const void* x_, const void* w_, const void* b_, void* y_, float* mean, float* rstd,
        int64_t rows, int64_t hidden, int64_t ld_x, int64_t ld_y, float eps,
        cudaStream_t stream) {
  const auto* x = static_cast<const typename D::T*>(x_);
  const auto *w = static_cast<const typename W::T*>(w_), *b = static_cast<const typename W::T*>(b_);
  auto* y = static_cast<typename D::T*>(y_);
  int grid = 0;
  auto rows_in_registers = [&](auto k, int per_cta) {
    if (int rc = persistent_grid((const void*)k, 0, (rows + per_cta - 1) / per_cta, &grid))
      return rc;
    launch_kernel(k, grid, 0, stream, x, w, b, y, mean, rstd, rows, (int)hidden, ld_x, ld_y, eps);
    return check_launch();
  };
  if (eights(hidden, {x, w, b, y}, {ld_x, ld_y}) && hidden <= 16384) {
    const int64_t n = hidden / kVec;
    if (n <= 32) return rows_in_registers(norm_fwd_rows<D, W, 8, 1, 32>, 8);
    if (n <= 64) return rows_in_registers(norm_fwd_rows<D, W, 8, 2, 32>, 8);
    if (n <= 128) return rows_in_registers(norm_fwd_rows<D, W, 8, 4, 32>, 8);
    if (n <= 256) return rows_in_registers(norm_fwd_rows<D, W, 8, 4, 64>, 4);
    if (n <= 512) return rows_in_registers(norm_fwd_rows<D, W, 8, 4, 128>, 2);
    if (n <= 1024) return rows_in_registers(norm_fwd_rows<D, W, 8, 4, 256>, 1);
    return rows_in_registers(norm_fwd_rows<D, W, 8, 8, 256>, 1);
  }
  // Single elements, bf16, us: 65536 x 255 with a warp to a row 20.5, with two 29.2; 32768 x 511
  // with a warp 35.2, with a CTA 45.4; 16384 x 1001 with a CTA 29.7 (fp32 29.8), with four warps
  // and 8 elements a thread 21.4 (26.1), with two and 16 36.1; 16384 x 2001 with a CTA 42.3, with
  // four warps 71.7; 8192 x 4001 with a CTA 69.2, with four warps and 32 elements a thread 62.9.
  if (hidden <= 256) return rows_in_registers(norm_fwd_rows<D, W, 1, 8, 32>, 8);
  if (hidden <= 512) return rows_in_registers(norm_fwd_rows<D, W, 1, 16, 32>, 8);
  if (hidden <= 1024) return rows_in_registers(norm_fwd_rows<D, W, 1, 4, 256>, 1);
  if (hidden <= 2048) return rows_in_registers(norm_fwd_rows<D, W, 1, 8, 256>, 1);
  if (hidden <= 4096) return rows_in_registers(norm_fwd_rows<D, W, 1, 16, 256>, 1);
  if (hidden <= 8192) return rows_in_registers(norm_fwd_rows<D, W, 1, 32, 256>, 1);
  auto k = norm_fwd_any<D, W>;
  if (int rc = persistent_grid((const void*)k, 0, rows, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, x, w, b, y, mean, rstd, rows, hidden, ld_x, ld_y, eps);
  return check_launch();
}

template <class D, class W>
int bwd(const void* gy_, const void* x_, const void* w_, const float* mean, const float* rstd,
        void* gx_, void* gw_, void* gb_, float* ws, int64_t rows, int64_t hidden, int64_t ld_gy,
        int64_t ld_x, int64_t ld_gx, int64_t stall, long long limit, cudaStream_t stream) {
  const auto* gy = static_cast<const typename D::T*>(gy_);
  const auto* x = static_cast<const typename D::T*>(x_);
  const auto* w = static_cast<const typename W::T*>(w_);
  auto* gx = static_cast<typename D::T*>(gx_);
  int groups = 0;
  float *pw = ws, *pb = nullptr;
  auto rows_in_registers = [&](auto k, int vec, int teams) {
    groups = norm_groups(rows, teams);
    pb = ws + groups * hidden;
    const int64_t stage = 2 * teams * hidden * (int64_t)sizeof(typename D::T);
    const int64_t fit = (kBwdSmem - hidden * 4) / stage;
    const int stages = vec == 8 ? (int)(fit < 8 ? fit : 8) : 0;
    // the ring and the weights; afterwards the teams' shares of the parameter gradients
    int64_t smem = vec == 8 ? stages * stage + hidden * 4 : 0;
    if (teams > 1 && smem < 2 * teams * hidden * 4) smem = 2 * teams * hidden * 4;
    if (int rc = ensure_smem_limit((const void*)k, kBwdSmem)) return rc;
    launch_kernel_block(k, groups, kBwdThreads, (size_t)smem, stream, gy, x, w, mean, rstd, gx, pw,
                        pb, rows, (int)hidden, ld_gy, ld_x, ld_gx, stages, stall, limit);
    return check_launch();
  };
  int rc = MOE_OK;
  const bool vec = eights(hidden, {gy, x, w, gx}, {ld_gy, ld_x, ld_gx});
  // 4 units a thread where the ring then holds two stages at least of every team (fp32: 2)
  constexpr int C = D::kBytes == 2 ? 4 : 2, F = 4 / C;
  constexpr bool kStalls = std::is_same<D, BF16>::value && std::is_same<W, F32>::value;
  if (kStalls && stall >= 0)
    rc = hidden <= 1024 ? rows_in_registers(norm_bwd_rows<D, W, 8, C, F, kStalls>, 8, 16 / F)
                        : rows_in_registers(norm_bwd_rows<D, W, 8, C, 8 * F, kStalls>, 8, 2 / F);
  else if (vec && hidden <= 256) rc = rows_in_registers(norm_bwd_rows<D, W, 8, 1, 1>, 8, 16);
  else if (vec && hidden <= 512) rc = rows_in_registers(norm_bwd_rows<D, W, 8, 2, 1>, 8, 16);
  else if (vec && hidden <= 1024) rc = rows_in_registers(norm_bwd_rows<D, W, 8, C, F>, 8, 16 / F);
  else if (vec && hidden <= 2048)
    rc = rows_in_registers(norm_bwd_rows<D, W, 8, C, 2 * F>, 8, 8 / F);
  else if (vec && hidden <= 4096)
    rc = rows_in_registers(norm_bwd_rows<D, W, 8, C, 4 * F>, 8, 4 / F);
  else if (vec && hidden <= 8192)
    rc = rows_in_registers(norm_bwd_rows<D, W, 8, C, 8 * F>, 8, 2 / F);
  else if (hidden <= 256) rc = rows_in_registers(norm_bwd_rows<D, W, 1, 8, 1>, 1, 16);
  else if (hidden <= 1024) rc = rows_in_registers(norm_bwd_rows<D, W, 1, 8, 4>, 1, 4);
  else if (hidden <= 4096) rc = rows_in_registers(norm_bwd_rows<D, W, 1, 8, 16>, 1, 1);
  else if (hidden <= 8192) rc = rows_in_registers(norm_bwd_rows<D, W, 1, 16, 16>, 1, 1);
  else {
    groups = norm_groups(rows);
    pb = ws + groups * hidden;
    int grid = 0;
    auto kr = norm_bwd_rows_any<D, W>;
    if (int e = persistent_grid((const void*)kr, 0, rows, &grid)) return e;
    launch_kernel(kr, grid, 0, stream, gy, x, w, mean, rstd, gx, rows, hidden, ld_gy, ld_x, ld_gx);
    if (int e = check_launch()) return e;
    const dim3 cols((unsigned)((hidden + kThreads - 1) / kThreads), (unsigned)groups);
    launch_kernel_grid(norm_bwd_cols_any<D>, cols, kThreads, 0, stream, gy, x, mean, rstd, pw, pb,
                       rows, hidden, ld_gy, ld_x);
    rc = check_launch();
  }
  if (rc) return rc;
  launch_kernel_block(norm_bwd_groups<W>, (int)((hidden + 31) / 32), kSumThreads, 0, stream,
                      (const float*)pw, (const float*)pb, static_cast<typename W::T*>(gw_),
                      static_cast<typename W::T*>(gb_), groups, hidden);
  return check_launch();
}

}  // namespace

bool layer_norm_bwd_width_ok(int64_t hidden) {
  return hidden >= 0 && hidden <= INT64_MAX / 8 / (2 * kNormGroups * (int64_t)sizeof(float));
}

int64_t layer_norm_bwd_workspace(int64_t rows, int64_t hidden) {
  return 2 * (int64_t)norm_groups(rows) * hidden * (int64_t)sizeof(float);
}

int layer_norm_device_errors(int32_t* bits, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_norm_errors, sizeof(int32_t));
  if (e != cudaSuccess) return cuda_fail(e);
  if (clear) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_norm_errors, &zero, sizeof(int32_t));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MOE_OK;
}

#define MOE_NORM_DISPATCH(F, ...)                                                    \
  switch (dt) {                                                                      \
    case MOE_BF16:                                                                   \
      return w_dt == MOE_FP32 ? F<BF16, F32>(__VA_ARGS__) : F<BF16, BF16>(__VA_ARGS__); \
    case MOE_FP16:                                                                   \
      return w_dt == MOE_FP32 ? F<F16, F32>(__VA_ARGS__) : F<F16, F16>(__VA_ARGS__); \
    default: return F<F32, F32>(__VA_ARGS__);                                        \
  }

int launch_layer_norm_fwd(const void* x, const void* w, const void* b, void* y, float* mean,
                          float* rstd, int64_t rows, int64_t hidden, int64_t ld_x, int64_t ld_y,
                          float eps, moe_dtype dt, moe_dtype w_dt, cudaStream_t stream) {
  MOE_NORM_DISPATCH(fwd, x, w, b, y, mean, rstd, rows, hidden, ld_x, ld_y, eps, stream)
}

int launch_layer_norm_bwd(const void* gy, const void* x, const void* w, const float* mean,
                          const float* rstd, void* gx, void* gw, void* gb, float* ws,
                          int64_t rows, int64_t hidden, int64_t ld_gy, int64_t ld_x,
                          int64_t ld_gx, moe_dtype dt, moe_dtype w_dt, cudaStream_t stream) {
  const int64_t stall = -1;
  const long long limit = tma::kWaitCycles;
  MOE_NORM_DISPATCH(bwd, gy, x, w, mean, rstd, gx, gw, gb, ws, rows, hidden, ld_gy, ld_x, ld_gx,
                    stall, limit, stream)
}

int launch_layer_norm_bwd_stalled(const void* gy, const void* x, const float* w,
                                  const float* mean, const float* rstd, void* gx, float* gw,
                                  float* ws, int64_t rows, int64_t hidden, int64_t stall,
                                  long long limit, cudaStream_t stream) {
  return bwd<BF16, F32>(gy, x, w, mean, rstd, gx, gw, nullptr, ws, rows, hidden, hidden, hidden,
                        hidden, stall, limit, stream);
}

}  // namespace moe
