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
// parameter gradients are summed in two fixed steps: kNormGroups groups of
// rows (group g holds rows g, g + kNormGroups, ...), each in row order, then
// the groups' partial sums in group order.  The number of groups is a
// constant, so the bits depend neither on the launch nor on the device.
#include "common.cuh"
#include "launch.cuh"

namespace moe {

namespace {

constexpr int kNormGroups = 148;   // row groups of the parameter gradients (one per SM)

inline int norm_groups(int64_t rows) { return (int)(rows < kNormGroups ? rows : kNormGroups); }

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

// Sums the groups' partials of 32 columns per CTA: warp i takes the groups
// i, i + 8, ..., in order, and the eight warps' sums are added in warp order.
template <class W>
__global__ void __launch_bounds__(kThreads)
norm_bwd_groups(const float* __restrict__ pw, const float* __restrict__ pb,
                typename W::T* __restrict__ gw, typename W::T* __restrict__ gb, int groups,
                int64_t hidden) {
  pdl_prologue();
  __shared__ float sw[kThreads / 32][32], sb[kThreads / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t h = (int64_t)blockIdx.x * 32 + lane;
  float dw = 0.f, db = 0.f;
  if (h < hidden) {
#pragma unroll 4
    for (int g = warp; g < groups; g += kThreads / 32) {
      dw += __ldg(pw + g * hidden + h);
      db += __ldg(pb + g * hidden + h);
    }
  }
  sw[warp][lane] = dw;
  sb[warp][lane] = db;
  __syncthreads();
  if (warp == 0 && h < hidden) {
    dw = db = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      dw += sw[i][lane];
      db += sb[i][lane];
    }
    store1<W>(gw + h, dw);
    if (gb) store1<W>(gb + h, db);
  }
}

// ------------------------------------------------------------ launchers

template <class D, class W>
int fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
        int64_t rows, int64_t hidden, int64_t ld_x, int64_t ld_y, float eps,
        cudaStream_t stream) {
  auto k = norm_fwd_any<D, W>;
  int grid = 0;
  if (int rc = persistent_grid((const void*)k, 0, rows, &grid)) return rc;
  launch_kernel(k, grid, 0, stream, static_cast<const typename D::T*>(x),
                static_cast<const typename W::T*>(w), static_cast<const typename W::T*>(b),
                static_cast<typename D::T*>(y), mean, rstd, rows, hidden, ld_x, ld_y, eps);
  return check_launch();
}

template <class D, class W>
int bwd(const void* gy_, const void* x_, const void* w_, const float* mean, const float* rstd,
        void* gx_, void* gw_, void* gb_, float* ws, int64_t rows, int64_t hidden, int64_t ld_gy,
        int64_t ld_x, int64_t ld_gx, cudaStream_t stream) {
  const auto* gy = static_cast<const typename D::T*>(gy_);
  const auto* x = static_cast<const typename D::T*>(x_);
  const auto* w = static_cast<const typename W::T*>(w_);
  auto* gx = static_cast<typename D::T*>(gx_);
  const int groups = norm_groups(rows);
  float *pw = ws, *pb = ws + groups * hidden;
  int grid = 0;
  auto kr = norm_bwd_rows_any<D, W>;
  if (int rc = persistent_grid((const void*)kr, 0, rows, &grid)) return rc;
  launch_kernel(kr, grid, 0, stream, gy, x, w, mean, rstd, gx, rows, hidden, ld_gy, ld_x, ld_gx);
  if (int rc = check_launch()) return rc;
  const dim3 cols((unsigned)((hidden + kThreads - 1) / kThreads), (unsigned)groups);
  launch_kernel_grid(norm_bwd_cols_any<D>, cols, kThreads, 0, stream, gy, x, mean, rstd, pw, pb,
                     rows, hidden, ld_gy, ld_x);
  if (int rc = check_launch()) return rc;
  launch_kernel(norm_bwd_groups<W>, (int)((hidden + 31) / 32), 0, stream, (const float*)pw,
                (const float*)pb, static_cast<typename W::T*>(gw_),
                static_cast<typename W::T*>(gb_), groups, hidden);
  return check_launch();
}

}  // namespace

int64_t layer_norm_bwd_workspace(int64_t rows, int64_t hidden) {
  return 2 * (int64_t)norm_groups(rows) * hidden * (int64_t)sizeof(float);
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
  MOE_NORM_DISPATCH(bwd, gy, x, w, mean, rstd, gx, gw, gb, ws, rows, hidden, ld_gy, ld_x, ld_gx,
                    stream)
}

}  // namespace moe
