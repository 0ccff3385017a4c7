// Layer norm of the rows of X [T, m] and its gradient.
//
//   mean = sum x / m;  var = sum (x - mean)^2 / m;  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd gamma + beta
//   xh = (x - mean) rstd;  g = dy gamma
//   dx = rstd (g - sum g / m - xh sum(g xh) / m);  dgamma = sum_rows dy xh;  dbeta = sum_rows dy
//
// All sums are fp32. The variance is summed from the deviations d from a first mean, not as
// E x^2 - mean^2, which loses every digit of rows whose offset is large against their spread; the
// deviations' own mean dm corrects the first one's rounding: mean = first + dm,
// var = sum d^2 / m - dm^2, x - mean = d - dm. Column sums are taken
// per range of rows and the ranges added in order: no atomics, the same bits on every run.
// Memory bound: each kernel reads its inputs once from HBM.
#include "norm.h"

#include <algorithm>

namespace poetx {
namespace norm {
namespace {

__device__ __forceinline__ float ld(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, int64_t i, float v) {
  p[i] = __float2bfloat16_rn(v);
}
// a weight of either type; NULL stands for `none` everywhere
__device__ __forceinline__ float ld_w(const void* w, int w_bf16, int64_t i, float none) {
  if (!w) return none;
  return w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                : static_cast<const float*>(w)[i];
}

// a variance that rounding left below zero counts as zero (NaN stays NaN)
__device__ __forceinline__ float rstd_of(float var, float eps) {
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

constexpr int kThreads = 256;

// sum over the block, the same value in every thread
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();   // the previous sum has been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

// One block per row, any width: the row is read again from cache for each sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) ln_fwd_any_kernel(const Fwd a) {
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
    const int64_t base = r * a.m;
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < a.m; i += kThreads) s += ld(x, base + i);
    const float mean = block_sum(s) / (float)a.m;
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = threadIdx.x; i < a.m; i += kThreads) {
      const float d = ld(x, base + i) - mean;
      s1 += d;
      s2 += d * d;
    }
    const float dm = block_sum(s1) / (float)a.m;
    const float rstd = rstd_of(block_sum(s2) / (float)a.m - dm * dm, a.eps);
    for (int64_t i = threadIdx.x; i < a.m; i += kThreads)
      st(y, base + i, (ld(x, base + i) - mean - dm) * rstd * ld_w(a.gamma, a.w_bf16, i, 1.f) +
                          ld_w(a.beta, a.w_bf16, i, 0.f));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean + dm;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_dx_any_kernel(const Bwd a) {
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.dx);
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
    const int64_t base = r * a.m;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = threadIdx.x; i < a.m; i += kThreads) {
      const float g = ld(dy, base + i) * ld_w(a.gamma, a.w_bf16, i, 1.f);
      s1 += g;
      s2 += g * ((ld(x, base + i) - mean) * rstd);
    }
    const float c1 = block_sum(s1) / (float)a.m, c2 = block_sum(s2) / (float)a.m;
    for (int64_t i = threadIdx.x; i < a.m; i += kThreads) {
      const float g = ld(dy, base + i) * ld_w(a.gamma, a.w_bf16, i, 1.f);
      const float xh = (ld(x, base + i) - mean) * rstd;
      st(dx, base + i, rstd * (g - c1 - xh * c2));
    }
  }
}

// Partial column sums of one range of rows: block (32 columns) x (8 rows at a time).
template <typename T>
__global__ void __launch_bounds__(kThreads) ln_cols_any_kernel(const Bwd a) {
  __shared__ float sg[8][33], sb[8][33];
  pdl_wait();
  pdl_trigger();
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  const int64_t per = (a.T + a.parts - 1) / a.parts;
  const int64_t lo = per * blockIdx.y, hi = min(a.T, lo + per);
  float g = 0.f, b = 0.f;
  if (c < a.m)
    for (int64_t r = lo + ty; r < hi; r += 8) {
      const float d = ld(dy, r * a.m + c);
      g += d * ((ld(x, r * a.m + c) - a.mean[r]) * a.rstd[r]);
      b += d;
    }
  sg[ty][tx] = g;
  sb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < a.m) {
    for (int k = 1; k < 8; ++k) {
      g += sg[k][tx];
      b += sb[k][tx];
    }
    a.part[(int64_t)blockIdx.y * a.m + c] = g;
    a.part[((int64_t)a.parts + blockIdx.y) * a.m + c] = b;
  }
}

// dgamma and dbeta: the ranges' sums added in order.
__global__ void __launch_bounds__(kThreads) ln_cols_sum_kernel(const Bwd a) {
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.m) return;
  float g = 0.f, b = 0.f;
  for (int p = 0; p < a.parts; ++p) {
    g += a.part[(int64_t)p * a.m + c];
    b += a.part[((int64_t)a.parts + p) * a.m + c];
  }
  if (a.dgamma) a.dgamma[c] = g;
  if (a.dbeta) a.dbeta[c] = b;
}

int row_blocks(int64_t T) { return (int)std::min<int64_t>(T, 148 * 8); }

}  // namespace

// ranges of rows that the column sums are split into
int parts_for(int64_t T, int64_t m) {
  (void)m;
  return (int)std::max<int64_t>(1, std::min<int64_t>(128, T / 64));
}

size_t bwd_ws_bytes(int64_t T, int64_t m) {
  if (T <= 0 || m <= 0) return 0;
  return (size_t)2 * (size_t)parts_for(T, m) * (size_t)m * sizeof(float);
}

cudaError_t fwd(const Fwd& a, DT t, cudaStream_t s) {
  TraceScope tr("ln_fwd", s);
  const dim3 grid((unsigned)row_blocks(a.T)), block(kThreads);
  return t == DT::BF16 ? launch_k(ln_fwd_any_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                       : launch_k(ln_fwd_any_kernel<float>, grid, block, 0, s, a);
}

cudaError_t bwd(Bwd a, DT t, void* ws, cudaStream_t s) {
  const dim3 block(kThreads);
  a.parts = parts_for(a.T, a.m);
  a.part = static_cast<float*>(ws);
  cudaError_t e = cudaSuccess;
  // the column sums first: dx may overwrite x or dy
  if (a.dgamma || a.dbeta) {
    {
      TraceScope tr("ln_bwd_cols", s);
      const dim3 grid((unsigned)((a.m + 31) / 32), (unsigned)a.parts);
      e = t == DT::BF16 ? launch_k(ln_cols_any_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                        : launch_k(ln_cols_any_kernel<float>, grid, block, 0, s, a);
      if (e != cudaSuccess) return e;
    }
    TraceScope tr("ln_bwd_sum", s);
    e = launch_k(ln_cols_sum_kernel, dim3((unsigned)((a.m + kThreads - 1) / kThreads)), block, 0,
                 s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dx) {
    TraceScope tr("ln_bwd_dx", s);
    const dim3 grid((unsigned)row_blocks(a.T));
    e = t == DT::BF16 ? launch_k(ln_dx_any_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                      : launch_k(ln_dx_any_kernel<float>, grid, block, 0, s, a);
  }
  return e;
}

}  // namespace norm
}  // namespace poetx
