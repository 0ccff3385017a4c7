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
// Memory bound: the kernels of rows in registers and of rows through a ring read their inputs once
// from HBM. Rows too wide for them (forward: more than 16384 columns; backward: also fp32 rows of more than
// about 14300, of which two do not fit the ring) are read again for each sum, x and dy by a launch for
// the column sums besides: 2048 x 20000 bf16 161 us forward, 212 us backward, of 25 and 38 us for the
// bytes. No input is read through the read-only cache: a block may start before the kernel that
// writes the input has ended.
#include "norm.h"
#include "umma_ptx.cuh"

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

// rstd of a row from the deviations from its first mean: sq = sum d^2 / m, dm = sum d / m. A
// variance that rounding left below zero counts as zero (NaN stays NaN). A dm of less than half an
// ulp of the deviations is dropped: values of few bits and one exponent all round alike when the
// first mean is subtracted, which looks like a dm of that size, while the first mean of such
// values is often exact.
__device__ __forceinline__ float rstd_of(float sq, float& dm, float eps) {
  float var = sq - dm * dm;
  var = var < 0.f ? 0.f : var;
  if (fabsf(dm) <= 0x1p-24f * sqrtf(var)) dm = 0.f;
  return 1.f / sqrtf(var + eps);
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
    float dm = block_sum(s1) / (float)a.m;
    const float rstd = rstd_of(block_sum(s2) / (float)a.m, dm, a.eps);
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

// dgamma and dbeta: the ranges' sums, 32 columns per block; 32 threads of a column take every 32nd
// range, and their sums are added by a fixed tree. A launch of its own, since it needs every block's
// sums: the last block to finish could take them, but would be known by a counter only, which has
// to be zero before every call. With few rows it costs most: 256 x 512 fp32 5.9 us for both.
__global__ void __launch_bounds__(1024) ln_cols_sum_kernel(const Bwd a) {
  __shared__ float sg[32][33], sb[32][33];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  float g = 0.f, b = 0.f;
  if (c < a.m) {
#pragma unroll 5
    for (int p = ty; p < a.parts; p += 32) {
      g += a.part[(int64_t)p * a.m + c];
      b += a.part[((int64_t)a.parts + p) * a.m + c];
    }
  }
  sg[ty][tx] = g;
  sb[ty][tx] = b;
  __syncthreads();
  // warp w adds column w's 32 sums
  g = sg[tx][ty];
  b = sb[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    g += __shfl_xor_sync(0xffffffffu, g, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int64_t col = (int64_t)blockIdx.x * 32 + ty;
  if (tx == 0 && col < a.m) {
    if (a.dgamma) a.dgamma[col] = g;
    if (a.dbeta) a.dbeta[col] = b;
  }
}

// ------------------------------------------------------------------ rows held in registers
// V consecutive elements as they lie in memory: 16 bytes, or one element where rows do not start
// on 16 bytes. Kept packed between the passes over a row: half of the registers for bf16.
template <typename T, int V>
struct Vec {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        f[k] = __uint_as_float(u[k]);
      } else {
        f[2 * k] = __uint_as_float(u[k] << 16);
        f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    }
  }
};
template <typename T>
struct Vec<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void clear() { st(&w, 0, 0.f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = ld(&w, 0); }
};
template <typename T, int V>
__device__ __forceinline__ void stv(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    st(p, 0, f[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
// V weights of type WT at p (NULL: `none`)
template <typename WT, int V>
__device__ __forceinline__ void ldw(const WT* p, int i, float none, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = p ? ld(p, i) : none;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = none;
    if (p) {
      if constexpr (sizeof(WT) == 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
          const float4 a = *reinterpret_cast<const float4*>(p + i + k);
          f[k] = a.x; f[k + 1] = a.y; f[k + 2] = a.z; f[k + 3] = a.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
          const uint2 u = *reinterpret_cast<const uint2*>(p + i + k);
          f[k] = __uint_as_float(u.x << 16); f[k + 1] = __uint_as_float(u.x & 0xffff0000u);
          f[k + 2] = __uint_as_float(u.y << 16); f[k + 3] = __uint_as_float(u.y & 0xffff0000u);
        }
      }
    }
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Sums of a few pairs as a tree: the chains of additions, and with them the rounding, stay short.
template <int P>
__device__ __forceinline__ float2 tree(const float2 (&f)[P]) {
  if constexpr (P == 2) return __fadd2_rn(f[0], f[1]);
  else return __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
}
template <int P>
__device__ __forceinline__ float2 tree_of_squares(const float2 (&f)[P]) {
  const float2 a = __ffma2_rn(f[1], f[1], __fmul2_rn(f[0], f[0]));
  if constexpr (P == 2) return a;
  else return __fadd2_rn(a, __ffma2_rn(f[3], f[3], __fmul2_rn(f[2], f[2])));
}

// Forward: W warps hold R rows, E elements of each per lane, packed as they came; blockDim.y such
// sets per block. A row is read once and stays in registers over its two sums. What bounds it is
// instructions as much as bytes, so what a row costs apart from its elements is kept small: W is
// compiled in (constant offsets; with a run-time width 16384 x 4096 bf16 took 60 us instead
// of 53), elements are worked on in pairs (fp32 x 2 instructions), and the R rows of a lane share
// its weights: fp32 gamma and beta of one bf16 row are four times the row's own traffic to L1, which
// bounded one row per warp (55 us, L1 78 % busy).
template <typename T, typename WT, int V, int E, int W, int R>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128, W > 4 ? 1 : 4) ln_fwd_kernel(const Fwd a) {
  constexpr int NV = E / V, Y = W > 4 ? 1 : 4 / W, STEP = 32 * W * V, P = V / 2;
  __shared__ float2 buf[2][Y][R][W];
  pdl_wait();
  pdl_trigger();
  const int64_t r0 = ((int64_t)blockIdx.x * Y + threadIdx.y) * R;
  const int rows = (int)max((int64_t)0, min((int64_t)R, a.T - r0));   // of this set
  const int c0 = threadIdx.x * V;         // vector i of a lane: column c0 + STEP i
  const int m = (int)a.m;
  const T* x = static_cast<const T*>(a.x) + r0 * a.m + c0;
  Vec<T, V> v[R][NV];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (j < rows && c0 + STEP * i < m) v[j][i].load(x + j * (int64_t)m + STEP * i);
  const float inv_m = 1.f / (float)m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto pairs = [](const Vec<T, V>& u, float2 (&f)[P]) {
    float e[V];
    u.get(e);
#pragma unroll
    for (int k = 0; k < P; ++k) f[k] = make_float2(e[2 * k], e[2 * k + 1]);
  };
  // sums of p over the W warps, per row
  auto reduce = [&](float2 (&p)[R], float2 (*b)[W]) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        p[j].x += __shfl_xor_sync(0xffffffffu, p[j].x, o);
        p[j].y += __shfl_xor_sync(0xffffffffu, p[j].y, o);
      }
    if constexpr (W > 1) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < R; ++j) b[j][warp] = p[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j) {
        p[j] = both(0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) p[j] = __fadd2_rn(p[j], b[j][w]);
      }
    }
  };
  float mean[R];
  float2 p[R], f[P];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (j < rows && c0 + STEP * i < m) {
        pairs(v[j][i], f);
        s = __fadd2_rn(s, tree(f));
      }
    }
    p[j] = make_float2(s.x + s.y, 0.f);
  }
  reduce(p, buf[0][threadIdx.y]);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mean[j] = p[j].x * inv_m;
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (j < rows && c0 + STEP * i < m) {
        pairs(v[j][i], f);
#pragma unroll
        for (int k = 0; k < P; ++k) f[k] = __fadd2_rn(f[k], both(-mean[j]));
        s1 = __fadd2_rn(s1, tree(f));
        s2 = __fadd2_rn(s2, tree_of_squares(f));
      }
    }
    p[j] = make_float2(s1.x + s1.y, s2.x + s2.y);
  }
  reduce(p, buf[1][threadIdx.y]);
#pragma unroll
  for (int j = 0; j < R; ++j) {   // p: dm and rstd
    p[j].x *= inv_m;
    p[j].y = rstd_of(p[j].y * inv_m, p[j].x, a.eps);
    if (threadIdx.x == 0 && j < rows) {
      if (a.mean) a.mean[r0 + j] = mean[j] + p[j].x;
      if (a.rstd) a.rstd[r0 + j] = p[j].y;
    }
  }
  T* y = static_cast<T*>(a.y) + r0 * a.m + c0;
  const WT* gamma = static_cast<const WT*>(a.gamma);
  const WT* beta = static_cast<const WT*>(a.beta);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + STEP * i;
    if (c < m) {
      float g[V], b[V];
      ldw<WT, V>(gamma, c, 1.f, g);
      ldw<WT, V>(beta, c, 0.f, b);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (j < rows) {
          // ((x - mean) - dm) rstd gamma + beta
          float e[V];
          pairs(v[j][i], f);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const float2 g2 = make_float2(g[2 * k], g[2 * k + 1]);
            const float2 b2 = make_float2(b[2 * k], b[2 * k + 1]);
            const float2 d = __fadd2_rn(__fadd2_rn(f[k], both(-mean[j])), both(-p[j].x));
            const float2 o = __ffma2_rn(__fmul2_rn(d, both(p[j].y)), g2, b2);
            e[2 * k] = o.x;
            e[2 * k + 1] = o.y;
          }
          stv<T, V>(y + j * (int64_t)m + STEP * i, e);
        }
      }
    }
  }
}

// The same for rows that do not start on 16 bytes: single elements, held as fp32 pairs (columns
// c and c + 32 W of a lane), one row at a time.
template <typename T, typename WT, int E, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) ln_fwd_odd_kernel(const Fwd a) {
  constexpr int P = E / 2, Y = W > 4 ? 1 : 4 / W, STEP = 32 * W;
  __shared__ float2 buf[2][Y][W];
  pdl_wait();
  pdl_trigger();
  const int64_t r = (int64_t)blockIdx.x * Y + threadIdx.y;
  const int m = r < a.T ? (int)a.m : 0;   // a row past the last one has no elements
  const int c0 = threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(a.x) + r * a.m + c0;
  float2 f[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + 2 * STEP * i;
    f[i].x = c < m ? ld(x, 2 * STEP * i) : 0.f;
    f[i].y = c + STEP < m ? ld(x, 2 * STEP * i + STEP) : 0.f;
  }
  auto reduce = [&](float2 v, float2* b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (W > 1) {
      if (lane == 0) b[warp] = v;
      __syncthreads();
      v = both(0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) v = __fadd2_rn(v, b[w]);
    }
    return v;
  };
  const float inv_m = 1.f / (float)a.m;
  float2 s = both(0.f);
#pragma unroll
  for (int i = 0; i < P; i += 4) {
    const float2 q[4] = {f[i], f[i + 1], f[i + 2], f[i + 3]};
    s = __fadd2_rn(s, tree(q));
  }
  const float mean = reduce(make_float2(s.x + s.y, 0.f), buf[0][threadIdx.y]).x * inv_m;
  float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
  for (int i = 0; i < P; i += 4) {
    float2 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 2 * STEP * (i + k);
      q[k] = __fadd2_rn(f[i + k], both(-mean));
      if (c >= m) q[k].x = 0.f;
      if (c + STEP >= m) q[k].y = 0.f;
      f[i + k] = q[k];
    }
    s1 = __fadd2_rn(s1, tree(q));
    s2 = __fadd2_rn(s2, tree_of_squares(q));
  }
  const float2 d = reduce(make_float2(s1.x + s1.y, s2.x + s2.y), buf[1][threadIdx.y]);
  float dm = d.x * inv_m;
  const float rstd = rstd_of(d.y * inv_m, dm, a.eps);
  T* y = static_cast<T*>(a.y) + r * a.m + c0;
  const WT* gamma = static_cast<const WT*>(a.gamma);
  const WT* beta = static_cast<const WT*>(a.beta);
  if (gamma) gamma += c0;
  if (beta) beta += c0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 2 * STEP * i + STEP * k;
      if (c0 + c < m) {
        const float g = gamma ? ld(gamma, c) : 1.f, b = beta ? ld(beta, c) : 0.f;
        st(y, c, ((k ? f[i].y : f[i].x) - dm) * rstd * g + b);
      }
    }
  }
  if (threadIdx.x == 0 && m) {
    if (a.mean) a.mean[r] = mean + dm;
    if (a.rstd) a.rstd[r] = rstd;
  }
}

constexpr int64_t kRegWidth = 16384;

template <typename T, typename WT, int V, int E, int W, int R>
cudaError_t launch_fwd(const Fwd& a, cudaStream_t s) {
  constexpr int Y = W > 4 ? 1 : 4 / W;
  return launch_k(ln_fwd_kernel<T, WT, V, E, W, R>,
                  dim3((unsigned)((a.T + Y * R - 1) / (Y * R))), dim3(32 * W, Y), 0, s, a);
}
// E x R values per lane. With rows enough to fill the GPU that way, as many as 64 registers hold
// (128 of bf16, 64 of fp32): rows of 32 elements up to 4096 columns and longer pieces of fewer rows
// beyond, so that a block stays at 128 threads (fp32: 256); the barriers of 512 threads cost more
// than shared weights save (2048 x 16384 bf16: 45 us against 35 us). With few rows, one row and
// 32 elements, or 8 where a warp then holds the row.
template <typename T, typename WT, int V>
cudaError_t fwd_width(const Fwd& a, cudaStream_t s) {
  constexpr int kHold = 256 / (int)sizeof(T), kRows = kHold / 32;
  const bool many = a.T * a.m >= (int64_t)kHold * 32 * 16 * 148;   // 16 warps on every SM
  if (a.m <= 256)
    return many ? launch_fwd<T, WT, V, 8, 1, kRows>(a, s) : launch_fwd<T, WT, V, 8, 1, 1>(a, s);
  if (many) {
    if (a.m <= 1024) return launch_fwd<T, WT, V, 32, 1, kRows>(a, s);
    if (a.m <= 2048) return launch_fwd<T, WT, V, 32, 2, kRows>(a, s);
    if (a.m <= 4096) return launch_fwd<T, WT, V, 32, 4, kRows>(a, s);
    if constexpr (kHold == 128) {
      if (a.m <= 8192) return launch_fwd<T, WT, V, 64, 4, 2>(a, s);
      return launch_fwd<T, WT, V, 128, 4, 1>(a, s);
    } else {
      if (a.m <= 8192) return launch_fwd<T, WT, V, 64, 4, 1>(a, s);
      return launch_fwd<T, WT, V, 64, 8, 1>(a, s);
    }
  }
  if (a.m <= 1024) return launch_fwd<T, WT, V, 32, 1, 1>(a, s);
  if (a.m <= 2048) return launch_fwd<T, WT, V, 32, 2, 1>(a, s);
  if (a.m <= 4096) return launch_fwd<T, WT, V, 32, 4, 1>(a, s);
  if (a.m <= 8192) return launch_fwd<T, WT, V, 32, 8, 1>(a, s);
  return launch_fwd<T, WT, V, 32, 16, 1>(a, s);
}
template <typename T, typename WT, int E, int W>
cudaError_t launch_odd(const Fwd& a, cudaStream_t s) {
  constexpr int Y = W > 4 ? 1 : 4 / W;
  return launch_k(ln_fwd_odd_kernel<T, WT, E, W>, dim3((unsigned)((a.T + Y - 1) / Y)),
                  dim3(32 * W, Y), 0, s, a);
}
// Few elements a lane and many warps a row: single-element loads wait one by one otherwise (32 a lane
// and a warp per row: 16384 x 1023 fp32 39 us against 25 us of 8 a lane, 1777 x 1023 9.8 against 5.4).
// Beyond 2048 columns 16 a lane (8192 x 4095 bf16 54 us against 61 us of 8 and 512 threads). The loads
// count, not the bytes: bf16 rows take as long as fp32 ones (16384 x 1023 25 us, bytes 10.4; 8192 x 4095 53,
// bytes 20.8; 4096 x 8191 72, bytes 20.8).
template <typename T, typename WT>
cudaError_t fwd_odd(const Fwd& a, cudaStream_t s) {
  if (a.m <= 256) return launch_odd<T, WT, 8, 1>(a, s);
  if (a.m <= 512) return launch_odd<T, WT, 8, 2>(a, s);
  if (a.m <= 1024) return launch_odd<T, WT, 8, 4>(a, s);
  if (a.m <= 2048) return launch_odd<T, WT, 8, 8>(a, s);
  if (a.m <= 4096) return launch_odd<T, WT, 16, 8>(a, s);
  if (a.m <= 8192) return launch_odd<T, WT, 16, 16>(a, s);
  return launch_odd<T, WT, 32, 16>(a, s);
}

// ------------------------------------------------------------------ rows through a ring
// A persistent block takes groups of consecutive rows. They come through a ring of shared-memory
// slots by bulk copies, groups ahead, so that bytes are in flight whatever the block waits for.
// Elements are worked on in pairs (fp32 x 2 instructions): at bf16's two bytes an element,
// instructions count as much as bytes.
// Rows that do not start on 16 bytes (V = 1) are copied as the 16-byte window around them.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

constexpr int kRingBytes = 224 * 1024;   // of the 227 KB of a block
constexpr int kMaxStages = 6;

struct RingShape {
  int stages, slot;                      // slot: bytes of one group of one array
};

// The ring of a block that reads ARR arrays [T][m] of one layout. All threads of the block make the
// same calls; thread 0 issues the copies. Waits are bounded: on expiry the device error word is
// set, wait() returns false and the block leaves through drain().
template <typename T, int V, int ARR>
struct Ring {
  const char* src[ARR];
  uint8_t* smem;
  uint64_t* full;
  umma::Ctl ctl;
  RingShape sh;
  int64_t group_bytes, total, groups, next;
  int rows, s, used;
  uint32_t ph;

  __device__ __forceinline__ int tid() const { return threadIdx.y * blockDim.x + threadIdx.x; }
  // bytes of group g: [lo, hi) of the arrays, copied as [from, end)
  __device__ __forceinline__ void window(int64_t g, int64_t& lo, int64_t& hi, int64_t& from,
                                         int64_t& end) const {
    lo = from = g * group_bytes;
    hi = end = min(total, lo + group_bytes);
    if constexpr (V == 1) {
      from = lo & ~(int64_t)15;
      end = min((hi + 15) & ~(int64_t)15, total & ~(int64_t)15);
      if (end < from) end = from;
    }
  }
  __device__ __forceinline__ void fetch(int64_t g, int slot) const {
    int64_t lo, hi, from, end;
    window(g, lo, hi, from, end);
    const uint32_t bytes = (uint32_t)(end - from), bar = umma::smem_u32(full + slot);
    umma::mbar_expect_tx(bar, ARR * bytes);
    if (bytes) {
#pragma unroll
      for (int k = 0; k < ARR; ++k)
        bulk_load(umma::smem_u32(smem + (size_t)(slot * ARR + k) * sh.slot), src[k] + from, bytes,
                  bar);
    }
  }
  __device__ __forceinline__ void init(uint8_t* buf, uint64_t* bars, int* abort_flag, int* err,
                                       RingShape shape, int64_t T_, int64_t m, int rows_) {
    smem = buf; full = bars; sh = shape; rows = rows_;
    ctl = umma::Ctl{abort_flag, err};
    group_bytes = rows * m * sizeof(T);
    total = T_ * m * sizeof(T);
    groups = (T_ + rows - 1) / rows;
    s = used = 0;
    ph = 0;
    if (tid() == 0) {
      *abort_flag = 0;
      for (int k = 0; k < sh.stages; ++k) umma::mbar_init(umma::smem_u32(full + k), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
  }
  __device__ __forceinline__ void start() {
    next = blockIdx.x;
    for (int k = 0; k < sh.stages; ++k, next += gridDim.x)
      if (tid() == 0 && next < groups) fetch(next, k);
  }
  // the current slot is filled (false: the wait ran out)
  __device__ __forceinline__ bool wait(int64_t g) {
    const bool ok = umma::wait_bounded(umma::smem_u32(full + s), ph, ctl, umma::kErrProducer,
                                       umma::kWaitLimitNs);
    if constexpr (V == 1) {
      // the arrays' last bytes, which no 16-byte copy inside them covers
      int64_t lo, hi, from, end;
      window(g, lo, hi, from, end);
      if (end < hi) {
        for (int64_t b = end + (int64_t)tid() * sizeof(T); b < hi;
             b += (int64_t)blockDim.x * blockDim.y * sizeof(T))
#pragma unroll
          for (int k = 0; k < ARR; ++k)
            *reinterpret_cast<T*>(smem + (size_t)(s * ARR + k) * sh.slot + (lo & 15) + (b - lo)) =
                *reinterpret_cast<const T*>(src[k] + b);
        __syncthreads();
      }
    }
    return ok;
  }
  // first row of the current slot's group
  __device__ __forceinline__ const T* row(int64_t g, int k) const {
    const T* p = reinterpret_cast<const T*>(smem + (size_t)(s * ARR + k) * sh.slot);
    if constexpr (V == 1) p += (g * group_bytes & 15) / sizeof(T);
    return p;
  }
  // After the barrier of the current group, on to the next slot. Its own slot has been read by every
  // thread and takes the next group to come.
  __device__ __forceinline__ void release() {
    refill(s);
    advance();
  }
  // The same where the slot is read once more behind the barrier: what takes the next group is the
  // slot of the group before.
  __device__ __forceinline__ void release_before() {
    if (used++ > 0) refill(s == 0 ? sh.stages - 1 : s - 1);
    advance();
  }
  __device__ __forceinline__ void refill(int slot) {
    if (tid() == 0 && next < groups) fetch(next, slot);
    next += gridDim.x;
  }
  __device__ __forceinline__ void advance() {
    if (++s == sh.stages) { s = 0; ph ^= 1u; }
  }
  // let the copies in flight land before the block leaves
  __device__ __forceinline__ void drain() {
    if (tid() == 0)
      for (int k = 0; k < sh.stages; ++k) {
        umma::wait_bounded(umma::smem_u32(full + s), ph, ctl, 0, umma::kDrainLimitNs,
                           /*stop_on_abort=*/false);
        if (++s == sh.stages) { s = 0; ph ^= 1u; }
      }
  }
};

// Column sums of a block: E per thread (vector i from column c0 + i step on), added over the sets of
// threads in order and written once.
template <int V, int E>
__device__ __forceinline__ void write_part(const Bwd& a, float* sh, int m, int step, int tid,
                                           const float* eg, const float* eb) {
  float* out_g = a.part + (int64_t)blockIdx.x * m;
  float* out_b = a.part + ((int64_t)gridDim.x + blockIdx.x) * m;
  const int c0 = threadIdx.x * V;
  __syncthreads();   // (the ring's memory: no copy is in flight any more)
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int c = c0 + i * step;
    if (c < m) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        sh[(threadIdx.y * 2) * m + c + k] = eg[i * V + k];
        sh[(threadIdx.y * 2 + 1) * m + c + k] = eb[i * V + k];
      }
    }
  }
  __syncthreads();
  for (int c = tid; c < m; c += blockDim.x * blockDim.y) {
    float g = 0.f, b = 0.f;
    for (int y = 0; y < (int)blockDim.y; ++y) {
      g += sh[(y * 2) * m + c];
      b += sh[(y * 2 + 1) * m + c];
    }
    out_g[c] = g;
    out_b[c] = b;
  }
}

// Backward, rows of up to 8192 columns. A thread has the same E columns in every row (vector i
// starts at column (i blockDim.x + threadIdx.x) V), so its shares of dgamma and dbeta and its
// gammas stay in registers; the block's column sums are written once. A group is R rows for each of
// blockDim.y sets of threads; per group there is one barrier, which completes the row sums and frees
// a slot. What is needed again behind the barrier stays in registers: as xh and g (16 a row of
// E = 8) where a thread may have 128 registers, else as loaded (PACKED).
// Besides the bytes what counts is instructions and each group's chain (sums, barrier, sums of the
// warps, dx). So the R rows' 2 R sums are reduced together: each step of the butterfly halves the
// values that a lane goes on with, until 32 / (2 R) lanes share one, in both levels. And dead columns
// cost no selects: their threads read the row's first column and have a gamma of zero. 16384 x 4096
// bf16 takes 76 us so (5.3 TB/s), 89 us with a reduction per row and a select per value. Not kept:
// two blocks per SM of 256 threads and E = 16 (95 us); two halves of a block one group apart (97 us).
template <typename T, typename WT, int V, int E, int R, int MAXT, bool PACKED>
__global__ void __launch_bounds__(MAXT, 1) ln_bwd_kernel(const Bwd a, const RingShape shape) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages];
  constexpr int N = 2 * R, G = 32 / N;            // row sums of a set; lanes that share one
  __shared__ float buf[2][MAXT / 32 * N];         // [set][sum][warp]
  __shared__ int abort_flag;
  constexpr int NV = E / V, P = E / 2;
  const int m = (int)a.m, warps = blockDim.x >> 5, step = blockDim.x * V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ring<T, V, 2> ring;
  ring.src[0] = static_cast<const char*>(a.x);
  ring.src[1] = static_cast<const char*>(a.dy);
  ring.init(smem, full, &abort_flag, a.err, shape, a.T, a.m, blockDim.y * R);
  pdl_wait();
  pdl_trigger();
  ring.start();
  const int c0 = threadIdx.x * V;
  int off[NV];                                    // columns as read
  float2 gm[P], ag[P], ab[P];
  {
    const WT* gamma = static_cast<const WT*>(a.gamma);
    float* e = reinterpret_cast<float*>(gm);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = c0 + i * step < m;
      off[i] = in ? c0 + i * step : 0;
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = 0.f;
      if (in) ldw<WT, V>(gamma, off[i], 1.f, v);
#pragma unroll
      for (int k = 0; k < V; ++k) e[i * V + k] = v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < P; ++k) ag[k] = ab[k] = both(0.f);
  float mean_n[R], rstd_n[R];                // of the next group's rows
  auto stats = [&](int64_t r, int64_t left) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean_n[j] = j < left ? a.mean[r + j] : 0.f;
      rstd_n[j] = j < left ? a.rstd[r + j] : 0.f;
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * ring.rows + threadIdx.y * R;
  const int64_t hop = (int64_t)gridDim.x * ring.rows;
  stats(r0, a.T - r0);
  // a row's vectors as fp32 pairs
  auto unpack = [](const Vec<T, V> (&u)[NV], float2 (&f)[P]) {
    float* e = reinterpret_cast<float*>(f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[V];
      u[i].get(v);
#pragma unroll
      for (int k = 0; k < V; ++k) e[i * V + k] = v[k];
    }
  };
  const float inv_m = 1.f / (float)m;
  bool bad = false;
  int turn = 0;
  for (int64_t g = blockIdx.x; g < ring.groups; g += gridDim.x, r0 += hop) {
    const int rows = a.T - r0 >= R ? R : max(0, (int)(a.T - r0));   // (r0 < T + the group's rows)
    float2 mean[R], rstd[R];                 // -mean, rstd
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean[j] = both(-mean_n[j]);
      rstd[j] = both(rstd_n[j]);
    }
    const bool ok = ring.wait(g);
    Vec<T, V> x[R][NV], d[R][NV];
    if (rows == R) {
      const T* px = ring.row(g, 0) + threadIdx.y * R * m;
      const T* pd = ring.row(g, 1) + threadIdx.y * R * m;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          x[j][i].load(px + j * m + off[i]);
          d[j][i].load(pd + j * m + off[i]);
        }
    } else {   // rows past the last one: some row's x and a dy of zero add nothing
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int r = j < rows ? threadIdx.y * R + j : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          x[j][i].load(ring.row(g, 0) + r * m + off[i]);
          if (j < rows) d[j][i].load(ring.row(g, 1) + r * m + off[i]);
          else d[j][i].clear();
        }
      }
    }
    float2 xh[R][P], gd[R][P];
    float s[N];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float2 s1 = both(0.f), s2 = both(0.f);
      unpack(x[j], xh[j]);
      unpack(d[j], gd[j]);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float2& h = xh[j][k];
        float2& q = gd[j][k];
        h = __fmul2_rn(__fadd2_rn(h, mean[j]), rstd[j]);
        ag[k] = __ffma2_rn(q, h, ag[k]);
        ab[k] = __fadd2_rn(ab[k], q);
        q = __fmul2_rn(q, gm[k]);
        s1 = __fadd2_rn(s1, q);
        s2 = __ffma2_rn(q, h, s2);
      }
      s[2 * j] = s1.x + s1.y;
      s[2 * j + 1] = s2.x + s2.y;
    }
    // lane l ends with the warp's sum l / G
    int o = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float give = up ? s[k] : s[k + n];
        s[k] = (up ? s[k + n] : s[k]) + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
#pragma unroll
    for (int q = G / 2; q > 0; q >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], q);
    float* mine = buf[turn] + (threadIdx.y * N + lane / G) * warps;   // (the other may still be read)
    turn ^= 1;
    if (lane % G == 0) mine[warp] = s[0];
    stats(r0 + hop, a.T - r0 - hop);
    bad = __syncthreads_or(!ok);
    if (bad) break;
    ring.release();
    if (a.dx) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < MAXT / 32; w += G)
        if (w + lane % G < warps) t += mine[w + lane % G];
#pragma unroll
      for (int q = G / 2; q > 0; q >>= 1) t += __shfl_xor_sync(0xffffffffu, t, q);
      t *= -inv_m;
      T* dx = static_cast<T*>(a.dx) + r0 * a.m;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float2 c1 = both(__shfl_sync(0xffffffffu, t, 2 * j * G));
        const float2 c2 = both(__shfl_sync(0xffffffffu, t, (2 * j + 1) * G));
        if constexpr (PACKED) {
          unpack(x[j], xh[j]);
          unpack(d[j], gd[j]);
        }
        // rstd (g - c1 - xh c2)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float2& h = xh[j][k];
          float2& q = gd[j][k];
          if constexpr (PACKED) {
            h = __fmul2_rn(__fadd2_rn(h, mean[j]), rstd[j]);
            q = __ffma2_rn(q, gm[k], c1);
          } else {
            q = __fadd2_rn(q, c1);
          }
          q = __fmul2_rn(__ffma2_rn(h, c2, q), rstd[j]);
        }
        const float* e = reinterpret_cast<const float*>(gd[j]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v[V];
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] = e[i * V + k];
          if (j < rows && c0 + i * step < m) stv<T, V>(dx + j * m + off[i], v);
        }
      }
    }
  }
  if (bad) {
    ring.drain();
    return;
  }
  if (a.part)
    write_part<V, E>(a, reinterpret_cast<float*>(smem), m, step, ring.tid(),
                     reinterpret_cast<const float*>(ag), reinterpret_cast<const float*>(ab));
}

// The same for rows of 8193 columns and more: one row a group, E = 32 columns per thread; the row is
// read from its slot a second time, which is freed one group later, and gamma comes from L1.
template <typename T, typename WT, int V>
__global__ void __launch_bounds__(512, 1) ln_bwd_wide_kernel(const Bwd a, const RingShape shape) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float buf[2][2][16];                 // [sum][warp]
  __shared__ int abort_flag;
  constexpr int E = 32, NV = E / V;
  const int m = (int)a.m, warps = blockDim.x >> 5, step = blockDim.x * V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ring<T, V, 2> ring;
  ring.src[0] = static_cast<const char*>(a.x);
  ring.src[1] = static_cast<const char*>(a.dy);
  ring.init(smem, full, &abort_flag, a.err, shape, a.T, a.m, 1);
  pdl_wait();
  pdl_trigger();
  ring.start();
  const WT* gamma = static_cast<const WT*>(a.gamma);
  const int c0 = threadIdx.x * V;
  float ag[E], ab[E];
#pragma unroll
  for (int k = 0; k < E; ++k) ag[k] = ab[k] = 0.f;
  const float inv_m = 1.f / (float)m;
  float mean_n = a.mean[blockIdx.x], rstd_n = a.rstd[blockIdx.x];
  bool bad = false;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
    const float mean = mean_n, rstd = rstd_n;
    const bool ok = ring.wait(r);
    const T* px = ring.row(r, 0) + c0;
    const T* pd = ring.row(r, 1) + c0;
    float(*sums)[16] = buf[turn];                 // (the other one may still be read)
    turn ^= 1;
    // vector i: xh and g, and dy
    auto get = [&](int i, float (&h)[V], float (&gk)[V], float (&d)[V]) {
      Vec<T, V> vx, vd;
      vx.load(px + i * step);
      vd.load(pd + i * step);
      vx.get(h);
      vd.get(d);
      ldw<WT, V>(gamma, c0 + i * step, 1.f, gk);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h[k] = (h[k] - mean) * rstd;
        gk[k] *= d[k];
      }
    };
    float s1[2] = {0.f, 0.f}, s2[2] = {0.f, 0.f};   // (two chains of sums each)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (c0 + i * step < m) {
        float h[V], gk[V], d[V];
        get(i, h, gk, d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int q = i * V + k;
          ag[q] += d[k] * h[k];
          ab[q] += d[k];
          s1[q & 1] += gk[k];
          s2[q & 1] += gk[k] * h[k];
        }
      }
    }
    // both sums at once: the lower half-warp goes on with s1, the upper one with s2
    const float t1 = s1[0] + s1[1], t2 = s2[0] + s2[1];
    float t = (lane & 16) ? t2 : t1;
    t += __shfl_xor_sync(0xffffffffu, (lane & 16) ? t1 : t2, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((lane & 15) == 0) sums[lane >> 4][warp] = t;
    if (r + gridDim.x < a.T) {
      mean_n = a.mean[r + gridDim.x];
      rstd_n = a.rstd[r + gridDim.x];
    }
    bad = __syncthreads_or(!ok);
    if (bad) break;
    ring.release_before();
    if (a.dx) {
      t = (lane & 15) < warps ? sums[lane >> 4][lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      const float c1 = __shfl_sync(0xffffffffu, t, 0) * inv_m;
      const float c2 = __shfl_sync(0xffffffffu, t, 16) * inv_m;
      T* dx = static_cast<T*>(a.dx) + r * a.m + c0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c0 + i * step < m) {
          float h[V], gk[V], d[V];
          get(i, h, gk, d);
#pragma unroll
          for (int k = 0; k < V; ++k) d[k] = rstd * (gk[k] - c1 - h[k] * c2);
          stv<T, V>(dx + i * step, d);
        }
      }
    }
  }
  if (bad) {
    ring.drain();
    return;
  }
  if (a.part)
    write_part<V, E>(a, reinterpret_cast<float*>(smem), m, step, ring.tid(), ag, ab);
}

constexpr int kMaxParts = 148;   // one block per SM

// Shape of the one-pass backward for a width; stages < 2: a row is too wide for the ring. E = 8 up to
// 5120 columns: 640 threads are five warps a scheduler of 96 registers each (8192 x 5120 bf16 58 us, with
// E = 16 71 us); the next warp is the sixth on one, which leaves 80 registers, and they spill (8192 x
// 5376 bf16 102 us, with E = 16 72 us). 16 up to 8192 (8192 x 6144, 7168, 8192 bf16 74, 82, 85 us; 1024
// threads of 8 columns and 64 registers spill: 145 us), 32 beyond. `sets` sets of threads and R rows
// each make a group: at most 96 KB of x and dy, no more than leaves a group for every SM. R = 2 with
// E = 8 (8192 x 5120 bf16 58.5 us against 67 us of one row; four rows spill: 16384 x 4096 bf16
// 92 us against 76 us), one row with E = 16 (8192 x 8192 bf16 two rows: 107 us).
struct GroupShape {
  int threads, sets, E, R;
  RingShape ring;
  size_t smem;
};
GroupShape group_shape(int64_t T, int64_t m, int esz) {
  GroupShape sh;
  sh.E = m <= 5120 ? 8 : m <= 8192 ? 16 : 32;
  sh.threads = 32 * (int)((m + 32 * sh.E - 1) / (32 * sh.E));
  const int most = sh.E == 8 ? 2 : 1;
  const int64_t fit = 96 * 1024 / (2 * m * esz);                  // rows in 96 KB
  const int64_t share = (T + kMaxParts - 1) / kMaxParts;          // rows per SM
  const int64_t rows = std::max<int64_t>(1, std::min(fit, share));
  sh.R = most;
  while (sh.R > rows) sh.R /= 2;
  const int block = std::max(sh.threads, 512);
  sh.sets = (int)std::max<int64_t>(1, std::min<int64_t>(block / sh.threads, rows / sh.R));
  // the window around unaligned rows needs up to 30 bytes more
  sh.ring.slot = (int)(((int64_t)sh.sets * sh.R * m * esz + 31) / 16 * 16);
  const int64_t stage = 2 * (int64_t)sh.ring.slot;
  sh.ring.stages = (int)std::min<int64_t>(kMaxStages, kRingBytes / stage);
  // at the end the ring's memory holds the block's column sums
  sh.smem = std::max((size_t)(sh.ring.stages * stage), (size_t)sh.sets * 2 * m * sizeof(float));
  return sh;
}

template <typename K>
cudaError_t launch_ring(K kern, const Bwd& a, const GroupShape& sh, cudaStream_t s) {
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sh.smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3((unsigned)a.parts), dim3((unsigned)sh.threads, (unsigned)sh.sets),
                  sh.smem, s, a, sh.ring);
}
template <typename T, typename WT, int V>
cudaError_t launch_bwd(const Bwd& a, const GroupShape& sh, cudaStream_t s) {
  if (sh.E == 32) return launch_ring(ln_bwd_wide_kernel<T, WT, V>, a, sh, s);
  if (sh.E == 16) return launch_ring(ln_bwd_kernel<T, WT, V, 16, 1, 512, true>, a, sh, s);
  if (sh.threads > 512)
    return sh.R == 2 ? launch_ring(ln_bwd_kernel<T, WT, V, 8, 2, 640, true>, a, sh, s)
                     : launch_ring(ln_bwd_kernel<T, WT, V, 8, 1, 640, true>, a, sh, s);
  return sh.R == 2 ? launch_ring(ln_bwd_kernel<T, WT, V, 8, 2, 512, false>, a, sh, s)
                   : launch_ring(ln_bwd_kernel<T, WT, V, 8, 1, 512, false>, a, sh, s);
}

int row_blocks(int64_t T) { return (int)std::min<int64_t>(T, 148 * 8); }

}  // namespace

// the most ranges of rows that the column sums are split into, whichever kernel runs
size_t bwd_ws_bytes(int64_t T, int64_t m) {
  if (T <= 0 || m <= 0) return 0;
  return (size_t)2 * (size_t)std::min<int64_t>(T, kMaxParts) * (size_t)m * sizeof(float);
}

cudaError_t fwd(const Fwd& a, DT t, cudaStream_t s) {
  TraceScope tr("ln_fwd", s);
  using bf16 = __nv_bfloat16;
  if (a.m <= kRegWidth && a.T < INT32_MAX) {
    const bool vec = a.m * (t == DT::BF16 ? 2 : 4) % 16 == 0;   // every row starts on 16 bytes
    if (t == DT::BF16) {
      if (vec) return a.w_bf16 ? fwd_width<bf16, bf16, 8>(a, s) : fwd_width<bf16, float, 8>(a, s);
      return a.w_bf16 ? fwd_odd<bf16, bf16>(a, s) : fwd_odd<bf16, float>(a, s);
    }
    if (vec) return a.w_bf16 ? fwd_width<float, bf16, 4>(a, s) : fwd_width<float, float, 4>(a, s);
    return a.w_bf16 ? fwd_odd<float, bf16>(a, s) : fwd_odd<float, float>(a, s);
  }
  const dim3 grid((unsigned)row_blocks(a.T)), block(kThreads);
  return t == DT::BF16 ? launch_k(ln_fwd_any_kernel<bf16>, grid, block, 0, s, a)
                       : launch_k(ln_fwd_any_kernel<float>, grid, block, 0, s, a);
}

cudaError_t bwd(Bwd a, DT t, void* ws, cudaStream_t s) {
  const dim3 block(kThreads);
  const bool cols = a.dgamma || a.dbeta;
  const int esz = t == DT::BF16 ? 2 : 4;
  const dim3 sum_grid((unsigned)((a.m + 31) / 32));
  a.part = cols ? static_cast<float*>(ws) : nullptr;
  a.err = device_error_word();
  if (!a.err) return cudaErrorUnknown;
  cudaError_t e = cudaSuccess;
  const bool vec = a.m * esz % 16 == 0;   // every row starts on 16 bytes
  const GroupShape sh = a.m <= kRegWidth ? group_shape(a.T, a.m, esz) : GroupShape{};
  if (a.m <= kRegWidth && sh.ring.stages >= 2) {
    const int64_t groups = (a.T + sh.sets * sh.R - 1) / (sh.sets * sh.R);
    a.parts = (int)std::min<int64_t>(groups, kMaxParts);
    using bf16 = __nv_bfloat16;
    {
      TraceScope tr("ln_bwd", s);
      if (t == DT::BF16 && vec)
        e = a.w_bf16 ? launch_bwd<bf16, bf16, 8>(a, sh, s) : launch_bwd<bf16, float, 8>(a, sh, s);
      else if (t == DT::BF16)
        e = a.w_bf16 ? launch_bwd<bf16, bf16, 1>(a, sh, s) : launch_bwd<bf16, float, 1>(a, sh, s);
      else if (vec)
        e = a.w_bf16 ? launch_bwd<float, bf16, 4>(a, sh, s) : launch_bwd<float, float, 4>(a, sh, s);
      else
        e = a.w_bf16 ? launch_bwd<float, bf16, 1>(a, sh, s) : launch_bwd<float, float, 1>(a, sh, s);
    }
    if (e != cudaSuccess || !cols) return e;
    TraceScope tr("ln_bwd_sum", s);
    return launch_k(ln_cols_sum_kernel, sum_grid, dim3(1024), 0, s, a);
  }
  // rows too wide for that: the column sums first, since dx may overwrite x or dy
  if (cols) {
    a.parts = (int)std::max<int64_t>(1, std::min<int64_t>(128, a.T / 64));
    {
      TraceScope tr("ln_bwd_cols", s);
      const dim3 grid((unsigned)((a.m + 31) / 32), (unsigned)a.parts);
      e = t == DT::BF16 ? launch_k(ln_cols_any_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                        : launch_k(ln_cols_any_kernel<float>, grid, block, 0, s, a);
      if (e != cudaSuccess) return e;
    }
    TraceScope tr("ln_bwd_sum", s);
    e = launch_k(ln_cols_sum_kernel, sum_grid, dim3(1024), 0, s, a);
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
