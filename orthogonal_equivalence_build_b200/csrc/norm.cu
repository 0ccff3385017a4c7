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

// dgamma and dbeta: the ranges' sums, 32 columns per block; eight threads of a column take every
// eighth range, and their sums are added in order.
__global__ void __launch_bounds__(kThreads) ln_cols_sum_kernel(const Bwd a) {
  __shared__ float sg[8][33], sb[8][33];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + tx;
  float g = 0.f, b = 0.f;
  if (c < a.m) {
#pragma unroll 4
    for (int p = ty; p < a.parts; p += 8) {
      g += a.part[(int64_t)p * a.m + c];
      b += a.part[((int64_t)a.parts + p) * a.m + c];
    }
  }
  sg[ty][tx] = g;
  sb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < a.m) {
    for (int k = 1; k < 8; ++k) {
      g += sg[k][tx];
      b += sb[k][tx];
    }
    if (a.dgamma) a.dgamma[c] = g;
    if (a.dbeta) a.dbeta[c] = b;
  }
}

// ------------------------------------------------------------------ rows held in registers
// V consecutive elements as they lie in memory: 16 bytes, or one element where rows do not start
// on 16 bytes. Kept packed between the passes over a row: half of the registers for bf16.
template <typename T, int V>
struct Vec {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
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
// V weights of either type
template <int V>
__device__ __forceinline__ void ldw(const void* w, int w_bf16, int64_t i, float none,
                                    float (&f)[V]) {
  if (!w) {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = none;
  } else if (w_bf16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w) + i;
    if constexpr (V == 8) {
      Vec<__nv_bfloat16, 8> v;
      v.load(p);
      v.get(f);
    } else if constexpr (V == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xffff0000u);
      f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
      f[0] = ld(p, 0);
    }
  } else {
    const float* p = static_cast<const float*>(w) + i;
    if constexpr (V == 1) {
      f[0] = *p;
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const float4 a = *reinterpret_cast<const float4*>(p + k);
        f[k] = a.x; f[k + 1] = a.y; f[k + 2] = a.z; f[k + 3] = a.w;
      }
    }
  }
}

// Sums of a and b over the threads of one row: blockDim.x threads (whole warps), row threadIdx.y of
// the block. `buf` holds a float2 per warp of the block; two calls in a row take different ones, so
// one barrier each is enough.
__device__ __forceinline__ float2 row_sum(float a, float b, float2* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  float2* mine = buf + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int w = 0; w < warps; ++w) {
    s.x += mine[w].x;
    s.y += mine[w].y;
  }
  return s;
}

// Forward: blockDim.x threads hold a row, V x NV elements each; blockDim.y rows per block, one
// block per group of rows. Many small blocks per SM keep enough rows in flight; a row is read
// once and stays in registers over its two sums.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) ln_fwd_kernel(const Fwd a) {
  __shared__ float2 buf[2][16];
  pdl_wait();
  pdl_trigger();
  const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int m = r < a.T ? (int)a.m : 0;   // a row past the last one has no elements
  const T* x = static_cast<const T*>(a.x) + r * a.m;
  Vec<T, V> v[NV];
  float f[V], s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < m) v[i].load(x + c);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * blockDim.x + threadIdx.x) * V < m) {
      v[i].get(f);
#pragma unroll
      for (int k = 0; k < V; ++k) s += f[k];
    }
  }
  const float mean = row_sum(s, 0.f, buf[0]).x / (float)a.m;
  float s1 = 0.f, s2 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * blockDim.x + threadIdx.x) * V < m) {
      v[i].get(f);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = f[k] - mean;
        s1 += d;
        s2 += d * d;
      }
    }
  }
  const float2 d = row_sum(s1, s2, buf[1]);
  const float dm = d.x / (float)a.m;
  const float rstd = rstd_of(d.y / (float)a.m - dm * dm, a.eps);
  T* y = static_cast<T*>(a.y) + r * a.m;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < m) {
      float g[V], b[V];
      ldw<V>(a.gamma, a.w_bf16, c, 1.f, g);
      ldw<V>(a.beta, a.w_bf16, c, 0.f, b);
      v[i].get(f);
#pragma unroll
      for (int k = 0; k < V; ++k) g[k] = (f[k] - mean - dm) * rstd * g[k] + b[k];
      stv<T, V>(y + c, g);
    }
  }
  if (threadIdx.x == 0 && m) {
    if (a.mean) a.mean[r] = mean + dm;
    if (a.rstd) a.rstd[r] = rstd;
  }
}

// Threads per row and rows per block of a width: V x NV elements per thread, whole warps.
struct RowShape {
  int threads, rows;
};
RowShape row_shape(int64_t m, int per_thread, int block) {
  const int warps = (int)((m + 32 * per_thread - 1) / (32 * per_thread));
  return {32 * warps, std::max(1, block / (32 * warps))};
}

constexpr int64_t kRegWidth = 16384;   // 512 threads x 32 elements

template <typename T, int V, int NV>
cudaError_t launch_fwd(const Fwd& a, cudaStream_t s) {
  const RowShape sh = row_shape(a.m, V * NV, 128);
  const int64_t blocks = (a.T + sh.rows - 1) / sh.rows;
  return launch_k(ln_fwd_kernel<T, V, NV>, dim3((unsigned)blocks),
                  dim3((unsigned)sh.threads, (unsigned)sh.rows), 0, s, a);
}
// Elements per thread: few for short rows (a warp holds up to 256 with 8), 32 for long ones.
template <typename T, int V>
cudaError_t fwd_width(const Fwd& a, cudaStream_t s) {
  if (a.m <= 256) return launch_fwd<T, V, 8 / V>(a, s);
  if (a.m <= 1024) return launch_fwd<T, V, 16 / V>(a, s);
  return launch_fwd<T, V, 32 / V>(a, s);
}

// ------------------------------------------------------------------ backward, one pass
// A persistent block takes groups of blockDim.y consecutive rows (blockDim.x threads each). The rows
// of x and dy come through a ring of shared-memory slots by bulk copies, several groups ahead, so
// that bytes are in flight whatever the block waits for; per group there is one barrier, which
// completes the row sums and frees the slot. dx leaves from registers; a thread's columns are the
// same in every row, so its shares of dgamma and dbeta stay in registers to the end, are added over
// the block's rows at a time in shared memory and written once per block.
// Rows that do not start on 16 bytes (V = 1) are copied as the 16-byte window around them.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Bounded waits: on expiry the device error word is set and the block leaves.
__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity, umma::Ctl c) {
  return umma::wait_bounded(bar, parity, c, umma::kErrProducer, umma::kWaitLimitNs);
}
__device__ __forceinline__ void drain_full(uint32_t bar, uint32_t parity, umma::Ctl c) {
  umma::wait_bounded(bar, parity, c, 0, umma::kDrainLimitNs, /*stop_on_abort=*/false);
}

constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 6;
constexpr int kMaxParts = 148;                   // one block per SM

struct Ring {
  int stages, slot;                              // slot: bytes of one group of x (and of dy)
};

template <typename T, int V, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) ln_bwd_kernel(const Bwd a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float2 buf[2][MAXT / 32];
  __shared__ int abort_flag;
  const int m = (int)a.m, rows = blockDim.y;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int64_t groups = (a.T + rows - 1) / rows;
  const umma::Ctl ctl{&abort_flag, a.err};
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < ring.stages; ++s) umma::mbar_init(umma::smem_u32(full + s), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  // bytes of a group: [lo, hi) of the array, copied as [lo & ~15, end)
  const int64_t row_bytes = (int64_t)m * sizeof(T), total = a.T * row_bytes;
  auto window = [&](int64_t g, int64_t& from, int64_t& end, int64_t& hi) {
    const int64_t lo = g * rows * row_bytes;
    hi = min(total, lo + rows * row_bytes);
    from = lo & ~(int64_t)15;
    end = min((hi + 15) & ~(int64_t)15, total & ~(int64_t)15);
    if (end < from) end = from;
  };
  auto fetch = [&](int64_t g, int s) {
    int64_t from, end, hi;
    window(g, from, end, hi);
    const uint32_t bytes = (uint32_t)(end - from), bar = umma::smem_u32(full + s);
    umma::mbar_expect_tx(bar, 2 * bytes);
    if (bytes) {
      const uint32_t dst = umma::smem_u32(smem + (size_t)s * 2 * ring.slot);
      bulk_load(dst, static_cast<const char*>(a.x) + from, bytes, bar);
      bulk_load(dst + ring.slot, static_cast<const char*>(a.dy) + from, bytes, bar);
    }
  };
  if (tid == 0)
    for (int s = 0; s < ring.stages; ++s) {
      const int64_t g = blockIdx.x + (int64_t)s * gridDim.x;
      if (g < groups) fetch(g, s);
    }

  float ag[NV][V], ab[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) ag[i][k] = ab[i][k] = 0.f;
  float mean_n = 0.f, rstd_n = 0.f;              // of the next group's row
  auto stats = [&](int64_t g) {
    const int64_t r = g * rows + threadIdx.y;
    if (r < a.T) {
      mean_n = __ldg(a.mean + r);
      rstd_n = __ldg(a.rstd + r);
    }
  };
  stats(blockIdx.x);

  int s = 0, turn = 0;
  uint32_t ph = 0;
  bool bad = false;
  int64_t issued = blockIdx.x + (int64_t)ring.stages * gridDim.x;   // next group to fetch
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t r = g * rows + threadIdx.y;
    const int live = r < a.T ? m : 0;
    const float mean = mean_n, rstd = rstd_n;
    const bool ok = wait_full(umma::smem_u32(full + s), ph, ctl);
    const int64_t lo = g * rows * row_bytes;
    uint8_t* sx = smem + (size_t)s * 2 * ring.slot + (lo & 15);
    if constexpr (V == 1) {
      // the array's last bytes, which no 16-byte copy inside it covers
      int64_t from, end, hi;
      window(g, from, end, hi);
      if (end < hi) {
        for (int64_t b = end + (int64_t)tid * sizeof(T); b < hi;
             b += (int64_t)blockDim.x * rows * sizeof(T)) {
          *reinterpret_cast<T*>(sx + (b - lo)) =
              *reinterpret_cast<const T*>(static_cast<const char*>(a.x) + b);
          *reinterpret_cast<T*>(sx + ring.slot + (b - lo)) =
              *reinterpret_cast<const T*>(static_cast<const char*>(a.dy) + b);
        }
        __syncthreads();
      }
    }
    const T* px = reinterpret_cast<const T*>(sx) + threadIdx.y * m;
    const T* pd = reinterpret_cast<const T*>(sx + ring.slot) + threadIdx.y * m;
    Vec<T, V> vx[NV], vd[NV];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (c < live) {
        vx[i].load(px + c);
        vd[i].load(pd + c);
        float x[V], d[V], w[V];
        vx[i].get(x);
        vd[i].get(d);
        ldw<V>(a.gamma, a.w_bf16, c, 1.f, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float xh = (x[k] - mean) * rstd, gk = d[k] * w[k];
          ag[i][k] += d[k] * xh;
          ab[i][k] += d[k];
          s1 += gk;
          s2 += gk * xh;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    const int warps = blockDim.x >> 5;
    float2* sums = buf[turn] + threadIdx.y * warps;   // (the other one may still be read)
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_float2(s1, s2);
    if (g + gridDim.x < groups) stats(g + gridDim.x);
    bad = __syncthreads_or(!ok);                 // the slot has been read by every thread
    if (bad) break;
    if (tid == 0 && issued < groups) fetch(issued, s);
    issued += gridDim.x;
    if (warps > 1) {
      s1 = s2 = 0.f;
      for (int w = 0; w < warps; ++w) {
        s1 += sums[w].x;
        s2 += sums[w].y;
      }
    }
    if (a.dx) {
      const float c1 = s1 / (float)m, c2 = s2 / (float)m;
      T* dx = static_cast<T*>(a.dx) + r * m;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < live) {
          float x[V], d[V], w[V];
          vx[i].get(x);
          vd[i].get(d);
          ldw<V>(a.gamma, a.w_bf16, c, 1.f, w);
#pragma unroll
          for (int k = 0; k < V; ++k)
            d[k] = rstd * (d[k] * w[k] - c1 - (x[k] - mean) * rstd * c2);
          stv<T, V>(dx + c, d);
        }
      }
    }
    if (++s == ring.stages) { s = 0; ph ^= 1u; }
  }
  if (bad) {
    // let the copies in flight land before the block leaves (its slots from s on, in ring order)
    if (tid == 0)
      for (int k = 0; k < ring.stages; ++k) {
        drain_full(umma::smem_u32(full + s), ph, ctl);
        if (++s == ring.stages) { s = 0; ph ^= 1u; }
      }
    return;
  }
  if (!a.part) return;
  // the block's column sums, its rows at a time added in order; no copy is in flight any more
  float* out_g = a.part + (int64_t)blockIdx.x * m;
  float* out_b = a.part + ((int64_t)gridDim.x + blockIdx.x) * m;
  float* sh = reinterpret_cast<float*>(smem);    // [rows][2][m]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < m) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        sh[(threadIdx.y * 2) * m + c + k] = ag[i][k];
        sh[(threadIdx.y * 2 + 1) * m + c + k] = ab[i][k];
      }
    }
  }
  __syncthreads();
  for (int c = tid; c < m; c += blockDim.x * rows) {
    float g = 0.f, b = 0.f;
    for (int y = 0; y < rows; ++y) {
      g += sh[(y * 2) * m + c];
      b += sh[(y * 2 + 1) * m + c];
    }
    out_g[c] = g;
    out_b[c] = b;
  }
}

// Shape of the one-pass kernel for a width, or stages < 2: too wide for the ring.
struct BwdShape {
  RowShape rows;
  Ring ring;
};
BwdShape bwd_shape(int64_t m, int esz) {
  BwdShape sh;
  sh.rows = row_shape(m, 16, 512);
  // x and dy of a group, the window's slack included; at the end the ring holds the column sums
  sh.ring.slot = (int)(((int64_t)sh.rows.rows * m * esz + 15 + 16) / 16 * 16);
  sh.ring.stages = (int)std::min<int64_t>(kMaxStages, kRingBytes / (2 * (int64_t)sh.ring.slot));
  return sh;
}

template <typename T, int V, int MAXT>
cudaError_t launch_bwd(const Bwd& a, const BwdShape& sh, int grid, cudaStream_t s) {
  auto kern = ln_bwd_kernel<T, V, 16 / V, MAXT>;
  const size_t smem = std::max((size_t)sh.ring.stages * 2 * sh.ring.slot,
                               (size_t)sh.rows.rows * 2 * a.m * sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3((unsigned)grid), dim3((unsigned)sh.rows.threads, (unsigned)sh.rows.rows),
                  smem, s, a, sh.ring);
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
  if (a.m <= kRegWidth && a.T < INT32_MAX) {
    const bool vec = a.m * (t == DT::BF16 ? 2 : 4) % 16 == 0;   // every row starts on 16 bytes
    if (t == DT::BF16)
      return vec ? fwd_width<__nv_bfloat16, 8>(a, s) : fwd_width<__nv_bfloat16, 1>(a, s);
    return vec ? fwd_width<float, 4>(a, s) : fwd_width<float, 1>(a, s);
  }
  const dim3 grid((unsigned)row_blocks(a.T)), block(kThreads);
  return t == DT::BF16 ? launch_k(ln_fwd_any_kernel<__nv_bfloat16>, grid, block, 0, s, a)
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
  const BwdShape sh = a.m <= kRegWidth ? bwd_shape(a.m, esz) : BwdShape{};
  if (a.m <= kRegWidth && sh.ring.stages >= 2) {
    const int64_t groups = (a.T + sh.rows.rows - 1) / sh.rows.rows;
    a.parts = (int)std::min<int64_t>(groups, kMaxParts);
    {
      TraceScope tr("ln_bwd", s);
      const bool vec = a.m * esz % 16 == 0;   // every row starts on 16 bytes
      if (sh.rows.threads <= 512) {
        if (t == DT::BF16)
          e = vec ? launch_bwd<__nv_bfloat16, 8, 512>(a, sh, a.parts, s)
                  : launch_bwd<__nv_bfloat16, 1, 512>(a, sh, a.parts, s);
        else
          e = vec ? launch_bwd<float, 4, 512>(a, sh, a.parts, s)
                  : launch_bwd<float, 1, 512>(a, sh, a.parts, s);
      } else {
        if (t == DT::BF16)
          e = vec ? launch_bwd<__nv_bfloat16, 8, 1024>(a, sh, a.parts, s)
                  : launch_bwd<__nv_bfloat16, 1, 1024>(a, sh, a.parts, s);
        else
          e = vec ? launch_bwd<float, 4, 1024>(a, sh, a.parts, s)
                  : launch_bwd<float, 1, 1024>(a, sh, a.parts, s);
      }
    }
    if (e != cudaSuccess || !cols) return e;
    TraceScope tr("ln_bwd_sum", s);
    return launch_k(ln_cols_sum_kernel, sum_grid, block, 0, s, a);
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
    e = launch_k(ln_cols_sum_kernel, sum_grid, block, 0, s, a);
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
