// Newton-Schulz orthogonalisation of small matrices (at most 128 x 128, packed blocks up to 128):
// one CTA per matrix and one launch for everything. X, A and B stay in shared memory as fp16 parts
// in the tensor core's operand layouts, accumulators in tensor memory; the formulas, scales, part
// products and their order are those of orth.cu, whose fifteen dependent products cost about 6 us
// each in round trips through L2 (100 us for 16 blocks of 64; here the time of one matrix).
//
// An operand is 128 rows x 128 columns per part: two chunks of 64 columns, 128 rows of 128 bytes
// each, 16-byte unit u of row i at u ^ (i & 7). As a left or right operand of gram and square, and
// as update's left operand, it is read K-major; X is update's right operand as it lies, N-major.
#include "orth_mma.cuh"

#include <algorithm>

namespace poetx {
namespace orth {
namespace {

constexpr int kSmallSide = 128;
constexpr int kThreads = kNormThreads;               // eight warps
constexpr uint32_t kChunkBytes = 128 * 128;          // 128 rows x 64 columns
constexpr uint32_t kPartBytes = 2 * kChunkBytes;     // one part of one operand
constexpr uint32_t kOperandBytes = 2 * kPartBytes;
constexpr int kOutLd = kSmallSide + 1;               // staged results: floats per row
constexpr size_t kSmem = 3 * kOperandBytes + 1024;
static_assert((size_t)kSmallSide * kOutLd * sizeof(float) <= 2 * kOperandBytes,
              "the result is staged over A and B");

struct Small {
  const void* x;
  void* out;
  int in_f32, out_f32, skew, tall, steps, exact, fmode;
  int m, n, r, k;                      // the caller's matrix; as worked on, r <= k
  long long elems;                     // values of one matrix in the caller's arrays
  double eps, sx;
  int* err;
  float f[3][kMaxSteps], fa[kMaxSteps], da[kMaxSteps];   // as in orth.cu
};

__device__ __forceinline__ uint32_t at16(int i, int j) {   // byte of element (i, j) in a part
  return (uint32_t)(j >> 6) * kChunkBytes + (uint32_t)i * 128 +
         ((((uint32_t)(j >> 3) & 7u) ^ ((uint32_t)i & 7u)) << 4) + ((uint32_t)j & 7u) * 2;
}

__global__ void __launch_bounds__(kThreads, 1) ns_small_kernel(const __grid_constant__ Small p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t done_bar;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* X = smem;
  uint8_t* A = smem + kOperandBytes;
  uint8_t* B = smem + 2 * kOperandBytes;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const Ctl ctl{&abort_flag, p.err};
  const long long base = (long long)blockIdx.x * p.elems;
  const int R = (p.r + 63) / 64 * 64, ld = (p.k + 63) / 64 * 64;   // padded with zeros

  if (tid == 0) {
    mbar_init(smem_u32(&done_bar), 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_holder)),
                 "r"(128u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (uint32_t i = tid; i < kOperandBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(X)[i] = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();
  pdl_trigger();

  // the norm in 64 bits, then X_0's parts
  double s = 0.0;
  for (int e = tid; e < (int)p.elems; e += kThreads) {
    const double v = ld_in(p.x, base + e, p.in_f32);
    s += v * v;
  }
  s = block_sum(s);   // (its barriers also order the zeros before the values)
  const double f0 = p.sx / (sqrt(p.skew ? 2.0 * s : s) + p.eps);
  auto put_x = [&](int i, int j, float v) {
    const __half h = __float2half_rn(v);
    *reinterpret_cast<__half*>(X + at16(i, j)) = h;
    *reinterpret_cast<__half*>(X + kPartBytes + at16(i, j)) = __float2half_rn(v - __half2float(h));
  };
  if (p.skew) {
    const int b = p.n;
    for (int i = tid >> 5; i < b; i += kThreads / 32)   // a warp per row of the triangle
      for (int j = i + 1 + lane; j < b; j += 32) {
        const float v = (float)((double)ld_in(p.x, base + i * b - i * (i + 1) / 2 - i - 1 + j,
                                              p.in_f32) * f0);
        put_x(i, j, v);
        put_x(j, i, -v);
      }
  } else {
    for (int i = tid >> 5; i < p.m; i += kThreads / 32)
      for (int j = lane; j < p.n; j += 32) {
        const float v = (float)((double)ld_in(p.x, base + i * p.n + j, p.in_f32) * f0);
        if (p.tall) put_x(j, i, v);
        else put_x(i, j, v);
      }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;

  const int quarter = warp & 3, c0 = (warp >> 2) * 64;   // this warp's rows and columns of a result
  const int row = quarter * 32 + lane;
  const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0;
  uint32_t phase = 0;
  bool ok = true;
  for (int q = 0; ok && q < 3 * p.steps; ++q) {
    const int t = q / 3, kind = q - 3 * t;
    const bool last = t + 1 == p.steps, out = kind == kUpdate && last;
    const int N = kind == kUpdate ? ld : R, K = kind == kGram ? ld : R;
    if (warp == 0) {
      const int ns = p.exact ? 3 : kind == kUpdate && !last ? 2 : 1;
      const uint32_t id = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24) |
                          (kind == kUpdate ? 1u << 16 : 0u);
      const uint32_t sa = smem_u32(kind == kGram ? X : kind == kSquare ? A : B);
      const uint32_t sb = smem_u32(kind == kSquare ? A : X);
      for (int seg = 0; seg < ns; ++seg) {
        // hi hi | hi lo, hi hi | lo hi, hi lo, hi hi
        const uint32_t pa = ns == 3 && seg == 0 ? kPartBytes : 0u;
        const uint32_t pb = ns > 1 && seg == ns - 2 ? kPartBytes : 0u;
        for (int k = 0; k < K; k += 16) {
          const uint32_t kmaj = (uint32_t)(k >> 6) * kChunkBytes + (uint32_t)(k & 63) * 2;
          const uint32_t a = desc_lo(sa + pa + kmaj, 16);
          const uint32_t b = kind == kUpdate ? desc_lo(sb + pb + (uint32_t)k * 128, kChunkBytes)
                                             : desc_lo(sb + pb + kmaj, 16);
          if (elect_one()) mma<1>(tmem, a, b, id, (seg > 0 || k > 0) ? 1u : 0u);
        }
      }
      if (elect_one()) umma_commit(smem_u32(&done_bar));
    }
    ok = wait_inline(smem_u32(&done_bar), phase, ctl, kErrMma);
    phase ^= 1u;
    ok = __syncthreads_and(ok);
    if (!ok) break;
    tc_fence_after();
    // columns past the result's padded width are not computed
    if (c0 < N) {
      float v[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t r[32];
        tmem_ld32(trow + (uint32_t)c, r);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[c + i] = __uint_as_float(r[i]);
      }
      const float f = p.f[kind][t];
      if (out) {
        float* stage = reinterpret_cast<float*>(A);
#pragma unroll
        for (int c = 0; c < 64; ++c) stage[row * kOutLd + c0 + c] = v[c] * f;
      } else {
        uint8_t* to = kind == kGram ? A : kind == kSquare ? B : X;
        const float fa = p.fa[t], da = p.da[t];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t at = at16(row, c0 + 8 * u);
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = v[8 * u + i] * f;
          if (kind == kSquare) {   // + fa A + da I
            const uint4 h = *reinterpret_cast<const uint4*>(A + at);
            const uint4 l = *reinterpret_cast<const uint4*>(A + kPartBytes + at);
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 a2 = __half22float2(*reinterpret_cast<const __half2*>(&hw[i]));
              const float2 b2 = p.exact ? __half22float2(*reinterpret_cast<const __half2*>(&lw[i]))
                                        : make_float2(0.f, 0.f);
              e[2 * i] += (a2.x + b2.x) * fa;
              e[2 * i + 1] += (a2.y + b2.y) * fa;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (row == c0 + 8 * u + i) e[i] += da;
          }
          uint32_t h[4], l[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 w = __floats2half2_rn(e[2 * i], e[2 * i + 1]);
            const __half2 z =
                __floats2half2_rn(e[2 * i] - __low2float(w), e[2 * i + 1] - __high2float(w));
            h[i] = *reinterpret_cast<const uint32_t*>(&w);
            l[i] = *reinterpret_cast<const uint32_t*>(&z);
          }
          *reinterpret_cast<uint4*>(to + at) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + kPartBytes + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (ok) {
    // the staged result, row by row of the caller's array
    const float* stage = reinterpret_cast<const float*>(A);
    if (p.fmode == kPacked) {
      const int b = p.n;
      for (int i = tid >> 5; i < b; i += kThreads / 32)
        for (int j = i + 1 + lane; j < b; j += 32)
          put(p.out, base + i * b - i * (i + 1) / 2 - i - 1 + j, stage[i * kOutLd + j], p.out_f32);
    } else {
      for (int i = tid >> 5; i < p.m; i += kThreads / 32)
        for (int j = lane; j < p.n; j += 32)
          put(p.out, base + i * p.n + j,
              p.tall ? stage[j * kOutLd + i] : stage[i * kOutLd + j], p.out_f32);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(128u)
                 : "memory");
  }
}

}  // namespace

bool small_fits(const Problem& p) { return std::max(p.m, p.n) <= kSmallSide; }

cudaError_t run_small(const Problem& p, const Plan& plan, const void* x, void* out,
                      cudaStream_t s) {
  Small q{};
  q.x = x;
  q.out = out;
  q.in_f32 = p.in_t == DT::F32;
  q.exact = q.out_f32 = p.out_t == DT::F32;
  q.skew = p.form == Form::Skew;
  q.tall = !q.skew && p.m > p.n;
  q.fmode = q.skew ? kPacked : kRows;
  q.steps = p.steps;
  q.m = (int)p.m;
  q.n = (int)p.n;
  q.r = (int)std::min(p.m, p.n);
  q.k = (int)std::max(p.m, p.n);
  q.elems = q.skew ? p.m * (p.m - 1) / 2 : p.m * p.n;
  q.eps = p.eps;
  q.sx = plan.sx[0];
  q.err = device_error_word();
  if (!q.err) return cudaErrorUnknown;
  fill_factors(p, plan, q.f, q.fa, q.da);
  cudaError_t e = cudaFuncSetAttribute(ns_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmem);
  if (e != cudaSuccess) return e;
  TraceScope t("ns_small", s);
  return launch_k(ns_small_kernel, dim3((unsigned)p.batch), dim3(kThreads), kSmem, s, q);
}

}  // namespace orth
}  // namespace poetx
