// Newton-Schulz orthogonalisation of small matrices (at most 128 x 128, packed blocks up to 128):
// one CTA per matrix and one launch for everything. X, A and B stay in shared memory as fp16 parts
// in the tensor core's operand layouts, accumulators in tensor memory; the formulas, scales, part
// products (three, for bf16 results too) and their order are those of orth.cu, whose fifteen dependent
// products cost about 6 us each in round trips through L2 (100 us for 16 blocks of 64; here 28 us, the
// time of one matrix).
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
// The large product is summed in several accumulators, four of 16 of K = 64 or two of 64 of K = 128,
// and those are added in registers: the tensor core truncates what it adds (see ns_kernel in orth.cu).
// Blocks of 32, 64, 128: 1.3, 0.8, 1.1 times the error of fp32 products; with one accumulator 1.5,
// 1.4, 1.7 times in 3 to 10 % less time (16 blocks of 64 27.1 us against 28.0, 3 of 128 42.6 us
// against 47.3).
constexpr int kMostAccs = 4;
constexpr uint32_t kTmemCols = kSmallSide * kMostAccs;
constexpr int kOutLd = kSmallSide + 1;               // staged results: floats per row
constexpr size_t kSmem = 3 * kOperandBytes + 1024;
static_assert((size_t)kSmallSide * kOutLd * sizeof(float) <= 2 * kOperandBytes,
              "the result is staged over A and B");

struct Small {
  const void* x;
  void* out;
  int in_f32, out_f32, skew, tall, steps, fmode;
  int m, n, r, k;                      // the caller's matrix; as worked on, r <= k
  long long elems;                     // values of one matrix in the caller's arrays
  double eps;
  float scale;
  float coeffs[3 * kMaxSteps];
  int* err;
  Plan plan;                           // of matrices whose norm is eps or more
};

__device__ __forceinline__ uint32_t at16(int i, int j) {   // byte of element (i, j) in a part
  return (uint32_t)(j >> 6) * kChunkBytes + (uint32_t)i * 128 +
         ((((uint32_t)(j >> 3) & 7u) ^ ((uint32_t)i & 7u)) << 4) + ((uint32_t)j & 7u) * 2;
}

// 32 columns of an accumulator on their way into registers, which tmem_arrived() hands out
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) ns_small_kernel(const __grid_constant__ Small p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t done_bar;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  __shared__ Plan plan;
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
                 "r"(kTmemCols)
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
  const double norm = sqrt(p.skew ? 2.0 * s : s), sum = norm + p.eps;
  const bool below = below_eps(norm, p.eps);
  const double f0 = (below ? x0_scale(norm / sum) : p.plan.x0) / sum;
  if (!below) {
    for (int i = tid; i < p.steps; i += kThreads) plan.step[i] = p.plan.step[i];
    if (tid == 0) plan.out = p.plan.out;
  } else if (tid == 0) {
    plan_from(norm / sum, p.coeffs, p.steps, p.scale, plan.step, &plan.out);
  }
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

  // this warp's rows of a result; of its columns the first or the second half
  const int quarter = warp & 3, half = warp >> 2;
  const int row = quarter * 32 + lane;
  const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
  uint32_t phase = 0;
  bool ok = true;
  for (int q = 0; ok && q < 3 * p.steps; ++q) {
    const int t = q / 3, kind = q - 3 * t;
    const bool out = kind == kUpdate && t + 1 == p.steps;
    const int N = kind == kUpdate ? ld : R, K = kind == kGram ? ld : R;
    if (warp == 0) {
      const int deep = K == 64 ? 4 : 6;   // 16 or 64 of K an accumulator
      const uint32_t id = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24) |
                          (kind == kUpdate ? 1u << 16 : 0u);
      const uint32_t sa = smem_u32(kind == kGram ? X : kind == kSquare ? A : B);
      const uint32_t sb = smem_u32(kind == kSquare ? A : X);
      for (int seg = 0; seg < 3; ++seg) {   // lo hi, hi lo, hi hi
        const uint32_t pa = seg == 0 ? kPartBytes : 0u, pb = seg == 1 ? kPartBytes : 0u;
        for (int k = 0; k < K; k += 16) {
          const uint32_t kmaj = (uint32_t)(k >> 6) * kChunkBytes + (uint32_t)(k & 63) * 2;
          const uint32_t a = desc_lo(sa + pa + kmaj, 16);
          const uint32_t b = kind == kUpdate ? desc_lo(sb + pb + (uint32_t)k * 128, kChunkBytes)
                                             : desc_lo(sb + pb + kmaj, 16);
          // the small products and the first part of the large one share an accumulator
          const int acc = seg == 2 ? k >> deep : 0;
          const bool more = acc > 0 ? (k & ((1 << deep) - 1)) > 0 : seg > 0 || k > 0;
          if (elect_one())
            mma<1>(tmem + (uint32_t)(acc * kSmallSide), a, b, id, more ? 1u : 0u);
        }
      }
      if (elect_one()) umma_commit(smem_u32(&done_bar));
    }
    const float f = plan.step[t].f[kind], fa = plan.step[t].fa, da = plan.step[t].da;
    ok = wait_inline(smem_u32(&done_bar), phase, ctl, kErrMma);
    phase ^= 1u;
    ok = __syncthreads_and(ok);
    if (!ok) break;
    tc_fence_after();
    // columns past the result's padded width N (64 or 128) are not computed
    for (int c0 = half * (N / 2); c0 < (half + 1) * (N / 2); c0 += 32) {
      float v[32];
      {
        uint32_t r[kMostAccs][32];
        const bool four = K == 64;
        tmem_ld32_start(trow + (uint32_t)c0, r[0]);
        tmem_ld32_start(trow + (uint32_t)(kSmallSide + c0), r[1]);
        if (four) {
          tmem_ld32_start(trow + (uint32_t)(2 * kSmallSide + c0), r[2]);
          tmem_ld32_start(trow + (uint32_t)(3 * kSmallSide + c0), r[3]);
        }
        tmem_arrived(r[0]);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[0][i]);
        tmem_arrived(r[1]);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(r[1][i]);
        if (four) {
          tmem_arrived(r[2]);
          tmem_arrived(r[3]);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] += __uint_as_float(r[2][i]) + __uint_as_float(r[3][i]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= f;
      }
      if (out) {
        float* stage = reinterpret_cast<float*>(A);
#pragma unroll
        for (int c = 0; c < 32; ++c) stage[row * kOutLd + c0 + c] = v[c] * plan.out;
        continue;
      }
      uint8_t* to = kind == kGram ? A : kind == kSquare ? B : X;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t at = at16(row, c0 + 8 * u);
        float* e = v + 8 * u;
        if (kind == kSquare) {   // + fa A + da I
          const uint4 h = *reinterpret_cast<const uint4*>(A + at);
          const uint4 l = *reinterpret_cast<const uint4*>(A + kPartBytes + at);
          const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a2 = __half22float2(*reinterpret_cast<const __half2*>(&hw[i]));
            const float2 b2 = __half22float2(*reinterpret_cast<const __half2*>(&lw[i]));
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
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
  q.out_f32 = p.out_t == DT::F32;
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
  q.err = device_error_word();
  if (!q.err) return cudaErrorUnknown;
  std::copy(p.coeffs, p.coeffs + 3 * p.steps, q.coeffs);
  q.scale = p.scale;
  q.plan = plan;
  cudaError_t e = cudaFuncSetAttribute(ns_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmem);
  if (e != cudaSuccess) return e;
  TraceScope t("ns_small", s);
  return launch_k(ns_small_kernel, dim3((unsigned)p.batch), dim3(kThreads), kSmem, s, q);
}

}  // namespace orth
}  // namespace poetx
