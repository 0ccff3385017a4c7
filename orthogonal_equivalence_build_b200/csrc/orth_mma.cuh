// Pieces shared by the two Newton-Schulz kernels (orth.cu, orth_small.cu). Local to the including
// translation unit.
#pragma once
#include "orth.h"
#include "umma_ptx.cuh"

#include <cuda_fp16.h>

namespace poetx {
namespace orth {
namespace {

using namespace umma;

enum : int { kGram = 0, kSquare = 1, kUpdate = 2 };
// Layout of the caller's output: rows, rows of the transposed result, packed strict upper triangles.
enum : int { kRows = 1, kTransposed = 2, kPacked = 3 };
// Waits may span whole products of other clusters.
constexpr uint64_t kLimitNs = 20000000000ull;
constexpr int kNormThreads = 256;

__device__ __forceinline__ float ld_in(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) s += part[w];
  __syncthreads();
  return s;
}

__device__ __forceinline__ void put(void* out, long long at, float x, int f32) {
  if (f32) static_cast<float*>(out)[at] = x;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

// ------------------------------------------------------------------ scales
// The exponent of the power of two that brings values of at most `most` to between half of fp16's
// range, 32768, and a half of that. (Nothing but zeros: any.)
__host__ __device__ inline int scale_exponent(double most) {
  if (!(most > 0.0)) return 0;
  int k;
  return frexp(most, &k) == 0.5 ? 16 - k : 15 - k;
}

// The scale of X_0 and the factors of every step for singular values of X_0 in [0, top].
__host__ __device__ inline double x0_scale(double top) {
  return ldexp(1.0, scale_exponent(1.02 * top));
}
__host__ __device__ inline bool plan_from(double top, const float* coeffs, int steps, float scale,
                                          Factors* step, float* out) {
  int ex = scale_exponent(1.02 * top);
  for (int t = 0; t < steps; ++t) {
    const double a = coeffs[3 * t], b = coeffs[3 * t + 1], c = coeffs[3 * t + 2];
    if (!isfinite(a) || !isfinite(b) || !isfinite(c)) return false;
    // With l = s^2: B's eigenvalues a + b l + c l^2 and the next singular values
    // s |a + b l + c l^2| over l in [0, top^2] have their extremes at the ends or where the
    // derivatives b + 2 c l and a + 3 b l + 5 c l^2 vanish.
    const double end = top * top;
    double bb = fabs(a), x = 0.0;
    auto look = [&](double l) {
      if (!(l > 0.0 && l <= end)) return;
      const double e = fabs(a + b * l + c * l * l);
      bb = fmax(bb, e);
      x = fmax(x, sqrt(l) * e);
    };
    look(end);
    if (c != 0.0) {
      look(-b / (2.0 * c));
      const double disc = 9.0 * b * b - 20.0 * a * c;
      if (disc >= 0.0) {
        look((-3.0 * b + sqrt(disc)) / (10.0 * c));
        look((-3.0 * b - sqrt(disc)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      look(-a / (3.0 * b));
    }
    // Entries of a matrix do not pass its spectral norm; 2 % for the rounding on the way. The scales
    // follow the singular values down as well as up: fp16's smallest numbers would cut off the
    // parts of what shrinks. The factors stay near 2^-15 all the same, since a polynomial's
    // coefficients are bounded by its largest value; terms that vanish in fp32 vanish beside the others.
    top = 1.02 * x;
    const int ea = scale_exponent(1.02 * end), eb = scale_exponent(1.02 * bb);
    const int next = scale_exponent(1.02 * top);
    Factors& o = step[t];
    o.f[0] = (float)ldexp(1.0, ea - 2 * ex);
    o.f[1] = (float)ldexp(c, eb - 2 * ea);
    o.fa = (float)ldexp(b, eb - ea);
    o.da = (float)ldexp(a, eb);
    // The last update takes the operands' scales off and the caller's scale after them: their product
    // can lie among fp32's smallest numbers where the result does not.
    const int off = eb + ex, first = off < 100 ? off : 100;
    o.f[2] = (float)ldexp(1.0, t + 1 < steps ? next - off : -first);
    *out = (float)ldexp((double)scale, first - off);
    ex = next;
    if (!(top < 1e6)) return false;
  }
  return true;
}

// A matrix whose norm is below eps has no singular value near 1 after the division by norm + eps, and
// its own scales: under those for [0, 1], fp16's smallest numbers would cut off its parts (with |X|_F =
// 1e-5 eps fp32 results were 3e-5 off, with 1e-9 eps zeros). The plan of all others comes with the launch.
__device__ __forceinline__ bool below_eps(double norm, double eps) { return norm > 0.0 && norm < eps; }

// One lane of a converged warp, always the same one. The issuing warps run their loops with all
// lanes and elect one for each copy, MMA and arrival: addresses and descriptors then are the same
// in every lane and stay in uniform registers. With a loop of lane 0 alone a K block took 600
// cycles to issue whatever its tile.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p)
      :
      : "memory");
  return p != 0;
}

// Shared-memory descriptors as two words (smem_desc of umma_ptx.cuh): the upper one is the same for
// every operand (128-byte swizzle, 8-row groups 1024 bytes apart); the lower one holds the
// address and the leading offset.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (saddr >> 4) | ((lbo >> 4) << 16);
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                    uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "r"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "r"(kDescHi)
        : "memory");
}

// wait_bounded (umma_ptx.cuh) without the call: a call would put the accumulated registers on the
// stack, and setmaxnreg allows none.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, Ctl c, int code,
                                            uint64_t limit_ns = kLimitNs,
                                            bool stop_on_abort = true) {
  auto test = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (test()) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    if (test()) return true;
    if ((it & 31) == 0) {
      if (stop_on_abort && *c.abort) return false;
      if (global_ns() - t0 > limit_ns) {
        *c.abort = 1;
        if (code) atomicCAS(c.err, 0, code);
        return false;
      }
    }
  }
}
}  // namespace
}  // namespace orth
}  // namespace poetx
