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
