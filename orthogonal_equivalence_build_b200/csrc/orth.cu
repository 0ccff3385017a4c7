// Newton-Schulz orthogonalisation of a stack of matrices on the tensor cores (tcgen05 / TMEM /
// TMA, sm_100a).
//
//   X_0 = X / (|X|_F + eps);   X_{t+1} = a_t X_t + (b_t A + c_t A^2) X_t,  A = X_t X_t^T
//
// with X laid out so that it has no more rows r than columns k (a taller input is transposed on
// its way in and back on its way out: X (X^T X) = (X X^T) X). Per step three products:
//   gram    A = X X^T, its epilogue also writes H = b I + c A          (symmetric)
//   square  B = a I + A H = a I + b A + c A^2                          (symmetric)
//   update  X <- B X                                                   (skew for skew X)
// The polynomial's lower terms ride on the diagonals of H and B, so no epilogue reads a matrix
// back. Symmetric (and skew) results are computed on the tiles on and above the diagonal; the
// epilogue stores every other tile twice, the second time transposed (and negated).
//
// Precision. Operands are fp16 parts of scaled values with fp32 accumulation: x = hi + lo,
// hi = fp16(x), lo = fp16(x - hi), which carries 22 bits. The scales are powers of two chosen on
// the host from the range of the singular values after each step (X_0 has them in [0, 1]; the
// quintic's range over an interval is known), so nothing overflows and the smallest entries that
// matter stay normal numbers.
//   fp32 results: every product is hi hi + hi lo + lo hi (three passes over K), error a few
//     2^-22 of the result's size.
//   bf16 results: one pass for gram and square; the update of every step but the last reads X in
//     both parts (two passes). X's rounding is what the iteration amplifies: a direction whose
//     singular value is 1e-3 of the largest is drowned by 2^-11 of the large ones, and it
//     is lifted by a = 3.4 a step while they stay. The rounding of A, H and B acts on the
//     directions in proportion and is not amplified. Against the exact result, in units of its
//     rms: 1.4e-3 for an update of a few strong directions over a background (single-part X
//     2.0e-3, and 9.5e-3 with a background of 3 % of the strongest); bf16 rounding alone is
//     1.7e-3.
#include "orth.h"
#include "umma_ptx.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

namespace poetx {
namespace orth {
namespace {

using namespace umma;

constexpr int BK = 64;
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;               // two per TMEM lane quarter, half of the columns each
constexpr int kThreads = 128 + 32 * kEpiWarps;
// Registers per thread at launch, then of warps 0..3 (which only issue copies and MMAs) and of the
// epilogue's: setmaxnreg moves them within what the block was launched with.
constexpr int kRegsLaunch = 168, kRegsIssue = 56, kRegsEpi = 224;
static_assert(128 * kRegsIssue + 32 * kEpiWarps * kRegsEpi <= kThreads * kRegsLaunch,
              "the register split must fit the launch's registers");
constexpr int kChunk = 2;                  // K blocks per accumulator of an fp32 result
constexpr int kPartBytes = 128 * BK * 2;   // one operand of one CTA and stage: 128 rows x 64
constexpr int kEpiStage = 8192;            // per epilogue warp
constexpr size_t kSmem = (size_t)kStages * 2 * kPartBytes + kEpiWarps * kEpiStage + 1024 + 256;

// ------------------------------------------------------------------ products
enum : int { kToMaps = 0, kRows = 1, kTransposed = 2, kPacked = 3 };

struct Prod {
  int tiles_m, tiles_n, per, total, sym, batch;
  int rows, cols;            // padded extents of the output (kToMaps)
  int nk, nseg;              // K blocks per segment; segment s multiplies parts pa[s], pb[s]
  int head, chunk;           // K blocks of a tile's first accumulator and of the later ones
  int pa[3], pb[3];
  float f0, d0, f1, d1;      // output o: acc * f + (i == j) * d
  int has1, lo;              // a second output; both outputs in two parts
  float mirror;              // sym: sign of the mirrored tile
  int fmode;                 // where the result goes
  void* out;                 // the caller's array (fmode != kToMaps)
  int out_f32, vec;          // its type; rows start on 16 bytes
  long long um, un;          // valid rows and columns of the result
  int* err;
};

struct Tile {
  int g, mb, nb;
};
// Symmetric results: row by row over the tiles on and above the diagonal. Others: bands of 16
// row tiles sweep the columns, so a band of the left operand stays in L2 while X streams.
__device__ __forceinline__ Tile decode(const Prod& p, int tile) {
  Tile t;
  t.g = tile / p.per;
  int l = tile - t.g * p.per;
  if (p.sym) {
    int i = 0;
    while (l >= p.tiles_n - i) l -= p.tiles_n - i++;
    t.mb = i;
    t.nb = i + l;
  } else {
    const int band = l / (16 * p.tiles_n), first = band * 16;
    const int gm = min(16, p.tiles_m - first), w = l - band * 16 * p.tiles_n;
    t.mb = first + w % gm;
    t.nb = w / gm;
  }
  return t;
}

template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y,
                                          int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}

// kind::f16, fp16 operands, fp32 accumulator, 128 CG x 128 CG tile
template <int CG, bool B_MN>
__device__ __forceinline__ constexpr uint32_t idesc() {
  return (1u << 4) | ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(128 * CG >> 3) << 17) |
         ((uint32_t)(128 * CG >> 4) << 24);
}

// wait_bounded (umma_ptx.cuh) without the call: a call would put the accumulated registers on the
// stack, and setmaxnreg allows none.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, Ctl c, int code,
                                            uint64_t limit_ns = kWaitLimitNs,
                                            bool stop_on_abort = true) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
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

// Four 8 x 8 blocks of 16-bit values: transposed out of shared memory, and back into it.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// One 32-row x 64-column piece of a warp to the fp16 maps: both outputs, both parts, and the
// mirrored piece of an off-diagonal tile. The warp's 8 KB stage is two halves that alternate, so
// a piece is packed while the previous one's copy still reads its half. A piece lies in its
// half in the 128-byte swizzle (16-byte unit u of row i at u ^ (i & 7)); the mirrored piece is
// read from there by transposing 8 x 8 blocks and lies in the 64-byte swizzle (unit u of row j at
// u ^ (j / 2 & 3)): neither side has bank conflicts.
__device__ __forceinline__ void emit_maps(const Prod& p, const CUtensorMap* out0,
                                          const CUtensorMap* out1, const CUtensorMap* mir0,
                                          const CUtensorMap* mir1, const float* v, int g, int row0,
                                          int col0, bool mirror, uint32_t stage, int lane,
                                          int& chunk) {
#pragma unroll 1
  for (int o = 0; o <= p.has1; ++o) {
    const float f = o ? p.f1 : p.f0, d = o ? p.d1 : p.d0;
#pragma unroll 1
    for (int part = 0; part <= p.lo; ++part) {
      int dq = row0 + lane - col0;            // the diagonal's column of this row's 64
      asm volatile("" : "+r"(dq));            // (not 64 comparisons kept over the loops)
      const int z = part * p.batch + g;
      const uint32_t half = stage + (chunk & 1) * 4096;
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 8 * u + 2 * q;
          const float a = v[c] * f + (dq == c ? d : 0.f);
          const float b = v[c + 1] * f + (dq == c + 1 ? d : 0.f);
          __half2 w = __floats2half2_rn(a, b);
          if (part) w = __floats2half2_rn(a - __low2float(w), b - __high2float(w));
          h[q] = *reinterpret_cast<uint32_t*>(&w);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         half + lane * 128 + ((u ^ (lane & 7)) << 4)),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        store_box(o ? out1 : out0, half, col0, row0, z);
        bulk_commit();
      }
      ++chunk;
      if (mirror) {
        const uint32_t other = stage + (chunk & 1) * 4096;
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        const uint32_t flip = p.mirror < 0.f ? 0x80008000u : 0u;
        // lane l names row l of the piece's 32 for the load, and for the store row l % 8 of the
        // unit's eight in 16-byte unit l / 8
        const uint32_t src = half + lane * 128;
        const int blk = lane >> 3, jj = lane & 7;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t r[4];
          ldmatrix4_trans(src + ((u ^ (lane & 7)) << 4), r);
#pragma unroll
          for (int q = 0; q < 4; ++q) r[q] ^= flip;
          stmatrix4(other + (8 * u + jj) * 64 + ((blk ^ ((jj >> 1) & 3)) << 4), r);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          store_box(o ? mir1 : mir0, other, row0, col0, z);
          bulk_commit();
        }
        ++chunk;
      }
    }
  }
}

__device__ __forceinline__ void put(void* out, long long at, float x, int f32) {
  if (f32) static_cast<float*>(out)[at] = x;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

// The same piece to the caller's array.
__device__ __forceinline__ void emit_user(const Prod& p, const float* v, int g, int row0,
                                          int col0, uint8_t* stage, int lane) {
  if (p.fmode == kTransposed) {
    // 32 rows of the piece are 32 neighbours of one output row
    const int i = row0 + lane, left = (int)min((long long)64, p.un - col0);
    if (i < p.um) {
      const long long at = ((long long)g * p.un + col0) * p.um + i;
      if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int q = 0; q < 64; ++q, o += p.um)
          if (q < left) *o = v[q] * p.f0;
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
        for (int q = 0; q < 64; ++q, o += p.um)
          if (q < left) *o = __float2bfloat16_rn(v[q] * p.f0);
      }
    }
    return;
  }
  // through the stage: row r in 256 bytes, 16-byte unit u at u ^ (r & 15)
#pragma unroll
  for (int u = 0; u < 16; ++u)
    *reinterpret_cast<float4*>(stage + lane * 256 + ((u ^ (lane & 15)) << 4)) =
        make_float4(v[4 * u] * p.f0, v[4 * u + 1] * p.f0, v[4 * u + 2] * p.f0, v[4 * u + 3] * p.f0);
  __syncwarp();
  auto unit = [&](int r, int u) {
    return *reinterpret_cast<const float4*>(stage + r * 256 + ((u ^ (r & 15)) << 4));
  };
  const int nrow = (int)min((long long)32, p.um - row0);
  if (p.fmode == kRows && p.vec) {
    const long long base = ((long long)g * p.um + row0) * p.un + col0;
    if (p.out_f32) {
      const int u = lane & 15;
      for (int r = lane >> 4; r < nrow; r += 2)
        if (col0 + 4 * u < p.un)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + base + r * p.un + 4 * u) =
              unit(r, u);
    } else {
      const int u = lane & 7;
      for (int r = lane >> 3; r < nrow; r += 4)
        if (col0 + 8 * u < p.un) {
          const float4 a = unit(r, 2 * u), b = unit(r, 2 * u + 1);
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + base + r * p.un + 8 * u) =
              make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                         pack_bf16x2(b.z, b.w));
        }
    }
  } else {
    for (int r = 0; r < nrow; ++r) {
      const int i = row0 + r;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h, j = col0 + c;
        const float x =
            *reinterpret_cast<const float*>(stage + r * 256 + (((c >> 2) ^ (r & 15)) << 4) +
                                            (c & 3) * 4);
        if (p.fmode == kPacked) {
          // packed strict upper triangle of block g
          const long long b = p.un;
          if (j > i && j < b)
            put(p.out, (long long)g * (b * (b - 1) / 2) + i * b - (long long)i * (i + 1) / 2 - i -
                           1 + j, x, p.out_f32);
        } else if (j < p.un) {
          put(p.out, ((long long)g * p.um + i) * p.un + j, x, p.out_f32);
        }
      }
    }
  }
  __syncwarp();   // the stage is read before it is written again
}

// C = A B on 128 CG x 128 CG tiles: CG = 1 one CTA, CG = 2 a CTA pair (cta_group::2, each CTA
// holds half of the tile's rows of A and half of its columns of B). A is K-major; B is K-major
// (gram and square: B^T has A's layout) or N-major (update: B = X). Persistent and
// warp-specialised: warp 0 streams operand tiles by TMA through a ring, one lane of warp 1
// issues the MMAs into one of two accumulators, warps 4..11 empty the other one (warps 2 and 3
// complete the first register group).
// The tensor core adds to its fp32 accumulator without rounding to nearest: every 16-deep step
// loses up to a whole unit in the last place, always towards zero, and K = 2048 in three
// passes came out 3.8e-5 off. So the parts' small products (hi lo, lo hi) come first, and for fp32
// results an accumulator of large products sums only kChunk K blocks; the epilogue warps add the
// accumulators in registers (round to nearest) while the next one fills.
// Every wait is bounded; on expiry the device error word is set, the roles leave their loops,
// copies and MMAs in flight are waited for (bounded) and TMEM is freed.
template <int CG, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1)
ns_product_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                  const __grid_constant__ CUtensorMap out0, const __grid_constant__ CUtensorMap out1,
                  const __grid_constant__ CUtensorMap mir0, const __grid_constant__ CUtensorMap mir1,
                  const __grid_constant__ Prod p) {
  constexpr int TILE = 128 * CG;
  constexpr uint32_t TMEM_COLS = 2 * TILE;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sa = smem;
  uint8_t* sb = smem + kStages * kPartBytes;
  uint8_t* sepi = sb + kStages * kPartBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sepi + kEpiWarps * kEpiStage);
  uint64_t* full = bars;              // leader only
  uint64_t* empty = bars + kStages;
  uint64_t* tfull = empty + kStages;  // [2]
  uint64_t* tempty = tfull + 2;       // [2], leader only
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const Ctl ctl{abort_flag, p.err};
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  const int nk = p.nk * p.nseg;   // K blocks of a tile: p.head, then p.chunk at a time

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(tfull + a), 1);
      mbar_init(smem_u32(tempty + a), kEpiWarps * CG);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_holder)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_holder)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();   // both CTAs' barriers exist before a remote arrive
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait();      // the operands belong to the previous kernel of the stream
  pdl_trigger();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        int it = 0, s = 0;        // K blocks issued; ring slot and its phase
        uint32_t ph = 1u;
        bool ok = true;
        uint32_t fb0 = smem_u32(full);
        if constexpr (CG == 2) fb0 = map_to_rank(fb0, 0);
        for (int tile = first; ok && tile < p.total; tile += step) {
          const Tile t = decode(p, tile);
          const int am = t.mb * TILE + (int)rank * 128, bn = t.nb * TILE + (int)rank * 128;
          for (int seg = 0; ok && seg < p.nseg; ++seg) {
            const int za = p.pa[seg] * p.batch + t.g, zb = p.pb[seg] * p.batch + t.g;
            for (int k = 0; k < p.nk * BK; k += BK, ++it) {
              // stops only when the wait runs out: both CTAs of a pair are released by the same
              // commits, so both have then issued the same loads
              if (!wait_inline(smem_u32(empty + s), ph, ctl, kErrProducer, kWaitLimitNs,
                               /*stop_on_abort=*/false)) {
                ok = false;
                break;
              }
              const uint32_t fb = fb0 + (uint32_t)(s * 8);
              if (leader) mbar_expect_tx(smem_u32(full + s), CG * 2 * kPartBytes);
              load_box<CG>(smem_u32(sa + s * kPartBytes), &tma_a, fb, k, am, za);
              const uint32_t db = smem_u32(sb + s * kPartBytes);
              if constexpr (B_MN) {
                load_box<CG>(db, &tma_b, fb, bn, k, zb);
                load_box<CG>(db + 64 * BK * 2, &tma_b, fb, bn + 64, k, zb);
              } else {
                load_box<CG>(db, &tma_b, fb, k, bn, zb);
              }
              if (++s == kStages) { s = 0; ph ^= 1u; }
            }
          }
        }
        if (!ok && leader)   // let the copies already issued land before the CTA leaves
          for (int j = max(0, it - kStages); j < it; ++j)
            wait_inline(smem_u32(full + j % kStages), (uint32_t)(j / kStages) & 1u, ctl, 0,
                         kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (leader && lane == 0) {
        constexpr uint32_t id = idesc<CG, B_MN>();
        auto commit = [](uint32_t bar) {
          if constexpr (CG == 2) umma_commit_pair_both(bar);
          else umma_commit(bar);
        };
        int s = 0, count = 0;   // ring slot, accumulators used
        uint32_t ph = 0u;
        bool ok = true;
        for (int tile = first; ok && tile < p.total; tile += step) {
          for (int kb = 0, end = p.head; ok && kb < nk; end = min(nk, end + p.chunk), ++count) {
            const int acc = count & 1;
            if (!wait_inline(smem_u32(tempty + acc), ((uint32_t)(count >> 1) & 1u) ^ 1u, ctl,
                             kErrMma)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * TILE);
            for (uint32_t more = 0u; kb < end; ++kb) {
              if (!wait_inline(smem_u32(full + s), ph, ctl, kErrMma)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t a0 = smem_u32(sa + s * kPartBytes), b0 = smem_u32(sb + s * kPartBytes);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk, more = 1u) {
                const uint64_t ad = smem_desc(a0 + kk * 32, 16, 1024);
                const uint64_t bd = B_MN ? smem_desc(b0 + kk * 2048, 64 * BK * 2, 1024)
                                         : smem_desc(b0 + kk * 32, 16, 1024);
                if constexpr (CG == 2) umma_bf16_pair(d, ad, bd, id, more);
                else umma_bf16(d, ad, bd, id, more);
              }
              commit(smem_u32(empty + s));
              if (++s == kStages) { s = 0; ph ^= 1u; }
            }
            if (ok) commit(smem_u32(tfull + acc));
          }
        }
        commit(smem_u32(drain));   // every MMA of this thread has retired once this completes
        wait_inline(smem_u32(drain), 0, ctl, ok ? kErrMma : 0, ok ? kWaitLimitNs : kDrainLimitNs);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 4..11)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    constexpr int COLS = TILE / 2;        // this warp's columns of the tile
    const int quarter = warp & 3;         // TMEM lanes 32 quarter .. + 31
    const int cbase = ((warp - 4) >> 2) * COLS;
    uint8_t* stage = sepi + (warp - 4) * kEpiStage;
    uint32_t back = smem_u32(tempty);
    if constexpr (CG == 2) back = map_to_rank(back, 0);
    int count = 0, chunk = 0;
    bool ok = true;
    for (int tile = first; ok && tile < p.total; tile += step) {
      const Tile t = decode(p, tile);
      const int row0 = t.mb * TILE + (int)rank * 128 + quarter * 32;
      const bool mirror = p.sym && t.mb != t.nb;
      float v[COLS];
#pragma unroll
      for (int q = 0; q < COLS; ++q) v[q] = 0.f;
      for (int done = 0; done < nk; done = done ? done + p.chunk : p.head, ++count) {
        const int acc = count & 1;
        if (!wait_inline(smem_u32(tfull + acc), (uint32_t)(count >> 1) & 1u, ctl, kErrEpilogue)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t trow = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                              (uint32_t)(acc * TILE + cbase);
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t r[32];
          tmem_ld32(trow + (uint32_t)c, r);
#pragma unroll
          for (int q = 0; q < 32; ++q) v[c + q] += __uint_as_float(r[q]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_remote_relaxed(back + (uint32_t)(acc * 8));
          else mbar_arrive(back + (uint32_t)(acc * 8));
        }
      }
      if (!ok) break;
      // pieces wholly in the padding (or below the diagonal of a packed result) are not stored
      const int rmax = p.fmode == kToMaps ? p.rows : (int)p.um;
      const int cmax = p.fmode == kToMaps ? p.cols : (int)p.un;
#pragma unroll
      for (int c = 0; c < COLS; c += 64) {
        const int col0 = t.nb * TILE + cbase + c;
        if (row0 >= rmax || col0 >= cmax || (p.fmode == kPacked && col0 + 63 <= row0)) continue;
        if (p.fmode == kToMaps)
          emit_maps(p, &out0, &out1, &mir0, &mir1, v + c, t.g, row0, col0, mirror,
                    smem_u32(stage), lane, chunk);
        else
          emit_user(p, v + c, t.g, row0, col0, stage, lane);
      }
    }
    if (lane == 0) bulk_wait_all();   // every store written before the CTA leaves
    __syncwarp();
  }

  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();   // no remote arrive may target a CTA that has left
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                   "r"(TMEM_COLS)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                   "r"(TMEM_COLS)
                   : "memory");
  }
}

// ------------------------------------------------------------------ norm and first split
constexpr int kNormThreads = 256;
constexpr int64_t kNormChunk = 16384;   // elements per block of the norm pass, at least
constexpr int kMaxChunks = 512;

int norm_chunks(int64_t elems) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxChunks, elems / kNormChunk));
}

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

// partial[g][chunk] = sum of the chunk's squares, in 64 bits: an fp32 square overflows at 1.8e19
// and vanishes at 1e-23, both of which are ordinary fp32 and bf16 values.
__global__ void __launch_bounds__(kNormThreads)
ns_norm_kernel(const void* __restrict__ x, int f32, long long elems, int chunks,
               double* __restrict__ partial) {
  pdl_wait();
  pdl_trigger();
  const long long base = (long long)blockIdx.y * elems;
  const long long per = (elems + chunks - 1) / chunks;
  const long long lo = per * blockIdx.x, hi = min(elems, lo + per);
  double s = 0.0;
  for (long long i = lo + threadIdx.x; i < hi; i += kNormThreads) {
    const double v = ld_in(x, base + i, f32);
    s += v * v;
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[(long long)blockIdx.y * chunks + blockIdx.x] = s;
}

// X_0 in two fp16 parts, [2][batch][R][ld], from the caller's array, one 64 x 64 tile per block:
// the tile goes through shared memory, so that reads follow the caller's rows and writes the
// workspace's, whichever way round they are. Padding is written as zeros.
struct Prep {
  const void* x;
  int f32, form, tall, chunks, batch, tiles_c;
  long long m, n;            // the caller's matrix (Skew: m = n = b)
  int r, k, R, ld;           // the workspace's: r x k in R x ld
  double eps, sx, norm_mult; // norm^2 = norm_mult * sum of the partials
  const double* partial;
  __half* out;
};
__global__ void __launch_bounds__(256) ns_prep_kernel(const __grid_constant__ Prep p) {
  __shared__ float tile[64][65];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, tid = threadIdx.x;
  double s = 0.0;
  for (int c = tid; c < p.chunks; c += 256) s += p.partial[(long long)g * p.chunks + c];
  s = block_sum(s);
  const double f = p.sx / (sqrt(p.norm_mult * s) + p.eps);
  const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  if (p.form == (int)Form::Skew && tr > tc) return;   // written by its mirror
  const int i0 = tr * 64, j0 = tc * 64;
#pragma unroll 4
  for (int e = tid; e < 4096; e += 256) {
    const int u = e >> 6, w = e & 63;     // w runs along the caller's rows
    float v = 0.f;
    if (p.form == (int)Form::Skew) {
      const int i = i0 + u, j = j0 + w;
      if (i < j && j < p.r)
        v = (float)((double)ld_in(p.x, (long long)g * (p.m * (p.m - 1) / 2) + i * p.m -
                                           (long long)i * (i + 1) / 2 - i - 1 + j, 1) * f);
      tile[u][w] = v;
    } else if (!p.tall) {
      if (i0 + u < p.r && j0 + w < p.k)
        v = (float)((double)ld_in(p.x, ((long long)g * p.m + i0 + u) * p.n + j0 + w, p.f32) * f);
      tile[u][w] = v;
    } else {   // the caller's row is a workspace column
      if (j0 + u < p.k && i0 + w < p.r)
        v = (float)((double)ld_in(p.x, ((long long)g * p.m + j0 + u) * p.n + i0 + w, p.f32) * f);
      tile[w][u] = v;
    }
  }
  __syncthreads();
  const bool diag = tr == tc;
  const long long part = (long long)p.batch * p.R * p.ld;
  auto store8 = [&](int i, int j, const float (&v)[8]) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 a = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
      const __half2 b = __floats2half2_rn(v[2 * q] - __low2float(a), v[2 * q + 1] - __high2float(a));
      h[q] = *reinterpret_cast<const uint32_t*>(&a);
      l[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __half* at = p.out + ((long long)g * p.R + i) * p.ld + j;
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at + part) = make_uint4(l[0], l[1], l[2], l[3]);
  };
#pragma unroll
  for (int e = tid; e < 512; e += 256) {
    const int u = e >> 3, w = (e & 7) * 8;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = tile[u][w + q];
      if (p.form == (int)Form::Skew && diag && u > w + q) v[q] = -tile[w + q][u];
    }
    store8(i0 + u, j0 + w, v);   // R and ld are multiples of 64
    if (p.form == (int)Form::Skew && !diag) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = -tile[w + q][u];
      store8(j0 + u, i0 + w, v);
    }
  }
}

// ------------------------------------------------------------------ host side
// fp16 stack [mats][rows][cols], box {bx, by, 1}
bool make_map3(CUtensorMap* m, const void* base, int64_t mats, int64_t rows, int64_t cols, int bx,
               int by, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)mats};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(rows * cols) * 2};
  cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A workspace stack and the ways the products address it.
struct Stack {
  __half* base = nullptr;
  int64_t rows = 0, cols = 0;
  CUtensorMap k, mn, st, mir;   // K-major operand, N-major operand, store, mirrored store
  bool init(__half* b, int64_t mats, int64_t r, int64_t c) {
    base = b; rows = r; cols = c;
    constexpr CUtensorMapSwizzle k128 = CU_TENSOR_MAP_SWIZZLE_128B, k64 = CU_TENSOR_MAP_SWIZZLE_64B;
    return make_map3(&k, b, mats, r, c, 64, 128, k128) &&
           make_map3(&mn, b, mats, r, c, 64, 64, k128) &&
           make_map3(&st, b, mats, r, c, 64, 32, k128) &&
           make_map3(&mir, b, mats, r, c, 32, 64, k64);
  }
};

struct Dims {
  int64_t r, k, R, ld;
  bool tall;
  int64_t elems;    // values of one matrix in the caller's array
  int chunks;
};
Dims dims_of(const Problem& p) {
  Dims d;
  d.tall = p.form == Form::Dense && p.m > p.n;
  d.r = std::min(p.m, p.n);
  d.k = std::max(p.m, p.n);
  d.R = (d.r + 63) / 64 * 64;
  d.ld = (d.k + 63) / 64 * 64;
  d.elems = p.form == Form::Skew ? p.m * (p.m - 1) / 2 : p.m * p.n;
  d.chunks = norm_chunks(d.elems);
  return d;
}

struct Ws {
  double* partial;
  __half *x[2], *a, *h, *b;
};
size_t layout(const Problem& p, void* base, Ws* o) {
  const Dims d = dims_of(p);
  Arena ar(base, SIZE_MAX);
  Ws w;
  w.partial = static_cast<double*>(ar.take((size_t)p.batch * d.chunks * sizeof(double)));
  const size_t xb = (size_t)(2 * p.batch * d.R * d.ld) * 2;
  const size_t gb = (size_t)(2 * p.batch * d.R * d.R) * 2;
  w.x[0] = static_cast<__half*>(ar.take(xb));
  w.x[1] = p.steps > 1 ? static_cast<__half*>(ar.take(xb)) : nullptr;
  w.a = static_cast<__half*>(ar.take(gb));
  w.h = static_cast<__half*>(ar.take(gb));
  w.b = static_cast<__half*>(ar.take(gb));
  if (o) *o = w;
  return ar.used;
}

int sm_total() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

template <int CG, bool B_MN>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const Stack* o0, const Stack* o1,
                   const Prod& p, int sms, const char* name, cudaStream_t s) {
  auto kern = ns_product_kernel<CG, B_MN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  // setmaxnreg waits for registers that the block was not launched with: refuse such a build
  static const int regs = [kern] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  set_pdl_attr(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(CG * std::min(p.total, sms / CG)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  TraceScope t(name, s);
  const CUtensorMap& s0 = o0 ? o0->st : a;
  const CUtensorMap& m0 = o0 ? o0->mir : a;
  return cudaLaunchKernelEx(&cfg, kern, a, b, s0, o1 ? o1->st : s0, m0, o1 ? o1->mir : m0, p);
}

}  // namespace

// ------------------------------------------------------------------ scales
namespace {
constexpr double kTop = 32768.0;   // largest scaled magnitude, half of fp16's range
// the power of two that brings values of at most `most` to at most kTop
float pow2_scale(double most) {
  const int e = (int)std::floor(std::log2(kTop / std::max(most, 1e-30)));
  return (float)std::ldexp(1.0, std::max(-100, std::min(15, e)));
}
}  // namespace

bool make_plan(const float* coeffs, int steps, Plan* plan) {
  constexpr int kSamples = 4096;
  double top = 1.0;   // the singular values of X lie in [0, top]
  for (int t = 0; t < steps; ++t) {
    const double a = coeffs[3 * t], b = coeffs[3 * t + 1], c = coeffs[3 * t + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    double h = 0.0, bb = 0.0, x = 0.0;
    for (int i = 0; i <= kSamples; ++i) {
      const double s = top * i / kSamples, l = s * s;
      h = std::max(h, std::fabs(b + c * l));
      bb = std::max(bb, std::fabs(a + b * l + c * l * l));
      x = std::max(x, s * std::fabs(a + b * l + c * l * l));
    }
    // entries of a matrix do not pass its spectral norm; 2 % for the samples and the rounding
    plan->sx[t] = pow2_scale(1.02 * top);
    plan->sa[t] = pow2_scale(1.02 * top * top);
    plan->sh[t] = pow2_scale(1.02 * h);
    plan->sb[t] = pow2_scale(1.02 * bb);
    top = 1.02 * x;
    if (!(top < 1e6) || !(h < 1e12) || !(bb < 1e12)) return false;
  }
  plan->sx[steps] = 1.f;
  return true;
}

size_t workspace_bytes(const Problem& p) { return layout(p, nullptr, nullptr); }

cudaError_t run(const Problem& p, const Plan& plan, const void* x, void* out, void* ws,
                cudaStream_t s) {
  const Dims d = dims_of(p);
  Ws w;
  layout(p, ws, &w);
  int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  const bool skew = p.form == Form::Skew;
  const bool exact = p.out_t == DT::F32;
  const int in_f32 = p.in_t == DT::F32;
  {
    TraceScope t("ns_norm", s);
    cudaError_t e = launch_k(ns_norm_kernel, dim3((unsigned)d.chunks, (unsigned)p.batch),
                             dim3(kNormThreads), 0, s, x, in_f32, (long long)d.elems, d.chunks,
                             w.partial);
    if (e != cudaSuccess) return e;
  }
  {
    Prep q;
    q.x = x; q.f32 = in_f32; q.form = (int)p.form; q.tall = d.tall; q.chunks = d.chunks;
    q.batch = (int)p.batch; q.tiles_c = (int)(d.ld / 64);
    q.m = p.m; q.n = p.n;
    q.r = (int)d.r; q.k = (int)d.k; q.R = (int)d.R; q.ld = (int)d.ld;
    q.eps = p.eps; q.sx = plan.sx[0]; q.norm_mult = skew ? 2.0 : 1.0;
    q.partial = w.partial; q.out = w.x[0];
    TraceScope t("ns_prep", s);
    cudaError_t e = launch_k(ns_prep_kernel, dim3((unsigned)(d.R / 64 * (d.ld / 64)), (unsigned)p.batch),
                             dim3(256), 0, s, q);
    if (e != cudaSuccess) return e;
  }
  Stack X[2], A, H, B;
  const int64_t mats = 2 * p.batch;
  if (!X[0].init(w.x[0], mats, d.R, d.ld) || (w.x[1] && !X[1].init(w.x[1], mats, d.R, d.ld)) ||
      !A.init(w.a, mats, d.R, d.R) || !H.init(w.h, mats, d.R, d.R) || !B.init(w.b, mats, d.R, d.R))
    return cudaErrorInvalidValue;

  const int sms = sm_total();
  // 256-wide pair tiles need half the operand traffic per product of 128-wide ones, which
  // fill the GPU with a quarter of the work
  auto tiles = [&](int64_t rows, int64_t cols, int tile, bool sym) {
    const int64_t tm = (rows + tile - 1) / tile, tn = (cols + tile - 1) / tile;
    return (sym ? tm * (tm + 1) / 2 : tm * tn) * p.batch;
  };
  auto product = [&](const CUtensorMap& a, const CUtensorMap& b, bool b_mn, int64_t cols, int64_t K,
                     bool sym, Prod q, const Stack* o0, const Stack* o1, const char* name) {
    const int64_t rows = d.R;
    const bool pair = tiles(rows, cols, 256, sym) >= sms / 4 && rows > 128;
    const int tile = pair ? 256 : 128;
    q.batch = (int)p.batch;
    q.tiles_m = (int)((rows + tile - 1) / tile);
    q.tiles_n = (int)((cols + tile - 1) / tile);
    q.sym = sym;
    q.per = (int)(tiles(rows, cols, tile, sym) / p.batch);
    q.total = (int)tiles(rows, cols, tile, sym);
    q.rows = (int)rows; q.cols = (int)cols;
    q.nk = (int)(K / BK);
    // the small products and the first of the large ones in one accumulator
    q.head = exact ? (q.nseg - 1) * q.nk + std::min(kChunk, q.nk) : q.nk * q.nseg;
    q.chunk = kChunk;
    q.err = err;
    if (b_mn)
      return pair ? launch<2, true>(a, b, o0, o1, q, sms, name, s)
                  : launch<1, true>(a, b, o0, o1, q, sms, name, s);
    return pair ? launch<2, false>(a, b, o0, o1, q, sms, name, s)
                : launch<1, false>(a, b, o0, o1, q, sms, name, s);
  };
  auto segments = [](Prod& q, int n) {
    // hi hi | hi lo, hi hi | lo hi, hi lo, hi hi: small products first
    q.nseg = n;
    const int pa[3] = {1, 0, 0}, pb[3] = {0, 1, 0};
    for (int i = 0; i < n; ++i) { q.pa[i] = pa[3 - n + i]; q.pb[i] = pb[3 - n + i]; }
  };

  for (int t = 0; t < p.steps; ++t) {
    const float* c = p.coeffs + 3 * t;
    const bool last = t + 1 == p.steps;
    const double sx = plan.sx[t], sa = plan.sa[t], sh = plan.sh[t], sb = plan.sb[t];
    const Stack& Xt = X[t & 1];
    Prod q{};
    segments(q, exact ? 3 : 1);
    q.lo = exact; q.mirror = 1.f; q.has1 = 1;
    q.f0 = (float)(sa / (sx * sx)); q.d0 = 0.f;
    q.f1 = (float)(sh * c[2] / (sx * sx)); q.d1 = (float)(sh * c[1]);
    cudaError_t e = product(Xt.k, Xt.k, false, d.R, d.ld, true, q, &A, &H, "ns_gram");
    if (e != cudaSuccess) return e;

    q.has1 = 0;
    q.f0 = (float)(sb / (sa * sh)); q.d0 = (float)(sb * c[0]);
    e = product(A.k, H.k, false, d.R, d.R, true, q, &B, nullptr, "ns_square");
    if (e != cudaSuccess) return e;

    q.d0 = 0.f;
    segments(q, exact ? 3 : (last ? 1 : 2));
    if (!last) {
      q.f0 = (float)(plan.sx[t + 1] / (sb * sx));
      q.lo = exact || t + 2 < p.steps;   // the last bf16 update reads one part
      q.mirror = -1.f;
      const Stack& Xn = X[(t + 1) & 1];
      e = product(B.k, Xt.mn, true, d.ld, d.R, skew, q, &Xn, nullptr, "ns_update");
    } else {
      q.f0 = (float)(p.scale / (sb * sx));
      q.fmode = skew ? kPacked : d.tall ? kTransposed : kRows;
      q.out = out; q.out_f32 = exact;
      q.um = d.r; q.un = d.k;
      q.vec = (d.k * (exact ? 4 : 2)) % 16 == 0;
      e = product(B.k, Xt.mn, true, d.ld, d.R, skew, q, nullptr, nullptr, "ns_update_out");
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace orth
}  // namespace poetx
