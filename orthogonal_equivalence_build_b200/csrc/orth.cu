// Newton-Schulz orthogonalisation of a stack of matrices on the tensor cores (tcgen05 / TMEM /
// TMA, sm_100a).
//
//   X_0 = X / (|X|_F + eps);   X_{t+1} = a_t X_t + (b_t A + c_t A^2) X_t,  A = X_t X_t^T
//
// with X laid out so that it has no more rows r than columns k (a taller input is transposed on
// its way in and back on its way out: X (X^T X) = (X X^T) X). Per step three products:
//   gram    A = X X^T                                  (symmetric)
//   square  B = a I + b A + c A A                      (symmetric; the epilogue reads A's tile)
//   update  X <- B X                                   (skew for skew X)
// a X rides on B's diagonal. Symmetric (and skew) results may be computed on the tiles on and above
// the diagonal only; the epilogue then stores every other tile twice, the second time
// transposed (and negated).
//
// All steps of all matrices run in one launch. Its tiles, in the order step, product, matrix,
// tile, are handed out one by one from a counter to the clusters that run; a tile's operands are
// loaded once the product before it is complete for its matrix (a count per matrix, raised by
// the epilogue warps after their stores). Every tile that a cluster waits for was handed out
// earlier, to a cluster that runs, so the waits end whatever else shares the GPU. Fifteen launches
// would pay for a ramp, a partial wave of tiles and a drain each: at 36 blocks of 512 two thirds
// of their time.
//
// Precision. Operands are fp16 parts of scaled values with fp32 accumulation: x = hi + lo,
// hi = fp16(x), lo = fp16(x - hi), which carries 22 bits. The scales are powers of two chosen
// from the range of the singular values after each step (X_0 has them in [0, 1]; the quintic's range
// over an interval is known), so nothing overflows and the smallest entries that matter stay
// normal numbers. A matrix whose norm is below eps has a smaller interval and scales of its own, which
// ns_prep_kernel finds; so every matrix has its row of factors in the workspace.
//   fp32 results, and bf16 results of up to 128 rows: every product is hi hi + hi lo + lo hi (three
//     passes over K), error a few 2^-22 of the result's size.
//   other bf16 results: one pass for gram and square; the update of every step but the last reads X
//     in both parts (two passes). X's rounding is what the iteration amplifies: a direction whose
//     singular value is 1e-3 of the largest is drowned by 2^-11 of the large ones, and it
//     is lifted by a = 3.4 a step while they stay. The rounding of A, H and B acts on the
//     directions in proportion and is not amplified. Against the exact result, in units of its
//     rms: 1.4e-3 for an update of a few strong directions over a background (single-part X
//     2.0e-3, and 9.5e-3 with a background of 3 % of the strongest); bf16 rounding alone is
//     1.7e-3. That is an average over the directions, each of which the roundings may move by up to
//     2e-2: 1.1e-3 of Gaussian matrices of 128 rows and more, but 1.7e-3 of 64 rows and 6e-3 of
//     two; 8e-3 of more rows where all singular values coincide, and 1e-2 where but a few rows are not
//     zero. No single rounding makes it (with X, A or B alone in two parts 1.2e-2 to 2.2e-2 are left of
//     2e-2); three passes for every size would be free of it and take 1.3 (200 x 300) to 2.2 times
//     as long (4096 x 14336 11.0 ms against 5.1 ms); up to 128 rows they take 1.2 to 1.3 times (64 x
//     300 104 us against 82).
#include "orth_mma.cuh"

#include <algorithm>
#include <cmath>

namespace poetx {
namespace orth {
namespace {

constexpr int BK = 64;
constexpr int kEpiWarps = 8;               // two per TMEM lane quarter, half of the columns each
constexpr int kThreads = 128 + 32 * kEpiWarps;
// Registers per thread at launch, then of warps 0..3 (which only issue copies and MMAs) and of the
// epilogue's: setmaxnreg moves them within what the block was launched with.
constexpr int kRegsLaunch = 168, kRegsIssue = 56, kRegsEpi = 224;
static_assert(128 * kRegsIssue + 32 * kEpiWarps * kRegsEpi <= kThreads * kRegsLaunch,
              "the register split must fit the launch's registers");
constexpr int kPiece = 4096;               // 32 rows x 64 columns of fp16
constexpr int kEpiStage = 2 * kPiece;      // per epilogue warp
// Tile numbers handed from the producer to the others. The producer is at most two tiles (the
// accumulators) and a ring of one-block tiles ahead of the epilogue, so that no slot's barriers
// pass two phases while a role still waits for the first.
constexpr int kSlots = 8;

// ------------------------------------------------------------------ the work
// Tile shapes. CG = 1: 128 x 128 tiles of one CTA; CG = 2: 256 x 256 tiles of a CTA pair
// (cta_group::2: each CTA holds 128 rows of A, half of B's columns and 128 rows of the result).
// TN = 64: 128 x 64 tiles of one CTA, whose epilogue is the first four warps' alone.
template <int CG_, int TN_>
struct Shape {
  static constexpr int CG = CG_, TM = 128 * CG_, TN = TN_;
  static constexpr int BN = TN / CG;                    // columns of B that a CTA loads
  static constexpr int EPI = TN >= 128 ? kEpiWarps : 4; // epilogue warps
  static constexpr int COLS = TN * 4 / EPI;             // result columns of each
};
constexpr int kOperand = 128 * BK * 2;     // bytes of a CTA's rows of A, and at most of its columns of B
// (three stages are enough while X fits L2, and cost 15 % where it does not)
constexpr int STAGES = 5;
constexpr size_t kSmem = (size_t)STAGES * 2 * kOperand + kEpiWarps * kEpiStage + 1024 + 512;

struct Kind {
  int tiles_m, tiles_n, per;   // tile grid of a matrix; tiles computed
  int sym, cols, nk;           // sym: on and above the diagonal; padded columns; K blocks a segment
};
struct Job {
  Kind k[3];
  int batch, steps, per_step, total;   // tiles per step (all matrices) and in all
  int R;                               // padded rows of every result
  int exact, chunk;                    // three part products; then K blocks per accumulator
  int fmode, out_f32, vec;             // the caller's array: layout, type, rows start on 16 bytes
  void* out;
  const float* factors;                // per matrix: Factors of every step, then Plan::out
  long long um, un;                    // its rows and columns (of the result as computed)
  int *counter, *done, *err;           // tiles handed out; per matrix: epilogue warps finished
};
struct Maps {
  CUtensorMap xk[2], xr[2], xn[2];   // X: left operand, right operand read K- and N-major,
  CUtensorMap xs[2], xm[2];   //    pieces as computed and mirrored
  CUtensorMap ak, ar, as, am; // A: left and right operand, pieces
  CUtensorMap bk, bs, bm;     // B: left operand, pieces
};

static_assert(sizeof(Factors) == 5 * sizeof(float), "the epilogue indexes them as floats");
// floats of a matrix's row; the same for every number of steps, and so is the workspace's size beyond one
constexpr int kFactors = 5 * kMaxSteps + 1;

struct Work {
  int t, kind, g, mb, nb;
  bool last;
};
// Tile numbers count through step, product, matrix, tile. Symmetric results: row by row over the
// tiles on and above the diagonal. Others: bands of 16 row tiles sweep the columns, so a band
// of the left operand stays in L2 while X streams.
__device__ __forceinline__ Work decode(const Job& j, int tile) {
  Work w;
  w.t = tile / j.per_step;
  w.last = w.t + 1 == j.steps;
  int l = tile - w.t * j.per_step;
  w.kind = kGram;
  while (w.kind < kUpdate && l >= j.batch * j.k[w.kind].per) l -= j.batch * j.k[w.kind++].per;
  const Kind& k = j.k[w.kind];
  w.g = l / k.per;
  l -= w.g * k.per;
  if (k.sym) {
    int i = 0;
    while (l >= k.tiles_n - i) l -= k.tiles_n - i++;
    w.mb = i;
    w.nb = i + l;
  } else {
    const int band = l / (16 * k.tiles_n), first = band * 16;
    const int gm = min(16, k.tiles_m - first), r = l - band * 16 * k.tiles_n;
    w.mb = first + r % gm;
    w.nb = r / gm;
  }
  return w;
}
// Part products of a tile: hi hi | hi lo, hi hi | lo hi, hi lo, hi hi, the small ones first.
__device__ __forceinline__ int segments(const Job& j, const Work& w) {
  return j.exact ? 3 : w.kind == kUpdate && !w.last ? 2 : 1;
}
__device__ __forceinline__ int part_a(int n, int seg) { return n == 3 && seg == 0; }
__device__ __forceinline__ int part_b(int n, int seg) { return n > 1 && seg == n - 2; }
// K blocks that the first accumulator of a tile sums: the small products and the first job.chunk of
// the large one with three part products, everything otherwise
__device__ __forceinline__ int head_blocks(const Job& j, int n, int nk) {
  return j.exact ? (n - 1) * nk + min(j.chunk, nk) : n * nk;
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

// kind::f16, fp16 operands, fp32 accumulator, TM x TN tile; bit 16: B is N-major
template <typename S>
__device__ __forceinline__ constexpr uint32_t idesc() {
  return (1u << 4) | ((uint32_t)(S::TN >> 3) << 17) | ((uint32_t)(S::TM >> 4) << 24);
}

// until *cnt >= target
__device__ __forceinline__ bool wait_done(const int* cnt, int target, Ctl c) {
  if (ld_acquire_gpu(cnt) >= target) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    __nanosleep(64);
    if (ld_acquire_gpu(cnt) >= target) return true;
    if ((it & 15) == 0) {
      if (*c.abort) return false;
      if (global_ns() - t0 > kLimitNs) {
        *c.abort = 1;
        atomicCAS(c.err, 0, (int)kErrDependency);
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

// One 32-row x 64-column piece of a warp to the fp16 maps, in one or two parts, and the mirrored
// piece of an off-diagonal tile. The value of element (i, j) is v f + (i == j) d. The parts are
// packed into the halves of the warp's stage in the 128-byte swizzle (16-byte unit u of row i at
// u ^ (i & 7)) and copied out together. For the mirror each half is then transposed in place, in 8 x 8
// blocks through registers, into the 64-byte swizzle (unit u of row j at u ^ (j / 2 & 3)): no bank
// conflicts either way. (Plain 16-byte stores instead of the copies: the same time where many tiles
// hide it, 15 to 30 % more where a product waits for the one before, which then waits for the
// stores' fence.)
__device__ __forceinline__ void emit_maps(const CUtensorMap* out, const CUtensorMap* mir,
                                          const float* v, float f, float d, int parts, int batch,
                                          int g, int row0, int col0, bool mirror, uint32_t flip,
                                          uint32_t stage, int lane) {
  if (lane == 0) bulk_wait_read<0>();   // the copies of the piece before have read the stage
  __syncwarp();
#pragma unroll 1
  for (int part = 0; part < parts; ++part) {
    int dq = row0 + lane - col0;        // the diagonal's column of this row's 64
    asm volatile("" : "+r"(dq));        // (not 64 comparisons kept over the parts)
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
        h[q] = *reinterpret_cast<const uint32_t*>(&w);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                       stage + part * kPiece + lane * 128 + ((u ^ (lane & 7)) << 4)),
                   "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    for (int part = 0; part < parts; ++part)
      store_box(out, stage + part * kPiece, col0, row0, part * batch + g);
    bulk_commit();
  }
  if (!mirror) return;
  // lane l names row l of the piece's 32 for the load, and for the store row l % 8 of the unit's
  // eight in 16-byte unit l / 8
  const int blk = lane >> 3, jj = lane & 7;
#pragma unroll 1
  for (int part = 0; part < parts; ++part) {
    const uint32_t half = stage + part * kPiece;
    uint32_t r[8][4];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      ldmatrix4_trans(half + lane * 128 + ((u ^ (lane & 7)) << 4), r[u]);
#pragma unroll
      for (int q = 0; q < 4; ++q) r[u][q] ^= flip;
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u)
      stmatrix4(half + (8 * u + jj) * 64 + ((blk ^ ((jj >> 1) & 3)) << 4), r[u]);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    for (int part = 0; part < parts; ++part)
      store_box(mir, stage + part * kPiece, row0, col0, part * batch + g);
    bulk_commit();
  }
}

// The same piece to the caller's array: v f out_scale.
__device__ __forceinline__ void emit_user(const Job& p, const float* v, float f, float out_scale, int g,
                                          int row0, int col0, uint8_t* stage, int lane) {
  if (p.fmode == kTransposed) {
    // 32 rows of the piece are 32 neighbours of one output row
    const int i = row0 + lane, left = (int)min((long long)64, p.un - col0);
    if (i < p.um) {
      const long long at = ((long long)g * p.un + col0) * p.um + i;
      if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int q = 0; q < 64; ++q, o += p.um)
          if (q < left) *o = v[q] * f * out_scale;
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
        for (int q = 0; q < 64; ++q, o += p.um)
          if (q < left) *o = __float2bfloat16_rn(v[q] * f * out_scale);
      }
    }
    return;
  }
  // through the stage: row r in 256 bytes, 16-byte unit u at u ^ (r & 15)
#pragma unroll
  for (int u = 0; u < 16; ++u)
    *reinterpret_cast<float4*>(stage + lane * 256 + ((u ^ (lane & 15)) << 4)) =
        make_float4(v[4 * u] * f * out_scale, v[4 * u + 1] * f * out_scale,
                    v[4 * u + 2] * f * out_scale, v[4 * u + 3] * f * out_scale);
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

// Persistent and warp-specialised. Warp 0 of the leader (rank 0) takes tile numbers from the counter
// and hands them to the other roles through kSlots slots; warp 0 of every CTA streams operand
// tiles by TMA through a ring of stages; one lane of the leader's warp 1 issues the MMAs into one
// of two accumulators; warps 4..11 empty the other one (warps 2 and 3 complete the first register
// group).
// The tensor core adds to its fp32 accumulator without rounding to nearest: every 16-deep step
// loses up to a whole unit in the last place, always towards zero, and K = 2048 in three
// passes came out 3.8e-5 off. So the parts' small products (hi lo, lo hi) come first, and for fp32
// results an accumulator of large products sums only job.chunk K blocks; the epilogue warps add the
// accumulators in registers (round to nearest) while the next one fills.
// Every wait is bounded; on expiry the device error word is set, the roles leave their loops,
// copies and MMAs in flight are waited for (bounded) and TMEM is freed.
template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
ns_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Job job) {
  constexpr int CG = S::CG, TN = S::TN;
  constexpr uint32_t TMEM_COLS = 2 * TN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sa = smem;
  uint8_t* sb = smem + STAGES * kOperand;
  uint8_t* sepi = sb + STAGES * kOperand;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sepi + kEpiWarps * kEpiStage);
  uint64_t* full = bars;                     // [STAGES], leader only
  uint64_t* empty = full + STAGES;           // [STAGES]
  uint64_t* tfull = empty + STAGES;          // [2]
  uint64_t* tempty = tfull + 2;              // [2], leader only
  uint64_t* wfull = tempty + 2;              // [kSlots]: a tile number is in its slot
  uint64_t* wempty = wfull + kSlots;         // [kSlots], leader only: every role has read it
  uint64_t* wready = wempty + kSlots;        // [kSlots]: the product before the tile's is complete
  uint64_t* aload = wready + kSlots;         // [kEpiWarps]: a warp's tile of A
  uint64_t* drain = aload + kEpiWarps;
  volatile int* wtile = reinterpret_cast<volatile int*>(drain + 1);   // [kSlots]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1) + kSlots;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // known to be uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const Ctl ctl{abort_flag, job.err};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(tfull + a), 1);
      mbar_init(smem_u32(tempty + a), S::EPI * CG);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(wfull + s), 1);
      mbar_init(smem_u32(wready + s), 1);
      // the MMA lane, the other CTA's producer, every epilogue warp
      mbar_init(smem_u32(wempty + s), CG + S::EPI * CG);
    }
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(aload + i), 1);
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

  // Next tile number for a role (a converged warp) other than the leader's producer; job.total or
  // more: there are no more. n counts the role's tiles.
  auto take = [&](int n, int& tile) {
    const int s = n % kSlots;
    const uint32_t ph = (uint32_t)(n / kSlots) & 1u;
    const bool ok = wait_inline<CG == 2>(smem_u32(wfull + s), ph, ctl, kErrEpilogue);
    tile = __shfl_sync(0xffffffffu, wtile[s], 0);
    if (!__all_sync(0xffffffffu, ok)) return false;
    if (elect_one()) {
      if constexpr (CG == 2) mbar_arrive_remote(map_to_rank(smem_u32(wempty + s), 0));
      else mbar_arrive(smem_u32(wempty + s));
    }
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0) {
      // ------------------------------------------------------------ tile numbers, TMA producer
      int it = 0, s = 0;        // K blocks issued; ring stage and its phase
      uint32_t ph = 1u;
      bool ok = true;
      uint32_t fb0 = smem_u32(full);
      if constexpr (CG == 2) fb0 = map_to_rank(fb0, 0);
      for (int n = 0; ok; ++n) {
        int tile = 0;
        if (leader) {
          // taken when it can be started, not earlier: a number held back by a busy cluster is work
          // that an idle one does not get
          if (lane == 0) tile = atomicAdd(job.counter, 1);
          tile = __shfl_sync(0xffffffffu, tile, 0);
          const int w = n % kSlots;
          ok = wait_inline<CG == 2>(smem_u32(wempty + w), ((uint32_t)(n / kSlots) & 1u) ^ 1u, ctl,
                                    kErrProducer);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (elect_one()) {
            wtile[w] = tile;
            mbar_arrive(smem_u32(wfull + w));
            if constexpr (CG == 2) {
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(
                               smem_u32(const_cast<int*>(wtile) + w), 1)),
                           "r"(tile)
                           : "memory");
              mbar_arrive_remote(map_to_rank(smem_u32(wfull + w), 1));
            }
          }
        } else if (!(ok = take(n, tile))) {
          break;
        }
        if (tile >= job.total) break;
        const Work w = decode(job, tile);
        const Kind& k = job.k[w.kind];
        const int before = w.t * (job.k[0].per + job.k[1].per + job.k[2].per) +
                           (w.kind > 0 ? job.k[0].per : 0) + (w.kind > 1 ? job.k[1].per : 0);
        if (before > 0) {
          // the product before this one is complete for this matrix; then order the loads of the
          // asynchronous proxy behind that
          if (lane == 0) ok = wait_done(job.done + w.g, before * S::EPI * CG, ctl);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          __syncwarp();
          asm volatile("fence.proxy.async.global;" ::: "memory");
        }
        if (elect_one()) mbar_arrive(smem_u32(wready + n % kSlots));
        const int x = w.t & 1;
        const CUtensorMap* ma =
            w.kind == kGram ? &maps.xk[x] : w.kind == kSquare ? &maps.ak : &maps.bk;
        const CUtensorMap* mb =
            w.kind == kGram ? &maps.xr[x] : w.kind == kSquare ? &maps.ar : &maps.xn[x];
        const int am = w.mb * S::TM + (int)rank * 128, bn = w.nb * TN + (int)rank * S::BN;
        const int ns = segments(job, w);
        for (int seg = 0; ok && seg < ns; ++seg) {
          const int za = part_a(ns, seg) * job.batch + w.g, zb = part_b(ns, seg) * job.batch + w.g;
          for (int kk = 0; kk < k.nk * BK; kk += BK, ++it) {
            // stops only when the wait runs out: both CTAs of a pair are released by the same
            // commits, so both have then issued the same loads
            ok = wait_inline(smem_u32(empty + s), ph, ctl, kErrProducer, kLimitNs,
                             /*stop_on_abort=*/false);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const uint32_t fb = fb0 + (uint32_t)(s * 8);
            const uint32_t da = smem_u32(sa) + (uint32_t)(s * kOperand);
            const uint32_t db = smem_u32(sb) + (uint32_t)(s * kOperand);
            if (elect_one()) {
              if (leader) mbar_expect_tx(smem_u32(full + s), CG * (kOperand + S::BN * BK * 2));
              load_box<CG>(da, ma, fb, kk, am, za);
              if (w.kind == kUpdate) {
                load_box<CG>(db, mb, fb, bn, kk, zb);
                if constexpr (S::BN == 128) load_box<CG>(db + 64 * BK * 2, mb, fb, bn + 64, kk, zb);
              } else {
                load_box<CG>(db, mb, fb, kk, bn, zb);
              }
            }
            if (++s == STAGES) { s = 0; ph ^= 1u; }
          }
        }
      }
      if (!ok && leader)   // let the copies already issued land before the CTA leaves
        for (int j = max(0, it - STAGES); j < it; ++j)
          wait_inline(smem_u32(full + j % STAGES), (uint32_t)(j / STAGES) & 1u, ctl, 0,
                      kDrainLimitNs, /*stop_on_abort=*/false);
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (leader) {
        auto commit = [](uint32_t bar) {
          if (elect_one()) {
            if constexpr (CG == 2) umma_commit_pair_both(bar);
            else umma_commit(bar);
          }
        };
        int s = 0, count = 0;   // ring stage, accumulators used
        uint32_t ph = 0u;
        bool ok = true;
        for (int n = 0; ok; ++n) {
          int tile;
          if (!(ok = take(n, tile)) || tile >= job.total) break;
          const Work w = decode(job, tile);
          const int ns = segments(job, w), nk1 = job.k[w.kind].nk, nk = ns * nk1;
          const bool mn = w.kind == kUpdate;
          const uint32_t id = idesc<S>() | (mn ? 1u << 16 : 0u);
          const uint32_t bstep = mn ? 2048u >> 4 : 32u >> 4;
          const uint32_t a_lo = desc_lo(smem_u32(sa), 16), b_lo = desc_lo(smem_u32(sb), mn ? 64 * BK * 2 : 16);
          for (int kb = 0, end = head_blocks(job, ns, nk1); ok && kb < nk;
               end = min(nk, end + job.chunk), ++count) {
            const int acc = count & 1;
            ok = wait_inline(smem_u32(tempty + acc), ((uint32_t)(count >> 1) & 1u) ^ 1u, ctl, kErrMma);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * TN);
            for (uint32_t more = 0u; kb < end; ++kb, more = 1u) {
              ok = wait_inline(smem_u32(full + s), ph, ctl, kErrMma);
              if (!(ok = __all_sync(0xffffffffu, ok))) break;
              tc_fence_after();
              const uint32_t a = a_lo + (uint32_t)s * (kOperand >> 4);
              const uint32_t b = b_lo + (uint32_t)s * (kOperand >> 4);
              if (elect_one()) {
                mma<CG>(d, a, b, id, more);
#pragma unroll
                for (int kk = 1; kk < BK / 16; ++kk) mma<CG>(d, a + 2 * kk, b + bstep * kk, id, 1u);
              }
              commit(smem_u32(empty + s));
              if (++s == STAGES) { s = 0; ph ^= 1u; }
            }
            if (ok) commit(smem_u32(tfull + acc));
          }
        }
        commit(smem_u32(drain));   // every MMA of this lane has retired once this completes
        wait_inline(smem_u32(drain), 0, ctl, ok ? kErrMma : 0, ok ? kLimitNs : kDrainLimitNs,
                    /*stop_on_abort=*/false);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 4..11)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    constexpr int COLS = S::COLS;         // this warp's columns of the tile
    const int quarter = warp & 3;         // TMEM lanes 32 quarter .. + 31
    const int cbase = ((warp - 4) >> 2) * COLS;
    uint8_t* stage = sepi + (warp - 4) * kEpiStage;
    uint32_t back = smem_u32(tempty);
    if constexpr (CG == 2) back = map_to_rank(back, 0);
    uint64_t* abar = aload + (warp - 4);
    uint32_t aphase = 0;
    int count = 0;
    bool ok = true, loading = false;   // (a tile of A is on its way into the stage)
    for (int n = 0; ok && warp - 4 < S::EPI; ++n) {
      int tile;
      if (!take(n, tile) || tile >= job.total) break;
      const Work w = decode(job, tile);
      const Kind& k = job.k[w.kind];
      const int ns = segments(job, w), nk = ns * k.nk, head = head_blocks(job, ns, k.nk);
      const int row0 = w.mb * S::TM + (int)rank * 128 + quarter * 32;
      const int base0 = w.nb * TN + cbase;
      // (asked for early: they arrive while the accumulators fill)
      const float* fac = job.factors + (long long)w.g * kFactors;
      const float f = fac[5 * w.t + w.kind], fa = fac[5 * w.t + 3], da = fac[5 * w.t + 4];
      const float scale = fac[5 * job.steps];
      // A's 64 columns from c on, for b A, into the stage (which the warp has finished with)
      auto load_a = [&](int c) {
        if (lane == 0) {
          asm volatile("fence.proxy.async;" ::: "memory");
          const int parts = job.exact ? 2 : 1;
          mbar_expect_tx(smem_u32(abar), parts * kPiece);
          for (int part = 0; part < parts; ++part)
            load_box<1>(smem_u32(stage) + part * kPiece, &maps.as, smem_u32(abar), base0 + c, row0,
                        part * job.batch + w.g);
        }
        loading = true;
      };
      if (w.kind == kSquare) {
        // requested before the accumulators are ready, once A is complete
        ok = wait_inline(smem_u32(wready + n % kSlots), (uint32_t)(n / kSlots) & 1u, ctl,
                         kErrDependency);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        load_a(0);
      }
      float v[COLS];
#pragma unroll
      for (int q = 0; q < COLS; ++q) v[q] = 0.f;
      for (int done = 0; done < nk; done = done ? done + job.chunk : head, ++count) {
        const int acc = count & 1;
        ok = wait_inline(smem_u32(tfull + acc), (uint32_t)(count >> 1) & 1u, ctl, kErrEpilogue);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t trow = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                              (uint32_t)(acc * TN + cbase);
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
      const bool out = w.kind == kUpdate && w.last;
      if (out) {
#pragma unroll
        for (int c = 0; c < COLS; c += 64) {
          // (nothing of a packed result lies below the diagonal)
          const int col0 = base0 + c;
          if (row0 < job.um && col0 < job.un && !(job.fmode == kPacked && col0 + 63 <= row0))
            emit_user(job, v + c, f, scale, w.g, row0, col0, stage, lane);
        }
        continue;
      }
      if (w.kind == kSquare) {
        // v <- v f + A fa
#pragma unroll
        for (int c = 0; c < COLS; c += 64) {
          if (c > 0) load_a(c);
          ok = wait_inline(smem_u32(abar), aphase, ctl, kErrDependency);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          aphase ^= 1u;
          loading = false;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint8_t* at = stage + lane * 128 + ((u ^ (lane & 7)) << 4);
            const uint4 h = *reinterpret_cast<const uint4*>(at);
            const uint4 l = job.exact ? *reinterpret_cast<const uint4*>(at + kPiece)
                                      : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 a2 = __half22float2(*reinterpret_cast<const __half2*>(&hw[q]));
              const float2 b2 = __half22float2(*reinterpret_cast<const __half2*>(&lw[q]));
              float* at2 = v + c + 8 * u + 2 * q;
              at2[0] = at2[0] * f + (a2.x + b2.x) * fa;
              at2[1] = at2[1] * f + (a2.y + b2.y) * fa;
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      const int x = ~w.t & 1;   // X_{t+1}'s buffer
      const CUtensorMap* to =
          w.kind == kGram ? &maps.as : w.kind == kSquare ? &maps.bs : &maps.xs[x];
      const CUtensorMap* to_mirror =
          w.kind == kGram ? &maps.am : w.kind == kSquare ? &maps.bm : &maps.xm[x];
      const bool mirror = k.sym && w.nb > w.mb;
      // bf16 results: the last update reads one part of X
      const int parts = job.exact || (w.kind == kUpdate && w.t + 2 < job.steps) ? 2 : 1;
#pragma unroll
      for (int c = 0; c < COLS; c += 64) {
        const int col0 = base0 + c;   // pieces wholly in the padding are not stored
        if (row0 < job.R && col0 < k.cols)
          emit_maps(to, to_mirror, v + c, w.kind == kSquare ? 1.f : f,
                    w.kind == kSquare ? da : 0.f, parts, job.batch, w.g, row0, col0, mirror,
                    w.kind == kUpdate ? 0x80008000u : 0u, smem_u32(stage), lane);
      }
      // publish: this warp's copies are complete, then the matrix's count goes up
      if (lane == 0) {
        bulk_wait_all();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        red_release_gpu_add(job.done + w.g, 1);
      }
      __syncwarp();
    }
    if (loading) wait_inline(smem_u32(abar), aphase, ctl, 0, kDrainLimitNs, /*stop_on_abort=*/false);
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
constexpr int64_t kNormChunk = 16384;   // elements per block of the norm pass, at least
constexpr int kMaxChunks = 512;

int norm_chunks(int64_t elems) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxChunks, elems / kNormChunk));
}

// partial[g][chunk] = sum of the chunk's squares, in 64 bits: an fp32 square overflows at 1.8e19
// and vanishes at 1e-23, both of which are ordinary fp32 and bf16 values. (Plain loads: a block may
// start before the kernel that writes x has ended.)
__global__ void __launch_bounds__(kNormThreads)
ns_norm_kernel(const void* x, int f32, int vec, long long elems, int chunks, double* partial,
               int* counts, int ncounts) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0)   // the products' counters start at zero
    for (int i = threadIdx.x; i < ncounts; i += kNormThreads) counts[i] = 0;
  const long long base = (long long)blockIdx.y * elems;
  const long long per = ((elems + chunks - 1) / chunks + 7) / 8 * 8;
  const long long lo = min(elems, per * blockIdx.x), hi = min(elems, lo + per);
  double s = 0.0;
  if (vec) {   // every matrix, and so every range, starts on 16 bytes
    if (f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + base);
#pragma unroll 4
      for (long long i = lo / 4 + threadIdx.x; i < hi / 4; i += kNormThreads) {
        const float4 v = p[i];
        s += (double)v.x * v.x + (double)v.y * v.y + (double)v.z * v.z + (double)v.w * v.w;
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + base);
#pragma unroll 4
      for (long long i = lo / 8 + threadIdx.x; i < hi / 8; i += kNormThreads) {
        const uint4 v = p[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const double a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xffff0000u);
          s += a * a + b * b;
        }
      }
    }
  } else {
    for (long long i = lo + threadIdx.x; i < hi; i += kNormThreads) {
      const double v = ld_in(x, base + i, f32);
      s += v * v;
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[(long long)blockIdx.y * chunks + blockIdx.x] = s;
}

// X_0 in two fp16 parts, [2][batch][R][ld], from the caller's array: eight values at a time where
// the caller's rows are the workspace's, else by 64 x 64 tiles through shared memory, so that reads
// follow the caller's rows and writes the workspace's. Padding is written as zeros.
struct Prep {
  const void* x;
  int f32, form, tall, vec, chunks, batch, tiles, tiles_c;
  long long m, n;            // the caller's matrix (Skew: m = n = b)
  int r, k, R, ld;           // the workspace's: r x k in R x ld
  double eps, norm_mult;     // norm^2 = norm_mult * sum of the partials
  const double* partial;
  __half* out;
  float* factors;            // per matrix, see Job
  int steps;
  float scale;
  float coeffs[3 * kMaxSteps];
  Plan plan;                 // of matrices whose norm is eps or more
};
__global__ void __launch_bounds__(256) ns_prep_kernel(const __grid_constant__ Prep p) {
  __shared__ float tile[64][65];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, tid = threadIdx.x;
  double s = 0.0;
  for (int c = tid; c < p.chunks; c += 256) s += p.partial[(long long)g * p.chunks + c];
  s = block_sum(s);
  const double norm = sqrt(p.norm_mult * s), sum = norm + p.eps;
  const bool below = below_eps(norm, p.eps);
  const double f = (below ? x0_scale(norm / sum) : p.plan.x0) / sum;
  if (blockIdx.x == 0) {
    float* fac = p.factors + (long long)g * kFactors;
    if (!below) {
      const float* all = reinterpret_cast<const float*>(p.plan.step);
      for (int i = tid; i < 5 * p.steps; i += 256) fac[i] = all[i];
      if (tid == 0) fac[5 * p.steps] = p.plan.out;
    } else if (tid == 0) {
      plan_from(norm / sum, p.coeffs, p.steps, p.scale, reinterpret_cast<Factors*>(fac),
                fac + 5 * p.steps);
    }
  }
  const long long part = (long long)p.batch * p.R * p.ld;
  auto store8 = [&](int i, int j, const float (&v)[8]) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 a = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
      const __half2 b =
          __floats2half2_rn(v[2 * q] - __low2float(a), v[2 * q + 1] - __high2float(a));
      h[q] = *reinterpret_cast<const uint32_t*>(&a);
      l[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __half* at = p.out + ((long long)g * p.R + i) * p.ld + j;
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at + part) = make_uint4(l[0], l[1], l[2], l[3]);
  };
  if (p.vec) {   // the caller's rows are the workspace's and start on 16 bytes
    const int per_row = p.ld / 8, total = p.R * per_row;
#pragma unroll 2
    for (int e = blockIdx.x * 256 + tid; e < total; e += gridDim.x * 256) {
      const int i = e / per_row, j = (e - i * per_row) * 8;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (i < p.r) {
        const long long at = ((long long)g * p.m + i) * p.n + j;
        if (p.f32) {
#pragma unroll
          for (int q = 0; q < 8; q += 4)
            if (j + q < p.k) {
              const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + at + q);
              v[q] = x.x; v[q + 1] = x.y; v[q + 2] = x.z; v[q + 3] = x.w;
            }
        } else if (j < p.k) {
          const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + at);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = (float)((double)v[q] * f);
      store8(i, j, v);
    }
    return;
  }
  for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
    const int tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
    if (p.form == (int)Form::Skew && tr > tc) continue;   // written by its mirror
    const int i0 = tr * 64, j0 = tc * 64;
    __syncthreads();   // the tile before has been stored
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

// Three part products, or fewer where a bf16 result's directions are many.
bool three_products(const Problem& p) {
  return p.out_t == DT::F32 || std::min(p.m, p.n) <= 128;
}

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
  int* counts;              // tiles handed out, then one count per matrix
  float* factors;
  __half *x[2], *a, *b;
};
size_t layout(const Problem& p, void* base, Ws* o) {
  const Dims d = dims_of(p);
  Arena ar(base, SIZE_MAX);
  Ws w;
  w.partial = static_cast<double*>(ar.take((size_t)p.batch * d.chunks * sizeof(double)));
  w.counts = static_cast<int*>(ar.take((size_t)(p.batch + 1) * sizeof(int)));
  w.factors = static_cast<float*>(
      ar.take((size_t)p.batch * kFactors * sizeof(float)));
  const size_t xb = (size_t)(2 * p.batch * d.R * d.ld) * 2;
  const size_t gb = (size_t)(2 * p.batch * d.R * d.R) * 2;
  w.x[0] = static_cast<__half*>(ar.take(xb));
  w.x[1] = p.steps > 1 ? static_cast<__half*>(ar.take(xb)) : nullptr;
  w.a = static_cast<__half*>(ar.take(gb));
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

Kind kind_of(int64_t rows, int64_t cols, int64_t K, int tm, int tn, bool sym) {
  Kind k;
  k.tiles_m = (int)((rows + tm - 1) / tm);
  k.tiles_n = (int)((cols + tn - 1) / tn);
  k.sym = sym;
  k.cols = (int)cols;
  k.nk = (int)(K / BK);
  k.per = sym ? k.tiles_n * (k.tiles_n + 1) / 2 : k.tiles_m * k.tiles_n;   // (sym: square)
  return k;
}

// Tile shape and use of symmetry of a problem.
struct Choice {
  int cg, tn;
  bool sym;
};
// The fastest of four by a model of one step: the work of all matrices shared out over the GPU, and
// one matrix's three products one after the other, each in whole waves of tiles; the longer of the
// two and a third of the other. Its figures (us) are a fit to 57 problems of 1 to 100 matrices of
// 60 to 4096 rows: the choice takes at most 9 % more than the best of the four, runs of one choice
// differing by half of that. Where each pays (256 x 256 symmetric, 128 x 128 symmetric, 128 x 128
// full, 128 x 64, us in one run): 4096 x 4096 bf16 1462, 1990, 2678, 4633; 100 blocks of 256 355, 307,
// 368, 516; 4096 x 1024 bf16 313, 260, 256, 310; 3 of 1000 x 333 fp32 306, 230, 215, 199. Never the
// fastest, and so not here: 256 x 256 full (36 blocks of 512 534, of 128 x 128 symmetric 464); 256 x
// 128 tiles of a pair (at most 3 % ahead of 128 x 128).
Choice choose(const Problem& p, const Dims& d, int sms) {
  const bool exact = three_products(p), skew = p.form == Form::Skew;
  Choice best{};
  double best_t = 1e30;
  for (const Choice c : {Choice{2, 256, true}, Choice{1, 128, true}, Choice{1, 128, false},
                         Choice{1, 64, false}}) {
    if (c.sym && d.R <= 128) continue;   // one row of tiles: nothing to mirror
    const int tm = 128 * c.cg, workers = sms / c.cg;
    // a K block with every SM busy and in a chain; a tile's way out per part, and what a product
    // takes besides from its last store to the next one's first load
    const double busy_us = c.cg == 2 ? 0.47 : c.tn == 128 ? 0.33 : 0.25;
    const double block_us = c.cg == 2 ? 0.28 : c.tn == 128 ? 0.17 : 0.11;
    const double part_us = c.cg == 2 ? 3.6 : 2.6, gap_us = c.cg == 2 ? 4.0 : 2.2;
    double work = 0.0, chain = 0.0;
    for (int kind = 0; kind < 3; ++kind) {
      const bool sym = c.sym && (kind < 2 || skew);
      const Kind k = kind_of(d.R, kind < 2 ? d.R : d.ld, kind == 0 ? d.ld : d.R, tm, c.tn, sym);
      const int blocks = k.nk * (exact ? 3 : kind == 2 ? 2 : 1);
      const double out =
          part_us * (exact || kind == 2 ? 2 : 1) * (sym && k.per > 1 ? 1.25 : 1.0);
      work += (double)p.batch * k.per * std::max(blocks * busy_us, out) / workers;
      chain += std::ceil((double)k.per / workers) * blocks * block_us + out + gap_us;
    }
    const double t = std::max(work, chain) + std::min(work, chain) / 3.0;
    if (t < best_t) { best_t = t; best = c; }
  }
  return best;
}

template <typename S>
cudaError_t launch(const Maps& maps, const Job& job, int sms, cudaStream_t s) {
  auto kern = ns_kernel<S>;
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
  attr[1].val.clusterDim.x = S::CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  // as many clusters as one product of all matrices has tiles, at most one CTA per SM
  int most = 0;
  for (const Kind& k : job.k) most = std::max(most, k.per * job.batch);
  cfg.gridDim = dim3((unsigned)(S::CG * std::min(most, sms / S::CG)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = S::CG == 2 ? 2 : 1;
  TraceScope t("ns_products", s);
  return cudaLaunchKernelEx(&cfg, kern, maps, job);
}

}  // namespace

bool make_plan(const Problem& p, Plan* plan) {
  plan->x0 = x0_scale(1.0);
  return plan_from(1.0, p.coeffs, p.steps, p.scale, plan->step, &plan->out);
}

size_t workspace_bytes(const Problem& p) {
  return small_fits(p) ? 0 : layout(p, nullptr, nullptr);
}

cudaError_t run(const Problem& p, const Plan& plan, const void* x, void* out, void* ws,
                cudaStream_t s) {
  if (small_fits(p)) return run_small(p, plan, x, out, s);
  const Dims d = dims_of(p);
  Ws w;
  layout(p, ws, &w);
  int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  const bool skew = p.form == Form::Skew;
  const bool exact = three_products(p), out_f32 = p.out_t == DT::F32;
  const int in_f32 = p.in_t == DT::F32;
  {
    TraceScope t("ns_norm", s);
    cudaError_t e = launch_k(ns_norm_kernel, dim3((unsigned)d.chunks, (unsigned)p.batch),
                             dim3(kNormThreads), 0, s, x, in_f32, d.elems % (in_f32 ? 4 : 8) == 0 ? 1 : 0,
                             (long long)d.elems, d.chunks,
                             w.partial, w.counts, (int)p.batch + 1);
    if (e != cudaSuccess) return e;
  }
  {
    Prep q;
    q.x = x; q.f32 = in_f32; q.form = (int)p.form; q.tall = d.tall; q.chunks = d.chunks;
    q.batch = (int)p.batch; q.tiles_c = (int)(d.ld / 64);
    q.tiles = (int)(d.R / 64 * (d.ld / 64));
    q.vec = !skew && !d.tall && p.n * (in_f32 ? 4 : 2) % 16 == 0;
    q.m = p.m; q.n = p.n;
    q.r = (int)d.r; q.k = (int)d.k; q.R = (int)d.R; q.ld = (int)d.ld;
    q.eps = p.eps; q.norm_mult = skew ? 2.0 : 1.0;
    q.partial = w.partial; q.out = w.x[0];
    q.factors = w.factors; q.steps = p.steps; q.scale = p.scale; q.plan = plan;
    std::copy(p.coeffs, p.coeffs + 3 * p.steps, q.coeffs);
    // few blocks per matrix when there are many, each summing the norm's partials once
    const int64_t blocks = std::min<int64_t>(q.tiles, std::max<int64_t>(8, 148 * 8 / p.batch));
    TraceScope t("ns_prep", s);
    cudaError_t e = launch_k(ns_prep_kernel, dim3((unsigned)blocks, (unsigned)p.batch),
                             dim3(256), 0, s, q);
    if (e != cudaSuccess) return e;
  }
  const int sms = sm_total();
  const Choice c = choose(p, d, sms);
  const int tm = 128 * c.cg, bn = c.tn / c.cg;

  Maps maps{};
  const int64_t mats = 2 * p.batch;
  constexpr CUtensorMapSwizzle k128 = CU_TENSOR_MAP_SWIZZLE_128B, k64 = CU_TENSOR_MAP_SWIZZLE_64B;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    if (!w.x[i]) continue;
    ok = ok && make_map3(&maps.xk[i], w.x[i], mats, d.R, d.ld, 64, 128, k128) &&
         make_map3(&maps.xr[i], w.x[i], mats, d.R, d.ld, 64, bn, k128) &&
         make_map3(&maps.xn[i], w.x[i], mats, d.R, d.ld, 64, 64, k128) &&
         make_map3(&maps.xs[i], w.x[i], mats, d.R, d.ld, 64, 32, k128) &&
         make_map3(&maps.xm[i], w.x[i], mats, d.R, d.ld, 32, 64, k64);
  }
  ok = ok && make_map3(&maps.ak, w.a, mats, d.R, d.R, 64, 128, k128) &&
       make_map3(&maps.ar, w.a, mats, d.R, d.R, 64, bn, k128) &&
       make_map3(&maps.as, w.a, mats, d.R, d.R, 64, 32, k128) &&
       make_map3(&maps.am, w.a, mats, d.R, d.R, 32, 64, k64) &&
       make_map3(&maps.bk, w.b, mats, d.R, d.R, 64, 128, k128) &&
       make_map3(&maps.bs, w.b, mats, d.R, d.R, 64, 32, k128) &&
       make_map3(&maps.bm, w.b, mats, d.R, d.R, 32, 64, k64);
  if (!ok) return cudaErrorInvalidValue;

  Job job{};
  job.k[kGram] = kind_of(d.R, d.R, d.ld, tm, c.tn, c.sym);
  job.k[kSquare] = kind_of(d.R, d.R, d.R, tm, c.tn, c.sym);
  job.k[kUpdate] = kind_of(d.R, d.ld, d.R, tm, c.tn, c.sym && skew);
  job.batch = (int)p.batch;
  job.steps = p.steps;
  int64_t per_step = 0;
  for (const Kind& k : job.k) per_step += (int64_t)k.per * p.batch;
  // a matrix's count rises by one per epilogue warp of a tile
  if (per_step * p.steps * (c.tn == 64 ? 4 : kEpiWarps * c.cg) > INT32_MAX)
    return cudaErrorInvalidValue;
  job.per_step = (int)per_step;
  job.total = job.per_step * p.steps;
  job.R = (int)d.R;
  job.exact = exact;
  // A truncated accumulator of 128 terms shrinks what is summed of one sign by 2^-18 or so. Of matrices
  // with many rows the result hardly feels it (640 x 2000: 0.9 times the error of fp32 products,
  // 2048 x 2048 0.5 times); with up to 512, whose spectrum is narrow, it was up to twice that error
  // (500 x 260), and 64 terms an accumulator bring it to 1.2 times for 6 to 11 % more time (200 ->
  // 213 us for 3 of 1000 x 333; 2048 x 2048 would take 620 -> 690 us).
  job.chunk = d.R <= 512 ? 1 : 2;
  job.fmode = skew ? kPacked : d.tall ? kTransposed : kRows;
  job.out = out;
  job.factors = w.factors;
  job.out_f32 = out_f32;
  job.um = d.r;
  job.un = d.k;
  job.vec = (d.k * (out_f32 ? 4 : 2)) % 16 == 0;
  job.counter = w.counts;
  job.done = w.counts + 1;
  job.err = err;
  if (c.cg == 2) return launch<Shape<2, 256>>(maps, job, sms, s);
  return c.tn == 128 ? launch<Shape<1, 128>>(maps, job, sms, s)
                     : launch<Shape<1, 64>>(maps, job, sms, s);
}

}  // namespace orth
}  // namespace poetx
