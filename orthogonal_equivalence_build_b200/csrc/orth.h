// Newton-Schulz orthogonalisation — interface of orth.cu.
#pragma once
#include "internal.h"

namespace poetx {
namespace orth {

constexpr int kMaxSteps = 64;

// Where the matrices come from and go to.
enum class Form : int {
  Dense = 0,   // batch x [m][n]
  Skew = 1,    // batch x packed strict upper triangles of b x b skew matrices (m = n = b)
};

struct Problem {
  Form form = Form::Dense;
  int64_t batch = 0, m = 0, n = 0;
  DT in_t = DT::F32, out_t = DT::F32;
  int steps = 0;
  const float* coeffs = nullptr;   // host, [steps][3]
  float eps = 0.f, scale = 1.f;
};

// How the epilogues of one step scale their accumulators: gram, square and update results are f[0..2]
// times the accumulator, square adds fa A + da I (operands as stored, scales included).
struct Factors {
  float f[3], fa, da;
};
// Powers of two that hold every operand of every step inside fp16 (see plan_from in orth_mma.cuh).
struct Plan {
  double x0;               // X_0 is stored times this
  Factors step[kMaxSteps]; // (the last update's f leaves the result itself, or 2^j times it)
  float out;               // the caller's scale, times 2^-j
};
// For matrices of a norm of eps and more. false: the coefficients are not finite or let the singular
// values grow past every bound
bool make_plan(const Problem& p, Plan* plan);

// One CTA per matrix (orth_small.cu), where a matrix fits into shared memory.
bool small_fits(const Problem& p);
cudaError_t run_small(const Problem& p, const Plan& plan, const void* x, void* out,
                      cudaStream_t s);

size_t workspace_bytes(const Problem& p);
cudaError_t run(const Problem& p, const Plan& plan, const void* x, void* out, void* ws,
                cudaStream_t s);

}  // namespace orth
}  // namespace poetx
