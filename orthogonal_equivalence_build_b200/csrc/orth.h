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

// Powers of two that hold every operand of every step inside fp16 (see orth.cu).
struct Plan {
  float sx[kMaxSteps + 1];   // scale of X before step t
  float sa[kMaxSteps], sb[kMaxSteps];   // of A and B
};
// false: the coefficients are not finite or let the singular values grow past every bound
bool make_plan(const float* coeffs, int steps, Plan* plan);

// Factors of the epilogues: gram, square and update results are f[0..2][t] times the accumulator;
// square adds fa[t] A and da[t] I (operands as stored, scales included).
void fill_factors(const Problem& p, const Plan& plan, float (*f)[kMaxSteps], float* fa, float* da);

// One CTA per matrix (orth_small.cu), where a matrix fits into shared memory.
bool small_fits(const Problem& p);
cudaError_t run_small(const Problem& p, const Plan& plan, const void* x, void* out,
                      cudaStream_t s);

size_t workspace_bytes(const Problem& p);
cudaError_t run(const Problem& p, const Plan& plan, const void* x, void* out, void* ws,
                cudaStream_t s);

}  // namespace orth
}  // namespace poetx
