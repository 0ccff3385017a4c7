// Layer norm and its gradient — interface of norm.cu.
#pragma once
#include "internal.h"

namespace poetx {
namespace norm {

struct Fwd {
  const void* x;              // [T][m]
  int64_t T, m;
  const void *gamma, *beta;   // [m] or NULL (ones, zeros)
  int w_bf16;
  float eps;
  void* y;                    // [T][m], may be x
  float *mean, *rstd;         // [T] or NULL
};
struct Bwd {
  const void *x, *dy;
  int64_t T, m;
  const void* gamma;
  int w_bf16;
  const float *mean, *rstd;
  void* dx;                   // [T][m] or NULL, may be x or dy
  float *dgamma, *dbeta;      // [m] or NULL
  float* part;                // [2][parts][m]: column sums per range of rows
  int parts;
  int* err;                   // device error word (bounded waits)
};

size_t bwd_ws_bytes(int64_t T, int64_t m);
cudaError_t fwd(const Fwd& a, DT t, cudaStream_t s);
cudaError_t bwd(Bwd a, DT t, void* ws, cudaStream_t s);

}  // namespace norm
}  // namespace poetx
