// Interfaces of the row operators: the RMS norm and its gradient (norm.cu),
// rows sorted by expert and back (permute.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace swg {

constexpr int64_t kMaxNormWidth = 32768;

struct NormCall {
  const void* x;
  const void* residual;   // or null
  const void* weight;     // [d]
  void* out;              // [M, d]: x's type, or e4m3 codes where `scales`
  float* scales;          // [M], or null
  void* sum;              // [M, d] where `residual`
  int64_t M, d;
  float eps;
  int f32, weight_f32;
};
cudaError_t launch_rms_norm(const NormCall& c, int num_sms, cudaStream_t st);

struct NormBackwardCall {
  const void* dy;
  const void* s;
  const void* weight;
  const void* ds;         // or null
  void* dx;
  void* dweight;          // [d], weight's type
  int64_t M, d;
  float eps;
  int f32, weight_f32;
};
// The partial sums of dweight: one row of d f32 values per CTA or cluster.
size_t rms_norm_backward_bytes(int64_t M, int64_t d, int f32, int num_sms);
cudaError_t launch_rms_norm_backward(const NormBackwardCall& c, float* part, int num_sms,
                                     cudaStream_t st);

// out[position[t, j]] = x[t]; rows from offsets[E] on are zero.  d elements of
// `elem` bytes to a row.  scales: null, or a scale per row that goes with it.
struct PermuteCall {
  const void* x;
  const float* scales;
  const int* position;
  const int* offsets;
  void* out;
  float* out_scales;
  int64_t T, k, E, d;
  int elem;
};
cudaError_t launch_permute(const PermuteCall& c, int num_sms, cudaStream_t st);

// y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]] (weights null: 1).
struct UnpermuteCall {
  const void* z;
  const int* position;
  const float* weights;
  const void* residual;
  void* y;
  int64_t T, k, d;
  int f32;
};
cudaError_t launch_unpermute(const UnpermuteCall& c, int num_sms, cudaStream_t st);

// dz[position[t, j]] = weights[t, j] dy[t], zero from offsets[E] on;
// dweights[t, j] = dy[t] . z[position[t, j]], 0 where there is no place.
struct UnpermuteBackwardCall {
  const void* dy;
  const void* z;
  const int* position;
  const int* offsets;
  const float* weights;
  void* dz;
  float* dweights;
  int64_t T, k, E, d;
  int f32;
};
cudaError_t launch_unpermute_backward(const UnpermuteBackwardCall& c, int num_sms,
                                      cudaStream_t st);

}  // namespace swg
