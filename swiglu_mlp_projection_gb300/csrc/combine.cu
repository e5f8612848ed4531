// The weighted sum over a token's choices, which ends the experts' down
// projection:
//
//   y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]]
//
// j ascending, in f32, rounded once.  Bound by memory: each z row is read
// once (16-byte loads, a warp covers consecutive columns), y written once.
#include "common.cuh"
#include "grouped.h"
#include "tc_common.cuh"

namespace swg {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 8;   // columns per thread
constexpr int kBatch = 4; // choices whose loads are in flight together

__global__ void __launch_bounds__(kThreads)
combine_kernel(const float* __restrict__ z, const int* __restrict__ position,
               const float* __restrict__ weights, const uint16_t* resid, uint16_t* y, int64_t T,
               int k, int64_t rows, int64_t d) {
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int64_t per = d / kVec;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < T * per;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per, c = (i - t * per) * kVec;
    float acc[kVec];
    if (resid) {
      const uint4 r = *reinterpret_cast<const uint4*>(resid + t * d + c);
      acc[0] = bf16_lo(r.x); acc[1] = bf16_hi(r.x);
      acc[2] = bf16_lo(r.y); acc[3] = bf16_hi(r.y);
      acc[4] = bf16_lo(r.z); acc[5] = bf16_hi(r.z);
      acc[6] = bf16_lo(r.w); acc[7] = bf16_hi(r.w);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
    }
    // four choices at a time: their rows' loads are in flight together
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      float w[kBatch];
      float4 a[kBatch], b[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        int p = -1;
        if (j0 + i < k) {
          p = position[t * k + j0 + i];
          w[i] = weights[t * k + j0 + i];
        }
        a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < 0 || p >= rows) {
          w[i] = 0.f;   // no term (whatever its weight)
        } else {
          const float4* src = reinterpret_cast<const float4*>(z + (int64_t)p * d + c);
          a[i] = __ldcs(src);
          b[i] = __ldcs(src + 1);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        acc[0] = fmaf(w[i], a[i].x, acc[0]); acc[1] = fmaf(w[i], a[i].y, acc[1]);
        acc[2] = fmaf(w[i], a[i].z, acc[2]); acc[3] = fmaf(w[i], a[i].w, acc[3]);
        acc[4] = fmaf(w[i], b[i].x, acc[4]); acc[5] = fmaf(w[i], b[i].y, acc[5]);
        acc[6] = fmaf(w[i], b[i].z, acc[6]); acc[7] = fmaf(w[i], b[i].w, acc[7]);
      }
    }
    uint4 o;
    o.x = pack_bf16x2(acc[0], acc[1]);
    o.y = pack_bf16x2(acc[2], acc[3]);
    o.z = pack_bf16x2(acc[4], acc[5]);
    o.w = pack_bf16x2(acc[6], acc[7]);
    *reinterpret_cast<uint4*>(y + t * d + c) = o;
  }
}

}  // namespace

cudaError_t launch_combine(const float* z, const int* position, const float* weights,
                           const void* residual, void* y, int64_t T, int64_t k, int64_t rows,
                           int64_t d, int num_sms, cudaStream_t st) {
  if (T == 0 || d == 0) return cudaSuccess;
  int64_t blocks = (T * (d / kVec) + kThreads - 1) / kThreads;
  const int64_t most = (int64_t)num_sms * 16;
  if (blocks > most) blocks = most;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel, z, position, weights, (const uint16_t*)residual,
                            (uint16_t*)y, T, (int)k, rows, d);
}

}  // namespace swg
