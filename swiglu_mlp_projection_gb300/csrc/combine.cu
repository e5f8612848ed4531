// The weighted sum over a token's choices, which ends the experts' down
// projection:
//
//   y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]]
//
// j ascending, in f32, rounded once.  A row of z whose unit of the product was
// cut along K is the sum of that unit's shares, in k order.  Bound by memory:
// each z row is read once (16-byte loads, a warp covers consecutive columns),
// y written once.
#include "common.cuh"
#include "grouped.h"
#include "grouped_plan.cuh"
#include "tc_common.cuh"

namespace swg {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 8;   // columns per thread
constexpr int kBatch = 8; // choices whose loads are in flight together

// Columns c .. c + 7 of sorted row p, if its unit was cut.
__device__ __forceinline__ bool cut_row(const Work& w, const Schedule& sch, const int* s_row,
                                        const int* s_chunk, int p, int c, float4* lo, float4* hi) {
  int a = 0, b = w.E;   // s_row[a] <= p < s_row[b]
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (s_row[mid] <= p) a = mid;
    else b = mid;
  }
  const int m = s_row[a + 1] - s_row[a], nc = s_chunk[a + 1] - s_chunk[a];
  if (nc < 1 || p < s_row[a]) return false;
  const int per = (m + nc - 1) / nc;
  const int chunk = (p - s_row[a]) / per;
  const uint32_t u = (uint32_t)s_chunk[a] * (uint32_t)w.ncg + (uint32_t)((c >> 8) * nc + chunk);
  if (u < sch.whole || u >= sch.units || chunk >= nc) return false;
  float v[8];
  add_row_shares<4>(w, shares_of(w, sch, u - sch.whole), (uint32_t)((c >> 7) & 1),
                 (p - s_row[a] - chunk * per) * 128 + (c & 127), v);
  *lo = make_float4(v[0], v[1], v[2], v[3]);
  *hi = make_float4(v[4], v[5], v[6], v[7]);
  return true;
}

template <bool CUT>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const float* __restrict__ z, const __grid_constant__ Work w,
               const int* __restrict__ position, const float* __restrict__ weights,
               const uint16_t* resid, uint16_t* y, int64_t T, int k, int64_t rows, int64_t d) {
  extern __shared__ int s_row[];   // [E + 1] first rows, then [E + 1] first chunks
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  // (the plan is read only where the product says that it cut units)
  Schedule sch{0, 0, 0, 1};
  int* s_chunk = s_row + w.E + 1;
  if (CUT) {
    const uint4 q = __ldcg(w.sched);
    sch = Schedule{q.x, q.y, q.z, q.w};
    if (sch.cut_iters > 0) {
      plan_chunks(w, s_row, s_chunk);
      __syncthreads();
    }
  }
  const int64_t per = d / kVec;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < T * per;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per, c = (i - t * per) * kVec;
    // (the residual is used only after the first rows' loads are under way)
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (resid) r = *reinterpret_cast<const uint4*>(resid + t * d + c);
    float acc[kVec];
    int p[kBatch];
    float wt[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      p[i] = i < k ? position[t * k + i] : -1;
      wt[i] = i < k ? weights[t * k + i] : 0.f;
    }
    // several choices at a time: their rows' loads are in flight together
    for (int j0 = 0; j0 == 0 || j0 < k; j0 += kBatch) {
      float4 a[kBatch], b[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p[i] < 0 || p[i] >= rows) {
          wt[i] = 0.f;   // no term (whatever its weight)
        } else if (CUT && sch.cut_iters > 0 &&
                   cut_row(w, sch, s_row, s_chunk, p[i], (int)c, &a[i], &b[i])) {
          // (the sums of the shares)
        } else {
          const float4* src = reinterpret_cast<const float4*>(z + (int64_t)p[i] * d + c);
          a[i] = __ldcs(src);
          b[i] = __ldcs(src + 1);
        }
      }
      int pn[kBatch];
      float wn[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {   // the next choices
        const int j = j0 + kBatch + i;
        pn[i] = j < k ? position[t * k + j] : -1;
        wn[i] = j < k ? weights[t * k + j] : 0.f;
      }
      if (j0 == 0) {
        acc[0] = bf16_lo(r.x); acc[1] = bf16_hi(r.x);
        acc[2] = bf16_lo(r.y); acc[3] = bf16_hi(r.y);
        acc[4] = bf16_lo(r.z); acc[5] = bf16_hi(r.z);
        acc[6] = bf16_lo(r.w); acc[7] = bf16_hi(r.w);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        acc[0] = fmaf(wt[i], a[i].x, acc[0]); acc[1] = fmaf(wt[i], a[i].y, acc[1]);
        acc[2] = fmaf(wt[i], a[i].z, acc[2]); acc[3] = fmaf(wt[i], a[i].w, acc[3]);
        acc[4] = fmaf(wt[i], b[i].x, acc[4]); acc[5] = fmaf(wt[i], b[i].y, acc[5]);
        acc[6] = fmaf(wt[i], b[i].z, acc[6]); acc[7] = fmaf(wt[i], b[i].w, acc[7]);
        p[i] = pn[i];
        wt[i] = wn[i];
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

cudaError_t launch_combine(const float* z, const Work* w, const int* position,
                           const float* weights, const void* residual, void* y, int64_t T,
                           int64_t k, int64_t rows, int64_t d, int num_sms, cudaStream_t st) {
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
  if (z && w->shares) {
    cfg.dynamicSmemBytes = (size_t)(2 * (w->E + 1)) * sizeof(int);
    return cudaLaunchKernelEx(&cfg, combine_kernel<true>, z, *w, position, weights,
                              (const uint16_t*)residual, (uint16_t*)y, T, (int)k, rows, d);
  }
  return cudaLaunchKernelEx(&cfg, combine_kernel<false>, z, *w, position, weights,
                            (const uint16_t*)residual, (uint16_t*)y, T, (int)k, rows, d);
}

}  // namespace swg
