// The root-mean-square norm that begins an MLP block, with the residual's
// addition before it, and its gradient.
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
//
// in f32 from the operands on; s and y are each rounded once.  A row stays in
// registers as t = s * weight, so that one reduction over the row gives both
// the sum of s^2 and, for 8-bit rows, max |t|: with r = 1 / sqrt(...), y = t r,
// the row's largest |y| is max |t| r, and its codes e4m3(y 448 / amax) are
// e4m3(t 448 / max |t|), without r.
#include "rows.cuh"
#include "rows.h"

namespace swg {
namespace {

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* out;
  float* scales;
  void* sum;
  int64_t M;
  int d;
  float eps;
  int weight_f32;
};

// Below this max |t| a row is 0 in 8 bits (448 / max |t| would leave binary32).
constexpr float kLeastAmax = 0x1p-118f;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Largest of values that are not negative (their bits order like the values; NaN is largest).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// One row per warp (WARP) or per CTA; VPT 16-byte pieces per thread.
template <bool F32, int VPT, bool FP8, bool RAGGED, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = Row<F32>::kVec;
  __shared__ float red_sum[32], red_max[32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int lanes = WARP ? 32 : blockDim.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                           : (int64_t)blockIdx.x;
  if (WARP && row >= a.M) return;
  const Pieces<F32, RAGGED> pc(row, a.d);

  uint4 xr[VPT], rr[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i < pc.n) {
      xr[j] = pc.load(a.x, i);
      if (a.residual) rr[j] = pc.load(a.residual, i);
    }
  }
  float t[VPT][V];
  float q = 0.f, m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i >= pc.n) continue;
    unpack<F32>(xr[j], t[j]);
    if (a.residual) {
      float r[V];
      unpack<F32>(rr[j], r);
#pragma unroll
      for (int e = 0; e < V; ++e) t[j][e] += r[e];
      pc.store(a.sum, i, t[j]);
    }
    float w[V];
    pc.weight(a.weight, a.weight_f32, i, w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      q = fmaf(t[j][e], t[j][e], q);
      t[j][e] *= w[e];
      if (FP8) m = fmaxf(m, fabsf(t[j][e]));
    }
  }
  q = warp_sum(q);
  if (FP8) m = warp_max(m);
  if (!WARP) {
    const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (l == 0) {
      red_sum[warp] = q;
      if (FP8) red_max[warp] = m;
    }
    __syncthreads();
    const bool in = l < (int)(blockDim.x >> 5);
    q = warp_sum(in ? red_sum[l] : 0.f);
    if (FP8) m = warp_max(in ? red_max[l] : 0.f);
  }
  const float r = 1.0f / sqrtf(q / (float)a.d + a.eps);
  const float f = FP8 ? (m >= kLeastAmax ? 448.0f / m : 0.f) : r;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i >= pc.n) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) t[j][e] *= f;
    if constexpr (FP8) {
      uint8_t* o = (uint8_t*)a.out + pc.first + (int64_t)i * V;
      uint32_t c[V / 4];
#pragma unroll
      for (int h = 0; h < V / 4; ++h)
        c[h] = e4m3x2(t[j][4 * h], t[j][4 * h + 1]) | (e4m3x2(t[j][4 * h + 2], t[j][4 * h + 3]) << 16);
      if (pc.whole(i)) {
        if constexpr (V == 8) *reinterpret_cast<uint2*>(o) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<uint32_t*>(o) = c[0];
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (pc.has(i, e)) o[e] = (uint8_t)(c[e / 4] >> (8 * (e & 3)));
      }
    } else {
      pc.store(a.out, i, t[j]);
    }
  }
  if (FP8 && lane == 0) a.scales[row] = (m >= kLeastAmax ? m : 0.f) * r / 448.0f;
}

// How a row's pieces are dealt out.
struct Shape {
  int vpt;       // pieces per thread
  int threads;   // threads per row
  bool warp;     // 32 of them, eight rows to a CTA
};
Shape shape_of(int64_t pieces, int vec, int64_t M, int num_sms) {
  // Many rows of up to 1024 elements: a warp each.  Otherwise a CTA with 16
  // elements per thread: 8 where the rows are few and only latency counts, 32
  // where 1024 threads would not do.
  int e = 8;
  if (M > num_sms) {
    while (e < 32 && 32 * (e / vec) < pieces) e *= 2;
    if (32 * (e / vec) >= pieces) return {e / vec, 32, true};
    e = 16;
  }
  while (e < 32 && 1024 * (e / vec) < pieces) e *= 2;
  const int vpt = e / vec;
  return {vpt, (int)((pieces + vpt * 32 - 1) / (vpt * 32) * 32), false};
}

template <bool F32, int VPT, bool FP8, bool RAGGED>
cudaError_t launch_norm(const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (s.warp)
    return launch_chained(norm_kernel<F32, VPT, FP8, RAGGED, true>, dim3((unsigned)((a.M + 7) / 8)),
                          dim3(256), 0, st, a);
  return launch_chained(norm_kernel<F32, VPT, FP8, RAGGED, false>, dim3((unsigned)a.M),
                        dim3(s.threads), 0, st, a);
}

template <bool F32, bool FP8, bool RAGGED>
cudaError_t launch_vpt(const NormArgs& a, const Shape& s, cudaStream_t st) {
  constexpr int base = 8 / Row<F32>::kVec;   // pieces of 8 elements
  if (s.vpt == base) return launch_norm<F32, base, FP8, RAGGED>(a, s, st);
  if (s.vpt == 2 * base) return launch_norm<F32, 2 * base, FP8, RAGGED>(a, s, st);
  return launch_norm<F32, 4 * base, FP8, RAGGED>(a, s, st);
}

template <bool F32>
cudaError_t launch_type(const NormArgs& a, bool fp8, bool ragged, const Shape& s, cudaStream_t st) {
  if (fp8)
    return ragged ? launch_vpt<F32, true, true>(a, s, st) : launch_vpt<F32, true, false>(a, s, st);
  return ragged ? launch_vpt<F32, false, true>(a, s, st) : launch_vpt<F32, false, false>(a, s, st);
}

// ---- gradient -------------------------------------------------------------------
//
//   r = 1 / sqrt(mean(s^2) + eps), g = dy * weight
//   dx = ds + r (g - s r^2 mean(g s)),  dweight = sum over rows of dy s r
//
// A CTA takes rows in a fixed order and keeps the columns' sums of dweight for
// all of them (in registers, or in shared memory for the widest rows); each CTA
// then writes one row of partial sums, and a second kernel adds those in a
// fixed order.

struct BackArgs {
  const void* dy;
  const void* s;
  const void* weight;
  const void* ds;
  void* dx;
  float* part;   // [gridDim.x, d]
  int64_t M;
  int d;
  float eps;
  int weight_f32;
};

template <bool F32, int VPT, bool RAGGED, bool SMEM>
__global__ void __launch_bounds__(SMEM ? 1024 : 512)
norm_backward_kernel(const __grid_constant__ BackArgs a) {
  constexpr int V = Row<F32>::kVec;
  extern __shared__ float s_acc[];   // SMEM: [VPT][V][threads]
  __shared__ float2 red[2][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int lanes = blockDim.x, warp = threadIdx.x >> 5, l = threadIdx.x & 31;
  float acc[SMEM ? 1 : VPT][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (SMEM) s_acc[(j * V + e) * lanes + threadIdx.x] = 0.f;
      else acc[SMEM ? 0 : j][e] = 0.f;
    }
  int side = 0;
  // (ragged: all rows of a CTA start at one place in their 16 bytes, since
  // gridDim.x is a multiple of 8 or every CTA has one row)
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, side ^= 1) {
    const Pieces<F32, RAGGED> pc(row, a.d);
    uint4 sr[VPT], dr[VPT], er[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = threadIdx.x + j * lanes;
      if (i < pc.n) {
        sr[j] = pc.load(a.s, i);
        dr[j] = pc.load(a.dy, i);
        if (a.ds) er[j] = pc.load(a.ds, i);
      }
    }
    float q = 0.f, p = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = threadIdx.x + j * lanes;
      if (i >= pc.n) continue;
      float s[V], g[V], w[V];
      unpack<F32>(sr[j], s);
      unpack<F32>(dr[j], g);
      pc.weight(a.weight, a.weight_f32, i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        q = fmaf(s[e], s[e], q);
        p = fmaf(g[e] * w[e], s[e], p);
      }
    }
    q = warp_sum(q);
    p = warp_sum(p);
    if (l == 0) red[side][warp] = make_float2(q, p);
    __syncthreads();   // (one is enough: the next row writes the other side)
    const float2 v = l < (lanes >> 5) ? red[side][l] : make_float2(0.f, 0.f);
    q = warp_sum(v.x);
    p = warp_sum(v.y);
    const float r = 1.0f / sqrtf(q / (float)a.d + a.eps);
    const float c = r * r * (p / (float)a.d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = threadIdx.x + j * lanes;
      if (i >= pc.n) continue;
      float s[V], g[V], w[V], o[V];
      unpack<F32>(sr[j], s);
      unpack<F32>(dr[j], g);
      pc.weight(a.weight, a.weight_f32, i, w);
      if (a.ds) {
        unpack<F32>(er[j], o);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = g[e] * (s[e] * r);
        if (SMEM) s_acc[(j * V + e) * lanes + threadIdx.x] += t;
        else acc[SMEM ? 0 : j][e] += t;
        o[e] = fmaf(r, fmaf(g[e], w[e], -s[e] * c), o[e]);
      }
      pc.store(a.dx, i, o);
    }
  }
  const Pieces<F32, RAGGED> pc(blockIdx.x, a.d);
  float* part = a.part + (int64_t)blockIdx.x * a.d;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = threadIdx.x + j * lanes;
    if (i >= pc.n) continue;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (pc.has(i, e))
        part[pc.col(i) + e] = SMEM ? s_acc[(j * V + e) * lanes + threadIdx.x] : acc[SMEM ? 0 : j][e];
  }
}

constexpr int kSumCols = 32, kSumRows = 32;

// dweight = the partial sums of n CTAs, added in a fixed order.
__global__ void __launch_bounds__(kSumCols * kSumRows)
dweight_kernel(const float* __restrict__ part, int n, int d, void* __restrict__ out, int f32) {
  __shared__ float red[kSumRows][kSumCols + 1];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * kSumCols + x;
  float v = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int i = y; i < n; i += kSumRows) v += part[(int64_t)i * d + c];
  }
  red[y][x] = v;
  __syncthreads();
  v = warp_sum(red[x][y]);   // column y of this block
  const int o = blockIdx.x * kSumCols + y;
  if (x == 0 && o < d) {
    if (f32) ((float*)out)[o] = v;
    else set_elem((uint16_t*)out + o, v);
  }
}

// CTAs of the gradient's kernel.
int back_grid(int64_t M, int num_sms) {
  const int64_t most = (int64_t)num_sms * 2 / 8 * 8;
  return (int)(M < most ? M : most);
}

template <bool F32, bool RAGGED>
cudaError_t launch_back(const BackArgs& a, int64_t pieces, int grid, cudaStream_t st) {
  constexpr int kTwo = 16 / Row<F32>::kVec;   // pieces of 16 elements
  const auto threads = [&](int vpt) { return (int)((pieces + vpt * 32 - 1) / (vpt * 32) * 32); };
  const int t = threads(kTwo);
  if (t <= 512)
    return launch_chained(norm_backward_kernel<F32, kTwo, RAGGED, false>, dim3(grid), dim3(t), 0,
                          st, a);
  const int w = threads(2 * kTwo);
  const size_t smem = (size_t)w * 2 * 16 * sizeof(float);
  const auto k = norm_backward_kernel<F32, 2 * kTwo, RAGGED, true>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(grid), dim3(w), smem, st, a);
}

}  // namespace

cudaError_t launch_rms_norm(const NormCall& c, int num_sms, cudaStream_t st) {
  if (c.M == 0 || c.d == 0) return cudaSuccess;
  const NormArgs a{c.x, c.residual, c.weight, c.out, c.scales, c.sum, c.M, (int)c.d, c.eps,
                   c.weight_f32};
  const int vec = c.f32 ? 4 : 8;
  const bool ragged = c.d % vec != 0;
  const int64_t pieces = ragged ? c.d / vec + 2 : c.d / vec;
  const Shape s = shape_of(pieces, vec, c.M, num_sms);
  return c.f32 ? launch_type<true>(a, c.scales != nullptr, ragged, s, st)
               : launch_type<false>(a, c.scales != nullptr, ragged, s, st);
}

size_t rms_norm_backward_bytes(int64_t M, int64_t d, int f32, int num_sms) {
  return (size_t)back_grid(M, num_sms) * (size_t)d * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackwardCall& c, float* part, int num_sms,
                                     cudaStream_t st) {
  if (c.d == 0) return cudaSuccess;
  const int grid = back_grid(c.M, num_sms);
  if (c.M > 0) {
    const BackArgs a{c.dy, c.s, c.weight, c.ds, c.dx, part, c.M, (int)c.d, c.eps, c.weight_f32};
    const int vec = c.f32 ? 4 : 8;
    const bool ragged = c.d % vec != 0;
    const int64_t pieces = ragged ? c.d / vec + 2 : c.d / vec;
    const cudaError_t e =
        c.f32 ? (ragged ? launch_back<true, true>(a, pieces, grid, st)
                        : launch_back<true, false>(a, pieces, grid, st))
              : (ragged ? launch_back<false, true>(a, pieces, grid, st)
                        : launch_back<false, false>(a, pieces, grid, st));
    if (e != cudaSuccess) return e;
  }
  return launch_chained(dweight_kernel, dim3((unsigned)((c.d + kSumCols - 1) / kSumCols)),
                        dim3(kSumCols * kSumRows), 0, st, (const float*)part, grid, (int)c.d,
                        c.dweight, c.weight_f32);
}

}  // namespace swg
