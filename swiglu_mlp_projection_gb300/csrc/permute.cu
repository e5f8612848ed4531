// Rows sorted by expert, and back, with their gradients (see rows.h):
//
//   permute:    out[position[t, j]] = x[t]
//   unpermute:  y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]]
//   gradient of unpermute:
//               dz[position[t, j]] = weights[t, j] dy[t]
//               dweights[t, j] = dy[t] . z[position[t, j]]
//
// (the gradient of permute is unpermute without weights).  All go by token, not
// by sorted row, so that x and dy are read once however many choices there
// are.  Bound by memory.  Rows from offsets[E] on belong to no pair; as many
// choices are dropped as there are such rows, so the (t, j) whose flat index is
// such a row's clears it.
#include "rows.cuh"
#include "rows.h"

namespace swg {
namespace {

constexpr int kBatch = 8;   // choices whose loads are in flight together

// A CTA has blockDim.y tokens at a time, blockDim.x threads for a piece of each row.
struct Team {
  int64_t t;
  int w;   // first word of this thread
};
__device__ __forceinline__ Team team() {
  return {(int64_t)blockIdx.x * blockDim.y + threadIdx.y,
          (int)(blockIdx.y * blockDim.x + threadIdx.x)};
}

__device__ __forceinline__ int64_t sorted_end(const int* offsets, int E, int64_t rows) {
  const int64_t n = offsets[E];
  return n < 0 ? 0 : n < rows ? n : rows;
}

// W: the widest word that divides a row's bytes; `per` words to a row.
template <typename W>
__global__ void __launch_bounds__(256)
permute_kernel(const W* __restrict__ x, const float* __restrict__ scales,
               const int* __restrict__ position, const int* __restrict__ offsets,
               W* __restrict__ out, float* __restrict__ out_scales, int64_t T, int k, int E,
               int per) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const Team tm = team();
  if (tm.t >= T) return;
  const int64_t rows = T * k, end = sorted_end(offsets, E, rows), f0 = tm.t * k;
  const int* pos = position + f0;
  for (int w = tm.w; w < per; w += gridDim.y * blockDim.x) {
    const W v = x[tm.t * per + w];
    for (int j = 0; j < k; ++j) {
      const int p = pos[j];
      if (p >= 0 && p < rows) out[(int64_t)p * per + w] = v;
      if (f0 + j >= end) out[(f0 + j) * per + w] = W{};
    }
  }
  if (scales && tm.w == 0) {
    const float s = scales[tm.t];
    for (int j = 0; j < k; ++j) {
      const int p = pos[j];
      if (p >= 0 && p < rows) out_scales[p] = s;
      if (f0 + j >= end) out_scales[f0 + j] = 0.f;
    }
  }
}

// N elements of a row as one word.
template <bool F32, int N>
struct Word {
  using E = typename Row<F32>::elem;
  static constexpr int kBytes = N * (int)sizeof(E);
  __device__ static __forceinline__ void load(const E* p, float (&v)[N]) {
    if constexpr (kBytes == 16) {
      unpack<F32>(load_once(p), v);
    } else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      if constexpr (F32) {
        v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
      } else {
        v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
      }
    } else if constexpr (N == 2) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(p);
      v[0] = bf16_lo(q); v[1] = bf16_hi(q);
    } else {
      v[0] = elem_f32(*p);
    }
  }
  __device__ static __forceinline__ void store(E* p, const float (&v)[N]) {
    if constexpr (kBytes == 16) {
      *reinterpret_cast<uint4*>(p) = pack<F32>(v);
    } else if constexpr (kBytes == 8) {
      if constexpr (F32)
        *reinterpret_cast<uint2*>(p) = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
      else
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    } else if constexpr (N == 2) {
      *reinterpret_cast<uint32_t*>(p) = bf16x2(v[0], v[1]);
    } else {
      set_elem(p, v[0]);
    }
  }
};

template <bool F32, int N>
__global__ void __launch_bounds__(256)
unpermute_kernel(const typename Row<F32>::elem* __restrict__ z, const int* __restrict__ position,
                 const float* __restrict__ weights, const typename Row<F32>::elem* residual,
                 typename Row<F32>::elem* y, int64_t T, int k, int64_t d, int per) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const Team tm = team();
  if (tm.t >= T) return;
  const int64_t rows = T * k;
  const int* pos = position + tm.t * k;
  const float* wt = weights ? weights + tm.t * k : nullptr;
  for (int w = tm.w; w < per; w += gridDim.y * blockDim.x) {
    float acc[N];
    if (residual) {
      Word<F32, N>::load(residual + tm.t * d + (int64_t)w * N, acc);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = 0.f;
    }
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      float v[kBatch][N], c[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = j0 + i < k ? pos[j0 + i] : -1;
        const bool live = p >= 0 && p < rows;
        c[i] = !live ? 0.f : wt ? wt[j0 + i] : 1.f;
        if (live) {
          Word<F32, N>::load(z + (int64_t)p * d + (int64_t)w * N, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) v[i][e] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(c[i], v[i][e], acc[e]);
    }
    Word<F32, N>::store(y + tm.t * d + (int64_t)w * N, acc);
  }
}

// One token per CTA row of threads; the dot products meet in shared memory.
template <bool F32, int N>
__global__ void __launch_bounds__(256)
unpermute_backward_kernel(const typename Row<F32>::elem* __restrict__ dy,
                          const typename Row<F32>::elem* __restrict__ z,
                          const int* __restrict__ position, const int* __restrict__ offsets,
                          const float* __restrict__ weights, typename Row<F32>::elem* dz,
                          float* __restrict__ dweights, int64_t T, int k, int E, int64_t d,
                          int per) {
  __shared__ float red[8][kBatch];   // by warp of the CTA
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool here = t < T;
  const int64_t rows = T * k, end = sorted_end(offsets, E, rows), f0 = t * k;
  const int warps = blockDim.x >> 5;   // of a token
  const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, l = threadIdx.x & 31;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    int p[kBatch];
    float c[kBatch], dot[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const bool in = here && j0 + i < k;
      p[i] = in ? position[f0 + j0 + i] : -1;
      if (p[i] >= rows) p[i] = -1;
      c[i] = in && p[i] >= 0 ? weights[f0 + j0 + i] : 0.f;
      dot[i] = 0.f;
    }
    for (int w = threadIdx.x; here && w < per; w += blockDim.x) {
      float g[N], v[kBatch][N];
      Word<F32, N>::load(dy + t * d + (int64_t)w * N, g);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (p[i] >= 0) Word<F32, N>::load(z + (int64_t)p[i] * d + (int64_t)w * N, v[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (p[i] >= 0) {
          float o[N];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            dot[i] = fmaf(g[e], v[i][e], dot[i]);
            o[e] = c[i] * g[e];
          }
          Word<F32, N>::store(dz + (int64_t)p[i] * d + (int64_t)w * N, o);
        }
        if (j0 + i < k && f0 + j0 + i >= end) {
          float o[N];
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] = 0.f;
          Word<F32, N>::store(dz + (f0 + j0 + i) * d + (int64_t)w * N, o);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
    }
    if (l == 0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) red[warp][i] = dot[i];
    }
    __syncthreads();
    if (here && threadIdx.x < kBatch && j0 + (int)threadIdx.x < k) {
      float s = 0.f;
      for (int i = 0; i < warps; ++i) s += red[threadIdx.y * warps + i][threadIdx.x];
      dweights[f0 + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// Threads for a row of `per` words: a power of two, 32 ... 256.
int row_threads(int64_t per) {
  int n = 32;
  while (n < 256 && n < per) n *= 2;
  return n;
}

// Few tokens: their rows are spread over several CTAs.
dim3 grid_of(int64_t T, int64_t per, dim3 block) {
  int64_t parts = (per + block.x - 1) / block.x;
  if (parts > 64) parts = 64;
  if (parts < 1) parts = 1;   // (rows of nothing, whose scales are moved all the same)
  return dim3((unsigned)((T + block.y - 1) / block.y), (unsigned)parts);
}

template <typename W>
cudaError_t permute_words(const PermuteCall& c, int64_t bytes, cudaStream_t st) {
  const int64_t per = bytes / (int64_t)sizeof(W);
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(permute_kernel<W>, grid_of(c.T, per, block), block, 0, st, (const W*)c.x,
                        c.scales, c.position, c.offsets, (W*)c.out, c.out_scales, c.T, (int)c.k,
                        (int)c.E, (int)per);
}

template <bool F32, int N>
cudaError_t unpermute_words(const UnpermuteCall& c, cudaStream_t st) {
  using E = typename Row<F32>::elem;
  const int64_t per = c.d / N;
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(unpermute_kernel<F32, N>, grid_of(c.T, per, block), block, 0, st,
                        (const E*)c.z, c.position, c.weights, (const E*)c.residual, (E*)c.y, c.T,
                        (int)c.k, c.d, (int)per);
}

template <bool F32, int N>
cudaError_t backward_words(const UnpermuteBackwardCall& c, cudaStream_t st) {
  using E = typename Row<F32>::elem;
  const int64_t per = c.d / N;
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(unpermute_backward_kernel<F32, N>,
                        dim3((unsigned)((c.T + block.y - 1) / block.y)), block, 0, st,
                        (const E*)c.dy, (const E*)c.z, c.position, c.offsets, c.weights, (E*)c.dz,
                        c.dweights, c.T, (int)c.k, (int)c.E, c.d, (int)per);
}

}  // namespace

cudaError_t launch_permute(const PermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.k == 0 || (c.d == 0 && !c.scales)) return cudaSuccess;
  const int64_t bytes = c.d * c.elem;
  if (bytes % 16 == 0) return permute_words<uint4>(c, bytes, st);
  if (bytes % 8 == 0) return permute_words<uint2>(c, bytes, st);
  if (bytes % 4 == 0) return permute_words<uint32_t>(c, bytes, st);
  if (bytes % 2 == 0) return permute_words<uint16_t>(c, bytes, st);
  return permute_words<uint8_t>(c, bytes, st);
}

cudaError_t launch_unpermute(const UnpermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.d == 0) return cudaSuccess;
  if (c.f32)
    return c.d % 4 == 0 ? unpermute_words<true, 4>(c, st)
           : c.d % 2 == 0 ? unpermute_words<true, 2>(c, st) : unpermute_words<true, 1>(c, st);
  return c.d % 8 == 0   ? unpermute_words<false, 8>(c, st)
         : c.d % 4 == 0 ? unpermute_words<false, 4>(c, st)
         : c.d % 2 == 0 ? unpermute_words<false, 2>(c, st) : unpermute_words<false, 1>(c, st);
}

cudaError_t launch_unpermute_backward(const UnpermuteBackwardCall& c, int num_sms,
                                      cudaStream_t st) {
  if (c.T == 0 || c.k == 0) return cudaSuccess;
  if (c.f32)
    return c.d % 4 == 0 ? backward_words<true, 4>(c, st)
           : c.d % 2 == 0 ? backward_words<true, 2>(c, st) : backward_words<true, 1>(c, st);
  return c.d % 8 == 0   ? backward_words<false, 8>(c, st)
         : c.d % 4 == 0 ? backward_words<false, 4>(c, st)
         : c.d % 2 == 0 ? backward_words<false, 2>(c, st) : backward_words<false, 1>(c, st);
}

}  // namespace swg
