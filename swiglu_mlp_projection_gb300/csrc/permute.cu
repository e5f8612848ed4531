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
//
// Rows are moved in 16-byte pieces that start on 16-byte boundaries of the
// tensor that is written.  Where a row's bytes are no multiple of 16 (RAGGED),
// the source starts elsewhere in its 16 bytes: two of its pieces are read (the
// second is a neighbour's first, from L1) and shifted together.
#include "rows.cuh"
#include "rows.h"

namespace swg {
namespace {

constexpr int kBatch = 8;   // choices whose loads are in flight together

// A CTA has blockDim.y tokens, blockDim.x threads for a piece of each row.
__device__ __forceinline__ int64_t token() {
  return (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
}

__device__ __forceinline__ int64_t sorted_end(const int* offsets, int E, int64_t rows) {
  const int64_t n = offsets[E];
  return n < 0 ? 0 : n < rows ? n : rows;
}

// Rows of `bytes` bytes (a multiple of sizeof(E)), row r's at byte r * bytes.
template <typename E, bool RAGGED>
struct Span16 {
  int64_t base;     // the row's first byte
  int shift;        // ... within its 16 bytes
  int n;            // pieces
  int bytes;
  __device__ __forceinline__ Span16(int64_t row, int bytes_) : base(row * bytes_), bytes(bytes_) {
    shift = RAGGED ? (int)(base & 15) : 0;
    n = RAGGED ? (shift + bytes_ + 15) / 16 : bytes_ / 16;
  }
  // Bytes 16 i - shift ... of row `src`, that is, what piece i of this row would
  // be if it held that row; neighbours' bytes where they are not the row's.
  __device__ __forceinline__ uint4 of(const void* p, int64_t src, int64_t total, int i) const {
    const int64_t at = src * bytes + (int64_t)i * 16 - shift;
    if (!RAGGED) return __ldg(reinterpret_cast<const uint4*>((const char*)p + at));
    const int sh = (int)(at & 15);
    const uint4 lo = load_inside<E>(p, at - sh, total);
    if (sh == 0) return lo;
    return shift_bytes(lo, load_inside<E>(p, at - sh + 16, total), sh);
  }
  __device__ __forceinline__ void put(void* p, int i, const uint4& q) const {
    char* o = (char*)p + base + (int64_t)i * 16 - shift;
    const int c = i * 16 - shift;
    if (!RAGGED || (c >= 0 && c + 16 <= bytes)) {
      *reinterpret_cast<uint4*>(o) = q;
    } else {
      union {
        uint4 q;
        E e[16 / sizeof(E)];
      } u;
      u.q = q;
#pragma unroll
      for (int m = 0; m < (int)(16 / sizeof(E)); ++m)
        if (c + m * (int)sizeof(E) >= 0 && c + m * (int)sizeof(E) < bytes)
          *reinterpret_cast<E*>(o + m * sizeof(E)) = u.e[m];
    }
  }
};

template <typename E, bool RAGGED>
__global__ void __launch_bounds__(256)
permute_kernel(const void* __restrict__ x, const float* __restrict__ scales,
               const int* __restrict__ position, const int* __restrict__ offsets,
               void* __restrict__ out, float* __restrict__ out_scales, int64_t T, int k, int n_exp,
               int bytes) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  if (t >= T) return;
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows), f0 = t * k;
  const int* pos = position + f0;
  const int w0 = blockIdx.y * blockDim.x + threadIdx.x, step = gridDim.y * blockDim.x;
  if constexpr (RAGGED) {
    for (int j = 0; j < k; ++j) {
      const int p = pos[j];
      if (p >= 0 && p < rows) {
        const Span16<E, true> o(p, bytes);
        for (int i = w0; i < o.n; i += step) o.put(out, i, o.of(x, t, T * bytes, i));
      }
      if (f0 + j >= end) {
        const Span16<E, true> o(f0 + j, bytes);
        for (int i = w0; i < o.n; i += step) o.put(out, i, make_uint4(0u, 0u, 0u, 0u));
      }
    }
  } else {
    const int per = bytes / 16;
    uint4* o = (uint4*)out;
    for (int w = w0; w < per; w += step) {
      const uint4 v = __ldg((const uint4*)x + t * per + w);
      for (int j = 0; j < k; ++j) {
        const int p = pos[j];
        if (p >= 0 && p < rows) o[(int64_t)p * per + w] = v;
        if (f0 + j >= end) o[(f0 + j) * per + w] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  if (scales && w0 == 0) {
    const float s = scales[t];
    for (int j = 0; j < k; ++j) {
      const int p = pos[j];
      if (p >= 0 && p < rows) out_scales[p] = s;
      if (f0 + j >= end) out_scales[f0 + j] = 0.f;
    }
  }
}

template <bool F32, bool RAGGED>
__global__ void __launch_bounds__(256, RAGGED ? 2 : 4)
unpermute_kernel(const void* __restrict__ z, const int* __restrict__ position,
                 const float* __restrict__ weights, const void* residual, void* y, int64_t T, int k,
                 int bytes) {
  using E = typename Row<F32>::elem;
  constexpr int V = Row<F32>::kVec;
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  if (t >= T) return;
  const int64_t rows = T * k;
  const int* pos = position + t * k;
  const float* wt = weights ? weights + t * k : nullptr;
  const Span16<E, RAGGED> o(t, bytes);
  for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < o.n; i += gridDim.y * blockDim.x) {
    // (the residual is used only after the first rows' loads are under way)
    uint4 rq = make_uint4(0u, 0u, 0u, 0u);
    if (residual) {
      const int64_t at = o.base - o.shift + (int64_t)i * 16;
      rq = RAGGED ? load_inside<E>(residual, at, T * bytes) : load_once((const char*)residual + at);
    }
    float acc[V];
    for (int j0 = 0; j0 == 0 || j0 < k; j0 += kBatch) {
      uint4 q[kBatch];
      float c[kBatch];
      bool live[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int p = j0 + b < k ? pos[j0 + b] : -1;
        live[b] = p >= 0 && p < rows;
        c[b] = !live[b] ? 0.f : wt ? wt[j0 + b] : 1.f;
        if (live[b]) q[b] = o.of(z, p, rows * bytes, i);
      }
      if (j0 == 0) unpack<F32>(rq, acc);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!live[b]) continue;
        float v[V];
        unpack<F32>(q[b], v);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(c[b], v[e], acc[e]);
      }
    }
    o.put(y, i, pack<F32>(acc));
  }
}

// The sums over a warp of v[0 ... 7]; lane 4 j (and its three neighbours) ends
// with that of v[j].  Halves of the values change sides, so that there are 9
// exchanges and not 40.
__device__ __forceinline__ float warp_sums8(float (&v)[8], int lane) {
#pragma unroll
  for (int h = 4, o = 16; h >= 1; h >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], o);
      v[i] = (up ? v[i + h] : v[i]) + other;
    }
  }
  float s = v[0];
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  return s;
}

// blockDim.x threads to a token; the warps' sums of the dot products meet in
// shared memory.
template <bool F32, bool RAGGED>
__global__ void __launch_bounds__(256, RAGGED ? 2 : 3)
unpermute_backward_kernel(const void* __restrict__ dy, const void* __restrict__ z,
                          const int* __restrict__ position, const int* __restrict__ offsets,
                          const float* __restrict__ weights, void* __restrict__ dz,
                          float* __restrict__ dweights, int64_t T, int k, int n_exp, int bytes) {
  using E = typename Row<F32>::elem;
  constexpr int V = Row<F32>::kVec;
  __shared__ float red[8][kBatch];   // by warp of the CTA
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  const bool here = t < T;
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows), f0 = t * k;
  const int warps = blockDim.x >> 5;   // of a token
  const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, l = threadIdx.x & 31;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    int p[kBatch];
    float c[kBatch], dot[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool in = here && j0 + b < k;
      p[b] = in ? position[f0 + j0 + b] : -1;
      if (p[b] >= rows) p[b] = -1;
      c[b] = in && p[b] >= 0 ? weights[f0 + j0 + b] : 0.f;
      dot[b] = 0.f;
    }
    if constexpr (RAGGED) {
      // in the pieces of z's and dz's row, so that these move as they are
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (p[b] >= 0) {
          const Span16<E, true> o(p[b], bytes);
          for (int i = threadIdx.x; i < o.n; i += blockDim.x) {
            const uint4 zq = load_inside<E>(z, o.base - o.shift + (int64_t)i * 16, rows * bytes);
            float g[V], v[V];
            unpack<F32>(o.of(dy, t, T * bytes, i), g);
            unpack<F32>(zq, v);
            const int c0 = i * V - o.shift / (16 / V), d = bytes / (16 / V);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const bool own = c0 + e >= 0 && c0 + e < d;
              dot[b] = own ? fmaf(g[e], v[e], dot[b]) : dot[b];
              g[e] *= c[b];
            }
            o.put(dz, i, pack<F32>(g));
          }
        }
      }
    } else {
      for (int i = threadIdx.x; here && i < bytes / 16; i += blockDim.x) {
        uint4 q[kBatch];
        const uint4 gq = __ldg(reinterpret_cast<const uint4*>((const char*)dy + t * bytes) + i);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (p[b] >= 0) q[b] = load_once((const char*)z + (int64_t)p[b] * bytes + (int64_t)i * 16);
        float g[V];
        unpack<F32>(gq, g);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (p[b] < 0) continue;
          float v[V];
          unpack<F32>(q[b], v);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dot[b] = fmaf(g[e], v[e], dot[b]);
            v[e] = c[b] * g[e];
          }
          *reinterpret_cast<uint4*>((char*)dz + (int64_t)p[b] * bytes + (int64_t)i * 16) = pack<F32>(v);
        }
      }
    }
    // rows of no pair
    for (int j = j0; here && j < k && j < j0 + kBatch; ++j) {
      if (f0 + j < end) continue;
      const Span16<E, RAGGED> o(f0 + j, bytes);
      for (int i = threadIdx.x; i < o.n; i += blockDim.x) o.put(dz, i, make_uint4(0u, 0u, 0u, 0u));
    }
    const float s = warp_sums8(dot, l);
    if ((l & 3) == 0) red[warp][l >> 2] = s;
    __syncthreads();
    if (here && threadIdx.x < kBatch && j0 + (int)threadIdx.x < k) {
      float v = 0.f;
      for (int i = 0; i < warps; ++i) v += red[threadIdx.y * warps + i][threadIdx.x];
      dweights[f0 + j0 + threadIdx.x] = v;
    }
    if (j0 + kBatch < k) __syncthreads();
  }
}

// Threads for a row of `per` pieces: a power of two, 32 ... 256.
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

int64_t pieces_of(int64_t bytes) { return bytes % 16 ? bytes / 16 + 2 : bytes / 16; }

template <typename E, bool RAGGED>
cudaError_t permute_rows(const PermuteCall& c, cudaStream_t st) {
  const int64_t bytes = c.d * c.elem, per = pieces_of(bytes);
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(permute_kernel<E, RAGGED>, grid_of(c.T, per, block), block, 0, st, c.x,
                        c.scales, c.position, c.offsets, c.out, c.out_scales, c.T, (int)c.k,
                        (int)c.E, (int)bytes);
}

template <bool F32, bool RAGGED>
cudaError_t unpermute_rows(const UnpermuteCall& c, int64_t bytes, cudaStream_t st) {
  const int64_t per = pieces_of(bytes);
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(unpermute_kernel<F32, RAGGED>, grid_of(c.T, per, block), block, 0, st, c.z,
                        c.position, c.weights, c.residual, c.y, c.T, (int)c.k, (int)bytes);
}

template <bool F32, bool RAGGED>
cudaError_t backward_rows(const UnpermuteBackwardCall& c, int64_t bytes, cudaStream_t st) {
  const int tx = row_threads(pieces_of(bytes));
  const dim3 block(tx, 256 / tx);
  return launch_chained(unpermute_backward_kernel<F32, RAGGED>,
                        dim3((unsigned)((c.T + block.y - 1) / block.y)), block, 0, st, c.dy, c.z,
                        c.position, c.offsets, c.weights, c.dz, c.dweights, c.T, (int)c.k,
                        (int)c.E, (int)bytes);
}

}  // namespace

cudaError_t launch_permute(const PermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.k == 0 || (c.d == 0 && !c.scales)) return cudaSuccess;
  if (c.d * c.elem % 16 == 0) return permute_rows<uint8_t, false>(c, st);
  if (c.elem == 4) return permute_rows<uint32_t, true>(c, st);
  if (c.elem == 2) return permute_rows<uint16_t, true>(c, st);
  return permute_rows<uint8_t, true>(c, st);
}

cudaError_t launch_unpermute(const UnpermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.d == 0) return cudaSuccess;
  const int64_t bytes = c.d * (c.f32 ? 4 : 2);
  if (c.f32)
    return bytes % 16 ? unpermute_rows<true, true>(c, bytes, st)
                      : unpermute_rows<true, false>(c, bytes, st);
  return bytes % 16 ? unpermute_rows<false, true>(c, bytes, st)
                    : unpermute_rows<false, false>(c, bytes, st);
}

cudaError_t launch_unpermute_backward(const UnpermuteBackwardCall& c, int num_sms,
                                      cudaStream_t st) {
  if (c.T == 0 || c.k == 0) return cudaSuccess;
  const int64_t bytes = c.d * (c.f32 ? 4 : 2);
  if (c.f32)
    return bytes % 16 ? backward_rows<true, true>(c, bytes, st)
                      : backward_rows<true, false>(c, bytes, st);
  return bytes % 16 ? backward_rows<false, true>(c, bytes, st)
                    : backward_rows<false, false>(c, bytes, st);
}

}  // namespace swg
