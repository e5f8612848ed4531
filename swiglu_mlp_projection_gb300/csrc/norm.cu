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
      xr[j] = pc.load(a.x, a.M, i);
      if (a.residual) rr[j] = pc.load(a.residual, a.M, i);
    }
  }
  float t[VPT][V];
  float q = 0.f, m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i >= pc.n) continue;
    unpack<F32>(xr[j], t[j]);
    pc.mask(i, t[j]);
    if (a.residual) {
      float r[V];
      unpack<F32>(rr[j], r);
      pc.mask(i, r);
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
// A CTA takes rows in a fixed order, several at a time where they are short,
// and keeps the columns' sums of dweight over all of them in registers; each
// CTA then writes one row of partial sums, and a second kernel adds those in a
// fixed order.  The next rows are on their way (cp.async, into slots that only
// the copying thread reads) while one is reduced.

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

// 16 bytes of which `bytes` are read and the rest zero.
__device__ __forceinline__ void copy_piece(uint4* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// W warps to a row, two pieces to a thread.
constexpr int kBackPieces = 2;
constexpr int back_threads(int w) { return w <= 8 ? 256 : 32 * w; }
constexpr int back_stages(int w) { return w <= 8 ? 3 : 2; }
constexpr int back_ctas(int w) { return w <= 8 ? 3 : w == 16 ? 2 : 1; }   // per SM

template <bool F32, int W, bool RAGGED>
__global__ void __launch_bounds__(back_threads(W), back_ctas(W))
norm_backward_kernel(const __grid_constant__ BackArgs a) {
  constexpr int V = Row<F32>::kVec, P = kBackPieces, T = back_threads(W), S = back_stages(W);
  constexpr int R = T / 32 / W;     // rows at a time
  extern __shared__ uint4 ring[];   // [S][arrays][P][T]: a thread reads what it copied itself
  __shared__ float2 red[2][T / 32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int team = warp / W, lane = threadIdx.x - team * W * 32;
  const int arrays = a.ds ? 3 : 2;
  const int64_t unit = (int64_t)blockIdx.x * R + team, units = (int64_t)gridDim.x * R;
  const int64_t total = a.M * a.d;
  // (ragged: all rows of a team start at one place in their 16 bytes, since
  // `units` is a multiple of 8 or every team has one row at most)
  const Pieces<F32, RAGGED> pc(unit, a.d);
  const auto slot = [&](int stage, int array, int j) {
    return ring + ((stage * arrays + array) * P + j) * T + threadIdx.x;
  };
  const auto fetch = [&](int64_t row, int stage) {
    if (row < a.M) {
      const int64_t first = row * a.d - pc.shift;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int i = lane + j * W * 32;
        if (i >= pc.n) continue;
        const int64_t at = first + (int64_t)i * V;
        // (the last piece of the tensor may be cut short)
        const int bytes = !RAGGED || total - at >= V ? 16 : (int)(total - at) * (16 / V);
        copy_piece(slot(stage, 0, j), (const char*)a.s + at * (16 / V), bytes);
        copy_piece(slot(stage, 1, j), (const char*)a.dy + at * (16 / V), bytes);
        if (a.ds) copy_piece(slot(stage, 2, j), (const char*)a.ds + at * (16 / V), bytes);
      }
    }
    copies_commit();
  };

  float w[P][V], acc[P][V];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = lane + j * W * 32;
    if (i < pc.n) pc.weight(a.weight, a.weight_f32, i, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[j][e] = 0.f;
  }
  const auto piece = [&](int stage, int array, int j, float (&v)[V]) {
    unpack<F32>(*slot(stage, array, j), v);
    pc.mask(lane + j * W * 32, v);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(unit + i * units, i);
  const float inv_d = 1.0f / (float)a.d;
  int side = 0, stage = 0, next = S - 1;
  for (int64_t row = unit; row < a.M; row += units) {
    fetch(row + (S - 1) * units, next);
    copies_wait<S - 1>();
    float q = 0.f, p = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (lane + j * W * 32 >= pc.n) continue;
      float s[V], g[V];
      piece(stage, 0, j, s);
      piece(stage, 1, j, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        q = fmaf(s[e], s[e], q);
        p = fmaf(g[e] * w[j][e], s[e], p);
      }
    }
    q = warp_sum(q);
    p = warp_sum(p);
    if (W > 1) {
      if (l == 0) red[side][warp] = make_float2(q, p);
      // (one barrier a row: the next row writes the other side)
      if (R == 1) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
      const float2 v = l < W ? red[side][team * W + l] : make_float2(0.f, 0.f);
      q = warp_sum(v.x);
      p = warp_sum(v.y);
    }
    const float r = 1.0f / sqrtf(fmaf(q, inv_d, a.eps));
    const float c = r * r * (p * inv_d);
    const int64_t first = row * a.d - pc.shift;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = lane + j * W * 32;
      if (i >= pc.n) continue;
      float s[V], g[V], o[V];
      piece(stage, 0, j, s);
      piece(stage, 1, j, g);
      if (a.ds) {
        piece(stage, 2, j, o);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[j][e] = fmaf(g[e], s[e] * r, acc[j][e]);
        o[e] = fmaf(r, fmaf(g[e], w[j][e], -s[e] * c), o[e]);
      }
      pc.store_at(a.dx, first, i, o);
    }
    side ^= 1;
    stage = stage + 1 == S ? 0 : stage + 1;
    next = next + 1 == S ? 0 : next + 1;
  }
  // The CTA's sums, team after team.
  copies_wait<0>();
  __syncthreads();
  float* part = a.part + (int64_t)blockIdx.x * a.d;
  float* sums = R > 1 ? reinterpret_cast<float*>(ring) + team * a.d : part;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = lane + j * W * 32;
    if (i >= pc.n) continue;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (pc.has(i, e)) sums[pc.col(i) + e] = acc[j][e];
  }
  if (R > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += T) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) v += reinterpret_cast<const float*>(ring)[i * a.d + c];
      part[c] = v;
    }
  }
}

// Rows wider than 32 warps' two pieces: a CTA per row reads it twice (the
// second time from L2) and keeps its sums of dweight in shared memory.
template <bool F32, bool RAGGED>
__global__ void __launch_bounds__(1024)
norm_backward_wide_kernel(const __grid_constant__ BackArgs a) {
  constexpr int V = Row<F32>::kVec;
  extern __shared__ float acc[];   // [V][pieces]
  __shared__ float2 red[2][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const Pieces<F32, RAGGED> p0(blockIdx.x, a.d);   // (the rows' shift: as above)
  for (int i = threadIdx.x; i < p0.n; i += 1024)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e * p0.n + i] = 0.f;
  const float inv_d = 1.0f / (float)a.d;
  int side = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, side ^= 1) {
    const Pieces<F32, RAGGED> pc(row, a.d);
    float q = 0.f, p = 0.f;
#pragma unroll 2
    for (int i = threadIdx.x; i < pc.n; i += 1024) {
      float s[V], g[V], w[V];
      unpack<F32>(pc.load(a.s, a.M, i), s);
      unpack<F32>(pc.load(a.dy, a.M, i), g);
      pc.mask(i, s);
      pc.mask(i, g);
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
    __syncthreads();
    q = warp_sum(red[side][l].x);
    p = warp_sum(red[side][l].y);
    const float r = 1.0f / sqrtf(fmaf(q, inv_d, a.eps));
    const float c = r * r * (p * inv_d);
#pragma unroll 2
    for (int i = threadIdx.x; i < pc.n; i += 1024) {
      float s[V], g[V], w[V], o[V];
      unpack<F32>(pc.load(a.s, a.M, i), s);
      unpack<F32>(pc.load(a.dy, a.M, i), g);
      pc.mask(i, s);
      pc.mask(i, g);
      pc.weight(a.weight, a.weight_f32, i, w);
      if (a.ds) {
        unpack<F32>(pc.load(a.ds, a.M, i), o);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[e * pc.n + i] += g[e] * (s[e] * r);
        o[e] = fmaf(r, fmaf(g[e], w[e], -s[e] * c), o[e]);
      }
      pc.store(a.dx, i, o);
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.d;
  for (int i = threadIdx.x; i < p0.n; i += 1024)
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (p0.has(i, e)) part[p0.col(i) + e] = acc[e * p0.n + i];
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

// How the gradient's rows are dealt out: W warps to a row (0: the wide kernel),
// `grid` CTAs.
struct BackShape {
  int warps, grid;
};
BackShape back_shape(int64_t M, int64_t d, bool f32, int num_sms) {
  const int vec = f32 ? 4 : 8;
  const int64_t pieces = d % vec ? d / vec + 2 : d / vec;
  int w = 1;
  while (w <= 32 && 32 * kBackPieces * w < pieces) w *= 2;
  const int rows = w > 32 ? 1 : back_threads(w) / 32 / w;
  int64_t grid = (M + rows - 1) / rows;
  const int64_t most = (int64_t)num_sms * (w > 32 ? 1 : back_ctas(w)) / 8 * 8;
  if (grid > most) grid = most;
  return {w > 32 ? 0 : w, (int)grid};
}

template <bool F32, int W, bool RAGGED>
cudaError_t launch_back_warps(const BackArgs& a, int grid, cudaStream_t st) {
  const auto k = norm_backward_kernel<F32, W, RAGGED>;
  size_t smem = (size_t)back_stages(W) * (a.ds ? 3 : 2) * kBackPieces * back_threads(W) * 16;
  static_assert(back_stages(W) * 2 * kBackPieces * 16 * 32 * W >= 512 * W * 4, "no room for the sums");
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(grid), dim3(back_threads(W)), smem, st, a);
}

template <bool F32, bool RAGGED>
cudaError_t launch_back(const BackArgs& a, const BackShape& s, cudaStream_t st) {
  switch (s.warps) {
    case 1: return launch_back_warps<F32, 1, RAGGED>(a, s.grid, st);
    case 2: return launch_back_warps<F32, 2, RAGGED>(a, s.grid, st);
    case 4: return launch_back_warps<F32, 4, RAGGED>(a, s.grid, st);
    case 8: return launch_back_warps<F32, 8, RAGGED>(a, s.grid, st);
    case 16: return launch_back_warps<F32, 16, RAGGED>(a, s.grid, st);
    case 32: return launch_back_warps<F32, 32, RAGGED>(a, s.grid, st);
  }
  const auto k = norm_backward_wide_kernel<F32, RAGGED>;
  const size_t smem = (size_t)(a.d + 16) * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(s.grid), dim3(1024), smem, st, a);
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
  return (size_t)back_shape(M, d, f32 != 0, num_sms).grid * (size_t)d * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackwardCall& c, float* part, int num_sms,
                                     cudaStream_t st) {
  if (c.d == 0) return cudaSuccess;
  const BackShape s = back_shape(c.M, c.d, c.f32 != 0, num_sms);
  if (c.M > 0) {
    const BackArgs a{c.dy, c.s, c.weight, c.ds, c.dx, part, c.M, (int)c.d, c.eps, c.weight_f32};
    const bool ragged = c.d % (c.f32 ? 4 : 8) != 0;
    const cudaError_t e =
        c.f32 ? (ragged ? launch_back<true, true>(a, s, st) : launch_back<true, false>(a, s, st))
              : (ragged ? launch_back<false, true>(a, s, st) : launch_back<false, false>(a, s, st));
    if (e != cudaSuccess) return e;
  }
  return launch_chained(dweight_kernel, dim3((unsigned)((c.d + kSumCols - 1) / kSumCols)),
                        dim3(kSumCols * kSumRows), 0, st, (const float*)part, s.grid, (int)c.d,
                        c.dweight, c.weight_f32);
}

}  // namespace swg
