// Routing of tokens to experts, and the order in which the experts' products
// read them.
//
// route: scores s = softmax(l) or sigmoid(l) of a token's E logits; the
// candidates are ordered by l (both scores grow with it), or by s + bias where
// there is a balance bias; with groups, only the experts of the topk_groups
// best groups are candidates; the k best candidates are chosen, ties to the
// lowest index, and their weights are s, divided by their sum on request,
// times a factor.  An expert whose logit is -inf or NaN (or whose biased score
// is) cannot be chosen; where fewer than k can be, the rest of the row is
// expert -1 with weight 0.
//
// dispatch: a stable counting sort of the T k choices by expert.
#include "common.cuh"
#include "grouped.h"
#include "tc_common.cuh"

namespace swg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kAll = 0xffffffffu;

// Order-preserving map of f32 to unsigned; -inf and NaN map to 0, which no
// other value does.  (-0 maps to +0: they tie.)
__device__ __forceinline__ unsigned sort_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const unsigned u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int* ids;
  float* weights;
  int64_t T;
  int E, k, sigmoid, groups, topk_groups, group_top2, renormalize, logits_f32;
  float scale;
};

// One warp per token; lane l holds experts l VPL .. l VPL + VPL - 1, so the
// lowest lane with the largest key holds the lowest index.
template <int VPL>
__global__ void __launch_bounds__(kThreads)
route_kernel(const RouteArgs a) {
  extern __shared__ float s_mem[];   // groups: per warp E candidate values, then the groups' keys
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    float l[VPL], s[VPL];
    unsigned key[VPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      l[i] = -INFINITY;
      if (e < E) {
        const float v = a.logits_f32 ? ((const float*)a.logits)[t * E + e]
                                     : bf16_lo(((const uint16_t*)a.logits)[t * E + e]);
        if (v > -INFINITY) l[i] = v;   // NaN counts as -inf
      }
      m = fmaxf(m, l[i]);
    }
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = 1.0f / (1.0f + expf(-l[i]));
    } else {
      m = warp_max(m);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        // (an infinite logit has exp(inf - inf) = 1)
        s[i] = l[i] > -INFINITY ? (l[i] == m ? 1.0f : expf(l[i] - m)) : 0.f;
        sum += s[i];
      }
      sum = warp_sum(sum);
      if (sum > 0.f) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = s[i] / sum;
      }
    }
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      v[i] = l[i];
      if (a.bias && e < E && l[i] > -INFINITY) v[i] = s[i] + a.bias[e];
      key[i] = sort_key(v[i]);
    }
    if (a.groups > 1) {
      // the groups' values: the largest candidate, or the sum of the two largest
      float* vals = s_mem + warp * (E + 32);
      unsigned* gk = reinterpret_cast<unsigned*>(vals + E);
      const bool scores = a.group_top2 && !a.bias;   // the top-two sum is of scores
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        if (e < E) vals[e] = key[i] ? (scores ? s[i] : v[i]) : -INFINITY;
      }
      __syncwarp();
      const int size = E / a.groups;
      unsigned mine = 0u;
      if (lane < a.groups) {
        float b0 = -INFINITY, b1 = -INFINITY;
        for (int q = 0; q < size; ++q) {
          int i = q + lane;   // start apart: other banks
          if (i >= size) i %= size;
          const float x = vals[lane * size + i];
          if (x > b0) {
            b1 = b0;
            b0 = x;
          } else if (x > b1) {
            b1 = x;
          }
        }
        mine = sort_key(a.group_top2 && b1 > -INFINITY ? b0 + b1 : b0);
      }
      gk[lane] = mine;
      __syncwarp();
      int better = 0;
      for (int g = 0; g < a.groups; ++g) {
        const unsigned o = gk[g];
        better += (o > mine || (o == mine && g < lane)) ? 1 : 0;
      }
      const unsigned kept = __ballot_sync(kAll, lane < a.groups && better < a.topk_groups);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        if (e >= E || !((kept >> (e / size)) & 1u)) key[i] = 0u;
      }
    }
    // k times the best that is left; lane j keeps choice j
    int my_id = -1;
    float my_w = 0.f, total = 0.f;
    for (int j = 0; j < a.k; ++j) {
      unsigned best = 0u;
      int bi = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] > best) {
          best = key[i];
          bi = i;
        }
      const unsigned top = __reduce_max_sync(kAll, best);
      if (top == 0u) break;
      const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
      float sv = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == bi) {
          sv = s[i];
          if (lane == owner) key[i] = 0u;
        }
      const int id = __shfl_sync(kAll, lane * VPL + bi, owner);
      const float w = __shfl_sync(kAll, sv, owner);
      total += w;
      if (lane == j) {
        my_id = id;
        my_w = w;
      }
    }
    if (a.renormalize && total > 0.f) my_w = my_w / total;
    if (lane < a.k) {
      a.ids[t * a.k + lane] = my_id;
      a.weights[t * a.k + lane] = my_w * a.scale;
    }
  }
}

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;

// Counts of each block's segment of the choices: hist [blocks][E].
__global__ void __launch_bounds__(kSortThreads)
hist_kernel(const int* __restrict__ ids, int* __restrict__ hist, int64_t R, int E, int64_t seg) {
  extern __shared__ int s_cnt[];
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  for (int e = threadIdx.x; e < E; e += kSortThreads) s_cnt[e] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * seg, r1 = r0 + seg < R ? r0 + seg : R;
  for (int64_t r = r0 + threadIdx.x; r < r1; r += kSortThreads) {
    const int e = ids[r];
    if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
}

// Stable scatter of one block's segment.  Each warp has a contiguous part of
// it: the warps' counts give every (warp, expert) its first place, and a warp
// places 32 choices at a time, equal ones in lane order.
__global__ void __launch_bounds__(kSortThreads)
scatter_kernel(const int* __restrict__ ids, const int* __restrict__ hist, int* __restrict__ offsets,
               int* __restrict__ order, int* __restrict__ position, int64_t R, int E, int64_t seg) {
  extern __shared__ int s_place[];   // [warps][E] counts, then places; then [E] totals
  int* s_tot = s_place + kSortWarps * E;
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nb = gridDim.x;
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) s_place[i] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * seg, r1 = r0 + seg < R ? r0 + seg : R;
  const int64_t part = (seg + kSortWarps - 1) / kSortWarps;
  const int64_t w0 = r0 + warp * part;
  const int64_t w1 = w0 + part < r1 ? w0 + part : r1;
  for (int64_t r = w0 + lane; r < w1; r += 32) {
    const int e = ids[r];
    if (e >= 0 && e < E) atomicAdd(&s_place[warp * E + e], 1);
  }
  __syncthreads();
  // per expert: all blocks' total, and what the blocks before this one hold
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int before = 0, all = 0;
    if (hist) {
      for (int b = 0; b < nb; ++b) {
        const int c = hist[(int64_t)b * E + e];
        if (b < (int)blockIdx.x) before += c;
        all += c;
      }
    } else {
      for (int w = 0; w < kSortWarps; ++w) all += s_place[w * E + e];
    }
    int run = before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = s_place[w * E + e];
      s_place[w * E + e] = run;
      run += c;
    }
    s_tot[e] = all;
  }
  __syncthreads();
  // exclusive prefix of the totals: the experts' offsets
  if (warp == 0) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < E ? s_tot[e] : 0;
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, inc, o);
        if (lane >= o) inc += v;
      }
      if (e < E) s_tot[e] = base + inc - c;
      base += __shfl_sync(kAll, inc, 31);
    }
    if (lane == 0) s_tot[E] = base;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = s_tot[e];
  const int valid = s_tot[E];
  for (int64_t base = w0; base < w1; base += 32) {
    const int64_t r = base + lane;
    int e = -1;
    if (r < w1) {
      e = ids[r];
      if (e < 0 || e >= E) e = -1;
    }
    const unsigned same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int place = -1;
    if (e >= 0) place = s_tot[e] + s_place[warp * E + e] + rank;
    __syncwarp();
    if (e >= 0 && rank == 0) s_place[warp * E + e] += __popc(same);
    __syncwarp();
    if (r < w1) {
      position[r] = place;
      if (place >= 0) order[place] = (int)r;
    }
  }
  // places that no choice takes
  for (int64_t r = (int64_t)valid + (int64_t)blockIdx.x * kSortThreads + threadIdx.x; r < R;
       r += (int64_t)nb * kSortThreads)
    order[r] = -1;
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, size_t smem,
                       cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Choices per block of the sort.
int64_t sort_segment(int64_t R) {
  int64_t seg = 2048;
  while ((R + seg - 1) / seg > 128) seg *= 2;
  return seg;
}

}  // namespace

cudaError_t launch_route(const RouteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0) return cudaSuccess;
  RouteArgs a;
  a.logits = c.logits;
  a.bias = c.bias;
  a.ids = c.ids;
  a.weights = c.weights;
  a.T = c.T;
  a.E = (int)c.E;
  a.k = (int)c.k;
  a.sigmoid = c.sigmoid;
  a.groups = c.groups;
  a.topk_groups = c.topk_groups;
  a.group_top2 = c.group_top2;
  a.renormalize = c.renormalize;
  a.logits_f32 = c.logits_f32;
  a.scale = c.scale;
  int64_t blocks = (c.T + kWarps - 1) / kWarps;
  if (blocks > (int64_t)num_sms * 16) blocks = (int64_t)num_sms * 16;
  const size_t smem = c.groups > 1 ? (size_t)kWarps * (c.E + 32) * sizeof(float) : 0;
  const unsigned g = (unsigned)blocks;
  if (c.E <= 32) return launch_pdl(route_kernel<1>, g, kThreads, smem, st, a);
  if (c.E <= 64) return launch_pdl(route_kernel<2>, g, kThreads, smem, st, a);
  if (c.E <= 128) return launch_pdl(route_kernel<4>, g, kThreads, smem, st, a);
  if (c.E <= 256) return launch_pdl(route_kernel<8>, g, kThreads, smem, st, a);
  if (c.E <= 512) return launch_pdl(route_kernel<16>, g, kThreads, smem, st, a);
  return launch_pdl(route_kernel<32>, g, kThreads, smem, st, a);
}

size_t dispatch_scratch_bytes(int64_t R, int64_t E) {
  const int64_t nb = (R + sort_segment(R) - 1) / sort_segment(R);
  return nb > 1 ? (size_t)nb * E * sizeof(int) : 0;
}

cudaError_t launch_dispatch(const int* ids, int* offsets, int* order, int* position, int64_t R,
                            int64_t E, int* scratch, cudaStream_t st) {
  const int64_t seg = sort_segment(R);
  int64_t nb = (R + seg - 1) / seg;
  if (nb < 1) nb = 1;
  const size_t smem = (size_t)(kSortWarps * E + E + 1) * sizeof(int);   // 36 KB at E = 1024
  if (nb > 1) {
    cudaError_t e = launch_pdl(hist_kernel, (unsigned)nb, kSortThreads, (size_t)E * sizeof(int), st,
                               ids, scratch, R, (int)E, seg);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(scatter_kernel, (unsigned)nb, kSortThreads, smem, st, ids,
                    nb > 1 ? scratch : (int*)nullptr, offsets, order, position, R, (int)E, seg);
}

}  // namespace swg
