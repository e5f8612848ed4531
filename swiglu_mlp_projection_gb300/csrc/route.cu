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
//
// A warp takes a token, a lane 1 ... 32 neighbouring experts in registers: the
// scores, the groups' ranks and the choices need only shuffles and warp-wide
// maxima, and the logits are read once.  Up to 16 tokens one block also sorts
// (one launch).  Above, the routing's blocks leave their counts per expert, and
// scatter_kernel, with the same split of the tokens, places the choices: each
// block adds up all blocks' counts itself, so that there is no third launch and
// no atomic whose order decides a place.
//
// What bounds it, on a GB300 (in a graph): 16384 tokens, E = 256, k = 8,
// sigmoid, bias, 4 of 8 groups: 25.9 us, where the 18.9 MB would take 2.8.
// route_kernel issues 1020 warp instructions per token and keeps the issue slots
// 67 % busy; the scatter's chain (counts, offsets, places) is L2 latency.  5001
// tokens, E = 60: 8.6 us, latency of the two kernels.  One token: 3.6 us, launch.
// Reading the next token's row ahead (prefetch) changed nothing: 26.0 us.
// Dispatch alone: 4096 tokens, k = 8, E = 64 6.5 us, 40000 tokens, E = 256 10.7.
#include "common.cuh"
#include "grouped.h"
#include "tc_common.cuh"

namespace swg {
namespace {

constexpr unsigned kAll = 0xffffffffu;
// Threads per block of the routing and of the sort.  Up to 256 experts a token
// takes 64 registers per thread, so that 32 warps fit on an SM; above that the
// scores alone take 16 or 32 registers, and 16 warps fit.
constexpr int block_threads(int64_t E) { return E <= 256 ? 1024 : 512; }
constexpr int vpl_threads(int vpl) { return vpl <= 8 ? 1024 : 512; }
// A block that routes a few tokens and sorts them by itself: its latency is
// that of its barriers and of clearing the warps' counts.
constexpr int kFewThreads = 256;

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

__device__ __forceinline__ float sigmoid(float v) { return __frcp_rn(1.0f + expf(-v)); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  int* ids;
  float* weights;
  int64_t T;
  int E, k, score_sigmoid, groups, topk_groups, group_top2, renormalize, logits_f32;
  int vec;   // rows of logits start on 16-byte boundaries
  float scale;
};

// The sorted choices' outputs and scratch.
struct SortArgs {
  const int* ids;
  int* offsets;
  int* order;
  int* position;
  int64_t R;       // choices
  int64_t seg;     // choices per block
  int E;
  int* counts;     // [blocks][count_stride(E)]: choices of its segment each block found
};
__host__ __device__ constexpr int count_stride(int E) { return (E + 3) / 4 * 4; }

// VPL values of row t, experts lane VPL ..; -inf past E and for NaN.
template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float* l) {
  const int e0 = lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = -INFINITY;
  if (a.logits_f32) {
    const float* src = (const float*)a.logits + t * a.E + e0;
    if (VPL >= 4 && a.vec) {   // E is a multiple of 4
#pragma unroll
      for (int i = 0; i < VPL; i += 4)
        if (e0 + i < a.E) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(src + i));
          l[i] = q.x;
          if constexpr (VPL >= 4) { l[i + 1] = q.y; l[i + 2] = q.z; l[i + 3] = q.w; }
        }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < a.E) l[i] = __ldg(src + i);
    }
  } else {
    const uint16_t* src = (const uint16_t*)a.logits + t * a.E + e0;
    if (VPL >= 8 && a.vec) {   // E is a multiple of 8
#pragma unroll
      for (int i = 0; i < VPL; i += 8)
        if (e0 + i < a.E) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(src + i));
          if constexpr (VPL >= 8) {
            l[i] = bf16_lo(q.x); l[i + 1] = bf16_hi(q.x);
            l[i + 2] = bf16_lo(q.y); l[i + 3] = bf16_hi(q.y);
            l[i + 4] = bf16_lo(q.z); l[i + 5] = bf16_hi(q.z);
            l[i + 6] = bf16_lo(q.w); l[i + 7] = bf16_hi(q.w);
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < a.E) l[i] = bf16_lo(__ldg(src + i));
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) l[i] = l[i] > -INFINITY ? l[i] : -INFINITY;   // NaN: -inf
}

// Larger and second of the pairs (b0, b1) and (c0, c1), each in order.
__device__ __forceinline__ void merge_two(float& b0, float& b1, float c0, float c1) {
  b1 = fmaxf(fminf(b0, c0), fmaxf(b1, c1));
  b0 = fmaxf(b0, c0);
}

// Keys of the experts outside the kept groups become 0.  cand: the values a
// group is ranked by, -inf for experts that cannot be chosen.
template <int VPL>
__device__ __forceinline__ void limit_groups(const RouteArgs& a, int lane, const float* cand,
                                             unsigned* key, float* vals) {
  const int size = a.E / a.groups;
  unsigned mine = 0u;   // lane g: group g's key
  const int lpg = size / VPL;   // lanes per group, where groups are whole lanes
  const bool aligned = lpg * VPL == size && lpg > 0 && (lpg & (lpg - 1)) == 0;
  const int own = aligned ? lane / lpg : 0;   // this lane's group
  if (aligned) {
    float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) merge_two(b0, b1, cand[i], -INFINITY);
    for (int o = 1; o < lpg; o <<= 1) {
      const float c0 = __shfl_xor_sync(kAll, b0, o), c1 = __shfl_xor_sync(kAll, b1, o);
      merge_two(b0, b1, c0, c1);
    }
    const unsigned k = sort_key(a.group_top2 && b1 > -INFINITY ? b0 + b1 : b0);
    // lane g takes group g's key (the lanes of a group hold the same one)
    const int from = lane * lpg;
    mine = __shfl_sync(kAll, k, from & 31);
    if (lane >= a.groups) mine = 0u;
  } else {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i < a.E) vals[lane * VPL + i] = cand[i];
    __syncwarp();
    if (lane < a.groups) {
      float b0 = -INFINITY, b1 = -INFINITY;
      for (int q = 0; q < size; ++q) {
        int i = q + lane;   // start apart: other banks
        if (i >= size) i %= size;
        merge_two(b0, b1, vals[lane * size + i], -INFINITY);
      }
      mine = sort_key(a.group_top2 && b1 > -INFINITY ? b0 + b1 : b0);
    }
  }
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    const unsigned o = __shfl_sync(kAll, mine, g);
    better += (o > mine || (o == mine && g < lane)) ? 1 : 0;
  }
  const unsigned kept = __ballot_sync(kAll, lane < a.groups && better < a.topk_groups);
  if (aligned) {
    if (own >= a.groups || !((kept >> own) & 1u)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e >= a.E || !((kept >> (e / size)) & 1u)) key[i] = 0u;
    }
  }
}

// A lane's three largest keys that are not used (0: none), the first of equal
// ones first, and where they are.
struct Best {
  unsigned key[3];
  int at[3];
};
template <int VPL>
__device__ __forceinline__ Best three_best(const unsigned* key, unsigned used) {
  Best b{};
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const unsigned q = (used >> i) & 1u ? 0u : key[i];
    const bool p0 = q > b.key[0], p1 = q > b.key[1], p2 = q > b.key[2];
    b.key[2] = p1 ? b.key[1] : p2 ? q : b.key[2];
    b.at[2] = p1 ? b.at[1] : p2 ? i : b.at[2];
    b.key[1] = p0 ? b.key[0] : p1 ? q : b.key[1];
    b.at[1] = p0 ? b.at[0] : p1 ? i : b.at[1];
    b.key[0] = p0 ? q : b.key[0];
    b.at[0] = p0 ? i : b.at[0];
  }
  return b;
}

// One warp, one token.  Lane l holds experts l VPL .. l VPL + VPL - 1, so the
// lowest lane with the largest key holds the lowest index.  vals: E floats of
// shared memory of the warp's own.  Lane j < k returns choice j.  ALL: the choice
// needs every expert's score (a bias, or groups ranked by sums of scores);
// otherwise it goes by logits, s is the logit or the exponential, and only the
// chosen experts' scores are finished (8192 tokens, E = 256, sigmoid: 12.9
// against 14.2 us; 5001 tokens, E = 60, softmax: 8.6 against 9.4).
template <int VPL, bool ALL>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t, int lane,
                                           const float* bias, float* vals, float* weight) {
  float l[VPL], s[VPL];
  unsigned key[VPL];
  load_logits<VPL>(a, t, lane, l);
  float sum = 0.f;
  if (a.score_sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = ALL ? sigmoid(l[i]) : l[i];
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // (an infinite logit has exp(inf - inf) = 1)
      s[i] = l[i] > -INFINITY ? (l[i] == m ? 1.0f : expf(l[i] - m)) : 0.f;
      sum += s[i];
    }
    sum = warp_sum(sum);
    if (ALL && sum > 0.f) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = s[i] / sum;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (ALL && a.bias && l[i] > -INFINITY) l[i] = s[i] + bias[i];
    key[i] = sort_key(l[i]);
  }
  if (a.groups > 1) {
    float cand[VPL];
    const bool scores = ALL && a.group_top2 && !a.bias;   // the top-two sum is of scores
#pragma unroll
    for (int i = 0; i < VPL; ++i) cand[i] = key[i] ? (scores ? s[i] : l[i]) : -INFINITY;
    limit_groups<VPL>(a, lane, cand, key, vals);
  }
  // the scores, for the lanes that end up with a choice
  __syncwarp();
  if constexpr (VPL >= 4) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<float4*>(vals + lane * VPL + i) =
          make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) vals[lane * VPL + i] = s[i];
  }
  __syncwarp();
  // k times the best that is left; lane j keeps choice j.  A lane knows its
  // three best and looks through its values again only when all of them have
  // been chosen: few lanes hold four of a token's choices.
  unsigned used = 0u;
  int have = 3;
  Best b = three_best<VPL>(key, used);
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    const unsigned top = __reduce_max_sync(kAll, b.key[0]);
    if (top == 0u) break;
    const int owner = __ffs(__ballot_sync(kAll, b.key[0] == top)) - 1;
    const int id = owner * VPL + __shfl_sync(kAll, b.at[0], owner);
    if (lane == j) my_id = id;
    const bool mine = lane == owner;
    if (mine) {
      used |= 1u << b.at[0];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b.key[i] = b.key[i + 1];
        b.at[i] = b.at[i + 1];
      }
      --have;
    }
    if (VPL > 3 && __any_sync(kAll, have == 0)) {
      if (have == 0) {
        b = three_best<VPL>(key, used);
        have = 3;
      }
    }
  }
  float w = 0.f;
  if (my_id >= 0) {
    w = vals[my_id];
    if (!ALL) w = a.score_sigmoid ? sigmoid(w) : w / sum;   // (sum >= 1: some logit can be chosen)
  }
  if (a.renormalize) {
    const float total = warp_sum(w);
    if (total > 0.f) w = w / total;
  }
  *weight = w * a.scale;
  return my_id;
}

// Stable scatter of the choices of this block's segment.  Each warp has a
// contiguous part of them: offsets, the earlier blocks' counts and the earlier
// warps' give every (warp, expert) its first place, and a warp places 32
// choices at a time, equal ones in lane order.  Shared memory: s_place
// [warps][E], s_tot [E + 1], s_before [E].
template <int THREADS>
__device__ void scatter_block(const SortArgs& a, const int* ids, int* s_place) {
  constexpr int kWarps = THREADS / 32, kRouteThreads = THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  const int nb = (int)gridDim.x, blk = (int)blockIdx.x;
  int* s_tot = s_place + kWarps * E;
  int* s_before = s_tot + E + 1;
  const int64_t r0 = (int64_t)blk * a.seg < a.R ? (int64_t)blk * a.seg : a.R;
  const int64_t r1 = r0 + a.seg < a.R ? r0 + a.seg : a.R;
  for (int i = threadIdx.x; i < kWarps * E; i += kRouteThreads) s_place[i] = 0;
  __syncthreads();
  int64_t part = (r1 - r0 + kWarps - 1) / kWarps;
  part = (part + 31) / 32 * 32;
  const int64_t w0 = r0 + warp * part;
  const int64_t w1 = w0 + part < r1 ? w0 + part : r1;
  // (the first 32 choices are loaded here and counted further down, with other
  // loads under way)
  const int e_first = w0 + lane < w1 ? ids[w0 + lane] : -1;
  auto count_own = [&]() {
    if (e_first >= 0 && e_first < E) atomicAdd(&s_place[warp * E + e_first], 1);
    for (int64_t r = w0 + lane + 32; r < w1; r += 32) {
      const int e = ids[r];
      if (e >= 0 && e < E) atomicAdd(&s_place[warp * E + e], 1);
    }
  };
  if (nb > 1) {
    // All blocks' counts, and those of the blocks before: `parts` threads per
    // four experts, each over a range of blocks, kBatch loads at a time (an L2
    // round trip each).
    constexpr int kBatch = 10;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) s_tot[e] = s_before[e] = 0;
    __syncthreads();
    const int stride = count_stride(E), quads = stride / 4;
    const int parts = quads < kRouteThreads ? kRouteThreads / quads : 1;
    const int span = (nb + parts - 1) / parts;
    for (int i = threadIdx.x; i < parts * quads; i += kRouteThreads) {
      const int p = i / quads, e = (i - p * quads) * 4;
      const int b0 = p * span, b1 = b0 + span < nb ? b0 + span : nb;
      int4 all = make_int4(0, 0, 0, 0), before = all;
      for (int b = b0; b < b1; b += kBatch) {
        int4 c[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
          c[q] = b + q < b1
                     ? __ldcg(reinterpret_cast<const int4*>(a.counts + (int64_t)(b + q) * stride + e))
                     : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          all.x += c[q].x; all.y += c[q].y; all.z += c[q].z; all.w += c[q].w;
          if (b + q < blk) {
            before.x += c[q].x; before.y += c[q].y; before.z += c[q].z; before.w += c[q].w;
          }
        }
      }
      const int va[4] = {all.x, all.y, all.z, all.w};
      const int vb[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (what pads a row of counts is 0 and adds nothing)
        if (va[j]) atomicAdd(&s_tot[e + j], va[j]);
        if (vb[j]) atomicAdd(&s_before[e + j], vb[j]);
      }
    }
    count_own();
    __syncthreads();
  } else {
    count_own();
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all += s_place[w * E + e];
      s_tot[e] = all;
      s_before[e] = 0;
    }
    __syncthreads();
  }
  // exclusive prefix of the totals: the experts' offsets (a lane has
  // consecutive experts, so that one scan of the warp does)
  if (warp == 0) {
    const int per = (E + 31) / 32, e0 = lane * per;
    const int e1 = e0 + per < E ? e0 + per : E;
    int own = 0;
    for (int e = e0; e < e1; ++e) own += s_tot[e];
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_tot[E] = inc;
    int run = inc - own;
    for (int e = e0; e < e1; ++e) {
      const int c = s_tot[e];
      s_tot[e] = run;
      run += c;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    int run = s_tot[e] + s_before[e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int c = s_place[w * E + e];
      s_place[w * E + e] = run;
      run += c;
    }
  }
  if (blk == 0)
    for (int e = threadIdx.x; e <= E; e += kRouteThreads) a.offsets[e] = s_tot[e];
  __syncthreads();
  for (int64_t b = w0; b < w1; b += 32) {
    const int64_t r = b + lane;
    int e = -1;
    if (r < w1) {
      e = ids[r];
      if (e < 0 || e >= E) e = -1;
    }
    const unsigned same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int place = -1;
    if (e >= 0) place = s_place[warp * E + e] + rank;
    __syncwarp();
    if (e >= 0 && rank == 0) s_place[warp * E + e] += __popc(same);
    __syncwarp();
    if (r < w1) {
      a.position[r] = place;
      if (place >= 0) a.order[place] = (int)r;
    }
  }
  // places that no choice takes
  for (int64_t r = (int64_t)s_tot[E] + (int64_t)blk * kRouteThreads + threadIdx.x; r < a.R;
       r += (int64_t)nb * kRouteThreads)
    a.order[r] = -1;
}

enum SortMode : int { kNoSort = 0, kSortHere = 1, kCount = 2 };

// Routing.  kSortHere: one block, which also sorts its choices.  kCount: block
// b has a contiguous range of tokens and leaves its experts' counts for the
// scatter kernel.
constexpr int route_threads(int vpl, int sort) {
  return sort == kSortHere ? kFewThreads : vpl_threads(vpl);
}

template <int VPL, int SORT, bool ALL>
__global__ void __launch_bounds__(route_threads(VPL, SORT), 1)
route_kernel(const RouteArgs a, const SortArgs so) {
  constexpr int kRouteThreads = route_threads(VPL, SORT), kWarps = kRouteThreads / 32;
  extern __shared__ __align__(16) int s_mem[];
  // scores of the warps' tokens (32 VPL each); afterwards (kSortHere) the sort's
  float* vals = reinterpret_cast<float*>(s_mem) + (threadIdx.x >> 5) * (32 * VPL);
  int* s_cnt = s_mem + kWarps * 32 * VPL;   // [E]
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (SORT == kCount) {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_cnt[e] = 0;
    __syncthreads();
  }
  const int64_t per = (a.T + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = (int64_t)blockIdx.x * per;
  const int64_t t1 = t0 + per < a.T ? t0 + per : a.T;
  float bias[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    bias[i] = ALL && a.bias && lane * VPL + i < a.E ? a.bias[lane * VPL + i] : 0.f;
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    float w;
    const int id = route_token<VPL, ALL>(a, t, lane, bias, vals, &w);
    if (lane < a.k) {
      a.ids[t * a.k + lane] = id;
      a.weights[t * a.k + lane] = w;
      if (SORT == kCount && id >= 0) atomicAdd(&s_cnt[id], 1);
    }
  }
  if constexpr (SORT == kSortHere) {
    __syncthreads();
    scatter_block<kRouteThreads>(so, a.ids, s_mem);
  }
  if constexpr (SORT == kCount) {
    __syncthreads();
    const int stride = count_stride(a.E);
    for (int e = threadIdx.x; e < stride; e += kRouteThreads)
      so.counts[(int64_t)blockIdx.x * stride + e] = e < a.E ? s_cnt[e] : 0;
  }
}

// Counts of each block's segment of given choices.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
count_kernel(const SortArgs a) {
  constexpr int kRouteThreads = THREADS;
  extern __shared__ int s_mem[];
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_mem[e] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * a.seg, r1 = r0 + a.seg < a.R ? r0 + a.seg : a.R;
  for (int64_t r = r0 + threadIdx.x; r < r1; r += kRouteThreads) {
    const int e = a.ids[r];
    if (e >= 0 && e < a.E) atomicAdd(&s_mem[e], 1);
  }
  __syncthreads();
  const int stride = count_stride(a.E);
  for (int e = threadIdx.x; e < stride; e += kRouteThreads)
    a.counts[(int64_t)blockIdx.x * stride + e] = e < a.E ? s_mem[e] : 0;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
scatter_kernel(const SortArgs a) {
  extern __shared__ int s_mem[];
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  scatter_block<THREADS>(a, a.ids, s_mem);
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

size_t sort_smem(int64_t E) {
  return (size_t)((block_threads(E) / 32 + 2) * E + 1) * sizeof(int);
}

// Blocks of a sort of R choices: one up to 2048 of them, else up to one per SM.
int64_t sort_blocks(int64_t R, int num_sms) {
  if (R <= 2048) return 1;
  const int64_t nb = (R + 511) / 512;
  return nb < num_sms ? nb : num_sms;
}

// Tokens that one block routes and sorts by itself (one launch).
constexpr int64_t kOneBlockTokens = 16;

// Blocks of the routing: 16 tokens or more each, up to one block per SM.
int64_t route_blocks(int64_t T, int num_sms) {
  const int64_t nb = (T + 15) / 16;
  return nb < 1 ? 1 : nb < num_sms ? nb : num_sms;
}

// (up to 74 KB at 1024 experts)
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int VPL, bool ALL>
cudaError_t launch_route_as(const RouteArgs& a, const SortArgs& so, int mode, unsigned grid,
                             cudaStream_t st) {
  constexpr int threads = vpl_threads(VPL);
  // the warps' scores and the block's counts, or the sort's
  size_t smem = (size_t)(threads * VPL + a.E) * sizeof(int);
  if (smem < sort_smem(a.E)) smem = sort_smem(a.E);
  cudaError_t e;
  if (mode == kSortHere) {
    if ((e = allow_smem(route_kernel<VPL, kSortHere, ALL>, smem)) != cudaSuccess) return e;
    return launch_pdl(route_kernel<VPL, kSortHere, ALL>, 1, kFewThreads, smem, st, a, so);
  }
  if (mode == kCount) {
    if ((e = allow_smem(route_kernel<VPL, kCount, ALL>, smem)) != cudaSuccess) return e;
    return launch_pdl(route_kernel<VPL, kCount, ALL>, grid, threads, smem, st, a, so);
  }
  if ((e = allow_smem(route_kernel<VPL, kNoSort, ALL>, smem)) != cudaSuccess) return e;
  return launch_pdl(route_kernel<VPL, kNoSort, ALL>, grid, threads, smem, st, a, so);
}

template <int VPL>
cudaError_t launch_route_vpl(const RouteArgs& a, const SortArgs& so, int mode, unsigned grid,
                             cudaStream_t st) {
  return a.bias || (a.groups > 1 && a.group_top2) ? launch_route_as<VPL, true>(a, so, mode, grid, st)
                                                  : launch_route_as<VPL, false>(a, so, mode, grid, st);
}

template <int THREADS>
cudaError_t launch_scatter(const SortArgs& so, unsigned grid, cudaStream_t st) {
  const size_t smem = sort_smem(so.E);
  cudaError_t e = allow_smem(scatter_kernel<THREADS>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(scatter_kernel<THREADS>, grid, THREADS, smem, st, so);
}

cudaError_t launch_scatter(const SortArgs& so, unsigned grid, cudaStream_t st) {
  // (one block of given choices; 2 to 16 where 17 to 256 tokens were routed)
  if (so.R <= 256) return launch_scatter<kFewThreads>(so, grid, st);
  return block_threads(so.E) == 1024 ? launch_scatter<1024>(so, grid, st)
                                     : launch_scatter<512>(so, grid, st);
}

}  // namespace

size_t dispatch_scratch_bytes(int64_t R, int64_t E, int num_sms) {
  const int64_t nb = sort_blocks(R, num_sms);
  return nb > 1 ? (size_t)nb * count_stride((int)E) * sizeof(int) : 0;
}

size_t route_scratch_bytes(int64_t T, int64_t E, int num_sms) {
  return T > kOneBlockTokens ? (size_t)route_blocks(T, num_sms) * count_stride((int)E) * sizeof(int) : 0;
}

cudaError_t launch_route(const RouteCall& c, const SortCall* sort, int num_sms, cudaStream_t st) {
  RouteArgs a;
  a.logits = c.logits;
  a.bias = c.bias;
  a.ids = c.ids;
  a.weights = c.weights;
  a.T = c.T;
  a.E = (int)c.E;
  a.k = (int)c.k;
  a.score_sigmoid = c.sigmoid;
  a.groups = c.groups;
  a.topk_groups = c.topk_groups;
  a.group_top2 = c.group_top2;
  a.renormalize = c.renormalize;
  a.logits_f32 = c.logits_f32;
  a.vec = ((uintptr_t)c.logits & 15u) == 0 && c.E % (c.logits_f32 ? 4 : 8) == 0;
  a.scale = c.scale;
  SortArgs so{};
  int mode = kNoSort;
  const int64_t nb = route_blocks(c.T, num_sms);
  if (sort) {
    // (kCount: the sort's segments are the routing's ranges of tokens)
    mode = c.T <= kOneBlockTokens ? kSortHere : kCount;
    so = SortArgs{c.ids, sort->offsets, sort->order, sort->position, c.T * c.k,
                  mode == kCount ? (c.T + nb - 1) / nb * c.k : c.T * c.k, (int)c.E, sort->scratch};
  }
  const unsigned g = (unsigned)nb;
  cudaError_t e = c.E <= 32    ? launch_route_vpl<1>(a, so, mode, g, st)
                  : c.E <= 64  ? launch_route_vpl<2>(a, so, mode, g, st)
                  : c.E <= 128 ? launch_route_vpl<4>(a, so, mode, g, st)
                  : c.E <= 256 ? launch_route_vpl<8>(a, so, mode, g, st)
                  : c.E <= 512 ? launch_route_vpl<16>(a, so, mode, g, st)
                               : launch_route_vpl<32>(a, so, mode, g, st);
  if (e != cudaSuccess || mode != kCount) return e;
  return launch_scatter(so, g, st);
}

cudaError_t launch_dispatch(const int* ids, const SortCall& s, int64_t R, int64_t E, int num_sms,
                            cudaStream_t st) {
  const int64_t nb = sort_blocks(R, num_sms);
  SortArgs so{ids, s.offsets, s.order, s.position, R, (R + nb - 1) / nb, (int)E, s.scratch};
  cudaError_t e;
  if (nb > 1) {
    e = launch_pdl(count_kernel<512>, (unsigned)nb, 512, (size_t)E * sizeof(int), st, so);
    if (e != cudaSuccess) return e;
  }
  return launch_scatter(so, (unsigned)nb, st);
}

}  // namespace swg
