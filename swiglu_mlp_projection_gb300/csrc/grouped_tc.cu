// Grouped products on the tensor cores (bf16): every expert's rows of x times
// that expert's weights, in one launch, and the general linear product as the
// case of one group.
//
//   experts, up:    h[r]  = silu(x[t(r)] . W_gate[e]) * (x[t(r)] . W_up[e])
//   experts, down:  z[r]  = h[r] . W_down[e]        (weighted and added up over
//                                                    a token's choices afterwards)
//   linear:         y[m]  = act(x[m] . W + bias) + residual[m]
//
// Rows r are sorted by expert; offsets[e] .. offsets[e + 1] are expert e's.
// They are known on the device only, so the kernel plans its own work: a
// chunk is up to n_max rows of one expert (an expert's rows are spread evenly
// over its chunks), a unit is a chunk and a group of output columns, and the
// grid is one CTA pair per two SMs, whatever the routing.
//
// Orientation: the weights are the MMA's A operand and the rows its B operand
// (D^T = W^T x^T), because the count of rows varies from one to thousands and
// N takes any multiple of 32, where M is 256.  64 experts of 512 rows on
// average, unevenly loaded, would leave 20 % of 256-row tiles empty; chunks of
// up to 256 rows, rounded to 32, leave 7 %.
//
// A pair (cta_group::2) computes 256 rows of W^T times N <= 256 rows of x;
// each CTA stages 128 weight columns and half of the x rows per 64-deep k
// block.  SwiGLU: a CTA's 128 weight columns are 64 gate columns and the 64
// up columns with the same indices, so a unit is 128 columns of h and gate and
// up meet in one CTA (through shared memory, in the epilogue).  Otherwise a
// unit is 256 adjacent output columns.
//
// Units run whole, round robin, as long as they fill the pairs; the units of
// a last, partial wave are cut along K in equal shares (grouped_plan.cuh).  A
// pair whose share ends inside a unit writes the f32 sums so far to the
// workspace.  They are added in k order: in short chunks (32 rows; 64 in the up
// projection) by the last pair to arrive, where they are few, and otherwise by
// a second kernel, linear_join_kernel or the weighted sum that follows the down
// projection anyway.  (The last pair alone took 13 of the router logits' 31 us
// at M = 4096, K = 4096, N = 64; the join takes 4.)  The up projection's longer
// chunks are not cut.  No output depends on an order of arrival.
//
// What bounds it, on a GB300 (6785 GB/s copy, 1878 TFLOP/s bf16 in a library
// product), replayed from a graph in bursts of a few ms:
//   few rows: HBM.  8 experts of d = 4096, d_ff = 14336, 32 tokens: 269 us for
//   1.88 GB (7.0 TB/s).  8 of 64 experts of d = 2048, d_ff = 1024 (67 MB, one
//   token): 16.3 us, 10 of them streaming, the rest the chain from the previous
//   kernel's end through offsets, order, rows and the first stages;
//   many rows: the MMAs, once operands arrive at 32 KB per CTA and k block:
//   one group, 4096 rows, d = 4096, d_ff = 14336 478-491 us (1960-2010 TFLOP/s);
//   64 experts of 512 rows on average 189-195 us (1420 TFLOP/s: chunks have 220
//   columns on average, 7 % of them padding, and the last wave is not full); 8
//   experts, K = 14336: 700 us with the weighted sum (1370 TFLOP/s), 622 for the
//   product alone under a profiler, the tensor pipe active 89 % of it at the
//   power cap's clock (the loads alone take 0.36 us per k block there, 0.24 at
//   K = 4096).  In loops of seconds the cap's clock (1540 MHz) bounds the others
//   too: 224 us for the 64 experts.
#include <atomic>

#include "common.cuh"
#include "grouped.h"
#include "grouped_plan.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "tc_pair.cuh"

namespace swg {
namespace {

using namespace tc;

constexpr int kBK = 64;
// Warps: 0 loads weights (TMA), 1 issues MMAs (rank 0) or relays (rank 1),
// 2-9 are the epilogue (two groups of four, each covering the 128 accumulator
// lanes), 10 and up load rows (one warp of TMA, or four of cp.async).  One warp
// issuing both operands in 16-row boxes took 419 us where this takes 250
// (M = 4096, K = 4096, N = 14336), and four-row TMA gathers 741 us where
// cp.async takes 190 (64 experts' up projection of 4096 tokens).
constexpr int kEpiThreads = 128;                  // one epilogue group
constexpr int kRowWarp = 10;
constexpr int kGatherThreads = 128;
constexpr int threads_of(bool gather) { return kRowWarp * 32 + (gather ? kGatherThreads : 32); }
constexpr uint32_t kChunkBytes = 64 * kBK * 2;    // one 64-column weight box
constexpr uint32_t kABytes = 2 * kChunkBytes;     // a CTA's 128 weight columns
// 10 stages at 32 rows per chunk, 6 at 192 and above.  (8 experts' decode up
// projection, 32 tokens: 269 us with 10 or 9 stages, 276 with 7, 287 with 5.)
constexpr uint32_t kRingBytes = 192u * 1024u;
constexpr int kMaxStages = 12;
constexpr uint32_t kTmemCols = 512;               // two accumulators of up to 256 columns
constexpr int kAccCols = 256;
// An epilogue group's staging.  SwiGLU: halves of 32 rows of gate and up,
// [16][64] f32 each, and 32 rows of h, [32][72] bf16; linear: 16 rows of
// f32, [16][132] (128 columns and 16 bytes, against bank conflicts).
constexpr int kStageCols = 132, kHCols = 72;
constexpr uint32_t kStagingBytes = 2 * 16 * 64 * 4 + 32 * kHCols * 2;
static_assert(kStagingBytes >= 16 * kStageCols * 4, "staging too small");
constexpr size_t kFixedBytes = 1024 + 2 * kStagingBytes + (2 * kMaxStages + 5) * 8 + 64;
static_assert(kFixedBytes + kRingBytes + 2 * (kMaxExperts + 1) * 4 <= 232448,
              "shared memory exceeded");

// Tensor maps of the row operand with boxes of 128, 64, 32 and 16 rows.
struct RowMaps {
  CUtensorMap box[4];
};

struct Args : Work {
  const uint16_t* x;       // gathered rows: [tokens, K]
  int K;
  const int* order;        // up: sorted row -> token * top_k + choice
  int top_k, tokens;
  int stages;
  uint32_t stage_bytes;
  int kmajor;              // weights stored [n_out, K]
  int joined;              // linear: a kernel that adds up shares follows
  int self_join;           // the last pair of a cut unit adds up its shares
  int prefetch_kb;         // linear: k blocks whose weights are asked into L2 early
  void* out;
  int out_f32;
  const void* bias;        // linear
  int bias_f32, act;
  const void* resid;       // linear, in the output's type
  unsigned* counters;      // self_join: two per pair, zero on entry, left at zero
  unsigned* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The same box into L2 only (a hint).
__device__ __forceinline__ void tma_prefetch_l2_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   (uint64_t)map),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// 16 bytes global -> shared, asynchronously; `bytes` 0 writes zeros instead.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// This thread's arrival on `bar` once its cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// (acquires at cluster scope: a stage's other half is the other CTA's)
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// As mbar_wait, for all lanes of a warp (the same answer for each) and a
// barrier given by its shared address.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned* status, uint64_t timeout_ns) {
  if (__all_sync(0xffffffffu, try_wait_at(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  bool up = false;   // gave up
  for (uint32_t i = 1;; ++i) {
    const bool done = try_wait_at(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) up = true;
      if (globaltimer_ns() - t0 > timeout_ns) {
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout);
        up = true;
      }
      if (__any_sync(0xffffffffu, up)) return false;
    }
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// mma_bf16_pair with the descriptors' halves apart: only the low ones change
// from one MMA to the next.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                         uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// mma_commit_pair_mc for both CTAs, the barrier given by its shared address.
__device__ __forceinline__ void commit_pair_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)0x3)
      : "memory");
}

__device__ __forceinline__ bool wait_drain(uint64_t* bar, uint32_t parity, unsigned* status,
                                           uint64_t timeout_ns) {
  int never = 0;
  return mbar_wait(bar, parity, &never, status, timeout_ns);
}

// Lets a producer's loads land (those of the last round of the ring; earlier
// ones have been waited for).
__device__ __forceinline__ void drain_loads(uint64_t* full, int64_t issued, const Args& a) {
  for (int64_t i = issued > a.stages ? issued - a.stages : 0; i < issued; ++i)
    wait_drain(&full[i % a.stages], (uint32_t)((i / a.stages) & 1), a.status, a.timeout_ns);
}

// v sigma(z).  For z < 0 it is v e^z / (1 + e^z): 1 + e^-z ends at z = -88.7,
// where v e^z is still a normal number.  The accurate functions serve f32
// outputs.  bf16 outputs take the fast exponential and divide: the error of
// the exponential grows with |z|, to 2^-16 of the value where e^z ends, well
// below the half ulp (2^-9) of the rounding that follows.
template <bool ACCURATE>
__device__ __forceinline__ float times_sigma(float v, float z) {
  const float e = ACCURATE ? expf(-fabsf(z)) : __expf(-fabsf(z));
  const float n = z >= 0.f ? v : v * e;
  return ACCURATE ? n / (1.0f + e) : __fdividef(n, 1.0f + e);
}

// act(v).  tanh form: 0.5 v (1 + tanh z) = v sigma(2 z),
// z = sqrt(2 / pi) (v + 0.044715 v^3).
template <int ACT, bool ACCURATE>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == kActRelu) return v > 0.f ? v : (v != v ? v : 0.f);
  if constexpr (ACT == kActSilu) return times_sigma<ACCURATE>(v, v);
  if constexpr (ACT == kActGelu) return 0.5f * v * erfcf(-0.70710678118654752f * v);
  if constexpr (ACT == kActGeluTanh)
    return times_sigma<ACCURATE>(v, 1.5957691216057308f * (v + 0.044715f * v * v * v));
  return v;
}

template <int ACT, bool ACCURATE, int N>
__device__ __forceinline__ void activate_all(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = activate<ACT, ACCURATE>(v[i]);
}

template <int N>
__device__ __forceinline__ void activate_n(float* v, int act, bool accurate) {
  switch (act * 2 + (accurate ? 1 : 0)) {
    case kActRelu * 2: case kActRelu * 2 + 1: activate_all<kActRelu, true, N>(v); break;
    case kActSilu * 2: activate_all<kActSilu, false, N>(v); break;
    case kActSilu * 2 + 1: activate_all<kActSilu, true, N>(v); break;
    case kActGelu * 2: case kActGelu * 2 + 1: activate_all<kActGelu, true, N>(v); break;
    case kActGeluTanh * 2: activate_all<kActGeluTanh, false, N>(v); break;
    case kActGeluTanh * 2 + 1: activate_all<kActGeluTanh, true, N>(v); break;
    default: break;
  }
}

// Two f32 -> packed bf16, to nearest even (`lo` in the low half).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t cvt_bf16(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}

// L2 prefetch of the weights of this CTA's first k blocks (linear).
template <int COLS>
__device__ void prefetch_weights(const Args& a, const CUtensorMap& tm_w, const int* s_row,
                                 const int* s_chunk, uint32_t pair, uint32_t pairs, uint32_t rank) {
  const Schedule sch = make_schedule(a, (uint32_t)s_chunk[a.E], pairs);
  WorkIter w(sch, pair);
  uint32_t u;
  int kb0, kb1, left = a.prefetch_kb, e_at = 0;
  while (left > 0 && w.next(a, sch, pairs, u, kb0, kb1)) {
    const Unit un = find_unit<COLS>(a, s_row, s_chunk, u, e_at);
    const int ca = un.col0 + 128 * (int)rank;
    for (int kb = kb0; kb < kb1 && left > 0; ++kb, --left) {
      if (a.kmajor) {
        tma_prefetch_l2_3d(&tm_w, kb * kBK, ca, un.e);
      } else {
        tma_prefetch_l2_3d(&tm_w, ca, kb * kBK, un.e);
        tma_prefetch_l2_3d(&tm_w, ca + 64, kb * kBK, un.e);
      }
    }
  }
}

// v[0 .. 4 NQ) = the sum of `nseg` shares, in order: the first one's, then
// those of the pairs after it.  NS shares are loaded at a time, because a
// share costs an L2 round trip, not its bytes.  `rows` of the chunk are used.
template <int NQ, int NS>
__device__ __forceinline__ void add_shares(float* v, const float* first, const float* rest,
                                           int64_t stride, int nseg, int rows) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < nseg; s0 += NS) {
    float4 t[NS][NQ];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float* src = s0 + s == 0 ? first : rest + (int64_t)(s0 + s - 1) * stride;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        t[s][q] = s0 + s < nseg && 4 * q < rows
                      ? __ldcg(reinterpret_cast<const float4*>(src + q * 512))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        v[4 * q] += t[s][q].x;
        v[4 * q + 1] += t[s][q].y;
        v[4 * q + 2] += t[s][q].z;
        v[4 * q + 3] += t[s][q].w;
      }
  }
}

// The residual at eight neighbouring outputs (element `o`, `left` columns of the
// row remain from there), as it lies in memory.
struct Residual8 {
  uint4 lo, hi;
};

__device__ __forceinline__ Residual8 load_residual8(const Args& a, int64_t o, int left) {
  Residual8 r;
  r.lo = r.hi = make_uint4(0u, 0u, 0u, 0u);
  if (!a.resid) return r;
  if (a.n_out & 7) {   // rows off 16-byte boundaries: element by element
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = 0u;
      if (i < left)
        q[i] = a.out_f32 ? ((const uint32_t*)a.resid)[o + i] : (uint32_t)((const uint16_t*)a.resid)[o + i];
    }
    if (a.out_f32) {
      r.lo = make_uint4(q[0], q[1], q[2], q[3]);
      r.hi = make_uint4(q[4], q[5], q[6], q[7]);
    } else {
      r.lo = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16);
    }
  } else if (a.out_f32) {
    const uint4* p = reinterpret_cast<const uint4*>((const float*)a.resid + o);
    r.lo = p[0];
    r.hi = p[1];
  } else {
    r.lo = *reinterpret_cast<const uint4*>((const uint16_t*)a.resid + o);
  }
  return r;
}

// v + residual, rounded to the output type, to eight neighbouring outputs.
__device__ __forceinline__ void store_row8(const Args& a, int64_t o, int left, float* v,
                                           const Residual8& r) {
  if (a.resid) {
    const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] += a.out_f32 ? __uint_as_float(w[i]) : (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
  if (a.n_out & 7) {   // rows off 16-byte boundaries: element by element
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= left) break;
      if (a.out_f32) ((float*)a.out)[o + i] = v[i];
      else ((uint16_t*)a.out)[o + i] = cvt_bf16(v[i]);
    }
    return;
  }
  if (a.out_f32) {
    float4* dst = reinterpret_cast<float4*>((float*)a.out + o);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint4 q;
  q.x = cvt_bf16x2(v[0], v[1]);
  q.y = cvt_bf16x2(v[2], v[3]);
  q.z = cvt_bf16x2(v[4], v[5]);
  q.w = cvt_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>((uint16_t*)a.out + o) = q;
}

template <int MODE, bool GATHER>
__global__ void __launch_bounds__(threads_of(GATHER), 1)
grouped_tc_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_wa,
                  const __grid_constant__ CUtensorMap tm_wb, const Args a) {
  constexpr int kCols = MODE == kGroupedSwiGLU ? 128 : 256;   // output columns of a unit
  constexpr int kPrefetchWarp = 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;
  uint8_t* staging_base = stages + (size_t)a.stages * a.stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging_base + 2 * kStagingBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned* ticket_slot = reinterpret_cast<volatile unsigned*>(tmem_slot + 2);
  uint32_t* half_slot = tmem_slot + 3;   // where rank 1's word about a stage is stored
  int* s_row = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_chunk = s_row + a.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pair = blockIdx.x >> 1;
  const uint32_t pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    // A stage is full once the weight box, this CTA's rows (one TMA arrival,
    // or one per gathering thread) and, on rank 0, rank 1's word that its
    // half has landed (4 bytes) have arrived.
    const uint32_t arrivals = 1u + (GATHER ? (uint32_t)kGatherThreads : 1u);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], arrivals);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * 2 * kEpiThreads);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_wa);
    tma_prefetch_desc(&tm_wb);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  // Without a routing the work is known at once.
  if (!a.offsets) plan_chunks(a, s_row, s_chunk);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  // ... and the first weights are asked into L2 while the previous kernel ends
  // (by a warp that nothing waits for: issuing blocks while the TMA unit is busy)
  if (!a.offsets && a.prefetch_kb > 0 && warp == kPrefetchWarp && lane == 0)
    prefetch_weights<kCols>(a, tm_wa, s_row, s_chunk, pair, pairs, rank);
  // All of the above overlaps the previous kernel's tail; the routing, the
  // operands and the outputs are touched only after it has finished.
  pdl_wait();
  // The next kernel may be placed at once, except where it adds up this one's
  // results: its small blocks would all be placed on the few SMs that finish
  // first (see the weights' thread).
  const bool late = MODE == kGroupedPlain || (MODE == kGroupedLinear && a.joined);
  if (!late) pdl_launch_dependents();
  if (a.offsets) {
    plan_chunks(a, s_row, s_chunk);
    __syncthreads();
  }
  const uint32_t tmem = *tmem_slot;
  // The pair's MMAs address both TMEMs with one column address; if the two
  // allocations disagree, neither CTA does any work.
  const bool skip = ld_shared_cluster_u32(mapa_shared(smem_u32(tmem_slot), rank ^ 1u)) != tmem;
  if (skip && threadIdx.x == 0) atomicOr(a.status, kStatusPairTmem);
  const Schedule sch = make_schedule(a, (uint32_t)s_chunk[a.E], pairs);
  if (MODE == kGroupedPlain && blockIdx.x == 0 && threadIdx.x == 32)
    *a.sched = make_uint4(sch.units, sch.whole, sch.cut_iters, sch.q);

  int64_t issued = 0;   // a producer's stages
  if (warp == 0) {
    // ---------------- weights (TMA, one thread of each CTA) ----------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = !skip;
      WorkIter w(sch, pair);
      uint32_t u;
      int kb0, kb1, e_at = 0;
      while (ok && w.next(a, sch, pairs, u, kb0, kb1)) {
        const Unit un = find_unit<kCols>(a, s_row, s_chunk, u, e_at);
        // columns of the CTA's two weight boxes
        const int ca = un.col0 + (MODE == kGroupedSwiGLU ? 64 : 128) * (int)rank;
        const int cb = MODE == kGroupedSwiGLU ? ca : ca + 64;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status, a.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* st = stages + (size_t)stage * a.stage_bytes;
          mbar_arrive_expect_tx(&full[stage], kABytes + (rank == 0 ? 4u : 0u));
          if (a.kmajor) {
            tma_load_3d(st, &tm_wa, &full[stage], kb * kBK, ca, un.e);
            // (one 128-column box where the columns are neighbours)
            if constexpr (MODE == kGroupedSwiGLU)
              tma_load_3d(st + kChunkBytes, &tm_wb, &full[stage], kb * kBK, cb, un.e);
          } else {
            tma_load_3d(st, &tm_wa, &full[stage], ca, kb * kBK, un.e);
            tma_load_3d(st + kChunkBytes, &tm_wb, &full[stage], cb, kb * kBK, un.e);
          }
          ++issued;
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every CTA is within a ring of its end by now, so the blocks of the
      // kernel that adds up find most SMs free.  (Decode linear, M = 8,
      // K = 14336, N = 4096: 26.6 us per call, 28.7 with its 32 joining blocks
      // placed at once, on the two SMs that have no work.)
      if (late) pdl_launch_dependents();
    }
    __syncwarp();
  } else if (warp >= kRowWarp) {
    // ---------------- rows of x ----------------
    if constexpr (GATHER) {
      // Rows gathered through `order`: 128 threads copy 16 bytes each, 16 rows
      // at a time, into the 128-byte-swizzled layout (16-byte chunk c of row r
      // at chunk c ^ (r & 7)).  Each thread's arrival on the stage's barrier
      // follows its copies by itself; whoever waits for the stage fences the
      // generic proxy, which wrote the rows, against the async proxy, through
      // which the MMAs read them.
      const int gt = threadIdx.x - kRowWarp * 32;
      const int c16 = gt & 7, r16 = gt >> 3;
      const uint32_t dst0 = kABytes + (uint32_t)r16 * 128u + (uint32_t)((c16 ^ (r16 & 7)) * 16);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = !skip;
      WorkIter w(sch, pair);
      uint32_t u;
      int kb0, kb1, e_at = 0;
      // The next unit's entries of `order` are fetched a unit ahead.
      int half = 0, next_half = 0, next0 = 0, next1 = 0;
      int flat[8];   // -1: past the chunk, zeros
      auto fetch = [&]() -> bool {
        if (!w.next(a, sch, pairs, u, next0, next1)) return false;
        const Unit un = find_unit<kCols>(a, s_row, s_chunk, u, e_at);
        next_half = un.n >> 1;
        const int r0 = un.row0 + (int)rank * next_half + r16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + j * 16;
          flat[j] = j * 16 < next_half && r < un.row0 + un.nrows ? a.order[r] : -1;
        }
        return true;
      };
      bool more = ok && fetch();
      while (ok && more) {
        const uint16_t* src[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t t = (uint32_t)flat[j] / (uint32_t)a.top_k;
          src[j] = flat[j] >= 0 && t < (uint32_t)a.tokens ? a.x + (int64_t)t * a.K : nullptr;
        }
        half = next_half;
        kb0 = next0;
        kb1 = next1;
        const int nb = half >> 4;
        more = fetch();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status, a.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32(stages + (size_t)stage * a.stage_bytes) + dst0;
          const int k = kb * kBK + c16 * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < nb) {
              const bool in = src[j] != nullptr && k < a.K;
              cp_async_16(dst + j * 2048, in ? src[j] + k : a.x, in ? 16u : 0u);
            }
          cp_async_arrive(&full[stage]);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      cp_async_wait_all();   // nothing is in flight when the CTA ends
    } else if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = !skip;
      WorkIter w(sch, pair);
      uint32_t u;
      int kb0, kb1, e_at = 0;
      while (ok && w.next(a, sch, pairs, u, kb0, kb1)) {
        const Unit un = find_unit<kCols>(a, s_row, s_chunk, u, e_at);
        const int half = un.n >> 1;
        const int brow = un.row0 + (int)rank * half;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status, a.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* sb = stages + (size_t)stage * a.stage_bytes + kABytes;
          mbar_arrive_expect_tx(&full[stage], (uint32_t)half * 128u);
          // boxes of 128, 64, 32 and 16 rows, as the bits of `half` ask
          int r = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int n = 128 >> b;
            if (half & n) {
              tma_load_2d(sb + r * 128, &tm_x.box[b], &full[stage], kb * kBK, brow + r);
              r += n;
            }
          }
          ++issued;
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer (rank 0 of the pair) ----------------
    // The whole warp runs the loop and one elected lane issues: with uniform
    // control flow the descriptors stay in uniform registers.  A loop of lane 0
    // alone took 580 clocks per k block, 70 of them per MMA, against the 512
    // that the MMAs of a full chunk take (64 experts' up projection of 4096
    // tokens 232 -> 191 us; M = 4096, K = 4096, N = 14336 261 -> 250 us).
    const bool elected = elect_one();
    const uint32_t a_step16 = (a.kmajor ? 32u : 2048u) >> 4, stage16 = a.stage_bytes >> 4;
    const uint64_t ad = smem_desc_sw128(smem_u32(stages), a.kmajor ? 16u : kChunkBytes, 1024u);
    const uint64_t bd = smem_desc_sw128(smem_u32(stages) + kABytes, 16u, 1024u);
    // (low halves: the address in 16-byte units; the high ones do not change)
    const uint32_t a_hi = (uint32_t)(ad >> 32), b_hi = (uint32_t)(bd >> 32);
    const uint32_t a_first = (uint32_t)ad, a_end = a_first + (uint32_t)a.stages * stage16;
    const uint32_t ab = (uint32_t)bd - (uint32_t)ad;
    const uint32_t full_first = smem_u32(full), to_empty = smem_u32(empty) - full_first;
    uint32_t al = a_first, bar = full_first;   // the stage's A descriptor and full barrier
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = !skip;
    WorkIter w(sch, pair);
    uint32_t u;
    int kb0, kb1, e_at = 0;
    while (ok && w.next(a, sch, pairs, u, kb0, kb1)) {
      const Unit un = find_unit<kCols>(a, s_row, s_chunk, u, e_at);
      // D format f32, A and B bf16; A (weights) MN-major for [K, n_out] weights
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((a.kmajor ? 0u : 1u) << 15) |
                             ((uint32_t)(un.n >> 3) << 17) | (16u << 24);
      ok = warp_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, a.status, a.timeout_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + (uint32_t)(acc * kAccCols);
      uint32_t accumulate = 0;
      for (int n = kb1 - kb0; n > 0; --n) {
        ok = warp_wait(bar, phase, abort_flag, a.status, a.timeout_ns);
        if (!ok) break;
        if constexpr (GATHER) fence_async_smem();
        tc_fence_after();
        if (elected) {
          const uint32_t bl = al + ab;
          mma_pair(d_tmem, al, a_hi, bl, b_hi, idesc, accumulate);
          mma_pair(d_tmem, al + a_step16, a_hi, bl + 2, b_hi, idesc, 1);
          mma_pair(d_tmem, al + 2 * a_step16, a_hi, bl + 4, b_hi, idesc, 1);
          mma_pair(d_tmem, al + 3 * a_step16, a_hi, bl + 6, b_hi, idesc, 1);
          commit_pair_both(bar + to_empty);
        }
        accumulate = 1;
        al += stage16;
        bar += 8;
        if (al == a_end) {
          al = a_first;
          bar = full_first;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elected) commit_pair_both(smem_u32(&tfull[acc]));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (elected) {
      mma_commit_pair(drain);
      wait_drain(drain, 0, a.status, a.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- rank 1: tell rank 0 when this CTA's half has landed ----------------
    // Gathered rows were written by this CTA's threads (cp.async, the generic
    // proxy), and rank 0's MMAs read them, so the word has to release at
    // cluster scope.  The completion of an asynchronous store does, and its
    // issue does not wait for that (64 experts' up projection of 4096 tokens
    // 193.1 us, 192.5 with an arrival that releases at CTA scope; an arrival
    // that releases at cluster scope holds the thread: 632 us).
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0u);
      const uint32_t slot0 = mapa_shared(smem_u32(half_slot), 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = !skip;
      WorkIter w(sch, pair);
      uint32_t u;
      int kb0, kb1;
      while (ok && w.next(a, sch, pairs, u, kb0, kb1)) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, a.status, a.timeout_ns)) {
            ok = false;
            break;
          }
          if constexpr (GATHER) fence_async_smem();
          st_async_u32(slot0, 1u, full0 + (uint32_t)stage * 8u);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: warps 2..9 (each CTA) ----------------
    // Two groups of four warps; group g takes the chunks of 32 rows c = g, g + 2, ...
    const int grp = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int col = quarter * 32 + lane;   // accumulator lane = weight column of this CTA
    const int et = (warp - 2 - 4 * grp) * 32 + lane;
    const uint32_t gbar = 1u + (uint32_t)grp;
    constexpr uint32_t kBothBar = 3;
    float* staging = reinterpret_cast<float*>(staging_base + grp * kStagingBytes);
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0u);
    int acc = 0;
    uint32_t acc_phase = 0;
    WorkIter w(sch, pair);
    uint32_t u;
    int kb0, kb1, e_at = 0;
    while (!skip && w.next(a, sch, pairs, u, kb0, kb1)) {
      const Unit un = find_unit<kCols>(a, s_row, s_chunk, u, e_at);
      // Both groups go on, or both end: what follows has barriers of one group
      // and of both.
      const bool ready = mbar_wait(&tfull[acc], acc_phase, abort_flag, a.status, a.timeout_ns);
      __syncwarp();
      if (!named_bar_all(kBothBar, 2 * kEpiThreads, ready)) break;
      tc_fence_after();
      const uint32_t t_acc = tmem + lane_off + (uint32_t)(acc * kAccCols);
      const bool whole = kb0 == 0 && kb1 == a.n_kb;
      const int nchunk = (un.nrows + 31) >> 5;
      const int cbase = un.col0 + (MODE == kGroupedSwiGLU ? 64 : 128) * (int)rank;   // output columns
      Shares sh{0, 0, 0};
      if (!whole) {
        // A share of a cut unit: store the sums so far.  A second kernel adds
        // them up or, in short chunks (self_join), the last of the unit's pairs
        // to take a ticket does.
        const uint32_t rel = u - sch.whole;
        const uint32_t slot = pair * sch.q / (uint32_t)a.n_kb == rel ? 0 : 1;
        float* mine = part_slot(a, pair, slot, rank);
#pragma unroll 1
        for (int c = grp; c < nchunk; c += 2) {
          uint32_t v[32];
          tmem_ld_x32(t_acc + (uint32_t)(c * 32), v);
          tmem_wait_ld();
          if (MODE == kGroupedSwiGLU || a.self_join) {
            // [32-row chunk][4-row group][column][4 rows]
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c * 32 + 4 * i < un.nrows)
                __stcg(reinterpret_cast<float4*>(mine + col * 4 + (c * 8 + i) * 512),
                       make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                   __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])));
          } else {
            // [row][column]
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i < un.nrows && cbase + col < a.n_out) __stcg(mine + (c * 32 + i) * 128 + col, __uint_as_float(v[i]));
          }
        }
        tc_fence_before();
        if (rank == 1) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
        else mbar_arrive(&tempty[acc]);
        bool last = false;
        if (MODE == kGroupedSwiGLU || a.self_join) {
          sh = shares_of(a, sch, rel);
          __threadfence();
          named_bar_sync(kBothBar, 2 * kEpiThreads);
          unsigned* counter = a.counters + sh.first * 2 + rank;
          if (grp == 0 && et == 0) *ticket_slot = atomicAdd(counter, 1u);
          named_bar_sync(kBothBar, 2 * kEpiThreads);
          const unsigned ticket = *ticket_slot;
          last = ticket + 1u == sh.count;
          // (a counter left over by a call that gave up)
          if (ticket >= sh.count && grp == 0 && et == 0) atomicOr(a.status, kStatusStaleCounter);
          if (last) {
            __threadfence();
            if (grp == 0 && et == 0) *counter = 0u;   // left at zero for the next call
          }
        }
        if (!last) {
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
          continue;
        }
      }
      // the bias of this thread's column
      float bias = 0.f;
      if constexpr (MODE == kGroupedLinear) {
        if (a.bias && cbase + col < a.n_out)
          bias = a.bias_f32 ? ((const float*)a.bias)[cbase + col]
                            : bf16_lo(((const uint16_t*)a.bias)[cbase + col]);
      }
#pragma unroll 1
      for (int c = grp; c < nchunk; c += 2) {
        float v[32];
        if (whole) {
          uint32_t* vu = reinterpret_cast<uint32_t*>(v);
          tmem_ld_x32(t_acc + (uint32_t)(c * 32), vu);
          tmem_wait_ld();
        } else {
          const float* first = part_slot(a, sh.first, sh.slot, rank) + c * 4096 + col * 4;
          const float* rest = part_slot(a, sh.first + 1, 0, rank) + c * 4096 + col * 4;
          if (un.nrows - c * 32 <= 8)
            add_shares<2, 8>(v, first, rest, part_stride(a), (int)sh.count, un.nrows - c * 32);
          else
            add_shares<8, 2>(v, first, rest, part_stride(a), (int)sh.count, un.nrows - c * 32);
        }
        if constexpr (MODE == kGroupedSwiGLU) {
          // Columns 0-63 hold x.W_gate, 64-127 x.W_up of the same 64 columns
          // of h.  The halves swap 16 rows: the gate threads finish rows 0-15
          // of the chunk, the up threads rows 16-31.
          const bool is_up = col >= 64;
          const int j = col & 63;
          float* give = staging + (is_up ? 16 * 64 : 0) + j;   // gate: [0], up: [1]
          const float* take = staging + (is_up ? 0 : 16 * 64) + j;
          uint16_t* hs = reinterpret_cast<uint16_t*>(staging + 2 * 16 * 64);
#pragma unroll
          for (int i = 0; i < 16; ++i) give[i * 64] = is_up ? v[i] : v[16 + i];
          named_bar_sync(gbar, kEpiThreads);
          uint16_t* hrow = hs + (is_up ? 16 * kHCols : 0) + j;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float other = take[i * 64];
            const float g = is_up ? other : v[i];
            const float up = is_up ? v[16 + i] : other;
            hrow[i * kHCols] = cvt_bf16(times_sigma<false>(g, g) * up);
          }
          named_bar_sync(gbar, kEpiThreads);
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int g = it * kEpiThreads + et;
            const int r = g >> 3, c8 = (g & 7) * 8;
            if (c * 32 + r < un.nrows && cbase + c8 < a.n_out)
              *reinterpret_cast<uint4*>((uint16_t*)a.out +
                                        (int64_t)(un.row0 + c * 32 + r) * a.n_out + cbase + c8) =
                  *reinterpret_cast<const uint4*>(hs + r * kHCols + c8);
          }
        } else if constexpr (MODE == kGroupedPlain) {
          // one column, 32 rows: a warp's stores cover 32 neighbouring columns
          // (128 bytes; staged through shared memory 2 % slower)
          if (cbase + col < a.n_out) {
            float* dst = (float*)a.out + (int64_t)(un.row0 + c * 32) * a.n_out + cbase + col;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i < un.nrows) dst[(int64_t)i * a.n_out] = v[i];
          }
        } else {
#pragma unroll
          for (int hp = 0; hp < 2; ++hp) {   // 16 rows at a time
            if (hp) {
              if (c * 32 + 16 >= un.nrows) break;
              named_bar_sync(gbar, kEpiThreads);   // rows 0-15 have been copied out
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[hp * 16 + i] += bias;
            activate_n<16>(v + hp * 16, a.act, a.out_f32 != 0);
#pragma unroll
            for (int i = 0; i < 16; ++i) staging[i * kStageCols + col] = v[hp * 16 + i];
            named_bar_sync(gbar, kEpiThreads);
#pragma unroll
            for (int it = 0; it < 2; ++it) {
              const int g = it * kEpiThreads + et;
              const int r = g >> 4, c8 = (g & 15) * 8;
              const int row = c * 32 + hp * 16 + r;
              if (row >= un.nrows || cbase + c8 >= a.n_out) continue;
              const int64_t o = (int64_t)(un.row0 + row) * a.n_out + cbase + c8;
              const int left = a.n_out - cbase - c8;
              const Residual8 rs = load_residual8(a, o, left);
              const float4* sp = reinterpret_cast<const float4*>(staging + r * kStageCols + c8);
              const float4 lo = sp[0], hi = sp[1];
              float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
              store_row8(a, o, left, f, rs);
            }
          }
          named_bar_sync(gbar, kEpiThreads);   // staging is free
        }
      }
      // every accumulator column of this buffer is read
      if (whole) {
        tc_fence_before();
        if (rank == 1) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
        else mbar_arrive(&tempty[acc]);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if constexpr (MODE == kGroupedSwiGLU) {
      // rows that no expert has (dropped choices) are zero
      const int first = s_row[a.E];
      const int per = a.n_out / 8;
      for (int64_t r = first + (int64_t)(blockIdx.x * 2 + grp); r < a.rows; r += 2 * gridDim.x)
        for (int c8 = et; c8 < per; c8 += kEpiThreads)
          *reinterpret_cast<uint4*>((uint16_t*)a.out + r * a.n_out + (int64_t)c8 * 8) =
              make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // Where a wait has given up, loads may still be in flight, whichever role it
  // was: they land before the CTA's shared memory goes away.  So do rank 1's
  // words that rank 0 no longer waits for: rank 1 lets 100 us pass after its
  // last one, and rank 0 stays until then.  (Where rank 0 gives up before its
  // last MMA, so does rank 1's epilogue.)
  if (*abort_flag) {
    drain_loads(full, issued, a);
    const uint64_t t0 = globaltimer_ns();
    while (rank == 1 && globaltimer_ns() - t0 < 100000u) __nanosleep(1000);
    __syncwarp();
  }
  // Neither CTA of a pair leaves (or frees its TMEM) while the other may still
  // signal its barriers or read its shared memory.
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The cut units of a linear product: y = act(sum of the shares + bias) +
// residual, eight columns of one row per thread, the shares in k order.
// Bound by L2 latency: a share is one round trip, so eight are loaded at a time.
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads)
linear_join_kernel(const __grid_constant__ Args a, int chunks, const Schedule sch) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t i = blockIdx.x * kJoinThreads + threadIdx.x;
  int row0, nrows;
  chunk_rows(a.rows, chunks, 0, &row0, &nrows);   // the first chunk has the most rows
  const uint32_t per = (uint32_t)nrows * 32u;
  const uint32_t rel = i / per;
  if (rel >= sch.units - sch.whole) return;
  const uint32_t rem = i - rel * per;
  const int r = (int)(rem >> 5), o = (int)(rem & 31);
  const uint32_t u = sch.whole + rel;
  const int cg = (int)(u / (uint32_t)chunks), chunk = (int)(u - (uint32_t)cg * (uint32_t)chunks);
  chunk_rows(a.rows, chunks, chunk, &row0, &nrows);
  const int c = cg * 256 + o * 8;
  if (r >= nrows || c >= a.n_out) return;
  // (bias and residual are used only after the shares' loads are under way)
  const int64_t out = (int64_t)(row0 + r) * a.n_out + c;
  const int left = a.n_out - c;
  const Residual8 rs = load_residual8(a, out, left);
  uint32_t bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bias[j] = 0u;
    if (a.bias && j < left)
      bias[j] = a.bias_f32 ? ((const uint32_t*)a.bias)[c + j] : (uint32_t)((const uint16_t*)a.bias)[c + j] << 16;
  }
  const Shares sh = shares_of(a, sch, rel);
  float v[8];
  add_row_shares<8>(a, sh, (uint32_t)(o >> 4), r * 128 + (o & 15) * 8, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(bias[j]);
  activate_n<8>(v, a.act, a.out_f32 != 0);
  store_row8(a, out, left, v, rs);
}

// y = act(bias) + residual, for products over nothing (K = 0).
__global__ void __launch_bounds__(256)
empty_linear_kernel(const void* bias, int bias_f32, int act, const void* resid, void* y, int out_f32,
                    int64_t M, int64_t N) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * N;
       i += (int64_t)gridDim.x * 256) {
    const int64_t n = i % N;
    float v = 0.f;
    if (bias) v = bias_f32 ? ((const float*)bias)[n] : bf16_lo(((const uint16_t*)bias)[n]);
    activate_n<1>(&v, act, out_f32 != 0);
    if (resid) v += out_f32 ? ((const float*)resid)[i] : bf16_lo(((const uint16_t*)resid)[i]);
    if (out_f32) ((float*)y)[i] = v;
    else ((uint16_t*)y)[i] = (uint16_t)f32_to_bf16_bits(v);
  }
}

// [K, N] weights whose rows are no multiple of 16 bytes, copied to rows of
// round8(N) (zeros behind N), which TMA can read.  Element by element, in every
// call: K = 4096, N = 50257, M = 8 516 us, 74 with N = 50264, 67 with the same
// weights as [N, K].
__global__ void __launch_bounds__(256)
pad_rows_kernel(const uint16_t* __restrict__ w, uint16_t* __restrict__ out, int64_t K, int64_t N,
                int64_t Np) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < K * Np;
       i += (int64_t)gridDim.x * 256) {
    const int64_t k = i / Np, n = i - k * Np;
    out[i] = n < N ? w[k * N + n] : (uint16_t)0;
  }
}

size_t smem_bytes(const GroupedPlan& p, int E) {
  return kFixedBytes + (size_t)p.stages * p.stage_bytes + (size_t)(2 * (E + 1)) * sizeof(int);
}

template <int MODE, bool GATHER>
cudaError_t launch_mode(const RowMaps& mx, const CUtensorMap& ma, const CUtensorMap& mb,
                        const Args& a, int pairs, size_t smem, cudaStream_t st) {
  auto kern = grouped_tc_kernel<MODE, GATHER>;
  static std::atomic<int> configured[64];   // zero: not yet set on that device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(threads_of(GATHER));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mx, ma, mb, a);
}

}  // namespace

GroupedPlan plan_grouped(int64_t rows, int64_t tokens, int64_t E, bool swiglu, int pairs,
                         const Tuning& tn) {
  GroupedPlan p{};
  // Rows per chunk.  An expert has rows / E rows on average, and no more than
  // `tokens` where a token chooses it once; chunks for twice the average keep
  // most experts in one chunk, so that their weights are read once.  Longer
  // chunks cost ring stages (10 at 32 rows, 6 at 192 and above), shorter ones
  // repeat the weights: 333 tokens over 8 experts (d_ff = 4864, d = 896) take
  // 24.3 us in chunks of up to 192 rows, 24.7 of 128, 30.0 of 64; the router
  // logits of 4096 rows 15.0 us in chunks of 256, 18.5 of 128, 24.6 of 64.
  int64_t want = E == 1 ? rows : 2 * ((rows + E - 1) / E) + 16;
  if (want > tokens) want = tokens;
  if (E == 1 && want > 256) {
    const int64_t c = (want + 255) / 256;
    want = (want + c - 1) / c;
  }
  if (want > 256) want = 256;
  if (tn.gr_rows > 0) want = tn.gr_rows < 256 ? tn.gr_rows : 256;
  p.n_max = (int)((want + 31) / 32 * 32);
  if (p.n_max < 32) p.n_max = 32;
  p.stage_bytes = kABytes + (uint32_t)(p.n_max / 2) * 128u;
  p.stages = (int)(kRingBytes / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.pairs = pairs < 1 ? 1 : pairs;
  p.counters_bytes = ((size_t)p.pairs * 2 * sizeof(unsigned) + 255) / 256 * 256;
  // (256 bytes behind the shares: the schedule)
  p.part_bytes = (size_t)p.pairs * 4 * (size_t)p.n_max * 128 * sizeof(float);
  // Shares of 16 k blocks or more: shorter ones only add shares to read (router
  // logits: 15.0 us at 16, 15.8 at 4 and 8, 18.4 at 32).  make_schedule takes 8
  // where few pairs would have work.
  p.min_kb = tn.gr_min_kb > 0 ? tn.gr_min_kb : 16;
  // Cutting: 24.3 against 34.9 us for the 333 tokens above, 24 against 73 us for
  // the decode linear below; the up projection of 4096 tokens over 64 experts
  // 233 us uncut, 238 cut (joined by the last pair).
  // Joined by the last pair up to 32 rows, by the next kernel above: decode
  // linear, K = 14336, N = 4096: M = 8 22.7 against 24.3 us, M = 64 29.7 against
  // 28.7; 333 tokens over 8 experts 31 against 24.3.
  p.self_join = swiglu || (tn.gr_self >= 0 ? tn.gr_self : p.n_max <= 32);
  p.cut = tn.gr_cut >= 0 ? tn.gr_cut : (!swiglu || p.n_max <= 64);
  // L2 prefetch before the dependency wait: 384 KB of weights per CTA (decode
  // linear, M = 8, K = 14336, N = 4096: 22.4 us with 24 k blocks, 23.1 with 16,
  // 22.8 with 32, 24.5 with none, 24.8 with 64).  Many rows hide it.
  p.prefetch_kb = tn.gr_prefetch >= 0 ? tn.gr_prefetch : (E == 1 && p.n_max <= 64 ? 24 : 0);
  return p;
}

void fill_work(Work* w, int mode, const GroupedCall& c, const GroupedPlan& p, float* part) {
  const int cols = mode == kGroupedSwiGLU ? 128 : 256;
  w->offsets = c.offsets;
  w->E = (int)c.E;
  w->rows = (int)c.rows;
  w->n_kb = (int)((c.K + kBK - 1) / kBK);
  w->n_out = (int)c.n_out;
  w->ncg = (int)((c.n_out + cols - 1) / cols);
  w->n_max = p.n_max;
  w->cut = p.cut;
  w->shares = p.cut && !p.self_join;
  w->min_kb = p.min_kb;
  w->part = part;
  w->sched = (uint4*)((char*)part + p.part_bytes);
}

cudaError_t launch_grouped(int mode, const GroupedCall& c, const GroupedPlan& p, float* part,
                           unsigned* counters, bool counters_clean, unsigned* status,
                           uint64_t timeout_ns, cudaStream_t st) {
  if (c.rows == 0 || c.n_out == 0) return cudaSuccess;
  cudaError_t e;
  if (c.K == 0) {
    if (mode != kGroupedLinear)
      return cudaMemsetAsync(c.out, 0, (size_t)c.rows * c.n_out * (c.out_f32 ? 4 : 2), st);
    int64_t blocks = (c.rows * c.n_out + 255) / 256;
    if (blocks > 1216) blocks = 1216;
    empty_linear_kernel<<<(unsigned)blocks, 256, 0, st>>>(c.bias, c.bias_f32, c.act, c.resid, c.out,
                                                         c.out_f32, c.rows, c.n_out);
    return cudaGetLastError();
  }
  RowMaps mx{};
  CUtensorMap ma, mb;
  const bool gather = mode == kGroupedSwiGLU;
  // (a CTA loads at most n_max / 2 rows at a time: larger boxes are never used)
  if (!gather)
    for (int b = 0; b < 4; ++b)
      if ((128 >> b) <= p.n_max / 2 &&
          (e = make_tmap_bf16_2d(&mx.box[b], c.x, c.rows, c.K, kBK, 128 >> b)) != cudaSuccess)
        return e;
  const bool kmajor = c.wlayout == kWeightsNK;
  const void* wa = c.wa;
  int64_t wcols = c.n_out;
  if (!kmajor && c.n_out % 8 != 0) {
    if (!c.padded || mode != kGroupedLinear) return cudaErrorInvalidValue;
    wcols = (c.n_out + 7) / 8 * 8;
    int64_t blocks = (c.K * wcols + 255) / 256;
    if (blocks > 1216) blocks = 1216;
    pad_rows_kernel<<<(unsigned)blocks, 256, 0, st>>>((const uint16_t*)c.wa, (uint16_t*)c.padded,
                                                     c.K, c.n_out, wcols);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    wa = c.padded;
  }
  const int64_t wr = kmajor ? c.n_out : c.K, wc = kmajor ? c.K : wcols;
  if ((e = make_tmap_bf16_3d(&ma, wa, c.E, wr, wc, 64, kmajor && !gather ? 128 : 64)) != cudaSuccess) return e;
  if (mode == kGroupedSwiGLU) {
    if ((e = make_tmap_bf16_3d(&mb, c.wb, c.E, wr, wc, 64, 64)) != cudaSuccess) return e;
  } else {
    mb = ma;
  }
  Args a{};
  a.x = (const uint16_t*)c.x;
  a.K = (int)c.K;
  a.order = c.order;
  a.top_k = (int)(c.top_k > 0 ? c.top_k : 1);
  a.tokens = (int)c.tokens;
  fill_work(&a, mode, c, p, part);
  a.stages = p.stages;
  a.stage_bytes = p.stage_bytes;
  a.kmajor = kmajor ? 1 : 0;
  a.prefetch_kb = c.offsets ? 0 : p.prefetch_kb;
  a.out = c.out;
  a.out_f32 = c.out_f32;
  a.bias = c.bias;
  a.bias_f32 = c.bias_f32;
  a.act = c.act;
  a.resid = c.resid;
  a.counters = counters;
  a.status = status;
  a.timeout_ns = timeout_ns;
  a.self_join = p.self_join;
  if (p.self_join && p.cut && !counters_clean &&
      (e = cudaMemsetAsync(counters, 0, p.counters_bytes, st)) != cudaSuccess)
    return e;
  const size_t smem = smem_bytes(p, a.E);
  switch (mode) {
    case kGroupedSwiGLU: return launch_mode<kGroupedSwiGLU, true>(mx, ma, mb, a, p.pairs, smem, st);
    case kGroupedPlain: return launch_mode<kGroupedPlain, false>(mx, ma, mb, a, p.pairs, smem, st);
    default: break;
  }
  // cut units: a second kernel adds their shares
  const uint32_t chunks = (uint32_t)((c.rows + p.n_max - 1) / p.n_max);
  const Schedule sch = make_schedule(a, chunks, (uint32_t)p.pairs);
  const uint32_t cut = sch.units - sch.whole;
  a.joined = cut > 0 && !p.self_join;
  if ((e = launch_mode<kGroupedLinear, false>(mx, ma, mb, a, p.pairs, smem, st)) != cudaSuccess)
    return e;
  if (!a.joined) return cudaSuccess;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = (c.rows + chunks - 1) / chunks;   // rows of a chunk
  cfg.gridDim = dim3((unsigned)((cut * most * 32 + kJoinThreads - 1) / kJoinThreads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_join_kernel, a, (int)chunks, sch);
}

}  // namespace swg
