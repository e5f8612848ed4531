// How a grouped product's work is cut up (grouped_tc.cu), shared with the
// kernels that add up the shares of cut units (linear_join_kernel,
// combine_kernel).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace swg {

struct Work {
  const int* offsets;      // [E + 1]; null: one group of `rows` rows
  int E;
  int rows;                // rows of the sorted operand (an upper bound of offsets[E])
  int n_kb;                // 64-deep k blocks
  int n_out;
  int ncg;                 // column groups (units) per chunk
  int n_max;               // most rows of a chunk, a multiple of 32
  int cut;                 // whether units of a partial wave are cut along K
  int shares;              // cut units' shares are left for the kernel after the product
  int min_kb;              // fewest k blocks of a share of a cut unit
  float* part;             // shares of cut units
  uint4* sched;            // the product's schedule (Schedule), for the kernel after it
};

// The work of a launch, from the offsets; the same in every thread.  (Units
// fit 32 bits: a unit is at least 128 columns of at least one row.)
struct Schedule {
  uint32_t units, whole;   // units [0, whole) run whole
  uint32_t cut_iters, q;   // the others (fewer than one per pair): k blocks in
                           // all, and per pair
};

struct Unit {
  int e, col0, row0, nrows, n;   // n: nrows rounded up to a multiple of 32
};

// A partial wave of at most three quarters of the pairs is cut: above that,
// sharing the units out evenly saves less than adding the shares costs (64
// units on 76 pairs, cut against whole: linear K = 4096, M = 8 26.6 / 24.9 us,
// M = 256 45.7 / 32.5; one token's up projection 20.4 / 16.2).  Below it, short
// chunks gain (40 units: M = 8 18.2 / 21.9, M = 64 22.4 / 25.0) and the longest
// would do without from half the pairs up (50 units: M = 8 22.0 / 22.3, M = 64
// 25.6 / 25.4, M = 256 39.0 / 29.6).
__host__ __device__ inline Schedule make_schedule(const Work& w, uint32_t chunks, uint32_t pairs) {
  Schedule s;
  s.units = chunks * (uint32_t)w.ncg;
  s.whole = s.units;
  s.cut_iters = 0;
  s.q = 1;
  const uint32_t rem = s.units % pairs;
  if (w.cut && rem > 0 && rem * 4 <= pairs * 3) {
    uint32_t q = (rem * (uint32_t)w.n_kb + pairs - 1) / pairs;
    // Shares half as long where the cut units would give work to at most a
    // quarter of the pairs and have two shares or more each (K = 4096, N = 64,
    // 256 rows: 10.1 against 11.3 us; 1 row 7.7 against 9.1; K = 2048, 1024 rows
    // 9.5 against 11.1).  Elsewhere they cost (M = 8, K = N = 896: 8.8 against
    // 7.1; M = 4096, K = 4096, N = 64: 15.9 against 15.0).
    const uint32_t n_kb = (uint32_t)w.n_kb, full = (uint32_t)w.min_kb;
    const uint32_t least = n_kb >= 2 * full && rem * n_kb * 4 <= pairs * full ? (full + 1) / 2 : full;
    if (q < least) q = least;
    if (q < (uint32_t)w.n_kb) {
      s.whole = s.units - rem;
      s.cut_iters = rem * (uint32_t)w.n_kb;
      s.q = q;
    }
  }
  return s;
}

// The work items of one pair: whole units, then its share of the cut units.
struct WorkIter {
  uint32_t u_next, it, it_end;
  __host__ __device__ WorkIter(const Schedule& s, uint32_t pair) : u_next(pair) {
    it = pair * s.q < s.cut_iters ? pair * s.q : s.cut_iters;
    it_end = (pair + 1) * s.q < s.cut_iters ? (pair + 1) * s.q : s.cut_iters;
  }
  __host__ __device__ bool next(const Work& a, const Schedule& s, uint32_t pairs, uint32_t& u, int& kb0,
                       int& kb1) {
    if (u_next < s.whole) {
      u = u_next;
      u_next += pairs;
      kb0 = 0;
      kb1 = a.n_kb;
      return true;
    }
    if (it < it_end) {
      const uint32_t n_kb = (uint32_t)a.n_kb;
      const uint32_t rel = it / n_kb;
      const uint32_t stop = (rel + 1) * n_kb < it_end ? (rel + 1) * n_kb : it_end;
      u = s.whole + rel;
      kb0 = (int)(it - rel * n_kb);
      kb1 = (int)(stop - rel * n_kb);
      it = stop;
      return true;
    }
    return false;
  }
};

// A cut unit's shares: those of pairs first .. first + count - 1, in k order.
// A pair has two slots: slot 0 for the unit its range begins in, slot 1 for
// the unit its range ends in (only the first pair's share can be in slot 1).
struct Shares {
  uint32_t first, count, slot;
};
__host__ __device__ inline Shares shares_of(const Work& w, const Schedule& s, uint32_t rel) {
  const uint32_t n_kb = (uint32_t)w.n_kb;
  Shares r;
  r.first = rel * n_kb / s.q;
  r.count = ((rel + 1) * n_kb - 1) / s.q - r.first + 1;
  r.slot = r.first * s.q / n_kb == rel ? 0 : 1;
  return r;
}

// f32 sums of one CTA's 128 columns of a share (slot, rank).
__device__ __forceinline__ int64_t part_stride(const Work& w) { return (int64_t)w.n_max * 128 * 4; }
__device__ __forceinline__ float* part_slot(const Work& w, uint32_t pair, uint32_t slot,
                                            uint32_t rank) {
  return w.part + (int64_t)pair * part_stride(w) + (int64_t)(slot * 2 + rank) * (w.n_max * 128);
}

// v[0 .. 8) = the sums of the shares at element `at` (row-major [row][128]),
// in k order.  NS shares are loaded at a time: each is an L2 round trip.
template <int NS>
__device__ __forceinline__ void add_row_shares(const Work& w, const Shares& sh, uint32_t rank,
                                               int at, float* v) {
  const float* first = part_slot(w, sh.first, sh.slot, rank) + at;
  const float* rest = part_slot(w, sh.first + 1, 0, rank) + at;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 1
  for (uint32_t s0 = 0; s0 < sh.count; s0 += NS) {
    float4 lo[NS], hi[NS];
#pragma unroll
    for (uint32_t s = 0; s < NS; ++s) {
      lo[s] = hi[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + s < sh.count) {
        const float* src = s0 + s == 0 ? first : rest + (int64_t)(s0 + s - 1) * part_stride(w);
        lo[s] = __ldcg(reinterpret_cast<const float4*>(src));
        hi[s] = __ldcg(reinterpret_cast<const float4*>(src) + 1);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      v[0] += lo[s].x; v[1] += lo[s].y; v[2] += lo[s].z; v[3] += lo[s].w;
      v[4] += hi[s].x; v[5] += hi[s].y; v[6] += hi[s].z; v[7] += hi[s].w;
    }
  }
}

// First row of expert e, within the rows there are (whatever the caller's
// offsets say, no row outside them is touched).
__device__ __forceinline__ int first_row(const Work& w, int e) {
  if (!w.offsets) return e == 0 ? 0 : w.rows;
  const int v = w.offsets[e];
  return v < 0 ? 0 : v > w.rows ? w.rows : v;
}

// s_row[e], s_chunk[e]: first row and first chunk of expert e (E + 1 entries).
// All threads of the block; they meet once more before reading s_chunk.
__device__ inline void plan_chunks(const Work& w, int* s_row, int* s_chunk) {
  for (int e = threadIdx.x; e <= w.E; e += blockDim.x) s_row[e] = first_row(w, e);
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int e0 = 0; e0 < w.E; e0 += 32) {
      const int e = e0 + (int)threadIdx.x;
      int c = 0;
      if (e < w.E) {
        const int m = s_row[e + 1] - s_row[e];
        c = m > 0 ? (m + w.n_max - 1) / w.n_max : 0;
      }
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if ((int)threadIdx.x >= o) inc += v;
      }
      if (e < w.E) s_chunk[e] = base + inc - c;
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (threadIdx.x == 0) s_chunk[w.E] = base;
  }
}

// Rows of one chunk: expert rows m over nc chunks, evenly.
__host__ __device__ inline void chunk_rows(int m, int nc, int chunk, int* first, int* count) {
  const int per = (m + nc - 1) / nc;
  *first = chunk * per;
  int n = m - chunk * per;
  if (n > per) n = per;
  *count = n < 0 ? 0 : n;
}

// Unit u: units run expert by expert, column group by column group, chunk by
// chunk, so that the pairs at work share an expert's weights and rows in L2.
// `e`: the expert of a unit before u, or 0 (callers go through their units in
// ascending order); left at u's expert.
template <int COLS>
__device__ __forceinline__ Unit find_unit(const Work& w, const int* s_row, const int* s_chunk,
                                          uint32_t u, int& e) {
  const int c = (int)(u / (uint32_t)w.ncg);
  if (s_chunk[e + 1] <= c) {   // s_chunk[e] <= c < s_chunk[hi]
    int hi = w.E;
    while (hi - e > 1) {
      const int mid = (e + hi) >> 1;
      if (s_chunk[mid] <= c) e = mid;
      else hi = mid;
    }
  }
  const int nc = s_chunk[e + 1] - s_chunk[e];
  const int l = (int)(u - (uint32_t)s_chunk[e] * (uint32_t)w.ncg);
  const int cg = l / nc, chunk = l - cg * nc;
  Unit r;
  int first;
  chunk_rows(s_row[e + 1] - s_row[e], nc, chunk, &first, &r.nrows);
  r.e = e;
  r.col0 = cg * COLS;
  r.row0 = s_row[e] + first;
  r.n = r.nrows <= 32 ? 32 : (r.nrows + 31) / 32 * 32;
  return r;
}

}  // namespace swg
