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
//
// Bound by memory: each operand is read and each result written once.  Rows of
// whole 16-byte pieces have a CTA each (a warp, up to 1024 elements), enough of
// which fit on an SM to keep its loads under way: 8192 x 8192 bf16 with a residual
// to e4m3 70.5 us in a graph (6670 GB/s, where a copy reaches 6780), 16384 x 2048
// 41.3 us, 8192 x 8192 f32 158 us; one row of 4096 takes 1.7 us, the launch.  Other
// widths stream through teams of warps (below): 8192 x 4099 44.9 us, 5001 x 897 f32
// 7.5 us (as the first kind, with partial pieces moved one by one, 58 and 9.3 us).
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

__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The larger of two; NaN if either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest of values that are not negative, or max_nan's NaN (their bits order like
// the values, and that NaN's, 0x7fffffff, come last).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// A piece of the row on its way: s (stored where there is a residual) and its squares ...
template <bool F32, bool RAGGED, bool MASK>
__device__ __forceinline__ void add_piece(const Pieces<F32, RAGGED>& pc, const NormArgs& a,
                                          int64_t first, int i, const uint4& xq, const uint4& rq,
                                          float2 (&t)[Row<F32>::kVec / 2], float2& q) {
  constexpr int H = Row<F32>::kVec / 2;
  unpack<F32>(xq, t);
  if (a.residual) {
    float2 r[H];
    unpack<F32>(rq, r);
#pragma unroll
    for (int h = 0; h < H; ++h) t[h] = add2(t[h], r[h]);
  }
  if (MASK) pc.mask(i, t);
  if (a.residual) pc.store_at(a.sum, first, i, t);
#pragma unroll
  for (int h = 0; h < H; ++h) q = fma2(t[h], t[h], q);
}
// ... then t = s * w, and the largest so far.
template <bool FP8, int H>
__device__ __forceinline__ void weigh(float2 (&t)[H], const float2 (&w)[H], float& m) {
#pragma unroll
  for (int h = 0; h < H; ++h) {
    t[h] = mul2(t[h], w[h]);
    if (FP8) m = max_nan(m, max_nan(fabsf(t[h].x), fabsf(t[h].y)));
  }
}

// ... and on its way out, as t * f.
template <bool F32, bool FP8, bool RAGGED>
__device__ __forceinline__ void put_piece(const Pieces<F32, RAGGED>& pc, void* out, int64_t first,
                                          int i, float2 (&t)[Row<F32>::kVec / 2], float f) {
  constexpr int V = Row<F32>::kVec;
#pragma unroll
  for (int h = 0; h < V / 2; ++h) t[h] = mul2(t[h], make_float2(f, f));
  if constexpr (FP8) {
    uint32_t c[V / 4];
#pragma unroll
    for (int h = 0; h < V / 4; ++h) c[h] = e4m3x2(t[2 * h]) | (e4m3x2(t[2 * h + 1]) << 16);
    pc.store_codes(out, first, i, c);
  } else {
    pc.store_at(out, first, i, t);
  }
}

struct RowFactors {
  float f;       // of t
  float scale;   // FP8: the row's
};
template <bool FP8>
__device__ __forceinline__ RowFactors row_factors(float q, float m, const NormArgs& a) {
  const float r = 1.0f / sqrtf(q / (float)a.d + a.eps);
  if (!FP8) return {r, 0.f};
  const bool some = !(m < kLeastAmax);   // (NaN gives NaN)
  return {some ? 448.0f / m : 0.f, (some ? m : 0.f) * r / 448.0f};
}

// One row per warp (WARP) or per CTA; VPT pieces per thread.
template <bool F32, int VPT, bool FP8, bool RAGGED, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int H = Row<F32>::kVec / 2;
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
  float2 t[VPT][H];
  float2 q2 = make_float2(0.f, 0.f);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i >= pc.n) continue;
    add_piece<F32, RAGGED, true>(pc, a, pc.first, i, xr[j], rr[j], t[j], q2);
    float2 w[H];
    pc.weight(a.weight, a.weight_f32, i, w);
    weigh<FP8>(t[j], w, m);
  }
  float q = warp_sum(q2.x + q2.y);
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
  const RowFactors rf = row_factors<FP8>(q, m, a);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = lane + j * lanes;
    if (i < pc.n) put_piece<F32, FP8, RAGGED>(pc, a.out, pc.first, i, t[j], rf.f);
  }
  if (FP8 && lane == 0) a.scales[row] = rf.scale;
}

// ---- rows that stream through a CTA ---------------------------------------------
//
// The gradient, and the norm of rows that are no multiple of 16 bytes, keep
// something per column across rows (sums of dweight; the weight, moved to where
// such rows start).  One CTA per SM holds R teams of W warps; a team takes row
// after row, two pieces to a thread, and copies the next rows (cp.async) into
// slots that only the copying thread reads, while one is reduced.  Rows go to
// the CTAs first, then to their teams.  The gradient's widest rows are shared by
// the CTAs of a cluster, whose warps hand their sums to all of them.

constexpr int kPieces = 2;
constexpr int team_threads(int w) { return 24 % w ? 32 * w : 768; }
constexpr int team_rows(int w) { return team_threads(w) / 32 / w; }   // R
// Stages of the copies, of `arrays` tensors each.  More is not better: with 768
// threads the gradient of 8192 x 4096 takes 44.3 us with two (147 KB) and 47.1 with
// three (221 KB), 16384 x 896 22.5 and 23.0.  A third is for what has little under
// way: 512 threads (4096 x 8192 48.0 with two, 47.6 with three; 8192 x 4096 f32 80.6
// and 81.1), the gradient's rows of a warp (16384 x 512 14.2 and 14.1; x 256 8.4 and
// 8.6), the norm's of four warps and less (5001 x 897 f32 7.55 and 7.45).
constexpr int team_stages(int w, int arrays, int cluster) {
  if (cluster > 1) return w == 16 ? 4 : 3;
  return w == 16 || w <= (arrays == 3 ? 1 : 4) ? 3 : 2;
}

enum Second { kNone, kSum, kMax };   // what becomes of the second value of join

// ARRAYS tensors are copied; C CTAs share a row (C > 1: one team to a CTA).
template <bool F32, int W, bool RAGGED, int ARRAYS, int C>
struct Team {
  static constexpr int V = Row<F32>::kVec, P = kPieces, T = team_threads(W),
                       S = team_stages(W, ARRAYS, C), R = team_rows(W);
  static_assert(C == 1 || R == 1, "a cluster's CTAs meet once a row");
  using Shared = float2[S][C > 1 ? C * W : 32];   // the warps' values
  int warp, l, team, rank, lane;
  int64_t unit, units;   // rows unit, unit + units, ...
  int64_t M;
  uint4* slots;
  // (ragged: all rows of a team start at one place of their 16 bytes, since
  // `units` is a multiple of row_period or every team has one row at most)
  Pieces<F32, RAGGED> pc;

  __device__ __forceinline__ Team(uint4* ring, int64_t M_, int d)
      : warp(threadIdx.x >> 5), l(threadIdx.x & 31), team(warp / W),
        rank(C > 1 ? blockIdx.x % C : 0), lane(threadIdx.x - team * W * 32),
        unit(blockIdx.x / C + (int64_t)team * (gridDim.x / C)),
        units((int64_t)(gridDim.x / C) * R), M(M_), slots(ring + threadIdx.x), pc(unit, d) {
    if (C > 1) tc::cluster_sync_all();   // the others run: their shared memory is there
  }
  __device__ __forceinline__ int piece(int j) const { return rank * (P * W * 32) + lane + j * W * 32; }
  __device__ __forceinline__ uint4* slot(int stage, int array, int j) const {
    return slots + stage * (ARRAYS * P * T) + (array * P + j) * T;
  }
  // The row's first and last piece: ones where it has elements.  The threads that
  // have them keep them, because the others wait for those every row.  (Not for
  // f32, whose four elements are masked as fast: 8192 x 4095 90 us, so 92; nor with
  // 32 warps, whose 64 registers it overruns: 2048 x 16001 58.5 us, so 65.6.)
  static constexpr bool kEdges = RAGGED && !F32 && W < 32;
  using Edges = uint4[kEdges ? R : 1][2];
  __device__ __forceinline__ void find_edges(Edges& edges) const {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = piece(j);
      if (kEdges && (i == 0 || i == pc.n - 1)) edges[team][i != 0] = pc.ones(i);
    }
  }
  // A piece of a row, with kEdges 0 where it is a neighbour's.
  __device__ __forceinline__ uint4 read(int stage, int array, int j, const Edges& edges) const {
    uint4 q = *slot(stage, array, j);
    const int i = piece(j);
    if (kEdges && !pc.whole(i)) {
      const uint4 m = edges[team][i != 0];
      q = make_uint4(q.x & m.x, q.y & m.y, q.z & m.z, q.w & m.w);
    }
    return q;
  }
  __device__ __forceinline__ int64_t first(int64_t row) const { return row * pc.d - pc.shift; }
  // This thread's pieces of `row`, a group of copies (an empty one past the last row).
  __device__ __forceinline__ void fetch(int64_t row, int stage, const void* p0, const void* p1,
                                        const void* p2) const {
    if (row < M) {
      const int64_t at = (first(row) + (int64_t)piece(0) * V) * (16 / V);   // in bytes
      const int64_t left = M * pc.d * (16 / V) - at;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (piece(j) >= pc.n) continue;
        // (the last piece of the tensor may be cut short)
        const int to = j * W * 32 * 16, bytes = !RAGGED || left >= to + 16 ? 16 : (int)left - to;
        copy_piece(slot(stage, 0, j), (const char*)p0 + at + to, bytes);
        if (p1) copy_piece(slot(stage, 1, j), (const char*)p1 + at + to, bytes);
        if (p2) copy_piece(slot(stage, 2, j), (const char*)p2 + at + to, bytes);
      }
    }
    copies_commit();
  }
  // The first rows' copies.
  __device__ __forceinline__ void begin(const void* p0, const void* p1, const void* p2) const {
#pragma unroll
    for (int i = 0; i < (C > 1 ? S : S - 1); ++i) fetch(unit + i * units, i, p0, p1, p2);
  }
  // Values of the threads added up (the second: see Second) over the row's threads,
  // in a fixed order: a warp's ...
  template <Second SECOND>
  __device__ __forceinline__ static float2 of_warp(float2 v) {
    v.x = warp_sum(v.x);
    if (SECOND != kNone) v.y = SECOND == kMax ? warp_max(v.y) : warp_sum(v.y);
    return v;
  }
  // ... and the row's (one barrier a row: the next row writes another stage's place).
  template <Second SECOND>
  __device__ __forceinline__ float2 join(Shared& red, int stage, float2 v) const {
    if (W == 1) return v;
    if (l == 0) red[stage][warp] = v;
    if (R == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
    if (W & (W - 1)) return of_warp<SECOND>(l < W ? red[stage][team * W + l] : make_float2(0.f, 0.f));
    // (a power of two takes log2 W steps: 5001 x 897 f32 7.5 us, with five 7.7)
    v = red[stage][team * W + l % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(~0u, v.x, o);
      if (SECOND == kNone) continue;
      const float u = __shfl_xor_sync(~0u, v.y, o);
      v.y = SECOND == kMax ? max_nan(v.y, u) : v.y + u;
    }
    return v;
  }
  // The same among a cluster's CTAs, in two halves.
  __device__ __forceinline__ void send(Shared& red, int stage, float2 v) const {
    if (l < C) {
      const uint32_t to = tc::mapa_shared(tc::smem_u32(&red[stage][rank * W + warp]), l);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y)
                   : "memory");
    }
    __syncwarp();   // (the barrier wants the warp together)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  template <Second SECOND>
  __device__ __forceinline__ float2 receive(const Shared& red, int stage) const {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < C * W; i += 32) {
      const float2 u = i + l < C * W ? red[stage][i + l] : make_float2(0.f, 0.f);
      v.x += u.x;
      v.y = SECOND == kMax ? max_nan(v.y, u.y) : v.y + u.y;
    }
    return of_warp<SECOND>(v);
  }
  // For each row of the team: first(row, stage) gives a thread's values, and
  // second(row, stage, v) gets the row's.  The next rows are on their way.  A
  // cluster's barrier takes longer than a CTA's, so there the first half of the
  // next row stands between its two ends, and the second half of the row before.
  // (unrolled, so that the slots' addresses are constants)
  template <Second SECOND, typename First, typename Last>
  __device__ __forceinline__ void rows(const void* p0, const void* p1, const void* p2, Shared& red,
                                       First first_half, Last second_half) const {
    int64_t row = unit;
    if constexpr (C > 1) {
      copies_wait<S - 1>();
      send(red, 0, of_warp<SECOND>(first_half(row, 0)));
    }
    while (true) {
#pragma unroll
      for (int stage = 0; stage < S; ++stage) {
        if (row >= M) return;
        if constexpr (C > 1) {
          const bool more = row + units < M;
          float2 mine = make_float2(0.f, 0.f);
          if (more) {
            copies_wait<S - 2>();
            mine = of_warp<SECOND>(first_half(row + units, (stage + 1) % S));
          }
          const float2 v = receive<SECOND>(red, stage);
          if (more) send(red, (stage + 1) % S, mine);
          second_half(row, stage, v);
          fetch(row + S * units, stage, p0, p1, p2);
        } else {
          fetch(row + (S - 1) * units, (stage + S - 1) % S, p0, p1, p2);
          copies_wait<S - 1>();
          second_half(row, stage,
                      join<SECOND>(red, stage, of_warp<SECOND>(first_half(row, stage))));
        }
        row += units;
      }
    }
  }
};

template <bool F32, int W, bool FP8>
__global__ void __launch_bounds__(team_threads(W), 1)
norm_stream_kernel(const __grid_constant__ NormArgs a) {
  using Tm = Team<F32, W, true, 2, 1>;
  constexpr int P = Tm::P, H = Tm::V / 2;
  extern __shared__ uint4 ring[];
  __shared__ typename Tm::Shared red;
  __shared__ typename Tm::Edges edges;
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const Tm tm(ring, a.M, a.d);
  tm.begin(a.x, a.residual, nullptr);
  tm.find_edges(edges);
  float2 w[P][H], t[P][H];
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (tm.piece(j) < tm.pc.n) tm.pc.weight(a.weight, a.weight_f32, tm.piece(j), w[j]);
  const auto add = [&](int64_t row, int stage) {
    float2 q = make_float2(0.f, 0.f);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = tm.piece(j);
      if (i >= tm.pc.n) continue;
      add_piece<F32, true, !Tm::kEdges>(tm.pc, a, tm.first(row), i, tm.read(stage, 0, j, edges),
                                  a.residual ? tm.read(stage, 1, j, edges) : uint4{}, t[j], q);
      weigh<FP8>(t[j], w[j], m);
    }
    return make_float2(q.x + q.y, m);
  };
  const auto put = [&](int64_t row, int stage, float2 v) {
    const RowFactors rf = row_factors<FP8>(v.x, v.y, a);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = tm.piece(j);
      if (i >= tm.pc.n) continue;
      put_piece<F32, FP8, true>(tm.pc, a.out, tm.first(row), i, t[j], rf.f);
    }
    if (FP8 && tm.lane == 0) a.scales[row] = rf.scale;
  };
  tm.template rows<FP8 ? kMax : kNone>(a.x, a.residual, nullptr, red, add, put);
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
  // where 512 threads would not do (4096 rows of 16384, bf16: 81 us, against 88
  // with 16 elements and 1024 threads, of which one CTA fits on an SM).
  int e = 8;
  if (M > num_sms) {
    while (e < 32 && 32 * (e / vec) < pieces) e *= 2;
    if (32 * (e / vec) >= pieces) return {e / vec, 32, true};
    e = 512 * (16 / vec) < pieces ? 32 : 16;
  }
  while (e < 32 && 1024 * (e / vec) < pieces) e *= 2;
  const int vpt = e / vec;
  return {vpt, (int)((pieces + vpt * 32 - 1) / (vpt * 32) * 32), false};
}

int64_t pieces_of(int64_t d, int vec) { return d % vec ? d / vec + 2 : d / vec; }

// How a streaming kernel is launched: `warps` of each CTA to a row, the CTAs of a
// cluster to the widest rows (of more than 2048 pieces), `units` CTAs or clusters.
struct TeamShape {
  int warps, cluster, units;
};
constexpr int64_t kOneCtaPieces = 32 * kPieces * 32;
TeamShape team_shape(int64_t M, int64_t d, int vec, int num_sms) {
  const int64_t pieces = pieces_of(d, vec);
  TeamShape s{0, 1, 0};
  for (int w : {32, 24, 16, 12, 8, 6, 4, 3, 2, 1})
    if (32 * kPieces * w >= pieces) s.warps = w;
  // (Two CTAs of 16 warps for 2048 pieces lose to one of 32: 2048 x 16384 58.8 us
  // against 56.1.  Above, one CTA that reads rows twice and keeps dweight's sums in
  // shared memory took 109 us for 2048 x 12288 f32, 146 for 2048 x 16384 f32 and 99
  // for 1024 x 32768 bf16, where the clusters take 68, 97 and 63.)
  if (!s.warps) {
    constexpr int kOf24 = 24 * 32 * kPieces;   // what a CTA of 24 warps holds
    s.cluster = pieces <= 2 * kOf24 ? 2 : pieces <= 4 * kOf24 ? 4 : 8;
    s.warps = pieces <= 1024 * s.cluster ? 16 : 24;
  }
  // (clusters of 4 and 8 must fit whole parts of the GPU: 36 and 15 do)
  int64_t most = num_sms / s.cluster;
  if (s.cluster == 4) most = most * 95 / 100;
  if (s.cluster == 8) most = most * 80 / 100;
  // Rows so many apart start at one place of their 16 bytes: see Team::pc.
  int period = vec;
  for (int64_t low = d; period > 1 && low % 2 == 0; low /= 2) period /= 2;
  most = most < period ? period : most / period * period;
  s.units = (int)(M < most ? M : most);
  return s;
}

template <auto kernel, int W, int ARRAYS, int C, typename A>
cudaError_t launch_team(const A& a, int units, cudaStream_t st) {
  constexpr int smem = team_stages(W, ARRAYS, C) * ARRAYS * kPieces * team_threads(W) * 16;
  return launch_chained_smem<kernel, C>(smem, dim3(units * C), dim3(team_threads(W)), smem, st, a);
}

template <bool F32, int VPT, bool FP8>
cudaError_t launch_norm(const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (s.warp)
    return launch_chained(norm_kernel<F32, VPT, FP8, false, true>, dim3((unsigned)((a.M + 7) / 8)),
                          dim3(256), 0, st, a);
  return launch_chained(norm_kernel<F32, VPT, FP8, false, false>, dim3((unsigned)a.M),
                        dim3(s.threads), 0, st, a);
}

template <bool F32, bool FP8>
cudaError_t launch_rows(const NormArgs& a, int num_sms, cudaStream_t st) {
  constexpr int V = Row<F32>::kVec, base = 8 / V;   // pieces of 8 elements
  if (a.d % V == 0) {
    const Shape s = shape_of(a.d / V, V, a.M, num_sms);
    if (s.vpt == base) return launch_norm<F32, base, FP8>(a, s, st);
    if (s.vpt == 2 * base) return launch_norm<F32, 2 * base, FP8>(a, s, st);
    return launch_norm<F32, 4 * base, FP8>(a, s, st);
  }
  const int64_t pieces = pieces_of(a.d, V);
  if (pieces > kOneCtaPieces)   // too wide for a team: as the others, with partial pieces
    return launch_chained(norm_kernel<F32, 4 * base, FP8, true, false>, dim3((unsigned)a.M),
                          dim3((unsigned)((pieces + 128 * base - 1) / (128 * base) * 32)), 0, st, a);
  const TeamShape s = team_shape(a.M, a.d, V, num_sms);
  switch (s.warps) {
    case 1: return launch_team<norm_stream_kernel<F32, 1, FP8>, 1, 2, 1>(a, s.units, st);
    case 2: return launch_team<norm_stream_kernel<F32, 2, FP8>, 2, 2, 1>(a, s.units, st);
    case 3: return launch_team<norm_stream_kernel<F32, 3, FP8>, 3, 2, 1>(a, s.units, st);
    case 4: return launch_team<norm_stream_kernel<F32, 4, FP8>, 4, 2, 1>(a, s.units, st);
    case 6: return launch_team<norm_stream_kernel<F32, 6, FP8>, 6, 2, 1>(a, s.units, st);
    case 8: return launch_team<norm_stream_kernel<F32, 8, FP8>, 8, 2, 1>(a, s.units, st);
    case 12: return launch_team<norm_stream_kernel<F32, 12, FP8>, 12, 2, 1>(a, s.units, st);
    case 16: return launch_team<norm_stream_kernel<F32, 16, FP8>, 16, 2, 1>(a, s.units, st);
    case 24: return launch_team<norm_stream_kernel<F32, 24, FP8>, 24, 2, 1>(a, s.units, st);
    case 32: return launch_team<norm_stream_kernel<F32, 32, FP8>, 32, 2, 1>(a, s.units, st);
  }
  return cudaErrorInvalidValue;   // (team_shape gives none other)
}

// ---- gradient -------------------------------------------------------------------
//
//   r = 1 / sqrt(mean(s^2) + eps), g = dy * weight
//   dx = ds + r (g - s r^2 mean(g s)),  dweight = sum over rows of dy s r
//
// A team's columns' sums of dweight stay in registers over all of its rows; each
// CTA then writes one row of partial sums, and a second kernel adds those in a
// fixed order.  Bound by memory but for its ends: 8192 x 4096 bf16 with ds 44.4 us
// in a graph (6050 GB/s), of which the second kernel and the first rows' latency
// take about 5; f32 80.6 us (6660 GB/s).  Without rows copied ahead it took 72 us,
// with every CTA's own partial sums (456 of them) 63.6.

struct BackArgs {
  const void* dy;
  const void* s;
  const void* weight;
  const void* ds;
  void* dx;
  float* part;   // [teams' CTAs or clusters, d]
  int64_t M;
  int d;
  float eps;
  int weight_f32;
};

template <bool F32, int W, bool RAGGED, int C>
__global__ void __launch_bounds__(team_threads(W), 1)
norm_backward_kernel(const __grid_constant__ BackArgs a) {
  using Tm = Team<F32, W, RAGGED, 3, C>;
  constexpr int P = Tm::P, H = Tm::V / 2, R = Tm::R;
  // whether a row's values stay unpacked for both halves
  constexpr bool kHold = C == 1 && (F32 || Tm::T <= 512);
  extern __shared__ uint4 ring[];
  __shared__ typename Tm::Shared red;
  __shared__ typename Tm::Edges edges;
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const Tm tm(ring, a.M, a.d);
  tm.begin(a.s, a.dy, a.ds);
  tm.find_edges(edges);
  float2 w[P][H], acc[P][H], s[P][H], g[P][H];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (tm.piece(j) < tm.pc.n) tm.pc.weight(a.weight, a.weight_f32, tm.piece(j), w[j]);
#pragma unroll
    for (int h = 0; h < H; ++h) acc[j][h] = make_float2(0.f, 0.f);
  }
  const float inv_d = 1.0f / (float)a.d;
  const auto sums_of = [&](int64_t, int stage) {   // s^2, g s
    float2 q = make_float2(0.f, 0.f), p = q;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = tm.piece(j);
      if (i >= tm.pc.n) continue;
      unpack<F32>(tm.read(stage, 0, j, edges), s[j]);
      unpack<F32>(tm.read(stage, 1, j, edges), g[j]);
      if (!Tm::kEdges) {
        tm.pc.mask(i, s[j]);
        tm.pc.mask(i, g[j]);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        q = fma2(s[j][h], s[j][h], q);
        p = fma2(mul2(g[j][h], w[j][h]), s[j][h], p);
      }
    }
    return make_float2(q.x + q.y, p.x + p.y);
  };
  // t = s r:  dx = ds + r g - t r^2 mean(g s),  dweight += dy t
  const auto put = [&](int64_t row, int stage, float2 v) {
    const float r = rsqrtf(fmaf(v.x, inv_d, a.eps));
    // (not r * r first, which leaves binary32 where eps is subnormal and s about 0)
    const float c = -r * (v.y * inv_d * r);
    const float2 r2 = make_float2(r, r), c2 = make_float2(c, c);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = tm.piece(j);
      if (i >= tm.pc.n) continue;
      float2 o[H];
      if (!kHold) {   // (ragged: what is a neighbour's is not stored)
        unpack<F32>(*tm.slot(stage, 0, j), s[j]);
        unpack<F32>(*tm.slot(stage, 1, j), g[j]);
      }
      if (a.ds) {
        unpack<F32>(*tm.slot(stage, 2, j), o);
      } else {
#pragma unroll
        for (int h = 0; h < H; ++h) o[h] = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float2 t = mul2(s[j][h], r2);
        acc[j][h] = fma2(g[j][h], t, acc[j][h]);
        o[h] = fma2(c2, t, fma2(r2, mul2(g[j][h], w[j][h]), o[h]));
      }
      tm.pc.store_at(a.dx, tm.first(row), i, o);
    }
  };
  tm.template rows<kSum>(a.s, a.dy, a.ds, red, sums_of, put);
  // The CTA's sums, team after team.
  copies_wait<0>();
  __syncthreads();
  float* part = a.part + (int64_t)(blockIdx.x / C) * a.d;
  float* all = reinterpret_cast<float*>(ring);
  float* sums = R > 1 ? all + tm.team * a.d : part;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = tm.piece(j);
    if (i >= tm.pc.n) continue;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (tm.pc.has(i, 2 * h)) sums[tm.pc.col(i) + 2 * h] = acc[j][h].x;
      if (tm.pc.has(i, 2 * h + 1)) sums[tm.pc.col(i) + 2 * h + 1] = acc[j][h].y;
    }
  }
  if (R > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += Tm::T) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) v += all[i * a.d + c];
      part[c] = v;
    }
  }
}

constexpr int kSumCols = 32, kSumRows = 32;

// dweight = the partial sums of n CTAs, added in a fixed order.
__global__ void __launch_bounds__(kSumCols * kSumRows)
dweight_kernel(const float* part, int n, int d, void* out, int f32) {
  __shared__ float red[kSumRows][kSumCols + 1];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * kSumCols + x;
  float v = 0.f;
  if (c < d) {
#pragma unroll 5
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

template <bool F32, bool RAGGED>
cudaError_t launch_back(const BackArgs& a, const TeamShape& s, cudaStream_t st) {
  // (the teams' sums take the place of their stages: R rows of at most 512 W
  // elements, 2 KB, and each stage has as much)
  switch (s.cluster > 1 ? 100 * s.cluster + s.warps : s.warps) {
    case 1: return launch_team<norm_backward_kernel<F32, 1, RAGGED, 1>, 1, 3, 1>(a, s.units, st);
    case 2: return launch_team<norm_backward_kernel<F32, 2, RAGGED, 1>, 2, 3, 1>(a, s.units, st);
    case 3: return launch_team<norm_backward_kernel<F32, 3, RAGGED, 1>, 3, 3, 1>(a, s.units, st);
    case 4: return launch_team<norm_backward_kernel<F32, 4, RAGGED, 1>, 4, 3, 1>(a, s.units, st);
    case 6: return launch_team<norm_backward_kernel<F32, 6, RAGGED, 1>, 6, 3, 1>(a, s.units, st);
    case 8: return launch_team<norm_backward_kernel<F32, 8, RAGGED, 1>, 8, 3, 1>(a, s.units, st);
    case 12: return launch_team<norm_backward_kernel<F32, 12, RAGGED, 1>, 12, 3, 1>(a, s.units, st);
    case 16: return launch_team<norm_backward_kernel<F32, 16, RAGGED, 1>, 16, 3, 1>(a, s.units, st);
    case 24: return launch_team<norm_backward_kernel<F32, 24, RAGGED, 1>, 24, 3, 1>(a, s.units, st);
    case 32: return launch_team<norm_backward_kernel<F32, 32, RAGGED, 1>, 32, 3, 1>(a, s.units, st);
    case 224: return launch_team<norm_backward_kernel<F32, 24, RAGGED, 2>, 24, 3, 2>(a, s.units, st);
    case 416: return launch_team<norm_backward_kernel<F32, 16, RAGGED, 4>, 16, 3, 4>(a, s.units, st);
    case 424: return launch_team<norm_backward_kernel<F32, 24, RAGGED, 4>, 24, 3, 4>(a, s.units, st);
    case 816: return launch_team<norm_backward_kernel<F32, 16, RAGGED, 8>, 16, 3, 8>(a, s.units, st);
  }
  return cudaErrorInvalidValue;   // (team_shape gives none other)
}

}  // namespace

cudaError_t launch_rms_norm(const NormCall& c, int num_sms, cudaStream_t st) {
  if (c.M == 0 || c.d == 0) return cudaSuccess;
  const NormArgs a{c.x, c.residual, c.weight, c.out, c.scales, c.sum, c.M, (int)c.d, c.eps,
                   c.weight_f32};
  if (c.f32)
    return c.scales ? launch_rows<true, true>(a, num_sms, st)
                    : launch_rows<true, false>(a, num_sms, st);
  return c.scales ? launch_rows<false, true>(a, num_sms, st)
                  : launch_rows<false, false>(a, num_sms, st);
}

size_t rms_norm_backward_bytes(int64_t M, int64_t d, int f32, int num_sms) {
  return (size_t)team_shape(M, d, f32 ? 4 : 8, num_sms).units * (size_t)d * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackwardCall& c, float* part, int num_sms,
                                     cudaStream_t st) {
  if (c.d == 0) return cudaSuccess;
  const TeamShape s = team_shape(c.M, c.d, c.f32 ? 4 : 8, num_sms);
  if (c.M > 0) {
    const BackArgs a{c.dy, c.s, c.weight, c.ds, c.dx, part, c.M, (int)c.d, c.eps, c.weight_f32};
    const bool ragged = c.d % (c.f32 ? 4 : 8) != 0;
    const cudaError_t e =
        c.f32 ? (ragged ? launch_back<true, true>(a, s, st) : launch_back<true, false>(a, s, st))
              : (ragged ? launch_back<false, true>(a, s, st) : launch_back<false, false>(a, s, st));
    if (e != cudaSuccess) return e;
  }
  return launch_chained(dweight_kernel, dim3((unsigned)((c.d + kSumCols - 1) / kSumCols)),
                        dim3(kSumCols * kSumRows), 0, st, (const float*)part, s.units, (int)c.d,
                        c.dweight, c.weight_f32);
}

}  // namespace swg
