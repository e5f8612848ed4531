// Rows sorted by expert, and back, with their gradients (see rows.h):
//
//   permute:    out[position[t, j]] = x[t]
//   unpermute:  y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]]
//   gradient of unpermute:
//               dz[position[t, j]] = weights[t, j] dy[t]
//               dweights[t, j] = dy[t] . z[position[t, j]]
//
// (the gradient of permute is unpermute without weights).  All go by token, not
// by sorted row, so that x and dy come from memory once however many choices
// there are (where a kernel reads them again, they are in L2).  Rows from
// offsets[E] on belong to no pair; as many choices are dropped as there are such
// rows, so the (t, j) whose flat index is such a row's clears it.
//
// Rows are moved in 16-byte pieces that start on 16-byte boundaries of the
// tensor that is written.  Where a row's bytes are no multiple of 16 (RAGGED),
// the source starts elsewhere in its 16 bytes: two of its pieces are shifted
// together.
//
// Bound by memory.  In a graph: 16384 tokens to 8 experts each, e4m3 rows of 4096
// with scales, 91.9 us (6580 GB/s, where a copy reaches 6780); the weighted sum
// back of 4096 tokens, k = 8, bf16, d = 4096 49.1 us (6570); its gradients, d =
// 2048, 42.6 us (6550), d = 4096 86.5; the eight rows of one token 1.8, 2.0 and 3.3.
#include "rows.cuh"
#include "rows.h"

namespace swg {
namespace {

// A CTA has blockDim.y tokens, blockDim.x threads (whole warps) for a piece of each row.
__device__ __forceinline__ int64_t token() {
  return (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
}

__device__ __forceinline__ int64_t sorted_end(const int* offsets, int E, int64_t rows) {
  const int64_t n = offsets[E];
  return n < 0 ? 0 : n < rows ? n : rows;
}

// A token's choices (k <= 32), one per lane: place (-1: none) and weight, which
// a warp reads once and hands around.
struct Choices {
  int p;
  float w;
  __device__ __forceinline__ Choices(const int* position, const float* weights, int64_t t, int k,
                                     int64_t rows)
      : p(-1), w(0.f) {
    const int l = threadIdx.x & 31;
    if (l < k) {
      p = position[t * k + l];
      if (p >= rows) p = -1;
      if (p >= 0) w = weights ? weights[t * k + l] : 1.f;
    }
  }
  __device__ __forceinline__ int place(int j) const { return __shfl_sync(0xffffffffu, p, j); }
  __device__ __forceinline__ float weight(int j) const { return __shfl_sync(0xffffffffu, w, j); }
};

// 16 bytes that may be in two pieces of their tensor.
struct Two {
  uint4 lo, hi;
};

// Rows of `bytes` bytes (a multiple of sizeof(E)); this one in 16-byte pieces
// that start on 16-byte boundaries of its tensor.
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
  // What piece i of this row would be if it held row `src` of the tensor of
  // `total` bytes at `p`: the loads, and afterwards the value, with neighbours'
  // bytes where they are not the row's.  (In two steps, and without a branch
  // around the loads, so that the loads of several rows are under way together.
  // The tensor's last bytes, where they fill no 16, are read one by one.)
  __device__ __forceinline__ Two begin(const void* p, int64_t src, int64_t total, int i) const {
    const int64_t at = src * bytes + (int64_t)i * 16 - shift;
    Two q;
    if (!RAGGED) {
      q.lo = load_once((const char*)p + at);
    } else {
      const int64_t last = (total & ~(int64_t)15) - 16, a0 = at & ~(int64_t)15;
      const int64_t l = a0 < 0 ? 0 : a0 < last ? a0 : last, h = a0 + 16 < last ? a0 + 16 : last;
      if (last >= 0) {
        q.lo = *reinterpret_cast<const uint4*>((const char*)p + l);
        q.hi = *reinterpret_cast<const uint4*>((const char*)p + h);
      }
    }
    return q;
  }
  __device__ __forceinline__ uint4 end(const Two& q, const void* p, int64_t src, int64_t total,
                                       int i) const {
    if (!RAGGED) return q.lo;
    const int64_t at = src * bytes + (int64_t)i * 16 - shift, a0 = at & ~(int64_t)15;
    const int sh = (int)(at & 15);
    if (a0 + 32 <= total) return shift_bytes(q.lo, q.hi, sh);
    return shift_bytes(load_inside<E>(p, a0, total), load_inside<E>(p, a0 + 16, total), sh);
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

// Rows of whole 16-byte pieces, `per` of them.
__global__ void __launch_bounds__(256, 6)
permute_kernel(const uint4* x, const float* scales, const int* position, const int* offsets,
               uint4* out, float* out_scales, int64_t T, int k, int n_exp, int per) {
  constexpr int B = 8;   // choices whose places are read together
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  if (t >= T) return;
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows), f0 = t * k;
  const int w0 = blockIdx.y * blockDim.x + threadIdx.x, step = gridDim.y * blockDim.x;
  const float s = scales && w0 == 0 ? scales[t] : 0.f;
  for (int j0 = 0; j0 < k; j0 += B) {
    int p[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      p[b] = j0 + b < k ? position[f0 + j0 + b] : -1;
      if (p[b] >= rows) p[b] = -1;
    }
    // (the rows of no pair that these choices clear: z ... last - 1)
    const int64_t last = f0 + (j0 + B < k ? j0 + B : k);
    const int64_t z = f0 + j0 > end ? f0 + j0 : end;
    for (int w = w0; w < per; w += step) {
      const uint4 v = load_once(x + t * per + w);
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (p[b] >= 0) out[(int64_t)p[b] * per + w] = v;
      for (int64_t r = z; r < last; ++r) out[r * per + w] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (scales && w0 == 0) {
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (p[b] >= 0) out_scales[p[b]] = s;
      for (int64_t r = z; r < last; ++r) out_scales[r] = 0.f;
    }
  }
}

// ---- rows that stream through a warp ---------------------------------------------
//
// A warp takes items (a token and 32 U pieces of its row) one after the other,
// B choices at a time, and copies what the next steps need (cp.async) into its
// own slots in shared memory while it works on one: no barrier but the warp's,
// no registers for what is under way, and a row that starts elsewhere in its 16
// bytes is read once, each thread taking its second half from its neighbour's
// slot.

constexpr int kPermuteWarps = 16;   // of permute's CTA for ragged rows, two per SM

// Pieces m of 16 bytes from byte `at` of a tensor of `total` bytes into
// slots[m], m < count <= N; zero where they are outside it.
template <bool RAGGED, int N>
__device__ __forceinline__ void copy_row(uint4* slots, const void* p, int64_t at, int64_t total,
                                         int count, int l) {
  const char* src = (const char*)p + at;
  const bool inside = !RAGGED || (at >= 0 && at + (int64_t)count * 16 <= total);
#pragma unroll
  for (int i = 0; i < (N + 31) / 32; ++i) {
    const int m = l + 32 * i;
    if (m >= count || m >= N) continue;
    if (inside) {
      copy_piece(slots + m, src + m * 16, 16);
    } else {
      const int64_t a = at + m * 16;
      const int bytes = a < 0 || a >= total ? 0 : total - a < 16 ? (int)(total - a) : 16;
      copy_piece(slots + m, bytes ? src + m * 16 : (const char*)p, bytes);
    }
  }
}

// The steps of a warp: its items (token t, part a of na) are spread over the
// warps of the grid, and each takes nb steps b.
struct Steps {
  int64_t t, dt;
  int a, na, da, b, nb;
  __device__ __forceinline__ Steps(int na_, int nb_) : na(na_), b(0), nb(nb_) {
    const int64_t g = (int64_t)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    t = g / na;
    a = (int)(g - t * na);
    dt = step / na;
    da = (int)(step - dt * na);
  }
  __device__ __forceinline__ bool last() const { return b + 1 == nb; }
  __device__ __forceinline__ void next() {
    if (++b < nb) return;
    b = 0;
    t += dt;
    a += da;
    if (a >= na) {
      a -= na;
      ++t;
    }
  }
};
// k choices B at a time (one step where there are none).
template <int B>
__device__ __forceinline__ int batches(int k) {
  return k > B ? (k + B - 1) / B : 1;
}

// Choices as they are copied (into slots c of place and weight): choice b of the
// B from j on of token t.  Lanes 0 ... B - 1 take the places, 8 ... 8 + B - 1
// the weights.
template <int B, typename Slots>
__device__ __forceinline__ void copy_choices(Slots& slots, int c, const int* position,
                                             const float* weights, int64_t t, int64_t T, int j,
                                             int k) {
  const int l = threadIdx.x & 31, b = l & 7;
  if (l >= 16 || b >= B || t >= T || j + b >= k) return;
  const int64_t f = t * k + j + b;
  if (l < 8) copy_word(&slots.place[c][b], position + f);
  else if (weights) copy_word(&slots.weight[c][b], weights + f);
}
// ... and its place, or -1.
template <typename Slots>
__device__ __forceinline__ int choice_place(const Slots& slots, int c, int j, int b, int k,
                                            int64_t rows) {
  const int p = slots.place[c][b];
  return j + b < k && p >= 0 && p < rows ? p : -1;
}
__device__ __forceinline__ int wrap(int i, int n) { return i + 1 == n ? 0 : i + 1; }

// Ragged permute: a warp's stages hold 64 pieces of a token's row, with one more
// on either side; the token's choices are copied S - 1 steps earlier.
struct PermuteSlots {
  static constexpr int S = 4, C = 2 * S - 1, U = 2;
  uint4 x[S][32 * U + 2];
  float scale[S][4];
  int place[C][32];
};

template <typename E>
__global__ void __launch_bounds__(32 * kPermuteWarps, 2)
permute_ragged_kernel(const void* x, const float* scales, const int* position,
                      const int* offsets, void* out, float* out_scales, int64_t T, int k, int n_exp,
                      int bytes, int segs) {
  constexpr int S = PermuteSlots::S, C = PermuteSlots::C, U = PermuteSlots::U;
  extern __shared__ uint4 smem[];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int l = threadIdx.x & 31;
  PermuteSlots& slots = reinterpret_cast<PermuteSlots*>(smem)[threadIdx.x >> 5];
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows);
  Steps ask(segs, 1), in = ask, out_s = ask;   // a: segments, all choices in one step
  int ask_c = 0, out_c = 0;
  const auto choices = [&]() {
    if (l < k && ask.t < T) copy_word(&slots.place[ask_c][l], position + ask.t * k + l);
    ask.next();
    ask_c = wrap(ask_c, C);
  };
  const auto fetch = [&](int stage) {
    if (in.t < T) {
      const int64_t base = in.t * bytes;
      copy_row<true, 32 * U + 2>(slots.x[stage], x, (base & ~(int64_t)15) + ((int64_t)in.a * 32 * U - 1) * 16,
                                 T * bytes, 32 * U + 2, l);
      if (scales && l == 0) copy_word(&slots.scale[stage][0], scales + in.t);
    }
    in.next();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) choices();
  copies_commit();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(i);
    choices();
    copies_commit();
  }
  int stage = 0, free_stage = S - 1;
  while (out_s.t < T) {
    copies_wait<S - 2>();
    __syncwarp();
    fetch(free_stage);
    choices();
    copies_commit();
    const int64_t t = out_s.t, f0 = t * k, src = t * bytes;
    const int i0 = out_s.a * 32 * U;
    for (int j = 0; j < k; ++j) {
      const int p = slots.place[out_c][j];
      if (p >= 0 && p < rows) {
        const Span16<E, true> o(p, bytes);
        // piece i of the output is in the source's pieces i + off and i + off + 1
        const int off = (int)(((src - o.shift) >> 4) - (src >> 4));
        const int sh = (int)((src - o.shift) & 15);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int m = l + 32 * u;
          if (i0 + m < o.n)
            o.put(out, i0 + m, shift_bytes(slots.x[stage][m + 1 + off], slots.x[stage][m + 2 + off], sh));
        }
        if (scales && out_s.a == 0 && l == 0) out_scales[p] = slots.scale[stage][0];
      }
      if (f0 + j >= end) {
        const Span16<E, true> o(f0 + j, bytes);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + l + 32 * u < o.n) o.put(out, i0 + l + 32 * u, make_uint4(0u, 0u, 0u, 0u));
        if (scales && out_s.a == 0 && l == 0) out_scales[f0 + j] = 0.f;
      }
    }
    out_s.next();
    out_c = wrap(out_c, C);
    stage = wrap(stage, S);
    free_stage = wrap(free_stage, S);
  }
}

// Few pieces (see kFewPieces): each has a thread of its own.
template <bool F32, bool RAGGED>
__global__ void __launch_bounds__(256)
unpermute_few_kernel(const void* z, const int* position, const float* weights,
                     const void* residual, void* y, int64_t T, int k, int bytes) {
  using E = typename Row<F32>::elem;
  constexpr int H = Row<F32>::kVec / 2, B = 8;
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  if (t >= T) return;
  const int64_t rows = T * k;
  const Choices ch(position, weights, t, k, rows);
  const Span16<E, RAGGED> o(t, bytes);
  const int i = blockIdx.y * blockDim.x + threadIdx.x;
  uint4 rq = make_uint4(0u, 0u, 0u, 0u);
  if (residual && i < o.n) rq = load_inside<E>(residual, o.base - o.shift + (int64_t)i * 16, T * bytes);
  float2 acc[H];
  unpack<F32>(rq, acc);
  for (int j0 = 0; j0 < k; j0 += B) {
    Two q[B];
    int p[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      p[b] = ch.place(j0 + b);
      if (p[b] >= 0 && i < o.n) q[b] = o.begin(z, p[b], rows * bytes, i);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float c = ch.weight(j0 + b);
      if (p[b] < 0 || i >= o.n) continue;
      float2 v[H];
      unpack<F32>(o.end(q[b], z, p[b], rows * bytes, i), v);
#pragma unroll
      for (int h = 0; h < H; ++h) acc[h] = fma2(make_float2(c, c), v[h], acc[h]);
    }
  }
  if (i < o.n) o.put(y, i, pack<F32>(acc));
}

// What a warp of unpermute keeps: S stages of pieces, and the steps' choices,
// which are copied S - 1 steps before the rows that they name.
template <bool F32, bool RAGGED, int B, int U>
struct UnpermuteSlots {
  static constexpr int kWarps = 16;   // of a CTA, one CTA per SM (12 with a stage more: 51.2 us
                                      // for 4096 tokens, k = 8, d = 4096, where 16 take 49.6)
  static constexpr int S = U == 1 && !RAGGED ? 3 : 2, C = 2 * S - 1;
  uint4 z[S][B][32 * U + (RAGGED ? 1 : 0)];
  uint4 residual[S][32 * U];
  int place[C][8];
  float weight[C][8];
};

// B choices of U pieces each to a step.
template <bool F32, bool RAGGED, int B, int U>
__global__ void __launch_bounds__(32 * UnpermuteSlots<F32, RAGGED, B, U>::kWarps, 1)
unpermute_kernel(const void* z, const int* position, const float* weights, const void* residual,
                 void* y, int64_t T, int k, int bytes, int segs) {
  using E = typename Row<F32>::elem;
  using Slots = UnpermuteSlots<F32, RAGGED, B, U>;
  constexpr int H = Row<F32>::kVec / 2, S = Slots::S, C = Slots::C;
  extern __shared__ uint4 smem[];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int l = threadIdx.x & 31;
  Slots& slots = reinterpret_cast<Slots*>(smem)[threadIdx.x >> 5];
  const int64_t rows = T * k;

  // choices copied, rows copied, at work (a: segments, b: batches of choices)
  Steps ask(segs, batches<B>(k)), in = ask, out = ask;
  int ask_c = 0, in_c = 0, out_c = 0;   // their places among the C
  const auto choices = [&]() {
    copy_choices<B>(slots, ask_c, position, weights, ask.t, T, ask.b * B, k);
    ask.next();
    ask_c = wrap(ask_c, C);
  };
  const auto fetch = [&](int stage) {
    if (in.t < T) {
      const Span16<E, RAGGED> o(in.t, bytes);
      const int i0 = in.a * 32 * U;
      const int count = o.n - i0 < 32 * U ? o.n - i0 : 32 * U;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int p = choice_place(slots, in_c, in.b * B, b, k, rows);
        if (p < 0) continue;
        const int64_t at = (int64_t)p * bytes + (int64_t)i0 * 16 - o.shift;
        copy_row<RAGGED, 32 * U + (RAGGED ? 1 : 0)>(slots.z[stage][b], z, at & ~(int64_t)15,
                                                    rows * bytes, RAGGED ? count + 1 : count, l);
      }
      if (residual && in.b == 0)
        copy_row<RAGGED, 32 * U>(slots.residual[stage], residual,
                                 o.base - o.shift + (int64_t)i0 * 16, T * bytes, count, l);
    }
    in.next();
    in_c = wrap(in_c, C);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) choices();
  copies_commit();
  copies_wait<0>();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(i);
    choices();
    copies_commit();
  }
  int stage = 0, free_stage = S - 1;
  float2 acc[U][H];
  while (out.t < T) {
    // this step's rows are here, and the choices of the step S - 1 ahead
    copies_wait<S - 2>();
    __syncwarp();
    fetch(free_stage);
    choices();
    copies_commit();
    const Span16<E, RAGGED> o(out.t, bytes);
    const int i0 = out.a * 32 * U;
    if (out.b == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (residual) {
          unpack<F32>(slots.residual[stage][l + 32 * u], acc[u]);
        } else {
#pragma unroll
          for (int h = 0; h < H; ++h) acc[u][h] = make_float2(0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int p = choice_place(slots, out_c, out.b * B, b, k, rows);
      if (p < 0) continue;
      const float w = weights ? slots.weight[out_c][b] : 1.f;
      const int sh = RAGGED ? (int)((unsigned)p * (unsigned)bytes - o.shift) & 15 : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + 32 * u >= o.n) break;
        uint4 q = slots.z[stage][b][l + 32 * u];
        if (RAGGED) q = shift_bytes(q, slots.z[stage][b][l + 32 * u + 1], sh);
        float2 v[H];
        unpack<F32>(q, v);
#pragma unroll
        for (int h = 0; h < H; ++h) acc[u][h] = fma2(make_float2(w, w), v[h], acc[u][h]);
      }
    }
    if (out.last()) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + l + 32 * u < o.n) o.put(y, i0 + l + 32 * u, pack<F32>(acc[u]));
    }
    out.next();
    out_c = wrap(out_c, C);
    stage = wrap(stage, S);
    free_stage = wrap(free_stage, S);
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

// One piece of dz and of the dot product: piece i of row o of dz and z, where dyq
// and zq are dy's and z's values.
template <bool F32, bool RAGGED, typename S>
__device__ __forceinline__ void backward_piece(const S& o, void* dz, int i, const uint4& dyq,
                                               const uint4& zq, float w, float2& dot) {
  constexpr int V = Row<F32>::kVec, H = V / 2;
  float2 v[H], m[H];
  unpack<F32>(zq, v);
  unpack<F32>(dyq, m);
  if (RAGGED) {
    const int c0 = i * V - o.shift / (16 / V), d = o.bytes / (16 / V);
    if (c0 < 0 || c0 + V > d) {   // (not the neighbours' values, which may be NaN)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (c0 + 2 * h < 0 || c0 + 2 * h >= d) v[h].x = m[h].x = 0.f;
        if (c0 + 2 * h + 1 < 0 || c0 + 2 * h + 1 >= d) v[h].y = m[h].y = 0.f;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    dot = fma2(m[h], v[h], dot);
    v[h] = mul2(make_float2(w, w), m[h]);
  }
  o.put(dz, i, pack<F32>(v));
}

// Gradient of unpermute.  A warp has B choices of a token for the whole row, so
// that it ends with their dot products: nothing is shared between warps, and
// there are enough items for an even spread (dy is read again for the next B,
// from L2).  The pieces are those of z's and dz's row, so that these move as they
// are; dy, where it starts elsewhere in its 16 bytes, is shifted.
template <bool RAGGED, int B, int U>
struct BackwardSlots {
  // Of a CTA, one CTA per SM.  With runs of 256 pieces there may also be too much
  // under way: 8 / 10 / 12 / 14 warps take 88.5 / 86.5 / 95.8 / 98.6 us for 4096
  // tokens, k = 8, d = 4096, and 44.6 / 42.6 / 43.0 / 44.6 for d = 2048.
  static constexpr int kWarps = U == 8 ? 10 : 16;
  static constexpr int S = U == 1 ? 3 : 2, C = 2 * S - 1;
  uint4 z[S][B][32 * U];
  uint4 dy[S][32 * U + (RAGGED ? 2 : 0)];   // ragged: one more on either side
  int place[C][8];
  float weight[C][8];
};

template <bool F32, bool RAGGED, int B, int U>
__global__ void __launch_bounds__(32 * BackwardSlots<RAGGED, B, U>::kWarps, 1)
unpermute_backward_kernel(const void* dy, const void* z, const int* position, const int* offsets,
                          const float* weights, void* dz, float* dweights, int64_t T, int k,
                          int n_exp, int bytes, int segs) {
  using E = typename Row<F32>::elem;
  using Slots = BackwardSlots<RAGGED, B, U>;
  constexpr int S = Slots::S, C = Slots::C;
  extern __shared__ uint4 smem[];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int l = threadIdx.x & 31;
  Slots& slots = reinterpret_cast<Slots*>(smem)[threadIdx.x >> 5];
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows);

  // choices copied, rows copied, at work (a: batches of choices, b: segments)
  Steps ask(batches<B>(k), segs), in = ask, out = ask;
  int ask_c = 0, in_c = 0, out_c = 0;
  const auto choices = [&]() {
    copy_choices<B>(slots, ask_c, position, weights, ask.t, T, ask.a * B, k);
    ask.next();
    ask_c = wrap(ask_c, C);
  };
  const auto fetch = [&](int stage) {
    if (in.t < T) {
      const int i0 = in.b * 32 * U;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int p = choice_place(slots, in_c, in.a * B, b, k, rows);
        if (p < 0) continue;
        const Span16<E, RAGGED> o(p, bytes);
        copy_row<RAGGED, 32 * U>(slots.z[stage][b], z, o.base - o.shift + (int64_t)i0 * 16,
                                 rows * bytes, o.n - i0, l);
      }
      const int64_t src = in.t * bytes;
      if (RAGGED)
        copy_row<true, 32 * U + 2>(slots.dy[stage], dy, (src & ~(int64_t)15) + (int64_t)(i0 - 1) * 16,
                                   T * bytes, 32 * U + 2, l);
      else
        copy_row<false, 32 * U>(slots.dy[stage], dy, src + (int64_t)i0 * 16, T * bytes,
                                bytes / 16 - i0, l);
    }
    in.next();
    in_c = wrap(in_c, C);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) choices();
  copies_commit();
  copies_wait<0>();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(i);
    choices();
    copies_commit();
  }
  int stage = 0, free_stage = S - 1;
  float2 dot[B];
#pragma unroll
  for (int b = 0; b < B; ++b) dot[b] = make_float2(0.f, 0.f);
  while (out.t < T) {
    copies_wait<S - 2>();
    __syncwarp();
    fetch(free_stage);
    choices();
    copies_commit();
    const int i0 = out.b * 32 * U, j0 = out.a * B;
    const int64_t f0 = out.t * k + j0;
    const unsigned src = (unsigned)out.t * (unsigned)bytes;   // (its low bits count)
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int p = choice_place(slots, out_c, j0, b, k, rows);
      if (p >= 0) {
        const Span16<E, RAGGED> o(p, bytes);
        const float w = slots.weight[out_c][b];
        // dy's bytes for piece i are in its pieces i + off and i + off + 1
        const int off = RAGGED ? ((int)(src & 15) < o.shift ? -1 : 0) : 0;
        const int sh = RAGGED ? (int)(src - o.shift) & 15 : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int m = l + 32 * u, i = i0 + m;
          if (i >= o.n) continue;
          const uint4* d4 = &slots.dy[stage][RAGGED ? m + 1 + off : m];
          backward_piece<F32, RAGGED>(o, dz, i, RAGGED ? shift_bytes(d4[0], d4[1], sh) : d4[0],
                                      slots.z[stage][b][m], w, dot[b]);
        }
      }
      if (j0 + b < k && f0 + b >= end) {   // a row of no pair
        const Span16<E, RAGGED> o(f0 + b, bytes);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + l + 32 * u < o.n) o.put(dz, i0 + l + 32 * u, make_uint4(0u, 0u, 0u, 0u));
      }
    }
    if (out.last()) {
      float sums[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) sums[b] = b < B ? dot[b].x + dot[b].y : 0.f;
#pragma unroll
      for (int b = 0; b < B; ++b) dot[b] = make_float2(0.f, 0.f);
      const float v = warp_sums8(sums, l);
      if ((l & 3) == 0 && (l >> 2) < B && j0 + (l >> 2) < k) dweights[f0 + (l >> 2)] = v;
    }
    out.next();
    out_c = wrap(out_c, C);
    stage = wrap(stage, S);
    free_stage = wrap(free_stage, S);
  }
}

// Few pieces (see kFewPieces): blockDim.x threads to a token.
template <bool F32, bool RAGGED>
__global__ void __launch_bounds__(256)
unpermute_backward_few_kernel(const void* dy, const void* z, const int* position,
                              const int* offsets, const float* weights, void* dz, float* dweights,
                              int64_t T, int k, int n_exp, int bytes) {
  using E = typename Row<F32>::elem;
  constexpr int B = 8;
  __shared__ float red[8][8];   // by warp of the CTA
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int64_t t = token();
  const bool here = t < T;
  const int64_t rows = T * k, end = sorted_end(offsets, n_exp, rows), f0 = t * k;
  const int warps = blockDim.x >> 5;   // of a token
  const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, l = threadIdx.x & 31;
  const Choices ch(position, weights, t, here ? k : 0, rows);
  const int most = RAGGED ? bytes / 16 + 2 : bytes / 16;   // pieces of a row
  for (int j0 = 0; j0 < k; j0 += B) {
    int p[B];
    float c[B];
    float2 dot[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      p[b] = ch.place(j0 + b);
      c[b] = ch.weight(j0 + b);
      dot[b] = make_float2(0.f, 0.f);
    }
    for (int i = threadIdx.x; here && i < most; i += blockDim.x) {
      uint4 q[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const Span16<E, RAGGED> o(p[b], bytes);
        if (p[b] < 0 || i >= o.n) continue;
        const int64_t at = o.base - o.shift + (int64_t)i * 16;
        // (z may end inside the piece: its last row's, or of rows shorter than a
        // piece one that has several)
        if (!RAGGED || at + 16 <= rows * bytes) q[b] = load_once((const char*)z + at);
        else q[b] = load_inside<E>(z, at, rows * bytes);
      }
      Two g;
      if (!RAGGED) g.lo = load_once((const char*)dy + t * bytes + (int64_t)i * 16);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (p[b] < 0) continue;
        const Span16<E, RAGGED> o(p[b], bytes);
        if (i >= o.n) continue;
        if (RAGGED) g = o.begin(dy, t, T * bytes, i);
        backward_piece<F32, RAGGED>(o, dz, i, o.end(g, dy, t, T * bytes, i), q[b], c[b], dot[b]);
      }
    }
    // rows of no pair
    for (int j = j0; here && j < k && j < j0 + B; ++j) {
      if (f0 + j < end) continue;
      const Span16<E, RAGGED> o(f0 + j, bytes);
      for (int i = threadIdx.x; i < o.n; i += blockDim.x) o.put(dz, i, make_uint4(0u, 0u, 0u, 0u));
    }
    float sums[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) sums[b] = dot[b].x + dot[b].y;
    const float s = warp_sums8(sums, l);
    if ((l & 3) == 0) red[warp][l >> 2] = s;
    __syncthreads();
    if (here && threadIdx.x < B && j0 + (int)threadIdx.x < k) {
      float v = 0.f;
      for (int i = 0; i < warps; ++i) v += red[threadIdx.y * warps + i][threadIdx.x];
      dweights[f0 + j0 + threadIdx.x] = v;
    }
    if (j0 + B < k) __syncthreads();
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

// CTAs of a streaming kernel: no more than there are items.
int stream_grid(int64_t items, int most) { return (int)(items < most ? items : most); }

template <typename E>
cudaError_t permute_ragged(const PermuteCall& c, int num_sms, cudaStream_t st) {
  constexpr int smem = kPermuteWarps * (int)sizeof(PermuteSlots);
  static_assert(2 * smem <= 225 * 1024, "shared memory");
  const int64_t bytes = c.d * c.elem, piece = 32 * PermuteSlots::U;
  const int64_t segs = (pieces_of(bytes) + piece - 1) / piece;
  return launch_chained_smem<permute_ragged_kernel<E>>(
      smem, dim3(stream_grid(c.T * segs, 2 * num_sms)), dim3(32 * kPermuteWarps), smem, st, c.x,
      c.scales, c.position, c.offsets, c.out, c.out_scales, c.T, (int)c.k, (int)c.E, (int)bytes,
      (int)segs);
}

// Up to this many 16-byte pieces of y (or dy) each has a thread, and nothing is
// copied ahead: one wave of threads, or little more.  In a graph, few / streamed:
// unpermute d = 4096, k = 2, 64 tokens (32768 pieces) 2.3 / 2.5 us, 256 tokens
// 2.5 / 2.8, 512 tokens 4.6 / 3.9; its gradient 2.7 / 5.1, 3.0 / 5.1, 6.1 / 5.2,
// and d = 1024, k = 8, 512 tokens (65536 pieces) 3.5 / 4.3, 1024 tokens 7.7 / 5.9.
// With more than four choices, unpermute's threads have as much under way
// themselves: d = 4096, k = 8, 256 tokens 4.2 / 4.8, 1024 tokens 13.7 / 15.8, 2048
// tokens 25.0 / 28.4, 4096 tokens 53.8 / 53.3.
constexpr int64_t kFewPieces = 152 * 640, kFewPiecesManyChoices = (int64_t)1 << 20;

template <bool F32, bool RAGGED>
cudaError_t unpermute_few(const UnpermuteCall& c, int64_t bytes, cudaStream_t st) {
  const int64_t per = pieces_of(bytes);
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(unpermute_few_kernel<F32, RAGGED>,
                        dim3((unsigned)((c.T + block.y - 1) / block.y), (unsigned)((per + tx - 1) / tx)),
                        block, 0, st, c.z, c.position, c.weights, c.residual, c.y, c.T, (int)c.k,
                        (int)bytes);
}

template <bool F32, bool RAGGED, int B, int U>
cudaError_t unpermute_batch(const UnpermuteCall& c, int64_t bytes, int num_sms, cudaStream_t st) {
  using Slots = UnpermuteSlots<F32, RAGGED, B, U>;
  constexpr int smem = Slots::kWarps * (int)sizeof(Slots);
  static_assert(smem <= 232448, "shared memory");
  const int64_t segs = (pieces_of(bytes) + 32 * U - 1) / (32 * U);
  return launch_chained_smem<unpermute_kernel<F32, RAGGED, B, U>>(
      smem, dim3(stream_grid(c.T * segs, num_sms)), dim3(32 * Slots::kWarps), smem, st, c.z,
      c.position, c.weights, c.residual, c.y, c.T, (int)c.k, (int)bytes, (int)segs);
}

template <bool F32, bool RAGGED>
cudaError_t unpermute_rows(const UnpermuteCall& c, int64_t bytes, int num_sms, cudaStream_t st) {
  const int64_t per = pieces_of(bytes);
  if (c.T * per <= (c.k > 4 ? kFewPiecesManyChoices : kFewPieces))
    return unpermute_few<F32, RAGGED>(c, bytes, st);
  if (per >= 128 || c.k <= 2) return unpermute_batch<F32, RAGGED, 2, 4>(c, bytes, num_sms, st);
  if (per >= 64 || c.k <= 4) return unpermute_batch<F32, RAGGED, 4, 2>(c, bytes, num_sms, st);
  return unpermute_batch<F32, RAGGED, 8, 1>(c, bytes, num_sms, st);
}

template <bool F32, bool RAGGED, int B, int U>
cudaError_t backward_batch(const UnpermuteBackwardCall& c, int64_t bytes, int num_sms,
                           cudaStream_t st) {
  using Slots = BackwardSlots<RAGGED, B, U>;
  constexpr int smem = Slots::kWarps * (int)sizeof(Slots);
  static_assert(smem <= 232448, "shared memory");
  const int64_t segs = (pieces_of(bytes) + 32 * U - 1) / (32 * U);
  return launch_chained_smem<unpermute_backward_kernel<F32, RAGGED, B, U>>(
      smem, dim3(stream_grid(c.T * ((c.k + B - 1) / B), num_sms)), dim3(32 * Slots::kWarps), smem, st,
      c.dy, c.z, c.position, c.offsets, c.weights, c.dz, c.dweights, c.T, (int)c.k, (int)c.E, (int)bytes,
      (int)segs);
}

template <bool F32, bool RAGGED>
cudaError_t backward_rows(const UnpermuteBackwardCall& c, int64_t bytes, int num_sms,
                          cudaStream_t st) {
  const int64_t per = pieces_of(bytes);
  if (c.T * per <= kFewPieces || c.d == 0) {
    const int tx = row_threads(per);
    const dim3 block(tx, 256 / tx);
    return launch_chained(unpermute_backward_few_kernel<F32, RAGGED>,
                          dim3((unsigned)((c.T + block.y - 1) / block.y)), block, 0, st, c.dy, c.z,
                          c.position, c.offsets, c.weights, c.dz, c.dweights, c.T, (int)c.k,
                          (int)c.E, (int)bytes);
  }
  // Long rows: the longer a run of a row that a step moves, the better, also at
  // the price of reading dy once for each choice (from L2; 4096 tokens, k = 8, d =
  // 2048: 51.9 us in runs of 32 pieces, 46.7 of 64, 44.6 of 128, 42.7 of 256).
  // Ragged ones, which are bound by instructions, are better off with two choices
  // (d = 2047: 80 us with one, 60 with two).
  if constexpr (!RAGGED)
    if (per >= 256) return backward_batch<F32, RAGGED, 1, 8>(c, bytes, num_sms, st);
  if (per >= 128 || c.k <= 2) return backward_batch<F32, RAGGED, 2, 4>(c, bytes, num_sms, st);
  if (per >= 64 || c.k <= 4) return backward_batch<F32, RAGGED, 4, 2>(c, bytes, num_sms, st);
  return backward_batch<F32, RAGGED, 8, 1>(c, bytes, num_sms, st);
}

}  // namespace

cudaError_t launch_permute(const PermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.k == 0 || (c.d == 0 && !c.scales)) return cudaSuccess;
  if (c.d * c.elem % 16) {
    if (c.elem == 4) return permute_ragged<uint32_t>(c, num_sms, st);
    if (c.elem == 2) return permute_ragged<uint16_t>(c, num_sms, st);
    return permute_ragged<uint8_t>(c, num_sms, st);
  }
  const int64_t per = c.d * c.elem / 16;
  const int tx = row_threads(per);
  const dim3 block(tx, 256 / tx);
  return launch_chained(permute_kernel, grid_of(c.T, per, block), block, 0, st, (const uint4*)c.x,
                        c.scales, c.position, c.offsets, (uint4*)c.out, c.out_scales, c.T, (int)c.k,
                        (int)c.E, (int)per);
}

cudaError_t launch_unpermute(const UnpermuteCall& c, int num_sms, cudaStream_t st) {
  if (c.T == 0 || c.d == 0) return cudaSuccess;
  const int64_t bytes = c.d * (c.f32 ? 4 : 2);
  if (c.f32)
    return bytes % 16 ? unpermute_rows<true, true>(c, bytes, num_sms, st)
                      : unpermute_rows<true, false>(c, bytes, num_sms, st);
  return bytes % 16 ? unpermute_rows<false, true>(c, bytes, num_sms, st)
                    : unpermute_rows<false, false>(c, bytes, num_sms, st);
}

cudaError_t launch_unpermute_backward(const UnpermuteBackwardCall& c, int num_sms,
                                      cudaStream_t st) {
  if (c.T == 0 || c.k == 0) return cudaSuccess;
  const int64_t bytes = c.d * (c.f32 ? 4 : 2);
  if (c.f32)
    return bytes % 16 ? backward_rows<true, true>(c, bytes, num_sms, st)
                      : backward_rows<true, false>(c, bytes, num_sms, st);
  return bytes % 16 ? backward_rows<false, true>(c, bytes, num_sms, st)
                    : backward_rows<false, false>(c, bytes, num_sms, st);
}

}  // namespace swg
