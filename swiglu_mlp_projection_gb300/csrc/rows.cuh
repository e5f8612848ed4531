// Device helpers of the row operators: 16-byte pieces of bf16 or f32 rows.
#pragma once

#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "tc_common.cuh"

namespace swg {

template <bool F32> struct Row;
template <> struct Row<true> {
  using elem = float;
  static constexpr int kVec = 4;   // elements of 16 bytes
};
template <> struct Row<false> {
  using elem = uint16_t;
  static constexpr int kVec = 8;
};

// (the instruction rounds to nearest even and keeps NaN)
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(uint16_t v) { return bf16_lo(v); }
__device__ __forceinline__ void set_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void set_elem(uint16_t* p, float v) { *p = (uint16_t)bf16x2(v, 0.f); }

// 16 bytes as pairs of f32 values, and back.
template <bool F32>
__device__ __forceinline__ void unpack(const uint4& q, float2 (&v)[Row<F32>::kVec / 2]) {
  if constexpr (F32) {
    v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
  } else {
    v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
    v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
    v[2] = make_float2(bf16_lo(q.z), bf16_hi(q.z));
    v[3] = make_float2(bf16_lo(q.w), bf16_hi(q.w));
  }
}

template <bool F32>
__device__ __forceinline__ uint4 pack(const float2 (&v)[Row<F32>::kVec / 2]) {
  if constexpr (F32)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
  else
    return make_uint4(bf16x2(v[0].x, v[0].y), bf16x2(v[1].x, v[1].y), bf16x2(v[2].x, v[2].y),
                      bf16x2(v[3].x, v[3].y));
}

// Two f32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

// 16 bytes that are read once.  (No .nc: the caller's output may be the input.)
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The 16 bytes from byte `sh` (0 ... 15) of lo and hi, one after the other.
__device__ __forceinline__ uint4 shift_bytes(const uint4& lo, const uint4& hi, int sh) {
  uint32_t w[6] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y};
  if (sh & 8) {
    w[0] = w[2]; w[1] = w[3]; w[2] = w[4]; w[3] = w[5]; w[4] = hi.z; w[5] = hi.w;
  }
  if (sh & 4) {
    w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = w[4]; w[4] = w[5];
  }
  const int b = 8 * (sh & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b),
                    __funnelshift_r(w[2], w[3], b), __funnelshift_r(w[3], w[4], b));
}

// The 16 bytes at byte `at` (a multiple of 16) of a tensor of `total` bytes;
// zero where that is outside it.  E: the tensor's elements.
template <typename E>
__device__ __forceinline__ uint4 load_inside(const void* p, int64_t at, int64_t total) {
  if (at >= 0 && at + 16 <= total) return *reinterpret_cast<const uint4*>((const char*)p + at);
  union {
    uint4 q;
    E e[16 / sizeof(E)];
  } u;
  u.q = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(E)); ++i)
    if (at >= 0 && at + (int64_t)(i * sizeof(E)) < total)
      u.e[i] = *reinterpret_cast<const E*>((const char*)p + at + i * sizeof(E));
  return u.q;
}

// A row of d elements in 16-byte pieces that start on 16-byte boundaries of
// the tensor, whatever d is: piece i holds the row's elements i * kVec - shift
// and on, of which those in 0 ... d - 1 are the row's own (the others are its
// neighbours': not used when the first or last piece is read, not touched when
// it is written).  Without RAGGED (d a multiple of kVec) shift is 0 and every
// piece is whole.
template <bool F32, bool RAGGED>
struct Pieces {
  static constexpr int V = Row<F32>::kVec;
  using E = typename Row<F32>::elem;
  int64_t first;   // flat index of piece 0's first element
  int shift, n, d;

  __device__ __forceinline__ Pieces(int64_t row, int d_) : d(d_) {
    const int64_t base = row * d_;
    shift = RAGGED ? (int)(base & (V - 1)) : 0;
    first = base - shift;
    n = RAGGED ? (shift + d_ + V - 1) / V : d_ / V;
  }
  __device__ __forceinline__ int col(int i) const { return i * V - shift; }
  __device__ __forceinline__ bool whole(int i) const {
    return !RAGGED || (col(i) >= 0 && col(i) + V <= d);
  }
  __device__ __forceinline__ bool has(int i, int e) const {
    return !RAGGED || (col(i) + e >= 0 && col(i) + e < d);
  }
  // Piece i of bf16 with all bits set where it has the row's elements.
  __device__ __forceinline__ uint4 ones(int i) const {
    uint32_t m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = (has(i, 2 * k) ? 0xffffu : 0u) | (has(i, 2 * k + 1) ? 0xffff0000u : 0u);
    return make_uint4(m[0], m[1], m[2], m[3]);
  }
  // Elements that are not the row's become 0.
  __device__ __forceinline__ void mask(int i, float2 (&v)[V / 2]) const {
    if (!whole(i)) {
#pragma unroll
      for (int h = 0; h < V / 2; ++h) {
        if (!has(i, 2 * h)) v[h].x = 0.f;
        if (!has(i, 2 * h + 1)) v[h].y = 0.f;
      }
    }
  }

  // Piece i of the tensor of `rows` rows at `p`, with neighbours' elements (see mask).
  __device__ __forceinline__ uint4 load(const void* p, int64_t rows, int i) const {
    const int64_t at = first + (int64_t)i * V;
    if (!RAGGED || at + V <= rows * d) return load_once((const E*)p + at);
    return load_inside<E>(p, at * (16 / V), rows * d * (16 / V));
  }
  __device__ __forceinline__ void store(void* p, int i, const float2 (&v)[V / 2]) const {
    store_at(p, first, i, v);
  }
  // Into another row that starts at the same place of its 16 bytes: its piece 0 at `at`.
  __device__ __forceinline__ void store_at(void* p, int64_t at, int i,
                                           const float2 (&v)[V / 2]) const {
    E* q = (E*)p + at + (int64_t)i * V;
    if (whole(i)) {
      *reinterpret_cast<uint4*>(q) = pack<F32>(v);
    } else {
      if constexpr (F32) {
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
          if (has(i, 2 * h)) q[2 * h] = v[h].x;
          if (has(i, 2 * h + 1)) q[2 * h + 1] = v[h].y;
        }
      } else {
        store_part(q, pack<F32>(v), col(i) < 0 ? -col(i) : 0, col(i) + V <= d ? V : d - col(i));
      }
    }
  }
  // Elements [lo, hi) of eight, and not all: the warps that have a row's ends keep
  // the others waiting, so three stores at most in place of one for each element
  // (with the norm's masks of such pieces, the gradient of 4096 x 8191 72 -> 57 us,
  // of 2048 x 12001 54 -> 46; of f32's four elements the plain form is the faster).
  __device__ __forceinline__ static void store_part(uint16_t* q, const uint4& u, int lo, int hi) {
    if (lo == 0) {   // 4, 2 and 1 of them, as hi has them
      const bool four = hi & 4, two = hi & 2;
      if (four) *reinterpret_cast<uint2*>(q) = make_uint2(u.x, u.y);
      if (two) *reinterpret_cast<uint32_t*>(q + (hi & 4)) = four ? u.z : u.x;
      if (hi & 1) q[hi - 1] = (uint16_t)(four ? (two ? u.w : u.z) : two ? u.y : u.x);
    } else if (hi == 8) {   // the same from the end
      const int n = 8 - lo;
      const bool four = n & 4, two = n & 2;
      if (four) *reinterpret_cast<uint2*>(q + 4) = make_uint2(u.z, u.w);
      if (two) *reinterpret_cast<uint32_t*>(q + (6 - (n & 4))) = four ? u.y : u.w;
      if (n & 1) q[lo] = (uint16_t)((four ? (two ? u.x : u.y) : two ? u.z : u.w) >> 16);
    } else {   // a row inside a piece
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= lo && e < hi) q[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
  }
  // The piece's e4m3 codes into a tensor of codes, which has V bytes where this one has 16.
  __device__ __forceinline__ void store_codes(void* p, int64_t at, int i,
                                              const uint32_t (&c)[V / 4]) const {
    uint8_t* o = (uint8_t*)p + at + (int64_t)i * V;
    if (whole(i)) {
      if constexpr (V == 8) *reinterpret_cast<uint2*>(o) = make_uint2(c[0], c[1]);
      else *reinterpret_cast<uint32_t*>(o) = c[0];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (has(i, e)) o[e] = (uint8_t)(c[e / 4] >> (8 * (e & 3)));
    }
  }
  // What piece i of a vector [d] of bf16 or f32 values (the norm's weight) would
  // be if it started where the row does; 0 past its ends.
  __device__ __forceinline__ void weight(const void* w, int w_f32, int i,
                                         float2 (&v)[V / 2]) const {
    if (!RAGGED) {
      if (w_f32) {
        const float4* q = reinterpret_cast<const float4*>((const float*)w + i * V);
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
          const float4 f = q[h];
          v[2 * h] = make_float2(f.x, f.y);
          v[2 * h + 1] = make_float2(f.z, f.w);
        }
      } else if constexpr (V == 8) {
        unpack<false>(*reinterpret_cast<const uint4*>((const uint16_t*)w + i * V), v);
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>((const uint16_t*)w + i * V);
        v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
        v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
      }
    } else if (w_f32 == (F32 ? 1 : 0)) {   // the row's own type: two pieces, shifted
      constexpr int es = 16 / V;
      const int64_t at = (int64_t)(shift ? i - 1 : i) * 16;
      const uint4 lo = load_inside<E>(w, at, (int64_t)d * es);
      const uint4 hi = load_inside<E>(w, at + 16, (int64_t)d * es);
      unpack<F32>(shift ? shift_bytes(lo, hi, 16 - shift * es) : lo, v);
    } else {
      const auto one = [&](int e) {
        return !has(i, e) ? 0.f
               : w_f32    ? ((const float*)w)[col(i) + e]
                          : bf16_lo(((const uint16_t*)w)[col(i) + e]);
      };
#pragma unroll
      for (int h = 0; h < V / 2; ++h) v[h] = make_float2(one(2 * h), one(2 * h + 1));
    }
  }
};

// 16 bytes of which `bytes` are read and the rest zero.
__device__ __forceinline__ void copy_piece(uint4* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_word(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A launch that may begin while the previous kernel of the stream ends (the
// kernel waits in pdl_wait before it touches memory; it is running while that one
// still writes, so it reads nothing through the non-coherent path: no __ldg, no
// const __restrict__).
// `cluster` CTAs in a row are a cluster.
template <typename... Params, typename... Args>
inline cudaError_t launch_clustered(int cluster, void (*kernel)(Params...), dim3 grid, dim3 block,
                                    size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                  cudaStream_t st, Args... args) {
  return launch_clustered(1, kernel, grid, block, smem, st, args...);
}

// The same for a kernel that needs up to `most` bytes of shared memory, which is
// asked for once on each device.
template <auto kernel, int CLUSTER = 1, typename... Args>
inline cudaError_t launch_chained_smem(int most, dim3 grid, dim3 block, size_t smem,
                                       cudaStream_t st, Args... args) {
  static std::atomic<int> configured[64];   // zero: not yet set on that device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev].store(1, std::memory_order_release);
  }
  return launch_clustered(CLUSTER, kernel, grid, block, smem, st, args...);
}

}  // namespace swg
