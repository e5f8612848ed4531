// Interfaces of the mixture-of-experts kernels and of the general linear
// product: grouped products (grouped_tc.cu), routing and dispatch (route.cu),
// the weighted sum over a token's choices (combine.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace swg {

// The grouped kernel's epilogues.
enum GroupedMode : int { kGroupedSwiGLU = 0, kGroupedPlain = 1, kGroupedLinear = 2 };

// swiglu_activation values.
enum Activation : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxGroups = 32;

struct GroupedPlan {
  int pairs;             // CTA pairs of the launch
  int n_max;             // most rows of a chunk (a multiple of 32, at most 256)
  int stages;            // shared-memory ring
  uint32_t stage_bytes;
  int cut;               // whether units of a partial wave are cut along K
  int self_join;         // the last pair of a cut unit adds up its shares
  int min_kb;            // fewest k blocks of a share of a cut unit
  int prefetch_kb;       // linear: k blocks of weights asked into L2 per CTA before the
                         // previous kernel has ended
  size_t counters_bytes, part_bytes;
};

// rows: rows of the sorted operand; tokens: most rows that one expert can have.
GroupedPlan plan_grouped(int64_t rows, int64_t tokens, int64_t E, bool swiglu, int pairs,
                         const Tuning& tn);

struct GroupedCall {
  const void* x;           // [tokens, K] (SwiGLU) or [rows, K]
  const void* wa;          // [E, K, n_out] or [E, n_out, K]; SwiGLU: W_gate
  const void* wb;          // SwiGLU: W_up
  const int* offsets;      // [E + 1], or null: one group
  const int* order;        // SwiGLU: sorted row -> token * top_k + choice
  void* out;               // [rows, n_out]
  int out_f32;
  const void* bias;        // linear: [n_out] or null
  int bias_f32, act;
  const void* resid;       // linear: [rows, n_out] in out's type, or null
  int64_t rows, tokens, E, top_k, K, n_out;
  int wlayout;             // kWeightsKN or kWeightsNK
  void* padded = nullptr;  // linear, [K, n_out] with n_out no multiple of 8: room for
                           // K x round8(n_out) bf16
};

cudaError_t launch_grouped(int mode, const GroupedCall& c, const GroupedPlan& p, float* part,
                           unsigned* counters, bool counters_clean, unsigned* status,
                           uint64_t timeout_ns, cudaStream_t st);

struct Work;   // grouped_plan.cuh
void fill_work(Work* w, int mode, const GroupedCall& c, const GroupedPlan& p, float* part);

// y[t] = residual[t] + sum_j weights[t, j] z[position[t, j]], j ascending, in
// f32, rounded once (bf16).  position -1: no term.  `w`: the grouped product
// that wrote z (row r of a cut unit is in its shares instead); z null: no term
// at all.
cudaError_t launch_combine(const float* z, const Work* w, const int* position,
                           const float* weights, const void* residual, void* y, int64_t T,
                           int64_t k, int64_t rows, int64_t d, int num_sms, cudaStream_t st);

struct RouteCall {
  const void* logits;
  int logits_f32;
  const float* bias;
  int* ids;
  float* weights;
  int64_t T, E, k;
  int sigmoid, groups, topk_groups, group_top2, renormalize;
  float scale;
};

// Counting sort of the R = T k choices by expert, stable.
struct SortCall {
  int* offsets;
  int* order;
  int* position;
  int* scratch;        // dispatch_scratch_bytes or route_scratch_bytes
};
size_t dispatch_scratch_bytes(int64_t R, int64_t E, int num_sms);
size_t route_scratch_bytes(int64_t T, int64_t E, int num_sms);
cudaError_t launch_dispatch(const int* ids, const SortCall& s, int64_t R, int64_t E, int num_sms,
                            cudaStream_t st);
// sort: null, or where the sorted choices go.
cudaError_t launch_route(const RouteCall& c, const SortCall* sort, int num_sms, cudaStream_t st);

}  // namespace swg
