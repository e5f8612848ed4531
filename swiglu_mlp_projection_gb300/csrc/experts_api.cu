// C ABI of the mixture-of-experts operators and the general linear product:
// argument checks, workspace, launches.  See include/swiglu.h for the contract
// of each entry point.
#include <stdio.h>

#include "grouped.h"
#include "grouped_plan.cuh"
#include "internal.h"
#include "swiglu.h"

namespace swg {
namespace {

struct Span {
  const char* name;
  const void* p;
  size_t bytes;
  unsigned align = 16;   // what the kernels' loads of it need
};

int failf(int status, const char* fmt, const char* a, const char* b = "") {
  char text[256];
  snprintf(text, sizeof text, fmt, a, b);
  return api_fail(status, text);
}

// Every non-empty tensor has a pointer, aligned as its loads need.
int check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (s[i].bytes && !s[i].p)
      return failf(SWIGLU_ERR_INVALID_ARG, "null pointer for a non-empty tensor (%s)", s[i].name);
    if ((uintptr_t)s[i].p & (s[i].align - 1))
      return failf(SWIGLU_ERR_ALIGNMENT, "%s must be %s-byte aligned", s[i].name,
                   s[i].align == 16 ? "16" : s[i].align == 4 ? "4" : "2");
  }
  return SWIGLU_OK;
}

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

int check_apart(const Span& out, const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(out, s[i])) return failf(SWIGLU_ERR_INVALID_ARG, "%s overlaps %s", out.name, s[i].name);
  return SWIGLU_OK;
}

// Sizes of a product: within 31 bits, rows on 16-byte boundaries.
// (any_n: N may be any number, see swiglu_linear)
int check_product(int64_t rows, int64_t K, int64_t N, const char* kname, const char* nname,
                  bool any_n = false) {
  if (rows < 0 || K < 0 || N < 0) return api_fail(SWIGLU_ERR_INVALID_ARG, "negative size");
  if (rows > (int64_t)1 << 30 || K > (int64_t)1 << 30 || N > (int64_t)1 << 30)
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "a size exceeds 2^30");
  // (a TMA descriptor's strides, here the bytes of one matrix, end at 2^40)
  if (N > 0 && K >= ((int64_t)1 << 39) / N)
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "a weight matrix of 2^40 bytes or more");
  if (any_n && K % 8 != 0) return failf(SWIGLU_ERR_ALIGNMENT, "%s must be a multiple of 8", kname);
  if (!any_n && (K % 8 != 0 || N % 8 != 0))
    return failf(SWIGLU_ERR_ALIGNMENT, "%s and %s must be multiples of 8", kname, nname);
  return SWIGLU_OK;
}

int check_routing(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 0 || E < 1) return api_fail(SWIGLU_ERR_INVALID_ARG, "negative size or no experts");
  if (E > kMaxExperts) return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 1024 experts");
  if (k > kMaxTopK) return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 32 choices per token");
  if (k > E) return api_fail(SWIGLU_ERR_INVALID_ARG, "more choices per token than experts");
  if (T > (int64_t)1 << 30 || T * k > (int64_t)1 << 30)
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 2^30 choices");
  return SWIGLU_OK;
}

int check_layout(int layout) {
  if (layout != SWIGLU_WEIGHTS_KN && layout != SWIGLU_WEIGHTS_NK)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown weight layout");
  return SWIGLU_OK;
}

int wlayout_of(int layout) { return layout == SWIGLU_WEIGHTS_NK ? kWeightsNK : kWeightsKN; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The shares of cut units, and 256 bytes for the schedule.
size_t part_region(const GroupedPlan& p) { return round256(p.part_bytes) + 256; }

struct Device {
  int dev = 0, num_sms = 0, pairs = 0;
};

int get_device(Device* d) {
  int v = api_current_device(&d->dev, &d->num_sms);
  if (v != SWIGLU_OK) return v;
  const int most = api_max_pairs(d->dev);
  d->pairs = d->num_sms / 2 < most ? d->num_sms / 2 : most;
  return SWIGLU_OK;
}

// For a call without a workspace of its own: until it returns, no other
// thread's call on the stream comes between its kernels.
std::unique_lock<std::mutex> lock_calls(const Device& dv, cudaStream_t st, const void* workspace) {
  return workspace ? std::unique_lock<std::mutex>() : api_lock_enqueue(dv.dev, st);
}

// One grouped product with its workspace; `extra` bytes (z of the down
// projection, or padded weights) follow the partial sums.  The caller frees ws.pooled.
int run_grouped(int mode, GroupedCall c, const GroupedPlan& p, const Device& dv, void* workspace,
                size_t ws_bytes, size_t extra, Workspace* ws, cudaStream_t st) {
  const size_t body = part_region(p) + extra;
  int v = api_take_workspace(dv.dev, st, workspace, ws_bytes, p.counters_bytes, body, ws);
  if (v != SWIGLU_OK) return v;
  if (extra && mode == kGroupedPlain) c.out = ws->body + part_region(p);
  else if (extra) c.padded = ws->body + part_region(p);
  cudaError_t e = launch_grouped(mode, c, p, (float*)ws->body, ws->counters, ws->counters_clean,
                                 api_status_word(dv.dev), api_wait_timeout_ns(), st);
  if (e != cudaSuccess) {
    if (ws->pooled) cudaFreeAsync(ws->pooled, st);
    ws->pooled = nullptr;
    return api_cuda_fail(e, "kernel launch");
  }
  return SWIGLU_OK;
}

int free_workspace(const Workspace& ws, cudaStream_t st) {
  if (!ws.pooled) return SWIGLU_OK;
  const cudaError_t e = cudaFreeAsync(ws.pooled, st);
  return e == cudaSuccess ? SWIGLU_OK : api_cuda_fail(e, "cudaFreeAsync(workspace)");
}

GroupedPlan plan_experts(int64_t T, int64_t k, int64_t E, bool up, int pairs) {
  return plan_grouped(T * k, T, E, up, pairs, read_tuning());
}

// Room for [K, N] weights with padded rows (launch_grouped), where N asks for it.
size_t padded_bytes(int64_t K, int64_t N) {
  return N % 8 ? round256((size_t)K * (size_t)((N + 7) / 8 * 8) * 2) : 0;
}

size_t z_bytes(int64_t rows, int64_t d) { return round256((size_t)rows * d * sizeof(float)); }

}  // namespace
}  // namespace swg

using namespace swg;

extern "C" {

size_t swiglu_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_product(M, K, N, "K", "N", true) != SWIGLU_OK) return 0;
  Device dv;
  if (get_device(&dv) != SWIGLU_OK) return 0;
  const GroupedPlan p = plan_grouped(M, M, 1, false, dv.pairs, read_tuning());
  api_clear_error();
  return p.counters_bytes + part_region(p) + padded_bytes(K, N);
}

int swiglu_linear(const void* x, const void* w, const void* bias, const void* residual, void* y,
                  int64_t M, int64_t K, int64_t N, int activation, int bias_dtype, int out_dtype,
                  int layout, void* workspace, size_t workspace_bytes, void* stream) {
  int v = check_product(M, K, N, "K", "N", true);
  if (v != SWIGLU_OK) return v;
  if ((v = check_layout(layout)) != SWIGLU_OK) return v;
  if (activation < SWIGLU_ACT_NONE || activation > SWIGLU_ACT_GELU_TANH)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown activation");
  if ((bias_dtype != SWIGLU_F32 && bias_dtype != SWIGLU_BF16) ||
      (out_dtype != SWIGLU_F32 && out_dtype != SWIGLU_BF16))
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown dtype");
  const size_t oe = out_dtype == SWIGLU_F32 ? 4 : 2, be = bias_dtype == SWIGLU_F32 ? 4 : 2;
  const Span out = {"y", y, (size_t)M * N * oe};
  const Span in[] = {{"x", x, (size_t)M * K * 2}, {"w", w, (size_t)K * N * 2},
                     {"bias", bias, bias ? (size_t)N * be : 0, (unsigned)be},
                     {"residual", residual, residual ? out.bytes : 0},
                     {"workspace", workspace, workspace ? workspace_bytes : 0}};
  if ((v = check_spans(&out, 1)) != SWIGLU_OK || (v = check_spans(in, 4)) != SWIGLU_OK) return v;
  if ((v = check_apart(out, in, 3)) != SWIGLU_OK) return v;
  if (residual != y && (v = check_apart(out, in + 3, 1)) != SWIGLU_OK) return v;
  if ((v = check_apart(out, in + 4, 1)) != SWIGLU_OK) return v;
  Device dv;
  if ((v = get_device(&dv)) != SWIGLU_OK) return v;
  if (M == 0 || N == 0) {
    api_clear_error();
    return SWIGLU_OK;
  }
  const GroupedPlan p = plan_grouped(M, M, 1, false, dv.pairs, read_tuning());
  GroupedCall c{};
  c.x = x;
  c.wa = w;
  c.out = y;
  c.out_f32 = out_dtype == SWIGLU_F32;
  c.bias = bias;
  c.bias_f32 = bias_dtype == SWIGLU_F32;
  c.act = activation;
  c.resid = residual;
  c.rows = c.tokens = M;
  c.E = 1;
  c.top_k = 1;
  c.K = K;
  c.n_out = N;
  c.wlayout = wlayout_of(layout);
  const cudaStream_t st = (cudaStream_t)stream;
  const std::unique_lock<std::mutex> lock = lock_calls(dv, st, workspace);
  Workspace ws;
  if ((v = run_grouped(kGroupedLinear, c, p, dv, workspace, workspace_bytes,
                       layout == SWIGLU_WEIGHTS_KN && K > 0 ? padded_bytes(K, N) : 0, &ws, st)) != SWIGLU_OK)
    return v;
  if ((v = free_workspace(ws, st)) != SWIGLU_OK) return v;
  api_clear_error();
  return SWIGLU_OK;
}

// The sort's scratch.
static int sort_workspace(const Device& dv, size_t scratch, Workspace* ws, SortCall* s,
                          cudaStream_t st) {
  if (!scratch) return SWIGLU_OK;
  int v = api_take_workspace(dv.dev, st, nullptr, 0, 0, round256(scratch), ws);
  if (v == SWIGLU_OK) s->scratch = (int*)ws->body;
  return v;
}

int swiglu_dispatch(const int32_t* ids, int32_t* offsets, int32_t* order, int32_t* position,
                    int64_t T, int64_t k, int64_t E, void* stream) {
  int v = check_routing(T, k, E);
  if (v != SWIGLU_OK) return v;
  const size_t n = (size_t)T * k * 4;
  const Span in[] = {{"ids", ids, n, 4}};
  const Span out[] = {{"offsets", offsets, (size_t)(E + 1) * 4, 4}, {"order", order, n, 4},
                      {"position", position, n, 4}};
  if ((v = check_spans(in, 1)) != SWIGLU_OK || (v = check_spans(out, 3)) != SWIGLU_OK) return v;
  for (int i = 0; i < 3; ++i) {
    if ((v = check_apart(out[i], in, 1)) != SWIGLU_OK) return v;
    if ((v = check_apart(out[i], out, i)) != SWIGLU_OK) return v;
  }
  Device dv;
  if ((v = get_device(&dv)) != SWIGLU_OK) return v;
  const cudaStream_t st = (cudaStream_t)stream;
  const std::unique_lock<std::mutex> lock = lock_calls(dv, st, nullptr);
  Workspace ws;
  SortCall sort{offsets, order, position, nullptr};
  if ((v = sort_workspace(dv, dispatch_scratch_bytes(T * k, E, dv.num_sms), &ws, &sort, st)) != SWIGLU_OK) return v;
  const cudaError_t e = launch_dispatch(ids, sort, T * k, E, dv.num_sms, st);
  v = free_workspace(ws, st);
  if (e != cudaSuccess) return api_cuda_fail(e, "kernel launch");
  if (v != SWIGLU_OK) return v;
  api_clear_error();
  return SWIGLU_OK;
}

int swiglu_route(const void* logits, const float* bias, int32_t* ids, float* weights,
                 int32_t* offsets, int32_t* order, int32_t* position, int64_t T, int64_t E,
                 int64_t k, int logits_dtype, int score, int64_t groups, int64_t topk_groups,
                 int group_score, int renormalize, float scale, void* stream) {
  int v = check_routing(T, k, E);
  if (v != SWIGLU_OK) return v;
  if (logits_dtype != SWIGLU_F32 && logits_dtype != SWIGLU_BF16)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown dtype");
  if (score != SWIGLU_SCORE_SOFTMAX && score != SWIGLU_SCORE_SIGMOID)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown score");
  if (group_score != SWIGLU_GROUP_MAX && group_score != SWIGLU_GROUP_TOP2)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown group score");
  if (groups < 1 || E % groups != 0)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "the experts do not divide into the groups");
  if (groups > kMaxGroups) return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 32 groups");
  if (topk_groups < 1 || topk_groups > groups)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "topk_groups must be 1 ... groups");
  const bool sort = offsets || order || position;
  const size_t n = (size_t)T * k * 4;
  const Span in[] = {{"logits", logits, (size_t)T * E * (logits_dtype == SWIGLU_F32 ? 4 : 2),
                      logits_dtype == SWIGLU_F32 ? 4u : 2u},
                     {"bias", bias, bias ? (size_t)E * 4 : 0, 4}};
  const Span out[] = {{"ids", ids, n, 4}, {"weights", weights, n, 4},
                      {"offsets", offsets, sort ? (size_t)(E + 1) * 4 : 0, 4},
                      {"order", order, sort ? n : 0, 4}, {"position", position, sort ? n : 0, 4}};
  if ((v = check_spans(in, 2)) != SWIGLU_OK || (v = check_spans(out, 5)) != SWIGLU_OK) return v;
  for (int i = 0; i < 5; ++i) {
    if ((v = check_apart(out[i], in, 2)) != SWIGLU_OK) return v;
    if ((v = check_apart(out[i], out, i)) != SWIGLU_OK) return v;
  }
  Device dv;
  if ((v = get_device(&dv)) != SWIGLU_OK) return v;
  const cudaStream_t st = (cudaStream_t)stream;
  if (!sort && (T == 0 || k == 0)) {
    api_clear_error();
    return SWIGLU_OK;
  }
  const RouteCall c{logits, logits_dtype == SWIGLU_F32, bias, ids, weights, T, E, k,
                    score == SWIGLU_SCORE_SIGMOID, (int)groups, (int)topk_groups,
                    group_score == SWIGLU_GROUP_TOP2, renormalize != 0, scale};
  const std::unique_lock<std::mutex> lock = lock_calls(dv, st, nullptr);
  Workspace ws;
  SortCall sc{offsets, order, position, nullptr};
  if (sort && (v = sort_workspace(dv, route_scratch_bytes(T, E, dv.num_sms), &ws, &sc, st)) != SWIGLU_OK) return v;
  const cudaError_t e = launch_route(c, sort ? &sc : nullptr, dv.num_sms, st);
  v = free_workspace(ws, st);
  if (e != cudaSuccess) return api_cuda_fail(e, "kernel launch");
  if (v != SWIGLU_OK) return v;
  api_clear_error();
  return SWIGLU_OK;
}

static size_t experts_workspace(int64_t T, int64_t k, int64_t E, int64_t K, int64_t N, bool up) {
  if (check_product(0, K, N, "d", "d_ff") != SWIGLU_OK || check_routing(T, k, E) != SWIGLU_OK) return 0;
  Device dv;
  if (get_device(&dv) != SWIGLU_OK) return 0;
  const GroupedPlan p = plan_experts(T, k, E, up, dv.pairs);
  api_clear_error();
  return p.counters_bytes + part_region(p) + (up ? 0 : z_bytes(T * k, N));
}

size_t swiglu_experts_up_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t d, int64_t d_ff) {
  return experts_workspace(T, k, E, d, d_ff, true);
}

size_t swiglu_experts_down_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t d_ff, int64_t d) {
  return experts_workspace(T, k, E, d_ff, d, false);
}

int swiglu_experts_up(const void* x, const void* w_gate, const void* w_up, const int32_t* offsets,
                      const int32_t* order, void* h, int64_t T, int64_t k, int64_t E, int64_t d,
                      int64_t d_ff, int layout, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int v = check_routing(T, k, E);
  if (v != SWIGLU_OK) return v;
  const int64_t rows = T * k;
  if ((v = check_product(rows, d, d_ff, "d", "d_ff")) != SWIGLU_OK) return v;
  if ((v = check_layout(layout)) != SWIGLU_OK) return v;
  const size_t nw = (size_t)E * d * d_ff * 2;
  const Span out = {"h", h, (size_t)rows * d_ff * 2};
  const Span in[] = {{"x", x, (size_t)T * d * 2}, {"w_gate", w_gate, nw}, {"w_up", w_up, nw},
                     {"offsets", offsets, (size_t)(E + 1) * 4, 4}, {"order", order, (size_t)rows * 4, 4},
                     {"workspace", workspace, workspace ? workspace_bytes : 0}};
  if ((v = check_spans(&out, 1)) != SWIGLU_OK || (v = check_spans(in, 5)) != SWIGLU_OK) return v;
  if ((v = check_apart(out, in, 6)) != SWIGLU_OK) return v;
  Device dv;
  if ((v = get_device(&dv)) != SWIGLU_OK) return v;
  if (rows == 0 || d_ff == 0) {
    api_clear_error();
    return SWIGLU_OK;
  }
  GroupedCall c{};
  c.x = x;
  c.wa = w_gate;
  c.wb = w_up;
  c.offsets = offsets;
  c.order = order;
  c.out = h;
  c.rows = rows;
  c.tokens = T;
  c.E = E;
  c.top_k = k;
  c.K = d;
  c.n_out = d_ff;
  c.wlayout = wlayout_of(layout);
  const cudaStream_t st = (cudaStream_t)stream;
  const std::unique_lock<std::mutex> lock = lock_calls(dv, st, workspace);
  Workspace ws;
  if ((v = run_grouped(kGroupedSwiGLU, c, plan_experts(T, k, E, true, dv.pairs), dv, workspace,
                       workspace_bytes, 0, &ws, st)) != SWIGLU_OK)
    return v;
  if ((v = free_workspace(ws, st)) != SWIGLU_OK) return v;
  api_clear_error();
  return SWIGLU_OK;
}

int swiglu_experts_down(const void* h, const void* w_down, const int32_t* offsets,
                        const int32_t* position, const float* weights, const void* residual,
                        void* y, int64_t T, int64_t k, int64_t E, int64_t d_ff, int64_t d,
                        int layout, void* workspace, size_t workspace_bytes, void* stream) {
  int v = check_routing(T, k, E);
  if (v != SWIGLU_OK) return v;
  const int64_t rows = T * k;
  if ((v = check_product(rows, d_ff, d, "d_ff", "d")) != SWIGLU_OK) return v;
  if ((v = check_layout(layout)) != SWIGLU_OK) return v;
  const Span out = {"y", y, (size_t)T * d * 2};
  const Span in[] = {{"h", h, (size_t)rows * d_ff * 2}, {"w_down", w_down, (size_t)E * d * d_ff * 2},
                     {"offsets", offsets, (size_t)(E + 1) * 4, 4},
                     {"position", position, (size_t)rows * 4, 4}, {"weights", weights, (size_t)rows * 4, 4},
                     {"residual", residual, residual ? out.bytes : 0},
                     {"workspace", workspace, workspace ? workspace_bytes : 0}};
  if ((v = check_spans(&out, 1)) != SWIGLU_OK || (v = check_spans(in, 6)) != SWIGLU_OK) return v;
  if ((v = check_apart(out, in, 5)) != SWIGLU_OK) return v;
  if (residual != y && (v = check_apart(out, in + 5, 1)) != SWIGLU_OK) return v;
  if ((v = check_apart(out, in + 6, 1)) != SWIGLU_OK) return v;
  Device dv;
  if ((v = get_device(&dv)) != SWIGLU_OK) return v;
  if (T == 0 || d == 0) {
    api_clear_error();
    return SWIGLU_OK;
  }
  const cudaStream_t st = (cudaStream_t)stream;
  const std::unique_lock<std::mutex> lock = lock_calls(dv, st, workspace);
  Workspace ws;
  const float* z = nullptr;
  Work work{};
  if (rows > 0 && d_ff > 0) {
    GroupedCall c{};
    c.x = h;
    c.wa = w_down;
    c.offsets = offsets;
    c.out_f32 = 1;
    c.rows = rows;
    c.tokens = T;
    c.E = E;
    c.top_k = k;
    c.K = d_ff;
    c.n_out = d;
    c.wlayout = wlayout_of(layout);
    const GroupedPlan p = plan_experts(T, k, E, false, dv.pairs);
    if ((v = run_grouped(kGroupedPlain, c, p, dv, workspace, workspace_bytes, z_bytes(rows, d), &ws,
                         st)) != SWIGLU_OK)
      return v;
    z = (const float*)(ws.body + part_region(p));
    fill_work(&work, kGroupedPlain, c, p, (float*)ws.body);
  }
  // (a product over nothing: y = residual, or 0)
  const cudaError_t e = launch_combine(z, &work, position, weights, residual, y, T,
                                       z ? k : 0, rows, d, dv.num_sms, st);
  v = free_workspace(ws, st);
  if (e != cudaSuccess) return api_cuda_fail(e, "kernel launch");
  if (v != SWIGLU_OK) return v;
  api_clear_error();
  return SWIGLU_OK;
}

}  // extern "C"
