// C ABI of libmoeq.so: argument validation, workspace layout and launches.
// Every exported function is declared, with its contract, in include/moeq.h.
#include "common.cuh"
#include "grouped.cuh"
#include "lora.cuh"
#include "mx.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <stdarg.h>
#include <stdio.h>
#include <vector>

#define MQ_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

// ---------------------------------------------------------------------------
// Launch accounting and optional per-kernel CUDA-event timing.
// ---------------------------------------------------------------------------
std::atomic<long long> g_launches{0};
std::atomic<int> g_prof_on{0};
std::mutex g_prof_mu;
struct ProfRec {
  int slot;
  cudaEvent_t a, b;
};
std::vector<ProfRec> g_prof_pending;
std::vector<cudaEvent_t> g_event_pool;
double g_prof_ms[MQ_PROF_SLOTS];
long long g_prof_n[MQ_PROF_SLOTS];

cudaEvent_t pool_event() {
  std::lock_guard<std::mutex> lock(g_prof_mu);
  if (!g_event_pool.empty()) {
    cudaEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// Counts one kernel launch and, while profiling is on, brackets it with a
// pair of events on its stream.
struct LaunchScope {
  int slot;
  cudaStream_t st;
  cudaEvent_t a = nullptr;
  LaunchScope(int s, cudaStream_t stream) : slot(s), st(stream) {
    g_launches.fetch_add(1, std::memory_order_relaxed);
    if (g_prof_on.load(std::memory_order_relaxed)) {
      a = pool_event();
      if (a) cudaEventRecord(a, st);
    }
  }
  ~LaunchScope() {
    if (!a) return;
    cudaEvent_t b = pool_event();
    if (!b) return;
    cudaEventRecord(b, st);
    std::lock_guard<std::mutex> lock(g_prof_mu);
    g_prof_pending.push_back({slot, a, b});
  }
};

thread_local char g_msg[512] = "";

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

int cuda_fail(cudaError_t err, const char* what) {
  return fail(MQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device status word (one per device, in this library's module).
__device__ unsigned g_dev_status;

constexpr int kMaxDevices = 64;
unsigned* g_status_ptr[kMaxDevices];
std::mutex g_status_mu;

unsigned* status_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_status_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_dev_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<unsigned*>(p);
  }
  return g_status_ptr[dev];
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace layout of moe_quant_forward: align arrays (16-slot blocks) and
// the chunk table of the GEMMs' token tiles, gathered activations (f16) and
// their row scales, act (bf16, then f16 in place) and its row scales,
// split-K partial outputs (fp32).
constexpr int kAlignBlock = 16;

// Which consumers the expert GEMMs run.  With a few token-slots per expert
// the converter warps can multiply with warp-level MMAs themselves
// (TcPlan::sync1 / sync2; token tiles of 16 or 32 rows) instead of feeding
// the tcgen05.mma issuers.  That mode was the faster gate/up GEMM for 8-bit
// batches of up to 32 tokens while each converter group had one
// tensor-memory stage (Mixtral-shaped T=8: 150 vs 163 us per launch).  With
// three stages shared by two issuers, tcgen05 is faster at every size
// measured (Mixtral-shaped gate/up T=1: 56.4 vs 57.8 us, T=8: 148.6 vs
// 158.3, T=32: 161.7 vs 174.0; fine-grained T=8: 25.1 vs 26.0), so the
// default takes tcgen05 and the warp-MMA mode runs when forced
// (MQ_FWD_PATH_DECODE).  Each mma.sync takes about 8 cycles of its
// scheduler's issue that dequant instructions cannot overlap.

// The one-launch layer by default where it measured faster than two
// launches (fine-grained E=128, k=8, H=2048, I=768 with Zipf routing, step
// with the L2 flushed: T=128 83.0 -> 77.2 us, T=512 132.4 -> 124.1 us): layers
// of many small experts with 128-row token tiles, where each GEMM alone runs
// few MMA steps per SM.  At T=64 (64-row tiles) both take 59-60 us, at
// T=4096 both 574 us; Mixtral-shaped layers (E=8) lose with it (T=64: 291 ->
// 305 us, as 64-row tiles replace the 32-row ones).  For one or two tokens
// in layers of a few experts the down GEMM's start-up hides behind the
// gate/up GEMM's tail: Mixtral-shaped T=1 step 79.6 -> 76.5 us (L2 flushed:
// 90.7 -> 85.3), T=2 80.1 -> 77.7 us; from T=4 on two launches are as fast
// or faster.
bool layer_default(int T, int E) { return E > 16 ? (T > 64 && T <= 2048) : T <= 2; }

TcPlan fwd_plan(int T, int H, int I, int E, int k, int bits, int group_size, unsigned flags) {
  TcPlan pl = tc_plan(T, H, I, E, k, bits);
  const bool ok = dec_supported(bits, group_size, H, I);
  if (flags & MQ_FWD_PATH_TENSOR_CORE) return pl;
  if (flags & MQ_FWD_PATH_LAYER) {  // 8-bit only (checked by the caller)
    pl.layer = true;
    return pl;
  }
  if (flags & MQ_FWD_PATH_DECODE) {
    if (!ok) return pl;
    pl.sync1 = pl.sync2 = true;
    // an expert receives at most one slot per token: up to 16 tokens every
    // expert fits one 16-row tile (uint4 keeps 16-row tiles: their register
    // budget holds two 8-token MMA groups)
    pl.bn = (bits == 8 && T > 16) ? 32 : 16;
    // the workspace holds the warp-MMA splits for batches where that mode is
    // the default's size class, else the tcgen05 plan's
    if (T <= 64) pl.splits = dec_splits(T, H, I, E, k, bits);
    return pl;
  }
  // default: tcgen05 for both GEMMs; one launch for both GEMMs of 8-bit
  // layers of many experts (measured rule above)
  (void)ok;
  if (bits == 8 && layer_default(T, E)) pl.layer = true;
  // 8-bit down GEMM on f16 operands after the in-place act -> f16 pass, for
  // layers of a few experts at 8-64 tokens: the f16 conversion of the codes
  // takes about half the instructions of bf16, which outweighs the pass
  // (Mixtral-shaped step T=64 248.3 -> 240.7 us, T=8 218.7 -> 213.1 us; T=1
  // 79.5 -> 81.9, fine-grained T=64 51.9 -> 57.4, prefill T=4096 2456 ->
  // 2556 us, where the pass costs more than it saves)
  if (bits == 8 && !pl.layer && E <= 16 && T >= 8 && T <= 64) pl.f16down = true;
  return pl;
}

struct WsLayout {
  size_t sorted, block_expert, offsets, num_padded, chunk_expert, chunk_start, counts, dep, xs,
      xinv, act, act_inv, y, topk_w, topk_ids, total;
  int64_t cap;
  TcPlan plan;
};

// with_route: the forward routes itself (router logits in), holding topk_w
// and topk_ids in the workspace too.
WsLayout ws_layout(int T, int H, int I, int E, int k, int bits, int group_size,
                   bool with_route = false) {
  WsLayout L;
  L.plan = tc_plan(T, H, I, E, k, bits);
  // partial outputs for every consumer choice (the warp-MMA plan's splits
  // and the tcgen05 plan's), so that a forced choice fits the same workspace
  const TcPlan fp = fwd_plan(T, H, I, E, k, bits, group_size, MQ_FWD_PATH_DECODE);
  const int ysplits = L.plan.splits > fp.splits ? L.plan.splits : fp.splits;
  const int bm = kAlignBlock;
  const int64_t S = (int64_t)T * k;
  const int64_t cap = moe_align_capacity(T, k, E, bm);
  L.cap = cap;
  size_t off = 0;
  L.sorted = off;       off += align256(sizeof(int32_t) * (size_t)cap);
  L.block_expert = off; off += align256(sizeof(int32_t) * (size_t)(cap / bm));
  L.offsets = off;      off += align256(sizeof(int32_t) * (size_t)(E + 1));
  L.num_padded = off;   off += align256(sizeof(int32_t));
  L.chunk_expert = off; off += align256(sizeof(int32_t) * (size_t)(cap / bm));
  L.chunk_start = off;  off += align256(sizeof(int32_t) * (size_t)(E + 1));
  L.counts = off;       off += align256(sizeof(int32_t) * (size_t)E);
  L.dep = off;          off += align256(sizeof(int32_t) * (size_t)(cap / bm));
  L.xs = off;           off += align256(sizeof(__half) * (size_t)cap * (size_t)H);
  L.xinv = off;         off += align256(sizeof(float) * (size_t)cap);
  L.act = off;          off += align256(sizeof(__nv_bfloat16) * (size_t)cap * (size_t)I);
  L.act_inv = off;      off += align256(sizeof(float) * (size_t)cap);
  L.y = off;            off += align256(sizeof(float) * (size_t)ysplits * (size_t)S * (size_t)H);
  L.topk_w = off;       if (with_route) off += align256(sizeof(float) * (size_t)S);
  L.topk_ids = off;     if (with_route) off += align256(sizeof(int32_t) * (size_t)S);
  L.total = off;
  return L;
}

bool fmt_ok(int bits, int group_size, int has_zp) {
  if (bits == 8) return group_size == -1 && has_zp == 0;
  if (bits == 4)
    return (group_size == 32 || group_size == 64 || group_size == 128 || group_size == 256) &&
           (has_zp == 0 || has_zp == 1);
  return false;
}

}  // namespace

int mq_set_error(int status, const char* msg) { return fail(status, "%s", msg); }

MQ_EXPORT const char* mq_status_string(int status) {
  switch (status) {
    case MQ_OK: return "ok";
    case MQ_ERR_INVALID_ARG: return "invalid argument";
    case MQ_ERR_UNSUPPORTED: return "unsupported";
    case MQ_ERR_CUDA: return "CUDA error";
    case MQ_ERR_WORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

MQ_EXPORT const char* mq_last_error_message(void) { return g_msg; }

MQ_EXPORT long long mq_kernel_launch_count(void) { return g_launches.load(); }

MQ_EXPORT int mq_test_layer_wait_extra(int extra) {
  if (extra < 0) return fail(MQ_ERR_INVALID_ARG, "extra must be >= 0");
  set_layer_wait_extra(extra);
  return MQ_OK;
}

MQ_EXPORT int mq_profile_enable(int on) {
  g_prof_on.store(on ? 1 : 0);
  return MQ_OK;
}

MQ_EXPORT int mq_profile_read(double* total_ms, long long* launches, int n_slots) {
  if (!total_ms || !launches || n_slots < 1) return fail(MQ_ERR_INVALID_ARG, "bad profile buffers");
  std::vector<ProfRec> recs;
  {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    recs.swap(g_prof_pending);
  }
  int status = MQ_OK;
  for (const ProfRec& r : recs) {
    float ms = 0.0f;
    cudaError_t err = cudaEventSynchronize(r.b);
    if (err == cudaSuccess) err = cudaEventElapsedTime(&ms, r.a, r.b);
    if (err != cudaSuccess) status = cuda_fail(err, "mq_profile_read");
    g_prof_ms[r.slot] += ms;
    g_prof_n[r.slot] += 1;
  }
  std::lock_guard<std::mutex> lock(g_prof_mu);
  for (const ProfRec& r : recs) {
    g_event_pool.push_back(r.a);
    g_event_pool.push_back(r.b);
  }
  for (int i = 0; i < n_slots; ++i) {
    total_ms[i] = i < MQ_PROF_SLOTS ? g_prof_ms[i] : 0.0;
    launches[i] = i < MQ_PROF_SLOTS ? g_prof_n[i] : 0;
  }
  for (int i = 0; i < MQ_PROF_SLOTS; ++i) {
    g_prof_ms[i] = 0.0;
    g_prof_n[i] = 0;
  }
  return status;
}

MQ_EXPORT int mq_device_status(void* stream, uint32_t* flags) {
  if (!flags) return fail(MQ_ERR_INVALID_ARG, "flags is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err = cudaStreamSynchronize(st);
  if (err != cudaSuccess) return cuda_fail(err, "mq_device_status: stream synchronize");
  unsigned v = 0;
  err = cudaMemcpyFromSymbol(&v, g_dev_status, sizeof(v));
  if (err != cudaSuccess) return cuda_fail(err, "mq_device_status: read");
  const unsigned zero = 0;
  err = cudaMemcpyToSymbol(g_dev_status, &zero, sizeof(zero));
  if (err != cudaSuccess) return cuda_fail(err, "mq_device_status: clear");
  *flags = v;
  return MQ_OK;
}

MQ_EXPORT int moe_quantize_int8_per_channel(const void* w, int64_t rows, int64_t cols, int8_t* q,
                                            float* scale, void* stream) {
  if (rows < 0 || cols < 0) return fail(MQ_ERR_INVALID_ARG, "negative size");
  if (cols % 8 || cols > (int64_t(1) << 31) - 8)
    return fail(MQ_ERR_INVALID_ARG, "cols must be a multiple of 8 below 2^31");
  if (rows == 0) return MQ_OK;
  if (cols == 0) return fail(MQ_ERR_INVALID_ARG, "cols must be positive");
  if (!w || !q || !scale) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(w) || !aligned16(q)) return fail(MQ_ERR_INVALID_ARG, "w and q must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_QUANT, st);
  cudaError_t err = launch_quant_int8(w, rows, cols, q, scale, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "quantize_int8 launch");
}

MQ_EXPORT int moe_quantize_uint4_group(const void* w, int64_t rows, int64_t cols, int group_size,
                                       uint8_t* qweight, uint16_t* scales, uint8_t* qzeros,
                                       void* stream) {
  if (rows < 0 || cols <= 0) return fail(MQ_ERR_INVALID_ARG, "bad size");
  if (rows % 2) return fail(MQ_ERR_INVALID_ARG, "rows must be even (zero points pack two rows)");
  if (!(group_size == 32 || group_size == 64 || group_size == 128 || group_size == 256))
    return fail(MQ_ERR_INVALID_ARG, "group_size must be 32, 64, 128 or 256");
  if (cols % group_size) return fail(MQ_ERR_INVALID_ARG, "group_size must divide cols");
  if (cols > (int64_t(1) << 30)) return fail(MQ_ERR_INVALID_ARG, "cols too large");
  if (rows == 0) return MQ_OK;
  if (!w || !qweight || !scales || !qzeros) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(w) || !aligned16(qweight)) return fail(MQ_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_QUANT, st);
  cudaError_t err = launch_quant_uint4(w, rows, cols, group_size, qweight, scales, qzeros, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "quantize_uint4 launch");
}

MQ_EXPORT int moe_topk_route(const float* logits, int T, int E, int k, int renormalize,
                             float* topk_w, int32_t* topk_ids, void* stream) {
  if (T < 0) return fail(MQ_ERR_INVALID_ARG, "T must be >= 0");
  if (E < 1 || E > 1024) return fail(MQ_ERR_UNSUPPORTED, "E must be in [1, 1024]");
  if (k < 1 || k > E || k > 32) return fail(MQ_ERR_INVALID_ARG, "need 1 <= k <= min(E, 32)");
  if (T == 0) return MQ_OK;
  if (!logits || !topk_w || !topk_ids) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_ROUTE, st);
  cudaError_t err = launch_route(logits, T, E, k, renormalize ? 1 : 0, topk_w, topk_ids, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "route launch");
}

// mq_route_opts -> RouteOpts, with the checks moe_topk_route_ex documents.
static int route_opts_from(const mq_route_opts* opts, int E, int k, RouteOpts* o) {
  if (!opts) return fail(MQ_ERR_INVALID_ARG, "null route options");
  if (opts->scoring_func != MQ_SCORING_SOFTMAX && opts->scoring_func != MQ_SCORING_SIGMOID)
    return fail(MQ_ERR_INVALID_ARG, "unknown scoring_func %d", opts->scoring_func);
  const int G = opts->num_expert_group;
  if (G < 0 || G > 32) return fail(MQ_ERR_INVALID_ARG, "num_expert_group must be in [0, 32]");
  if (G > 1) {
    if (E % G) return fail(MQ_ERR_INVALID_ARG, "num_expert_group must divide E");
    if (opts->topk_group < 1 || opts->topk_group > G)
      return fail(MQ_ERR_INVALID_ARG, "topk_group must be in [1, num_expert_group]");
    if ((int64_t)k > (int64_t)opts->topk_group * (E / G))
      return fail(MQ_ERR_INVALID_ARG, "k exceeds the experts of topk_group groups");
  }
  if (!std::isfinite(opts->routed_scaling_factor))
    return fail(MQ_ERR_INVALID_ARG, "routed_scaling_factor must be finite");
  if (opts->e_score_correction_bias && !aligned16(opts->e_score_correction_bias))
    return fail(MQ_ERR_INVALID_ARG, "e_score_correction_bias must be 16-byte aligned");
  o->scoring = opts->scoring_func;
  o->renorm = opts->renormalize ? 1 : 0;
  o->groups = G > 1 ? G : 0;
  o->topk_group = G > 1 ? opts->topk_group : 0;
  o->bias = opts->e_score_correction_bias;
  o->scale = opts->routed_scaling_factor;
  return MQ_OK;
}

MQ_EXPORT int moe_topk_route_ex(const float* logits, int T, int E, int k,
                                const mq_route_opts* opts, float* topk_w, int32_t* topk_ids,
                                void* stream) {
  if (T < 0) return fail(MQ_ERR_INVALID_ARG, "T must be >= 0");
  if (E < 1 || E > 1024) return fail(MQ_ERR_UNSUPPORTED, "E must be in [1, 1024]");
  if (k < 1 || k > E || k > 32) return fail(MQ_ERR_INVALID_ARG, "need 1 <= k <= min(E, 32)");
  RouteOpts o;
  const int rc = route_opts_from(opts, E, k, &o);
  if (rc != MQ_OK) return rc;
  if (T == 0) return MQ_OK;
  if (!logits || !topk_w || !topk_ids) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_ROUTE, st);
  cudaError_t err = launch_route_ex(logits, T, E, k, o, topk_w, topk_ids, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "route launch");
}

MQ_EXPORT int64_t moe_align_capacity(int T, int k, int E, int block_m) {
  if (T < 0 || k < 1 || E < 1 || block_m < 1) return -1;
  const int64_t S = (int64_t)T * k;
  const int64_t cap = S + (int64_t)(E < S ? E : S) * (block_m - 1);
  return (cap + block_m - 1) / block_m * block_m;
}

MQ_EXPORT int moe_align_block(const int32_t* topk_ids, int T, int k, int E, int block_m,
                              int32_t* sorted_slot_ids, int32_t* block_expert,
                              int32_t* expert_offsets, int32_t* num_padded, int64_t capacity,
                              void* stream) {
  if (T < 0 || k < 1 || E < 1) return fail(MQ_ERR_INVALID_ARG, "bad T, k or E");
  if (E > 1024) return fail(MQ_ERR_UNSUPPORTED, "E must be <= 1024");
  if (block_m < 1 || block_m > 1024) return fail(MQ_ERR_INVALID_ARG, "block_m must be in [1, 1024]");
  if ((int64_t)T * k > (int64_t(1) << 30)) return fail(MQ_ERR_UNSUPPORTED, "too many slots");
  if (capacity < moe_align_capacity(T, k, E, block_m))
    return fail(MQ_ERR_INVALID_ARG, "capacity below moe_align_capacity()");
  if ((T > 0 && !topk_ids) || !sorted_slot_ids || !block_expert || !expert_offsets || !num_padded)
    return fail(MQ_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned* status = status_ptr();
  LaunchScope ls(MQ_PROF_ALIGN, st);
  cudaError_t err = launch_align(topk_ids, T, k, E, block_m, sorted_slot_ids, block_expert,
                                 expert_offsets, num_padded, status, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "align launch");
}

MQ_EXPORT size_t moe_quant_forward_workspace(int T, int H, int I, int E, int k, int bits,
                                             int group_size) {
  if (T < 0 || H <= 0 || I <= 0 || E < 1 || k < 1 || k > E) return 0;
  if (!fmt_ok(bits, group_size, 0)) return 0;
  return ws_layout(T, H, I, E, k, bits, group_size).total;
}

MQ_EXPORT int moe_quant_forward_ex(const void* x, int T, int H, int I, int E, int k, int bits,
                                   int group_size, int has_zp, const void* w13, const void* w2,
                                   const void* s13, const void* s2, const uint8_t* z13,
                                   const uint8_t* z2, const float* topk_w,
                                   const int32_t* topk_ids, void* workspace, size_t ws_bytes,
                                   void* out, unsigned flags, void* stream);

MQ_EXPORT int moe_quant_forward(const void* x, int T, int H, int I, int E, int k, int bits,
                                int group_size, int has_zp, const void* w13, const void* w2,
                                const void* s13, const void* s2, const uint8_t* z13,
                                const uint8_t* z2, const float* topk_w, const int32_t* topk_ids,
                                void* workspace, size_t ws_bytes, void* out, void* stream) {
  return moe_quant_forward_ex(x, T, H, I, E, k, bits, group_size, has_zp, w13, w2, s13, s2, z13,
                              z2, topk_w, topk_ids, workspace, ws_bytes, out, 0u, stream);
}

// The forward.  With logits (router logits [T, E]) it routes itself, into
// the workspace; otherwise topk_w / topk_ids are the caller's.
static int forward_impl(const void* x, int T, int H, int I, int E, int k, int bits,
                        int group_size, int has_zp, const void* w13, const void* w2,
                        const void* s13, const void* s2, const uint8_t* z13, const uint8_t* z2,
                        const float* topk_w, const int32_t* topk_ids, const float* logits,
                        const RouteOpts& ro, void* workspace, size_t ws_bytes, void* out,
                        unsigned flags, void* stream) {
  constexpr unsigned kW8Flags = MQ_FWD_W8_UINT8 | MQ_FWD_SCALE_F16 | MQ_FWD_SCALE_BF16 |
                                MQ_FWD_SCALE_PER_TENSOR;
  constexpr unsigned kAllFlags = kW8Flags | MQ_FWD_ACT_F16 | MQ_FWD_ROUTER_WEIGHT_ON_INPUT |
                                 MQ_FWD_PATH_TENSOR_CORE | MQ_FWD_PATH_DECODE |
                                 MQ_FWD_PATH_LAYER;
  if (T < 0 || H <= 0 || I <= 0 || E < 1) return fail(MQ_ERR_INVALID_ARG, "bad T, H, I or E");
  if (k < 1 || k > E || k > 32) return fail(MQ_ERR_INVALID_ARG, "need 1 <= k <= min(E, 32)");
  if (E > 1024) return fail(MQ_ERR_UNSUPPORTED, "E must be <= 1024");
  if (flags & ~kAllFlags) return fail(MQ_ERR_UNSUPPORTED, "unknown flags 0x%x", flags & ~kAllFlags);
  if (bits == 4 && (flags & kW8Flags))
    return fail(MQ_ERR_UNSUPPORTED, "uint8 codes and scale options apply to bits = 8 only");
  if ((flags & MQ_FWD_SCALE_F16) && (flags & MQ_FWD_SCALE_BF16))
    return fail(MQ_ERR_UNSUPPORTED, "scales are float16 or bfloat16, not both");
  {
    const unsigned paths = flags & (MQ_FWD_PATH_TENSOR_CORE | MQ_FWD_PATH_DECODE | MQ_FWD_PATH_LAYER);
    if (paths & (paths - 1))
      return fail(MQ_ERR_INVALID_ARG, "at most one of the MQ_FWD_PATH_* flags");
  }
  if ((flags & MQ_FWD_PATH_LAYER) && bits != 8)
    return fail(MQ_ERR_UNSUPPORTED, "the one-launch layer takes 8-bit codes");
  if ((flags & MQ_FWD_PATH_DECODE) && !dec_supported(bits, group_size, H, I))
    return fail(MQ_ERR_UNSUPPORTED, "the warp-MMA consumers take 8-bit codes or uint4 with group_size 128 or 256");
  const bool w8zp = bits == 8 && group_size == -1 && has_zp == 1 && (flags & MQ_FWD_W8_UINT8);
  if (!fmt_ok(bits, group_size, has_zp) && !w8zp)
    return fail(MQ_ERR_UNSUPPORTED,
                "format must be (8, -1, 0), (8, -1, 1) with uint8 codes, or (4, 32..256, 0|1)");
  if (H % 128 || I % 128) return fail(MQ_ERR_UNSUPPORTED, "H and I must be multiples of 128");
  if (bits == 4 && (H % group_size || I % group_size))
    return fail(MQ_ERR_UNSUPPORTED, "group_size must divide H and I");
  if ((int64_t)T * k > (int64_t(1) << 24)) return fail(MQ_ERR_UNSUPPORTED, "too many token-slots");
  if (T == 0) return MQ_OK;
  if (!x || !w13 || !w2 || !s13 || !s2 || !out || !workspace ||
      (logits ? false : (!topk_w || !topk_ids)))
    return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (has_zp && (!z13 || !z2)) return fail(MQ_ERR_INVALID_ARG, "null zero points");
  if (!has_zp && (z13 || z2)) return fail(MQ_ERR_INVALID_ARG, "zero points given with has_zp = 0");
  if (!aligned16(x) || !aligned16(w13) || !aligned16(w2) || !aligned16(out) || !aligned16(workspace))
    return fail(MQ_ERR_INVALID_ARG, "x, w13, w2, out and workspace must be 16-byte aligned");
  if (!aligned16(s13) || !aligned16(s2) || (z13 && !aligned16(z13)) || (z2 && !aligned16(z2)))
    return fail(MQ_ERR_INVALID_ARG, "scales and zero points must be 16-byte aligned");
  {
    const char* xb = static_cast<const char*>(x);
    const char* ob = static_cast<const char*>(out);
    const size_t nb = (size_t)T * H * 2;
    // out == x is fused_experts' inplace: x is read (gathered) before any
    // output is written
    if (ob != xb && ob < xb + nb && xb < ob + nb)
      return fail(MQ_ERR_INVALID_ARG, "out overlaps x (only out == x is allowed)");
  }
  const WsLayout L = ws_layout(T, H, I, E, k, bits, group_size, logits != nullptr);
  const TcPlan plan = fwd_plan(T, H, I, E, k, bits, group_size, flags);
  const int bm = kAlignBlock;
  if (ws_bytes < L.total)
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, L.total);

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float* rw = logits ? reinterpret_cast<float*>(ws + L.topk_w) : nullptr;
  int32_t* rid = logits ? reinterpret_cast<int32_t*>(ws + L.topk_ids) : nullptr;
  if (logits) {
    topk_w = rw;
    topk_ids = rid;
  }
  MoeArgs a;
  a.x = x;
  a.flags = flags;
  a.T = T; a.H = H; a.I = I; a.E = E; a.k = k;
  a.bits = bits; a.group_size = group_size; a.has_zp = has_zp;
  a.w13 = w13; a.w2 = w2; a.s13 = s13; a.s2 = s2; a.z13 = z13; a.z2 = z2;
  a.topk_w = topk_w; a.topk_ids = topk_ids;
  a.out = out;
  a.status = status_ptr();
  a.sorted = reinterpret_cast<int32_t*>(ws + L.sorted);
  a.block_expert = reinterpret_cast<int32_t*>(ws + L.block_expert);
  a.offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  a.num_padded = reinterpret_cast<int32_t*>(ws + L.num_padded);
  a.chunk_expert = reinterpret_cast<int32_t*>(ws + L.chunk_expert);
  a.chunk_start = reinterpret_cast<int32_t*>(ws + L.chunk_start);
  a.counts = reinterpret_cast<int32_t*>(ws + L.counts);
  a.dep = reinterpret_cast<int32_t*>(ws + L.dep);
  a.act = reinterpret_cast<__nv_bfloat16*>(ws + L.act);
  a.y = reinterpret_cast<float*>(ws + L.y);
  a.bm = bm;
  a.cap = L.cap;

  cudaError_t err;
  // the plain softmax router of small batches runs inside the align kernel
  const bool plain = route_opts_plain(ro);
  const bool fused = logits && plain && route_fused(T, k, E);
  if (logits && !fused) {  // otherwise the router kernel first
    LaunchScope ls(MQ_PROF_ROUTE, st);
    err = plain ? launch_route(logits, T, E, k, ro.renorm, rw, rid, st)
                : launch_route_ex(logits, T, E, k, ro, rw, rid, st);
    if (err != cudaSuccess) return cuda_fail(err, "forward: route launch");
  }
  const int chunk = plan.bn;  // token rows per tile of the chunk table
  {
    LaunchScope ls(MQ_PROF_ALIGN, st);
    if (fused)
      err = launch_route_align(logits, ro.renorm, rw, rid, T, k, E, bm, a.sorted, a.block_expert,
                               a.offsets, a.num_padded, a.status, st, chunk, a.chunk_expert,
                               a.chunk_start, a.counts, plan.layer ? a.dep : nullptr);
    else
      err = launch_align(topk_ids, T, k, E, bm, a.sorted, a.block_expert, a.offsets,
                         a.num_padded, a.status, st, chunk, a.chunk_expert, a.chunk_start,
                         a.counts, plan.layer ? a.dep : nullptr);
  }
  if (err != cudaSuccess) return cuda_fail(err, "forward: align launch");
  void* xs = ws + L.xs;
  float* xinv = reinterpret_cast<float*>(ws + L.xinv);
  {
    LaunchScope ls(MQ_PROF_GATHER, st);
    err = launch_gather_rows(a, xs, xinv, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "forward: gather launch");
  if (plan.layer) {
    {
      LaunchScope ls(MQ_PROF_LAYER, st);
      err = launch_layer_tc(a, plan, xs, xinv, a.y, st);
    }
    if (err != cudaSuccess) return cuda_fail(err, "forward: expert layer launch");
    LaunchScope ls(MQ_PROF_COMBINE, st);
    err = launch_combine_splits(a, a.y, plan.splits, st);
    if (err != cudaSuccess) return cuda_fail(err, "forward: combine launch");
    return MQ_OK;
  }
  {
    LaunchScope ls(MQ_PROF_GEMM1, st);
    err = launch_gemm1_tc(a, plan, xs, xinv, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "forward: gate/up GEMM launch");
  float* act_inv = reinterpret_cast<float*>(ws + L.act_inv);
  if ((bits == 4 && !plan.sync2) || plan.f16down) {
    // the tcgen05 uint4 down GEMM runs f16 operands (and the 8-bit one where
    // the plan says so); otherwise the 8-bit one and the warp-MMA mode read
    // bf16 act
    LaunchScope ls(MQ_PROF_ACTF16, st);
    err = launch_act_to_f16(a, act_inv, st);
    if (err != cudaSuccess) return cuda_fail(err, "forward: act conversion launch");
  }
  {
    LaunchScope ls(MQ_PROF_GEMM2, st);
    err = launch_gemm2_tc(a, plan, act_inv, a.y, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "forward: down GEMM launch");
  {
    LaunchScope ls(MQ_PROF_COMBINE, st);
    err = launch_combine_splits(a, a.y, plan.splits, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "forward: combine launch");
  return MQ_OK;
}

MQ_EXPORT int moe_quant_forward_ex(const void* x, int T, int H, int I, int E, int k, int bits,
                                   int group_size, int has_zp, const void* w13, const void* w2,
                                   const void* s13, const void* s2, const uint8_t* z13,
                                   const uint8_t* z2, const float* topk_w,
                                   const int32_t* topk_ids, void* workspace, size_t ws_bytes,
                                   void* out, unsigned flags, void* stream) {
  const RouteOpts none = {MQ_SCORING_SOFTMAX, 0, 0, 0, nullptr, 1.0f};
  return forward_impl(x, T, H, I, E, k, bits, group_size, has_zp, w13, w2, s13, s2, z13, z2,
                      topk_w, topk_ids, nullptr, none, workspace, ws_bytes, out, flags, stream);
}

MQ_EXPORT size_t moe_quant_forward_logits_workspace(int T, int H, int I, int E, int k, int bits,
                                                    int group_size) {
  if (T < 0 || H <= 0 || I <= 0 || E < 1 || k < 1 || k > E) return 0;
  if (!fmt_ok(bits, group_size, 0)) return 0;
  return ws_layout(T, H, I, E, k, bits, group_size, true).total;
}

MQ_EXPORT int moe_quant_forward_logits(const void* x, const float* router_logits, int T, int H,
                                       int I, int E, int k, int renormalize, int bits,
                                       int group_size, int has_zp, const void* w13,
                                       const void* w2, const void* s13, const void* s2,
                                       const uint8_t* z13, const uint8_t* z2, void* workspace,
                                       size_t ws_bytes, void* out, unsigned flags, void* stream) {
  if (T > 0 && !router_logits) return fail(MQ_ERR_INVALID_ARG, "null router_logits");
  const RouteOpts ro = {MQ_SCORING_SOFTMAX, renormalize ? 1 : 0, 0, 0, nullptr, 1.0f};
  return forward_impl(x, T, H, I, E, k, bits, group_size, has_zp, w13, w2, s13, s2, z13, z2,
                      nullptr, nullptr, router_logits, ro, workspace, ws_bytes, out, flags, stream);
}

MQ_EXPORT int moe_quant_forward_logits_ex(const void* x, const float* router_logits, int T,
                                          int H, int I, int E, int k, const mq_route_opts* opts,
                                          int bits, int group_size, int has_zp, const void* w13,
                                          const void* w2, const void* s13, const void* s2,
                                          const uint8_t* z13, const uint8_t* z2, void* workspace,
                                          size_t ws_bytes, void* out, unsigned flags,
                                          void* stream) {
  if (k < 1 || k > E || k > 32) return fail(MQ_ERR_INVALID_ARG, "need 1 <= k <= min(E, 32)");
  RouteOpts ro;
  const int rc = route_opts_from(opts, E, k, &ro);
  if (rc != MQ_OK) return rc;
  if (T > 0 && !router_logits) return fail(MQ_ERR_INVALID_ARG, "null router_logits");
  return forward_impl(x, T, H, I, E, k, bits, group_size, has_zp, w13, w2, s13, s2, z13, z2,
                      nullptr, nullptr, router_logits, ro, workspace, ws_bytes, out, flags, stream);
}

// ---------------------------------------------------------------------------
// Microscaled formats.
// ---------------------------------------------------------------------------
static bool dtype_ok(int dtype) {
  return dtype == MQ_DTYPE_BF16 || dtype == MQ_DTYPE_F16 || dtype == MQ_DTYPE_F32;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks that the quantiser and its inverse share.
static int mx_args(const void* x, int dtype, int64_t rows, int64_t cols, int bits,
                   const uint8_t* q, const uint8_t* scale) {
  if (!dtype_ok(dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (bits != 4 && bits != 8) return fail(MQ_ERR_INVALID_ARG, "bits must be 4 or 8");
  if (rows < 0) return fail(MQ_ERR_INVALID_ARG, "rows must be >= 0");
  if (cols <= 0 || cols % 32) return fail(MQ_ERR_INVALID_ARG, "cols must be a positive multiple of 32");
  if (rows == 0) return MQ_OK;
  if (cols > (int64_t(1) << 40) / rows) return fail(MQ_ERR_UNSUPPORTED, "too many elements");
  if (!x || !q || !scale) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(q) || !aligned4(scale))
    return fail(MQ_ERR_INVALID_ARG, "x / out and q must be 16-byte aligned, scale 4-byte");
  return MQ_OK;
}

MQ_EXPORT int moe_quantize_mx(const void* x, int dtype, int64_t rows, int64_t cols,
                              int64_t row_stride, int bits, uint8_t* q, uint8_t* scale,
                              void* stream) {
  if (row_stride != cols && cols >= int64_t(1) << 35)  // (the kernel's vectors per row: 32 bits)
    return fail(MQ_ERR_UNSUPPORTED, "rows of 2^35 elements or more must be dense");
  const int rc = mx_args(x, dtype, rows, cols, bits, q, scale);
  if (rc != MQ_OK) return rc;
  if (row_stride < cols || row_stride % 8)
    return fail(MQ_ERR_INVALID_ARG, "row_stride must be a multiple of 8, at least cols");
  if (rows == 0) return MQ_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_QUANT, st);
  const cudaError_t err = launch_quant_mx(x, dtype, rows, cols, row_stride, bits, q, scale, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "quantize_mx launch");
}

MQ_EXPORT int moe_dequantize_mx(const uint8_t* q, const uint8_t* scale, int64_t rows,
                                int64_t cols, int bits, void* out, int dtype, void* stream) {
  const int rc = mx_args(out, dtype, rows, cols, bits, q, scale);
  if (rc != MQ_OK || rows == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_QUANT, st);
  const cudaError_t err = launch_dequant_mx(q, scale, rows * cols, bits, out, dtype, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "dequantize_mx launch");
}

// Whether T dense 16-bit rows at `out` reach into T such rows `stride` elements
// apart at `in`, other than as the very same rows: another CTA may read there
// after the write.
static bool rows_clash(const void* out, const void* in, int T, int H, int64_t stride) {
  if (!out || !in || (out == in && (stride == H || T == 1))) return false;
  const int64_t o = (int64_t)reinterpret_cast<uintptr_t>(out);
  const int64_t i = (int64_t)reinterpret_cast<uintptr_t>(in);
  const int64_t row = 2 * (int64_t)H, step = 2 * stride;
  const int64_t r = o < i + row ? 0 : (o - i - row) / step + 1;  // first row that ends behind out
  return r < T && i + r * step < o + T * row;
}

MQ_EXPORT int moe_rmsnorm_mx(const void* x, const void* residual, const void* weight, int dtype,
                             int weight_f32, int T, int H, int64_t x_stride,
                             int64_t residual_stride, float eps, void* residual_out, void* y_out,
                             int bits, uint8_t* q, uint8_t* scale, void* stream) {
  if (!dtype_ok(dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (dtype == MQ_DTYPE_F32) return fail(MQ_ERR_UNSUPPORTED, "rows must be bfloat16 or float16");
  if (bits != 4 && bits != 8) return fail(MQ_ERR_INVALID_ARG, "bits must be 4 or 8");
  if (T < 0) return fail(MQ_ERR_INVALID_ARG, "T must be >= 0");
  if (H <= 0 || H % 32) return fail(MQ_ERR_INVALID_ARG, "H must be a positive multiple of 32");
  if (H > 32768) return fail(MQ_ERR_UNSUPPORTED, "H must be at most 32768");
  if (!(eps >= 0.0f) || !std::isfinite(eps))
    return fail(MQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (x_stride < H || x_stride % 8 || (residual && (residual_stride < H || residual_stride % 8)))
    return fail(MQ_ERR_INVALID_ARG, "row strides must be multiples of 8, at least H");
  if (T == 0) return MQ_OK;
  if (!x || !weight || !q || !scale) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  for (const void* out : {residual_out, y_out})
    if (rows_clash(out, x, T, H, x_stride) || rows_clash(out, residual, T, H, residual_stride))
      return fail(MQ_ERR_INVALID_ARG,
                  "residual_out and y_out may share memory with x or residual only as the same dense rows");
  if (rows_clash(y_out, residual_out, T, H, H))
    return fail(MQ_ERR_INVALID_ARG, "residual_out and y_out share memory");
  if (!aligned16(x) || (residual && !aligned16(residual)) || !aligned16(weight) ||
      (residual_out && !aligned16(residual_out)) || (y_out && !aligned16(y_out)) ||
      !aligned16(q) || !aligned4(scale))
    return fail(MQ_ERR_INVALID_ARG, "pointers must be 16-byte aligned, scale 4-byte");
  NormArgs a;
  a.x = x; a.residual = residual; a.weight = weight;
  a.dtype = dtype; a.weight_f32 = weight_f32 ? 1 : 0;
  a.T = T; a.H = H;
  a.x_stride = x_stride; a.residual_stride = residual_stride;
  a.eps = eps;
  a.residual_out = residual_out; a.y = y_out;
  a.bits = bits; a.q = q; a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(MQ_PROF_NORM, st);
  const cudaError_t err = launch_rmsnorm_mx(a, st);
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "rmsnorm_mx launch");
}

// The kernels count their units of work (at most 16 K splits of 16 rows by 256
// outputs) in 32 bits.
static bool mx_units_ok(int64_t rows, int64_t N, int E) {
  return (rows / 16 + E) * ((N + 255) / 256) < (int64_t(1) << 27);
}

// Weight rows and k are rounded up to 256 and 512 in 32 bits.
static bool mx_rounds_up(int64_t n) { return n <= INT32_MAX - 511; }

static bool mx_product_sizes_ok(int64_t R, int K, int N, int E) {
  return R >= 0 && K > 0 && N > 0 && E >= 1 && K % 128 == 0 && E <= 1024 &&
         R < (int64_t(1) << 30) && mx_rounds_up(K) && mx_rounds_up(N) && mx_units_ok(R, N, E);
}

MQ_EXPORT size_t moe_mx_product_workspace(int64_t R, int K, int N, int E) {
  if (!mx_product_sizes_ok(R, K, N, E) || R == 0) return 0;
  const int splits = std::max(mx_plan(R, E, K, N, false, 8).splits,
                              mx_plan(R, E, K, N, false, 4).splits);
  return splits > 1 ? align256(sizeof(float) * (size_t)splits * (size_t)R * (size_t)N) : 0;
}

MQ_EXPORT int moe_mx_product(const uint8_t* a, const uint8_t* a_scale, int a_bits, int64_t R,
                             int K, int N, int E, const uint8_t* w, const uint8_t* w_scale,
                             const int32_t* expert_offsets, void* out, int out_dtype,
                             void* workspace, size_t ws_bytes, void* stream) {
  if (R < 0 || K <= 0 || N <= 0 || E < 1) return fail(MQ_ERR_INVALID_ARG, "bad R, K, N or E");
  if (a_bits != 4 && a_bits != 8) return fail(MQ_ERR_INVALID_ARG, "a_bits must be 4 or 8");
  if (!dtype_ok(out_dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown out_dtype %d", out_dtype);
  if (!mx_product_sizes_ok(R, K, N, E))
    return fail(MQ_ERR_UNSUPPORTED, "need K %% 128 == 0, E <= 1024, R < 2^30, K and N <= 2^31 - 512 and R * N < 2^39");
  if (!expert_offsets && E != 1)
    return fail(MQ_ERR_INVALID_ARG, "expert_offsets may be NULL with E = 1 only");
  if (R == 0) return MQ_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(w_scale) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(w) & 31u) || (expert_offsets && !aligned4(expert_offsets)))
    return fail(MQ_ERR_INVALID_ARG,
                "pointers must be 16-byte aligned, w 32-byte, expert_offsets 4-byte");
  const MxPlan pl = mx_plan(R, E, K, N, false, a_bits);
  const size_t need = moe_mx_product_workspace(R, K, N, E);
  if (need && (!workspace || ws_bytes < need))
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  if (need && !aligned16(workspace))
    return fail(MQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  MxGemm g = {};
  g.a_bits = a_bits;
  g.epi = pl.splits > 1 ? MX_EPI_PART : MX_EPI_OUT;
  g.a = a; g.a_scale = a_scale; g.w = w; g.w_scale = w_scale;
  g.R = R; g.S = R; g.E = E; g.K = K; g.N = N; g.wrows = N;
  g.weight_bytes = (int64_t)std::min<int64_t>(E, R) * N * K / 2;
  g.seg_start = expert_offsets;
  g.out = out; g.out_dtype = out_dtype;
  g.part = static_cast<float*>(workspace); g.part_rows = R;
  g.status = status_ptr();
  cudaError_t err;
  {
    LaunchScope ls(MQ_PROF_GEMM1, st);
    err = launch_mx_gemm(g, pl, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "mx_product launch");
  if (pl.splits > 1) {
    LaunchScope ls(MQ_PROF_COMBINE, st);
    err = launch_mx_reduce(g.part, pl.splits, R, N, expert_offsets, E, out, out_dtype, st);
    if (err != cudaSuccess) return cuda_fail(err, "mx_product: reduce launch");
  }
  return MQ_OK;
}

namespace {

struct MxLayout {
  size_t sorted, block_expert, offsets, num_padded, counts, xa, xs, act, act_s, y, total;
  int64_t cap;
  MxPlan up, down;
};

MxLayout mx_layout(int T, int H, int I, int E, int k, int bits) {
  MxLayout L;
  const int64_t S = (int64_t)T * k;
  L.up = mx_plan(S, E, H, I, true, bits);
  L.down = mx_plan(S, E, I, H, false, bits);
  const int64_t cap = moe_align_capacity(T, k, E, kAlignBlock);
  L.cap = cap;
  size_t off = 0;
  L.sorted = off;       off += align256(sizeof(int32_t) * (size_t)cap);
  L.block_expert = off; off += align256(sizeof(int32_t) * (size_t)(cap / kAlignBlock));
  L.offsets = off;      off += align256(sizeof(int32_t) * (size_t)(E + 1));
  L.num_padded = off;   off += align256(sizeof(int32_t));
  L.counts = off;       off += align256(sizeof(int32_t) * (size_t)E);
  L.xa = off;           off += align256((size_t)cap * (size_t)H * bits / 8);
  L.xs = off;           off += align256((size_t)cap * (size_t)H / 32);
  L.act = off;          off += align256((size_t)cap * (size_t)I * bits / 8);
  L.act_s = off;        off += align256((size_t)cap * (size_t)I / 32);
  L.y = off;            off += align256(sizeof(float) * (size_t)L.down.splits * (size_t)S * (size_t)H);
  L.total = off;
  return L;
}

// Refuses sizes that the forward does not take.
int mx_forward_sizes(int T, int H, int I, int E, int k, int a_bits) {
  if (T < 0 || H <= 0 || I <= 0 || E < 1) return fail(MQ_ERR_INVALID_ARG, "bad T, H, I or E");
  if (k < 1 || k > E || k > 32) return fail(MQ_ERR_INVALID_ARG, "need 1 <= k <= min(E, 32)");
  if (a_bits != 4 && a_bits != 8) return fail(MQ_ERR_INVALID_ARG, "a_bits must be 4 or 8");
  if (E > 1024) return fail(MQ_ERR_UNSUPPORTED, "E must be <= 1024");
  if (H % 128 || I % 128) return fail(MQ_ERR_UNSUPPORTED, "H and I must be multiples of 128");
  // (2I weight rows; H * a_bits bits of a row, counted in 32 bits)
  if (!mx_rounds_up(2 * (int64_t)I) || H >= 1 << 28)
    return fail(MQ_ERR_UNSUPPORTED, "need I <= 2^30 - 256 and H < 2^28");
  if ((int64_t)T * k > (int64_t(1) << 24) || !mx_units_ok((int64_t)T * k, 2 * (int64_t)I, E) ||
      !mx_units_ok((int64_t)T * k, H, E))
    return fail(MQ_ERR_UNSUPPORTED, "too many token-slots");
  return MQ_OK;
}

}  // namespace

MQ_EXPORT size_t moe_mx_forward_workspace(int T, int H, int I, int E, int k, int a_bits) {
  return mx_forward_sizes(T, H, I, E, k, a_bits) == MQ_OK ? mx_layout(T, H, I, E, k, a_bits).total : 0;
}

MQ_EXPORT int moe_mx_forward(const uint8_t* a, const uint8_t* a_scale, int a_bits, int T, int H,
                             int I, int E, int k, const uint8_t* w13, const uint8_t* s13,
                             const uint8_t* w2, const uint8_t* s2, const float* topk_w,
                             const int32_t* topk_ids, void* out, int out_dtype, void* workspace,
                             size_t ws_bytes, void* stream) {
  const int rc = mx_forward_sizes(T, H, I, E, k, a_bits);
  if (rc != MQ_OK) return rc;
  if (out_dtype != MQ_DTYPE_BF16 && out_dtype != MQ_DTYPE_F16)
    return fail(MQ_ERR_INVALID_ARG, "out_dtype must be MQ_DTYPE_BF16 or MQ_DTYPE_F16");
  if (T == 0) return MQ_OK;
  if (!a || !a_scale || !w13 || !s13 || !w2 || !s2 || !topk_w || !topk_ids || !out || !workspace)
    return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(s13) || !aligned16(s2) ||
      !aligned16(out) || !aligned16(workspace) || !aligned4(topk_w) || !aligned4(topk_ids) ||
      (reinterpret_cast<uintptr_t>(w13) & 31u) || (reinterpret_cast<uintptr_t>(w2) & 31u))
    return fail(MQ_ERR_INVALID_ARG, "pointers must be 16-byte aligned, w13 and w2 32-byte");
  const MxLayout L = mx_layout(T, H, I, E, k, a_bits);
  if (ws_bytes < L.total)
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, L.total);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + L.sorted);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  int32_t* num_padded = reinterpret_cast<int32_t*>(ws + L.num_padded);
  int32_t* counts = reinterpret_cast<int32_t*>(ws + L.counts);
  unsigned* status = status_ptr();
  const int S = T * k;
  cudaError_t err;
  // Rows in expert order: one launch for up to 2048 slots, else the align
  // kernel and a gather (see mx_arrange).
  const bool small = S <= 2048;
  {
    LaunchScope ls(MQ_PROF_ALIGN, st);
    err = small ? launch_mx_arrange(topk_ids, S, k, E, a, a_scale, H * a_bits / 8, H / 32, sorted,
                                    offsets, ws + L.xa, ws + L.xs, status, st)
                : launch_align(topk_ids, T, k, E, kAlignBlock, sorted,
                               reinterpret_cast<int32_t*>(ws + L.block_expert), offsets,
                               num_padded, status, st, 0, nullptr, nullptr, counts);
  }
  if (err != cudaSuccess) return cuda_fail(err, "mx_forward: align launch");
  if (!small) {
    LaunchScope ls(MQ_PROF_GATHER, st);
    err = launch_mx_gather(a, a_scale, H * a_bits / 8, H / 32, sorted, num_padded, k, S, L.cap,
                           ws + L.xa, ws + L.xs, st);
    if (err != cudaSuccess) return cuda_fail(err, "mx_forward: gather launch");
  }
  MxGemm g = {};
  g.a_bits = a_bits;
  g.R = L.cap; g.S = S; g.E = E;
  g.weight_bytes = (int64_t)std::min<int64_t>(E, S) * 3 * H * I / 2;
  g.seg_start = offsets; g.seg_count = small ? nullptr : counts;
  g.status = status;
  g.epi = MX_EPI_GATED;
  g.a = ws + L.xa; g.a_scale = ws + L.xs; g.w = w13; g.w_scale = s13;
  g.K = H; g.N = I; g.wrows = 2 * I;
  g.act = ws + L.act; g.act_scale = ws + L.act_s;
  {
    LaunchScope ls(MQ_PROF_GEMM1, st);
    err = launch_mx_gemm(g, L.up, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "mx_forward: gate/up launch");
  g.epi = MX_EPI_PART;
  g.a = ws + L.act; g.a_scale = ws + L.act_s; g.w = w2; g.w_scale = s2;
  g.K = I; g.N = H; g.wrows = H;
  g.part = reinterpret_cast<float*>(ws + L.y); g.part_rows = S;
  g.dest = sorted; g.dest_w = topk_w;
  {
    LaunchScope ls(MQ_PROF_GEMM2, st);
    err = launch_mx_gemm(g, L.down, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "mx_forward: down launch");
  {
    LaunchScope ls(MQ_PROF_COMBINE, st);
    err = launch_mx_combine(g.part, L.down.splits, topk_ids, T, k, E, H, out, out_dtype, st);
  }
  return err == cudaSuccess ? MQ_OK : cuda_fail(err, "mx_forward: combine launch");
}

// ---------------------------------------------------------------------------
// 16-bit weights.
// ---------------------------------------------------------------------------
static bool half_ok(int dtype) { return dtype == MQ_DTYPE_BF16 || dtype == MQ_DTYPE_F16; }

// Units of work are counted in 32 bits, with up to 16 splits of each.
static bool gg_units_ok(int64_t rows, int64_t M, int E) {
  return (rows / 16 + E) * ((M + 127) / 128) < (int64_t(1) << 27);
}

static bool gg_sizes_ok(int64_t R, int K, int N, int E) {
  constexpr int kTop = INT32_MAX - 511;  // (sizes are rounded up to tiles in 32 bits)
  return R >= 0 && K > 0 && N > 0 && E >= 1 && E <= 1024 && R < (int64_t(1) << 30) && K <= kTop &&
         N <= kTop && gg_units_ok(R, N, E) && gg_units_ok(R, K, E) &&
         (int64_t)E * ((N + 127) / 128) < (int64_t(1) << 27) / ((K + 127) / 128) &&
         (int64_t)N * K < (int64_t(1) << 52) / E;
}

static size_t gg_part_bytes(GgForm form, int64_t R, int E, int M, int N, int K) {
  const int splits = gg_plan(form, R, E, M, N, K).splits;
  const size_t n = form == GG_ROWS ? (size_t)E * M * N : (size_t)R * M;
  return splits > 1 ? align256(sizeof(float) * splits * n) : 0;
}

MQ_EXPORT size_t moe_grouped_product_workspace(int64_t R, int K, int N, int E) {
  if (!gg_sizes_ok(R, K, N, E) || R == 0) return 0;
  return std::max(gg_part_bytes(GG_W_K, R, E, N, 0, K), gg_part_bytes(GG_W_M, R, E, N, 0, K));
}

MQ_EXPORT size_t moe_grouped_product_grad_workspace(int64_t R, int K, int N, int E) {
  if (!gg_sizes_ok(R, K, N, E) || R == 0) return 0;
  return std::max({gg_part_bytes(GG_W_K, R, E, K, 0, N), gg_part_bytes(GG_W_M, R, E, K, 0, N),
                   gg_part_bytes(GG_ROWS, R, E, N, K, 0),
                   gg_part_bytes(GG_ROWS, R, E, K, N, 0)});
}

static int gg_workspace(const GgGemm& g, const void* workspace, size_t ws_bytes) {
  const size_t need = gg_part_bytes(g.form, g.R, g.E, g.M, g.N, g.K);
  if (need && (!workspace || ws_bytes < need))
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  if (need && !aligned16(workspace))
    return fail(MQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return MQ_OK;
}

// One product: the kernel, and the sum of its splits.
static int gg_run(GgGemm g, void* workspace, size_t ws_bytes, cudaStream_t st) {
  const GgPlan pl = gg_plan(g.form, g.R, g.E, g.M, g.N, g.K);
  const int ws = gg_workspace(g, workspace, ws_bytes);
  if (ws != MQ_OK) return ws;
  g.part = static_cast<float*>(workspace);
  g.status = status_ptr();
  cudaError_t err;
  {
    LaunchScope ls(MQ_PROF_GEMM1, st);
    err = launch_gg(g, pl, st);
  }
  if (err != cudaSuccess) return cuda_fail(err, "grouped product launch");
  if (pl.splits > 1) {
    LaunchScope ls(MQ_PROF_COMBINE, st);
    err = g.form == GG_ROWS
              ? launch_mx_reduce(g.part, pl.splits, (int64_t)g.E * g.M, g.N, nullptr, g.E, g.out, g.out_dtype, st)
              : launch_mx_reduce(g.part, pl.splits, g.R, g.M, g.offsets, g.E, g.out, g.out_dtype, st);
    if (err != cudaSuccess) return cuda_fail(err, "grouped product: reduce launch");
  }
  return MQ_OK;
}

// Checks that the product and its gradients share: sizes, and the weights' strides.
static int gg_args(int dtype, int64_t R, int K, int N, int E, int64_t w_stride,
                   int64_t w_expert_stride, int w_transposed, bool w_read,
                   const int32_t* expert_offsets) {
  if (!dtype_ok(dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (dtype == MQ_DTYPE_F32) return fail(MQ_ERR_UNSUPPORTED, "rows and weights must be bfloat16 or float16");
  if (R < 0 || K <= 0 || N <= 0 || E < 1) return fail(MQ_ERR_INVALID_ARG, "bad R, K, N or E");
  if (!gg_sizes_ok(R, K, N, E))
    return fail(MQ_ERR_UNSUPPORTED, "need E <= 1024, R < 2^30, K and N <= 2^31 - 512 and fewer than 2^27 tiles");
  if (!expert_offsets && E != 1)
    return fail(MQ_ERR_INVALID_ARG, "expert_offsets may be NULL with E = 1 only");
  const int row = w_transposed ? N : K, rows = w_transposed ? K : N;
  if (!w_read) return MQ_OK;
  if ((rows > 1 && w_stride < row) || w_stride < 0 || w_stride % 8 || (E > 1 && (w_expert_stride <= 0 || w_expert_stride % 8)))
    return fail(MQ_ERR_INVALID_ARG, "the weights' strides must be multiples of 8, a row's at least its length");
  return MQ_OK;
}

static bool gg_row_stride_ok(int64_t stride, int64_t cols, int64_t R) {
  return stride % 8 == 0 && stride >= 0 && (R <= 1 || stride >= cols);
}

// The largest stride of a tensor map is below 2^40 bytes; a stride that is never
// taken (one row, one expert) is replaced.
static bool gg_map_strides(int64_t& row, int64_t rows, int64_t len, int64_t* expert, int E) {
  const int64_t round = (len + 7) / 8 * 8;
  if (rows <= 1) row = round;
  if (expert && E == 1) *expert = round;
  constexpr int64_t kTop = int64_t(1) << 39;
  return row < kTop && (!expert || *expert < kTop);
}

// The bytes from the first to the last one of an array (none where it is missing).
struct Span {
  uintptr_t lo, hi;
  Span(const void* p, int64_t elements, int64_t size)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(p ? lo + (uintptr_t)(elements * size) : lo) {}
  bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

static Span row_span(const void* p, int64_t R, int64_t stride, int64_t cols) {
  return Span(p, (R - 1) * stride + cols, 2);
}

// Whether one of R rows of `len` bytes, `stride` bytes apart, meets a span.
static bool rows_meet(const void* p, int64_t R, int64_t stride, int64_t len, const Span& s) {
  if (!p || s.lo == s.hi) return false;
  const int64_t first = (int64_t)reinterpret_cast<uintptr_t>(p), lo = (int64_t)s.lo, hi = (int64_t)s.hi;
  int64_t i = 0;  // the first row that ends behind the span's beginning
  if (R > 1 && first + len <= lo) i = (lo - len - first) / stride + 1;
  return i < R && first + i * stride + len > lo && first + i * stride < hi;
}

static int workspace_shared() {
  return fail(MQ_ERR_INVALID_ARG, "the workspace must not share memory with an input or a result");
}

static Span weight_span(const void* w, int K, int N, int E, int64_t stride, int64_t expert, int transposed) {
  const int64_t rows = transposed ? K : N, len = transposed ? N : K;
  return Span(w, (E - 1) * expert + (rows - 1) * stride + len, 2);
}

static int64_t dtype_size(int dtype) { return dtype == MQ_DTYPE_F32 ? 4 : 2; }

MQ_EXPORT int moe_grouped_product(const void* a, int64_t a_stride, int dtype, int64_t R, int K,
                                  int N, int E, const void* w, int64_t w_stride,
                                  int64_t w_expert_stride, int w_transposed,
                                  const int32_t* expert_offsets, void* out, int out_dtype,
                                  void* workspace, size_t ws_bytes, void* stream) {
  const int rc = gg_args(dtype, R, K, N, E, w_stride, w_expert_stride, w_transposed, true, expert_offsets);
  if (rc != MQ_OK) return rc;
  if (!dtype_ok(out_dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown out_dtype %d", out_dtype);
  if (!gg_row_stride_ok(a_stride, K, R))
    return fail(MQ_ERR_INVALID_ARG, "a_stride must be a multiple of 8, at least K");
  if (R == 0) return MQ_OK;
  if (!a || !w || !out) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(a) || !aligned16(w) || !aligned16(out) || (expert_offsets && !aligned4(expert_offsets)))
    return fail(MQ_ERR_INVALID_ARG, "pointers must be 16-byte aligned, expert_offsets 4-byte");
  if (!gg_map_strides(a_stride, R, K, nullptr, 1) ||
      !gg_map_strides(w_stride, w_transposed ? K : N, w_transposed ? N : K, &w_expert_stride, E))
    return fail(MQ_ERR_UNSUPPORTED, "strides of 2^39 elements or more");
  GgGemm g = {};
  g.form = w_transposed ? GG_W_M : GG_W_K;
  g.bf16 = dtype == MQ_DTYPE_BF16;
  g.w = w; g.w_stride = w_stride; g.w_expert = w_expert_stride;
  g.a = a; g.a_stride = a_stride;
  g.R = R; g.E = E; g.M = N; g.K = K;
  g.offsets = expert_offsets;
  g.out = out; g.out_dtype = out_dtype;
  const int ws = gg_workspace(g, workspace, ws_bytes);
  if (ws != MQ_OK) return ws;
  const Span written(out, R * N, dtype_size(out_dtype));
  if (written.meets(row_span(a, R, a_stride, K)) ||
      written.meets(weight_span(w, K, N, E, w_stride, w_expert_stride, w_transposed)) ||
      written.meets(Span(expert_offsets, E + 1, 4)))
    return fail(MQ_ERR_INVALID_ARG, "out must not share memory with a, w or expert_offsets");
  const Span used(workspace, (int64_t)gg_part_bytes(g.form, R, E, N, 0, K), 1);
  if (used.meets(written) || rows_meet(a, R, a_stride * 2, (int64_t)K * 2, used) ||
      used.meets(weight_span(w, K, N, E, w_stride, w_expert_stride, w_transposed)) ||
      used.meets(Span(expert_offsets, E + 1, 4)))
    return workspace_shared();
  return gg_run(g, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

MQ_EXPORT int moe_grouped_product_grad(const void* dy, int64_t dy_stride, const void* a,
                                       int64_t a_stride, int dtype, int64_t R, int K, int N, int E,
                                       const void* w, int64_t w_stride, int64_t w_expert_stride,
                                       int w_transposed, const int32_t* expert_offsets, void* da,
                                       void* dw, int dw_dtype, void* workspace, size_t ws_bytes,
                                       void* stream) {
  const int rc = gg_args(dtype, R, K, N, E, w_stride, w_expert_stride, w_transposed, da != nullptr, expert_offsets);
  if (rc != MQ_OK) return rc;
  if (!dtype_ok(dw_dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown dw_dtype %d", dw_dtype);
  if (!gg_row_stride_ok(a_stride, K, R) || !gg_row_stride_ok(dy_stride, N, R))
    return fail(MQ_ERR_INVALID_ARG, "row strides must be multiples of 8, at least a row's length");
  if (!aligned16(dy) || !aligned16(a) || !aligned16(w) || !aligned16(da) || !aligned16(dw) ||
      (expert_offsets && !aligned4(expert_offsets)))
    return fail(MQ_ERR_INVALID_ARG, "pointers must be 16-byte aligned, expert_offsets 4-byte");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (R == 0) {  // no rows: the weights' gradient is zero
    if (!dw) return MQ_OK;
    const size_t bytes = (size_t)E * N * K * (dw_dtype == MQ_DTYPE_F32 ? 4 : 2);
    const cudaError_t err = cudaMemsetAsync(dw, 0, bytes, st);
    return err == cudaSuccess ? MQ_OK : cuda_fail(err, "grouped product's gradient: memset");
  }
  if ((da || dw) && (!dy || (da && !w) || (dw && !a))) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  if (!gg_map_strides(a_stride, R, K, nullptr, 1) || !gg_map_strides(dy_stride, R, N, nullptr, 1) ||
      !gg_map_strides(w_stride, w_transposed ? K : N, w_transposed ? N : K, &w_expert_stride, E))
    return fail(MQ_ERR_UNSUPPORTED, "strides of 2^39 elements or more");
  const size_t need = moe_grouped_product_grad_workspace(R, K, N, E);
  if (need && (!workspace || ws_bytes < need))
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  const Span da_span(da, R * K, 2), dw_span(dw, (int64_t)E * N * K, dtype_size(dw_dtype));
  const Span read[4] = {row_span(dy, R, dy_stride, N), row_span(dw ? a : nullptr, R, a_stride, K),
                        weight_span(da ? w : nullptr, K, N, E, w_stride, w_expert_stride, w_transposed),
                        Span(expert_offsets, E + 1, 4)};
  for (const Span& in : read)
    if (da_span.meets(in) || dw_span.meets(in))
      return fail(MQ_ERR_INVALID_ARG, "da and dw must not share memory with dy, a, w or expert_offsets");
  if (da_span.meets(dw_span)) return fail(MQ_ERR_INVALID_ARG, "da and dw must not share memory");
  if (need && !aligned16(workspace)) return fail(MQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const Span used(workspace, (int64_t)need, 1);
  if (used.meets(da_span) || used.meets(dw_span) || rows_meet(dy, R, dy_stride * 2, (int64_t)N * 2, used) ||
      (dw && rows_meet(a, R, a_stride * 2, (int64_t)K * 2, used)) || used.meets(read[2]) || used.meets(read[3]))
    return workspace_shared();
  GgGemm g = {};
  g.bf16 = dtype == MQ_DTYPE_BF16;
  g.R = R; g.E = E;
  g.offsets = expert_offsets;
  GgGemm of_rows = g, of_weights = g;
  if (da) {  // W's outputs are the contraction: the other of the two storages
    of_rows.form = w_transposed ? GG_W_K : GG_W_M;
    of_rows.w = w; of_rows.w_stride = w_stride; of_rows.w_expert = w_expert_stride;
    of_rows.a = dy; of_rows.a_stride = dy_stride;
    of_rows.M = K; of_rows.K = N;
    of_rows.out = da; of_rows.out_dtype = dtype;
    of_rows.zero_outside = true;
  }
  if (dw) {  // laid out as the weights are
    of_weights.form = GG_ROWS;
    of_weights.w = w_transposed ? a : dy; of_weights.w_stride = w_transposed ? a_stride : dy_stride;
    of_weights.a = w_transposed ? dy : a; of_weights.a_stride = w_transposed ? dy_stride : a_stride;
    of_weights.M = w_transposed ? K : N; of_weights.N = w_transposed ? N : K;
    of_weights.out = dw; of_weights.out_dtype = dw_dtype;
  }
  if (da && dw && gg_side_by_side(of_rows, of_weights)) {
    of_rows.status = of_weights.status = status_ptr();
    LaunchScope ls(MQ_PROF_GEMM1, st);
    const cudaError_t err = launch_gg_both(of_rows, of_weights, st);
    return err == cudaSuccess ? MQ_OK : cuda_fail(err, "grouped product's gradients launch");
  }
  if (da) {
    const int r = gg_run(of_rows, workspace, ws_bytes, st);
    if (r != MQ_OK) return r;
  }
  return dw ? gg_run(of_weights, workspace, ws_bytes, st) : MQ_OK;
}

static bool lora_sizes_ok(int64_t R, int K, int N, int r, int L, int E) {
  constexpr int kTop = 1 << 30;
  return R >= 0 && R < kTop && K > 0 && N > 0 && K % 8 == 0 && K < kTop && N < kTop && r >= 8 && r <= 128 &&
         r % 8 == 0 && L >= 1 && E >= 1 && E <= 1024 && (int64_t)L * E < kTop &&
         (R + 127) / 128 * (((int64_t)N + 127) / 128) < (int64_t(1) << 27) &&
         (int64_t)L * E < (int64_t(1) << 48) / ((int64_t)K + N);
}

MQ_EXPORT size_t moe_lora_product_workspace(int64_t R, int K, int N, int r, int L, int E) {
  if (!lora_sizes_ok(R, K, N, r, L, E) || R == 0) return 0;
  const LoraPlan pl = lora_plan(R, K, N, r, L, E);
  return pl.rows ? 0 : align256(lora_workspace(pl, R, r));
}

// Whether R rows of `len` bytes, `stride` bytes apart, share a byte with R others.
// (With equal strides exactly; with others, whether the ranges do.)
static bool rows_overlap(const void* p, int64_t stride, int64_t len, const void* q, int64_t q_stride,
                         int64_t q_len, int64_t R) {
  const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(p), b = (int64_t)reinterpret_cast<uintptr_t>(q);
  if (a + (R - 1) * stride + len <= b || b + (R - 1) * q_stride + q_len <= a) return false;
  if (stride != q_stride || R <= 1) return true;
  const int64_t d = b >= a ? (b - a) % stride : stride - 1 - (a - b - 1) % stride;  // of q's rows in p's
  return d < len || d + q_len > stride;
}

MQ_EXPORT int moe_lora_product(const void* x, int64_t x_stride, int dtype, int64_t R, int K, int N, int r,
                               int L, int E, const void* lora_a, const void* lora_b,
                               const int32_t* adapter_ids, const int32_t* expert_offsets,
                               const float* scaling, const void* base, int64_t base_stride, void* out,
                               int64_t out_stride, int out_dtype, void* workspace, size_t ws_bytes,
                               void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return fail(MQ_ERR_INVALID_ARG, "unknown dtype");
  if (!half_ok(dtype)) return fail(MQ_ERR_UNSUPPORTED, "rows and adapters must be bfloat16 or float16");
  if (R < 0 || K <= 0 || N <= 0 || r <= 0 || L < 1 || E < 1)
    return fail(MQ_ERR_INVALID_ARG, "bad R, K, N, r, L or E");
  if (K % 8 || r % 8) return fail(MQ_ERR_INVALID_ARG, "K and r must be multiples of 8");
  if (!lora_sizes_ok(R, K, N, r, L, E))
    return fail(MQ_ERR_UNSUPPORTED, "need r <= 128, E <= 1024, and R, K, N and L * E < 2^30, fewer than 2^27 tiles");
  if (!expert_offsets && E != 1)
    return fail(MQ_ERR_INVALID_ARG, "expert_offsets may be NULL with E = 1 only");
  if (!gg_row_stride_ok(x_stride, K, R))
    return fail(MQ_ERR_INVALID_ARG, "x_stride must be a multiple of 8, at least K");
  if (R > 1 && (out_stride < N || (base && base_stride < N)))
    return fail(MQ_ERR_INVALID_ARG, "row strides must be at least a row's length");
  if (R == 0) return MQ_OK;
  if (!x || !lora_a || !lora_b || !adapter_ids || !out) return fail(MQ_ERR_INVALID_ARG, "null pointer");
  const int64_t size = out_dtype == MQ_DTYPE_F32 ? 4 : 2;
  if (!aligned16(x) || !aligned16(lora_a) || !aligned16(lora_b) || !aligned4(adapter_ids) ||
      (expert_offsets && !aligned4(expert_offsets)) || (scaling && !aligned4(scaling)) ||
      reinterpret_cast<uintptr_t>(out) % size || reinterpret_cast<uintptr_t>(base) % size)
    return fail(MQ_ERR_INVALID_ARG, "x and the adapters must be 16-byte aligned, other pointers to their elements");
  if (!gg_map_strides(x_stride, R, K, nullptr, 1) || !gg_map_strides(out_stride, R, N, nullptr, 1) ||
      !gg_map_strides(base_stride, base ? R : 1, N, nullptr, 1))
    return fail(MQ_ERR_UNSUPPORTED, "strides of 2^39 elements or more");
  if (rows_overlap(out, out_stride * size, N * size, x, x_stride * 2, (int64_t)K * 2, R) ||
      (base && !(base == out && (base_stride == out_stride || R == 1)) &&
       rows_overlap(out, out_stride * size, N * size, base, base_stride * size, N * size, R)))
    return fail(MQ_ERR_INVALID_ARG, "out must not share memory with x, or with base other than as the same rows");
  const LoraPlan pl = lora_plan(R, K, N, r, L, E);
  const size_t need = moe_lora_product_workspace(R, K, N, r, L, E);
  if (need && (!workspace || ws_bytes < need))
    return fail(MQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace ? ws_bytes : 0, need);
  if (need && !aligned16(workspace)) return fail(MQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const Span written(out, (R - 1) * out_stride + N, size);
  const int64_t groups = (int64_t)L * E;
  if (written.meets(Span(lora_a, groups * r * K, 2)) || written.meets(Span(lora_b, groups * r * N, 2)) ||
      written.meets(Span(adapter_ids, R, 4)) || written.meets(Span(expert_offsets, E + 1, 4)) ||
      written.meets(Span(scaling, L, 4)))
    return fail(MQ_ERR_INVALID_ARG, "out must not share memory with the adapters, their ids, scaling or expert_offsets");
  const Span used(workspace, (int64_t)need, 1);
  if (rows_meet(out, R, out_stride * size, N * size, used) || rows_meet(base, R, base_stride * size, N * size, used) ||
      rows_meet(x, R, x_stride * 2, (int64_t)K * 2, used) || used.meets(Span(lora_a, groups * r * K, 2)) ||
      used.meets(Span(lora_b, groups * r * N, 2)) || used.meets(Span(adapter_ids, R, 4)) ||
      used.meets(Span(expert_offsets, E + 1, 4)) || used.meets(Span(scaling, L, 4)))
    return workspace_shared();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LoraArgs g = {};
  g.bf16 = dtype == MQ_DTYPE_BF16;
  g.x = x; g.x_stride = x_stride;
  g.R = R; g.K = K; g.N = N; g.r = r; g.L = L; g.E = E;
  g.a = lora_a; g.b = lora_b;
  g.ids = adapter_ids; g.offsets = expert_offsets; g.scaling = scaling;
  g.base = base; g.base_stride = base_stride;
  g.out = out; g.out_stride = out_stride; g.out_dtype = out_dtype;
  g.workspace = static_cast<uint8_t*>(workspace);
  g.status = status_ptr();
  for (int which = 0; which < (pl.rows ? 1 : 2); ++which) {
    LaunchScope ls(which ? MQ_PROF_GEMM2 : MQ_PROF_GEMM1, st);
    const cudaError_t err = launch_lora(g, pl, which, st);
    if (err != cudaSuccess) return cuda_fail(err, "lora_product launch");
  }
  return MQ_OK;
}
