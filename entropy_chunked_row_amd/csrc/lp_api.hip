// C ABI of liblp.so (declared in include/lp.h): argument validation, chunk /
// tile scheduling and stream-ordered launches.  Every check runs on the host
// before anything is launched; a rejected call touches no output.
#include <initializer_list>
#include <mutex>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "../../include/lp.h"
#include "lp_internal.hpp"

namespace {

thread_local char g_err[512] = {0};

lp_status fail(lp_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

lp_status ok() {
  g_err[0] = 0;
  return LP_OK;
}

lp_status hip_fail(hipError_t e, const char* where) {
  return fail(LP_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

// The launchers read hipGetLastError() after each launch; an error left
// pending on this thread by an earlier, unrelated runtime call (the caller's
// or another library's) would be reported as ours.  Clear it first.
void clear_pending_hip_error() { (void)hipGetLastError(); }

constexpr double kLog2eD = 1.44269504088896340736;
constexpr int64_t kMaxV = (int64_t(1) << 30);

bool temperature_applies(float t) { return t > 0.f && t != 1.f; }

// c = log2(e) / tau_effective, rounded once.
float exp2_scale(float temperature) {
  const double tau = temperature_applies(temperature) ? static_cast<double>(temperature) : 1.0;
  return static_cast<float>(kLog2eD / tau);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Every fp32 array argument (NULL allowed) must be 4-byte aligned.
bool f32_aligned(std::initializer_list<const float*> ps) {
  for (const float* p : ps)
    if (p && !aligned(p, 4)) return false;
  return true;
}

size_t dtype_bytes(int d) { return d == LP_FP32 ? 4 : 2; }

}  // namespace

// Scratch of lp_lm_head_logprobs_entropy_noalloc: one copy per GPU the
// library runs on, held until the process ends.  Host code never passes this
// name to a kernel (on the host it is only a stand-in for the symbol): the
// device address of each GPU's copy comes from hipGetSymbolAddress below.
static __device__ __align__(256) unsigned char scratch[LP_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's scratch, looked up once per device
// (with that device current) and kept.
hipError_t scratch_of_current_device(int* device, void** out) {
  hipError_t e = hipGetDevice(device);
  if (e != hipSuccess) return e;
  if (*device < 0 || *device >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[*device]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    g_scratch_ptr[*device] = p;
  }
  *out = g_scratch_ptr[*device];
  return hipSuccess;
}

}  // namespace

extern "C" {

int lp_version(void) { return 100; }

const char* lp_status_string(int status) {
  switch (status) {
    case LP_OK: return "LP_OK";
    case LP_ERR_INVALID_ARGUMENT: return "LP_ERR_INVALID_ARGUMENT";
    case LP_ERR_UNSUPPORTED: return "LP_ERR_UNSUPPORTED";
    case LP_ERR_WORKSPACE_TOO_SMALL: return "LP_ERR_WORKSPACE_TOO_SMALL";
    case LP_ERR_HIP: return "LP_ERR_HIP";
    default: return "unknown status";
  }
}

const char* lp_last_error(void) { return g_err; }

static lp_status logprobs_entropy_impl(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                       const int64_t* targets, int64_t K, const uint8_t* mask, float temperature,
                                       int64_t chunk_rows, float* logprob, float* entropy, void* stream) {
  if (K < 1 || K > lp::kMaxTargets)
    return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: K must be in 1..%d", lp::kMaxTargets);
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: unknown dtype %d", static_cast<int>(dtype));
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: T < 0");
  if (V <= 0 || V > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: V out of range (1..2^30)");
  if (ld < V) return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: ld < V");
  if (!isfinite(temperature)) return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: temperature not finite");
  if (T == 0) return ok();
  if (!logits || !targets || !logprob)
    return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: logits, targets and logprob are required");
  if (!aligned(logits, dtype_bytes(dtype)) || !aligned(logprob, 4) || (entropy && !aligned(entropy, 4)) ||
      !aligned(targets, 8))
    return fail(LP_ERR_INVALID_ARGUMENT, "lp_logprobs_entropy: misaligned pointer");
  // Chunks bound the rows whose fp32 copy exists at once in the page's
  // design; here no fp32 copy exists (rows are widened in registers), so all
  // chunks of the call run back to back in one launch, in row order: one
  // drain of the grid per call instead of one per chunk, and results that do
  // not depend on chunk_rows.
  (void)chunk_rows;
  hipStream_t s = static_cast<hipStream_t>(stream);
  lp::RowArgs a;
  a.x = logits;
  a.ld = ld;
  a.V = static_cast<int>(V);
  a.targets = targets;
  a.K = static_cast<int>(K);
  a.mask = mask;
  a.c = exp2_scale(temperature);
  a.logprob = logprob;
  a.entropy = entropy;
  a.row0 = 0;
  a.rows = T;
  clear_pending_hip_error();
  hipError_t e = lp::launch_logprobs_entropy(static_cast<int>(dtype), a, s);
  if (e != hipSuccess) return hip_fail(e, "lp_logprobs_entropy launch");
  return ok();
}

lp_status lp_logprobs_entropy(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                              const int64_t* targets, const uint8_t* mask, float temperature,
                              int64_t chunk_rows, float* logprob, float* entropy, void* stream) {
  return logprobs_entropy_impl(logits, dtype, T, V, ld, targets, 1, mask, temperature, chunk_rows, logprob, entropy,
                               stream);
}

lp_status lp_logprobs_entropy_k(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                const int64_t* targets, int64_t K, const uint8_t* mask, float temperature,
                                int64_t chunk_rows, float* logprob, float* entropy, void* stream) {
  return logprobs_entropy_impl(logits, dtype, T, V, ld, targets, K, mask, temperature, chunk_rows, logprob, entropy,
                               stream);
}

int lp_lm_head_fast_tiles(int64_t T, int64_t h, int64_t V, int64_t ld_h, int64_t ld_w, int64_t tile_rows,
                          int backward) {
  if (T < 0 || h <= 0 || V <= 0 || V > kMaxV || h > kMaxV || ld_h < h || ld_w < h || tile_rows <= 0) return -1;
  return lp::lmhead_fast_tiles(T, h, V, ld_h, ld_w, tile_rows, backward ? 1 : 0) ? 1 : 0;
}

size_t lp_lm_head_workspace_bytes(int64_t T, int64_t h, int64_t V, int64_t tile_rows, int backward) {
  lp::LMHeadWorkspace w;
  if (!lp::lmhead_workspace_layout(T, h, V, tile_rows, backward, &w)) return 0;
  return w.total;
}

// static_scratch: the call brings no workspace (the no-alloc form checks its
// own scratch), so `workspace` is not examined.
static lp_status check_lmhead(const char* fn, const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                              int64_t T, int64_t h, int64_t V, const int64_t* targets, float temperature,
                              int64_t tile_rows, void* workspace, size_t workspace_bytes, int backward,
                              lp::LMHeadWorkspace* w, bool static_scratch = false) {
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  if (h <= 0 || V <= 0 || V > kMaxV || h > kMaxV)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: h and V must be in 1..2^30", fn);
  if (ld_h < h || ld_w < h) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_h and ld_w must be >= h", fn);
  if (tile_rows <= 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: tile_rows must be > 0", fn);
  if (!isfinite(temperature)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: temperature not finite", fn);
  if (h % 8 || ld_h % 8 || ld_w % 8)
    return fail(LP_ERR_UNSUPPORTED, "%s: h, ld_h and ld_w must be multiples of 8", fn);
  if (T == 0) return LP_OK;
  if (!hidden || !weight || !targets) return fail(LP_ERR_INVALID_ARGUMENT, "%s: hidden, weight, targets required", fn);
  if (!aligned(hidden, 16) || !aligned(weight, 16))
    return fail(LP_ERR_UNSUPPORTED, "%s: hidden and weight must be 16-byte aligned", fn);
  if (!aligned(targets, 8)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned targets", fn);
  if (!lp::lmhead_workspace_layout(T, h, V, tile_rows, backward, w))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: sizes overflow the workspace layout", fn);
  if (!lp::lmhead_launches_fit(T, h, V, tile_rows, backward))
    return fail(LP_ERR_UNSUPPORTED, "%s: a launch would exceed 2^32-1 work-items; use a smaller tile_rows", fn);
  if (static_scratch) return LP_OK;
  if (!workspace || workspace_bytes < w->total)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes, got %zu", fn, w->total,
                workspace ? workspace_bytes : size_t(0));
  if (!aligned(workspace, 256)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  return LP_OK;
}

static lp::LMHeadShape make_shape(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w, int64_t T,
                                  int64_t h, int64_t V, const int64_t* targets, int64_t K, const uint8_t* mask,
                                  float temperature, int64_t tile_rows) {
  lp::LMHeadShape sh;
  sh.hidden = static_cast<const uint16_t*>(hidden);
  sh.ld_h = ld_h;
  sh.weight = static_cast<const uint16_t*>(weight);
  sh.ld_w = ld_w;
  sh.T = T;
  sh.h = static_cast<int>(h);
  sh.V = static_cast<int>(V);
  sh.targets = targets;
  sh.K = static_cast<int>(K);
  sh.mask = mask;
  sh.c = exp2_scale(temperature);
  sh.inv_tau = temperature_applies(temperature) ? 1.0f / temperature : 1.0f;
  sh.tile_rows = tile_rows;
  return sh;
}

static lp_status lm_head_forward_impl(const char* fn, const void* hidden, int64_t ld_h, const void* weight,
                                      int64_t ld_w, int64_t T, int64_t h, int64_t V, const int64_t* targets,
                                      int64_t K, const uint8_t* mask, float temperature, int64_t tile_rows,
                                      float* logprob, float* entropy, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (K < 1 || K > lp::kMaxTargets) return fail(LP_ERR_INVALID_ARGUMENT, "%s: K must be in 1..%d", fn, lp::kMaxTargets);
  lp::LMHeadWorkspace w;
  lp_status st = check_lmhead(fn, hidden, ld_h, weight, ld_w, T, h, V, targets, temperature, tile_rows,
                              workspace, workspace_bytes, 0, &w);
  if (st != LP_OK) return st;
  if (T == 0) return ok();
  if (!logprob) return fail(LP_ERR_INVALID_ARGUMENT, "%s: logprob is required", fn);
  if (!f32_aligned({logprob, entropy, lse})) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned fp32 output", fn);
  lp::LMHeadShape sh = make_shape(hidden, ld_h, weight, ld_w, T, h, V, targets, K, mask, temperature, tile_rows);
  clear_pending_hip_error();
  hipError_t e = lp::launch_lmhead_forward(sh, logprob, entropy, lse, static_cast<char*>(workspace), w,
                                           static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_lm_head_logprobs_entropy(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                                      int64_t T, int64_t h, int64_t V, const int64_t* targets,
                                      const uint8_t* mask, float temperature, int64_t tile_rows,
                                      float* logprob, float* entropy, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return lm_head_forward_impl("lp_lm_head_logprobs_entropy", hidden, ld_h, weight, ld_w, T, h, V, targets, 1, mask,
                              temperature, tile_rows, logprob, entropy, lse, workspace, workspace_bytes, stream);
}

lp_status lp_lm_head_logprobs_entropy_k(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                                        int64_t T, int64_t h, int64_t V, const int64_t* targets, int64_t K,
                                        const uint8_t* mask, float temperature, int64_t tile_rows, float* logprob,
                                        float* entropy, float* lse, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  return lm_head_forward_impl("lp_lm_head_logprobs_entropy_k", hidden, ld_h, weight, ld_w, T, h, V, targets, K, mask,
                              temperature, tile_rows, logprob, entropy, lse, workspace, workspace_bytes, stream);
}

lp_status lp_lm_head_logprobs_entropy_noalloc(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                                              int64_t T, int64_t h, int64_t V, const int64_t* targets,
                                              const uint8_t* mask, float temperature, int64_t tile_rows,
                                              float* logprob, float* entropy, float* lse, void* stream) {
  const char* fn = "lp_lm_head_logprobs_entropy_noalloc";
  lp::LMHeadWorkspace w;
  lp_status st = check_lmhead(fn, hidden, ld_h, weight, ld_w, T, h, V, targets, temperature, tile_rows, nullptr, 0,
                              0, &w, true);
  if (st != LP_OK) return st;
  if (T == 0) return ok();
  if (w.total > LP_NOALLOC_SCRATCH_BYTES)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL,
                "%s: this shape needs %zu bytes of scratch, the static scratch holds %zu; use a smaller tile_rows "
                "or the workspace form",
                fn, w.total, static_cast<size_t>(LP_NOALLOC_SCRATCH_BYTES));
  if (!logprob) return fail(LP_ERR_INVALID_ARGUMENT, "%s: logprob is required", fn);
  if (!f32_aligned({logprob, entropy, lse})) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned fp32 output", fn);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int device = 0;
  void* ws = nullptr;
  hipError_t e = scratch_of_current_device(&device, &ws);
  if (e != hipSuccess) return hip_fail(e, fn);
  if (s) {
    hipDevice_t sd = 0;
    e = hipStreamGetDevice(s, &sd);
    if (e != hipSuccess) return hip_fail(e, fn);
    if (sd != device)
      return fail(LP_ERR_INVALID_ARGUMENT, "%s: the stream belongs to device %d, the current device is %d", fn,
                  static_cast<int>(sd), device);
  }
  lp::LMHeadShape sh = make_shape(hidden, ld_h, weight, ld_w, T, h, V, targets, 1, mask, temperature, tile_rows);
  clear_pending_hip_error();
  e = lp::launch_lmhead_forward(sh, logprob, entropy, lse, static_cast<char*>(ws), w, s);
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

static lp_status lm_head_backward_impl(const char* fn, const void* hidden, int64_t ld_h, const void* weight,
                                       int64_t ld_w, int64_t T, int64_t h, int64_t V, const int64_t* targets,
                                       int64_t K, const uint8_t* mask, float temperature, int64_t tile_rows,
                                       const float* lse, const float* entropy, const float* grad_logprob,
                                       const float* grad_entropy, float* grad_hidden, float* grad_weight,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  if (K < 1 || K > lp::kMaxTargets) return fail(LP_ERR_INVALID_ARGUMENT, "%s: K must be in 1..%d", fn, lp::kMaxTargets);
  lp::LMHeadWorkspace w;
  lp_status st = check_lmhead(fn, hidden, ld_h, weight, ld_w, T, h, V, targets, temperature, tile_rows,
                              workspace, workspace_bytes, 1, &w);
  if (st != LP_OK) return st;
  if (!f32_aligned({lse, entropy, grad_logprob, grad_entropy, grad_hidden, grad_weight}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned fp32 argument", fn);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0) {
    // no rows: the weight gradient is still defined (all zero)
    if (grad_weight) {
      clear_pending_hip_error();
      hipError_t e = lp::launch_zero_f32(grad_weight, V * h, s);
      if (e != hipSuccess) return hip_fail(e, fn);
    }
    return ok();
  }
  if (!lse || !entropy || !grad_logprob)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: lse, entropy and grad_logprob are required", fn);
  lp::LMHeadShape sh = make_shape(hidden, ld_h, weight, ld_w, T, h, V, targets, K, mask, temperature, tile_rows);
  clear_pending_hip_error();
  hipError_t e = lp::launch_lmhead_backward(sh, lse, entropy, grad_logprob, grad_entropy, grad_hidden,
                                            grad_weight, static_cast<char*>(workspace), w, s);
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_lm_head_logprobs_entropy_backward(const void* hidden, int64_t ld_h, const void* weight,
                                               int64_t ld_w, int64_t T, int64_t h, int64_t V,
                                               const int64_t* targets, const uint8_t* mask,
                                               float temperature, int64_t tile_rows, const float* lse,
                                               const float* entropy, const float* grad_logprob,
                                               const float* grad_entropy, float* grad_hidden,
                                               float* grad_weight, void* workspace, size_t workspace_bytes,
                                               void* stream) {
  return lm_head_backward_impl("lp_lm_head_logprobs_entropy_backward", hidden, ld_h, weight, ld_w, T, h, V, targets,
                               1, mask, temperature, tile_rows, lse, entropy, grad_logprob, grad_entropy, grad_hidden,
                               grad_weight, workspace, workspace_bytes, stream);
}

lp_status lp_lm_head_logprobs_entropy_backward_k(const void* hidden, int64_t ld_h, const void* weight,
                                                 int64_t ld_w, int64_t T, int64_t h, int64_t V,
                                                 const int64_t* targets, int64_t K, const uint8_t* mask,
                                                 float temperature, int64_t tile_rows, const float* lse,
                                                 const float* entropy, const float* grad_logprob,
                                                 const float* grad_entropy, float* grad_hidden, float* grad_weight,
                                                 void* workspace, size_t workspace_bytes, void* stream) {
  return lm_head_backward_impl("lp_lm_head_logprobs_entropy_backward_k", hidden, ld_h, weight, ld_w, T, h, V, targets,
                               K, mask, temperature, tile_rows, lse, entropy, grad_logprob, grad_entropy, grad_hidden,
                               grad_weight, workspace, workspace_bytes, stream);
}

size_t lp_lm_head_kl_workspace_bytes(int64_t T, int64_t h_student, int64_t V, int64_t tile_rows, int backward) {
  lp::LMHeadWorkspace w;
  if (!lp::lmhead_workspace_layout(T, h_student, V, tile_rows, backward ? 3 : 2, &w)) return 0;
  return w.total;
}

// Checks of one head's operands (T > 0).
static lp_status check_head(const char* fn, const char* who, const void* hidden, int64_t ld_h, const void* weight,
                            int64_t ld_w, int64_t h) {
  if (h <= 0 || h > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "%s: %s h must be in 1..2^30", fn, who);
  if (ld_h < h || ld_w < h) return fail(LP_ERR_INVALID_ARGUMENT, "%s: %s ld_h and ld_w must be >= h", fn, who);
  if (h % 8 || ld_h % 8 || ld_w % 8)
    return fail(LP_ERR_UNSUPPORTED, "%s: %s h, ld_h and ld_w must be multiples of 8", fn, who);
  if (!hidden || !weight) return fail(LP_ERR_INVALID_ARGUMENT, "%s: %s hidden and weight are required", fn, who);
  if (!aligned(hidden, 16) || !aligned(weight, 16))
    return fail(LP_ERR_UNSUPPORTED, "%s: %s hidden and weight must be 16-byte aligned", fn, who);
  return LP_OK;
}

static lp_status check_kl_heads(const char* fn, const void* hs, int64_t ld_hs, const void* ws_, int64_t ld_ws,
                                int64_t h_s, const void* ht, int64_t ld_ht, const void* wt, int64_t ld_wt,
                                int64_t h_t, int64_t T, int64_t V, int64_t tile_rows, void* workspace,
                                size_t workspace_bytes, int backward, lp::LMHeadWorkspace* w) {
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  if (V <= 0 || V > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "%s: V must be in 1..2^30", fn);
  if (h_s <= 0 || h_s > kMaxV || h_t <= 0 || h_t > kMaxV)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: h_student and h_teacher must be in 1..2^30", fn);
  if (tile_rows <= 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: tile_rows must be > 0", fn);
  if (T == 0) return LP_OK;
  lp_status st = check_head(fn, "student", hs, ld_hs, ws_, ld_ws, h_s);
  if (st != LP_OK) return st;
  if ((st = check_head(fn, "teacher", ht, ld_ht, wt, ld_wt, h_t)) != LP_OK) return st;
  if (!lp::lmhead_workspace_layout(T, h_s, V, tile_rows, backward ? 3 : 2, w))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: sizes overflow the workspace layout", fn);
  if (!lp::lmhead_launches_fit(T, h_s > h_t ? h_s : h_t, V, tile_rows, backward ? 3 : 2))
    return fail(LP_ERR_UNSUPPORTED, "%s: a launch would exceed 2^32-1 work-items; use a smaller tile_rows", fn);
  if (!workspace || workspace_bytes < w->total)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes, got %zu", fn, w->total,
                workspace ? workspace_bytes : size_t(0));
  if (!aligned(workspace, 256)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  return LP_OK;
}

lp_status lp_lm_head_kl(const void* student_hidden, int64_t ld_hs, const void* student_weight, int64_t ld_ws,
                        int64_t h_student, const void* teacher_hidden, int64_t ld_ht, const void* teacher_weight,
                        int64_t ld_wt, int64_t h_teacher, int64_t T, int64_t V, const uint8_t* mask,
                        const int64_t* targets, const uint8_t* diff_mask, int64_t tile_rows, float* kl,
                        float* lp_student, float* lp_teacher, float* prob_diff, float* lse_student,
                        float* lse_teacher, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_lm_head_kl";
  lp::LMHeadWorkspace w;
  lp_status st = check_kl_heads(fn, student_hidden, ld_hs, student_weight, ld_ws, h_student, teacher_hidden, ld_ht,
                                teacher_weight, ld_wt, h_teacher, T, V, tile_rows, workspace, workspace_bytes, 0, &w);
  if (st != LP_OK) return st;
  if (!targets && (lp_student || lp_teacher || prob_diff))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: lp_student/lp_teacher/prob_diff need targets", fn);
  if (T == 0) return ok();
  if (!kl) return fail(LP_ERR_INVALID_ARGUMENT, "%s: kl is required", fn);
  if (targets && !aligned(targets, 8)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned targets", fn);
  if (!f32_aligned({kl, lp_student, lp_teacher, prob_diff, lse_student, lse_teacher}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned fp32 output", fn);
  const lp::LMHeadShape su = make_shape(student_hidden, ld_hs, student_weight, ld_ws, T, h_student, V, targets, 1,
                                        mask, 1.0f, tile_rows);
  const lp::LMHeadShape te = make_shape(teacher_hidden, ld_ht, teacher_weight, ld_wt, T, h_teacher, V, targets, 1,
                                        mask, 1.0f, tile_rows);
  const lp::KLHeadOutputs out{kl, lp_student, lp_teacher, prob_diff, lse_student, lse_teacher};
  clear_pending_hip_error();
  hipError_t e = lp::launch_lmhead_kl_forward(su, te, targets, diff_mask, out, static_cast<char*>(workspace), w,
                                              static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_lm_head_kl_backward(const void* student_hidden, int64_t ld_hs, const void* student_weight,
                                 int64_t ld_ws, int64_t h_student, const void* teacher_hidden, int64_t ld_ht,
                                 const void* teacher_weight, int64_t ld_wt, int64_t h_teacher, int64_t T, int64_t V,
                                 const uint8_t* mask, int64_t tile_rows, const float* lse_student,
                                 const float* lse_teacher, const float* grad_kl, float* grad_hidden,
                                 float* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_lm_head_kl_backward";
  lp::LMHeadWorkspace w;
  lp_status st = check_kl_heads(fn, student_hidden, ld_hs, student_weight, ld_ws, h_student, teacher_hidden, ld_ht,
                                teacher_weight, ld_wt, h_teacher, T, V, tile_rows, workspace, workspace_bytes, 1, &w);
  if (st != LP_OK) return st;
  if (!f32_aligned({lse_student, lse_teacher, grad_kl, grad_hidden, grad_weight}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned fp32 argument", fn);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0) {
    if (grad_weight) {
      clear_pending_hip_error();
      hipError_t e = lp::launch_zero_f32(grad_weight, V * h_student, s);
      if (e != hipSuccess) return hip_fail(e, fn);
    }
    return ok();
  }
  if (!lse_student || !lse_teacher || !grad_kl)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: lse_student, lse_teacher and grad_kl are required", fn);
  const lp::LMHeadShape su = make_shape(student_hidden, ld_hs, student_weight, ld_ws, T, h_student, V, nullptr, 1,
                                        mask, 1.0f, tile_rows);
  const lp::LMHeadShape te = make_shape(teacher_hidden, ld_ht, teacher_weight, ld_wt, T, h_teacher, V, nullptr, 1,
                                        mask, 1.0f, tile_rows);
  clear_pending_hip_error();
  hipError_t e = lp::launch_lmhead_kl_backward(su, te, lse_student, lse_teacher, grad_kl, grad_hidden, grad_weight,
                                               static_cast<char*>(workspace), w, s);
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_kl_full_vocab(const void* student, const void* teacher, lp_dtype dtype, int64_t T, int64_t V,
                           int64_t ld_s, int64_t ld_t, float* kl, const int64_t* targets,
                           const uint8_t* diff_mask, float* lp_student, float* lp_teacher, float* prob_diff,
                           void* stream) {
  const char* fn = "lp_kl_full_vocab";
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: dtype must be LP_BF16, LP_FP16 or LP_FP32", fn);
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  if (V <= 0 || V > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "%s: V out of range (1..2^30)", fn);
  if (ld_s < V || ld_t < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_s and ld_t must be >= V", fn);
  if (!targets && (lp_student || lp_teacher || prob_diff))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: lp_student/lp_teacher/prob_diff need targets", fn);
  if (T == 0) return ok();
  if (T > 0x7fffffff) return fail(LP_ERR_UNSUPPORTED, "%s: more than 2^31-1 rows", fn);
  if (!student || !teacher || !kl) return fail(LP_ERR_INVALID_ARGUMENT, "%s: student, teacher, kl required", fn);
  if (!aligned(student, dtype_bytes(dtype)) || !aligned(teacher, dtype_bytes(dtype)) ||
      (targets && !aligned(targets, 8)) || !f32_aligned({kl, lp_student, lp_teacher, prob_diff}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  lp::KLArgs a;
  a.student = student;
  a.teacher = teacher;
  a.ld_s = ld_s;
  a.ld_t = ld_t;
  a.V = static_cast<int>(V);
  a.T = T;
  a.row0 = 0;
  a.c = static_cast<float>(kLog2eD);
  a.kl = kl;
  a.targets = targets;
  a.diff_mask = diff_mask;
  a.lp_student = lp_student;
  a.lp_teacher = lp_teacher;
  a.prob_diff = prob_diff;
  clear_pending_hip_error();
  hipError_t e = lp::launch_kl_full_vocab(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_prob_diff(const float* lp_a, const float* lp_b, const uint8_t* mask, int64_t n, float* out,
                       void* stream) {
  if (n < 0) return fail(LP_ERR_INVALID_ARGUMENT, "lp_prob_diff: n < 0");
  if (n == 0) return ok();
  if (!lp_a || !lp_b || !out) return fail(LP_ERR_INVALID_ARGUMENT, "lp_prob_diff: lp_a, lp_b, out required");
  if (!f32_aligned({lp_a, lp_b, out})) return fail(LP_ERR_INVALID_ARGUMENT, "lp_prob_diff: misaligned pointer");
  clear_pending_hip_error();
  hipError_t e = lp::launch_prob_diff(lp_a, lp_b, mask, n, out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "lp_prob_diff");
  return ok();
}

size_t lp_prob_diff_stats_workspace_bytes(void) { return lp::prob_diff_stats_workspace_bytes(); }

lp_status lp_prob_diff_stats(const float* lp_a, const float* lp_b, const uint8_t* mask, int64_t n, double* out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_prob_diff_stats";
  if (n < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: n < 0", fn);
  if (!out) return fail(LP_ERR_INVALID_ARGUMENT, "%s: out is required", fn);
  if (n > 0 && (!lp_a || !lp_b)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: lp_a and lp_b are required", fn);
  if (!f32_aligned({lp_a, lp_b})) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned lp_a or lp_b", fn);
  if (!workspace || workspace_bytes < lp::prob_diff_stats_workspace_bytes())
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes", fn, lp::prob_diff_stats_workspace_bytes());
  if (!aligned(workspace, 256) || !aligned(out, 8))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned workspace or out", fn);
  clear_pending_hip_error();
  hipError_t e = lp::launch_prob_diff_stats(lp_a, lp_b, mask, n, out, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

// ---------------------------------------------------------------------------
// logit rules
// ---------------------------------------------------------------------------

static bool i32_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned(p, 4)) return false;
  return true;
}

// A row-major block in memory: `width` bytes of each of `rows` rows, `pitch`
// bytes apart.
struct Block {
  uintptr_t at;
  uint64_t rows, width, pitch;
  Block(const void* p, int64_t n, int64_t w, int64_t ld, size_t e)
      : at(reinterpret_cast<uintptr_t>(p)), rows(n), width(uint64_t(w) * e), pitch(uint64_t(ld) * e) {}
  Block(const void* p, int64_t n, size_t e) : Block(p, 1, n, n, e) {}
  uintptr_t end() const { return at + (rows - 1) * pitch + width; }
};

// Whether two blocks share bytes.  Address ranges that do not meet share none,
// and neither do rows of one pitch that lie beside each other; all else counts
// as shared.
static bool share_bytes(const Block& a, const Block& b) {
  if (a.at >= b.end() || b.at >= a.end()) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  // a single row may be taken at the other block's pitch
  const uint64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  if (b.rows > 1 && b.pitch != pitch) return true;
  const uint64_t apart = a.at < b.at ? (b.at - a.at) % pitch : (pitch - (a.at - b.at) % pitch) % pitch;
  return apart < a.width || apart + b.width > pitch;
}

// Checks shared by the calls under rules; fills the fields every one of them
// has.  T == 0 passes with nothing examined beyond the sizes.
static lp_status check_rules(const char* fn, const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                             const lp_logit_rules* rules, const uint8_t* mask, lp::RulesArgs* a) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  if (V <= 0 || V > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "%s: V out of range (1..2^30)", fn);
  if (ld < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld < V", fn);
  if (T > (int64_t(1) << 40) || ld > (int64_t(1) << 40) / (T > 0 ? T : 1))
    return fail(LP_ERR_UNSUPPORTED, "%s: T x ld past 2^40 elements", fn);
  memset(a, 0, sizeof(*a));
  a->x = logits;
  a->ld = ld;
  a->V = static_cast<int>(V);
  a->T = T;
  a->mask = mask;
  if (T == 0) return LP_OK;
  if (!logits) return fail(LP_ERR_INVALID_ARGUMENT, "%s: logits are required", fn);
  if (!aligned(logits, dtype_bytes(dtype))) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned logits", fn);
  if (!rules) return LP_OK;
  const lp_logit_rules& r = *rules;
  if (!i32_aligned({r.tokens, r.row_buffer, r.prompt_len, r.hist_len, r.repetition, r.frequency, r.presence,
                    r.bias_tokens, r.bias_values, r.allowed}) ||
      (r.bias_offsets && !aligned(r.bias_offsets, 8)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned rules array", fn);
  if (r.tokens) {
    if (!r.hist_len) return fail(LP_ERR_INVALID_ARGUMENT, "%s: tokens need hist_len", fn);
    if (r.buffers < 1 || r.max_len < 1 || r.buffers > 0x7fffffff || r.max_len > 0x7fffffff ||
        r.ld_tokens < r.max_len || r.ld_tokens > (int64_t(1) << 40) / r.buffers)
      return fail(LP_ERR_INVALID_ARGUMENT,
                  "%s: buffers and max_len must be in 1..2^31-1, ld_tokens >= max_len, the buffers below 2^40 tokens",
                  fn);
    if (!r.row_buffer && r.buffers < T)
      return fail(LP_ERR_INVALID_ARGUMENT, "%s: without row_buffer every row needs a buffer of its own", fn);
  } else if (r.repetition || r.frequency || r.presence) {
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: penalties need tokens and hist_len", fn);
  }
  if (r.bias_offsets) {
    if (r.bias_count < 0 || r.bias_count > 0x7fffffff)
      return fail(LP_ERR_INVALID_ARGUMENT, "%s: bias_count must be in 0..2^31-1", fn);
    if (r.bias_count > 0 && (!r.bias_tokens || !r.bias_values))
      return fail(LP_ERR_INVALID_ARGUMENT, "%s: biases need bias_tokens and bias_values", fn);
  } else if (r.bias_tokens || r.bias_values) {
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: biases need bias_offsets", fn);
  }
  if (r.allowed && r.ld_allowed < (V + 31) / 32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_allowed must be >= ceil(V / 32)", fn);
  // a history without any penalty changes nothing and is not read
  if (r.tokens && (r.repetition || r.frequency || r.presence)) {
    a->tokens = r.tokens;
    a->buffers = r.buffers;
    a->ld_tokens = r.ld_tokens;
    a->max_len = r.max_len;
    a->row_buffer = r.row_buffer;
    a->prompt_len = r.prompt_len;
    a->hist_len = r.hist_len;
    a->repetition = r.repetition;
    a->frequency = r.frequency;
    a->presence = r.presence;
  }
  if (r.bias_offsets && r.bias_count > 0) {
    a->bias_offsets = r.bias_offsets;
    a->bias_tokens = r.bias_tokens;
    a->bias_values = r.bias_values;
    a->bias_count = r.bias_count;
  }
  a->allowed = r.allowed;
  a->ld_allowed = r.ld_allowed;
  return LP_OK;
}

lp_status lp_process_logits(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                            const lp_logit_rules* rules, const uint8_t* mask, void* out, int64_t ld_out,
                            void* stream) {
  const char* fn = "lp_process_logits";
  lp::RulesArgs a;
  lp_status st = check_rules(fn, logits, dtype, T, V, ld, rules, mask, &a);
  if (st != LP_OK) return st;
  if (ld_out < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_out < V", fn);
  if (T == 0) return ok();
  if (ld_out > (int64_t(1) << 40) / T) return fail(LP_ERR_UNSUPPORTED, "%s: T x ld_out past 2^40 elements", fn);
  if (!out || !aligned(out, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: out is required and must be aligned", fn);
  const size_t e_bytes = dtype_bytes(dtype);
  if (!(out == logits && ld_out == ld) && share_bytes({logits, T, V, ld, e_bytes}, {out, T, V, ld_out, e_bytes}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: out overlaps the logits without being them", fn);
  a.out = out;
  a.ld_out = ld_out;
  clear_pending_hip_error();
  hipError_t e = lp::launch_process_logits(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

size_t lp_processed_workspace_bytes(int64_t T, int64_t V) {
  if (T < 0 || T > (int64_t(1) << 40) || V <= 0 || V > kMaxV) return 0;
  const size_t n = lp::processed_workspace_bytes(T, V);
  return n > 256 ? n : 256;
}

lp_status lp_processed_logprobs_entropy(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                        const lp_logit_rules* rules, const int64_t* targets, const uint8_t* mask,
                                        float temperature, float* logprob, float* entropy, float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_processed_logprobs_entropy";
  lp::RulesArgs a;
  lp_status st = check_rules(fn, logits, dtype, T, V, ld, rules, mask, &a);
  if (st != LP_OK) return st;
  if (!isfinite(temperature)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: temperature not finite", fn);
  if (T == 0) return ok();
  if (!targets || !logprob) return fail(LP_ERR_INVALID_ARGUMENT, "%s: targets and logprob are required", fn);
  if (!aligned(targets, 8) || !f32_aligned({logprob, entropy, lse}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t need = lp_processed_workspace_bytes(T, V);
  if (!workspace || workspace_bytes < need)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes, got %zu", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (!aligned(workspace, 256)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  a.targets = targets;
  a.c = exp2_scale(temperature);
  a.logprob = logprob;
  a.entropy_out = entropy;
  a.lse_out = lse;
  clear_pending_hip_error();
  hipError_t e = lp::launch_processed_score(static_cast<int>(dtype), a, static_cast<char*>(workspace),
                                            static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_processed_logprobs_entropy_backward(const void* logits, lp_dtype dtype, int64_t T, int64_t V,
                                                 int64_t ld, const lp_logit_rules* rules, const int64_t* targets,
                                                 const uint8_t* mask, float temperature, const float* lse,
                                                 const float* entropy, const float* grad_logprob,
                                                 const float* grad_entropy, void* grad_logits, int64_t ld_grad,
                                                 void* stream) {
  const char* fn = "lp_processed_logprobs_entropy_backward";
  lp::RulesArgs a;
  lp_status st = check_rules(fn, logits, dtype, T, V, ld, rules, mask, &a);
  if (st != LP_OK) return st;
  if (!isfinite(temperature)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: temperature not finite", fn);
  if (ld_grad < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_grad < V", fn);
  if (T == 0) return ok();
  if (ld_grad > (int64_t(1) << 40) / T) return fail(LP_ERR_UNSUPPORTED, "%s: T x ld_grad past 2^40 elements", fn);
  if (!targets || !lse || !grad_logprob || !grad_logits || (grad_entropy && !entropy))
    return fail(LP_ERR_INVALID_ARGUMENT,
                "%s: targets, lse, grad_logprob and grad_logits are required, and entropy with grad_entropy", fn);
  if (!aligned(targets, 8) || !f32_aligned({lse, entropy, grad_logprob, grad_entropy}) ||
      !aligned(grad_logits, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t e_bytes = dtype_bytes(dtype);
  if (share_bytes({logits, T, V, ld, e_bytes}, {grad_logits, T, V, ld_grad, e_bytes}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: grad_logits overlaps the logits", fn);
  a.targets = targets;
  a.c = exp2_scale(temperature);
  a.inv_tau = temperature_applies(temperature) ? 1.0f / temperature : 1.0f;
  a.lse = lse;
  a.entropy = entropy;
  a.grad_logprob = grad_logprob;
  a.grad_entropy = grad_entropy;
  a.out = grad_logits;
  a.ld_out = ld_grad;
  clear_pending_hip_error();
  hipError_t e = lp::launch_processed_grad(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------

static lp_status check_embedding(const char* fn, lp_dtype dtype, int64_t V, int64_t h, int64_t N, int64_t ld_a,
                                 int64_t ld_b, float scale) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
  if (N < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: N < 0", fn);
  if (V <= 0 || V > kMaxV || h <= 0 || h > kMaxV)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: h and V must be in 1..2^30", fn);
  if (ld_a < h || ld_b < h) return fail(LP_ERR_INVALID_ARGUMENT, "%s: leading dimensions must be >= h", fn);
  if (!isfinite(scale)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: scale not finite", fn);
  constexpr int64_t kMost = int64_t(1) << 60;
  if (ld_a > kMost / (N > V ? N : V) || ld_b > kMost / (N > V ? N : V))
    return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 elements", fn);
  return LP_OK;
}

lp_status lp_embedding(const void* weight, lp_dtype dtype, int64_t V, int64_t h, int64_t ld_w, const int64_t* tokens,
                       int64_t N, float scale, void* out, int64_t ld_out, void* stream) {
  const char* fn = "lp_embedding";
  lp_status st = check_embedding(fn, dtype, V, h, N, ld_w, ld_out, scale);
  if (st != LP_OK) return st;
  if (N == 0) return ok();
  if (!weight || !tokens || !out) return fail(LP_ERR_INVALID_ARGUMENT, "%s: weight, tokens and out are required", fn);
  if (!aligned(weight, dtype_bytes(dtype)) || !aligned(out, dtype_bytes(dtype)) || !aligned(tokens, 8))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t e_bytes = dtype_bytes(dtype);
  const Block written(out, N, h, ld_out, e_bytes);
  if (share_bytes(written, {weight, V, h, ld_w, e_bytes}) || share_bytes(written, {tokens, N, 8}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: out overlaps an input", fn);
  lp::EmbedArgs a;
  a.weight = weight;
  a.ld_w = ld_w;
  a.V = static_cast<int>(V);
  a.h = static_cast<int>(h);
  a.tokens = tokens;
  a.N = N;
  a.scale = scale;
  a.out = out;
  a.ld_out = ld_out;
  clear_pending_hip_error();
  hipError_t e = lp::launch_embedding(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

size_t lp_embedding_workspace_bytes(int64_t N, int64_t h, int64_t V) {
  lp::EmbedWorkspace w;
  return lp::embedding_workspace_layout(N, h, V, &w) ? w.total : 0;
}

lp_status lp_embedding_backward(const void* grad_out, lp_dtype dtype, int64_t N, int64_t h, int64_t ld_g,
                                const int64_t* tokens, int64_t V, float scale, int accumulate, float* grad_weight,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_embedding_backward";
  lp_status st = check_embedding(fn, dtype, V, h, N, ld_g, ld_g, scale);
  if (st != LP_OK) return st;
  lp::EmbedWorkspace w;
  if (!lp::embedding_workspace_layout(N, h, V, &w)) return fail(LP_ERR_UNSUPPORTED, "%s: more than 2^31-1 positions", fn);
  if (!grad_weight || (N > 0 && (!grad_out || !tokens)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: grad_out, tokens and grad_weight are required", fn);
  if (!aligned(grad_out, dtype_bytes(dtype)) || !aligned(grad_weight, 4) || !aligned(tokens, 8))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {
    // no positions: the gradient is still defined
    if (accumulate) return ok();
    clear_pending_hip_error();
    hipError_t e = lp::launch_zero_f32(grad_weight, V * h, s);
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
  }
  if (!workspace || workspace_bytes < w.total)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes, got %zu", fn, w.total,
                workspace ? workspace_bytes : size_t(0));
  if (!aligned(workspace, 256)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  const Block gradient(grad_weight, V * h, 4), scratch(workspace, static_cast<int64_t>(w.total), 1);
  const Block grads(grad_out, N, h, ld_g, dtype_bytes(dtype)), ids(tokens, N, 8);
  if (share_bytes(gradient, grads) || share_bytes(gradient, ids) || share_bytes(gradient, scratch) ||
      share_bytes(scratch, grads) || share_bytes(scratch, ids))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: grad_weight or the workspace overlaps an operand", fn);
  lp::EmbedGradArgs a;
  memset(&a, 0, sizeof(a));
  a.grad = grad_out;
  a.ld_g = ld_g;
  a.N = N;
  a.h = static_cast<int>(h);
  a.V = static_cast<int>(V);
  a.tokens = tokens;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  a.grad_weight = grad_weight;
  clear_pending_hip_error();
  hipError_t e = lp::launch_embedding_backward(static_cast<int>(dtype), a, static_cast<char*>(workspace), w, s);
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

// ---------------------------------------------------------------------------
// 4-bit head
// ---------------------------------------------------------------------------

static lp_status check_w4(const char* fn, int64_t V, int64_t h, int64_t group, const void* packed, int64_t ld_packed,
                          const void* scales, int64_t ld_scales) {
  if (V <= 0 || V > kMaxV || h <= 0 || h > kMaxV)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: h and V must be in 1..2^30", fn);
  if (h % 32) return fail(LP_ERR_UNSUPPORTED, "%s: h must be a multiple of 32", fn);
  if (group != 32 && group != 64 && group != 128)
    return fail(LP_ERR_UNSUPPORTED, "%s: group must be 32, 64 or 128", fn);
  if (ld_packed < h / 2 || ld_scales < (h + group - 1) / group)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_packed must be >= h / 2 and ld_scales >= ceil(h / group)", fn);
  if (ld_packed > (int64_t(1) << 60) / V || ld_scales > (int64_t(1) << 60) / V)
    return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 bytes", fn);
  if (ld_packed % 16) return fail(LP_ERR_UNSUPPORTED, "%s: ld_packed must be a multiple of 16", fn);
  if (!packed || !scales) return fail(LP_ERR_INVALID_ARGUMENT, "%s: packed and scales are required", fn);
  if (!aligned(packed, 16)) return fail(LP_ERR_UNSUPPORTED, "%s: packed must be 16-byte aligned", fn);
  if (!aligned(scales, 2)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned scales", fn);
  return LP_OK;
}

lp_status lp_lm_head_w4_quantize(const void* weight, lp_dtype dtype, int64_t V, int64_t h, int64_t ld_w,
                                 int64_t group, void* packed, int64_t ld_packed, void* scales, int64_t ld_scales,
                                 void* stream) {
  const char* fn = "lp_lm_head_w4_quantize";
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
  lp_status st = check_w4(fn, V, h, group, packed, ld_packed, scales, ld_scales);
  if (st != LP_OK) return st;
  if (ld_w < h) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_w < h", fn);
  if (ld_w > (int64_t(1) << 59) / V) return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 bytes", fn);
  if (!weight || !aligned(weight, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: weight is required and must be aligned", fn);
  const Block dense(weight, V, h, ld_w, dtype_bytes(dtype)), head(packed, V, h / 2, ld_packed, 1);
  const Block steps(scales, V, (h + group - 1) / group, ld_scales, 2);
  if (share_bytes(dense, head) || share_bytes(dense, steps) || share_bytes(head, steps))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: weight, packed and scales overlap", fn);
  lp::W4QuantArgs a;
  a.weight = weight;
  a.ld_w = ld_w;
  a.V = static_cast<int>(V);
  a.h = static_cast<int>(h);
  a.group = static_cast<int>(group);
  a.groups = static_cast<int>((h + group - 1) / group);
  a.packed = packed;
  a.ld_p = ld_packed;
  a.scales = static_cast<uint16_t*>(scales);
  a.ld_s = ld_scales;
  clear_pending_hip_error();
  hipError_t e = lp::launch_w4_quantize(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_lm_head_w4_logits(const void* hidden, lp_dtype dtype, int64_t T, int64_t h, int64_t ld_h,
                               const void* packed, int64_t ld_packed, const void* scales, int64_t ld_scales, int64_t V,
                               int64_t group, void* out, lp_dtype out_dtype, int64_t ld_out, void* stream) {
  const char* fn = "lp_lm_head_w4_logits";
  if (dtype == LP_FP32) return fail(LP_ERR_UNSUPPORTED, "%s: hidden must be bf16 or fp16", fn);
  if ((dtype != LP_BF16 && dtype != LP_FP16) ||
      (out_dtype != LP_BF16 && out_dtype != LP_FP16 && out_dtype != LP_FP32))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d or %d", fn, static_cast<int>(dtype),
                static_cast<int>(out_dtype));
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  lp_status st = check_w4(fn, V, h, group, packed, ld_packed, scales, ld_scales);
  if (st != LP_OK) return st;
  if (ld_h < h || ld_out < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_h must be >= h and ld_out >= V", fn);
  if (ld_h % 8) return fail(LP_ERR_UNSUPPORTED, "%s: ld_h must be a multiple of 8", fn);
  if (T == 0) return ok();
  if (T > (int64_t(1) << 40) || ld_h > (int64_t(1) << 59) / T || ld_out > (int64_t(1) << 59) / T)
    return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 bytes", fn);
  if (!hidden || !out) return fail(LP_ERR_INVALID_ARGUMENT, "%s: hidden and out are required", fn);
  if (!aligned(hidden, 16)) return fail(LP_ERR_UNSUPPORTED, "%s: hidden must be 16-byte aligned", fn);
  if (!aligned(out, dtype_bytes(out_dtype))) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned out", fn);
  const Block written(out, T, V, ld_out, dtype_bytes(out_dtype));
  if (share_bytes(written, {hidden, T, h, ld_h, 2}) || share_bytes(written, {packed, V, h / 2, ld_packed, 1}) ||
      share_bytes(written, {scales, V, (h + group - 1) / group, ld_scales, 2}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: out overlaps an input", fn);
  lp::W4Args a;
  a.hidden = static_cast<const uint16_t*>(hidden);
  a.ld_h = ld_h;
  a.T = T;
  a.h = static_cast<int>(h);
  a.V = static_cast<int>(V);
  a.group = static_cast<int>(group);
  a.packed = packed;
  a.ld_p = ld_packed;
  a.scales = static_cast<const uint16_t*>(scales);
  a.ld_s = ld_scales;
  a.out = out;
  a.out_dtype = static_cast<int>(out_dtype);
  a.ld_out = ld_out;
  clear_pending_hip_error();
  hipError_t e = lp::launch_w4_logits(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

// ---------------------------------------------------------------------------
// the largest logits, distillation from them, beams
// ---------------------------------------------------------------------------

// Checks of T rows of V logits and a temperature that the calls below share.
static lp_status check_rows(const char* fn, const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                            float temperature) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  if (V <= 0 || V > kMaxV) return fail(LP_ERR_INVALID_ARGUMENT, "%s: V out of range (1..2^30)", fn);
  if (ld < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld < V", fn);
  if (T > (int64_t(1) << 40) || ld > (int64_t(1) << 40) / (T > 0 ? T : 1))
    return fail(LP_ERR_UNSUPPORTED, "%s: T x ld past 2^40 elements", fn);
  if (!isfinite(temperature)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: temperature not finite", fn);
  if (T == 0) return LP_OK;
  if (!logits || !aligned(logits, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: logits are required and must be aligned", fn);
  return LP_OK;
}

static double inverse(float temperature) {
  return temperature_applies(temperature) ? 1.0 / static_cast<double>(temperature) : 1.0;
}

static lp_status check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need)
    return fail(LP_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %zu bytes, got %zu", fn, need,
                workspace ? bytes : size_t(0));
  if (!aligned(workspace, 256)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  return LP_OK;
}

// True if nothing written shares bytes with anything read or written besides
// (NULL blocks aside).
static bool apart(std::initializer_list<Block> written, std::initializer_list<Block> read) {
  for (const Block* w = written.begin(); w != written.end(); ++w) {
    if (!w->at) continue;
    for (const Block* o = w + 1; o != written.end(); ++o)
      if (o->at && share_bytes(*w, *o)) return false;
    for (const Block& o : read)
      if (o.at && share_bytes(*w, o)) return false;
  }
  return true;
}

static int64_t bytes_of(size_t n) { return static_cast<int64_t>(n); }

size_t lp_top_workspace_bytes(lp_dtype dtype, int64_t T, int64_t V, int64_t K) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32) return 0;
  if (T < 0 || T > (int64_t(1) << 40) || V <= 0 || V > kMaxV || K < 1 || K > lp::kMaxTop || K > V) return 0;
  const size_t n = lp::top_workspace_bytes(static_cast<int>(dtype), T, V, K);
  return n > 256 ? n : 256;
}

lp_status lp_top_logits(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld, int64_t K,
                        const uint8_t* mask, float temperature, int64_t* ids, float* logprob, float* rest,
                        float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_top_logits";
  lp_status st = check_rows(fn, logits, dtype, T, V, ld, temperature);
  if (st != LP_OK) return st;
  if (K < 1 || K > lp::kMaxTop || K > V)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: K must be in 1..min(V, %d)", fn, lp::kMaxTop);
  if (T == 0) return ok();
  if (!ids || !logprob) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ids and logprob are required", fn);
  if (!aligned(ids, 8) || !f32_aligned({logprob, rest, lse}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t need = lp_top_workspace_bytes(dtype, T, V, K);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != LP_OK) return st;
  if (!apart({{ids, T * K, 8}, {logprob, T * K, 4}, {rest, T, 4}, {lse, T, 4}, {workspace, bytes_of(need), 1}},
             {{logits, T, V, ld, dtype_bytes(dtype)}, {mask, T, 1}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: an output or the workspace overlaps an operand", fn);
  lp::TopArgs a;
  memset(&a, 0, sizeof(a));
  a.x = logits;
  a.ld = ld;
  a.V = static_cast<int>(V);
  a.T = T;
  a.K = static_cast<int>(K);
  a.mask = mask;
  a.c = exp2_scale(temperature);
  a.inv_tau = inverse(temperature);
  a.ids = ids;
  a.logprob = logprob;
  a.rest = rest;
  a.lse = lse;
  clear_pending_hip_error();
  hipError_t e = lp::launch_top_logits(static_cast<int>(dtype), a, static_cast<char*>(workspace),
                                       static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

static lp_status check_distill(const char* fn, const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld,
                               int64_t K, const int64_t* teacher_ids, const float* teacher_logprob,
                               const float* teacher_rest, const uint8_t* mask, float temperature,
                               lp::DistillArgs* a) {
  lp_status st = check_rows(fn, logits, dtype, T, V, ld, temperature);
  if (st != LP_OK) return st;
  if (K < 1 || K > lp::kMaxTop) return fail(LP_ERR_INVALID_ARGUMENT, "%s: K must be in 1..%d", fn, lp::kMaxTop);
  memset(a, 0, sizeof(*a));
  if (T == 0) return LP_OK;
  if (!teacher_ids || !teacher_logprob)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: teacher_ids and teacher_logprob are required", fn);
  if (!aligned(teacher_ids, 8) || !f32_aligned({teacher_logprob, teacher_rest}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  a->x = logits;
  a->ld = ld;
  a->V = static_cast<int>(V);
  a->T = T;
  a->K = static_cast<int>(K);
  a->ids = teacher_ids;
  a->logprob = teacher_logprob;
  a->rest = teacher_rest;
  a->mask = mask;
  a->c = exp2_scale(temperature);
  a->inv_tau = inverse(temperature);
  return LP_OK;
}

size_t lp_distill_top_workspace_bytes(lp_dtype dtype, int64_t T, int64_t V) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32) return 0;
  if (T < 0 || T > (int64_t(1) << 40) || V <= 0 || V > kMaxV) return 0;
  const size_t n = lp::distill_workspace_bytes(static_cast<int>(dtype), T, V);
  return n > 256 ? n : 256;
}

lp_status lp_distill_top(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld, int64_t K,
                         const int64_t* teacher_ids, const float* teacher_logprob, const float* teacher_rest,
                         const uint8_t* mask, float temperature, float* loss, float* lse, float* lse_rest,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "lp_distill_top";
  lp::DistillArgs a;
  lp_status st = check_distill(fn, logits, dtype, T, V, ld, K, teacher_ids, teacher_logprob, teacher_rest, mask,
                               temperature, &a);
  if (st != LP_OK) return st;
  if (T == 0) return ok();
  if (!loss) return fail(LP_ERR_INVALID_ARGUMENT, "%s: loss is required", fn);
  if (!f32_aligned({loss, lse, lse_rest})) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t need = lp_distill_top_workspace_bytes(dtype, T, V);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != LP_OK) return st;
  if (!apart({{loss, T, 4}, {lse, T, 4}, {lse_rest, T, 4}, {workspace, bytes_of(need), 1}},
             {{logits, T, V, ld, dtype_bytes(dtype)}, {teacher_ids, T * K, 8}, {teacher_logprob, T * K, 4},
              {teacher_rest, T, 4}, {mask, T, 1}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: an output or the workspace overlaps an operand", fn);
  a.loss = loss;
  a.lse_out = lse;
  a.lse_rest_out = lse_rest;
  clear_pending_hip_error();
  hipError_t e = lp::launch_distill(static_cast<int>(dtype), a, static_cast<char*>(workspace),
                                    static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_distill_top_backward(const void* logits, lp_dtype dtype, int64_t T, int64_t V, int64_t ld, int64_t K,
                                  const int64_t* teacher_ids, const float* teacher_logprob,
                                  const float* teacher_rest, const uint8_t* mask, float temperature,
                                  const float* lse, const float* lse_rest, const float* grad_loss,
                                  void* grad_logits, int64_t ld_grad, void* stream) {
  const char* fn = "lp_distill_top_backward";
  lp::DistillArgs a;
  lp_status st = check_distill(fn, logits, dtype, T, V, ld, K, teacher_ids, teacher_logprob, teacher_rest, mask,
                               temperature, &a);
  if (st != LP_OK) return st;
  if (ld_grad < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_grad < V", fn);
  if (T == 0) return ok();
  if (ld_grad > (int64_t(1) << 40) / T) return fail(LP_ERR_UNSUPPORTED, "%s: T x ld_grad past 2^40 elements", fn);
  if (!lse || !lse_rest || !grad_loss || !grad_logits)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: lse, lse_rest, grad_loss and grad_logits are required", fn);
  if (!f32_aligned({lse, lse_rest, grad_loss}) || !aligned(grad_logits, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t e_bytes = dtype_bytes(dtype);
  if (!apart({{grad_logits, T, V, ld_grad, e_bytes}},
             {{logits, T, V, ld, e_bytes}, {teacher_ids, T * K, 8}, {teacher_logprob, T * K, 4}, {teacher_rest, T, 4},
              {mask, T, 1}, {lse, T, 4}, {lse_rest, T, 4}, {grad_loss, T, 4}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: grad_logits overlaps an operand", fn);
  a.lse = lse;
  a.lse_rest = lse_rest;
  a.grad_loss = grad_loss;
  a.out = grad_logits;
  a.ld_out = ld_grad;
  clear_pending_hip_error();
  hipError_t e = lp::launch_distill_grad(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

static bool beam_sizes(int64_t B, int64_t W, int64_t N) {
  return B >= 0 && B <= (int64_t(1) << 34) && W >= 1 && W <= lp::kMaxBeams && N >= 1 && N <= lp::kMaxTop &&
         W * N <= lp::kMaxBeamLists;
}

size_t lp_beam_workspace_bytes(lp_dtype dtype, int64_t B, int64_t W, int64_t V, int64_t N) {
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32) return 0;
  if (!beam_sizes(B, W, N) || V <= 0 || V > kMaxV) return 0;
  const size_t n = lp::beam_workspace_bytes(static_cast<int>(dtype), B, W, V, N);
  return n > 256 ? n : 256;
}

lp_status lp_beam_select(const void* logits, lp_dtype dtype, int64_t B, int64_t W, int64_t V, int64_t ld,
                         const float* beam_scores, const uint8_t* finished, int64_t N, int64_t end_token,
                         float temperature, float* scores, int32_t* parents, int64_t* tokens, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const char* fn = "lp_beam_select";
  if (!beam_sizes(B, W, N))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: B in 0..2^34, W in 1..%d, N in 1..%d, W N up to %d", fn, lp::kMaxBeams,
                lp::kMaxTop, lp::kMaxBeamLists);
  lp_status st = check_rows(fn, logits, dtype, B * W, V, ld, temperature);
  if (st != LP_OK) return st;
  if (end_token < 0 || end_token >= V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: end_token must be in 0..V-1", fn);
  if (B == 0) return ok();
  if (!beam_scores || !scores || !parents || !tokens)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: beam_scores, scores, parents and tokens are required", fn);
  if (!f32_aligned({beam_scores, scores}) || !aligned(parents, 4) || !aligned(tokens, 8))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", fn);
  const size_t need = lp_beam_workspace_bytes(dtype, B, W, V, N);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != LP_OK) return st;
  if (!apart({{scores, B * N, 4}, {parents, B * N, 4}, {tokens, B * N, 8}, {workspace, bytes_of(need), 1}},
             {{logits, B * W, V, ld, dtype_bytes(dtype)}, {beam_scores, B * W, 4}, {finished, B * W, 1}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: an output or the workspace overlaps an operand", fn);
  lp::TopArgs a;
  memset(&a, 0, sizeof(a));
  a.x = logits;
  a.ld = ld;
  a.V = static_cast<int>(V);
  a.T = B * W;
  a.K = static_cast<int>(N);
  a.W = static_cast<int>(W);
  a.c = exp2_scale(temperature);
  a.inv_tau = inverse(temperature);
  a.beam_scores = beam_scores;
  a.finished = finished;
  a.end_token = end_token;
  a.scores = scores;
  a.parents = parents;
  a.ids = tokens;
  clear_pending_hip_error();
  hipError_t e = lp::launch_beam_select(static_cast<int>(dtype), a, B, static_cast<char*>(workspace),
                                        static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

lp_status lp_beam_reorder(const void* src, int64_t src_outer, int64_t src_row, int64_t src_mid, int64_t outer,
                          int64_t mid, int64_t width, const int32_t* parents, int64_t B, int64_t W, int64_t N,
                          void* dst, int64_t dst_outer, int64_t dst_row, int64_t dst_mid, void* stream) {
  const char* fn = "lp_beam_reorder";
  constexpr int64_t kMost = int64_t(1) << 40;  // bytes of a stride or a width; the products below stay in 64 bits
  if (W < 1 || W > lp::kMaxTop || N < 1 || N > lp::kMaxTop)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: W and N must be in 1..%d", fn, lp::kMaxTop);
  if (B < 0 || outer < 0 || mid < 0 || width < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: a negative size", fn);
  for (int64_t x : {src_outer, src_row, src_mid, dst_outer, dst_row, dst_mid, width})
    if (x < 0 || x > kMost) return fail(LP_ERR_INVALID_ARGUMENT, "%s: strides and width must be in 0..2^40 bytes", fn);
  if (B == 0 || outer == 0 || mid == 0 || width == 0) return ok();
  constexpr int64_t kSegs = 0x7fffffff;
  if (B > kSegs || mid > kSegs || outer > kSegs || B > kSegs / mid || B * mid > kSegs / outer)
    return fail(LP_ERR_UNSUPPORTED, "%s: more than 2^31-1 of B x mid x outer", fn);
  if (!src || !dst || !parents) return fail(LP_ERR_INVALID_ARGUMENT, "%s: src, dst and parents are required", fn);
  if (!aligned(parents, 4)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned parents", fn);
  // sizes are below 2^40 and 2^31 each: whole extents as doubles, where a
  // rounding does not matter, before they are formed
  auto extent = [&](int64_t o, int64_t row, int64_t rows, int64_t m) {
    return static_cast<double>(outer) * o + static_cast<double>(rows) * row + static_cast<double>(mid) * m + width;
  };
  if (extent(src_outer, src_row, B * W, src_mid) > 1e18 || extent(dst_outer, dst_row, B * N, dst_mid) > 1e18)
    return fail(LP_ERR_UNSUPPORTED, "%s: states past 10^18 bytes", fn);
  const int64_t part = (mid - 1) * dst_mid + width, rows = (B * N - 1) * dst_row + part;
  if ((mid > 1 && dst_mid < width) || (B * N > 1 && dst_row < part) || (outer > 1 && dst_outer < rows))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: the strides of dst must be nested: width, mid, row, outer", fn);
  const Block from(src, (outer - 1) * src_outer + (B * W - 1) * src_row + (mid - 1) * src_mid + width, 1);
  if (!apart({{dst, (outer - 1) * dst_outer + rows, 1}}, {from, {parents, B * N, 4}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: dst overlaps src or parents", fn);
  lp::ReorderArgs a;
  memset(&a, 0, sizeof(a));
  a.src = src;
  a.dst = dst;
  a.outer = outer;
  a.mid = mid;
  a.width = width;
  a.src_outer = outer > 1 ? src_outer : 0;
  a.src_row = B * W > 1 ? src_row : 0;
  a.src_mid = mid > 1 ? src_mid : 0;
  a.dst_outer = outer > 1 ? dst_outer : 0;
  a.dst_row = B * N > 1 ? dst_row : 0;
  a.dst_mid = mid > 1 ? dst_mid : 0;
  a.B = B;
  a.W = static_cast<int>(W);
  a.N = static_cast<int>(N);
  a.parents = parents;
  if (!lp::beam_reorder_fits(a)) return fail(LP_ERR_UNSUPPORTED, "%s: rows too long for one launch", fn);
  clear_pending_hip_error();
  hipError_t e = lp::launch_beam_reorder(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

// ---------------------------------------------------------------------------
// 8-bit head
// ---------------------------------------------------------------------------

constexpr int64_t kMaxFp8H = int64_t(1) << 20, kMaxFp8Pitch = int64_t(1) << 23;

static lp_status check_fp8(const char* fn, int64_t V, int64_t h, const void* q, int64_t ld_q, const float* scales,
                           int64_t ld_scales) {
  if (V <= 0 || V > kMaxV || h <= 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: h >= 1 and V in 1..2^30", fn);
  if (h % 16 || h > kMaxFp8H) return fail(LP_ERR_UNSUPPORTED, "%s: h must be a multiple of 16 up to 2^20", fn);
  if (ld_q < h || ld_scales < (h + 127) / 128)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_q must be >= h and ld_scales >= ceil(h / 128)", fn);
  if (ld_q % 16 || ld_q > kMaxFp8Pitch)
    return fail(LP_ERR_UNSUPPORTED, "%s: ld_q must be a multiple of 16 up to 2^23", fn);
  if (ld_scales > (int64_t(1) << 58) / V) return fail(LP_ERR_UNSUPPORTED, "%s: scales past 2^60 bytes", fn);
  if (!q || !scales) return fail(LP_ERR_INVALID_ARGUMENT, "%s: q and scales are required", fn);
  if (!aligned(q, 16)) return fail(LP_ERR_UNSUPPORTED, "%s: q must be 16-byte aligned", fn);
  if (!aligned(scales, 4)) return fail(LP_ERR_INVALID_ARGUMENT, "%s: misaligned scales", fn);
  return LP_OK;
}

lp_status lp_lm_head_fp8_quantize(const void* weight, lp_dtype dtype, int64_t V, int64_t h, int64_t ld_w, void* q,
                                  int64_t ld_q, float* scales, int64_t ld_scales, void* stream) {
  const char* fn = "lp_lm_head_fp8_quantize";
  if (dtype != LP_BF16 && dtype != LP_FP16 && dtype != LP_FP32)
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
  lp_status st = check_fp8(fn, V, h, q, ld_q, scales, ld_scales);
  if (st != LP_OK) return st;
  if (ld_w < h) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_w < h", fn);
  if (ld_w > (int64_t(1) << 58) / V) return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 bytes", fn);
  if (!weight || !aligned(weight, dtype_bytes(dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: weight is required and must be aligned", fn);
  if (!apart({{q, V, h, ld_q, 1}, {scales, (V + 127) / 128, (h + 127) / 128, ld_scales, 4}},
             {{weight, V, h, ld_w, dtype_bytes(dtype)}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: weight, q and scales overlap", fn);
  lp::Fp8QuantArgs a;
  a.weight = weight;
  a.ld_w = ld_w;
  a.V = static_cast<int>(V);
  a.h = static_cast<int>(h);
  a.q = static_cast<uint8_t*>(q);
  a.ld_q = ld_q;
  a.scales = scales;
  a.ld_s = ld_scales;
  clear_pending_hip_error();
  hipError_t e = lp::launch_fp8_quantize(static_cast<int>(dtype), a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

size_t lp_lm_head_fp8_workspace_bytes(int64_t T, int64_t h, int64_t V) {
  if (T < 0 || T > (int64_t(1) << 36) || V <= 0 || V > kMaxV || h <= 0 || h % 16 || h > kMaxFp8H) return 0;
  const size_t n = lp::fp8_workspace_bytes(T, h, V);
  return n > 256 ? n : 256;
}

lp_status lp_lm_head_fp8_logits(const void* hidden, lp_dtype dtype, int64_t T, int64_t h, int64_t ld_h, const void* q,
                                int64_t ld_q, const float* scales, int64_t ld_scales, int64_t V, void* out,
                                lp_dtype out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const char* fn = "lp_lm_head_fp8_logits";
  if (dtype == LP_FP32) return fail(LP_ERR_UNSUPPORTED, "%s: hidden must be bf16 or fp16", fn);
  if ((dtype != LP_BF16 && dtype != LP_FP16) ||
      (out_dtype != LP_BF16 && out_dtype != LP_FP16 && out_dtype != LP_FP32))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d or %d", fn, static_cast<int>(dtype),
                static_cast<int>(out_dtype));
  if (T < 0) return fail(LP_ERR_INVALID_ARGUMENT, "%s: T < 0", fn);
  lp_status st = check_fp8(fn, V, h, q, ld_q, scales, ld_scales);
  if (st != LP_OK) return st;
  if (ld_h < h || ld_out < V) return fail(LP_ERR_INVALID_ARGUMENT, "%s: ld_h must be >= h and ld_out >= V", fn);
  if (T == 0) return ok();
  if (T > (int64_t(1) << 36) || ld_h > (int64_t(1) << 58) / T || ld_out > (int64_t(1) << 58) / T)
    return fail(LP_ERR_UNSUPPORTED, "%s: operands past 2^60 bytes", fn);
  if (!hidden || !out || !aligned(hidden, 2) || !aligned(out, dtype_bytes(out_dtype)))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: hidden and out are required and must be aligned", fn);
  const size_t need = lp_lm_head_fp8_workspace_bytes(T, h, V);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != LP_OK) return st;
  if (!apart({{out, T, V, ld_out, dtype_bytes(out_dtype)}, {workspace, bytes_of(need), 1}},
             {{hidden, T, h, ld_h, 2}, {q, V, h, ld_q, 1}, {scales, (V + 127) / 128, (h + 127) / 128, ld_scales, 4}}))
    return fail(LP_ERR_INVALID_ARGUMENT, "%s: out or the workspace overlaps an operand", fn);
  lp::Fp8Args a;
  a.hidden = static_cast<const uint16_t*>(hidden);
  a.ld_h = ld_h;
  a.T = T;
  a.h = static_cast<int>(h);
  a.V = static_cast<int>(V);
  a.weight = static_cast<const uint8_t*>(q);
  a.ld_w = ld_q;
  a.scales = scales;
  a.ld_s = ld_scales;
  a.out = out;
  a.out_dtype = static_cast<int>(out_dtype);
  a.ld_out = ld_out;
  clear_pending_hip_error();
  hipError_t e = lp::launch_fp8_logits(static_cast<int>(dtype), a, static_cast<char*>(workspace),
                                       static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, fn);
  return ok();
}

}  // extern "C"
