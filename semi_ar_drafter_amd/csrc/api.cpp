// C ABI of libdspark (declared in include/dspark.h): host-side argument
// validation, workspace sizing, status reporting and dispatch to the HIP
// launchers.  Every check runs before anything is enqueued, so argument
// errors are reported synchronously and without touching the GPU.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/dspark.h"
#include "launch.h"

namespace {

thread_local char g_last_error[512] = "";

dspark_status fail(dspark_status s, const char* fmt, const char* detail = nullptr) {
  if (detail)
    std::snprintf(g_last_error, sizeof g_last_error, fmt, detail);
  else
    std::snprintf(g_last_error, sizeof g_last_error, "%s", fmt);
  return s;
}

dspark_status hip_fail(hipError_t e) {
  std::snprintf(g_last_error, sizeof g_last_error, "HIP error %d: %s", int(e), hipGetErrorString(e));
  return DSPARK_ERR_HIP;
}

std::atomic<int> g_draft_launch{DSPARK_LAUNCH_COOPERATIVE};

constexpr int kMaxGamma = 64;
constexpr int kMaxD = 65536;
constexpr int kMaxV = 1 << 24;

}  // namespace

extern "C" {

const char* dspark_status_string(dspark_status s) {
  switch (s) {
    case DSPARK_OK: return "ok";
    case DSPARK_ERR_INVALID_ARG: return "invalid argument";
    case DSPARK_ERR_UNSUPPORTED: return "unsupported shape or type";
    case DSPARK_ERR_WORKSPACE: return "workspace missing, too small or misaligned";
    case DSPARK_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

const char* dspark_last_error(void) { return g_last_error; }

dspark_status dspark_set_draft_launch(dspark_launch mode) {
  g_last_error[0] = '\0';
  if (mode != DSPARK_LAUNCH_COOPERATIVE && mode != DSPARK_LAUNCH_EXCLUSIVE)
    return fail(DSPARK_ERR_INVALID_ARG, "unknown launch mode");
  g_draft_launch.store(int(mode));
  return DSPARK_OK;
}

dspark_launch dspark_get_draft_launch(void) { return dspark_launch(g_draft_launch.load()); }

size_t dspark_draft_workspace_bytes(int B, int gamma, int V, int r) {
  (void)V;
  (void)r;
  if (B <= 0 || gamma <= 0) return 0;
  return dspark::draft_workspace_layout(B, gamma, 0).total;
}

size_t dspark_serve_workspace_bytes(int B, int gamma, int V, int r) {
  const size_t draft = dspark_draft_workspace_bytes(B, gamma, V, r);
  if (draft == 0) return 0;
  return draft + dspark::schedule_workspace_bytes(B, gamma);
}

size_t dspark_rnn_draft_workspace_bytes(int B, int gamma, int V, int r) {
  (void)V;
  if (B <= 0 || gamma <= 0 || r <= 0) return 0;
  return dspark::draft_workspace_layout(B, gamma, r).total;
}

namespace {

// Shared by the Markov-head and RNN-head entry points (decay == nullptr: Markov).
dspark_status draft_impl(int B, int gamma, int V, int r, int d, dspark_dtype dtype, const int32_t* anchor,
                         const void* U, const void* h, const void* W1, const void* W2, const float* decay,
                         bool rnn, const float* conf_w, float conf_b, const float* sts_T, dspark_sampling mode,
                         uint64_t seed, int32_t* tokens, float* logit, float* conf, float* surv, void* workspace,
                         size_t workspace_bytes, hipStream_t stream, bool noalloc = false,
                         const dspark::StepArgs* step = nullptr, bool* fused = nullptr, bool check_only = false) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0 || V < 0 || r < 0 || d < 0)
    return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (mode != DSPARK_GREEDY && mode != DSPARK_GUMBEL) return fail(DSPARK_ERR_INVALID_ARG, "unknown sampling mode");
  if (rnn && dtype != DSPARK_BF16) return fail(DSPARK_ERR_UNSUPPORTED, "the RNN head needs bf16 storage");
  if (B == 0 || gamma == 0) return DSPARK_OK;
  if (V < 1 || r < 1) return fail(DSPARK_ERR_INVALID_ARG, "V and r must be positive");
  if (!anchor || !U || !W1 || !W2 || !conf_w || !sts_T || !tokens || !logit || !conf || !surv ||
      (d > 0 && !h) || (rnn && !decay))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (gamma > kMaxGamma) return fail(DSPARK_ERR_UNSUPPORTED, "gamma > 64");
  if (d > kMaxD) return fail(DSPARK_ERR_UNSUPPORTED, "d > 65536");
  if (V > kMaxV) return fail(DSPARK_ERR_UNSUPPORTED, "V > 2^24");
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(W1) % 16 || reinterpret_cast<uintptr_t>(U) % elem ||
      reinterpret_cast<uintptr_t>(W2) % elem || (h && reinterpret_cast<uintptr_t>(h) % elem) ||
      (rnn && reinterpret_cast<uintptr_t>(decay) % 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor (W1 needs 16-byte alignment)");
  const size_t need = rnn ? dspark_rnn_draft_workspace_bytes(B, gamma, V, r) : dspark_draft_workspace_bytes(B, gamma, V, r);
  if (noalloc) {
    // allocation-free entry point: the launcher takes the static per-device
    // scratch in place of a workspace, once every check has passed
    if (need > dspark::kNoAllocScratchBytes)
      return fail(DSPARK_ERR_UNSUPPORTED, "shape needs more workspace than the 8 MiB static scratch");
  } else if (!workspace || workspace_bytes < need)
    return fail(DSPARK_ERR_WORKSPACE, rnn ? "workspace missing or smaller than dspark_rnn_draft_workspace_bytes()"
                                          : "workspace missing or smaller than dspark_draft_workspace_bytes()");
  if (!noalloc && reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(DSPARK_ERR_WORKSPACE, "workspace not 256-byte aligned");

  dspark::DraftArgs a;
  a.B = B;
  a.gamma = gamma;
  a.V = V;
  a.r = r;
  a.d = d;
  a.bf16 = dtype == DSPARK_BF16;
  a.gumbel = mode == DSPARK_GUMBEL;
  a.seed = seed;
  a.anchor = anchor;
  a.U = U;
  a.h = h;
  a.W1 = W1;
  a.W2 = W2;
  a.conf_w = conf_w;
  a.conf_b = conf_b;
  a.sts_T = sts_T;
  a.tokens = tokens;
  a.logit = logit;
  a.conf = conf;
  a.surv = surv;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  a.exclusive = g_draft_launch.load() == DSPARK_LAUNCH_EXCLUSIVE;
  a.decay = rnn ? decay : nullptr;
  a.noalloc = noalloc;
  a.step = step;
  a.check_only = check_only;
  const char* why = nullptr;
  hipError_t e = dspark::launch_markov_draft(a, stream, &why, fused);
  if (why) return fail(DSPARK_ERR_UNSUPPORTED, "%s", why);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

}  // namespace

dspark_status dspark_markov_draft(int B, int gamma, int V, int r, int d, dspark_dtype dtype,
                                  const int32_t* anchor, const void* U, const void* h, const void* W1,
                                  const void* W2, const float* conf_w, float conf_b, const float* sts_T,
                                  dspark_sampling mode, uint64_t seed, int32_t* tokens, float* logit,
                                  float* conf, float* surv, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  return draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, nullptr, false, conf_w, conf_b, sts_T, mode, seed,
                    tokens, logit, conf, surv, workspace, workspace_bytes, stream);
}

dspark_status dspark_markov_draft_noalloc(int B, int gamma, int V, int r, int d, dspark_dtype dtype,
                                          const int32_t* anchor, const void* U, const void* h, const void* W1,
                                          const void* W2, const float* conf_w, float conf_b, const float* sts_T,
                                          dspark_sampling mode, uint64_t seed, int32_t* tokens, float* logit,
                                          float* conf, float* surv, hipStream_t stream) {
  return draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, nullptr, false, conf_w, conf_b, sts_T, mode, seed,
                    tokens, logit, conf, surv, nullptr, 0, stream, /*noalloc=*/true);
}

dspark_status dspark_rnn_draft(int B, int gamma, int V, int r, int d, dspark_dtype dtype, const int32_t* anchor,
                               const void* U, const void* h, const void* W1, const void* W2, const float* decay,
                               const float* conf_w, float conf_b, const float* sts_T, dspark_sampling mode,
                               uint64_t seed, int32_t* tokens, float* logit, float* conf, float* surv,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, decay, true, conf_w, conf_b, sts_T, mode, seed,
                    tokens, logit, conf, surv, workspace, workspace_bytes, stream);
}

size_t dspark_schedule_workspace_bytes(int B, int gamma) {
  if (B < 0 || gamma < 0) return 0;
  return dspark::schedule_workspace_bytes(B, gamma);
}

dspark_status dspark_schedule(int B, int gamma, const float* surv, const double* t_step, int n_min, int n_count,
                              int32_t* lens, int32_t* m_out, double* objective, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0 || n_count < 1) return fail(DSPARK_ERR_INVALID_ARG, "negative size or empty step-cost table");
  if (!t_step || !m_out || (B > 0 && (!lens || (gamma > 0 && !surv))))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (n_min > B || (long long)n_min + n_count - 1 < B)
    return fail(DSPARK_ERR_INVALID_ARG, "step-cost table must cover n = B (n_min <= B <= n_min + n_count - 1)");
  if ((long long)B * gamma > dspark::kMaxScheduleItems)
    return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 16384");
  if (workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(DSPARK_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (workspace_bytes < dspark::schedule_workspace_bytes(B, gamma))
      return fail(DSPARK_ERR_WORKSPACE, "workspace smaller than dspark_schedule_workspace_bytes(B, gamma)");
  }
  hipError_t e =
      dspark::launch_schedule(B, gamma, surv, t_step, n_min, n_count, lens, m_out, objective, workspace, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

dspark_status dspark_parallel_draft(int B, int gamma, int V, dspark_dtype dtype, const void* U,
                                    dspark_sampling mode, uint64_t seed, int32_t* tokens, float* logit,
                                    hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0 || V < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (mode != DSPARK_GREEDY && mode != DSPARK_GUMBEL) return fail(DSPARK_ERR_INVALID_ARG, "unknown sampling mode");
  if (B == 0 || gamma == 0) return DSPARK_OK;
  if (V < 1) return fail(DSPARK_ERR_INVALID_ARG, "V must be positive");
  if (!U || !tokens || !logit) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (V > kMaxV) return fail(DSPARK_ERR_UNSUPPORTED, "V > 2^24");
  if ((long long)B * gamma > 0x7FFFFFFFLL) return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 2^31 - 1");
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(U) % elem) return fail(DSPARK_ERR_INVALID_ARG, "misaligned U");
  hipError_t e = dspark::launch_parallel_draft(B, gamma, V, dtype == DSPARK_BF16, U, mode == DSPARK_GUMBEL, seed,
                                               tokens, logit, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

dspark_status dspark_gumbel_from_words(int n, const uint32_t* words, float* out, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (n < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (n == 0) return DSPARK_OK;
  if (!words || !out) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (reinterpret_cast<uintptr_t>(words) % 4 || reinterpret_cast<uintptr_t>(out) % 4)
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned array");
  hipError_t e = dspark::launch_gumbel_words(n, words, out, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

dspark_status dspark_schedule_threshold(int B, int gamma, const float* surv, float tau, int32_t* lens,
                                        int32_t* m_out, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (!m_out || (B > 0 && (!lens || (gamma > 0 && !surv)))) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if ((long long)B * gamma > 0x7FFFFFFFLL) return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 2^31 - 1");
  hipError_t e = dspark::launch_schedule_threshold(B, gamma, surv, tau, lens, m_out, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

dspark_status dspark_serve(int iters, int B, int gamma, int V, int r, int d, dspark_dtype dtype,
                           const int32_t* anchor0, const void* U, const void* h, const void* W1, const void* W2,
                           const float* conf_w, float conf_b, const float* sts_T, dspark_sampling mode,
                           uint64_t seed, const int32_t* target, const double* t_step, int n_min, int n_count,
                           dspark_policy policy, float tau, int32_t* tokens, float* logit, float* conf,
                           float* surv, int32_t* lens, int32_t* accepted, int32_t* bonus, int32_t* m_out,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (iters < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative iteration count");
  if (policy != DSPARK_POLICY_GLOBAL && policy != DSPARK_POLICY_GLOBAL_DELAYED2 && policy != DSPARK_POLICY_THRESHOLD)
    return fail(DSPARK_ERR_INVALID_ARG, "unknown scheduling policy");
  if (B < 0 || gamma < 0 || V < 0 || r < 0 || d < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (iters == 0 || B == 0 || gamma == 0) return DSPARK_OK;
  if (!target || !lens || !accepted || !bonus || !m_out || (policy != DSPARK_POLICY_THRESHOLD && !t_step))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (policy != DSPARK_POLICY_THRESHOLD) {
    if (n_count < 1) return fail(DSPARK_ERR_INVALID_ARG, "empty step-cost table");
    if (n_min > B || (long long)n_min + n_count - 1 < B)
      return fail(DSPARK_ERR_INVALID_ARG, "step-cost table must cover n = B (n_min <= B <= n_min + n_count - 1)");
    if ((long long)B * gamma > dspark::kMaxScheduleItems) return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 16384");
  }
  // the draft's workspace first, the scheduler's after it
  const size_t draft_bytes = dspark_draft_workspace_bytes(B, gamma, V, r);
  const size_t sched_bytes = policy == DSPARK_POLICY_THRESHOLD ? 0 : dspark::schedule_workspace_bytes(B, gamma);
  if (workspace && workspace_bytes >= draft_bytes && workspace_bytes - draft_bytes < sched_bytes)
    return fail(DSPARK_ERR_WORKSPACE, "workspace smaller than dspark_serve_workspace_bytes(B, gamma, V, r)");
  void* sched_ws = workspace ? static_cast<unsigned char*>(workspace) + draft_bytes : nullptr;
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  const size_t bg = size_t(B) * size_t(gamma);
  for (int t = 0; t < iters; ++t) {
    const int32_t* anchor = t == 0 ? anchor0 : bonus + size_t(t - 1) * B;
    const unsigned char* Ut = static_cast<const unsigned char*>(U) + size_t(t) * bg * size_t(V) * elem;
    const unsigned char* ht = h ? static_cast<const unsigned char*>(h) + size_t(t) * bg * size_t(d) * elem : nullptr;
    float* surv_t = surv + size_t(t) * bg;
    // iteration 0 validates the draft arguments before anything is enqueued;
    // later iterations differ only by offsets that keep the same alignment
    dspark_status st = dspark_markov_draft(B, gamma, V, r, d, dtype, anchor, Ut, ht, W1, W2, conf_w, conf_b, sts_T,
                                           mode, seed + uint64_t(t), tokens + size_t(t) * bg, logit + size_t(t) * bg,
                                           conf + size_t(t) * bg, surv_t, workspace, workspace_bytes, stream);
    if (st != DSPARK_OK) return st;
    hipError_t e;
    if (policy == DSPARK_POLICY_THRESHOLD) {
      e = dspark::launch_schedule_threshold(B, gamma, surv_t, tau, lens + size_t(t) * B, m_out + t, stream);
    } else {
      const float* src = (policy == DSPARK_POLICY_GLOBAL_DELAYED2 && t >= 2) ? surv + size_t(t - 2) * bg : surv_t;
      e = dspark::launch_schedule(B, gamma, src, t_step, n_min, n_count, lens + size_t(t) * B, m_out + t, nullptr,
                                  sched_ws, stream);
    }
    if (e != hipSuccess) return hip_fail(e);
    e = dspark::launch_verify(B, gamma, tokens + size_t(t) * bg, target + size_t(t) * bg + size_t(t) * B,
                              lens + size_t(t) * B, accepted + size_t(t) * B, bonus + size_t(t) * B, stream);
    if (e != hipSuccess) return hip_fail(e);
  }
  return DSPARK_OK;
}

size_t dspark_sts_workspace_bytes(int N, int G, int n_bins) {
  if (N < 0 || G < 1 || n_bins < 1 || G > dspark::kMaxStsGrid || n_bins > dspark::kMaxStsBins) return 0;
  return dspark::sts_workspace_layout(N, G, n_bins).total;
}

dspark_status dspark_sts_fit(int N, int gamma, const float* logit, const int32_t* accepted, const float* grid,
                             int G, int n_bins, int32_t* choice, float* T_out, double* ece, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (N < 0 || gamma < 0 || G < 0 || n_bins < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (gamma == 0) return DSPARK_OK;
  if (G < 1 || n_bins < 1) return fail(DSPARK_ERR_INVALID_ARG, "G and n_bins must be positive");
  if (!grid || !choice || !T_out || !ece || (N > 0 && (!logit || !accepted)))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (G > dspark::kMaxStsGrid) return fail(DSPARK_ERR_UNSUPPORTED, "G > 4096");
  if (n_bins > dspark::kMaxStsBins) return fail(DSPARK_ERR_UNSUPPORTED, "n_bins > 256");
  if ((long long)G * n_bins > dspark::kMaxStsHist) return fail(DSPARK_ERR_UNSUPPORTED, "G * n_bins > 8192");
  if (N > dspark::kMaxStsBlocks) return fail(DSPARK_ERR_UNSUPPORTED, "N > 2^24");
  if ((long long)N * gamma > 0x7FFFFFFFLL) return fail(DSPARK_ERR_UNSUPPORTED, "N * gamma > 2^31 - 1");
  if (reinterpret_cast<uintptr_t>(logit) % 4 || reinterpret_cast<uintptr_t>(accepted) % 4 ||
      reinterpret_cast<uintptr_t>(grid) % 4 || reinterpret_cast<uintptr_t>(ece) % 8)
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_sts_workspace_bytes(N, G, n_bins);
  if (!workspace || workspace_bytes < need)
    return fail(DSPARK_ERR_WORKSPACE, "workspace missing or smaller than dspark_sts_workspace_bytes()");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(DSPARK_ERR_WORKSPACE, "workspace not 256-byte aligned");
  dspark::StsArgs a;
  a.N = N;
  a.gamma = gamma;
  a.G = G;
  a.nbins = n_bins;
  a.logit = logit;
  a.accepted = accepted;
  a.grid = grid;
  a.choice = choice;
  a.T_out = T_out;
  a.ece = ece;
  a.ws = workspace;
  hipError_t e = dspark::launch_sts_fit(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

dspark_status dspark_verify(int B, int gamma, const int32_t* tokens, const int32_t* target, const int32_t* lens,
                            int32_t* accepted, int32_t* bonus, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (B == 0) return DSPARK_OK;
  if (!target || !lens || !accepted || !bonus || (gamma > 0 && !tokens))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  hipError_t e = dspark::launch_verify(B, gamma, tokens, target, lens, accepted, bonus, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_step_workspace_bytes(int B, int gamma, int V, int r) { return dspark_serve_workspace_bytes(B, gamma, V, r); }

dspark_status dspark_step(int B, int gamma, int V, int r, int d, dspark_dtype dtype, const int32_t* anchor,
                          const void* U, const void* h, const void* W1, const void* W2, const float* conf_w,
                          float conf_b, const float* sts_T, dspark_sampling mode, uint64_t seed,
                          const int32_t* target, const double* t_step, int n_min, int n_count, int32_t* tokens,
                          float* logit, float* conf, float* surv, int32_t* lens, int32_t* m_out, int32_t* accepted,
                          int32_t* bonus, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0 || V < 0 || r < 0 || d < 0 || n_count < 1)
    return fail(DSPARK_ERR_INVALID_ARG, "negative size or empty step-cost table");
  if (B == 0) return DSPARK_OK;
  if (!target || !t_step || !lens || !m_out || !accepted || !bonus)
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (n_min > B || (long long)n_min + n_count - 1 < B)
    return fail(DSPARK_ERR_INVALID_ARG, "step-cost table must cover n = B (n_min <= B <= n_min + n_count - 1)");
  if ((long long)B * gamma > dspark::kMaxScheduleItems) return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 16384");
  // the drafting workspace first, the scheduler's after it
  const size_t draft_bytes = dspark_draft_workspace_bytes(B, gamma, V, r);
  const size_t sched_bytes = dspark::schedule_workspace_bytes(B, gamma);
  if (workspace && workspace_bytes >= draft_bytes && workspace_bytes - draft_bytes < sched_bytes)
    return fail(DSPARK_ERR_WORKSPACE, "workspace smaller than dspark_step_workspace_bytes(B, gamma, V, r)");
  if (gamma == 0) {   // nothing to draft or schedule: every length 0, bonus = target[b][0]
    hipError_t e = dspark::launch_schedule(B, 0, nullptr, t_step, n_min, n_count, lens, m_out, nullptr, nullptr,
                                           stream);
    if (e == hipSuccess) e = dspark::launch_verify(B, 0, nullptr, target, lens, accepted, bonus, stream);
    if (e != hipSuccess) return hip_fail(e);
    return DSPARK_OK;
  }
  dspark::StepArgs st;
  st.t_step = t_step;
  st.n_min = n_min;
  st.n_count = n_count;
  st.target = target;
  st.lens = lens;
  st.m_out = m_out;
  st.accepted = accepted;
  st.bonus = bonus;
  st.sched_ws = workspace ? static_cast<unsigned char*>(workspace) + draft_bytes : nullptr;
  bool fused = false;
  dspark_status ds = draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, nullptr, false, conf_w, conf_b,
                                sts_T, mode, seed, tokens, logit, conf, surv, workspace, workspace_bytes, stream,
                                false, &st, &fused);
  if (ds != DSPARK_OK || fused) return ds;
  hipError_t e = dspark::launch_schedule(B, gamma, surv, t_step, n_min, n_count, lens, m_out, nullptr, st.sched_ws,
                                         stream);
  if (e == hipSuccess) e = dspark::launch_verify(B, gamma, tokens, target, lens, accepted, bonus, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

namespace {

bool known_dtype(dspark_dtype t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool misaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// Whether [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}
struct Span {
  const void* p;
  size_t n;
};
// Whether any output (the workspace is one) shares memory with an input or
// with another output.
bool any_overlap(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (overlap(o->p, o->n, i.p, i.n)) return true;
    for (const Span* q = out.begin(); q != o; ++q)
      if (overlap(o->p, o->n, q->p, q->n)) return true;
  }
  return false;
}
dspark_status overlap_refused() { return fail(DSPARK_ERR_INVALID_ARG, "an output or the workspace overlaps another array"); }

// Checks shared by the linear layer's two directions.
dspark_status linear_sizes(int M, int N, int K, dspark_dtype dtype, dspark_activation act) {
  if (M < 0 || N < 0 || K < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (!known_dtype(dtype)) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (act != DSPARK_ACT_NONE && act != DSPARK_ACT_RELU && act != DSPARK_ACT_GELU && act != DSPARK_ACT_SILU)
    return fail(DSPARK_ERR_INVALID_ARG, "unknown activation");
  if (M > dspark::kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "M > 2^20");
  if (N > kMaxV) return fail(DSPARK_ERR_UNSUPPORTED, "N > 2^24");
  if (K > kMaxD) return fail(DSPARK_ERR_UNSUPPORTED, "K > 65536");
  return DSPARK_OK;
}

dspark_status check_workspace(const void* ws, size_t have, size_t need, const char* name) {
  if (need == 0) return DSPARK_OK;
  if (!ws || have < need) return fail(DSPARK_ERR_WORKSPACE, "workspace missing or smaller than %s()", name);
  if (misaligned(ws, 256)) return fail(DSPARK_ERR_WORKSPACE, "workspace not 256-byte aligned");
  return DSPARK_OK;
}

}  // namespace

size_t dspark_linear_workspace_bytes(int M, int N, int K, dspark_dtype dtype) {
  if (M <= 0 || N <= 0 || K < 0 || M > dspark::kMaxRows || N > kMaxV || K > kMaxD || !known_dtype(dtype)) return 0;
  return dspark::linear_workspace_bytes(M, N, K, dtype == DSPARK_BF16);
}

dspark_status dspark_linear(int M, int N, int K, dspark_dtype dtype, const void* x, const void* w, const void* bias,
                            dspark_activation act, const void* residual, void* y, float* pre, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = linear_sizes(M, N, K, dtype, act);
  if (st != DSPARK_OK) return st;
  if (M == 0 || N == 0) return DSPARK_OK;
  if (!y || (K > 0 && (!x || !w))) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(x, 16) || misaligned(w, 16)) return fail(DSPARK_ERR_INVALID_ARG, "x and w need 16-byte alignment");
  if (misaligned(bias, elem) || misaligned(residual, elem) || misaligned(y, elem) || misaligned(pre, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_linear_workspace_bytes(M, N, K, dtype);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_linear_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t m = size_t(M), n = size_t(N), k = size_t(K);
  if (any_overlap({{y, m * n * elem}, {pre, m * n * 4}, {workspace, need}},
                  {{x, m * k * elem},
                   {w, n * k * elem},
                   {bias, n * elem},
                   {residual == y ? nullptr : residual, m * n * elem}}))
    return overlap_refused();
  dspark::LinearArgs a;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = dtype == DSPARK_BF16;
  a.act = int(act);
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.pre = pre;
  a.ws = workspace;
  hipError_t e = dspark::launch_linear(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_linear_backward_act_workspace_bytes(int M, int N, int K, dspark_dtype dtype, dspark_activation act) {
  if (M < 0 || N <= 0 || K < 0 || M > dspark::kMaxRows || N > kMaxV || K > kMaxD || !known_dtype(dtype)) return 0;
  return dspark::linear_backward_workspace_bytes(M, N, K, dtype == DSPARK_BF16, act != DSPARK_ACT_NONE);
}

size_t dspark_linear_backward_workspace_bytes(int M, int N, int K, dspark_dtype dtype) {
  return dspark_linear_backward_act_workspace_bytes(M, N, K, dtype, DSPARK_ACT_RELU);
}

dspark_status dspark_linear_backward(int M, int N, int K, dspark_dtype dtype, const void* dy, const void* x,
                                     const void* w, dspark_activation act, const float* pre, void* dx, void* dw,
                                     void* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = linear_sizes(M, N, K, dtype, act);
  if (st != DSPARK_OK) return st;
  const bool some = M > 0 && N > 0;
  if ((some && !dy) || (some && act != DSPARK_ACT_NONE && !pre) || (some && dx && K > 0 && !w) ||
      (some && dw && K > 0 && !x))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(dy, 16))
    return fail(DSPARK_ERR_INVALID_ARG, "x, w and dy need 16-byte alignment");
  if (misaligned(dx, elem) || misaligned(dw, elem) || misaligned(dbias, elem) || misaligned(pre, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_linear_backward_act_workspace_bytes(M, N, K, dtype, act);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_linear_backward_act_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t m = size_t(M), n = size_t(N), k = size_t(K);
  if (any_overlap({{dx, m * k * elem}, {dw, n * k * elem}, {dbias, n * elem}, {workspace, need}},
                  {{dy, m * n * elem}, {x, m * k * elem}, {w, n * k * elem}, {pre, m * n * 4}}))
    return overlap_refused();
  if (!dx && !dw && !dbias) return DSPARK_OK;
  dspark::LinearBackwardArgs a;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = dtype == DSPARK_BF16;
  a.act = int(act);
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.pre = pre;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.ws = workspace;
  hipError_t e = dspark::launch_linear_backward(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

namespace {

bool loss_sizes_fit(int N, int V, int d, int r) {
  return N >= 0 && V >= 1 && d >= 0 && r >= 0 && N <= dspark::kMaxRows && V <= kMaxV && d <= kMaxD && r <= kMaxD;
}

// Checks shared by the loss and its gradient.
dspark_status loss_inputs(const dspark::LossArgs& a, dspark_dtype dtype) {
  if (a.N < 0 || a.V < 0 || a.d < 0 || a.r < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (!known_dtype(dtype)) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (a.V < 1) return fail(DSPARK_ERR_INVALID_ARG, "V must be positive");
  if ((a.d > 0) != (a.Wo != nullptr) || (a.d == 0 && a.h) || (a.r > 0) != (a.W2 != nullptr) ||
      (a.r == 0 && (a.W1 || a.prev)))
    return fail(DSPARK_ERR_INVALID_ARG, "h and Wo go with d > 0, prev, W1 and W2 with r > 0");
  if (a.N > 0 && (!a.label || (a.d > 0 && !a.h) || (a.r > 0 && (!a.W1 || !a.prev))))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (a.N > 0 && !a.U && a.d == 0 && a.r == 0)
    return fail(DSPARK_ERR_INVALID_ARG, "no logits: give U, h and Wo, or prev, W1 and W2");
  if (a.N > dspark::kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "N > 2^20");
  if (a.V > kMaxV) return fail(DSPARK_ERR_UNSUPPORTED, "V > 2^24");
  if (a.d > kMaxD || a.r > kMaxD) return fail(DSPARK_ERR_UNSUPPORTED, "d or r > 65536");
  if (misaligned(a.h, 16) || misaligned(a.Wo, 16) || misaligned(a.W1, 16) || misaligned(a.W2, 16))
    return fail(DSPARK_ERR_INVALID_ARG, "h, Wo, W1 and W2 need 16-byte alignment");
  if (misaligned(a.U, a.bf16 ? 2 : 4) || misaligned(a.label, 4) || misaligned(a.prev, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  return DSPARK_OK;
}

dspark::LossArgs loss_args(int N, int V, int d, int r, dspark_dtype dtype, const int32_t* label, const void* U,
                           const void* h, const void* Wo, const int32_t* prev, const void* W1, const void* W2,
                           void* ws) {
  dspark::LossArgs a = {};
  a.N = N;
  a.V = V;
  a.d = d;
  a.r = r;
  a.bf16 = dtype == DSPARK_BF16;
  a.label = label;
  a.prev = prev;
  a.U = U;
  a.h = h;
  a.Wo = Wo;
  a.W1 = W1;
  a.W2 = W2;
  a.ws = ws;
  return a;
}

// any_overlap() with the inputs that the loss and its gradient share.
bool overlaps_loss(std::initializer_list<Span> out, const dspark::LossArgs& a) {
  const size_t elem = a.bf16 ? 2 : 4, n = size_t(a.N), v = size_t(a.V), d = size_t(a.d), r = size_t(a.r);
  return any_overlap(out, {{a.label, n * 4},
                           {a.prev, n * 4},
                           {a.U, n * v * elem},
                           {a.h, n * d * elem},
                           {a.Wo, v * d * elem},
                           {a.W1, v * r * elem},
                           {a.W2, r * v * elem}});
}

}  // namespace

size_t dspark_markov_loss_workspace_bytes(int N, int V, int d, int r, dspark_dtype dtype) {
  if (!loss_sizes_fit(N, V, d, r) || !known_dtype(dtype) || N == 0) return 0;
  return dspark::loss_workspace_bytes(N, V, d, r, dtype == DSPARK_BF16, false);
}

dspark_status dspark_markov_loss(int N, int V, int d, int r, dspark_dtype dtype, const int32_t* label, const void* U,
                                 const void* h, const void* Wo, const int32_t* prev, const void* W1, const void* W2,
                                 float* nll, float* lse, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark::LossArgs a = loss_args(N, V, d, r, dtype, label, U, h, Wo, prev, W1, W2, workspace);
  dspark_status st = loss_inputs(a, dtype);
  if (st != DSPARK_OK) return st;
  if (N == 0) return DSPARK_OK;
  if (!nll || !lse) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  // 256 threads for each 128 x 128 logits (the least that so many rows take): a launch holds less than 2^32
  if ((long long)((V + 127) / 128) * ((N + 127) / 128) >= 1ll << 24)
    return fail(DSPARK_ERR_UNSUPPORTED, "N * V (both rounded up to 128) >= 2^38");
  if (misaligned(nll, 4) || misaligned(lse, 4)) return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_markov_loss_workspace_bytes(N, V, d, r, dtype);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_markov_loss_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t rows = size_t(N) * 4;
  if (overlaps_loss({{nll, rows}, {lse, rows}, {workspace, need}}, a)) return overlap_refused();
  a.nll = nll;
  a.lse = lse;
  hipError_t e = dspark::launch_markov_loss(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_markov_loss_backward_workspace_bytes(int N, int V, int d, int r, dspark_dtype dtype) {
  if (!loss_sizes_fit(N, V, d, r) || !known_dtype(dtype)) return 0;
  return dspark::loss_workspace_bytes(N, V, d, r, dtype == DSPARK_BF16, true);
}

dspark_status dspark_markov_loss_backward(int N, int V, int d, int r, dspark_dtype dtype, const float* g,
                                          const float* lse, const int32_t* label, const void* U, const void* h,
                                          const void* Wo, const int32_t* prev, const void* W1, const void* W2,
                                          void* dU, void* dh, void* dWo, void* dW1, void* dW2, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark::LossArgs a = loss_args(N, V, d, r, dtype, label, U, h, Wo, prev, W1, W2, workspace);
  dspark_status st = loss_inputs(a, dtype);
  if (st != DSPARK_OK) return st;
  if (N > 0 && (!g || !lse)) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if ((dU && N > 0 && !U) || (d == 0 && (dh || dWo)) || (r == 0 && (dW1 || dW2)))
    return fail(DSPARK_ERR_INVALID_ARG, "gradient of an input that is not there");
  const size_t elem = a.bf16 ? 2 : 4;
  if (misaligned(g, 4) || misaligned(lse, 4) || misaligned(dU, elem) || misaligned(dh, elem) ||
      misaligned(dWo, elem) || misaligned(dW1, elem) || misaligned(dW2, elem))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_markov_loss_backward_workspace_bytes(N, V, d, r, dtype);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_markov_loss_backward_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t n = size_t(N) * elem, v = size_t(V) * elem, rows = size_t(N) * 4;
  const std::initializer_list<Span> out = {
      {dU, n * V}, {dh, n * d}, {dWo, v * d}, {dW1, v * r}, {dW2, v * r}, {workspace, need}};
  if (overlaps_loss(out, a) || any_overlap(out, {{g, rows}, {lse, rows}})) return overlap_refused();
  if (!dU && !dh && !dWo && !dW1 && !dW2) return DSPARK_OK;
  a.lse_in = lse;
  a.g = g;
  a.dU = dU;
  a.dh = dh;
  a.dWo = dWo;
  a.dW1 = dW1;
  a.dW2 = dW2;
  hipError_t e = dspark::launch_markov_loss_backward(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_hidden_draft_workspace_bytes(int B, int gamma, int V, int r, int d, dspark_dtype dtype) {
  const size_t draft = dspark_draft_workspace_bytes(B, gamma, V, r);
  if (draft == 0 || (long long)B * gamma > dspark::kMaxRows) return draft;
  return draft + dspark_linear_workspace_bytes(B * gamma, V, d, dtype);
}

dspark_status dspark_hidden_draft(int B, int gamma, int V, int r, int d, dspark_dtype dtype, const int32_t* anchor,
                                  const void* h, const void* Wo, const void* bias, const void* W1, const void* W2,
                                  const float* conf_w, float conf_b, const float* sts_T, dspark_sampling mode,
                                  uint64_t seed, void* U, int32_t* tokens, float* logit, float* conf, float* surv,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || gamma < 0 || V < 0 || r < 0 || d < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if ((long long)B * gamma > dspark::kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "B * gamma > 2^20");
  // every check of the draft before the product is enqueued
  dspark_status st = draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, nullptr, false, conf_w, conf_b, sts_T,
                                mode, seed, tokens, logit, conf, surv, workspace, workspace_bytes, stream, false,
                                nullptr, nullptr, /*check_only=*/true);
  // (they ask the device last: what is wrong with the arrays is said where there is none, too)
  if ((st != DSPARK_OK && st != DSPARK_ERR_HIP) || B == 0 || gamma == 0) return st;
  const size_t draft = dspark_draft_workspace_bytes(B, gamma, V, r);
  if (workspace_bytes < dspark_hidden_draft_workspace_bytes(B, gamma, V, r, d, dtype))
    return fail(DSPARK_ERR_WORKSPACE, "workspace smaller than dspark_hidden_draft_workspace_bytes()");
  {
    const size_t elem = dtype == DSPARK_BF16 ? 2 : 4, n = size_t(B) * gamma, v = size_t(V);
    if (any_overlap({{U, n * v * elem},
                     {tokens, n * 4},
                     {logit, n * 4},
                     {conf, n * 4},
                     {surv, n * 4},
                     {workspace, dspark_hidden_draft_workspace_bytes(B, gamma, V, r, d, dtype)}},
                    {{anchor, size_t(B) * 4},
                     {h, n * d * elem},
                     {Wo, v * d * elem},
                     {bias, v * elem},
                     {W1, v * r * elem},
                     {W2, v * r * elem},
                     {conf_w, (size_t(d) + r) * 4},
                     {sts_T, size_t(gamma) * 4}}))
      return overlap_refused();
  }
  if (st != DSPARK_OK) return st;
  st = dspark_linear(B * gamma, V, d, dtype, h, Wo, bias, DSPARK_ACT_NONE, nullptr, U, nullptr,
                     static_cast<unsigned char*>(workspace) + draft, workspace_bytes - draft, stream);
  if (st != DSPARK_OK) return st;
  return draft_impl(B, gamma, V, r, d, dtype, anchor, U, h, W1, W2, nullptr, false, conf_w, conf_b, sts_T, mode, seed,
                    tokens, logit, conf, surv, workspace, workspace_bytes, stream);
}

size_t dspark_gated_linear_workspace_bytes(int M, int N, int K, dspark_dtype dtype) {
  if (M <= 0 || N <= 0 || K < 0 || M > dspark::kMaxRows || N > kMaxV || K > kMaxD || !known_dtype(dtype)) return 0;
  return dspark::gated_workspace_bytes(M, N, K, dtype == DSPARK_BF16);
}

dspark_status dspark_gated_linear(int M, int N, int K, dspark_dtype dtype, const void* x, const void* wg,
                                  const void* wu, const void* bg, const void* bu, dspark_activation act, void* y,
                                  float* pre, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = linear_sizes(M, N, K, dtype, act);
  if (st != DSPARK_OK) return st;
  if (M == 0 || N == 0) return DSPARK_OK;
  if (!y || (K > 0 && (!x || !wg || !wu))) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(x, 16) || misaligned(wg, 16) || misaligned(wu, 16))
    return fail(DSPARK_ERR_INVALID_ARG, "x, wg and wu need 16-byte alignment");
  if (misaligned(bg, elem) || misaligned(bu, elem) || misaligned(y, elem) || misaligned(pre, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_gated_linear_workspace_bytes(M, N, K, dtype);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_gated_linear_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t m = size_t(M), n = size_t(N), k = size_t(K);
  if (any_overlap({{y, m * n * elem}, {pre, m * n * 8}, {workspace, need}},
                  {{x, m * k * elem}, {wg, n * k * elem}, {wu, n * k * elem}, {bg, n * elem}, {bu, n * elem}}))
    return overlap_refused();
  dspark::GatedArgs a;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = dtype == DSPARK_BF16;
  a.act = int(act);
  a.x = x;
  a.wg = wg;
  a.wu = wu;
  a.bg = bg;
  a.bu = bu;
  a.y = y;
  a.pre = pre;
  a.ws = workspace;
  hipError_t e = dspark::launch_gated(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_gated_linear_backward_workspace_bytes(int M, int N, int K, dspark_dtype dtype) {
  if (M < 0 || N < 0 || K < 0 || M > dspark::kMaxRows || N > kMaxV || K > kMaxD || !known_dtype(dtype)) return 0;
  return dspark::gated_backward_workspace_bytes(M, N, K, dtype == DSPARK_BF16);
}

dspark_status dspark_gated_linear_backward(int M, int N, int K, dspark_dtype dtype, const void* dy, const void* x,
                                           const void* wg, const void* wu, dspark_activation act, const float* pre,
                                           void* dx, void* dwg, void* dwu, void* dbg, void* dbu, void* workspace,
                                           size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = linear_sizes(M, N, K, dtype, act);
  if (st != DSPARK_OK) return st;
  const bool some = M > 0 && N > 0;
  if (some && (!dy || !pre || (dx && K > 0 && (!wg || !wu)) || ((dwg || dwu) && K > 0 && !x)))
    return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(x, 16) || misaligned(wg, 16) || misaligned(wu, 16) || misaligned(dy, 16))
    return fail(DSPARK_ERR_INVALID_ARG, "x, wg, wu and dy need 16-byte alignment");
  if (misaligned(dx, elem) || misaligned(dwg, elem) || misaligned(dwu, elem) || misaligned(dbg, elem) ||
      misaligned(dbu, elem) || misaligned(pre, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_gated_linear_backward_workspace_bytes(M, N, K, dtype);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_gated_linear_backward_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t m = size_t(M), n = size_t(N), k = size_t(K);
  if (any_overlap({{dx, m * k * elem},
                   {dwg, n * k * elem},
                   {dwu, n * k * elem},
                   {dbg, n * elem},
                   {dbu, n * elem},
                   {workspace, need}},
                  {{dy, m * n * elem}, {x, m * k * elem}, {wg, n * k * elem}, {wu, n * k * elem}, {pre, m * n * 8}}))
    return overlap_refused();
  if (!dx && !dwg && !dwu && !dbg && !dbu) return DSPARK_OK;
  dspark::GatedBackwardArgs a;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = dtype == DSPARK_BF16;
  a.act = int(act);
  a.dy = dy;
  a.x = x;
  a.wg = wg;
  a.wu = wu;
  a.pre = pre;
  a.dx = dx;
  a.dwg = dwg;
  a.dwu = dwu;
  a.dbg = dbg;
  a.dbu = dbu;
  a.ws = workspace;
  hipError_t e = dspark::launch_gated_backward(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

namespace {

dspark_status norm_sizes(int M, int C, dspark_dtype dtype, dspark_norm_kind kind) {
  if (M < 0 || C < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (!known_dtype(dtype)) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (kind != DSPARK_NORM_LAYER && kind != DSPARK_NORM_RMS)
    return fail(DSPARK_ERR_INVALID_ARG, "unknown normalisation");
  if (M > dspark::kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "M > 2^20");
  if (C > dspark::kMaxChannels) return fail(DSPARK_ERR_UNSUPPORTED, "C > 32768");
  return DSPARK_OK;
}

}  // namespace

dspark_status dspark_norm(int M, int C, dspark_dtype dtype, dspark_norm_kind kind, const void* x, const void* residual,
                          const void* weight, const void* bias, float eps, void* sum, void* y, float* stat,
                          hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = norm_sizes(M, C, dtype, kind);
  if (st != DSPARK_OK) return st;
  if (!(eps >= 0.f && eps <= 3.4e38f)) return fail(DSPARK_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (M == 0 || C == 0) return DSPARK_OK;
  if (!x || !y) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if ((residual != nullptr) != (sum != nullptr)) return fail(DSPARK_ERR_INVALID_ARG, "sum goes with residual");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(x, elem) || misaligned(residual, elem) || misaligned(weight, elem) || misaligned(bias, elem) ||
      misaligned(sum, elem) || misaligned(y, elem) || misaligned(stat, 8))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t rows = size_t(M) * C * elem, row = size_t(C) * elem, stats = size_t(M) * 8;
  // the sum may take its place over either of its parts, whose other overlaps are refused all the same
  if (any_overlap({{sum, rows}}, {{sum == x ? nullptr : x, rows}, {sum == residual ? nullptr : residual, rows}}) ||
      any_overlap({{sum, rows}, {y, rows}, {stat, stats}}, {{weight, row}, {bias, row}}) ||
      any_overlap({{y, rows}, {stat, stats}}, {{x, rows}, {residual, rows}, {sum, rows}}))
    return overlap_refused();
  dspark::NormArgs a;
  a.M = M;
  a.C = C;
  a.bf16 = dtype == DSPARK_BF16;
  a.center = kind == DSPARK_NORM_LAYER;
  a.x = x;
  a.residual = residual;
  a.w = weight;
  a.b = bias;
  a.eps = eps;
  a.sum = sum;
  a.y = y;
  a.stat = stat;
  hipError_t e = dspark::launch_norm(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_norm_backward_workspace_bytes(int M, int C, dspark_dtype dtype) {
  if (M <= 0 || C <= 0 || M > dspark::kMaxRows || C > dspark::kMaxChannels || !known_dtype(dtype)) return 0;
  return dspark::norm_backward_workspace_bytes(M, C, dtype == DSPARK_BF16);
}

dspark_status dspark_norm_backward(int M, int C, dspark_dtype dtype, dspark_norm_kind kind, const void* dy,
                                   const void* x, const float* stat, const void* weight, const void* dsum, void* dx,
                                   void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark_status st = norm_sizes(M, C, dtype, kind);
  if (st != DSPARK_OK) return st;
  if (C == 0 || (!dx && !dweight && !dbias)) return DSPARK_OK;
  if (M > 0 && (!dy || !x || !stat)) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = dtype == DSPARK_BF16 ? 2 : 4;
  if (misaligned(dy, elem) || misaligned(x, elem) || misaligned(stat, 8) || misaligned(weight, elem) ||
      misaligned(dsum, elem) || misaligned(dx, elem) || misaligned(dweight, elem) || misaligned(dbias, elem))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dweight || dbias ? dspark_norm_backward_workspace_bytes(M, C, dtype) : 0;
  st = check_workspace(workspace, workspace_bytes, need, "dspark_norm_backward_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const size_t rows = size_t(M) * C * elem, row = size_t(C) * elem;
  if (any_overlap({{dx, rows}, {dweight, row}, {dbias, row}, {workspace, need}},
                  {{dy, rows}, {x, rows}, {stat, size_t(M) * 8}, {weight, row}, {dsum == dx ? nullptr : dsum, rows}}) ||
      any_overlap({{dweight, row}, {dbias, row}, {workspace, need}}, {{dsum, rows}}))
    return overlap_refused();
  dspark::NormBackwardArgs a;
  a.M = M;
  a.C = C;
  a.bf16 = dtype == DSPARK_BF16;
  a.center = kind == DSPARK_NORM_LAYER;
  a.dy = dy;
  a.x = x;
  a.stat = stat;
  a.w = weight;
  a.dsum = dsum;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.ws = workspace;
  hipError_t e = dspark::launch_norm_backward(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

namespace {

bool recurrence_sizes_fit(int T, int S, int C) {
  return T >= 0 && S >= 0 && C >= 0 && T <= dspark::kMaxTokens && S <= dspark::kMaxRows && C <= kMaxD;
}
bool known_gate(dspark_gate k) { return k == DSPARK_GATE_SIGMOID || k == DSPARK_GATE_DECAY; }

// Checks shared by the recurrence and its gradient.
dspark_status recurrence_inputs(const dspark::RecurrenceArgs& a, dspark_dtype dtype, dspark_gate kind) {
  if (a.T < 0 || a.S < 0 || a.C < 0) return fail(DSPARK_ERR_INVALID_ARG, "negative size");
  if (!known_dtype(dtype)) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype");
  if (!known_gate(kind)) return fail(DSPARK_ERR_INVALID_ARG, "unknown gate");
  if (a.T > dspark::kMaxTokens) return fail(DSPARK_ERR_UNSUPPORTED, "T > 2^24");
  if (a.S > dspark::kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "S > 2^20");
  if (a.C > kMaxD) return fail(DSPARK_ERR_UNSUPPORTED, "C > 65536");
  if (!a.offsets && (a.S == 0 ? a.T > 0 : a.T % a.S != 0))
    return fail(DSPARK_ERR_INVALID_ARG, "without offsets S has to divide T");
  if (a.T > 0 && a.C > 0 && !a.x) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (!a.gate && a.C > 0 && (a.T > 0 || !a.sigmoid)) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = a.bf16 ? 2 : 4;
  if (misaligned(a.x, elem) || misaligned(a.gate, a.sigmoid ? elem : 4) || misaligned(a.offsets, 4) ||
      misaligned(a.h0, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  return DSPARK_OK;
}

dspark::RecurrenceArgs recurrence_args(int T, int S, int C, dspark_dtype dtype, dspark_gate kind,
                                       const int32_t* offsets, const void* x, const void* gate, const float* h0,
                                       void* ws) {
  dspark::RecurrenceArgs a = {};
  a.T = T;
  a.S = S;
  a.C = C;
  a.bf16 = dtype == DSPARK_BF16;
  a.sigmoid = kind == DSPARK_GATE_SIGMOID;
  a.offsets = offsets;
  a.x = x;
  a.gate = gate;
  a.h0 = h0;
  a.ws = ws;
  return a;
}

// Bytes of the arrays by row and channel, of the gate, by sequence and of the kept states.
struct RecurrenceBytes {
  size_t rows, gate, ends, states, offsets;
};
RecurrenceBytes recurrence_bytes(const dspark::RecurrenceArgs& a) {
  const size_t c = size_t(a.C), rows = size_t(a.T) * c * (a.bf16 ? 2 : 4);
  return {rows, a.sigmoid ? rows : c * 4, size_t(a.S) * c * 4,
          (size_t(a.T) + DSPARK_RECURRENCE_BLOCK - 1) / DSPARK_RECURRENCE_BLOCK * c * 4, (size_t(a.S) + 1) * 4};
}

}  // namespace

size_t dspark_recurrence_workspace_bytes(int T, int S, int C, dspark_dtype dtype, dspark_gate kind) {
  if (!recurrence_sizes_fit(T, S, C) || !known_dtype(dtype) || !known_gate(kind) || T == 0 || S == 0 || C == 0) return 0;
  return dspark::recurrence_workspace_bytes(T, S, C, dtype == DSPARK_BF16, kind == DSPARK_GATE_SIGMOID);
}

dspark_status dspark_recurrence(int T, int S, int C, dspark_dtype dtype, dspark_gate kind, const int32_t* offsets,
                                const void* x, const void* gate, const float* h0, void* h, float* last, float* states,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark::RecurrenceArgs a = recurrence_args(T, S, C, dtype, kind, offsets, x, gate, h0, workspace);
  dspark_status st = recurrence_inputs(a, dtype, kind);
  if (st != DSPARK_OK) return st;
  if (C == 0 || S == 0 || (T == 0 && !last)) return DSPARK_OK;
  if (T > 0 && !h) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  if (misaligned(h, a.bf16 ? 2 : 4) || misaligned(last, 4) || misaligned(states, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_recurrence_workspace_bytes(T, S, C, dtype, kind);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_recurrence_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const RecurrenceBytes n = recurrence_bytes(a);
  if (any_overlap({{h, n.rows}, {last, n.ends}, {states, n.states}, {workspace, need}},
                  {{offsets, n.offsets}, {x, n.rows}, {gate, n.gate}, {h0 == last ? nullptr : h0, n.ends}}) ||
      any_overlap({{h, n.rows}, {states, n.states}, {workspace, need}}, {{h0, n.ends}}))
    return overlap_refused();
  a.h = h;
  a.last = last;
  a.states = states;
  hipError_t e = dspark::launch_recurrence(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

size_t dspark_recurrence_backward_workspace_bytes(int T, int S, int C, dspark_dtype dtype, dspark_gate kind) {
  if (!recurrence_sizes_fit(T, S, C) || !known_dtype(dtype) || !known_gate(kind) || S == 0 || C == 0) return 0;
  return dspark::recurrence_backward_workspace_bytes(T, S, C, dtype == DSPARK_BF16, kind == DSPARK_GATE_SIGMOID);
}

dspark_status dspark_recurrence_backward(int T, int S, int C, dspark_dtype dtype, dspark_gate kind,
                                         const int32_t* offsets, const void* dh, const void* x, const void* gate,
                                         const float* h0, const float* dlast, const float* states, void* dx,
                                         void* dgate, float* dh0, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
  g_last_error[0] = '\0';
  dspark::RecurrenceArgs a = recurrence_args(T, S, C, dtype, kind, offsets, x, gate, h0, workspace);
  dspark_status st = recurrence_inputs(a, dtype, kind);
  if (st != DSPARK_OK) return st;
  if (C == 0 || (!dx && !dgate && !dh0)) return DSPARK_OK;
  if (T > 0 && S > 0 && (!dh || !states)) return fail(DSPARK_ERR_INVALID_ARG, "null pointer argument");
  const size_t elem = a.bf16 ? 2 : 4;
  if (misaligned(dh, elem) || misaligned(dx, elem) || misaligned(dgate, a.sigmoid ? elem : 4) ||
      misaligned(dlast, 4) || misaligned(states, 4) || misaligned(dh0, 4))
    return fail(DSPARK_ERR_INVALID_ARG, "misaligned tensor");
  const size_t need = dspark_recurrence_backward_workspace_bytes(T, S, C, dtype, kind);
  st = check_workspace(workspace, workspace_bytes, need, "dspark_recurrence_backward_workspace_bytes");
  if (st != DSPARK_OK) return st;
  const RecurrenceBytes n = recurrence_bytes(a);
  if (any_overlap({{dx, n.rows}, {dgate, n.gate}, {dh0, n.ends}, {workspace, need}},
                  {{offsets, n.offsets},
                   {dh, n.rows},
                   {x, n.rows},
                   {gate, n.gate},
                   {h0, n.ends},
                   {dlast == dh0 ? nullptr : dlast, n.ends},
                   {states, n.states}}) ||
      any_overlap({{dx, n.rows}, {dgate, n.gate}, {workspace, need}}, {{dlast, n.ends}}))
    return overlap_refused();
  a.dh = dh;
  a.dlast = dlast;
  a.states_in = states;
  a.dx = dx;
  a.dgate = dgate;
  a.dh0 = dh0;
  hipError_t e = dspark::launch_recurrence_backward(a, stream);
  if (e != hipSuccess) return hip_fail(e);
  return DSPARK_OK;
}

}  // extern "C"
