// Host-side launch interface between the C ABI layer (api.cpp) and the
// kernel translation units.  Arguments arrive here already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dspark {

// Upper bound on the draft kernel's grid (one workgroup per compute unit).
constexpr int kMaxDraftWorkgroups = 512;
// Largest number of requests one workgroup can own for the confidence epilogue.
constexpr int kMaxOwnedRows = 64;
// Requests per group in the draft kernel (LDS holds one group's embeddings).
constexpr int kMaxGroupRows = 128;
// Batches of at most this many requests (one group of at most 16 rows)
// synchronise the draft positions through per-workgroup winner keys instead
// of arrival counters.
constexpr int kSmallBatch = 16;
// Distance (in 32-bit words) between the per-group arrival counters (one
// 128-byte line each: every workgroup polls them).
constexpr int kBarStride = 32;
// Scheduler: one workgroup sorts all (request, position) keys in LDS.
constexpr int kMaxScheduleItems = 16384;
// dspark_step runs draft, schedule and verify in one launch up to this many
// verify candidates (B * gamma), and makes three launches above it.
constexpr int kFusedStepItems = 1024;

// The schedule and verify part of a fused step (dspark_step).
struct StepArgs {
  const double* t_step;
  int n_min, n_count;
  const int32_t* target;
  int32_t *lens, *m_out, *accepted, *bonus;
  void* sched_ws;   // the scheduler's workspace (schedule_workspace_bytes)
};

struct DraftArgs {
  int B, gamma, V, r, d;
  bool bf16, gumbel;
  uint64_t seed;
  const int32_t* anchor;
  const void *U, *h, *W1, *W2;
  const float* conf_w;
  float conf_b;
  const float* sts_T;
  int32_t* tokens;
  float *logit, *conf, *surv;
  void* ws;
  size_t ws_bytes;
  bool exclusive;   // plain launch: the caller guarantees nothing else runs on the device
  const float* decay = nullptr;   // non-null: RNN head with this per-channel state decay [r] (bf16 only)
  bool noalloc = false;           // ws ignored: the per-device static scratch is used (Markov head)
  bool check_only = false;        // nothing is launched: the shape's checks alone
  const StepArgs* step = nullptr;  // non-null: schedule and verify in the same launch when the shape allows
};

// Workspace carve-up of the draft call (byte offsets, 256-aligned).  Every
// section before zpart must be zero when a call starts (each call leaves it
// so); wkeys and wz are empty unless B <= kSmallBatch.
struct DraftWorkspace {
  size_t ctrl, bar, slots, wkeys, wz, zpart, hdot, state, total;
};
// r_state: the RNN head's rank (its bf16 state [2][B][r] is carved out too), 0 for the Markov head.
DraftWorkspace draft_workspace_layout(int B, int gamma, int r_state);

// Returns hipSuccess or the first HIP error; sets *unsupported (with a reason)
// when the shape is outside what the kernels handle.
// *fused (optional) tells whether the schedule and verify of a.step ran in the
// same launch (else the caller launches them).
hipError_t launch_markov_draft(const DraftArgs& a, hipStream_t stream, const char** unsupported,
                               bool* fused = nullptr);

// Allocation-free draft entry point: size of the per-device static scratch
// that replaces the caller's workspace, and its device address (set up and
// zero-filled on `stream` at the first call on the current device).
constexpr size_t kNoAllocScratchBytes = size_t(8) << 20;
// A call whose shape (B << 32 | gamma) differs from the previous one on the
// device clears the first zero_bytes (its counters and slots) first.
hipError_t noalloc_scratch(hipStream_t stream, void** out, uint64_t shape, size_t zero_bytes);

// Bytes of the multi-workgroup scheduler's workspace (0 for B*gamma == 0 or
// above kMaxScheduleItems).
size_t schedule_workspace_bytes(int B, int gamma);
// workspace == nullptr: the one-workgroup kernel; else the multi-workgroup
// kernel on a workspace of schedule_workspace_bytes(B, gamma) bytes.
hipError_t launch_schedule(int B, int gamma, const float* surv, const double* t_step, int n_min, int n_count,
                           int32_t* lens, int32_t* m_out, double* objective, void* workspace, hipStream_t stream);

hipError_t launch_schedule_threshold(int B, int gamma, const float* surv, float tau, int32_t* lens, int32_t* m_out,
                                    hipStream_t stream);

hipError_t launch_parallel_draft(int B, int gamma, int V, bool bf16, const void* U, bool gumbel, uint64_t seed,
                                 int32_t* tokens, float* logit, hipStream_t stream);
hipError_t launch_gumbel_words(int n, const uint32_t* words, float* out, hipStream_t stream);

// Sequential-temperature fit: limits of one workgroup's LDS histogram.
constexpr int kMaxStsGrid = 4096;
constexpr int kMaxStsBins = 256;
constexpr int kMaxStsHist = 8192;     // nbins * G
constexpr int kMaxStsBlocks = 1 << 24;

struct StsArgs {
  int N, gamma, G, nbins;
  const float* logit;
  const int32_t* accepted;
  const float* grid;
  int32_t* choice;
  float* T_out;
  double* ece;
  void* ws;
};

struct StsWorkspace {
  size_t ctrl, hist, S, total;
};
StsWorkspace sts_workspace_layout(int N, int G, int nbins);
size_t sts_lds_bytes(int G, int nbins);

hipError_t launch_sts_fit(const StsArgs& a, hipStream_t stream);

hipError_t launch_verify(int B, int gamma, const int32_t* tokens, const int32_t* target,
                         const int32_t* lens, int32_t* accepted, int32_t* bonus, hipStream_t stream);

// Linear layer (x [M][K], w [N][K]) and its gradients.
struct LinearArgs {
  int M, N, K;
  bool bf16;
  int act;
  const void *x, *w, *bias, *residual;
  void* y;
  float* pre;
  void* ws;
};
struct LinearBackwardArgs {
  int M, N, K;
  bool bf16;
  int act;
  const void *dy, *x, *w;
  const float* pre;
  void *dx, *dw, *dbias;
  void* ws;
};
constexpr int kMaxRows = 1 << 20;   // rows of the linear layer and of the loss
size_t linear_workspace_bytes(int M, int N, int K, bool bf16);
size_t linear_backward_workspace_bytes(int M, int N, int K, bool bf16, bool act);
hipError_t launch_linear(const LinearArgs& a, hipStream_t stream);
hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t stream);

// Cross entropy over the heads' logits; the gradient's members are unused by
// the forward call and the other way round.
struct LossArgs {
  int N, V, d, r;
  bool bf16;
  const int32_t *label, *prev;
  const void *U, *h, *Wo, *W1, *W2;
  float *nll, *lse;
  const float *lse_in, *g;
  void *dU, *dh, *dWo, *dW1, *dW2;
  void* ws;
};
size_t loss_workspace_bytes(int N, int V, int d, int r, bool bf16, bool backward);
hipError_t launch_markov_loss(const LossArgs& a, hipStream_t stream);
hipError_t launch_markov_loss_backward(const LossArgs& a, hipStream_t stream);

// Normalisation of rows (x [M][C]) with the residual stream's sum, and its gradients.
struct NormArgs {
  int M, C;
  bool bf16, center;   // center: layer normalisation, else root mean square
  const void *x, *residual, *w, *b;
  float eps;
  void *sum, *y;
  float* stat;
};
struct NormBackwardArgs {
  int M, C;
  bool bf16, center;
  const void *dy, *x;
  const float* stat;
  const void *w, *dsum;
  void *dx, *dw, *db;
  void* ws;
};
constexpr int kMaxChannels = 32768;   // of a normalised row: 1024 threads keep it in registers
size_t norm_backward_workspace_bytes(int M, int C, bool bf16);
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t stream);

// Gated linear recurrence over packed sequences (x [T][C]) and its gradients;
// the gradient's members are unused by the forward call and the other way
// round.
struct RecurrenceArgs {
  int T, S, C;
  bool bf16, sigmoid;   // sigmoid: gate [T][C] in the storage type, else decay: fp32 [C]
  const int32_t* offsets;
  const void *x, *gate;
  const float* h0;
  void* h;
  float *last, *states;
  const void* dh;
  const float *dlast, *states_in;
  void *dx, *dgate;
  float* dh0;
  void* ws;
};
constexpr int kMaxTokens = 1 << 24;   // rows of the recurrence
size_t recurrence_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid);
size_t recurrence_backward_workspace_bytes(int T, int S, int C, bool bf16, bool sigmoid);
hipError_t launch_recurrence(const RecurrenceArgs& a, hipStream_t stream);
hipError_t launch_recurrence_backward(const RecurrenceArgs& a, hipStream_t stream);

// Gated feed-forward projection (x [M][K], wg and wu [N][K], pre [2][M][N]) and its gradients.
struct GatedArgs {
  int M, N, K;
  bool bf16;
  int act;
  const void *x, *wg, *wu, *bg, *bu;
  void* y;
  float* pre;
  void* ws;
};
struct GatedBackwardArgs {
  int M, N, K;
  bool bf16;
  int act;
  const void *dy, *x, *wg, *wu;
  const float* pre;
  void *dx, *dwg, *dwu, *dbg, *dbu;
  void* ws;
};
size_t gated_workspace_bytes(int M, int N, int K, bool bf16);
size_t gated_backward_workspace_bytes(int M, int N, int K, bool bf16);
hipError_t launch_gated(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_backward(const GatedBackwardArgs& a, hipStream_t stream);

}  // namespace dspark
