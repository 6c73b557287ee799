/*
 * muon.h - C ABI of libmuon.so, the Muon / MuonGS optimizer step for a stack of
 * 2-D weight matrices on NVIDIA B200 (sm_100a).
 *
 * What one step computes, per matrix W (rows x cols, the storage shape; an
 * nn.Linear weight is (out, in)):
 *   a1  M_t = mu*M_{t-1} + G_t                       (SGD momentum)
 *   a2  U   = G_t + mu*M_t     (Nesterov; U = M_t without MUON_NESTEROV)
 *   a3  X_0 = U / (||U||_F + eps)
 *   a4  tall matrices (rows > cols) are iterated through X^T (exact identity)
 *   a5  ns_steps times: S = X X^T; P = b*S + c*S*S; X = a*X + P*X
 *   a6  optional row-or-column RMS equilibration          (MUON_EQUILIBRATE)
 *   a7  O = s*O, s = scale_k*sqrt(max(rows, cols))       (MUON_SCALE_MOONLIGHT)
 *   a8  MuonGS: O~ = O - (<W,O>_F / ||W||_F^2) W         (MUON_MODE_MUONGS)
 *   a9  W <- (1 - lr*weight_decay) W - lr*O~
 * Sources (page title, section):
 *   "LLM Pretraining Loss Spike 진단과 처방 ... 그리고 Muon 전환 판단", section
 *     "AdamW에서 Muon으로 갈아탈 것인가": the Newton-Schulz listing (a3, a5, the
 *     Keller shape correction), the defaults (lr 0.02, momentum 0.95, Nesterov,
 *     5 steps) and the Moonlight sub-section (decoupled weight decay, a7, a9).
 *   "MuonGS: Pretraining LLMs with Relaxed Weight-Norm Control", section
 *     "전제와 한계": the Gram-Schmidt projection a8 and the C_T statistics.
 *   "[논문 AI 리뷰] MUON IS SCALABLE FOR LLM TRAINING TECHNICAL REPORT", section 2:
 *     the Newton-Schulz recurrence (a5) and the Eq. 4 update scale (a7).
 *   "행과 열을 함께 정규화하는 사전학습 옵티마이저 MeqMuon 공개", section "핵심 내용":
 *     row or column normalisation of the orthogonalised update (a6).
 *   "[Deep Learning] Muon — 행렬 업데이트를 직교화하는 옵티마이저", sections 3 and 5:
 *     the step order and the API conventions (a list of 2-D params; lr,
 *     momentum, weight_decay; a non-2-D parameter is an error).
 *
 * Precision: G is bf16 or fp32, W and M are fp32 and are updated in place.
 * Default Newton-Schulz path: bf16 operands on the tcgen05 tensor cores with
 * fp32 accumulation; X, S and P are stored in bf16 between the GEMMs, as in the
 * printed listing. MUON_NS_FP32 runs the iteration in fp32 on the CUDA cores.
 *
 * Conventions common to every call:
 *   - All matrix pointers are DEVICE pointers owned by the caller. The library
 *     never allocates device memory: scratch space is the caller's workspace.
 *   - Matrices are row-major with a leading dimension (elements) >= cols.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls are asynchronous on that stream and never synchronise, except
 *     muon_query_device_status.
 *   - Host-side validation happens before anything is enqueued; on error the
 *     call returns the status and nothing runs.
 *   - A plan object is not thread-safe; distinct plans may be used concurrently
 *     on distinct streams with distinct workspaces.
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 1

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1,  /* null pointer, bad enum, n < 0, bad hyper-parameter */
  MUON_ERR_SHAPE = 2,        /* rows or cols < 1, ld < cols, rows*cols >= 2^31 */
  MUON_ERR_DTYPE = 3,        /* W must be F32; grad F32 or BF16 */
  MUON_ERR_ALIAS = 4,        /* a written buffer (W, momentum) overlaps another buffer */
  MUON_ERR_WORKSPACE = 5,    /* workspace null, misaligned (256 B) or too small */
  MUON_ERR_CUDA = 6,         /* a CUDA runtime/driver call or a launch failed */
  MUON_ERR_TIMEOUT = 7,      /* device side: a bounded wait inside a kernel gave up */
  MUON_ERR_UNSUPPORTED = 8   /* the current device is not sm_100 (B200) */
} muon_status_t;

typedef enum { MUON_F32 = 0, MUON_BF16 = 1 } muon_dtype_t;

typedef enum {
  MUON_MODE_MUON = 0,    /* plain Muon (with decoupled weight decay when wd > 0) */
  MUON_MODE_MUONGS = 1,  /* MuonGS: radial (Gram-Schmidt) projection before the update */
  MUON_MODE_MUONH = 2,   /* MuonH: fixed radius, W_{t+1} = ||W_t|| W' / ||W'|| with W' the
                            plain Muon update ("MuonGS: Pretraining LLMs with Relaxed
                            Weight-Norm Control", section 무엇과 다른가, names fixed-norm
                            control; the retraction form is this library's reading) */
  MUON_MODE_TWOSIDED = 3 /* for 2-D parameters that are not orthogonalised ("행과 열을 함께
                            정규화하는 ... MeqMuon 공개", section 핵심 내용): no Newton-Schulz;
                            the Frobenius-normalised Nesterov direction X is normalised along
                            rows and columns at once, N_ij = X_ij rho / ((sqrt(r_i)+eps)
                            (sqrt(c_j)+eps)), r / c the row / column mean squares of X and rho
                            its RMS (this library's reading; no formula on the page). Use
                            scale MUON_SCALE_NONE for an update of RMS about 1. ns_steps and
                            MUON_EQUILIBRATE are ignored; stats report w_norm only (the
                            other fields are NaN). */
} muon_mode_t;

typedef enum {
  MUON_SCALE_MOONLIGHT = 0, /* s = scale_k * sqrt(max(rows, cols)), scale_k = 0.2 by default */
  MUON_SCALE_KELLER = 1,    /* s = sqrt(max(1, rows/cols)) */
  MUON_SCALE_NONE = 2       /* s = 1 */
} muon_scale_t;

enum {
  MUON_NESTEROV = 1u,      /* U = G + mu*M (else U = M) */
  MUON_EQUILIBRATE = 2u,   /* row-or-column RMS equilibration after orthogonalisation */
  MUON_NS_FP32 = 4u,       /* fp32 Newton-Schulz on CUDA cores (else bf16 tensor cores) */
  MUON_WANT_STATS = 8u     /* reserved; stats are written whenever stats_dev != NULL */
};

/* One weight matrix. W: F32, updated in place. grad: F32 or BF16, read only.
 * momentum: F32, updated in place (it holds M_t after the call; zero it before
 * the first step). Leading dimensions are in elements. */
typedef struct {
  void* W;
  const void* grad;
  void* momentum;
  int64_t rows, cols;
  int64_t ld_w, ld_g, ld_m;
  int32_t w_dtype;   /* muon_dtype_t, must be MUON_F32 */
  int32_t g_dtype;   /* muon_dtype_t */
} muon_matrix_t;

typedef struct {
  float lr;              /* eta, 0.02 by default */
  float momentum;        /* mu, 0.95 */
  float weight_decay;    /* lambda, 0 (decay multiplies lr: W <- (1 - lr*wd) W) */
  float ns_coeffs[3];    /* (a, b, c) = (3.4445, -4.7750, 2.0315) */
  int32_t ns_steps;      /* 5; 0 <= ns_steps <= 64 */
  float eps;             /* 1e-7, added to ||U||_F (and to row/col RMS in a6) */
  int32_t mode;          /* muon_mode_t */
  int32_t scale;         /* muon_scale_t */
  float scale_k;         /* 0.2 */
  uint32_t flags;        /* MUON_NESTEROV | ... ; default MUON_NESTEROV */
} muon_hparams_t;

/* Per-matrix statistics of the step just taken (device memory, one entry per
 * matrix in the caller's order). C_T of the MuonGS page accumulates lr/w_norm. */
typedef struct {
  float w_norm;       /* ||W_t||_F before the step */
  float w_dot_o;      /* <W_t, O>_F with O after equilibration and scale */
  float o_norm;       /* ||O~||_F, the applied direction */
  float update_rms;   /* ||O~||_F / sqrt(rows*cols) */
  int32_t equil_axis; /* 0 none, 1 rows, 2 columns */
  int32_t reserved;
} muon_stats_t;

/* Library ABI version (MUON_ABI_VERSION). */
MUON_API int muon_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
MUON_API const char* muon_status_string(muon_status_t status);

/* Fills *hp with the defaults listed in muon_hparams_t. */
MUON_API muon_status_t muon_hparams_default(muon_hparams_t* hp);

/* Host-only validation of a matrix list and hyper-parameters (no CUDA call). */
MUON_API muon_status_t muon_validate(const muon_matrix_t* mats, int n, const muon_hparams_t* hp);

/* Workspace bytes muon_step_batched needs for this list (0 if the list is
 * invalid). Host only. The workspace must be 256-byte aligned device memory. */
MUON_API size_t muon_workspace_size(const muon_matrix_t* mats, int n, const muon_hparams_t* hp);

/* One step over n matrices. Groups the matrices by shape on the host, copies a
 * descriptor table into the workspace and launches the kernels on `stream`.
 * stats_dev: device array of n muon_stats_t, or NULL. n == 0 is a no-op. */
MUON_API muon_status_t muon_step_batched(const muon_matrix_t* mats, int n, const muon_hparams_t* hp,
                                void* workspace, size_t ws_bytes, muon_stats_t* stats_dev,
                                void* stream);

/* ---- cached plan: grouping and descriptor table built once for a fixed list ---- */
typedef struct muon_plan_s* muon_plan_t;

/* Validates and groups the list (host only, no CUDA call). On success *out owns
 * a copy of the list; the pointers inside must stay valid while the plan is used. */
MUON_API muon_status_t muon_plan_create(const muon_matrix_t* mats, int n, const muon_hparams_t* hp,
                               muon_plan_t* out);
MUON_API size_t muon_plan_workspace_size(muon_plan_t plan);
/* Replaces the hyper-parameters (e.g. a learning-rate schedule). Flags that change
 * the workspace layout (MUON_NS_FP32, MUON_EQUILIBRATE) must not change. */
MUON_API muon_status_t muon_plan_set_hparams(muon_plan_t plan, const muon_hparams_t* hp);
/* One step. The descriptor table is uploaded into the workspace on the first call
 * with a given workspace pointer and reused afterwards. */
MUON_API muon_status_t muon_plan_step(muon_plan_t plan, void* workspace, size_t ws_bytes,
                             muon_stats_t* stats_dev, void* stream);
MUON_API void muon_plan_destroy(muon_plan_t plan);

/* ---- Newton-Schulz only: O = NS(X / (||X||_F + eps)), for tests and benchmarks ----
 * X and O are device matrices of the given dtype (X and O may not overlap).
 * Uses ns_coeffs, ns_steps, eps and MUON_NS_FP32 from hp; other fields ignored.
 * The workspace size is muon_ns_workspace_size for the same list. */
typedef struct {
  const void* X;
  void* O;
  int64_t rows, cols, ld_x, ld_o;
  int32_t dtype;     /* MUON_F32 or MUON_BF16, for both X and O */
  int32_t reserved;
} muon_ns_matrix_t;

MUON_API size_t muon_ns_workspace_size(const muon_ns_matrix_t* mats, int n, const muon_hparams_t* hp);
MUON_API muon_status_t muon_newton_schulz_batched(const muon_ns_matrix_t* mats, int n,
                                         const muon_hparams_t* hp, void* workspace,
                                         size_t ws_bytes, void* stream);

/* ---- per-kernel device timing of a plan (CUDA events around each launch) ----
 * Kernel kinds: "ingest", "ns_gram", "ns_poly", "ns_apply", "post_reduce",
 * "post_finalize", "post_apply", "ns_fused" (the fp32 path's single launch over all
 * iterations of small matrices), "post_stats" (the statistics of MUON_MODE_MUON and
 * MUON_MODE_TWOSIDED, after post_apply). flops / bytes are the algorithmic work of the
 * recorded launches: Newton-Schulz flops count the symmetric Gram and polynomial
 * once (m(m+1)n and m^2(m+1)) and the apply 2m^2n; bytes count each kernel's own
 * inputs and outputs once (ingest: G, M read, M and X_0 written; post_reduce: W and
 * O read, or O alone in MUON_MODE_MUON and MUON_MODE_TWOSIDED, whose update needs no
 * scalar of W; post_apply: W read and written, O read). */
typedef struct {
  char name[32];
  int32_t launches;   /* launches recorded since the last read */
  float total_ms;     /* their summed device time */
  double flops;       /* their algorithmic flops */
  double bytes;       /* their algorithmic bytes */
} muon_profile_entry_t;

/* Turns event recording on (1) or off (0) for later muon_plan_step calls. */
MUON_API muon_status_t muon_plan_profile_enable(muon_plan_t plan, int enable);
/* Waits for the recorded events, writes up to max_entries kinds (in the order
 * listed above) and clears the record. Returns the number of kinds written,
 * or -1 on a CUDA error. */
MUON_API int muon_plan_profile_read(muon_plan_t plan, muon_profile_entry_t* out, int max_entries);

/* ---- Newton-Schulz of one matrix without any caller workspace ----
 * The pages have no counterpart of this call: it exists for callers that cannot
 * call cudaMalloc. Examples: code that runs under a memory pool or framework
 * allocator owning all device memory, which must not be bypassed; code that
 * cannot afford the device-wide synchronisation cudaMalloc/cudaFree may imply.
 * Same result as muon_newton_schulz_batched for that one matrix (X in, O out,
 * device pointers, dtype F32 or BF16 for both): the arguments are validated by
 * the same host checks (so they get the same status) and the same kernels and tile
 * shapes run. Scratch is the library's own
 * 32 MiB static device array, which every GPU that loads the library keeps
 * until exit. A matrix whose scratch needs exceed it is rejected with
 * MUON_ERR_WORKSPACE before anything is enqueued. In bf16 that is 2*(m*ld_n +
 * m*ld_m)*2 bytes plus 2 KiB, with m <= n the sorted sides and ld_* rounded up
 * to 64, so 1024 x 4096 fits and 2048 x 2048 does not.
 * All calls share that array: calls that overlap on the GPU (two streams or
 * two host threads) race and must be serialised by the caller. The first call
 * on each device looks up the array's device address (cudaGetSymbolAddress,
 * with that device current), so make it before any stream capture.
 * status_dev: optional uint32 in device memory of the current device (anything
 * else is rejected with MUON_ERR_INVALID_ARG) that receives MUON_ERR_TIMEOUT if a
 * bounded wait inside a kernel gives up; it is cleared to 0 at the start of the
 * call. With status_dev == NULL a timeout is not reported anywhere: the word it
 * lands in belongs to the shared scratch and the next call clears it, and O may
 * then hold garbage. Pass a status word whenever the result matters. */
MUON_API muon_status_t muon_newton_schulz_noalloc(const muon_ns_matrix_t* mat,
                                                  const muon_hparams_t* hp, uint32_t* status_dev,
                                                  void* stream);

/* ---- QK-Clip (MuonClip) ----
 * "LLM Pretraining Loss Spike 진단과 처방", section "Moonlight와 MuonClip이 추가한 것"
 * (QK-Clip listing): for attention head h whose largest pre-softmax logit S_max[h]
 * exceeds tau, gamma_h = tau / S_max[h] (else 1); the head's non-rotary query and key
 * projection rows are multiplied by gamma_h^0.5, its rotary query rows by gamma_h,
 * and the rotary key shared by all heads is not touched.
 * A slice names rows [row0, row0 + rows) of a row-major fp32 device matrix W (all
 * `cols` columns, leading dimension ld) that belong to head `head` and are scaled by
 * gamma_head^power (0.5 or 1.0 in the listing). s_max_dev: device array of n_heads
 * floats (the caller's forward pass measures them). Slices of one call may not
 * overlap (MUON_ERR_ALIAS; a slice of zero rows overlaps nothing). cols is at most
 * 2^26 (MUON_ERR_SHAPE). Asynchronous on `stream`; no workspace. */
typedef struct {
  void* W;
  int64_t row0, rows, cols, ld;
  int32_t head;
  float power;
} muon_qk_slice_t;

MUON_API muon_status_t muon_qk_clip(const muon_qk_slice_t* slices, int n, const float* s_max_dev,
                                    int n_heads, float tau, void* stream);

/* ---- the step's inputs: 8-bit activation checkpoints, weight gradients, attention ----
 * muon_plan_step reads one gradient per matrix and muon_qk_clip the largest attention
 * logit of every head. The calls below produce both from a training step's own tensors.
 * They are asynchronous on `stream`, allocate nothing and can be captured into a graph.
 * Calls that write the same buffers, or share a workspace, must be ordered by the caller.
 *
 * status_dev (where present): optional uint32 in device memory that receives
 * MUON_ERR_TIMEOUT if a bounded wait inside a kernel gives up (the outputs may then hold
 * garbage). The calls never clear it: zero it before its first use. */

/* One activation X (rows x cols, row-major, F32 or BF16) and its 8-bit checkpoint: int8
 * values q (rows x cols, ld_q) and one power-of-two scale per row and group of 32
 * columns, held as a biased exponent byte (rows x ceil(cols/32), ld_e):
 *   amax = max |x| over the group, E = max(floor(log2 amax) - 6, -126), byte = E + 127
 *   q = clamp(round_half_even(x 2^-E), -127, 127),      restored value = q 2^E
 * |x - q 2^E| <= 2^E / 2 (2^E where |x| rounds past 127), 2^E <= amax / 64. A restored
 * value has 7 significant bits, so BF16 and F32 hold it exactly. A group with a NaN or an
 * infinity gets byte 255 and zeros: byte 255 stands for an infinite scale, so the group
 * restores as NaN throughout. Byte 0 stands for a scale of zero; store never writes it.
 * q and exps are 16-byte aligned, ld_q and ld_e multiples of 16; every leading dimension is at
 * least the width (MUON_ERR_SHAPE), so that no two rows share an address. rows may be 0. Bytes of q
 * and exps beyond cols are neither read nor written. */
typedef struct {
  void* X;             /* read by muon_act8_store, written by muon_act8_restore */
  int8_t* q;
  uint8_t* exps;
  int64_t rows, cols, ld_x, ld_q, ld_e;
  int32_t dtype;       /* muon_dtype_t of X */
  int32_t reserved;
} muon_act8_t;

/* Stores / restores n activations, up to 128 per launch. Nothing written may overlap
 * anything else of the call (MUON_ERR_ALIAS). A matrix counts from its first to its last
 * element here: two column slices of one buffer are written by two calls. */
MUON_API muon_status_t muon_act8_store(const muon_act8_t* items, int n, void* stream);
MUON_API muon_status_t muon_act8_restore(const muon_act8_t* items, int n, void* stream);

/* Weight gradients from a checkpoint. For each group g of consecutive tokens:
 *   dW_g[o, i] (+)= sum over t in [offsets[g], offsets[g+1]) of dY[t, o] q[t, i] 2^E[t, i/32]
 * One group is a dense matrix, several are the experts of a layer, with their tokens
 * sorted by expert; a group may be empty (dW_g = 0, or left alone with accumulate).
 * dY (tokens x out) is BF16, 16-byte aligned, ld_dy a multiple of 8. dW is F32 or BF16,
 * aligned to its element: group g starts stride_w elements after group g - 1, rows are
 * ld_w apart. Products are exact, sums are FP32, and a BF16 dW (with accumulate: its sum
 * with the old value) is rounded once. offsets: groups + 1 int32 in device memory (NULL:
 * one group of all tokens); each is read as clamped to [0, tokens], and a group whose end
 * lies before its start is empty. Tokens outside every group are not read.
 * The workspace (256-byte aligned) may be NULL when muon_weight_grad_workspace_size is 0. */
typedef struct {
  const void* dY;
  const int8_t* q;
  const uint8_t* exps;
  void* dW;
  const int32_t* offsets;
  uint32_t* status_dev;
  int64_t tokens, out, in;
  int64_t ld_dy, ld_q, ld_e, ld_w, stride_w;
  int32_t groups;
  int32_t w_dtype;     /* muon_dtype_t of dW */
  int32_t accumulate;  /* 0: dW = sum, 1: dW += sum */
  int32_t reserved;
} muon_weight_grad_t;

MUON_API size_t muon_weight_grad_workspace_size(const muon_weight_grad_t* a);
MUON_API muon_status_t muon_weight_grad(const muon_weight_grad_t* a, void* workspace,
                                        size_t ws_bytes, void* stream);

/* Softmax attention over packed sequences, with what its backward pass and QK-Clip need.
 * Sequence s has the query rows [q_offsets[s], q_offsets[s+1]) and the keys
 * [k_offsets[s], k_offsets[s+1]); query head h reads key head h / (heads / kv_heads).
 *   S_ij = scale q_i . k_j for the visible keys: all of the sequence, or with causal, of m
 *          queries and n keys, j <= i + n - m (rows aligned at the end of the keys)
 *   lse_i = log sum_j exp(S_ij),  o_i = sum_j exp(S_ij - lse_i) v_j
 *   s_max[h] = max(s_max[h], largest S_ij of head h over all sequences)
 * A row that sees no key has o = 0 and lse = -inf. s_max is raised, never lowered, so it
 * collects the maximum over micro-batches: set it to -inf before the first (NaN logits do
 * not raise it). Rows outside every sequence are not written, and what they hold does not
 * matter.
 * The backward pass recomputes P = exp(S - lse) and needs the forward pass's o and lse:
 *   delta_i = o_i . dout_i,  dV = P^T dout,  dS = P (dout V^T - delta)
 *   dQ = scale dS K,  dK = scale dS^T Q   (dK and dV summed over the heads of a key head)
 * o and lse may be those of more keys than the call's: the gradients are then these keys'
 * terms of the whole. A row whose softmax is one key alone has dQ = 0 exactly.
 * Keys that no row sees get zero gradients. Sums are taken in a fixed order: the results
 * of equal calls are equal bit for bit.
 * Tensors q, o, dout, dq (q_tokens x heads x head_dim) and k, v, dk, dv (k_tokens x
 * kv_heads x head_dim) are BF16 with unit stride along head_dim, 16-byte aligned, their
 * token and head strides (in elements) multiples of 8. Views of one buffer (packed q, k,
 * v) may interleave; no two elements of a tensor share an address, also of those only read
 * (broadcast heads or tokens are refused: MUON_ERR_SHAPE). lse is heads x q_tokens F32,
 * contiguous. head_dim is a multiple of 8 up to 128, the same for q, k and v; scale is
 * positive and finite (MUON_ERR_INVALID_ARG).
 * All sums are FP32. P (both passes) and dS are rounded to BF16 for the products. The backward
 * pass adds the product with that rounding's rest where it costs little: in dQ of 128 rows that
 * see at most 128 keys, and in dK and dV of keys that at most 128 rows see (of one query head, or
 * of a few that several blocks share). With head_dim up to 64 it does so only in calls of up to
 * 296 tiles of 128 rows or keys, so that the gradients of a short sequence may be more exact alone
 * than packed with many others (relative error 0.0017 against 0.0024), within the same bound.
 * Offsets are n_seq + 1 int32 in device memory; with n_seq == 1 either pointer may be NULL,
 * which stands for all rows (q_offsets) or all keys (k_offsets), with more neither may
 * (MUON_ERR_INVALID_ARG). Each offset is read as clamped to [0, tokens], and a sequence whose
 * end lies before its start is empty. Offsets must not decrease. A NaN or infinity of a sequence stays within it. */
typedef struct {
  void* ptr;
  int64_t ld;          /* stride between tokens */
  int64_t head;        /* stride between heads */
} muon_heads_t;

typedef struct {
  muon_heads_t q, k, v, o;
  muon_heads_t dout, dq, dk, dv;   /* backward only */
  float* lse;
  float* s_max;                    /* heads floats or NULL; forward only */
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  uint32_t* status_dev;
  int64_t q_tokens, k_tokens;
  int32_t n_seq;
  int32_t heads, kv_heads, head_dim;
  int32_t causal;
  float scale;
} muon_attention_t;

MUON_API muon_status_t muon_attention_forward(const muon_attention_t* a, void* stream);
/* The backward pass's scratch: 4 bytes per head and query row, rounded up. */
MUON_API size_t muon_attention_workspace_size(const muon_attention_t* a);
MUON_API muon_status_t muon_attention_backward(const muon_attention_t* a, void* workspace,
                                               size_t ws_bytes, void* stream);

/* Self-test of the device-side timeout path: launches one thread that waits, with
 * the same bounded wait the pipelined kernels use, on an mbarrier nothing arrives
 * at, for limit_cycles SM clock cycles (1 .. 2e9), then records MUON_ERR_TIMEOUT
 * in the workspace's error word (read it with muon_query_device_status). The
 * workspace needs only its first 256 bytes. Nothing faults and nothing hangs. */
MUON_API muon_status_t muon_wait_probe(void* workspace, int64_t limit_cycles, void* stream);

/* Reads the sticky device-side error word of the workspace (MUON_OK or
 * MUON_ERR_TIMEOUT) behind the work already enqueued on `stream`, clears it on that
 * stream, and synchronises `stream` only (no other stream and no device-wide wait). The word is zeroed when
 * a plan first uses a workspace and on every muon_step_batched /
 * muon_newton_schulz_batched call, so after those it reflects that call only. */
MUON_API muon_status_t muon_query_device_status(void* workspace, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_H_ */
