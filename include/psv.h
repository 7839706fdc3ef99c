/*
 * psv.h — C ABI of libpsv: single-GPU serving of autoregressive-denoising
 * DiT world models on GB300 (sm_103a).
 *
 * The problem these calls serve (AREX article "vLLM 与 Physis-AI 联合介绍
 * PhysisServe 推理系统", §难题 and §三层设计; BAAI announcement
 * "智源悟界·PhysisServe：首个兼顾智能与高频吞吐的物理 AI 推理系统",
 * §新一代物理 AI 的基础设施 Fig. 1 and §PhysisServe Fig. 2–3):
 *   - a stream produces latent chunks; every chunk starts from pure noise
 *     and is denoised over S steps;
 *   - at step s and transformer block b a chunk attends to its own tokens
 *     plus the still-noisy keys/values that the W preceding chunks left at
 *     the same (block, step), so chunk c step s may run once chunk c step
 *     s-1 and chunk c-1 step s are done;
 *   - every ready (chunk, step) task of every stream is time-shared on the
 *     one GPU: a "wave" runs them all, block by block, each block as one
 *     batched launch per operation (same-block batching, Fig. 3 right).
 *
 * Conventions
 *   - every call returns 0 (PSV_OK) or a negative PSV_E* code; on error
 *     psv_last_error() describes it; PSV_ECUDA and PSV_EDEVICE are sticky;
 *   - the library never frees caller memory; host inputs are copied before
 *     a call returns, so the caller may reuse its buffers at once;
 *   - device work is issued on the caller's CUDA stream (given at create)
 *     and is asynchronous unless a call says otherwise;
 *   - all matrices are row-major; linear weights use the [out, in] layout.
 */
#ifndef PSV_H
#define PSV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define PSV_OK          0
#define PSV_EINVAL     (-1)  /* bad argument, shape or state                   */
#define PSV_ENOMEM     (-2)  /* arena too small / host allocation failed       */
#define PSV_EAGAIN     (-3)  /* nothing to return yet / queue full: retry later */
#define PSV_ETIMEDOUT  (-4)  /* psv_sync deadline passed (host-side polling)    */
#define PSV_ECUDA      (-5)  /* a CUDA runtime call failed (sticky)             */
#define PSV_EDEVICE    (-6)  /* a kernel raised its error word (sticky)         */

/* ---- create flags -------------------------------------------------------- */
#define PSV_FLAG_PLAN_ONLY   1  /* host scheduler only: no device, no arena     */
#define PSV_FLAG_SEQUENTIAL  2  /* one task per wave, lowest (stream, chunk,
                                   step) first: strictly sequential order       */
#define PSV_FLAG_CHUNK_COND  4  /* reserve per-chunk conditioning tables, for
                                   psv_submit_chunk_cond                       */
#define PSV_FLAG_LATENCY     8  /* latency mode: a wave runs only each stream's
                                   oldest ready chunk, so a chunk goes through
                                   its S steps in S consecutive waves (response
                                   time S single-chunk waves instead of S full
                                   waves), at the cost of smaller batches      */

/* ---- model description --------------------------------------------------
 * B blocks, S Euler steps (t_s = 1 - s/S), model width d = H*dh, MLP width
 * F, latent channels C (already patchified), T tokens per chunk, KV window
 * W (a chunk sees its own KV plus that of the W preceding chunks).
 * Requirements: d % 128 == 0, F % 64 == 0, dh in {32, 64, 128}, T >= 1,
 * W >= 0, 1 <= S <= 8, t_embed % 2 == 0 and <= 1024, C <= 256.
 * max_inflight: chunks of one stream alive at once (submitted and not yet
 * polled); 0 selects S + 4. */
typedef struct psv_model_desc {
  int32_t B, S, d, H, dh, F, C, T, W;
  int32_t max_streams;
  int32_t max_inflight;
  int32_t t_embed;      /* sinusoidal timestep-embedding width (256)       */
  float   ln_eps;       /* LayerNorm epsilon (1e-6)                        */
  float   rope_theta;   /* RoPE base (1e4)                                 */
  int32_t flags;        /* PSV_FLAG_*                                      */
} psv_model_desc;

/* ---- weights --------------------------------------------------------------
 * Global tensors (block = -1):
 *   IN_W [d, C]  IN_B [d]        latent -> residual stream
 *   T1_W [d, t_embed] T1_B [d]   time MLP, first layer (SiLU after it)
 *   T2_W [d, d]  T2_B [d]        time MLP, second layer
 *   FMOD_W [2d, d] FMOD_B [2d]   final adaLN: [shift_f, scale_f]
 *   OUT_W [C, d] OUT_B [C]       velocity head
 * Per block b (block = b):
 *   QKV_W [3d, d] QKV_B [3d]     rows [q | k | v], head h = rows h*dh..
 *   O_W [d, d]   O_B [d]
 *   UP_W [F, d]  UP_B [F]        GELU (tanh form) after it
 *   DOWN_W [d, F] DOWN_B [d]
 *   MOD_W [6d, d] MOD_B [6d]     adaLN: [shift1, scale1, gate1, shift2,
 *                                scale2, gate2] = MOD_W SiLU(e_s) + MOD_B
 * Matrices are stored in bf16 (f32 input is rounded to nearest even);
 * biases are stored in f32.  All tensors must be loaded before
 * psv_open_stream. */
enum {
  PSV_W_IN_W = 0, PSV_W_IN_B, PSV_W_T1_W, PSV_W_T1_B, PSV_W_T2_W, PSV_W_T2_B,
  PSV_W_FMOD_W, PSV_W_FMOD_B, PSV_W_OUT_W, PSV_W_OUT_B,
  PSV_W_QKV_W = 16, PSV_W_QKV_B, PSV_W_O_W, PSV_W_O_B, PSV_W_UP_W, PSV_W_UP_B,
  PSV_W_DOWN_W, PSV_W_DOWN_B, PSV_W_MOD_W, PSV_W_MOD_B
};
#define PSV_DTYPE_F32   0
#define PSV_DTYPE_BF16  1
#define PSV_LOC_HOST    0
#define PSV_LOC_DEVICE  1

typedef struct psv_weight {
  int32_t id;          /* PSV_W_*                                   */
  int32_t block;       /* -1 for global tensors, else 0..B-1        */
  const void* data;    /* host or device pointer, see location      */
  int32_t dtype;       /* PSV_DTYPE_F32 or PSV_DTYPE_BF16           */
  int32_t location;    /* PSV_LOC_HOST or PSV_LOC_DEVICE            */
  int64_t numel;       /* must equal the tensor's element count     */
} psv_weight;

/* One scheduled task, for introspection (psv_wave_plan). */
typedef struct psv_task {
  int32_t stream;      /* stream id                                          */
  int32_t chunk;       /* chunk index c within the stream                    */
  int32_t step;        /* denoising step s                                   */
  int32_t slot;        /* KV ring slot the task writes: c mod (W+1)          */
  int32_t kv_len;      /* keys the task attends to: (min(c, W) + 1) * T      */
  int32_t row_off;     /* first row of the task in the wave's batch          */
  int32_t state_slot;  /* latent state slot holding x of this chunk          */
  int32_t cond_table;  /* adaLN tables the task reads: its stream id, or
                          max_streams + state_slot for a chunk submitted with
                          its own conditioning (psv_submit_chunk_cond)       */
} psv_task;

/* Per-kernel timing, filled when profiling is on (psv_set_profiling). */
typedef struct psv_kernel_time {
  char    name[32];
  int64_t launches;
  double  total_ms;
  double  flops;       /* algorithmic FLOPs of all launches              */
  double  bytes;       /* algorithmic HBM bytes of all launches          */
} psv_kernel_time;

typedef struct psv_ctx psv_ctx;

/* Device bytes psv_create needs for this description (weights, KV rings
 * for max_streams, activations for the largest wave, latent state, tables):
 * the memory footprint a stream placement checks against (AREX article,
 * section 三层设计, third layer: a stream is admitted only if it fits). */
int psv_arena_bytes(const psv_model_desc* desc, size_t* bytes);

/* Create a context: one served model on one GPU, whose device memory holds
 * the model's weights, every stream's noisy-KV rings and the activations of
 * the largest wave (AREX article, section 三层设计, second layer: one GPU
 * time-shares the stages of many (block, step) pairs and keeps their state).
 * dev_arena/arena_bytes: caller-owned device memory of at
 * least psv_arena_bytes() bytes, 1024-byte aligned, used until psv_destroy;
 * cuda_stream: caller-owned cudaStream_t all device work is issued on
 * (NULL = legacy default stream).  With PSV_FLAG_PLAN_ONLY the arena and
 * stream are ignored (may be NULL) and no CUDA call is made.
 * Errors: PSV_EINVAL (bad shape), PSV_ENOMEM (arena too small), PSV_ECUDA. */
int psv_create(const psv_model_desc* desc, void* dev_arena, size_t arena_bytes,
               void* cuda_stream, psv_ctx** out);

/* Copy n tensors into the arena (see the weight table above).  The model is
 * served as loaded: unpruned, uncompressed, unquantised weights (AREX article,
 * section 实测数字), here bf16 matrices and f32 biases.  Synchronous
 * with respect to the host buffers.  Errors: PSV_EINVAL (unknown id, wrong
 * numel or dtype), PSV_ECUDA. */
int psv_load_weights(psv_ctx* ctx, const psv_weight* w, int n);

/* Open a stream: one agent's sequence of chunks, generated autoregressively
 * and conditioned on that agent (AREX article, section 难题: an
 * action-conditioned world model generates the next frames from the current
 * observation and action; section 三层设计, third layer: each stream is
 * scheduled as a unit).  cond: the stream's conditioning vector (host, f32
 * [d]).  Builds the
 * stream's adaLN tables on the device: for every step s,
 * e_s = T2 SiLU(T1 emb(t_s) + b1) + b2 + cond, mod[s][b] = MOD_W,b SiLU(e_s)
 * + MOD_B,b, fmod[s] = FMOD_W SiLU(e_s) + FMOD_B.  Stream ids are assigned
 * lowest-free-first.  Errors: PSV_EAGAIN (max_streams open), PSV_EINVAL. */
int psv_open_stream(psv_ctx* ctx, const float* cond, int* stream_id);

/* Submit the next chunk of a stream: noise (host, f32 [T, C], the chunk's
 * x_0).  Every chunk starts from pure noise and is denoised over S steps;
 * it may start before its predecessor has finished, reading at each step the
 * predecessor's still-noisy KV of that step (BAAI announcement, section
 * 新一代物理 AI 的基础设施, Fig. 1 right).  Chunks are numbered 0, 1, ... in
 * submission order.  Errors:
 * PSV_EAGAIN (max_inflight chunks alive: poll first), PSV_EINVAL. */
int psv_submit_chunk(psv_ctx* ctx, int stream_id, const float* noise);

/* Submit the next chunk with its own conditioning vector cond (host, f32
 * [d]): an action / observation embedding for this chunk only.  Every step
 * of the chunk uses e_s = temb(t_s) + cond in place of the stream's vector
 * (the pages' action-conditioned world models condition each generated
 * chunk on the agent's action: AREX article, section 难题; BAAI
 * announcement, section 新一代物理 AI 的基础设施).  The chunk's adaLN tables are
 * built on the device before this call returns (asynchronously on the
 * context stream, ahead of any later wave).  Needs a context created with
 * PSV_FLAG_CHUNK_COND.  Errors: PSV_EINVAL (flag missing, null argument),
 * PSV_EAGAIN (max_inflight chunks alive), PSV_ECUDA. */
int psv_submit_chunk_cond(psv_ctx* ctx, int stream_id, const float* noise, const float* cond);

/* Run one wave: every task whose dependencies are met, all streams batched
 * block by block.  The tasks that sit on the same transformer block, from
 * different chunks, denoising steps and streams, run as one batch, so that
 * weight loads and kernel launches are shared (AREX article, section 三层设计,
 * second layer; BAAI announcement, section PhysisServe, time-sharing and
 * Fig. 3 right, cross-stream batching on one card).  Asynchronous on the
 * context stream.  *n_tasks = tasks run (0 = nothing ready; no device work
 * issued). */
int psv_run_wave(psv_ctx* ctx, int* n_tasks);

/* Return the oldest finished, not yet returned chunk of a stream, in chunk
 * order: the stream's output, one chunk per steady interval (BAAI
 * announcement, Fig. 1 right and Fig. 2: once the pipeline is full a new
 * chunk comes out every interval; AREX article, section 实测数字: the output
 * latency is that interval).  Copies
 * its final latent x_S (f32 [T, C]) to host `out` and its index to
 * *chunk_idx.  Non-blocking: PSV_EAGAIN if that chunk's wave has not
 * finished on the device (or no chunk of the stream has been run to its
 * last step).  Checks the device error word: PSV_EDEVICE if set. */
int psv_poll_chunk(psv_ctx* ctx, int stream_id, float* out, int64_t* chunk_idx);

/* Wait (host-side polling, no device spin) until all issued work is done:
 * the end of the time slices issued so far on the one time-shared GPU
 * (AREX article, section 三层设计, second layer).
 * timeout_ms < 0 waits without deadline.  PSV_ETIMEDOUT on deadline. */
int psv_sync(psv_ctx* ctx, int timeout_ms);

/* The task list the next psv_run_wave would run (no state change): the
 * ready (stream, chunk, step) tasks of the dependency DAG of the pages
 * (BAAI announcement, Fig. 2, upper part: one row per stage, one column per
 * chunk).
 * Writes min(n, cap) entries; *n = number of ready tasks. */
int psv_wave_plan(psv_ctx* ctx, psv_task* buf, int cap, int* n);

/* Close a stream; its id and rings become free for a later stream (AREX
 * article, section 三层设计, third layer: streams arrive and leave while
 * others keep running).  Queued work is not
 * cancelled: call after its chunks were polled. */
int psv_close_stream(psv_ctx* ctx, int stream_id);

/* ---- admission control (one GPU) -----------------------------------------
 * The pages admit a new stream only when the whole stream fits and its
 * service objective (SLO) can be met, never migrate running streams, and so
 * keep the service of the streams already admitted stable (AREX article,
 * section 三层设计, third layer; BAAI announcement, section PhysisServe,
 * multi-stream scheduling).  On one GPU: a stream's state is its KV rings
 * (one of the max_streams ring sets reserved at create), and in steady state
 * every open stream gets one chunk per wave, so every stream's ms per chunk
 * is the shared wave time, which a new stream lengthens for all of them.
 *
 * Predicted steady wave time with n open streams (n*S tasks, full windows).
 * The library times every wave on the device and keeps the mean of the
 * full-window waves per task count; a count measured before is predicted by
 * its mean, another one from the nearest measured count in proportion to
 * the algorithmic FLOPs, and with no measurement at all from the
 * algorithmic FLOPs at 1 PFLOP/s.  Errors: PSV_EINVAL (n < 1 or >
 * max_streams). */
int psv_predict_wave_ms(psv_ctx* ctx, int n_streams, double* ms);

/* Open a stream (as psv_open_stream) only if a ring set is free and the
 * predicted wave time with it meets slo_ms (ms per chunk, <= 0: none) and the
 * SLO every open stream was admitted with.  *predicted_ms (may be NULL) gets
 * the prediction.  Errors: PSV_EAGAIN (rejected: no ring set free, or an SLO
 * would be missed; the reason is in psv_last_error), PSV_EINVAL, PSV_ECUDA. */
int psv_admit_stream(psv_ctx* ctx, const float* cond, double slo_ms, int* stream_id,
                     double* predicted_ms);

/* Destroy the context (synchronises the stream first); the arena returns to
 * the caller.  NULL is a no-op.  (Housekeeping: the pages have no
 * counterpart.) */
void psv_destroy(psv_ctx* ctx);

/* Last error message of this context ("" if none); NULL ctx gives the
 * message of the last failed psv_create.  (Housekeeping: the pages have no
 * counterpart.) */
const char* psv_last_error(const psv_ctx* ctx);

/* ---- executor controls and introspection -------------------------------- */

/* Replay each wave shape (task count) as a CUDA graph (default on). */
int psv_set_graphs(psv_ctx* ctx, int enabled);

/* Record CUDA events around every kernel launch (forces eager launches
 * while on).  psv_kernel_times returns per-kernel totals since enabling;
 * it synchronises the stream.  Writes min(cap, kinds) entries, *n = kinds. */
int psv_set_profiling(psv_ctx* ctx, int enabled);
int psv_kernel_times(psv_ctx* ctx, psv_kernel_time* out, int cap, int* n);

/* Debug tap for parity tests: during the next psv_run_wave (run eagerly),
 * copy the residual stream h (f32 [n_tasks*T, d], rows in task order) into
 * the caller's device buffers h_in (before block `block`) and h_out (after
 * it).  Cleared after that wave. */
int psv_debug_tap(psv_ctx* ctx, int block, float* h_in, float* h_out);

/* Debug read of one KV ring (stream, block, step) into host f32 buffers:
 * k [(W+1)*T, d] and v [(W+1)*T, d], rows = slot*T + token.  Synchronous. */
int psv_debug_read_kv(psv_ctx* ctx, int stream_id, int block, int step,
                      float* k, float* v);

/* Debug: byte offset, from the start of the arena given to psv_create, of
 * the int error word that a kernel sets when a device-side wait times out or
 * a bounds check fails (psv_poll_chunk and psv_sync then return the sticky
 * PSV_EDEVICE).  Lets a test raise the word from the host, without any
 * kernel fault, to check that path.  Errors: PSV_EINVAL (plan-only
 * context). */
int psv_debug_error_word(psv_ctx* ctx, size_t* arena_offset);

/* ---- kernel-level window attention ---------------------------------------
 * The attention step of the wave (AREX article "vLLM 与 Physis-AI 联合介绍
 * PhysisServe 推理系统", §难题: a chunk's queries attend to its own keys and
 * the still-noisy keys the preceding chunks left) as a standalone call on
 * caller buffers: n independent query blocks; the T queries of block i
 * attend to the L keys of block i with softmax scale 1/sqrt(dh), no mask.
 *   q   bf16 [n*T][H*dh]            row-major; head h = columns [h*dh, (h+1)*dh)
 *   k   bf16 [n][k_rows][H*dh]      keys of block i at rows [0, L)
 *   vt  bf16 [n][H][dh][vt_cols]    values transposed per head, keys at cols [0, L)
 *   o   bf16 [n*T][H*dh]            output (written)
 * Requirements: dh in {32, 64, 128}; H*dh % 8 == 0; 1 <= L <= k_rows;
 * L <= vt_cols, vt_cols % 8 == 0; all pointers 16-byte aligned device memory.
 * scratch: caller-owned device memory of at least psv_attention_scratch_bytes
 * bytes (task table, the work queue of the persistent CTA pairs and the
 * split-key arrival counters, split-key partials), 256-byte aligned;
 * it is overwritten and must not be shared by calls that may overlap on the
 * GPU.  Asynchronous on cuda_stream; the int at the start of scratch is set
 * nonzero if a device-side pipeline wait timed out.  Errors: PSV_EINVAL. */
typedef struct psv_attn_problem {
  int32_t n, T, H, dh, L, k_rows, vt_cols;
} psv_attn_problem;

int psv_attention_scratch_bytes(const psv_attn_problem* p, size_t* bytes);
int psv_attention(const psv_attn_problem* p, const void* q, const void* k, const void* vt,
                  void* o, void* scratch, size_t scratch_bytes, void* cuda_stream);

/* Allocation-free psv_attention (the pages have no counterpart: this is a
 * deployment convenience).  For callers that cannot allocate device memory
 * at call time, e.g. a real-time control loop that must not enter the CUDA
 * allocator after start-up, or a host framework that owns all device memory
 * and provides no scratch.  Same arguments and results as psv_attention,
 * without scratch: the library uses a fixed array of
 * PSV_ATTN_NOALLOC_SCRATCH_BYTES bytes inside its CUDA module, which every
 * device that loads the module holds until the process exits.  Problems
 * whose scratch (psv_attention_scratch_bytes) exceeds that size are rejected
 * with PSV_ENOMEM; bad shapes or pointers with PSV_EINVAL.
 * Set-up: the first call on a device, with that device current, looks up
 * the array's device address.  Under CUDA's default lazy module loading that
 * is also when the module is loaded on the device and the array reserved, so
 * the first call may fail with PSV_ECUDA if the device is out of memory; make
 * it at start-up, and before any stream capture.  Later calls allocate
 * nothing, on the host or on the device.  Every call shares the one array
 * (each call clears the parts that must start at zero), and the array keeps
 * the last call's contents; calls whose work may overlap on the GPU race on
 * it and must be ordered by the caller (e.g. issued on one stream). */
#define PSV_ATTN_NOALLOC_SCRATCH_BYTES (16u << 20)
int psv_attention_noalloc(const psv_attn_problem* p, const void* q, const void* k,
                          const void* vt, void* o, void* cuda_stream);

/* Status of the last psv_attention_noalloc call on the current device:
 * waits for cuda_stream, then *status = the error word of the shared array
 * (0, or nonzero if a device-side pipeline wait of that call timed out and
 * its output is not valid).  Allocates nothing.  Errors: PSV_EINVAL,
 * PSV_ECUDA. */
int psv_attention_noalloc_status(int* status, void* cuda_stream);

/* ---- kernel-level operators of a rolling key/value cache ------------------
 *
 * The pages keep the keys and values of the preceding chunks in a rolling
 * window (AREX article, §难题) and say nothing about positions in space,
 * masks or what leaves the window.  These calls give a program that drives
 * its own cache the operators around psv_attention: rotary positions with
 * several axes, attention over a cache with masks, a score cap and a distance
 * bias, the attention weight every key received, and the eviction of the keys
 * that received least.
 *
 * Conventions of these calls
 *   - strides are counted in elements; the innermost index (a head's dh
 *     values) is contiguous; offsets are 64-bit;
 *   - every pointer is device memory of the current device unless its line
 *     says host; work goes to cuda_stream and is asynchronous; nothing is
 *     allocated and no host memory is read after the call returns, so a call
 *     can be captured into a CUDA graph;
 *   - lengths, positions, documents and prefixes are read on the device when
 *     the kernels run (a captured call sees their values at replay); their
 *     pointers, as every pointer, are aligned to their type;
 *   - errors: PSV_EINVAL (shapes, strides, alignment, null pointers; host
 *     memory, or another device's, as the first input or the first output),
 *     PSV_ECUDA; psv_cache_last_error() names the reason.  What other pointers
 *     point to is not looked at;
 *   - outputs that meet an input or one another (as each call says) are refused
 *     (PSV_EINVAL).  Tensors packed into one buffer, row by row or block by
 *     block, pass where their strides agree; where they do not, the stretches
 *     from a tensor's first to its last byte have to be apart. */

#define PSV_DTYPE_F16 2 /* besides PSV_DTYPE_F32 and PSV_DTYPE_BF16 */

/* Reason of this thread's last failed call of this section ("" if none). */
const char* psv_cache_last_error(void);

/* Rotary positions with several axes.  x [B][L][H][dh]; the first
 * R = axis_dims[0] + .. + axis_dims[n_axes-1] values of a head are rotated,
 * the others copied.  Rotated pair p (0 <= p < R/2) belongs to axis a, whose
 * pairs are numbered consecutively (axis 0 first), and turns by
 *   angle = pos[b][l][a] * f_p,  f_p = theta^(-2 j / axis_dims[a])
 * with j the pair's number within its axis; freqs, where given, holds f_p
 * itself (any schedule).  (u, w) -> (u cos - w sin, u sin + w cos); inverse
 * turns by -angle (un-rotates cached keys; also the gradient of the forward
 * call).  Layout PAIRS: pair p is (2p, 2p+1), as on the wave path; HALVES:
 * (p, p + R/2).  Angles are reduced in 64-bit fixed point, so positions up to
 * 2^31 keep f32 accuracy; the rotation is done in f32 and rounded once.
 * In place (out == x with equal strides) is allowed; an out that meets x
 * otherwise, or pos, is refused.
 * Rows l >= lens[b] of out are left as they were.
 * Requirements: dtype F32, BF16 or F16; 1 <= n_axes <= 4; axis_dims even and
 * positive; R <= dh <= 256; dh even; 1 <= B <= 65535; L, H >= 1 and L x H
 * below 2^24; strides in [0, 2^40], out's rows distinct.  Bases and strides that are multiples of 16 bytes use 16-byte accesses. */
#define PSV_ROPE_PAIRS  0
#define PSV_ROPE_HALVES 1
typedef struct psv_rope_problem {
  int32_t dtype, B, L, H, dh;
  int32_t n_axes, axis_dims[4];
  int32_t layout, inverse;
  double theta;
  const double* freqs;     /* host [R/2], radians per position; NULL: from theta */
  int64_t x_stride[3];     /* batch, row, head */
  int64_t out_stride[3];
  int64_t pos_stride[2];   /* batch (0: shared), row; axes are contiguous */
  const int32_t* lens;     /* [B] rows in use; NULL: L */
} psv_rope_problem;

/* pos int32 [B][L][n_axes]. */
int psv_rope(const psv_rope_problem* p, const void* x, const int32_t* pos, void* out,
             void* cuda_stream);

/* Attention over a cache.  q, o [B][Lq][Hq][dh]; k, v [B][Lk][Hkv][dh] (values
 * as written, not transposed); query head h reads key head h / (Hq / Hkv).
 *   s = scale * q.k;  softcap > 0: s = softcap * tanh(s / softcap);
 *   slopes: s -= slopes[h] * |q_pos - k_pos|
 * A row sees key j if j < k_lens[b], q_doc == k_doc (where documents are
 * given) and, with causal set, k_pos <= q_pos or k_pos < prefix[b].
 *   o = softmax(s) v over the visible keys;  lse = log sum exp s  [B][Hq][Lq]
 * A row that sees nothing gets o = 0 and lse = -infinity; a row that sees a NaN
 * score gets NaN in o and lse.  Rows i >= q_lens[b] of o and lse are left as they
 * were.  Lengths are clamped to [0, Lq] and [0, Lk].  o may be q itself (equal
 * strides); otherwise o and lse meet neither q, k, v nor one another.  Default
 * positions: k_pos = j, q_pos = k_len - q_len + i (the rows are the last ones of
 * the sequence).  Positions lie within +-2^30.
 * Keys and values behind k_lens[b] may hold anything (NaN too); keys that are
 * only masked may hold anything finite, their scores are not used.
 * Products take bf16/f16 operands and accumulate in f32; scores, maxima, sums
 * and lse are f32 (the cap's tanh is good to 2^-21 of the capped score, with a
 * cap of up to 128 to 2^-21 of the cap); the weights are rounded to the operand
 * type for their product with v, the output once.  Results do not depend on other sequences
 * of the batch, and repeat bit for bit.
 * Requirements: dtype BF16 or F16; B, Hkv >= 1; Hq a multiple of Hkv; B x Hq
 * <= 2^24; 0 <= Lq <= 2^24, 0 <= Lk <= 2^28; 1 <= dh <= 256; strides in [0,
 * 2^40], o's rows distinct; scale >= 0 and softcap >= 0 finite; k_doc and
 * q_doc both or neither; prefix needs causal.
 * The tensor-core paths (one for up to 16 rows a kv head, Lq x Hq / Hkv, as in
 * single-token calls, one for more) take dh <= 128, dh % 8 == 0, Hq / Hkv <=
 * 128, bases and strides in multiples of 16 bytes (positive where the extent
 * is over 1); every other problem runs on a slower general kernel. */
typedef struct psv_cache_problem {
  int32_t dtype, B, Hq, Hkv, dh, Lq, Lk;
  int32_t causal;
  float scale;              /* 0: 1 / sqrt(dh) */
  float softcap;            /* 0: none */
  int64_t q_stride[3];      /* batch, row, head */
  int64_t k_stride[3], v_stride[3], o_stride[3];
  const int32_t* q_lens;    /* [B]; NULL: Lq */
  const int32_t* k_lens;    /* [B]; NULL: Lk */
  const int32_t* q_pos;     /* [B][Lq]; NULL: see above */
  const int32_t* q_doc;     /* [B][Lq]; NULL: one document */
  int64_t q_meta_stride;    /* batch stride of q_pos and q_doc */
  const int32_t* k_pos;     /* [B][Hkv][Lk]; NULL: j */
  const int32_t* k_doc;     /* [B][Hkv][Lk] */
  int64_t k_meta_stride[2]; /* batch and kv-head strides of k_pos and k_doc (0: shared) */
  const int32_t* prefix;    /* [B]; NULL: 0 */
  const float* slopes;      /* [Hq], at most 1e30 in size; NULL: no distance bias */
} psv_cache_problem;

/* Workspace of psv_cache_attention and psv_cache_mass for this problem (its
 * size depends on the shapes, on softcap, on which of the pointers are given and
 * on whether k_meta_stride[1] is 0, as the kv heads' notes are then one; a larger
 * one serves as well):
 * 256-byte aligned device memory whose first PSV_CACHE_SCRATCH_HEAD bytes the
 * caller zeroes once, before its first use.  It may serve any number of calls
 * (captured ones too) that do not overlap on the GPU.  The int at its start
 * becomes nonzero, and stays so, if a device-side wait of a call timed out (2 s
 * without progress); that call's output is not valid, and the workspace is
 * zeroed before reuse.  The calls return before the GPU has done its work, so
 * they cannot say so: psv_cache_status does. */
#define PSV_CACHE_SCRATCH_HEAD 256
int psv_cache_scratch_bytes(const psv_cache_problem* p, size_t* bytes);

/* Whether a call on this workspace timed out: waits for cuda_stream, then
 * *status = the workspace's first int.  Not while the stream is captured.
 * Errors: PSV_EINVAL, PSV_ECUDA. */
int psv_cache_status(const void* scratch, int* status /* host */, void* cuda_stream);

int psv_cache_attention(const psv_cache_problem* p, const void* q, const void* k, const void* v,
                        void* o, float* lse /* may be NULL */, void* scratch, size_t scratch_bytes,
                        void* cuda_stream);

/* Attention weight that each cached key received, from the rows' lse of
 * psv_cache_attention on the same problem (v and o are not used):
 *   mass_out[b][g][j] = mass_in[b][g][j]
 *                     + sum over rows i < q_lens[b] and heads h of group g of exp(s_ij - lse)
 * over visible pairs (a row whose lse is NaN gives NaN to the keys it sees, and
 * may give it to others of its sequence and kv head); mass f32 [B][Hkv][Lk];
 * mass_in may be NULL (zeros) or mass_out (accumulate in place); mass_out meets
 * neither q, k nor lse.  Entries j >= k_lens[b] are left as they were.  Sums are
 * f32 in a fixed order (repeats are equal bit for bit).
 * Requirements as above. */
int psv_cache_mass(const psv_cache_problem* p, const void* q, const void* k, const float* lse,
                   const float* mass_in, float* mass_out, void* scratch, size_t scratch_bytes,
                   void* cuda_stream);

/* Eviction by accumulated weight.  Of the n = k_lens[b] keys of each (sequence,
 * kv head), min(n, budget) are kept: the first `sinks` slots, the last
 * `recent` ones, and of the others those with the greatest mass, the lower
 * slot among equals (NaN counts as the greatest).  Kept keys, values and mass
 * are written in slot order to other buffers (k_out, v_out [B][budget][Hkv][dh];
 * mass_out, idx_out, pos_out, doc_out [B][Hkv][budget]); idx_out holds the
 * slots they came from, lens_out[b] = min(n, budget).  Rows behind lens_out
 * are left as they were.  pos_out without k_pos receives the slots.  Out
 * buffers that meet an input or one another are refused (k_out and v_out may be
 * packed into one buffer).
 * Requirements: dtype F32, BF16 or F16; B, Hkv, budget >= 1; 1 <= L <= 2^30;
 * budget <= L; 1 <= dh; sinks, recent >= 0, sinks + recent <= budget; B <= 65535 and budget
 * x Hkv x dh below 2^32; strides in [0, 2^40], rows of k_out and v_out
 * distinct; doc_out needs k_doc. */
typedef struct psv_evict_problem {
  int32_t dtype, B, Hkv, dh, L, budget, sinks, recent;
  int64_t k_stride[3], v_stride[3];         /* batch, row, head */
  int64_t k_out_stride[3], v_out_stride[3];
  const int32_t* k_lens;    /* [B]; NULL: L */
  const int32_t* k_pos;     /* [B][Hkv][L] or NULL */
  const int32_t* k_doc;     /* [B][Hkv][L] or NULL */
  int64_t k_meta_stride[2]; /* batch and kv-head strides of k_pos and k_doc (0: shared) */
  int32_t* pos_out;         /* or NULL */
  int32_t* doc_out;         /* or NULL */
  int32_t* lens_out;        /* [B] or NULL; not k_lens */
} psv_evict_problem;

int psv_cache_evict(const psv_evict_problem* p, const void* k, const void* v, const float* mass,
                    void* k_out, void* v_out, float* mass_out, int32_t* idx_out, void* cuda_stream);

/* ---- kernel-level operators of a paged key/value cache ---------------------
 *
 * The pages keep the keys and values of the preceding chunks (AREX article,
 * §难题) and say nothing about how a server of many streams holds them.  These
 * calls keep the caches of all streams in one pool of pages, in 16 bits or in
 * 8 with a scale for each token and head: rows are written (and quantised) into
 * pages, read back as plain tensors, which psv_cache_attention takes for a
 * chunk's many rows, and looked at by a new token, or a few, in place.
 *
 * The conventions of the rolling cache's calls hold, psv_cache_last_error()
 * among them.  Tables, starts and lengths are read on the device when the kernels
 * run.  What rows of a call read or see of the pages is psv_page_write's, or equal to
 * what it would write. */

#define PSV_PAGE_BF16 1 /* values as they are (rounded, from F32 rows)                */
#define PSV_PAGE_F16  2
#define PSV_PAGE_E4M3 3 /* 8-bit floats, scale = (largest size of the row) / 448      */
#define PSV_PAGE_I8   4 /* 8-bit integers of -127 to 127, scale = (largest size) / 127 */

/* The cache.  Position j of sequence b lies in row j mod page_size of page
 * table[b][j / page_size].  An entry outside [0, n_pages) names no page, and
 * positions behind max_pages x page_size have none: rows written there are
 * dropped, they read back as zeros, and attention does not see them.  Sequences
 * may share pages.
 * A row (one head's dh values of one key or value) is kept, in 8 bits, as
 * code = nearest(x * (M / size)), ties to even, and scale = size / M, with size the
 * largest |x| of the row and M = 448 or 127, in f32 arithmetic; it stands for
 * code * scale.  A row with size below 2^-100 is kept as zeros with scale 0; one
 * that holds a NaN or an infinity has the scale NaN and reads back as NaN.
 * Requirements: 1 <= B <= 65535; n_pages, page_size, max_pages, Hkv >= 1;
 * max_pages x page_size <= 2^30; B x Hkv <= 2^24; 1 <= dh <= 256; strides in
 * [0, 2^40]. */
typedef struct psv_page_cache {
  int32_t format, B, n_pages, page_size, max_pages, Hkv, dh;
  int64_t k_stride[3], v_stride[3]; /* page, row, head, in stored values */
  int64_t scale_stride[3];          /* page, row, head, of k_scales and v_scales */
  int64_t table_stride;             /* of a sequence (0: shared) */
  const int32_t* table;             /* [B][max_pages] */
  void *k_pages, *v_pages;          /* [n_pages][page_size][Hkv][dh] in any order of the indexes */
  float *k_scales, *v_scales;       /* [n_pages][page_size][Hkv]; NULL for 16-bit pages */
} psv_page_cache;

/* Rows k, v [B][L][Hkv][dh] of a program: row i of sequence b is position
 * starts[b] + i.  dtype F32, BF16 or F16 (16-bit pages: their own type or F32);
 * L >= 0, L x Hkv <= 2^30. */
typedef struct psv_page_rows {
  int32_t dtype, L;
  int64_t k_stride[3], v_stride[3]; /* batch, row, head */
  const int32_t* starts;            /* [B]; NULL: 0 */
  const int32_t* lens;              /* [B] rows in use, clamped to [0, L]; NULL: L */
} psv_page_rows;

/* Writes the rows in use into their pages.  Of two rows that one call writes to one
 * place either's values may stay, and the other's scale.  Rows of pages must be
 * distinct; pages and scales that meet an input or one another are refused (k and
 * v may be packed into one buffer).  Multiples of 8 as dh and strides of pages,
 * and of 16 bytes as strides of k and v and as all bases, use wide accesses. */
int psv_page_write(const psv_page_cache* c, const psv_page_rows* r, const void* k, const void* v,
                   void* cuda_stream);

/* Reads positions back into k and v, rounded once; rows not in use are left as
 * they were.  k and v meet neither the cache nor one another. */
int psv_page_read(const psv_page_cache* c, const psv_page_rows* r, void* k, void* v, void* cuda_stream);

/* Attention of rows over the pages.  q, o [B][Lq][Hq][dh]; query head h reads key
 * head h / (Hq / Hkv).  With n = k_lens[b] (append: + q_lens[b], where k_lens
 * counts the keys before this call's rows), row i stands at position
 * p = n - q_lens[b] + i and sees key j < n if it has a page and
 *   causal: j <= p;     window > 0: j > p - window, or j < sinks
 *   s = scale * q.k; softcap > 0: s = softcap * tanh(s / softcap)
 *   o = softmax(s) v;  lse = log sum exp s  [B][Hq][Lq]
 * A row that sees nothing gets o = 0 and lse = -infinity; one that sees a NaN score
 * gets NaN in both.  Rows i >= q_lens[b] of o and lse are left as they were.  o may
 * be q itself (equal strides).  Keys that no row sees may hold anything, and so may
 * keys and values that are masked for some rows, as far as those rows go: codes that are
 * NaN, scales and values that are not finite reach the rows that see them only.
 * Products take f16 operands (bf16 ones for BF16 pages) and accumulate in f32: 8-bit
 * codes are exact in f16, bf16 queries get a power of two for each row first (and are
 * exact down to 2^-31 of the row's largest), a key's scale is applied to its score
 * and a value's to its weight, in f32.  Scores,
 * maxima, sums and lse are f32; the weights are rounded to the operand type for
 * their product with v, the output once.  f16 weights have fixed steps below 2^-21 of a
 * row's largest (weight times value's scale for 8-bit pages): each is off by at most
 * 2^-32 of that, n keys together by n 2^-32.  Results repeat bit for bit for the same
 * lengths; those of a sequence may differ in their roundings where the lengths
 * of others change, as the work is shared out among the SMs by all of them.
 * Requirements: dtype BF16 or F16 (16-bit pages: their own); Hq a multiple of Hkv;
 * B x Hq <= 2^24; 0 <= Lq <= 2^20, B x Lq x Hq <= 2^30; window, sinks >= 0, sinks
 * need a window; scale, softcap >= 0 finite; o's rows distinct.
 * The tensor-core kernel takes dh % 8 == 0, bases and strides of q and o in
 * multiples of 16 bytes, of pages in multiples of eight values, strides of pages, rows
 * and scales below 4 GB; every other problem runs on a general kernel, tens to
 * thousands of times slower (pad the rows of other widths to a multiple of 8).  It is
 * made for few rows: it reads the pages once for every 16 rows a kv head, Lq x Hq / Hkv (8, where dh > 128;
 * 32 of long caches in 16 bits, heads of 72 to 128).
 * (A chunk's many rows: psv_page_read, then psv_cache_attention.)  Pages of a multiple
 * of eight rows are read fastest.  max_pages is what the host knows of the lengths:
 * where it is small, calls need no second kernel. */
typedef struct psv_page_query {
  int32_t dtype, Lq, Hq, causal, window, sinks, append;
  float scale;                      /* 0: 1 / sqrt(dh) */
  float softcap;                    /* 0: none */
  int64_t q_stride[3], o_stride[3]; /* batch, row, head */
  const int32_t* q_lens;            /* [B], clamped to [0, Lq]; NULL: Lq */
  const int32_t* k_lens;            /* [B], clamped to [0, max_pages x page_size]; NULL: that (append: 0) */
} psv_page_query;

/* Workspace of psv_page_attention: 256-byte aligned device memory of any content.  It
 * may serve any number of calls (captured ones too, of any problem that it is large
 * enough for) that do not overlap on the GPU.  5.2 MB (10^6 bytes) at most. */
int psv_page_scratch_bytes(const psv_page_cache* c, const psv_page_query* q, size_t* bytes);

int psv_page_attention(const psv_page_cache* c, const psv_page_query* q, const void* x /* q */, void* o,
                       float* lse /* may be NULL */, void* scratch, size_t scratch_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* PSV_H */
