/*
 * statekv.h -- C ABI of libstatekv, the GB300 (sm_103a) implementation of
 * StateKV streaming video prefill.
 *
 * Method: "Linear Scaling Video VLMs for Long Video Understanding" (StateKV,
 * ECCV 2026), papernotes.org summary, section 方法详解:
 *   整体框架 (overall framework) -- frames arrive one at a time, T visual tokens
 *     each; in every layer the frame attends only to a fixed-capacity
 *     compressed state C_{n-1} and to itself, so the per-frame cost is
 *     O(T^2 + BT) and the prefill is linear in the number of frames N;
 *   关键设计 1 (dual state) -- per layer a detailed state D_n holding every
 *     frame's K/V (kept for text decoding) and a compressed state C_n with
 *     |K̄_n| = B; Q_n attends over [K̄_{n-1}; K_n];
 *   关键设计 2 (temporal-sink update) -- candidate pool U_n = S̄_{n-1} ∪ {1..T},
 *     score s_j = mean attention the frame's queries pay to key j,
 *     S̄_n = TopK({s_j}, B) rebuilds C_n;
 *   关键设计 3 (virtual length, static RoPE scale) -- RoPE angles use the
 *     logical stream position L_n = nT (+ i); one global scale alpha is fixed
 *     before prefill and never changes.
 *
 * Readings of points the page leaves open (fixed here, per KV head):
 *   - mask: compressed keys fully visible; frame key i' visible to query i iff
 *     i' <= i;
 *   - s_j averages P over all G*T query rows of the G query heads that share
 *     the KV head (a query that cannot see j contributes 0);
 *   - Top-B ties go to the lower virtual position;
 *   - positions p = position_offset + n*T + i, n 0-based;
 *   - alpha != 1 is YaRN NTK-by-parts (beta_fast 32, beta_slow 1) with logit
 *     factor mscale^2, mscale = 0.1 ln(alpha) + 1;
 *   - C and D hold post-RoPE keys in the storage dtype.
 *
 * Threading and streams: a handle is not thread-safe; calls on one handle
 * must be serialised by the caller.  All device work of a call is enqueued
 * asynchronously on the caller's CUDA stream (cudaStream_t passed as void*,
 * NULL = the legacy default stream); results are valid once that stream has
 * reached the point after the call.
 *
 * Errors: every entry point returns an int status (STATEKV_OK or a negative
 * STATEKV_E_*).  Nothing aborts and no C++ exception crosses the ABI.  Host
 * argument checks happen before any device work, so a call rejected with
 * E_INVALID_ARG / E_UNSUPPORTED / E_CAPACITY leaves the handle unchanged.
 * E_CUDA means a CUDA call failed (the handle's device state is then
 * unspecified; destroy it); the call clears the CUDA runtime's last-error
 * state before returning, so a refused launch does not resurface in later
 * calls.  Device-side bounded waits that give up record a
 * status that statekv_check_device_status() reports as E_TIMEOUT.
 */
#ifndef STATEKV_H_
#define STATEKV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------ selection policy */
#define STATEKV_SELECT_TOPB    0    /* Top-B by attention score (StateKV)    */
#define STATEKV_SELECT_WINDOW  1    /* the B most recent tokens (ReKV-style)  */

/* ---------------------------------------------------------------- status */
#define STATEKV_OK              0
#define STATEKV_E_INVALID_ARG  -1   /* null pointer, bad size, bad index      */
#define STATEKV_E_UNSUPPORTED  -2   /* valid but not implemented (e.g. d=96)  */
#define STATEKV_E_CAPACITY     -3   /* detailed state full (n == max_frames)  */
#define STATEKV_E_OOM          -4   /* device allocation failed at create     */
#define STATEKV_E_CUDA         -5   /* a CUDA runtime/driver call failed      */
#define STATEKV_E_TIMEOUT      -6   /* a device-side bounded wait gave up     */
#define STATEKV_E_DEVICE       -7   /* a device-side consistency check failed */

/* storage dtypes */
#define STATEKV_BF16 0              /* bf16 storage, fp32 accumulation        */
#define STATEKV_F32  1              /* fp32 storage and arithmetic            */

/* kernels, for statekv_profile_read() */
#define STATEKV_KERNEL_ROPE_TABLE 0 /* cos/sin table (computed once, at create: */
                                    /* no launches inside a prefill)            */
#define STATEKV_KERNEL_ROPE       1 /* RoPE at virtual positions + appends    */
#define STATEKV_KERNEL_ATTENTION  2 /* two-sweep attention + key column sums  */
#define STATEKV_KERNEL_SELECT     3 /* score finish, Top-B, slot-reuse gather */
#define STATEKV_NUM_KERNELS       4

typedef struct statekv_handle statekv_handle;   /* opaque */

/*
 * Configuration of one handle.  Every (stream, layer, KV head) is an
 * independent unit with its own C and D; all units advance together, one
 * frame per statekv_prefill_frame call.
 *   num_streams   S >= 1   independent videos stepped together
 *   num_layers    L >= 1   transformer layers (inputs per layer are given)
 *   num_q_heads   Hq       query heads; Hq % Hkv == 0, G = Hq / Hkv
 *   num_kv_heads  Hkv >= 1 KV heads (query head j uses KV head j / G)
 *   head_dim      d        64 or 128
 *   frame_tokens  T >= 1   visual tokens per frame
 *   budget        B >= 0   compressed-state capacity (关键设计 1, |K̄| = B)
 *   max_frames    N_max    capacity of the detailed state D, in frames
 *   dtype         STATEKV_BF16 or STATEKV_F32
 *   device        CUDA device ordinal the handle lives on
 *   rope_theta    RoPE base theta (> 1)
 *   rope_alpha    static global RoPE scale alpha >= 1, fixed for the
 *                 handle's lifetime (关键设计 3)
 *   rope_orig_ctx YaRN original context L_orig (> 0 when alpha != 1)
 *   position_offset virtual position of the first video token (>= 0)
 *   select_policy STATEKV_SELECT_TOPB (the method, 关键设计 2) or
 *                 STATEKV_SELECT_WINDOW: keep the B most recent tokens
 *                 instead, the sliding-window baseline the page compares
 *                 against (ReKV, R frames = B/T).  Full self-attention is
 *                 budget >= max_frames*T with either policy (nothing is ever
 *                 evicted).
 * Limits: G*T <= 65536 query rows per unit; B + T <= 24576 unless
 * B >= max_frames*T (no eviction: then only memory bounds the pool);
 * positions must fit in int32.
 * The bf16 attention runs one CTA per 128-row query tile.  Some tiles are
 * split over their keys among the CTAs of a thread-block cluster, which
 * exchange their row log-sum-exps and partial outputs through distributed
 * shared memory (results agree with whole tiles up to rounding, and are
 * deterministic): with at least one full wave of tiles (one per SM), the
 * tiles of the last, partial wave when it fills at most half the SMs, as
 * pairs; with fewer tiles than SMs (for example one layer per call), every
 * tile, over 2..8 CTAs chosen from how many such clusters the device holds
 * at once.  The selection likewise spreads each unit over a cluster of up to
 * 8 CTAs when the units are few.  Test overrides, read at every prefill
 * launch: STATEKV_ATTN_SPLIT (0 = no split, all = every tile, n = the last n
 * tiles) with STATEKV_ATTN_SPLIT_WAYS (2..8, default 2), and
 * STATEKV_SELECT_CLUSTER (1, 2, 4 or 8 CTAs per unit).
 */
typedef struct statekv_config {
    int32_t num_streams;
    int32_t num_layers;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t frame_tokens;
    int32_t budget;
    int32_t max_frames;
    int32_t dtype;
    int32_t device;
    double  rope_theta;
    double  rope_alpha;
    int64_t rope_orig_ctx;
    int64_t position_offset;
    int32_t select_policy;
} statekv_config;

/* Human-readable name of a status code (static storage, never NULL). */
const char* statekv_status_string(int status);

/*
 * Create a handle: validates cfg, allocates on cfg->device (current device is
 * restored on return) the compressed pool [S][L][Hkv][B+T][d] for K and V,
 * its positions [S][L][Hkv][B+T] int32, the detailed state
 * [S][L][Hkv][N_max*T][d] for K and V, scratch (rotated queries, per-tile key
 * column sums, scores) and one frame of staging for the host-buffer entry
 * point.  This memory is zero-filled (buffers that later calls allocate on
 * first use are not).  The handle owns it all.
 * On failure *out is set to NULL and nothing is leaked.
 */
int statekv_create(const statekv_config* cfg, statekv_handle** out);

/* Free everything the handle owns (synchronises the device first). NULL ok. */
int statekv_destroy(statekv_handle* h);

/*
 * One frame step n (= statekv_frame_index(h)) for every unit (整体框架,
 * 关键设计 1-3):
 *   1. rotate Q and K at p = position_offset + n*T + i with the static
 *      frequencies, store K' and V into D rows [n*T, n*T+T) and into the
 *      compressed pool after the c = min(B, n*T) live slots;
 *   2. O = softmax(Q' [K̄_{n-1}; K'_n]^T * mscale^2/sqrt(d), masked) [V̄; V];
 *   3. s_j for every pool slot, Top-B with ties to the lower position;
 *   4. C_n keeps the B winners: evicted slots are refilled in place by the
 *      surviving frame rows (slot order is not position order).
 * Pointers are DEVICE pointers on the handle's device, caller-owned,
 * contiguous, in the storage dtype:
 *   q, o : [S][L][Hq][T][d]      (o is written, never read)
 *   k, v : [S][L][Hkv][T][d]     (pre-RoPE keys; values)
 * q/k/v must not alias o or handle memory.  Returns E_CAPACITY when
 * n == max_frames.  On success the frame index advances by one.
 * The rotation may start as soon as the kernel before it on the stream
 * releases its dependents (programmatic dependent launch).  This library's own
 * kernels do so only where that is safe; a caller's kernel that writes q, k or
 * v, or reads handle memory, has to leave it to its end (the default).
 */
int statekv_prefill_frame(statekv_handle* h, const void* q, const void* k,
                          const void* v, void* o, void* cuda_stream);

/*
 * Same step with HOST buffers (same layouts): copies q/k/v into the handle's
 * device staging, runs the step and copies o back, all enqueued on
 * cuda_stream.  Host buffers should be page-locked for the copies to be
 * asynchronous; they must stay valid and unmodified until the stream passes
 * the call.
 */
int statekv_prefill_frame_host(statekv_handle* h, const void* q_host,
                               const void* k_host, const void* v_host,
                               void* o_host, void* cuda_stream);

/*
 * `frames` consecutive steps from HOST buffers holding the frames back to
 * back (frame-major, each frame in the layouts above):
 *   q, o : [frames][S][L][Hq][T][d]      k, v : [frames][S][L][Hkv][T][d]
 * The same computation as `frames` calls of statekv_prefill_frame_host, but
 * the copies overlap the device work: the handle holds two staging slots,
 * and on side streams of its own (four per direction, each copying a quarter
 * of a frame's bytes) it copies frame i+1 in and frame i-1 out while frame i
 * runs on cuda_stream.  The whole batch is ordered on
 * cuda_stream like a single call: the side streams first wait for the work
 * already enqueued there, and cuda_stream waits for the last copy out, so
 * every o frame is valid (and q/k/v may be reused) once the stream passes
 * the call.  Host buffers should be page-locked.  Returns E_CAPACITY, with
 * nothing done, when n + frames > max_frames; frames == 0 is a no-op.  The
 * side streams and events are created on the first call (E_CUDA if that
 * fails); a handle's calls must not overlap with each other.
 * This entry point has no counterpart in the page; it streams a video from
 * host memory at device speed.
 */
int statekv_prefill_frames_host(statekv_handle* h, int32_t frames, const void* q_host,
                                const void* k_host, const void* v_host, void* o_host,
                                void* cuda_stream);

/*
 * Text decode over the detailed state (关键设计 1: D_n keeps every frame's
 * K/V for text decoding; 关键设计 3: text continues the virtual positions
 * with the same static scale).  `tokens` new text tokens (1..16, and at most
 * T) take positions p = position_offset + n*T + j, j counting every text
 * token decoded since the last frame; their K', V are appended to D after
 * the rows already there, and each query row attends over all earlier D rows
 * (the whole video and earlier text) and, causally, over the new tokens:
 *   O = softmax(Q' [D_K]^T * mscale^2/sqrt(d), causal on the new rows) D_V.
 * Device pointers, contiguous, storage dtype:
 *   q, o : [S][L][Hq][tokens][d]     k, v : [S][L][Hkv][tokens][d] (pre-RoPE)
 * Supported: bf16 storage, d = 128, G*tokens <= 64 (else E_UNSUPPORTED).
 * Returns E_CAPACITY (nothing done) when the new rows do not fit in D
 * (n*T + decoded + tokens > max_frames*T).  Once a handle has decoded text,
 * the prefill entry points return E_INVALID_ARG until statekv_reset.  The
 * first call allocates the handle's decode scratch (partial results per
 * 2048-key chunk of D; E_OOM if that fails).  The first call of this and the
 * entry points below that allocate cannot be captured into a CUDA graph.
 * A captured call counts as made: its graph has to be replayed once before the
 * handle's next call, and a further replay repeats it at the same positions.
 */
int statekv_decode(statekv_handle* h, int32_t tokens, const void* q, const void* k,
                   const void* v, void* o, void* cuda_stream);

/*
 * RMS norm of the heads of Q and K ahead of the rotation, for models that
 * have one (Qwen3-VL): from this call on the prefill and decode entry points
 * compute x * w / sqrt(mean(x^2) + eps) in fp32 for every head of q and k
 * before they rotate it, w = q_weight or k_weight of the head's layer, float
 * [num_layers][head_dim], DEVICE memory (16-byte aligned) copied on
 * cuda_stream.  Both NULL turns the norm off again; one NULL is
 * E_INVALID_ARG.  The first call allocates the handle's copy.
 */
int statekv_set_qk_norm(statekv_handle* h, const float* q_weight, const float* k_weight, float eps,
                        void* cuda_stream);

/*
 * One verification step of speculative decoding over the detailed state: a
 * tree of `tokens` (1..64, at most T) drafted tokens attends over every D row
 * and, among itself, where its masks say.
 *   tree:  uint64 DEVICE [num_streams][tokens], bit j of entry i set where node
 *          i sees node j (its ancestors and itself);
 *   depth: int32 DEVICE [num_streams][tokens]: node i is at position
 *          position_offset + n*T + decoded text + depth[i].
 * q, k, v, o as for statekv_decode.  The drafted K', V stay in the handle's
 * own draft rows: D, its count and the text count do not change, so a call can
 * be repeated, until statekv_accept takes a path over.  bf16, head_dim 64 or
 * 128, G <= 64 (else E_UNSUPPORTED).  The first call allocates the draft rows
 * and the workspace (E_OOM).
 */
int statekv_decode_tree(statekv_handle* h, int32_t tokens, const void* q, const void* k, const void* v,
                        const uint64_t* tree, const int32_t* depth, void* o, void* cuda_stream);

/*
 * The accepted path of the last statekv_decode_tree becomes text: K', V of
 * nodes path[s][0..count-1] (int32 DEVICE [num_streams][count], a path from a
 * node of depth 0 down, so that node i of it is at depth i; the same count
 * for every stream) are appended to D and the text count grows by count.
 * E_INVALID_ARG without such a step before it, or count > its tokens;
 * E_CAPACITY when the rows do not fit.  A node out of range is recorded in the
 * device status and its row skipped.  count = 0 drops the draft.
 */
int statekv_accept(statekv_handle* h, int32_t count, const int32_t* path, void* cuda_stream);

/*
 * statekv_decode with block-sparse attention (statekv_sparse_attention below):
 * each new token attends to the `top` (1..1024) 64-row blocks of D that 8-bit
 * scores of its query choose per KV head, and to the rows since the last
 * complete block.  Block summaries of D are kept by the handle and brought up
 * to date by this call.  tokens 1..T; bf16, head_dim 64 or 128, G <= 16, D of
 * at most 2,097,152 rows (else E_UNSUPPORTED).  The first call allocates the
 * summaries (E_OOM).
 */
int statekv_decode_sparse(statekv_handle* h, int32_t tokens, int32_t top, const void* q, const void* k,
                          const void* v, void* o, void* cuda_stream);

/*
 * statekv_decode for a whole text prompt: 1..T tokens at once, d = 64 or 128,
 * any G <= 64 (the attention is that of statekv_paged_attention below; bf16,
 * else E_UNSUPPORTED).  The first call allocates the workspace (E_OOM).
 */
int statekv_decode_prompt(statekv_handle* h, int32_t tokens, const void* q, const void* k, const void* v,
                          void* o, void* cuda_stream);

/* Text tokens decoded since the last reset (-1 for a NULL handle). */
int64_t statekv_text_tokens(const statekv_handle* h);

/*
 * Borrowed DEVICE pointers to the compressed state C_{n-1} of (stream s,
 * layer) after the last step: k, v -> [Hkv][pitch][d], pos -> [Hkv][pitch]
 * int32 virtual positions; the first *count slots of each head are live
 * (count = min(B, n*T)), in slot order.  *pitch = B + T.  Valid until the
 * next call that changes the handle.  Any output pointer may be NULL.
 */
int statekv_get_compressed(statekv_handle* h, int32_t s, int32_t layer,
                           const void** k, const void** v, const int32_t** pos,
                           int32_t* count, int32_t* pitch);

/*
 * Borrowed DEVICE pointers to the detailed state D_{n-1} of (s, layer):
 * k, v -> [Hkv][pitch][d] with row r = virtual position r - position_offset
 * (post-RoPE K, V as given); *count = n*T (+ decoded text tokens) live rows per head,
 * *pitch = max_frames*T.  Any output pointer may be NULL.
 */
int statekv_get_detailed(statekv_handle* h, int32_t s, int32_t layer,
                         const void** k, const void** v, int64_t* count,
                         int64_t* pitch);

/* Frames processed so far (n). */
int64_t statekv_frame_index(const statekv_handle* h);

/* Forget all frames: n = 0, c = 0 (allocations kept, contents stale). */
int statekv_reset(statekv_handle* h);

/*
 * Synchronise cuda_stream, then report and clear the device status word:
 * STATEKV_OK, STATEKV_E_TIMEOUT (a bounded wait inside a kernel gave up; that
 * launch's outputs are invalid) or STATEKV_E_DEVICE.
 */
int statekv_check_device_status(statekv_handle* h, void* cuda_stream);

/* ------------------------------------------------------------- test hooks */

/*
 * Importance scores of the last step (关键设计 2) for (s, layer):
 * scores -> [Hkv][pitch] fp32, pool_pos -> [Hkv][pitch] int32, both in pool
 * slot order before the Top-B update (slots [0,c) held C_{n-1}, slots
 * [c, c+T) the frame's tokens); *m = c + T candidates.  Borrowed DEVICE
 * pointers, valid until the next step.
 */
int statekv_get_scores(statekv_handle* h, int32_t s, int32_t layer,
                       const float** scores, const int32_t** pool_pos,
                       int32_t* m, int32_t* pitch);

/* Borrowed DEVICE pointer to the rotated queries Q' of the last frame step
 * ([S][L][Hq][T][d], storage dtype) or, after a text decode (dense, sparse or
 * a prompt or a tree), of the last such step ([S][L][Hq][tokens][d]).  Valid until the next step. */
int statekv_get_rotated_query(statekv_handle* h, const void** q_rot);

/* Set the frame index n (teacher forcing / resume); 0 <= n < max_frames. */
int statekv_set_frame_index(statekv_handle* h, int64_t n);

/*
 * Teacher forcing / resume: overwrite C of (s, layer) with count rows per KV
 * head from DEVICE buffers k, v [Hkv][count][d] (post-RoPE, storage dtype)
 * and pos [Hkv][count] int32.  count must equal min(B, n*T) for the current
 * frame index n.  Copies are enqueued on cuda_stream.
 */
int statekv_set_compressed(statekv_handle* h, int32_t s, int32_t layer,
                           const void* k, const void* v, const int32_t* pos,
                           int32_t count, void* cuda_stream);

/*
 * Per-kernel timing with CUDA events recorded on the launch stream around
 * every launch while enabled.  statekv_profile_read synchronises, then
 * returns for kernel id (STATEKV_KERNEL_*) the summed device milliseconds
 * and the number of launches since profiling was last enabled.
 * statekv_profile_kernels restricts the bracketing to the kernels whose bit
 * (1 << STATEKV_KERNEL_*) is set in mask (default: all).  An event recorded
 * between two launches also ends the overlap of the second launch's start
 * with the first one's end (below), so timing only the kernel of interest
 * keeps the others' overlap.
 *
 * Overlap of consecutive launches within a frame sequence: the RoPE kernel
 * of frame n+1 starts while the selection of frame n still runs (its query
 * rows do not depend on it; its writes of the frame's keys into the pool
 * wait for the selection to finish), the attention kernel's set-up
 * overlaps the RoPE kernel's end, and the selection is launched while the
 * attention kernel still runs and starts work as soon as it has finished
 * (programmatic dependent launch).  Any other
 * operation on the stream between two calls separates them as usual.
 */
int statekv_profile_enable(statekv_handle* h, int enable);
int statekv_profile_kernels(statekv_handle* h, uint32_t mask);
int statekv_profile_read(statekv_handle* h, int32_t kernel, double* total_ms,
                         int64_t* launches);

/* ------------------------------------------------- allocation-free entry */

/*
 * No counterpart in the paper: a deployment convenience.
 *
 * Frame attention and importance scores for callers that cannot allocate
 * device memory -- whose memory is owned by another allocator (an inference
 * server's pool, a framework hosting this library as a plugin) or that must
 * avoid the device-wide synchronisation cudaMalloc/cudaFree can cause.  It
 * creates no handle and calls no cudaMalloc, cudaFree or other allocating
 * routine; its only scratch (the per-query-tile column sums of P) is a
 * file-scope 16 MiB __device__ array that every GPU loading this library
 * holds until the process exits.
 *
 * Computes, per unit u (one KV head of one layer and stream), exactly the
 * attention and scores of one statekv_prefill_frame step:
 *   o      = softmax(q_rot pool_k^T * logit_scale, masked) pool_v
 *   scores = s_j, the mean over the group*frame_tokens query rows of P[:, j]
 * where pool rows [0, compressed) are compressed keys (visible to every
 * query) and rows [compressed, compressed + frame_tokens) are the frame's
 * keys in token order (frame key i' visible to query token i iff i' <= i).
 * DEVICE pointers on the current device, caller-owned, contiguous, storage
 * dtype (STATEKV_BF16 or STATEKV_F32), 16-byte aligned:
 *   q_rot  [units][group * frame_tokens][head_dim]  rotated queries, g-major
 *   pool_k, pool_v [units][pool_rows][head_dim]     pool_rows >= compressed + frame_tokens
 *   o      [units][group * frame_tokens][head_dim]  written
 *   scores [units][compressed + frame_tokens] fp32  written
 *   status uint32[4] device status word, required (4-byte aligned): the
 *          call first zeroes it on cuda_stream; a bounded device wait that
 *          gives up then writes STATEKV_E_TIMEOUT into status[0] (the wait
 *          site into status[1]) and leaves o and scores unspecified.  Read
 *          it once the stream has passed the call.
 * logit_scale = mscale^2 / sqrt(head_dim).  Returns STATEKV_E_CAPACITY when
 * units * ceil(group*frame_tokens / R) * round_up(pool_rows, 128) * 4 bytes
 * exceeds the 16 MiB scratch (R = 128 query rows per tile for bf16, 16 for
 * fp32), STATEKV_E_UNSUPPORTED for head_dim not in {64, 128}.
 * The first call on a device takes the scratch's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  All calls on a device share the scratch:
 * calls that overlap on the GPU race and must be serialised by the caller.
 * Work is enqueued on cuda_stream; results are valid once it passes the call.
 */
int statekv_attend_scores_static(const void* q_rot, const void* pool_k,
                                 const void* pool_v, int32_t units,
                                 int32_t group, int32_t frame_tokens,
                                 int32_t head_dim, int32_t pool_rows,
                                 int32_t compressed, double logit_scale,
                                 int32_t dtype, void* o, float* scores,
                                 uint32_t* status, void* cuda_stream);

/* ------------------------------------------- text operators, handle-free */

/*
 * Operators of text decoding over a cache of keys and values (a handle's
 * detailed state D, or any other cache), for callers that hold their own
 * tensors.  No counterpart in the page except for the rotation (关键设计 3);
 * the handle's statekv_decode_tree, statekv_accept and statekv_decode_sparse
 * run the same kernels over D.
 *
 * Tensors are views [batch][heads][tokens][head_dim] of DEVICE memory on the
 * current device: the last dimension contiguous, the other strides (in
 * elements) free but not negative, every row on a 16-byte boundary (the stride
 * of a dimension of one entry is not looked at).  An input
 * may repeat its entries (stride 0), but for the keys and values of
 * statekv_tree_attention, which are read in tiles; no two rows of an output may
 * share memory (E_INVALID_ARG unless, taken from the smallest up, each stride
 * spans all that the smaller ones reach).  The batch is sequences x layers:
 * batch entry n belongs to sequence n / layers, and lengths, trees, paths and
 * destination rows have one entry per sequence.  Query head j uses KV head j / (q_heads / kv_heads).  Outputs
 * must not overlap inputs unless said otherwise.
 *
 * `lengths` (int32, device) gives each sequence's rows in the cache; where it
 * is NULL every sequence has `length` rows.  A length, count, row or node out
 * of range is known only on the device: the kernel clamps or skips it, and
 * records STATEKV_E_DEVICE in the status word.  `status` is a device
 * uint32[4] (4-byte aligned, required), zeroed once by the caller and kept
 * over any number of calls: the first failure stays in it (status[0] a
 * STATEKV_E_* code, as for statekv_check_device_status) until the caller
 * clears it.
 *
 * Calls allocate nothing, keep nothing between calls and may be captured into
 * CUDA graphs.  Calls that overlap on the GPU need workspaces of their own;
 * they may share a status word.  Scales of scores are in (1e-30, 1e30).
 */
typedef struct statekv_view {
    void*   data;
    int64_t batch_stride, head_stride, token_stride;   /* in elements */
} statekv_view;

#define STATEKV_BLOCK 64            /* cache rows per summarised block */

/*
 * RMS norm of every head of Q and K, rotation at the tokens' virtual
 * positions, and the store of Q, K and V, in one pass:
 *   y = x * w / sqrt(mean(x^2) + eps), rotated by the angles p * omega[k]
 * (element k with element k + head_dim/2), in fp32, rounded once.
 *   q -> q_out rows t; k -> k_out and v -> v_out rows out_rows[sequence] + t
 *   (row t where out_rows is NULL), of out_capacity rows.
 * q_weight, k_weight [weight_rows][head_dim] in weight_dtype (16-byte
 * aligned), batch entry n using row n % weight_rows (1: one weight for all;
 * the number of layers: one per layer); NULL: no norm of that tensor.  omega:
 * float64 [head_dim/2], radians per position.  Token t is at position
 * position0 + positions[n / position_layers][t] (int32, rows position_stride
 * >= tokens apart, 0 for one row shared by all), position0 + t where
 * positions is NULL.  v.data
 * and v_out.data may both be NULL.  Each output may be its own input (the
 * same view).  A sequence whose rows do not fit in k_out is recorded, and its
 * K and V are not stored.
 * dtype: STATEKV_BF16 or STATEKV_F32; head_dim 64 or 128.
 */
typedef struct statekv_norm_rope_args {
    statekv_view q, k, v, q_out, k_out, v_out;
    const void* q_weight;
    const void* k_weight;
    const double* omega;
    const int32_t* positions;
    const int32_t* out_rows;
    uint32_t* status;
    int64_t position0;
    int32_t position_stride, position_layers;
    int32_t batch, layers, q_heads, kv_heads, tokens, head_dim;
    int32_t out_capacity, weight_rows;
    int32_t dtype, weight_dtype;
    float eps;
} statekv_norm_rope_args;
int statekv_norm_rope(const statekv_norm_rope_args* args, void* cuda_stream);

/*
 * Attention of a tree of `tokens` (1..64) drafted tokens over the cache:
 *   o = softmax(q [cache_K[:length]; K_new]^T * scale, masked) [cache_V; V_new]
 * Every cache row is visible; drafted token j is visible to drafted token i
 * iff bit j of tree[i] is set (the node's ancestors and itself; any mask is
 * allowed).  q and k_new are already rotated.  A key that is masked, and
 * cache rows from `length` on, contribute nothing whatever they hold
 * (infinities and NaN included); a row that sees no key at all gets zeros.
 * Scores, softmax sums and the output are fp32; the probabilities are rounded
 * to bf16 (2^-8 of each) for the product with V, their sum takes them unrounded.
 * tree: uint64 [sequences][tree_stride >= tokens], or tree_stride 0 for one
 * tree shared by all; bits from `tokens` on are ignored.
 * bf16, head_dim 64 or 128, q_heads / kv_heads <= 64, cache_rows >= 0 rows
 * per head in the cache views.  workspace: device memory of
 * statekv_tree_attention_workspace() bytes, 16-byte aligned, contents
 * irrelevant (NULL where that is 0: a few short caches); the function depends
 * on the current device and returns -1 for sizes that the call would refuse.
 * With the same kv_heads it rises or stays with every other argument, so one
 * workspace for the largest serves all; with more KV heads for the same query
 * heads it may fall.  The results do not depend on the workspace or on the
 * other calls, but sums are grouped by the whole batch: they agree between
 * batchings up to rounding.
 */
typedef struct statekv_tree_args {
    statekv_view q, out, k_new, v_new, k_cache, v_cache;
    const uint64_t* tree;
    const int32_t* lengths;
    uint32_t* status;
    void* workspace;
    int64_t workspace_bytes;
    double scale;
    int32_t tree_stride, length;
    int32_t batch, layers, q_heads, kv_heads, tokens, head_dim, cache_rows;
} statekv_tree_args;
int64_t statekv_tree_attention_workspace(int32_t batch, int32_t q_heads, int32_t kv_heads,
                                         int32_t tokens, int32_t head_dim, int32_t cache_rows);
int statekv_tree_attention(const statekv_tree_args* args, void* cuda_stream);

/*
 * The accepted drafted tokens join the cache: for i < counts[sequence],
 *   cache row length + i = new row path[sequence][i],
 * K and V of every layer and head; other rows stay as they are.  path: int32
 * [sequences][path_stride >= path_len] (path_stride 0: shared), each entry in
 * [0, tokens), in any order.  counts (int32, each 0..path_len) NULL: path_len
 * for all.  new_lengths, if not NULL, receives length + count (memory of its
 * own, not the `lengths` or `counts` array).  A sequence whose rows do not
 * fit appends nothing; an entry out of range is skipped.  Any head_dim of
 * whole 16-byte units up to 512; dtype STATEKV_BF16 or STATEKV_F32.
 */
typedef struct statekv_append_args {
    statekv_view k_new, v_new, k_cache, v_cache;
    const int32_t* path;
    const int32_t* counts;
    const int32_t* lengths;
    int32_t* new_lengths;
    uint32_t* status;
    int32_t path_stride, path_len, length;
    int32_t batch, layers, kv_heads, tokens, head_dim, cache_rows, dtype;
} statekv_append_args;
int statekv_append_accepted(const statekv_append_args* args, void* cuda_stream);

/*
 * Summaries of the complete blocks of STATEKV_BLOCK cache rows, block b =
 * rows [64 b, 64 b + 64): the mean key (fp32, from a sum exact to fp32) as
 * 8-bit codes of one scale,
 *   scale = max |mean| / 127,  code = round_to_even(mean * (127 / max |mean|)),
 * in fp32 (where max |mean| < 2^-100, mean and maximum are multiplied by 2^64
 * for the code, so that the factor stays finite; zeros give zeros).
 * Brings up to date the blocks that the last `appended` rows completed, [
 * (length - appended) / 64, length / 64 ); the others are left as they are.
 * codes: int8 [batch][kv_heads][blocks][head_dim] (8-byte aligned), scales:
 * float [batch][kv_heads][blocks], blocks >= cache_rows / 64 (else
 * E_CAPACITY).  Keys, and their sums over a block in fp32, must be finite.
 * bf16, head_dim 64 or 128.
 */
typedef struct statekv_summary_args {
    statekv_view k_cache;
    int8_t* codes;
    float* scales;
    const int32_t* lengths;
    uint32_t* status;
    int32_t length, appended, blocks;
    int32_t batch, layers, kv_heads, head_dim, cache_rows;
} statekv_summary_args;
int statekv_block_summaries(const statekv_summary_args* args, void* cuda_stream);

/*
 * Block-sparse attention of the last `tokens` rows of each sequence over the
 * cache they are already part of (token j is row length - tokens + j).  With
 * first = length - tokens, each token and KV head
 *   1. scores the complete blocks of rows [0, first): the head group's query
 *      rows are rounded to 8 bits with one scale, qi = round_to_even(q * (127 /
 *      max |q|)) as for the summaries, and score_b = float(max over the group
 *      of qi . code_b) * scale_b.  The products are whole numbers, so the scores, and the choice,
 *      do not depend on the order of summation;
 *   2. keeps the `top` best (1..1024), ties to the lower block;
 *   3. attends over those blocks' rows, the rows since the last complete block
 *      and, causally, the new rows.
 * With top >= first / 64 this is full attention.  Precision of the attention as
 * in statekv_tree_attention.  selected, if not NULL:
 * int32 [batch][kv_heads][tokens][top], the chosen blocks in ascending order,
 * -1 from the last one on.  codes and scales as statekv_block_summaries
 * writes them, up to date for every complete block before `first`, codes
 * 16-byte aligned.  bf16, head_dim 64 or 128, q_heads / kv_heads <= 16,
 * at most 32768 blocks, tokens <= length (a shorter sequence gives zeros for the
 * tokens before its first row).  No workspace.
 */
typedef struct statekv_sparse_args {
    statekv_view q, out, k_cache, v_cache;
    const int8_t* codes;
    const float* scales;
    const int32_t* lengths;
    int32_t* selected;
    uint32_t* status;
    double scale;
    int32_t length, top, blocks;
    int32_t batch, layers, q_heads, kv_heads, tokens, head_dim, cache_rows;
} statekv_sparse_args;
int statekv_sparse_attention(const statekv_sparse_args* args, void* cuda_stream);

/*
 * ------------------------------------------------------ paged caches
 *
 * A pool of pages holds the rows of many sequences: views
 * [pages][kv_heads][page_rows][head_dim] (batch_stride is the stride of a
 * page), num_pages of them.  table: int32 [batch][table_stride], row i of batch
 * entry n is row i % page_rows of page table[n][i / page_rows]; a table row
 * holds table_pages <= table_stride entries, and with them a sequence at most
 * table_pages x page_rows rows (2^31 - 257 at most, of a plain cache too).
 * Entries past the last page in use are not looked
 * at; one in use that is out of [0, num_pages) is recorded (E_DEVICE): its rows
 * read as zeros, and nothing is written there.  Pages may be shared by entries
 * that only read them.  page_rows is a multiple of 16.  table NULL: a plain
 * cache, batch entry n is page n (num_pages >= batch), of any number of rows.
 * lengths (or length) and counts have one entry per sequence, as above; counts
 * NULL: `tokens` for all.  A count below 0, or past `tokens`, is recorded and
 * clamped.
 */

/*
 * New rows join their sequences: for i < counts[sequence],
 *   cache row length + i = new row i,
 * K and V of every layer and head; other rows stay as they are.  new_lengths,
 * if not NULL, receives length + count (memory of its own).  A sequence whose
 * rows do not fit in its table row appends nothing (recorded).  Batch entries
 * that write one page write the same row of it in any order: pages that are
 * appended to are not shared.  k_pages and v_pages do not overlap each other
 * (E_INVALID_ARG; they may lie side by side in one tensor) or the new rows.  Any
 * head_dim of whole 16-byte units up to 512; dtype STATEKV_BF16 or STATEKV_F32.
 */
typedef struct statekv_paged_append_args {
    statekv_view k_new, v_new, k_pages, v_pages;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* counts;
    int32_t* new_lengths;
    uint32_t* status;
    int32_t length, table_stride, table_pages, num_pages, page_rows;
    int32_t batch, layers, kv_heads, tokens, head_dim, dtype;
} statekv_paged_append_args;
int statekv_paged_append(const statekv_paged_append_args* args, void* cuda_stream);

/*
 * Attention of the last tokens of each sequence over the cache they are already
 * part of: with first = length - count, token j < count is row first + j and
 * sees the rows up to itself,
 *   o = softmax(q K[:first + j + 1]^T * scale) V[:first + j + 1],
 *   lse = log(sum over those rows of exp(q . k * scale)).
 * Any number of tokens (one, or a whole prompt), q already rotated.  Tokens from
 * count on (a padded batch), and those of a sequence shorter than its count
 * (recorded) past its length, give zeros and -infinity.  Rows that a token does
 * not see contribute nothing to it whatever they hold (infinities and NaN
 * included); a row whose scores are all -infinity gives zeros.
 * Scores, softmax sums and the output are fp32; the probabilities are rounded
 * to bf16 (2^-8 of each) for the product with V, their sum takes them unrounded.
 * lse, if not NULL: float [batch][q_heads][tokens].
 * bf16, head_dim 64 or 128, q_heads / kv_heads <= 64, that times tokens below 2^26.
 * K and V are read in tiles: their entries do not share memory (strides above 0).  workspace: device memory of
 * statekv_paged_attention_workspace() bytes, 16-byte aligned, contents
 * irrelevant (NULL where that is 0: a few short caches; cache_rows: the most that
 * a sequence can hold); the size depends on the current device and, with the
 * same kv_heads, rises or stays with every argument (-1 for sizes that the call
 * would refuse).  The results do not
 * depend on the workspace or on other calls, but sums are grouped by the whole
 * batch: they agree between batchings up to rounding.
 */
typedef struct statekv_paged_attention_args {
    statekv_view q, out, k_pages, v_pages;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* counts;
    float* lse;
    uint32_t* status;
    void* workspace;
    int64_t workspace_bytes;
    double scale;
    int32_t length, table_stride, table_pages, num_pages, page_rows;
    int32_t batch, layers, q_heads, kv_heads, tokens, head_dim;
} statekv_paged_attention_args;
int64_t statekv_paged_attention_workspace(int32_t batch, int32_t q_heads, int32_t kv_heads,
                                          int32_t tokens, int32_t head_dim, int32_t cache_rows);
int statekv_paged_attention(const statekv_paged_attention_args* args, void* cuda_stream);

/*
 * What attention every cache row received from the tokens of a
 * statekv_paged_attention call, from its queries and log-sum-exps:
 *   out[row] = before[row] + sum over the head group's queries that see the row
 *              of exp(q . k * scale - lse),
 * rows from the length on as before.  q, lengths and counts as for that call;
 * a query whose lse is infinite adds nothing (a key that is not finite gives
 * its own row what comes of it, and no other).  before, out: float
 * [batch][kv_heads][weight_rows] (before NULL: zeros; out may be before, and shares
 * no memory with it otherwise), weight_rows at least the rows a sequence can hold (E_CAPACITY).  Scores and sums in
 * fp32, each row's sum in a fixed order (the same bits on every run).
 * bf16, head_dim 64 or 128, q_heads / kv_heads <= 64, that times tokens below 2^26;
 * q and K are read in tiles: their entries do not share memory.  No workspace.
 */
typedef struct statekv_attention_weights_args {
    statekv_view q, k_pages;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* counts;
    const float* lse;
    const float* before;
    float* out;
    uint32_t* status;
    double scale;
    int32_t length, table_stride, table_pages, num_pages, page_rows, weight_rows;
    int32_t batch, layers, q_heads, kv_heads, tokens, head_dim;
} statekv_attention_weights_args;
int statekv_attention_weights(const statekv_attention_weights_args* args, void* cuda_stream);

/*
 * Eviction by accumulated weight: every batch entry and KV head keeps
 * min(length, keep) of its rows, and they become, in their order, rows 0.. of
 * the pages that out_table names.  Rows below `sinks` and the last `recent`
 * stay (sinks + recent <= keep); of the others those of the largest weight,
 * ties to the lower row, NaN below all.
 * k_out and v_out are pools of their own, or k_pages and v_pages themselves;
 * pages that out_table names are read by no entry of the call and named once.
 * (The rows move to fresh pages so that pages shared with other sequences stay as
 * they are.)  Rows of out pages past the last kept row stay as they are.
 *   weights      float [batch][kv_heads][weight_rows], weight_rows at least the
 *                rows a sequence can hold
 *   weights_out  float [batch][kv_heads][out_rows]: the kept rows' weights, then zeros
 *   kept         int32 [batch][kv_heads][keep]: the kept rows, then -1
 *   new_lengths  int32 [sequences]: min(length, keep), if not NULL
 * none of which shares memory with another or an input.  out_rows >= keep; the
 * out table holds out_table_pages * out_page_rows >= keep rows (E_CAPACITY); the pools
 * may have pages of different sizes, and either table may be NULL.  out_table NULL:
 * batch entry n's rows go to page n, a plain cache of out_page_rows >= keep rows.
 * Where either table is NULL no row of k_out or v_out shares memory with one of the
 * source's, and never K's with V's (E_INVALID_ARG).  Any head_dim of whole 16-byte
 * units up to 512; dtype STATEKV_BF16 or STATEKV_F32; a sequence holds at
 * most 2^22 rows.
 */
typedef struct statekv_evict_args {
    statekv_view k_pages, v_pages, k_out, v_out;
    const int32_t* table;
    const int32_t* out_table;
    const int32_t* lengths;
    const float* weights;
    float* weights_out;
    int32_t* kept;
    int32_t* new_lengths;
    uint32_t* status;
    int32_t length, table_stride, table_pages, num_pages, page_rows, weight_rows;
    int32_t out_table_stride, out_table_pages, out_num_pages, out_page_rows, out_rows;
    int32_t keep, sinks, recent;
    int32_t batch, layers, kv_heads, head_dim, dtype;
} statekv_evict_args;
int statekv_evict_rows(const statekv_evict_args* args, void* cuda_stream);

/*
 * Verification of a drafted tree against the target's probabilities, with
 * random numbers from the caller: which path of it stands, and the token after
 * it, so that the tokens are distributed as if drawn from the target one by one.
 *   tree     uint64 [sequences][tree_stride >= tokens] (0: one for all), as for
 *            statekv_tree_attention; node i's parent is the highest lower node
 *            that its mask names, none: it follows the text so far
 *   target   float, rows [sequences][tokens + 1][vocab] (strides in elements):
 *            the target's probabilities after the text (row 0) and after node i (row i + 1)
 *   draft    the same of the draft's, from which the children of a node were
 *            drawn independently; rows of nodes without children are not read.  NULL: the
 *            children of a node are proposals without probabilities
 *   drafted  int32 [sequences][tokens], the nodes' tokens
 *   uniforms float [sequences][tokens + 1] in [0, 1): one per node, then one for
 *            the token at the end
 * From the text on, with p and q the current node's rows, c = 0 and R = 1, for
 * its children x in ascending order, u their uniforms:
 *   r(v) = max(p(v) - c q(v), 0);  if u q(x) R < r(x), x stands and is the
 *   current node; else c += R, R = sum of max(p(v) - c q(v), 0) over v.
 * Without q: if u R < r(x), r = p without the refused tokens, x stands; else
 * R = max(R - r(x), 0).
 * When no child is left, the token is the lowest v with
 *   sum over w <= v of r(w) > u * sum of r
 * (where that sum is 0, of p instead of r; where that is 0 too, token 0).
 * A child's own test is in 64 bits.  In sums each r(v) is off by at most 2^-47 and
 * rounded to a whole number of 2^-60, and whole numbers are added: the results do not
 * depend on the other sequences of the call.  Probabilities are in [0, 1] and sum to 1
 * up to rounding; NaN and negative ones count as 0, uniforms are clamped to [0, 1).
 * (Of other rows some nodes and some token come out.)
 *   path     int32 [sequences][tokens]: the accepted nodes, then -1
 *   counts   int32 [sequences], how many
 *   next     int32 [sequences]
 * as statekv_append_accepted takes them.  A drafted token out of [0, vocab) is recorded and
 * refused.  tokens 1..64, vocab below 2^26.
 */
typedef struct statekv_verify_args {
    const float* target;
    const float* draft;
    const int32_t* drafted;
    const uint64_t* tree;
    const float* uniforms;
    int32_t* path;
    int32_t* counts;
    int32_t* next;
    uint32_t* status;
    int64_t target_stride, target_row, draft_stride, draft_row;   /* of a sequence, of a row */
    int32_t tree_stride, sequences, tokens, vocab;
} statekv_verify_args;
int statekv_verify_tree(const statekv_verify_args* args, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* STATEKV_H_ */
