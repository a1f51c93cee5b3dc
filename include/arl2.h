/*
 * arl2.h — C ABI of the ARL2 hybrid attention layer for NVIDIA B200 (sm_100a).
 *
 * The layer ("Attend Locally, Remember Linearly", technical summary §2.1
 * Hybrid Attention Decomposition and §2.2 Memory State Management) runs once
 * per latent frame and denoising pass.  For every stream b and head h:
 *
 *   O = softmax(Q K^T * scale) V  +  (Q W_q[h]) S_{N-1}[b,h]
 *
 * the first term being the intra-frame bidirectional softmax branch over the
 * frame's L tokens (§2.1 item 1) and the second the inter-frame read of the
 * fixed-size state through the per-head feature map phi_q (§2.1 "Adaptation",
 * "Output"), every token reading the same pre-update state (§2.2 "Frame-Level
 * Access").  On the clean pass only (§2.2 "Clean-Pass Updates"), after the
 * read, the state is updated once for the frame (§2.1 "State Update"):
 *
 *   K' = rownorm(K W_k[h]),  V' = V W_v[h]
 *   S_N = alpha S_{N-1} + K'^T diag(beta) (V' - K' S_{N-1})
 *
 * Conventions used by every entry point:
 *   - Token tensors (q, k, v, out, x) are [B][L][H][d], dense, in the
 *     handle's dtype, device memory, 16-byte aligned.
 *   - Feature maps W are [H][d][d] with row = input feature (x' = x W).
 *   - The state S is fp32 [B][H][d][d], row = key feature, column = value
 *     feature.  It is owned by the handle.
 *   - alpha is fp32 [B][H] (one forget gate per stream and head for the
 *     frame; headwise gating, the form the pages adopt), or, for a handle
 *     created with gating = ARL2_GATE_ELEMENTWISE, fp32 [B][H][d] (one gate
 *     per key feature: S_N = diag(alpha) S_{N-1} + ..., the variant the
 *     atlas summary's "Surprising findings" compares).  beta is fp32
 *     [B][H][L] (one rate per token).
 *   - Every call is asynchronous and stream-ordered on the given stream: it
 *     makes no host synchronisation and allocates nothing after
 *     arl2_create.  A call that returns anything but ARL2_OK enqueued
 *     nothing, except ARL2_ERR_CUDA, which reports a failed launch or copy.
 *   - The caller keeps ownership of every pointer it passes; the handle owns
 *     the state, its derived copies, the weight copies and all workspaces.
 *   - The caller's current CUDA device must be the handle's device.
 *   - A handle is not thread-safe: calls on one handle must be serialised
 *     by the caller, and calls enqueued on different streams must not
 *     overlap on the GPU.
 */
#ifndef ARL2_H
#define ARL2_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ARL2_OK = 0,
    ARL2_ERR_INVALID_ARG = -1,  /* null pointer, bad flag, wrong device     */
    ARL2_ERR_SHAPE = -2,        /* a dimension out of the supported range   */
    ARL2_ERR_ALIGN = -3,        /* a tensor pointer not 16-byte aligned     */
    ARL2_ERR_CUDA = -4,         /* a CUDA runtime or driver call failed     */
    ARL2_ERR_OOM = -5,          /* device allocation failed in arl2_create  */
    ARL2_ERR_TIMEOUT = -6,      /* a kernel's bounded wait ran out          */
    ARL2_ERR_UNSUPPORTED = -7   /* valid, but not built for this dtype/size */
} arl2_status;

typedef enum { ARL2_BF16 = 0, ARL2_FP32 = 1 } arl2_dtype;

/* Kernel family.  AUTO picks the tensor-core (tcgen05) kernels for bf16 with
 * head_dim 128 and the fp32 SIMT kernels for fp32.  SIMT forces the SIMT
 * kernels (fp32 arithmetic) for either dtype; it exists to cross-check the
 * tensor-core kernels on the GPU and is not a fallback: AUTO never falls
 * back to it. */
typedef enum { ARL2_IMPL_AUTO = 0, ARL2_IMPL_SIMT = 1 } arl2_impl;

/* Granularity of the forget gate alpha (see the conventions above). */
typedef enum { ARL2_GATE_HEADWISE = 0, ARL2_GATE_ELEMENTWISE = 1 } arl2_gating;

/* How the frame's tokens reach the state.  FRAME (the method, technical
 * summary §2.2 "Frame-Level Access"): every token reads S_{N-1} and the
 * clean pass updates once.  TOKEN (the ablation the pages compare with it):
 * token i reads the state left by tokens 0..i-1 of the pass and then updates
 * it with the delta rule, S <- G_i S + beta_i k'_i^T (v'_i - k'_i S), the
 * forget gate acting once with token 0 (G_0 = alpha, G_i = 1); every pass
 * reads through its own sequential states, so alpha and beta are required on
 * every pass, and only the clean pass keeps the final state.  With bf16 and
 * d = 128 TOKEN runs on tensor-core kernels (a per-chunk preparation, then a
 * scan over 128-token chunks with the fp32 state in TMEM and bf16 chunk
 * operands); otherwise on fp32 SIMT kernels (bf16 inputs are widened).  With
 * bf16 its output is rounded twice (the intra-frame term, then the sum). */
typedef enum { ARL2_ACCESS_FRAME = 0, ARL2_ACCESS_TOKEN = 1 } arl2_access;

typedef struct arl2_handle arl2_handle;

typedef struct {
    int batch;             /* B >= 1: independent streams                     */
    int heads;             /* H >= 1                                          */
    int head_dim;          /* d: 128 for bf16 tensor-core kernels; 1..128 SIMT */
    int tokens_per_frame;  /* L >= 1                                          */
    arl2_dtype dtype;      /* dtype of q, k, v, out and the feature maps      */
    const void* w_q;       /* device [H][d][d], dtype; copied at create       */
    const void* w_k;
    const void* w_v;
    float softmax_scale;   /* 0 selects 1/sqrt(d)                             */
    int host_staging;      /* 0: none; 1: device staging buffers for the
                              host-buffer calls (arl2_frame_forward_host,
                              arl2_frame_forward_hidden_host), copies on the
                              caller's stream; 2: two sets of them, and the
                              copies run on the handle's own streams so that
                              one call's input copies overlap the previous
                              call's pass and output copy (see
                              arl2_frame_forward_host); other nonzero values
                              act as 1                                        */
    arl2_impl impl;
    int max_ctas;          /* 0: the tensor-core attention kernel may use every
                              SM; > 0 caps its persistent grid (co-scheduling
                              with other work, tests of the split schedule)   */
    arl2_gating gating;    /* HEADWISE: alpha [B][H]; ELEMENTWISE: [B][H][d]  */
    arl2_access access;    /* FRAME (the method) or TOKEN (the ablation)      */
    /* Optional gate projections (see arl2_frame_forward_hidden).  NULL w_gate:
     * none, and hidden_dim, b_gate are ignored. */
    int hidden_dim;        /* D: width of the hidden states; a multiple of 8;
                              needs 2 H <= 96                                 */
    const void* w_gate;    /* device [D][2H] in dtype, 16-byte aligned; column
                              h gives head h's alpha logit, column H + h its
                              beta logit; copied at create                    */
    const float* b_gate;   /* device fp32 [2H], 16-byte aligned; copied       */
} arl2_config;

/* Create a layer on the current device.  Validates cfg, allocates the zeroed
 * state S_0 = 0 and every workspace, and copies the three feature maps
 * (stream-ordered on `stream`).  On success *out receives the handle.
 * Errors: INVALID_ARG (null cfg/out/weights, w_gate without b_gate), SHAPE
 * (also hidden_dim with w_gate), ALIGN (weights), UNSUPPORTED (dtype/head_dim
 * the chosen kernels do not handle; gate projections with elementwise
 * gating), OOM, CUDA. */
arl2_status arl2_create(const arl2_config* cfg, cudaStream_t stream, arl2_handle** out);

/* One denoising pass of one latent frame (technical summary §2.1, §2.2).
 * Writes out = O_intra + O_inter for every token, reading S_{N-1}.  When
 * clean_pass is nonzero, then also updates the state in place to S_N; alpha
 * and beta are read only in that case and may be NULL otherwise (with
 * access = ARL2_ACCESS_TOKEN they are read on every pass, see above).
 * q, k, v, out: device [B][L][H][d] dtype, 16-byte aligned; out must not
 * alias q, k or v.  alpha: device fp32 [B][H] ([B][H][d] with elementwise
 * gating); beta: device fp32 [B][H][L]. */
arl2_status arl2_frame_forward(arl2_handle* h, const void* q, const void* k, const void* v,
                               const float* alpha, const float* beta, int clean_pass,
                               void* out, cudaStream_t stream);

/* arl2_frame_forward on HOST buffers: copies q, k, v (and alpha, beta on a
 * clean pass) from host memory into the handle's device staging buffers,
 * runs the pass, and copies out back to host memory.  The call is complete
 * when `stream` reaches its end; host buffers should be pinned for the
 * copies to be asynchronous, and the caller must not touch them until then.
 * host_staging = 1: every copy is ordered on `stream`.  host_staging = 2:
 * consecutive calls alternate between two staging sets; the input copies
 * run on the handle's copy-in stream (once the pass that last used the set
 * is done) and may start before earlier work on `stream` has finished, so
 * the host inputs must hold their values when the call is made; the pass
 * runs on `stream` after them; the output copy runs on the copy-out stream
 * and `stream` waits for it.  Needs a handle created with host_staging != 0
 * (INVALID_ARG otherwise). */
arl2_status arl2_frame_forward_host(arl2_handle* h, const void* q, const void* k, const void* v,
                                    const float* alpha, const float* beta, int clean_pass,
                                    void* out, cudaStream_t stream);

/* Gate projections (technical summary §2.1 "State Update": alpha and beta
 * are learned per-token projections; the pages give no form, and this is
 * the reading the library takes).  For hidden states x (device [B][L][D] in
 * dtype, 16-byte aligned; the input of the layer's QKV projection):
 *   a_ih = x_i . w_gate[:, h] + b_gate[h],  g_ih = x_i . w_gate[:, H+h] + b_gate[H+h]
 *   beta[b][h][i] = sigmoid(g_ih)
 *   alpha[b][h]   = sigmoid((1/L) sum_i a_ih)   (one forget gate per frame)
 * Writes alpha (device fp32 [B][H]) and beta (device fp32 [B][H][L]).
 * Needs a handle created with w_gate (INVALID_ARG otherwise); fp32
 * accumulation; one kernel. */
arl2_status arl2_gates_apply(arl2_handle* h, const void* x, float* alpha, float* beta, cudaStream_t stream);

/* arl2_frame_forward with the gates projected from the hidden states x
 * (arl2_gates_apply into the handle's own buffers) on the passes that read
 * them: the clean pass (and, with token-level access, every pass).  x may be
 * NULL on other passes.  Needs a handle created with w_gate. */
arl2_status arl2_frame_forward_hidden(arl2_handle* h, const void* q, const void* k, const void* v,
                                      const void* x, int clean_pass, void* out, cudaStream_t stream);

/* arl2_frame_forward_hidden on HOST buffers (q, k, v, out [B][L][H][d] and x
 * [B][L][D], pinned for asynchronous copies), stream-ordered like
 * arl2_frame_forward_host.  Needs host_staging and w_gate at create. */
arl2_status arl2_frame_forward_hidden_host(arl2_handle* h, const void* q, const void* k, const void* v,
                                           const void* x, int clean_pass, void* out, cudaStream_t stream);

/* S := 0 for every stream and head (the start of a new video stream). */
arl2_status arl2_state_reset(arl2_handle* h, cudaStream_t stream);

/* Copy the fp32 state [B][H][d][d] to device memory dst (checkpoint, parity). */
arl2_status arl2_state_get(arl2_handle* h, float* dst_device, cudaStream_t stream);

/* Replace the state by the fp32 [B][H][d][d] device buffer src (resume). */
arl2_status arl2_state_set(arl2_handle* h, const float* src_device, cudaStream_t stream);

/* Apply one of the handle's per-head feature maps to a token tensor:
 * which = 0: out = x W_q;  1: out = rownorm(x W_k);  2: out = x W_v
 * (technical summary §2.1 "Adaptation").  x, out: device [B][L][H][d] in
 * the handle's dtype.  This is the stand-alone form of the projection the
 * forward pass fuses; it exists for step-level checks. */
arl2_status arl2_phi_apply(arl2_handle* h, int which, const void* x, void* out,
                           cudaStream_t stream);

/* Synchronise `stream`, then read and clear the handle's device error word.
 * Returns ARL2_ERR_TIMEOUT if a kernel gave up a bounded wait since the last
 * check (its outputs are then undefined), ARL2_ERR_CUDA on a CUDA error,
 * else ARL2_OK.  This is the one call that blocks the host. */
arl2_status arl2_device_status(arl2_handle* h, cudaStream_t stream);

/* Self-test of the failure path: one thread waits, with the bounded spin
 * the kernels' inter-CTA waits use, for a device word that nothing ever
 * sets; after limit_us (1 .. 1,000,000) it gives up, sets the handle's error
 * word and returns.  arl2_device_status then reports ARL2_ERR_TIMEOUT and
 * clears it; the context stays usable.  No fault, trap or unbounded wait. */
arl2_status arl2_selftest_wait_timeout(arl2_handle* h, unsigned limit_us, cudaStream_t stream);

/* Device bytes the handle holds (state, copies, weights, workspaces). */
size_t arl2_device_bytes(const arl2_handle* h);

/* Number of kernels this handle has enqueued (or recorded into a CUDA graph
 * capture) since creation; memsets and copies are not counted.  0 for NULL. */
unsigned long long arl2_kernel_launches(const arl2_handle* h);

/* Largest batch * tokens * heads * head_dim that arl2_state_update_noalloc
 * accepts: 4,194,304 elements (a 1560-token, 12-head, 128-wide frame of one
 * stream is 2,396,160). */
#define ARL2_NOALLOC_MAX_ELEMENTS (1u << 22)

/* The clean-pass state update, for callers that cannot allocate device
 * memory.  The ARL2 pages have no counterpart to this call: it exists for
 * deployment.  Some callers cannot call cudaMalloc where they run this step
 * (a plugin that only gets fixed buffers from its host framework, or a
 * process whose caching allocator has already reserved the device memory),
 * and arl2_create allocates.  This call allocates nothing: the caller owns
 * the state, and the two fp32 scratch arrays the update needs live in a
 * static device array inside the library (2 x ARL2_NOALLOC_MAX_ELEMENTS
 * floats = 32 MiB, held on every GPU that loads the library until exit).
 *
 * Computes, in place on `state` (fp32 [B][H][d][d], row = key feature):
 *   S = alpha S + K'^T diag(beta) (V' - K' S),  K' = rownorm(K W_k), V' = V W_v
 * k, v: device [B][L][H][d] in dtype; w_k, w_v: device [H][d][d] in dtype;
 * alpha: device fp32 [B][H]; beta: device fp32 [B][H][L].  All pointers
 * 16-byte aligned.  Uses the fp32 SIMT kernels for either dtype.
 *
 * The first call on each device looks up the scratch array's device address
 * (cudaGetSymbolAddress, with that device current) and sets kernel
 * attributes; make that first call before any stream capture.  That set-up
 * is cached for the life of the process, so do not use this call across a
 * cudaDeviceReset (the cached address and attributes would be stale).  Every
 * call shares the one scratch array and leaves its contents behind, so calls
 * whose work overlaps on the GPU (other streams, other threads) race: keep
 * them ordered.  Errors: INVALID_ARG (null pointer, bad dtype), SHAPE (a
 * dimension out of range: batch above 65535, heads above 1024, head_dim
 * above 128, or B*L*H*d > ARL2_NOALLOC_MAX_ELEMENTS), ALIGN, CUDA; nothing
 * is enqueued on an error other than CUDA. */
arl2_status arl2_state_update_noalloc(int batch, int heads, int head_dim, int tokens,
                                      arl2_dtype dtype, const void* k, const void* v,
                                      const void* w_k, const void* w_v, const float* alpha,
                                      const float* beta, float* state, cudaStream_t stream);

/* Release everything the handle owns.  Synchronises the device first.
 * NULL is ignored. */
void arl2_destroy(arl2_handle* h);

/* ------------------------------------------------------------------------
 * Softmax teacher layer with a KV cache.
 *
 * The attention the hybrid layer replaces, kept by the layers of a stack
 * that stay softmax: technical summary §1 ("KV Cache Growth": the cache of
 * keys and values grows with every generated frame) and §4 ("Efficiency":
 * the speedup of the hybrid stack grows with video length as that cache
 * comes to dominate).  The pages fix the cache's role, not its arithmetic;
 * this layer reads it as chunk-causal attention at frame granularity.  For
 * one pass of frame N (N = arl2_kv_frames before the call):
 *   O = softmax([Q Kc^T, Q K^T] * scale) [Vc; V]
 * where (Kc, Vc) hold the keys and values of the clean passes of frames
 * 0..N-1 in frame order, and (K, V) are this pass's own, attended
 * bidirectionally.  A clean pass then appends its k and v to the cache (the
 * same passes that update the hybrid layer's state, §2.2 "Clean-Pass
 * Updates"); other passes leave the cache alone.
 *
 * The cache holds max_frames frames and is allocated by arl2_kv_create; no
 * later call allocates.  Device memory held: 2 B max_frames L H d elements
 * of dtype plus workspaces; the part in use grows by 2 B L H d elements per
 * frame (arl2_kv_cache_bytes). */
typedef struct arl2_kv_handle arl2_kv_handle;

typedef struct {
    int batch;             /* B >= 1                                          */
    int heads;             /* H >= 1                                          */
    int head_dim;          /* d: 128 for the bf16 tensor-core kernel; 1..128 SIMT */
    int tokens_per_frame;  /* L >= 1                                          */
    int max_frames;        /* cache capacity in frames, >= 1; max_frames * L
                              <= 2^26                                         */
    arl2_dtype dtype;      /* dtype of q, k, v, out and the cache             */
    float softmax_scale;   /* 0 selects 1/sqrt(d)                             */
    int host_staging;      /* nonzero: staging buffers for
                              arl2_kv_frame_forward_host                      */
    arl2_impl impl;
    int max_ctas;          /* as in arl2_config                               */
} arl2_kv_config;

/* Create a teacher layer with an empty cache on the current device.
 * Errors: INVALID_ARG, SHAPE, UNSUPPORTED (dtype/head_dim), OOM, CUDA. */
arl2_status arl2_kv_create(const arl2_kv_config* cfg, cudaStream_t stream, arl2_kv_handle** out);

/* One pass of one frame: out = the attention above over the cached frames
 * and this pass's k, v; with clean_pass nonzero, then appends k and v to the
 * cache.  q, k, v, out: device [B][L][H][d] dtype, 16-byte aligned; out must
 * not alias q, k or v.  SHAPE (nothing enqueued) for a clean pass when the
 * cache already holds max_frames frames.  The frame count lives on the host:
 * a call recorded into a CUDA graph keeps the cache length it saw. */
arl2_status arl2_kv_frame_forward(arl2_kv_handle* h, const void* q, const void* k, const void* v,
                                  int clean_pass, void* out, cudaStream_t stream);

/* arl2_kv_frame_forward on HOST buffers (pinned for asynchronous copies):
 * q, k, v are copied into the handle's staging buffers, and out back, all
 * stream-ordered.  Needs host_staging != 0 (INVALID_ARG otherwise). */
arl2_status arl2_kv_frame_forward_host(arl2_kv_handle* h, const void* q, const void* k, const void* v,
                                       int clean_pass, void* out, cudaStream_t stream);

/* Empty the cache (the start of a new video stream).  Host-side only. */
arl2_status arl2_kv_reset(arl2_kv_handle* h);

/* Frames in the cache; -1 for NULL. */
int arl2_kv_frames(const arl2_kv_handle* h);

/* Copy the cached keys and values to device buffers k_dst, v_dst, each
 * [B][frames * L][H][d] dtype (dense).  Nothing is copied while empty. */
arl2_status arl2_kv_cache_get(arl2_kv_handle* h, void* k_dst, void* v_dst, cudaStream_t stream);

/* Replace the cache by `frames` frames from device buffers k_src, v_src,
 * each [B][frames * L][H][d] dtype (dense): resume from a checkpoint taken
 * with arl2_kv_cache_get.  frames = 0 empties the cache.  Errors:
 * INVALID_ARG, SHAPE (frames > max_frames), CUDA. */
arl2_status arl2_kv_cache_set(arl2_kv_handle* h, const void* k_src, const void* v_src, int frames,
                              cudaStream_t stream);

/* As arl2_device_status, for the teacher layer's kernels. */
arl2_status arl2_kv_device_status(arl2_kv_handle* h, cudaStream_t stream);

/* Device bytes the handle holds (the whole cache capacity included). */
size_t arl2_kv_device_bytes(const arl2_kv_handle* h);

/* Bytes of the cache in use: 2 B frames L H d elements of dtype. */
size_t arl2_kv_cache_bytes(const arl2_kv_handle* h);

/* Kernels this handle has enqueued since creation. */
unsigned long long arl2_kv_kernel_launches(const arl2_kv_handle* h);

/* Release the handle (synchronises the device first); NULL is ignored. */
void arl2_kv_destroy(arl2_kv_handle* h);

/* ------------------------------------------------------------------------
 * Rotary positions with up to four axes (a video token's time, height and
 * width; a text token's index).
 *
 * The first R = sum of axis_dim features of a head form R / 2 pairs; axis a
 * owns axis_dim[a] / 2 consecutive ones, in order.  Pair p, the i-th of axis
 * a, turns by the angle pos[n][a] * f_p:
 *   (x, y) -> (x cos - y sin, x sin + y cos)
 *   f_p = base^(-2 i / axis_dim[a])   (ARL2_FREQS_PER_AXIS)
 *   f_p = base^(-2 p / R)             (ARL2_FREQS_SHARED)
 * Features from R on pass through.  inverse turns by the opposite angle:
 * the rotation's transpose, hence the gradient with respect to its input.
 *
 * An arl2_rotary is a host-side plan (the frequencies); it holds no device
 * memory, is never written after its creation and may be used by several
 * threads, streams and devices at once. */
typedef enum { ARL2_PAIRS_ADJACENT = 0, ARL2_PAIRS_HALVES = 1 } arl2_pairs;
typedef enum { ARL2_FREQS_PER_AXIS = 0, ARL2_FREQS_SHARED = 1 } arl2_freqs;

typedef struct arl2_rotary arl2_rotary;

typedef struct {
    int head_dim;          /* d: 2..256                                       */
    int axes;              /* columns of the positions: 1..4                  */
    int axis_dim[4];       /* features of each axis: even, >= 0, sum in 2..d  */
    double base;           /* >= 1                                            */
    arl2_pairs pairs;      /* ADJACENT: features 2p, 2p + 1; HALVES: p, p + R/2 */
    arl2_freqs freqs;
} arl2_rotary_config;

/* Create a plan.  Errors: INVALID_ARG, SHAPE, OOM.  No CUDA call. */
arl2_status arl2_rotary_create(const arl2_rotary_config* cfg, arl2_rotary** out);

/* Turn q [tokens][q_heads][d] and k [tokens][k_heads][d] (dtype, device; the
 * heads of a token are contiguous, tokens are *_stride elements apart, 0 for
 * dense) by positions (device int32 [tokens][axes], any sign) into q_out and
 * k_out, in one launch.  An output may be its own input (in place) but not
 * overlap any tensor otherwise.  q_heads or k_heads may be 0 (pointers
 * unused then); tokens may be 0 (nothing to do), and 2^30 at most.  The angle is formed as an
 * exact product in 2^-64 turns and reduced before it is rounded, so far
 * positions lose nothing.  Errors: INVALID_ARG, SHAPE, ALIGN (a pointer not
 * aligned to its elements), CUDA. */
arl2_status arl2_rotary_apply(const arl2_rotary* r, arl2_dtype dtype, int tokens, const int* positions,
                              int q_heads, const void* q, long long q_stride, void* q_out,
                              long long q_out_stride, int k_heads, const void* k, long long k_stride,
                              void* k_out, long long k_out_stride, int inverse, cudaStream_t stream);

/* Release the plan; NULL is ignored. */
void arl2_rotary_destroy(arl2_rotary* r);

/* ------------------------------------------------------------------------
 * Paged KV cache and the attention that reads it.
 *
 * The teacher layer's cache (above) is one dense run of whole frames and all
 * its streams are at the same frame.  Here every sequence (a video stream, a
 * text) has its own length and its keys and values lie in pages of a pool
 * that the caller owns, found through a page table, as they are or quantised
 * to 8 bits.
 *
 * Pool of one layer:
 *   k, v:             [pages][kv_heads][page_tokens][d], dtype or e4m3 codes
 *   k_scale, v_scale: fp32 [pages][kv_heads][page_tokens] (e4m3 only)
 * Key j of sequence s lies in page page_table[s][j / page_tokens], slot
 * j % page_tokens.
 *
 * Quantised rows (one row: the d features of one token and head):
 *   scale = max(max|x| / 448, 2^-126),  code = e4m3(x * (1 / scale))
 * in fp32, codes rounded to nearest even; a row reads back as code * scale.
 * A row that holds an infinity or NaN gets scale NaN and codes 0: it reads
 * back as NaN.  (The NaN codes 0x7f and 0xff are never written; in a pool that
 * the caller filled they must not be in rows that a query sees.)
 *
 * A batch names, for each of its sequences, the chunk of new tokens and the
 * length with them; they are the sequence's last ones.  Row i of sequence s's
 * new = q_offsets[s+1] - q_offsets[s] rows (rows q_offsets[s] on of the token
 * tensors) has the position kv_lens[s] - new + i.  Rows at negative positions
 * (a chunk padded on the left) and rows from q_offsets[seqs] on belong to no
 * token: they are not written to the cache; the former's outputs are zeros,
 * the latter's outputs are left as they were.
 *
 * The query at position p, with c = floor(p / block), sees the keys
 *   j < min(kv_lens[s], (c + 1) block)   and
 *   j >= (c + 1 - window) block  or  j < sinks block   (if window > 0)
 * block = 1 is causal by token; block = tokens per frame is bidirectional
 * within a frame and causal between frames (the teacher layer's mask).
 * window counts blocks, the query's own among them; 0: no window.  sinks
 * counts first blocks that stay visible.  A query that sees nothing gives
 * zeros.  A key that a query does not see has no effect on it, whatever it
 * holds.
 *
 * The lengths, offsets and tables are device memory, read when the kernels
 * run: a captured graph may be replayed with other values in them.  They are
 * checked there, before they are used as an address.  A sequence whose
 * offsets are out of order or past `tokens`, whose length is negative or
 * beyond max_pages pages, or a page number outside the pool sets the
 * handle's error word: the sequence (or the page) is skipped, outputs of
 * the sequence are undefined, and arl2_paged_device_status reports
 * INVALID_ARG.  With offsets out of order, rows that belong to another
 * sequence's range as well may be skipped with it, and what they share is
 * undefined; no row is written to or read from a position other than its own. */
typedef enum { ARL2_CACHE_NATIVE = 0, ARL2_CACHE_E4M3 = 1 } arl2_cache_format;

typedef struct arl2_paged_handle arl2_paged_handle;

typedef struct {
    int q_heads;           /* Hq: a multiple of kv_heads                      */
    int kv_heads;          /* Hk >= 1; Hq / Hk <= 64                          */
    int head_dim;          /* d: 128 for the bf16 tensor-core kernels; 1..128 SIMT */
    int pages;             /* pages of a pool, >= 1                           */
    int page_tokens;       /* 16, 32, 64, 128 or 256                          */
    arl2_dtype dtype;      /* dtype of q, k, v and out                        */
    arl2_cache_format format; /* NATIVE: the pool holds dtype                 */
    float softmax_scale;   /* 0 selects 1/sqrt(d)                             */
    arl2_impl impl;
    int max_ctas;          /* as in arl2_config                               */
} arl2_paged_config;

/* One layer's pages (device memory of the caller, 16-byte aligned).  The
 * same handle may serve the pools of many layers. */
typedef struct {
    void* k;
    void* v;
    float* k_scale;        /* NULL unless the format is E4M3 */
    float* v_scale;
} arl2_paged_pool;

typedef struct {
    int seqs;              /* 0..1024                                         */
    int tokens;            /* rows of the token tensors: 0..2^30              */
    int max_pages;         /* columns of page_table; max_pages * page_tokens
                              <= 2^30                                         */
    int max_new;           /* the largest number of new tokens of a sequence,
                              or 0 if unknown: which kernel runs depends on
                              it, results only within their rounding          */
    const int* q_offsets;  /* device int32 [seqs + 1], ascending              */
    const int* kv_lens;    /* device int32 [seqs]                             */
    const int* page_table; /* device int32 [seqs][max_pages]                  */
} arl2_paged_batch;

/* Create a handle on the current device (workspace and error word; no pool).
 * Errors: INVALID_ARG, SHAPE, UNSUPPORTED (dtype/head_dim), OOM, CUDA. */
arl2_status arl2_paged_create(const arl2_paged_config* cfg, cudaStream_t stream, arl2_paged_handle** out);

/* Write the batch's new keys and values, k and v [tokens][kv_heads][d] dtype
 * (tokens *_stride elements apart, 0 for dense), into their pages, quantised
 * if the format says so.  Two rows of a batch must not share a slot.  Rows
 * that go to the same pages as another sequence's (a shared prefix) are the
 * caller's to keep apart. */
arl2_status arl2_paged_write(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                             const void* k, long long k_stride, const void* v, long long v_stride,
                             cudaStream_t stream);

/* Read keys and values back: rows offsets[s] .. offsets[s+1] - 1 of k_dst and
 * v_dst ([tokens][kv_heads][d] dtype, dense) get sequence s's positions
 * starts[s], starts[s] + 1, ... (starts NULL: from 0).  offsets: device int32
 * [seqs + 1]; starts: device int32 [seqs]; page_table: [seqs][max_pages].
 * Rows from offsets[seqs] on are left as they were. */
arl2_status arl2_paged_read(arl2_paged_handle* h, const arl2_paged_pool* pool, int seqs, int tokens,
                            int max_pages, const int* offsets, const int* starts, const int* page_table,
                            void* k_dst, void* v_dst, cudaStream_t stream);

/* Attention of the batch's new tokens, q [tokens][q_heads][d] (tokens
 * q_stride elements apart, 0 for dense), over their sequences' keys; query
 * head i reads key head i / (Hq / Hk).  out: [tokens][q_heads][d], dense, not
 * overlapping q or the pool.  block >= 1, window >= 0, sinks >= 0 (see
 * above).  Scores, statistics and sums are fp32.  The tensor-core kernels round
 * the softmax weights (times the value's scale, in E4M3) before the product
 * with v: to bf16, or, for at most 16 query rows of a key head and E4M3, to 12
 * bits; with E4M3 they take q to within 2^-17 of its row's largest element.
 * q, k and v may be 0 or of magnitudes from 2^-100 to 2^100, scores (q.k times
 * the scale) up to 2^29; beyond, scores, weights or sums may leave fp32's range.
 * Pages none of whose keys a query of the chunk sees are not looked up (a
 * rolling cache may have given them away).  A value that is not finite reaches
 * the queries that see it, as what it is; if not all queries of a tile see it,
 * the keys at the mask's edges are looked at twice more.  One launch. */
arl2_status arl2_paged_attend(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                              int block, int window, int sinks, const void* q, long long q_stride, void* out,
                              cudaStream_t stream);

/* One softmax layer's step: k and q turned by the plan (rotary NULL: not
 * turned), k and v written to their pages, then the attention of the turned
 * q.  The results, cache and output, are bit for bit those of
 * arl2_rotary_apply, arl2_paged_write and arl2_paged_attend.  turned: device
 * scratch of the caller, [tokens][q_heads + kv_heads][d] dtype, for the
 * turned q and k (unused and may be NULL without rotary).  positions: as in
 * arl2_rotary_apply. */
arl2_status arl2_paged_forward(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                               const arl2_rotary* rotary, const int* positions, int block, int window, int sinks,
                               const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                               long long v_stride, void* turned, void* out, cudaStream_t stream);

/* As arl2_device_status: TIMEOUT if a kernel gave up a bounded wait,
 * INVALID_ARG if a batch's tables were wrong (see above), since the last
 * check. */
arl2_status arl2_paged_device_status(arl2_paged_handle* h, cudaStream_t stream);

/* Device bytes the handle holds. */
size_t arl2_paged_device_bytes(const arl2_paged_handle* h);

/* Kernels this handle has enqueued since creation. */
unsigned long long arl2_paged_kernel_launches(const arl2_paged_handle* h);

/* Release the handle (synchronises the device first); NULL is ignored. */
void arl2_paged_destroy(arl2_paged_handle* h);

/* Static string for a status code. */
const char* arl2_status_string(arl2_status s);

/* ABI version: major * 10000 + minor * 100 + patch. */
int arl2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ARL2_H */
