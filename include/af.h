/*
 * af.h -- C ABI of the B200 affine-autoregressive-flow library (libaf.so).
 *
 * The operations are those of STARFlow-V ("STARFlow-V: End-to-End Video
 * Generative Modeling with Autoregressive Normalizing Flows", CVPR 2026 paper
 * notes, papernotes.org):
 *   - the affine AF block z = (x - mu(x*m)) / sigma(x*m), sigma > 0, m the
 *     self-exclusive causal mask (section "Key design 1: global-local
 *     architecture", affine-flow equation), with log|det dz/dx| = -sum log sigma
 *     (the change of variables behind L_NF, section "Loss / training strategy");
 *   - its inverse by video-aware block-wise Jacobi iteration
 *     x^(k+1) = mu(x^(k)*m) + sigma(x^(k)*m) * z, blocks of B tokens in
 *     sequence, parallel inside a block, finished blocks kept in a KV cache,
 *     warm start from the previous frame's converged x, stop when
 *     ||x^(k+1)-x^(k)||^2 / ||x^(k+1)||^2 < tau (section "Key design 3:
 *     video-aware block-wise Jacobi iteration");
 *   - stacks of T blocks of alternating direction, inverted last to first
 *     (section "Key design 1": T >= 3 alternating blocks).
 *
 * Model inside one AF block (the pages only say "causal Transformer"; the
 * readings taken): the input at sequence position p is x_{p-1} (zero at p=0),
 * i.e. the self-exclusive mask as a one-token shift; h = x_in W_in^T + b_in +
 * P_space[p mod frame_len] + P_time[p div frame_len]; `layers` pre-LN blocks
 * (LayerNorm eps 1e-5, causal multi-head attention j <= i with scale
 * 1/sqrt(d/heads), exact-erf GELU MLP of width mlp_ratio*d); final LayerNorm;
 * head [mu | s] = h W_head^T + b_head with sigma = exp(s).  Direction R2L
 * reverses each sample's token order before the block and restores it after.
 *
 * Conventions for every call below:
 *   - x, z: float32 [batch, L, C] row-major, logdet: float32 [batch],
 *     iters: int32; all are caller-owned DEVICE pointers.  x and z never alias.
 *   - ws: caller-owned device workspace of at least af_workspace_bytes(...)
 *     bytes, 256-byte aligned.  The library allocates nothing per call.
 *   - Every call only enqueues work on `stream` (a cudaStream_t, passed as
 *     void*) and returns.  The returned status covers argument checks and
 *     launch errors; device-side failures (a bounded wait that timed out) are
 *     reported by af_device_error().
 *   - Results are deterministic: the same inputs give the same bits.
 */
#ifndef AF_H_
#define AF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  AF_OK = 0,
  AF_ERR_ARG = 1,        /* a bad argument: nothing was enqueued */
  AF_ERR_CUDA = 2,       /* a CUDA call failed; af_last_error_string() tells which */
  AF_ERR_WORKSPACE = 3,  /* ws is null, misaligned or smaller than af_workspace_bytes() */
  AF_NOT_CONVERGED = 4,  /* from af_last_convergence(): some block hit max_iter */
  AF_ERR_DEVICE = 5      /* from af_device_error(): a kernel gave up a bounded wait */
} af_status;

typedef enum { AF_L2R = 0, AF_R2L = 1 } af_dir;
typedef enum { AF_FP32 = 0, AF_BF16 = 1 } af_dtype;

/* Shape of one AF block.  max_len = frame_len * max_frames bounds L.
 * Every config needs positive sizes, d % heads == 0, C % 8 == 0, d % 4 == 0.
 * AF_BF16 also requires C % 64 == 0, d % 128 == 0, (mlp_ratio * d) % 128 == 0
 * and d / heads in {64, 128} (the tensor-core tile shapes);
 * AF_FP32 requires d / heads in {16, 32, 64, 128}. */
typedef struct {
  int C, d, heads, layers, mlp_ratio;
  int frame_len, max_frames;
  af_dtype dtype;
} af_config;

typedef struct af_model af_model;

/* Number of float32 host tensors af_model_create() expects: 4 + 12*layers + 4,
 * in this order ([out, in] row-major matrices):
 *   W_in [d,C], b_in [d], P_space [frame_len,d], P_time [max_frames,d],
 *   per layer: ln1_g [d], ln1_b [d], W_qkv [3d,d] (q;k;v rows, heads as
 *     consecutive d/heads slices), b_qkv [3d], W_o [d,d], b_o [d],
 *     ln2_g [d], ln2_b [d], W_1 [fd,d], b_1 [fd], W_2 [d,fd], b_2 [d]
 *     (fd = mlp_ratio*d),
 *   lnf_g [d], lnf_b [d], W_head [2C,d] (rows 0..C-1 give mu, C..2C-1 give s),
 *   b_head [2C]. */
int af_num_tensors(const af_config* cfg);

/* Copies the weights to the current CUDA device (rounded to bf16, nearest
 * even, for AF_BF16) and returns an opaque model that owns them.  `tensors`
 * are HOST pointers; the call is synchronous.  AF_ERR_ARG on a bad config. */
af_status af_model_create(const af_config* cfg, const float* const* tensors, int n_tensors,
                          af_model** out);
af_status af_model_destroy(af_model* m);

/* Workspace bytes for a call on `batch` sequences of L tokens whose Jacobi
 * blocks hold at most B tokens (pass B = L for af_forward; B need not divide
 * L).  Includes the KV cache of all layers over L positions.  The same
 * workspace serves every block of a stack made of models with the same
 * config.  0 on bad arguments. */
size_t af_workspace_bytes(const af_model* m, int batch, int L, int B);

/* Forward pass of one AF block: z and logdet (= -sum_{i,c} s_{i,c} per
 * sample) from x.  Requires 1 <= L <= max_len. */
af_status af_forward(const af_model* m, const float* x, int batch, int L, af_dir dir,
                     float* z, float* logdet, void* ws, size_t ws_bytes, void* stream);

/* Block-wise Jacobi inverse of one AF block.  Requires L % B == 0,
 * max_iter >= 1, tau >= 0 and finite.  Block b starts from z_b, or, when
 * warm_start != 0, from the previous frame's converged state ("Key design
 * 3": a new frame is warm-started from the previous frame's converged x):
 * the token at working-order position p starts from the converged x at
 * p - k*frame_len, the same spatial position in the most recent finished
 * frame (smallest k >= 1 landing before the block), and from z where no
 * frame before it has finished.  With B = frame_len this is "block b starts
 * from block b-1's final x".  A sample leaves the iteration of a block at
 * the first update whose residual is < tau (0/0 counts as converged);
 * iters[s * (L/B) + b] counts the updates computed.  All iterations, tests
 * and block changes run on the device: one graph launch per call (after one
 * small kernel that writes the block table into ws), no host round trip per
 * iteration. */
af_status af_inverse_jacobi(const af_model* m, const float* z, int batch, int L, af_dir dir,
                            int B, float tau, int max_iter, int warm_start, float* x,
                            int32_t* iters, void* ws, size_t ws_bytes, void* stream);

/* T blocks applied in order t = 0..T-1 (directions dirs[t]); logdet sums the
 * blocks' logdets.  All models must share one af_config. */
af_status flow_stack_forward(const af_model* const* blocks, const af_dir* dirs, int T,
                             const float* x, int batch, int L, float* z, float* logdet,
                             void* ws, size_t ws_bytes, void* stream);

/* Inverse of flow_stack_forward: Jacobi-inverts t = T-1 .. 0.
 * iters is [T, batch, L/B] (block t's counts at offset t*batch*(L/B)). */
af_status flow_stack_inverse(const af_model* const* blocks, const af_dir* dirs, int T,
                             const float* z, int batch, int L, int B, float tau, int max_iter,
                             int warm_start, float* x, int32_t* iters, void* ws,
                             size_t ws_bytes, void* stream);

/* Block-wise Jacobi inverse with a schedule of block sizes, over a range of
 * blocks (section "Key findings": runtime is U-shaped in the block size, and
 * the method uses a smaller block for the first frame and larger ones after;
 * "A complete example": I2V / V2V generation continues a sequence whose
 * first frames are observed).  block_sizes[0 .. n_blocks-1] (HOST array,
 * each >= 1, summing to L) cut the sequence into consecutive blocks; the
 * call inverts blocks b_begin .. b_end-1 (0 <= b_begin < b_end <= n_blocks)
 * with the rules of af_inverse_jacobi (warm start per frame as described
 * there), writing x and iters[s * n_blocks + b] of those blocks only.
 * ws needs af_workspace_bytes(m, batch, L, largest block).  When
 * b_begin > 0, x must already hold the final values of the blocks before
 * b_begin, and ws the K/V of the positions before block b_begin - 1 -- as
 * left by an earlier call on the same ws that ended at b_begin, or by
 * af_prefix_encode of those positions (the first update of block b_begin
 * recomputes block b_begin - 1's K/V from x).  af_last_convergence counts
 * accumulate over calls and restart with a call whose b_begin is 0. */
af_status af_inverse_jacobi_schedule(const af_model* m, const float* z, int batch, int L, af_dir dir,
                                     const int* block_sizes, int n_blocks, int b_begin, int b_end, float tau,
                                     int max_iter, int warm_start, float* x, int32_t* iters, void* ws,
                                     size_t ws_bytes, void* stream);

/* Flow-encode of observed tokens ("A complete example": I2V / V2V -- the
 * flow's forward pass writes the observed frames into the KV cache, no
 * separate encoder): writes the K/V of working-order positions
 * 0 .. n_tokens-1, computed from x, into the cache of a workspace laid out
 * for (batch, L, B) (size af_workspace_bytes(m, batch, L, B)), ready for
 * af_inverse_jacobi_schedule to continue at the block starting at n_tokens
 * (x must then hold the observed tokens too).  Runs passes of at most 2B
 * positions each; writes nothing but the cache and workspace scratch.
 * Requires 1 <= n_tokens <= L. */
af_status af_prefix_encode(const af_model* m, const float* x, int batch, int L, af_dir dir, int B, int n_tokens,
                           void* ws, size_t ws_bytes, void* stream);

/* Streaming generation past the model's length ("A complete example": a
 * sliding window over the deep flow -- after a chunk of latents is
 * produced, f_D is re-run on the last `overlap` latents to rebuild the KV
 * cache, and the next frames are generated).  z, x: [batch, n_frames *
 * frame_len, C], any n_frames; direction L->R, one frame per Jacobi block.
 * Window w covers `window` frames (<= max_frames) starting at frame
 * s_w = w * (window - overlap) (the last window may be shorter); it runs at
 * the model's positions 0 .. window*frame_len - 1.  Its first `overlap`
 * frames (after the first window) are the previous window's output,
 * flow-encoded into the cache (af_prefix_encode); the rest are generated by
 * block-Jacobi (tau, max_iter, warm_start as in af_inverse_jacobi).
 * iters [batch, n_frames] holds each frame's count from the window that
 * generated it.  ws: af_stream_workspace_bytes(m, batch, window) (the most
 * that a window of up to `window` frames needs, plus staging of its x and z).
 * 0 <= overlap < window. */
size_t af_stream_workspace_bytes(const af_model* m, int batch, int window);
af_status af_inverse_jacobi_stream(const af_model* m, const float* z, int batch, int n_frames, int window, int overlap,
                                   float tau, int max_iter, int warm_start, float* x, int32_t* iters, void* ws,
                                   size_t ws_bytes, void* stream);

/* Bytes of the shallow-side workspace of flow_pipeline_inverse for T shallow
 * blocks (config of `shallow`), `batch` videos, frames of frame_len tokens,
 * up to `group` frames per shallow call (a shorter last group can need more
 * than a full one); 0 on a bad argument. */
size_t flow_pipeline_workspace_bytes(const af_model* shallow, int T, int batch, int frame_len, int group);

/* Pipelined deep -> shallow decoding ("Key design 3": the deep flow
 * f_D runs without pause while the shallow blocks f_S consume its output
 * frame by frame; end-to-end latency is set by the deep block):
 * x = f_S^{-1}(f_D^{-1}(z)) with f_S applied to each frame on its own.
 * f_D^{-1} (`deep`, direction L->R, blocks of B tokens, tau, max_iter_deep,
 * warm_start) runs on stream_deep, one frame's blocks per graph launch.
 * Frames are handed to the shallow side in groups of `group` consecutive
 * frames (the last group may be shorter; 1 <= group <= L / frame_len): when
 * the deep flow has finished a group, an event lets stream_shallow run the
 * T-block stack inverse of the group's frames of every video as one batch of
 * batch * group one-frame samples (blocks shallow[0..T-1], directions
 * shallow_dirs, one Jacobi block per frame, no warm start, tau,
 * max_iter_shallow) while the deep flow moves on.  group 1 hands over every
 * frame at once (the shortest tail after the deep flow ends); larger groups
 * run fewer, larger shallow calls beside it.  z, x: [batch, L, C];
 * frame_len = the deep model's frame_len (the shallow models must accept
 * frames of that length and C); L % frame_len == 0 and frame_len % B == 0.
 * iters_deep [batch, L/B], iters_shallow [T, batch, L/frame_len].  ws_deep:
 * af_workspace_bytes(deep, batch, L, B); ws_shallow:
 * flow_pipeline_workspace_bytes(shallow[0], T, batch, frame_len, group).  The
 * two streams may be the same stream (no overlap).  On return all work is
 * enqueued; stream_deep waits for the last group's shallow work, so
 * synchronising stream_deep covers the whole call.  The result is
 * bit-identical to af_inverse_jacobi followed by flow_stack_inverse of each
 * group's frames as one batch. */
af_status flow_pipeline_inverse(const af_model* deep, const af_model* const* shallow, const af_dir* shallow_dirs, int T,
                                const float* z, int batch, int L, int B, float tau, int max_iter_deep,
                                int max_iter_shallow, int warm_start, int group, float* x, int32_t* iters_deep,
                                int32_t* iters_shallow, void* ws_deep, size_t ws_deep_bytes, void* ws_shallow,
                                size_t ws_shallow_bytes, void* stream_deep, void* stream_shallow);

/* The flow-score-matching denoiser s_phi ("Key design 2": a light causal
 * Transformer trained to regress sigma * grad log p of the flow at the noisy
 * sample, with one frame of look-ahead, s_phi(x_{<=n+1}) ~ (sigma grad log
 * p)_n; it refines the flow's slightly noisy output).  Same af_config and
 * tensor order as af_model_create except the head: W_head [C, d], b_head [C]
 * (plain outputs, no (mu, s) pairs).  Readings (the pages give only "8-layer
 * Transformer, width of the shallow blocks"): the input is x_noisy itself
 * (no shift); h = x W_in^T + b_in + P_space[p mod frame_len] + P_time[p div
 * frame_len]; pre-LN layers as in the AF block, with attention by frames of
 * frame_len tokens -- in the first layer a token of frame n attends every
 * token of frames <= n + 1, in later layers frames <= n -- so frame n's
 * output depends on frames <= n + 1 exactly; final LayerNorm and head give
 * s_phi.  AF_BF16 / AF_FP32 as for the AF block; an AF_BF16 denoiser also
 * needs C % 128 == 0 or C % 192 == 0 (its head has C outputs).  The model
 * can only be used with af_denoise (the flow calls reject it). */
int af_denoiser_num_tensors(const af_config* cfg);
af_status af_denoiser_create(const af_config* cfg, const float* const* tensors, int n_tensors,
                             af_model** out);

/* x = x_noisy + sigma * s_phi(x_noisy) (the Tweedie step with s_phi ~ sigma
 * grad log p), x_noisy and x [batch, L, C], L <= max_len, sigma finite.
 * ws: af_workspace_bytes(m, batch, L, L). */
af_status af_denoise(const af_model* m, const float* x_noisy, int batch, int L, float sigma, float* x, void* ws,
                     size_t ws_bytes, void* stream);

/* af_forward for callers that cannot allocate device memory -- a host that
 * owns the whole GPU memory through its own allocator, or a plugin that is
 * handed only its input and output buffers, and so cannot provide a
 * workspace.  No counterpart in the paper.  Same arguments and
 * results as af_forward minus the workspace: the call runs in a scratch array
 * inside the library, 32 MiB per device, held by every GPU that loads libaf.so
 * until the process exits.  Returns AF_ERR_WORKSPACE (with a message in
 * af_last_error_string) when af_workspace_bytes(m, batch, L, L) exceeds
 * 32 MiB.  The first call on a device looks up the array's address; make it
 * before any stream capture.  Calls share the array: calls whose GPU work
 * overlaps (other streams, other threads) race; serialise them.  Allocates
 * nothing and launches its kernels directly on `stream`. */
af_status af_forward_noalloc(const af_model* m, const float* x, int batch, int L, af_dir dir,
                             float* z, float* logdet, void* stream);

/* ---- Operators of one attention layer ------------------------------------
 *
 * The calls below are the parts of an attention layer with rotary positions
 * and a compressed cache, for callers that run their own layers.  No
 * counterpart in the paper.  They take no model: all pointers are device
 * memory of the current device, `stream` belongs to it, data pointers are
 * 16-byte aligned, and strides are in elements, with every row starting on a
 * 16-byte boundary.  A row's heads are consecutive slices of head_dim
 * elements, so q, k and v may be slices of the rows of one QKV product.  Every
 * call only enqueues work on `stream` and can be captured into a CUDA graph;
 * it allocates nothing and keeps nothing.  Zero rows or sequences are allowed
 * and enqueue nothing. */

/* Rotary positions on three axes (time, height, width) and the norm of each
 * head.  pairs[a] channel pairs turn with axis a, in this order, the rest
 * (head_dim / 2 minus their sum, >= 0) stay as they are; pair j of the n of
 * an axis turns by position * theta^(-j / n).  Pair i is channels (2i, 2i+1)
 * (AF_ROPE_PAIRS) or (i, i + head_dim / 2) (AF_ROPE_HALVES).  head_dim 16, 32,
 * 64, 128 or 256; theta >= 1, eps > 0, both finite. */
typedef enum { AF_ROPE_PAIRS = 0, AF_ROPE_HALVES = 1 } af_rope_layout;
typedef struct {
  double theta;
  int head_dim;
  int pairs[3];
  af_rope_layout layout;
  float eps;
} af_rope;

/* Queries and keys of `rows` tokens: each head's row x becomes
 * y = x * rsqrt(mean(x^2) + eps) * gain (gain float32 [head_dim], shared by the
 * heads; null: y = x), then turns by its token's position pos[3 row ..] (int32
 * [rows, 3], any values).  Squares are summed, the rotation is done in fp32,
 * angles are formed in fp64, and the result is rounded once to `dtype`.  q
 * [rows, heads * head_dim], k [rows, kv_heads * head_dim], the outputs
 * likewise, each with its row stride; kv_heads 0 leaves k out (its pointers
 * may be null), heads 0 leaves q out.  An output may be its input (same
 * pointer and stride); otherwise they must not overlap. */
af_status af_qk_norm_rope(const af_rope* rope, af_dtype dtype, int rows, const void* q, int64_t q_stride, int heads,
                          const void* k, int64_t k_stride, int kv_heads, const float* q_gain, const float* k_gain,
                          const int32_t* pos, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                          void* stream);

/* One layer's key/value cache in 4 bits: `batch` sequences of up to `capacity`
 * (at most 2^30) positions, kv_heads heads of head_dim (64 or 128) channels, in one
 * caller-owned buffer of af_cache_bytes bytes (256-byte aligned; 0 on a bad
 * config).  It needs no initialisation: a position's content is what was last
 * written to it, and positions never written must not be attended or read.
 *
 * Contents, for callers that move or make caches themselves: four parts, each
 * on a 256-byte boundary -- key codes, key parameters, value codes, value
 * parameters --, each laid out [batch][kv_heads][capacity][row].  Channels form
 * groups of 32; a group's parameters are its step s (bf16) and its lowest value
 * lo (bf16), in this order, and channel c stands for lo + n_c * s with n_c in
 * 0..15.  A row's codes are 4 * head_dim / 32 little-endian 32-bit words: word
 * t * (head_dim / 32) + g holds channels 32 g + 8 t + i, i = 0..7, the code of
 * an even i in bits 2i .. 2i+3, of an odd i in bits 14 + 2i .. 17 + 2i. */
typedef struct {
  int batch, kv_heads, head_dim, capacity;
} af_cache_config;
size_t af_cache_bytes(const af_cache_config* cfg);

/* Quantises the bf16 rows k, v [batch, rows, kv_heads * head_dim] as it writes
 * them: row i of sequence b goes to position start[b] + i for i < count[b]
 * (int32 device arrays [batch]; start null: 0, count null: rows; counts are
 * clamped to 0..rows).  Rows that fall outside 0..capacity-1 are dropped.
 * For a group with least value lo and largest hi: s = bf16((hi - lo) / 15),
 * n_c = min(15, round-half-even((x_c - lo) / s)), all 0 where s is 0, with
 * fp32 differences and quotients; |x_c - (lo + n_c s)| <= s / 2, plus at most
 * 2^-8 (hi - lo) at the upper end where s was rounded down.  A token whose k
 * or v row of a head holds a NaN or an infinity (or a group with |lo| + 15 s
 * beyond bf16) reads back as NaN in that head's whole k and v row, and every
 * query of the head that attends it gets NaN; queries that mask it are not
 * touched. */
af_status af_cache_write(const af_cache_config* cfg, void* cache, int rows, const void* k, int64_t k_batch_stride,
                         int64_t k_row_stride, const void* v, int64_t v_batch_stride, int64_t v_row_stride,
                         const int32_t* start, const int32_t* count, void* stream);

/* Reads positions start[b] .. start[b] + count[b] - 1 back into rows 0 .. of
 * k, v [batch, rows, kv_heads * head_dim] of `dtype` (the values lo + n s,
 * rounded once), start, count and dropped rows as for af_cache_write; rows
 * not read are left as they were. */
af_status af_cache_read(const af_cache_config* cfg, const void* cache, int rows, const int32_t* start,
                        const int32_t* count, af_dtype dtype, void* k, void* v, int64_t batch_stride,
                        int64_t row_stride, void* stream);

/* Attention over the cache: for each of `heads` query heads (a multiple of
 * kv_heads; consecutive heads share a key head)
 *   out_i = sum_j p_ij v_j,  p_ij = softmax_j(scale * q_i . k_j)
 * over the positions j that query i attends.  Sequence b has length[b] live
 * positions (clamped to 0..capacity) and n_q[b] queries (null: rows; clamped to
 * 0..rows), which are its last n_q[b] positions when causal != 0: query i
 * attends j <= length[b] - n_q[b] + i; when causal == 0, every live position.
 * A query that attends nothing gives zeros; one that attends keys but has no
 * finite score for any of them (a query row that is not finite) gives NaN.
 * Rows n_q[b] .. rows-1 of a sequence are left as they were.  q, out: bf16
 * [batch, rows, heads * head_dim]; length, n_q: int32 device arrays [batch].
 * 0 < scale <= 2^127.
 * rows * heads / kv_heads is at most 2^20.  Sums, softmax statistics and the
 * output are fp32, rounded once; what enters the products is rounded once more
 * at most: weights and values to bf16, and, by the number of query rows, keys
 * to bf16, or queries to 16 bits of their row's largest value (24 bits where a
 * group of 32 channels would lose more than 2^-13 of its values by that).  out
 * must not overlap q.  ws: af_cache_attention_workspace_bytes(cfg, heads, rows) bytes (the
 * current device decides; fewer rows can need more, since more splits of the
 * keys then share the work), 256-byte aligned, not shared by calls that may
 * overlap; it needs no initialisation and holds nothing between calls. */
size_t af_cache_attention_workspace_bytes(const af_cache_config* cfg, int heads, int rows);
af_status af_cache_attention(const af_cache_config* cfg, const void* cache, int rows, int heads, const void* q,
                             int64_t q_batch_stride, int64_t q_row_stride, const int32_t* length, const int32_t* n_q,
                             int causal, float scale, void* out, int64_t out_batch_stride, int64_t out_row_stride,
                             void* ws, size_t ws_bytes, void* stream);

/* The same in a model's own layers, for every call on the model after it
 * (flows and, for rotary positions, the denoiser).  No counterpart in the
 * paper.
 *
 * af_set_rotary: after a layer's QKV projection the heads of q and k are
 * normed (q_gain, k_gain: HOST float32 [layers, d / heads], rounded to bf16 for
 * AF_BF16; null: no norm) and turned by the token's position: with p the
 * working-order position, (p div frame_len, (p mod frame_len) div width,
 * (p mod frame_len) mod width).  rope->head_dim must be d / heads and width
 * divide frame_len; the learned tables P_space and P_time are added as before
 * (zeros leave them out).  The description and the gains are copied; null rope:
 * as created.  Synchronous, on the model's device.
 *
 * af_set_cache_bits: 4 keeps the KV cache of an AF_BF16 block quantised as
 * af_cache_write does, and attends it as af_cache_attention does (forward,
 * Jacobi inverse and flow-encode alike): per layer 5 bits a value instead of
 * 16, plus one layer's K and V in bf16.  16: as created.  Changes what
 * af_workspace_bytes returns and what a workspace holds, so set it before the
 * first call on a workspace; the blocks of a stack need one setting. */
af_status af_set_rotary(af_model* m, const af_rope* rope, int width, const float* q_gain, const float* k_gain);
af_status af_set_cache_bits(af_model* m, int bits);

/* Failure detection of the calls above, as af_set_wait_limit and
 * af_device_error are a model's: the limit of one pipeline wait of the
 * tensor-core kernel (default 2 s, the whole process), and the error word of
 * the current device (synchronises it; AF_ERR_DEVICE and *code, a bit mask, if
 * a wait gave up, and clears the word). */
af_status af_operator_wait_limit(double seconds);
af_status af_operator_error(int* code);

/* Synchronises `stream` and reports how many (sample, block) pairs of the
 * last inverse call on this workspace (of the calls since the last one that
 * started at block 0, for af_inverse_jacobi_schedule) stopped at max_iter
 * without passing the test: AF_OK if none, AF_NOT_CONVERGED otherwise
 * (*n_unconverged set). */
af_status af_last_convergence(void* ws, int* n_unconverged, void* stream);

/* Failure detection: every wait of the tensor-core kernels' pipelines (on a
 * TMA load, an MMA, a buffer hand-off between warps) is bounded.  A wait that
 * runs past `seconds` (default 2) makes its CTA abort: every role stops, the
 * loads and MMAs already in flight are waited for (each with its own 2 s
 * bound), tensor memory is freed, and the model's error word is set for
 * af_device_error.  The results of that call are then undefined; later calls
 * are unaffected.  Applies to calls enqueued after it (graphs captured with
 * another limit are captured anew).  AF_ERR_ARG unless 0 < seconds <= 60.
 * No counterpart in the paper. */
af_status af_set_wait_limit(af_model* m, double seconds);

/* Synchronises the device and returns AF_ERR_DEVICE (and clears the word)
 * if any kernel of this model gave up a bounded wait; *code is a bit mask of
 * where: 1 a GEMM pipeline wait, 4 an attention pipeline wait, 2 a drain
 * after an abort that did not see its in-flight work complete in time. */
af_status af_device_error(const af_model* m, int* code);

const char* af_status_string(af_status s);
const char* af_last_error_string(void);

#ifdef __cplusplus
}
#endif
#endif /* AF_H_ */
