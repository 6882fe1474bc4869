/*
 * tq.h - TurboQuant-style KV-cache compression and decode attention over the
 * compressed cache, for NVIDIA GB300 (sm_103a).  C ABI of libtq.so.
 *
 * What is computed (sources are cited by page title and section):
 *
 *   Encode, per (token, KV head) vector x of head_dim d
 *   ("TurboQuant+ KV cache compression", Stage 1 and Stage 2 step lists):
 *     n = ||x||, x_hat = x / n;  y = H_d diag(s) x_hat  (seeded random signs s,
 *     orthonormal Walsh-Hadamard H_d);  idx_i = Lloyd-Max index of y_i for the
 *     Gaussian N(0, 1/d) with 2^b levels;  store idx and n.
 *     K formats add the QJL stage: r = y - c[idx], store rnorm = n ||r|| and
 *     sigma_j = [(S r)_j > 0] for an iid N(0, 1) d x d matrix S
 *     ("TurboQuant+ deep dive", section 2.3: sign of the projection).
 *     V formats keep stage 1 only ("TurboQuant+ KV cache compression",
 *     K/V asymmetric strategy).
 *
 *   Decode attention, one query token per sequence:
 *     q_rot = H_d diag(s) q;  Sq = S q_rot;
 *     score_j = scale (n_j <q_rot, c[idx_j]> + rnorm_j sqrt(pi/2)/d <Sq, 2 sigma_j - 1>);
 *     online softmax over the context; V accumulated in the rotated space as
 *     n_j c_V[idx_j], skipping tokens whose weight is below skip_threshold
 *     ("TurboQuant+: 3.8x compression ...", core content item 4, Sparse V);
 *     split-K partials merged by log-sum-exp; out = diag(s) H_d acc / l.
 *
 * Conventions for every function below
 *   - All device pointers are CUDA device (or managed) memory of the device that
 *     was current when the context was created; host pointers are noted "host".
 *   - The caller allocates and owns every buffer: inputs, caches, workspace,
 *     outputs.  The library allocates only the small tables inside a context.
 *   - Device work is enqueued on `stream` (NULL = the legacy default stream) and
 *     is asynchronous; nothing is synchronised unless stated.
 *   - Arguments are validated on the host before any launch; an invalid call
 *     launches nothing and returns TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED /
 *     TQ_ERR_WORKSPACE.  A failed launch returns TQ_ERR_CUDA.  Nothing aborts,
 *     nothing throws across the ABI.
 *   - Values that only the device can see (sequence lengths, block-table
 *     entries, slot ids) are bounds-checked in the kernels: an offending item is
 *     skipped and a bit is set in the context's device status word, read with
 *     tq_get_status().
 */
#ifndef TQ_H_
#define TQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (the runtime's stream handle); NULL is the legacy default stream. */
typedef struct CUstream_st* tq_stream_t;

typedef enum tq_status {
  TQ_OK = 0,
  TQ_ERR_INVALID_ARG = 1,  /* bad pointer, size, format, stride or a device-side bounds flag */
  TQ_ERR_UNSUPPORTED = 2,  /* valid request outside what this build implements (e.g. d = 96) */
  TQ_ERR_WORKSPACE = 3,    /* workspace smaller than tq_decode_workspace_bytes() */
  TQ_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed */
  TQ_ERR_OOM = 5           /* context tables could not be allocated */
} tq_status;

/*
 * Storage formats.  Stage-1 bits and QJL bit per element follow the format
 * table of "TurboQuant+ KV cache compression" (turbo2 = 1+1, turbo3 = 2+1,
 * turbo4 = 3+1); the _MSE variants are the V forms with stage 1 only (turbo4
 * V = 3 bits, same page, K/V asymmetric strategy).  Q8_0 is the pages' int8
 * baseline cache type (absmax / 127 per block of 32, "TurboQuant+ deep dive"
 * section 2.1 with n = 8).  MINMAX is the per-group asymmetric min-max
 * quantiser of "mac-code TurboQuant analysis" section 2.1 (group 64,
 * cache_view.bits = 2, 3 or 4).
 */
typedef enum tq_format {
  TQ_FMT_TURBO2 = 0,
  TQ_FMT_TURBO3 = 1,
  TQ_FMT_TURBO4 = 2,
  TQ_FMT_TURBO2_MSE = 3,
  TQ_FMT_TURBO3_MSE = 4,
  TQ_FMT_TURBO4_MSE = 5,
  TQ_FMT_Q8_0 = 6,
  TQ_FMT_MINMAX = 7,
  TQ_FMT_F8_BLOCK = 8 /* e4m3 with a scale per 16 tokens and head (tq_append_kv, tq_read_kv, tq_chunk_attention) */
} tq_format;

/*
 * Byte layout of one stored vector (one token of one KV head of one layer).
 * Each vector has a payload and a header, kept in two separate arrays.
 *
 *   turbo (K and V): each coordinate i has a w-bit code, w = b (+1 for K):
 *     bits [0, b) = Lloyd-Max index (ascending level order), bit b = QJL sign
 *     (K only, 1 = positive projection).  Codes are packed little-endian,
 *     coordinate i at bit offset w*i of the payload; so every group of 32
 *     coordinates ("block-32") fills exactly w 32-bit words.
 *     payload = d*w/8 bytes.  header: K = {fp16 n, fp16 rnorm}, V = {fp16 n}.
 *   q8_0: payload = d int8 values; header = d/32 fp16 scales (block order).
 *   minmax: codes of `bits` bits packed as for turbo; header = d/64 pairs
 *     {fp16 scale, fp16 zero} (group order).
 *   f8_block: payload = d e4m3 codes (1 sign, 4 exponent, 3 mantissa bits, largest value 448); the header belongs to a
 *     block of 16 vectors, the tokens [16 k, 16 k + 16) of a page (page_size is a multiple of 16): one 32-bit word
 *     2^e as fp32, -80 <= e <= 80, whose low 16 bits mark tokens: bit i of a marked token i, every coordinate of which
 *     reads back as NaN.  A value is code * 2^e.  The codes 0x7F and 0xFF (NaN) are never written; where a cache that
 *     was filled in another way holds them, what is read from it is not specified.
 *
 * Cache view: a 4-D array of vectors [n_layers][num_pages][n_kv_heads][page_size].
 * The vector at (layer, page, head, p) has index
 *     v = ((layer * num_pages + page) * n_kv_heads + head) * page_size + p
 * and lives at payload + v * tq_payload_bytes(), header + v * tq_header_bytes() (f8_block: header + v / 16 * 4, the
 * word of its block).
 * Token slot t of a layer means page = t / page_size, p = t % page_size, so a
 * contiguous cache of capacity C per sequence is the view with page_size = C
 * and page = sequence index (block_table = NULL in tq_decode_attention).
 */
typedef struct tq_cache_view {
  int32_t format;      /* tq_format */
  int32_t head_dim;    /* d: 64, 128 or 256 */
  int32_t n_kv_heads;  /* H >= 1 */
  int32_t page_size;   /* tokens per page >= 1 */
  int64_t num_pages;   /* pages per layer >= 1 */
  int32_t n_layers;    /* layers held by this view >= 1 */
  int32_t bits;        /* TQ_FMT_MINMAX only: 2, 3 or 4; ignored otherwise */
  void* payload;       /* device, 16-byte aligned */
  void* header;        /* device, 4-byte aligned */
} tq_cache_view;

typedef struct tq_context tq_context;

/* ---- sizes and names (host, pure functions) ---- */

const char* tq_status_string(tq_status s);
const char* tq_format_name(tq_format f);
/* Payload / header bytes of one vector; 0 for an invalid (format, head_dim, bits).  An f8_block vector has no header of
 * its own: tq_header_bytes() is 0 for it. */
size_t tq_payload_bytes(tq_format f, int head_dim, int bits);
size_t tq_header_bytes(tq_format f, int head_dim, int bits);
/* Bytes of a view's whole header array (the pointers are not looked at); 0 for an invalid view. */
size_t tq_view_header_bytes(const tq_cache_view* view);
/* payload + header, the compressed bytes of one vector. */
size_t tq_vector_bytes(tq_format f, int head_dim, int bits);

/* ---- host math ---- */

/*
 * Lloyd-Max quantiser for N(0, 1/head_dim) with 2^bits levels, bits in 1..4
 * ("TurboQuant+ KV cache compression", Stage 1 step 3: optimal codebook for the
 * Gaussian precomputed with Lloyd's algorithm).  Iterated in double precision:
 * boundaries = midpoints, centroids = conditional means of their cells, until no
 * centroid moves by more than 1e-13 sigma.  Writes (host) centroids[2^bits] and
 * boundaries[2^bits - 1], ascending, rounded to float (boundaries are the
 * double midpoints rounded once).  head_dim >= 1.
 */
tq_status tq_codebook_build(int bits, int head_dim, float* centroids, float* boundaries);

/*
 * Default random tables, counter based (SplitMix64 of Steele, Lea and Flood,
 * evaluated at counter (seed << 32) + k).  seed < 2^32.
 *   signs[i] = -1 if the top bit of SplitMix64(c_i) is set else +1   (host int8 [d])
 *   S[j*d + i] = sqrt(-2 ln u1) cos(2 pi u2), u = ((SplitMix64(c) >> 11) + 1) 2^-53
 *                at counters 2(j*d+i), 2(j*d+i)+1, computed in double, rounded
 *                to float                                           (host float [d*d])
 */
tq_status tq_signs_generate(uint32_t seed, int head_dim, int8_t* signs);
tq_status tq_qjl_matrix_generate(uint32_t seed, int head_dim, float* S);

/* ---- context: the per-head_dim tables on the current device ---- */

/*
 * Creates a context for one head_dim (64, 128 or 256) on the current device:
 * the sign diagonal, the QJL matrix S (row j = projection j) and the turbo
 * codebooks for 1, 2 and 3 bits.  `signs` (host int8 [d], +-1) and `qjl` (host
 * float [d*d]) may be NULL, in which case the default generators are used with
 * wht_seed / qjl_seed; when given they are copied.  Synchronous.  The context
 * is immutable afterwards (except its status word) and may be used from any
 * stream of that device.  Returns TQ_ERR_UNSUPPORTED for other head_dim.
 */
tq_status tq_context_create(int head_dim, uint32_t wht_seed, uint32_t qjl_seed,
                            const int8_t* signs, const float* qjl, tq_context** out);
tq_status tq_context_destroy(tq_context* ctx);

/*
 * Copies the context's tables to host memory (any pointer may be NULL):
 * signs int8 [d]; qjl float [d*d]; centroids float [3][8] and boundaries
 * float [3][7] for bits 1, 2, 3 (unused entries zero).  Synchronous.
 */
tq_status tq_context_get_tables(const tq_context* ctx, int8_t* signs, float* qjl,
                                float* centroids, float* boundaries);

/*
 * Reads and clears the context's device status word (synchronises the device).
 * *flags (host, may be NULL) receives the bits: 1 = a sequence length above
 * max_ctx or the view's capacity was clamped, 2 = a block-table entry out of
 * [0, num_pages) was skipped, 4 = a slot id out of range was skipped, 8 = a
 * bounded wait for the tensor cores ran out (the results of that call are not
 * valid).  Returns TQ_ERR_INVALID_ARG if any bit was set, else TQ_OK.
 */
tq_status tq_get_status(tq_context* ctx, uint32_t* flags);

/* ---- encode ---- */

/*
 * Compresses fp16 K and/or V vectors into cache views (either pair may be NULL,
 * not both).  Input element (l, t, h, i) of K is
 *     k[l * in_layer_stride + t * in_token_stride + h * d + i]
 * for l < n_layers, t < n_tokens, h < n_kv_heads of the view, i < d (same for V);
 * strides are in elements and heads are contiguous d-vectors.  k and v must be
 * 16-byte aligned and both strides multiples of 8 elements (the inputs are read
 * with 16-byte loads), else TQ_ERR_INVALID_ARG.  Layer l of the
 * input goes to layer layer_begin + l of the view.  Token t goes to slot
 * slots[t] (device int64 [n_tokens]) when `slots` is non-NULL, else to slot
 * slot_begin + t; a slot outside [0, num_pages * page_size) is skipped and
 * flagged.  K views take any format except the _MSE ones; V views take any
 * format; both views must share head_dim and n_kv_heads with the context's d.
 * Turbo K: stage 1 + QJL; turbo _MSE: stage 1; Q8_0; MINMAX.  F8_BLOCK:
 * TQ_ERR_UNSUPPORTED (its blocks are filled in the order of a sequence:
 * tq_append_kv).
 */
tq_status tq_encode_kv(const tq_context* ctx,
                       const tq_cache_view* k_view, const void* k,
                       const tq_cache_view* v_view, const void* v,
                       int layer_begin, int n_layers, int n_tokens,
                       int64_t in_layer_stride, int64_t in_token_stride,
                       const int64_t* slots, int64_t slot_begin,
                       tq_stream_t stream);

/* ---- decode attention ---- */

/*
 * Bytes of workspace tq_decode_attention needs for these sizes (split-K
 * partials plus the rotated queries).  Depends only on its arguments and on the
 * context's device.
 */
size_t tq_decode_workspace_bytes(const tq_context* ctx, int n_layers, int batch,
                                 int n_q_heads, int max_ctx);

/*
 * One decode step of attention for `batch` sequences over n_layers layers.
 *   q:   device [n_layers][batch][n_q_heads][d], fp32 (q_is_fp16 = 0) or fp16 (1).
 *   out: device float [n_layers][batch][n_q_heads][d].
 *   Layer l reads layer layer_begin + l of k_view and v_view.
 *   Query head h reads KV head h / (n_q_heads / n_kv_heads); n_q_heads must be
 *   a multiple of n_kv_heads.
 *   seq_lens: device int32 [batch]; sequence b attends to its tokens [0, seq_lens[b]).
 *   max_ctx: host upper bound on every seq_lens[b] (sizes the split-K grid).
 *   block_table: device int32 [batch][max_blocks_per_seq] mapping logical page
 *     t / page_size of sequence b to a physical page, or NULL for page = b.
 *   softmax_scale: the logit scale (1/sqrt(d) in the usual model).
 *   skip_threshold: V terms whose weight exp(s - running max) is below it are
 *     not accumulated (Sparse V); 0 keeps every term.  The softmax denominator
 *     keeps every token.
 *   workspace: device scratch of tq_decode_workspace_bytes() bytes, 256-byte
 *     aligned; its contents are undefined after the call (the combine drops the
 *     split partials from L2 without writing them back).
 *   K formats: turbo (with or without QJL) or Q8_0.  V formats: turbo _MSE or
 *   Q8_0.  A sequence of length 0 yields zeros.
 *   The call is three kernels on `stream`: the query prologue, the split-K
 *   attention (launched as a programmatic dependent of the prologue) and the
 *   combine (a dependent of the attention); work queued after it on the stream
 *   sees the finished result, as after any kernel.
 */
tq_status tq_decode_attention(const tq_context* ctx,
                              const void* q, int q_is_fp16,
                              int n_layers, int batch, int n_q_heads,
                              const tq_cache_view* k_view, const tq_cache_view* v_view,
                              int layer_begin,
                              const int32_t* seq_lens, int max_ctx,
                              const int32_t* block_table, int max_blocks_per_seq,
                              float softmax_scale, float skip_threshold,
                              void* workspace, size_t workspace_bytes,
                              float* out, tq_stream_t stream);

/*
 * tq_decode_attention without a caller workspace, for callers that cannot
 * allocate device memory when they run decode attention (a process whose
 * device memory is all reserved by its own pool, code inside an allocator
 * callback, a plug-in that only receives its inputs and outputs).  The paper
 * has no counterpart: this is a deployment variant of the same computation.
 *
 * Same arguments and result as tq_decode_attention minus the workspace pair.
 * The workspace is a fixed 16 MiB array inside libtq.so (every GPU that loads
 * the library keeps it until exit); a call whose tq_decode_workspace_bytes()
 * exceeds 16 MiB returns TQ_ERR_WORKSPACE and launches nothing.  The first call
 * on a device looks the array's device address up (with that device current)
 * and should come before any stream capture; the address is kept for the life
 * of the process, so the entry point must not be used on a device after
 * cudaDeviceReset (the library's module, and the array with it, is gone).  All
 * calls share the array: calls that overlap on the GPU race.  The context's
 * device must be current.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 */
tq_status tq_decode_attention_static(const tq_context* ctx,
                                     const void* q, int q_is_fp16,
                                     int n_layers, int batch, int n_q_heads,
                                     const tq_cache_view* k_view, const tq_cache_view* v_view,
                                     int layer_begin,
                                     const int32_t* seq_lens, int max_ctx,
                                     const int32_t* block_table, int max_blocks_per_seq,
                                     float softmax_scale, float skip_threshold,
                                     float* out, tq_stream_t stream);

/* ---- per-layer views: a K and a V format per layer ---- */

/*
 * Layer policies that give some layers another format, as in Boundary V ("TurboQuant+: 3.8x
 * compression ...", core content item 3: q8_0 V on the first 2 and last 2 layers, turbo2 V
 * elsewhere; "TurboQuant+ deep dive", section 3.2, layer-wise V strategy), or asymmetric K/V
 * pairs per layer (same page's item 2; deep dive section 3.1), are expressed with one view per
 * layer: layer l is stored at layer k_view_layers[l] of k_views[l] (host arrays [n_layers]) and
 * at layer v_view_layers[l] of v_views[l].  Views may repeat (a view holding several layers).
 * Every layer's views must share head_dim (the context's) and n_kv_heads; the K and V views of a
 * layer must share page_size and num_pages.
 */

/*
 * tq_encode_kv over per-layer views: input layer l (at k + l * in_layer_stride elements, same for
 * v) is encoded into layer k_view_layers[l] of k_views[l] (and v_*).  k_views (with k_view_layers
 * and k) or v_views (with v_view_layers and v) may be NULL, not both.  Every layer is validated
 * before anything is launched; then runs of consecutive layers that share their views at
 * consecutive view layers are encoded by one call of tq_encode_kv each.  Errors as tq_encode_kv.
 */
tq_status tq_encode_kv_layers(const tq_context* ctx,
                              const tq_cache_view* k_views, const int32_t* k_view_layers,
                              const tq_cache_view* v_views, const int32_t* v_view_layers, int n_layers,
                              const void* k, const void* v, int n_tokens,
                              int64_t in_layer_stride, int64_t in_token_stride,
                              const int64_t* slots, int64_t slot_begin, tq_stream_t stream);

/*
 * tq_decode_attention over per-layer views, in one call: q, out, seq_lens, block_table, the scale,
 * the skip threshold and the workspace as for tq_decode_attention (layer l of q and out is query
 * layer l), the workspace sized by tq_decode_workspace_bytes(ctx, n_layers, batch, n_q_heads,
 * max_ctx).  Every layer is validated before anything is launched (TQ_ERR_INVALID_ARG /
 * TQ_ERR_UNSUPPORTED / TQ_ERR_WORKSPACE as for tq_decode_attention; more than 65535 layers or
 * view layers: TQ_ERR_UNSUPPORTED); then the layers are grouped by their (K view, V view) pair,
 * wherever they sit, and each group (128 layers at most per launch) runs the decode kernels once,
 * with the split plan tq_decode_attention would take for that group alone when it fits in the
 * workspace, else the whole call's.  The result then equals tq_decode_attention run on each group.
 */
tq_status tq_decode_attention_layers(const tq_context* ctx, const void* q, int q_is_fp16,
                                     int n_layers, int batch, int n_q_heads,
                                     const tq_cache_view* k_views, const int32_t* k_view_layers,
                                     const tq_cache_view* v_views, const int32_t* v_view_layers,
                                     const int32_t* seq_lens, int max_ctx,
                                     const int32_t* block_table, int max_blocks_per_seq,
                                     float softmax_scale, float skip_threshold,
                                     void* workspace, size_t workspace_bytes,
                                     float* out, tq_stream_t stream);

/* ---- chunked-prefill attention ---- */

/* Bytes of workspace tq_prefill_attention needs (the prepared queries). */
size_t tq_prefill_workspace_bytes(const tq_context* ctx, int n_tokens, int n_q_heads);

/*
 * Attention of a prefill chunk over the compressed cache ("TurboQuant+: 3.8x compression ...",
 * core content item 1: prefill reads the quantised cache).  The chunk's n_tokens tokens sit at
 * positions start .. start + n_tokens - 1 of one sequence and are already encoded into the cache
 * (tq_encode_kv); chunk token i attends to the cached tokens 0 .. start + i (causal, its own
 * token included), with the same compressed-domain scores as tq_decode_attention (q rotated once,
 * n_j <q', c[idx_j]> + rnorm_j sqrt(pi/2)/d <S q', sign_j>) and no Sparse V.
 *   q:   device [n_tokens][n_q_heads][d], fp32 (q_is_fp16 = 0) or fp16 (1).
 *   out: device float [n_tokens][n_q_heads][d].
 *   Query head h reads KV head h / (n_q_heads / n_kv_heads).
 *   The sequence: layer `layer` of k_view and v_view; block_table (device int32 [max_blocks],
 *   logical page -> physical page) or NULL for page `seq` of a contiguous cache.
 *   workspace: device, tq_prefill_workspace_bytes() bytes, 256-byte aligned.
 * This build: head_dim 128, K turbo2/3/4 (with the QJL stage), V turbo2/3/4_mse; other formats or
 * head_dims return TQ_ERR_UNSUPPORTED.  The products run on the fifth-generation tensor cores.
 * A block-table entry out of range sets status bit 2, and its keys are left out.
 */
tq_status tq_prefill_attention(const tq_context* ctx, const void* q, int q_is_fp16, int n_tokens, int n_q_heads,
                               const tq_cache_view* k_view, const tq_cache_view* v_view, int layer, int seq,
                               const int32_t* block_table, int max_blocks, int start, float softmax_scale,
                               void* workspace, size_t workspace_bytes, float* out, tq_stream_t stream);

/* ---- one serving step over the compressed cache: rotate, append, attend a ragged batch ---- */

/* Element type of the activations that the calls below read and write. */
typedef enum tq_dtype { TQ_DTYPE_F32 = 0, TQ_DTYPE_F16 = 1, TQ_DTYPE_BF16 = 2 } tq_dtype;

/* Rotary positions: which coordinates form a pair. */
typedef enum tq_rope_layout {
  TQ_ROPE_HALF = 0,        /* pair i = coordinates (i, i + rotary_dim / 2) */
  TQ_ROPE_INTERLEAVED = 1  /* pair i = coordinates (2 i, 2 i + 1) */
} tq_rope_layout;

/* How the angles f_i = base^(-2 i / rotary_dim) per position are changed for contexts `factor` times longer. */
typedef enum tq_rope_scaling {
  TQ_ROPE_NONE = 0,
  TQ_ROPE_LINEAR = 1,      /* f_i / factor */
  TQ_ROPE_NTK = 2,         /* base * factor^(r / (r - 2)) in place of base, r = rotary_dim > 2 */
  TQ_ROPE_WAVELENGTH = 3,  /* s f_i + (1 - s) f_i / factor,
                              s = clamp((original_ctx f_i / 2 pi - low) / (high - low), 0, 1):
                              pairs that turn more than `high` times within original_ctx keep their angle, pairs
                              that turn less than `low` times are stretched (defaults low 1, high 4) */
  TQ_ROPE_YARN = 4         /* g_i f_i / factor + (1 - g_i) f_i, g_i = clamp((i - a) / max(b - a, 0.001), 0, 1),
                              a = max(floor(dim(high)), 0), b = min(ceil(dim(low)), r - 1),
                              dim(t) = r ln(original_ctx / (2 pi t)) / (2 ln base) (defaults low 1, high 32);
                              the rotated coordinates are multiplied by 0.1 ln factor + 1 */
} tq_rope_scaling;

typedef struct tq_rope_params {
  int32_t head_dim;     /* 64, 128 or 256 */
  int32_t rotary_dim;   /* even, 2 .. head_dim: coordinates [rotary_dim, head_dim) are not rotated */
  int32_t layout;       /* tq_rope_layout */
  int32_t scaling;      /* tq_rope_scaling */
  double base;          /* > 1 */
  double factor;        /* > 0 (ignored by TQ_ROPE_NONE) */
  double original_ctx;  /* > 0 (TQ_ROPE_WAVELENGTH, TQ_ROPE_YARN) */
  double low, high;     /* 0: the scaling's default; low < high */
  double attn_factor;   /* factor on the rotated coordinates; 0: the scaling's default (1; see TQ_ROPE_YARN) */
} tq_rope_params;

/*
 * The rotation in the form the kernels take: turns[i] is pair i's angle per position as a fraction of a turn in
 * units of 2^-64.  position * turns[i] modulo 2^64 is the angle at any position, negative ones included, without
 * the loss that a product in fp32 has at far positions.  Filled by tq_rope_build, passed by value to the kernels
 * (no device memory); the caller owns it and may change it after a call returns.
 */
typedef struct tq_rope_table {
  int32_t head_dim, rotary_dim, layout;
  float attn_factor;
  uint64_t turns[128];
} tq_rope_table;

/* Host; TQ_ERR_INVALID_ARG for values outside those noted above and where an angle leaves the range of double (a factor
 * of 1e-320, say), TQ_ERR_UNSUPPORTED for another head_dim. */
tq_status tq_rope_build(const tq_rope_params* params, tq_rope_table* table);

/*
 * Rotates n_tokens x n_heads vectors: element (t, h, i) is x[t * x_token_stride + h * d + i], the result goes to
 * out[t * out_token_stride + h * d + i] in the same type (strides in elements, >= n_heads * d).  Token t turns by
 * positions[t] (device int32 [n_tokens]) times the table's angles, in the other direction with inverse = 1, which is
 * the gradient of the rotation (its transpose, attn_factor included).  Computed in fp32, rounded once.  out may be x
 * with the same stride (in place); other overlaps are not allowed.  x and out 16-byte aligned, strides multiples of
 * 16 bytes, else TQ_ERR_INVALID_ARG; without tokens (n_tokens = 0, here and in the calls below) the arrays of rows and
 * positions may be NULL.  The context's device must be current (TQ_ERR_INVALID_ARG otherwise, here and in the calls
 * below); the table's head_dim must be the context's.
 */
tq_status tq_rope(const tq_context* ctx, const tq_rope_table* table, const void* x, tq_dtype dtype, int n_tokens,
                  int n_heads, int64_t x_token_stride, const int32_t* positions, int inverse, void* out,
                  int64_t out_token_stride, tq_stream_t stream);

/*
 * Norms of queries and keys per head, and the rotation, in the same pass.  Of each vector x (token t, head h), in fp32:
 *   r = 1 / sqrt(sum_i x_i^2 / d + eps),  y_i = r x_i weight[i],  out = y rotated as by tq_rope
 * over all d coordinates, the ones that are not rotated among them.  q and k describe the rows of the queries and of the
 * keys: either may be NULL (not both), each has its own weight (device [d] of type weight_dtype, any alignment of an
 * element; NULL: ones), heads and strides; x and out are as in tq_rope (out may be x with the same stride; other overlaps
 * are not allowed, nor between the two).  eps > 0, 2^-126 at least.  A vector whose squares pass the range of fp32 is
 * normed all the same; one with a NaN gives NaN in every coordinate, one with an infinity NaN in that coordinate and the
 * one rotated with it and 0 in the others.  Errors as tq_rope.
 */
typedef struct tq_norm_rows {
  const void* x;             /* element (t, h, i) at t * x_token_stride + h * d + i */
  int64_t x_token_stride;    /* elements, >= n_heads * d, a multiple of 16 bytes */
  void* out;
  int64_t out_token_stride;
  const void* weight;
  int32_t n_heads;           /* >= 1 */
} tq_norm_rows;

tq_status tq_norm_rope(const tq_context* ctx, const tq_rope_table* table, const tq_norm_rows* q, const tq_norm_rows* k,
                       tq_dtype dtype, tq_dtype weight_dtype, float eps, int n_tokens, const int32_t* positions,
                       tq_stream_t stream);

/*
 * The gradient of tq_norm_rope.  With g = dout rotated back (its transpose, attn_factor included) and x' = r x:
 *   dx_i = r (g_i weight[i] - x'_i sum_j(g_j weight[j] x'_j) / d),  dweight[i] = sum over tokens and heads of g_i x'_i.
 * x, dout and dx are of type dtype (dx may be dout with the same stride); dweight is device float [d], 4-byte aligned,
 * written and not added to, NULL where it is not wanted.  Sums are fp32 (the last ones, over partial results, with what
 * each addition loses), in an order that depends on the sizes alone.  workspace: device,
 * tq_norm_rope_grad_workspace_bytes() bytes, 256-byte aligned (TQ_ERR_WORKSPACE); calls that may overlap need their own.
 * n_heads: the heads of q and k together.
 */
typedef struct tq_norm_grad_rows {
  const void* x;
  int64_t x_token_stride;
  const void* dout;
  int64_t dout_token_stride;
  const void* weight;
  void* dx;
  int64_t dx_token_stride;
  float* dweight;
  int32_t n_heads;
} tq_norm_grad_rows;

size_t tq_norm_rope_grad_workspace_bytes(const tq_context* ctx, int n_tokens, int n_heads);
tq_status tq_norm_rope_grad(const tq_context* ctx, const tq_rope_table* table, const tq_norm_grad_rows* q,
                            const tq_norm_grad_rows* k, tq_dtype dtype, tq_dtype weight_dtype, float eps, int n_tokens,
                            const int32_t* positions, void* workspace, size_t workspace_bytes, tq_stream_t stream);

/*
 * A ragged batch of new tokens.  Sequence b has the tokens [cu_tokens[b], cu_tokens[b + 1]) of the call's n_tokens
 * rows (device int32 [n_seqs + 1], from 0 on, not decreasing; rows behind cu_tokens[n_seqs] are padding: what they
 * hold has no effect, and in every output they are left as they are) and seq_lens[b] tokens in all (device int32
 * [n_seqs]), the new ones included: its new token i of n sits at position seq_lens[b] - n + i.  block_table (device
 * int32 [n_seqs][max_blocks]) maps page position / page_size of a sequence to a physical page; NULL: sequence b is
 * page b.
 * max_tokens and max_ctx (host) bound the new tokens and the length of every sequence.  A sequence whose device values
 * break these bounds (more new tokens than max_tokens or than its length, a length above max_ctx, rows outside
 * [0, n_tokens)) is left out of the call: status bit 1 is set, its outputs are zeros (attention, read) or not written
 * (append).
 */
typedef struct tq_batch {
  int32_t n_seqs;      /* >= 0 */
  int32_t n_tokens;    /* rows of q, k, v and the outputs, >= 0 */
  int32_t max_tokens;  /* >= 0 */
  int32_t max_ctx;     /* >= 0, at most max_blocks * page_size, or page_size without a block table */
  int32_t max_blocks;
  const int32_t* cu_tokens;
  const int32_t* seq_lens;
  const int32_t* block_table;
} tq_batch;

/*
 * Appends the batch's new keys and values to layer `layer` of the views, keys rotated on the way when `rope` is not
 * NULL (to positions[t], device int32 [n_tokens], or where positions is NULL to the token's position in its sequence).
 * k / v element (t, h, i): k[t * k_token_stride + h * d + i], same type for both, 16-byte aligned, strides multiples
 * of 16 bytes and >= H d.  The rotated key is quantised from fp32 without a rounding in between.  K: Q8_0.  V: Q8_0
 * or turbo2/3/4_mse; or F8_BLOCK for both.  Others return TQ_ERR_UNSUPPORTED (turbo K: tq_rope, then tq_encode_kv).
 * Values in fp16 without a rotation give the bytes of tq_encode_kv for Q8_0.  A NaN element of a Q8_0 vector is stored as 0; an
 * infinite one, or one so large that the fp16 scale overflows (a magnitude of 127 * 65520 or more), gives an infinite
 * scale and codes of 0, which read back as NaN in its block of 32.  A turbo vector with a NaN or an infinite element,
 * or whose norm passes fp16 (65520), reads back as NaN in every coordinate (tq_read_kv, tq_chunk_attention).  A token
 * whose page is out of range is skipped and sets status bit 2.  Two tokens of one call must not share a slot.
 *
 * F8_BLOCK: the positions [16 k, 16 k + 16) of a sequence are a block, with a scale for each head.  Of the new vectors
 * (keys rotated) that go to it, those with a NaN, an infinity or a magnitude above 448 * 2^80 are marked, with codes of
 * 0.  e is the smallest integer with max |x| <= 448 * 2^e over the others, -80 at least, and at least the block's e
 * so far where the block holds earlier tokens of the sequence (positions before the new ones); where that raises e, the
 * earlier tokens' codes become the e4m3 values nearest to code * 2^(e_before - e), which is exact unless the value falls
 * below 2^-6 * 2^e.  A new code is the e4m3 value nearest to x / 2^e (a tie goes to the even one).  So the stored values
 * depend on what was appended in which calls, not on timing; a block that two sequences share must be full, or not
 * be appended to.
 */
tq_status tq_append_kv(const tq_context* ctx, const tq_batch* batch, const void* k, int64_t k_token_stride,
                       const void* v, int64_t v_token_stride, tq_dtype dtype, const tq_rope_table* rope,
                       const int32_t* positions, const tq_cache_view* k_view, const tq_cache_view* v_view, int layer,
                       tq_stream_t stream);

/*
 * Reads the batch's rows back from layer `layer`: k_out and v_out [n_tokens][H][d] of type dtype, contiguous, 16-byte
 * aligned, in the original space (K as stored, its rotation kept).  Either pair may be NULL, not both.  With
 * cu_tokens covering whole sequences this gathers them.  Formats: Q8_0, turbo2/3/4_mse and F8_BLOCK; others
 * TQ_ERR_UNSUPPORTED.
 * Tokens whose page is out of range give zeros and status bit 2.
 */
tq_status tq_read_kv(const tq_context* ctx, const tq_batch* batch, const tq_cache_view* k_view, void* k_out,
                     const tq_cache_view* v_view, void* v_out, tq_dtype dtype, int layer, tq_stream_t stream);

/* Changes to the scores of tq_chunk_attention; zeros and NULLs: none. */
typedef struct tq_score_mods {
  float softcap;               /* c > 0: s = c tanh(s / c), before the distance bias; any finite c */
  int32_t window;              /* w > 0: the token at position p sees no key j <= p - w */
  const float* slopes;         /* device float [n_q_heads]: s -= slopes[h] |p - j| */
  const int32_t* first_keys;   /* device int32 [n_tokens]: token t sees no key j < first_keys[t] (packed documents) */
  const int32_t* prefix_lens;  /* device int32 [n_seqs]: the keys j < prefix_lens[b] of sequence b are seen by all its
                                  tokens, before or after them (the window and first_keys still apply) */
} tq_score_mods;

/*
 * Workspace of tq_chunk_attention for a batch of these host sizes (the device pointers are not looked at); 0 for
 * invalid arguments.
 */
size_t tq_chunk_workspace_bytes(const tq_context* ctx, const tq_batch* batch, int n_q_heads, int n_kv_heads);

/*
 * The workspace with which tq_chunk_attention runs these views and modifications (may be NULL) fastest; never less
 * than tq_chunk_workspace_bytes(), with which every call runs.  0 for invalid arguments.  What it has more are keys
 * and values as fp16 operands: 4 bytes for each coordinate of a key and its value, of n_seqs sequences of max_ctx
 * (rounded up to 128) tokens each, 8 GiB at most (beyond, it is the least one).  (Where most runs of 128 keys hold
 * f8_block scales more than 2^8 apart, the least workspace is the faster one: 2.1 and 3.2 ms for 4096 tokens at 32K.)
 * The size given to a call chooses the kernel, so its results agree with those of another size to rounding, not bit
 * by bit.
 */
size_t tq_chunk_workspace_for(const tq_context* ctx, const tq_batch* batch, int n_q_heads, const tq_cache_view* k_view,
                              const tq_cache_view* v_view, const tq_score_mods* mods);

/*
 * Attention of a ragged batch of chunks, one token to thousands per sequence, over the paged cache, whose new tokens
 * are already in it (tq_append_kv).  A decode step over Q8_0 K can take this call or tq_decode_attention.  This one:
 * one layer a call, as a model runs them (one token at 32K, 8 KV heads of 128, 4 query heads each: 27 us, 37 there;
 * 64 sequences of 1K to 16K: 145 us, 228 there; turbo4 V 32 and 35, 196 and 207), 16-bit outputs, the score
 * modifications below. tq_decode_attention: turbo K, Sparse V, or many layers' queries at hand at once (17 and 199 us
 * a layer).
 * The token at position p of a sequence of length n sees the keys j < n with j <= p or j < its prefix length, as the
 * score modifications leave them;
 *   s_j = softmax_scale <q, k_j> (capped, then biased), out = sum_j softmax(s)_j v_j;
 * a row that sees no key gives zeros.  A row that sees a key whose stored K or V has an infinite or NaN scale or norm
 * is NaN in all coordinates; a key that a row does not see never reaches it, whatever is stored there.
 *   q: element (t, h, i) at q[t * q_token_stride + h * d + i], type q_dtype, 16-byte aligned, stride a multiple of 16
 *   bytes and >= n_q_heads d.  out: [n_tokens][n_q_heads][d] of type out_dtype, contiguous, 16-byte aligned, apart
 *   from q.
 *   Query head h reads KV head h / (n_q_heads / n_kv_heads); n_q_heads a multiple of n_kv_heads.
 *   K: Q8_0 with V: Q8_0 or turbo2/3/4_mse; or F8_BLOCK for both.  Others: TQ_ERR_UNSUPPORTED (turbo K:
 *   tq_decode_attention, tq_prefill_attention).  F8_BLOCK codes are fp16 numbers: keys and values are not rounded, and a
 *   block's scale goes to its scores and weights.  A weight is rounded to fp16 (few rows: to 22 bits) with V's scale in
 *   it, relative to the row's largest such product: keys that the row does not see, or hardly weighs, take nothing from
 *   the others whatever their scale; a key whose product is below 2^-29 of the largest (2^-21 with the workspace of
 *   tq_chunk_workspace_for()) may count as 0.  Scores are fp32: beyond 2^22 in magnitude their steps pass what a weight
 *   can tell apart, and a row may come out as NaN from 2^28 on.
 *   workspace: device, tq_chunk_workspace_bytes() bytes, 256-byte aligned; calls that may overlap need their own.
 * max_tokens chooses the kernel: a batch of at most 16 rows (max_tokens * n_q_heads / n_kv_heads; 8 at head_dim 256)
 * per sequence and KV head takes one that is about twice as fast for them, so a decode step passes max_tokens = 1.
 * The operands of the products are fp16: queries (scaled by a power of two per row, so that no type overflows), keys
 * and values as scale * code (turbo: norm * level), weights; the sums and the softmax are fp32.  Few rows: keys are
 * exact and fp32 queries have 22 bits.  Against fp64, N(0, 1) queries on a cache with 1 % of its channels 20 times
 * larger (2-norm of all outputs, the output's own rounding included: 2e-4 in fp16, 1.7e-3 in bf16): few rows 3.3e-4 to
 * 4.5e-4 (F8_BLOCK: 2e-4), many 5e-4 to 2.0e-3 (fp16 out) and 1.9e-3 to 2.7e-3 (bf16 out).  Stored q8_0 scales above
 * 511.5 (values above 64960) are read as 511.5.  The result of a call does not depend on what else runs.  A block-table
 * entry out of range sets status bit 2, and its keys are left out.
 */
tq_status tq_chunk_attention(const tq_context* ctx, const tq_batch* batch, const void* q, tq_dtype q_dtype,
                             int64_t q_token_stride, int n_q_heads, const tq_cache_view* k_view,
                             const tq_cache_view* v_view, int layer, float softmax_scale, const tq_score_mods* mods,
                             void* workspace, size_t workspace_bytes, void* out, tq_dtype out_dtype,
                             tq_stream_t stream);

/*
 * The same with sinks, first tokens that stay visible: where sinks s > 0, the window of mods hides no key j < f + s,
 * f = first_keys[t] (0 without first_keys, and where that is negative).  Without a window they change nothing.  (A call of
 * its own, so that tq_score_mods keeps its size for programs that were built without them.)
 */
tq_status tq_chunk_attention_sinks(const tq_context* ctx, const tq_batch* batch, const void* q, tq_dtype q_dtype,
                                   int64_t q_token_stride, int n_q_heads, const tq_cache_view* k_view,
                                   const tq_cache_view* v_view, int layer, float softmax_scale, const tq_score_mods* mods,
                                   int sinks, void* workspace, size_t workspace_bytes, void* out, tq_dtype out_dtype,
                                   tq_stream_t stream);

/* ---- dequantize (reconstruction; test and debugging path) ---- */

/*
 * Reconstructs n slots of one layer of a view into out (device float
 * [n][n_kv_heads][d]) in the original, unrotated space.  Slot t = slots[t]
 * (device int64 [n]) or slot_begin + t.  Turbo: n diag(s) H c[idx], plus for K
 * formats with include_qjl != 0 the QJL vector-form residual
 * diag(s) H (rnorm sqrt(pi/2)/d S^T (2 sigma - 1)).  Q8_0: q * scale.
 * MINMAX: q * scale + zero.  F8_BLOCK: code * 2^e.  Skipped (out-of-range) slots are written as zeros.
 */
tq_status tq_dequantize(const tq_context* ctx, const tq_cache_view* view, int layer,
                        const int64_t* slots, int64_t slot_begin, int n,
                        int include_qjl, float* out, tq_stream_t stream);

/* ---- persistence of a compressed cache (host; out of the hot path) ---- */

/*
 * A compressed cache saved to disk and read back ("mac-code TurboQuant analysis",
 * section 2.4: the compressed arrays are serialised with a small JSON metadata
 * record; here both go into one file).  File layout:
 *   the 9 bytes "TQCACHE1\n";
 *   one JSON object on one line followed by "\n", with the keys version, format,
 *     format_id, head_dim, n_kv_heads, page_size, num_pages, n_layers, bits,
 *     payload_bytes, header_bytes, wht_seed, qjl_seed, tables_hash (16 hex
 *     digits), data_hash (16 hex digits) and layout;
 *   zero bytes up to the next multiple of 4096;
 *   the view's payload array (all its layers, in the view's own order), then its
 *     header array.
 * tables_hash is FNV-1a 64 over head_dim (int32), the sign diagonal (int8 [d]),
 * the QJL matrix (float [d*d]) and the codebook tables (float [3][8], [3][7]) of
 * the context; data_hash is FNV-1a 64 over the two arrays as 64-bit
 * little-endian words, taken in blocks of 64 MiB per array (each block's trailing
 * bytes one at a time).  Codes are only meaningful with the tables they were made
 * with, so a load checks tables_hash against its context.
 */

/* FNV-1a 64 hash of the context's tables (the file's tables_hash). */
tq_status tq_context_tables_hash(const tq_context* ctx, uint64_t* hash);

/*
 * Writes every layer of `view` to `path` (created or replaced: written to
 * path + ".partial" and renamed on success).  host_memory = 0: the view's arrays
 * are device memory of the current device (the device is synchronised, the
 * arrays are copied through a host buffer of at most 64 MiB); 1: host memory.
 * ctx (may be NULL: seeds and tables_hash are then written as 0) supplies the
 * seeds and the tables hash; its head_dim must match the view's.  Synchronous.
 * Errors: TQ_ERR_INVALID_ARG (bad view, I/O failure), TQ_ERR_OOM, TQ_ERR_CUDA.
 */
tq_status tq_cache_save(const tq_context* ctx, const tq_cache_view* view, int host_memory, const char* path);

/*
 * Reads the geometry of a file written by tq_cache_save: format, head_dim,
 * n_kv_heads, page_size, num_pages, n_layers and bits into *geometry (payload and
 * header set to NULL), the tables hash into *tables_hash (may be NULL), so that a
 * caller can allocate the view to load into.  TQ_ERR_INVALID_ARG if the file is
 * missing or not such a file.
 */
tq_status tq_cache_file_info(const char* path, tq_cache_view* geometry, uint64_t* tables_hash);

/*
 * Reads a file written by tq_cache_save into `view`, whose format, head_dim,
 * n_kv_heads, page_size, num_pages, n_layers and bits must equal the file's
 * (host_memory as for tq_cache_save).  With a context, the file's tables_hash
 * must equal the context's.  The data hash is checked after the copy; on any
 * mismatch (geometry, tables, size, trailing bytes, data hash) the call returns
 * TQ_ERR_INVALID_ARG, and when the data hash alone fails the view already holds
 * the file's (corrupt) bytes.  Synchronous.
 */
tq_status tq_cache_load(const tq_context* ctx, const tq_cache_view* view, int host_memory, const char* path);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H_ */
