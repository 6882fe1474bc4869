// Host side of the serving step: the rotation table, argument checks and the exported entry points of the rotary,
// norm, append, read and chunk-attention kernels (tq_rope.cu, tq_norm.cu, tq_append.cu, tq_append_f8.cu, tq_chunk.cu).
#include <cmath>

#include "tq_internal.h"

using namespace tq;

namespace {

cudaStream_t cuda_stream(tq_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
tq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA; }

// Bytes of an element, 0 for an unknown type.
int dtype_bytes(tq_dtype t) {
  return t == TQ_DTYPE_F32 ? 4 : (t == TQ_DTYPE_F16 || t == TQ_DTYPE_BF16) ? 2 : 0;
}

// The kernels read and write rows with 16-byte accesses.  Without rows (n == 0) there need not be memory for them.
bool rows_ok(const void* p, int64_t stride, int64_t row, int esz, int n) {
  return (p || n == 0) && !(reinterpret_cast<uintptr_t>(p) & 15) && stride >= row && (stride * esz) % 16 == 0;
}

// A launch goes to the current device: a context of another one would be read from the wrong GPU.
bool on_device(const tq_context* ctx) {
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == ctx->device;
}

bool table_ok(const tq_context* ctx, const tq_rope_table* t) {
  return t->head_dim == ctx->d && t->rotary_dim >= 2 && t->rotary_dim <= ctx->d && t->rotary_dim % 2 == 0 &&
         (t->layout == TQ_ROPE_HALF || t->layout == TQ_ROPE_INTERLEAVED);
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// What the norm calls share; eps: a normal number, so that its square root has an inverse.
bool norm_call_ok(const tq_context* ctx, const tq_rope_table* table, tq_dtype dtype, tq_dtype weight_dtype, float eps,
                  int n_tokens, const int32_t* positions) {
  return ctx && table && table_ok(ctx, table) && dtype_bytes(dtype) && dtype_bytes(weight_dtype) && eps >= 0x1p-126f &&
         std::isfinite(eps) && n_tokens >= 0 && (positions || n_tokens == 0);
}

// Rows read from x and written to out (in place: the same stride).
bool norm_rows_ok(const tq_context* ctx, const void* x, int64_t x_stride, const void* out, int64_t out_stride, int n_heads,
                  tq_dtype dtype, int n_tokens) {
  const int esz = dtype_bytes(dtype);
  const int64_t row = (int64_t)n_heads * ctx->d;
  return n_heads >= 1 && n_heads <= (1 << 20) && rows_ok(x, x_stride, row, esz, n_tokens) &&
         rows_ok(out, out_stride, row, esz, n_tokens) && (x != out || n_tokens == 0 || x_stride == out_stride);
}

NormArgs norm_args(const tq_rope_table* table, int weight_dtype, float eps, int n_tokens, const int32_t* positions) {
  NormArgs a{};
  a.rope = *table;
  a.positions = positions;
  a.eps = eps;
  a.n_tokens = n_tokens;
  a.weight_dtype = weight_dtype;
  return a;
}

// The sizes of a batch; the device pointers too when it is not empty.
bool batch_ok(const tq_batch* b) {
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_tokens < 0 || b->max_ctx < 0) return false;
  return b->n_seqs == 0 || b->n_tokens == 0 || (b->cu_tokens && b->seq_lens);
}

bool batch_fits(const tq_batch* b, const DevView& v) {
  if (b->n_seqs == 0) return true;
  if (b->block_table) return b->max_blocks >= 1 && (int64_t)b->max_blocks * v.page_size >= b->max_ctx;
  return b->max_ctx <= v.page_size && b->n_seqs <= v.num_pages;
}

DevBatch dev_batch(const tq_batch* b) {
  return DevBatch{b->n_seqs, b->n_tokens, b->max_tokens, b->max_ctx, b->max_blocks, b->cu_tokens, b->seq_lens,
                  b->block_table};
}

bool is_f8(const DevView& v) { return v.format == TQ_FMT_F8_BLOCK; }

bool mods_ok(const tq_score_mods* m) {
  return !m || (m->softcap >= 0.0f && std::isfinite(m->softcap) && m->window >= 0);
}

bool stored_ok(const DevView& v) { return v.format == TQ_FMT_Q8_0 || (format_is_turbo(v.format) && !v.has_qjl); }

}  // namespace

extern "C" {

tq_status tq_rope_build(const tq_rope_params* p, tq_rope_table* out) {
  if (!p || !out) return TQ_ERR_INVALID_ARG;
  const int d = p->head_dim, r = p->rotary_dim;
  if (d != 64 && d != 128 && d != 256) return TQ_ERR_UNSUPPORTED;
  if (r < 2 || r > d || r % 2 || (p->layout != TQ_ROPE_HALF && p->layout != TQ_ROPE_INTERLEAVED))
    return TQ_ERR_INVALID_ARG;
  if (p->scaling < TQ_ROPE_NONE || p->scaling > TQ_ROPE_YARN) return TQ_ERR_INVALID_ARG;
  if (!(p->base > 1.0) || !std::isfinite(p->base) || !(p->attn_factor >= 0.0) || !std::isfinite(p->attn_factor))
    return TQ_ERR_INVALID_ARG;
  const bool banded = p->scaling == TQ_ROPE_WAVELENGTH || p->scaling == TQ_ROPE_YARN;
  if (p->scaling != TQ_ROPE_NONE && (!(p->factor > 0.0) || !std::isfinite(p->factor))) return TQ_ERR_INVALID_ARG;
  if (p->scaling == TQ_ROPE_NTK && r <= 2) return TQ_ERR_INVALID_ARG;
  const double low = p->low == 0.0 ? 1.0 : p->low;
  const double high = p->high == 0.0 ? (p->scaling == TQ_ROPE_YARN ? 32.0 : 4.0) : p->high;
  if (banded && (!(p->original_ctx > 0.0) || !std::isfinite(p->original_ctx) || !(low > 0.0) || !(high > low) ||
                 !std::isfinite(high)))
    return TQ_ERR_INVALID_ARG;

  const double two_pi = 6.283185307179586476925;
  const double base = p->scaling == TQ_ROPE_NTK ? p->base * std::pow(p->factor, (double)r / (r - 2)) : p->base;
  if (!std::isfinite(base) || !(base > 0.0)) return TQ_ERR_INVALID_ARG;
  double from = 0.0, width = 1.0, attn = 1.0;
  if (p->scaling == TQ_ROPE_YARN) {
    auto dim = [&](double turns) { return r * std::log(p->original_ctx / (two_pi * turns)) / (2.0 * std::log(base)); };
    from = std::fmax(std::floor(dim(high)), 0.0);
    width = std::fmax(std::fmin(std::ceil(dim(low)), r - 1.0) - from, 0.001);
    attn = 0.1 * std::log(p->factor) + 1.0;
  }
  if (p->attn_factor > 0.0) attn = p->attn_factor;
  if (!std::isfinite((float)attn)) return TQ_ERR_INVALID_ARG;
  tq_rope_table t{};
  t.head_dim = d;
  t.rotary_dim = r;
  t.layout = p->layout;
  t.attn_factor = (float)attn;
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (p->scaling == TQ_ROPE_LINEAR) f /= p->factor;
    if (p->scaling == TQ_ROPE_WAVELENGTH) {
      const double s = std::fmin(std::fmax((p->original_ctx * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = s * f + (1.0 - s) * f / p->factor;
    }
    if (p->scaling == TQ_ROPE_YARN) {
      const double g = std::fmin(std::fmax((i - from) / width, 0.0), 1.0);
      f = g * f / p->factor + (1.0 - g) * f;
    }
    if (!std::isfinite(f)) return TQ_ERR_INVALID_ARG;  // (its fraction of a turn would be whatever the machine makes of NaN)
    const double turn = f / two_pi, frac = turn - std::floor(turn);
    t.turns[i] = (uint64_t)std::ldexp(frac, 64);  // frac < 1 has 53 bits: below 2^64
  }
  *out = t;
  return TQ_OK;
}

tq_status tq_rope(const tq_context* ctx, const tq_rope_table* table, const void* x, tq_dtype dtype, int n_tokens,
                  int n_heads, int64_t x_token_stride, const int32_t* positions, int inverse, void* out,
                  int64_t out_token_stride, tq_stream_t stream) {
  const int esz = dtype_bytes(dtype);
  if (!ctx || !table || !table_ok(ctx, table) || !esz || n_tokens < 0 || n_heads < 1 || n_heads > (1 << 20))
    return TQ_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return TQ_ERR_INVALID_ARG;
  const int64_t row = (int64_t)n_heads * ctx->d;
  if (!rows_ok(x, x_token_stride, row, esz, n_tokens) || !rows_ok(out, out_token_stride, row, esz, n_tokens) ||
      (!positions && n_tokens))
    return TQ_ERR_INVALID_ARG;
  if (x == out && n_tokens && x_token_stride != out_token_stride) return TQ_ERR_INVALID_ARG;
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return TQ_OK;
  return cuda_status(launch_rope(*table, x, dtype, n_tokens, n_heads, x_token_stride, positions, inverse, out,
                                 out_token_stride, ctx->sm_count, cuda_stream(stream)));
}

tq_status tq_norm_rope(const tq_context* ctx, const tq_rope_table* table, const tq_norm_rows* q, const tq_norm_rows* k,
                       tq_dtype dtype, tq_dtype weight_dtype, float eps, int n_tokens, const int32_t* positions,
                       tq_stream_t stream) {
  if (!norm_call_ok(ctx, table, dtype, weight_dtype, eps, n_tokens, positions) || (!q && !k)) return TQ_ERR_INVALID_ARG;
  NormArgs a = norm_args(table, weight_dtype, eps, n_tokens, positions);
  for (int i = 0; i < 2; ++i) {
    const tq_norm_rows* r = i ? k : q;
    if (!r) continue;
    if (!norm_rows_ok(ctx, r->x, r->x_token_stride, r->out, r->out_token_stride, r->n_heads, dtype, n_tokens))
      return TQ_ERR_INVALID_ARG;
    if (!aligned(r->weight, dtype_bytes(weight_dtype))) return TQ_ERR_INVALID_ARG;
    a.rows[i] = NormRows{r->x, r->out, nullptr, r->weight, nullptr, r->x_token_stride, r->out_token_stride, 0, r->n_heads};
  }
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return TQ_OK;
  return cuda_status(launch_norm(a, dtype, ctx->sm_count, cuda_stream(stream)));
}

size_t tq_norm_rope_grad_workspace_bytes(const tq_context* ctx, int n_tokens, int n_heads) {
  if (!ctx || n_tokens < 0 || n_heads < 1 || n_heads > (1 << 21)) return 0;
  return norm_grad_workspace(ctx->sm_count, ctx->d, n_heads);
}

tq_status tq_norm_rope_grad(const tq_context* ctx, const tq_rope_table* table, const tq_norm_grad_rows* q,
                            const tq_norm_grad_rows* k, tq_dtype dtype, tq_dtype weight_dtype, float eps, int n_tokens,
                            const int32_t* positions, void* workspace, size_t workspace_bytes, tq_stream_t stream) {
  if (!norm_call_ok(ctx, table, dtype, weight_dtype, eps, n_tokens, positions) || (!q && !k)) return TQ_ERR_INVALID_ARG;
  NormArgs a = norm_args(table, weight_dtype, eps, n_tokens, positions);
  bool sums = false;
  for (int i = 0; i < 2; ++i) {
    const tq_norm_grad_rows* r = i ? k : q;
    if (!r) continue;
    if (!norm_rows_ok(ctx, r->x, r->x_token_stride, r->dx, r->dx_token_stride, r->n_heads, dtype, n_tokens) ||
        !norm_rows_ok(ctx, r->dout, r->dout_token_stride, r->dx, r->dx_token_stride, r->n_heads, dtype, n_tokens))
      return TQ_ERR_INVALID_ARG;
    if (!aligned(r->weight, dtype_bytes(weight_dtype)) || !aligned(r->dweight, sizeof(float))) return TQ_ERR_INVALID_ARG;
    a.rows[i] = NormRows{r->x, r->dx, r->dout, r->weight, r->dweight, r->x_token_stride, r->dx_token_stride,
                         r->dout_token_stride, r->n_heads};
    sums = sums || r->dweight;
  }
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  if (n_tokens == 0 && !sums) return TQ_OK;
  if (!workspace || workspace_bytes < norm_grad_workspace(ctx->sm_count, ctx->d, a.rows[0].n_heads + a.rows[1].n_heads) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return TQ_ERR_WORKSPACE;
  return cuda_status(launch_norm_grad(a, dtype, workspace, ctx->sm_count, cuda_stream(stream)));
}

tq_status tq_append_kv(const tq_context* ctx, const tq_batch* batch, const void* k, int64_t k_token_stride,
                       const void* v, int64_t v_token_stride, tq_dtype dtype, const tq_rope_table* rope,
                       const int32_t* positions, const tq_cache_view* k_view, const tq_cache_view* v_view, int layer,
                       tq_stream_t stream) {
  const int esz = dtype_bytes(dtype);
  if (!ctx || !batch_ok(batch) || !esz || layer < 0) return TQ_ERR_INVALID_ARG;
  AppendArgs a{};
  if (!make_dev_view(k_view, &a.k) || !make_dev_view(v_view, &a.v)) return TQ_ERR_INVALID_ARG;
  if (a.k.d != ctx->d || a.v.d != ctx->d || a.k.H != a.v.H || a.k.page_size != a.v.page_size ||
      a.k.num_pages != a.v.num_pages || layer >= a.k.n_layers || layer >= a.v.n_layers)
    return TQ_ERR_INVALID_ARG;
  if (rope && !table_ok(ctx, rope)) return TQ_ERR_INVALID_ARG;
  const int64_t row = (int64_t)a.k.H * ctx->d;
  if (!rows_ok(k, k_token_stride, row, esz, batch->n_tokens) || !rows_ok(v, v_token_stride, row, esz, batch->n_tokens))
    return TQ_ERR_INVALID_ARG;
  if (!batch_fits(batch, a.k) || !on_device(ctx)) return TQ_ERR_INVALID_ARG;
  const bool f8 = is_f8(a.k) && is_f8(a.v);
  if (!f8 && (a.k.format != TQ_FMT_Q8_0 || !stored_ok(a.v))) return TQ_ERR_UNSUPPORTED;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return TQ_OK;
  a.b = dev_batch(batch);
  a.tab = ctx->tables;
  a.layer = layer;
  a.xk = k;
  a.xv = v;
  a.k_stride = k_token_stride;
  a.v_stride = v_token_stride;
  a.positions = positions;
  a.has_rope = rope ? 1 : 0;
  if (rope) a.rope = *rope;
  return cuda_status(f8 ? launch_append_f8(a, dtype, ctx->sm_count, cuda_stream(stream))
                        : launch_append(a, dtype, ctx->sm_count, cuda_stream(stream)));
}

tq_status tq_read_kv(const tq_context* ctx, const tq_batch* batch, const tq_cache_view* k_view, void* k_out,
                     const tq_cache_view* v_view, void* v_out, tq_dtype dtype, int layer, tq_stream_t stream) {
  const int esz = dtype_bytes(dtype);
  if (!ctx || !batch_ok(batch) || !esz || layer < 0 || (!k_view && !v_view)) return TQ_ERR_INVALID_ARG;
  if ((!k_view && k_out) || (!v_view && v_out)) return TQ_ERR_INVALID_ARG;
  if (batch->n_tokens && (!k_view != !k_out || !v_view != !v_out)) return TQ_ERR_INVALID_ARG;
  AppendArgs a{};
  for (int i = 0; i < 2; ++i) {
    const tq_cache_view* view = i ? v_view : k_view;
    DevView* dv = i ? &a.v : &a.k;
    if (!view) continue;
    if (!make_dev_view(view, dv) || dv->d != ctx->d || layer >= dv->n_layers || !batch_fits(batch, *dv))
      return TQ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(i ? v_out : k_out) & 15) return TQ_ERR_INVALID_ARG;
  }
  if (k_view && v_view && (a.k.H != a.v.H || a.k.page_size != a.v.page_size || a.k.num_pages != a.v.num_pages))
    return TQ_ERR_INVALID_ARG;
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  const bool k_f8 = k_view && is_f8(a.k), v_f8 = v_view && is_f8(a.v);
  if ((k_view && !k_f8 && !stored_ok(a.k)) || (v_view && !v_f8 && !stored_ok(a.v))) return TQ_ERR_UNSUPPORTED;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return TQ_OK;
  a.b = dev_batch(batch);
  a.tab = ctx->tables;
  a.layer = layer;
  // (one launch, or one for each of two kinds of formats)
  for (int f8 = 0; f8 < 2; ++f8) {
    a.k_out = k_f8 == (f8 != 0) ? k_out : nullptr;
    a.v_out = v_f8 == (f8 != 0) ? v_out : nullptr;
    if (!a.k_out && !a.v_out) continue;
    const cudaError_t e = f8 ? launch_read_f8(a, dtype, ctx->sm_count, cuda_stream(stream))
                             : launch_read(a, dtype, ctx->sm_count, cuda_stream(stream));
    if (e != cudaSuccess) return TQ_ERR_CUDA;
  }
  return TQ_OK;
}

size_t tq_chunk_workspace_bytes(const tq_context* ctx, const tq_batch* batch, int n_q_heads, int n_kv_heads) {
  if (!ctx || !batch || batch->n_seqs < 0 || batch->n_tokens < 0 || batch->max_tokens < 0 || batch->max_ctx < 0 ||
      n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads)
    return 0;
  return chunk_workspace(ctx->sm_count, ctx->d, *batch, n_q_heads, n_kv_heads);
}

size_t tq_chunk_workspace_for(const tq_context* ctx, const tq_batch* batch, int n_q_heads, const tq_cache_view* k_view,
                              const tq_cache_view* v_view, const tq_score_mods* mods) {
  DevView k{}, v{};
  if (!make_dev_view(k_view, &k) || !make_dev_view(v_view, &v) || !mods_ok(mods)) return 0;
  const size_t least = tq_chunk_workspace_bytes(ctx, batch, n_q_heads, k.H);
  if (!least || k.d != ctx->d) return 0;
  return chunk_workspace_most(ctx->sm_count, k, *batch, n_q_heads, mods && mods->first_keys, mods ? mods->window : 0);
}

tq_status tq_chunk_attention(const tq_context* ctx, const tq_batch* batch, const void* q, tq_dtype q_dtype,
                             int64_t q_token_stride, int n_q_heads, const tq_cache_view* k_view,
                             const tq_cache_view* v_view, int layer, float softmax_scale, const tq_score_mods* mods,
                             void* workspace, size_t workspace_bytes, void* out, tq_dtype out_dtype,
                             tq_stream_t stream) {
  return tq_chunk_attention_sinks(ctx, batch, q, q_dtype, q_token_stride, n_q_heads, k_view, v_view, layer, softmax_scale,
                                  mods, 0, workspace, workspace_bytes, out, out_dtype, stream);
}

tq_status tq_chunk_attention_sinks(const tq_context* ctx, const tq_batch* batch, const void* q, tq_dtype q_dtype,
                                   int64_t q_token_stride, int n_q_heads, const tq_cache_view* k_view,
                                   const tq_cache_view* v_view, int layer, float softmax_scale, const tq_score_mods* mods,
                                   int sinks, void* workspace, size_t workspace_bytes, void* out, tq_dtype out_dtype,
                                   tq_stream_t stream) {
  const int esz = dtype_bytes(q_dtype), osz = dtype_bytes(out_dtype);
  if (!ctx || !batch_ok(batch) || !esz || !osz || layer < 0 || n_q_heads < 1 || !std::isfinite(softmax_scale))
    return TQ_ERR_INVALID_ARG;
  ChunkArgs a{};
  if (!make_dev_view(k_view, &a.k) || !make_dev_view(v_view, &a.v)) return TQ_ERR_INVALID_ARG;
  const int d = ctx->d;
  if (a.k.d != d || a.v.d != d || a.k.H != a.v.H || a.k.page_size != a.v.page_size ||
      a.k.num_pages != a.v.num_pages || layer >= a.k.n_layers || layer >= a.v.n_layers)
    return TQ_ERR_INVALID_ARG;
  const int64_t row = (int64_t)n_q_heads * d;
  if (!rows_ok(q, q_token_stride, row, esz, batch->n_tokens) || !rows_ok(out, row, row, osz, batch->n_tokens))
    return TQ_ERR_INVALID_ARG;
  if (!mods_ok(mods) || sinks < 0) return TQ_ERR_INVALID_ARG;
  if (!batch_fits(batch, a.k) || !on_device(ctx)) return TQ_ERR_INVALID_ARG;
  const bool f8 = is_f8(a.k) && is_f8(a.v);
  if ((!f8 && (a.k.format != TQ_FMT_Q8_0 || !stored_ok(a.v))) || n_q_heads % a.k.H) return TQ_ERR_UNSUPPORTED;
  // row numbers of a sequence and tile numbers are 32-bit in the kernels
  if ((int64_t)batch->max_tokens * (n_q_heads / a.k.H) >= (int64_t(1) << 30) || batch->max_ctx >= (1 << 30))
    return TQ_ERR_UNSUPPORTED;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return TQ_OK;
  if (!workspace || workspace_bytes < chunk_workspace(ctx->sm_count, d, *batch, n_q_heads, a.k.H) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return TQ_ERR_WORKSPACE;
  a.b = dev_batch(batch);
  a.tab = ctx->tables;
  a.layer = layer;
  a.n_q_heads = n_q_heads;
  a.G = n_q_heads / a.k.H;
  a.q = q;
  a.q_dtype = q_dtype;
  a.out_dtype = out_dtype;
  a.q_stride = q_token_stride;
  a.out = out;
  a.scale = softmax_scale;
  if (mods) {
    a.softcap = mods->softcap;
    a.window = mods->window;
    a.slopes = mods->slopes;
    a.first_keys = mods->first_keys;
    a.prefix_lens = mods->prefix_lens;
    a.sinks = mods->window ? sinks : 0;
  }
  const float lam_v = a.v.format == TQ_FMT_Q8_0 || f8 ? 1.f : ctx->f16_scale_h[a.v.idx_bits - 1];
  return cuda_status(launch_chunk(a, lam_v, workspace, workspace_bytes, ctx->sm_count, cuda_stream(stream)));
}

}  // extern "C"
