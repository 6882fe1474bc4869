// Attention of a ragged batch of chunks over the paged cache: one warp per row (token, query head), one pass over the
// row's visible keys with the running maximum and sum of the softmax.
#include "tq_batch.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;

template <int D>
__device__ __forceinline__ void load_vector(const DevView& V, const float* cb, long long vec, int lane,
                                            float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const unsigned char* pay = V.payload + vec * V.pay_bytes;
  const __half* hdr = reinterpret_cast<const __half*>(V.header + vec * V.hdr_bytes);
  if (V.format == TQ_FMT_Q8_0) {
    const float delta = __half2float(hdr[E * lane / 32]);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (float)reinterpret_cast<const int8_t*>(pay)[E * lane + e] * delta;
  } else {
    const float n = __half2float(hdr[0]);
#pragma unroll
    for (int e = 0; e < E; ++e)
      x[e] = n * cb[stream_code(reinterpret_cast<const uint32_t*>(pay), E * lane + e, V.code_bits)];
  }
}

__device__ __forceinline__ float q_at(const ChunkArgs& a, long long i) {
  if (a.q_dtype == TQ_DTYPE_F32) return static_cast<const float*>(a.q)[i];
  if (a.q_dtype == TQ_DTYPE_F16) return __half2float(static_cast<const __half*>(a.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[i]);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(row / a.n_q_heads), h = (int)(row - (long long)t * a.n_q_heads);
  if (t >= a.b.n_tokens) return;
  const int b = seq_of_row(a.b, t);
  if (b == a.b.n_seqs) return;
  const SeqOf s = seq_of(a.b, b);
  float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (!s.ok) {
    if (lane == 0) atomicOr(a.tab.status, kFlagSeqLen);
  } else {
    const int pos = s.len - s.n + (t - s.first);
    int lo = 0, hi = pos + 1;
    if (a.prefix_lens) hi = min(s.len, max(hi, a.prefix_lens[b]));
    if (a.window) lo = max(lo, pos - a.window + 1);
    if (a.first_keys) lo = max(lo, a.first_keys[t]);
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = q_at(a, (long long)t * a.q_stride + (long long)h * D + E * lane + e);
    const float slope = a.slopes ? a.slopes[h] : 0.f;
    const float* cb = a.tab.centroids + (a.v.format == TQ_FMT_Q8_0 ? 0 : (a.v.idx_bits - 1) * 8);
    for (int j = lo; j < hi; ++j) {
      const long long v0 = position_vector(a.b, a.k, a.layer, b, j);
      if (v0 < 0) {
        if (lane == 0) atomicOr(a.tab.status, kFlagBlockTable);
        continue;
      }
      const long long vec = v0 + (long long)(h / a.G) * a.k.page_size;
      float k[E], v[E];
      load_vector<D>(a.k, cb, vec, lane, k);
      float sc = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) sc = fmaf(q[e], k[e], sc);
      sc = warp_sum(sc) * a.scale;
      if (a.softcap > 0.f) sc = a.softcap * tanhf(sc / a.softcap);
      sc -= slope * (float)abs(pos - j);
      const __half* vh = reinterpret_cast<const __half*>(a.v.header + vec * a.v.hdr_bytes);
      for (int i = 0; i < a.v.hdr_bytes / 2; ++i)
        if (!isfinite(__half2float(vh[i]))) sc = NAN;
      const float mn = fmaxf(m, sc), mu = mn == -INFINITY ? 0.f : mn, al = __expf(m - mu), p = __expf(sc - mu);
      load_vector<D>(a.v, cb, vec, lane, v);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], al, p * v[e]);
      l = fmaf(l, al, p);
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    if (a.v.format != TQ_FMT_Q8_0) {
      warp_wht<D>(acc, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= (float)a.tab.signs[E * lane + e];
    }
  }
  const long long o = row * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (a.out_dtype == TQ_DTYPE_F32) from_float(static_cast<float*>(a.out) + o + e, acc[e]);
    else if (a.out_dtype == TQ_DTYPE_F16) from_float(static_cast<__half*>(a.out) + o + e, acc[e]);
    else from_float(static_cast<__nv_bfloat16*>(a.out) + o + e, acc[e]);
  }
}

}  // namespace

size_t chunk_workspace(int, int, const tq_batch&, int, int) { return 256; }

cudaError_t launch_chunk(const ChunkArgs& a, float, void*, int, cudaStream_t s) {
  const long long rows = (long long)a.b.n_tokens * a.n_q_heads;
  const long long grid = (rows + kWarps - 1) / kWarps;
  if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
  if (a.k.d == 64) chunk_kernel<64><<<(unsigned)grid, kWarps * 32, 0, s>>>(a);
  else if (a.k.d == 128) chunk_kernel<128><<<(unsigned)grid, kWarps * 32, 0, s>>>(a);
  else chunk_kernel<256><<<(unsigned)grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
