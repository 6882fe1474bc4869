// Rotary positions of n_tokens x n_heads vectors: y = m R(p f) x on the first rotary_dim coordinates.
//
// One pass over the data: 2 bytes read and written per fp16 element, so HBM bounds it.  A thread owns P pairs of one
// head position (P as wide as 16-byte accesses and the pair layout allow) and walks over `hpt` heads of its token, so
// that the angles are computed once for them: an exact 64-bit fixed-point product and one sincospi per pair.  4096 x 32
// heads of 128 in bf16: 13.8 us, 4.9 TB/s, 72 % of the copy bandwidth.
#include "tq_batch.cuh"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  tq_rope_table t;
  const void* x;
  void* out;
  long long x_stride, out_stride;
  const int32_t* positions;
  int n_tokens, n_heads, d;
  int hpt;        // heads per thread
  int splits;     // ceil(n_heads / hpt)
  int rot_units;  // threads per (token, head split) that rotate P pairs each
  int units;      // and those behind them that copy 2 P coordinates each (none in place)
  float m, sign;
};

// Units of one token are consecutive threads: (head split, unit) with the unit fastest, so that a warp's accesses
// cover whole rows.
template <class T, int P, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int per_token = a.splits * a.units;
  const long long id = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int t = (int)(id / per_token);
  if (t >= a.n_tokens) return;
  const int r = (int)(id - (long long)t * per_token);
  const int split = r / a.units, u = r - split * a.units;
  const int h0 = split * a.hpt, h1 = min(a.n_heads, h0 + a.hpt);
  const T* x = static_cast<const T*>(a.x) + (long long)t * a.x_stride;
  T* y = static_cast<T*>(a.out) + (long long)t * a.out_stride;
  if (u >= a.rot_units) {  // coordinates behind the rotated ones
    const int c = a.t.rotary_dim + (u - a.rot_units) * 2 * P;
    for (int h = h0; h < h1; ++h) {
      float v[2 * P];
      load_row<2 * P>(x + (long long)h * a.d + c, v);
      store_row<2 * P>(y + (long long)h * a.d + c, v);
    }
    return;
  }
  const int pos = a.positions[t];
  float cs[P], sn[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 f = rope_at(a.t.turns[u * P + i], pos, a.m);
    cs[i] = f.x;
    sn[i] = a.sign * f.y;
  }
  const int half = a.t.rotary_dim / 2;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const long long o = (long long)h * a.d;
    if constexpr (HALF) {
      float p[P], q[P], yp[P], yq[P];
      load_row<P>(x + o + u * P, p);
      load_row<P>(x + o + half + u * P, q);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        yp[i] = p[i] * cs[i] - q[i] * sn[i];
        yq[i] = p[i] * sn[i] + q[i] * cs[i];
      }
      store_row<P>(y + o + u * P, yp);
      store_row<P>(y + o + half + u * P, yq);
    } else {
      float p[2 * P], yp[2 * P];
      load_row<2 * P>(x + o + 2 * u * P, p);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        yp[2 * i] = p[2 * i] * cs[i] - p[2 * i + 1] * sn[i];
        yp[2 * i + 1] = p[2 * i] * sn[i] + p[2 * i + 1] * cs[i];
      }
      store_row<2 * P>(y + o + 2 * u * P, yp);
    }
  }
}

template <class T, int P>
cudaError_t launch_p(RopeArgs& a, int sm_count, bool in_place, cudaStream_t s) {
  a.rot_units = a.t.rotary_dim / 2 / P;
  a.units = a.rot_units + (in_place ? 0 : (a.d - a.t.rotary_dim) / (2 * P));
  const long long one = (long long)a.n_tokens * a.units;
  // As many heads per thread (up to 8: the angles then cost a few percent) as leave 1024 threads on every SM; a call
  // that cannot fill the GPU takes one head per thread, the shortest chain.
  int hpt = 1;
  while (hpt < 8 && hpt * 2 <= a.n_heads && one * (a.n_heads / (hpt * 2)) >= (long long)sm_count * 1024) hpt *= 2;
  a.hpt = hpt;
  a.splits = (a.n_heads + hpt - 1) / hpt;
  const long long threads = one * a.splits;
  const long long grid = (threads + kRopeThreads - 1) / kRopeThreads;
  if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
  if (a.t.layout == TQ_ROPE_HALF) rope_kernel<T, P, true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
  else rope_kernel<T, P, false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_t(RopeArgs& a, int sm_count, bool in_place, cudaStream_t s) {
  // The widest accesses that the layout allows: every unit starts at a multiple of its width, both in the rotated
  // part (rotary_dim / 2 a multiple of P; interleaved pairs are together, so half the pairs fill 16 bytes) and
  // behind it (2 P coordinates).
  constexpr int kWide = 16 / sizeof(T);
  const int half = a.t.rotary_dim / 2;
  const bool two = a.t.layout == TQ_ROPE_HALF;
  if (two && half % kWide == 0) return launch_p<T, kWide>(a, sm_count, in_place, s);
  if (half % (kWide / 2) == 0) return launch_p<T, kWide / 2>(a, sm_count, in_place, s);
  if constexpr (kWide == 8)
    if (half % 2 == 0) return launch_p<T, 2>(a, sm_count, in_place, s);
  return launch_p<T, 1>(a, sm_count, in_place, s);
}

}  // namespace

cudaError_t launch_rope(const tq_rope_table& rope, const void* x, int dtype, int n_tokens, int n_heads,
                        long long x_stride, const int32_t* positions, int inverse, void* out, long long out_stride,
                        int sm_count, cudaStream_t s) {
  RopeArgs a{};
  a.t = rope;
  a.x = x;
  a.out = out;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.positions = positions;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  a.d = rope.head_dim;
  a.m = rope.attn_factor;
  a.sign = inverse ? -1.f : 1.f;
  const bool in_place = x == out;
  if (dtype == TQ_DTYPE_F32) return launch_t<float>(a, sm_count, in_place, s);
  if (dtype == TQ_DTYPE_F16) return launch_t<__half>(a, sm_count, in_place, s);
  return launch_t<__nv_bfloat16>(a, sm_count, in_place, s);
}

}  // namespace tq
