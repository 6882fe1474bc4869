// Norms of queries and keys per head with the rotation in the same pass, and their gradient.
//
//   r = 1 / sqrt(sum x_i^2 / d + eps), y = r x w, out = m R(p) y;  with g = m R(p)^T dout and x' = r x:
//   dx = r (g w - x' sum(g w x') / d), dw = sum over rows g x'.
//
// One pass over the data: 2 (gradient 3) elements moved per element, so HBM bounds it.  d / 16 lanes hold a vector, 8 pairs
// of coordinates each, whose sums they share by shuffles; such a group walks over heads of one token with the angles and
// the weight in registers, and asks for the next heads' words before it turns to the first ones.  Queries and keys are
// heads of one launch.  4096 tokens of 32 + 8 heads of 128 in bf16: 17.7 us for 84 MB, where a plain copy of them takes 16.2
// (4 heads per group 18.4; blocks of 256 threads 20.5, of 128 with four on an SM 19.4; two heads in flight and six blocks
// 20.0); the gradient 33 us for 126 MB, of which the first kernel 28 (4 heads per group 38, 16 41; two heads in flight and
// four blocks instead of four and three 34.8, one and four 43; twice or half the blocks for the partial sums the same).
// What did not pay: two coordinates per instruction (the pairs' moves: 21.9 and 36.5), the next heads' lines asked into L2
// at once (19.2 and 36).
//
// The weight's gradient: a lane adds up its 16 coordinates over the rows of its group, the CTA's groups are joined in
// shared memory and leave one row of partial sums, and a second kernel adds those rows in their order, with what each sum
// loses carried along (fp64 sums, at this GPU's rate for them, took 21 us for 1210 rows of 128).
#include <type_traits>

#include "tq_batch.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;
constexpr int kPairs = 8;            // of a lane
constexpr int kHeads = 8;            // most heads of a group
constexpr int kGradCtasPerSm = 16;
constexpr int kJoin = 32;            // rows of partial sums that the second kernel adds side by side

// How a lane's pairs lie: two runs of 8 (halves), one run of 16 (interleaved), or halves whose border no run meets.
enum Mode { kRuns, kInterleaved, kScattered };

// Coordinates of pair i of lane l.
template <int MODE>
struct At {
  int l, r;  // rotary_dim
  __device__ __forceinline__ int a(int i) const {
    if (MODE == kInterleaved) return 16 * l + 2 * i;
    if (MODE == kRuns) return 16 * l < r ? 8 * l + i : r + 16 * (l - r / 16) + i;
    const int j = 8 * l + i;
    return 2 * j < r ? j : 2 * j;
  }
  __device__ __forceinline__ int b(int i) const {
    if (MODE == kInterleaved) return 16 * l + 2 * i + 1;
    if (MODE == kRuns) return 16 * l < r ? r / 2 + 8 * l + i : r + 16 * (l - r / 16) + 8 + i;
    const int j = 8 * l + i;
    return 2 * j < r ? j + r / 2 : 2 * j + 1;
  }
};

template <class T>
struct Raw {
  static constexpr int W = 16 * sizeof(T) / 16;
  uint4 w[W];
};

template <int MODE, class T>
__device__ __forceinline__ void fetch(const T* row, const At<MODE>& at, bool on, Raw<T>& x) {
  constexpr int W = Raw<T>::W;
#pragma unroll
  for (int k = 0; k < W; ++k) x.w[k] = make_uint4(0u, 0u, 0u, 0u);
  if (!on) return;
  if constexpr (MODE == kScattered) {
    T* e = reinterpret_cast<T*>(x.w);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      e[i] = row[at.a(i)];
      e[kPairs + i] = row[at.b(i)];
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(row + at.a(0));
    const uint4* q = MODE == kRuns ? reinterpret_cast<const uint4*>(row + at.b(0)) : p + W / 2;
#pragma unroll
    for (int k = 0; k < W / 2; ++k) {
      x.w[k] = __ldcs(p + k);
      x.w[W / 2 + k] = __ldcs(q + k);
    }
  }
}

template <int MODE, class T>
__device__ __forceinline__ void unpack(const Raw<T>& x, float (&a)[kPairs], float (&b)[kPairs]) {
  float y[16];
  load_row<16>(reinterpret_cast<const T*>(x.w), y);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    a[i] = MODE == kInterleaved ? y[2 * i] : y[i];
    b[i] = MODE == kInterleaved ? y[2 * i + 1] : y[kPairs + i];
  }
}

template <int MODE, class T>
__device__ __forceinline__ void put(T* row, const At<MODE>& at, const float (&a)[kPairs], const float (&b)[kPairs]) {
  if constexpr (MODE == kScattered) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      from_float(row + at.a(i), a[i]);
      from_float(row + at.b(i), b[i]);
    }
  } else if constexpr (MODE == kRuns) {
    store_row<kPairs>(row + at.a(0), a);
    store_row<kPairs>(row + at.b(0), b);
  } else {
    float y[16];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      y[2 * i] = a[i];
      y[2 * i + 1] = b[i];
    }
    store_row<16>(row + at.a(0), y);
  }
}

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
  if (!w) return 1.f;
  if (dtype == TQ_DTYPE_F32) return static_cast<const float*>(w)[i];
  if (dtype == TQ_DTYPE_F16) return to_float(static_cast<const __half*>(w)[i]);
  return to_float(static_cast<const __nv_bfloat16*>(w)[i]);
}

template <int LPV>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = 1; m < LPV; m <<= 1) x += __shfl_xor_sync(kFull, x, m);
  return x;
}

// 1 / sqrt(mean square + eps) of the group's vector.  Squares that pass the range of fp32 are summed again of x 2^-70: x is
// scaled then, and the result belongs to the scaled one; returns the scale.
template <int LPV, class T>
__device__ __forceinline__ float norm_of(float (&a)[kPairs], float (&b)[kPairs], float eps, float* r) {
  constexpr float kInv = 1.f / (16 * LPV);
  auto sum = [&]() {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      s0 = fmaf(a[i], a[i], s0);
      s1 = fmaf(b[i], b[i], s1);
    }
    return group_sum<LPV>(s0 + s1);
  };
  float ss = sum(), scale = 1.f;
  if constexpr (!std::is_same<T, __half>::value) {  // (fp16 squares do not pass it)
    const bool large = !(fmaf(ss, kInv, eps) < 3.0e38f);
    if (__any_sync(kFull, large)) {
      if (large) {
        scale = 0x1p-70f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          a[i] *= scale;
          b[i] *= scale;
        }
      }
      ss = sum();
    }
  }
  *r = rsqrtf(fmaf(ss, kInv, eps * scale * scale));
  return scale;
}

struct Launch {
  NormArgs n;
  int hpt;            // heads per group
  int splits_q, splits;
  int ctas;           // gradient: CTAs per split
  float* part;        // gradient: [splits * ctas][d]
};

template <int MODE>
__device__ __forceinline__ void angles(const NormArgs& n, int l, int pos, bool on, float (&cs)[kPairs], float (&sn)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int j = kPairs * l + i;
    float2 f = make_float2(1.f, 0.f);
    if (on && 2 * j < n.rope.rotary_dim) f = rope_at(n.rope.turns[j], pos, n.rope.attn_factor);
    cs[i] = f.x;
    sn[i] = f.y;
  }
}

// Of heads that are rotated in part (PART), the pairs of lane l that are, its first ones.  The others are not pairs: they are
// left out of the rotation, not turned by 0, which would hand an infinity or a NaN on to the neighbour in the lane.  (Without
// the form for wholly rotated heads, which selects nothing: 18.0 us instead of 17.5 for the call at the head.)
__device__ __forceinline__ int turned(const NormArgs& n, int l) { return n.rope.rotary_dim / 2 - kPairs * l; }

template <class T, int D, int MODE, bool PART>
__global__ void __launch_bounds__(kThreads, MODE == kScattered ? 4 : 5) norm_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / 16, U = 8 / sizeof(T);  // heads in flight: as many as have the registers
  pdl_launch_dependents();  // the next kernel's start overlaps this one, as this one's the last
  pdl_wait();
  const long long group = ((long long)blockIdx.x * kThreads + threadIdx.x) / LPV;
  const int l = threadIdx.x % LPV, token = (int)(group / L.splits), split = (int)(group - (long long)token * L.splits);
  const bool of_k = split >= L.splits_q, on = token < L.n.n_tokens;
  const NormRows& R = L.n.rows[of_k];
  const int h0 = (of_k ? split - L.splits_q : split) * L.hpt, h1 = min(R.n_heads, h0 + L.hpt);
  const At<MODE> at{l, L.n.rope.rotary_dim};
  const T* x = static_cast<const T*>(R.x) + (long long)token * R.x_stride;
  T* y = static_cast<T*>(R.out) + (long long)token * R.out_stride;
  Raw<T> raw[U];
  auto ask = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) fetch<MODE>(x + (long long)(h + u) * D, at, on && h + u < h1, raw[u]);
  };
  ask(h0);
  float cs[kPairs], sn[kPairs], wa[kPairs], wb[kPairs];
  angles<MODE>(L.n, l, on ? L.n.positions[token] : 0, on, cs, sn);
  const int pairs = turned(L.n, l);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    wa[i] = weight_at(R.weight, L.n.weight_dtype, at.a(i));
    wb[i] = weight_at(R.weight, L.n.weight_dtype, at.b(i));
  }
  for (int i0 = 0; i0 < L.hpt; i0 += U) {  // (the warp's groups alike: the sums are the warp's)
    if (i0) ask(h0 + i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= L.hpt) break;
      const int h = h0 + i0 + u;
      float a[kPairs], b[kPairs], r;
      unpack<MODE>(raw[u], a, b);
      norm_of<LPV, T>(a, b, L.n.eps, &r);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float p = a[i] * r * wa[i], q = b[i] * r * wb[i];
        const bool turn = !PART || i < pairs;
        a[i] = turn ? p * cs[i] - q * sn[i] : p;
        b[i] = turn ? p * sn[i] + q * cs[i] : q;
      }
      if (on && h < h1) put<MODE>(y + (long long)h * D, at, a, b);
    }
  }
}

template <class T, int D, int MODE, bool PART>
__global__ void __launch_bounds__(kThreads, 3) norm_grad_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / 16, GPC = kThreads / LPV, U = 8 / sizeof(T);
  __shared__ float joined[kThreads / 32][D];
  const int l = threadIdx.x % LPV, g = threadIdx.x / LPV, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x / L.ctas, c = blockIdx.x - split * L.ctas;
  pdl_launch_dependents();
  pdl_wait();
  const bool of_k = split >= L.splits_q;
  const NormRows& R = L.n.rows[of_k];
  const int h0 = (of_k ? split - L.splits_q : split) * L.hpt, h1 = min(R.n_heads, h0 + L.hpt);
  const At<MODE> at{l, L.n.rope.rotary_dim};
  const int pairs = turned(L.n, l);
  float wa[kPairs], wb[kPairs], da[kPairs], db[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    wa[i] = weight_at(R.weight, L.n.weight_dtype, at.a(i));
    wb[i] = weight_at(R.weight, L.n.weight_dtype, at.b(i));
    da[i] = db[i] = 0.f;
  }
  for (int t0 = c * GPC; t0 < L.n.n_tokens; t0 += L.ctas * GPC) {
    const int token = t0 + g;
    const bool on = token < L.n.n_tokens;
    const T* x = static_cast<const T*>(R.x) + (long long)token * R.x_stride;
    const T* d_out = static_cast<const T*>(R.dout) + (long long)token * R.dout_stride;
    T* dx = static_cast<T*>(R.out) + (long long)token * R.out_stride;
    Raw<T> raw[U], grad[U];
    auto ask = [&](int h) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        fetch<MODE>(x + (long long)(h + u) * D, at, on && h + u < h1, raw[u]);
        fetch<MODE>(d_out + (long long)(h + u) * D, at, on && h + u < h1, grad[u]);
      }
    };
    ask(h0);
    float cs[kPairs], sn[kPairs];
    angles<MODE>(L.n, l, on ? L.n.positions[token] : 0, on, cs, sn);
    for (int i0 = 0; i0 < L.hpt; i0 += U) {
      if (i0) ask(h0 + i0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u >= L.hpt) break;
        const int h = h0 + i0 + u;
        const bool row = on && h < h1;
        float a[kPairs], b[kPairs], p[kPairs], q[kPairs], r;
        unpack<MODE>(raw[u], a, b);
        unpack<MODE>(grad[u], p, q);
        const float scale = norm_of<LPV, T>(a, b, L.n.eps, &r);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const bool turn = !PART || i < pairs;
          const float ga = turn ? p[i] * cs[i] + q[i] * sn[i] : p[i], gb = turn ? q[i] * cs[i] - p[i] * sn[i] : q[i];
          a[i] *= r;
          b[i] *= r;
          if (row) {
            da[i] = fmaf(ga, a[i], da[i]);
            db[i] = fmaf(gb, b[i], db[i]);
          }
          p[i] = ga * wa[i];
          q[i] = gb * wb[i];
          dot = fmaf(p[i], a[i], fmaf(q[i], b[i], dot));
        }
        dot = group_sum<LPV>(dot) * (1.f / D);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          p[i] = r * fmaf(-a[i], dot, p[i]) * scale;
          q[i] = r * fmaf(-b[i], dot, q[i]) * scale;
        }
        if (row) put<MODE>(dx + (long long)h * D, at, p, q);
      }
    }
  }
  if (!R.dweight) return;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
#pragma unroll
    for (int m = LPV; m < 32; m <<= 1) {
      da[i] += __shfl_xor_sync(kFull, da[i], m);
      db[i] += __shfl_xor_sync(kFull, db[i], m);
    }
    if (lane < LPV) {
      joined[warp][at.a(i)] = da[i];
      joined[warp][at.b(i)] = db[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += joined[w][i];
    L.part[(long long)blockIdx.x * D + i] = s;
  }
}

// s += x; what the rounding of the sum leaves goes to lost (the two-sum of Knuth), nothing of a sum beyond fp32.
__device__ __forceinline__ void add_exactly(float& s, float& lost, float x) {
  const float t = __fadd_rn(s, x), v = __fsub_rn(t, s);
  const float rest = __fadd_rn(__fsub_rn(s, __fsub_rn(t, v)), __fsub_rn(x, v));
  if (isfinite(t)) lost += rest;
  s = t;
}

// The weight's gradient from the CTAs' rows: 32 coordinates of q's (y = 0) or k's weight.
__global__ void __launch_bounds__(32 * kJoin) weight_kernel(const __grid_constant__ Launch L, int d) {
  __shared__ float2 sums[kJoin][33];
  pdl_launch_dependents();
  pdl_wait();
  const bool of_k = blockIdx.y != 0;
  const NormRows& R = L.n.rows[of_k];
  if (!R.dweight) return;
  const int first = of_k ? L.splits_q * L.ctas : 0, end = of_k ? L.splits * L.ctas : L.splits_q * L.ctas;
  const int i = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
  float s = 0.f, lost = 0.f;
#pragma unroll 8
  for (int c = first + y; c < end; c += kJoin) add_exactly(s, lost, L.part[(long long)c * d + i]);
  sums[y][threadIdx.x % 32] = make_float2(s, lost);
  __syncthreads();
  if (y == 0) {
    for (int k = 1; k < kJoin; ++k) {
      const float2 x = sums[k][threadIdx.x];
      add_exactly(s, lost, x.x);
      lost += x.y;
    }
    R.dweight[i] = s + lost;
  }
}

// As many heads per group, up to 8, as leave 512 threads on every SM (the angles then cost a few percent); a call that cannot
// fill the GPU takes one head per group, the shortest chain.
int heads_per_group(const NormArgs& n, int d, int sm_count) {
  const int heads = n.rows[0].n_heads + n.rows[1].n_heads;
  int hpt = 1;
  while (hpt < kHeads && (long long)n.n_tokens * (heads / (2 * hpt)) * (d / 16) >= (long long)sm_count * 512) hpt *= 2;
  return hpt;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <class T, int D, int MODE, bool PART>
cudaError_t launch_forward(Launch& L, int sm_count, cudaStream_t s) {
  const NormArgs& n = L.n;
  const int hpt = heads_per_group(n, D, sm_count);
  L.hpt = hpt;
  L.splits_q = ceil_div(n.rows[0].n_heads, hpt);
  L.splits = L.splits_q + ceil_div(n.rows[1].n_heads, hpt);
  const long long threads = (long long)n.n_tokens * L.splits * (D / 16), grid = (threads + kThreads - 1) / kThreads;
  if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(norm_kernel<T, D, MODE, PART>, dim3((unsigned)grid), dim3(kThreads), 0, s, L);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <class T, int D, int MODE, bool PART>
cudaError_t launch_gradient(Launch& L, int sm_count, cudaStream_t s) {
  constexpr int GPC = kThreads / (D / 16);
  const NormArgs& n = L.n;
  L.hpt = heads_per_group(n, D, sm_count);
  const int hpt = L.hpt;
  L.splits_q = ceil_div(n.rows[0].n_heads, hpt);
  L.splits = L.splits_q + ceil_div(n.rows[1].n_heads, hpt);
  L.ctas = max(1, min(ceil_div(n.n_tokens, GPC), kGradCtasPerSm * sm_count / L.splits));
  cudaError_t e = launch_pdl(norm_grad_kernel<T, D, MODE, PART>, dim3((unsigned)(L.splits * L.ctas)), dim3(kThreads), 0, s, L);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || (!n.rows[0].dweight && !n.rows[1].dweight)) return e;
  e = launch_pdl(weight_kernel, dim3(D / 32, 2), dim3(32 * kJoin), 0, s, L, D);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <class T, int D, int MODE, bool PART>
cudaError_t launch_m(Launch& L, bool grad, int sm_count, cudaStream_t s) {
  return grad ? launch_gradient<T, D, MODE, PART>(L, sm_count, s) : launch_forward<T, D, MODE, PART>(L, sm_count, s);
}

template <class T, int D>
cudaError_t launch_d(Launch& L, bool grad, int sm_count, cudaStream_t s) {
  const tq_rope_table& t = L.n.rope;
  const bool part = t.rotary_dim < D;
  if (t.layout == TQ_ROPE_INTERLEAVED)
    return part ? launch_m<T, D, kInterleaved, true>(L, grad, sm_count, s) : launch_m<T, D, kInterleaved, false>(L, grad, sm_count, s);
  if (t.rotary_dim % 16 == 0)
    return part ? launch_m<T, D, kRuns, true>(L, grad, sm_count, s) : launch_m<T, D, kRuns, false>(L, grad, sm_count, s);
  return launch_m<T, D, kScattered, true>(L, grad, sm_count, s);
}

template <class T>
cudaError_t launch_t(Launch& L, bool grad, int sm_count, cudaStream_t s) {
  if (L.n.rope.head_dim == 64) return launch_d<T, 64>(L, grad, sm_count, s);
  if (L.n.rope.head_dim == 128) return launch_d<T, 128>(L, grad, sm_count, s);
  return launch_d<T, 256>(L, grad, sm_count, s);
}

cudaError_t launch_any(Launch& L, bool grad, int dtype, int sm_count, cudaStream_t s) {
  if (dtype == TQ_DTYPE_F32) return launch_t<float>(L, grad, sm_count, s);
  if (dtype == TQ_DTYPE_F16) return launch_t<__half>(L, grad, sm_count, s);
  return launch_t<__nv_bfloat16>(L, grad, sm_count, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int sm_count, cudaStream_t s) {
  Launch L{};
  L.n = a;
  return launch_any(L, false, dtype, sm_count, s);
}

size_t norm_grad_workspace(int sm_count, int d, int n_heads) {
  // splits: at most n_heads, which are as many CTAs where they pass kGradCtasPerSm per SM
  return (size_t)max(n_heads, kGradCtasPerSm * sm_count) * d * sizeof(float);
}

cudaError_t launch_norm_grad(const NormArgs& a, int dtype, void* workspace, int sm_count, cudaStream_t s) {
  Launch L{};
  L.n = a;
  L.part = static_cast<float*>(workspace);
  return launch_any(L, true, dtype, sm_count, s);
}

}  // namespace tq
