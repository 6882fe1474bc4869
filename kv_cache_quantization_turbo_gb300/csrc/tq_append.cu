// Appending a ragged batch's keys (rotated on the way) and values to the paged cache, and reading rows back.
//
// A group of d / 16 lanes holds one vector, 16 consecutive coordinates per lane, and walks over `hpt` heads of its
// token, so that the token's place in the cache and the angles of its rotation are found once.  Everything between the
// load and the stored bytes stays in registers: the q8_0 scale of a 32-block is shared by two lanes, the turbo
// rotation runs four butterfly stages in a lane and log2(d / 16) across the group.  K and V are the two halves of one
// launch.  Bytes: both inputs once, the stored vectors once (append), the reverse (read).
#include "tq_batch.cuh"

namespace tq {
namespace {

constexpr int kApThreads = 128;
constexpr int kE = 16;  // coordinates per lane

struct Launch {
  AppendArgs a;
  int hpt, splits;  // heads per group, ceil(H / hpt)
};

// The group's place: token t, heads [h0, h1), the vector of (position, head 0), or vec < 0: nothing to do there.
struct Place {
  int t, h0, h1, seq, pos;
  long long vec;
  bool padding;  // behind the last sequence
};

template <int D>
__device__ __forceinline__ Place place_of(const Launch& L, const DevView& v, bool report) {
  constexpr int LPV = D / kE;
  Place p;
  const int g = (blockIdx.x * kApThreads + threadIdx.x) / LPV;
  p.t = g / L.splits;
  const int split = g - p.t * L.splits;
  p.h0 = split * L.hpt;
  p.h1 = min(v.H, p.h0 + L.hpt);
  p.vec = -1;
  p.padding = true;
  p.pos = 0;
  if (p.t >= L.a.b.n_tokens) return p;
  p.seq = seq_of_row(L.a.b, p.t);
  if (p.seq == L.a.b.n_seqs) return p;
  p.padding = false;
  const SeqOf s = seq_of(L.a.b, p.seq);
  if (!s.ok) {
    if (report && p.h0 == 0) atomicOr(L.a.tab.status, kFlagSeqLen);
    return p;
  }
  p.pos = s.len - s.n + (p.t - s.first);
  p.vec = position_vector(L.a.b, v, L.a.layer, p.seq, p.pos);
  if (p.vec < 0 && report && p.h0 == 0) atomicOr(L.a.tab.status, kFlagBlockTable);
  return p;
}

// H x / sqrt(D) of a vector held by a group, unscaled: lane `sub` owns coordinates [16 sub, 16 sub + 16).
template <int D>
__device__ __forceinline__ void group_wht(float (&x)[kE], int sub) {
#pragma unroll
  for (int s = 1; s < kE; s <<= 1) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if ((i & s) == 0) {
        const float u = x[i], v = x[i + s];
        x[i] = u + v;
        x[i + s] = u - v;
      }
    }
  }
#pragma unroll
  for (int m = 1; m < D / kE; m <<= 1) {
    const float f = sub & m ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = fmaf(x[i], f, __shfl_xor_sync(kFull, x[i], m));
  }
}

// round(x / delta), halves away from zero, as tq_encode_kv has it (the IEEE quotient, then roundf).
__device__ __forceinline__ int q8_code(float x, float delta) { return (int)roundf(__fdiv_rn(x, delta)); }

// Stores a vector as q8_0: 16 code bytes per lane, a scale per pair of lanes.
__device__ __forceinline__ void store_q8(const float (&x)[kE], unsigned char* pay, unsigned char* hdr, int sub,
                                         bool keep) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  const float delta = __fdiv_rn(amax, 127.0f);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (delta > 0.f) {
#pragma unroll
    for (int i = 0; i < kE; ++i) w[i / 4] |= (uint32_t)(uint8_t)(int8_t)q8_code(x[i], delta) << (8 * (i % 4));
  }
  if (!keep) return;
  *reinterpret_cast<uint4*>(pay + 16 * sub) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((sub & 1) == 0) reinterpret_cast<__half*>(hdr)[sub / 2] = __float2half_rn(delta);
}

// Stores a vector as turbo-MSE codes of B bits: n = |x|, y = H diag(s) x / n, the count of boundaries <= y.
template <int D, int B>
__device__ __forceinline__ void store_turbo(float (&x)[kE], const float (&bnd)[7], unsigned char* pay,
                                            unsigned char* hdr, int sub, bool keep) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int m = 1; m < D / kE; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
  group_wht<D>(x, sub);
  const float n = sqrtf(ss);
  const float f = n > 0.f ? __fdiv_rn(inv_sqrt_dim<D>(), n) : 0.f;
  uint64_t codes = 0;  // 16 B <= 48 bits
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const float y = x[i] * f;
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < (1 << B) - 1; ++k) c += y >= bnd[k] ? 1u : 0u;
    codes |= (uint64_t)c << (B * i);
  }
  if (!keep) return;
  uint16_t* dst = reinterpret_cast<uint16_t*>(pay) + B * sub;
#pragma unroll
  for (int k = 0; k < B; ++k) dst[k] = (uint16_t)(codes >> (16 * k));
  if (sub == 0) *reinterpret_cast<__half*>(hdr) = __float2half_rn(n);
}

template <class T, int D, int VB>  // VB: 0 q8_0 values, else turbo-MSE index bits
__global__ void __launch_bounds__(kApThreads) append_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE;
  const bool is_v = blockIdx.y != 0;
  const DevView& V = is_v ? L.a.v : L.a.k;
  const int sub = threadIdx.x % LPV;
  const Place p = place_of<D>(L, V, sub == 0 && !is_v);
  const bool keep = p.vec >= 0;  // the shuffles below are warp-wide: groups with nothing to store go along
  // heads per group may be cut short by H: the trip count is the launch's, the same for all groups
  const long long stride = is_v ? L.a.v_stride : L.a.k_stride;
  const T* row = static_cast<const T*>(is_v ? L.a.xv : L.a.xk) + (long long)(keep ? p.t : 0) * stride + 16 * sub;
  if (!is_v && L.a.has_rope) {
    const tq_rope_table& R = L.a.rope;
    const int half = R.rotary_dim / 2;
    const bool interleaved = R.layout == TQ_ROPE_INTERLEAVED;
    const int pos = keep && L.a.positions ? __ldg(L.a.positions + p.t) : p.pos;
    float c[kE], s[kE];
    // half layout: the partners of 16 consecutive coordinates are consecutive too unless a border of the rotated
    // halves falls inside; interleaved pairs never leave the lane
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int e = 16 * sub + i;
      c[i] = 1.f;
      s[i] = 0.f;
      if (e < R.rotary_dim) {
        const int pair = interleaved ? e >> 1 : (e < half ? e : e - half);
        const bool first = interleaved ? (e & 1) == 0 : e < half;
        if (interleaved && (i & 1)) {  // the even coordinate's angle
          c[i] = c[i - 1];
          s[i] = -s[i - 1];
        } else {
          const float2 f = rope_at(R.turns[pair], pos, R.attn_factor);
          c[i] = f.x;
          s[i] = first ? -f.y : f.y;
        }
      }
    }
    const bool whole = !interleaved && half % kE == 0;  // partners: one aligned block of 16
    const int to = 16 * sub < half ? half : -half;
    for (int j = 0; j < L.hpt; ++j) {
      const int h = p.h0 + j;
      const bool on = keep && h < p.h1;
      float x[kE], y[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] = y[i] = 0.f;
      if (on) {
        const T* src = row + (long long)h * D;
        load_row<kE>(src, x);
        if (interleaved) {
#pragma unroll
          for (int i = 0; i < kE; ++i) y[i] = x[i ^ 1];
        } else if (whole) {
          if (16 * sub < R.rotary_dim) load_row<kE>(src + to, y);
        } else {
#pragma unroll
          for (int i = 0; i < kE; ++i) {
            const int e = 16 * sub + i;
            if (e < R.rotary_dim) load_row<1>(src + i + (e < half ? half : -half), *reinterpret_cast<float(*)[1]>(&y[i]));
          }
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) x[i] = fmaf(c[i], x[i], s[i] * y[i]);
      }
      const long long vec = p.vec + (long long)h * V.page_size;
      store_q8(x, V.payload + vec * V.pay_bytes, V.header + vec * V.hdr_bytes, sub, on);
    }
    return;
  }
  float bnd[7];
  uint32_t neg = 0;  // sign flips of the lane's coordinates
  if constexpr (VB > 0) {
#pragma unroll
    for (int k = 0; k < 7; ++k) bnd[k] = k < (1 << VB) - 1 ? L.a.tab.boundaries[(VB - 1) * 7 + k] : 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) neg |= (L.a.tab.signs[16 * sub + i] < 0 ? 1u : 0u) << i;
  }
  for (int j = 0; j < L.hpt; ++j) {
    const int h = p.h0 + j;
    const bool on = keep && h < p.h1;
    float x[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = 0.f;
    if (on) load_row<kE>(row + (long long)h * D, x);
    const long long vec = p.vec + (long long)h * V.page_size;
    unsigned char* pay = V.payload + vec * V.pay_bytes;
    unsigned char* hdr = V.header + vec * V.hdr_bytes;
    if constexpr (VB > 0) {
      if (is_v) {
#pragma unroll
        for (int i = 0; i < kE; ++i) x[i] = (neg >> i) & 1u ? -x[i] : x[i];
        store_turbo<D, VB>(x, bnd, pay, hdr, sub, on);
        continue;
      }
    }
    store_q8(x, pay, hdr, sub, on);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kApThreads) read_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE;
  const bool is_v = L.a.k_out == nullptr || blockIdx.y != 0;
  const DevView& V = is_v ? L.a.v : L.a.k;
  const int sub = threadIdx.x % LPV;
  const Place p = place_of<D>(L, V, sub == 0 && blockIdx.y == 0);
  T* out = static_cast<T*>(is_v ? L.a.v_out : L.a.k_out);
  const int b = V.idx_bits;
  const bool q8 = V.format == TQ_FMT_Q8_0;
  const float* cb = L.a.tab.centroids + (q8 ? 0 : (b - 1) * 8);
  for (int j = 0; j < L.hpt; ++j) {
    const int h = p.h0 + j;
    const bool on = !p.padding && h < p.h1;
    float x[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = 0.f;
    const long long vec = p.vec + (long long)h * V.page_size;
    if (on && p.vec >= 0) {
      const unsigned char* pay = V.payload + vec * V.pay_bytes;
      const unsigned char* hdr = V.header + vec * V.hdr_bytes;
      if (q8) {
        const uint4 u = *reinterpret_cast<const uint4*>(pay + 16 * sub);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        const float delta = __half2float(reinterpret_cast<const __half*>(hdr)[sub / 2]);
#pragma unroll
        for (int i = 0; i < kE; ++i) x[i] = (float)(int8_t)(w[i / 4] >> (8 * (i % 4))) * delta;
      } else {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(pay) + b * sub;
        uint64_t codes = 0;
        for (int k = 0; k < b; ++k) codes |= (uint64_t)src[k] << (16 * k);
        const float n = __half2float(*reinterpret_cast<const __half*>(hdr));
#pragma unroll
        for (int i = 0; i < kE; ++i) x[i] = n * __ldg(cb + ((uint32_t)(codes >> (b * i)) & ((1u << b) - 1u)));
      }
    }
    if (!q8) {  // uniform over the launch's half
      group_wht<D>(x, sub);
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] *= inv_sqrt_dim<D>() * (float)L.a.tab.signs[16 * sub + i];
    }
    if (on) store_row<kE>(out + ((long long)p.t * V.H + h) * D + 16 * sub, x);
  }
}

// Heads per group: up to 8 (place and angles found once for them) while 512 threads are left for every SM.
template <class F>
cudaError_t with_launch(const AppendArgs& a, int d, int H, int sm_count, F run) {
  Launch L{};
  L.a = a;
  const int lpv = d / kE;
  int hpt = 1;
  while (hpt < 8 && hpt * 2 <= H && (long long)a.b.n_tokens * (H / (hpt * 2)) * lpv >= (long long)sm_count * 512) hpt *= 2;
  L.hpt = hpt;
  L.splits = (H + hpt - 1) / hpt;
  const long long groups = (long long)a.b.n_tokens * L.splits;
  const long long grid = (groups * lpv + kApThreads - 1) / kApThreads;
  if (groups * lpv >= (1LL << 31) - kApThreads) return cudaErrorInvalidValue;
  run(L, (unsigned)grid);
  return cudaGetLastError();
}

template <class T, int D>
cudaError_t append_td(const AppendArgs& a, int sm_count, cudaStream_t s) {
  return with_launch(a, D, a.k.H, sm_count, [&](const Launch& L, unsigned grid) {
    const dim3 g(grid, 2);
    switch (a.v.format == TQ_FMT_Q8_0 ? 0 : a.v.idx_bits) {
      case 0: append_kernel<T, D, 0><<<g, kApThreads, 0, s>>>(L); break;
      case 1: append_kernel<T, D, 1><<<g, kApThreads, 0, s>>>(L); break;
      case 2: append_kernel<T, D, 2><<<g, kApThreads, 0, s>>>(L); break;
      default: append_kernel<T, D, 3><<<g, kApThreads, 0, s>>>(L); break;
    }
  });
}

template <class T, int D>
cudaError_t read_td(const AppendArgs& a, int sm_count, cudaStream_t s) {
  return with_launch(a, D, a.k_out ? a.k.H : a.v.H, sm_count, [&](const Launch& L, unsigned grid) {
    read_kernel<T, D><<<dim3(grid, a.k_out && a.v_out ? 2 : 1), kApThreads, 0, s>>>(L);
  });
}

template <class T>
cudaError_t append_t(const AppendArgs& a, int sm_count, cudaStream_t s) {
  if (a.k.d == 64) return append_td<T, 64>(a, sm_count, s);
  if (a.k.d == 128) return append_td<T, 128>(a, sm_count, s);
  return append_td<T, 256>(a, sm_count, s);
}

template <class T>
cudaError_t read_t(const AppendArgs& a, int sm_count, cudaStream_t s) {
  const int d = a.k_out ? a.k.d : a.v.d;
  if (d == 64) return read_td<T, 64>(a, sm_count, s);
  if (d == 128) return read_td<T, 128>(a, sm_count, s);
  return read_td<T, 256>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int dtype, int sm_count, cudaStream_t s) {
  if (dtype == TQ_DTYPE_F32) return append_t<float>(a, sm_count, s);
  if (dtype == TQ_DTYPE_F16) return append_t<__half>(a, sm_count, s);
  return append_t<__nv_bfloat16>(a, sm_count, s);
}

cudaError_t launch_read(const AppendArgs& a, int dtype, int sm_count, cudaStream_t s) {
  if (dtype == TQ_DTYPE_F32) return read_t<float>(a, sm_count, s);
  if (dtype == TQ_DTYPE_F16) return read_t<__half>(a, sm_count, s);
  return read_t<__nv_bfloat16>(a, sm_count, s);
}

}  // namespace tq
