// Appending a ragged batch's keys (rotated on the way) and values to the paged cache, and reading rows back.
//
// A CTA takes `tc` consecutive tokens, K or V.  A group of d / 16 lanes holds one vector, 16 consecutive coordinates per
// lane; its first vector is asked for before anything else.  Meanwhile one warp per token finds the token's sequence and
// place in the cache, and the CTA computes the rotation's angles once per token for all its heads (16 sincospi per lane
// and vector instead made a 4096-token chunk of 8 heads of 128 take 23 us; it takes 18, of which the bytes need 4: bound by
// the chain of dependent loads that finds a place, and its two barriers).  From the load to the stored bytes a vector stays
// in registers: the q8_0 scale of a 32-block is shared by two lanes, the turbo rotation runs four butterfly stages
// in a lane and log2(d / 16) across the group.  Bytes: both inputs once, the stored vectors once (append), the reverse
// (read: 11 us for the rows of that chunk).
#include "tq_append.cuh"

namespace tq {
namespace {

constexpr int kApThreads = 256;

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

// Stores a vector as q8_0: 16 code bytes per lane, a scale per pair of lanes.  The codes are round(x / delta), halves away
// from zero, as tq_encode_kv has them (the IEEE quotient, then roundf).  x * (1 / delta) is within 127 * 2^-21 of the
// quotient, so its nearest integer is the code unless it lies that near a half: only then are the 16 quotients taken.
// A scale that fp16 does not hold is stored as infinite, with codes of 0: every reader then finds NaN in the block, and not
// infinities beside them.
__device__ __forceinline__ void store_q8(const float (&x)[kE], unsigned char* pay, unsigned char* hdr, int sub,
                                         bool keep) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  const float delta = __fdiv_rn(amax, 127.0f);
  if (!keep) return;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (delta > 0.f && delta < 65520.f) {  // (65520 and more round to infinity)
    const float inv = __fdiv_rn(1.0f, delta), magic = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are the integer
    bool near = !(inv < 3.0e38f);  // (a subnormal delta: its reciprocal is not finite)
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float t = x[i] * inv, r = t + magic;
      near |= !(fabsf(t - (r - magic)) < 0.4999f);  // also NaN
      w[i / 4] |= (__float_as_uint(r) & 255u) << (8 * (i % 4));
    }
    if (near) {
      w[0] = w[1] = w[2] = w[3] = 0u;
#pragma unroll
      for (int i = 0; i < kE; ++i)
        w[i / 4] |= (uint32_t)(uint8_t)(int8_t)(int)roundf(__fdiv_rn(x[i], delta)) << (8 * (i % 4));
    }
  }
  *reinterpret_cast<uint4*>(pay + 16 * sub) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((sub & 1) == 0) reinterpret_cast<__half*>(hdr)[sub / 2] = __float2half_rn(delta);
}

// Stores a vector as turbo-MSE codes of B bits: n = |x|, y = H diag(s) x / n, the count of boundaries <= y.  A coordinate
// nearer to a boundary than fp32 butterflies can tell (2^-18 of a standard deviation: about one vector in a thousand has
// one) is summed again in fp64, the group together, and compared as sum_j +-x_j >= boundary sqrt(D) |x|: a code on the
// wrong side would move it by a whole step.
template <int D, int B>
__device__ __forceinline__ void store_turbo(float (&x)[kE], const float (&bnd)[7], unsigned char* pay,
                                            unsigned char* hdr, int sub, bool keep) {
  constexpr int LPV = D / kE;
  float raw[kE], ss = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    raw[i] = x[i];
    ss = fmaf(x[i], x[i], ss);
  }
#pragma unroll
  for (int m = 1; m < LPV; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
  group_wht<D>(x, sub);
  const float n = sqrtf(ss);
  const float f = n > 0.f ? __fdiv_rn(inv_sqrt_dim<D>(), n) : 0.f;
  constexpr float kBand = inv_sqrt_dim<D>() * 0x1p-18f;
  uint64_t codes = 0;  // 16 B <= 48 bits
  uint32_t near = 0;
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const float y = x[i] * f;
    uint32_t c = 0;
    bool at = false;
#pragma unroll
    for (int k = 0; k < (1 << B) - 1; ++k) {
      c += y >= bnd[k] ? 1u : 0u;
      at |= fabsf(y - bnd[k]) < kBand;
    }
    codes |= (uint64_t)c << (B * i);
    near |= (at ? 1u : 0u) << i;
  }
  if (!keep || n == 0.f) near = 0;
  if (__any_sync(kFull, near != 0)) {
    double zz = 0.0;
#pragma unroll 1
    for (int i = 0; i < kE; ++i) zz = fma((double)raw[i], (double)raw[i], zz);
#pragma unroll 1
    for (int m = 1; m < LPV; m <<= 1) zz += __shfl_xor_sync(kFull, zz, m);
    zz *= D;
    double r = rsqrtf((float)zz);  // 1 / sqrt(D zz), two Newton steps
    r *= 1.5 - 0.5 * zz * r * r;
    r *= 1.5 - 0.5 * zz * r * r;
    const int lane = threadIdx.x & 31, base = lane & ~(LPV - 1);
    for (;;) {  // one coordinate of every group at a time
      const uint32_t have = __ballot_sync(kFull, near != 0);
      if (!have) break;
      const uint32_t mine = (have >> base) & (LPV == 32 ? 0xFFFFFFFFu : (1u << LPV) - 1u);
      const int owner = mine ? __ffs(mine) - 1 : 0;  // lane of the group
      const int i = near ? __ffs(near) - 1 : 0;
      const int e = 16 * owner + __shfl_sync(kFull, i, base + owner);
      double z = 0.0;
#pragma unroll 1
      for (int j = 0; j < kE; ++j) z += __popc(e & (16 * sub + j)) & 1 ? -(double)raw[j] : (double)raw[j];
#pragma unroll 1
      for (int m = 1; m < LPV; m <<= 1) z += __shfl_xor_sync(kFull, z, m);
      if (mine && sub == owner) {
        uint32_t c = 0;
        for (int k = 0; k < (1 << B) - 1; ++k) c += z * r >= (double)bnd[k] ? 1u : 0u;
        codes = (codes & ~((uint64_t)((1 << B) - 1) << (B * i))) | ((uint64_t)c << (B * i));
        near &= near - 1;
      }
    }
  }
  if (!keep) return;
  uint16_t* dst = reinterpret_cast<uint16_t*>(pay) + B * sub;
#pragma unroll
  for (int k = 0; k < B; ++k) dst[k] = (uint16_t)(codes >> (16 * k));
  if (sub == 0) *reinterpret_cast<__half*>(hdr) = __float2half_rn(n);
}

template <class T, int D, int VB>  // VB: 0 q8_0 values, else turbo-MSE index bits
__global__ void __launch_bounds__(kApThreads, VB == 0 ? 4 : 2) append_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE, GROUPS = kApThreads / LPV, ANG = D / 2 + D / 8;
  constexpr int NV = 2, W = kE * sizeof(T) / 16;  // vectors in flight, their 16-byte words
  __shared__ Place place[kMaxTc];
  __shared__ __align__(16) float cs[kMaxTc][ANG], sn[kMaxTc][ANG];
  const bool is_v = blockIdx.y != 0;
  const DevView& V = is_v ? L.a.v : L.a.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = tid % LPV;
  const int t0 = blockIdx.x * L.tc, H = V.H;
  const int n_tok = min(L.tc, L.a.b.n_tokens - t0), n_vec = n_tok * H;
  const long long stride = is_v ? L.a.v_stride : L.a.k_stride;
  const T* in = static_cast<const T*>(is_v ? L.a.xv : L.a.xk) + (long long)t0 * stride + 16 * sub;
  const int g = tid / LPV;
  uint4 raw[NV][W];
  auto fetch = [&](int v0) {  // vectors v0 + g, v0 + GROUPS + g of the CTA: vector v is token v / H, head v % H
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = v0 + u * GROUPS + g, t = v / H, h = v - t * H;
      const uint4* src = reinterpret_cast<const uint4*>(in + (long long)t * stride + (long long)h * D);
#pragma unroll
      for (int k = 0; k < W; ++k) raw[u][k] = v < n_vec ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(0);

  for (int k = warp; k < n_tok; k += kApThreads / 32) {
    const Place p = find_place(L.a, V, t0 + k, lane, !is_v);
    if (lane == 0) place[k] = p;
  }
  __syncthreads();
  const tq_rope_table& R = L.a.rope;
  const int half = R.rotary_dim / 2;
  const bool turn = !is_v && L.a.has_rope;
  if (turn) {
    for (int i = tid; i < n_tok * half; i += kApThreads) {
      const int k = i / half, p = i - k * half;
      const int pos = L.a.positions ? __ldg(L.a.positions + t0 + k) : place[k].pos;
      const float2 f = rope_at(R.turns[p], pos, R.attn_factor);
      cs[k][angle_at(p)] = f.x;
      sn[k][angle_at(p)] = f.y;
    }
    __syncthreads();
  }
  float bnd[7];
  uint32_t neg = 0;  // sign flips of the lane's coordinates
  if constexpr (VB > 0) {
    if (is_v) {
#pragma unroll
      for (int k = 0; k < 7; ++k) bnd[k] = k < (1 << VB) - 1 ? L.a.tab.boundaries[(VB - 1) * 7 + k] : 0.f;
#pragma unroll
      for (int i = 0; i < kE; ++i) neg |= (L.a.tab.signs[16 * sub + i] < 0 ? 1u : 0u) << i;
    }
  }
  // the trip counts are the CTA's: the shuffles inside are warp-wide
  for (int v0 = 0; v0 < n_vec; v0 += NV * GROUPS) {
    if (v0 > 0) fetch(v0);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (v0 + u * GROUPS >= n_vec) break;
      const int v = v0 + u * GROUPS + g, t = v / H, h = v - t * H;
      const Place p = v < n_vec ? place[t] : Place{-1, 0, true};
      const bool on = p.vec >= 0;
      const int tt = on ? t : 0;
      float x[kE];
      load_row<kE>(reinterpret_cast<const T*>(raw[u]), x);
      if (turn)
        turn_part<T, D>(x, raw[u], [&] { return in + (long long)t * stride + (long long)h * D; }, R, cs[tt], sn[tt], sub,
                        lane, on);
      const long long vec = p.vec + (long long)h * V.page_size;
      unsigned char* pay = V.payload + vec * V.pay_bytes;
      unsigned char* hdr = V.header + vec * V.hdr_bytes;
      if (VB > 0 && is_v) {
        if constexpr (VB > 0) {
#pragma unroll
          for (int i = 0; i < kE; ++i) x[i] = (neg >> i) & 1u ? -x[i] : x[i];
          store_turbo<D, VB>(x, bnd, pay, hdr, sub, on);
        }
      } else {
        store_q8(x, pay, hdr, sub, on);
      }
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kApThreads) read_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE, GROUPS = kApThreads / LPV;
  __shared__ Place place[kMaxTc];
  const bool is_v = L.a.k_out == nullptr || blockIdx.y != 0;
  const DevView& V = is_v ? L.a.v : L.a.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = tid % LPV;
  const int t0 = blockIdx.x * L.tc, H = V.H;
  const int n_tok = min(L.tc, L.a.b.n_tokens - t0), n_vec = n_tok * H;
  for (int k = warp; k < n_tok; k += kApThreads / 32) {
    const Place p = find_place(L.a, V, t0 + k, lane, blockIdx.y == 0);
    if (lane == 0) place[k] = p;
  }
  __syncthreads();
  T* out = static_cast<T*>(is_v ? L.a.v_out : L.a.k_out);
  const int b = V.idx_bits;
  const bool q8 = V.format == TQ_FMT_Q8_0;
  const float* cb = L.a.tab.centroids + (q8 ? 0 : (b - 1) * 8);
  for (int v0 = 0; v0 < n_vec; v0 += GROUPS) {
    const int v = v0 + tid / LPV, t = v / H, h = v - t * H;
    const bool in_range = v < n_vec;
    const Place p = in_range ? place[t] : Place{-1, 0, true};
    float x[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = 0.f;
    if (p.vec >= 0) {
      const long long vec = p.vec + (long long)h * V.page_size;
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
        float n = __half2float(*reinterpret_cast<const __half*>(hdr));
        n += n - n;  // an infinite norm is NaN in every coordinate (its levels alone could add up to infinities)
#pragma unroll
        for (int i = 0; i < kE; ++i) x[i] = n * __ldg(cb + ((uint32_t)(codes >> (b * i)) & ((1u << b) - 1u)));
      }
    }
    if (!q8) {  // uniform over the CTA
      group_wht<D>(x, sub);
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] *= inv_sqrt_dim<D>() * (float)L.a.tab.signs[16 * sub + i];
    }
    if (in_range && !p.padding) store_row<kE>(out + ((long long)(t0 + t) * H + h) * D + 16 * sub, x);
  }
}

template <class T, int D>
cudaError_t append_td(const AppendArgs& a, int sm_count, cudaStream_t s) {
  return with_launch(a, sm_count, [&](const Launch& L, unsigned grid) {
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
  return with_launch(a, sm_count, [&](const Launch& L, unsigned grid) {
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
