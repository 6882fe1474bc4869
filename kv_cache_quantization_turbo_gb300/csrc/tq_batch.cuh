// Device helpers of the serving step's kernels: element types, the ragged batch, the page of a token, the rotation.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_device.cuh"

namespace tq {

// Sequence b of a batch: its rows [first, first + n) and its length; ok is false where the device values break the
// bounds of the call (documented at tq_batch).
struct SeqOf {
  int first, n, len;
  bool ok;
};

__device__ __forceinline__ SeqOf seq_of(const DevBatch& b, int i) {
  SeqOf s;
  const int c0 = __ldg(b.cu + i), c1 = __ldg(b.cu + i + 1);
  s.first = c0;
  s.len = __ldg(b.seq_lens + i);
  // the differences below cannot overflow once the ends are in [0, n_tokens]
  s.ok = c0 >= 0 && c1 >= c0 && c1 <= b.n_tokens && s.len >= 0 && s.len <= b.max_ctx && c1 - c0 <= b.max_tokens &&
         c1 - c0 <= s.len;
  s.n = s.ok ? c1 - c0 : 0;
  return s;
}

// The sequence that row t belongs to: the first b with cu[b + 1] > t; n_seqs for a padding row.
__device__ __forceinline__ int seq_of_row(const DevBatch& b, int t) {
  int lo = 0, hi = b.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(b.cu + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < b.n_seqs && __ldg(b.cu + lo) <= t ? lo : b.n_seqs;
}

// Index of the vector (layer, head 0) of a sequence's position, or -1 where its page is out of range; consecutive
// heads are page_size vectors apart.
__device__ __forceinline__ long long position_vector(const DevBatch& b, const DevView& v, int layer, int seq, int pos) {
  const int lp = pos / v.page_size;
  long long page = seq;
  if (b.block_table) page = lp < b.max_blocks ? __ldg(b.block_table + (long long)seq * b.max_blocks + lp) : -1;
  if (page < 0 || page >= v.num_pages) return -1;
  return ((long long)layer * v.num_pages + page) * v.H * v.page_size + (pos - lp * v.page_size);
}

// The end of the first s keys from `first` on, which a window does not hide.
__device__ __forceinline__ int sink_end(int first, int s) { return first > 0x7FFFFFFF - s ? 0x7FFFFFFF : first + s; }

// cos and sin of pair angle `turns` (2^-64 turns per position) at a position, times m.  The product wraps modulo one
// turn exactly; its top 32 bits, as a signed fraction of half a turn, are what sincospi takes (error below 2^-25 half
// turns, 1e-7 in the results).
__device__ __forceinline__ float2 rope_at(uint64_t turns, int pos, float m) {
  const int top = (int)((turns * (uint64_t)(long long)pos) >> 32);
  float s, c;
  sincospif((float)top * 0x1p-31f, &s, &c);
  return make_float2(m * c, m * s);
}

// N consecutive elements as fp32 (vector accesses of up to 16 bytes; p aligned to min(16, N * element) bytes).
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p[i];
  }
}

__device__ __forceinline__ float2 widen(uint32_t w, const __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 widen(uint32_t w, const __nv_bfloat16*) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t narrow(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }

template <int N, class T>
__device__ __forceinline__ void load_row(const T* p, float (&x)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = widen(w[k], p);
        x[i + 2 * k] = f.x; x[i + 2 * k + 1] = f.y;
      }
    }
  } else if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 f = widen(v.x, p), g = widen(v.y, p);
    x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
  } else if constexpr (N == 2) {
    const float2 f = widen(*reinterpret_cast<const uint32_t*>(p), p);
    x[0] = f.x; x[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_float(p[i]);
  }
}

template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&x)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = x[i];
  }
}

template <int N, class T>
__device__ __forceinline__ void store_row(T* p, const float (&x)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(narrow(x[i], x[i + 1], p), narrow(x[i + 2], x[i + 3], p),
                                                    narrow(x[i + 4], x[i + 5], p), narrow(x[i + 6], x[i + 7], p));
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(narrow(x[0], x[1], p), narrow(x[2], x[3], p));
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint32_t*>(p) = narrow(x[0], x[1], p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) from_float(p + i, x[i]);
  }
}

}  // namespace tq
