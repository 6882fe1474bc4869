// Appending to and reading from an f8_block cache: e4m3 codes with a power-of-two scale for each 16 tokens and head.
//
// A block takes part in an append as a whole: its scale is the maximum over its new vectors and what it had.  The CTA
// whose rows hold a block's first new token takes the block, K or V, and a warp at a time one of its heads: the up to 16
// vectors go to registers once, 16 coordinates per lane (d / 16 lanes to a vector), are rotated, give the maximum by
// shuffles, and leave as codes.  Where the scale rises and the block holds earlier tokens, their codes are read, brought
// to the new scale and written back; a power of two makes that exact but for values that fall below the smallest normal
// code, so a block can be appended to token by token without losing bits each time.
//
// Bytes: the inputs once, d bytes per vector and a word per block (append), the reverse (read).  4096 tokens of 8 heads of 128 in
// bf16: 16.5 us, where the bytes need 3.8; bound by the chain of dependent loads that finds a block's place, its angles and rows,
// in 1.7 rounds of CTAs (registers: two on an SM).  Reading them back 10.8 us, the same chain.  64 single tokens 6.8 and 5.6.
#include <cuda_fp8.h>

#include "tq_append.cuh"

namespace tq {
namespace {

constexpr int kF8Threads = 256, kF8Warps = kF8Threads / 32;
constexpr uint32_t kTooLarge = 0x6BE00000u;  // 448 * 2^80 as fp32: what is above, infinities and NaN are marked

// As rope_at, with the bits of the angle that a float does not hold: the turn is off by 2^-32 then, and what is left is the
// rounding of sincospi.  A key's code is decided by these, and so is nearly always that of the exact rotation.
__device__ __forceinline__ float2 rope_finely(uint64_t turns, int pos, float m) {
  const int top = (int)((turns * (uint64_t)(long long)pos) >> 32);
  const float f = (float)top, d = (float)(top - (int)f) * (3.14159265f * 0x1p-31f);
  float s, c;
  sincospif(f * 0x1p-31f, &s, &c);
  return make_float2(m * fmaf(-s, d, c), m * fmaf(c, d, s));
}

// A row's place (as Place has it) and the rows [first, end) of its sequence.
struct Row {
  long long vec;
  int pos, first, end;
  bool padding;
};

// The rows [t0, t0 + n) of a CTA, by all its warps.  Up to a row per warp each looks for its own; more rows are mostly of one
// sequence: every warp looks for the first, whose followers in its block lie behind it and in others need a look at the block
// table each, by a lane; the warps share the rest.
__device__ __forceinline__ void find_rows(const AppendArgs& a, const DevView& v, int t0, int n, int warp, int lane, bool report,
                                          Row* rows) {
  int seq, same = 0;
  SeqOf s{};
  auto put = [&](int k, const Place& p) { rows[k] = Row{p.vec, p.pos, s.first, s.first + s.n, p.padding}; };
  if (n > kF8Warps) {
    Place p = find_row(a, v, t0, lane, report && warp == 0, seq, s);
    same = s.ok ? min(n, s.first + s.n - t0) : 1;
    if (warp == 0 && lane < same) {
      const int first = p.pos;
      p.pos += lane;
      if (p.pos / kF8Block == first / kF8Block) {  // (a block lies in one page)
        p.vec = p.vec < 0 ? -1 : p.vec + lane;
      } else {
        p.vec = position_vector(a.b, v, a.layer, seq, p.pos);
        if (p.vec < 0 && report) atomicOr(a.tab.status, kFlagBlockTable);
      }
      put(lane, p);
    }
  }
  for (int k = same + warp; k < n; k += kF8Warps) {
    s = SeqOf{};
    const Place p = find_row(a, v, t0 + k, lane, report, seq, s);
    if (lane == 0) put(k, p);
  }
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ void values4(uint32_t w, float (&x)[4]) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3)));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

template <class T, int D>
__global__ void __launch_bounds__(kF8Threads, D == 256 ? 1 : 2) append_f8_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE, VPP = 32 / LPV, NP = kF8Block / VPP;  // lanes per vector, vectors per pass, passes
  constexpr int ANG = D / 2 + D / 8, W = kE * sizeof(T) / 16;
  __shared__ Row rows[kMaxTc];
  __shared__ __align__(16) float cs[kF8Block][ANG], sn[kF8Block][ANG];
  const AppendArgs& a = L.a;
  const bool is_v = blockIdx.y != 0;
  const DevView& V = is_v ? a.v : a.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LPV, g = lane / LPV;
  const int t0 = blockIdx.x * L.tc, H = V.H, n_tok = min(L.tc, a.b.n_tokens - t0);
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const T* in = static_cast<const T*>(is_v ? a.xv : a.xk) + 16 * sub;
  pdl_launch_dependents();  // the next kernel's start overlaps this one, as this one's the last
  pdl_wait();
  // The rows are on their way to L2 while the first one's sequence is looked for.
  constexpr int LINES = D * (int)sizeof(T) / 128;  // of a vector
  for (int h = warp; h < H; h += kF8Warps) {
    const T* row = static_cast<const T*>(is_v ? a.xv : a.xk) + (long long)t0 * stride + (long long)h * D;
    for (int i = lane; i < n_tok * LINES; i += 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (long long)(i / LINES) * stride + i % LINES * (128 / (int)sizeof(T))));
  }
  const bool many = n_tok > kF8Warps;
  if (!many) {
    find_rows(a, V, t0, n_tok, warp, lane, !is_v, rows);
    __syncthreads();
  }
  const tq_rope_table& R = a.rope;
  const int half = R.rotary_dim / 2;
  const bool turn = !is_v && a.has_rope;
  // Block by block (the CTA's threads alike).  Up to a row per warp the rows have been found side by side; of more, mostly of
  // one sequence, every warp finds the first of a block itself (handed on through shared memory, with two searches of a warp
  // one after the other: 20 us for 4096 tokens of 8 heads of 128, where this takes 16).
  for (int k = 0; k < n_tok;) {
    Row r;
    if (many) {
      SeqOf s{};
      int seq;
      const Place p = find_row(a, V, t0 + k, lane, !is_v && warp == 0, seq, s);
      if (seq == a.b.n_seqs) break;
      r = Row{p.vec, p.pos, s.first, s.first + s.n, p.padding || !s.ok};
    } else {
      r = rows[k];
    }
    struct {  // the slot of the block's first token (head 0), its first new row, the new tokens, the offset of the first
      long long vec;
      int row, n, off;
    } q;
    q.off = r.pos % kF8Block;
    q.vec = r.vec - q.off;
    q.row = t0 + k;
    q.n = min(kF8Block - q.off, r.end - q.row);
    k += many && !r.padding ? q.n : 1;
    if (r.vec < 0 || (q.off && q.row != r.first)) continue;  // no place, or no block begins here
    if (turn) {
      __syncthreads();  // the angles of the block before have been used
      for (int i = tid; i < q.n * half; i += kF8Threads) {
        const int j = i / half, k = i - j * half;
        const float2 f = rope_finely(R.turns[k], a.positions ? __ldg(a.positions + q.row + j) : r.pos + j, R.attn_factor);
        cs[j][angle_at(k)] = f.x;
        sn[j][angle_at(k)] = f.y;
      }
      __syncthreads();
    }
    for (int h = warp; h < H; h += kF8Warps) {
      const long long vec = q.vec + (long long)h * V.page_size;  // a multiple of 16
      uint32_t* word = reinterpret_cast<uint32_t*>(V.header) + vec / kF8Block;
      uint4* pay = reinterpret_cast<uint4*>(V.payload + vec * D) + sub;  // vector i of the block: LPV i further on
      const T* src = in + (long long)q.row * stride + (long long)h * D;
      const uint32_t before = q.off ? *word : 0u;
      uint4 raw[NP][W];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int j = p * VPP + g;
#pragma unroll
        for (int w = 0; w < W; ++w)
          raw[p][w] = j < q.n ? __ldg(reinterpret_cast<const uint4*>(src + (long long)j * stride) + w)
                              : make_uint4(0u, 0u, 0u, 0u);
      }
      float x[NP][kE];
      uint32_t top = 0, marks = 0;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int j = p * VPP + g;
        load_row<kE>(reinterpret_cast<const T*>(raw[p]), x[p]);
        if (p * VPP >= q.n) continue;
        const bool on = j < q.n;
        if (turn)
          turn_part<T, D>(x[p], raw[p], [&] { return src + (long long)j * stride; }, R, cs[on ? j : 0], sn[on ? j : 0],
                          sub, lane, on);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kE; ++i) m = max(m, __float_as_uint(x[p][i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int s = 1; s < LPV; s <<= 1) m = max(m, __shfl_xor_sync(kFull, m, s));
        const bool bad = on && m > kTooLarge;
        if (bad) {
#pragma unroll
          for (int i = 0; i < kE; ++i) x[p][i] = 0.f;
        } else if (on) {
          top = max(top, m);
        }
        const uint32_t b = __ballot_sync(kFull, bad && sub == 0);
#pragma unroll
        for (int i = 0; i < VPP; ++i) marks |= ((b >> (i * LPV)) & 1u) << (p * VPP + i);
      }
#pragma unroll
      for (int s = LPV; s < 32; s <<= 1) top = max(top, __shfl_xor_sync(kFull, top, s));
      // the smallest e with top <= 448 2^e = 1.75 * 2^(e + 8)
      int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), kF8MinExp);
      if (q.off) {
        const int old = min(max((int)(before >> 23) - 127, kF8MinExp), kF8MaxExp);
        if (e > old) {  // (the warp's lanes alike)
          const float f = pow2(old - e < -126 ? -126 : old - e);
          for (int j = g; j < q.off; j += VPP) {
            const uint4 c = pay[j * LPV];
            const uint32_t in4[4] = {c.x, c.y, c.z, c.w};
            uint32_t out4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y[4];
              values4(in4[i], y);
              out4[i] = codes4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
            }
            pay[j * LPV] = make_uint4(out4[0], out4[1], out4[2], out4[3]);
          }
        } else {
          e = old;
        }
        marks = marks << q.off | (before & ((1u << q.off) - 1u));
      }
      const float f = pow2(-e);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int j = p * VPP + g;
        if (j >= q.n) continue;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = codes4(x[p][4 * i] * f, x[p][4 * i + 1] * f, x[p][4 * i + 2] * f, x[p][4 * i + 3] * f);
        pay[(q.off + j) * LPV] = make_uint4(c[0], c[1], c[2], c[3]);
      }
      if (lane == 0) *word = (uint32_t)(e + 127) << 23 | marks;
    }
  }
}

// Rows of f8_block views back in the original space: a group of d / 16 lanes per vector.
template <class T, int D>
__global__ void __launch_bounds__(kF8Threads) read_f8_kernel(const __grid_constant__ Launch L) {
  constexpr int LPV = D / kE, GROUPS = kF8Threads / LPV, NV = 4;
  __shared__ Row rows[kMaxTc];
  const bool is_v = L.a.k_out == nullptr || blockIdx.y != 0;
  const DevView& V = is_v ? L.a.v : L.a.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = tid % LPV;
  const int t0 = blockIdx.x * L.tc, H = V.H;
  const int n_tok = min(L.tc, L.a.b.n_tokens - t0), n_vec = n_tok * H;
  pdl_launch_dependents();
  pdl_wait();
  find_rows(L.a, V, t0, n_tok, warp, lane, blockIdx.y == 0, rows);
  __syncthreads();
  T* out = static_cast<T*>(is_v ? L.a.v_out : L.a.k_out) + (long long)t0 * H * D + 16 * sub;
  for (int v0 = tid / LPV; v0 < n_vec; v0 += NV * GROUPS) {
    uint4 c[NV];
    uint32_t w[NV];
    bool padding[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = v0 + u * GROUPS, t = v / H, h = v - t * H;
      const Row p = v < n_vec ? rows[t] : Row{-1, 0, 0, 0, true};
      padding[u] = p.padding;
      c[u] = make_uint4(0u, 0u, 0u, 0u);
      w[u] = 0u;
      if (p.vec >= 0) {
        const long long vec = p.vec + (long long)h * V.page_size;
        c[u] = *(reinterpret_cast<const uint4*>(V.payload + vec * D) + sub);
        w[u] = reinterpret_cast<const uint32_t*>(V.header)[vec / kF8Block];
        w[u] = (w[u] >> (vec % kF8Block)) & 1u ? 0x7FC00000u : w[u] & 0xFFFF0000u;
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (padding[u]) continue;
      const uint32_t in4[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      float x[kE];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4];
        values4(in4[i], y);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[4 * i + k] = y[k] * __uint_as_float(w[u]);
      }
      store_row<kE>(out + (long long)(v0 + u * GROUPS) * D, x);
    }
  }
}

template <class T, int D>
cudaError_t append_td(const AppendArgs& a, int sm_count, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const cudaError_t last = with_launch(a, sm_count, [&](const Launch& L, unsigned grid) {
    e = launch_pdl(append_f8_kernel<T, D>, dim3(grid, 2), dim3(kF8Threads), 0, s, L);
  });
  return e == cudaSuccess ? last : e;
}

template <class T, int D>
cudaError_t read_td(const AppendArgs& a, int sm_count, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const cudaError_t last = with_launch(a, sm_count, [&](const Launch& L, unsigned grid) {
    e = launch_pdl(read_f8_kernel<T, D>, dim3(grid, a.k_out && a.v_out ? 2 : 1), dim3(kF8Threads), 0, s, L);
  });
  return e == cudaSuccess ? last : e;
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

cudaError_t launch_append_f8(const AppendArgs& a, int dtype, int sm_count, cudaStream_t s) {
  if (dtype == TQ_DTYPE_F32) return append_t<float>(a, sm_count, s);
  if (dtype == TQ_DTYPE_F16) return append_t<__half>(a, sm_count, s);
  return append_t<__nv_bfloat16>(a, sm_count, s);
}

cudaError_t launch_read_f8(const AppendArgs& a, int dtype, int sm_count, cudaStream_t s) {
  if (dtype == TQ_DTYPE_F32) return read_t<float>(a, sm_count, s);
  if (dtype == TQ_DTYPE_F16) return read_t<__half>(a, sm_count, s);
  return read_t<__nv_bfloat16>(a, sm_count, s);
}

}  // namespace tq
