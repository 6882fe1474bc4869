// Chunk attention of entries of few rows (decode, short speculative steps).
//
// A tensor instruction of tcgen05 takes as long for 4 rows as for 128, and a tile's way through its two buffers, five
// roles and their barriers is what a decode step then waits for.  Here a warp works alone: it takes every NW-th slice of 16
// keys of its CTA's range, copies the next slices' codes and scales asynchronously to a ring of its own, turns codes into
// fp16 fragments in registers, and keeps its own softmax reference, sum and output; no barrier until the range ends.  The
// products are the warp-wide m16n8k16 ones (fp16 operands, fp32 sums):
//   S^T = K Q^T: M = 16 keys, N = 8 rows; the codes are integers that fp16 holds, the scale of a block of 32 goes to its sum
//     in fp32, so K is not rounded; what fp16 leaves of fp32 queries has products of its own.  A lane holds 8 coordinates of a block at a time: the contraction index is permuted,
//     alike for K and Q.
//   O^T = V^T P^T: M = 16 coordinates, N = 8 rows; a lane pairs the codes of two keys by byte permutes, and P^T is S^T's
//     accumulators with two 8 x 8 transposes.  A lane's columns are the same rows of Q in both products.
// The ranges, the join of entries that several CTAs share and the meaning of every mask are those of tq_chunk_tc.cuh;
// weights are taken against a reference that is raised only when a weight would pass 2^15.
//
// What bounds it.  64 sequences of 1K to 16K tokens, 8 KV heads of 128, 4 rows: 147 us for 0.87 GB, 5.9 TB/s, 87 % of the
// copy bandwidth, at 64 % of the instruction slots (511 instructions per slice, of which 180 turn codes into fp16).  Keys as
// the right operand, 8 of 16 rows idle, took 170 us; scales multiplied into K's fragments 149 us, and rounded K: an error of
// 1.3e-3 instead of 3.6e-4.  Turbo values: more instructions (a lookup by byte permutes) for fewer bytes, 149 us for 48 such
// sequences, bound by the instruction slots.  One token at 32K: 20 us after the plan, of which the range's 7 slices per
// warp take 9 (instruction slots), finding the range, the first copies and Q 5, the join of 38 shares 5.
#pragma once

#include <type_traits>

#include "tq_chunk_tc.cuh"
#include "tq_warp_mma.cuh"

namespace tq {
namespace ck {
namespace few {

constexpr int SK = 16;     // keys of a slice
constexpr float kMaxExp = 15.f;

// Two CTAs per SM hide each other's starts and ends of ranges.
template <int D, int NT, int VB>  // VB: 0 q8_0 values, else turbo-MSE index bits
struct Few {
  static constexpr int NW = D == 256 || NT > 1 ? 6 : 8;  // warps of a CTA: as many as have the registers
  static constexpr int VP = VB == 0 ? D : D * VB / 8;    // payload and header bytes of a V vector
  static constexpr int VH = VB == 0 ? D / 16 : 2;
  static constexpr int k = 0, v = SK * D;                // parts of a slice
  static constexpr int ks = v + SK * VP, vs = ks + SK * D / 16;
  static constexpr int slice = vs + SK * VH;
  static constexpr int most = 108 * 1024 / (NW * slice);
  static constexpr int NS = most > 8 ? 8 : most;         // slices of a warp's ring
  static constexpr int ring = NW * NS * slice;
  static constexpr int items = ring;                     // Item [2]
  static constexpr int row = items + 2 * 128;            // Row [16]
  static constexpr int ml = row + 16 * 32;               // float2 [NW][16]
  static constexpr int miss = ml + NW * 16 * 8;          // uint32 [NW][8]: keys of the slice whose page is out of range
  static constexpr int tab = miss + NW * 8 * 4;          // uint32 [4]: the V codebook in fp16, low bytes, high bytes
  static constexpr int flag = tab + 16;
  static constexpr int walk = flag + 16;                 // Items<D>
  static constexpr int ql = walk + 64;                   // uint4 [NT][D / 32][32 lanes]: what fp16 leaves of fp32 queries
  static constexpr int total = ql + NT * D * 16;
  static constexpr int OS = D + 4;                       // floats of a row of a warp's O (in the ring, once it is read)
  static constexpr int mo = NW * 8 * NT * OS * 4, sh = 8 * NT * 320 * 8;  // the warps' O, or the weights of 320 shares
  static constexpr int fin = mo > sh ? mo : sh;          // behind them, float [8 NT][D]: joined rows before their transform
  static_assert(slice % 32 == 0 && ring % 16 == 0, "alignment");
  static_assert(NS >= 2 && fin + 8 * NT * D * 4 + NW * 32 * 16 <= ring, "merge area");
  static_assert(2 * (total + 1024) <= 228 * 1024, "two CTAs per SM");
};

// Chunk of 16 bytes of a row, so that the lanes' reads of the products' operands meet different banks: a K read takes 32
// bytes of each of four keys, a V read two chunks of every second key.
template <int D>
__device__ __forceinline__ int k_at(int key, int chunk) {
  return key * D + ((D == 64 ? chunk ^ (key & 2) : chunk ^ ((key & 3) << 1)) << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int key, int chunk) {
  return key * D + ((D == 64 ? chunk ^ ((key >> 1) & 3) : chunk ^ (key & 6)) << 4);
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {  // an 8 x 8 matrix of fp16, a pair per lane
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  if constexpr (N == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
  else if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}

struct Row {
  int lo, hi, pos;  // the keys [lo, hi) it sees; its position
  float slope;      // in log2 units
  float sl;         // what its scores are multiplied by, in log2 units
  int pad[3];
};

struct Spot {
  int page, off;
};

// Page and offset of a key, -1 where the key is not wanted.  pages: the sequence's row of the block table, if there is
// one.  inv: floor((2^32 - 1) / page_size), with which the quotient is at most one too small.
__device__ __forceinline__ Spot spot_of(const Args& a, const int32_t* pages, int seq, int j, int end, uint32_t inv) {
  Spot s{-1, 0};
  if (j < end) {
    if (!pages) return Spot{seq, j};
    const int ps = a.c.k.page_size;
    int lp = (int)__umulhi((uint32_t)j, inv);
    s.off = j - lp * ps;
    if (s.off >= ps) {
      ++lp;
      s.off -= ps;
    }
    if (lp < a.c.b.max_blocks) s.page = __ldg(pages + lp);
  }
  return s;
}

// A lane's part of a row of Q as fragments of the right operand, times a power of two that brings the row's largest magnitude
// to [1, 2); returns that power's inverse.  16-bit queries are exact in fp16 then, down to 2^-24 of the largest.  Of fp32
// ones rest takes what the rounding leaves, in fp16 again (22 bits in all), which a second product adds to the scores: rest
// [D / 32] at a stride of 32 lanes, null where another warp writes it.  (Without it 64 decode rows of fp32 queries are off by
// 5.5e-4, 2.7e-3 at most, with it by 3.5e-4 and 1.7e-3, as fp16 ones are; it costs 2 us of 164, and its branch 1 % elsewhere.)
template <int D, class T>
__device__ __forceinline__ float load_q(const Args& a, const T* src, bool valid, int t, uint32_t (&f)[D / 16][2], uint4* rest) {
  uint32_t top = 0;
  float x[D / 32][8];  // coordinates 8 t .. 8 t + 7 of every 32
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    if (valid) {
      load_row<8>(src + 32 * i + 8 * t, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7FFFFFFFu);
  }
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  top = max(top, __shfl_xor_sync(kFull, top, 2));
  uint32_t ex = min(max(top >> 23, 1u), 253u);
  if (top >= 0x7F800000u) ex = 127u;  // infinite or NaN: as it is
  const float m = a.q_sign * __uint_as_float((254u - ex) << 23);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      f[2 * i + w][0] = narrow(x[i][4 * w] * m, x[i][4 * w + 1] * m, (const __half*)nullptr);
      f[2 * i + w][1] = narrow(x[i][4 * w + 2] * m, x[i][4 * w + 3] * m, (const __half*)nullptr);
    }
  if constexpr (sizeof(T) == 4) {
    if (rest) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t r[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 h = widen(f[2 * i + w / 2][w % 2], (const __half*)nullptr);
          r[w] = narrow(fmaf(x[i][2 * w], m, -h.x), fmaf(x[i][2 * w + 1], m, -h.y), (const __half*)nullptr);
        }
        rest[32 * i] = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
  }
  return __uint_as_float(ex << 23);
}

template <int D>
__device__ __forceinline__ float load_q_any(const Args& a, long long at, bool valid, int t, uint32_t (&f)[D / 16][2],
                                            uint4* rest) {
  if (a.c.q_dtype == TQ_DTYPE_F32) return load_q<D>(a, static_cast<const float*>(a.c.q) + at, valid, t, f, rest);
  if (a.c.q_dtype == TQ_DTYPE_F16) return load_q<D>(a, static_cast<const __half*>(a.c.q) + at, valid, t, f, rest);
  return load_q<D>(a, static_cast<const __nv_bfloat16*>(a.c.q) + at, valid, t, f, rest);
}

// Clamps N scales as the large kernel does (a turbo norm is left as it is); true where one is not finite (it becomes 0).
static __device__ __noinline__ bool mend_scales(__half* s, int n, bool clamp) {
  bool poison = false;
  for (int i = 0; i < n; ++i) {
    const uint32_t h = __half_as_ushort(s[i]);
    if (not_finite(h)) {
      poison = true;
      s[i] = __ushort_as_half(0);
    } else if (clamp && (h & 0x7FFFu) > 0x5FFEu) {
      s[i] = __ushort_as_half((unsigned short)((h & 0x8000u) | 0x5FFEu));  // 511.5
    }
  }
  return poison;
}

// Codes 0-3 of VB bits to the nibbles of a byte permute's selector.
template <int VB>
__device__ __forceinline__ uint32_t nibbles(uint32_t x) {
  if constexpr (VB == 1) {
    x = (x | x << 6) & 0x0303u;
    return (x | x << 3) & 0x1111u;
  } else if constexpr (VB == 2) {
    x = (x | x << 4) & 0x0F0Fu;
    return (x | x << 2) & 0x3333u;
  } else {
    x = (x & 0x3Fu) | (x << 2 & 0x3F00u);
    return (x & 0x0707u) | (x << 1 & 0x7070u);
  }
}

// Four key-paired coordinates of V (fp16 pairs) from the codes of keys a and b; sel: their nibbles.
__device__ __forceinline__ void turbo_pairs(const uint32_t (&tab)[4], uint32_t sa, uint32_t sb, uint32_t scale,
                                            uint32_t (&y)[4]) {
  const uint32_t la = __byte_perm(tab[0], tab[1], sa), ha = __byte_perm(tab[2], tab[3], sa);
  const uint32_t lb = __byte_perm(tab[0], tab[1], sb), hb = __byte_perm(tab[2], tab[3], sb);
  const uint32_t a0 = __byte_perm(la, ha, 0x5140), a1 = __byte_perm(la, ha, 0x7362);
  const uint32_t b0 = __byte_perm(lb, hb, 0x5140), b1 = __byte_perm(lb, hb, 0x7362);
  y[0] = mul_h2(__byte_perm(a0, b0, 0x5410), scale);
  y[1] = mul_h2(__byte_perm(a0, b0, 0x7632), scale);
  y[2] = mul_h2(__byte_perm(a1, b1, 0x5410), scale);
  y[3] = mul_h2(__byte_perm(a1, b1, 0x7632), scale);
}

template <int D, int NT, int VB>
__global__ void __launch_bounds__(Few<D, NT, VB>::NW * 32, 2) few_kernel(const __grid_constant__ Args a) {
  using F = Few<D, NT, VB>;
  constexpr int NS = F::NS, NW = F::NW;
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  Item* items = reinterpret_cast<Item*>(sm + F::items);
  unsigned char* ring = sm + warp * NS * F::slice;
  const uint32_t ring_s = tc::smem_addr(ring);
  uint32_t* miss = reinterpret_cast<uint32_t*>(sm + F::miss) + warp * 8;
  float2* ml = reinterpret_cast<float2*>(sm + F::ml);
  Row* row_of = reinterpret_cast<Row*>(sm + F::row);
  int* flag = reinterpret_cast<int*>(sm + F::flag);
  uint4* q_rest = reinterpret_cast<uint4*>(sm + F::ql);
  const bool fine = a.c.q_dtype == TQ_DTYPE_F32;
  const DevView &K = a.c.k, &V = a.c.v;
  const bool mods = a.c.softcap > 0.f || a.c.slopes != nullptr;
  // where the 16 keys of a slice, which begin at a multiple of 16, are consecutive vectors
  const bool runs = !a.c.b.block_table || K.page_size % SK == 0;
  const uint32_t inv = 0xFFFFFFFFu / (uint32_t)K.page_size;
  uint32_t tab[4] = {0u, 0u, 0u, 0u};
  if constexpr (VB > 0) {
    if (tid < 4) {  // word tid: low (0, 1) or high (2, 3) bytes of four levels
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 4 * (tid & 1) + i;
        const float x = n < (1 << VB) ? a.c.tab.f16_scale[VB - 1] * a.c.tab.centroids[(VB - 1) * 8 + n] : 0.f;
        const uint32_t h = __half_as_ushort(__float2half_rn(x));
        w |= ((tid & 2 ? h >> 8 : h) & 0xFFu) << (8 * i);
      }
      reinterpret_cast<uint32_t*>(sm + F::tab)[tid] = w;
    }
  }
  pdl_wait();  // the plan
  Items<D>* walk = reinterpret_cast<Items<D>*>(sm + F::walk);
  static_assert(sizeof(Items<D>) <= 64, "items");
  if (tid == 0) {
    walk->start(a);
    walk->next(a, items[0]);
  }
  __syncthreads();
  if constexpr (VB > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tab[i] = reinterpret_cast<const uint32_t*>(sm + F::tab)[i];
  }
  for (int n_item = 0;; ++n_item) {
    const Item& it = items[n_item & 1];
    if (it.kind == 0) break;
    const int G = a.c.G, rows = it.rows;
    auto out_of = [&](int r) {  // where row r's result goes
      const int row = it.row0 + r, ti = row / G;
      return ((long long)(it.tok0 + ti) * a.c.n_q_heads + it.kvh * G + (row - ti * G)) * D;
    };
    auto next_item = [&]() {
      if (tid == 0) walk->next(a, items[(n_item + 1) & 1]);
    };
    if (it.kind == 2) {
      next_item();
      for (int i = tid; i < rows * (D / 8); i += NW * 32) {
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store8(a.c.out, a.c.out_dtype, out_of(i / (D / 8)) + 8 * (i % (D / 8)), z);
      }
      __syncthreads();
      continue;
    }
    constexpr int BN = Shape<D>::BN;
    const int j0 = max(it.tile * BN, it.lo) & ~(SK - 1), end = min((it.tile + it.n) * BN, it.hi);
    const int seq = it.seq, low = it.lo;
    const int32_t* pages = a.c.b.block_table ? a.c.b.block_table + (long long)seq * a.c.b.max_blocks : nullptr;
    // payload bytes of a page; where the layer's bytes of the head begin
    const long long page_b = (long long)K.H * K.page_size * D;
    const long long first_b = (long long)a.c.layer * K.num_pages * page_b + (long long)it.kvh * K.page_size * D;
    // Asks for the slice that begins at key n0 into stage st; sp: the place of key lane % 16 of it, or (runs) of its first
    // key.  Returns the norm of V's key lane % 16 (turbo values), which goes to the stage later.
    bool missed = false;  // some slice of this warp has keys whose page is out of range: miss[] is valid
    auto issue = [&](int n0, int st, const Spot& sp) {
      uint16_t norm = 0;
      if (n0 < end) {
        const bool there = sp.page >= 0 && sp.page < K.num_pages;
        const uint32_t base = ring_s + st * F::slice;
        constexpr int LPK = D / 16, KPI = 32 / LPK;  // lanes of a key, keys of a copy
        const int kl = lane / LPK, c = lane % LPK;
        const long long at0 = there ? first_b + (uint32_t)sp.page * page_b + (long long)sp.off * D : 0;  // of K's payload
        auto mark = [&](uint32_t off) {
          if (off && !missed) {
            missed = true;
            if (lane < NS) miss[lane] = 0u;
            __syncwarp();
          }
          if (missed && lane == 0) {
            miss[st] = off;
            if (off) atomicOr(a.c.tab.status, kFlagBlockTable);
          }
        };
        const int c0 = max(low - n0, 0), c1 = min(end - n0, SK);  // the keys [c0, c1) are wanted
        if (runs) {
          const unsigned char *pk = K.payload + at0 + 16 * lane, *hk = K.header + (at0 >> 4) + 4 * lane;
          auto go = [&](auto on) {  // on(key): the key is there
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              copy_async<16>(base + F::k + k_at<D>(i * KPI + kl, c), pk + 512 * i, on(i * KPI + kl));
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
              const int at = 4 * lane + 128 * i;
              if (D >= 128 || lane < D / 4) copy_async<4>(base + F::ks + at, hk + 128 * i, on(at / (D / 16)));
            }
            if constexpr (VB == 0) {
              const unsigned char *pv = V.payload + at0 + 16 * lane, *hv = V.header + (at0 >> 4) + 4 * lane;
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                copy_async<16>(base + F::v + v_at<D>(i * KPI + kl, c), pv + 512 * i, on(i * KPI + kl));
#pragma unroll
              for (int i = 0; i < (D + 127) / 128; ++i) {
                const int at = 4 * lane + 128 * i;
                if (D >= 128 || lane < D / 4) copy_async<4>(base + F::vs + at, hv + 128 * i, on(at / (D / 16)));
              }
            } else {
              const long long vec = at0 / D;
              const unsigned char* pv = V.payload + vec * F::VP + 8 * lane;
#pragma unroll
              for (int i = 0; i < (F::VP + 15) / 16; ++i) {
                const int at = 8 * lane + 256 * i;
                if (at < SK * F::VP) copy_async<8>(base + F::v + at, pv + 256 * i, on(at / F::VP));
              }
              if (on(lane & 15)) norm = __ldg(reinterpret_cast<const uint16_t*>(V.header) + vec + (lane & 15));
            }
          };
          if (there && low <= n0 && n0 + SK <= end) {
            go([](int) { return true; });
            if (missed) mark(0u);
          } else {
            go([&](int key) { return there && key >= c0 && key < c1; });
            mark(there ? 0u : (1u << c1) - (1u << c0));
          }
        } else {
          const int mk = lane & 15;
          const bool want = mk >= c0 && mk < c1, on = there && want;
          mark(__ballot_sync(kFull, want && !there) & 0xFFFFu);
          const unsigned char* hk = K.header + (on ? at0 >> 4 : 0);
#pragma unroll
          for (int i = 0; i < D / 64; ++i)
            if (lane < 16) copy_async<4>(base + F::ks + mk * (D / 16) + 4 * i, hk + 4 * i, on);
            else if (VB == 0) copy_async<4>(base + F::vs + mk * (D / 16) + 4 * i, V.header + (on ? at0 >> 4 : 0) + 4 * i, on);
          if (VB > 0 && on) norm = __ldg(reinterpret_cast<const uint16_t*>(V.header) + at0 / D);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int key = i * KPI + kl;
            const long long kv = __shfl_sync(kFull, on ? at0 : -1, key);
            const long long at = (kv < 0 ? 0 : kv) + 16 * c;
            copy_async<16>(base + F::k + k_at<D>(key, c), K.payload + at, kv >= 0);
            if (VB == 0) copy_async<16>(base + F::v + v_at<D>(key, c), V.payload + at, kv >= 0);
          }
          if constexpr (VB > 0) {
#pragma unroll
            for (int i = 0; i < (F::VP + 15) / 16; ++i) {
              const int at = 8 * lane + 256 * i, key = min(at / F::VP, SK - 1);
              const long long kv = __shfl_sync(kFull, on ? at0 / D : -1, key);
              if (at < SK * F::VP)
                copy_async<8>(base + F::v + at, V.payload + (kv < 0 ? 0 : kv) * F::VP + at % F::VP, kv >= 0);
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return norm;
    };
    auto put_norm = [&](int st, uint16_t norm) {
      if (VB > 0 && lane < 16) *reinterpret_cast<uint16_t*>(ring + st * F::slice + F::vs + 2 * lane) = norm;
    };
    constexpr int STEP = SK * NW;
    auto spot = [&](int n0) { return spot_of(a, pages, seq, n0 + (runs ? 0 : lane & 15), end, inv); };
    int ask = j0 + SK * warp;  // the next slice to ask for
    {
      Spot sp[NS - 1];
      uint16_t norm[NS - 1];
#pragma unroll
      for (int k = 0; k < NS - 1; ++k) sp[k] = spot(ask + STEP * k);
#pragma unroll
      for (int k = 0; k < NS - 1; ++k) norm[k] = issue(ask + STEP * k, k, sp[k]);
#pragma unroll
      for (int k = 0; k < NS - 1; ++k) put_norm(k, norm[k]);
      ask += STEP * (NS - 1);
    }
    Spot ahead = spot(ask);
    uint16_t norm = 0;
    next_item();

    if (tid < 16) {
      Row r{0, 0x7FFFFFFF, 0, 0.f, 0.f, {0, 0, 0}};  // rows that are not there see everything: they never need a mask
      if (tid < rows) {
        const int row = it.row0 + tid, ti = row / G;
        r.pos = it.pos0 + ti;
        r.hi = min(it.len, max(r.pos + 1, it.prefix));
        if (a.c.window) r.lo = max(r.lo, r.pos - a.c.window + 1);
        if (a.c.first_keys) r.lo = max(r.lo, a.c.first_keys[it.tok0 + ti]);
        if (a.c.slopes) r.slope = a.c.slopes[it.kvh * G + (row - ti * G)] * kLog2e;
      }
      row_of[tid].lo = r.lo;
      row_of[tid].hi = r.hi;
      row_of[tid].pos = r.pos;
      row_of[tid].slope = r.slope;
    }
    // Q's row g (and 8 + g) as fragments; everything else of this lane belongs to the rows 2 t, 2 t + 1 (and 8 more)
    uint32_t q[NT][D / 16][2];
    float f[NT][2], m[NT][2], mu[NT][2], l[NT][2];  // f: scores to log2 units; mu: m, or 0 where that is unset
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int r = g + 8 * u;
      const bool valid = r < rows;
      const int row = it.row0 + (valid ? r : 0), ti = row / G, head = it.kvh * G + (row - ti * G), tok = it.tok0 + ti;
      const float rs = load_q_any<D>(a, (long long)tok * a.c.q_stride + (long long)head * D, valid, t, q[u],
                                     warp == 0 ? q_rest + u * D + lane : nullptr);
      const float x = fmaxf(a.scale * rs, 1.2e-38f);
      if (warp == 0 && t == 0) row_of[r].sl = x;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[u][e] = __shfl_sync(kFull, x, 8 * t + 4 * e);
        if (mods) f[u][e] = 1.f;  // (scores with modifications are in log2 units already)
        m[u][e] = -INFINITY;
        mu[u][e] = l[u][e] = 0.f;
      }
    }
    __syncthreads();  // the rows
    // every row sees the keys [all_lo, all_hi), and they are this range's
    const int all_lo = max(it.lo, __reduce_max_sync(kFull, row_of[lane & 15].lo));
    const int all_hi = min(end, __reduce_min_sync(kFull, row_of[lane & 15].hi));
    // scales from here on (of K's key lane % 16, of V's) do not pass: the clamp, or not finite (a turbo norm)
    const bool of_k = lane < 16;
    const uint32_t bump = of_k || VB == 0 ? 0x20012001u : 0x04000400u;
    const int sc_at = of_k ? F::ks + lane * (D / 16) : F::vs + (lane - 16) * F::VH;
    float o[NT][D / 16][4];
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][i][e] = 0.f;

    int st = 0;
#pragma unroll 1
    for (int key0 = j0 + SK * warp; key0 < end; key0 += STEP, st = st + 1 == NS ? 0 : st + 1) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      const int last = st == 0 ? NS - 1 : st - 1;  // the stage read before, asked for below
      if (VB > 0 && ask > j0 + SK * warp + STEP * (NS - 1)) put_norm(last == 0 ? NS - 1 : last - 1, norm);
      __syncwarp();  // the slice is there, and the one before it has been read
      norm = issue(ask, last, ahead);
      ask += STEP;
      ahead = spot(ask);
      unsigned char* sk = ring + st * F::slice;
      uint32_t poison = 0;
      {
        __half* s = reinterpret_cast<__half*>(sk + sc_at);
        uint32_t big = 0;
        if constexpr (VB == 0) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) big |= (reinterpret_cast<const uint32_t*>(s)[i] & 0x7FFF7FFFu) + bump;
        } else {
          if (of_k) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) big |= (reinterpret_cast<const uint32_t*>(s)[i] & 0x7FFF7FFFu) + bump;
          } else {
            big = (__half_as_ushort(*s) & 0x7FFFu) + (bump & 0xFFFFu);
          }
        }
        if (__any_sync(kFull, (big & 0x80008000u) != 0)) {
          const uint32_t p = __ballot_sync(kFull, mend_scales(s, of_k || VB == 0 ? D / 32 : 1, of_k || VB == 0));
          poison = (p | p >> 16) & 0xFFFFu;
          __syncwarp();
        }
      }
      // scores: x[rows 8 u + ..][key g of rows 2 t, 2 t + 1, then key g + 8]
      float x[NT][4];
      {
        uint32_t sa[D / 64], sb[D / 64];  // the scales of both keys
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          sa[i] = *reinterpret_cast<const uint32_t*>(sk + F::ks + g * (D / 16) + 4 * i);
          sb[i] = *reinterpret_cast<const uint32_t*>(sk + F::ks + (g + 8) * (D / 16) + 4 * i);
        }
        auto products = [&](auto with_rest) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {  // a block of 32: two products of the codes, exact, then its scale
            const uint2 wa = *reinterpret_cast<const uint2*>(sk + F::k + k_at<D>(g, 2 * i + (t >> 1)) + 8 * (t & 1));
            const uint2 wb = *reinterpret_cast<const uint2*>(sk + F::k + k_at<D>(g + 8, 2 * i + (t >> 1)) + 8 * (t & 1));
            const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&sa[i / 2]));
            const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&sb[i / 2]));
            const float ka = i & 1 ? fa.y : fa.x, kb = i & 1 ? fb.y : fb.x;
            uint32_t a0[2], a1[2], a2[2], a3[2];
            q8_pairs(wa.x, a0[0], a2[0]);
            q8_pairs(wb.x, a1[0], a3[0]);
            q8_pairs(wa.y, a0[1], a2[1]);
            q8_pairs(wb.y, a1[1], a3[1]);
#pragma unroll
            for (int u = 0; u < NT; ++u) {
              float c[4];
              wm::mma_16816_zc(c, a0[0], a1[0], a2[0], a3[0], q[u][2 * i][0], q[u][2 * i][1]);
              wm::mma_16816(c, a0[1], a1[1], a2[1], a3[1], q[u][2 * i + 1][0], q[u][2 * i + 1][1]);
              if constexpr (with_rest.value) {
                const uint4 r = q_rest[u * D + 32 * i + lane];
                wm::mma_16816(c, a0[0], a1[0], a2[0], a3[0], r.x, r.y);
                wm::mma_16816(c, a0[1], a1[1], a2[1], a3[1], r.z, r.w);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) x[u][e] = i == 0 ? (e < 2 ? ka : kb) * c[e] : fmaf(e < 2 ? ka : kb, c[e], x[u][e]);
            }
          }
        };
        if (fine) products(std::true_type{});
        else products(std::false_type{});
      }
      const uint32_t gone = missed ? miss[st] : 0u;
      const bool masked = key0 < all_lo || key0 + SK > all_hi || (gone | poison) != 0u;
      if (mods || masked) {
        const float2 cap = cap_factors(a.c.softcap);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& s = x[u][e];
            const Row r = row_of[8 * u + 2 * t + (e & 1)];
            const int c = g + 4 * (e & 2), j = key0 + c;
            if (mods) {
              s *= r.sl;
              if (a.c.softcap > 0.f) s = cap_score(s, cap.x, cap.y);  // (sl holds log2 e)
              if (r.slope != 0.f) s = fmaf(-r.slope, fabsf((float)(r.pos - j)), s);
            }
            if ((poison >> c) & 1u) s = __uint_as_float(0x7FC00000u);
            if (j < r.lo || j >= r.hi || j < low || j >= end || ((gone >> c) & 1u)) s = -INFINITY;
          }
        }
      }
      bool raise = false;
      float mx[NT][2];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[u][e] = fmaxf(x[u][e], x[u][2 + e]) * f[u][e];
          raise |= mx[u][e] - m[u][e] > kMaxExp;
        }
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = mx[u][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
            const float mn = fmaxf(m[u][e], top - kBias);
            al[e] = mn == -INFINITY ? 1.f : ex2(m[u][e] - mn);
            m[u][e] = mn;
            mu[u][e] = mn == -INFINITY ? 0.f : mn;
            l[u][e] *= al[e];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][i][e] *= al[e & 1];
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[e] = ex2(fmaf(x[u][e], f[u][e], -mu[u][e]));
          w[2 + e] = ex2(fmaf(x[u][2 + e], f[u][e], -mu[u][e]));
          l[u][e] += w[e] + w[2 + e];
        }
        p[u][0] = transpose8(narrow(w[0], w[1], (const __half*)nullptr));
        p[u][1] = transpose8(narrow(w[2], w[3], (const __half*)nullptr));
      }
      // O^T += V^T P^T: this lane's coordinates are D / 8 consecutive ones (D = 256: two runs of 16) of four keys
      const int keys[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
#pragma unroll
      for (int c = 0; c < (D + 127) / 128; ++c) {
        constexpr int W = D == 64 ? 2 : 4;
        const int chunk = D == 64 ? g >> 1 : 8 * c + g;
        uint32_t w[4][W], s1[4];  // q8_0: the codes of a key; turbo: the selectors of W quads
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if constexpr (VB == 0) {
            const unsigned char* at = sk + F::v + v_at<D>(keys[y], chunk);
            if constexpr (D == 64) {
              const uint2 z = *reinterpret_cast<const uint2*>(at + 8 * (g & 1));
              w[y][0] = z.x; w[y][1] = z.y;
            } else {
              const uint4 z = *reinterpret_cast<const uint4*>(at);
              w[y][0] = z.x; w[y][1] = z.y; w[y][W - 2] = z.z; w[y][W - 1] = z.w;
            }
            s1[y] = *reinterpret_cast<const uint16_t*>(sk + F::vs + keys[y] * (D / 16) + (chunk >> 1) * 2);
          } else {
            s1[y] = *reinterpret_cast<const uint16_t*>(sk + F::vs + keys[y] * 2);
            constexpr int CB = W * VB / 2;  // bytes of this lane's codes
            const unsigned char* at = sk + F::v + keys[y] * F::VP + (8 * c + g) * CB;
            uint32_t x0 = 0, x1 = 0;  // codes of the first and of the last W / 2 quads
            if constexpr (D == 64) {
              x0 = at[0];
              if constexpr (VB == 2) x0 |= (uint32_t)at[1] << 8;
              if constexpr (VB == 3) x0 |= (uint32_t)at[1] << 8 | (uint32_t)at[2] << 16;
              w[y][0] = nibbles<VB>(x0 & ((1u << 4 * VB) - 1u));
              w[y][1] = nibbles<VB>(x0 >> 4 * VB);
            } else {
              const uint16_t* h = reinterpret_cast<const uint16_t*>(at);
              if constexpr (VB == 1) {
                x0 = h[0] & 0xFFu;
                x1 = h[0] >> 8;
              } else if constexpr (VB == 2) {
                x0 = h[0];
                x1 = h[1];
              } else {
                const uint32_t mid = h[1];
                x0 = h[0] | (mid & 0xFFu) << 16;
                x1 = mid >> 8 | (uint32_t)h[2] << 8;
              }
              w[y][0] = nibbles<VB>(x0 & ((1u << 4 * VB) - 1u));
              w[y][1] = nibbles<VB>(x0 >> 4 * VB);
              w[y][W - 2] = nibbles<VB>(x1 & ((1u << 4 * VB) - 1u));
              w[y][W - 1] = nibbles<VB>(x1 >> 4 * VB);
            }
          }
        }
        const uint32_t sab = __byte_perm(s1[0], s1[1], 0x5410), scd = __byte_perm(s1[2], s1[3], 0x5410);
#pragma unroll
        for (int z = 0; z < W; ++z) {
          uint32_t y[2][4];  // coordinates 0 to 3 of the first two keys, of the second two
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (VB == 0) {
              q8_pairs(__byte_perm(w[2 * h][z], w[2 * h + 1][z], 0x5140), y[h][0], y[h][1]);
              q8_pairs(__byte_perm(w[2 * h][z], w[2 * h + 1][z], 0x7362), y[h][2], y[h][3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[h][e] = mul_h2(y[h][e], h ? scd : sab);
            } else {
              turbo_pairs(tab, w[2 * h][z], w[2 * h + 1][z], h ? scd : sab, y[h]);
            }
          }
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            wm::mma_16816(o[u][(c * W + z) * 2], y[0][0], y[0][1], y[1][0], y[1][1], p[u][0], p[u][1]);
            wm::mma_16816(o[u][(c * W + z) * 2 + 1], y[0][2], y[0][3], y[1][2], y[1][3], p[u][0], p[u][1]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the rings have been read

    // ---- the warps' results, joined in their order ----
    float* mo = reinterpret_cast<float*>(sm);  // [NW][8 NT][OS]
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[u][e] += __shfl_xor_sync(kFull, l[u][e], d);
        if (g == 0) ml[warp * 16 + 8 * u + 2 * t + e] = make_float2(m[u][e], l[u][e]);
        float* row = mo + (warp * 8 * NT + 8 * u + 2 * t + e) * F::OS;
        constexpr int W = D == 64 ? 2 : 4;
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c)
#pragma unroll
          for (int z = 0; z < W; ++z) {
            const float(&x)[4] = o[u][(c * W + z) * 2], (&y)[4] = o[u][(c * W + z) * 2 + 1];
            *reinterpret_cast<float4*>(row + (D == 64 ? 8 * g : 128 * c + 16 * g) + 4 * z) =
                make_float4(x[e], x[2 + e], y[e], y[2 + e]);
          }
      }
    }
    __syncthreads();
    const bool whole = it.n_ctas == 1;
    auto slot_of = [&](int cta, int which) { return ((long long)cta * 2 + which) * a.rows_cap; };
    auto store4 = [&](long long at, const float (&y)[4]) {
      if (a.c.out_dtype == TQ_DTYPE_F32) store_row<4>(static_cast<float*>(a.c.out) + at, y);
      else if (a.c.out_dtype == TQ_DTYPE_F16) store_row<4>(static_cast<__half*>(a.c.out) + at, y);
      else store_row<4>(static_cast<__nv_bfloat16*>(a.c.out) + at, y);
    };
    const long long my_slot = slot_of(blockIdx.x, it.slot);
    float* fin = reinterpret_cast<float*>(sm + F::fin);
    // four columns of a finished row: out, or (turbo values) to the transform
    auto finish = [&](int r, int c, const float (&y)[4]) {
      if constexpr (VB == 0) store4(out_of(r) + 4 * c, y);
      else *reinterpret_cast<float4*>(fin + r * D + 4 * c) = make_float4(y[0], y[1], y[2], y[3]);
    };
    // out = diag(s) H of the finished rows, a row per warp, E coordinates per lane; folds 1 / lambda and 1 / sqrt(D)
    auto transform = [&]() {
      if constexpr (VB > 0) {
        constexpr int E = D / 32;
        __syncthreads();
        for (int r = warp; r < rows; r += NW) {
          float y[E];
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = fin[r * D + E * lane + e];
          thread_wht<E>(y);
#pragma unroll
          for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = fmaf(y[e], lane & d ? -1.f : 1.f, __shfl_xor_sync(kFull, y[e], d));
          const float n = a.inv_lam_v * inv_sqrt_dim<D>();
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] *= n * (float)a.c.tab.signs[E * lane + e];
          const long long at = out_of(r) + E * lane;
          if (a.c.out_dtype == TQ_DTYPE_F32) store_row<E>(static_cast<float*>(a.c.out) + at, y);
          else if (a.c.out_dtype == TQ_DTYPE_F16) store_row<E>(static_cast<__half*>(a.c.out) + at, y);
          else store_row<E>(static_cast<__nv_bfloat16*>(a.c.out) + at, y);
        }
      }
    };
    for (int i = tid; i < rows * (D / 4); i += NW * 32) {
      const int r = i / (D / 4), c = i % (D / 4);
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w * 16 + r].x);
      const float at_m = top == -INFINITY ? 0.f : top;
      float y[4] = {0.f, 0.f, 0.f, 0.f}, lt = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 z = ml[w * 16 + r];
        if (z.y == 0.f) continue;  // a share without weight is not looked at
        const float f = ex2(z.x - at_m);
        const float4 v = *reinterpret_cast<const float4*>(mo + (w * 8 * NT + r) * F::OS + 4 * c);
        lt = fmaf(f, z.y, lt);
        y[0] = fmaf(f, v.x, y[0]);
        y[1] = fmaf(f, v.y, y[1]);
        y[2] = fmaf(f, v.z, y[2]);
        y[3] = fmaf(f, v.w, y[3]);
      }
      if (whole) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= inv;
        finish(r, c, y);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (my_slot + r) * D + 4 * c) = make_float4(y[0], y[1], y[2], y[3]);
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + (my_slot + r) * 2) = make_float2(top, lt);
      }
    }
    if (whole) transform();
    else {
      __threadfence();
      __syncthreads();
      if (tid == 0) *flag = (int)atomicAdd(a.counters + it.counter, 1u) == it.n_ctas - 1;
      __syncthreads();
      if (*flag) {
        __threadfence();
        // the shares' references and sums first, then, per four columns of a row, PG threads take every PG-th share each
        const int n_sh = it.n_ctas;
        constexpr int TH = NW * 32;
        float2* sh = reinterpret_cast<float2*>(sm);  // [n_sh][rows]: weight of a share, its sum times that
        auto share = [&](int p) { return slot_of(it.first_cta + p, p == 0 ? 1 : 0); };
        for (int i = tid; i < n_sh * rows; i += TH)
          sh[i] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (share(i / rows) + i % rows) * 2));
        __syncthreads();
        for (int r = warp; r < rows; r += NW) {
          float top = -INFINITY;
          for (int p = lane; p < n_sh; p += 32) top = fmaxf(top, sh[p * rows + r].y != 0.f ? sh[p * rows + r].x : -INFINITY);
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
          if (top == -INFINITY) top = 0.f;
          float lt = 0.f;
          for (int p = lane; p < n_sh; p += 32) {
            const float2 z = sh[p * rows + r];
            const float w = z.y == 0.f ? 0.f : ex2(z.x - top);
            lt += w * z.y;
            sh[p * rows + r] = make_float2(w, z.y);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) lt += __shfl_xor_sync(kFull, lt, d);
          if (lane == 0) ml[r] = make_float2(lt == 0.f ? 0.f : 1.f / lt, 0.f);
        }
        __syncthreads();
        float4* part = reinterpret_cast<float4*>(sm + F::ring) - TH;  // (behind the weights)
        const int units = rows * (D / 4);
        int pg = 1;  // threads of a unit
        while (2 * pg * units <= TH) pg *= 2;
        for (int i0 = 0; i0 < units; i0 += TH / pg) {
          const int i = i0 + tid % (TH / pg), q0 = tid / (TH / pg);
          const int r = i / (D / 4), c = i % (D / 4);
          float y[4] = {0.f, 0.f, 0.f, 0.f};
          if (i < units && q0 < pg) {
#pragma unroll 1
            for (int p0 = q0; p0 < n_sh; p0 += 12 * pg) {
              float4 v[12];
#pragma unroll
              for (int k = 0; k < 12; ++k)
                v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (share(min(p0 + k * pg, n_sh - 1)) + r) * D + 4 * c));
#pragma unroll
              for (int k = 0; k < 12; ++k) {
                if (p0 + k * pg >= n_sh) continue;
                const float2 z = sh[(p0 + k * pg) * rows + r];
                if (z.y == 0.f) continue;  // a share without weight is not looked at
                y[0] = fmaf(z.x, v[k].x, y[0]);
                y[1] = fmaf(z.x, v[k].y, y[1]);
                y[2] = fmaf(z.x, v[k].z, y[2]);
                y[3] = fmaf(z.x, v[k].w, y[3]);
              }
            }
          }
          if (pg > 1) {
            part[tid] = make_float4(y[0], y[1], y[2], y[3]);
            __syncthreads();
          }
          if (i < units && q0 == 0) {
            for (int q = 1; q < pg; ++q) {
              const float4 z = part[tid + q * (TH / pg)];
              y[0] += z.x;
              y[1] += z.y;
              y[2] += z.z;
              y[3] += z.w;
            }
            const float n = ml[r].x;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= n;
            finish(r, c, y);
          }
        }
        transform();
      }
    }
    __syncthreads();  // before the rings, the item and the flag are written again
  }
}

template <int D, int NT, int VB>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t s) {
  using F = Few<D, NT, VB>;
  // (the weights of an entry's shares, at most one per CTA, lie where the warps' results were)
  if (2LL * sm_count * 8 * NT * 8 > F::fin) return cudaErrorInvalidValue;
  auto kern = few_kernel<D, NT, VB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::total);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)(2 * sm_count)), dim3(F::NW * 32), F::total, s, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int NT>
cudaError_t launch_v(const Args& a, int vb, int sm_count, cudaStream_t s) {
  switch (vb) {
    case 0: return launch<D, NT, 0>(a, sm_count, s);
    case 1: return launch<D, NT, 1>(a, sm_count, s);
    case 2: return launch<D, NT, 2>(a, sm_count, s);
    default: return launch<D, NT, 3>(a, sm_count, s);
  }
}

}  // namespace few
}  // namespace ck
}  // namespace tq
