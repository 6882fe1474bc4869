// Chunk attention on the fifth-generation tensor cores: one kernel for every row count, from one token to thousands.
//
// Per KV head, the rows of a sequence are its (new token, query head of the group) pairs, row = token * G + head.  An
// entry is up to MT consecutive rows and the key tiles that any of them sees (the plan kernel lists them).  The tiles of
// all entries of all KV heads form one line of work units, cut into equal ranges, one per CTA (one CTA per SM): a CTA
// takes the end of one entry, whole entries, and the start of another.  Entries that several CTAs share are joined from
// partial results by the last CTA that finishes, in a fixed order, so that results do not depend on timing.  With one
// decode row the long axis is so split over the whole GPU; with a large chunk every SM works to the end.
//
// A tile is BN keys.  A step is one score product S = Q K^T (M 128, N BN, K D), its softmax and O += P V (M 128, N D,
// K BN).  Entries of more than 128 rows (D <= 128) have two row tiles, and steps alternate between them on one key tile;
// smaller ones have one, and steps alternate between two independent accumulators on successive key tiles, joined at
// the end like any other partial results.  Either way step u uses score buffer u % 2 and warpgroup u % 2, and the
// tensor core works on one buffer while the other is in the softmax.  At D = 256 tensor memory holds one accumulator,
// and one warpgroup takes every step.
//
// Warps, meeting on mbarriers only:
//   0-3, 4-7   softmax: one row per thread.  S from tensor memory to registers, score modifications and masks, online
//              softmax with a lazily raised reference (O in tensor memory is rescaled only when the maximum passes the
//              reference by 2^8), P as fp16 into the columns of S, the left operand of the value product.
//   8-11       producers: codes to fp16 values, K and V alike, 16 coordinates per step of a thread, into swizzled
//              operand tiles (K: K-major; the same bytes read MN-major are V).  A q8_0 code becomes its value by a byte
//              permute into 1024 + u, an exact subtraction and one rounded product with the scale.
//   12         one thread issues the products, in the order QK(0), QK(1), PV(0), QK(2), PV(1), ...
//   13         finds each key's place through the block table a few tiles ahead, and asks for its bytes in L2
//   14         reads the plan a few items ahead
// The scales of fp16 operands: queries are multiplied by a power of two per row (any input type fits then), turbo
// values carry lambda so that the codebook is nearly exact in fp16.  Rounding to fp16 (2^-11 relative at most per
// operand) is what the tensor core's full rate asks for; sums are fp32.
#pragma once

#include "tq_batch.cuh"
#include "tq_chunk.h"
#include "tq_tc.cuh"

namespace tq {
namespace ck {

constexpr int kThreads = 512;
constexpr int kProdWarps = 4;
constexpr int kIssuer = 12, kLocator = 13, kScheduler = 14;
constexpr int kItemReaders = 8 + kProdWarps + 2;
constexpr int NI = 3;       // items known ahead
constexpr int NL = 6;       // tiles located ahead of the producers
constexpr int kMissRing = 16;
constexpr int kMinUnits = 2;
constexpr float kLazy = 8.0f;
constexpr float kLog2e = 1.4426950408889634074f;
// registers per thread after the split: 256 * 168 + 128 * 112 + 128 * 56 <= 512 * 128
constexpr int kRegsSoftmax = 168, kRegsProducer = 112, kRegsOther = 56;
static_assert(256 * kRegsSoftmax + 128 * kRegsProducer + 128 * kRegsOther <= 512 * 128, "register split");
constexpr int kRegsNeeded = 256 * kRegsSoftmax + 128 * kRegsProducer + 128 * kRegsOther;

template <int D>
struct Shape {
  static constexpr int BN = D == 256 ? 64 : 128;
  static constexpr int kTileB = BN * D * 2;            // bytes of a K or V operand tile
  static constexpr int kQTile = 128 * D * 2;           // bytes of a row tile's queries
  static constexpr int kQTiles = D == 256 ? 1 : 2;
  static constexpr int NB = D == 64 ? 3 : 2;           // K and V tile buffers each
  static constexpr int q = 0;
  static constexpr int k = q + kQTiles * kQTile;
  static constexpr int v = k + NB * kTileB;
  static constexpr int loc = v + NB * kTileB;          // long long [NL][BN]
  static constexpr int miss = loc + NL * BN * 8;       // uint32 [kMissRing][4]
  static constexpr int rs = miss + kMissRing * 16;     // float [256]: row scales
  static constexpr int items = rs + 256 * 4;           // Item [NI]
  static constexpr int tab = items + NI * 128;         // fp16 [8]: the V codebook
  static constexpr int bars = tab + 16;
  static constexpr int total = bars + 64 * 8;
  static constexpr int alloc = total + 1024;
  static_assert(alloc <= 227 * 1024, "shared memory");
  // tensor memory columns: S [2][BN], O [kQTiles][D]
  static constexpr int tO = 2 * BN;
};

struct Item {
  int kind;        // 0: no more; 1: tiles; 2: rows that see nothing
  int kvh, seq, tok0, pos0, len, prefix;
  int row0, rows;  // of the sequence's rows
  int lo, hi;      // keys that some row sees
  int tile, n;     // key tiles of this CTA
  int two;         // two row tiles
  int first_cta, n_ctas, slot;  // CTAs that share the entry; this CTA's partial slot
  int counter;
};
static_assert(sizeof(Item) <= 128, "item");

struct Bars {
  uint64_t k_full[3], k_free[3], v_full[3], v_free[3];
  uint64_t s_done[2], p_full[2], pv_done[2];
  uint64_t drained, q_full, item_full[NI], item_free[NI], loc_full[NL], loc_free[NL];
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 64 * 8, "barriers");

// Byte offset of (row, 16-byte chunk of 8 elements) in an operand tile of R rows: 64-element blocks of R 128-byte rows,
// chunks of a row XOR-swizzled by the row.
template <int R>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (uint32_t)((chunk >> 3) * (128 * R) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Start offset of a K step (16 elements) in a K-major tile of R rows.
template <int R>
__host__ __device__ constexpr uint32_t kstep(int ks) {
  return (uint32_t)((ks >> 2) * (128 * R) + (ks & 3) * 32);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A wait that gives up for good once one has run out: the role then runs through its loops without waiting (every
// named barrier is still met), and the error is reported at the end.
__device__ __forceinline__ void wait(bool& ok, uint64_t* bar, uint32_t parity) {
  if (ok) ok = tc::mbar_wait(bar, parity & 1u);
}

// The same for a whole warp, whose lanes stay of one mind.
__device__ __forceinline__ void wait_warp(bool& ok, uint64_t* bar, uint32_t parity) {
  wait(ok, bar, parity);
  ok = __all_sync(kFull, ok);
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four int8 codes to two fp16 pairs: u = code + 128 permuted under the exponent of 1024, minus 1152 (exact).
__device__ __forceinline__ void q8_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  w ^= 0x80808080u;
  const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 c = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), c);
  const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&y), c);
  a = *reinterpret_cast<const uint32_t*>(&p);
  b = *reinterpret_cast<const uint32_t*>(&q);
}

// A scale clamped to where 127 times it is finite in fp16, duplicated; the sign of bad is left to the caller.
__device__ __forceinline__ uint32_t clamp_scale(uint16_t s) {
  const __half lim = __ushort_as_half(0x5FFE), nlim = __ushort_as_half(0xDFFE);  // 511.5
  const __half h = __hmax(__hmin(__ushort_as_half(s), lim), nlim);
  return (uint32_t)__half_as_ushort(h) * 0x10001u;
}
__device__ __forceinline__ bool not_finite(uint32_t s) { return (s & 0x7C00u) == 0x7C00u; }

__device__ __forceinline__ void arrive_smem(uint64_t* bar, int lane) {
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// ---------------------------------------------------------------------------
// scheduler: the CTA's items, in order
// ---------------------------------------------------------------------------
template <int D>
__device__ void schedule(const Args& a, Bars* B, Item* items, bool& ok) {
  const PlanHead head = *a.plan;
  const long long T = head.units, U = T * a.c.k.H;
  // every CTA that takes part has at least kMinUnits units (so no CTA inside an entry's range is without work)
  const long long nC = max(1LL, min((long long)gridDim.x, U / kMinUnits)), c = blockIdx.x;
  long long u = c < nC ? U * c / nC : 0;
  const long long u1 = c < nC ? U * (c + 1) / nC : 0;
  // the CTA whose range holds a unit
  auto cta_of = [&](long long x) { return (int)(((x + 1) * nC - 1) / U); };
  int cnt = 0;
  auto put = [&](const Item& it) {
    const int s = cnt % NI;
    if (cnt >= NI) wait(ok, &B->item_free[s], cnt / NI - 1);
    items[s] = it;
    tc::mbar_arrive(&B->item_full[s]);
    ++cnt;
  };
  if (u < u1) {
    int h = (int)(u / T);
    long long off = u - (long long)h * T;
    int e = 0;  // the last entry that starts at or before off
    for (int step = 1 << 30; step > 0; step >>= 1)
      if (e + step < head.n_entries && a.entries[e + step].start <= off) e += step;
    while (u < u1) {
      const Entry en = a.entries[e];
      const long long base = (long long)h * T + en.start, w = en.n_tiles + kOverhead;
      Item it;
      it.kvh = h;
      it.seq = en.seq;
      it.row0 = en.row0;
      const SeqOf s = seq_of(a.c.b, en.seq);
      it.tok0 = s.first;
      it.len = s.len;
      it.pos0 = s.len - s.n;
      it.prefix = a.c.prefix_lens ? a.c.prefix_lens[en.seq] : 0;
      it.rows = min(s.n * a.c.G - en.row0, Shape<D>::kQTiles * 128);
      it.lo = en.lo;
      it.hi = en.hi;
      it.two = D != 256 && it.rows > 128;
      it.counter = (h * head.n_entries + e) * 2;
      const long long t0 = max(0LL, u - base - kOverhead), t1 = min((long long)en.n_tiles, u1 - base - kOverhead);
      if (en.n_tiles == 0) {
        it.kind = u == base ? 2 : 0;  // by the CTA that holds its first unit
        it.n = 0;
      } else {
        it.kind = t0 < t1 ? 1 : 0;
        it.tile = en.lo / Shape<D>::BN + (int)t0;
        it.n = (int)(t1 - t0);
        it.first_cta = cta_of(base + kOverhead);
        it.n_ctas = cta_of(base + kOverhead + en.n_tiles - 1) - it.first_cta + 1;
        it.slot = t0 == 0 ? 1 : 0;
      }
      if (it.kind) put(it);
      u = base + w;
      if (++e == head.n_entries) {
        e = 0;
        ++h;
      }
    }
  }
  Item end;
  end.kind = 0;
  put(end);
}

// ---------------------------------------------------------------------------
// locator: the vector of every key of a tile, and its bytes asked for in L2
// ---------------------------------------------------------------------------
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int D>
__device__ void locate_tile(const Args& a, const Item& it, int t, long long* loc, uint32_t* miss, int lane) {
  constexpr int BN = Shape<D>::BN;
  const DevView &K = a.c.k, &V = a.c.v;
#pragma unroll
  for (int i = 0; i < BN / 32; ++i) {
    const int j = t * BN + 32 * i + lane;
    long long vec = -1;
    bool bad = false;
    if (j >= it.lo && j < it.hi) {
      vec = position_vector(a.c.b, K, a.c.layer, it.seq, j);
      bad = vec < 0;
      if (!bad) {
        vec += (long long)it.kvh * K.page_size;
        const unsigned char* pk = K.payload + vec * K.pay_bytes;
        const unsigned char* pv = V.payload + vec * V.pay_bytes;
        prefetch_l2(pk);
        prefetch_l2(pv);
        if constexpr (D == 256) {
          prefetch_l2(pk + 128);
          if (V.pay_bytes > 128) prefetch_l2(pv + 128);
        }
        prefetch_l2(K.header + vec * K.hdr_bytes);
        prefetch_l2(V.header + vec * V.hdr_bytes);
      }
    }
    loc[32 * i + lane] = vec;
    const uint32_t m = __ballot_sync(kFull, bad);
    if (lane == 0) {
      miss[i] = m;
      if (m) atomicOr(a.c.tab.status, kFlagBlockTable);
    }
  }
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
template <int D, int VB>
struct Producer {
  static constexpr int BN = Shape<D>::BN;
  static constexpr int CH = D / 16;                       // units (16 coordinates) per vector
  static constexpr int UN = BN * CH / (32 * kProdWarps);  // units per thread and tile
  static constexpr int VW = VB == 0 ? 4 : VB == 3 ? 2 : 1;  // words of a V unit's codes

  struct Raw {
    uint4 k[UN];
    uint32_t sc[UN];  // K scale in the low half, V scale (or norm) in the high half
  };

  // Codes of K and the scales of K and V for the thread's units of a located tile.
  static __device__ __forceinline__ void load_k(const Args& a, const long long* loc, int ptid, Raw& r) {
    const DevView &K = a.c.k, &V = a.c.v;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int unit = ptid + 32 * kProdWarps * i, row = unit / CH, c = unit % CH;
      const long long vec = loc[row];
      r.k[i] = make_uint4(0u, 0u, 0u, 0u);
      r.sc[i] = 0u;
      if (vec >= 0) {
        r.k[i] = __ldg(reinterpret_cast<const uint4*>(K.payload + vec * D) + c);
        const uint32_t hk = __ldg(reinterpret_cast<const unsigned short*>(K.header + vec * (D / 16)) + (c >> 1));
        const uint32_t hv =
            VB == 0 ? __ldg(reinterpret_cast<const unsigned short*>(V.header + vec * (D / 16)) + (c >> 1))
                    : __ldg(reinterpret_cast<const unsigned short*>(V.header + vec * 2));
        r.sc[i] = hk | (hv << 16);
      }
    }
  }

  static __device__ __forceinline__ void load_v(const Args& a, const long long* loc, int ptid, uint32_t (&v)[UN][VW]) {
    const DevView& V = a.c.v;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int unit = ptid + 32 * kProdWarps * i, row = unit / CH, c = unit % CH;
      const long long vec = loc[row];
#pragma unroll
      for (int k = 0; k < VW; ++k) v[i][k] = 0u;
      if (vec >= 0) {
        if constexpr (VB == 0) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(V.payload + vec * D) + c);
          v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
        } else {
          const unsigned short* p = reinterpret_cast<const unsigned short*>(V.payload + vec * (D * VB / 8)) + VB * c;
          v[i][0] = __ldg(p);
          if constexpr (VB >= 2) v[i][0] |= (uint32_t)__ldg(p + 1) << 16;
          if constexpr (VB == 3) v[i][1] = __ldg(p + 2);
        }
      }
    }
  }

  // 16 values (8 fp16 pairs) of a unit to its two chunks of the tile; lanes of odd 64-blocks store the second chunk
  // first, so that the eight lanes of a row hit eight different chunks.
  static __device__ __forceinline__ void put(unsigned char* tile, int row, int c, const uint32_t (&h)[8]) {
    const bool swap = (c >> 2) & 1;
    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
    *reinterpret_cast<uint4*>(tile + tile_at<BN>(row, 2 * c + (swap ? 1 : 0))) = swap ? hi : lo;
    *reinterpret_cast<uint4*>(tile + tile_at<BN>(row, 2 * c + (swap ? 0 : 1))) = swap ? lo : hi;
  }

  static __device__ __forceinline__ void q8_unit(const uint32_t (&w)[4], uint32_t scale2, uint32_t (&h)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t x, y;
      q8_pairs(w[k], x, y);
      h[2 * k] = mul_h2(x, scale2);
      h[2 * k + 1] = mul_h2(y, scale2);
    }
  }

  static __device__ __forceinline__ void convert_k(const Raw& r, unsigned char* tile, int ptid) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int unit = ptid + 32 * kProdWarps * i, row = unit / CH, c = unit % CH;
      const uint32_t w[4] = {r.k[i].x, r.k[i].y, r.k[i].z, r.k[i].w};
      uint32_t s2 = clamp_scale((uint16_t)r.sc[i]);
      // a key whose stored K or V is not finite poisons the scores of the rows that see it (the value product of the
      // others must not meet it)
      if (not_finite(r.sc[i]) || not_finite(r.sc[i] >> 16)) s2 = 0x7E007E00u;
      uint32_t h[8];
      q8_unit(w, s2, h);
      put(tile, row, c, h);
    }
  }

  static __device__ __forceinline__ void convert_v(const uint32_t (&v)[UN][VW], const uint32_t (&sc)[UN],
                                                   const uint32_t* tab, unsigned char* tile, int ptid) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int unit = ptid + 32 * kProdWarps * i, row = unit / CH, c = unit % CH;
      const uint32_t raw = sc[i] >> 16;
      uint32_t h[8];
      if constexpr (VB == 0) {
        const uint32_t s2 = not_finite(raw) ? 0u : clamp_scale((uint16_t)raw);
        const uint32_t w[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
        q8_unit(w, s2, h);
      } else {
        const uint32_t s2 = not_finite(raw) ? 0u : raw * 0x10001u;
        // the codebook (up to 8 fp16 levels) as byte tables: low bytes in lo0, lo1, high bytes in hi0, hi1
        const uint32_t lo0 = tab[0], lo1 = tab[1], hi0 = tab[2], hi1 = tab[3];
        const uint64_t codes = VB == 3 ? (uint64_t)v[i][0] | ((uint64_t)v[i][VW - 1] << 32) : (uint64_t)v[i][0];
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // four codes: nibble selectors of a byte permute
          const uint32_t x = (uint32_t)(codes >> (4 * VB * g));
          constexpr uint32_t m = (1u << VB) - 1u;
          const uint32_t sel = (x & m) | ((x << (4 - VB)) & (m << 4)) | ((x << (8 - 2 * VB)) & (m << 8)) |
                               ((x << (12 - 3 * VB)) & (m << 12));
          const uint32_t lb = __byte_perm(lo0, lo1, sel), hb = __byte_perm(hi0, hi1, sel);
          h[2 * g] = mul_h2(__byte_perm(lb, hb, 0x5140), s2);
          h[2 * g + 1] = mul_h2(__byte_perm(lb, hb, 0x7362), s2);
        }
      }
      put(tile, row, c, h);
    }
  }
};

// ---------------------------------------------------------------------------
// the queries of an item: row r at row r % 128 of row tile r / 128, times a power of two that brings the row's largest
// element into [1, 2), whose inverse goes to rs[r]
// ---------------------------------------------------------------------------
template <int D, class T>
__device__ __forceinline__ void load_queries(const Args& a, const Item& it, const T* q, unsigned char* sq, float* rs,
                                             int warp, int lane) {
  constexpr int LQ = D / 8, RP = 32 / LQ;  // lanes per row, rows per warp and pass
  const int c = lane % LQ, G = a.c.G;
  constexpr int U = 4;
  for (int r0 = warp * RP + lane / LQ; __any_sync(kFull, r0 < it.rows); r0 += 8 * RP * U) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 8 * RP * u;
      if (r < it.rows) {
        const int row = it.row0 + r, i = row / G, g = row - i * G;
        load_row<8>(q + (long long)(it.tok0 + i) * a.c.q_stride + (long long)(it.kvh * G + g) * D + 8 * c, x[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 8 * RP * u;
      const bool on = r < it.rows;
      uint32_t top = 0;  // bits of the largest magnitude (NaN above all)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, on ? __float_as_uint(x[u][e]) & 0x7FFFFFFFu : 0u);
#pragma unroll
      for (int m = 1; m < LQ; m <<= 1) top = max(top, __shfl_xor_sync(kFull, top, m));
      uint32_t ex = min(max(top >> 23, 1u), 253u);
      if (top >= 0x7F800000u) ex = 127u;  // infinite or NaN: as it is
      const float f = a.q_sign * __uint_as_float((254u - ex) << 23);
      if (on) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = narrow(x[u][2 * e] * f, x[u][2 * e + 1] * f, (const __half*)nullptr);
        *reinterpret_cast<uint4*>(sq + (r >> 7) * Shape<D>::kQTile + tile_at<128>(r & 127, c)) =
            make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0) rs[r] = __uint_as_float(ex << 23);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// epilogue helpers
// ---------------------------------------------------------------------------

// Unscaled Walsh-Hadamard transform of N values of one thread.
template <int N>
__device__ __forceinline__ void thread_wht(float (&x)[N]) {
#pragma unroll
  for (int s = 1; s < N; s <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((i & s) == 0) {
        const float u = x[i], v = x[i + s];
        x[i] = u + v;
        x[i + s] = u - v;
      }
    }
  }
}

__device__ __forceinline__ void store8(void* out, int dtype, long long at, const float (&x)[8]) {
  if (dtype == TQ_DTYPE_F32) store_row<8>(static_cast<float*>(out) + at, x);
  else if (dtype == TQ_DTYPE_F16) store_row<8>(static_cast<__half*>(out) + at, x);
  else store_row<8>(static_cast<__nv_bfloat16*>(out) + at, x);
}

template <int D, int VB>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
  using Sh = Shape<D>;
  constexpr int BN = Sh::BN, NB = Sh::NB;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = tc::smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Bars* B = reinterpret_cast<Bars*>(sm + Sh::bars);
  Item* items = reinterpret_cast<Item*>(sm + Sh::items);
  long long* loc = reinterpret_cast<long long*>(sm + Sh::loc);
  uint32_t* miss = reinterpret_cast<uint32_t*>(sm + Sh::miss);
  float* rs = reinterpret_cast<float*>(sm + Sh::rs);

  if (warp == 0) {
    tc::tmem_alloc(&B->tmem, 512);
    if (lane == 0) {
      for (int i = 0; i < 3; ++i) {
        tc::mbar_init(&B->k_full[i], kProdWarps);
        tc::mbar_init(&B->v_full[i], kProdWarps);
        tc::mbar_init(&B->k_free[i], 1);
        tc::mbar_init(&B->v_free[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&B->s_done[i], 1);
        tc::mbar_init(&B->p_full[i], 4);
        tc::mbar_init(&B->pv_done[i], 1);
      }
      tc::mbar_init(&B->q_full, 8);
      tc::mbar_init(&B->drained, 1);
      for (int i = 0; i < NI; ++i) {
        tc::mbar_init(&B->item_full[i], 1);
        tc::mbar_init(&B->item_free[i], kItemReaders);
      }
      for (int i = 0; i < NL; ++i) {
        tc::mbar_init(&B->loc_full[i], 1);
        tc::mbar_init(&B->loc_free[i], kProdWarps);
      }
    }
  }
  if constexpr (VB > 0) {
    if (tid < 4) {  // byte tables of lambda * level: words 0, 1 the low bytes, 2, 3 the high ones
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * (tid & 1) + i;
        const float c = e < (1 << VB) ? a.c.tab.f16_scale[VB - 1] * a.c.tab.centroids[(VB - 1) * 8 + e] : 0.f;
        w |= ((narrow(c, 0.f, (const __half*)nullptr) >> (tid < 2 ? 0 : 8)) & 255u) << (8 * i);
      }
      reinterpret_cast<uint32_t*>(sm + Sh::tab)[tid] = w;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = B->tmem;
  pdl_wait();  // the plan
  bool ok = true;
  int icnt = 0;  // items so far
  int gu = 0;    // steps so far
  int gt = 0;    // key tiles so far

  if (warp >= 12) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kScheduler) {
      if (lane == 0) schedule<D>(a, B, items, ok);
    } else if (warp == kLocator) {
      for (;; ++icnt) {
        const int is = icnt % NI;
        wait_warp(ok, &B->item_full[is], icnt / NI);
        const Item it = items[is];
        if (!ok || it.kind == 0) break;
        for (int j = 0; j < it.n && ok; ++j, ++gt) {
          const int s = gt % NL;
          if (gt >= NL) wait_warp(ok, &B->loc_free[s], gt / NL - 1);
          locate_tile<D>(a, it, it.tile + j, loc + s * BN, miss + (gt % kMissRing) * 4, lane);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&B->loc_full[s]);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
      }
    } else if (warp == kIssuer) {
      if (lane == 0) {
        constexpr uint32_t id_qk = tc::idesc_f16_f32(128, BN);
        constexpr uint32_t id_pv = tc::idesc_f16_f32(128, D) | (1u << 16);  // B (V) MN-major
        for (;; ++icnt) {
          const int is = icnt % NI;
          wait(ok, &B->item_full[is], icnt / NI);
          const int kind = items[is].kind, n = items[is].n, two = items[is].two;
          if (!ok || kind == 0) break;
          if (kind == 1) {
            wait(ok, &B->q_full, icnt);
            const int steps = n << two;
            auto qk = [&](int u) {
              const int j = gt + (u >> two), b = j % NB, s = (gu + u) & 1;
              if (!two || !(u & 1)) wait(ok, &B->k_full[b], j / NB);
              if (!ok) return;
              tc::fence_after_sync();
              const uint64_t dq = tc::desc_sw128(sb + Sh::q + (two ? (u & 1) * Sh::kQTile : 0));
              const uint64_t dk = tc::desc_sw128(sb + Sh::k + b * Sh::kTileB);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                tc::mma_f16(tmem + s * BN, dq + (kstep<128>(ks) >> 4), dk + (kstep<BN>(ks) >> 4), id_qk, ks > 0);
              tc::commit(&B->s_done[s]);
              if (!two || (u & 1)) tc::commit(&B->k_free[b]);
            };
            auto pv = [&](int u) {
              const int j = gt + (u >> two), b = j % NB, s = (gu + u) & 1;
              wait(ok, &B->p_full[s], (gu + u) >> 1);
              if (!two || !(u & 1)) wait(ok, &B->v_full[b], j / NB);
              if (!ok) return;
              tc::fence_after_sync();
              const uint32_t o = tmem + Sh::tO + (D == 256 ? 0 : (u & 1) * D);
              const bool fresh = u < (D == 256 ? 1 : 2);
              const uint64_t dv = tc::desc_sw128_mn(sb + Sh::v + b * Sh::kTileB, BN * 128);
#pragma unroll
              for (int ks = 0; ks < BN / 16; ++ks)
                tc::mma_f16_ts(o, tmem + s * BN + 8 * ks, dv + (uint64_t)(ks * (2048 >> 4)), id_pv, !fresh || ks > 0);
              tc::commit(&B->pv_done[s]);
              if (!two || (u & 1)) tc::commit(&B->v_free[b]);
            };
            qk(0);
            for (int u = 0; u < steps && ok; ++u) {
              if (u + 1 < steps) qk(u + 1);
              pv(u);
            }
            gu += steps;
            gt += n;
          } else {
            wait(ok, &B->q_full, icnt);
          }
          tc::mbar_arrive(&B->item_free[is]);
        }
        tc::commit(&B->drained);  // products still in flight end before the tensor memory is freed
        tc::mbar_wait(&B->drained, 0u, 1 << 16);
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegsProducer>();
    using P = Producer<D, VB>;
    const int ptid = tid - 256;
    uint32_t tab[4] = {0u, 0u, 0u, 0u};
    if constexpr (VB > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) tab[i] = reinterpret_cast<const uint32_t*>(sm + Sh::tab)[i];
    }
    typename P::Raw kr;
    bool loaded = false;  // kr holds the next tile
    for (;; ++icnt) {
      const int is = icnt % NI;
      wait_warp(ok, &B->item_full[is], icnt / NI);
      const int kind = items[is].kind, n = items[is].n;
      if (!ok || kind == 0) break;
      for (int j = 0; j < n && ok; ++j, ++gt) {
        const int s = gt % NL, b = gt % NB;
        const long long* lv = loc + s * BN;
        if (!loaded) {
          wait_warp(ok, &B->loc_full[s], gt / NL);
          P::load_k(a, lv, ptid, kr);
        }
        loaded = false;
        uint32_t vr[P::UN][P::VW], sc[P::UN];
        P::load_v(a, lv, ptid, vr);  // in flight while K is converted
#pragma unroll
        for (int i = 0; i < P::UN; ++i) sc[i] = kr.sc[i];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B->loc_free[s]);
        if (gt >= NB) wait_warp(ok, &B->k_free[b], gt / NB - 1);
        P::convert_k(kr, sm + Sh::k + b * Sh::kTileB, ptid);
        arrive_smem(&B->k_full[b], lane);
        if (j + 1 < n) {  // the next tile's K in flight while V is converted
          const int s1 = (gt + 1) % NL;
          wait_warp(ok, &B->loc_full[s1], (gt + 1) / NL);
          P::load_k(a, loc + s1 * BN, ptid, kr);
          loaded = true;
        }
        if (gt >= NB) wait_warp(ok, &B->v_free[b], gt / NB - 1);
        P::convert_v(vr, sc, tab, sm + Sh::v + b * Sh::kTileB, ptid);
        arrive_smem(&B->v_full[b], lane);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float cap = a.c.softcap;
    const bool mods = cap > 0.f || a.c.slopes != nullptr;
    for (;; ++icnt) {
      const int is = icnt % NI;
      wait_warp(ok, &B->item_full[is], icnt / NI);
      const Item& it = items[is];
      // A role that gave up leaves here: its partner's waits run out in their turn, and both meet no more barriers.
      if (tc::bar_sync_and(1, 256, ok && it.kind != 0) == false) break;  // (also: the last item's queries are not read any more)
      if (it.kind == 1) {
        if (a.c.q_dtype == TQ_DTYPE_F32)
          load_queries<D>(a, it, static_cast<const float*>(a.c.q), sm + Sh::q, rs, warp, lane);
        else if (a.c.q_dtype == TQ_DTYPE_F16)
          load_queries<D>(a, it, static_cast<const __half*>(a.c.q), sm + Sh::q, rs, warp, lane);
        else
          load_queries<D>(a, it, static_cast<const __nv_bfloat16*>(a.c.q), sm + Sh::q, rs, warp, lane);
      }
      arrive_smem(&B->q_full, lane);
      tc::bar_sync(1, 256);

      // this thread's row
      const int rr = (it.two ? 128 * wg : 0) + r;
      const bool valid = rr < it.rows;
      const int row = it.row0 + (valid ? rr : 0), ti = row / a.c.G, head = it.kvh * a.c.G + (row - ti * a.c.G);
      const int tok = it.tok0 + ti, pos = it.pos0 + ti;
      const long long out_at = ((long long)tok * a.c.n_q_heads + head) * D;
      if (it.kind == 2) {
        if (valid && (it.two || wg == 0)) {
          const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int c = 0; c < D / 8; ++c) store8(a.c.out, a.c.out_dtype, out_at + 8 * c, z);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
        continue;
      }
      int lo = 0, hi = 0x7FFFFFFF;  // rows that are not there see everything: they never need a mask
      float sl = 1.f, slope = 0.f;
      if (valid) {
        hi = min(it.len, max(pos + 1, it.prefix));
        if (a.c.window) lo = max(lo, pos - a.c.window + 1);
        if (a.c.first_keys) lo = max(lo, a.c.first_keys[tok]);
        sl = fmaxf(a.scale * rs[rr], 1.2e-38f);
        if (a.c.slopes) slope = a.c.slopes[head] * kLog2e;
      }
      const int all_lo = __reduce_max_sync(kFull, lo), all_hi = __reduce_min_sync(kFull, hi);
      const int steps = it.n << it.two;
      const int u0 = D == 256 ? (wg == 0 ? 0 : steps) : wg, du = D == 256 ? 1 : 2;
      const uint32_t t_o = tmem + Sh::tO + (D == 256 ? 0 : wg * D) + lanes;
      float m = -INFINITY, l = 0.f;
      int last = -1;
      for (int u = u0; u < steps; u += du) {
        const int jt = u >> it.two, s = (gu + u) & 1;
        const int key0 = (it.tile + jt) * BN;
        wait_warp(ok, &B->s_done[s], (gu + u) >> 1);
        tc::fence_after_sync();
        const uint32_t t_s = tmem + s * BN + lanes;
        float x[BN];
        {
          uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) tc::tmem_ld32_nw(t_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(w + 32 * c));
          tc::tmem_wait_ld();
        }
        float f = sl;
        if (mods) {  // to log2 units here
          if (cap > 0.f) {
            const float fi = 2.f * sl / cap, fo = cap * kLog2e;  // sl holds log2 e: 2^(fi x) = e^(2 s / cap)
#pragma unroll
            for (int e = 0; e < BN; ++e) x[e] = fo * (1.f - __fdividef(2.f, 1.f + ex2(x[e] * fi)));
          } else {
#pragma unroll
            for (int e = 0; e < BN; ++e) x[e] *= sl;
          }
          const float d0 = (float)(pos - key0);
#pragma unroll
          for (int e = 0; e < BN; ++e) x[e] = fmaf(-slope, fabsf(d0 - (float)e), x[e]);
          f = 1.f;
        }
        const uint32_t* mw = miss + ((gt + jt) % kMissRing) * 4;
        uint32_t any_miss = 0;
#pragma unroll
        for (int i = 0; i < BN / 32; ++i) any_miss |= mw[i];
        if (key0 < all_lo || key0 + BN > all_hi || any_miss) {
#pragma unroll
          for (int i = 0; i < BN / 32; ++i) {
            // visible keys of this 32-group as a bit mask
            const int p = min(max(lo - key0 - 32 * i, 0), 32), q = min(max(hi - key0 - 32 * i, 0), 32);
            const uint32_t below_q = q == 32 ? 0xFFFFFFFFu : (1u << q) - 1u;
            const uint32_t from_p = p == 32 ? 0u : 0xFFFFFFFFu << p;
            const uint32_t vis = below_q & from_p & ~mw[i];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[32 * i + e] = (vis >> e) & 1u ? x[32 * i + e] : -INFINITY;
          }
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int e = 4; e < BN; e += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = e + 4 + k < BN ? fmaxf(fmaxf(mx[k], x[e + k]), x[e + 4 + k]) : fmaxf(mx[k], x[e + k]);
        }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
        // (rows that are not there hold whatever shared memory had: they have no say, so that results do not vary)
        if (__any_sync(kFull, valid && mt > m + kLazy)) {
          const float mn = fmaxf(m, mt);
          const float al = mn == -INFINITY ? 1.f : ex2(m - mn);
          l *= al;
          if (last >= 0) {  // the product of this warpgroup's last step is complete
            if constexpr (D == 256) {
              wait_warp(ok, &B->pv_done[last & 1], last >> 1);
              tc::fence_after_sync();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(t_o + 32 * c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc::tmem_st32(t_o + 32 * c, o);
            }
          }
          m = mn;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const float2 f2 = make_float2(f, f), m2 = make_float2(-mu, -mu);
        float2 l2[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int i = 64 * c + 2 * e;
            float2 p = __ffma2_rn(make_float2(x[i], x[i + 1]), f2, m2);
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            l2[e & 1] = __fadd2_rn(l2[e & 1], p);
            pk[e] = narrow(p.x, p.y, (const __half*)nullptr);
          }
          tc::tmem_st32(t_s + 32 * c, pk);
        }
        l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B->p_full[s]);
        last = gu + u;
      }
      if (last >= 0) wait_warp(ok, &B->pv_done[last & 1], last >> 1);
      tc::fence_after_sync();
      gu += steps;
      gt += it.n;
      const bool mine = D != 256 || wg == 0;  // this warpgroup holds rows

      // ---- the result: O / l where this warpgroup alone has the rows, else a partial result ----
      const int parts = D == 256 || it.two ? it.n_ctas : 2 * it.n_ctas;
      const bool whole = parts == 1;
      // partial slots: [CTA][start or end of its range][warpgroup][rows][D], then m and l of each
      auto slot_of = [&](int cta, int which, int w) { return ((long long)cta * 2 + which) * 2 + w; };
      const long long my_slot = slot_of(blockIdx.x, it.slot, wg);
      float* po = a.part_o + my_slot * a.rows_cap * D + (long long)r * D;
      float norm = a.inv_lam_v;  // folds 1 / lambda and the transform's 1 / sqrt(D)
      if constexpr (VB > 0) norm *= inv_sqrt_dim<D>();
      if (mine) {
        if (whole) norm *= l == 0.f ? 0.f : __fdividef(1.f, l);
        if (!whole && valid) {
          float* ml = a.part_ml + my_slot * a.rows_cap * 2 + 2 * r;
          ml[0] = m;
          ml[1] = l;
        }
        if (last >= 0) {
          // a row without any weight (l = 0) is zeros whatever its accumulator holds
          const bool zero = l == 0.f;
          auto emit = [&](int col, const float (&y)[8]) {  // eight columns of this thread's row
            if (!valid) return;
            if (whole) store8(a.c.out, a.c.out_dtype, out_at + col, y);
            else store_row<8>(po + col, y);
          };
          if constexpr (VB == 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(t_o + 32 * c, o);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = zero ? 0.f : __uint_as_float(o[8 * k + e]) * norm;
                emit(32 * c + 8 * k, y);
              }
            }
          } else {
            constexpr int N = D == 256 ? 128 : D;
            float o[N];
            float4* half = reinterpret_cast<float4*>(sm + Sh::q);  // D = 256: the transform of the first half
#pragma unroll
            for (int p = 0; p < D / N; ++p) {
              {
                uint32_t* w = reinterpret_cast<uint32_t*>(o);
#pragma unroll
                for (int c = 0; c < N / 32; ++c)
                  tc::tmem_ld32_nw(t_o + p * N + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(w + 32 * c));
                tc::tmem_wait_ld();
              }
              thread_wht<N>(o);
              if (D == 256 && p == 0) {
#pragma unroll
                for (int c = 0; c < 32; ++c) half[r * 32 + (c ^ (r & 31))] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
              }
            }
#pragma unroll
            for (int k = 0; k < N / 8; ++k) {
              float y[8], z[8];
#pragma unroll
              for (int e = 0; e < 8; e += 4) {
                float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
                if (D == 256) b = half[r * 32 + ((2 * k + e / 4) ^ (r & 31))];
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int c = 8 * k + e + i;
                  const float sgn = norm * (float)a.c.tab.signs[c];
                  if (D == 256) {
                    y[e + i] = zero ? 0.f : (bb[i] + o[c]) * sgn;
                    z[e + i] = zero ? 0.f : (bb[i] - o[c]) * norm * (float)a.c.tab.signs[128 + c];
                  } else {
                    y[e + i] = zero ? 0.f : o[c] * sgn;
                  }
                }
              }
              emit(8 * k, y);
              if (D == 256) emit(128 + 8 * k, z);
            }
          }
        } else if (whole && valid) {
          const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int c = 0; c < D / 8; ++c) store8(a.c.out, a.c.out_dtype, out_at + 8 * c, z);
        }
        if (!whole) {
          // the last of the warpgroups that share the rows joins them, in the order of the key ranges
          __threadfence();
          tc::bar_sync(2 + wg, 128);
          int done = 0;
          if (r == 0) done = (int)atomicAdd(a.counters + it.counter + (it.two ? wg : 0), 1u) == parts - 1;
          const bool join = tc::bar_sync_or(2 + wg, 128, done != 0);
          if (join) {
            __threadfence();
            const int nrows = min(128, it.rows - (it.two ? 128 * wg : 0));
            const int per = D == 256 || it.two ? 1 : 2;  // partial results per CTA
            for (int i = r; i < nrows * (D / 8); i += 128) {
              const int jr = i / (D / 8), jc = i % (D / 8);
              float top = -INFINITY;
              for (int p = 0; p < parts; ++p) {
                const int ci = p / per;
                const long long sl_ = slot_of(it.first_cta + ci, ci == 0 ? 1 : 0, per == 2 ? p % 2 : wg);
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + sl_ * a.rows_cap * 2) + jr);
                if (ml.y != 0.f) top = fmaxf(top, ml.x);
              }
              if (top == -INFINITY) top = 0.f;
              float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, lt = 0.f;
              for (int p = 0; p < parts; ++p) {
                const int ci = p / per;
                const long long sl_ = slot_of(it.first_cta + ci, ci == 0 ? 1 : 0, per == 2 ? p % 2 : wg);
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + sl_ * a.rows_cap * 2) + jr);
                if (ml.y == 0.f) continue;
                const float w = ex2(ml.x - top);
                lt = fmaf(w, ml.y, lt);
                const float4* src = reinterpret_cast<const float4*>(a.part_o + (sl_ * a.rows_cap + jr) * D + 8 * jc);
                const float4 x0 = __ldcg(src), x1 = __ldcg(src + 1);
                acc[0] = fmaf(w, x0.x, acc[0]); acc[1] = fmaf(w, x0.y, acc[1]);
                acc[2] = fmaf(w, x0.z, acc[2]); acc[3] = fmaf(w, x0.w, acc[3]);
                acc[4] = fmaf(w, x1.x, acc[4]); acc[5] = fmaf(w, x1.y, acc[5]);
                acc[6] = fmaf(w, x1.z, acc[6]); acc[7] = fmaf(w, x1.w, acc[7]);
              }
              const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] *= inv;
              const int jrow = it.row0 + (it.two ? 128 * wg : 0) + jr, jt = jrow / a.c.G;
              const int jh = it.kvh * a.c.G + (jrow - jt * a.c.G);
              store8(a.c.out, a.c.out_dtype, ((long long)(it.tok0 + jt) * a.c.n_q_heads + jh) * D + 8 * jc, acc);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
    }
  }
  if (!ok && lane == 0) atomicOr(a.c.tab.status, kFlagTimeout);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int D, int VB>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t s) {
  auto kern = chunk_kernel<D, VB>;
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, kern);
  if (e != cudaSuccess) return e;
  if (at.numRegs * kThreads < kRegsNeeded) return cudaErrorLaunchOutOfResources;  // the split would wait for ever
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::alloc);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)sm_count), dim3(kThreads), Shape<D>::alloc, s, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D>
cudaError_t launch_d(const Args& a, int vb, int sm_count, cudaStream_t s) {
  switch (vb) {
    case 0: return launch<D, 0>(a, sm_count, s);
    case 1: return launch<D, 1>(a, sm_count, s);
    case 2: return launch<D, 2>(a, sm_count, s);
    default: return launch<D, 3>(a, sm_count, s);
  }
}

}  // namespace ck
}  // namespace tq
