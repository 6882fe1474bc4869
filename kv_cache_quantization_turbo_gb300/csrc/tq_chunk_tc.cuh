// Chunk attention on the fifth-generation tensor cores, for entries of more than a few rows.
//
// Per KV head, the rows of a sequence are its (new token, query head of the group) pairs, row = token * G + head.  An
// entry is up to MT consecutive rows and the key tiles that any of them sees (the plan kernel lists them).  The tiles of
// all entries of all KV heads form one line of work units, cut into equal ranges, one per CTA (one CTA per SM): a CTA
// takes the end of one entry, whole entries, and the start of another.  Entries that several CTAs share are joined from
// partial results by a second kernel, in a fixed order, so that results do not depend on timing.  With one
// decode row the long axis is so split over the whole GPU; with a large chunk every SM works to the end.  Where entries are so
// many and so alike that ranges of whole ones are nearly even, the plan does not cut them.
//
// A tile is BN keys.  A step is one score product S = Q K^T (M 128, N BN, K D), its softmax and O += P V (M 128, N D,
// K BN), the last two in parts of 64 keys.  Entries of more than 128 rows (D <= 128) have two row tiles, and steps
// alternate between them on one key tile; smaller ones have one, and steps alternate between two independent
// accumulators on successive key tiles, joined at the end like any other partial results.  Either way step u uses score
// buffer u % 2 and warpgroup u % 2, and the tensor core works for one while the other is in the softmax.  At D = 256
// tensor memory holds one accumulator, and one warpgroup takes every step.
//
// Warps, meeting on mbarriers only:
//   0-3, 4-7   softmax: one row per thread, 64 scores at a time.  The weights 2^(s - reference) are taken against the
//              reference so far; only where it is unset, or a row's 64 keys sum to more than fp16 weights can hold, does a
//              second reading find their maximum, raise the reference and rescale O in tensor memory.  Scores with
//              modifications or masks are changed in place before.  P as fp16 goes over S, the left operand of the value
//              product.
//   8-11, 12-15  producers of the K and of the V tiles: codes to fp16 values in swizzled operand tiles (K: K-major; the
//              same bytes read MN-major are V).  A q8_0 code becomes its value by a byte permute into 1024 + u, an exact
//              subtraction and one rounded product with the scale; a turbo code by byte permutes over the level table.
//   16, 17     issue the products, one warp for each softmax warpgroup: QK, PV, PV, QK, ... in order.  (One warp for both
//              took longer to go round than the products.)
//   18, 19     18 reads the plan; both find each key's place through the block table a few tiles ahead, and ask for its
//              bytes in L2
// The scales of fp16 operands: queries are multiplied by a power of two per row (any input type fits then), turbo
// values carry lambda so that the codebook is nearly exact in fp16.  Rounding to fp16 (2^-11 relative at most per
// operand) is what the tensor core's full rate asks for; sums are fp32.
//
// What bounds it.  Many rows: a tensor instruction of M 128, K 16 takes 65 cycles for any N up to 128 (measured alone),
// so a tile of two row tiles (32 instructions) takes 2.1 K cycles; it takes 4.9 K.  A row tile's steps follow one another
// (its scores and weights share one buffer): score product 0.95 K, two softmax parts of 64 keys with 0.4 K around each,
// value product 0.3 K.  The two row tiles' steps run side by side, so a tile takes as long as one of them, and most of
// that is the softmax: a part takes 0.43 K cycles alone and 1.0 K beside the producers, which convert every tile again
// for each entry and share the instruction slots of its SM sub-partition, as do the polls of barriers (5 K of 13.9 K
// instructions). Without the softmax the loop runs at 1.56 ms, without softmax and conversion at 1.22 ms, with both at
// 2.04 ms for a 4096-token chunk at 32K context, 32 query heads of 128; the call takes 2.05 ms (1.00 PFLOP/s), 0.5 % more
// since the join is a kernel of its own, which saves small batches most of their time (below, at join_kernel).  64-key
// score products with twice the buffers take the same 65 cycles each for half the keys: 2.15 ms.  Few rows: a tile is
// 34.8 KB of cache, 1.5 K cycles of this GPU's bandwidth; it takes 3.5 K, bound by the round of a tile through its two
// buffers.  Entries of up to 16 rows have a kernel of their own (tq_chunk_few.cuh).
//
// Error against fp64 (2-norm of all outputs, N(0, 1) queries, 1 % of the channels 20 times larger): 512 tokens at 32K, fp16,
// 2.0e-3; 4096 tokens, bf16, 2.7e-3, of which the output's type is 1.6e-3; without such channels 5e-4.  Nearly all of it is
// the rounding of scale * code in K, 2^-12 of each product at most: the scales of a key differ by block of 32, so exact
// codes would want a score product, and its scores in tensor memory, for each block.
#pragma once

#include "tq_batch.cuh"
#include "tq_chunk.h"
#include "tq_tc.cuh"

namespace tq {
namespace ck {

constexpr int kThreads = 640;
constexpr int kProdWarps = 8;
constexpr int kIssuer = 16, kLocator = 18, kLocWarps = 2;
constexpr int NI = 3;       // items known ahead
constexpr int NL = 6;       // tiles located ahead of the producers
constexpr int kMissRing = 16;
constexpr float kBias = 4.0f;     // a fresh reference makes the row's largest weight 2^kBias
constexpr float kTop = 32768.0f;  // the reference is raised where a tile's weights sum to more: each is below 65504
constexpr float kLog2e = 1.4426950408889634074f;
// Registers per thread after the split; its sum has to be within the launch's (checked at the launch).
constexpr int kRegsSoftmax = 136, kRegsProducer = 72, kRegsOther = 64;
constexpr int kRegsNeeded = 256 * kRegsSoftmax + 32 * kProdWarps * kRegsProducer + 128 * kRegsOther;
static_assert(kRegsNeeded <= kThreads * 96, "register split");

constexpr int HN = 64;  // keys of a part

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
  static constexpr int words = miss + kMissRing * 16;  // uint32 [kMissRing][2][8]: f8_block words of a tile's K and V
  static constexpr int rs = words + kMissRing * 64;    // float [256]: row scales
  static constexpr int items = rs + 256 * 4;           // Item [NI]
  static constexpr int tab = items + NI * 128;         // fp16 [8]: the V codebook
  static constexpr int bars = tab + 16;
  static constexpr int total = bars + 64 * 8;
  static constexpr int alloc = total + 1024;
  static_assert(alloc <= 227 * 1024, "shared memory");
  static constexpr int PH = BN / HN;                   // parts of a step
  // At 256 the first issuer has every step and the second takes no part: it would poll through the whole of every item.
  static constexpr int kIssuers = D == 256 ? 1 : 2;
  static constexpr int kItemReaders = 8 + kProdWarps + kIssuers + kLocWarps - 1;  // (the first locator writes the items)
  // tensor memory columns: S [2][BN], O [kQTiles][D]
  static constexpr int tO = 2 * BN;
  static_assert(tO + kQTiles * D <= 512, "tensor memory");
};

struct Item {
  int kind;        // 0: no more; 1: tiles; 2: rows that see nothing
  int kvh, seq, tok0, pos0, len, prefix;
  int row0, rows;  // of the sequence's rows
  int lo, hi;      // keys that some row sees
  int tile, n;     // key tiles of this CTA, the first s_n of them sinks ahead of the windows: tile_of()
  int s_n, s_lo, s_hi, s_tile;
  int two;         // two row tiles
  int first_cta, n_ctas, slot;  // CTAs that share the entry; this CTA's partial slot
  int counter;
};
static_assert(sizeof(Item) <= 128, "item");

// Number of the CTA's tile j; the keys wanted from it.
__device__ __forceinline__ int tile_of(const Item& it, int j) { return (j < it.s_n ? it.s_tile : it.tile) + j; }
__device__ __forceinline__ int2 keys_of(const Item& it, int j) {
  return j < it.s_n ? make_int2(it.s_lo, it.s_hi) : make_int2(it.lo, it.hi);
}

struct Bars {
  uint64_t k_full[3], k_free[3], v_full[3], v_free[3];
  uint64_t s_done[2], p_full[4], pv_done[4];  // per buffer, per buffer and part
  // q_full is one per item slot: nothing makes the softmax warps wait for an issuer without a step in an item, and with one
  // barrier for all items they could complete a second phase before it has seen the first.  An item slot is written again
  // only once all have left the item.
  uint64_t turn[2][4];  // (staged kernel) of softmax warp w % 4 of each warpgroup: its partner has done a step
  uint64_t drained[2], q_full[NI], item_full[NI], item_free[NI], loc_full[NL], loc_free[NL];
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 64 * 8, "barriers");

// Byte offset of (row, 16-byte chunk of 8 elements) in an operand tile of R rows: 64-element blocks of R 128-byte rows,
// chunks of a row XOR-swizzled by the row.
template <int R>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (uint32_t)((chunk >> 3) * (128 * R) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c tanh(s / c) of a score s in log2 units; c2 = c log2 e, i2 = 2 / c (cap_factors).  With z = 2 (s / c) log2 e it is
// c (1 - 2 / (1 + 2^z)), whose difference keeps about 2.5e-7 of c and nothing of an s far below that: where |s / c| is
// below 1/4 its series s (1 - y^2 / 3 + 2 y^4 / 15 - 17 y^6 / 315), y = z ln 2 / 2, is taken instead (62 y^8 / 2835 is
// left out: 3.4e-7 relative at most).  So the error is 1e-6 relative for every c; a c that no score comes near leaves s.
// (Eight chunks of up to 700 tokens, 256 wide, capped: 58.7 us without the series, 60.6 with it.)
__device__ __forceinline__ float cap_score(float s, float c2, float i2) {
  constexpr float kY2 = 0.12011325347955035f;  // (ln 2 / 2)^2
  const float z = s * i2, w = z * z;
  const float far = c2 * (1.f - __fdividef(2.f, 1.f + ex2(z)));
  const float near = s * fmaf(w, fmaf(w, fmaf(w, -17.f / 315.f * kY2 * kY2 * kY2, 2.f / 15.f * kY2 * kY2), -kY2 / 3.f), 1.f);
  return fabsf(z) < 0.72134752f ? near : far;  // |y| < 1/4
}
// c2 and i2 of a cap c > 0, finite for the smallest and the largest (a score of 0 stays 0).
__device__ __forceinline__ float2 cap_factors(float c) {
  return make_float2(fminf(c * 1.4426950408889634f, 3.4e38f), fminf(2.f / c, 3.4e38f));
}

// Waits for this thread's tensor-memory loads, x among them (an operand, so that no use of x moves before the wait).
__device__ __forceinline__ void loaded(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                 "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]),
                 "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                 "+r"(x[30]), "+r"(x[31])::"memory");
}
__device__ __forceinline__ void loaded(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]),
                 "+r"(x[15])::"memory");
}
// 64 consecutive columns of this warp's tensor-memory lanes, waited for in the same statement: no use of x can move
// before the wait, and no register is copied to keep it so.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&x)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
        "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
        "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
        "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31]),
        "=r"(x[32]), "=r"(x[33]), "=r"(x[34]), "=r"(x[35]), "=r"(x[36]), "=r"(x[37]), "=r"(x[38]), "=r"(x[39]),
        "=r"(x[40]), "=r"(x[41]), "=r"(x[42]), "=r"(x[43]), "=r"(x[44]), "=r"(x[45]), "=r"(x[46]), "=r"(x[47]),
        "=r"(x[48]), "=r"(x[49]), "=r"(x[50]), "=r"(x[51]), "=r"(x[52]), "=r"(x[53]), "=r"(x[54]), "=r"(x[55]),
        "=r"(x[56]), "=r"(x[57]), "=r"(x[58]), "=r"(x[59]), "=r"(x[60]), "=r"(x[61]), "=r"(x[62]), "=r"(x[63])
      : "r"(taddr)
      : "memory");
}
// Stores 16 consecutive 32-bit columns of this warp's tensor-memory lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// A wait that gives up for good once one has run out: the role then runs through its loops without waiting (every
// named barrier is still met), and the error is reported at the end.
// Polls without a suspend-time hint (with one of 1 us waits took longer); 2^23 polls are some tenths of a second at least.
// SLEEP: nanoseconds between polls, for roles with time in hand (polling takes instruction slots
// from the others).
template <int SLEEP = 0>
__device__ __forceinline__ void wait(bool& ok, uint64_t* bar, uint32_t parity) {
  if (!ok) return;
  uint32_t done = 0;
  const uint32_t at = tc::smem_addr(bar);
  for (int i = 0; i < (1 << 23) && !done; ++i) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(at), "r"(parity & 1u)
        : "memory");
    if (SLEEP > 0 && !done) __nanosleep(SLEEP);
  }
  ok = done != 0;
}

// A value that all lanes share, in a form that the compiler knows to be shared.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFull, x, 0); }

// Four tensor instructions of the lane with one = 1, K = 64 in all: D += A B^T.  Descriptors as low word and the common
// high word; acc = 0 starts the sum.  mma4_ss: A and B K-major in shared memory, one 64-element block of each.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc,
                                        uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a, b;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.u32 e, %6, 0;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t"
      "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\tmov.b64 x, {a, %3};\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(one));
}
// mma4_ts: A in tensor memory (8 columns per instruction), B MN-major (2048 bytes per instruction).
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc,
                                        uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a, b;\n\t.reg .b64 y;\n\t"
      "setp.ne.u32 e, %6, 0;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\tmov.b64 y, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(one));
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(tc::smem_addr(bar)),
      "r"(one)
      : "memory");
}

// The same for a whole warp, whose lanes stay of one mind.
template <int SLEEP = 0>
__device__ __forceinline__ void wait_warp(bool& ok, uint64_t* bar, uint32_t parity) {
  wait<SLEEP>(ok, bar, parity);
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

// A duplicated scale clamped to where 127 times it is finite in fp16.
__device__ __forceinline__ uint32_t clamp_scale(uint32_t s2) {
  const uint32_t lim = 0x5FFE5FFEu, nlim = 0xDFFEDFFEu;  // 511.5
  const __half2 h = __hmax2(__hmin2(*reinterpret_cast<const __half2*>(&s2), *reinterpret_cast<const __half2*>(&lim)),
                            *reinterpret_cast<const __half2*>(&nlim));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four e4m3 codes to two fp16 pairs, exact.
__device__ __forceinline__ void f8_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
// The exponent of an f8_block word's scale, and the scale.
__device__ __forceinline__ int f8_exponent(uint32_t w) { return (int)(w >> 23 & 255u) - 127; }
__device__ __forceinline__ float f8_scale(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The word of a block that is not there: the smallest scale, which moves no other block's, and no marks.
constexpr uint32_t kF8None = (uint32_t)(kF8MinExp + 127) << 23;

// f8_block.  A row's output is a sum of weights times 2^(exponent of V's block) times codes, and its weights go to fp16 with
// that power: s + exponent, s the score in log2 units, is what has to stay within fp16's range, for the keys that the row
// sees.  So a row has two references, integers (powers of two then move between weights, sum and accumulator exactly): m of
// its scores, for the sum l, and m + ve of s + exponent, for O, which is in units of 2^ve.  Raises them to kBias below
// top and top_v, the largest s and s + exponent of the keys at hand (-INFINITY: none), with the sum; returns O's factor.
__device__ __forceinline__ float raised(float& m, float& ve, float& l, float top, float top_v) {
  const float mn = fmaxf(m, rintf(top) - kBias), mv = m + ve, mvn = fmaxf(mv, rintf(top_v) - kBias);
  const float al = mvn == -INFINITY ? 1.f : ex2(mv - mvn);
  l *= mn == -INFINITY ? 1.f : ex2(m - mn);
  m = mn;
  ve = mn == -INFINITY ? 0.f : mvn - mn;
  return al;
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
// the CTA's items, in order
// ---------------------------------------------------------------------------
template <int D>
struct Items {
  long long T, U, nC, u, u1;
  int n_entries, h, e, whole;

  // A quotient of numbers >= 0; those of fewer than 32 bits, as good as always, are divided as such.
  static __device__ __forceinline__ long long div(long long x, long long y) {
    return ((unsigned long long)(x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
  }

  // the CTA whose range holds a unit
  __device__ __forceinline__ int cta_of(long long x) const { return (int)div((x + 1) * nC - 1, U); }

  __device__ void start(const Args& a) {
    const PlanHead head = *a.plan;
    T = head.units;
    n_entries = head.n_entries;
    U = T * a.c.k.H;
    // every CTA that takes part has at least kMinUnits units (so no CTA inside an entry's range is without work)
    whole = head.whole;
    nC = whole ? (long long)gridDim.x : max(1LL, min((long long)gridDim.x, U / kMinUnits));
    const long long c = blockIdx.x;
    u = c < nC ? div(U * c, nC) : 0;
    u1 = c < nC ? div(U * (c + 1), nC) : 0;
    h = e = 0;
    if (u < u1) {
      h = (int)div(u, T);
      const long long off = u - (long long)h * T;
      for (int step = 1 << 30; step > 0; step >>= 1)  // the last entry that starts at or before off
        if (e + step < n_entries && a.entries[e + step].start <= off) e += step;
      if (whole && a.entries[e].start < off && ++e == n_entries) {
        e = 0;
        ++h;
      }
      if (whole) u = h < a.c.k.H ? (long long)h * T + a.entries[e].start : U;
    }
  }

  __device__ void next(const Args& a, Item& it) {
    it.kind = 0;
    it.n = 0;
    while (u < u1 && it.kind == 0) {
      const Entry en = a.entries[e];
      const long long base = (long long)h * T + en.start;
      it.kvh = h;
      it.seq = en.seq;
      it.row0 = en.row0;
      it.rows = en.rows;
      it.tok0 = en.tok0;
      it.pos0 = en.pos0;
      it.len = en.len;
      it.prefix = en.prefix;
      it.lo = en.lo;
      it.hi = en.hi;
      it.two = D != 256 && it.rows > 128;
      it.counter = (h * n_entries + e) * 2;
      const long long t0 = max(0LL, u - base - kOverhead);
      const long long t1 = whole ? en.n_tiles : min((long long)en.n_tiles, u1 - base - kOverhead);
      if (en.n_tiles == 0) {
        it.kind = u == base ? 2 : 0;  // by the CTA that holds its first unit
      } else if (t0 < t1) {
        it.kind = 1;
        it.tile = en.lo / Shape<D>::BN + (int)t0;
        it.n = (int)(t1 - t0);
        it.s_n = 0;
        if (en.s_tiles) {
          it.tile -= en.s_tiles;
          it.s_lo = en.s_lo;
          it.s_hi = en.s_hi;
          it.s_tile = en.s_lo / Shape<D>::BN + (int)t0;
          it.s_n = max(0, min(en.s_tiles, (int)t1) - (int)t0);
        }
        it.first_cta = whole ? (int)blockIdx.x : cta_of(base + kOverhead);
        it.n_ctas = whole ? 1 : cta_of(base + kOverhead + en.n_tiles - 1) - it.first_cta + 1;
        it.slot = t0 == 0 ? 1 : 0;
      }
      u = base + en.n_tiles + kOverhead;
      if (++e == n_entries) {
        e = 0;
        ++h;
      }
    }
  }
};

// ---------------------------------------------------------------------------
// locator: the vector of every key of a tile, and its bytes asked for in L2
// ---------------------------------------------------------------------------
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The two locator warps take half of a tile's rows each; lane's rows are BN / 2 * half + lane + 32 i.  page[i] is the
// physical page of a row, read one tile ahead.
template <int D>
__device__ __forceinline__ void read_pages(const Args& a, const Item& it, int tile, int half, int lane,
                                           int (&page)[Shape<D>::BN / 64]) {
  const DevBatch& b = a.c.b;
  const int t = tile_of(it, tile);
  const int2 keys = keys_of(it, tile);
#pragma unroll
  for (int i = 0; i < Shape<D>::BN / 64; ++i) {
    const int j = t * Shape<D>::BN + Shape<D>::BN / 2 * half + 32 * i + lane;
    const int lp = (int)((uint32_t)j / (uint32_t)a.c.k.page_size);
    page[i] = b.block_table ? -1 : it.seq;
    if (b.block_table && j >= keys.x && j < keys.y && lp < b.max_blocks)
      page[i] = __ldg(b.block_table + (long long)it.seq * b.max_blocks + lp);
  }
}

template <int D, int VB>
__device__ __forceinline__ void locate_tile(const Args& a, const Item& it, int tile, int half, int lane,
                                            const int (&page)[Shape<D>::BN / 64], long long* loc, uint32_t* miss,
                                            uint32_t* words) {
  constexpr int BN = Shape<D>::BN;
  const DevView &K = a.c.k, &V = a.c.v;
  const int t = tile_of(it, tile);
  const int2 keys = keys_of(it, tile);
  const long long first = (long long)a.c.layer * K.num_pages;
#pragma unroll
  for (int i = 0; i < BN / 64; ++i) {
    const int at = BN / 2 * half + 32 * i + lane, j = t * BN + at;
    const bool want = j >= keys.x && j < keys.y;
    const bool on = want && page[i] >= 0 && page[i] < K.num_pages;
    const int off = j - (int)((uint32_t)j / (uint32_t)K.page_size) * K.page_size;
    const long long vec = on ? ((first + page[i]) * K.H + it.kvh) * K.page_size + off : -1;
    loc[at] = vec;
    const uint32_t m = __ballot_sync(kFull, want && !on);
    if (lane == 0) {
      miss[BN / 64 * half + i] = m;
      if (m) atomicOr(a.c.tab.status, kFlagBlockTable);
    }
    if (on) {
      // (a line per lane: bulk requests for the runs of a page measured 7 % slower on a paged decode batch)
      const unsigned char* pk = K.payload + vec * D;
      const unsigned char* pv = V.payload + vec * V.pay_bytes;
      prefetch_l2(pk);
      prefetch_l2(pv);
      if constexpr (D == 256) {
        prefetch_l2(pk + 128);
        if (V.pay_bytes > 128) prefetch_l2(pv + 128);
      }
      if constexpr (VB != kF8) {
        prefetch_l2(K.header + vec * K.hdr_bytes);
        prefetch_l2(V.header + vec * V.hdr_bytes);
      }
    }
    if constexpr (VB == kF8) {  // the words of the two blocks: lanes 0 and 16 K's, 1 and 17 V's
      const uint32_t there = __ballot_sync(kFull, on) >> (lane & 16) & 0xFFFFu;
      const long long some = __shfl_sync(kFull, vec, (lane & 16) + (there ? __ffs(there) - 1 : 0));
      if ((lane & 14) == 0) {
        const unsigned char* hdr = lane & 1 ? V.header : K.header;
        words[8 * (lane & 1) + (BN / 2 * half + 32 * i + (lane & 16)) / 16] =
            there ? __ldg(reinterpret_cast<const uint32_t*>(hdr) + some / kF8Block) : kF8None;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------

// Loads that leave zeros where on is false, without a branch around them and without a use of the value: all of a
// tile's loads are in flight at once.
__device__ __forceinline__ uint4 load16(const void* p, bool on) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "l"(p), "r"((uint32_t)on));
  return v;
}
__device__ __forceinline__ uint32_t load4(const void* p, bool on) {
  uint32_t v = 0u;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.nc.u32 %0, [%1];\n\t}\n"
               : "+r"(v)
               : "l"(p), "r"((uint32_t)on));
  return v;
}
__device__ __forceinline__ uint16_t load2(const void* p, bool on) {
  uint16_t v = 0;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.nc.u16 %0, [%1];\n\t}\n"
               : "+h"(v)
               : "l"(p), "r"((uint32_t)on));
  return v;
}

// Four warps make the K tiles, four the V tiles.  A thread's units (16 coordinates each) of a tile: rows row0 + 32 i, and
// of each the quarter lane % 4 of every 64 coordinates; row i of the next tile is asked for as soon as row i of this one
// is converted.  The eight lanes that a 16-byte store is served together for are then two neighbouring rows of four
// chunks, all in different banks; a row's place is looked up once for all its blocks.
template <int D, int VB>
struct Producer {
  static constexpr int BN = Shape<D>::BN;
  static constexpr int RN = BN / 32, BK = D / 64;  // rows and 64-blocks per thread
  static_assert(kProdWarps / 2 * 8 == 32, "rows per pass");

  static constexpr bool kBytes = VB == 0 || VB == kF8;  // V's codes are bytes

  struct RawK {
    uint4 w[RN][BK];
    uint32_t k[VB == kF8 ? 1 : RN][BK];               // K scales of the two 32-blocks of a 64-block
    uint32_t v[VB == kF8 ? 1 : RN][VB == 0 ? BK : 1];  // V scales, or the norm
  };
  struct RawV {
    uint32_t s[VB == kF8 ? 1 : RN][VB == 0 ? BK : 1];  // scales, or the norm
    uint4 w[kBytes ? RN : 1][BK];
    uint32_t c[VB == 2 ? RN : 1][BK];                  // 16 codes of 2 bits
    uint16_t h[VB & 1 ? RN : 1][BK][VB == 3 ? 3 : 1];  // 16 codes of 1 or 3 bits
  };

  static __device__ __forceinline__ int row_of(int ptid, int i) { return 32 * i + (ptid >> 2); }

  // Row i of a located tile.
  static __device__ __forceinline__ void load_k(const Args& a, const long long* loc, int ptid, int i, RawK& r) {
    const DevView &K = a.c.k, &V = a.c.v;
    const int c = ptid & 3;
    const long long vec = loc[row_of(ptid, i)];
    const bool on = vec >= 0;
    const unsigned char* pk = K.payload + vec * D + 16 * c;
    if constexpr (VB == kF8) {
#pragma unroll
      for (int b = 0; b < BK; ++b) r.w[i][b] = load16(pk + 64 * b, on);
      return;
    }
    const unsigned char* hk = K.header + vec * (D / 16);
    const unsigned char* hv = V.header + vec * (VB == 0 ? D / 16 : 2);
#pragma unroll
    for (int b = 0; b < BK; ++b) r.w[i][b] = load16(pk + 64 * b, on);
#pragma unroll
    for (int b = 0; b < BK; ++b) r.k[i][b] = load4(hk + 4 * b, on);
    if constexpr (VB == 0) {
#pragma unroll
      for (int b = 0; b < BK; ++b) r.v[i][b] = load4(hv + 4 * b, on);
    } else {
      r.v[i][0] = load2(hv, on);
    }
  }

  static __device__ __forceinline__ void load_v(const Args& a, const long long* loc, int ptid, int i, RawV& r) {
    const DevView& V = a.c.v;
    const int c = ptid & 3;
    const long long vec = loc[row_of(ptid, i)];
    const bool on = vec >= 0;
    const unsigned char* p = V.payload + vec * (kBytes ? D : D * VB / 8) + (kBytes ? 16 : 2 * VB) * c;
    const unsigned char* hv = V.header + vec * (VB == 0 ? D / 16 : 2);
#pragma unroll
    for (int b = 0; b < BK; ++b) {
      if constexpr (kBytes) r.w[i][b] = load16(p + 64 * b, on);
      if constexpr (VB == 0) r.s[i][b] = load4(hv + 4 * b, on);
      if constexpr (VB == 2) r.c[i][b] = load4(p + 16 * b, on);
      if constexpr (VB == 1 || VB == 3) {
#pragma unroll
        for (int k = 0; k < VB; ++k) r.h[i][b][k] = load2(p + 8 * VB * b + 2 * k, on);
      }
    }
    if constexpr (!kBytes) r.s[i][0] = load2(hv, on);
  }

  // The same for 16 e4m3 codes.
  static __device__ __forceinline__ void put_f8(unsigned char* tile, uint32_t c0, uint32_t c1, const uint4& w) {
    uint4 h;
    f8_pairs(w.x, h.x, h.y);
    f8_pairs(w.y, h.z, h.w);
    *reinterpret_cast<uint4*>(tile + c0) = h;
    f8_pairs(w.z, h.x, h.y);
    f8_pairs(w.w, h.z, h.w);
    *reinterpret_cast<uint4*>(tile + c1) = h;
  }

  // Converts the 16 codes of a q8_0 unit and stores them as chunks 2 c, 2 c + 1 of 64-block b of a row; at: the
  // chunks' offsets in the block, c0 and c1.
  static __device__ __forceinline__ void put_q8(unsigned char* tile, uint32_t c0, uint32_t c1, const uint4& w,
                                                uint32_t s2) {
    uint32_t x, y;
    uint4 h;
    q8_pairs(w.x, x, y);
    h.x = mul_h2(x, s2);
    h.y = mul_h2(y, s2);
    q8_pairs(w.y, x, y);
    h.z = mul_h2(x, s2);
    h.w = mul_h2(y, s2);
    *reinterpret_cast<uint4*>(tile + c0) = h;
    q8_pairs(w.z, x, y);
    h.x = mul_h2(x, s2);
    h.y = mul_h2(y, s2);
    q8_pairs(w.w, x, y);
    h.z = mul_h2(x, s2);
    h.w = mul_h2(y, s2);
    *reinterpret_cast<uint4*>(tile + c1) = h;
  }

  // The thread's half of a pair of scales, duplicated.
  static __device__ __forceinline__ uint32_t scale_of(uint32_t pair, int c) {
    return __byte_perm(pair, 0u, c & 2 ? 0x3232 : 0x1010);
  }

  static __device__ __forceinline__ void convert_k(const RawK& r, unsigned char* tile, int ptid, int i) {
    const int c = ptid & 3, row = row_of(ptid, i);
    const uint32_t c0 = tile_at<BN>(row, 2 * c), c1 = tile_at<BN>(row, 2 * c + 1);
#pragma unroll
    for (int b = 0; b < BK; ++b) {
      if constexpr (VB == kF8) {
        put_f8(tile + b * (128 * BN), c0, c1, r.w[i][b]);
        continue;
      }
      const uint32_t sk = scale_of(r.k[i][b], c);
      const uint32_t sv = VB == 0 ? scale_of(r.v[i][VB == 0 ? b : 0], c) : r.v[i][0];
      uint32_t s2 = clamp_scale(sk);
      // a key whose stored K or V is not finite poisons the scores of the rows that see it (the value product of the
      // others must not meet it)
      if (not_finite(sk) || not_finite(sv)) s2 = 0x7E007E00u;
      put_q8(tile + b * (128 * BN), c0, c1, r.w[i][b], s2);
    }
  }

  static __device__ __forceinline__ void convert_v(const RawV& r, const uint32_t (&tab)[4], unsigned char* tile, int ptid,
                                                   int i) {
    const int c = ptid & 3, row = row_of(ptid, i);
    const uint32_t c0 = tile_at<BN>(row, 2 * c), c1 = tile_at<BN>(row, 2 * c + 1);
#pragma unroll
    for (int b = 0; b < BK; ++b) {
      if constexpr (VB == kF8) {
        put_f8(tile + b * (128 * BN), c0, c1, r.w[i][b]);
      } else if constexpr (VB == 0) {
        const uint32_t s = scale_of(r.s[i][b], c);
        put_q8(tile + b * (128 * BN), c0, c1, r.w[i][b], not_finite(s) ? 0u : clamp_scale(s));
      } else {
        const uint32_t s2 = not_finite(r.s[i][0]) ? 0u : r.s[i][0] * 0x10001u;
        uint64_t codes;
        if constexpr (VB == 2) codes = r.c[i][b];
        else if constexpr (VB == 1) codes = r.h[i][b][0];
        else codes = (uint64_t)r.h[i][b][0] | ((uint64_t)r.h[i][b][VB - 2] << 16) | ((uint64_t)r.h[i][b][VB - 1] << 32);
        uint32_t h[8];
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // four codes: nibble selectors of byte permutes over the level table
          const uint32_t x = (uint32_t)(codes >> (4 * VB * g));
          constexpr uint32_t m = (1u << VB) - 1u;
          const uint32_t sel = (x & m) | ((x << (4 - VB)) & (m << 4)) | ((x << (8 - 2 * VB)) & (m << 8)) |
                               ((x << (12 - 3 * VB)) & (m << 12));
          const uint32_t lb = __byte_perm(tab[0], tab[1], sel), hb = __byte_perm(tab[2], tab[3], sel);
          h[2 * g] = mul_h2(__byte_perm(lb, hb, 0x5140), s2);
          h[2 * g + 1] = mul_h2(__byte_perm(lb, hb, 0x7362), s2);
        }
        *reinterpret_cast<uint4*>(tile + b * (128 * BN) + c0) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(tile + b * (128 * BN) + c1) = make_uint4(h[4], h[5], h[6], h[7]);
      }
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
  constexpr int W = sizeof(T) / 2;         // 16-byte words of 8 elements
  constexpr int U = 8 / W;                 // rows in flight
  const int c = lane % LQ, G = a.c.G;
  for (int r0 = warp * RP + lane / LQ; __any_sync(kFull, r0 < it.rows); r0 += 8 * RP * U) {
    uint4 raw[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 8 * RP * u, row = it.row0 + r, i = row / G, g = row - i * G;
      const T* src = q + (long long)(it.tok0 + i) * a.c.q_stride + (long long)(it.kvh * G + g) * D + 8 * c;
#pragma unroll
      for (int k = 0; k < W; ++k) raw[u][k] = load16(reinterpret_cast<const uint4*>(src) + k, r < it.rows);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 8 * RP * u;
      float x[8];
      load_row<8>(reinterpret_cast<const T*>(raw[u]), x);
      uint32_t top = 0;  // bits of the largest magnitude (NaN above all)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
      for (int m = 1; m < LQ; m <<= 1) top = max(top, __shfl_xor_sync(kFull, top, m));
      uint32_t ex = min(max(top >> 23, 1u), 253u);
      if (top >= 0x7F800000u) ex = 127u;  // infinite or NaN: as it is
      const float f = a.q_sign * __uint_as_float((254u - ex) << 23);
      if (r < it.rows) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = narrow(x[2 * e] * f, x[2 * e + 1] * f, (const __half*)nullptr);
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

// ---------------------------------------------------------------------------
// the issuer of warpgroup w: its products, QK, PV, PV, QK, ... in order (D = 256: all)
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void issue_products(Bars* B, const Item* items, uint32_t sb, uint32_t tmem, int w, int lane,
                                               bool& ok) {
  using Sh = Shape<D>;
  constexpr int BN = Sh::BN, NB = Sh::NB, PH = Sh::PH;
  int icnt = 0, gt = 0;  // items and key tiles so far
  // The whole warp runs the same code, one lane's predicate on the tensor instructions: descriptors and addresses
  // then stay in uniform registers, where those instructions take them from.  (With one lane in a branch, every
  // operand was moved there first, and issuing a product took longer than the product.)
  const uint32_t one = lane == 0;
  int c = 0;  // this warpgroup's steps so far
  auto buffer = [&](int x) { return D == 256 ? x & 1 : w; };
  auto phase = [&](int x) { return D == 256 ? x >> 1 : x; };
  constexpr uint32_t id_qk = tc::idesc_f16_f32(128, BN);
  constexpr uint32_t id_pv = tc::idesc_f16_f32(128, D) | (1u << 16);  // B (V) MN-major
  const uint32_t hi = (uint32_t)(tc::desc_sw128(0) >> 32);  // the same for all operands
  const uint32_t q_lo = (uint32_t)tc::desc_sw128(sb + Sh::q), k_lo = (uint32_t)tc::desc_sw128(sb + Sh::k);
  const uint32_t v_lo = (uint32_t)tc::desc_sw128_mn(sb + Sh::v, BN * 128);
  for (;; ++icnt) {
    const int is = icnt % NI;
    wait_warp(ok, &B->item_full[is], icnt / NI);
    const int kind = uniform(items[is].kind), n = uniform(items[is].n), two = uniform(items[is].two);
    if (!ok || kind == 0) break;
    wait_warp(ok, &B->q_full[is], icnt / NI);
    if (kind == 1) {
      // own steps: every tile with two row tiles, else every other one; D = 256: all
      const int first = two || D == 256 ? 0 : w, stride = two || D == 256 ? 1 : 2;
      const int steps = (n - first + stride - 1) / stride;
      const uint32_t dq = q_lo + (uint32_t)(two ? w * (Sh::kQTile >> 4) : 0);
      const bool alone = !two;  // no other issuer uses the tile
      auto qk = [&](int i) {
        const int j = gt + first + stride * i, b = j % NB, s = buffer(c + i);
        wait_warp(ok, &B->k_full[b], j / NB);
        if (!ok) return;
        // (no tcgen05 fence: K comes through shared memory, and the score buffer's last readers were seen by the
        // value product that took their weights)
        const uint32_t dk = k_lo + (uint32_t)(b * (Sh::kTileB >> 4));
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          mma4_ss(tmem + s * BN, dq + kb * (128 * 128 >> 4), dk + kb * (128 * BN >> 4), hi, id_qk, kb > 0, one);
        commit(&B->s_done[s], one);
        commit(&B->k_free[b], one);
        if (alone) commit(&B->k_free[b], one);
      };
      auto pv = [&](int i) {
        const int j = gt + first + stride * i, b = j % NB, s = buffer(c + i);
        wait_warp(ok, &B->v_full[b], j / NB);
#pragma unroll
        for (int h = 0; h < PH; ++h) {
          wait_warp(ok, &B->p_full[s * PH + h], phase(c + i));
          if (!ok) return;
          tc::fence_after_sync();
          mma4_ts(tmem + Sh::tO + w * D, tmem + s * BN + h * (HN / 2),
                  v_lo + (uint32_t)(b * (Sh::kTileB >> 4) + h * (HN * 128 >> 4)), hi, id_pv, i > 0 || h > 0, one);
          commit(&B->pv_done[s * PH + h], one);
        }
        commit(&B->v_free[b], one);
        if (alone) commit(&B->v_free[b], one);
      };
      // D = 256: one score buffer ahead; else a step's score product needs the buffer of the step before
      constexpr int kAhead = D == 256 ? 1 : 0;
      if (steps > 0) qk(0);
      for (int i = 0; i < steps && ok; ++i) {
        if (kAhead && i + 1 < steps) qk(i + 1);
        pv(i);
        if (!kAhead && i + 1 < steps) qk(i + 1);
      }
      c += steps;
      gt += n;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
  }
  commit(&B->drained[w], one);  // products still in flight end before the tensor memory is freed
  tc::mbar_wait(&B->drained[w], 0u, 1 << 16);
}

// Partial slots: [CTA][start or end of its range][warpgroup], O and then m and l of each.
__device__ __forceinline__ long long partial_slot(int cta, int which, int w) { return ((long long)cta * 2 + which) * 2 + w; }

// Four columns from 4 jc on of row `row` of a sequence.
__device__ __forceinline__ void store4(const Args& a, int D, int kvh, int tok0, int row, int jc, const float (&y)[4]) {
  const int t = row / a.c.G, head = kvh * a.c.G + (row - t * a.c.G);
  const long long at = ((long long)(tok0 + t) * a.c.n_q_heads + head) * D + 4 * jc;
  if (a.c.out_dtype == TQ_DTYPE_F32) store_row<4>(static_cast<float*>(a.c.out) + at, y);
  else if (a.c.out_dtype == TQ_DTYPE_F16) store_row<4>(static_cast<__half*>(a.c.out) + at, y);
  else store_row<4>(static_cast<__nv_bfloat16*>(a.c.out) + at, y);
}

// Partial results `shares` of one row, columns jc0, jc0 + step, ... (C of them) below D / 4, joined in the order of the shares;
// share(p): slot of share p.  S shares' loads are in flight together; what a share without weight holds is not looked at.
template <int D, int C, int S, class Share>
__device__ __forceinline__ void join_columns(const Args& a, int shares, int row, int jc0, int step, Share share,
                                             float (&acc)[C][4]) {
  auto ml_of = [&](int p) {
    return __ldcg(reinterpret_cast<const float2*>(a.part_ml + share(min(p, shares - 1)) * a.rows_cap * 2) + row);
  };
  float2 ml[S];
  float4 x[S][C];
  auto ask = [&](int p0) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (p0 + k >= shares) break;  // (the block's threads alike)
      ml[k] = ml_of(p0 + k);
      const float4* o = reinterpret_cast<const float4*>(a.part_o + share(p0 + k) * a.rows_cap * D) + row;
#pragma unroll
      for (int c = 0; c < C; ++c) x[k][c] = __ldcg(o + (long long)min(jc0 + c * step, D / 4 - 1) * a.rows_cap);
    }
  };
  ask(0);
  float top = -INFINITY, lt = 0.f;
#pragma unroll
  for (int k = 0; k < S; ++k) top = fmaxf(top, k < shares && ml[k].y != 0.f ? ml[k].x : -INFINITY);
#pragma unroll 1
  for (int p0 = S; p0 < shares; p0 += 8) {
    float2 z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = ml_of(p0 + k);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, z[k].y != 0.f ? z[k].x : -INFINITY);
  }
  if (top == -INFINITY) top = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
#pragma unroll 1
  for (int p0 = 0; p0 < shares; p0 += S) {
    if (p0) ask(p0);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (p0 + k >= shares || ml[k].y == 0.f) continue;
      const float w = ex2(ml[k].x - top);
      lt = fmaf(w, ml[k].y, lt);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        acc[c][0] = fmaf(w, x[k][c].x, acc[c][0]);
        acc[c][1] = fmaf(w, x[k][c].y, acc[c][1]);
        acc[c][2] = fmaf(w, x[k][c].z, acc[c][2]);
        acc[c][3] = fmaf(w, x[k][c].w, acc[c][3]);
      }
    }
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[c][e] *= inv;
}

// The rows of an entry that one CTA has, from its two warpgroups' results, by 128 threads, r: their index.  A thread keeps to
// one row.  Not inlined: what it holds in registers would push out what the loop over the tiles keeps.
template <int D>
__device__ __noinline__ void join_pair(const Args& a, const Item& it, int r) {
  const int groups = 128 / it.rows, row = r % it.rows, g = r / it.rows;
  if (g >= groups) return;
  constexpr int C = 8;
#pragma unroll 1
  for (int c0 = g; c0 < D / 4; c0 += C * groups) {
    float acc[C][4];
    join_columns<D, C, 2>(a, 2, row, c0, groups, [&](int p) { return partial_slot(blockIdx.x, it.slot, p); }, acc);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c0 + c * groups < D / 4) store4(a, D, it.kvh, it.tok0, it.row0 + row, c0 + c * groups, acc[c]);
  }
}

// Remembers an item whose entry begins in this CTA's range and ends behind it (the last one, if there is one).
__device__ __forceinline__ void note_shared(const Item& it, Shared& s) {
  if (it.kind == 1 && it.n_ctas > 1 && it.slot == 1) s = Shared{it.n_ctas, it.kvh, it.tok0, it.row0, it.rows};
}

// The rows of entries that several CTAs share: blocks (c, ...) those of the entry that begins in CTA c's range and ends behind
// it, a row per thread and kJoinColumns groups of four columns per block.  (The last CTA to finish joined them itself, a
// warpgroup alone: 54 us for 64 tokens of 32 heads of 128 that see 1024 keys, most of it in this.)
constexpr int kJoinColumns = 2;
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Args a) {
  constexpr int kBlocks = D / 4 / kJoinColumns;
  pdl_wait();  // the shares
  const Shared en = a.shared[blockIdx.x];
  const bool two = D != 256 && en.rows > 128;
  const int w = blockIdx.y / kBlocks, row = threadIdx.x, first = blockIdx.x;
  if (en.n_ctas == 0 || (w == 1 && !two) || row >= min(128, en.rows - 128 * w)) return;
  const int per = D == 256 || two ? 1 : 2;  // partial results per CTA
  auto share = [&](int p) {
    const int ci = per == 2 ? p >> 1 : p;
    return partial_slot(first + ci, ci == 0 ? 1 : 0, per == 2 ? p & 1 : w);
  };
  const int jc0 = blockIdx.y % kBlocks * kJoinColumns;
  float acc[kJoinColumns][4];
  join_columns<D, kJoinColumns, 4>(a, per * en.n_ctas, row, jc0, 1, share, acc);
#pragma unroll
  for (int c = 0; c < kJoinColumns; ++c) store4(a, D, en.kvh, en.tok0, en.row0 + 128 * w + row, jc0 + c, acc[c]);
}

template <int D>
cudaError_t launch_join(const Args& a, int sm_count, cudaStream_t s) {
  const cudaError_t e = launch_pdl(join_kernel<D>, dim3((unsigned)sm_count, (D == 256 ? 1 : 2) * D / 4 / kJoinColumns),
                                   dim3(128), 0, s, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// ---------------------------------------------------------------------------
// the result of an item's rows: O / l where this warpgroup alone has the rows, else a partial result, joined with the others
// at once where they are this CTA's.  Row r of warpgroup wg; some: O holds something, in units of `unit`; m, l: its reference and sum.
// ---------------------------------------------------------------------------
template <int D, bool kTurbo>
__device__ __forceinline__ void finish_rows(const Args& a, const Item& it, int wg, int r, bool valid, bool any_valid,
                                            long long out_at, uint32_t t_o, bool some, float m, float l, float unit) {
  const bool mine = D != 256 || wg == 0;  // this warpgroup holds rows
  const int shares = D == 256 || it.two ? it.n_ctas : 2 * it.n_ctas;
  const bool whole = shares == 1;
  const long long my_slot = partial_slot(blockIdx.x, it.slot, wg);
  // (a share's O: [D / 4][rows_cap] float4, so that the rows of a warp are consecutive)
  float4* po = reinterpret_cast<float4*>(a.part_o + my_slot * a.rows_cap * D) + r;
  float norm = a.inv_lam_v;  // folds 1 / lambda and the transform's 1 / sqrt(D)
  if constexpr (kTurbo) norm *= inv_sqrt_dim<D>();
  if (mine) {
    if (whole) norm *= l == 0.f ? 0.f : __fdividef(1.f, l);
    if (!whole && valid) {
      float* ml = a.part_ml + my_slot * a.rows_cap * 2 + 2 * r;
      ml[0] = m;
      ml[1] = l;
    }
    if (some) {
      // a row without any weight (l = 0) is zeros whatever its accumulator holds
      const bool zero = l == 0.f;
      auto emit = [&](int col, const float (&y)[8]) {  // eight columns of this thread's row
        if (!valid) return;
        if (whole) store8(a.c.out, a.c.out_dtype, out_at + col, y);
        else {
          po[(col >> 2) * a.rows_cap] = make_float4(y[0], y[1], y[2], y[3]);
          po[((col >> 2) + 1) * a.rows_cap] = make_float4(y[4], y[5], y[6], y[7]);
        }
      };
      if constexpr (!kTurbo) {
#pragma unroll 1
        for (int c = 0; c < D / 32 && any_valid; ++c) {
          uint32_t o[32];
          tc::tmem_ld32_nw(t_o + 32 * c, o);
          loaded(o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = zero ? 0.f : __uint_as_float(o[8 * k + e]) * norm * unit;
            emit(32 * c + 8 * k, y);
          }
        }
      } else {
        // diag(s) H: the transform of D = 64 n coordinates is one over the n blocks, taken while they are read
        // (block p of the result: the blocks with signs (-1)^|p & k|), then one over 64 in registers
#pragma unroll 1
        for (int p = 0; p < D / 64 && any_valid; ++p) {
          float z[64];
#pragma unroll
          for (int e = 0; e < 64; ++e) z[e] = 0.f;
#pragma unroll 1
          for (int k = 0; k < D / 64; ++k) {
            const float sgn = __popc(p & k) & 1 ? -1.f : 1.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t o[32];
              tc::tmem_ld32_nw(t_o + 64 * k + 32 * c, o);
              loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) z[32 * c + e] = fmaf(sgn, __uint_as_float(o[e]), z[32 * c + e]);
            }
          }
          thread_wht<64>(z);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              y[e] = zero ? 0.f : z[8 * k + e] * norm * (float)a.c.tab.signs[64 * p + 8 * k + e];
            emit(64 * p + 8 * k, y);
          }
        }
      }
    } else if (whole && valid) {
      const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < D / 8; ++c) store8(a.c.out, a.c.out_dtype, out_at + 8 * c, z);
    }
    if (!whole && it.n_ctas == 1) {
      // the last of the two warpgroups joins them (what several CTAs share: join_kernel)
      __threadfence();
      tc::bar_sync(2 + wg, 128);
      int done = 0;
      if (r == 0) done = (int)atomicAdd(a.counters + it.counter, 1u) == 1;
      const bool join = tc::bar_sync_or(2 + wg, 128, done != 0);
      if (join) {
        __threadfence();
        join_pair<D>(a, it, r);
      }
    }
  }
}

template <int D, int VB>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
  using Sh = Shape<D>;
  constexpr int BN = Sh::BN, NB = Sh::NB, PH = Sh::PH;
  constexpr bool kTurbo = VB > 0 && VB < kF8;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = tc::smem_addr(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Bars* B = reinterpret_cast<Bars*>(sm + Sh::bars);
  Item* items = reinterpret_cast<Item*>(sm + Sh::items);
  long long* loc = reinterpret_cast<long long*>(sm + Sh::loc);
  uint32_t* miss = reinterpret_cast<uint32_t*>(sm + Sh::miss);
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + Sh::words);
  float* rs = reinterpret_cast<float*>(sm + Sh::rs);

  if (warp == 0) {
    tc::tmem_alloc(&B->tmem, 512);
    if (lane == 0) {
      for (int i = 0; i < 3; ++i) {
        tc::mbar_init(&B->k_full[i], kProdWarps / 2);
        tc::mbar_init(&B->v_full[i], kProdWarps / 2);
        tc::mbar_init(&B->k_free[i], 2);  // one by each issuer, or both by the only one that uses the tile
        tc::mbar_init(&B->v_free[i], 2);
      }
      tc::mbar_init(&B->s_done[0], 1);
      tc::mbar_init(&B->s_done[1], 1);
      for (int i = 0; i < 4; ++i) {
        tc::mbar_init(&B->p_full[i], 4);
        tc::mbar_init(&B->pv_done[i], 1);
      }
      tc::mbar_init(&B->drained[0], 1);
      tc::mbar_init(&B->drained[1], 1);
      for (int i = 0; i < NI; ++i) {
        tc::mbar_init(&B->q_full[i], 8);
        tc::mbar_init(&B->item_full[i], 1);
        tc::mbar_init(&B->item_free[i], Sh::kItemReaders);
      }
      for (int i = 0; i < NL; ++i) {
        tc::mbar_init(&B->loc_full[i], kLocWarps);
        tc::mbar_init(&B->loc_free[i], kProdWarps);
      }
    }
  }
  if constexpr (kTurbo) {
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
  const uint32_t tmem = (uint32_t)uniform((int)B->tmem);
  pdl_wait();  // the plan
  pdl_launch_dependents();  // the join's start overlaps the last CTAs
  bool ok = true;
  int icnt = 0;  // items so far
  int gt = 0;    // key tiles so far

  if (warp >= 8 + kProdWarps) {
    setmaxnreg_dec<kRegsOther>();
    if (warp >= kLocator) {
      const int half = warp - kLocator;
      Items<D> src;
      if (half == 0) src.start(a);
      for (;; ++icnt) {
        const int is = icnt % NI;
        if (half == 0) {
          if (icnt >= NI) wait_warp<100>(ok, &B->item_free[is], icnt / NI - 1);
          Item it;
          src.next(a, it);  // (the lanes alike)
          if (lane == 0) {
            items[is] = it;
            tc::mbar_arrive(&B->item_full[is]);
          }
          __syncwarp();
        } else {
          wait_warp<100>(ok, &B->item_full[is], icnt / NI);
        }
        const Item& it = items[is];
        if (!ok || it.kind == 0) break;
        const int n = it.n;
        int page[BN / 64], next[BN / 64];
        if (n > 0) read_pages<D>(a, it, 0, half, lane, page);
        for (int j = 0; j < n && ok; ++j, ++gt) {
          const int s = gt % NL;
          if (j + 1 < n) read_pages<D>(a, it, j + 1, half, lane, next);
          if (gt >= NL) wait_warp<100>(ok, &B->loc_free[s], gt / NL - 1);
          locate_tile<D, VB>(a, it, j, half, lane, page, loc + s * BN, miss + (gt % kMissRing) * 4,
                             words + (gt % kMissRing) * 16);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&B->loc_full[s]);
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) page[i] = next[i];
        }
        __syncwarp();
        if (half && lane == 0) tc::mbar_arrive(&B->item_free[is]);
      }
    } else if (warp - kIssuer < Sh::kIssuers) {
      issue_products<D>(B, items, sb, tmem, warp - kIssuer, lane, ok);
    }
    __syncwarp();
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegsProducer>();
    using P = Producer<D, VB>;
    const int ptid = tid & 127;
    // One role's tiles: convert row i, ask for row i of the next tile; raw holds the codes between.
    auto produce = [&](auto& raw, auto load, auto convert, uint64_t* full, uint64_t* free, int tiles_at) {
      for (;; ++icnt) {
        const int is = icnt % NI;
        wait_warp<40>(ok, &B->item_full[is], icnt / NI);
        const int kind = items[is].kind, n = items[is].n;
        if (!ok || kind == 0) break;
        if (n > 0) {
          wait_warp<40>(ok, &B->loc_full[gt % NL], gt / NL);
#pragma unroll
          for (int i = 0; i < P::RN; ++i) load(a, loc + (gt % NL) * BN, ptid, i, raw);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&B->loc_free[gt % NL]);
        }
        for (int j = 0; j < n && ok; ++j, ++gt) {
          const int b = gt % NB, s1 = (gt + 1) % NL;
          const bool more = j + 1 < n;
          if (more) wait_warp<40>(ok, &B->loc_full[s1], (gt + 1) / NL);
          if (gt >= NB) wait_warp<40>(ok, &free[b], gt / NB - 1);
#pragma unroll
          for (int i = 0; i < P::RN; ++i) {
            convert(raw, sm + tiles_at + b * Sh::kTileB, ptid, i);
            if (more) load(a, loc + s1 * BN, ptid, i, raw);
          }
          arrive_smem(&full[b], lane);
          if (more && lane == 0) tc::mbar_arrive(&B->loc_free[s1]);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
      }
    };
    if (warp < 8 + kProdWarps / 2) {
      typename P::RawK raw;
      produce(raw, P::load_k, P::convert_k, B->k_full, B->k_free, Sh::k);
    } else {
      uint32_t tab[4] = {0u, 0u, 0u, 0u};
      if constexpr (kTurbo) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tab[i] = reinterpret_cast<const uint32_t*>(sm + Sh::tab)[i];
      }
      typename P::RawV raw;
      produce(raw, P::load_v, [&](const typename P::RawV& r, unsigned char* tile, int t, int i) { P::convert_v(r, tab, tile, t, i); },
              B->v_full, B->v_free, Sh::v);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    const int wg = warp >> 2, r = tid & 127;
    int c0 = 0;  // this warpgroup's steps so far
    auto buffer = [&](int x) { return D == 256 ? x & 1 : wg; };
    auto phase = [&](int x) { return D == 256 ? x >> 1 : x; };
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const bool mods = a.c.softcap > 0.f || a.c.slopes != nullptr;
    Shared shared{0, 0, 0, 0, 0};
    for (;; ++icnt) {
      const int is = icnt % NI;
      wait_warp(ok, &B->item_full[is], icnt / NI);
      const Item& it = items[is];
      if (tid == 0) note_shared(it, shared);
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
      arrive_smem(&B->q_full[is], lane);
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
      int s_lo = 0;                 // and the sinks from s_lo on
      float sl = 1.f, slope = 0.f;
      if (valid) {
        hi = min(it.len, max(pos + 1, it.prefix));
        if (a.c.window) lo = max(lo, pos - a.c.window + 1);
        if (a.c.first_keys) s_lo = max(0, a.c.first_keys[tok]);
        lo = max(lo, s_lo);
        sl = fmaxf(a.scale * rs[rr], 1.2e-38f);
        if (a.c.slopes) slope = a.c.slopes[head] * kLog2e;
      }
      const int all_lo = __reduce_max_sync(kFull, lo), all_hi = __reduce_min_sync(kFull, hi);
      const int first = it.two || D == 256 ? 0 : wg, stride = it.two || D == 256 ? 1 : 2;
      const int steps = D == 256 && wg ? 0 : (it.n - first + stride - 1) / stride;
      const uint32_t t_o = tmem + Sh::tO + (D == 256 ? 0 : wg * D) + lanes;
      const bool live = valid && lo < hi;  // sees some key
      const bool any_valid = __any_sync(kFull, valid);  // a warp without rows only keeps the barriers
      float m = -INFINITY, l = 0.f;
      bool unset = true;  // (of the warp) a row that sees keys has no reference yet
      float ve = 0.f;  // f8_block: O is in units of 2^ve, see raised()
      int last = -1, last_phase = 0;  // barrier and phase of the last part's value product
      for (int i = 0; i < steps; ++i) {
        const int s = buffer(c0 + i), jt = first + stride * i, tile0 = tile_of(it, jt) * BN;
        wait_warp(ok, &B->s_done[s], phase(c0 + i));
        tc::fence_after_sync();
#pragma unroll 1
        for (int h = 0; h < PH; ++h) {
          const int key0 = tile0 + h * HN;
          const uint32_t t_s = tmem + s * BN + h * HN + lanes;
          if (any_valid) {
            const uint2 mw = *reinterpret_cast<const uint2*>(miss + ((gt + jt) % kMissRing) * 4 + 2 * h);
            // steps that need more than a scale are changed in place, in tensor memory
            uint32_t kw[4], vw[4], marks = 0;  // f8_block: the words of the part's blocks
            if constexpr (VB == kF8) {
              const uint32_t* w = words + ((gt + jt) % kMissRing) * 16 + 4 * h;
              const uint4 x = *reinterpret_cast<const uint4*>(w), y = *reinterpret_cast<const uint4*>(w + 8);
              kw[0] = x.x; kw[1] = x.y; kw[2] = x.z; kw[3] = x.w;
              vw[0] = y.x; vw[1] = y.y; vw[2] = y.z; vw[3] = y.w;
#pragma unroll
              for (int b = 0; b < 4; ++b) marks |= (kw[b] | vw[b]) & 0xFFFFu;
            }
            const bool special = mods || key0 < all_lo || key0 + HN > all_hi || (mw.x | mw.y | marks) != 0u;
            if (special) {
              uint32_t xa[16];
              const bool capped = a.c.softcap > 0.f;
              const float2 cap = cap_factors(a.c.softcap);
              const int s_hi = valid ? min(sink_end(s_lo, a.c.sinks), hi) : 0;
#pragma unroll 1
              for (int c = 0; c < HN / 16; ++c) {
                tc::tmem_ld16_nw(t_s + 16 * c, xa);
                loaded(xa);
                uint32_t poison = 0;
                if constexpr (VB == kF8) {
                  const uint32_t* w = words + ((gt + jt) % kMissRing) * 16 + 4 * h + c;
                  poison = (w[0] | w[8]) & 0xFFFFu;
                  if (mods) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) xa[e] = __float_as_uint(__uint_as_float(xa[e]) * f8_scale(w[0]));
                  }
                }
                if (capped) {
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    xa[e] = __float_as_uint(cap_score(__uint_as_float(xa[e]) * sl, cap.x, cap.y));
                } else if (mods) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) xa[e] = __float_as_uint(__uint_as_float(xa[e]) * sl);
                }
                if (slope != 0.f) {
                  const float d0 = (float)(pos - key0 - 16 * c);
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    xa[e] = __float_as_uint(fmaf(-slope, fabsf(d0 - (float)e), __uint_as_float(xa[e])));
                }
                // visible keys of these 16 as a bit mask
                const int p = min(max(lo - key0 - 16 * c, 0), 16), q = min(max(hi - key0 - 16 * c, 0), 16);
                const int sp = min(max(s_lo - key0 - 16 * c, 0), 16), sq = min(max(s_hi - key0 - 16 * c, 0), 16);
                const uint32_t vis = ((((1u << q) - 1u) & (0xFFFFFFFFu << p)) | (((1u << sq) - 1u) & (0xFFFFFFFFu << sp))) &
                                     ~((c & 2 ? mw.y : mw.x) >> (16 * (c & 1)));
                if (poison) {  // a key whose K or V is marked makes the rows that see it NaN
#pragma unroll
                  for (int e = 0; e < 16; ++e) xa[e] = (poison >> e) & 1u ? 0x7FC00000u : xa[e];
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) xa[e] = (vis >> e) & 1u ? xa[e] : 0xFF800000u;
                tmem_st16(t_s + 16 * c, xa);
              }
              tc::tmem_wait_st();
            }
            // Weights against the reference so far, and only where that is unset or turns out too low (a row's tile sums
            // to more than kTop) the row's maximum, a new reference and the weights again: S is still there.
            const float f = mods ? 1.f : sl;  // scores to log2 units (special tiles are in them already where mods is set)
            bool raise = unset;
            uint32_t pk[HN / 2];
            float sum, top_sum;
#pragma unroll 1
            for (;;) {
              uint32_t x[64];
              if (raise) {
                float mx0 = -INFINITY, mx1 = -INFINITY, top = -INFINITY, top_v = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < HN / 16; ++c) {
                  uint32_t y[16];
                  tc::tmem_ld16_nw(t_s + 16 * c, y);
                  loaded(y);
#pragma unroll
                  for (int e = 0; e < 16; e += 4) {
                    mx0 = fmaxf(fmaxf(mx0, __uint_as_float(y[e])), __uint_as_float(y[e + 1]));
                    mx1 = fmaxf(fmaxf(mx1, __uint_as_float(y[e + 2])), __uint_as_float(y[e + 3]));
                  }
                  if constexpr (VB == kF8) {  // (a block's scores at its scale; the part's so far in top)
                    const uint32_t* w = words + ((gt + jt) % kMissRing) * 16 + 4 * h + c;
                    const float s1 = fmaxf(mx0, mx1) * (mods ? 1.f : fmaxf(f * f8_scale(w[0]), 1.2e-38f));
                    top = fmaxf(top, s1);
                    top_v = fmaxf(top_v, s1 + (float)f8_exponent(w[8]));
                    mx0 = mx1 = -INFINITY;
                  }
                }
                float al;
                if constexpr (VB == kF8) {
                  al = raised(m, ve, l, top, top_v);
                } else {
                  const float mn = fmaxf(m, fmaf(fmaxf(mx0, mx1), f, -kBias));
                  al = mn == -INFINITY ? 1.f : ex2(m - mn);
                  m = mn;
                  l *= al;
                }
                unset = __any_sync(kFull, live && m == -INFINITY);
                if (last >= 0) {  // O, once the product of this warpgroup's last part is complete
                  wait_warp(ok, &B->pv_done[last], last_phase);
                  tc::fence_after_sync();
#pragma unroll 1
                  for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tc::tmem_ld16_nw(t_o + 16 * c, o);
                    loaded(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                    tmem_st16(t_o + 16 * c, o);
                  }
                }
              }
              tmem_ld64(t_s, x);
              const float mu = m == -INFINITY ? 0.f : m;
              if constexpr (VB == kF8) {
                // Weights times their V block's scale over 2^ve; the sum takes that back.  (A scale below 2^-40 of 2^ve
                // counts as that: its weights, below 2^15 2^-40, are 0 in fp16.)
                sum = top_sum = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const float sh = fmaxf((float)f8_exponent(vw[b]) - ve, -40.f);
                  const float fb = mods ? 1.f : fmaxf(f * f8_scale(kw[b]), 1.2e-38f);
                  const float2 f2 = make_float2(fb, fb), m2 = make_float2(sh - mu, sh - mu);
                  float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
                  for (int e = 8 * b; e < 8 * b + 8; ++e) {
                    float2 p = __ffma2_rn(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f2, m2);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    l2 = __fadd2_rn(l2, p);
                    pk[e] = narrow(p.x, p.y, (const __half*)nullptr);
                  }
                  sum = fmaf(l2.x + l2.y, ex2(-sh), sum);
                  top_sum += l2.x + l2.y;
                }
                top_sum = fmaxf(top_sum, sum);
              } else {
              const float2 f2 = make_float2(f, f), m2 = make_float2(-mu, -mu);
              float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                float2 p = __ffma2_rn(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f2, m2);
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                l2[e & 1] = __fadd2_rn(l2[e & 1], p);
                pk[e] = narrow(p.x, p.y, (const __half*)nullptr);
              }
              sum = top_sum = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
              }
              // (rows that are not there hold whatever shared memory had: they have no say, so that results do not vary)
              if (raise || !__any_sync(kFull, live && top_sum > kTop)) break;
              raise = true;
            }
            l += sum;
            tc::tmem_st32(tmem + s * BN + h * (HN / 2) + lanes, pk);  // over scores that have been read
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&B->p_full[s * PH + h]);
          last = s * PH + h;
          last_phase = phase(c0 + i);
        }
      }
      if (last >= 0) wait_warp(ok, &B->pv_done[last], last_phase);
      tc::fence_after_sync();
      c0 += steps;
      gt += it.n;
      finish_rows<D, kTurbo>(a, it, wg, r, valid, any_valid, out_at, t_o, last >= 0, m, l, VB == kF8 ? ex2(ve) : 1.f);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&B->item_free[is]);
    }
    if (tid == 0) a.shared[blockIdx.x] = shared;
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
    case kF8: return launch<D, kF8>(a, sm_count, s);
    default: return launch<D, 3>(a, sm_count, s);
  }
}

}  // namespace ck
}  // namespace tq
