// Chunk attention over f8_block caches whose tiles many entries use, head sizes 64 and 128.
//
// A first kernel writes every key tile that some row sees once, as the tensor core takes it: fp16 values in swizzled operand
// tiles, relative to the tile's largest scale where its blocks' scales lie within 2^8 of one another, else without scales,
// which then go to scores and weights block by block; exact either way.  The main kernel's tiles are then plain bulk copies by
// one thread, without producers, which in the kernel that converts for each entry (tq_chunk_tc.cuh) share the instruction
// slots with the softmax.  Its registers go to the softmax instead: a row's 128 scores are read from tensor memory at once,
// masks and score modifications happen in registers, and weights are written only when their sum is known not to pass what
// fp16 holds, so that the scores are still there where it does.  Entries, ranges, products, the running references and the
// join of shared entries are those of tq_chunk_tc.cuh.
//
// What bounds it.  Eight tensor instructions of M 128, N 128, K 16 take 584 cycles by themselves, for scores as for values,
// so a tile of two row tiles (32 of them) 2.34 K cycles; it takes 3.1 to 3.3 K.  Scores and weights of a row tile share one
// buffer, so its step is a chain: value products of the last tile's second half, score product, the scores' way to
// registers, weights (720 cycles for 128 keys by themselves, most of them the exponentials), stores.  The chains of the two
// row tiles do not fill each other's gaps wholly, and the operands and copies of a tile, 256 KB, keep shared memory busy for
// 2 K cycles meanwhile.  4096 tokens at 32K, 32 query heads of 128 on 8 KV heads, bf16: 1.55 ms with staging (42 us) and
// join (15 us), 1.33 PFLOP/s; 2.13 ms in the other kernel.  Steps on the way: without producers 1.74 ms; the two softmax
// warps of a sub-partition taking turns 1.65 (left alone they fall into step); the check for a new reference by the scores'
// maximum before the turn 1.58, by the weights' sum, with the weights in registers until it is known, 1.57; the join 1.53,
// its loads 1.51; with references of each row's own for its weights' exponents, instead of the warp's, 1.55.  Where every
// other block of V has a scale 2^12 larger, so that every tile's scales are applied by block: 3.19 ms, 2.14 in the other
// kernel.  A version that kept the scores in registers for that check spilled: 1.71.  Pairs of CTAs that share the operands
// (two thirds of the shared-memory traffic) are the way on.
#pragma once

#include <type_traits>

#include "tq_chunk_tc.cuh"

namespace tq {
namespace ck {
namespace staged {

// ---------------------------------------------------------------------------
// staging: a CTA per tile and KV head
// ---------------------------------------------------------------------------
constexpr int kStageThreads = 256;
// Tiles whose blocks' scales differ by at most 2^kSpan have operands relative to the largest one, for keys and values; the
// others' are the codes alone.  Weights of the former count by the tile's scale: a row's weights below 2^-29 of its largest
// are 0 in fp16, which are then up to 2^(8 - 29) of it where a block's own scale is 2^-8 of its tile's.
constexpr int kSpan = 8;

// Orders this thread's accesses to global memory with those of asynchronous copies.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const __grid_constant__ Args a) {
  constexpr int BN = Shape<D>::BN, LPR = D / 16, RPP = kStageThreads / LPR, NP = BN / RPP;  // lanes per row, rows per pass
  __shared__ long long loc[BN];
  __shared__ uint32_t words[2][BN / 16], missing[4], marked[4];
  const ChunkArgs& c = a.c;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();  // the plan, and with it what was written before this call
  const SeqOf s = seq_of(c.b, b);
  // the keys that some row sees: the sinks [0, s_hi) and [lo, len)
  const int lo = c.window ? max(0, s.len - s.n - c.window + 1) : 0, s_hi = min(c.sinks, lo);
  const bool wanted_tile = s.n > 0 && t * BN < s.len && ((t + 1) * BN > lo || t * BN < s_hi);
  if (wanted_tile) {
    const DevView &K = c.k, &V = c.v;
    if (tid < 4) missing[tid] = marked[tid] = 0u;
    if (tid < BN) {
      const int j = t * BN + tid;
      const bool want = j < s.len && (j >= lo || j < s_hi);
      const int lp = (int)((uint32_t)j / (uint32_t)K.page_size);
      int page = c.b.block_table ? -1 : b;
      if (c.b.block_table && want && lp < c.b.max_blocks) page = __ldg(c.b.block_table + (long long)b * c.b.max_blocks + lp);
      const bool on = want && page >= 0 && page < K.num_pages;
      const long long vec =
          on ? (((long long)c.layer * K.num_pages + page) * K.H + h) * K.page_size + (j - lp * K.page_size) : -1;
      loc[tid] = vec;
      const uint32_t m = __ballot_sync(kFull, want && !on), there = __ballot_sync(kFull, on) >> (lane & 16) & 0xFFFFu;
      const long long some = __shfl_sync(kFull, vec, (lane & 16) + (there ? __ffs(there) - 1 : 0));
      if ((lane & 14) == 0) {  // lanes 0 and 16: K's words of two blocks, 1 and 17: V's (0: no key of it is wanted)
        const unsigned char* hdr = lane & 1 ? V.header : K.header;
        words[lane & 1][tid / 16] = there ? __ldg(reinterpret_cast<const uint32_t*>(hdr) + some / kF8Block) : 0u;
      }
      __syncwarp();
      if (lane == 0) {
        missing[tid / 32] = m;
        const uint32_t* kw = words[0] + tid / 16;
        const uint32_t* vw = words[1] + tid / 16;
        marked[tid / 32] = ((kw[0] | vw[0]) & 0xFFFFu) | (kw[1] | vw[1]) << 16;
        if (m && h == 0) atomicOr(c.tab.status, kFlagBlockTable);
      }
    }
    __syncthreads();
    int top[2], least[2];  // exponents of K's scales, of V's
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      top[x] = kF8MinExp;
      least[x] = kF8MaxExp;
#pragma unroll
      for (int i = 0; i < BN / 16; ++i) {
        const uint32_t w = words[x][i];
        top[x] = max(top[x], w ? f8_exponent(w) : kF8MinExp);
        least[x] = min(least[x], w ? f8_exponent(w) : kF8MaxExp);
      }
    }
    const bool wide = top[0] - least[0] > kSpan || top[1] - least[1] > kSpan;
    const long long at = ((long long)b * a.staged.tiles + t) * K.H + h;
    const int row0 = tid / LPR, ch = tid % LPR;
    // a code's last bit, 2^-9, is above fp16's 2^-24 kSpan further down
    static_assert(kSpan <= 15, "exact operands");
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const unsigned char* pay = (x ? V.payload : K.payload) + 16 * ch;
      unsigned char* tile = (x ? a.staged.v : a.staged.k) + at * Shape<D>::kTileB;
      uint4 w[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const long long vec = loc[p * RPP + row0];
        w[p] = load16(pay + (vec < 0 ? 0 : vec) * D, vec >= 0);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + row0, e = wide ? 0 : max(f8_exponent(words[x][row / 16]) - top[x], -kSpan);
        const uint32_t f2 = (uint32_t)(e + 15) << 10 | (uint32_t)(e + 15) << 26;  // 2^e
        uint32_t y[8];
        f8_pairs(w[p].x, y[0], y[1]);
        f8_pairs(w[p].y, y[2], y[3]);
        f8_pairs(w[p].z, y[4], y[5]);
        f8_pairs(w[p].w, y[6], y[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = mul_h2(y[i], f2);
        *reinterpret_cast<uint4*>(tile + tile_at<BN>(row, 2 * ch)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(tile + tile_at<BN>(row, 2 * ch + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    if (tid == 0) {
      StagedHead q{};
      q.k_scale = ex2((float)top[0]);
      q.v_exp = top[1];
      q.wide = wide;
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) {
        q.missing[i] = missing[i];
        q.marked[i] = marked[i];
        q.any |= missing[i] | marked[i];
      }
#pragma unroll
      for (int i = 0; i < BN / 16; ++i) {
        q.k_exps[i] = (signed char)f8_exponent(words[0][i]);
        q.v_exps[i] = (signed char)f8_exponent(words[1][i]);
      }
      a.staged.heads[at] = q;
    }
    fence_async_global();  // the tiles, for the copies
  }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kThreads = 384;  // warps 0-3, 4-7 softmax; 8, 9 issuers; 10 loads tiles; 11 idle
constexpr int kIssuer = 8, kLoader = 10;
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kRegsNeeded = 256 * kRegsSoftmax + 128 * kRegsOther;
static_assert(kRegsNeeded <= kThreads * kRegsLaunch, "register split");

// 64 columns of this warp's tensor-memory lanes, asked for; arrived() waits for them.
__device__ __forceinline__ void tmem_ask64(uint32_t taddr, uint32_t (&x)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
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
__device__ __forceinline__ void arrived(uint32_t (&x)[64]) {
  loaded(reinterpret_cast<uint32_t(&)[32]>(x[0]));
  loaded(reinterpret_cast<uint32_t(&)[32]>(x[32]));
}

// A row's view of the keys.
struct RowOf {
  int lo, hi, s_lo, s_hi, pos;
  float sl, slope;
};

// Scores of 64 keys from key0 on that need more than a scale: modified, to log2 units where mods is set, and masked.  gone and
// marked: bits of the 64 keys.
__device__ __forceinline__ void modify(uint32_t (&x)[64], const ChunkArgs& c, const RowOf& row, int key0, float k_scale,
                                       bool mods, uint2 gone, uint2 marked) {
  if (mods) {
    const float2 cap = cap_factors(c.softcap);
    const float f = fmaxf(row.sl * k_scale, 1.2e-38f), d0 = (float)(row.pos - key0);
    const bool capped = c.softcap > 0.f, sloped = row.slope != 0.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) {
      float s = __uint_as_float(x[e]) * f;
      if (capped) s = cap_score(s, cap.x, cap.y);
      if (sloped) s = fmaf(-row.slope, fabsf(d0 - (float)e), s);
      x[e] = __float_as_uint(s);
    }
  }
  auto ones = [](int from, int to) {  // bits [from, to) of 32
    const int p = min(max(from, 0), 32), q = min(max(to, 0), 32);
    return p < q ? (0xFFFFFFFFu >> (32 - (q - p))) << p : 0u;
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = key0 + 32 * k;
    const uint32_t vis = (ones(row.lo - j, row.hi - j) | ones(row.s_lo - j, row.s_hi - j)) & ~(k ? gone.y : gone.x);
    const uint32_t bad = k ? marked.y : marked.x;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if ((bad >> e) & 1u) x[32 * k + e] = 0x7FC00000u;
      if (!((vis >> e) & 1u)) x[32 * k + e] = 0xFF800000u;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) staged_kernel(const __grid_constant__ Args a) {
  using Sh = Shape<D>;
  static_assert(D <= 128, "at 256 the other kernel is faster for every batch");
  constexpr int BN = Sh::BN, NB = Sh::NB, PH = 2;  // parts of a step
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = tc::smem_addr(sm);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Bars* B = reinterpret_cast<Bars*>(sm + Sh::bars);
  Item* items = reinterpret_cast<Item*>(sm + Sh::items);
  float* rs = reinterpret_cast<float*>(sm + Sh::rs);

  if (warp == 0) {
    tc::tmem_alloc(&B->tmem, 512);
    if (lane == 0) {
      for (int i = 0; i < 3; ++i) {
        tc::mbar_init(&B->k_full[i], 1);
        tc::mbar_init(&B->v_full[i], 1);
        tc::mbar_init(&B->k_free[i], 2);  // one by each issuer, or both by the only one that uses the tile
        tc::mbar_init(&B->v_free[i], 2);
      }
      tc::mbar_init(&B->s_done[0], 1);
      tc::mbar_init(&B->s_done[1], 1);
      for (int i = 0; i < 4; ++i) {
        tc::mbar_init(&B->p_full[i], 4);
        tc::mbar_init(&B->pv_done[i], 1);
      }
      for (int i = 0; i < 4; ++i) {
        tc::mbar_init(&B->turn[0][i], 1);
        tc::mbar_init(&B->turn[1][i], 1);
      }
      tc::mbar_init(&B->drained[0], 1);
      tc::mbar_init(&B->drained[1], 1);
      for (int i = 0; i < NI; ++i) {
        tc::mbar_init(&B->q_full[i], 8);
        tc::mbar_init(&B->item_full[i], 1);
        tc::mbar_init(&B->item_free[i], 8 + Sh::kIssuers);
      }
    }
    tc::fence_async_smem();  // the barriers, for the copies
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = (uint32_t)uniform((int)B->tmem);
  pdl_wait();  // the staged tiles and the plan
  pdl_launch_dependents();  // the join's start overlaps the last CTAs
  bool ok = true;
  int icnt = 0;  // items so far
  int gt = 0;    // key tiles so far

  if (warp >= kIssuer) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kLoader) {
      fence_async_global();
      Items<D> src;
      src.start(a);
      for (;; ++icnt) {
        const int is = icnt % NI;
        if (icnt >= NI) wait_warp<100>(ok, &B->item_free[is], icnt / NI - 1);
        Item it;
        src.next(a, it);  // (the lanes alike)
        if (lane == 0) {
          items[is] = it;
          tc::mbar_arrive(&B->item_full[is]);
        }
        __syncwarp();
        if (!ok || it.kind == 0) break;
        for (int j = 0; j < it.n && ok; ++j, ++gt) {
          const int b = gt % NB;
          const long long at = ((long long)it.seq * a.staged.tiles + tile_of(it, j)) * a.c.k.H + it.kvh;
          if (gt >= NB) wait_warp<20>(ok, &B->k_free[b], gt / NB - 1);
          if (ok && lane == 0) {
            tc::mbar_arrive_expect_tx(&B->k_full[b], Sh::kTileB);
            tc::bulk_load(sb + Sh::k + b * Sh::kTileB, a.staged.k + at * Sh::kTileB, Sh::kTileB, &B->k_full[b]);
          }
          if (gt >= NB) wait_warp<20>(ok, &B->v_free[b], gt / NB - 1);
          if (ok && lane == 0) {
            tc::mbar_arrive_expect_tx(&B->v_full[b], Sh::kTileB);
            tc::bulk_load(sb + Sh::v + b * Sh::kTileB, a.staged.v + at * Sh::kTileB, Sh::kTileB, &B->v_full[b]);
          }
          __syncwarp();
        }
      }
      // copies still in flight end before the block does
      for (int i = 0; i < NB; ++i) {
        const int n = (gt - i + NB - 1) / NB;  // tiles that went through buffer i
        if (n > 0) {
          tc::mbar_wait(&B->k_full[i], (n - 1) & 1, 1 << 16);
          tc::mbar_wait(&B->v_full[i], (n - 1) & 1, 1 << 16);
        }
      }
      __syncwarp();
    } else if (warp - kIssuer < Sh::kIssuers) {
      issue_products<D>(B, items, sb, tmem, warp - kIssuer, lane, ok);
    }
    __syncwarp();
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    const int wg = warp >> 2, r = tid & 127;
    int c0 = 0, c1 = 0;  // this warpgroup's steps so far, the other's
    const int s = wg;  // its score buffer
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
      const int tok = it.tok0 + ti;
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
      RowOf me{0, 0x7FFFFFFF, 0, 0, it.pos0 + ti, 1.f, 0.f};  // rows that are not there see everything: they never need a mask
      if (valid) {
        me.hi = min(it.len, max(me.pos + 1, it.prefix));
        if (a.c.window) me.lo = max(0, me.pos - a.c.window + 1);
        me.s_hi = min(a.c.sinks, me.hi);
        me.sl = fmaxf(a.scale * rs[rr], 1.2e-38f);
        if (a.c.slopes) me.slope = a.c.slopes[head] * kLog2e;
      }
      const int all_lo = __reduce_max_sync(kFull, me.lo), all_hi = __reduce_min_sync(kFull, me.hi);
      const int first = it.two ? 0 : wg, stride = it.two ? 1 : 2, steps = (it.n - first + stride - 1) / stride;
      const uint32_t t_o = tmem + Sh::tO + wg * D + lanes;
      const bool live = valid && me.lo < me.hi;  // sees some key
      const bool any_valid = __any_sync(kFull, valid);  // a warp without rows only keeps the barriers
      float m = -INFINITY, l = 0.f;
      bool unset = true;  // (of the warp) a row that sees keys has no reference yet
      float ve = 0.f;  // O is in units of 2^ve, see raised()
      int last = -1, last_phase = 0;  // barrier and phase of the last part's value product
      const int H = a.c.k.H, s_n = it.s_n, main_tile = it.tile, sink_tile = it.s_tile;
      const StagedHead* heads = a.staged.heads + (long long)it.seq * a.staged.tiles * H + it.kvh;
      auto tile_at_step = [&](int i) {
        const int j = first + stride * i;
        return (j < s_n ? sink_tile : main_tile) + j;
      };
      auto head_of = [&](int tile) {  // as far as every step needs it
        return __ldg(reinterpret_cast<const uint4*>(heads + (long long)tile * H));
      };
      int next_tile = tile_at_step(0);
      uint4 next = steps > 0 ? head_of(next_tile) : make_uint4(0u, 0u, 0u, 0u);
      for (int i = 0; i < steps; ++i) {
        const int tile = next_tile;
        const uint4 hd = next;
        next_tile = tile_at_step(i + 1);
        if (i + 1 < steps) next = head_of(next_tile);
        const bool wide = hd.w != 0;  // operands are codes, the blocks' scales in the head
        const float k_scale = wide ? 1.f : __uint_as_float(hd.x), v_exp = (float)(int)hd.y;
        const int key0 = tile * BN;
        const float f = mods ? 1.f : fmaxf(me.sl * k_scale, 1.2e-38f);  // scores to log2 units
        const uint32_t t_s = tmem + s * BN + lanes;
        wait_warp(ok, &B->s_done[s], c0 + i);
        tc::fence_after_sync();
        const bool special = mods || key0 < all_lo || key0 + BN > all_hi || hd.z;
        auto change = [&](uint32_t (&x)[64], int h) {
          uint2 gone = make_uint2(0u, 0u), marked = gone;
          if (hd.z) {
            const StagedHead* q = heads + (long long)tile * H;
            gone = make_uint2(q->missing[2 * h], q->missing[2 * h + 1]);
            marked = make_uint2(q->marked[2 * h], q->marked[2 * h + 1]);
          }
          modify(x, a.c, me, key0 + h * HN, k_scale, mods, gone, marked);
        };
        // Weights times 2^(v_exp - ve), in fp16; the sum takes that factor back.  (A scale below 2^-40 of 2^ve counts as that:
        // its weights, at most 2^15 2^-40, are 0 in fp16.)
        const float2 f2 = make_float2(f, f);
        const float sh = fmaxf(v_exp - ve, -40.f), mu = sh - (m == -INFINITY ? 0.f : m);
        const float2 m2 = make_float2(mu, mu);
        // of 32 keys from half * 32 on
        auto weights = [&](const uint32_t (&y)[64], auto half, uint32_t (&pk)[32], float2 (&l2)[2]) {
          constexpr int k0 = half.value * 32;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = k0 + 2 * e;
            float2 p = __ffma2_rn(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), f2, m2);
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            l2[e & 1] = __fadd2_rn(l2[e & 1], p);
            pk[k / 2] = narrow(p.x, p.y, (const __half*)nullptr);
          }
        };
        constexpr std::integral_constant<int, 0> lower{};
        constexpr std::integral_constant<int, 1> upper{};
        auto sum_of = [&](const float2 (&l2)[2]) { return (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y); };
        // (rows that are not there hold whatever shared memory had: they have no say, so that results do not vary)
        const float back = ex2(-sh), most = kTop * fminf(1.f, ex2(sh));
        auto too_large = [&](float sum) { return __any_sync(kFull, live && sum > most); };
        auto store = [&](int h, const uint32_t (&pk)[32]) {  // over scores that have been read
          tc::tmem_st32(t_s + h * (HN / 2), pk);
        };
        auto publish = [&](int h) {
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&B->p_full[s * PH + h]);
          last = s * PH + h;
          last_phase = c0 + i;
        };
        // The two softmax warps of an SM sub-partition take turns, step by step: then one's products run while the other has
        // the sub-partition to itself.  Left alone they fall into step, and the tensor core and the softmax take turns.
        auto pass_on = [&]() {
          if (lane == 0) tc::mbar_arrive(&B->turn[1 - wg][warp & 3]);
        };
        int todo = 0;  // parts before this one are published
        if (any_valid && !unset && !wide) {
          uint32_t x0[64], pk[32];
          float2 u[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          tmem_ask64(t_s, x0);
          uint32_t x1[64], qk[32];
          float2 w[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          tmem_ask64(t_s + HN, x1);
          arrived(x0);
          arrived(x1);
          if (special) {
            change(x0, 0);
            change(x1, 1);
          }
          wait_warp(ok, &B->turn[wg][warp & 3], wg ? c1 + i : c1 + i - 1);
          weights(x0, lower, pk, u);
          weights(x0, upper, pk, u);
          float sum = sum_of(u);
          weights(x1, lower, qk, w);  // (while the first part's sum is looked at)
          if (!too_large(sum)) {
            l = fmaf(sum, back, l);
            store(0, pk);
            weights(x1, upper, qk, w);  // (while the first part's weights are stored)
            publish(0);
            todo = 1;
            sum = sum_of(w);
            if (!too_large(sum)) {
              l = fmaf(sum, back, l);
              store(1, qk);
              pass_on();
              publish(1);
              todo = 2;
            }
          }
        } else {
          wait_warp(ok, &B->turn[wg][warp & 3], wg ? c1 + i : c1 + i - 1);
        }
        // The references are raised, and O and the sum with them, where they are unset, and where weights against those so far
        // turned out too large: their scores are still there.  Wide tiles come here, too: a block of 16 keys at a time.
        if (todo < PH) {
          const StagedHead* q = heads + (long long)tile * H;
#pragma unroll 1
          for (int h = todo; h < PH; ++h) {
            if (any_valid) {
              uint32_t x[64], pk[32];
              tmem_ld64(t_s + h * HN, x);
              float es[4] = {v_exp, v_exp, v_exp, v_exp};
              if (wide) {
                const uint32_t ke = *reinterpret_cast<const uint32_t*>(q->k_exps + 4 * h);
                const uint32_t ev = *reinterpret_cast<const uint32_t*>(q->v_exps + 4 * h);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const float k_b = ex2((float)(signed char)(ke >> 8 * b & 255u));
                  es[b] = (float)(signed char)(ev >> 8 * b & 255u);
#pragma unroll
                  for (int e = 16 * b; e < 16 * b + 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * k_b);
                }
              }
              if (special) change(x, h);
              float top = -INFINITY, top_v = -INFINITY;
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 16 * b; e < 16 * b + 16; ++e) mx[e & 1] = fmaxf(mx[e & 1], __uint_as_float(x[e]));
                const float s1 = fmaxf(mx[0], mx[1]) * f;
                top = fmaxf(top, s1);
                top_v = fmaxf(top_v, s1 + es[b]);
              }
              const float al = raised(m, ve, l, top, top_v);
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
              const float m1 = m == -INFINITY ? 0.f : m;
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const float shb = fmaxf(es[b] - ve, -40.f);
                const float2 mb = make_float2(shb - m1, shb - m1);
                float2 u = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 8 * b; e < 8 * b + 8; ++e) {
                  float2 p = __ffma2_rn(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f2, mb);
                  p.x = ex2(p.x);
                  p.y = ex2(p.y);
                  u = __fadd2_rn(u, p);
                  pk[e] = narrow(p.x, p.y, (const __half*)nullptr);
                }
                l = fmaf(u.x + u.y, ex2(-shb), l);
              }
              store(h, pk);
            }
            publish(h);
          }
          pass_on();
        }
      }
      if (last >= 0) wait_warp(ok, &B->pv_done[last], last_phase);
      tc::fence_after_sync();
      c0 += steps;
      c1 += (it.n - (it.two ? 0 : 1 - wg) + stride - 1) / stride;
      gt += it.n;
      finish_rows<D, false>(a, it, wg, r, valid, any_valid, out_at, t_o, last >= 0, m, l, ex2(ve));
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

template <int D>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t s) {
  cudaError_t e = launch_pdl(stage_kernel<D>, dim3((unsigned)a.staged.tiles, (unsigned)a.c.k.H, (unsigned)a.c.b.n_seqs),
                             dim3(kStageThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  auto kern = staged_kernel<D>;
  cudaFuncAttributes at;
  e = cudaFuncGetAttributes(&at, kern);
  if (e != cudaSuccess) return e;
  if (at.numRegs * kThreads < kRegsNeeded) return cudaErrorLaunchOutOfResources;  // the split would wait for ever
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::alloc);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)sm_count), dim3(kThreads), Shape<D>::alloc, s, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace staged
}  // namespace ck
}  // namespace tq
