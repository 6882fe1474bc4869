// Plan and host side of the chunk attention (the attention itself: tq_chunk_tc.cuh).
//
// The sequences' lengths are on the device, so a one-block kernel lists the entries (up to rows_per_entry rows of a
// sequence and the keys that any of them sees) and sums up their work.  It runs in a few microseconds for the sizes
// that a step has, and clears the counters with which the main kernel joins partial results.
#include "tq_batch.cuh"
#include "tq_chunk.h"

namespace tq {
namespace {

using ck::Args;
using ck::Entry;
using ck::PlanHead;

constexpr int kPlanThreads = 512;
constexpr int kNear = 1024;  // sequences whose entry counts are kept in shared memory

struct PlanArgs {
  ChunkArgs c;
  PlanHead* head;
  Entry* entries;
  int* seq_base;  // [n_seqs + 1]: entries of the sequences before
  unsigned int* counters;
  int max_entries, rows, keys;
};

// What an entry's tokens see: the call's row and the position of its first token, their number, length and prefix of the
// sequence; then (row, tokens) hold the first key that one of them sees and the end of the last.
struct Look {
  int row, tokens, pos, len, prefix;
};

// Exclusive prefix sum of x over the block; *total receives the sum.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long y = __shfl_up_sync(kFull, v, m);
    if (lane >= m) v += y;
  }
  __syncthreads();  // the sums of the scan before are not read any more
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long w = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long y = __shfl_up_sync(kFull, w, m);
    if (lane >= m) w += y;
  }
  *total = __shfl_sync(kFull, w, 31);
  return __shfl_sync(kFull, w, warp) - warp_sums[warp] + v - x;
}

// The sequences b0 + tid whose threads say refused break their bounds: flagged, and their rows (those that are in range)
// are zeros, written by the whole block: 0.5 ms for 8192 tokens of 8 heads of 128 in fp32, 8.5 ms from one thread.
// Rare: a plan without such a sequence meets one barrier more.
__device__ __noinline__ void zero_refused(const ChunkArgs& a, int b0, bool refused, uint32_t* refused_of) {
  const int tid = threadIdx.x;
  const uint32_t m = __ballot_sync(kFull, refused);
  if ((tid & 31) == 0) refused_of[tid >> 5] = m;
  if (tid == 0) atomicOr(a.tab.status, kFlagSeqLen);
  __syncthreads();
  const long long row = (long long)a.n_q_heads * a.k.d * (a.out_dtype == TQ_DTYPE_F32 ? 4 : 2) / 16;  // 16-byte units
  uint4* o = static_cast<uint4*>(a.out);
  for (int w = 0; w < kPlanThreads / 32; ++w)
    for (uint32_t left = refused_of[w]; left; left &= left - 1) {
      const int b = b0 + 32 * w + __ffs(left) - 1;
      const long long r0 = max(0, a.b.cu[b]), r1 = min(a.b.n_tokens, a.b.cu[b + 1]);
      for (long long i = r0 * row + tid; i < r1 * row; i += kPlanThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  __syncthreads();  // before refused_of is written again
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs p) {
  __shared__ long long warp_sums[kPlanThreads / 32];
  __shared__ int near_base[kNear];
  __shared__ uint32_t refused_of[kPlanThreads / 32];
  __shared__ Look look[kPlanThreads];
  const ChunkArgs& a = p.c;
  const int tid = threadIdx.x, G = a.G;
  pdl_launch_dependents();  // the main kernel's start overlaps this one
  long long carry = 0, total;
  for (int b0 = 0; b0 < a.b.n_seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long ne = 0;
    bool refused = false;
    if (b < a.b.n_seqs) {
      const SeqOf s = seq_of(a.b, b);
      ne = ((long long)s.n * G + p.rows - 1) / p.rows;
      refused = !s.ok;
    }
    if (__syncthreads_or(refused)) zero_refused(a, b0, refused, refused_of);
    const long long at = carry + block_scan(ne, warp_sums, &total);
    if (b < a.b.n_seqs) (a.b.n_seqs <= kNear ? near_base : p.seq_base)[b] = (int)min(at, (long long)p.max_entries);
    carry += total;
  }
  // more entries than rows can hold: sequences that overlap (cu_tokens not ascending); the last ones are left out
  if (carry > p.max_entries) {
    if (tid == 0) atomicOr(a.tab.status, kFlagSeqLen);
    carry = p.max_entries;
  }
  const int E = (int)carry;
  const int* seq_base = a.b.n_seqs <= kNear ? near_base : p.seq_base;
  __syncthreads();
  carry = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    Entry en{};
    SeqOf s{};
    int i0 = 0, i1 = -1, prefix = 0;  // tokens of the entry
    if (e < E) {
      int lo = 0, hi = a.b.n_seqs;  // the last sequence with seq_base <= e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_base[mid] <= e) lo = mid;
        else hi = mid;
      }
      s = seq_of(a.b, lo);
      en.seq = lo;
      en.row0 = (e - seq_base[lo]) * p.rows;
      const int rows = min(p.rows, s.n * G - en.row0);
      en.rows = rows;
      en.tok0 = s.first;
      en.pos0 = s.len - s.n;
      en.len = s.len;
      i0 = en.row0 / G;
      i1 = (en.row0 + rows - 1) / G;
      prefix = en.prefix = a.prefix_lens ? a.prefix_lens[lo] : 0;
    }
    int first = 0x7FFFFFFF, last = 0;
    if (a.first_keys) {
      // a warp per entry, 32 tokens at a time (a thread's warp looking at its lanes' entries one after another took 13 us
      // for 7 entries of up to 256 tokens; the call went from 49 to 44 us)
      look[tid] = Look{s.first + i0, i1 - i0 + 1, s.len - s.n + i0, s.len, prefix};
      __syncthreads();
      for (int k = tid >> 5; k < min(kPlanThreads, E - e0); k += kPlanThreads / 32) {
        const Look y = look[k];
        int f = 0x7FFFFFFF, t = 0;
#pragma unroll 4
        for (int i = tid & 31; i < y.tokens; i += 32) {
          const int pos = y.pos + i, h = min(y.len, max(pos + 1, y.prefix));
          int lo = max(0, __ldg(a.first_keys + y.row + i));
          if (a.window) lo = max(lo, pos - a.window + 1);
          if (lo < h) {
            f = min(f, lo);
            t = max(t, h);
          }
        }
        f = __reduce_min_sync(kFull, f);
        t = __reduce_max_sync(kFull, t);
        __syncwarp();
        if ((tid & 31) == 0) {
          look[k].row = f;
          look[k].tokens = t;
        }
      }
      __syncthreads();
      first = look[tid].row;
      last = look[tid].tokens;
    } else if (e < E) {
      const int pos0 = s.len - s.n;
      first = a.window ? max(0, pos0 + i0 - a.window + 1) : 0;
      last = min(s.len, max(pos0 + i1 + 1, prefix));
    }
    if (first < last) {
      en.lo = first;
      en.hi = last;
      en.n_tiles = (last + p.keys - 1) / p.keys - first / p.keys;
    }
    const long long at = carry + block_scan(e < E ? en.n_tiles + ck::kOverhead : 0, warp_sums, &total);
    if (e < E) {
      en.start = at;
      p.entries[e] = en;
    }
    carry += total;
  }
  for (long long i = tid; i < (long long)E * a.k.H * 2; i += kPlanThreads) p.counters[i] = 0u;
  if (tid == 0) *p.head = PlanHead{carry, E};
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// The parts of the workspace, in order: head, entries, seq_base, counters, partial results.
struct Layout {
  size_t entries, seq_base, counters, part_o, part_ml, bytes;
  long long max_entries;
  int rows_cap;
};

Layout layout(int sm_count, int d, long long n_seqs, long long n_tokens, long long max_tokens, int n_q_heads,
              int n_kv_heads) {
  Layout l;
  const long long G = n_q_heads / n_kv_heads, rows = ck::rows_per_entry(d);
  const long long of_tokens = (n_tokens * G) / rows + n_seqs, per_seq = (max_tokens * G + rows - 1) / rows;
  // sum of ceil(n_b G / rows): at most both bounds
  l.max_entries = per_seq == 0 ? 0 : (of_tokens < n_seqs * per_seq ? of_tokens : n_seqs * per_seq);
  l.rows_cap = (int)(max_tokens * G < 128 ? max_tokens * G : 128);
  l.entries = 256;
  l.seq_base = l.entries + up(l.max_entries * sizeof(Entry));
  l.counters = l.seq_base + up((n_seqs + 1) * sizeof(int));
  l.part_o = l.counters + up(l.max_entries * n_kv_heads * 2 * sizeof(unsigned));
  l.part_ml = l.part_o + up((size_t)sm_count * 4 * l.rows_cap * d * sizeof(float));
  l.bytes = l.part_ml + up((size_t)sm_count * 4 * l.rows_cap * 2 * sizeof(float));
  return l;
}

}  // namespace

size_t chunk_workspace(int sm_count, int d, const tq_batch& b, int n_q_heads, int n_kv_heads) {
  return layout(sm_count, d, b.n_seqs, b.n_tokens, b.max_tokens, n_q_heads, n_kv_heads).bytes;
}

cudaError_t launch_chunk(const ChunkArgs& c, float lam_v, void* workspace, int sm_count, cudaStream_t s) {
  const Layout l = layout(sm_count, c.k.d, c.b.n_seqs, c.b.n_tokens, c.b.max_tokens, c.n_q_heads, c.k.H);
  if (l.max_entries * c.k.H * 2 >= (1LL << 31)) return cudaErrorInvalidValue;  // counter indices are 32-bit
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  PlanArgs p{};
  p.c = c;
  p.head = reinterpret_cast<PlanHead*>(ws);
  p.entries = reinterpret_cast<Entry*>(ws + l.entries);
  p.seq_base = reinterpret_cast<int*>(ws + l.seq_base);
  p.counters = reinterpret_cast<unsigned int*>(ws + l.counters);
  p.max_entries = (int)l.max_entries;
  p.rows = ck::rows_per_entry(c.k.d);
  p.keys = ck::keys_per_tile(c.k.d);
  plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  Args a{};
  a.c = c;
  a.plan = p.head;
  a.entries = p.entries;
  a.counters = p.counters;
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  a.part_ml = reinterpret_cast<float*>(ws + l.part_ml);
  a.rows_cap = l.rows_cap;
  a.scale = (c.scale < 0.f ? -c.scale : c.scale) * 1.4426950408889634074f;
  a.q_sign = c.scale > 0.f ? 1.f : c.scale < 0.f ? -1.f : 0.f;
  a.inv_lam_v = 1.f / lam_v;
  const int vb = c.v.format == TQ_FMT_Q8_0 ? 0 : c.v.idx_bits;
  // Entries of few rows.  48 sequences of 1K to 16K tokens, 8 KV heads of 128, 4 rows each: q8_0 128 us there and 253 in
  // the large kernel, turbo4 149 and 382; 16 rows: 152 and 275, turbo4 204 and 400; head size 64: 85 and 195; 256: 215 and
  // 330; 4 sequences of 500 tokens: 20 and 24.  At 256 a lane's registers hold 8 rows.
  const long long most = (long long)c.b.max_tokens * c.G;  // rows of an entry
  if (most <= ck::few_rows(c.k.d)) {
    if (c.k.d == 64) return ck::launch_few64(a, (int)most, vb, sm_count, s);
    if (c.k.d == 128) return ck::launch_few128(a, (int)most, vb, sm_count, s);
    return ck::launch_few256(a, (int)most, vb, sm_count, s);
  }
  if (c.k.d == 64) return ck::launch_d64(a, vb, sm_count, s);
  if (c.k.d == 128) return ck::launch_d128(a, vb, sm_count, s);
  return ck::launch_d256(a, vb, sm_count, s);
}

}  // namespace tq
