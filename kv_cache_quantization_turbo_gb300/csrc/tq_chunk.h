// What the chunk attention's plan (tq_chunk.cu) hands to its main kernel (tq_chunk_tc.cuh).
#pragma once

#include "tq_internal.h"

namespace tq {
namespace ck {

// Work units of an entry besides its key tiles: loading its queries and storing its result takes about as long.
constexpr int kOverhead = 2;

constexpr int rows_per_entry(int d) { return d == 256 ? 128 : 256; }
constexpr int keys_per_tile(int d) { return d == 256 ? 64 : 128; }

// Up to rows_per_entry rows of a sequence, the keys [lo, hi) that any of them sees and the tiles that cover them; start:
// work units of the entries before it.
struct Entry {
  long long start;
  int seq, row0, rows, lo, hi, n_tiles;
  int tok0, pos0, len, prefix;  // of its sequence: first row and position of the new tokens, length, prefix length
};

struct PlanHead {
  long long units;  // of all entries of one KV head
  int n_entries;
};

struct Args {
  ChunkArgs c;
  const PlanHead* plan;
  const Entry* entries;
  unsigned int* counters;  // [KV head][entry][row tile]: partial results so far
  float* part_o;           // [CTA][2][2][D / 4][rows_cap][4]
  float* part_ml;          // [CTA][2][2][rows_cap][2]: reference (log2 units), sum
  int rows_cap;
  float scale, q_sign;     // |softmax_scale| log2 e and its sign (0 for a scale of 0)
  float inv_lam_v;
};

cudaError_t launch_d64(const Args& a, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_d128(const Args& a, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_d256(const Args& a, int vb, int sm_count, cudaStream_t s);

// Entries of at most few_rows(d) rows (tq_chunk_few.cuh); their 2 sm_count CTAs use two partial results each.
constexpr int few_rows(int d) { return d == 256 ? 8 : 16; }
cudaError_t launch_few64(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_few128(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_few256(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);

}  // namespace ck
}  // namespace tq
