// What the chunk attention's plan (tq_chunk.cu) hands to its main kernel (tq_chunk_tc.cuh).
#pragma once

#include "tq_internal.h"

namespace tq {
namespace ck {

// Work units of an entry besides its key tiles: loading its queries and storing its result takes about as long.
constexpr int kOverhead = 2;
// A CTA that takes part has at least as many, where entries are cut.
constexpr int kMinUnits = 2;

constexpr int rows_per_entry(int d) { return d == 256 ? 128 : 256; }
constexpr int keys_per_tile(int d) { return d == 256 ? 64 : 128; }

// Kinds of V in the kernels: q8_0, turbo-MSE index bits 1 to 3 (both over q8_0 K), or f8_block for K and V.
constexpr int kF8 = 4;

// Up to rows_per_entry rows of a sequence, the keys that any of them sees and the tiles that cover them: the keys
// [s_lo, s_hi) ahead of the window (sinks) in the first s_tiles ones, then [lo, hi); start: work units of the entries
// before it.
struct Entry {
  long long start;
  int seq, row0, rows, lo, hi, n_tiles, s_lo, s_hi, s_tiles;
  int tok0, pos0, len, prefix;  // of its sequence: first row and position of the new tokens, length, prefix length
};

struct PlanHead {
  long long units;  // of all entries of one KV head
  int n_entries;
  int whole;        // entries are not cut: a CTA takes those that begin in its range
};

// f8_block tiles as operands, staged in the workspace (tq_chunk_staged.cuh): tile t of KV head h of sequence b is number
// (b * tiles + t) * H + h of k, v (tile_bytes each, as the tensor core takes them) and heads.
struct StagedHead {
  float k_scale;      // of the tile's K operand; its V operand's is 2^v_exp
  int v_exp;
  uint32_t any;       // some bit of missing or marked is set
  uint32_t wide;      // its blocks' scales lie too far apart for one: the operands are codes, without scales
  uint32_t missing[4], marked[4];  // by key: its page is out of range; its K or V is marked
  signed char k_exps[8], v_exps[8];  // by block of 16 keys: the exponents of its scales
};
struct Staged {
  unsigned char* k;
  unsigned char* v;
  StagedHead* heads;
  int tiles;          // of a sequence
};
constexpr int tile_bytes(int d) { return keys_per_tile(d) * d * 2; }

// The entry that begins in a CTA's range and ends behind it: the CTAs that share it (0: there is none), its rows.
struct Shared {
  int n_ctas, kvh, tok0, row0, rows;
};

struct Args {
  ChunkArgs c;
  const PlanHead* plan;
  const Entry* entries;
  unsigned int* counters;  // [KV head][entry][2]: partial results so far
  float* part_o;           // [CTA][2][2][D / 4][rows_cap][4]
  float* part_ml;          // [CTA][2][2][rows_cap][2]: reference (log2 units), sum
  Shared* shared;          // [CTA]
  int rows_cap;
  float scale, q_sign;     // |softmax_scale| log2 e and its sign (0 for a scale of 0)
  float inv_lam_v;
  Staged staged;           // launch_staged*
};

cudaError_t launch_d64(const Args& a, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_d128(const Args& a, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_d256(const Args& a, int vb, int sm_count, cudaStream_t s);
// After these or the staged ones: the rows that several CTAs share.
cudaError_t launch_join64(const Args& a, int sm_count, cudaStream_t s);
cudaError_t launch_join128(const Args& a, int sm_count, cudaStream_t s);
cudaError_t launch_join256(const Args& a, int sm_count, cudaStream_t s);

// f8_block views whose tiles are staged first.
cudaError_t launch_staged64(const Args& a, int sm_count, cudaStream_t s);
cudaError_t launch_staged128(const Args& a, int sm_count, cudaStream_t s);

// Entries of at most few_rows(d) rows (tq_chunk_few.cuh); their 2 sm_count CTAs use two partial results each.
constexpr int few_rows(int d) { return d == 256 ? 8 : 16; }
cudaError_t launch_few64(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_few128(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);
cudaError_t launch_few256(const Args& a, int rows, int vb, int sm_count, cudaStream_t s);

}  // namespace ck
}  // namespace tq
