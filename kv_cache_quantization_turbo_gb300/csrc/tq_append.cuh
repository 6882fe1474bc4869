// What the append kernels of the formats share: a token's place in the cache, the rotation on the way, tokens per CTA.
#pragma once

#include "tq_batch.cuh"

namespace tq {

constexpr int kE = 16;     // coordinates per lane
constexpr int kMaxTc = 16;  // tokens per CTA

struct Launch {
  AppendArgs a;
  int tc;
};

// A token's place: the vector of (position, head 0), -1: nothing to do there; pos: its position in the sequence.
struct Place {
  long long vec;
  int pos;
  bool padding;  // behind the last sequence
};

// Row t's place, its sequence's number (n_seqs behind the last one) and its data in s.  Called by a whole warp.
__device__ __forceinline__ Place find_row(const AppendArgs& a, const DevView& v, int t, int lane, bool report, int& seq,
                                          SeqOf& s) {
  Place p{-1, 0, true};
  seq = a.b.n_seqs;
  if (t >= a.b.n_tokens) return p;
  // the sequence with cu[b] <= t < cu[b + 1]: 32 probes at a time of a shrinking range [lo, hi)
  int lo = 0, hi = a.b.n_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, at = min(lo + step * (lane + 1), hi) - 1;  // ends of 32 parts
    const uint32_t above = __ballot_sync(kFull, __ldg(a.b.cu + at + 1) > t);
    if (!above) {
      lo = hi = a.b.n_seqs;
      break;
    }
    const int k = __ffs(above) - 1;
    const int end = min(lo + step * (k + 1), hi);
    lo += step * k;
    hi = step == 1 ? lo : end;
  }
  if (lo >= a.b.n_seqs) return p;
  seq = lo;
  if (__ldg(a.b.cu + lo) > t) return p;
  p.padding = false;
  s = seq_of(a.b, lo);
  if (!s.ok) {
    if (report && lane == 0) atomicOr(a.tab.status, kFlagSeqLen);
    return p;
  }
  p.pos = s.len - s.n + (t - s.first);
  p.vec = position_vector(a.b, v, a.layer, lo, p.pos);
  if (p.vec < 0 && report && lane == 0) atomicOr(a.tab.status, kFlagBlockTable);
  return p;
}

__device__ __forceinline__ Place find_place(const AppendArgs& a, const DevView& v, int t, int lane, bool report) {
  SeqOf s;
  int seq;
  return find_row(a, v, t, lane, report, seq, s);
}

// Angle p of a token's table, padded so that the lanes of a group read different banks.
__device__ __forceinline__ int angle_at(int p) { return p + (p >> 4) * 4; }

// The rotation of a lane's coordinates [16 sub, 16 sub + 16) of a vector, held as raw words and as x.  row(): the vector's
// coordinate 16 sub in memory, read again only where a half's border lies inside lanes; cs, sn: the token's angles.  The
// lanes of a warp call it together; on: the vector has a place.
template <class T, int D, class Row>
__device__ __forceinline__ void turn_part(float (&x)[kE], const uint4 (&raw)[kE * sizeof(T) / 16], Row row_at,
                                          const tq_rope_table& R, const float* cs, const float* sn, int sub, int lane,
                                          bool on) {
  constexpr int W = kE * sizeof(T) / 16;
  const int half = R.rotary_dim / 2;
  if (R.layout == TQ_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < kE; i += 2) {
      const int e = 16 * sub + i;
      if (e < R.rotary_dim) {
        const float c = cs[angle_at(e >> 1)], s = sn[angle_at(e >> 1)], a = x[i], b = x[i + 1];
        x[i] = a * c - b * s;
        x[i + 1] = a * s + b * c;
      }
    }
  } else if (half % kE == 0) {  // the partners of the lane's coordinates: those of one other lane
    const bool rot = 16 * sub < R.rotary_dim, first = 16 * sub < half;
    const int from = rot ? (first ? half / kE : -half / kE) : 0;
    uint4 other[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      other[k].x = __shfl_sync(kFull, raw[k].x, lane + from);
      other[k].y = __shfl_sync(kFull, raw[k].y, lane + from);
      other[k].z = __shfl_sync(kFull, raw[k].z, lane + from);
      other[k].w = __shfl_sync(kFull, raw[k].w, lane + from);
    }
    if (rot) {
      float y[kE];
      load_row<kE>(reinterpret_cast<const T*>(other), y);
      const int p0 = angle_at(first ? 16 * sub : 16 * sub - half);
#pragma unroll
      for (int i = 0; i < kE; i += 4) {
        const float4 c = *reinterpret_cast<const float4*>(cs + p0 + i);
        const float4 s = *reinterpret_cast<const float4*>(sn + p0 + i);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i + k] = fmaf(cc[k], x[i + k], (first ? -ss[k] : ss[k]) * y[i + k]);
      }
    }
  } else if (on) {  // borders of the halves inside lanes
    const T* row = row_at();
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int e = 16 * sub + i;
      if (e < R.rotary_dim) {
        const bool first = e < half;
        float y[1];
        load_row<1>(row + i + (first ? half : -half), y);
        const int pr = angle_at(first ? e : e - half);
        x[i] = fmaf(cs[pr], x[i], (first ? -sn[pr] : sn[pr]) * y[0]);
      }
    }
  }
}

// Tokens per CTA: as many, up to 16, as leave a CTA of each half for every SM (a decode batch takes one token each, the
// shortest chain; a chunk shares places and angles: 16 instead of 8 tokens are 16 us instead of 19 for 1.7K tokens of 8
// heads of 64, and the same 17 us for 4096 tokens of 8 heads of 128).
template <class F>
cudaError_t with_launch(const AppendArgs& a, int sm_count, F run) {
  Launch L{};
  L.a = a;
  int tc = 1;
  while (tc < kMaxTc && a.b.n_tokens / (tc * 2) >= sm_count) tc *= 2;
  L.tc = tc;
  run(L, (unsigned)((a.b.n_tokens + tc - 1) / tc));
  return cudaGetLastError();
}

}  // namespace tq
