// wattn_common.cuh -- what the kernels of the window attention with sinks
// share: the problem, its mask and the split of the sinks' gradients.
//
// Key j is visible to the query at position i (query t sits at T - Tq + t)
// when j <= i and (j > i - window or j < sinks), both below the sequence's
// length.  out_i = sum_j softmax_j(scale q_i . k_j) v_j over the visible keys,
// lse_i = log sum_j exp(scale q_i . k_j); a row at or past its sequence's
// length gets out 0 and lse -inf and has no gradient.  Query head h reads key
// head h / (H / Hkv).
#pragma once

#include "rotary_kernels.cuh"

namespace lact {

struct WattnParams {
  View4 q, k, v, out, dout;          // forward: out is written; backward: read
  View4 dq, dk, dv;
  float* lse;                        // [B, H, Tq]
  const int* lengths;                // [B] or null: T
  float* delta;                      // backward: rowsum(dout * out) [B, H, Tq]
  float* part;                       // backward: the sink tiles' partial dk, dv
  float scale;
  int B, H, Hkv, group, T, Tq, d;    // group = H / Hkv
  int window, sinks;                 // each at most T
  int far_rows;                      // query rows of one far part of a sink tile
  int heads_first, by_length;        // order of the query tiles (query_tile_at)
};

__device__ __forceinline__ int seq_len(const WattnParams& p, int b) {
  return p.lengths ? max(0, min(p.lengths[b], p.T)) : p.T;
}

// The v-th query tile of 128 rows in the order in which persistent CTAs take
// them.  by_length (the forward of a few sequences, for their lengths are walked):
// first the tiles that hold tokens, then the tiles behind the lengths, which are
// only filled; else sequence after sequence.  (dQ gains nothing by it: over 90 ragged
// batches the backward took 1% less to 7% more, by the number of sequences.)  The
// later positions of a sequence first (the first
// window's tiles see fewer keys).  heads_first: all heads of a sequence at one
// position together, so that its short tiles are its last: for few rounds (B 2, H 6,
// T 8192, d 256, window 2048: the backward 933 us, 983 head by head; the forward
// 194, 204).  Else head by head, whose CTAs share keys in L2 (H 64, T 16384, d 128,
// window 4096: the backward 8674 us, 9045 the other way; the forward gains nothing
// by it: 844 and 839 at B 2, H 6, T 32768, d 256).
struct TileAt {
  int b, h, m;
};
__device__ __forceinline__ TileAt query_tile_at(const WattnParams& p, int nb, int v) {
  TileAt t;
  const int off = p.T - p.Tq;
  for (int behind = 0; behind < 2; ++behind)
    for (t.b = 0; t.b < p.B; ++t.b) {
      const int some = p.by_length ? min(nb, (max(seq_len(p, t.b) - off, 0) + 127) >> 7) : nb;
      if (!p.by_length) {   // every sequence alike
        t.b = v / (nb * p.H);
        v %= nb * p.H;
      }
      const int tiles = behind ? nb - some : some, n = tiles * p.H;
      if (v < n) {
        t.h = p.heads_first ? v % p.H : v / tiles;
        t.m = (behind ? nb : some) - 1 - (p.heads_first ? v / p.H : v % tiles);
        return t;
      }
      v -= n;
    }
  t.b = t.h = t.m = 0;   // not reached: v is below B * H * nb
  return t;
}

// Gradients of keys [kt BN, (kt + 1) BN): the queries that see any of them
// through the window are positions [kt BN, kt BN + BN - 1 + window).  A tile
// that holds sink keys is also seen by every later query; those positions are
// cut into far parts of `far_rows`, one CTA each, and the tile's partial sums
// are joined in a fixed order afterwards.  Part 0 is the near one.
struct KeyPart {
  int lo, hi;      // query positions
};
__host__ __device__ __forceinline__ int near_end(int kt, int bn, int window, int T) {
  const int64_t e = static_cast<int64_t>(kt) * bn + bn - 1 + window;
  return e < T ? static_cast<int>(e) : T;
}
// far parts of a sink tile; the same for each sink tile: positions from the
// first tile's near end on (a later tile's parts that its near part covers
// are empty)
__host__ __device__ __forceinline__ int far_parts(int bn, int window, int T, int far_rows) {
  const int e = near_end(0, bn, window, T);
  return (T - e + far_rows - 1) / far_rows;
}
__host__ __device__ __forceinline__ KeyPart key_part(int kt, int part, int bn, int window, int T, int far_rows) {
  KeyPart r;
  const int near = near_end(kt, bn, window, T);
  if (part == 0) {
    r.lo = kt * bn;
    r.hi = near;
  } else {
    const int64_t lo = near_end(0, bn, window, T) + static_cast<int64_t>(part - 1) * far_rows;
    const int64_t hi = lo + far_rows;
    r.lo = static_cast<int>(lo > near ? lo : near);
    r.hi = static_cast<int>(hi < T ? hi : T);
  }
  return r;
}

}  // namespace lact
