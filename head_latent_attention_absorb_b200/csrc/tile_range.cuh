// Equal shares of the concatenated key tiles of a ragged batch: share c of nc takes tiles
// [c total / nc, (c + 1) total / nc) of the sequences laid end to end, so a long sequence is cut over many
// SMs and short ones share one.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace mla {

struct TileRange {
  long long lo, hi;  // this share, in the order of all tiles
  long long tb;      // first tile of sequence b in that order
  int b;             // the sequence that holds tile lo
};

// Tiles of a sequence; a length outside [T, n_max] has none.
template <int kTile>
__device__ __forceinline__ int tiles_of_length(int len, int T, int n_max) {
  return len < T || len > n_max ? 0 : (len + kTile - 1) / kTile;
}

// One warp: share c of nc.  Share 0 reports lengths outside [T, n_max].
template <int kTile>
__device__ __forceinline__ void tile_range(const int32_t* lengths, int B, int T, int n_max, int c, int nc, int32_t* err,
                                           TileRange* out) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  bool bad = false;
  for (int b = lane; b < B; b += 32) {
    const int len = lengths[b];
    bad |= len < T || len > n_max;
    total += tiles_of_length<kTile>(len, T, n_max);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (__any_sync(0xffffffffu, bad) && c == 0 && lane == 0) raise_error(err, MLA_ERR_LENGTH);
  TileRange r;
  r.lo = total * c / nc;
  r.hi = total * (c + 1) / nc;
  r.b = B;
  r.tb = 0;
  if (r.lo < r.hi) {
    long long base = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int nt = b0 + lane < B ? tiles_of_length<kTile>(lengths[b0 + lane], T, n_max) : 0;
      int sum = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + sum > r.lo);
      if (hit) {
        const int l = __ffs(hit) - 1;
        r.b = b0 + l;
        r.tb = base + __shfl_sync(0xffffffffu, sum - nt, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  if (lane == 0) *out = r;
}

// Calls f(b, length, first tile, end tile) for every piece of a sequence in the share, until f returns false.
template <int kTile, typename F>
__device__ __forceinline__ void for_each_piece(const TileRange& r, const int32_t* lengths, int B, int T, int n_max, F f) {
  long long t = r.lo, tb = r.tb;
  for (int b = r.b; b < B && t < r.hi; ++b) {
    const int len = lengths[b], nt = tiles_of_length<kTile>(len, T, n_max);
    if (tb + nt > t) {
      const int begin = (int)(t - tb), end = (int)((r.hi < tb + nt ? r.hi : tb + nt) - tb);
      if (!f(b, len, begin, end)) return;
      t = tb + end;
    }
    tb += nt;
  }
}

}  // namespace mla
