// Eviction from a cache by accumulated attention weight.
//
// Per sequence with L > keep rows: kept are the first `sink` rows, the `recent` newest rows, and the
// keep - sink - recent rows of largest accumulated weight among the rest (ties: the lower row; NaN
// counts as the least).  Attention does not depend on the order of the rows (the rotary key carries
// each row's position), so nothing is shifted: the kept rows behind `keep` move into the holes before
// it, j-th hole from j-th row.  That moves the fewest bytes, and since sources lie at or behind `keep` and
// destinations before it, no row is read after it was written: the move needs no order and no copy.
//
// Which rows are the newest: without positions the last ones, which holds while rows stand in order of age.  The move
// itself ends that order (the newest rows go into holes anywhere), so a cache that is cut again brings its rows'
// positions, which move along.  The newest are then found by a radix selection of their own, over (position, row),
// whose keys are all distinct, and enter the selection by weight with a key above every weight's.  The sinks need no
// positions: the first `sink` rows are always kept and never move.
//
// Two launches: the selection writes row_map (a cluster of eight CTAs per sequence, each with a slice of the
// rows, or one CTA for a short sequence; counts, ranks and the list of moved rows cross through distributed
// shared memory), the move reads it.
//
// Bound: the selection by latency, a chain of passes over keys in shared memory, scans and meetings (17 us for 4
// sequences of up to 32768 rows, 12 for 32 of 4096, alone with cold caches); the move by its bytes, with
// few warps when few rows move.  Both together, back to back: 4 sequences of 20000 to 32768 rows of 1152 bytes cut to
// 16384 25 us (63 MB: 2.5 TB/s), 32 sequences of 4-bit rows that lose up to 256 of 4096 12.6 us.  With positions 38 and
// 21 us: one pass for the bits in which positions differ and mostly two for the newest rows.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;  // of a CTA of the selection
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;     // CTAs that share a sequence
// Rows that one CTA selects from by itself: always; as far as its shared memory goes; for each sequence of the batch.
constexpr int kOneCta = 8192, kOneCtaFull = 32768, kOneCtaPer = 1024;
constexpr int kSelectSmem = 220 * 1024;
constexpr int kMaxRows = 400000;  // a slice of them is counted in 16 bits
constexpr int kWord = 32;       // rows of one word of the kept mask
constexpr int kBatch = 4;       // keys, or words of the mask, that are read together
// Digits of the radix selection, from the top.  One CTA takes 11, 11 and 10 bits: the first digit holds the sign,
// the exponent and two bits of the fraction, which spreads weights of one size over enough counters that a warp's
// additions seldom meet, and two digits mostly decide.  A cluster, which reads eight arrays of counts, takes 8 bits.
template <int C>
constexpr int kDigitBits = C == 1 ? 11 : 8;
template <int C>
constexpr int kBins = 1 << kDigitBits<C>;
template <int C>
constexpr int kPasses = (32 + kDigitBits<C> - 1) / kDigitBits<C>;

// Order-preserving map of a float to 32 bits: NaN is the least, -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Rows in order of age as one number; of equal positions the higher row is the newer one.
constexpr int kRowBits = 19;  // of a row's number
static_assert(kMaxRows < 1 << kRowBits, "a row's number is the low part of the key");
__device__ __forceinline__ uint64_t age_key(int32_t position, int row) {
  return (uint64_t)((uint32_t)position ^ 0x80000000u) << 32 | (uint32_t)row;
}

// Position of the n-th (from 0) set bit of m.
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return __ffs(m) - 1;
}

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(sm100::mapa(sm100::smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(int* p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(sm100::mapa(sm100::smem_u32(p), rank)), "r"(v) : "memory");
}

// Integers of the list of a slice of `per` words; the counts of the digits lie there before.  The moved rows are at
// most half of all rows: they lie behind `keep` and fill holes before it.
template <int C>
__host__ __device__ constexpr int list_ints(int per) {
  return per * kWord / 2 > kPasses<C> * kBins<C> ? per * kWord / 2 : kPasses<C> * kBins<C>;
}

struct Found {
  int digit, rank;  // the digit that holds the threshold, and how many of its rows are to be taken
  int rows, lower;  // the rows that have it, and those of them in the slices before this one
};
struct SelectSmem {
  uint32_t sums[kPasses<kCluster> + 2][kWarps];
  Found found[2];
  int mine[2];  // this CTA's holes and moved rows
  int differ;   // bits in which the positions of this CTA's rows differ
};

// Inclusive prefix sum over the block's threads; the array is written by this call alone.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t (&warp_sums)[kWarps]) {
  static_assert(kWarps == 32, "a lane has a warp's sum");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  return x + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0u);
}

// Sum of the lower-ranked CTAs' value, once the cluster has met.
template <int C>
__device__ __forceinline__ int before_me(const int* p, uint32_t rank) {
  int sum = 0;
#pragma unroll
  for (uint32_t r = 0; r < C; ++r) {
    const int v = C == 1 ? 0 : ld_cluster(p, r);
    sum += r < rank ? v : 0;
  }
  return sum;
}

// All threads of the C CTAs of a sequence.
template <int C>
__device__ __forceinline__ void meet() {
  if constexpr (C == 1)
    __syncthreads();
  else
    sm100::cluster_sync();
}

// Clears the counts of an earlier pass, after a later pass's meeting: by then every CTA has read them.
template <int C>
__device__ __forceinline__ void clear_counts(int* hist, int pass) {
  if (pass < 0) return;
  for (int i = threadIdx.x; i < kBins<C>; i += kThreads) hist[pass % kPasses<C> * kBins<C> + i] = 0;
}

// The digit that holds the `left`-th largest of the keys counted in the cluster's `count`; every thread of every CTA.
template <int C>
__device__ __forceinline__ Found find_digit(const int* count, int left, uint32_t rank, uint32_t (&sums)[kWarps], Found& found) {
  // thread t sums its digits over the cluster, in descending order, each CTA for itself
  constexpr int kOwn = kBins<C> > kThreads ? kBins<C> / kThreads : 1;
  const int top = kBins<C> - 1 - kOwn * (int)threadIdx.x;
  int n[kOwn] = {}, lower[kOwn] = {}, sum = 0;
  if (top >= 0) {
#pragma unroll
    for (uint32_t r = 0; r < C; ++r)
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int v = C == 1 ? count[top - i] : ld_cluster(&count[top - i], r);
        n[i] += v;
        lower[i] += r < rank ? v : 0;
        sum += v;
      }
  }
  const int x = block_scan(sum, sums);  // the prefix sums find the digit that holds rank `left`
  int above = x - sum;
  if (x >= left && above < left) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (above < left && above + n[i] >= left) found = {top - i, left - above, n[i], lower[i]};
      above += n[i];
    }
  }
  __syncthreads();
  return found;
}

// The age_key of the `recent`-th newest of the sequence's rows from lo on, of which this CTA has [c0, c1); 1 <= recent <=
// their number.  `pass` counts the passes, which take turns with the kPasses arrays of counts; the last one's is left as
// it is, since other CTAs may be reading it.
template <int C>
__device__ __forceinline__ uint64_t newest_from(const int32_t* positions, int lo, int c0, int c1, int recent, uint32_t rank,
                                                int* hist, SelectSmem& sm, int& pass) {
  const int tid = threadIdx.x;
  const int32_t some = positions[lo];
  uint32_t differ = 0u;
  for (int t = c0 + tid; t < c1; t += kThreads) differ |= (uint32_t)(positions[t] ^ some);
  differ = __reduce_or_sync(0xffffffffu, differ);
  if ((tid & 31) == 0) atomicOr(&sm.differ, (int)differ);
  meet<C>();
  for (uint32_t r = 0; r < C; ++r) differ |= (uint32_t)(C == 1 ? sm.differ : ld_cluster(&sm.differ, r));
  // from the highest bit in which positions differ; the bits between a position and a row's number are zeros
  int bits = differ != 0u ? 64 - __clz(differ) : kRowBits, left = recent;
  uint64_t mask = bits < 64 ? ~uint64_t(0) << bits : 0u, prefix = age_key(some, 0) & mask;
  for (bool found = false; !found && bits > 0; ++pass) {
    const int width = min(bits > 32 ? bits - 32 : bits, kDigitBits<C>), shift = bits - width;
    const uint32_t digit = (1u << width) - 1u;
    int* count = hist + pass % kPasses<C> * kBins<C>;
    for (int t = c0 + tid; t < c1; t += kThreads) {
      const uint64_t key = age_key(positions[t], t);
      if ((key & mask) == prefix) atomicAdd(&count[(uint32_t)(key >> shift) & digit], 1);
    }
    meet<C>();
    clear_counts<C>(hist, pass - 1);
    const Found f = find_digit<C>(count, left, rank, sm.sums[pass % kPasses<C>], sm.found[pass & 1]);
    prefix |= (uint64_t)f.digit << shift;
    mask |= (uint64_t)digit << shift;
    left = f.rank;
    found = f.rows == f.rank;
    bits = shift > kRowBits && shift <= 32 ? kRowBits : shift;
  }
  return prefix;  // (its lower bits are zeros)
}

// C CTAs (a cluster) per sequence; CTA r has the r-th slice of its rows (whole words of the mask).  kAged: the newest
// rows by position.
template <int C, bool kAged>
__device__ __forceinline__ void select_rows(const EvictArgs& a, bool keys_in_smem) {
  __shared__ SelectSmem sm;
  extern __shared__ __align__(16) int dyn[];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = C == 1 ? 0u : sm100::cluster_ctarank();
  const int len = a.lengths[b];
  int32_t* map = a.row_map + (int64_t)b * a.keep;
  const bool bad = len < 0 || len > a.n_max;
  if (bad || len <= a.keep) {
    const int n = bad ? 0 : len;
    for (int i = rank * kThreads + tid; i < a.keep; i += C * kThreads) map[i] = i < n ? i : -1;
    meet<C>();  // every thread has read lengths, which new_lengths may alias
    if (rank == 0 && tid == 0) {
      if (bad) raise_error(a.err, MLA_ERR_LENGTH);
      a.new_lengths[b] = n;
    }
    return;
  }
  const float* acc = a.acc + b * a.acc_b;
  const int words = (len + kWord - 1) / kWord, per = (words + C - 1) / C;  // words, of a slice
  const int r0 = min((int)rank * per * kWord, len), r1 = min(r0 + per * kWord, len);
  uint32_t* kept = reinterpret_cast<uint32_t*>(dyn);   // [per] kept rows of the slice
  uint32_t* tied = kept + per;                         // [per] rows at the threshold
  uint32_t* counts_before = tied + per;                // [per] holes and moved rows of the slice before each word
  int* list = dyn + (3 * per + 3) / 4 * 4;             // a part of the moved rows, in order
  int* hist = list;  // [kPasses][kBins] this CTA's counts of each digit, before the list is made
  uint32_t* keys = reinterpret_cast<uint32_t*>(list) + list_ints<C>(per);  // [per * 32], where they fit
  // rows that compete, and how many of them stay (kAged: the newest compete too, with the largest key)
  const int lo = a.sink, hi = kAged ? len : len - a.recent;
  const int c0 = max(r0, lo), c1 = min(r1, hi);
  const int want = a.keep - a.sink - (kAged ? 0 : a.recent);

  for (int i = tid; i < kPasses<C> * kBins<C>; i += kThreads) hist[i] = 0;
  if (kAged && tid == 0) sm.differ = 0;
  __syncthreads();
  const int32_t* positions = kAged ? a.positions + b * a.pos_b : nullptr;
  uint64_t newest = 0u;
  int pass = 0;
  if constexpr (kAged) newest = newest_from<C>(positions, lo, c0, c1, a.recent, rank, hist, sm, pass);
  auto row_key = [&](int t, float weight) {
    if (kAged && age_key(positions[t], t) >= newest) return 0xffffffffu;  // (above that of +infinity)
    return order_key(weight);
  };
  // radix select from the top: the want-th largest key, or as much of it as tells the kept rows from the others
  uint32_t prefix = 0u, mask = 0u;
  int left = want;  // keys equal to the prefix still to be taken
  int ties_before = 0;
  bool ties_all = true;  // every row at the threshold is kept
  for (int bits = 32; bits > 0 && want > 0; ++pass) {
    const int width = min(bits, kDigitBits<C>), shift = bits - width;
    const uint32_t digit = (1u << width) - 1u;
    int* count = hist + (kAged ? pass % kPasses<C> : pass) * kBins<C>;
    for (int f = c0; f < c1; f += kBatch * kThreads) {
      const int t0 = f + tid, some = (c1 - f + kThreads - 1) / kThreads;  // the block has keys in so many of the batch
      uint32_t k[kBatch];
      if (bits == 32 || !keys_in_smem) {
        float v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i < some) v[i] = t0 + i * kThreads < c1 ? acc[t0 + i * kThreads] : 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i < some) {
            k[i] = kAged && t0 + i * kThreads >= c1 ? 0u : row_key(t0 + i * kThreads, v[i]);
            if (keys_in_smem && t0 + i * kThreads < c1) keys[t0 + i * kThreads - r0] = k[i];
          }
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i < some) k[i] = t0 + i * kThreads < c1 ? keys[t0 + i * kThreads - r0] : 0u;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < some && t0 + i * kThreads < c1 && (k[i] & mask) == prefix) atomicAdd(&count[(k[i] >> shift) & digit], 1);
    }
    meet<C>();
    if (kAged) clear_counts<C>(hist, pass - 1);
    const Found f = find_digit<C>(count, left, rank, sm.sums[kAged ? pass % kPasses<C> : pass], sm.found[pass & 1]);
    prefix |= (uint32_t)f.digit << shift;
    mask |= digit << shift;
    left = f.rank;
    ties_before = f.lower;
    ties_all = f.rows == f.rank;
    bits = ties_all ? 0 : shift;
  }

  // kept and tied rows of the slice
  for (int wb = warp; wb < per; wb += kBatch * kWarps) {
    const int some = (per - wb + kWarps - 1) / kWarps;
    uint32_t k[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = r0 + (wb + i * kWarps) * kWord + lane;
      k[i] = 0u;
      if (i < some && t >= c0 && t < c1 && want > 0) k[i] = keys_in_smem ? keys[t - r0] : row_key(t, acc[t]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= some) break;
      const int w = wb + i * kWarps, t = r0 + w * kWord + lane;
      const bool inside = t >= lo && t < hi && t < r1;
      const uint32_t keep_w = __ballot_sync(0xffffffffu, inside ? want > 0 && (k[i] & mask) > prefix : t < r1);
      const uint32_t tie_w = __ballot_sync(0xffffffffu, inside && want > 0 && (k[i] & mask) == prefix);
      if (lane == 0) {
        kept[w] = keep_w;
        tied[w] = tie_w;
      }
    }
  }
  __syncthreads();
  // contiguous chunks of words for each thread, so that ranks follow from a scan over the threads
  const int chunk = (per + kThreads - 1) / kThreads;
  const int w0 = min(tid * chunk, per), w1 = min(w0 + chunk, per);
  int before = 0;  // rows at the threshold before this thread's
  if (!ties_all) {
    uint32_t ties = 0;
    for (int w = w0; w < w1; ++w) ties += __popc(tied[w]);
    before = ties_before + (int)(block_scan(ties, sm.sums[kPasses<kCluster>]) - ties);
  }
  auto below = [&](int w) {  // bits of the word whose row is below keep
    const int first = r0 + w * kWord;
    return first + kWord <= a.keep ? 0xffffffffu : first >= a.keep ? 0u : (1u << (a.keep - first)) - 1u;
  };
  auto rows_of = [&](int w) {  // bits of the word that are rows
    const int n = r1 - (r0 + w * kWord);
    return n >= kWord ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  };
  uint32_t count = 0u;  // holes, and 65536 times moved rows: a slice has at most 50000 rows
  for (int w = w0; w < w1; ++w) {
    const uint32_t tie = tied[w];
    const int here = __popc(tie), take = ties_all ? here : max(0, min(here, left - before));
    before += here;
    uint32_t k = kept[w];
    if (take == here)
      k |= tie;
    else if (take > 0)
      k |= tie & ((1u << nth_bit(tie, take)) - 1u);
    kept[w] = k;
    counts_before[w] = count;
    count += __popc(~k & rows_of(w) & below(w)) + (__popc(k & ~below(w)) << 16);
  }
  const uint32_t upto = block_scan(count, sm.sums[kPasses<kCluster> + 1]);
  for (int w = w0; w < w1; ++w) counts_before[w] += upto - count;
  if (tid == kThreads - 1) {
    sm.mine[0] = upto & 0xffffu;
    sm.mine[1] = upto >> 16;
  }
  meet<C>();
  const int holes0 = before_me<C>(&sm.mine[0], rank), moved0 = before_me<C>(&sm.mine[1], rank);
  // the moved rows in order, dealt out over the cluster
  for (int wb = warp; wb < per; wb += kBatch * kWarps) {
    const int some = (per - wb + kWarps - 1) / kWarps;
    uint32_t k[kBatch];
    int m[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int w = wb + i * kWarps;
      if (i >= some) break;
      k[i] = kept[w] & ~below(w);
      m[i] = moved0 + (int)(counts_before[w] >> 16) + __popc(k[i] & ((1u << lane) - 1u));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < some && ((k[i] >> lane) & 1u)) {
        const int row = r0 + (wb + i * kWarps) * kWord + lane;
        if (C == 1)
          list[m[i]] = row;
        else
          st_cluster(&list[(uint32_t)m[i] / C], (uint32_t)m[i] % C, row);
      }
  }
  meet<C>();
  // hole j takes the j-th of them
  for (int wb = warp; wb < per; wb += kBatch * kWarps) {
    const int some = (per - wb + kWarps - 1) / kWarps;
    int h[kBatch], src[kBatch];
    uint32_t in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int w = wb + i * kWarps;
      if (i >= some) break;
      in[i] = rows_of(w) & below(w);
      const uint32_t hole = ~kept[w] & in[i];
      src[i] = r0 + w * kWord + lane;
      h[i] = (hole >> lane) & 1u ? holes0 + (int)(counts_before[w] & 0xffffu) + __popc(hole & ((1u << lane) - 1u)) : -1;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < some && h[i] >= 0) src[i] = C == 1 ? list[h[i]] : ld_cluster(&list[(uint32_t)h[i] / C], (uint32_t)h[i] % C);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < some && ((in[i] >> lane) & 1u)) map[r0 + (wb + i * kWarps) * kWord + lane] = src[i];
  }
  if (rank == 0 && tid == 0) a.new_lengths[b] = a.keep;
  if (C > 1) meet<C>();  // no CTA leaves while another one may read its part of the list
}

template <bool kAged>
__global__ void __launch_bounds__(kThreads) evict_select_one(EvictArgs a, bool keys_in_smem) {
  select_rows<1, kAged>(a, keys_in_smem);
}
template <bool kAged>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    evict_select_cluster(EvictArgs a, bool keys_in_smem) {
  select_rows<kCluster, kAged>(a, keys_in_smem);
}

// The rows that move: a CTA compacts kMoveEntries entries of row_map to those that do; a warp copies two rows at a time,
// all planes' 16-byte (or smaller) elements numbered through, so that eight loads are under way per lane.
// (Entries of a CTA 256, 128, 64, 32: 29, 25, 23, 24 us for 4 sequences cut from 32768 rows to 16384, 12.5, 12.4, 13.3,
// 15.3 for 32 of 4096 rows that lose a few.)
constexpr int kMoveThreads = 256, kMoveEntries = 128;
template <typename V, bool kPositions>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
  __shared__ int dst[kMoveEntries], src[kMoveEntries], warp_n[kMoveEntries / 32];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int i = blockIdx.x * kMoveEntries + tid;
  const int from = tid < kMoveEntries && i < a.keep ? a.row_map[(int64_t)b * a.keep + i] : -1;
  const bool moves = from >= 0 && from != i && from < a.n_max;
  const uint32_t ballot = __ballot_sync(0xffffffffu, moves);
  if (lane == 0 && warp < kMoveEntries / 32) warp_n[warp] = __popc(ballot);
  __syncthreads();
  int at = __popc(ballot & ((1u << lane) - 1u)), n = 0;
#pragma unroll
  for (int w = 0; w < kMoveEntries / 32; ++w) {
    at += w < warp ? warp_n[w] : 0;
    n += warp_n[w];
  }
  if (moves) {
    dst[at] = i;
    src[at] = from;
    if constexpr (kPositions) a.positions[b * a.pos_b + i] = a.positions[b * a.pos_b + from];
  }
  __syncthreads();
  int first[MLA_MAX_PLANES + 1];  // elements of the planes before each one
  first[0] = 0;
#pragma unroll
  for (int p = 0; p < MLA_MAX_PLANES; ++p)
    first[p + 1] = first[p] + (p < a.n_planes ? a.planes[p].row_bytes / (int)sizeof(V) : 0);
  const int elements = first[MLA_MAX_PLANES];
  for (int e = warp; e < n; e += 2 * (kMoveThreads / 32))
    for (int c0 = lane; c0 < elements; c0 += 4 * 32) {
      V v[2][4];
      V* to[4];
      int64_t step[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 32 * k;
        if (c >= elements) break;
        int p = 0;
#pragma unroll
        for (int q = 1; q < MLA_MAX_PLANES; ++q) p += c >= first[q] ? 1 : 0;
        const mla_rows& pl = a.planes[p];
        uint8_t* base = static_cast<uint8_t*>(pl.base) + b * pl.bstride + (int64_t)(c - first[p]) * (int)sizeof(V);
        to[k] = reinterpret_cast<V*>(base);
        step[k] = pl.rstride;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int at_e = e + r * (kMoveThreads / 32);
          if (at_e < n) v[r][k] = *reinterpret_cast<const V*>(base + src[at_e] * pl.rstride);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int at_e = e + r * (kMoveThreads / 32);
          if (c0 + 32 * k < elements && at_e < n)
            *reinterpret_cast<V*>(reinterpret_cast<uint8_t*>(to[k]) + dst[at_e] * step[k]) = v[r][k];
        }
    }
}

template <typename V>
cudaError_t move_launch(const EvictArgs& a, dim3 grid, cudaStream_t st) {
  return launch_pdl(a.positions != nullptr ? evict_move_kernel<V, true> : evict_move_kernel<V, false>, grid, dim3(kMoveThreads), 0,
                    st, a);
}

// Shared memory of a CTA of the selection: masks and counts for each word, the list (or, before it, the
// counts of the digits) and the keys.
template <int C>
size_t select_smem_bytes(int n_max, bool keys) {
  const size_t words = (n_max + kWord - 1) / kWord, per = (words + C - 1) / C;
  return 16 * ((3 * per + 3) / 4) + 4 * ((size_t)list_ints<C>((int)per) + (keys ? per * kWord : 0));
}

}  // namespace

int evict_max_rows() { return kMaxRows; }

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  // One CTA for a short sequence, a cluster for a long one: the meetings of a cluster take longer than one CTA's passes
  // over some thousand keys in its shared memory, and a cluster's CTAs share the SMs with those of the other sequences.
  // The border moves up with their number.  One CTA / a cluster, us a call:
  //    8 sequences of 1024 rows 13 / 18, 4096 16 / 20, 8192 20 / 23, 16384 30 / 25
  //   16 of 8192 19 / 30, 16384 32 / 36, 24000 43 / 39;   26 of 16384 36 / 43, 24000 50 / 50, 32768 65 / 59
  //   37 of 24000 57 / 70, 32768 76 / 84;   64 of 4096 19 / 66, 16384 51 / 93, 32768 110 / 150
  const bool one = a.n_max <= kOneCta || (a.n_max <= kOneCtaFull && a.n_max / kOneCtaPer <= a.B);
  const auto bytes = one ? select_smem_bytes<1> : select_smem_bytes<kCluster>;
  const bool keys = bytes(a.n_max, true) <= kSelectSmem;
  const size_t smem = bytes(a.n_max, keys);
  const bool aged = a.positions != nullptr && a.recent > 0;
  const auto kernel = one ? aged ? evict_select_one<true> : evict_select_one<false>
                          : aged ? evict_select_cluster<true> : evict_select_cluster<false>;
  static PerDevice allowed[4];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSelectSmem, allowed[2 * one + aged]);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(a.B * (one ? 1 : kCluster)), dim3(kThreads), smem, st, a, keys);
  if (e != cudaSuccess) return e;
  // the widest element that every plane's base, strides and rows are multiples of
  uintptr_t bits = 0;
  for (int p = 0; p < a.n_planes; ++p)
    bits |= reinterpret_cast<uintptr_t>(a.planes[p].base) | (uintptr_t)a.planes[p].bstride |
            (uintptr_t)a.planes[p].rstride | (uintptr_t)a.planes[p].row_bytes;
  const dim3 grid((a.keep + kMoveEntries - 1) / kMoveEntries, a.B);
  if (bits % 16 == 0) return move_launch<uint4>(a, grid, st);
  if (bits % 4 == 0) return move_launch<uint32_t>(a, grid, st);
  return move_launch<uint8_t>(a, grid, st);
}

}  // namespace mla
