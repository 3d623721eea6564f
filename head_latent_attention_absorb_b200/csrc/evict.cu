// Eviction from a cache by accumulated attention weight.
//
// Per sequence with L > keep rows: kept are the first `sink` rows, the last `recent` rows, and the
// keep - sink - recent rows of largest accumulated weight among the rest (ties: the lower row; NaN
// counts as the least).  Attention does not depend on the order of the rows (the rotary key carries
// each row's position), so nothing is shifted: the kept rows behind `keep` move into the holes before
// it, j-th hole from j-th row.  That moves the fewest bytes, and since sources lie at or behind `keep` and
// destinations before it, no row is read after it was written: the move needs no order and no copy.
//
// Two launches: the selection writes row_map (a cluster of eight CTAs per sequence, each with a slice of the
// rows; counts, ranks and the list of moved rows cross through distributed shared memory), the move reads it.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512;   // of a CTA of the selection
constexpr int kCluster = 8;     // CTAs that share a sequence
constexpr int kMaxRows = 400000;  // 4 bytes of a CTA's shared memory for kCluster rows, and an eighth
constexpr int kWord = 32;       // rows of one word of the kept mask

// Order-preserving map of a float to 32 bits: NaN is the least, -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
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

struct SelectSmem {
  int hist[4][256];        // this CTA's counts, one array for each digit
  int warp_sums[16];
  int bin, rank;           // the digit found and what is still to be taken of its keys
  int mine[3];             // this CTA's ties, holes and moved rows
};

// Exclusive prefix sum of v over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s = warp_sums[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  return x - v + before;
}

// Sum of the lower-ranked CTAs' value, once the cluster has met.
__device__ __forceinline__ int before_me(const int* p, uint32_t rank) {
  int sum = 0;
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r) {
    const int v = ld_cluster(p, r);
    sum += r < rank ? v : 0;
  }
  return sum;
}

// One cluster per sequence; CTA r has the r-th slice of its rows (whole words of the mask).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
  __shared__ SelectSmem sm;
  extern __shared__ int dyn[];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int b = blockIdx.x / kCluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = sm100::cluster_ctarank();
  const int len = a.lengths[b];
  int32_t* map = a.row_map + (int64_t)b * a.keep;
  const bool bad = len < 0 || len > a.n_max;
  if (bad || len <= a.keep) {
    const int n = bad ? 0 : len;
    for (int i = rank * kThreads + tid; i < a.keep; i += kCluster * kThreads) map[i] = i < n ? i : -1;
    sm100::cluster_sync();  // every thread has read lengths, which new_lengths may alias
    if (rank == 0 && tid == 0) {
      if (bad) raise_error(a.err, MLA_ERR_LENGTH);
      a.new_lengths[b] = n;
    }
    return;
  }
  const float* acc = a.acc + b * a.acc_b;
  const int words = (len + kWord - 1) / kWord, per = (words + kCluster - 1) / kCluster;  // words, of a slice
  const int r0 = min((int)rank * per * kWord, len), r1 = min(r0 + per * kWord, len);
  uint32_t* kept = reinterpret_cast<uint32_t*>(dyn);  // [per] kept rows of the slice
  uint32_t* tied = kept + per;                        // [per] rows at the threshold
  int* list = dyn + 2 * per;                          // [per * 32] a part of the moved rows, in order
  const int lo = a.sink, hi = len - a.recent;         // rows that compete
  const int c0 = max(r0, lo), c1 = min(r1, hi);
  const int want = a.keep - a.sink - a.recent;

  // radix select, eight bits a pass from the top: the want-th largest key
  for (int i = tid; i < 4 * 256; i += kThreads) sm.hist[i >> 8][i & 255] = 0;
  __syncthreads();
  uint32_t prefix = 0u, mask = 0u;
  int left = want;  // keys equal to the prefix still to be taken
  for (int pass = 0; pass < 4 && want > 0; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll 4
    for (int t = c0 + tid; t < c1; t += kThreads) {
      const uint32_t k = order_key(acc[t]);
      if ((k & mask) == prefix) atomicAdd(&sm.hist[pass][(k >> shift) & 255u], 1);
    }
    sm100::cluster_sync();
    // warp w sums digits 16 w .. 16 w + 15 over the cluster, each CTA for itself
    if (tid < 256) {
      int n = 0;
#pragma unroll
      for (uint32_t r = 0; r < kCluster; ++r) n += ld_cluster(&sm.hist[pass][255 - tid], r);
      // descending digits: inclusive prefix sums find the one that holds rank `left`
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sm.warp_sums[warp] = x;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int w = 0; w < warp; ++w) x += sm.warp_sums[w];
      if (x >= left && x - n < left) {
        sm.bin = 255 - tid;
        sm.rank = left - (x - n);
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sm.bin << shift;
    left = sm.rank;
    mask |= 255u << shift;
    __syncthreads();
  }

  // kept and tied rows of the slice
  int n_ties = 0;
  for (int w = warp; w < per; w += kThreads / 32) {
    const int t = r0 + w * kWord + lane;
    const bool inside = t >= lo && t < hi && t < r1;
    const uint32_t k = inside && want > 0 ? order_key(acc[t]) : 0u;
    const uint32_t keep_w = __ballot_sync(0xffffffffu, inside ? want > 0 && k > prefix : t < r1);
    const uint32_t tie_w = __ballot_sync(0xffffffffu, inside && want > 0 && k == prefix);
    n_ties += __popc(tie_w);
    if (lane == 0) {
      kept[w] = keep_w;
      tied[w] = tie_w;
    }
  }
  if (lane == 0) sm.warp_sums[warp] = n_ties;
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int w = 0; w < kThreads / 32; ++w) n += sm.warp_sums[w];
    sm.mine[0] = n;
  }
  sm100::cluster_sync();
  // contiguous chunks of words for each thread, so that ranks follow from a scan over the threads
  const int chunk = (per + kThreads - 1) / kThreads;
  const int w0 = min(tid * chunk, per), w1 = min(w0 + chunk, per);
  int ties = 0, total;
  for (int w = w0; w < w1; ++w) ties += __popc(tied[w]);
  int before = before_me(&sm.mine[0], rank) + block_scan(ties, sm.warp_sums, &total);
  auto below = [&](int w) {  // bits of the word whose row is below keep
    const int first = r0 + w * kWord;
    return first + kWord <= a.keep ? 0xffffffffu : first >= a.keep ? 0u : (1u << (a.keep - first)) - 1u;
  };
  auto rows_of = [&](int w) {  // bits of the word that are rows
    const int n = r1 - (r0 + w * kWord);
    return n >= kWord ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  };
  int holes = 0, moved = 0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t tie = tied[w];
    const int here = __popc(tie), take = max(0, min(here, left - before));
    before += here;
    uint32_t k = kept[w];
    if (take == here)
      k |= tie;
    else if (take > 0)
      k |= tie & ((1u << nth_bit(tie, take)) - 1u);
    kept[w] = k;
    holes += __popc(~k & rows_of(w) & below(w));
    moved += __popc(k & ~below(w));
  }
  int h = block_scan(holes, sm.warp_sums, &total);
  if (tid == 0) sm.mine[1] = total;
  int m = block_scan(moved, sm.warp_sums, &total);
  if (tid == 0) sm.mine[2] = total;
  sm100::cluster_sync();
  h += before_me(&sm.mine[1], rank);
  m += before_me(&sm.mine[2], rank);
  // the moved rows in order, spread over the cluster (there are fewer than rows, so a slice's worth fits)
  const int room = per * kWord;
  for (int w = w0; w < w1; ++w)
    for (uint32_t k = kept[w] & ~below(w); k != 0u; k &= k - 1, ++m)
      st_cluster(&list[m % room], (uint32_t)(m / room) % kCluster, r0 + w * kWord + __ffs(k) - 1);
  sm100::cluster_sync();
  // hole j takes the j-th of them
  for (int w = w0; w < w1; ++w) {
    const int first = r0 + w * kWord;
    const uint32_t in = rows_of(w) & below(w);
    for (uint32_t k = in; k != 0u; k &= k - 1) {
      const int i = __ffs(k) - 1;
      int src = first + i;
      if (!((kept[w] >> i) & 1u)) {
        src = ld_cluster(&list[h % room], (uint32_t)(h / room) % kCluster);
        ++h;
      }
      map[first + i] = src;
    }
  }
  if (rank == 0 && tid == 0) a.new_lengths[b] = a.keep;
  sm100::cluster_sync();  // no CTA leaves while another one may read its part of the list
}

// The rows that move: a CTA compacts 256 entries of row_map to those that do; a warp copies two rows at a time,
// all planes' 16-byte (or smaller) elements numbered through, so that eight loads are under way per lane.
constexpr int kMoveThreads = 256;
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
  __shared__ int dst[kMoveThreads], src[kMoveThreads], warp_n[kMoveThreads / 32];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int i = blockIdx.x * kMoveThreads + tid;
  const int from = i < a.keep ? a.row_map[(int64_t)b * a.keep + i] : -1;
  const bool moves = from >= 0 && from != i && from < a.n_max;
  const uint32_t ballot = __ballot_sync(0xffffffffu, moves);
  if (lane == 0) warp_n[warp] = __popc(ballot);
  __syncthreads();
  int at = __popc(ballot & ((1u << lane) - 1u)), n = 0;
#pragma unroll
  for (int w = 0; w < kMoveThreads / 32; ++w) {
    at += w < warp ? warp_n[w] : 0;
    n += warp_n[w];
  }
  if (moves) {
    dst[at] = i;
    src[at] = from;
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

// Shared memory of the selection: two words of masks and a list entry for every row of a slice
size_t select_smem_bytes(int n_max) {
  const size_t words = (n_max + kWord - 1) / kWord, per = (words + kCluster - 1) / kCluster;
  return per * (8 + 4 * kWord);
}

}  // namespace

int evict_max_rows() { return kMaxRows; }

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  const size_t smem = select_smem_bytes(a.n_max);
  static int allowed[kMaxDevices];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), (int)smem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(evict_select_kernel, dim3(a.B * kCluster), dim3(kThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  // the widest element that every plane's base, strides and rows are multiples of
  uintptr_t bits = 0;
  for (int p = 0; p < a.n_planes; ++p)
    bits |= reinterpret_cast<uintptr_t>(a.planes[p].base) | (uintptr_t)a.planes[p].bstride |
            (uintptr_t)a.planes[p].rstride | (uintptr_t)a.planes[p].row_bytes;
  const dim3 grid((a.keep + kMoveThreads - 1) / kMoveThreads, a.B);
  if (bits % 16 == 0) return launch_pdl(evict_move_kernel<uint4>, grid, dim3(kMoveThreads), 0, st, a);
  if (bits % 4 == 0) return launch_pdl(evict_move_kernel<uint32_t>, grid, dim3(kMoveThreads), 0, st, a);
  return launch_pdl(evict_move_kernel<uint8_t>, grid, dim3(kMoveThreads), 0, st, a);
}

}  // namespace mla
