// Eviction from a cache by accumulated attention weight.
//
// Per sequence with L > keep rows: kept are the first `sink` rows, the last `recent` rows, and the
// keep - sink - recent rows of largest accumulated weight among the rest (ties: the lower row; NaN
// counts as the least).  Attention does not depend on the order of the rows (the rotary key carries
// each row's position), so nothing is shifted: the kept rows behind `keep` move into the holes before
// it, j-th hole from j-th row.  That moves the fewest bytes, and since sources lie at or behind `keep` and
// destinations before it, no row is read after it was written: the move needs no order and no copy.
//
// Two launches: the selection writes row_map (one CTA per sequence), the move reads it.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMaxRows = 400000;  // twelve bytes of shared memory for 32 rows

// Order-preserving map of a float to 32 bits: NaN is the least, -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

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
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Rows of a sequence that one 32-bit word of the kept mask holds.
constexpr int kWord = 32;

// Position of the n-th (from 0) set bit of m.
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return __ffs(m) - 1;
}

// Shared arrays of one selection: per word of 32 rows the kept mask, and the rows that go before it
// (holes, rows < keep) or that move from before it (rows >= keep).
struct SelectSmem {
  uint32_t* kept;
  int* holes;
  int* moved;
};
size_t select_smem_bytes(int n_max) { return (size_t)((n_max + kWord - 1) / kWord) * 12; }

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rank;
  extern __shared__ uint32_t dyn[];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int len = a.lengths[b];
  int32_t* map = a.row_map + (int64_t)b * a.keep;
  const bool bad = len < 0 || len > a.n_max;
  if (bad || len <= a.keep) {
    const int n = bad ? 0 : len;
    for (int i = tid; i < a.keep; i += kSelThreads) map[i] = i < n ? i : -1;
    __syncthreads();  // every thread has read lengths, which new_lengths may alias
    if (tid == 0) {
      if (bad) raise_error(a.err, MLA_ERR_LENGTH);
      a.new_lengths[b] = n;
    }
    return;
  }
  const float* acc = a.acc + b * a.acc_b;
  const int lo = a.sink, hi = len - a.recent;  // rows that compete
  const int want = a.keep - a.sink - a.recent;
  // radix select, eight bits a pass from the top: the want-th largest key
  uint32_t prefix = 0u, mask = 0u;
  int rank = want;  // keys equal to the prefix still to be taken
  for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t k = order_key(acc[t]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, r = rank;
      while (d > 0 && hist[d] < r) r -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_rank = r;
    }
    __syncthreads();
    prefix = s_prefix;
    rank = s_rank;
    mask |= 255u << shift;
    __syncthreads();
  }
  const int words = (a.n_max + kWord - 1) / kWord, used = (len + kWord - 1) / kWord;
  const SelectSmem sm{dyn, reinterpret_cast<int*>(dyn + words), reinterpret_cast<int*>(dyn + 2 * words)};
  uint32_t* ties = reinterpret_cast<uint32_t*>(sm.holes);  // until the ties are settled
  for (int w = tid / 32; w < used; w += kSelThreads / 32) {
    const int t = w * kWord + lane;
    const bool inside = t >= lo && t < hi;
    const uint32_t k = inside && want > 0 ? order_key(acc[t]) : 0u;
    const uint32_t keep_w = __ballot_sync(0xffffffffu, inside ? want > 0 && k > prefix : t < len);
    const uint32_t tie_w = __ballot_sync(0xffffffffu, inside && want > 0 && k == prefix);
    if (lane == 0) {
      sm.kept[w] = keep_w;
      ties[w] = tie_w;
    }
  }
  __syncthreads();
  // contiguous chunks of words for each thread, so that ranks follow from a scan over the threads
  const int chunk = (used + kSelThreads - 1) / kSelThreads;
  const int w0 = min(tid * chunk, used), w1 = min(w0 + chunk, used);
  int n_ties = 0, total;
  for (int w = w0; w < w1; ++w) n_ties += __popc(ties[w]);
  int before = block_scan(n_ties, warp_sums, &total);
  int n_holes = 0, n_moved = 0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t tie = ties[w];
    const int here = __popc(tie), take = max(0, min(here, rank - before));
    before += here;
    uint32_t k = sm.kept[w];
    if (take == here)
      k |= tie;
    else if (take > 0)
      k |= tie & ((1u << nth_bit(tie, take)) - 1u);
    sm.kept[w] = k;
    const int first = w * kWord;  // bits of this word whose row is below keep
    const uint32_t low = first + kWord <= a.keep ? 0xffffffffu : first >= a.keep ? 0u : (1u << (a.keep - first)) - 1u;
    n_holes += __popc(~k & low);
    n_moved += __popc(k & ~low);
  }
  int h = block_scan(n_holes, warp_sums, &total);
  int m = block_scan(n_moved, warp_sums, &total);
  for (int w = w0; w < w1; ++w) {
    const uint32_t k = sm.kept[w];
    const int first = w * kWord;
    const uint32_t low = first + kWord <= a.keep ? 0xffffffffu : first >= a.keep ? 0u : (1u << (a.keep - first)) - 1u;
    sm.holes[w] = h;
    sm.moved[w] = m;
    h += __popc(~k & low);
    m += __popc(k & ~low);
  }
  __syncthreads();
  // hole j takes the j-th kept row from keep on: the last word with at most j such rows before it
  const int first_word = a.keep / kWord;
  for (int i = tid; i < a.keep; i += kSelThreads) {
    const uint32_t k = sm.kept[i / kWord];
    int src = i;
    if (!((k >> (i % kWord)) & 1u)) {
      const int j = sm.holes[i / kWord] + __popc(~k & ((1u << (i % kWord)) - 1u));
      int l = first_word, r = used - 1;
      while (l < r) {
        const int mid = (l + r + 1) / 2;
        if (sm.moved[mid] <= j)
          l = mid;
        else
          r = mid - 1;
      }
      uint32_t k2 = sm.kept[l];
      if (l == first_word) k2 &= ~((1u << (a.keep % kWord)) - 1u);
      src = l * kWord + nth_bit(k2, j - sm.moved[l]);
    }
    map[i] = src;
  }
  if (tid == 0) a.new_lengths[b] = a.keep;
}

// One warp per 32 entries of row_map: the entries that move are copied plane by plane.
template <typename V>
__global__ void __launch_bounds__(128) evict_move_kernel(EvictArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int i0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 32;
  const int i = i0 + lane;
  const int src = i < a.keep ? a.row_map[(int64_t)b * a.keep + i] : -1;
  uint32_t todo = __ballot_sync(0xffffffffu, src >= 0 && src != i);
  while (todo) {
    const int j = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t from = __shfl_sync(0xffffffffu, src, j), to = i0 + j;
    for (int p = 0; p < a.n_planes; ++p) {
      const mla_rows& pl = a.planes[p];
      uint8_t* base = static_cast<uint8_t*>(pl.base) + b * pl.bstride;
      const V* s = reinterpret_cast<const V*>(base + from * pl.rstride);
      V* d = reinterpret_cast<V*>(base + to * pl.rstride);
      for (int k = lane; k < pl.row_bytes / (int)sizeof(V); k += 32) d[k] = s[k];
    }
  }
}

}  // namespace

int evict_max_rows() { return kMaxRows; }

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  const size_t smem = select_smem_bytes(a.n_max);
  static int allowed[kMaxDevices];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), (int)smem, allowed);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<a.B, kSelThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the widest element that every plane's base, strides and rows are multiples of
  uintptr_t bits = 0;
  for (int p = 0; p < a.n_planes; ++p)
    bits |= reinterpret_cast<uintptr_t>(a.planes[p].base) | (uintptr_t)a.planes[p].bstride |
            (uintptr_t)a.planes[p].rstride | (uintptr_t)a.planes[p].row_bytes;
  const dim3 grid((a.keep + 127) / 128, a.B);
  if (bits % 16 == 0)
    evict_move_kernel<uint4><<<grid, 128, 0, st>>>(a);
  else if (bits % 4 == 0)
    evict_move_kernel<uint32_t><<<grid, 128, 0, st>>>(a);
  else
    evict_move_kernel<uint8_t><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
