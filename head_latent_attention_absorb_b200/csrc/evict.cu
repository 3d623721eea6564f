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
// rows, or one CTA for a short sequence; counts, ranks and the list of moved rows cross through distributed shared memory), the move reads it.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512;   // of a CTA of the selection
constexpr int kCluster = 8;     // CTAs that share a sequence
constexpr int kOneCta = 8192;     // rows that one CTA selects from by itself
constexpr int kSelectSmem = 220 * 1024;
constexpr int kMaxRows = 400000;  // 4.5 bytes of a CTA's shared memory for kCluster rows
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
  int warp_sums[2][kThreads / 32];
  int bin, rank;           // the digit found and what is still to be taken of its keys
  int mine[2];             // this CTA's holes and moved rows
};

// Exclusive prefix sums of two values over the block's threads; total gets the sums.
__device__ __forceinline__ int2 block_scan(int2 v, int (&warp_sums)[2][kThreads / 32], int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, x.x, o), y1 = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += y0;
      x.y += y1;
    }
  }
  __syncthreads();
  if (lane == 31) {
    warp_sums[0][warp] = x.x;
    warp_sums[1][warp] = x.y;
  }
  __syncthreads();
  int2 before = make_int2(0, 0), all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s0 = warp_sums[0][w], s1 = warp_sums[1][w];
    before.x += w < warp ? s0 : 0;
    before.y += w < warp ? s1 : 0;
    all.x += s0;
    all.y += s1;
  }
  *total = all;
  return make_int2(x.x - v.x + before.x, x.y - v.y + before.y);
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

// C CTAs (a cluster) per sequence; CTA r has the r-th slice of its rows (whole words of the mask).
template <int C>
__device__ __forceinline__ void select_rows(const EvictArgs& a, bool keys_in_smem) {
  __shared__ SelectSmem sm;
  extern __shared__ int dyn[];
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
  int* holes_before = dyn + 2 * per;                   // [per]
  int* moved_before = dyn + 3 * per;                   // [per]
  int* list = dyn + 4 * per;                           // [per * 32] a part of the moved rows, in order
  uint32_t* keys = reinterpret_cast<uint32_t*>(list) + per * kWord;  // [per * 32], where they fit
  const int lo = a.sink, hi = len - a.recent;          // rows that compete
  const int c0 = max(r0, lo), c1 = min(r1, hi);
  const int want = a.keep - a.sink - a.recent;
  auto key = [&](int t) { return keys_in_smem ? keys[t - r0] : order_key(acc[t]); };

  for (int i = tid; i < 4 * 256; i += kThreads) sm.hist[i >> 8][i & 255] = 0;
  if (keys_in_smem) {
#pragma unroll 8
    for (int t = r0 + tid; t < r1; t += kThreads) keys[t - r0] = order_key(acc[t]);
  }
  __syncthreads();
  // radix select, eight bits a pass from the top: the want-th largest key
  uint32_t prefix = 0u, mask = 0u;
  int left = want;  // keys equal to the prefix still to be taken
  int ties_before = 0;
  for (int pass = 0; pass < 4 && want > 0; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll 4
    for (int t = c0 + tid; t < c1; t += kThreads) {
      const uint32_t k = key(t);
      if ((k & mask) == prefix) atomicAdd(&sm.hist[pass][(k >> shift) & 255u], 1);
    }
    meet<C>();
    if (tid < 256) {  // thread t sums digit 255 - t over the cluster, each CTA for itself
      int n = 0, lower = 0;
#pragma unroll
      for (uint32_t r = 0; r < C; ++r) {
        const int v = C == 1 ? sm.hist[pass][255 - tid] : ld_cluster(&sm.hist[pass][255 - tid], r);
        n += v;
        lower += r < rank ? v : 0;
      }
      // descending digits: inclusive prefix sums find the one that holds rank `left`
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sm.warp_sums[0][warp] = x;
      asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
      for (int w = 0; w < 7; ++w) x += w < warp ? sm.warp_sums[0][w] : 0;
      if (x >= left && x - n < left) {
        sm.bin = 255 - tid;
        sm.rank = left - (x - n);
        sm.mine[0] = lower;  // (in the last pass: rows at the threshold in the slices before this one)
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sm.bin << shift;
    left = sm.rank;
    ties_before = sm.mine[0];
    mask |= 255u << shift;
    __syncthreads();
  }

  // kept and tied rows of the slice
  for (int w = warp; w < per; w += kThreads / 32) {
    const int t = r0 + w * kWord + lane;
    const bool inside = t >= lo && t < hi && t < r1;
    const uint32_t k = inside && want > 0 ? key(t) : 0u;
    const uint32_t keep_w = __ballot_sync(0xffffffffu, inside ? want > 0 && k > prefix : t < r1);
    const uint32_t tie_w = __ballot_sync(0xffffffffu, inside && want > 0 && k == prefix);
    if (lane == 0) {
      kept[w] = keep_w;
      tied[w] = tie_w;
    }
  }
  __syncthreads();
  // contiguous chunks of words for each thread, so that ranks follow from a scan over the threads
  const int chunk = (per + kThreads - 1) / kThreads;
  const int w0 = min(tid * chunk, per), w1 = min(w0 + chunk, per);
  int ties = 0;
  int2 total;
  for (int w = w0; w < w1; ++w) ties += __popc(tied[w]);
  int before = ties_before + block_scan(make_int2(ties, 0), sm.warp_sums, &total).x;
  auto below = [&](int w) {  // bits of the word whose row is below keep
    const int first = r0 + w * kWord;
    return first + kWord <= a.keep ? 0xffffffffu : first >= a.keep ? 0u : (1u << (a.keep - first)) - 1u;
  };
  auto rows_of = [&](int w) {  // bits of the word that are rows
    const int n = r1 - (r0 + w * kWord);
    return n >= kWord ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  };
  int2 count = make_int2(0, 0);  // holes, moved rows
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
    holes_before[w] = count.x;
    moved_before[w] = count.y;
    count.x += __popc(~k & rows_of(w) & below(w));
    count.y += __popc(k & ~below(w));
  }
  const int2 at = block_scan(count, sm.warp_sums, &total);
  for (int w = w0; w < w1; ++w) {
    holes_before[w] += at.x;
    moved_before[w] += at.y;
  }
  if (tid == 0) {
    sm.mine[0] = total.x;
    sm.mine[1] = total.y;
  }
  meet<C>();
  const int holes0 = before_me<C>(&sm.mine[0], rank), moved0 = before_me<C>(&sm.mine[1], rank);
  // the moved rows in order, spread over the cluster (there are fewer than rows, so a slice's worth fits)
  const int room = per * kWord;
  for (int w = warp; w < per; w += kThreads / 32) {
    const uint32_t k = kept[w] & ~below(w);
    if ((k >> lane) & 1u) {
      const int m = moved0 + moved_before[w] + __popc(k & ((1u << lane) - 1u)), row = r0 + w * kWord + lane;
      if (C == 1)
        list[m % room] = row;
      else
        st_cluster(&list[m % room], (uint32_t)(m / room) % C, row);
    }
  }
  meet<C>();
  // hole j takes the j-th of them
  for (int w = warp; w < per; w += kThreads / 32) {
    const uint32_t in = rows_of(w) & below(w);
    if (in == 0u) continue;
    const uint32_t hole = ~kept[w] & in;
    int src = r0 + w * kWord + lane;
    if ((hole >> lane) & 1u) {
      const int h = holes0 + holes_before[w] + __popc(hole & ((1u << lane) - 1u));
      src = C == 1 ? list[h % room] : ld_cluster(&list[h % room], (uint32_t)(h / room) % C);
    }
    if ((in >> lane) & 1u) map[r0 + w * kWord + lane] = src;
  }
  if (rank == 0 && tid == 0) a.new_lengths[b] = a.keep;
  if (C > 1) meet<C>();  // no CTA leaves while another one may read its part of the list
}

__global__ void __launch_bounds__(kThreads) evict_select_one(EvictArgs a, bool keys_in_smem) {
  select_rows<1>(a, keys_in_smem);
}
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    evict_select_cluster(EvictArgs a, bool keys_in_smem) {
  select_rows<kCluster>(a, keys_in_smem);
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

// Shared memory of a CTA of the selection: four words of masks and counts and a list entry for every row of a slice,
// and the keys.
size_t select_smem_bytes(int n_max, int ctas, bool keys) {
  const size_t words = (n_max + kWord - 1) / kWord, per = (words + ctas - 1) / ctas;
  return per * (16 + 4 * kWord * (keys ? 2 : 1));
}

}  // namespace

int evict_max_rows() { return kMaxRows; }

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  // One CTA for a sequence of up to kOneCta rows: a meeting of a cluster takes about a microsecond, a pass of one
  // CTA over that many keys in shared memory less.
  const bool one = a.n_max <= kOneCta;
  const int ctas = one ? 1 : kCluster;
  const bool keys = select_smem_bytes(a.n_max, ctas, true) <= kSelectSmem;
  const size_t smem = select_smem_bytes(a.n_max, ctas, keys);
  static int allowed_one[kMaxDevices], allowed_cluster[kMaxDevices];
  cudaError_t e = one ? allow_smem(reinterpret_cast<const void*>(evict_select_one), kSelectSmem, allowed_one)
                      : allow_smem(reinterpret_cast<const void*>(evict_select_cluster), kSelectSmem, allowed_cluster);
  if (e != cudaSuccess) return e;
  e = launch_pdl(one ? evict_select_one : evict_select_cluster, dim3(a.B * ctas), dim3(kThreads), smem, st, a, keys);
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
