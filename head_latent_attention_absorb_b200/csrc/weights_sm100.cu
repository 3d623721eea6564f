// Attention weights of the cached rows on tcgen05 tensor cores (sm_100a):
//   out[t] = [t < L - T] decay acc[t] + sum over query rows r of exp(scale (q_r . key_t) - lse_r)
// with the R = T n_h query rows of a sequence, q_r = [q~ | q_pe] and key_t = [c_t | k^R_t] (576 features).
//
// The scores are computed transposed, S^T = K Q^T: the 128 keys of a tile are the rows (TMEM lanes) of the
// accumulator and up to 128 query rows its columns, so the sum over query rows is a sum within a thread and
// nothing is exchanged.  Since lse is known there is no running maximum and no second pass.
//
// Bound: a bf16 cache by its bytes (1152 a row): B = 32, N = 4096, 128 heads 29.1 us, 151 MB at 5.2 TB/s (N = 16384:
// 91 us, 6.6 TB/s); a tile takes 5500 cycles of the bytes' and 3850 of the MMAs' time.  A 4-bit cache (416 bytes a
// row) by the decode beside the MMAs, some 6500 cycles a tile in which neither the tensor pipe nor the ALUs nor
// shared memory is half busy: the slabs' proxy fences wait for the loads under way.  B = 8, up to 16384 rows 21 us,
// B = 32, N = 16384 111 us.  7 us go before the first tile (launch, share of the work, the first slabs) and 2 after
// the last.  (A CTA pair that splits the query rows, with a ring of nine slabs, took 35 and 25 us instead of 29 and
// 21: its start and end cost 4 us more.  Sixteen decode warps instead of eight: the same.)
//
// * One CTA per SM takes an equal share of the batch's 128-key tiles.  The query rows of its sequence (144 KB
//   in nine 64-feature slabs) stay in shared memory; the keys pass through a ring of five 16 KB slabs.
// * bf16 cache: TMA boxes fill the ring.  4-bit cache: eight warps load codes and scales into registers one
//   tile ahead and write bf16 slabs (code * scale * latent_scale is exact in bf16) in the same layout.
// * The accumulator is double-buffered, so the four warps that take exponentials and sums run beside the
//   next tile's MMAs.
// * More than 128 query rows: groups of 128, one after the other over pieces of four tiles, so that the
//   repeated reads of the keys come from L2.
// * Every wait is bounded; on expiry the kernel records MLA_ERR_TIMEOUT, lets its copies land and returns.
#include <math.h>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "tile_range.cuh"
#include "tma_host.h"

namespace mla {
namespace weights_tc {

using namespace sm100;

constexpr int kDC = 512, kDR = 64;
constexpr int kTile = 128;                   // keys per tile: the rows of an MMA
constexpr int kRows = 128;                   // query rows per group: its columns
constexpr int kSlabs = (kDC + kDR) / 64;     // 64-feature slabs of a row
constexpr int kSlabBytes = kTile * 128;      // 128 rows of 64 bf16 features
constexpr int kStages = 5;
// Tiles per piece when several groups of query rows pass over them.  (1, 4, 16: 52, 43 and 43 us for 4 sequences of 8192
// bf16 rows with 8 tokens of 128 heads; a short piece keeps its keys in L2 between the groups.)
constexpr int kGroupPiece = 4;
constexpr int kQWarp = 6, kKeyWarp = 5, kMmaWarp = 4, kDecodeWarp0 = 7, kDecodeWarps = 8;
constexpr int kThreadsBf16 = 32 * kDecodeWarp0, kThreadsFp4 = 32 * (kDecodeWarp0 + kDecodeWarps);
constexpr uint32_t kTmemCols = 256;          // two accumulators of 128 columns
constexpr uint64_t kWaitLimitNs = 1000000000ull;

struct Params {
  CUtensorMap tm_ckv;  // bf16 cache: (d_c, n_max, B), box (64, 128, 1), 128-byte swizzle
  CUtensorMap tm_kr;   // (d_r, n_max, B), same box
  CUtensorMap tm_q;    // (d_c, R, B) query rows, same box: rows past R read as zeros
  CUtensorMap tm_qp;   // (d_r, R, B)
  CacheView kv;        // 4-bit cache
  const int32_t* lengths;
  int B, T, n_h, n_max, ckv_z, kr_z;  // z: 0 where all sequences share one cache (batch stride 0)
  float scale_log2;
  const float* lse;
  const float* acc;
  int64_t acc_b;
  float decay;
  float* out;
  int64_t out_b;
  int32_t* err;
};

struct Smem {
  uint64_t full[kStages], empty[kStages], q_full[kSlabs], q_empty, s_full[2], s_empty[2], drain;
  alignas(16) float neg_lse[kRows];  // -lse in log2 units, -inf for absent and dropped rows
  int dropped[4];        // some present row of the quarter has no softmax
  uint32_t tmem_base;
  int abort, never;
  TileRange range;
};
constexpr int kRingOff = kSlabs * kSlabBytes;
constexpr int kSmemOff = kRingOff + kStages * kSlabBytes;
constexpr int kSmemBytes = kSmemOff + (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory above 227 KB");

// Bounded wait that records its own expiry.
__device__ __forceinline__ bool wait(Smem& sm, uint64_t& bar, uint32_t parity, int32_t* err) {
  if (mbar_wait(smem_u32(&bar), parity, &sm.abort, kWaitLimitNs)) return true;
  raise_error(err, MLA_ERR_TIMEOUT);
  sm.abort = 1;
  return false;
}

// Calls f(b, length, group, first tile, end tile) for every pass of this CTA: all groups of query rows over
// a piece of a sequence, then the next piece.
template <typename F>
__device__ __forceinline__ void for_each_pass(const Params& p, const Smem& sm, F f) {
  const int groups = (p.T * p.n_h + kRows - 1) / kRows;
  for_each_piece<kTile>(sm.range, p.lengths, p.B, p.T, p.n_max, [&](int b, int len, int begin, int end) {
    const int step = groups > 1 ? kGroupPiece : end - begin;
    for (int t0 = begin; t0 < end; t0 += step)
      for (int g = 0; g < groups; ++g)
        if (!f(b, len, g, t0, min(t0 + step, end))) return false;
    return true;
  });
}

// One lane's part of the 16 keys that a warp decodes of a tile.  Four lanes cover the 64 bytes of codes that a
// key has in two slabs, so an instruction of 512 bytes looks up eight lines; lanes of the second slab are two
// rows ahead, so that the eight lanes of a store phase hit distinct banks.
struct KeyPart {
  uint4 code[4][2];   // [pair of slabs][keys 0..7, 8..15]
  uint4 scale[2][2];  // all 32 scales of the two keys
  uint4 rope[4];      // eight lanes cover a key's rotary row: keys lane / 8 + 4 i
};
struct KeySource {
  const uint8_t *code, *scale, *rope;  // the lane's first key
  int left, left_rope;                 // keys from that one on that are in the sequence
};
__device__ __forceinline__ int code_row(int lane) { return ((lane >> 2) + (lane & 2)) & 7; }
__device__ __forceinline__ KeySource key_source(const Params& p, int b, int64_t first, int len, int lane) {
  const int64_t t = first + code_row(lane), u = first + (lane >> 3);
  return {p.kv.c4 + b * p.kv.c4_b + t * p.kv.c4_r + 16 * (lane & 3), p.kv.sc + b * p.kv.sc_b + t * p.kv.sc_r,
          static_cast<const uint8_t*>(p.kv.k_r) + 2 * (b * p.kv.kr_b + u * p.kv.kr_r) + 16 * (lane & 7),
          (int)(len - t), (int)(len - u)};
}
// Rows behind the sequence may hold anything, or not exist: they are zeros.  (Plain loads: the kernel before this one may
// still be writing the cache when this one starts, which a load through the non-coherent path does not allow.)
__device__ __forceinline__ uint4 load_row(const uint8_t* src, bool present) {
  return present ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void load_codes(const Params& p, const KeySource& s, int pair, KeyPart& k) {
#pragma unroll
  for (int i = 0; i < 2; ++i) k.code[pair][i] = load_row(s.code + 8 * i * p.kv.c4_r + 64 * pair, 8 * i < s.left);
}
__device__ __forceinline__ void load_scales(const Params& p, const KeySource& s, int h, KeyPart& k) {
#pragma unroll
  for (int i = 0; i < 2; ++i) k.scale[i][h] = load_row(s.scale + 8 * i * p.kv.sc_r + 16 * h, 8 * i < s.left);
}
__device__ __forceinline__ void load_rope(const Params& p, const KeySource& s, KeyPart& k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) k.rope[i] = load_row(s.rope + 8 * i * p.kv.kr_r, 4 * i < s.left_rope);
}

// The sum of exp over a key's columns [0, cols) of the accumulator at `src`; kSelect: without those before `first`,
// whose tokens do not see the key, and those whose -lse at `nl` (log2 units) is -infinity.
template <bool kSelect>
__device__ __forceinline__ float key_sum(uint32_t src, uint32_t nl, int cols, float scale_log2, int first) {
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < cols; c += 32) {
    uint32_t s[32];
    tmem_ld32(src + c, s);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 l4 = ld_shared_v4(nl + 4 * (c + i));
      const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = ex2f_approx(fmaf(__uint_as_float(s[i + e]), scale_log2, l[e]));
        w[e] += kSelect && (c + i + e < first || l[e] == -INFINITY) ? 0.f : x;
      }
    }
  }
  return (w[0] + w[1]) + (w[2] + w[3]);
}

template <bool kFp4>
__global__ void __launch_bounds__(kFp4 ? kThreadsFp4 : kThreadsBf16, 1) weights_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem& sm = *reinterpret_cast<Smem*>(smem + kSmemOff);
  const uint32_t q_addr = smem_u32(smem), ring = smem_u32(smem + kRingOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.T * p.n_h;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), kFp4 ? kDecodeWarps : 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int j = 0; j < kSlabs; ++j) mbar_init(smem_u32(&sm.q_full[j]), 1);
    mbar_init(smem_u32(&sm.q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.s_empty[i]), 4);
    }
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort = sm.never = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  if (warp == 0) tile_range<kTile>(p.lengths, p.B, p.T, p.n_max, blockIdx.x, gridDim.x, p.err, &sm.range);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == kQWarp) {
    // ---------------------------------------------------------------- the query rows of each pass
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      uint32_t pass = 0;
      for_each_pass(p, sm, [&](int b, int, int g, int, int) {
        if (!wait(sm, sm.q_empty, (pass & 1u) ^ 1u, p.err)) return false;
        for (int j = 0; j < kSlabs; ++j) {
          const uint32_t bar = smem_u32(&sm.q_full[j]), dst = q_addr + j * kSlabBytes;
          mbar_arrive_expect_tx(bar, kSlabBytes);
          if (j < kSlabs - 1)
            tma_load_3d(dst, &p.tm_q, bar, 64 * j, kRows * g, b, pol);
          else
            tma_load_3d(dst, &p.tm_qp, bar, 0, kRows * g, b, pol);
        }
        ++pass;
        return true;
      });
      for (int j = 0; j < kSlabs && pass > 0; ++j)
        mbar_wait(smem_u32(&sm.q_full[j]), (pass - 1) & 1u, &sm.never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (!kFp4 && warp == kKeyWarp) {
    // ---------------------------------------------------------------- bf16 keys by TMA
    if (lane == 0) {
      const uint64_t pol = R > kRows ? policy_evict_last() : policy_evict_first();
      uint32_t n = 0;
      for_each_pass(p, sm, [&](int b, int, int, int t0, int t1) {
        for (int t = t0; t < t1; ++t)
          for (int j = 0; j < kSlabs; ++j, ++n) {
            const uint32_t st = n % kStages;
            if (!wait(sm, sm.empty[st], ((n / kStages) & 1u) ^ 1u, p.err)) return false;
            const uint32_t bar = smem_u32(&sm.full[st]), dst = ring + st * kSlabBytes;
            mbar_arrive_expect_tx(bar, kSlabBytes);
            if (j < kSlabs - 1)
              tma_load_3d(dst, &p.tm_ckv, bar, 64 * j, t * kTile, b * p.ckv_z, pol);
            else
              tma_load_3d(dst, &p.tm_kr, bar, 0, t * kTile, b * p.kr_z, pol);
          }
        return true;
      });
      for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k)
        mbar_wait(smem_u32(&sm.full[k % kStages]), (k / kStages) & 1u, &sm.never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- S^T = K Q^T
    if (elect_one()) {
      uint32_t n = 0, tile = 0, pass = 0;
      for_each_pass(p, sm, [&](int, int, int g, int t0, int t1) {
        const int cols = (min(R - kRows * g, kRows) + 31) & ~31;  // zero rows pad to the readers' 32 columns
        const uint32_t idesc = idesc_bf16_f32(kTile, cols, 0, 0);
        for (int t = t0; t < t1; ++t, ++tile) {
          const uint32_t buf = tile & 1u;
          if (!wait(sm, sm.s_empty[buf], ((tile >> 1) & 1u) ^ 1u, p.err)) return false;
          tc_fence_after();
          for (int j = 0; j < kSlabs; ++j, ++n) {
            const uint32_t st = n % kStages;
            if (t == t0 && !wait(sm, sm.q_full[j], pass & 1u, p.err)) return false;
            if (!wait(sm, sm.full[st], (n / kStages) & 1u, p.err)) return false;
            tc_fence_after();
            const uint32_t a = ring + st * kSlabBytes, q = q_addr + j * kSlabBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + buf * kRows, smem_desc(a + 32 * k, 16, 1024, kSwizzle128),
                     smem_desc(q + 32 * k, 16, 1024, kSwizzle128), idesc, j > 0 || k > 0 ? 1u : 0u);
            mma_commit(smem_u32(&sm.empty[st]));
          }
          mma_commit(smem_u32(&sm.s_full[buf]));
        }
        mma_commit(smem_u32(&sm.q_empty));
        ++pass;
        return true;
      });
      mma_commit(smem_u32(&sm.drain));
      mbar_wait(smem_u32(&sm.drain), 0, &sm.never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- exponentials and sums, one key per thread
    // After a failed wait the warp still walks its passes, without the tiles: the four warps meet there.
    uint32_t tile = 0;
    bool dead = false;
    for_each_pass(p, sm, [&](int b, int len, int g, int t0, int t1) {
      const int rows = min(R - kRows * g, kRows), cols = (rows + 31) & ~31;
      named_bar_sync(1, 128);  // the previous pass has read its values
      {
        const int r = threadIdx.x;
        const float lse = r < rows ? p.lse[(int64_t)b * R + kRows * g + r] : -INFINITY;
        sm.neg_lse[r] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
        const bool d = __any_sync(0xffffffffu, r < rows && lse == -INFINITY);
        if (lane == 0) sm.dropped[warp] = d;
      }
      named_bar_sync(1, 128);
      const bool dropped = sm.dropped[0] | sm.dropped[1] | sm.dropped[2] | sm.dropped[3];
      const uint32_t nl = smem_u32(sm.neg_lse);
      for (int t = t0; t < t1 && !dead; ++t, ++tile) {
        const uint32_t buf = tile & 1u, src = tmem + ((uint32_t)(32 * warp) << 16) + buf * kRows;
        const int key = t * kTile + 32 * warp + lane;
        float* out = p.out + b * p.out_b + key;
        float old = 0.f;  // on its way while the scores are made
        if (key < len) {
          if (g > 0)
            old = *out;
          else if (p.acc != nullptr && key < len - p.T)
            old = p.acc[b * p.acc_b + key];
        }
        dead = !__all_sync(0xffffffffu, wait(sm, sm.s_full[buf], (tile >> 1) & 1u, p.err));
        if (dead) break;
        tc_fence_after();
        // some row of this tile is not seen by every token, or a query row gave no weight: select
        const bool select = dropped || (p.T > 1 && (t + 1) * kTile > len - p.T);
        const int first = max(0, key - (len - p.T)) * p.n_h - kRows * g;  // first query row that sees the key
        const float sum = select ? key_sum<true>(src, nl, cols, p.scale_log2, first)
                                 : key_sum<false>(src, nl, cols, p.scale_log2, first);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[buf]));
        if (key < len) *out = fmaf(g > 0 ? 1.f : p.decay, old, sum);
      }
      return true;
    });
  } else if (kFp4 && warp >= kDecodeWarp0) {
    // ---------------------------------------------------------------- 4-bit keys to bf16 slabs
    // (Every producer takes every use of every stage in order: a wait by parity that skipped uses of a stage could
    // take an older phase for the one it needs.)
    // Each load of the next tile follows the last use of its registers, so a tile's time passes before it is
    // needed.
    const int row0 = 16 * (warp - kDecodeWarp0), row = code_row(lane), slab = (lane >> 1) & 1, half = lane & 1;
    const uint32_t dst_codes = ring + (row0 + row) * 128, dst_rope = ring + (row0 + (lane >> 3)) * 128;
    uint32_t n = 0;
    KeyPart k;
    for_each_pass(p, sm, [&](int b, int len, int, int t0, int t1) {
      KeySource s = key_source(p, b, (int64_t)t0 * kTile + row0, len, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) load_codes(p, s, j, k);
      load_scales(p, s, 0, k);
      load_scales(p, s, 1, k);
      load_rope(p, s, k);
      for (int t = t0; t < t1; ++t) {
        s = key_source(p, b, (int64_t)(t + 1) * kTile + row0, t + 1 < t1 ? len : 0, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j, n += 2) {
          bool ok = true;
          for (uint32_t m = n; m < n + 2; ++m) ok &= wait(sm, sm.empty[m % kStages], ((m / kStages) & 1u) ^ 1u, p.err);
          if (!__all_sync(0xffffffffu, ok)) return false;
          const uint32_t dst = dst_codes + (n + slab) % kStages * kSlabBytes;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 q = k.scale[i][j >> 1];
            const uint32_t sw = (j & 1) ? (slab ? q.w : q.z) : (slab ? q.y : q.x);
            const float2 s2 = unpack_f16x2(fp4::scales_to_f16(sw >> (16 * half)));
            const float s0 = s2.x * p.kv.latent_scale, s1 = s2.y * p.kv.latent_scale;
            const uint32_t scale[2] = {pack_bf16x2(s0, s0), pack_bf16x2(s1, s1)};
            const uint32_t words[4] = {k.code[j][i].x, k.code[j][i].y, k.code[j][i].z, k.code[j][i].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t h[4];
              fp4::codes_to_bf16(words[w], h);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = fp4::mul_bf16x2(h[e], scale[w >> 1]);
              st_shared_v4_b32(dst + 1024 * i + (((4 * half + w) ^ row) << 4), h[0], h[1], h[2], h[3]);
            }
          }
          load_codes(p, s, j, k);
          if (j & 1) load_scales(p, s, j >> 1, k);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane < 2) mbar_arrive(smem_u32(&sm.full[(n + lane) % kStages]));
        }
        const uint32_t st = n % kStages;
        if (!__all_sync(0xffffffffu, wait(sm, sm.empty[st], ((n / kStages) & 1u) ^ 1u, p.err))) return false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4_b32(dst_rope + st * kSlabBytes + 512 * i + (((lane & 7) ^ ((lane >> 3) + 4 * (i & 1))) << 4),
                           k.rope[i].x, k.rope[i].y, k.rope[i].z, k.rope[i].w);
        load_rope(p, s, k);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.full[st]));
        ++n;
      }
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

bool make_map(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1_bytes,
              uint64_t s2_bytes) {
  const uint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1_bytes, s2_bytes};
  const uint32_t box[3] = {64, 128, 1};
  return make_tensor_map_bf16(m, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A cache map; sequences that share one cache (batch stride 0) become one.
bool make_cache_map(CUtensorMap* m, const void* base, int width, int n_max, int B, int64_t row, int64_t batch, int* z) {
  *z = B > 1 && batch != 0;
  const uint64_t rb = (uint64_t)row * 2;
  return make_map(m, base, width, n_max, *z ? B : 1, rb, *z ? (uint64_t)batch * 2 : rb * n_max);
}

template <bool kFp4>
cudaError_t launch(const Params& p, int grid, cudaStream_t st) {
  static PerDevice allowed;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(weights_kernel<kFp4>), kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(weights_kernel<kFp4>, dim3(grid), dim3(kFp4 ? kThreadsFp4 : kThreadsBf16), kSmemBytes, st, p);
}

}  // namespace weights_tc

cudaError_t weights_tc_launch(const WeightsArgs& a, cudaStream_t st) {
  using namespace weights_tc;
  const bool fp4 = a.kv.c4 != nullptr;
  const int R = a.T * a.n_h;
  Params p{};
  if (!make_map(&p.tm_q, a.q_tilde, kDC, R, a.B, (uint64_t)a.ldqt * 2, (uint64_t)a.ldqt * 2 * R) ||
      !make_map(&p.tm_qp, a.q_pe, kDR, R, a.B, (uint64_t)a.ldqp * 2, (uint64_t)a.ldqp * 2 * R))
    return cudaErrorInvalidValue;
  if (!fp4 && (!make_cache_map(&p.tm_ckv, a.kv.c_kv, kDC, a.n_max, a.B, a.kv.ckv_r, a.kv.ckv_b, &p.ckv_z) ||
               !make_cache_map(&p.tm_kr, a.kv.k_r, kDR, a.n_max, a.B, a.kv.kr_r, a.kv.kr_b, &p.kr_z)))
    return cudaErrorInvalidValue;
  p.kv = a.kv;
  p.lengths = a.lengths;
  p.B = a.B; p.T = a.T; p.n_h = a.n_h; p.n_max = a.n_max;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.lse = a.lse; p.acc = a.acc; p.acc_b = a.acc_b; p.decay = a.decay;
  p.out = a.out; p.out_b = a.out_b; p.err = a.err;
  const int sms = sm_count();
  const int64_t tiles = (int64_t)a.B * ((a.n_max + kTile - 1) / kTile);
  const int grid = (int)(tiles < sms ? tiles : sms);
  return fp4 ? launch<true>(p, grid, st) : launch<false>(p, grid, st);
}

}  // namespace mla
