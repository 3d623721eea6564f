// Absorbed decode over the 4-bit latent cache on tcgen05 tensor cores (sm_100a):
//   z[r, t] = scale (q~_r . c_t + q_pe,r . k^R_t),  ctx_r = sum_t softmax(z)_t c_t,  lse_r = log sum_t exp z
// for the R = T n_h query rows r of a sequence (row r belongs to new token r / n_h and sees the rows
// t <= L - T + r / n_h), c_t = code * scale decoded on chip.
//
// Bound: the tensor pipe.  A cached row costs 2 R (2 d_c + d_r) operations against 416 bytes: at R = 128
// 669 a byte, far right of the GPU's ridge.
//
// Why this split.  The fp32 context of 128 rows x 512 features fills TMEM, so no SM can hold it beside
// scores.  A CTA therefore keeps one half of the latent features of the context (256 columns) and computes
// all 576 features of the scores itself: the score work is done twice, 27.3 instead of 17.8 MFLOP per 64
// rows and two CTAs, and in return nothing is exchanged, no CTA waits for another one and the halves need
// not even run at the same time.  (Exchanging partial scores between two CTAs through distributed shared
// memory holds the bf16 decode at one third of the tensor peak.)
//
// * Operands are fp16: code * scale has at most six significant bits and lies in 2^-10 .. 2688, so the cache
//   is exact; a query row is scaled by a power of two that puts its largest element into [2^14, 2^15), so that
//   bf16 elements are exact down to 2^-31 of it, and the power goes into the row's softmax scale.  The rotary
//   part stays in bf16 (separate MMAs into the same accumulator).  Probabilities are rounded to fp16.
// * Tiles of 64 keys.  TMEM: context 256 columns, scores 64, query features [0, 384) 192 columns as the A
//   operand; the other query features and the probabilities are A operands in shared memory.
// * Nine warps decode: lane pairs own a key, 16-byte loads of codes two tiles ahead in registers, cvt to fp16,
//   one product with the block's scale, stores in the 128-byte-swizzled layout.  The four slabs of the
//   CTA's own half serve the scores (K-major) and the values (MN-major) and stay until the values are used: three
//   buffers.  The other half's slabs and the rotary slab are free once the scores are done: a ring of eight.
// * MMA order S(t + 1), O(t), S(t + 2), ...: the softmax of tile t runs under S(t + 1), and the tensor pipe
//   works on O(t - 1) while S(t) is read from TMEM.
// * Four softmax warps, one query row per thread; base-2 exponentials, their reference moved (and the context
//   rescaled in TMEM) only when the running maximum grows by more than 8.
// * Work: chunks of single sequences when each can have CTAs of its own and the chunks come out balanced, else
//   equal ranges of all tiles.  A sequence that is cut leaves fp32 partials and a second kernel joins them in a
//   fixed order.
// * Every wait is bounded; on expiry the kernel records MLA_ERR_TIMEOUT and all warps run out their barriers.
#include <math.h>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"
#include "tma_host.h"

namespace mla {
namespace decode_fp4 {

using namespace sm100;

constexpr int kDC = 512, kDR = 64;
constexpr int kTile = 64;                        // keys per tile
constexpr int kRows = 128;                       // query rows per group: the rows of every MMA
constexpr int kSlabBytes = kTile * 128;          // 64 keys of 64 features
constexpr int kKvStages = 3, kKvBytes = 4 * kSlabBytes;
constexpr int kKSlots = 8, kKPerTile = 5;        // rotary slab and the other half's four slabs
constexpr int kQSlabBytes = kRows * 128;         // 128 query rows of 64 features
constexpr int kQTmemSlabs = 6;                   // query slabs in TMEM; the other two and the rotary one in shared memory
constexpr int kKOff = kKvStages * kKvBytes;
constexpr int kQOff = kKOff + kKSlots * kSlabBytes;
constexpr int kPOff = kQOff + 3 * kQSlabBytes;
constexpr int kSmemOff = kPOff + kRows * 128;
static_assert(kQTmemSlabs * kQSlabBytes <= kQOff, "the query is staged in the key buffers");
static_assert(kRows * 256 * 4 <= kQOff, "the partial context is staged in the key buffers");
constexpr int kMmaWarp = 4, kKvWarp0 = 5, kKWarp0 = 9, kRopeWarp = 13;
constexpr int kPrefetchWarp = 14;
constexpr int kThreads = 32 * 15;
constexpr uint32_t kTmemCols = 512, kColO = 0, kColS = 256, kColQ = 320;
// Probabilities are 2^(z - ref): ref is set kRaise below the largest score so far (log2 units) and moved up
// only when a score passes it by kRescale.  So they reach 2^15 at most (fp16 ends at 2^16), the sum is at
// least 2^kRaise, and a probability that fp16's subnormals round (2^-25) is off by 2^-32 of the sum.
constexpr float kRaise = 7.f, kRescale = 15.f;
constexpr int kPrefetch = 4;                     // tiles that L2 is ahead of the decode warps
constexpr int kPlanRegs = 3;                     // items per lane that the chunk search holds (more than the pairs)
constexpr int kSwitchTiles = 5;                  // what a second piece costs a CTA, in tiles
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Params {
  CUtensorMap tm_q;   // (d_c, R, B) query rows, box (64, 128, 1), 128-byte swizzle: rows past R read as zeros
  CUtensorMap tm_qp;  // (d_r, R, B), same box
  CacheView kv;
  const int32_t* lengths;
  int B, T, n_h, n_max, R, groups, pairs;
  float scale_log2;
  __nv_bfloat16* ctx;
  float* lse;
  int4* table;    // [B * groups] partials of an item: first slot, first CTA pair, number
  float2* ws_ml;  // [2 pairs slots][2 halves][128] (reference in log2 units, sum)
  float* ws_o;    // [slots][2 halves][min(R, 128)][256], 16-byte chunk j of row r at (j + r) % 64
  int32_t* err;
};

// An item is a group of up to 128 query rows of one sequence.  Keys its last row sees, 0 for a bad length.
__device__ __forceinline__ int item_keys(const Params& p, int i) {
  const int len = p.lengths[i / p.groups];
  if (len < p.T || len > p.n_max) return 0;
  const int last = min(p.R, kRows * (i % p.groups + 1)) - 1;
  return len - p.T + last / p.n_h + 1;
}
__device__ __forceinline__ int item_tiles(const Params& p, int i) { return (item_keys(p, i) + kTile - 1) / kTile; }

// A CTA pair's share: pieces of items.
struct Plan {
  long long lo, hi, tb, total;  // tiles [lo, hi) of all items' tiles laid end to end; first tile of `item`
  int item, chunk, c0, n;       // chunk > 0: one piece, the (pair - c0)-th of item's n chunks
  int nc;                       // pairs that have work
};
struct Piece {
  int item, begin, end, tiles;  // item < 0: none left
  int slot, c0, n;              // where its partial goes; first pair and number of the item's pieces
};

struct Smem {
  uint64_t kv_full[kKvStages], kv_empty[kKvStages], k_full[kKSlots], k_empty[kKSlots];
  uint64_t q_full, s_full, s_empty, p_full, pv_done, drain;
  alignas(16) float row_scale[kRows];  // softmax scale of a query row, log2 units
  Plan plan;
  Piece piece;
  float row_max[2][kRows];  // largest element of a query row, each half of its slabs
  uint32_t tmem_base;
  int abort, never, progress;
};
constexpr int kSmemBytes = kSmemOff + (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory above 227 KB");

__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

// Bounded wait that records its own expiry; what follows a first failed try is one shared function, since the
// roles' loops together have to fit the instruction cache.
__device__ __noinline__ bool wait_more(Smem& sm, uint32_t bar, uint32_t parity, int32_t* err) {
  if (mbar_wait(bar, parity, &sm.abort, kWaitLimitNs)) return true;
  raise_error(err, MLA_ERR_TIMEOUT);
  sm.abort = 1;
  return false;
}
__device__ __forceinline__ bool wait(Smem& sm, uint64_t& bar, uint32_t parity, int32_t* err) {
  return mbar_try_wait(smem_u32(&bar), parity) || wait_more(sm, smem_u32(&bar), parity, err);
}
// All lanes wait; the warp goes on only if all of them saw the phase complete.
__device__ __forceinline__ bool wait_warp(Smem& sm, uint64_t& bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, wait(sm, bar, parity, err));
}

// total c / nc, in 32 bits where they hold the product.
__device__ __forceinline__ long long share(long long total, int c, int nc) {
  return total < (1 << 22) ? (long long)((uint32_t)total * (uint32_t)c / (uint32_t)nc) : total * c / nc;
}
// The pair that holds tile t: ((t + 1) nc - 1) / total.
__device__ __forceinline__ int holder(long long t, long long total, int nc) {
  return total < (1 << 22) ? (int)(((uint32_t)(t + 1) * (uint32_t)nc - 1u) / (uint32_t)total)
                           : (int)(((t + 1) * nc - 1) / total);
}

// One warp: the share of pair c.
__device__ __noinline__ void make_plan(const Params& p, int c, Plan* out) {
  const int lane = threadIdx.x & 31, items = p.B * p.groups;
  long long total = 0;
  int longest = 0, nonempty = 0, nt[kPlanRegs];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kPlanRegs; ++k) nt[k] = 0;
#pragma unroll 1
  for (int i0 = 0, k = 0; i0 < items; i0 += 32, ++k) {
    const int n = i0 + lane < items ? item_tiles(p, i0 + lane) : 0;
    bad |= i0 + lane < items && n == 0;
#pragma unroll
    for (int j = 0; j < kPlanRegs; ++j)
      if (j == k) nt[j] = n;
    total += n;
    longest = max(longest, n);
    nonempty += n > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  longest = __reduce_max_sync(0xffffffffu, longest);
  nonempty = __reduce_add_sync(0xffffffffu, nonempty);
  if (__any_sync(0xffffffffu, bad) && c == 0 && lane == 0) raise_error(p.err, MLA_ERR_LENGTH);
  Plan r;
  r.total = total;
  r.nc = (int)(total < p.pairs ? total : p.pairs);
  r.lo = r.hi = r.tb = 0;
  r.item = items;
  r.chunk = r.c0 = r.n = 0;
  if (c >= r.nc) {
    if (lane == 0) *out = r;
    return;
  }
  // the smallest chunk whose chunks fit the pairs, if that is little above the even share
  const int even = (int)share(total + r.nc - 1, 1, r.nc);
  if (items <= 32 * kPlanRegs && nonempty <= r.nc && longest < (1 << 22)) {
#pragma unroll 1
    for (int size = even; size <= even + kSwitchTiles; ++size) {
      const float inv = 1.f / (float)size;
      int n = 0;
#pragma unroll
      for (int k = 0; k < kPlanRegs; ++k) {
        // ceil(nt / size): the float quotient is within one of the exact one
        int q = (int)((float)nt[k] * inv);
        q += (q * size < nt[k]) + ((q + 1) * size < nt[k]) - ((q - 1) * size >= nt[k] && q > 0);
        n += q;
      }
      if ((int)__reduce_add_sync(0xffffffffu, n) <= r.nc) {
        r.chunk = size;
        break;
      }
    }
  }
  if (r.chunk == 0) {
    r.lo = share(total, c, r.nc);
    r.hi = share(total, c + 1, r.nc);
  }
  long long base = 0;  // chunks or tiles before item i0
  const long long at = r.chunk > 0 ? c : r.lo;
#pragma unroll 1
  for (int i0 = 0; i0 < items; i0 += 32) {
    const int tiles = i0 + lane < items ? item_tiles(p, i0 + lane) : 0;
    const int n = r.chunk > 0 ? (tiles + r.chunk - 1) / r.chunk : tiles;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + sum > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      r.item = i0 + l;
      r.tb = base + __shfl_sync(0xffffffffu, sum - n, l);
      r.n = __shfl_sync(0xffffffffu, n, l);
      break;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  r.c0 = (int)r.tb;  // chunk plan: the item's first chunk is its first pair's
  if (lane == 0) *out = r;
}

// One thread: the next piece of pair c.
__device__ __noinline__ void next_piece(const Params& p, int c, Plan& s, Piece* out) {
  Piece r;
  r.item = -1;
  r.begin = r.end = r.tiles = r.slot = r.c0 = r.n = 0;
  const int items = p.B * p.groups;
  if (s.chunk > 0) {
    if (s.item < items) {
      r.item = s.item;
      r.tiles = item_tiles(p, s.item);
      r.begin = (c - s.c0) * s.chunk;
      r.end = min(r.begin + s.chunk, r.tiles);
      r.slot = 2 * c;
      r.c0 = s.c0;
      r.n = s.n;
      s.item = items;
    }
    *out = r;
    return;
  }
  for (; s.item < items && s.lo < s.hi; ++s.item) {
    const int nt = item_tiles(p, s.item);
    if (s.tb + nt > s.lo) {
      const long long end = s.hi < s.tb + nt ? s.hi : s.tb + nt;
      r.item = s.item;
      r.tiles = nt;
      r.begin = (int)(s.lo - s.tb);
      r.end = (int)(end - s.tb);
      r.c0 = holder(s.tb, s.total, s.nc);
      r.n = holder(s.tb + nt - 1, s.total, s.nc) - r.c0 + 1;
      r.slot = 2 * c + (share(s.total, c, s.nc) < s.tb ? 1 : 0);  // a pair's first and its later pieces
      s.lo = end;
      s.tb += nt;
      ++s.item;
      *out = r;
      return;
    }
    s.tb += nt;
  }
  *out = r;
}

// A decode warp's lane: 32 features of one 64-feature slab for four keys of a tile (lane / 2 + 16 i).
struct Part {
  uint4 code[4];
  uint32_t scale[4];
};
struct PartSource {
  const uint8_t* code;
  const uint8_t* scale;
  int64_t code16, scale16;  // 16 rows on
};
__device__ __forceinline__ PartSource part_source(const Params& p, int b, int tile, int slab, int lane) {
  const int64_t t = (int64_t)tile * kTile + (lane >> 1);
  return {p.kv.c4 + b * p.kv.c4_b + t * p.kv.c4_r + 32 * slab + 16 * (lane & 1),
          p.kv.sc + b * p.kv.sc_b + t * p.kv.sc_r + 4 * slab + 2 * (lane & 1), 16 * p.kv.c4_r, 16 * p.kv.sc_r};
}
// Loads the source's tile and moves on to the next one; `left` keys from the lane's first one are in the sequence.
__device__ __forceinline__ void load_part(PartSource& s, int left, Part& k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k.code[i] = make_uint4(0u, 0u, 0u, 0u);
    k.scale[i] = 0u;
    if (16 * i < left) {  // rows behind the sequence may hold anything, or not exist
      k.code[i] = __ldg(reinterpret_cast<const uint4*>(s.code));
      k.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(s.scale));
    }
    s.code += s.code16;
    s.scale += s.scale16;
  }
}
__device__ __forceinline__ void store_part(const Part& k, uint32_t dst, int lane) {
  const int half = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * i + (lane >> 1);
    const uint32_t s2 = fp4::scales_to_f16(k.scale[i]);
    const uint32_t s[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
    const uint32_t words[4] = {k.code[i].x, k.code[i].y, k.code[i].z, k.code[i].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t h[4];
      fp4::codes_to_f16(words[w], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = fp4::mul_f16x2(h[e], s[w >> 1]);
      st_shared_v4_b32(dst + row * 128 + (((4 * half + w) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}
// The rotary warp's lane: half of the rotary row of the same four keys.
__device__ __forceinline__ void load_rope(const uint8_t*& src, int64_t rows16, int left, uint4 (&k)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      k[4 * i + j] = 16 * i < left ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0u, 0u, 0u, 0u);
    src += rows16;
  }
}
__device__ __forceinline__ void store_rope(const uint4 (&k)[16], uint32_t dst, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * i + (lane >> 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4_b32(dst + row * 128 + (((4 * (lane & 1) + j) ^ (row & 7)) << 4), k[4 * i + j].x, k[4 * i + j].y,
                       k[4 * i + j].z, k[4 * i + j].w);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One thread: the item's query rows as they are (bf16, rows past R as zeros): the six slabs of TMEM over the
// value buffers, the other two and the rotary one to their place.  Slabs count from the CTA's own half.
__device__ __noinline__ void fetch_query(const Params& p, Smem& sm, uint32_t base, int b, int g, int hf) {
  fence_proxy_async_smem();  // the buffers were read and written by threads before
  const uint64_t pol = policy_evict_last();
  const uint32_t bar = smem_u32(&sm.q_full);
  mbar_arrive_expect_tx(bar, 9 * kQSlabBytes);
#pragma unroll 1
  for (int j = 0; j < 8; ++j)
    tma_load_3d(base + (j < kQTmemSlabs ? 0 : kQOff - kQTmemSlabs * kQSlabBytes) + j * kQSlabBytes, &p.tm_q, bar,
                64 * (j ^ (4 * hf)), kRows * g, b, pol);
  tma_load_3d(base + kQOff + 2 * kQSlabBytes, &p.tm_qp, bar, 0, kRows * g, b, pol);
}

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The query rows in place, by the softmax warps (h = 0: the own half's slabs) and the four warps that decode the
// other half (h = 1: its slabs and the rotary one), one row per thread of each: the row's power of two, its latent
// part to fp16 (in TMEM, or where it is), its rotary part scaled where it is.
__device__ __noinline__ bool place_query(const Params& p, Smem& sm, uint32_t base, uint32_t tmem, int h, uint32_t parity) {
  const int r = 32 * ((threadIdx.x >> 5) & 3) + (threadIdx.x & 31);  // the row is the warp's TMEM lane
  const bool ok = wait_warp(sm, sm.q_full, parity, p.err);
  auto chunk = [&](int j, int c) {  // address of 16-byte chunk c of slab j (8: rotary)
    return base + (j < kQTmemSlabs ? 0 : kQOff - kQTmemSlabs * kQSlabBytes) + j * kQSlabBytes + r * 128 + ((c ^ (r & 7)) << 4);
  };
  const float ls = p.kv.latent_scale;
  float m = 0.f;
  uint32_t big = 0u;
#pragma unroll 1
  for (int j = 4 * h; j < 4 + 5 * h; ++j) {
    if (j == 8) {
      m = fmaxf(bf16_lo(big), bf16_hi(big)) * ls;
      big = 0u;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = ld_shared_v4_b32(chunk(j, c));
      big = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(big, u.x), u.y), u.z), u.w);
    }
  }
  m = fmaxf(m, fmaxf(bf16_lo(big), bf16_hi(big)) * (h ? 1.f : ls));
  sm.row_max[h][r] = m;
  named_bar_sync(1, 256);
  m = fmaxf(m, sm.row_max[1 - h][r]);
  // 2^e that puts the row's largest element into [2^14, 2^15)
  const int e = m > 0.f ? max(-126, min(126, 14 + 127 - (int)(__float_as_uint(m) >> 23))) : 0;
  const float mul = __uint_as_float((uint32_t)(127 + e) << 23);
  if (h == 0) sm.row_scale[r] = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 1.2e-38f);
#pragma unroll 1
  for (int j = 4 * h; j < 4 + 5 * h; ++j) {
    const float a = j < 8 ? ls : 1.f;
    uint32_t v[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = ld_shared_v4_b32(chunk(j, c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = bf16_lo(w[i]) * a * mul, hi = bf16_hi(w[i]) * a * mul;
        v[4 * c + i] = j < 8 ? pack_f16x2_ieee(lo, hi) : pack_bf16x2(lo, hi);
      }
    }
    if (j < kQTmemSlabs) {
      tmem_st32(tmem + ((uint32_t)(r & 96) << 16) + kColQ + 32 * j, v);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_v4_b32(chunk(j, c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
  }
  tmem_st_wait();
  tc_fence_before();
  fence_proxy_async_smem();
  return ok;
}

// What a role needs to know of the piece at hand.  The roles are functions of their own so that each has the
// registers to itself: inlined together they spill.
struct Work {
  uint32_t base, tmem;   // shared memory, TMEM
  uint32_t it0, n;       // tiles of the earlier pieces, tiles of this one
  int begin, b, g, len, hf;
  int slot, c0, pieces;  // as in Piece
};

// A 128-byte-swizzled shared-memory descriptor whose address is at + 32 k: the low word counts 16 bytes.
__device__ __forceinline__ uint64_t step_desc(uint32_t at, int k, uint32_t lbo_bytes = 16) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (kSwizzle128 << 29);
  return ((uint64_t)hi << 32) | ((lbo_bytes >> 4) << 16 | ((at >> 4) + 2 * k));
}

// One 64-feature slab of the scores, the query slab in TMEM columns q or in shared memory at q.
__device__ __forceinline__ void slab_ts(uint32_t s, uint32_t q, uint32_t keys, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    mma_ts(s, q + 8 * k, step_desc(keys, k), idesc_f16_f32(kRows, kTile, 0, 0), first && k == 0 ? 0u : 1u);
}
__device__ __forceinline__ void slab_ss(uint32_t s, uint32_t q, uint32_t keys, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_ss(s, step_desc(q, k), step_desc(keys, k), idesc, 1u);
}

// One warp: the MMAs of a piece, issued by one thread: S(t), then O(t - 1).  Query slabs are counted from the
// CTA's own half: 0..3 its half, 4..7 the other one; 0..5 are in TMEM.
__device__ __noinline__ bool mma_role(const Params& p, uint32_t it0, uint32_t n) {
  uint8_t* smem = shared_base();
  Smem& sm = *reinterpret_cast<Smem*>(smem + kSmemOff);
  const uint32_t base = smem_u32(smem), tmem = sm.tmem_base, tS = tmem + kColS, tQ = tmem + kColQ;
  bool ok = true;
  if (elect_one()) {
#pragma unroll 1
    for (uint32_t t = 0; t <= n; ++t) {
      if (t < n) {
        // All waits first: they run under O(t - 2), and the issue below then stays ahead of the tensor pipe.
        const uint32_t it = it0 + t, st = it % kKvStages, kv = base + st * kKvBytes, k = kKPerTile * it;
        ok = wait(sm, sm.s_empty, (it & 1u) ^ 1u, p.err) && wait(sm, sm.kv_full[st], (it / kKvStages) & 1u, p.err);
#pragma unroll 1
        for (uint32_t j = 0; j < kKPerTile && ok; ++j)
          ok = wait(sm, sm.k_full[(k + j) % kKSlots], ((k + j) / kKSlots) & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) slab_ts(tS, tQ + 32 * j, kv + j * kSlabBytes, j == 0);
#pragma unroll
        for (int j = 0; j < kKPerTile; ++j) {
          const uint32_t slot = (k + j) % kKSlots, keys = base + kKOff + slot * kSlabBytes;
          if (j == 0)
            slab_ss(tS, base + kQOff + 2 * kQSlabBytes, keys, idesc_bf16_f32(kRows, kTile, 0, 0));
          else if (j < 3)
            slab_ts(tS, tQ + 96 + 32 * j, keys, false);
          else
            slab_ss(tS, base + kQOff + (j - 3) * kQSlabBytes, keys, idesc_f16_f32(kRows, kTile, 0, 0));
          mma_commit(smem_u32(&sm.k_empty[slot]));
        }
        mma_commit(smem_u32(&sm.s_full));
      }
      if (t > 0) {
        const uint32_t it = it0 + t - 1, st = it % kKvStages, kv = base + st * kKvBytes;
        ok = wait(sm, sm.p_full, it & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tmem + kColO, step_desc(base + kPOff, k), step_desc(kv + 2048 * k, 0, kSlabBytes),
                 idesc_f16_f32(kRows, 256, 0, 1), t > 1 || k > 0 ? 1u : 0u);
        mma_commit(smem_u32(&sm.kv_empty[st]));
        mma_commit(smem_u32(&sm.pv_done));
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Four warps, one query row per thread: probabilities, and the piece's result.
__device__ __noinline__ bool softmax_role(const Params& p, Smem& sm, Work w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x;
  const uint32_t base = w.base, n = w.n, it0 = w.it0;
  const int b = w.b, g = w.g, len = w.len, hf = w.hf, rows = min(p.R - kRows * g, kRows);
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t tS = w.tmem + lanes + kColS, tO = w.tmem + lanes + kColO;
  const uint32_t p_row = base + kPOff + r * 128;
  const float sl = sm.row_scale[r];
  // keys that the row, and the group's first row, see
  const int limit = len - p.T + (kRows * g + min(r, rows - 1)) / p.n_h + 1;
  const int all_see = len - p.T + (kRows * g) / p.n_h + 1;
  float ref = -INFINITY, l = 0.f;
  bool ok = true;
#pragma unroll 1
  for (uint32_t t = 0; t < n && ok; ++t) {
    const uint32_t it = it0 + t;
    const int k0 = (w.begin + (int)t) * kTile;
    ok = wait_warp(sm, sm.s_full, it & 1u, p.err);
    if (!ok) break;
    tc_fence_after();
    uint32_t s[2][32];
    tmem_ld32(tS, s[0]);
    tmem_ld32(tS + 32, s[1]);
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty));
    if (k0 + kTile > all_see) {
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (k0 + i >= limit) s[i >> 5][i & 31] = 0xff800000u;  // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i >> 5][i & 31]));
    const float z = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
    float f = 1.f;
    const bool raise = z > ref + kRescale;  // ref = -inf: any finite maximum
    if (raise) {
      f = ex2f_approx(ref - (z - kRaise));
      l *= f;
      ref = z - kRaise;
    }
    const float neg = ref == -INFINITY ? 0.f : -ref;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    auto half = [&](int k) {  // probabilities of 32 keys, as fp16 pairs in the first 16 words
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float a = ex2f_approx(fmaf(__uint_as_float(s[k][i]), sl, neg));
        const float c = ex2f_approx(fmaf(__uint_as_float(s[k][i + 1]), sl, neg));
        sum[i & 2] += a;
        sum[(i & 2) + 1] += c;
        s[k][i / 2] = pack_f16x2_ieee(a, c);
      }
    };
    auto store = [&](int k) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4_b32(p_row + (((4 * k + c) ^ (r & 7)) << 4), s[k][4 * c], s[k][4 * c + 1], s[k][4 * c + 2],
                         s[k][4 * c + 3]);
    };
    half(0);
    if (t > 0) {  // the last tile's probabilities are used up, its context complete
      ok = wait_warp(sm, sm.pv_done, (it - 1) & 1u, p.err);
      if (!ok) break;
      if (__any_sync(0xffffffffu, raise)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(tO + c, o);
        }
        tmem_st_wait();
        tc_fence_before();
      }
    }
    store(0);
    half(1);
    store(1);
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.p_full));
  }
  if (ok) ok = wait_warp(sm, sm.pv_done, (it0 + n - 1) & 1u, p.err);
  if (ok) {
    // -------------------------------------------------------------- the piece's result
    // through the idle key buffers, 16-byte chunks rotated by the row so that neither the row-wise
    // writes nor the copies out conflict
    tc_fence_after();
    const uint32_t out_row = (uint32_t)b * p.R + kRows * g;  // first query row of the group
    if (w.pieces == 1) {
      const float inv = (l == 0.f ? 0.f : 1.f / l) * p.kv.latent_scale;
      const uint32_t dst = base + r * 512;
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
          st_shared_v4_b32(dst + (((c / 8 + i + r) & 31) << 4), v[0], v[1], v[2], v[3]);
        }
      }
      __syncwarp();
      for (int k = 32 * warp; k < min(32 * warp + 32, rows); ++k) {
        const uint4 v = ld_shared_v4_b32(base + k * 512 + (((lane + k) & 31) << 4));
        reinterpret_cast<uint4*>(p.ctx + (int64_t)(out_row + k) * kDC + 256 * hf)[lane] = v;
      }
      if (hf == 0 && r < rows && p.lse != nullptr)
        p.lse[out_row + r] = l == 0.f ? -INFINITY : ref * kLn2 + logf(l);
    } else {
      const uint32_t dst = base + r * 1024;
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4_b32(dst + (((c / 4 + i + r) & 63) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      const int64_t part = 2 * (int64_t)w.slot + hf;
      const int mine = min(32, rows - 32 * warp);
      if (lane == 0 && mine > 0) {
        bulk_store_s2g(p.ws_o + (part * min(p.R, kRows) + 32 * warp) * 256, base + 32 * warp * 1024, mine * 1024);
        bulk_group_commit();
        bulk_group_wait_read_all();
      }
      if (r < rows) p.ws_ml[part * kRows + r] = make_float2(ref, l);
    }
    if (threadIdx.x == 0 && hf == 0 && w.begin == 0) p.table[w.b * p.groups + w.g] = make_int4(w.slot, w.c0, w.pieces, 0);
    tc_fence_before();
    fence_proxy_async_smem();
  }
  return ok;
}

// One warp: its latent slab of every tile, loaded one tile ahead (from L2: the rotary warp prefetches).
__device__ __noinline__ bool latent_role(const Params& p, Smem& sm, Work w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool own = warp < kKWarp0;  // a slab of this CTA's half
  const int j = own ? warp - kKvWarp0 : warp - kKWarp0;
  PartSource src = part_source(p, w.b, w.begin, 4 * (own ? w.hf : 1 - w.hf) + j, lane);
  int left = w.len - w.begin * kTile - (lane >> 1);
  Part k;
  load_part(src, left, k);
#pragma unroll 1
  for (uint32_t t = 0; t < w.n; ++t) {
    const uint32_t it = w.it0 + t, q = kKPerTile * it + 1 + j;
    const uint32_t slot = own ? it % kKvStages : q % kKSlots, use = own ? it / kKvStages : q / kKSlots;
    if (!wait_warp(sm, own ? sm.kv_empty[slot] : sm.k_empty[slot], (use & 1u) ^ 1u, p.err)) return false;
    store_part(k, w.base + (own ? slot * kKvBytes + j * kSlabBytes : kKOff + slot * kSlabBytes), lane);
    if (lane == 0) mbar_arrive(smem_u32(own ? &sm.kv_full[slot] : &sm.k_full[slot]));
    if (warp == kKvWarp0 && lane == 0) *const_cast<volatile int*>(&sm.progress) = (int)t;
    left -= kTile;
    load_part(src, left, k);
  }
  return true;
}

__device__ __forceinline__ void prefetch_l2(const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); }
// One warp: the cached rows of a tile into L2.
__device__ __forceinline__ void prefetch_tile(const Params& p, int b, int tile, int len, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = (int64_t)tile * kTile + 32 * i + lane;
    if (t >= len) return;
    const uint8_t* c = p.kv.c4 + b * p.kv.c4_b + t * p.kv.c4_r;
    prefetch_l2(c);
    prefetch_l2(c + 128);
    prefetch_l2(p.kv.sc + b * p.kv.sc_b + t * p.kv.sc_r);
    prefetch_l2(static_cast<const __nv_bfloat16*>(p.kv.k_r) + b * p.kv.kr_b + t * p.kv.kr_r);
  }
}

// One warp: the tiles' way into L2, kPrefetch tiles ahead of the decode warps.
__device__ __noinline__ void prefetch_role(const Params& p, Smem& sm, Work w) {
  const int lane = threadIdx.x & 31;
  const volatile int* progress = &sm.progress;
  const volatile int* abort = &sm.abort;
#pragma unroll 1
  for (int t = kPrefetch; t < (int)w.n; ++t) {
    while (*progress + kPrefetch < t && !*abort) __nanosleep(100);  // the decode warps' waits are bounded
    prefetch_tile(p, w.b, w.begin + t, w.len, lane);
  }
}

// One warp: the rotary slab of every tile.
__device__ __noinline__ bool rope_role(const Params& p, Smem& sm, Work w) {
  const int lane = threadIdx.x & 31;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(static_cast<const __nv_bfloat16*>(p.kv.k_r) + w.b * p.kv.kr_b +
                                                        ((int64_t)w.begin * kTile + (lane >> 1)) * p.kv.kr_r) + 64 * (lane & 1);
  int left = w.len - w.begin * kTile - (lane >> 1);
  uint4 k[16];
  load_rope(src, 32 * p.kv.kr_r, left, k);
#pragma unroll 1
  for (uint32_t t = 0; t < w.n; ++t) {
    const uint32_t q = kKPerTile * (w.it0 + t), slot = q % kKSlots;
    if (!wait_warp(sm, sm.k_empty[slot], ((q / kKSlots) & 1u) ^ 1u, p.err)) return false;
    store_rope(k, w.base + kKOff + slot * kSlabBytes, lane);
    if (lane == 0) mbar_arrive(smem_u32(&sm.k_full[slot]));
    left -= kTile;
    load_rope(src, 32 * p.kv.kr_r, left, k);
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Params p) {
  uint8_t* smem = shared_base();
  Smem& sm = *reinterpret_cast<Smem*>(smem + kSmemOff);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, hf = blockIdx.x & 1;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(smem_u32(&sm.kv_full[s]), 4);
      mbar_init(smem_u32(&sm.kv_empty[s]), 1);
    }
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(smem_u32(&sm.k_full[s]), 1);
      mbar_init(smem_u32(&sm.k_empty[s]), 1);
    }
    mbar_init(smem_u32(&sm.q_full), 1);
    mbar_init(smem_u32(&sm.s_full), 1);
    mbar_init(smem_u32(&sm.s_empty), 4);
    mbar_init(smem_u32(&sm.p_full), 4);
    mbar_init(smem_u32(&sm.pv_done), 1);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort = sm.never = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  if (warp == 0) {
    make_plan(p, pair, &sm.plan);
    __syncwarp();
    if (lane == 0) next_piece(p, pair, sm.plan, &sm.piece);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // it0: tiles of the earlier pieces.  All warps take every barrier of every piece, also after a failed wait.
  uint32_t it0 = 0, pieces = 0;
  bool dead = false;
  while (true) {
    if (sm.piece.item < 0) break;
    Work w;
    w.base = base;
    w.tmem = tmem;
    w.it0 = it0;
    w.begin = sm.piece.begin;
    w.n = (uint32_t)(sm.piece.end - w.begin);
    w.b = sm.piece.item / p.groups;
    w.g = sm.piece.item % p.groups;
    w.len = p.lengths[w.b];
    w.hf = hf;
    w.slot = sm.piece.slot;
    w.c0 = sm.piece.c0;
    w.pieces = sm.piece.n;
    if (threadIdx.x == 0) {
      sm.progress = 0;
      fetch_query(p, sm, base, w.b, w.g, hf);
    }
    if (warp == kPrefetchWarp)
      for (int t = 0; t < kPrefetch && t < (int)w.n; ++t) prefetch_tile(p, w.b, w.begin + t, w.len, lane);
    __syncwarp();
    // (all eight warps come here in every piece: they meet inside)
    if (warp < 4 || (warp >= kKWarp0 && warp < kRopeWarp))
      dead |= !place_query(p, sm, base, tmem, warp >= kKWarp0 ? 1 : 0, pieces & 1u);
    ++pieces;
    __syncthreads();
    tc_fence_after();
    if (sm.abort) dead = true;
    if (!dead) {
      bool ok = true;
      if (warp < 4)
        ok = softmax_role(p, sm, w);
      else if (warp > kMmaWarp)
        ok = warp < kRopeWarp ? latent_role(p, sm, w) : warp > kRopeWarp || rope_role(p, sm, w);
      else
        ok = mma_role(p, it0, w.n);
      if (warp == kPrefetchWarp) prefetch_role(p, sm, w);
      dead = !ok;
    }
    __syncwarp();
    it0 += w.n;
    if (threadIdx.x == 0) next_piece(p, pair, sm.plan, &sm.piece);
    __syncthreads();
    tc_fence_after();
    if (sm.abort) dead = true;
  }
  if (warp == kMmaWarp) {
    if (lane == 0) {
      mma_commit(smem_u32(&sm.drain));
      mbar_wait(smem_u32(&sm.drain), 0, &sm.never, kWaitLimitNs);
    }
    __syncwarp();
  }
  if (threadIdx.x == 0 && sm.abort && pieces > 0)  // a query still on its way lands before the block leaves
    mbar_wait(smem_u32(&sm.q_full), (pieces - 1) & 1u, &sm.never, kWaitLimitNs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partials of items that were cut: one warp per query row and latent half, in slot order.  Rows of
// sequences with a bad length become zeros.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, hf = (int)(w & 1);
  const int64_t row = w >> 1;
  if (row >= (int64_t)p.B * p.R) return;
  const int b = (int)(row / p.R), r = (int)(row % p.R), g = r / kRows, i = r % kRows;
  uint4* dst = reinterpret_cast<uint4*>(p.ctx + row * kDC + 256 * hf);
  if (item_keys(p, b * p.groups + g) == 0) {
    dst[lane] = make_uint4(0u, 0u, 0u, 0u);
    if (hf == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = -INFINITY;
    return;
  }
  int4 e = p.table[b * p.groups + g];
  if (e.z == 1) return;
  // a decode that gave up may have left no entry
  if ((unsigned)e.x >= 2u * p.pairs || e.y < 0 || e.z < 0 || e.z > p.pairs || e.y > p.pairs - e.z) e.z = 0;
  const int stride = min(p.R, kRows);
  auto part = [&](int k) { return 2 * (int64_t)(k == 0 ? e.x : 2 * (e.y + k)) + hf; };
  float M = -INFINITY;
  for (int k = lane; k < e.z; k += 32) M = fmaxf(M, p.ws_ml[part(k) * kRows + i].x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // lane l holds features 8 l .. 8 l + 7: chunks 2 l and 2 l + 1 of the rotated row
#pragma unroll 4
  for (int k = 0; k < e.z; ++k) {
    const float2 ml = p.ws_ml[part(k) * kRows + i];
    const float4* src = reinterpret_cast<const float4*>(p.ws_o + (part(k) * stride + i) * 256);
    const float4 a = src[(2 * lane + i) & 63], c = src[(2 * lane + 1 + i) & 63];
    if (ml.y == 0.f) continue;  // the row saw none of this piece's keys
    const float f = exp2f(ml.x - ref);
    L = fmaf(f, ml.y, L);
    const float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = fmaf(f, v[j], o[j]);
  }
  const float inv = (L == 0.f ? 0.f : 1.f / L) * p.kv.latent_scale;
  dst[lane] = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                         pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
  if (hf == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

bool query_map(CUtensorMap* m, const void* base, int width, int R, int B, int64_t ld) {
  const uint64_t dims[3] = {(uint64_t)width, (uint64_t)R, (uint64_t)B};
  const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * R};
  const uint32_t box[3] = {64, kRows, 1};
  return make_tensor_map_bf16(m, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
int max_pairs() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 1 ? sms / 2 : 1;
}
// Pairs that this shape can keep busy at most
int shape_pairs(int n_h, int B, int T, int n_max) {
  const int64_t groups = ((int64_t)n_h * T + kRows - 1) / kRows, tiles = groups * B * ((n_max + kTile - 1) / kTile);
  const int pairs = max_pairs();
  return (int)(tiles < pairs ? tiles : pairs);
}
size_t table_bytes(int n_h, int B, int T) { return (size_t)B * (((size_t)n_h * T + kRows - 1) / kRows) * sizeof(int4); }
size_t ml_bytes(int pairs) { return (size_t)pairs * 2 * 2 * kRows * sizeof(float2); }

}  // namespace decode_fp4

size_t decode_fp4_tc_workspace(int n_h, int B, int T, int n_max) {
  using namespace decode_fp4;
  const int pairs = shape_pairs(n_h, B, T, n_max), R = n_h * T;
  return table_bytes(n_h, B, T) + ml_bytes(pairs) + (size_t)pairs * 2 * 2 * (R < kRows ? R : kRows) * 256 * sizeof(float);
}

cudaError_t decode_fp4_tc_launch(const Fp4DecodeArgs& a, void* ws, cudaStream_t st) {
  using namespace decode_fp4;
  Params p{};
  p.kv = a.kv;
  p.lengths = a.lengths;
  p.B = a.B; p.T = a.T; p.n_h = a.n_h; p.n_max = a.n_max;
  p.R = a.T * a.n_h;
  p.groups = (p.R + kRows - 1) / kRows;
  if (!query_map(&p.tm_q, a.q_tilde, kDC, p.R, a.B, a.ldqt) || !query_map(&p.tm_qp, a.q_pe, kDR, p.R, a.B, a.ldqp))
    return cudaErrorInvalidValue;
  p.pairs = shape_pairs(a.n_h, a.B, a.T, a.n_max);
  p.scale_log2 = a.scale * kLog2e;
  p.ctx = static_cast<__nv_bfloat16*>(a.ctx);
  p.lse = a.lse;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.table = reinterpret_cast<int4*>(w);
  w += table_bytes(a.n_h, a.B, a.T);
  p.ws_ml = reinterpret_cast<float2*>(w);
  w += ml_bytes(p.pairs);
  p.ws_o = reinterpret_cast<float*>(w);
  p.err = a.err;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_kernel, dim3(2 * p.pairs), dim3(kThreads), kSmemBytes, st, p);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)p.B * p.R * 2;
  return launch_pdl(join_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace mla
