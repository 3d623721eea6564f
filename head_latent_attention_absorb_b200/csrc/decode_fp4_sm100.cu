// Absorbed decode over the 4-bit latent cache on tcgen05 tensor cores (sm_100a):
//   z[r, t] = scale (q~_r . c_t + q_pe,r . k^R_t),  ctx_r = sum_t softmax(z)_t c_t,  lse_r = log sum_t exp z
// for the R = T n_h query rows r of a sequence (row r belongs to new token r / n_h and sees the rows
// t <= L - T + r / n_h), c_t = code * scale decoded on chip.
//
// Bound: the tensor pipe.  A cached row costs 2 R (2 d_c + d_r) operations against 416 bytes: at R = 128
// 669 a byte, far right of the GPU's ridge.  Measured (one call, replayed in a graph): B = 32, N = 4096, 128 heads
// 51.7 us, 706 TFLOP/s; B = 8, 1024 to 65536 rows 85 us; 32 query rows (16 heads, 2 tokens), B = 32, up to 8191 rows
// 56 us, a quarter of each MMA's rows in use; B = 1, N = 1000 18.4 us.  A tile of 128 keys takes a pair 4000 cycles, 2190
// of them in the MMAs: the loop from a released buffer over the decode of its next keys, the scores and the softmax
// to the values crosses between the CTAs four times.  Some 17 us of a call lie outside its tiles: work split and
// query (8), the end of the pipeline and the partials (6), the join (3).
//
// Why this split.  The fp32 context of 128 rows x 512 features fills TMEM, so no SM can hold it beside
// scores.  Every MMA therefore spans a CTA pair (cta_group::2, M = 128): each CTA holds 64 of the rows with their
// whole context (256 columns).  The pair's MMAs take B from both CTAs' shared memory, the scores' keys split
// by position (64 of a tile's 128 each), the values' by feature (256 of 512 each).  So a CTA decodes 64 whole
// rows, and the values of its 256 features for the other 64 rows: 1.5 times the cache's elements per pair, and
// no data crosses between the CTAs, only barrier arrivals.  Pair MMAs of these shapes run at the full rate also
// with A in shared memory (2190 cycles a tile measured alone; single-CTA M = 128 MMAs with N = 64 need 42 cycles
// instead of 32, and 75 with A in shared memory).
//
// * Operands are fp16: code * scale has at most six significant bits and lies in 2^-10 .. 2688, so the cache
//   is exact; a query row is scaled by a power of two that puts its largest element into [2^14, 2^15), so that
//   bf16 elements are exact down to 2^-31 of it, and the power goes into the row's softmax scale.  The rotary
//   part stays in bf16 (separate MMAs into the same accumulator).  Probabilities are rounded to fp16.
// * Shared memory (224 KB): region X holds the key slabs of features 0..255 (three buffers), region Y those of
//   256..511 (two), the rotary slab, query features 256..511 and the rotary query, the probabilities.
//   One of the regions holds the CTA's own half of the features: its slabs serve the scores (K-major) and are the
//   values of these 64 rows (MN-major).  In the other one the values of the other 64 rows replace the slabs once
//   the scores are done.  Then X holds the values of the tile's first 64 rows and Y of its last 64, in both CTAs.
// * TMEM: context 256 columns, scores two buffers of 64, query features 0..255 128 columns (A operand, in both
//   lane halves).
// * Thirteen warps decode: 16-byte loads of codes one tile ahead in registers, cvt to fp16, one product with the
//   block's scale, stores in the 128-byte-swizzled layout.
// * MMA order S(t + 1), O(t), S(t + 2), ...: the softmax of tile t runs under O(t - 1) and S(t + 1).  (With one
//   score buffer S(t + 1) waited for both CTAs to have read S(t): an arrival at the other CTA takes some hundred
//   cycles.)  The scores start with X, whose third buffer is decoded ahead,
//   while Y's are decoded behind O.
// * Eight softmax warps: a thread has 32 keys of a query row and agrees with the three threads that have the row's
//   others on the reference of the base-2 exponentials, which moves (and the context is rescaled in TMEM) only when the
//   running maximum grows by more than 8.
// * Work: chunks of single sequences when each can have pairs of its own and the chunks come out balanced, else
//   equal ranges of all tiles.  A sequence that is cut leaves fp32 partials and a second kernel joins them in a
//   fixed order.
// * The roles are functions with compact loops: together they have to fit the instruction cache (unrolled, the
//   loops took twice as long).
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
constexpr int kTile = 128, kKeys = 64;           // keys per tile, and of it per CTA
constexpr int kRows = 128, kMyRows = 64;         // query rows per group, and per CTA
constexpr int kSlabBytes = 64 * 128;             // 64 rows (keys or query rows) of 64 features
constexpr int kRegion = 4 * kSlabBytes;          // half of the latent features of 64 keys
constexpr int kXBufs = 3, kYBufs = 2;
constexpr int kQTmemSlabs = 4;                   // query slabs in TMEM; the other four and the rotary one in shared memory
constexpr int kYOff = kXBufs * kRegion;
constexpr int kRopeOff = kYOff + kYBufs * kRegion;
constexpr int kQOff = kRopeOff + kSlabBytes;
constexpr int kPOff = kQOff + 5 * kSlabBytes;    // probabilities of the first and the last 64 keys
constexpr int kSmemOff = kPOff + 2 * kSlabBytes;
static_assert(kQTmemSlabs * kSlabBytes <= kRegion, "the query for TMEM is staged in a buffer of region X");
static_assert(kMyRows * kDC * 4 <= kRopeOff, "the partial context is staged in the regions");
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kKWarp0 = 9, kVWarp0 = 17, kRopeWarp = 21;
constexpr int kKWarps = 8, kVWarps = 4;
constexpr int kThreads = 32 * (kRopeWarp + 1);
constexpr uint32_t kTmemCols = 512, kColO = 0, kColS = 256, kColQ = 384;  // scores: two buffers of 64
// Probabilities are 2^(z - ref): ref is set kRaise below the largest score so far (log2 units) and moved up
// only when a score passes it by kRescale.  So they reach 2^15 at most (fp16 ends at 2^16), the sum is at
// least 2^kRaise, and a probability that fp16's subnormals round (2^-25) is off by 2^-32 of the sum.
constexpr float kRaise = 7.f, kRescale = 15.f;
constexpr int kPlanRegs = 3;                     // items per lane that the chunk search holds (more than the pairs)
constexpr int kJoin = 4;                         // partials that a warp of the join reads at once
// What a second piece costs a pair, in tiles: the end of the pipeline, the result and the next query, some 13 us against
// 2 us a tile.  (Measured with 3, 9 and 12: 60 sequences of 4096 rows 87, 82 and 81 us, 40 of 2048 49, 46 and 47,
// 44 of 4096 72, 73 and 82.)
constexpr int kSwitchTiles = 9;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The roles read their arguments from shared memory: handed to functions that are not inlined, a reference to the
// kernel's parameters becomes loads through L1, some hundred cycles each.
struct Args {
  CacheView kv;
  const int32_t* lengths;
  int B, T, n_h, n_max, R, groups, pairs;
  float scale_log2;
  __nv_bfloat16* ctx;
  float* lse;
  int4* table;    // [B * groups] partials of an item: first slot, first CTA pair, number
  float2* ws_ml;  // [2 pairs slots][128] (reference in log2 units, sum)
  float* ws_o;    // [slots][4 quarters of the features][min(R, 128)][128], 16-byte chunk j of row r at (j + r) % 32
  int32_t* err;
};
struct Params {
  CUtensorMap tm_q;   // (d_c, R, B) query rows, box (64, 64, 1), 128-byte swizzle: rows past R read as zeros
  CUtensorMap tm_qp;  // (d_r, R, B), same box
  Args a;
};

// An item is a group of up to 128 query rows of one sequence.  Keys its last row sees, 0 for a bad length.
__device__ __forceinline__ int item_keys(const Args& p, int b, int g) {
  const int len = p.lengths[b];
  if (len < p.T || len > p.n_max) return 0;
  return g == p.groups - 1 ? len : len - p.T + (kRows * (g + 1) - 1) / p.n_h + 1;
}
__device__ __noinline__ int item_tiles(const Args& p, int i) {
  const int b = p.groups == 1 ? i : i / p.groups;
  return (item_keys(p, b, i - b * p.groups) + kTile - 1) / kTile;
}

// A CTA pair's share: pieces of items.
struct Plan {
  int lo, hi, tb;          // tiles [lo, hi) of all items' tiles laid end to end; first tile of `item`
  int item, chunk, c0, n;  // chunk > 0: one piece, the (pair - c0)-th of item's n chunks
  int nc, q, rem;          // pairs that have work; total tiles = q nc + rem
};
struct Piece {
  int item;              // < 0: none left
  int b, g, len;         // its sequence, group of query rows, and the sequence's length
  int begin, n;          // first tile, tiles
  int slot, c0, pieces;  // where its partial goes; first pair and number of the item's pieces
  int hiding;            // its first tile, from `begin` on, with a key that the group's first row does not see
};

struct Smem {
  // Waited for in the even CTA only; arrivals from both CTAs.  (The waiting thread reads nothing that they
  // guard, it issues MMAs; an acquire at cluster scope would cost it some hundred cycles a wait.)
  uint64_t x_full[kXBufs], y_full[kYBufs], rope_full, v_full[2], s_empty[2], p_full, q_ready;
  // in each CTA; arrivals from the MMAs
  uint64_t x_empty[kXBufs], y_empty[kYBufs], rope_empty, s_full[2], pv_done, drain;
  uint64_t q_full, q_placed;
  float share[2][4][kMyRows];          // exchange between the four threads of a row
  Args args;
  Plan plan;
  Piece piece[2];  // the one at hand, the next one
  uint32_t tmem_base;
  int abort, never;
};
constexpr int kSmemBytes = kSmemOff + (int)sizeof(Smem);
static_assert(kSmemBytes <= 232448, "shared memory above 227 KB");

// (the kernel checks that the hardware places it on a 1024-byte boundary: there is no room to round it up)
__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  return smem_raw;
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
// The MMA thread polls before it lets the hardware put it to sleep: waking up takes some hundred cycles, and one
// polling thread costs the others little.
__device__ __forceinline__ bool wait_awake(Smem& sm, uint64_t& bar, uint32_t parity, int32_t* err) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_test(smem_u32(&bar), parity)) return true;
  return wait_more(sm, smem_u32(&bar), parity, err);
}
// All lanes wait; the warp goes on only if all of them saw the phase complete.
__device__ __forceinline__ bool wait_warp(Smem& sm, uint64_t& bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, wait(sm, bar, parity, err));
}
// Arrival on a barrier of the even CTA.
__device__ __forceinline__ void arrive_even(uint64_t& bar, uint32_t rank) {
  if (rank == 0)
    mbar_arrive(smem_u32(&bar));
  else
    mbar_arrive_remote_cta(mapa(smem_u32(&bar), 0));
}

// First tile of pair c's share: floor(total c / nc).  (The launch refuses totals of 2^31 tiles.)
__device__ __forceinline__ int share(const Plan& s, int c) { return s.q * c + s.rem * c / s.nc; }
// The pair whose share holds tile t.
__device__ __forceinline__ int holder(const Plan& s, int t) {
  int c = t / (s.q + 1);
  while (c + 1 < s.nc && share(s, c + 1) <= t) ++c;
  return c;
}

// One thread: the next piece of pair c.
__device__ __noinline__ void next_piece(const Args& p, int c, Plan& s, Piece& r) {
  const int items = p.B * p.groups;
  r.item = -1;
  if (s.chunk > 0) {
    if (s.item >= items) return;
    r.item = s.item;
    r.begin = (c - s.c0) * s.chunk;
    r.n = min(s.chunk, item_tiles(p, s.item) - r.begin);
    r.slot = 2 * c;
    r.c0 = s.c0;
    r.pieces = s.n;
    s.item = items;
  } else {
#pragma unroll 1
    for (; r.item < 0 && s.item < items && s.lo < s.hi; ++s.item) {
      const int nt = item_tiles(p, s.item), tb = s.tb;
      s.tb += nt;
      if (s.tb <= s.lo) continue;
      r.item = s.item;
      r.begin = s.lo - tb;
      r.n = min(s.hi, s.tb) - s.lo;
      r.c0 = holder(s, tb);
      r.pieces = holder(s, tb + nt - 1) - r.c0 + 1;
      r.slot = 2 * c + (share(s, c) < tb ? 1 : 0);  // a pair's first and its later pieces
      s.lo += r.n;
    }
    if (r.item < 0) return;
  }
  r.b = p.groups == 1 ? r.item : r.item / p.groups;
  r.g = r.item - r.b * p.groups;
  r.len = p.lengths[r.b];
  r.hiding = p.T == 1 ? 0x7fffffff : (r.len - p.T + (kRows * r.g) / p.n_h + 1) / kTile - r.begin;
}

// One warp: the share of pair c and its first piece.
__device__ __noinline__ void make_plan(const Args& p, int c, Plan* out, Piece* piece) {
  const int lane = threadIdx.x & 31, items = p.B * p.groups;
  int total = 0, longest = 0, nonempty = 0, nt[kPlanRegs];
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
  total = __reduce_add_sync(0xffffffffu, total);
  longest = __reduce_max_sync(0xffffffffu, longest);
  nonempty = __reduce_add_sync(0xffffffffu, nonempty);
  if (__any_sync(0xffffffffu, bad) && c == 0 && lane == 0) raise_error(p.err, MLA_ERR_LENGTH);
  Plan r;
  r.nc = min(total, p.pairs);
  r.q = r.nc > 0 ? total / r.nc : 0;
  r.rem = total - r.q * r.nc;
  r.lo = r.hi = r.tb = 0;
  r.item = items;
  r.chunk = r.c0 = r.n = 0;
  if (c < r.nc) {
    // the smallest chunk whose chunks fit the pairs, if that is little above the even share
    const int even = r.q + (r.rem > 0);
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
      r.lo = share(r, c);
      r.hi = share(r, c + 1);
    }
    int base = 0;  // chunks or tiles before item i0
    const int at = r.chunk > 0 ? c : r.lo;
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += 32) {
      int n = i0 == 0 ? nt[0] : i0 + lane < items ? item_tiles(p, i0 + lane) : 0;
      if (r.chunk > 0) n = (n + r.chunk - 1) / r.chunk;
      int sum = n;
#pragma unroll 1
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
    r.c0 = r.tb;  // chunk plan: the item's first chunk is its first pair's
  }
  if (lane == 0) {
    *out = r;
    next_piece(p, c, *out, *piece);
  }
  __syncwarp();
}

// A decode warp has 4 G of 64 keys and one half of the latent features, 128 bytes of codes, at a time: eight lanes cover a
// key's, so an instruction reads four keys in about six cache lines (one key per lane pair, 64 features each,
// needed sixteen, and the L1 lookups then bounded the kernel).  Lane l has 32 features, of slab (l & 7) / 2, and
// of the keys 4 i + r, i < G, the r that makes the eight lanes of a store phase hit distinct banks: the four
// slabs take four different rows.
template <int G>
struct Part {
  uint4 code[G];
  uint32_t scale[G];
};
struct PartSource {
  const uint8_t* code;
  const uint8_t* scale;
  int64_t code4, scale4;  // four rows on
  int left;               // keys from the lane's first one on that are in the sequence
};
__device__ __forceinline__ int part_row(int lane) { return ((lane >> 3) + ((lane & 7) >> 1)) & 3; }
// From key `first` on, half `region` of the features
__device__ __forceinline__ PartSource part_source(const Args& p, int b, int len, int first, int region, int lane) {
  const int64_t t = (int64_t)first + part_row(lane);
  return {p.kv.c4 + b * p.kv.c4_b + t * p.kv.c4_r + 128 * region + 16 * (lane & 7),
          p.kv.sc + b * p.kv.sc_b + t * p.kv.sc_r + 16 * region + 2 * (lane & 7), 4 * p.kv.c4_r, 4 * p.kv.sc_r,
          (int)(len - t)};
}
// Loads the source's keys; those of the other half of the features, too, lie `half` halves away.  (Plain loads: the append
// or eviction before this kernel may still be writing rows when it starts, so the cache is not read-only for the kernel's
// lifetime, as a load through the non-coherent path requires.)
template <int G>
__device__ __forceinline__ void load_part(const PartSource& s, int half, Part<G>& k) {
#pragma unroll
  for (int i = 0; i < G; ++i) {
    k.code[i] = make_uint4(0u, 0u, 0u, 0u);
    k.scale[i] = 0u;
    if (4 * i < s.left) {  // rows behind the sequence may hold anything, or not exist
      k.code[i] = *reinterpret_cast<const uint4*>(s.code + i * s.code4 + 128 * half);
      k.scale[i] = *reinterpret_cast<const uint16_t*>(s.scale + i * s.scale4 + 16 * half);
    }
  }
}
__device__ __forceinline__ void next_tile(PartSource& s) {
  s.code += kTile / 4 * s.code4;
  s.scale += kTile / 4 * s.scale4;
  s.left -= kTile;
}
// A key that some query rows do not see gets the probability 0 from them, but 0 times a NaN value is NaN.  So in tiles with
// such keys (Piece::hiding) NaN scales count as 0, and the rotary row of their key is NaN instead, which makes the key's
// scores NaN for the rows that do see it.
template <int G>
__device__ __forceinline__ void drop_nan(Part<G>& k) {
#pragma unroll
  for (int i = 0; i < G; ++i) k.scale[i] &= ~(((((k.scale[i] & 0x7f7fu) + 0x0101u) & 0x8080u) >> 7) * 0xffu);
}
// Decodes into the region at `dst`, keys 4 G j on.
template <int G>
__device__ __forceinline__ void store_part(const Part<G>& k, uint32_t dst, int j, int lane) {
  const int half = lane & 1, r = part_row(lane);
  dst += ((lane & 7) >> 1) * kSlabBytes + (4 * G * j + r) * 128;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const uint32_t s2 = fp4::scales_to_f16(k.scale[i]);
    const uint32_t s[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
    const uint32_t words[4] = {k.code[i].x, k.code[i].y, k.code[i].z, k.code[i].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t h[4];
      fp4::codes_to_f16(words[w], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = fp4::mul_f16x2(h[e], s[w >> 1]);
      st_shared_v4_b32(dst + 512 * i + (((4 * (half ^ (i & 1)) + w) ^ r) << 4), h[0], h[1], h[2], h[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}
// The rotary warp: eight lanes cover a key's row, lane l has the keys l / 8 + 4 i.
__device__ __forceinline__ void load_rope(const uint8_t*& src, int64_t rows4, int left, uint4 (&k)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    k[i] = 4 * i < left ? *reinterpret_cast<const uint4*>(src + i * rows4) : make_uint4(0u, 0u, 0u, 0u);
  src += kTile / 4 * rows4;
}
__device__ __forceinline__ void store_rope(const uint4 (&k)[16], uint32_t dst, int lane) {
  dst += (lane >> 3) * 128;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    st_shared_v4_b32(dst + 512 * i + (((lane & 7) ^ (lane >> 3) ^ (4 * (i & 1))) << 4), k[i].x, k[i].y, k[i].z, k[i].w);
}
// The rotary chunks of keys with a NaN among their scales, of which a lane looks at four, become NaN; `t`, `left` as above.
__device__ __noinline__ void mark_nan(const Args& p, int b, int t, int left, uint32_t dst, int lane) {
  const uint8_t* src = p.kv.sc + b * p.kv.sc_b + t * p.kv.sc_r + 4 * (lane & 7);
  dst += (lane >> 3) * 128;
#pragma unroll 1
  for (int i = 0; i < 16 && 4 * i < left; ++i) {
    const uint32_t s = *reinterpret_cast<const uint32_t*>(src + 4 * i * p.kv.sc_r);
    if (((s & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)
      st_shared_v4_b32(dst + 512 * i + (((lane & 7) ^ (lane >> 3) ^ (4 * (i & 1))) << 4), 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u,
                       0x7fc07fc0u);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Where slab j of the query lands (8: the rotary one): those for TMEM at `stage`.
__device__ __forceinline__ uint32_t query_slab(uint32_t base, uint32_t stage, int j) {
  return j < kQTmemSlabs ? stage + j * kSlabBytes : base + kQOff + (j - kQTmemSlabs) * kSlabBytes;
}

// One thread: the CTA's 64 query rows of the item as they are (bf16, rows past R as zeros).
__device__ __noinline__ void fetch_query(const CUtensorMap* maps, Smem& sm, uint32_t base, uint32_t stage, int b, int row) {
  fence_proxy_async_smem();  // the buffers were read and written by threads before
  const uint64_t pol = policy_evict_first();
  const uint32_t bar = smem_u32(&sm.q_full);
  mbar_arrive_expect_tx(bar, 9 * kSlabBytes);
#pragma unroll 1
  for (int j = 0; j < 8; ++j) tma_load_3d(query_slab(base, stage, j), maps, bar, 64 * j, row, b, pol);
  tma_load_3d(query_slab(base, stage, 8), maps + 1, bar, 0, row, b, pol);
}

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The query rows in place, by the softmax warps, one row per thread and TMEM lane (lanes 64.. repeat the rows): the
// row's power of two; the latent part to fp16, slabs 0..3 in TMEM (the first four warps), the others where they are
// (the other four warps, with the rotary part, which is only scaled).  `scale`: the row's softmax scale, log2 units.
__device__ __noinline__ bool place_query(Smem& sm, uint32_t base, uint32_t tmem, uint32_t stage,
                                         uint32_t parity, float* scale) {
  const Args& p = sm.args;
  const int lane = threadIdx.x & (kRows - 1), r = lane & (kMyRows - 1), h = threadIdx.x >> 7, hi = lane >> 6;
  const bool ok = wait_warp(sm, sm.q_full, parity, p.err);
  auto chunk = [&](int j, int c) { return query_slab(base, stage, j) + r * 128 + ((c ^ (r & 7)) << 4); };
  const float ls = p.kv.latent_scale;
  // two latent slabs each, the rotary one by the last
  const int j0 = 4 * h + 2 * hi;
  float m = 0.f;
#pragma unroll 1
  for (int j = j0; j < (h + hi == 2 ? 9 : j0 + 2); ++j) {
    uint32_t big = 0u;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = ld_shared_v4_b32(chunk(j, c));
      big = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(big, u.x), u.y), u.z), u.w);
    }
    m = fmaxf(m, fmaxf(bf16_lo(big), bf16_hi(big)) * (j < 8 ? ls : 1.f));
  }
  float(&x)[4][kMyRows] = sm.share[0];
  x[2 * h + hi][r] = m;
  named_bar_sync(1, 256);
  m = fmaxf(fmaxf(x[0][r], x[1][r]), fmaxf(x[2][r], x[3][r]));
  // 2^e that puts the largest element into [2^14, 2^15); the latent part takes 2^e times latent_scale
  const int le = (int)(__float_as_uint(ls) >> 23) - 127;
  const int e = m > 0.f ? max(max(-126, -126 - le), min(min(126, 126 - le), 14 + 127 - (int)(__float_as_uint(m) >> 23))) : 0;
  *scale = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 1.2e-38f);
  const float mul_pe = __uint_as_float((uint32_t)(127 + e) << 23), mul_lat = __uint_as_float((uint32_t)(127 + e + le) << 23);
  // h = 0: slabs 0..3;  h = 1: 4, 5 and 8 by the rows of lanes 0.., 6 and 7 by their repetition
  const int jn = h == 0 ? 4 : hi == 0 ? 3 : 2;
#pragma unroll 1
  for (int k = 0; k < jn; ++k) {
    const int j = h == 0 ? k : k == 2 ? 8 : j0 + k;
    uint32_t v[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = ld_shared_v4_b32(chunk(j, c));
      v[4 * c] = u.x;
      v[4 * c + 1] = u.y;
      v[4 * c + 2] = u.z;
      v[4 * c + 3] = u.w;
    }
    if (j < 8) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = pack_f16x2_ieee(bf16_lo(v[i]) * mul_lat, bf16_hi(v[i]) * mul_lat);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = pack_bf16x2(bf16_lo(v[i]) * mul_pe, bf16_hi(v[i]) * mul_pe);
    }
    if (h == 0) {
      tmem_st32(tmem + ((uint32_t)(lane & 96) << 16) + kColQ + 32 * j, v);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_v4_b32(chunk(j, c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
  }
  if (h == 0) tmem_st_wait();
  tc_fence_before();
  fence_proxy_async_smem();
  return ok;
}

// The roles are functions of their own so that each has the registers to itself (inlined together they spill), and
// read the piece at hand from shared memory.

// A 128-byte-swizzled shared-memory descriptor whose address is at + 32 k: the low word counts 16 bytes.
__device__ __forceinline__ uint64_t step_desc(uint32_t at, int k, uint32_t lbo_bytes = 16) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (kSwizzle128 << 29);
  return ((uint64_t)hi << 32) | ((lbo_bytes >> 4) << 16 | ((at >> 4) + 2 * k));
}

// One 64-feature slab of the scores, the query slab in TMEM columns q or in shared memory at q.
__device__ __forceinline__ void slab_ts(uint32_t s, uint32_t q, uint32_t keys) {
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_pair_ts(s, q + 8 * k, step_desc(keys, k), idesc_f16_f32(kRows, kTile, 0, 0), 1u);
}
__device__ __forceinline__ void slab_ss(uint32_t s, uint32_t q, uint32_t keys, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_pair_ss(s, step_desc(q, k), step_desc(keys, k), idesc, first && k == 0 ? 0u : 1u);
}
// The context from 64 keys: their values at `v`, their probabilities at `pr`; 128 of each CTA's features at a time.
__device__ __forceinline__ void values(uint32_t o, uint32_t pr, uint32_t v, bool first) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_pair_ss(o + 128 * i, step_desc(pr, k), step_desc(v + 2 * i * kSlabBytes + 2048 * k, 0, kSlabBytes),
                  idesc_f16_f32(kRows, 256, 0, 1), first && k == 0 ? 0u : 1u);
}

// One warp of the even CTA: the pair's MMAs of a piece, issued by one thread: S(t), then O(t - 1).
__device__ __noinline__ bool mma_role(uint32_t it0, uint32_t n, uint32_t parity) {
  uint8_t* smem = shared_base();
  Smem& sm = *reinterpret_cast<Smem*>(smem + kSmemOff);
  const Args& p = sm.args;
  const uint32_t base = smem_u32(smem), tmem = sm.tmem_base, tQ = tmem + kColQ, tO = tmem + kColO;
  constexpr uint16_t kBoth = 3;
  bool ok = true;
  if (elect_one()) {
    ok = wait_awake(sm, sm.q_ready, parity, p.err);
#pragma unroll 1
    for (uint32_t t = 0; t <= n && ok; ++t) {
      if (t < n) {
        const uint32_t it = it0 + t, xb = it % kXBufs, yb = it % kYBufs, tS = tmem + kColS + 64 * (it & 1u);
        ok = wait_awake(sm, sm.s_empty[it & 1u], ((it >> 1) & 1u) ^ 1u, p.err) && wait_awake(sm, sm.x_full[xb], (it / kXBufs) & 1u, p.err) &&
             wait_awake(sm, sm.rope_full, it & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t x = base + xb * kRegion, y = base + kYOff + yb * kRegion;
        slab_ss(tS, base + kQOff + 4 * kSlabBytes, base + kRopeOff, idesc_bf16_f32(kRows, kTile, 0, 0), true);
        mma_commit_pair(smem_u32(&sm.rope_empty), kBoth);
#pragma unroll
        for (int j = 0; j < 4; ++j) slab_ts(tS, tQ + 32 * j, x + j * kSlabBytes);
        ok = wait_awake(sm, sm.y_full[yb], (it / kYBufs) & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          slab_ss(tS, base + kQOff + j * kSlabBytes, y + j * kSlabBytes, idesc_f16_f32(kRows, kTile, 0, 0), false);
        mma_commit_pair(smem_u32(&sm.s_full[it & 1u]), kBoth);
      }
      if (t > 0) {
        const uint32_t it = it0 + t - 1, xb = it % kXBufs, yb = it % kYBufs;
        ok = wait_awake(sm, sm.v_full[it & 1u], (it >> 1) & 1u, p.err) && wait_awake(sm, sm.p_full, it & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
        values(tO, base + kPOff + kSlabBytes, base + kYOff + yb * kRegion, t == 1);
        mma_commit_pair(smem_u32(&sm.y_empty[yb]), kBoth);
        values(tO, base + kPOff, base + xb * kRegion, false);
        mma_commit_pair(smem_u32(&sm.x_empty[xb]), kBoth);
        mma_commit_pair(smem_u32(&sm.pv_done), kBoth);
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Eight warps, 32 keys of a query row per thread: probabilities, and the piece's result.
__device__ __noinline__ bool softmax_role(Smem& sm, const Piece& w, uint32_t it0, float sl, bool ok) {
  const Args& p = sm.args;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, col = warp >> 2;
  const int tl = 32 * quad + lane, r = tl & (kMyRows - 1), half = tl >> 6;  // TMEM lane, row, half of the tile's keys
  const int part = 2 * half + col;                                          // the row's quarter of keys and features
  const uint32_t base = smem_u32(&sm) - kSmemOff, tmem = sm.tmem_base, n = w.n, rank = cluster_ctarank();
  const int g = w.g, len = w.len;
  const int row = kMyRows * (int)rank + r, rows = min(p.R - kRows * g, kRows);  // row of the group, rows that it has
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  const uint32_t tS = tmem + lanes + kColS + 32 * col, tO = tmem + lanes + kColO + 128 * col;
  const uint32_t p_row = base + kPOff + half * kSlabBytes + r * 128;
  // keys that the row, and the group's first row, see
  const int limit = len - p.T + (kRows * g + min(row, rows - 1)) / p.n_h + 1;
  const int all_see = len - p.T + (kRows * g) / p.n_h + 1;
  float ref = -INFINITY, l = 0.f;
  // The four warps that have the same rows meet once a tile and once more at the end.  A warp whose wait failed
  // still comes to all the meetings.
  uint32_t met = 0;
  auto meet = [&]() {
    named_bar_sync(2 + (quad & 1), 128);
    ++met;
  };
#pragma unroll 1
  for (uint32_t t = 0; t < n && ok; ++t) {
    const uint32_t it = it0 + t;
    const int k0 = (w.begin + (int)t) * kTile + 32 * part;
    ok = wait_warp(sm, sm.s_full[it & 1u], (it >> 1) & 1u, p.err);
    if (!ok) break;
    tc_fence_after();
    uint32_t s[32];
    tmem_ld32(tS + 64 * (it & 1u), s);
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_even(sm.s_empty[it & 1u], rank);
    if (k0 + 32 > all_see) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (k0 + i >= limit) s[i] = 0xff800000u;  // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
    const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
    float(&x)[4][kMyRows] = sm.share[it & 1u];
    x[part][r] = mine;
    meet();
    const float z = fmaxf(fmaxf(x[0][r], x[1][r]), fmaxf(x[2][r], x[3][r]));
    float f = 1.f;
    const bool raise = z > ref + kRescale;  // ref = -inf: any finite maximum
    if (raise) {
      f = ex2f_approx(ref - (z - kRaise));
      l *= f;
      ref = z - kRaise;
    }
    const float neg = ref == -INFINITY ? 0.f : -ref;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {  // fp16 pairs in the first 16 words
      const float a = ex2f_approx(fmaf(__uint_as_float(s[i]), sl, neg));
      const float c = ex2f_approx(fmaf(__uint_as_float(s[i + 1]), sl, neg));
      sum[i & 2] += a;
      sum[(i & 2) + 1] += c;
      s[i / 2] = pack_f16x2_ieee(a, c);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if (t > 0) {  // the last tile's probabilities are used up, its context complete
      ok = wait_warp(sm, sm.pv_done, (it - 1) & 1u, p.err);
      if (!ok) break;
      if (__any_sync(0xffffffffu, raise)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
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
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_shared_v4_b32(p_row + (((4 * col + c) ^ (r & 7)) << 4), s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_even(sm.p_full, rank);
  }
  if (ok) {  // the row's sum (the last tile used the other buffer)
    float(&x)[4][kMyRows] = sm.share[(it0 + n) & 1u];
    x[part][r] = l;
    meet();
    l = (x[0][r] + x[1][r]) + (x[2][r] + x[3][r]);
    ok = wait_warp(sm, sm.pv_done, (it0 + n - 1) & 1u, p.err);
  }
  while (met <= n) meet();
  if (ok) {
    // -------------------------------------------------------------- the piece's result
    // The thread has the row's features [128 part, 128 part + 128).  They go through the idle regions, 16-byte
    // chunks rotated by the row so that neither the row-wise writes nor the copies out conflict.
    tc_fence_after();
    const int64_t out_row = (int64_t)w.b * p.R + kRows * g + kMyRows * (int)rank;  // the CTA's first query row
    const int first = 32 * (quad & 1), mine = min(32, rows - kMyRows * (int)rank - first);  // the warp's rows of it
    const bool whole = w.pieces == 1;
    const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) * p.kv.latent_scale : 1.f;
    const uint32_t src = base + warp * (32 * 512), dst = src + lane * 512;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t o[32];
      tmem_ld32(tO + c, o);
      tmem_ld_wait();
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
          st_shared_v4_b32(dst + (((c / 8 + i + r) & 15) << 4), v[0], v[1], v[2], v[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4_b32(dst + (((c / 4 + i + r) & 31) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (whole) {
#pragma unroll 4
      for (int k = lane >> 4; k < mine; k += 2)
        reinterpret_cast<uint4*>(p.ctx + (out_row + first + k) * kDC + 128 * part)[lane & 15] =
            ld_shared_v4_b32(src + k * 512 + (((lane + first + k) & 15) << 4));
      if (part == 0 && row < rows && p.lse != nullptr)
        p.lse[out_row + r] = l == 0.f ? -INFINITY : ref * kLn2 + logf(l);
    } else {
      if (lane == 0 && mine > 0) {
        const int64_t at = (4 * (int64_t)w.slot + part) * min(p.R, kRows) + kMyRows * (int)rank + first;
        bulk_store_s2g(p.ws_o + at * 128, src, mine * 512);
        bulk_group_commit();
        bulk_group_wait_read_all();
      }
      if (part == 0 && row < rows) p.ws_ml[(int64_t)w.slot * kRows + row] = make_float2(ref, l);
    }
    if (threadIdx.x == 0 && rank == 0 && w.begin == 0) p.table[w.item] = make_int4(w.slot, w.c0, w.pieces, 0);
    tc_fence_before();
    fence_proxy_async_smem();
  }
  return ok;
}

// One of eight warps: eight of the CTA's keys of every tile, loaded one tile ahead; first the half in region X, then,
// when the values of two tiles before have been used, the one in region Y.
__device__ __noinline__ bool key_role(Smem& sm, const Piece& w, uint32_t it0, uint32_t parity) {
  const Args& p = sm.args;
  const uint32_t base = smem_u32(&sm) - kSmemOff, n = w.n, rank = cluster_ctarank();
  const int lane = threadIdx.x & 31, j = (threadIdx.x >> 5) - kKWarp0;
  PartSource src = part_source(p, w.b, w.len, w.begin * kTile + kKeys * (int)rank + 8 * j, 0, lane);
  Part<2> x, y;
  load_part(src, 0, x);
  load_part(src, 1, y);
#pragma unroll 1
  for (uint32_t t = 0; t < n; ++t) {
    const uint32_t it = it0 + t, xb = it % kXBufs, yb = it % kYBufs;
    if (!wait_warp(sm, sm.x_empty[xb], ((it / kXBufs) & 1u) ^ 1u, p.err)) return false;
    // (the first use of the third buffer: the query has left it)
    if (t == 2 && !wait_warp(sm, sm.q_placed, parity, p.err)) return false;
    if ((int)t >= w.hiding) {
      drop_nan(x);
      drop_nan(y);
    }
    store_part(x, base + xb * kRegion, j, lane);
    if (lane == 0) arrive_even(sm.x_full[xb], rank);
    next_tile(src);
    load_part(src, 0, x);
    if (!wait_warp(sm, sm.y_empty[yb], ((it / kYBufs) & 1u) ^ 1u, p.err)) return false;
    store_part(y, base + kYOff + yb * kRegion, j, lane);
    if (lane == 0) arrive_even(sm.y_full[yb], rank);
    load_part(src, 1, y);
  }
  return true;
}

// One of four warps: of every tile, the values of 16 of the other CTA's keys replace slabs of the half that is not
// this CTA's, once the tile's scores are done.
__device__ __noinline__ bool value_role(Smem& sm, const Piece& w, uint32_t it0) {
  const Args& p = sm.args;
  const uint32_t base = smem_u32(&sm) - kSmemOff, n = w.n, rank = cluster_ctarank();
  const int lane = threadIdx.x & 31, j = (threadIdx.x >> 5) - kVWarp0;
  PartSource src = part_source(p, w.b, w.len, w.begin * kTile + kKeys * (1 - (int)rank) + 16 * j, (int)rank, lane);
  Part<4> v;
  load_part(src, 0, v);
#pragma unroll 1
  for (uint32_t t = 0; t < n; ++t) {
    const uint32_t it = it0 + t;
    if (!wait_warp(sm, sm.s_full[it & 1u], (it >> 1) & 1u, p.err)) return false;
    if ((int)t >= w.hiding) drop_nan(v);
    store_part(v, base + (rank == 0 ? kYOff + it % kYBufs * kRegion : it % kXBufs * kRegion), j, lane);
    if (lane == 0) arrive_even(sm.v_full[it & 1u], rank);
    next_tile(src);
    load_part(src, 0, v);
  }
  return true;
}

// One warp: the rotary slab of every tile.
__device__ __noinline__ bool rope_role(Smem& sm, const Piece& w, uint32_t it0) {
  const Args& p = sm.args;
  const uint32_t base = smem_u32(&sm) - kSmemOff, n = w.n;
  const int rank = (int)cluster_ctarank();
  const int lane = threadIdx.x & 31, keys = w.begin * kTile + kKeys * rank;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(static_cast<const __nv_bfloat16*>(p.kv.k_r) + w.b * p.kv.kr_b +
                                                        ((int64_t)keys + (lane >> 3)) * p.kv.kr_r) + 16 * (lane & 7);
  int left = w.len - keys - (lane >> 3);
  uint4 k[16];
  load_rope(src, 8 * p.kv.kr_r, left, k);
#pragma unroll 1
  for (uint32_t t = 0; t < n; ++t) {
    if (!wait_warp(sm, sm.rope_empty, ((it0 + t) & 1u) ^ 1u, p.err)) return false;
    store_rope(k, base + kRopeOff, lane);
    if ((int)t >= w.hiding) mark_nan(p, w.b, keys + (int)t * kTile + (lane >> 3), left, base + kRopeOff, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_even(sm.rope_full, rank);
    left -= kTile;
    load_rope(src, 8 * p.kv.kr_r, left, k);
  }
  return true;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Params p) {
  uint8_t* smem = shared_base();
  Smem& sm = *reinterpret_cast<Smem*>(smem + kSmemOff);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, rank = (int)cluster_ctarank();

  griddep_launch_dependents();
  if (base & 1023u) {
    if (threadIdx.x == 0) raise_error(p.a.err, MLA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kXBufs; ++i) {
      mbar_init(smem_u32(&sm.x_full[i]), 2 * kKWarps);
      mbar_init(smem_u32(&sm.x_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.y_full[i]), 2 * kKWarps);
      mbar_init(smem_u32(&sm.y_empty[i]), 1);
      mbar_init(smem_u32(&sm.v_full[i]), 2 * kVWarps);
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.s_empty[i]), 2 * kSoftmaxWarps);
    }
    mbar_init(smem_u32(&sm.rope_full), 2);
    mbar_init(smem_u32(&sm.rope_empty), 1);
    mbar_init(smem_u32(&sm.p_full), 2 * kSoftmaxWarps);
    mbar_init(smem_u32(&sm.q_ready), 2 * kSoftmaxWarps);
    mbar_init(smem_u32(&sm.q_placed), kSoftmaxWarps);
    mbar_init(smem_u32(&sm.q_full), 1);
    mbar_init(smem_u32(&sm.pv_done), 1);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort = sm.never = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_qp);
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  // nothing arrives on the other CTA's barriers before they are there
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  griddep_wait();
  if (warp == 0) {
    static_assert(sizeof(Args) % 4 == 0, "copied by words");
    for (int i = lane; i < (int)sizeof(Args) / 4; i += 32)
      reinterpret_cast<uint32_t*>(&sm.args)[i] = reinterpret_cast<const uint32_t*>(&p.a)[i];
    __syncwarp();
    make_plan(sm.args, pair, &sm.plan, &sm.piece[0]);
  }
  tc_fence_before();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  tc_fence_after();

  // it0: tiles of the earlier pieces.  Both CTAs walk the same pieces, and all warps take every barrier of every
  // piece, also after a failed wait.
  uint32_t it0 = 0, pieces = 0;
  bool dead = false;
  while (true) {
    const uint32_t parity = pieces & 1u;
    const Piece& w = sm.piece[parity];
    if (w.item < 0) break;
    ++pieces;
    // the query for TMEM is staged in the buffer of region X that is used last
    const uint32_t stage = base + (it0 + kXBufs - 1) % kXBufs * kRegion;
    if (threadIdx.x == 0) fetch_query(&p.tm_q, sm, base, stage, w.b, kRows * w.g + kMyRows * rank);
    __syncwarp();
    if (dead) {
      if (warp == kRopeWarp && lane == 0) next_piece(sm.args, pair, sm.plan, sm.piece[parity ^ 1u]);
    } else {
      bool ok = true;
      if (warp < kSoftmaxWarps) {
        float scale;
        ok = place_query(sm, base, sm.tmem_base, stage, parity, &scale);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.q_placed));
          arrive_even(sm.q_ready, rank);
        }
        ok = softmax_role(sm, w, it0, scale, ok);
      } else if (warp == kMmaWarp) {
        ok = rank != 0 || mma_role(it0, w.n, parity);
      } else if (warp < kRopeWarp) {
        ok = warp < kVWarp0 ? key_role(sm, w, it0, parity) : value_role(sm, w, it0);
      } else {
        if (lane == 0) next_piece(sm.args, pair, sm.plan, sm.piece[parity ^ 1u]);
        __syncwarp();
        ok = rope_role(sm, w, it0);
      }
      dead = !ok;
    }
    __syncwarp();
    it0 += w.n;
    __syncthreads();
    tc_fence_after();
    if (sm.abort) dead = true;
  }
  if (sm.abort) {  // what is still on its way, the query and the MMAs, ends before the block leaves
    if (threadIdx.x == 0 && pieces > 0) mbar_wait(smem_u32(&sm.q_full), (pieces - 1) & 1u, &sm.never, kWaitLimitNs);
    __syncwarp();
    if (warp == kMmaWarp && rank == 0) {
      if (elect_one()) {
        mma_commit_pair(smem_u32(&sm.drain), 1);
        mbar_wait(smem_u32(&sm.drain), 0, &sm.never, kWaitLimitNs);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still arrive on its barriers or read its shared memory
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(sm.tmem_base, kTmemCols);
}

// Joins the partials of items that were cut: one warp per query row and latent half, in slot order.  Rows of
// sequences with a bad length become zeros.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args p) {
  griddep_launch_dependents();
  griddep_wait();
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, hf = (int)(w & 1);
  const int row = w >> 1;
  if (row >= p.B * p.R) return;  // (at most 65535 query groups of 128 rows)
  const int b = row / p.R, r = row - b * p.R, g = r / kRows, i = r % kRows;
  uint4* dst = reinterpret_cast<uint4*>(p.ctx + (int64_t)row * kDC + 256 * hf);
  int4 e = p.table[b * p.groups + g];  // (on its way beside the length; a sequence without keys has left none)
  if (item_keys(p, b, g) == 0) {
    dst[lane] = make_uint4(0u, 0u, 0u, 0u);
    if (hf == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = -INFINITY;
    return;
  }
  if (e.z == 1) return;
  // a decode that gave up may have left no entry
  if ((unsigned)e.x >= 2u * p.pairs || e.y < 0 || e.z < 0 || e.z > p.pairs || e.y > p.pairs - e.z) e.z = 0;
  const int stride = min(p.R, kRows);
  auto slot = [&](int k) { return (int64_t)(k == 0 ? e.x : 2 * (e.y + k)); };
  float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // lane l holds features 8 l .. 8 l + 7 of the half: two chunks of a rotated row
  // The loads of kJoin pieces at once: with a branch on what was loaded between them they came one after the other,
  // and a sequence of 32 pieces took 31 us instead of 24.  (Eight at once: 23, but 54 instead of 51 for 32 sequences
  // of two or three pieces each, whose many warps no longer fit the SMs.)
#pragma unroll 1
  for (int k0 = 0; k0 < e.z; k0 += kJoin) {
    float2 ml[kJoin];
    float4 v[kJoin][2];
#pragma unroll
    for (int u = 0; u < kJoin; ++u) {
      ml[u] = make_float2(0.f, 0.f);
      if (k0 + u < e.z) {
        const int64_t s = slot(k0 + u);
        ml[u] = p.ws_ml[s * kRows + i];
        const float4* src = reinterpret_cast<const float4*>(p.ws_o + ((4 * s + 2 * hf + (lane >> 4)) * stride + i) * 128);
        v[u][0] = src[(2 * lane + i) & 31];
        v[u][1] = src[(2 * lane + 1 + i) & 31];
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kJoin; ++u)
      if (ml[u].y != 0.f) top = fmaxf(top, ml[u].x);
    const float ref = top == -INFINITY ? 0.f : top;
    if (k0 > 0) {
      const float f = exp2f(M - ref);
      L *= f;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= f;
    }
    M = top;
#pragma unroll
    for (int u = 0; u < kJoin; ++u) {
      if (ml[u].y == 0.f) continue;  // the row saw none of the piece's keys
      const float f = exp2f(ml[u].x - ref);
      L = fmaf(f, ml[u].y, L);
      const float x[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(f, x[j], o[j]);
    }
  }
  const float inv = (L == 0.f ? 0.f : 1.f / L) * p.kv.latent_scale;
  dst[lane] = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                         pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
  if (hf == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

bool query_map(CUtensorMap* m, const void* base, int width, int R, int B, int64_t ld) {
  const uint64_t dims[3] = {(uint64_t)width, (uint64_t)R, (uint64_t)B};
  const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * R};
  const uint32_t box[3] = {64, kMyRows, 1};
  return make_tensor_map_bf16(m, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
int max_pairs() { return sm_count() > 1 ? sm_count() / 2 : 1; }
// Pairs that this shape can keep busy at most
int shape_pairs(int pairs, int n_h, int B, int T, int n_max) {
  const int64_t groups = ((int64_t)n_h * T + kRows - 1) / kRows, tiles = groups * B * ((n_max + kTile - 1) / kTile);
  return (int)(tiles < pairs ? tiles : pairs);
}
// Pairs that are resident at once (a GPC with an odd number of SMs leaves one over): one wave.  Per device.
int resident_pairs() {
  static PerDevice cache;
  const int dev = current_device();
  if (cache.get(dev) > 0) return cache.get(dev);
  int pairs = max_pairs(), active = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaOccupancyMaxActiveClusters(&active, decode_kernel, &cfg) == cudaSuccess && active > 0 && active < pairs)
    pairs = active;
  cudaGetLastError();  // a failed query leaves no sticky state
  cache.set(dev, pairs);
  return pairs;
}
size_t table_bytes(int n_h, int B, int T) { return (size_t)B * (((size_t)n_h * T + kRows - 1) / kRows) * sizeof(int4); }
size_t ml_bytes(int pairs) { return (size_t)pairs * 2 * kRows * sizeof(float2); }

}  // namespace decode_fp4

size_t decode_fp4_tc_workspace(int n_h, int B, int T, int n_max) {
  using namespace decode_fp4;
  const int pairs = shape_pairs(max_pairs(), n_h, B, T, n_max), R = n_h * T;
  return table_bytes(n_h, B, T) + ml_bytes(pairs) + (size_t)pairs * 2 * 2 * (R < kRows ? R : kRows) * 256 * sizeof(float);
}

cudaError_t decode_fp4_tc_launch(const Fp4DecodeArgs& a, void* ws, cudaStream_t st) {
  using namespace decode_fp4;
  Params params{};
  Args& p = params.a;
  p.kv = a.kv;
  p.lengths = a.lengths;
  p.B = a.B; p.T = a.T; p.n_h = a.n_h; p.n_max = a.n_max;
  p.R = a.T * a.n_h;
  p.groups = (p.R + kRows - 1) / kRows;
  if (!query_map(&params.tm_q, a.q_tilde, kDC, p.R, a.B, a.ldqt) || !query_map(&params.tm_qp, a.q_pe, kDR, p.R, a.B, a.ldqp))
    return cudaErrorInvalidValue;
  static PerDevice allowed;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(decode_kernel), kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  p.pairs = shape_pairs(resident_pairs(), a.n_h, a.B, a.T, a.n_max);
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
  e = launch_pdl(decode_kernel, dim3(2 * p.pairs), dim3(kThreads), kSmemBytes, st, params);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)p.B * p.R * 2;
  return launch_pdl(join_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace mla
