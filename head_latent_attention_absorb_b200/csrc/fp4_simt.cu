// CUDA-core kernels of the 4-bit decode and of the attention-weight pass in fp32, generic in the dimensions.
//
//   decode   z[h,t] = scale (q~_h . c_t + q_pe,h . k^R_t), softmax over t <= length - T + s,
//            ctx_h = sum_t p c_t, lse = log sum exp z      (split over the rows, merged by a second pass)
//   weights  out[t] = [t < length - T] decay acc[t] + sum over tokens s and heads h of exp(z - lse)
//
// One warp per (head, query, split) in the decode and per cached row in the weights; lane l owns the
// 16-feature blocks l and l + 32 of a latent row, so a 4-bit row costs a lane one 8-byte load and
// one scale per block.
//
// Bound: latency, at the few rows and heads that fp32 is used with: a row is a chain of loads, a sum across the warp
// and an exponential, so a warp of the decode takes four rows at once and the splits are short.  3 sequences of 64 to
// 193 rows and 4 heads: 11.4 us (168 with one row at a time in longer splits).  The splits are cut from n_max, since the
// lengths are on the device: in a cache of 65536 rows the same sequences lie in one split each and take 83 us.
// The weights take one query row after the other for each cached row: 4.3 us for those sequences (26 in the large cache, by
// its blocks without rows), 109 us for 4 sequences of 500 rows with 9 heads, 4 tokens and 640 features (their decode 97).
#include <math.h>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kAhead = 4;      // rows that a warp of the decode works on at once
// Rows of a split while there are few of them.  (4, 16 and 64: 9, 11 and 27 us for one sequence of 64 rows and 4 heads,
// 18, 14 and 25 for 3 of 200 rows.)
constexpr int kRowsSplit = 16;
constexpr int kMaxSplits = 64;

// The lane's blocks of latent row t of sequence b (kFp4: decoded; otherwise as it is).
template <int NB, bool kFp4>
__device__ __forceinline__ void load_row(const QueryArgs& a, int b, int t, int lane, float (&c)[NB][16]) {
  const int blocks = (a.d_c + fp4::kBlock - 1) / fp4::kBlock;
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int blk = lane + 32 * k;
#pragma unroll
    for (int i = 0; i < 16; ++i) c[k][i] = 0.f;
    if (blk >= blocks) continue;
    if constexpr (kFp4) {
      const uint8_t* src = a.kv.c4 + b * a.kv.c4_b + t * a.kv.c4_r + 8 * blk;
      const float s = fp4::scale_value(a.kv.sc[b * a.kv.sc_b + t * a.kv.sc_r + blk]) * a.kv.latent_scale;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t word = 0u, h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) word |= (uint32_t)src[4 * w + j] << (8 * j);
        fp4::codes_to_f16(word, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = sm100::unpack_f16x2(h[j]);
          c[k][8 * w + 2 * j] = f.x * s;
          c[k][8 * w + 2 * j + 1] = f.y * s;
        }
      }
    } else {
      const float* src = static_cast<const float*>(a.kv.c_kv) + b * a.kv.ckv_b + t * a.kv.ckv_r + 16 * blk;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * blk + i < a.d_c) c[k][i] = src[i];
    }
  }
}

// A lane's features of query row r.
template <int NB>
struct Query {
  float c[NB][16], pe[4];  // d_r <= 128
  __device__ __forceinline__ void load(const QueryArgs& a, int64_t r, int lane) {
    const float* q = static_cast<const float*>(a.q_tilde) + r * a.ldqt;
    const float* qp = static_cast<const float*>(a.q_pe) + r * a.ldqp;
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int f = 16 * (lane + 32 * k) + i;
        c[k][i] = f < a.d_c ? q[f] : 0.f;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) pe[i] = lane + 32 * i < a.d_r ? qp[lane + 32 * i] : 0.f;
  }
};

// scale (q~ . c_t + q_pe . k^R_t), summed over the warp.  (load_row leaves zeros past d_c.)
template <int NB>
__device__ __forceinline__ float score(const QueryArgs& a, const Query<NB>& q, const float* k_row, int lane,
                                       const float (&c)[NB][16]) {
  float dot = 0.f;
#pragma unroll
  for (int k = 0; k < NB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) dot = fmaf(q.c[k][i], c[k][i], dot);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.d_r) dot = fmaf(q.pe[i], k_row[lane + 32 * i], dot);
  return warp_sum(dot) * a.scale;
}

template <int NB>
__global__ void __launch_bounds__(32 * kWarps) decode_fp4_simt(Fp4DecodeArgs a, int n_splits, float* ws_o, float2* ws_ml) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int h = blockIdx.x * kWarps + warp;
  const int q = blockIdx.y, split = blockIdx.z;
  if (h >= a.n_h) return;
  const int b = q / a.T, s = q % a.T;
  const int len = a.lengths[b];
  const bool bad = len < a.T || len > a.n_max;
  if (bad && lane == 0 && h == 0 && split == 0) raise_error(a.err, MLA_ERR_LENGTH);
  const int n = bad ? 0 : len - a.T + s + 1;  // rows this token sees
  const int chunk = (a.n_max + n_splits - 1) / n_splits;
  const int t0 = split * chunk, t1 = min(t0 + chunk, n);
  const int64_t r = (int64_t)q * a.n_h + h;
  float acc[NB][16];
#pragma unroll
  for (int k = 0; k < NB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[k][i] = 0.f;
  Query<NB> query;
  query.load(a, r, lane);
  float m = -INFINITY, l = 0.f;
  // four rows at a time: their loads and sums overlap, and the running maximum is settled once
  for (int t = t0; t < t1; t += kAhead) {
    float c[kAhead][NB][16], z[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) load_row<NB, true>(a, b, min(t + e, t1 - 1), lane, c[e]);
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int row = min(t + e, t1 - 1);
      z[e] = score<NB>(a, query, static_cast<const float*>(a.kv.k_r) + b * a.kv.kr_b + row * a.kv.kr_r, lane, c[e]);
    }
    float m_new = m;
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (t + e < t1) m_new = fmaxf(m_new, z[e]);
    const bool none = m_new == -INFINITY;  // nothing to weigh yet (NaN scores pass through below)
    const float corr = none ? 1.f : expf(m - m_new);
    l *= corr;
    float p[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      p[e] = t + e >= t1 ? 0.f : none ? (z[e] != z[e] ? z[e] : 0.f) : expf(z[e] - m_new);
      l += p[e];
    }
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float v = acc[k][i] * corr;
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (t + e < t1) v = fmaf(p[e], c[e][k][i], v);
        acc[k][i] = v;
      }
    m = m_new;
  }
  const bool whole = n_splits == 1;
  const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
  const int64_t row = whole ? r : ((int64_t)split * a.B * a.T + q) * a.n_h + h;
#pragma unroll
  for (int k = 0; k < NB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int f = 16 * (lane + 32 * k) + i;
      if (f >= a.d_c) continue;
      if (whole)
        static_cast<float*>(a.ctx)[row * a.d_c + f] = acc[k][i] * inv;
      else
        ws_o[row * a.d_c + f] = acc[k][i];
    }
  if (lane != 0) return;
  if (!whole)
    ws_ml[row] = make_float2(m, l);
  else if (a.lse != nullptr)
    a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

// One CTA per query row: the splits' factors once, then features with eight splits' loads under way.  (The partials are
// not __restrict__: the decode writes them while this kernel may have started, so they are not read-only for its lifetime.)
__global__ void __launch_bounds__(128) combine_fp4_simt(Fp4DecodeArgs a, int n_splits, const float* ws_o, const float2* ws_ml) {
  __shared__ float factor[kMaxSplits];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int64_t r = (int64_t)blockIdx.y * a.n_h + blockIdx.x, rows = (int64_t)a.B * a.T * a.n_h;
  const int lane = threadIdx.x & 31;
  // every warp for itself: lane l has splits l and l + 32
  float2 ml[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    ml[k] = lane + 32 * k < n_splits ? ws_ml[(lane + 32 * k) * rows + r] : make_float2(-INFINITY, 0.f);
  const float M = warp_max(fmaxf(ml[0].x, ml[1].x));
  float L = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float f = ml[k].y != 0.f ? expf(ml[k].x - M) : 0.f;  // (0: the row saw none of the split's keys)
    L = fmaf(f, ml[k].y, L);
    if (threadIdx.x < 32) factor[lane + 32 * k] = f;
  }
  L = warp_sum(L);
  __syncthreads();
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int c = threadIdx.x; c < a.d_c; c += blockDim.x) {
    float acc = 0.f;
#pragma unroll 1
    for (int s0 = 0; s0 < n_splits; s0 += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i < n_splits) v[i] = ws_o[((s0 + i) * rows + r) * a.d_c + c];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i < n_splits && factor[s0 + i] != 0.f) acc = fmaf(factor[s0 + i], v[i], acc);
    }
    static_cast<float*>(a.ctx)[r * a.d_c + c] = acc * inv;
  }
  if (a.lse != nullptr && threadIdx.x == 0) a.lse[r] = L == 0.f ? -INFINITY : M + logf(L);
}

template <int NB, bool kFp4>
__global__ void __launch_bounds__(32 * kWarps) weights_simt(WeightsArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5), b = blockIdx.y;
  const int len = a.lengths[b];
  if (len < a.T || len > a.n_max) {
    if (t == 0 && lane == 0) raise_error(a.err, MLA_ERR_LENGTH);
    return;
  }
  if (t >= len) return;
  float c[NB][16];
  load_row<NB, kFp4>(a, b, t, lane, c);
  const float* k_row = static_cast<const float*>(a.kv.k_r) + b * a.kv.kr_b + t * a.kv.kr_r;
  float w = 0.f;
  // new token s sees rows t <= len - T + s
  for (int s = max(0, t - (len - a.T)); s < a.T; ++s)
    for (int h = 0; h < a.n_h; ++h) {
      const int64_t r = ((int64_t)b * a.T + s) * a.n_h + h;
      const float lse = a.lse[r];
      Query<NB> query;
      query.load(a, r, lane);
      const float z = score<NB>(a, query, k_row, lane, c);
      if (lse != -INFINITY) w += expf(z - lse);  // a row without a softmax gave no weight
    }
  if (lane != 0) return;
  // a new token's row starts from nothing, whatever an evicted row left in its place
  if (a.acc != nullptr && t < len - a.T) w = fmaf(a.decay, a.acc[b * a.acc_b + t], w);
  a.out[b * a.out_b + t] = w;
}

}  // namespace

int decode_fp4_simt_splits(int B, int n_max) {
  // a warp's rows are a chain of loads and sums, about 2 us for four of them: short splits while the GPU has room
  // for more of them, then enough (head group, query, split) blocks to cover it a few times over
  const int by_rows = (n_max + kRowsSplit - 1) / kRowsSplit, want = (4 * 148 + B - 1) / B;
  const int s = by_rows < want ? by_rows : want;
  return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s;
}

size_t decode_fp4_simt_workspace(int n_h, int d_c, int B, int n_max) {
  const int s = decode_fp4_simt_splits(B, n_max);
  return s == 1 ? 256 : (size_t)s * B * n_h * (d_c * sizeof(float) + sizeof(float2)) + 256;
}

cudaError_t decode_fp4_simt_launch(const Fp4DecodeArgs& a, void* ws, cudaStream_t st) {
  const int q = a.B * a.T, splits = decode_fp4_simt_splits(q, a.n_max);
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + (size_t)splits * q * a.n_h * a.d_c);
  const dim3 grid((a.n_h + kWarps - 1) / kWarps, q, splits);
  const cudaError_t e = launch_pdl(a.d_c <= 512 ? decode_fp4_simt<1> : decode_fp4_simt<2>, grid,
                                   dim3(32 * kWarps), 0, st, a, splits, ws_o, ws_ml);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_pdl(combine_fp4_simt, dim3(a.n_h, q), dim3(128), 0, st, a, splits, (const float*)ws_o,
                    (const float2*)ws_ml);
}

cudaError_t weights_simt_launch(const WeightsArgs& a, cudaStream_t st) {
  const dim3 grid((a.n_max + kWarps - 1) / kWarps, a.B);
  const bool fp4 = a.kv.c4 != nullptr;
  if (a.d_c <= 512)
    (fp4 ? weights_simt<1, true> : weights_simt<1, false>)<<<grid, 32 * kWarps, 0, st>>>(a);
  else
    (fp4 ? weights_simt<2, true> : weights_simt<2, false>)<<<grid, 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
