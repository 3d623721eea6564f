// Append to and read-back from the 4-bit latent cache (the format is in fp4.cuh).
//
// Append ("Key-value down-projection", mla-kv excerpt; "Key-value latent RMSNorm"): for token i of
// sequence b, x = kv_a[b, i, 0:d_c],
//   y = g x / sqrt(mean(x^2) + eps) / latent_scale,
//   per block of 16: s = e4m3(max|y| / 6), code = e2m1(y / s)   (nearest, ties to even, saturating)
// and the rotary key y[2j] + j y[2j+1] turned by position * base^(-2j/d_r).
//
// One warp per token: lane l owns blocks l and l + 32, so the block maximum never leaves the lane, and
// only the sum of squares crosses the warp (five shuffles).  A token is 1152 bytes read and 416 written in bf16,
// but a prompt is bound by the instructions and latencies of the quantisation: 11,551 tokens in a batch of four prompts
// padded to 4095 take 16.0 us and their read-back, with its zeros, 9.2 us (each alone, cold caches; 39 and 31 % of the
// issue slots, 1.1 and 2.2 TB/s), together 18.7 us back to back.  The next token's row is on its way while one is
// quantised.  32 single tokens: 4.9 us with the read-back, latency.  fp32 rows, loaded and stored element by element:
// 2000 tokens of 640 features 7.9 us, their read-back 10.3.
//
// A 4-bit code is a step of up to a third of its value, so a value next to a rounding border has to
// fall on the side that the formula puts it on.  The fp32 pass carries a relative error below
// 32 * 2^-24 = 2^-19 (sum of up to 32 squares per lane and five exchanges, halved by the square root:
// 19; reciprocal root 4; two products, the scale's reciprocal and the product with it 5).  It rounds
// each quotient twice, moved down and up by 2^-19; where the two disagree (in about one row of 160), or
// where the sum of squares leaves fp32's safe range, the warp redoes the block in fp64: the scale reaches the
// fp32 converter through round-to-odd, so the second rounding cannot undo the first, and the codes come from
// comparisons with the borders (quotients took most of the kernel's time on prompts).
#include <math.h>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 64;  // rotary pairs: d_r <= 128
constexpr float kDelta = 1.f / 524288.f;  // 2^-19

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// fp64 to fp32 by round-to-odd: a later rounding to few bits then equals the direct one.
__device__ __forceinline__ float to_odd(double v) {
  const float f = __double2float_rz(v);
  if (f == f && (double)f != v) return __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// A block of 16 consecutive elements (bf16 rows are 16-byte aligned, fp32 rows element-aligned) and a rotary pair,
// as loaded and as fp32.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float x[16], k[2];
};
template <> struct Raw<__nv_bfloat16> {
  uint4 x[2];
  uint32_t k;
};
__device__ __forceinline__ void load16(const float* p, Raw<float>& r) {
#pragma unroll
  for (int i = 0; i < 16; ++i) r.x[i] = p[i];
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.x[0] = reinterpret_cast<const uint4*>(p)[0];
  r.x[1] = reinterpret_cast<const uint4*>(p)[1];
}
__device__ __forceinline__ void load2(const float* p, Raw<float>& r) {
  r.k[0] = p[0];
  r.k[1] = p[1];
}
__device__ __forceinline__ void load2(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.k = *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = r.x[i];
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w[4] = {r.x[k].x, r.x[k].y, r.x[k].z, r.x[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
      x[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float2 pair_of(const Raw<float>& r) { return make_float2(r.k[0], r.k[1]); }
__device__ __forceinline__ float2 pair_of(const Raw<__nv_bfloat16>& r) {
  return make_float2(__uint_as_float(r.k << 16), __uint_as_float(r.k & 0xffff0000u));
}

__device__ __forceinline__ void store2(float* p, float a, float b) {
  p[0] = a;
  p[1] = b;
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = sm100::pack_bf16x2(a, b);
}

// NaN-keeping maximum of magnitudes.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// One block in fp32; returns false when a rounding is too close to call.
__device__ __forceinline__ bool quantise_fast(const float (&x)[16], const float* g, float mul, uint32_t (&code)[2],
                                              uint32_t& s8) {
  float y[16], m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = x[i] * mul;
    if (g != nullptr) y[i] *= g[32 * i];
    m = max_abs(m, y[i]);
  }
  const float q = m * (1.f / 6.f);
  const uint32_t s2 = fp4::to_scales(q - q * kDelta, q + q * kDelta);
  s8 = s2 & 0xffu;
  bool ok = s8 == (s2 >> 8);
  const float s = fp4::scale_value(s8);
  const float inv = s > 0.f ? 1.f / s : 0.f;  // a zero or NaN scale: all codes zero
  code[0] = code[1] = 0u;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float a = y[i] * inv, b = y[i + 1] * inv;
    const uint32_t lo = fp4::to_codes(a - a * kDelta, b - b * kDelta);
    ok &= lo == fp4::to_codes(a + a * kDelta, b + b * kDelta);
    code[i >> 3] |= lo << (4 * (i & 7));
  }
  return ok;
}

// The blocks of a row whose bits are set in `redo` (bit l of word k: block l + 32 k), in fp64, 16 lanes to a block.
template <typename T, int NB>
__device__ __noinline__ void quantise_exact(const AppendFp4Args& a, const T* row, const uint32_t (&redo)[NB], uint8_t* c_dst,
                                            uint8_t* s_dst) {
  const int lane = threadIdx.x & 31, e = lane & 15;
  double s64 = 0.0;
  for (int f = lane; f < a.d_c; f += 32) {
    const double v = (double)to_f32(row[f]);
    s64 = fma(v, v, s64);
  }
  const double mul = 1.0 / sqrt(warp_sum_f64(s64) / a.d_c + (double)a.eps), unscale = 1.0 / (double)a.latent_scale;
  for (int k = 0; k < NB; ++k)
    for (uint32_t left = redo[k]; left != 0u; left &= left - 1) {
      const int blk = 32 * k + __ffs(left) - 1, f = 16 * blk + e;
      double y = (double)to_f32(row[f]) * mul;
      if (a.gain != nullptr) y *= (double)a.gain[f];
      y *= unscale;
      double m = fabs(y);
      for (int o = 8; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool nan = __any_sync(0xffffffffu, y != y);
      const float q = nan ? nanf("") : to_odd(m / 6.0);
      const uint32_t s8 = fp4::to_scales(q, q) & 0xffu;
      const double s = (double)fp4::scale_value(s8), v = fabs(y);
      // a code counts the borders that |y| has passed; a tie goes to the even code.  Border times scale is exact.
      uint32_t code = 0u;
      if (s > 0.0) {  // (a zero or NaN scale: all codes zero)
        code = (v > 0.25 * s) + (v >= 0.75 * s) + (v > 1.25 * s) + (v >= 1.75 * s) + (v > 2.5 * s) + (v >= 3.5 * s) + (v > 5.0 * s);
        code |= y < 0.0 ? 8u : 0u;
      }
      const uint32_t high = __shfl_down_sync(0xffffffffu, code, 1);
      if (lane < 16 && (lane & 1) == 0) c_dst[8 * blk + lane / 2] = (uint8_t)(code | high << 4);
      if (lane == 0) s_dst[blk] = (uint8_t)s8;
    }
}

// Turns per position of each rotary pair, base^(-2j / d_r) / (2 pi), by the host: in the kernel the fp64
// logarithm and exponentials took longer than a token's rows.
struct RotaryTurns {
  double turn[kMaxPairs];
};

// NB blocks of 16 features and NB rotary pairs per lane.
template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 8 : 4) append_fp4_kernel(const __grid_constant__ AppendFp4Args a,
                                                              const __grid_constant__ RotaryTurns rot) {
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t n_rows = (uint32_t)a.B * (uint32_t)a.T, stride = gridDim.x * (kThreads / 32);
  const int blocks = a.d_c / fp4::kBlock;
  // the gains by lane and element: read from global memory for every token, 64 bytes apart, they took more L1
  // lookups than the rows, and in registers they cost a third of the resident warps
  __shared__ float gain[NB][16][32];
  if (a.gain != nullptr) {
    for (int f = threadIdx.x; f < a.d_c; f += kThreads) gain[f >> 9][f & 15][(f >> 4) & 31] = a.gain[f];
    __syncthreads();
  }
  // the next token's row and indices are on their way while a token is worked on.  Rows of padding are not read: a
  // padded batch would pay for them, and there may be no memory there.  (A sequence's first row is there, and does not
  // wait for the count: 32 single tokens 4.9 us instead of 5.1.)
  struct Token {
    Raw<T> raw[NB];
    const T* row;
    int b, i, pos, dst, n;
  };
  auto fetch = [&](uint32_t w, Token& t) {
    t.b = a.T == 1 ? (int)w : (int)(w / (uint32_t)a.T);
    t.i = (int)(w - (uint32_t)t.b * (uint32_t)a.T);
    t.pos = a.positions[t.b];
    t.dst = a.rows != nullptr ? a.rows[t.b] : t.pos;
    t.n = a.counts != nullptr ? a.counts[t.b] : a.T;
    t.row = static_cast<const T*>(a.kv_a) + t.b * a.lda_b + t.i * a.lda;
    if (t.i > 0 && (t.i >= t.n || t.n > a.T)) return;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int at = lane + 32 * k;
      if (at < blocks) load16(t.row + at * fp4::kBlock, t.raw[k]);
      if (at < a.d_r / 2) load2(t.row + a.d_c + 2 * at, t.raw[k]);
    }
  };
  Token next;
  const uint32_t first = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (first < n_rows) fetch(first, next);
  for (uint32_t w = first; w < n_rows; w += stride) {
    const Token t = next;
    if (n_rows - w > stride) fetch(w + stride, next);
    const int b = t.b, i = t.i;
    const int64_t pos = (int64_t)t.pos + i, dst = (int64_t)t.dst + i;
    if (t.n < 0 || t.n > a.T) {
      if (lane == 0 && i == 0) raise_error(a.err, MLA_ERR_LENGTH);
      continue;
    }
    if (i >= t.n) continue;
    if (t.pos < 0 || dst < 0 || dst >= a.n_max) {  // would land outside the cache: report, write nothing
      if (lane == 0) raise_error(a.err, MLA_ERR_INDEX);
      continue;
    }
    float x[NB][16];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NB; ++k)
      if (lane + 32 * k < blocks) {
        widen(t.raw[k], x[k]);
#pragma unroll
        for (int j = 0; j < 16; ++j) ss = fmaf(x[k][j], x[k][j], ss);
      }
    ss = warp_sum(ss);
    const float inv = rsqrtf(ss / (float)a.d_c + a.eps) * (1.f / a.latent_scale);
    uint32_t code[NB][2], s8[NB];
    const bool safe = ss > 1e-30f && ss < 1e36f;
    uint8_t* c_dst = a.c4 + b * a.c4_b + dst * a.c4_r;
    uint8_t* s_dst = a.sc + b * a.sc_b + dst * a.sc_r;
    uint32_t redo[NB], any = 0u;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int blk = lane + 32 * k;
      bool ok = true;
      if (blk < blocks) {
        ok = quantise_fast(x[k], a.gain != nullptr ? &gain[k][0][lane] : nullptr, inv, code[k], s8[k]) && safe;
        if (ok) {
          if constexpr (sizeof(T) == 2) {  // bf16 caches are 16-byte aligned
            *reinterpret_cast<uint2*>(c_dst + 8 * blk) = make_uint2(code[k][0], code[k][1]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c_dst[8 * blk + j] = (uint8_t)(code[k][j >> 2] >> (8 * (j & 3)));
          }
          s_dst[blk] = (uint8_t)s8[k];
        }
      }
      redo[k] = __ballot_sync(0xffffffffu, !ok);
      any |= redo[k];
    }
    if (any != 0u) quantise_exact<T, NB>(a, t.row, redo, c_dst, s_dst);
    // rotary key: the angle in turns, reduced in fp64 (at position 65535 an fp32 product is off by
    // 4e-3 rad), then sin and cos of at most half a turn in fp32
    T* k_dst = static_cast<T*>(a.k_r) + b * a.kr_b + dst * a.kr_r;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int j = lane + 32 * k;
      if (j >= a.d_r / 2) continue;
      const double turns = (double)pos * rot.turn[j];
      const float2 y = pair_of(t.raw[k]);
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      store2(k_dst + 2 * j, y.x * c - y.y * s, y.x * s + y.y * c);
    }
  }
}

// Read-back: one thread per block of 16 features; rows past counts[b] come back as zeros.
template <typename T>
__global__ void __launch_bounds__(256) read_fp4_kernel(ReadFp4Args a) {
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int blocks = a.d_c / fp4::kBlock;
  const int64_t total = (int64_t)a.B * a.n * blocks;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
    const int blk = (int)(u % blocks);
    const int64_t r = u / blocks;
    const int b = (int)(r / a.n), i = (int)(r % a.n);
    const int n = a.counts != nullptr ? a.counts[b] : a.n;
    const int64_t src = (a.first != nullptr ? a.first[b] : 0) + (int64_t)i;
    bool live = i < n;
    if (n < 0 || n > a.n) {
      if (blk == 0 && i == 0) raise_error(a.err, MLA_ERR_LENGTH);
      live = false;
    } else if (live && (src < 0 || src >= a.n_max)) {
      if (blk == 0) raise_error(a.err, MLA_ERR_INDEX);
      live = false;
    }
    uint32_t w[2] = {0u, 0u};
    float s = 0.f;
    if (live) {
      const uint8_t* c = a.c4 + b * a.c4_b + src * a.c4_r + 8 * blk;
      if constexpr (sizeof(T) == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(c);
        w[0] = v.x;
        w[1] = v.y;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)c[j] << (8 * (j & 3));
      }
      s = fp4::scale_value(a.sc[b * a.sc_b + src * a.sc_r + blk]) * a.latent_scale;
    }
    float v[16];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t h[4];
      fp4::codes_to_f16(w[k], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = sm100::unpack_f16x2(h[j]);
        v[8 * k + 2 * j] = f.x * s;
        v[8 * k + 2 * j + 1] = f.y * s;
      }
    }
    T* o = static_cast<T*>(a.out) + b * a.out_b + i * a.out_r + blk * fp4::kBlock;
    if constexpr (sizeof(T) == 2) {
      uint32_t p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = sm100::pack_bf16x2(v[2 * j], v[2 * j + 1]);
      reinterpret_cast<uint4*>(o)[0] = make_uint4(p[0], p[1], p[2], p[3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(p[4], p[5], p[6], p[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = v[j];
    }
  }
}

}  // namespace

template <typename T>
cudaError_t cache_append_fp4_launch(const AppendFp4Args& a, cudaStream_t st) {
  // the last table made by this thread: a program appends with one base and width
  static thread_local float base = 0.f;
  static thread_local int d_r = 0;
  static thread_local RotaryTurns rot;
  if (base != a.rope_base || d_r != a.d_r) {
    for (int j = 0; j < kMaxPairs; ++j)
      rot.turn[j] = exp(-(2.0 * j / a.d_r) * log((double)a.rope_base)) * 0.15915494309189533577;  // 1 / (2 pi)
    base = a.rope_base;
    d_r = a.d_r;
  }
  const int64_t ctas = ((int64_t)a.B * a.T + kThreads / 32 - 1) / (kThreads / 32), most = 8 * sm_count();
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  // the usual widths leave a lane one block and one pair, and half the registers of two
  if (a.d_c <= 512 && a.d_r <= 64) return launch_pdl(append_fp4_kernel<T, 1>, grid, dim3(kThreads), 0, st, a, rot);
  return launch_pdl(append_fp4_kernel<T, 2>, grid, dim3(kThreads), 0, st, a, rot);
}

template <typename T>
cudaError_t cache_read_fp4_launch(const ReadFp4Args& a, cudaStream_t st) {
  const int64_t ctas = ((int64_t)a.B * a.n * (a.d_c / fp4::kBlock) + 255) / 256;
  const int64_t most = 8 * sm_count();
  return launch_pdl(read_fp4_kernel<T>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(256), 0, st, a);
}

template cudaError_t cache_append_fp4_launch<float>(const AppendFp4Args&, cudaStream_t);
template cudaError_t cache_append_fp4_launch<__nv_bfloat16>(const AppendFp4Args&, cudaStream_t);
template cudaError_t cache_read_fp4_launch<float>(const ReadFp4Args&, cudaStream_t);
template cudaError_t cache_read_fp4_launch<__nv_bfloat16>(const ReadFp4Args&, cudaStream_t);

}  // namespace mla
