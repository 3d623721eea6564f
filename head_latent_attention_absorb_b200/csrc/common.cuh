// Shared helpers of the MLA CUDA library: element conversion, warp reductions, the device error
// flag and the argument blocks handed from the C-ABI layer to the kernel launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>

#include "mla_api.h"

namespace mla {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// First error wins: a later error never overwrites an earlier one.
__device__ __forceinline__ void raise_error(int32_t* flag, int32_t code) {
  if (flag != nullptr) atomicCAS(flag, 0, code);
}

// Whether a persistent decode launch may use the sliced merge, in which every cluster holding a
// piece of a sequence waits for all the others' partials.  That wait needs every cluster of the
// launch resident at once.  The launcher passes `one_wave` = the occupancy query confirmed that the
// whole grid fits on the GPU in one wave; MLA_DECODE_SLICED_MERGE=0 in the environment turns the
// sliced merge off as well, for GPUs whose SMs another context may hold for the length of a launch
// (MPS clients, another process's long-running kernel).  Without it the last cluster to arrive
// merges every partial, which waits only on clusters that have already run.
inline bool sliced_merge_allowed(bool one_wave) {
  const char* e = getenv("MLA_DECODE_SLICED_MERGE");
  return one_wave && !(e != nullptr && e[0] == '0' && e[1] == '\0');
}

// Validated arguments of one decode call (pointers already checked on the host).
struct DecodeArgs {
  int n_h, d_c, d_r, B, n_max, topk;
  int T = 1;  // new tokens per cache sequence: B query groups over B / T cache sequences
  const void* q_tilde; int64_t ldqt;
  const void* q_pe;    int64_t ldqp;
  const void* c_kv;    int64_t ckv_b, ckv_r;
  const void* k_r;     int64_t kr_b, kr_r;
  const int32_t* lengths;
  const int32_t* topk_idx;
  float scale;
  void* ctx;
  float* lse;
  int32_t* err;
  // FP8 latent cache (mla_decode_absorb_fp8kv): e4m3 rows replace c_kv; strides in bytes for c8 and
  // in floats for kv_scale (one fp32 scale per 128 latent features of a row)
  const void* c8 = nullptr;        int64_t c8_b = 0, c8_r = 0;
  const float* kv_scale = nullptr; int64_t sc_b = 0, sc_r = 0;
};

struct PrefillArgs {
  int n_h, d_c, d_r, d_h, d_v, B, S, causal;
  const void* q;
  const void* c_kv; int64_t ckv_r;
  const void* k_r;  int64_t kr_r;
  const void* w;
  float scale;
  void* out;
  void* kv;  // expanded [B, S, n_h, d_h + d_v] in the input dtype
};

// Validated arguments of one cache append (one new token per sequence).
struct AppendArgs {
  int d_c, d_r, B, n_max;
  const void* kv_a; int64_t lda;  // [B, d_c + d_r] rows: latent first, rotary key last
  const float* gain;              // [d_c] RMSNorm gain, or nullptr for ones
  float eps, rope_base;
  const int32_t* positions;       // [B] position of each new token
  const int32_t* rows = nullptr;  // [B] cache row of each new token, or nullptr: row = position
  void* c_kv; int64_t ckv_b, ckv_r;
  void* k_r;  int64_t kr_b, kr_r;
  int32_t* err;
};

// The caches an operator reads: latent rows in the element type (c_kv, strides in elements) or in
// 4 bits (c4 codes and sc scales, strides in bytes), and the rotary rows.
struct CacheView {
  const void* c_kv = nullptr;  int64_t ckv_b = 0, ckv_r = 0;
  const uint8_t* c4 = nullptr; int64_t c4_b = 0, c4_r = 0;
  const uint8_t* sc = nullptr; int64_t sc_b = 0, sc_r = 0;
  const void* k_r = nullptr;   int64_t kr_b = 0, kr_r = 0;
  float latent_scale = 1.f;    // 4-bit rows: value = code * scale * latent_scale (a power of two)
};

// Validated arguments of the 4-bit decode and of the attention-weight pass: T new tokens for each of
// B sequences, query rows ((b * T + s) * n_h + h).
struct QueryArgs {
  int n_h, d_c, d_r, B, T, n_max;
  const void* q_tilde; int64_t ldqt;
  const void* q_pe;    int64_t ldqp;
  CacheView kv;
  const int32_t* lengths;
  float scale;
  int32_t* err;
};
struct Fp4DecodeArgs : QueryArgs {
  void* ctx;
  float* lse;
};
struct WeightsArgs : QueryArgs {
  const float* lse;
  const float* acc; int64_t acc_b;  // nullptr: nothing accumulated so far
  float decay;
  float* out; int64_t out_b;
};

// Validated arguments of the 4-bit append (T tokens per sequence) and of the read-back.
struct AppendFp4Args {
  int d_c, d_r, B, T, n_max;
  const void* kv_a; int64_t lda_b, lda;
  const float* gain;
  float eps, rope_base, latent_scale;
  const int32_t* positions; const int32_t* rows; const int32_t* counts;
  uint8_t* c4; int64_t c4_b, c4_r;
  uint8_t* sc; int64_t sc_b, sc_r;
  void* k_r;   int64_t kr_b, kr_r;
  int32_t* err;
};
struct ReadFp4Args {
  int d_c, B, n, n_max;
  const int32_t* first; const int32_t* counts;
  const uint8_t* c4; int64_t c4_b, c4_r;
  const uint8_t* sc; int64_t sc_b, sc_r;
  float latent_scale;
  void* out; int64_t out_b, out_r;
  int32_t* err;
};

// Validated arguments of the eviction: row planes with strides in bytes.
struct EvictArgs {
  int B, n_max, n_planes, keep, sink, recent;
  mla_rows planes[MLA_MAX_PLANES];
  const float* acc; int64_t acc_b;
  const int32_t* lengths;
  int32_t* positions; int64_t pos_b;  // nullptr: the rows stand in order of age
  int32_t* new_lengths;
  int32_t* row_map;
  int32_t* err;
};

// The current device's index (below kMaxDevices) and multiprocessors, looked up once per device.
constexpr int kMaxDevices = 64;
inline int current_device() {
  int dev = 0;
  cudaGetDevice(&dev);
  return dev >= 0 && dev < kMaxDevices ? dev : 0;
}
// What is looked up once per device, in static storage (0: not yet).  Any thread may look it up, and all find the same, so
// the accesses need no order.
struct PerDevice {
  std::atomic<int> value[kMaxDevices];
  int get(int dev) const { return value[dev].load(std::memory_order_relaxed); }
  void set(int dev, int v) { value[dev].store(v, std::memory_order_relaxed); }
};
inline int sm_count() {
  static PerDevice cache;
  const int dev = current_device();
  int n = cache.get(dev);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cache.set(dev, n);
  }
  return n;
}
// Raises a kernel's dynamic shared memory limit, once per device; `allowed` is the kernel's own record.
inline cudaError_t allow_smem(const void* kernel, int bytes, PerDevice& allowed) {
  const int dev = current_device();
  if (allowed.get(dev) >= bytes) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed.set(dev, bytes);
  return e;
}

// Launch with programmatic stream serialization: the kernel may start while the preceding kernel
// in the stream is still running, and synchronises with it through griddepcontrol.wait before it
// touches that kernel's data (every kernel of this library does).
template <typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mla
