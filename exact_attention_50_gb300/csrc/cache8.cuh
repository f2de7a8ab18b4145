// cache8.cuh -- the 8-bit cache codes shared by the kernels that write and read them.
#pragma once
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "kernels.h"
#include "ptx.cuh"

namespace attn {

// Code types: the largest magnitude a code stands for, float -> code (round to nearest even,
// within range) and code -> float (exact).
struct CodeI8 {
  static constexpr float kInvTop = 1.0f / 127.0f;
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    auto one = [](float x) { return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f))) & 0xffu; };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
};
struct CodeE4m3 {
  static constexpr float kInvTop = 1.0f / 448.0f;
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    uint32_t h0, h1;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
};

// Batch b's cache length; a length outside [0, Nk] counts as an empty cache (reported when the
// caller asks for it, once per batch).
__device__ __forceinline__ int cache_len(const int32_t* lens, int b, int Nk, unsigned* status, bool report) {
  if (!lens) return Nk;
  const int L = lens[b];
  if (L < 0 || L > Nk) {
    if (report) raise_status(status, ATTN_ERR_DEVICE_INPUT);
    return 0;
  }
  return L;
}

// Programmatic dependent launch: the first kernel lets the next one's CTAs start as soon as there is
// room; those wait, before they read its results, until all of it has completed.
__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}

// Runs `set_up` at the first call on each device (its result is not kept when it fails).
template <typename F>
cudaError_t once_per_device(std::atomic<unsigned long long>& ready, F set_up) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = set_up();
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace attn
