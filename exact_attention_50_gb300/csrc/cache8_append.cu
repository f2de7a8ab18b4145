// cache8_append.cu -- writes new tokens into an 8-bit KV cache: per block of tokens and head a
// scale s = max |x| / top (top = 127 or 448) and codes round(x / s).
//
// A CTA owns one touched block of one (batch, kv head) of keys or of values: it reads the block's
// new tokens once into registers (16 bytes per load, up to eight in flight per thread), reduces
// max |x|, and writes the codes.  HBM-bound: four prompts of 8k to 16k
// tokens, 317 MB, take 56 us, 83% of the copy rate (72 us when the tokens were read twice, the second
// time from L2); a decode step's single tokens 2.5 us.  The block at the cache's end may hold
// tokens already: its scale only grows, and when it does the codes there are recoded by the same CTA,
// so no other CTA ever touches them.  Every operation is one IEEE rounding (no contraction), so
// codes and scales are a function of the inputs alone.
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kVecs = 8;  // vectors of eight elements that a thread holds

// Eight consecutive elements as they lie in memory, and as floats.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <>
struct Vec8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x; x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// The bits of |x|: ordered like |x|, with infinity above every number and NaN above that.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <typename T, typename Code, int kThreads>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  __shared__ uint32_t s_max[kThreads / 32];
  const int per_bh = 2 * p.blocks_per_head;
  const int bh = blockIdx.x / per_bh;
  const int rem = blockIdx.x % per_bh;
  const int side = rem / p.blocks_per_head;  // 0: keys, 1: values
  const int b = bh / p.Hkv;
  const int L = p.cache_seqlens ? p.cache_seqlens[b] : 0;
  const int n = p.new_seqlens ? p.new_seqlens[b] : p.Nn;
  if (L < 0 || n < 0 || n > p.Nn || L > p.Nk - n) {
    if (rem == 0 && threadIdx.x == 0) raise_status(p.status, ATTN_ERR_DEVICE_INPUT);
    return;
  }
  const int blk = L / p.block + rem % p.blocks_per_head;
  const long long blk0 = static_cast<long long>(blk) * p.block;
  const int t0 = static_cast<int>(max(blk0, static_cast<long long>(L)));                       // new tokens [t0, t1)
  const int t1 = static_cast<int>(min(blk0 + p.block, static_cast<long long>(L) + n));
  if (t0 >= t1) return;
  const T* src = static_cast<const T*>(p.x_new[side]) + (static_cast<size_t>(bh) * p.Nn + (t0 - L)) * p.d;
  uint8_t* const head = p.x8[side] + static_cast<size_t>(bh) * p.Nk * p.d;
  float* const scale = p.scale[side] + static_cast<size_t>(bh) * p.n_blocks + blk;
  const int nvec = (t1 - t0) * p.d / 8;  // vectors of 8 elements: rows are contiguous on both sides
  // all of the block's new tokens at once: block * d <= 8 * kVecs * kThreads
  Vec8<T> raw[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int i = u * kThreads + threadIdx.x;
    if (i < nvec) raw[u].load(src + static_cast<size_t>(i) * 8);
  }
  uint32_t mx = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    if (u * kThreads + static_cast<int>(threadIdx.x) >= nvec) break;
    float x[8];
    raw[u].get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = max(mx, abs_bits(x[e]));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) mx = max(mx, s_max[w]);
  constexpr float kTiny = 1.17549435e-38f;  // 2^-126
  float s = __fmul_rn(__uint_as_float(mx), Code::kInvTop);
  if (s < kTiny) s = 0.f;
  const bool held = t0 > blk0;  // the block holds tokens already
  const float s_old = held ? *scale : 0.f;
  if (held && !(s_old <= s) && !(s != s)) s = s_old;  // larger, or NaN: it stays
  const float inv = s == 0.f ? 0.f : __frcp_rn(s);
  uint8_t* const dst = head + static_cast<size_t>(t0) * p.d;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int i = u * kThreads + threadIdx.x;
    if (i >= nvec) break;
    float x[8];
    raw[u].get(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], inv);
    reinterpret_cast<uint2*>(dst)[i] = make_uint2(Code::encode4(x[0], x[1], x[2], x[3]), Code::encode4(x[4], x[5], x[6], x[7]));
  }
  if (held && s > s_old) {
    const float f = __fmul_rn(s_old, inv);
    uint2* const old = reinterpret_cast<uint2*>(head + static_cast<size_t>(blk0) * p.d);
    const int nold = static_cast<int>(t0 - blk0) * p.d / 8;
    for (int i = threadIdx.x; i < nold; i += kThreads) {
      const uint2 w = old[i];
      float a[4], c[4];
      Code::decode4(w.x, a);
      Code::decode4(w.y, c);
      old[i] = make_uint2(Code::encode4(__fmul_rn(a[0], f), __fmul_rn(a[1], f), __fmul_rn(a[2], f), __fmul_rn(a[3], f)),
                          Code::encode4(__fmul_rn(c[0], f), __fmul_rn(c[1], f), __fmul_rn(c[2], f), __fmul_rn(c[3], f)));
    }
  }
  __syncthreads();  // every thread has read the old scale
  if (threadIdx.x == 0) *scale = s;
}

template <typename T>
cudaError_t run(const AppendParams& p, attn_cache_dtype_t cache, cudaStream_t stream) {
  const int grid = p.B * p.Hkv * 2 * p.blocks_per_head;
  const bool small = p.block * p.d <= 8 * kVecs * 128;
  if (cache == ATTN_CACHE_I8) {
    if (small) append_kernel<T, CodeI8, 128><<<grid, 128, 0, stream>>>(p);
    else append_kernel<T, CodeI8, 256><<<grid, 256, 0, stream>>>(p);
  } else {
    if (small) append_kernel<T, CodeE4m3, 128><<<grid, 128, 0, stream>>>(p);
    else append_kernel<T, CodeE4m3, 256><<<grid, 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache8_append(const AppendParams& p, attn_dtype_t dtype, attn_cache_dtype_t cache, cudaStream_t stream) {
  if (dtype == ATTN_F32) return run<float>(p, cache, stream);
  if (dtype == ATTN_F16) return run<__half>(p, cache, stream);
  return run<__nv_bfloat16>(p, cache, stream);
}

}  // namespace attn
