// cache8_wide.cu -- attention of many query rows over an 8-bit KV cache.
//
// CUDA-core kernel: a CTA of 128 threads owns one query row of a (batch, kv head) and walks the
// keys in tiles of 128, a thread per key for the scores, an online softmax over the tile, a thread
// per column for P V.  The key scale multiplies the score, the value scale the weight.
#include "cache8.cuh"

namespace attn {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, typename Code>
__global__ void __launch_bounds__(128) simple_kernel(const Cache8Params p) {
  __shared__ float s_q[128], s_p[128], s_red[4];
  const int bh = blockIdx.x / p.R, r = blockIdx.x % p.R, b = bh / p.Hkv, tid = threadIdx.x;
  const int L = cache_len(p.cache_seqlens, b, p.Nk, p.status, tid == 0 && r == 0 && bh % p.Hkv == 0);
  const int last = p.causal ? min(L - p.Nq + r % p.Nq, L - 1) : L - 1;
  const size_t row = static_cast<size_t>(bh) * p.R + r;
  if (tid < p.d) s_q[tid] = to_f<T>(static_cast<const T*>(p.q)[row * p.d + tid]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j0 = 0; j0 <= last; j0 += 128) {
    const int j = j0 + tid;
    float s = -INFINITY, vs = 0.f;
    if (j <= last) {
      const size_t at = static_cast<size_t>(bh) * p.n_blocks + (j >> p.block_shift);
      const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k8 + (static_cast<size_t>(bh) * p.Nk + j) * p.d);
      float dot = 0.f;
      for (int c = 0; c < p.d / 4; ++c) {
        float x[4];
        Code::decode4(k[c], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) dot = fmaf(x[i], s_q[4 * c + i], dot);
      }
      s = dot * p.k_scale[at] * p.scale_log2;
      vs = p.v_scale[at];
    }
    float mx = s;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float e = j <= last ? exp2f(s - mn) : 0.f;
    s_p[tid] = e == 0.f ? 0.f : e * vs;
    float sum = e;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    __syncthreads();
    if ((tid & 31) == 0) s_red[tid >> 5] = sum;
    __syncthreads();
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    l = l * alpha + (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
    m = mn;
    o *= alpha;
    const int n = min(128, last + 1 - j0);
    if (tid < p.d) {
      const uint8_t* v = p.v8 + (static_cast<size_t>(bh) * p.Nk + j0) * p.d + (tid & ~3);
      for (int i = 0; i < n; ++i) {
        float x[4];
        Code::decode4(*reinterpret_cast<const uint32_t*>(v + static_cast<size_t>(i) * p.d), x);
        o = fmaf(s_p[i], x[tid & 3], o);
      }
    }
    __syncthreads();
  }
  o = l > 0.f ? o / l : (l == 0.f ? 0.f : l);
  if (tid < p.d) {
    if (p.out_f32) static_cast<float*>(p.o)[row * p.d + tid] = o;
    else from_f(static_cast<T*>(p.o) + row * p.d + tid, o);
  }
  if (tid == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <typename T>
cudaError_t run(const Cache8Params& p, attn_cache_dtype_t cache, cudaStream_t stream) {
  const int grid = p.B * p.Hkv * p.R;
  if (cache == ATTN_CACHE_I8) simple_kernel<T, CodeI8><<<grid, 128, 0, stream>>>(p);
  else simple_kernel<T, CodeE4m3><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache8_wide(const Cache8Params& p, attn_dtype_t dtype, attn_cache_dtype_t cache, cudaStream_t stream) {
  return dtype == ATTN_F16 ? run<__half>(p, cache, stream) : run<__nv_bfloat16>(p, cache, stream);
}

}  // namespace attn
