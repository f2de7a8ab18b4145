// cache_weights.cu -- the attention weight that each cached key receives, added up over queries, for
// float32 (fp16 and bf16 run on the tensor cores, cache_weights_tc.cu):
//   w_out[j] = w_in[j] + sum_r exp(scale Q_r . K_j - LSE_r) over the rows r = (head, query) of the
//   key's kv head that see it.
//
// CUDA-core kernel: a CTA of 256 threads owns 64 keys of one (batch, kv head), staged transposed
// ([d][64 + 4], fp32) in shared memory, and walks the rows in tiles of 64; a thread forms a 4 x 4
// block of scores and keeps four keys' sums in registers, reduced over the 16 threads of a row at
// the end.  No atomics: the order of the sum is fixed.  8 x 8 heads of 16k-32k keys, 4 rows: 1160 us for 128 of
// bytes (60 of the 64 rows of its tile are padding, and the staging's stores meet four to a bank); 4 x 8
// heads of 4k-8k keys, 192 rows: 391 us, 26 TFLOP/s.
#include <algorithm>
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kTile = 64, kPad = kTile + 4;

__device__ __forceinline__ void stage(float* dst, const float* src, int rows, int d) {
  for (int i = threadIdx.x; i < kTile * d; i += 256) {
    const int r = i / d, c = i % d;
    dst[c * kPad + r] = r < rows ? src[static_cast<size_t>(r) * d + c] : 0.f;
  }
}

__global__ void __launch_bounds__(256) weights_f32_kernel(const WeightParams p, int key_tiles) {
  extern __shared__ __align__(16) float smem[];
  float* sK = smem;
  float* sQ = smem + p.d * kPad;
  __shared__ float s_nl[kTile];   // -LSE log2(e); -inf: the row adds nothing
  __shared__ int s_last[kTile];   // the last key the row sees
  const int bh = blockIdx.x / key_tiles, key0 = (blockIdx.x % key_tiles) * kTile;
  const int b = bh / p.Hkv, tid = threadIdx.x;
  const int L = cache_len(p.cache_seqlens, b, p.Nk, p.status, tid == 0 && key0 == 0 && bh % p.Hkv == 0);
  const int tk = tid & 15, tr = tid >> 4;  // keys 4 tk .. + 3, rows 4 tr .. + 3
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (key0 < L) {
    stage(sK, static_cast<const float*>(p.k) + (static_cast<size_t>(bh) * p.Nk + key0) * p.d, min(kTile, L - key0), p.d);
    for (int r0 = 0; r0 < p.R; r0 += kTile) {
      // under the causal mask a tile of rows within one head may end before this key
      const int r1 = min(r0 + kTile, p.R) - 1;
      if (p.causal && r0 / p.Nq == r1 / p.Nq && L - p.Nq + r1 % p.Nq < key0) continue;
      __syncthreads();
      stage(sQ, static_cast<const float*>(p.q) + (static_cast<size_t>(bh) * p.R + r0) * p.d, min(kTile, p.R - r0), p.d);
      if (tid < kTile) {
        const int r = r0 + tid;
        s_nl[tid] = r < p.R ? -p.lse[static_cast<size_t>(bh) * p.R + r] * 1.4426950408889634f : -INFINITY;
        if (s_nl[tid] == INFINITY) s_nl[tid] = -INFINITY;  // LSE -inf: no key
        s_last[tid] = r < p.R ? (p.causal ? min(L - p.Nq + r % p.Nq, L - 1) : L - 1) : -1;
      }
      __syncthreads();
      float s[4][4] = {};
      for (int c = 0; c < p.d; ++c) {
        const float4 k = *reinterpret_cast<const float4*>(sK + c * kPad + tk * 4);
        const float4 q = *reinterpret_cast<const float4*>(sQ + c * kPad + tr * 4);
        const float kk[4] = {k.x, k.y, k.z, k.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[a][e] = fmaf(kk[a], qq[e], s[a][e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float nl = s_nl[tr * 4 + e];
        const int last = s_last[tr * 4 + e];
#pragma unroll
        for (int a = 0; a < 4; ++a)
          if (nl != -INFINITY && key0 + tk * 4 + a <= last) acc[a] += exp2f(fmaf(s[a][e], p.scale_log2, nl));
      }
    }
  }
  __syncthreads();
  float* red = sQ;  // [16][64]
#pragma unroll
  for (int a = 0; a < 4; ++a) red[tr * kTile + tk * 4 + a] = acc[a];
  __syncthreads();
  if (tid < kTile && key0 + tid < p.Nk) {
    float sum = 0.f;
    for (int i = 0; i < 16; ++i) sum += red[i * kTile + tid];
    const size_t at = static_cast<size_t>(bh) * p.Nk + key0 + tid;
    p.w_out[at] = (p.w_in ? p.w_in[at] : 0.f) + (key0 + tid < L ? sum : 0.f);
  }
}

}  // namespace

cudaError_t launch_cache_weights_f32(const WeightParams& p, cudaStream_t stream) {
  const int key_tiles = (p.Nk + kTile - 1) / kTile;
  const int bytes = std::max(2 * p.d, p.d + 16) * kPad * 4;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(weights_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 128 * kPad * 4);
  });
  if (e != cudaSuccess) return e;
  weights_f32_kernel<<<p.B * p.Hkv * key_tiles, 256, bytes, stream>>>(p, key_tiles);
  return cudaGetLastError();
}

}  // namespace attn
