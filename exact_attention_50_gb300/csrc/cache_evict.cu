// cache_evict.cu -- eviction from a KV cache by accumulated attention weight: per (batch, kv head)
// the `keep` keys of the largest weight among all but the last `recent`, and those, copied in the
// order of their positions to the front of another cache.
//
// Two kernels. select: a CTA per (batch, kv head) finds the keep-th largest weight by radix
// selection over the weights' ordered bits (four passes of 8 bits, each a histogram in shared
// memory), then walks the keys once in order, numbering the kept ones with a block-wide scan;
// among keys that equal the threshold the lowest positions are taken.  gather: all SMs copy the
// rows, 16 bytes per thread.
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kThreads = 1024;

// Weights as unsigned integers in the same order; -0 counts as 0 and every NaN is the largest.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the CTA of two counts packed in 16-bit halves (each at most 1024).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const uint32_t w = s_warp[lane];
    uint32_t y = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y - w;
    if (lane == 31) s_warp[32] = y;
  }
  __syncthreads();
  const uint32_t r = s_warp[warp] + x - v;
  total = s_warp[32];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const EvictParams p) {
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_warp[33];
  __shared__ uint32_t s_pick[2];
  const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x;
  const int L = cache_len(p.cache_seqlens, b, p.Nk, p.status, bh % p.Hkv == 0 && tid == 0);
  const int left = min(L, p.M);
  const float* w = p.w + static_cast<size_t>(bh) * p.Nk;
  int32_t* index = p.index + static_cast<size_t>(bh) * p.M;
  float* w_out = p.w_out + static_cast<size_t>(bh) * p.cap;
  if (bh % p.Hkv == 0 && tid == 0) p.out_seqlens[b] = left;
  const int n = L <= p.M ? 0 : L - p.recent;  // the candidates
  uint32_t prefix = 0, want = p.keep;         // the threshold's known leading bits; its rank among the keys that have them
  if (n > 0 && p.keep > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = tid; j < n; j += kThreads) {
        const uint32_t u = ordered(w[j]);
        if ((u & mask) == prefix) atomicAdd(&s_hist[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      // the bin that holds the want-th largest: counts from the top
      if (tid < 32) {
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = s_hist[255 - (tid * 8 + i)];
          sum += c[i];
        }
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (tid >= o) x += y;
        }
        uint32_t above = x - sum;  // keys in larger bins
        if (above < want && x >= want) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (above < want && above + c[i] >= want) {
              s_pick[0] = 255 - (tid * 8 + i);
              s_pick[1] = above;
            }
            above += c[i];
          }
        }
      }
      __syncthreads();
      prefix |= s_pick[0] << shift;
      want -= s_pick[1];
      __syncthreads();
    }
  }
  // numbered in order: every key above the threshold, the first `want` that equal it, the recent
  uint32_t done = 0, equal = 0;
  for (int j0 = 0; j0 < L; j0 += kThreads) {
    const int j = j0 + tid;
    float x = 0.f;
    bool take = false, eq = false;
    if (j < L) {
      x = w[j];
      if (j >= n) {
        take = true;
      } else if (p.keep > 0) {
        const uint32_t u = ordered(x);
        take = u > prefix;
        eq = u == prefix;
      }
    }
    uint32_t total;
    const uint32_t r = block_scan((take ? 1u : 0u) | (eq ? 0x10000u : 0u), s_warp, total);
    // equals before this key in the whole sequence; of them, the first `want` are kept
    const uint32_t eq_before = equal + (r >> 16);
    if (eq && eq_before < want) take = true;
    if (take) {
      const uint32_t at = done + (r & 0xffffu) + (min(eq_before, want) - min(equal, want));
      index[at] = j;
      w_out[at] = x;
    }
    const uint32_t eq_end = equal + (total >> 16);
    done += (total & 0xffffu) + (min(eq_end, want) - min(equal, want));
    equal = eq_end;
  }
  for (int i = left + tid; i < p.M; i += kThreads) index[i] = -1;
  for (int i = left + tid; i < p.cap; i += kThreads) w_out[i] = 0.f;
}

// One thread per 16 bytes of a kept row, keys and values.
__global__ void __launch_bounds__(256) gather_kernel(const EvictParams p) {
  const int chunks = p.row_bytes / 16;
  const long long per_bh = static_cast<long long>(p.M) * chunks;
  const long long total = per_bh * p.B * p.Hkv;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<long long>(gridDim.x) * 256) {
    const long long bh = i / per_bh;
    const int rem = static_cast<int>((i % per_bh) / chunks), c = static_cast<int>(i % chunks);
    const int j = p.index[bh * p.M + rem];
    if (j < 0) continue;
    const size_t src = (static_cast<size_t>(bh) * p.Nk + j) * chunks + c, dst = (static_cast<size_t>(bh) * p.cap + rem) * chunks + c;
    const uint4 k = static_cast<const uint4*>(p.k)[src], v = static_cast<const uint4*>(p.v)[src];
    static_cast<uint4*>(p.k_out)[dst] = k;
    static_cast<uint4*>(p.v_out)[dst] = v;
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t stream) {
  const int bhs = p.B * p.Hkv;
  select_kernel<<<bhs, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long total = static_cast<long long>(bhs) * p.M * (p.row_bytes / 16);
  long long blocks = (total + 255) / 256;
  if (blocks > 152L * 32) blocks = 152L * 32;
  gather_kernel<<<static_cast<int>(blocks), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
