// cache_evict.cu -- eviction from a KV cache by accumulated attention weight: per (batch, kv head)
// the `keep` keys of the largest weight among all but the last `recent`, and those, copied in the
// order of their positions to the front of another cache.
//
// Two kernels.  select: a CTA per (batch, kv head) finds the keep-th largest weight by radix
// selection over the weights' ordered bits and numbers the kept keys in order; among keys that
// equal the threshold the lowest positions are taken.  Caches of up to 32768 keys: the weights are
// read once into registers, three passes of 11, 11 and 10 bits over them (histograms in shared memory;
// a warp whose keys all fall in one bin adds once, so equal weights do not serialise), and one
// scan over the 32-key groups' counts.  Longer ones: four passes of 8 bits over the weights in L2, then
// a walk with a scan per 1024 keys.  gather: all SMs copy the rows, 16 bytes per thread and step; it
// is launched while select runs and waits for it inside.
// 8 x 8 heads, 16k-32k keys to 4096: select 44 us with the second form, REPL_SEL with the first; gather
// REPL_GAT for 236 MB.
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

// Exclusive prefix sum over the CTA; total: the whole sum.
__device__ __forceinline__ uint32_t scan_all(uint32_t v, uint32_t* s_warp, uint32_t& total) {
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

// Up to E * 1024 keys: key i * 1024 + tid in register i of thread tid.
template <int E>
__global__ void __launch_bounds__(kThreads) select_reg_kernel(const EvictParams p) {
  __shared__ uint32_t s_hist[2048];
  __shared__ uint32_t s_warp[33];
  __shared__ uint32_t s_pick[2];
  __shared__ uint32_t s_take[E * 32], s_eq[E * 32];  // per 32 keys, in order
  dependents_launch();
  const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = cache_len(p.cache_seqlens, b, p.Nk, p.status, bh % p.Hkv == 0 && tid == 0);
  const int left = min(L, p.M);
  const float* w = p.w + static_cast<size_t>(bh) * p.Nk;
  int32_t* index = p.index + static_cast<size_t>(bh) * p.M;
  float* w_out = p.w_out + static_cast<size_t>(bh) * p.cap;
  if (bh % p.Hkv == 0 && tid == 0) p.out_seqlens[b] = left;
  const int n = L <= p.M ? 0 : L - p.recent;  // the candidates
  float x[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int j = i * kThreads + tid;
    x[i] = j < L ? w[j] : 0.f;
  }
  uint32_t prefix = 0, want = p.keep;
  if (n > 0 && p.keep > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1024 : 2048, known = pass == 0 ? 0u : 0xffffffffu << (shift + (pass == 2 ? 10 : 11));
      s_hist[tid] = 0;
      s_hist[tid + 1024] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i * kThreads >= n) break;
        const uint32_t u = ordered(x[i]);
        const bool in = i * kThreads + tid < n && (u & known) == prefix;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (!who) continue;
        const uint32_t bin = (u >> shift) & (bins - 1);
        const uint32_t first = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !in || bin == first)) {
          if (lane == 0) atomicAdd(&s_hist[first], static_cast<uint32_t>(__popc(who)));
        } else if (in) {
          atomicAdd(&s_hist[bin], 1u);
        }
      }
      __syncthreads();
      // bins from the top, two a thread: the one that holds the want-th largest
      const uint32_t c0 = 2 * tid < bins ? s_hist[bins - 1 - 2 * tid] : 0, c1 = 2 * tid < bins ? s_hist[bins - 2 - 2 * tid] : 0;
      uint32_t total;
      const uint32_t above = scan_all(c0 + c1, s_warp, total);
      if (above < want && above + c0 + c1 >= want) {
        const bool second = above + c0 < want;
        s_pick[0] = bins - 1 - 2 * tid - (second ? 1 : 0);
        s_pick[1] = above + (second ? c0 : 0);
      }
      __syncthreads();
      prefix |= s_pick[0] << shift;
      want -= s_pick[1];
      __syncthreads();
    }
  }
  // the candidates above the threshold and the first `want` that equal it, numbered in order
  if (n > 0 && p.keep > 0) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool in = i * kThreads + tid < n;
      const uint32_t u = ordered(x[i]);
      const unsigned take = __ballot_sync(0xffffffffu, in && u > prefix), eq = __ballot_sync(0xffffffffu, in && u == prefix);
      if (lane == 0) {
        s_take[i * 32 + warp] = __popc(take);
        s_eq[i * 32 + warp] = __popc(eq);
      }
    }
    __syncthreads();
    // E * 32 groups of 32 keys: at most one per thread
    uint32_t total;
    const bool has = tid < E * 32;
    const uint32_t t0 = scan_all(has ? s_take[has ? tid : 0] : 0, s_warp, total);
    const uint32_t e0 = scan_all(has ? s_eq[has ? tid : 0] : 0, s_warp, total);
    if (has) {
      s_take[tid] = t0;
      s_eq[tid] = e0;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int j = i * kThreads + tid;
      const uint32_t u = ordered(x[i]);
      const bool over = j < n && u > prefix, same = j < n && u == prefix;
      const unsigned take = __ballot_sync(0xffffffffu, over), eq = __ballot_sync(0xffffffffu, same);
      const uint32_t eq_before = s_eq[i * 32 + warp] + __popc(eq & below);
      if (over || (same && eq_before < want)) {
        const uint32_t at = s_take[i * 32 + warp] + __popc(take & below) + min(eq_before, want);
        index[at] = j;
        w_out[at] = x[i];
      }
    }
  }
  // behind them the last keys: all of them from n on
  const int base = n > 0 ? p.keep : 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int j = i * kThreads + tid;
    if (j >= n && j < L) {
      index[base + j - n] = j;
      w_out[base + j - n] = x[i];
    }
  }
  for (int i = left + tid; i < p.M; i += kThreads) index[i] = -1;
  for (int i = left + tid; i < p.cap; i += kThreads) w_out[i] = 0.f;
}

// 16-byte chunks of the kept rows, keys and values, four per thread.
constexpr int kGather = 256 * 4;
__global__ void __launch_bounds__(256) gather_kernel(const EvictParams p, int ctas_per_bh) {
  const int chunks = p.row_bytes / 16;
  const int bh = blockIdx.x / ctas_per_bh;
  const long long first = static_cast<long long>(blockIdx.x % ctas_per_bh) * kGather + threadIdx.x, n = static_cast<long long>(p.M) * chunks;
  const uint4* const k = static_cast<const uint4*>(p.k) + static_cast<size_t>(bh) * p.Nk * chunks;
  const uint4* const v = static_cast<const uint4*>(p.v) + static_cast<size_t>(bh) * p.Nk * chunks;
  uint4* const ko = static_cast<uint4*>(p.k_out) + static_cast<size_t>(bh) * p.cap * chunks;
  uint4* const vo = static_cast<uint4*>(p.v_out) + static_cast<size_t>(bh) * p.cap * chunks;
  dependency_wait();
  long long src[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const long long i = first + u * 256;
    const int row = i < n ? static_cast<int>(i / chunks) : 0;
    const int j = i < n ? p.index[static_cast<size_t>(bh) * p.M + row] : -1;
    src[u] = j < 0 ? -1 : static_cast<long long>(j) * chunks + static_cast<int>(i - static_cast<long long>(row) * chunks);
  }
  uint4 a[4], b[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (src[u] >= 0) {
      a[u] = k[src[u]];
      b[u] = v[src[u]];
    }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (src[u] >= 0) {
      ko[first + u * 256] = a[u];
      vo[first + u * 256] = b[u];
    }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t stream) {
  const int bhs = p.B * p.Hkv;
  if (p.Nk <= 2 * kThreads) select_reg_kernel<2><<<bhs, kThreads, 0, stream>>>(p);
  else if (p.Nk <= 8 * kThreads) select_reg_kernel<8><<<bhs, kThreads, 0, stream>>>(p);
  else if (p.Nk <= 32 * kThreads) select_reg_kernel<32><<<bhs, kThreads, 0, stream>>>(p);
  else select_kernel<<<bhs, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per_bh = static_cast<int>((static_cast<long long>(p.M) * (p.row_bytes / 16) + kGather - 1) / kGather);
  return launch_dependent(gather_kernel, dim3(static_cast<unsigned>(bhs) * per_bh), 256, stream, p, per_bh);
}

}  // namespace attn
