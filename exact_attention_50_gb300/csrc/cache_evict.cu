// cache_evict.cu -- eviction from a KV cache by accumulated attention weight: per (batch, kv head)
// the `keep` keys of the largest weight among all but the last `recent`, and those, copied in the
// order of their positions to the front of another cache.
//
// Two kernels.  select, per (batch, kv head), finds the keep-th largest weight by radix
// selection over the weights' ordered bits and numbers the kept keys in order; among keys that
// equal the threshold the lowest positions are taken.  A CTA -- with few pairs a cluster of up to eight,
// which add up their histograms through distributed shared memory -- reads the weights once into
// registers (32 a thread at most), makes three passes of 11, 11 and 10 bits (histograms in shared
// memory; a warp whose keys all fall in one bin adds once, so equal weights do not serialise), the
// later two over the list of the weights in the first one's bin, and one scan over the 32-key groups' counts.  Longer caches: four passes of 8 bits over the weights in L2, then
// a walk with a scan per 1024 keys.  gather: all SMs copy the rows, 16 bytes per thread and step; it
// is launched while select runs and waits for it inside.
// 8 x 8 heads, 16k-32k keys to 4096: select 44 us with the second form, 19 us with the first; gather 39
// us for 268 MB (6.9 TB/s, what a copy reaches).  Both kernels, 65536 keys each: 69 us; where the second form
// begins, with one key more, 135 us, 131072 keys 227, 262144 keys 403; 8 heads of 262144 keys 38 us, of one more 328.
#include <cooperative_groups.h>
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kThreads = 1024;

// Weights as unsigned integers in the same order: the addition makes -0 a 0 and every NaN the same
// positive one, which is above infinity.
__device__ __forceinline__ uint32_t ordered(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// The weight of its ordered bits, unless it is a zero or a NaN: those are read again, so that they are handed on as they
// were.  (Reading every kept weight again takes 2 us of 62 for 8 x 8 heads of 16k-32k keys.)
__device__ __forceinline__ float weight_of(uint32_t u, const float* w) {
  if (u == 0x80000000u || u == 0xffffffffu) return *w;
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

// Exclusive prefix sum over the CTA; total: the whole sum.  (Also of two counts in 16-bit halves, at most 1024 each.)
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
    const uint32_t r = scan_all((take ? 1u : 0u) | (eq ? 0x10000u : 0u), s_warp, total);
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

// A cluster of C CTAs per (batch, kv head), up to C * E * 1024 keys: CTA r has keys [r E 1024, (r + 1) E
// 1024), key i * 1024 + tid of them in register i of thread tid.
template <int E, int C>
__global__ void __launch_bounds__(kThreads) select_reg_kernel(const EvictParams p) {
  constexpr uint32_t kList = 2048;
  __shared__ uint32_t s_hist[2][2048];
  __shared__ uint32_t s_list[kList];  // the CTA's weights in the first pass's bin
  __shared__ uint32_t s_warp[33];
  __shared__ uint32_t s_pick[3], s_total[2];
  __shared__ uint32_t s_take[E * 32], s_eq[E * 32];            // masks of 32 keys, in order
  __shared__ uint32_t s_take_at[E * 32], s_eq_at[E * 32];      // and the counts before them
  dependents_launch();
  const int rank = C == 1 ? 0 : blockIdx.x % C;
  const int bh = blockIdx.x / C, b = bh / p.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = cache_len(p.cache_seqlens, b, p.Nk, p.status, bh % p.Hkv == 0 && rank == 0 && tid == 0);
  const int left = min(L, p.M);
  const float* w = p.w + static_cast<size_t>(bh) * p.Nk;
  int32_t* index = p.index + static_cast<size_t>(bh) * p.M;
  float* w_out = p.w_out + static_cast<size_t>(bh) * p.cap;
  if (bh % p.Hkv == 0 && rank == 0 && tid == 0) p.out_seqlens[b] = left;
  const int n = L <= p.M ? 0 : L - p.recent;  // the candidates
  const int key0 = rank * E * kThreads;
  auto everyone = [] {  // all CTAs of the cluster, their shared memory visible to each other
    if constexpr (C == 1) __syncthreads();
    else cooperative_groups::this_cluster().sync();
  };
  auto at_rank = [](uint32_t* x, int r) {
    if constexpr (C == 1) return x;
    else return cooperative_groups::this_cluster().map_shared_rank(x, r);
  };
  if (n > 0 && p.keep > 0) {
    uint32_t u[E];  // 0 for what is no candidate: below the bits of every weight
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int j = key0 + i * kThreads + tid;
      u[i] = j < n ? ordered(w[j]) : 0u;
    }
    s_hist[0][tid] = s_hist[0][tid + 1024] = 0;
    if (tid == 0) s_pick[2] = 0;
    __syncthreads();
    uint32_t prefix = 0, want = p.keep;  // the threshold's known leading bits; its rank among the keys that have them
    uint32_t held = 0;                   // the weights listed
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1024 : 2048;
      uint32_t* const hist = s_hist[pass & 1];
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (key0 + i * kThreads >= n) break;
          const uint32_t bin = u[i] >> 21;
          // a warp of one bin (equal weights) adds once instead of 32 times in turn
          if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
            if (lane == 0) atomicAdd(&hist[bin], 32u);
          } else {
            atomicAdd(&hist[bin], 1u);
          }
        }
      } else if (held <= kList) {
        const uint32_t known = 0xffffffffu << (shift + (pass == 2 ? 10 : 11));
        for (uint32_t i = tid; i < (held + 31) / 32 * 32; i += kThreads) {  // whole warps
          const uint32_t x = i < held ? s_list[i] : 0u;
          const bool in = i < held && (x & known) == prefix;
          const uint32_t bin = (x >> shift) & (bins - 1);
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (!who) continue;
          const uint32_t one = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
          if (__all_sync(0xffffffffu, !in || bin == one)) {
            if (lane == 0) atomicAdd(&hist[one], static_cast<uint32_t>(__popc(who)));
          } else if (in) {
            atomicAdd(&hist[bin], 1u);
          }
        }
      } else {  // more weights in one bin than the list holds
        const uint32_t known = 0xffffffffu << (shift + (pass == 2 ? 10 : 11));
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const bool in = (u[i] & known) == prefix;
          const uint32_t bin = (u[i] >> shift) & (bins - 1);
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (!who) continue;
          const uint32_t one = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
          if (__all_sync(0xffffffffu, !in || bin == one)) {
            if (lane == 0) atomicAdd(&hist[one], static_cast<uint32_t>(__popc(who)));
          } else if (in) {
            atomicAdd(&hist[bin], 1u);
          }
        }
      }
      everyone();
      // bins from the top, two a thread: the one that holds the want-th largest
      uint32_t c0 = 0, c1 = 0;
      if (2 * tid < bins) {
#pragma unroll
        for (int r = 0; r < C; ++r) {
          const uint32_t* h = at_rank(hist, r);
          c0 += h[bins - 1 - 2 * tid];
          c1 += h[bins - 2 - 2 * tid];
        }
      }
      s_hist[(pass + 1) & 1][tid] = s_hist[(pass + 1) & 1][tid + 1024] = 0;  // read by nobody since the last pass
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
      if (pass == 0) {  // the later passes look at the weights of that bin alone
        const uint32_t bin = prefix >> 21;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const bool in = (u[i] >> 21) == bin;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (!who) continue;
          uint32_t at = 0;
          if (lane == 0) at = atomicAdd(&s_pick[2], static_cast<uint32_t>(__popc(who)));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
          if (in && at < kList) s_list[at] = u[i];
        }
      }
      __syncthreads();
      held = s_pick[2];
    }
    // the candidates above the threshold and the first `want` that equal it, numbered in order
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const unsigned take = __ballot_sync(0xffffffffu, u[i] > prefix), eq = __ballot_sync(0xffffffffu, u[i] == prefix);
      if (lane == 0) {
        s_take[i * 32 + warp] = take;
        s_eq[i * 32 + warp] = eq;
      }
    }
    __syncthreads();
    // E * 32 groups of 32 keys: at most one per thread
    uint32_t takes, eqs;
    const bool has = tid < E * 32;
    uint32_t t0 = scan_all(has ? __popc(s_take[has ? tid : 0]) : 0, s_warp, takes);
    uint32_t e0 = scan_all(has ? __popc(s_eq[has ? tid : 0]) : 0, s_warp, eqs);
    if constexpr (C > 1) {  // behind those of the CTAs before this one
      if (tid == 0) {
        s_total[0] = takes;
        s_total[1] = eqs;
      }
      everyone();
      for (int r = 0; r < rank; ++r) {
        const uint32_t* x = at_rank(s_total, r);
        t0 += x[0];
        e0 += x[1];
      }
    }
    if (has) {
      s_take_at[tid] = t0;
      s_eq_at[tid] = e0;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int group = i * 32 + warp;
      const bool over = u[i] > prefix, same = u[i] == prefix;
      if (!over && !same) continue;
      const uint32_t eq_before = s_eq_at[group] + __popc(s_eq[group] & below);
      if (same && eq_before >= want) continue;
      const uint32_t at = s_take_at[group] + __popc(s_take[group] & below) + min(eq_before, want);
      const int j = key0 + i * kThreads + tid;
      index[at] = j;
      w_out[at] = weight_of(u[i], w + j);
    }
  }
  // behind them the last keys: all of them from n on; then the fill
  const int base = n > 0 ? p.keep : 0, step = C * kThreads, first = rank * kThreads + tid;
  for (int j = n + first; j < L; j += step) {
    index[base + j - n] = j;
    w_out[base + j - n] = w[j];
  }
  for (int i = left + first; i < p.M; i += step) index[i] = -1;
  for (int i = left + first; i < p.cap; i += step) w_out[i] = 0.f;
  if constexpr (C > 1) everyone();  // the others may still read this CTA's totals
}

template <int E, int C>
cudaError_t run_select(const EvictParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_reg_kernel<E, C>, p);
}

template <int C>
cudaError_t select_c(const EvictParams& p, cudaStream_t stream) {
  const int e = (p.Nk + C * kThreads - 1) / (C * kThreads);
  return e <= 1 ? run_select<1, C>(p, stream) : e <= 4 ? run_select<4, C>(p, stream) : e <= 16 ? run_select<16, C>(p, stream) : run_select<32, C>(p, stream);
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
  // CTAs per (batch, kv head): as many as find an SM each and have four thousand keys (2048 keys took
  // a cluster of two 11 us, one CTA 7.5 us; 16k-32k keys two 19 us, one 26 us)
  int c = 1;
  while (c < 8 && bhs * 2 * c <= 152 && p.Nk > c * 4 * kThreads) c *= 2;
  cudaError_t e;
  if (p.Nk > c * 32 * kThreads) {
    select_kernel<<<bhs, kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
  } else {
    e = c == 1 ? select_c<1>(p, stream) : c == 2 ? select_c<2>(p, stream) : c == 4 ? select_c<4>(p, stream) : select_c<8>(p, stream);
  }
  if (e != cudaSuccess) return e;
  const int per_bh = static_cast<int>((static_cast<long long>(p.M) * (p.row_bytes / 16) + kGather - 1) / kGather);
  return launch_dependent(gather_kernel, dim3(static_cast<unsigned>(bhs) * per_bh), 256, stream, p, per_bh);
}

}  // namespace attn
