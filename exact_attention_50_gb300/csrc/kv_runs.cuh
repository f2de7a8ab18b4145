// kv_runs.cuh -- attention of few query rows over caches of different lengths: dealing the work, joining it.
//
// The caches are cut into tiles of p.tile_keys keys, and all tiles of all (batch, kv head) pairs, one after the other,
// are dealt in equal runs to the workers, whatever the sequences' lengths.  A run may begin and end inside a
// pair: such parts go to the workspace, normalised with their log-sum-exp, and a second kernel merges them.
// P is the caller's parameter struct (Cache8Params, PagedParams): the sizes, lengths, outputs and parts of the same names.
#pragma once
#include <algorithm>
#include <type_traits>
#include "cache8.cuh"

namespace attn {

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack2(const __half*, float a, float b) { return pack_half(a, b); }
__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Batch b's tiles per kv head.
template <typename P>
__device__ __forceinline__ int tiles_of(const P& p, int b) {
  return (cache_len(p.cache_seqlens, b, p.Nk, nullptr, false) + p.tile_keys - 1) / p.tile_keys;
}

// The runs: all tiles of all (batch, kv head) pairs in one numbering, the first total % runs runs one
// tile longer than the others; runs without a tile come last.
struct Deal {
  int total, base, rest;
  __device__ __forceinline__ void set(int tiles, int runs) {
    total = tiles;
    base = tiles / runs;
    rest = tiles % runs;
  }
  __device__ __forceinline__ int start(int run) const { return run * base + min(run, rest); }
  __device__ __forceinline__ int holder(int tile) const {  // the run that holds a tile
    const int longer = rest * (base + 1);
    return tile < longer ? tile / (base + 1) : rest + (tile - longer) / base;
  }
};

// Walks the parts of (batch, kv head) pairs that tiles [t, end) cover.
struct Walk {
  int t, end;    // the next tile and the end
  int b, h, nt;  // the pair that holds tile t, its tiles
  int j;         // tile t's number within the pair
  __device__ __forceinline__ int part() const { return min(end - t, nt - j); }  // tiles of this pair within the run
  template <typename P>
  __device__ __forceinline__ void next(const P& p) {
    t += part();
    j = 0;
    if (t >= end) return;
    if (++h == p.Hkv) {
      h = 0;
      do {
        ++b;
        nt = b < p.B ? tiles_of(p, b) : 1;
      } while (nt == 0);
      if (b >= p.B) t = end;  // not reached
    }
  }
};

// The deal, and the walk of one run; whole warps call it. The lengths are read by 32 lanes at a
// time: once for up to 32 batches, twice for more.
template <typename P>
__device__ __forceinline__ void deal_and_find(const P& p, int runs, int run, Deal& deal, Walk& w) {
  const int lane = threadIdx.x & 31;
  auto scan = [&](int b0, int& mine) {  // inclusive sum of the tiles of batches b0 .. b0 + lane
    mine = b0 + lane < p.B ? tiles_of(p, b0 + lane) : 0;
    int x = mine * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  int mine, x = scan(0, mine);
  int total = __shfl_sync(0xffffffffu, x, 31);
  for (int b0 = 32; b0 < p.B; b0 += 32) {
    int m2;
    total += __shfl_sync(0xffffffffu, scan(b0, m2), 31);
  }
  deal.set(total, runs);
  w.t = deal.start(run);
  w.end = deal.start(run + 1);
  w.b = w.h = w.nt = w.j = 0;
  if (w.t >= w.end) return;
  int off = 0;  // tiles before the 32 batches at b0
  for (int b0 = 0;;) {
    const unsigned hit = __ballot_sync(0xffffffffu, off + x > w.t);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int before = off + __shfl_sync(0xffffffffu, x - mine * p.Hkv, src);
      w.nt = __shfl_sync(0xffffffffu, mine, src);
      w.b = b0 + src;
      w.h = (w.t - before) / w.nt;
      w.j = (w.t - before) % w.nt;
      return;
    }
    off += __shfl_sync(0xffffffffu, x, 31);
    b0 += 32;
    if (b0 >= p.B) {  // not reached: tile t is below the total
      w.end = w.t;
      return;
    }
    x = scan(b0, mine);
  }
}

// Merges the parts of the pairs that several runs share.  A row is one warp's (W = 1) or a CTA's
// eight warps' (W = 8), each taking every W-th part, kAhead at a time.
template <typename OutT, int W, int kAhead, typename P>
__global__ void __launch_bounds__(256) runs_merge_kernel(const P p) {
  __shared__ float4 s_o[8][32];
  __shared__ float2 s_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = W == 8 ? blockIdx.x : static_cast<long long>(blockIdx.x) * 8 + warp;
  dependency_wait();
  if (row >= static_cast<long long>(p.B) * p.Hkv * p.R) return;
  const int bh = static_cast<int>(row / p.R), r = static_cast<int>(row % p.R);
  const int2 parts = p.parts[bh];
  // none, or (left by a run that ended with an error status) anything
  if (parts.y <= 0 || parts.x < 0 || parts.x >= p.runs || parts.y > p.runs - parts.x) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = W == 8 ? warp : 0; k0 < parts.y; k0 += kAhead * W) {
    float e[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u * W;
      const bool in = k < parts.y;
      // the first run's part ends inside the pair, the others' begin there
      const size_t at = (static_cast<size_t>(parts.x + k) * 2 + (k == 0 ? 1 : 0)) * p.R + r;
      e[u] = in ? p.lse_part[at] : -INFINITY;
      x[u] = in && lane * 4 < p.d ? *reinterpret_cast<const float4*>(p.o_part + at * p.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) top = fmaxf(top, e[u]);
    const float a = m == top ? 1.f : ex2_approx(m - top);  // m = -inf: 0
    acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
    l *= a;
    m = top;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      // a NaN part stays; an empty one (no key that the row sees) has no weight
      const float b = e[u] == -INFINITY ? 0.f : ex2_approx(e[u] - top);
      acc.x += x[u].x * b;
      acc.y += x[u].y * b;
      acc.z += x[u].z * b;
      acc.w += x[u].w * b;
      l += b;
    }
  }
  if (W == 8) {
    s_o[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
    m = -INFINITY;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = fmaxf(m, s_ml[u].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float b = s_ml[u].x == -INFINITY ? 0.f : ex2_approx(s_ml[u].x - m);
      const float4 x = s_o[u][lane];
      acc.x += x.x * b; acc.y += x.y * b; acc.z += x.z * b; acc.w += x.w * b;
      l += s_ml[u].y * b;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (lane * 4 < p.d) {
    if constexpr (std::is_same<OutT, float>::value) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * p.d + lane * 4) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
      const OutT* tag = nullptr;
      *reinterpret_cast<uint2*>(static_cast<OutT*>(p.o) + row * p.d + lane * 4) =
          make_uint2(pack2(tag, acc.x * inv, acc.y * inv), pack2(tag, acc.z * inv, acc.w * inv));
    }
  }
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

// A cache of capacity 0: O = 0, LSE = -inf for every row.
template <typename P>
__global__ void __launch_bounds__(256) runs_none_kernel(const P p) {
  const size_t rows = static_cast<size_t>(p.B) * p.Hkv * p.R, n16 = rows * p.d * (p.out_f32 ? 4 : 2) / 16;
  const size_t first = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = first; i < n16; i += step) static_cast<uint4*>(p.o)[i] = make_uint4(0, 0, 0, 0);
  if (p.lse)
    for (size_t i = first; i < rows; i += step) p.lse[i] = -INFINITY;
  if (first < static_cast<size_t>(p.B)) cache_len(p.cache_seqlens, static_cast<int>(first), p.Nk, p.status, true);
}

// By the parts that a pair has on average: 228 of them (1 x 8 heads of 32k keys) a warp's share in two rounds
// of loads, 28 (8 x 8 heads) in one, a few for one warp; 16 loads ahead for those of 64 x 8 heads, 3 each,
// took 8 us more.
template <typename OutT, typename P>
cudaError_t launch_merge(const P& p, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(p.B) * p.Hkv, rows = pairs * p.R;
  if (p.runs < 8 * pairs) return launch_dependent(runs_merge_kernel<OutT, 1, 8, P>, dim3(static_cast<unsigned>((rows + 7) / 8)), 256, stream, p);
  if (p.runs < 64 * pairs) return launch_dependent(runs_merge_kernel<OutT, 8, 4, P>, dim3(static_cast<unsigned>(rows)), 256, stream, p);
  return launch_dependent(runs_merge_kernel<OutT, 8, 16, P>, dim3(static_cast<unsigned>(rows)), 256, stream, p);
}

template <typename P>
cudaError_t launch_none(const P& p, cudaStream_t stream) {
  const size_t work = std::max(static_cast<size_t>(p.B) * p.Hkv * p.R * p.d / 4, static_cast<size_t>(p.B));
  runs_none_kernel<<<static_cast<int>(std::min<size_t>((work + 255) / 256, 1u << 20)), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
