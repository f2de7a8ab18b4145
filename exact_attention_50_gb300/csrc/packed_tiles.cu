// packed_tiles.cu -- the list of tiles of packed sequences, heaviest first, for the forward and the backward of
// packed attention with grouped heads; and what lies behind the last sequence.
//
// The lengths are on the device, so the host knows only bounds.  A grid over (longest sequence, sequences) is mostly
// empty when the lengths differ: 1000 sequences of which one has 4096 tokens would be 97% items without a row.  The
// list holds the tiles that there are.  Under the causal mask a forward tile's cost grows with its number, a
// backward (key) tile's with its distance from the sequence's end; call that the tile's level, 0 .. n - 1 in a
// sequence of n tiles.  Level l holds one tile of each sequence longer than l, so with the sequences counted by n
// (one histogram, two suffix sums) every tile's place is known without a sort:
//   A[n] = sequences of more than n tiles,  first[l] = sum of A[l'] over l' > l,
//   place(level l of a sequence of n tiles, r-th of its length) = first[l] + A[n] + r.
// Without the mask all tiles of a sequence cost the same, and longer sequences come first:
//   place = sum of m over the sequences of m > n tiles (= first[n] + (n + 1) A[n]) + r n + l.
// Sequences of more than kLevels tiles take 2^shift tiles a level.  One CTA: 16 sequences 3 us, 1000 sequences 5 us.
#include <algorithm>
#include "kernels.h"
#include "ptx.cuh"
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kLevels = 2048, kThreads = 1024, kEach = kLevels / kThreads;

// In place: x[i] -> the sum of x[i'] over i' > i, for kLevels values.
__device__ __forceinline__ void suffix_sums(int* x, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = kLevels - 1 - kEach * static_cast<int>(threadIdx.x);  // this thread: i0, i0 - 1, ..
  int v[kEach], sum = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    v[k] = x[i0 - k];
    sum += v[k];
  }
  int y = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) s_warp[warp] = y;
  __syncthreads();
  int before = y - sum;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    x[i0 - k] = before;
    before += v[k];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) packed_tiles_kernel(const int32_t* __restrict__ cu, int nseq, int T, int max_seqlen, int tile, int shift,
                                                                int causal, int backward, int bound, int* head, int4* out, unsigned* status) {
  __shared__ int A[kLevels + 1], first[kLevels], seen[kLevels + 1];
  __shared__ int s_warp[32];
  dependents_launch();
  for (int i = threadIdx.x; i < kLevels; i += kThreads) A[i] = first[i] = seen[i] = 0;
  if (threadIdx.x == 0) A[kLevels] = seen[kLevels] = 0;
  __syncthreads();
  // the sequence's start and length (0: none, or not to be computed), and its levels
  const auto look = [&](int s, int& c0, bool report) -> int {
    c0 = cu[s];
    const int c1 = cu[s + 1];
    if (c0 < 0 || c1 < c0 || c1 > T || c1 - c0 > max_seqlen || (s == 0 && c0 != 0)) {
      if (report) raise_status(status, ATTN_ERR_DEVICE_INPUT);
      return 0;
    }
    return c1 - c0;
  };
  const auto levels_of = [&](int len) { return ((len + tile - 1) / tile + (1 << shift) - 1) >> shift; };
  // the histogram, n tiles at place n - 1: its suffix sum there is A[n]
  for (int s = threadIdx.x; s < nseq; s += kThreads) {
    int c0;
    const int n = levels_of(look(s, c0, true));
    if (n > 0) atomicAdd(first + n - 1, 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kLevels; i += kThreads) A[i + 1] = first[i];  // for now: sequences of i + 1 tiles
  __syncthreads();
  suffix_sums(first, s_warp);  // first[n - 1]: sequences of more than n tiles
  int keep[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int n = static_cast<int>(threadIdx.x) + k * kThreads;
    keep[k] = first[n] + A[n + 1];  // A of n: sequences of more than n tiles, n = 0 ..
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) A[threadIdx.x + k * kThreads] = first[threadIdx.x + k * kThreads] = keep[k];
  if (threadIdx.x == 0) A[kLevels] = 0;
  __syncthreads();
  suffix_sums(first, s_warp);
  const long long count = (static_cast<long long>(first[0]) + A[0]) << shift;
  const bool fits = count <= bound;  // always, when cu does not decrease
  if (threadIdx.x == 0) {
    const int end = cu[nseq];
    head[0] = fits ? static_cast<int>(count) : 0;
    head[1] = end >= 0 && end <= T ? end : T;
    if (!fits) raise_status(status, ATTN_ERR_DEVICE_INPUT);
  }
  if (!fits) return;
  const int lane = threadIdx.x & 31, sub = 1 << shift;
  const auto put = [&](int c0, int len, int n, int r, int at) {  // tile `at` (level at >> shift) of the r-th sequence of n levels
    const int l = at >> shift, in = at & (sub - 1);
    const int place = causal ? first[l] + A[n] + r : first[min(n, kLevels - 1)] + (n < kLevels ? (n + 1) * A[n] : 0) + r * n + l;
    // backward under the mask: key tiles in ascending order as the levels fall
    const bool turn = causal && backward;
    const int no = turn ? n * sub - 1 - at : at;
    const bool there = no < (len + tile - 1) / tile;
    out[static_cast<long long>(place) * sub + (turn ? sub - 1 - in : in)] = make_int4(c0, there ? len : 0, no, 0);
  };
  for (int s0 = threadIdx.x - lane; s0 < nseq; s0 += kThreads) {
    int c0 = 0, len = 0;
    if (s0 + lane < nseq) len = look(s0 + lane, c0, false);
    const int n = levels_of(len);
    int r = 0;
    if (n > 0) r = atomicAdd(seen + n, 1);
    const bool small = n * sub <= 8;
    if (small)
      for (int at = 0; at < n * sub; ++at) put(c0, len, n, r, at);
    for (unsigned big = __ballot_sync(0xffffffffu, !small); big; big &= big - 1) {
      const int src = __ffs(big) - 1;
      const int bc = __shfl_sync(0xffffffffu, c0, src), bl = __shfl_sync(0xffffffffu, len, src);
      const int bn = __shfl_sync(0xffffffffu, n, src), br = __shfl_sync(0xffffffffu, r, src);
      for (int at = lane; at < bn * sub; at += 32) put(bc, bl, bn, br, at);
    }
  }
}

// Rows [end, T) of up to three tensors of `bytes` a row: zeros; and of lse [H, T]: -inf.
struct TailParams {
  uint4* x[3];
  int vecs[3];             // 16-byte vectors of a row
  float* lse;
  int H, T;
  const int32_t* end;
};
__global__ void __launch_bounds__(256) packed_tail_kernel(const TailParams p) {
  const int end = min(max(*p.end, 0), p.T);
  for (int k = 0; k < 3; ++k) {
    if (!p.x[k]) continue;
    const long long n = static_cast<long long>(p.T - end) * p.vecs[k];
    uint4* const x = p.x[k] + static_cast<long long>(end) * p.vecs[k];
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<long long>(gridDim.x) * 256) x[i] = make_uint4(0, 0, 0, 0);
  }
  if (p.lse)
    for (int t = end + blockIdx.x; t < p.T; t += gridDim.x)
      for (int h = threadIdx.x; h < p.H; h += 256) p.lse[static_cast<size_t>(h) * p.T + t] = -INFINITY;
}

}  // namespace

int packed_shift(int max_seqlen, int tile) {
  int shift = 0;
  while (((static_cast<long long>(max_seqlen) + tile - 1) / tile + (1LL << shift) - 1) >> shift > kLevels) ++shift;
  return shift;
}
long long packed_bound(int T, int nseq, int max_seqlen, int tile) {
  return T / tile + (static_cast<long long>(nseq) << packed_shift(max_seqlen, tile));
}

cudaError_t launch_packed_tiles(const int32_t* cu, int nseq, int T, int max_seqlen, int tile, bool causal, bool backward, int* head, int4* tiles,
                                unsigned* status, cudaStream_t stream) {
  packed_tiles_kernel<<<1, kThreads, 0, stream>>>(cu, nseq, T, max_seqlen, tile, packed_shift(max_seqlen, tile), causal, backward,
                                                  static_cast<int>(packed_bound(T, nseq, max_seqlen, tile)), head, tiles, status);
  return cudaGetLastError();
}

cudaError_t launch_packed_tail(void* const x[3], const int row_bytes[3], float* lse, int H, int T, const int32_t* end, cudaStream_t stream) {
  TailParams p{};
  for (int k = 0; k < 3; ++k) {
    p.x[k] = static_cast<uint4*>(x[k]);
    p.vecs[k] = row_bytes[k] / 16;
  }
  p.lse = lse;
  p.H = H; p.T = T;
  p.end = end;
  packed_tail_kernel<<<152, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
