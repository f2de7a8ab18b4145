// packed_tiles.cu -- the list of tiles of packed sequences, heaviest first, for the forward and the backward of
// packed attention with grouped heads; and what lies behind the last sequence.
//
// The lengths are on the device, so the host knows only bounds.  A grid over (longest sequence, sequences) is mostly
// empty when the lengths differ: 1000 sequences of which one has 4096 tokens would be 97% items without a row.  The
// list holds the tiles that there are.  Under the causal mask a forward tile's cost grows with its number, a
// backward (key) tile's with its distance from the sequence's end; call that the tile's level, 0 .. n - 1 in a
// sequence of n tiles.  Level l holds one tile of each sequence longer than l, so with the sequences counted by n
// (one histogram and its suffix sums) every tile's place is known without a sort:
//   A[n] = sequences of more than n tiles,  first[l] = sum of A[l'] over l' > l,
//   place(level l of a sequence of n tiles, r-th of its length) = first[l] + A[n] + r.
// Without the mask all tiles of a sequence cost the same, and longer sequences come first:
//   place = sum of m over the sequences of m > n tiles + r n + l.
// Both sums come from one pass over the levels, with h[m] = sequences of m tiles: A[n] = sum of h[m], M[n] = sum of m h[m]
// over m > n;  first[l] = M[l + 1] - (l + 1) A[l + 1], and without the mask the place is M[n] + r n + l.
// Sequences of more than kLevels tiles take 2^shift tiles a level.
//
// One CTA, a chain of one read of cu, a barrier, the sums and the writes; a thread keeps its sequence in registers when
// there are no more than threads.
#include <algorithm>
#include "kernels.h"
#include "ptx.cuh"
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kLevels = 2048, kThreads = 1024;

struct ListParams {
  const int32_t* cu;
  int nseq, T, max_seqlen, tile, shift, levels, by_level, backward, bound;
  int* head;
  int4* out;
  unsigned* status;
};

__global__ void __launch_bounds__(kThreads) packed_tiles_kernel(const ListParams p) {
  __shared__ int A[kLevels + 2], M[kLevels + 2], seen[kLevels + 2];  // by number of levels, 0 .. levels + 1
  __shared__ int s_a[32], s_m[32];
  dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = 1 << p.shift, top = p.levels;
  const int32_t* const cu = p.cu;
  // the sequence's start and length (0: none, or not to be computed), and its levels
  const auto look = [&](int s, int& c0, bool report) -> int {
    c0 = cu[s];
    const int c1 = cu[s + 1];
    if (c0 < 0 || c1 < c0 || c1 > p.T || c1 - c0 > p.max_seqlen || (s == 0 && c0 != 0)) {
      if (report) raise_status(p.status, ATTN_ERR_DEVICE_INPUT);
      return 0;
    }
    return c1 - c0;
  };
  const auto levels_of = [&](int len) { return ((len + p.tile - 1) / p.tile + sub - 1) >> p.shift; };
  const bool once = p.nseq <= kThreads;  // a thread's sequence stays in registers
  const int mine = lane * 32 + warp;     // few sequences are spread over the warps, which write their tiles
  int c0 = 0, len = 0, n = 0, r = 0;
  if (once && mine < p.nseq) len = look(mine, c0, true);
  for (int i = threadIdx.x; i <= top + 1; i += kThreads) A[i] = seen[i] = 0;
  __syncthreads();
  if (once) {
    n = levels_of(len);
    if (n > 0) r = atomicAdd(A + n, 1);
  } else {
    for (int s = threadIdx.x; s < p.nseq; s += kThreads) {
      const int m = levels_of(look(s, c0, true));
      if (m > 0) atomicAdd(A + m, 1);
    }
  }
  __syncthreads();
  // the sums behind each number of levels: a thread takes neighbouring ones from the top down
  {
    const int each = (top + kThreads) / kThreads + 1;  // covers 0 .. top + 1
    const int hi = top + 1 - each * static_cast<int>(threadIdx.x);
    int a = 0, m = 0;
    for (int k = 0; k < each; ++k)
      if (hi - k >= 0) {
        a += A[hi - k];
        m += A[hi - k] * (hi - k);
      }
    int xa = a, xm = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ya = __shfl_up_sync(0xffffffffu, xa, o), ym = __shfl_up_sync(0xffffffffu, xm, o);
      if (lane >= o) {
        xa += ya;
        xm += ym;
      }
    }
    if (lane == 31) {
      s_a[warp] = xa;
      s_m[warp] = xm;
    }
    __syncthreads();
    xa -= a;
    xm -= m;
    // (as many warps as there are levels for)
    for (int w = 0; w < warp && w * 32 * each <= top + 1; ++w) {
      xa += s_a[w];
      xm += s_m[w];
    }
    for (int k = 0; k < each; ++k)
      if (hi - k >= 0) {
        const int h = A[hi - k];
        A[hi - k] = xa;
        M[hi - k] = xm;
        xa += h;
        xm += h * (hi - k);
      }
  }
  __syncthreads();
  const long long count = static_cast<long long>(M[0]) << p.shift;  // all tiles (no sequence has 0)
  const bool fits = count <= p.bound;  // always, when cu does not decrease
  if (threadIdx.x == 0) {
    const int end = cu[p.nseq];
    p.head[0] = fits ? static_cast<int>(count) : 0;
    p.head[1] = end >= 0 && end <= p.T ? end : p.T;
    if (!fits) raise_status(p.status, ATTN_ERR_DEVICE_INPUT);
  }
  if (!fits) return;
  const bool turn = p.by_level && p.backward;  // key tiles in ascending order as the levels fall
  const auto put = [&](int c0, int len, int n, int r, int held, int at) {  // tile `at` of the r-th sequence of n levels, `held` tiles
    const int l = at >> p.shift, in = at & (sub - 1);
    const int place = p.by_level ? M[l + 1] - (l + 1) * A[l + 1] + A[n] + r : M[n] + r * n + l;
    const int no = turn ? n * sub - 1 - at : at;
    p.out[static_cast<long long>(place) * sub + (turn ? sub - 1 - in : in)] = make_int4(c0, no < held ? len : 0, no, 0);
  };
  for (int s0 = 0; s0 < p.nseq; s0 += kThreads) {
    if (!once) {
      len = n = r = 0;
      if (s0 + mine < p.nseq) len = look(s0 + mine, c0, false);
      n = levels_of(len);
      if (n > 0) r = atomicAdd(seen + n, 1);
    }
    const int held = (len + p.tile - 1) / p.tile;
    const bool small = n * sub <= 4;
    if (small)
      for (int at = 0; at < n * sub; ++at) put(c0, len, n, r, held, at);
    for (unsigned big = __ballot_sync(0xffffffffu, !small); big; big &= big - 1) {
      const int src = __ffs(big) - 1;
      const int bc = __shfl_sync(0xffffffffu, c0, src), bl = __shfl_sync(0xffffffffu, len, src);
      const int bn = __shfl_sync(0xffffffffu, n, src), br = __shfl_sync(0xffffffffu, r, src), bh = __shfl_sync(0xffffffffu, held, src);
      for (int at = lane; at < bn * sub; at += 32) put(bc, bl, bn, br, bh, at);
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

cudaError_t launch_packed_tiles(const int32_t* cu, int nseq, int T, int max_seqlen, int tile, bool by_level, bool backward, int* head, int4* tiles,
                                unsigned* status, cudaStream_t stream) {
  ListParams p{};
  p.cu = cu;
  p.nseq = nseq; p.T = T; p.max_seqlen = max_seqlen; p.tile = tile;
  p.shift = packed_shift(max_seqlen, tile);
  p.levels = static_cast<int>(((static_cast<long long>(max_seqlen) + tile - 1) / tile + (1LL << p.shift) - 1) >> p.shift);
  p.by_level = by_level; p.backward = backward;
  p.bound = static_cast<int>(packed_bound(T, nseq, max_seqlen, tile));
  p.head = head;
  p.out = tiles;
  p.status = status;
  packed_tiles_kernel<<<1, kThreads, 0, stream>>>(p);
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
