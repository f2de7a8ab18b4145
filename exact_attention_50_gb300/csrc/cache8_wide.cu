// cache8_wide.cu -- many query rows over an 8-bit KV cache (chunks of a prompt): the cache is expanded
// to 16 bits once, in the caller's workspace, and the tcgen05 forward runs on that.
//
// With R rows per kv head the forward reads every key R / 128 times, so expanding inside it would
// repeat the conversion as often, on the warps whose exponentials bound it; once costs 5 bytes of
// traffic per code.  K and V are expanded to bare codes, exact in either 16-bit type; K's scales multiply
// the scores in fp32, and log2 of V's, in units of the head's largest, goes into P's exponent.  So the one
// rounding is that of P (fp16 whatever the type, half a step 2^-11), relative to the largest P vs of the
// row's own keys: scale / unit in V (a chunk of 2048 queries took 817 to 859 us with that, now 820 to 832) would lose
// the digits of rows that see small scales only.  A block whose scale is below 2^-60 of the head's largest, or below 2^-126,
// counts as values of zero.
#include <algorithm>
#include "cache8.cuh"

namespace attn {
namespace {

__device__ __forceinline__ uint32_t pair(const __half*, float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pair(const __nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, typename Code>
__device__ __forceinline__ void expand16(const uint4 w, uint4* dst) {
  const T* tag = nullptr;
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4];
    Code::decode4(in[i], x);
    out[2 * i] = pair(tag, x[0], x[1]);
    out[2 * i + 1] = pair(tag, x[2], x[3]);
  }
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// One key range: the rows of a 128-row block that sees no key have no work item; O = 0, LSE = -inf. Blocks first,
// first + step, .. of one (batch, kv head).
__device__ __forceinline__ void unseen_rows(const Cache8Params& p, int bh, int L, int first, int step) {
  const int es = p.out_f32 ? 4 : 2;
  for (int rb = first; rb < (p.R + 127) / 128; rb += step) {
    if (kv_needed_keys(L, p.Nq, p.R, rb, p.causal != 0) > 0) continue;
    const int rows = min(128, p.R - rb * 128);
    const size_t row = static_cast<size_t>(bh) * p.R + rb * 128;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.o) + row * p.d * es);
    for (int i = threadIdx.x; i < rows * p.d * es / 16; i += 256) dst[i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = threadIdx.x; i < rows; i += 256) p.lse[row + i] = -INFINITY;
  }
}

// A CTA expands 128 tokens of one (batch, kv head), and every per-th 128 behind them: 16 codes of K and of V
// per thread and step.  Each CTA looks through all of the head's scales for the unit, which it should not
// read more of than a quarter of its codes' traffic, while there are 16 CTAs per SM (4 heads of 2^20 tokens
// in blocks of 16, 128 rows: 1066 us, with a CTA for each 128 tokens 1557; in blocks of 128: 960 and 956).
template <typename T, typename Code>
__global__ void __launch_bounds__(256) expand_kernel(const Cache8Params p, T* k16, __half* v16, float* v_unit, float* v_log, int per, bool final_rows) {
  constexpr float kSpread = 60.f;
  __shared__ float s_max[8];
  const int bh = blockIdx.x / per, first = blockIdx.x % per;
  const int L = cache_len(p.cache_seqlens, bh / p.Hkv, p.Nk, nullptr, false);
  if (final_rows) unseen_rows(p, bh, L, first, per);
  const int tiles = (L + 127) / 128, chunks = p.d / 16;
  if (first >= tiles) return;
  uint4 kw[4], vw[4];  // all of a thread's codes on their way at once (128 tokens, 8 chunks of 16: four each)
  auto load = [&](int tile) {
    const int j0 = tile * 128;
    const size_t base = (static_cast<size_t>(bh) * p.Nk + j0) * p.d;
    const uint4* k = reinterpret_cast<const uint4*>(p.k8 + base);
    const uint4* v = reinterpret_cast<const uint4*>(p.v8 + base);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i < 128 * chunks && j0 + i / chunks < L) {
        kw[u] = k[i];
        vw[u] = v[i];
      }
    }
  };
  load(first);
  // the unit: the largest scale of the blocks that hold tokens; one that is infinite or NaN shows in its block's values
  const float* vs = p.v_scale + static_cast<size_t>(bh) * p.n_blocks;
  float unit = 0.f;
  for (int i = threadIdx.x; i <= (L - 1) >> p.block_shift; i += 256)
    if (vs[i] < INFINITY) unit = fmaxf(unit, vs[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) unit = fmaxf(unit, __shfl_xor_sync(0xffffffffu, unit, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = unit;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) unit = fmaxf(unit, s_max[i]);
  if (first == 0 && threadIdx.x == 0) v_unit[bh] = unit;
  const float least = fmaxf(unit * 0x1p-60f, 0x1p-126f);  // scales below it count as 0
  for (int tile = first;;) {
    const int j0 = tile * 128, n = min(128, p.Nk - j0) * chunks;
    const size_t base = (static_cast<size_t>(bh) * p.Nk + j0) * p.d;
    uint4* ko = reinterpret_cast<uint4*>(k16 + base);
    uint4* vo = reinterpret_cast<uint4*>(v16 + base);
    const int block = (j0 >> p.block_shift) + threadIdx.x;  // of the blocks that hold tokens
    if (block <= (min(j0 + 128, L) - 1) >> p.block_shift)
      v_log[static_cast<size_t>(bh) * p.n_blocks + block] =
          vs[block] < least ? -kSpread : vs[block] < INFINITY ? log2f(vs[block] / unit) : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (i >= n) break;
      const int j = j0 + i / chunks;
      if (j < L) {
        expand16<T, Code>(kw[u], ko + 2 * i);
        const float s = vs[j >> p.block_shift];
        expand16<__half, Code>(s < least ? make_uint4(0, 0, 0, 0) : vw[u], vo + 2 * i);
        if (!(s < INFINITY)) vo[2 * i] = vo[2 * i + 1] = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);  // NaN
      } else {  // the tile's rest: a weight of zero times what lies there has to be zero
        const uint4 z = make_uint4(0, 0, 0, 0);
        ko[2 * i] = ko[2 * i + 1] = vo[2 * i] = vo[2 * i + 1] = z;
      }
    }
    tile += per;
    if (tile >= tiles) break;
    load(tile);
  }
}

template <typename T>
cudaError_t expand(const Cache8Params& p, void* k16, void* v16, float* v_unit, float* v_log, bool final_rows, attn_cache_dtype_t cache,
                   cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const long long tiles = (p.Nk + 127) / 128, each = std::max(1, p.n_blocks / (40 * p.d));
  const int per = static_cast<int>(std::min(tiles, std::max((tiles + each - 1) / each, (16 * 152 + heads - 1) / heads)));
  const int grid = static_cast<int>(heads) * per;
  if (cache == ATTN_CACHE_I8)
    expand_kernel<T, CodeI8><<<grid, 256, 0, stream>>>(p, static_cast<T*>(k16), static_cast<__half*>(v16), v_unit, v_log, per, final_rows);
  else
    expand_kernel<T, CodeE4m3><<<grid, 256, 0, stream>>>(p, static_cast<T*>(k16), static_cast<__half*>(v16), v_unit, v_log, per, final_rows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache8_expand(const Cache8Params& p, void* k16, void* v16, float* v_unit, float* v_log, bool final_rows, attn_dtype_t dtype,
                                 attn_cache_dtype_t cache, cudaStream_t stream) {
  return dtype == ATTN_F16 ? expand<__half>(p, k16, v16, v_unit, v_log, final_rows, cache, stream)
                           : expand<__nv_bfloat16>(p, k16, v16, v_unit, v_log, final_rows, cache, stream);
}

}  // namespace attn
