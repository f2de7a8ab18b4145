// cache8_fwd.cu -- attention of few query rows over an 8-bit KV cache (decode, drafts of a few
// tokens): HBM-bound, each code is read once.
//
// A row r is query i = r % Nq of head g = r / Nq of a kv head's group, R = G Nq rows share its
// keys.  With code c and block scales ks, vs:
//   s_j = scale ks_j (q . ck_j), masked;  l = sum_j exp(s_j - m);  o = sum_j exp(s_j - m) vs_j cv_j / l.
//
// Work: the caches are cut into tiles of 32 keys (48 for more than 8 rows, 64 for long caches of 64
// columns), and all tiles of all (batch, kv head) pairs, one after the other, are dealt in equal runs
// to the workers, whatever the sequences' lengths.  A worker is one warp per block of rows, four warps a CTA, as many CTAs as
// fit.  A run may begin and end inside a pair: such parts go to the workspace, normalised with
// their log-sum-exp, and a second kernel merges them; a pair that lies within one run is
// finished by its worker.  (Warps of a CTA that shared a run and joined their sums in shared memory
// for every pair took 55 us for 256 sequences of 100 to 200 keys, now 31 us.)  Small problems take a
// cluster of CTAs per pair instead.
//
// A worker keeps its own ring of tiles full: when a tile's codes are in registers its first warp
// starts the copies of the tile that follows in that stage -- TMA tile loads of K and V, swizzled,
// and 4-byte asynchronous copies of the scales -- so there is no producer warp and, with one
// row block, no barrier but the copies' own.  Codes become fp16 in registers and are multiplied
// with mma.sync.m16n8k16, fp32 sums, keys (or columns of V) as the 16 rows and query rows as the 8
// columns: S^T = K Q^T, O^T = V^T P^T.  A tcgen05 product would have to take the converted tiles
// through shared memory again, 5 times the traffic of the codes, and has at least 64 rows of
// which the few queries of a decode fill 4.
//
// The contraction index is permuted so that a thread's fragments are whole 16-byte chunks: columns
// 32 t .. 32 t + 31 of a key for K Q^T (t = lane % 4), columns 16 g .. 16 g + 15 of four keys for
// V^T P^T (g = lane / 4); the swizzle makes both conflict-free.  P^T goes from the layout of S^T to
// that of an operand by an 8 x 8 transposition between the lanes (movmatrix).
//
// Conversion: K's int8 codes as fp16 subnormals, (code + 128) 2^-24, exact, two instructions a pair;
// the sum starts at -128 2^-24 sum(q), so it rounds at the size of 255 sum|q| instead of sum|q code|: scores
// are off by about 2e-7 (rms, q.k of size one), 2e-6 with one column of K far above the others.  V's by placing code + 128 in the mantissa of 1024 + u and
// subtracting 1152: there the offset would be far larger than the sums.  e4m3 by the conversion
// instruction.
//
// What it reaches (8 sequences of 16k to 32k keys, 32 over 8 heads, d = 128, int8): 77 us, 5.5 TB/s, 81% of
// the copy rate: 71 us in this kernel, the rest the merge (5 us alone, partly hidden) and the launch; 75 us with
// one query row per kv head.  With 16 rows (NB = 2) 85 us.  With 32 (two warps per tile, the codes converted
// twice) 145 us: 253 registers leave two warps per scheduler, which issue in 45% of the cycles, waiting
// mostly for results of fixed latency; ALU 45%, tensor pipe 34%, DRAM 38%, so no unit bounds it.  With 64 264 us.
//
// Rounding: q in bf16 becomes fp16 after a multiplication by a power of two per row (largest
// element in [2^14, 2^15)), exact but for elements below 2^-28 of that.  P vs is rounded to fp16 (half a
// step 2^-11) in units near the largest P vs among the keys that the row sees, so an error
// is relative to the row's own terms, whatever the scales of other blocks; a term below 2^-14 of the largest
// has an absolute error of 2^-25 of that.  A block whose scale is below 2^-60 of the largest of a worker's
// keys, and one below 2^-126, counts as values of zero.
#include <algorithm>
#include <atomic>
#include <type_traits>
#include <cooperative_groups.h>
#include "kv_runs.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLazy = 8.0f;   // log2 units by which a tile's maximum may exceed the running one
constexpr int kSpread = 60;     // powers of two that value scales may lie apart

// NB: blocks of 8 query rows per warp, 1 or 2.
template <int DP, int NB, int KEYS>
struct Layout {
  static constexpr int kKeys = KEYS;
  static constexpr int kGroups = kKeys / 16;                  // 16 keys share a scale
  static constexpr int kCtas = cache8_ctas_per_sm(NB);
  static constexpr int kTile = kKeys * DP;                    // bytes of codes
  static constexpr int kStages = (NB == 1 ? 16 : 24) * 1024 / (2 * kTile);  // per warp: 64 or 96 KB a CTA
  static constexpr int kOffV = kTile;                         // within a stage: K, V
  static constexpr int kStage = 2 * kTile;
  static constexpr int kOffScale = kWarps * kStages * kStage; // per stage: (ks, vs) of each group
  static constexpr int kOffBar = kOffScale + kWarps * kStages * 32;  // full[], empty[]
  static constexpr int kOffMisc = kOffBar + 2 * kWarps * kStages * 8;  // pad, abort flag, wait limit
  static constexpr int kBytes = kOffMisc + 16;
  static_assert((kBytes + 1024) * kCtas <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Four codes of K as two pairs of fp16, less the offset and in units of kUnitK.
template <typename Code>
constexpr float kUnitK = 1.f;
template <>
constexpr float kUnitK<CodeI8> = 16777216.f;  // 2^24
__device__ __forceinline__ void k_to_half(CodeI8, uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  lo = __byte_perm(w, 0u, 0x4140);
  hi = __byte_perm(w, 0u, 0x4342);
}
__device__ __forceinline__ void k_to_half(CodeE4m3 c, uint32_t w, uint32_t& lo, uint32_t& hi);

// Four codes as two pairs of fp16.
__device__ __forceinline__ void to_half(CodeI8, uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;  // code + 128, 0 .. 255
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);  // 1024 + code + 128
  const uint32_t off = 0x64806480u;                                                                  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&off));
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&off));
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void to_half(CodeE4m3, uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void k_to_half(CodeE4m3 c, uint32_t w, uint32_t& lo, uint32_t& hi) { to_half(c, w, lo, hi); }

__device__ __forceinline__ void unpack2(const __half*, uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x; b = f.y;
}
__device__ __forceinline__ void unpack2(const __nv_bfloat16*, uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

// SPREAD: a cluster of CTAs per pair, whose workers take its tiles in turn and join their sums through
// distributed shared memory; no workspace and no second kernel.
template <typename T, typename Code, int DP, int NB, int KEYS, bool SPREAD>
__global__ void __launch_bounds__(kThreads, (Layout<DP, NB, KEYS>::kCtas))
    cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Cache8Params p) {
  using L = Layout<DP, NB, KEYS>;
  constexpr int kKeys = L::kKeys, kGroups = L::kGroups;
  constexpr int kSteps = DP / 16;  // contraction steps of K Q^T
  constexpr int kCols = DP / 16;   // 16-column blocks of V
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle needs aligned tiles
    if (threadIdx.x == 0) raise_status(p.status, ATTN_ERR_CUDA);
    return;
  }
  const uint32_t abort_flag = smem_u32(smem + L::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a worker: RB warps, one per 8 NB rows, in RBW (a power of two) places
  const int RB = SPREAD ? 1 : (p.R + 8 * NB - 1) / (8 * NB);
  const int RBW = RB <= 1 ? 1 : RB <= 2 ? 2 : 4;
  const int rb = warp % RBW, first_warp = warp - rb;
  const uint32_t stages = L::kStages * RBW;  // of the worker's ring
  uint8_t* const ring = smem + first_warp * L::kStages * L::kStage;
  float* const s_scale = reinterpret_cast<float*>(smem + L::kOffScale) + first_warp * L::kStages * 8;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::kOffBar) + first_warp * L::kStages;
  uint64_t* const empty = full + kWarps * L::kStages;
  if (threadIdx.x == 0) {
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
    for (int i = 0; i < kWarps * L::kStages; ++i) {
      mbar_init(bars + i, 1 + 2 * kGroups);  // the tile's bytes, and its scales
      mbar_init(bars + kWarps * L::kStages + i, RB);
    }
    abort_set(abort_flag, 0);
    wait_limit_set(abort_flag, p.wait_ns);
    mbar_init_fence();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  if (!SPREAD) dependents_launch();
  const int per_cta = kWarps / RBW;
  const int run = blockIdx.x * per_cta + warp / RBW;
  const int stride = SPREAD ? p.cluster * kWarps : 1;  // from a worker's tile of a pair to its next
  Deal deal{};
  Walk w;
  if constexpr (SPREAD) {
    const int bh = blockIdx.x / p.cluster;
    w.b = bh / p.Hkv;
    w.h = bh % p.Hkv;
    w.j = run % stride;
    const int len = cache_len(p.cache_seqlens, w.b, p.Nk, p.status, w.h == 0 && w.j == 0 && lane == 0);
    w.nt = (len + kKeys - 1) / kKeys;
    w.t = w.j;
    w.end = w.nt;
  } else {
    deal_and_find(p, p.runs, run, deal, w);
  }

  // ---- the copies of the run's next tile, into the stage of its number
  Walk ahead = w;
  uint32_t issued = 0;
  bool ok = true;
  auto issue = [&]() {
    if (ahead.t >= ahead.end) return;
    const uint32_t st = issued % stages;
    if (RB > 1 && issued >= stages && !mbar_wait_warp(empty + st, ((issued / stages) - 1) & 1, abort_flag, p.status)) {
      ok = false;
      return;
    }
    const int bh = ahead.b * p.Hkv + ahead.h, key0 = ahead.j * kKeys;
    if (lane == 0) {
      mbar_expect_tx(full + st, L::kStage);
      tma_load_3d(ring + st * L::kStage, &tmK, full + st, 0, key0, bh);
      tma_load_3d(ring + st * L::kStage + L::kOffV, &tmV, full + st, 0, key0, bh);
    }
    if (lane < 2 * kGroups) {
      // the scale of 16 keys; of none that the cache holds: 0, the scale there is not read
      const int key = key0 + (lane >> 1) * 16;
      float* dst = s_scale + st * 8 + lane;
      if (key < cache_len(p.cache_seqlens, ahead.b, p.Nk, nullptr, false)) {
        const float* src = ((lane & 1) == 0 ? p.k_scale : p.v_scale) + static_cast<size_t>(bh) * p.n_blocks + (key >> p.block_shift);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + st)) : "memory");
      } else {
        *dst = 0.f;
        mbar_arrive(full + st);
      }
    }
    __syncwarp();
    ++issued;
    if (SPREAD) {
      ahead.t = ahead.j += stride;
    } else if (ahead.j + 1 < ahead.nt) {
      ++ahead.t;
      ++ahead.j;
    } else {
      ahead.next(p);  // the pair's last tile: its part is this one
    }
  };
  if (rb == 0)
    for (uint32_t i = 0; i < stages; ++i) issue();

  const int g = lane >> 2, t = lane & 3;
  const bool works = rb < RB;
  const uint32_t tiles = smem_u32(ring);
  const int row0 = rb * 8 * NB;  // this warp's rows; as columns of S^T and O^T this thread has rows 8 b + 2 t + e of them
  uint32_t n = 0;                // tiles of the run passed
  for (; SPREAD || (works && ok && w.t < w.end); w.next(p)) {
    const int len = cache_len(p.cache_seqlens, w.b, p.Nk, nullptr, false);
    const size_t bh = static_cast<size_t>(w.b) * p.Hkv + w.h;
    const int part = SPREAD ? (max(w.nt - w.j, 0) + stride - 1) / stride : w.part();
    // ---- Q as B fragments: step s holds columns (DP / 4) t + 4 s .. + 3 of row g
    uint32_t qb[NB][kSteps][2];
    float f[NB][2], start[NB][2];  // per row: scale log2(e) over its power of two; where its sums start
    int last[NB][2];               // the last key the row sees
    {
      const T* q = static_cast<const T*>(p.q) + bh * p.R * p.d;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = row0 + 8 * b + g;
        uint2 raw[kSteps];
        uint32_t mx = 0;  // an ordered maximum of magnitudes that keeps infinity and NaN
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int c = (DP / 4) * t + 4 * s;
          raw[s] = r < p.R && c < p.d ? *reinterpret_cast<const uint2*>(q + static_cast<size_t>(r) * p.d + c) : make_uint2(0, 0);
          if (!std::is_same<T, __half>::value) {
            const uint32_t x = raw[s].x & 0x7fff7fffu, y = raw[s].y & 0x7fff7fffu;
            mx = max(max(mx, max(x << 16, x & 0xffff0000u)), max(y << 16, y & 0xffff0000u));
          }
        }
        float up = 1.f, down = 1.f;
        if (!std::is_same<T, __half>::value) {
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int k = 0;  // q 2^k has its largest element in [2^14, 2^15)
          if (mx != 0 && mx < 0x7f800000u) k = min(100, 14 + 127 - static_cast<int>(mx >> 23));
          up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
          down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        }
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          float a, c, a2, c2;
          if (std::is_same<T, __half>::value) {
            qb[b][s][0] = raw[s].x;
            qb[b][s][1] = raw[s].y;
          } else {
            unpack2(q, raw[s].x, a, c);
            qb[b][s][0] = pack_half(a * up, c * up);
            unpack2(q, raw[s].y, a, c);
            qb[b][s][1] = pack_half(a * up, c * up);
          }
          if (std::is_same<Code, CodeI8>::value) {
            unpack2(static_cast<const __half*>(nullptr), qb[b][s][0], a, c);
            unpack2(static_cast<const __half*>(nullptr), qb[b][s][1], a2, c2);
            sum += (a + c) + (a2 + c2);
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[b][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + e)) * p.scale_log2 * kUnitK<Code>;
          start[b][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e)) * (-128.f / 16777216.f);
          if (std::is_same<Code, CodeE4m3>::value) start[b][e] = 0.f;
          const int i = (row0 + 8 * b + 2 * t + e) % p.Nq;
          last[b][e] = p.causal ? min(len - p.Nq + i, len - 1) : len - 1;
        }
      }
    }
    float o[kCols][NB][4];
#pragma unroll
    for (int i = 0; i < kCols; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) o[i][b][0] = o[i][b][1] = o[i][b][2] = o[i][b][3] = 0.f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      m[b][0] = m[b][1] = -INFINITY;
      l[b][0] = l[b][1] = 0.f;
    }
    // The value scales lie in the exponents: with w = log2(vs) and m the running maximum of s + w over the keys
    // that a row sees,
    //   o = sum 2^(s + w - m) cv,  l = sum 2^(s + w - m) 2^(c - w):  O = 2^c o / l,  LSE = m - c + log2(l).
    // c, of the first tile's largest scale, only keeps l's terms within float's range.
    int vexp = 0;
    float vhigh = 0.f;  // 2^(c + kSpread); 0 before the first scale
    bool finite = true; // the value scales; one that is not leaves the LSE alone
    {
      for (int x = 0; x < part; ++x, ++n) {
        const uint32_t st = n % stages;
        // several warps read a tile: the one before has been read by all of them before its stage is filled again
        if (RB > 1 && rb == 0 && n > 0) issue();
        if (!ok || !mbar_wait_warp(full + st, (n / stages) & 1, abort_flag, p.status)) { ok = false; break; }
        const uint32_t kt = tiles + st * L::kStage, vt = kt + L::kOffV;
        float kg[kGroups], vg[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const float2 kv = *reinterpret_cast<const float2*>(s_scale + st * 8 + 2 * i);
          kg[i] = kv.x;
          vg[i] = kv.y;
        }
        // ---- S^T = K Q^T: blocks of 16 keys, side by side
        float s[kGroups][NB][4];
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            s[i][b][0] = s[i][b][2] = start[b][0];
            s[i][b][1] = s[i][b][3] = start[b][1];
          }
        constexpr int kChunks = DP / 64;  // 16-byte chunks of a thread
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint4 kw[kGroups][2];
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = i * 16 + e * 8 + g;
              const int chunk = kChunks * t + c;
              const int sw = DP == 128 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3));
              kw[i][e] = lds128(kt + row * DP + sw * 16);
            }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              uint32_t a[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t word = k == 0 ? kw[i][e].x : k == 1 ? kw[i][e].y : k == 2 ? kw[i][e].z : kw[i][e].w;
                k_to_half(Code{}, word, a[e], a[2 + e]);
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816(s[i][b], a, qb[b][c * 4 + k][0], qb[b][c * 4 + k][1]);
            }
        }
        // ---- scale, mask, running maximum
        const int key0 = (w.j + x * stride) * kKeys;
        float largest = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          if (!(vg[i] < INFINITY)) {
            finite = false;
            vg[i] = 0.f;
          }
          largest = fmaxf(largest, vg[i]);
        }
        if (largest > vhigh) {  // the first scale, or one that leaves c far behind
          const int e = min(max(static_cast<int>(__float_as_uint(largest) >> 23), 1), 254);
          const float up = static_cast<float>(e - 127 - vexp), down = ex2_approx(-up);
          vexp = e - 127;
          vhigh = __uint_as_float(static_cast<uint32_t>(min(e + kSpread, 255)) << 23);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            m[b][0] += up;
            m[b][1] += up;
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              o[i][b][0] *= down; o[i][b][1] *= down; o[i][b][2] *= down; o[i][b][3] *= down;
            }
          }
        }
        // per group: w, 2^(c - w), and what P is masked with: nothing of a scale of 0, or of one too small to
        // count beside the largest
        float wv[kGroups], lw[kGroups];
        uint32_t counts[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const float least = static_cast<float>(vexp - kSpread), x = __log2f(vg[i]);
          const bool none = __float_as_uint(vg[i]) < 0x00800000u || x < least;
          wv[i] = none ? least : x;
          lw[i] = ex2_approx(static_cast<float>(vexp) - wv[i]);
          counts[i] = none ? 0u : 0xffffffffu;
        }
        bool move = false;
        float mx[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            const float f0 = f[b][0] * kg[i], f1 = f[b][1] * kg[i];
            s[i][b][0] = fmaf(s[i][b][0], f0, wv[i]); s[i][b][1] = fmaf(s[i][b][1], f1, wv[i]);
            s[i][b][2] = fmaf(s[i][b][2], f0, wv[i]); s[i][b][3] = fmaf(s[i][b][3], f1, wv[i]);
          }
          if (__any_sync(0xffffffffu, key0 + kKeys - 1 > min(last[b][0], last[b][1]))) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              const int key = key0 + i * 16 + g;
              if (key > last[b][0]) s[i][b][0] = -INFINITY;
              if (key > last[b][1]) s[i][b][1] = -INFINITY;
              if (key + 8 > last[b][0]) s[i][b][2] = -INFINITY;
              if (key + 8 > last[b][1]) s[i][b][3] = -INFINITY;
            }
          }
          mx[b][0] = mx[b][1] = -INFINITY;
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            mx[b][0] = max3f(mx[b][0], s[i][b][0], s[i][b][2]);
            mx[b][1] = max3f(mx[b][1], s[i][b][1], s[i][b][3]);
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            mx[b][0] = fmaxf(mx[b][0], __shfl_xor_sync(0xffffffffu, mx[b][0], d));
            mx[b][1] = fmaxf(mx[b][1], __shfl_xor_sync(0xffffffffu, mx[b][1], d));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) move |= mx[b][e] > m[b][e] + kLazy || (m[b][e] == -INFINITY && mx[b][e] != -INFINITY);
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = fmaxf(m[b][e], mx[b][e]);
              a[e] = m[b][e] == top ? 1.f : m[b][e] == -INFINITY ? 0.f : ex2_approx(m[b][e] - top);
              m[b][e] = top;
              l[b][e] *= a[e];
            }
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              o[i][b][0] *= a[0]; o[i][b][1] *= a[1]; o[i][b][2] *= a[0]; o[i][b][3] *= a[1];
            }
          }
        }
        // ---- P = exp2(S + w - m), its sum, and fp16 B fragments
        uint32_t pb[kGroups][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float n0 = m[b][0] == -INFINITY ? 0.f : m[b][0], n1 = m[b][1] == -INFINITY ? 0.f : m[b][1];
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            const float e0 = ex2_approx(s[i][b][0] - n0), e1 = ex2_approx(s[i][b][1] - n1);
            const float e2 = ex2_approx(s[i][b][2] - n0), e3 = ex2_approx(s[i][b][3] - n1);
            l[b][0] = fmaf(e0 + e2, lw[i], l[b][0]);
            l[b][1] = fmaf(e1 + e3, lw[i], l[b][1]);
            pb[i][b][0] = transpose8x8(pack_half(e0, e1) & counts[i]);
            pb[i][b][1] = transpose8x8(pack_half(e2, e3) & counts[i]);
          }
        }
        // a code behind the cache's end may be e4m3's NaN, which a weight of zero does not cancel
        const int over = std::is_same<Code, CodeE4m3>::value ? len - key0 : kKeys;
        // ---- O^T += V^T P^T: per 16 keys, this thread's columns (DP / 8) g .. of keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          uint32_t vw[4][DP / 32];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = j * 16 + 2 * t + (e & 1) + (e >> 1) * 8;
            if constexpr (DP == 128) {
              const uint4 v = lds128(vt + row * DP + ((g ^ (row & 7)) << 4));
              vw[e][0] = v.x; vw[e][1] = v.y; vw[e][2] = v.z; vw[e][3] = v.w;
            } else {
              const uint2 v = lds64(vt + row * DP + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
              vw[e][0] = v.x; vw[e][1] = v.y;
            }
            if (over < kKeys && row >= over) {
#pragma unroll
              for (int k = 0; k < DP / 32; ++k) vw[e][k] = 0;
            }
          }
          if (j == kGroups - 1) {  // the tile is in registers: the next one into its stage
            __syncwarp();
            if (RB > 1 && lane == 0) mbar_arrive(empty + st);
            if (RB == 1) issue();
          }
#pragma unroll
          for (int k = 0; k < DP / 32; ++k)
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // columns 4 k + 2 c and + 1 of the chunk
              uint32_t a[4];
              to_half(Code{}, __byte_perm(vw[0][k], vw[1][k], c ? 0x7362 : 0x5140), a[0], a[1]);
              to_half(Code{}, __byte_perm(vw[2][k], vw[3][k], c ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816(o[2 * k + c][b], a, pb[j][b][0], pb[j][b][1]);
            }
        }
      }
    }
    if (!SPREAD && !ok) break;
    // ---- this warp's part: sums over the eight lanes that share a row; the output, normalised before it is
    // multiplied by 2^c, so that it overflows only where the values do; m and l in units of one
    const float unit = finite ? __uint_as_float(static_cast<uint32_t>(vexp + 127) << 23) : __int_as_float(0x7fffffff);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float il[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
        m[b][e] -= static_cast<float>(vexp);
        il[e] = l[b][e] == 0.f ? 0.f : 1.f / l[b][e];
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        o[i][b][0] = o[i][b][0] * il[0] * unit; o[i][b][1] = o[i][b][1] * il[1] * unit;
        o[i][b][2] = o[i][b][2] * il[0] * unit; o[i][b][3] = o[i][b][3] * il[1] * unit;
      }
    }
    if constexpr (SPREAD) {
      // ---- the workers' parts in their CTAs' shared memory (the ring, read to its end), then every
      // thread of the cluster sums some outputs over them
      const auto cluster = cooperative_groups::this_cluster();
      const int rank = blockIdx.x % p.cluster, workers = min(stride, w.nt);  // those with a tile
      constexpr int kRows = 8 * NB;
      float* const part_o = reinterpret_cast<float*>(smem);                            // [kWarps][kRows][DP]
      float2* const part_ml = reinterpret_cast<float2*>(smem + kWarps * kRows * DP * 4);  // [kWarps][kRows]
      float2* const all_ml = part_ml + kWarps * kRows;                                 // [workers][kRows]
      static_assert(kWarps * kRows * DP * 4 + 9 * kWarps * kRows * 8 <= L::kOffScale, "the parts lie in the ring");
      if (!ok || abort_read(abort_flag))  // let the copies land before their stages are written
        for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i) mbar_drain(full + i % stages, (i / stages) & 1);
      __syncthreads();
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * b + 2 * t + e;
          if (g == 0) part_ml[warp * kRows + r] = make_float2(m[b][e], l[b][e]);
          float* dst = part_o + (warp * kRows + r) * DP + (DP / 8) * g;
#pragma unroll
          for (int c = 0; c < DP / 8; c += 4)
            *reinterpret_cast<float4*>(dst + c) = make_float4(o[c / 2][b][e], o[c / 2][b][2 + e], o[c / 2 + 1][b][e], o[c / 2 + 1][b][2 + e]);
        }
      cluster.sync();
      for (int i = threadIdx.x; i < workers * kRows; i += kThreads) {
        const int k = i / kRows;
        all_ml[i] = *cluster.map_shared_rank(part_ml + (k % kWarps) * kRows + i % kRows, k / kWarps);
      }
      __syncthreads();
      const int half = p.d / 2;
      for (int i = rank * kThreads + threadIdx.x; i < p.R * half; i += p.cluster * kThreads) {
        const int r = i / half, c = i % half * 2;
        float top = -INFINITY;
        for (int k = 0; k < workers; ++k) top = fmaxf(top, all_ml[k * kRows + r].x);
        float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll 4
        for (int k = 0; k < workers; ++k) {
          const float2 ml = all_ml[k * kRows + r];
          const float2 v = *reinterpret_cast<const float2*>(cluster.map_shared_rank(part_o + ((k % kWarps) * kRows + r) * DP + c, k / kWarps));
          const float a = ml.y * (ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top));
          sum += a;
          x += v.x * a;
          y += v.y * a;
        }
        const float il = sum == 0.f ? 0.f : 1.f / sum;
        const size_t row = bh * p.R + r;
        if (p.out_f32) {
          *reinterpret_cast<float2*>(static_cast<float*>(p.o) + row * p.d + c) = make_float2(x * il, y * il);
        } else {
          const T* tag = nullptr;
          *reinterpret_cast<uint32_t*>(static_cast<T*>(p.o) + row * p.d + c) = pack2(tag, x * il, y * il);
        }
        if (c == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : add_log2(top, sum) * 0.69314718055994531f;
      }
      cluster.sync();  // the others may still read this CTA's parts
      return;
    }
    // ---- the pair's output, or this run's part of it
    {
      const bool whole = part == w.nt;
      // a run's first part may begin inside a pair (slot 0), another one ends inside it (slot 1)
      const size_t slot = static_cast<size_t>(run) * 2 + (w.j > 0 ? 0 : 1);
      // for the merge: the pair's first run and its number of runs
      if (w.j == 0 && rb == 0 && lane == 0)
        p.parts[bh] = make_int2(run, whole ? 0 : deal.holder(w.t + w.nt - 1) - run + 1);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = row0 + 8 * b + 2 * t + e;
          if (r >= p.R) continue;
          const float lse2 = l[b][e] == 0.f ? -INFINITY : add_log2(m[b][e], l[b][e]);
          const size_t row = whole ? bh * p.R + r : slot * p.R + r;
          if (g == 0) {
            if (!whole) p.lse_part[row] = lse2;
            else if (p.lse) p.lse[row] = lse2 * 0.69314718055994531f;
          }
          // columns (DP / 8) g + i: element 2 (i % 2) + e of block i / 2
#pragma unroll
          for (int i = 0; i < DP / 8; i += 8) {
            const int col = (DP / 8) * g + i;
            if (col >= p.d) continue;
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = o[(i + k) / 2][b][2 * (k & 1) + e];
            if (!whole || p.out_f32) {
              float4* dst = reinterpret_cast<float4*>((whole ? static_cast<float*>(p.o) : p.o_part) + row * p.d + col);
              dst[0] = make_float4(y[0], y[1], y[2], y[3]);
              dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              const T* tag = nullptr;
              *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + row * p.d + col) =
                  make_uint4(pack2(tag, y[0], y[1]), pack2(tag, y[2], y[3]), pack2(tag, y[4], y[5]), pack2(tag, y[6], y[7]));
            }
          }
        }
    }
  }
  if (rb == 0 && (!ok || abort_read(abort_flag)))  // let the copies land before the shared memory goes away
    for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i) mbar_drain(full + i % stages, (i / stages) & 1);
  // ---- batches without a key: O = 0, LSE = -inf, nothing to merge; dealt to the CTAs
  if (p.cache_seqlens) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (cache_len(p.cache_seqlens, b, p.Nk, p.status, threadIdx.x == 0) > 0) continue;
      const size_t rows = static_cast<size_t>(p.Hkv) * p.R;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.o) + b * rows * p.d * (p.out_f32 ? 4 : 2));
      const size_t n16 = rows * p.d * (p.out_f32 ? 4 : 2) / 16;
      for (size_t i = threadIdx.x; i < n16; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (size_t i = threadIdx.x; i < rows; i += kThreads) p.lse[b * rows + i] = -INFINITY;
      for (int i = threadIdx.x; i < p.Hkv; i += kThreads) p.parts[static_cast<size_t>(b) * p.Hkv + i] = make_int2(0, 0);
    }
  }
}

template <typename T, typename Code, int DP, int NB, int KEYS, bool SPREAD>
cudaError_t run(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, cudaStream_t stream) {
  using L = Layout<DP, NB, KEYS>;
  auto kern = cache8_kernel<T, Code, DP, NB, KEYS, SPREAD>;
  static std::atomic<unsigned long long> ready{0};  // devices on which the kernel is set up
  cudaError_t e = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  });
  if (e != cudaSuccess) return e;
  if (SPREAD) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, k, v, p);
  }
  kern<<<p.ctas, kThreads, L::kBytes, stream>>>(k, v, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while the first kernel runs (it takes its SMs' room as that ends), waits for it inside
  return p.out_f32 ? launch_merge<float>(p, stream) : launch_merge<T>(p, stream);
}

template <typename T, typename Code, int DP, int NB>
cudaError_t run_s(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, cudaStream_t stream) {
  constexpr int kKeys = NB == 1 ? 32 : 48;
  if (p.cluster) return run<T, Code, DP, NB, kKeys, true>(k, v, p, stream);
  if constexpr (DP == 64)
    if (p.tile_keys == 64) return run<T, Code, DP, NB, 64, false>(k, v, p, stream);
  return run<T, Code, DP, NB, kKeys, false>(k, v, p, stream);
}

template <typename T, typename Code>
cudaError_t run_c(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, cudaStream_t stream) {
  const bool few = cache8_row_blocks(p.R) == 1;
  if (p.d <= 64) return few ? run_s<T, Code, 64, 1>(k, v, p, stream) : run_s<T, Code, 64, 2>(k, v, p, stream);
  return few ? run_s<T, Code, 128, 1>(k, v, p, stream) : run_s<T, Code, 128, 2>(k, v, p, stream);
}

template <typename T>
cudaError_t run_t(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, attn_cache_dtype_t cache, cudaStream_t stream) {
  return cache == ATTN_CACHE_I8 ? run_c<T, CodeI8>(k, v, p, stream) : run_c<T, CodeE4m3>(k, v, p, stream);
}

}  // namespace

cudaError_t launch_cache8_none(const Cache8Params& p, cudaStream_t stream) { return launch_none(p, stream); }

cudaError_t launch_cache8_fwd(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, attn_dtype_t dtype,
                              attn_cache_dtype_t cache, cudaStream_t stream) {
  return dtype == ATTN_F16 ? run_t<__half>(k, v, p, cache, stream) : run_t<__nv_bfloat16>(k, v, p, cache, stream);
}

}  // namespace attn
