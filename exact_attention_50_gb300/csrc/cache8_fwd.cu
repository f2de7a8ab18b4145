// cache8_fwd.cu -- attention of few query rows over an 8-bit KV cache (decode, drafts of a few
// tokens): HBM-bound, each code is read once.
//
// A row r is query i = r % Nq of head g = r / Nq of a kv head's group, R = G Nq rows share its
// keys.  With code c and block scales ks, vs:
//   s_j = scale ks_j (q . ck_j), masked;  l = sum_j exp(s_j - m);  o = sum_j exp(s_j - m) vs_j cv_j / l.
//
// Work: the caches are cut into tiles of 48 keys, and all tiles of all (batch, kv head) pairs, one
// after the other, are dealt to the CTAs (two per SM) in equal runs, whatever the sequences'
// lengths.  A run may begin and end inside a sequence: such parts go to the workspace, normalised
// with their log-sum-exp, and a second kernel merges them; a sequence that lies within one run
// is finished by its CTA.
//
// A CTA is one producer warp and four consumer warps.  The producer keeps a ring of tiles full
// with TMA tile loads (K and V, swizzled, 12 KB a tile for d = 128) and 4-byte asynchronous
// copies of the scales.  A tile belongs to one consumer warp per 16 rows, which converts codes to
// fp16 in registers (exact: int8 by placing the byte in the mantissa of 1024 + u and subtracting,
// e4m3 by the conversion instruction) and multiplies with mma.sync.m16n8k16, fp32 sums. A tcgen05
// product would have to take the converted tiles through shared memory again, 5 times the
// traffic of the codes, to fill 4 of its 128 rows.  The contraction index is permuted so that a
// thread's B fragments are whole 16-byte chunks: columns 32 t .. 32 t + 31 of a key for Q K^T
// (t = lane % 4), columns 16 g .. 16 g + 15 of four keys for P V (g = lane / 4); the swizzle
// makes both conflict-free.
//
// Rounding: q in bf16 becomes fp16 after a multiplication by a power of two per row (largest
// element in [2^14, 2^15)), exact but for elements below 2^-28 of that.  P is rounded to fp16
// (half a step 2^-11) after its multiplication by vs / (the largest vs so far): a block whose
// scale is below 2^-14 of that has absolute errors of 2^-25 times the largest value instead.
#include <algorithm>
#include <type_traits>
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kKeys = kCache8Keys;  // keys of a tile: 48
constexpr int kGroups = kKeys / 16; // 16 keys share a scale
constexpr int kConsumers = 4;   // consumer warps of a CTA
constexpr int kThreads = 2 * kConsumers * 32;  // a warpgroup of consumers, one that holds the producer
// Registers: launched at 128 a thread (two CTAs fill the SM's file), then split by setmaxnreg; a
// consumer holds 64 sums of O, 32 of S and 32 registers of Q.
constexpr uint32_t kLaunchRegs = 128, kRegsConsumer = 216, kRegsProducer = 40;
static_assert(kRegsConsumer + kRegsProducer == 2 * kLaunchRegs, "register split must match the launch");
constexpr float kLazy = 8.0f;   // log2 units by which a tile's maximum may exceed the running one

template <int DP>
struct Layout {
  static constexpr int kTile = kKeys * DP;                    // bytes of codes
  // A multiple of the consumer warps: tile n of the run goes to stage n % kStages and to the warps
  // with tg == n % TG, so a stage has the same readers in every turn and none of them can
  // run ahead of its phase. Two stages a warp (d = 128) with 48 keys; 64 would leave room for one.
  static constexpr int kStages = DP == 128 ? 8 : 16;
  static_assert(kStages % kConsumers == 0, "a stage belongs to one consumer");
  static constexpr int kOffV = kTile;                         // within a stage: K, V
  static constexpr int kStage = 2 * kTile;
  static constexpr int kOffMerge = kStages * kStage;          // two warps' O: [DP / 8][32] float4
  static constexpr int kMerge = 16 * DP * 4;
  static constexpr int kOffStat = kOffMerge + 2 * kMerge;     // two warps' (m, l) of 16 rows
  static constexpr int kOffScale = kOffStat + 2 * 16 * 8;     // per stage: (ks, vs) of each group
  static constexpr int kOffBar = kOffScale + kStages * 32;    // full[], empty[], merge
  static constexpr int kOffMisc = kOffBar + (2 * kStages + 1) * 8;  // pad, abort flag, wait limit
  static constexpr int kBytes = kOffMisc + 16;
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

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack2(const __half*, uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x; b = f.y;
}
__device__ __forceinline__ void unpack2(const __nv_bfloat16*, uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ uint32_t pack2(const __half*, float a, float b) { return pack_half(a, b); }
__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Batch b's tiles per kv head.
__device__ __forceinline__ int tiles_of(const Cache8Params& p, int b) {
  return (cache_len(p.cache_seqlens, b, p.Nk, nullptr, false) + kKeys - 1) / kKeys;
}

// All tiles of all (batch, kv head) pairs; every lane of a warp calls it and gets the sum.
__device__ __forceinline__ long long total_tiles(const Cache8Params& p) {
  if (!p.cache_seqlens) return static_cast<long long>(p.B) * p.Hkv * ((p.Nk + kKeys - 1) / kKeys);
  long long sum = 0;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) sum += tiles_of(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * p.Hkv;
}

// Walks the parts of (batch, kv head) pairs that tiles [t, end) of the common numbering cover.
struct Walk {
  long long t, end;    // the next tile and the end
  int b, h, nt;        // the pair that holds tile t, its tiles
  int j;               // tile t's number within the pair
  // Whole warps call start: the batch that holds tile t is found by a scan over the lengths.
  __device__ __forceinline__ void start(const Cache8Params& p, long long first, long long last) {
    t = first;
    end = last;
    b = h = nt = j = 0;
    if (t >= end) return;
    const int lane = threadIdx.x & 31;
    long long off = 0;  // tiles before the 32 batches at b0
    for (int b0 = 0;; b0 += 32) {
      const int mine = b0 + lane < p.B ? tiles_of(p, b0 + lane) : 0;
      long long x = static_cast<long long>(mine) * p.Hkv;
      const long long own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, off + x > t);
      if (hit) {
        const int src = __ffs(hit) - 1;
        const long long before = off + __shfl_sync(0xffffffffu, x - own, src);
        nt = __shfl_sync(0xffffffffu, mine, src);
        b = b0 + src;
        h = static_cast<int>((t - before) / nt);
        j = static_cast<int>((t - before) % nt);
        return;
      }
      off += __shfl_sync(0xffffffffu, x, 31);
      if (b0 + 32 >= p.B) {  // not reached: t is below the total
        end = t;
        return;
      }
    }
  }
  __device__ __forceinline__ int part() const {  // tiles of this pair within the run
    const long long rest = end - t;
    return rest < nt - j ? static_cast<int>(rest) : nt - j;
  }
  __device__ __forceinline__ void next(const Cache8Params& p) {
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

__device__ __forceinline__ long long run_start(long long total, int c, int ctas) { return total * c / ctas; }
// The CTA whose run holds tile t.
__device__ __forceinline__ int run_of(long long total, long long t, int ctas) {
  return static_cast<int>(((t + 1) * ctas + total - 1) / total) - 1;
}

template <typename T, typename Code, int DP>
__global__ void __launch_bounds__(kThreads, 2)
    cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Cache8Params p) {
  using L = Layout<DP>;
  constexpr int kSteps = DP / 16;  // contraction steps of Q K^T
  constexpr int kCols = DP / 8;    // 8-column blocks of O
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle needs aligned tiles
    if (threadIdx.x == 0) raise_status(p.status, ATTN_ERR_CUDA);
    return;
  }
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* const empty = full + L::kStages;
  uint64_t* const merge = empty + L::kStages;
  float* const s_scale = reinterpret_cast<float*>(smem + L::kOffScale);
  const uint32_t abort_flag = smem_u32(smem + L::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps by row block and by tile: RBW row blocks of 16 (a power of two), TG tiles at a time
  const int RB = (p.R + 15) / 16;
  const int RBW = RB <= 1 ? 1 : RB <= 2 ? 2 : 4, TG = kConsumers / RBW;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(full + i, 1 + 2 * kGroups);  // the tile's bytes, and its scales
      mbar_init(empty + i, RB);
    }
    mbar_init(merge, kConsumers);
    abort_set(abort_flag, 0);
    wait_limit_set(abort_flag, p.wait_ns);
    mbar_init_fence();
  }
  __syncthreads();
  const long long total = total_tiles(p);
  Walk w;
  w.start(p, run_start(total, blockIdx.x, gridDim.x), run_start(total, blockIdx.x + 1, gridDim.x));

  if (warp >= kConsumers) {
    regs_dec<kRegsProducer>();
    if (warp > kConsumers) return;
    // ================================================================ producer
    uint32_t n = 0;  // tiles issued
    bool ok = true;
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    for (; ok && w.t < w.end; w.next(p)) {
      const int len = cache_len(p.cache_seqlens, w.b, p.Nk, nullptr, false);
      const int bh = w.b * p.Hkv + w.h;
      const int part = w.part();
      for (int i = 0; i < part; ++i, ++n) {
        const uint32_t st = n % L::kStages;
        if (n >= L::kStages && !mbar_wait_warp(empty + st, ((n / L::kStages) - 1) & 1, abort_flag, p.status)) { ok = false; break; }
        const int key0 = (w.j + i) * kKeys;
        if (lane == 0) {
          mbar_expect_tx(full + st, L::kStage);
          tma_load_3d(smem + st * L::kStage, &tmK, full + st, 0, key0, bh);
          tma_load_3d(smem + st * L::kStage + L::kOffV, &tmV, full + st, 0, key0, bh);
        }
        if (lane < 2 * kGroups) {
          // the scale of 16 keys; of none that the cache holds: 0, the scale there is not read
          const int key = key0 + (lane >> 1) * 16;
          float* dst = s_scale + st * 8 + lane;
          if (key < len) {
            const float* src = ((lane & 1) == 0 ? p.k_scale : p.v_scale) + static_cast<size_t>(bh) * p.n_blocks + (key >> p.block_shift);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + st)) : "memory");
          } else {
            *dst = 0.f;
            mbar_arrive(full + st);
          }
        }
      }
    }
    if (!ok || abort_read(abort_flag))  // let the copies land before the shared memory goes away
      for (uint32_t i = n > L::kStages ? n - L::kStages : 0; i < n; ++i) mbar_drain(full + i % L::kStages, (i / L::kStages) & 1);
    return;
  }

  regs_inc<kRegsConsumer>();
  // ================================================================ consumers
  const int g = lane >> 2, t = lane & 3;
  const int rb = warp % RBW, tg = warp / RBW;
  const bool works = rb < RB;
  const uint32_t tiles = smem_u32(smem);
  const int r0 = rb * 16 + g, r1 = r0 + 8;  // this thread's rows
  const int i0 = r0 % p.Nq, i1 = r1 % p.Nq;
  uint32_t n = 0;       // tiles of the run passed
  uint32_t merges = 0;  // phases of the merge barrier
  bool ok = true;       // after a failed wait: no more waits or sums, but the same barriers
  for (; w.t < w.end; w.next(p)) {
    const int len = cache_len(p.cache_seqlens, w.b, p.Nk, nullptr, false);
    const size_t bh = static_cast<size_t>(w.b) * p.Hkv + w.h;
    const int part = w.part();
    const int active = min(TG, part);  // warps (of a row block) with a tile: those with place < active
    const int place = (tg - static_cast<int>(n % TG) + TG) % TG;  // this warp's first tile of the part
    // ---- Q as A fragments: step s holds columns (DP / 4) t + 4 s .. + 3
    uint32_t qa[kSteps][4];
    float f0 = 0.f, f1 = 0.f;  // scale log2(e) over the row's power of two
    if (works && place < active) {
      const T* q = static_cast<const T*>(p.q) + bh * p.R * p.d;
      float mx[2] = {0.f, 0.f};
      uint2 raw[2][kSteps];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = e ? r1 : r0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int c = (DP / 4) * t + 4 * s;
          raw[e][s] = r < p.R && c < p.d ? *reinterpret_cast<const uint2*>(q + static_cast<size_t>(r) * p.d + c) : make_uint2(0, 0);
          float a, b, c2, d2;
          unpack2(q, raw[e][s].x, a, b);
          unpack2(q, raw[e][s].y, c2, d2);
          // an ordered maximum of magnitudes that keeps infinity and NaN
          const uint32_t hi = max(max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu),
                                  max(__float_as_uint(c2) & 0x7fffffffu, __float_as_uint(d2) & 0x7fffffffu));
          mx[e] = __uint_as_float(max(__float_as_uint(mx[e]), hi));
        }
        uint32_t u = __float_as_uint(mx[e]);
        u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
        u = max(u, __shfl_xor_sync(0xffffffffu, u, 2));
        mx[e] = __uint_as_float(u);
      }
      float up[2], down[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int k = 0;  // q 2^k has its largest element in [2^14, 2^15)
        const uint32_t u = __float_as_uint(mx[e]);
        if (sizeof(T) == 2 && !std::is_same<T, __half>::value && u != 0 && u < 0x7f800000u)
          k = min(100, 14 + 127 - static_cast<int>(u >> 23));
        up[e] = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        down[e] = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      }
      f0 = p.scale_log2 * down[0];
      f1 = p.scale_log2 * down[1];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (std::is_same<T, __half>::value) {
            qa[s][e] = raw[e][s].x;
            qa[s][2 + e] = raw[e][s].y;
          } else {
            float a, b;
            unpack2(q, raw[e][s].x, a, b);
            qa[s][e] = pack_half(a * up[e], b * up[e]);
            unpack2(q, raw[e][s].y, a, b);
            qa[s][2 + e] = pack_half(a * up[e], b * up[e]);
          }
        }
    }
    const int last0 = p.causal ? min(len - p.Nq + i0, len - 1) : len - 1;  // the last key each row sees
    const int last1 = p.causal ? min(len - p.Nq + i1, len - 1) : len - 1;
    float o[kCols][4];
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float vref = 0.f;  // the largest value scale so far: o is in units of it
    if (works) {
      for (int x = place; x < part; x += TG) {
        const uint32_t at = n + x, st = at % L::kStages;
        if (ok) ok = mbar_wait_warp(full + st, (at / L::kStages) & 1, abort_flag, p.status);
        if (!ok) break;
        const uint32_t kt = tiles + st * L::kStage, vt = kt + L::kOffV;
        float kg[kGroups], vg[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const float2 kv = *reinterpret_cast<const float2*>(s_scale + st * 8 + 2 * i);
          kg[i] = kv.x;
          vg[i] = kv.y;
        }
        // ---- S = Q K^T: six blocks of 8 keys, three at a time
        float s[2 * kGroups][4];
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kGroups; i += 3) {
          constexpr int kChunks = DP / 64;  // 16-byte chunks of a thread
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint4 kw[3];
#pragma unroll
            for (int e = 0; e < 3; ++e) {
              const int row = (i + e) * 8 + g;
              const int chunk = kChunks * t + c;
              const int sw = DP == 128 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3));
              kw[e] = lds128(kt + row * DP + sw * 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                const uint32_t word = k == 0 ? kw[e].x : k == 1 ? kw[e].y : k == 2 ? kw[e].z : kw[e].w;
                uint32_t b0, b1;
                to_half(Code{}, word, b0, b1);
                mma16816(s[i + e], qa[c * 4 + k], b0, b1);
              }
          }
        }
        // ---- scale, mask, running maximum
        const int key0 = (w.j + x) * kKeys + 2 * t;
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          const float a = f0 * kg[i >> 1], b = f1 * kg[i >> 1];
          s[i][0] *= a; s[i][1] *= a; s[i][2] *= b; s[i][3] *= b;
        }
        if (key0 - 2 * t + kKeys - 1 > min(last0, last1)) {
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            const int key = key0 + i * 8;
            if (key > last0) s[i][0] = -INFINITY;
            if (key + 1 > last0) s[i][1] = -INFINITY;
            if (key > last1) s[i][2] = -INFINITY;
            if (key + 1 > last1) s[i][3] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          mx0 = max3f(mx0, s[i][0], s[i][1]);
          mx1 = max3f(mx1, s[i][2], s[i][3]);
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float v_old = vref;
        vref = fmaxf(fmaxf(fmaxf(vg[0], vg[1]), vg[2]), vref);
        const bool move0 = mx0 > m0 + kLazy || (m0 == -INFINITY && mx0 != -INFINITY);
        const bool move1 = mx1 > m1 + kLazy || (m1 == -INFINITY && mx1 != -INFINITY);
        if (__any_sync(0xffffffffu, move0 || move1 || vref != v_old)) {
          const float back = v_old == vref ? 1.f : v_old / vref;
          const float a0 = !move0 ? 1.f : m0 == -INFINITY ? 0.f : ex2_approx(m0 - mx0);
          const float a1 = !move1 ? 1.f : m1 == -INFINITY ? 0.f : ex2_approx(m1 - mx1);
          if (move0) m0 = mx0;
          if (move1) m1 = mx1;
          l0 *= a0;
          l1 *= a1;
          const float c0 = a0 * back, c1 = a1 * back;
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            o[i][0] *= c0; o[i][1] *= c0; o[i][2] *= c1; o[i][3] *= c1;
          }
        }
        const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
        // ---- P = exp2(S - m), its sum, and P vs / vref as fp16 A fragments
        float ratio[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) ratio[i] = vref == 0.f ? 0.f : vg[i] / vref;
        uint32_t pa[kGroups][4];
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          const float rv = ratio[i >> 1];
          const float e0 = ex2_approx(s[i][0] + n0), e1 = ex2_approx(s[i][1] + n0);
          const float e2 = ex2_approx(s[i][2] + n1), e3 = ex2_approx(s[i][3] + n1);
          l0 += e0 + e1;
          l1 += e2 + e3;
          pa[i >> 1][(i & 1) * 2] = pack_half(e0 * rv, e1 * rv);
          pa[i >> 1][(i & 1) * 2 + 1] = pack_half(e2 * rv, e3 * rv);
        }
        // a code behind the cache's end may be e4m3's NaN, which a weight of zero does not cancel
        const int over = std::is_same<Code, CodeE4m3>::value ? len - (w.j + x) * kKeys : kKeys;
        // ---- O += P V: per 16 keys, this thread's columns (DP / 8) g .. of keys 2t, 2t+1, 2t+8, 2t+9
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
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t x0[4], x1[4];  // pairs of keys (0, 1) and (2, 3) at four columns
            to_half(Code{}, __byte_perm(vw[0][k], vw[1][k], 0x5140), x0[0], x0[1]);
            to_half(Code{}, __byte_perm(vw[0][k], vw[1][k], 0x7362), x0[2], x0[3]);
            to_half(Code{}, __byte_perm(vw[2][k], vw[3][k], 0x5140), x1[0], x1[1]);
            to_half(Code{}, __byte_perm(vw[2][k], vw[3][k], 0x7362), x1[2], x1[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) mma16816(o[k * 4 + c], pa[j], x0[c], x1[c]);
          }
        }
        mbar_arrive_warp(empty + st);
      }
    }
    n += part;
    // ---- this warp's part: sums over the four threads of a row, o in units of one
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      o[i][0] *= vref; o[i][1] *= vref; o[i][2] *= vref; o[i][3] *= vref;
    }
    // ---- joined over the warps of a row block: the upper half hands its part to the lower
    float4* const mo = reinterpret_cast<float4*>(smem + L::kOffMerge);
    float2* const ms = reinterpret_cast<float2*>(smem + L::kOffStat);
    for (int half = TG / 2; half >= 1; half >>= 1) {
      if (active <= half) continue;  // the upper half had no tile
      const bool gives = place >= half && place < 2 * half;
      const int slot = (gives ? place - half : place) * RBW + rb;
      if (gives) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) mo[(slot * kCols + i) * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        if (t == 0) {
          ms[slot * 16 + g] = make_float2(m0, l0);
          ms[slot * 16 + 8 + g] = make_float2(m1, l1);
        }
      }
      mbar_arrive_warp(merge);
      if (ok) ok = mbar_wait_warp(merge, merges & 1, abort_flag, p.status);
      ++merges;
      if (place < half) {
        const float2 y0 = ms[slot * 16 + g], y1 = ms[slot * 16 + 8 + g];
        const float M0 = fmaxf(m0, y0.x), M1 = fmaxf(m1, y1.x);
        const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - M0), b0 = y0.x == -INFINITY ? 0.f : ex2_approx(y0.x - M0);
        const float a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - M1), b1 = y1.x == -INFINITY ? 0.f : ex2_approx(y1.x - M1);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const float4 y = mo[(slot * kCols + i) * 32 + lane];
          o[i][0] = o[i][0] * a0 + y.x * b0;
          o[i][1] = o[i][1] * a0 + y.y * b0;
          o[i][2] = o[i][2] * a1 + y.z * b1;
          o[i][3] = o[i][3] * a1 + y.w * b1;
        }
        l0 = l0 * a0 + y0.y * b0;
        l1 = l1 * a1 + y1.y * b1;
        m0 = M0;
        m1 = M1;
      }
      mbar_arrive_warp(merge);
      if (ok) ok = mbar_wait_warp(merge, merges & 1, abort_flag, p.status);
      ++merges;
    }
    // ---- the pair's output, or this run's part of it
    if (works && place == 0) {
      const bool whole = part == w.nt;
      // a run's first part may begin inside a pair (slot 0), another one ends inside it (slot 1)
      const size_t slot = static_cast<size_t>(blockIdx.x) * 2 + (w.j > 0 ? 0 : 1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = e ? r1 : r0;
        if (r >= p.R) continue;
        const float l = e ? l1 : l0, m = e ? m1 : m0;
        const float il = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
        const size_t row = whole ? bh * p.R + r : slot * p.R + r;
        if (t == 0) {
          if (!whole) p.lse_part[row] = lse2;
          else if (p.lse) p.lse[row] = lse2 * 0.69314718055994531f;
        }
        // columns (DP / 4) t + i (element 2e of block i) and + DP / 8 (element 2e + 1)
#pragma unroll
        for (int c = 0; c < DP / 4; c += 8) {
          const int col = (DP / 4) * t + c;
          if (col >= p.d) continue;
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = o[(c + k) % kCols][2 * e + (c + k) / kCols] * il;
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
  // ---- batches without a key: O = 0, LSE = -inf, dealt to the CTAs
  if (p.cache_seqlens) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (cache_len(p.cache_seqlens, b, p.Nk, p.status, threadIdx.x == 0) > 0) continue;
      const size_t rows = static_cast<size_t>(p.Hkv) * p.R;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.o) + b * rows * p.d * (p.out_f32 ? 4 : 2));
      const size_t n16 = rows * p.d * (p.out_f32 ? 4 : 2) / 16;
      for (size_t i = threadIdx.x; i < n16; i += kConsumers * 32) dst[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (size_t i = threadIdx.x; i < rows; i += kConsumers * 32) p.lse[b * rows + i] = -INFINITY;
    }
  }
}

// Merges the parts of the pairs that lie in several runs.  CTA (c, r): if run c + 1 is the first to
// begin inside a pair, that pair's row r; four warps take every fourth part each.
template <typename OutT>
__global__ void __launch_bounds__(128) cache8_merge_kernel(const Cache8Params p, int ctas) {
  __shared__ float4 s_o[4][32];
  __shared__ float2 s_ml[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long total = total_tiles(p);
  const int c = blockIdx.x;
  const long long cut = run_start(total, c + 1, ctas);
  if (cut >= total || cut == 0) return;
  Walk w;
  w.start(p, cut, total);
  if (w.j == 0) return;  // the cut lies between two pairs
  const long long first = cut - w.j;
  const int c0 = run_of(total, first, ctas), c1 = run_of(total, first + w.nt - 1, ctas);
  // one of the cuts inside the pair works: the first (an empty run's cut comes again with the next)
  if (c > 0 && run_start(total, c, ctas) > first) return;
  for (int r = blockIdx.y; r < p.R; r += gridDim.y) {
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = c0 + warp; k0 <= c1; k0 += 16) {
      float e[4];
      float4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + 4 * u;
        // run k's part of this pair begins at its start, or where the pair begins
        const bool in = k <= c1 && run_start(total, k, ctas) < run_start(total, k + 1, ctas);
        const size_t row = (static_cast<size_t>(k) * 2 + (run_start(total, k, ctas) > first ? 0 : 1)) * p.R + r;
        e[u] = in ? p.lse_part[row] : -INFINITY;
        x[u] = in && lane * 4 < p.d ? *reinterpret_cast<const float4*>(p.o_part + row * p.d + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (e[u] == -INFINITY) continue;
        const float M = fmaxf(m, e[u]);
        const float a = m == -INFINITY ? 0.f : ex2_approx(m - M), b = ex2_approx(e[u] - M);
        acc.x = acc.x * a + x[u].x * b;
        acc.y = acc.y * a + x[u].y * b;
        acc.z = acc.z * a + x[u].z * b;
        acc.w = acc.w * a + x[u].w * b;
        l = l * a + b;
        m = M;
      }
    }
    s_o[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp == 0) {
      float M = -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) M = fmaxf(M, s_ml[u].x);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float b = s_ml[u].x == -INFINITY ? 0.f : ex2_approx(s_ml[u].x - M);
        const float4 x = s_o[u][lane];
        y.x += x.x * b; y.y += x.y * b; y.z += x.z * b; y.w += x.w * b;
        sum += s_ml[u].y * b;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t row = (static_cast<size_t>(w.b) * p.Hkv + w.h) * p.R + r;
      if (lane * 4 < p.d) {
        if constexpr (std::is_same<OutT, float>::value) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * p.d + lane * 4) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        } else {
          const OutT* tag = nullptr;
          *reinterpret_cast<uint2*>(static_cast<OutT*>(p.o) + row * p.d + lane * 4) =
              make_uint2(pack2(tag, y.x * inv, y.y * inv), pack2(tag, y.z * inv, y.w * inv));
        }
      }
      if (lane == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (M + __log2f(sum)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

// A cache of capacity 0: O = 0, LSE = -inf for every row.
__global__ void __launch_bounds__(256) cache8_none_kernel(const Cache8Params p) {
  const size_t rows = static_cast<size_t>(p.B) * p.Hkv * p.R, n16 = rows * p.d * (p.out_f32 ? 4 : 2) / 16;
  const size_t first = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = first; i < n16; i += step) static_cast<uint4*>(p.o)[i] = make_uint4(0, 0, 0, 0);
  if (p.lse)
    for (size_t i = first; i < rows; i += step) p.lse[i] = -INFINITY;
  if (first < static_cast<size_t>(p.B)) cache_len(p.cache_seqlens, static_cast<int>(first), p.Nk, p.status, true);
}

template <typename T, typename Code, int DP>
cudaError_t run(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, cudaStream_t stream) {
  auto kern = cache8_kernel<T, Code, DP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP>::kBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;  // the register split assumes the launch's allocation; never launch otherwise
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != static_cast<int>(kLaunchRegs)) return cudaErrorInvalidConfiguration;
  kern<<<p.ctas, kThreads, Layout<DP>::kBytes, stream>>>(k, v, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.ctas == 1) return e;
  const dim3 grid(p.ctas - 1, std::min(p.R, 64));
  if (p.out_f32) cache8_merge_kernel<float><<<grid, 128, 0, stream>>>(p, p.ctas);
  else cache8_merge_kernel<T><<<grid, 128, 0, stream>>>(p, p.ctas);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_t(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, attn_cache_dtype_t cache, cudaStream_t stream) {
  if (p.d <= 64)
    return cache == ATTN_CACHE_I8 ? run<T, CodeI8, 64>(k, v, p, stream) : run<T, CodeE4m3, 64>(k, v, p, stream);
  return cache == ATTN_CACHE_I8 ? run<T, CodeI8, 128>(k, v, p, stream) : run<T, CodeE4m3, 128>(k, v, p, stream);
}

}  // namespace

cudaError_t launch_cache8_none(const Cache8Params& p, cudaStream_t stream) {
  const size_t work = std::max(static_cast<size_t>(p.B) * p.Hkv * p.R * p.d / 4, static_cast<size_t>(p.B));
  cache8_none_kernel<<<static_cast<int>(std::min<size_t>((work + 255) / 256, 1u << 20)), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache8_fwd(const CUtensorMap& k, const CUtensorMap& v, const Cache8Params& p, attn_dtype_t dtype,
                              attn_cache_dtype_t cache, cudaStream_t stream) {
  return dtype == ATTN_F16 ? run_t<__half>(k, v, p, cache, stream) : run_t<__nv_bfloat16>(k, v, p, cache, stream);
}

}  // namespace attn
