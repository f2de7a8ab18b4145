// cache_weights_tc.cu -- accumulated attention weights for fp16 / bf16 on the tensor cores:
//   w_out[j] = w_in[j] + sum_r exp(scale Q_r . K_j - LSE_r)
// over the rows r = (head, query) of the key's kv head that see it.
//
// S^T = K Q^T: a key is a TMEM lane, so its sum over the rows is one thread's sum over columns -- no
// reduction over threads, no atomics, an order fixed by the sizes.  A work item is 256 keys of
// one (batch, kv head): two 128-key tiles that stay in shared memory while the rows' Q tiles
// (of up to 128 rows, as even as R allows) stream past both, which halves Q's traffic out of L2,
// the bound of a 128-key item (32 KB of Q per 128 x 128 x 128 product).  With few rows (decode)
// every item has one Q tile and K streams from HBM; up to eight rows are summed over their eight
// columns alone (8 x 8 heads of 16k-32k keys, 4 rows: 72.7 us, 6.1 TB/s; 4 us more over the tile's 32 columns).
// Items are numbered by key tile, those that the most queries see first, and dealt to the CTAs in snake
// order.  When there are fewer items than half the SMs, a cluster of CTAs takes each one's Q tiles in
// turn and adds its sums up in distributed shared memory, in order (one 2048-token prompt, 32 over 8
// heads: 45 us, 72 without).
//
// 640 threads: sixteen warps that sum (tcgen05.ld, one paired FMA and two ex2 per pair of scores), four
// for each key tile and each of its two S^T buffers of 128 columns, the buffers taken in turn;
// then a warp for the TMA loads, one MMA issuer per key tile, on two sub-partitions (one thread
// issues 16 of them in about 1700 cycles, more than they take), and one that prepares the rows'
// -LSE log2(e) and last visible keys.  2048-token prompts (B = 4, 32 over 8 heads, d = 128) take 130 us
// without and 77 us (889 TFLOP/s) with the causal mask, 86 with integer divisions in every role's walk
// over the tiles.  Measured beside 131 and 86, with those: eight summing warps and one issuer 160 and
// 116; eight warps that take a whole tile into registers first 149 and 92; two groups that halve every
// tile's columns 135 and 90; loads of 32 columns ahead of the sums 162 and 102; tiles handed over in
// parts of 64 columns, with twice the products to issue, 183 and 108.  Tiles of 256 rows, one buffer per
// key tile, halved by the two groups: beside 132 and 78, 138 and 84.
#include <algorithm>
#include <atomic>
#include <type_traits>
#include <cooperative_groups.h>
#include "cache8.cuh"

namespace attn {
namespace {

constexpr int kMaxStages = 12;  // of the Q ring, and of both K rings together
constexpr int kRing = kMaxStages / 2;
constexpr int kNl = 4;          // stages of row terms; even: a stage is read by the groups of one buffer

// Shared memory: a ring of 128-key tiles for each of an item's two, the Q ring, then the fixed part.  Every
// ring's barriers are waited for in every turn by the same threads: an issuer that waited only for its
// own tiles of a common K ring could be two turns off, where the parity says nothing.
struct Smem {
  static constexpr int kNlOff = 0;                 // [kNl][128] float
  static constexpr int kLimOff = kNlOff + kNl * 512;   // [kNl][128] int
  static constexpr int kMinOff = kLimOff + kNl * 512;  // [kNl] int: the least of them
  static constexpr int kSumOff = kMinOff + kNl * 4;    // [2][128] float: one buffer's sums for the other's warps
  static constexpr int kPartOff = kSumOff + 2 * 512;   // [2][128] float: this CTA's share of a cluster's sums
  // k_full, k_empty, q_full, q_empty [12]; nl_full, nl_empty [4]; s_full, s_free [2][2]; sum_full, sum_free [2]; drain [2]
  static constexpr int kBarOff = kPartOff + 2 * 512;
  static constexpr int kMiscOff = kBarOff + (4 * kMaxStages + 2 * kNl + 8 + 4 + 2) * 8;  // tmem base, abort flag, wait limit
  static constexpr int kBytes = kMiscOff + 16;
};

// Eight columns of this warp's TMEM lanes, waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// n / d for 0 <= n < 2^31: with m = ceil(2^(31 + s) / d), 2^s >= d, the product's error stays below 1 / d.
// (Every role finds every item by two divisions.  With the compiler's the decode case took 73.9 us, with 64
// columns 65.7, four windows of 48 queries 22.7 us; now 72.7, 54.9 and 21.6.)
struct Divisor {
  uint32_t m, s;
  explicit Divisor(uint32_t d) : s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ int of(int n) const { return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> 31 >> s); }
};

struct Item {
  int bh, key0, L;
};

// The CTA's k-th item; a cluster of `split` CTAs has one.
template <bool SPLIT>
__device__ __forceinline__ int snake(int k, int split) {
  const int G = gridDim.x, c = blockIdx.x;
  if (SPLIT) return k == 0 ? c / split : 0x7fffffff;
  return k * G + ((k & 1) ? G - 1 - c : c);
}

struct Heads {
  Divisor all, kv, query;  // B Hkv, Hkv and Nq
};
__device__ __forceinline__ Item item_of(const WeightParams& p, const Heads& heads, int idx) {
  const int tile = heads.all.of(idx);
  Item it;
  it.bh = idx - tile * (p.B * p.Hkv);
  it.key0 = tile * 256;
  it.L = cache_len(p.cache_seqlens, heads.kv.of(it.bh), p.Nk, nullptr, false);
  return it;
}

// A Q tile, and the first row of the head that its first row belongs to (kept under the causal mask when a
// head is longer than a tile).  Every role walks them, so without a division per tile.
struct Tile {
  int rb, head;
};

// From tile t on the first with a row that sees a key of the item (or one past the last): under the causal
// mask the rows of queries i >= key0 - (L - Nq) of each head, of which a tile as long as a head has one.
__device__ __forceinline__ void seek(const WeightParams& p, const Item& it, int qn, Tile& t) {
  if (!p.causal || p.Nq <= qn) return;
  const int r0 = t.rb * qn, least = it.key0 - (it.L - p.Nq);
  if (r0 >= p.R) return;
  if (r0 - t.head >= p.Nq) t.head += p.Nq;
  if (r0 - t.head < least) t.rb = (t.head + least) / qn;
}

// FEW: one Q tile per item, so the sets of summing warps take the items in turn and join no sums.
// SPLIT: a cluster of `split` CTAs per item.  (Both are compile-time: the tile walk with a step costs the
// decode case 30%.)
template <bool BF16, int DP, bool FEW, bool SPLIT>
__global__ void __launch_bounds__(640, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const WeightParams p,
                      const Heads heads, int n_items, int qn, int k_stages, int q_stages, int split) {
  constexpr int kChunks = DP / 64;
  constexpr int kTileK = 128 * DP * 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle needs aligned tiles
    if (threadIdx.x == 0) raise_status(p.status, ATTN_ERR_CUDA);
    return;
  }
  const int q_bytes = qn * DP * 2;
  uint8_t* const sK = smem;  // [key tile][stage]
  uint8_t* const sQ = smem + 2 * k_stages * kTileK;
  uint8_t* const fixed = sQ + q_stages * q_bytes;
  float* const s_nl = reinterpret_cast<float*>(fixed + Smem::kNlOff);
  int* const s_lim = reinterpret_cast<int*>(fixed + Smem::kLimOff);
  int* const s_min = reinterpret_cast<int*>(fixed + Smem::kMinOff);
  uint64_t* const k_full = reinterpret_cast<uint64_t*>(fixed + Smem::kBarOff);
  uint64_t* const k_empty = k_full + kMaxStages;
  uint64_t* const q_full = k_empty + kMaxStages;
  uint64_t* const q_empty = q_full + kMaxStages;
  uint64_t* const nl_full = q_empty + kMaxStages;
  uint64_t* const nl_empty = nl_full + kNl;
  uint64_t* const s_full = nl_empty + kNl;  // [key tile][buffer]
  uint64_t* const s_free = s_full + 4;
  uint64_t* const sum_full = s_free + 4;  // [key tile]
  uint64_t* const sum_free = sum_full + 2;
  uint64_t* const drain = sum_free + 2;
  float* const s_sum = reinterpret_cast<float*>(fixed + Smem::kSumOff);
  float* const s_part = reinterpret_cast<float*>(fixed + Smem::kPartOff);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(fixed + Smem::kMiscOff);
  const uint32_t abort_flag = smem_u32(fixed + Smem::kMiscOff + 4);
  constexpr int kSums = 16;  // summing warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 2);  // both issuers
    }
    for (int i = 0; i < kNl; ++i) {
      mbar_init(nl_full + i, 1);
      mbar_init(nl_empty + i, 8);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sum_full + i, 4);
      mbar_init(sum_free + i, 4);
      mbar_init(drain + i, 1);
    }
    abort_set(abort_flag, 0);
    wait_limit_set(abort_flag, p.wait_ns);
    mbar_init_fence();
  }
  if (warp == kSums) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_rb = (p.R + qn - 1) / qn;
  const int G = gridDim.x, rank = SPLIT ? blockIdx.x % split : 0;
  // this CTA's Q tiles of an item: those that see its keys, every split-th
  auto step = [&](const Item& it, Tile& t) {
    ++t.rb;
    seek(p, it, qn, t);
  };
  auto next_tile = [&](const Item& it, Tile& t) {
    step(it, t);
    if constexpr (SPLIT)
      for (int i = 1; i < split && t.rb < n_rb; ++i) step(it, t);
  };
  auto first_tile = [&](const Item& it) {
    Tile t{0, 0};
    seek(p, it, qn, t);
    if constexpr (SPLIT)
      for (int i = 0; i < rank && t.rb < n_rb; ++i) step(it, t);
    return t;
  };

  if (warp == kSums) {
    // ================================================================ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      uint32_t nk0 = 0, nk1 = 0, nq = 0;  // tiles issued
      bool ok = true;
      for (int k = 0; ok && k * G < n_items; ++k) {
        const int idx = snake<SPLIT>(k, split);
        if (idx >= n_items) continue;
        const Item it = item_of(p, heads, idx);
        if (it.key0 >= it.L) continue;
        Tile t = first_tile(it);
        if (t.rb >= n_rb) continue;
        for (int h = 0; ok && h < 2 && it.key0 + 128 * h < it.L; ++h) {
          const uint32_t nk = h ? nk1 : nk0, st = h * kRing + nk % k_stages;
          if (nk >= static_cast<uint32_t>(k_stages) && !mbar_wait(k_empty + st, ((nk / k_stages) - 1) & 1, abort_flag, p.status)) { ok = false; break; }
          mbar_expect_tx(k_full + st, kTileK);
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d(sK + (h * k_stages + nk % k_stages) * kTileK + c * 128 * 128, &tmK, k_full + st, c * 64, it.key0 + 128 * h, it.bh);
          nk0 += 1 - h;
          nk1 += h;
        }
        for (; ok && t.rb < n_rb; next_tile(it, t)) {
          const uint32_t st = nq % q_stages;
          if (nq >= static_cast<uint32_t>(q_stages) && !mbar_wait(q_empty + st, ((nq / q_stages) - 1) & 1, abort_flag, p.status)) { ok = false; break; }
          mbar_expect_tx(q_full + st, q_bytes);
          for (int c = 0; c < kChunks; ++c) tma_load_3d(sQ + st * q_bytes + c * qn * 128, &tmQ, q_full + st, c * 64, t.rb * qn, it.bh);
          ++nq;
        }
      }
      if (!ok || abort_read(abort_flag)) {  // let the copies land before the shared memory goes away
        for (int h = 0; h < 2; ++h) {
          const uint32_t nk = h ? nk1 : nk0;
          for (uint32_t i = nk > static_cast<uint32_t>(k_stages) ? nk - k_stages : 0; i < nk; ++i) mbar_drain(k_full + h * kRing + i % k_stages, (i / k_stages) & 1);
        }
        for (uint32_t i = nq > static_cast<uint32_t>(q_stages) ? nq - q_stages : 0; i < nq; ++i) mbar_drain(q_full + i % q_stages, (i / q_stages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kSums + 1 || warp == kSums + 2) {
    // ================================================================ MMA issuers, one per key tile
    if (lane == 0) {
      const int h = warp - kSums - 1;
      const uint32_t id = idesc_f16(BF16, false, false, 128, qn);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024), dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      uint32_t nk = 0, nq = 0, ns0 = 0, ns1 = 0;  // this ring's K tiles and the Q tiles passed; tiles put into either buffer
      bool ok = true;
      for (int k = 0; ok && k * G < n_items; ++k) {
        const int idx = snake<SPLIT>(k, split);
        if (idx >= n_items) continue;
        const Item it = item_of(p, heads, idx);
        if (it.key0 >= it.L) continue;
        Tile t = first_tile(it);
        if (t.rb >= n_rb) continue;
        const int halves = it.key0 + 128 < it.L ? 2 : 1;
        const uint32_t ks = nk % k_stages;
        if (h < halves && !mbar_wait(k_full + h * kRing + ks, (nk / k_stages) & 1, abort_flag, p.status)) { ok = false; break; }
        for (; t.rb < n_rb; next_tile(it, t), ++nq) {
          const uint32_t qs = nq % q_stages, b = nq & 1;
          if (!mbar_wait(q_full + qs, (nq / q_stages) & 1, abort_flag, p.status)) { ok = false; break; }
          if (h >= halves) {  // no keys of this tile: its share of the Q stage is done
            mbar_arrive(q_empty + qs);
            continue;
          }
          const uint32_t ns = b ? ns1 : ns0;
          if (ns > 0 && !mbar_wait(s_free + 2 * h + b, (ns - 1) & 1, abort_flag, p.status)) { ok = false; break; }
          ns0 += 1 - b;
          ns1 += b;
          tc_fence_after();
          const uint64_t kx = dK + (((h * k_stages + ks) * kTileK) >> 4), qx = dQ + ((qs * q_bytes) >> 4);
#pragma unroll
          for (int s = 0; s < DP / 16; ++s)
            mma_ss(tmem + h * 256 + b * 128, kx + (((s >> 2) * 128 * 128 + (s & 3) * 32) >> 4),
                   qx + (((s >> 2) * qn * 128 + (s & 3) * 32) >> 4), id, s > 0 ? 1u : 0u);
          mma_commit(s_full + 2 * h + b);
          mma_commit(q_empty + qs);
        }
        if (!ok) break;
        if (h < halves) {
          mma_commit(k_empty + h * kRing + ks);
          ++nk;
        }
      }
      if (!ok) {
        mma_commit(drain + h);  // every MMA issued completes before this arrives
        mbar_drain(drain + h, 0);
      }
    }
    __syncwarp();
  } else if (warp == kSums + 3) {
    // ================================================================ row terms
    uint32_t n = 0;
    bool ok = true;
    for (int k = 0; ok && k * G < n_items; ++k) {
      const int idx = snake<SPLIT>(k, split);
      if (idx >= n_items) continue;
      const Item it = item_of(p, heads, idx);
      if (it.key0 >= it.L) continue;
      const float* lse = p.lse + static_cast<size_t>(it.bh) * p.R;
      for (Tile t = first_tile(it); t.rb < n_rb; next_tile(it, t), ++n) {
        const uint32_t st = n % kNl;
        auto query = [&](int r) {  // r % Nq
          if (p.Nq <= qn) return r - heads.query.of(r) * p.Nq;
          const int i = r - t.head;
          return i >= p.Nq ? i - p.Nq : i;
        };
        float nl[4];
        int lim[4], least = 0x7fffffff;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = u * 32 + lane, r = t.rb * qn + c;
          const bool in = c < qn && r < p.R;
          const float x = in ? lse[r] : -INFINITY;
          nl[u] = x == -INFINITY ? -INFINITY : -x * 1.4426950408889634f;  // a row without a key adds nothing
          lim[u] = in ? (p.causal ? min(it.L - p.Nq + query(r), it.L - 1) : it.L - 1) : c < qn ? -1 : 0x7fffffff;
          least = min(least, lim[u]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        if (n >= kNl && !mbar_wait_warp(nl_empty + st, ((n / kNl) - 1) & 1, abort_flag, p.status)) { ok = false; break; }
        // a row without a key sees none, like those that fill up the tile: an infinity or NaN that its q
        // makes stays out.  (Not above, ahead of the wait, where the LSE may not have come yet.)
        bool none = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool out = nl[u] == -INFINITY && u * 32 < qn;
          none |= out;
          s_nl[st * 128 + u * 32 + lane] = nl[u];
          s_lim[st * 128 + u * 32 + lane] = out ? -1 : lim[u];
        }
        if (__any_sync(0xffffffffu, none)) least = -1;
        if (lane == 0) s_min[st] = least;
        mbar_arrive_warp(nl_full + st);
      }
    }
  } else {
    // ================================================================ sums
    const int h = warp >> 3;             // key tile of the item
    const uint32_t mine = (warp >> 2) & 1;       // FEW: the buffer of this set
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + h * 256;
    const uint64_t scl = f2_pack(p.scale_log2, p.scale_log2);
    uint32_t n = 0, ns = 0, joins = 0;  // Q tiles passed, tiles summed, sums joined
    bool ok = true;
    for (int k = 0; ok && k * G < n_items; ++k) {
      const int idx = snake<SPLIT>(k, split);
      if (idx >= n_items) continue;
      const Item it = item_of(p, heads, idx);
      const int key = it.key0 + h * 128 + (threadIdx.x & 127);
      const size_t at = static_cast<size_t>(it.bh) * p.Nk + key;
      const bool writes = (n & 1) == mine;  // the set that has the item's first Q tile
      int tiles = 0;
      float before = 0.f;
      if (writes && p.w_in && key < p.Nk) before = p.w_in[at];
      if (it.key0 == 0 && it.bh % p.Hkv == 0 && rank == 0 && threadIdx.x == 0) cache_len(p.cache_seqlens, it.bh / p.Hkv, p.Nk, p.status, true);
      const bool works = it.key0 + h * 128 < it.L;
      float sum = 0.f;
      if (it.key0 < it.L) {
        for (Tile t = first_tile(it); t.rb < n_rb; next_tile(it, t), ++n) {
          const uint32_t b = n & 1, st = n % kNl;
          ++tiles;
          if (b != mine) continue;
          if (!mbar_wait_warp(nl_full + st, (n / kNl) & 1, abort_flag, p.status)) { ok = false; break; }
          if (works) {
            if (!mbar_wait_warp(s_full + 2 * h + b, ns & 1, abort_flag, p.status)) { ok = false; break; }
            ++ns;
            tc_fence_after();
            const float* nl = s_nl + st * 128;
            const int* lim = s_lim + st * 128;
            const bool mask = s_min[st] < it.key0 + h * 128 + 127;  // some row of the tile sees not all these keys
            uint64_t acc0 = 0, acc1 = 0;  // pairs of zeros
            auto add = [&](auto& r, int c0) {
              auto sums = [&](auto masked) {
#pragma unroll
                for (int c = 0; c < static_cast<int>(sizeof(r) / 4); c += 4) {
                  const float4 t4 = *reinterpret_cast<const float4*>(nl + c0 + c);
                  float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), scl, f2_pack(t4.x, t4.y)));
                  float2 y = f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), scl, f2_pack(t4.z, t4.w)));
                  if constexpr (decltype(masked)::value) {  // whatever its score and LSE, a row that does not see the key adds nothing
                    const int4 l4 = *reinterpret_cast<const int4*>(lim + c0 + c);
                    if (key > l4.x) x.x = -INFINITY;
                    if (key > l4.y) x.y = -INFINITY;
                    if (key > l4.z) y.x = -INFINITY;
                    if (key > l4.w) y.y = -INFINITY;
                  }
                  acc0 = f2_add(acc0, f2_pack(ex2_approx(x.x), ex2_approx(x.y)));
                  acc1 = f2_add(acc1, f2_pack(ex2_approx(y.x), ex2_approx(y.y)));
                }
              };
              if (mask) sums(std::true_type{});
              else sums(std::false_type{});
            };
            if (FEW && p.R <= 8) {  // a decode's rows: nothing to do for the tile's other columns
              uint32_t r[8];
              tmem_ld8(tl + b * 128, r);
              tc_fence_before();
              mbar_arrive_warp(s_free + 2 * h + b);
              add(r, 0);
            } else
#pragma unroll 1
            for (int c0 = 0; c0 < qn; c0 += 32) {
              uint32_t r[32];
              tmem_ld32(tl + b * 128 + c0, r);
              tmem_ld_wait();
              tmem_reg_fence(r);
              if (c0 + 32 >= qn) {
                tc_fence_before();
                mbar_arrive_warp(s_free + 2 * h + b);  // the buffer is in registers
              }
              add(r, c0);
            }
            const float2 a = f2_unpack(f2_add(acc0, acc1));
            sum += a.x + a.y;  // tile by tile: a long sum of partial sums
          }
          mbar_arrive_warp(nl_empty + st);
        }
        if (!ok) break;
      }
      if (!FEW && tiles > 1) {  // the other buffer's tiles
        float* const other = s_sum + h * 128 + (threadIdx.x & 127);
        if (!writes) {
          if (joins > 0 && !mbar_wait_warp(sum_free + h, (joins - 1) & 1, abort_flag, p.status)) { ok = false; break; }
          *other = sum;
          mbar_arrive_warp(sum_full + h);
        }
        // both sets wait here, so that no warp can be a phase ahead when they change places
        if (!mbar_wait_warp(sum_full + h, joins & 1, abort_flag, p.status)) { ok = false; break; }
        if (writes) {
          sum += *other;
          mbar_arrive_warp(sum_free + h);
        }
        ++joins;
      }
      if constexpr (SPLIT) {
        if (writes) s_part[h * 128 + (threadIdx.x & 127)] = key < it.L ? sum : 0.f;
      } else if (writes && key < p.Nk) {
        p.w_out[at] = before + (key < it.L ? sum : 0.f);
      }
    }
  }
  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kSums) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (SPLIT) {  // the cluster's sums, rank by rank
    const auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    const Item it = item_of(p, heads, snake<SPLIT>(0, split));
    const int key = it.key0 + threadIdx.x;
    if (rank == 0 && threadIdx.x < 256 && key < p.Nk) {
      const size_t at = static_cast<size_t>(it.bh) * p.Nk + key;
      float sum = 0.f;
      for (int r = 0; r < split; ++r) sum += *cluster.map_shared_rank(s_part + threadIdx.x, r);
      p.w_out[at] = (p.w_in ? p.w_in[at] : 0.f) + sum;
    }
    cluster.sync();  // rank 0 has read the others' shared memory
  }
}

template <bool BF16, int DP, bool FEW, bool SPLIT>
cudaError_t run(const CUtensorMap& q, const CUtensorMap& k, const WeightParams& p, int qn, int split, cudaStream_t stream) {
  // 208 KB for the rings: two Q stages (more gain nothing), the rest for K, six tiles of 128 columns with few
  // rows and four with many
  constexpr int kTileK = 128 * DP * 2, kData = 208 * 1024;
  const int q_bytes = qn * DP * 2;
  const int q_stages = 2;
  const int k_stages = std::min(kRing, (kData - q_stages * q_bytes) / (2 * kTileK));
  auto kern = weights_tc_kernel<BF16, DP, FEW, SPLIT>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = once_per_device(ready, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kData + Smem::kBytes);
  });
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(p.B) * p.Hkv * ((p.Nk + 255) / 256);
  const int grid = static_cast<int>(SPLIT ? items * split : std::min<long long>(items, 152));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(640);
  cfg.dynamicSmemBytes = 2 * k_stages * kTileK + q_stages * q_bytes + Smem::kBytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, q, k, p, Heads{Divisor(p.B * p.Hkv), Divisor(p.Hkv), Divisor(p.Nq)}, static_cast<int>(items), qn, k_stages, q_stages, split);
}

}  // namespace

cudaError_t launch_cache_weights_tc(const CUtensorMap& q, const CUtensorMap& k, const WeightParams& p, int q_rows, attn_dtype_t dtype,
                                    cudaStream_t stream) {
  const bool few = p.R <= q_rows;
  const long long items = static_cast<long long>(p.B) * p.Hkv * ((p.Nk + 255) / 256);
  int split = 1;
  const int q_tiles = (p.R + q_rows - 1) / q_rows;
  while (!few && split < 8 && items * 2 * split <= 152 && 2 * split <= q_tiles) split *= 2;
  // the first keys of a causal prompt have twice the average's Q tiles: two CTAs for them, the light ones
  // in a second wave (two prompts of 2048: 74 -> 55 us, one of 4096: 140 -> 85; without a mask 68 -> 81 and 130 -> 147)
  if (split == 1 && p.causal && items <= 152 && q_tiles >= 16) split = 2;
  auto pick = [&](auto bf16, auto dp) {
    constexpr bool kB = decltype(bf16)::value;
    constexpr int kD = decltype(dp)::value;
    if (few) return run<kB, kD, true, false>(q, k, p, q_rows, 1, stream);
    return split > 1 ? run<kB, kD, false, true>(q, k, p, q_rows, split, stream) : run<kB, kD, false, false>(q, k, p, q_rows, 1, stream);
  };
  auto by_d = [&](auto bf16) {
    return p.d <= 64 ? pick(bf16, std::integral_constant<int, 64>{}) : pick(bf16, std::integral_constant<int, 128>{});
  };
  return dtype == ATTN_BF16 ? by_d(std::true_type{}) : by_d(std::false_type{});
}

}  // namespace attn
