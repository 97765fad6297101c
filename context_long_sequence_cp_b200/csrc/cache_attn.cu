// cache_attn.cu — attention of a few new tokens of each sequence over its key/value
// cache (sm_100a, tcgen05 + TMEM + TMA): single tokens when decoding, chains or trees of
// drafted tokens when several are checked at once.
//
// The rows of a product are the (token, query head) pairs that share a key/value head, up
// to 128 of them (a query tile: whole tokens of G = Hq / Hkv rows each), so a cache row is
// read once for each query tile: once in all where T <= floor(128 / G). Token t sees the cached keys
// [0, lengths[b]) and, among the drafted ones (cache rows lengths[b] + u), those whose
// bit u is set in its tree word. Softmax, lse and partials are those of attn_fwd.cu.
//
// Bound: HBM, the cache read once per query tile (4 D bytes per key and key/value head; the
// later tiles of a head come at other times, so what they share in L2 is chance: 65536 keys,
// 4 key/value heads of 16 query heads, 64 tokens in eight tiles 200 us, 8 tokens in one 53). The 128-key
// tiles of all (sequence, head, query tile) units are laid end to end and cut into equal
// runs, one per CTA (one CTA per SM), so uneven lengths leave no SM idle. A run that
// covers a unit whole writes its output; pieces of a unit go to fp32 slots, two per CTA,
// that a second kernel joins by their maxima. Within a CTA two softmax warpgroups take
// the even and the odd key tiles, each with its own maximum, sum and accumulator (joined
// at the unit's end), so that one's softmax runs under the other's products.
//
// Measured, 131040 cached keys, 8 key/value heads of 4 query heads, D = 128, at an SM clock of
// 1965 MHz: 32 drafted tokens 108 us, of them 97 in the first kernel (5.5 TB/s, 0.85 of the copy
// rate) and 9 in the join, which starts when the last CTA is done; one token 94 us. Run without
// a pause the card reaches its power limit and the clock falls to 1490 MHz: 127 to 140 us
// and 112, so there the softmax's chain per tile bounds it and not HBM. Sixteen sequences of 0
// to 8176 keys, 16 drafted tokens each: 63 us, 4.3 TB/s (73 at 1730 MHz): about two units per
// CTA, whose start and end are not hidden under another's products. P is kept to 2^-17 in two
// bf16 terms, so that a row of a partial is as exact as its fp32 type says.
//
// Cache rows that no token sees, past the last key or a tree's padding, are never read as
// values: their scores are set to -inf and their rows of V are cleared in shared memory, so
// stale NaNs there do no harm.
#include "cache_attn.h"

#include <cmath>
#include <cstring>
#include <new>

#include "cp_attn.h"
#include "geometry.h"
#include "plan_view.h"
#include "sm100.cuh"

namespace cpattn {

using namespace sm100;

namespace {

constexpr int kCacheThreads = 384;
constexpr float kCacheRescale = 8.0f;   // log2 units: rescale when the maximum grows by > 256x
constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
constexpr int kBlock = kTile * 128;     // 128 rows x 128 B

template <int D>
struct CacheCfg {
  static constexpr int kBlocks = D / 64;
  static constexpr int kTileBytes = kBlocks * kBlock;
  static constexpr int kStages = D == 128 ? 5 : 11;
};

template <int D>
struct alignas(1024) CacheSmem {
  uint8_t q[CacheCfg<D>::kTileBytes];
  uint8_t kv[CacheCfg<D>::kStages][CacheCfg<D>::kTileBytes];
  uint64_t kv_full[CacheCfg<D>::kStages], kv_empty[CacheCfg<D>::kStages];
  uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_done[2], ml_ready, unit_done, drain;
  float2 ml[2][kTile];               // (max, sum) of each warpgroup's rows
  int2 before[kCacheMaxB + 1];       // see CacheSpan
  int2 warp_sum[kCacheThreads / 32];
  uint32_t tmem_base;
  WaitBlock wblk;
};
static_assert(sizeof(CacheSmem<128>) + 1024 <= 232448, "CacheSmem exceeds the per-CTA limit");
static_assert(sizeof(CacheSmem<64>) + 1024 <= 232448, "CacheSmem exceeds the per-CTA limit");

// Keys of sequence b: cached plus drafted; -1 for a length outside the cache.
__device__ __forceinline__ int key_count(const CacheParams& p, int b) {
  const int len = __ldg(p.lengths + b), extra = p.own ? p.T : 0;
  return len < 0 || len > p.cap - extra ? -1 : len + extra;
}

// The work of all units, laid end to end in slots and cut into equal runs, one per CTA: a
// unit's key tiles, after kUnitSlots empty slots that stand for its start and end (queries
// loaded, accumulators joined and written: about two tiles' time), from two tiles per CTA on.
// Measured without and with them, uneven lengths on 148 SMs: 128 tiles 11.9 and 12.7 us (fewer
// CTAs get tiles at all), 304 tiles 17.5 and 16.3, 608 tiles 27.8 and 19.0, 4480 tiles 93.7
// and 65.1.
constexpr int kUnitSlots = 2;
struct CacheSpan {
  const int2* before;   // key tiles of the sequences before b, and those of them that have keys
  int units;            // units of a sequence
  int extra;            // empty slots per unit
  int per, more;        // CTA c holds `per` slots, and one more where c < more
  __device__ __forceinline__ int start(int c) const { return c * per + min(c, more); }
  __device__ __forceinline__ int holder(int f) const {   // the CTA that holds slot f
    const int wide = more * (per + 1);
    return f < wide ? f / (per + 1) : more + (f - wide) / per;
  }
  __device__ __forceinline__ int slots_before(int b) const { return (before[b].x + extra * before[b].y) * units; }
  __device__ __forceinline__ int tiles(int b) const { return before[b + 1].x - before[b].x; }
};

// Fills before[0 .. B], by all threads of the block.
template <int THREADS>
__device__ __forceinline__ CacheSpan cache_span(const CacheParams& p, int2* before, int2* warp_sum) {
  int2 carry = make_int2(0, 0);
  if (threadIdx.x == 0) before[0] = carry;
  for (int b0 = 0; b0 < p.B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int2 v = make_int2(b < p.B ? (max(key_count(p, b), 0) + kTile - 1) / kTile : 0, 0);
    v.y = v.x > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ux = __shfl_up_sync(0xffffffffu, v.x, o), uy = __shfl_up_sync(0xffffffffu, v.y, o);
      if ((threadIdx.x & 31) >= o) {
        v.x += ux;
        v.y += uy;
      }
    }
    if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v.x += carry.x;
    v.y += carry.y;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x >> 5)) {
        v.x += warp_sum[w].x;
        v.y += warp_sum[w].y;
      }
      carry.x += warp_sum[w].x;
      carry.y += warp_sum[w].y;
    }
    if (b < p.B) before[b + 1] = v;
    __syncthreads();
  }
  CacheSpan s;
  s.before = before;
  s.units = p.Hkv * p.row_tiles;
  s.extra = static_cast<int64_t>(carry.x) * s.units >= 2 * p.n_cta ? kUnitSlots : 0;
  const int total = (carry.x + carry.y * s.extra) * s.units;   // the plan keeps it in int32
  s.per = total / p.n_cta;
  s.more = total - s.per * p.n_cta;
  return s;
}

// A run of key tiles of one unit (sequence b, key/value head hk, query tile rt); n may be
// 0 where the piece holds empty slots only.
struct CacheSeg {
  int b, hk, rt;
  int t0, n, nt;   // key tiles [t0, t0 + n) of nt
  int next;        // slot after the piece
};
// The piece of the slots that starts at f and ends at `end` at most.
__device__ __forceinline__ CacheSeg seg_at(const CacheParams& p, const CacheSpan& sp, int f, int end) {
  int lo = 0, hi = p.B - 1;   // last b that starts at f or before: never a sequence without keys
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sp.slots_before(mid) <= f) lo = mid;
    else hi = mid - 1;
  }
  CacheSeg s;
  s.b = lo;
  s.nt = sp.tiles(lo);
  const int rem = f - sp.slots_before(lo), len = s.nt + sp.extra;
  const int u = rem / len, pos = rem - u * len;
  s.hk = u / p.row_tiles;
  s.rt = u - s.hk * p.row_tiles;
  const int stop = min(pos + end - f, len);
  s.next = f + stop - pos;
  s.t0 = max(pos - sp.extra, 0);
  s.n = max(stop - sp.extra, 0) - s.t0;
  return s;
}

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tS, uint32_t q, uint32_t k) {
  const uint64_t dq = smem_desc_sw128(q, 16, 1024), dk = smem_desc_sw128(k, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kBlock + (kk & 3) * 32) >> 4;
    umma_ss_elect(tS, dq + off, dk + off, kIdescQK, kk > 0);
  }
}
// O (+)= P V over keys [16 KK0, 16 KK1): P is two bf16 terms, 32 columns of a score tile
// holding the high ones of their 32 keys, then the low ones.
template <int D, int KK0, int KK1>
__device__ __forceinline__ void issue_av(uint32_t tO, uint32_t tS, uint32_t v, bool accumulate) {
  const uint64_t dv = smem_desc_sw128(v, kBlock, 1024);
#pragma unroll
  for (int kk = KK0; kk < KK1; ++kk) {
    const uint32_t tP = tS + (kk >> 1) * 32 + (kk & 1) * 8;
    umma_ts_elect(tO, tP, dv + ((kk * 2048) >> 4), idesc_bf16_f32(128, D, 0, 1), accumulate || kk > 0);
    umma_ts_elect(tO, tP + 16, dv + ((kk * 2048) >> 4), idesc_bf16_f32(128, D, 0, 1), 1u);
  }
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
// Which of 32 columns a row sees: those before `lim` (cached keys), and from there on those
// of the drafted tokens' word.
__device__ __forceinline__ uint32_t keep_bits(uint64_t word, int lim) {
  const uint64_t tree = lim >= 32 || lim <= -64 ? 0ull : lim >= 0 ? word << lim : word >> -lim;
  return static_cast<uint32_t>(low_bits(lim) | tree);
}
__device__ __forceinline__ void mask_scores(uint32_t (&s)[32], uint32_t keep) {
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j] = keep >> j & 1u ? s[j] : 0xff800000u;   // -inf
}

// OR over the lanes of a warp.
__device__ __forceinline__ uint64_t any_lane(uint64_t x) {
  const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x));
  return static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x >> 32))) << 32 | lo;
}

// Row r of the query tile: which token and query head, and where its results go.
struct CacheRow {
  bool valid;
  int t, hq;
};
__device__ __forceinline__ CacheRow cache_row(const CacheParams& p, int hk, int rt, int r) {
  CacheRow c;
  const int tl = r / p.G;
  c.t = rt * p.tok_per_tile + tl;
  c.hq = hk * p.G + (r - tl * p.G);
  c.valid = tl < p.tok_per_tile && c.t < p.T;
  return c;
}
__device__ __forceinline__ void store_lse(const CacheParams& p, int b, const CacheRow& c, float lse) {
  if (p.lse == nullptr) return;
  if (p.o_part != nullptr) p.lse[(static_cast<int64_t>(b) * p.T + c.t) * p.Hq + c.hq] = lse;
  else p.lse[(static_cast<int64_t>(b) * p.Hq + c.hq) * p.T + c.t] = lse;
}

// 1 / sum and lse of a row; a row that sees nothing gets 0 and -inf, a NaN stays one.
__device__ __forceinline__ float inv_sum(float l) { return l > 0.f ? 1.f / l : l == 0.f ? 0.f : l; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}

template <int D>
__global__ void __launch_bounds__(kCacheThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheParams p) {
  using C = CacheCfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  CacheSmem<D>& sm = *reinterpret_cast<CacheSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                      ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_addr(&sm.kv_full[s]), 1);
      mbar_init(smem_addr(&sm.kv_empty[s]), 1);
    }
    mbar_init(smem_addr(&sm.q_full), 1);
    mbar_init(smem_addr(&sm.q_empty), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&sm.s_full[w]), 1);
      mbar_init(smem_addr(&sm.p_full[w][0]), 128);
      mbar_init(smem_addr(&sm.p_full[w][1]), 128);
      mbar_init(smem_addr(&sm.o_done[w]), 1);
    }
    mbar_init(smem_addr(&sm.ml_ready), 256);
    mbar_init(smem_addr(&sm.unit_done), 256);
    mbar_init(smem_addr(&sm.drain), 1);
    wait_block_init(sm.wblk, p.status, p.wait_limit_ns);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may get ready
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  const CacheSpan span = cache_span<kCacheThreads>(p, sm.before, sm.warp_sum);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const WaitCtl ctl = wait_ctl(sm.wblk);
  const int f0 = span.start(static_cast<int>(blockIdx.x)), f1 = span.start(static_cast<int>(blockIdx.x) + 1);
  auto wait = [&](uint64_t& bar, int phase) { return __all_sync(0xffffffffu, mbar_wait(smem_addr(&bar), phase & 1, ctl)); };

  if (warp == 9) {
    // ---------------------------------------------------------------- TMA
    const uint64_t pol = l2_policy_evict_first();
    bool ok = true;
    int kv = 0, unit = 0, q_loads = 0;
    for (int f = f0; f < f1 && ok;) {
      const CacheSeg s = seg_at(p, span, f, f1);
      f = s.next;
      if (s.n == 0) continue;
      // K(0), K(1), then V(i), K(i + 2): the order the products take them. The first of a unit
      // are loaded before its Q, which waits for the unit before to have read its own.
      bool q_loaded = false;
      for (int j = 0; j < 2 * s.n; ++j, ++kv) {
        if (j == (s.n == 1 ? 1 : 2)) {
          if (unit > 0 && !(ok = wait(sm.q_empty, unit - 1))) break;
          q_loaded = true;
          mbar_arrive_expect_tx_elect(smem_addr(&sm.q_full), C::kBlocks * p.G * p.tok_per_tile * 128);
          for (int blk = 0; blk < C::kBlocks; ++blk)
            tma_load_4d_elect(smem_addr(&sm.q[0]) + blk * kBlock, &tm_q, smem_addr(&sm.q_full), blk * 64, s.hk * p.G,
                              s.rt * p.tok_per_tile, s.b, pol);
        }
        const int key = j == 0 ? 0 : s.n == 1 ? -1 : j == 1 ? 1 : (j & 1) && (j + 1) / 2 < s.n ? (j + 1) / 2 : -1;
        const int tile = key >= 0 ? key : j == 2 * s.n - 1 ? s.n - 1 : (j - 2) / 2;
        const int st = kv % NS;
        if (kv >= NS && !(ok = wait(sm.kv_empty[st], kv / NS - 1))) break;
        mbar_arrive_expect_tx_elect(smem_addr(&sm.kv_full[st]), C::kTileBytes);
        for (int blk = 0; blk < C::kBlocks; ++blk)
          tma_load_4d_elect(smem_addr(&sm.kv[st][0]) + blk * kBlock, key >= 0 ? &tm_k : &tm_v,
                            smem_addr(&sm.kv_full[st]), blk * 64, s.hk, (s.t0 + tile) * kTile, s.b, pol);
      }
      q_loads += q_loaded;
      ++unit;
    }
    if (!ok) {   // abort: let every load this warp issued land before the CTA exits
      for (int k = kv - NS; k < kv; ++k)
        if (k >= 0) mbar_wait_drain(smem_addr(&sm.kv_full[k % NS]), (k / NS) & 1, p.wait_limit_ns);
      if (q_loads > 0) mbar_wait_drain(smem_addr(&sm.q_full), (q_loads - 1) & 1, p.wait_limit_ns);
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA
    const uint32_t q = smem_addr(&sm.q[0]);
    const uint32_t tS[2] = {tbase, tbase + 128}, tO[2] = {tbase + 256, tbase + 256 + D};
    bool ok = true, issued = false;
    int kv = 0, unit = 0, cnt[2] = {0, 0};
    for (int f = f0; f < f1 && ok;) {
      const CacheSeg s = seg_at(p, span, f, f1);
      f = s.next;
      if (s.n == 0) continue;
      if (!(ok = wait(sm.q_full, unit))) break;
      for (int i = 0; i < 2 && i < s.n; ++i, ++kv) {
        const int st = kv % NS;
        if (!(ok = wait(sm.kv_full[st], kv / NS))) break;
        tc_fence_after();
        issue_qk<D>(tS[i], q, smem_addr(&sm.kv[st][0]));
        umma_commit_elect(smem_addr(&sm.s_full[i]));
        umma_commit_elect(smem_addr(&sm.kv_empty[st]));
        if (i + 1 == s.n) umma_commit_elect(smem_addr(&sm.q_empty));
        issued = true;
      }
      for (int i = 0; i < s.n && ok; ++i) {
        const int w = i & 1;
        const int vs = kv % NS;
        if (!(ok = wait(sm.kv_full[vs], kv / NS))) break;
        ++kv;
        const bool next = i + 2 < s.n;
        int ks = 0;
        if (next) {
          ks = kv % NS;
          if (!(ok = wait(sm.kv_full[ks], kv / NS))) break;
          ++kv;
        }
        const uint32_t v = smem_addr(&sm.kv[vs][0]);
        if (!(ok = wait(sm.p_full[w][0], cnt[w]))) break;
        tc_fence_after();
        issue_av<D, 0, 4>(tO[w], tS[w], v, i >= 2);
        if (!(ok = wait(sm.p_full[w][1], cnt[w]))) break;
        tc_fence_after();
        issue_av<D, 4, 8>(tO[w], tS[w], v, true);
        ++cnt[w];
        if (i + 2 >= s.n) umma_commit_elect(smem_addr(&sm.o_done[w]));
        umma_commit_elect(smem_addr(&sm.kv_empty[vs]));
        if (next) {
          issue_qk<D>(tS[w], q, smem_addr(&sm.kv[ks][0]));
          umma_commit_elect(smem_addr(&sm.s_full[w]));
          umma_commit_elect(smem_addr(&sm.kv_empty[ks]));
          if (i + 3 == s.n) umma_commit_elect(smem_addr(&sm.q_empty));   // the unit's last scores
        }
      }
      ++unit;
    }
    if (issued) {   // every product and commit has to finish before TMEM is freed
      umma_commit_elect(smem_addr(&sm.drain));
      mbar_wait_drain(smem_addr(&sm.drain), 0, p.wait_limit_ns);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_off + wg * 128;
    const uint32_t tO = tbase + lane_off + 256 + wg * D;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int kv = 0, unit = 0, s_cnt = 0, od_cnt = 0;
    for (int f = f0; f < f1 && ok;) {
      const CacheSeg sg = seg_at(p, span, f, f1);
      f = sg.next;
      if (sg.n == 0) continue;
      const CacheRow cr = cache_row(p, sg.hk, sg.rt, row);
      const bool busy = __any_sync(0xffffffffu, cr.valid);   // a warp without rows only keeps the barriers' pace
      const int len = __ldg(p.lengths + sg.b), keys = len + (p.own ? p.T : 0);
      uint64_t word = 0;   // drafted tokens this row sees
      if (p.own && cr.valid)
        word = p.tree == nullptr ? low_bits(cr.t + 1)
                                 : __ldg(p.tree + static_cast<int64_t>(sg.b) * p.T + cr.t) & low_bits(p.T);
      uint64_t mine = low_bits(p.T);   // this lane's part of the drafted tokens that some token sees
      if (p.own && p.tree != nullptr) {
        const unsigned long long* words = p.tree + static_cast<int64_t>(sg.b) * p.T;
        mine = (lane < p.T ? __ldg(words + lane) : 0) | (lane + 32 < p.T ? __ldg(words + lane + 32) : 0);
      }
      // The accumulators and (max, sum) rows of the unit before have been read by both warpgroups.
      if (unit > 0 && !(ok = wait(sm.unit_done, unit - 1))) break;
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = wg; i < sg.n; i += 2) {
        if (!(ok = wait(sm.s_full[wg], s_cnt))) break;
        ++s_cnt;
        tc_fence_after();
        const int k0 = (sg.t0 + i) * kTile;
        if (len - k0 < kTile) {
          // A tile past the cached keys: clear the rows of V that no token sees, whatever the
          // cache holds there. V of tile i is load 2 i + 2 of the piece, of its last tile the last.
          const int idx = kv + min(2 * i + 2, 2 * sg.n - 1), end = min(keys - k0, kTile);
          const uint64_t seen = any_lane(mine);
          if (!(ok = wait(sm.kv_full[idx % NS], idx / NS))) break;
          uint8_t* v = &sm.kv[idx % NS][0];
          auto clear = [&](int r, int vec) {
            *reinterpret_cast<uint4*>(v + (vec / 8) * kBlock + r * 128 + (vec % 8) * 16) = make_uint4(0, 0, 0, 0);
          };
          for (int e = row; e < (kTile - end) * 8 * C::kBlocks; e += 128)
            clear(end + e / (8 * C::kBlocks), e % (8 * C::kBlocks));
          if (p.own && (~seen & low_bits(p.T)))
            for (int r = max(len - k0, 0) + row / (8 * C::kBlocks); r < end; r += 128 / (8 * C::kBlocks))
              if (!(seen >> (k0 + r - len) & 1)) clear(r, row % (8 * C::kBlocks));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (busy) {
          // Two walks over the row's scores, 32 columns at a time from TMEM: the maximum, then
          // the exponentials, P written over the columns just read. (Holding all 128 scores
          // needs the registers of both and straight-line code that outruns the instruction cache.)
          const int lim = len - k0;   // columns below it are cached keys
          float mt = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * c, s);
            if (lim < kTile) mask_scores(s, keep_bits(word, lim - 32 * c));
#pragma unroll
            for (int j = 0; j < 32; j += 2) mt = max3(mt, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          }
          // Online softmax with a lazily moved maximum, as in attn_fwd.cu.
          const float m_prev = m_run;
          const bool resc = mt * sl2 - m_run > kCacheRescale;   // false while both are -inf
          if (resc) m_run = mt * sl2;
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const float alpha = resc ? ex2_approx(m_prev - m_run) : 1.f;
          l_run *= alpha;
          if (i >= 2 && __any_sync(0xffffffffu, resc)) {
            // The accumulator holds the products before this tile, all complete.
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(tO + c, o);
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
              tmem_st16(tO + c, o);
            }
          }
          const uint64_t sl2_2 = f2_pack(sl2, sl2), nm_2 = f2_pack(-m_use, -m_use);
          float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32], hi[16], lo[16];
            tmem_ld32(tS + 32 * c, s);
            if (lim < kTile) mask_scores(s, keep_bits(word, lim - 32 * c));
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), sl2_2, nm_2), x0, x1);
              const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
              l0 += e0;
              l1 += e1;
              hi[j] = pack_bf16x2(e0, e1);
              f2_unpack(f2_sub(f2_pack(e0, e1), bf16x2_to_f2(hi[j])), x0, x1);
              lo[j] = pack_bf16x2(x0, x1);
            }
            tmem_st16(tS + 32 * c, hi);
            tmem_st16(tS + 32 * c + 16, lo);
            if (c & 1) {   // half the keys: their part of P V may start
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(smem_addr(&sm.p_full[wg][c >> 1]));
            }
          }
          l_run += l0 + l1;
        } else {
          mbar_arrive(smem_addr(&sm.p_full[wg][0]));
          mbar_arrive(smem_addr(&sm.p_full[wg][1]));
        }
      }
      if (!ok) break;
      kv += 2 * sg.n;
      // ---------------------------------------------------------- unit's end
      const bool two = sg.n > 1;
      if (wg == 0 || two) {
        if (!(ok = wait(sm.o_done[wg], od_cnt))) break;
        ++od_cnt;
      }
      sm.ml[wg][row] = make_float2(m_run, l_run);
      mbar_arrive(smem_addr(&sm.ml_ready));
      if (!(ok = wait(sm.ml_ready, unit))) break;
      tc_fence_after();
      const float2 m0 = sm.ml[0][row], m1 = sm.ml[1][row];
      const float M = fmaxf(m0.x, m1.x);
      const float a0 = m0.x == -INFINITY ? 0.f : ex2_approx(m0.x - M);
      const float a1 = m1.x == -INFINITY ? 0.f : ex2_approx(m1.x - M);
      const float l = m0.y * a0 + m1.y * a1;
      const bool whole = sg.n == sg.nt;
      // A unit cut at this CTA's start goes to its first slot, one cut at its end to the second.
      float* slot = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (sg.t0 > 0 ? 0 : 1)) * (kTile * (D + 2));
      const float inv = whole ? inv_sum(l) : 1.f;
      const int64_t out = (static_cast<int64_t>(sg.b) * p.T + cr.t) * p.Hq + cr.hq;
      if (busy) {
#pragma unroll
        for (int c = wg * (D / 2); c < (wg + 1) * (D / 2); c += 16) {
          uint32_t x0[16], x1[16];
          tmem_ld16(tbase + lane_off + 256 + c, x0);
          if (two) tmem_ld16(tbase + lane_off + 256 + D + c, x1);
          float y[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            y[q] = __uint_as_float(x0[q]) * a0;
            if (two) y[q] = fmaf(__uint_as_float(x1[q]), a1, y[q]);
            y[q] *= inv;
          }
          if (cr.valid) {
            if (!whole || p.o_part != nullptr) {
              float4* dst = reinterpret_cast<float4*>(whole ? p.o_part + out * D + c : slot + row * D + c);
#pragma unroll
              for (int q = 0; q < 4; ++q) dst[q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.o + out * D + c);
#pragma unroll
              for (int q = 0; q < 2; ++q)
                dst[q] = make_uint4(pack_bf16x2(y[8 * q], y[8 * q + 1]), pack_bf16x2(y[8 * q + 2], y[8 * q + 3]),
                                    pack_bf16x2(y[8 * q + 4], y[8 * q + 5]), pack_bf16x2(y[8 * q + 6], y[8 * q + 7]));
            }
          }
        }
      }
      if (wg == 0 && cr.valid) {
        if (whole) store_lse(p, sg.b, cr, row_lse(M, l));
        else *reinterpret_cast<float2*>(slot + kTile * D + 2 * row) = make_float2(M, l);
      }
      tc_fence_before();
      mbar_arrive(smem_addr(&sm.unit_done));
      ++unit;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the pieces of the units that were cut, one warp per row; writes the rows of
// sequences without keys (O = 0, lse = -inf) and of those whose length lies outside the
// cache (NaN).
template <int D>
__global__ void __launch_bounds__(256) cache_join_kernel(const __grid_constant__ CacheParams p, int row_blocks) {
  __shared__ int2 before[kCacheMaxB + 1];
  __shared__ int2 warp_sum[8];
  const CacheSpan span = cache_span<256>(p, before, warp_sum);
  __syncthreads();
  // Launched while the attention kernel still runs: wait for its results.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = static_cast<int>(blockIdx.x) / row_blocks;
  const int row = (static_cast<int>(blockIdx.x) % row_blocks) * 8 + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int b = unit / span.units, u = unit - b * span.units;
  const CacheRow cr = cache_row(p, u / p.row_tiles, u % p.row_tiles, row);
  if (row >= kTile || !cr.valid) return;
  const int nt = span.tiles(b);
  constexpr int kPer = D / 16;   // columns of a lane: half a warp spans the row, the halves take every other piece
  const int half = lane >> 4, col = (lane & 15) * kPer;
  float acc[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) acc[q] = 0.f;
  float lse = -INFINITY, inv = 0.f;
  if (nt == 0) {
    if (key_count(p, b) < 0) {
      lse = __int_as_float(0x7fc00000);
#pragma unroll
      for (int q = 0; q < kPer; ++q) acc[q] = lse;
      inv = 1.f;
    }
  } else {
    const int first = span.slots_before(b) + u * (nt + span.extra) + span.extra;   // slot of the first tile
    const int c0 = span.holder(first), c1 = span.holder(first + nt - 1);
    if (c0 == c1) return;   // written whole
    // A piece that starts inside the unit lies in its CTA's first slot, else in the second.
    auto slot_of = [&](int c) {
      return p.parts + (2 * static_cast<int64_t>(c) + (span.start(c) > first ? 0 : 1)) * (kTile * (D + 2));
    };
    // A lane per piece: the joint maximum and sum first, so that the sums' loads do not wait
    // on one another.
    float M = -INFINITY, l = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, slot_of(c)[kTile * D + 2 * row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int cb = c0; cb <= c1; cb += 32) {
      const int c = cb + lane;
      const float* slot = c <= c1 ? slot_of(c) : nullptr;
      float w = 0.f;
      if (slot != nullptr) {
        const float2 ml = *reinterpret_cast<const float2*>(slot + kTile * D + 2 * row);
        w = ml.x == -INFINITY ? ml.y : ex2_approx(ml.x - M);   // a sum without a maximum is 0 or NaN
        l = fmaf(ml.y, w, l);
      }
      const int np = min(32, c1 - cb + 1);
#pragma unroll 4
      for (int k = 0; k < np; k += 2) {
        const float wk = __shfl_sync(0xffffffffu, w, k + half);   // 0 past the last piece
        if (wk == 0.f) continue;                                  // its rows may hold anything
        const float4* from = reinterpret_cast<const float4*>(slot_of(cb + k + half) + row * D + col);
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
          const float4 v = from[q];
          acc[4 * q] = fmaf(v.x, wk, acc[4 * q]);
          acc[4 * q + 1] = fmaf(v.y, wk, acc[4 * q + 1]);
          acc[4 * q + 2] = fmaf(v.z, wk, acc[4 * q + 2]);
          acc[4 * q + 3] = fmaf(v.w, wk, acc[4 * q + 3]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) acc[q] += __shfl_xor_sync(0xffffffffu, acc[q], 16);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    inv = inv_sum(l);
    lse = row_lse(M, l);
  }
  const int64_t out = ((static_cast<int64_t>(b) * p.T + cr.t) * p.Hq + cr.hq) * D + col;
  if (half == 0) {
#pragma unroll
    for (int q = 0; q < kPer; q += 4) {
      const float y[4] = {acc[q] * inv, acc[q + 1] * inv, acc[q + 2] * inv, acc[q + 3] * inv};
      if (p.o_part != nullptr)
        *reinterpret_cast<float4*>(p.o_part + out + q) = make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2*>(p.o + out + q) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
  }
  if (lane == 0) store_lse(p, b, cr, lse);
}

template <int D>
bool launch_cache(const CacheLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(CacheSmem<D>) + 1024;
  auto kern = cache_attn_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  kern<<<L.p.n_cta, kCacheThreads, smem, stream>>>(L.tm_q, L.tm_k, L.tm_v, L.p);
  if (cudaGetLastError() != cudaSuccess) return false;
  const int rows = L.p.tok_per_tile * L.p.G;
  const int row_blocks = (rows + 7) / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.p.B * L.p.Hkv * L.p.row_tiles * row_blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D>, L.p, row_blocks) == cudaSuccess;
}

}  // namespace

}  // namespace cpattn

using namespace cpattn;

struct cp_cache_plan_s {
  int B, Hq, Hkv, D, cap, T;
  float scale;
  int device = -1, sms = 148;
  int* d_status = nullptr;
};

namespace {

// Query tiles: as many whole tokens (G rows each) as fit 128 rows.
int tokens_per_tile(const cp_cache_plan_s& c) {
  const int g = c.Hq / c.Hkv;
  return c.T < kTile / g ? c.T : kTile / g;
}

size_t cache_workspace(const cp_cache_plan_s& c) {
  return static_cast<size_t>(2) * c.sms * kTile * (c.D + 2) * sizeof(float);
}

int run_cache(cp_cache_plan_t plan, const void* q, const void* k, const void* v, const int32_t* lengths, int own,
              const int64_t* tree, void* o, float* o_part, float* lse, void* workspace, cp_stream_t stream) {
  if (plan == nullptr || q == nullptr || k == nullptr || v == nullptr || lengths == nullptr ||
      (o == nullptr && o_part == nullptr))
    return CP_ERR_INVALID_ARG;
  if (own != 0 && own != 1) return CP_ERR_INVALID_ARG;
  if (!is_aligned16(q) || !is_aligned16(k) || !is_aligned16(v) || !is_aligned16(o) || !is_aligned16(o_part) ||
      !is_aligned16(workspace) || (reinterpret_cast<uintptr_t>(lengths) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 || (reinterpret_cast<uintptr_t>(tree) & 7u) != 0)
    return CP_ERR_ALIGNMENT;
  if (workspace == nullptr) return CP_ERR_WORKSPACE;
  if (plan->d_status == nullptr) return CP_ERR_CUDA;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return CP_ERR_CUDA;
  if (dev != plan->device) return CP_ERR_INVALID_ARG;
  // Other CTAs read the cache, and the join reads the lengths again. Only the bf16 output may be
  // the queries themselves: a CTA that writes rows has read them, and no other one does.
  const size_t rows = static_cast<size_t>(plan->B) * plan->T * plan->Hq;
  const size_t cache = sizeof(__nv_bfloat16) * plan->B * plan->cap * plan->Hkv * plan->D;
  const size_t q_bytes = rows * plan->D * sizeof(__nv_bfloat16);
  if (overlaps({{o, q_bytes}, {o_part, rows * plan->D * sizeof(float)}, {lse, rows * sizeof(float)},
                {workspace, cache_workspace(*plan)}},
               {{o == q ? nullptr : q, q_bytes}, {k, cache}, {v, cache}, {lengths, plan->B * sizeof(int32_t)},
                {tree, static_cast<size_t>(plan->B) * plan->T * sizeof(int64_t)}}))
    return CP_ERR_INVALID_ARG;
  CacheLaunch L;
  CacheParams& p = L.p;
  p.B = plan->B;
  p.Hq = plan->Hq;
  p.Hkv = plan->Hkv;
  p.T = plan->T;
  p.G = plan->Hq / plan->Hkv;
  p.cap = plan->cap;
  p.own = own;
  p.tok_per_tile = tokens_per_tile(*plan);
  p.row_tiles = (plan->T + p.tok_per_tile - 1) / p.tok_per_tile;
  p.n_cta = plan->sms;
  p.scale_log2 = plan->scale * 1.4426950408889634f;
  p.lengths = lengths;
  p.tree = reinterpret_cast<const unsigned long long*>(tree);
  p.parts = static_cast<float*>(workspace);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o_part = o_part;
  p.lse = lse;
  p.status = plan->d_status;
  p.wait_limit_ns = kWaitLimitNs;
  if (!encode_map_4d(&L.tm_q, q, plan->D, plan->Hq, plan->T, plan->B, p.G, p.tok_per_tile) ||
      !encode_map_4d(&L.tm_k, k, plan->D, plan->Hkv, plan->cap, plan->B, 1, kTile) ||
      !encode_map_4d(&L.tm_v, v, plan->D, plan->Hkv, plan->cap, plan->B, 1, kTile))
    return CP_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return (plan->D == 128 ? launch_cache<128>(L, st) : launch_cache<64>(L, st)) ? CP_OK : CP_ERR_CUDA;
}

}  // namespace

extern "C" {

int cp_cache_plan(cp_cache_plan_t* out, int B, int Hq, int Hkv, int D, int capacity, int T, float softmax_scale) {
  if (out == nullptr) return CP_ERR_INVALID_ARG;
  *out = nullptr;
  if (B < 1 || Hq < 1 || Hkv < 1 || capacity < 1 || T < 1) return CP_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale)) return CP_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return CP_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0 || Hq / Hkv > kTile || T > kCacheMaxT || B > kCacheMaxB) return CP_ERR_UNSUPPORTED;
  // Tile counts, row blocks of the join and cache rows are int32.
  if (capacity > (1 << 30) || Hq > (1 << 20)) return CP_ERR_UNSUPPORTED;
  const int64_t tiles = (static_cast<int64_t>(capacity) + kTile - 1) / kTile;
  const int64_t per_tile = kTile / (Hq / Hkv);
  const int64_t units = static_cast<int64_t>(B) * Hkv * ((T + per_tile - 1) / per_tile);
  if (units * (kTile / 8) > INT32_MAX || units * (tiles + kUnitSlots) > INT32_MAX) return CP_ERR_UNSUPPORTED;
  cp_cache_plan_s* c = new (std::nothrow) cp_cache_plan_s;
  if (c == nullptr) return CP_ERR_CUDA;
  c->B = B;
  c->Hq = Hq;
  c->Hkv = Hkv;
  c->D = D;
  c->cap = capacity;
  c->T = T;
  c->scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(static_cast<float>(D));
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) == cudaSuccess && ndev > 0) {
    int sms = 0;
    if (cudaGetDevice(&c->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess || sms <= 0 ||
        cudaMalloc(&c->d_status, sizeof(int)) != cudaSuccess) {
      delete c;
      return CP_ERR_CUDA;
    }
    if (cudaMemset(c->d_status, 0, sizeof(int)) != cudaSuccess) {
      cudaFree(c->d_status);
      delete c;
      return CP_ERR_CUDA;
    }
    c->sms = sms;
  }
  *out = c;
  return CP_OK;
}

int cp_cache_plan_destroy(cp_cache_plan_t plan) {
  if (plan == nullptr) return CP_OK;
  if (plan->d_status != nullptr) cudaFree(plan->d_status);
  delete plan;
  return CP_OK;
}

size_t cp_cache_attn_workspace_bytes(cp_cache_plan_t plan) { return plan == nullptr ? 0 : cache_workspace(*plan); }

int cp_cache_attn(cp_cache_plan_t plan, const void* q, const void* k_cache, const void* v_cache, const int32_t* lengths,
                  const int64_t* tree, void* o, float* lse, void* workspace, cp_stream_t stream) {
  if (o == nullptr) return CP_ERR_INVALID_ARG;
  return run_cache(plan, q, k_cache, v_cache, lengths, 1, tree, o, nullptr, lse, workspace, stream);
}

int cp_cache_attn_partial(cp_cache_plan_t plan, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* lengths, int own_drafts, const int64_t* tree, float* o_part, float* lse_part,
                          void* workspace, cp_stream_t stream) {
  if (o_part == nullptr || lse_part == nullptr) return CP_ERR_INVALID_ARG;
  return run_cache(plan, q, k_cache, v_cache, lengths, own_drafts, tree, nullptr, o_part, lse_part, workspace, stream);
}

int cp_cache_check(cp_cache_plan_t plan, cp_stream_t stream) {
  if (plan == nullptr) return CP_ERR_INVALID_ARG;
  if (plan->d_status == nullptr) return CP_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return CP_ERR_CUDA;
  int status = 0;
  if (cudaMemcpy(&status, plan->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return CP_ERR_CUDA;
  if (status != 0) {
    cudaMemset(plan->d_status, 0, sizeof(int));
    return status;
  }
  return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // extern "C"
