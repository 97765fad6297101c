// linattn.cu — causal linear attention with a decay for each head (sm_100a,
// tcgen05 + TMEM + TMA), its gradients, and its recurrent form.
//
//   S_t = d S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   d = exp(log_decay[h]).
//
// One engine computes the output and every gradient. For rows a, b, c and a state Z0,
//   y_i = s_in sum_{j<=i} d^(i-j) (a_i . b_j) c_j + s_st d^(i+e) a_i^T Z0
// in one direction over the tokens:
//   o  : a, b, c = q, k, v     Z0 = S_0      e = 1   forward
//   dq : a, b, c = do, v, k    Z0 = S_0^T    e = 1   forward
//   dk : a, b, c = v, do, q    Z0 = dS_T^T   e = 0   backward over the tokens
//   dv : a, b, c = k, q, do    Z0 = dS_T     e = 0   backward; its final state is dS_0
// (sum_i d^(i+1) scale q_i do_i^T + d^S dS_T).
//
// Chunked form, chunks of 128 tokens (never across a rank's piece). With Z the state
// before a chunk of L tokens and p the row's index in walking order:
//   Y  = ((A B^T) o M) C + diag(d^(p+e)) A Z,   M_pj = d^(p-j) for j <= p,
//   Z' = d^L Z + B^T diag(d^(L-1-p+1-e)) C.
// Four products on the tensor core per chunk; the chunk's decay mask is built from 32
// powers of d and three row factors, so no exponential is taken per score.
//
// A CTA walks a run of chunks ("segment") of one (batch, head); Z stays in the registers
// of eight warps in fp32. Sequences with few (batch, head) are cut into segments: a first
// launch (OUT = false) computes each segment's own state, and the second, launched early,
// joins those before it at its start.
//
// Bound. The forward cannot do without 8 bytes per element (164 us for 32768 tokens, 32 heads,
// D = 128, at the card's copy rate); the two launches read B and C twice. Measured there, at an
// SM clock of 1965 MHz: 308 us, a quarter of them for the segments' states, and 351 (a third) where
// a last state is asked for; run without a pause, where the card's power limit holds the clock at
// 1640 to 1665 MHz, 363 and 413. With loads that all hit L2 302 instead of 320, so HBM is not what
// bounds it; the time follows the clock. A chunk takes
// ~5600 cycles of an SM, the tensor core ~2400 of them: the chain of the state's warps
// (weight C, the product, add, publish Z) and that of the score warps (scores, P, the
// product, output) meet once per chunk, and each is about that long. Not kept, measured:
// eight score warps (333 us: 96 registers a thread spill), output staged over A for a ring of
// six tiles (323), Z published after the next weighting (321), loads of TMEM a block ahead
// (319), parts of a segment's state on CTAs of their own (322).
//
// Precision. Where the last state is asked for, the state is exact to fp32: the weighted
// rows of C are split into three bf16 terms (8 + 8 + 8 bits of the fp32 product) multiplied
// one after the other; two terms (2^-17) do where it is only read as bf16 operand. The
// chunk sum starts from zero in TMEM and is added to d^L Z in registers, d^L as an fp32
// pair, because the tensor core's accumulation truncates and a long run of it would
// drift. Rounded to bf16: the masked scores (P), and the state where it is multiplied
// by A (Z); both once, as operands.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "cp_attn.h"
#include "linattn.h"
#include "plan_view.h"
#include "sm100.cuh"

namespace cpattn {

using namespace sm100;

namespace {

constexpr int kChunk = 128;          // tokens of a chunk: the 128 lanes of a tcgen05 product
constexpr int kBlk = kChunk * 128;   // 128 rows x 128 B: one swizzled 64-column block
constexpr int kHalf = kChunk / 2;    // tokens of C that one group of four warps weights

template <int D, bool OUT, int TERMS>
struct LinCfg {
  static constexpr int kBlocks = D / 64;
  static constexpr int kTileBytes = kBlocks * kBlk;       // a 128 x D tile
  static constexpr int kPerChunk = OUT ? 3 : 2;           // tiles per chunk: [A,] B, C
  static constexpr int kTiles = D == 128 ? (OUT ? 5 : 6) : (OUT ? 9 : 10);
  // Warps 0-7 weight C and hold the state; 8-11 (OUT) scores and output; then the issuers: the
  // chunk state's products, the TMA, and (OUT) the other products. Two issuing warps, because
  // one spends longer on its waits and commits than the tensor core on the products.
  static constexpr int kKvWarp = OUT ? 12 : 8, kTmaWarp = kKvWarp + 1, kOutWarp = kKvWarp + 2;
  static constexpr int kThreads = 32 * (OUT ? kOutWarp + 1 : kOutWarp);
  // Tokens a group of four warps weights at a time, and the buffers it alternates between.
  static constexpr int kStep = OUT && TERMS == 3 ? 32 : 64;
  static constexpr int kBufs = OUT ? 1 : 2;
  static constexpr int kSteps = kHalf / kStep;
  // TMEM columns: chunk state, transposed [0,128); weighted C^T from 128 on, a buffer's
  // terms side by side in bf16 pairs; with OUT: scores, P over their lower half [256,384),
  // output [384,512).
  static constexpr int kBufCols = TERMS * kStep / 2;
  static constexpr int kTmemCols = 512;
  static_assert(2 * kBufs * kBufCols <= (OUT ? 128 : 384), "weighted C^T columns");
};
constexpr int kColCw = 128, kColS = 256, kColY = 384;
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);   // A B^T
// A Z: both operands K-major. C^T B and P C: left operand in TMEM, right MN-major.
__host__ __device__ constexpr uint32_t idesc_az(int D) { return idesc_bf16_f32(128, D, 0, 0); }
__host__ __device__ constexpr uint32_t idesc_ts(int D) { return idesc_bf16_f32(128, D, 0, 1); }

template <int D, bool OUT, int TERMS>
struct alignas(1024) LinSmem {
  using C = LinCfg<D, OUT, TERMS>;
  uint8_t tile[C::kTiles][C::kTileBytes];            // ring of 128 x D tiles
  uint8_t z[OUT ? D * D * 2 : 1024];                 // bf16 Z^T: row = feature of C, 64-column blocks
  uint8_t y[OUT ? D / 64 : 1][OUT ? 4 : 1][OUT ? 32 * 128 : 1024];   // output: 32 rows x 64 columns per warp
  uint64_t full[C::kTiles], empty[C::kTiles];
  uint64_t cw_ready[2][2], cw_free[2][2];            // per group of weighting warps and buffer
  uint64_t s_full, p_ready, kv_done, kv_free, az_done, z_ready, y_full, y_free, drain[2];
  float diag[64];                                    // fast decays: [32 + x] = s_in d^x for x = 0 .. 31
  float2 w_full[kChunk / 2], w_tail[kChunk / 2];     // weights of the rows of C, of a whole and of a tail chunk
  uint32_t tmem_base;
  WaitBlock wblk;
};
static_assert(sizeof(LinSmem<128, true, 2>) + 1024 <= 232448, "LinSmem exceeds the per-CTA limit");
static_assert(sizeof(LinSmem<64, true, 2>) + 1024 <= 232448, "LinSmem exceeds the per-CTA limit");
static_assert(sizeof(LinSmem<128, false, 2>) + 1024 <= 232448, "LinSmem exceeds the per-CTA limit");
static_assert(sizeof(LinSmem<64, false, 2>) + 1024 <= 232448, "LinSmem exceeds the per-CTA limit");

// Decays slow enough that d^-128 stays below e^48: see the score warps.
constexpr double kSlowDecay = -48.0 / kChunk;

// Descriptor moved by a byte offset (the address field counts 16-byte units).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Four transposed 8 x 8 bf16 matrices: matrix m's rows (16 bytes) are at the addresses of
// lanes 8m .. 8m + 7; lane t gets column t / 4, rows 2 (t % 4) and the next.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes x 4 columns of TMEM from two such fragments: lanes t / 4 and 8 + t / 4 of column t % 4.
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, uint32_t r0, uint32_t r1) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r0), "r"(r1) : "memory");
}

// TMA store of a box from shared memory, one thread; its own group.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// This thread's stores: the sources of all but the newest N groups have been read; all are complete.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// d^n; n = 0 gives 1 also for d = 0.
__device__ __forceinline__ double decay_pow(double ld, int64_t n) {
  return n == 0 ? 1.0 : exp(ld * static_cast<double>(n));
}

// The chunks in walking order: where a chunk's rows are. Moved on by counting, since the
// divisions would sit in every role's way once per chunk.
struct ChunkWalk {
  int piece, off, len;
  __device__ __forceinline__ ChunkWalk(const LinParams& p, int ci) {
    const int cn = p.reverse ? p.nch - 1 - ci : ci;
    piece = cn / p.chunks_per_piece;
    off = (cn - piece * p.chunks_per_piece) * kChunk;
    len = min(kChunk, p.piece_len - off);
  }
  __device__ __forceinline__ void next(const LinParams& p) {
    off += p.reverse ? -kChunk : kChunk;
    if (off < 0 || off >= p.piece_len) {
      piece += p.reverse ? -1 : 1;
      off = p.reverse ? (p.chunks_per_piece - 1) * kChunk : 0;
    }
    len = min(kChunk, p.piece_len - off);
  }
  __device__ __forceinline__ bool whole() const { return len == kChunk; }
  // Zigzag: rank r holds piece r, then piece 2N - 1 - r.
  __device__ __forceinline__ int rank(const LinParams& p) const {
    return !p.zigzag || piece < p.N ? piece : 2 * p.N - 1 - piece;
  }
  __device__ __forceinline__ int token(const LinParams& p) const {   // first row, within the rank
    return (!p.zigzag || piece < p.N ? 0 : p.piece_len) + off;
  }
};
// Tokens walked before chunk ci.
__device__ __forceinline__ int walked_before(const LinParams& p, int ci) {
  if (ci >= p.nch) return p.S;
  const ChunkWalk c(p, ci);
  const int p0 = c.piece * p.piece_len + c.off;
  return p.reverse ? p.S - p0 - c.len : p0;
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// One arrival for a warp whose lanes have all fenced what they publish.
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&bar));
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One CTA per (scan, segment, batch, head). The backward's three scans are one launch: they
// are independent, so their CTAs fill the waves together, and those of one place in the
// sequence, which read the same rows, run next to each other. The direction is a run-time
// flag: as a template parameter it put three copies of the code side by side on the GPU, and
// a chunk took twice as long for want of instructions.
template <int D, bool OUT, int TERMS>
__global__ void __launch_bounds__(LinCfg<D, OUT, TERMS>::kThreads, 1)
    linattn_kernel(const __grid_constant__ LinLaunch launch) {
  const LinScan& L = launch.scan[blockIdx.x % launch.scans];
  const LinParams& p = L.p;
  const CUtensorMap &tm_a = L.tm_a, &tm_b = L.tm_b, &tm_c = L.tm_c, &tm_y = L.tm_y;
  const bool back = p.reverse;
  const int place = static_cast<int>(blockIdx.x) / launch.scans;
  const int bh = place % p.units;
  const int seg = OUT && back ? p.nseg - 1 - place / p.units : place / p.units;   // in walking order
  using C = LinCfg<D, OUT, TERMS>;
  constexpr int NT = C::kTiles;
  // Order of a chunk's tiles in the ring: A is the first to be free, so the next chunk's A and B
  // load while this one is multiplied.
  constexpr int kTA = 0, kTB = OUT ? 1 : 0, kTC = OUT ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  LinSmem<D, OUT, TERMS>& sm = *reinterpret_cast<LinSmem<D, OUT, TERMS>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = bh % p.H, b = bh / p.H;
  const int ci0 = static_cast<int>(static_cast<int64_t>(seg) * p.nch / p.nseg);
  const int ci1 = static_cast<int>(static_cast<int64_t>(seg + 1) * p.nch / p.nseg);
  const int n = ci1 - ci0;
  const double ld = static_cast<double>(__ldg(p.log_decay + h));
  const int tail = p.piece_len % kChunk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NT; ++s) {
      mbar_init(smem_addr(&sm.full[s]), 1);
      mbar_init(smem_addr(&sm.empty[s]), OUT ? 2 : 1);   // a commit of each reader of the tile
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(smem_addr(&sm.cw_ready[s >> 1][s & 1]), 4);
      mbar_init(smem_addr(&sm.cw_free[s >> 1][s & 1]), 1);
    }
    mbar_init(smem_addr(&sm.s_full), 1);
    mbar_init(smem_addr(&sm.p_ready), 4);
    mbar_init(smem_addr(&sm.kv_done), 1);
    mbar_init(smem_addr(&sm.kv_free), 8);
    mbar_init(smem_addr(&sm.az_done), 1);
    mbar_init(smem_addr(&sm.z_ready), 8);
    mbar_init(smem_addr(&sm.y_full), 1);
    mbar_init(smem_addr(&sm.y_free), 4);
    mbar_init(smem_addr(&sm.drain[0]), 1);
    mbar_init(smem_addr(&sm.drain[1]), 1);
    wait_block_init(sm.wblk, p.status, p.wait_limit_ns);
    fence_barrier_init();
  }
  const bool slow = ld >= kSlowDecay;
  if (OUT && threadIdx.x < 64)
    sm.diag[threadIdx.x] = threadIdx.x < 32 ? 0.f : static_cast<float>(decay_pow(ld, threadIdx.x - 32)) * p.s_in;
  if (threadIdx.x < 256) {
    const int r = threadIdx.x & 127, len = threadIdx.x < 128 ? kChunk : tail;
    const float w = r < len ? static_cast<float>(decay_pow(ld, back ? r + 1 : len - 1 - r)) * p.s_upd : 0.f;
    reinterpret_cast<float*>(threadIdx.x < 128 ? sm.w_full : sm.w_tail)[r] = w;
  }
  if (warp == C::kKvWarp) {
    tmem_alloc(smem_addr(&sm.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  if (!OUT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the rows' launch may get ready
  if (warp == C::kTmaWarp && lane == 0) {
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const WaitCtl ctl = wait_ctl(sm.wblk);
  float* zt_smem = reinterpret_cast<float*>(&sm.tile[0][0]);   // D x D, rows D + 1 apart
  static_assert(D * (D + 1) * 4 <= sizeof(sm.tile), "transposed state");
  const uint32_t tCw = tbase + kColCw, tS = tbase + kColS, tY = tbase + kColY;
  auto wait = [&](uint64_t& bar, int phase) { return all_ok(mbar_wait(smem_addr(&bar), phase & 1, ctl)); };
  auto tile_full = [&](int t) { return wait(sm.full[t % NT], t / NT); };

  if (warp == C::kTmaWarp) {
    // ---------------------------------------------------------------- TMA
    const uint64_t pol = l2_policy_evict_first();
    bool ok = true;
    int t = 0;
    // The ring holds less than two chunks, so the one after next is brought into L2 ahead.
    ChunkWalk ahead(p, ci0), c = ahead;
    auto prefetch = [&]() {
      ahead.next(p);
      const int rb = ahead.rank(p) * p.B + b, t0 = ahead.token(p);
      for (int which = 0; which < C::kPerChunk; ++which)
        for (int blk = 0; blk < C::kBlocks; ++blk)
          tma_prefetch_4d_elect(which == kTC ? &tm_c : which == kTB ? &tm_b : &tm_a, blk * 64, h, t0, rb);
    };
    if (n > 1) prefetch();
    for (int i = 0; i < n && ok; ++i, c.next(p)) {
      const int rb = c.rank(p) * p.B + b, t0 = c.token(p);
      if (i + 2 < n) prefetch();
      for (int which = 0; which < C::kPerChunk; ++which, ++t) {
        const int st = t % NT;
        if (t >= NT && !(ok = wait(sm.empty[st], t / NT - 1))) break;
        const uint32_t bar = smem_addr(&sm.full[st]);
        const CUtensorMap* map = which == kTC ? &tm_c : which == kTB ? &tm_b : &tm_a;
        mbar_arrive_expect_tx_elect(bar, C::kTileBytes);
        for (int blk = 0; blk < C::kBlocks; ++blk)
          tma_load_4d_elect(smem_addr(&sm.tile[st][0]) + blk * kBlk, map, bar, blk * 64, h, t0, rb, pol);
      }
    }
    if (!ok)   // abort: let every load this warp issued land before the CTA exits
      for (int k = t - NT; k < t; ++k)
        if (k >= 0) mbar_wait_drain(smem_addr(&sm.full[k % NT]), (k / NT) & 1, p.wait_limit_ns);
  } else if (warp == C::kKvWarp) {
    // ---------------------------------------- MMA: C^T B of a chunk, onto the chunk state
    constexpr uint32_t kIdescTS = idesc_ts(D);
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const int tB = i * C::kPerChunk + kTB, tC = i * C::kPerChunk + kTC;
      if (!(ok = tile_full(tB))) break;
      if (i > 0 && !(ok = wait(sm.kv_free, i - 1))) break;
      const uint64_t dB = smem_desc_sw128(smem_addr(&sm.tile[tB % NT][0]), kBlk, 1024);
      // As the weighted rows of C come, smallest term first.
#pragma unroll 1
      for (int part = 0; part < 2 * C::kSteps; ++part) {
        const int g = part & 1, step = part >> 1, u = i * C::kSteps + step, buf = u % C::kBufs;
        if (!(ok = wait(sm.cw_ready[g][buf], u / C::kBufs))) break;
        tc_fence_after();
        const uint64_t d = desc_at(dB, (g * kHalf + step * C::kStep) * 128);
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int kk = 0; kk < C::kStep / 16; ++kk)
            umma_ts_elect(tbase, tCw + (g * C::kBufs + buf) * C::kBufCols + term * (C::kStep / 2) + kk * 8,
                          desc_at(d, kk * 2048), kIdescTS, part > 0 || term > 0 || kk > 0);
        umma_commit_elect(smem_addr(&sm.cw_free[g][buf]));
      }
      if (!ok) break;
      umma_commit_elect(smem_addr(&sm.kv_done));
      umma_commit_elect(smem_addr(&sm.empty[tB % NT]));
      umma_commit_elect(smem_addr(&sm.empty[tC % NT]));   // its rows have been weighted
    }
    if (n > 0) {   // every product and commit has to finish before TMEM is freed
      umma_commit_elect(smem_addr(&sm.drain[0]));
      mbar_wait_drain(smem_addr(&sm.drain[0]), 0, p.wait_limit_ns);
    }
  } else if (OUT && warp == C::kOutWarp) {
    // ------------------------------------------- MMA: A Z, P C, and the next chunk's scores
    constexpr uint32_t kIdescAZ = idesc_az(D), kIdescTS = idesc_ts(D);
    const uint64_t dZ = smem_desc_sw128(smem_addr(&sm.z[0]), 16, 1024);
    bool ok = true;
    auto tile_addr = [&](int t) { return smem_addr(&sm.tile[t % NT][0]); };
#pragma unroll 1
    for (int j = 0; j <= n && ok; ++j) {
      const int i = j - 1;
      const int tA = i * C::kPerChunk + kTA, tC = i * C::kPerChunk + kTC;
      if (j > 0) {
        // A Z, onto the columns the output warps have read for the previous chunk.
        if (!(ok = wait(sm.z_ready, i))) break;
        if (i > 0 && !(ok = wait(sm.y_free, i - 1))) break;
        tc_fence_after();
        const uint64_t dA = smem_desc_sw128(tile_addr(tA), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_elect(tY, desc_at(dA, (kk >> 2) * kBlk + (kk & 3) * 32),
                        desc_at(dZ, (kk >> 2) * (D * 128) + (kk & 3) * 32), kIdescAZ, kk > 0);
        umma_commit_elect(smem_addr(&sm.az_done));
        umma_commit_elect(smem_addr(&sm.empty[tA % NT]));
        if (!(ok = tile_full(tC))) break;
        if (!(ok = wait(sm.p_ready, i))) break;   // P written (and A Z scaled): P C adds to A Z
        tc_fence_after();
        const uint64_t dC = smem_desc_sw128(tile_addr(tC), kBlk, 1024);
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk)
          umma_ts_elect(tY, tS + kk * 8, desc_at(dC, kk * 2048), kIdescTS, 1u);
        umma_commit_elect(smem_addr(&sm.y_full));
        umma_commit_elect(smem_addr(&sm.empty[tC % NT]));
      }
      if (j < n) {   // scores of chunk j, over the P whose product was issued before
        const int sA = j * C::kPerChunk + kTA, sB = j * C::kPerChunk + kTB;
        if (!(ok = tile_full(sA)) || !(ok = tile_full(sB))) break;
        tc_fence_after();
        const uint64_t dA = smem_desc_sw128(tile_addr(sA), 16, 1024), dB = smem_desc_sw128(tile_addr(sB), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBlk + (kk & 3) * 32;
          umma_ss_elect(tS, desc_at(dA, off), desc_at(dB, off), kIdescS, kk > 0);
        }
        umma_commit_elect(smem_addr(&sm.s_full));
        umma_commit_elect(smem_addr(&sm.empty[sA % NT]));
        umma_commit_elect(smem_addr(&sm.empty[sB % NT]));
      }
    }
    if (n > 0) {
      umma_commit_elect(smem_addr(&sm.drain[1]));
      mbar_wait_drain(smem_addr(&sm.drain[1]), 0, p.wait_limit_ns);
    }
  } else if (warp < 8) {
    // ---------------------- weighted C^T in bf16 terms, and the state; lanes are features of C
    const int quad = warp & 3, grp = warp >> 2;
    const int row = quad * 32 + lane;          // feature of C (column of Z)
    const int col0 = grp * (D / 2);            // features of B (rows of Z) held by this thread
    const bool busy = quad * 32 < D;           // warp-uniform; for D = 64 two quads have no rows
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const double d_full = decay_pow(ld, kChunk), d_tail = decay_pow(ld, tail);
    const float hi_full = static_cast<float>(d_full), hi_tail = static_cast<float>(d_tail);
    const float lo_full = static_cast<float>(d_full - static_cast<double>(hi_full));
    const float lo_tail = static_cast<float>(d_tail - static_cast<double>(hi_tail));
    float z[D / 2];
#pragma unroll
    for (int q = 0; q < D / 2; ++q) z[q] = 0.f;
    const int64_t state0 = static_cast<int64_t>(bh) * D * D;
    // A segment's own state is kept in the order the threads hold it: vector q of (group, row) at
    // q * 2D + group * D + row, so that a warp's accesses are contiguous.
    const int zt = grp * D + row;
    if (OUT && busy) {
      const int x = walked_before(p, ci0);
      if (p.z0 != nullptr) {
        const float w = static_cast<float>(decay_pow(ld, x));
#pragma unroll
        for (int q = 0; q < D / 2; ++q) {
          const int col = col0 + q;
          z[q] = w * __ldg(p.z0 + state0 + (p.z0_transposed ? row * D + col : col * D + row));
        }
      }
      // Launched while the segments' states are still being computed.
      if (p.nseg > 1) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int g = 0; g < seg; ++g) {
        const int end = walked_before(p, static_cast<int>(static_cast<int64_t>(g + 1) * p.nch / p.nseg));
        const float w = x == end ? 1.f : expf(static_cast<float>(ld * (x - end)));
        const float4* src = reinterpret_cast<const float4*>(
                                p.zseg + (static_cast<int64_t>(bh) * (p.nseg - 1) + g) * (D * D)) + zt;
#pragma unroll
        for (int q = 0; q < D / 8; ++q) {
          const float4 v = src[q * (2 * D)];
          z[4 * q] = fmaf(w, v.x, z[4 * q]);
          z[4 * q + 1] = fmaf(w, v.y, z[4 * q + 1]);
          z[4 * q + 2] = fmaf(w, v.z, z[4 * q + 2]);
          z[4 * q + 3] = fmaf(w, v.w, z[4 * q + 3]);
        }
      }
    }
    bool ok = true;
    // Steps in order; the state after chunk i is taken kAhead steps into chunk i + 1 (with two
    // buffers one step is weighted while the tensor core finishes the chunk).
    constexpr int kAhead = C::kBufs - 1;
    const int steps = n * C::kSteps;
    ChunkWalk cv(p, ci0), cz = cv;   // chunk being weighted, chunk whose state is taken
    int zi = 0;   // chunks whose state has been added
#pragma unroll 1
    for (int u = 0; u < steps + kAhead && ok; ++u) {
      if (OUT && u == zi * C::kSteps + (zi > 0 ? kAhead : 0) && zi < n) {   // bf16 Z^T for A Z of chunk zi
        if (zi > 0 && !(ok = wait(sm.az_done, zi - 1))) break;
        if (busy) {
#pragma unroll
          for (int v = 0; v < D / 16; ++v) {
            const int col = col0 + 8 * v;
            *reinterpret_cast<uint4*>(
                &sm.z[(col / 64) * (D * 128) + row * 128 + ((((col % 64) / 8) ^ (row & 7)) * 16)]) =
                make_uint4(pack_bf16x2(z[8 * v], z[8 * v + 1]), pack_bf16x2(z[8 * v + 2], z[8 * v + 3]),
                           pack_bf16x2(z[8 * v + 4], z[8 * v + 5]), pack_bf16x2(z[8 * v + 6], z[8 * v + 7]));
          }
        }
        fence_async_smem();
        warp_arrive(sm.z_ready);
      }
      if (u < steps) {
        // This warp's 32 features of one step's tokens into a TMEM buffer.
        const int i = u / C::kSteps, step = u % C::kSteps, buf = u % C::kBufs;
        const int tC = i * C::kPerChunk + kTC;
        if (step == 0 && !(ok = tile_full(tC))) break;
        if (u >= C::kBufs && !(ok = wait(sm.cw_free[grp][buf], u / C::kBufs - 1))) break;
        if (busy) {
          const bool whole = cv.whole();
          // The features: 16-byte vectors quad * 4 .. + 3 of the tile's rows (tokens).
          const uint32_t src = smem_addr(&sm.tile[tC % NT][0]) + (quad >> 1) * kBlk;
#pragma unroll 1
          for (int k = 0; k < C::kStep / 8; ++k) {   // 8 tokens at a time
            const int tok = grp * kHalf + step * C::kStep + 8 * k;
            uint32_t r[4], t[TERMS][4];
            ldmatrix_x4_trans(src + (tok + (lane & 7)) * 128 + ((((quad & 1) * 4 + (lane >> 3)) ^ (lane & 7)) * 16), r);
            const int pair = tok / 2 + (lane & 3);   // this lane's two tokens
            const float2 w = whole ? sm.w_full[pair] : sm.w_tail[pair];
            if (!whole) {   // rows past the chunk's tokens may hold anything
#pragma unroll
              for (int m = 0; m < 4; ++m)
                r[m] = 2 * pair + 1 < tail ? r[m] : 2 * pair < tail ? r[m] & 0xffffu : 0u;
            }
            const uint64_t ww = f2_pack(w.x, w.y);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              uint64_t x = f2_mul(bf16x2_to_f2(r[m]), ww);
#pragma unroll
              for (int e = TERMS - 1; e >= 0; --e) {   // term 0 is the smallest
                float x0, x1;
                f2_unpack(x, x0, x1);
                t[e][m] = pack_bf16x2(x0, x1);
                if (e > 0) x = f2_sub(x, bf16x2_to_f2(t[e][m]));
              }
            }
            const uint32_t dst = tCw + lane_off + (grp * C::kBufs + buf) * C::kBufCols + 4 * k;
#pragma unroll
            for (int e = 0; e < TERMS; ++e) {
              tmem_st_16x128b(dst + e * (C::kStep / 2), t[e][0], t[e][1]);
              tmem_st_16x128b(dst + e * (C::kStep / 2) + (16u << 16), t[e][2], t[e][3]);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        warp_arrive(sm.cw_ready[grp][buf]);
        if (step == C::kSteps - 1) cv.next(p);
      }
      if (u == (zi + 1) * C::kSteps + kAhead - 1) {   // the state after chunk zi
        if (!(ok = wait(sm.kv_done, zi))) break;
        tc_fence_after();
        const float hi = cz.whole() ? hi_full : hi_tail, lo = cz.whole() ? lo_full : lo_tail;
        const uint64_t hi2 = f2_pack(hi, hi), lo2 = f2_pack(lo, lo);
        cz.next(p);
        if (busy) {
#pragma unroll
          for (int q = 0; q < D / 2; q += 32) {
            uint32_t t0[32];
            tmem_ld32(tbase + lane_off + col0 + q, t0);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const uint64_t zz = f2_pack(z[q + k], z[q + k + 1]);
              const uint64_t sum = f2_pack(__uint_as_float(t0[k]), __uint_as_float(t0[k + 1]));
              f2_unpack(f2_fma(zz, hi2, f2_fma(zz, lo2, sum)), z[q + k], z[q + k + 1]);
            }
          }
        }
        tc_fence_before();
        if (++zi < n) warp_arrive(sm.kv_free);
      }
    }
    if (ok && busy) {
      if (!OUT) {
        float4* dst = reinterpret_cast<float4*>(
                          p.zseg + (static_cast<int64_t>(bh) * (p.nseg - 1) + seg) * (D * D)) + zt;
#pragma unroll
        for (int q = 0; q < D / 8; ++q)
          dst[q * (2 * D)] = make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
        if (p.zseg_t != nullptr) {   // through the ring's memory, whose tiles have all been read
#pragma unroll
          for (int q = 0; q < D / 2; ++q) zt_smem[(col0 + q) * (D + 1) + row] = z[q];
        }
      } else if (seg == p.nseg - 1 && p.z_out != nullptr) {
#pragma unroll
        for (int q = 0; q < D / 2; ++q) p.z_out[state0 + static_cast<int64_t>(col0 + q) * D + row] = z[q];
      }
    }
  } else if (OUT && warp < 12) {
    // --------------------------------- masked scores and output, one row per lane
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const float ldf = static_cast<float>(ld);
    // Score (row p, column j) is weighted by d^(p - j) and A Z's row by d^(p + e).
    // Slow decays: P_pj = S_pj d^(-j - e) adds to A Z as it is, and the row factor d^(p + e)
    // multiplies the sum. Fast ones, where d^-128 could overflow: d^(p - j) as a row factor
    // times a column power off the diagonal 32-column block, from a table on it, and A Z is
    // scaled in place. Either way a block's weights are 32 column powers, kept in registers,
    // times one factor per block (uniform, or the row's):
    //                          column power           block factor
    //   slow   forward         d^-jj                  d^(-32m - 1)
    //          backward        d^(jj - 31)            d^(-(L - 32 - 32m))
    //   fast   forward         d^(31 - jj)            d^(row - 32m - 31)
    //          backward        d^jj                   d^(32m - row)
    uint64_t off[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int up = back ? 2 * j - 31 : -2 * j;   // of the slow form, at column 2j
      const int x0 = slow ? up : up + 31, x1 = back ? x0 + 1 : x0 - 1;
      off[j] = f2_pack(x0 == 0 ? 1.f : expf(ldf * static_cast<float>(x0)),
                       x1 == 0 ? 1.f : expf(ldf * static_cast<float>(x1)));
    }
    const int step = back ? 1 : -1;
    const float* diag = &sm.diag[32 - lane * step];   // column jj at step * jj
    const uint32_t ydst = smem_addr(&sm.y[0][quad][0]) + lane * 128;
    const int first = back ? quad : 0, last = back ? 3 : quad;   // blocks that are not masked whole
    bool ok = true;
    const uint32_t keep = back ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);   // columns of the diagonal block
    ChunkWalk c(p, ci0);
    const float up32 = slow ? expf(ldf * (back ? 32.f : -32.f)) : 1.f;
#pragma unroll 1
    for (int i = 0; i < n; ++i, c.next(p)) {
      // d^(p + e) of this row, and the slow form's factor of the first block.
      const int x = back ? c.len - 1 - row : row + 1;
      const float w = x > 0 ? expf(ldf * static_cast<float>(x)) * p.s_st : p.s_st;
      float fs = expf(ldf * static_cast<float>(back ? 32 - c.len : -1)) * (p.s_in / p.s_st);
      if (!(ok = wait(sm.s_full, i))) break;
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m, fs *= up32) {   // P over the scores: block m's columns were read by block m / 2
        uint32_t s[32], pk[16];
        if (m < first || m > last) {
          const uint32_t zero[16] = {0u};
          tmem_st16(tS + lane_off + 16 * m, zero);
          continue;
        }
        tmem_ld32(tS + lane_off + 32 * m, s);
        if (back && c.len < kChunk) {   // columns past the chunk's tokens hold other rows
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) s[jj] = 32 * m + jj < c.len ? s[jj] : 0u;
        }
        if (slow || m != quad) {
          const float fm = slow ? fs : expf(ldf * static_cast<float>(back ? 32 * m - row : row - 32 * m - 31)) * p.s_in;
          const uint64_t ff = f2_pack(fm, fm);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float x0, x1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), f2_mul(off[j], ff)), x0,
                      x1);
            pk[j] = pack_bf16x2(x0, x1);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[j] = pack_bf16x2(__uint_as_float(s[2 * j]) * diag[2 * j * step],
                                __uint_as_float(s[2 * j + 1]) * diag[(2 * j + 1) * step]);
        }
        if (m == quad) {   // the masked side of the diagonal block, 0 whatever the scores
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            pk[j] &= (keep & (1u << (2 * j)) ? 0xffffu : 0u) | (keep & (2u << (2 * j)) ? 0xffff0000u : 0u);
          }
        }
        tmem_st16(tS + lane_off + 16 * m, pk);
      }
      if (!slow) {
        if (!(ok = wait(sm.az_done, i))) break;
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          uint32_t az[32];
          tmem_ld32(tY + lane_off + q, az);
#pragma unroll
          for (int k = 0; k < 32; ++k) az[k] = __float_as_uint(__uint_as_float(az[k]) * w);
          tmem_st16(tY + lane_off + q, az);
          tmem_st16(tY + lane_off + q + 16, az + 16);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(sm.p_ready);
      // Rows leave through shared memory and TMA stores of 32 rows x 64 columns (a thread's
      // own stores would touch 32 lines at a time and hold up the other warps' shared-memory
      // accesses); a warp whose rows end inside the chunk stores them itself, the rows after
      // may be another piece's.
      const bool staged = quad * 32 + 32 <= c.len;
      const int rb = c.rank(p) * p.B + b, t0 = c.token(p);
      __nv_bfloat16* dst = p.y + ((static_cast<int64_t>(rb) * p.T + t0 + row) * p.H + h) * D;
      if (lane == 0) bulk_wait_read<0>();   // the chunk before has left the buffers
      if (!(ok = wait(sm.y_full, i))) break;
      tc_fence_after();
      const uint64_t wy = slow ? f2_pack(w, w) : f2_pack(1.f, 1.f);
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t y[32];
        tmem_ld32(tY + lane_off + 32 * q, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x0, x1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(y[8 * k + 2 * e]), __uint_as_float(y[8 * k + 2 * e + 1])), wy), x0,
                      x1);
            v[e] = pack_bf16x2(x0, x1);
          }
          const int vec = 4 * (q & 1) + k;
          if (staged) st_shared_v4(ydst + (q >> 1) * (4 * 32 * 128) + ((vec ^ (lane & 7)) * 16), v);
          else if (row < c.len) reinterpret_cast<uint4*>(dst)[4 * q + k] = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      tc_fence_before();
      fence_async_smem();
      warp_arrive(sm.y_free);
      if (staged && lane == 0)
        for (int blk = 0; blk < C::kBlocks; ++blk)
          tma_store_4d(&tm_y, smem_addr(&sm.y[blk][quad][0]), blk * 64, h, t0 + quad * 32, rb);
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kKvWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
  if (!OUT && p.zseg_t != nullptr && warp < 8 && (warp & 3) * 32 < D) {
    const int row = (warp & 3) * 32 + lane, grp = warp >> 2;
    float4* dst = reinterpret_cast<float4*>(p.zseg_t + (static_cast<int64_t>(bh) * (p.nseg - 1) + seg) * (D * D)) +
                  grp * D + row;
    const float* src = zt_smem + row * (D + 1) + grp * (D / 2);
#pragma unroll
    for (int q = 0; q < D / 8; ++q)
      dst[q * (2 * D)] = make_float4(src[4 * q], src[4 * q + 1], src[4 * q + 2], src[4 * q + 3]);
  }
}

// ------------------------------------------------------------------ recurrent form
// A few tokens on a kept state, updated in place: per (batch, head) the D x D fp32
// state is read and written once (8 D^2 bytes, the bound) while the tokens' q, k, v are
// walked from shared memory. A CTA owns CW columns of one head's state: a thread holds
// rows rg, rg + RG, ... of four columns in registers; each token's output is summed
// over a warp's row groups by shuffles and over the warps through shared memory,
// four tokens at a time.
constexpr int kStepGroup = 4;   // tokens whose sums are joined at a time
template <int D, int CW>
struct alignas(16) StepSmem {
  float2 qk[kLinStepMaxT][D];
  float v[kLinStepMaxT][CW];       // v and red are also read and written as float4
  float red[kStepGroup][8][CW];
};

template <int D, int CW>
__global__ void __launch_bounds__(256) linattn_step_kernel(const LinStepParams p) {
  constexpr int CG = CW / 4;        // column groups of 4
  constexpr int RG = 256 / CG;      // row groups
  constexpr int RPT = D / RG;       // rows per thread
  static_assert(RPT >= 1 && CG <= 32, "tile");
  using Smem = StepSmem<D, CW>;
  static_assert(offsetof(Smem, v) % 16 == 0 && offsetof(Smem, red) % 16 == 0 && CW % 4 == 0, "float4 accesses");
  __shared__ Smem sm;
  constexpr int kSl = D / CW;
  const int sl = static_cast<int>(blockIdx.x) % kSl;
  const int64_t bh = blockIdx.x / kSl;
  const int h = static_cast<int>(bh % p.H);
  const int64_t b = bh / p.H;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* st = p.state + bh * D * D + sl * CW + cg * 4;
  float4 s[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) s[r] = *reinterpret_cast<const float4*>(st + static_cast<int64_t>(rg + r * RG) * D);
  for (int i = threadIdx.x; i < p.T * D; i += 256) {
    const int t = i / D, d = i % D;
    const int64_t at = ((b * p.T + t) * p.H + h) * D + d;
    sm.qk[t][d] = make_float2(__bfloat162float(p.q[at]) * p.scale, __bfloat162float(p.k[at]));
    if (d < CW) sm.v[t][d] = __bfloat162float(p.v[at + sl * CW]);
  }
  // d as an fp32 pair, as in the chunked form: one fp32 exponential is off by up to 2^-23 of it, the
  // same way at every call, and a state kept over thousands of tokens would show that.
  const double d = decay_pow(static_cast<double>(__ldg(p.log_decay + h)), 1);
  const float hi = static_cast<float>(d), lo = static_cast<float>(d - static_cast<double>(hi));
  const uint64_t hi2 = f2_pack(hi, hi), lo2 = f2_pack(lo, lo);
  __syncthreads();
  for (int t0 = 0; t0 < p.T; t0 += kStepGroup) {
    const int t1 = min(t0 + kStepGroup, p.T);
    for (int t = t0; t < t1; ++t) {
      const float4 v = *reinterpret_cast<const float4*>(&sm.v[t][cg * 4]);
      const uint64_t v0 = f2_pack(v.x, v.y), v1 = f2_pack(v.z, v.w);
      uint64_t o0 = f2_pack(0.f, 0.f), o1 = o0;
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float2 qk = sm.qk[t][rg + r * RG];
        const uint64_t qq = f2_pack(qk.x, qk.x), kk = f2_pack(qk.y, qk.y);
        const uint64_t z0 = f2_pack(s[r].x, s[r].y), z1 = f2_pack(s[r].z, s[r].w);
        const uint64_t s0 = f2_fma(z0, hi2, f2_fma(z0, lo2, f2_mul(kk, v0)));
        const uint64_t s1 = f2_fma(z1, hi2, f2_fma(z1, lo2, f2_mul(kk, v1)));
        o0 = f2_fma(qq, s0, o0);
        o1 = f2_fma(qq, s1, o1);
        f2_unpack(s0, s[r].x, s[r].y);
        f2_unpack(s1, s[r].z, s[r].w);
      }
      float4 o;
      f2_unpack(o0, o.x, o.y);
      f2_unpack(o1, o.z, o.w);
#pragma unroll
      for (int m = CG; m < 32; m <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
      }
      if (lane < CG) *reinterpret_cast<float4*>(&sm.red[t - t0][warp][lane * 4]) = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (t1 - t0) * CW; i += 256) {
      const int t = t0 + i / CW, c = i % CW;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) y += sm.red[t - t0][w][c];
      p.o[((b * p.T + t) * p.H + h) * D + sl * CW + c] = __float2bfloat16_rn(y);
    }
    if (t1 < p.T) __syncthreads();   // the sums have been read before the next group's are written
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) *reinterpret_cast<float4*>(st + static_cast<int64_t>(rg + r * RG) * D) = s[r];
}

template <int D, bool OUT, int TERMS>
bool launch_lin(const LinLaunch& L, int segments, bool early, cudaStream_t stream) {
  const size_t smem = sizeof(LinSmem<D, OUT, TERMS>) + 1024;
  auto kern = linattn_kernel<D, OUT, TERMS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.scans * L.scan[0].p.units * segments);
  cfg.blockDim = dim3(LinCfg<D, OUT, TERMS>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, L) == cudaSuccess;
}

// The launches of a forward or a backward: the segments' own states (all but the last),
// then the rows. The backward's last scan takes its states from the one before, transposed.
template <int D, int TERMS>
bool launch_scans(LinLaunch& L, cudaStream_t stream) {
  const int nseg = L.scan[0].p.nseg, scans = L.scans;
  if (nseg > 1) {
    L.scans = scans == 3 ? 2 : scans;
    if (!launch_lin<D, false, TERMS>(L, nseg - 1, false, stream)) return false;
    L.scans = scans;
  }
  return launch_lin<D, true, TERMS>(L, nseg, nseg > 1, stream);
}
bool launch_scans(LinLaunch& L, int D, cudaStream_t stream) {
  bool exact = false;   // a last state is asked for
  for (int i = 0; i < L.scans; ++i) exact = exact || L.scan[i].p.z_out != nullptr;
  if (D == 128) return exact ? launch_scans<128, 3>(L, stream) : launch_scans<128, 2>(L, stream);
  return exact ? launch_scans<64, 3>(L, stream) : launch_scans<64, 2>(L, stream);
}

// ------------------------------------------------------------------------ host side

// The memory view a plan's tensors are walked in: pieces of consecutive tokens in
// natural order. A contiguous batch of one, and a single rank, are one piece.
struct LinView {
  int N, zigzag, T, piece_len, pieces, chunks_per_piece, nch;
};
LinView lin_view(const PlanView& v) {
  LinView w;
  const bool plain = v.N == 1 || (v.layout == CP_LAYOUT_CONTIGUOUS && v.B == 1);
  w.N = plain ? 1 : v.N;
  w.zigzag = !plain && v.layout == CP_LAYOUT_ZIGZAG;
  w.T = v.S / w.N;
  w.pieces = w.zigzag ? 2 * w.N : w.N;
  w.piece_len = v.S / w.pieces;
  w.chunks_per_piece = (w.piece_len + kChunk - 1) / kChunk;
  w.nch = w.pieces * w.chunks_per_piece;
  return w;
}

// Segments a sequence is cut into, for `ctas` scans x (batch, head) of nch chunks. Modelled
// time in chunks of the output launch (3.1 us each): a wave costs its chunks, about 2.5 more
// to fill and drain, and 0.35 for each earlier segment's state to join; a chunk of the state
// launch 0.45. Measured on 148 SMs, us, the model's choice first: 32 heads of 256 chunks 4
// segments 309, 3 392, 5 418, 9 321, 1 759; 8 heads of 64 chunks 16 48.9, 12 52.1, 8 54.1, 18 51.7,
// 1 195; their backward 6 71, 4 88, 8 96, 1 198; the backward of 4 heads of 256 chunks 12 130, 9 153,
// 16 180, 1 763.
constexpr int kMaxSegments = 64;
int choose_segments(int64_t ctas, int64_t state_ctas, int nch, int sms) {
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= nch && s <= kMaxSegments; ++s) {
    const double per = (nch + s - 1) / s;
    const double waves = static_cast<double>((ctas * s + sms - 1) / sms);
    double cost = waves * (per + 2.5 + 0.35 * (s - 1));
    if (s > 1) cost += static_cast<double>((state_ctas * (s - 1) + sms - 1) / sms) * (0.45 * per + 2.0);
    if (s == 1 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

size_t tensor_bytes(const PlanView& v) { return sizeof(__nv_bfloat16) * v.B * v.S * v.H * v.D; }
size_t state_bytes(const PlanView& v, int nseg) {   // the segments' own states of one scan
  return static_cast<size_t>(v.B) * v.H * (nseg - 1) * v.D * v.D * sizeof(float);
}
int fwd_segments(const PlanView& v) {
  const int64_t units = static_cast<int64_t>(v.B) * v.H;
  return choose_segments(units, units, lin_view(v).nch, v.sms);
}
int bwd_segments(const PlanView& v) {
  const int64_t units = static_cast<int64_t>(v.B) * v.H;
  return choose_segments(3 * units, 2 * units, lin_view(v).nch, v.sms);
}

struct ScanCall {
  const void *a, *b, *c;
  void* y;
  const float* z0;
  bool z0_transposed, reverse;
  float s_in, s_st, s_upd;
  float* z_out;
};

bool make_scan(LinScan* L, const PlanView& v, const ScanCall& s, const float* log_decay, float* ws, int nseg) {
  const LinView w = lin_view(v);
  const int64_t rb = static_cast<int64_t>(w.N) * v.B;
  if (!encode_map_4d(&L->tm_a, s.a, v.D, v.H, w.T, rb, 1, kChunk) ||
      !encode_map_4d(&L->tm_b, s.b, v.D, v.H, w.T, rb, 1, kChunk) ||
      !encode_map_4d(&L->tm_c, s.c, v.D, v.H, w.T, rb, 1, kChunk) ||
      !encode_map_4d(&L->tm_y, s.y, v.D, v.H, w.T, rb, 1, 32))
    return false;
  LinParams& p = L->p;
  p.B = v.B;
  p.H = v.H;
  p.S = v.S;
  p.N = w.N;
  p.T = w.T;
  p.zigzag = w.zigzag;
  p.piece_len = w.piece_len;
  p.chunks_per_piece = w.chunks_per_piece;
  p.nch = w.nch;
  p.units = v.B * v.H;
  p.nseg = nseg;
  p.z0_transposed = s.z0_transposed;
  p.reverse = s.reverse;
  p.s_in = s.s_in;
  p.s_st = s.s_st;
  p.s_upd = s.s_upd;
  p.log_decay = log_decay;
  p.z0 = s.z0;
  p.z_out = s.z_out;
  p.zseg = ws;
  p.zseg_t = nullptr;
  p.y = static_cast<__nv_bfloat16*>(s.y);
  p.status = v.status;
  p.wait_limit_ns = kWaitLimitNs;
  return true;
}

bool supported(const PlanView& v) {
  if (v.layout == CP_LAYOUT_ULYSSES || !v.causal) return false;
  // one CTA per scan, (batch, head) and segment, indexed in int32
  return static_cast<int64_t>(v.B) * v.H <= (int64_t(1) << 29) / kMaxSegments;
}

// The plan of a forward or a backward.
int check_plan(cp_attn_plan_t plan, PlanView* v) {
  const int rc = plan_view(plan, v);
  return supported(*v) ? rc : CP_ERR_UNSUPPORTED;
}

}  // namespace

}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cp_linattn_workspace_bytes(cp_attn_plan_t plan) {
  if (plan == nullptr) return 0;
  PlanView v;
  plan_view(plan, &v);   // the sizes, whichever device is current
  if (!supported(v)) return 0;
  const size_t f = state_bytes(v, fwd_segments(v)), b = 3 * state_bytes(v, bwd_segments(v));
  return f > b ? f : b;
}

int cp_linattn_fwd(cp_attn_plan_t plan, const void* q, const void* k, const void* v, const float* log_decay,
                   const float* state_in, void* o, float* state_out, void* workspace, cp_stream_t stream) {
  if (plan == nullptr || q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || o == nullptr)
    return CP_ERR_INVALID_ARG;
  if (!is_aligned16(q) || !is_aligned16(k) || !is_aligned16(v) || !is_aligned16(o) || !is_aligned16(state_in) ||
      !is_aligned16(state_out) || !is_aligned16(workspace) || (reinterpret_cast<uintptr_t>(log_decay) & 3u) != 0)
    return CP_ERR_ALIGNMENT;
  if (state_in != nullptr && state_in == state_out) return CP_ERR_INVALID_ARG;   // read by every segment's CTAs
  PlanView pv;
  int rc = check_plan(plan, &pv);
  if (rc != CP_OK) return rc;
  const int nseg = fwd_segments(pv);
  const size_t ws_bytes = state_bytes(pv, nseg);
  if (workspace == nullptr && ws_bytes > 0) return CP_ERR_WORKSPACE;
  // Other CTAs would read rows already written, or write the same ones.
  const size_t t = tensor_bytes(pv), z = state_bytes(pv, 2), ld = pv.H * sizeof(float);
  if (overlaps({{o, t}, {state_out, z}, {workspace, ws_bytes}},
               {{q, t}, {k, t}, {v, t}, {log_decay, ld}, {state_in, z}}))
    return CP_ERR_INVALID_ARG;
  LinLaunch L;
  L.scans = 1;
  if (!make_scan(&L.scan[0], pv, {q, k, v, o, state_in, false, false, pv.scale, pv.scale, 1.f, state_out}, log_decay,
                 static_cast<float*>(workspace), nseg))
    return CP_ERR_CUDA;
  return launch_scans(L, pv.D, static_cast<cudaStream_t>(stream)) ? CP_OK : CP_ERR_CUDA;
}

int cp_linattn_bwd(cp_attn_plan_t plan, const void* q, const void* k, const void* v, const float* log_decay,
                   const void* dout, const float* state_in, const float* dstate_out, void* dq, void* dk, void* dv,
                   float* dstate_in, void* workspace, cp_stream_t stream) {
  if (plan == nullptr || q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || dout == nullptr ||
      dq == nullptr || dk == nullptr || dv == nullptr)
    return CP_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, dout, state_in, dstate_out, dq, dk, dv, dstate_in, workspace};
  for (const void* x : ptrs)
    if (!is_aligned16(x)) return CP_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(log_decay) & 3u) != 0) return CP_ERR_ALIGNMENT;
  if (dstate_out != nullptr && dstate_out == dstate_in) return CP_ERR_INVALID_ARG;
  PlanView pv;
  int rc = check_plan(plan, &pv);
  if (rc != CP_OK) return rc;
  const int nseg = bwd_segments(pv);
  const size_t part_bytes = state_bytes(pv, nseg), part = part_bytes / sizeof(float);
  if (workspace == nullptr && part > 0) return CP_ERR_WORKSPACE;
  const size_t t = tensor_bytes(pv), z = state_bytes(pv, 2), ld = pv.H * sizeof(float);
  if (overlaps({{dq, t}, {dk, t}, {dv, t}, {dstate_in, z}, {workspace, 3 * part_bytes}},
               {{q, t}, {k, t}, {v, t}, {log_decay, ld}, {dout, t}, {state_in, z}, {dstate_out, z}}))
    return CP_ERR_INVALID_ARG;
  const float sc = pv.scale;
  const ScanCall calls[3] = {{dout, v, k, dq, state_in, true, false, sc, sc, 1.f, nullptr},
                             {v, dout, q, dk, dstate_out, true, true, sc, 1.f, sc, nullptr},
                             {k, q, dout, dv, dstate_out, false, true, sc, 1.f, sc, dstate_in}};
  LinLaunch L;
  L.scans = 3;
  for (int i = 0; i < 3; ++i) {
    float* ws = part > 0 ? static_cast<float*>(workspace) + i * part : nullptr;
    if (!make_scan(&L.scan[i], pv, calls[i], log_decay, ws, nseg)) return CP_ERR_CUDA;
  }
  // dk's state sums do_i q_i^T and dv's its transpose, in the same direction with the same weights.
  if (part > 0) L.scan[1].p.zseg_t = L.scan[2].p.zseg;
  return launch_scans(L, pv.D, static_cast<cudaStream_t>(stream)) ? CP_OK : CP_ERR_CUDA;
}

int cp_linattn_step(int B, int T, int H, int D, const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, float* state, void* o, cp_stream_t stream) {
  if (B < 0 || T < 0 || H < 1) return CP_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return CP_ERR_UNSUPPORTED;
  if (T > kLinStepMaxT || static_cast<int64_t>(B) * H * (D / 32) > INT32_MAX) return CP_ERR_UNSUPPORTED;
  if (!(scale > -INFINITY && scale < INFINITY)) return CP_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return CP_OK;
  if (q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || state == nullptr || o == nullptr)
    return CP_ERR_INVALID_ARG;
  if (!is_aligned16(q) || !is_aligned16(k) || !is_aligned16(v) || !is_aligned16(state) || !is_aligned16(o) ||
      (reinterpret_cast<uintptr_t>(log_decay) & 3u) != 0)
    return CP_ERR_ALIGNMENT;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return CP_ERR_CUDA;
  const size_t t = sizeof(__nv_bfloat16) * B * T * H * D;
  if (overlaps({{o, t}, {state, sizeof(float) * B * H * D * D}}, {{q, t}, {k, t}, {v, t}, {log_decay, H * sizeof(float)}}))
    return CP_ERR_INVALID_ARG;
  LinStepParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.log_decay = log_decay;
  p.state = state;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.scale = scale;
  p.T = T;
  p.H = H;
  const int64_t heads = static_cast<int64_t>(B) * H;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // A whole head per CTA where there is one for each SM; else 32 columns each, for more CTAs.
  // Measured whole and cut on 148 SMs, D = 128: 32 heads 3.4 and 2.3 us (16 tokens: 10.2 and 6.6),
  // 148 heads 3.7 and 3.5 (10.6 and 12.9), 2048 heads 43.4 and 41.5 (114 and 147).
  const bool wide = heads >= sms;
  const int grid = static_cast<int>(heads * (wide ? 1 : D / 32));
  if (D == 128) {
    if (wide) linattn_step_kernel<128, 128><<<grid, 256, 0, st>>>(p);
    else linattn_step_kernel<128, 32><<<grid, 256, 0, st>>>(p);
  } else {
    if (wide) linattn_step_kernel<64, 64><<<grid, 256, 0, st>>>(p);
    else linattn_step_kernel<64, 32><<<grid, 256, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // extern "C"
