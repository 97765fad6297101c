// cache_attn.h — launch parameters of attention over a key/value cache (internal).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cpattn {

constexpr int kCacheMaxB = 1024;   // sequences: their tile prefix sums sit in shared memory
constexpr int kCacheMaxT = 64;     // drafted tokens: one bit each in a 64-bit word

struct CacheParams {
  int B, Hq, Hkv, T, G, cap;
  int own;              // cache rows lengths[b] .. lengths[b] + T - 1 hold the drafted tokens
  int tok_per_tile;     // drafted tokens per 128-row query tile
  int row_tiles;        // query tiles per (sequence, key/value head)
  int n_cta;
  float scale_log2;
  const int* lengths;            // [B]
  const unsigned long long* tree;   // [B][T] or null (a chain)
  float* parts;                  // [2 * n_cta] slots of 128 x D sums, then 128 (max, sum) pairs
  __nv_bfloat16* o;              // [B][T][Hq][D], or null
  float* o_part;                 // fp32 [B*T*Hq][D], or null
  float* lse;                    // [B][Hq][T] with o, [B*T*Hq] with o_part
  int* status;
  uint64_t wait_limit_ns;
};

struct CacheLaunch {
  CUtensorMap tm_q, tm_k, tm_v;   // 4-D views (D, Hq, T, B) and (D, Hkv, cap, B)
  CacheParams p;
};

}  // namespace cpattn
