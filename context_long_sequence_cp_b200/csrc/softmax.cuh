// softmax.cuh — the pieces of one score row's online softmax that the attention
// kernels share: a row of kTile scores per thread, P written back to TMEM as bf16.
#pragma once

#include <cstdint>

#include "geometry.h"
#include "sm100.cuh"

namespace cpattn {

using namespace sm100;

// Exponentials of one 32-column chunk c of a score row, packed to bf16 pairs and
// stored as 16 TMEM columns of P at tS + 64 + 16c (over the scores of keys
// 64-127, which are in registers by then); row-sum partials accumulate in ls.
// The scaling x = s * scale - m runs two columns per instruction (f32x2).
__device__ __forceinline__ void softmax_chunk(const float (&s)[kTile], int c, float sl2, float m_use,
                                              uint32_t tS, float (&ls)[8]) {
  uint32_t pk[16];
  const uint64_t sl2_2 = f2_pack(sl2, sl2);
  const uint64_t nm_2 = f2_pack(-m_use, -m_use);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int col = c * 32 + 2 * j;
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(s[col], s[col + 1]), sl2_2, nm_2), x0, x1);
    const float e0 = ex2_approx(x0);
    const float e1 = ex2_approx(x1);
    ls[j & 7] += e0 + e1;
    pk[j] = pack_bf16x2(e0, e1);
  }
  tmem_st16(tS + 64 + c * 16, pk);
}

// Maximum of the 64 scores s[32c .. 32c+63], four chains of 3-input maxima.
__device__ __forceinline__ float half_max(const float (&s)[kTile], int c) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = 32 * c + 16 * k;
    float x = max3(s[b], s[b + 1], s[b + 2]);
#pragma unroll
    for (int j = 3; j + 1 < 16; j += 2) x = max3(x, s[b + j], s[b + j + 1]);
    m[k] = fmaxf(x, s[b + 15]);
  }
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

}  // namespace cpattn
