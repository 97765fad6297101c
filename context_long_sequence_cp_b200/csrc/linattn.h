// linattn.h — launch parameters of linear attention (internal).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cpattn {

// One scan over a plan's tokens (see linattn.cu for the roles of a, b, c and Z).
struct LinParams {
  int B, H, S, N, T;        // batches, heads, tokens, ranks of the view, tokens per rank
  int zigzag;
  int piece_len;            // consecutive tokens in memory and in the sequence
  int chunks_per_piece, nch;
  int units;                // B * H
  int nseg;                 // segments a sequence is cut into
  int reverse;              // walk from the last token to the first
  int z0_transposed;
  float s_in, s_st, s_upd;  // factors of the scores, of A Z, and of the rows entering Z
  const float* log_decay;   // [H]
  const float* z0;          // [B][H][D][D] or null
  float* z_out;             // [B][H][D][D] or null
  float* zseg;              // [units][nseg - 1][D][D]: each segment's own state
  float* zseg_t;            // the same, transposed, for another scan (null: not wanted)
  __nv_bfloat16* y;
  int* status;
  uint64_t wait_limit_ns;
};

struct LinScan {
  CUtensorMap tm_a, tm_b, tm_c, tm_y;   // 4-D views (D, H, T, N*B)
  LinParams p;
};

struct LinLaunch {
  LinScan scan[3];   // the forward's one, or the backward's three
  int scans;
};

constexpr int kLinStepMaxT = 16;   // tokens of one recurrent call

struct LinStepParams {
  const __nv_bfloat16 *q, *k, *v;   // [B][T][H][D]
  const float* log_decay;           // [H]
  float* state;                     // [B][H][D][D], updated in place
  __nv_bfloat16* o;                 // [B][T][H][D]
  float scale;
  int T, H;
};

}  // namespace cpattn
