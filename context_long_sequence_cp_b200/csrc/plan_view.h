// plan_view.h — what entry points outside api.cu need of a plan, and the helpers
// they share with it (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "geometry.h"

struct cp_attn_plan_s;

namespace cpattn {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s per in-kernel wait

struct PlanView {
  int B, H, S, D, N, causal, layout;
  float scale;
  int sms;
  int* status;   // device status word
};

// Fills *out. Returns CP_ERR_CUDA when the plan was made without a device,
// CP_ERR_INVALID_ARG when another device than the plan's is current, else CP_OK.
int plan_view(const cp_attn_plan_s* plan, PlanView* out);

// Bytes are 16-byte aligned.
inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A buffer of a call; a null one is empty.
struct Buffer {
  const void* p;
  size_t bytes;
};
// One of the outputs shares bytes with an input or with another output.
inline bool overlaps(std::initializer_list<Buffer> outs, std::initializer_list<Buffer> ins) {
  auto meet = [](const Buffer& a, const Buffer& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Buffer* o = outs.begin(); o != outs.end(); ++o) {
    for (const Buffer& i : ins)
      if (meet(*o, i)) return true;
    for (const Buffer* other = outs.begin(); other != o; ++other)
      if (meet(*o, *other)) return true;
  }
  return false;
}

// 4-D bf16 tensor map (d0, d1, d2, d3) over a dense tensor stored [d3][d2][d1][d0],
// 128-byte swizzle, box (64, box1, box2, 1); false when the driver refuses it.
bool encode_map_4d(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t d3, int box1,
                   int box2);

}  // namespace cpattn
