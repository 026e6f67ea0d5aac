// Host-side pieces shared by the layer entry points (not part of the ABI).
#pragma once

#include <cmath>

#include "ffn_host.h"
#include "layers.cuh"

namespace igc {

inline bool is_type(int dtype) { return dtype == IGC_F32 || is_operand_type(dtype); }
// a, or fp32 beside it
inline bool is_type_or_f32(int dtype, int a) { return dtype == a || dtype == IGC_F32; }

// Dropout of an entry's (p, seed, offset, step): false for a p outside [0, 1] or NaN.
// *active: whether anything can be dropped (T < 65536).
inline bool make_drop(double p, uint64_t seed, uint64_t offset, const uint64_t* step, Drop* d,
                      bool* active) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  const uint32_t T = static_cast<uint32_t>(std::nearbyint((1.0 - p) * 65536.0));
  *active = T < 65536u;
  for (uint32_t r = 0; r < kPhiloxRounds; ++r) {
    d->key[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
    d->key[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
  }
  d->offset = offset;
  d->step = step;
  d->threshold = T << 16;
  d->scale = T == 0 ? 0.0f : static_cast<float>(65536.0 / T);
  return true;
}

// Whether the rows of a matrix of M rows start on 16-byte boundaries (a null one's do).  A single
// row's stride says nothing.
inline bool rows_vec(int64_t M, const void* p, int64_t ld, int dtype) {
  return p == nullptr || rows_aligned(p, M > 1 ? ld : 0, elem_size(dtype), 16);
}

// Division of 32-bit numbers by a fixed d >= 1 as a product and shifts (Granlund and
// Montgomery, "Division by invariant integers using multiplication", PLDI 1994, figure 4.1).
struct FastDiv {
  uint32_t d = 1, mul = 0, sh1 = 0, sh2 = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - div)) / div + 1);
    sh1 = l < 1 ? l : 1;
    sh2 = l < 1 ? 0 : l - 1;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(mul, n);
    return (t + ((n - t) >> sh1)) >> sh2;
  }
};

}  // namespace igc
