// Device pieces shared by the layer kernels: eight adjacent elements of a row as a unit of
// loads, stores and dropout, the counter-based generator, sums over the threads of a row.
#pragma once

#include "ffn_act.cuh"
#include "igc_layers.h"
#include "sm100_ptx.cuh"

namespace igc {

// Eight adjacent elements of type kT as they lie in memory.
template <int kT>
struct Raw8 {
  uint4 q[kT == IGC_F32 ? 2 : 1];
};

template <int kT>
__device__ __forceinline__ const char* row_at(const void* p, long long row, long long ld) {
  return static_cast<const char*>(p) + row * ld * (kT == IGC_F32 ? 4 : 2);
}
template <int kT>
__device__ __forceinline__ char* row_at(void* p, long long row, long long ld) {
  return static_cast<char*>(p) + row * ld * (kT == IGC_F32 ? 4 : 2);
}

// Elements [n, n + 8) of a row of N (0 past its end): by 16-byte loads where the row starts on
// a 16-byte boundary (vec) and has them all, else one by one.
template <int kT>
__device__ __forceinline__ Raw8<kT> load8(const char* row, int n, int N, bool vec) {
  Raw8<kT> r;
  if (vec && n + 8 <= N) {
    const uint4* p = reinterpret_cast<const uint4*>(row + static_cast<long long>(n) *
                                                              (kT == IGC_F32 ? 4 : 2));
    r.q[0] = p[0];
    if constexpr (kT == IGC_F32) r.q[1] = p[1];
    return r;
  }
  if constexpr (kT == IGC_F32) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = n + i < N ? p[n + i] : 0u;
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = n + 2 * i < N ? p[n + 2 * i] : 0u;
      const uint32_t hi = n + 2 * i + 1 < N ? p[n + 2 * i + 1] : 0u;
      w[i] = lo | (hi << 16);
    }
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

template <int kT>
__device__ __forceinline__ void unpack8(const Raw8<kT>& r, float (&v)[8]) {
  if constexpr (kT == IGC_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(r.q[i].x), v[4 * i + 1] = __uint_as_float(r.q[i].y);
      v[4 * i + 2] = __uint_as_float(r.q[i].z), v[4 * i + 3] = __uint_as_float(r.q[i].w);
    }
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(w[i], kT == IGC_BF16);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

// Rounds eight values and stores those before the row's end.
template <int kT>
__device__ __forceinline__ void store8(char* row, int n, int N, bool vec, const float (&v)[8]) {
  if constexpr (kT == IGC_F32) {
    float* p = reinterpret_cast<float*>(row) + n;
    if (vec && n + 8 <= N) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) p[i] = v[i];
  } else {
    constexpr bool bf16 = kT == IGC_BF16;
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + n;
    const uint32_t w[4] = {pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16),
                           pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16)};
    if (vec && n + 8 <= N) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) p[i] = static_cast<uint16_t>(i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
  }
}

// Elements [n, n + 8) of a vector of N that is fp32 (f32) or of type kT; `none` for no vector
// and past its end.  (Vectors may start anywhere: 16-byte loads where they can.)
template <int kT>
__device__ __forceinline__ void load_vec8(const void* p, int n, int N, bool f32, float none,
                                          float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
    return;
  }
  const bool vec = (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
  if (kT == IGC_F32 || f32)
    unpack8<IGC_F32>(load8<IGC_F32>(static_cast<const char*>(p), n, N, vec), v);
  else
    unpack8<kT>(load8<kT>(static_cast<const char*>(p), n, N, vec), v);
}

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011): ten rounds, each two 32 x 32 -> 64 bit
// products, two three-way exclusive ors and a step of the key.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return c;
}

struct Drop {
  uint32_t k0 = 0, k1 = 0;     // the seed
  uint64_t offset = 0;
  const uint64_t* step = nullptr;
  uint32_t threshold = 0;      // T << 16 (T < 65536; no dropout is another variant of a kernel)
  float scale = 1.0f;          // 65536 / T (0 for T = 0)
};

// v: eight elements of row `row` from column n (a multiple of 8) on, dropped and scaled.  One
// block of Philox for all eight, 16 bits each: 5 instructions an element beside the 10 that 32
// bits each would take, and p to 2^-17 is finer than a rate is ever set.  What is dropped is
// selected away, not multiplied by 0: an infinity there leaves nothing.
__device__ __forceinline__ void drop8(const Drop& d, uint64_t offset, long long row, int n,
                                      float (&v)[8]) {
  const uint4 q = philox4x32_10(
      make_uint4(static_cast<uint32_t>(n) / 8u, static_cast<uint32_t>(row),
                 static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)),
      d.k0, d.k1);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a half is under T just where the word that has it as its upper half is under T << 16
    v[2 * i] = (w[i] << 16) < d.threshold ? v[2 * i] * d.scale : 0.0f;
    v[2 * i + 1] = w[i] < d.threshold ? v[2 * i + 1] * d.scale : 0.0f;
  }
}

__device__ __forceinline__ uint64_t drop_offset(const Drop& d) {
  return d.offset + (d.step != nullptr ? *d.step : 0u);
}

// ---------------------------------------------------------------------------
// sums over the kThreads threads of a row, in every one of them, in a fixed order
// ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_sum_all(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// kThreads = 32: a warp; else the whole block of kThreads threads, through red (one array of
// kThreads / 32 values for each sum that may be in flight between two barriers).
template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum_all(v);
  if constexpr (kThreads > 32) {
    constexpr int kWarps = kThreads / 32;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s[4] = {};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s[i % 4] += red[i];
    v = (s[0] + s[1]) + (s[2] + s[3]);
  }
  return v;
}

}  // namespace igc
