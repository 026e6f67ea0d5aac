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

// Rounds eight values and stores them at p, a 16-byte boundary.
template <int kT>
__device__ __forceinline__ void store_unit(char* p, const float (&v)[8]) {
  if constexpr (kT == IGC_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    constexpr bool bf16 = kT == IGC_BF16;
    *reinterpret_cast<uint4*>(p) = make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16),
                                              pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16));
  }
}
// Eight elements at p, a 16-byte boundary.
template <int kT>
__device__ __forceinline__ void load_unit(const char* p, float (&v)[8]) {
  Raw8<kT> r;
  r.q[0] = reinterpret_cast<const uint4*>(p)[0];
  if constexpr (kT == IGC_F32) r.q[1] = reinterpret_cast<const uint4*>(p)[1];
  unpack8<kT>(r, v);
}

// Rounds eight values and stores those before the row's end.
template <int kT>
__device__ __forceinline__ void store8(char* row, int n, int N, bool vec, const float (&v)[8]) {
  if (vec && n + 8 <= N) {
    store_unit<kT>(row + static_cast<long long>(n) * (kT == IGC_F32 ? 4 : 2), v);
    return;
  }
  if constexpr (kT == IGC_F32) {
    float* p = reinterpret_cast<float*>(row) + n;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) p[i] = v[i];
  } else {
    constexpr bool bf16 = kT == IGC_BF16;
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + n;
    const uint32_t w[4] = {pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16),
                           pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16)};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) p[i] = static_cast<uint16_t>(i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
  }
}

template <int kT>
__device__ __forceinline__ float load1(const char* row, int n) {
  if constexpr (kT == IGC_F32)
    return reinterpret_cast<const float*>(row)[n];
  else
    return load16(row, n, kT == IGC_BF16);
}
template <int kT>
__device__ __forceinline__ void store1(char* row, int n, float v) {
  if constexpr (kT == IGC_F32)
    reinterpret_cast<float*>(row)[n] = v;
  else
    store16(row, n, v, kT == IGC_BF16);
}

// w moved up by `bytes` (a multiple of 4, less than 16) of its kN words: what lies past its end is
// undefined.
template <int kN>
__device__ __forceinline__ void shift_words(uint32_t (&w)[kN], uint32_t bytes) {
#pragma unroll
  for (int i = 0; i + 2 < kN; ++i) w[i] = bytes & 8u ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i + 1 < kN; ++i) w[i] = bytes & 4u ? w[i + 1] : w[i];
}

// load8 for a row off 16-byte boundaries: the 16-byte pieces that hold the unit, where they lie
// within the row, are loaded and shifted into place (what neighbours hold in them is not used);
// the units at the ends of a row are loaded one by one.  (Of use where a kernel has few registers
// to lose: beside the other loads of the dropout and the lookup it made their aligned rows slower
// by a sixth to a quarter, and rows off boundaries no faster.)
template <int kT>
__device__ __forceinline__ Raw8<kT> load8_shifted(const char* row, int n, int N) {
  if (n < 8 || n > N - 16) return load8<kT>(row, n, N, false);
  constexpr int kPieces = kT == IGC_F32 ? 3 : 2;
  const char* at = row + static_cast<long long>(n) * (kT == IGC_F32 ? 4 : 2);
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
  const uint4* p = reinterpret_cast<const uint4*>(at - off);
  uint32_t w[4 * kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint4 q = p[i];
    w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
  }
  shift_words(w, off);
  Raw8<kT> r;
  if constexpr (kT == IGC_F32) {
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const uint32_t s = (off & 3u) * 8u;
    r.q[0] = make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                        __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
  }
  return r;
}

// store8 by a whole warp whose lanes hold adjacent units of a row.  `there`: whether the lane has
// one.  Rows off 16-byte boundaries are written in aligned 16-byte pieces all the same: a lane writes
// the piece that its unit begins in, together with what the lane before it has of that piece.
template <int kT>
__device__ __forceinline__ void store8_warp(char* row, int n, int N, bool vec, bool there,
                                            const float (&v)[8]) {
  if (vec) {
    if (there) store8<kT>(row, n, N, true, v);
    return;
  }
  constexpr int kSize = kT == IGC_F32 ? 4 : 2, kWords = 2 * kSize;
  uint32_t w[kWords + 4];  // the last 16 bytes of the lane before, then this lane's
  if constexpr (kT == IGC_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[4 + i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = pack16(v[2 * i], v[2 * i + 1], kT == IGC_BF16);
  }
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[kWords + i], 1);
  const bool whole = there && n + 8 <= N;
  const uint32_t wholes = __ballot_sync(0xffffffffu, whole);
  if (!there) return;
  if (!whole) {
    store8<kT>(row, n, N, false, v);
    return;
  }
  char* at = row + static_cast<long long>(n) * kSize;
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
  if (off == 0) {
    store_unit<kT>(at, v);
    return;
  }
  const bool before = lane > 0 && (wholes >> (lane - 1) & 1u);
  const bool after = lane < 31 && (wholes >> (lane + 1) & 1u);
  const uint32_t from = 16u - off;  // bytes of this lane in the piece that it begins in
  if (!before || !after) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool first = static_cast<uint32_t>(i * kSize) < from;
      // (an fp32 unit has a whole piece between its ends)
      const bool last = static_cast<uint32_t>(i * kSize) >= 8 * kSize - off;
      if ((first && !before) || (last && !after)) {
        if constexpr (kT == IGC_F32)
          reinterpret_cast<float*>(at)[i] = v[i];
        else
          store16(at, i, v[i], kT == IGC_BF16);
      }
    }
  }
  shift_words(w, from);
  uint4* to = reinterpret_cast<uint4*>(at - off);
  if constexpr (kT == IGC_F32) {
    if (before) to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const uint32_t s = (from & 3u) * 8u;
    if (before)
      to[0] = make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                         __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
  }
}

// Of a unit of columns [n, n + 8) those past the row's end become v.
__device__ __forceinline__ void fill_past(float (&s)[8], int n, int N, float v) {
  if (n + 8 <= N) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (n + j >= N) s[j] = v;
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
// two fp32 values in one instruction
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(uint64_t p) {
  float lo, hi;
  unpair(p, lo, hi);
  return lo + hi;
}

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011): ten rounds, each two 32 x 32 -> 64 bit
// products and two three-way exclusive ors with the round's keys.
constexpr int kPhiloxRounds = 10;

struct Drop {
  uint32_t key[kPhiloxRounds][2] = {};  // the seed, stepped from round to round
  uint64_t offset = 0;
  const uint64_t* step = nullptr;
  uint32_t threshold = 0;  // T << 16 (T < 65536; no dropout is another variant of a kernel)
  float scale = 1.0f;      // 65536 / T (0 for T = 0)
};

__device__ __forceinline__ uint4 philox(const Drop& d, uint4 c) {
#pragma unroll
  for (int r = 0; r < kPhiloxRounds; ++r) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ d.key[r][0], static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ d.key[r][1], static_cast<uint32_t>(a));
  }
  return c;
}

// The random bits of eight elements of row `row` from column n (a multiple of 8) on.  One block
// of Philox for all eight, 16 bits each: 5 instructions an element beside the 10 that 32 bits
// each would take, and p to 2^-17 is finer than a rate is ever set.
__device__ __forceinline__ uint4 drop_bits(const Drop& d, uint64_t offset, long long row, int n) {
  return philox(d, make_uint4(static_cast<uint32_t>(n) / 8u, static_cast<uint32_t>(row),
                              static_cast<uint32_t>(offset),
                              static_cast<uint32_t>(offset >> 32)));
}

// v: eight elements; each becomes v * scale + r if its bits keep it, else r.  What is dropped is
// selected away, not multiplied by 0: an infinity there leaves nothing.
__device__ __forceinline__ void drop8(const Drop& d, uint4 q, float (&v)[8],
                                      const float (&r)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a half is under T just where the word that has it as its upper half is under T << 16
    v[2 * i] = (w[i] << 16) < d.threshold ? fmaf(v[2 * i], d.scale, r[2 * i]) : r[2 * i];
    v[2 * i + 1] = w[i] < d.threshold ? fmaf(v[2 * i + 1], d.scale, r[2 * i + 1]) : r[2 * i + 1];
  }
}
__device__ __forceinline__ void drop8(const Drop& d, uint4 q, float (&v)[8]) {
  const float none[8] = {};
  drop8(d, q, v, none);
}

// One element, of column n.
__device__ __forceinline__ float drop1(const Drop& d, uint64_t offset, long long row, int n,
                                       float v, float r) {
  const uint4 q = drop_bits(d, offset, row, n);
  const int i = n % 8 / 2;
  const uint32_t w = i < 2 ? (i == 0 ? q.x : q.y) : (i == 2 ? q.z : q.w);
  return (n % 2 ? w : w << 16) < d.threshold ? fmaf(v, d.scale, r) : r;
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

// A barrier of the kThreads threads of group `group` (of a block that is all of them, or several
// groups: each has a barrier of its own).
template <int kThreads>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (kThreads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kThreads) : "memory");
}

// kThreads <= 32: a warp or an aligned part of one; else a group of kThreads threads, through its
// red (16-byte aligned; one
// array of kThreads / 32 values for each sum that may be in flight between two barriers).
template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float* red, int group = 0) {
#pragma unroll
  for (int o = (kThreads < 32 ? kThreads : 32) / 2; o > 0; o /= 2)
    v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kThreads > 32) {
    constexpr int kWarps = kThreads / 32;
    if (threadIdx.x % 32 == 0) red[threadIdx.x % kThreads / 32] = v;
    group_sync<kThreads>(group);
    if constexpr (kWarps % 4 == 0) {
      uint64_t s = 0;
#pragma unroll
      for (int i = 0; i < kWarps / 4; ++i) {
        const float4 q = reinterpret_cast<const float4*>(red)[i];
        s = add2(s, add2(pair(q.x, q.y), pair(q.z, q.w)));
      }
      v = sum2(s);
    } else {
      v = red[0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) v += red[i];
    }
  }
  return v;
}

// a / n, rounded to nearest, from inv = 1 / n (rounded to nearest); fp32 holds n up to 2^24.  The
// product a * inv alone is a step off for many a even where n divides a, and a row of one value
// would not have it as its mean.  The remainder of the product, which is exact, corrects it (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990).  (A
// division there took 1 to 5 % of a pass over rows: its branch for extreme values holds registers.)
__device__ __forceinline__ float quotient(float a, int n, float inv) {
  const float q = a * inv;
  return fabsf(q) < INFINITY ? fmaf(fmaf(-q, static_cast<float>(n), a), inv, q) : q;
}

// Two sums at once over kThreads <= 32 lanes: half the lanes carry one sum on, half the other,
// which is the upper half's (of all kThreads).
template <int kThreads>
__device__ __forceinline__ float pair_sum(float a, float b, bool upper) {
  float v = upper ? b : a;
  v += __shfl_xor_sync(0xffffffffu, upper ? a : b, kThreads / 2);
#pragma unroll
  for (int o = kThreads / 4; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Both sums in every one of kThreads <= 32 lanes.
template <int kThreads>
__device__ __forceinline__ void lane_sums(float& a, float& b) {
  const bool upper = threadIdx.x % kThreads >= kThreads / 2;
  const float v = pair_sum<kThreads>(a, b, upper);
  const float other = __shfl_xor_sync(0xffffffffu, v, kThreads / 2);
  a = upper ? other : v;
  b = upper ? v : other;
}

// Both sums over kThreads >= 64 threads.  First each warp leaves its own in red (kThreads / 32
// pairs, 16-byte aligned); after a barrier every thread adds the warps'.
template <int kThreads>
__device__ __forceinline__ void leave_sums(float a, float b, float2* red) {
  const int lane = threadIdx.x % 32;
  const bool upper = lane >= 16;
  const float v = pair_sum<32>(a, b, upper);
  if (lane % 16 == 0) reinterpret_cast<float*>(red + threadIdx.x % kThreads / 32)[upper] = v;
}
template <int kThreads>
__device__ __forceinline__ void take_sums(float& a, float& b, const float2* red) {
  constexpr int kWarps = kThreads / 32;
  uint64_t s = kWarps % 2 ? pair(red[kWarps - 1].x, red[kWarps - 1].y) : 0;
#pragma unroll
  for (int i = 0; i < kWarps / 2; ++i) {
    const float4 q = reinterpret_cast<const float4*>(red)[i];
    s = add2(s, add2(pair(q.x, q.y), pair(q.z, q.w)));
  }
  unpair(s, a, b);
}

}  // namespace igc
