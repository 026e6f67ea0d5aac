// embedding_backward: dW[v] = scale * sum of dY[i] over the positions i of token v.
//
// Bound by memory: dY is read once and dW written once (a training batch touches a small part of
// a large table: most of the time goes to the zeros of the rest).
//
// Few positions: one launch.  A block per position (and 512 columns) looks through all tokens;
// the block of a token's first position adds the rows of all its positions, in four shares.
// Further blocks write the zeros of the rows that no token points to.
//
// Many: the positions are sorted by token first (stable, so that a token's positions stay in
// order), with a radix sort.  Blocks then walk chunks of 32 to 128 sorted positions and write each
// token's sum; the sums of a token that crosses a chunk's border go to the workspace, and a last
// kernel adds them in order.  No atomics on sums.  32768 positions of 131072 x 4096 bf16: 208 us,
// 1.34 GB at 6.5 TB/s, 21 us of it the sort.
#include <mutex>

#include "layers_host.h"

namespace igc {

namespace {

constexpr int kThreads = 128;       // of a block over 1024 columns
constexpr int kSmallUnits = 64, kSmallSubs = 4;  // few positions: 512 columns, four shares of rows
constexpr int kSmallThreads = kSmallUnits * kSmallSubs;
constexpr int kSmallM = 1024;       // positions up to which one launch does
constexpr int kMinChunk = 32, kMaxChunk = 128;  // sorted positions of a chunk
constexpr int kMaxSpan = 2048;                  // and of a block's chunks
constexpr int kAhead = 8, kSmallAhead = 4;  // rows that a thread loads before it adds the first
constexpr int kZeroRows = 64;       // of a block that writes zeros, at most
constexpr int kSortThreads = 1024, kSortBlocks = 64;
constexpr int kMaxDigit = 512;      // values of a digit of the radix sort
constexpr int kBatch = 4;           // steps of 32 positions that a warp of the sort has at once

struct EmbedParams {
  int M, D, vec, token64, accumulate;
  int slabs;                 // blocks to a row
  int chunk;                 // sorted positions that one thread adds
  int zero_rows;             // rows of a block that writes zeros, and those blocks
  unsigned zero_blocks;
  long long V;
  const void* tokens;
  const void* dY;
  void* dW;
  long long lddy, lddw;
  float scale;
  uint2* pairs[2];           // sorted: token (V: none of the table's) and position
  uint8_t* touched;          // 1 for each row of dW that a token points to
  uint32_t* counts;          // [block of the sort][digit]
  float* partial;            // [chunk][2][D]: sums of a chunk's first and last token
  int digit_bits, passes;
  int sort_steps;            // steps of 32 positions of a warp of the sort
  int lanes_log2;            // threads that share a chunk's row in a block of the sums
};

__device__ __forceinline__ long long token_at(const EmbedParams& p, int i) {
  return p.token64 ? static_cast<const long long*>(p.tokens)[i]
                   : static_cast<const int*>(p.tokens)[i];
}

// Tokens of the positions first + k * step (k < kN) before end, -1 for the others: all loaded
// before the first is looked at.
template <int kN>
__device__ __forceinline__ void tokens_at(const EmbedParams& p, long long first, int step,
                                          long long end, long long (&v)[kN]) {
  if (p.token64) {
    const long long* t = static_cast<const long long*>(p.tokens);
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = first + k * step < end ? t[first + k * step] : -1;
  } else {
    const int* t = static_cast<const int*>(p.tokens);
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = first + k * step < end ? t[first + k * step] : -1;
  }
}

// dW[v] (8 columns) = scale * acc, added to what is there when accumulating.
template <int kW>
__device__ __forceinline__ void finish8(const EmbedParams& p, long long v, int n, bool vec,
                                        const float (&acc)[8]) {
  char* row = row_at<kW>(p.dW, v, p.lddw);
  float out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = acc[j] * p.scale;
  if (p.accumulate) {
    float old[8];
    unpack8<kW>(load8<kW>(row, n, p.D, vec), old);
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] += old[j];
  }
  store8<kW>(row, n, p.D, vec, out);
}

template <int kY>
__device__ __forceinline__ void add8(const Raw8<kY>& y, float (&acc)[8]) {
  float f[8];
  unpack8<kY>(y, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] += f[j];
}

template <int kW, int kStep>
__device__ __forceinline__ void zero_row(const EmbedParams& p, long long v, bool vec) {
  const float zero[8] = {};
  char* row = row_at<kW>(p.dW, v, p.lddw);
  for (long long n = threadIdx.x * 8; n < p.D; n += kStep * 8)
    store8<kW>(row, static_cast<int>(n), p.D, vec, zero);
}

// ---------------------------------------------------------------------------
// few positions
// ---------------------------------------------------------------------------
template <int kY, int kW>
__global__ void __launch_bounds__(kSmallThreads, 4) embed_small_kernel(const EmbedParams p) {
  __shared__ uint32_t bits[kSmallM / 32];
  __shared__ float4 tot[kSmallSubs - 1][2][kSmallUnits];
  grid_dependency_wait();
  grid_dependents_launch();
  const bool vec = p.vec != 0;
  constexpr int kPer = kSmallM / kSmallThreads;
  if (blockIdx.x < p.zero_blocks) {
    // the rows [v0, v1): bits says which a token points to
    const long long v0 = static_cast<long long>(blockIdx.x) * p.zero_rows;
    const long long v1 = min(p.V, v0 + p.zero_rows);
    if (threadIdx.x < 2) bits[threadIdx.x] = 0;
    __syncthreads();
    long long v[kPer];
    tokens_at<kPer>(p, threadIdx.x, kSmallThreads, p.M, v);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (v[k] >= v0 && v[k] < v1) atomicOr(&bits[(v[k] - v0) / 32], 1u << ((v[k] - v0) % 32));
    __syncthreads();
    for (long long r = v0; r < v1; ++r)
      if (!(bits[(r - v0) / 32] >> ((r - v0) % 32) & 1u)) zero_row<kW, kSmallThreads>(p, r, vec);
    return;
  }
  const int i = static_cast<int>((blockIdx.x - p.zero_blocks) / p.slabs);
  // bit j: position j holds the same token as position i
  const int words = (p.M + 31) / 32;
  long long held[kPer];
  tokens_at<kPer>(p, threadIdx.x, kSmallThreads, p.M, held);
  const long long v = token_at(p, i);
  if (v < 0 || v >= p.V) return;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t same = __ballot_sync(0xffffffffu, held[k] == v);
    if (threadIdx.x % 32 == 0)
      bits[(k * kSmallThreads + static_cast<int>(threadIdx.x)) / 32] = same;
  }
  __syncthreads();
  uint32_t earlier = 0;
  for (int k = 0; k < i / 32; ++k) earlier |= bits[k];
  if (earlier != 0 || (bits[i / 32] & ((1u << (i % 32)) - 1u)) != 0) return;
  const int unit = static_cast<int>(threadIdx.x) % kSmallUnits;
  const int sub = static_cast<int>(threadIdx.x) / kSmallUnits;
  const int n =
      (static_cast<int>((blockIdx.x - p.zero_blocks) % p.slabs) * kSmallUnits + unit) * 8;
  // of the token's positions in order, each share has every kSmallSubs-th; it loads a few rows
  // before it adds the first
  float acc[8] = {};
  int k = i / 32, count = 0;
  uint32_t left = bits[k];
  for (bool more = n < p.D; more;) {
    Raw8<kY> y[kSmallAhead];
    int found = 0;
#pragma unroll
    for (int a = 0; a < kSmallAhead; ++a) {
      int j = -1;
      while (true) {
        while (left == 0 && k + 1 < words) left = bits[++k];
        if (left == 0) break;
        j = k * 32 + __ffs(static_cast<int>(left)) - 1;
        left &= left - 1;
        if (count++ % kSmallSubs == sub) break;
        j = -1;
      }
      if (j < 0) continue;
      y[a] = load8<kY>(row_at<kY>(p.dY, j, p.lddy), n, p.D, vec);
      found = a + 1;
    }
#pragma unroll
    for (int a = 0; a < kSmallAhead; ++a)
      if (a < found) add8<kY>(y[a], acc);
    more = found == kSmallAhead;
  }
  if (sub > 0) {
    tot[sub - 1][0][unit] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    tot[sub - 1][1][unit] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  if (sub > 0 || n >= p.D) return;
#pragma unroll
  for (int r = 0; r < kSmallSubs - 1; ++r) {
    const float4 a = tot[r][0][unit], b = tot[r][1][unit];
    acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
    acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
  }
  finish8<kW>(p, v, n, vec, acc);
}

// ---------------------------------------------------------------------------
// many positions: the sort
// ---------------------------------------------------------------------------
// One pass of the radix sort is two kernels of at most kSortBlocks blocks, each with a run of
// positions (kSortThreads of them up to 65536 positions in all, a multiple of that beyond),
// whose warps have runs of their own in it.  Every warp counts its digits; the first kernel
// writes each block's counts, the second adds those of the smaller digits and of the blocks
// before, and moves its run there.  (One cluster of eight blocks for all passes, with barriers
// in place of launches, took 25 us for 32768 positions; the four kernels take 21.)
struct SortRun {
  uint32_t key[kBatch], pos[kBatch], at[kBatch];
};

struct Sorter {
  const EmbedParams& p;
  const int pass, warp, lane, digits, steps;
  const long long first;
  uint32_t* mine;  // the warp's counts of digits

  __device__ __forceinline__ Sorter(const EmbedParams& q, int number, uint32_t* hist)
      : p(q), pass(number), warp(threadIdx.x / 32), lane(threadIdx.x % 32),
        digits(1 << q.digit_bits), steps(q.sort_steps),
        first((static_cast<long long>(blockIdx.x) * (kSortThreads / 32) + threadIdx.x / 32) *
              (q.sort_steps * 32)),
        mine(hist + threadIdx.x / 32 * (1 << q.digit_bits)) {}

  __device__ __forceinline__ uint32_t digit_of(uint32_t key) const {
    return (key >> (pass * p.digit_bits)) & static_cast<uint32_t>(digits - 1);
  }
  // kBatch steps of 32 positions
  __device__ __forceinline__ void load(SortRun& r, int batch) const {
    const long long from = first + batch * (kBatch * 32) + lane;
    const long long end = min(static_cast<long long>(p.M), first + steps * 32);
    if (pass == 0) {
      long long v[kBatch];
      tokens_at<kBatch>(p, from, 32, end, v);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        r.key[k] = static_cast<uint32_t>(v[k] >= 0 && v[k] < p.V ? v[k] : p.V);
        r.pos[k] = static_cast<uint32_t>(from + k * 32);
      }
    } else {
      const uint2* in = p.pairs[(pass + p.passes) & 1];
      uint2 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        v[k] = from + k * 32 < end ? in[from + k * 32] : make_uint2(0, 0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r.key[k] = v[k].x, r.pos[k] = v[k].y;
    }
  }
  __device__ __forceinline__ bool holds(int batch, int k) const {
    return batch * kBatch + k < steps && first + (batch * kBatch + k) * 32 + lane < p.M;
  }
  // at: the keys' places among those of their digit, counted in mine
  __device__ __forceinline__ void rank(SortRun& r, int batch) const {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (batch * kBatch + k >= steps) break;
      const bool valid = holds(batch, k);
      // (a lane past the last position has a digit that no other has)
      const uint32_t d = valid ? digit_of(r.key[k]) : 0xffffffffu;
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const uint32_t ahead = __popc(peers & ((1u << lane) - 1u));
      if (valid) r.at[k] = mine[d] + ahead;
      __syncwarp();
      if (valid && ahead == 0) mine[d] += __popc(peers);
      __syncwarp();
    }
  }
  // The rows of dW that a token points to: set by the positions whose neighbour holds another
  // token.  (In the second pass, where most of a token's positions are neighbours: set by every
  // position, the bytes of frequent tokens took 3 us of a training batch.  Warps that set the
  // same byte set it to the same.)
  __device__ __forceinline__ void mark(const SortRun& r, int batch) const {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t other = __shfl_up_sync(0xffffffffu, r.key[k], 1);
      if (holds(batch, k) && r.key[k] < p.V && (lane == 0 || other != r.key[k]))
        p.touched[r.key[k]] = 1;
    }
  }
  __device__ __forceinline__ void clear() const {
    for (int d = lane; d < digits; d += 32) mine[d] = 0;
    __syncwarp();
  }
  __device__ __forceinline__ int batches() const { return (steps + kBatch - 1) / kBatch; }
};

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const EmbedParams p, int pass) {
  extern __shared__ uint32_t hist[];  // [32 warps][digits]
  const Sorter s(p, pass, hist);
  s.clear();
  grid_dependency_wait();
  grid_dependents_launch();
  if (pass == 0 && p.touched != nullptr)  // (its place in the workspace is a multiple of 256)
    for (long long k = static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x;
         k < (p.V + 15) / 16; k += static_cast<long long>(gridDim.x) * kSortThreads)
      reinterpret_cast<uint4*>(p.touched)[k] = make_uint4(0, 0, 0, 0);
  SortRun r;
  for (int batch = 0; batch < s.batches(); ++batch) {
    s.load(r, batch);
    s.rank(r, batch);
    if (pass == 1 && p.touched != nullptr) s.mark(r, batch);
  }
  __syncthreads();
  const int d = static_cast<int>(threadIdx.x);
  if (d < s.digits) {
    uint32_t sum = 0;
#pragma unroll 16
    for (int w = 0; w < kSortThreads / 32; ++w) sum += hist[w * s.digits + d];
    p.counts[blockIdx.x * s.digits + d] = sum;
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_move_kernel(const EmbedParams p, int pass) {
  extern __shared__ uint32_t hist[];  // [32 warps][digits]: counts, then places
  __shared__ uint32_t part[2][kMaxDigit], scan[32];
  const Sorter s(p, pass, hist);
  s.clear();
  grid_dependency_wait();
  grid_dependents_launch();
  SortRun r;
  s.load(r, 0);
  // two threads to a digit, half of the blocks each: all blocks' counts, and those before this
  const int d = static_cast<int>(threadIdx.x) % kMaxDigit, half = threadIdx.x / kMaxDigit;
  const int rank = static_cast<int>(blockIdx.x), blocks = static_cast<int>(gridDim.x);
  uint32_t all = 0, before = 0;
  if (d < s.digits) {
#pragma unroll 16
    for (int c = half; c < blocks; c += 2) {
      const uint32_t v = p.counts[c * s.digits + d];
      all += v;
      if (c < rank) before += v;
    }
  }
  if (half == 1) {
    part[0][d] = all;
    part[1][d] = before;
  }
  const bool kept = s.batches() == 1;
  s.rank(r, 0);
  if (!kept) {
    for (int batch = 1; batch < s.batches(); ++batch) {
      s.load(r, batch);
      s.rank(r, batch);
    }
  }
  __syncthreads();
  if (half == 0) all += part[0][d], before += part[1][d];
  // the smaller digits' counts
  uint32_t upto = half == 0 ? all : 0;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (s.lane >= o) upto += v;
  }
  if (s.lane == 31) scan[s.warp] = upto;
  __syncthreads();
  uint32_t ahead = s.lane < s.warp ? scan[s.lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
  // the warps' counts become places
  if (half == 0 && d < s.digits) {
    uint32_t place = ahead + upto - all + before;
#pragma unroll 16
    for (int w = 0; w < kSortThreads / 32; ++w) {
      const uint32_t c = hist[w * s.digits + d];
      hist[w * s.digits + d] = place;
      place += c;
    }
  }
  __syncthreads();
  uint2* out = p.pairs[(pass + p.passes + 1) & 1];
  for (int batch = 0; batch < s.batches(); ++batch) {
    if (!kept) {
      s.load(r, batch);
      s.rank(r, batch);  // (from the places on now)
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!s.holds(batch, k)) continue;
      const uint32_t to = r.at[k] + (kept ? s.mine[s.digit_of(r.key[k])] : 0u);
      out[to] = make_uint2(r.key[k], r.pos[k]);
    }
    if (p.passes == 1 && p.touched != nullptr) s.mark(r, batch);
  }
}

// ---------------------------------------------------------------------------
// many positions: the sums
// ---------------------------------------------------------------------------
// A block has kThreads units of eight columns: of one chunk's rows or, where rows are narrow, of
// several chunks'.
template <int kY, int kW>
__global__ void __launch_bounds__(kThreads) embed_sums_kernel(const EmbedParams p) {
  __shared__ uint32_t keys[kMaxSpan + 2], pos[kMaxSpan];
  grid_dependency_wait();
  grid_dependents_launch();
  const bool vec = p.vec != 0;
  const int chunks = (p.M + p.chunk - 1) / p.chunk;
  const int subs = kThreads >> p.lanes_log2;  // chunks of a block
  const unsigned sum_blocks = static_cast<unsigned>((chunks + subs - 1) / subs) * p.slabs;
  if (blockIdx.x >= sum_blocks) {
    const long long v0 = static_cast<long long>(blockIdx.x - sum_blocks) * p.zero_rows;
    const long long v1 = min(p.V, v0 + p.zero_rows);
    if (v0 + static_cast<int>(threadIdx.x) < v1 && threadIdx.x < kZeroRows)
      keys[threadIdx.x] = p.touched[v0 + threadIdx.x];
    __syncthreads();
    for (long long v = v0; v < v1; ++v)
      if (keys[v - v0] == 0) zero_row<kW, kThreads>(p, v, vec);
    return;
  }
  const int sub = static_cast<int>(threadIdx.x) >> p.lanes_log2;
  const int lane = static_cast<int>(threadIdx.x) & ((1 << p.lanes_log2) - 1);
  const int c0 = static_cast<int>(blockIdx.x / p.slabs) * subs;
  const long long p0 = static_cast<long long>(c0) * p.chunk;
  const uint32_t none = static_cast<uint32_t>(p.V);
  // keys[k + 1]: token of the block's position k; a token that is not in the table before the
  // first position, after the last, and for what is not to be summed
  for (int k = threadIdx.x; k < subs * p.chunk + 2; k += kThreads) {
    const long long at = p0 + k - 1;
    const uint2 v = at >= 0 && at < p.M ? p.pairs[0][at] : make_uint2(none, 0);
    keys[k] = v.x;
    if (k > 0 && k <= subs * p.chunk) pos[k - 1] = v.y;
  }
  __syncthreads();
  const int n = (static_cast<int>(blockIdx.x % p.slabs) * kThreads + lane) * 8;
  if (n >= p.D) return;
  const uint32_t* key = keys + sub * p.chunk;
  const uint32_t* at = pos + sub * p.chunk;
  float acc[8] = {};
  bool from_start = key[0] == key[1];  // the token at hand began in an earlier chunk
  for (int k0 = 0; k0 < p.chunk; k0 += kAhead) {
    Raw8<kY> y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (key[k0 + k + 1] != none)
        y[k] = load8<kY>(row_at<kY>(p.dY, at[k0 + k], p.lddy), n, p.D, vec);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t v = key[k0 + k + 1];
      if (v == none) return;  // the rest holds no tokens of the table
      add8<kY>(y[k], acc);
      const bool last = k0 + k == p.chunk - 1, goes_on = key[k0 + k + 2] == v;
      if (goes_on && !last) continue;
      if (from_start || goes_on) {
        float* out =
            p.partial + (static_cast<long long>(c0 + sub) * 2 + (from_start ? 0 : 1)) * p.D;
        store8<IGC_F32>(reinterpret_cast<char*>(out), n, p.D,
                        (reinterpret_cast<uintptr_t>(out) & 15u) == 0, acc);
      } else {
        finish8<kW>(p, v, n, vec, acc);
      }
      from_start = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    }
  }
}

// Tokens that cross chunks: the sum of the chunk where one begins and of those it goes on in.
// A block has 256 columns and looks at 8 chunks, a warp at each: a token that goes on in few
// chunks is the warp's, one that goes on in many is then shared by all 8 warps.
constexpr int kJoinWarps = 8, kJoinAhead = 4;

template <int kW>
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const EmbedParams p) {
  __shared__ float tot[kJoinWarps][256];
  __shared__ int long_end[kJoinWarps];  // last chunk of the token that begins in a warp's chunk
  grid_dependency_wait();
  grid_dependents_launch();
  const bool vec = p.vec != 0;
  const int chunks = (p.M + p.chunk - 1) / p.chunk;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int col_blocks = (p.D + 255) / 256;
  const long long n0 = static_cast<long long>(blockIdx.x % col_blocks) * 256 + lane * 8;
  const int n = static_cast<int>(n0), c0 = static_cast<int>(blockIdx.x / col_blocks) * kJoinWarps;
  // chunk k's part of the token that begins in chunk c: of its last token there, of its first
  // in those after
  auto part = [&](int k, int c) {
    const float* from = p.partial + (static_cast<long long>(k) * 2 + (k == c ? 1 : 0)) * p.D;
    return load8<IGC_F32>(reinterpret_cast<const char*>(from), n, p.D,
                          (reinterpret_cast<uintptr_t>(from) & 15u) == 0);
  };
  const int mine = c0 + warp;
  const long long p0 = static_cast<long long>(mine) * p.chunk, next = p0 + p.chunk;
  int end = -1;
  uint32_t v = 0;
  if (next < p.M) {
    v = p.pairs[0][next - 1].x;
    const uint32_t after = p.pairs[0][next].x;
    const uint32_t ahead = p0 > 0 ? p.pairs[0][p0 - 1].x : ~v;
    if (v < p.V && after == v && ahead != v) {
      // the chunk that it ends in: the tokens ascend, 32 chunks are looked at at once
      end = mine + 1;
      while (true) {
        const long long k = static_cast<long long>(end) + 1 + lane;
        const uint32_t more =
            __ballot_sync(0xffffffffu, k < chunks && p.pairs[0][k * p.chunk].x == v);
        end += __popc(more);
        if (more != 0xffffffffu) break;
      }
    }
  }
  const bool shared = end - mine >= kJoinAhead;
  if (lane == 0) long_end[warp] = end >= 0 && shared ? end : -1;
  if (end >= 0 && !shared && n0 < p.D) {
    Raw8<IGC_F32> f[kJoinAhead];
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (mine + k <= end) f[k] = part(mine + k, mine);
    float acc[8] = {};
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (mine + k <= end) add8<IGC_F32>(f[k], acc);
    finish8<kW>(p, v, n, vec, acc);
  }
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) {
    const int last = long_end[w], c = c0 + w;
    if (last < 0) continue;
    float acc[8] = {};
    if (n0 < p.D) {
#pragma unroll 4
      for (int k = c + warp; k <= last; k += kJoinWarps) add8<IGC_F32>(part(k, c), acc);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) tot[warp][lane * 8 + j] = acc[j];
    __syncthreads();
    if (warp == 0 && n0 < p.D) {
      for (int r = 1; r < kJoinWarps; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += tot[r][lane * 8 + j];
      finish8<kW>(p, p.pairs[0][static_cast<long long>(c) * p.chunk + p.chunk - 1].x, n, vec, acc);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Fewer borders for tokens to cross where there is work for every SM without them.
inline int64_t chunk_of(int64_t M, int64_t D) {
  const int64_t units = (D + 7) / 8;
  int64_t chunk = kMinChunk;
  while (chunk < kMaxChunk && M > 128 * 1024 / units * chunk) chunk *= 2;
  return chunk;
}
inline int64_t chunks_of(int64_t M, int64_t D) {
  const int64_t chunk = chunk_of(M, D);
  return (M + chunk - 1) / chunk;
}
// Steps of 32 positions of a warp of the sort.
inline int64_t sort_steps(int64_t M) {
  const int64_t most = static_cast<int64_t>(kSortThreads) * kSortBlocks;
  return (M + most - 1) / most;
}
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct EmbedLayout {
  size_t pairs[2], touched, counts, partial, bytes;
};
EmbedLayout layout(int64_t M, int64_t V, int64_t D) {
  EmbedLayout l = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  if (M > kSmallM && V > 0 && D > 0) {
    for (int i = 0; i < 2; ++i) l.pairs[i] = take(static_cast<size_t>(M) * sizeof(uint2));
    l.touched = take(static_cast<size_t>(V));
    l.counts = take(static_cast<size_t>(kSortBlocks) * kMaxDigit * 4);
    l.partial = take(static_cast<size_t>(chunks_of(M, D)) * 2 * static_cast<size_t>(D) * 4);
  }
  l.bytes = at;
  return l;
}

// The sort's kernels may have their shared memory, on this device.
int sort_setup(const DeviceInfo& dev) {
  static std::once_flag once[64];
  static int rc[64];
  std::call_once(once[dev.device], [&] {
    rc[dev.device] = IGC_OK;
    for (auto kernel : {embed_count_kernel, embed_move_kernel}) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (kSortThreads / 32) * kMaxDigit * 4) != cudaSuccess) {
        (void)cudaGetLastError();
        rc[dev.device] = IGC_ERR_CUDA;
      }
    }
  });
  return rc[dev.device];
}

template <int kY, int kW>
int run(const DeviceInfo& dev, EmbedParams p, cudaStream_t stream) {
  const long long zero_blocks = p.accumulate ? 0 : (p.V + p.zero_rows - 1) / p.zero_rows;
  p.zero_blocks = static_cast<unsigned>(zero_blocks);
  if (p.M <= kSmallM) {
    const long long blocks = static_cast<long long>(p.M) * p.slabs + zero_blocks;
    if (blocks > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
    if (blocks == 0) return IGC_OK;
    return launch_pdl(embed_small_kernel<kY, kW>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kSmallThreads), 0, stream, p);
  }
  const int chunks = (p.M + p.chunk - 1) / p.chunk, subs = kThreads >> p.lanes_log2;
  const long long blocks =
      static_cast<long long>((chunks + subs - 1) / subs) * p.slabs + zero_blocks;
  const long long join_blocks = static_cast<long long>((chunks + kJoinWarps - 1) / kJoinWarps) *
                                ((static_cast<long long>(p.D) + 255) / 256);
  if (blocks > 0x7fffffff || join_blocks > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
  const int smem = (kSortThreads / 32) * (1 << p.digit_bits) * 4;
  int rc = sort_setup(dev);
  if (rc != IGC_OK) return rc;
  const int run = kSortThreads * p.sort_steps;
  const dim3 sort_grid(static_cast<unsigned>((p.M + static_cast<long long>(run) - 1) / run));
  for (int pass = 0; pass < p.passes; ++pass) {
    for (auto kernel : {embed_count_kernel, embed_move_kernel}) {
      rc = launch_pdl(kernel, sort_grid, dim3(kSortThreads), static_cast<size_t>(smem), stream, p,
                      pass);
      if (rc != IGC_OK) return rc;
    }
  }
  rc = launch_pdl(embed_sums_kernel<kY, kW>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                  0, stream, p);
  if (rc != IGC_OK) return rc;
  return launch_pdl(embed_join_kernel<kW>, dim3(static_cast<unsigned>(join_blocks)),
                    dim3(kJoinWarps * 32), 0, stream, p);
}

}  // namespace

}  // namespace igc

using namespace igc;

extern "C" {

size_t embedding_backward_workspace_size(int64_t M, int64_t V, int64_t D) {
  return M < 0 || V < 0 || D < 0 ? 0 : layout(M, V, D).bytes;
}

int embedding_backward(int64_t M, int64_t V, int64_t D, const void* tokens, int token_bytes,
                       const void* dY, int64_t lddy, int y_dtype, float scale, int accumulate,
                       void* dW, int64_t lddw, int dw_dtype, void* workspace,
                       size_t workspace_bytes, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || V < 0 || D < 0 || (token_bytes != 4 && token_bytes != 8) || !is_type(y_dtype) ||
      !is_type_or_f32(dw_dtype, y_dtype))
    return IGC_ERR_INVALID_ARG;
  if (V == 0 || D == 0 || (M == 0 && accumulate)) return IGC_OK;
  if (!fits32(M) || !fits32(V) || !fits32(D)) return IGC_ERR_UNSUPPORTED;
  if (dW == nullptr || lddw < D || (M > 0 && (tokens == nullptr || dY == nullptr || lddy < D)))
    return IGC_ERR_INVALID_ARG;
  if (is_any(dW, tokens, dY)) return IGC_ERR_INVALID_ARG;
  if (!elements_aligned(Mat{dY, lddy, y_dtype}, Mat{dW, lddw, dw_dtype}) ||
      reinterpret_cast<uintptr_t>(tokens) % token_bytes != 0)
    return IGC_ERR_MISALIGNED;
  DeviceInfo dev;
  const int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  const EmbedLayout l = layout(M, V, D);
  if (l.bytes > 0 && (workspace == nullptr || workspace_bytes < l.bytes ||
                      reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return IGC_ERR_WORKSPACE;
  EmbedParams p = {};
  p.M = static_cast<int>(M), p.D = static_cast<int>(D), p.V = V;
  p.vec = rows_vec(M, dY, lddy, y_dtype) && rows_vec(V, dW, lddw, dw_dtype);
  p.token64 = token_bytes == 8;
  p.accumulate = accumulate != 0;
  const int64_t slab = (M <= kSmallM ? kSmallUnits : kThreads) * 8;
  p.slabs = static_cast<int>((D + slab - 1) / slab);
  p.chunk = static_cast<int>(chunk_of(M, D));
  // chunks of narrow rows share a block
  p.lanes_log2 = 3;
  while ((1 << p.lanes_log2) < kThreads && (8 << p.lanes_log2) < D) ++p.lanes_log2;
  p.sort_steps = static_cast<int>(sort_steps(M));
  // about 64 KB of zeros to a block
  const int64_t rows = 65536 / (D * static_cast<int64_t>(elem_size(dw_dtype)));
  p.zero_rows = static_cast<int>(rows < 1 ? 1 : (rows > kZeroRows ? kZeroRows : rows));
  p.tokens = tokens, p.dY = dY, p.dW = dW;
  p.lddy = lddy, p.lddw = lddw;
  p.scale = scale;
  char* ws = static_cast<char*>(workspace);
  for (int i = 0; i < 2; ++i) p.pairs[i] = reinterpret_cast<uint2*>(ws + l.pairs[i]);
  p.touched = accumulate ? nullptr : reinterpret_cast<uint8_t*>(ws + l.touched);
  p.counts = reinterpret_cast<uint32_t*>(ws + l.counts);
  p.partial = reinterpret_cast<float*>(ws + l.partial);
  int bits = 1;
  while ((static_cast<int64_t>(1) << bits) <= V) ++bits;  // keys are 0 .. V
  p.passes = (bits + 8) / 9;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  if (y_dtype == IGC_F32) return run<IGC_F32, IGC_F32>(dev, p, stream);
  if (y_dtype == IGC_F16)
    return dw_dtype == IGC_F32 ? run<IGC_F16, IGC_F32>(dev, p, stream)
                               : run<IGC_F16, IGC_F16>(dev, p, stream);
  return dw_dtype == IGC_F32 ? run<IGC_BF16, IGC_F32>(dev, p, stream)
                             : run<IGC_BF16, IGC_BF16>(dev, p, stream);
}

}  // extern "C"
