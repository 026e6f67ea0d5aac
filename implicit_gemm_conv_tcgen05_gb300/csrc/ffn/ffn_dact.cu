// The pass through the activation of the feed-forward backward passes, with the bias
// gradients, and the forward pass of an empty contraction.
//
//   linear:  dZ = dY act'(Z)                    db  = column sums of dZ
//   gated:   dU = dH act(G), dG = dH U act'(G)  dbg, dbu = column sums of dG, dU
//
// One pass over memory: a thread keeps 8 adjacent columns (one 16-byte access per
// matrix and row) and walks down the rows of its chunk, so the column sums stay in its
// registers (fp32) and cost no second read.  The threads of a block that share columns
// meet in shared memory, one row of partial sums per chunk goes to the workspace, and a
// second kernel adds the chunks in order (no atomics).  Up to 512 rows, a cluster of up to
// 8 blocks covers a column block's rows and adds its sums through distributed shared memory
// instead: one launch less (2 to 3 us of host time in calls that take about 22).
//
// Bound by memory: gated 8192 x 16384 without sums 190 us, 1.34 GB at 7.1 TB/s; linear 4096 x
// 8192, tanh-GELU with sums, 37 us, 201 MB at 5.4 TB/s (27 instructions an element).
#include "ffn_act.cuh"
#include "ffn_host.h"
#include "ffn_tc.cuh"

namespace igc {

namespace {

constexpr int kThreads = 256;
// Columns of a block, 8 to a thread; the threads of a column walk every kRowLanes-th row.
// Narrow blocks (64 columns, 32 rows at a time) spread a short input over more SMs.
template <int kCols>
struct Block {
  static constexpr int kLanes = kCols / 8, kRowLanes = kThreads / kLanes;
};
constexpr int kWide = 256, kNarrow = 64;
constexpr int kMaxChunks = 256;

struct DactParams {
  int M, N;
  int rows_per_chunk;
  int bf16, act;
  const uint16_t* dO;
  const uint16_t* Z;
  const uint16_t* U;
  long long ldo, ldz, ldu;
  int o_vec, z_vec, u_vec;
  uint16_t* D0;
  uint16_t* D1;
  long long ldd;
  float* partial0;
  float* partial1;
  void* db0;
  void* db1;
  int db_f32;
};

// 8 elements of a row from column n one by one (zeros past N): rows that are not 16-byte
// aligned, and a row's last columns.
__device__ __forceinline__ uint4 load8_single(const uint16_t* row, int n, int N) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = n + 2 * i < N ? row[n + 2 * i] : 0u;
    const uint32_t hi = n + 2 * i + 1 < N ? row[n + 2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// dZ, dG and dU leave in 16 bits because the tensor cores take their operands so; as fp32
// operands (tf32) the products would run at half the rate on twice the bytes and keep 10 bits
// of them.  It is the one rounding that the fp32 form does not have: error against 64 bits of
// dX and dW 0.0023 instead of 0.0017 of their size (bf16), 0.00029 instead of 0.00021 (fp16),
// and fp16's range (igc_ffn.h).  The bias gradients sum what has not been rounded.
// The workspace rows are padded to a multiple of 8 columns: always whole.
__device__ __forceinline__ void save8(uint16_t* row, int n, bool bf16, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(row + n) =
      make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16), pack16(v[4], v[5], bf16),
                 pack16(v[6], v[7], bf16));
}

enum : int { kSumNone = 0, kSumChunks = 1, kSumCluster = 2 };
constexpr int kClusterMaxRows = 512;  // 8 blocks x 32 threads of a column x at most 2 rows

// The block's column sums, its threads' added in order: that of column threadIdx.x (for
// the first kCols threads).
template <int kCols>
__device__ __forceinline__ float block_sum(float (&red)[Block<kCols>::kRowLanes][kCols],
                                           const float (&s)[8]) {
  constexpr int kLanes = Block<kCols>::kLanes, kRowLanes = Block<kCols>::kRowLanes;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) red[threadIdx.x / kLanes][threadIdx.x % kLanes * 8 + i] = s[i];
  __syncthreads();
  float t = 0.0f;
  if (threadIdx.x < kCols) {
#pragma unroll
    for (int w = 0; w < kRowLanes; ++w) t += red[w][threadIdx.x];
  }
  return t;
}

__device__ __forceinline__ void store_sum(void* out, int n, float v, bool f32, bool bf16) {
  if (f32)
    static_cast<float*>(out)[n] = v;
  else
    store16(out, n, v, bf16);
}

// Column sums of the whole cluster from its blocks' sums (tot): each block writes its
// share of the columns.
__device__ __forceinline__ void cluster_sums(const DactParams& p, const float* tot, void* out) {
  const int blocks = static_cast<int>(gridDim.y), share = kNarrow / blocks;
  const int rank = static_cast<int>(cluster_ctarank());
  const int c = rank * share + static_cast<int>(threadIdx.x);
  const int n = static_cast<int>(blockIdx.x) * kNarrow + c;
  if (static_cast<int>(threadIdx.x) >= share || n >= p.N) return;
  float t = 0.0f;
  for (int r = 0; r < blocks; ++r)
    t += __uint_as_float(
        ld_shared_cluster_u32(mapa_shared(smem_u32(tot + c), static_cast<uint32_t>(r))));
  store_sum(out, n, t, p.db_f32, p.bf16);
}

// One row's 8 columns: o, z (and u) come in as dO, Z (U) and leave as D0 (z when gated,
// else o) and D1 (u).
template <bool kGated, int kAct>
__device__ __forceinline__ void dact8(float (&o)[8], float (&z)[8], float (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f, d;
    act_grad_f32<kAct>(z[i], f, d);
    if constexpr (kGated) {
      z[i] = o[i] * u[i] * d;  // dG
      u[i] = o[i] * f;         // dU
    } else {
      o[i] *= d;               // dZ
    }
  }
}

__device__ __forceinline__ void unpack8(uint4 q, bool bf16, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16(w[i], bf16);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}

// Bound by memory where it reads 16-byte vectors: kUnroll rows' loads are issued before
// the first is used, so that an SM keeps some 70 KB in flight.
template <bool kGated, int kAct, int kSum, bool kBf16, int kRowLanes>
__device__ __forceinline__ void dact_rows(const DactParams& p, int n, long long r0, long long r1,
                                          float (&s0)[8], float (&s1)[8]) {
  constexpr int kUnroll = kGated || kSum != kSumNone ? 2 : 4;
  constexpr bool kNeedZ = kGated || kAct != IGC_ACT_NONE;
  constexpr bool bf16 = kBf16;  // (as a run-time flag: 28 instructions an element)
  const bool fast = n + 8 <= p.N && p.o_vec && (!kNeedZ || p.z_vec) && (!kGated || p.u_vec);
  for (long long r = r0; r < r1; r += kUnroll * kRowLanes) {
    uint4 qo[kUnroll], qz[kUnroll], qu[kUnroll];
    if (fast) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const long long rj = r + j * kRowLanes;
        if (rj >= r1) continue;
        qo[j] = *reinterpret_cast<const uint4*>(p.dO + rj * p.ldo + n);
        if constexpr (kNeedZ) qz[j] = *reinterpret_cast<const uint4*>(p.Z + rj * p.ldz + n);
        if constexpr (kGated) qu[j] = *reinterpret_cast<const uint4*>(p.U + rj * p.ldu + n);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const long long rj = r + j * kRowLanes;
        if (rj >= r1) continue;
        qo[j] = load8_single(p.dO + rj * p.ldo, n, p.N);
        if constexpr (kNeedZ) qz[j] = load8_single(p.Z + rj * p.ldz, n, p.N);
        if constexpr (kGated) qu[j] = load8_single(p.U + rj * p.ldu, n, p.N);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const long long rj = r + j * kRowLanes;
      if (rj >= r1) continue;
      float o[8], z[8], u[8];
      unpack8(qo[j], bf16, o);
      if constexpr (kNeedZ) unpack8(qz[j], bf16, z);
      if constexpr (kGated) unpack8(qu[j], bf16, u);
      if constexpr (kNeedZ) dact8<kGated, kAct>(o, z, u);
      float(&d0)[8] = kGated ? z : o;
      if constexpr (kSum != kSumNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s0[i] += d0[i];
          if constexpr (kGated) s1[i] += u[i];
        }
      }
      if (p.D0 != nullptr) {
        save8(p.D0 + rj * p.ldd, n, bf16, d0);
        if constexpr (kGated) save8(p.D1 + rj * p.ldd, n, bf16, u);
      }
    }
  }
}

template <bool kGated, int kAct, int kSum, bool kBf16>
__global__ void __launch_bounds__(kThreads, kGated && kSum != kSumNone ? 2 : 3)
    dact_kernel(const DactParams p) {
  constexpr int kCols = kSum == kSumCluster ? kNarrow : kWide;
  constexpr int kLanes = Block<kCols>::kLanes, kRowLanes = Block<kCols>::kRowLanes;
  grid_dependency_wait();
  grid_dependents_launch();
  const int n = blockIdx.x * kCols + threadIdx.x % kLanes * 8;
  const long long r0 = static_cast<long long>(blockIdx.y) * p.rows_per_chunk;
  const long long r1 = min(static_cast<long long>(p.M), r0 + p.rows_per_chunk);
  float s0[8] = {}, s1[8] = {};
  if (n < p.N)
    dact_rows<kGated, kAct, kSum, kBf16, kRowLanes>(p, n, r0 + threadIdx.x / kLanes, r1, s0, s1);
  if constexpr (kSum != kSumNone) {
    __shared__ float red[kRowLanes][kCols];
    __shared__ float tot[2][kSum == kSumCluster ? kCols : 1];
    const float t0 = block_sum<kCols>(red, s0);
    const float t1 = kGated ? block_sum<kCols>(red, s1) : 0.0f;
    if constexpr (kSum == kSumChunks) {
      const int col = blockIdx.x * kCols + threadIdx.x;
      const long long at = static_cast<long long>(blockIdx.y) * p.N + col;
      if (col < p.N) {
        p.partial0[at] = t0;
        if constexpr (kGated) p.partial1[at] = t1;
      }
    } else {
      if (threadIdx.x < kCols) {
        tot[0][threadIdx.x] = t0;
        tot[1][threadIdx.x] = t1;
      }
      cluster_sync();
      cluster_sums(p, tot[0], p.db0);
      if constexpr (kGated) cluster_sums(p, tot[1], p.db1);
      cluster_sync();  // no block may exit while another reads its sums
    }
  }
}

template <bool kGated, int kSum, bool kBf16>
int launch_dact(const DactParams& p, dim3 grid, cudaStream_t stream) {
  void (*kern)(DactParams) = dact_kernel<kGated, IGC_ACT_NONE, kSum, kBf16>;
  switch (p.act) {
    case IGC_ACT_RELU: kern = dact_kernel<kGated, IGC_ACT_RELU, kSum, kBf16>; break;
    case IGC_ACT_GELU: kern = dact_kernel<kGated, IGC_ACT_GELU, kSum, kBf16>; break;
    case IGC_ACT_GELU_TANH: kern = dact_kernel<kGated, IGC_ACT_GELU_TANH, kSum, kBf16>; break;
    case IGC_ACT_SILU: kern = dact_kernel<kGated, IGC_ACT_SILU, kSum, kBf16>; break;
    default: break;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = grid.y;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kSum == kSumCluster ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return IGC_ERR_CUDA;
  }
  return IGC_OK;
}

template <bool kGated, bool kBf16>
int launch_dact_sum(const DactParams& p, int sum, dim3 grid, cudaStream_t stream) {
  switch (sum) {
    case kSumChunks: return launch_dact<kGated, kSumChunks, kBf16>(p, grid, stream);
    case kSumCluster: return launch_dact<kGated, kSumCluster, kBf16>(p, grid, stream);
    default: return launch_dact<kGated, kSumNone, kBf16>(p, grid, stream);
  }
}

// out[n] = sum over chunks of partial[chunk][n]; blockIdx.y: which vector.
__global__ void __launch_bounds__(256) sum_chunks_kernel(const float* partial0,
                                                         const float* partial1, int chunks, int N,
                                                         void* out0, void* out1, int f32,
                                                         int bf16, int late_wait) {
  __shared__ float red[8][32];
  ffn_dependency_wait(late_wait);
  const float* partial = blockIdx.y ? partial1 : partial0;
  void* out = blockIdx.y ? out1 : out0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (n < N)
    // (from L2: with a late wait nothing has told this SM's L1 of the new sums)
    for (int c = warp; c < chunks; c += 8) t += __ldcg(partial + static_cast<long long>(c) * N + n);
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && n < N) {
#pragma unroll
    for (int w = 1; w < 8; ++w) t += red[w][lane];
    store_sum(out, n, t, f32, bf16);
  }
  ffn_dependency_end(late_wait);
}

// ---------------------------------------------------------------------------
// forward pass over a contraction of length zero: Z = bias
// ---------------------------------------------------------------------------
struct BiasOnlyParams {
  int M, N;
  int bf16, act, gated;
  const void* bias0;
  const void* bias1;
  int bias_f32;
  const void* R;
  long long ldr;
  void* out[3];
  long long ld[3];
  int f32_0;
};

__global__ void __launch_bounds__(256) bias_only_kernel(const BiasOnlyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long total = static_cast<long long>(p.M) * p.N;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const bool bf16 = p.bf16 != 0;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += step) {
    const long long m = i / p.N;
    const int n = static_cast<int>(i - m * p.N);
    const float z = load_vec(p.bias0, n, p.bias_f32, bf16);
    float y = z;
    with_act(p.act, [&](auto a) { y = act_f32<decltype(a)::value>(z); });
    if (p.out[1] != nullptr) store16(p.out[1], m * p.ld[1] + n, z, bf16);
    if (p.gated) {
      const float u = load_vec(p.bias1, n, p.bias_f32, bf16);
      y *= u;
      if (p.out[2] != nullptr) store16(p.out[2], m * p.ld[2] + n, u, bf16);
    } else if (p.R != nullptr) {
      y += load16(p.R, m * p.ldr + n, bf16);
    }
    if (p.f32_0)
      static_cast<float*>(p.out[0])[m * p.ld[0] + n] = y;
    else
      store16(p.out[0], m * p.ld[0] + n, y, bf16);
  }
}

}  // namespace

// Rows of a chunk: a whole number of unrolled steps of a block's warps (8, 16 or a multiple
// of 32 rows), few enough that some 4096 blocks even out over the SMs.
static int64_t dact_rows(int64_t M, int64_t N) {
  const int64_t col_blocks = (N + kWide - 1) / kWide;
  int64_t chunks = col_blocks > 0 ? (4096 + col_blocks - 1) / col_blocks : 1;
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  const int64_t rows = (M + chunks - 1) / chunks;
  return rows <= 8 ? 8 : (rows <= 16 ? 16 : (rows + 31) / 32 * 32);
}

int64_t dact_chunks(int64_t M, int64_t N) {
  const int64_t rows = dact_rows(M, N);
  return M > 0 ? (M + rows - 1) / rows : 1;
}

int ffn_dact(const DactArgs& a, bool gated, cudaStream_t stream) {
  DactParams p = {};
  p.M = static_cast<int>(a.M), p.N = static_cast<int>(a.N);
  const int sum = a.db0 == nullptr ? kSumNone
                                   : (a.M <= kClusterMaxRows ? kSumCluster : kSumChunks);
  int64_t chunks = dact_chunks(a.M, a.N);
  p.rows_per_chunk = static_cast<int>(dact_rows(a.M, a.N));
  if (sum == kSumCluster) {
    for (chunks = 1; chunks < 8 && a.M > chunks * Block<kNarrow>::kRowLanes;) chunks *= 2;
    p.rows_per_chunk = static_cast<int>((a.M + chunks - 1) / chunks);
  }
  p.bf16 = a.dtype == IGC_BF16, p.act = a.act;
  p.dO = static_cast<const uint16_t*>(a.dO.ptr), p.ldo = a.dO.ld;
  p.Z = static_cast<const uint16_t*>(a.Z.ptr), p.ldz = a.Z.ld;
  p.U = static_cast<const uint16_t*>(a.U.ptr), p.ldu = a.U.ld;
  p.o_vec = operand_ok(a.dO.ptr, a.dO.ld);
  p.z_vec = operand_ok(a.Z.ptr, a.Z.ld);
  p.u_vec = operand_ok(a.U.ptr, a.U.ld);
  p.D0 = static_cast<uint16_t*>(a.D0), p.D1 = static_cast<uint16_t*>(a.D1);
  p.ldd = a.ldd;
  if (sum != kSumNone) {
    p.partial0 = a.partial;
    p.partial1 = gated ? a.partial + chunks * a.N : nullptr;
    p.db0 = a.db0, p.db1 = a.db1, p.db_f32 = a.db_dtype == IGC_F32;
  }
  const int64_t cols = sum == kSumCluster ? kNarrow : kWide;
  const dim3 grid(static_cast<unsigned>((a.N + cols - 1) / cols), static_cast<unsigned>(chunks));
  if (p.bf16)
    return gated ? launch_dact_sum<true, true>(p, sum, grid, stream)
                 : launch_dact_sum<false, true>(p, sum, grid, stream);
  return gated ? launch_dact_sum<true, false>(p, sum, grid, stream)
               : launch_dact_sum<false, false>(p, sum, grid, stream);
}

int ffn_dact_sums(const DactArgs& a, bool gated, bool late_wait, cudaStream_t stream) {
  if (a.M <= kClusterMaxRows) return IGC_OK;  // ffn_dact wrote the sums itself
  const int64_t chunks = dact_chunks(a.M, a.N);
  return launch_pdl(sum_chunks_kernel,
                    dim3(static_cast<unsigned>((a.N + 31) / 32), gated ? 2 : 1), dim3(256), 0,
                    stream, static_cast<const float*>(a.partial),
                    static_cast<const float*>(a.partial + (gated ? chunks * a.N : 0)),
                    static_cast<int>(chunks), static_cast<int>(a.N), a.db0, a.db1,
                    a.db_dtype == IGC_F32 ? 1 : 0, a.dtype == IGC_BF16 ? 1 : 0,
                    late_wait ? 1 : 0);
}

int ffn_bias_only(const PointwiseArgs& a, bool gated, cudaStream_t stream) {
  BiasOnlyParams p = {};
  p.M = static_cast<int>(a.M), p.N = static_cast<int>(a.N);
  p.bf16 = a.dtype == IGC_BF16, p.act = a.act, p.gated = gated;
  p.bias0 = a.bias[0], p.bias1 = a.bias[1], p.bias_f32 = a.bias_dtype == IGC_F32;
  p.R = a.R.ptr, p.ldr = a.R.ld;
  for (int i = 0; i < 3; ++i) {
    p.out[i] = const_cast<void*>(a.out[i].ptr);
    p.ld[i] = a.out[i].ld;
  }
  p.f32_0 = a.out[0].dtype == IGC_F32;
  const long long blocks = (static_cast<long long>(p.M) * p.N + 255) / 256;
  return launch_pdl(bias_only_kernel, dim3(static_cast<unsigned>(blocks < 4864 ? blocks : 4864)),
                    dim3(256), 0, stream, p);
}

}  // namespace igc
