// grad_norm_clip: the global 2-norm of many tensors and their clipping.
//
// Bound by memory: every gradient is read for the norm and, scaled, read again and written
// (1.2e9 bf16: 7.2 GB in 1.08 ms, 6.65 TB/s; 2 M elements in 48 tensors 12 us).  Two
// kernels.  The first deals chunks of all tensors over a fixed number of blocks in turn; a
// thread adds squares in fp32 over a chunk and chunks in fp64, a block writes one partial
// sum.  In the second every block adds the partial sums itself, in the same order (a few
// hundred doubles from L2, instead of a third launch between the two), and scales its
// chunks.  It walks them backwards: the chunks that the first kernel read last are still in
// L2.  No atomics, so the norm is the same every time.
//
// Dealt in turn, the blocks read neighbouring chunks at any time; runs of neighbouring
// chunks for each block were 3 % slower on 2.4 GB, streaming cache hints on the second
// kernel's loads and stores 4 %.
//
// The list of tensors travels in the kernel's parameters (up to 32764 bytes): nothing is
// copied to the device, and the host arrays are free once the call returns.
#include <algorithm>

#include "ffn_act.cuh"
#include "ffn_host.h"
#include "sm100_ptx.cuh"

namespace igc {

namespace {

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 2;        // (2.4 GB: 1.09 ms; three 1.10, four 1.14)
constexpr int kMaxBlocks = 512;       // partial sums of one launch
constexpr int kTable = 1024;          // tensors of one launch
constexpr int kSmallTable = 64;
constexpr long long kMinChunk = 2048, kMaxChunk = 131072, kChunkStep = 1024;  // elements

template <int NT>
struct Table {
  const void* g[NT];
  void* out[NT];
  long long n[NT];
  int first[NT + 1];  // first chunk of each tensor; first[count] = all chunks
  unsigned char dtype[NT];
  int count, blocks;
  int chunk;
};
static_assert(sizeof(Table<kTable>) + 64 <= 32764, "kernel parameter limit");

// Tensor that holds chunk c: the last one whose first chunk is at most c.
template <int NT>
__device__ __forceinline__ int tensor_of(const Table<NT>& t, int c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Sum over the lanes of a warp, in every lane.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float load_elem(const void* p, long long i, int dtype) {
  return dtype == IGC_F32 ? static_cast<const float*>(p)[i] : load16(p, i, dtype == IGC_BF16);
}

__device__ __forceinline__ void store_elem(void* p, long long i, int dtype, float v) {
  if (dtype == IGC_F32)
    static_cast<float*>(p)[i] = v;
  else
    store16(p, i, v, dtype == IGC_BF16);
}

// Elements before the first 16-byte boundary at or after p.
__device__ __forceinline__ int head_of(const void* p, int esize, long long n) {
  const int bytes = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u);
  return static_cast<int>(min(static_cast<long long>(bytes / esize), n));
}

template <int kDtype>
__device__ __forceinline__ float squares16(uint4 q) {
  if constexpr (kDtype == IGC_F32) {
    const float a = __uint_as_float(q.x), b = __uint_as_float(q.y), c = __uint_as_float(q.z),
                d = __uint_as_float(q.w);
    return (a * a + b * b) + (c * c + d * d);
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(w[i], kDtype == IGC_BF16);
      s[i] = f.x * f.x + f.y * f.y;
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
  }
}

// This thread's sum of squares of n elements at p (16-byte vectors between the ends).
template <int kDtype>
__device__ __forceinline__ float chunk_squares(const void* p, long long n) {
  constexpr int kEs = kDtype == IGC_F32 ? 4 : 2, kPer = 16 / kEs;
  const int head = head_of(p, kEs, n);
  const long long vecs = (n - head) / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + head * kEs);
  float acc[4] = {};
  long long i = threadIdx.x;
  for (; i + 3 * kThreads < vecs; i += 4 * kThreads) {
    uint4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = v[i + j * kThreads];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += squares16<kDtype>(q[j]);
  }
  for (; i < vecs; i += kThreads) acc[0] += squares16<kDtype>(v[i]);
  const long long tail0 = head + vecs * kPer;
  if (static_cast<int>(threadIdx.x) < head) {
    const float x = load_elem(p, threadIdx.x, kDtype);
    acc[1] += x * x;
  }
  if (tail0 + static_cast<int>(threadIdx.x) < n) {  // fewer than kPer elements
    const float x = load_elem(p, tail0 + threadIdx.x, kDtype);
    acc[2] += x * x;
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

template <int kDtype>
__device__ __forceinline__ uint4 scale16(uint4 q, float c) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == IGC_F32) {
      w[i] = __float_as_uint(__uint_as_float(w[i]) * c);
    } else {
      const float2 f = unpack16(w[i], kDtype == IGC_BF16);
      w[i] = pack16(f.x * c, f.y * c, kDtype == IGC_BF16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kDtype>
__device__ __forceinline__ void chunk_scale(const void* p, void* o, long long n, float c) {
  constexpr int kEs = kDtype == IGC_F32 ? 4 : 2, kPer = 16 / kEs;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15u) != 0) {
    for (long long i = threadIdx.x; i < n; i += kThreads)
      store_elem(o, i, kDtype, load_elem(p, i, kDtype) * c);
    return;
  }
  const int head = head_of(p, kEs, n);
  const long long vecs = (n - head) / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + head * kEs);
  uint4* w = reinterpret_cast<uint4*>(static_cast<char*>(o) + head * kEs);
  long long i = threadIdx.x;
  for (; i + 3 * kThreads < vecs; i += 4 * kThreads) {
    uint4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = v[i + j * kThreads];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i + j * kThreads] = scale16<kDtype>(q[j], c);
  }
  for (; i < vecs; i += kThreads) w[i] = scale16<kDtype>(v[i], c);
  const long long tail0 = head + vecs * kPer;
  if (static_cast<int>(threadIdx.x) < head)
    store_elem(o, threadIdx.x, kDtype, load_elem(p, threadIdx.x, kDtype) * c);
  if (tail0 + static_cast<int>(threadIdx.x) < n)
    store_elem(o, tail0 + threadIdx.x, kDtype, load_elem(p, tail0 + threadIdx.x, kDtype) * c);
}

template <int NT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    norm_kernel(const __grid_constant__ Table<NT> t, double* partial) {
  __shared__ double red[kThreads];
  const int chunks = t.first[t.count];
  grid_dependency_wait();
  grid_dependents_launch();
  double sum = 0.0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const long long at = static_cast<long long>(c - t.first[i]) * t.chunk;
    const long long n = min(static_cast<long long>(t.chunk), t.n[i] - at);
    const int d = t.dtype[i];
    const char* p = static_cast<const char*>(t.g[i]) + at * (d == IGC_F32 ? 4 : 2);
    sum += d == IGC_F32 ? chunk_squares<IGC_F32>(p, n)
                        : (d == IGC_BF16 ? chunk_squares<IGC_BF16>(p, n)
                                         : chunk_squares<IGC_F16>(p, n));
  }
  // one warp adds the threads' sums: fp64 additions are slow (about two a clock on an SM)
  red[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += red[w * 32 + threadIdx.x];
  sum = warp_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    scale_kernel(const __grid_constant__ Table<NT> t, const double* partial, int n_partial,
                 float max_norm, float eps, float* norm_out) {
  __shared__ float shared_norm;
  const int chunks = t.first[t.count];
  grid_dependency_wait();
  grid_dependents_launch();
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int k = threadIdx.x; k < n_partial; k += 32) sum += partial[k];
    sum = warp_sum(sum);
    if (threadIdx.x == 0) shared_norm = static_cast<float>(sqrt(sum));
  }
  __syncthreads();
  const float norm = shared_norm;
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float ratio = max_norm / (norm + eps);
  const float coef = ratio > 1.0f ? 1.0f : ratio;  // (NaN stays NaN)
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int i = tensor_of(t, c);
    if (coef == 1.0f && t.out[i] == t.g[i]) continue;  // in place, times one
    const long long at = static_cast<long long>(c - t.first[i]) * t.chunk;
    const long long n = min(static_cast<long long>(t.chunk), t.n[i] - at);
    const int d = t.dtype[i];
    const long long off = at * (d == IGC_F32 ? 4 : 2);
    const char* p = static_cast<const char*>(t.g[i]) + off;
    char* o = static_cast<char*>(t.out[i]) + off;
    if (d == IGC_F32)
      chunk_scale<IGC_F32>(p, o, n, coef);
    else if (d == IGC_BF16)
      chunk_scale<IGC_BF16>(p, o, n, coef);
    else
      chunk_scale<IGC_F16>(p, o, n, coef);
  }
}

// The tensors [t0, t1) of a call as a table for at most `most` blocks; its number of
// chunks, or -1 if there are more than an int holds.
template <int NT>
long long fill(Table<NT>& t, int64_t t0, int64_t t1, const void* const* grads,
               const int64_t* sizes, const int32_t* dtypes, void* const* out, long long chunk,
               int most) {
  t.count = static_cast<int>(t1 - t0);
  t.chunk = static_cast<int>(chunk);
  long long at = 0;
  for (int64_t i = t0; i < t1; ++i) {
    const int k = static_cast<int>(i - t0);
    t.g[k] = grads[i];
    t.out[k] = out ? out[i] : nullptr;
    t.n[k] = sizes[i];
    t.dtype[k] = static_cast<unsigned char>(dtypes[i]);
    t.first[k] = static_cast<int>(at);
    at += (sizes[i] + chunk - 1) / chunk;
    if (at > 0x7ffffff0LL) return -1;
  }
  t.first[t.count] = static_cast<int>(at);
  t.blocks = static_cast<int>(at < most ? (at < 1 ? 1 : at) : most);
  return at;
}

// Both kernels over tables of NT tensors.
template <int NT>
int run(const DeviceInfo& dev, int64_t count, const void* const* grads, const int64_t* sizes,
        const int32_t* dtypes, void* const* out, float max_norm, float eps, float* norm,
        double* partial, cudaStream_t stream) {
  int most = dev.sm_count * kBlocksPerSm;
  if (most > kMaxBlocks) most = kMaxBlocks;
  long long total = 0;
  for (int64_t i = 0; i < count; ++i) total += sizes[i];
  // Chunk: one per block where that is at most 16384 elements (with room for the tensors'
  // ragged ends), else about eight per block, so that they are dealt evenly.
  const long long one = (total + total / 4) / most;
  long long chunk = std::max(std::min(one, 16384LL), one / 8);
  chunk = (chunk + kChunkStep - 1) / kChunkStep * kChunkStep;
  chunk = std::min(std::max(chunk, kMinChunk), kMaxChunk);

  Table<NT> t;
  const int64_t groups = count == 0 ? 1 : (count + NT - 1) / NT;
  int n_partial = 0;
  for (int64_t g = 0; g < groups; ++g) {
    const int64_t t1 = (g + 1) * NT < count ? (g + 1) * NT : count;
    const long long chunks = fill(t, g * NT, t1, grads, sizes, dtypes, out, chunk, most);
    if (chunks < 0) return IGC_ERR_UNSUPPORTED;
    if (chunks == 0) continue;
    const int rc = launch_pdl(norm_kernel<NT>, dim3(t.blocks), dim3(kThreads), 0, stream, t,
                              partial + n_partial);
    if (rc != IGC_OK) return rc;
    n_partial += t.blocks;
  }
  // the norm alone: one block of an empty table
  const int64_t scaled = out != nullptr ? count : 0;
  for (int64_t g = 0; g < (scaled == 0 ? 1 : groups); ++g) {
    const int64_t t1 = (g + 1) * NT < scaled ? (g + 1) * NT : scaled;
    // (with a single group the table is the one that the norm used)
    if (groups > 1 || out == nullptr)
      if (fill(t, g * NT, t1, grads, sizes, dtypes, out, chunk, most) == 0 && g > 0) continue;
    const int rc = launch_pdl(scale_kernel<NT>, dim3(t.blocks), dim3(kThreads), 0, stream, t,
                              static_cast<const double*>(partial), n_partial, max_norm, eps,
                              g == 0 ? norm : static_cast<float*>(nullptr));
    if (rc != IGC_OK) return rc;
  }
  return IGC_OK;
}

}  // namespace

}  // namespace igc

using namespace igc;

extern "C" {

size_t grad_norm_clip_workspace_size(int64_t count) {
  if (count < 0) return 0;
  const size_t groups =
      count == 0 ? 1 : (static_cast<size_t>(count) + kSmallTable - 1) / kSmallTable;
  // tables of kSmallTable tensors are used only for a single group
  const size_t launches = groups == 1 ? 1 : (static_cast<size_t>(count) + kTable - 1) / kTable;
  return launches * kMaxBlocks * sizeof(double);
}

int grad_norm_clip(int64_t count, const void* const* grads, const int64_t* sizes,
                   const int32_t* dtypes, void* const* out, float max_norm, float eps,
                   float* norm, void* workspace, size_t workspace_bytes, igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (count < 0 || norm == nullptr || !(max_norm >= 0.0f) || !(eps >= 0.0f))
    return IGC_ERR_INVALID_ARG;
  if (count > 0 && (grads == nullptr || sizes == nullptr || dtypes == nullptr))
    return IGC_ERR_INVALID_ARG;
  if (count > 0x3fffffff) return IGC_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(norm) % sizeof(float) != 0) return IGC_ERR_MISALIGNED;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0) return IGC_ERR_INVALID_ARG;
    if (dtypes[i] != IGC_F32 && !is_operand_type(dtypes[i])) return IGC_ERR_INVALID_ARG;
    if (sizes[i] == 0) continue;
    const uintptr_t es = elem_size(dtypes[i]);
    if (grads[i] == nullptr || (out != nullptr && out[i] == nullptr)) return IGC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(grads[i]) % es != 0 ||
        (out != nullptr && reinterpret_cast<uintptr_t>(out[i]) % es != 0))
      return IGC_ERR_MISALIGNED;
  }
  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  if (workspace == nullptr || workspace_bytes < grad_norm_clip_workspace_size(count) ||
      reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return IGC_ERR_WORKSPACE;
  double* partial = static_cast<double*>(workspace);
  return count <= kSmallTable ? run<kSmallTable>(dev, count, grads, sizes, dtypes, out, max_norm,
                                                 eps, norm, partial, stream)
                              : run<kTable>(dev, count, grads, sizes, dtypes, out, max_norm, eps,
                                            norm, partial, stream);
}

}  // extern "C"
