// embedding_lookup: Y[i] = scale W[token[i]].
//
// Bound by memory: the rows that are asked for are read once (a second time mostly from L2), Y
// is written once (32768 rows of 131072 x 4096 bf16: 64 us, 366 MB at 5.7 TB/s).
#include "layers_host.h"

namespace igc {

namespace {

constexpr int kThreads = 256;

struct LookupParams {
  long long units;  // of eight columns, M * units_per_row
  FastDiv per_row;
  int D, vec, token64;
  long long V;
  const void* tokens;
  const void* W;
  void* Y;
  long long ldw, ldy;
  float scale;
};

// kW, kY: types of W and Y; kUnroll units to a thread.
template <int kW, int kY, int kUnroll>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long u0 = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll);
  const long long row0 = u0 / p.per_row.d;
  const uint32_t at0 = static_cast<uint32_t>(u0 - row0 * p.per_row.d) + threadIdx.x;
  const bool vec = p.vec != 0;
  long long row[kUnroll], token[kUnroll];
  int n[kUnroll];
  Raw8<kW> w[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint32_t at = at0 + i * kThreads, q = p.per_row.div(at);
    row[i] = row0 + q;
    n[i] = static_cast<int>(at - q * p.per_row.d) * 8;
    token[i] = -1;
    if (u0 + threadIdx.x + i * kThreads < p.units)
      token[i] = p.token64 ? static_cast<const long long*>(p.tokens)[row[i]]
                           : static_cast<const int*>(p.tokens)[row[i]];
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    w[i] = {};
    if (token[i] >= 0 && token[i] < p.V)
      w[i] = load8<kW>(row_at<kW>(p.W, token[i], p.ldw), n[i], p.D, vec);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (u0 + threadIdx.x + i * kThreads >= p.units) continue;
    float v[8];
    unpack8<kW>(w[i], v);
    const bool inside = token[i] >= 0 && token[i] < p.V;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = inside ? v[j] * p.scale : 0.0f;
    store8<kY>(row_at<kY>(p.Y, row[i], p.ldy), n[i], p.D, vec, v);
  }
}

// Two units to a thread where that still gives every SM a full set of threads (32768 rows of 4096,
// bf16: 64 us; one unit 88, four 65, eight 69).
template <int kW, int kY>
int launch(const DeviceInfo& dev, const LookupParams& p, cudaStream_t stream) {
  const int unroll = p.units >= static_cast<long long>(dev.sm_count) * 2048 * 2 ? 2 : 1;
  const long long blocks = (p.units + kThreads * unroll - 1) / (kThreads * unroll);
  if (blocks > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
  return launch_pdl(unroll == 2 ? lookup_kernel<kW, kY, 2> : lookup_kernel<kW, kY, 1>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

}  // namespace

}  // namespace igc

using namespace igc;

extern "C" int embedding_lookup(int64_t M, int64_t V, int64_t D, const void* tokens,
                                int token_bytes, const void* W, int64_t ldw, int w_dtype,
                                float scale, void* Y, int64_t ldy, int y_dtype,
                                igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || V < 0 || D < 0 || (token_bytes != 4 && token_bytes != 8) || !is_type(w_dtype) ||
      !is_type_or_f32(y_dtype, w_dtype))
    return IGC_ERR_INVALID_ARG;
  if (M == 0 || D == 0) return IGC_OK;
  if (!fits32(M) || !fits32(V) || !fits32(D)) return IGC_ERR_UNSUPPORTED;
  if (tokens == nullptr || Y == nullptr || ldy < D || (V > 0 && (W == nullptr || ldw < D)))
    return IGC_ERR_INVALID_ARG;
  if (is_any(Y, tokens, W)) return IGC_ERR_INVALID_ARG;
  if (!elements_aligned(Mat{W, ldw, w_dtype}, Mat{Y, ldy, y_dtype}) ||
      reinterpret_cast<uintptr_t>(tokens) % token_bytes != 0)
    return IGC_ERR_MISALIGNED;
  DeviceInfo dev;
  const int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  LookupParams p = {};
  p.per_row = FastDiv(static_cast<uint32_t>((D + 7) / 8));
  p.units = M * ((D + 7) / 8);
  p.D = static_cast<int>(D);
  p.vec = rows_vec(V, W, ldw, w_dtype) && rows_vec(M, Y, ldy, y_dtype);
  p.token64 = token_bytes == 8;
  p.V = V;
  p.tokens = tokens, p.W = W, p.Y = Y;
  p.ldw = ldw, p.ldy = ldy;
  p.scale = scale;
  if (w_dtype == IGC_F32) return launch<IGC_F32, IGC_F32>(dev, p, stream);
  if (w_dtype == IGC_F16)
    return y_dtype == IGC_F32 ? launch<IGC_F16, IGC_F32>(dev, p, stream)
                              : launch<IGC_F16, IGC_F16>(dev, p, stream);
  return y_dtype == IGC_F32 ? launch<IGC_BF16, IGC_F32>(dev, p, stream)
                            : launch<IGC_BF16, IGC_BF16>(dev, p, stream);
}
