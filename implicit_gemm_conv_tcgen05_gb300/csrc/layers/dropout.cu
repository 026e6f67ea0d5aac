// dropout_add: Y = R + drop(X).
//
// Bound by memory: X and R are read once, Y written once, and the mask is made on the way
// (16384 x 8192 bf16 with a residual: 117 us, 805 MB at 6.9 TB/s; 20 instructions an element, 8 of
// them the generator's).
#include "layers_host.h"

namespace igc {

namespace {

constexpr int kThreads = 256;

struct DropoutParams {
  long long units;  // of eight columns, M * units_per_row
  FastDiv per_row;
  int N, vec;
  const void* X;
  const void* R;
  void* Y;
  long long ldx, ldr, ldy;
  Drop drop;
};

// kX, kY: types of X, and of R and Y; kUnroll units of eight columns to a thread, loaded before
// the first is used.
template <int kX, int kY, int kUnroll, bool kDrop>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long u0 = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll);
  const long long row0 = u0 / p.per_row.d;
  const uint32_t at0 = static_cast<uint32_t>(u0 - row0 * p.per_row.d) + threadIdx.x;
  const uint64_t offset = kDrop ? drop_offset(p.drop) : 0;
  const bool vec = p.vec != 0;
  Raw8<kX> x[kUnroll];
  Raw8<kY> r[kUnroll];
  long long row[kUnroll];
  int n[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint32_t at = at0 + i * kThreads, q = p.per_row.div(at);
    row[i] = row0 + q;
    n[i] = static_cast<int>(at - q * p.per_row.d) * 8;
    if (u0 + threadIdx.x + i * kThreads < p.units) {
      x[i] = load8<kX>(row_at<kX>(p.X, row[i], p.ldx), n[i], p.N, vec);
      if (p.R != nullptr) r[i] = load8<kY>(row_at<kY>(p.R, row[i], p.ldr), n[i], p.N, vec);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (u0 + threadIdx.x + i * kThreads >= p.units) continue;
    float v[8], f[8] = {};
    unpack8<kX>(x[i], v);
    if (p.R != nullptr) unpack8<kY>(r[i], f);
    if constexpr (kDrop) {
      drop8(p.drop, drop_bits(p.drop, offset, row[i], n[i]), v, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
    store8<kY>(row_at<kY>(p.Y, row[i], p.ldy), n[i], p.N, vec, v);
  }
}

template <int kX, int kY, int kUnroll>
int launch(const DropoutParams& p, bool drop, cudaStream_t stream) {
  const long long blocks = (p.units + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  if (blocks > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
  return launch_pdl(drop ? dropout_kernel<kX, kY, kUnroll, true>
                         : dropout_kernel<kX, kY, kUnroll, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

// Four units to a thread where that still gives every SM a full set of threads, else one (on the
// device 64 x 4096 bf16 with residual 1.5 us, with four 2.3).
template <int kX, int kY>
int launch(const DeviceInfo& dev, const DropoutParams& p, bool drop, cudaStream_t stream) {
  return p.units >= static_cast<long long>(dev.sm_count) * 2048 * 4
             ? launch<kX, kY, 4>(p, drop, stream)
             : launch<kX, kY, 1>(p, drop, stream);
}

}  // namespace

}  // namespace igc

using namespace igc;

extern "C" int dropout_add(int64_t M, int64_t N, const void* X, int64_t ldx, int x_dtype,
                           const void* R, int64_t ldr, double p, uint64_t seed, uint64_t offset,
                           const uint64_t* step, void* Y, int64_t ldy, int y_dtype,
                           igc_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (M < 0 || N < 0 || !is_type(x_dtype) || !is_type(y_dtype)) return IGC_ERR_INVALID_ARG;
  if (x_dtype != y_dtype && x_dtype != IGC_F32 && y_dtype != IGC_F32) return IGC_ERR_INVALID_ARG;
  DropoutParams a = {};
  bool active = false;
  if (!make_drop(p, seed, offset, step, &a.drop, &active)) return IGC_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return IGC_OK;
  if (!fits32(M) || !fits32(N)) return IGC_ERR_UNSUPPORTED;
  if (X == nullptr || Y == nullptr || ldx < N || ldy < N || (R != nullptr && ldr < N))
    return IGC_ERR_INVALID_ARG;
  if ((Y == X && (x_dtype != y_dtype || ldx != ldy)) || (Y == R && ldr != ldy) ||
      is_any(Y, step))
    return IGC_ERR_INVALID_ARG;
  if (!elements_aligned(Mat{X, ldx, x_dtype}, Mat{R, ldr, y_dtype}, Mat{Y, ldy, y_dtype}) ||
      reinterpret_cast<uintptr_t>(step) % 8 != 0)
    return IGC_ERR_MISALIGNED;
  DeviceInfo dev;
  const int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;
  a.per_row = FastDiv(static_cast<uint32_t>((N + 7) / 8));
  a.units = M * ((N + 7) / 8);
  a.N = static_cast<int>(N);
  a.vec = rows_vec(M, X, ldx, x_dtype) && rows_vec(M, R, ldr, y_dtype) &&
          rows_vec(M, Y, ldy, y_dtype);
  a.X = X, a.R = R, a.Y = Y;
  a.ldx = ldx, a.ldr = ldr, a.ldy = ldy;
  switch (x_dtype * 3 + y_dtype) {
    case IGC_F32 * 3 + IGC_F32: return launch<IGC_F32, IGC_F32>(dev, a, active, stream);
    case IGC_F32 * 3 + IGC_F16: return launch<IGC_F32, IGC_F16>(dev, a, active, stream);
    case IGC_F32 * 3 + IGC_BF16: return launch<IGC_F32, IGC_BF16>(dev, a, active, stream);
    case IGC_F16 * 3 + IGC_F32: return launch<IGC_F16, IGC_F32>(dev, a, active, stream);
    case IGC_F16 * 3 + IGC_F16: return launch<IGC_F16, IGC_F16>(dev, a, active, stream);
    case IGC_BF16 * 3 + IGC_F32: return launch<IGC_BF16, IGC_F32>(dev, a, active, stream);
    default: return launch<IGC_BF16, IGC_BF16>(dev, a, active, stream);
  }
}
