// Host-side pieces shared by the feed-forward entry points (not part of the ABI).
#pragma once

#include "igc_ffn.h"
#include "igc_host.h"

namespace igc {

inline size_t elem_size(int dtype) { return dtype == IGC_F32 ? 4 : 2; }
inline bool is_operand_type(int dtype) { return dtype == IGC_F16 || dtype == IGC_BF16; }
// Sizes that tile coordinates (up to a tile past the end) hold in 32 bits.
inline bool fits32(int64_t v) { return v <= 0x7ffffe00; }
// Whether an output pointer is one of the others (a null output is none).
template <typename... P>
bool is_any(const void* out, P... others) {
  return out != nullptr && ((out == static_cast<const void*>(others)) || ...);
}
inline CUtensorMapDataType map_type(int dtype) {
  return dtype == IGC_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : (dtype == IGC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
}
inline bool rows_aligned(const void* p, int64_t ld, size_t esize, size_t to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && static_cast<uint64_t>(ld) * esize % to == 0;
}

// An M x N 16-bit operand that TMA reads.
inline bool operand_ok(const void* p, int64_t ld) { return rows_aligned(p, ld, 2, 16); }

// A matrix of the interface: pointer, row stride, element type.
struct Mat {
  const void* ptr = nullptr;
  int64_t ld = 0;
  int dtype = IGC_F32;
};

// Whether every matrix or vector starts on a boundary of its elements (null ones do): loads
// and stores of whole elements fault the GPU elsewhere.
template <typename... M>
bool elements_aligned(const M&... m) {
  return ((reinterpret_cast<uintptr_t>(m.ptr) % elem_size(m.dtype) == 0) && ...);
}

// How a product runs: on the kernel for small outputs (mt rows to a block, m_blocks of
// them, split CTAs to each) or on 256-row tiles of bn columns (tile_ctas CTAs); the
// estimated times of both.
struct ProductPlan {
  bool small = false;
  int mt = 16, m_blocks = 1, split = 1;
  int bn = 256, tile_ctas = 0;
  double small_us = 0.0, tiles_us = 0.0;
};

// Whether the dX of a backward pass goes to the tiles though the kernel for small outputs
// is estimated faster.  Tiles of both products that fit the SMs together run side by side;
// dX on the kernel for small outputs, which spreads over all SMs, leaves those of dW no room.
// Both gradients, device time with this rule and without, in us (linear; g: gated, with the
// activation's pass): 509 x 1001 x 777 10.6 and 16.2, 77 x 486 x 2638 9.1 and 12.5, 603 x
// 976 x 769 10.9 and 10.6, g 350 x 432 x 1407 12.8 and 17.2, g 1907 x 2489 x 467 31.9 and 39.7;
// of 21 sizes that it holds for it was the faster at 20.  dX by itself would be up to 8 us
// faster on the other kernel there (9.9 and 7.8 at the first size) and stays on the tiles, so
// that its bits do not depend on what else is asked for.
inline bool grad_x_beside_w(const ProductPlan& x, const ProductPlan& w, int sms) {
  const double beside = x.tiles_us > w.tiles_us ? x.tiles_us : w.tiles_us;
  return x.small && !w.small && x.tile_ctas + w.tile_ctas <= sms &&
         beside < x.small_us + w.tiles_us - 3.0;
}

// The products of a backward pass: dX = sum_s D[s] W[s] (ffn_gradx.cu) and dW[s] = D[s]^T X
// (ffn_gradw.cu), D[s] M x N, W[s] and dW[s] N x K, X and dX M x K, s < count.  The plans go
// by the sizes alone, as of operands with closely packed rows.
struct GradArgs {
  int64_t M = 0, N = 0, K = 0;
  int dtype = IGC_BF16;
  int count = 1;
  const Mat* D = nullptr;
  const Mat* W = nullptr;
  Mat X, dX;
  const Mat* dW = nullptr;
};
int ffn_plan_x(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan);
int ffn_plan_w(const DeviceInfo& dev, const GradArgs& a, ProductPlan* plan);
// late_wait: the kernel may run beside the one before it in the stream
// (ffn_dependency_wait, ffn_tc.cuh).
int ffn_grad_x(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream);
int ffn_grad_w(const DeviceInfo& dev, const GradArgs& a, const ProductPlan& plan, bool late_wait,
               cudaStream_t stream);

// Forward passes over the fp32 pre-activations of a contraction of length zero
// (the biases alone), and the backward passes over stored pre-activations (ffn_dact.cu).
struct PointwiseArgs {
  int64_t M = 0, N = 0;
  int dtype = IGC_BF16, act = IGC_ACT_NONE;
  const void* bias[2] = {};
  int bias_dtype = IGC_F32;
  Mat R, out[3];
};
int ffn_bias_only(const PointwiseArgs& a, bool gated, cudaStream_t stream);

// Backward through the activation: D0 = dO act'(Z) (linear), or D0 = dG and D1 = dU
// (gated, Z = G).  D0 / D1 may be null (not stored); db0 / db1 null: not summed.
struct DactArgs {
  int64_t M = 0, N = 0;
  int dtype = IGC_BF16, act = IGC_ACT_NONE;
  Mat dO, Z, U;
  void* D0 = nullptr;
  void* D1 = nullptr;
  int64_t ldd = 0;  // row stride of D0 and D1: a multiple of 8; both 16-byte aligned
  void* db0 = nullptr;
  void* db1 = nullptr;
  int db_dtype = IGC_F32;
  float* partial = nullptr;  // dact_chunks(M, N) x N floats per summed vector
};
int64_t dact_chunks(int64_t M, int64_t N);
int ffn_dact(const DactArgs& a, bool gated, cudaStream_t stream);
// The bias gradients from the partial sums that ffn_dact left (up to 512 rows it has
// written them already, and nothing is launched).
int ffn_dact_sums(const DactArgs& a, bool gated, bool late_wait, cudaStream_t stream);

}  // namespace igc

// For tests, through the binding: what a CTA of the kernel that igc_plan_ffn answers (the
// same arguments) takes of an SM: out[0] tensor-memory columns, out[1] bytes of dynamic
// shared memory.
extern "C" int igc_ffn_cta_resources(int op, int64_t M, int64_t N, int64_t K, int count, int sms,
                                     int32_t* out);
