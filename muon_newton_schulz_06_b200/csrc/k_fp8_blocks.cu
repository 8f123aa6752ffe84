// Block passes of the 8-bit format: quantise (with the activation), read back, and the
// activation's gradient from its checkpoint (dense, or quantised again).
//
//   quantise       q = code(f(x) 2^-e),  e from the block's largest magnitude
//   dequantise     x = value(q) 2^e
//   act backward   du = 2 sqrt(h) dy,    h = value(q) 2^e
//
// One CTA per 128 x 128 block, 512 threads; each thread holds 8 consecutive columns of
// 4 rows (rows t/16 + 32 i), so the whole block sits in registers between the maximum
// and the rounding and memory is touched once in each direction.  Half a warp covers the
// 128 columns of a row: row scales need shuffles only, square ones one exchange through
// shared memory.  Bound by memory traffic.
#include "fp8_blocks.cuh"

namespace muon {
namespace {

constexpr int kThreads = 512;
constexpr int kIter = 4;
constexpr int kStep = kThreads / 16;  // rows between a thread's rows
static_assert(kIter * kStep == kFp8Block, "a CTA holds one block");

// Maximum of m over the CTA.
__device__ __forceinline__ float cta_max(float m, float* warp_max) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, warp_max[w]);
  return m;
}

template <int OP, typename Params>
__global__ void __launch_bounds__(kThreads, 2) fp8_pass_kernel(const __grid_constant__ Params p) {
  __shared__ float warp_max[2][kThreads / 32];
  __shared__ __align__(16) float xch_all[kThreads / 16 * kF8Xch];
  __shared__ float slope[OP == kF8ActBackward ? kF8SlopeTable : 1];
  const int block = blockIdx.x;
  int lo = 0, hi = p.n - 1;  // last matrix whose block_begin <= block
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.m[mid].block_begin <= block) lo = mid;
    else hi = mid - 1;
  }
  const F8Pass& m = p.m[lo];
  const int local = block - m.block_begin;
  const int br = local / m.blocks_c, bc = local - br * m.blocks_c;
  const int rows = m.rows, cols = m.cols;
  const int col = bc * kFp8Block + (threadIdx.x & 15) * 8;
  const int row0 = br * kFp8Block + (threadIdx.x >> 4);

  float* xch = xch_all + (threadIdx.x >> 4) * kF8Xch;
  if constexpr (OP == kF8ActBackward) {
    if (p.relu2) {
      f8_slope_init(slope, m.saved.e5m2, threadIdx.x, kThreads);
      __syncthreads();
    }
  }
  f8_grid_wait();

  // entries outside the matrix are 0, and stay 0 through f and the gradient
  float v[kIter][8];
  if constexpr (OP == kF8Dequantize) {
    uint2 c[kIter];
    uint32_t sb[kIter];
    f8_load_code_rows<kIter>(m.saved, row0, kStep, rows, col, cols, c);
#pragma unroll
    for (int i = 0; i < kIter; ++i)
      sb[i] = row0 + i * kStep < rows ? *f8_scale_at(m.saved, row0 + i * kStep, bc) : 127u;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      if (m.saved.e5m2) f8_decode8<true>(c[i], f8_scale(sb[i]), v[i]);
      else f8_decode8<false>(c[i], f8_scale(sb[i]), v[i]);
    }
  } else {
    if (m.in.vec) f8_load_rows<kIter>(m.in, row0, kStep, rows, col, cols, v);
    else if (m.in.bf16) f8_load_rows_xch<kIter, true>(m.in, row0, kStep, rows, col, cols, v, xch);
    else f8_load_rows_xch<kIter, false>(m.in, row0, kStep, rows, col, cols, v, xch);
  }
  if constexpr (OP == kF8Quantize) {
    if (p.relu2) {
#pragma unroll
      for (int i = 0; i < kIter; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = f8_relu2(v[i][j]);
    }
  }
  if constexpr (OP == kF8ActBackward) {
    if (p.relu2) f8_times_slope<kIter>(m.saved, slope, row0, kStep, rows, col, cols, v);
  }

  if (OP == kF8Dequantize || (OP == kF8ActBackward && m.out.data != nullptr)) {
    if (m.out.vec) {
#pragma unroll
      for (int i = 0; i < kIter; ++i)
        if (row0 + i * kStep < rows && col < cols) f8_store8(m.out, row0 + i * kStep, col, cols, v[i]);
    } else {
      f8_store_rows_xch<kIter>(m.out, row0, kStep, rows, col, cols, v, xch);
    }
    return;
  }
  if constexpr (OP != kF8Dequantize) {
    if (m.out8.row_blocks) {
      f8_quantize_rows<kIter>(m.out8, row0, kStep, rows, col, cols, v);
      return;
    }
    float rmax[kIter], inv[kIter];
    f8_row_max<kIter>(v, rmax);
    float amax = cta_max(fmaxf(fmaxf(rmax[0], rmax[1]), fmaxf(rmax[2], rmax[3])), warp_max[0]);
    const bool inf = amax == kF8Inf;
    if (inf) {
      f8_row_max_finite<kIter>(v, rmax);
      amax = cta_max(fmaxf(fmaxf(rmax[0], rmax[1]), fmaxf(rmax[2], rmax[3])), warp_max[1]);
    }
    const int e = f8_exponent(amax, m.out8.e5m2);
    if (threadIdx.x == 0) *f8_scale_at(m.out8, br * kFp8Block, bc) = (uint8_t)(e + 127);
#pragma unroll
    for (int i = 0; i < kIter; ++i) inv[i] = f8_exp2(-e);
    f8_store_rows<kIter>(m.out8, row0, kStep, rows, col, cols, v, inv, inf);
  }
}

template <typename Params>
cudaError_t launch(int op, const Params& p, cudaStream_t st) {
  if (p.total_blocks == 0) return cudaSuccess;
  switch (op) {
    case kF8Quantize: return f8_launch(fp8_pass_kernel<kF8Quantize, Params>, p, p.total_blocks, kThreads, 0, 1, st);
    case kF8Dequantize: return f8_launch(fp8_pass_kernel<kF8Dequantize, Params>, p, p.total_blocks, kThreads, 0, 1, st);
    default: return f8_launch(fp8_pass_kernel<kF8ActBackward, Params>, p, p.total_blocks, kThreads, 0, 1, st);
  }
}

}  // namespace

cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kF8FewPasses>& p, cudaStream_t st) { return launch(op, p, st); }
cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kMaxF8Passes>& p, cudaStream_t st) { return launch(op, p, st); }

}  // namespace muon
