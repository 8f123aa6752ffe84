// Block passes of the 8-bit format: quantise (with the activation), read back, and the
// activation's gradient from its checkpoint (dense, or quantised again).
//
//   quantise       q = code(f(x) 2^-e),  e from the block's largest magnitude
//   dequantise     x = value(q) 2^e
//   act backward   du = 2 sqrt(h) dy,    h = value(q) 2^e
//
// One CTA per 128 x 128 block, 256 threads; each thread holds 8 consecutive columns of
// 8 rows (rows t/16 + 16 i), so the whole block sits in registers between the maximum
// and the rounding and memory is touched once in each direction.  Half a warp covers the
// 128 columns of a row: row scales need shuffles only, square ones one exchange through
// shared memory.  Bound by memory traffic.
#include "fp8_blocks.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kIter = 8;

// Maximum, scale and codes of one block, 8 rows x 8 columns per thread.  Entries outside
// the matrix are 0 (f(0) = 0, and so is the gradient there).
__device__ __forceinline__ void fp8_quantize_block(const F8Pass& m, int br, int bc, int row0, int col,
                                                   const float (&v)[kIter][8], float* warp_max) {
  const int rows = m.rows, cols = m.cols;
  const bool live_c = col < cols;
  float rmax[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    rmax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) rmax[i] = fmaxf(rmax[i], f8_finite_abs(v[i][j]));
  }
  const bool e5m2 = m.out8.e5m2;
  if (m.out8.row_blocks) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) rmax[i] = fmaxf(rmax[i], __shfl_xor_sync(0xffffffffu, rmax[i], d));
      const int row = row0 + 16 * i;
      const int e = f8_exponent(rmax[i], e5m2);
      if (row < rows) {
        if ((threadIdx.x & 15) == 0) *f8_scale_at(m.out8, row, bc) = (uint8_t)(e + 127);
        if (live_c) f8_store_codes8(m.out8, row, col, cols, f8_encode8(v[i], f8_exp2(-e), e5m2));
      }
    }
    return;
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; ++i) amax = fmaxf(amax, rmax[i]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  const int e = f8_exponent(amax, e5m2);
  if (threadIdx.x == 0) *f8_scale_at(m.out8, br * kFp8Block, bc) = (uint8_t)(e + 127);
  const float inv = f8_exp2(-e);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = row0 + 16 * i;
    if (row < rows && live_c) f8_store_codes8(m.out8, row, col, cols, f8_encode8(v[i], inv, e5m2));
  }
}

template <int OP>
__global__ void __launch_bounds__(kThreads) fp8_pass_kernel(const __grid_constant__ F8PassParams p) {
  __shared__ float warp_max[kThreads / 32];
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
  const bool live_c = col < cols;

  float v[kIter][8];
  if constexpr (OP != kF8Dequantize) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = row0 + 16 * i;
      if (row < rows && live_c) {
        f8_load8(m.in, row, col, cols, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      }
    }
  }
  if constexpr (OP == kF8Quantize) {
    if (p.relu2) {
#pragma unroll
      for (int i = 0; i < kIter; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = f8_relu2(v[i][j]);
    }
  }
  if constexpr (OP == kF8Dequantize || OP == kF8ActBackward) {
    if (OP == kF8Dequantize || p.relu2) {
      uint2 c[kIter];
      uint32_t sb[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int row = row0 + 16 * i;
        const bool live = row < rows && live_c;
        c[i] = live ? f8_load_codes8(m.saved, row, col, cols) : make_uint2(0u, 0u);
        sb[i] = live ? *f8_scale_at(m.saved, row, bc) : 127u;
      }
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        float h[8];
        f8_decode8(c[i], f8_scale(sb[i]), m.saved.e5m2, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (OP == kF8Dequantize) v[i][j] = h[j];
          else v[i][j] = __fmul_rn(f8_relu2_slope(h[j]), v[i][j]);
        }
      }
    }
  }

  if (OP == kF8Dequantize || (OP == kF8ActBackward && m.out.data != nullptr)) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = row0 + 16 * i;
      if (row < rows && live_c) f8_store8(m.out, row, col, cols, v[i]);
    }
    return;
  }

  if constexpr (OP != kF8Dequantize) fp8_quantize_block(p.m[lo], br, bc, row0, col, v, warp_max);
}

}  // namespace

cudaError_t launch_fp8_pass(int op, const F8PassParams& p, cudaStream_t st) {
  if (p.total_blocks == 0) return cudaSuccess;
  switch (op) {
    case kF8Quantize: fp8_pass_kernel<kF8Quantize><<<p.total_blocks, kThreads, 0, st>>>(p); break;
    case kF8Dequantize: fp8_pass_kernel<kF8Dequantize><<<p.total_blocks, kThreads, 0, st>>>(p); break;
    default: fp8_pass_kernel<kF8ActBackward><<<p.total_blocks, kThreads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace muon
