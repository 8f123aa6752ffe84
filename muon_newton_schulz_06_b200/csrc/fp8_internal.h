// Internal structures of the 8-bit operators, shared by their host driver (muon_fp8.cu)
// and kernels (k_fp8_blocks.cu, k_fp8_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace muon {

constexpr int kFp8Block = 128;

// The four bytes at `at` of a buffer [lo, hi), read as the aligned words that hold them, or one
// by one where such a word would reach out of the buffer (at its two ends, when it does not start
// or end at a multiple of four). word(a), byte(a): the reads.
template <typename Word, typename Byte>
__host__ __device__ __forceinline__ uint32_t f8_read4(uintptr_t at, uintptr_t lo, uintptr_t hi, Word word, Byte byte) {
  const uint32_t off = (uint32_t)(at & 3u);
  if (off == 0) return word(at);
  const uintptr_t first = at - off;
  if (first >= lo && first + 8 <= hi) return word(first) >> (8 * off) | word(first + 4) << (32 - 8 * off);
  return byte(at) | byte(at + 1) << 8 | byte(at + 2) << 16 | byte(at + 3) << 24;
}

// Launch of one of these kernels: `cluster` CTAs per cluster, and its start may overlap the
// end of the kernel before it on the stream (programmatic stream serialization).  Every
// kernel here lets the next one start as soon as all its CTAs run, and touches memory only
// after f8_grid_wait(), which returns when the kernel before has completed: chains of small
// calls hide their launch and set-up behind each other.
template <typename Params>
cudaError_t f8_launch(void (*kernel)(Params), const Params& p, int grid, int block, uint32_t smem, int cluster,
                      cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Raises a kernel's shared-memory limit, once per device (`ready`: one bit each).
inline cudaError_t f8_allow_smem(const void* kernel, uint32_t bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit != 0 && (ready.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A dense operand of a kernel (null data: absent).
struct F8Dense {
  void* data;
  int64_t ld;    // elements
  uint8_t bf16;  // else float32
  uint8_t vec;   // 8 consecutive entries starting at a multiple of 8 columns are 16-byte aligned
};

// An 8-bit operand (null codes: absent).  Scale byte of entry (i, j), counted in blocks
// of 128 columns kb = j / 128: row blocks: scales[kb * s_col + i], square blocks:
// scales[(i / 128) * s_row + kb].
struct F8Mat {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld;
  int32_t s_row, s_col;  // square: column blocks, unused; row: unused, rows
  uint8_t e5m2;
  uint8_t row_blocks;
};

// ------------------------------------------------------------------ block passes

enum F8Op : int { kF8Quantize = 0, kF8Dequantize = 1, kF8ActBackward = 2 };

// One matrix of a pass: out (dense or 8 bits) from in and / or saved.
struct F8Pass {
  F8Dense in;
  F8Mat saved;
  F8Dense out;
  F8Mat out8;
  int32_t rows, cols;
  int32_t blocks_c;     // 128-column blocks per row of blocks
  int32_t block_begin;  // first block of this matrix inside the launch
};
// A launch's parameters travel with it, so calls of a few matrices use a smaller struct (a
// launch copies all of it: 17 KB for 96 matrices).
constexpr int kMaxF8Passes = 96;
constexpr int kF8FewPasses = 4;
template <int N>
struct F8PassParamsN {
  F8Pass m[N];
  int n;
  int total_blocks;
  int relu2;
};
static_assert(sizeof(F8PassParamsN<kMaxF8Passes>) <= 32764,
              "parameters of the block passes must fit the kernel parameter space");

cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kF8FewPasses>& p, cudaStream_t st);
cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kMaxF8Passes>& p, cudaStream_t st);

// ------------------------------------------------------------------ products

// Scales of an operand as the product walks them: byte of row r (M or N index) and
// k-block kb at s[(by_row ? r : r / 128) * s_r + kb * s_k].
struct F8Scales {
  const uint8_t* s;
  int32_t s_r, s_k;
  int32_t by_row;
};

enum F8Epi : int { kF8EpiNone = 0, kF8EpiRelu2 = 1, kF8EpiRelu2Backward = 2 };

// How a result leaves the pair kernel.
enum F8Out : int { kF8OutBf16 = 0, kF8OutF32 = 1, kF8OutCodes = 2 };

struct F8Product {
  F8Scales sa, sb;
  F8Dense d, c;
  F8Mat d8, saved;
  int32_t m, n, k;
  uint8_t a_mn, b_mn;      // operand stored with M / N contiguous (contraction over its rows)
  uint8_t a_e5m2, b_e5m2;
  int32_t epi;
  int32_t out;             // F8Out
  int32_t out_align;       // largest of 32, 16 that divides the result's base and row pitch in bytes, else 0
  int32_t seg_kb;          // k-blocks that one accumulation may sum (pair kernel; >= all of them: no segments)
  int32_t tiles_m, tiles_n;
  int32_t tile_begin;      // first tile inside the launch
};
constexpr int kMaxF8Products = 16;
constexpr int kF8FewProducts = 3;
template <int N>
struct __align__(64) F8GemmParamsN {
  CUtensorMap map_a[N];
  CUtensorMap map_b[N];
  F8Product p[N];
  int n;
  int total_tiles;
  int stages;              // ring depth of k_fp8_gemm.cu: 6, or 3 for two CTAs per SM
  int backward;            // some product has the kF8EpiRelu2Backward epilogue
  int* status;
};
static_assert(sizeof(F8GemmParamsN<kMaxF8Products>) <= 32764,
              "parameters of the 8-bit products must fit the kernel parameter space");

// A float32 result sums this many k-blocks at most in tensor memory (4096 of the contraction; a
// multiple of the 4 of a scale group).
constexpr int32_t kF8SegmentBlocks = 32;
constexpr int32_t kF8TileAccs = 3;  // accumulators of a 128 x 128 tile with an SM of its own

// 256 x 256 tiles by pairs of CTAs, persistent: `clusters` pairs.
constexpr int kF8PairTile = 256;
constexpr int kF8PairProducts = 8;
struct __align__(64) F8PairParams : F8GemmParamsN<kF8PairProducts> {
  CUtensorMap map_saved[kF8PairProducts];  // checkpoints, boxes of 32 rows x 128 codes
};
cudaError_t launch_fp8_gemm_pair(const F8PairParams& p, int clusters, cudaStream_t st);

// Diagnostic: the products' bounded wait on a barrier that nothing completes.
cudaError_t launch_fp8_wait_selftest(int* status, long long limit_clocks, cudaStream_t st);

// 128 x 128 tiles, one CTA each; `split` CTAs (a cluster of 1, 2 or 4) share a tile's
// contraction and join their sums through distributed shared memory.  segments: shares longer
// than the accumulators' kF8TileAccs * kF8SegmentBlocks are summed in segments (six stages only).
cudaError_t launch_fp8_gemm_tile(const F8GemmParamsN<kF8FewProducts>& p, int split, bool segments, cudaStream_t st);
cudaError_t launch_fp8_gemm_tile(const F8GemmParamsN<kMaxF8Products>& p, int split, bool segments, cudaStream_t st);

}  // namespace muon
