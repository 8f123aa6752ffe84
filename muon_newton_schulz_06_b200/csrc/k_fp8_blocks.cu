// Block passes of the 8-bit format: quantise (with the activation), read back, and the
// activation's gradient from its checkpoint (dense, or quantised again).
//
//   quantise       q = code(f(x) 2^-e),  e from the block's largest magnitude
//   dequantise     x = value(q) 2^e
//   act backward   du = 2 sqrt(h) dy,    h = value(q) 2^e
//
// One CTA per 128 x 128 block, which sits in registers between the maximum and the rounding,
// so memory is touched once in each direction.  Two forms:
//
// Wide (rows that 32-byte accesses can address, a multiple of 16 columns): a thread holds 16
// consecutive columns (32 bytes of bf16, one sector; 16 codes) of rows t/8 + 32 i, packed as
// loaded until they are needed.  Bound by memory traffic, after the instructions per entry had
// been brought from 15 to about 5.
//
// General (any pitch, alignment and width): 512 threads, a thread holds 8 consecutive columns of
// rows t/16 + 32 i; half a block with 256 threads where no maximum spans the block.
//
// In both, a group of lanes covers the 128 columns of a row: row scales need shuffles only,
// square ones one exchange through shared memory.
#include "fp8_blocks.cuh"

namespace muon {
namespace {

constexpr int kIter = 4;

// Maximum of m over the CTA.
template <int kThreads>
__device__ __forceinline__ float cta_max(float m, float* warp_max) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, warp_max[w]);
  return m;
}

// SUB: CTAs per block, 1 or 2.
template <int OP, int SUB, typename Params>
__global__ void __launch_bounds__(512 / SUB, 2 * SUB) fp8_pass_kernel(const __grid_constant__ Params p) {
  constexpr int kThreads = 512 / SUB;
  constexpr int kStep = kThreads / 16;  // rows between a thread's rows
  __shared__ float warp_max[2][kThreads / 32];
  __shared__ __align__(16) float xch_all[kThreads / 16 * kF8Xch];
  __shared__ float slope[OP == kF8ActBackward ? kF8SlopeTable : 1];
  const int block = blockIdx.x / SUB;
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
  const int row0 = br * kFp8Block + (int)(blockIdx.x % SUB) * (kFp8Block / SUB) + (threadIdx.x >> 4);

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
    if (OP == kF8Quantize && !m.in.vec && !m.in.bf16) f8_load_rows_xch<kIter>(m.in, row0, kStep, rows, col, cols, v, xch);
    else f8_load_rows<kIter>(m.in, row0, kStep, rows, col, cols, v);
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
    float amax = cta_max<kThreads>(fmaxf(fmaxf(rmax[0], rmax[1]), fmaxf(rmax[2], rmax[3])), warp_max[0]);
    const bool inf = amax == kF8Inf;
    if (inf) {
      f8_row_max_finite<kIter>(v, rmax);
      amax = cta_max<kThreads>(fmaxf(fmaxf(rmax[0], rmax[1]), fmaxf(rmax[2], rmax[3])), warp_max[1]);
    }
    const int e = f8_exponent(amax, m.out8.e5m2);
    if (threadIdx.x == 0) *f8_scale_at(m.out8, br * kFp8Block, bc) = (uint8_t)(e + 127);
#pragma unroll
    for (int i = 0; i < kIter; ++i) inv[i] = f8_exp2(-e);
    f8_store_rows<kIter>(m.out8, row0, kStep, rows, col, cols, v, inv, inf);
  }
}

template <int OP, typename Params>
cudaError_t launch_op(const Params& p, bool halves, cudaStream_t st) {
  if (halves) return f8_launch<Params>(fp8_pass_kernel<OP, 2, Params>, p, 2 * p.total_blocks, 256, 0, 1, st);
  return f8_launch<Params>(fp8_pass_kernel<OP, 1, Params>, p, p.total_blocks, 512, 0, 1, st);
}

template <typename Params>
cudaError_t launch(int op, const Params& p, cudaStream_t st) {
  if (p.total_blocks == 0) return cudaSuccess;
  bool halves = p.total_blocks <= INT32_MAX / 2;
  for (int i = 0; i < p.n; ++i) halves = halves && (p.m[i].out8.codes == nullptr || p.m[i].out8.row_blocks);
  switch (op) {
    case kF8Quantize: return launch_op<kF8Quantize>(p, halves, st);
    case kF8Dequantize: return f8_launch<Params>(fp8_pass_kernel<kF8Dequantize, 2, Params>, p, 2 * p.total_blocks, 256, 0, 1, st);
    default: return launch_op<kF8ActBackward>(p, halves, st);
  }
}

// ---------------------------------------------------------------------- wide form

__device__ __forceinline__ void ld_global_32b(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Packed entry j of 16: a word holds two bf16 or one float32.
template <bool BF16>
__device__ __forceinline__ float unpack(const uint32_t* w, int j) {
  if constexpr (BF16) return __uint_as_float((j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  else return __uint_as_float(w[j]);
}
template <bool BF16>
__device__ __forceinline__ void store16(uint8_t* p, const float* v) {
  uint32_t w[BF16 ? 8 : 16];
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    st_global_32b(p, w);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[j]);
    st_global_32b(p, w);
    st_global_32b(p + 32, w + 8);
  }
}

// Codes of 16 values times inv.
template <bool E5M2>
__device__ __forceinline__ uint4 encode16(const float* v, float inv, bool inf) {
  uint2 a = f8_encode8<E5M2>(v, inv), b = f8_encode8<E5M2>(v + 8, inv);
  if (inf) {
    a = f8_encode_inf8<E5M2>(v, a);
    b = f8_encode_inf8<E5M2>(v + 8, b);
  }
  return make_uint4(a.x, a.y, b.x, b.y);
}

constexpr int kF8ActBackward8 = 3;

// OP (kF8ActBackward8: the gradient in 8 bits); BF16: type of the dense side; FMT: format of the 8-bit result (of the source for
// dequantise), 1 = e5m2.  bf16: 256 threads, 4 rows each; float32: 512 threads, 2 rows.
template <int OP, bool BF16, bool FMT>
__global__ void __launch_bounds__(BF16 ? 256 : 512, BF16 ? (OP == kF8ActBackward8 ? 2 : OP == kF8ActBackward ? 3 : 4) : 2)
    fp8_wide_kernel(const __grid_constant__ F8PassParamsN<kF8FewPasses> p) {
  constexpr int kThr = BF16 ? 256 : 512;
  constexpr int kRows = kThr / 8;           // rows between a thread's rows
  constexpr int kN = kFp8Block / kRows;     // rows per thread
  constexpr int kW = BF16 ? 8 : 16;         // words per 16 entries
  __shared__ float warp_max[2][kThr / 32];
  constexpr bool kGrad = OP == kF8ActBackward || OP == kF8ActBackward8;
  __shared__ float slope[kGrad ? kF8SlopeTable : 1];
  int mi = 0;
  while (mi + 1 < p.n && p.m[mi + 1].block_begin <= (int)blockIdx.x) ++mi;
  const F8Pass& m = p.m[mi];
  const int local = (int)blockIdx.x - m.block_begin;
  const int br = local / m.blocks_c, bc = local - br * m.blocks_c;
  const int rows = m.rows, cols = m.cols;
  const int col = bc * kFp8Block + (threadIdx.x & 7) * 16;
  const int row0 = br * kFp8Block + (threadIdx.x >> 3);
  const bool live_c = col < cols;
  if constexpr (kGrad) {
    if (p.relu2) {
      f8_slope_init(slope, m.saved.e5m2, threadIdx.x, kThr);
      __syncthreads();
    }
  }
  f8_grid_wait();

  // every load is issued before the first use; entries outside the matrix are 0
  uint32_t x[kN][kW];
  uint4 c[kN];
  uint32_t sb[kN];
  if constexpr (OP != kF8Dequantize) {
    const uint8_t* q = reinterpret_cast<const uint8_t*>(m.in.data) + ((int64_t)row0 * m.in.ld + col) * (BF16 ? 2 : 4);
    const int64_t step = (int64_t)kRows * m.in.ld * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int j = 0; j < kW; ++j) x[i][j] = 0u;
      if (live_c && row0 + i * kRows < rows) {
        ld_global_32b(q + i * step, x[i]);
        if constexpr (!BF16) ld_global_32b(q + i * step + 32, x[i] + 8);
      }
    }
  }
  if constexpr (OP != kF8Quantize) {
    const uint8_t* q = m.saved.codes + (int64_t)row0 * m.saved.ld + col;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const bool live = live_c && row0 + i * kRows < rows;
      c[i] = live ? *reinterpret_cast<const uint4*>(q + (int64_t)(i * kRows) * m.saved.ld) : make_uint4(0u, 0u, 0u, 0u);
      sb[i] = live ? *f8_scale_at(m.saved, row0 + i * kRows, bc) : 127u;
    }
  }

  if constexpr (OP == kF8Dequantize) {
    uint8_t* q = reinterpret_cast<uint8_t*>(m.out.data) + ((int64_t)row0 * m.out.ld + col) * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float v[16];
      const float scale = f8_scale(sb[i]);
      f8_decode8<FMT>(make_uint2(c[i].x, c[i].y), scale, v);
      f8_decode8<FMT>(make_uint2(c[i].z, c[i].w), scale, v + 8);
      if (live_c && row0 + i * kRows < rows) store16<BF16>(q + (int64_t)(i * kRows) * m.out.ld * (BF16 ? 2 : 4), v);
    }
    return;
  }

  // entry j of row i after f, or times f'
  const bool relu2 = p.relu2;
  auto values = [&](int i, float* v) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = unpack<BF16>(x[i], j);
    if constexpr (OP == kF8Quantize) {
      if (relu2) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = f8_relu2(v[j]);
      }
    }
    if constexpr (kGrad) {
      if (relu2) {
        const int e = (int)sb[i] - 127, parity = e & 1;
        const float scale = sb[i] == 255u ? __uint_as_float(0x7fc00000u) : f8_exp2((e - parity) / 2);
        const float* t = slope + 256 * parity;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(__fmul_rn(t[(w[j >> 2] >> (8 * (j & 3))) & 255u], scale), v[j]);
      }
    }
  };
  if constexpr (OP == kF8ActBackward) {
    uint8_t* q = reinterpret_cast<uint8_t*>(m.out.data) + ((int64_t)row0 * m.out.ld + col) * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float v[16];
      values(i, v);
      if (live_c && row0 + i * kRows < rows) store16<BF16>(q + (int64_t)(i * kRows) * m.out.ld * (BF16 ? 2 : 4), v);
    }
  }
  if constexpr (OP == kF8Quantize || OP == kF8ActBackward8) {
    // the gradient's entries are formed once; those to quantise stay packed, and are unpacked
    // again for the codes
    float g[OP == kF8ActBackward8 ? kN : 1][16];
    if constexpr (OP == kF8ActBackward8) {
#pragma unroll
      for (int i = 0; i < kN; ++i) values(i, g[i]);
    }
    // largest magnitude of row i's 16 entries (NaN is passed over, infinity is not); f is
    // monotonic, so relu^2 takes that of the largest entry
    auto row_max = [&](int i, bool finite) {
      float a = 0.f;
      if constexpr (OP == kF8ActBackward8) {
#pragma unroll
        for (int j = 0; j < 16; ++j) a = fmaxf(a, finite ? f8_finite_abs(g[i][j]) : fabsf(g[i][j]));
      } else if (finite) {
        float v[16];
        values(i, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) a = fmaxf(a, f8_finite_abs(v[j]));
      } else {
        if constexpr (BF16) {
          __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            const __nv_bfloat162 u = *reinterpret_cast<const __nv_bfloat162*>(&x[i][j]);
            m2 = __hmax2(m2, relu2 ? u : __habs2(u));
          }
          a = fmaxf(__low2float(m2), __high2float(m2));
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) a = fmaxf(a, relu2 ? unpack<BF16>(x[i], j) : fabsf(unpack<BF16>(x[i], j)));
        }
        if (relu2) a = __fmul_rn(a, a);
      }
      return a;
    };
    auto lanes_max = [&](float a) {  // over the 8 lanes of a row
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      return a;
    };
    auto block_max = [&](float a, float* slots) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = a;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThr / 32; ++w) a = fmaxf(a, slots[w]);
      return a;
    };
    float rmax[kN];
    bool inf = false;
    if (m.out8.row_blocks) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        rmax[i] = lanes_max(row_max(i, false));
        inf |= rmax[i] == kF8Inf;
      }
      inf = __any_sync(0xffffffffu, inf);
      if (inf) {
#pragma unroll
        for (int i = 0; i < kN; ++i) rmax[i] = lanes_max(row_max(i, true));
      }
    } else {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) a = fmaxf(a, row_max(i, false));
      a = block_max(a, warp_max[0]);
      inf = a == kF8Inf;
      if (inf) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) a = fmaxf(a, row_max(i, true));
        a = block_max(a, warp_max[1]);
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) rmax[i] = a;
    }
    uint8_t* q = m.out8.codes + (int64_t)row0 * m.out8.ld + col;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int row = row0 + i * kRows, e = f8_exponent(rmax[i], FMT);
      if (row < rows && (m.out8.row_blocks ? (threadIdx.x & 7) == 0 : threadIdx.x == 0 && i == 0))
        *f8_scale_at(m.out8, row, bc) = (uint8_t)(e + 127);
      uint4 code;
      if constexpr (OP == kF8ActBackward8) {
        code = encode16<FMT>(g[i], f8_exp2(-e), inf);
      } else {
        float v[16];
        values(i, v);
        code = encode16<FMT>(v, f8_exp2(-e), inf);
      }
      if (live_c && row < rows) *reinterpret_cast<uint4*>(q + (int64_t)(i * kRows) * m.out8.ld) = code;
    }
  }
}

// Dense side and matrices that the wide form can take, all of one type and format.
bool wide_dense(const F8Dense& x) {
  const int64_t esz = x.bf16 ? 2 : 4;
  return (reinterpret_cast<uintptr_t>(x.data) & 31u) == 0 && (x.ld * esz) % 32 == 0;
}
bool wide(int op, const F8PassParamsN<kF8FewPasses>& p, bool* bf16, bool* e5m2) {
  for (int i = 0; i < p.n; ++i) {
    const F8Pass& m = p.m[i];
    if (m.cols % 16) return false;
    const F8Dense& x = op == kF8Dequantize ? m.out : m.in;
    if (!wide_dense(x)) return false;
    if (op == kF8ActBackward && (m.out.data == nullptr || !wide_dense(m.out) || m.out.bf16 != m.in.bf16)) return false;
    if (op == kF8ActBackward8 && m.out8.codes == nullptr) return false;
    const bool f = op == kF8Dequantize ? m.saved.e5m2 : m.out8.codes != nullptr && m.out8.e5m2;
    if (i == 0) {
      *bf16 = x.bf16;
      *e5m2 = f;
    } else if (x.bf16 != *bf16 || f != *e5m2) {
      return false;
    }
  }
  return true;
}

template <int OP, bool FMT>
cudaError_t launch_wide(const F8PassParamsN<kF8FewPasses>& p, bool bf16, cudaStream_t st) {
  using P = F8PassParamsN<kF8FewPasses>;
  return bf16 ? f8_launch<P>(fp8_wide_kernel<OP, true, FMT>, p, p.total_blocks, 256, 0, 1, st)
              : f8_launch<P>(fp8_wide_kernel<OP, false, FMT>, p, p.total_blocks, 512, 0, 1, st);
}

}  // namespace

cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kF8FewPasses>& p, cudaStream_t st) {
  bool bf16 = false, e5m2 = false;
  const int wide_op = op == kF8ActBackward && p.m[0].out8.codes != nullptr ? (int)kF8ActBackward8 : op;
  if (p.total_blocks > 0 && wide(wide_op, p, &bf16, &e5m2)) {
    switch (wide_op) {
      case kF8Quantize:
        return e5m2 ? launch_wide<kF8Quantize, true>(p, bf16, st) : launch_wide<kF8Quantize, false>(p, bf16, st);
      case kF8Dequantize:
        return e5m2 ? launch_wide<kF8Dequantize, true>(p, bf16, st) : launch_wide<kF8Dequantize, false>(p, bf16, st);
      case kF8ActBackward:  // no 8-bit result
        return launch_wide<kF8ActBackward, false>(p, bf16, st);
      default:
        return e5m2 ? launch_wide<kF8ActBackward8, true>(p, bf16, st)
                    : launch_wide<kF8ActBackward8, false>(p, bf16, st);
    }
  }
  return launch(op, p, st);
}
cudaError_t launch_fp8_pass(int op, const F8PassParamsN<kMaxF8Passes>& p, cudaStream_t st) { return launch(op, p, st); }

}  // namespace muon
