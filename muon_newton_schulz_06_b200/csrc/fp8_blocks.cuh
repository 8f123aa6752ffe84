// Device arithmetic of the 8-bit block-scaled format, shared by the block passes
// (k_fp8_blocks.cu) and the products' epilogues (k_fp8_gemm.cu): scales, rounding into
// and out of the codes, dense loads and stores of 8 consecutive entries.
//
// A block with finite largest magnitude amax = m 2^p (m in [0.5, 1)) takes the scale 2^e
// with e the least integer such that amax <= top * 2^e.  Both formats have
// top = 0.875 * 2^P (P = 9 for e4m3, 16 for e5m2), so e = p - P, plus one if m > 0.875.
// A power of two makes the scaling exact: each entry is rounded once, into the code.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_internal.h"

namespace muon {
namespace {

// See f8_launch: the next kernel may be set up from here on; and the wait for the one before.
__device__ __forceinline__ void f8_grid_wait() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// 2^e as a float for e in [-127, 127].
__device__ __forceinline__ float f8_exp2(int e) {
  return e == -127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// Exponent of a block from its largest finite magnitude.
__device__ __forceinline__ int f8_exponent(float amax, bool e5m2) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return 0;
  const int e = (int)(b >> 23) - 126 - (e5m2 ? 16 : 9) + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -127);  // a subnormal amax lands here too; e <= 120 always
}

// Scale of a stored byte (255 is NaN).
__device__ __forceinline__ float f8_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : f8_exp2((int)byte - 127);
}

constexpr float kF8Inf = __builtin_huge_valf();

// |v| where finite, else 0.
__device__ __forceinline__ float f8_finite_abs(float v) {
  const float a = fabsf(v);
  return a < kF8Inf ? a : 0.f;
}

// f(u) = max(u, 0)^2; NaN stays NaN.
__device__ __forceinline__ float f8_relu2(float u) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(u));
  return __fmul_rn(r, r);
}
// f'(u) = 2 relu(u) = 2 sqrt(h) from h = f(u) = q 2^e: with p the parity of e,
// 2 sqrt(q 2^p) 2^((e - p) / 2), whose power of two is exact.  The first factor is one of 512
// numbers (code, parity), kept in shared memory: a lookup and a product per entry in the
// place of a square root with its rounding (the root took half of the gradient pass: 181 us
// against 77 us of traffic for 16384 x 6144 bf16).
constexpr int kF8SlopeTable = 512;
__device__ __forceinline__ void f8_slope_init(float* table, bool e5m2, int tid, int threads) {
  for (int i = tid; i < kF8SlopeTable; i += threads) {
    const uint16_t pair = (uint16_t)(i & 255);
    uint32_t h2;
    if (e5m2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(pair));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
    const float q = __low2float(*reinterpret_cast<const __half2*>(&h2));
    table[i] = __fmul_rn(2.f, __fsqrt_rn(i >= 256 ? __fmul_rn(2.f, q) : q));
  }
}

// 8 values times `inv` to 8 codes, round to nearest even.  The conversion saturates, so
// infinities need f8_encode_inf8 as well.
template <bool E5M2>
__device__ __forceinline__ uint2 f8_encode8(const float* v, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    const float a = __fmul_rn(v[4 * i], inv), b = __fmul_rn(v[4 * i + 1], inv);
    const float c = __fmul_rn(v[4 * i + 2], inv), d = __fmul_rn(v[4 * i + 3], inv);
    if constexpr (E5M2) {
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Puts right the codes of infinite values: NaN in e4m3, infinity in e5m2, sign kept.
template <bool E5M2>
__device__ __forceinline__ uint2 f8_encode_inf8(const float* v, uint2 c) {
  uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(v[i]) == kF8Inf) {
      const uint32_t code = (v[i] < 0.f ? 0x80u : 0u) | (E5M2 ? 0x7cu : 0x7fu);
      w[i >> 2] = (w[i >> 2] & ~(0xffu << (8 * (i & 3)))) | (code << (8 * (i & 3)));
    }
  return make_uint2(w[0], w[1]);
}

// 8 codes to 8 values times `scale` (both conversions are exact).
template <bool E5M2>
__device__ __forceinline__ void f8_decode8(uint2 c, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = (uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    uint32_t h2;
    if constexpr (E5M2)
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(pair));
    else
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

// N groups of 8 consecutive entries of a dense matrix (here in rows of 16-byte aligned groups),
// group i at (row0 + i * step, col): entries outside rows x cols read as 0.  Every load is issued
// before the first use.
template <int N, bool BF16>
__device__ __forceinline__ void f8_load_rows_t(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                               float (&v)[N][8]) {
  if (col + 8 <= cols) {
    if constexpr (BF16) {
      uint4 raw[N];
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(x.data) + (int64_t)row0 * x.ld + col;
#pragma unroll
      for (int i = 0; i < N; ++i)
        raw[i] = row0 + i * step < rows ? *reinterpret_cast<const uint4*>(p + (int64_t)(i * step) * x.ld)
                                        : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][2 * j] = __uint_as_float(w[j] << 16);
          v[i][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else {
      const float* p = reinterpret_cast<const float*>(x.data) + (int64_t)row0 * x.ld + col;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (row0 + i * step < rows) {
          a = reinterpret_cast<const float4*>(p + (int64_t)(i * step) * x.ld)[0];
          b = reinterpret_cast<const float4*>(p + (int64_t)(i * step) * x.ld)[1];
        }
        v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
        v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t at = (int64_t)(row0 + i * step) * x.ld + col;
    const bool live = row0 + i * step < rows;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = 0.f;
      if (live && col + j < cols)
        v[i][j] = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x.data)[at + j])
                       : reinterpret_cast<const float*>(x.data)[at + j];
    }
  }
}
// W words from byte `shift` (even, below 16) of w.
template <int W>
__device__ __forceinline__ void f8_shift_words(uint32_t (&w)[W + 4], int shift) {
  if (shift & 8) {
#pragma unroll
    for (int j = 0; j < W + 2; ++j) w[j] = w[j + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int j = 0; j < W + 1; ++j) w[j] = w[j + 1];
  }
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 8 * (shift & 2));
}

// f8_load_rows for rows whose groups of 8 are not 16-byte aligned: a thread reads the aligned
// blocks that hold its group (its neighbour reads the shared one too, from the L1 cache) and
// shifts; groups at a row's ends, whose blocks reach out of the row, go entry by entry.
// (16384 x 6139 bf16, quantised: 91 us; by 2-byte loads and shared memory 152 us; rows that
// 16-byte loads can address, 6136 columns: 69 us.)
template <int N, bool BF16>
__device__ __forceinline__ void f8_load_rows_shifted(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                                     float (&v)[N][8]) {
  constexpr int kEsz = BF16 ? 2 : 4, kWide = BF16 ? 1 : 2, kWords = 4 * kWide;
  constexpr int kBatch = BF16 && N > 1 ? 2 : 1;  // rows in flight (more spill)
  const uint8_t* p0 = reinterpret_cast<const uint8_t*>(x.data) + ((int64_t)row0 * x.ld + col) * kEsz;
  const int64_t pitch = x.ld * (int64_t)(step * kEsz);
  const int left = (cols - col) * kEsz;  // bytes to the row's end
#pragma unroll
  for (int i0 = 0; i0 < N; i0 += kBatch) {
    uint32_t w[kBatch][kWords + 4];
    int shift[kBatch];  // -1: entry by entry
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint8_t* p = p0 + (i0 + i) * pitch;
      const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
      const bool live = row0 + (i0 + i) * step < rows;
      const bool whole = s == 0 ? left >= 8 * kEsz : col > 0 && 16 * (kWide + 1) - s <= left;
      shift[i] = whole ? s : -1;
      if (whole) {
        const uint4* q = reinterpret_cast<const uint4*>(p - s);
#pragma unroll
        for (int b = 0; b <= kWide; ++b) {
          const uint4 y = live && (b < kWide || s > 0) ? q[b] : make_uint4(0u, 0u, 0u, 0u);
          w[i][4 * b] = y.x; w[i][4 * b + 1] = y.y; w[i][4 * b + 2] = y.z; w[i][4 * b + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[i][j] = 0u;
          if (live && j * kEsz < left)
            w[i][j] = BF16 ? (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << 16 : reinterpret_cast<const uint32_t*>(p)[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (shift[i] >= 0) {
        f8_shift_words<kWords>(w[i], shift[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i0 + i][j] =
              __uint_as_float(!BF16 ? w[i][j % kWords] : j & 1 ? w[i][j / 2] & 0xffff0000u : w[i][j / 2] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i0 + i][j] = __uint_as_float(w[i][j]);
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void f8_load_rows(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                             float (&v)[N][8]) {
  if (x.vec) {
    if (x.bf16) f8_load_rows_t<N, true>(x, row0, step, rows, col, cols, v);
    else f8_load_rows_t<N, false>(x, row0, step, rows, col, cols, v);
  } else {
    if (x.bf16) f8_load_rows_shifted<N, true>(x, row0, step, rows, col, cols, v);
    else f8_load_rows_shifted<N, false>(x, row0, step, rows, col, cols, v);
  }
}

// Stores of such rows: a half warp writes the 128 entries of a row as the aligned 16-byte blocks
// inside them, and the entries outside whole blocks one per lane (fewer than 8 at either end), by
// way of `xch`, kF8Xch floats of shared memory. Both half warps take part.  (16384 x 6139 bf16,
// read back: 77 us; entry by entry through shared memory 108 us; 6136 columns: 58 us.)
constexpr int kF8Xch = 144;  // floats per half warp: 33 blocks, and 16 banks between two of them
// Loads of such float32 rows where nothing else is in registers: 4 bytes per lane, all rows in
// flight at once, traded for groups of 8 in `xch` (4999 x 1531 quantised and read back: 22.5 us;
// by aligned blocks, with registers for one row in flight, 26.5).
template <int N>
__device__ __forceinline__ void f8_load_rows_xch(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                                 float (&v)[N][8], float* xch) {
  const int l = threadIdx.x & 15, c0 = col - 8 * l + l;
  const float* p = reinterpret_cast<const float*>(x.data) + (int64_t)row0 * x.ld + c0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[i][j] = row0 + i * step < rows && c0 + 16 * j < cols ? p[(int64_t)(i * step) * x.ld + 16 * j] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) xch[l + 16 * j] = v[i][j];
    __syncwarp();
    const float4 a = *reinterpret_cast<const float4*>(xch + 8 * l), b = *reinterpret_cast<const float4*>(xch + 8 * l + 4);
    v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
    v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    __syncwarp();
  }
}
template <int N, bool BF16>
__device__ __forceinline__ void f8_store_rows_xch_t(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                                    const float (&v)[N][8], float* xch) {
  constexpr int kEsz = BF16 ? 2 : 4, kWide = BF16 ? 1 : 2;
  const int l = threadIdx.x & 15, c0 = col - 8 * l;
  uint8_t* img = reinterpret_cast<uint8_t*>(xch);  // the entries start 16 bytes into it
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __syncwarp();
    uint4* own = reinterpret_cast<uint4*>(img + 16 + 16 * kWide * l);
    if constexpr (BF16) {
      uint4 raw;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[i][2 * j], v[i][2 * j + 1]);
      own[0] = raw;
    } else {
      reinterpret_cast<float4*>(own)[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
      reinterpret_cast<float4*>(own)[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
    }
    __syncwarp();
    const bool live = row0 + i * step < rows;
    // blocks are counted from the aligned address at or below the entries
    uint8_t* p = reinterpret_cast<uint8_t*>(x.data) + ((int64_t)(row0 + i * step) * x.ld + c0) * kEsz;
    const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15u), end = s + min(kFp8Block, cols - c0) * kEsz;
    p -= s;
    const int hb = s > 0 ? 1 : 0, tb = end >> 4;
#pragma unroll
    for (int b = 0; b < kWide; ++b) {
      const int k = l + 16 * b;
      // block k holds the entries' bytes from 16 k - s
      const uint4* q = reinterpret_cast<const uint4*>(img + 16 * (s == 0 ? k + 1 : k));
      const uint4 y = q[0], z = q[s == 0 ? 0 : 1];
      uint32_t w[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
      f8_shift_words<4>(w, (16 - s) & 15);
      if (live && k >= hb && k < tb) *reinterpret_cast<uint4*>(p + 16 * k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const int pos = l < 8 ? s + l * kEsz : 16 * tb + (l - 8) * kEsz;
    if (live && (l < 8 ? hb > 0 && pos < min(16, end) : tb >= hb && pos >= s && pos < end)) {
      const uint8_t* q = img + 16 + pos - s;
      if constexpr (BF16) *reinterpret_cast<uint16_t*>(p + pos) = *reinterpret_cast<const uint16_t*>(q);
      else *reinterpret_cast<uint32_t*>(p + pos) = *reinterpret_cast<const uint32_t*>(q);
    }
  }
}
template <int N>
__device__ __forceinline__ void f8_store_rows_xch(const F8Dense& x, int row0, int step, int rows, int col, int cols,
                                                  const float (&v)[N][8], float* xch) {
  if (x.bf16) f8_store_rows_xch_t<N, true>(x, row0, step, rows, col, cols, v, xch);
  else f8_store_rows_xch_t<N, false>(x, row0, step, rows, col, cols, v, xch);
}

__device__ __forceinline__ void f8_store8(const F8Dense& x, int64_t row, int col, int cols, const float* v) {
  const int64_t at = row * x.ld + col;
  if (x.vec && col + 8 <= cols) {
    if (x.bf16) {
      uint4 raw;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(x.data) + at) = raw;
    } else {
      float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(x.data) + at);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) {
      if (x.bf16)
        reinterpret_cast<__nv_bfloat16*>(x.data)[at + i] = __float2bfloat16_rn(v[i]);
      else
        reinterpret_cast<float*>(x.data)[at + i] = v[i];
    }
}

// N groups of 8 consecutive codes, in the manner of f8_load_rows (code 0 outside).  Codes
// are 16-byte aligned with a pitch that is a multiple of 16, so a multiple of 8 columns is
// 8-byte aligned.
template <int N>
__device__ __forceinline__ void f8_load_code_rows(const F8Mat& m, int row0, int step, int rows, int col, int cols,
                                                  uint2 (&c)[N]) {
  const uint8_t* p = m.codes + (int64_t)row0 * m.ld + col;
  if (col + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      c[i] = row0 + i * step < rows ? *reinterpret_cast<const uint2*>(p + (int64_t)(i * step) * m.ld)
                                    : make_uint2(0u, 0u);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t w[2] = {0u, 0u};
    const bool live = row0 + i * step < rows;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (live && col + j < cols) w[j >> 2] |= (uint32_t)p[(int64_t)(i * step) * m.ld + j] << (8 * (j & 3));
    c[i] = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ void f8_store_codes8(const F8Mat& m, int64_t row, int col, int cols, uint2 c) {
  uint8_t* p = m.codes + row * m.ld + col;
  if (col + 8 <= cols) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

// Where the scale byte of entry (row, 128-column block kb) lives.
__device__ __forceinline__ uint8_t* f8_scale_at(const F8Mat& m, int row, int kb) {
  return m.row_blocks ? m.scales + (int64_t)kb * m.s_col + row : m.scales + (int64_t)(row / kFp8Block) * m.s_row + kb;
}

// v[i] *= f'(u) from the checkpoint's entries at (row0 + i * step, col); table: f8_slope_init.
template <int N>
__device__ __forceinline__ void f8_times_slope(const F8Mat& saved, const float* table, int row0, int step, int rows,
                                               int col, int cols, float (&v)[N][8]) {
  uint2 c[N];
  uint32_t sb[N];
  f8_load_code_rows<N>(saved, row0, step, rows, col, cols, c);
#pragma unroll
  for (int i = 0; i < N; ++i)
    sb[i] = row0 + i * step < rows && col < cols ? *f8_scale_at(saved, row0 + i * step, col / kFp8Block) : 127u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (int)sb[i] - 127, parity = e & 1;
    const float scale = sb[i] == 255u ? __uint_as_float(0x7fc00000u) : f8_exp2((e - parity) / 2);
    const float* t = table + 256 * parity;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[i][j] = __fmul_rn(__fmul_rn(t[((j < 4 ? c[i].x : c[i].y) >> (8 * (j & 3))) & 255u], scale), v[i][j]);
  }
}

// Largest magnitude of v[i] (NaN is passed over, infinity is not).
template <int N>
__device__ __forceinline__ void f8_row_max(const float (&v)[N][8], float (&rmax)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rmax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) rmax[i] = fmaxf(rmax[i], fabsf(v[i][j]));
  }
}
// The same over finite entries.
template <int N>
__device__ __forceinline__ void f8_row_max_finite(const float (&v)[N][8], float (&rmax)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rmax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) rmax[i] = fmaxf(rmax[i], f8_finite_abs(v[i][j]));
  }
}
__device__ __forceinline__ float f8_half_warp_max(float m) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Stores the codes of v[i] at (row0 + i * step, col); inv[i]: 2^-e of the row's block;
// inf: some entry may be infinite.
template <int N, bool E5M2>
__device__ __forceinline__ void f8_store_rows_t(const F8Mat& m, int row0, int step, int rows, int col, int cols,
                                                const float (&v)[N][8], const float (&inv)[N], bool inf) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint2 c = f8_encode8<E5M2>(v[i], inv[i]);
    if (inf) c = f8_encode_inf8<E5M2>(v[i], c);
    if (row0 + i * step < rows && col < cols) f8_store_codes8(m, row0 + i * step, col, cols, c);
  }
}
template <int N>
__device__ __forceinline__ void f8_store_rows(const F8Mat& m, int row0, int step, int rows, int col, int cols,
                                              const float (&v)[N][8], const float (&inv)[N], bool inf) {
  if (m.e5m2) f8_store_rows_t<N, true>(m, row0, step, rows, col, cols, v, inv, inf);
  else f8_store_rows_t<N, false>(m, row0, step, rows, col, cols, v, inv, inf);
}

// Row blocks: each half warp holds whole rows of 128 columns.
template <int N>
__device__ __forceinline__ void f8_quantize_rows(const F8Mat& m, int row0, int step, int rows, int col, int cols,
                                                 const float (&v)[N][8]) {
  float rmax[N], inv[N];
  f8_row_max<N>(v, rmax);
  bool inf = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rmax[i] = f8_half_warp_max(rmax[i]);
    inf |= rmax[i] == kF8Inf;
  }
  inf = __any_sync(0xffffffffu, inf);
  if (inf) {
    f8_row_max_finite<N>(v, rmax);
#pragma unroll
    for (int i = 0; i < N; ++i) rmax[i] = f8_half_warp_max(rmax[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = f8_exponent(rmax[i], m.e5m2);
    inv[i] = f8_exp2(-e);
    if ((threadIdx.x & 15) == 0 && row0 + i * step < rows)
      *f8_scale_at(m, row0 + i * step, col / kFp8Block) = (uint8_t)(e + 127);
  }
  f8_store_rows<N>(m, row0, step, rows, col, cols, v, inv, inf);
}

}  // namespace
}  // namespace muon
