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

// |v| where finite, else 0.
__device__ __forceinline__ float f8_finite_abs(float v) {
  const float a = fabsf(v);
  return a < __uint_as_float(0x7f800000u) ? a : 0.f;
}

// f(u) = max(u, 0)^2; NaN stays NaN.
__device__ __forceinline__ float f8_relu2(float u) { return u > 0.f ? __fmul_rn(u, u) : (u == u ? 0.f : u); }
// f'(u) from h = f(u): 2 relu(u) = 2 sqrt(h).
__device__ __forceinline__ float f8_relu2_slope(float h) { return __fmul_rn(2.f, __fsqrt_rn(h)); }

// 8 scaled values to 8 codes, round to nearest even.  The conversion saturates, so
// infinities are put right afterwards (NaN in e4m3, infinity in e5m2).
__device__ __forceinline__ uint2 f8_encode8(const float* v, float inv, bool e5m2) {
  uint32_t w[2];
  float s[8];
  bool inf = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = __fmul_rn(v[i], inv);
    inf |= fabsf(v[i]) == __uint_as_float(0x7f800000u);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    if (e5m2) {
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(s[4 * i + 1]), "f"(s[4 * i]));
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(s[4 * i + 3]), "f"(s[4 * i + 2]));
    } else {
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(s[4 * i + 1]), "f"(s[4 * i]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(s[4 * i + 3]), "f"(s[4 * i + 2]));
    }
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  if (inf) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(v[i]) == __uint_as_float(0x7f800000u)) {
        const uint32_t c = (v[i] < 0.f ? 0x80u : 0u) | (e5m2 ? 0x7cu : 0x7fu);
        w[i >> 2] = (w[i >> 2] & ~(0xffu << (8 * (i & 3)))) | (c << (8 * (i & 3)));
      }
  }
  return make_uint2(w[0], w[1]);
}

// 8 codes to 8 values times `scale` (both conversions are exact).
__device__ __forceinline__ void f8_decode8(uint2 c, float scale, bool e5m2, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = (uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    uint32_t h2;
    if (e5m2)
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(pair));
    else
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

// 8 consecutive entries (row, col .. col + 7) of a dense matrix; entries at or past `cols`
// read as 0 and are not written.
__device__ __forceinline__ void f8_load8(const F8Dense& x, int64_t row, int col, int cols, float* v) {
  const int64_t at = row * x.ld + col;
  if (x.vec && col + 8 <= cols) {
    if (x.bf16) {
      const uint4 raw = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(x.data) + at);
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x.data) + at);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.f;
    if (col + i < cols)
      v[i] = x.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x.data)[at + i])
                    : reinterpret_cast<const float*>(x.data)[at + i];
  }
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

// 8 consecutive codes, with the same treatment of the row's end.  Codes are 16-byte
// aligned with a pitch that is a multiple of 16, so a multiple of 8 columns is 8-byte
// aligned.
__device__ __forceinline__ uint2 f8_load_codes8(const F8Mat& m, int64_t row, int col, int cols) {
  const uint8_t* p = m.codes + row * m.ld + col;
  if (col + 8 <= cols) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + i < cols) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
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

}  // namespace
}  // namespace muon
