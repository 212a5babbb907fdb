// The cache's affine quantizer (RAQ-MLA page, appendix Table 5): levels min + k * scale with an
// FP16 minimum rounded down and an FP16 scale rounded up, every code decided exactly. Files that
// use it are compiled without contraction (-fmad=false).
#pragma once
#include <cuda_fp16.h>

#include "kernels.cuh"

namespace mlaq {

// Is x on the upper side of the midpoint between levels j and j+1 (exact ties go to the even
// level)?
__device__ __forceinline__ bool above_midpoint(float x, float m, float s, int j) {
  const float h = (static_cast<float>(j) + 0.5f) * s;  // <= 16 significant bits: exact
  const float t_lo = __fadd_rd(m, h);
  const float t_hi = __fadd_ru(m, h);
  bool gt, eq;
  if (t_lo == t_hi) {  // m + h is exactly representable in float
    gt = x > t_lo;
    eq = x == t_lo;
  } else {  // exact in double (at most 46 significant bits)
    const double T = static_cast<double>(m) + static_cast<double>(h);
    const double xd = static_cast<double>(x);
    gt = xd > T;
    eq = xd == T;
  }
  return gt || (eq && ((j + 1) & 1) == 0);
}

__device__ __forceinline__ int quant_code(float x, float m, float s, float inv_s, int L) {
  if (!(s > 0.f)) return 0;
  int k = __float2int_rn(__fsub_rn(x, m) * inv_s);
  k = min(max(k, 0), L);
  while (k > 0 && !above_midpoint(x, m, s, k - 1)) --k;
  while (k < L && above_midpoint(x, m, s, k)) ++k;
  return k;
}

struct QParams {
  float m, s, inv_s;
  uint32_t meta;  // scale bits | min bits << 16
  int flags;
};

// FP16 minimum rounded down and FP16 scale rounded up from the exact range [lo, hi]:
// RU16(RU32(RU32(hi - m) / L)) equals RU16((hi - m) / L) because each upward rounding lands at
// or below the FP16 result (L * scale is exact in float).
__device__ __forceinline__ QParams make_qparams(float lo, float hi, int L) {
  QParams q;
  q.flags = 0;
  __half mh = __float2half_rd(lo);
  float m = __half2float(mh);
  if (isinf(m)) {
    q.flags |= kErrRange;
    m = -65504.f;
  }
  float d = __fsub_ru(hi, m);
  float r = __fdiv_ru(d, static_cast<float>(L));
  __half sh = __float2half_ru(r);
  float s = __half2float(sh);
  if (isinf(s) || hi > 65504.f) {
    q.flags |= kErrRange;
    s = 65504.f;
  }
  q.m = m;
  q.s = s;
  q.inv_s = s > 0.f ? 1.f / s : 0.f;
  uint32_t mb = __half_as_ushort(__float2half_rn(m));  // m, s are FP16 values: exact
  uint32_t sb = __half_as_ushort(__float2half_rn(s));
  if ((mb & 0x7fffu) == 0) mb = 0;  // zero is stored as +0
  if ((sb & 0x7fffu) == 0) sb = 0;
  q.meta = sb | (mb << 16);
  return q;
}

// make_qparams for 15 steps without a division: the smallest FP16 scale with min + 15 * scale >= hi. A
// first candidate from a rounded-up reciprocal is that scale or the next FP16 above it; 15 times the one
// below is exact in float32, and reaches the exact hi - m where it reaches that difference rounded up.
__device__ __forceinline__ QParams make_qparams15(float lo, float hi) {
  QParams q;
  q.flags = 0;
  float m = __half2float(__float2half_rd(lo));
  if (isinf(m)) {
    q.flags |= kErrRange;
    m = -65504.f;
  }
  const float d = __fsub_ru(hi, m);
  const __half top = __float2half_ru(__fmul_ru(d, 0.06666667f));  // >= 1 / 15
  const uint16_t bits = __half_as_ushort(top);
  const float below = __half2float(__ushort_as_half(static_cast<uint16_t>(bits ? bits - 1 : 0)));
  float s = bits && __fmul_rn(below, 15.f) >= d ? below : __half2float(top);
  if (isinf(s) || hi > 65504.f) {
    q.flags |= kErrRange;
    s = 65504.f;
  }
  q.m = m;
  q.s = s;
  q.inv_s = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t mb = __half_as_ushort(__float2half_rn(m));  // m, s are FP16 values: exact
  uint32_t sb = __half_as_ushort(__float2half_rn(s));
  if ((mb & 0x7fffu) == 0) mb = 0;  // zero is stored as +0
  if ((sb & 0x7fffu) == 0) sb = 0;
  q.meta = sb | (mb << 16);
  return q;
}

}  // namespace mlaq
