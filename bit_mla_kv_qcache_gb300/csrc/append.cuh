// What the appending kernels share: where a new row goes, and the rotation of channel pairs; small arithmetic that the
// attention over their pages takes too.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.cuh"
#include "kv4.cuh"

namespace mlaq {

// The largest b in [0, B) with cu[b] <= r, found by a whole warp: each round 32 lanes probe 32
// evenly spread entries of the remaining range (one round for B <= 32, two for B <= 1024).
__device__ __forceinline__ int warp_find_seq(const int32_t* cu, int B, int r) {
  int lo = 0, n = B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5, i = static_cast<int>(threadIdx.x & 31) * step;
    const bool le = i < n && __ldg(cu + lo + i) <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int hit = m ? 31 - __clz(m) : 0;
    lo += hit * step;
    n = min(step, n - hit * step);
  }
  return lo;
}

struct RowPlace {
  int64_t t;    // position, or -1: the row is skipped
  int32_t pid;  // page
  int tp;       // token within the page
  int flags;    // device error bits
  int b, len;   // its sequence, and the tokens that this held before
};

// Where row r of the call goes. Rows at and behind cu_new[B] belong to no sequence and are skipped
// without an error (a padded batch). Called by whole warps. Up to 32 sequences are looked at with one
// load per lane of the offsets and one of the lengths, so that only the page id waits for another load.
__device__ __forceinline__ RowPlace place_row(const int32_t* cu, const int32_t* lens, const int32_t* table, int B, int r,
                                              int max_new, int max_pages, int p_shift, int64_t n_pages, bool paged,
                                              int n_pos) {
  RowPlace z{-1, 0, 0, 0, 0, 0};
  int b = 0, r0, r1, s0;
  if (B <= 32) {
    const int lane = threadIdx.x & 31, i = min(lane, B - 1);
    const int end = __ldg(cu + i + 1), len = __ldg(lens + i), begin = __ldg(cu);
    b = __popc(__ballot_sync(0xffffffffu, lane < B && end <= r));
    if (b >= B) return z;
    r1 = __shfl_sync(0xffffffffu, end, b);
    r0 = __shfl_sync(0xffffffffu, end, b > 0 ? b - 1 : 0);
    if (b == 0) r0 = begin;
    s0 = __shfl_sync(0xffffffffu, len, b);
  } else {
    b = -1;
    if (r < B) {  // decode steps: one row per sequence
      r0 = __ldg(cu + r);
      r1 = __ldg(cu + r + 1);
      if (r0 == r && r1 == r + 1) b = r;
    }
    if (b < 0) {
      if (r >= __ldg(cu + B)) return z;
      b = warp_find_seq(cu, B, r);
      r0 = __ldg(cu + b);
      r1 = __ldg(cu + b + 1);
    }
    s0 = __ldg(lens + b);
  }
  if (r < r0 || r >= r1 || r1 - r0 > max_new) {
    z.flags = kErrRows;
    return z;
  }
  const int64_t t = static_cast<int64_t>(s0) + (r - r0);
  const int64_t pg = t >> p_shift;
  if (s0 < 0 || pg >= max_pages || t >= n_pos) {
    z.flags = kErrSeqOverflow;
    return z;
  }
  if (paged) {
    z.pid = __ldg(table + static_cast<size_t>(b) * max_pages + pg);
    if (z.pid < 0 || z.pid >= n_pages) {
      z.flags = kErrBadPage;
      return z;
    }
  }
  z.tp = static_cast<int>(t & ((1 << p_shift) - 1));
  z.t = t;
  z.b = b;
  z.len = s0;
  return z;
}

__device__ __forceinline__ float elem_lo(uint32_t w, bool f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w))) : __uint_as_float(w << 16);
}
__device__ __forceinline__ float elem_hi(uint32_t w, bool f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))) : __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack8(const uint4& w, bool f16, float (&x)[8]) {
  x[0] = elem_lo(w.x, f16), x[1] = elem_hi(w.x, f16), x[2] = elem_lo(w.y, f16), x[3] = elem_hi(w.y, f16);
  x[4] = elem_lo(w.z, f16), x[5] = elem_hi(w.z, f16), x[6] = elem_lo(w.w, f16), x[7] = elem_hi(w.w, f16);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, bool f16) {
  if (f16) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8], bool f16) {
  return make_uint4(pack2(x[0], x[1], f16), pack2(x[2], x[3], f16), pack2(x[4], x[5], f16), pack2(x[6], x[7], f16));
}

// The largest exponent E with max_abs * 2^E < 2^15 for every finite max_abs, at most 120: brings a row of queries into FP16.
__device__ __forceinline__ int fp16_exponent(float max_abs) {
  return max_abs > 0.f ? min(14 + 127 - static_cast<int>(__float_as_uint(max_abs) >> 23), 120) : 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two float32 operations in one instruction. A product and a sum that follow one another may still come
// out fused (seen with the 13.0 assembler), so these are used where that changes nothing.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The angles of one thread's eight channels 8 i .. 8 i + 7 at position t: with neighbouring pairs
// four (c, s), with pairs half a rotation apart eight (s negative for the first of a pair, so that
// both are x c + partner s); rows of the tables are 16-byte aligned (rot_dim / 2 is a multiple of 8).
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles load_angles(const Rotation& rot, int64_t t, int i) {
  Angles a;
#pragma unroll
  for (int k = 0; k < 8; ++k) a.c[k] = 1.f, a.s[k] = 0.f;
  if (8 * i >= rot.rot_dim) return a;
  const int half = rot.rot_dim >> 1;
  const size_t row = static_cast<size_t>(t) * half;
  if (rot.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(rot.cos_tab + row + 4 * i));
    const float4 s = __ldg(reinterpret_cast<const float4*>(rot.sin_tab + row + 4 * i));
    a.c[0] = c.x, a.c[1] = c.y, a.c[2] = c.z, a.c[3] = c.w;
    a.s[0] = s.x, a.s[1] = s.y, a.s[2] = s.z, a.s[3] = s.w;
  } else {
    const bool first = 8 * i < half;
    const int f = first ? 8 * i : 8 * i - half;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(rot.cos_tab + row + f) + k);
      const float4 s = __ldg(reinterpret_cast<const float4*>(rot.sin_tab + row + f) + k);
      a.c[4 * k] = c.x, a.c[4 * k + 1] = c.y, a.c[4 * k + 2] = c.z, a.c[4 * k + 3] = c.w;
      a.s[4 * k] = first ? -s.x : s.x, a.s[4 * k + 1] = first ? -s.y : s.y;
      a.s[4 * k + 2] = first ? -s.z : s.z, a.s[4 * k + 3] = first ? -s.w : s.w;
    }
  }
  return a;
}

// (a, b) -> (a cos - b sin, b cos + a sin) on the thread's eight channels (thread i of the head, in
// lane order); every product and sum is rounded by itself, so the keys' codes are reproducible.
// The partner of a pair half a rotation away sits in the lane rot_dim / 16 further up or down; the
// whole warp takes part.
__device__ __forceinline__ void rotate8(const Rotation& rot, const Angles& a, int i, const uint4& raw, bool f16,
                                        float (&x)[8]) {
  unpack8(raw, f16, x);
  if (rot.rot_dim == 0) return;
  if (rot.interleaved) {
    if (8 * i < rot.rot_dim) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float u = x[2 * k], w = x[2 * k + 1];
        x[2 * k] = __fsub_rn(__fmul_rn(u, a.c[k]), __fmul_rn(w, a.s[k]));
        x[2 * k + 1] = __fadd_rn(__fmul_rn(w, a.c[k]), __fmul_rn(u, a.s[k]));
      }
    }
    return;
  }
  const int d = rot.rot_dim >> 4, lane = threadIdx.x & 31;
  const bool in = i < 2 * d;
  const int src = !in ? lane : i < d ? lane + d : lane - d;
  uint4 o;
  o.x = __shfl_sync(0xffffffffu, raw.x, src);
  o.y = __shfl_sync(0xffffffffu, raw.y, src);
  o.z = __shfl_sync(0xffffffffu, raw.z, src);
  o.w = __shfl_sync(0xffffffffu, raw.w, src);
  if (!in) return;
  float y[8];
  unpack8(o, f16, y);
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = __fadd_rn(__fmul_rn(x[k], a.c[k]), __fmul_rn(y[k], a.s[k]));
}

}  // namespace mlaq
