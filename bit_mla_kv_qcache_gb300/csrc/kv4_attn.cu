// Attention over the grouped-query cache in 4 bits for few query rows per kv head (single tokens,
// drafted tokens); rows = (query token, head of the group), 8 or 16 to a work item.
//
//   out = sum_t softmax_t(scale q . k_t) v_t,   k_t = km_t + ks_t n_t,  v_t = vm_t + vs_t n'_t
//
// Codes go to the tensor cores as they are: a nibble masked in place is the FP16 subnormal
// n 2^-24 (or 16 n 2^-24), so q . n is exact products summed in float32, and a token's scale and
// minimum enter outside: score = ks (q . n) + km sum(q). The query is prescaled by a power of two
// to FP16 range. In the readout the weight of a token is w = p vs in FP16 (one rounding, 2^-11),
// scaled by a power of two that follows the largest vs seen; sum p vm stays in float32.
//
// A warp owns 16 tokens at a time: S^T[16 tokens x rows] = K q^T with the key codes as the A operand
// (each lane loads its fragment's 16 contiguous bytes straight from the page), softmax on the
// accumulators, movmatrix turns the weights into the B operand, O^T += V^T w^T with the value codes
// as A (token pairs joined by byte permutes). No shared memory and no barrier inside the loop; the
// next tile is in registers before this one is multiplied. Warps of a CTA meet once per work item.
//
// Work: (sequence, kv head, row block) x its 16-token tiles, laid on one line; CTA i takes tiles
// [i S, (i + 1) S). An item cut by CTA borders is joined by the CTA that arrives last (partials in
// CTA order, so the result does not depend on who that is).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "append.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTok = 16;           // tokens per warp tile
constexpr int kMinTiles = 8;       // tiles per CTA at least: two per warp
constexpr float kSlack = 8.f;      // the running max is raised when a score exceeds it by more than this
constexpr float kWeightRoom = 64.f;  // w / p stays at or below this: w <= 2^14 in FP16

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t float2_to_half2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What one lane holds of a tile: key words of tokens g and g + 8, value words of tokens 2q, 2q + 1,
// 2q + 8, 2q + 9, and the numbers of tokens g and g + 8 (per group: scale | min of key, of value).
template <int D, int NG>
struct Tile {
  uint32_t k[2][D / 32];
  uint32_t v[4][D / 64];
  uint2 meta[2][NG];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

struct Item {
  int b, h, rb;  // sequence, kv head, row block
};

// The length, rows and tiles per row block of sequence b.
template <int R>
__device__ __forceinline__ void sequence(const Kv4AttnParams& p, int b, int& T, int& n, int& r0, int& tiles, int& blocks,
                                         int& flags) {
  T = __ldg(p.seq_lens + b);
  r0 = b, n = 1;
  if (p.cu_q) {
    r0 = __ldg(p.cu_q + b);
    n = __ldg(p.cu_q + b + 1) - r0;
  }
  if (n < 0 || n > p.max_q || r0 < 0 || r0 > p.n_rows - n) {
    flags |= kErrRows;
    n = 0;
  }
  if (T < 0 || T > static_cast<int64_t>(p.max_pages) * p.P) {
    flags |= kErrSeqOverflow;
    T = 0;
  }
  tiles = (T + kTok - 1) / kTok;
  if (p.window) tiles = min(tiles, static_cast<int>((static_cast<int64_t>(p.window) + R / p.G + kTok) / kTok) + 1);
  tiles = max(tiles, 1);
  blocks = (n * p.G + R - 1) / R;
}

// Tokens that query row i of the sequence sees: [lo, hi).
__device__ __forceinline__ int2 visible(const Kv4AttnParams& p, int T, int n, int i) {
  const int pos = T - n + i;
  const int hi = p.causal ? max(0, min(T, pos + 1)) : T;
  const int lo = p.window ? max(0, pos - p.window + 1) : 0;
  return make_int2(lo, hi);
}

template <int D, int NG, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3) kv4_decode_kernel(const Kv4AttnParams p) {
  constexpr int R = 8 * NT, KW = D / 32, VW = D / 64, MT = D / 16;
  constexpr int kRowPad = D + 4;
  __shared__ __align__(16) float s_o[kWarps][R][kRowPad];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ long long s_sum[kThreads + 1];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  int flags = 0;

  // ---- this CTA's stretch of the line of tiles: thread i sums sequences [i c, (i + 1) c)
  const int chunk = (p.B + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int b = tid * chunk; b < min(p.B, (tid + 1) * chunk); ++b) {
    int T, n, r0, tiles, blocks;
    sequence<R>(p, b, T, n, r0, tiles, blocks, flags);
    mine += static_cast<long long>(tiles) * blocks * p.Hkv;
  }
  {
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    long long base = 0;
    for (int w = 0; w < warp; ++w) base += s_sum[w];
    __syncthreads();
    s_sum[tid + 1] = base + x;
    if (tid == 0) s_sum[0] = 0;
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    const int f = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && f) atomicOr(p.err, f);
  }
  flags = 0;
  const long long total = s_sum[kThreads];
  long long share = (total + gridDim.x - 1) / gridDim.x;
  if (share < kMinTiles) share = kMinTiles;
  long long at = share * blockIdx.x;
  const long long end = min(total, at + share);
  if (at >= end) return;

  // ---- the first item: the thread whose sequences hold tile `at`, then the sequence
  Item it;
  long long item0;  // line position of the item's first tile
  int T, n, r0, tiles, blocks;
  {
    int lo = 0, hi = kThreads - 1;  // s_sum[lo] <= at < s_sum[lo + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_sum[mid + 1] > at) hi = mid;
      else lo = mid + 1;
    }
    long long pos = s_sum[lo];
    it.b = lo * chunk;
    int ignore = 0;
    for (;; ++it.b) {
      if (it.b >= p.B) return;  // lengths that changed under the call
      sequence<R>(p, it.b, T, n, r0, tiles, blocks, ignore);
      const long long w = static_cast<long long>(tiles) * blocks * p.Hkv;
      if (at < pos + w) break;
      pos += w;
    }
    const long long k = (at - pos) / tiles;
    it.h = static_cast<int>(k / blocks);
    it.rb = static_cast<int>(k % blocks);
    item0 = pos + k * tiles;
  }

  while (at < end) {
    // ---- the item's tokens
    const int i0 = it.rb * R / p.G, i1 = min(n - 1, (it.rb * R + R - 1) / p.G);
    const int t_lo = visible(p, T, n, i0).x, t_hi = visible(p, T, n, i1).y;
    const int tile0 = t_lo / kTok;
    const int a0 = static_cast<int>(at - item0);                                  // this CTA's tiles of the item
    const int a1 = static_cast<int>(min(end - item0, static_cast<long long>(tiles)));
    const int tile_end = min(tile0 + a1, (t_hi + kTok - 1) / kTok);

    // ---- queries: B fragments of rows g (+ 8), channels 32 j + 8 q4 + (0 .. 7)
    uint32_t bq[NT][KW][4];
    float fr[NT][2], qs[NT][2][NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = it.rb * R + 8 * nt + g;  // row = (query token rr / G, head rr % G)
      const bool live = rr < n * p.G;
      float x[KW][8];
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live)
          w = __ldg(reinterpret_cast<const uint4*>(p.q.data + static_cast<int64_t>(r0 + rr / p.G) * p.q.row_stride +
                                                   (it.h * p.G + rr % p.G) * p.q.head_stride + 32 * j) + q4);
        unpack8(w, p.f16, x[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[j][k]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      bool range = false;
      const int E = prescale_exponent(mx, range);
      const float up = pow2_int(E);
      float sum[NG];
#pragma unroll
      for (int k = 0; k < NG; ++k) sum[k] = 0.f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {  // field a: channels a and a + 4 of the word; odd fields count 16 times
          const float down = (a & 1) ? up * 0.0625f : up;
          const uint32_t w = float2_to_half2(x[j][a] * down, x[j][a + 4] * down);
          bq[nt][j][a] = w;
          const float2 f = half2_to_float2(w);
          sum[j / (KW / NG)] += (f.x + f.y) * ((a & 1) ? 16.f : 1.f);
        }
      }
      const float back = pow2_int(-E) * p.scale_log2;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
        sum[k] *= back;
      }
      // the accumulators' columns are rows 2 q4 and 2 q4 + 1
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fr[nt][c] = __shfl_sync(0xffffffffu, back * 16777216.f, 4 * (2 * q4 + c));
#pragma unroll
        for (int k = 0; k < NG; ++k) qs[nt][c][k] = __shfl_sync(0xffffffffu, sum[k], 4 * (2 * q4 + c));
      }
    }
    int2 vis[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rr = it.rb * R + 8 * nt + 2 * q4 + c;
        vis[nt][c] = rr < n * p.G ? visible(p, T, n, rr / p.G) : make_int2(0, 0);
      }
    // tiles in [full_lo, full_hi) are seen whole by every row of the block
    const int full_lo = (visible(p, T, n, i1).x + kTok - 1) / kTok;
    const int full_hi = visible(p, T, n, i0).y / kTok;

    float o[NT][MT][4], m[NT][2], l[NT][2], om[NT][2][NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < MT; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) om[nt][c][k] = 0.f;
      }
    }
    float wf = 0.f, vs_most = -1.f;  // weight factor 2^Ev, and the scale above which it is lowered

    const size_t region = static_cast<size_t>(it.h) * kv4_head_bytes(D, NG, p.P);
    const int32_t* table = p.page_table + static_cast<size_t>(it.b) * p.max_pages;
    // a bad page id drops the tile: its numbers read as zero and its tokens are hidden
    auto load = [&](int tile, Tile<D, NG>& t) -> bool {
      const int tok = tile * kTok, tp = tok & (p.P - 1);
      const int32_t pid = __ldg(table + (tok >> p.p_shift));
      if (pid < 0 || pid >= p.n_pages) {
        flags |= kErrBadPage;
        return false;
      }
      const uint8_t* base = p.pool + static_cast<size_t>(pid) * p.page_bytes + region;
      const uint8_t* kp = base + (tp + g) * (D / 2) + q4 * (D / 8);
      load_words<KW>(t.k[0], kp);
      load_words<KW>(t.k[1], kp + 8 * (D / 2));
      const uint8_t* vp = base + p.P * (D / 2) + (tp + 2 * q4) * (D / 2) + g * (D / 16);
      load_words<VW>(t.v[0], vp);
      load_words<VW>(t.v[1], vp + D / 2);
      load_words<VW>(t.v[2], vp + 8 * (D / 2));
      load_words<VW>(t.v[3], vp + 9 * (D / 2));
      const uint8_t* mp = base + p.P * D + (tp + g) * (8 * NG);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (NG == 1) {
          t.meta[e][0] = __ldg(reinterpret_cast<const uint2*>(mp + e * 64));
        } else {
#pragma unroll
          for (int k = 0; k < NG / 2; ++k) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(mp + e * 64 * NG) + k);
            t.meta[e][2 * k] = make_uint2(x.x, x.y);
            t.meta[e][2 * k + 1] = make_uint2(x.z, x.w);
          }
        }
      }
      return true;
    };

    Tile<D, NG> nxt;
    int tile = tile0 + a0 + warp;
    bool ok = false;
    if (tile < tile_end) ok = load(tile, nxt);
    for (; tile < tile_end; tile += kWarps) {
      Tile<D, NG> cur = nxt;
      const bool cur_ok = ok;
      if (tile + kWarps < tile_end) ok = load(tile + kWarps, nxt);
      if (!cur_ok) continue;  // the same for all lanes

      const int tok = tile * kTok;
      if (tok + kTok > T) {  // numbers of tokens behind the sequence are not read as such
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (tok + 8 * e + g >= T)
#pragma unroll
            for (int k = 0; k < NG; ++k) cur.meta[e][k] = make_uint2(0, 0);
      }
      // ---- scores
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int j = k * (KW / NG); j < (k + 1) * (KW / NG); ++j) {
          const uint32_t u0 = cur.k[0][j], u1 = cur.k[1][j], v0 = u0 >> 8, v1 = u1 >> 8;
          const uint32_t a01[4] = {u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x00F000F0u};
          const uint32_t a23[4] = {v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(s[nt], a01, bq[nt][j][0], bq[nt][j][1]);
            mma_f16_16816(s[nt], a23, bq[nt][j][2], bq[nt][j][3]);
          }
        }
        const float2 k0 = half2_to_float2(cur.meta[0][k].x), k1 = half2_to_float2(cur.meta[1][k].x);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            x[nt][c] += k0.x * (fr[nt][c] * s[nt][c]) + k0.y * qs[nt][c][k];
            x[nt][2 + c] += k1.x * (fr[nt][c] * s[nt][2 + c]) + k1.y * qs[nt][c][k];
          }
      }
      if (tile < full_lo || tile >= full_hi) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = tok + 8 * e + g;
              if (t < vis[nt][c].x || t >= vis[nt][c].y) x[nt][2 * e + c] = -INFINITY;
            }
      }
      // ---- running max and weight factor, raised rarely
      float2 v0[NG], v1[NG];
      float vs = 0.f;
      bool raise = false;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        v0[k] = half2_to_float2(cur.meta[0][k].y);
        v1[k] = half2_to_float2(cur.meta[1][k].y);
        vs = fmaxf(vs, fmaxf(v0[k].x, v1[k].x));
      }
      raise = vs > vs_most;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) raise |= fmaxf(x[nt][c], x[nt][2 + c]) > m[nt][c] + kSlack;
      if (__any_sync(0xffffffffu, raise)) {
        float wr = 1.f;
        vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 4));
        vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 8));
        vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 16));
        if (vs > vs_most) {  // 2^Ev vs in [1, 2)
          const int e = vs > 0.f ? max(-24, static_cast<int>(__float_as_uint(vs) >> 23) - 127) : -24;
          const float f = pow2_int(-e);
          wr = wf > 0.f ? f / wf : 1.f;
          wf = f;
          vs_most = kWeightRoom * pow2_int(e);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float sc[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float t = fmaxf(x[nt][c], x[nt][2 + c]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float mn = fmaxf(m[nt][c], t);
            sc[c] = mn > m[nt][c] ? ex2(m[nt][c] - mn) : 1.f;
            m[nt][c] = mn;
            l[nt][c] *= sc[c];
#pragma unroll
            for (int k = 0; k < NG; ++k) om[nt][c][k] *= sc[c];
            sc[c] *= wr;
          }
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[nt][j][0] *= sc[0], o[nt][j][2] *= sc[0];
            o[nt][j][1] *= sc[1], o[nt][j][3] *= sc[1];
          }
        }
      }
      // ---- weights
      uint32_t bw[NT][NG][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mm = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
          w[c] = ex2(x[nt][c] - mm);
          w[2 + c] = ex2(x[nt][2 + c] - mm);
          l[nt][c] += w[c] + w[2 + c];
#pragma unroll
          for (int k = 0; k < NG; ++k) om[nt][c][k] += w[c] * v0[k].y + w[2 + c] * v1[k].y;
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          const float s0 = v0[k].x * wf, s1 = v1[k].x * wf;
          bw[nt][k][0] = movmatrix_t(float2_to_half2(w[0] * s0, w[1] * s0));
          bw[nt][k][1] = movmatrix_t(float2_to_half2(w[2] * s1, w[3] * s1));
        }
      }
      // ---- readout
#pragma unroll
      for (int u = 0; u < VW; ++u) {
        const uint32_t p0 = prmt(cur.v[0][u], cur.v[1][u], 0x5410), p1 = prmt(cur.v[0][u], cur.v[1][u], 0x7632);
        const uint32_t p2 = prmt(cur.v[2][u], cur.v[3][u], 0x5410), p3 = prmt(cur.v[2][u], cur.v[3][u], 0x7632);
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const int sh = 8 * hi;
          const uint32_t r0w = p0 >> sh, r1w = p1 >> sh, r2w = p2 >> sh, r3w = p3 >> sh;
          const uint32_t a0w[4] = {r0w & 0x000F000Fu, r1w & 0x000F000Fu, r2w & 0x000F000Fu, r3w & 0x000F000Fu};
          const uint32_t a1w[4] = {r0w & 0x00F000F0u, r1w & 0x00F000F0u, r2w & 0x00F000F0u, r3w & 0x00F000F0u};
          const int j = 4 * u + 2 * hi;
          constexpr int kPer = MT / NG;  // 16-channel blocks per group
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(o[nt][j], a0w, bw[nt][j / kPer][0], bw[nt][j / kPer][1]);
            mma_f16_16816(o[nt][j + 1], a1w, bw[nt][(j + 1) / kPer][0], bw[nt][(j + 1) / kPer][1]);
          }
        }
      }
    }

    // ---- the warps of the CTA meet
    const float undo = wf > 0.f ? 16777216.f / wf : 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[nt][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int row = 8 * nt + 2 * q4 + c;
        if (g == 0) s_m[warp][row] = m[nt][c], s_l[warp][row] = v;
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          float z = om[nt][c][k];
          z += __shfl_xor_sync(0xffffffffu, z, 4);
          z += __shfl_xor_sync(0xffffffffu, z, 8);
          z += __shfl_xor_sync(0xffffffffu, z, 16);
          om[nt][c][k] = z;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float f = (j & 1) ? undo * 0.0625f : undo;
          const float z = om[nt][c][j / (MT / NG)];
          s_o[warp][row][16 * j + g] = o[nt][j][c] * f + z;
          s_o[warp][row][16 * j + 8 + g] = o[nt][j][2 + c] * f + z;
        }
      }
    __syncthreads();
    const long long item_end = item0 + tiles;
    const bool whole = at == item0 && end >= item_end;
    const long long c0 = item0 / share, c1 = (item_end - 1) / share;  // CTAs of the item
    // partial slots: 2 c for the item that CTA c continues, 2 c + 1 for the one that it begins
    const int slot = 2 * static_cast<int>(blockIdx.x) + (at == item0 ? 1 : 0);
    auto store_row = [&](int row, int ch, float v, float M, float L) {  // M in log2 units
      const int rr = it.rb * R + row;
      if (rr >= n * p.G) return;
      const size_t orow = static_cast<size_t>(r0 + rr / p.G) * p.Hq + it.h * p.G + rr % p.G;
      const float y = L > 0.f ? v / L : (L == 0.f ? 0.f : v);
      p.out[orow * D + ch] = p.f16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
      if (ch == 0 && p.lse) p.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : (L == 0.f ? -INFINITY : L);
    };
    for (int e = tid; e < R * D; e += kThreads) {
      const int row = e / D, ch = e % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][row]);
      float v = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][row] == -INFINITY ? (s_l[w][row] == 0.f ? 0.f : 1.f) : ex2(s_m[w][row] - M);
        if (f != 0.f) v += f * s_o[w][row][ch], L += f * s_l[w][row];
      }
      if (whole) {
        store_row(row, ch, v, M, L);
      } else {
        p.part_o[(static_cast<size_t>(slot) * R + row) * D + ch] = v;
        if (ch == 0) {
          float* ml = p.part_ml + (static_cast<size_t>(slot) * R + row) * 2;
          ml[0] = M;
          ml[1] = L;
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t parts = static_cast<uint32_t>(c1 - c0 + 1);
        const uint32_t before = atomicAdd(p.arrive + c0, 1u);
        s_last = before == parts - 1;
        if (s_last) {
          p.arrive[c0] = 0;
          __threadfence();
        }
      }
      __syncthreads();
      if (s_last) {
        for (int e = tid; e < R * D; e += kThreads) {
          const int row = e / D, ch = e % D;
          float M = -INFINITY, L = 0.f, v = 0.f;
          for (long long c = c0; c <= c1; ++c) {
            const size_t sl = 2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + sl * R + row);
            if (ml.y == 0.f) continue;
            const float x = __ldcg(p.part_o + (sl * R + row) * D + ch);
            const float mn = fmaxf(M, ml.x);
            const float fa = M == -INFINITY ? 0.f : ex2(M - mn), fb = ml.x == -INFINITY ? 1.f : ex2(ml.x - mn);
            v = v * fa + x * fb;
            L = L * fa + ml.y * fb;
            M = mn;
          }
          store_row(row, ch, v, M, L);
        }
      }
    }
    __syncthreads();

    // ---- the next item
    at = min(end, item_end);
    if (at >= end) break;
    item0 = at;
    if (++it.rb == blocks) {
      it.rb = 0;
      if (++it.h == p.Hkv) {
        it.h = 0;
        int ignore = 0;
        do {
          if (++it.b >= p.B) return;
          sequence<R>(p, it.b, T, n, r0, tiles, blocks, ignore);
        } while (blocks == 0);
      }
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && flags) atomicOr(p.err, flags);
}

template <int D, int NG>
cudaError_t launch(const Kv4AttnParams& p, int rows, int ctas, cudaStream_t stream) {
  if (rows == 8) kv4_decode_kernel<D, NG, 1><<<ctas, kThreads, 0, stream>>>(p);
  else kv4_decode_kernel<D, NG, 2><<<ctas, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int kv4_decode_rows(int max_q, int G) { return static_cast<int64_t>(max_q) * G <= 8 ? 8 : 16; }
int kv4_decode_ctas(int rows, int num_sms) {
  return std::min(num_sms * (rows == 8 ? 4 : 3), static_cast<int>(kKv4CounterBytes / 4));
}
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms) {
  const size_t ctas = kv4_decode_ctas(rows, num_sms);
  return kKv4CounterBytes + 2 * ctas * rows * (static_cast<size_t>(D) + 2) * sizeof(float);
}

cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  const int rows = kv4_decode_rows(p.max_q, p.G), ctas = kv4_decode_ctas(rows, num_sms);
  if (D == 128) {
    if (n_groups == 1) return launch<128, 1>(p, rows, ctas, stream);
    if (n_groups == 2) return launch<128, 2>(p, rows, ctas, stream);
    return launch<128, 4>(p, rows, ctas, stream);
  }
  return n_groups == 1 ? launch<64, 1>(p, rows, ctas, stream) : launch<64, 2>(p, rows, ctas, stream);
}

}  // namespace mlaq
