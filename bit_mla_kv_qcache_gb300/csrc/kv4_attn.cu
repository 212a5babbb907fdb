// Attention over the grouped-query cache in 4 bits for few query rows per kv head (single tokens,
// drafted tokens); rows = (query token, head of the group), 8 or 16 to a work item.
//
//   out = sum_t softmax_t(scale q . k_t) v_t,   k_t = km_t + ks_t n_t,  v_t = vm_t + vs_t n'_t
//
// Codes go to the tensor cores as they are: a nibble masked in place is the FP16 subnormal
// n 2^-24 (or 16 n 2^-24), so q . n is exact products summed in float32, and a token's scale and
// minimum enter outside: score = ks (q . n) + km sum(q). The query is prescaled by a power of two
// to FP16 range. In the readout the weight of a token is w = p vs in FP16 (one rounding, 2^-11),
// scaled by a power of two that follows the largest vs seen (below 2^-18 of it, by 2^-29 of it); sum p vm stays in float32.
// Codes are 7.5 from zero on average, values are not: the weights' rounding errors enter multiplied by the codes, larger than the
// values. For FP16 rows 7.5 times the sum of the errors is put back, which leaves them multiplied by n - 7.5 (error of the output
// 5.1e-4 -> 3.1e-4 of it, half of that its own rounding; 64 ragged sequences up to 16K 49.4 -> 51.9 us). A BF16 output's
// own rounding, 1.7e-3, covers them.
//
// A warp owns steps of 32 tokens, two tiles of 16: S^T[16 tokens x rows] = K q^T with the key codes as the A operand
// (a lane's fragment is 16 contiguous bytes of the page), softmax on the accumulators, movmatrix
// turns the weights into the B operand, O^T += V^T w^T with the value codes as A (token pairs joined
// by byte permutes). Steps come through a ring of the warp by asynchronous copies, two ahead of their use (the
// ring in place of loads into registers: 94.6 -> 70.1 us for 32 sequences of 8K, 32 query heads on 8, D = 128); no
// barrier inside the loop. The warps of a CTA meet once per work item.
//
// Work: items (sequence, kv head, row block), each a row of 32-token steps. Where they can be cut so that
// every CTA has one part of one item, they are: the share is the smallest of a few multiples of
// total / CTAs for which the parts fit (a second, short segment costs a CTA ~12 us of latencies: ids,
// queries, first tokens, meeting, joining). Otherwise the items lie on one line that is cut into equal
// stretches (one sequence of 128K, 64 heads on 8: 47.3 us on the line, 39.6 with one part each). An item in several
// parts is joined by the CTA that arrives last (parts in CTA order, so the result does not depend on who that is).
//
// Rows: 8 or 16 to an item; two blocks of 16 up to 32 rows, above that the kernel for many rows. Measured on either
// side (eight ragged sequences up to 32K, 8 heads on each of 4, D = 128): 24 rows 79 us here and 79 there, 40 rows 117 and 81;
// one sequence of 4K: 24 rows 17 and 26 us, 40 rows 19 and 27; D = 64, 24 rows 49 and 52 us.
//
// Bound: the chain of a step within a warp. 32 sequences of 8K take 65 us where their bytes take 42 at the card's copy rate, and no
// unit is full: issue 55%, the ALU pipe (masks, shifts and byte permutes of codes) 53%, DRAM 54%, the tensor pipe 25%. Four warps
// share a scheduler; between two instructions a warp waits 1.5 issue slots for fixed latencies, 1.0 for its turn, 0.8 for
// the ALU pipe and 0.5 for shared memory. ~9 us are launch, the first tokens, and the joining (one sequence of 1K: 10.1 us).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "append.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

namespace mlaq {
namespace {

constexpr int kTile = 16;      // tokens of a tensor-core tile
constexpr int kTok = 32;       // tokens of a step: two tiles
constexpr int kMaxParts = 64;  // CTAs that one item is cut into, at most

template <int D, int NG, int NT>
struct Geom {
  static constexpr int kWarps = NT == 1 ? 8 : 6;  // two CTAs per SM: 16 warps of 128 registers, or 12 of 168
  static constexpr int kPair = NT == 1 ? 2 : 1;  // tiles multiplied side by side
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kMinSteps = 2 * kWarps;    // an item is not cut below this: joining costs more than it saves
  static constexpr int kR = 8 * NT;
  static constexpr int kCodes = kTok * D / 2;     // bytes of a step's key codes, and of its value codes
  static constexpr int kStage = 2 * kCodes + kTok * 8 * NG;
  static constexpr int kStages = 3 * kStage * 16 <= 210 * 1024 ? 3 : 2;
  static constexpr int kRowPad = D + 4;
  // a warp's ring, later its sums when the warps meet
  static constexpr int kRing = kStages * kStage > kR * kRowPad * 4 ? kStages * kStage : kR * kRowPad * 4;
  static constexpr int kSmem = kWarps * kRing;
};

constexpr float kSlack = 8.f;      // the running max is raised when a score exceeds it by more than this
constexpr float kNoMax = -1e30f;  // the running max before the first score
constexpr float kWeightRoom = 64.f;  // w / p stays at or below this: w <= 2^14 in FP16, whose half step below
                                     // 2^-14 is 2^-25, so a token's weight is off by at most 2^-29 of the largest vs

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

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Copies one tile (16 tokens from `tp` of the page region `base`) to its place in a ring stage: keys at
// `ks`, values at `vs`, numbers at `ms`. Key rows keep their order. The value row of token
// t = 8f + 2q + e goes to row 8f + 4e + q, at D = 128 with its 16-byte chunks exchanged by pairs for
// q >= 2, so that the 8-byte reads of a half warp (four q, four g) fall in distinct banks.
template <int D, int NG>
__device__ __forceinline__ void copy_tile(uint8_t* ks, uint8_t* vs, uint8_t* ms, const uint8_t* base, int tp, int P,
                                          int lane) {
  constexpr int CPR = D / 32;  // 16-byte chunks per row
  const int t = lane / CPR, c = lane % CPR, q = (t >> 1) & 3;
  const uint8_t* kp = base + (tp * (D / 2) + 16 * lane);
  uint8_t* vd = vs + ((t & 8) + 4 * (t & 1) + q) * (D / 2) + 16 * (D == 128 ? c ^ (q & 2) : c);
#pragma unroll
  for (int i = 0; i < CPR / 2; ++i) {  // 32 chunks cover eight rows (D = 128) or sixteen
    cp_async_cg16(ks + 16 * lane + 512 * i, kp + 512 * i);
    cp_async_cg16(vd + 512 * i, kp + P * (D / 2) + 512 * i);
  }
  if (lane < 8 * NG) cp_async_cg16(ms + 16 * lane, base + (P * D + tp * 8 * NG + 16 * lane));
}

// This lane's key words of tokens g and g + 8, channels 8 q4 .. 8 q4 + 7 of each block of 32.
template <int D>
__device__ __forceinline__ void read_keys(uint32_t (&k)[2][D / 32], const uint8_t* ks, int g, int q4) {
  load_words<D / 32>(k[0], ks + g * (D / 2) + q4 * (D / 8));
  load_words<D / 32>(k[1], ks + (g + 8) * (D / 2) + q4 * (D / 8));
}
// Its value words of tokens 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9.
template <int D>
__device__ __forceinline__ void read_values(uint32_t (&v)[4][D / 64], const uint8_t* vs, int g, int q4) {
  const int at = D == 128 ? 16 * ((g >> 1) ^ (q4 & 2)) + 8 * (g & 1) : 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) load_words<D / 64>(v[i], vs + q4 * (D / 2) + at + 4 * i * (D / 2));
}
// The numbers of tokens g and g + 8, per group: scale | min of the key, then of the value.
template <int NG>
__device__ __forceinline__ void read_numbers(uint2 (&m)[2][NG], const uint8_t* ms, int g) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if constexpr (NG == 1) {
      m[e][0] = *reinterpret_cast<const uint2*>(ms + (g + 8 * e) * 8);
    } else {
#pragma unroll
      for (int k = 0; k < NG / 2; ++k) {
        const uint4 x = *reinterpret_cast<const uint4*>(ms + (g + 8 * e) * 8 * NG + 16 * k);
        m[e][2 * k] = make_uint2(x.x, x.y);
        m[e][2 * k + 1] = make_uint2(x.z, x.w);
      }
    }
  }
}
// Keeps the loads that follow behind the work that came before (their registers are not needed yet).
__device__ __forceinline__ void no_loads_across() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ float sum_over_g(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

// The part of an item that a CTA works on. Kept in shared memory: the loop over the tokens needs the
// registers.
struct Place {
  int b, h, rb;                 // the item: sequence, kv head, row block
  int T, n, r0, tiles, blocks;  // of the sequence: length, query rows, first row, steps of an item, row blocks
  int a0, a1;                   // steps of the item done here
  int c0, parts;                // first CTA of the item, and how many
  long long at, end, item0, share;  // on the line: here, end of the CTA's stretch, the item's start, length of a stretch
};

// The item's steps that lie in the CTA's stretch of the line.
__device__ __forceinline__ void on_line(Place& s) {
  s.a0 = static_cast<int>(s.at - s.item0);
  s.a1 = static_cast<int>(min(s.end - s.item0, static_cast<long long>(s.tiles)));
  s.c0 = static_cast<int>(s.item0 / s.share);
  s.parts = static_cast<int>((s.item0 + s.tiles - 1) / s.share) - s.c0 + 1;
}

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
  const int lo = p.window && pos >= p.window ? pos - p.window + 1 : 0;  // no overflow before the first token
  return make_int2(lo, hi);
}

// Channels 4 c4 .. 4 c4 + 3 of row `row` of the item: sums v under the max M (log2 units) and sum L.
template <int D, int R>
__device__ __forceinline__ void store_out(const Kv4AttnParams& p, const Place& at, int row, int c4, float4 v, float M, float L) {
  const int rr = at.rb * R + row;
  if (rr >= at.n * p.G) return;
  const size_t orow = static_cast<size_t>(at.r0 + rr / p.G) * p.Hq + at.h * p.G + rr % p.G;
  const float y = L == 0.f ? 0.f : 1.f / L;
  reinterpret_cast<uint2*>(p.out + orow * D)[c4] = make_uint2(pack2(v.x * y, v.y * y, p.f16), pack2(v.z * y, v.w * y, p.f16));
  if (c4 == 0 && p.lse) p.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// The CTA that came last joins the item's parts, those of CTAs c0 .. c0 + parts - 1 in this order:
// first the parts' weights, then the outputs, which each thread copies to shared memory (`room`
// bytes) for as many parts as fit there at once, all in flight and none in registers.
template <int D, int R, int kThreads>
__device__ __forceinline__ void merge_parts(const Kv4AttnParams& p, const Place& at, uint8_t* smem, int room,
                                            float (&s_f)[kMaxParts + 1][R], float (&s_ml)[R][2]) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = at.c0, parts = at.parts, rows = min(R, at.n * p.G - at.rb * R);
  auto slot_of = [&](int i) { return static_cast<uint32_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)); };
  constexpr int kPer = (kMaxParts + 31) / 32, kPart = R * D * 4;
  const int batch = room / kPart, n_chunks = rows * (D / 4);  // 16-byte chunks of a part
  auto ask = [&](int e, int i0, int n) {
    for (int i = 0; i < n; ++i)
      cp_async_cg16(smem + i * kPart + e * 16, p.part_o + static_cast<size_t>(slot_of(i0 + i)) * (R * D) + 4 * e);
  };
  if (tid < n_chunks) ask(tid, 0, min(batch, parts));  // on their way while the weights are formed
  for (int row = warp; row < rows; row += kThreads / 32) {
    float M = kNoMax, L = 0.f;
    float2 ml[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = lane + 32 * k;
      ml[k] = i < parts ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(i) * R + row) : make_float2(kNoMax, 0.f);
      M = fmaxf(M, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = lane + 32 * k;
      const float f = ex2(ml[k].x - M);
      if (i < parts) s_f[i][row] = f;
      L += f * ml[k].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_ml[row][0] = M, s_ml[row][1] = L;
  }
  __syncthreads();
  for (int e = tid; e < n_chunks; e += kThreads) {
    const int row = e / (D / 4), c4 = e % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += batch) {
      const int n = min(batch, parts - i0);
      if (e != tid || i0 > 0) ask(e, i0, n);
      cp_async_wait_all();  // a thread reads what it copied itself
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(smem + i * kPart + e * 16);
        const float f = s_f[i0 + i][row];
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
    }
    store_out<D, R>(p, at, row, c4, v, s_ml[row][0], s_ml[row][1]);
  }
}

template <int D, int NG, int NT>
__global__ void __launch_bounds__(Geom<D, NG, NT>::kThreads, 2) kv4_decode_kernel(const Kv4AttnParams p) {
  using Ge = Geom<D, NG, NT>;
  constexpr int R = 8 * NT, KW = D / 32, VW = D / 64, MT = D / 16;
  constexpr int PT = Ge::kPair;
  constexpr int kWarps = Ge::kWarps, kThreads = Ge::kThreads, kRowPad = Ge::kRowPad;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ float s_f[kMaxParts + 1][R];  // weights of the parts of a cut item; then the rows' (M, L)
  __shared__ float s_ml[R][2];
  constexpr int kHeld = 256;  // sequences that the quick way of sharing the work takes
  __shared__ int s_last, s_steps[kHeld], s_items[kHeld];  // of each sequence: steps of an item, items
  __shared__ Place s_at;
  __shared__ int s_full[kWarps][4];  // steps that every row sees whole: from, to; tokens seen by any: end, begin
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  int flags = 0;

  // ---- which part of which item. Thread b looks at sequence b; then every warp works the rest out by
  // itself, lane i for sequences [i c, (i + 1) c). (Loops stay rolled: this code runs once, from cold
  // instruction caches.)
  {
    const int chunk = (p.B + 31) / 32, first = lane * chunk, n_ctas = static_cast<int>(gridDim.x);
    const int last = min(p.B, first + chunk);
    int share = 0, mine = 0;  // parts of the lane's items
    bool small = p.B <= kHeld;
    if (small) {
      for (int b = tid; b < p.B; b += kThreads) {
        int T, n, r0, tiles, blocks;
        sequence<R>(p, b, T, n, r0, tiles, blocks, flags);
        s_steps[b] = tiles;
        s_items[b] = blocks * p.Hkv;
      }
      if (blockIdx.x == 0) {
        const int f = __reduce_or_sync(0xffffffffu, flags);
        if (lane == 0 && f) atomicOr(p.err, f);
      }
      flags = 0;
      __syncthreads();
      float steps = 0.f;
      int items = 0, most = 0;
#pragma unroll 1
      for (int b = first; b < last; ++b) {
        steps += static_cast<float>(s_steps[b]) * static_cast<float>(s_items[b]);
        items = min(items + s_items[b], 1 << 20);
        if (s_items[b] > 0) most = max(most, s_steps[b]);
      }
      items = __reduce_add_sync(0xffffffffu, items);
      small = items <= n_ctas && __all_sync(0xffffffffu, steps < 3e7f);  // 32 lanes: below 2^30
      if (small) {
        const int total = __reduce_add_sync(0xffffffffu, static_cast<int>(steps)), top = __reduce_max_sync(0xffffffffu, most);
        const int least = max(min(Ge::kMinSteps, top), (top + kMaxParts - 2) / (kMaxParts - 1));
        const float base = static_cast<float>(total) / static_cast<float>(n_ctas);
        float times = 1.f;
#pragma unroll 1
        for (int k = 0; k < 9 && share == 0; ++k, times *= 1.08f) {  // up to about twice
          const int s = max(least, static_cast<int>(base * times) + 1);
          mine = 0;
#pragma unroll 1
          for (int b = first; b < last; ++b) mine += s_items[b] * ((s_steps[b] + s - 1) / s);
          if (__reduce_add_sync(0xffffffffu, mine) <= n_ctas) share = s;
        }
      }
    }
    if (share > 0) {
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int x = static_cast<int>(blockIdx.x);
      if (x >= __shfl_sync(0xffffffffu, upto, 31)) return;
      if (x >= upto - mine && x < upto) {  // one lane; every warp stores the same
        Place s{};
        int r = x - (upto - mine), ignore = 0;
#pragma unroll 1
        for (s.b = first; s.b + 1 < last; ++s.b) {
          const int w = s_items[s.b] * ((s_steps[s.b] + share - 1) / share);
          if (r < w) break;
          r -= w;
        }
        sequence<R>(p, s.b, s.T, s.n, s.r0, s.tiles, s.blocks, ignore);
        s.tiles = s_steps[s.b];
        s.parts = (s.tiles + share - 1) / share;
        const uint32_t part = r % s.parts;
        const int item = min(r / s.parts, max(1, s.blocks * p.Hkv) - 1);  // (lengths may change under the call)
        s.h = s.blocks > 1 ? item / s.blocks : item;
        s.rb = s.blocks > 1 ? item - s.h * s.blocks : 0;
        s.a0 = static_cast<uint32_t>(s.tiles) * part / s.parts;  // steps < 2^25, parts <= 64
        s.a1 = static_cast<uint32_t>(s.tiles) * (part + 1) / s.parts;
        s.c0 = x - part;  // at = end: not on the line
        s_at = s;
      }
    } else {
      long long steps = 0;
      int most = 0;
      for (int b = first; b < last; ++b) {
        int T, n, r0, tiles, blocks;
        sequence<R>(p, b, T, n, r0, tiles, blocks, flags);
        steps += static_cast<long long>(tiles) * blocks * p.Hkv;
        if (blocks > 0) most = max(most, tiles);
      }
      if (blockIdx.x == 0 && warp == 0) {
        const int f = __reduce_or_sync(0xffffffffu, flags);
        if (lane == 0 && f) atomicOr(p.err, f);
      }
      flags = 0;
      const int top = __reduce_max_sync(0xffffffffu, most);
      long long before = steps;  // of the lanes up to this one
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const long long total = __shfl_sync(0xffffffffu, before, 31);
      before -= steps;
      const long long stretch = max((total + n_ctas - 1) / n_ctas, static_cast<long long>(max(min(Ge::kMinSteps, top), (top + kMaxParts - 2) / (kMaxParts - 1))));
      const long long x = stretch * blockIdx.x;
      if (x >= total) return;
      if (x >= before && x < before + steps) {  // one lane; every warp stores the same
        Place s{};
        s.at = x;
        s.end = min(total, x + stretch);
        s.share = stretch;
        long long pos = before;
        int ignore = 0;
        for (s.b = first;; ++s.b) {
          sequence<R>(p, s.b, s.T, s.n, s.r0, s.tiles, s.blocks, ignore);
          const long long w = static_cast<long long>(s.tiles) * s.blocks * p.Hkv;
          if (x < pos + w || s.b + 1 >= p.B) break;
          pos += w;
        }
        const long long k = min((x - pos) / s.tiles, static_cast<long long>(max(1, s.blocks * p.Hkv)) - 1);
        s.h = s.blocks > 0 ? static_cast<int>(k / s.blocks) : 0;
        s.rb = s.blocks > 0 ? static_cast<int>(k % s.blocks) : 0;
        s.item0 = pos + k * s.tiles;
        on_line(s);
        s_at = s;
      }
    }
    __syncwarp();
  }

  while (true) {
    // ---- the item's tokens
    int tile, tile_end;
    {
      const int i0 = s_at.rb * R / p.G, i1 = min(s_at.n - 1, (s_at.rb * R + R - 1) / p.G);
      const int2 first = visible(p, s_at.T, s_at.n, i0), last = visible(p, s_at.T, s_at.n, i1);
      const int tile0 = first.x / kTok;
      tile = tile0 + s_at.a0 + warp;
      tile_end = min(tile0 + s_at.a1, (last.y + kTok - 1) / kTok);
      // steps in [full_lo, full_hi) are seen whole by every row of the block
      if (lane == 0) {
        s_full[warp][0] = (last.x + kTok - 1) / kTok;
        s_full[warp][1] = first.y / kTok;
        s_full[warp][2] = last.y;
        s_full[warp][3] = first.x;
      }
      __syncwarp();
    }
    const volatile int* const full = s_full[warp];  // read where needed: the loop has no registers to spare

    // ---- this warp's steps tile, tile + kWarps, ...: the first ones are on their way before the
    // queries are read. Lane i holds the page id of tile i & 1 of the next step to be copied; a bad one
    // drops its tile. (Any id may stand in the table, so whether a tile was asked for is told by its tokens.)
    constexpr int kStages = Ge::kStages;
    uint8_t* const ring = smem + warp * Ge::kRing;
    int next = tile;
    uint32_t next_st = 0, present = 0;  // two bits per stage
    // tiles that no row sees are not asked for: their pages may be gone (behind a sliding window)
    auto asked = [&](int tok) { return tok < full[2] && tok + kTile > full[3]; };
    auto page_id = [&](int t) {
      const int tok = t * kTok + kTile * (lane & 1);
      return asked(tok) ? __ldg(p.page_table + static_cast<size_t>(s_at.b) * p.max_pages + (tok >> p.p_shift)) : -1;
    };
    int32_t pid = page_id(next);
    auto issue = [&]() {
      if (next < tile_end) {
        uint8_t* const st = ring + next_st * Ge::kStage;
        const int h = *const_cast<const volatile int*>(&s_at.h);
        present &= ~(3u << (2 * next_st));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int32_t id = __shfl_sync(0xffffffffu, pid, r);
          if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.n_pages)) {
            const uint8_t* base = p.pool + static_cast<uint64_t>(static_cast<uint32_t>(id)) * static_cast<uint32_t>(p.page_bytes) +
                                  static_cast<uint32_t>(h * kv4_head_bytes(D, NG, p.P));
            copy_tile<D, NG>(st + r * (Ge::kCodes / 2), st + Ge::kCodes + r * (Ge::kCodes / 2),
                             st + 2 * Ge::kCodes + r * (kTile * 8 * NG), base, (next * kTok + r * kTile) & (p.P - 1), p.P, lane);
            present |= 1u << (2 * next_st + r);
          } else if (asked(next * kTok + r * kTile)) {
            flags |= kErrBadPage;
          }
        }
        next += kWarps;
        next_st = next_st + 1 == kStages ? 0 : next_st + 1;
        if (next < tile_end) pid = page_id(next);
      }
      cp_async_commit();
    };
    // ---- queries: B fragments of rows g (+ 8), channels 32 j + 8 q4 + (0 .. 7); read before the first
    // copies are asked for (those wait for the page ids), used after
    uint32_t bq[NT][KW][4];
    float fr[NT][2], qs[NT][2][NG];
    uint4 qraw[NT][KW];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = s_at.rb * R + 8 * nt + g;  // row = (query token rr / G, head rr % G)
      const bool live = rr < s_at.n * p.G;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        qraw[nt][j] = make_uint4(0, 0, 0, 0);
        if (live)
          qraw[nt][j] = __ldg(reinterpret_cast<const uint4*>(p.q.data +
                                                             static_cast<int64_t>(s_at.r0 + rr / p.G) * p.q.row_stride +
                                                             (s_at.h * p.G + rr % p.G) * p.q.head_stride + 32 * j) + q4);
      }
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[KW][8];
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        unpack8(qraw[nt][j], p.f16, x[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[j][k]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int E = fp16_exponent(mx);
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
    float o[NT][MT][4], m[NT][2], l[NT][2], om[NT][2][NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < MT; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = kNoMax;
        l[nt][c] = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) om[nt][c][k] = 0.f;
      }
    }
    float wf = 0.f;  // weight factor 2^Ev, lowered when a scale times it exceeds kWeightRoom; 0: none yet

    uint32_t stage = 0;
    for (; tile < tile_end; tile += kWarps) {
      cp_async_wait_group<kStages - 2>();
      __syncwarp();  // this step's copies of every lane have landed, and the stage before it is read
      issue();
      const uint8_t* const st = ring + stage * Ge::kStage;
      const uint32_t here = present >> (2 * stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if ((here & 3) == 0) continue;  // the same for all lanes
      const bool edge = (here & 3) != 3 || tile < full[0] || tile >= full[1];
#pragma unroll 1
      for (int r0 = 0; r0 < 2; r0 += PT) {
        uint2 num[PT][2][NG];
#pragma unroll
        for (int r = 0; r < PT; ++r) read_numbers<NG>(num[r], st + 2 * Ge::kCodes + (r0 + r) * (kTile * 8 * NG), g);
        if (edge) {  // numbers of tokens behind the sequence, or of no page, are not read as such
#pragma unroll
          for (int r = 0; r < PT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tile * kTok + (r0 + r) * kTile + 8 * e + g >= s_at.T || !((here >> (r0 + r)) & 1))
#pragma unroll
                for (int k = 0; k < NG; ++k) num[r][e][k] = make_uint2(0, 0);
        }
        // ---- scores
        uint32_t kw[PT][2][KW];
#pragma unroll
        for (int r = 0; r < PT; ++r) read_keys<D>(kw[r], st + (r0 + r) * (Ge::kCodes / 2), g, q4);
        float x[PT][NT][4];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          float s[PT][NT][4];
#pragma unroll
          for (int j = k * (KW / NG); j < (k + 1) * (KW / NG); ++j) {
            uint32_t a01[PT][4], a23[PT][4];
#pragma unroll
            for (int r = 0; r < PT; ++r) {
              const uint32_t u0 = kw[r][0][j], u1 = kw[r][1][j], v0 = u0 >> 8, v1 = u1 >> 8;
              a01[r][0] = u0 & 0x000F000Fu, a01[r][1] = u1 & 0x000F000Fu, a01[r][2] = u0 & 0x00F000F0u, a01[r][3] = u1 & 0x00F000F0u;
              a23[r][0] = v0 & 0x000F000Fu, a23[r][1] = v1 & 0x000F000Fu, a23[r][2] = v0 & 0x00F000F0u, a23[r][3] = v1 & 0x00F000F0u;
            }
#pragma unroll
            for (int r = 0; r < PT; ++r)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (j == k * (KW / NG)) mma_f16_16816_z(s[r][nt], a01[r], bq[nt][j][0], bq[nt][j][1]);
                else mma_f16_16816(s[r][nt], a01[r], bq[nt][j][0], bq[nt][j][1]);
              }
#pragma unroll
            for (int r = 0; r < PT; ++r)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[r][nt], a23[r], bq[nt][j][2], bq[nt][j][3]);
          }
#pragma unroll
          for (int r = 0; r < PT; ++r) {
            const float2 k0 = half2_to_float2(num[r][0][k].x), k1 = half2_to_float2(num[r][1][k].x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float m0 = k0.y * qs[nt][c][k], m1 = k1.y * qs[nt][c][k];
                x[r][nt][c] = (k == 0 ? m0 : x[r][nt][c] + m0) + k0.x * (fr[nt][c] * s[r][nt][c]);
                x[r][nt][2 + c] = (k == 0 ? m1 : x[r][nt][2 + c] + m1) + k1.x * (fr[nt][c] * s[r][nt][2 + c]);
              }
          }
        }
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int rr = s_at.rb * R + 8 * nt + 2 * q4 + c;
              const int2 v = rr < s_at.n * p.G ? visible(p, s_at.T, s_at.n, rr / p.G) : make_int2(0, 0);
#pragma unroll
              for (int r = 0; r < PT; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int t = tile * kTok + (r0 + r) * kTile + 8 * e + g;
                  if (t < v.x || t >= v.y || !((here >> (r0 + r)) & 1)) x[r][nt][2 * e + c] = -INFINITY;
                }
            }
        }
        // ---- running max and weight factor, raised rarely
        float vs = 0.f;
#pragma unroll
        for (int r = 0; r < PT; ++r)
#pragma unroll
          for (int k = 0; k < NG; ++k)
            vs = fmaxf(vs, fmaxf(half2_to_float2(num[r][0][k].y).x, half2_to_float2(num[r][1][k].y).x));
        float top[NT][2];
        bool raise = vs * wf > kWeightRoom;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            top[nt][c] = fmaxf(x[0][nt][c], x[0][nt][2 + c]);
            if constexpr (PT == 2) top[nt][c] = fmaxf(top[nt][c], fmaxf(x[PT - 1][nt][c], x[PT - 1][nt][2 + c]));
            raise |= top[nt][c] > m[nt][c] + kSlack;
          }
        if (__any_sync(0xffffffffu, raise)) {
          float wr = 1.f;
          vs = max_over_g(vs);
          if (wf == 0.f || vs * wf > kWeightRoom) {  // 2^Ev vs in [16, 32): room upwards, and far down before FP16 ends
            const int e = vs > 0.f ? max(-24, static_cast<int>(__float_as_uint(vs) >> 23) - 127) : -24;
            const float f = pow2_int(4 - e);
            wr = wf > 0.f ? f / wf : 1.f;
            wf = f;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float sc[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float mn = fmaxf(m[nt][c], max_over_g(top[nt][c]));
              sc[c] = ex2(m[nt][c] - mn);
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
        const float mid = wf > 0.f ? 7.5f * __uint_as_float(0x7F000000u - __float_as_uint(wf)) : 0.f;  // 7.5 / wf, a power of two
        uint32_t bw[PT][NT][NG][2];
#pragma unroll
        for (int r = 0; r < PT; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              w[c] = ex2(x[r][nt][c] - m[nt][c]);
              w[2 + c] = ex2(x[r][nt][2 + c] - m[nt][c]);
              l[nt][c] += w[c] + w[2 + c];
            }
#pragma unroll
            for (int k = 0; k < NG; ++k) {
              const float2 v0 = half2_to_float2(num[r][0][k].y), v1 = half2_to_float2(num[r][1][k].y);
#pragma unroll
              for (int c = 0; c < 2; ++c) om[nt][c][k] += w[c] * v0.y + w[2 + c] * v1.y;
              const float s0 = v0.x * wf, s1 = v1.x * wf;
              const uint32_t h0 = float2_to_half2(w[0] * s0, w[1] * s0), h1 = float2_to_half2(w[2] * s1, w[3] * s1);
              if (p.f16) {  // codes are about 7.5 from zero, values are not: the weights' rounding errors times 7.5 are put back
                const float2 r0 = half2_to_float2(h0), r1 = half2_to_float2(h1);
                om[nt][0][k] += mid * (fmaf(w[0], s0, -r0.x) + fmaf(w[2], s1, -r1.x));
                om[nt][1][k] += mid * (fmaf(w[1], s0, -r0.y) + fmaf(w[3], s1, -r1.y));
              }
              bw[r][nt][k][0] = movmatrix_t(h0);
              bw[r][nt][k][1] = movmatrix_t(h1);
            }
          }
        // ---- readout
#pragma unroll
        for (int r = 0; r < PT; ++r) {
          no_loads_across();
          uint32_t vw[4][VW];
          read_values<D>(vw, st + Ge::kCodes + (r0 + r) * (Ge::kCodes / 2), g, q4);
#pragma unroll
          for (int u = 0; u < VW; ++u) {
            const uint32_t p0 = prmt(vw[0][u], vw[1][u], 0x5410), p1 = prmt(vw[0][u], vw[1][u], 0x7632);
            const uint32_t p2 = prmt(vw[2][u], vw[3][u], 0x5410), p3 = prmt(vw[2][u], vw[3][u], 0x7632);
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const int sh = 8 * hi;
              const uint32_t w0 = p0 >> sh, w1 = p1 >> sh, w2 = p2 >> sh, w3 = p3 >> sh;
              const uint32_t a0w[4] = {w0 & 0x000F000Fu, w1 & 0x000F000Fu, w2 & 0x000F000Fu, w3 & 0x000F000Fu};
              const uint32_t a1w[4] = {w0 & 0x00F000F0u, w1 & 0x00F000F0u, w2 & 0x00F000F0u, w3 & 0x00F000F0u};
              const int j = 4 * u + 2 * hi;
              constexpr int kPer = MT / NG;  // 16-channel blocks per group
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(o[nt][j], a0w, bw[r][nt][j / kPer][0], bw[r][nt][j / kPer][1]);
                mma_f16_16816(o[nt][j + 1], a1w, bw[r][nt][(j + 1) / kPer][0], bw[r][nt][(j + 1) / kPer][1]);
              }
            }
          }
        }
      }
    }
    cp_async_wait_group<0>();
    __syncwarp();

    // ---- the warps of the CTA meet: a common max per row, then each leaves its scaled sums
    const float undo = wf > 0.f ? 16777216.f / wf : 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] = sum_over_g(l[nt][c]);
#pragma unroll
        for (int k = 0; k < NG; ++k) om[nt][c][k] = sum_over_g(om[nt][c][k]);
        if (g == 0) s_m[warp][8 * nt + 2 * q4 + c] = m[nt][c], s_l[warp][8 * nt + 2 * q4 + c] = l[nt][c];
      }
    __syncthreads();
    float(*const mine_o)[kRowPad] = reinterpret_cast<float(*)[kRowPad]>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * nt + 2 * q4 + c;
        float M = m[nt][c];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][row]);
        const float f = ex2(m[nt][c] - M), fo = f * undo;
#pragma unroll
        for (int k = 0; k < NG; ++k) om[nt][c][k] *= f;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float fj = (j & 1) ? fo * 0.0625f : fo;
          mine_o[row][16 * j + g] = o[nt][j][c] * fj + om[nt][c][j / (MT / NG)];
          mine_o[row][16 * j + 8 + g] = o[nt][j][2 + c] * fj + om[nt][c][j / (MT / NG)];
        }
      }
    if (tid < R) {
      float M = kNoMax, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L += ex2(s_m[w][tid] - M) * s_l[w][tid];
      s_ml[tid][0] = M, s_ml[tid][1] = L;
    }
    __syncthreads();
    const bool whole = s_at.parts == 1;
    // partial slots: 2 c for an item that CTA c goes on with, 2 c + 1 for one that it begins
    const int slot = 2 * static_cast<int>(blockIdx.x) + (s_at.a0 == 0 ? 1 : 0);
    for (int e = tid; e < R * D / 4; e += kThreads) {
      const int row = e / (D / 4), c4 = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(smem + w * Ge::kRing + (row * kRowPad + 4 * c4) * 4);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      if (whole) {
        store_out<D, R>(p, s_at, row, c4, v, s_ml[row][0], s_ml[row][1]);
      } else {
        reinterpret_cast<float4*>(p.part_o + (static_cast<size_t>(slot) * R + row) * D)[c4] = v;
        if (c4 == 0)
          reinterpret_cast<float2*>(p.part_ml)[static_cast<size_t>(slot) * R + row] = make_float2(s_ml[row][0], s_ml[row][1]);
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_last = atomicAdd(p.arrive + s_at.c0, 1u) == static_cast<uint32_t>(s_at.parts - 1);
        if (s_last) {
          p.arrive[s_at.c0] = 0;
          __threadfence();
        }
      }
      __syncthreads();
      if (s_last) merge_parts<D, R, kThreads>(p, s_at, smem, Ge::kSmem, s_f, s_ml);
    }
    __syncthreads();

    // ---- the next item on the line
    if (tid == 0) {
      Place& s = s_at;
      if (s.at < s.end) s.at = min(s.end, s.item0 + s.tiles);
      if (s.at < s.end) {
        s.item0 = s.at;
        if (++s.rb == s.blocks) {
          s.rb = 0;
          if (++s.h == p.Hkv) {
            s.h = 0;
            int ignore = 0;
            do {
              if (++s.b >= p.B) {  // lengths that changed under the call
                s.at = s.end;
                break;
              }
              sequence<R>(p, s.b, s.T, s.n, s.r0, s.tiles, s.blocks, ignore);
            } while (s.blocks == 0);
          }
        }
        on_line(s);
      }
    }
    __syncthreads();
    if (s_at.at >= s_at.end) break;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && flags) atomicOr(p.err, flags);
}

template <int D, int NG, int NT>
cudaError_t launch_rows(const Kv4AttnParams& p, int ctas, cudaStream_t stream) {
  using Ge = Geom<D, NG, NT>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kv4_decode_kernel<D, NG, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ge::kSmem);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  kv4_decode_kernel<D, NG, NT><<<ctas, Ge::kThreads, Ge::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int NG>
cudaError_t launch(const Kv4AttnParams& p, int rows, int ctas, cudaStream_t stream) {
  return rows == 8 ? launch_rows<D, NG, 1>(p, ctas, stream) : launch_rows<D, NG, 2>(p, ctas, stream);
}

}  // namespace

int kv4_decode_rows(int max_q, int G) { return static_cast<int64_t>(max_q) * G <= 8 ? 8 : 16; }
int kv4_decode_ctas(int num_sms) { return std::min(2 * num_sms, static_cast<int>(kKv4CounterBytes / 4)); }
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms) {
  const size_t ctas = kv4_decode_ctas(num_sms);
  return kKv4CounterBytes + 2 * ctas * rows * (static_cast<size_t>(D) + 2) * sizeof(float);
}

cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  const int rows = kv4_decode_rows(p.max_q, p.G), ctas = kv4_decode_ctas(num_sms);
  if (D == 128) {
    if (n_groups == 1) return launch<128, 1>(p, rows, ctas, stream);
    if (n_groups == 2) return launch<128, 2>(p, rows, ctas, stream);
    return launch<128, 4>(p, rows, ctas, stream);
  }
  return n_groups == 1 ? launch<64, 1>(p, rows, ctas, stream) : launch<64, 2>(p, rows, ctas, stream);
}

}  // namespace mlaq
