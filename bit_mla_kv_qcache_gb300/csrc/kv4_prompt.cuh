// Attention over the grouped-query cache in 4 bits for many query rows per kv head (chunks of a
// prompt, several drafted tokens of many heads), on the fifth-generation tensor cores. Rows = (query
// token, head of the group), 128 to a tile of queries.
//
// One CTA per SM, 16 warps. Per tile of 128 cached tokens:
//   unpacking    one token per thread: the token's codes become FP16 values min + code * scale (one
//                rounding) in shared memory, keys and values, two stages each;
//   warp 12      one lane issues S = Q K^T (128 rows x 128 tokens, both operands in shared memory)
//                and O += P V (P from tensor memory);
//   warp 13      asks for the codes of later tiles in L2 or copies them to shared memory, a lane per page;
//   softmax      one row per thread: S is read from tensor memory once (its maximum, then the weights), P
//                replaces it there as FP16, handed over in two halves. The running max is raised,
//                and O rescaled in place, only when a score exceeds it by more than 2^8.
// The softmax groups take the registers that the others give up (setmaxnreg), so every role has its own
// loop over the CTA's work. The kernel exists in two forms:
//   two tiles of queries (more than 128 rows): two softmax groups of four warps, which alternate so that the
//     tensor cores work for one while the other takes its softmax; warps 8-11 unpack keys and values, loaded into
//     registers a tile ahead. Against one tile of queries per CTA: 649 and 1004 us (two chunks of 4K, the second of each
//     prompt, 32 heads on 8, D = 128), 133 and 143 us (256 rows of eight sequences up to 32K).
//   one tile: warps 0-3 take the softmax of every token tile, 4-7 unpack values, 8-11 keys, from copies of the pages
//     in shared memory, two tiles ahead (loaded into registers: 93 us for 40 rows of eight sequences up to 32K, copied
//     82). With at most 64 rows the tile holds them twice: one twin takes the first 64 tokens of a token tile, the
//     other the rest, and their sums join at the end (84 us without the twins, 80 with; 64 rows 86 and 83). Queries lie in
//     tensor memory, so that a score product reads keys alone from shared memory, which is busy with the unpacked tiles, and the
//     values' group unpacks the last quarter of the keys (16 nodes of 64 sequences of 8K, 32 heads on 8, D = 128: 399 us,
//     with the first 360, the second 371, both 343; 16 sequences of 32K 355, 310, 321 and 289; 40 rows 80.5 and 78.5). The
//     products then set the pace: 25 of ~70 cycles to a token tile.
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D each; one tile: the queries in place of O1). A step's S overwrites the P of two steps
// before; products of one thread run in the order of their issue.
//
// Channels keep the order in which a code word unpacks: eight channels of a word in the order 0 4 1 5
// 2 6 3 7, for keys matched by the queries, for values undone when a row is stored.
//
// kExact (the rounding of a key to FP16, up to 2^-11 of it, shows in the log-sum-exp as
// ~1e-4): scores from exact products. With the scale s = s1 + s2 cut after seven bits, n s1 and n s2 fit FP16
// for every code n: two key operands. (From 4096 on 15 s1 would not: such a token's numbers are quartered and its
// scores taken four times. Smaller numbers stay as they are, subnormal ones too: quartered, FP16 would drop their last
// bits.) The minimum enters as sixteen more channels: its value for each
// group against the sum of the group's queries, in two FP16 parts. One stage of keys then has the room; its halves
// (of the channels) fill and empty one by one. Taken when the log-sum-exp is asked for, and always with one tile of queries
// of 128 channels, where it costs little (40 rows: 81 us, rounded keys 79), and beside weights in two parts (kSplit).
//
// Work: one CTA per item (sequence, kv head, row block), those that see the most tokens first (of trees the longest
// sequences, up to 512 of them: 16 nodes of 64 sequences up to 8K 254 us in the order given, 231 by length); or items cut
// over the SMs (see kv4_prompt_plan), so that every SM has one part of one item, or, where the parts do
// not fit, laid on one line and cut evenly (as in the kernel for few rows). A launch of its own joins the parts.
//
// Bound: the chain of a group's tile: S, its way to the registers, exponentials, P V. Two chunks of 4K over 8K (824
// GFLOP) take 648 us where the card's rate for large BF16 products gives 424: the tensor pipe is 47% busy, issue 45%; tensor memory
// is full at D = 128, so a group's next S waits for its P V. 40 rows of eight sequences up to 32K: 78.5 us, 16 for their bytes: per
// token tile of ~2.5 k cycles 25 products take 1.7 k.
//
// kTree: as in the kernel for few rows; a row's bits of 32 tokens are read at the tiles of the tree alone.
// kSplit, for trees with FP16 outputs: weights enter in two FP16 parts, the second in the columns of S that the first leaves free: what is
// rounded off them counts as much as the output's own rounding (error of the output 3.4e-4 -> 2.8e-4 of it, of which that is
// 2.1e-4; 16 nodes of 64 sequences up to 8K 239 -> 254 us).
#pragma once
#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "append.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "kv4_tree.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 512;
// registers by role; over the four groups of 128 threads they come to the 512 of the launch
template <bool two>
struct Regs {  // two: one group unpacks, else two groups do
  static constexpr int softmax = 184, unpack = two ? 96 : 120, issue = two ? 48 : 88;
};
constexpr int kAhead = 3;         // tiles that warp 13 runs ahead
constexpr int kTok = 128;         // tokens per tile
constexpr int kMaxParts = 32;     // CTAs that one item is cut into, at most
constexpr int kStart = 6;         // tiles' worth of time that an item costs besides its tiles: queries, first tiles, results
constexpr float kSlack = 8.f;     // the running max is raised when a score exceeds it by more than this
constexpr float kNoMax = -1e30f;  // the running max before the first score
// Weights carry a factor of 2^kRoom, and so do their sums: at most 2^15 in FP16, and those below its smallest normal
// number off by at most 2^-32 of the weight at the running max (one token 17.4 nats above 16383 others: their
// share of the output, 4.5e-4, is off by 3e-6; without the factor it is lost).
constexpr float kRoom = 7.f;
constexpr long long kBudget = 4ll << 30;  // cycles of a wait before it is given up

// Shared memory in tiles of 128 x D FP16: queries (one or two tiles), keys (two stages, or two operands),
// values (two stages); kExact: the sixteen further channels of each tile of queries, and of the keys.
template <int D, int NG, bool kExact>
struct Geom {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kMore = kExact ? 128 * 16 * 2 : 0;
  static constexpr uint32_t kColS = 0, kColO = 256, kColQ = kColO + D;
  __host__ __device__ static constexpr int k_at(bool two) { return (two ? 2 : 1) * kTile; }
  __host__ __device__ static constexpr int v_at(bool two) { return k_at(two) + 2 * kTile; }
  __host__ __device__ static constexpr int more_q_at(bool two) { return v_at(two) + 2 * kTile; }
  __host__ __device__ static constexpr int more_k_at(bool two) { return more_q_at(two) + (two ? 2 : 1) * kMore; }
  __host__ __device__ static constexpr int ring_at(bool two) { return more_k_at(two) + kMore; }
  // one tile of queries: codes and numbers of two token tiles as they lie in the pages (key codes, value codes, numbers)
  static constexpr int kCodes = kTok * D / 2, kStage = 2 * kCodes + kTok * 8 * NG;
  __host__ __device__ static constexpr int smem(bool two) { return ring_at(two) + (two ? 0 : 2 * kStage) + 1024; }  // slack to align the start
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_shared_v2(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// (a, b) * (f, f) + (c, c) in one instruction
__device__ __forceinline__ void fma_pair(float& a, float& b, float f, float c) {
  asm("{ .reg .b64 x, f, c; mov.b64 x, {%0, %1}; mov.b64 f, {%2, %2}; mov.b64 c, {%3, %3}; fma.rn.f32x2 x, x, f, c;"
      " mov.b64 {%0, %1}, x; }"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(c));
}
__device__ __forceinline__ void add_pair(float& a, float& b, float x, float y) {
  asm("{ .reg .b64 u, v; mov.b64 u, {%0, %1}; mov.b64 v, {%2, %3}; add.rn.f32x2 u, u, v; mov.b64 {%0, %1}, u; }"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
__device__ __forceinline__ void bulk_prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void softmax_barrier(int threads) { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

// The two codes at bits 0-3 (kHigh: 4-7) of the halves of w as min + code * scale: 1024 + n (1024 + 16 n)
// is put together by bits, n comes out exactly, then one rounding.
template <bool kHigh>
__device__ __forceinline__ uint32_t dequant2(uint32_t w, __half2 s, __half2 m) {
  const uint32_t b = and_or(w, kHigh ? 0x00F000F0u : 0x000F000Fu, 0x64006400u);
  const __half2 x = *reinterpret_cast<const __half2*>(&b);
  const __half2 n = kHigh ? __hfma2(x, __float2half2_rn(0.0625f), __float2half2_rn(-64.f))
                          : __hadd2(x, __float2half2_rn(-1024.f));
  const __half2 v = __hfma2(n, s, m);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The codes of the same pair, times two factors (exact: see kExact).
template <bool kHigh>
__device__ __forceinline__ void codes2_times(uint32_t w, __half2 s1, __half2 s2, uint32_t& y1, uint32_t& y2) {
  const uint32_t b = and_or(w, kHigh ? 0x00F000F0u : 0x000F000Fu, 0x64006400u);
  const __half2 x = *reinterpret_cast<const __half2*>(&b);
  const __half2 n = kHigh ? __hfma2(x, __float2half2_rn(0.0625f), __float2half2_rn(-64.f))
                          : __hadd2(x, __float2half2_rn(-1024.f));
  const __half2 a = __hmul2(n, s1), c = __hmul2(n, s2);
  y1 = *reinterpret_cast<const uint32_t*>(&a);
  y2 = *reinterpret_cast<const uint32_t*>(&c);
}

// The part of an item that the CTA works on.
struct Seg {
  int b, h, rb;          // sequence, kv head, row block
  int T, n, r0;          // of the sequence: length, query rows, first row
  int base;              // kTree: tokens before the tree
  int tile, tiles;       // first token tile here, and how many
  int part, c0, parts;   // slot of the partial result, or -1 (the item is whole here); CTAs of the item
  int valid;
  // line mode: position, end of the CTA's stretch, the item's first tile and its tiles, CTA stretch, (b, rb) pair
  long long at, end, item0, share;
  int item_tiles, pair;
};

template <bool kTree>
__device__ __forceinline__ void load_sequence(const Kv4AttnParams& p, int b, int& T, int& n, int& r0, int& base, int& flags) {
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
  if constexpr (kTree) base = tree_base(p, b, T, n, flags);
}

// Tokens that query row i of the sequence sees: [lo, hi).
__device__ __forceinline__ int2 visible(const Kv4AttnParams& p, int T, int n, int i) {
  const int pos = T - n + i;
  const int hi = p.causal ? max(0, min(T, pos + 1)) : T;
  const int lo = p.window && pos >= p.window ? pos - p.window + 1 : 0;  // no overflow before the first token
  return make_int2(lo, hi);
}

// Tokens that some row of row block rb may see: [x, y).
template <bool kTree>
__device__ __forceinline__ int2 block_tokens(const Kv4AttnParams& p, int T, int n, int base, int rb, int R) {
  if constexpr (kTree) return tree_tokens(p, T, base);
  const int i0 = rb * R / p.G, i1 = min(n - 1, (rb * R + R - 1) / p.G);  // rows * G < 2^31
  return make_int2(visible(p, T, n, i0).x, visible(p, T, n, i1).y);
}
// First token tile of row block rb and the number of tiles (at least one, to store rows that see nothing).
template <bool kTree>
__device__ __forceinline__ int2 block_tiles(const Kv4AttnParams& p, int T, int n, int base, int rb, int R) {
  const int2 seen = block_tokens<kTree>(p, T, n, base, rb, R);
  const int t0 = seen.x / kTok, t1 = (seen.y + kTok - 1) / kTok;
  return make_int2(t0, max(1, t1 - t0));
}
__device__ __forceinline__ int row_blocks(const Kv4AttnParams& p, int n, int R) { return (n * p.G + R - 1) / R; }

// Line mode: the segment that starts at s.at (b, h, rb and the sequence are set). An item takes its tiles and kStart more
// places of the line.
template <bool kTree>
__device__ __forceinline__ void line_segment(const Kv4AttnParams& p, Seg& s, int R) {
  const int2 t = block_tiles<kTree>(p, s.T, s.n, s.base, s.rb, R);
  s.item_tiles = t.y;
  const int a0 = static_cast<int>(s.at - s.item0);
  const int a1 = static_cast<int>(min(s.end - s.item0, static_cast<long long>(t.y)));
  s.tile = t.x + a0;
  s.tiles = a1 - a0;
  s.c0 = static_cast<int>(s.item0 / s.share);
  s.parts = static_cast<int>((s.item0 + t.y - 1) / s.share) - s.c0 + 1;
  s.part = s.parts == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (a0 == 0 ? 1 : 0);
  s.valid = 1;
}

// Line mode: goes on to the item at s.at, the next head or row block (`line` of them per sequence) or sequence.
template <bool kTree>
__device__ __forceinline__ void next_item(const Kv4AttnParams& p, Seg& s, int line, int R) {
  s.valid = 0;
  if (s.at >= s.end) return;
  s.item0 = s.at;
  if (++s.h == p.Hkv) {  // the next pair with rows
    s.h = 0;
    int f = 0;
    do {
      if (++s.pair >= p.B * line) return;  // lengths that changed under the call
      s.b = s.pair / line;
      s.rb = s.pair - s.b * line;
      load_sequence<kTree>(p, s.b, s.T, s.n, s.r0, s.base, f);
    } while (s.rb >= row_blocks(p, s.n, R));
  }
  line_segment<kTree>(p, s, R);
}

template <int D, int NG, bool kExact, bool two, bool kTree, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(const Kv4AttnParams p, const int rows, const int line) {
  using Ge = Geom<D, NG, kExact>;
  constexpr int KW = D / 32, VW = D / 64, CB = D / 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[19];  // k_full[2] k_free[2] v_full[2] v_free[2] s_full[2] p_ready[2] o_done c_full[2] c_free[2]
  __shared__ uint32_t s_tmem;
  __shared__ Seg s_seg, s_next;  // here, and the one after it
  __shared__ long long s_part[kThreads / 32];
  __shared__ int s_most[kThreads / 32];
  __shared__ Kv4Joined s_joined;  // the item that the CTA begins and others go on with
  __shared__ float2 s_side[kTok];  // max and sum of a row under half of the tokens
  constexpr int kTry = 9;
  __shared__ int s_count[kTry + 1];  // parts that a share would make; tiles in all
  __shared__ volatile int s_abort, s_any_odd;  // s_any_odd: a bit of s_hidden or s_large has been set
  __shared__ volatile uint32_t s_unpacked;  // two tiles of queries: token tiles that warp 8 has unpacked so far
  __shared__ uint32_t s_bad_pages[2];  // of a stage of codes: bit i, its i-th page
  __shared__ __align__(16) uint32_t s_hidden[4][4];  // tokens of a tile (modulo four) whose page id is bad
  __shared__ __align__(16) uint32_t s_large[4][4];   // kExact: tokens of a tile whose scale and minimum are quartered
  uint64_t *const k_full = bars, *const k_free = bars + 2, *const v_full = bars + 4, *const v_free = bars + 6,
           *const s_full = bars + 8, *const p_ready = bars + 10, *const o_done = bars + 12, *const c_full = bars + 13, *const c_free = bars + 15, *const p_half = bars + 17;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
  long long* const s_sum = reinterpret_cast<long long*>(smem);  // tiles before each pair, until the first queries come
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = two ? 256 : rows;
  const bool half = R == 64;
  const uint32_t k_tiles = base + Ge::k_at(two), v_tiles = base + Ge::v_at(two);
  int flags = 0;

  if (warp == 12) tc5::alloc512(&s_tmem);
  if (tid == 0) s_joined = Kv4Joined{};
  // ---- which part of which item
  if (!line) {
    const int per = p.B * p.Hkv, blocks = static_cast<int>(gridDim.x) / per;
    if constexpr (kTree) {  // the longest sequences first: a node sees as much of its sequence as any other
      const int bh = static_cast<int>(blockIdx.x) / p.Hkv;
      if (tid == 0) {
        s_seg.h = static_cast<int>(blockIdx.x) % p.Hkv;
        s_seg.rb = bh % blocks;
        s_seg.b = bh / blocks;
      }
      if (p.B > 1 && p.B <= kThreads) {
        int* const lens = reinterpret_cast<int*>(smem);
        const int mine = tid < p.B ? __ldg(p.seq_lens + tid) : 0;
        lens[tid] = mine;
        __syncthreads();
        int before = 0;
#pragma unroll 4
        for (int b = 0; b < p.B; ++b) before += lens[b] > mine || (lens[b] == mine && b < tid);
        if (tid < p.B && before == bh / blocks) s_seg.b = tid;
        __syncthreads();
      }
    }
    if (tid == 0) {
      Seg& s = s_seg;
      const int bh = static_cast<int>(blockIdx.x) % per;
      if constexpr (!kTree) {
        s.rb = blocks - 1 - static_cast<int>(blockIdx.x) / per;
        s.b = bh / p.Hkv;
        s.h = bh % p.Hkv;
      }
      int f = 0;
      load_sequence<kTree>(p, s.b, s.T, s.n, s.r0, s.base, f);
      flags |= f;
      s.valid = s.rb < row_blocks(p, s.n, R);
      s.part = -1;
      s.parts = 1;
      if (s.valid) {
        const int2 t = block_tiles<kTree>(p, s.T, s.n, s.base, s.rb, R);
        s.tile = t.x;
        s.tiles = t.y;
      }
    }
  } else {
    const int blocks_most = line;  // row blocks of the longest sequence
    const int pairs = p.B * blocks_most;  // (sequence, row block), in order; a pair's heads in a row
    // Thread or lane i looks at pair i: its tiles, and its places on the line.
    auto look = [&](int i, int& t) -> long long {
      t = 0;
      if (i >= pairs) return 0;
      int T, n, r0, base_ = 0, f = 0;
      const int b = i / blocks_most, rb = i - b * blocks_most;
      load_sequence<kTree>(p, b, T, n, r0, base_, f);
      if (blockIdx.x == 0) flags |= f;
      if (rb < row_blocks(p, n, R)) t = block_tiles<kTree>(p, T, n, base_, rb, R).y;
      return t > 0 ? static_cast<long long>(t + kStart) * p.Hkv : 0;
    };
    // fewest tiles of a part; items of fewer than 2048 tokens stay whole
    auto least_of = [](int most) { return most < 2048 / kTok ? max(1, most) : max(4, (most + kMaxParts - 2) / (kMaxParts - 1)); };
    // shares for which every part could have a CTA of its own: the smallest of a few multiples of the mean, or
    // items uncut where the longest is little more than the line's stretch
    auto share_of = [&](int k, int most, int least, int tiles, long long total) {
      const float mean = static_cast<float>(tiles) / static_cast<float>(gridDim.x);
      const float stretch = static_cast<float>(total) / static_cast<float>(gridDim.x);
      const bool uncut = most + kStart <= 1.2f * (stretch + kStart);
      return k == kTry - 1 && uncut ? max(1, most) : max(least, static_cast<int>(mean * (1.f + 0.12f * k)) + 1);
    };
    // What lies at the CTA's place: pair `lo`, whose places begin at `before`. share > 0: parts of one CTA each; else stretches of the line.
    auto locate = [&](Seg& s, int share, int lo, long long before) {
      int f = 0;
      s.pair = lo;
      s.b = lo / blocks_most;
      s.rb = lo - s.b * blocks_most;
      load_sequence<kTree>(p, s.b, s.T, s.n, s.r0, s.base, f);
      if (s.rb >= row_blocks(p, s.n, R)) return;  // the lengths changed under the call
      const int2 tiles = block_tiles<kTree>(p, s.T, s.n, s.base, s.rb, R);
      const int at = static_cast<int>(s.at - before);
      if (share > 0) {
        const int parts = (tiles.y + share - 1) / share, part = at % parts;
        s.h = min(at / parts, p.Hkv - 1);
        s.tile = tiles.x + tiles.y * part / parts;
        s.tiles = tiles.x + tiles.y * (part + 1) / parts - s.tile;
        s.parts = parts;
        s.c0 = static_cast<int>(blockIdx.x) - part;
        s.part = parts == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (part == 0 ? 1 : 0);
        s.valid = 1;
        s.item0 = s.end = s.at;  // and nothing after it
        s.item_tiles = tiles.y;
      } else {
        s.h = min(at / (tiles.y + kStart), p.Hkv - 1);
        s.item0 = before + static_cast<long long>(s.h) * (tiles.y + kStart);
        if (s.at < s.item0 + tiles.y) {
          line_segment<kTree>(p, s, R);
        } else {
          s.at = s.item0 + tiles.y + kStart;
          next_item<kTree>(p, s, line, R);
        }
      }
    };
    if (pairs <= 32) {  // one warp, without the block's barriers (2.9 us to here, by the block 6.4)
      if (warp == 0) {
        int t;
        const long long x = look(lane, t);
        auto scan = [&](long long v) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
          }
          return v;
        };
        const int most = __reduce_max_sync(0xffffffffu, t), least = least_of(most);
        long long upto = scan(x);
        const long long total = __shfl_sync(0xffffffffu, upto, 31);
        const bool small = total < (1 << 24);
        const int tiles = __reduce_add_sync(0xffffffffu, small ? p.Hkv * t : 0);
        int share = 0;
#pragma unroll 1
        for (int k = 0; k < kTry && share == 0 && small; ++k) {
          const int sh = share_of(k, most, least, tiles, total);
          if (__reduce_add_sync(0xffffffffu, p.Hkv * ((t + sh - 1) / sh)) <= static_cast<int>(gridDim.x)) share = sh;
        }
        long long mine = x, places = total;
        if (share > 0) {
          mine = p.Hkv * ((t + share - 1) / share);
          upto = scan(mine);
          places = __shfl_sync(0xffffffffu, upto, 31);
        }
        Seg& s = s_seg;
        if (lane == 0) {
          s.share = share > 0 ? 1 : max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(least));
          s.at = s.share * blockIdx.x;
          s.end = min(places, s.at + s.share);
          s.valid = 0;
        }
        __syncwarp();
        const long long at = s.at;
        if (at < s.end && at >= upto - mine && at < upto) locate(s, share, lane, upto - mine);  // one lane
        __syncwarp();
      }
    } else {
      int t;
      long long x = look(tid, t);
      const int warp_most = __reduce_max_sync(0xffffffffu, t);
      auto scan = [&](long long v) {  // inclusive, over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        if (lane == 31) s_part[warp] = v;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < warp; ++w) v += s_part[w];
        return v;
      };
      if (lane == 0) s_most[warp] = warp_most;
      if (tid <= kTry) s_count[tid] = 0;
      x = scan(x);
      s_sum[tid + 1] = x;
      if (tid == 0) s_sum[0] = 0;
      __syncthreads();
      int most = 0;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) most = max(most, s_most[w]);
      const long long total = s_sum[kThreads];
      const int least = least_of(most);
      const bool small = total < (1 << 24);
      const int tiles_here = __reduce_add_sync(0xffffffffu, small ? p.Hkv * t : 0);
      if (lane == 0) atomicAdd(&s_count[kTry], tiles_here);
      __syncthreads();
      const int tiles = s_count[kTry];
#pragma unroll 1
      for (int k = 0; k < kTry; ++k) {
        const int sh = share_of(k, most, least, tiles, total);
        const int parts = __reduce_add_sync(0xffffffffu, small ? p.Hkv * ((t + sh - 1) / sh) : 1 << 20);
        if (lane == 0) atomicAdd(&s_count[k], parts);
      }
      __syncthreads();
      int share = 0;
#pragma unroll 1
      for (int k = 0; k < kTry && share == 0; ++k)
        if (s_count[k] <= static_cast<int>(gridDim.x)) share = share_of(k, most, least, tiles, total);
      if (share > 0) {  // the parts before each pair
        x = scan(p.Hkv * ((t + share - 1) / share));
        __syncthreads();
        s_sum[tid + 1] = x;
        __syncthreads();
      }
      if (tid == 0) {
        Seg& s = s_seg;
        s.share = share > 0 ? 1 : max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(least));
        s.at = s.share * blockIdx.x;
        s.end = min(s_sum[kThreads], s.at + s.share);
        s.valid = 0;
        if (s.at < s.end) {
          int lo = 0, hi = kThreads - 1;  // s_sum[lo] <= at < s_sum[lo + 1]
#pragma unroll 1
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_sum[mid + 1] > s.at) hi = mid;
            else lo = mid + 1;
          }
          locate(s, share, lo, s_sum[lo]);
        }
      }
    }
  }
  if (tid == 0) {
    s_abort = 0;
    s_any_odd = 0;
    s_unpacked = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, !two && kExact && D == 128 && i == 1 ? 8 : 4);  // one arrival per warp
      mbar_init(v_full + i, 4);
      mbar_init(p_ready + i, 4);
      mbar_init(p_half + i, 4);
      mbar_init(k_free + i, 1);
      mbar_init(v_free + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(c_full + i, 1);
      mbar_init(c_free + i, 8);
    }
    mbar_init(o_done, 1);
    fence_mbar_init();
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (!s_seg.valid) {
    if (line && tid == 0) p.joined[blockIdx.x] = Kv4Joined{};
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && flags) atomicOr(p.err, flags);
    tc5::fence_before();
    __syncthreads();
    if (warp == 12) tc5::dealloc512(s_tmem);
    return;
  }
  const uint32_t tmem = s_tmem;

  // A wait that runs out raises the abort flag, which ends every other wait too. Threads go on all the
  // same (on whatever is there, within their buffers) and leave their loop together, by the flag, which is
  // looked at where it costs nothing; only the warp that issues products asks whether the wait was done.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
      if (s_abort) return false;
      if (clock64() - t0 > kBudget) {
        s_abort = 1;
        flags |= kErrTimeout;
        return false;
      }
    }
    return true;
  };
  auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  auto any = [](bool x) { return __any_sync(0xffffffffu, x) != 0; };
  // Stages and barrier phases go on from segment to segment: token tiles and steps of the earlier ones.
  uint32_t tiles_done = 0, steps_done[2] = {0, 0}, segs = 0;
  const int group = warp >> 2;  // 0, 1: softmax; 2: unpacking; 3: products, prefetch
  const Seg& sg = s_seg;
  auto steps_of = [&]() { return two ? 2 * sg.tiles : sg.tiles; };  // step s: S buffer s & 1, token tile two ? s / 2 : s
  // Two barriers of all warps frame a segment: queries in place; results stored and the next segment set.
  auto leave_segment = [&](int n_tiles, int steps) -> bool {
    __syncthreads();
    if (line) {
      constexpr int kWords = sizeof(Seg) / 4;
      if (tid < kWords) reinterpret_cast<volatile uint32_t*>(&s_seg)[tid] = reinterpret_cast<volatile uint32_t*>(&s_next)[tid];
      __syncthreads();
    }
    tiles_done += n_tiles;
    steps_done[0] += (steps + 1) >> 1;
    steps_done[1] += steps >> 1;
    ++segs;
    return !s_abort && line && sg.valid;
  };
  constexpr bool one_k = kExact;  // one stage of keys
  constexpr bool kTmemQ = !two && !kSplit;  // queries in tensor memory; with weights in two parts it is the busier side (229 us, so 241)

  if (group == 2 || (group == 1 && !two)) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<two>::unpack));
    // ---- unpacking: thread = token of the tile
    const int tok_row = tid & 127;
    const bool keys = group == 2, vals = two || group == 1;
    const uint32_t page_sh = min(p.p_shift, 7);
    constexpr int CH = D / 32;  // 16-byte chunks of a token's codes
    const int rot = two ? 0 : tok_row / (4 / CH * 2);  // lanes take chunks from shared memory in turned orders: distinct banks
    int n_tiles, steps;
    do {
      n_tiles = sg.tiles, steps = steps_of();
      const int tile0 = sg.tile;
      const int2 t_seen = block_tokens<kTree>(p, sg.T, sg.n, sg.base, sg.rb, R);
      const int t_begin = t_seen.x, t_end = t_seen.y;  // pages before the first may be gone (behind a sliding window)
      auto scale_of = [](uint32_t w) { return __ushort_as_half(static_cast<unsigned short>(w)); };
      auto min_of = [](uint32_t w) { return __ushort_as_half(static_cast<unsigned short>(w >> 16)); };
      constexpr int kHalves = one_k ? 2 : 1;  // one stage of keys: its halves (of the channels) fill and empty one by one
      auto key_chunk = [&](int i) { return i / (CH / kHalves) * (CH / kHalves) + ((i + rot) & (CH / kHalves - 1)); };
      constexpr bool kShared = !two && kExact && CH == 4;  // the values' group takes the last chunk of the keys
      auto takes = [&](int i) { return keys ? !kShared || i < CH - 1 : kShared && i == CH - 1; };
      auto value_chunk = [&](int i) { return (i + rot) & (CH - 1); };
      // Two tiles of queries leave no room for codes in shared memory: each thread loads its token's into registers, a
      // tile ahead. With one tile warp 13 copies them.
      const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
      const size_t region = static_cast<size_t>(sg.h) * kv4_head_bytes(D, NG, p.P);
      uint32_t kw[D / 8], vw[D / 8];
      uint2 num[NG], cur[NG];
      auto asked = [&](int j) {  // by its token, not by the id: any may stand in the table
        const int tok = (tile0 + j) * kTok + tok_row;
        return j < n_tiles && tok >= t_begin && tok < t_end;
      };
      auto page_of = [&](int j) -> int32_t { return asked(j) ? __ldg(table + (((tile0 + j) * kTok + tok_row) >> p.p_shift)) : -1; };
      bool bad = false;  // the token that the registers hold has no page
      auto token_base = [&](int32_t id, int j) -> const uint8_t* {
        bad = false;
        if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.n_pages))
          return p.pool + static_cast<size_t>(static_cast<uint32_t>(id)) * p.page_bytes + region;
        bad = asked(j);
        if (bad) flags |= kErrBadPage;
        return nullptr;
      };
      auto load_codes = [&](uint32_t (&w)[D / 8], const uint8_t* src) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint4 x = src ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
          w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
      };
      auto load_nums = [&](const uint8_t* src) {
#pragma unroll
        for (int g = 0; g < NG; ++g) num[g] = src ? __ldg(reinterpret_cast<const uint2*>(src) + g) : make_uint2(0, 0);
      };
      int32_t id = -1;
      if (two) {
        id = page_of(0);
        const uint8_t* src = token_base(id, 0);
        const int tp = (tile0 * kTok + tok_row) & (p.P - 1);
        load_nums(src ? src + p.P * D + tp * 8 * NG : nullptr);
        load_codes(kw, src ? src + tp * (D / 2) : nullptr);
        load_codes(vw, src ? src + p.P * (D / 2) + tp * (D / 2) : nullptr);
        id = page_of(1);
      }
      __syncthreads();
      for (int j = 0; j < n_tiles; ++j) {
        const uint32_t J = tiles_done + j, st = J & 1, ph = (J >> 1) & 1;
        const uint8_t* next = nullptr;
        const int tp = ((tile0 + j + 1) * kTok + tok_row) & (p.P - 1);
        uint32_t hidden;
        if (two) {
          hidden = __ballot_sync(0xffffffffu, bad);
          next = token_base(id, j + 1);
          id = page_of(j + 2);
#pragma unroll
          for (int g = 0; g < NG; ++g) cur[g] = num[g];
        } else {
          const uint32_t codes = base + Ge::ring_at(two) + st * Ge::kStage;
          wait(c_full + st, ph);
          bad = (s_bad_pages[st] >> (tok_row >> page_sh)) & 1;
          const int tok = (tile0 + j) * kTok + tok_row;
          const bool none = bad || tok < t_begin || tok >= t_end;
          hidden = __ballot_sync(0xffffffffu, bad);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            ld_shared_v2(codes + 2 * Ge::kCodes + tok_row * 8 * NG + 8 * g, cur[g].x, cur[g].y);
            if (none) cur[g] = make_uint2(0, 0);
          }
#pragma unroll
          for (int i = 0; i < CH; ++i)
            if (takes(i)) ld_shared_v4(codes + tok_row * (D / 2) + 16 * key_chunk(i), kw[4 * i], kw[4 * i + 1], kw[4 * i + 2], kw[4 * i + 3]);
          if (!keys) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
              ld_shared_v4(codes + Ge::kCodes + tok_row * (D / 2) + 16 * value_chunk(i), vw[4 * i], vw[4 * i + 1], vw[4 * i + 2],
                           vw[4 * i + 3]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(c_free + st);
        }
        if (keys || kShared) {
          __half2 s1[NG], s2[NG];
          uint32_t more[4] = {0, 0, 0, 0}, large = 0;
          if constexpr (kExact) {  // the scale in seven bits and the rest; the minimum
            bool over = false;
#pragma unroll
            for (int g = 0; g < NG; ++g) over |= (cur[g].x & 0xffffu) >= 0x6C00u;  // FP16 4096; scales are not negative
            large = __ballot_sync(0xffffffffu, over);
            const __half2 down = __float2half2_rn(over ? 0.25f : 1.f);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const __half2 s = __hmul2(__half2half2(scale_of(cur[g].x)), down);
              const uint32_t top = *reinterpret_cast<const uint32_t*>(&s) & 0xFFF0FFF0u;
              s1[g] = *reinterpret_cast<const __half2*>(&top);
              s2[g] = __hsub2(s, s1[g]);
              const __half2 mn = __hmul2(__half2half2(min_of(cur[g].x)), down);
              more[g] = *reinterpret_cast<const uint32_t*>(&mn);
            }
          }
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            if (!keys && hf < kHalves - 1) continue;
            const uint32_t ks = one_k ? hf : st;
            wait(k_free + ks, (one_k ? J & 1 : ph) ^ 1);
            if (kExact && hf == 0) st_shared_v4(base + Ge::more_k_at(two) + 16 * tok_row, more[0], more[1], more[2], more[3]);
#pragma unroll
            for (int i = hf * (CH / kHalves); i < (hf + 1) * (CH / kHalves); ++i) {
              if (!takes(i)) continue;
              const uint32_t kd = k_tiles + (one_k ? 0 : st * Ge::kTile) + 16 * tok_row + 8192 * key_chunk(i);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int g = (k % KW) / (KW / NG);
                const uint32_t w = kw[4 * i + k], w8 = w >> 8;
                if constexpr (kExact) {
                  uint32_t y[4], z[4];
                  codes2_times<false>(w, s1[g], s2[g], y[0], z[0]);
                  codes2_times<true>(w, s1[g], s2[g], y[1], z[1]);
                  codes2_times<false>(w8, s1[g], s2[g], y[2], z[2]);
                  codes2_times<true>(w8, s1[g], s2[g], y[3], z[3]);
                  st_shared_v4(kd + k * 2048, y[0], y[1], y[2], y[3]);
                  st_shared_v4(kd + Ge::kTile + k * 2048, z[0], z[1], z[2], z[3]);
                } else {
                  const __half2 s = __half2half2(scale_of(cur[g].x)), mn = __half2half2(min_of(cur[g].x));
                  st_shared_v4(kd + k * 2048, dequant2<false>(w, s, mn), dequant2<true>(w, s, mn), dequant2<false>(w8, s, mn),
                               dequant2<true>(w8, s, mn));
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {  // the tile four back has had its softmax: its values were freed two tiles ago
              if (hf == 0) {
                s_hidden[J & 3][warp & 3] = hidden;
                if constexpr (kExact) s_large[J & 3][warp & 3] = large;
                if (hidden | large) s_any_odd = 1;
              }
              mbar_arrive(k_full + ks);
            }
          }
          if (two) load_codes(kw, next ? next + tp * (D / 2) : nullptr);
        }
        if (two) load_nums(next ? next + p.P * D + tp * 8 * NG : nullptr);
        if (vals) {
          wait(v_free + st, ph ^ 1);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const uint32_t vd = v_tiles + st * Ge::kTile + 16 * tok_row + 8192 * value_chunk(c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // word 4 chunk + k, pair i: channels 64 (k % VW) + 16 i + {0, 8} + word / VW
              uint32_t y[4];
              const uint32_t w = vw[4 * c + k], w8 = w >> 8;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t nm = cur[(64 * (k % VW) + 16 * i) / (D / NG)].y;
                const __half2 s = __half2half2(scale_of(nm)), mn = __half2half2(min_of(nm));
                const uint32_t src = i < 2 ? w : w8;
                y[i] = (i & 1) ? dequant2<true>(src, s, mn) : dequant2<false>(src, s, mn);
              }
              st_shared_v4(vd + k * 2048, y[0], y[1], y[2], y[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_full + st);
            if (two && warp == 8) s_unpacked = J + 1;
          }
          if (two) load_codes(vw, next ? next + p.P * (D / 2) + tp * (D / 2) : nullptr);
        }
        if (any(s_abort)) break;  // the warp together: it votes again at the next tile
      }
    } while (leave_segment(n_tiles, steps));
  } else if (group == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<two>::issue));
    int n_tiles, steps;
    do {
      n_tiles = sg.tiles, steps = steps_of();
      if (warp == 13) {
        // ---- a lane per page of the tile, its key codes, value codes and numbers: copied (one tile of queries), and asked
        // into L2 some tiles ahead
        const int32_t* table = p.page_table + static_cast<size_t>(sg.b) * p.max_pages;
        const size_t region = static_cast<size_t>(sg.h) * kv4_head_bytes(D, NG, p.P);
        const int2 t_seen = block_tokens<kTree>(p, sg.T, sg.n, sg.base, sg.rb, R);
        const int tile0 = sg.tile, t_begin = t_seen.x, t_end = t_seen.y;
        const int part = min(p.P, kTok);  // tokens of a page that are in a tile
        auto asked = [&](int j) {  // by the tokens, not by the id: any may stand in the table
          const int tok = (tile0 + j) * kTok + lane * part;
          return j < n_tiles && lane * part < kTok && tok + part > t_begin && tok < t_end;
        };
        auto page_of = [&](int j) -> int32_t { return asked(j) ? __ldg(table + (((tile0 + j) * kTok + lane * part) >> p.p_shift)) : -1; };
        auto good = [&](int32_t id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.n_pages); };
        auto page_at = [&](int32_t id, int j, int& tp) -> const uint8_t* {
          tp = ((tile0 + j) * kTok + lane * part) & (p.P - 1);
          return p.pool + static_cast<size_t>(static_cast<uint32_t>(id)) * p.page_bytes + region;
        };
        auto prefetch = [&](int j) {
          const int32_t id = page_of(j);
          if (!good(id)) return;
          int tp;
          const uint8_t* const src = page_at(id, j, tp);
          bulk_prefetch_l2(src + tp * (D / 2), part * (D / 2));
          bulk_prefetch_l2(src + (p.P + tp) * (D / 2), part * (D / 2));
          bulk_prefetch_l2(src + p.P * D + tp * 8 * NG, part * 8 * NG);
        };
        auto copy = [&](int j, int32_t id) -> bool {
          const uint32_t J = tiles_done + j, cs = J & 1;
          if (!all(wait(c_free + cs, ((J >> 1) & 1) ^ 1))) return false;
          const bool have = good(id), none = !have && asked(j);
          if (none) flags |= kErrBadPage;
          const uint32_t bad = __ballot_sync(0xffffffffu, none), here = __ballot_sync(0xffffffffu, have);
          if (lane == 0) {
            s_bad_pages[cs] = bad;
            mbar_arrive_expect_tx(c_full + cs, __popc(here) * part * (D + 8 * NG));
          }
          __syncwarp();
          if (have) {
            int tp;
            const uint8_t* const src = page_at(id, j, tp);
            uint8_t* const dst = smem + Ge::ring_at(two) + cs * Ge::kStage;
            bulk_g2s(dst + lane * part * (D / 2), src + tp * (D / 2), part * (D / 2), c_full + cs);
            bulk_g2s(dst + Ge::kCodes + lane * part * (D / 2), src + (p.P + tp) * (D / 2), part * (D / 2), c_full + cs);
            bulk_g2s(dst + 2 * Ge::kCodes + lane * part * 8 * NG, src + p.P * D + tp * 8 * NG, part * 8 * NG, c_full + cs);
          }
          return true;
        };
        int32_t id = two ? -1 : page_of(0);
        int sent = !two && copy(0, id) ? 1 : 0;
        if (!two) id = page_of(1);
        for (int j = 1; j < kAhead; ++j) prefetch(j);
        __syncthreads();
        if (two) {
          // A tile for each that is unpacked, by a count that only grows: nothing waits for this warp, so a barrier's phase
          // could come and go while it is late. Where the count does not come the other waits end the call.
          for (int j = 0; j < n_tiles && !s_abort; ++j) {
            prefetch(j + kAhead);
            const long long t0 = clock64();
            while (static_cast<int32_t>(s_unpacked - (tiles_done + j)) <= 0 && !s_abort && clock64() - t0 <= kBudget) __nanosleep(64);
          }
        }
        for (; sent > 0 && sent < n_tiles; ++sent) {
          prefetch(sent + kAhead - 1);
          if (!copy(sent, id)) break;
          id = page_of(sent + 1);
        }
        // copies in flight end before the segment does, whatever happened
        for (int j = max(0, sent - 2); j < sent; ++j) {
          const uint32_t J = tiles_done + j;
          if (!mbar_wait_bounded(c_full + (J & 1), (J >> 1) & 1, kBudget >> 4)) s_abort = 1;
        }
      } else {
        __syncthreads();
        if (warp == 15 && lane == 0 && line) {  // the next segment of the CTA's stretch, meanwhile
          s_next = s_seg;
          s_next.at = min(s_next.end, s_next.item0 + s_next.item_tiles + kStart);
          next_item<kTree>(p, s_next, line, R);
        }
      }
      if (warp == 12) {
        // ---- products, issued by one lane of the whole warp
        constexpr uint32_t kDescS = tc5::instr_desc(kTok, false), kDescO = tc5::instr_desc(D, true);
        const uint32_t leader = tc5::elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        auto scores = [&](int s) -> bool {
          const int u = s & 1, j = two ? s >> 1 : s;
          const uint32_t J = tiles_done + j, st = one_k ? 0 : J & 1;
          const uint64_t qa = tc5::smem_desc(base + (two ? u * Ge::kTile : 0), 2048, 128);
          const uint64_t ka = tc5::smem_desc(k_tiles + st * Ge::kTile, 2048, 128);
          constexpr int kHalves = one_k ? 2 : 1;
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            const uint32_t ks = one_k ? hf : st;
            if ((!two || u == 0) && !all(wait(k_full + ks, one_k ? J & 1 : (J >> 1) & 1))) return false;
            tc5::fence_after();
#pragma unroll
            for (int k = hf * (D / 32); k < (hf + 1) * (D / 16 / kHalves); ++k) {  // descriptor addresses count 16 bytes
              if constexpr (!kTmemQ) tc5::mma_ss(tm + Ge::kColS + 128 * u, qa + 256 * k, ka + 256 * k, kDescS, k > 0, leader);
              else tc5::mma_ts(tm + Ge::kColS + 128 * u, tm + Ge::kColQ + 8 * k, ka + 256 * k, kDescS, k > 0, leader);
              if constexpr (kExact && !kTmemQ)
                tc5::mma_ss(tm + Ge::kColS + 128 * u, qa + 256 * k, ka + Ge::kTile / 16 + 256 * k, kDescS, true, leader);
              else if constexpr (kExact)
                tc5::mma_ts(tm + Ge::kColS + 128 * u, tm + Ge::kColQ + 8 * k, ka + Ge::kTile / 16 + 256 * k, kDescS, true, leader);
            }
            if constexpr (kExact) {
              const uint64_t more_k = tc5::smem_desc(base + Ge::more_k_at(two), 2048, 128);
              if (hf > 0) {
              } else if constexpr (!kTmemQ) {
                tc5::mma_ss(tm + Ge::kColS + 128 * u, tc5::smem_desc(base + Ge::more_q_at(two) + (two ? u * Ge::kMore : 0), 2048, 128), more_k,
                            kDescS, true, leader);
              } else {
                tc5::mma_ts(tm + Ge::kColS + 128 * u, tm + Ge::kColQ + D / 2, more_k, kDescS, true, leader);
              }
            }
            if (hf == kHalves - 1) tc5::commit(s_full + u, leader);
            if (!two || u == 1) tc5::commit(k_free + ks, leader);
          }
          return true;
        };
        bool ok = scores(0) && (steps < 2 || scores(1));
        for (int s = 0; ok && s < steps; ++s) {
          const int u = s & 1, j = two ? s >> 1 : s;
          const uint32_t J = tiles_done + j, st = J & 1;
          ok = all(wait((two ? p_half : p_ready) + u, (steps_done[u] + (s >> 1)) & 1) && ((two && u == 1) || wait(v_full + st, (J >> 1) & 1)));
          if (!ok) break;
          tc5::fence_after();
          const uint64_t va = tc5::smem_desc(v_tiles + st * Ge::kTile, 128, 2048);
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k) {
            if (two && k == kTok / 32) {
              ok = all(wait(p_ready + u, (steps_done[u] + (s >> 1)) & 1));
              tc5::fence_after();
            }
            tc5::mma_ts(tm + Ge::kColO + (two ? D * u : 0), tm + Ge::kColS + 128 * u + 8 * k, va + 16 * k, kDescO,
                        s >= (two ? 2 : 1) || k > 0, leader);
            if (kSplit)
              tc5::mma_ts(tm + Ge::kColO + (two ? D * u : 0), tm + Ge::kColS + 128 * u + 64 + 8 * k, va + 16 * k, kDescO, true, leader);
          }
          if (!two || u == 1) tc5::commit(v_free + st, leader);
          if (s + 2 < steps) ok = scores(s + 2);
        }
        tc5::commit(o_done, leader);  // the products in flight end before anyone goes on, whatever happened
        if (!mbar_wait_bounded(o_done, segs & 1, ok ? kBudget : kBudget >> 4)) {
          s_abort = 1;
          flags |= kErrTimeout;
        }
      }
      __syncwarp();
    } while (leave_segment(n_tiles, steps));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<two>::softmax));
    const int lane_row = tid & 127, side = lane_row >> 6;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t oc = tmem + lane_base + Ge::kColO + D * group;
    const int n_softmax = two ? 256 : 128;  // threads of the softmax groups
    int n_tiles, steps;
    do {
      n_tiles = sg.tiles, steps = steps_of();
      const int tile0 = sg.tile;
      const int rows_left = sg.n * p.G - sg.rb * R;  // live rows of the block
      const int row = two ? 128 * group + lane_row : half ? lane_row & 63 : lane_row, rr = sg.rb * R + row;
      const bool live = row < rows_left;
      float m = kNoMax, l = 0.f, fr = 0.f;
      int2 vis = make_int2(0, 0);
      {
        // ---- queries: the warp's 32 rows, eight rows x 64 bytes with one load (lane: row lane & 7 of the
        // eight, 16-byte chunk lane >> 3 of the four); prescaled by a power of two and stored in the keys' channel
        // order, eight rows of a chunk side by side; this thread keeps its own row's factor
        if (!kTree && live) vis = visible(p, sg.T, sg.n, rr / p.G);
        uint4 w[4][CB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r2 = row - lane + 8 * i + (lane & 7), q2 = sg.rb * R + r2;  // row of the block
          const uint16_t* src = p.q.data + static_cast<int64_t>(sg.r0 + q2 / p.G) * p.q.row_stride +
                                static_cast<int64_t>(sg.h * p.G + q2 % p.G) * p.q.head_stride;
#pragma unroll
          for (int j = 0; j < CB / 4; ++j)
            w[i][j] = r2 < rows_left ? __ldg(reinterpret_cast<const uint4*>(src) + 4 * j + (lane >> 3)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mx = 0.f;
#pragma unroll
          for (int j = 0; j < CB / 4; ++j) {
            float x[8];
            unpack8(w[i][j], p.f16, x);
#pragma unroll
            for (int k = 0; k < 8; k += 2) mx = max3(mx, fabsf(x[k]), fabsf(x[k + 1]));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const int E = fp16_exponent(mx) - (kExact ? 8 : 0);  // kExact: below 2^7, so that the sums fit
          if ((lane >> 3) == i)  // a hidden score, -inf, stays one at scale 0
            fr = fmaxf(pow2_int(-E) * fabsf(p.scale_log2), 1e-37f);
          if (two || group == 0) {
            const float up = p.scale_log2 < 0.f ? -pow2_int(E) : pow2_int(E);
            const uint32_t dst = base + (two ? group * Ge::kTile : 0) + 16 * (32 * (warp & 3) + 8 * i + (lane & 7));
            float sum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
            for (int j = 0; j < CB / 4; ++j) {  // channels 32 j + 8 (lane >> 3) ..: chunk (D / 32) (lane >> 3) + j
              float x[8];
              uint32_t y[4];
              unpack8(w[i][j], p.f16, x);
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = h2(x[k] * up, x[k + 4] * up);
              st_shared_v4(dst + ((lane >> 3) * KW + j) * 2048, y[0], y[1], y[2], y[3]);
              if constexpr (kExact) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y[k]));
                  sum[j / (KW / NG)] += v.x + v.y;
                }
              }
            }
            if constexpr (kExact) {
              uint32_t more[4] = {0, 0, 0, 0};
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 8);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 16);
                const float high = __half2float(__float2half_rn(sum[g]));
                more[g] = h2(high, sum[g] - high);
              }
              const uint32_t at = base + Ge::more_q_at(two) + (two ? group * Ge::kMore : 0) +
                                  16 * (32 * (warp & 3) + 8 * i + (lane & 7));
              if (lane < 8) st_shared_v4(at, more[0], more[1], more[2], more[3]);
              else if (lane < 16) st_shared_v4(at + 2048, 0, 0, 0, 0);
              else if (lane < 24 && (!two || group == 0))  // and the keys' last eight channels: nothing
                st_shared_v4(base + Ge::more_k_at(two) + 2048 + 16 * (32 * (warp & 3) + 8 * i + (lane & 7)), 0, 0, 0, 0);
            }
          }
        }
        if constexpr (!kTmemQ) {
          fence_proxy_async_smem();
        } else {  // on to tensor memory, a thread its row
          __syncwarp();
          const uint32_t at = base + 16 * lane_row, to = tmem + lane_base + Ge::kColQ;
#pragma unroll
          for (int c = 0; c < CB; c += 4) {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) ld_shared_v4(at + 2048 * (c + i), y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            tc5::st16(to + 4 * c, y);
          }
          if constexpr (kExact) {
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              ld_shared_v4(at + Ge::more_q_at(two) + 2048 * i, y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            tc5::st8(to + D / 2, y);
            fence_proxy_async_smem();  // the keys' last channels
          }
          tc5::wait_st();
          tc5::fence_before();
        }
      }
      int full_lo, full_hi;  // tiles that every live row of the block sees whole
      if constexpr (kTree) {
        const int2 every = tree_tokens_of_all(p, sg.T, sg.base);
        full_lo = (every.x + kTok - 1) / kTok;
        full_hi = every.y / kTok;
      } else {
        const int i0 = sg.rb * R / p.G, i1 = min(sg.n - 1, (sg.rb * R + R - 1) / p.G);
        full_lo = (visible(p, sg.T, sg.n, i1).x + kTok - 1) / kTok;
        full_hi = visible(p, sg.T, sg.n, i0).y / kTok;
      }
      __syncthreads();
      // ---- softmax: thread = row
      auto tile_weights = [&](auto chunks, int k) {
        constexpr int NC = decltype(chunks)::value;  // chunks of 32 tokens that a thread takes
        const int first = NC == 4 ? 0 : 2 * side;    // the first of them
        const int t = tile0 + k, u = two ? group : k & 1;  // S buffer
        const uint32_t sc = tmem + lane_base + Ge::kColS + 128 * u;
        const uint32_t ph = two ? steps_done[group] + k : steps_done[u] + (k >> 1);
        wait(s_full + u, ph & 1);
        tc5::fence_after();
        uint32_t raw[NC][32];
#pragma unroll
        for (int c = 0; c < NC; ++c) tc5::ld32(sc + 32 * (first + c), raw[c]);
#pragma unroll
        for (int c = 0; c < NC; ++c) tc5::wait_ld(raw[c]);
        if (s_any_odd) {  // some tile so far
          if constexpr (kExact) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint32_t four = s_large[(tiles_done + k) & 3][first + c];
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((four >> i) & 1) raw[c][i] = __float_as_uint(4.f * __uint_as_float(raw[c][i]));
            }
          }
          uint32_t bits[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) bits[c] = s_hidden[(tiles_done + k) & 3][first + c];
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bits[c] >> i) & 1) raw[c][i] = 0xff800000u;  // -inf
        }
        if constexpr (kTree) {
          if (t < full_lo || t >= full_hi) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const uint32_t seen = live ? tree_bits(p, sg.r0 + rr / p.G, sg.T, sg.base, t * kTok + 32 * (first + c)) : 0u;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((seen >> i) & 1)) raw[c][i] = 0xff800000u;  // -inf
            }
          }
        } else if (t < full_lo || t >= full_hi) {
          const int lo = vis.x - t * kTok - 32 * first, hi = vis.y - t * kTok - 32 * first;  // columns that this row sees: [lo, hi)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < lo || 32 * c + i >= hi) raw[c][i] = 0xff800000u;  // -inf
        }
        // The weights are formed under the running max as it is, unless a score is more than 2^8 above it (a warp's
        // first tile always finds its max).
        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            mx = max3(mx, __uint_as_float(raw[c][i]), __uint_as_float(raw[c][i + 1]));
            my = max3(my, __uint_as_float(raw[c][i + 2]), __uint_as_float(raw[c][i + 3]));
          }
        mx = fmaxf(mx, my);
        if (k == 0 || __any_sync(0xffffffffu, mx * fr > m + kSlack)) {
          const float mn = fmaxf(m, mx * fr), a = ex2(m - mn);
          m = mn;
          l *= a;
          if (k > 0) {
            if (!two) {  // the products of the tile before still add to O
              const uint32_t J = tiles_done + k - 1;
              wait(v_free + (J & 1), (J >> 1) & 1);
              tc5::fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t v[16];
              tc5::ld16(oc + 16 * c, v);
              tc5::wait_ld16(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * a);
              tc5::st16(oc + 16 * c, v);
            }
            tc5::wait_st();
          }
        }
        float l0 = 0.f, l1 = 0.f;
        const float neg = kRoom - m;
        auto half_ready = [&]() {
          tc5::wait_st();
          tc5::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_half + u);
        };
        if constexpr (kSplit) {  // sixteen at a time: both parts of 32 would not fit the registers
#pragma unroll
          for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int i0 = 0; i0 < 32; i0 += 16) {
              uint32_t w[8], rest[8];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                float a = __uint_as_float(raw[c][i0 + i]), b = __uint_as_float(raw[c][i0 + i + 1]);
                fma_pair(a, b, fr, neg);
                a = ex2(a);
                b = ex2(b);
                add_pair(l0, l1, a, b);
                w[i >> 1] = h2(a, b);
                const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&w[i >> 1]));
                rest[i >> 1] = h2(a - r.x, b - r.y);
              }
              tc5::st8(sc + 16 * (first + c) + i0 / 2, w);
              tc5::st8(sc + 64 + 16 * (first + c) + i0 / 2, rest);
            }
            if (two && c == 1) half_ready();
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a = __uint_as_float(raw[c][i]), b = __uint_as_float(raw[c][i + 1]);
              fma_pair(a, b, fr, neg);
              a = ex2(a);
              b = ex2(b);
              add_pair(l0, l1, a, b);
              w[i >> 1] = h2(a, b);
            }
            tc5::st16(sc + 16 * (first + c), w);
            if (two && c == 1) half_ready();
          }
        }
        l += l0 + l1;
        if constexpr (NC == 2) {  // the other half's weights are its twin's
          uint32_t none[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) none[i] = 0;
          tc5::st16(sc + 16 * (2 - first), none);
          tc5::st16(sc + 16 * (3 - first), none);
          if (kSplit) {
            tc5::st16(sc + 64 + 16 * (2 - first), none);
            tc5::st16(sc + 64 + 16 * (3 - first), none);
          }
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + u);
      };
      for (int k = 0; k < n_tiles && !any(s_abort); ++k) {
        if (half) tile_weights(std::integral_constant<int, 2>{}, k);
        else tile_weights(std::integral_constant<int, 4>{}, k);
      }
      const bool done = all(wait(o_done, segs & 1) && !s_abort);
      tc5::fence_after();

              constexpr int kPartRow = D * 4;
              uint8_t* const part_st = smem + (two ? Ge::k_at(true) : Ge::v_at(false));  // 32 rows of floats per warp
              float f = 1.f;
              if (half) {  // the row and its twin: a common max, the twin's sums by way of shared memory
                s_side[lane_row] = make_float2(m, l);
                softmax_barrier(n_softmax);
                const float2 a = s_side[row], b = s_side[row + 64];
                const float M = fmaxf(a.x, b.x);
                f = ex2(m - M);
                l = ex2(a.x - M) * a.y + ex2(b.x - M) * b.y;
                m = M;
                if (side) {
                  uint8_t* const st = part_st + (warp & 3) * 32 * kPartRow;
#pragma unroll
                  for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tc5::ld32(oc + 32 * c, v);
                    tc5::wait_ld(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                      *reinterpret_cast<float4*>(st + lane * kPartRow + 16 * ((8 * c + i) ^ (lane & 7))) =
                          make_float4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f,
                                      __uint_as_float(v[4 * i + 2]) * f, __uint_as_float(v[4 * i + 3]) * f);
                  }
                }
                softmax_barrier(n_softmax);
              }
      // ---- results: thread = row
      if (done) {
        auto load_sums = [&](int c, float (&x)[32]) {  // columns 32 c ..
          uint32_t v[32];
          tc5::ld32(oc + 32 * c, v);
          tc5::wait_ld(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]);
          if (half) {
            const uint8_t* const st = part_st + ((warp & 1) + 2) * 32 * kPartRow;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 o = *reinterpret_cast<const float4*>(st + lane * kPartRow + 16 * ((8 * c + i) ^ (lane & 7)));
              x[4 * i] = fmaf(x[4 * i], f, o.x), x[4 * i + 1] = fmaf(x[4 * i + 1], f, o.y);
              x[4 * i + 2] = fmaf(x[4 * i + 2], f, o.z), x[4 * i + 3] = fmaf(x[4 * i + 3], f, o.w);
            }
          }
        };
        const bool stores = !half || side == 0;
        const float y = l == 0.f ? 0.f : 1.f / l;
        auto out_row = [&](int row_of_block) {
          const int q2 = sg.rb * R + row_of_block;
          return static_cast<size_t>(sg.r0 + q2 / p.G) * p.Hq + sg.h * p.G + q2 % p.G;
        };
        // rows go out by way of shared memory (each warp its 32 rows), so that lanes store along a row; 16-byte
        // chunks are exchanged by the row's low bits: distinct banks both ways
        const int first = (two ? 128 * group : 0) + 32 * (warp & 3);
        if (!stores) {
        } else if (sg.part >= 0) {
          constexpr int kRow = kPartRow, kChunks = D / 4;
          uint8_t* const st = part_st + (first >> 5) * 32 * kRow;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float x[32];
            load_sums(c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(st + lane * kRow + 16 * ((8 * c + i) ^ (lane & 7))) =
                  make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
          __syncwarp();
          const int left = min(32, rows_left - first);
          float4* const dst = reinterpret_cast<float4*>(p.part_o + (static_cast<size_t>(sg.part) * R + first) * D);
          for (int e = lane; e < left * kChunks; e += 32) {
            const int r2 = e / kChunks, ch = e % kChunks;
            dst[e] = *reinterpret_cast<const float4*>(st + r2 * kRow + 16 * (ch ^ (r2 & 7)));
          }
          if (live) reinterpret_cast<float2*>(p.part_ml)[static_cast<size_t>(sg.part) * R + row] = make_float2(m, l);
          if (tid == 0 && sg.c0 == static_cast<int>(blockIdx.x)) s_joined = Kv4Joined{sg.h, sg.rb, sg.parts, sg.r0, sg.n * p.G};
        } else {
          uint32_t res[D / 2];
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float x[32];
            load_sums(c, x);
            // column 8 wi + 2 i + e is channel 64 (wi % VW) + 16 i + 8 e + wi / VW: neighbouring channels are
            // columns VW * 8 apart, in the same 32
#pragma unroll
            for (int i = 0; i < 8 * VW; ++i) {  // i = 8 w + 2 pair + e
              constexpr int kPairs = 32 / (16 * VW);  // channel pairs per 32 columns
#pragma unroll
              for (int k = 0; k < kPairs; ++k) {
                const int col = (2 * k) * 8 * VW + i;
                res[i * 4 + c * kPairs + k] = pack2(x[col] * y, x[col + 8 * VW] * y, p.f16);
              }
            }
          }
          constexpr int kRow = D * 2, kChunks = D / 8;  // chunk i holds channels 8 i .. 8 i + 7
          uint8_t* const st = smem + (first >> 5) * 32 * kRow;  // where the queries were
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            *reinterpret_cast<uint4*>(st + lane * kRow + 16 * (i ^ (lane & 7))) =
                make_uint4(res[4 * i], res[4 * i + 1], res[4 * i + 2], res[4 * i + 3]);
          __syncwarp();
          const int left = min(32, rows_left - first);
          for (int e = lane; e < left * kChunks; e += 32) {
            const int r2 = e / kChunks, ch = e % kChunks;
            reinterpret_cast<uint4*>(p.out + out_row(first + r2) * D)[ch] =
                *reinterpret_cast<const uint4*>(st + r2 * kRow + 16 * (ch ^ (r2 & 7)));
          }
          if (live && p.lse) p.lse[out_row(row)] = l == 0.f ? -INFINITY : (m + (log2f(l) - kRoom)) * 0.69314718055994531f;
        }
      }
      tc5::fence_before();
    } while (leave_segment(n_tiles, steps));
  }
  tc5::fence_before();
  __syncthreads();
  if (warp == 12) tc5::dealloc512(tmem);
  if (line && tid == 0) p.joined[blockIdx.x] = s_joined;
  if (line && s_abort) {  // some warp may have given up before it stored its rows: neither part counts
    float2* const ml = reinterpret_cast<float2*>(p.part_ml) + static_cast<size_t>(blockIdx.x) * 2 * R;
    for (int i = tid; i < 2 * R; i += kThreads) ml[i] = make_float2(kNoMax, -1.f);
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && flags) atomicOr(p.err, flags);
}

template <int D, int NG, bool kExact, bool two, bool kTree, bool kSplit>
cudaError_t launch_as(const Kv4AttnParams& p, int rows, int line, int ctas, cudaStream_t stream) {
  static bool attr_done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kv4_prompt_kernel<D, NG, kExact, two, kTree, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Geom<D, NG, kExact>::smem(two));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  kv4_prompt_kernel<D, NG, kExact, two, kTree, kSplit><<<ctas, kThreads, Geom<D, NG, kExact>::smem(two), stream>>>(p, rows, line);
  return cudaGetLastError();
}

template <int D, int NG, bool kTree, bool kSplit>
cudaError_t launch_many(const Kv4AttnParams& p, int rows, int line, int ctas, cudaStream_t stream) {
  // Keys rounded to FP16 where nothing asks for exact scores, but not beside weights in two parts: an FP16 output would be off by 4.6e-4
  // in place of 2.8e-4 of it, and by more or less as a log-sum-exp is asked for.
  if constexpr (!kSplit) {
    if (rows == 256 && !p.lse) return launch_as<D, NG, false, true, kTree, false>(p, rows, line, ctas, stream);
    if constexpr (D == 64) {
      if (rows < 256 && !p.lse) return launch_as<D, NG, false, false, kTree, false>(p, rows, line, ctas, stream);
    }
  }
  return rows == 256 ? launch_as<D, NG, true, true, kTree, kSplit>(p, rows, line, ctas, stream)
                     : launch_as<D, NG, true, false, kTree, kSplit>(p, rows, line, ctas, stream);
}

template <bool kTree, bool kSplit>
cudaError_t launch_prompt_part(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  const int ctas = static_cast<int>(z.ctas);
  if (D == 128) {
    if (n_groups == 1) return launch_many<128, 1, kTree, kSplit>(p, z.rows, z.line, ctas, stream);
    if (n_groups == 2) return launch_many<128, 2, kTree, kSplit>(p, z.rows, z.line, ctas, stream);
    return launch_many<128, 4, kTree, kSplit>(p, z.rows, z.line, ctas, stream);
  }
  return n_groups == 1 ? launch_many<64, 1, kTree, kSplit>(p, z.rows, z.line, ctas, stream) : launch_many<64, 2, kTree, kSplit>(p, z.rows, z.line, ctas, stream);
}

template <bool kTree, bool kSplit>
cudaError_t launch_prompt_kernel(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  const cudaError_t e = launch_prompt_part<kTree, kSplit>(p, z, D, n_groups, stream);
  return e != cudaSuccess || !z.line ? e : launch_kv4_join(p, z, D, stream);
}

}  // namespace
}  // namespace mlaq
