// Verification of drafted tokens (chains and trees) against the target model, from given random numbers or greedily.
//
// A sequence's rows are nodes of a tree, row 0 its root; p_r is the target's distribution behind node r, q_r the one that
// the children of r were drawn from. From the root on, the children of the node reached so far are tried in order. After k
// rejections there,
//   res_k = max(p - c_k q, 0),  c_0 = 0, Z_0 = 1,  c_(k+1) = c_k + Z_k,  Z_k = sum res_k  (k > 0),
// is in proportion to what the residual distributions max(p/Z - q, 0), one formed of the other, leave: one number instead of a
// row that changes. A child x is accepted, and its children are next, where u q(x) Z_k < res_k(x); where none is, the new
// token is drawn from the last res by its running sum. Without q (drafts picked without chance) a child is accepted where
// u Z < p(x), and a rejected child's probability goes from the row and from Z.
//
// Sums decide whole numbers here, so they are pairs of float32 (a sum and the exact error of its additions, after Knuth's and Dekker's
// two-sums, products by a fused multiply-add; ~2^-42 of it): in 64 bits,
// which a B300 adds at a sixty-fourth of the float32 rate, five drafts of 64 sequences took 102 us, with pairs 19.
//
// A cluster of eight CTAs takes a sequence: the row that is summed is cut over them, their sums meet in distributed shared memory. The first CTA
// reads all of a node's numbers (parent, token, p(x), q(x), u), a thread per node, its warp 0 walks, and tells the others which row
// to sum: they take the same way whatever happens to the inputs meanwhile. Reads: only the rows that are summed.
#include <cfloat>
#include <utility>

#include <cooperative_groups.h>

#include "append.cuh"
#include "kernels.cuh"
#include "verify.cuh"

namespace mlaq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;  // of a cluster

// A sequence's nodes. parent -2: never accepted.
struct __align__(8) Node {
  int parent, token;
  int first;  // whether it is accepted as the first child that is tried
  float u, p, q;  // its random number; p and q of its token at its parent
};

// Rows of sequence b; none where the offsets do not fit.
__device__ __forceinline__ int rows_of(const VerifyParams& p, int b, int& r0, int& flags) {
  r0 = __ldg(p.cu_rows + b);
  const int n = __ldg(p.cu_rows + b + 1) - r0;
  if (n < 0 || n > p.max_rows || r0 < 0 || r0 > p.n_rows - n) {
    flags |= kErrRows;
    return 0;
  }
  return n;
}

// The highest node before i in row r's mask; -1: none.
__device__ __forceinline__ int parent_of(const VerifyParams& p, int r, int i) {
  if (!p.mask) return i - 1;
  for (int w = min((i - 1) >> 5, p.mask_words - 1); w >= 0; --w) {
    uint32_t bits = __ldg(p.mask + static_cast<size_t>(r) * p.mask_words + w);
    if (32 * w + 32 > i) bits &= (1u << (i - 32 * w)) - 1u;
    if (bits) return 32 * w + 31 - __clz(bits);
  }
  return -1;
}

// The first node behind `after` that is a child of `at` and, with match, carries `token`; n: none. By a whole warp.
__device__ __forceinline__ int next_child(const Node* nodes, int n, int at, int after, bool match, int token) {
  const int lane = threadIdx.x & 31;
  for (int i0 = (after + 1) & ~31; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const bool hit = i > after && i < n && nodes[i].parent == at && (!match || nodes[i].token == token);
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (m) return i0 + __ffs(m) - 1;
  }
  return n;
}

// A probability that counts: not NaN, not negative, finite.
__device__ __forceinline__ float mass(float x) { return x > 0.f && x <= FLT_MAX ? x : 0.f; }

// max(p - c q, 0) as an exact difference d + e (to ~2^-48 of p).
struct Pair {
  float d, e;
};
__device__ __forceinline__ Pair residual(float p, float q, float ch, float cl) {
  const float h = __fmul_rn(ch, q), l = __fmaf_rn(cl, q, __fmaf_rn(ch, q, -h));
  const float d = __fsub_rn(p, h), t = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, t)), __fadd_rn(h, t)), l);
  return __fadd_rn(d, e) > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}
// s + e += d + x, the error of the addition to s going to e
__device__ __forceinline__ void add_exact(float& s, float& e, float d, float x) {
  const float t = __fadd_rn(s, d), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(x, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(d, z))));
  s = t;
}

// The entries of a row in vectors of four that lie on 16-byte boundaries (the first begins up to three entries before the
// row); vectors first .. last - 1 are the warp's.
struct Slice {
  int shift, vectors, first, last;
};
// A warp's part of a slice that so many share, in whole rounds of a warp.
__device__ __forceinline__ Slice part_of(Slice s, int warp, int warps) {
  const int round = warps * 32, per = static_cast<int>((static_cast<int64_t>(s.last) - s.first + round - 1) / round) * 32;
  const int end = s.last;
  s.first = static_cast<int>(min(s.first + static_cast<int64_t>(warp) * per, static_cast<int64_t>(end)));
  s.last = static_cast<int>(min(static_cast<int64_t>(s.first) + per, static_cast<int64_t>(end)));
  return s;
}
template <int kPer, typename T>
__device__ __forceinline__ Slice slice_of(const T* row, int vocab, int warp, int warps) {  // the warp's of so many
  Slice s;
  s.shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kPer);
  s.vectors = static_cast<int>((static_cast<int64_t>(vocab) + s.shift + kPer - 1) / kPer);
  s.first = 0, s.last = s.vectors;
  return part_of(s, warp, warps);
}
// Vector v of a row, entries outside it 0.
__device__ __forceinline__ float4 load4(const float* row, int shift, int v, int vocab, bool even) {
  const int64_t j = 4ll * v - shift;
  if (even && j >= 0 && j + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + j));
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = j + k >= 0 && j + k < vocab ? __ldg(row + j + k) : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

// What is left of the row at a node.
struct Rest {
  const float *p, *q;  // the row, and the draft's, or nullptr
  float ch, cl;        // c
  int n_gone;          // tokens whose probability is gone
  bool q_even;         // q's entries lie on the same boundaries
};
// How many tokens a warp has to look for in its vectors: all, or 0 where none of them lies there.
__device__ __forceinline__ int gone_within(const Rest& w, const int* gone, const Slice& s) {
  bool here = false;
  for (int i = threadIdx.x & 31; i < w.n_gone; i += 32) {
    const int64_t v = (static_cast<int64_t>(gone[i]) + s.shift) >> 2;
    here |= v >= s.first && v < s.last;
  }
  return __any_sync(0xffffffffu, here) ? w.n_gone : 0;
}
// Entries of vector v that are gone become 0.
__device__ __forceinline__ void take_gone(float4& x, const int* gone, int n_gone, int shift, int v) {
#pragma unroll 1
  for (int i = 0; i < n_gone; ++i) {
    const unsigned at = static_cast<unsigned>(gone[i]) + shift;
    if (at >> 2 == static_cast<unsigned>(v)) {
      x.x = (at & 3) == 0 ? 0.f : x.x, x.y = (at & 3) == 1 ? 0.f : x.y;
      x.z = (at & 3) == 2 ? 0.f : x.z, x.w = (at & 3) == 3 ? 0.f : x.w;
    }
  }
}
// What is left of four entries (those that are gone are 0).
__device__ __forceinline__ void left4(const Rest& w, const float4& pv, const float4& qv, Pair (&r)[4]) {
  const float a[4] = {mass(pv.x), mass(pv.y), mass(pv.z), mass(pv.w)};
  if (w.q) {
    const float b[4] = {mass(qv.x), mass(qv.y), mass(qv.z), mass(qv.w)};
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = residual(a[k], b[k], w.ch, w.cl);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = Pair{a[k], 0.f};
  }
}

// A sum and its error. (|e| is at most half a step of s: comparisons go by the difference.)
struct Sum {
  float s, e;
};
__device__ __forceinline__ Sum operator+(const Sum& a, const Sum& b) {
  float s = a.s, e = a.e;
  add_exact(s, e, b.s, b.e);
  const float t = __fadd_rn(s, e);
  return {t, __fsub_rn(e, __fsub_rn(t, s))};
}
__device__ __forceinline__ Sum operator*(const Sum& a, const Sum& b) {
  const float h = __fmul_rn(a.s, b.s), l = __fmaf_rn(a.s, b.s, -h);
  return Sum{h, 0.f} + Sum{l, __fmaf_rn(a.s, b.e, __fmul_rn(a.e, b.s))};
}
__device__ __forceinline__ bool above(const Sum& a, const Sum& b) {
  return __fadd_rn(__fsub_rn(a.s, b.s), __fsub_rn(a.e, b.e)) > 0.f;
}
// Inclusive sums over the lanes (the first kLanes of a warp).
template <int kLanes = 32>
__device__ __forceinline__ Sum upto(Sum x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const Sum y = {__shfl_up_sync(0xffffffffu, x.s, o), __shfl_up_sync(0xffffffffu, x.e, o)};
    if (lane >= o) x = y + x;
  }
  return x;
}
__device__ __forceinline__ Sum of_lane(const Sum& x, int lane) {
  return {__shfl_sync(0xffffffffu, x.s, lane), __shfl_sync(0xffffffffu, x.e, lane)};
}

// Two sums with their errors, side by side.
struct Sum2 {
  float2 s, e;
};
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {  // one instruction: b (-1) + a, rounded once
  float2 r;
  asm("{ .reg .b64 x, y, m; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 m, {%6, %6}; fma.rn.f32x2 x, y, m, x; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(-1.f));
  return r;
}
// s + e += d, the error of the addition to s going to e (additions alone: nothing here can be fused)
__device__ __forceinline__ void add_exact2(Sum2& a, float2 d) {
  const float2 t = add2(a.s, d), z = sub2(t, a.s);
  a.e = add2(a.e, add2(sub2(a.s, sub2(t, z)), sub2(d, z)));
  a.s = t;
}
__device__ __forceinline__ bool all_count(const float4& x) {  // none negative, infinite or NaN
  return max(max(__float_as_uint(x.x), __float_as_uint(x.y)), max(__float_as_uint(x.z), __float_as_uint(x.w))) <= 0x7f7fffffu;
}
__device__ __forceinline__ float4 masses(const float4& x) { return make_float4(mass(x.x), mass(x.y), mass(x.z), mass(x.w)); }

// How what is left of an entry is formed.
enum class Left { kRow, kOnce, kAny };  // p, less what is gone; max(p - q, 0); max(p - c q, 0)

// Adds what is left of four entries. For p - q the smaller of p and q is taken away, so that the difference is 0 or of a larger and a
// smaller number, whose error is (p - d) - q.
template <Left kLeft>
__device__ __forceinline__ void add_left(Sum2 (&part)[2], const Rest& w, float4 p, float4 q) {
  if constexpr (kLeft == Left::kAny) {
    Pair r[4];
    left4(w, p, q, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      add_exact(part[i].s.x, part[i].e.x, r[2 * i].d, r[2 * i].e);
      add_exact(part[i].s.y, part[i].e.y, r[2 * i + 1].d, r[2 * i + 1].e);
    }
  } else {
    if (!all_count(p)) p = masses(p);
    if (kLeft == Left::kRow) {
      add_exact2(part[0], make_float2(p.x, p.y));
      add_exact2(part[1], make_float2(p.z, p.w));
    } else {
      if (!all_count(q)) q = masses(q);
      const float2 p0 = make_float2(p.x, p.y), p1 = make_float2(p.z, p.w);
      const float2 q0 = make_float2(fminf(p.x, q.x), fminf(p.y, q.y)), q1 = make_float2(fminf(p.z, q.z), fminf(p.w, q.w));
      const float2 d0 = sub2(p0, q0), d1 = sub2(p1, q1);
      add_exact2(part[0], d0);
      add_exact2(part[1], d1);
      part[0].e = add2(part[0].e, sub2(sub2(p0, d0), q0));
      part[1].e = add2(part[1].e, sub2(sub2(p1, d1), q1));
    }
  }
}

// The sum of what is left of a row in a warp's vectors; every lane has it. Vectors that lie in the row as a whole are loaded without a
// look, four rounds ahead; the row's ends, and a q on other boundaries, entry by entry.
template <Left kLeft>
__device__ __forceinline__ Sum sum_left(const Rest& w, const Slice& s, int vocab, const int* gone = nullptr, int n_gone = 0) {
  const int lane = threadIdx.x & 31;
  constexpr int kAhead = 4;
  Sum2 part[2] = {};
  const bool has_q = kLeft != Left::kRow && w.q;
  int lo = s.first, hi = s.last;
  // one by one: the row's ends (lanes 0 and 1), or all
  int one = lo + lane, ones = hi;
  const bool even = !has_q || w.q_even;
  if (even) {
    const int whole = static_cast<int>((static_cast<int64_t>(vocab) + s.shift) >> 2);  // behind the last vector that is whole
    const bool head = lo == 0 && hi > 0 && s.shift > 0;
    const bool tail = hi > whole && whole >= lo + (head ? 1 : 0);
    one = head && lane == 0 ? 0 : tail && lane == 1 ? whole : hi;
    ones = min(one + 1, hi);
    lo += head ? 1 : 0;
    hi = min(hi, whole);
  }
#pragma unroll 1
  for (int v = one; v < ones; v += 32) {
    const float4 q = has_q ? load4(w.q, s.shift, v, vocab, w.q_even) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 x = load4(w.p, s.shift, v, vocab, true);
    if (kLeft == Left::kRow) take_gone(x, gone, n_gone, s.shift, v);
    add_left<kLeft>(part, w, x, q);
  }
  if (even) {
    const float4* const P = reinterpret_cast<const float4*>(w.p - s.shift) + lane;
    const float4* const Q = has_q ? reinterpret_cast<const float4*>(w.q - s.shift) + lane : P;
    for (int v = lo; v < hi; v += 32 * kAhead) {
      float4 pv[kAhead], qv[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool in = v + 32 * k + lane < hi;
        pv[k] = qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) pv[k] = __ldg(P + v + 32 * k);
        if (has_q && in) qv[k] = __ldg(Q + v + 32 * k);
      }
      if (kLeft == Left::kRow && n_gone) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) take_gone(pv[k], gone, n_gone, s.shift, v + 32 * k + lane);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (v + 32 * k < hi) add_left<kLeft>(part, w, pv[k], qv[k]);
    }
  }
  Sum x = (Sum{part[0].s.x, part[0].e.x} + Sum{part[0].s.y, part[0].e.y}) + (Sum{part[1].s.x, part[1].e.x} + Sum{part[1].s.y, part[1].e.y});
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = x + Sum{__shfl_xor_sync(0xffffffffu, x.s, o), __shfl_xor_sync(0xffffffffu, x.e, o)};
  return of_lane(x, 0);
}
__device__ __forceinline__ Sum sum_of(const Rest& w, const int* gone, const Slice& s, int vocab) {
  if (!w.q) return sum_left<Left::kRow>(w, s, vocab, gone, gone_within(w, gone, s));
  if (w.ch == 1.f && w.cl == 0.f) return sum_left<Left::kOnce>(w, s, vocab);
  return sum_left<Left::kAny>(w, s, vocab);
}

// Of a list of sums, one to a lane, the part in which the running sum passes pos: the last with something in it whose predecessors
// together do not; -1: nothing anywhere. start: what comes before the list, and what comes before the part.
struct Found {
  int part;
  Sum start;
};
template <int kLanes>
__device__ __forceinline__ Found find_part(Sum x, Sum pos, Sum start) {
  const Sum up = upto<kLanes>((threadIdx.x & 31) == 0 ? start + x : x);
  Sum prior = {__shfl_up_sync(0xffffffffu, up.s, 1), __shfl_up_sync(0xffffffffu, up.e, 1)};
  if ((threadIdx.x & 31) == 0) prior = start;
  const unsigned some = __ballot_sync(0xffffffffu, x.s > 0.f), open = __ballot_sync(0xffffffffu, x.s > 0.f && !above(prior, pos));
  const int part = open ? 31 - __clz(open) : some ? __ffs(some) - 1 : -1;
  return {part, of_lane(prior, max(part, 0))};
}

// The first entry in a warp's vectors at which the running sum, `run` before them, passes pos; the last entry with something in it,
// if rounding lets none.
__device__ __forceinline__ int find_entry(const Rest& w, const int* gone, const Slice& s, int vocab, Sum run, const Sum& pos) {
  const int lane = threadIdx.x & 31, n_gone = gone_within(w, gone, s);
  int64_t last = -1;
  for (int v0 = s.first; v0 < s.last; v0 += 32) {
    const int v = v0 + lane;
    float4 pv = make_float4(0.f, 0.f, 0.f, 0.f), qv = pv;
    if (v < s.last) {
      pv = load4(w.p, s.shift, v, vocab, true);
      if (w.q) qv = load4(w.q, s.shift, v, vocab, w.q_even);
    }
    take_gone(pv, gone, n_gone, s.shift, v);
    Pair r[4];
    left4(w, pv, qv, r);
    Sum x = {0.f, 0.f};
    int own = -1;  // the lane's last entry with something in it
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x = x + Sum{r[i].d, r[i].e};
      if (r[i].d + r[i].e > 0.f) own = i;
    }
    const Sum here = run + upto(x);
    const unsigned passed = __ballot_sync(0xffffffffu, own >= 0 && above(here, pos)), some = __ballot_sync(0xffffffffu, own >= 0);
    if (passed) {
      Sum to = {__shfl_up_sync(0xffffffffu, here.s, 1), __shfl_up_sync(0xffffffffu, here.e, 1)};
      if (lane == 0) to = run;
      bool over = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        to = to + Sum{r[i].d, r[i].e};
        if (!over && r[i].d + r[i].e > 0.f && above(to, pos)) own = i, over = true;
      }
      return static_cast<int>(__shfl_sync(0xffffffffu, 4ll * v - s.shift + own, __ffs(passed) - 1));
    }
    if (some) last = __shfl_sync(0xffffffffu, 4ll * v - s.shift + own, 31 - __clz(some));
    run = of_lane(here, 31);
  }
  return static_cast<int>(last);
}

// What the first CTA asks of all: the sum of what is left of a row and, with `last`, the new token from it.
struct __align__(16) Ask {
  Rest rest;
  int last, count;  // count: nodes kept
  float u;
};
constexpr int kAlone = 64;  // vectors in which one warp finds the new token by itself
struct Find {  // a CTA's warp 0 to its others: the slice in which the new token is, the sum before it, the sum that it passes
  Rest rest;
  int here;
  Slice at;
  Sum start, pos;
};

template <int kThreads>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1024 / kThreads) verify_sampled_kernel(const VerifyParams p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Node nodes[kMaxTreeRows];
  __shared__ Sum s_cta[2][kCtas], s_warp[kWarps];
  __shared__ Ask s_ask;
  __shared__ Find s_find;
  __shared__ int s_gone[kMaxTreeRows], s_kept[kMaxTreeRows + 1];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = static_cast<int>(cl.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kCtas;
  const float* const target = static_cast<const float*>(p.target);
  auto started = cl.barrier_arrive();
  int turn = 0;
  // One round, of every CTA: what s_ask says is summed, every warp's part in s_warp, every CTA's in s_cta[turn] of each.
  auto round = [&](const Rest& w) {
    const Sum x = sum_of(w, s_gone, slice_of<4>(w.p, p.vocab, rank * kWarps + warp, kCtas * kWarps), p.vocab);
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    turn ^= 1;
    if (warp == 0) {
      const Sum all = of_lane(upto<kWarps>(lane < kWarps ? s_warp[lane] : Sum{0.f, 0.f}), kWarps - 1);
      if (lane < kCtas) cl.map_shared_rank(&s_cta[turn][0], lane)[rank] = all;
    }
    cl.sync();
  };
  auto total = [&]() { return of_lane(upto<kCtas>(lane < kCtas ? s_cta[turn][lane] : Sum{0.f, 0.f}), kCtas - 1); };
  auto store_new = [&](int count, int token) {
    if (lane == 0) p.new_tokens[static_cast<size_t>(b) * p.max_rows + count - 1] = token;
  };

  // ---- the first CTA, its warp 0, walks from the root. Its state stands in shared memory between rounds.
  __shared__ int s_n, s_r0, s_at, s_after, s_count, s_n_gone, s_fresh;
  __shared__ Sum s_c, s_Z;
  if (rank == 0) {
    // Where every sequence has max_rows rows, what stands at b max_rows is this one's: asked for while the offsets come.
    const bool even = static_cast<int64_t>(p.B) * p.max_rows == p.n_rows && tid < p.max_rows;
    const int guess = b * p.max_rows;
    int token = 0, r0, flags = 0;
    float u = 0.f;
    if (even) token = __ldg(p.tokens + guess + tid), u = __ldg(p.u_accept + guess + tid);
    const int n = rows_of(p, b, r0, flags), i = tid;
    if (i < n) {
      const int r = r0 + i;
      if (!even || r0 != guess) token = __ldg(p.tokens + r), u = __ldg(p.u_accept + r);
      Node x = {-2, token, 0, u, 0.f, 0.f};
      const int parent = i == 0 ? -1 : parent_of(p, r, i);
      if (x.token >= 0 && x.token < p.vocab && parent >= 0) {
        x.parent = parent;
        x.p = mass(__ldg(target + (r0 + parent) * p.target_stride + x.token));
        x.q = p.draft ? mass(__ldg(p.draft + (r0 + parent) * p.draft_stride + x.token)) : 1.f;
        const float h = __fmul_rn(x.u, x.q), l = __fmaf_rn(x.u, x.q, -h);  // u q < p, exactly: the product and its error
        x.first = h < x.p || (h == x.p && l < 0.f);
      }
      nodes[i] = x;
    }
    if (tid == 0) {
      if (flags) atomicOr(p.err, flags);
      s_n = n, s_r0 = r0, s_at = s_after = s_n_gone = 0, s_fresh = 1, s_count = n > 0 ? 1 : 0, s_kept[0] = 0;
      s_c = Sum{0.f, 0.f}, s_Z = Sum{1.f, 0.f};
    }
    __syncthreads();
  }
  cl.barrier_wait(std::move(started));  // every CTA is there
  // On to the next row that has to be summed: the walk's next question, to every CTA. (By warp 0 of the first CTA.)
  auto walk = [&]() {
    const int n = s_n;
    int at = s_at, after = s_after, count = s_count, n_gone = s_n_gone;
    bool fresh = s_fresh, last = false;  // fresh: no child of the node refused yet
    Sum c = s_c, Z = s_Z;
    bool done = false;
    if (n <= 32 && fresh) {  // while every node is accepted as its parent's first child
      const int parent = lane < n ? nodes[lane].parent : -2;
      const unsigned ok = __ballot_sync(0xffffffffu, lane < n && nodes[lane].first);
      while (true) {
        const unsigned m = __ballot_sync(0xffffffffu, parent == at && lane > after), first = m & -m;
        if (first & ok) {
          at = after = __ffs(first) - 1;
          if (lane == 0) s_kept[count] = at;
          ++count;
          continue;
        }
        if (!m) {
          last = done = true;
        } else if (p.draft) {  // the first child is refused: the row has to be summed
          after = __ffs(first) - 1;
          fresh = false;
          c = Sum{1.f, 0.f};
          last = m == first;
          done = true;
        }
        break;
      }
    }
    while (!done) {
      const int x = next_child(nodes, n, at, after, false, 0);
      if (x >= n) {
        last = true;
        break;
      }
      after = x;
      const Node y = nodes[x];
      bool ok, gone = false;
      if (fresh) {
        ok = y.first;
      } else {
        for (int i0 = 0; i0 < n_gone; i0 += 32) gone |= __any_sync(0xffffffffu, i0 + lane < n_gone && s_gone[i0 + lane] == y.token);
        if (p.draft) {
          const Pair left = residual(y.p, y.q, c.s, c.e);
          ok = above(Sum{left.d, left.e}, Sum{y.u, 0.f} * Sum{y.q, 0.f} * Z);
        } else {  // u Z < p
          const float h = __fmul_rn(y.u, Z.s), l = __fmaf_rn(y.u, Z.e, __fmaf_rn(y.u, Z.s, -h));
          ok = __fsub_rn(__fsub_rn(gone ? 0.f : y.p, h), l) > 0.f;
        }
      }
      if (ok) {
        at = x;
        c = Sum{0.f, 0.f}, Z = Sum{1.f, 0.f}, n_gone = 0;
        fresh = true;
        if (lane == 0) s_kept[count] = x;
        ++count;
        continue;
      }
      fresh = false;
      if (p.draft) {
        c = c + Z;
        last = next_child(nodes, n, at, after, false, 0) >= n;  // no further child: the new token comes from this sum
        break;
      }
      if (!gone) {
        Z = Z + Sum{-y.p, 0.f};
        if (lane == 0) s_gone[n_gone] = y.token;
        ++n_gone;
        __syncwarp();
      }
    }
    __syncwarp();
    if (lane == 0) s_at = at, s_after = after, s_count = count, s_n_gone = n_gone, s_fresh = fresh, s_c = c;
    Ask a;
    a.rest.p = target + (s_r0 + at) * p.target_stride;
    a.rest.q = p.draft && !fresh ? p.draft + (s_r0 + at) * p.draft_stride : nullptr;
    a.rest.ch = c.s, a.rest.cl = c.e, a.rest.n_gone = n_gone;
    a.rest.q_even = a.rest.q && ((reinterpret_cast<uintptr_t>(a.rest.p) ^ reinterpret_cast<uintptr_t>(a.rest.q)) & 15) == 0;
    a.last = last, a.count = count;
    a.u = __ldg(p.u_sample + b);
    if (lane < kCtas) {
      *cl.map_shared_rank(&s_ask, lane) = a;
      int* const gone = cl.map_shared_rank(s_gone, lane);
      if (lane > 0)
        for (int i = 0; i < n_gone; ++i) gone[i] = s_gone[i];
    }
  };
  while (true) {
    if (rank == 0 && warp == 0) {
      if (s_n > 0) {
        walk();
      } else if (lane < kCtas) {
        Ask* const a = cl.map_shared_rank(&s_ask, lane);
        a->last = 1, a->count = 0;
      }
    }
    cl.sync();
    if (s_ask.last) break;
    round(s_ask.rest);
    if (rank == 0 && warp == 0) {
      const Sum z = total();
      if (lane == 0) s_Z = z;
      __syncwarp();
    }
  }
  // ---- the new token: every CTA sums and finds out by itself whether it is in its part
  const int count = s_ask.count;
  if (count > 0) {
    Rest w = s_ask.rest;
    round(w);
    if (!(total().s > 0.f)) {  // nothing is left: the row as it is (every thread of the cluster sees the same sums)
      w.q = nullptr;
      w.n_gone = 0;
      round(w);
    }
    if (warp == 0) {
      const Sum all = total(), pos = Sum{s_ask.u, 0.f} * all;
      Found cta = find_part<kCtas>(lane < kCtas ? s_cta[turn][lane] : Sum{0.f, 0.f}, pos, Sum{0.f, 0.f});
      if (!(all.s <= FLT_MAX)) cta.part = -1;  // a part that overflowed: the others' sums are not the row's
      int here = 0;
      if (cta.part == rank) {
        const Found at = find_part<kWarps>(lane < kWarps ? s_warp[lane] : Sum{0.f, 0.f}, pos, cta.start);
        const Slice slice = slice_of<4>(w.p, p.vocab, rank * kWarps + at.part, kCtas * kWarps);
        here = slice.last - slice.first > kAlone;
        if (!here) store_new(count, find_entry(w, s_gone, slice, p.vocab, at.start, pos));
        else if (lane == 0) s_find = Find{w, 1, slice, at.start, pos};
      } else if (cta.part < 0 && rank == 0) {
        if (lane == 0) atomicOr(p.err, kErrRange);
        store_new(count, -1);
      }
      if (lane == 0 && !here) s_find.here = 0;
    }
    __syncthreads();
    if (s_find.here) {  // a long part of a warp is cut over the CTA's warps once more
      const Slice mine = part_of(s_find.at, warp, kWarps);
      const Sum x = sum_of(s_find.rest, s_gone, mine, p.vocab);
      if (lane == 0) s_warp[warp] = x;
      __syncthreads();
      const Found at = find_part<kWarps>(lane < kWarps ? s_warp[lane] : Sum{0.f, 0.f}, s_find.pos, s_find.start);
      if (at.part == warp) store_new(count, find_entry(s_find.rest, s_gone, mine, p.vocab, at.start, s_find.pos));
    }
  }
  if (rank == 0) {
    for (int i = tid; i < p.max_rows; i += kThreads) {
      p.kept[static_cast<size_t>(b) * p.max_rows + i] = i < count ? s_kept[i] : -1;
      if (i != count - 1)
        p.new_tokens[static_cast<size_t>(b) * p.max_rows + i] = i < count ? nodes[s_kept[i + 1]].token : -1;
    }
    if (tid == 0) p.n_kept[b] = count;
  }
}

// ---------------------------------------------------------------- greedy
// Larger keys are larger values, and among equal ones lower indices; 0: no number.
__device__ __forceinline__ unsigned long long key_of(float x, int j) {
  const uint32_t w = __float_as_uint(__fadd_rn(x, 0.f));  // -0 equals +0
  const uint32_t o = w & 0x80000000u ? ~w : w | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long key) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  return key;
}
template <typename T>
__device__ __forceinline__ float value_of(T x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// The largest entry of 16 bytes; NaN only where all are.
template <typename T>
__device__ __forceinline__ float largest(const uint4& w);
template <>
__device__ __forceinline__ float largest<float>(const uint4& w) {
  return fmaxf(max3(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z)), __uint_as_float(w.w));
}
template <typename T2>
__device__ __forceinline__ T2 max_of4(const uint4& w) {
  const T2* const x = reinterpret_cast<const T2*>(&w);
  return __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
}
template <>
__device__ __forceinline__ float largest<__half>(const uint4& w) {
  const float2 m = __half22float2(max_of4<__half2>(w));
  return fmaxf(m.x, m.y);
}
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>(const uint4& w) {
  const float2 m = __bfloat1622float2(max_of4<__nv_bfloat162>(w));
  return fmaxf(m.x, m.y);
}

// Vector v of a row of `vocab` entries; those outside the row as `none`.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* row, int shift, int v, int vocab, T none) {
  constexpr int kPer = 16 / sizeof(T);
  const int64_t j = static_cast<int64_t>(kPer) * v - shift;
  if (j >= 0 && j + kPer <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + j));
  uint4 w;
  T* const x = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int k = 0; k < kPer; ++k) x[k] = j + k >= 0 && j + k < vocab ? row[j + k] : none;
  return w;
}

// The key of the largest entry among a warp's vectors of a row. Vectors are looked at as a whole; the first of a lane's that
// holds its largest value is read again for the entry. Where nothing is above -inf they are all read again, entry by entry.
template <typename T>
__device__ __forceinline__ unsigned long long best_of(const T* row, int vocab, const Slice& s) {
  constexpr int kPer = 16 / sizeof(T), kAhead = 8;
  const int lane = threadIdx.x & 31;
  const T none = static_cast<T>(NAN);
  float best = -INFINITY;
  int where = -1;
  auto look = [&](const uint4& w, int v) {
    const float m = largest<T>(w);
    if (m > best) best = m, where = v;
  };
  const int lo = s.first == 0 && s.shift > 0 ? 1 : s.first;  // vectors that lie in the row as a whole
  const int hi = min(s.last, static_cast<int>((static_cast<int64_t>(vocab) + s.shift) / kPer));
  if (lane == 0 && lo > s.first && s.last > 0) look(load16(row, s.shift, 0, vocab, none), 0);
  const uint4* const x = reinterpret_cast<const uint4*>(row - s.shift) + lane;
  for (int v = lo; v < hi; v += 32 * kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (v + 32 * k + lane < hi) w[k] = __ldg(x + v + 32 * k);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (v + 32 * k + lane < hi) look(w[k], v + 32 * k + lane);
  }
  if (lane == 0 && s.last > hi && hi >= lo) look(load16(row, s.shift, hi, vocab, none), hi);
  unsigned long long key = 0;
  auto entries = [&](int v) {
    const uint4 w = load16(row, s.shift, v, vocab, none);
    const T* const y = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float f = value_of<T>(y[k]);
      if (f == best) key = max(key, key_of(f, static_cast<int>(static_cast<int64_t>(kPer) * v - s.shift + k)));
    }
  };
  if (where >= 0) entries(where);
  key = warp_max(key);
  if (key == 0) {
    for (int v = s.first + lane; v < s.last; v += 32) entries(v);
    key = warp_max(key);
  }
  return key;
}

// The walk is one row after the other: a cluster takes the largest of the row that is reached, all its CTAs at once. A tree of up
// to eight nodes may be taken at once instead (`whole`): every CTA has a row or a part of one, and they meet a single time.
template <typename T, int kThreads>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1024 / kThreads) verify_greedy_kernel(const VerifyParams p, const bool whole) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Node nodes[kMaxTreeRows];
  __shared__ unsigned long long s_best[2][kCtas], s_warp[kWarps];
  __shared__ int s_kept[kMaxTreeRows + 1], s_n, s_r0;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = static_cast<int>(cl.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kCtas;
  const T* const target = static_cast<const T*>(p.target);
  auto started = cl.barrier_arrive();
  // At most eight rows, taken at once: every CTA meets the others once, whatever the offsets are by then. Else the first CTA reads the
  // nodes and gives them to the others: the CTAs take the same way whatever happens to the inputs meanwhile.
  int n, r0, token = 0, flags = 0;
  if (whole) {
    n = rows_of(p, b, r0, flags);
    if (rank == 0 && tid < n) token = __ldg(p.tokens + r0 + tid);
    if (rank == 0 && tid == 0 && flags) atomicOr(p.err, flags);
    cl.barrier_wait(std::move(started));
  } else {
    if (rank == 0) {
      n = rows_of(p, b, r0, flags);
      int parent = -2;
      if (tid < n) {
        token = __ldg(p.tokens + r0 + tid);
        parent = tid == 0 ? -2 : parent_of(p, r0 + tid, tid);
      }
      if (tid == 0 && flags) atomicOr(p.err, flags);
      cl.barrier_wait(std::move(started));
      if (tid < n) {
#pragma unroll
        for (int c = 0; c < kCtas; ++c) *reinterpret_cast<int2*>(&(cl.map_shared_rank(nodes, c) + tid)->parent) = make_int2(parent, token);
      }
      if (tid < kCtas) *cl.map_shared_rank(&s_n, tid) = n, *cl.map_shared_rank(&s_r0, tid) = r0;
    } else {
      cl.barrier_wait(std::move(started));
    }
    cl.sync();
    n = s_n, r0 = s_r0;
  }
  constexpr int kPer = 16 / sizeof(T);
  int turn = 0;
  // The CTA's part of row `row`, one of `parts`; its key to every CTA.
  auto meet = [&](int row, int part, int parts) {
    unsigned long long key = 0;
    if (part < parts) {
      const T* const x = target + (r0 + row) * p.target_stride;
      key = best_of<T>(x, p.vocab, slice_of<kPer>(x, p.vocab, part * kWarps + warp, parts * kWarps));
    }
    if (lane == 0) s_warp[warp] = key;
    __syncthreads();
    turn ^= 1;
    if (warp == 0) {
      key = warp_max(lane < kWarps ? s_warp[lane] : 0ull);
      if (lane < kCtas) cl.map_shared_rank(&s_best[turn][0], lane)[rank] = key;
    }
    cl.sync();
  };
  int count = 0, at = n > 0 ? 0 : -1, last = -1;
  // One step of the walk, by any warp: the token behind node `at`, and the child that carries it.
  auto step = [&](unsigned long long key) {
    if (warp == 0 && lane == 0) s_kept[count] = at;
    ++count;
    last = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    if (!key && rank == 0 && tid == 0) atomicOr(p.err, kErrNonFinite);
    const int x = last < 0 ? n : next_child(nodes, n, at, at, true, last);
    at = x < n ? x : -1;
  };
  if (whole) {
    const int parts = n > 0 ? kCtas / n : 0, row = n > 0 ? rank % n : 0;
    meet(row, n > 0 ? rank / n : 0, parts);
    if (rank > 0 || warp > 0) return;
    if (lane < n) nodes[lane].token = token, nodes[lane].parent = lane == 0 ? -2 : parent_of(p, r0 + lane, lane);
    __syncwarp();
    while (at >= 0) {
      const bool mine = lane < kCtas && lane % n == at && lane / n < parts;
      step(warp_max(mine ? s_best[turn][lane] : 0ull));
    }
  } else {
    while (at >= 0) {
      meet(at, rank, kCtas);
      step(warp_max(lane < kCtas ? s_best[turn][lane] : 0ull));
    }
    if (rank > 0 || warp > 0) return;
  }
  __syncwarp();
  for (int i = lane; i < p.max_rows; i += 32) {
    p.kept[static_cast<size_t>(b) * p.max_rows + i] = i < count ? s_kept[i] : -1;
    p.new_tokens[static_cast<size_t>(b) * p.max_rows + i] = i < count - 1 ? nodes[s_kept[i + 1]].token : i == count - 1 ? last : -1;
  }
  if (lane == 0) p.n_kept[b] = count;
}

// ---------------------------------------------------------------- masks
__global__ void __launch_bounds__(kMaxTreeRows) tree_mask_kernel(const TreeMaskParams p) {
  __shared__ int s_parent[kMaxTreeRows];
  const int b = blockIdx.x, i = threadIdx.x;
  const int r0 = __ldg(p.cu_rows + b), n = __ldg(p.cu_rows + b + 1) - r0;
  if (n < 0 || n > p.max_rows || r0 < 0 || r0 > p.n_rows - n) {
    if (i == 0) atomicOr(p.err, kErrRows);
    return;
  }
  bool bad = false;
  if (i < n) {
    int x = __ldg(p.parents + r0 + i);
    bad = x < -1 || x >= i;
    s_parent[i] = bad ? -1 : x;
  }
  if (__syncthreads_or(bad) && i == 0) atomicOr(p.err, kErrRows);
  if (i >= n) return;
  uint32_t w[kMaxTreeRows / 32] = {};
  for (int x = i; x >= 0; x = s_parent[x]) {  // a parent comes before its child: this ends
#pragma unroll
    for (int k = 0; k < kMaxTreeRows / 32; ++k)
      if (x >> 5 == k) w[k] |= 1u << (x & 31);
  }
#pragma unroll
  for (int k = 0; k < kMaxTreeRows / 32; ++k)
    if (k < p.mask_words) p.mask[static_cast<size_t>(r0 + i) * p.mask_words + k] = w[k];
}

// Clusters of a kernel that the GPU holds at once: asked for once on each device.
template <auto kKernel, int kThreads>
cudaError_t clusters_held(int* out) {
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (known[dev] == 0) {
    cudaLaunchConfig_t at{};
    at.gridDim = dim3(kCtas);
    at.blockDim = dim3(kThreads);
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kKernel, &at)) != cudaSuccess) return e;
    known[dev] = n;
  }
  *out = known[dev];
  return cudaSuccess;
}

// 512 threads to a CTA, for the latency of a row, as long as the GPU holds every sequence's cluster at once (36 of them); with more, 256,
// of which it holds twice as many. 512 and 256, sampled chains of five drafts, 102400 entries: 32 sequences 13.0 and 13.5 us, 36 13.1 and
// 14.0, 37 19.1 and 14.3, 48 22.1 and 15.5; greedy in float32 32 20.8 and 30.6, 36 21.9 and 31.5, 37 36.3 and 31.5, 48 37.5 and 33.0.
template <auto kWide, auto kNarrow, typename... Args>
cudaError_t launch_clusters(const VerifyParams& p, cudaStream_t stream, Args... more) {
  int held = 0;
  const cudaError_t e = clusters_held<kWide, 512>(&held);
  if (e != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>(p.B) * kCtas;
  if (p.B <= held) kWide<<<ctas, 512, 0, stream>>>(p, more...);
  else kNarrow<<<ctas, 256, 0, stream>>>(p, more...);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_greedy(const VerifyParams& p, cudaStream_t stream) {
  // All rows at once save a meeting of ~2 us for each row on the path, and read rows that the path never reaches: the more bytes these
  // are, the dearer. At once and one after the other (geometric means over 30, 60 and 80% of the drafts accepted, all but the smallest from
  // DRAM): six BF16 rows of 150001 of one sequence 9.0 and 12.3 us, of 8 12.7 and 19.2, 32 (55 MB) 16.6 and 21.7, 48 (82 MB) 24.1 and 24.4, 128
  // (220 MB) 51.3 and 37.9; float32 rows of 102400, four of 32 (50 MB) 15.4 and 15.2, six (75 MB) 22.2 and 18.3, six of 64 (150 MB) 36.6 and 21.3.
  // Over 330 sizes up to 256 MB the time is 0.742 of one after the other with this bound, 0.750 with half of it, 0.764 with three times as much.
  const bool whole = p.max_rows <= kCtas && static_cast<int64_t>(p.n_rows) * p.vocab * sizeof(T) <= (80 << 20);
  return launch_clusters<verify_greedy_kernel<T, 512>, verify_greedy_kernel<T, 256>>(p, stream, whole);
}

}  // namespace

cudaError_t launch_verify_sampled(const VerifyParams& p, cudaStream_t stream) {
  return launch_clusters<verify_sampled_kernel<512>, verify_sampled_kernel<256>>(p, stream);
}

cudaError_t launch_verify_greedy(const VerifyParams& p, cudaStream_t stream) {
  return p.type == 0 ? launch_greedy<__nv_bfloat16>(p, stream) : p.type == 1 ? launch_greedy<__half>(p, stream) : launch_greedy<float>(p, stream);
}

cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t stream) {
  tree_mask_kernel<<<p.B, kMaxTreeRows, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mlaq
