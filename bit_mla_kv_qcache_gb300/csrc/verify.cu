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
// Sums decide whole numbers here, so they are held in two float32 (a sum and the exact error of its additions, ~2^-45 of it) and
// joined in 64 bits, which a B300 adds at a sixty-fourth of the float32 rate: two additions exact by themselves cost ten times less.
//
// A cluster of eight CTAs takes a sequence: the row that is summed is cut over them, their sums meet in distributed shared memory. All of
// a node's numbers (parent, token, p(x), q(x), u) are read at the start, a thread per node, and stored to every CTA of the
// cluster: the CTAs take the same way because they hold the same bits. Reads: only the rows that are summed.
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
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Nodes {  // of the sequence, the same in every CTA of its cluster
  int parent[kMaxTreeRows], token[kMaxTreeRows];
  float p[kMaxTreeRows], q[kMaxTreeRows], u[kMaxTreeRows];  // p and q of the node's token at its parent
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
__device__ __forceinline__ int next_child(const Nodes& nodes, int n, int at, int after, bool match, int token) {
  const int lane = threadIdx.x & 31;
  for (int i0 = (after + 1) & ~31; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const bool hit = i > after && i < n && nodes.parent[i] == at && (!match || nodes.token[i] == token);
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
template <int kPer, typename T>
__device__ __forceinline__ Slice slice_of(const T* row, int vocab, int rank_warp) {
  Slice s;
  s.shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kPer);
  s.vectors = static_cast<int>((static_cast<int64_t>(vocab) + s.shift + kPer - 1) / kPer);
  const int per = (s.vectors + kCtas * kWarps * 32 - 1) / (kCtas * kWarps * 32) * 32;  // whole rounds of a warp
  s.first = static_cast<int>(min(static_cast<int64_t>(rank_warp) * per, static_cast<int64_t>(s.vectors)));
  s.last = min(s.first + per, s.vectors);
  return s;
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
__device__ __forceinline__ void rest4(const Rest& w, const int* gone, int shift, int v, const float4& pv, const float4& qv, Pair (&r)[4]) {
  const float a[4] = {mass(pv.x), mass(pv.y), mass(pv.z), mass(pv.w)};
  if (w.q) {
    const float b[4] = {mass(qv.x), mass(qv.y), mass(qv.z), mass(qv.w)};
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = residual(a[k], b[k], w.ch, w.cl);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = Pair{a[k], 0.f};
  }
  for (int i = 0; i < w.n_gone; ++i) {
    const int64_t at = static_cast<int64_t>(gone[i]) + shift;
    if (at >> 2 == v) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((at & 3) == k) r[k] = Pair{0.f, 0.f};
    }
  }
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ double warp_upto(double x) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 2) verify_sampled_kernel(const VerifyParams p) {
  __shared__ Nodes nodes;
  __shared__ double s_cta[2][kCtas], s_warp[kWarps];
  __shared__ int s_gone[kMaxTreeRows], s_kept[kMaxTreeRows], s_n, s_r0;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = static_cast<int>(cl.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kCtas;
  const float* const target = static_cast<const float*>(p.target);
  int flags = 0;
  for (int i = tid; i < kMaxTreeRows; i += kThreads) nodes.parent[i] = -2;
  auto started = cl.barrier_arrive();  // every CTA is there, its nodes empty
  {
    int r0;
    const int n = rows_of(p, b, r0, flags), i = tid;
    int parent = -2, token = 0;
    float px = 0.f, qx = 0.f, u = 0.f;
    if (i < n && i % kCtas == rank) {
      const int r = r0 + i;
      parent = i == 0 ? -1 : parent_of(p, r, i);
      token = __ldg(p.tokens + r);
      u = __ldg(p.u_accept + r);
      if (token < 0 || token >= p.vocab || parent < 0) {
        parent = -2;  // never tried
      } else {
        px = mass(__ldg(target + (r0 + parent) * p.target_stride + token));
        qx = p.draft ? mass(__ldg(p.draft + (r0 + parent) * p.draft_stride + token)) : 1.f;
      }
    }
    cl.barrier_wait(std::move(started));
    if (i < n && i % kCtas == rank) {
#pragma unroll 1
      for (int c = 0; c < kCtas; ++c) {
        Nodes* const to = cl.map_shared_rank(&nodes, c);
        to->parent[i] = parent, to->token[i] = token, to->p[i] = px, to->q[i] = qx, to->u[i] = u;
      }
    }
    if (rank == 0 && tid < kCtas) *cl.map_shared_rank(&s_n, tid) = n, *cl.map_shared_rank(&s_r0, tid) = r0;
    cl.sync();
  }
  const int n = s_n, r0 = s_r0;
  const int rank_warp = rank * kWarps + warp;

  // ---- the sum of what is left of a row: of every warp's part in s_warp, of every CTA's in s_cta[turn]
  int turn = 0;
  auto sum = [&](const Rest& w) -> double {
    const Slice s = slice_of<4>(w.p, p.vocab, rank_warp);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, err[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 4;
    for (int v0 = s.first + lane; v0 < s.last; v0 += 32 * kAhead) {
      float4 pv[kAhead], qv[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int v = v0 + 32 * k;
        pv[k] = qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v < s.last) {
          pv[k] = load4(w.p, s.shift, v, p.vocab, true);
          if (w.q) qv[k] = load4(w.q, s.shift, v, p.vocab, w.q_even);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        Pair r[4];
        rest4(w, s_gone, s.shift, v0 + 32 * k, pv[k], qv[k], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exact(acc[i], err[i], r[i].d, r[i].e);
      }
    }
    double x = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) x += static_cast<double>(acc[i]) + static_cast<double>(err[i]);
    x = warp_sum(x);
    __syncthreads();  // the sums of the turn before have been read
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    turn ^= 1;
    if (warp == 0) {
      const double c = warp_sum(lane < kWarps ? s_warp[lane] : 0.0);
      if (lane < kCtas) cl.map_shared_rank(&s_cta[turn][0], lane)[rank] = c;
    }
    cl.sync();
    double all = 0.0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) all += s_cta[turn][c];
    return all;
  };

  int count = n > 0 ? 1 : 0;
  if (n > 0) {
    int at = 0, after = 0, n_gone = 0;
    double c = 0.0, Z = 1.0;
    bool summed = false;
    auto rest = [&]() {
      Rest w;
      w.p = target + (r0 + at) * p.target_stride;
      w.q = p.draft && c > 0.0 ? p.draft + (r0 + at) * p.draft_stride : nullptr;
      w.ch = static_cast<float>(c);
      w.cl = static_cast<float>(c - static_cast<double>(w.ch));
      w.n_gone = n_gone;
      w.q_even = w.q && ((reinterpret_cast<uintptr_t>(w.p) ^ reinterpret_cast<uintptr_t>(w.q)) & 15) == 0;
      return w;
    };
    double total = 0.0;
    if (tid == 0) s_kept[0] = 0;
    while (true) {
      const int x = next_child(nodes, n, at, after, false, 0);
      if (x >= n) break;
      after = x;
      const double px = nodes.p[x], qx = nodes.q[x], u = nodes.u[x];
      bool gone = false;
      if (!p.draft)
        for (int i = 0; i < n_gone; ++i) gone |= s_gone[i] == nodes.token[x];
      const double left = gone ? 0.0 : p.draft ? fmax(px - c * qx, 0.0) : px;
      if (u * qx * Z < left) {
        at = x;
        c = 0.0, Z = 1.0, n_gone = 0;
        summed = false;
        if (tid == 0) s_kept[count] = x;
        ++count;
        __syncthreads();  // s_gone is free again
      } else if (p.draft) {
        c += Z;
        Z = total = sum(rest());
        summed = true;
      } else if (!gone) {
        Z -= px;
        if (tid == 0) s_gone[n_gone] = nodes.token[x];
        ++n_gone;
        __syncthreads();
      }
    }
    // ---- the new token
    Rest w = rest();
    if (!summed) total = sum(w);
    if (!(total > 0.0)) {  // nothing is left: the row as it is
      w.q = nullptr;
      w.n_gone = 0;
      total = sum(w);
    }
    const double pos = static_cast<double>(__ldg(p.u_sample + b)) * total;
    // the CTA, then the warp, in whose part the running sum passes pos; behind the last (rounding): the last with a part
    int cta = -1;
    double before = 0.0, upto = 0.0;
    for (int i = 0; i < kCtas; ++i) {
      const double x = s_cta[turn][i];
      if (x > 0.0 && (cta < 0 || upto <= pos)) cta = i, before = upto;
      upto += x;
    }
    if (cta < 0 && rank == 0 && tid == 0) {
      flags |= kErrRange;
      p.new_tokens[static_cast<size_t>(b) * p.max_rows + count - 1] = -1;
    }
    if (cta == rank) {
      int part = -1;
      upto = before;
      for (int i = 0; i < kWarps; ++i) {
        const double x = s_warp[i];
        if (x > 0.0 && (part < 0 || upto <= pos)) part = i, before = upto;
        upto += x;
      }
      if (part == warp) {
        const Slice s = slice_of<4>(w.p, p.vocab, rank_warp);
        int64_t found = -1, last = -1;
        for (int v0 = s.first; v0 < s.last && found < 0; v0 += 32) {
          const int v = v0 + lane;
          Pair r[4] = {};
          if (v < s.last) {
            const float4 pv = load4(w.p, s.shift, v, p.vocab, true);
            const float4 qv = w.q ? load4(w.q, s.shift, v, p.vocab, w.q_even) : make_float4(0.f, 0.f, 0.f, 0.f);
            rest4(w, s_gone, s.shift, v, pv, qv, r);
          }
          double x = 0.0;
          int64_t mine = -1;  // the lane's last entry with a part
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x += static_cast<double>(r[k].d) + static_cast<double>(r[k].e);
            if (r[k].d + r[k].e > 0.f) mine = 4ll * v + k - s.shift;
          }
          const double inclusive = before + warp_upto(x);
          const unsigned passed = __ballot_sync(0xffffffffu, mine >= 0 && inclusive > pos), some = __ballot_sync(0xffffffffu, mine >= 0);
          if (passed) {
            int64_t j = mine;
            double run = inclusive - x;
#pragma unroll
            for (int k = 3; k >= 0; --k) {  // the first entry at which the sum passes
              double to = run;
              for (int m = 0; m <= k; ++m) to += static_cast<double>(r[m].d) + static_cast<double>(r[m].e);
              if (r[k].d + r[k].e > 0.f && to > pos) j = 4ll * v + k - s.shift;
            }
            found = __shfl_sync(0xffffffffu, j, __ffs(passed) - 1);
          } else if (some) {
            last = __shfl_sync(0xffffffffu, mine, 31 - __clz(some));
          }
          before = __shfl_sync(0xffffffffu, inclusive, 31);
        }
        if (lane == 0) p.new_tokens[static_cast<size_t>(b) * p.max_rows + count - 1] = static_cast<int32_t>(found >= 0 ? found : last);
      }
    }
  }
  if (rank == 0) {
    __syncthreads();
    for (int i = tid; i < p.max_rows; i += kThreads) {
      p.kept[static_cast<size_t>(b) * p.max_rows + i] = i < count ? s_kept[i] : -1;
      if (i != count - 1)
        p.new_tokens[static_cast<size_t>(b) * p.max_rows + i] = i < count ? nodes.token[s_kept[i + 1]] : -1;
    }
    if (tid == 0) {
      p.n_kept[b] = count;
      if (flags) atomicOr(p.err, flags);
    }
  }
}

// ---------------------------------------------------------------- greedy
// Larger keys are larger values, and among equal ones lower indices; 0: no number.
__device__ __forceinline__ unsigned long long key_of(float x, int j) {
  const uint32_t w = __float_as_uint(x);
  const uint32_t o = w & 0x80000000u ? ~w : w | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(j));
}
template <typename T>
__device__ __forceinline__ float value_of(T x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 2) verify_greedy_kernel(const VerifyParams p) {
  __shared__ Nodes nodes;
  __shared__ unsigned long long s_best[2][kCtas], s_warp[kWarps];
  __shared__ int s_kept[kMaxTreeRows], s_n, s_r0;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = static_cast<int>(cl.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kCtas;
  const T* const target = static_cast<const T*>(p.target);
  int flags = 0;
  for (int i = tid; i < kMaxTreeRows; i += kThreads) nodes.parent[i] = -2;
  auto started = cl.barrier_arrive();
  {
    int r0;
    const int n = rows_of(p, b, r0, flags), i = tid;
    int parent = -2, token = 0;
    if (i < n && i % kCtas == rank) {
      parent = i == 0 ? -2 : parent_of(p, r0 + i, i);
      token = __ldg(p.tokens + r0 + i);
    }
    cl.barrier_wait(std::move(started));
    if (i < n && i % kCtas == rank) {
#pragma unroll 1
      for (int c = 0; c < kCtas; ++c) {
        Nodes* const to = cl.map_shared_rank(&nodes, c);
        to->parent[i] = parent < 0 ? -2 : parent, to->token[i] = token;
      }
    }
    if (rank == 0 && tid < kCtas) *cl.map_shared_rank(&s_n, tid) = n, *cl.map_shared_rank(&s_r0, tid) = r0;
    cl.sync();
  }
  const int n = s_n, r0 = s_r0, rank_warp = rank * kWarps + warp;
  constexpr int kPer = 16 / sizeof(T);
  int count = 0, turn = 0, at = 0, last = -1;
  while (n > 0) {
    const T* const row = target + (r0 + at) * p.target_stride;
    const Slice s = slice_of<kPer>(row, p.vocab, rank_warp);
    float best = -INFINITY;
    int64_t where = -1;
    constexpr int kAhead = 4;
    for (int v0 = s.first + lane; v0 < s.last; v0 += 32 * kAhead) {
      uint4 raw[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t j = static_cast<int64_t>(kPer) * (v0 + 32 * k) - s.shift;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (v0 + 32 * k < s.last && j >= 0 && j + kPer <= p.vocab) raw[k] = __ldg(reinterpret_cast<const uint4*>(row + j));
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t j = static_cast<int64_t>(kPer) * (v0 + 32 * k) - s.shift;
        if (v0 + 32 * k >= s.last) break;
        const bool inside = j >= 0 && j + kPer <= p.vocab;
        const T* const x = reinterpret_cast<const T*>(&raw[k]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (!inside && (j + i < 0 || j + i >= p.vocab)) continue;
          const float y = inside ? value_of<T>(x[i]) : value_of<T>(row[j + i]);
          if (y > best || (where < 0 && y == best)) best = y, where = j + i;
        }
      }
    }
    unsigned long long key = where < 0 ? 0ull : key_of(best + 0.f, static_cast<int>(where));  // -0 equals +0
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
    __syncthreads();
    if (lane == 0) s_warp[warp] = key;
    __syncthreads();
    turn ^= 1;
    if (warp == 0) {
      key = lane < kWarps ? s_warp[lane] : 0ull;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
      if (lane < kCtas) cl.map_shared_rank(&s_best[turn][0], lane)[rank] = key;
    }
    cl.sync();
    key = 0ull;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) key = max(key, s_best[turn][c]);
    if (tid == 0) s_kept[count] = at;
    ++count;
    last = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    if (!key && rank == 0) flags |= kErrNonFinite;
    const int x = last < 0 ? n : next_child(nodes, n, at, at, true, last);
    if (x >= n) break;
    at = x;
  }
  if (rank == 0) {
    __syncthreads();
    for (int i = tid; i < p.max_rows; i += kThreads) {
      p.kept[static_cast<size_t>(b) * p.max_rows + i] = i < count ? s_kept[i] : -1;
      p.new_tokens[static_cast<size_t>(b) * p.max_rows + i] = i < count - 1 ? nodes.token[s_kept[i + 1]] : i == count - 1 ? last : -1;
    }
    if (tid == 0) {
      p.n_kept[b] = count;
      if (flags) atomicOr(p.err, flags);
    }
  }
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

}  // namespace

cudaError_t launch_verify_sampled(const VerifyParams& p, cudaStream_t stream) {
  verify_sampled_kernel<<<static_cast<unsigned>(p.B) * kCtas, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_verify_greedy(const VerifyParams& p, cudaStream_t stream) {
  const unsigned ctas = static_cast<unsigned>(p.B) * kCtas;
  if (p.type == 0) verify_greedy_kernel<__nv_bfloat16><<<ctas, kThreads, 0, stream>>>(p);
  else if (p.type == 1) verify_greedy_kernel<__half><<<ctas, kThreads, 0, stream>>>(p);
  else verify_greedy_kernel<float><<<ctas, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t stream) {
  tree_mask_kernel<<<p.B, kMaxTreeRows, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mlaq
