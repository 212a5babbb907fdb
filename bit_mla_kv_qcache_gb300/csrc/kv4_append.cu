// Append of new K/V rows to the grouped-query cache in 4 bits, keys (and the step's queries)
// rotated to their positions on the way.
//
// A thread holds eight channels of one head (one 16-byte load); the D / 8 threads of a head are
// neighbouring lanes. Rotation partners and group statistics are lane shuffles, a key-code word is
// one thread's eight channels, and a value-code word is a column of the 8 x 8 matrix of codes that
// eight lanes hold (transposed by three rounds of exchanges). CTA r serves row r: its threads
// cover 512 / D or 2048 / D heads at a time and keep the row's angles in registers over all heads; rows are
// loaded two rounds ahead. Bound: with many rows the wait for a warp's own loads with 44% of the warps resident (of eleven issue slots
// between two instructions five are that, two fixed latencies); issue is 64% busy, DRAM 46%, the ALU pipe 42%: 16K rows of 8 + 8 heads of
// 128 with 32 query heads take 107 us, their bytes, read and written once, 63 at the card's copy rate. A
// decode step of 32 rows takes 5.8 us: 32 SMs, each behind the launch and three dependent loads (offsets, page, row; with these
// alone the latent append takes 2.8) in three rounds of 16 heads.
#include "append.cuh"
#include "quant.cuh"

namespace mlaq {
namespace {

// Eight codes against the exact midpoints, 4 bits each. Rarely called, and not inlined.
__device__ __noinline__ uint32_t quant_codes8_exactly(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                                      float x7, float m, float s, float inv_s) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  uint32_t word = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) word |= static_cast<uint32_t>(quant_code(x[k], m, s, inv_s, 15)) << (4 * k);
  return word;
}

// The codes of eight values with few instructions: t = (x - m) / s from two rounded operations and a
// rounded reciprocal is off by at most 16 * 3 * 2^-24 < 3e-6, so a t further than 1e-4 from every
// midpoint has its nearest level already; where one of the eight is nearer, or the group is reported (`odd`: NaN,
// infinities, beyond the range), they are decided against the exact midpoints, within 0 .. 15 (NaN: 0). Adding 1.5 * 2^23 (bits 0x4B400000) rounds to the nearest whole number and
// leaves it in the low bits (0 <= t <= 15 but for that error; whichever way the packed operations round,
// the distance from t decides). n: the codes as numbers; returned: as fields.
__device__ __forceinline__ uint32_t quant_codes8(const float (&x)[8], const QParams& q, bool odd, float (&n)[8]) {
  constexpr float kRound = 12582912.f;
  float far = 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float2 t = mul2(add2(make_float2(x[k], x[k + 1]), make_float2(-q.m, -q.m)), make_float2(q.inv_s, q.inv_s));
    const float2 r = add2(t, make_float2(kRound, kRound)), c = add2(r, make_float2(-kRound, -kRound));
    const float2 d = add2(t, make_float2(-c.x, -c.y));
    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    n[k] = c.x, n[k + 1] = c.y;
    word += (__float_as_uint(r.x) << (4 * k)) + (__float_as_uint(r.y) << (4 * k + 4));
  }
  word -= 0x3F400000u;  // the sum of 0x4B400000 << 4 k, modulo 2^32
  if (!(far <= 0.4999f) || odd) {
    word = quant_codes8_exactly(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], q.m, q.s, q.inv_s);
#pragma unroll
    for (int k = 0; k < 8; ++k) n[k] = static_cast<float>((word >> (4 * k)) & 15u);
  }
  return word;
}

// 8 x 8 transpose of 4-bit fields: lane i (of eight) holds row i, field c at bits 4c; afterwards it
// holds column i, field r at bits 4r.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t v, int i) {
  const uint32_t keep[3] = {0x0F0F0F0Fu, 0x00FF00FFu, 0x0000FFFFu};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int d = 1 << k, sh = 4 << k;
    const uint32_t o = __shfl_xor_sync(0xffffffffu, v, d);
    v = (i & d) ? (v & ~keep[k]) | ((o >> sh) & keep[k]) : (v & keep[k]) | ((o << sh) & ~keep[k]);
  }
  return v;
}

// fields 0 2 4 6 1 3 5 7 -> 0 .. 7
__device__ __forceinline__ uint32_t even_fields_first(uint32_t v) {
  uint32_t e = v & 0x0F0F0F0Fu, o = (v >> 4) & 0x0F0F0F0Fu;
  e = (e | (e >> 4)) & 0x00FF00FFu;
  o = (o | (o >> 4)) & 0x00FF00FFu;
  e = (e | (e >> 8)) & 0x0000FFFFu;
  o = (o | (o >> 8)) & 0x0000FFFFu;
  return e | (o << 16);
}

// What the cache holds for a group that is reported: finite numbers, so that rows that do not see the token are not
// reached by it (a weight of zero times infinity or NaN). With an infinity or without a number: zeros. Beyond
// FP16: the largest scale whose top level fits.
__device__ __noinline__ QParams settle_qparams(QParams q, float lo, float hi) {
  if (!(lo > -INFINITY && hi < INFINITY)) {
    q.m = q.s = 0.f;
  } else if (q.flags & kErrRange) {
    q.s = __half2float(__float2half_rd(__fdiv_rd(65504.f - q.m, 15.f)));
  }
  q.inv_s = q.s > 0.f ? 1.f / q.s : 0.f;
  q.meta = __half_as_ushort(__float2half_rn(q.s)) | static_cast<uint32_t>(__half_as_ushort(__float2half_rn(q.m + 0.f))) << 16;
  return q;
}

// Quantizes the group that this lane's eight values belong to (LG lanes per group).
template <int LG>
__device__ __forceinline__ QParams quantize8(const float (&x)[8], uint32_t& word, float (&n)[8]) {
  float lo = fminf(x[0], x[1]), hi = fmaxf(x[0], x[1]);
#pragma unroll
  for (int k = 2; k < 8; k += 2) lo = min3(lo, x[k], x[k + 1]), hi = max3(hi, x[k], x[k + 1]);
  float2 none = make_float2(0.f, 0.f);  // NaN if a value is NaN or infinite
#pragma unroll
  for (int k = 0; k < 8; k += 2) none = add2(none, mul2(make_float2(x[k], x[k + 1]), make_float2(0.f, 0.f)));
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  QParams qp = make_qparams15(lo, hi);
  if (!(none.x + none.y == 0.f)) qp.flags |= kErrNonFinite;
  if (__fmaf_rn(15.f, qp.s, qp.m) >= 65520.f) qp.flags |= kErrRange;  // the top level would not fit FP16
  if (qp.flags) qp = settle_qparams(qp, lo, hi);
  word = quant_codes8(x, qp, qp.flags != 0, n);
  return qp;
}

template <int D, int NG, bool F16, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int kLanes = D / 8;                 // threads of one head
  constexpr int kSlots = kThreads / kLanes;     // heads at a time
  constexpr int kGroupLanes = kLanes / NG;
  const int tid = threadIdx.x, i = tid % kLanes, slot = tid / kLanes;
  const int r = blockIdx.x;
  if (r >= p.n_rows) {  // the blocks behind the rows: the new lengths
    const int b = (r - p.n_rows) * kThreads + tid;
    if (b < p.B) p.seq_next[b] = __ldg(p.seq_lens + b) + __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
    return;
  }
  const int Hq = p.q.data ? p.Hq : 0, Hkv2 = 2 * p.Hkv;
  auto load_q = [&](int h) {
    return h < Hq ? __ldg(reinterpret_cast<const uint4*>(p.q.data + r * p.q.row_stride + h * p.q.head_stride) + i)
                  : make_uint4(0, 0, 0, 0);
  };
  auto load_kv = [&](int h) {  // keys, then values
    if (h >= Hkv2) return make_uint4(0, 0, 0, 0);
    const uint16_t* src = h < p.Hkv ? p.k.data + r * p.k.row_stride + h * p.k.head_stride
                                    : p.v.data + r * p.v.row_stride + (h - p.Hkv) * p.v.head_stride;
    return __ldg(reinterpret_cast<const uint4*>(src) + i);
  };
  // two heads of each kind ahead of their use; the first ones while the row's place is found
  uint4 kv0 = load_kv(slot), kv1 = load_kv(slot + kSlots), q0 = load_q(slot), q1 = load_q(slot + kSlots);
  const RowPlace at = place_row(p.cu_new, p.seq_lens, p.page_table, p.B, r, p.max_new, p.max_pages, p.p_shift, p.n_pages,
                                true, p.rot.rot_dim && !p.tree_mask ? p.rot.n_pos : 0x7fffffff);
  if (at.t < 0) {
    if (tid == 0 && at.flags) atomicOr(p.err, at.flags);
    return;
  }
  int64_t pos = at.t;  // that the rotation turns to
  if (p.tree_mask) {  // a node of a tree: as many behind the tree's base as it has ancestors
    pos = (p.tree_base ? __ldg(p.tree_base + at.b) : at.len) - 1;
    for (int w = 0; w < p.mask_words; ++w) pos += __popc(__ldg(p.tree_mask + static_cast<size_t>(r) * p.mask_words + w));
    if (p.rot.rot_dim && (pos < 0 || pos >= p.rot.n_pos)) {
      if (tid == 0) atomicOr(p.err, kErrSeqOverflow);
      return;
    }
  }
  const Angles ang = load_angles(p.rot, pos, i);
  uint8_t* page = p.pool + static_cast<size_t>(at.pid) * p.page_bytes;
  const int head_bytes = kv4_head_bytes(D, NG, p.P);
  int flags = 0;
  const int warp_slot = (tid & ~31) / kLanes;  // the warp's first slot: its loops end together
#pragma unroll 1
  for (int h0 = 0; h0 + warp_slot < Hkv2; h0 += kSlots) {
    const int hh = h0 + slot;
    const uint4 raw = kv0;
    kv0 = kv1;
    kv1 = load_kv(hh + 2 * kSlots);
    const bool is_k = hh < p.Hkv;
    float x[8];
    if (__any_sync(0xffffffffu, is_k)) rotate8(p.rot, ang, i, raw, F16, x);  // all lanes of the warp
    if (!is_k) unpack8(raw, F16, x);
    uint32_t word;
    float n[8];
    const QParams qp = quantize8<kGroupLanes>(x, word, n);
    uint32_t col = 0;
    if (__any_sync(0xffffffffu, !is_k)) col = even_fields_first(transpose_nibbles(word, i & 7));
    if (hh >= Hkv2) continue;
    const int h = is_k ? hh : hh - p.Hkv;
    flags |= qp.flags;
    uint8_t* region = page + h * head_bytes;
    uint32_t* codes = reinterpret_cast<uint32_t*>(region + (is_k ? 0 : p.P * (D / 2)) + at.tp * (D / 2));
    if (is_k) codes[(i & 3) * (D / 32) + (i >> 2)] = word;
    else codes[(i & 7) * (D / 64) + (i >> 3)] = col;
    if (i % kGroupLanes == 0)
      reinterpret_cast<uint32_t*>(region + p.P * D + (at.tp * NG + i / kGroupLanes) * 8)[is_k ? 0 : 1] = qp.meta;
    uint16_t* deq = is_k ? p.k_deq : p.v_deq;
    if (deq) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 v = add2(mul2(make_float2(n[k], n[k + 1]), make_float2(qp.s, qp.s)), make_float2(qp.m, qp.m));
        n[k] = v.x, n[k + 1] = v.y;
      }
      reinterpret_cast<uint4*>(deq + (static_cast<size_t>(r) * p.Hkv + h) * D)[i] = pack8(n, F16);
    }
  }
#pragma unroll 1
  for (int h0 = 0; h0 + warp_slot < Hq; h0 += kSlots) {
    const int h = h0 + slot;
    const uint4 raw = q0;
    q0 = q1;
    q1 = load_q(h + 2 * kSlots);
    float x[8];
    rotate8(p.rot, ang, i, raw, F16, x);
    if (h < Hq) reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(r) * p.Hq + h) * D)[i] = pack8(x, F16);
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if ((tid & 31) == 0 && flags) atomicOr(p.err, flags);
}

template <int D, int NG, bool F16, int kThreads>
cudaError_t launch_as(const Kv4AppendParams& p, cudaStream_t stream) {
  const int tail = p.seq_next ? (p.B + kThreads - 1) / kThreads : 0;
  kv4_append_kernel<D, NG, F16, kThreads><<<p.n_rows + tail, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// Few rows (decode steps): 256 threads to a row, for its latency. Many: 64, which place the row and
// read its angles less often. 256 and 64 threads, 8 + 8 and 32 heads of 128: 64 rows 5.8 and 11.5 us, 512 rows 8.4 and
// 13.4, 1K 13.0 and 15.8, 2K 23.1 and 22.7; 16K rows 105 with 64.
template <int D, int NG>
cudaError_t launch(const Kv4AppendParams& p, cudaStream_t stream) {
  const bool few = p.n_rows < 2048;
  if (p.f16) return few ? launch_as<D, NG, true, 256>(p, stream) : launch_as<D, NG, true, 64>(p, stream);
  return few ? launch_as<D, NG, false, 256>(p, stream) : launch_as<D, NG, false, 64>(p, stream);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, int D, int n_groups, cudaStream_t stream) {
  if (D == 128) {
    if (n_groups == 1) return launch<128, 1>(p, stream);
    if (n_groups == 2) return launch<128, 2>(p, stream);
    return launch<128, 4>(p, stream);
  }
  return n_groups == 1 ? launch<64, 1>(p, stream) : launch<64, 2>(p, stream);
}

}  // namespace mlaq
