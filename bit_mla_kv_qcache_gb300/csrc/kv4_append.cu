// Append of new K/V rows to the grouped-query cache in 4 bits, keys (and the step's queries)
// rotated to their positions on the way.
//
// A thread holds eight channels of one head (one 16-byte load); the D / 8 threads of a head are
// neighbouring lanes. Rotation partners and group statistics are lane shuffles, a key-code word is
// one thread's eight channels, and a value-code word is a column of the 8 x 8 matrix of codes that
// eight lanes hold (transposed by three rounds of exchanges). CTA r serves row r: its threads
// cover 2048 / D heads at a time and keep the row's angles in registers over all heads. Bound:
// the bytes of the rows, read and written once.
#include "append.cuh"
#include "quant.cuh"

namespace mlaq {
namespace {

constexpr int kAppendThreads = 256;

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

// Quantizes the group that this lane's eight values belong to (LG lanes per group).
template <int LG>
__device__ __forceinline__ QParams quantize8(const float (&x)[8], uint32_t& word, float (&val)[8], int& flags) {
  float lo = x[0], hi = x[0], zero = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    lo = fminf(lo, x[k]);
    hi = fmaxf(hi, x[k]);
    zero = __fadd_rn(zero, __fmul_rn(x[k], 0.f));  // NaN if a value is NaN or infinite
  }
#pragma unroll
  for (int o = 1; o < LG; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const QParams qp = make_qparams(lo, hi, 15);
  flags |= qp.flags | (zero == 0.f ? 0 : kErrNonFinite);
  word = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = quant_code4(x[k], qp);
    word |= static_cast<uint32_t>(c) << (4 * k);
    val[k] = __fadd_rn(__fmul_rn(static_cast<float>(c), qp.s), qp.m);
  }
  return qp;
}

template <int D, int NG>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int kLanes = D / 8;                       // threads of one head
  constexpr int kSlots = kAppendThreads / kLanes;     // heads at a time
  constexpr int kGroupLanes = kLanes / NG;
  constexpr int kLoads = 4;                           // heads of a thread that are read at once
  const int tid = threadIdx.x, i = tid % kLanes, slot = tid / kLanes;
  const int r = blockIdx.x;
  if (r >= p.n_rows) {  // the blocks behind the rows: the new lengths
    const int b = (r - p.n_rows) * kAppendThreads + tid;
    if (b < p.B) p.seq_next[b] = __ldg(p.seq_lens + b) + __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
    return;
  }
  const int Hq = p.q.data ? p.Hq : 0, total = Hq + 2 * p.Hkv;  // queries, then keys, then values
  uint4 raw[kLoads];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int hh = h0 + u * kSlots + slot;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (hh < total) {
        const HeadView& src = hh < Hq ? p.q : hh < Hq + p.Hkv ? p.k : p.v;
        const int h = hh < Hq ? hh : hh < Hq + p.Hkv ? hh - Hq : hh - Hq - p.Hkv;
        raw[u] = __ldg(reinterpret_cast<const uint4*>(src.data + r * src.row_stride + h * src.head_stride) + i);
      }
    }
  };
  load(0);  // on their way while the row's place is found
  const RowPlace at = place_row(p.cu_new, p.seq_lens, p.page_table, p.B, r, p.max_new, p.max_pages, p.p_shift, p.n_pages,
                                true, p.rot.rot_dim ? p.rot.n_pos : 0x7fffffff);
  if (at.t < 0) {
    if (tid == 0 && at.flags) atomicOr(p.err, at.flags);
    return;
  }
  const Angles ang = load_angles(p.rot, at.t, i);
  uint8_t* page = p.pool + static_cast<size_t>(at.pid) * p.page_bytes;
  const int head_bytes = kv4_head_bytes(D, NG, p.P);
  int flags = 0;
  for (int h0 = 0; h0 < total; h0 += kLoads * kSlots) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int hh = h0 + u * kSlots + slot;
      if (h0 + u * kSlots >= total) break;
      const bool is_q = hh < Hq, is_k = !is_q && hh < Hq + p.Hkv, live = hh < total;
      const int h = is_q ? hh : is_k ? hh - Hq : hh - Hq - p.Hkv;
      float x[8];
      rotate8(p.rot, ang, i, raw[u], p.f16, x);  // all lanes of the warp, whatever head each one holds
      if (!is_q && !is_k) unpack8(raw[u], p.f16, x);
      if (is_q) reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(r) * p.Hq + h) * D)[i] = pack8(x, p.f16);
      if (__all_sync(0xffffffffu, is_q)) continue;
      uint32_t word;
      float val[8];
      int fl = 0;
      const QParams qp = quantize8<kGroupLanes>(x, word, val, fl);
      const uint32_t col = even_fields_first(transpose_nibbles(word, i & 7));
      if (!live || is_q) continue;
      flags |= fl;
      uint8_t* region = page + h * head_bytes;
      uint32_t* codes = reinterpret_cast<uint32_t*>(region + (is_k ? 0 : p.P * (D / 2)) + at.tp * (D / 2));
      if (is_k) codes[(i & 3) * (D / 32) + (i >> 2)] = word;
      else codes[(i & 7) * (D / 64) + (i >> 3)] = col;
      if (i % kGroupLanes == 0)
        reinterpret_cast<uint32_t*>(region + p.P * D + (at.tp * NG + i / kGroupLanes) * 8)[is_k ? 0 : 1] = qp.meta;
      uint16_t* deq = is_k ? p.k_deq : p.v_deq;
      if (deq) reinterpret_cast<uint4*>(deq + (static_cast<size_t>(r) * p.Hkv + h) * D)[i] = pack8(val, p.f16);
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if ((tid & 31) == 0 && flags) atomicOr(p.err, flags);
}

template <int D, int NG>
cudaError_t launch(const Kv4AppendParams& p, cudaStream_t stream) {
  const int tail = p.seq_next ? (p.B + kAppendThreads - 1) / kAppendThreads : 0;
  kv4_append_kernel<D, NG><<<p.n_rows + tail, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
