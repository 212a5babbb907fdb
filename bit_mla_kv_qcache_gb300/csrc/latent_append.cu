// Append of new latent rows to the paged BF16 cache (the one the unquantized decode reads): RMS
// norm of the latent, rotation of the positional key and of the queries' positional part.
//
// CTA r serves row r. Warp 0 normalizes the latent (sixteen channels per lane, sum of squares in
// float32 over the warp); the other warps rotate the positional key and the queries, eight lanes
// per head of 64 channels. Bound: the bytes of the rows, read and written once.
#include "append.cuh"

namespace mlaq {
namespace {

constexpr int kLatThreads = 128;

__global__ void __launch_bounds__(kLatThreads) latent_append_kernel(const LatentAppendParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x;
  if (r >= p.n_rows) {  // the blocks behind the rows: the new lengths
    const int b = (r - p.n_rows) * kLatThreads + tid;
    if (b < p.B) p.seq_next[b] = __ldg(p.seq_lens + b) + __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
    return;
  }
  const uint16_t* row = p.kv.data + r * p.kv.row_stride;
  const int n_pos = p.rot.rot_dim ? p.rot.n_pos : 0x7fffffff;
  if (warp == 0) {
    uint4 w[2], g[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // on their way while the row's place is found
      w[k] = __ldg(reinterpret_cast<const uint4*>(row) + lane + 32 * k);
      g[k] = p.weight ? __ldg(reinterpret_cast<const uint4*>(p.weight) + lane + 32 * k) : make_uint4(0, 0, 0, 0);
    }
    const RowPlace at = place_row(p.cu_new, p.seq_lens, p.page_table, p.B, r, p.max_new, p.max_pages, p.p_shift, p.n_pages,
                                  p.pool != nullptr, n_pos);
    if (at.t < 0) {
      if (lane == 0 && at.flags) atomicOr(p.err, at.flags);
      return;
    }
    if (p.weight) {
      float x[2][8], ss = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        unpack8(w[k], false, x[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x[k][j] * x[k][j];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = 1.f / sqrtf(ss * (1.f / kLatent) + p.eps);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float y[8];
        unpack8(g[k], false, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[k][j] = x[k][j] * inv * y[j];
        w[k] = pack8(x[k], false);
      }
    }
    uint16_t* dst = p.pool ? p.pool + (static_cast<size_t>(at.pid) * p.P + at.tp) * kRow : nullptr;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (dst) reinterpret_cast<uint4*>(dst)[lane + 32 * k] = w[k];
      if (p.c_out) reinterpret_cast<uint4*>(p.c_out + static_cast<size_t>(r) * kLatent)[lane + 32 * k] = w[k];
    }
    return;
  }
  constexpr int kSlots = (kLatThreads - 32) / 8, kLoads = 4;
  const int i = tid & 7, slot = (tid - 32) / 8;
  const int heads = 1 + (p.q.data ? p.H : 0);  // the positional key, then the queries
  uint4 raw[kLoads];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int h = h0 + u * kSlots + slot;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (h < heads)
        raw[u] = __ldg(reinterpret_cast<const uint4*>(
                           h == 0 ? row + kLatent : p.q.data + r * p.q.row_stride + (h - 1) * p.q.head_stride) + i);
    }
  };
  load(0);
  const RowPlace at = place_row(p.cu_new, p.seq_lens, p.page_table, p.B, r, p.max_new, p.max_pages, p.p_shift, p.n_pages,
                                p.pool != nullptr, n_pos);
  if (at.t < 0) return;  // warp 0 reports it
  const Angles ang = load_angles(p.rot, at.t, i);
  for (int h0 = 0; h0 < heads; h0 += kLoads * kSlots) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int h = h0 + u * kSlots + slot;
      if (h0 + u * kSlots >= heads) break;
      float x[8];
      rotate8(p.rot, ang, i, raw[u], false, x);
      const uint4 y = pack8(x, false);
      if (h == 0) {
        if (p.pool)
          reinterpret_cast<uint4*>(p.pool + (static_cast<size_t>(at.pid) * p.P + at.tp) * kRow + kLatent)[i] = y;
        if (p.kr_out) reinterpret_cast<uint4*>(p.kr_out + static_cast<size_t>(r) * kRope)[i] = y;
      } else if (h < heads) {
        reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(r) * p.H + h - 1) * kRope)[i] = y;
      }
    }
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream) {
  const int tail = p.seq_next ? (p.B + kLatThreads - 1) / kLatThreads : 0;
  latent_append_kernel<<<p.n_rows + tail, kLatThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mlaq
