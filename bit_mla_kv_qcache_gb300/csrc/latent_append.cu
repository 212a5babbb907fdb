// Append of new latent rows to the paged BF16 cache (the one the unquantized decode reads): RMS
// norm of the latent, rotation of the positional key and of the queries' positional part.
//
// With few rows a CTA of four warps serves one: warp 0 normalizes the latent (sixteen channels per lane,
// sum of squares in float32 over the warp), the others rotate the positional key and the queries, eight
// lanes per head of 64 channels. With many, each warp serves a row of its own, which is placed once and
// whose angles are read once. Bound: for many rows the latency of a row's loads (16K rows with 16 heads 18 us, their
// bytes, read and written once, 10 at the card's copy rate; issue 52%, long waits on loads); for a decode step the launch and
// three dependent loads (32 rows 2.8 us).
#include "append.cuh"

namespace mlaq {
namespace {

constexpr int kLatThreads = 128;

// kWarps: warps of one row, 1 or 4.
template <int kWarps>
__global__ void __launch_bounds__(kLatThreads, 8) latent_append_kernel(const LatentAppendParams p, const int row_ctas) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) >= row_ctas) {  // the blocks behind the rows: the new lengths
    const int b = (blockIdx.x - row_ctas) * kLatThreads + tid;
    if (b < p.B) p.seq_next[b] = __ldg(p.seq_lens + b) + __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
    return;
  }
  const int r = kWarps == 4 ? blockIdx.x : blockIdx.x * 4 + (tid >> 5), sub = kWarps == 4 ? tid >> 5 : 0;
  if (r >= p.n_rows) return;
  const uint16_t* row = p.kv.data + r * p.kv.row_stride;
  const bool latent = sub == 0, turns = kWarps == 1 || sub > 0;
  // the first loads are on their way while the row's place is found
  uint4 w[2];
  if (latent) {
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(row) + lane + 32 * k);
  }
  constexpr int kSlots = kWarps == 4 ? 12 : 4, kLoads = kWarps == 4 ? 2 : 5;  // heads at a time; of those, asked for at once
  const int i = lane & 7, slot = (kWarps == 4 ? 4 * (sub - 1) : 0) + (lane >> 3);
  const int heads = 1 + (p.q.data ? p.H : 0);  // the positional key, then the queries
  uint4 raw[kLoads];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int h = h0 + u * kSlots + slot;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (turns && h < heads)
        raw[u] = __ldg(reinterpret_cast<const uint4*>(
                           h == 0 ? row + kLatent : p.q.data + r * p.q.row_stride + (h - 1) * p.q.head_stride) + i);
    }
  };
  load(0);
  const RowPlace at = place_row(p.cu_new, p.seq_lens, p.page_table, p.B, r, p.max_new, p.max_pages, p.p_shift, p.n_pages,
                                p.pool != nullptr, p.rot.rot_dim ? p.rot.n_pos : 0x7fffffff);
  if (at.t < 0) {
    if (latent && lane == 0 && at.flags) atomicOr(p.err, at.flags);
    return;
  }
  uint16_t* const dst = p.pool ? p.pool + (static_cast<size_t>(at.pid) * p.P + at.tp) * kRow : nullptr;
  if (latent) {
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
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight) + lane + 32 * k), false, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[k][j] = x[k][j] * inv * g[j];
        w[k] = pack8(x[k], false);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (dst) reinterpret_cast<uint4*>(dst)[lane + 32 * k] = w[k];
      if (p.c_out) reinterpret_cast<uint4*>(p.c_out + static_cast<size_t>(r) * kLatent)[lane + 32 * k] = w[k];
    }
  }
  if (!turns) return;
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
        if (dst) reinterpret_cast<uint4*>(dst + kLatent)[i] = y;
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
  // Four warps to a row and one, 16 heads: 256 rows 3.0 and 3.8 us, 1K 3.5 and 4.0, 2K 5.4 and 4.9, 4K 9.1 and 6.2
  // (below 2K rows a warp to a row leaves SMs idle).
  if (p.n_rows < 2048) {
    latent_append_kernel<4><<<p.n_rows + tail, kLatThreads, 0, stream>>>(p, p.n_rows);
  } else {
    const int ctas = (p.n_rows + 3) / 4;
    latent_append_kernel<1><<<ctas + tail, kLatThreads, 0, stream>>>(p, ctas);
  }
  return cudaGetLastError();
}

}  // namespace mlaq
