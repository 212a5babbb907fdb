// Attention over the 4-bit grouped-query cache for many query rows per kv head: rows of a sequence's last positions.
#include "kv4_prompt.cuh"

namespace mlaq {

bool kv4_uses_prompt(int max_q, int G) { return static_cast<int64_t>(max_q) * G > 32; }

// An item is worth cutting, which costs a schedule, a second store and a join, when its tokens are many. 48 items
// of 256 rows, one CTA each against cut: 2K tokens 39 and 43 us, 3K 53 and 47, 8K 122 and 72; four of 40 rows: 1K 20 and 25, 2K 30
// and 26. Between a half and all of the SMs whole items fill one wave and a cut makes two (96 items, 8K: 123 and 126 us).
// Up to twice the SMs a cut fills the second wave: 192 items, 4K: 103 and 104, 8K: 215 and 173 us. The lengths are on
// the device: the room of the page table stands for them here, and there short items stay whole.
Kv4PromptPlan kv4_prompt_plan(int B, int Hkv, int n_rows, int max_q, int64_t max_tokens, int G, int num_sms) {
  Kv4PromptPlan z;
  const int64_t rows = static_cast<int64_t>(std::min(max_q, n_rows)) * G;
  z.rows = rows > 128 ? 256 : rows > 64 ? 128 : 64;
  const int64_t items = static_cast<int64_t>(B) * Hkv * ((rows + z.rows - 1) / z.rows);
  const int64_t blocks = (rows + z.rows - 1) / z.rows;
  const bool cut = 2 * items <= num_sms ? max_tokens > 2048 : items > num_sms && items < 2 * num_sms && max_tokens > 4096;
  z.line = cut && B * blocks <= kThreads ? static_cast<int>(blocks) : 0;
  z.ctas = z.line ? std::min(num_sms, static_cast<int>(kKv4CounterBytes / 4)) : items;
  return z;
}

size_t kv4_prompt_workspace_bytes(const Kv4PromptPlan& z, int D) {
  return kKv4CounterBytes + (z.line ? static_cast<size_t>(z.ctas) * (2 * z.rows * (static_cast<size_t>(D) + 2) * sizeof(float) + sizeof(Kv4Joined)) : 0);
}

namespace {

// Joins the parts of the items that were cut: D / 4 lanes to a row of the item that CTA blockIdx.x began, a lane to four columns. By
// the CTA that came last, within the kernel, this took 18 us for 9 parts of 256 rows and 5 for parts of 64: one SM reads 1.2 MB no
// faster. As a launch of its own it takes 10 and 6 with its start (64 nodes of a document of 64K: 141 -> 124 us with the quicker
// sharing of the work; 40 rows of eight sequences up to 32K: 79 -> 80).
constexpr int kJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnParams p, const int R) {
  constexpr int kLanes = D / 4, VW = D / 64, kPer = kMaxParts / kLanes, kBatch = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  const int lane = threadIdx.x % kLanes, c0 = static_cast<int>(blockIdx.x);
  const int row = (static_cast<int>(blockIdx.y) * kJoinThreads + static_cast<int>(threadIdx.x)) / kLanes;  // of the block
  const unsigned group = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  auto slot_of = [&](int i) { return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)); };  // of the CTA's two: the item that it begins
  const Kv4Joined it = p.joined[c0];
  float2 ml[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = lane + k * kLanes;
    ml[k] = c0 + i < static_cast<int>(gridDim.x) ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(i) * R + row) : make_float2(kNoMax, 0.f);
  }
  if (it.parts < 2 || it.rb * R + row >= it.rows) return;  // (all lanes of the row)
  const int parts = min(min(it.parts, kMaxParts), static_cast<int>(gridDim.x) - c0);
  float M = kNoMax, L = 0.f;
  bool whole = true;  // an item with a part that is not there stays as it is
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (lane + k * kLanes >= parts) ml[k] = make_float2(kNoMax, 0.f);
    else whole &= !(ml[k].y < 0.f);
    M = fmaxf(M, ml[k].x);
  }
  if (!__all_sync(group, whole)) return;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(group, M, o, kLanes));
  float w[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    w[k] = ex2(ml[k].x - M);
    L += w[k] * ml[k].y;
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) L += __shfl_xor_sync(group, L, o, kLanes);
  const float y = L == 0.f ? 0.f : 1.f / L;
  const int q2 = it.rb * R + row;
  const size_t out_row = static_cast<size_t>(it.r0 + q2 / p.G) * p.Hq + it.h * p.G + q2 % p.G;
  if (lane == 0 && p.lse) p.lse[out_row] = L == 0.f ? -INFINITY : (M + (log2f(L) - kRoom)) * 0.69314718055994531f;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const float4* const src = reinterpret_cast<const float4*>(p.part_o) + static_cast<size_t>(row) * kLanes + lane;
  for (int i0 = 0; i0 < parts; i0 += kBatch) {
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < parts) x[i] = __ldcg(src + slot_of(i0 + i) * R * kLanes);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= parts) break;
      float f = __shfl_sync(group, w[0], (i0 + i) % kLanes, kLanes);
      if constexpr (kPer > 1) {
        const float g = __shfl_sync(group, w[kPer - 1], (i0 + i) % kLanes, kLanes);
        if (i0 + i >= kLanes) f = g;
      }
      v[0] += f * x[i].x, v[1] += f * x[i].y, v[2] += f * x[i].z, v[3] += f * x[i].w;
    }
  }
  // Channel 64 a + 16 i + 8 e + b is column 8 (b VW + a) + 2 i + e: a lane stores four neighbouring channels, which four lanes hold.
  const int a = lane / 16, i = lane / 4 % 4, e = lane / 2 % 2;
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int from = 2 * ((4 * (lane & 1) + j) * VW + a) + (i >> 1);
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __shfl_sync(group, v[k], from, kLanes);
    z[j] = y * ((i & 1) ? (e ? t[3] : t[2]) : (e ? t[1] : t[0]));
  }
  reinterpret_cast<uint2*>(p.out + out_row * D)[lane] = make_uint2(pack2(z[0], z[1], p.f16), pack2(z[2], z[3], p.f16));
}

}  // namespace

cudaError_t launch_kv4_join(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, cudaStream_t stream) {
  cudaLaunchAttribute early{};  // launched while the kernel before it ends
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t at{};
  at.gridDim = dim3(static_cast<unsigned>(z.ctas), z.rows * (D / 4) / kJoinThreads);
  at.blockDim = dim3(kJoinThreads);
  at.stream = stream;
  at.attrs = &early;
  at.numAttrs = 1;
  return D == 128 ? cudaLaunchKernelEx(&at, kv4_join_kernel<128>, p, z.rows) : cudaLaunchKernelEx(&at, kv4_join_kernel<64>, p, z.rows);
}

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  return launch_prompt_kernel<false, false>(p, z, D, n_groups, stream);
}

}  // namespace mlaq
