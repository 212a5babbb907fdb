// Calls the launch that joins the parts of cut items (csrc/kv4_prompt.cu) on parts that the test lays out itself.
#include <cstdint>

#include "kv4.cuh"

// joined [ctas][5]: kv head, row block, parts, first row, rows. Heads of D, one kv head, `G` query heads on it.
extern "C" int join_parts(int ctas, int rows, int D, int G, const float* part_o, const float* part_ml, const int32_t* joined, int f16,
                          void* out, float* lse, void* stream) {
  static_assert(sizeof(mlaq::Kv4Joined) == 20, "as the test lays it out");
  mlaq::Kv4AttnParams p{};
  p.part_o = const_cast<float*>(part_o);
  p.part_ml = const_cast<float*>(part_ml);
  p.joined = reinterpret_cast<mlaq::Kv4Joined*>(const_cast<int32_t*>(joined));
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.Hq = p.G = G;
  p.Hkv = 1;
  p.f16 = f16 != 0;
  mlaq::Kv4PromptPlan z{};
  z.rows = rows;
  z.line = 1;
  z.ctas = ctas;
  return static_cast<int>(mlaq::launch_kv4_join(p, z, D, static_cast<cudaStream_t>(stream)));
}
