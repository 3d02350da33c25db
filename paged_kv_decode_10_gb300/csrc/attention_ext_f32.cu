// EXT builds (prefix partials, scores, row sums) of the split-KV paged decode
// attention kernel: CUDA-core consumer, float32.
#include "attention_kernel.cuh"

namespace pkv {

bool attn_variant_ext_f32(int D, int G, AttnVariant *v) {
  using T = float;
  if (G <= 2) G = 2;
  if (D == 64) {
    if (G == 2) { *v = AttnLauncher<T, 64, 4, 8, 1, 2>::variant_ext(); return true; }
    if (G == 4) { *v = AttnLauncher<T, 64, 4, 8, 1, 4>::variant_ext(); return true; }
    if (G == 8) { *v = AttnLauncher<T, 64, 4, 8, 1, 8>::variant_ext(); return true; }
  } else if (D == 128) {
    if (G == 2) { *v = AttnLauncher<T, 128, 4, 4, 1, 2>::variant_ext(); return true; }
    if (G == 4) { *v = AttnLauncher<T, 128, 4, 4, 1, 4>::variant_ext(); return true; }
    if (G == 8) { *v = AttnLauncher<T, 128, 4, 4, 1, 8>::variant_ext(); return true; }
  }
  return false;
}

}  // namespace pkv
