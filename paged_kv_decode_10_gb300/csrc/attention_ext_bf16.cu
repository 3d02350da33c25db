// EXT builds (prefix partials, scores, row sums) of the split-KV paged decode
// attention kernel: tensor-core consumer, bf16.
#include "attention_kernel.cuh"

namespace pkv {

bool attn_variant_ext_bf16(int D, AttnVariant *v) {
  switch (D) {
    case 64: *v = AttnLauncher<__nv_bfloat16, 64, 4, 16, 0, 8>::variant_ext(); return true;
    case 128: *v = AttnLauncher<__nv_bfloat16, 128, 4, 8, 0, 8>::variant_ext(); return true;
    default: return false;
  }
}

}  // namespace pkv
