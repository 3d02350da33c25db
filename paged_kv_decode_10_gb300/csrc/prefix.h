// The prefix part of pkv_decode_attn_shared: parameters of its kernels.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "shared_plan.h"

namespace pkv {

struct PrefixParams {
  const void *q;                 // [B, Hq, D] rotated queries
  const void *k_cache, *v_cache;
  const int32_t *tables;         // [n_prefixes, pt_stride]
  const int32_t *plan;
  float *o, *lse;                // partials: [slots, Hq, D] normalised, [slots, Hq] base 2
  int32_t *err;
  int B, Hq, Hkv, G, num_blocks, n_prefixes, pt_stride, plan_ints, slots, C;
  float scale_log2;
  long long wait_limit;
};

// One work item as the plan states it, checked against the call: false (and
// PKV_DEVERR_BAD_PLAN) when it does not fit, and the item is then skipped.
struct PrefixItem {
  int prefix, g, r0, rows, t0, t1, split;
};
__device__ __forceinline__ bool prefix_plan_ok(const PrefixParams &p) {
  return p.plan[0] == kSharedMagic && p.plan[2] == p.B && p.plan[4] == p.C &&
         p.plan[5] == p.Hkv && p.plan[6] == p.G && p.plan[1] >= 0 &&
         p.plan[1] <= (p.plan_ints - plan_items_at(p.B, p.C)) / kPlanItem;
}
__device__ __forceinline__ bool prefix_item(const PrefixParams &p, int i, int max_rows,
                                            PrefixItem *it) {
  const int4 *w = reinterpret_cast<const int4 *>(p.plan + plan_items_at(p.B, p.C) +
                                                 static_cast<size_t>(i) * kPlanItem);
  const int4 a = w[0], b = w[1];
  *it = PrefixItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  return it->prefix >= 0 && it->prefix < p.n_prefixes && it->g >= 0 && it->g < p.Hkv &&
         it->r0 >= 0 && it->rows > 0 && it->rows * p.G <= max_rows && it->r0 <= p.B - it->rows &&
         it->t0 >= 0 && it->t0 % kBlockTokens == 0 && it->t0 < it->t1 && it->t1 <= 16ll * p.pt_stride && it->split >= 0;
}
// Batch row i of an item and the slot its partial goes to (-1: does not fit).
__device__ __forceinline__ int prefix_row(const PrefixParams &p, const PrefixItem &it, int i,
                                          int *slot) {
  const int row = p.plan[plan_order_at(p.B) + it.r0 + i];
  *slot = -1;
  if (row < 0 || row >= p.B) return -1;
  const int s0 = p.plan[plan_rows_at() + 2 * row], n = p.plan[plan_rows_at() + 2 * row + 1];
  if (s0 < 0 || it.split >= n || s0 > p.slots - n) return -1;
  *slot = s0 + it.split;
  return row;
}

cudaError_t launch_prefix_f32(const PrefixParams &p, int D, cudaStream_t s);
cudaError_t launch_prefix_bf16(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                               int D, cudaStream_t s);

}  // namespace pkv
