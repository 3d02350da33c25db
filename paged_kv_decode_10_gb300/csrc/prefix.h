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
// (The header in two 16-byte reads, without branches between them.)
__device__ __forceinline__ bool prefix_plan_ok(const PrefixParams &p, int *n_items) {
  const int4 *w = reinterpret_cast<const int4 *>(p.plan);
  const int4 a = w[0], b = w[1];
  *n_items = a.y;
  return (a.x == kSharedMagic) & (a.z == p.B) & (b.x == p.C) & (b.y == p.Hkv) & (b.z == p.G) &
         (a.y >= 0) & (a.y <= (p.plan_ints - plan_items_at(p.B, p.C)) / kPlanItem);
}
__device__ __forceinline__ bool prefix_item(const PrefixParams &p, int i, int max_rows,
                                            PrefixItem *it) {
  const int4 *w = reinterpret_cast<const int4 *>(p.plan + plan_items_at(p.B, p.C) +
                                                 static_cast<size_t>(i) * kPlanItem);
  const int4 a = w[0], b = w[1];
  *it = PrefixItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  return (it->prefix >= 0) & (it->prefix < p.n_prefixes) & (it->g >= 0) & (it->g < p.Hkv) &
         (it->r0 >= 0) & (it->rows > 0) & (it->rows <= max_rows / p.G) &
         (it->r0 <= p.B - it->rows) & (it->t0 >= 0) & (it->t0 % kBlockTokens == 0) &
         (it->t0 < it->t1) & (it->t1 <= 16ll * p.pt_stride) & (it->split >= 0);
}
// Batch row i of an item and the slot its partial goes to (-1: does not fit).
__device__ __forceinline__ int prefix_row(const PrefixParams &p, const PrefixItem &it, int i,
                                          int *slot) {
  const int at = plan_order_at(p.B) + 2 * (it.r0 + i);   // (even: the pair is one 8-byte read)
  const int2 w = *reinterpret_cast<const int2 *>(p.plan + at);
  const bool ok = w.x >= 0 && w.x < p.B && w.y >= 0 && it.split < p.slots - w.y;
  *slot = ok ? w.y + it.split : -1;
  return ok ? w.x : -1;
}

// The form of the whole call for short contexts (shared_short.cu).
struct ShortParams {
  const void *q, *k_cache, *v_cache;
  const int32_t *block_tables, *seq_lens, *prefix_tables, *plan, *mass_lens;   // plan: nullable
  const float *bias;
  float *mass, *lse_out;
  void *out;
  int32_t *err;
  int B, Hq, Hkv, C, num_blocks, n_prefixes, pt_stride, bt_stride, bias_stride;
  int cluster, pages;            // CTAs to a (row, KV head), pages one of them may get
  float scale_log2, decay;
};
constexpr int kShortMaxSmem = 160 * 1024;
int shared_short_cluster(const pkv_shared_args &a, bool prefixes, int *per_cta);
cudaError_t launch_shared_short(const ShortParams &p, int D, int G, int dtype, cudaStream_t s);

cudaError_t launch_prefix_f32(const PrefixParams &p, int D, cudaStream_t s);
cudaError_t launch_prefix_bf16(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                               int D, cudaStream_t s);

}  // namespace pkv
