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
  int32_t *status;               // [C] what each CTA did, stored by every call
  int32_t *err;
  int B, Hq, Hkv, G, num_blocks, n_prefixes, pt_stride, plan_ints, slots, C;
  float scale_log2;
  long long wait_limit;
};

// A CTA's status: the (row, KV head) partials of its items, or why some of them may be
// from an earlier call.  The join reads the status of all CTAs and takes partials only if
// they add up to the plan's.
enum : int32_t {
  kPrefixSkipped = -1,   // an item or a row that does not fit
  kPrefixGaveUp = -2,    // a wait did
};

// The plan's header, checked against the call (in two 16-byte reads, without branches
// between them).
struct PlanHeader {
  int items, slots;
  bool ok;
};
__device__ __forceinline__ PlanHeader plan_header(const int32_t *plan, int B, int C, int Hkv, int G,
                                                  int plan_ints, int slots) {
  const int4 *w = reinterpret_cast<const int4 *>(plan);   // (L2: the join reads ahead of its wait)
  const int4 a = __ldcg(w), b = __ldcg(w + 1);
  const bool ok = (a.x == kSharedMagic) & (a.z == B) & (b.x == C) & (b.y == Hkv) & (b.z == G) &
                  (a.y >= 0) & (a.y <= (plan_ints - plan_items_at(B, C)) / kPlanItem) & (a.w >= 0) &
                  (a.w <= slots);
  return PlanHeader{a.y, a.w, ok};
}
// A row's record (first slot, partials, prefix or -1, its length), checked against the call:
// a row whose record does not fit has no prefix.
__device__ __forceinline__ bool plan_row_ok(const int4 &r, int n_prefixes, int pt_stride, int slots) {
  return (r.z < n_prefixes) & (r.w >= 0) & (r.w <= kBlockTokens * pt_stride) & (r.x >= 0) &
         (r.y >= 0) & (r.y <= slots - r.x);
}

// One work item as the plan states it, checked against the call.  Where it does not fit,
// PKV_DEVERR_BAD_PLAN is set and it is not computed: kItemUnread names partials of rows
// whose prefix lies outside the call's tables (they become "no token"), kItemBad nothing.
struct PrefixItem {
  int prefix, g, r0, rows, t0, t1, split;
};
enum : int { kItemBad, kItemUnread, kItemOk };
__device__ __forceinline__ int prefix_item(const PrefixParams &p, int i, int max_rows,
                                           PrefixItem *it) {
  const int4 *w = reinterpret_cast<const int4 *>(p.plan + plan_items_at(p.B, p.C) +
                                                 static_cast<size_t>(i) * kPlanItem);
  const int4 a = w[0], b = w[1];
  *it = PrefixItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  const bool named = (it->g >= 0) & (it->g < p.Hkv) & (it->r0 >= 0) & (it->rows > 0) &
                     (it->rows <= max_rows / p.G) & (it->r0 <= p.B - it->rows) & (it->split >= 0) &
                     (it->prefix >= 0) & (it->t0 >= 0) & (it->t0 % kBlockTokens == 0) &
                     (it->t0 < it->t1);
  const bool there = (it->prefix < p.n_prefixes) & (it->t1 <= 16ll * p.pt_stride);
  return !named ? kItemBad : there ? kItemOk : kItemUnread;
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
// kItemUnread: its partials as of no token (by `threads` threads; false if a row does not
// fit).
__device__ __forceinline__ bool prefix_unread(const PrefixParams &p, const PrefixItem &it, int tid,
                                              int threads) {
  bool ok = true;
  for (int e = tid; e < it.rows * p.G; e += threads) {
    int slot;
    if (prefix_row(p, it, e / p.G, &slot) < 0)
      ok = false;
    else
      p.lse[static_cast<size_t>(slot) * p.Hq + it.g * p.G + e % p.G] = -INFINITY;
  }
  return ok;
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
