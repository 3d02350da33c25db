// Layout of a shared-prefix plan (pkv_shared_plan), shared by the host planner
// and the kernels that read it (not part of the C ABI).
#pragma once
#include <stdint.h>

namespace pkv {

// int32 words: a header of kPlanHead, [B][4] (first partial slot, partials, prefix or
// -1, its length) per row, [B][2] the rows grouped by prefix (row, first partial slot), [C + 1] first
// item of every CTA, then (at a multiple of 4) items of kPlanItem words.
constexpr int32_t kSharedMagic = 0x53506c31;
constexpr int kPlanHead = 16;   // magic, items, B, slots, C, Hkv, G, rows per tile
constexpr int kMaxPlanCtas = 4096;
constexpr int kPlanItem = 8;    // prefix, KV head, first in the row list, rows, t0, t1, split

inline __host__ __device__ int plan_rows_at() { return kPlanHead; }
inline __host__ __device__ int plan_order_at(int B) { return kPlanHead + 4 * B; }
inline __host__ __device__ int plan_ctas_at(int B) { return kPlanHead + 6 * B; }
inline __host__ __device__ int plan_items_at(int B, int C) {
  return (kPlanHead + 6 * B + C + 1 + 3) / 4 * 4;
}

// Query rows (batch rows x group heads) one work item covers at most.
constexpr int kTileRowsBf16 = 256;
constexpr int kTileRowsF32 = 64;
// Prefixes are split at multiples of this many tokens (a step of the kernels).
constexpr int kSplitTokens = 128;
constexpr int kSplitTokensF32 = 32;

}  // namespace pkv
