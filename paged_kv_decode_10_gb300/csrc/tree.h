// The attention of drafted tokens (pkv_decode_attn_tree): parameters of its kernels, and
// how its work is dealt to CTAs.
//
// Work.  The queries of one row's nodes (tokens of the row that have a query) under one
// KV head are the rows of a matrix: node i, head h of the group is row i * G + h.  An item
// is up to `tile` such rows against all tokens that they may see, kStep tokens at a time.
// Items lie end to end in the order row, KV head, row tile, as positions: kBoundary for
// what an item costs by itself, one for each step.  CTA c of C owns positions
// [floor(c P / C), floor((c + 1) P / C)) and the steps in them, so the work is shared
// evenly whatever the lengths, and every CTA finds its share from the lengths alone:
// no plan, no counters, the same partition in every call.
//
// An item whose steps lie in one CTA is finished there.  Of the others every CTA leaves a
// partial (float32 output, base-2 log-sum-exp) in a slot of its own: a CTA has at most
// two cut items, the one it begins with (slot 2 c) and the one it ends with (slot
// 2 c + 1), and writes for each slot which item and which CTAs it belongs to (TreeCut).  The
// join kernel combines an item's parts in the order of the tokens, every slot's share of
// its rows on its own, so that an item of many parts is joined by many.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace pkv {

constexpr int kMaxTreeCtas = 1024;

// A slot's item: its parts lie in slot 2 first + 1 and slots 2 (first + 1), ...,
// 2 (first + parts - 1); parts == 0: the slot is not used.
struct alignas(16) TreeCut {
  int32_t parts, first, q0, rows;   // first query row, rows
  int32_t g, base, n, pad;          // KV head; the row's tokens ahead of its nodes, its nodes
};

struct TreeParams {
  const void *q;                 // [T, Hq, D]
  const void *k_cache, *v_cache;
  const int32_t *tables, *lens, *starts;
  const uint32_t *mask;          // nullable [T, mask_words]
  void *out;                     // [T, Hq, D]
  float *lse_out;                // nullable [T, Hq]
  float *part_o, *part_lse;      // [2 C, tile, D], [2 C, tile]
  TreeCut *cuts;                 // [2 C]
  int32_t *err;
  int B, T, Hq, Hkv, G, num_blocks, bt_stride, mask_words;
  int C, tile, lg_nodes, lg_g;   // CTAs, rows of an item, log2 of the nodes that these are, of G
  float scale_log2;
  long long wait_limit;
};

struct TreeItem {
  int b, g, n0, nodes, q0;       // batch row, KV head, first node and nodes, first query row
  int base, n, tokens;           // the row's tokens ahead of its nodes, its nodes; tokens the item sees
  int t0, t1, steps;             // this CTA's steps of the item's
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == steps; }
  __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 == 0 ? 1 : 0); }
};

// Nodes and length of a row; false where they do not fit the call.  (Plain loads: constant
// ones, which depend on nothing, might be moved ahead of the wait for the grid before.)
__device__ __forceinline__ bool tree_row(const TreeParams &p, int b, int *s0, int *n, int *len) {
  const int a = p.starts[b], e = p.starts[b + 1];
  *len = p.lens[b];
  *s0 = a;
  *n = e - a;
  return a >= 0 && e >= a && e <= p.T && *len >= *n && *len <= 16ll * p.bt_stride &&
         (!p.mask || *n <= 32ll * p.mask_words);
}

// Tokens that the nodes up to `last` of a row may see.
__device__ __forceinline__ int tree_tokens(const TreeParams &p, int n, int len, int last) {
  return p.mask ? len : len - n + min(last, n);
}

// Positions of one KV head of a row (0 for a row without nodes).  STEP: tokens of a step,
// BOUND: what an item costs by itself.
template <int STEP, int BOUND>
__device__ __forceinline__ unsigned long long tree_head_cost(const TreeParams &p, int n, int len) {
  const uint32_t tiles = (static_cast<uint32_t>(n) + (1u << p.lg_nodes) - 1) >> p.lg_nodes;
  if (p.mask) return static_cast<unsigned long long>(tiles) * (BOUND + (len + STEP - 1) / STEP);
  unsigned long long sum = static_cast<unsigned long long>(tiles) * BOUND;
  for (uint32_t c = 1; c <= tiles; ++c)
    sum += (tree_tokens(p, n, len, static_cast<int>(c << p.lg_nodes)) + STEP - 1) / STEP;
  return sum;
}

// Writes down a cut item's CTAs: it ends ahead of position `end` of `all`, shared by `ctas`
// CTAs.  (A function, for its 64-bit divisions: inline, they took the kernels 1 to 2 % longer.)
static __device__ __noinline__ void tree_cut(const TreeParams &p, const TreeItem it, int cta, uint32_t end,
                                      uint32_t all, uint32_t ctas) {
  // the CTA that has the step at position x
  auto owner = [&](uint32_t x) {
    return static_cast<int>((static_cast<unsigned long long>(x + 1) * ctas - 1) / all);
  };
  const int from = owner(end - it.steps);
  p.cuts[it.slot(cta)] =
      TreeCut{owner(end - 1) - from + 1, from, it.q0, it.nodes * p.G, it.g, it.base, it.n, 0};
}

// The items of a CTA, in order.  (32 bits: a call of 2^31 positions and more is refused.)
template <int STEP, int BOUND>
struct TreeWalk {
  uint32_t at, lo, hi;           // position of the next item; this CTA's
  uint32_t all, ctas;            // of the whole call, CTAs with a share
  int cta;
  int b, g, c;                   // the next item
  int s0, n, len;                // its row
  bool loaded;

  __device__ __forceinline__ bool next(const TreeParams &p, TreeItem *it) {
    const int per = 1 << p.lg_nodes;
    while (at < hi) {
      if (!loaded) {
        if (b >= p.B) return false;
        if (!tree_row(p, b, &s0, &n, &len) || n == 0) {
          ++b;
          continue;
        }
        loaded = true;
        g = c = 0;
        if (at < lo) {   // (the first row: whole heads ahead of the CTA's share)
          const uint32_t head = static_cast<uint32_t>(tree_head_cost<STEP, BOUND>(p, n, len));
          while (g + 1 < p.Hkv && at + head <= lo) {
            at += head;
            ++g;
          }
        }
      }
      const int tokens = tree_tokens(p, n, len, (c + 1) * per);
      const int steps = (tokens + STEP - 1) / STEP;
      const uint32_t first = at + BOUND;
      it->b = b;
      it->g = g;
      it->n0 = c * per;
      it->nodes = min(per, n - c * per);
      it->q0 = s0 + it->n0;
      it->base = len - n;
      it->n = n;
      it->tokens = tokens;
      it->steps = steps;
      at = first + steps;
      it->t0 = static_cast<int>(max(lo, first) - first);
      it->t1 = static_cast<int>(min(hi, at)) - static_cast<int>(first);
      if ((c + 1) * per < n) {
        ++c;
      } else {
        c = 0;
        if (++g == p.Hkv) {
          ++b;
          loaded = false;
        }
      }
      if (it->t0 < it->t1) return true;
    }
    return false;
  }
};

// A CTA's share of `sum` positions: floor(c all / ctas) by 32-bit divisions.  (The rest
// dealt to the first CTAs, one each, instead of evenly, took 3 % longer.)  A call of fewer
// positions than CTAs leaves the rest of them without any.
template <int STEP, int BOUND>
__device__ __forceinline__ TreeWalk<STEP, BOUND> tree_share(const TreeParams &p, int cta,
                                                            unsigned long long sum, bool bad) {
  const bool fits = sum < 1ull << 31;
  const uint32_t all = fits ? static_cast<uint32_t>(sum) : 0;
  if (cta == 0 && (bad || !fits)) set_dev_err(p.err, PKV_DEVERR_BAD_LEN);
  const uint32_t ctas = max(1u, min(all, static_cast<uint32_t>(p.C)));
  const uint32_t share = all / ctas, rest = all - share * ctas;
  const uint32_t c = min(static_cast<uint32_t>(cta), ctas), c1 = min(c + 1, ctas);
  const uint32_t lo = c * share + c * rest / ctas, hi = c1 * share + c1 * rest / ctas;
  return TreeWalk<STEP, BOUND>{hi, lo, hi, all, ctas, cta, p.B, 0, 0, 0, 0, 0, false};
}
template <int STEP, int BOUND>
__device__ __forceinline__ unsigned long long tree_row_cost(const TreeParams &p, int b, bool *bad) {
  int s0, n, len;
  if (!tree_row(p, b, &s0, &n, &len)) {
    *bad = true;
    return 0;
  }
  return tree_head_cost<STEP, BOUND>(p, n, len) * p.Hkv;
}
__device__ __forceinline__ unsigned long long warp_sum_up(unsigned long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Where CTA `cta` of p.C begins, from the rows' lengths (rows that do not fit have no
// positions; CTA 0 reports them): found by one warp, for batches of at most 32 rows ...
constexpr int kWarpRows = 32;
template <int STEP, int BOUND>
__device__ __forceinline__ TreeWalk<STEP, BOUND> tree_begin_warp(const TreeParams &p, int cta) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  const unsigned long long mine = lane < p.B ? tree_row_cost<STEP, BOUND>(p, lane, &bad) : 0;
  const unsigned long long incl = warp_sum_up(mine, lane);
  auto walk = tree_share<STEP, BOUND>(p, cta, __shfl_sync(0xffffffffu, incl, 31),
                                           __any_sync(0xffffffffu, bad));
  const uint32_t row =   // the lane that has the first position
      __ballot_sync(0xffffffffu, walk.lo < walk.hi && incl - mine <= walk.lo && walk.lo < incl);
  if (row) {
    walk.b = __ffs(row) - 1;
    walk.at = static_cast<uint32_t>(__shfl_sync(0xffffffffu, incl - mine, walk.b));
  }
  return walk;
}
// ... or by all NT threads of the CTA together.
template <int STEP, int BOUND, int NT>
__device__ __forceinline__ TreeWalk<STEP, BOUND> tree_begin(const TreeParams &p, int cta) {
  __shared__ unsigned long long sums[NT / 32];
  __shared__ int start[2];   // first row, its position
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = p.B <= NT ? 1 : (p.B + NT - 1) / NT;
  const int b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
  unsigned long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) mine += tree_row_cost<STEP, BOUND>(p, b, &bad);
  bad = __any_sync(0xffffffffu, bad);
  if (bad && cta == 0 && lane == 0) set_dev_err(p.err, PKV_DEVERR_BAD_LEN);
  const unsigned long long incl = warp_sum_up(mine, lane);
  if (lane == 31) sums[warp] = incl;
  if (tid == 0) start[0] = p.B;
  __syncthreads();
  unsigned long long before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sums[w];
    sum += sums[w];
  }
  auto walk = tree_share<STEP, BOUND>(p, cta, sum, false);
  unsigned long long at = before + incl - mine;
  if (walk.lo < walk.hi && at <= walk.lo && walk.lo < at + mine) {   // one thread has the row
    int b = b0;
    for (; b + 1 < b1; ++b) {   // (more rows than threads)
      const unsigned long long rows = tree_row_cost<STEP, BOUND>(p, b, &bad);
      if (walk.lo < at + rows) break;
      at += rows;
    }
    start[0] = b;
    start[1] = static_cast<int>(at);
  }
  __syncthreads();
  walk.b = start[0];
  if (walk.b < p.B) walk.at = static_cast<uint32_t>(start[1]);
  return walk;
}

// 32 visibility bits of a query row: tokens tok .. tok + 31 of its row, bit j for token
// tok + j (node: the node's number in its row, words: its mask or NULL for a chain).
__device__ __forceinline__ uint32_t tree_sees(const uint32_t *words, int n_words, int node, int base,
                                              int tokens, int tok) {
  uint32_t w;
  const int j = tok - base;   // node of the first token
  if (j <= -32) {
    w = 0xffffffffu;
  } else if (!words) {
    const int last = node - j;   // of the 32, the last one that it sees
    w = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
  } else {
    const int i = j >> 5;        // (rounds down)
    const uint32_t lo = i < 0 ? 0xffffffffu : i < n_words ? __ldg(words + i) : 0u;
    const uint32_t hi = i + 1 < n_words ? __ldg(words + i + 1) : 0u;
    w = __funnelshift_r(lo, hi, j & 31);
  }
  const int left = tokens - tok;
  return left >= 32 ? w : left <= 0 ? 0u : w & ((1u << left) - 1u);
}

// Whether a node of a row of n sees any token at all (where all its scores are -inf the
// formula gives NaN, and zeros only where it sees nothing).
__device__ __forceinline__ bool tree_sees_any(const TreeParams &p, int q_row, int base, int n) {
  if (base > 0 || !p.mask) return true;
  const uint32_t *w = p.mask + static_cast<size_t>(q_row) * p.mask_words;
  for (int i = 0; 32 * i < n; ++i)
    if (w[i] & (n - 32 * i >= 32 ? 0xffffffffu : (1u << (n - 32 * i)) - 1u)) return true;
  return false;
}
// What a row's normaliser becomes: 1 / den, 0 for a row without tokens, NaN for one whose
// scores are all -inf or not numbers.
__device__ __forceinline__ float tree_inverse(float den, bool sees_any) {
  return den > 0.f ? 1.f / den : den == 0.f && !sees_any ? 0.f : __int_as_float(0x7fffffff);
}
// Natural log-sum-exp from the largest base-2 score and the sum relative to it.
__device__ __forceinline__ float tree_lse(float mx, float den, bool sees_any) {
  return den > 0.f ? (mx + log2f(den)) * 0.6931471805599453f
                   : den == 0.f && !sees_any ? -INFINITY : __int_as_float(0x7fffffff);
}

// After a wait that gave up (by all NT threads of the CTA): no output of it counts.
template <typename T, int D, int STEP, int BOUND, int NT>
__device__ __noinline__ void tree_all_nan(const TreeParams &p) {
  const int cta = blockIdx.x;
  auto walk = tree_begin<STEP, BOUND, NT>(p, cta);
  TreeItem it;
  const float nan = __int_as_float(0x7fffffff);
  while (walk.next(p, &it)) {
    // (what was not come to was not written down either)
    if (!it.whole() && threadIdx.x == 0) tree_cut(p, it, cta, walk.at, walk.all, walk.ctas);
    for (int e = threadIdx.x; e < it.nodes * p.G; e += NT) {
      if (!it.whole()) {   // (the join makes NaN of it)
        p.part_lse[static_cast<size_t>(it.slot(cta)) * p.tile + e] = INFINITY;
        continue;
      }
      const size_t at = static_cast<size_t>(it.q0 + e / p.G) * p.Hq + it.g * p.G + e % p.G;
      if (p.lse_out) p.lse_out[at] = nan;
      for (int c = 0; c < D; ++c) static_cast<T *>(p.out)[at * D + c] = from_f32<T>(nan);
    }
  }
}

cudaError_t launch_tree_f32(const TreeParams &p, int D, cudaStream_t s);
cudaError_t launch_tree_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                             const TreeParams &p, int D, cudaStream_t s);

}  // namespace pkv
