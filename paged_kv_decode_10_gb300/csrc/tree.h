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
// 2 c + 1).  The CTA that has an item's first step writes which slots hold the rest
// (TreeCut), and the join kernel combines them, in the order of the tokens.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace pkv {

constexpr int kMaxTreeCtas = 1024;

// Of the item whose first part lies in CTA c's slot 2 c + 1 (more == 0: there is none):
// `more` further parts in slots 2 (c + 1), 2 (c + 2), ...
struct TreeCut {
  int32_t more, q0, rows, g;     // first query row, rows, KV head
  int32_t base, n, pad[2];       // the row's tokens ahead of its nodes, its nodes
};

struct TreeParams {
  const void *q;                 // [T, Hq, D]
  const void *k_cache, *v_cache;
  const int32_t *tables, *lens, *starts;
  const uint32_t *mask;          // nullable [T, mask_words]
  void *out;                     // [T, Hq, D]
  float *lse_out;                // nullable [T, Hq]
  float *part_o, *part_lse;      // [2 C, tile, D], [2 C, tile]
  TreeCut *cuts;                 // [C]
  int32_t *err;
  int B, T, Hq, Hkv, G, num_blocks, bt_stride, mask_words;
  int C, tile;                   // CTAs, rows of an item
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

// Nodes and length of a row; false where they do not fit the call.
__device__ __forceinline__ bool tree_row(const TreeParams &p, int b, int *s0, int *n, int *len) {
  const int a = __ldg(p.starts + b), e = __ldg(p.starts + b + 1);
  *len = __ldg(p.lens + b);
  *s0 = a;
  *n = e - a;
  return a >= 0 && e >= a && e <= p.T && *len >= *n && *len <= 16ll * p.bt_stride &&
         (!p.mask || *n <= 32ll * p.mask_words);
}

// Tokens that the nodes up to `last` of a row may see.
__device__ __forceinline__ int tree_tokens(const TreeParams &p, int n, int len, int last) {
  return p.mask ? len : len - n + min(last, n);
}

// The items of a CTA, in order.  STEP: tokens of a step, BOUND: kBoundary.
template <int STEP, int BOUND>
struct TreeWalk {
  const TreeParams &p;
  long long at, lo, hi, all;     // position of the next item; this CTA's; of the whole call
  int ctas, cta;                 // CTAs with a share
  int b, g, c;                   // the next item
  int s0 = 0, n = 0, len = 0;    // its row
  bool loaded = false;

  static __device__ __forceinline__ int steps_of(int tokens) { return (tokens + STEP - 1) / STEP; }
  // positions of one KV head of a row
  static __device__ __forceinline__ long long head_cost(const TreeParams &p, int n, int len) {
    const int per = p.tile / p.G, tiles = (n + per - 1) / per;
    if (p.mask) return static_cast<long long>(tiles) * (BOUND + steps_of(len));
    long long sum = 0;
    for (int c = 0; c < tiles; ++c) sum += BOUND + steps_of(tree_tokens(p, n, len, (c + 1) * per));
    return sum;
  }

  __device__ __forceinline__ bool next(TreeItem *it) {
    const int per = p.tile / p.G;
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
          const long long head = head_cost(p, n, len);
          g = static_cast<int>(min((lo - at) / head, static_cast<long long>(p.Hkv - 1)));
          at += g * head;
        }
      }
      const int tokens = tree_tokens(p, n, len, (c + 1) * per);
      const int steps = steps_of(tokens);
      const long long first = at + BOUND;
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
      it->t1 = static_cast<int>(min(hi, at) - first);
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
  // CTAs behind this one that have steps of the item that next() gave last.
  __device__ __forceinline__ int more() const {
    return static_cast<int>((at * ctas - 1) / all) - cta;   // (the CTA of its last step)
  }
};

// Where CTA `cta` of p.C begins, found by all NT threads of the CTA together from the
// rows' lengths (rows that do not fit have no positions; CTA 0 reports them).
// MIN: positions a CTA gets at least, while there are CTAs to spare.
template <int STEP, int BOUND, int MIN, int NT>
__device__ __forceinline__ TreeWalk<STEP, BOUND> tree_begin(const TreeParams &p, int cta) {
  using Walk = TreeWalk<STEP, BOUND>;
  __shared__ long long sums[NT / 32], start_at[1];
  __shared__ int start_row[1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.B + NT - 1) / NT, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
  long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    int s0, n, len;
    if (!tree_row(p, b, &s0, &n, &len))
      bad = true;
    else
      mine += p.Hkv * Walk::head_cost(p, n, len);
  }
  if (bad && cta == 0) set_dev_err(p.err, PKV_DEVERR_BAD_LEN);
  long long incl = mine;   // positions up to this thread's rows, them included
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  if (tid == 0) start_row[0] = p.B;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  incl += before;
  long long shares = all / MIN;
  shares = shares < 1 ? 1 : shares;
  const int ctas = static_cast<int>(min(shares, static_cast<long long>(p.C)));
  const long long lo = cta < ctas ? cta * all / ctas : all;
  const long long hi = cta < ctas ? (cta + 1) * all / ctas : all;
  if (lo < hi && incl - mine <= lo && lo < incl) {   // one thread has the row
    long long at = incl - mine;
    for (int b = b0; b < b1; ++b) {
      int s0, n, len;
      const long long cost =
          tree_row(p, b, &s0, &n, &len) ? p.Hkv * Walk::head_cost(p, n, len) : 0;
      if (lo < at + cost) {
        start_row[0] = b;
        start_at[0] = at;
        break;
      }
      at += cost;
    }
  }
  __syncthreads();
  const int row = start_row[0];
  return Walk{p, row < p.B ? start_at[0] : hi, lo, hi, all, ctas, cta, row, 0, 0};
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

cudaError_t launch_tree_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                             const TreeParams &p, int D, cudaStream_t s);

}  // namespace pkv
