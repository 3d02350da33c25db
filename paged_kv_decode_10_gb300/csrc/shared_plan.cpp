// Host planner of the shared-prefix attention (pkv_shared_plan): rows grouped by
// prefix, prefixes split along their tokens, work items dealt to CTAs.
//
// An item is up to 256 query rows (64 in float32) x one KV head x a range of a
// prefix's tokens.  Splitting a prefix into s ranges fills the GPU, but every
// row then leaves s partials (float32, d values a head) that are written and
// read again, so s is chosen by trying the useful values and estimating
//   makespan of the items, dealt longest first to the least loaded CTA
//   + the partials' bytes at the rate L2 takes them.
#ifndef __CUDACC__
#define __host__
#define __device__
#endif
#include <algorithm>
#include <cstdint>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "shared_plan.h"
#include "status.h"

namespace pkv {
int current_sms(int *sms);   // attention.cu
}

namespace {

constexpr int kMaxB = 65536;

struct Bounds {
  int64_t items, slots;
};

// What a plan may use at most: one item and one slot per row tile, plus what
// splitting over twice the CTAs adds.
Bounds bounds(int32_t B, int32_t n_prefixes, int32_t Hq, int32_t Hkv, int32_t C) {
  const int64_t G = Hq / Hkv;
  const int64_t tiles = std::min<int64_t>(
      B, (B * G + pkv::kTileRowsF32 - 1) / pkv::kTileRowsF32 + n_prefixes);
  Bounds b;
  b.items = tiles * Hkv + 2 * static_cast<int64_t>(C);
  b.slots = B + (2 * static_cast<int64_t>(C) + Hkv - 1) / Hkv * std::min<int64_t>(B, 128);
  return b;
}

int check(int32_t B, int32_t n_prefixes, int32_t Hq, int32_t Hkv, int32_t *num_ctas) {
  PKV_REQUIRE(B >= 0 && B <= kMaxB, PKV_ERR_UNSUPPORTED, "B = %d (max %d)", B, kMaxB);
  PKV_REQUIRE(n_prefixes >= 0, PKV_ERR_INVALID_ARG, "n_prefixes < 0");
  PKV_REQUIRE(Hkv > 0 && Hq > 0 && Hq % Hkv == 0, PKV_ERR_INVALID_ARG,
              "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  const int G = Hq / Hkv;
  PKV_REQUIRE(G == 1 || G == 2 || G == 4 || G == 8, PKV_ERR_UNSUPPORTED,
              "group size %d (built: 1, 2, 4, 8)", G);
  PKV_REQUIRE(*num_ctas <= pkv::kMaxPlanCtas, PKV_ERR_INVALID_ARG, "num_ctas must be <= %d",
              pkv::kMaxPlanCtas);
  if (*num_ctas <= 0) {
    int sms = 0;
    const int rc = pkv::current_sms(&sms);
    if (rc != PKV_OK) return rc;
    *num_ctas = sms;
  }
  return PKV_OK;
}

}  // namespace

extern "C" int pkv_shared_plan_cap(int32_t B, int32_t n_prefixes, int32_t Hq, int32_t Hkv,
                                   int32_t num_ctas, int32_t *plan_cap, int32_t *max_slots) {
  pkv::clear_error();
  PKV_REQUIRE(plan_cap && max_slots, PKV_ERR_INVALID_ARG, "NULL output");
  const int rc = check(B, n_prefixes, Hq, Hkv, &num_ctas);
  if (rc != PKV_OK) return rc;
  const Bounds b = bounds(B, n_prefixes, Hq, Hkv, num_ctas);
  const int64_t cap = pkv::plan_items_at(B, num_ctas) + b.items * pkv::kPlanItem;
  PKV_REQUIRE(cap < (int64_t(1) << 31) && b.slots < (int64_t(1) << 31), PKV_ERR_UNSUPPORTED,
              "plan too large");
  *plan_cap = static_cast<int32_t>(cap);
  *max_slots = static_cast<int32_t>(b.slots);
  return PKV_OK;
}

extern "C" int pkv_shared_plan(const int32_t *row_prefix, int32_t B, const int32_t *prefix_lens,
                               int32_t n_prefixes, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t dtype, int32_t num_ctas, int32_t *plan, int32_t plan_cap,
                               int32_t *plan_ints, int32_t *slots) {
  pkv::clear_error();
  PKV_REQUIRE(plan && plan_ints && slots, PKV_ERR_INVALID_ARG, "NULL output");
  PKV_REQUIRE(dtype == PKV_F32 || dtype == PKV_BF16, PKV_ERR_UNSUPPORTED, "dtype %d", dtype);
  PKV_REQUIRE(d == 64 || d == 128, PKV_ERR_UNSUPPORTED, "head_dim %d (built: 64, 128)", d);
  int rc = check(B, n_prefixes, Hq, Hkv, &num_ctas);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE((B == 0 || row_prefix) && (n_prefixes == 0 || prefix_lens), PKV_ERR_INVALID_ARG,
              "NULL argument");
  for (int32_t p = 0; p < n_prefixes; ++p)
    PKV_REQUIRE(prefix_lens[p] >= 0 && prefix_lens[p] < (1 << 30), PKV_ERR_INVALID_ARG,
                "prefix %d: length %d", p, prefix_lens[p]);
  for (int32_t b = 0; b < B; ++b)
    PKV_REQUIRE(row_prefix[b] < n_prefixes, PKV_ERR_INVALID_ARG, "row %d: prefix %d of %d", b,
                row_prefix[b], n_prefixes);
  const int32_t C = num_ctas, G = Hq / Hkv;
  const int32_t R = (dtype == PKV_BF16 ? pkv::kTileRowsBf16 : pkv::kTileRowsF32) / G;
  const int32_t grain = dtype == PKV_BF16 ? pkv::kSplitTokens : pkv::kSplitTokensF32;
  const Bounds bd = bounds(B, n_prefixes, Hq, Hkv, C);
  const int64_t items_at = pkv::plan_items_at(B, C);
  PKV_REQUIRE(plan_cap >= items_at, PKV_ERR_INVALID_ARG, "plan_cap %d < %lld", plan_cap,
              (long long)items_at);
  try {
    // rows grouped by prefix, each group in row order
    std::vector<int32_t> first(static_cast<size_t>(n_prefixes) + 1, 0);
    for (int32_t b = 0; b < B; ++b)
      if (row_prefix[b] >= 0 && prefix_lens[row_prefix[b]] > 0) ++first[row_prefix[b] + 1];
    for (int32_t p = 0; p < n_prefixes; ++p) first[p + 1] += first[p];
    std::vector<int32_t> order(first[n_prefixes]);
    {
      std::vector<int32_t> at(first.begin(), first.end() - 1);
      for (int32_t b = 0; b < B; ++b)
        if (row_prefix[b] >= 0 && prefix_lens[row_prefix[b]] > 0) order[at[row_prefix[b]]++] = b;
    }
    struct Group {
      int32_t p, rows, tiles, grains;
    };
    std::vector<Group> groups;
    int32_t longest = 0;
    for (int32_t p = 0; p < n_prefixes; ++p) {
      const int32_t rows = first[p + 1] - first[p];
      if (rows == 0) continue;
      const int32_t gr = (prefix_lens[p] + grain - 1) / grain;
      groups.push_back({p, rows, (rows + R - 1) / R, gr});
      longest = std::max(longest, gr);
    }
    // time estimates, ns: a grain of tokens for one item, an item's fixed cost.  (Half
    // of what a grain takes alone on an SM: weighed at its full time, or with idle
    // SMs credited, the choice came out longer ranges, which lost 4 % on 256 rows of
    // five prefixes and nothing was gained elsewhere.)
    auto grain_ns = [&](int32_t rows) {
      const double q = static_cast<double>(rows) * G, w = d / 128.0;
      if (dtype == PKV_F32) return 500.0 / (pkv::kSplitTokens / pkv::kSplitTokensF32) * w * q;
      return (q > 128 ? 1100.0 : 700.0) * (d == 128 ? 1.0 : 0.7);
    };
    const double fixed_ns = 3000.0;
    auto tile_rows = [&](const Group &g, int32_t t) {
      // even shares, so that no tile is left with a remainder of a few rows
      const int32_t a = static_cast<int32_t>(static_cast<int64_t>(g.rows) * t / g.tiles);
      const int32_t e = static_cast<int32_t>(static_cast<int64_t>(g.rows) * (t + 1) / g.tiles);
      return std::pair<int32_t, int32_t>(a, e);
    };
    std::vector<double> costs;
    double best = -1.0;
    int32_t best_c = std::max(longest, 1), last_c = -1;
    for (int32_t j = 1; j <= std::min(longest, 256); ++j) {
      const int32_t c = (longest + j - 1) / j;
      if (c == last_c) continue;
      last_c = c;
      int64_t n = 0, ns = 0;
      for (const Group &g : groups) {
        const int64_t s = (g.grains + c - 1) / c;
        n += static_cast<int64_t>(g.tiles) * Hkv * s;
        ns += static_cast<int64_t>(g.rows) * s;
      }
      if (j > 1 && (n > bd.items || ns > bd.slots)) break;
      costs.clear();
      for (const Group &g : groups) {
        const int32_t s = (g.grains + c - 1) / c;
        const double len = static_cast<double>(g.grains) / s;
        for (int32_t t = 0; t < g.tiles; ++t) {
          const auto r = tile_rows(g, t);
          for (int64_t k = 0; k < static_cast<int64_t>(Hkv) * s; ++k)
            costs.push_back(fixed_ns + len * grain_ns(r.second - r.first));
        }
      }
      std::sort(costs.begin(), costs.end(), std::greater<double>());
      std::priority_queue<double, std::vector<double>, std::greater<double>> load;
      for (int32_t i = 0; i < C; ++i) load.push(0.0);
      double span = 0.0;
      for (double x : costs) {
        const double l = load.top() + x;
        load.pop();
        load.push(l);
        span = std::max(span, l);
      }
      const double est = span + static_cast<double>(ns) * Hq * d * 8.0 / 5000.0;
      if (best < 0.0 || est < best) {
        best = est;
        best_c = c;
      }
    }
    // the plan itself
    struct Item {
      int32_t v[pkv::kPlanItem];
      double cost;
    };
    std::vector<Item> items;
    int32_t *rows_out = plan + pkv::plan_rows_at();
    for (int32_t b = 0; b < B; ++b) {
      const int32_t len = row_prefix[b] < 0 ? 0 : prefix_lens[row_prefix[b]];
      rows_out[4 * b] = rows_out[4 * b + 1] = 0;
      rows_out[4 * b + 2] = len > 0 ? row_prefix[b] : -1;
      rows_out[4 * b + 3] = len;
    }
    int64_t slot = 0;
    for (const Group &g : groups) {
      const int32_t s = (g.grains + best_c - 1) / best_c;
      const int32_t L = prefix_lens[g.p];
      for (int32_t i = 0; i < g.rows; ++i) {
        const int32_t b = order[first[g.p] + i];
        rows_out[4 * b] = static_cast<int32_t>(slot);
        rows_out[4 * b + 1] = s;
        slot += s;
      }
      for (int32_t t = 0; t < g.tiles; ++t) {
        const auto r = tile_rows(g, t);
        for (int32_t k = 0; k < s; ++k) {
          const int32_t a = static_cast<int32_t>(static_cast<int64_t>(g.grains) * k / s);
          const int32_t e = static_cast<int32_t>(static_cast<int64_t>(g.grains) * (k + 1) / s);
          for (int32_t h = 0; h < Hkv; ++h) {
            Item it{{g.p, h, first[g.p] + r.first, r.second - r.first, a * grain,
                     std::min(L, e * grain), k, 0},
                    fixed_ns + (e - a) * grain_ns(r.second - r.first)};
            items.push_back(it);
          }
        }
      }
    }
    const int64_t n = static_cast<int64_t>(items.size());
    PKV_REQUIRE(n <= bd.items && slot <= bd.slots &&
                    items_at + n * pkv::kPlanItem <= plan_cap,
                PKV_ERR_INVALID_ARG, "plan_cap %d < %lld", plan_cap,
                (long long)(items_at + n * pkv::kPlanItem));
    // longest first, each to the CTA with the least so far (the lowest of equals)
    std::vector<int32_t> by(n);
    for (int64_t i = 0; i < n; ++i) by[i] = static_cast<int32_t>(i);
    std::stable_sort(by.begin(), by.end(),
                     [&](int32_t x, int32_t y) { return items[x].cost > items[y].cost; });
    using Load = std::pair<double, int32_t>;
    std::priority_queue<Load, std::vector<Load>, std::greater<Load>> load;
    for (int32_t i = 0; i < C; ++i) load.push({0.0, i});
    std::vector<std::vector<int32_t>> of(C);
    for (int32_t i : by) {
      const Load l = load.top();
      load.pop();
      of[l.second].push_back(i);
      load.push({l.first + items[i].cost, l.second});
    }
    int32_t *order_out = plan + pkv::plan_order_at(B);
    for (int32_t i = 0; i < B; ++i) {
      const int32_t b = i < static_cast<int32_t>(order.size()) ? order[i] : -1;
      order_out[2 * i] = b;
      order_out[2 * i + 1] = b < 0 ? 0 : rows_out[4 * b];
    }
    int32_t *ctas = plan + pkv::plan_ctas_at(B);
    int32_t *out = plan + items_at;
    int32_t at = 0;
    for (int32_t c = 0; c < C; ++c) {
      ctas[c] = at;
      for (int32_t i : of[c]) {
        std::copy(items[i].v, items[i].v + pkv::kPlanItem, out + static_cast<int64_t>(at) * pkv::kPlanItem);
        ++at;
      }
    }
    ctas[C] = at;
    for (int64_t i = pkv::plan_ctas_at(B) + C + 1; i < items_at; ++i) plan[i] = 0;
    for (int i = 0; i < pkv::kPlanHead; ++i) plan[i] = 0;
    plan[0] = pkv::kSharedMagic;
    plan[1] = at;
    plan[2] = B;
    plan[3] = static_cast<int32_t>(slot);
    plan[4] = C;
    plan[5] = Hkv;
    plan[6] = G;
    plan[7] = R;
    *plan_ints = static_cast<int32_t>(items_at + n * pkv::kPlanItem);
    *slots = static_cast<int32_t>(slot);
  } catch (...) {
    return pkv::fail(PKV_ERR_INVALID_ARG, "out of host memory");
  }
  return PKV_OK;
}
