// pkv_decode_attn_shared: attention over shared prefixes and own tokens, with the
// weights of the own tokens accumulated per cache slot.
//
// Launches: the prefix kernel (partials of every row over its prefix), the EXT
// build of the split-KV kernel over the rows' own tokens (a programmatic
// dependent of the prefix kernel that reads nothing of it, so it fills whatever
// SMs that one leaves), the merge of the two and, with mass, the fold of the
// scores.  Without prefixes only the second and the last.  Short contexts take one
// launch of another kernel (shared_short.cu).
//
// Each kernel is launched behind the one before as its programmatic dependent and
// waits for it before it reads what it left.
//
// The merge is a kernel of its own because joining the partials in the split-KV
// kernel's epilogue made its consumers wait, first for the prefix kernel and then
// for chains of partial reads, while no page was streamed: that took 31 us of the
// 122 us which the kernel needed for 64 rows of 1..4096 tokens (32/8 heads of 128)
// behind an 8192-token prefix.
#include <cuda.h>

#include "attention_host.h"
#include "attention_kernel.cuh"
#include "prefix.h"

namespace pkv {
namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct SharedSpace {
  size_t lse2, own_lse, own_o, status, pre_lse, pre_o, bytes;   // offsets behind the attention workspace
};

SharedSpace shared_space(size_t attn_bytes, int B, int Hq, int d, int slots) {
  SharedSpace s;
  s.lse2 = align256(attn_bytes);
  s.own_lse = s.lse2 + align256(static_cast<size_t>(B) * Hq * sizeof(float));
  s.own_o = s.own_lse + align256(static_cast<size_t>(B) * Hq * sizeof(float));
  s.status = s.own_o + (slots > 0 ? align256(static_cast<size_t>(B) * Hq * d * sizeof(float)) : 0);
  s.pre_lse = s.status + (slots > 0 ? kMaxPlanCtas * sizeof(int32_t) : 0);
  s.pre_o = s.pre_lse + align256(static_cast<size_t>(slots) * Hq * sizeof(float));
  s.bytes = s.pre_o + align256(static_cast<size_t>(slots) * Hq * d * sizeof(float));
  return s;
}

// ---- prefix partials and own tokens joined -------------------------------------
// out = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M) over the own tokens' partial
// and the row's n prefix partials (merge_acc_add).  D / 4 lanes own one (row, head),
// a float4 column each; the reads of eight partials go out together.  Bound by L2
// latency: the partials were just written (64 rows of 32 heads of 128, 17 MB: 6 us
// behind the kernel before it).
//
// The partials count only if every one of the plan's was stored by this call's prefix
// kernel, which its CTAs' status tells: otherwise what lies there may be an earlier
// call's.  A plan that does not fit leaves the rows their own tokens; where a wait gave
// up, the rows behind prefixes are NaN.
struct JoinParams {
  const int32_t *plan, *status;
  const float *own_o, *own_lse, *pre_o, *pre_lse;
  void *out;
  float *lse2, *lse_out;
  int32_t *err;
  int rows, B, Hq, Hkv, C, n_prefixes, pt_stride, plan_ints, slots;   // rows: B * Hq
};

template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  pdl_launch_dependents();
  constexpr int LPR = D / 4, K = 8;
  __shared__ uint32_t sums[8], flags[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at_row = blockIdx.x * (256 / LPR) + tid / LPR, d4 = tid % LPR;
  const bool on_row = at_row < p.rows;
  const int u = on_row ? at_row : 0;
  const int b = u / p.Hq, h = u - b * p.Hq;
  const PlanHeader head = plan_header(p.plan, p.B, p.C, p.Hkv, p.Hq / p.Hkv, p.plan_ints, p.slots);
  const int4 part = __ldcg(reinterpret_cast<const int4 *>(p.plan + plan_rows_at() + 4 * b));
  const bool fits = head.ok && plan_row_ok(part, p.n_prefixes, p.pt_stride, head.slots);
  const int n = fits ? part.y : 0;
  pdl_wait();   // the partials come from the kernels before this one
  uint32_t done = 0;
  int worst = 0;
  if (warp == 0)
    for (int c0 = 0; c0 < p.C; c0 += 256) {
      int s[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = c0 + 32 * q + lane < p.C ? __ldcg(p.status + c0 + 32 * q + lane) : 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        done += static_cast<uint32_t>(max(s[q], 0));
        worst |= s[q] == kPrefixGaveUp ? 2 : s[q] < 0 ? 1 : 0;
      }
    }
  MergeAcc a{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  float l1[1] = {__ldcg(p.own_lse + u)};
  float4 v1[1] = {__ldcg(reinterpret_cast<const float4 *>(p.own_o + static_cast<size_t>(u) * D) + d4)};
  for (int i0 = 0; i0 < n; i0 += K) {
    float l[K];
    float4 v[K];
#pragma unroll
    for (int t = 0; t < K; ++t) {
      const bool on = i0 + t < n;
      const size_t at = static_cast<size_t>(part.x + (on ? i0 + t : 0)) * p.Hq + h;
      l[t] = on ? __ldcg(p.pre_lse + at) : -INFINITY;
      v[t] = __ldcg(reinterpret_cast<const float4 *>(p.pre_o + at * D) + d4);
    }
    merge_acc_add<K>(a, l, v);
  }
  // (the status last: the partials' reads need not wait for it)
  if (warp == 0) {
    done = __reduce_add_sync(0xffffffffu, done);
    worst = __reduce_or_sync(0xffffffffu, worst);
    if (lane == 0) {
      sums[0] = done;
      flags[0] = worst;
    }
  }
  __syncthreads();
  done = sums[0];
  worst = flags[0];
  // (both sides modulo 2^32)
  const bool whole = worst == 0 && done == static_cast<uint32_t>(head.slots) * p.Hkv;
  if (!whole || !fits) {
    a = MergeAcc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (worst < 2 && d4 == 0 && on_row) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
  }
  merge_acc_add<1>(a, l1, v1);
  if (worst >= 2 && n > 0) a.den = __int_as_float(0x7fffffff);
  if (!on_row) return;
  keep_nan(a);
  merge_store<T>(static_cast<T *>(p.out) + static_cast<size_t>(u) * D, d4, D, a);
  if (d4 == 0) {
    const float l2 = a.den > 0.f ? a.M + log2f(a.den) : -INFINITY;
    if (p.lse2) p.lse2[u] = l2;
    if (p.lse_out) p.lse_out[u] = l2 * 0.6931471805599453f;
  }
}

// ---- the weights of the own tokens --------------------------------------------
// Token t of row b has base-2 scores s_h for the G heads of a KV head and the row
// sums 2^lse_h over prefix and own tokens: its weight is sum_h 2^(s_h - lse_h).
// A CTA takes pages_per_cta pages of one row; an item is one (page, KV head,
// token): the scores of consecutive items lie side by side, as do the weights.
// Memory bound: 4 G + 8 bytes a token and KV head, mostly from L2 (64 rows of 1..4096
// tokens, 32/8 heads: 25 MB, 14 us behind the attention kernel; 760 looping CTAs in place
// of one grid over all pages took 3 us more).
struct MassParams {
  const float *scores, *lse2;
  float *mass;
  const int32_t *block_tables, *seq_lens, *mass_lens;
  int bt_stride, bias_stride, Hq, Hkv, num_blocks, chunks, has_bias;
  float decay;
};
constexpr int kMassPages = 8;

template <int G>
__global__ void __launch_bounds__(256, 5) mass_kernel(const MassParams p) {
  constexpr int kBatch = G == 8 ? 2 : 4;   // items of a thread whose reads are under way together
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x - b * p.chunks;
  // Lengths, tables and the weights so far are read ahead of the wait, which takes 2 us off
  // (103 against 105; mass_prefix_f32 34.7 against 36.7).  They were there before the first
  // kernel of the call went on from its own wait, flushed to L2, from where they are read.
  const int L = __ldcg(p.seq_lens + b);
  bool bad;
  const int n = pages_of_len(L, p.bt_stride, p.has_bias != 0, p.bias_stride, &bad);
  const int known = p.mass_lens ? __ldcg(p.mass_lens + b) : L - 1;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const int per_page = p.Hkv * kBlockTokens;
  bool waited = false;
  for (int j0 = chunk * kMassPages; j0 < n; j0 += p.chunks * kMassPages) {
    const int j1 = min(n, j0 + kMassPages);
    // this thread's items, 256 apart, by page and place (no division in the loop)
    int j = j0 + threadIdx.x / per_page, r = threadIdx.x % per_page;
    while (j < j1) {
      int heads[kBatch];
      int at[kBatch];   // cache row of the item, -1: nothing to do
      float old[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        at[u] = -1;
        heads[u] = r / kBlockTokens;
        const int t = j * kBlockTokens + r % kBlockTokens;
        const int blk = j < j1 ? __ldcg(table + j) : -1;
        if (t < L && blk >= 0 && blk < p.num_blocks) {   // (others: flagged by the attention kernel)
          at[u] = blk * per_page + r;   // (the pool has fewer than 2^31 rows)
          old[u] = t < known ? p.decay * __ldcg(p.mass + at[u]) : 0.f;
        }
        r += 256;
        while (r >= per_page) {
          r -= per_page;
          ++j;
        }
      }
      if (!waited) pdl_wait();   // scores and row sums come from the kernels before this one
      waited = true;
      float s[kBatch][G];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (at[u] < 0) continue;
        const float *src = p.scores + static_cast<size_t>(at[u]) * G;
        if constexpr (G >= 4) {
#pragma unroll
          for (int q = 0; q < G / 4; ++q)
            reinterpret_cast<float4 *>(s[u])[q] = __ldcs(reinterpret_cast<const float4 *>(src) + q);
        } else {
#pragma unroll
          for (int q = 0; q < G; ++q) s[u][q] = __ldcs(src + q);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (at[u] < 0) continue;
        const float *l = p.lse2 + static_cast<size_t>(b) * p.Hq + heads[u] * G;
        float w = 0.f;
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const float x = __ldcg(l + q);
          w += x == -INFINITY ? 0.f : ex2(s[u][q] - x);
        }
        p.mass[at[u]] = old[u] + w;
      }
    }
  }
  if (!waited) pdl_wait();   // (what follows this kernel follows those before it)
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_shared_default_parts(int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                                        int32_t dtype, int32_t bt_stride, int32_t *num_parts) {
  clear_error();
  PKV_REQUIRE(num_parts, PKV_ERR_INVALID_ARG, "num_parts is NULL");
  PKV_REQUIRE(bt_stride > 0 && bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              bt_stride);
  int rc = check_shapes(B, Hq, Hkv, d, dtype);
  if (rc != PKV_OK) return rc;
  int most = 0;
  rc = default_parts(d, dtype, 0, Hq / Hkv, &most);
  if (rc != PKV_OK) return rc;
  // Parts of one page cost their prologue and a merge each: 4 rows of up to 64 tokens
  // behind a 500-token prefix (8/2 heads of 64) take 28.8 us in 304 parts, 14.4 in 16,
  // 12.3 in 8.
  const long long positions =
      static_cast<long long>(B) * Hkv * (static_cast<long long>(bt_stride) + seg_cost(d));
  const long long parts = (positions + 7) / 8;
  *num_parts = parts < 1 ? 1 : parts < most ? static_cast<int>(parts) : most;
  return PKV_OK;
}

extern "C" int pkv_shared_short(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                                int32_t bt_stride, int32_t pt_stride, int32_t *short_form) {
  clear_error();
  PKV_REQUIRE(short_form, PKV_ERR_INVALID_ARG, "short_form is NULL");
  const int rc = check_shapes(B, Hq, Hkv, d, dtype);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(bt_stride >= 0 && pt_stride >= 0, PKV_ERR_INVALID_ARG, "negative width");
  pkv_shared_args a = {};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.dtype = dtype;
  a.bt_stride = bt_stride;
  a.pt_stride = pt_stride;
  int per_cta = 0;
  *short_form = shared_short_cluster(a, pt_stride > 0, &per_cta) > 0;
  return PKV_OK;
}

extern "C" int pkv_shared_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                                          int32_t num_parts, int32_t slots, size_t *bytes) {
  size_t attn = 0;
  const int rc = pkv_attn_workspace_bytes(B, Hq, Hkv, d, num_parts, &attn);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(bytes, PKV_ERR_INVALID_ARG, "bytes is NULL");
  PKV_REQUIRE(slots >= 0, PKV_ERR_INVALID_ARG, "slots < 0");
  *bytes = shared_space(attn, B, Hq, d, slots).bytes;
  return PKV_OK;
}

extern "C" int pkv_decode_attn_shared(const pkv_shared_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  int rc = check_shapes(a->B, a->Hq, a->Hkv, a->d, a->dtype);
  if (rc != PKV_OK) return rc;
  if (a->B == 0) return PKV_OK;
  const int G = a->Hq / a->Hkv;
  PKV_REQUIRE((a->flags & ~(PKV_ATTN_CHECK_PLAN | PKV_ATTN_SHORT_WAITS)) == 0, PKV_ERR_UNSUPPORTED,
              "flags %d", a->flags);
  PKV_REQUIRE(a->q_rot && a->k_cache && a->v_cache && a->block_tables && a->seq_lens && a->out &&
                  a->workspace,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  const long long out_bytes =
      static_cast<long long>(a->B) * a->Hq * a->d * static_cast<long long>(dtype_size(a->dtype));
  PKV_REQUIRE(!rows_overlap(a->out, 0, out_bytes, a->q_rot, 0, out_bytes, 1), PKV_ERR_INVALID_ARG,
              "out must not overlap q_rot");
  PKV_REQUIRE(std::isfinite(a->scale), PKV_ERR_INVALID_ARG, "scale must be finite");
  PKV_REQUIRE(a->num_blocks > 0, PKV_ERR_INVALID_ARG, "num_blocks must be positive");
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->k_cache) & 15) == 0 &&
                  (reinterpret_cast<uintptr_t>(a->v_cache) & 15) == 0 &&
                  (reinterpret_cast<uintptr_t>(a->q_rot) & 15) == 0,
              PKV_ERR_INVALID_ARG, "caches and q_rot must be 16-byte aligned");
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->out) & 15) == 0, PKV_ERR_INVALID_ARG,
              "out must be 16-byte aligned");
  PKV_REQUIRE(a->bt_stride > 0 && a->bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              a->bt_stride);
  PKV_REQUIRE(!a->attn_bias || a->bias_stride > 0, PKV_ERR_INVALID_ARG,
              "bias_stride must be positive when attn_bias is given");
  PKV_REQUIRE(!a->plan || (reinterpret_cast<uintptr_t>(a->plan) & 15) == 0, PKV_ERR_INVALID_ARG,
              "plan must be 16-byte aligned");
  PKV_REQUIRE(!a->mass || a->scores, PKV_ERR_INVALID_ARG, "mass needs the scores buffer");
  PKV_REQUIRE(!a->mass || std::isfinite(a->mass_decay), PKV_ERR_INVALID_ARG,
              "mass_decay must be finite");
  PKV_REQUIRE(!a->mass || (reinterpret_cast<uintptr_t>(a->scores) & 15) == 0, PKV_ERR_INVALID_ARG,
              "scores must be 16-byte aligned");
  int num_parts = a->num_parts;
  if (num_parts <= 0) {
    PKV_REQUIRE(!a->plan, PKV_ERR_INVALID_ARG, "a plan is made for a given num_parts: pass it");
    rc = pkv_shared_default_parts(a->B, a->Hq, a->Hkv, a->d, a->dtype, a->bt_stride, &num_parts);
    if (rc != PKV_OK) return rc;
  }
  // (a plan without partials -- no row has a prefix -- leaves the own tokens alone)
  const bool prefixes = a->prefix_tables != nullptr && a->n_prefixes > 0 && a->slots > 0;
  if (a->num_parts <= 0 && prefixes && a->dtype == PKV_F32) {
    // One part to an SM leaves room for a CTA of the float32 prefix kernel beside it; with
    // two the kernels follow one another (24 rows of 300 tokens, 16/8 heads of 64, behind
    // 1000: 28 us against 40; behind 300: 25 against 30).
    int sms = 0;
    rc = current_sms(&sms);
    if (rc != PKV_OK) return rc;
    if (num_parts > sms) num_parts = sms;
  }
  int C = a->num_ctas;
  if (prefixes) {
    if (C <= 0) {
      rc = current_sms(&C);
      if (rc != PKV_OK) return rc;
    }
    PKV_REQUIRE(C <= kMaxPlanCtas, PKV_ERR_INVALID_ARG, "num_ctas must be <= %d", kMaxPlanCtas);
    PKV_REQUIRE(a->prefix_plan && (reinterpret_cast<uintptr_t>(a->prefix_plan) & 15) == 0,
                PKV_ERR_INVALID_ARG, "prefix_plan must be given, 16-byte aligned");
    PKV_REQUIRE(a->pt_stride > 0 && a->pt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "pt_stride %d",
                a->pt_stride);
    PKV_REQUIRE(a->plan_ints >= plan_items_at(a->B, C), PKV_ERR_INVALID_ARG,
                "plan of %d ints < %d: not made for B = %d, num_ctas = %d", a->plan_ints,
                plan_items_at(a->B, C), a->B, C);
  }
  PKV_REQUIRE(a->slots >= 0, PKV_ERR_INVALID_ARG, "slots < 0");
  const int slots = prefixes ? a->slots : 0;
  size_t attn = 0;
  rc = pkv_attn_workspace_bytes(a->B, a->Hq, a->Hkv, a->d, num_parts, &attn);
  if (rc != PKV_OK) return rc;
  const SharedSpace sp = shared_space(attn, a->B, a->Hq, a->d, slots);
  PKV_REQUIRE(a->workspace_bytes >= sp.bytes, PKV_ERR_INVALID_ARG,
              "workspace of %zu bytes < %zu needed", a->workspace_bytes, sp.bytes);
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->workspace) & 255) == 0, PKV_ERR_INVALID_ARG,
              "workspace must be 256-byte aligned");
  const long long rows = static_cast<long long>(a->num_blocks) * a->Hkv * kBlockTokens;
  PKV_REQUIRE(rows < (1ll << 31), PKV_ERR_UNSUPPORTED,
              "pool too large for 32-bit TMA row coordinates");
  unsigned char *ws = static_cast<unsigned char *>(a->workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->num_parts <= 0 && a->flags == 0) {   // short contexts: one launch
    ShortParams p = {};
    p.cluster = shared_short_cluster(*a, prefixes, &p.pages);
    if (p.cluster > 0) {
      p.q = a->q_rot;
      p.k_cache = a->k_cache;
      p.v_cache = a->v_cache;
      p.block_tables = a->block_tables;
      p.seq_lens = a->seq_lens;
      p.prefix_tables = prefixes ? a->prefix_tables : a->block_tables;
      p.plan = prefixes ? a->prefix_plan : nullptr;
      p.mass_lens = a->mass_lens;
      p.bias = a->attn_bias;
      p.mass = a->mass;
      p.lse_out = a->lse_out;
      p.out = a->out;
      p.err = a->dev_err_flag;
      p.B = a->B;
      p.Hq = a->Hq;
      p.Hkv = a->Hkv;
      p.C = C;
      p.num_blocks = a->num_blocks;
      p.n_prefixes = a->n_prefixes;
      p.pt_stride = prefixes ? a->pt_stride : 0;
      p.bt_stride = a->bt_stride;
      p.bias_stride = a->attn_bias ? a->bias_stride : 0;
      p.scale_log2 = a->scale * kLog2e;
      p.decay = a->mass_decay;
      const cudaError_t e = launch_shared_short(p, a->d, G, a->dtype, s);
      PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "shared_short_kernel launch: %s",
                  cudaGetErrorString(e));
      return PKV_OK;
    }
  }
  AttnExt ext = {};
  ext.scores = a->mass ? a->scores : nullptr;
  ext.lse2 = a->mass ? reinterpret_cast<float *>(ws + sp.lse2) : nullptr;
  ext.lse_out = a->lse_out;
  if (prefixes) {
    PrefixParams p = {};
    p.q = a->q_rot;
    p.k_cache = a->k_cache;
    p.v_cache = a->v_cache;
    p.tables = a->prefix_tables;
    p.plan = a->prefix_plan;
    p.lse = reinterpret_cast<float *>(ws + sp.pre_lse);
    p.o = reinterpret_cast<float *>(ws + sp.pre_o);
    p.status = reinterpret_cast<int32_t *>(ws + sp.status);
    p.err = a->dev_err_flag;
    p.B = a->B;
    p.Hq = a->Hq;
    p.Hkv = a->Hkv;
    p.G = G;
    p.num_blocks = a->num_blocks;
    p.n_prefixes = a->n_prefixes;
    p.pt_stride = a->pt_stride;
    p.plan_ints = a->plan_ints;
    p.slots = slots;
    p.C = C;
    p.scale_log2 = a->scale * kLog2e;
    p.wait_limit = (a->flags & PKV_ATTN_SHORT_WAITS) ? 64 : kWaitLimitCycles;
    cudaError_t e;
    if (a->dtype == PKV_BF16) {
      CUtensorMap tk, tv;
      rc = get_tmap(a->k_cache, rows, a->d, a->dtype, &tk);
      if (rc != PKV_OK) return rc;
      rc = get_tmap(a->v_cache, rows, a->d, a->dtype, &tv);
      if (rc != PKV_OK) return rc;
      e = launch_prefix_bf16(tk, tv, p, a->d, s);
    } else {
      e = launch_prefix_f32(p, a->d, s);
    }
    PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "prefix kernel launch: %s", cudaGetErrorString(e));
    ext.own_o = reinterpret_cast<float *>(ws + sp.own_o);
    ext.lse2 = reinterpret_cast<float *>(ws + sp.own_lse);
    ext.lse_out = nullptr;
    ext.dependent = 1;
  }
  rc = attn_launch_ext(*a, num_parts, ext, stream);
  if (rc != PKV_OK) return rc;
  float *lse2 = reinterpret_cast<float *>(ws + sp.lse2);
  if (ext.own_o) {
    JoinParams j;
    j.plan = a->prefix_plan;
    j.status = reinterpret_cast<const int32_t *>(ws + sp.status);
    j.own_o = ext.own_o;
    j.own_lse = ext.lse2;
    j.pre_o = reinterpret_cast<const float *>(ws + sp.pre_o);
    j.pre_lse = reinterpret_cast<const float *>(ws + sp.pre_lse);
    j.out = a->out;
    j.lse2 = a->mass ? lse2 : nullptr;
    j.lse_out = a->lse_out;
    j.err = a->dev_err_flag;
    j.rows = a->B * a->Hq;
    j.B = a->B;
    j.Hq = a->Hq;
    j.Hkv = a->Hkv;
    j.C = C;
    j.n_prefixes = a->n_prefixes;
    j.pt_stride = a->pt_stride;
    j.plan_ints = a->plan_ints;
    j.slots = slots;
    const int per_cta = 256 / (a->d / 4);
    const unsigned grid = static_cast<unsigned>((j.rows + per_cta - 1) / per_cta);
    const cudaError_t e =
        a->dtype == PKV_BF16
            ? (a->d == 64 ? launch_waiting(join_kernel<__nv_bfloat16, 64>, grid, 256, 0, s, j)
                          : launch_waiting(join_kernel<__nv_bfloat16, 128>, grid, 256, 0, s, j))
            : (a->d == 64 ? launch_waiting(join_kernel<float, 64>, grid, 256, 0, s, j)
                          : launch_waiting(join_kernel<float, 128>, grid, 256, 0, s, j));
    PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "join kernel launch: %s", cudaGetErrorString(e));
  }
  if (a->mass) {
    MassParams m;
    m.scores = a->scores;
    m.lse2 = lse2;
    m.mass = a->mass;
    m.block_tables = a->block_tables;
    m.seq_lens = a->seq_lens;
    m.mass_lens = a->mass_lens;
    m.bt_stride = a->bt_stride;
    m.bias_stride = a->attn_bias ? a->bias_stride : 0;
    m.has_bias = a->attn_bias ? 1 : 0;
    m.Hq = a->Hq;
    m.Hkv = a->Hkv;
    m.num_blocks = a->num_blocks;
    m.decay = a->mass_decay;
    // at most 64 CTAs a row... or enough for one long row to fill the GPU
    int chunks = (a->bt_stride + kMassPages - 1) / kMassPages;
    const int most = a->B >= 64 ? 64 : 4096 / a->B;
    m.chunks = chunks < most ? chunks : most;
    const unsigned grid = static_cast<unsigned>(a->B) * m.chunks;
    const cudaError_t e = G == 1   ? launch_waiting(mass_kernel<1>, grid, 256, 0, s, m)
                          : G == 2 ? launch_waiting(mass_kernel<2>, grid, 256, 0, s, m)
                          : G == 4 ? launch_waiting(mass_kernel<4>, grid, 256, 0, s, m)
                                   : launch_waiting(mass_kernel<8>, grid, 256, 0, s, m);
    PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "mass kernel launch: %s", cudaGetErrorString(e));
  }
  return PKV_OK;
}
