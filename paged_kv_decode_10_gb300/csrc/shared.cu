// pkv_decode_attn_shared: attention over shared prefixes and own tokens, with the
// weights of the own tokens accumulated per cache slot.
//
// Launches: the prefix kernel (partials of every row over its prefix), the EXT
// build of the split-KV kernel over the rows' own tokens (a programmatic
// dependent of the prefix kernel: it streams pages while that one runs and waits
// for it before joining the partials) and, with mass, the fold of the scores.
#include <cuda.h>

#include "attention_host.h"
#include "attention_kernel.cuh"
#include "prefix.h"

namespace pkv {
namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct SharedSpace {
  size_t lse2, pre_lse, pre_o, bytes;   // offsets behind the attention workspace
};

SharedSpace shared_space(size_t attn_bytes, int B, int Hq, int d, int slots) {
  SharedSpace s;
  s.lse2 = align256(attn_bytes);
  s.pre_lse = s.lse2 + align256(static_cast<size_t>(B) * Hq * sizeof(float));
  s.pre_o = s.pre_lse + align256(static_cast<size_t>(slots) * Hq * sizeof(float));
  s.bytes = s.pre_o + align256(static_cast<size_t>(slots) * Hq * d * sizeof(float));
  return s;
}

// ---- the weights of the own tokens --------------------------------------------
// Token t of row b has base-2 scores s_h for the G heads of a KV head and the row
// sums 2^lse_h over prefix and own tokens: its weight is sum_h 2^(s_h - lse_h).
// A CTA takes pages_per_cta pages of one row; an item is one (page, KV head,
// token): the scores of consecutive items lie side by side, as do the weights.
// Memory bound: 4 G + 8 bytes a token and KV head.
struct MassParams {
  const float *scores, *lse2;
  float *mass;
  const int32_t *block_tables, *seq_lens, *mass_lens;
  int bt_stride, bias_stride, Hq, Hkv, num_blocks, chunks, has_bias;
  float decay;
};
constexpr int kMassPages = 16;

template <int G>
__global__ void __launch_bounds__(256) mass_kernel(const MassParams p) {
  pdl_wait();   // scores and row sums come from the kernel before this one
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x - b * p.chunks;
  const int L = p.seq_lens[b];
  bool bad;
  const int n = pages_of_len(L, p.bt_stride, p.has_bias != 0, p.bias_stride, &bad);
  const int known = p.mass_lens ? p.mass_lens[b] : L - 1;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const int per_page = p.Hkv * kBlockTokens;
  for (int j0 = chunk * kMassPages; j0 < n; j0 += p.chunks * kMassPages) {
    const int items = min(kMassPages, n - j0) * per_page;
    for (int e = threadIdx.x; e < items; e += blockDim.x) {
      const int j = j0 + e / per_page, r = e % per_page;
      const int g = r / kBlockTokens, t = j * kBlockTokens + r % kBlockTokens;
      if (t >= L) continue;
      const int blk = table[j];
      if (blk < 0 || blk >= p.num_blocks) continue;   // flagged by the attention kernel
      const size_t at = static_cast<size_t>(blk) * per_page + r;
      const float *l = p.lse2 + static_cast<size_t>(b) * p.Hq + g * G;
      float s[G];
      if constexpr (G >= 4) {
#pragma unroll
        for (int q = 0; q < G / 4; ++q)
          reinterpret_cast<float4 *>(s)[q] = __ldcs(reinterpret_cast<const float4 *>(p.scores + at * G) + q);
      } else {
#pragma unroll
        for (int q = 0; q < G; ++q) s[q] = p.scores[at * G + q];
      }
      const float old = t < known ? p.decay * p.mass[at] : 0.f;
      float w = 0.f;
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const float x = l[q];
        w += x == -INFINITY ? 0.f : ex2(s[q] - x);
      }
      p.mass[at] = old + w;
    }
  }
}

template <int G>
cudaError_t launch_mass(const MassParams &p, unsigned grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mass_kernel<G>, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

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
  PKV_REQUIRE(a->out != a->q_rot, PKV_ERR_INVALID_ARG, "out must not be q_rot");
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
  PKV_REQUIRE(!a->mass || (reinterpret_cast<uintptr_t>(a->scores) & 15) == 0, PKV_ERR_INVALID_ARG,
              "scores must be 16-byte aligned");
  int num_parts = a->num_parts;
  if (num_parts <= 0) {
    PKV_REQUIRE(!a->plan, PKV_ERR_INVALID_ARG, "a plan is made for a given num_parts: pass it");
    rc = default_parts(a->d, a->dtype, 0, G, &num_parts);
    if (rc != PKV_OK) return rc;
  }
  const bool prefixes = a->prefix_tables != nullptr && a->n_prefixes > 0;
  int C = a->num_ctas;
  if (prefixes) {
    if (C <= 0) {
      rc = current_sms(&C);
      if (rc != PKV_OK) return rc;
    }
    PKV_REQUIRE(C <= 4096, PKV_ERR_INVALID_ARG, "num_ctas must be <= 4096");
    PKV_REQUIRE(a->prefix_plan && (reinterpret_cast<uintptr_t>(a->prefix_plan) & 15) == 0,
                PKV_ERR_INVALID_ARG, "prefix_plan must be given, 16-byte aligned");
    PKV_REQUIRE(a->pt_stride > 0 && a->pt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "pt_stride %d",
                a->pt_stride);
    PKV_REQUIRE(a->plan_ints >= plan_items_at(a->B, C), PKV_ERR_INVALID_ARG,
                "plan of %d ints < %d: not made for B = %d, num_ctas = %d", a->plan_ints,
                plan_items_at(a->B, C), a->B, C);
    PKV_REQUIRE(a->slots >= 0, PKV_ERR_INVALID_ARG, "slots < 0");
  }
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
    ext.row_part = a->prefix_plan + plan_rows_at();
    ext.pre_o = p.o;
    ext.pre_lse = p.lse;
    ext.slots = slots;
    ext.dependent = 1;
  }
  rc = attn_launch_ext(*a, num_parts, ext, stream);
  if (rc != PKV_OK) return rc;
  if (a->mass) {
    MassParams m;
    m.scores = a->scores;
    m.lse2 = ext.lse2;
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
    cudaError_t e = G == 1   ? launch_mass<1>(m, grid, s)
                    : G == 2 ? launch_mass<2>(m, grid, s)
                    : G == 4 ? launch_mass<4>(m, grid, s)
                             : launch_mass<8>(m, grid, s);
    PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "mass kernel launch: %s", cudaGetErrorString(e));
  }
  return PKV_OK;
}
