// pkv_decode_attn_tree: attention of drafted tokens over the paged cache.  Here the call
// and the join of items that several CTAs shared.
//
// Mathematics.  Node i of a row sees the row's tokens ahead of its nodes and those nodes
// that its mask names (without one, the nodes up to itself): out = sum_t softmax_t(s) v_t
// over what it sees, by an online softmax in base 2 over steps of the tokens; parts of the
// tokens are joined by their log-sum-exp.
#include "tree.h"

#include <cstring>

#include "attention_host.h"
#include "attention_kernel.cuh"

namespace pkv {
namespace {

__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// ---- the join ---------------------------------------------------------------------
// out = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M), M the largest lse_s, over the parts
// of an item, in the order of its tokens.  Every slot stands for one share of its item's
// rows, kJoinChunks CTAs to a slot, D / 4 lanes to a row.  Bound by the launch and by L2
// latency (the partials were just written, by other SMs: about 1 us a round trip), so 8
// reads of a lane are under way together: K parts of F rows.  (Joined by the CTAs of an
// item's first part alone, one item of 131072 tokens and 19 parts took 20 us; two parts at
// once whatever their number, 8 parts took 7 us, now 3.)
constexpr int kJoinChunks = 2;

template <typename T, int D, int F, int K>
__device__ __forceinline__ void join_rows(const TreeParams &p, const TreeCut &cut, int first, int end,
                                          int step) {
  const int d4 = threadIdx.x % (D / 4);
  for (int r = first; r < end; r += F * step) {
    float M[F], den[F];
    float4 acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      M[f] = -INFINITY;
      den[f] = 0.f;
      acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i = 0; i < cut.parts; i += K) {
      float l[F][K];
      float4 v[F][K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // (what does not count is read from the last part or row: a branch would make the
        // reads wait for one another)
        const int part = min(i + k, cut.parts - 1);
        const size_t slot =
            static_cast<size_t>(part == 0 ? 2 * cut.first + 1 : 2 * (cut.first + part)) * p.tile;
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const size_t at = slot + min(r + f * step, end - 1);
          l[f][k] = __ldcg(p.part_lse + at);
          v[f][k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at * D) + d4);
        }
      }
#pragma unroll
      for (int f = 0; f < F; ++f) {
        float top = M[f];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (i + k >= cut.parts) l[f][k] = -INFINITY;
          top = fmaxf(top, l[f][k]);
        }
        const float mu = top == -INFINITY ? 0.f : top, al = ex2(M[f] - mu);
        den[f] *= al;
        acc[f] = make_float4(acc[f].x * al, acc[f].y * al, acc[f].z * al, acc[f].w * al);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          // (a part of which the row sees nothing counts for nothing, whatever it holds)
          if (l[f][k] == -INFINITY) continue;
          const float w = ex2(l[f][k] - mu);
          den[f] += w;
          acc[f].x = fmaf(w, v[f][k].x, acc[f].x);
          acc[f].y = fmaf(w, v[f][k].y, acc[f].y);
          acc[f].z = fmaf(w, v[f][k].z, acc[f].z);
          acc[f].w = fmaf(w, v[f][k].w, acc[f].w);
        }
        M[f] = top;
      }
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int row = r + f * step;
      if (row >= end) continue;
      const int q_row = cut.q0 + (row >> p.lg_g);
      const size_t at = static_cast<size_t>(q_row) * p.Hq + cut.g * p.G + (row & (p.G - 1));
      const bool any = den[f] > 0.f || tree_sees_any(p, q_row, cut.base, cut.n);
      const float inv = tree_inverse(den[f], any);
      store4(static_cast<T *>(p.out) + at * D + 4 * d4,
             make_float4(acc[f].x * inv, acc[f].y * inv, acc[f].z * inv, acc[f].w * inv));
      if (d4 == 0 && p.lse_out) p.lse_out[at] = tree_lse(M[f], den[f], any);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeParams p) {
  constexpr int kRows = 256 / (D / 4);
  pdl_launch_dependents();   // (every CTA waits before it ends)
  pdl_wait();
  const int mine = blockIdx.x / kJoinChunks, chunk = blockIdx.x % kJoinChunks;
  const int4 *said = reinterpret_cast<const int4 *>(p.cuts + mine);
  const int4 c0 = __ldcg(said), c1 = __ldcg(said + 1);
  const TreeCut cut{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  if (cut.parts <= 0) return;
  const int part = mine / 2 - cut.first;   // this slot's place among the item's
  const int r0 = cut.rows * part / cut.parts + chunk * kRows + threadIdx.x / (D / 4),
            r1 = cut.rows * (part + 1) / cut.parts;
  if (cut.parts <= 2)
    join_rows<T, D, 4, 2>(p, cut, r0, r1, kJoinChunks * kRows);
  else if (cut.parts <= 4)
    join_rows<T, D, 2, 4>(p, cut, r0, r1, kJoinChunks * kRows);
  else
    join_rows<T, D, 1, 8>(p, cut, r0, r1, kJoinChunks * kRows);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Rows of an item, CTAs, and the workspace they need.
struct TreeSpace {
  int tile, ctas;
  size_t lse, o, bytes;
};
int tree_space(int d, int dtype, TreeSpace *s) {
  int sms = 0;
  const int rc = current_sms(&sms);
  if (rc != PKV_OK) return rc;
  s->tile = dtype == PKV_BF16 ? 256 : 64;
  s->ctas = dtype == PKV_F32 && d == 64 ? 2 * sms : sms;
  if (s->ctas > kMaxTreeCtas) s->ctas = kMaxTreeCtas;
  const size_t rows = 2 * static_cast<size_t>(s->ctas) * s->tile;
  s->lse = align256(2 * s->ctas * sizeof(TreeCut));
  s->o = s->lse + align256(rows * sizeof(float));
  s->bytes = s->o + align256(rows * d * sizeof(float));
  return PKV_OK;
}

// Queries [T, Hq, D] (bf16) as a 3-D tensor; the box is one 128-byte column slab of 128 rows,
// 128 / G tokens of the G heads of one KV head, swizzled 128B.
int query_tmap(const void *base, int T, int Hq, int G, int D, CUtensorMap *out) {
  static const auto encode = [] {   // the driver's function, through the runtime
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess
               ? reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn)
               : nullptr;
  }();
  PKV_REQUIRE(encode, PKV_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  std::memset(out, 0, sizeof(*out));
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  PKV_REQUIRE(r == CUDA_SUCCESS, PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)",
              static_cast<int>(r));
  return PKV_OK;
}

int tree_shapes(int B, int T, int Hq, int Hkv, int d, int dtype) {
  const int rc = check_shapes(B, Hq, Hkv, d, dtype);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(T >= 0, PKV_ERR_INVALID_ARG, "T %d < 0", T);
  return PKV_OK;
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_tree_workspace_bytes(int32_t Hq, int32_t Hkv, int32_t d, int32_t dtype,
                                        size_t *bytes) {
  clear_error();
  PKV_REQUIRE(bytes, PKV_ERR_INVALID_ARG, "bytes is NULL");
  int rc = tree_shapes(1, 1, Hq, Hkv, d, dtype);
  if (rc != PKV_OK) return rc;
  TreeSpace sp;
  rc = tree_space(d, dtype, &sp);
  if (rc != PKV_OK) return rc;
  *bytes = sp.bytes;
  return PKV_OK;
}

extern "C" int pkv_decode_attn_tree(const pkv_tree_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  int rc = tree_shapes(a->B, a->T, a->Hq, a->Hkv, a->d, a->dtype);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE((a->flags & ~PKV_ATTN_SHORT_WAITS) == 0, PKV_ERR_UNSUPPORTED, "flags %d", a->flags);
  if (a->B == 0 || a->T == 0) return PKV_OK;
  PKV_REQUIRE(a->q_rot && a->k_cache && a->v_cache && a->block_tables && a->seq_lens &&
                  a->node_starts && a->out && a->workspace,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  const long long out_bytes = static_cast<long long>(a->T) * a->Hq * a->d *
                              static_cast<long long>(dtype_size(a->dtype));
  PKV_REQUIRE(!rows_overlap(a->out, 0, out_bytes, a->q_rot, 0, out_bytes, 1), PKV_ERR_INVALID_ARG,
              "out must not overlap q_rot");
  PKV_REQUIRE(std::isfinite(a->scale), PKV_ERR_INVALID_ARG, "scale must be finite");
  PKV_REQUIRE(a->num_blocks > 0, PKV_ERR_INVALID_ARG, "num_blocks must be positive");
  PKV_REQUIRE(((reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) |
                reinterpret_cast<uintptr_t>(a->q_rot) | reinterpret_cast<uintptr_t>(a->out)) &
               15) == 0,
              PKV_ERR_INVALID_ARG, "caches, q_rot and out must be 16-byte aligned");
  PKV_REQUIRE(a->bt_stride > 0 && a->bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              a->bt_stride);
  PKV_REQUIRE(!a->mask || (a->mask_words > 0 && a->mask_words < (1 << 26)), PKV_ERR_INVALID_ARG,
              "mask_words %d", a->mask_words);
  const long long rows = static_cast<long long>(a->num_blocks) * a->Hkv * kBlockTokens;
  PKV_REQUIRE(rows < (1ll << 31), PKV_ERR_UNSUPPORTED,
              "pool too large for 32-bit TMA row coordinates");
  TreeSpace sp;
  rc = tree_space(a->d, a->dtype, &sp);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(a->workspace_bytes >= sp.bytes, PKV_ERR_INVALID_ARG,
              "workspace of %zu bytes < %zu needed", a->workspace_bytes, sp.bytes);
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->workspace) & 255) == 0, PKV_ERR_INVALID_ARG,
              "workspace must be 256-byte aligned");
  unsigned char *ws = static_cast<unsigned char *>(a->workspace);
  TreeParams p = {};
  p.q = a->q_rot;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.tables = a->block_tables;
  p.lens = a->seq_lens;
  p.starts = a->node_starts;
  p.mask = reinterpret_cast<const uint32_t *>(a->mask);
  p.out = a->out;
  p.lse_out = a->lse_out;
  p.cuts = reinterpret_cast<TreeCut *>(ws);
  p.part_lse = reinterpret_cast<float *>(ws + sp.lse);
  p.part_o = reinterpret_cast<float *>(ws + sp.o);
  p.err = a->dev_err_flag;
  p.B = a->B;
  p.T = a->T;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.num_blocks = a->num_blocks;
  p.bt_stride = a->bt_stride;
  p.mask_words = a->mask ? a->mask_words : 0;
  p.C = sp.ctas;
  p.tile = sp.tile;
  while (p.G << p.lg_nodes < sp.tile) ++p.lg_nodes;
  while (1 << p.lg_g < p.G) ++p.lg_g;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.wait_limit = (a->flags & PKV_ATTN_SHORT_WAITS) ? 64 : kWaitLimitCycles;
  cudaError_t e;
  if (a->dtype == PKV_BF16) {
    CUtensorMap tq, tk, tv;
    rc = query_tmap(a->q_rot, a->T, a->Hq, p.G, a->d, &tq);
    if (rc != PKV_OK) return rc;
    rc = get_tmap(a->k_cache, rows, a->d, a->dtype, &tk);
    if (rc != PKV_OK) return rc;
    rc = get_tmap(a->v_cache, rows, a->d, a->dtype, &tv);
    if (rc != PKV_OK) return rc;
    e = launch_tree_bf16(tq, tk, tv, p, a->d, s);
  } else {
    e = launch_tree_f32(p, a->d, s);
  }
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "tree kernel launch: %s", cudaGetErrorString(e));
  const unsigned grid = 2 * static_cast<unsigned>(sp.ctas) * kJoinChunks;
  e = a->dtype == PKV_BF16
          ? (a->d == 64 ? launch_waiting(tree_join_kernel<__nv_bfloat16, 64>, grid, 256, 0, s, p)
                        : launch_waiting(tree_join_kernel<__nv_bfloat16, 128>, grid, 256, 0, s, p))
          : (a->d == 64 ? launch_waiting(tree_join_kernel<float, 64>, grid, 256, 0, s, p)
                        : launch_waiting(tree_join_kernel<float, 128>, grid, 256, 0, s, p));
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "tree join launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}
