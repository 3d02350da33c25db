// pkv_decode_attn_tree: attention of drafted tokens over the paged cache.  Here the call,
// the float32 kernel (CUDA cores) and the join of items that several CTAs shared.
//
// Mathematics.  Node i of a row sees the row's tokens ahead of its nodes and those nodes
// that its mask names (without one, the nodes up to itself): out = sum_t softmax_t(s) v_t
// over what it sees, by an online softmax in base 2 over steps of the tokens; parts of the
// tokens are joined by their log-sum-exp.
#include "tree.h"

#include "attention_host.h"
#include "attention_kernel.cuh"

namespace pkv {
namespace {

// ---- float32 -----------------------------------------------------------------
// 64 rows (queries) against 64 tokens a step: 16 x 16 threads, thread (ty, tx) has rows
// ty + 16 i and, for the scores, tokens tx + 16 j, for the output columns 4 tx + 64 m.
// Items of at most 16 or 32 rows use one or two of the four row registers.
constexpr int kStep = 64, kTile = 64, kThreads = 256, kBoundary = 1, kMin = 2;

template <int D>
struct Lay {
  static constexpr int LD = D + 4;                  // floats between staged rows
  static constexpr int kQ = 0, kK = kQ + kTile * LD, kV = kK + kStep * LD;
  static constexpr int kLP = kStep + 4, kP = kV + kStep * LD;
  static constexpr int kPages = kP + kTile * kLP;   // of the step: in the pool?
  static constexpr int kFloats = kPages + kStep / kBlockTokens;
};

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <int D, int NR>
__device__ __forceinline__ void f32_item(const TreeParams &p, const TreeItem &it, float *sm) {
  using L = Lay<D>;
  constexpr int LD = L::LD, M = D / 64, kCols = D / 4;
  float *qs = sm + L::kQ, *ks = sm + L::kK, *vs = sm + L::kV, *ps = sm + L::kP;
  volatile int *pages = reinterpret_cast<volatile int *>(sm + L::kPages);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int rows = it.nodes * p.G;
  const int32_t *table = p.tables + static_cast<size_t>(it.b) * p.bt_stride;
  const float *kc = static_cast<const float *>(p.k_cache), *vc = static_cast<const float *>(p.v_cache);
  for (int e = tid; e < 16 * NR * kCols; e += kThreads) {
    const int r = e / kCols, c = e % kCols * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      x = load4(static_cast<const float *>(p.q) +
                (static_cast<size_t>(it.q0 + r / p.G) * p.Hq + it.g * p.G + r % p.G) * D + c);
      x.x *= p.scale_log2;
      x.y *= p.scale_log2;
      x.z *= p.scale_log2;
      x.w *= p.scale_log2;
    }
    store4(qs + r * LD + c, x);
  }
  float mx[NR], l[NR];
  float4 acc[NR][M];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) acc[i][m] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int t = it.t0; t < it.t1; ++t) {
    const int tok0 = t * kStep;
    __syncthreads();   // (the step before is done with shared memory)
    for (int e = tid; e < kStep * kCols; e += kThreads) {
      const int r = e / kCols, c = e % kCols * 4, tok = tok0 + r;
      float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
      if (tok < it.tokens) {
        const int blk = table[tok / kBlockTokens];
        const bool on = blk >= 0 && blk < p.num_blocks;
        if (on) {
          const size_t at =
              ((static_cast<size_t>(blk) * p.Hkv + it.g) * kBlockTokens + tok % kBlockTokens) * D + c;
          k = load4(kc + at);
          v = load4(vc + at);
        }
        if (c == 0 && r % kBlockTokens == 0) {
          pages[r / kBlockTokens] = on;
          if (!on) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
        }
      }
      store4(ks + r * LD + c, k);
      store4(vs + r * LD + c, v);
    }
    __syncthreads();
    float s[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * j) * LD + c);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float4 q = *reinterpret_cast<const float4 *>(qs + (ty + 16 * i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(q.x, k[j].x, fmaf(q.y, k[j].y, fmaf(q.z, k[j].z, fmaf(q.w, k[j].w, s[i][j]))));
      }
    }
    uint32_t there = 0;   // pages of the step that are in the pool
#pragma unroll
    for (int pg = 0; pg < kStep / kBlockTokens; ++pg)
      there |= (tok0 + pg * kBlockTokens < it.tokens && pages[pg] ? 1u : 0u) << pg;
    // a step that every row sees whole needs no masks
    const bool masked = tok0 + kStep > it.base || there != (1u << (kStep / kBlockTokens)) - 1u;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = ty + 16 * i;
      uint32_t sees[2] = {0xffffffffu, 0xffffffffu};
      if (masked) {
        const int node = min(r / p.G, it.nodes - 1);
        const uint32_t *words =
            p.mask ? p.mask + static_cast<size_t>(it.q0 + node) * p.mask_words : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sees[h] = tree_sees(words, p.mask_words, it.n0 + node, it.base, it.tokens, tok0 + 32 * h) &
                    ((there >> 2 * h & 1 ? 0xffffu : 0u) | (there >> (2 * h + 1) & 1 ? 0xffff0000u : 0u));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!(sees[j >> 1] >> (tx + 16 * (j & 1)) & 1)) s[i][j] = -INFINITY;
      }
      float top = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(mx[i], top), mu = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(mx[i] - mu);
      mx[i] = mn;
      l[i] *= al;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = ex2(s[i][j] - mu);
        l[i] += w;
        // (a weight of -1: what lies there is not looked at)
        ps[r * L::kLP + tx + 16 * j] = sees[j >> 1] >> (tx + 16 * (j & 1)) & 1 ? w : -1.f;
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        acc[i][m].x *= al;
        acc[i][m].y *= al;
        acc[i][m].z *= al;
        acc[i][m].w *= al;
      }
    }
    __syncwarp();   // (a row's weights come from its own half warp)
    auto weighted = [&](auto check) {
#pragma unroll 2
      for (int u = 0; u < kStep; u += 4) {
        float4 w[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i)
          w[i] = *reinterpret_cast<const float4 *>(ps + (ty + 16 * i) * L::kLP + u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const float4 v = *reinterpret_cast<const float4 *>(vs + (u + e) * LD + 4 * tx + 64 * m);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              const float x = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
              if (decltype(check)::value && x < 0.f) continue;
              acc[i][m].x = fmaf(x, v.x, acc[i][m].x);
              acc[i][m].y = fmaf(x, v.y, acc[i][m].y);
              acc[i][m].z = fmaf(x, v.z, acc[i][m].z);
              acc[i][m].w = fmaf(x, v.w, acc[i][m].w);
            }
          }
      }
    };
    if (masked)
      weighted(std::true_type());
    else
      weighted(std::false_type());
  }
  const bool whole = it.whole();
  const int slot = it.slot(blockIdx.x);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = ty + 16 * i;
    float den = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (r >= rows) continue;
    const int q_row = it.q0 + r / p.G;
    const size_t at = static_cast<size_t>(q_row) * p.Hq + it.g * p.G + r % p.G;
    const bool any = !whole || den > 0.f || tree_sees_any(p, q_row, it.base, it.n);
    const float inv = whole ? tree_inverse(den, any) : den > 0.f ? 1.f / den : 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float4 o = make_float4(acc[i][m].x * inv, acc[i][m].y * inv, acc[i][m].z * inv,
                                   acc[i][m].w * inv);
      const int c = 4 * tx + 64 * m;
      if (whole)
        store4(static_cast<float *>(p.out) + at * D + c, o);
      else
        store4(p.part_o + (static_cast<size_t>(slot) * p.tile + r) * D + c, o);
    }
    if (tx == 0) {
      if (!whole)
        p.part_lse[static_cast<size_t>(slot) * p.tile + r] = part_lse(mx[i], den);
      else if (p.lse_out)
        p.lse_out[at] = tree_lse(mx[i], den, any);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
    tree_f32_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(16) float sm[];
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: what starts then may read what was there before)
  const int cta = blockIdx.x;
  auto walk = tree_begin<kStep, kBoundary, kMin, kThreads>(p, cta);
  TreeCut cuts[2] = {};
  TreeItem it;
  while (walk.next(&it)) {
    if (!it.whole()) (it.t0 == 0 ? cuts[1] : cuts[0]) = walk.cut(it, walk.at);
    const int rows = it.nodes * p.G;
    __syncthreads();   // (the item before is done with the queries)
    if (rows <= 16)
      f32_item<D, 1>(p, it, sm);
    else if (rows <= 32)
      f32_item<D, 2>(p, it, sm);
    else
      f32_item<D, 4>(p, it, sm);
  }
  if (threadIdx.x == 0) {
    p.cuts[2 * cta] = cuts[0];
    p.cuts[2 * cta + 1] = cuts[1];
  }
}

template <int D>
cudaError_t launch_f32(const TreeParams &p, cudaStream_t s) {
  constexpr int smem = Lay<D>::kFloats * 4;
  auto kern = tree_f32_kernel<D>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  return launch_waiting(kern, p.C, kThreads, smem, s, p);
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
  s->tile = dtype == PKV_BF16 ? 256 : kTile;
  s->ctas = dtype == PKV_F32 && d == 64 ? 2 * sms : sms;
  if (s->ctas > kMaxTreeCtas) s->ctas = kMaxTreeCtas;
  const size_t rows = 2 * static_cast<size_t>(s->ctas) * s->tile;
  s->lse = align256(2 * s->ctas * sizeof(TreeCut));
  s->o = s->lse + align256(rows * sizeof(float));
  s->bytes = s->o + align256(rows * d * sizeof(float));
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
    e = a->d == 64 ? launch_f32<64>(p, s) : launch_f32<128>(p, s);
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
