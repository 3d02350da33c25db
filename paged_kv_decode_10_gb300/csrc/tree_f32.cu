// Attention of drafted tokens in float32, on CUDA cores (there is no tensor-core product of
// that precision): up to 64 query rows (nodes x group heads of one batch row and KV head)
// against 64 tokens a step, online softmax in base 2.
//
// Eight warps compute, 16 x 16 threads: thread (ty, tx) has rows ty + 16 i and, of the scores,
// tokens tx + 16 j, of the output, columns 4 tx + 64 m.  A half warp shares its rows, so
// row maxima, weights and queries never leave it and the warps do not wait for one another.
// Items of at most 16 or 32 rows use one or two of the four row registers.  Keys lie in
// shared memory with rows 4 floats longer than a head, so that a warp's reads spread over
// the banks.  A ninth warp finds the CTA's items (tree.h), hands them out through a short
// queue and loads K and V a step ahead, a bulk copy for every token.  (By tensor copies
// into swizzled slabs the loads of a call of two steps a CTA were 2 us sooner, but the
// permuted addresses took the products 10 to 20 % longer.)  Multiplications and additions
// go two to an instruction (16 rows of 1000 tokens, 16 nodes, 32/8 heads of 128: 139 -> 119
// us).  Twice the rows to a thread, with half the threads to a step, took 10 % less for 16
// to 32 rows of 64-wide heads, but 18 % more for full tiles, and 1.7 times as long for
// 128-wide heads, whose accumulators did not fit the registers.
//
// Masks.  Only steps that reach past the tokens every row sees look at mask bits.  What a row
// does not see may hold anything, the tail of a last page and pages outside the pool
// included (they are not even loaded): where one of those values is not finite (sums of
// four that overflow count as such), what a row does not see gets a weight of -1 and is
// skipped in the product with V instead of being multiplied by zero.
//
// Bound by the FMA and shared-memory pipes where rows are many (4 rows of 4000 tokens, 32
// nodes, 32/8 heads of 128: 199 us, 42 TFLOP/s), by the loads' latency where they are few
// (one row of 500 tokens, 8 nodes, 8/2 heads of 64: 13 us).
#include "tensor_core.cuh"
#include "tree.h"

namespace pkv {
namespace {

constexpr int kStep = 64, kTile = 64, kCompute = 256, kThreads = kCompute + 32, kBoundary = 1;
constexpr int kStages = 2, kQueue = 4;
constexpr long long kDrainCycles = 1ll << 31;
constexpr long long kPollLimit = 4096;

// An item as it is handed out: 64 bytes.
struct Handed {
  int q0, nodes, g, b;
  int base, n, tokens, n0;
  int t0, t1, part, pad[5];      // part: partial slot or -1 (whole)
};

template <int D>
struct Lay {
  static constexpr int LD = D + 4;                  // floats between staged rows
  static constexpr int kMat = kStep * LD;
  static constexpr int kQ = 0, kKV = kTile * LD;    // K, V of every stage
  static constexpr int kLP = kStep + 4, kP = kKV + 2 * kStages * kMat;
  static constexpr int kItems = kP + kTile * kLP;
  static constexpr int kBars = kItems + kQueue * 16;
  static constexpr int kThere = kBars + 2 * (2 * kStages + 2 * kQueue);   // pages of a stage in the pool
  static constexpr int kMisc = kThere + kStages;    // a wait gave up
  static constexpr int kBytes = 4 * (kMisc + 2);
};

template <int D, int NR, typename Wait>
__device__ __forceinline__ bool compute_item(const TreeParams &p, const Handed &it, float *sm,
                                             uint64_t *full, uint64_t *empty, const Wait &wait, int *step) {
  using L = Lay<D>;
  constexpr int LD = L::LD, M = D / 64;
  float *qs = sm + L::kQ, *ps = sm + L::kP;
  const volatile int *there_s = reinterpret_cast<const volatile int *>(sm + L::kThere);
  const int tid = threadIdx.x, lane = tid & 31, tx = tid & 15, ty = tid >> 4;
  const int rows = it.nodes * p.G;
  __syncwarp();   // (the item before is done with the queries)
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = ty + 16 * i;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        x = *reinterpret_cast<const float4 *>(
            static_cast<const float *>(p.q) +
            (static_cast<size_t>(it.q0 + (r >> p.lg_g)) * p.Hq + it.g * p.G + (r & (p.G - 1))) * D + 4 * tx +
            64 * m);
        x = make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
      }
      *reinterpret_cast<float4 *>(qs + r * LD + 4 * tx + 64 * m) = x;
    }
  }
  __syncwarp();
  float mx[NR], l[NR];
  uint64_t acc[NR][M][2];   // columns 4 tx + 64 m ..., two in one
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) acc[i][m][0] = acc[i][m][1] = 0;
  }
  for (int t = it.t0; t < it.t1; ++t, ++*step) {
    const int tok0 = t * kStep, st = *step % kStages;
    if (!wait.warp(&full[st], static_cast<uint32_t>(*step / kStages) & 1u)) return false;
    const float *ks = sm + L::kKV + 2 * st * L::kMat, *vs = ks + L::kMat;
    const uint32_t there = there_s[st];
    // scores: sums over the even and the odd elements of a head, two in one instruction
    uint64_t s2[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = 0;   // (two zeros)
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      ulonglong2 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        k[j] = *reinterpret_cast<const ulonglong2 *>(ks + (tx + 16 * j) * LD + c);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(qs + (ty + 16 * i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = fma2(q.y, k[j].y, fma2(q.x, k[j].x, s2[i][j]));
      }
    }
    float s[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = unpair(s2[i][j]);
        s[i][j] = x.x + x.y;
      }
    // a step that every row sees whole needs no masks
    const int special = it.base + (p.mask ? 0 : it.n0);
    bool odd = there != (1u << (kStep / kBlockTokens)) - 1u;
    const bool masked = tok0 + kStep > special || odd;
    if (masked) {   // (every warp looks for itself: 16 tokens of 64 are 8 reads a lane)
#pragma unroll 4
      for (int e = max(special - tok0, 0) * (D / 4) + lane; e < kStep * (D / 4); e += 32) {
        const float4 v = *reinterpret_cast<const float4 *>(vs + e / (D / 4) * LD + e % (D / 4) * 4);
        odd |= !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY);
      }
      odd = __any_sync(0xffffffffu, odd);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = ty + 16 * i;
      uint32_t sees[2] = {0xffffffffu, 0xffffffffu};
      if (masked) {
        const int node = min(r >> p.lg_g, it.nodes - 1);
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
        ps[r * L::kLP + tx + 16 * j] =
            odd && !(sees[j >> 1] >> (tx + 16 * (j & 1)) & 1) ? -1.f : w;
      }
      const uint64_t al2 = pair(al, al);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[i][m][h] = mul2(acc[i][m][h], al2);
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
        for (int e = 0; e < 4; ++e) {
          uint64_t x2[NR];
          bool on[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const float x = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
            x2[i] = pair(x, x);
            on[i] = !decltype(check)::value || !(x < 0.f);
          }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(vs + (u + e) * LD + 4 * tx + 64 * m);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              if (!on[i]) continue;
              acc[i][m][0] = fma2(x2[i], v.x, acc[i][m][0]);
              acc[i][m][1] = fma2(x2[i], v.y, acc[i][m][1]);
            }
          }
        }
      }
    };
    if (odd)
      weighted(std::true_type());
    else
      weighted(std::false_type());
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  const bool whole = it.part < 0;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = ty + 16 * i;
    float den = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (r >= rows) continue;
    const int q_row = it.q0 + (r >> p.lg_g);
    const size_t at = static_cast<size_t>(q_row) * p.Hq + it.g * p.G + (r & (p.G - 1));
    const size_t part = static_cast<size_t>(max(it.part, 0)) * p.tile + r;
    const bool any = !whole || den > 0.f || tree_sees_any(p, q_row, it.base, it.n);
    const float inv = whole ? tree_inverse(den, any) : den > 0.f ? 1.f / den : 0.f;
    float *to = whole ? static_cast<float *>(p.out) + at * D : p.part_o + part * D;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float2 x = unpair(acc[i][m][0]), y = unpair(acc[i][m][1]);
      *reinterpret_cast<float4 *>(to + 4 * tx + 64 * m) =
          make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
    }
    if (tx == 0) {
      if (!whole)
        p.part_lse[part] = part_lse(mx[i], den);
      else if (p.lse_out)
        p.lse_out[at] = tree_lse(mx[i], den, any);
    }
  }
  return true;
}

template <int D, bool POLL>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
    tree_f32_kernel(const __grid_constant__ TreeParams p) {
  using L = Lay<D>;
  extern __shared__ __align__(16) float sm[];
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::kBars), *empty = full + kStages;
  uint64_t *i_full = empty + kStages, *i_empty = i_full + kQueue;
  Handed *items = reinterpret_cast<Handed *>(sm + L::kItems);
  volatile int *there_s = reinterpret_cast<volatile int *>(sm + L::kThere);
  volatile int *gave_up = reinterpret_cast<volatile int *>(sm + L::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kCompute / 32);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], kCompute / 32);
    }
    *gave_up = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: what starts then may read what was there before)
  const int cta = blockIdx.x;
  // (few rows: the loading warp finds its share by itself)
  TreeWalk<kStep, kBoundary> walk = {};
  if (p.B > kWarpRows)
    walk = tree_begin<kStep, kBoundary, kThreads>(p, cta);   // (synchronises the CTA)
  else
    __syncthreads();
  const Waiter<POLL> wait{gave_up, p.err, p.wait_limit};
  if (warp == kCompute / 32) {
    // ======================= items, K and V =======================
    if (p.B <= kWarpRows) walk = tree_begin_warp<kStep, kBoundary>(p, cta);
    int x = 0;   // steps so far
    uint32_t cut = 0;   // slots that were written down
    bool ok = true;
    for (int i = 0; ok; ++i) {
      TreeItem w;
      const bool some = walk.next(p, &w);
      ok = wait.warp(&i_empty[i % kQueue], (static_cast<uint32_t>(i / kQueue) & 1u) ^ 1u);
      if (!ok) break;
      if (lane == 0) {
        items[i % kQueue] = some ? Handed{w.q0, w.nodes, w.g, w.b, w.base, w.n, w.tokens, w.n0, w.t0,
                                          w.t1, w.whole() ? -1 : w.slot(cta), {}}
                                 : Handed{};
        mbar_arrive(&i_full[i % kQueue]);
      }
      __syncwarp();
      if (!some) break;
      const int32_t *table = p.tables + static_cast<size_t>(w.b) * p.bt_stride;
      // lane's tokens of a step: lane and lane + 32
      auto page_id = [&](int t, int h) {
        const int tok = t * kStep + lane + 32 * h;
        return t < w.t1 && tok < w.tokens ? table[tok / kBlockTokens] : -1;
      };
      int next[2] = {page_id(w.t0, 0), page_id(w.t0, 1)};
      for (int t = w.t0; t < w.t1; ++t, ++x) {
        const int blk[2] = {next[0], next[1]};
        next[0] = page_id(t + 1, 0);
        next[1] = page_id(t + 1, 1);
        const int st = x % kStages;
        ok = wait.warp(&empty[st], (static_cast<uint32_t>(x / kStages) & 1u) ^ 1u);
        if (!ok) break;
        uint32_t bad = 0, tokens = 0;   // pages outside the pool
        bool on[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          on[h] = blk[h] >= 0 && blk[h] < p.num_blocks;
          tokens += __popc(__ballot_sync(0xffffffffu, on[h]));
          const uint32_t b = __ballot_sync(0xffffffffu, !on[h] && t * kStep + lane + 32 * h < w.tokens);
          bad |= ((b & 0xffffu ? 1u : 0u) | (b >> 16 ? 2u : 0u)) << (2 * h);
        }
        if (lane == 0) {
          // (pages behind the last token count as there: their tokens are masked by number)
          there_s[st] = static_cast<int>(~bad & 0xfu);
          if (bad) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
          mbar_arrive_expect_tx(&full[st], tokens * 2 * D * 4);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!on[h]) continue;
          const size_t at =
              ((static_cast<size_t>(blk[h]) * p.Hkv + w.g) * kBlockTokens + lane % kBlockTokens) * D;
          const uint32_t to = smem_u32(sm + L::kKV + 2 * st * L::kMat + (lane + 32 * h) * L::LD);
          bulk_copy_g2s(to, static_cast<const float *>(p.k_cache) + at, D * 4, &full[st]);
          bulk_copy_g2s(to + L::kMat * 4, static_cast<const float *>(p.v_cache) + at, D * 4, &full[st]);
        }
        __syncwarp();
      }
      if (!w.whole()) {   // (at most two of them)
        cut |= w.t0 == 0 ? 2u : 1u;
        if (lane == 0) tree_cut(p, w, cta, walk.at, walk.all, walk.ctas);
      }
    }
    if (lane < 2 && !(cut >> lane & 1u)) p.cuts[2 * cta + lane] = TreeCut{};
    // every copy has landed before the CTA ends (after a normal run they have)
    for (int n = max(0, x - kStages); n < x; ++n)
      mbar_wait_bounded(&full[n % kStages], static_cast<uint32_t>(n / kStages) & 1u, kDrainCycles);
  } else {
    int step = 0;
    for (int i = 0;; ++i) {
      if (!wait.warp(&i_full[i % kQueue], static_cast<uint32_t>(i / kQueue) & 1u)) break;
      const Handed &it = items[i % kQueue];   // (read again where it is used)
      if (it.t1 <= it.t0) break;
      const int rows = it.nodes * p.G;
      const bool ok = rows <= 16   ? compute_item<D, 1>(p, it, sm, full, empty, wait, &step)
                      : rows <= 32 ? compute_item<D, 2>(p, it, sm, full, empty, wait, &step)
                                   : compute_item<D, 4>(p, it, sm, full, empty, wait, &step);
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[i % kQueue]);
    }
  }
  __syncthreads();
  if (*gave_up) tree_all_nan<float, D, kStep, kBoundary, kThreads>(p);
}

template <int D, bool POLL>
cudaError_t launch(const TreeParams &p, cudaStream_t s) {
  constexpr int smem = Lay<D>::kBytes;
  auto kern = tree_f32_kernel<D, POLL>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  return launch_waiting(kern, p.C, kThreads, smem, s, p);
}

}  // namespace

cudaError_t launch_tree_f32(const TreeParams &p, int D, cudaStream_t s) {
  if (p.wait_limit <= kPollLimit) return D == 64 ? launch<64, true>(p, s) : launch<128, true>(p, s);
  return D == 64 ? launch<64, false>(p, s) : launch<128, false>(p, s);
}

}  // namespace pkv
