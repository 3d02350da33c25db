// pkv_decode_attn_shared for short contexts: prefix and own tokens of one (row, KV head)
// by one CTA or a cluster of them, in one launch, weights included.
//
// Mathematics: softmax in base 2 over prefix ++ own, online per page of 16 tokens, the
// warps' and then the CTAs' partials joined by log-sum-exp; the weights follow from the
// scores kept in shared memory once the row sums are known.  Everything is float32.
//
// A warp takes every eighth page of its CTA's share.  Scores: two lanes to a token, each
// half of the head's elements against all of the group's queries (shared memory, read as
// broadcasts); weighted values: a lane owns D / 32 columns and takes the weights by
// shuffle.  A page's keys and values are read together.  What bounds it is the latency of
// a few dependent steps (4 rows of up to 64 tokens behind 500, 8/2 heads of 64: 4.8 us,
// 8.7 as three kernels).  A prefix is read by every row behind it, from L2 mostly, which
// is why this form is for few rows and short contexts.
#include "attention_host.h"
#include "attention_kernel.cuh"
#include "prefix.h"

namespace pkv {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote_f32(const float *local, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// N consecutive elements (16-byte aligned when N elements are 16 bytes or more).
template <typename T, int N>
struct Piece {
  static constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        *reinterpret_cast<uint4 *>(w + 4 * i) = reinterpret_cast<const uint4 *>(p)[i];
    } else if constexpr (kWords == 2) {
      *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 2)
      return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else
      return __uint_as_float(w[i]);
  }
};

// CTAs that fit an SM by registers (a page's keys and values and the accumulators of the
// group are held in them).
constexpr int resident(int elem, int d, int G) {
  return elem * d * (G < 4 ? 1 : G / 2) <= 256 ? 2 : 1;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads, resident(sizeof(T), D, G))
    shared_short_kernel(const __grid_constant__ ShortParams p) {
  constexpr int DPL = D / 32, QS = D + 8;   // (the halves of a query 4 floats apart: other banks)
  extern __shared__ __align__(16) float sm[];
  float *qs = sm;                             // [G][QS]
  float *red_o = qs + G * QS;                 // [warps][G][D]
  float *red_ml = red_o + kWarps * G * D;     // [warps][G][2]
  float *all_o = red_ml + kWarps * G * 2;     // [G][D], relative to all_ml's maximum
  float *all_ml = all_o + G * D;              // [G][2]
  float *lse_s = all_ml + G * 2;              // [G]
  float *own_s = lse_s + 8;                   // [tokens][G + 1] scores, decayed weight
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.cluster, rank = S > 1 ? static_cast<int>(ctarank()) : 0;
  const int u = blockIdx.x / S, b = u / p.Hkv, g = u - b * p.Hkv;
  pdl_wait();
  const int L = p.seq_lens[b];
  // the row's prefix, as the plan states it
  int4 pre = make_int4(0, 0, -1, 0);
  if (p.plan) {
    // (nothing is kept in slots here; what plan_header and plan_row_ok check beyond this
    // took 0.2 us of 4.9)
    const int4 *w = reinterpret_cast<const int4 *>(p.plan);
    const int4 h0 = w[0], h1 = w[1];
    pre = *reinterpret_cast<const int4 *>(p.plan + plan_rows_at() + 4 * b);
    const bool fits = (h0.x == kSharedMagic) & (h0.z == p.B) & (h1.x == p.C) & (h1.y == p.Hkv) &
                      (h1.z == G) & (pre.z < p.n_prefixes) & (pre.w >= 0) &
                      (pre.w <= kBlockTokens * p.pt_stride);
    if (!fits || pre.z < 0) {
      if (!fits && tid == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
      pre.z = -1;
      pre.w = 0;
    }
  }
  bool bad;
  const int n_own = pages_of_len(L, p.bt_stride, p.bias != nullptr, p.bias_stride, &bad);
  if (bad && tid == 0 && g == 0 && rank == 0) set_dev_err(p.err, PKV_DEVERR_BAD_LEN);
  const int n_pre = (pre.w + kBlockTokens - 1) / kBlockTokens, total = n_pre + n_own;
  const int j0 = total * rank / S, j1 = total * (rank + 1) / S;
  const int32_t *own = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const int32_t *shared = p.prefix_tables + static_cast<size_t>(max(pre.z, 0)) * p.pt_stride;
  auto block_of = [&](int j) { return j < n_pre ? shared[j] : own[j - n_pre]; };
  int ids = -1;   // block of this warp's page number `lane`
  {
    const int j = j0 + warp + kWarps * lane;
    if (j < j1) ids = block_of(j);
  }
  const T *q = static_cast<const T *>(p.q) + (static_cast<size_t>(b) * p.Hq + g * G) * D;
  for (int e = tid; e < G * D; e += kThreads) {
    const int h = e / D, x = e % D;
    qs[h * QS + x + (x >= D / 2 ? 4 : 0)] = to_f32(q[e]) * p.scale_log2;
  }
  __syncthreads();

  const int tok = lane >> 1, half = lane & 1;
  const int known = p.mass ? (p.mass_lens ? p.mass_lens[b] : L - 1) : 0;
  float m[G], l[G], o[G][DPL];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int c = 0; c < DPL; ++c) o[h][c] = 0.f;
  }
  for (int j = j0 + warp, i = 0; j < j1; j += kWarps, ++i) {
    const int blk = __shfl_sync(0xffffffffu, ids, i);
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
      continue;
    }
    const bool mine = j >= n_pre;   // own tokens
    const int t0 = (mine ? j - n_pre : j) * kBlockTokens;
    const int valid = min(kBlockTokens, (mine ? L : pre.w) - t0);
    const size_t page = (static_cast<size_t>(blk) * p.Hkv + g) * kBlockTokens;
    Piece<T, D / 2> k;
    Piece<T, DPL> v[kBlockTokens];
    k.load(static_cast<const T *>(p.k_cache) + (page + tok) * D + half * (D / 2));
#pragma unroll
    for (int t = 0; t < kBlockTokens; ++t)
      v[t].load(static_cast<const T *>(p.v_cache) + (page + t) * D + lane * DPL);
    float bias = 0.f;
    if (mine && p.bias && tok < valid)
      bias = p.bias[static_cast<size_t>(b) * p.bias_stride + t0 + tok] * kLog2e;
    float old = 0.f;
    if (mine && p.mass && half && tok < valid && t0 + tok < known) old = p.decay * p.mass[page + tok];
    float s[G];
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 2; e += 4) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float4 x = *reinterpret_cast<const float4 *>(qs + h * QS + half * (D / 2 + 4) + e);
        s[h] = fmaf(k.at(e), x.x, fmaf(k.at(e + 1), x.y, fmaf(k.at(e + 2), x.z, fmaf(k.at(e + 3), x.w, s[h]))));
      }
    }
    // (a token behind the last one, or excluded by the mask, may hold anything)
    const bool counts = tok < valid && bias != -INFINITY;
    const uint32_t live = __ballot_sync(0xffffffffu, counts);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
      s[h] = counts ? s[h] + bias : -INFINITY;
    }
    if (mine && p.mass) {
      float *dst = own_s + ((j - j0) * kBlockTokens + tok) * (G + 1);
#pragma unroll
      for (int h = 0; h < G; ++h)
        if (half == 0) dst[h] = s[h];
      if (half) dst[G] = old;
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float top = s[h];
#pragma unroll
      for (int x = 2; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m[h], top), mu = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(m[h] - mu);
      m[h] = mn;
      s[h] = ex2(s[h] - mu);
      l[h] = l[h] * al + (half ? 0.f : s[h]);   // this lane's tokens
#pragma unroll
      for (int c = 0; c < DPL; ++c) o[h][c] *= al;
    }
#pragma unroll
    for (int t = 0; t < kBlockTokens; ++t) {
      if (!(live >> (2 * t) & 1u)) continue;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float w = __shfl_sync(0xffffffffu, s[h], 2 * t);
#pragma unroll
        for (int c = 0; c < DPL; ++c) o[h][c] = fmaf(w, v[t].at(c), o[h][c]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < G; ++h) {
    float sum = l[h];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) {
      red_ml[(warp * G + h) * 2] = m[h];
      red_ml[(warp * G + h) * 2 + 1] = sum;
    }
#pragma unroll
    for (int c = 0; c < DPL; ++c) red_o[(warp * G + h) * D + lane * DPL + c] = o[h][c];
  }
  __syncthreads();
  // ---- the CTA's partial ----
  for (int e = tid; e < G * D; e += kThreads) {
    const int h = e / D;
    float M = -INFINITY, den = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[(w * G + h) * 2]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = M == -INFINITY ? 0.f : ex2(red_ml[(w * G + h) * 2] - M);
      den = fmaf(f, red_ml[(w * G + h) * 2 + 1], den);
      x = fmaf(f, red_o[w * G * D + e], x);
    }
    all_o[e] = x;
    if (e % D == 0) {
      all_ml[2 * h] = M;
      all_ml[2 * h + 1] = den;
    }
  }
  if (S > 1)
    cluster_barrier();
  else
    __syncthreads();
  // ---- the row: every CTA stores its share of the columns and knows the row sums ----
  const int share = G * D / S;   // (S at most 8, G * D at least 64)
  T *out = static_cast<T *>(p.out) + (static_cast<size_t>(b) * p.Hq + g * G) * D;
  // (what is read of the other CTAs is read together, then added: one by one the round
  // trips took 2 us of 7)
  auto sums = [&](int h, float *M, float (&f)[kMaxCluster]) {   // the CTAs' factors, the denominator
    float m[kMaxCluster], d[kMaxCluster], den = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      m[r] = r >= S ? -INFINITY : S > 1 ? remote_f32(all_ml + 2 * h, r) : all_ml[2 * h];
      d[r] = r >= S ? 0.f : S > 1 ? remote_f32(all_ml + 2 * h + 1, r) : all_ml[2 * h + 1];
    }
    *M = -INFINITY;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) *M = fmaxf(*M, m[r]);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      f[r] = *M == -INFINITY ? 0.f : ex2(m[r] - *M);
      den = fmaf(f[r], d[r], den);
    }
    return den;
  };
  float M, f[kMaxCluster];
  for (int e = rank * share + tid; e < (rank + 1) * share; e += kThreads) {
    float part[kMaxCluster], x = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      part[r] = r >= S ? 0.f : S > 1 ? remote_f32(all_o + e, r) : all_o[e];
    const float den = sums(e / D, &M, f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) x = fmaf(f[r], part[r], x);
    out[e] = from_f32<T>(den == 0.f ? 0.f : x / den);
  }
  if (tid < G) {
    const float den = sums(tid, &M, f);
    const float l2 = den == 0.f ? -INFINITY : M + log2f(den);   // (NaN stays NaN)
    lse_s[tid] = den != den ? den : l2;
    if (rank == 0 && p.lse_out)
      p.lse_out[static_cast<size_t>(b) * p.Hq + g * G + tid] = lse_s[tid] * 0.6931471805599453f;
  }
  if (S > 1)
    cluster_barrier();   // (also: a CTA's shared memory outlives its readers)
  else
    __syncthreads();
  if (!p.mass) return;
  for (int i = tid; i < (j1 - j0) * kBlockTokens; i += kThreads) {
    const int j = j0 + i / kBlockTokens, t = (j - n_pre) * kBlockTokens + i % kBlockTokens;
    if (j < n_pre || t >= L) continue;
    const int blk = own[j - n_pre];
    if (blk < 0 || blk >= p.num_blocks) continue;
    const float *src = own_s + i * (G + 1);
    float w = src[G];
    float add = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) add += lse_s[h] == -INFINITY ? 0.f : ex2(src[h] - lse_s[h]);
    p.mass[(static_cast<size_t>(blk) * p.Hkv + g) * kBlockTokens + i % kBlockTokens] = w + add;
  }
}

template <typename T, int D, int G>
cudaError_t launch(const ShortParams &p, cudaStream_t s) {
  auto kern = shared_short_kernel<T, D, G>;
  const size_t fixed = (G * (D + 8) + kWarps * G * D + kWarps * G * 2 + G * D + G * 2 + 8) * 4;
  const size_t smem = fixed + (p.mass ? static_cast<size_t>(p.pages) * kBlockTokens * (G + 1) * 4 : 0);
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kShortMaxSmem);
  });
  if (e != cudaSuccess) return e;
  if (smem > static_cast<size_t>(kShortMaxSmem)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, int D>
cudaError_t launch_g(const ShortParams &p, int G, cudaStream_t s) {
  return G == 1   ? launch<T, D, 1>(p, s)
         : G == 2 ? launch<T, D, 2>(p, s)
         : G == 4 ? launch<T, D, 4>(p, s)
                  : launch<T, D, 8>(p, s);
}

}  // namespace

// CTAs to a (row, KV head) and the pages one of them may get; 0: the other form.
// As many clusters of S are on the GPU at once as its groups of SMs hold (152, 76, 36 and
// 15 with a CTA to an SM).  Up to two pages a warp this form wins (4 heads of 128 to a KV
// head, bf16: 1 row of 4 KV heads and 512 tokens 6.4 us against 10.5 in parts, 16 rows
// behind 448 shared tokens 9.6 against 15.2; 8 heads to a KV head with weights 13.3
// against 18.8); at four they are even, and beyond it loses.  One CTA to a pair may also
// take several waves, where the other form pays for more kernels (prefixes) or for its
// partition (float32): 608 pairs of 16 own tokens behind 40, bf16, 4 heads of 64: 8.6
// against 18.3; 250 tokens, float32, 4 heads of 128: 51 against 64.  Two waves of the
// bf16 form without prefixes lose (304 pairs of 100 tokens, heads of 128: 12 against 7).
int shared_short_cluster(const pkv_shared_args &a, bool prefixes, int *per_cta) {
  constexpr int kMostUnits[4] = {152, 76, 34, 14};
  const long long units = static_cast<long long>(a.B) * a.Hkv;
  const long long pages = static_cast<long long>(a.bt_stride) + (prefixes ? a.pt_stride : 0);
  int i = 0;
  while (i < 3 && units <= kMostUnits[i + 1] && pages > static_cast<long long>(kWarps) << i) ++i;
  const long long s = 1ll << i;
  const long long rounds = (pages + kWarps * s - 1) / (kWarps * s);   // pages of a warp
  const int r = resident(static_cast<int>(dtype_size(a.dtype)), a.d, a.Hq / a.Hkv);
  const long long waves = i > 0 ? 1 : (units + 152 * r - 1) / (152 * r);
  const int most = i > 0 ? 2 : a.dtype == PKV_F32 ? 8 / r : prefixes ? 2 * r : 2;
  if (rounds > 2 || waves * rounds > most || (waves > 1 && !prefixes && a.dtype == PKV_BF16)) return 0;
  *per_cta = static_cast<int>((pages + s - 1) / s);
  return static_cast<int>(s);
}

cudaError_t launch_shared_short(const ShortParams &p, int D, int G, int dtype, cudaStream_t s) {
  if (dtype == PKV_BF16)
    return D == 64 ? launch_g<__nv_bfloat16, 64>(p, G, s) : launch_g<__nv_bfloat16, 128>(p, G, s);
  return D == 64 ? launch_g<float, 64>(p, G, s) : launch_g<float, 128>(p, G, s);
}

}  // namespace pkv
