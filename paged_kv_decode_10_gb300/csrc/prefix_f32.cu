// Prefix partials on CUDA cores: a tile of up to 64 query rows against a range
// of a prefix's tokens, online softmax in base 2.
//
// Eight warps of eight query rows each; 32 tokens at a time are staged in shared
// memory as float32.  Scores: a lane holds one token and all eight rows, keys
// read as float4 (rows padded by 4 floats, so that a warp's reads spread over
// the banks), queries as broadcasts.  Weighted values: a lane holds D/32
// columns, the weights come by shuffle.
#include "prefix.h"

namespace pkv {
namespace {

constexpr int kTok = 32, kWarps = 8, kRowsPerWarp = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) prefix_simt_kernel(const PrefixParams p,
                                                                  int max_rows) {
  constexpr int M = kWarps * kRowsPerWarp, LD = D + 4, DPL = D / 32;
  extern __shared__ float sm[];
  float *qs = sm, *ks = qs + M * D, *vs = ks + kTok * LD;
  int *rows = reinterpret_cast<int *>(vs + kTok * LD), *slots = rows + M;
  int *ok_s = slots + M;   // [kTok]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  int n_items;
  if (!prefix_plan_ok(p, &n_items)) {
    if (tid == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
    return;
  }
  const int *ctas = p.plan + plan_ctas_at(p.B);
  const int i0 = max(0, ctas[blockIdx.x]), i1 = min(n_items, ctas[blockIdx.x + 1]);
  for (int i = i0; i < i1; ++i) {
    PrefixItem it;
    if (!prefix_item(p, i, max_rows, &it)) {
      if (tid == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
      continue;
    }
    const int total = it.rows * p.G;
    for (int m0 = 0; m0 < total; m0 += M) {
      const int mq = min(M, total - m0);   // query rows of this tile
      __syncthreads();
      if (tid < M) {
        int row = -1, slot = -1;
        if (tid < mq) {
          row = prefix_row(p, it, (m0 + tid) / p.G, &slot);
          if (row < 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
        }
        rows[tid] = row;
        slots[tid] = slot;
      }
      __syncthreads();
      for (int e = tid; e < M * D; e += kWarps * 32) {
        const int m = e / D, c = e - m * D;
        float x = 0.f;
        if (rows[m] >= 0)
          x = to_f32(static_cast<const T *>(
                  p.q)[(static_cast<size_t>(rows[m]) * p.Hq + it.g * p.G + (m0 + m) % p.G) * D + c]) *
              p.scale_log2;
        qs[e] = x;
      }
      float mx[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][DPL];
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        mx[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) acc[r][e] = 0.f;
      }
      const int32_t *table = p.tables + static_cast<size_t>(it.prefix) * p.pt_stride;
      for (int t0 = it.t0; t0 < it.t1; t0 += kTok) {
        __syncthreads();
        constexpr int VEC = 16 / sizeof(T);
        for (int e = tid; e < kTok * (D / VEC); e += kWarps * 32) {
          const int t = e / (D / VEC), c = (e - t * (D / VEC)) * VEC;
          const int tok = t0 + t;
          bool ok = tok < it.t1;
          T kx[VEC], vx[VEC];
          if (ok) {
            const int blk = table[tok >> 4];
            ok = blk >= 0 && blk < p.num_blocks;
            if (!ok) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
            if (ok) {
              const size_t at =
                  ((static_cast<size_t>(blk) * p.Hkv + it.g) * kBlockTokens + (tok & 15)) * D + c;
              *reinterpret_cast<uint4 *>(kx) =
                  *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_cache) + at);
              *reinterpret_cast<uint4 *>(vx) =
                  *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v_cache) + at);
            }
          }
#pragma unroll
          for (int q = 0; q < VEC; ++q) {
            ks[t * LD + c + q] = ok ? to_f32(kx[q]) : 0.f;
            vs[t * LD + c + q] = ok ? to_f32(vx[q]) : 0.f;
          }
          if (c == 0) ok_s[t] = ok;
        }
        __syncthreads();
        float s[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) s[r] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
          const float4 k = *reinterpret_cast<const float4 *>(ks + lane * LD + c);
#pragma unroll
          for (int r = 0; r < kRowsPerWarp; ++r) {
            const float4 q =
                *reinterpret_cast<const float4 *>(qs + (warp * kRowsPerWarp + r) * D + c);
            s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
          }
        }
        const bool ok = ok_s[lane] != 0;
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
          if (!ok) s[r] = -INFINITY;
          float t = s[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
          const float mn = fmaxf(mx[r], t), mu = mn == -INFINITY ? 0.f : mn;
          const float al = ex2(mx[r] - mu);
          mx[r] = mn;
          s[r] = ex2(s[r] - mu);
          l[r] = l[r] * al + s[r];   // this lane's tokens
#pragma unroll
          for (int e = 0; e < DPL; ++e) acc[r][e] *= al;
        }
#pragma unroll 4
        for (int t = 0; t < kTok; ++t) {
          float v[DPL];
#pragma unroll
          for (int e = 0; e < DPL; ++e) v[e] = vs[t * LD + e * 32 + lane];
#pragma unroll
          for (int r = 0; r < kRowsPerWarp; ++r) {
            const float w = __shfl_sync(0xffffffffu, s[r], t);
#pragma unroll
            for (int e = 0; e < DPL; ++e) acc[r][e] = fmaf(w, v[e], acc[r][e]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        float sum = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int m = warp * kRowsPerWarp + r;
        if (slots[m] < 0) continue;
        const size_t at = static_cast<size_t>(slots[m]) * p.Hq + it.g * p.G + (m0 + m) % p.G;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) p.o[at * D + e * 32 + lane] = acc[r][e] * inv;
        if (lane == 0) p.lse[at] = sum > 0.f ? mx[r] + log2f(sum) : -INFINITY;
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch(const PrefixParams &p, int max_rows, cudaStream_t s) {
  constexpr int M = kWarps * kRowsPerWarp;
  constexpr int smem = (M * D + 2 * kTok * (D + 4)) * 4 + (2 * M + kTok) * 4;
  auto kern = prefix_simt_kernel<T, D>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  kern<<<p.C, kWarps * 32, smem, s>>>(p, max_rows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_f32(const PrefixParams &p, int D, cudaStream_t s) {
  return D == 64 ? launch<float, 64>(p, kTileRowsF32, s) : launch<float, 128>(p, kTileRowsF32, s);
}

}  // namespace pkv
