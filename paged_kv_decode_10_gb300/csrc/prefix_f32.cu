// Prefix partials in float32, on CUDA cores: a tile of up to 64 query rows against a
// range of a prefix's tokens, online softmax in base 2.
//
// Eight warps share the tile's rows evenly (row r of warp w is query row 8 r + w), so
// that a few rows still keep all of them busy.  32 tokens at a time are copied to
// shared memory asynchronously, one step ahead.  Scores: a lane holds one token and
// all of the warp's rows, keys read as float4 (rows padded by 4 floats, so that a
// warp's reads spread over the banks), queries as broadcasts.  Weighted values: a
// lane holds D/32 columns, the weights come by shuffle.  Bound by the FMA and
// shared-memory pipes (float32 has no tensor-core product of its precision): 24 rows of
// 16 heads of 64 behind prefixes of 250..1000 tokens take 13 us (22 with eight rows to
// a warp and synchronous copies).  Items of 32 tokens, a step, fill the GPU where the
// prefixes are short (24 rows behind 250 tokens: 41 us a call with items of 128, 29 so).
#include "prefix.h"

namespace pkv {
namespace {

constexpr int kTok = 32, kWarps = 8, kRowsPerWarp = 8, kRows = kWarps * kRowsPerWarp;

template <int D>
struct Lay {
  static constexpr int LD = D + 4;                     // floats between staged tokens
  static constexpr int kStage = 2 * kTok * LD;         // K, then V
  static constexpr int kQ = 2 * kStage;                // [64][D]
  static constexpr int kOk = kQ + kRows * D;           // [2][32] token counts (int)
  static constexpr int kRow = kOk + 2 * kTok;          // [64] batch row, [64] slot (int)
  static constexpr int kState = kRow + 2 * kRows;      // something did not fit, partials (int)
  static constexpr int kFloats = kState + 2;
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool on) {   // zeros if not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}

template <int D>
struct Rows {
  float mx[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][D / 32];
};

// One staged step for the warp's first NR rows.
template <int D, int NR>
__device__ __forceinline__ void step(Rows<D> &st, const float *ks, const float *vs, const float *qs,
                                     bool ok, int warp, int lane) {
  constexpr int LD = Lay<D>::LD, DPL = D / 32;
  float s[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) s[r] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    const float4 k = *reinterpret_cast<const float4 *>(ks + lane * LD + c);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float4 q = *reinterpret_cast<const float4 *>(qs + (r * kWarps + warp) * D + c);
      s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (!ok) s[r] = -INFINITY;
    float t = s[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    const float mn = fmaxf(st.mx[r], t), mu = mn == -INFINITY ? 0.f : mn;
    const float al = ex2(st.mx[r] - mu);
    st.mx[r] = mn;
    s[r] = ex2(s[r] - mu);
    st.l[r] = st.l[r] * al + s[r];   // this lane's tokens
#pragma unroll
    for (int e = 0; e < DPL; ++e) st.acc[r][e] *= al;
  }
#pragma unroll 4
  for (int t = 0; t < kTok; ++t) {
    float v[DPL];
#pragma unroll
    for (int e = 0; e < DPL; ++e) v[e] = vs[t * LD + e * 32 + lane];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float w = __shfl_sync(0xffffffffu, s[r], t);
#pragma unroll
      for (int e = 0; e < DPL; ++e) st.acc[r][e] = fmaf(w, v[e], st.acc[r][e]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) prefix_f32_kernel(const PrefixParams p) {
  using L = Lay<D>;
  extern __shared__ __align__(16) float sm[];
  float *qs = sm + L::kQ;
  int *ok_s = reinterpret_cast<int *>(sm + L::kOk);
  int *rows = reinterpret_cast<int *>(sm + L::kRow), *slots = rows + kRows;
  volatile int *state = reinterpret_cast<volatile int *>(sm + L::kState);
  const float *kc = static_cast<const float *>(p.k_cache), *vc = static_cast<const float *>(p.v_cache);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: what starts then may read what was there before)
  const int *ctas = p.plan + plan_ctas_at(p.B);
  int i0 = ctas[blockIdx.x], i1 = ctas[blockIdx.x + 1];
  const PlanHeader head = plan_header(p.plan, p.B, p.C, p.Hkv, p.G, p.plan_ints, p.slots);
  if (!head.ok) {
    if (tid == 0) {
      set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
      p.status[blockIdx.x] = kPrefixSkipped;
    }
    return;
  }
  i0 = max(0, i0);
  i1 = min(head.items, i1);
  if (tid == 0) state[0] = state[1] = 0;
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    PrefixItem it;
    const int fits = prefix_item(p, i, kTileRowsF32, &it);
    if (tid == 0) state[1] = state[1] + it.rows;   // (not read where the item is kItemBad)
    if (fits != kItemOk) {
      if (tid == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
      if (fits == kItemBad || !prefix_unread(p, it, tid, kWarps * 32)) state[0] = 1;
      continue;
    }
    const int total = it.rows * p.G;   // at most 64
    const int nr = (total + kWarps - 1) / kWarps;
    const int32_t *table = p.tables + static_cast<size_t>(it.prefix) * p.pt_stride;
    const int steps = (it.t1 - it.t0 + kTok - 1) / kTok;
    // this thread's tokens of a step are t, t + per, ...: its 16-byte column of each
    constexpr int kCols = D / 4, kPer = kWarps * 32 / kCols, kN = kTok / kPer;
    const int col = tid % kCols * 4, tok = tid / kCols;
    auto ids = [&](int s, int (&blk)[kN]) {   // block of each (-1: no such token)
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const int t = it.t0 + s * kTok + tok + n * kPer;
        blk[n] = s < steps && t < it.t1 ? table[t >> 4] : -1;
      }
    };
    auto stage = [&](int s, const int (&blk)[kN]) {
      float *base = sm + (s & 1) * L::kStage;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const int local = tok + n * kPer, t = it.t0 + s * kTok + local;
        const bool there = s < steps && t < it.t1;
        const bool on = there && blk[n] >= 0 && blk[n] < p.num_blocks;
        if (there && !on) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
        const size_t at =
            on ? ((static_cast<size_t>(blk[n]) * p.Hkv + it.g) * kBlockTokens + (t & 15)) * D + col : 0;
        copy16(base + local * L::LD + col, kc + at, on);
        copy16(base + kTok * L::LD + local * L::LD + col, vc + at, on);
        if (col == 0) ok_s[(s & 1) * kTok + local] = on;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int blk[kN];
    ids(0, blk);
    __syncthreads();   // (the item before is done with shared memory)
    stage(0, blk);
    ids(1, blk);
    if (tid < kRows) {
      int row = -1, slot = -1;
      if (tid < total) {
        row = prefix_row(p, it, tid / p.G, &slot);
        if (row < 0) {
          set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
          state[0] = 1;
        }
      }
      rows[tid] = row;
      slots[tid] = slot;
    }
    __syncthreads();
    for (int e = tid; e < nr * kWarps * kCols; e += kWarps * 32) {
      const int m = e / kCols, c = e % kCols * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rows[m] >= 0) {
        x = *reinterpret_cast<const float4 *>(
            static_cast<const float *>(p.q) +
            (static_cast<size_t>(rows[m]) * p.Hq + it.g * p.G + m % p.G) * D + c);
        x.x *= p.scale_log2;
        x.y *= p.scale_log2;
        x.z *= p.scale_log2;
        x.w *= p.scale_log2;
      }
      *reinterpret_cast<float4 *>(qs + m * D + c) = x;
    }
    Rows<D> st;
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      st.mx[r] = -INFINITY;
      st.l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) st.acc[r][e] = 0.f;
    }
    for (int s = 0; s < steps; ++s) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();   // step s has landed, and step s - 1's buffer is free
      if (s + 1 < steps) {
        stage(s + 1, blk);
        ids(s + 2, blk);
      }
      const float *ks = sm + (s & 1) * L::kStage, *vs = ks + kTok * L::LD;
      const bool ok = ok_s[(s & 1) * kTok + lane] != 0;
      if (nr <= 1)
        step<D, 1>(st, ks, vs, qs, ok, warp, lane);
      else if (nr <= 2)
        step<D, 2>(st, ks, vs, qs, ok, warp, lane);
      else if (nr <= 4)
        step<D, 4>(st, ks, vs, qs, ok, warp, lane);
      else
        step<D, 8>(st, ks, vs, qs, ok, warp, lane);
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const int m = r * kWarps + warp;
      if (m >= total || slots[m] < 0) continue;   // (the same for the warp)
      float sum = st.l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const size_t at = static_cast<size_t>(slots[m]) * p.Hq + it.g * p.G + m % p.G;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) p.o[at * D + e * 32 + lane] = st.acc[r][e] * inv;
      if (lane == 0) p.lse[at] = part_lse(st.mx[r], sum);
    }
  }
  __syncthreads();
  if (tid == 0) p.status[blockIdx.x] = state[0] ? kPrefixSkipped : state[1];
}

template <int D>
cudaError_t launch(const PrefixParams &p, cudaStream_t s) {
  constexpr int smem = Lay<D>::kFloats * 4;
  auto kern = prefix_f32_kernel<D>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  return launch_waiting(kern, p.C, kWarps * 32, smem, s, p);
}

}  // namespace

cudaError_t launch_prefix_f32(const PrefixParams &p, int D, cudaStream_t s) {
  return D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace pkv
