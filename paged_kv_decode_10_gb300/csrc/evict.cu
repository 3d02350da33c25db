// Eviction from the paged cache by accumulated attention weight (pkv_evict):
// choose the tokens to keep per (row, KV head), then compact keys, values and
// weights in place.
//
// Choice.  The m-th largest of a row's candidate weights is found by radix
// selection on order-preserving 32-bit keys (digits of 11, 11 and 10 bits, from
// the top): after each digit only the keys that share the threshold's digits so
// far still count.  Tokens above the threshold are kept, and of those equal to
// it the first few by index, so the choice does not depend on any order of
// execution.  One scan in token order then writes the kept indices ascending.  A
// row's keys are read once and stay on chip; rows too long for one CTA, and
// rows too few to fill the GPU, are shared by clusters whose histograms are added
// through distributed shared memory.  Bound by latency: three passes of a handful
// of barriers each.
//
// Compaction.  The i-th kept token comes from index >= i.
//  * Many rows: a CTA walks the kept tokens of one (row, KV head), K or V, in
//    order.  A step's stores can only reach slots that this or an earlier step has
//    read: read a step into registers, barrier, store it.
//  * Few rows: chunks of T kept tokens go to CTAs of their own.  A chunk may be
//    stored once every token that still lies in its T slots has been read; at most
//    T kept tokens come from there, consecutive ones, so they belong to at most two
//    chunks, earlier ones or itself: a chunk waits for two flags (the choice notes how
//    many kept tokens lie below each chunk's first slot, which names them).  Chunks are taken
//    by ticket in order and reading never waits, so every wait ends.
//  * Short rows: one CTA chooses and compacts (evict_small_kernel).
// The first two are memory bound: each kept row is read and written once.  The walk needs
// no flags and keeps its steps back to back (64 rows of 8 heads, 1500..2600 tokens of 128
// down to 1024, bf16: 78 us, 5.9 TB/s, against 150 us in chunks, the choice before it
// 17 us); with 4 (row, head) pairs it leaves the GPU empty (131072 tokens down to 32768:
// 130 us against 31 us in chunks, the choice 23 us).
#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 256;
constexpr int kBins = 2048, kBinsPer = kBins / kSelThreads;
constexpr int kWarps = kSelThreads / 32;
constexpr int kTileTokens = 4 * kSelThreads;       // a thread holds 4 consecutive tokens of a tile
constexpr int kMaxCluster = 16, kMaxCached = 48;   // CTAs, steps (of 4 KB of keys)
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;                       // 16-byte pieces of K (and of V) a thread moves
constexpr int kChunkBytes = kMoveThreads * kMoveVecs * 16;
constexpr int kWalkVecs = 4;                       // pieces of a walking thread's step
constexpr int kWalkTokens = 1024;                  // tokens of its list
constexpr int kChunkUnits = 76;                    // (row, head) pairs from which rows are walked
constexpr long long kWaitCycles = 1ll << 31;

struct EvictParams {
  unsigned char *k_cache, *v_cache;
  float *mass;
  const int32_t *block_tables, *seq_lens, *keep_lens;
  int32_t *kept, *err;
  int32_t *ticket, *flags;           // workspace: [1], [B * Hkv][chunks]
  int32_t *below;                    // [B * Hkv][chunks + 1] kept tokens with index < chunk * c;
                                     // NULL: rows are walked
  int num_blocks, bt_stride, kept_stride, sink, recent;
  int B, Hkv, row_bytes;
  int chunk, chunks;                 // tokens of a chunk, chunks of kept_stride tokens
  int cached;                        // steps whose keys the select kernel keeps
};

// Larger key <=> larger weight; -0 and +0 are equal, every NaN is the largest.  No
// weight has key 0 (the lowest, -inf's, is 0x007fffff): that marks other tokens.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Words of CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t remote_addr(const void *local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t remote_u32(const void *local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote_addr(local, rank)) : "memory");
  return v;
}
// Sum over the threads before this one of v, and the total (kSelThreads threads).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t w = lane < kSelThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < kSelThreads / 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, kSelThreads / 32 - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + incl - v;
}

// One (row, KV head) per cluster.  CTA r of the cluster has `per` tiles' worth of
// consecutive tokens, of which each warp has a consecutive share, 128 tokens (four a
// lane) at a time: warp, step, lane, place is token order, so the final scan needs
// one exchange between the warps.  The keys are kept in shared memory and the loops
// over them stay rolled: with the keys in registers the code was unrolled 16 times
// and run once a pass, and fetching it took 40 us instead of 12 for 131072 tokens.
// Steps beyond p.cached read the weights again in every pass.
// kRead: steps read at once (few: more CTAs fit an SM; many: fewer rounds of reads).
template <int kRead>
__global__ void __launch_bounds__(kSelThreads, kRead > 4 ? 2 : 4)
    evict_select_kernel(const EvictParams p) {
  extern __shared__ uint4 keys_s[];   // [cached][kSelThreads]
  // bin i counts digit kBins - 1 - i: ascending order of bins is descending order
  // of keys.  Two histograms: one is cleared while the other is in use.
  __shared__ __align__(16) uint32_t hist[2][kBins];
  __shared__ uint32_t warp_sums[kWarps];
  __shared__ uint32_t counts[kWarps][2], totals[2];
  __shared__ uint32_t bad, segment;
  __shared__ __align__(8) uint32_t found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), nc = cluster_size();
  pdl_wait();
  pdl_launch_dependents();
  const int u = blockIdx.x / nc;
  const int b = u / p.Hkv, g = u - b * p.Hkv;
  const int L = p.seq_lens[b], K = p.keep_lens[b];
  int32_t *kept = p.kept + static_cast<size_t>(u) * p.kept_stride;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const bool bad_len = L < 0 || K < 0 || static_cast<long long>(L) > 16ll * p.bt_stride ||
                       min(L, K) > p.kept_stride;
  const int step = static_cast<int>(nc) * kSelThreads, me = static_cast<int>(rank) * kSelThreads + tid;
  // what the chunks need: flags and ticket
  int32_t *below = nullptr;
  if (p.below) {
    for (int j = me; j < p.chunks; j += step) p.flags[static_cast<size_t>(u) * p.chunks + j] = 0;
    below = p.below + static_cast<size_t>(u) * (p.chunks + 1);
  }
  if (blockIdx.x == 0 && tid == 0) *p.ticket = 0;
  for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int n_recent = min(p.recent, max(K, 0)), n_sink = min(p.sink, max(K, 0) - n_recent);
  const int c0 = n_sink, c1 = L - n_recent;   // candidates [c0, c1)
  const int m = K - n_recent - n_sink;        // of which m stay
  const int len = bad_len ? 0 : L;
  const int tiles = (len + kTileTokens - 1) / kTileTokens;
  const int per = (tiles + static_cast<int>(nc) - 1) / static_cast<int>(nc);   // steps of a warp
  // this lane's tokens of step i: t_of(i) .. t_of(i) + 3
  auto t_of = [&](int i) {
    return ((static_cast<int>(rank) * kWarps + warp) * per + i) * 128 + 4 * lane;
  };
  auto page_ok = [&](int blk) { return blk >= 0 && blk < p.num_blocks; };
  auto weights = [&](int blk, int t) {
    return __ldcg(reinterpret_cast<const float4 *>(
        p.mass + (static_cast<size_t>(blk) * p.Hkv + g) * kBlockTokens + (t & 15)));
  };
  auto keys4 = [&](const float4 &x, int t) {   // 0: not a candidate
    return make_uint4(t >= c0 && t < c1 ? mass_key(x.x) : 0u,
                      t + 1 >= c0 && t + 1 < c1 ? mass_key(x.y) : 0u,
                      t + 2 >= c0 && t + 2 < c1 ? mass_key(x.z) : 0u,
                      t + 3 >= c0 && t + 3 < c1 ? mass_key(x.w) : 0u);
  };
  const int cached = min(per, p.cached);
  bool wrong = false;
  // the table, then the weights: two rounds of reads for every kRead steps
#pragma unroll 1
  for (int i0 = 0; i0 < per; i0 += kRead) {
    int blk[kRead];
#pragma unroll
    for (int i = 0; i < kRead; ++i) {
      const int t = t_of(i0 + i);
      const bool mine = i0 + i < per && t < len;
      blk[i] = mine ? table[t >> 4] : -1;
      wrong |= mine && !page_ok(blk[i]);
    }
    float4 x[kRead];
#pragma unroll
    for (int i = 0; i < kRead; ++i)
      if (i0 + i < cached && page_ok(blk[i])) x[i] = weights(blk[i], t_of(i0 + i));
#pragma unroll
    for (int i = 0; i < kRead; ++i)
      if (i0 + i < cached)
        keys_s[(i0 + i) * kSelThreads + tid] =
            page_ok(blk[i]) ? keys4(x[i], t_of(i0 + i)) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (wrong) bad = 1;
  bool skip = bad_len;   // (the same in every CTA of the cluster)
  if (nc > 1) {
    cluster_sync();
    // (a lane a CTA: the remote reads are under way together)
    skip |= __any_sync(0xffffffffu, static_cast<uint32_t>(lane) < nc && remote_u32(&bad, lane) != 0);
  } else {
    __syncthreads();
    skip |= bad != 0;
  }
  if (skip && tid == 0 && g == 0 && rank == 0)
    set_dev_err(p.err, bad_len ? PKV_DEVERR_BAD_LEN : PKV_DEVERR_BAD_BLOCK);
  const int n = skip ? 0 : min(L, K);
  for (int j = n + me; j < p.kept_stride; j += step) kept[j] = -1;
  if (!skip && L <= K)
    for (int j = me; j < L; j += step) kept[j] = j;
  if (!skip && L > K) {
    for (int j = me; j < n_sink; j += step) kept[j] = j;
    for (int j = me; j < n_recent; j += step) kept[K - n_recent + j] = c1 + j;
    // below, where the choice has no say: among the first and the last tokens, or
    // where all between go
    for (int c = below ? me : p.chunks + 1; c <= p.chunks; c += step) {
      const long long x = static_cast<long long>(c) * p.chunk;
      if (x <= c0 || x >= c1 || m <= 0)
        below[c] = static_cast<int>(x <= c0   ? x
                                    : x >= c1 ? min(static_cast<long long>(K), K - n_recent + (x - c1))
                                              : n_sink);
    }
  }
  if (skip || K >= L || m <= 0) {
    if (nc > 1) cluster_sync();   // a CTA's shared memory outlives its readers
    return;
  }

  auto each_step = [&](auto &&f) {   // f(first token, keys), whole warps
#pragma unroll 2
    for (int i = 0; i < cached; ++i) f(t_of(i), keys_s[i * kSelThreads + tid]);
#pragma unroll 1
    for (int i = cached; i < per; ++i) {
      const int t = t_of(i);
      f(t, t < len ? keys4(weights(table[t >> 4], t), t) : make_uint4(0u, 0u, 0u, 0u));
    }
  };
  // ---- the threshold: the m-th largest key ----
  uint32_t prefix = 0, mask = 0;   // the threshold's bits so far
  uint32_t left = m;               // its rank among the keys with that prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t dm = pass == 2 ? 1023u : 2047u;
    uint32_t *h = hist[pass & 1];
    // (tokens that are no candidates count in the last bin, behind every weight's)
    auto count = [&](uint32_t k) {
      if ((k & mask) == prefix) atomicAdd(&h[kBins - 1 - ((k >> shift) & dm)], 1u);
    };
    each_step([&](int, const uint4 &x) {
      count(x.x);
      count(x.y);
      count(x.z);
      count(x.w);
    });
    if (nc > 1)
      cluster_sync();
    else
      __syncthreads();
    // The bins are shared out over the cluster (reading all of every CTA's histogram
    // took 8 times as long): thread i of CTA r has nb bins of segment r.
    // (a cluster of 16 leaves every second thread without a bin)
    const int nb = max(1, kBinsPer / static_cast<int>(nc));
    const bool busy = nc <= kBinsPer || tid < kSelThreads / 2;
    const int first = nc <= kBinsPer ? (static_cast<int>(rank) * kSelThreads + tid) * nb
                                     : static_cast<int>(rank) * (kSelThreads / 2) + (busy ? tid : 0);
    uint32_t c[kBinsPer], sum = 0, total;
    if (nc == 1) {
#pragma unroll
      for (int q = 0; q < kBinsPer; q += 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(&h[first + q]);
        c[q] = x.x;
        c[q + 1] = x.y;
        c[q + 2] = x.z;
        c[q + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < kBinsPer; ++q) {
        c[q] = 0;
        if (q < nb && busy) {
          uint32_t y[kMaxCluster];   // read together, then added
          y[0] = h[first + q];
#pragma unroll
          for (int r = 1; r < kMaxCluster; ++r)
            y[r] = r < static_cast<int>(nc) ? remote_u32(&h[first + q], (rank + r) % nc) : 0u;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) c[q] += y[r];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kBinsPer; ++q) sum += c[q];
#pragma unroll
    for (int q = 0; q < kBinsPer; q += 4)
      *reinterpret_cast<uint4 *>(&hist[(pass & 1) ^ 1][kBinsPer * tid + q]) =
          make_uint4(0u, 0u, 0u, 0u);
    uint32_t above = block_scan(sum, warp_sums, &total);
    if (nc > 1) {
      if (tid == 0) segment = total;
      cluster_sync();
      above += __reduce_add_sync(0xffffffffu,
                                 static_cast<uint32_t>(lane) < rank ? remote_u32(&segment, lane) : 0u);
    }
    uint32_t at = 0, rest = 0;   // (one thread of the cluster finds it)
#pragma unroll
    for (int q = 0; q < kBinsPer; ++q) {
      if (above < left && above + c[q] >= left) {
        at = kBins - 1 - (first + q);
        rest = left - above;
      }
      above += c[q];
    }
    if (rest) {
#pragma unroll 1
      for (uint32_t r = 0; r < nc; ++r)
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote_addr(found, r)),
                     "r"(at), "r"(rest)
                     : "memory");
    }
    if (nc > 1)
      cluster_sync();   // (and the histograms have been read)
    else
      __syncthreads();
    prefix |= found[0] << shift;
    mask |= dm << shift;
    left = found[1];
  }
  // ---- kept indices in token order: above the threshold, and the first
  // `left` of those equal to it ----
  uint32_t gt = 0, eq = 0;
  each_step([&](int, const uint4 &x) {
    gt += (x.x > prefix) + (x.y > prefix) + (x.z > prefix) + (x.w > prefix);
    eq += (x.x == prefix) + (x.y == prefix) + (x.z == prefix) + (x.w == prefix);
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    counts[warp][0] = gt;
    counts[warp][1] = eq;
  }
  __syncthreads();
  uint32_t g_at = 0, e_at = 0;   // above the threshold, and equal, ahead of this warp's tokens
  if (nc > 1) {
    if (tid < 2) {
      uint32_t t = 0;
      for (int w = 0; w < kWarps; ++w) t += counts[w][tid];
      totals[tid] = t;
    }
    cluster_sync();
    const bool ahead = static_cast<uint32_t>(lane) < rank;
    g_at = __reduce_add_sync(0xffffffffu, ahead ? remote_u32(&totals[0], lane) : 0u);
    e_at = __reduce_add_sync(0xffffffffu, ahead ? remote_u32(&totals[1], lane) : 0u);
  }
  for (int w = 0; w < warp; ++w) {
    g_at += counts[w][0];
    e_at += counts[w][1];
  }
  each_step([&](int t, const uint4 &x) {
    const uint32_t k[4] = {x.x, x.y, x.z, x.w};
    uint32_t is_gt = 0, is_eq = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      is_gt |= (k[q] > prefix ? 1u : 0u) << q;
      is_eq |= (k[q] == prefix ? 1u : 0u) << q;
    }
    const uint32_t v = __popc(is_gt) << 16 | __popc(is_eq);   // of at most 128 tokens
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
    uint32_t ga = g_at + ((incl - v) >> 16), ea = e_at + ((incl - v) & 0xffffu);
    const int c = below ? (t + 3) / p.chunk : 0;   // a chunk's first slot among these?
    const int edge = c * p.chunk;
    const bool mark = below && edge >= t && edge > c0 && edge < c1 && c <= p.chunks;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (mark && edge == t + q) below[c] = static_cast<int>(n_sink + ga + min(ea, left));
      const bool one_gt = is_gt >> q & 1u, one_eq = is_eq >> q & 1u;
      if (one_gt || (one_eq && ea < left)) kept[n_sink + ga + min(ea, left)] = t + q;
      ga += one_gt;
      ea += one_eq;
    }
    g_at += all >> 16;
    e_at += all & 0xffffu;
  });
  if (nc > 1) cluster_sync();   // a CTA's shared memory outlives its readers
}

// Rows of up to NT tokens: choice and compaction by one CTA per (row, KV head), a token
// a thread.  A candidate stays if fewer than m candidates come before it in order of
// weight (ties: of index), which a thread counts over all keys in shared memory; the
// places follow from a scan of the ballots.  Every weight is in a register and every
// step's keys and values are read before anything is written where they lay.  Bound by
// latency and, for many rows, by the keys' n^2 comparisons.  8 heads of 128 in bf16, half
// kept: 1 row of 256 tokens 5.5 us (choice and compaction apart 11.3), 64 rows 11.5
// (19.9); 512 tokens: 1 row 10.0 (12.6), 64 rows 31.5 (29.1).
template <int NT>
__global__ void __launch_bounds__(NT) evict_small_kernel(const EvictParams p) {
  __shared__ __align__(16) uint32_t keys[NT];
  __shared__ int table_s[NT / kBlockTokens], from_s[NT];
  __shared__ int counts[NT / 32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x, b = u / p.Hkv, g = u - b * p.Hkv;
  const int L = p.seq_lens[b], K = p.keep_lens[b];
  int32_t *kept = p.kept + static_cast<size_t>(u) * p.kept_stride;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const bool bad_len = L < 0 || K < 0 || L > kBlockTokens * p.bt_stride ||
                       min(L, K) > p.kept_stride;
  const int len = bad_len ? 0 : L;   // (at most NT)
  const int blk = tid < len ? table[tid >> 4] : -1;
  const bool there = blk >= 0 && blk < p.num_blocks;
  const bool skip = __syncthreads_or(tid < len && !there) || bad_len;
  if (skip && tid == 0 && g == 0)
    set_dev_err(p.err, bad_len ? PKV_DEVERR_BAD_LEN : PKV_DEVERR_BAD_BLOCK);
  const int n = skip ? 0 : min(L, K);
  for (int j = n + tid; j < p.kept_stride; j += NT) kept[j] = -1;
  if (skip || L <= K) {
    if (tid < n) kept[tid] = tid;
    return;
  }
  const int n_recent = min(p.recent, K), n_sink = min(p.sink, K - n_recent);
  const int c0 = n_sink, c1 = L - n_recent;            // candidates [c0, c1)
  const int m = K - n_recent - n_sink;                 // of which m stay
  const int row = there ? (blk * p.Hkv + g) * kBlockTokens + (tid & 15) : 0;
  const float x = there ? p.mass[row] : 0.f;
  const bool candidate = tid >= c0 && tid < c1;
  const uint32_t key = candidate ? mass_key(x) : 0u;
  keys[tid] = key;
  if (there && (tid & 15) == 0) table_s[tid >> 4] = blk;
  __syncthreads();
  // rank: keys ahead of this warp's count from equal on, those behind it from larger on
  int rank = 0;
  const uint4 *k4 = reinterpret_cast<const uint4 *>(keys);
  const int w0 = 8 * warp, w1 = w0 + 8, end = (c1 + 3) / 4;
  for (int i = c0 / 4; i < min(w0, end); ++i) {
    const uint4 k = k4[i];
    rank += (k.x >= key) + (k.y >= key) + (k.z >= key) + (k.w >= key);
  }
  for (int i = max(w0, c0 / 4); i < min(w1, end); ++i) {
    const uint4 k = k4[i];
    rank += (k.x > key || (k.x == key && 4 * i < tid)) + (k.y > key || (k.y == key && 4 * i + 1 < tid)) +
            (k.z > key || (k.z == key && 4 * i + 2 < tid)) +
            (k.w > key || (k.w == key && 4 * i + 3 < tid));
  }
  for (int i = max(w1, c0 / 4); i < end; ++i) {
    const uint4 k = k4[i];
    rank += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
  }
  const bool stays = tid < len && (candidate ? rank < m : true);
  const uint32_t votes = __ballot_sync(0xffffffffu, stays);
  if (lane == 0) counts[warp] = __popc(votes);
  __syncthreads();
  int at = __popc(votes & ((1u << lane) - 1u));
  for (int w = 0; w < warp; ++w) at += counts[w];
  auto row_at = [&](int j) { return (table_s[j >> 4] * p.Hkv + g) * kBlockTokens + (j & 15); };
  if (stays) {
    kept[at] = tid;
    from_s[at] = row;
    if (at != tid) p.mass[row_at(at)] = x;   // (every weight has been read)
  }
  __syncthreads();
  const int pieces = p.row_bytes / 16, per = NT / pieces;
  const int lt = tid / pieces, lc = tid - lt * pieces;
  for (int j0 = 0; j0 < K; j0 += per * kWalkVecs) {
    uint4 xk[kWalkVecs], xv[kWalkVecs];
    int to[kWalkVecs];
#pragma unroll
    for (int q = 0; q < kWalkVecs; ++q) {
      const int j = j0 + q * per + lt, jc = min(j, K - 1);
      const int from = from_s[jc];
      to[q] = row_at(jc);
      if (lt >= per || j >= K || from == to[q]) to[q] = -1;
      if (to[q] >= 0) {
        const size_t off = static_cast<size_t>(from) * p.row_bytes + 16 * lc;
        xk[q] = *reinterpret_cast<const uint4 *>(p.k_cache + off);
        xv[q] = *reinterpret_cast<const uint4 *>(p.v_cache + off);
      }
    }
    __syncthreads();   // the step is read before any of it is written
#pragma unroll
    for (int q = 0; q < kWalkVecs; ++q)
      if (to[q] >= 0) {
        const size_t off = static_cast<size_t>(to[q]) * p.row_bytes + 16 * lc;
        *reinterpret_cast<uint4 *>(p.k_cache + off) = xk[q];
        *reinterpret_cast<uint4 *>(p.v_cache + off) = xv[q];
      }
  }
}

// CTA (row, head, part): part 0 walks K, 1 walks V, 2 the weights.
//
// The kept tokens ahead of the first dropped one stay where they are: one round of
// probes finds where they end.  From there on, kWalkTokens at a time, the cache rows
// they come from and go to are listed in shared memory (two round trips for all of
// them; looked up step by step they were two of every step's three), and while a step
// is stored the next one's reads are under way.
__global__ void __launch_bounds__(kMoveThreads, 4) evict_walk_kernel(const EvictParams p) {
  __shared__ int2 list[kWalkTokens];   // cache rows: from, to
  pdl_wait();
  const int u = blockIdx.x / 3, part = blockIdx.x - 3 * u;
  const int b = u / p.Hkv, g = u - b * p.Hkv;
  const int L = p.seq_lens[b], K = p.keep_lens[b];
  if (K >= L || K <= 0 || K > p.kept_stride) return;
  const int32_t *kept = p.kept + static_cast<size_t>(u) * p.kept_stride;
  const int tid = threadIdx.x;
  const int span = (K + kMoveThreads - 1) / kMoveThreads;
  const int probe = min((tid + 1) * span, K) - 1, last = kept[K - 1];
  const int stay = __syncthreads_count(kept[probe] == probe) * span;   // (kept[j] - j never falls)
  // (last < 0: the choice left this row alone, for a bad length or block)
  if (last < 0 || stay >= K) return;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  auto row_of = [&](int t) {   // (the pool has fewer than 2^31 rows)
    return (table[t >> 4] * p.Hkv + g) * kBlockTokens + (t & 15);
  };
  unsigned char *cache = part == 0 ? p.k_cache : p.v_cache;
  const int pieces = p.row_bytes / 16;           // 16-byte pieces of a token's row
  const int per = kMoveThreads / pieces;         // tokens in one round of the CTA
  const int lt = tid / pieces, lc = tid - lt * pieces;
  cache += 16 * lc;
  for (int j0 = stay; j0 < K; j0 += kWalkTokens) {
    const int n = min(kWalkTokens, K - j0);
    constexpr int kPer = kWalkTokens / kMoveThreads;
    int src[kPer], to[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) src[q] = kept[j0 + min(q * kMoveThreads + tid, n - 1)];
#pragma unroll
    for (int q = 0; q < kPer; ++q) to[q] = row_of(j0 + min(q * kMoveThreads + tid, n - 1));
#pragma unroll
    for (int q = 0; q < kPer; ++q) src[q] = row_of(src[q]);
    if (part == 2) {
      float x[kPer];
#pragma unroll
      for (int q = 0; q < kPer; ++q) x[q] = p.mass[src[q]];
      __syncthreads();   // read before any of it is written
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (q * kMoveThreads + tid < n) p.mass[to[q]] = x[q];
      continue;
    }
    __syncthreads();   // (the list before is done with)
#pragma unroll
    for (int q = 0; q < kPer; ++q) list[q * kMoveThreads + tid] = make_int2(src[q], to[q]);
    __syncthreads();
    const int step = per * kWalkVecs;
    auto load = [&](uint4(&x)[kWalkVecs], int(&dst)[kWalkVecs], int i0) {
#pragma unroll
      for (int q = 0; q < kWalkVecs; ++q) {
        const int i = i0 + q * per + lt;
        const int2 r = list[min(i, kWalkTokens - 1)];
        dst[q] = lt < per && i < n && r.x != r.y ? r.y : -1;
        if (dst[q] >= 0)
          x[q] = *reinterpret_cast<const uint4 *>(cache + static_cast<size_t>(r.x) * p.row_bytes);
      }
    };
    auto store = [&](const uint4(&x)[kWalkVecs], const int(&dst)[kWalkVecs]) {
#pragma unroll
      for (int q = 0; q < kWalkVecs; ++q)
        if (dst[q] >= 0)
          *reinterpret_cast<uint4 *>(cache + static_cast<size_t>(dst[q]) * p.row_bytes) = x[q];
    };
    uint4 x[kWalkVecs], y[kWalkVecs];
    int dx[kWalkVecs], dy[kWalkVecs];
    load(x, dx, 0);
    for (int i = 0; i < n; i += 2 * step) {
      load(y, dy, i + step);   // (its tokens lie behind every slot that is written by then)
      __syncthreads();         // a step is read before any of it is written
      store(x, dx);
      load(x, dx, i + 2 * step);
      __syncthreads();
      store(y, dy);
    }
  }
}

// One chunk of one (row, KV head): keys, values and weights.
__global__ void __launch_bounds__(kMoveThreads, 4) evict_chunk_kernel(const EvictParams p) {
  __shared__ int task_s, ok_s;
  __shared__ int2 lens_s[kChunkUnits];
  const int tid = threadIdx.x;
  const int units = p.B * p.Hkv;
  // (every row's lengths, so that they need not wait for the ticket; the choice's own
  // wait was over before it released this kernel: what came before it is in L2)
  if (tid < p.B) lens_s[tid] = make_int2(__ldcg(p.seq_lens + tid), __ldcg(p.keep_lens + tid));
  pdl_wait();
  if (tid == 0) {
    task_s = atomicAdd(p.ticket, 1);
    ok_s = 1;
  }
  __syncthreads();
  const int chunk = task_s / units, u = task_s - chunk * units;
  const int b = u / p.Hkv, g = u - b * p.Hkv;
  const int L = lens_s[b].x, K = lens_s[b].y;
  const int j0 = chunk * p.chunk;
  if (K >= L || j0 >= K || K > p.kept_stride) return;
  const int32_t *kept = p.kept + static_cast<size_t>(u) * p.kept_stride;
  const int nj = min(p.chunk, K - j0);
  const int pieces = p.row_bytes / 16;
  int src[kMoveVecs];   // where this thread's pieces come from (read beside what follows)
#pragma unroll
  for (int q = 0; q < kMoveVecs; ++q)
    src[q] = kept[j0 + min((tid + q * kMoveThreads) / pieces, nj - 1)];
  const int last = kept[j0 + nj - 1];
  // the chunks whose tokens lie in this chunk's slots (threads 0 and 1)
  int lo = 0, hi = 0;
  if (tid < 2) {
    const int32_t *below = p.below + static_cast<size_t>(u) * (p.chunks + 1) + chunk;
    lo = below[0];
    hi = below[1];
  }
  if (last < 0) return;   // the choice left this row alone (bad length or block)
  int32_t *flags = p.flags + static_cast<size_t>(u) * p.chunks;
  if (last == j0 + nj - 1) {   // every token up to here is where it belongs
    if (tid == 0) asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flags + chunk) : "memory");
    return;
  }
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  auto row_of = [&](int t) {
    return (static_cast<size_t>(table[t >> 4]) * p.Hkv + g) * kBlockTokens + (t & 15);
  };
  uint4 xk[kMoveVecs], xv[kMoveVecs];
  int dst[kMoveVecs];   // cache row, -1: nothing to move
  float xm[4];          // weights (a chunk has at most 1024 tokens)
  int msrc[4];
  // (each kind of read for all pieces before the next kind, and no branch between, so
  // that a round trip serves them all: one by one this phase took 3 to 6 us of a CTA's 7)
#pragma unroll
  for (int q = 0; q < 4; ++q) msrc[q] = kept[j0 + min(tid + q * kMoveThreads, nj - 1)];
  int from[kMoveVecs];
#pragma unroll
  for (int q = 0; q < kMoveVecs; ++q) {
    const int j = (tid + q * kMoveThreads) / pieces;
    from[q] = static_cast<int>(row_of(src[q]));
    const int to = static_cast<int>(row_of(j0 + min(j, nj - 1)));
    dst[q] = j < nj && src[q] != j0 + j ? to : -1;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) msrc[q] = static_cast<int>(row_of(msrc[q]));
#pragma unroll
  for (int q = 0; q < kMoveVecs; ++q) {
    const size_t at =
        static_cast<size_t>(from[q]) * p.row_bytes + 16 * ((tid + q * kMoveThreads) % pieces);
    if (dst[q] >= 0) {
      xk[q] = __ldcg(reinterpret_cast<const uint4 *>(p.k_cache + at));
      xv[q] = __ldcg(reinterpret_cast<const uint4 *>(p.v_cache + at));
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (tid + q * kMoveThreads < nj) xm[q] = __ldcg(p.mass + msrc[q]);
  // the chunks that have to have been read: mostly they were long ago, so a first
  // look goes out beside the reads
  int need = lo < hi ? (tid == 0 ? lo : hi - 1) / p.chunk : -1;
  if (need >= chunk) need = -1;   // (this one)
  auto is_read = [&]() {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flags + need) : "memory");
    return v != 0;
  };
  if (need >= 0 && is_read()) need = -1;
  __threadfence();   // this thread's reads are done before the flag is seen
  __syncthreads();
  // (the flag before any wait: what has been read never waits)
  if (tid == 0) asm volatile("st.relaxed.gpu.global.s32 [%0], 1;" ::"l"(flags + chunk) : "memory");
  if (need >= 0) {
    const long long t0 = clock64();
    while (!is_read()) {
      if (clock64() - t0 > kWaitCycles) {
        set_dev_err(p.err, PKV_DEVERR_TIMEOUT);
        ok_s = 0;
        break;
      }
    }
  }
  __syncthreads();
  if (!ok_s) return;
#pragma unroll
  for (int q = 0; q < kMoveVecs; ++q)
    if (dst[q] >= 0) {
      const size_t at =
          static_cast<size_t>(dst[q]) * p.row_bytes + 16 * ((tid + q * kMoveThreads) % pieces);
      *reinterpret_cast<uint4 *>(p.k_cache + at) = xk[q];
      *reinterpret_cast<uint4 *>(p.v_cache + at) = xv[q];
    }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = tid + q * kMoveThreads;
    if (j < nj) p.mass[row_of(j0 + j)] = xm[q];
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int chunk_tokens(int row_bytes) { return kChunkBytes / row_bytes; }

int check_sizes(int B, int Hkv, int d, int dtype, int kept_stride) {
  PKV_REQUIRE(dtype_ok(dtype), PKV_ERR_UNSUPPORTED, "dtype %d", dtype);
  PKV_REQUIRE(B >= 0 && B <= 65536 && Hkv > 0 && Hkv <= 4096, PKV_ERR_UNSUPPORTED,
              "B = %d, Hkv = %d", B, Hkv);
  const long long row_bytes = static_cast<long long>(d) * dtype_size(dtype);
  PKV_REQUIRE(d > 0 && row_bytes % 16 == 0 && row_bytes <= 1024, PKV_ERR_UNSUPPORTED,
              "head_dim * sizeof(dtype) must be a multiple of 16, at most 1024 (d=%d)", d);
  PKV_REQUIRE(kept_stride > 0, PKV_ERR_INVALID_ARG, "kept_stride must be positive");
  const long long chunks = (kept_stride + chunk_tokens(static_cast<int>(row_bytes)) - 1ll) /
                           chunk_tokens(static_cast<int>(row_bytes));
  PKV_REQUIRE(static_cast<long long>(B) * Hkv * chunks < (1ll << 31) &&
                  static_cast<long long>(B) * Hkv * kMaxCluster < (1ll << 31),
              PKV_ERR_UNSUPPORTED, "too many rows, heads and kept tokens");
  return PKV_OK;
}

template <typename K>
cudaError_t launch(K kern, long long grid, int threads, size_t smem, int cluster,
                   const EvictParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];   // (every kernel here waits before it touches memory)
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_evict_workspace_bytes(int32_t B, int32_t Hkv, int32_t d, int32_t dtype,
                                         int32_t kept_stride, size_t *bytes) {
  clear_error();
  PKV_REQUIRE(bytes, PKV_ERR_INVALID_ARG, "bytes is NULL");
  const int rc = check_sizes(B, Hkv, d, dtype, kept_stride);
  if (rc != PKV_OK) return rc;
  const int chunk = chunk_tokens(d * static_cast<int>(dtype_size(dtype)));
  const size_t chunks = (kept_stride + chunk - 1ll) / chunk;
  *bytes = 256 + align256(static_cast<size_t>(B) * Hkv * (2 * chunks + 1) * sizeof(int32_t));
  return PKV_OK;
}

extern "C" int pkv_evict(const pkv_evict_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  int rc = check_sizes(a->B, a->Hkv, a->d, a->dtype, a->kept_stride);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(a->sink >= 0 && a->recent >= 0, PKV_ERR_INVALID_ARG, "negative sink or recent");
  PKV_REQUIRE(a->num_blocks > 0, PKV_ERR_INVALID_ARG, "num_blocks must be positive");
  PKV_REQUIRE(a->bt_stride > 0 && a->bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              a->bt_stride);
  if (a->B == 0) return PKV_OK;
  PKV_REQUIRE(a->k_cache && a->v_cache && a->mass && a->block_tables && a->seq_lens &&
                  a->keep_lens && a->kept && a->workspace,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) |
               reinterpret_cast<uintptr_t>(a->mass)) %
                      16 == 0,
              PKV_ERR_INVALID_ARG, "caches and mass must be 16-byte aligned");
  PKV_REQUIRE(reinterpret_cast<uintptr_t>(a->workspace) % 256 == 0, PKV_ERR_INVALID_ARG,
              "workspace must be 256-byte aligned");
  size_t need = 0;
  rc = pkv_evict_workspace_bytes(a->B, a->Hkv, a->d, a->dtype, a->kept_stride, &need);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(a->workspace_bytes >= need, PKV_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed",
              a->workspace_bytes, need);
  EvictParams p;
  p.k_cache = static_cast<unsigned char *>(a->k_cache);
  p.v_cache = static_cast<unsigned char *>(a->v_cache);
  p.mass = a->mass;
  p.block_tables = a->block_tables;
  p.seq_lens = a->seq_lens;
  p.keep_lens = a->keep_lens;
  p.kept = a->kept;
  p.err = a->dev_err_flag;
  p.ticket = static_cast<int32_t *>(a->workspace);
  p.flags = p.ticket + 64;
  p.chunk = chunk_tokens(a->d * static_cast<int>(dtype_size(a->dtype)));
  p.chunks = static_cast<int>((a->kept_stride + p.chunk - 1ll) / p.chunk);
  p.below = p.flags + static_cast<size_t>(a->B) * a->Hkv * p.chunks;
  p.num_blocks = a->num_blocks;
  p.bt_stride = a->bt_stride;
  p.kept_stride = a->kept_stride;
  p.sink = a->sink;
  p.recent = a->recent;
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.row_bytes = a->d * static_cast<int>(dtype_size(a->dtype));
  const long long rows = static_cast<long long>(a->num_blocks) * a->Hkv * kBlockTokens;
  PKV_REQUIRE(rows < (1ll << 31), PKV_ERR_UNSUPPORTED, "pool too large for 32-bit row numbers");
  PKV_REQUIRE(!rows_overlap(a->k_cache, 0, rows * p.row_bytes, a->v_cache, 0, rows * p.row_bytes, 1),
              PKV_ERR_INVALID_ARG, "the caches overlap");
  // CTAs per row and head: 8 steps of keys each for the longest row, and while the
  // rows are few, enough to share it out (two steps at least)
  const long long units = static_cast<long long>(a->B) * a->Hkv;
  const long long longest = 16ll * a->bt_stride;
  int cluster = 1;
  while (cluster < kMaxCluster &&
         (longest > 8ll * cluster * kTileTokens ||
          (units * cluster < 152 && longest > 2ll * cluster * kTileTokens)))
    cluster *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (longest <= 256 || (longest <= 512 && units <= 152)) {   // (512: a CTA to an SM)
    const cudaError_t e = longest <= 256
                              ? launch(evict_small_kernel<256>, units, 256, 0, 1, p, s)
                              : launch(evict_small_kernel<512>, units, 512, 0, 1, p, s);
    PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "evict_small_kernel launch: %s",
                cudaGetErrorString(e));
    return PKV_OK;
  }
  const bool walk = units >= kChunkUnits;   // two CTAs a pair (K, V) fill the GPU
  if (walk) p.below = nullptr;
  const long long tiles = ((longest + kTileTokens - 1) / kTileTokens + cluster - 1) / cluster;
  p.cached = static_cast<int>(tiles < kMaxCached ? tiles : kMaxCached);
  static std::atomic<unsigned long long> attrs_set{0};
  PKV_CUDA_CHECK(set_attributes_once(attrs_set, [] {
    for (auto kern : {evict_select_kernel<4>, evict_select_kernel<8>}) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMaxCached * kTileTokens * 4);
      if (e == cudaSuccess)   // clusters of 16
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }));
  cudaError_t e = launch(tiles > 4 ? evict_select_kernel<8> : evict_select_kernel<4>,
                         units * cluster, kSelThreads,
                         static_cast<size_t>(p.cached) * kTileTokens * 4, cluster, p, s);
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "evict_select_kernel launch: %s",
              cudaGetErrorString(e));
  if (walk)
    e = launch(evict_walk_kernel, units * 3, kMoveThreads, 0, 1, p, s);
  else
    e = launch(evict_chunk_kernel, units * p.chunks, kMoveThreads, 0, 1, p, s);
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "evict compaction launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}
