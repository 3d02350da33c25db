// Eviction from the paged cache by accumulated attention weight (pkv_evict):
// choose the tokens to keep per (row, KV head), then compact keys, values and
// weights in place.
//
// Choice.  The m-th largest of a row's candidate weights is found by radix
// selection on order-preserving 32-bit keys (digits of 11, 11 and 10 bits, from
// the top): after each digit only the keys that share the threshold's digits so
// far still count.  Tokens above the threshold are kept, and of those equal to
// it the first few by index, so the choice does not depend on any order of
// execution.  One scan in token order then writes the kept indices ascending.
//
// Compaction.  The i-th kept token comes from index >= i, so when a CTA walks
// its kept tokens in order, a chunk's stores can only reach slots that this or
// an earlier chunk has already read: load a chunk into registers, barrier,
// store it.  CTAs share nothing: each owns one (row, KV head), one of K and V,
// and a column slice of the rows.
#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kScanPer = 8;          // tokens a thread takes in a step of the final scan
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;        // 16-byte pieces a thread has in flight

struct EvictParams {
  unsigned char *k_cache, *v_cache;
  float *mass;
  const int32_t *block_tables, *seq_lens, *keep_lens;
  int32_t *kept, *err;
  int num_blocks, bt_stride, kept_stride, sink, recent;
  int B, Hkv, row_bytes;
  int cached;                        // keys the select kernel keeps in shared memory
  int slices, slice_bytes;           // column slices of a K (or V) row
};

// Larger key <=> larger weight; -0 and +0 are equal, every NaN is the largest.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the threads before this one of v, and the total (kSelThreads threads).
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long *warp_sums,
                                                         unsigned long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const unsigned long long s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys_s[];   // [cached]
  __shared__ uint32_t hist[kBins];
  __shared__ unsigned long long warp_sums[kSelThreads / 32];
  __shared__ int bad, digit_s, left_s;
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv;
  const int L = p.seq_lens[b], K = p.keep_lens[b];
  int32_t *kept = p.kept + static_cast<size_t>(blockIdx.x) * p.kept_stride;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const bool bad_len = L < 0 || K < 0 || static_cast<long long>(L) > 16ll * p.bt_stride ||
                       min(L, K) > p.kept_stride;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (bad_len) {
    if (tid == 0 && g == 0) set_dev_err(p.err, PKV_DEVERR_BAD_LEN);
  } else {
    for (int j = tid; j < (L + 15) / 16; j += kSelThreads) {
      const int blk = table[j];
      if (blk < 0 || blk >= p.num_blocks) bad = 1;
    }
    __syncthreads();
    if (bad && tid == 0 && g == 0) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
  }
  const bool skip = bad_len || bad;
  const int n = skip ? 0 : min(L, K);
  for (int j = n + tid; j < p.kept_stride; j += kSelThreads) kept[j] = -1;
  if (skip) return;
  if (L <= K) {
    for (int j = tid; j < L; j += kSelThreads) kept[j] = j;
    return;
  }
  const int n_recent = min(p.recent, K), n_sink = min(p.sink, K - n_recent);
  const int c0 = n_sink, count = L - n_recent - n_sink;   // candidates [c0, c0 + count)
  const int m = K - n_recent - n_sink;                    // of which m stay, m < count
  for (int j = tid; j < n_sink; j += kSelThreads) kept[j] = j;
  for (int j = tid; j < n_recent; j += kSelThreads) kept[K - n_recent + j] = L - n_recent + j;
  if (m == 0) return;
  auto read_key = [&](int i) {
    const int t = c0 + i;
    return mass_key(
        p.mass[(static_cast<size_t>(table[t >> 4]) * p.Hkv + g) * kBlockTokens + (t & 15)]);
  };
  const int cached = min(count, p.cached);
  for (int i = tid; i < cached; i += kSelThreads) keys_s[i] = read_key(i);
  auto key_of = [&](int i) { return i < cached ? keys_s[i] : read_key(i); };
  // ---- the threshold: the m-th largest key ----
  uint32_t prefix = 0, mask = 0;   // the threshold's bits so far
  int left = m;                    // its rank among the keys with that prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t dm = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += kSelThreads) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dm], 1u);
    }
    __syncthreads();
    // bins from the top: thread i takes bins top - 4i .. top - 4i - 3
    uint32_t c[kBins / kSelThreads];
    unsigned long long sum = 0, total;
#pragma unroll
    for (int q = 0; q < kBins / kSelThreads; ++q) {
      c[q] = hist[kBins - 1 - (tid * (kBins / kSelThreads) + q)];
      sum += c[q];
    }
    unsigned long long above = block_scan(sum, warp_sums, &total);
#pragma unroll
    for (int q = 0; q < kBins / kSelThreads; ++q) {
      if (above < static_cast<unsigned long long>(left) &&
          above + c[q] >= static_cast<unsigned long long>(left)) {
        digit_s = kBins - 1 - (tid * (kBins / kSelThreads) + q);
        left_s = left - static_cast<int>(above);
      }
      above += c[q];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(digit_s) << shift;
    mask |= dm << shift;
    left = left_s;
    __syncthreads();
  }
  // ---- kept indices in token order: above the threshold, and the first
  // `left` of those equal to it ----
  int base_gt = 0, base_eq = 0;
  for (int i0 = 0; i0 < count; i0 += kSelThreads * kScanPer) {
    const int i1 = i0 + tid * kScanPer;
    uint32_t gt = 0, eq = 0;   // bit q: token i1 + q
#pragma unroll
    for (int q = 0; q < kScanPer; ++q)
      if (i1 + q < count) {
        const uint32_t k = key_of(i1 + q);
        gt |= (k > prefix ? 1u : 0u) << q;
        eq |= (k == prefix ? 1u : 0u) << q;
      }
    unsigned long long total;
    const unsigned long long v = static_cast<unsigned long long>(__popc(gt)) << 32 | __popc(eq);
    const unsigned long long before = block_scan(v, warp_sums, &total);
    int g_at = base_gt + static_cast<int>(before >> 32);
    int e_at = base_eq + static_cast<int>(before & 0xffffffffu);
#pragma unroll
    for (int q = 0; q < kScanPer; ++q) {
      const bool is_gt = gt >> q & 1u, is_eq = eq >> q & 1u;
      if (is_gt || (is_eq && e_at < left))
        kept[n_sink + g_at + min(e_at, left)] = c0 + i1 + q;
      g_at += is_gt;
      e_at += is_eq;
    }
    base_gt += static_cast<int>(total >> 32);
    base_eq += static_cast<int>(total & 0xffffffffu);
  }
}

// CTA (row, head, part): part < 2 * slices moves column slice part / 2 of K (even)
// or V (odd); part 2 * slices moves the weights.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  const int parts = 2 * p.slices + 1;
  const int u = blockIdx.x / parts, part = blockIdx.x - u * parts;
  const int b = u / p.Hkv, g = u - b * p.Hkv;
  const int L = p.seq_lens[b], K = p.keep_lens[b];
  if (K >= L || K <= 0 || K > p.kept_stride) return;
  const int32_t *kept = p.kept + static_cast<size_t>(u) * p.kept_stride;
  if (kept[0] < 0) return;   // the choice left this row alone (bad length or block)
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const int tid = threadIdx.x;
  auto row_of = [&](int t) {
    return (static_cast<size_t>(table[t >> 4]) * p.Hkv + g) * kBlockTokens + (t & 15);
  };
  if (part == 2 * p.slices) {
    for (int j0 = 0; j0 < K; j0 += kMoveThreads * kMoveBatch) {
      float x[kMoveBatch];
      bool go[kMoveBatch];
#pragma unroll
      for (int q = 0; q < kMoveBatch; ++q) {
        const int j = j0 + q * kMoveThreads + tid;
        const int s = j < K ? kept[j] : j;
        go[q] = s != j;
        if (go[q]) x[q] = p.mass[row_of(s)];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kMoveBatch; ++q) {
        const int j = j0 + q * kMoveThreads + tid;
        if (go[q]) p.mass[row_of(j)] = x[q];
      }
    }
    return;
  }
  unsigned char *cache = (part & 1 ? p.v_cache : p.k_cache) +
                         static_cast<size_t>(part >> 1) * p.slice_bytes;
  const int width = min(p.slice_bytes, p.row_bytes - (part >> 1) * p.slice_bytes);
  const int pieces = width / 16;                 // 16-byte pieces of a token's slice
  const int per = kMoveThreads / pieces;         // tokens in one round of the CTA
  const int lt = tid / pieces, lc = tid - lt * pieces;
  const bool on = lt < per;
  for (int j0 = 0; j0 < K; j0 += per * kMoveBatch) {
    uint4 x[kMoveBatch];
    bool go[kMoveBatch];
#pragma unroll
    for (int q = 0; q < kMoveBatch; ++q) {
      const int j = j0 + q * per + lt;
      const int s = on && j < K ? kept[j] : j;
      go[q] = s != j;
      if (go[q]) x[q] = *reinterpret_cast<const uint4 *>(cache + row_of(s) * p.row_bytes + 16 * lc);
    }
    __syncthreads();   // the chunk is read before any of it is written
#pragma unroll
    for (int q = 0; q < kMoveBatch; ++q) {
      const int j = j0 + q * per + lt;
      if (go[q]) *reinterpret_cast<uint4 *>(cache + row_of(j) * p.row_bytes + 16 * lc) = x[q];
    }
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_evict(const pkv_evict_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  PKV_REQUIRE(dtype_ok(a->dtype), PKV_ERR_UNSUPPORTED, "dtype %d", a->dtype);
  PKV_REQUIRE(a->B >= 0 && a->B <= 65536 && a->Hkv > 0 && a->Hkv <= 4096, PKV_ERR_UNSUPPORTED,
              "B = %d, Hkv = %d", a->B, a->Hkv);
  const long long row_bytes = static_cast<long long>(a->d) * dtype_size(a->dtype);
  PKV_REQUIRE(a->d > 0 && row_bytes % 16 == 0 && row_bytes <= 1024, PKV_ERR_UNSUPPORTED,
              "head_dim * sizeof(dtype) must be a multiple of 16, at most 1024 (d=%d)", a->d);
  PKV_REQUIRE(a->sink >= 0 && a->recent >= 0, PKV_ERR_INVALID_ARG, "negative sink or recent");
  PKV_REQUIRE(a->num_blocks > 0, PKV_ERR_INVALID_ARG, "num_blocks must be positive");
  PKV_REQUIRE(a->bt_stride > 0 && a->bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              a->bt_stride);
  PKV_REQUIRE(a->kept_stride > 0, PKV_ERR_INVALID_ARG, "kept_stride must be positive");
  if (a->B == 0) return PKV_OK;
  PKV_REQUIRE(a->k_cache && a->v_cache && a->mass && a->block_tables && a->seq_lens &&
                  a->keep_lens && a->kept,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE((reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache)) %
                      16 == 0,
              PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  EvictParams p;
  p.k_cache = static_cast<unsigned char *>(a->k_cache);
  p.v_cache = static_cast<unsigned char *>(a->v_cache);
  p.mass = a->mass;
  p.block_tables = a->block_tables;
  p.seq_lens = a->seq_lens;
  p.keep_lens = a->keep_lens;
  p.kept = a->kept;
  p.err = a->dev_err_flag;
  p.num_blocks = a->num_blocks;
  p.bt_stride = a->bt_stride;
  p.kept_stride = a->kept_stride;
  p.sink = a->sink;
  p.recent = a->recent;
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.row_bytes = static_cast<int>(row_bytes);
  const long long longest = 16ll * a->bt_stride;
  p.cached = static_cast<int>(longest < 40960 ? longest : 40960);
  // column slices: split rows (down to a 32-byte sector) until the CTAs fill the GPU
  const long long units = static_cast<long long>(a->B) * a->Hkv;
  p.slices = 1;
  p.slice_bytes = p.row_bytes;
  while (units * 2 * p.slices < 2 * 152 && p.slice_bytes % 64 == 0) {
    p.slices *= 2;
    p.slice_bytes /= 2;
  }
  const long long grid = units * (2 * p.slices + 1);
  PKV_REQUIRE(grid < (1ll << 31), PKV_ERR_UNSUPPORTED, "too many rows and heads");
  static std::atomic<unsigned long long> attrs_set{0};
  PKV_CUDA_CHECK(set_attributes_once(attrs_set, [] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                40960 * 4);
  }));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  evict_select_kernel<<<static_cast<unsigned>(units), kSelThreads, p.cached * sizeof(uint32_t), s>>>(
      p);
  PKV_LAUNCH_CHECK("evict_select_kernel");
  evict_move_kernel<<<static_cast<unsigned>(grid), kMoveThreads, 0, s>>>(p);
  PKV_LAUNCH_CHECK("evict_move_kernel");
  return PKV_OK;
}
