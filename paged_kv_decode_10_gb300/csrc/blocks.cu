// Moves within and between the pools of a paged cache: whole blocks (pkv_copy_blocks:
// forks' last blocks, a pool of another size) and the accepted path of a tree of drafted
// tokens to the front of the tree's slots (pkv_tree_accept).  Both take the pools of
// every layer, keys and values, in one launch.  Bytes move as they are, whatever the type.
#include <algorithm>
#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
// Pools that a small call has room for: the parameters of a call of 256 pools, 2 to 4 KB, are
// handed over at every launch.
constexpr int kFewPools = 8;

// ---- whole blocks ---------------------------------------------------------------
// A CTA copies one chunk of one block of one pool: kWide 16-byte pieces a thread, all
// read before the first is written.  Bound by memory: 1023 blocks of 32 KB in 16 pools, 156
// us, 6.9 TB/s.  (A few blocks: by the call, 1.6 us in a graph.)
template <int POOLS>
struct CopyParams {
  const int32_t *src_blocks, *dst_blocks;
  int32_t *err;
  int n, src_num, dst_num, chunks;
  long long pieces;                    // of 16 bytes, a block
  const uint4 *src[POOLS];
  uint4 *dst[POOLS];
};

template <int WIDE, int POOLS>
__global__ void __launch_bounds__(kThreads)
    copy_blocks_kernel(const __grid_constant__ CopyParams<POOLS> p) {
  pdl_wait();
  const unsigned u = blockIdx.x / static_cast<unsigned>(p.chunks);
  const int chunk = static_cast<int>(blockIdx.x - u * p.chunks);
  const unsigned pool = u / static_cast<unsigned>(p.n);
  const int i = static_cast<int>(u - pool * p.n);
  const int from = p.src_blocks[i], to = p.dst_blocks[i];
  if (from < 0 || to < 0) return;
  if (from >= p.src_num || to >= p.dst_num) {
    if (threadIdx.x == 0) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
    return;
  }
  const uint4 *s = p.src[pool] + from * p.pieces;
  uint4 *d = p.dst[pool] + to * p.pieces;
  const long long at = static_cast<long long>(chunk) * (WIDE * kThreads) + threadIdx.x;
  uint4 v[WIDE];
#pragma unroll
  for (int k = 0; k < WIDE; ++k)
    if (at + k * kThreads < p.pieces) v[k] = __ldcs(s + at + k * kThreads);
#pragma unroll
  for (int k = 0; k < WIDE; ++k)
    if (at + k * kThreads < p.pieces) __stcs(d + at + k * kThreads, v[k]);
}

// ---- the accepted path ----------------------------------------------------------
// Token base + j of row b takes the key and value of token base + path[j].  path ascends
// strictly, so path[j] >= j: going up in j, whatever is overwritten has been read, and a
// thread that owns one 16-byte column of one head of one pool needs nobody else for
// that.  A CTA serves kThreads columns of one row at a time; it checks the row first (every
// CTA of a row comes to the same answer) and lists its moves in shared memory.  A piece is a
// head of a token (256 bytes, the next head's 4 KB further).  64 rows that accept 1 to 12
// nodes, 64 pools of 8 heads of 128: 21 us, 4.6 TB/s, in two waves of CTAs whose shares are
// uneven (DRAM 34 % busy); 3 rows, 2 pools: 3 us, the chain of reads before the moves.
template <int POOLS>
struct AcceptParams {
  const int32_t *block_tables, *seq_lens, *node_starts, *path, *accept_lens;
  int32_t *err;
  int B, T, Hkv, num_blocks, bt_stride, path_stride, n_pools, chunks;
  unsigned cols;                       // of 16 bytes, a head
  uint4 *pool[POOLS];
};
constexpr int kMoves = 256;   // listed at a time
constexpr int kFlight = 8;    // tokens a thread reads before it writes them

template <int POOLS>
__global__ void __launch_bounds__(kThreads)
    tree_accept_kernel(const __grid_constant__ AcceptParams<POOLS> p) {
  __shared__ long long from_s[kMoves], to_s[kMoves];   // offsets in a pool, of head 0's column 0
  pdl_wait();
  const int tid = threadIdx.x;
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.chunks));
  const int chunk = static_cast<int>(blockIdx.x - static_cast<unsigned>(b) * p.chunks);
  const int s0 = p.node_starts[b], s1 = p.node_starts[b + 1], len = p.seq_lens[b];
  const int a = p.accept_lens[b];
  const int32_t *path = p.path + static_cast<size_t>(b) * p.path_stride;
  const int32_t *table = p.block_tables + static_cast<size_t>(b) * p.bt_stride;
  const long long n = static_cast<long long>(s1) - s0;
  bool bad = s0 < 0 || n < 0 || s1 > p.T || len < n || len > 16ll * p.bt_stride || a < 0 ||
             a > p.path_stride || a > n;
  bool bad_block = false;
  const int base = bad ? 0 : len - static_cast<int>(n);
  auto slot = [&](int t) {   // of token t (-1: its block lies outside the pool)
    const int blk = table[t / kBlockTokens];
    return blk >= 0 && blk < p.num_blocks ? blk * kBlockTokens + t % kBlockTokens : -1;
  };
  if (!bad)
    for (int j = tid; j < a; j += kThreads) {
      const int i = path[j], before = j > 0 ? path[j - 1] : -1;
      if (i <= before || i >= n)
        bad = true;
      else if (i != j && (slot(base + i) < 0 || slot(base + j) < 0))
        bad_block = true;
    }
  bad = __syncthreads_or(bad);
  bad_block = __syncthreads_or(bad_block);
  if (bad || bad_block) {
    if (tid == 0) set_dev_err(p.err, bad ? PKV_DEVERR_BAD_LEN : PKV_DEVERR_BAD_BLOCK);
    return;
  }
  auto offset = [&](int slot) {   // [num_blocks, Hkv, 16, cols]
    return (static_cast<long long>(slot / kBlockTokens) * p.Hkv * kBlockTokens + slot % kBlockTokens) *
           p.cols;
  };
  const unsigned per_pool = static_cast<unsigned>(p.Hkv * p.cols), items = per_pool * p.n_pools;
  for (int j0 = 0; j0 < a; j0 += kMoves) {
    const int m = min(kMoves, a - j0);
    if (j0) __syncthreads();
    if (tid < m) {
      const int j = j0 + tid, i = path[j];
      from_s[tid] = i == j ? -1 : offset(slot(base + i));   // (-1: stays where it is)
      to_s[tid] = i == j ? -1 : offset(slot(base + j));
    }
    __syncthreads();
    for (unsigned item = chunk * kThreads + tid; item < items; item += p.chunks * kThreads) {
      const unsigned pool = item / per_pool, r = item - pool * per_pool;
      const unsigned h = r / p.cols, c = r - h * p.cols;
      uint4 *mine = p.pool[pool] + static_cast<size_t>(h) * (kBlockTokens * p.cols) + c;
      for (int j = 0; j < m; j += kFlight) {
        uint4 v[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k)
          if (j + k < m && from_s[j + k] >= 0) v[k] = mine[from_s[j + k]];
#pragma unroll
        for (int k = 0; k < kFlight; ++k)
          if (j + k < m && from_s[j + k] >= 0) mine[to_s[j + k]] = v[k];
      }
    }
  }
}
static_assert(kMoves <= kThreads, "a thread lists one move");

// Whether a pool that is written overlaps another pool (given ones may be read and
// written at once, if they are the same pool).
struct Span {
  uintptr_t at;
  long long bytes;
  bool written;
};
bool written_overlap(Span *spans, int n) {
  std::sort(spans, spans + n, [](const Span &x, const Span &y) { return x.at < y.at; });
  uintptr_t read_end = 0, written_end = 0;
  for (int i = 0; i < n; ++i) {
    const Span &x = spans[i];
    if (x.at < written_end || (x.written && x.at < read_end)) return true;
    uintptr_t &end = x.written ? written_end : read_end;
    end = std::max(end, x.at + static_cast<uintptr_t>(x.bytes));
  }
  return false;
}

template <int POOLS>
int copy_blocks(const pkv_copy_args *a, void *stream) {
  CopyParams<POOLS> p;
  for (int i = 0; i < a->n_pools; ++i) {
    PKV_REQUIRE(a->src[i] && a->dst[i], PKV_ERR_INVALID_ARG, "pool %d is NULL", i);
    PKV_REQUIRE(((reinterpret_cast<uintptr_t>(a->src[i]) | reinterpret_cast<uintptr_t>(a->dst[i])) &
                 15) == 0,
                PKV_ERR_INVALID_ARG, "pool %d must be 16-byte aligned", i);
    p.src[i] = static_cast<const uint4 *>(a->src[i]);
    p.dst[i] = static_cast<uint4 *>(a->dst[i]);
  }
  const long long src_bytes = a->src_num_blocks * a->block_bytes,
                  dst_bytes = a->dst_num_blocks * a->block_bytes;
  Span spans[2 * POOLS];
  int n_spans = 0;
  for (int i = 0; i < a->n_pools; ++i) {
    spans[n_spans++] = Span{reinterpret_cast<uintptr_t>(a->dst[i]), dst_bytes, true};
    if (a->src[i] != a->dst[i])
      spans[n_spans++] = Span{reinterpret_cast<uintptr_t>(a->src[i]), src_bytes, false};
  }
  PKV_REQUIRE(!written_overlap(spans, n_spans), PKV_ERR_INVALID_ARG,
              "a destination pool overlaps another pool");
  p.src_blocks = a->src_blocks;
  p.dst_blocks = a->dst_blocks;
  p.err = a->dev_err_flag;
  p.n = a->n;
  p.src_num = a->src_num_blocks;
  p.dst_num = a->dst_num_blocks;
  p.pieces = a->block_bytes / 16;
  // Chunks of 8 KB (2 pieces a thread) while larger ones would leave SMs without work, 32 KB
  // once they give each of the 152 SMs 8 and more.
  const long long blocks = static_cast<long long>(a->n) * a->n_pools;
  const int wide = blocks * p.pieces >= 8ll * 8 * kThreads * 152 ? 8 : 2;
  const long long chunks = (p.pieces + wide * kThreads - 1) / (wide * kThreads);
  PKV_REQUIRE(blocks * chunks < (1ll << 31), PKV_ERR_UNSUPPORTED, "too many blocks for one call");
  p.chunks = static_cast<int>(chunks);
  const unsigned grid = static_cast<unsigned>(blocks * chunks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = wide == 8 ? launch_waiting(copy_blocks_kernel<8, POOLS>, grid, kThreads, 0, s, p)
                                  : launch_waiting(copy_blocks_kernel<2, POOLS>, grid, kThreads, 0, s, p);
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "copy_blocks launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

template <int POOLS>
int tree_accept(const pkv_accept_args *a, long long head, void *stream) {
  AcceptParams<POOLS> p;
  Span spans[POOLS];
  const long long bytes = a->num_blocks * kBlockTokens * head * a->Hkv;
  for (int i = 0; i < a->n_pools; ++i) {
    PKV_REQUIRE(a->pools[i] && (reinterpret_cast<uintptr_t>(a->pools[i]) & 15) == 0,
                PKV_ERR_INVALID_ARG, "pool %d must be given, 16-byte aligned", i);
    spans[i] = Span{reinterpret_cast<uintptr_t>(a->pools[i]), bytes, true};
    p.pool[i] = static_cast<uint4 *>(a->pools[i]);
  }
  PKV_REQUIRE(!written_overlap(spans, a->n_pools), PKV_ERR_INVALID_ARG, "two pools overlap");
  p.block_tables = a->block_tables;
  p.seq_lens = a->seq_lens;
  p.node_starts = a->node_starts;
  p.path = a->path;
  p.accept_lens = a->accept_lens;
  p.err = a->dev_err_flag;
  p.B = a->B;
  p.T = a->T;
  p.Hkv = a->Hkv;
  p.cols = static_cast<unsigned>(head / 16);
  p.num_blocks = a->num_blocks;
  p.bt_stride = a->bt_stride;
  p.path_stride = a->path_stride;
  p.n_pools = a->n_pools;
  const long long items = static_cast<long long>(a->Hkv) * p.cols * a->n_pools;   // below 2^28
  // As many CTAs as there are pieces of kThreads columns, but no more than about 8 to each of
  // the 152 SMs (two waves: at 58 registers 4 fit at once): looking the row over takes a CTA
  // longer than a piece's moves.
  const long long pieces = (items + kThreads - 1) / kThreads, most = a->B < 1216 ? 1216 / a->B : 1;
  p.chunks = static_cast<int>(pieces < most ? pieces : most);
  const unsigned grid = static_cast<unsigned>(p.chunks) * a->B;
  const cudaError_t e =
      launch_waiting(tree_accept_kernel<POOLS>, grid, kThreads, 0, static_cast<cudaStream_t>(stream), p);
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "tree_accept launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_copy_blocks(const pkv_copy_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  PKV_REQUIRE(a->n >= 0 && a->n_pools >= 0, PKV_ERR_INVALID_ARG, "negative size");
  PKV_REQUIRE(a->n_pools <= PKV_MAX_POOLS, PKV_ERR_UNSUPPORTED, "%d pools > %d", a->n_pools,
              PKV_MAX_POOLS);
  if (a->n == 0 || a->n_pools == 0) return PKV_OK;
  PKV_REQUIRE(a->src && a->dst && a->src_blocks && a->dst_blocks, PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(a->src_num_blocks > 0 && a->dst_num_blocks > 0, PKV_ERR_INVALID_ARG,
              "pools must have blocks");
  PKV_REQUIRE(a->block_bytes > 0 && a->block_bytes % 16 == 0 && a->block_bytes < (1ll << 31),
              PKV_ERR_INVALID_ARG, "block_bytes %lld must be a positive multiple of 16 below 2^31",
              (long long)a->block_bytes);
  PKV_REQUIRE(static_cast<long long>(a->n) * a->n_pools < (1ll << 31), PKV_ERR_UNSUPPORTED,
              "too many blocks for one call");
  return a->n_pools <= kFewPools ? copy_blocks<kFewPools>(a, stream) : copy_blocks<PKV_MAX_POOLS>(a, stream);
}

extern "C" int pkv_tree_accept(const pkv_accept_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a, PKV_ERR_INVALID_ARG, "args is NULL");
  PKV_REQUIRE(a->B >= 0 && a->T >= 0 && a->n_pools >= 0, PKV_ERR_INVALID_ARG, "negative size");
  PKV_REQUIRE(a->B <= 65536, PKV_ERR_UNSUPPORTED, "B %d > 65536", a->B);
  PKV_REQUIRE(a->n_pools <= PKV_MAX_POOLS, PKV_ERR_UNSUPPORTED, "%d pools > %d", a->n_pools,
              PKV_MAX_POOLS);
  PKV_REQUIRE(dtype_ok(a->dtype), PKV_ERR_UNSUPPORTED, "dtype %d", a->dtype);
  if (a->B == 0 || a->n_pools == 0) return PKV_OK;
  PKV_REQUIRE(a->pools && a->block_tables && a->seq_lens && a->node_starts && a->path &&
                  a->accept_lens,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(a->Hkv > 0 && a->d > 0, PKV_ERR_INVALID_ARG, "non-positive size");
  PKV_REQUIRE(a->num_blocks > 0, PKV_ERR_INVALID_ARG, "num_blocks must be positive");
  PKV_REQUIRE(static_cast<long long>(a->num_blocks) * kBlockTokens < (1ll << 31), PKV_ERR_UNSUPPORTED,
              "pool too large for 32-bit slots");
  PKV_REQUIRE(a->bt_stride > 0 && a->bt_stride < (1 << 26), PKV_ERR_INVALID_ARG, "bt_stride %d",
              a->bt_stride);
  PKV_REQUIRE(a->path_stride > 0, PKV_ERR_INVALID_ARG, "path_stride %d", a->path_stride);
  const long long head = static_cast<long long>(a->d) * static_cast<long long>(dtype_size(a->dtype));
  PKV_REQUIRE(head % 16 == 0, PKV_ERR_UNSUPPORTED, "a head of %lld bytes is no multiple of 16", head);
  PKV_REQUIRE(a->Hkv * (head / 16) <= (1 << 20), PKV_ERR_UNSUPPORTED, "too many heads");
  return a->n_pools <= kFewPools ? tree_accept<kFewPools>(a, head, stream)
                                 : tree_accept<PKV_MAX_POOLS>(a, head, stream);
}
