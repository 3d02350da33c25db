// Attention of drafted tokens on the 5th-generation tensor cores (bf16): up to 256 query
// rows (nodes x group heads of one batch row and KV head) against 128 tokens a step.
//
// Mathematics.  S = Q K^T and O = P V with P = 2^(S c - m), two 128 x 128 x d products per
// 128 rows and 128 tokens, online softmax between them; tokens that a node does not see
// have P = 0.  The cached tokens are read once for all nodes of the row and all heads of
// the group.
//
// Roles (one CTA per SM, its share of the positions of tree.h):
//  * warp 8 finds the CTA's items, hands them out through a short queue in shared memory
//    and loads Q and K by TMA; warp 11 loads V.  16-token pages go into 128-byte-swizzled
//    slabs, K-major for the first product, the same bytes MN-major for the second.  (With
//    one warp for both, a K tile waited for the V tile ahead of it, which waits for a
//    product: a load's latency a tile, 3.7 TB/s.)
//  * warps 0-3 and 4-7: a softmax warpgroup per slot.  A slot is a Q tile and an
//    accumulator pair (S, O) in tensor memory; thread r owns query row r, weights go back
//    as bf16 over their scores.
//  * warps 9 and 10 issue the products of one slot each.
// An item of more than 128 rows takes both slots, which share its K and V tiles and take
// turns in the products.  Smaller ones take one slot each, alternately: while one slot
// finishes an item and writes it out, the other is at work on the next, so the loads never
// pause between items.  The largest score is followed only when it grows by more than 2^8
// (kLazy): weights up to 2^8 are exact enough in bf16.
//
// Masks.  Only steps that reach past the tokens every row sees (the cached ones, and in a
// chain the nodes ahead of the item's) look at mask bits, 32 at a time.  What a node does not
// see may be anything, and 0 * NaN is NaN: so the issuing warp (of a tile that both slots use,
// slot 0's) looks over the values of such tokens while the softmax is at work, and where one
// is not finite the element is zeroed in shared memory for the product and added at the end
// to the rows that see it (any positive weight leaves NaN and infinity what they are).
//
// The code is kept short: rare paths are functions of their own, the rows' output is written
// in a loop.  A first form of 150 KB (two slots merged at the end of every item, everything
// unrolled) spent 8 us an item, mostly on instructions that were not in the cache.
//
// Bound by the loads while rows are few (64 rows of 4000 tokens, 4 nodes, 32/8 heads of 128:
// 169 us with the join, 6.2 TB/s), by the chain product, exponentials, product of the two
// slots where they are many: a step of 256 rows takes 2850 clocks, 2048 of them products (one
// row of 131072 tokens, 61 nodes, 32/4 heads of 128: 98 us with the join, 1.3 PFLOP/s).  The
// largest scores come with their load (a search of its own: 103 us against 101), the next tile
// of K is looked for while there is time (101 to 98).  A third stage for K or V, and Q loaded
// ahead of K, gained nothing or lost 2 %.
#include "tensor_core.cuh"
#include "tree.h"

namespace pkv {
namespace {

constexpr int kTile = 128;                    // tokens of a step, rows of a slot
constexpr int kPages = kTile / kBlockTokens;  // pages of a step
constexpr int kSoftmax = 256, kThreads = 384;
// registers a thread: 168 at launch; the softmax warpgroups hold a row of 128
// scores and take 216, what the third warpgroup gives up (2 * 216 + 72 = 3 * 168)
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr float kLazy = 8.0f;
constexpr int kHalf = 2;                      // 32-token pieces of P after which P V starts
constexpr long long kDrainCycles = 1ll << 31;
constexpr long long kPollLimit = 4096;
constexpr int kBoundary = 2;
constexpr int kQueue = 8;                     // items handed out and not yet written out
constexpr int kBadRing = 16, kOddRing = 4;

template <int D>
struct Lay {
  static constexpr int kSlabs = D / 64;                   // 128-byte column slabs
  static constexpr int kSlab = kTile * 128;               // bytes of a slab of a tile
  static constexpr int kMat = kSlabs * kSlab;             // bytes of a tile of Q, K or V
  static constexpr int NS = D == 128 ? 2 : 4;             // K and V stages
  static constexpr int kQ = 0;                            // [2] tiles, one per slot
  static constexpr int kK = 2 * kMat;                     // [NS]
  static constexpr int kV = kK + NS * kMat;               // [NS]
  static constexpr int kItems = kV + NS * kMat;           // [kQueue] 64 bytes
  static constexpr int kBars = kItems + kQueue * 64;
  static constexpr int kNumBars = 4 * NS + 2 * kQueue + 16;
  static constexpr int kBad = kBars + kNumBars * 8;       // [kBadRing] pages outside the pool
  static constexpr int kMisc = kBad + kBadRing;
  static constexpr int kBytes = kMisc + 4 * (kOddRing + 4) + 1024;   // + alignment slack
};

using Walk = TreeWalk<kTile, kBoundary>;

// An item as it is handed out: 64 bytes.
struct Handed {
  int q0, nodes, g, b;
  int base, n, tokens, n0;
  int t0, t1, slots, part;       // slots: 1, 2 or both; part: partial slot or -1 (whole)
  int special, pad[3];           // first token that rows may differ in
};

// Bits 15 and 31: a half's exponent is all ones (its sum with the lowest exponent bit
// carries into the sign's place).
__device__ __forceinline__ uint32_t odd_word(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t clean_word(uint32_t w) {
  const uint32_t odd = odd_word(w);
  return w & ~((odd & 0x8000u ? 0xffffu : 0u) | (odd >> 31 ? 0xffff0000u : 0u));
}

__device__ __forceinline__ bool in_pool(const TreeParams &p, int blk) {
  return blk >= 0 && blk < p.num_blocks;
}

// A wait of the whole warp: what is not there at once is waited for in a function (of 30
// waits, each with its own loop, the kernel would be a third longer).
template <bool POLL>
__device__ __noinline__ bool wait_longer(const Waiter<POLL> w, uint64_t *bar, uint32_t parity) {
  return w(bar, parity);
}
template <bool POLL>
struct WarpWaiter {
  Waiter<POLL> w;
  __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, w.done(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_longer<POLL>(w, bar, parity));
  }
};

// Until the copies of more than `tile` tiles were started.  A barrier says only whether its
// phase is even or odd, and a slot that comes back to the stages after the other slot's items
// does not know how many phases went by: once its tile's copies are under way, the phase is
// the tile's until this slot hands the stage back.
template <bool POLL>
__device__ __noinline__ bool wait_started(const Waiter<POLL> w, volatile int *started, int tile) {
  const long long t0 = clock64();
  while (*started <= tile) {
    if (*w.abort) return false;
    if (clock64() - t0 > w.limit) {
      *w.abort = 1;
      set_dev_err(w.err, PKV_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Values of rows [first, last) of a V tile that are not finite become zero (one warp).
template <int D>
__device__ __noinline__ void clean_values(unsigned char *vt, int first, int last, int lane) {
  for (int s = 0; s < Lay<D>::kSlabs; ++s)
    for (int c = first * 8 + lane; c < last * 8; c += 32) {
      uint4 *at = reinterpret_cast<uint4 *>(vt + s * Lay<D>::kSlab + c * 16);
      const uint4 v = *at;
      *at = make_uint4(clean_word(v.x), clean_word(v.y), clean_word(v.z), clean_word(v.w));
    }
}
// Rows of a V tile that do not count become zero (one warp): pages of `bad`, and those behind
// the last token within its page.
template <int D>
__device__ __noinline__ void zero_values(unsigned char *vt, int valid, uint32_t bad, int lane) {
  for (int pg = 0; pg * kBlockTokens < valid; ++pg) {
    const int end = (pg + 1) * kBlockTokens;
    const int from = bad >> pg & 1 ? end - kBlockTokens : min(end, valid);
    for (int s = 0; s < Lay<D>::kSlabs; ++s)
      for (int c = from * 8 + lane; c < end * 8; c += 32)
        *reinterpret_cast<uint4 *>(vt + s * Lay<D>::kSlab + c * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// What clean_values left out, added to the outputs of one query row (`out`: bf16 or, of a
// part, float32): any positive weight leaves infinity and NaN what they are.
template <int D>
__device__ __noinline__ void add_odd_values(const TreeParams &p, const Handed it, int node, void *out,
                                            bool part) {
  const int32_t *table = p.tables + static_cast<size_t>(it.b) * p.bt_stride;
  const uint32_t *words =
      p.mask ? p.mask + static_cast<size_t>(it.q0 + node) * p.mask_words : nullptr;
  for (int tok = max(it.special, it.t0 * kTile); tok < min(it.tokens, it.t1 * kTile); ++tok) {
    const int blk = table[tok / kBlockTokens];
    if (!in_pool(p, blk) ||
        !(tree_sees(words, p.mask_words, it.n0 + node, it.base, it.tokens, tok) & 1u))
      continue;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                             ((static_cast<size_t>(blk) * p.Hkv + it.g) * kBlockTokens +
                              tok % kBlockTokens) * D;
    for (int c = 0; c < D; ++c) {
      const float x = __bfloat162float(v[c]);
      if (isfinite(x)) continue;
      if (part) {
        static_cast<float *>(out)[c] += x;
      } else {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out) + c;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + x);
      }
    }
  }
}

template <int D, bool POLL>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TreeParams p) {
  using L = Lay<D>;
  constexpr int NS = L::NS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *k_full = bars, *k_empty = bars + NS, *v_full = bars + 2 * NS, *v_empty = bars + 3 * NS;
  uint64_t *i_full = bars + 4 * NS, *i_empty = i_full + kQueue;
  uint64_t *s_full = i_empty + kQueue, *p_ready = s_full + 2, *o_full = s_full + 4;   // [2] each
  uint64_t *q_full = s_full + 6, *q_empty = s_full + 8, *turn = s_full + 10, *p_half = s_full + 12;
  uint64_t *drain = s_full + 14;
  volatile uint8_t *bad_s = reinterpret_cast<volatile uint8_t *>(smem + L::kBad);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  // misc: a wait gave up, tmem, items with values that are not finite [kOddRing] (number + 1),
  // tiles whose copies of K and of V were started
  constexpr int kStartedK = 2 + kOddRing, kStartedV = kStartedK + 1;

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);   // one arrival per slot
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], 3 + kSoftmax / 32);   // V, issuers, softmax warps
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&p_ready[m], kTile / 32);   // one arrival per warp
      mbar_init(&p_half[m], kTile / 32);
      mbar_init(&o_full[m], 1);
      mbar_init(&q_full[m], 1);
      mbar_init(&q_empty[m], 1);
      mbar_init(&turn[m], 1);
    }
    mbar_init(drain, 2);
    misc[0] = 0;
    for (int i = 0; i < kOddRing + 2; ++i) misc[2 + i] = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(const_cast<int *>(misc + 1)))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: what starts then may read what was there before)
  const int cta = blockIdx.x;
  // (few rows: warp 8 finds its share by itself, while nobody waits for it)
  Walk walk = {};
  if (p.B > kWarpRows)
    walk = tree_begin<kTile, kBoundary, kThreads>(p, cta);   // (synchronises the CTA)
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(static_cast<uint32_t>(misc[1]));
  // (by arithmetic: arrays indexed by the slot would live in local memory)
  auto tS = [tmem](int m) { return tmem + 128u * m; };
  auto tO = [tmem](int m) { return tmem + 256u + 128u * m; };
  const Waiter<POLL> wait_here{misc, p.err, p.wait_limit};
  const WarpWaiter<POLL> wait_there{wait_here};
  Handed *items = reinterpret_cast<Handed *>(smem + L::kItems);
  // The i-th item of the queue (for the whole warp; t1 == 0: there are no more).
  auto take = [&](int i, Handed *it) {
    if (!wait_there.warp(&i_full[i % kQueue], static_cast<uint32_t>(i / kQueue) & 1u)) return false;
    *it = items[i % kQueue];
    __syncwarp();
    if (lane == 0) mbar_arrive(&i_empty[i % kQueue]);
    return it->t1 > 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    const auto &wait = wait_there;
    if (warp == 8 || warp == 11) {
      // ======================= loads: items, Q and K (warp 8), V (warp 11) =======================
      const bool is_v = warp == 11;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const void *tmap = is_v ? &tmap_v : &tmap_k;
      const uint32_t base = smem_u32(smem + (is_v ? L::kV : L::kK)) + lane * (kBlockTokens * 128);
      int x = 0;                      // tiles so far
      int used[2] = {0, 0};           // items of each slot so far
      int single = 0;                 // the slot of the next item that takes one
      TreeItem first = {}, last = {};             // the cut items, and where they end
      uint32_t first_end = 0, last_end = 0;
      bool ok = true;
      if (!is_v && p.B <= kWarpRows) walk = tree_begin_warp<kTile, kBoundary>(p, cta);
      for (int i = 0; ok; ++i) {
        Handed it;
        if (is_v) {
          if (!take(i, &it)) break;
        } else {
          TreeItem w;
          const bool some = walk.next(p, &w);
          if (some) {
            if (!w.whole()) {   // (at most two of them)
              (w.t0 == 0 ? last : first) = w;
              (w.t0 == 0 ? last_end : first_end) = walk.at;
            }
            const bool two = w.nodes * p.G > kTile;
            it = Handed{w.q0, w.nodes, w.g, w.b, w.base, w.n, w.tokens, w.n0, w.t0, w.t1,
                        two ? 3 : 1 << single, w.whole() ? -1 : w.slot(cta),
                        w.base + (p.mask ? 0 : w.n0), {}};
            if (!two) single ^= 1;
          } else {
            it = Handed{};
          }
          ok = wait.warp(&i_empty[i % kQueue], (static_cast<uint32_t>(i / kQueue) & 1u) ^ 1u);
          if (!ok) break;
          if (lane == 0) {
            items[i % kQueue] = it;
            mbar_arrive(&i_full[i % kQueue]);
          }
          __syncwarp();
          if (!some) break;
        }
        const int32_t *table = p.tables + static_cast<size_t>(it.b) * p.bt_stride;
        const int tiles = it.t1 - it.t0;
        auto page_id = [&](int t) {   // block of page `lane` of tile t (-1: no such page)
          const int tok = (it.t0 + t) * kTile + lane * kBlockTokens;
          return lane < kPages && tok < it.tokens ? table[tok >> 4] : -1;
        };
        int next = page_id(0);
        for (int t = 0; t < tiles; ++t, ++x) {
          const int blk = next;
          next = t + 1 < tiles ? page_id(t + 1) : -1;
          const int st = x % NS;
          const bool good = in_pool(p, blk);
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, good))) *
                                 (kBlockTokens * D * 2);
          const int y = (blk * p.Hkv + it.g) * kBlockTokens;
          ok = wait.warp(&empty[st], (static_cast<uint32_t>(x / NS) & 1u) ^ 1u);
          if (!ok) break;
          if (!is_v) {
            const uint32_t bad =
                __ballot_sync(0xffffffffu, !good && lane < kPages &&
                                               (it.t0 + t) * kTile + lane * kBlockTokens < it.tokens);
            if (lane == 0) {
              bad_s[x % kBadRing] = static_cast<uint8_t>(bad);
              if (bad) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
            }
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[st], bytes);
            __threadfence_block();
            misc[is_v ? kStartedV : kStartedK] = x + 1;
          }
          __syncwarp();
          if (good) {
#pragma unroll
            for (int s = 0; s < L::kSlabs; ++s)
              tma_load_2d(base + st * L::kMat + s * L::kSlab, tmap, s * 64, y, &full[st]);
          }
          __syncwarp();
          if (is_v || t > 0) continue;
          // the queries of the item's slots, once the slots' last item is done with them
          for (int m = 0; m < 2; ++m) {
            if (!(it.slots >> m & 1)) continue;
            ok = ok && wait.warp(&q_empty[m], (static_cast<uint32_t>(used[m]) & 1u) ^ 1u);
            if (!ok) break;
            ++used[m];
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full[m], L::kMat);
#pragma unroll
              for (int s = 0; s < L::kSlabs; ++s)
                tma_load_3d(smem_u32(smem + L::kQ) + m * L::kMat + s * L::kSlab, &tmap_q, s * 64,
                            it.g * p.G, it.q0 + (it.slots == 3 ? m * (kTile / p.G) : 0), &q_full[m]);
            }
            __syncwarp();
          }
          if (!ok) {
            ++x;
            break;
          }
        }
      }
      if (lane == 0 && !is_v) {
        p.cuts[2 * cta] = p.cuts[2 * cta + 1] = TreeCut{};
        if (first_end) tree_cut(p, first, cta, first_end, walk.all, walk.ctas);
        if (last_end) tree_cut(p, last, cta, last_end, walk.all, walk.ctas);
      }
      // every copy has landed before the CTA ends (after a normal run they have)
      for (int n = max(0, x - NS); n < x; ++n)
        mbar_wait_bounded(&full[n % NS], static_cast<uint32_t>(n / NS) & 1u, kDrainCycles);
      for (int m = 0; m < 2; ++m)
        if (used[m]) mbar_wait_bounded(&q_full[m], static_cast<uint32_t>(used[m] - 1) & 1u, kDrainCycles);
    } else {
      // ======================= products of slot m =======================
      const int m = warp - 9;
      constexpr uint32_t kIdescO = inst_desc(D, true);
      // a negative scale is taken into Q (bit 13: A negated), so that the largest score
      // stays the largest
      const uint32_t idesc_s = inst_desc(kTile, false) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
      const uint32_t q_addr = smem_u32(smem + L::kQ) + m * L::kMat, k_addr = smem_u32(smem + L::kK),
                     v_addr = smem_u32(smem + L::kV);
      int x = 0, used = 0;
      uint32_t p_ph = 0, turn_ph = 0;
      bool ok = true;
      for (int i = 0;; ++i) {
        Handed it;
        if (!take(i, &it)) break;
        const int first = uniform(it.t0), tiles = uniform(it.t1) - first, tokens = uniform(it.tokens);
        const int slots = uniform(it.slots), special = uniform(it.special);
        if (!(slots >> m & 1)) {   // the other slot's
          x += tiles;
          continue;
        }
        const bool two = slots == 3;
        // With two slots at work on the same tiles their products alternate in whole batches:
        // interleaved one by one, both would finish late and then share the exponential
        // unit as well.
        auto my_turn = [&]() {
          if (!two) return true;
          const bool r = wait.warp(&turn[m], turn_ph ^ (m == 0 ? 1u : 0u));
          turn_ph ^= 1u;
          return r;
        };
        // (one lane; a tile that one slot alone uses is handed back by it for both)
        auto next_turn = [&]() {
          if (two) mbar_arrive(&turn[m ^ 1]);
        };
        auto wait_tile = [&](uint64_t *full, int started, int t) {
          const bool r = t >= NS || __all_sync(0xffffffffu, misc[started] > x + t) ||
                         __all_sync(0xffffffffu, wait_started<POLL>(wait_here, misc + started, x + t));
          return r && wait.warp(&full[(x + t) % NS], static_cast<uint32_t>((x + t) / NS) & 1u);
        };
        auto tile_there = [&](uint64_t *full, int started, int t) {
          return __all_sync(0xffffffffu, (t >= NS || misc[started] > x + t) &&
                                             mbar_test_wait(&full[(x + t) % NS],
                                                            static_cast<uint32_t>((x + t) / NS) & 1u));
        };
        auto release = [&](uint64_t *empty) {
          mma_commit(empty);
          if (!two) mma_commit(empty);
        };
        ok = wait.warp(&q_full[m], static_cast<uint32_t>(used) & 1u);
        if (!ok) break;
        ++used;
        for (int t = -1; t < tiles; ++t) {   // P V of tile t, then the scores of tile t + 1
          if (t >= 0) {
            const int st = (x + t) % NS, tok0 = (first + t) * kTile, valid = min(kTile, tokens - tok0);
            ok = wait_tile(v_full, kStartedV, t);
            if (!ok) break;
            // values of tokens that do not count may be anything: their weights are zero,
            // and so must they be.  (Of a tile that both slots use slot 0's issuer sees to
            // it: its product comes first, and its turn, handed over behind the fence,
            // orders what it wrote ahead of slot 1's.)
            unsigned char *vt = smem + L::kV + st * L::kMat;
            bool changed = false;
            const uint32_t bad = uniform(static_cast<uint32_t>(bad_s[(x + t) % kBadRing]));
            const bool mine = !two || m == 0;
            if (mine && (valid % kBlockTokens || bad)) {
              zero_values<D>(vt, valid, bad, lane);
              changed = true;
            }
            const int look = max(0, special - tok0);
            if (mine && look < valid) {
              uint32_t odd = 0;
#pragma unroll 1
              for (int s = 0; s < L::kSlabs; ++s)
#pragma unroll 4
                for (int c = look * 8 + lane; c < valid * 8; c += 32) {
                  const uint4 v = *reinterpret_cast<const uint4 *>(vt + s * L::kSlab + c * 16);
                  odd |= odd_word(v.x) | odd_word(v.y) | odd_word(v.z) | odd_word(v.w);
                }
              if (__any_sync(0xffffffffu, odd != 0)) {
                if (lane == 0) misc[2 + i % kOddRing] = i + 1;
                clean_values<D>(vt, look, valid, lane);
                changed = true;
              }
            }
            if (changed) {
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          // (looked for here, where there is time, the next tile of K does not hold up the
          // products: S follows P V at once)
          const bool k_there = t + 1 == tiles || tile_there(k_full, kStartedK, t + 1);
          ok = (t < 0 || wait.warp(&p_half[m], p_ph)) && my_turn();
          if (!ok) break;
          const int vst = (x + t + NS) % NS, valid = min(kTile, tokens - (first + t) * kTile);
          auto weighted = [&](int from, int to) {   // O += P V, a page at a time
#pragma unroll
            for (int ks = from; ks < to; ++ks)
              if (ks * kBlockTokens < valid)
                mma_ts(tO(m), tS(m) + ks * 8,
                       smem_desc(v_addr + vst * L::kMat + ks * (kBlockTokens * 128), L::kSlab, 1024),
                       kIdescO, t > 0 || ks > 0);
          };
          if (t >= 0) {
            tc_fence_after();
            if (elect_one()) weighted(0, 2 * kHalf);
            __syncwarp();
          }
          if (t >= 0) {
            ok = wait.warp(&p_ready[m], p_ph);
            if (!ok) break;
            p_ph ^= 1u;
          }
          tc_fence_after();
          auto rest = [&]() {
            if (t < 0) return;
            weighted(2 * kHalf, kPages);
            release(&v_empty[vst]);
            if (t + 1 == tiles) mma_commit(&o_full[m]);
          };
          if (!k_there) {
            if (elect_one()) rest();
            __syncwarp();
            ok = wait_tile(k_full, kStartedK, t + 1);
            if (!ok) break;
            tc_fence_after();
          }
          const int st = (x + t + 1) % NS;
          if (elect_one()) {
            if (k_there) rest();
            if (t + 1 < tiles) {   // S = Q K^T
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks / 4) * L::kSlab + (ks % 4) * 32;
                mma_ss(tS(m), smem_desc(q_addr + off, 16, 1024),
                       smem_desc(k_addr + st * L::kMat + off, 16, 1024), idesc_s, ks > 0);
              }
              mma_commit(&s_full[m]);
              release(&k_empty[st]);
              if (t + 2 == tiles) mma_commit(&q_empty[m]);
            }
            next_turn();
          }
          __syncwarp();
        }
        if (!ok) break;
        x += tiles;
      }
      // every product is done before tensor memory is given back (the lane that issued
      // them commits)
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, kDrainCycles);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const auto &wait = wait_here;
    // ======================= softmax =======================
    const int m = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // this warp's 32 lanes
    const uint32_t sS = tS(m) + lanes, sO = tO(m) + lanes;
    const float c = fmaxf(fabsf(p.scale_log2), 1e-37f);
    const int lg = p.lg_g;
    int x = 0;
    uint32_t s_ph = 0, o_ph = 0;
    auto arrive = [&](uint64_t *bar) {   // for the warp, after all of its lanes
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    for (int i = 0;; ++i) {
      // (an item stays in the queue until its results are out, and is read there again: what
      // it says would take 16 of the registers that hold the scores)
      const Handed &it = items[i % kQueue];
      if (!wait.warp(&i_full[i % kQueue], static_cast<uint32_t>(i / kQueue) & 1u)) break;
      const int tiles = it.t1 - it.t0;
      if (tiles <= 0) break;
      if (!(it.slots >> m & 1)) {   // the other slot's
        x += tiles;
        arrive(&i_empty[i % kQueue]);
        continue;
      }
      const int total = it.nodes << lg;
      const int row0 = (it.slots == 3 ? m * kTile : 0) + (warp & 3) * 32;   // this warp's first row
      const bool active = row0 < total;
      const int node = min((row0 + lane) >> lg, it.nodes - 1);
      const uint32_t *words =
          p.mask ? p.mask + static_cast<size_t>(it.q0 + node) * p.mask_words : nullptr;
      float mx = -INFINITY, l = 0.f;
      for (int t = 0; t < tiles; ++t, ++x) {
        const int tok0 = (it.t0 + t) * kTile;
        bool masked = tok0 + kTile > it.special;
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (masked && active) {   // (ahead of the scores)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            vis[q] = tree_sees(words, p.mask_words, it.n0 + node, it.base, it.tokens, tok0 + 32 * q);
        }
        ok = wait.warp(&s_full[m], s_ph);
        if (!ok) break;
        s_ph ^= 1u;
        tc_fence_after();
        const uint32_t bad = bad_s[x % kBadRing];
        if (bad) {
          masked = true;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            vis[q] &= (bad >> 2 * q & 1 ? 0u : 0xffffu) | (bad >> (2 * q + 1) & 1 ? 0u : 0xffff0000u);
        }
        if (active) {
          float s[kTile], t4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) tm_ld32_max(sS + 32 * q, s + 32 * q, &t4[q]);
          tm_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) pin32(s + 32 * q);
          asm volatile("" : "+f"(t4[0]), "+f"(t4[1]), "+f"(t4[2]), "+f"(t4[3]));
          if (masked) {
            t4[0] = t4[1] = t4[2] = t4[3] = -INFINITY;
#pragma unroll
            for (int e = 0; e < kTile; e += 2) {
              if (!(vis[e / 32] >> (e % 32) & 1u)) s[e] = -INFINITY;
              if (!(vis[e / 32] >> (e % 32 + 1) & 1u)) s[e + 1] = -INFINITY;
              t4[(e >> 1) & 3] = max3(t4[(e >> 1) & 3], s[e], s[e + 1]);
            }
          }
          const float top = fmaxf(mx, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c);
          if (__any_sync(0xffffffffu, top > mx + kLazy)) {
            const float al = top == -INFINITY ? 1.f : ex2(mx - top);   // 0 before the first score
            mx = top;
            l *= al;
            if (t > 0) {   // the slot's last P V is done: its scores came after it
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float o[32];
                tm_ld32(sO + 32 * q, o);
                tm_wait_ld();
                pin32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= al;
                tm_st32(sO + 32 * q, o);
              }
            }
          }
          const float mu = mx == -INFINITY ? 0.f : mx;
          const uint64_t c2 = pair(c, c), mu2 = pair(-mu, -mu);
          uint64_t l2[2] = {0, 0};   // (two zeros)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y =
                  unpair(fma2(pair(s[32 * q + 2 * e], s[32 * q + 2 * e + 1]), c2, mu2));
              const float a = ex2(y.x), b = ex2(y.y);
              l2[e & 1] = add2(l2[e & 1], pair(a, b));
              w[e] = pack_bf16(a, b);
            }
            tm_st16(sS + 16 * q, w);
            if (q == kHalf - 1) {   // the product may start on these
              tm_wait_st();
              tc_fence_before();
              arrive(&p_half[m]);
            }
          }
          const float2 ls = unpair(add2(l2[0], l2[1]));
          l += ls.x + ls.y;
          tm_wait_st();
        } else {
          arrive(&p_half[m]);
        }
        tc_fence_before();
        arrive(&p_ready[m]);
      }
      if (!ok) break;
      ok = wait.warp(&o_full[m], o_ph);
      if (!ok) break;
      o_ph ^= 1u;
      tc_fence_after();
      if (!active) {
        arrive(&i_empty[i % kQueue]);
        continue;
      }
      // ---- results: a lane writes its row, whole 32-byte sectors at a time ----
      const bool whole = it.part < 0, on = row0 + lane < total;
      auto out_at = [&](int row) {   // of the outputs [T, Hq]
        return static_cast<size_t>(it.q0 + (row >> lg)) * p.Hq + it.g * p.G + (row & (p.G - 1));
      };
      const size_t part0 = static_cast<size_t>(max(it.part, 0)) * p.tile;
      float inv = l > 0.f ? 1.f / l : 0.f;
      if (on) {
        if (whole) {
          const bool any = l > 0.f || tree_sees_any(p, it.q0 + node, it.base, it.n);
          inv = tree_inverse(l, any);
          if (p.lse_out) p.lse_out[out_at(row0 + lane)] = tree_lse(mx, l, any);
        } else {
          p.part_lse[part0 + row0 + lane] = part_lse(mx, l);
        }
      }
      unsigned char *to =
          whole ? static_cast<unsigned char *>(p.out) + out_at(min(row0 + lane, total - 1)) * (D * 2)
                : reinterpret_cast<unsigned char *>(p.part_o + (part0 + row0 + lane) * D);
      const bool sectors = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        __syncwarp();
        tm_ld32(sO + 32 * q, o);
        tm_wait_ld();
        pin32(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (!on) continue;   // (the warp meets again ahead of the next load)
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) store8(reinterpret_cast<float *>(to) + 32 * q + e, o + e);
          continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
        if (sectors) {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            store8(reinterpret_cast<float *>(to + 64 * q) + e, reinterpret_cast<const float *>(w) + e);
        } else {   // (outputs need not be aligned to more than 16 bytes)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4 *>(to + 64 * q + 4 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
      }
      __syncwarp();
      if (misc[2 + i % kOddRing] == i + 1 && on)
        add_odd_values<D>(p, it, node, to, !whole);
      arrive(&i_empty[i % kQueue]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (misc[0]) tree_all_nan<__nv_bfloat16, D, kTile, kBoundary, kThreads>(p);
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int D, bool POLL>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                   cudaStream_t s) {
  auto kern = tree_tc_kernel<D, POLL>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_waiting(kern, p.C, kThreads, Lay<D>::kBytes, s, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_tree_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                             const TreeParams &p, int D, cudaStream_t s) {
  if (p.wait_limit <= kPollLimit)
    return D == 64 ? launch<64, true>(tq, tk, tv, p, s) : launch<128, true>(tq, tk, tv, p, s);
  return D == 64 ? launch<64, false>(tq, tk, tv, p, s) : launch<128, false>(tq, tk, tv, p, s);
}

}  // namespace pkv
