// Attention of drafted tokens on the 5th-generation tensor cores (bf16): up to 256 query
// rows (nodes x group heads of one batch row and KV head) against 128 tokens a step.
//
// Mathematics.  S = Q K^T and O = P V with P = 2^(S c - m), two 128 x 128 x d products per
// 128 rows and 128 tokens, online softmax between them; tokens that a node does not see
// have P = 0.  The cached tokens are read once for all nodes of the row and all heads of
// the group.
//
// Roles (one CTA per SM, its share of the positions of tree.h):
//  * warps 0-3 and 4-7: a softmax warpgroup per slot, an accumulator pair (S, O) in tensor
//    memory; thread r owns query row r, weights go back as bf16 over their scores.
//  * warps 8 and 11: TMA producers of K and of V, 16-token pages into 128-byte-swizzled slabs,
//    K-major for the first product, the same bytes MN-major for the second.  (With one warp
//    for both, a K tile waited for the V tile ahead of it, which waits for a product: a
//    load's latency a tile, 3.7 TB/s.)
//  * warps 9 and 10: issue the products of one slot each.
// Above 128 query rows the slots are two row tiles that share every K and V tile; up to 128
// they take turns in the tokens and are merged at the end.  The largest score is followed
// only when it grows by more than 2^8 (kLazy): weights up to 2^8 are exact enough in bf16.
//
// Nothing holds the producers and issuers back between items: the queries come by TMA once
// the last scores of the item before are done, and the next item's first scores are
// computed while the softmax warps still write out.
//
// Masks.  Only steps that reach past the tokens every row sees (the cached ones, and in a
// chain the nodes ahead of the item's) look at mask bits, 32 at a time.  What a node does not
// see may be anything, and 0 * NaN is NaN: so the issuing warp looks over the values of such
// tokens while the softmax is at work, and where one is not finite the element is zeroed in
// shared memory for the product and added at the end to the rows that see it (any positive
// weight leaves NaN and infinity what they are).
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
constexpr int kBoundary = 2, kMin = 1;

template <int D>
struct Lay {
  static constexpr int kSlabs = D / 64;                   // 128-byte column slabs
  static constexpr int kSlab = kTile * 128;               // bytes of a slab of a tile
  static constexpr int kMat = kSlabs * kSlab;             // bytes of a tile of Q, K or V
  static constexpr int NS = D == 128 ? 2 : 4;             // K and V stages
  static constexpr int kQ = 0;                            // [2] tiles
  static constexpr int kK = 2 * kMat;                     // [NS]
  static constexpr int kV = kK + NS * kMat;               // [NS]
  static constexpr int kScratch = kV + NS * kMat;         // half of the second slot's O
  static constexpr int kBars = kScratch + kTile * D / 2 * 4;
  static constexpr int kNumBars = 4 * NS + 14;
  static constexpr int kSums = kBars + kNumBars * 8;      // m, l of the second slot
  static constexpr int kBad = kSums + 2 * kTile * 4;      // [kBadRing] pages outside the pool
  static constexpr int kBadRing = 16;
  static constexpr int kMisc = kBad + kBadRing;
  static constexpr int kBytes = kMisc + 32 + 1024;        // + alignment slack
};

using Walk = TreeWalk<kTile, kBoundary>;

// First token from which on rows of an item may differ in what they see.
__device__ __forceinline__ int first_special(const TreeParams &p, const TreeItem &it) {
  return it.base + (p.mask ? 0 : it.n0);
}
__device__ __forceinline__ bool odd_bf16(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }
// Bits 15 and 31: a half's exponent is all ones (its sum with the lowest exponent bit
// carries into the sign's place).
__device__ __forceinline__ uint32_t odd_word(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t clean_word(uint32_t w) {
  return (odd_bf16(w) ? 0u : w & 0xffffu) | (odd_bf16(w >> 16) ? 0u : w & 0xffff0000u);
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
  uint64_t *s_full = bars + 4 * NS, *p_ready = s_full + 2, *o_full = s_full + 4;   // [2] each
  uint64_t *q_full = s_full + 6, *both = s_full + 7, *drain = s_full + 8;
  uint64_t *turn = s_full + 9, *p_half = s_full + 11;   // [2] each
  uint64_t *q_empty = s_full + 13;
  volatile uint8_t *bad_s = reinterpret_cast<volatile uint8_t *>(smem + L::kBad);
  float *sums_s = reinterpret_cast<float *>(smem + L::kSums);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  // misc: a wait gave up, tmem, the last item of odd and of even number with values that are
  // not finite [2] (its number + 1)

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);   // one arrival per slot
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&p_ready[m], kTile / 32);   // one arrival per warp
      mbar_init(&p_half[m], kTile / 32);
      mbar_init(&o_full[m], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);   // one arrival per slot
    mbar_init(both, kSoftmax / 32);
    mbar_init(drain, 2);
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);
    misc[0] = 0;
    misc[2] = misc[3] = 0;
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
  Walk walk = tree_begin<kTile, kBoundary, kMin, kThreads>(p, cta);   // (synchronises the CTA)
  TreeItem it;
  tc_fence_after();
  const uint32_t tmem = uniform(static_cast<uint32_t>(misc[1]));
  // (by arithmetic: arrays indexed by the slot would live in local memory)
  auto tS = [tmem](int m) { return tmem + 128u * m; };
  auto tO = [tmem](int m) { return tmem + 256u + 128u * m; };
  const Waiter<POLL> wait{misc, p.err, p.wait_limit};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8 || warp == 11) {
      // ======================= producers: K (warp 8), V (warp 11) =======================
      const bool is_v = warp == 11;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const void *tmap = is_v ? &tmap_v : &tmap_k;
      const uint32_t base = smem_u32(smem + (is_v ? L::kV : L::kK)) + lane * (kBlockTokens * 128);
      int x = 0;       // tiles of the items before
      int armed = 0;   // tiles whose copies were started
      int n_items = 0, armed_q = 0;
      bool ok = true;
      TreeCut cut = {};
      while (ok && walk.next(&it)) {
        if (it.t0 == 0 && it.t1 < it.steps)
          cut = TreeCut{walk.more(), it.q0, it.nodes * p.G, it.g, it.base, it.n};
        const int32_t *table = p.tables + static_cast<size_t>(it.b) * p.bt_stride;
        const int tiles = it.t1 - it.t0;
        auto page_id = [&](int t) {   // block of page `lane` of tile t (-1: no such page)
          const int tok = (it.t0 + t) * kTile + lane * kBlockTokens;
          return lane < kPages && tok < it.tokens ? table[tok >> 4] : -1;
        };
        int next = page_id(0);
        for (int t = 0; t < tiles; ++t) {
          const int blk = next;
          next = t + 1 < tiles ? page_id(t + 1) : -1;
          const int st = (x + t) % NS;
          const bool good = blk >= 0 && blk < p.num_blocks;
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, good))) *
                                 (kBlockTokens * D * 2);
          const int y = (blk * p.Hkv + it.g) * kBlockTokens;
          ok = wait.warp(&empty[st], (static_cast<uint32_t>((x + t) / NS) & 1u) ^ 1u);
          if (!ok) break;
          if (!is_v) {
            const uint32_t bad =
                __ballot_sync(0xffffffffu, !good && lane < kPages &&
                                               (it.t0 + t) * kTile + lane * kBlockTokens < it.tokens);
            if (lane == 0) {
              bad_s[(x + t) % L::kBadRing] = static_cast<uint8_t>(bad);
              if (bad) set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
            }
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
          __syncwarp();
          if (good) {
#pragma unroll
            for (int s = 0; s < L::kSlabs; ++s)
              tma_load_2d(base + st * L::kMat + s * L::kSlab, tmap, s * 64, y, &full[st]);
          }
          __syncwarp();
          armed = x + t + 1;
          if (is_v && t == 0) {   // the queries, once the products of the item before are done with them
            ok = wait.warp(q_empty, (static_cast<uint32_t>(n_items) & 1u) ^ 1u);
            if (!ok) break;
            const int q_tiles = it.nodes * p.G > kTile ? 2 : 1;
            if (elect_one()) {
              mbar_arrive_expect_tx(q_full, q_tiles * L::kMat);
              for (int e = 0; e < q_tiles; ++e)
#pragma unroll
                for (int s = 0; s < L::kSlabs; ++s)
                  tma_load_3d(smem_u32(smem + L::kQ) + e * L::kMat + s * L::kSlab, &tmap_q, s * 64,
                              it.g * p.G, it.q0 + e * (kTile / p.G), q_full);
            }
            __syncwarp();
            armed_q = ++n_items;
          }
        }
        x += tiles;
      }
      if (lane == 0 && !is_v) p.cuts[cta] = cut;
      // every copy has landed before the CTA ends (after a normal run they have)
      for (int n = max(0, armed - NS); n < armed; ++n)
        mbar_wait_bounded(&full[n % NS], static_cast<uint32_t>(n / NS) & 1u, kDrainCycles);
      if (armed_q) mbar_wait_bounded(q_full, static_cast<uint32_t>(armed_q - 1) & 1u, kDrainCycles);
    } else {
      // ======================= products of slot m =======================
      const int m = warp - 9;
      constexpr uint32_t kIdescO = inst_desc(D, true);
      // a negative scale is taken into Q (bit 13: A negated), so that the largest score
      // stays the largest
      const uint32_t idesc_s = inst_desc(kTile, false) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
      const uint32_t q_addr = smem_u32(smem + L::kQ), k_addr = smem_u32(smem + L::kK),
                     v_addr = smem_u32(smem + L::kV);
      int x = 0, n_items = 0;
      uint32_t p_ph = 0, turn_ph = 0;
      bool ok = true;
      while (ok && walk.next(&it)) {
        const int first = uniform(it.t0), tiles = uniform(it.t1) - first, tokens = uniform(it.tokens);
        const bool two = uniform(it.nodes) * p.G > kTile;   // the slots are two row tiles
        const int n = two ? tiles : (tiles + 1 - m) / 2;
        ok = wait.warp(q_full, static_cast<uint32_t>(n_items) & 1u);
        if (!ok) break;
        tc_fence_after();
        const int special = first_special(p, it);
        ++n_items;
        const int turns = two ? tiles : (tiles + 1) / 2;   // slot 0's tiles, at least this slot's
        auto tile_of = [&](int j) { return two ? j : 2 * j + m; };
        // the slots' products alternate in whole batches: interleaved one by one, both
        // slots would finish late and then share the exponential unit as well
        auto my_turn = [&]() {
          const bool r = wait.warp(&turn[m], turn_ph ^ (m == 0 ? 1u : 0u));
          turn_ph ^= 1u;
          return r;
        };
        auto next_turn = [&]() { mbar_arrive(&turn[m ^ 1]); };   // (one lane)
        auto wait_k = [&](int t) {
          return wait.warp(&k_full[(x + t) % NS], static_cast<uint32_t>((x + t) / NS) & 1u);
        };
        // a tile that one slot alone uses is handed back by it for both
        auto release = [&](uint64_t *empty) {
          mma_commit(empty);
          if (!two) mma_commit(empty);
        };
        // S = Q K^T for the slot's tile j (issued by one lane)
        auto issue_scores = [&](int j) {
          const int t = tile_of(j);
          const int st = (x + t) % NS;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks / 4) * L::kSlab + (ks % 4) * 32;
            mma_ss(tS(m), smem_desc(q_addr + (two ? m * L::kMat : 0) + off, 16, 1024),
                   smem_desc(k_addr + st * L::kMat + off, 16, 1024), idesc_s, ks > 0);
          }
          mma_commit(&s_full[m]);
          release(&k_empty[st]);
          if (j + 1 == n) mma_commit(q_empty);
        };
        ok = (n == 0 || wait_k(tile_of(0))) && my_turn();
        if (ok && elect_one()) {
          if (n > 0)
            issue_scores(0);
          else
            mbar_arrive(q_empty);
          next_turn();
        }
        __syncwarp();
        for (int j = 0; j < turns && ok; ++j) {
          if (j >= n) {   // slot 1 has a tile less: its turn goes by
            ok = my_turn();
            if (ok && elect_one()) next_turn();
            __syncwarp();
            continue;
          }
          const int t = tile_of(j), st = (x + t) % NS;
          const int tok0 = (first + t) * kTile, valid = min(kTile, tokens - tok0);
          const bool more = j + 1 < n;
          // the values first (they are there well before the weights)
          ok = wait.warp(&v_full[st], static_cast<uint32_t>((x + t) / NS) & 1u);
          if (!ok) break;
          unsigned char *vt = smem + L::kV + st * L::kMat;
          // 16-byte pieces of the tile's tokens from `first` to `last`: piece e, or where it lies
          auto piece = [&](int e, int first, int last) {
            const int s = e / ((last - first) * 8), c = e - s * ((last - first) * 8);
            return reinterpret_cast<uint4 *>(vt + s * L::kSlab + first * 128 + c * 16);
          };
          bool changed = false;
          const uint32_t bad = bad_s[(x + t) % L::kBadRing];
          if (valid % kBlockTokens || bad) {
            // values of tokens that do not count may be anything: their weights are
            // zero, and so must they be (both slots of a shared tile write the zeros)
            for (int pg = 0; pg * kBlockTokens < valid; ++pg) {
              const int end = (pg + 1) * kBlockTokens;
              const int from = bad >> pg & 1 ? end - kBlockTokens : min(end, valid);
              for (int e = lane; e < (end - from) * 8 * L::kSlabs; e += 32)
                *piece(e, from, end) = make_uint4(0u, 0u, 0u, 0u);
            }
            changed = true;
          }
          const int look = max(0, special - tok0);
          if (look < valid) {
            uint32_t odd = 0;
            for (int e = lane; e < (valid - look) * 8 * L::kSlabs; e += 32) {
              const uint4 v = *piece(e, look, valid);
              odd |= odd_word(v.x) | odd_word(v.y) | odd_word(v.z) | odd_word(v.w);
            }
            if (__any_sync(0xffffffffu, odd != 0)) {
              // (the note first: the other slot may find the tile clean already)
              if (lane == 0) misc[2 + (n_items & 1)] = n_items;
              __threadfence_block();
              __syncwarp();
              for (int e = lane; e < (valid - look) * 8 * L::kSlabs; e += 32) {
                uint4 *at = piece(e, look, valid);
                const uint4 v = *at;
                *at = make_uint4(clean_word(v.x), clean_word(v.y), clean_word(v.z), clean_word(v.w));
              }
              changed = true;
            }
          }
          if (changed) {
            fence_proxy_async_smem();
            __syncwarp();
          }
          auto weighted = [&](int from, int to) {   // O += P V, a page at a time
#pragma unroll
            for (int ks = from; ks < to; ++ks)
              if (ks * kBlockTokens < valid)
                mma_ts(tO(m), tS(m) + ks * 8,
                       smem_desc(v_addr + st * L::kMat + ks * (kBlockTokens * 128), L::kSlab, 1024),
                       kIdescO, j > 0 || ks > 0);
          };
          ok = wait.warp(&p_half[m], p_ph) && my_turn();
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) weighted(0, 2 * kHalf);
          __syncwarp();
          ok = wait.warp(&p_ready[m], p_ph);
          if (!ok) break;
          p_ph ^= 1u;
          tc_fence_after();
          if (elect_one()) {
            weighted(2 * kHalf, kPages);
            release(&v_empty[st]);
            if (!more) mma_commit(&o_full[m]);
          }
          __syncwarp();
          ok = !more || wait_k(tile_of(j + 1));
          if (!ok) break;
          if (elect_one()) {
            if (more) issue_scores(j + 1);
            next_turn();
          }
          __syncwarp();
        }
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
    // ======================= softmax =======================
    const int m = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // this warp's 32 lanes
    const uint32_t sS = tS(m) + lanes, sO = tO(m) + lanes;
    const float c = fmaxf(fabsf(p.scale_log2), 1e-37f);
    const int lg = __ffs(p.G) - 1;
    int x = 0, n_items = 0;
    uint32_t s_ph = 0, o_ph = 0, b_ph = 0;
    bool ok = true;
    auto arrive = [&](uint64_t *bar) {   // for the warp, after all of its lanes
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto meet = [&]() {   // both warpgroups
      arrive(both);
      ok = ok && wait.warp(both, b_ph);
      b_ph ^= 1u;
    };
    while (ok && walk.next(&it)) {
      const int total = it.nodes * p.G;
      const int tiles = it.t1 - it.t0;
      const bool two = total > kTile;
      const int n = two ? tiles : (tiles + 1 - m) / 2;
      const int32_t *table = p.tables + static_cast<size_t>(it.b) * p.bt_stride;
      const int special = first_special(p, it);
      const int end = min(it.tokens, it.t1 * kTile);   // of this CTA's tokens
      ++n_items;
      const int from = max(special, it.t0 * kTile);    // of them, first that rows may differ in
      const int mine = (two ? m * kTile : 0) + r;   // this thread's row of the item
      const bool active = (two ? m * kTile : 0) + (warp & 3) * 32 < total;
      const int node = min(mine >> lg, it.nodes - 1);
      const uint32_t *words =
          p.mask ? p.mask + static_cast<size_t>(it.q0 + node) * p.mask_words : nullptr;
      auto sees = [&](int tok) {
        return tree_sees(words, p.mask_words, it.n0 + node, it.base, it.tokens, tok);
      };
      float mx = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int t = two ? j : 2 * j + m;
        const int tok0 = (it.t0 + t) * kTile;
        bool masked = tok0 + kTile > special;
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (masked && active) {   // (ahead of the scores)
#pragma unroll
          for (int q = 0; q < 4; ++q) vis[q] = sees(tok0 + 32 * q);
        }
        ok = wait.warp(&s_full[m], s_ph);
        if (!ok) break;
        s_ph ^= 1u;
        tc_fence_after();
        const uint32_t bad = bad_s[(x + t) % L::kBadRing];
        if (bad) {
          masked = true;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            vis[q] &= (bad >> 2 * q & 1 ? 0u : 0xffffu) | (bad >> (2 * q + 1) & 1 ? 0u : 0xffff0000u);
        }
        if (active) {
          float s[kTile];
#pragma unroll
          for (int q = 0; q < 4; ++q) tm_ld32(sS + 32 * q, s + 32 * q);
          tm_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) pin32(s + 32 * q);
          if (masked) {
#pragma unroll
            for (int e = 0; e < kTile; ++e)
              if (!(vis[e / 32] >> (e % 32) & 1u)) s[e] = -INFINITY;
          }
          float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int e = 4; e + 1 < kTile; e += 2)
            t4[(e >> 1) & 3] = max3(t4[(e >> 1) & 3], s[e], s[e + 1]);
          const float top = fmaxf(mx, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c);
          if (__any_sync(0xffffffffu, top > mx + kLazy)) {
            const float al = top == -INFINITY ? 1.f : ex2(mx - top);   // 0 before the first score
            mx = top;
            l *= al;
            if (j > 0) {   // the slot's last P V is done: its scores came after it
#pragma unroll
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
              const float2 x =
                  unpair(fma2(pair(s[32 * q + 2 * e], s[32 * q + 2 * e + 1]), c2, mu2));
              const float a = ex2(x.x), b = ex2(x.y);
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
      x += tiles;
      if (ok && n > 0) {
        ok = wait.warp(&o_full[m], o_ph);
        o_ph ^= 1u;
        tc_fence_after();
      }
      // ---- results: the second slot of a single row tile is merged into the first ----
      float w0 = 1.f, w1 = 0.f;
      const bool merge = !two && tiles > 1;
      if (merge && m == 1 && ok) {
        sums_s[r] = mx;
        sums_s[kTile + r] = l;
      }
      float *scratch = reinterpret_cast<float *>(smem + L::kScratch);   // [D/2][128]
      const bool whole = it.whole();
      const bool on = mine < total;
      const size_t out_at = static_cast<size_t>(it.q0 + node) * p.Hq + it.g * p.G + (mine & (p.G - 1));
      const size_t part_at = static_cast<size_t>(it.slot(cta)) * p.tile + mine;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (merge) {
          if (m == 1 && active && ok) {
#pragma unroll
            for (int q = 0; q < D / 64; ++q) {
              float o[32];
              tm_ld32(sO + h * (D / 2) + 32 * q, o);
              tm_wait_ld();
              pin32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) scratch[(32 * q + e) * kTile + r] = o[e];
            }
          }
          meet();
        }
        if ((two || m == 0) && active && ok) {
          // (behind the merge's meeting: the other slot's products are done, too)
          const bool odd = misc[2 + (n_items & 1)] == n_items;
          if (h == 0) {
            float den = l;
            if (merge) {
              const float m1 = sums_s[r], l1 = sums_s[kTile + r];
              const float M = fmaxf(mx, m1);
              w0 = M == -INFINITY ? 0.f : ex2(mx - M);
              w1 = M == -INFINITY ? 0.f : ex2(m1 - M);
              den = l * w0 + l1 * w1;
              mx = M;
            }
            float inv = den > 0.f ? 1.f / den : 0.f;
            if (on && whole) {
              const bool any = den > 0.f || tree_sees_any(p, it.q0 + node, it.base, it.n);
              inv = tree_inverse(den, any);
              if (p.lse_out) p.lse_out[out_at] = tree_lse(mx, den, any);
            } else if (on) {
              p.part_lse[part_at] = part_lse(mx, den);
            }
            w0 *= inv;
            w1 *= inv;
          }
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            float o[32];
            const int col = h * (D / 2) + 32 * q;
            __syncwarp();
            tm_ld32(sO + col, o);
            tm_wait_ld();
            pin32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              o[e] *= w0;
              if (merge) o[e] = fmaf(w1, scratch[(32 * q + e) * kTile + r], o[e]);
            }
            if (on && odd) {   // what was left out of the products
#pragma unroll 1
              for (int tok = from; tok < end; ++tok) {
                if (!(sees(tok) & 1u)) continue;
                const int blk = table[tok / kBlockTokens];
                if (blk < 0 || blk >= p.num_blocks) continue;
                const uint4 *v = reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(p.v_cache) +
                    ((static_cast<size_t>(blk) * p.Hkv + it.g) * kBlockTokens + tok % kBlockTokens) * D +
                    col);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint4 w = v[e];
                  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                  for (int f = 0; f < 4; ++f) {
                    if (odd_bf16(u[f])) o[8 * e + 2 * f] += bf16_lo(u[f]);
                    if (odd_bf16(u[f] >> 16)) o[8 * e + 2 * f + 1] += bf16_hi(u[f]);
                  }
                }
              }
            }
            if (on && whole) {
              uint4 *dst =
                  reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + out_at * D + col);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dst[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                    pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                    pack_bf16(o[8 * e + 6], o[8 * e + 7]));
            } else if (on) {
              float *dst = p.part_o + part_at * D + col;
#pragma unroll
              for (int e = 0; e < 32; e += 8) store8(dst + e, o + e);
            }
          }
        }
        if (merge) meet();
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (misc[0]) {   // a wait gave up: no output of this CTA's counts
    Walk again = tree_begin<kTile, kBoundary, kMin, kThreads>(p, cta);
    const float nan = __int_as_float(0x7fffffff);
    while (again.next(&it)) {
      for (int e = tid; e < it.nodes * p.G; e += kThreads) {
        if (!it.whole()) {
          p.part_lse[static_cast<size_t>(it.slot(cta)) * p.tile + e] = INFINITY;   // (the join makes NaN of it)
          continue;
        }
        const size_t at = static_cast<size_t>(it.q0 + e / p.G) * p.Hq + it.g * p.G + e % p.G;
        if (p.lse_out) p.lse_out[at] = nan;
        for (int col = 0; col < D; ++col)
          static_cast<__nv_bfloat16 *>(p.out)[at * D + col] = __float2bfloat16_rn(nan);
      }
    }
  }
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
