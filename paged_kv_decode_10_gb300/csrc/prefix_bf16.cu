// Prefix partials on the 5th-generation tensor cores (bf16): up to 256 query rows
// against a range of a prefix's tokens, 128 tokens at a time.
//
// Mathematics.  For one KV head the queries of all rows that share the prefix are
// the rows of one matrix Q (batch rows x group heads), so the scores are
// S = Q K^T and the partial output O = P V with P = 2^(S c - m): two 128 x 128 x d
// products per 128 query rows and 128 tokens, online softmax between them.
//
// Roles (one CTA per SM, work items from the plan):
//  * warps 0-3 and 4-7: one softmax warpgroup per slot.  A slot is an accumulator
//    pair (S, O) in tensor memory; thread r of a warpgroup owns query row r, so
//    row maxima and sums need no shuffles.  Scores are read from tensor memory,
//    weights go back as bf16 over the scores they came from.
//  * warp 8: TMA producer.  16-token pages of K and V land in 128-byte-swizzled
//    slabs, eight pages to a tile; for K a slab is the K-major operand, for V the
//    same bytes are the MN-major operand, so neither is transposed.
//  * warps 9 and 10: issue the products of one slot each (warp 11 only completes the
//    warpgroup).  While one slot is in its softmax the tensor cores work for the other.
//    An issuer's waits and bookkeeping take about as long as its products, which
//    is why there are two: one warp for both slots left the tensor cores idle for
//    1400 of 3700 clocks a step.
// Above 128 query rows the slots are the two row tiles and share every K and V
// tile; up to 128 rows they take turns in the tokens and are merged at the end.
//
// The largest score seen is only followed when it grows by more than 2^8
// (kLazy): until then weights up to 2^8 are exact enough in bf16 and the
// accumulator needs no rescaling; l and O use the same m, so the result is the
// same quotient.  Sums and accumulators are float32, weights are rounded to
// bf16 once, for the product; the normaliser sums them before that.
//
// Measured: 128 rows x 8 heads of 128 against 65531 tokens of 4 KV heads, 137 GFLOP, in
// 107 us (1.28 PFLOP/s, tensor pipe active 58 % of the time).  What bounds it is the
// softmax of a step (scores in, 128 exponentials a row, weights out) between its two
// products: a step of both slots takes 3140 clocks, its products 2048.
#include "prefix.h"
#include "tensor_core.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;                    // tokens of a tile, rows of a slot
constexpr int kPages = kTile / kBlockTokens;  // pages of a tile
constexpr int kSoftmax = 256, kThreads = 384;
// registers a thread: 168 at launch; the softmax warpgroups hold a row of 128
// scores and take 216, what the third warpgroup gives up (2 * 216 + 72 = 3 * 168)
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr float kLazy = 8.0f;
constexpr int kHalf = 2;                      // 32-token pieces of P after which P V starts
constexpr long long kDrainCycles = 1ll << 31;
constexpr long long kPollLimit = 4096;

template <int D>
struct Lay {
  static constexpr int kSlabs = D / 64;                   // 128-byte column slabs
  static constexpr int kSlab = kTile * 128;               // bytes of a slab of a tile
  static constexpr int kMat = kSlabs * kSlab;             // bytes of a tile of Q, K or V
  static constexpr int NS = D == 128 ? 2 : 4;             // K and V stages
  static constexpr int kQ = 0;                            // [2] tiles
  static constexpr int kK = 2 * kMat;                     // [NS]
  static constexpr int kV = kK + NS * kMat;               // [NS]
  static constexpr int kBars = kV + NS * kMat;
  static constexpr int kNumBars = 4 * NS + 13;
  static constexpr int kRows = kBars + kNumBars * 8;      // row, partial index of each query row
  static constexpr int kSums = kRows + 2 * kSoftmax * 4;  // m, l of the second slot
  static constexpr int kMisc = kSums + 2 * kTile * 4;
  static constexpr int kBytes = kMisc + 64 + 1024;        // + alignment slack
};

template <int D, bool POLL>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PrefixParams p) {
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
  int *rows_s = reinterpret_cast<int *>(smem + L::kRows);   // [256] batch row, [256] slot
  float *sums_s = reinterpret_cast<float *>(smem + L::kSums);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  // misc: a wait gave up, tmem, bad pages [2], a row does not fit, partials or kPrefixSkipped

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
    mbar_init(q_full, kSoftmax / 32);
    mbar_init(both, kSoftmax / 32);
    mbar_init(drain, 2);
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);
    misc[0] = 0;
    misc[2] = misc[3] = misc[4] = misc[5] = 0;
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
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: what starts then may read what was there before)
  // the plan's header and this CTA's items
  const int *ctas = p.plan + plan_ctas_at(p.B);
  int i0 = ctas[blockIdx.x], i1 = ctas[blockIdx.x + 1];
  const PlanHeader head = plan_header(p.plan, p.B, p.C, p.Hkv, p.G, p.plan_ints, p.slots);
  i0 = uniform(head.ok ? max(0, i0) : 0);
  i1 = uniform(head.ok ? min(head.items, i1) : 0);
  if (!head.ok && tid == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(static_cast<uint32_t>(misc[1]));
  // (by arithmetic: arrays indexed by the slot would live in local memory)
  auto tS = [tmem](int m) { return tmem + 128u * m; };
  auto tO = [tmem](int m) { return tmem + 256u + 128u * m; };
  const Waiter<POLL> wait{misc, p.err, p.wait_limit};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      // ======================= producer =======================
      int x = 0;                     // tiles of the items before
      int armed_k = 0, armed_v = 0;  // tiles whose copies were started
      int partials = 0;              // of the items, which
      bool fits = head.ok;           // fit
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        PrefixItem it;
        const int kind = prefix_item(p, i, kTileRowsBf16, &it);
        partials += it.rows;
        if (kind != kItemOk) {
          if (lane == 0) set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
          if (kind == kItemBad || __any_sync(0xffffffffu, !prefix_unread(p, it, lane, 32))) fits = false;
          continue;
        }
        const int32_t *table = p.tables + static_cast<size_t>(it.prefix) * p.pt_stride;
        const int tiles = (it.t1 - it.t0 + kTile - 1) / kTile;
        auto page_id = [&](int t) {   // block of page `lane` of tile t (-1: no such page)
          const int tok = it.t0 + t * kTile + lane * kBlockTokens;
          return lane < kPages && tok < it.t1 ? table[tok >> 4] : -1;
        };
        int next = page_id(0);
        for (int t = 0; t < tiles && ok; ++t) {
          const int blk = next;
          next = t + 1 < tiles ? page_id(t + 1) : -1;
          const int st = (x + t) % NS;
          const uint32_t ph = static_cast<uint32_t>((x + t) / NS) & 1u;
          const bool good = blk >= 0 && blk < p.num_blocks;
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, good))) *
                                 (kBlockTokens * D * 2);
          const int y = (blk * p.Hkv + it.g) * kBlockTokens;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            uint64_t *full = kv ? &v_full[st] : &k_full[st];
            ok = ok && wait.warp(kv ? &v_empty[st] : &k_empty[st], ph ^ 1u);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            if (good) {
              const uint32_t dst =
                  smem_u32(smem + (kv ? L::kV : L::kK) + st * L::kMat) + lane * (kBlockTokens * 128);
#pragma unroll
              for (int s = 0; s < L::kSlabs; ++s)
                tma_load_2d(dst + s * L::kSlab, kv ? &tmap_v : &tmap_k, s * 64, y, full);
            }
            __syncwarp();
            (kv ? armed_v : armed_k) = x + t + 1;
          }
        }
        x += tiles;
      }
      // (the account of the items is kept here: in a warp of its own, or at the head of the
      // softmax, it took 2 us of 137)
      if (lane == 0) misc[5] = fits ? partials : kPrefixSkipped;
      // every copy has landed before the CTA ends (after a normal run they have)
      for (int n = max(0, armed_k - NS); n < armed_k; ++n)
        mbar_wait_bounded(&k_full[n % NS], static_cast<uint32_t>(n / NS) & 1u, kDrainCycles);
      for (int n = max(0, armed_v - NS); n < armed_v; ++n)
        mbar_wait_bounded(&v_full[n % NS], static_cast<uint32_t>(n / NS) & 1u, kDrainCycles);
    } else if (warp <= 10) {
      // ======================= products of slot m =======================
      const int m = warp - 9;
      constexpr uint32_t kIdescS = inst_desc(kTile, false), kIdescO = inst_desc(D, true);
      const uint32_t q_addr = smem_u32(smem + L::kQ), k_addr = smem_u32(smem + L::kK),
                     v_addr = smem_u32(smem + L::kV);
      int x = 0, n_items = 0;
      uint32_t p_ph = 0, turn_ph = 0;
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        PrefixItem it;
        if (uniform(prefix_item(p, i, kTileRowsBf16, &it)) != kItemOk) continue;
        it.t0 = uniform(it.t0);
        it.t1 = uniform(it.t1);
        it.rows = uniform(it.rows);
        const int tiles = (it.t1 - it.t0 + kTile - 1) / kTile;
        const bool two = it.rows * p.G > kTile;   // the slots are two row tiles
        const int n = two ? tiles : (tiles + 1 - m) / 2;
        ok = wait.warp(q_full, static_cast<uint32_t>(n_items) & 1u);
        if (!ok) break;
        tc_fence_after();
        const bool bad_pages = uniform(misc[2 + (n_items & 1)] + 0) != 0;
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
        // S = Q K^T for tile t (issued by one lane)
        auto issue_scores = [&](int t) {
          const int st = (x + t) % NS;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks / 4) * L::kSlab + (ks % 4) * 32;
            mma_ss(tS(m), smem_desc(q_addr + (two ? m * L::kMat : 0) + off, 16, 1024),
                   smem_desc(k_addr + st * L::kMat + off, 16, 1024), kIdescS, ks > 0);
          }
          mma_commit(&s_full[m]);
          release(&k_empty[st]);
        };
        ok = (n == 0 || wait_k(tile_of(0))) && my_turn();
        if (ok && elect_one()) {
          if (n > 0) issue_scores(tile_of(0));
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
          const int valid = min(kTile, it.t1 - it.t0 - t * kTile);
          const bool more = j + 1 < n;
          // the tiles first (they are there well before the weights)
          ok = wait.warp(&v_full[st], static_cast<uint32_t>((x + t) / NS) & 1u) &&
               (!more || wait_k(tile_of(j + 1)));
          if (!ok) break;
          if (valid % kBlockTokens || bad_pages) {
            // values of tokens that do not count may be anything: their weights are
            // zero, and so must they be (both slots of a shared tile write the zeros)
            const int32_t *table = p.tables + static_cast<size_t>(it.prefix) * p.pt_stride;
            unsigned char *vt = smem + L::kV + st * L::kMat;
            for (int pg = 0; pg * kBlockTokens < valid; ++pg) {
              const int blk = table[(it.t0 + t * kTile) / kBlockTokens + pg];
              const int first =
                  blk < 0 || blk >= p.num_blocks ? 0 : min(kBlockTokens, valid - pg * kBlockTokens);
              for (int e = lane; e < (kBlockTokens - first) * 8 * L::kSlabs; e += 32) {
                const int s = e / ((kBlockTokens - first) * 8), c = e % ((kBlockTokens - first) * 8);
                *reinterpret_cast<uint4 *>(vt + s * L::kSlab + (pg * kBlockTokens + first) * 128 +
                                           c * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
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
            if (more)
              issue_scores(tile_of(j + 1));
            else
              mma_commit(&o_full[m]);
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
    // a negative scale is taken into Q, so that the largest score stays the largest
    const float c = fmaxf(fabsf(p.scale_log2), 1e-37f);
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    int n_items = 0;
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
    for (int i = i0; i < i1 && ok; ++i) {
      PrefixItem it;
      if (prefix_item(p, i, kTileRowsBf16, &it) != kItemOk) continue;
      const int total = it.rows * p.G;
      const int tiles = (it.t1 - it.t0 + kTile - 1) / kTile;
      const bool two = total > kTile;
      const int n = two ? tiles : (tiles + 1 - m) / 2;
      const int32_t *table = p.tables + static_cast<size_t>(it.prefix) * p.pt_stride;
      volatile int *bad = misc + 2 + (n_items & 1);
      if (tid == 0) misc[2 + ((n_items + 1) & 1)] = 0;   // (read last in the item before)
      ++n_items;
      {
        int row = -1, at = -1;
        if (tid < total) {
          int slot;
          row = prefix_row(p, it, tid / p.G, &slot);
          if (row < 0) {
            set_dev_err(p.err, PKV_DEVERR_BAD_PLAN);
            misc[4] = 1;
          } else {
            at = slot * p.Hq + it.g * p.G + tid % p.G;
          }
        }
        rows_s[tid] = row;
        rows_s[kSoftmax + tid] = at;
      }
      for (int j = it.t0 / kBlockTokens + tid; j < (it.t1 + kBlockTokens - 1) / kBlockTokens;
           j += kSoftmax) {
        const int blk = table[j];
        if (blk < 0 || blk >= p.num_blocks) {
          *bad = 1;
          set_dev_err(p.err, PKV_DEVERR_BAD_BLOCK);
        }
      }
      meet();
      if (!ok) break;
      constexpr int kStep = kSoftmax / (D / 8);   // rows between a thread's pieces
      const int ch = tid % (D / 8);
      for (int r0 = tid / (D / 8); r0 < (two ? 2 : 1) * kTile; r0 += 16 * kStep) {
        uint4 v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          // (rows that do not count read row 0: a branch here would make the loads
          // wait for one another)
          const int row = r0 + u * kStep, b = row < kSoftmax ? rows_s[row] : 0;
          v[u] = *reinterpret_cast<const uint4 *>(
              static_cast<const __nv_bfloat16 *>(p.q) +
              (static_cast<size_t>(max(b, 0)) * p.Hq + it.g * p.G + (row & (p.G - 1))) * D + ch * 8);
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int row = r0 + u * kStep;
          uint4 x = make_uint4(v[u].x ^ flip, v[u].y ^ flip, v[u].z ^ flip, v[u].w ^ flip);
          if (row >= kSoftmax || rows_s[row] < 0) x = make_uint4(0u, 0u, 0u, 0u);
          if (row < (two ? 2 : 1) * kTile)
            *reinterpret_cast<uint4 *>(smem + L::kQ + (row / kTile) * L::kMat +
                                       (ch / 8) * L::kSlab + (row % kTile) * 128 +
                                       (((ch & 7) ^ (row & 7)) << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();   // the reads of the item before's O
      arrive(q_full);
      const bool bad_pages = *bad != 0;
      const bool active = (two ? m * kTile : 0) + (warp & 3) * 32 < total;
      float mx = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = wait.warp(&s_full[m], s_ph);
        if (!ok) break;
        s_ph ^= 1u;
        tc_fence_after();
        if (active) {
          const int t = two ? j : 2 * j + m;
          const int valid = min(kTile, it.t1 - it.t0 - t * kTile);
          float s[kTile];
#pragma unroll
          for (int q = 0; q < 4; ++q) tm_ld32(sS + 32 * q, s + 32 * q);
          tm_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) pin32(s + 32 * q);
          if (valid < kTile || bad_pages) {
            uint32_t pages = 0xffu;
            if (bad_pages) {
              pages = 0;
              for (int pg = 0; pg * kBlockTokens < valid; ++pg) {
                const int blk = table[(it.t0 + t * kTile) / kBlockTokens + pg];
                pages |= (blk >= 0 && blk < p.num_blocks ? 1u : 0u) << pg;
              }
            }
#pragma unroll
            for (int q = 0; q < kTile; ++q)
              if (q >= valid || !(pages >> (q / kBlockTokens) & 1u)) s[q] = -INFINITY;
          }
          float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int q = 4; q + 1 < kTile; q += 2)
            t4[(q >> 1) & 3] = max3(t4[(q >> 1) & 3], s[q], s[q + 1]);
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
      float *scratch = reinterpret_cast<float *>(smem + L::kQ + L::kMat);   // [D/2][128]
      const int at = rows_s[kSoftmax + (two ? m * kTile : 0) + r];
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
            const float inv = den > 0.f ? 1.f / den : 0.f;
            w0 *= inv;
            w1 *= inv;
            if (at >= 0) p.lse[at] = part_lse(mx, den);
          }
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            float o[32];
            tm_ld32(sO + h * (D / 2) + 32 * q, o);
            tm_wait_ld();
            pin32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              o[e] *= w0;
              if (merge) o[e] = fmaf(w1, scratch[(32 * q + e) * kTile + r], o[e]);
            }
            if (at >= 0) {
              float *dst = p.o + static_cast<size_t>(at) * D + h * (D / 2) + 32 * q;
#pragma unroll
              for (int e = 0; e < 32; e += 8) store8(dst + e, o + e);
            }
          }
        }
        if (merge) meet();
      }
      meet();   // both are done with the item
    }
    tc_fence_before();
  }
  __syncthreads();
  if (tid == 0)
    p.status[blockIdx.x] = misc[0] ? kPrefixGaveUp : misc[4] ? kPrefixSkipped : misc[5];
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int D, bool POLL>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                   cudaStream_t s) {
  auto kern = prefix_tc_kernel<D, POLL>;
  static std::atomic<unsigned long long> attrs_set{0};
  cudaError_t e = set_attributes_once(attrs_set, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_waiting(kern, p.C, kThreads, Lay<D>::kBytes, s, tk, tv, p);
}

}  // namespace

cudaError_t launch_prefix_bf16(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                               int D, cudaStream_t s) {
  if (p.wait_limit <= kPollLimit)
    return D == 64 ? launch<64, true>(tk, tv, p, s) : launch<128, true>(tk, tv, p, s);
  return D == 64 ? launch<64, false>(tk, tv, p, s) : launch<128, false>(tk, tv, p, s);
}

}  // namespace pkv
