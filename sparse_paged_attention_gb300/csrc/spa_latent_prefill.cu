// spa_latent_prefill.cu - expanded latent attention over ragged causal sequences: per head, keys
// [k_nope | k_rope] (k_rope shared by all heads) and values v.
//
//   s_ij = scale q_i . [k_nope_j | k_rope_j],   out_i = sum_{j <= i + n_k - n_q} softmax(s_i)_j v_j
//
// Bound by the tensor cores: 2 (d_k + d_v) flops a visible (query, key) pair and head against a few
// bytes.  A CTA takes 256 queries of one head as two tiles of 128 and streams tiles of 128 keys:
//
//   S_t = Q_t K^T    tcgen05, M = 128 queries, N = 128 keys, both operands in shared memory
//   O_t += P_t V     M = 128 queries, N = d_v, A = P_t from TMEM (bf16, in the columns of its own S_t)
//
// TMEM holds one S (128 columns, fp32), P_0 and P_1 (64 each) and O_0, O_1 (128 each).  S is the query
// tiles' in turn: it is free again as soon as a tile's softmax has its row in registers, so the next S
// (the other tile's) is worked out under the exponentials of this one, and neither waits for PV.
//
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread has one query's row of S: maximum, exponentials and
//                    sum without any exchange; P to TMEM; O rescaled only when a row's maximum has
//                    grown by more than 2^8; epilogue
//   warp 8           MMAs of S;  warp 9: MMAs of O (apart, so that neither one's waits keep the tensor
//                    core idle)
//   warp 10          schedule and tensor-map copies: Q once an item; K in chunks of 64 dimensions (the
//                    rotary ones last) through a ring of four, each free as soon as the second tile's
//                    MMAs have read it; V through two slots
//
// Items (256 queries, head) go to CTAs statically, sequence after sequence, in an order that starts with
// the last queries (the longest rows) of all heads and folds back and forth over the CTAs, so that long
// and short items add up alike; a last round that would leave half of the CTAs idle is shared out by
// single tiles.  The copies zero-fill what lies past a width (any multiple of 8); rows past a sequence's
// end are other data: masked as keys, blanked as values, not stored as queries.
//
// Measured (nope 128, rotary 64, v 128, 64 heads): 8,192 tokens in 0.91 ms (1,500 TFLOP/s: 80% of the
// measured bf16 burst rate; 0.99 ms and 1,386 TFLOP/s when the chip has been busy for seconds, 82% of
// the sustained rate), 1,075 and 1,096 tokens after 12,000 in 0.92 ms (1,210 TFLOP/s: 512 items of two
// tiles and 128 of one on 152 CTAs; 0.97 ms without the halves of the last round).  A step of
// both tiles takes about 3,900 cycles against 2,560 of its MMAs: S keeps shared memory busy all the time
// that it runs (8 KB an MMA of 64 cycles), so the copies of K and V stretch it, and between two S pass
// a commit, the read into registers and an arrival, about 500 cycles, which PV fills only in part.
// Steps on the way, 8,192 tokens: S_0 and S_1 apart with P in their columns 1.29 ms, P in halves 1.15,
// one S buffer 0.99, two fp32 operations an instruction and MMAs without waits between them 0.94, one
// mask instead of two 0.91.  Tried and slower: one warp for both products in a fixed order (1.06 ms;
// 1.24 with the waits moved under the MMAs), five K chunks and V by halves (1.06), prefetches of K and
// V into L2 (1.03).
#include "spa_errors.h"
#include "spa_latent.h"
#include "spa_launch.h"

namespace spa {

namespace {

constexpr int kTile = 128;                       // queries of a tile, keys of a step
constexpr int kChunk = kTile * 128;              // 128 rows of 64 bf16 values
constexpr int kKs = 4, kVs = 2;                  // ring slots: chunks of K, tiles of V
constexpr int kThreads = 352;
constexpr int kItems = 2;                        // item infos in flight
constexpr int kTmemCols = 512;
constexpr int kPCol = 128, kOCol = 256;          // S: columns 0 .. 127
constexpr float kTau = 8.f;                      // lazy rescale threshold (log2 units)

constexpr int kQOff = 0;                                     // [2 tiles][3 chunks]
constexpr int kKOff = kQOff + 6 * kChunk;
constexpr int kVOff = kKOff + kKs * kChunk;
constexpr int kInfoOff = kVOff + kVs * 2 * kChunk;

struct Item {
  int q0, n;          // first query row, queries of the item (0: no more items)
  int k0, nk;         // first key row, keys of the sequence
  int pos;            // position of the item's first query (may be negative: it sees no key)
  int head;
  int steps[2];       // key tiles of query tile 0, 1
};

enum {
  B_QFULL = 0, B_QEMPTY = B_QFULL + 2, B_KFULL = B_QEMPTY + 2, B_KEMPTY = B_KFULL + kKs,
  B_VFULL = B_KEMPTY + kKs, B_VEMPTY = B_VFULL + kVs, B_SFULL = B_VEMPTY + kVs, B_SEMPTY = B_SFULL + 2,
  B_PREADY = B_SEMPTY + 1, B_PVDONE = B_PREADY + 4, B_OFREE = B_PVDONE + 2, B_IFULL = B_OFREE + 2,
  B_IEMPTY = B_IFULL + kItems, B_DRAIN = B_IEMPTY + kItems, B_COUNT = B_DRAIN + 2
};
constexpr int kBarOff = kInfoOff + kItems * (int)sizeof(Item);
constexpr int kMiscOff = kBarOff + B_COUNT * 8;
constexpr int kSmem = kMiscOff + 8;
static_assert(kSmem <= 232448, "shared memory budget");

struct PrefillParams {
  CUtensorMap q, kn, kr, v;
  LatentPrefillArgs a;
  float scale_log2;        // |scale| log2(e), never 0 (times a masked key's -inf it would be NaN): a scale of
  int q_zero;              // 0 is q = 0, read past the last row, instead
  int negate;              // scale < 0
};

__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int warp = (int)warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kMiscOff + 4);
  Item* items = reinterpret_cast<Item*>(sm + kInfoOff);
#define BAR(i) (sb + (uint32_t)kBarOff + 8u * (uint32_t)(i))
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKs; ++i) {
      mbar_init(BAR(B_KFULL + i), 1);
      mbar_init(BAR(B_KEMPTY + i), 1);
    }
    for (int i = 0; i < kVs; ++i) {
      mbar_init(BAR(B_VFULL + i), 1);
      mbar_init(BAR(B_VEMPTY + i), 1);
    }
    mbar_init(BAR(B_SEMPTY), 4);             // lane 0 of the four softmax warps that have read it
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_QFULL + i), 1);
      mbar_init(BAR(B_QEMPTY + i), 1);
      mbar_init(BAR(B_SFULL + i), 1);
      mbar_init(BAR(B_PREADY + i), 4);       // lane 0 of the tile's four softmax warps: P's first half,
      mbar_init(BAR(B_PREADY + 2 + i), 4);   // and its second
      mbar_init(BAR(B_PVDONE + i), 1);
      mbar_init(BAR(B_OFREE + i), 4);
      mbar_init(BAR(B_DRAIN + i), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(BAR(B_IFULL + i), 1);
      mbar_init(BAR(B_IEMPTY + i), 10);      // eight softmax and two MMA warps
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc(sb + kMiscOff, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*reinterpret_cast<volatile uint32_t*>(sm + kMiscOff));
  pdl_launch_dependents();
  pdl_wait();   // nothing global before the grid before this one is done

  const LatentPrefillArgs& a = p.a;
  const int nkc = (a.dn + 63) >> 6, nvc = (a.dv + 63) >> 6;   // 64-wide chunks of k_nope, v
  const bool rope = a.dr > 0;

  // Item info n of this CTA (0, 1, ..), read by every consumer warp; false when the CTA gives up.
  const auto next_item = [&](int n, Item& it) -> bool {
    const int s = n % kItems;
    if (!warp_wait(BAR(B_IFULL + s), (uint32_t)((n / kItems) & 1), abort_flag)) return false;
    const volatile int* src = reinterpret_cast<const volatile int*>(items + s);
    int* dst = reinterpret_cast<int*>(&it);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) dst[i] = (int)warp_uniform((uint32_t)src[i]);
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(B_IEMPTY + s));
    return true;
  };

  if (warp == 10) {
    // ================================ schedule and copies =================================
    // Tiles of 256 queries of the sequences b0 + lane, their bounds, and the inclusive sum over the lanes.
    // A sequence with bad bounds has none, nor has one that begins before an earlier sequence's end (no
    // two items write one row).  `highest`: the largest bound of the sequences before b0.
    const auto tiles_at = [&](int b0, int& highest, int& q0, int& q1, int& k0, int& k1, int& mine, bool& bad) {
      const int b = b0 + lane;
      q0 = q1 = k0 = k1 = 0;
      bad = false;
      if (b < a.B) {
        q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
        k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
      }
      int top = b < a.B ? q0 : 0;              // largest bound up to and with this sequence's first
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, x);
      }
      top = max(top, highest);
      if (b < a.B)
        bad = q0 < top || q1 < q0 || q1 > a.num_q || k0 < 0 || k1 < k0 || k1 > a.num_k;
      mine = bad ? 0 : (q1 - q0 + 2 * kTile - 1) / (2 * kTile);
      int scan = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
      }
      highest = __shfl_sync(0xffffffffu, top, 31);
      return scan;
    };
    // The 32 sequences with the next item's tile; a CTA's items come in their order, so that every
    // sequence's bounds are read once for the sum and once on the way.
    int c_q0, c_q1, c_k0, c_k1, c_mine, c_highest = 0, c_b0 = 0;
    bool c_bad;
    int c_scan = tiles_at(0, c_highest, c_q0, c_q1, c_k0, c_k1, c_mine, c_bad);
    int c_before = 0, c_tiles = __shfl_sync(0xffffffffu, c_scan, 31);   // tiles before them, theirs
    if (c_bad) flag_error(SPA_ERR_INDEX);
    int total = c_tiles;
    for (int b0 = 32, highest = c_highest; b0 < a.B; b0 += 32) {
      int q0, q1, k0, k1, mine;
      bool bad;
      const int scan = tiles_at(b0, highest, q0, q1, k0, k1, mine, bad);
      if (bad) flag_error(SPA_ERR_INDEX);
      total += __shfl_sync(0xffffffffu, scan, 31);
    }
    const long long n_items = (long long)total * a.H;
    // Rounds of one item a CTA; where a last round would leave half of the CTAs idle its items are taken
    // by single tiles (which take half as long).
    const long long whole = n_items / gridDim.x * gridDim.x;
    const bool halves = 2 * (n_items - whole) <= gridDim.x;
    const int nc = nkc + (rope ? 1 : 0);       // chunks of a key
    int n = 0, qs[2] = {0, 0};                 // items, query tiles copied
    uint32_t kc = 0, vc = 0;                   // chunks of K, tiles of V copied
    bool ok = true;
    for (; ok; ++n) {
      // the n-th item of this CTA; every other round goes backwards
      long long i = (long long)n * gridDim.x + ((n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      int from = 0, upto = 2 * kTile;        // queries of the item that this CTA takes
      if (halves && i >= whole) {
        from = (int)((i - whole) & 1) * kTile;
        upto = from + kTile;
        i = whole + (i - whole) / 2;
      }
      Item it = {};
      if (i < n_items) {
        const int tile = (int)(i / a.H);
        it.head = (int)(i % a.H);
        while (tile >= c_before + c_tiles) {           // (below the sum of all)
          c_before += c_tiles;
          c_b0 += 32;
          c_scan = tiles_at(c_b0, c_highest, c_q0, c_q1, c_k0, c_k1, c_mine, c_bad);
          c_tiles = __shfl_sync(0xffffffffu, c_scan, 31);
        }
        const int k = __ffs(__ballot_sync(0xffffffffu, tile < c_before + c_scan)) - 1;
        // a sequence's last tiles, which see the most keys, come first
        const int after = __shfl_sync(0xffffffffu, c_before + c_scan, k) - 1 - tile;
        const int q0 = __shfl_sync(0xffffffffu, c_q0, k), q1 = __shfl_sync(0xffffffffu, c_q1, k);
        const int k0 = __shfl_sync(0xffffffffu, c_k0, k), k1 = __shfl_sync(0xffffffffu, c_k1, k);
        const int r = after * 2 * kTile + from;
        it.q0 = q0 + r;
        it.n = max(0, min(upto - from, q1 - q0 - r));    // (0, a second half of nothing: the last)
        it.k0 = k0;
        it.nk = k1 - k0;
        it.pos = it.nk - (q1 - q0) + r;
        // (position of a tile's last query, and the key tiles up to it)
        const int last0 = it.pos + min(it.n, kTile) - 1, last1 = it.pos + it.n - 1;
        it.steps[0] = last0 >= 0 ? last0 / kTile + 1 : 0;
        it.steps[1] = it.n > kTile && last1 >= 0 ? last1 / kTile + 1 : 0;
      }
      const int s = n % kItems;
      ok = warp_wait(BAR(B_IEMPTY + s), (uint32_t)(((n / kItems) & 1) ^ 1), abort_flag);
      if (!ok) break;
      if (lane == 0) {
        items[s] = it;
        __threadfence_block();
        mbar_arrive(BAR(B_IFULL + s));
      }
      __syncwarp();
      if (it.n == 0) break;
      const int steps = max(it.steps[0], it.steps[1]);
      if (steps == 0) continue;
      const bool lead = elect_one();
      // the item's queries
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (it.steps[t] == 0 || !ok) continue;
        ok = warp_wait(BAR(B_QEMPTY + t), (uint32_t)((qs[t] & 1) ^ 1), abort_flag);
        if (!ok) continue;
        ++qs[t];
        if (lead) {
          mbar_arrive_expect_tx(BAR(B_QFULL + t), (uint32_t)(nc * kChunk));
          for (int c = 0; c < nc; ++c)
            tma_box3(sb + kQOff + (t * 3 + c) * kChunk, &p.q, c < nkc ? 64 * c : a.dn, it.head,
                     p.q_zero ? a.num_q : it.q0 + t * kTile, BAR(B_QFULL + t));
        }
        __syncwarp();
      }
      for (int j = 0; j < steps && ok; ++j) {
        const int row = it.k0 + j * kTile;
        // Where the keys end inside the tile, a softmax warp will wait for its V by parity.  That needs the
        // fill before in the slot to have landed, which a query tile that had no part in it (of an item of
        // one query tile, before one whose first tile sees no key) has not seen: seen here, before
        // the keys without which there is no S.
        if (it.nk - j * kTile < kTile && vc >= kVs) {
          const uint32_t f = vc - kVs;
          if (!(ok = warp_wait(BAR(B_VFULL + f % kVs), (f / kVs) & 1, abort_flag))) break;
        }
        for (int c = 0; c < nc; ++c, ++kc) {
          const uint32_t sl = kc % kKs, full = BAR(B_KFULL + sl);
          if (!(ok = warp_wait(BAR(B_KEMPTY + sl), ((kc / kKs) & 1) ^ 1, abort_flag))) break;
          if (lead) {
            mbar_arrive_expect_tx(full, (uint32_t)kChunk);
            if (c < nkc) tma_box3(sb + kKOff + sl * kChunk, &p.kn, 64 * c, it.head, row, full);
            else tma_box3(sb + kKOff + sl * kChunk, &p.kr, 0, 0, row, full);
          }
          __syncwarp();
        }
        if (!ok) break;
        const uint32_t sl = vc % kVs, full = BAR(B_VFULL + sl);
        if (!(ok = warp_wait(BAR(B_VEMPTY + sl), ((vc / kVs) & 1) ^ 1, abort_flag))) break;
        if (lead) {
          mbar_arrive_expect_tx(full, (uint32_t)(nvc * kChunk));
          for (int c = 0; c < nvc; ++c)
            tma_box3(sb + kVOff + (sl * 2 + c) * kChunk, &p.v, 64 * c, it.head, row, full);
        }
        __syncwarp();
        ++vc;
      }
    }
    // copies in flight must land before the CTA ends (at once after a normal run)
    if (lane == 0) {
      for (int t = 0; t < 2; ++t)
        if (qs[t] > 0) mbar_wait_drain(BAR(B_QFULL + t), (uint32_t)((qs[t] - 1) & 1));
      for (uint32_t f = kc > kKs ? kc - kKs : 0; f < kc; ++f)
        mbar_wait_drain(BAR(B_KFULL + f % kKs), (f / kKs) & 1);
      for (uint32_t f = vc > kVs ? vc - kVs : 0; f < vc; ++f)
        mbar_wait_drain(BAR(B_VFULL + f % kVs), (f / kVs) & 1);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ================================= MMAs of S ==========================================
    // (bit 13 of the instruction descriptor negates A: a negative scale)
    const uint32_t idS = idesc_bf16(kTile, kTile, 0, 0) | (p.negate ? 1u << 13 : 0u);
    const uint64_t dq0 = sdesc(sb + kQOff, 16, 1024), dk0 = sdesc(sb + kKOff, 16, 1024);
    const bool lead = elect_one();
    const int nc = nkc + (rope ? 1 : 0);
    uint32_t kc = 0, issued = 0;                 // chunks of K seen, S issued
    int qs[2] = {0, 0};                          // query tiles seen
    bool ok = true;
    Item it;
    for (int n = 0; ok && (ok = next_item(n, it)) && it.n > 0; ++n) {
      const int steps = max(it.steps[0], it.steps[1]);
      for (int j = 0; j < steps && ok; ++j, kc += nc) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= it.steps[t] || !ok) continue;
          const bool last = t == 1 || j >= it.steps[1];      // the last tile to read this step's keys
          if (t == 0 || it.steps[0] <= j)                    // the first
            for (int c = 0; c < nc && ok; ++c)
              ok = warp_wait(BAR(B_KFULL + (kc + c) % kKs), ((kc + c) / kKs) & 1, abort_flag);
          if (ok && j == 0) ok = warp_wait(BAR(B_QFULL + t), (uint32_t)(qs[t]++ & 1), abort_flag);
          // the S before has been read
          if (ok && issued > 0) ok = warp_wait(BAR(B_SEMPTY), (issued - 1) & 1, abort_flag);
          if (!ok) continue;
          ++issued;
          tc_fence_after();
          if (lead) {
            for (int c = 0; c < nc; ++c) {
              const uint32_t sl = (kc + c) % kKs;
              const int ks = ((c < nkc ? min(64, a.dn - 64 * c) : a.dr) + 15) >> 4;
              const uint64_t dq = desc_add(dq0, (t * 3 + c) * kChunk), dk = desc_add(dk0, sl * kChunk);
              mma_bf16(tmem, dq, dk, idS, c != 0);
              if (ks == 4) {
#pragma unroll
                for (int st = 1; st < 4; ++st) mma_bf16(tmem, desc_add(dq, st * 32), desc_add(dk, st * 32), idS, 1u);
              } else {
                for (int st = 1; st < ks; ++st) mma_bf16(tmem, desc_add(dq, st * 32), desc_add(dk, st * 32), idS, 1u);
              }
              if (last) mma_commit(BAR(B_KEMPTY + sl));
            }
            mma_commit(BAR(B_SFULL + t));
            if (j == it.steps[t] - 1) mma_commit(BAR(B_QEMPTY + t));
          }
          __syncwarp();
        }
      }
    }
    // nothing may still write TMEM when it is released
    if (lead) {
      mma_commit(BAR(B_DRAIN));
      mbar_wait_drain(BAR(B_DRAIN), 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ================================= MMAs of O ==========================================
    const int nv = (a.dv + 15) & ~15;
    const uint32_t idO = idesc_bf16(kTile, nv, 0, 1);
    const uint64_t dv0 = sdesc(sb + kVOff, kChunk, 1024);         // MN-major: 64 values a chunk
    const bool lead = elect_one();
    uint32_t vc = 0;
    int done[2] = {0, 0}, opened[2] = {0, 0};
    bool ok = true;
    Item it;
    for (int n = 0; ok && (ok = next_item(n, it)) && it.n > 0; ++n) {
      const int steps = max(it.steps[0], it.steps[1]);
      for (int j = 0; j < steps && ok; ++j, ++vc) {
        const uint32_t sl = vc % kVs;
        ok = warp_wait(BAR(B_VFULL + sl), (vc / kVs) & 1, abort_flag);
        if (!ok) break;
        const uint64_t dv = desc_add(dv0, sl * 2 * kChunk);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= it.steps[t]) continue;
          ok = warp_wait(BAR(B_PREADY + t), (uint32_t)(done[t] & 1), abort_flag);
          if (ok && j == 0) {                    // O of the item before has been stored
            ok = warp_wait(BAR(B_OFREE + t), (uint32_t)((opened[t] & 1) ^ 1), abort_flag);
            ++opened[t];
          }
          if (!ok) break;
          ++done[t];
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)       // 16 keys a step
              mma_bf16_ts(tmem + kOCol + t * kTile, tmem + kPCol + t * 64 + kk * 8, desc_add(dv, kk * 2048), idO,
                          (j > 0 || kk > 0) ? 1u : 0u);
          }
          __syncwarp();
          ok = warp_wait(BAR(B_PREADY + 2 + t), (uint32_t)((done[t] - 1) & 1), abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int kk = 4; kk < 8; ++kk)
              mma_bf16_ts(tmem + kOCol + t * kTile, tmem + kPCol + t * 64 + kk * 8, desc_add(dv, kk * 2048), idO, 1u);
            mma_commit(BAR(B_PVDONE + t));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lead) mma_commit(BAR(B_VEMPTY + sl));
        __syncwarp();
      }
    }
    if (lead) {
      mma_commit(BAR(B_DRAIN + 1));
      mbar_wait_drain(BAR(B_DRAIN + 1), 0);
    }
    __syncwarp();
  } else {
    // ================================ softmax and epilogue ================================
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;      // query tile, row in it == TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t pc = lanes + kPCol + t * 64, oc = lanes + kOCol + t * kTile;
    const float s2 = p.scale_log2;
    int done = 0;                                // steps of this tile done
    uint32_t vc = 0;                             // tiles of V seen
    bool ok = true;
    Item it;
    for (int n = 0; ok && (ok = next_item(n, it)) && it.n > 0; ++n) {
      const int steps = it.steps[t], all_steps = max(it.steps[0], it.steps[1]);
      const int pos = it.pos + t * kTile + row;  // this query sees keys 0 .. pos
      const int pos_min = it.pos + t * kTile + (warp & 3) * 32;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++done) {
        if (!(ok = warp_wait(BAR(B_SFULL + t), (uint32_t)(done & 1), abort_flag))) break;
        tc_fence_after();
        const int left = pos - j * kTile;        // keys 0 .. left of the tile are visible
        const bool masked = pos_min - j * kTile < kTile - 1;
        float x[4][32];                          // the row's 128 scores
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lanes + 32 * c, x[c]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_SEMPTY));
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) x[c][i] = 32 * c + i <= left ? x[c][i] : -INFINITY;
        }
        float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2) y[c] = fmaxf(y[c], fmaxf(x[c][i], x[c][i + 1]));
        const float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        const float mt = mx == -INFINITY ? -INFINITY : mx * s2;
        const float mn = mt > m + kTau ? mt : m;
        const bool grow = __any_sync(0xffffffffu, mn != m);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = fast_exp2(m - ref);
        m = mn;
        if (j > 0) {
          // PV of the step before has read P and added to O
          if (!(ok = warp_wait(BAR(B_PVDONE + t), (uint32_t)((done - 1) & 1), abort_flag))) break;
          tc_fence_after();
        }
        if (grow && j > 0) {
          // some row's maximum moved: rescale this warp's rows of O
#pragma unroll 1
          for (int c = 0; c < nvc * 4; ++c) {
            float o[16];
            tmem_ld16(oc + 16 * c, o);
            tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * al);
            tmem_st16(oc + 16 * c, w);
          }
        }
        const int keys = it.nk - j * kTile;      // keys of the tile that are the sequence's
        if (keys < kTile) {
          // values of other rows: a probability of zero times a NaN would still be one.  (Both tiles'
          // warps write the same zeros before their own PV.)
          const uint32_t sl = (vc + j) % kVs;
          if (!(ok = warp_wait(BAR(B_VFULL + sl), ((vc + j) / kVs) & 1, abort_flag))) break;
          for (int u = (threadIdx.x & 127); u < (kTile - keys) * nvc * 8; u += 128) {
            const int r = keys + u / (nvc * 8), w = u % (nvc * 8);
            *reinterpret_cast<uint4*>(sm + kVOff + sl * 2 * kChunk + (w >> 3) * kChunk + r * 128 +
                                      (w & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // P in two halves of 64 keys: PV starts on the first while the second is worked out
        l *= al;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              fma_f32x2(x[c][i], x[c][i + 1], s2, -ref);
              x[c][i] = fast_exp2(x[c][i]);
              x[c][i + 1] = fast_exp2(x[c][i + 1]);
            }
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(x[c][2 * i], x[c][2 * i + 1]);
            tmem_st16(pc + 16 * c, w);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_PREADY + 2 * hf + t));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2) add_f32x2(sum[c & 2], sum[(c & 2) + 1], x[c][i], x[c][i + 1]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      vc += all_steps;
      // ---- epilogue ----
      const bool mine = t * kTile + row < it.n;
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)(it.q0 + t * kTile + row) * a.H + it.head) * a.dv * 2);
      const int nu = a.dv >> 3;                  // 16-byte units of a row
      if (steps == 0) {
        if (mine)
          for (int u = 0; u < nu; ++u) dst[u] = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!(ok = warp_wait(BAR(B_PVDONE + t), (uint32_t)((done - 1) & 1), abort_flag))) break;
      tc_fence_after();
      const float inv = m == -INFINITY ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < nvc * 2; ++c) {
        float o[32];
        tmem_ld32(oc + 32 * c, o);
        tmem_wait_ld();
        if (mine) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (4 * c + u < nu)
              dst[4 * c + u] = make_uint4(pack_bf16x2(o[8 * u] * inv, o[8 * u + 1] * inv),
                                          pack_bf16x2(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                          pack_bf16x2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                          pack_bf16x2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_OFREE + t));
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t prepare_latent_prefill() {
  return cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, int sms, cudaStream_t stream) {
  PrefillParams p = {};
  p.a = a;
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;
  p.negate = a.scale < 0.f;
  p.q_zero = p.scale_log2 == 0.f;
  if (p.q_zero) p.scale_log2 = 1.f;
  if (!encode_bf16_3d(&p.q, a.q, a.dn + a.dr, a.H, a.q_sh, a.num_q, a.q_st, 1, kTile))
    return cudaErrorInvalidValue;
  if (a.num_k > 0) {   // (without keys every output row is zero and none of these is used)
    if (!encode_bf16_3d(&p.kn, a.k_nope, a.dn, a.H, a.kn_sh, a.num_k, a.kn_st, 1, kTile) ||
        !encode_bf16_3d(&p.v, a.v, a.dv, a.H, a.v_sh, a.num_k, a.v_st, 1, kTile))
      return cudaErrorInvalidValue;
    if (a.dr > 0 && !encode_bf16_3d(&p.kr, a.k_rope, a.dr, 1, 0, a.num_k, a.kr_st, 1, kTile))
      return cudaErrorInvalidValue;
  }
  // at most this many items, in two halves each; a CTA without one ends at once
  const long long items = 2 * ((long long)a.num_q / (2 * kTile) + a.B + 1) * a.H;
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  return launch_with_pdl(latent_prefill_kernel, dim3(grid), dim3(kThreads), kSmem, stream, 2LL * grid <= sms,
                         p);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t latent_prefill_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
