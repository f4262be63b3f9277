// spa_latent_tree.cu - latent attention of drafted tokens: the tokens of a sequence's tree lie behind its
// context in the latent cache, and each attends to the whole context and to those of the tree that its
// mask names (its ancestors and itself).
//
//   s_j = scale (q_c . c_j + q_r . r_j),   out = sum_j softmax(s)_j c_j
//
// All heads of all drafted tokens of a sequence are rows of one matrix against the same cached rows: n H of
// them, each 2 (2L + R) flops a cached row, so from 128 rows on the tensor cores are the bound.  A unit is 128 such
// rows; a pair of CTAs takes it (64 rows each) with tcgen05 MMAs of both (cta_group::2, M = 128):
//
//   S[row][j]  = q_row . x_j      N = 128 entries, of which each CTA brings 64: whole rows of the cache
//   O[row][d] += P[row][j] c_j[d] N = 256 channels a MMA, of which each CTA brings 128: of all 128 entries
//
// One CTA alone cannot hold O of 128 rows and L = 512 beside S (512 columns of TMEM), and with 64 rows its MMAs
// run at half the rate or wait for their operands: measured, 77 cycles for M = 128, N = 64, K = 16 with both
// operands in shared memory, where the pair's M = 128, N = 128 takes 32 (the full rate of both).  The price is that
// a CTA reads its share of channels of all entries besides its entries' whole rows: 1.85 times the tile.  (Not
// taken: the channels split between two CTAs that exchange parts of S.  Distributed shared memory moves 32 KB each way
// in 1,608 cycles, more than the MMAs of 64 entries take.)
//
// TMEM of a CTA (rows 0-63 in lanes 0-63 and, their other half of the columns, in lanes 64-127): O 256
// columns, four S of 64.  Shared memory: q, P, and two rings of cached rows: K (the CTA's own 64 entries of a tile,
// whole rows, three 128-byte chunks a fill) and V (its channels of all 128 entries, two chunks of 64 a fill).
//
//   softmax warps  (8, e4m3 16) a thread has a row and 32 (16) of a tile's entries; epilogue
//   roles 0, 3     (of the first CTA) issue the MMAs of S, and those of O
//   role 1         schedule, page tables
//   role 2         sees every fill of V land, cleans it where a tile holds what not all rows may see, and tells the
//                  first CTA
//   roles 4-7      q of a unit; role 4 the copies of V, role 5 those of K, which complete on the first CTA's
//                  barrier.  (Roles 6 and 7 only where q or cached rows go by cp.async: heads that neither divide 64
//                  nor are a multiple of it, pages that are not a multiple of eight entries.)
//
// The running maximum of a row, which its 4 (8) threads have to agree on, costs no barrier: a thread's maximum of
// tile k + 1 goes into one word of shared memory a row and tile, by an atomic maximum (whose result does not depend
// on an order), before the exponentials of tile k, and is read a tile later.  In fp32: as the reference of the
// exponentials it may be off by no more than an exponent can hold, however large the scores are.
//
// Measured (L = 512, R = 64, device time of calls in a graph, inputs that change from call to call; a call from Python
// adds about 5 us).  In bursts, at 2,070 MHz: for seconds on end the 32 drafts reach the power limit, 1,700 MHz, and
// take 394 us either way:
//   32 drafts of 5 to 16 tokens behind up to 8,187 entries, 128 heads, bf16: 361 us (1,268 TFLOP/s, 67% of the
//     measured bf16 rate); 172 tiles and 4.6 units a pair, some 3,500 cycles a tile, everything counted, of which 2,180
//     are its 52 MMAs and about 3,100 what it moves through shared memory (399 KB: the MMAs 245, the copies 138)
//   12 drafts of 20 to 60 tokens behind up to 16,004 entries, 16 heads, e4m3, pages of 24: 193 us (734 TFLOP/s)
//   one draft of 8 tokens behind 4,097 entries, 64 heads, bf16: 30 us, two tiles a pair
// These cycles are computed, from the MMAs' measured rate and 128 bytes a cycle of shared memory; by them shared
// memory is what a bf16 tile waits for.  Under ncu tensor cores are active 58% of the kernel (e4m3 48%).  Before
// it was the roles' code, each loop fetched anew for every tile: with 139 KB of it a warp that issued had waited 5.6
// cycles for its next instruction, now 0.5.  Steps, for the 32 drafts: one warp for all copies and one for all MMAs
// 755 us; a warp each 487; page tables apart from K's copies 459; polls and divisions out of line, one place for
// each fill 441; P of two tiles in turn 394; q by tensor maps and the unit's cost in the schedule 371; the merge's
// search by ballots 361.  Arrivals on the other CTA's barriers at cluster scope, 980 cycles each, had taken 1,339.
// Tried and slower: sixteen softmax warps for bf16 (464 for 441), V by whole groups through two slots (440 for 435).
// Maxima in fp32 by an atomic maximum cost what bf16 ones in places of their own did (360.2 for 359.7; e4m3, whose were
// fp32 before, 193.0 for 193.9), and those were wrong: from scores of 3e4 on off by more than an exponent holds.
//
// Cleaning: a masked entry has a weight of zero, but zero times a NaN or infinity is none.  Rows that do not
// exist are zeroed.  A drafted token's row that is not finite makes the score of whoever sees it NaN or
// infinite; its values are taken as zero, so that those who do not see it are not touched.
//
// Schedule: the tiles of all units are one line, each unit with kUnitCost tiles' room for its q and its epilogue;
// each pair takes an equal stretch.  Units cut by that leave normalised parts with their log-sum-exp, which
// tree_merge_kernel joins in the order of the pairs.
//
// e4m3 rows enter as codes: q as two e4m3 terms times a power of two a row, the weights p_j scale_j as three e5m2
// terms of an f16 number (see spa_latent_decode.cu).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_errors.h"
#include "spa_latent.h"
#include "spa_launch.h"

namespace spa {

namespace {

constexpr int kRows = 64;            // rows of a CTA
constexpr int kUnitRows = 128;       // of a pair
constexpr int kGroup = 64;           // entries of a fill
constexpr int kTile = 128;           // entries of a tile
constexpr int kChunk = kGroup * 128;
constexpr int kKFill = 3, kVFill = 2;   // chunks of a fill
constexpr int kInfos = 4;            // tile infos in flight
constexpr int kRoles = 8;            // warps besides the softmax warps
constexpr int kSBufs = 4;            // S buffers in TMEM
constexpr int kMaxTiles = 8;         // tiles whose maxima have a place: see the softmax warps
constexpr int kQScales = 8;          // units whose scales of q may be in use: S runs up to kSBufs tiles ahead
constexpr int kTmemCols = 512;
constexpr int kSCol = 256;           // O from column 0, S of 64 columns each
constexpr int kUnitCost = 4;         // tiles' worth of a unit's q and epilogue (2, 3, 6: 392, 375, 377 us for 371,
                                     // 32 drafts; 210, 204, 215 for 205, 12 e4m3 drafts)
constexpr int kMaxSlices = 128;

constexpr float kPUnit = 1024.f;     // e4m3: unit of the weights (times 2^5 at most: an e5m2 number)

enum { kFirst = 1, kLast = 2, kFinal = 4, kEnd = 8, kClean = 16 };

template <bool kFp8>
struct Cfg {
  static constexpr int kKSlots = kFp8 ? 2 : 3, kVSlots = kFp8 ? 2 : 3;
  // Softmax warps: e4m3's longer arithmetic is faster on sixteen (278 us against 308), bf16's on eight (441 against
  // 464, both at the time).
  static constexpr int kSoftmaxWarps = kFp8 ? 16 : 8;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + kRoles);
  static constexpr int kParts = kSoftmaxWarps / 2, kKeys = kTile / kParts;   // threads of a row, entries of a thread
  static constexpr int kCw = kFp8 ? 128 : 64;        // channels of a chunk
  static constexpr int kMaxChunks = kFp8 ? 5 : 9;    // of a row
  static constexpr float kTau = kFp8 ? 5.f : 8.f;    // lazy rescale threshold (log2 units)
  struct Info {
    int flags, slot, first_row, rows;                // part slot (-1: none); global row of the unit, its rows
    int tok0, unit_row, rel, seq;                    // sequence's first token, unit's first row in it, base - context
    uint32_t valid[4];                               // bit i of word w: entry 32 w + i exists
    int boxes[16];                                   // first rows of the tile's boxes
    float scale[kFp8 ? kTile : 1];                   // kPUnit times the rows' scales, and log2 of their sizes
    float lscale[kFp8 ? kTile : 1];
  };
  static constexpr int kQBytes = kFp8 ? kMaxChunks * 2 * kChunk : kMaxChunks * kChunk;
  static constexpr int kPBytes = kFp8 ? 3 * kChunk : 2 * kChunk;
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + kQBytes;
  static constexpr int kKOff = kPOff + 2 * kPBytes;              // (P of two tiles)
  static constexpr int kVOff = kKOff + kKSlots * kKFill * kChunk;
  static constexpr int kVEnd = kVOff + kVSlots * kVFill * kChunk;
  static constexpr int kMaxOff = kVEnd;                            // int [kMaxTiles][64 rows], see ordered()
  static constexpr int kQScaleOff = kMaxOff + kMaxTiles * kRows * 4;   // e4m3: float [kQScales][64]
  static constexpr int kInfoOff = kQScaleOff + (kFp8 ? kQScales * kRows * 4 : 0);
  static constexpr int kInfoEnd = kInfoOff + kInfos * (int)sizeof(Info);
  // Without boxes, the rows of the tiles' entries: int [kInfos][128].  bf16: in the last slot of V, which is
  // then not used.
  static constexpr int kRowOff = kFp8 ? kInfoEnd : kVEnd - kVFill * kChunk;
  static constexpr int kBarOff = ((kFp8 ? kRowOff + kInfos * kTile * 4 : kInfoEnd) + 7) & ~7;
  // Barriers at the same place in both CTAs.  Those marked L are used in the first CTA alone, whose MMA warp
  // waits for both; those marked 2 are completed in both by the MMAs' commits.  Every wait by parity comes when
  // that phase is the next to complete or the last that did: each role passes every phase of what it waits for.
  static constexpr int bKFull = 0 /* cp.async */, bKReady = bKFull + kKSlots /* L */,
                       bKEmpty = bKReady + kKSlots /* 2 */,
                       bVFull = bKEmpty + kKSlots, bVReady = bVFull + kVSlots /* L */,
                       bVEmpty = bVReady + kVSlots /* 2 */, bSFull = bVEmpty + kVSlots /* 2 */,
                       bSEmpty = bSFull + kSBufs /* L */, bPReady = bSEmpty + kSBufs /* L */,
                       bMax = bPReady + 2, bLFull = bMax + 2, bLEmpty = bLFull + 1, bPvDone = bLEmpty + 1 /* 2 */,
                       bQFull = bPvDone + 2 /* L */, bQLocal = bQFull + 1, bQEmpty = bQLocal + 1 /* 2 */,
                       bOFree = bQEmpty + 1 /* L */, bInfoFull = bOFree + 1, bInfoEmpty = bInfoFull + kInfos,
                       bDrain = bInfoEmpty + kInfos, kNumB = bDrain + 2;
  static constexpr int kMiscOff = kBarOff + kNumB * 8;             // TMEM base, abort flag
  static constexpr int kSmem = kMiscOff + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct Part {                 // the unit cut at the end of a slice: its first row, rows, last slice (-1: none)
  int row, rows, last, pad;
};

struct TreeParams {
  CUtensorMap chunk;          // the pool's rows, boxes of 128 bytes by `box` rows
  CUtensorMap q_lat, q_rope;  // bf16, with q_box: q by 128-byte chunks, boxes of 64 rows
  CUtensorMap k_box, v_box;   // the same by whole 128-byte chunks, boxes of a fill's chunks by 64 rows (box 64)
  LatentTreeArgs a;
  int box, box_shift;         // rows of a box: 8, 16, 32 or 64 (0: cp.async), and log2 of them
  int slices;
  // |scale| log2(e); bf16: never 0 (times a masked score's -inf it would be NaN), a scale of 0 is q = 0 instead
  float scale_log2;
  int q_zero, negate, q_box;
  Part* cut;                  // [slices]
  float* lse;                 // [slices][2][128], log2 units
  float* part;                // [slices][2][128][L]
  uint8_t* q_codes;           // e4m3: [q slots][2 CTAs][chunks][64 rows of the high term, 64 of the low][128]
  float* q_scale;             // e4m3: [q slots][128], 1 / kPUnit over the power of two in the codes
};

// The q slot of unit g of sequence b, whose first token is lo: no two units share one, and there are at most
// T H / 128 + B of them.
__host__ __device__ __forceinline__ long long q_slot(long long lo, int H, int b, int g) {
  return lo * H / kUnitRows + b + g;
}

// MMAs of the pair, issued by one thread of its first CTA; operands and results at the same places in both.
template <bool kFp8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` in both CTAs once every MMA of this thread so far has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Arrive on a barrier of either CTA (a shared::cluster address).  What the MMAs wait for is a CTA's own shared or
// tensor memory, read by that CTA's own tensor core, so the arrival orders it within the CTA: at cluster
// scope an arrival took its warp 980 cycles, and a tile of 128 entries 15,000 instead of 5,000.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// An fp32 number that is no NaN as an integer of the same order, and back.
__device__ __forceinline__ int ordered(int bits) { return bits >= 0 ? bits : bits ^ 0x7fffffff; }

// Waits whose polls are out of line: each role's loop is fetched anew every tile, and the less there is of it the
// better.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, abort_flag);
}
__device__ __noinline__ void drain(uint32_t bar, uint32_t parity) { mbar_wait_drain(bar, parity); }

// Copies of a CTA of the pair into its own shared memory that complete on a barrier of the first CTA.
__device__ __forceinline__ void tma_row_pair(uint32_t dst, const CUtensorMap* map, int x, int r, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_box3_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// A ring whose length is not known at compile time (see spa_latent_ring.h).
struct Slots {
  int n, slot = 0;
  uint32_t parity = 0;
  __device__ explicit Slots(int count) : n(count) {}
  __device__ __forceinline__ void next() {
    if (++slot == n) {
      slot = 0;
      parity ^= 1;
    }
  }
};

__device__ __noinline__ long long quotient(long long x, long long y) { return x / y; }

// A sequence as the schedule sees it: its tokens and entries, units and tiles of a unit (no units: none to do).
struct Seq {
  int lo, n, ctx, tiles;
  long long units;
  bool bad;
};
// Sequences b0 + lane; `top`: the largest bound before them, and then after.
__device__ __noinline__ Seq load_seqs(const LatentTreeArgs& a, int b0, int& top) {
  const int lane = threadIdx.x & 31, b = b0 + lane;
  Seq s = {};
  int hi = 0;
  if (b < a.pool.B) {
    s.lo = __ldg(a.cu_tokens + b);
    hi = __ldg(a.cu_tokens + b + 1);
    s.ctx = __ldg(a.context_lens + b);
  }
  int highest = b < a.pool.B ? s.lo : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, highest, o);
    if (lane >= o) highest = max(highest, x);
  }
  highest = max(highest, top);
  top = __shfl_sync(0xffffffffu, highest, 31);
  if (b >= a.pool.B) return s;
  long long cap = (long long)a.pool.bt_stride * a.pool.ps;
  cap = cap < 0x7fffff00LL ? cap : 0x7fffff00LL;    // (a tile's entries stay below 2^31)
  s.bad = s.lo < highest || hi < s.lo || hi > a.T || s.ctx < 0 || (long long)s.ctx + hi - s.lo > cap;
  if (s.bad || hi == s.lo) return s;
  s.n = hi - s.lo;
  s.tiles = (s.ctx + s.n + kTile - 1) / kTile;
  s.units = ((long long)s.n * a.H + kUnitRows - 1) / kUnitRows;
  return s;
}

// e4m3: q as two e4m3 terms times a power of two a row, in the order of the MMA's operand.  A warp takes a row; the
// last R columns repeat the rotary part, against the low codes of the rows.  (Rows of a unit's last that
// belong to no token keep what they hold: their results are not stored.)
// A warp's rows are counted on from sequence to sequence: 12 drafts, 7,500 rows, in 11 us alone; with every sequence
// begun at the first warp, which left most of them idle, it took 21.
__global__ void __launch_bounds__(256)
    tree_q_kernel(const __grid_constant__ LatentTreeArgs a, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nlp = a.pool.L >> 3, nrp = a.pool.R >> 3, n_chunks = (a.pool.row_bytes + 127) >> 7;
  int top = 0;
  long long r = (long long)blockIdx.x * 8 + warp;   // this warp's next row, counted on through the sequences
  for (int b0 = 0; b0 < a.pool.B; b0 += 32) {
    const Seq all = load_seqs(a, b0, top);
    for (int k = 0; k < 32 && b0 + k < a.pool.B; ++k) {
      const int lo = __shfl_sync(0xffffffffu, all.lo, k), n = __shfl_sync(0xffffffffu, all.n, k);
      const long long rows = (long long)n * a.H;
      for (; r < rows; r += (long long)gridDim.x * 8) {
        const long long t = lo + r / a.H, h = r % a.H;
        const uint4* ql = reinterpret_cast<const uint4*>(a.q_latent + t * a.ql_st + h * a.ql_sh);
        const uint4* qr = reinterpret_cast<const uint4*>(a.q_rope + t * a.qr_st + h * a.qr_sh);
        uint4 x[3];                              // pieces of eight values
        uint32_t mb = 0;                         // largest magnitude (NaN if there is one)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int o = lane + 32 * i, z = o - nlp;
          x[i] = make_uint4(0, 0, 0, 0);
          if (z < 2 * nrp) x[i] = z < 0 ? __ldg(ql + o) : __ldg(qr + (z < nrp ? z : z - nrp));
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) mb = max(mb, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        mb = __reduce_max_sync(0xffffffffu, mb);
        const float m = bf16_lo(mb);
        const bool finite = mb < 0x7f80u;        // (else the row's scores become NaN through its scale)
        const float qs = finite && m > 0.f ? pow2_floor(448.f / m) : 1.f;
        const long long slot = q_slot(lo, a.H, b0 + k, 0) + r / kUnitRows;
        const int ur = (int)(r % kUnitRows), half = ur / kRows, hr = ur % kRows;
        if (lane == 0) scales[slot * kUnitRows + ur] = finite ? (1.f / kPUnit) / qs : __int_as_float(0x7fffffff);
        uint8_t* dst = codes + (slot * 2 + half) * ((long long)n_chunks * 2 * kChunk) + hr * 128;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int o = lane + 32 * i;           // piece o: chunk o / 16, 16-byte unit (o / 2) & 7 of the row
          if (o >= 16 * n_chunks) continue;
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t high[4], low[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = bf16_lo(w[e]) * qs, z = bf16_hi(w[e]) * qs;
            high[e] = e4m3x2(y, z);
            const __half2_raw hh = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)high[e], __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hh));
            low[e] = e4m3x2(y - v.x, z - v.y);
          }
          uint8_t* d = dst + (o >> 4) * (2 * kChunk) + ((((o >> 1) & 7) ^ (hr & 7)) << 4) + (o & 1) * 8;
          *reinterpret_cast<uint2*>(d) = make_uint2(high[0] | (high[1] << 16), high[2] | (high[3] << 16));
          *reinterpret_cast<uint2*>(d + kChunk) = make_uint2(low[0] | (low[1] << 16), low[2] | (low[3] << 16));
        }
      }
      r -= rows;
    }
  }
}

// kN consecutive columns of this warp's TMEM lanes.
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&x)[kN]) {
  static_assert(kN == 16 || kN == 32, "widths of the loads");
  if constexpr (kN == 16) tmem_ld16(at, x);
  else tmem_ld32(at, x);
}

// 16-byte units u[0 .. 3] of the rows of four neighbouring lanes, transposed: lane j of the four then has unit j of
// all four rows.
__device__ __forceinline__ void transpose4(uint4 (&u)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s <= 2; s *= 2) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
      uint4 &x = u[i], &y = u[i + s];            // lanes without bit s give y and take the other's x
      uint4 give = up ? x : y;
      give.x = __shfl_xor_sync(0xffffffffu, give.x, s);
      give.y = __shfl_xor_sync(0xffffffffu, give.y, s);
      give.z = __shfl_xor_sync(0xffffffffu, give.z, s);
      give.w = __shfl_xor_sync(0xffffffffu, give.w, s);
      if (up) x = give;
      else y = give;
    }
  }
}

// A 16-byte piece of cached values with zeros for what is not finite.
template <bool kFp8>
__device__ __forceinline__ uint4 finite_only(uint4 u) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kFp8) {
#pragma unroll
      for (int b = 0; b < 32; b += 8)
        if (((w[i] >> b) & 0x7fu) == 0x7fu) w[i] &= ~(0xffu << b);
    } else {
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
  }
  return u;
}

// kBox: cached rows by tensor maps, else (pages that are not a multiple of eight entries) by cp.async.
template <bool kFp8, bool kBox>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<kFp8>::kThreads, 1)
    latent_tree_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int warp = (int)warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int role = warp - C::kSoftmaxWarps;      // (negative: softmax)
  const int rank = (int)cluster_ctarank();
  const int slice = blockIdx.x >> 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kMiscOff + 4);
  typename C::Info* infos = reinterpret_cast<typename C::Info*>(sm + C::kInfoOff);
#define BAR(i) (sb + (uint32_t)C::kBarOff + 8u * (uint32_t)(i))
  const uint32_t lead_bars = mapa_cluster(sb + (uint32_t)C::kBarOff, 0);
  const auto lead_bar = [&](int i) { return lead_bars + 8u * (uint32_t)i; };   // in the first CTA

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKSlots; ++i) {
      mbar_init(BAR(C::bKFull + i), 128);
      mbar_init(BAR(C::bKReady + i), kBox ? 1 : 2);     // armed by the first CTA's loader, or role 2 of both CTAs
      mbar_init(BAR(C::bKEmpty + i), 1);
    }
    for (int i = 0; i < C::kVSlots; ++i) {
      mbar_init(BAR(C::bVFull + i), kBox ? 1 : 128);
      mbar_init(BAR(C::bVReady + i), 2);
      mbar_init(BAR(C::bVEmpty + i), 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(BAR(C::bSFull + i), 1);
      mbar_init(BAR(C::bSEmpty + i), 2 * C::kSoftmaxWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(BAR(C::bMax + i), C::kSoftmaxWarps);
    mbar_init(BAR(C::bLFull), C::kSoftmaxWarps);
    mbar_init(BAR(C::bLEmpty), C::kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::bPReady + i), 2 * C::kSoftmaxWarps);
      mbar_init(BAR(C::bPvDone + i), 1);
    }
    mbar_init(BAR(C::bQFull), kFp8 || p.q_box ? 2 : 8);
    mbar_init(BAR(C::bQLocal), 1);
    mbar_init(BAR(C::bQEmpty), 1);
    mbar_init(BAR(C::bOFree), 2 * C::kSoftmaxWarps);
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(BAR(C::bInfoFull + i), 1);
      mbar_init(BAR(C::bInfoEmpty + i), C::kSoftmaxWarps + (rank == 0 ? 7 : 5));   // (roles 0 and 3: the first CTA)
    }
    mbar_init(BAR(C::bDrain), 1);
    mbar_init(BAR(C::bDrain + 1), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = threadIdx.x; i < kMaxTiles * kRows; i += C::kThreads)
    reinterpret_cast<int*>(sm + C::kMaxOff)[i] = ordered(__float_as_int(-INFINITY));
  if (role == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + C::kMiscOff),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*reinterpret_cast<volatile uint32_t*>(sm + C::kMiscOff));
  pdl_launch_dependents();
  pdl_wait();   // nothing global before the grid before this one is done

  const LatentTreeArgs& a = p.a;
  const int L = a.pool.L, W = a.pool.row_bytes;
  const int n_chunks = (W + 127) >> 7;                         // of a row
  const int n_half = ((L + C::kCw - 1) / C::kCw + 1) >> 1;     // chunks of values a CTA brings
  const int k_fills = (n_chunks + kKFill - 1) / kKFill;
  const int v_fills = (n_half + kVFill - 1) / kVFill;          // of a group
  Slots ks(C::kKSlots), vs(kBox || kFp8 ? C::kVSlots : C::kVSlots - 1);   // where a role is in the rings
  // (lanes that copy boxes: chunk of the fill and box of the group)
  const int per_group = kGroup >> p.box_shift, my_c = lane >> (6 - p.box_shift), my_box = lane & (per_group - 1);
  const uint32_t my_off = my_c * kChunk + ((my_box << p.box_shift) << 7);
  if (role == 1) {
    // ================================ schedule and loads ==================================
    int top = 0, s0 = 0;
    Seq cur = load_seqs(a, 0, top);
    if (slice == 0 && rank == 0 && cur.bad) flag_error(SPA_ERR_INDEX);
    long long tiles = cur.units * cur.tiles, units = cur.units;
    {
      int t = top;
      for (int b0 = 32; b0 < a.pool.B; b0 += 32) {
        const Seq s = load_seqs(a, b0, t);
        if (slice == 0 && rank == 0 && s.bad) flag_error(SPA_ERR_INDEX);
        tiles += s.units * s.tiles;
        units += s.units;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
      units += __shfl_xor_sync(0xffffffffu, units, o);
    }
    // The line: a unit that begins at w has its tile 0 there, and tile j > 0 at w + cost + j.  A slice takes the
    // tiles from per * slice to before per * (slice + 1).  (cost < per, so that a unit has tiles in every slice
    // from its first to its last.)
    const long long each = quotient(tiles + p.slices - 1, p.slices);
    const long long cost = min((long long)(units > 1 ? kUnitCost : 0), max(each, 1LL) - 1);
    const long long per = max(quotient(tiles + cost * units + p.slices - 1, p.slices), 1LL);
    const long long begin = per * slice, end = begin + per;
    int it_s = 0;                                // next tile: sequence (in the chunk), unit, tile of the unit
    long long it_u = 0, w_unit = 0, left_all = 0;
    int it_j = 0;
    {
      bool found = false;
      int chunk = 0, chunk_top = 0, t = 0;
      long long w0 = 0;
      for (int b0 = 0; b0 < a.pool.B; b0 += 32) {
        const int t_before = t;
        const Seq s = load_seqs(a, b0, t);
        const long long span = s.tiles + cost, mine = s.units * span;
        long long sum = mine;                    // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const long long w = w0 + sum - mine;
        const auto before = [&](long long x) {   // tiles of this lane's sequence before x
          if (x <= w || s.units == 0) return 0LL;
          const long long u = min(quotient(x - w, span), s.units);
          const long long y = x - w - u * span;
          return u * s.tiles + (u < s.units && y > 0 ? min((long long)s.tiles, max(1LL, y - cost)) : 0);
        };
        const long long lo = before(begin), hi = before(end);
        left_all += hi - lo;
        const unsigned m = __ballot_sync(0xffffffffu, lo < s.units * s.tiles);
        if (!found && m) {
          const int k = __ffs(m) - 1;
          found = true;
          chunk = b0;
          chunk_top = t_before;
          it_s = k;
          const long long l = __shfl_sync(0xffffffffu, lo, k), wk = __shfl_sync(0xffffffffu, w, k);
          const int tl = __shfl_sync(0xffffffffu, s.tiles, k);
          it_u = quotient(l, tl);
          it_j = (int)(l - it_u * tl);
          w_unit = wk + it_u * (tl + cost);
        }
        w0 += __shfl_sync(0xffffffffu, sum, 31);
        if (w0 >= end) break;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) left_all += __shfl_xor_sync(0xffffffffu, left_all, o);
      if (chunk != 0) {
        s0 = chunk;
        top = chunk_top;
        cur = load_seqs(a, s0, top);
      }
    }
    // The current unit
    int u_lo = 0, u_n = 0, u_ctx = 0, u_tiles = 0, u_seq = 0, u_len = 0;
    long long u_units = 0;
    bool started = false, fresh = true;
    int left = 0;
    Part cut = {0, 0, -1, 0};
    const auto begin_unit = [&]() {
      while (it_u >= __shfl_sync(0xffffffffu, cur.units, it_s)) {   // (there is a unit to come)
        it_u = 0;
        if (++it_s == 32) {
          it_s = 0;
          s0 += 32;
          cur = load_seqs(a, s0, top);
        }
      }
      u_lo = __shfl_sync(0xffffffffu, cur.lo, it_s);
      u_n = __shfl_sync(0xffffffffu, cur.n, it_s);
      u_ctx = __shfl_sync(0xffffffffu, cur.ctx, it_s);
      u_tiles = __shfl_sync(0xffffffffu, cur.tiles, it_s);
      u_units = __shfl_sync(0xffffffffu, cur.units, it_s);
      u_seq = s0 + it_s;
      u_len = u_ctx + u_n;
      started = it_j == 0;
      left = u_tiles - it_j;
      fresh = true;
      if (started && left > left_all) {          // (the line ends inside it)
        const long long unit_row = it_u * kUnitRows;
        cut.row = (int)((long long)u_lo * a.H + unit_row);
        cut.rows = (int)min((long long)kUnitRows, (long long)u_n * a.H - unit_row);
        cut.last = (int)quotient(w_unit + cost + u_tiles - 1, per);
      }
    };
    struct Tile {
      int flags, slot, base, first_row, rows, tok0, unit_row, rel, valid_len;
      int blk[4];                                // boxed: of box `lane`; else of entries lane + 32 e
    };
    const auto page_of = [&](int key) { return a.pool.ps_shift >= 0 ? key >> a.pool.ps_shift : key / a.pool.ps; };
    const int my_key = kBox ? lane << p.box_shift : lane;        // first entry of this lane's box
    const bool has_box = kBox && my_key < kTile;
    const auto next_tile = [&](Tile& x) {        // the next tile, its block-table reads under way
      x.flags = kEnd;
      if (left_all == 0) return;
      if (left == 0) {
        if (u_tiles > 0) {                       // (0: the line's first unit, which may begin at any tile)
          w_unit += cost + u_tiles;
          ++it_u;
          it_j = 0;
        }
        begin_unit();
      }
      const bool last = left == 1 || left_all == 1;
      x.base = it_j * kTile;
      x.slot = started && left == 1 ? -1 : (started ? 1 : 0);
      x.unit_row = (int)(it_u * kUnitRows);
      x.first_row = (int)((long long)u_lo * a.H + it_u * kUnitRows);
      x.rows = (int)min((long long)kUnitRows, (long long)u_n * a.H - it_u * kUnitRows);
      x.tok0 = u_lo;
      x.rel = x.base - u_ctx;
      x.valid_len = u_len - x.base;
      x.flags = (fresh ? kFirst : 0) | (last ? kLast : 0) | (left_all == 1 ? kFinal : 0);
      // (the q slot of the unit goes with the sequence; see the published info)
      x.blk[0] = x.blk[1] = x.blk[2] = x.blk[3] = -2;
      const int32_t* bt = a.pool.bt + (size_t)u_seq * a.pool.bt_stride;
      if (kBox) {
        if (has_box && my_key < x.valid_len) x.blk[0] = __ldg(bt + page_of(x.base + my_key));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (lane + 32 * e < x.valid_len) x.blk[e] = __ldg(bt + page_of(x.base + lane + 32 * e));
      }
      fresh = false;
      --left_all;
      --left;
      ++it_j;
    };
    const int total_rows = (int)(a.pool.num_blocks * a.pool.ps);
    bool ok = true;
    Tile nxt = {}, x = {};
    int box_rows = 0;
#pragma unroll 1
    for (int k = -1; ok; ++k) {
      x = nxt;
      const int seq = u_seq;
      if (k < 0 || !(x.flags & (kEnd | kFinal))) next_tile(nxt);
      if (k < 0) continue;
      // rows of the tile
      int rows4[4];
      uint32_t valid[4];
      bool clean = false;
      if (!(x.flags & kEnd)) {
        if (kBox) {
          const bool good = x.blk[0] >= 0 && (long long)x.blk[0] < a.pool.num_blocks;
          if (x.blk[0] != -2 && !good) flag_error(SPA_ERR_INDEX);
          // a box without entries starts past the last row and is filled with zeros
          const int key = x.base + my_key;
          box_rows = good ? x.blk[0] * a.pool.ps + (key - page_of(key) * a.pool.ps) : total_rows;
          const uint32_t okb = __ballot_sync(0xffffffffu, good);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // a bit an entry: the boxes' bits spread, cut off at the sequence's end
            const uint32_t b = okb >> ((32 * e) >> p.box_shift);
            uint32_t m = p.box >= 32   ? 0u - (b & 1u)
                         : p.box == 16 ? (b & 1u) * 0xffffu | (b >> 1 & 1u) * 0xffff0000u
                                       : (b & 1u) * 0xffu | (b >> 1 & 1u) * 0xff00u | (b >> 2 & 1u) * 0xff0000u |
                                             (b >> 3 & 1u) * 0xff000000u;
            const int n = x.valid_len - 32 * e;
            if (n < 32) m &= n <= 0 ? 0u : (1u << n) - 1u;
            valid[e] = m;
            if constexpr (kFp8) {
              const int i = lane + 32 * e;
              rows4[e] = __shfl_sync(0xffffffffu, box_rows, i >> p.box_shift) + (i & (p.box - 1));
              if (!(m >> lane & 1u)) rows4[e] = -1;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = x.base + lane + 32 * e;
            const bool good = x.blk[e] >= 0 && (long long)x.blk[e] < a.pool.num_blocks;
            if (x.blk[e] != -2 && !good) flag_error(SPA_ERR_INDEX);
            rows4[e] = good ? x.blk[e] * a.pool.ps + (key - page_of(key) * a.pool.ps) : -1;
            valid[e] = __ballot_sync(0xffffffffu, good);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) clean |= valid[e] != 0xffffffffu;
        clean |= x.rel + kTile > 0;              // drafted tokens' entries among them
      }
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
      if (kFp8 && !(x.flags & kEnd)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (rows4[e] >= 0) sc[e] = __ldg(a.pool.scale + rows4[e]);
      }
      // publish the tile (before its copies: the MMAs go by its flags)
      const int ri = k % kInfos;
      ok = tree_wait(BAR(C::bInfoEmpty + ri), ((k / kInfos) & 1) ^ 1, abort_flag);
      if (!ok) break;
      typename C::Info& info = infos[ri];
      if (x.flags & kEnd) {                      // (nothing to do at all: k is 0)
        if (lane == 0) {
          info.flags = kEnd;
          __threadfence_block();
          mbar_arrive(BAR(C::bInfoFull + ri));
        }
        break;
      }
      if (kBox) {
        if (lane < 16) info.boxes[lane] = box_rows;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          reinterpret_cast<int*>(sm + C::kRowOff)[ri * kTile + lane + 32 * e] = rows4[e];
      }
      if constexpr (kFp8) {
        bool one = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) one |= sc[e] == 1.f;
        if (__any_sync(0xffffffffu, one)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[e] = latent_scale_of(a.pool.rows, W, rows4[e], sc[e]);
        }
        // the maximum of a tile is taken over p_j |scale_j|, the weights that enter the value product (a scale
        // below 2^-60 counts as that: the sums of p_j alone must stay finite)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          info.scale[lane + 32 * e] = kPUnit * sc[e];
          info.lscale[lane + 32 * e] = rows4[e] >= 0 ? fmaxf(__log2f(fabsf(sc[e])), -60.f) : -INFINITY;
        }
      }
      if (lane == 0) {
        info.flags = x.flags | (clean ? kClean : 0);
        info.slot = x.slot;
        info.first_row = x.first_row;
        info.rows = x.rows;
        info.tok0 = x.tok0;
        info.unit_row = x.unit_row;
        info.rel = x.rel;
        info.seq = seq;
#pragma unroll
        for (int e = 0; e < 4; ++e) info.valid[e] = valid[e];
      }
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::bInfoFull + ri));
      if (x.flags & kFinal) break;
    }
    if (rank == 0 && lane == 0) p.cut[slice] = cut;
    __syncwarp();
  } else if (role == 0) {
    // ================================= MMAs of S ==========================================
    if (rank == 0) {
      // (bit 13 negates A: a negative scale)
      const uint32_t idS =
          (kFp8 ? idesc_e4m3(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0)) | (p.negate ? 1u << 13 : 0u);
      const uint64_t dq = sdesc(sb + C::kQOff, 16, 1024), dk0 = sdesc(sb + C::kKOff, 16, 1024);
      constexpr uint32_t kQChunk = (kFp8 ? 2 : 1) * kChunk;
      const bool lead = elect_one();
      uint32_t units = 0;
#pragma unroll 1
      for (int k = 0;; ++k) {
        const int ri = k % kInfos, sn = k % kSBufs;
        if (!tree_wait(BAR(C::bInfoFull + ri), (uint32_t)((k / kInfos) & 1), abort_flag)) break;
        const int flags = (int)warp_uniform(*reinterpret_cast<volatile int*>(&infos[ri].flags));
        if (lead) mbar_arrive(BAR(C::bInfoEmpty + ri));
        if (flags & kEnd) break;
        if ((flags & kFirst) && !tree_wait(BAR(C::bQFull), units++ & 1, abort_flag)) break;
        if (!tree_wait(BAR(C::bSEmpty + sn), (uint32_t)(((k / kSBufs) & 1) ^ 1), abort_flag)) break;
        const uint32_t dS = tmem + kSCol + sn * 64;
        bool ok = true;
#pragma unroll 1
        for (int f = 0; f < k_fills; ++f) {
          if (!(ok = tree_wait(BAR(C::bKReady + ks.slot), ks.parity, abort_flag))) break;
          tc_fence_after();
          // (the loops that issue are short, without predicates in whole chunks, and all but the issue itself is the
          // whole warp's, so that it stays in uniform registers)
          const uint64_t b0 = desc_add(dk0, ks.slot * (kKFill * kChunk)), q0 = desc_add(dq, f * kKFill * kQChunk);
          const int n = min(kKFill, n_chunks - f * kKFill), left = W - f * kKFill * 128;   // chunks, bytes to come
          const uint32_t acc = f != 0;
          const auto chunk = [&](int c, uint32_t acc0) {
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              const uint64_t q = desc_add(q0, c * kQChunk + st * 32), b = desc_add(b0, c * kChunk + st * 32);
              mma_pair<kFp8>(dS, q, b, idS, st ? 1u : acc0);
              if (kFp8) mma_pair<kFp8>(dS, desc_add(q, kChunk), b, idS, 1u);
            }
          };
          if (left >= kKFill * 128) {
            if (lead) {
              chunk(0, acc);
              chunk(1, 1u);
              chunk(2, 1u);
            }
          } else {
            for (int c = 0; c < n; ++c) {
              const int steps = min(4, (left - c * 128 + 31) >> 5);
              for (int st = 0; st < steps; ++st) {
                const uint64_t q = desc_add(q0, c * kQChunk + st * 32), b = desc_add(b0, c * kChunk + st * 32);
                if (lead) {
                  mma_pair<kFp8>(dS, q, b, idS, (acc | c | st) != 0);
                  if (kFp8) mma_pair<kFp8>(dS, desc_add(q, kChunk), b, idS, 1u);
                }
              }
            }
          }
          if (lead) {
            commit_pair(BAR(C::bKEmpty + ks.slot));
            if (f == k_fills - 1) {
              commit_pair(BAR(C::bSFull + sn));
              if (flags & kLast) commit_pair(BAR(C::bQEmpty));
            }
          }
          __syncwarp();
          ks.next();
        }
        if (!ok || (flags & kFinal)) break;
      }
      // nothing may still write TMEM when it is released
      if (lead) {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(BAR(C::bDrain))
                     : "memory");
        drain(BAR(C::bDrain), 0);
      }
      __syncwarp();
    }
  } else if (role == 3) {
    // ================================= MMAs of O ==========================================
    if (rank == 0) {
      // (A: P in bf16, or in e5m2)
      const auto idO = [&](int n) { return kFp8 ? idesc_e4m3(128, n, 0, 1) | (1u << 7) : idesc_bf16(128, n, 0, 1); };
      const uint64_t dp = sdesc(sb + C::kPOff, 16, 1024), dv0 = sdesc(sb + C::kVOff, kChunk, 1024);
      const bool lead = elect_one();
      uint32_t units = 0;
#pragma unroll 1
      for (int k = 0;; ++k) {
        const int ri = k % kInfos;
        if (!tree_wait(BAR(C::bInfoFull + ri), (uint32_t)((k / kInfos) & 1), abort_flag)) break;
        const int flags = (int)warp_uniform(*reinterpret_cast<volatile int*>(&infos[ri].flags));
        if (lead) mbar_arrive(BAR(C::bInfoEmpty + ri));
        if (flags & kEnd) break;
        if (!tree_wait(BAR(C::bPReady + (k & 1)), (uint32_t)((k >> 1) & 1), abort_flag)) break;
        const bool first = flags & kFirst;
        // (O of the unit before has been stored)
        if (first && units++ > 0 && !tree_wait(BAR(C::bOFree), units & 1, abort_flag)) break;
        bool ok = true;
#pragma unroll 1
        for (int f = 0; f < 2 * v_fills; ++f) {  // fill f of the tile: of group grp, from chunk c0 on
          if (!(ok = tree_wait(BAR(C::bVReady + vs.slot), vs.parity, abort_flag))) break;
          tc_fence_after();
          const int grp = f >= v_fills, c0 = kVFill * (f - grp * v_fills);
          const uint64_t pa = desc_add(dp, (k & 1) * C::kPBytes + grp * (kFp8 ? 64 : kChunk));
          const uint64_t b = desc_add(dv0, vs.slot * (kVFill * kChunk));
          const uint32_t d = tmem + c0 * C::kCw, acc = !(first && grp == 0);
          if (lead) {
            if (kFp8) {
              // 128 channels of each CTA a chunk
              const auto block = [&](int c) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {          // 32 entries a step
                  const uint64_t pk = desc_add(pa, kk * 32), bk = desc_add(b, c * kChunk + kk * 4096);
                  mma_pair<kFp8>(d + c * 128, pk, bk, idO(256), kk ? 1u : acc);
                  mma_pair<kFp8>(d + c * 128, desc_add(pk, kChunk), bk, idO(256), 1u);
                  mma_pair<kFp8>(d + c * 128, desc_add(pk, 2 * kChunk), bk, idO(256), 1u);
                }
              };
              block(0);
              if (c0 + 1 < n_half) block(1);
            } else {
              // 128 channels of each CTA, or the last 64 of an odd number of chunks
              const uint32_t id = c0 + 1 < n_half ? idO(256) : idO(128);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)              // 16 entries a step
                mma_pair<kFp8>(d, desc_add(pa, kk * 32), desc_add(b, kk * 2048), id, kk ? 1u : acc);
            }
            commit_pair(BAR(C::bVEmpty + vs.slot));
            if (f == 2 * v_fills - 1) commit_pair(BAR(C::bPvDone + (k & 1)));
          }
          __syncwarp();
          vs.next();
        }
        if (!ok || (flags & kFinal)) break;
      }
      if (lead) {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(BAR(C::bDrain + 1))
                     : "memory");
        drain(BAR(C::bDrain + 1), 0);
      }
      __syncwarp();
    }
  } else if (role == 2) {
    // ===================== every fill as it lands: cleaned, handed on =====================
    bool ok = true;
    const auto k_part = [&]() {                  // (cp.async)
#pragma unroll 1
      for (int f = 0; f < k_fills && ok; ++f) {
        if (!(ok = tree_wait(BAR(C::bKFull + ks.slot), ks.parity, abort_flag))) return;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_bar(C::bKReady + ks.slot));
        ks.next();
      }
    };
    const auto v_part = [&](int k) {
      const int ri = k % kInfos;
      const typename C::Info& info = infos[ri];
      const bool clean = info.flags & kClean;
#pragma unroll 1
      for (int f = 0; f < 2 * v_fills; ++f) {
        if (!(ok = tree_wait(BAR(C::bVFull + vs.slot), vs.parity, abort_flag))) return;
        if (clean) {
          const int grp = f >= v_fills, n = min(kVFill, n_half - kVFill * (f - grp * v_fills));
          uint8_t* src = sm + C::kVOff + vs.slot * (kVFill * kChunk);
          const uint32_t lo = info.valid[2 * grp], hi = info.valid[2 * grp + 1];
          const int ctx = max(-info.rel - grp * kGroup, 0);        // the first row that not all may see
          // from the first row that needs it: two a step, a half-warp each, four steps' loads in flight
          const int gone = ~lo ? __ffs(~lo) - 1 : ~hi ? 31 + __ffs(~hi) : kGroup;
          const int c = (lane >> 3) & 1, half = lane >> 4;
          uint4* at_row = reinterpret_cast<uint4*>(src + c * kChunk + half * 128) + (lane & 7);
#pragma unroll 1
          for (int r0 = min(ctx, gone) & ~7; r0 < kGroup; r0 += 8) {
            uint4 old[4];
            const uint32_t exists = (r0 < 32 ? lo >> r0 : hi >> (r0 - 32)) >> half;
#pragma unroll
            for (int z = 0; z < 4; ++z) old[z] = at_row[(r0 + 2 * z) * 8];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint4 now = exists >> (2 * z) & 1u ? finite_only<kFp8>(old[z]) : make_uint4(0, 0, 0, 0);
              if (c < n && (now.x != old[z].x || now.y != old[z].y || now.z != old[z].z || now.w != old[z].w))
                at_row[(r0 + 2 * z) * 8] = now;
            }
          }
        }
        if (clean || !kBox) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_bar(C::bVReady + vs.slot));
        vs.next();
      }
      if (lane == 0) mbar_arrive(BAR(C::bInfoEmpty + ri));
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int ri = k % kInfos;
      if (!tree_wait(BAR(C::bInfoFull + ri), (uint32_t)((k / kInfos) & 1), abort_flag)) break;
      const int flags = *reinterpret_cast<volatile int*>(&infos[ri].flags);
      if (flags & kEnd) break;
      if (!kBox) k_part();
      if (ok) v_part(k);
      if (flags & kFinal) break;
    }
  } else if (role >= 4) {
    // ======= q of every unit; copies of V (role 4) and K (5), or all rows by cp.async =====
    const int tid = threadIdx.x - 32 * (C::kSoftmaxWarps + 4);
    const bool lead = elect_one();
    uint32_t units = 0;
    long long fills = 0;
    bool ok = true;
    // cp.async of a fill: n chunks from c0 on of entry group grp of the tile of info ri
    const auto fill = [&](int ri, int grp, uint32_t dst0, uint32_t full, int c0, int n) {
      const int* rows = reinterpret_cast<const int*>(sm + C::kRowOff) + ri * kTile + grp * kGroup;
      const int jj = tid & 7, r0 = tid >> 3;
      const uint32_t dst = dst0 + r0 * 128 + ((jj ^ (r0 & 7)) << 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = rows[r0 + 16 * i];
        const uint8_t* src = a.pool.rows + (size_t)(row < 0 ? 0 : row) * W;
        for (int c = 0; c < n; ++c) {
          const int col = (c0 + c) * 128 + jj * 16;
          const bool has = row >= 0 && col < W;
          cp_async_16(dst + c * kChunk + i * 2048, has ? src + col : a.pool.rows, has ? 16u : 0u);
        }
      }
      cp_async_arrive_noinc(full);
    };
    // K of a tile: this CTA's 64 entries
    const auto k_part = [&](int ri) {
      const int row = kBox ? infos[ri].boxes[rank * per_group + my_box] : 0;
#pragma unroll 1
      for (int f = 0; f < k_fills; ++f) {
        if (!(ok = tree_wait(BAR(C::bKEmpty + ks.slot), ks.parity ^ 1, abort_flag))) return;
        if (kBox) {
          const uint32_t dst = sb + C::kKOff + ks.slot * (kKFill * kChunk), ready = lead_bar(C::bKReady + ks.slot);
          const int c0 = f * kKFill, n = min(kKFill, n_chunks - c0);
          if (lead && rank == 0) mbar_arrive_expect_tx(BAR(C::bKReady + ks.slot), (uint32_t)(2 * n * kChunk));
          if (p.box == kGroup && (c0 + kKFill) * 128 <= W) {
            if (lead) tma_box3_pair(dst, &p.k_box, 0, row, c0, ready);
          } else if (my_c < n) {
            tma_row_pair(dst + my_off, &p.chunk, (c0 + my_c) * 128, row, ready);
          }
          __syncwarp();
          ++fills;
          ks.next();
          continue;
        }
        fill(ri, rank, sb + C::kKOff + ks.slot * (kKFill * kChunk), BAR(C::bKFull + ks.slot), f * kKFill,
             min(kKFill, n_chunks - f * kKFill));
        ks.next();
      }
    };
    const auto v_part = [&](int k) {
      const int ri = k % kInfos;
      if (!kBox || role == 4) {
#pragma unroll 1
        for (int f = 0; f < 2 * v_fills; ++f) {
          const int grp = f >= v_fills, c = kVFill * (f - grp * v_fills), c0 = rank * n_half + c;
          const int row = kBox ? infos[ri].boxes[grp * per_group + my_box] : 0, n = min(kVFill, n_half - c);
          if (!(ok = tree_wait(BAR(C::bVEmpty + vs.slot), vs.parity ^ 1, abort_flag))) return;
          const uint32_t dst = sb + C::kVOff + vs.slot * (kVFill * kChunk), full = BAR(C::bVFull + vs.slot);
          if (!kBox) {
            fill(ri, grp, dst, full, c0, n);
          } else {
            if (lead) mbar_arrive_expect_tx(full, (uint32_t)(n * kChunk));
            if (p.box == kGroup && n == kVFill && (c0 + kVFill) * 128 <= W) {
              if (lead) tma_box3(dst, &p.v_box, 0, row, c0, full);
            } else if (my_c < n) {
              tma_row(dst + my_off, &p.chunk, (c0 + my_c) * 128, row, full);
            }
            __syncwarp();
            ++fills;
          }
          vs.next();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::bInfoEmpty + ri));
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int ri = k % kInfos;
      if (!tree_wait(BAR(C::bInfoFull + ri), (uint32_t)((k / kInfos) & 1), abort_flag)) break;
      const typename C::Info& info = infos[ri];
      const int flags = info.flags;
      if (flags & kEnd) break;
      const bool first = flags & kFirst;
      if (!kBox || role == 5) k_part(ri);
      if (first && ok) {
        const uint32_t ph = (units & 1) ^ 1;
        ++units;
        if (kFp8 || p.q_box) {
          if (role == 4) {
            ok = tree_wait(BAR(C::bQEmpty), ph, abort_flag);
            if (ok && lead) {
              if (kFp8) {
                const long long slot = q_slot(info.tok0, a.H, info.seq, info.unit_row / kUnitRows);
                const uint32_t bytes = (uint32_t)n_chunks * 2 * kChunk;
                mbar_arrive_expect_tx(BAR(C::bQLocal), bytes + kRows * 4);
                bulk_load(sb + C::kQOff, p.q_codes + (slot * 2 + rank) * bytes, bytes, BAR(C::bQLocal));
                bulk_load(sb + C::kQScaleOff + (units % kQScales) * kRows * 4,
                          p.q_scale + slot * kUnitRows + rank * kRows,
                          kRows * 4, BAR(C::bQLocal));
              } else {
                // (rows behind the unit's last are other tokens' or past the last, then zeros: not stored)
                const int sr = info.unit_row + rank * kRows, h = sr % a.H;
                const int t = p.q_zero ? a.T : info.tok0 + sr / a.H;
                mbar_arrive_expect_tx(BAR(C::bQLocal), (uint32_t)n_chunks * kChunk);
                tma_box4(sb + C::kQOff, &p.q_lat, 0, h, t, 0, BAR(C::bQLocal));
                if (a.pool.R > 0) tma_box3(sb + C::kQOff + (L >> 6) * kChunk, &p.q_rope, 0, h, t, BAR(C::bQLocal));
              }
            }
            __syncwarp();
            if (ok) ok = tree_wait(BAR(C::bQLocal), ph ^ 1, abort_flag);
            if (ok && lane == 0) mbar_arrive_pair(lead_bar(C::bQFull));
          }
        } else {
          const int jj = tid & 7;
          ok = tree_wait(BAR(C::bQEmpty), ph, abort_flag);
          if (ok) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int r = (tid >> 3) + 16 * i, ur = rank * kRows + r;
              const bool has = ur < info.rows && !p.q_zero;
              const int sr = info.unit_row + (has ? ur : 0);
              const long long t = info.tok0 + sr / a.H, h = sr % a.H;
              const uint8_t *ql = a.q_latent + t * a.ql_st + h * a.ql_sh, *qr = a.q_rope + t * a.qr_st + h * a.qr_sh;
              const uint32_t dst = sb + C::kQOff + r * 128 + ((jj ^ (r & 7)) << 4);
              for (int c = 0; c < n_chunks; ++c) {
                const int col = c * 128 + jj * 16;
                const bool in = has && col < W;
                const uint8_t* src = !in ? a.q_latent : (col < 2 * L ? ql + col : qr + (col - 2 * L));
                cp_async_16(dst + c * kChunk, src, in ? 16u : 0u);
              }
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead_bar(C::bQFull));
          }
        }
      }
      if (ok) v_part(k);
      if (flags & kFinal) break;
    }
    cp_async_wait_all();
    // copies in flight must land before the CTA ends (at once after a normal run)
    if (role == 4 && lane == 0) {
      if ((kFp8 || p.q_box) && units > 0) drain(BAR(C::bQLocal), (units - 1) & 1);
      for (long long f = max(0LL, fills - vs.n); f < fills; ++f)
        drain(BAR(C::bVFull + (int)(f % vs.n)), (uint32_t)((f / vs.n) & 1));
    }
    if (role == 5 && lane == 0 && rank == 0)    // (both CTAs' copies of K complete here)
      for (long long f = max(0LL, fills - C::kKSlots); f < fills; ++f)
        drain(BAR(C::bKReady + (int)(f % C::kKSlots)), (uint32_t)((f / C::kKSlots) & 1));
    __syncwarp();
  } else {
    // ================================ softmax and epilogue ================================
    // TMEM lanes 32 quad ..: rows 32 (quad & 1) .., entry group (of S) or channel half (of O) quad >> 1; this
    // warp takes part `ch` of each one's columns
    constexpr int kKeys = C::kKeys, kParts = C::kParts;
    constexpr uint32_t kAll = 0xffffffffu >> (32 - kKeys);
    constexpr int kOCols = 128 / (kParts / 2);   // columns of a 128-channel block of O
    const int quad = warp & 3, ch = warp >> 2, grp = quad >> 1;
    const int row = (quad & 1) * 32 + lane, part = kParts / 2 * grp + ch, e0 = kKeys * part;   // first entry of a tile
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    uint8_t* pb = sm + C::kPOff;
    // this thread's units of P (e4m3: its unit of each term)
    uint8_t* p_at = pb + row * 128 + (kFp8 ? ((part ^ (row & 7)) << 4) : grp * kChunk);
    int* max_at = reinterpret_cast<int*>(sm + C::kMaxOff) + row;
    float m = -INFINITY, l = 0.f;
    uint32_t units = 0, units_next = 0;          // begun, by the tile at hand and by the one after it
    // flags and visible entries (bits) of the tile at hand, and of the one after it
    int flags = 0, flags_next = 0;
    uint32_t seen = 0, seen_next = 0;
    // q's scale for a row of unit u
    const auto row_arg = [&](uint32_t u) {
      return kFp8 ? p.scale_log2 * reinterpret_cast<const float*>(sm + C::kQScaleOff)[(u % kQScales) * kRows + row]
                  : p.scale_log2;
    };
    // Maxima of tile n and weights of tile k, in turn: n runs one ahead of k, but for tiles whose S waits for what may
    // itself wait for P of the tile before: the first of a unit (its q comes after that tile's V), and all without
    // boxes (K comes after it).
    int k = 0, n = 0;
    bool all = false;                            // the last tile's maxima are done
#pragma unroll 1
    for (;;) {
      if (!all) {
        // ---- maxima of tile n ----
        const int ri = n % kInfos;
        if (!tree_wait(BAR(C::bInfoFull + ri), (uint32_t)((n / kInfos) & 1), abort_flag)) break;
        const typename C::Info& info = infos[ri];
        flags_next = info.flags;
        if (flags_next & kEnd) break;
        if (n == k || (kBox && !(flags_next & kFirst))) {
          if (flags_next & kFirst) ++units_next;
          seen_next = info.valid[e0 >> 5] >> (e0 & 31) & kAll;
          const int rel = info.rel + e0;
          if (rel > -kKeys) {
            // drafted tokens among entries e0 ..: by the mask of this row's token
            const int ur = rank * kRows + row;
            uint32_t bits = 0;
            if (ur < info.rows) {
              const int i = (info.unit_row + ur) / a.H;            // the row's drafted token
              if (a.mask) {
                const uint32_t* mk = a.mask + (size_t)(info.tok0 + i) * a.mask_words;
                const int at = rel < 0 ? 0 : rel >> 5;
                const uint32_t w0 = at < a.mask_words ? __ldg(mk + at) : 0u;
                if (rel < 0) bits = (w0 << -rel) | ((1u << -rel) - 1u);
                else {
                  const uint32_t w1 = at + 1 < a.mask_words ? __ldg(mk + at + 1) : 0u;
                  bits = __funnelshift_r(w0, w1, rel & 31);
                }
              } else {
                const int c = i - rel + 1;                         // entries up to token i's
                bits = c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
              }
            }
            seen_next &= bits;
          }
          if (!tree_wait(BAR(C::bSFull + n % kSBufs), (uint32_t)((n / kSBufs) & 1), abort_flag)) break;
          __syncwarp();
          tc_fence_after();
          float x[kKeys];
          tmem_ld(lanes + kSCol + (n % kSBufs) * 64 + kKeys * ch, x);
          tmem_wait_ld();
          const float arg = row_arg(units_next);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if constexpr (kFp8) {
            // of the weights that enter the value product, p_j scale_j
            const float4* ks = reinterpret_cast<const float4*>(info.scale + e0);
            const float4* ls = reinterpret_cast<const float4*>(info.lscale + e0);
#pragma unroll
            for (int j = 0; j < kKeys / 4; ++j) {
              const float4 c = ks[j], d = ls[j];
              const float cs[4] = {c.x, c.y, c.z, c.w}, ds[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float z = fmaf(arg, x[4 * j + e] * cs[e], ds[e]);
                mx[e] = fmaxf(mx[e], (seen_next >> (4 * j + e)) & 1u ? z : -INFINITY);
              }
            }
          } else {
            if (seen_next != kAll) {
#pragma unroll
              for (int j = 0; j < kKeys; ++j) x[j] = (seen_next >> j) & 1u ? x[j] : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < kKeys; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // The place for tile n + 2 is cleared: that of tile n - 6, whose maxima everybody has read, as the value
          // products of tile n - 4 were waited for at tile n - 2; who writes there has waited for tile n.  (Two
          // barriers: a warp is here for tile n + 1 after it has waited for tile n, but before others have.)
          if (part == 0) max_at[(n + 2) % kMaxTiles * kRows] = ordered(__float_as_int(-INFINITY));
          atomicMax(max_at + n % kMaxTiles * kRows, ordered(__float_as_int(kFp8 ? mt : mt * arg)));   // (bf16: arg > 0)
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(C::bMax + (n & 1)));
          __syncwarp();
          ++n;
          all = flags_next & kFinal;
          if (n == k + 1) {
            flags = flags_next;
            seen = seen_next;
            units = units_next;
            continue;
          }
        }
      }
      // ---- weights of tile k ----
      const int ri = k % kInfos;
      const typename C::Info& info = infos[ri];
      const bool first = flags & kFirst;
      if (first) {
        m = -INFINITY;
        l = 0.f;
      }
      float x[kKeys];
      tmem_ld(lanes + kSCol + (k % kSBufs) * 64 + kKeys * ch, x);
      if (!tree_wait(BAR(C::bMax + (k & 1)), (uint32_t)((k >> 1) & 1), abort_flag)) break;
      const float mt = __int_as_float(ordered(*reinterpret_cast<volatile int*>(max_at + k % kMaxTiles * kRows)));
      // lazy: the reference moves only where it is exceeded by more than tau
      float al = 1.f;
      if (mt > m + C::kTau) {
        al = fast_exp2(m - mt);
        l *= al;
        m = mt;
      }
      const bool grow = __any_sync(0xffffffffu, al != 1.f);
      __syncwarp();
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(lead_bar(C::bSEmpty + k % kSBufs));
      // (a row without any entry so far: everything is masked, the reference does not matter)
      const float arg = row_arg(units), ref = m == -INFINITY ? 0.f : m;
      if constexpr (kFp8) {
        const float4* ks = reinterpret_cast<const float4*>(info.scale + e0);
#pragma unroll
        for (int j = 0; j < kKeys / 4; ++j) {
          const float4 c = ks[j];
          const float cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[4 * j + e] = (seen >> (4 * j + e)) & 1u ? fast_exp2(fmaf(arg, x[4 * j + e] * cs[e], -ref)) : 0.f;
        }
      } else {
        if (seen != kAll) {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) x[j] = (seen >> j) & 1u ? x[j] : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kKeys; j += 2) {
          fma_f32x2(x[j], x[j + 1], arg, -ref);
          x[j] = fast_exp2(x[j]);
          x[j + 1] = fast_exp2(x[j + 1]);
        }
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kKeys; j += 2) add_f32x2(sum[j & 2], sum[(j & 2) + 1], x[j], x[j + 1]);
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // P in registers: 16-byte units of eight entries, or (e4m3) of sixteen for each term
      constexpr int kUnits = kFp8 ? 3 : kKeys / 8;
      uint4 pu[kUnits];
      if constexpr (kFp8) {
        // u = kPUnit p scale in f16 as three e5m2 terms, each the nearest to what is left
        const float4* ks = reinterpret_cast<const float4*>(info.scale + e0);
        const auto upper = [](uint32_t f16x2) { return (f16x2 + 0x00800080u) & 0xff00ff00u; };
        uint32_t w[3][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 c = ks[q];
          const float* e = x + 4 * q;
          // (a weight of zero stays one, whatever the scale of a row that is not seen)
          const float f[4] = {e[0] == 0.f ? 0.f : e[0] * c.x, e[1] == 0.f ? 0.f : e[1] * c.y,
                              e[2] == 0.f ? 0.f : e[2] * c.z, e[3] == 0.f ? 0.f : e[3] * c.w};
          uint32_t t[3][2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            __half2 y = __floats2half2_rn(f[2 * z], f[2 * z + 1]);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              t[i][z] = upper(*reinterpret_cast<const uint32_t*>(&y));
              if (i < 2) y = __hsub2(y, *reinterpret_cast<const __half2*>(&t[i][z]));
            }
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) w[i][q] = __byte_perm(t[i][0], t[i][1], 0x7531);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) pu[i] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
      } else {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const float* e = x + 8 * u;
          pu[u] = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                             pack_bf16x2(e[6], e[7]));
        }
      }
      // the products of the tile before the last have read P
      if (k > 1 && !tree_wait(BAR(C::bPvDone + (k & 1)), (uint32_t)(((k >> 1) & 1) ^ 1), abort_flag)) break;
      if (grow && !first) {
        // (and those of the last have added to O)
        if (!tree_wait(BAR(C::bPvDone + ((k - 1) & 1)), (uint32_t)(((k - 1) >> 1) & 1), abort_flag)) break;
        __syncwarp();
        tc_fence_after();
        const int n_mt = (n_half * C::kCw + 127) / 128;
#pragma unroll 1
        for (int c = 0; c < n_mt * kOCols / 32; ++c) {           // 32 columns a time of a 128-channel block
          const uint32_t at = lanes + c / (kOCols / 32) * 128 + kOCols * ch + c % (kOCols / 32) * 32;
          float o[32];
          tmem_ld32(at, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= al;
          tmem_st32(at, o);
        }
        tmem_wait_st();
        tc_fence_before();
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        *reinterpret_cast<uint4*>(p_at + (k & 1) * C::kPBytes +
                                  (kFp8 ? u * kChunk : ((kUnits * ch + u) ^ (row & 7)) << 4)) = pu[u];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(lead_bar(C::bPReady + (k & 1)));
      int slot = 0, n_rows = 0, first_row = 0;
      if (flags & kLast) slot = info.slot, n_rows = info.rows, first_row = info.first_row;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::bInfoEmpty + ri));
      if (flags & kLast) {
        // ---- epilogue: denominators, then O ----
        if (!tree_wait(BAR(C::bPvDone + (k & 1)), (uint32_t)((k >> 1) & 1), abort_flag)) break;
        // The parts' sums, in P's place: its products are done, and whoever goes on waits until everybody has read them.
        const auto sums = [&](int e) { return reinterpret_cast<float*>(pb + (k & 1) * C::kPBytes) + e * kRows; };
        sums(part)[row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::bLFull));
        if (!tree_wait(BAR(C::bLFull), (units - 1) & 1, abort_flag)) break;
        float ls = 0.f;
#pragma unroll
        for (int e = 0; e < kParts; ++e) ls += sums(e)[row];
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::bLEmpty));
        // (0: no entry at all.  A NaN among the scores is in the sum, whatever the maximum is.)
        const float inv = ls == 0.f ? 0.f : (kFp8 ? 1.f / kPUnit : 1.f) / ls;
        const int ur = rank * kRows + row;
        const size_t prow = ((size_t)slice * 2 + (slot > 0 ? 1 : 0)) * kUnitRows + ur;
        if (slot >= 0 && part == 0) p.lse[prow] = ls == 0.f ? -INFINITY : m + __log2f(ls);
        __syncwarp();
        tc_fence_after();
        const int n_mt = (n_half * C::kCw + 127) / 128;
#pragma unroll 1
        for (int c = 0; c < n_mt * kOCols / 32; ++c) {
          const int block = c / (kOCols / 32), col = kOCols * ch + c % (kOCols / 32) * 32;
          const int d = grp * n_half * C::kCw + block * 128 + col;
          // (bf16: the last block of an odd number of chunks is one chunk wide)
          const bool there = (kFp8 || 2 * block + 1 < n_half || col < 64) && d < L;
          float o[32];
          tmem_ld32(lanes + block * 128 + col, o);
          tmem_wait_ld();
          // (d and L are multiples of 32: all 32 channels exist.)  A lane's sixteen bytes at a time would touch 32 rows a
          // store; of four lanes' units transposed, a store has 64 bytes of each of eight rows.
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          const int u0 = rank * kRows + (row & ~3), unit = lane & 3;
          const size_t prow0 = ((size_t)slice * 2 + (slot > 0 ? 1 : 0)) * kUnitRows + u0;
          if (slot >= 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 u[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = make_uint4(__float_as_uint(o[16 * h + 4 * e]), __float_as_uint(o[16 * h + 4 * e + 1]),
                                  __float_as_uint(o[16 * h + 4 * e + 2]), __float_as_uint(o[16 * h + 4 * e + 3]));
              transpose4(u);
              uint4* dst = reinterpret_cast<uint4*>(p.part + prow0 * L + d + 16 * h) + unit;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (there && u0 + e < n_rows) dst[(size_t)e * (L / 4)] = u[e];
            }
          } else {
            uint4 u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
            transpose4(u);
            uint4* dst = reinterpret_cast<uint4*>(a.out + (((size_t)first_row + u0) * L + d) * 2) + unit;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (there && u0 + e < n_rows) dst[(size_t)e * (L / 8)] = u[e];
          }
          __syncwarp();                          // (the loads from TMEM are the whole warp's)
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_bar(C::bOFree));
        if (!tree_wait(BAR(C::bLEmpty), (units - 1) & 1, abort_flag)) break;
      }
      if (flags & kFinal) break;
      ++k;                                       // (where n is k now, the next trip sets these)
      flags = flags_next;
      seen = seen_next;
      units = units_next;
    }
  }
#undef BAR
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (role == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the parts of the units that were cut: out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M), in the
// order of the slices.  A warp takes 128 channels of a row, eight parts in flight.  The 32 drafts above: 19 us alone
// (27 while a row's item was looked for one by one, each step a load that waits for the last), one draft 9.  Four
// CTAs an SM: with 6, 8 or 12 the call takes 1 to 2 us more.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const Part* __restrict__ cut, const float* __restrict__ lse, const float* __restrict__ part,
                      __nv_bfloat16* __restrict__ out, int slices, int L) {
  __shared__ int4 item[kMaxSlices];       // row, slice, last slice, rows of the items up to and with this one
  __shared__ int n_items;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nq = (L + 127) >> 7;
  pdl_wait();
  if (warp == 0) {
    int n = 0, rows = 0;
    for (int s0 = 0; s0 < slices; s0 += 32) {
      Part c = {0, 0, -1, 0};
      if (s0 + lane < slices) c = cut[s0 + lane];
      const unsigned m = __ballot_sync(0xffffffffu, c.last >= 0);
      int scan = c.last >= 0 ? c.rows : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
      }
      if (c.last >= 0) item[n + __popc(m & ((1u << lane) - 1u))] = make_int4(c.row, s0 + lane, c.last, rows + scan);
      n += __popc(m);
      rows += __shfl_sync(0xffffffffu, scan, 31);
    }
    if (lane == 0) n_items = n;
  }
  __syncthreads();
  if (n_items == 0) return;
  const int work = item[n_items - 1].w * nq;
  for (int u = blockIdx.x * kMergeWarps + warp; u < work; u += gridDim.x * kMergeWarps) {
    const int r_all = u / nq, d = (u % nq) * 128 + 4 * lane;
    int i = 0;                               // items that end before the row (their ends never fall)
    for (int b = 0; b < n_items; b += 32)
      i += __popc(__ballot_sync(0xffffffffu, b + lane < n_items && item[b + lane].w <= r_all));
    const int4 it = item[i];
    const int r = r_all - (i ? item[i - 1].w : 0), n = it.z - it.y + 1;
    const auto at = [&](int s) { return ((size_t)(it.y + s) * 2 + (s == 0 ? 1 : 0)) * kUnitRows + r; };
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, tot = 0.f;
    for (int s0 = 0; s0 < n; s0 += 8) {
      float e[8];
      float4 v[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        e[z] = -INFINITY;
        v[z] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 + z < n) {
          e[z] = lse[at(s0 + z)];
          if (d < L) v[z] = *reinterpret_cast<const float4*>(part + at(s0 + z) * L + d);
        }
      }
      float mx = M;
#pragma unroll
      for (int z = 0; z < 8; ++z) mx = fmaxf(mx, e[z]);
      // (a NaN among the parts' sums is not seen by the maximum but comes back in its weight)
      const float ref = mx == -INFINITY ? 0.f : mx, f = exp2f(M - ref);
      M = mx;
      tot *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const float w = exp2f(e[z] - ref);
        tot += w;
        acc.x = fmaf(w, v[z].x, acc.x);
        acc.y = fmaf(w, v[z].y, acc.y);
        acc.z = fmaf(w, v[z].z, acc.z);
        acc.w = fmaf(w, v[z].w, acc.w);
      }
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    if (d < L)
      *reinterpret_cast<uint2*>(out + ((size_t)it.x + r) * L + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int slices_of(int sms) { return sms / 2 < 1 ? 1 : sms / 2 > kMaxSlices ? kMaxSlices : sms / 2; }

struct Workspace {
  size_t cut, lse, part, codes, scale, bytes;
};
Workspace workspace_layout(const LatentTreeArgs& a, bool fp8, int sms) {
  const size_t slots = (size_t)slices_of(sms) * 2 * kUnitRows;
  Workspace w;
  w.cut = 0;
  w.lse = align256(slices_of(sms) * sizeof(Part));
  w.part = w.lse + align256(slots * sizeof(float));
  w.codes = align256(w.part + slots * (size_t)a.pool.L * sizeof(float));
  const size_t units = fp8 ? (size_t)((long long)a.T * a.H / kUnitRows + a.pool.B + 1) : 0;
  w.scale = w.codes + units * 2 * ((a.pool.L + 2 * a.pool.R + 127) / 128) * 2 * kChunk;
  w.bytes = w.scale + units * kUnitRows * sizeof(float);
  return w;
}

template <bool kFp8>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  using C = Cfg<kFp8>;
  // (e4m3: a dependent of tree_q_kernel, launched right before)
  return launch_with_pdl(p.box ? latent_tree_kernel<kFp8, true> : latent_tree_kernel<kFp8, false>, dim3(2 * p.slices),
                         dim3(C::kThreads), C::kSmem, stream, kFp8, p);
}

}  // namespace

cudaError_t prepare_latent_tree() {
  const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(latent_tree_kernel<false, true>, most, Cfg<false>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_tree_kernel<false, false>, most, Cfg<false>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_tree_kernel<true, true>, most, Cfg<true>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_tree_kernel<true, false>, most, Cfg<true>::kSmem);
  return e;
}

size_t latent_tree_workspace(const LatentTreeArgs& a, bool fp8, int sms) {
  return workspace_layout(a, fp8, sms).bytes;
}

cudaError_t launch_latent_tree(const LatentTreeArgs& a, bool fp8, void* workspace, int sms, cudaStream_t stream) {
  TreeParams p = {};
  p.a = a;
  p.slices = slices_of(sms);
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;
  p.negate = a.scale < 0.f;
  p.q_zero = !fp8 && p.scale_log2 == 0.f;
  if (p.q_zero) p.scale_log2 = 1.f;
  const Workspace w = workspace_layout(a, fp8, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cut = reinterpret_cast<Part*>(ws + w.cut);
  p.lse = reinterpret_cast<float*>(ws + w.lse);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.q_codes = ws + w.codes;
  p.q_scale = reinterpret_cast<float*>(ws + w.scale);
  // Pages of a multiple of eight entries: boxes of as many rows as divide the page (at most a fill's 64).
  p.box = 0;
  for (int b = 8; b <= kGroup; b *= 2)
    if (a.pool.ps % b == 0) p.box = b;
  if (p.box) {
    const unsigned long long W = a.pool.row_bytes;
    const unsigned long long d[2] = {W, (unsigned long long)(a.pool.num_blocks * a.pool.ps)}, st[1] = {W};
    const unsigned bx[2] = {128, (unsigned)p.box};
    if (!encode_bytes(&p.chunk, a.pool.rows, 2, d, st, bx)) return cudaErrorInvalidValue;
    while (1 << p.box_shift < p.box) ++p.box_shift;
    if (p.box == kGroup && W >= 128) {
      const unsigned long long d3[3] = {128, d[1], W / 128}, st3[2] = {W, 128};
      const unsigned kb[3] = {128, kGroup, kKFill}, vb[3] = {128, kGroup, kVFill};
      if (!encode_bytes(&p.k_box, a.pool.rows, 3, d3, st3, kb) || !encode_bytes(&p.v_box, a.pool.rows, 3, d3, st3, vb))
        return cudaErrorInvalidValue;
    }
  }
  // bf16 q by tensor maps, where 64 rows are whole tokens or part of one (else by cp.async).
  if (!fp8 && (a.H % kRows == 0 || kRows % a.H == 0)) {
    p.q_box = 1;
    const unsigned hb = a.H < kRows ? (unsigned)a.H : (unsigned)kRows, tb = kRows / hb;
    const auto stride = [](long long n, long long s, long long other) {
      return (unsigned long long)(n > 1 ? s : other);
    };
    const unsigned long long H = a.H, T = a.T;
    const unsigned long long lh = stride(a.H, a.ql_sh, 2LL * a.pool.L), rh = stride(a.H, a.qr_sh, 2LL * a.pool.R);
    const unsigned long long d[4] = {128, H, T, (unsigned long long)(a.pool.L / 64)};
    const unsigned long long st[3] = {lh, stride(a.T, a.ql_st, lh * H), 128};
    const unsigned bx[4] = {128, hb, tb, (unsigned)(a.pool.L / 64)};
    if (!encode_bytes(&p.q_lat, a.q_latent, 4, d, st, bx)) return cudaErrorInvalidValue;
    if (a.pool.R > 0) {
      const unsigned long long dr[3] = {2ull * a.pool.R, H, T}, sr[2] = {rh, stride(a.T, a.qr_st, rh * H)};
      const unsigned br[3] = {128, hb, tb};
      if (!encode_bytes(&p.q_rope, a.q_rope, 3, dr, sr, br)) return cudaErrorInvalidValue;
    }
  }
  const long long rows = (long long)a.T * a.H;
  cudaError_t e = cudaSuccess;
  if (fp8) {
    const long long blocks = (rows + 7) / 8;
    e = launch_with_pdl(tree_q_kernel, dim3((unsigned)(blocks < 8LL * sms ? blocks : 8LL * sms)), dim3(256), 0, stream,
                        false, a, p.q_codes, p.q_scale);
    if (e != cudaSuccess) return e;
  }
  if (fp8) e = launch_tree<true>(p, stream);
  else e = launch_tree<false>(p, stream);
  if (e != cudaSuccess) return e;
  const long long units = (rows * ((a.pool.L + 127) / 128) + kMergeWarps - 1) / kMergeWarps;
  const unsigned merge_blocks = (unsigned)(units < 4LL * sms ? units : 4LL * sms);
  return launch_with_pdl(tree_merge_kernel, dim3(merge_blocks), dim3(32 * kMergeWarps),
                         0, stream, true, (const Part*)p.cut, (const float*)p.lse, (const float*)p.part,
                         reinterpret_cast<__nv_bfloat16*>(a.out), p.slices, a.pool.L);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t latent_tree_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
