// spa_latent_decode.cu - absorbed latent attention over the paged cache: every head of a query
// attends to the same rows x_j = [c_j | r_j], which are its keys and (their latent part) its values.
//
//   s_j = scale (q_c . c_j + q_r . r_j),   out = sum_j softmax(s)_j c_j,   j <= position
//
// A row serves 64 heads of a token once it is in shared memory: 2 (2L + R) flops a head and row, so 64 heads
// do about 121 flops a byte of a bf16 row (L = 512, R = 64) and 128 heads 242, where the machine
// turns from HBM-bound to tensor-bound.  (More heads copy it again for every 64, and so does every further
// token of its sequence: from L2, or from HBM where other rows have come between.)  Both limits matter, so the
// products run on the tcgen05 tensor cores from one copy of the row, in tiles of 64 entries and 64 heads:
//
//   S[h][j]   = q_h . x_j           bf16: M = 128 stacks the two halves of the latent dimension,
//                                   [q_h first half; q_h second half] against [rows' first half;
//                                   rows' second half] with N = 128, and the two diagonal blocks
//                                   add up to S (an MMA of M = 64 runs at half the rate of M = 128:
//                                   measured 46 cycles for N = 64, and 64 for M = N = 128).
//                                   e4m3: M = 128 stacks q_hi over q_lo, the blocks add up likewise.
//   O^T[d][h] += c_j[d] P[h][j]     M = 128 latent channels, N = 64 heads, K = 64 entries: A = the
//                                   same rows read MN-major, B = P.
//
// bf16 queries sit in TMEM (the A operand of S), which leaves shared memory for three tiles of rows:
// one is loaded, one multiplied, one waits for its softmax.  P takes the place of its own tile's
// rotary chunk, which nobody reads any more.  TMEM: O^T 256 columns, S 128, q 128.  (e4m3 queries stay
// in shared memory: there is room, and TMEM then has two S buffers, which measured faster, 194 us
// against 217 for the 48 sequences below at the time.)
//
// What bounds a tile is shared memory's 128 bytes a cycle as much as the tensor core (bf16, L = 512,
// R = 64: the MMAs read 184 KB, the copy writes 74, the softmax moves 40: 2,330 cycles, against 2,090
// of the MMAs alone).
//
//   warps 0-7   softmax: a thread has one head and a quarter of a tile's entries; it adds the other
//               stacked block's part of S (through shared memory), then maximum and sum are in
//               registers; epilogue.  (With four warps, half a tile a thread, the softmax took longer
//               than the tile's MMAs.)
//   warps 8-11  the next token's q: into TMEM (bf16), or (e4m3) a copy of the codes that latent_q_kernel
//               made of it; and the rows by cp.async where a tile is not one box of a page
//   warp 12     issues the MMAs of S, warp 14 those of O: two warps, so that neither one's waits keep
//               the tensor core idle while the other has work
//   warp 13     schedule and page tables, two tiles ahead; tensor-map copies (pages of a multiple of 64
//               entries: a tile is then one box of rows by 128-byte chunks, a single copy)
//
// Schedule: the tiles of all tokens are one long line, each token with a few tiles' room for what it costs
// beside them (its q, its epilogue); each slice of CTAs (one CTA for every 64 heads) takes an equal
// stretch of it.  So the work is balanced whatever the sequence lengths, without knowing them on the
// host.  A token whose tiles lie in one slice is finished there;
// the parts of a token that was cut go to the workspace, normalised, with their log-sum-exp, and
// latent_merge_kernel joins them in the order of the slices.
//
// e4m3 rows enter the MMAs as codes.  q becomes q_hi + q_lo (e4m3, times a power of two per head);
// the row's scale multiplies the score.  The weights p_j scale_j enter as f16 numbers cut into three e5m2
// terms, each the nearest to what the terms before it leave, in a unit that puts the largest weight of the
// sequence so far between 2^10 and 2^15 (the last binade but one of e5m2).  So a weight is off
//   by 2^-11 of itself at most (f16's rounding: the terms lose nothing more), or, below about 2^-16 of
//   the largest, by 2^-17 of the unit, 2^-27 of the largest.
// Small weights matter as much as large ones: 100,000 entries at 2^-13 of the largest outweigh it.  With an
// e5m2 and an e4m3 term (ten bits less of range; 128 us for the 48 sequences below where this takes 138) the
// weights of such a tail were off by up to 11%.  A reference that may be exceeded by 2^4, 2^5 or 2^6 before O is rescaled took
// 141, 138 and 138 us.  A row of zeros, whose stored scale is 1, would raise the reference by the seven or
// so bits that this is above other rows': its scale counts as 0 here (its score is 0 and so are its values).
//
// Measured (L = 512, R = 64, calls one after the other, inputs larger than L2):
//   64 sequences of up to 16,004 entries, 128 heads, bf16: 182 us (797 TFLOP/s, 42% of the measured bf16
//     rate; 3.4 TB/s), some 10 of them the merge; 107 tiles a CTA, tensor cores active 55% of the kernel
//   48 sequences of up to 11,581 entries, 2 tokens each, 64 heads, e4m3: 138 us; 63 tiles a CTA, tensor cores
//     active 36%: of about 3,900 cycles a tile, everything counted, 2,110 are its 44 MMAs; the softmax warps'
//     parts (swap, maxima, exponentials, the three terms of P) follow one after the other
//   one sequence of 131,071 entries, 16 heads, e4m3: 39 us; one of 4,097, 64 heads, bf16: 22.5 us, of which
//     about 5 are the way to the first product, 3 the parts' stores and 8 the merge, its launch included
// Figures of variants, each against the kernel of its time:
//   The loops that issue MMAs are kept short (no predicates in the whole chunks, not unrolled across them): 145,
//   184 and 44 us became 131, 179 and 40.
//   Tried and slower: a softmax of two groups of four warps on alternate e4m3 tiles (181 us against 153: the
//   code twice as long costs more in instruction fetches than the overlap gives), a prefetch of the next tile
//   into L2, a separate warp for copies, S waiting on half tiles, the next tile's S read under the sum of this
//   one's weights (190 and 147 us against 183 and 143), longer and shorter polls; and, no faster, e4m3's
//   swap in one round.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_errors.h"
#include "spa_latent.h"
#include "spa_latent_ring.h"
#include "spa_launch.h"

namespace spa {

namespace {

constexpr int kHeads = 64;        // heads of a CTA
constexpr int kKeys = 64;         // entries of a tile
constexpr int kChunkBytes = kKeys * 128;
constexpr int kBufs = LatentTileRing::kSlots;   // tiles of rows in shared memory
constexpr int kRing = 4;          // tile infos in flight
constexpr int kTmemCols = 512;
constexpr int kSCol = 256, kQCol = 384;   // TMEM columns: O^T from 0, S, q
constexpr int kSoftmax = 256;     // threads of the softmax warps
constexpr int kThreads = kSoftmax + 224;
constexpr int kMinTiles = 2;      // tiles of a slice at least: fewer would cost more in merging
constexpr int kTokenCost = 6;     // what a token costs its CTA beside its tiles, in tiles (measured: 0 took 190
                                  // and 150 us where 6 took 183 and 144)

// e4m3: the unit of the weights, and how far (log2) one may exceed the reference before O is rescaled.  Their
// product is 2^15, so that a weight rounds to an e5m2 number.
constexpr float kPUnit = 1024.f;
constexpr float kTau8 = 5.f;

// first and last tile of this CTA's part of a token, its last tile of all, no tile at all
enum { kFirst = 1, kLast = 2, kFinal = 4, kEnd = 8 };

template <bool kFp8>
struct Cfg {
  static constexpr int kSlots = kFp8 ? 5 : 9;        // 128-byte chunks of a row
  static constexpr int kPerTile = kFp8 ? 1 : 2;      // slots of 128 channels
  static constexpr int kBufBytes = kSlots * kChunkBytes;
  static constexpr int kSBufs = kFp8 ? 2 : 1;        // S buffers in TMEM (64 or 128 columns)
  static constexpr float kTau = kFp8 ? kTau8 : 8.f;    // lazy rescale threshold (log2 units)
  struct Info {
    int t, flags, slot, pad;
    uint32_t valid[2];                               // bit j: entry j (32 + j) takes part
    uint32_t pad2[2];
    int row[kKeys];                                  // pool rows (-1: none), for cp.async
    float scale[kFp8 ? kKeys : 4];                   // the rows' scales, and log2 of them
    float lscale[kFp8 ? kKeys : 4];
  };
  // q first: bf16 has its rotary chunk there (64 rows; the MMA reads 128, the rest is ignored)
  static constexpr int kQBytes = kFp8 ? 5 * 16384 : 8192;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQBytes;
  // P's first 8 KB take the place of the tile's last slot (e4m3: the first two terms); e4m3's third term
  // has a place of its own for each buffer
  static constexpr int kPOff = kKOff + kBufs * kBufBytes;
  static constexpr int kRedOff = kPOff + (kFp8 ? kBufs * 4096 : 0);  // float [4][64], e4m3 two of them
  static constexpr int kQScaleOff = kRedOff + (kFp8 ? 2 : 1) * 4 * kHeads * 4;    // e4m3: float [4][64]
  static constexpr int kInfoOff = kQScaleOff + (kFp8 ? 4 * kHeads * 4 : 0);
  static constexpr int kBarOff = kInfoOff + kRing * (int)sizeof(Info);
  // Barriers (each in its own word; those of one kind side by side).  EMPTY of a tile's buffer, completed
  // by the MMAs of O that read it, is also what the softmax warps wait for before they touch O.  Every wait
  // by parity is at most one phase from its barrier, whatever the warps' pace:
  //   FULL, EMPTY, P-ready, by tile k modulo three: S of tile k needs FULL of its buffer, whose copy
  //     waited for EMPTY of tile k - 3, and that for P-ready of tile k - 3.  So whoever has S of tile k
  //     finds EMPTY and P-ready of its slot at phase k / 3, and those of tiles k - 1 and k - 2 no more
  //     than one phase from theirs; and none of them goes on to tile k + 3 before P of tile k.
  //   S full, S free: S of tile k waits for the softmax to have read the S before it in that buffer.
  //   q full, q free, O free: completed once a token, each by the side that waits for the other.
  //   info full, info free: all fourteen readers arrive before a slot is written again.
  static constexpr int kFullB = 0, kEmptyB = kFullB + kBufs, kQFullB = kEmptyB + kBufs,
                       kQEmptyB = kQFullB + 1, kSFullB = kQEmptyB + 1, kSEmptyB = kSFullB + 2,
                       kPFullB = kSEmptyB + 2, kOFreeB = kPFullB + kBufs, kInfoFullB = kOFreeB + 1,
                       kInfoEmptyB = kInfoFullB + kRing, kDrainB = kInfoEmptyB + kRing,
                       kTokenB = kDrainB + 2, kNumB = kTokenB + 1;
  static constexpr int kMiscOff = kBarOff + kNumB * 8;   // TMEM base, abort flag, first token
  static constexpr int kSmem = kMiscOff + 12;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct DecodeParams {
  // With `boxed`: the pool's 128-byte chunks of 64 rows, one chunk a box; and the first `whole` slots of
  // 64 rows in one box (0: none).
  CUtensorMap chunk, block;
  LatentDecodeArgs a;
  int boxed, whole;
  int groups;                  // of 64 heads
  int slices;
  float scale_log2;
  int2* cut;                   // [slices * groups]: the token cut at the end of a slice, its last slice
  float* lse;                  // [slices * groups][2][64], log2 units
  float* part;                 // [slices * groups][2][64][L]
  uint8_t* q_codes;            // e4m3: [T * groups][chunks][64 rows of the high term, 64 of the low][128]
  float* q_scale;              // e4m3: [T * groups][64], 1 / kPUnit over the power of two in the codes
};

__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kKeys - 1) / kKeys : 1; }

// Entries of a token (0 for one that attends to nothing) at position `pos` of sequence b.
__device__ __forceinline__ int token_len(const LatentDecodeArgs& a, int pos, int b, bool& bad) {
  long long cap = (long long)a.pool.bt_stride * a.pool.ps;
  cap = cap < 0x7fffffc0LL ? cap : 0x7fffffc0LL;   // (a tile's entries stay below 2^31)
  bad = b < 0 || b >= a.pool.B || (long long)pos >= cap;
  if (b < 0 || b >= a.pool.B || pos < 0) return 0;
  return (int)((long long)pos + 1 < cap ? (long long)pos + 1 : cap);
}

// e4m3: q as two e4m3 terms times a power of two per head, in the order of the MMA's operand in shared
// memory (a chunk of 128 columns: 64 rows of the high term, 64 of the low, swizzled), once a token
// instead of once in every CTA that takes part in it (which measured 18,000 cycles before the first
// product, the code being cold and its conversions slow).  A warp takes a head; the last R columns
// repeat the rotary part, against the low codes of the rows.
__global__ void __launch_bounds__(256)
    latent_q_kernel(const __grid_constant__ LatentDecodeArgs a, int groups, uint8_t* __restrict__ codes,
                    float* __restrict__ scales) {
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nlp = a.pool.L >> 3, nrp = a.pool.R >> 3, n_chunks = (a.pool.row_bytes + 127) >> 7;
  const long long units = (long long)a.T * groups * (kHeads / 8);
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long tg = u / (kHeads / 8), t = tg / groups;
    const int h = (int)(u % (kHeads / 8)) * 8 + warp, hg = (int)(tg % groups) * kHeads + h;
    const uint4* ql = reinterpret_cast<const uint4*>(a.q_latent + t * a.ql_st + hg * a.ql_sh);
    const uint4* qr = reinterpret_cast<const uint4*>(a.q_rope + t * a.qr_st + hg * a.qr_sh);
    uint4 x[3];                                // pieces of eight values
    uint32_t mb = 0;                           // largest magnitude (NaN if there is one)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int o = lane + 32 * i, r = o - nlp;
      x[i] = make_uint4(0, 0, 0, 0);
      if (hg < a.H && r < 2 * nrp) x[i] = r < 0 ? __ldg(ql + o) : __ldg(qr + (r < nrp ? r : r - nrp));
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mb = max(mb, w[e] & 0x7fffu);          // (bf16's bits order as their magnitudes do)
        mb = max(mb, (w[e] >> 16) & 0x7fffu);
      }
    }
    mb = __reduce_max_sync(0xffffffffu, mb);
    const float m = bf16_lo(mb);
    const bool finite = mb < 0x7f80u;          // (else the head's scores become NaN through its scale)
    const float qs = finite && m > 0.f ? pow2_floor(448.f / m) : 1.f;
    if (lane == 0) scales[tg * kHeads + h] = finite ? (1.f / kPUnit) / qs : __int_as_float(0x7fffffff);
    // piece o: chunk o / 16, 16-byte unit (o / 2) & 7 of the row
    uint8_t* dst = codes + tg * ((long long)n_chunks * 16384) + h * 128;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int o = lane + 32 * i;
      if (o >= 16 * n_chunks) continue;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = bf16_lo(w[e]) * qs, z = bf16_hi(w[e]) * qs;
        hi[e] = e4m3x2(y, z);
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[e], __NV_E4M3);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        lo[e] = e4m3x2(y - v.x, z - v.y);
      }
      uint8_t* d = dst + (o >> 4) * 16384 + ((((o >> 1) & 7) ^ (h & 7)) << 4) + (o & 1) * 8;
      *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2*>(d + 8192) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
    }
  }
}

// The scale of an e4m3 row (-1: none), 0 if its codes are nothing but zeros (of either sign).  Out of line:
// hardly ever called, and the decode kernel's code is long as it is.
__device__ __noinline__ float without_zero_row(const uint8_t* rows, int width, int row, float scale) {
  if (row < 0 || scale != 1.f) return scale;
  const uint4* src = reinterpret_cast<const uint4*>(rows + (size_t)row * width);
  uint32_t any = 0;
  for (int i = 0; i < (width >> 4) && any == 0; i += 4) {
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const uint4 u = i + z < (width >> 4) ? __ldg(src + i + z) : make_uint4(0, 0, 0, 0);
      any |= (u.x | u.y | u.z | u.w) & 0x7f7f7f7fu;
    }
  }
  return any ? scale : 0.f;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int warp = (int)warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kMiscOff + 4);
  typename C::Info* infos = reinterpret_cast<typename C::Info*>(sm + C::kInfoOff);
#define BAR(i) (sb + (uint32_t)C::kBarOff + 8u * (uint32_t)(i))

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(BAR(C::kFullB + i), p.boxed ? 1 : 128);   // armed by the loader, or cp.async's threads
      mbar_init(BAR(C::kEmptyB + i), 1);
      // (lane 0 of every softmax warp arrives: an arrival of every thread on one barrier takes the
      // barrier a cycle or two each, hundreds of cycles a tile)
      mbar_init(BAR(C::kPFullB + i), 8);
    }
    mbar_init(BAR(C::kQFullB), kFp8 ? 1 : 4);
    mbar_init(BAR(C::kQEmptyB), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::kSFullB + i), 1);
      mbar_init(BAR(C::kSEmptyB + i), 8);
      mbar_init(BAR(C::kDrainB + i), 1);
    }
    mbar_init(BAR(C::kOFreeB), 8);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(BAR(C::kInfoFullB + i), 1);
      mbar_init(BAR(C::kInfoEmptyB + i), 14);  // two MMA, eight softmax and four q warps
    }
    mbar_init(BAR(C::kTokenB), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(sb + C::kMiscOff, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*reinterpret_cast<volatile uint32_t*>(sm + C::kMiscOff));
  pdl_launch_dependents();
  // Nothing global before the grid before this one is done: e4m3, latent_q_kernel, whose results only the
  // q warps read (it began after everything before it was done).
  if (!kFp8) pdl_wait();

  const LatentDecodeArgs& a = p.a;
  const int L = a.pool.L, R = a.pool.R, W = a.pool.row_bytes;
  const int n_chunks = (W + 127) >> 7;
  // bf16: latent chunk c goes to slot 2c (c < nh) or 2(c - nh) + 1, so that slots 2i, 2i + 1 hold the
  // same columns of the two halves; the rotary chunk follows in slot 2 nh.  e4m3: slot = chunk.
  const int nl = L >> 6, nh = (nl + 1) >> 1;
  const int n_mt = kFp8 ? (L + 127) >> 7 : nh;          // 128-channel tiles of O^T
  const auto slot_of = [&](int c) {
    return kFp8 ? c : (c < nh ? 2 * c : (c < nl ? 2 * (c - nh) + 1 : 2 * nh));
  };
  const int g = blockIdx.x % p.groups;                  // this CTA's 64 heads
  const int slice = blockIdx.x / p.groups;

  if (warp == 13) {
    // ================================ schedule and loads ==================================
    // the iterator: token t of the chunk of 32 whose lengths and sequences the lanes hold
    int t0 = 0, c_len = 0, c_seq = 0, c_bad = 0;
    auto load_chunk = [&](int at) {
      t0 = at;
      const int t = at + lane;
      c_len = c_seq = c_bad = 0;
      if (t < a.T) {
        const int pos = __ldg(a.positions + t);
        if (a.seq_of_token) c_seq = __ldg(a.seq_of_token + t);
        bool bad;
        c_len = token_len(a, pos, c_seq, bad);
        c_bad = bad;
      }
    };
    load_chunk(0);
    const auto quotient = [](long long x, long long y) {   // (a 64-bit division takes some 100 instructions)
      return x < 0x80000000LL && y < 0x80000000LL ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
    };
    // The line: a token that begins at w has its tile 0 there, and tile j > 0 at w + cost + j.  A slice takes
    // the tiles from per * slice to before per * (slice + 1).  (cost < per, so that a token has tiles in
    // every slice from its first to its last.)
    int cost = 0;
    long long per;
    int it_t = 0, it_j = 0;                    // next tile: token, tile of the token
    long long w_tok = 0;                       // where that token begins
    int left_all = 0;                          // tiles to go
    if (a.T == 1) {                            // nothing to weigh
      const int n = tiles_of(__shfl_sync(0xffffffffu, c_len, 0));
      const int each = max((n + p.slices - 1) / p.slices, kMinTiles);
      it_j = (int)min((long long)each * slice, (long long)n);
      left_all = min(each, n - it_j);
      per = each;
    } else {
      long long total = lane < a.T ? tiles_of(c_len) : 0;
      for (int at = 32; at < a.T; at += 4 * 32) {   // (four tokens' loads of a lane in flight)
        int pos[4], seq[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = min(at + 32 * i + lane, a.T - 1);
          pos[i] = __ldg(a.positions + t);
          if (a.seq_of_token) seq[i] = __ldg(a.seq_of_token + t);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool bad;
          if (at + 32 * i + lane < a.T) total += tiles_of(token_len(a, pos[i], seq[i], bad));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      cost = (int)min((long long)kTokenCost,
                      max(quotient(total + p.slices - 1, p.slices), (long long)kMinTiles) - 1);
      per = max(quotient(total + (long long)cost * a.T + p.slices - 1, p.slices), (long long)kMinTiles);
      const long long begin = per * slice, end = begin + per;
      bool found = false;
      int chunk = 0;
      long long w0 = 0;
      for (;; load_chunk(t0 + 32)) {
        const int n = t0 + lane < a.T ? tiles_of(c_len) : 0;
        int sum = n;                           // inclusive scan (32 tokens: below 2^31 tiles)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const long long w = w0 + (sum - n) + (long long)cost * lane;
        const auto before = [&](long long x) {   // tiles of this lane's token before x
          return x <= w ? 0 : (int)min((long long)n, max(1LL, x - w - cost));
        };
        const int lo = before(begin);
        left_all += before(end) - lo;
        const unsigned m = __ballot_sync(0xffffffffu, lo < n);
        if (!found && m) {
          const int k = __ffs(m) - 1;
          found = true;
          chunk = t0;
          it_t = t0 + k;
          it_j = __shfl_sync(0xffffffffu, lo, k);
          w_tok = __shfl_sync(0xffffffffu, w, k);
        }
        w0 += __shfl_sync(0xffffffffu, sum, 31) + 32LL * cost;
        if (t0 + 32 >= a.T || w0 >= end) break;
      }
      left_all = __reduce_add_sync(0xffffffffu, left_all);
      if (t0 != chunk) load_chunk(chunk);
    }
    if (lane == 0) {                           // the first token's q can be on its way
      *reinterpret_cast<volatile int*>(sm + C::kMiscOff + 8) = left_all > 0 ? it_t : -1;
      mbar_arrive(BAR(C::kTokenB));
    }
    struct Tile {
      int t, flags, slot;
      int blk[2], off[2];                      // block and slot in it of entries lane, 32 + lane
    };
    // The token of the next tile: its sequence, tiles to go, entries to go, whether its first tile is
    // this CTA's; and, boxed (tiles lie in one page each), the slot in the page and the blocks of tiles
    // c_tile .. c_tile + 31, one a lane.
    int b_t = 0, n_tok = 0, left = 0, entries = 0, started = 0, off = 0, c_tile = 0, c_blk = -1;
    bool fresh = true;
    int2 cut = make_int2(-1, 0);
    const auto begin_token = [&]() {
      if (it_t >= t0 + 32) load_chunk(it_t);
      const int k = it_t - t0;
      const int len = __shfl_sync(0xffffffffu, c_len, k);
      b_t = __shfl_sync(0xffffffffu, c_seq, k);
      started = it_j == 0;
      if (started && __shfl_sync(0xffffffffu, c_bad, k) && lane == 0) flag_error(SPA_ERR_INDEX);
      n_tok = tiles_of(len);
      left = n_tok - it_j;
      entries = len - it_j * kKeys;
      if (started && left > left_all)          // (the line ends inside it: the slice where it ends)
        cut = make_int2(it_t, (int)quotient(w_tok + cost + n_tok - 1, per));
      if (p.boxed) off = it_j % (a.pool.ps / kKeys) * kKeys;
      c_tile = it_j - 32;
      fresh = true;
    };
    if (left_all > 0) begin_token();
    auto next_tile = [&](Tile& x) {            // the next tile, its block-table reads under way
      x.t = -1;
      if (left_all == 0) return;
      if (left == 0) {
        w_tok += cost + n_tok;
        ++it_t;
        it_j = 0;
        begin_token();
      }
      x.t = it_t;
      const bool last = left == 1 || left_all == 1;
      x.flags = (fresh ? kFirst : 0) | (last ? kLast : 0) | (left_all == 1 ? kFinal : 0);
      x.slot = started && left == 1 ? -1 : started;
      if (p.boxed) {
        if (it_j >= c_tile + 32) {
          c_tile = it_j;
          const int page = (it_j * kKeys + min(lane, left - 1) * kKeys) / a.pool.ps;
          c_blk = entries > 0 ? __ldg(a.pool.bt + (size_t)b_t * a.pool.bt_stride + page) : -1;
        }
        const int blk = __shfl_sync(0xffffffffu, c_blk, it_j - c_tile);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x.blk[e] = lane + 32 * e < entries ? blk : -2;   // -2: not of the sequence
          x.off[e] = off + lane + 32 * e;
        }
        off = off + kKeys == a.pool.ps ? 0 : off + kKeys;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x.blk[e] = -2;
          x.off[e] = 0;
          if (lane + 32 * e < entries) {
            const int key = it_j * kKeys + lane + 32 * e;
            const int page = key / a.pool.ps;
            x.off[e] = key - page * a.pool.ps;
            x.blk[e] = __ldg(a.pool.bt + (size_t)b_t * a.pool.bt_stride + page);
          }
        }
      }
      fresh = false;
      --left_all;
      --left;
      ++it_j;
      entries -= kKeys;
    };
    // Rows of a tile (-1: no such entry) and, e4m3, their scales.
    auto resolve = [&](const Tile& x, int (&row)[2], float (&sc)[2]) {
      row[0] = row[1] = -1;
      if (x.t < 0) return;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (x.blk[e] >= 0 && (long long)x.blk[e] < a.pool.num_blocks)
          row[e] = x.blk[e] * a.pool.ps + x.off[e];        // (below 2^30)
        else if (x.blk[e] != -2)
          flag_error(SPA_ERR_INDEX);
        sc[e] = kFp8 && row[e] >= 0 ? __ldg(a.pool.scale + row[e]) : 0.f;
      }
    };
    // A tile's blocks are read two tiles ahead of its copy and its scales one ahead; nothing loaded is
    // touched (not even copied to another register) before it is needed.
    Tile nxt = {};
    int row[2], t_cur, flags_cur, slot_cur;
    float sc[2] = {0.f, 0.f};
    const auto take = [&]() {                  // the tile read last becomes the current one
      t_cur = nxt.t;
      flags_cur = nxt.flags;
      slot_cur = nxt.slot;
      resolve(nxt, row, sc);
      next_tile(nxt);
    };
    next_tile(nxt);
    take();
    const int total_rows = (int)(a.pool.num_blocks * a.pool.ps);
    int k = 0, fills = 0;
    LatentTileRing at;
    bool ok = true;
    if (t_cur < 0) {                           // nothing to do: tell the others
      if (lane == 0) {
        infos[0].flags = kEnd;
        __threadfence_block();
        mbar_arrive(BAR(C::kInfoFullB));
      }
    }
    for (; t_cur >= 0; ++k) {
      if (p.boxed) {                           // its copy first: everything else can wait for that
        ok = warp_wait(BAR(C::kEmptyB + at.slot), at.parity ^ 1, abort_flag);
        if (!ok) break;
        // a tile without entries starts past the last row and is filled with zeros
        const int base = (int)warp_uniform(row[0] >= 0 ? row[0] : total_rows);
        if (elect_one()) {
          const uint32_t dst = sb + C::kKOff + at.slot * C::kBufBytes, full = BAR(C::kFullB + at.slot);
          mbar_arrive_expect_tx(full, (uint32_t)(n_chunks * kChunkBytes));
          if (p.whole > 0) {
            if (kFp8) tma_box3(dst, &p.block, 0, base, 0, full);
            else tma_box4(dst, &p.block, 0, base, 0, 0, full);
          }
          for (int c = p.whole; c < n_chunks; ++c)
            tma_row(dst + slot_of(c) * kChunkBytes, &p.chunk, c * 128, base, full);
        }
        __syncwarp();
        ++fills;
        at.next();
      }
      // publish the tile
      const int ri = k % kRing;
      ok = warp_wait(BAR(C::kInfoEmptyB + ri), ((k / kRing) & 1) ^ 1, abort_flag);
      if (!ok) break;
      const unsigned lo = __ballot_sync(0xffffffffu, row[0] >= 0);
      const unsigned hi = __ballot_sync(0xffffffffu, row[1] >= 0);
      typename C::Info& info = infos[ri];
      if (!p.boxed) {
        info.row[lane] = row[0];
        info.row[lane + 32] = row[1];
      }
      if (kFp8) {
        // (a scale of exactly 1 is that of a row of zeros or, rarely, of one whose largest value is 448)
        if (__any_sync(0xffffffffu, sc[0] == 1.f || sc[1] == 1.f)) {
          sc[0] = without_zero_row(a.pool.rows, W, row[0], sc[0]);
          sc[1] = without_zero_row(a.pool.rows, W, row[1], sc[1]);
        }
        // the maximum of a tile is taken over p_j |scale_j|, the weights that enter the value
        // product (a scale below 2^-60 counts as that: the sums of p_j alone must stay finite)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          info.scale[lane + 32 * e] = kPUnit * sc[e];
          info.lscale[lane + 32 * e] = row[e] >= 0 ? fmaxf(__log2f(fabsf(sc[e])), -60.f) : -INFINITY;
        }
      }
      if (lane == 0) {
        info.t = t_cur;
        info.flags = flags_cur;
        info.slot = slot_cur;
        info.valid[0] = lo;
        info.valid[1] = hi;
      }
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kInfoFullB + ri));
      take();
    }
    if (lane == 0) {
      p.cut[blockIdx.x] = cut;
      // copies in flight must land before the CTA ends (at once after a normal run)
      for (int q = max(0, fills - kBufs); q < fills; ++q)
        mbar_wait_drain(BAR(C::kFullB + q % kBufs), (uint32_t)((q / kBufs) & 1));
    }
  } else if (warp == 12) {
    // ================================= MMAs of S ==========================================
    // The warp runs as one (its waits too); one elected lane issues.  The MMAs of one tile execute in
    // the order of issue.
    const uint32_t idS2 = idesc_bf16(128, 128, 0, 0), idS1 = idesc_bf16(128, 64, 0, 0);
    const uint32_t idS8 = idesc_e4m3(128, 64, 0, 0);
    const uint64_t dq0 = sdesc(sb + C::kQOff, 16, 1024);
    const uint64_t dk0 = sdesc(sb + C::kKOff, 16, 1024);            // rows, K-major
    const bool lead = elect_one();
    LatentTileRing at;
    uint32_t q_ph = 0;
    for (int k = 0;; ++k) {
      const int ri = k % kRing, sn = k % C::kSBufs;
      if (!warp_wait(BAR(C::kInfoFullB + ri), (uint32_t)((k / kRing) & 1), abort_flag)) break;
      const int flags = (int)warp_uniform(*reinterpret_cast<volatile int*>(&infos[ri].flags));
      if (lead) mbar_arrive(BAR(C::kInfoEmptyB + ri));
      if (flags & kEnd) break;
      if (flags & kFirst) {
        if (!warp_wait(BAR(C::kQFullB), q_ph, abort_flag)) break;
        q_ph ^= 1;
      }
      if (!warp_wait(BAR(C::kFullB + at.slot), at.parity, abort_flag)) break;
      if (!warp_wait(BAR(C::kSEmptyB + sn), ((k / C::kSBufs) & 1) ^ 1, abort_flag)) break;
      if (!p.boxed) fence_proxy_async_smem();   // (rows copied by cp.async)
      tc_fence_after();
      if (lead) {
        const uint32_t dS = tmem + kSCol + sn * 64;
        const uint64_t dk = desc_add(dk0, at.slot * C::kBufBytes);
        if (kFp8) {
          for (int c = 0; c < n_chunks; ++c) {
            const int steps = (W - c * 128 + 31) >> 5;             // 32-byte steps left in the row
            const uint64_t dqc = desc_add(dq0, c * 16384), dkc = desc_add(dk, c * kChunkBytes);
            mma_f8(dS, dqc, dkc, idS8, c != 0);
            if (steps >= 4) {
#pragma unroll
              for (int st = 1; st < 4; ++st) mma_f8(dS, desc_add(dqc, st * 32), desc_add(dkc, st * 32), idS8, 1u);
            } else {
              for (int st = 1; st < steps; ++st) mma_f8(dS, desc_add(dqc, st * 32), desc_add(dkc, st * 32), idS8, 1u);
            }
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < nh; ++i) {
            const uint32_t id = nh + i < nl ? idS2 : idS1;         // (an odd last chunk stands alone)
#pragma unroll
            for (int st = 0; st < 4; ++st)
              mma_bf16_ts(dS, tmem + kQCol + i * 32 + st * 8,
                          desc_add(dk, 2 * i * kChunkBytes + st * 32), id, (i | st) != 0);
          }
          const int steps = (2 * R + 31) >> 5;
#pragma unroll
          for (int st = 0; st < 4; ++st)
            if (st < steps)
              mma_bf16(dS, desc_add(dq0, st * 32), desc_add(dk, 2 * nh * kChunkBytes + st * 32), idS1, 1u);
        }
        mma_commit(BAR(C::kSFullB + sn));
        if (flags & kLast) mma_commit(BAR(C::kQEmptyB));
      }
      __syncwarp();
      at.next();
      if (flags & kFinal) break;
    }
    // nothing may still write TMEM when it is released
    if (lead) {
      mma_commit(BAR(C::kDrainB));
      mbar_wait_drain(BAR(C::kDrainB), 0);
    }
    __syncwarp();
  } else if (warp == 14) {
    // ================================= MMAs of O ==========================================
    const uint32_t idO = kFp8 ? idesc_e4m3(128, 64, 1, 0) : idesc_bf16(128, 64, 1, 0);
    const uint32_t idO5 = idO | (1u << 10);            // B in e5m2: the terms of P
    const uint64_t dv0 = sdesc(sb + C::kKOff, kChunkBytes, 1024);   // rows, MN-major
    const uint32_t p_at = sb + C::kKOff + (C::kSlots - 1) * kChunkBytes;
    const uint64_t dp0 = kFp8 ? sdesc64(p_at, 16, 512) : sdesc(p_at, 16, 1024);
    const uint64_t dp3 = sdesc64(sb + C::kPOff, 16, 512);           // e4m3's third term
    const bool lead = elect_one();
    LatentTileRing at;
    uint32_t o_ph = 0;
    bool any = warp_wait(BAR(C::kInfoFullB), 0, abort_flag);
    if (any) any = !(warp_uniform(*reinterpret_cast<volatile int*>(&infos[0].flags)) & kEnd);
    for (int k = 0; any; ++k) {
      const int ri = k % kRing;
      if (!warp_wait(BAR(C::kPFullB + at.slot), at.parity, abort_flag)) break;
      // (P of the tile comes after its S, and that after its info)
      const int flags = (int)warp_uniform(*reinterpret_cast<volatile int*>(&infos[ri].flags));
      if (lead) mbar_arrive(BAR(C::kInfoEmptyB + ri));
      const bool first = flags & kFirst;
      if (first) {
        if (!warp_wait(BAR(C::kOFreeB), o_ph ^ 1, abort_flag)) break;
        o_ph ^= 1;
      }
      if (!p.boxed) fence_proxy_async_smem();
      tc_fence_after();
      if (lead) {
        const uint32_t acc0 = first ? 0u : 1u;
        const uint64_t dp = desc_add(dp0, at.slot * C::kBufBytes), dq = desc_add(dp3, at.slot * 4096);
#pragma unroll 1
        for (int mt = 0; mt < n_mt; ++mt) {
          const uint32_t dO = tmem + mt * 64;
          const uint64_t dv = desc_add(dv0, at.slot * C::kBufBytes + mt * C::kPerTile * kChunkBytes);
          if (!kFp8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)               // 16 entries a step
              mma_bf16(dO, desc_add(dv, kk * 2048), desc_add(dp, kk * 32), idO, kk ? 1u : acc0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {             // 32 entries a step
              mma_f8(dO, desc_add(dv, kk * 4096), desc_add(dp, kk * 32), idO5, kk ? 1u : acc0);
              mma_f8(dO, desc_add(dv, kk * 4096), desc_add(dp, 4096 + kk * 32), idO5, 1u);
              mma_f8(dO, desc_add(dv, kk * 4096), desc_add(dq, kk * 32), idO5, 1u);
            }
          }
        }
        mma_commit(BAR(C::kEmptyB + at.slot));
      }
      __syncwarp();
      at.next();
      if (flags & kFinal) break;
    }
    if (lead) {
      mma_commit(BAR(C::kDrainB + 1));
      mbar_wait_drain(BAR(C::kDrainB + 1), 0);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // =================================== queries ==========================================
    // Each token's q is read into registers as soon as its first tile is announced, and put in
    // place once the token before has no S left to compute.
    const int tid = threadIdx.x - kSoftmax;
    int items = 0, flags = 0;
    if (kFp8) pdl_wait();           // (for latent_q_kernel, launched right before)
    auto put_q = [&](int t) -> bool {
      if constexpr (!kFp8) {
        // TMEM lane 32w + l is head 32(w & 1) + l; its first (w < 2) or second half of the latents
        const int qw = warp - 8, h = g * kHeads + (qw & 1) * 32 + lane;
        const int c0 = qw < 2 ? 0 : nh, nc = qw < 2 ? nh : nl - nh;
        const uint4* src = reinterpret_cast<const uint4*>(a.q_latent + t * a.ql_st + h * a.ql_sh) + 8 * c0;
        const auto load = [&](int b, uint4 (&u)[16]) {      // sixteen 16-byte units in flight
#pragma unroll
          for (int i = 0; i < 16; ++i)
            u[i] = (h < a.H && 16 * b + i < 8 * nc) ? __ldg(src + 16 * b + i) : make_uint4(0, 0, 0, 0);
        };
        const auto put = [&](int b, const uint4 (&u)[16]) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              w[4 * i] = __uint_as_float(u[8 * q + i].x);
              w[4 * i + 1] = __uint_as_float(u[8 * q + i].y);
              w[4 * i + 2] = __uint_as_float(u[8 * q + i].z);
              w[4 * i + 3] = __uint_as_float(u[8 * q + i].w);
            }
            tmem_st32(tmem + ((uint32_t)(qw * 32) << 16) + kQCol + 64 * b + 32 * q, w);
          }
        };
        if (h < a.H)                    // the second sixteen units on their way to L2
          for (int i = 16; i < 8 * nc; i += 8)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
        uint4 u[16];
        load(0, u);
        uint4 v[4];                     // rotary part: 64 rows of eight 16-byte units
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hr = (tid >> 3) + 16 * i, hg = g * kHeads + hr;
          v[i] = make_uint4(0, 0, 0, 0);
          if (hg < a.H && (tid & 7) * 8 < R)
            v[i] = __ldg(reinterpret_cast<const uint4*>(a.q_rope + t * a.qr_st + hg * a.qr_sh) + (tid & 7));
        }
        if (!warp_wait(BAR(C::kQEmptyB), (uint32_t)((items & 1) ^ 1), abort_flag)) return false;
        tc_fence_after();
        put(0, u);
        load(1, u);
        put(1, u);
        tmem_wait_st();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hr = (tid >> 3) + 16 * i;
          *reinterpret_cast<uint4*>(sm + C::kQOff + hr * 128 + (((tid & 7) ^ (hr & 7)) << 4)) = v[i];
        }
      } else {
        // latent_q_kernel's codes and scales of 64 heads: two plain copies
        if (warp == 8) {
          if (!warp_wait(BAR(C::kQEmptyB), (uint32_t)((items & 1) ^ 1), abort_flag)) return false;
          if (elect_one()) {
            const size_t at = (size_t)t * p.groups + g;
            const uint32_t bytes = (uint32_t)n_chunks * 16384;
            mbar_arrive_expect_tx(BAR(C::kQFullB), bytes + kHeads * 4);
            bulk_load(sb + C::kQOff, p.q_codes + at * bytes, bytes, BAR(C::kQFullB));
            bulk_load(sb + C::kQScaleOff + (items & 3) * kHeads * 4, p.q_scale + at * kHeads, kHeads * 4,
                      BAR(C::kQFullB));
          }
          __syncwarp();
        }
        ++items;
        return true;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kQFullB));
      ++items;
      return true;
    };
    // (a boxed CTA's first token does not wait for the page table; cp.async copies rows first)
    bool ok = true;
    if (p.boxed) {
      ok = warp_wait(BAR(C::kTokenB), 0, abort_flag);
      const int t = *reinterpret_cast<volatile int*>(sm + C::kMiscOff + 8);
      if (ok && t >= 0) ok = put_q(t);
    }
    LatentTileRing at;
    for (int k = 0; ok && !(flags & kFinal); ++k) {
      const int ri = k % kRing;
      if (!warp_wait(BAR(C::kInfoFullB + ri), (uint32_t)((k / kRing) & 1), abort_flag)) break;
      const int t = infos[ri].t;
      flags = infos[ri].flags;
      if (flags & kEnd) break;
      if (!p.boxed) {
        // the tile's rows by cp.async: unit jj (16 bytes) of every chunk of rows r0, r0 + 16, ..;
        // what is no entry, or past the row, is filled with zeros
        const int jj = tid & 7, r0 = tid >> 3;
        const uint8_t* src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = infos[ri].row[r0 + 16 * i];
          src[i] = row >= 0 ? a.pool.rows + (size_t)row * W : nullptr;
        }
        const uint32_t dst = sb + C::kKOff + at.slot * C::kBufBytes + r0 * 128 + ((jj ^ (r0 & 7)) << 4);
        if (!warp_wait(BAR(C::kEmptyB + at.slot), at.parity ^ 1, abort_flag)) break;
        for (int c = 0; c < n_chunks; ++c) {
          const int col = c * 128 + jj * 16;
          const uint32_t d = dst + slot_of(c) * kChunkBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool has = src[i] != nullptr && col < W;
            cp_async_16(d + i * 2048, has ? src[i] + col : a.pool.rows, has ? 16u : 0u);
          }
        }
        cp_async_arrive_noinc(BAR(C::kFullB + at.slot));
        at.next();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kInfoEmptyB + ri));
      if ((flags & kFirst) && !(p.boxed && k == 0) && !put_q(t)) break;
    }
    cp_async_wait_all();
    if (kFp8 && warp == 8 && items > 0) {      // (a copy in flight, where the CTA gave up)
      mbar_wait_drain(BAR(C::kQFullB), (uint32_t)((items - 1) & 1));
      __syncwarp();
    }
  } else {
    // ================================ softmax and epilogue ================================
    const int tid = threadIdx.x;
    // TMEM lanes 32 quad ..: stacked block `half` of heads 32 pair ..; this warp takes columns of part
    // `ch`: entries 32 half + 16 ch .. of the tile, and channels' heads 32 ch .. of O^T
    const int quad = warp & 3, ch = warp >> 2, half = quad >> 1, pair = quad & 1;
    const int head = pair * 32 + lane, part = 2 * half + ch;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    float* red = reinterpret_cast<float*>(sm + C::kRedOff);
    const bool two = kFp8 || nl > 1;               // the second stacked block holds anything
    // own head and head ^ 32 (whose channels this warp may have to rescale)
    float m = -INFINITY, mo = -INFINITY, l = 0.f;
    int items = -1, reds = 0;
    // Named barriers join the eight warps (1) and the two that swap parts of S (2 .. 5).  A wait that
    // gives up does not leave the loop: every warp reaches every barrier, and all leave together, where
    // they agree that one of them gave up.
    bool ok = true;
    // The four parts' values of the own head and of head ^ 32.  (All eight warps pass a barrier between
    // one use of a buffer and its next: e4m3 the other buffer's, bf16 that of the vote.)
    auto exchange = [&](float mine, float (&own)[4], float (&other)[4]) -> bool {
      float* r = red + (kFp8 ? (reds & 1) * 256 : 0);
      ++reds;
      r[part * 64 + head] = mine;
      ok = named_bar_and(1, kSoftmax, ok);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        own[e] = r[e * 64 + head];
        other[e] = r[e * 64 + (head ^ 32)];
      }
      return ok;
    };
    // Factor of head c (lane c of the warps that own it, or their own copy) for columns c of O^T
    auto column = [&](float own, float other, int c) {
      return __shfl_sync(0xffffffffu, (c >= 32) == (pair != 0) ? own : other, c & 31);
    };
    int flags = 0;
    LatentTileRing at, at1;                        // this tile, the one before
    // the MMAs of O of a tile are done
    const auto pv_done = [&](const LatentTileRing& tile) {
      return warp_wait(BAR(C::kEmptyB + tile.slot), tile.parity, abort_flag);
    };
    ok = warp_wait(BAR(C::kInfoFullB), 0, abort_flag);
    const bool any = named_bar_and(1, kSoftmax, ok && !(infos[0].flags & kEnd));
    for (int k = 0; any && !(flags & kFinal); ++k) {
      const int ri = k % kRing, s = k % C::kSBufs;
      if (k > 0) {
        at1 = at;
        at.next();
      }
      ok = warp_wait(BAR(C::kSFullB + s), (uint32_t)((k / C::kSBufs) & 1), abort_flag) && ok;
      tc_fence_after();
      // (S of the tile comes after its info)
      const typename C::Info& info = infos[ri];
      const int t = info.t, slot = info.slot;
      flags = info.flags;
      const uint32_t va = info.valid[0], vb = info.valid[1];
      const bool first = flags & kFirst, last = flags & kLast;
      if (first) {
        ++items;
        m = mo = -INFINITY;
        l = 0.f;
      }
      float x[16];
      // P of this tile: in its last slot, whose rotary part only S needed
      uint8_t* pb = sm + C::kKOff + at.slot * C::kBufBytes + (C::kSlots - 1) * kChunkBytes;
      {
        float th[16];
        const uint32_t sa = lane_base + kSCol + (kFp8 ? s * 64 : half * 64) + 16 * ch;
        tmem_ld16(sa + (half ^ 1) * 32, th);
        tmem_ld16(sa + half * 32, x);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kSEmptyB + s));
        if (!two && half == 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) th[j] = x[j] = 0.f;
        }
        // The warps of the other block have the other part of S: swap the entries that are not one's
        // own with one of them, eight at a time, through a quarter of P's rows.  A warp's second eight
        // go where it has just read, so one barrier a round is enough.
        uint8_t* quarter = pb + (2 * pair + ch) * 2048;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float4* put = reinterpret_cast<float4*>(quarter + (half ^ 1 ^ r) * 1024);
          const float4* get = reinterpret_cast<const float4*>(quarter + (half ^ r) * 1024);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            put[j * 32 + lane] = make_float4(th[8 * r + 4 * j], th[8 * r + 4 * j + 1],
                                             th[8 * r + 4 * j + 2], th[8 * r + 4 * j + 3]);
          named_bar_sync(2 + 2 * pair + ch, 64);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 o = get[j * 32 + lane];
            x[8 * r + 4 * j] += o.x;
            x[8 * r + 4 * j + 1] += o.y;
            x[8 * r + 4 * j + 2] += o.z;
            x[8 * r + 4 * j + 3] += o.w;
          }
        }
      }
      const int e0 = 32 * half + 16 * ch;          // this thread's first entry
      const uint32_t valid = ((half ? vb : va) >> (16 * ch)) & 0xffffu;
      float mt = -INFINITY, arg = 1.f;              // log2 of the weights: arg x
      if (kFp8) {
        // (info.scale holds kPUnit times the rows' scales, and this table 1 / kPUnit over the heads')
        arg = p.scale_log2 *
              reinterpret_cast<const float*>(sm + C::kQScaleOff)[(items & 3) * kHeads + head];
        const float4* ks4 = reinterpret_cast<const float4*>(info.scale + e0);
        const float4* ls4 = reinterpret_cast<const float4*>(info.lscale + e0);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 4; ++j) {                // (lscale is -inf where no entry takes part)
          const float4 c = ks4[j], d = ls4[j];
          x[4 * j] *= c.x;
          x[4 * j + 1] *= c.y;
          x[4 * j + 2] *= c.z;
          x[4 * j + 3] *= c.w;
          mx[0] = fmaxf(mx[0], fmaf(arg, x[4 * j], d.x));
          mx[1] = fmaxf(mx[1], fmaf(arg, x[4 * j + 1], d.y));
          mx[2] = fmaxf(mx[2], fmaf(arg, x[4 * j + 2], d.z));
          mx[3] = fmaxf(mx[3], fmaf(arg, x[4 * j + 3], d.w));
        }
        mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= p.scale_log2;
        if (valid != 0xffffu) {
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = (valid >> j) & 1u ? x[j] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 16; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
        mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      }
      // bf16: most tiles leave every running maximum within tau of what it was: one vote tells (and tells
      // that the swaps are over), and the maxima are exchanged only where one head's has to move.  (With
      // e4m3's smaller tau so many tiles would need both that the exchange alone measured faster.)
      float own[4], other[4], al = 1.f, alo = 1.f;
      uint32_t grow0 = 0, grow1 = 0;
      if (kFp8 || !named_bar_and(1, kSoftmax, ok && !(mt > m + C::kTau))) {
        if (!exchange(mt, own, other)) break;      // (all eight warps, or none)
        const float t0 = fmaxf(fmaxf(own[0], own[1]), fmaxf(own[2], own[3]));
        const float t1 = fmaxf(fmaxf(other[0], other[1]), fmaxf(other[2], other[3]));
        const float n0 = t0 > m + C::kTau ? t0 : m, n1 = t1 > mo + C::kTau ? t1 : mo;
        grow0 = __ballot_sync(0xffffffffu, n0 != m);
        grow1 = __ballot_sync(0xffffffffu, n1 != mo);
        al = fast_exp2(m - n0);                    // (only used where n0 is not -inf)
        alo = fast_exp2(mo - n1);
        if (n0 != m) l *= al;
        else al = 1.f;
        if (n1 == mo) alo = 1.f;
        m = n0;
        mo = n1;
      }
      const bool grow = (grow0 | grow1) != 0;
      // (a head without any entry so far: everything is masked, the reference does not matter)
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = kFp8 ? fast_exp2(fmaf(arg, x[j], -ref)) : fast_exp2(x[j] - ref);
        if (kFp8 && valid != 0xffffu) x[j] = (valid >> j) & 1u ? x[j] : 0.f;
      }
      if (!kFp8) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {              // 16-byte unit: eight entries
          const float* e = x + 8 * u;
          *reinterpret_cast<uint4*>(pb + head * 128 + (((2 * part + u) ^ (head & 7)) << 4)) =
              make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                         pack_bf16x2(e[6], e[7]));
        }
      } else {
        // u = kPUnit p scale (at most 2^15) in f16, whose upper byte is an e5m2 number: the nearest one by
        // adding half a step to the bits, then the same of what it leaves (exact in f16), and again.
        // (A NaN's bits run over here; it comes back through the denominator.)
        const float4* ks4 = reinterpret_cast<const float4*>(info.scale + e0);
        uint32_t w[3][4];                          // of each term one 16-byte unit: sixteen entries
        const auto upper = [](uint32_t f16x2) { return (f16x2 + 0x00800080u) & 0xff00ff00u; };
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 c = ks4[q];
          const float* e = x + 4 * q;
          uint32_t t[3][2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            __half2 y = z ? __floats2half2_rn(e[2] * c.z, e[3] * c.w) : __floats2half2_rn(e[0] * c.x, e[1] * c.y);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              t[i][z] = upper(*reinterpret_cast<const uint32_t*>(&y));
              if (i < 2) y = __hsub2(y, *reinterpret_cast<const __half2*>(&t[i][z]));
            }
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) w[i][q] = __byte_perm(t[i][0], t[i][1], 0x7531);
        }
        const int unit = head * 64 + ((part ^ ((head >> 1) & 3)) << 4);
        *reinterpret_cast<uint4*>(pb + unit) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
        *reinterpret_cast<uint4*>(pb + 4096 + unit) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
        *reinterpret_cast<uint4*>(sm + C::kPOff + at.slot * 4096 + unit) =
            make_uint4(w[2][0], w[2][1], w[2][2], w[2][3]);
      }
      if ((va & vb) != 0xffffffffu) {
        // entries that take no part: their rows hold other data or none, and a probability of zero
        // times a NaN would still be one
        for (int e = 0; e < 2; ++e) {
          uint32_t gone = ~(e ? vb : va);
          while (gone) {
            const int r = 32 * e + __ffs(gone) - 1;
            gone &= gone - 1;
            for (int u = tid; u < n_mt * C::kPerTile * 8; u += kSoftmax)   // 16-byte units of its values
              *reinterpret_cast<uint4*>(sm + C::kKOff + at.slot * C::kBufBytes + (u >> 3) * kChunkBytes +
                                        r * 128 + (u & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      if (grow && !first) {
        // the running maximum of some head moved: rescale its quarter of O (sixteen heads) once PV of
        // the tile before is done
        ok = pv_done(at1) && ok;
        tc_fence_after();
        const uint32_t g0 = pair ? grow1 : grow0, g1 = pair ? grow0 : grow1;   // heads 0-31, 32-63
#pragma unroll 1
        for (int q = 2 * ch; q < 2 * ch + 2; ++q) {
          if ((((q >= 2 ? g1 : g0) >> (16 * (q & 1))) & 0xffffu) == 0) continue;
          float f[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = column(al, alo, q * 16 + c);
#pragma unroll 1
          for (int i = 0; i < n_mt; i += 2) {
            const uint32_t ta = lane_base + i * 64 + q * 16;
            float o[2][16];
            tmem_ld16(ta, o[0]);
            if (i + 1 < n_mt) tmem_ld16(ta + 64, o[1]);
            tmem_wait_ld();
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t w[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) w[c] = __float_as_uint(o[z][c] * f[c]);
              if (i + z < n_mt) tmem_st16(ta + z * 64, w);
            }
          }
        }
        tmem_wait_st();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(BAR(C::kPFullB + at.slot));
        mbar_arrive(BAR(C::kInfoEmptyB + ri));
      }
      // (nobody waits for the denominators)
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[j & 3] += x[j];
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (!last) continue;

      // ---- epilogue: denominators, then O ----
      if (!kFp8) named_bar_sync(1, kSoftmax);      // (the last exchange has been read by all)
      if (!exchange(l, own, other)) break;
      const float ls = (own[0] + own[1]) + (own[2] + own[3]);
      const float lso = (other[0] + other[1]) + (other[2] + other[3]);
      // (0: no entry at all.  A NaN among the scores is in the sum, whatever the maximum is.)
      constexpr float kUnit = kFp8 ? 1.f / kPUnit : 1.f;
      const float inv = ls == 0.f ? 0.f : kUnit / ls, invo = lso == 0.f ? 0.f : kUnit / lso;
      const int Hg = min(kHeads, a.H - g * kHeads);
      const size_t pslot = (size_t)blockIdx.x * 2 + (slot > 0 ? 1 : 0);
      if (slot >= 0 && part == 0)
        p.lse[pslot * kHeads + head] = ls == 0.f ? -INFINITY : m + __log2f(ls);
      ok = pv_done(at) && ok;
      tc_fence_after();
      // TMEM lane -> channel of tile i of O^T: d0 + i dstep; sixteen heads (columns) at a time
      const int ln = quad * 32 + lane;
      const int d0 = kFp8 || ln < 64 ? ln : 64 * nh + ln - 64, dstep = kFp8 ? 128 : 64;
#pragma unroll 1
      for (int q = 2 * ch; q < 2 * ch + 2; ++q) {
        const int n_h = min(16, Hg - q * 16);
        if (n_h <= 0) break;
        float iv[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) iv[c] = column(inv, invo, q * 16 + c);
        const auto store = [&](int i, const float (&o)[16]) {
          const int d = d0 + i * dstep;
          if (slot >= 0) {
            float* wo = p.part + (pslot * kHeads + q * 16) * L + d;
            if (d < L) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (c < n_h) wo[(uint32_t)(c * L)] = o[c] * iv[c];
            }
          } else {
            // lanes 2m and 2m + 1 swap halves so that each stores two adjacent channels
            const bool up = lane & 1;
            __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(a.out) +
                                ((size_t)t * a.H + g * kHeads + q * 16) * L + (d & ~1);
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float x0 = o[c] * iv[c], x1 = o[c + 1] * iv[c + 1];
              const float recv = __shfl_xor_sync(0xffffffffu, up ? x0 : x1, 1);
              const uint32_t pr = up ? pack_bf16x2(recv, x1) : pack_bf16x2(x0, recv);
              const int hh = c + (up ? 1 : 0);
              if (hh < n_h && d < L) *reinterpret_cast<uint32_t*>(ob + (uint32_t)(hh * L)) = pr;
            }
          }
        };
        // two tiles of O^T a round: the next one is read from TMEM while one is stored
#pragma unroll 1
        for (int i = 0; i < n_mt; i += 2) {
          float o0[16], o1[16];
          tmem_ld16(lane_base + i * 64 + q * 16, o0);
          tmem_wait_ld();
          if (i + 1 < n_mt) tmem_ld16(lane_base + (i + 1) * 64 + q * 16, o1);
          store(i, o0);
          tmem_wait_ld();
          if (i + 1 < n_mt) store(i + 1, o1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kOFreeB));
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the tokens that were cut: out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).
// Most tokens are cut in two or three: a warp takes a head of one, with all its loads in flight at
// once.  A token of more than kWarpParts parts (few long sequences) takes a block for every 128 channels
// of a head, its eight warps every eighth part each, added up in warp order.  Bound by reading the
// parts.
constexpr int kMergeWarps = 8;
constexpr int kMergeMaxCuts = 1024;
constexpr int kWarpParts = 8;
constexpr int kParts = 20;          // loads in flight a warp: all of its parts of 152 slices

__global__ void __launch_bounds__(32 * kMergeWarps)
    latent_merge_kernel(const int2* __restrict__ cut, const float* __restrict__ lse,
                        const float* __restrict__ part, __nv_bfloat16* __restrict__ out, int slices,
                        int groups, int H, int L) {
  __shared__ __align__(16) float sum[kMergeWarps][128];
  // of every cut token: the slice where it begins, its last slice, itself, units of the tokens before it
  __shared__ __align__(16) int4 item[kMergeMaxCuts];
  __shared__ int2 cuts[kMergeMaxCuts];
  __shared__ float2 stat[kMergeWarps];
  __shared__ int n_items, n_units;
  __shared__ int2 warp_sum[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = (L + 127) >> 7;
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kMergeMaxCuts / (32 * kMergeWarps); ++i) {     // (all loads in flight together)
    const int s = threadIdx.x + i * 32 * kMergeWarps;
    if (s < slices) cuts[s] = cut[(size_t)s * groups];
  }
  __syncthreads();
  // A thread takes a slice; the items and units before it are its warp's scan and the warps' before.
  for (int s0 = 0; s0 < slices; s0 += 32 * kMergeWarps) {
    const int s = s0 + threadIdx.x;
    const int2 c = s < slices ? cuts[s] : make_int2(-1, 0);
    const unsigned m = __ballot_sync(0xffffffffu, c.x >= 0);
    const int mine = c.x < 0 ? 0 : (c.y - s + 1 <= kWarpParts ? (H + kMergeWarps - 1) / kMergeWarps : H * nq);
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) warp_sum[warp] = make_int2(__popc(m), scan);
    __syncthreads();
    int n = s0 == 0 ? 0 : n_items, units = s0 == 0 ? 0 : n_units;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      const int2 x = warp_sum[w];
      if (w < warp) n += x.x, units += x.y;
    }
    if (c.x >= 0) item[n + __popc(m & ((1u << lane) - 1u))] = make_int4(s, c.y, c.x, units + scan - mine);
    __syncthreads();
    if (threadIdx.x == 32 * kMergeWarps - 1) {
      n_items = n + __popc(m);
      n_units = units + scan;
    }
    __syncthreads();
  }
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    int lo = 0, hi = n_items - 1;          // the last token whose units begin at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item[mid].w <= u) lo = mid; else hi = mid - 1;
    }
    const int4 it = item[lo];
    const int n = it.y - it.x + 1;
    const bool by_warp = n <= kWarpParts;
    const int h = by_warp ? (u - it.w) * kMergeWarps + warp : (u - it.w) / nq;
    const int g = h / kHeads, hl = h % kHeads;
    // part i: the first slice's second slot, then every later slice's first
    const auto slot = [&](int i) { return (((size_t)(it.x + i) * groups + g) * 2 + (i == 0 ? 1 : 0)) * kHeads + hl; };
    __nv_bfloat16* row = out + ((size_t)it.z * H + h) * L;
    if (by_warp) {
      if (h >= H) continue;
      // (a lane's four channels of every 128; parts past n count as the first with weight 0)
      float4 v[2][4];
      const auto load = [&](int i0) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float* src = part + slot(i0 + z < n ? i0 + z : i0) * L;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int d = 4 * lane + 128 * q;
            v[z][q] = d < L ? *reinterpret_cast<const float4*>(src + d) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      };
      const float mine = lane < n ? lse[slot(lane)] : -INFINITY;
      load(0);
      float4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      float M = mine;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float ref = M == -INFINITY ? 0.f : M;
      const float w = exp2f(mine - ref);
      float tot = w;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      const float inv = M == -INFINITY ? 0.f : 1.f / tot;
      for (int i0 = 0; i0 < n; i0 += 2) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float f = __shfl_sync(0xffffffffu, w * inv, i0 + z);
          if (i0 + z >= n) break;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[q].x = fmaf(f, v[z][q].x, acc[q].x);
            acc[q].y = fmaf(f, v[z][q].y, acc[q].y);
            acc[q].z = fmaf(f, v[z][q].z, acc[q].z);
            acc[q].w = fmaf(f, v[z][q].w, acc[q].w);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 4 * lane + 128 * q;
        if (d < L)
          *reinterpret_cast<uint2*>(row + d) = make_uint2(pack_bf16x2(acc[q].x, acc[q].y),
                                                          pack_bf16x2(acc[q].z, acc[q].w));
      }
      continue;
    }
    // kParts parts in flight, weighted against the largest of this warp's so far
    const int d = 128 * ((u - it.w) % nq) + 4 * lane;      // (L may end inside the last 128)
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, tot = 0.f;
    for (int i0 = warp; i0 < n; i0 += kParts * kMergeWarps) {
      float e[kParts];
      float4 v[kParts];
#pragma unroll
      for (int z = 0; z < kParts; ++z) {
        const int i = i0 + z * kMergeWarps;
        e[z] = -INFINITY;
        v[z] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          const size_t at = slot(i);
          e[z] = lse[at];
          if (d < L) v[z] = *reinterpret_cast<const float4*>(part + at * L + d);
        }
      }
      float mx = M;
#pragma unroll
      for (int z = 0; z < kParts; ++z) mx = fmaxf(mx, e[z]);
      // (a NaN among the parts' sums is not seen by the maximum but comes back in its weight)
      const float ref = mx == -INFINITY ? 0.f : mx, f = exp2f(M - ref);
      M = mx;
      tot *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int z = 0; z < kParts; ++z) {
        const float w = exp2f(e[z] - ref);
        tot += w;
        acc.x = fmaf(w, v[z].x, acc.x);
        acc.y = fmaf(w, v[z].y, acc.y);
        acc.z = fmaf(w, v[z].z, acc.z);
        acc.w = fmaf(w, v[z].w, acc.w);
      }
    }
    *reinterpret_cast<float4*>(&sum[warp][4 * lane]) = acc;
    if (lane == 0) stat[warp] = make_float2(M, tot);
    __syncthreads();
    const int e = 2 * threadIdx.x, de = 128 * ((u - it.w) % nq) + e;
    if (threadIdx.x < 64 && de < L) {
      float all = -INFINITY, t = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) all = fmaxf(all, stat[w].x);
      const float ref = all == -INFINITY ? 0.f : all;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = exp2f(stat[w].x - ref);
        t = fmaf(f, stat[w].y, t);
        x = fmaf(f, sum[w][e], x);
        y = fmaf(f, sum[w][e + 1], y);
      }
      // (t is 0 where no part has an entry, NaN where a part's sum is)
      const float inv = t == 0.f ? 0.f : 1.f / t;
      *reinterpret_cast<uint32_t*>(row + de) = pack_bf16x2(x * inv, y * inv);
    }
    __syncthreads();
  }
}

int slices_of(const LatentDecodeArgs& a, int sms) {
  const int groups = (a.H + kHeads - 1) / kHeads;
  int s = sms / groups;
  if (s > kMergeMaxCuts) s = kMergeMaxCuts;
  return s < 1 ? 1 : s;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Workspace {
  size_t cut, lse, part, codes, scale, bytes;
};
Workspace workspace_layout(const LatentDecodeArgs& a, bool fp8, int sms) {
  const size_t ctas = (size_t)slices_of(a, sms) * ((a.H + kHeads - 1) / kHeads);
  Workspace w;
  w.cut = 0;
  w.lse = align256(ctas * sizeof(int2));
  w.part = w.lse + align256(ctas * 2 * kHeads * sizeof(float));
  w.codes = align256(w.part + ctas * 2 * kHeads * (size_t)a.pool.L * sizeof(float));
  const size_t tokens = fp8 ? (size_t)a.T * ((a.H + kHeads - 1) / kHeads) : 0;
  w.scale = w.codes + tokens * ((a.pool.L + 2 * a.pool.R + 127) / 128) * 16384;
  w.bytes = w.scale + tokens * kHeads * sizeof(float);
  return w;
}

template <bool kFp8>
cudaError_t launch(const DecodeParams& p, cudaStream_t stream, unsigned grid) {
  using C = Cfg<kFp8>;
  return launch_with_pdl(latent_decode_kernel<kFp8>, dim3(grid), dim3(kThreads), C::kSmem, stream,
                         kFp8, p);
}

}  // namespace

cudaError_t prepare_latent_decode() {
  const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel<false>, most, Cfg<false>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_decode_kernel<true>, most, Cfg<true>::kSmem);
  return e;
}

size_t latent_decode_workspace(const LatentDecodeArgs& a, bool fp8, int sms) {
  return workspace_layout(a, fp8, sms).bytes;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void* workspace, int sms,
                                 cudaStream_t stream) {
  DecodeParams p = {};
  p.a = a;
  p.groups = (a.H + kHeads - 1) / kHeads;
  p.slices = slices_of(a, sms);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const Workspace w = workspace_layout(a, fp8, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cut = reinterpret_cast<int2*>(ws + w.cut);
  p.lse = reinterpret_cast<float*>(ws + w.lse);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.q_codes = ws + w.codes;
  p.q_scale = reinterpret_cast<float*>(ws + w.scale);
  // Pages of a multiple of 64 entries: a tile is 64 consecutive rows, and one tensor-map copy brings all
  // its whole 128-byte chunks in slot order (bf16: pairs of the two halves, so only where all pair
  // up); the chunks left over come one by one.  Other pages: cp.async, any row anywhere.
  p.boxed = a.pool.ps % kKeys == 0;
  if (p.boxed) {
    const long long rows = a.pool.num_blocks * a.pool.ps;
    const unsigned long long W = a.pool.row_bytes;
    const int nl = a.pool.L / 64;
    const unsigned long long cd[2] = {W, (unsigned long long)rows}, cs[1] = {W};
    const unsigned cb[2] = {128, kKeys};
    if (!encode_bytes(&p.chunk, a.pool.rows, 2, cd, cs, cb)) return cudaErrorInvalidValue;
    if (fp8 && W >= 128) {
      p.whole = (int)(W / 128);
      const unsigned long long d[3] = {128, (unsigned long long)rows, W / 128}, st[2] = {W, 128};
      const unsigned bx[3] = {128, kKeys, (unsigned)p.whole};
      if (!encode_bytes(&p.block, a.pool.rows, 3, d, st, bx)) return cudaErrorInvalidValue;
    } else if (!fp8 && nl % 2 == 0) {
      p.whole = nl;
      const unsigned long long half = nl / 2;
      const unsigned long long d[4] = {128, (unsigned long long)rows, 2, half}, st[3] = {W, half * 128, 128};
      const unsigned bx[4] = {128, kKeys, 2, (unsigned)half};
      if (!encode_bytes(&p.block, a.pool.rows, 4, d, st, bx)) return cudaErrorInvalidValue;
    }
  }
  const unsigned grid = (unsigned)p.slices * (unsigned)p.groups;
  cudaError_t e;
  if (fp8) {
    // The codes first.  Not as a dependent grid itself, so that what the decode kernel reads before it
    // waits for the codes is there.
    const long long units = (long long)a.T * p.groups * (kHeads / 8);
    const unsigned blocks = (unsigned)(units < 8LL * sms ? units : 8LL * sms);
    e = launch_with_pdl(latent_q_kernel, dim3(blocks), dim3(256), 0, stream, false, a, p.groups, p.q_codes,
                        p.q_scale);
    if (e == cudaSuccess) e = launch<true>(p, stream, grid);
  } else {
    e = launch<false>(p, stream, grid);
  }
  if (e != cudaSuccess) return e;
  // (no more units than this; blocks without one would only delay the others' start)
  const long long units = (long long)a.T * a.H * ((a.pool.L + 127) / 128);
  const unsigned blocks = (unsigned)(units < 4LL * sms ? units : 4LL * sms);
  return launch_with_pdl(latent_merge_kernel, dim3(blocks), dim3(32 * kMergeWarps), 0, stream, true,
                         (const int2*)p.cut, (const float*)p.lse, (const float*)p.part,
                         reinterpret_cast<__nv_bfloat16*>(a.out), p.slices, p.groups, a.H, a.pool.L);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t latent_decode_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
