// spa_latent_decode.cu - absorbed latent attention over the paged cache: every head of a query
// attends to the same rows x_j = [c_j | r_j], which are its keys and (their latent part) its values.
//
//   s_j = scale (q_c . c_j + q_r . r_j),   out = sum_j softmax(s)_j c_j,   j <= position
//
// Each row is read once from HBM and used by every head: 2 (2L + R) flops a head and row, so 64 heads
// do about 121 flops a byte of a bf16 row (L = 512, R = 64) and 128 heads 242, where the machine
// turns from HBM-bound to tensor-bound.  Both limits matter, so the products run on the tcgen05 tensor
// cores from one copy of the row in shared memory:
//
//   S^T[j][h] = x_j . q_h          M = 64 entries, N = heads: A = rows (K-major)
//   O^T[d][h] += c_j[d] P^T[j][h]  M = 128 latent channels, N = 64 heads: A = the same rows read
//                                  MN-major, B = P^T
//
// A CTA holds q of one token's 64 heads and streams tiles of 64 entries through two (bf16) or three
// (e4m3) buffers by tensor-map copies, so that a tile is loaded while another is multiplied.  O^T
// takes 256 TMEM columns, which leaves room for two S^T buffers: S of the next tile is computed
// before the softmax of the current one is done.
//
//   warps 0-3   softmax: S^T from TMEM as fragments (16 entries x 64 heads a warp, two rows and 16
//               heads a thread), online maximum and sums, P^T to shared memory, epilogue
//   warp 4      issues the MMAs
//   warp 5      schedule, page tables, tensor-map copies
//   warps 6-9   (e4m3 only) q as two e4m3 terms
//
// Schedule: the tiles of all tokens are one long line; each slice of CTAs (one CTA for every 64
// heads) takes an equal stretch of it.  So the work is balanced whatever the sequence lengths,
// without knowing them on the host.  A token whose tiles lie in one slice is finished there;
// the parts of a token that was cut go to the workspace, normalised, with their log-sum-exp, and
// latent_merge_kernel joins them in the order of the slices.
//
// e4m3 rows enter the MMAs as codes.  q becomes q_hi + q_lo (e4m3, times a power of two per token
// and 64 heads), read as N = 128; the row's scale multiplies the score.  The weights p_j scale_j
// enter as an e5m2 and an e4m3 term: the first has the exponents to keep small weights of long
// sequences (24 bits below the largest), the second the mantissa of the large ones.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_latent.h"
#include "spa_launch.h"

namespace spa {

namespace {

constexpr int kHeads = 64;        // heads of a CTA
constexpr int kKeys = 64;         // entries of a tile
constexpr int kChunkBytes = kKeys * 128;
constexpr int kRing = 4;          // tile infos in flight
constexpr int kTmemCols = 512;
constexpr int kOCol = 256;        // first TMEM column of O^T
constexpr int kMinTiles = 2;      // tiles of a slice at least: fewer would cost more in merging

enum { kFirst = 1, kLast = 2, kEnd = 4 };

template <bool kFp8>
struct Cfg {
  static constexpr int kBufs = kFp8 ? 3 : 2;
  static constexpr int kChunks = kFp8 ? 5 : 9;       // 128-byte chunks of a row
  static constexpr int kGroupChunks = kFp8 ? 1 : 2;  // chunks of 128 channels
  static constexpr int kGroups = 5;                  // barriers a buffer
  static constexpr int kBufBytes = kChunks * kChunkBytes;
  static constexpr int kQRows = kFp8 ? 2 * kHeads : kHeads;
  static constexpr int kQChunk = kQRows * 128;
  static constexpr int kSCols = kFp8 ? 128 : 64;
  static constexpr int kThreads = kFp8 ? 320 : 192;
  static constexpr float kTau = kFp8 ? 1.f : 8.f;    // lazy rescale threshold (log2 units)
  struct Info {
    int t, flags, slot, pad;
    uint32_t even, odd;                              // bit k: entry 2k (2k + 1) takes part
    uint32_t pad2[2];
    float scale[kFp8 ? kKeys : 4];
  };
  static constexpr int kKOff = 0;
  static constexpr int kQOff = kBufs * kBufBytes;
  static constexpr int kPOff = kQOff + kChunks * kQChunk;
  static constexpr int kRedOff = kPOff + 8192;                       // float2 [2][4][32]
  static constexpr int kInfoOff = kRedOff + 2 * 4 * 32 * 8;
  static constexpr int kBarOff = kInfoOff + kRing * (int)sizeof(Info);
  // barriers
  static constexpr int kFullB = 0, kEmptyB = kBufs * kGroups, kQFullB = 2 * kBufs * kGroups,
                       kQEmptyB = kQFullB + 1, kSFullB = kQFullB + 2, kSEmptyB = kSFullB + 2,
                       kPFullB = kSEmptyB + 2, kPvDoneB = kPFullB + 1, kOFreeB = kPFullB + 2,
                       kInfoFullB = kPFullB + 3, kInfoEmptyB = kInfoFullB + kRing,
                       kDrainB = kInfoEmptyB + kRing, kRedB = kDrainB + 1, kQRedB = kRedB + 2,
                       kNumB = kQRedB + 1;
  // TMEM base, abort flag, q scales [4], q maxima of the q warps [2][4]
  static constexpr int kMiscOff = kBarOff + kNumB * 8;
  static constexpr int kSmem = kMiscOff + 8 + 16 + 32;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct DecodeParams {
  CUtensorMap rows;            // the pool's rows, boxes of box_rows rows (one row for gathers)
  CUtensorMap ql, qr;          // bf16 pools: q as [T][H][width], boxes of 64 heads
  LatentDecodeArgs a;
  int box_rows;                // 0: gathers of four single rows
  int groups;                  // of 64 heads
  int slices;
  float scale_log2;
  int2* cut;                   // [slices * groups]: the token cut at the end of a slice, its last slice
  float* lse;                  // [slices * groups][2][64], log2 units
  float* part;                 // [slices * groups][2][64][L]
};

__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kKeys - 1) / kKeys : 1; }

// Entries of token t (0 for a token that attends to nothing) and its sequence.
__device__ __forceinline__ int token_len(const LatentDecodeArgs& a, int t, int& b, bool& bad) {
  const int pos = __ldg(a.positions + t);
  b = a.seq_of_token ? __ldg(a.seq_of_token + t) : 0;
  long long cap = (long long)a.pool.bt_stride * a.pool.ps;
  cap = cap < 0x7fffffc0LL ? cap : 0x7fffffc0LL;   // (a tile's entries stay below 2^31)
  bad = b < 0 || b >= a.pool.B || (long long)pos >= cap;
  if (b < 0 || b >= a.pool.B || pos < 0) return 0;
  return (int)((long long)pos + 1 < cap ? (long long)pos + 1 : cap);
}

template <bool kFp8>
__global__ void __launch_bounds__(Cfg<kFp8>::kThreads, 1)
    latent_decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kMiscOff + 4);
  volatile float* q_scales = reinterpret_cast<volatile float*>(sm + C::kMiscOff + 8);
  typename C::Info* infos = reinterpret_cast<typename C::Info*>(sm + C::kInfoOff);
#define BAR(i) (sb + (uint32_t)C::kBarOff + 8u * (uint32_t)(i))

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBufs * C::kGroups; ++i) {
      mbar_init(BAR(C::kFullB + i), 1);
      mbar_init(BAR(C::kEmptyB + i), 1);
    }
    mbar_init(BAR(C::kQFullB), kFp8 ? 128 : 1);
    mbar_init(BAR(C::kQEmptyB), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::kSFullB + i), 1);
      mbar_init(BAR(C::kSEmptyB + i), 128);
    }
    mbar_init(BAR(C::kPFullB), 128);
    mbar_init(BAR(C::kPvDoneB), 1);
    mbar_init(BAR(C::kOFreeB), 128);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(BAR(C::kInfoFullB + i), 1);
      mbar_init(BAR(C::kInfoEmptyB + i), kFp8 ? 9 : 5);
    }
    mbar_init(BAR(C::kDrainB), 1);
    mbar_init(BAR(C::kRedB), 4);
    mbar_init(BAR(C::kRedB + 1), 4);
    mbar_init(BAR(C::kQRedB), 4);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4) tmem_alloc(sb + C::kMiscOff, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::kMiscOff);
  pdl_launch_dependents();
  pdl_wait();   // nothing global before the grid before this one is done

  const LatentDecodeArgs& a = p.a;
  const int L = a.pool.L, R = a.pool.R, W = a.pool.row_bytes;
  const int n_chunks = (W + 127) >> 7;
  const int n_groups = (n_chunks + C::kGroupChunks - 1) / C::kGroupChunks;
  const int n_mt = (L + 127) >> 7;             // 128-channel tiles of O^T (groups that hold values)
  const int g = blockIdx.x % p.groups;         // this CTA's 64 heads
  const int slice = blockIdx.x / p.groups;

  if (warp == 5) {
    // ================================ schedule and loads ==================================
    long long total = 0;
    for (int t = lane; t < a.T; t += 32) {
      int b;
      bool bad;
      total += tiles_of(token_len(a, t, b, bad));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    long long per = (total + p.slices - 1) / p.slices;
    if (per < kMinTiles) per = kMinTiles;
    const long long begin = per * slice;
    const long long end = begin + per < total ? begin + per : total;

    // the iterator: token t of the chunk of 32 whose lengths and sequences the lanes hold
    int t0 = 0, c_len = 0, c_seq = 0, c_bad = 0;
    auto load_chunk = [&](int at) {
      t0 = at;
      const int t = at + lane;
      c_len = c_seq = c_bad = 0;
      if (t < a.T) {
        bool bad;
        c_len = token_len(a, t, c_seq, bad);
        c_bad = bad;
      }
    };
    int it_t = 0, it_j = 0;                    // next tile: token, tile of the token
    long long it_pos = begin;                  // its place in the line
    if (begin < end) {
      long long before = 0;
      for (load_chunk(0);; load_chunk(t0 + 32)) {
        const int n = t0 + lane < a.T ? tiles_of(c_len) : 0;
        int sum = n;                           // inclusive scan (32 tokens: below 2^31 tiles)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (begin < before + all) {
          const unsigned m = __ballot_sync(0xffffffffu, begin < before + sum);
          const int k = __ffs(m) - 1;
          it_t = t0 + k;
          it_j = (int)(begin - before - (__shfl_sync(0xffffffffu, sum, k) -
                                         __shfl_sync(0xffffffffu, n, k)));
          break;
        }
        before += all;
      }
    }
    struct Tile {
      int t, flags, slot, n;                   // n: entries of the tile that are in the sequence
      int blk[2], off[2];                      // block of entries 2 lane, 2 lane + 1 (-1: none)
    };
    int started = it_j == 0;                   // the current token's first tile is this CTA's
    bool fresh = true;
    int2 cut = make_int2(-1, 0);
    auto next_tile = [&](Tile& x) {            // the next tile, its block-table reads under way
      x.t = -1;
      if (it_pos >= end) return;
      if (it_t >= t0 + 32) load_chunk(it_t);
      const int k = it_t - t0;
      const int len = __shfl_sync(0xffffffffu, c_len, k);
      const int b = __shfl_sync(0xffffffffu, c_seq, k);
      const int bad = __shfl_sync(0xffffffffu, c_bad, k);
      if (bad && it_j == 0 && lane == 0) flag_error(SPA_ERR_INDEX);
      const int nt = tiles_of(len);
      x.t = it_t;
      x.n = min(kKeys, len - it_j * kKeys);
      const bool item_end = it_j == nt - 1;
      const bool last = item_end || it_pos == end - 1;
      x.flags = (fresh ? kFirst : 0) | (last ? kLast : 0);
      x.slot = started && item_end ? -1 : started;
      if (last && !item_end && started)
        cut = make_int2(it_t, (int)((it_pos + (nt - 1 - it_j)) / per));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * lane + e;
        x.blk[e] = -2;                         // not of the sequence
        x.off[e] = 0;
        if (j < x.n) {
          const int key = it_j * kKeys + j;
          const int page = key / a.pool.ps;
          x.off[e] = key - page * a.pool.ps;
          x.blk[e] = __ldg(a.pool.bt + (size_t)b * a.pool.bt_stride + page);
        }
      }
      fresh = last;
      ++it_pos;
      ++it_j;
      if (item_end) {
        ++it_t;
        it_j = 0;
        started = 1;
      }
    };
    Tile cur, nxt, nxt2;
    float sc_cur[2] = {0.f, 0.f};
    int row_cur[2] = {-1, -1};
    auto resolve = [&](const Tile& x, int (&row)[2], float (&sc)[2]) {
      row[0] = row[1] = -1;
      if (x.t < 0) return;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (x.blk[e] >= 0 && (long long)x.blk[e] < a.pool.num_blocks)
          row[e] = (int)((long long)x.blk[e] * a.pool.ps + x.off[e]);
        else if (x.blk[e] != -2)
          flag_error(SPA_ERR_INDEX);
        sc[e] = kFp8 && row[e] >= 0 ? __ldg(a.pool.scale + row[e]) : 0.f;
      }
    };
    next_tile(cur);
    next_tile(nxt);
    next_tile(nxt2);
    resolve(cur, row_cur, sc_cur);
    const int total_rows = (int)(a.pool.num_blocks * a.pool.ps);
    const int nb = p.box_rows > 0 ? kKeys / p.box_rows : kKeys / 4;   // copies a chunk
    int k = 0, items = 0;
    bool ok = true;
    for (; cur.t >= 0 && ok; ++k) {
      int row_nxt[2];
      float sc_nxt[2] = {0.f, 0.f};
      resolve(nxt, row_nxt, sc_nxt);
      Tile nxt3;
      next_tile(nxt3);
      // publish the tile
      const int ri = k % kRing;
      if (lane == 0) ok = mbar_wait(BAR(C::kInfoEmptyB + ri), ((k / kRing) & 1) ^ 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const unsigned even = __ballot_sync(0xffffffffu, row_cur[0] >= 0);
      const unsigned odd = __ballot_sync(0xffffffffu, row_cur[1] >= 0);
      typename C::Info& info = infos[ri];
      if (kFp8) {
        info.scale[2 * lane] = sc_cur[0];
        info.scale[2 * lane + 1] = sc_cur[1];
      }
      if (lane == 0) {
        info.t = cur.t;
        info.flags = cur.flags;
        info.slot = cur.slot;
        info.even = even;
        info.odd = odd;
      }
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kInfoFullB + ri));
      // q of a new token
      if (!kFp8 && (cur.flags & kFirst)) {
        if (lane == 0) {
          ok = mbar_wait(BAR(C::kQEmptyB), (items & 1) ^ 1, abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(BAR(C::kQFullB), (uint32_t)(n_chunks * C::kQChunk));
            for (int c = 0; c < n_chunks; ++c) {
              const uint32_t dst = sb + C::kQOff + c * C::kQChunk;
              if (64 * c < L)
                tma_box3(dst, &p.ql, 64 * c, g * kHeads, cur.t, BAR(C::kQFullB));
              else
                tma_box3(dst, &p.qr, 0, g * kHeads, cur.t, BAR(C::kQFullB));
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++items;
        if (!ok) break;
      }
      // the rows, group by group: lane o issues copy o of the group
      const int buf = k % C::kBufs;
      for (int gr = 0; gr < n_groups && ok; ++gr) {
        const int bi = buf * C::kGroups + gr;
        const int nc = min(C::kGroupChunks, n_chunks - gr * C::kGroupChunks);
        if (lane == 0) {
          ok = mbar_wait(BAR(C::kEmptyB + bi), ((k / C::kBufs) & 1) ^ 1, abort_flag);
          mbar_arrive_expect_tx(BAR(C::kFullB + bi), ok ? (uint32_t)(nc * kChunkBytes) : 0u);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        const int cc = lane / nb, box = lane % nb;   // (at most 16 copies a chunk, two chunks)
        const int c = gr * C::kGroupChunks + cc;
        const uint32_t dst0 = sb + C::kKOff + buf * C::kBufBytes + c * kChunkBytes;
        if (p.box_rows > 0) {
          const int row = __shfl_sync(0xffffffffu, row_cur[0], (box * p.box_rows) >> 1);
          // a box with no entry starts past the last row and is filled with zeros
          if (ok && cc < nc)
            tma_row(dst0 + box * p.box_rows * 128, &p.rows, c * 128, row >= 0 ? row : total_rows,
                    BAR(C::kFullB + bi));
        } else {
          const int r0 = __shfl_sync(0xffffffffu, row_cur[0], 2 * box);
          const int r1 = __shfl_sync(0xffffffffu, row_cur[1], 2 * box);
          const int r2 = __shfl_sync(0xffffffffu, row_cur[0], 2 * box + 1);
          const int r3 = __shfl_sync(0xffffffffu, row_cur[1], 2 * box + 1);
          // (a missing row is read as row 0; the softmax warps blank it)
          if (ok && cc < nc)
            tma_gather4(dst0 + box * 4 * 128, &p.rows, c * 128, max(r0, 0), max(r1, 0), max(r2, 0),
                        max(r3, 0), BAR(C::kFullB + bi));
        }
      }
      cur = nxt;
      nxt = nxt2;
      nxt2 = nxt3;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_cur[e] = row_nxt[e];
        sc_cur[e] = sc_nxt[e];
      }
    }
    if (lane == 0) {
      if (ok && !*abort_flag) {
        const int ri = k % kRing;
        if (mbar_wait(BAR(C::kInfoEmptyB + ri), ((k / kRing) & 1) ^ 1, abort_flag)) {
          infos[ri].flags = kEnd;
          __threadfence_block();
          mbar_arrive(BAR(C::kInfoFullB + ri));
        }
      }
      p.cut[blockIdx.x] = cut;
      // copies in flight must land before the CTA ends (at once after a normal run)
      for (int q = max(0, k - C::kBufs); q < k; ++q)
        for (int gr = 0; gr < n_groups; ++gr)
          mbar_wait_drain(BAR(C::kFullB + (q % C::kBufs) * C::kGroups + gr),
                          (uint32_t)((q / C::kBufs) & 1));
      if (!kFp8 && items > 0) mbar_wait_drain(BAR(C::kQFullB), (uint32_t)((items - 1) & 1));
    }
  } else if (warp == 4) {
    // ====================================== MMA ===========================================
    if (lane == 0) {
      const uint32_t idS = kFp8 ? idesc_e4m3(64, 128, 0, 0) : idesc_bf16(64, 64, 0, 0);
      const uint32_t idO = kFp8 ? idesc_e4m3(128, 64, 1, 1) : idesc_bf16(128, 64, 1, 1);
      const uint32_t idO5 = idO | (1u << 10);            // B in e5m2: the high term of P
      const uint64_t dq0 = sdesc(sb + C::kQOff, 16, 1024);
      const uint64_t dp0 = kFp8 ? sdesc64(sb + C::kPOff, 4096, 512) : sdesc(sb + C::kPOff, 8192, 1024);
      int ks = 0, kp = 0;                                 // tiles whose S, PV were issued
      uint32_t q_ph = 0, o_ph = 0;
      auto issue_s = [&](int flags) -> bool {
        const int buf = ks % C::kBufs, s = ks & 1;
        if (flags & kFirst) {
          if (!mbar_wait(BAR(C::kQFullB), q_ph, abort_flag)) return false;
          q_ph ^= 1;
        }
        if (!mbar_wait(BAR(C::kSEmptyB + s), ((ks >> 1) & 1) ^ 1, abort_flag)) return false;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t dS = tmem + s * C::kSCols;
        for (int gr = 0; gr < n_groups; ++gr) {
          const int bi = buf * C::kGroups + gr;
          if (!mbar_wait(BAR(C::kFullB + bi), (uint32_t)((ks / C::kBufs) & 1), abort_flag)) return false;
          tc_fence_after();
          for (int cc = 0; cc < C::kGroupChunks; ++cc) {
            const int c = gr * C::kGroupChunks + cc;
            if (c >= n_chunks) break;
            const uint64_t da = sdesc(sb + C::kKOff + buf * C::kBufBytes + c * kChunkBytes, 16, 1024);
            const uint64_t db = desc_add(dq0, c * C::kQChunk);
            const int steps = min(4, (W - c * 128 + 31) >> 5);
            for (int st = 0; st < steps; ++st) {
              if (kFp8)
                mma_f8(dS, desc_add(da, st * 32), desc_add(db, st * 32), idS, (c | st) != 0);
              else
                mma_bf16(dS, desc_add(da, st * 32), desc_add(db, st * 32), idS, (c | st) != 0);
            }
          }
          if (gr >= n_mt) mma_commit(BAR(C::kEmptyB + bi));   // no values in this group
        }
        mma_commit(BAR(C::kSFullB + s));
        if (flags & kLast) mma_commit(BAR(C::kQEmptyB));
        ++ks;
        return true;
      };
      auto issue_pv = [&](int flags) -> bool {
        const int buf = kp % C::kBufs;
        if (!mbar_wait(BAR(C::kPFullB), (uint32_t)(kp & 1), abort_flag)) return false;
        const bool first = flags & kFirst;
        if (first) {
          if (!mbar_wait(BAR(C::kOFreeB), o_ph ^ 1, abort_flag)) return false;
          o_ph ^= 1;
        }
        fence_proxy_async_smem();
        tc_fence_after();
        for (int mt = 0; mt < n_mt; ++mt) {
          const uint32_t dO = tmem + kOCol + mt * 64;
          const uint32_t kv = sb + C::kKOff + buf * C::kBufBytes + mt * C::kGroupChunks * kChunkBytes;
          const uint64_t dv = sdesc(kv, kChunkBytes, 1024);
          if (!kFp8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)               // 16 entries a step
              mma_bf16(dO, desc_add(dv, kk * 2048), desc_add(dp0, kk * 2048), idO,
                       (first && kk == 0) ? 0u : 1u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {             // 32 entries a step
              mma_f8(dO, desc_add(dv, kk * 4096), desc_add(dp0, kk * 2048), idO5,
                     (first && kk == 0) ? 0u : 1u);
              mma_f8(dO, desc_add(dv, kk * 4096), desc_add(dp0, 4096 + kk * 2048), idO, 1u);
            }
          }
          mma_commit(BAR(C::kEmptyB + buf * C::kGroups + mt));
        }
        mma_commit(BAR(C::kPvDoneB));
        ++kp;
        return true;
      };
      // S of tile k + 1 is issued before PV of tile k, except where a new token begins
      int flags_s = 0, ki = 0;
      auto read_info = [&](int& flags) -> bool {
        const int ri = ki % kRing;
        if (!mbar_wait(BAR(C::kInfoFullB + ri), (uint32_t)((ki / kRing) & 1), abort_flag)) return false;
        flags = *reinterpret_cast<volatile int*>(&infos[ri].flags);
        mbar_arrive(BAR(C::kInfoEmptyB + ri));
        ++ki;
        return true;
      };
      bool ok = read_info(flags_s);
      while (ok && !(flags_s & kEnd)) {
        ok = issue_s(flags_s);
        while (ok) {
          const int flags_p = flags_s;
          if (!(flags_p & kLast)) {
            ok = read_info(flags_s) && issue_s(flags_s);
            if (!ok) break;
          }
          ok = issue_pv(flags_p);
          if (flags_p & kLast) break;
        }
        if (ok) ok = read_info(flags_s);
      }
      // nothing may still write TMEM when it is released
      mma_commit(BAR(C::kDrainB));
      mbar_wait_drain(BAR(C::kDrainB), 0);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ======================= q as two e4m3 terms (e4m3 pools only) ========================
    if constexpr (kFp8) {
      const int tid = threadIdx.x - 192;
      volatile float* qmax = reinterpret_cast<volatile float*>(sm + C::kMiscOff + 24);
      int items = 0;
      for (int k = 0;; ++k) {
        const int ri = k % kRing;
        if (!warp_wait(BAR(C::kInfoFullB + ri), (uint32_t)((k / kRing) & 1), abort_flag)) break;
        const int flags = infos[ri].flags, t = infos[ri].t;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::kInfoEmptyB + ri));
        if (flags & kEnd) break;
        if (!(flags & kFirst)) continue;
        const int nl = L >> 3, nr = R >> 3, np = nl + 2 * nr;    // pieces of eight values of K
        const int npad = n_chunks * 16;                          // pieces of the padded row
        auto piece = [&](int h, int i) {                         // q's values of piece i, or zeros
          const int hg = g * kHeads + h;
          if (hg >= a.H || i >= np) return make_uint4(0, 0, 0, 0);
          const uint8_t* src = i < nl ? a.q_latent + t * a.ql_st + hg * a.ql_sh + 16 * i
                                      : a.q_rope + t * a.qr_st + hg * a.qr_sh + 16 * ((i - nl) % nr);
          return __ldg(reinterpret_cast<const uint4*>(src));
        };
        float m = 0.f;
        for (int i = tid; i < kHeads * (nl + nr); i += 128) {
          const uint4 u = piece(i / (nl + nr), i % (nl + nr));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        volatile float* qm = qmax + 4 * (items & 1);
        if (lane == 0) {
          qm[warp - 6] = m;
          mbar_arrive(BAR(C::kQRedB));
        }
        if (!warp_wait(BAR(C::kQRedB), (uint32_t)(items & 1), abort_flag)) break;
        m = fmaxf(fmaxf(qm[0], qm[1]), fmaxf(qm[2], qm[3]));
        const float qs = m > 0.f ? pow2_floor(448.f / m) : 1.f;
        if (!warp_wait(BAR(C::kQEmptyB), (uint32_t)((items & 1) ^ 1), abort_flag)) break;
        if (tid == 0) q_scales[items & 3] = qs;
        for (int i = tid; i < kHeads * npad; i += 128) {
          const int h = i / npad, pc = i % npad;
          const uint4 u = piece(h, pc);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = bf16_lo(w[e]) * qs, y = bf16_hi(w[e]) * qs;
            hi[e] = e4m3x2(x, y);
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[e], __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            lo[e] = e4m3x2(x - v.x, y - v.y);
          }
          // piece pc: bytes 8 pc of the row, chunk pc / 16, 16-byte unit (pc / 2) & 7 swizzled by row
          const uint32_t off = (pc >> 4) * C::kQChunk + h * 128 + ((((pc >> 1) & 7) ^ (h & 7)) << 4) + (pc & 1) * 8;
          *reinterpret_cast<uint2*>(sm + C::kQOff + off) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(sm + C::kQOff + off + 64 * 128) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        }
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::kQFullB));
        ++items;
      }
    }
  } else {
    // ================================ softmax and epilogue ================================
    const int tid = threadIdx.x;
    const int fr = lane >> 2, fc = lane & 3;       // fragment row, column pair
    const int r0 = 16 * warp + fr, r1 = r0 + 8;    // this thread's entries of the tile
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    float2* red = reinterpret_cast<float2*>(sm + C::kRedOff);
    float2 m = make_float2(-INFINITY, -INFINITY);  // running maxima of heads 2 lane, 2 lane + 1
    float l[16];                                   // this thread's sums of heads 8i + 2fc + e
    int items = -1, reds = 0;                      // tokens begun, exchanges between the warps done
    // The warps' values of heads 2 lane, 2 lane + 1, all four in every thread: through one of two
    // buffers in turn, with a wait that ends (false) when the CTA gives up.
    auto exchange = [&](float2 mine, float2 (&all)[4]) -> bool {
      float2* rr = red + (reds & 1) * 128;
      rr[warp * 32 + lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kRedB + (reds & 1)));
      if (!warp_wait(BAR(C::kRedB + (reds & 1)), (uint32_t)((reds >> 1) & 1), abort_flag)) return false;
      ++reds;
#pragma unroll
      for (int w = 0; w < 4; ++w) all[w] = rr[w * 32 + lane];
      return true;
    };
    for (int k = 0;; ++k) {
      const int ri = k % kRing, s = k & 1;
      if (!warp_wait(BAR(C::kInfoFullB + ri), (uint32_t)((k / kRing) & 1), abort_flag)) break;
      const typename C::Info& info = infos[ri];
      const int t = info.t, flags = info.flags, slot = info.slot;
      const uint32_t even = info.even, odd = info.odd;
      float ks0 = 1.f, ks1 = 1.f;
      if (kFp8) ks0 = info.scale[r0], ks1 = info.scale[r1];
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::kInfoEmptyB + ri));
      if (flags & kEnd) break;
      const bool first = flags & kFirst, last = flags & kLast;
      // (r1 = r0 + 8 has r0's parity)
      const uint32_t word = (r0 & 1) ? odd : even;
      const bool v0 = (word >> (r0 >> 1)) & 1u, v1 = (word >> (r1 >> 1)) & 1u;
      if (first) {
        ++items;
        m = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int i = 0; i < 16; ++i) l[i] = 0.f;
      }
      if (!warp_wait(BAR(C::kSFullB + s), (uint32_t)((k >> 1) & 1), abort_flag)) break;
      tc_fence_after();
      float x[32];
      tmem_ld_frag64(lane_base + s * C::kSCols, x);
      float c0 = p.scale_log2, c1 = p.scale_log2, b0 = 0.f, b1 = 0.f;
      if (kFp8) {
        float y[32];
        tmem_ld_frag64(lane_base + s * C::kSCols + 64, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] += y[i];
        const float qi = p.scale_log2 / q_scales[items & 3];
        c0 = qi * ks0;
        c1 = qi * ks1;
        // the maximum is taken over p_j |scale_j|, the weights that enter the value product (a scale
        // below 2^-60 counts as that: the sums of p_j alone must stay finite)
        b0 = fmaxf(__log2f(fabsf(ks0)), -60.f);
        b1 = fmaxf(__log2f(fabsf(ks1)), -60.f);
      } else {
        tmem_wait_ld();
      }
      tc_fence_before();
      mbar_arrive(BAR(C::kSEmptyB + s));
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = (i & 2) ? (v1 ? x[i] * c1 : -INFINITY) : (v0 ? x[i] * c0 : -INFINITY);
      // tile maxima: over this thread's two entries, then over the eight lanes of equal fc, halving
      // the columns each step so that lane 4i + fc ends with columns 8i + 2fc, + 1
      float mx[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mx[2 * i] = fmaxf(x[4 * i] + b0, x[4 * i + 2] + b1);
        mx[2 * i + 1] = fmaxf(x[4 * i + 1] + b0, x[4 * i + 3] + b1);
      }
#pragma unroll
      for (int w = 8; w >= 2; w >>= 1) {           // 16 -> 8 -> 4 -> 2 values; lane bits 4, 3, 2
        const bool up = lane & (2 * w);
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const float send = up ? mx[i] : mx[i + w], keep = up ? mx[i + w] : mx[i];
          mx[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 2 * w));
        }
      }
      float2 ex[4];
      if (!exchange(make_float2(mx[0], mx[1]), ex)) break;
      const float2 mt = make_float2(fmaxf(fmaxf(ex[0].x, ex[1].x), fmaxf(ex[2].x, ex[3].x)),
                                    fmaxf(fmaxf(ex[0].y, ex[1].y), fmaxf(ex[2].y, ex[3].y)));
      const float2 mn = make_float2(mt.x > m.x + C::kTau ? mt.x : m.x, mt.y > m.y + C::kTau ? mt.y : m.y);
      const bool grow = __any_sync(0xffffffffu, mn.x != m.x || mn.y != m.y);
      // a head without any entry so far: everything is masked, the reference does not matter
      const float2 ref = make_float2(mn.x == -INFINITY ? 0.f : mn.x, mn.y == -INFINITY ? 0.f : mn.y);
      const float2 al = make_float2(fast_exp2(m.x - ref.x), fast_exp2(m.y - ref.y));
      m = mn;
      if (grow && !first) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          l[2 * i] *= __shfl_sync(0xffffffffu, al.x, 4 * i + fc);
          l[2 * i + 1] *= __shfl_sync(0xffffffffu, al.y, 4 * i + fc);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float mc0 = __shfl_sync(0xffffffffu, ref.x, 4 * i + fc);
        const float mc1 = __shfl_sync(0xffffffffu, ref.y, 4 * i + fc);
        x[4 * i] = fast_exp2(x[4 * i] - mc0);
        x[4 * i + 1] = fast_exp2(x[4 * i + 1] - mc1);
        x[4 * i + 2] = fast_exp2(x[4 * i + 2] - mc0);
        x[4 * i + 3] = fast_exp2(x[4 * i + 3] - mc1);
        l[2 * i] += x[4 * i] + x[4 * i + 2];
        l[2 * i + 1] += x[4 * i + 1] + x[4 * i + 3];
      }
      // P^T words: bf16 pairs, or four codes of each term gathered over a lane pair
      uint32_t pw[16];
      if (!kFp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pw[2 * i] = pack_bf16x2(x[4 * i], x[4 * i + 1]);
          pw[2 * i + 1] = pack_bf16x2(x[4 * i + 2], x[4 * i + 3]);
        }
      } else {
        // u = 2^7 p scale (at most 2^8, as tau = 1): e5m2, then e4m3 of what that leaves.  Invalid
        // rows have p = 0, but a scale that may be anything.
        const float s0 = v0 ? ks0 * 128.f : 0.f, s1 = v1 ? ks1 * 128.f : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t w2[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float ua = x[4 * i + 2 * r] * (r ? s1 : s0), ub = x[4 * i + 2 * r + 1] * (r ? s1 : s0);
            const uint32_t hi = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(ua, ub), __NV_SATFINITE, __NV_E5M2);
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E5M2);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            w2[r] = hi | (e4m3x2(ua - v.x, ub - v.y) << 16);
          }
          // even lanes take row r0's four codes (heads 8i + 2fc ..+3), odd lanes row r1's
          const uint32_t o = __shfl_xor_sync(0xffffffffu, (lane & 1) ? w2[0] : w2[1], 1);
          const uint32_t mine = (lane & 1) ? w2[1] : w2[0];
          const uint32_t lo_h = (lane & 1) ? o : mine, hi_h = (lane & 1) ? mine : o;
          pw[2 * i] = __byte_perm(lo_h, hi_h, 0x5410);       // high terms
          pw[2 * i + 1] = __byte_perm(lo_h, hi_h, 0x7632);   // low terms
        }
      }
      if (!first) {
        // PV of the tile before: then O can be rescaled and the P buffer reused
        if (!warp_wait(BAR(C::kPvDoneB), (uint32_t)((k - 1) & 1), abort_flag)) break;
        tc_fence_after();
        if (grow) {
          for (int hf = 0; hf < 2; ++hf) {
            for (int i = 0; i < n_mt; ++i) {
              float o[32];
              const uint32_t ta = lane_base + kOCol + i * 64 + hf * 32;
              tmem_ld32(ta, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c)
                o[c] *= __shfl_sync(0xffffffffu, (c & 1) ? al.y : al.x, hf * 16 + (c >> 1));
              tmem_st32(ta, o);
            }
          }
          tmem_wait_st();
        }
      }
      if (!kFp8) {
        uint8_t* p0 = sm + C::kPOff + r0 * 128 + fc * 4;     // (r1's swizzle is r0's: 8 apart)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          *reinterpret_cast<uint32_t*>(p0 + ((i ^ (r0 & 7)) << 4)) = pw[2 * i];
          *reinterpret_cast<uint32_t*>(p0 + 1024 + ((i ^ (r0 & 7)) << 4)) = pw[2 * i + 1];
        }
      } else {
        const int row = (lane & 1) ? r1 : r0;
        uint8_t* pr = sm + C::kPOff + row * 64 + (fc >> 1) * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {      // heads 8i + 4(fc / 2): 16-byte unit i / 2, half i & 1
          const int off = (((i >> 1) ^ ((row >> 1) & 3)) << 4) + (i & 1) * 8;
          *reinterpret_cast<uint32_t*>(pr + off) = pw[2 * i];
          *reinterpret_cast<uint32_t*>(pr + 4096 + off) = pw[2 * i + 1];
        }
      }
      if ((even & odd) != 0xffffffffu) {
        // entries that take no part: their rows hold other data or none, and a probability of zero
        // times a NaN would still be one
        const int buf = k % C::kBufs;
        const int u16 = n_mt * C::kGroupChunks * 8;          // 16-byte units of a row's values
        for (int e = 0; e < 2; ++e) {
          uint32_t gone = ~(e ? odd : even);
          while (gone) {
            const int r = 2 * (__ffs(gone) - 1) + e;
            gone &= gone - 1;
            for (int u = tid; u < u16 && (u >> 3) < n_chunks; u += 128)
              *reinterpret_cast<uint4*>(sm + C::kKOff + buf * C::kBufBytes + (u >> 3) * kChunkBytes +
                                        r * 128 + (u & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(BAR(C::kPFullB));
      if (!last) continue;

      // ---- epilogue: denominators, then O ----
#pragma unroll
      for (int w = 8; w >= 2; w >>= 1) {
        const bool up = lane & (2 * w);
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const float send = up ? l[i] : l[i + w], keep = up ? l[i + w] : l[i];
          l[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * w);
        }
      }
      if (!exchange(make_float2(l[0], l[1]), ex)) break;
      const float2 ls = make_float2((ex[0].x + ex[1].x) + (ex[2].x + ex[3].x),
                                    (ex[0].y + ex[1].y) + (ex[2].y + ex[3].y));
      constexpr float kUnit = kFp8 ? 1.f / 128.f : 1.f;
      const float2 inv = make_float2(m.x == -INFINITY ? 0.f : kUnit / ls.x, m.y == -INFINITY ? 0.f : kUnit / ls.y);
      const int Hg = min(kHeads, a.H - g * kHeads);
      const size_t pslot = (size_t)blockIdx.x * 2 + (slot > 0 ? 1 : 0);
      if (slot >= 0 && warp == 0) {
        float* le = p.lse + pslot * kHeads;
        le[2 * lane] = m.x == -INFINITY ? -INFINITY : m.x + __log2f(ls.x);
        le[2 * lane + 1] = m.y == -INFINITY ? -INFINITY : m.y + __log2f(ls.y);
      }
      if (!warp_wait(BAR(C::kPvDoneB), (uint32_t)(k & 1), abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        if (hf * 32 >= Hg) break;
        float iv[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
          iv[c] = __shfl_sync(0xffffffffu, (c & 1) ? inv.y : inv.x, hf * 16 + (c >> 1));
        const int nh = min(32, Hg - hf * 32);
#pragma unroll 1
        for (int i = 0; i < n_mt; ++i) {
          const int d = i * 128 + tid;
          float o[32];
          tmem_ld32(lane_base + kOCol + i * 64 + hf * 32, o);
          tmem_wait_ld();
          if (slot >= 0) {
            float* wo = p.part + (pslot * kHeads + hf * 32) * L + d;
            if (d < L) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c < nh) wo[(uint32_t)(c * L)] = o[c] * iv[c];
            }
          } else {
            // lanes 2m and 2m + 1 swap halves so that each stores two adjacent channels
            const bool up = lane & 1;
            __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(a.out) +
                                ((size_t)t * a.H + g * kHeads + hf * 32) * L + (d & ~1);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float x0 = o[c] * iv[c], x1 = o[c + 1] * iv[c + 1];
              const float recv = __shfl_xor_sync(0xffffffffu, up ? x0 : x1, 1);
              const uint32_t pr = up ? pack_bf16x2(recv, x1) : pack_bf16x2(x0, recv);
              const int hh = c + (up ? 1 : 0);
              if (hh < nh && d < L) *reinterpret_cast<uint32_t*>(ob + (uint32_t)(hh * L)) = pr;
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(BAR(C::kOFreeB));
    }
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the tokens that were cut: out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).
// A unit is one head of one such token; the eight warps of a block take every eighth part each, and
// add up in warp order.
constexpr int kMergeWarps = 8;
constexpr int kMergeMaxCuts = 1024;

__global__ void __launch_bounds__(32 * kMergeWarps)
    latent_merge_kernel(const int2* __restrict__ cut, const float* __restrict__ lse,
                        const float* __restrict__ part, __nv_bfloat16* __restrict__ out, int slices,
                        int groups, int H, int L) {
  __shared__ __align__(16) float sum[kMergeWarps][kLatMaxDim];
  __shared__ __align__(16) int2 item[kMergeMaxCuts];   // slice where the token begins, its last slice
  __shared__ int n_items;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (warp == 0) {
    int n = 0;
    for (int s0 = 0; s0 < slices; s0 += 32) {
      const int s = s0 + lane;
      const int2 c = s < slices ? cut[(size_t)s * groups] : make_int2(-1, 0);
      const unsigned m = __ballot_sync(0xffffffffu, c.x >= 0);
      if (c.x >= 0) item[n + __popc(m & ((1u << lane) - 1u))] = make_int2(s, c.y);
      n += __popc(m);
    }
    if (lane == 0) n_items = n;
  }
  __syncthreads();
  const long long units = (long long)n_items * H;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int2 it = item[u / H];
    const int h = (int)(u % H), g = h / kHeads, hl = h % kHeads;
    const int n = it.y - it.x + 1;
    // part i: the first slice's second slot, then every later slice's first
    const auto slot = [&](int i) { return ((size_t)(it.x + i) * groups + g) * 2 + (i == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, lse[slot(i) * kHeads + hl]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // (a NaN among the parts' sums is not seen by the maximum but comes back in its weight)
    const float ref = M == -INFINITY ? 0.f : M;
    float tot = 0.f;
    for (int i = lane; i < n; i += 32) tot += exp2f(lse[slot(i) * kHeads + hl] - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    float4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = warp; i < n; i += kMergeWarps) {
      const float w = exp2f(lse[slot(i) * kHeads + hl] - ref);
      const float* src = part + (slot(i) * kHeads + hl) * L;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int d = 4 * lane + 128 * q;
        if (d < L) {
          const float4 v = *reinterpret_cast<const float4*>(src + d);
          acc[q].x = fmaf(w, v.x, acc[q].x);
          acc[q].y = fmaf(w, v.y, acc[q].y);
          acc[q].z = fmaf(w, v.z, acc[q].z);
          acc[q].w = fmaf(w, v.w, acc[q].w);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<float4*>(&sum[warp][4 * lane + 128 * q]) = acc[q];
    __syncthreads();
    const int t = cut[(size_t)it.x * groups].x;
    const float inv = M == -INFINITY ? 0.f : 1.f / tot;
    for (int d = 2 * threadIdx.x; d < L; d += 2 * 32 * kMergeWarps) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        x += sum[w][d];
        y += sum[w][d + 1];
      }
      *reinterpret_cast<uint32_t*>(out + ((size_t)t * H + h) * L + d) = pack_bf16x2(x * inv, y * inv);
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
  size_t cut, lse, part, bytes;
};
Workspace workspace_layout(const LatentDecodeArgs& a, int sms) {
  const size_t ctas = (size_t)slices_of(a, sms) * ((a.H + kHeads - 1) / kHeads);
  Workspace w;
  w.cut = 0;
  w.lse = align256(ctas * sizeof(int2));
  w.part = w.lse + align256(ctas * 2 * kHeads * sizeof(float));
  w.bytes = w.part + ctas * 2 * kHeads * (size_t)a.pool.L * sizeof(float);
  return w;
}

template <bool kFp8>
cudaError_t launch(const DecodeParams& p, cudaStream_t stream, unsigned grid) {
  using C = Cfg<kFp8>;
  const cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel<kFp8>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_with_pdl(latent_decode_kernel<kFp8>, dim3(grid), dim3(C::kThreads), C::kSmem, stream,
                         false, p);
}

}  // namespace

size_t latent_decode_workspace(const LatentDecodeArgs& a, int sms) {
  return workspace_layout(a, sms).bytes;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void* workspace, int sms,
                                 cudaStream_t stream) {
  DecodeParams p = {};
  p.a = a;
  p.groups = (a.H + kHeads - 1) / kHeads;
  p.slices = slices_of(a, sms);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const Workspace w = workspace_layout(a, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cut = reinterpret_cast<int2*>(ws + w.cut);
  p.lse = reinterpret_cast<float*>(ws + w.lse);
  p.part = reinterpret_cast<float*>(ws + w.part);
  // Boxes of as many rows as divide a page and a tile: a box then lies in one page.  Pages that
  // leave fewer than four rows take gathers of four single rows instead.
  int box = a.pool.ps & -a.pool.ps;
  box = box > kKeys ? kKeys : box;
  p.box_rows = box >= 4 ? box : 0;
  const long long rows = a.pool.num_blocks * a.pool.ps;
  if (!encode_rows(&p.rows, a.pool.rows, rows, a.pool.row_bytes, p.box_rows > 0 ? p.box_rows : 1))
    return cudaErrorInvalidValue;
  if (!fp8) {
    if (!encode_bf16_3d(&p.ql, a.q_latent, a.pool.L, a.H, a.ql_sh, a.T, a.ql_st, kHeads, 1))
      return cudaErrorInvalidValue;
    if (a.pool.R > 0 &&
        !encode_bf16_3d(&p.qr, a.q_rope, a.pool.R, a.H, a.qr_sh, a.T, a.qr_st, kHeads, 1))
      return cudaErrorInvalidValue;
  }
  const unsigned grid = (unsigned)p.slices * (unsigned)p.groups;
  cudaError_t e = fp8 ? launch<true>(p, stream, grid) : launch<false>(p, stream, grid);
  if (e != cudaSuccess) return e;
  return launch_with_pdl(latent_merge_kernel, dim3(4 * (unsigned)sms), dim3(32 * kMergeWarps), 0,
                         stream, true, (const int2*)p.cut, (const float*)p.lse,
                         (const float*)p.part, reinterpret_cast<__nv_bfloat16*>(a.out), p.slices,
                         p.groups, a.H, a.pool.L);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t read_and_clear_latent_decode_error_word(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_spa_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_spa_error, &zero, sizeof(int));
}

}  // namespace spa
