// spa_latent_cache.cu - the latent cache's write and read: rows [c | r] of new tokens go to their
// pool slots, copied (bf16 pools) or quantised to e4m3 with one scale a row, and come back as bf16.
//
//   scale = max|x| / 448,  code(c) = e4m3(c / scale),
//   high(r) = e4m3(r / scale),  low(r) = e4m3(r / scale - high(r))      (the difference is exact)
//
// The rotary part keeps two codes a value (about 8 bits) because it carries the position: its
// rounding moves the scores of near and far entries against one another, and it is a ninth of the
// row.  A row's bytes go in and a row's bytes out, with no reuse.  One warp takes one token, all of whose
// row is loaded before any of it is used; the row maximum is a warp reduction; the slot's dependent
// loads (position, block table) run beside the row's.  No shared memory and few registers, so that
// enough warps stay resident to cover HBM's latency without a staged pipeline (one, with the next row's
// loads under this row's codes, measured slower: 42 us against 31 for 65,536 e4m3 rows).
//
// Measured, L = 512, R = 64: 65,536 rows written as e4m3 in 24.8 us (4.8 TB/s, 70% of the measured copy
// rate; its arithmetic takes two thirds of the issue slots: with one value an instruction it took
// 31, with IEEE divisions for the rotary part and 12 CTAs an SM 27.4), read back in 22.8 us (5.2 TB/s,
// 76%); 65,536 bf16 rows written in 26.8 us and read in 27.0 (5.6 TB/s, 83%), 30,001 of them in pages of 24
// written in 14.4, launch included (two to four rows in flight a warp: the same or slower).  Eight tokens
// take 2 us, and the call's host side 13.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_kvwrite_quant.cuh"
#include "spa_errors.h"
#include "spa_latent.h"

namespace spa {

namespace {

constexpr int kWarps = 4;            // tokens in flight a CTA
constexpr int kBlocks = 16;          // CTAs an SM, all resident: 64 warps of 32 registers (e4m3 write of 65,536
                                     // rows: 26.3 us where 41 registers, and 12 CTAs resident, took 28.1; the
                                     // rotary part's divisions as above brought 24.8)
constexpr int kChunks = kLatMaxDim / 8 / 32;   // 16-byte chunks of the latent part a lane
static_assert(kChunks == 2, "the write's slow path picks one of two");

// Pool row of token t, or -1 (a position, page, block or sequence that does not exist).
__device__ __forceinline__ int token_row(const LatentCacheArgs& a, int t) {
  const int x = __ldg(a.positions + t);
  const int b = a.seq_of_token ? __ldg(a.seq_of_token + t) : 0;
  if (x < 0 || b < 0 || b >= a.pool.B) return -1;
  return latent_row(a.pool, b, x);
}

// Maximum of two pairs of bf16 magnitudes (a NaN does not enter it).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t m, uint32_t w) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
  return r;
}

// (x0, x1) / scale by kvq_div's operations, two values an instruction: r = RN(1 / scale), one correction
// with the exact residual; the sign of a zero is lost.  For a scale that is RN(m / 448) of a bf16 m (what
// a row has) and bf16 x the quotients are the correctly rounded ones: true of all 128 x 128 mantissas
// wherever the residual is exact (|x| >= 2^-100); below that they are too small to have codes.
__device__ __forceinline__ void div_bf16x2(float& x0, float& x1, float scale, float r) {
  asm("{ .reg .b64 x, r, s, q, e; mov.b64 x, {%0, %1}; mov.b64 r, {%2, %2}; mov.b64 s, {%3, %3}; "
      "mul.rn.f32x2 q, x, r; fma.rn.f32x2 e, q, s, x; fma.rn.f32x2 q, e, r, q; mov.b64 {%0, %1}, q; }"
      : "+f"(x0), "+f"(x1)
      : "f"(r), "f"(-scale));
}

// kvq_chunk's reciprocal path; x's sign is put into the codes, four at a time, instead of into the
// quotients.
__device__ __forceinline__ uint2 latent_codes(const uint4& u, float scale, float r) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q0 = __uint_as_float(w[i] << 16), q1 = __uint_as_float(w[i] & 0xffff0000u);
    div_bf16x2(q0, q1, scale, r);
    c[i] = kvq_e4m3x2(q0, q1);
  }
  const auto with_signs = [](uint32_t codes, uint32_t upper) {
    return (codes & 0x7f7f7f7fu) | (upper & 0x80808080u);
  };
  return make_uint2(with_signs(c[0] | (c[1] << 16), __byte_perm(w[0], w[1], 0x7531)),
                    with_signs(c[2] | (c[3] << 16), __byte_perm(w[2], w[3], 0x7531)));
}

// value pairs of two e4m3 codes
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A lane takes chunks lane and 32 + lane of the latent part and word lane of the rotary part (two values:
// at most 64 of them).  Spread like that the rotary part's quotients and second codes cost every lane two
// of each; as 16-byte chunks they kept eight lanes busy with eight of each while the others
// waited, and the e4m3 write of 65,536 tokens took half as long again.
struct NewRow {
  uint4 u[kChunks];
  uint32_t r;
};

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) latent_write_kernel(const LatentCacheArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nl = a.pool.L >> 3, nr = a.pool.R >> 1;   // 16-byte chunks, 4-byte words
  const long long step = (long long)gridDim.x * kWarps;
  for (long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += step) {
    NewRow x;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = lane + 32 * i;
      x.u[i] = c < nl ? __ldg(reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride) + c)
                      : make_uint4(0, 0, 0, 0);
    }
    x.r = lane < nr ? __ldg(reinterpret_cast<const uint32_t*>(a.rope + t * a.rope_stride) + lane) : 0u;
    const int row = token_row(a, (int)t);
    if (row < 0) {
      if (lane == 0) flag_error(SPA_ERR_INDEX);
      continue;
    }
    uint8_t* dst = a.pool.rows + (size_t)row * a.pool.row_bytes;
    if constexpr (!kFp8) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        if (c < nl) reinterpret_cast<uint4*>(dst)[c] = x.u[i];
      }
      if (lane < nr) reinterpret_cast<uint32_t*>(dst + 2 * a.pool.L)[lane] = x.r;
    } else {
      const float ra = kvq_bf16_to_f32(x.r & 0xFFFFu), rb = kvq_bf16_to_f32(x.r >> 16);
      uint32_t mb = absmax_bf16x2(0u, x.r);
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        for (const uint32_t w : {x.u[i].x, x.u[i].y, x.u[i].z, x.u[i].w}) mb = absmax_bf16x2(mb, w);
      // (bf16's bits order as their magnitudes do)
      mb = __reduce_max_sync(0xffffffffu, max(mb & 0xffffu, mb >> 16));
      const float amax = __uint_as_float(mb << 16);
      const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      const float r = __frcp_rn(scale);
      const bool fast = kvq_fast_scale(scale);
      float p = ra, q = rb;
      if (fast) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = lane + 32 * i;
          if (c < nl) *reinterpret_cast<uint2*>(dst + 8 * c) = latent_codes(x.u[i], scale, r);
        }
        div_bf16x2(p, q, scale, r);
        p = copysignf(p, ra);
        q = copysignf(q, rb);
      } else {
#pragma unroll 1
        for (int i = 0; i < kChunks; ++i) {
          const int c = lane + 32 * i;
          if (c < nl) *reinterpret_cast<uint2*>(dst + 8 * c) = kvq_chunk(i == 0 ? x.u[0] : x.u[1], scale, r, false);
        }
        p = __fdiv_rn(ra, scale);
        q = __fdiv_rn(rb, scale);
      }
      if (lane < nr) {
        // (the low code sees the quotient's last bits)
        const uint32_t high = kvq_e4m3x2(p, q);
        const float2 v = e4m3x2_to_f32(high);
        uint16_t* rope = reinterpret_cast<uint16_t*>(dst + a.pool.L) + lane;
        rope[0] = (uint16_t)high;
        rope[nr] = (uint16_t)kvq_e4m3x2(p - v.x, q - v.y);
      }
      if (lane == 0) a.pool.scale[row] = scale;
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) latent_read_kernel(const LatentCacheArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nl = a.pool.L >> 3, nr = a.pool.R >> 1;
  const long long step = (long long)gridDim.x * kWarps;
  for (long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += step) {
    const int row = token_row(a, (int)t);
    if (row < 0 && lane == 0) flag_error(SPA_ERR_INDEX);
    const uint8_t* src = a.pool.rows + (size_t)(row < 0 ? 0 : row) * a.pool.row_bytes;
    uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.out_stride);
    uint32_t* dst_r = reinterpret_cast<uint32_t*>(a.out + t * a.out_stride + 2 * a.pool.L);
    if constexpr (!kFp8) {
      NewRow x;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        x.u[i] = row >= 0 && c < nl ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
      }
      x.r = row >= 0 && lane < nr ? __ldg(reinterpret_cast<const uint32_t*>(src + 2 * a.pool.L) + lane) : 0u;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        if (c < nl) dst[c] = x.u[i];
      }
      if (lane < nr) dst_r[lane] = x.r;
    } else {
      uint2 code[kChunks];
      uint32_t high = 0, low = 0;
      const float scale = row >= 0 ? __ldg(a.pool.scale + row) : 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        code[i] = row >= 0 && c < nl ? __ldg(reinterpret_cast<const uint2*>(src) + c) : make_uint2(0, 0);
      }
      if (row >= 0 && lane < nr) {
        const uint16_t* rope = reinterpret_cast<const uint16_t*>(src + a.pool.L) + lane;
        high = __ldg(rope);
        low = __ldg(rope + nr);
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        const uint32_t h[2] = {code[i].x, code[i].y};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = e4m3x2_to_f32((h[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
          o[k] = bf16x2(v.x * scale, v.y * scale);
        }
        if (c < nl) dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (lane < nr) {
        const float2 v = e4m3x2_to_f32(high), w = e4m3x2_to_f32(low);
        dst_r[lane] = bf16x2((v.x + w.x) * scale, (v.y + w.y) * scale);
      }
    }
  }
}

unsigned cache_blocks(int T, int sms) {
  const long long b = ((long long)T + kWarps - 1) / kWarps, cap = (long long)kBlocks * sms;
  return (unsigned)(b < cap ? b : cap);
}

}  // namespace

cudaError_t launch_latent_write(const LatentCacheArgs& a, bool fp8, int sms, cudaStream_t stream) {
  const unsigned blocks = cache_blocks(a.T, sms);
  return launch_with_pdl(fp8 ? latent_write_kernel<true> : latent_write_kernel<false>,
                         dim3(blocks), dim3(32 * kWarps), 0, stream, 2LL * blocks <= sms, a);
}

cudaError_t launch_latent_read(const LatentCacheArgs& a, bool fp8, int sms, cudaStream_t stream) {
  const unsigned blocks = cache_blocks(a.T, sms);
  return launch_with_pdl(fp8 ? latent_read_kernel<true> : latent_read_kernel<false>, dim3(blocks),
                         dim3(32 * kWarps), 0, stream, 2LL * blocks <= sms, a);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t latent_cache_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
