// spa_latent_cache.cu - the latent cache's write and read: rows [c | r] of new tokens go to their
// pool slots, copied (bf16 pools) or quantised to e4m3 with one scale a row, and come back as bf16.
//
//   scale = max|x| / 448,  code(c) = e4m3(c / scale),
//   high(r) = e4m3(r / scale),  low(r) = e4m3(r / scale - high(r))      (the difference is exact)
//
// The rotary part keeps two codes a value (about 8 bits) because it carries the position: its
// rounding moves the scores of near and far entries against one another, and it is a ninth of the
// row.  Both kernels are bound by HBM (a row's bytes in, a row's bytes out, no reuse).  One warp
// takes one token: a row is at most 72 16-byte chunks, three a lane, all loaded before any is used;
// the row maximum is a shuffle reduction; the slot's dependent loads (position, block table) run
// beside the row's.  No shared memory and few registers, so that enough warps stay resident to
// cover HBM's latency without a staged pipeline.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_kvwrite_quant.cuh"
#include "spa_latent.h"

namespace spa {

namespace {

constexpr int kWarps = 4;            // tokens in flight a CTA
constexpr int kChunks = (kLatMaxDim + kLatMaxRope) / 8 / 32 + 1;   // 16-byte chunks a lane (3)

// Pool row of token t, or -1 (a position, page, block or sequence that does not exist).
__device__ __forceinline__ int token_row(const LatentCacheArgs& a, int t) {
  const int x = __ldg(a.positions + t);
  const int b = a.seq_of_token ? __ldg(a.seq_of_token + t) : 0;
  if (x < 0 || b < 0 || b >= a.pool.B) return -1;
  return latent_row(a.pool, b, x);
}

__device__ __forceinline__ float chunk_absmax(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = fmaxf(m, fabsf(kvq_bf16_to_f32(w[i] & 0xFFFFu)));
    m = fmaxf(m, fabsf(kvq_bf16_to_f32(w[i] >> 16)));
  }
  return m;
}

// value pairs of two e4m3 codes
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight rotary values -> high and low codes.  IEEE divisions: the low code sees the quotient's
// last bits, which the reciprocal path of the latent part is not held to.
__device__ __forceinline__ void rope_codes(const uint4& u, float scale, uint2& high, uint2& low) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = __fdiv_rn(kvq_bf16_to_f32(w[i] & 0xFFFFu), scale);
    const float y = __fdiv_rn(kvq_bf16_to_f32(w[i] >> 16), scale);
    h[i] = kvq_e4m3x2(x, y);
    const float2 v = e4m3x2_to_f32(h[i]);
    l[i] = kvq_e4m3x2(x - v.x, y - v.y);
  }
  high = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  low = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps) latent_write_kernel(const LatentCacheArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int L = a.pool.L, R = a.pool.R;
  const int nl = L >> 3, n = (L + R) >> 3;   // chunks of the latent part, of the row
  const long long step = (long long)gridDim.x * kWarps;
  for (long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += step) {
    uint4 u[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = lane + 32 * i;
      u[i] = make_uint4(0, 0, 0, 0);
      if (c < nl)
        u[i] = __ldg(reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride) + c);
      else if (c < n)
        u[i] = __ldg(reinterpret_cast<const uint4*>(a.rope + t * a.rope_stride) + (c - nl));
    }
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
        if (c < n) reinterpret_cast<uint4*>(dst)[c] = u[i];
      }
    } else {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) amax = fmaxf(amax, chunk_absmax(u[i]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      const float r = __frcp_rn(scale);
      const bool fast = kvq_fast_scale(scale);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        if (c < nl) {
          *reinterpret_cast<uint2*>(dst + 8 * c) = kvq_chunk(u[i], scale, r, fast);
        } else if (c < n) {
          uint2 high, low;
          rope_codes(u[i], scale, high, low);
          *reinterpret_cast<uint2*>(dst + 8 * c) = high;
          *reinterpret_cast<uint2*>(dst + R + 8 * c) = low;
        }
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
__global__ void __launch_bounds__(32 * kWarps) latent_read_kernel(const LatentCacheArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int L = a.pool.L, R = a.pool.R;
  const int nl = L >> 3, n = (L + R) >> 3;
  const long long step = (long long)gridDim.x * kWarps;
  for (long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += step) {
    const int row = token_row(a, (int)t);
    if (row < 0 && lane == 0) flag_error(SPA_ERR_INDEX);
    const uint8_t* src = a.pool.rows + (size_t)(row < 0 ? 0 : row) * a.pool.row_bytes;
    uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.out_stride);
    if constexpr (!kFp8) {
      uint4 u[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        u[i] = make_uint4(0, 0, 0, 0);
        if (row >= 0 && c < n) u[i] = __ldg(reinterpret_cast<const uint4*>(src) + c);
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        if (c < n) dst[c] = u[i];
      }
    } else {
      uint2 hi[kChunks], lo[kChunks];
      float scale = 0.f;
      if (row >= 0) scale = __ldg(a.pool.scale + row);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        hi[i] = lo[i] = make_uint2(0, 0);
        if (row >= 0 && c < n) hi[i] = __ldg(reinterpret_cast<const uint2*>(src + 8 * c));
        if (row >= 0 && c >= nl && c < n)
          lo[i] = __ldg(reinterpret_cast<const uint2*>(src + R + 8 * c));
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = lane + 32 * i;
        if (c < n) {
          const uint32_t h[2] = {hi[i].x, hi[i].y}, l[2] = {lo[i].x, lo[i].y};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = e4m3x2_to_f32((h[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
            const float2 y = e4m3x2_to_f32((l[k >> 1] >> (16 * (k & 1))) & 0xFFFFu);
            o[k] = c < nl ? bf16x2(x.x * scale, x.y * scale)
                          : bf16x2((x.x + y.x) * scale, (x.y + y.y) * scale);
          }
          dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

unsigned cache_blocks(int T, int sms) {
  const long long b = ((long long)T + kWarps - 1) / kWarps, cap = 16LL * sms;
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
cudaError_t read_and_clear_latent_cache_error_word(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_spa_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_spa_error, &zero, sizeof(int));
}

}  // namespace spa
