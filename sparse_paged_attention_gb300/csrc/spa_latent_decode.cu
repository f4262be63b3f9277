// spa_latent_decode.cu - absorbed latent attention over the paged cache, first form: one CTA a
// (token, head), fp32 arithmetic, an online softmax over tiles of 128 entries.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_latent.h"

namespace spa {

namespace {

constexpr int kTile = 128;

template <bool kFp8>
__device__ __forceinline__ float row_value(const LatentPoolDev& p, const uint8_t* row, float scale,
                                           int i) {
  if (!kFp8) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  __nv_fp8_e4m3 v;
  v.__x = row[i];
  float x = (float)v;
  if (i >= p.L) {
    v.__x = row[i + p.R];
    x += (float)v;
  }
  return x * scale;
}

template <bool kFp8>
__global__ void __launch_bounds__(kTile) latent_decode_simple(const LatentDecodeArgs a) {
  __shared__ float q[kLatMaxDim + kLatMaxRope], pr[kTile], red[4];
  __shared__ int rows[kTile];
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const int L = a.pool.L, W = a.pool.L + a.pool.R;
  for (int i = tid; i < W; i += kTile) {
    const uint8_t* src = i < L ? a.q_latent + t * a.ql_st + h * a.ql_sh + 2 * i
                               : a.q_rope + t * a.qr_st + h * a.qr_sh + 2 * (i - L);
    q[i] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(src) << 16);
  }
  const int b = a.seq_of_token ? a.seq_of_token[t] : 0;
  int n = a.positions[t];
  n = n < 0 ? 0 : n + 1;
  if (n < 0) n = 0x7fffffff;
  if (b < 0 || b >= a.pool.B) {
    n = 0;
    if (tid == 0) flag_error(SPA_ERR_INDEX);
  }
  const long long cap = (long long)a.pool.bt_stride * a.pool.ps;
  if (n > cap) {
    n = (int)cap;
    if (tid == 0) flag_error(SPA_ERR_INDEX);
  }
  float m = -INFINITY, l = 0.f, o[kLatMaxDim / kTile] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < n; j0 += kTile) {
    __syncthreads();
    const int j = j0 + tid;
    const int row = j < n ? latent_row(a.pool, b, j) : -1;
    if (j < n && row < 0) flag_error(SPA_ERR_INDEX);
    rows[tid] = row;
    float s = -INFINITY;
    if (row >= 0) {
      const uint8_t* x = a.pool.rows + (size_t)row * a.pool.row_bytes;
      const float sc = kFp8 ? a.pool.scale[row] : 1.f;
      s = 0.f;
      for (int i = 0; i < W; ++i) s += q[i] * row_value<kFp8>(a.pool, x, sc, i);
      s *= a.scale;
    }
    float mx = s;
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - ref);
    pr[tid] = row >= 0 ? expf(s - ref) : 0.f;
    __syncthreads();
    l *= c;
    for (int k = 0; k < kTile; ++k) l += pr[k];
    for (int d = 0; d < kLatMaxDim / kTile; ++d) o[d] *= c;
    for (int k = 0; k < kTile; ++k) {
      if (rows[k] < 0) continue;
      const uint8_t* x = a.pool.rows + (size_t)rows[k] * a.pool.row_bytes;
      const float sc = kFp8 ? a.pool.scale[rows[k]] : 1.f;
      for (int d = 0; d < kLatMaxDim / kTile; ++d)
        if (d * kTile + tid < L) o[d] += pr[k] * row_value<kFp8>(a.pool, x, sc, d * kTile + tid);
    }
    m = mn;
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + ((size_t)t * a.H + h) * L;
  for (int d = 0; d < kLatMaxDim / kTile; ++d)
    if (d * kTile + tid < L) out[d * kTile + tid] = __float2bfloat16_rn(m == -INFINITY ? 0.f : o[d] / l);
}

}  // namespace

size_t latent_decode_workspace(const LatentDecodeArgs&, int) { return 0; }

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void*, int, cudaStream_t stream) {
  const long long blocks = (long long)a.T * a.H;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (fp8) latent_decode_simple<true><<<(unsigned)blocks, kTile, 0, stream>>>(a);
  else latent_decode_simple<false><<<(unsigned)blocks, kTile, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t read_and_clear_latent_decode_error_word(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_spa_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_spa_error, &zero, sizeof(int));
}

}  // namespace spa
