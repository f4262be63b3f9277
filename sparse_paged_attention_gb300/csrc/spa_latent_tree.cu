// spa_latent_tree.cu - latent attention of drafted tokens: the tokens of a sequence's tree lie behind its
// context in the latent cache, and each attends to the whole context and to those of the tree that its
// mask names (its ancestors and itself).
//
//   s_j = scale (q_c . c_j + q_r . r_j),   out = sum_j softmax(s)_j c_j
//
// One block a token and head, 64 entries at a time: scores by warps, then every thread its channels.
#include "spa_errors.h"
#include "spa_latent.h"
#include "spa_launch.h"

namespace spa {

namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;

template <bool kFp8>
__device__ __forceinline__ float row_value(const LatentPoolDev& p, const uint8_t* row, float scale, int d) {
  if (!kFp8) return bf16_lo(reinterpret_cast<const uint16_t*>(row)[d]);
  const auto value = [](uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return (float)v;
  };
  return (value(row[d]) + (d < p.L ? 0.f : value(row[d + p.R]))) * scale;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads) latent_tree_kernel(const LatentTreeArgs a) {
  __shared__ float q[kLatMaxDim + kLatMaxRope], s[kTile];
  __shared__ int rows[kTile], seq;
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H, L = a.pool.L, R = a.pool.R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    seq = -1;
    int top = 0;
    for (int b = 0; b < a.pool.B; ++b) {
      const int lo = a.cu_tokens[b], hi = a.cu_tokens[b + 1];
      const bool bad = lo < top || hi < lo || hi > a.T || a.context_lens[b] < 0 ||
                       (long long)a.context_lens[b] + (hi - lo) > (long long)a.pool.bt_stride * a.pool.ps;
      top = max(top, lo);
      if (bad && blockIdx.x == 0) flag_error(SPA_ERR_INDEX);
      if (!bad && t >= lo && t < hi) seq = b;
    }
  }
  for (int d = threadIdx.x; d < L + R; d += kThreads)
    q[d] = bf16_lo(d < L ? reinterpret_cast<const uint16_t*>(a.q_latent + t * a.ql_st + h * a.ql_sh)[d]
                         : reinterpret_cast<const uint16_t*>(a.q_rope + t * a.qr_st + h * a.qr_sh)[d - L]);
  __syncthreads();
  const int b = seq;
  if (b < 0) return;
  const int ctx = a.context_lens[b], first = a.cu_tokens[b], len = ctx + a.cu_tokens[b + 1] - first;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int j0 = 0; j0 < len; j0 += kTile) {
    if (threadIdx.x < kTile) {
      const int j = j0 + threadIdx.x, i = j - ctx;
      bool seen = j < len;
      if (seen && i >= 0)
        seen = a.mask ? i < 32 * a.mask_words && (a.mask[(size_t)t * a.mask_words + (i >> 5)] >> (i & 31) & 1u)
                      : i <= t - first;
      int row = -1;
      if (j < len && (row = latent_row(a.pool, b, j)) < 0) flag_error(SPA_ERR_INDEX);
      rows[threadIdx.x] = seen ? row : -1;
    }
    __syncthreads();
    for (int i = warp; i < kTile; i += kThreads / 32) {
      const int row = rows[i];
      float x = 0.f;
      if (row >= 0) {
        const uint8_t* src = a.pool.rows + (size_t)row * a.pool.row_bytes;
        const float sc = kFp8 ? a.pool.scale[row] : 1.f;
        for (int d = lane; d < L + R; d += 32) x = fmaf(q[d], row_value<kFp8>(a.pool, src, sc, d), x);
      }
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) x += __shfl_xor_sync(0xffffffffu, x, e);
      if (lane == 0) s[i] = row >= 0 ? x * a.scale : -INFINITY;
    }
    __syncthreads();
    float mt = m;
    for (int i = 0; i < kTile; ++i) mt = fmaxf(mt, s[i]);
    const float ref = mt == -INFINITY ? 0.f : mt, f = __expf(m - ref);
    l *= f;
    o[0] *= f;
    o[1] *= f;
    m = mt;
    for (int i = 0; i < kTile; ++i) {
      const int row = rows[i];
      if (row < 0) continue;
      const float p = __expf(s[i] - ref);
      l += p;
      const uint8_t* src = a.pool.rows + (size_t)row * a.pool.row_bytes;
      const float sc = kFp8 ? a.pool.scale[row] : 1.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = threadIdx.x + e * kThreads;
        if (d < L) o[e] = fmaf(p, row_value<kFp8>(a.pool, src, sc, d), o[e]);
      }
    }
    __syncthreads();
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int e = 0; e < 2; ++e) {
    const int d = threadIdx.x + e * kThreads;
    if (d < L) reinterpret_cast<__nv_bfloat16*>(a.out)[((size_t)t * a.H + h) * L + d] = __float2bfloat16(o[e] * inv);
  }
}

}  // namespace

cudaError_t prepare_latent_tree() { return cudaSuccess; }

size_t latent_tree_workspace(const LatentTreeArgs&, bool, int) { return 0; }

cudaError_t launch_latent_tree(const LatentTreeArgs& a, bool fp8, void*, int, cudaStream_t stream) {
  return launch_with_pdl(fp8 ? latent_tree_kernel<true> : latent_tree_kernel<false>, dim3((unsigned)a.T * a.H),
                         dim3(kThreads), 0, stream, false, a);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t latent_tree_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
