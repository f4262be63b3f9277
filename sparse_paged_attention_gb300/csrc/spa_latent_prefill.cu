// spa_latent_prefill.cu - expanded latent attention over ragged causal sequences, first form: one
// CTA a (query row, head), fp32 arithmetic, an online softmax over tiles of 128 keys.
#include "spa_latent.h"

namespace spa {

namespace {

constexpr int kTile = 128;

__device__ __forceinline__ float bf(const uint8_t* p, int i) {
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// Sequence bounds of sequence b; false (and the error word) when they are not usable.
__device__ __forceinline__ bool bounds(const LatentPrefillArgs& a, int b, int& q0, int& q1, int& k0,
                                       int& k1) {
  q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  return 0 <= q0 && q0 <= q1 && q1 <= a.num_q && 0 <= k0 && k0 <= k1 && k1 <= a.num_k;
}

__global__ void __launch_bounds__(kTile) latent_prefill_simple(const LatentPrefillArgs a) {
  __shared__ float q[192], pr[kTile], red[4];
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  bool own = false;
  for (int b = 0; b < a.B && !own; ++b) {
    const bool ok = bounds(a, b, q0, q1, k0, k1);
    if (!ok && tid == 0) flag_error(SPA_ERR_INDEX);
    own = ok && q0 <= t && t < q1;
  }
  if (!own) return;
  const uint8_t* qr = a.q + t * a.q_st + h * a.q_sh;
  for (int i = tid; i < a.dn + a.dr; i += kTile) q[i] = bf(qr, i);
  const long long n = (long long)(t - q0) + 1 + (k1 - k0) - (q1 - q0);   // keys seen
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (long long j0 = 0; j0 < n; j0 += kTile) {
    __syncthreads();
    const long long j = k0 + j0 + tid;
    float s = -INFINITY;
    if (j0 + tid < n) {
      const uint8_t* kn = a.k_nope + j * a.kn_st + h * a.kn_sh;
      const uint8_t* kr = a.k_rope + j * a.kr_st;
      s = 0.f;
      for (int i = 0; i < a.dn; ++i) s += q[i] * bf(kn, i);
      for (int i = 0; i < a.dr; ++i) s += q[a.dn + i] * bf(kr, i);
      s *= a.scale;
    }
    float mx = s;
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - ref);
    pr[tid] = j0 + tid < n ? expf(s - ref) : 0.f;
    __syncthreads();
    l *= c;
    o *= c;
    for (int k = 0; k < kTile && j0 + k < n; ++k) {
      l += pr[k];
      if (tid < a.dv) o += pr[k] * bf(a.v + (k0 + j0 + k) * a.v_st + h * a.v_sh, tid);
    }
    m = mn;
  }
  if (tid < a.dv)
    reinterpret_cast<__nv_bfloat16*>(a.out)[((size_t)t * a.H + h) * a.dv + tid] =
        __float2bfloat16_rn(n <= 0 ? 0.f : o / l);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, int, cudaStream_t stream) {
  const long long blocks = (long long)a.num_q * a.H;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  latent_prefill_simple<<<(unsigned)blocks, kTile, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t read_and_clear_latent_prefill_error_word(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_spa_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_spa_error, &zero, sizeof(int));
}

}  // namespace spa
