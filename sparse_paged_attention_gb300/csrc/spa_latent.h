// spa_latent.h - parameters and launchers of the latent-attention kernels, shared by the kernel
// files and their C ABI file.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "spa_device.cuh"

namespace spa {

constexpr int kLatMaxDim = 512;    // latent_dim at most (a multiple of 64)
constexpr int kLatMaxRope = 64;    // rope_dim at most (a multiple of 8)

// A latent pool as the kernels see it.
struct LatentPoolDev {
  uint8_t* rows;          // [num_blocks * ps] rows of row_bytes
  float* scale;           // e4m3 pools
  const int32_t* bt;      // [B][bt_stride]
  long long num_blocks;
  int ps, bt_stride, B;
  int ps_shift;           // log2 of ps, or -1
  int L, R;               // latent and rotary widths
  int row_bytes;          // 2 (L + R), or L + 2 R
};

// Row of the entry at position x >= 0 of sequence b (checked by the caller), or -1.
__device__ __forceinline__ int latent_row(const LatentPoolDev& p, int b, int x) {
  const int page = p.ps_shift >= 0 ? x >> p.ps_shift : x / p.ps;
  if (page >= p.bt_stride) return -1;
  const int blk = __ldg(p.bt + (size_t)b * p.bt_stride + page);
  if (blk < 0 || (long long)blk >= p.num_blocks) return -1;
  return (int)((long long)blk * p.ps + (x - page * p.ps));   // (num_blocks * ps <= 2^30)
}

struct LatentCacheArgs {        // write and read
  LatentPoolDev pool;
  const uint8_t* latent;        // write: bf16 rows, strides in bytes
  const uint8_t* rope;
  long long latent_stride, rope_stride;
  uint8_t* out;                 // read: bf16 rows, stride in bytes
  long long out_stride;
  const int32_t* positions;
  const int32_t* seq_of_token;
  int T;
};
cudaError_t launch_latent_write(const LatentCacheArgs& a, bool fp8, int sms, cudaStream_t stream);
cudaError_t launch_latent_read(const LatentCacheArgs& a, bool fp8, int sms, cudaStream_t stream);

struct LatentDecodeArgs {
  LatentPoolDev pool;
  const uint8_t* q_latent;      // bf16, strides in bytes
  const uint8_t* q_rope;
  long long ql_st, ql_sh, qr_st, qr_sh;
  uint8_t* out;                 // bf16 [T][H][L]
  const int32_t* positions;
  const int32_t* seq_of_token;
  float scale;
  int T, H;
};
cudaError_t prepare_latent_decode();   // per-device one-time attributes (dynamic shared memory)
size_t latent_decode_workspace(const LatentDecodeArgs& a, bool fp8, int sms);
cudaError_t launch_latent_decode(const LatentDecodeArgs& a, bool fp8, void* workspace, int sms,
                                 cudaStream_t stream);

struct LatentPrefillArgs {
  const uint8_t *q, *k_nope, *k_rope, *v;   // bf16, strides in bytes
  long long q_st, q_sh, kn_st, kn_sh, kr_st, v_st, v_sh;
  uint8_t* out;                 // bf16 [num_q][H][dv]
  const int32_t *cu_q, *cu_k;
  float scale;
  int num_q, num_k, B, H, dn, dr, dv;
};
cudaError_t prepare_latent_prefill();
cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, int sms, cudaStream_t stream);

}  // namespace spa
