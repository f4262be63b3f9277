// spa_rotary.h - parameters and launchers of the rotation, norm and append kernels, shared by the kernel
// file and its C ABI file.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "spa_latent.h"

namespace spa {

constexpr int kRopeMaxDim = 1024;     // head_dim at most (a multiple of 8)
constexpr int kRopeMaxPart = 256;     // rope_dim at most (a multiple of 8)

struct RotaryDev {
  const long long* turns;   // [R / 2], turns a position as 64-bit binary fractions
  float scale;              // rotated values times this
  int R, start;             // values rotated, the first of them
  int half;                 // pairs (i, i + R / 2) instead of (2i, 2i + 1)
  int inverse;
};

// The checks that the entry points share: SPA_OK or what is wrong.
int check_rotary(int32_t rope_dim, int32_t rope_start, int32_t width, float rope_scale, const int64_t* turns);
int check_norm(const void* weight, int32_t weight_dtype, float eps);
// The append's arguments but for the pool; widths as checked.
int check_append(const spa_append_t* pr, int k_width, int v_width);
void fill_append(struct AppendArgs& a, const spa_append_t* pr);

struct HeadRows {           // rows of one tensor, strides in bytes
  const uint8_t* x;
  uint8_t* out;
  const void* weight;       // NULL: ones
  long long x_st, x_sh, out_st, out_sh;
  int H;
};

struct RopeArgs {
  HeadRows q, k;            // k.H 0: none
  RotaryDev rot;
  const int32_t* positions;
  float eps;
  int T, D;
  int weight_bf16;
};
// The rotation alone, or after the norm of every head.
cudaError_t launch_rope(const RopeArgs& a, bool norm, int sms, cudaStream_t stream);

struct AppendArgs {         // K and V rows into a paged pool, or [c | r] rows into a latent pool
  RotaryDev rot;
  const uint8_t *k, *v;     // bf16 rows, strides in bytes (latent: c and r)
  long long k_st, v_st;
  const void* weight;       // NULL: ones
  const int32_t *positions, *entries, *seq_of_token;
  LatentPoolDev pool;       // rows: a latent pool, or (paged) [rows][2][D] with L = D
  float *k_scale, *v_scale;
  float eps;
  int T, norm, weight_bf16;
};
cudaError_t launch_kv_append(const AppendArgs& a, bool fp8, int sms, cudaStream_t stream);
cudaError_t launch_latent_append(const AppendArgs& a, bool fp8, int sms, cudaStream_t stream);

}  // namespace spa
