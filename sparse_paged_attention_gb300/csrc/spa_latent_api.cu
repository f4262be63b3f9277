// spa_latent_api.cu - the latent-attention entry points of the C ABI: host-side validation and
// launches.
#include <cmath>
#include <cstring>

#include "sparse_attn_paged.h"
#include "spa_latent.h"
#include "spa_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// element strides up to 2^38: byte offsets stay in 63 bits, and a tensor map holds 2^40 bytes
bool stride_ok(int64_t s) { return s >= 0 && s <= (1ll << 38); }

// The kernels take the scale times log2(e) in fp32.
bool scale_ok(float s) { return std::isfinite(s * 1.4426950408889634f); }

// Geometry that needs no pointer: checked even when there is nothing to do.
int check_dims(const spa_latent_pool_t* pl) {
  if (pl->latent_dim < 1 || pl->rope_dim < 0) return SPA_ERR_SHAPE;
  if (pl->latent_dim % 64 != 0 || pl->latent_dim > spa::kLatMaxDim || pl->rope_dim % 8 != 0 ||
      pl->rope_dim > spa::kLatMaxRope)
    return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

int check_pool(const spa_latent_pool_t* pl, bool fp8) {
  if (!pl->rows || !pl->block_table) return SPA_ERR_NULL;
  if (pl->num_blocks < 1 || pl->page_size < 1 || pl->bt_stride < 1) return SPA_ERR_SHAPE;
  if ((long double)pl->num_blocks * pl->page_size > (long double)(1ll << 30))
    return SPA_ERR_UNSUPPORTED;
  if (!aligned16(pl->rows)) return SPA_ERR_ALIGN;
  if (fp8 && !pl->scale) return SPA_ERR_NULL;
  return SPA_OK;
}

void fill_pool(spa::LatentPoolDev& d, const spa_latent_pool_t* pl, int num_seqs, bool fp8) {
  d.rows = static_cast<uint8_t*>(const_cast<void*>(pl->rows));   // written by the write alone
  d.scale = const_cast<float*>(pl->scale);
  d.bt = pl->block_table;
  d.num_blocks = pl->num_blocks;
  d.ps = pl->page_size;
  d.ps_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (d.ps == 1 << i) d.ps_shift = i;
  d.bt_stride = pl->bt_stride;
  d.B = num_seqs;
  d.L = pl->latent_dim;
  d.R = pl->rope_dim;
  d.row_bytes = fp8 ? pl->latent_dim + 2 * pl->rope_dim : 2 * (pl->latent_dim + pl->rope_dim);
}

int latent_write(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                 int32_t T, const int32_t* positions, const int32_t* seq_of_token, int32_t B,
                 const spa_latent_pool_t* pool, void* stream, bool fp8) {
  if (!pool) return SPA_ERR_NULL;
  if (T < 0 || B < 1 || !stride_ok(latent_stride) || !stride_ok(rope_stride)) return SPA_ERR_SHAPE;
  int st = check_dims(pool);
  if (st) return st;
  if (T == 0) return SPA_OK;
  const bool has_rope = pool->rope_dim > 0;
  if (!latent || (has_rope && !rope) || !positions) return SPA_ERR_NULL;
  st = check_pool(pool, fp8);
  if (st) return st;
  if (!aligned16(latent) || latent_stride % 8 != 0) return SPA_ERR_ALIGN;
  if (has_rope && (!aligned16(rope) || rope_stride % 8 != 0)) return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::LatentCacheArgs a;
  std::memset(&a, 0, sizeof a);
  fill_pool(a.pool, pool, B, fp8);
  a.latent = static_cast<const uint8_t*>(latent);
  a.rope = static_cast<const uint8_t*>(rope);
  a.latent_stride = 2 * latent_stride;
  a.rope_stride = 2 * rope_stride;
  a.positions = positions;
  a.seq_of_token = seq_of_token;
  a.T = T;
  const cudaError_t e = spa::launch_latent_write(a, fp8, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "latent write kernel launch");
}

int latent_read(const spa_latent_pool_t* pool, int32_t n, const int32_t* positions,
                const int32_t* seq_of_token, int32_t B, void* out, int64_t out_stride, void* stream,
                bool fp8) {
  if (!pool) return SPA_ERR_NULL;
  if (n < 0 || B < 1 || !stride_ok(out_stride)) return SPA_ERR_SHAPE;
  int st = check_dims(pool);
  if (st) return st;
  if (n == 0) return SPA_OK;
  if (n > 1 && out_stride < pool->latent_dim + pool->rope_dim) return SPA_ERR_SHAPE;
  if (!positions || !out) return SPA_ERR_NULL;
  st = check_pool(pool, fp8);
  if (st) return st;
  if (!aligned16(out) || out_stride % 8 != 0) return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::LatentCacheArgs a;
  std::memset(&a, 0, sizeof a);
  fill_pool(a.pool, pool, B, fp8);
  a.out = static_cast<uint8_t*>(out);
  a.out_stride = 2 * out_stride;
  a.positions = positions;
  a.seq_of_token = seq_of_token;
  a.T = n;
  const cudaError_t e = spa::launch_latent_read(a, fp8, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "latent read kernel launch");
}

// The sizes of a decode call; *work says whether there is anything to compute.
int check_decode(const spa_latent_pool_t* pool, const spa_latent_problem_t* pr, bool* work) {
  if (!pool || !pr) return SPA_ERR_NULL;
  if (pr->num_tokens < 0 || pr->num_seqs < 1 || pr->num_heads < 1 || !scale_ok(pr->scale) ||
      !stride_ok(pr->q_latent_stride_t) || !stride_ok(pr->q_latent_stride_h) ||
      !stride_ok(pr->q_rope_stride_t) || !stride_ok(pr->q_rope_stride_h))
    return SPA_ERR_SHAPE;
  const int st = check_dims(pool);
  if (st) return st;
  if ((long long)pr->num_tokens * pr->num_heads > 0x7fffffffLL) return SPA_ERR_UNSUPPORTED;
  *work = pr->num_tokens > 0;
  return SPA_OK;
}

void fill_decode(spa::LatentDecodeArgs& a, const spa_latent_pool_t* pool,
                 const spa_latent_problem_t* pr, void* out, bool fp8) {
  std::memset(&a, 0, sizeof a);
  fill_pool(a.pool, pool, pr->num_seqs, fp8);
  a.q_latent = static_cast<const uint8_t*>(pr->q_latent);
  a.q_rope = static_cast<const uint8_t*>(pr->q_rope);
  a.ql_st = 2 * pr->q_latent_stride_t;
  a.ql_sh = 2 * pr->q_latent_stride_h;
  a.qr_st = 2 * pr->q_rope_stride_t;
  a.qr_sh = 2 * pr->q_rope_stride_h;
  a.out = static_cast<uint8_t*>(out);
  a.positions = pr->positions;
  a.seq_of_token = pr->seq_of_token;
  a.scale = pr->scale;
  a.T = pr->num_tokens;
  a.H = pr->num_heads;
}

int latent_decode(const spa_latent_pool_t* pool, const spa_latent_problem_t* pr, void* out,
                  void* workspace, size_t workspace_bytes, void* stream, bool fp8) {
  bool work = false;
  int st = check_decode(pool, pr, &work);
  if (st || !work) return st;
  const bool has_rope = pool->rope_dim > 0;
  // rows that overlap or repeat are refused: a tensor map walks distinct rows
  const auto rows_ok = [&](int64_t st, int64_t sh, int width) {
    return (pr->num_tokens <= 1 || st >= width) && (pr->num_heads <= 1 || sh >= width);
  };
  if (!rows_ok(pr->q_latent_stride_t, pr->q_latent_stride_h, pool->latent_dim) ||
      (has_rope && !rows_ok(pr->q_rope_stride_t, pr->q_rope_stride_h, pool->rope_dim)))
    return SPA_ERR_SHAPE;
  if (!pr->positions || !pr->q_latent || (has_rope && !pr->q_rope) || !out) return SPA_ERR_NULL;
  st = check_pool(pool, fp8);
  if (st) return st;
  if (!aligned16(out) || !aligned16(pr->q_latent) || pr->q_latent_stride_t % 8 != 0 ||
      pr->q_latent_stride_h % 8 != 0)
    return SPA_ERR_ALIGN;
  if (has_rope && (!aligned16(pr->q_rope) || pr->q_rope_stride_t % 8 != 0 ||
                   pr->q_rope_stride_h % 8 != 0))
    return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::LatentDecodeArgs a;
  fill_decode(a, pool, pr, out, fp8);
  const size_t need = spa::latent_decode_workspace(a, fp8, sms);
  if (need > 0) {
    if (!workspace) return SPA_ERR_NULL;
    if (!aligned16(workspace)) return SPA_ERR_ALIGN;
    if (workspace_bytes < need) return SPA_ERR_WORKSPACE;
  }
  const cudaError_t e = spa::launch_latent_decode(a, fp8, workspace, sms,
                                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "latent decode kernel launch");
}

}  // namespace

extern "C" {

int sparse_attn_latent_write(const void* latent, int64_t latent_stride, const void* rope,
                             int64_t rope_stride, int32_t num_tokens, const int32_t* positions,
                             const int32_t* seq_of_token, int32_t num_seqs,
                             const spa_latent_pool_t* pool, void* stream) {
  return latent_write(latent, latent_stride, rope, rope_stride, num_tokens, positions, seq_of_token,
                      num_seqs, pool, stream, false);
}

int sparse_attn_latent_write_fp8(const void* latent, int64_t latent_stride, const void* rope,
                                 int64_t rope_stride, int32_t num_tokens, const int32_t* positions,
                                 const int32_t* seq_of_token, int32_t num_seqs,
                                 const spa_latent_pool_t* pool, void* stream) {
  return latent_write(latent, latent_stride, rope, rope_stride, num_tokens, positions, seq_of_token,
                      num_seqs, pool, stream, true);
}

int sparse_attn_latent_read(const spa_latent_pool_t* pool, int32_t num_rows,
                            const int32_t* positions, const int32_t* seq_of_token, int32_t num_seqs,
                            void* out, int64_t out_stride, void* stream) {
  return latent_read(pool, num_rows, positions, seq_of_token, num_seqs, out, out_stride, stream,
                     false);
}

int sparse_attn_latent_read_fp8(const spa_latent_pool_t* pool, int32_t num_rows,
                                const int32_t* positions, const int32_t* seq_of_token,
                                int32_t num_seqs, void* out, int64_t out_stride, void* stream) {
  return latent_read(pool, num_rows, positions, seq_of_token, num_seqs, out, out_stride, stream,
                     true);
}

size_t sparse_attn_latent_decode_workspace_size(const spa_latent_problem_t* prob,
                                                const spa_latent_pool_t* pool) {
  bool work = false;
  if (check_decode(pool, prob, &work) || !work || pool->num_blocks < 1 || pool->page_size < 1 ||
      pool->bt_stride < 1)
    return 0;
  int dev = 0, sms = 0;
  if (spa::api_current_device(&dev, &sms) != SPA_OK) return 0;
  spa::LatentDecodeArgs a;
  fill_decode(a, pool, prob, nullptr, false);
  return spa::latent_decode_workspace(a, pool->scale != nullptr, sms);
}

int sparse_attn_latent_decode(const spa_latent_pool_t* pool, const spa_latent_problem_t* prob,
                              void* out, void* workspace, size_t workspace_bytes, void* stream) {
  return latent_decode(pool, prob, out, workspace, workspace_bytes, stream, false);
}

int sparse_attn_latent_decode_fp8(const spa_latent_pool_t* pool, const spa_latent_problem_t* prob,
                                  void* out, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  return latent_decode(pool, prob, out, workspace, workspace_bytes, stream, true);
}

int sparse_attn_latent_prefill(const spa_latent_prefill_t* pr, void* out, void* stream) {
  if (!pr) return SPA_ERR_NULL;
  if (pr->num_q < 0 || pr->num_k < 0 || pr->num_seqs < 0 || pr->num_heads < 1 || pr->nope_dim < 1 ||
      pr->rope_dim < 0 || pr->v_dim < 1 || !scale_ok(pr->scale))
    return SPA_ERR_SHAPE;
  if (pr->nope_dim % 8 != 0 || pr->nope_dim > 128 || pr->v_dim % 8 != 0 || pr->v_dim > 128 ||
      pr->rope_dim % 8 != 0 || pr->rope_dim > 64)
    return SPA_ERR_UNSUPPORTED;
  if ((long long)pr->num_q * pr->num_heads > 0x7fffffffLL) return SPA_ERR_UNSUPPORTED;
  if (pr->num_q == 0 || pr->num_seqs == 0) return SPA_OK;
  const int64_t H = pr->num_heads;
  struct {
    const void* p;
    int64_t st, sh;
    int width, rows;
    bool heads;
  } in[4] = {{pr->q, pr->q_stride_t, pr->q_stride_h, pr->nope_dim + pr->rope_dim, pr->num_q, true},
             {pr->k_nope, pr->k_nope_stride_t, pr->k_nope_stride_h, pr->nope_dim, pr->num_k, true},
             {pr->v, pr->v_stride_t, pr->v_stride_h, pr->v_dim, pr->num_k, true},
             {pr->k_rope, pr->k_rope_stride_t, 0, pr->rope_dim, pr->num_k, false}};
  if (!pr->cu_q || !pr->cu_k || !out) return SPA_ERR_NULL;
  for (const auto& x : in) {
    if (x.width == 0 || x.rows == 0) continue;
    if (!x.p) return SPA_ERR_NULL;
    if (!stride_ok(x.st) || !stride_ok(x.sh)) return SPA_ERR_SHAPE;
    if ((x.rows > 1 && x.st < x.width) || (x.heads && H > 1 && x.sh < x.width))
      return SPA_ERR_SHAPE;
    if (!aligned16(x.p) || x.st % 8 != 0 || x.sh % 8 != 0) return SPA_ERR_ALIGN;
  }
  if (!aligned16(out)) return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  const int st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::LatentPrefillArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = static_cast<const uint8_t*>(pr->q);
  a.k_nope = static_cast<const uint8_t*>(pr->k_nope);
  a.k_rope = static_cast<const uint8_t*>(pr->k_rope);
  a.v = static_cast<const uint8_t*>(pr->v);
  a.q_st = 2 * pr->q_stride_t;
  a.q_sh = 2 * pr->q_stride_h;
  a.kn_st = 2 * pr->k_nope_stride_t;
  a.kn_sh = 2 * pr->k_nope_stride_h;
  a.kr_st = 2 * pr->k_rope_stride_t;
  a.v_st = 2 * pr->v_stride_t;
  a.v_sh = 2 * pr->v_stride_h;
  a.out = static_cast<uint8_t*>(out);
  a.cu_q = pr->cu_q;
  a.cu_k = pr->cu_k;
  a.scale = pr->scale;
  a.num_q = pr->num_q;
  a.num_k = pr->num_k;
  a.B = pr->num_seqs;
  a.H = pr->num_heads;
  a.dn = pr->nope_dim;
  a.dr = pr->rope_dim;
  a.dv = pr->v_dim;
  const cudaError_t e = spa::launch_latent_prefill(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "latent prefill kernel launch");
}

}  // extern "C"
