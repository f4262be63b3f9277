// spa_rotary_api.cu - the entry points of the rotation, the norms and the paged append: host-side
// validation and launches.
#include <cmath>
#include <cstring>

#include "sparse_attn_paged.h"
#include "spa_launch.h"
#include "spa_rotary.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stride_ok(int64_t s) { return s >= 0 && s <= (1ll << 38); }

spa::RotaryDev rotary(int R, int start, int interleaved, int inverse, float scale, const int64_t* turns) {
  spa::RotaryDev r;
  r.turns = reinterpret_cast<const long long*>(turns);
  r.scale = scale;
  r.R = R;
  r.start = start;
  r.half = !interleaved;
  r.inverse = inverse != 0;
  return r;
}

// Rows of one tensor of a rope call (norm or not).
int check_rows(const spa_head_rows_t& x, const spa_rope_problem_t* pr, bool norm) {
  if (!x.x || !x.out) return SPA_ERR_NULL;
  const int64_t st[4] = {x.x_stride_t, x.x_stride_h, x.out_stride_t, x.out_stride_h};
  for (const int64_t s : st)
    if (!stride_ok(s)) return SPA_ERR_SHAPE;
  // output rows are distinct: a token's heads lie within its stride, or a head's tokens within its own
  const int64_t D = pr->head_dim, ot = x.out_stride_t, oh = x.out_stride_h;
  const int T = pr->num_tokens, H = x.num_heads;
  if ((T > 1 && ot < D) || (H > 1 && oh < D) ||
      (T > 1 && H > 1 && (ot - D) / (H - 1) < oh && (oh - D) / (T - 1) < ot))
    return SPA_ERR_SHAPE;
  if (x.x == x.out && ((pr->num_tokens > 1 && x.x_stride_t != x.out_stride_t) ||
                       (x.num_heads > 1 && x.x_stride_h != x.out_stride_h)))
    return SPA_ERR_SHAPE;
  if (!aligned16(x.x) || !aligned16(x.out)) return SPA_ERR_ALIGN;
  for (const int64_t s : st)
    if (s % 8 != 0) return SPA_ERR_ALIGN;
  return norm ? spa::check_norm(x.weight, pr->weight_dtype, pr->eps) : SPA_OK;
}

spa::HeadRows rows(const spa_head_rows_t& x) {
  spa::HeadRows r;
  r.x = static_cast<const uint8_t*>(x.x);
  r.out = static_cast<uint8_t*>(x.out);
  r.weight = x.weight;
  r.x_st = 2 * x.x_stride_t;
  r.x_sh = 2 * x.x_stride_h;
  r.out_st = 2 * x.out_stride_t;
  r.out_sh = 2 * x.out_stride_h;
  r.H = x.num_heads;
  return r;
}

int rope(const spa_rope_problem_t* pr, void* stream, bool norm) {
  if (!pr) return SPA_ERR_NULL;
  if (pr->num_tokens < 0 || pr->head_dim < 1 || pr->q.num_heads < 0 || pr->k.num_heads < 0) return SPA_ERR_SHAPE;
  if (pr->head_dim % 8 != 0 || pr->head_dim > spa::kRopeMaxDim) return SPA_ERR_UNSUPPORTED;
  int st = spa::check_rotary(pr->rope_dim, pr->rope_start, pr->head_dim, pr->rope_scale, pr->turns);
  if (st) return st;
  if (norm && !(pr->eps > 0.f && std::isfinite(pr->eps))) return SPA_ERR_SHAPE;
  const long long heads = (long long)pr->q.num_heads + pr->k.num_heads;
  if ((long long)pr->num_tokens * heads > (1ll << 30)) return SPA_ERR_UNSUPPORTED;
  if (pr->num_tokens == 0 || heads == 0) return SPA_OK;
  if (!pr->positions) return SPA_ERR_NULL;
  for (const spa_head_rows_t* x : {&pr->q, &pr->k}) {
    if (x->num_heads == 0) continue;
    st = check_rows(*x, pr, norm);
    if (st) return st;
  }
  int dev = 0, sms = 0;
  st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::RopeArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = rows(pr->q);
  a.k = rows(pr->k);
  a.rot = rotary(pr->rope_dim, pr->rope_start, pr->interleaved, pr->inverse, pr->rope_scale, pr->turns);
  a.positions = pr->positions;
  a.eps = pr->eps;
  a.T = pr->num_tokens;
  a.D = pr->head_dim;
  a.weight_bf16 = pr->weight_dtype;
  const cudaError_t e = spa::launch_rope(a, norm, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "rope kernel launch");
}

int kv_append(const spa_append_t* pr, const spa_pool_t* pool, void* stream, bool fp8) {
  if (!pr || !pool) return SPA_ERR_NULL;
  if (pr->head_dim < 1) return SPA_ERR_SHAPE;
  if (pr->head_dim % 64 != 0 || pr->head_dim > 512) return SPA_ERR_UNSUPPORTED;
  int st = spa::check_rotary(pr->rope_dim, pr->rope_start, pr->head_dim, pr->rope_scale, pr->turns);
  if (st) return st;
  st = spa::check_append(pr, pr->head_dim, pr->head_dim);
  if (st || pr->num_tokens == 0) return st;
  if (!pool->kv || !pool->block_table || (fp8 && (!pool->k_scale || !pool->v_scale))) return SPA_ERR_NULL;
  if (pool->num_blocks < 1 || pool->page_size < 1 || pool->bt_stride < 1) return SPA_ERR_SHAPE;
  if ((long double)pool->num_blocks * pool->page_size > (long double)(1ll << 30)) return SPA_ERR_UNSUPPORTED;
  if (!aligned16(pool->kv)) return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  st = spa::api_current_device(&dev, &sms);
  if (st) return st;
  spa::AppendArgs a;
  spa::fill_append(a, pr);
  a.pool.rows = static_cast<uint8_t*>(const_cast<void*>(pool->kv));   // written by these calls
  a.pool.bt = pool->block_table;
  a.pool.num_blocks = pool->num_blocks;
  a.pool.ps = pool->page_size;
  a.pool.ps_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.pool.ps == 1 << i) a.pool.ps_shift = i;
  a.pool.bt_stride = pool->bt_stride;
  a.pool.B = pr->num_seqs;
  a.pool.L = pr->head_dim;
  a.k_scale = const_cast<float*>(pool->k_scale);
  a.v_scale = const_cast<float*>(pool->v_scale);
  const cudaError_t e = spa::launch_kv_append(a, fp8, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPA_OK : spa::api_cuda_fail(e, "KV append kernel launch");
}

}  // namespace

namespace spa {

int check_rotary(int32_t rope_dim, int32_t rope_start, int32_t width, float rope_scale, const int64_t* turns) {
  if (rope_dim < 0 || rope_start < 0 || (int64_t)rope_start + rope_dim > width || !std::isfinite(rope_scale))
    return SPA_ERR_SHAPE;
  if (rope_dim % 8 != 0 || rope_dim > kRopeMaxPart || rope_start % 8 != 0) return SPA_ERR_UNSUPPORTED;
  if (rope_dim > 0 && !turns) return SPA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(turns) % 8 != 0) return SPA_ERR_ALIGN;
  return SPA_OK;
}

int check_norm(const void* weight, int32_t weight_dtype, float eps) {
  if (!(eps > 0.f && std::isfinite(eps)) || (weight_dtype != 0 && weight_dtype != 1)) return SPA_ERR_SHAPE;
  return aligned16(weight) ? SPA_OK : SPA_ERR_ALIGN;
}

int check_append(const spa_append_t* pr, int k_width, int v_width) {
  if (pr->num_tokens < 0 || pr->num_seqs < 1 || !stride_ok(pr->k_stride) || !stride_ok(pr->v_stride))
    return SPA_ERR_SHAPE;
  if (pr->norm) {
    const int st = check_norm(pr->weight, pr->weight_dtype, pr->eps);
    if (st) return st;
  }
  if (pr->num_tokens == 0) return SPA_OK;
  if (!pr->positions || (k_width > 0 && !pr->k) || (v_width > 0 && !pr->v)) return SPA_ERR_NULL;
  if (!aligned16(pr->k) || pr->k_stride % 8 != 0) return SPA_ERR_ALIGN;
  if (v_width > 0 && (!aligned16(pr->v) || pr->v_stride % 8 != 0)) return SPA_ERR_ALIGN;
  return SPA_OK;
}

void fill_append(AppendArgs& a, const spa_append_t* pr) {
  std::memset(&a, 0, sizeof a);
  a.rot = rotary(pr->rope_dim, pr->rope_start, pr->interleaved, 0, pr->rope_scale, pr->turns);
  a.k = static_cast<const uint8_t*>(pr->k);
  a.v = static_cast<const uint8_t*>(pr->v);
  a.k_st = 2 * pr->k_stride;
  a.v_st = 2 * pr->v_stride;
  a.weight = pr->weight;
  a.positions = pr->positions;
  a.entries = pr->entries ? pr->entries : pr->positions;
  a.seq_of_token = pr->seq_of_token;
  a.eps = pr->eps;
  a.T = pr->num_tokens;
  a.norm = pr->norm != 0;
  a.weight_bf16 = pr->weight_dtype;
}

}  // namespace spa

extern "C" {

int sparse_attn_rope(const spa_rope_problem_t* prob, void* stream) { return rope(prob, stream, false); }

int sparse_attn_norm_rope(const spa_rope_problem_t* prob, void* stream) { return rope(prob, stream, true); }

int sparse_attn_paged_kv_append(const spa_append_t* prob, const spa_pool_t* pool, void* stream) {
  return kv_append(prob, pool, stream, false);
}

int sparse_attn_paged_kv_append_fp8(const spa_append_t* prob, const spa_pool_t* pool, void* stream) {
  return kv_append(prob, pool, stream, true);
}

}  // extern "C"
