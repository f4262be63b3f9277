// spa_rotary.cu - what lies between a layer's projections and its attention: the norm of every head, the
// rotation of its rotary part by the token's position, and both on the way into a paged cache.
//
//   y = x rsqrt(mean(x^2) + eps) w,      (a, b)_i -> m (a cos t - b sin t, b cos t + a sin t),  t = pos f_i
//
// All of it is a row in, a row out: bound by HBM, or by latency where there are few rows.  A warp takes a
// token's rows of several heads, all loads in flight before any is used; statistics and rotation are
// fp32, with one rounding at the end.  The token's angles are worked out once a warp and serve its heads.
//
// Angles: a position times a frequency loses the angle's fraction in fp32 (at position 2^20 a step is 1/16
// of a radian).  The frequencies come as turns a position in 64-bit binary fractions, so the product modulo
// 2^64 is the fraction of a turn, exactly that of the given frequency at any position; its upper 32 bits
// go to fp32 (off by 2^-32 turns and 2^-24 of itself).  In 64-bit floating point, which this machine
// does at a sixty-fourth of the rate, the angles of 65,536 tokens alone would take about 10 us.
//
// Measured (device time of calls in a graph, inputs that change; % of the measured copy rate):
//   norm and rotation, 8,192 tokens, 64 + 1 heads of 512     173.5 us   6.28 TB/s  93%
//   rotation of 8,192 x 128 heads of 64 in rows of 192        22.1 us   6.07 TB/s  89%
//   norm and rotation, 3,001 tokens, 20 + 4 heads of 128      12.8 us   2.88 TB/s  (issue slots 77% full)
//   K/V append, 65,536 tokens, bf16                           46.7 us   5.76 TB/s  85%   (e4m3 49.5)
//   latent append, 65,536 tokens, e4m3                        27.9 us   4.25 TB/s  63%   (bf16 29.0)
//   one to eight tokens: 2 to 3 us, which is a launch
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_errors.h"
#include "spa_kvwrite_quant.cuh"
#include "spa_rotary.h"
#include "spa_rotary_turn.h"

namespace spa {

namespace {

constexpr int kWarps = 4;

// cos and sin (times the amplitude; sin negated for the inverse) of a pair.
__device__ __forceinline__ float2 cos_sin(const RotaryDev& r, int pos, int pair) {
  float c, s;
  sincospif((float)turn_of(pos, __ldg(r.turns + pair)) * 0x1p-31f, &s, &c);     // (half turns in [-1, 1))
  return make_float2(c * r.scale, s * (r.inverse ? -r.scale : r.scale));
}
// Those of pairs 2w and 2w + 1.
struct Angles {
  float2 t[2];
};
__device__ __forceinline__ Angles angles(const RotaryDev& r, int pos, int w) {
  return Angles{{cos_sin(r, pos, 2 * w), cos_sin(r, pos, 2 * w + 1)}};
}
// The same for w = lane & 15 of a rotary part of at most 64 values: a lane works out one pair (the function is some
// 25 instructions) and takes its two from others.
__device__ __forceinline__ Angles angles_shared(const RotaryDev& r, int pos) {
  const int lane = threadIdx.x & 31, from = (lane & 15) * 2;
  float2 mine = make_float2(0.f, 0.f);
  if (2 * lane < r.R) mine = cos_sin(r, pos, lane);
  Angles a;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    a.t[e] = make_float2(__shfl_sync(0xffffffffu, mine.x, from + e), __shfl_sync(0xffffffffu, mine.y, from + e));
  return a;
}

// Pairs 2w and 2w + 1 of a row's rotary part: (a, b) of each.  Interleaved they are four values in a row, in
// halves two of the first and two of the second half.
struct Pairs {
  uint32_t u, v;
};
__device__ __forceinline__ Pairs load_pairs(const uint8_t* part, const RotaryDev& r, int w) {
  Pairs p;
  if (r.half) {
    p.u = *reinterpret_cast<const uint32_t*>(part + 4 * w);
    p.v = *reinterpret_cast<const uint32_t*>(part + r.R + 4 * w);
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(part + 8 * w);
    p.u = x.x;
    p.v = x.y;
  }
  return p;
}
// The four values in the order in which they lie: half: a0 a1, b0 b1; else a0 b0, a1 b1.
__device__ __forceinline__ void rotate(float (&x)[4], const RotaryDev& r, const Angles& t) {
  const float a0 = x[0], b0 = r.half ? x[2] : x[1], a1 = r.half ? x[1] : x[2], b1 = x[3];
  const float a2 = a0 * t.t[0].x - b0 * t.t[0].y, b2 = b0 * t.t[0].x + a0 * t.t[0].y;
  const float a3 = a1 * t.t[1].x - b1 * t.t[1].y, b3 = b1 * t.t[1].x + a1 * t.t[1].y;
  x[0] = a2;
  x[1] = r.half ? a3 : b2;
  x[2] = r.half ? b2 : a3;
  x[3] = b3;
}
__device__ __forceinline__ void unpack(const Pairs& p, float (&x)[4]) {
  x[0] = bf16_lo(p.u);
  x[1] = bf16_hi(p.u);
  x[2] = bf16_lo(p.v);
  x[3] = bf16_hi(p.v);
}
__device__ __forceinline__ void store_pairs(uint8_t* part, const RotaryDev& r, int w, const float (&x)[4]) {
  const uint32_t u = pack_bf16x2(x[0], x[1]), v = pack_bf16x2(x[2], x[3]);
  if (r.half) {
    *reinterpret_cast<uint32_t*>(part + 4 * w) = u;
    *reinterpret_cast<uint32_t*>(part + r.R + 4 * w) = v;
  } else {
    *reinterpret_cast<uint2*>(part + 8 * w) = make_uint2(u, v);
  }
}

// Weights of eight adjacent values, or of the values of pairs 2w and 2w + 1.
__device__ __forceinline__ void weight8(const void* w, bool bf16, int at, float (&x)[8]) {
  if (bf16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at));
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(v[i]);
      x[2 * i + 1] = bf16_hi(v[i]);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 u = __ldg(f), v = __ldg(f + 1);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  }
}
__device__ __forceinline__ void weight_pairs(const void* wt, bool bf16, const RotaryDev& r, int w, float (&x)[4]) {
  const int at = r.start + (r.half ? 2 * w : 4 * w), to = r.half ? at + r.R / 2 : at + 2;
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(wt);
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p + at)), v = __ldg(reinterpret_cast<const uint32_t*>(p + to));
    x[0] = bf16_lo(u), x[1] = bf16_hi(u), x[2] = bf16_lo(v), x[3] = bf16_hi(v);
  } else {
    const float* p = static_cast<const float*>(wt);
    const float2 u = __ldg(reinterpret_cast<const float2*>(p + at)), v = __ldg(reinterpret_cast<const float2*>(p + to));
    x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float sum_squares(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), s);
    s = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), s);
  }
  return s;
}

// The column of 16-byte chunk c of the values that are not rotated.
__device__ __forceinline__ int plain_column(const RotaryDev& r, int c) { return 8 * c < r.start ? 8 * c : 8 * c + r.R; }

// (x, y) *= (a, b), two values an instruction
__device__ __forceinline__ void mul_f32x2(float& x, float& y, float a, float b) {
  asm("{ .reg .b64 v, c; mov.b64 v, {%0, %1}; mov.b64 c, {%2, %3}; mul.rn.f32x2 v, v, c; mov.b64 {%0, %1}, v; }"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// kC: 16-byte chunks a lane of the values that are not rotated (0: none, or they stay where they are); kW: fours of
// rotated values a lane and row, or 0: rows of at most 64 rotated values, two rows at once, a half-warp each;
// kRows: heads of a token a warp takes at once, enough that their loads cover the latency and not so many that
// registers leave too few warps.  Measured: norm, 8,192 x 65 rows of 512: 4 rows 173 us, 2 rows 200 to 224, 1 row 265.
// Rotation alone of 64 values, 8,192 x 128 rows: 16 rows 22.2 us, 8 rows 24 to 26, 4 rows 36, 2 rows 53; of rows of
// 128 values 4 rows 12.6 us, 8 rows 14.4, 2 rows 15.4, 16 rows 20.6.
template <int kC, int kW, int kRows, bool kNorm>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const RopeArgs a, int units_q, int units_k) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kP = kW ? kRows * kW : (kRows + 1) / 2;    // fours of rotated values a lane
  const int lane = threadIdx.x & 31;
  // row (of the group) and four (of the row) of slot i
  const auto row_of = [&](int i) { return kW ? i / (kW ? kW : 1) : 2 * i + (lane >> 4); };
  const auto four_of = [&](int i) { return kW ? lane + 32 * (i % (kW ? kW : 1)) : lane & 15; };
  const int per_token = units_q + units_k;
  const int units = a.T * per_token;             // (checked by the caller to fit)
  const int n_plain = (a.D - a.rot.R) >> 3, n_pairs = a.rot.R >> 2;
  const float inv_d = 1.f / (float)a.D;
  for (int u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const int t = u / per_token, g = u - t * per_token;
    const bool is_k = g >= units_q;
    const HeadRows& x = is_k ? a.k : a.q;
    const int h0 = (is_k ? g - units_q : g) * kRows;
    const int pos = __ldg(a.positions + t);
    const uint8_t* src = x.x + t * x.x_st + h0 * x.x_sh;
    uint8_t* dst = x.out + t * x.out_st + h0 * x.out_sh;
    const int rows = min(kRows, x.H - h0);
    uint4 plain[kRows][kC ? kC : 1];
    Pairs pair[kP];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint8_t* row = src + (i < rows ? i : 0) * x.x_sh;
#pragma unroll
      for (int c = 0; c < kC; ++c)
        plain[i][c] = lane + 32 * c < n_plain
                          ? *reinterpret_cast<const uint4*>(row + 2 * plain_column(a.rot, lane + 32 * c))
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int r = row_of(i), w = four_of(i);
      pair[i].u = pair[i].v = 0;
      if (w < n_pairs && r < rows) pair[i] = load_pairs(src + r * x.x_sh + 2 * a.rot.start, a.rot, w);
    }
    float inv[kRows];
    if constexpr (kNorm) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) s += sum_squares(plain[i][c]);
        inv[i] = s;
      }
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float s = sum_squares(make_uint4(pair[i].u, pair[i].v, 0, 0));
        if (kW) {
          inv[i / (kW ? kW : 1)] += s;
        } else {
          inv[2 * i] += lane < 16 ? s : 0.f;
          if (2 * i + 1 < kRows) inv[2 * i + 1] += lane < 16 ? 0.f : s;
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) inv[i] = rsqrtf(fmaf(warp_sum(inv[i]), inv_d, a.eps));
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (lane + 32 * c >= n_plain) continue;
      const int col = plain_column(a.rot, lane + 32 * c);
      float wt[8];
      if constexpr (kNorm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) wt[e] = 1.f;
        if (x.weight) weight8(x.weight, a.weight_bf16, col, wt);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        uint4 o = plain[i][c];
        if constexpr (kNorm) {
          uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float p = bf16_lo(v[e]), q = bf16_hi(v[e]);
            mul_f32x2(p, q, inv[i], inv[i]);
            mul_f32x2(p, q, wt[2 * e], wt[2 * e + 1]);
            v[e] = pack_bf16x2(p, q);
          }
          o = make_uint4(v[0], v[1], v[2], v[3]);
        }
        *reinterpret_cast<uint4*>(dst + i * x.out_sh + 2 * col) = o;
      }
    }
    Angles an[kW ? kW : 1];
    if constexpr (kW == 0) {
      an[0] = angles_shared(a.rot, pos);
    } else {
#pragma unroll
      for (int w = 0; w < kW; ++w)
        if (lane + 32 * w < n_pairs) an[w] = angles(a.rot, pos, lane + 32 * w);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const int r = row_of(i), w = four_of(i);
      if (w >= n_pairs || r >= rows) continue;
      float v[4];
      unpack(pair[i], v);
      if constexpr (kNorm) {
        float wt[4] = {1.f, 1.f, 1.f, 1.f};
        if (x.weight) weight_pairs(x.weight, a.weight_bf16, a.rot, w, wt);
        const float f = kW ? inv[i / (kW ? kW : 1)]
                           : lane < 16 ? inv[2 * i < kRows ? 2 * i : 0] : inv[2 * i + 1 < kRows ? 2 * i + 1 : 0];
        mul_f32x2(v[0], v[1], f, f);
        mul_f32x2(v[2], v[3], f, f);
        mul_f32x2(v[0], v[1], wt[0], wt[1]);
        mul_f32x2(v[2], v[3], wt[2], wt[3]);
      }
      rotate(v, a.rot, an[kW ? i % (kW ? kW : 1) : 0]);
      store_pairs(dst + r * x.out_sh + 2 * a.rot.start, a.rot, w, v);
    }
  }
}

template <int kC, int kW, int kRows>
cudaError_t launch_rope_as(const RopeArgs& a, bool norm, int sms, cudaStream_t stream) {
  const int uq = (a.q.H + kRows - 1) / kRows, uk = (a.k.H + kRows - 1) / kRows;
  const long long blocks = ((long long)a.T * (uq + uk) + kWarps - 1) / kWarps, cap = 64LL * sms;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  return launch_with_pdl(norm ? rope_kernel<kC, kW, kRows, true> : rope_kernel<kC, kW, kRows, false>, dim3(grid),
                         dim3(32 * kWarps), 0, stream, 2LL * grid <= sms, a, uq, uk);
}

template <int kC, int kRows, int kWide = kRows>
cudaError_t launch_rope_width(const RopeArgs& a, bool norm, int sms, cudaStream_t stream) {
  if (a.rot.R <= 64) return launch_rope_as<kC, 0, kRows>(a, norm, sms, stream);
  return a.rot.R <= 128 ? launch_rope_as<kC, 1, kWide>(a, norm, sms, stream)
                        : launch_rope_as<kC, 2, kWide>(a, norm, sms, stream);
}

// ---- appends --------------------------------------------------------------------------------
__device__ __forceinline__ int append_row(const AppendArgs& a, int t) {
  const int x = __ldg(a.entries + t);
  const int b = a.seq_of_token ? __ldg(a.seq_of_token + t) : 0;
  if (x < 0 || b < 0 || b >= a.pool.B) return -1;
  return latent_row(a.pool, b, x);
}

// (At least fp32's smallest number: normalised or rotated values may be so small that the quotient is zero, and zeros
// over it would be NaN.)
__device__ __forceinline__ float row_scale(float amax) {
  return amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), __int_as_float(1)) : 1.f;
}
__device__ __forceinline__ float warp_max(float m) {   // of values >= 0 (their bits order as they do)
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// A row's values in fp32: a lane's 16-byte chunks (two: rows of up to 512) and fours of rotated ones.
template <int kW>
struct Row {
  float x[2][8], r[kW][4];
};
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <int N>
__device__ __forceinline__ void scale_by(float (&x)[N], float f) {
#pragma unroll
  for (int e = 0; e < N; e += 2) mul_f32x2(x[e], x[e + 1], f, f);
}
template <int N>
__device__ __forceinline__ void scale_by(float (&x)[N], const float (&w)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 2) mul_f32x2(x[e], x[e + 1], w[e], w[e + 1]);
}
template <int N>
__device__ __forceinline__ float abs_max(const float (&x)[N], float m) {   // (a NaN does not enter it)
#pragma unroll
  for (int e = 0; e < N; ++e) m = fmaxf(m, fabsf(x[e]));
  return m;
}
template <int N>
__device__ __forceinline__ float squares(const float (&x)[N], float s) {
#pragma unroll
  for (int e = 0; e < N; ++e) s = fmaf(x[e], x[e], s);
  return s;
}

// A K row, normalised.
template <int kW>
__device__ __forceinline__ void norm_row(Row<kW>& y, const AppendArgs& a, int width, int n_plain, int n_pairs) {
  const int lane = threadIdx.x & 31;
  float s = squares(y.x[1], squares(y.x[0], 0.f));
#pragma unroll
  for (int w = 0; w < kW; ++w) s = squares(y.r[w], s);
  const float inv = rsqrtf(warp_sum(s) / (float)width + a.eps);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    scale_by(y.x[c], inv);
    if (a.weight && lane + 32 * c < n_plain) {
      float wt[8];
      weight8(a.weight, a.weight_bf16, plain_column(a.rot, lane + 32 * c), wt);
      scale_by(y.x[c], wt);
    }
  }
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    scale_by(y.r[w], inv);
    if (a.weight && lane + 32 * w < n_pairs) {
      float wt[4];
      weight_pairs(a.weight, a.weight_bf16, a.rot, lane + 32 * w, wt);
      scale_by(y.r[w], wt);
    }
  }
}

template <int kW>
__device__ __forceinline__ float row_amax(const Row<kW>& y) {
  float m = abs_max(y.x[1], abs_max(y.x[0], 0.f));
#pragma unroll
  for (int w = 0; w < kW; ++w) m = abs_max(y.r[w], m);
  return warp_max(m);
}

// Values over the row's scale, in place: by its reciprocal where that is a normal number (the quotient is then off by
// two units in its last place, next to which the values' own roundings are no smaller), else divided.  Out of
// line: rows with so small a scale are rare, and a division for every value would be most of the kernel's code.
__device__ __noinline__ float divided(float x, float scale) { return __fdiv_rn(x, scale); }
template <int kC, int kR>
__device__ __forceinline__ void divide(float (&x)[kC][8], float (&r)[kR], float scale) {
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[c][e] = divided(x[c][e], scale);
#pragma unroll
  for (int e = 0; e < kR; ++e) r[e] = divided(r[e], scale);
}
template <int kW>
__device__ __forceinline__ void over_scale(Row<kW>& y, float scale) {
  if (!kvq_fast_scale(scale)) {
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w == 0) divide(y.x, y.r[0], scale);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) y.r[w][e] = divided(y.r[w][e], scale);
    }
    return;
  }
  const float r = __frcp_rn(scale);
  scale_by(y.x[0], r);
  scale_by(y.x[1], r);
#pragma unroll
  for (int w = 0; w < kW; ++w) scale_by(y.r[w], r);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return kvq_e4m3x2(a, b) | (kvq_e4m3x2(c, d) << 16);
}
__device__ __forceinline__ uint2 codes8(const float (&e)[8]) {
  return make_uint2(codes4(e[0], e[1], e[2], e[3]), codes4(e[4], e[5], e[6], e[7]));
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
// Four codes of a rotary part (of bytes).
__device__ __forceinline__ void store_codes(uint8_t* part, const RotaryDev& r, int w, uint32_t code) {
  if (r.half) {
    *reinterpret_cast<uint16_t*>(part + 2 * w) = (uint16_t)code;
    *reinterpret_cast<uint16_t*>(part + r.R / 2 + 2 * w) = (uint16_t)(code >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(part + 4 * w) = code;
  }
}

// CTAs an SM.  Measured at 65,536 tokens: K/V, bf16: 8 CTAs 46.6 us, 6 52.5, 12 58, 16 97; latent, e4m3: 8 CTAs
// 27.9 us, 7 30.6, 6 31.5, 10 33.
constexpr int kAppendBlocks = 8, kLatentBlocks = 8;

// K rows (normalised, rotated) and V rows (as they are) of new tokens into their slots.  A warp a token; kW: fours
// of rotated values a lane, 0: at most 64 values.
template <bool kFp8, int kW>
__global__ void __launch_bounds__(32 * kWarps, kAppendBlocks) kv_append_kernel(const AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kR = kW ? kW : 1;
  const int lane = threadIdx.x & 31, D = a.pool.L;
  const int n_plain = (D - a.rot.R) >> 3, n_pairs = a.rot.R >> 2, n_all = D >> 3;
  const long long step = (long long)gridDim.x * kWarps;
  for (long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += step) {
    const uint8_t *k = a.k + t * a.k_st, *v = a.v + t * a.v_st;
    uint4 kx[2], vx[2];
    Pairs kp[kR];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      kx[c] = vx[c] = make_uint4(0, 0, 0, 0);
      if (lane + 32 * c < n_plain)
        kx[c] = __ldg(reinterpret_cast<const uint4*>(k + 2 * plain_column(a.rot, lane + 32 * c)));
      if (lane + 32 * c < n_all) vx[c] = __ldg(reinterpret_cast<const uint4*>(v) + lane + 32 * c);
    }
#pragma unroll
    for (int w = 0; w < kR; ++w) {
      kp[w].u = kp[w].v = 0;
      if (lane + 32 * w < n_pairs) kp[w] = load_pairs(k + 2 * a.rot.start, a.rot, lane + 32 * w);
    }
    const int pos = __ldg(a.positions + t), row = append_row(a, (int)t);
    if (row < 0) {
      if (lane == 0) flag_error(SPA_ERR_INDEX);
      continue;
    }
    Row<kR> y;
#pragma unroll
    for (int c = 0; c < 2; ++c) unpack8(kx[c], y.x[c]);
#pragma unroll
    for (int w = 0; w < kR; ++w) unpack(kp[w], y.r[w]);
    if (a.norm) norm_row(y, a, D, n_plain, n_pairs);
    if constexpr (kW == 0) {
      rotate(y.r[0], a.rot, angles_shared(a.rot, pos));    // (zeros where a lane has none)
    } else {
#pragma unroll
      for (int w = 0; w < kR; ++w)
        if (lane + 32 * w < n_pairs) rotate(y.r[w], a.rot, angles(a.rot, pos, lane + 32 * w));
    }
    if constexpr (!kFp8) {
      uint8_t* dst = a.pool.rows + (size_t)row * 4 * D;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (lane + 32 * c < n_plain)
          *reinterpret_cast<uint4*>(dst + 2 * plain_column(a.rot, lane + 32 * c)) = pack8(y.x[c]);
        if (lane + 32 * c < n_all) reinterpret_cast<uint4*>(dst + 2 * D)[lane + 32 * c] = vx[c];
      }
#pragma unroll
      for (int w = 0; w < kR; ++w)
        if (lane + 32 * w < n_pairs) store_pairs(dst + 2 * a.rot.start, a.rot, lane + 32 * w, y.r[w]);
    } else {
      const float ks = row_scale(row_amax(y));
      over_scale(y, ks);
      uint32_t vm = 0;                           // (bf16's bits order as their magnitudes do)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        for (const uint32_t z : {vx[c].x, vx[c].y, vx[c].z, vx[c].w}) {
          asm("max.bf16x2 %0, %0, %1;" : "+r"(vm) : "r"(z & 0x7fff7fffu));
        }
      vm = __reduce_max_sync(0xffffffffu, max(vm & 0xffffu, vm >> 16));
      const float vs = row_scale(bf16_lo(vm)), vr = __frcp_rn(vs);
      uint8_t* dst = a.pool.rows + (size_t)row * 2 * D;
      uint2* dst_v = reinterpret_cast<uint2*>(dst + D);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (lane + 32 * c < n_plain)
          *reinterpret_cast<uint2*>(dst + plain_column(a.rot, lane + 32 * c)) = codes8(y.x[c]);
      if (kvq_fast_scale(vs)) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (lane + 32 * c < n_all) dst_v[lane + 32 * c] = kvq_chunk(vx[c], vs, vr, true);
      } else {
#pragma unroll 1
        for (int c = 0; c < 2; ++c)
          if (lane + 32 * c < n_all) dst_v[lane + 32 * c] = kvq_chunk(c == 0 ? vx[0] : vx[1], vs, vr, false);
      }
#pragma unroll
      for (int w = 0; w < kR; ++w)
        if (lane + 32 * w < n_pairs)
          store_codes(dst + a.rot.start, a.rot, lane + 32 * w, codes4(y.r[w][0], y.r[w][1], y.r[w][2], y.r[w][3]));
      if (lane == 0) {
        a.k_scale[row] = ks;
        a.v_scale[row] = vs;
      }
    }
  }
}

// Latent rows [norm(c) | rotated r] of new tokens into their slots; e4m3: r as a high and a low code.  A half-warp a
// token (four 16-byte chunks a lane, and its rotary part fills sixteen lanes): what is done once a row, addresses,
// reductions and angles, then costs two rows one instruction.  With a warp a token it was 419 instructions a row, and
// the e4m3 append of 65,536 rows took 35 us.
template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps, kLatentBlocks) latent_append_kernel(const AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kC = kLatMaxDim / 8 / 16;
  const int w = threadIdx.x & 15, L = a.pool.L;
  const int nl = L >> 3, n_pairs = a.rot.R >> 2;
  const float inv_l = 1.f / (float)L;
  const long long step = 2LL * gridDim.x * kWarps;
  // (both halves of a warp take the same trips)
  for (long long t0 = 2LL * (blockIdx.x * kWarps + (threadIdx.x >> 5)); t0 < a.T; t0 += step) {
    const long long t = t0 + ((threadIdx.x >> 4) & 1);
    const bool there = t < a.T;
    const uint8_t* k = a.k + t * a.k_st;
    uint4 raw[kC];
    Pairs p;
    p.u = p.v = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      raw[c] = there && w + 16 * c < nl ? __ldg(reinterpret_cast<const uint4*>(k) + w + 16 * c) : make_uint4(0, 0, 0, 0);
    if (there && w < n_pairs) p = load_pairs(a.v + t * a.v_st, a.rot, w);
    int row = -1, pos = 0;
    if (there) {
      pos = __ldg(a.positions + t);
      row = append_row(a, (int)t);
      if (row < 0 && w == 0) flag_error(SPA_ERR_INDEX);
    }
    float x[kC][8], r[4];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      unpack8(raw[c], x[c]);
      if (a.norm) s = squares(x[c], s);
    }
    unpack(p, r);
    if (a.norm) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float inv = rsqrtf(fmaf(s, inv_l, a.eps));
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        scale_by(x[c], inv);
        if (a.weight && w + 16 * c < nl) {
          float wt[8];
          weight8(a.weight, a.weight_bf16, 8 * (w + 16 * c), wt);
          scale_by(x[c], wt);
        }
      }
    }
    if (w < n_pairs) rotate(r, a.rot, angles(a.rot, pos, w));
    uint8_t* dst = a.pool.rows + (size_t)(row < 0 ? 0 : row) * a.pool.row_bytes;
    if constexpr (!kFp8) {
      if (row >= 0) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (w + 16 * c < nl) reinterpret_cast<uint4*>(dst)[w + 16 * c] = pack8(x[c]);
        if (w < n_pairs) store_pairs(dst + 2 * L, a.rot, w, r);
      }
    } else {
      float m = abs_max(r, 0.f);
#pragma unroll
      for (int c = 0; c < kC; ++c) m = abs_max(x[c], m);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float scale = row_scale(m);
      if (kvq_fast_scale(scale)) {
        const float f = __frcp_rn(scale);
#pragma unroll
        for (int c = 0; c < kC; ++c) scale_by(x[c], f);
        scale_by(r, f);
      } else {
        divide(x, r, scale);
      }
      if (row >= 0) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (w + 16 * c < nl) reinterpret_cast<uint2*>(dst)[w + 16 * c] = codes8(x[c]);
        if (w < n_pairs) {
          uint32_t high[2], low[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            high[i] = kvq_e4m3x2(r[2 * i], r[2 * i + 1]);
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)high[i], __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            low[i] = kvq_e4m3x2(r[2 * i] - f.x, r[2 * i + 1] - f.y);
          }
          store_codes(dst + L, a.rot, w, high[0] | (high[1] << 16));
          store_codes(dst + L + a.rot.R, a.rot, w, low[0] | (low[1] << 16));
        }
        if (w == 0) a.k_scale[row] = scale;
      }
    }
  }
}

unsigned append_blocks(long long warps, long long cap) {
  const long long b = (warps + kWarps - 1) / kWarps;
  return (unsigned)(b < cap ? b : cap);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool norm, int sms, cudaStream_t stream) {
  // In place and without a norm the values that are not rotated stay as they are.
  const bool in_place = !norm && a.q.x == a.q.out && (a.k.H == 0 || a.k.x == a.k.out);
  const int chunks = in_place ? 0 : (a.D - a.rot.R) / 8;
  if (chunks == 0) return launch_rope_width<0, 16, 4>(a, norm, sms, stream);
  if (chunks <= 32) return launch_rope_width<1, 4>(a, norm, sms, stream);
  if (chunks <= 64) return launch_rope_width<2, 4>(a, norm, sms, stream);
  return launch_rope_width<4, 2>(a, norm, sms, stream);
}

cudaError_t launch_kv_append(const AppendArgs& a, bool fp8, int sms, cudaStream_t stream) {
  const unsigned blocks = append_blocks(a.T, 2LL * kAppendBlocks * sms);
  const auto kern = a.rot.R <= 64 ? (fp8 ? kv_append_kernel<true, 0> : kv_append_kernel<false, 0>)
                                  : (fp8 ? kv_append_kernel<true, 2> : kv_append_kernel<false, 2>);
  return launch_with_pdl(kern, dim3(blocks), dim3(32 * kWarps), 0, stream, 2LL * blocks <= sms, a);
}

cudaError_t launch_latent_append(const AppendArgs& a, bool fp8, int sms, cudaStream_t stream) {
  const unsigned blocks = append_blocks(((long long)a.T + 1) / 2, (long long)kLatentBlocks * sms);
  return launch_with_pdl(fp8 ? latent_append_kernel<true> : latent_append_kernel<false>, dim3(blocks),
                         dim3(32 * kWarps), 0, stream, 2LL * blocks <= sms, a);
}

// This translation unit's copy of the device error word (see spa_device.cuh).
cudaError_t rotary_error_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_spa_error);
}

}  // namespace spa
