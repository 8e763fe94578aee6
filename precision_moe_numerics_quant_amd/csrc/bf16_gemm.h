// Shared pieces of the BF16 expert products (gfx950): the calls' arguments,
// the gathered rows and the epilogues.
#pragma once
#include "gemm_common.h"
#include "moe4_internal.h"

namespace moe4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The products with row groups, all C[rows of e] = A[rows of e] . B_e:
//   FWD     B_e = w[e]^T, w [E, N, K];  c = act(z + bias) + residual, pre = z + bias
//   GATED   B_e = w[e]^T, w [E, 2, N, K] (N the block's hidden width): z_0 and
//           z_1 of one column together;  h = act(z_0 + bias) (z_1 + bias), both kept
//   DGRAD   B_e = w[e], w [E, K, N] (the contraction runs over w's rows);
//           c = scale z act'(pre), hs = scale act(pre)
//   GDGRAD  as DGRAD through the gated product: dh = scale z,
//           dg = dh u act'(g), du = dh act(g), hs = scale act(g) u
enum Bf16Mode { FWD, GATED, DGRAD, GDGRAD };

struct Bf16Args {
  const uint16_t* a;    // [a_rows, K]; row r of the product is a[map[r] / div] (no map: a[r])
  const int32_t* map;
  const uint16_t* w;
  const int32_t* off;   // [E + 1]
  const float* bias;    // FWD [E, N], GATED [E, 2, N], or NULL
  const float* scale;   // [a_rows div] by the map's entry (no map: [M] by row), or NULL
  const uint16_t* in;   // DGRAD pre, GDGRAD gu, or NULL
  const void* res;      // FWD, DGRAD: added at the end (c's type), or NULL
  void* c;              // FWD, DGRAD: [M, N] float32 or bf16; GATED h [M, N]; GDGRAD dgu [M, 2, N]
  uint16_t* aux;        // pre, gu or hs (bf16), or NULL
  int64_t a_rows, M, N, K;  // N: C's columns, K: the contraction
  uint32_t div, magic;  // magic = floor(2^32 / div), 2^32 - 1 for div = 1
  int E, act;
};

// n / div for n < 2^32: the high word of n magic is the quotient or one below
// it (n (2^32 mod div) / (2^32 div) < 1).
__device__ inline uint32_t udiv_magic(uint32_t n, uint32_t div, uint32_t magic) {
  const uint32_t q = __umulhi(n, magic);
  return q + (n - q * div >= div ? 1u : 0u);
}

// Row r of the routed matrix in memory, or -1 (reported) for a map entry
// outside [0, a_rows div).
__device__ inline int64_t mapped_row(const int32_t* map, int64_t r, uint32_t div, uint32_t magic, int64_t rows, uint32_t* err) {
  if (map == nullptr) return r;
  const uint32_t t = udiv_magic((uint32_t)map[r], div, magic);
  if (map[r] < 0 || t >= rows) {
    atomicOr(err, MOE4_DEVERR_INDEX);
    return -1;
  }
  return t;
}

// The scale of row r (0 for a map entry outside [0, n), whose row is zeros).
__device__ inline float row_scale(const float* scale, const int32_t* map, int64_t r, int64_t n) {
  if (scale == nullptr) return 1.0f;
  if (map == nullptr) return scale[r];
  const int32_t i = map[r];
  return i >= 0 && i < n ? scale[i] : 0.0f;
}

// ------------------------------------------------------------- activations
// act(x) = x t with t = sigmoid(p): p = x (SiLU), or GELU by its tanh form,
// whose (1 + tanh(v)) / 2 is sigmoid(2 v); act'(x) = t + x t (1 - t) p'.
// EXACT (float32 results): exp and the division to within an ulp; otherwise
// the hardware's exp2 and reciprocal, whose relative error (|p| 2^-24 and 1 ulp)
// is far below the half step of 2^-9 that rounding to bf16 costs.
// Infinities: act(-inf) = -0, act(inf) = inf, act' = 0 and 1 there.
template <bool EXACT>
__device__ inline float sigmoid_of(float p) {
  if (EXACT) return 1.0f / (1.0f + expf(-p));
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(p * -1.44269504f));
}
template <bool EXACT>
__device__ inline void act_of(int act, float x, float& f, float& df) {
  constexpr float C = 1.5957691216f, B = 0.044715f;  // 2 sqrt(2 / pi)
  if (act == MOE4_ACT_NONE) {
    f = x;
    df = 1.0f;
    return;
  }
  float p = x, dp = 1.0f;
  if (act == MOE4_ACT_GELU) {
    const float x2 = x * x;
    p = C * fmaf(B * x2, x, x);
    dp = fmaf(3.0f * B * C, x2, C);
  }
  const float t = sigmoid_of<EXACT>(p), s = t * (1.0f - t);
  f = t == 0.0f ? -0.0f : x * t;
  // (x s before dp: x^2 alone may exceed the range where s x dp does not)
  df = s == 0.0f ? t : fmaf(x * s, dp, t);
}

// ---------------------------------------------------------------- epilogues
// W consecutive values, W % 4 == 0
template <int W>
__device__ inline void load_bf16(const uint16_t* p, float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(p + i);
    v[i] = bf16_bits_to_f32(q[0] & 0xFFFFu);
    v[i + 1] = bf16_bits_to_f32(q[0] >> 16);
    v[i + 2] = bf16_bits_to_f32(q[1] & 0xFFFFu);
    v[i + 3] = bf16_bits_to_f32(q[1] >> 16);
  }
}
template <int W>
__device__ inline void load_f32(const float* p, float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const f32x4 q = *reinterpret_cast<const f32x4*>(p + i);
    v[i] = q[0]; v[i + 1] = q[1]; v[i + 2] = q[2]; v[i + 3] = q[3];
  }
}
template <int W>
__device__ inline void store_bf16(uint16_t* p, const float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) *reinterpret_cast<u32x2*>(p + i) = u32x2{bf16_pair(v[i], v[i + 1]), bf16_pair(v[i + 2], v[i + 3])};
}
template <int W>
__device__ inline void store_f32(float* p, const float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// c = q + res, at element `at`
template <bool OUT_BF16, int W>
__device__ inline void add_store(const Bf16Args& p, int64_t at, float (&q)[W]) {
  if (p.res) {
    float v[W];
    if (OUT_BF16) load_bf16<W>(static_cast<const uint16_t*>(p.res) + at, v);
    else load_f32<W>(static_cast<const float*>(p.res) + at, v);
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = q[i] + v[i];
  }
  if (OUT_BF16) store_bf16<W>(static_cast<uint16_t*>(p.c) + at, q);
  else store_f32<W>(static_cast<float*>(p.c) + at, q);
}

// The W results z (GATED: z and z1) of row r, columns n .. n + W - 1, of expert e.
template <int MODE, bool OUT_BF16, int W>
__device__ inline void bf16_epilogue(const Bf16Args& p, int e, int64_t r, int64_t n, const float (&z)[W], const float (&z1)[W]) {
  const int64_t at = r * p.N + n;
  float v[W], h[W];
  if (MODE == FWD) {
    float q[W];
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = z[i];
    if (p.bias) {
      load_f32<W>(p.bias + e * p.N + n, v);
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = q[i] + v[i];
    }
    if (p.aux) store_bf16<W>(p.aux + at, q);
    if (p.act != MOE4_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float d;
        act_of<!OUT_BF16>(p.act, q[i], h[i], d);
        q[i] = h[i];
      }
    }
    add_store<OUT_BF16, W>(p, at, q);
  } else if (MODE == GATED) {
    float g[W], u[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      g[i] = z[i];
      u[i] = z1[i];
    }
    if (p.bias) {
      load_f32<W>(p.bias + (int64_t)e * 2 * p.N + n, v);
#pragma unroll
      for (int i = 0; i < W; ++i) g[i] = g[i] + v[i];
      load_f32<W>(p.bias + ((int64_t)e * 2 + 1) * p.N + n, v);
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] = u[i] + v[i];
    }
    if (p.aux) {
      store_bf16<W>(p.aux + 2 * r * p.N + n, g);
      store_bf16<W>(p.aux + (2 * r + 1) * p.N + n, u);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float d;
      act_of<false>(p.act, g[i], h[i], d);
      h[i] = h[i] * u[i];
    }
    store_bf16<W>(static_cast<uint16_t*>(p.c) + at, h);
  } else {
    const float s = row_scale(p.scale, p.map, r, p.a_rows * p.div);
    float q[W];
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = s * z[i];
    if (MODE == DGRAD) {
      if (p.in) {
        load_bf16<W>(p.in + at, v);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          float d;
          act_of<!OUT_BF16>(p.act, v[i], h[i], d);
          q[i] = q[i] * d;
          h[i] = s * h[i];
        }
        if (p.aux) store_bf16<W>(p.aux + at, h);
      }
      add_store<OUT_BF16, W>(p, at, q);
    } else {
      float u[W];
      const uint16_t* gu = p.in + 2 * r * p.N + n;
      load_bf16<W>(gu, v);
      load_bf16<W>(gu + p.N, u);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float f, d;
        act_of<false>(p.act, v[i], f, d);
        h[i] = s * (f * u[i]);
        v[i] = q[i] * u[i] * d;
        u[i] = q[i] * f;
      }
      if (p.aux) store_bf16<W>(p.aux + at, h);
      uint16_t* d = static_cast<uint16_t*>(p.c) + 2 * r * p.N + n;
      store_bf16<W>(d, v);
      store_bf16<W>(d + p.N, u);
    }
  }
}

// The weight gradient: dw[e] = beta dw[e] + sum over e's rows r of dy[r]^T a[r],
// db[e] = beta db[e] + sum of db_scale[r] dy[r]; each operand with a map or without.
struct Bf16Wgrad {
  const uint16_t *dy, *a;
  const int32_t *dy_map, *a_map, *off;
  const float* db_scale;
  float *dw, *db;
  int64_t dy_rows, a_rows, M, N, K;
  uint32_t div, magic;
  int E;
  float beta;
  bool zero_empty;
};

}  // namespace moe4
