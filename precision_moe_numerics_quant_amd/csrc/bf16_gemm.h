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
// act(x) = x t with t = sigmoid(p), p = x (c1 + c3 x^2): SiLU has c1 = 1, c3 = 0;
// GELU by its tanh form, whose (1 + tanh(v)) / 2 is sigmoid(2 v), c1 = 2 sqrt(2 / pi)
// and c3 = 0.044715 c1.  act'(x) = t + x t (1 - t) p'.
// EXACT (float32 results): exp and the division to within an ulp; otherwise
// the hardware's exp2 and reciprocal, whose relative error (|p| 2^-24 and 1 ulp)
// is far below the half step of 2^-8 that rounding to bf16 costs.
// Infinities: act(-inf) = -0, act(inf) = inf, act' = 0 and 1 there.
// Below p = FAR t leaves float32's range before x t does (exp(-p) overflows at
// -88.7: SiLU of -89 is -2e-37), and 1 + exp(-p) is exp(-p) to all bits: there t =
// h^2 with h = exp(p / 2), a factor at a time.  Hardly any value is so far out, so the
// values of one store are looked at together: a minimum each, one branch.
struct ActCoef {
  float c1, c3;
  __host__ __device__ ActCoef(int act) : c1(act == MOE4_ACT_GELU ? 1.5957691216f : 1.0f), c3(act == MOE4_ACT_GELU ? 1.5957691216f * 0.044715f : 0.0f) {}
};
template <bool EXACT>
__device__ inline float sigmoid_of(float p) {
  if (EXACT) return 1.0f / (1.0f + expf(-p));
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(p * -1.44269504f));
}
constexpr float FAR = -80.0f;
template <bool EXACT, int W>
__device__ inline void act_of(const ActCoef& a, const float (&x)[W], float (&f)[W], float (&df)[W]) {
  float least = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float x2 = fminf(x[i] * x[i], 1e30f);   // (x^2 past the range, times c3 = 0)
    const float p = x[i] * fmaf(a.c3, x2, a.c1), t = sigmoid_of<EXACT>(p), s = t * (1.0f - t);
    least = fminf(least, p);
    f[i] = x[i] * t;
    // (x s before p': x^2 alone may exceed the range where s x p' does not)
    df[i] = s == 0.0f ? t : fmaf(x[i] * s, fmaf(3.0f * a.c3, x2, a.c1), t);
  }
  if (least < FAR) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x2 = fminf(x[i] * x[i], 1e30f), p = x[i] * fmaf(a.c3, x2, a.c1);
      const float h = EXACT ? expf(0.5f * p) : __builtin_amdgcn_exp2f(p * 0.72134752f);
      if (p < FAR) {
        f[i] = h == 0.0f ? -0.0f : x[i] * h * h;
        df[i] = h == 0.0f ? 0.0f : h * fmaf(x[i], fmaf(3.0f * a.c3, x2, a.c1), 1.0f) * h;
      }
    }
  }
}

// ---------------------------------------------------------------- epilogues
// Buffer accesses of W consecutive values (4 or 8) at an element offset from
// the descriptor's base; PAST as the offset reads zeros and stores nothing.
constexpr uint32_t PAST = 0x20000000u;   // (times 4 or 2 bytes: past 2^30, the largest descriptor here, and no wrap)
template <int W>
__device__ inline void load_words(const __amdgpu_buffer_rsrc_t& rs, uint32_t o, uint32_t (&q)[W / 2]) {   // W bf16 values
  if (W == 8) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b128(rs, o * 2, 0, 0);
    q[0] = x[0]; q[1] = x[1]; q[W / 2 - 2] = x[2]; q[W / 2 - 1] = x[3];
  } else {
    const auto x = __builtin_amdgcn_raw_buffer_load_b64(rs, o * 2, 0, 0);
    q[0] = x[0]; q[1] = x[1];
  }
}
template <int W>
__device__ inline void values_of(const uint32_t (&q)[W / 2], float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = bf16_bits_to_f32((i & 1) ? q[i / 2] >> 16 : q[i / 2] & 0xFFFFu);
}
template <int W>
__device__ inline void load_f32(const __amdgpu_buffer_rsrc_t& rs, uint32_t o, float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b128(rs, (o + i) * 4, 0, 0);
#pragma unroll
    for (int n = 0; n < 4; ++n) v[i + n] = __uint_as_float(x[n]);
  }
}
// (POLICY: NT_STORE passes the line on to memory instead of keeping it in L2.  The
// tiled kernels store so, whose operands are read again and results are not:
// 16384 x 1536 from 4096 254 -> 217 us, 384 experts' weight gradients 2.55 -> 2.41 ms.)
constexpr int NT_STORE = 2;
template <int W, int POLICY>
__device__ inline void store_bf16(const __amdgpu_buffer_rsrc_t& rs, uint32_t o, const float (&v)[W]) {
  if (W == 8)
    __builtin_amdgcn_raw_buffer_store_b128(
        u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[W - 4], v[W - 3]), bf16_pair(v[W - 2], v[W - 1])}, rs, o * 2, 0, POLICY);
  else
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, rs, o * 2, 0, POLICY);
}
template <int W, int POLICY>
__device__ inline void store_f32(const __amdgpu_buffer_rsrc_t& rs, uint32_t o, const float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])},
                                           rs, (o + i) * 4, 0, POLICY);
}

// A tile's epilogue: descriptors that start with its first row and end with its
// last, so that rows past it are neither read nor stored.  Element (r, n) of
// them is at offset r N + n (of gu and dgu: (2 r + half) N + n).
template <int MODE, bool OUT_BF16, int POLICY>
struct Bf16Epilogue {
  static constexpr int CW = MODE == GDGRAD ? 2 : 1, XW = MODE == GATED ? 2 : 1, IW = MODE == GDGRAD ? 2 : 1;
  static constexpr int CB = OUT_BF16 ? 2 : 4;
  __amdgpu_buffer_rsrc_t c, aux, in, res, bias;
  uint32_t N;
  ActCoef act;
  bool has_act, has_aux, has_in, has_res, has_bias;

  __device__ Bf16Epilogue(const Bf16Args& p, int e, int64_t row0, int32_t rows) : act(p.act) {
    N = (uint32_t)p.N;
    has_act = p.act != MOE4_ACT_NONE;
    has_aux = p.aux != nullptr;
    has_in = p.in != nullptr;
    has_res = p.res != nullptr;
    has_bias = p.bias != nullptr;
    const int64_t at = row0 * p.N, n = (int64_t)rows * p.N;
    c = make_rsrc(static_cast<uint8_t*>(p.c) + at * CW * CB, (uint64_t)n * CW * CB);
    aux = make_rsrc(p.aux + at * XW, has_aux ? (uint64_t)n * XW * 2 : 0);
    in = make_rsrc(p.in + at * IW, has_in ? (uint64_t)n * IW * 2 : 0);
    res = make_rsrc(static_cast<const uint8_t*>(p.res) + at * CB, has_res ? (uint64_t)n * CB : 0);
    const int64_t nb = p.N * (MODE == GATED ? 2 : 1);
    bias = make_rsrc(p.bias + e * nb, has_bias ? (uint64_t)nb * 4 : 0);
  }
  // What the results of row r, columns n .. n + W - 1 need from memory: requested
  // for several rows before the first is used.
  template <int W>
  struct Need {
    uint32_t in[W / 2], in1[MODE == GDGRAD ? W / 2 : 1], res16[OUT_BF16 ? W / 2 : 1];
    float res[OUT_BF16 ? 1 : W];
  };
  template <int W>
  struct Bias {
    float b[W], b1[MODE == GATED ? W : 1];
  };
  template <int W>
  __device__ void request(Need<W>& x, uint32_t r, uint32_t n) const {
    const uint32_t o = n < N ? (MODE == GDGRAD ? 2 * r * N : r * N) + n : PAST;
    if (MODE == GDGRAD) {
      load_words<W>(in, o, x.in);
      load_words<W>(in, n < N ? o + N : PAST, reinterpret_cast<uint32_t(&)[W / 2]>(x.in1));
    }
    if (MODE == DGRAD && has_in) load_words<W>(in, o, x.in);
    if ((MODE == FWD || MODE == DGRAD) && has_res) {
      if (OUT_BF16) load_words<W>(res, o, reinterpret_cast<uint32_t(&)[W / 2]>(x.res16));
      else load_f32<W>(res, o, reinterpret_cast<float(&)[W]>(x.res));
    }
  }
  template <int W>
  __device__ void request(Bias<W>& x, uint32_t n) const {
    if ((MODE == FWD || MODE == GATED) && has_bias) {
      load_f32<W>(bias, n < N ? n : PAST, x.b);
      if (MODE == GATED) load_f32<W>(bias, n < N ? n + N : PAST, reinterpret_cast<float(&)[W]>(x.b1));
    }
  }
  template <bool EXACT, int W>
  __device__ void act_or_none(const float (&x)[W], float (&f)[W], float (&df)[W]) const {
    if (has_act) {
      act_of<EXACT, W>(act, x, f, df);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        f[i] = x[i];
        df[i] = 1.0f;
      }
    }
  }
  template <int W>
  __device__ void add_store(uint32_t o, float (&q)[W], const Need<W>& x) const {
    if (has_res) {
      float v[W];
      if (OUT_BF16) values_of<W>(reinterpret_cast<const uint32_t(&)[W / 2]>(x.res16), v);
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = q[i] + (OUT_BF16 ? v[i] : x.res[OUT_BF16 ? 0 : i]);
    }
    if (OUT_BF16) store_bf16<W, POLICY>(c, o, q);
    else store_f32<W, POLICY>(c, o, q);
  }
  // The W results z (GATED: z and z1) of row r of the tile, columns n .. n + W -
  // 1 (n >= N: nothing happens); s: the row's scale.
  template <int W>
  __device__ void put(uint32_t r, uint32_t n, float s, const float (&z)[W], const float (&z1)[W], const Need<W>& x, const Bias<W>& bs) const {
    const bool ok = n < N;
    const uint32_t o = ok ? r * N + n : PAST, o0 = ok ? 2 * r * N + n : PAST, o1 = ok ? o0 + N : PAST;
    float v[W], h[W], q[W], d[W];
    if (MODE == FWD) {
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = has_bias ? z[i] + bs.b[i] : z[i];
      if (has_aux) store_bf16<W, POLICY>(aux, o, q);
      act_or_none<!OUT_BF16, W>(q, h, d);
      add_store<W>(o, h, x);
    } else if (MODE == GATED) {
      float u[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        q[i] = has_bias ? z[i] + bs.b[i] : z[i];
        u[i] = has_bias ? z1[i] + bs.b1[MODE == GATED ? i : 0] : z1[i];
      }
      if (has_aux) {
        store_bf16<W, POLICY>(aux, o0, q);
        store_bf16<W, POLICY>(aux, o1, u);
      }
      act_or_none<false, W>(q, h, d);
#pragma unroll
      for (int i = 0; i < W; ++i) h[i] = h[i] * u[i];
      store_bf16<W, POLICY>(c, o, h);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = s * z[i];
      if (MODE == DGRAD) {
        if (has_in) {
          values_of<W>(x.in, v);
          act_or_none<!OUT_BF16, W>(v, h, d);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            q[i] = q[i] * d[i];
            h[i] = s * h[i];
          }
          if (has_aux) store_bf16<W, POLICY>(aux, o, h);
        }
        add_store<W>(o, q, x);
      } else {
        float u[W];
        values_of<W>(x.in, v);
        values_of<W>(reinterpret_cast<const uint32_t(&)[W / 2]>(x.in1), u);
        act_or_none<false, W>(v, h, d);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float f = h[i];
          h[i] = s * (f * u[i]);
          v[i] = q[i] * u[i] * d[i];
          u[i] = q[i] * f;
        }
        if (has_aux) store_bf16<W, POLICY>(aux, o, h);
        store_bf16<W, POLICY>(c, o0, v);
        store_bf16<W, POLICY>(c, o1, u);
      }
    }
  }
};

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
  int slices, db_slices;             // of each expert's rows (1: dw and db themselves are written)
  float *dw_part, *db_part;          // the slices' sums [E, slices, N, K] and [E, db_slices, N]
};

}  // namespace moe4
