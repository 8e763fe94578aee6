// The layer's tail with dropout (gfx950): gate-weighted combine, dropout and
// residual in one pass, and the gradient of the dropout.
//
// Element i = t d + c of [T, d] is kept iff its 16 random bits (the library's
// counter hash of (seed, stream, i), one 32-bit word for two elements) are below
// q = round((1 - p) 65536), and then scaled by 65536 / q; so the expectation is
// exact for any p, and the mask is recomputed where it is needed.
#include <math.h>

#include "moe4_internal.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_dropout() { return take_device_word(&g_dev_err); }

struct Dropout {
  uint32_t base, q;  // sr_base_key(seed, stream), threshold
  float scale;       // 65536 / q (0 for q = 0)
};

// Whether elements i .. i + 3 (i % 4 == 0) are kept: two words of the hash.
__device__ inline void keep4(const Dropout& dr, uint64_t i, bool (&k)[4]) {
  const uint64_t j = i >> 1;
  const uint32_t key = fmix32(dr.base ^ (uint32_t)(j >> 32));
  const uint32_t w0 = fmix32((uint32_t)j ^ key), w1 = fmix32((uint32_t)(j + 1) ^ key);
  k[0] = (w0 & 0xFFFFu) < dr.q;
  k[1] = (w0 >> 16) < dr.q;
  k[2] = (w1 & 0xFFFFu) < dr.q;
  k[3] = (w1 >> 16) < dr.q;
}

// Four columns a thread: 16 bytes of each of the k rows.  Bound: the bytes; 16384
// tokens of 8 rows of 4096, with a residual 2.42 GB in 500 us, 4.85 TB/s (a copy: 5.1).
__global__ void __launch_bounds__(256) k_combine_dropout(const float* __restrict__ yp, const float* __restrict__ gates,
                                                         const int32_t* __restrict__ inv, int64_t T, int k, int64_t d,
                                                         Dropout dr, const uint16_t* residual, uint16_t* y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= T * d) return;
  const int64_t t = i / d, c = i - t * d;
  f32x4 acc = {};
  for (int j = 0; j < k; ++j) {
    int64_t row = inv[t * k + j];
    if (row < 0 || row >= T * k) {
      atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
      row = row < 0 ? 0 : T * k - 1;
    }
    const float g = gates[t * k + j];
    const f32x4 v = *reinterpret_cast<const f32x4*>(yp + row * d + c);
    for (int n = 0; n < 4; ++n) acc[n] = acc[n] + g * v[n];
  }
  bool keep[4];
  keep4(dr, (uint64_t)i, keep);
  u32x2 r = {};
  if (residual) r = *reinterpret_cast<const u32x2*>(residual + i);
  float o[4];
  for (int n = 0; n < 4; ++n) {
    o[n] = keep[n] ? acc[n] * dr.scale : 0.0f;
    if (residual) o[n] = bf16_bits_to_f32((n & 1) ? r[n >> 1] >> 16 : r[n >> 1] & 0xFFFFu) + o[n];
  }
  *reinterpret_cast<u32x2*>(y + i) = u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
}

// Bound: the bytes; 16384 x 4096, 268 MB in 51 us, 5.2 TB/s.
__global__ void __launch_bounds__(256) k_dropout_bwd(const uint16_t* dy, int64_t n, Dropout dr, uint16_t* dx) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  bool keep[4];
  keep4(dr, (uint64_t)i, keep);
  const u32x2 r = *reinterpret_cast<const u32x2*>(dy + i);
  float o[4];
  for (int m = 0; m < 4; ++m) o[m] = keep[m] ? bf16_bits_to_f32((m & 1) ? r[m >> 1] >> 16 : r[m >> 1] & 0xFFFFu) * dr.scale : 0.0f;
  *reinterpret_cast<u32x2*>(dx + i) = u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
}

static Dropout make_dropout(double p, uint64_t seed, uint32_t stream_id) {
  const uint32_t q = (uint32_t)nearbyint((1.0 - p) * 65536.0);
  return Dropout{sr_base_key(seed, stream_id), q, q ? 65536.0f / (float)q : 0.0f};
}

}  // namespace moe4

using namespace moe4;

extern "C" int moe_combine_dropout(const float* yp, const float* gates, const int32_t* inv_perm, int64_t T, int32_t k, int64_t d, double p,
                                   uint64_t seed, uint32_t stream_id, const uint16_t* residual, uint16_t* y, void* stream) {
  MOE4_REQUIRE(T >= 0 && k >= 1 && k <= 16 && d > 0 && d % 4 == 0, MOE4_EINVAL, "moe_combine_dropout: bad sizes (1 <= k <= 16, d % 4 == 0)");
  MOE4_REQUIRE(p >= 0.0 && p <= 1.0, MOE4_EINVAL, "moe_combine_dropout: p must be in [0, 1]");
  MOE4_REQUIRE(T < ((int64_t)1 << 31) && d < ((int64_t)1 << 31) && T * k < ((int64_t)1 << 31) && grid_fits((T * d + 1023) / 1024, 256),
               MOE4_EINVAL, "moe_combine_dropout: too large");
  MOE4_REQUIRE(T == 0 || (yp && gates && inv_perm && y), MOE4_EINVAL, "moe_combine_dropout: NULL pointer");
  MOE4_REQUIRE(aligned16(yp) && aligned16(y) && aligned16(residual), MOE4_EALIGN, "moe_combine_dropout: misaligned pointer");
  if (T == 0) return MOE4_OK;
  hipLaunchKernelGGL(k_combine_dropout, dim3((unsigned)((T * d + 1023) / 1024)), dim3(256), 0, as_stream(stream), yp, gates, inv_perm, T, k,
                     d, make_dropout(p, seed, stream_id), residual, y);
  return check_launch("moe_combine_dropout");
}

extern "C" int moe_dropout_backward(const uint16_t* dy, int64_t T, int64_t d, double p, uint64_t seed, uint32_t stream_id, uint16_t* dx,
                                    void* stream) {
  MOE4_REQUIRE(T >= 0 && d > 0 && d % 4 == 0, MOE4_EINVAL, "moe_dropout_backward: bad sizes (d % 4 == 0)");
  MOE4_REQUIRE(p >= 0.0 && p <= 1.0, MOE4_EINVAL, "moe_dropout_backward: p must be in [0, 1]");
  MOE4_REQUIRE(T < ((int64_t)1 << 31) && d < ((int64_t)1 << 31) && grid_fits((T * d + 1023) / 1024, 256), MOE4_EINVAL,
               "moe_dropout_backward: too large");
  MOE4_REQUIRE(T == 0 || (dy && dx), MOE4_EINVAL, "moe_dropout_backward: NULL pointer");
  MOE4_REQUIRE(aligned16(dy) && aligned16(dx), MOE4_EALIGN, "moe_dropout_backward: misaligned pointer");
  if (T == 0) return MOE4_OK;
  hipLaunchKernelGGL(k_dropout_bwd, dim3((unsigned)((T * d + 1023) / 1024)), dim3(256), 0, as_stream(stream), dy, T * d,
                     make_dropout(p, seed, stream_id), dx);
  return check_launch("moe_dropout_backward");
}
