// Weight gradients of the BF16 expert products (gfx950): per expert
// dw = dy^T a over its rows (v_mfma_f32_16x16x32_bf16, float32 accumulation),
// and the column sums of dy for the bias.
#include "bf16_gemm.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16_wgrad() { return take_device_word(&g_dev_err); }

namespace b16w {
constexpr int BN = 64, BK = 64, BR = 32, LD = BR + 8;
}

__global__ void __launch_bounds__(256) k_wgrad_bf16(Bf16Wgrad p) {
  using namespace b16w;
  __shared__ __attribute__((aligned(16))) uint16_t as[BN * LD], bs[BK * LD];
  const int e = blockIdx.z;
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4, w = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.y * BN, k0 = (int64_t)blockIdx.x * BK;
  int64_t r0 = p.off[e], r1 = p.off[e + 1];
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 < p.M ? r1 : p.M;
  if (r0 >= r1 && (p.beta != 0.0f || !p.zero_empty)) return;
  f32x4 acc[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) acc[b] = f32x4{};
  for (int64_t r = r0; r < r1; r += BR) {
    __syncthreads();
    const int64_t row = r + tid / 8;
    const int c = 8 * (tid % 8);
    u32x4 v = {}, x = {};
    if (row < r1) {
      const int64_t rd = mapped_row(p.dy_map, row, p.div, p.magic, p.dy_rows, &g_dev_err);
      const int64_t ra = mapped_row(p.a_map, row, p.div, p.magic, p.a_rows, &g_dev_err);
      if (rd >= 0 && n0 + c < p.N) v = *reinterpret_cast<const u32x4*>(p.dy + rd * p.N + n0 + c);
      if (ra >= 0 && k0 + c < p.K) x = *reinterpret_cast<const u32x4*>(p.a + ra * p.K + k0 + c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      as[(c + i) * LD + tid / 8] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
      bs[(c + i) * LD + tid / 8] = (uint16_t)(x[i / 2] >> (16 * (i & 1)));
    }
    __syncthreads();
    const bf16x8 fa = *reinterpret_cast<const bf16x8*>(as + (16 * w + li) * LD + 8 * q);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(bs + (16 * b + li) * LD + 8 * q);
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb, fa, acc[b], 0, 0, 0);
    }
  }
  const int64_t n = n0 + 16 * w + li;
  if (n >= p.N) return;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int64_t k = k0 + 16 * b + 4 * q;
    if (k >= p.K) continue;
    float* d = p.dw + ((int64_t)e * p.N + n) * p.K + k;
    f32x4 v = acc[b];
    if (p.beta != 0.0f) v = *reinterpret_cast<const f32x4*>(d) + v;
    *reinterpret_cast<f32x4*>(d) = v;
  }
}

// db: one wave per 64 columns of one expert, its rows in order.
__global__ void __launch_bounds__(64) k_bias_grad_bf16(Bf16Wgrad p) {
  const int e = blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x;
  int64_t r0 = p.off[e], r1 = p.off[e + 1];
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 < p.M ? r1 : p.M;
  if (n >= p.N || (r0 >= r1 && (p.beta != 0.0f || !p.zero_empty))) return;
  float s = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t rd = mapped_row(p.dy_map, r, p.div, p.magic, p.dy_rows, &g_dev_err);
    if (rd < 0) continue;
    const float v = bf16_bits_to_f32(p.dy[rd * p.N + n]);
    s = s + row_scale(p.db_scale, p.dy_map, r, p.dy_rows * p.div) * v;
  }
  float* d = p.db + (int64_t)e * p.N + n;
  *d = p.beta != 0.0f ? *d + s : s;
}

}  // namespace moe4

using namespace moe4;

extern "C" int moe_grouped_gemm_bf16_wgrad(const uint16_t* dy, int64_t dy_rows, const int32_t* dy_map, const uint16_t* a, int64_t a_rows,
                                           const int32_t* a_map, int32_t map_div, const int32_t* expert_off, int32_t E, int64_t M_total,
                                           int64_t N, int64_t K, float* dw, float beta, int flags, const float* db_scale, float* db,
                                           void* stream) {
  const std::string s("moe_grouped_gemm_bf16_wgrad");
  MOE4_REQUIRE(E >= 1 && E <= 2048 && M_total >= 0 && N > 0 && K > 0 && N % 8 == 0 && K % 8 == 0, MOE4_EINVAL,
               s + ": need 1 <= E <= 2048 and widths that are multiples of 8");
  MOE4_REQUIRE(M_total < ((int64_t)1 << 31) && dy_rows >= 0 && a_rows >= 0 && dy_rows < ((int64_t)1 << 31) && a_rows < ((int64_t)1 << 31) &&
                   N < ((int64_t)1 << 20) && K < ((int64_t)1 << 20) && N * K < ((int64_t)1 << 29),
               MOE4_EINVAL, s + ": rows must be below 2^31, widths below 2^20, each expert's matrix below 2 GiB");
  MOE4_REQUIRE((beta == 0.0f || beta == 1.0f) && (flags & ~MOE4_WGRAD_SKIP_EMPTY) == 0, MOE4_EINVAL, s + ": beta must be 0 or 1, flags known");
  MOE4_REQUIRE(expert_off && dw, MOE4_EINVAL, s + ": NULL pointer");
  MOE4_REQUIRE(M_total == 0 || (dy && a), MOE4_EINVAL, s + ": NULL pointer");
  MOE4_REQUIRE((!dy_map && !a_map) || map_div >= 1, MOE4_EINVAL, s + ": map_div must be positive");
  MOE4_REQUIRE(dy_map ? M_total == 0 || dy_rows >= 1 : dy_rows == M_total, MOE4_EINVAL, s + ": dy's rows do not fit");
  MOE4_REQUIRE(a_map ? M_total == 0 || a_rows >= 1 : a_rows == M_total, MOE4_EINVAL, s + ": a's rows do not fit");
  MOE4_REQUIRE((!dy_map || dy_rows * N < ((int64_t)1 << 30)) && (!a_map || a_rows * K < ((int64_t)1 << 30)), MOE4_EINVAL,
               s + ": a mapped operand must be below 2 GiB");
  MOE4_REQUIRE(db || !db_scale, MOE4_EINVAL, s + ": db_scale needs db");
  MOE4_REQUIRE(aligned16(dy) && aligned16(a) && aligned16(dw) && aligned16(db) && aligned4(db_scale) && aligned4(dy_map) && aligned4(a_map),
               MOE4_EALIGN, s + ": misaligned pointer");
  const uint32_t magic = map_div <= 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / (uint32_t)map_div);
  const Bf16Wgrad p{dy, a, dy_map, a_map, expert_off, db_scale, dw, db, dy_rows, a_rows, M_total, N, K, (uint32_t)map_div, magic, E, beta,
                    (flags & MOE4_WGRAD_SKIP_EMPTY) == 0};
  hipStream_t st = as_stream(stream);
  const int64_t nx = (K + 63) / 64, ny = (N + 63) / 64;
  hipLaunchKernelGGL(k_wgrad_bf16, dim3((unsigned)nx, (unsigned)ny, (unsigned)E), dim3(256), 0, st, p);
  if (db) hipLaunchKernelGGL(k_bias_grad_bf16, dim3((unsigned)ny, (unsigned)E), dim3(64), 0, st, p);
  return check_launch(s.c_str());
}
