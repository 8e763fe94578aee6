// Expert-grouped BF16 products with their epilogues (gfx950): forward with
// bias, activation and residual, the gated block, and their input gradients.
// v_mfma_f32_16x16x32_bf16, float32 accumulation, each result rounded once.
#include "bf16_gemm.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16() { return take_device_word(&g_dev_err); }

namespace b16 {
constexpr int BM = 64, BN = 64, BK = 32, LD = BK + 8;  // (80-byte LDS rows)
}

// 64 x 64 tiles (GATED: 64 x 32, both halves of a column in one wave), four
// waves of 16 rows.  The weights take the MFMA's M side, so that a lane holds
// four consecutive columns of one row.
template <int MODE, bool OUT_BF16>
__global__ void __launch_bounds__(256) k_gemm_bf16(Bf16Args p) {
  using namespace b16;
  constexpr int NW = MODE == GATED ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) uint16_t as[BM * LD], bs[BN * LD];
  int e;
  int64_t mt;
  if (!find_m_tile(p.off, p.E, BM, blockIdx.y, e, mt)) return;
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4, w = tid >> 6;
  const int64_t r0 = (int64_t)p.off[e] + mt * BM, n0 = (int64_t)blockIdx.x * NW;
  const int64_t re = (int64_t)p.off[e + 1] < p.M ? (int64_t)p.off[e + 1] : p.M;
  if (r0 < 0) return;
  const int64_t ar = r0 + tid / 4;
  const int64_t arow = ar < re ? mapped_row(p.map, ar, p.div, p.magic, p.a_rows, &g_dev_err) : -1;
  f32x4 acc[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) acc[b] = f32x4{};
  for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
    __syncthreads();
    const int64_t k = k0 + 8 * (tid % 4);
    u32x4 v = {};
    if (arow >= 0 && k < p.K) v = *reinterpret_cast<const u32x4*>(p.a + arow * p.K + k);
    *reinterpret_cast<u32x4*>(as + (tid / 4) * LD + 8 * (tid % 4)) = v;
    u32x4 x = {};
    if (MODE == FWD || MODE == GATED) {
      const int r = tid / 4;
      const int64_t n = n0 + (MODE == GATED ? r % NW : r);
      const int64_t row = MODE == GATED ? ((int64_t)e * 2 + r / NW) * p.N + n : (int64_t)e * p.N + n;
      if (n < p.N && k < p.K) x = *reinterpret_cast<const u32x4*>(p.w + row * p.K + k);
      *reinterpret_cast<u32x4*>(bs + r * LD + 8 * (tid % 4)) = x;
    } else {
      const int64_t kk = k0 + tid / 8, n = n0 + 8 * (tid % 8);
      if (n < p.N && kk < p.K) x = *reinterpret_cast<const u32x4*>(p.w + ((int64_t)e * p.K + kk) * p.N + n);
#pragma unroll
      for (int i = 0; i < 8; ++i) bs[(8 * (tid % 8) + i) * LD + tid / 8] = (uint16_t)(x[i / 2] >> (16 * (i & 1)));
    }
    __syncthreads();
    const bf16x8 fa = *reinterpret_cast<const bf16x8*>(as + (16 * w + li) * LD + 8 * q);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(bs + (16 * b + li) * LD + 8 * q);
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb, fa, acc[b], 0, 0, 0);
    }
  }
  const int64_t r = r0 + 16 * w + li;
  if (r >= re) return;
#pragma unroll
  for (int b = 0; b < NW / 16; ++b) {
    const int64_t n = n0 + 16 * b + 4 * q;
    if (n >= p.N) continue;
    const f32x4 z0 = acc[b], z1 = acc[MODE == GATED ? b + 2 : b];
    const float z[4] = {z0[0], z0[1], z0[2], z0[3]}, y[4] = {z1[0], z1[1], z1[2], z1[3]};
    bf16_epilogue<MODE, OUT_BF16, 4>(p, e, r, n, z, y);
  }
}

template <int MODE, bool OUT_BF16>
static int launch_bf16(const Bf16Args& p, void* stream, const char* name) {
  constexpr int NW = MODE == GATED ? b16::BN / 2 : b16::BN;
  const int64_t nt = (p.N + NW - 1) / NW, mt = p.M / b16::BM + p.E;
  MOE4_REQUIRE(mt < 65536 && grid_fits(nt, 256), MOE4_EINVAL, std::string(name) + ": too large");
  hipLaunchKernelGGL((k_gemm_bf16<MODE, OUT_BF16>), dim3((unsigned)nt, (unsigned)mt), dim3(256), 0, as_stream(stream), p);
  return check_launch(name);
}

// What the four calls check alike.  rows of a: M without a map.
static int check_bf16(const Bf16Args& p, const char* name) {
  const std::string s(name);
  MOE4_REQUIRE(p.E >= 1 && p.E <= 4096 && p.M >= 0 && p.N > 0 && p.K > 0 && p.N % 8 == 0 && p.K % 8 == 0, MOE4_EINVAL,
               s + ": need 1 <= E <= 4096 and widths that are multiples of 8");
  MOE4_REQUIRE(p.M < ((int64_t)1 << 31) && p.a_rows >= 0 && p.a_rows < ((int64_t)1 << 31) && p.N < ((int64_t)1 << 20) &&
                   p.K < ((int64_t)1 << 20) && p.N * p.K < ((int64_t)1 << 29),
               MOE4_EINVAL, s + ": rows must be below 2^31, widths below 2^20, each expert's matrix below 1 GiB");
  MOE4_REQUIRE(p.act >= MOE4_ACT_NONE && p.act <= MOE4_ACT_GELU, MOE4_EINVAL, s + ": bad activation");
  MOE4_REQUIRE(p.off, MOE4_EINVAL, s + ": NULL pointer");
  if (p.map) {
    MOE4_REQUIRE(p.div >= 1 && p.div < (1u << 31), MOE4_EINVAL, s + ": map_div must be positive");
    MOE4_REQUIRE(p.M == 0 || p.a_rows >= 1, MOE4_EINVAL, s + ": a map needs rows to point at");
    MOE4_REQUIRE(p.a_rows * p.K < ((int64_t)1 << 30), MOE4_EINVAL, s + ": a mapped operand must be below 2 GiB");
  } else {
    MOE4_REQUIRE(p.a_rows == p.M, MOE4_EINVAL, s + ": without a map the operand has M_total rows");
  }
  MOE4_REQUIRE(p.M == 0 || (p.a && p.w && p.c), MOE4_EINVAL, s + ": NULL pointer");
  MOE4_REQUIRE(aligned16(p.a) && aligned16(p.w) && aligned16(p.c) && aligned16(p.in) && aligned16(p.res) && aligned16(p.aux) && aligned16(p.bias) &&
                   aligned4(p.scale) && aligned4(p.map),
               MOE4_EALIGN, s + ": misaligned pointer");
  return MOE4_OK;
}
static uint32_t div_magic(int32_t div) { return div <= 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / (uint32_t)div); }

}  // namespace moe4

using namespace moe4;

extern "C" int moe_grouped_gemm_bf16(const uint16_t* a, int64_t a_rows, const int32_t* row_map, int32_t map_div, const uint16_t* w,
                                     const float* bias, const int32_t* expert_off, int32_t E, int64_t M_total, int64_t N, int64_t K,
                                     int act, const void* residual, void* c, int c_dtype, uint16_t* pre, void* stream) {
  const char* name = "moe_grouped_gemm_bf16";
  const Bf16Args p{a, row_map, w, expert_off, bias, nullptr, nullptr, residual, c, pre, a_rows, M_total, N, K, (uint32_t)map_div, div_magic(map_div), E, act};
  MOE4_REQUIRE(c_dtype == MOE4_F32 || c_dtype == MOE4_BF16, MOE4_EINVAL, "moe_grouped_gemm_bf16: c_dtype must be F32 or BF16");
  if (const int rc = check_bf16(p, name)) return rc;
  if (M_total == 0) return MOE4_OK;
  return c_dtype == MOE4_BF16 ? launch_bf16<FWD, true>(p, stream, name) : launch_bf16<FWD, false>(p, stream, name);
}

extern "C" int moe_gated_gemm_bf16(const uint16_t* a, int64_t a_rows, const int32_t* row_map, int32_t map_div, const uint16_t* w,
                                   const float* bias, const int32_t* expert_off, int32_t E, int64_t M_total, int64_t F, int64_t K,
                                   int act, uint16_t* h, uint16_t* gu, void* stream) {
  const char* name = "moe_gated_gemm_bf16";
  const Bf16Args p{a, row_map, w, expert_off, bias, nullptr, nullptr, nullptr, h, gu, a_rows, M_total, F, K, (uint32_t)map_div, div_magic(map_div), E, act};
  if (const int rc = check_bf16(p, name)) return rc;
  if (M_total == 0) return MOE4_OK;
  return launch_bf16<GATED, true>(p, stream, name);
}

extern "C" int moe_grouped_gemm_bf16_dgrad(const uint16_t* dy, int64_t dy_rows, const int32_t* row_map, int32_t map_div,
                                           const float* row_scale, const uint16_t* w, const int32_t* expert_off, int32_t E,
                                           int64_t M_total, int64_t N, int64_t K, int act, const uint16_t* pre, const void* add,
                                           void* dx, int dx_dtype, uint16_t* hs, void* stream) {
  const char* name = "moe_grouped_gemm_bf16_dgrad";
  const Bf16Args p{dy, row_map, w, expert_off, nullptr, row_scale, pre, add, dx, hs, dy_rows, M_total, K, N, (uint32_t)map_div, div_magic(map_div), E, act};
  MOE4_REQUIRE(dx_dtype == MOE4_F32 || dx_dtype == MOE4_BF16, MOE4_EINVAL, "moe_grouped_gemm_bf16_dgrad: dx_dtype must be F32 or BF16");
  MOE4_REQUIRE(pre || (act == MOE4_ACT_NONE && !hs), MOE4_EINVAL, "moe_grouped_gemm_bf16_dgrad: an activation or hs needs pre");
  if (const int rc = check_bf16(p, name)) return rc;
  if (M_total == 0) return MOE4_OK;
  return dx_dtype == MOE4_BF16 ? launch_bf16<DGRAD, true>(p, stream, name) : launch_bf16<DGRAD, false>(p, stream, name);
}

extern "C" int moe_gated_gemm_bf16_dgrad(const uint16_t* dy, int64_t dy_rows, const int32_t* row_map, int32_t map_div,
                                         const float* row_scale, const uint16_t* w, const int32_t* expert_off, int32_t E,
                                         int64_t M_total, int64_t N, int64_t F, int act, const uint16_t* gu, uint16_t* dgu, uint16_t* hs,
                                         void* stream) {
  const char* name = "moe_gated_gemm_bf16_dgrad";
  const Bf16Args p{dy, row_map, w, expert_off, nullptr, row_scale, gu, nullptr, dgu, hs, dy_rows, M_total, F, N, (uint32_t)map_div, div_magic(map_div), E, act};
  if (const int rc = check_bf16(p, name)) return rc;
  MOE4_REQUIRE(M_total == 0 || gu, MOE4_EINVAL, "moe_gated_gemm_bf16_dgrad: NULL pointer");
  if (M_total == 0) return MOE4_OK;
  return launch_bf16<GDGRAD, true>(p, stream, name);
}
