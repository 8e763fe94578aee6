// Expert-grouped product of MXFP4 operands (gfx950): C[rows of e] = A[rows of
// e] . B[e]^T on the block-scaled FP4 MFMA, whose E8M0 scale per 32 values
// along K is exactly MXFP4's.  Products of two E2M1 values and their power-of-
// two scales are exact; the accumulation is float32.
#include "gemm_common.h"
#include "moe4_internal.h"

namespace moe4 {

constexpr int FP4 = 4;  // the MFMA's operand format code of E2M1

namespace m4s {
constexpr int NT = 256, TR = 16;  // rows of A per workgroup
constexpr int KB = 128;           // K per MFMA
}  // namespace m4s

// A wave takes 16 rows of B[e] (the MFMA's M side) and 16 rows of A (its N
// side); lane (li, q) holds the 32 values k = 128 s + 32 q .. of row li.
template <bool OUT_BF16>
__global__ void __launch_bounds__(m4s::NT)
    k_gemm_mx4_rows(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_sf,
                    const uint8_t* __restrict__ b_codes, const uint8_t* __restrict__ b_sf,
                    const int32_t* __restrict__ off, int E, int64_t M_total, int64_t N, int64_t K, int n_nt,
                    void* __restrict__ c) {
  using namespace m4s;
  int e;
  int64_t mt;
  if (!find_m_tile(off, E, TR, blockIdx.x / n_nt, e, mt)) return;
  const int l = threadIdx.x & 63, li = l & 15, qg = l >> 4;
  const int64_t n0 = ((int64_t)(blockIdx.x % n_nt) * (NT / 64) + (threadIdx.x >> 6)) * 16;
  if (n0 >= N) return;
  const int64_t r0 = (int64_t)off[e] + mt * TR;
  const int64_t r1 = (int64_t)off[e + 1] < M_total ? (int64_t)off[e + 1] : M_total;
  if (r0 < 0 || r0 >= r1) return;
  const int64_t ra = r0 + li < r1 ? r0 + li : r1 - 1;  // (rows past the expert are never stored)
  const int64_t KS = K / 32;
  const uint8_t* ac = a_codes + ra * (K / 2);
  const uint8_t* as = a_sf + ra * KS;
  const uint8_t* bc = b_codes + ((int64_t)e * N + n0 + li) * (K / 2);
  const uint8_t* bs = b_sf + ((int64_t)e * N + n0 + li) * KS;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t s = 0; s * KB < K; ++s) {
    const int64_t kb = 4 * s + qg;  // this lane's block
    u32x4 wa = {0u, 0u, 0u, 0u}, wb = wa;
    int ya = 0, yb = 0;
    if (kb < KS) {
      wa = *reinterpret_cast<const u32x4*>(ac + 16 * kb);
      wb = *reinterpret_cast<const u32x4*>(bc + 16 * kb);
      ya = as[kb];
      yb = bs[kb];
    }
    const i32x8 fb = {(int)wb[0], (int)wb[1], (int)wb[2], (int)wb[3], 0, 0, 0, 0};
    const i32x8 fa = {(int)wa[0], (int)wa[1], (int)wa[2], (int)wa[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, FP4, FP4, 0, yb, 0, ya);
  }
  const int64_t row = r0 + li, col = n0 + 4 * qg;
  if (row >= r1) return;
  if (OUT_BF16)
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(c) + row * N + col) =
        u32x2{f32_to_bf16_bits(acc[0]) | (f32_to_bf16_bits(acc[1]) << 16),
              f32_to_bf16_bits(acc[2]) | (f32_to_bf16_bits(acc[3]) << 16)};
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(c) + row * N + col) = acc;
}

}  // namespace moe4

using namespace moe4;

extern "C" int moe_grouped_gemm_mx4(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* b_codes,
                                    const uint8_t* b_sf, const int32_t* expert_off, int32_t E, int64_t M_total, int64_t N,
                                    int64_t K, void* c, int c_dtype, void* stream) {
  MOE4_REQUIRE(c_dtype == MOE4_F32 || c_dtype == MOE4_BF16, MOE4_EINVAL, "moe_grouped_gemm_mx4: c_dtype must be F32 or BF16");
  MOE4_REQUIRE(E >= 1 && M_total >= 0 && N > 0 && K > 0 && K % 32 == 0 && N % 32 == 0, MOE4_EINVAL,
               "moe_grouped_gemm_mx4: need K % 32 == 0 and N % 32 == 0");
  MOE4_REQUIRE(M_total < ((int64_t)1 << 31) && N * K < ((int64_t)1 << 32), MOE4_EINVAL,
               "moe_grouped_gemm_mx4: M must be below 2^31 and each expert's B below 2 GiB");
  MOE4_REQUIRE(expert_off && (M_total == 0 || (a_codes && a_sf && b_codes && b_sf && c)), MOE4_EINVAL,
               "moe_grouped_gemm_mx4: NULL pointer");
  MOE4_REQUIRE(aligned16(a_codes) && aligned16(b_codes) && aligned16(c), MOE4_EALIGN,
               "moe_grouped_gemm_mx4: a_codes, b_codes and c must be 16-byte aligned");
  if (M_total == 0) return MOE4_OK;
  const int64_t m_tiles = (M_total + m4s::TR - 1) / m4s::TR + E;
  const int n_nt = (int)((N + 63) / 64);
  MOE4_REQUIRE(m_tiles * n_nt < ((int64_t)1 << 31), MOE4_EINVAL, "moe_grouped_gemm_mx4: too large");
  const dim3 grid((unsigned)(m_tiles * n_nt));
  if (c_dtype == MOE4_BF16)
    hipLaunchKernelGGL(k_gemm_mx4_rows<true>, grid, dim3(m4s::NT), 0, as_stream(stream), a_codes, a_sf, b_codes, b_sf,
                       expert_off, E, M_total, N, K, n_nt, c);
  else
    hipLaunchKernelGGL(k_gemm_mx4_rows<false>, grid, dim3(m4s::NT), 0, as_stream(stream), a_codes, a_sf, b_codes, b_sf,
                       expert_off, E, M_total, N, K, n_nt, c);
  return check_launch("moe_grouped_gemm_mx4");
}
