// MXFP4 quantisation and decoding (gfx950).  MXFP4 = E2M1 elements (two to a
// byte, the even element in the low nibble) with one E8M0 scale byte per 32
// consecutive values of a row: the 4-bit format whose scales gfx950's
// block-scaled MFMA applies itself.
//
// Per block: e = the least integer with amax <= 6 * 2**e (nothing saturates;
// the rule MXFP8 follows here with 448), clamped to [-127, 127], -127 for an
// all-zero block; code = E2M1(x * 2**-e), ties to even, signs kept.  A block
// that holds an infinity or a NaN gets the scale byte 255 (E8M0's NaN) and
// zero codes, so the block decodes to NaN and every product with it is NaN.
//
// Both kernels move bytes and nothing else bounds them: a lane takes 8
// values (one 16-byte load of bf16, two of float32; one 4-byte code word), so
// a wave's loads and stores are whole cache lines, and the block's maximum
// is two DPP steps over the four lanes that share it.
#include "act.h"
#include "moe4_internal.h"

namespace moe4 {

// This file's device-side error word (moe4_debug_check reads and clears it).
static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_mxfp4() { return take_device_word(&g_dev_err); }

namespace m4q {
constexpr int THREADS = 256, VALS = 8;  // values per lane and step
}

// Scale byte of a block from the bits of its largest |x| (as an integer, so
// an infinity or NaN is the largest of all).
__device__ inline uint32_t mx4_scale_byte(uint32_t amax_bits) {
  const int ex = (int)(amax_bits >> 23);
  if (ex == 255) return 255u;
  // amax = 1.m * 2**(ex - 127) <= 6 * 2**e = 1.5 * 2**(e + 2)
  const int e = ex - 127 - ((amax_bits & 0x7FFFFFu) <= 0x400000u ? 2 : 1);
  return (uint32_t)((e < -127 ? -127 : e) + 127);
}

// The 8 values of one lane: the code word (value i in nibble i) and the scale
// byte of the block that lanes 4m .. 4m + 3 share.
__device__ inline uint32_t mx4_encode8(const float (&v)[8], uint32_t& sbyte) {
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  a = max(a, dpp_u<DPP_XOR1>(a));
  a = max(a, dpp_u<DPP_XOR2>(a));
  sbyte = mx4_scale_byte(a);
  const float p = __builtin_amdgcn_ldexpf(1.0f, 127 - (int)sbyte);
  uint32_t w = 0u;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * p, v[1] * p, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * p, v[3] * p, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * p, v[5] * p, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * p, v[7] * p, 1.0f, 3);
  return sbyte == 255u ? 0u : w;
}

// PRE: silu(x) of bf16 x.  MAP: row r goes to the output rows
// out_map[r * copies + j], j < copies (an index outside [0, out_rows) is
// reported and its copy dropped).
template <int DT, bool PRE, bool MAP>
__global__ void __launch_bounds__(m4q::THREADS) k_mx4_rows(const void* __restrict__ x, int64_t pieces, uint32_t ppr,
                                                           const int32_t* __restrict__ out_map, int copies,
                                                           int64_t out_rows, uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ sf, const float* __restrict__ act_tab) {
  using namespace m4q;
  __shared__ float tab[PRE ? ACT_TAB : 1];
  if (PRE) stage_act_table(tab, act_tab);
  const int64_t p0 = (int64_t)blockIdx.x * THREADS, p = p0 + threadIdx.x;
  if (p >= pieces) return;  // (whole blocks: pieces is a multiple of 4)
  float v[8];
  if (DT == MOE4_F32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + p * VALS);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const u32x4 q = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + p * VALS);
    if (PRE) {
      const uint32_t w[4] = {q[0], q[1], q[2], q[3]};
      act_eval_packed<false>(w, tab, v);
      // the table's domain is finite: a NaN or infinity stays one
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = (i & 1) ? q[i >> 1] >> 16 : q[i >> 1] & 0xFFFFu;
        if ((h & 0x7F80u) == 0x7F80u && h != 0xFF80u) v[i] = bf16_bits_to_f32(h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits_to_f32(q[i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(q[i] >> 16);
      }
    }
  }
  uint32_t sb;
  const uint32_t w = mx4_encode8(v, sb);
  if (!MAP) {
    codes[p] = w;
    if ((threadIdx.x & 3) == 0) sf[p >> 2] = (uint8_t)sb;
    return;
  }
  // the row and the piece in it: one 64-bit division per workgroup, a 32-bit
  // one per lane
  const int64_t r0 = p0 / ppr;
  const uint32_t rel = (uint32_t)(p0 - r0 * ppr) + threadIdx.x, dr = rel / ppr, c = rel - dr * ppr;
  const int64_t r = r0 + dr;
  for (int j = 0; j < copies; ++j) {
    const int64_t o = out_map[r * copies + j];
    if (o < 0 || o >= out_rows) {
      if (c == 0) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
      continue;
    }
    codes[o * ppr + c] = w;
    if ((threadIdx.x & 3) == 0) sf[o * (ppr >> 2) + (c >> 2)] = (uint8_t)sb;
  }
}

// Values of MXFP4 codes, 8 per lane, exact in bf16 and float32 (NaN for the
// scale byte 255; a value of 2**128 is an infinity).
template <int DT>
__global__ void __launch_bounds__(m4q::THREADS) k_mx4_dequant(const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ sf, int64_t pieces,
                                                              void* __restrict__ out) {
  const int64_t p = (int64_t)blockIdx.x * m4q::THREADS + threadIdx.x;
  if (p >= pieces) return;
  const uint32_t w = codes[p], sb = sf[p >> 2];
  float v[8];
  mx4_decode8(w, (int)sb - 127, v);
  if (sb == 255u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7FC00000u);
  }
  if (DT == MOE4_F32) {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + p * 8);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + p * 8) = o;
  }
}

}  // namespace moe4

using namespace moe4;

extern "C" int mxfp4_quant(const void* x, int dtype, int64_t rows, int64_t cols, const int32_t* out_map, int32_t copies,
                           int64_t out_rows, int pre_op, uint8_t* codes, uint8_t* sf, void* stream) {
  MOE4_REQUIRE(dtype == MOE4_BF16 || dtype == MOE4_F32, MOE4_EINVAL, "mxfp4_quant: dtype must be BF16 or F32");
  MOE4_REQUIRE(rows >= 0 && cols > 0 && cols % 32 == 0 && cols < ((int64_t)1 << 31), MOE4_EINVAL,
               "mxfp4_quant: cols must be a positive multiple of 32");
  MOE4_REQUIRE(pre_op == MOE4_PRE_NONE || (pre_op == MOE4_PRE_SILU && dtype == MOE4_BF16), MOE4_EINVAL,
               "mxfp4_quant: pre_op must be NONE, or SILU with bf16 x");
  if (out_map)
    MOE4_REQUIRE(copies >= 1 && out_rows >= 0 && rows * copies < ((int64_t)1 << 31), MOE4_EINVAL,
                 "mxfp4_quant: out_map needs copies >= 1, out_rows >= 0 and rows * copies below 2^31");
  else
    MOE4_REQUIRE(copies == 1 && out_rows == rows, MOE4_EINVAL, "mxfp4_quant: without out_map, copies = 1 and out_rows = rows");
  if (rows == 0 || out_rows == 0) return MOE4_OK;
  MOE4_REQUIRE(x && codes && sf, MOE4_EINVAL, "mxfp4_quant: NULL pointer");
  MOE4_REQUIRE(aligned16(x) && aligned16(codes), MOE4_EALIGN, "mxfp4_quant: x and codes must be 16-byte aligned");
  const int64_t pieces = rows * (cols / 8), wg = (pieces + m4q::THREADS - 1) / m4q::THREADS;
  MOE4_REQUIRE(wg < ((int64_t)1 << 31), MOE4_EINVAL, "mxfp4_quant: tensor too large");
  const float* tab = nullptr;
  if (pre_op == MOE4_PRE_SILU) {
    const int rc = act_tables(&tab);
    if (rc) return rc;
  }
#define MOE4_MX4Q(DT, PRE, MAP)                                                                                       \
  hipLaunchKernelGGL((k_mx4_rows<DT, PRE, MAP>), dim3((unsigned)wg), dim3(m4q::THREADS), 0, as_stream(stream), x,     \
                     pieces, (uint32_t)(cols / 8), out_map, copies, out_rows, reinterpret_cast<uint32_t*>(codes), sf, \
                     tab)
  if (dtype == MOE4_F32) {
    if (out_map) MOE4_MX4Q(MOE4_F32, false, true);
    else MOE4_MX4Q(MOE4_F32, false, false);
  } else if (pre_op == MOE4_PRE_SILU) {
    if (out_map) MOE4_MX4Q(MOE4_BF16, true, true);
    else MOE4_MX4Q(MOE4_BF16, true, false);
  } else {
    if (out_map) MOE4_MX4Q(MOE4_BF16, false, true);
    else MOE4_MX4Q(MOE4_BF16, false, false);
  }
#undef MOE4_MX4Q
  return check_launch("mxfp4_quant");
}

extern "C" int mxfp4_dequant(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t cols, void* out,
                             int out_dtype, void* stream) {
  MOE4_REQUIRE(out_dtype == MOE4_BF16 || out_dtype == MOE4_F32, MOE4_EINVAL, "mxfp4_dequant: out_dtype must be BF16 or F32");
  MOE4_REQUIRE(rows >= 0 && cols > 0 && cols % 32 == 0, MOE4_EINVAL, "mxfp4_dequant: cols must be a positive multiple of 32");
  if (rows == 0) return MOE4_OK;
  MOE4_REQUIRE(codes && sf && out, MOE4_EINVAL, "mxfp4_dequant: NULL pointer");
  MOE4_REQUIRE(aligned16(codes) && aligned16(out), MOE4_EALIGN, "mxfp4_dequant: codes and out must be 16-byte aligned");
  const int64_t pieces = rows * (cols / 8), wg = (pieces + m4q::THREADS - 1) / m4q::THREADS;
  MOE4_REQUIRE(wg < ((int64_t)1 << 31), MOE4_EINVAL, "mxfp4_dequant: tensor too large");
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(codes);
  if (out_dtype == MOE4_F32)
    hipLaunchKernelGGL(k_mx4_dequant<MOE4_F32>, dim3((unsigned)wg), dim3(m4q::THREADS), 0, as_stream(stream), cw, sf, pieces, out);
  else
    hipLaunchKernelGGL(k_mx4_dequant<MOE4_BF16>, dim3((unsigned)wg), dim3(m4q::THREADS), 0, as_stream(stream), cw, sf, pieces, out);
  return check_launch("mxfp4_dequant");
}
