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
// Both kernels move bytes and nothing else bounds them.  The quantiser's lane
// loads pieces of 8 values (16 bytes of bf16, 32 of float32: whole lines
// across the wave), a block's maximum is two DPP steps over the four lanes that
// share it, and four pieces a lane are then transposed within those four lanes,
// so that each holds one block: 16 code bytes and a scale byte to store, a
// quarter of the store instructions (which is what the dispatch, storing
// every block `copies` times, spends its time on).  16384 x 4096 bf16 to eight
// rows each (0.44 GB): 73 us, 6.0 TB/s; 73728 x 4096 float32 (1.37 GB): 238 us,
// 5.7 TB/s; 131072 x 4096 decoded to bf16 (1.38 GB, mostly written): 252 us.
// With SiLU the VALU takes over (busy 82 %): 131072 x 1536 bf16 (0.51 GB): 111 us.
#include "act.h"
#include "moe4_internal.h"
#include "mx_requant.h"

namespace moe4 {

// This file's device-side error word (moe4_debug_check reads and clears it).
static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_mxfp4() { return take_device_word(&g_dev_err); }

namespace m4q {
constexpr int THREADS = 256, THREADS_SILU = 512;
constexpr int UNIT = 256;  // pieces of 8 values per wave and step
constexpr int MAPS = 8;    // output rows looked up at a time
constexpr int SILU_WG = 768;  // workgroups of the SiLU form (three per CU by their registers; 24 KB of table each)
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

// 16 bytes of piece p (float32: half h).  bf16 is loaded nontemporally: nothing
// reads it again and a dispatch's stores keep the caches (91 -> 72 us at 16384 x
// 4096, eight copies).  A float32 piece's two halves share their lines, so it is
// not (248 -> 265 us); there the stores are (248 -> 231 us at 73728 x 4096).
template <int DT>
__device__ inline u32x4 load_piece(const void* x, int64_t p, int h) {
  const u32x4* q = static_cast<const u32x4*>(x);
  if (DT == MOE4_F32) return q[2 * p + h];
  return __builtin_nontemporal_load(q + p);
}

// One wave: units of 256 pieces (64 blocks); piece 64 u + l of a unit is lane
// l's u-th, and block 16 j + m of it ends up in lane 4 m + j.  PRE: silu(x) of
// bf16 x (a grid of a few workgroups per CU walks the units, so that the table
// is staged once for many of them).  MAP: row r goes to the output rows
// out_map[r * copies + j], j < copies (an index outside [0, out_rows) is
// reported and its copy dropped).
template <int DT, bool PRE, bool MAP>
__global__ void __launch_bounds__(PRE ? m4q::THREADS_SILU : m4q::THREADS)
    k_mx4_rows(const void* __restrict__ x, int64_t pieces, int64_t units,
                                                           uint32_t bpr, const int32_t* __restrict__ out_map, int copies,
                                                           int64_t out_rows, u32x4* __restrict__ codes,
                                                           uint8_t* __restrict__ sf, const float* __restrict__ act_tab) {
  using namespace m4q;
  constexpr int WAVES = (PRE ? THREADS_SILU : THREADS) / 64;
  __shared__ float tab[PRE ? ACT_TAB : 1];
  if (PRE) stage_act_table(tab, act_tab);
  const int l = threadIdx.x & 63, j = l & 3;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t unit = (int64_t)blockIdx.x * WAVES + w; unit < units; unit += (int64_t)gridDim.x * WAVES) {
    u32x4 raw[4][DT == MOE4_F32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t p = unit * UNIT + 64 * u + l;
#pragma unroll
      for (int h = 0; h < (DT == MOE4_F32 ? 2 : 1); ++h)
        raw[u][h] = p < pieces ? load_piece<DT>(x, p, h) : u32x4{0u, 0u, 0u, 0u};
    }
    uint32_t cw[4], sb[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[8];
      if (DT == MOE4_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(raw[u][DT == MOE4_F32 ? i >> 2 : 0][i & 3]);
      } else if (PRE) {
        const uint32_t q[4] = {raw[u][0][0], raw[u][0][1], raw[u][0][2], raw[u][0][3]};
        act_eval_packed<false>(q, tab, v);
        // the table's domain is finite: a NaN and +infinity stay what they are
        uint32_t odd = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= ((q[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        if (__any(odd != 0u)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t h = (i & 1) ? q[i >> 1] >> 16 : q[i >> 1] & 0xFFFFu;
            if ((h & 0x7F80u) == 0x7F80u && h != 0xFF80u) v[i] = bf16_bits_to_f32(h);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16_bits_to_f32(raw[u][0][i] & 0xFFFFu);
          v[2 * i + 1] = bf16_bits_to_f32(raw[u][0][i] >> 16);
        }
      }
      cw[u] = mx4_encode8(v, sb[u]);
    }
    // transpose cw over the four lanes and the four pieces
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      const uint32_t y = dpp_u<DPP_XOR1>((j & 1) ? cw[u] : cw[u + 1]);
      if (j & 1) cw[u] = y;
      else cw[u + 1] = y;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t y = dpp_u<DPP_XOR2>((j & 2) ? cw[u] : cw[u + 2]);
      if (j & 2) cw[u] = y;
      else cw[u + 2] = y;
    }
    const u32x4 code = {cw[0], cw[1], cw[2], cw[3]};
    const uint8_t scale = (uint8_t)(j == 0 ? sb[0] : j == 1 ? sb[1] : j == 2 ? sb[2] : sb[3]);
    const int64_t b0 = unit * (UNIT / 4);
    const uint32_t db = 16u * j + (l >> 2);
    if (b0 + db >= pieces / 4) continue;
    if (!MAP) {
      if (DT == MOE4_F32) __builtin_nontemporal_store(code, codes + b0 + db);
      else codes[b0 + db] = code;
      sf[b0 + db] = scale;
      continue;
    }
    // the row and the block in it: one 64-bit division per unit, a 32-bit one
    // per lane
    const int64_t r0 = b0 / bpr;
    const uint32_t rel = (uint32_t)(b0 - r0 * bpr) + db, dr = rel / bpr, c = rel - dr * bpr;
    const int32_t* to = out_map + (r0 + dr) * copies;
    for (int i = 0; i < copies; i += MAPS) {
      int64_t o[MAPS];
#pragma unroll
      for (int k = 0; k < MAPS; ++k) o[k] = i + k < copies ? to[i + k] : -1;
#pragma unroll
      for (int k = 0; k < MAPS; ++k) {
        if (i + k >= copies) break;
        if (o[k] < 0 || o[k] >= out_rows) {
          if (c == 0) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
          continue;
        }
        codes[o[k] * bpr + c] = code;
        sf[o[k] * bpr + c] = scale;
      }
    }
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
    // (nontemporal: whole lines, larger than what was read: 145 -> 104 us at 73728 x 4096 with the codes in cache)
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + p * 8));
  }
}

// ------------------------------------------------- transposed requantisation
// MXFP4 [R, C] -> exact values -> transpose -> MXFP8 with stochastic rounding,
// group-major (tiles, LDS staging and random words as the other sources'
// kernel: 128 padded rows x 512 columns per workgroup, a wave per 32-row MX
// block, lane l the columns c0 + 8 l ..).
//
// The arithmetic per value is the random word's share (3 instructions) and what
// the format needs.  The power of two of a source block goes into the FP4
// decoder's scale operand and that of a result block into the stochastic
// converter's, so a value costs half a decode and one conversion in each of
// the two passes (maxima, then codes).  That holds while every scale byte met
// is in [20, 251] (values and results then normal floats); a block outside
// takes its powers of two by ldexp.  A source scale byte of 255 gives each
// column block that meets it the scale byte 255.
//
// A wave's 32 x 16 scale bytes come as eight loads of 64 bytes and are turned
// through LDS into each lane's 32 (32 byte loads a lane before: 150 -> 124 us at
// 131072 x 1536).
//
// The codes leave in two halves of the lane's columns, so that a wave needs 8 KB
// of LDS and three waves fit a SIMD (two with all columns at once: 125 -> 115 us
// at 131072 x 1536, 280 -> 252 at 131072 x 4096); each half hashes its rows' keys
// again.  Its 13 VALU instructions a value keep the VALU busy for 67 % of the
// cycles (112 us under the profiler); the 1.56 bytes a value would take 62.
namespace rq4 {
// any byte of w zero
__device__ inline uint32_t zero_byte(uint32_t w) { return (w - 0x01010101u) & ~w & 0x80808080u; }
// any byte below 20 or above 251
__device__ inline bool odd_scales(uint32_t w) {
  const uint32_t big = zero_byte(~(w | 0x03030303u));                 // 252 .. 255
  // below 20: bit 7 clear, and clear after adding 108 to the other seven
  const uint32_t small = ~((w & 0x7F7F7F7Fu) + 0x6C6C6C6Cu) & ~w & 0x80808080u;  // below 20
  return (big | small) != 0u;
}
}  // namespace rq4

__global__ void __launch_bounds__(rq::THREADS, 3) k_requant_mx4_T(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ sf, int64_t C,
                                                               const int32_t* __restrict__ off,
                                                               const int32_t* __restrict__ offp, int G, int64_t R,
                                                               int64_t max_pr, int64_t n_ct, uint32_t base, int sfb,
                                                               uint8_t* __restrict__ out_c, uint8_t* __restrict__ out_s) {
  using namespace rq;
  __shared__ __attribute__((aligned(16))) uint8_t lq[COLS / 2 * ROWS];  // half of each lane's columns
  __shared__ __attribute__((aligned(16))) uint8_t lsc[WAVES][16][32];  // [wave][source block][row]
  __shared__ uint8_t lsf[COLS * WAVES];  // [column][block]
  __shared__ int64_t lblk[WAVES][3];     // block's code offset at column 0, P (0: no block), scale offset at column 0
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int64_t c0 = (int64_t)(blockIdx.x % n_ct) * COLS;
  const int64_t pr = ((int64_t)(blockIdx.x / n_ct) * WAVES + w) * 32;
  const int64_t ptot = offp[G];
  int64_t P = 0, pr_in_g = 0, src0 = 0, obase = 0, sbase = 0;
  int nvalid = 0, g = 0;
  // the block's group; offsets that would lead out of the outputs are reported
  // and their blocks left alone
  bool present = pr < ptot, bad = ptot > max_pr;
  if (present) {
    g = find_group(offp, G, pr);
    const int64_t o0 = offp[g], o1 = offp[g + 1];
    bad = bad || o0 < 0 || o0 > pr || o1 <= pr || o1 > max_pr || ((o0 | o1) & 31) != 0;
  }
  if (bad && l == 0) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
  present = present && !bad;
  if (present) {
    pr_in_g = pr - offp[g];
    P = (int64_t)offp[g + 1] - offp[g];
    src0 = (int64_t)off[g] + pr_in_g;
    const int64_t gend = (int64_t)off[g + 1] < R ? (int64_t)off[g + 1] : R;
    const int64_t n = gend - src0;
    nvalid = n < 0 || src0 < 0 ? 0 : (n > 32 ? 32 : (int)n);
    obase = C * (int64_t)offp[g] + pr_in_g;
    sbase = C * (int64_t)offp[g] / 32 + (sfb ? (pr_in_g / 32) * C : pr_in_g / 32);
  }
  if (l == 0) {
    lblk[w][0] = obase;
    lblk[w][1] = P;
    lblk[w][2] = sbase;
  }
  const int64_t c = c0 + LCOLS * l;
  // code words (8 columns) of the 32 rows; rows past the group are zeros
  uint32_t cw[32];
  const uint8_t* crow = codes + src0 * (C / 2) + c / 2;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    cw[i] = i < nvalid && c < C ? *reinterpret_cast<const uint32_t*>(crow + (int64_t)i * (C / 2)) : 0u;
  // scale bytes: load i takes rows 4 i .. 4 i + 3 of the wave's 16 source blocks
  {
    const int64_t nb = C / 32, b = c0 / 32 + (l & 15);
    uint32_t s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (l >> 4);
      s[i] = r < nvalid && b < nb ? (uint32_t)sf[(src0 + r) * nb + b] : 127u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) lsc[w][l & 15][4 * i + (l >> 4)] = (uint8_t)s[i];
  }
  __syncthreads();
  // row group k (rows 4k..4k+3 of block w) of the lane's column 4 h + q: dword
  // k % 4 of 16-byte chunk 2w + k / 4 of LDS run 4 l + q
  auto put = [&](int k, int q, uint32_t v) {
    const int col = LCOLS / 2 * l + q;
    *reinterpret_cast<uint32_t*>(lq + col * ROWS + swz(col, 2 * w + (k >> 2)) * 16 + (k & 3) * 4) = v;
  };
  int ex[8];
  bool nan = false;
  uint32_t sbp[8];  // the lane's scale bytes, four rows a register
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(&lsc[w][l >> 2][16 * k]);
    sbp[4 * k] = v[0]; sbp[4 * k + 1] = v[1]; sbp[4 * k + 2] = v[2]; sbp[4 * k + 3] = v[3];
  }
  bool odd = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) odd |= rq4::odd_scales(sbp[k]);
  const int64_t j0 = src0 * (C / 2) + c / 2;  // pair index of (row src0, column c)
  const uint32_t key0 = fmix32(base);
  const bool fast = src0 * (C / 2) + 32 * (C / 2) < ((int64_t)1 << 32);
  const bool plain = fast && !__any(odd);  // (uniform over the wave)
  auto scale = [&](int i) { return __uint_as_float(((sbp[i >> 2] >> (8 * (i & 3))) & 0xFFu) << 23); };  // 2**(byte - 127)
  auto byte = [&](int i) { return (int)((sbp[i >> 2] >> (8 * (i & 3))) & 0xFFu); };
  float sc[8];  // the result blocks' scales (any for an all-zero one)
  {
    float am[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) am[q] = 0.0f;
    if (plain) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float s = scale(i);
        const f32x2 d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], s, 0), d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], s, 1);
        const f32x2 d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], s, 2), d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], s, 3);
        const float v[8] = {d0[0], d0[1], d1[0], d1[1], d2[0], d2[1], d3[0], d3[1]};
#pragma unroll
        for (int q = 0; q < 8; ++q) am[q] = fmaxf(am[q], fabsf(v[q]));
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) ex[q] = mx_exponent(am[q]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) nan |= rq4::zero_byte(~sbp[k]) != 0u;  // a byte of 255
      // a quarter of each value (MXFP4 reaches 6 * 2**127, past float32)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float v[8];
        mx4_decode8(cw[i], byte(i) - 129, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) am[q] = fmaxf(am[q], fabsf(v[q]));
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) ex[q] = am[q] < 1.0f ? mx_exponent(4.0f * am[q]) : mx_exponent(am[q]) + 2;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sc[q] = ex[q] == -127 ? 1.0f : __uint_as_float((uint32_t)(ex[q] + 127) << 23);
  }
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {  // columns 4 h .. 4 h + 3 of the lane
    // (decoded and hashed again, instead of keeping 256 values live)
    int64_t jh = j0;
    asm volatile("" : "+v"(jh));
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+v"(cw[i]));
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sbp[i]));
    if (plain) {
      const uint32_t hm = 0u - (uint32_t)h;
      float hs[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) hs[q] = h ? sc[4 + q] : sc[q];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t od[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) od[q] = 0u;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const int i = 4 * k + ii;
          const uint32_t cv = cw[i] >> (16 * h);
          const float s = scale(i);
          const f32x2 d[2] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cv, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cv, s, 1)};
          Fmix32x4 hw((uint32_t)jh + (uint32_t)i * (uint32_t)(C / 2), key0);
          hw.m0 += hw.d2 & hm;  // (words 2 h and 2 h + 1)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t word = hw.word(p);
            od[2 * p] = sr_fp8_scaled(od[2 * p], d[p][0], word << 16, hs[2 * p], ii);
            od[2 * p + 1] = sr_fp8_scaled(od[2 * p + 1], d[p][1], word & 0xFFFF0000u, hs[2 * p + 1], ii);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) put(k, q, od[q]);
      }
    } else {
      // (both halves are made and one is dropped.  A block of zeros has the scale
      // byte 0, so a wave that meets one comes here: 131072 x 1536 by events 119 us
      // without zero rows, 147 with one in a thousand, 182 in a hundred, 218 in ten)
      auto deqw = [&](int i, float (&q)[8]) {  // q * 2**(sb - 127 - ex)
        mx4_decode8(cw[i], 0, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_ldexpf(q[j], byte(i) - 127 - ex[j]);
      };
      uint32_t lo[4];
      const float one[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      requant_block<false, true>(deqw, 32, 1.0f, one, jh, C / 2, base, key0, [&](int k, int q, uint32_t v) {
        if (q < 4) lo[q] = v;
        else put(k, q - 4, h ? v : lo[q & 3]);
      });
    }
    // the half's codes as 128-byte column runs, 8 lanes per run
    __syncthreads();
#pragma unroll
    for (int it = 0; it < COLS / 2 * 8 / THREADS; ++it) {
      const int idx = it * THREADS + tid, col = idx >> 3, chunk = idx & 7, b = chunk >> 1;
      const int64_t Pb = lblk[b][1], gc = c0 + (col >> 2) * LCOLS + 4 * h + (col & 3);
      if (Pb != 0 && gc < C)
        *reinterpret_cast<u32x4*>(out_c + lblk[b][0] + gc * Pb + (chunk & 1) * 16) =
            *reinterpret_cast<const u32x4*>(lq + col * ROWS + swz(col, chunk) * 16);
    }
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) lsf[(LCOLS * l + q) * WAVES + w] = nan ? 255u : (uint8_t)(ex[q] + 127);
  __syncthreads();
  rq_store_scales(lsf, lblk, c0, C, sfb, out_s);
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
  if (rows == 0) return MOE4_OK;  // (an empty map's pointer is NULL)
  if (out_map)
    MOE4_REQUIRE(copies >= 1 && out_rows >= 0 && rows * copies < ((int64_t)1 << 31), MOE4_EINVAL,
                 "mxfp4_quant: out_map needs copies >= 1, out_rows >= 0 and rows * copies below 2^31");
  else
    MOE4_REQUIRE(copies == 1 && out_rows == rows, MOE4_EINVAL, "mxfp4_quant: without out_map, copies = 1 and out_rows = rows");
  // (no output rows: nothing is written, but every entry of out_map is reported)
  MOE4_REQUIRE(x && (out_rows == 0 || (codes && sf)), MOE4_EINVAL, "mxfp4_quant: NULL pointer");
  MOE4_REQUIRE(aligned16(x) && aligned16(codes), MOE4_EALIGN, "mxfp4_quant: x and codes must be 16-byte aligned");
  const int64_t pieces = rows * (cols / 8), units = (pieces + m4q::UNIT - 1) / m4q::UNIT;
  const int threads = pre_op == MOE4_PRE_SILU ? m4q::THREADS_SILU : m4q::THREADS;
  int64_t wg = (units + threads / 64 - 1) / (threads / 64);
  if (pre_op == MOE4_PRE_SILU && wg > m4q::SILU_WG) wg = m4q::SILU_WG;
  MOE4_REQUIRE(grid_fits(wg, threads), MOE4_EINVAL, "mxfp4_quant: tensor too large");
  const float* tab = nullptr;
  if (pre_op == MOE4_PRE_SILU) {
    const int rc = act_tables(&tab);
    if (rc) return rc;
  }
#define MOE4_MX4Q(DT, PRE, MAP)                                                                                       \
  hipLaunchKernelGGL((k_mx4_rows<DT, PRE, MAP>), dim3((unsigned)wg), dim3(threads), 0, as_stream(stream), x,          \
                     pieces, units, (uint32_t)(cols / 32), out_map, copies, out_rows, reinterpret_cast<u32x4*>(codes), \
                     sf, tab)
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
  MOE4_REQUIRE(grid_fits(wg, m4q::THREADS), MOE4_EINVAL, "mxfp4_dequant: tensor too large");
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(codes);
  if (out_dtype == MOE4_F32)
    hipLaunchKernelGGL(k_mx4_dequant<MOE4_F32>, dim3((unsigned)wg), dim3(m4q::THREADS), 0, as_stream(stream), cw, sf, pieces, out);
  else
    hipLaunchKernelGGL(k_mx4_dequant<MOE4_BF16>, dim3((unsigned)wg), dim3(m4q::THREADS), 0, as_stream(stream), cw, sf, pieces, out);
  return check_launch("mxfp4_dequant");
}

extern "C" int mxfp8_requant_mx4_sr_T(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t cols,
                                     const int32_t* group_row_off, const int32_t* group_off_pad, int32_t n_groups,
                                     int64_t max_padded_rows, uint64_t seed, uint32_t stream_id, int sf_layout,
                                     uint8_t* out_codes, uint8_t* out_sf, void* stream) {
  MOE4_REQUIRE(rows >= 0 && cols > 0 && cols % 32 == 0, MOE4_EINVAL, "mxfp8_requant_mx4_sr_T: cols must be a positive multiple of 32");
  MOE4_REQUIRE(n_groups >= 1 && group_row_off && group_off_pad, MOE4_EINVAL, "mxfp8_requant_mx4_sr_T: group offsets required");
  MOE4_REQUIRE(max_padded_rows >= 0 && max_padded_rows % 32 == 0, MOE4_EINVAL,
               "mxfp8_requant_mx4_sr_T: max_padded_rows must be a multiple of 32");
  MOE4_REQUIRE(sf_layout == MOE4_SF_ROWS || sf_layout == MOE4_SF_BLOCKS, MOE4_EINVAL,
               "mxfp8_requant_mx4_sr_T: sf_layout must be MOE4_SF_ROWS or MOE4_SF_BLOCKS");
  if (max_padded_rows == 0) return MOE4_OK;
  MOE4_REQUIRE((rows == 0 || (codes && sf)) && out_codes && out_sf, MOE4_EINVAL, "mxfp8_requant_mx4_sr_T: NULL pointer");
  MOE4_REQUIRE(aligned16(codes) && aligned16(out_codes), MOE4_EALIGN, "mxfp8_requant_mx4_sr_T: misaligned pointer");
  const int64_t n_ct = (cols + rq::COLS - 1) / rq::COLS, n_rt = (max_padded_rows + rq::ROWS - 1) / rq::ROWS;
  MOE4_REQUIRE(grid_fits(n_ct * n_rt, rq::THREADS), MOE4_EINVAL, "mxfp8_requant_mx4_sr_T: tensor too large");
  hipLaunchKernelGGL(k_requant_mx4_T, dim3((unsigned)(n_ct * n_rt)), dim3(rq::THREADS), 0, as_stream(stream), codes, sf,
                     cols, group_row_off, group_off_pad, n_groups, rows, max_padded_rows, n_ct,
                     sr_base_key(seed, stream_id), (int)(sf_layout == MOE4_SF_BLOCKS), out_codes, out_sf);
  return check_launch("mxfp8_requant_mx4_sr_T");
}
