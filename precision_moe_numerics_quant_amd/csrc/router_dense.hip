// The router's backward for a dense logit gradient (gfx950): a balance loss
// puts a gradient on every expert's logit, so the products that only visit
// each token's k selected experts (router.hip) do not cover it.
//
//   k_router_dx_dense  dx[t] = bf16(sum_j dXp[row(t, j)] + sum_e dz[t, e] W_r[e]):
//                      the un-permuting sum with the GEMM dz . W_r under it,
//                      64 x 128 tiles (T x d), the sum added in the epilogue.
//   k_router_dw_dense  dW_r [E, d] = dz^T . x, 128 x 128 tiles (E x d), the
//                      tokens split over workgroups whose partial tiles
//                      k_router_dw_join adds in order.
//
// dz is float32 and the other operand bf16.  A float32 from 2^-110 on is exactly
// the sum of three bf16 numbers (its 24 significand bits cut 8 + 8 + 8; the MFMA
// keeps bf16's subnormals), so three bf16 MFMAs per fragment
// (v_mfma_f32_32x32x16_bf16) give exact products with float32 accumulation:
// nothing of dz is rounded, at three bf16 MFMAs where a float32 MFMA would take
// eight times as long as one.  Below 2^-110 the last part ends at bf16's
// smallest subnormal: dz is cut by less than 2^-133.
//
// Both contractions run along a dimension that is not contiguous in memory
// (W_r's rows; dz's and x's tokens): a thread loads 8 consecutive k of one or
// two columns (whole cache lines across the wave) and the bytes are put into
// fragment order on the way to LDS, [k / 8][row][8 k]: a fragment read is then
// 16 consecutive bytes per lane, without bank conflicts.
//
// Measured at 16384 tokens, k = 8, d = 4096, 384 experts: dx 507 us, against 427
// for the un-permuting sum alone (2.1 GB gathered at 5.2 TB/s, the bound) and 213
// for the GEMM alone, which hides partly behind the other workgroups' gathers:
// six per CU (one LDS stage, one register set; 128-row tiles with two stages, 2 per
// CU: 587).  dW 216 us (181 to 256 from launch to launch: power moves the clock
// about 1.7 GHz) and 11 for the join, 113 at the bf16 MFMA rate of a large
// product; the MFMAs and the VALU are busy 40 % of the cycles each: its operands
// cross from token-major rows through registers into LDS, three parts of dz each.
// 64-deep slabs or 256-wide tiles would cut the workgroups per CU again.
#include "gemm_common.h"
#include "moe4_internal.h"

namespace moe4 {

namespace rd {
constexpr int TM = 128, TN = 128, BK = 32, NT = 256;
constexpr int KC = BK / 8;                  // 8-deep k chunks of a slab
constexpr int PART_B = KC * TM * 16;        // bytes of one bf16 operand slab
constexpr int STAGE = 4 * PART_B;           // three parts of dz, one of the other operand
constexpr int MAXK = 16;
constexpr int CUS = 256;  // (MI355X; not asked of the device: the workspace query, which names none, uses it too)
constexpr int64_t MAXE = (1 << 20) - 1, MAXD = (1 << 28) - 1;  // (128 rows of dz and a row of W_r: 31-bit byte ranges)
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
}  // namespace rd

constexpr int CLASS_INF = 0x204;  // -infinity, +infinity

// 8 float32 values -> their three bf16 parts (the high 8 significand bits,
// the next 8, the last 8; each subtraction is exact), 8 bf16 each.  An infinity
// is all in the first part (less itself it would be a NaN).
__device__ inline void split3(const float (&v)[8], u32x4 (&o)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[2], m[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float a = v[2 * i + j];
      h[j] = __float_as_uint(a) & 0xFFFF0000u;
      const float r = __builtin_amdgcn_classf(a, CLASS_INF) ? 0.0f : a - __uint_as_float(h[j]);
      m[j] = __float_as_uint(r) & 0xFFFF0000u;
      lo[j] = __float_as_uint(r - __uint_as_float(m[j]));
    }
    o[0][i] = (h[0] >> 16) | h[1];
    o[1][i] = (m[0] >> 16) | m[1];
    o[2][i] = (lo[0] >> 16) | (lo[1] & 0xFFFF0000u);
  }
}

// 8 dwords of two bf16 columns each (row i in w[i]) -> the 8 k of each column.
__device__ inline void columns2(const uint32_t (&w)[8], u32x4& c0, u32x4& c1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c0[i] = (w[2 * i] & 0xFFFFu) | (w[2 * i + 1] << 16);
    c1[i] = (w[2 * i] >> 16) | (w[2 * i + 1] & 0xFFFF0000u);
  }
}

// A thread's share of one slab in registers: 8 k of a row (dx) or two columns (dW)
// of dz and of two columns of the other operand.
struct RdRegs {
  float a[2][8];
  uint32_t b[8];
};

// One slab of a tile of ROWS rows: wave (wm, wn) owns 32 MI x 32 NJ of it, in
// MFMA blocks of 32 x 32.
template <int ROWS, int MI, int NJ>
__device__ inline void rd_compute(const uint8_t* st, int wm, int wn, f32x16 (&acc)[MI][NJ]) {
  using namespace rd;
  constexpr int PART_A = KC * ROWS * 16;
  const int l = threadIdx.x & 63, li = l & 31, g = l >> 5;
#pragma unroll
  for (int kk = 0; kk < BK / 16; ++kk) {
    const int c = 2 * kk + g;  // lane half g holds k = 16 kk + 8 g .. + 7
    bf16x8 a[3][MI], b[NJ];
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int i = 0; i < MI; ++i)
        a[p][i] = *reinterpret_cast<const bf16x8*>(st + p * PART_A + (c * ROWS + wm + 32 * i + li) * 16);
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = *reinterpret_cast<const bf16x8*>(st + 3 * PART_A + (c * TN + wn + 32 * j + li) * 16);
#pragma unroll
    for (int p = 2; p >= 0; --p)  // the smallest parts first
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[p][i], b[j], acc[i][j], 0, 0, 0);
  }
}

// idx clamped to [0, n); a clamp is reported
__device__ inline int64_t clamp_row(int64_t i, int64_t n, uint32_t* err) {
  if (i < 0 || i >= n) {
    atomicOr(err, MOE4_DEVERR_INDEX);
    return i < 0 ? 0 : n - 1;
  }
  return i;
}

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_router_dense() { return take_device_word(&g_dev_err); }

// ROWS x 128 tiles: a tile's gathers follow one another, so many small tiles side
// by side hide them best until W_r's slabs are read too often.  64 rows: 525 us at
// 16384 tokens (128 rows 531, 32 rows 544; at k = 2, 8000 tokens 156, 150, 190).
// 32 rows where 64 would leave CUs with one tile or none: 512 tokens 25 - 28, 333
// tokens with 130 experts, k = 6, d = 520 10 us (128 rows: 27).
template <int ROWS>
__global__ void __launch_bounds__(rd::NT, 4)
    k_router_dx_dense(const float* __restrict__ dxp, const int32_t* __restrict__ inv, int64_t T, int k, int64_t d,
                      const float* __restrict__ dz, int E, const uint16_t* __restrict__ w, int64_t n_nt, int64_t n_all,
                      uint16_t* __restrict__ dx) {
  using namespace rd;
  constexpr int PART_A = KC * ROWS * 16, SLAB = 3 * PART_A + PART_B;
  constexpr int MI = ROWS / 32;
  constexpr int HROWS = 32;  // rows of the float32 tile in LDS at a time
  __shared__ __attribute__((aligned(16))) uint8_t lds[SLAB > HROWS * TN * 4 ? SLAB : HROWS * TN * 4];
  __shared__ int32_t rows[ROWS * MAXK];  // dXp's rows of the tile's tokens
  const int64_t tile = xcd_tile(blockIdx.x, n_all);
  if (tile >= n_all) return;
  const int64_t t0 = (tile / n_nt) * ROWS, c0 = (tile % n_nt) * TN;
  const int tid = threadIdx.x, l = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = 32 * wv;  // the wave's columns
  for (int i = tid; i < ROWS * k; i += NT)  // (tokens past T: any row)
    rows[i] = t0 * k + i < T * k ? (int32_t)clamp_row(inv[t0 * k + i], T * k, &g_dev_err) : 0;
  // dz: unit (row tid / 4, chunk tid % 4; 32 rows: the first half of the threads); W_r: unit (chunk tid / 64, columns 2 l, 2 l + 1)
  const int ach = tid & 3, ar = tid >> 2;
  const int64_t bc = c0 + 2 * l;
  // (a descriptor that ends with the tile's rows, and one per row of W_r: rows
  // past T or E and columns past d come as zeros)
  const __amdgpu_buffer_rsrc_t rz = make_rsrc(dz + t0 * E, (uint64_t)(T - t0 < ROWS ? T - t0 : ROWS) * E * 4);
  const uint32_t zo = (uint32_t)ar * E * 4 + 32u * ach;
  const uint32_t wo = (uint32_t)bc * 2;
  auto load = [&](RdRegs& q, int k0) {
    const uint32_t o = zo + (uint32_t)k0 * 4;
    const u32x4 x0 = __builtin_amdgcn_raw_buffer_load_b128(rz, o, 0, 0), x1 = __builtin_amdgcn_raw_buffer_load_b128(rz, o + 16, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q.a[0][i] = __uint_as_float(x0[i]);
      q.a[0][4 + i] = __uint_as_float(x1[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = k0 + 8 * wv + i;
      q.b[i] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(w + (int64_t)(e < E ? e : 0) * d, e < E ? (uint64_t)d * 2 : 0), wo, 0, 0);
    }
  };
  // (k0: the slab's first expert; past E the row's values are the next row's)
  auto store = [&](RdRegs& q, uint8_t* st, int k0) {
    if (k0 + BK > E) {  // (uniform)
#pragma unroll
      for (int i = 0; i < 8; ++i) q.a[0][i] = k0 + 8 * ach + i < E ? q.a[0][i] : 0.0f;
    }
    if (ar < ROWS) {
      u32x4 o[3];
      split3(q.a[0], o);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4*>(st + p * PART_A + (ach * ROWS + ar) * 16) = o[p];
    }
    u32x4 b0, b1;
    columns2(q.b, b0, b1);
    *reinterpret_cast<u32x4*>(st + 3 * PART_A + (wv * TN + 2 * l) * 16) = b0;
    *reinterpret_cast<u32x4*>(st + 3 * PART_A + (wv * TN + 2 * l + 1) * 16) = b1;
  };
  f32x16 acc[MI][1];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i][0] = f32x16{};
  const int nk = (E + BK - 1) / BK;
  RdRegs q;
  load(q, 0);
  for (int s = 0; s < nk; ++s) {
    store(q, lds, s * BK);
    __syncthreads();
    if (s + 1 < nk) load(q, (s + 1) * BK);  // in flight during this slab's MFMAs
    rd_compute<ROWS>(lds, 0, wn, acc);
    __syncthreads();
  }
  // the tile through LDS, HROWS rows at a time, so that a thread adds whole
  // 16-byte pieces of rows
  float* tl = reinterpret_cast<float*>(lds);
  const int li = l & 31, g = l >> 5;
  const int64_t col = c0 + 4 * (tid & 31);
#pragma unroll
  for (int h = 0; h < ROWS / HROWS; ++h) {
#pragma unroll
    for (int v = 0; v < 16; ++v) tl[((v >> 2) * 8 + 4 * g + (v & 3)) * TN + wn + li] = acc[h][0][v];
    __syncthreads();
    // many tiles: the rows, read once, leave W_r in the L2 (nontemporal: 524 -> 505 us at
    // 16384 tokens, 236 -> 212 at 8000 with 64 experts; 24.5 -> 26.4 for the 32-row tiles' batches,
    // which the caches hold)
    constexpr int JS = 8;  // row loads in flight per lane (with more, fewer workgroups fit: slower)
    if (col < d)
      for (int r = tid >> 5; r < HROWS && t0 + HROWS * h + r < T; r += NT / 32) {
        const int32_t* rw = rows + (HROWS * h + r) * k;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j0 = 0; j0 < k; j0 += JS) {
          f32x4 v[JS];
#pragma unroll
          for (int j = 0; j < JS; ++j)
            if (j0 + j < k) {
              const f32x4* q = reinterpret_cast<const f32x4*>(dxp + (int64_t)rw[j0 + j] * d + col);
              v[j] = ROWS == 64 ? __builtin_nontemporal_load(q) : *q;
            }
#pragma unroll
          for (int j = 0; j < JS; ++j)
            if (j0 + j < k) s = s + v[j];
        }
        s = s + *reinterpret_cast<const f32x4*>(tl + r * TN + 4 * (tid & 31));
        *reinterpret_cast<u32x2*>(dx + (t0 + HROWS * h + r) * d + col) = u32x2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
      }
    __syncthreads();
  }
}

// Workgroup (tile, token share z): out + z * E * d gets the share's partial
// products (out is dW itself when there is one share).
__global__ void __launch_bounds__(rd::NT, 4)
    k_router_dw_dense(const uint16_t* __restrict__ x, const float* __restrict__ dz, int64_t T, int E, int64_t d,
                      int64_t n_nt, int64_t share, float* __restrict__ out) {
  using namespace rd;
  __shared__ __attribute__((aligned(16))) uint8_t lds[STAGE];
  const int64_t e0 = (blockIdx.x / n_nt) * TM, c0 = (blockIdx.x % n_nt) * TN;
  const int64_t ta = (int64_t)blockIdx.y * share, tb = ta + share < T ? ta + share : T;
  const int tid = threadIdx.x, l = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wv >> 1) * 64, wn = (wv & 1) * 64;
  // dz: units (chunk wv, expert l + 64 j); x: unit (chunk wv, columns 2 l, 2 l + 1)
  const int64_t bc = c0 + 2 * l;
  const uint32_t zo = (uint32_t)(e0 + l) * 4, xo = (uint32_t)bc * 2;
  auto load = [&](RdRegs& q, int64_t k0) {  // a descriptor per row: tokens past the share, experts past E, columns past d are 0
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = k0 + 8 * wv + i, tr = t < tb ? t : 0;
      const __amdgpu_buffer_rsrc_t rz = make_rsrc(dz + tr * E, t < tb ? (uint64_t)E * 4 : 0);
      const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + tr * d, t < tb ? (uint64_t)d * 2 : 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) q.a[j][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rz, zo + 256 * j, 0, 0));
      q.b[i] = __builtin_amdgcn_raw_buffer_load_b32(rx, xo, 0, 0);
    }
  };
  auto store = [&](const RdRegs& q, uint8_t* st) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 o[3];
      split3(q.a[j], o);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x4*>(st + p * PART_B + (wv * TM + l + 64 * j) * 16) = o[p];
    }
    u32x4 b0, b1;
    columns2(q.b, b0, b1);
    *reinterpret_cast<u32x4*>(st + 3 * PART_B + (wv * TN + 2 * l) * 16) = b0;
    *reinterpret_cast<u32x4*>(st + 3 * PART_B + (wv * TN + 2 * l + 1) * 16) = b1;
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  const int nk = tb > ta ? (int)((tb - ta + BK - 1) / BK) : 0;
  RdRegs q;
  load(q, ta);
  for (int s = 0; s < nk; ++s) {
    store(q, lds);
    __syncthreads();
    if (s + 1 < nk) load(q, ta + (int64_t)(s + 1) * BK);  // in flight during this slab's MFMAs
    rd_compute<TM>(lds, wm, wn, acc);
    __syncthreads();
  }
  const int li = l & 31, g = l >> 5;
  float* o = out + (int64_t)blockIdx.y * E * d;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = c0 + wn + 32 * j + li;
      if (col >= d) continue;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t e = e0 + wm + 32 * i + (v >> 2) * 8 + 4 * g + (v & 3);
        if (e < E) o[e * d + col] = acc[i][j][v];
      }
    }
}

// dw = the partial products of the n shares, added in order (n4 = E d / 4).
__global__ void __launch_bounds__(256) k_router_dw_join(const f32x4* __restrict__ part, int n, int64_t n4,
                                                        f32x4* __restrict__ dw) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4 s = part[i];
  for (int z = 1; z < n; ++z) s = s + part[z * n4 + i];
  dw[i] = s;
}

// Token shares of the weight gradient: enough workgroups for four per CU, at
// least 8 slabs each; where that does not give every CU one, at least 2
// slabs (333 tokens, 130 experts, d = 520: 20 us in one share, 9.5 + 3 in five
// with the join).
inline int dw_shares(int64_t T, int E, int64_t d) {
  const int64_t tiles = ((E + rd::TM - 1) / rd::TM) * ((d + rd::TN - 1) / rd::TN);
  int64_t n = 1024 / tiles;
  const int64_t most = T / (8 * rd::BK);
  if (n > most) n = most;
  if (n < 1) n = 1;
  if (n * tiles < rd::CUS) {
    n = rd::CUS / tiles;
    if (n > T / (2 * rd::BK)) n = T / (2 * rd::BK);
  }
  return (int)(n < 1 ? 1 : n);
}

}  // namespace moe4

using namespace moe4;

extern "C" int moe_unpermute_sum_router_dense(const float* dxp, const int32_t* inv_perm, int64_t T, int32_t k, int64_t d,
                                              const float* dlogits, int32_t E, const uint16_t* w, uint16_t* dx,
                                              void* stream) {
  MOE4_REQUIRE(T >= 0 && E >= 1 && E <= rd::MAXE && k >= 1 && k <= rd::MAXK && d > 0 && d <= rd::MAXD && d % 4 == 0, MOE4_EINVAL,
               "moe_unpermute_sum_router_dense: need 1 <= k <= 16, 1 <= E < 2^20, 0 < d < 2^28 and d % 4 == 0");
  MOE4_REQUIRE(T * (int64_t)k < ((int64_t)1 << 31), MOE4_EINVAL, "moe_unpermute_sum_router_dense: T * k must be below 2^31");
  MOE4_REQUIRE(T == 0 || (dxp && inv_perm && dlogits && w && dx), MOE4_EINVAL, "moe_unpermute_sum_router_dense: NULL pointer");
  MOE4_REQUIRE(aligned16(dxp) && aligned16(dlogits) && aligned16(w) && aligned16(dx), MOE4_EALIGN,
               "moe_unpermute_sum_router_dense: dxp, dlogits, w and dx must be 16-byte aligned");
  if (T == 0) return MOE4_OK;
  const int64_t n_nt = (d + rd::TN - 1) / rd::TN, n64 = n_nt * ((T + 63) / 64), n32 = n_nt * ((T + 31) / 32);
  MOE4_REQUIRE(grid_fits(xcd_grid(n64), rd::NT), MOE4_EINVAL, "moe_unpermute_sum_router_dense: too large");
#define MOE4_RDX(ROWS, TILES)                                                                                        \
  hipLaunchKernelGGL(k_router_dx_dense<ROWS>, dim3((unsigned)xcd_grid(TILES)), dim3(rd::NT), 0, as_stream(stream), dxp, \
                     inv_perm, T, k, d, dlogits, E, w, n_nt, TILES, dx)
  if (n64 < 2 * rd::CUS) MOE4_RDX(32, n32);
  else MOE4_RDX(64, n64);
#undef MOE4_RDX
  return check_launch("moe_unpermute_sum_router_dense");
}

extern "C" size_t moe_router_wgrad_dense_ws_bytes(int64_t T, int32_t E, int64_t d) {
  if (T < 0 || E < 1 || d < 1) return 0;
  const int n = dw_shares(T, E, d);
  return n > 1 ? (size_t)n * (size_t)E * (size_t)d * 4 : 0;
}

extern "C" int moe_router_wgrad_dense(const uint16_t* x, const float* dlogits, int64_t T, int32_t E, int64_t d, float* dw,
                                      void* ws, size_t ws_bytes, void* stream) {
  MOE4_REQUIRE(T >= 0 && E >= 1 && E <= rd::MAXE && d > 0 && d <= rd::MAXD && d % 4 == 0, MOE4_EINVAL,
               "moe_router_wgrad_dense: need T >= 0, 1 <= E < 2^20, 0 < d < 2^28 and d % 4 == 0");
  MOE4_REQUIRE(dw && (T == 0 || (x && dlogits)), MOE4_EINVAL, "moe_router_wgrad_dense: NULL pointer");
  MOE4_REQUIRE(aligned16(x) && aligned16(dlogits) && aligned16(dw), MOE4_EALIGN,
               "moe_router_wgrad_dense: x, dlogits and dw must be 16-byte aligned");
  const int64_t n_nt = (d + rd::TN - 1) / rd::TN, tiles = n_nt * ((E + rd::TM - 1) / rd::TM);
  MOE4_REQUIRE(grid_fits(tiles, rd::NT), MOE4_EINVAL, "moe_router_wgrad_dense: too large");
  const int n = dw_shares(T, E, d);
  const size_t need = moe_router_wgrad_dense_ws_bytes(T, E, d);
  MOE4_REQUIRE(need == 0 || (ws && ws_bytes >= need), MOE4_EWORKSPACE,
               "moe_router_wgrad_dense: workspace of moe_router_wgrad_dense_ws_bytes() bytes required");
  MOE4_REQUIRE(need == 0 || aligned16(ws), MOE4_EALIGN, "moe_router_wgrad_dense: ws must be 16-byte aligned");
  const int64_t share = ((T + n - 1) / n + rd::BK - 1) / rd::BK * rd::BK;
  const hipStream_t s = as_stream(stream);
  float* out = n > 1 ? static_cast<float*>(ws) : dw;
  hipLaunchKernelGGL(k_router_dw_dense, dim3((unsigned)tiles, (unsigned)n), dim3(rd::NT), 0, s, x, dlogits, T, E, d, n_nt,
                     share, out);
  if (n > 1) {
    const int64_t n4 = (int64_t)E * d / 4;
    hipLaunchKernelGGL(k_router_dw_join, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s,
                       reinterpret_cast<const f32x4*>(ws), n, n4, reinterpret_cast<f32x4*>(dw));
  }
  return check_launch("moe_router_wgrad_dense");
}
