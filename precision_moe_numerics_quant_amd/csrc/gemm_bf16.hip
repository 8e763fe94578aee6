// Expert-grouped BF16 products with their epilogues (gfx950): forward with
// bias, activation and residual, the gated block, and their input gradients.
// v_mfma_f32_16x16x32_bf16, float32 accumulation, each result rounded once.
#include <type_traits>

#include "bf16_tile.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16() { return take_device_word(&g_dev_err); }

template <int N>
using Int = std::integral_constant<int, N>;

namespace t16 {
constexpr int MAX_E = 4096;
constexpr int GM = 4;            // m-tiles of a group (see tile order)
}  // namespace t16

// One m-tile: rows row0 .. row0 + rows - 1 of expert e, 64 mi rows of LDS.
struct MTile {
  int e;
  int32_t row0, rows, mi;
};

template <int MODE, bool OUT_BF16>
__global__ void __launch_bounds__(t16::NT, 1) k_bf16_tile(Bf16Args p, int cap, uint32_t n_nt) {
  using namespace t16;
  constexpr bool TR = MODE == DGRAD || MODE == GDGRAD;   // w's columns are the product's: read transposed
  constexpr int NW = MODE == GATED ? TN / 2 : TN;        // the tile's columns
  __shared__ __attribute__((aligned(16))) uint8_t ring[RING];
  __shared__ uint32_t s_first[MAX_E + 1];
  __shared__ uint32_t s_scan[4];
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w >> 1, wn = w & 1;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)ring);

  // the experts' first m-tiles: thread t counts experts t P .. t P + P - 1
  const int E = p.E;
  const int32_t M = (int32_t)p.M;
  auto tiles_of = [&](int32_t n) __attribute__((always_inline)) { return n > 0 ? ((uint32_t)n + (1u << cap) - 1) >> cap : 0u; };
  auto rows_of = [&](int32_t r0, int32_t r1) __attribute__((always_inline)) { return (r1 < M ? r1 : M) - (r0 > 0 ? r0 : 0); };
  {
    const int P = (E + NT - 1) / NT;
    uint32_t mine = 0;
    for (int e = tid * P; e < (tid + 1) * P && e < E; ++e) {
      mine += tiles_of(rows_of(p.off[e], p.off[e + 1]));
    }
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t y = __shfl_up(inc, o, 64);
      if (l >= o) inc += y;
    }
    if (l == 63) s_scan[w] = inc;
    __syncthreads();
    uint32_t run = inc - mine;
    for (int i = 0; i < w; ++i) run += s_scan[i];
    for (int e = tid * P; e < (tid + 1) * P && e < E; ++e) {
      s_first[e] = run;
      run += tiles_of(rows_of(p.off[e], p.off[e + 1]));
    }
    if (tid == NT - 1) s_first[E] = run;   // (threads past E hold the total too)
    __syncthreads();
  }
  const uint32_t n_mt = __builtin_amdgcn_readfirstlane(s_first[E]), total = n_mt * n_nt;
  // this workgroup's tiles: its XCD's share in order, every gridDim / 8-th of it
  const uint32_t xcd = blockIdx.x % 8, stride = gridDim.x / 8, per = (total + 7) / 8;
  const uint32_t t_end = (xcd + 1) * per < total ? (xcd + 1) * per : total, t_begin = xcd * per + blockIdx.x / 8;
  if (t_begin >= t_end) return;

  // tile t -> its m-tile and n-tile
  auto locate = [&](uint32_t t, MTile& m, uint32_t& nt) __attribute__((always_inline)) {
    const uint32_t gsz = GM * n_nt, g = t / gsz, r = t - g * gsz;
    const uint32_t gm = n_mt - g * GM < GM ? n_mt - g * GM : GM;
    nt = r / gm;
    const uint32_t mi = g * GM + (r - nt * gm);
    // the last expert e with s_first[e] <= mi (experts without tiles share their successor's)
    int lo = 0;
    for (int step = E <= 64 ? 1 : (E <= 64 * 64 ? 64 : 4096); step >= 1; step /= 64) {
      const int at = lo + l * step;
      const unsigned long long b = __ballot(at <= E && s_first[at <= E ? at : E] <= mi);
      lo += (63 - __clzll((long long)b)) * step;
    }
    m.e = __builtin_amdgcn_readfirstlane(lo);
    // (scalar loads: a vector load here would wait for the loads in flight)
    const int32_t r0 = ld_const(p.off, m.e), n = rows_of(r0, ld_const(p.off, m.e + 1));
    const uint32_t cnt = tiles_of(n), even = (((uint32_t)n + cnt - 1) / cnt + 63) / 64 * 64;   // rows of all tiles but the last
    const int32_t at = (int32_t)((mi - __builtin_amdgcn_readfirstlane(s_first[m.e])) * even);
    m.row0 = (r0 > 0 ? r0 : 0) + at;
    m.rows = n - at < (int32_t)even ? (n > at ? n - at : 0) : (int32_t)even;
    m.mi = (m.rows + 63) / 64;
  };

  const uint32_t K = (uint32_t)p.K, N = (uint32_t)p.N, KB = K * 2, nk0 = ((K + BK - 1) / BK + 1) / 2 * 2, nk = nk0 < S ? S : nk0;
  const uint32_t ldb = TR ? N * 2 : KB;                     // bytes of a row of w

  // ------------------------------------------------------------- load stream
  // (past the last tile it goes on with descriptors of nothing, so that every
  // step issues as many loads)
  uint32_t lt = t_begin, ls = 0;
  u32x4 ra, rb;
  uint32_t voa[4], vob[4];
  const uint32_t ca = (l & 3) ^ ((l >> 4) & 3);             // A: the chunk that lands in slot l & 3 of row l >> 2
  auto cb = [&](int t) __attribute__((always_inline)) { return TR ? ((uint32_t)(l & 31) ^ (4 * ((2 * t + (l >> 5)) & 3))) : ((uint32_t)(l & 3) ^ ((2 * t + (l >> 5)) & 3)); };
  auto seek = [&]() __attribute__((always_inline)) {
    ls = 0;
    if (lt >= t_end) {
      ra = rsrc4(p.a, 0);
      rb = ra;
      return;
    }
    MTile m;
    uint32_t nt;
    locate(lt, m, nt);
    const int64_t n0 = (int64_t)nt * NW;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = 64 * w + 16 * t + (l >> 2);
      uint32_t o = OOB;
      if (r < m.rows) {
        const int64_t row = mapped_row(p.map, (int64_t)m.row0 + r, p.div, p.magic, p.a_rows, &g_dev_err);
        if (row >= 0) o = (uint32_t)(p.map ? row : r) * KB + 16 * ca;
      }
      voa[t] = o;
    }
    ra = rsrc4(p.map ? p.a : p.a + (int64_t)m.row0 * p.K, (uint64_t)(p.map ? p.a_rows : m.rows) * KB);
    if (TR) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t k = 8 * w + 2 * t + (l >> 5), c = cb(t);
        vob[t] = n0 + 8 * c < N ? k * ldb + 16 * c : OOB;
      }
      rb = rsrc4(p.w + (int64_t)m.e * p.K * p.N + n0, (uint64_t)(K * (uint64_t)N - n0) * 2);
    } else {
      const int64_t row0 = MODE == GATED ? (int64_t)m.e * 2 * p.N : (int64_t)m.e * p.N;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t R = 64 * w + 16 * t + (l >> 2);      // GATED: 64 gate and 64 up columns for each wave column
        const uint32_t n = MODE == GATED ? (uint32_t)n0 + 64 * (R >> 7) + (R & 63) : (uint32_t)n0 + R;
        const uint32_t row = MODE == GATED ? ((R >> 6) & 1) * N + n : n;
        vob[t] = n < N ? row * KB + 16 * cb(t) : OOB;
      }
      rb = rsrc4(p.w + row0 * p.K, (uint64_t)(MODE == GATED ? 2 : 1) * N * KB);
    }
  };
  // this wave's loads of a stage, four of each operand
  auto load_a = [&](int t, uint32_t stage) __attribute__((always_inline)) {
    load_lds(ra, lds0 + stage * STAGE + (4 * w + t) * 1024, 4 * ls + ca < K / 8 ? voa[t] : OOB, ls * (BK * 2));
  };
  auto load_b = [&](int t, uint32_t stage) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + stage * STAGE + HALF + (4 * w + t) * 1024;
    // (TR: rows past K lie past the descriptor, so all of the offset in the operand that is checked)
    if (TR) load_lds(rb, dst, vob[t] + ls * BK * ldb, 0);
    else load_lds(rb, dst, 4 * ls + cb(t) < K / 8 ? vob[t] : OOB, ls * (BK * 2));
  };
  // --------------------------------------------------------------- fragments
  uint32_t lb[4];                                            // TR: the lane's offset for each pair of column blocks
  uint32_t la = 0, lbn = 0;
  if (TR) {
    const int j = li >> 2, s = li & 3;
#pragma unroll
    for (int pb = 0; pb < 4; ++pb) lb[pb] = HALF + (8 * q + j) * 512 + 16 * (16 * wn + 4 * (pb ^ j) + s);
  } else {
    lbn = HALF + (128 * wn + 8 * (li >> 2) + (li & 3)) * 64 + 16 * (q ^ (li >> 2));
  }
  auto frag_a = [&](bf16x8& f, int i, uint32_t st) __attribute__((always_inline)) { f = *reinterpret_cast<const bf16x8*>(ring + st + la + 1024 * i); };
  auto frag_b = [&](bf16x8& f, int i, uint32_t st) __attribute__((always_inline)) {
    const int pb = i >> 1, b = i & 1;
    if (TR) {
      typedef __attribute__((address_space(3))) s16x4* lp;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + st + lb[pb] + 8 * b));
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + st + lb[pb] + 8 * b + 2048));
      f = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      f = *reinterpret_cast<const bf16x8*>(ring + st + lbn + 2048 * pb + 256 * b);
    }
  };

  // waits until all of this wave's loads but those of the S - 2 latest stages
  // have landed
  auto landed = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * LOADS));
  };
  auto barrier = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };

  seek();
  for (int s = 0; s < S; ++s) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      load_a(t, s);
      load_b(t, s);
    }
    ++ls;
  }

  uint32_t gs = 0;   // stage counter of the compute stream
  for (uint32_t ct = t_begin; ct < t_end; ct += stride) {
    MTile m;
    uint32_t nt;
    locate(ct, m, nt);
    auto run = [&](auto mb) __attribute__((always_inline)) {
      constexpr int MB = decltype(mb)::value;
      f32x4 acc[MB][8];
      bf16x8 fa[2][MB], fb[2][8];
      // One step: the MFMAs of set CUR, the loads into this step's stage (every
      // wave has read it), the reads of the next stage into the other set.
      auto step = [&](auto cur) __attribute__((always_inline)) {
        constexpr int CUR = decltype(cur)::value;
        landed();
        barrier();
        const uint32_t nst = ((gs + 1) % S) * STAGE, stg = gs % S;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i < MB) frag_a(fa[1 - CUR][i < MB ? i : 0], i, nst);
          frag_b(fb[1 - CUR][i], i, nst);
          if (i < 4) load_a(i, stg);
          else load_b(i - 4, stg);
          if (i < MB) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
              acc[i < MB ? i : 0][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[CUR][n], fa[CUR][i < MB ? i : 0], acc[i < MB ? i : 0][n], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        ++ls;
        gs = __builtin_amdgcn_readfirstlane(gs + 1);
      };
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[i][n] = f32x4{};
      la = (16 * MB * wm + li) * 64 + 16 * (q ^ (li >> 2));
      __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * LOADS));
      barrier();
      {
        const uint32_t st = (gs % S) * STAGE;
#pragma unroll
        for (int i = 0; i < MB; ++i) frag_a(fa[0][i], i, st);
#pragma unroll
        for (int i = 0; i < 8; ++i) frag_b(fb[0][i], i, st);
      }
      // the loads are S steps ahead: from step nk - S on they are the next tile's.
      // (The last step reads fragments of the next tile's first stage, of no use:
      // its rows lie differently over the waves.)
      for (uint32_t s = 0; s < nk; s += 2) {
        if (s == nk - S) {
          lt += stride;
          seek();
        }
        step(Int<0>{});
        step(Int<1>{});
      }
      const Bf16Epilogue<MODE, OUT_BF16> epi(p, m.e, m.row0, m.rows);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = 16 * MB * wm + 16 * i + li;
        const float sc = (MODE == DGRAD || MODE == GDGRAD) && r < m.rows ? row_scale(p.scale, p.map, (int64_t)m.row0 + r, p.a_rows * p.div) : 1.0f;
#pragma unroll
        for (int pb = 0; pb < (MODE == GATED ? 2 : 4); ++pb) {
          const uint32_t n = nt * NW + (MODE == GATED ? 64 : 128) * wn + 32 * pb + 8 * q;
          const f32x4 x = acc[i][2 * pb], y = acc[i][2 * pb + 1];
          const f32x4 x1 = acc[i][MODE == GATED ? 2 * pb + 4 : 0], y1 = acc[i][MODE == GATED ? 2 * pb + 5 : 0];
          const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
          const float z1[8] = {x1[0], x1[1], x1[2], x1[3], y1[0], y1[1], y1[2], y1[3]};
          epi.template put<8>(r, n, sc, z, z1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    if (m.mi >= 4) run(Int<8>{});
    else if (m.mi == 3) run(Int<6>{});
    else if (m.mi == 2) run(Int<4>{});
    else run(Int<2>{});
  }
  __builtin_amdgcn_s_waitcnt(wait_vm(0));   // (no load into this workgroup's LDS outlives it)
}

static int cu_count() {
  static int n[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (n[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    n[dev] = v;
  }
  return n[dev];
}

template <int MODE, bool OUT_BF16>
static int launch_bf16(const Bf16Args& p, void* stream, const char* name) {
  using namespace t16;
  constexpr int NW = MODE == GATED ? TN / 2 : TN;
  const int64_t nt = (p.N + NW - 1) / NW;
  const int cus = cu_count() / 8 * 8 < 8 ? 8 : cu_count() / 8 * 8;
  int cap = 8;   // log2 of a tile's most rows
  while (cap > 6 && ((p.M >> cap) + (p.M < p.E ? p.M : p.E)) * nt < cus) --cap;
  MOE4_REQUIRE(((p.M >> cap) + p.E) * nt < ((int64_t)1 << 31), MOE4_EINVAL, std::string(name) + ": too large");
  hipLaunchKernelGGL((k_bf16_tile<MODE, OUT_BF16>), dim3((unsigned)cus), dim3(NT), 0, as_stream(stream), p, cap, (uint32_t)nt);
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
