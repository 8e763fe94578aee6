// Weight gradients of the BF16 expert products (gfx950): per expert
// dw = dy^T a over its rows (v_mfma_f32_16x16x32_bf16, float32 accumulation),
// and the column sums of dy for the bias.
#include "bf16_tile.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16_wgrad() { return take_device_word(&g_dev_err); }

// A tile of an expert's gradient: n-tile nt (of dy's columns), k-tile kt (of a's;
// at = nt 2^16 + kt), the expert's rows.
struct WTile {
  int32_t e, at, row0, rows;
};

// The tiled products' structure (gemm_bf16.hip) with the rows as the
// contraction: a slab is 64 rows of both operands, 512 bytes of each, read
// transposed from LDS.  A map's entries come through LDS, those of eight slabs at a
// time.  order: the experts are visited in steps of
// `order` (coprime to E), so that popular and rare ones, whose tiles multiply
// and store in different proportions, run side by side.
__global__ void __launch_bounds__(t16::NT, 1) k_bf16_wgrad(Bf16Wgrad p, uint32_t n_nt, uint32_t n_kt, uint32_t order) {
  using namespace t16;
  __shared__ __attribute__((aligned(16))) uint8_t ring[RING];
  __shared__ __attribute__((aligned(16))) WTile s_tile[NT];   // this workgroup's next tiles
  __shared__ int32_t s_off[MAX_E + 1];                   // the experts' first rows, clamped
  __shared__ __attribute__((aligned(16))) uint32_t s_map[2][2][8][64];   // map entries: operand, half of them, wave, slab and row
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w >> 1, wn = w & 1, grp = w >> 2;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)ring);
  const uint32_t ldsm = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)(uint8_t*)s_map);
  const int E = p.E;
  const int32_t M = (int32_t)p.M;
  for (int e = tid; e <= E; e += NT) {
    const int32_t o = p.off[e];
    s_off[e] = o < 0 ? 0 : (o < M ? o : M);
  }
  __syncthreads();
  const uint32_t per_e = n_nt * n_kt, total = per_e * E, xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const uint32_t chunk = total >= 16 * per_e ? per_e : (total + gridDim.x - 1) / gridDim.x;
  const uint32_t N = (uint32_t)p.N, K = (uint32_t)p.K, ldd = N * 2, lda = K * 2;
  auto lane = [&]() __attribute__((always_inline)) {   // (kept from the optimiser, as in gemm_bf16.hip)
    int x = l;
    asm volatile("" : "+v"(x));
    return x;
  };

  // ------------------------------------------------------------- load stream
  uint32_t ln = 0, n_my = 0;
  int32_t lr = 0, left = 0;          // the next slab's first row in its expert, the expert's rows from there
  u32x4 rd, ra;
  uint32_t vod[4], voa[4], cd[4], ca[4];   // offsets; with a map those of the columns
  uint32_t batch = 0;                // eight slabs' map entries that have been taken up
  auto tile = [&](uint32_t i) __attribute__((always_inline)) {
    const WTile x = s_tile[i];
    return WTile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.at), __builtin_amdgcn_readfirstlane(x.row0),
                 __builtin_amdgcn_readfirstlane(x.rows)};
  };
  // the chunk (16 bytes) that lands in this lane's slot l % 32 of load t, row 8 w + 2 t + l / 32 of the slab
  auto chunk_of = [&](int t, int l) __attribute__((always_inline)) { return (uint32_t)(l & 31) ^ (4 * ((2 * t + (l >> 5)) & 3)) ^ (2 * (w & 1)); };
  // requests the map entries of the eight slabs from row r of the expert's rows
  // (row0 .., n of them) on: this wave's rows 8 w + 2 t + h of slab s to s 8 + h 4 + t
  auto fetch = [&](int32_t row0, int32_t n, int32_t r) __attribute__((always_inline)) {
    const int x = lane();
    const uint32_t o = 4 * (r + BK * (x >> 3) + 8 * w + 2 * (x & 3) + ((x >> 2) & 1));
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);   // (the entries there have been read)
    const uint32_t to = ldsm + ((batch & 1) * 8 + w) * 256;
    if (p.dy_map) load_lds4(rsrc4(p.dy_map + row0, (uint64_t)n * 4), to, o);
    if (p.a_map) load_lds4(rsrc4(p.a_map + row0, (uint64_t)n * 4), to + 4096, o);
    ++batch;
  };
  // a mapped operand's offsets for the next slab
  auto gather = [&](uint32_t (&vo)[4], int op, const uint32_t (&c)[4], uint32_t rows, uint32_t ld) __attribute__((always_inline)) {
    // (the half being read is the one not being filled)
    const u32x4 m = *reinterpret_cast<const u32x4*>(&s_map[op][batch & 1][w][8 * ((lr / BK) & 7) + 4 * (l >> 5)]);
    bool bad = false;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t row = udiv_magic(m[t], p.div, p.magic);
      const bool in = 8 * w + 2 * t + (l >> 5) < left, ok = (int32_t)m[t] >= 0 && row < rows;
      bad |= in && !ok;
      vo[t] = in && ok ? row * ld + c[t] : OOB;
    }
    if (__any(bad) && l == 0) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
  };
  WTile lt{0, 0, 0, 0};              // the tile being loaded
  const bool mapped = p.dy_map || p.a_map;
  auto skip = [&](uint32_t i) __attribute__((always_inline)) {   // the first tile from i on that has rows
    WTile x{0, 0, 0, 0};
    while (i < n_my && (x = tile(i)).rows == 0) ++i;
    ln = i;
    return x;
  };
  // the mapped operands at the next slab; with its first of eight the next
  // eight are requested: this tile's, or the next tile's first
  auto set_rows = [&]() __attribute__((always_inline)) {
    if (((lr / BK) & 7) == 0) {
      if (left > 8 * BK) {
        fetch(lt.row0, lt.rows, lr + 8 * BK);
      } else {
        const uint32_t keep = ln;
        const WTile x = skip(ln);
        fetch(x.row0, x.rows, 0);
        ln = keep;
      }
    }
    if (p.dy_map) gather(vod, 0, cd, (uint32_t)p.dy_rows, ldd);
    if (p.a_map) gather(voa, 1, ca, (uint32_t)p.a_rows, lda);
  };
  // the loads go on with tile ln, passing over those of experts without rows
  auto bind = [&]() __attribute__((always_inline)) {
    const WTile x = lt = skip(ln);
    ++ln;
    lr = 0;
    left = x.rows;
    if (left == 0) {   // (descriptors of nothing: every slab has as many loads)
      rd = rsrc4(p.dy, 0);
      ra = rd;
      return;
    }
    const int l = lane();
    const uint32_t n0 = (uint32_t)(x.at >> 16) * TM, k0 = (uint32_t)(x.at & 0xFFFF) * TN;
    rd = p.dy_map ? rsrc4(p.dy, (uint64_t)p.dy_rows * ldd) : rsrc4(p.dy + (int64_t)x.row0 * p.N, (uint64_t)left * ldd);
    ra = p.a_map ? rsrc4(p.a, (uint64_t)p.a_rows * lda) : rsrc4(p.a + (int64_t)x.row0 * p.K, (uint64_t)left * lda);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t c = chunk_of(t, l), k = 8 * w + 2 * t + (l >> 5);
      cd[t] = n0 + 8 * c < N ? 2 * n0 + 16 * c : OOB;
      ca[t] = k0 + 8 * c < K ? 2 * k0 + 16 * c : OOB;
      vod[t] = k * ldd + cd[t];
      voa[t] = k * lda + ca[t];
    }
  };
  auto step = [&](u32x4& rs, uint32_t ld) __attribute__((always_inline)) {
    const uint64_t base = ((uint64_t)rs[1] << 32 | rs[0]) + BK * ld;
    rs = rsrc4(reinterpret_cast<const void*>(base), (uint64_t)left * ld);
  };
  // the next slab of the stream into a slot of the ring
  auto issue = [&](uint32_t stage) __attribute__((always_inline)) {
    if (left == 0) bind();
    if (mapped && left) set_rows();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      load_lds(rd, lds0 + stage * STAGE + (4 * w + t) * 1024, vod[t], 0);
      load_lds(ra, lds0 + stage * STAGE + HALF + (4 * w + t) * 1024, voa[t], 0);
    }
    lr += BK;
    left = left > BK ? left - BK : 0;
    if (!p.dy_map) step(rd, ldd);
    if (!p.a_map) step(ra, lda);
  };

  // --------------------------------------------------------------- fragments
  // (swizzle and columns as in gemm_bf16.hip's float32 results)
  const uint32_t lb = HALF + (8 * q + (li >> 2)) * 512 + 16 * (16 * wn + (((li & 3) >> 1) ^ (4 * (li >> 2)) ^ (2 * (q & 1)))) + 8 * (li & 1);
  typedef __attribute__((address_space(3))) s16x4* lp;
  auto read_tr = [&](bf16x8& f, uint32_t at) __attribute__((always_inline)) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at + 2048));
    f = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto barrier = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };

  for (uint32_t j0 = 0;; j0 += NT) {
    {
      const uint32_t J = (j0 + tid) * stride + blockIdx.x / 8, c = J / chunk, t = (c * 8 + xcd) * chunk + (J - c * chunk);
      WTile x{0, 0, 0, 0};
      if (t < total) {
        const uint32_t i = t / per_e, r = t - i * per_e;
        x.e = (int32_t)((uint64_t)i * order % (uint32_t)E);
        const uint32_t nt = r / n_kt;
        x.at = (int32_t)(nt << 16 | (r - nt * n_kt));
        x.row0 = s_off[x.e];
        x.rows = s_off[x.e + 1] > x.row0 ? s_off[x.e + 1] - x.row0 : 0;
      }
      s_tile[tid] = x;
      n_my = __syncthreads_count(t < total);
    }
    if (n_my == 0) break;
    ln = 0;
    left = 0;
    if (mapped) {
      const WTile x = skip(0);
      fetch(x.row0, x.rows, 0);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
    issue(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    barrier();
    if (grp) barrier();
    uint32_t gs = 0;       // the slab's place in the ring
    int stored = -1;       // memory operations of the last epilogue, at least (-1: there was none)
    for (uint32_t ct = 0; ct < n_my; ++ct) {
      const WTile m = tile(ct);
      const uint32_t nt = (uint32_t)(m.at >> 16), kt = (uint32_t)(m.at & 0xFFFF), nk = ((uint32_t)m.rows + BK - 1) / BK;
      if (nk == 0 && (p.beta != 0.0f || !p.zero_empty)) continue;
      const uint32_t tn = N - nt * TM < TM ? N - nt * TM : TM;
      const int mb = (int)((tn + 63) / 64);   // blocks of 16 of a wave
      f32x4 acc[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[i][n] = f32x4{};
      uint32_t ao[4];   // and for A's blocks: chunks 2 mb wm + 2 i and + 1 of the row
      {
        const int x = lane() & 15, q = lane() >> 4, j = x >> 2, s = x & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) ao[i] = (8 * q + j) * 512 + 8 * (s & 1) + 16 * ((2 * mb * wm + 2 * i + (s >> 1)) ^ (4 * j) ^ (2 * (q & 1)));
      }
      bf16x8 fa[4], fb[8];
      auto reads = [&](int h) __attribute__((always_inline)) {
        const uint32_t st = gs * STAGE + 16384 * h;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          read_tr(fb[i], (st + lb) ^ (32 * i));
          if (i < 4) read_tr(fa[i], st + ao[i]);
        }
      };
      auto mfmas = [&](bool bar) __attribute__((always_inline)) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (i < mb) {
#pragma unroll
            for (int n = 0; n < (i ? 8 : 4); ++n) acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[i], acc[i][n], 0, 0, 0);
          }
        }
        if (bar) barrier();
#pragma unroll
        for (int n = 4; n < 8; ++n) acc[0][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[0], acc[0][n], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
      };
      for (uint32_t s = 0; s < nk; ++s) {
        reads(0);
        if (stored < 0) {
          issue(1 - gs);
          stored = 0;
        }
        barrier();
        mfmas(true);
        reads(1);
        if (grp) wait_but(stored);
        barrier();
        if (!grp) wait_but(stored);
        stored = -1;
        mfmas(!(grp && s == nk - 1));
        gs = 1 - gs;
      }
      if (nk) {
        issue(1 - gs);
        stored = 8 * mb;
      }
      const int64_t row0 = (int64_t)m.e * p.N + (int64_t)nt * TM;
      const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.dw + row0 * p.K, (uint64_t)tn * K * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < mb) {
          const int li = lane() & 15, q = lane() >> 4;
          const uint32_t r = 16 * mb * wm + 16 * i + li;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const uint32_t k = kt * TN + 128 * wn + 16 * n + 4 * q, o = k < K ? r * K + k : PAST;
            float z[4] = {acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]};
            if (p.beta != 0.0f) {
              float v[4];
              load_f32<4>(rc, o, v);
#pragma unroll
              for (int x = 0; x < 4; ++x) z[x] = v[x] + z[x];
            }
            store_f32<4>(rc, o, z);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (grp && nk) barrier();
    }
    if (!grp) barrier();
    __builtin_amdgcn_s_waitcnt(wait_vm(0));   // (no load into this workgroup's LDS outlives it)
    __syncthreads();
  }
}

// db: 64 columns of one expert per workgroup, eight a thread; thread row y sums
// rows y, y + 128, ... in order, then the 128 sums are added in order.
__global__ void __launch_bounds__(1024) k_bias_grad_bf16(Bf16Wgrad p) {
  __shared__ float s[128][65];
  const int e = blockIdx.y, cx = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t n = (int64_t)blockIdx.x * 64 + 8 * cx;
  int64_t r0 = p.off[e], r1 = p.off[e + 1];
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 < p.M ? r1 : p.M;
  if (r0 >= r1 && (p.beta != 0.0f || !p.zero_empty)) return;
  float v[8] = {};
  if (n < p.N)
    for (int64_t r = r0 + y; r < r1; r += 128) {
      const int64_t rd = mapped_row(p.dy_map, r, p.div, p.magic, p.dy_rows, &g_dev_err);
      if (rd < 0) continue;
      const u32x4 q = *reinterpret_cast<const u32x4*>(p.dy + rd * p.N + n);
      const float sc = row_scale(p.db_scale, p.dy_map, r, p.dy_rows * p.div);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] + sc * bf16_bits_to_f32((i & 1) ? q[i / 2] >> 16 : q[i / 2] & 0xFFFFu);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[y][8 * cx + i] = v[i];
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || c >= p.N) return;
  float t = 0.0f;
  for (int i = 0; i < 128; ++i) t = t + s[i][threadIdx.x];
  float* d = p.db + (int64_t)e * p.N + c;
  *d = p.beta != 0.0f ? *d + t : t;
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
  const int64_t nt = (N + t16::TM - 1) / t16::TM, kt = (K + t16::TN - 1) / t16::TN;
  MOE4_REQUIRE(nt * kt * E < ((int64_t)1 << 31), MOE4_EINVAL, s + ": too large");
  // a step through the experts near the golden section of E, coprime to it
  uint32_t order = (uint32_t)(0.618 * E);
  const auto gcd = [](uint32_t a, uint32_t b) {
    while (b) {
      const uint32_t c = a % b;
      a = b;
      b = c;
    }
    return a;
  };
  while (order < 1 || gcd(order, (uint32_t)E) != 1) ++order;
  hipLaunchKernelGGL(k_bf16_wgrad, dim3((unsigned)tile_grid()), dim3(t16::NT), 0, st, p, (uint32_t)nt, (uint32_t)kt, order);
  if (db) hipLaunchKernelGGL(k_bias_grad_bf16, dim3((unsigned)((N + 63) / 64), (unsigned)E), dim3(1024), 0, st, p);
  return check_launch(s.c_str());
}
