// Expert-grouped BF16 products with their epilogues (gfx950): forward with
// bias, activation and residual, the gated block, and their input gradients.
// v_mfma_f32_16x16x32_bf16, float32 accumulation, each result rounded once.
#include "bf16_tile.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16() { return take_device_word(&g_dev_err); }

namespace t16 {
constexpr int GM = 4;            // m-tiles of a group (see tile order)
}  // namespace t16

// A tile: rows row0 .. row0 + rows - 1 of expert e, n-tile nt.
struct Tile {
  int e;
  int32_t row0, rows;
  uint32_t nt;
};

// The tiled products: tiles of 256 rows of one expert x 256 columns by eight waves
// of 64 x 128, whose sums fill half of the registers.  A slab of 64 values of K
// (whole 128-byte lines) is 64 KB, two of them a ring in LDS that direct loads fill
// through the tiles' ends; FWD and GATED have K contiguous in both operands, DGRAD
// and GDGRAD read w transposed from LDS.  Workgroups stay, one per CU, and find
// their tiles from the offsets on the device.  Tiles of few rows issue no MFMAs for the
// missing blocks of 16.
// Bound: a slab is 2048 cycles of MFMA per SIMD; the LDS gives its fragments (192 KB)
// and takes the next one in about 1500, so the reads of one half of the waves run
// under the MFMAs of the other half, and loads go between MFMAs (eight at once took
// a turn of 1250 cycles, not 780).  16384 x 4096 from 4096: 438 us, 1254 TFLOP/s
// (zeros: 363; torch's library product 399), its input gradient in float32 459 us
// (449); 131072 gated rows of eight experts (1024 from 4096) 1286 TFLOP/s, of 384 even ones
// with 256 rows 1047, with 341 (a second tile of 85 costs four fifths of a full one)
// 766; some 10 rows each, uneven: the weights at 4.7 TB/s.
// cap: log2 of a tile's most rows
template <int MODE, bool OUT_BF16>
__global__ void __launch_bounds__(t16::NT, 1) k_bf16_tile(Bf16Args p, int cap, uint32_t n_nt) {
  using namespace t16;
  constexpr bool TR = MODE == DGRAD || MODE == GDGRAD;   // w's columns are the product's: read transposed
  constexpr int NW = MODE == GATED ? TN / 2 : TN;        // the tile's columns
  // Column of block n, lane quarter q, value v of a wave's 128: with float32
  // results 16 n + 4 q + v, with bf16 ones 32 (n / 2) + 8 q + 4 (n % 2) + v: four
  // lanes have 64 consecutive bytes of a row either way (see store_order).
  constexpr bool PAIR = OUT_BF16;
  __shared__ __attribute__((aligned(16))) uint8_t ring[RING];
  __shared__ __attribute__((aligned(16))) Tile s_tile[NT];   // this workgroup's next tiles
  __shared__ int32_t s_off[MAX_E + 1];                   // the experts' first rows, clamped
  __shared__ uint32_t s_first[MAX_E + 1];                // and first m-tiles
  __shared__ int32_t s_map[8 * 64];                      // the next tile's map entries, 32 of each wave
  __shared__ uint32_t s_scan[8];
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w >> 1, wn = w & 1, grp = w >> 2;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)ring);
  const uint32_t ldsm = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)(uint8_t*)(s_map + 64 * w));

  // the experts' first m-tiles: thread t counts experts t P .. t P + P - 1
  const int E = p.E;
  const int32_t M = (int32_t)p.M;
  for (int e = tid; e <= E; e += NT) {
    const int32_t o = p.off[e];
    s_off[e] = o < 0 ? 0 : (o < M ? o : M);
  }
  __syncthreads();
  auto tiles_of = [&](int e) __attribute__((always_inline)) {
    const int32_t n = s_off[e + 1] - s_off[e];
    return n > 0 ? ((uint32_t)n + (1u << cap) - 1) >> cap : 0u;
  };
  {
    const int P = (E + NT - 1) / NT;
    uint32_t mine = 0;
    for (int e = tid * P; e < (tid + 1) * P && e < E; ++e) mine += tiles_of(e);
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
      run += tiles_of(e);
    }
    if (tid == NT - 1) s_first[E] = run;   // (threads past E hold the total too)
    __syncthreads();
  }
  // Tile order: groups of GM m-tiles, in a group the m-tiles fastest, so that
  // the 32 workgroups of an XCD work on GM row blocks and the column blocks of
  // one or two experts at a time.  The XCDs take chunks of tiles in turn: whole
  // groups where there are enough of them, else single tiles or a few.
  const uint32_t n_mt = __builtin_amdgcn_readfirstlane(s_first[E]), total = n_mt * n_nt, gsz = GM * n_nt;
  const uint32_t xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const uint32_t chunk = total >= 16 * gsz ? gsz : (total + gridDim.x - 1) / gridDim.x;

  // The lane number, kept from the optimiser: what a tile's start and end make
  // of it would be hoisted out of the tile loop and fill the registers that the
  // contraction needs.
  auto lane = [&]() __attribute__((always_inline)) {
    int x = l;
    asm volatile("" : "+v"(x));
    return x;
  };

  const uint32_t K = (uint32_t)p.K, N = (uint32_t)p.N, KB = K * 2, nk = (K + BK - 1) / BK;
  const uint32_t ldb = TR ? N * 2 : KB;                     // bytes of a row of w

  // ------------------------------------------------------------- load stream
  // It runs two slabs ahead; the map entries of the tile after the one being
  // loaded are fetched a tile ahead.  Past the last tile it goes on with
  // descriptors of nothing, so that every slab has as many loads.
  uint32_t ln = 0, n_my = 0, ls = 0;   // the next tile to load, this batch's tiles, slab
  u32x4 ra, rb;
  uint32_t voa[4], vob[4];
  // the chunk (16 bytes) that lands in this lane's slot: load t of A has rows 32 w
  // + 8 t + l / 8, slot l % 8; so has B, or with TR k rows 8 w + 2 t + l / 32, slot l % 32
  auto ca = [&](int t, int l) __attribute__((always_inline)) { return (uint32_t)(l & 7) ^ (4 * (t & 1) + (l >> 4)); };
  auto cb = [&](int t, int l) __attribute__((always_inline)) {
    if (TR) return (uint32_t)(l & 31) ^ (4 * ((2 * t + (l >> 5)) & 3)) ^ (PAIR ? 0 : 2 * (w & 1));
    return (uint32_t)(l & 7) ^ (PAIR ? 2 * (t & 3) + ((l >> 4) & 1) : 4 * (t & 1) + (l >> 4));
  };
  auto tile = [&](uint32_t i) __attribute__((always_inline)) {
    const Tile x = s_tile[i];
    return Tile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.row0), __builtin_amdgcn_readfirstlane(x.rows),
                (uint32_t)__builtin_amdgcn_readfirstlane((int)x.nt)};
  };
  auto fetch_map = [&](uint32_t i) __attribute__((always_inline)) {
    if (!p.map || i >= n_my) return;
    const Tile x = tile(i);
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);   // (the entries there have been read)
    load_lds4(rsrc4(p.map + x.row0, (uint64_t)x.rows * 4), ldsm, 4 * (16 * ((x.rows + 63) / 64) * (w >> 1) + 32 * (w & 1) + lane()));
  };
  // the loads go on with tile ln (its map entries have landed: they are older
  // than a slab that has been waited for, unless tiles have but one)
  auto bind = [&]() __attribute__((always_inline)) {
    ls = 0;
    if (p.map && nk == 1) __builtin_amdgcn_s_waitcnt(wait_vm(0));
    if (ln >= n_my) {
      ra = rsrc4(p.a, 0);
      rb = ra;
      return;
    }
    const Tile m = tile(ln);
    const int l = lane(), mb = (m.rows + 63) / 64;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // row x of a wave row's 64 in LDS is row 16 mb wm + x of the tile
      const int x = 32 * (w & 1) + 8 * t + (l >> 3), r = 16 * mb * (w >> 1) + x;
      uint32_t row = (uint32_t)r;
      bool ok = x < 16 * mb && r < m.rows;
      if (p.map && ok) {
        const int32_t i = s_map[64 * w + 8 * t + (l >> 3)];
        row = udiv_magic((uint32_t)i, p.div, p.magic);
        ok = i >= 0 && row < (uint32_t)p.a_rows;
        if (!ok) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
      }
      voa[t] = ok ? row * KB + 16 * ca(t, l) : OOB;
    }
    ra = rsrc4(p.map ? p.a : p.a + (int64_t)m.row0 * p.K, (uint64_t)(p.map ? p.a_rows : m.rows) * KB);
    const uint32_t n0 = m.nt * NW;
    if (TR) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t k = 8 * w + 2 * t + (l >> 5), c = cb(t, l);
        vob[t] = n0 + 8 * c < N ? k * ldb + 16 * c : OOB;
      }
      rb = rsrc4(p.w + (int64_t)m.e * p.K * p.N + n0, (uint64_t)(K * (uint64_t)N - n0) * 2);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t R = 32 * w + 8 * t + (l >> 3);       // GATED: 64 gate and 64 up columns for each wave column
        const uint32_t n = MODE == GATED ? n0 + 64 * (R >> 7) + (R & 63) : n0 + R;
        const uint32_t row = MODE == GATED ? ((R >> 6) & 1) * N + n : n;
        vob[t] = n < N ? row * KB + 16 * cb(t, l) : OOB;
      }
      rb = rsrc4(p.w + (MODE == GATED ? 2 : 1) * (int64_t)m.e * p.N * p.K, (uint64_t)(MODE == GATED ? 2 : 1) * N * KB);
    }
    if (K < BK) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (ca(t, l) >= K / 8) voa[t] = OOB;
        if (!TR && cb(t, l) >= K / 8) vob[t] = OOB;
      }
    }
    ++ln;
    fetch_map(ln);
  };
  // this wave's loads of a slab, four of each operand.  (Their offsets stay in
  // registers of their own: one that is written again for the next load waits
  // until the load before has left for the memory pipeline, and the MFMAs behind
  // it wait too.)
  auto load_a = [&](int t, uint32_t stage) __attribute__((always_inline)) {
    load_lds(ra, lds0 + stage * STAGE + (4 * w + t) * 1024, voa[t], ls * (BK * 2));
  };
  auto load_b = [&](int t, uint32_t stage) __attribute__((always_inline)) {
    load_lds(rb, lds0 + stage * STAGE + HALF + (4 * w + t) * 1024, vob[t], TR ? 0 : ls * (BK * 2));
  };
  // the next slab of the tile: B's k rows by the descriptor; before a last slab
  // that ends inside it, the chunks past K drop out
  auto advance = [&]() __attribute__((always_inline)) {
    ++ls;
    if (TR) {
      const uint64_t base = ((uint64_t)rb[1] << 32 | rb[0]) + BK * ldb;
      const uint32_t left = rb[2] > BK * ldb ? rb[2] - BK * ldb : 0;
      rb = rsrc4(reinterpret_cast<const void*>(base), left);
    }
    if (8 * ls + 8 > K / 8 && 8 * ls < K / 8) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (8 * ls + ca(t, l) >= K / 8) voa[t] = OOB;
        if (!TR && 8 * ls + cb(t, l) >= K / 8) vob[t] = OOB;
      }
    }
  };

  // --------------------------------------------------------------- fragments
  // Swizzles (through the chunk that each lane loads): a row's 16-byte chunk c
  // sits at c ^ x(row) such that the 16 lanes (transposed reads of 32 bytes a row:
  // 32 lanes) of a fragment read hit different banks.
  uint32_t lb[4];    // lane offsets of B's fragments: !TR one for each half of the slab, TR PAIR for each pair of blocks, TR one
  uint32_t la[2];    // A: for each half of the slab
  if (TR) {
    const int j = li >> 2, s = li & 3;
    if (PAIR) {
#pragma unroll
      for (int pb = 0; pb < 4; ++pb) lb[pb] = HALF + (8 * q + j) * 512 + 16 * (16 * wn + 4 * (pb ^ j) + s);
    } else {
      lb[0] = HALF + (8 * q + j) * 512 + 16 * (16 * wn + ((s >> 1) ^ (4 * j) ^ (2 * (q & 1)))) + 8 * (s & 1);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) lb[h] = HALF + (128 * wn + (PAIR ? 8 * (li >> 2) + (li & 3) : li)) * 128 + 16 * ((4 * h + q) ^ (li >> 1));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) la[h] = (64 * wm + li) * 128 + 16 * ((4 * h + q) ^ (li >> 1));
  auto frag_a = [&](bf16x8& f, int i, int h, uint32_t st) __attribute__((always_inline)) {
    f = *reinterpret_cast<const bf16x8*>(ring + st + la[h] + 2048 * i);
  };
  auto frag_b = [&](bf16x8& f, int i, int h, uint32_t st) __attribute__((always_inline)) {
    if (TR) {
      typedef __attribute__((address_space(3))) s16x4* lp;
      const uint32_t at = PAIR ? st + lb[i >> 1] + 8 * (i & 1) : (st + lb[0]) ^ (32 * i);
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at + 16384 * h));
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at + 16384 * h + 2048));
      f = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      f = *reinterpret_cast<const bf16x8*>(ring + st + lb[h] + (PAIR ? 4096 * (i >> 1) + 512 * (i & 1) : 2048 * i));
    }
  };
  auto barrier = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };

  // -------------------------------------------------------- batches of tiles
  for (uint32_t j0 = 0;; j0 += NT) {
    {
      const uint32_t J = (j0 + tid) * stride + blockIdx.x / 8, c = J / chunk, t = (c * 8 + xcd) * chunk + (J - c * chunk);
      Tile x{0, 0, 0, 0};
      if (t < total) {
        const uint32_t g = t / gsz, r = t - g * gsz, gm = n_mt - g * GM < GM ? n_mt - g * GM : GM;
        x.nt = r / gm;
        const uint32_t mi = g * GM + (r - x.nt * gm);
        // the last expert e with s_first[e] <= mi (experts without tiles share their successor's)
        int lo = 0, hi = E;
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (s_first[mid] <= mi) lo = mid;
          else hi = mid;
        }
        x.e = lo;
        x.row0 = s_off[lo] + (int32_t)((mi - s_first[lo]) << cap);
        const int32_t n = s_off[lo + 1] - x.row0;
        x.rows = n < (1 << cap) ? n : 1 << cap;
      }
      s_tile[tid] = x;
      n_my = __syncthreads_count(t < total);
    }
    if (n_my == 0) break;
    ln = 0;
    fetch_map(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    for (int s = 0; s < 2; ++s) {   // slabs 0 and 1
      if (s == 0 || ls == nk) bind();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        load_a(t, s);
        load_b(t, s);
      }
      advance();
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(8));
    barrier();
    // The two groups of waves take turns: one runs the MFMAs of half a slab
    // while the other reads its fragments of the next half, a barrier between
    // the turns; group 1 is a turn behind.  A slab's place in the ring is filled
    // again as it is read to its end: the rows of A that only group 0 reads,
    // by group 0, from its second turn at the MFMAs on, the rest from group 1's
    // second turn on.  The loads go between the MFMAs: eight of them at once
    // keep the memory pipeline busy for as long as a turn lasts, and a reading
    // turn would last longer than the other group's MFMAs.
    if (grp) barrier();
    uint32_t gs = 0;       // the slab's place in the ring
    int stored = 0;        // memory operations of the last epilogue, at least
    for (uint32_t ct = 0; ct < n_my; ++ct) {
      const Tile m = tile(ct);
      const int mb = (m.rows + 63) / 64;   // blocks of 16 rows of a wave
      f32x4 acc[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[i][n] = f32x4{};
      bf16x8 fa[4], fb[8];
      auto reads = [&](int h) __attribute__((always_inline)) {
        const uint32_t st = gs * STAGE;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          frag_b(fb[i], i, h, st);
          if (i < 4) frag_a(fa[i], i, h, st);
        }
      };
      // A turn at the MFMAs, with the loads that `load` makes in its four gaps.
      // Its barrier comes four MFMAs before its end: the other group's first
      // ones then follow without a gap.
      auto mfmas = [&](auto load, auto hand_over) __attribute__((always_inline)) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (i < mb) {
#pragma unroll
            for (int n = 0; n < (i ? 8 : 4); ++n) acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[i], acc[i][n], 0, 0, 0);
          }
          load(3 - i);
        }
        hand_over();
#pragma unroll
        for (int n = 4; n < 8; ++n) acc[0][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[0], acc[0][n], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
      };
      // group 0: B of the next slab, in its first turn; group 1: half its share
      // of it while it reads (both before a tile's results are stored, so in the
      // tile's first slab they have been made)
      auto late = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (!grp || t >= 2) load_b(t, 1 - gs);
        advance();
      };
      for (uint32_t s = 0; s < nk; ++s) {
        reads(0);
        if (grp && s) late();
        barrier();
        mfmas([&](int t) __attribute__((always_inline)) { if (!grp && s) load_b(t, 1 - gs); }, barrier);
        if (!grp && s) advance();
        reads(1);
        if (ls == nk) bind();
        if (grp) wait_but(stored);   // (the next slab; the last tile's results need not have been stored)
        barrier();
        mfmas(
            [&](int t) __attribute__((always_inline)) {
              load_a(t, gs);
              if (grp && t < 2) load_b(t, gs);
            },
            [&]() __attribute__((always_inline)) {
              if (!grp) wait_but(stored + 4);
              // (a tile's last turn: group 1 stores its results before the
              // barrier, while group 0 stores its own behind it)
              if (!(grp && s == nk - 1)) barrier();
            });
        stored = 0;
        gs = 1 - gs;
      }
      late();
      stored = (MODE == GATED ? (p.aux ? 6 : 2) : MODE == GDGRAD || !OUT_BF16 ? 8 : 4) * mb;
      typedef Bf16Epilogue<MODE, OUT_BF16, NT_STORE> Epi;
      const Epi epi(p, m.e, m.row0, m.rows);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < mb) {
          const int l = lane(), r = 16 * mb * wm + 16 * i + (l >> 3);
          auto scale = [&](int r) __attribute__((always_inline)) {
            return (MODE == DGRAD || MODE == GDGRAD) && r < m.rows ? row_scale(p.scale, p.map, (int64_t)m.row0 + r, p.a_rows * p.div) : 1.0f;
          };
          const float s0 = scale(r), s1 = scale(r + 8);
          constexpr int W = PAIR ? 8 : 4, NB = MODE == GATED ? 4 : 8;   // values of a lane, blocks of columns
          const uint32_t n0 = m.nt * NW + (MODE == GATED ? 64 : 128) * wn + W * (l & 7);
          constexpr int GB = 4;                 // (as many are requested at once as registers hold)
#pragma unroll
          for (int g = 0; g < NB; g += GB) {
            typename Epi::template Need<W> need[GB / (W / 2)][2];
            typename Epi::template Bias<W> bias[GB / (W / 2)];
#pragma unroll
            for (int b = g; b < g + GB; b += W / 2) {
              epi.template request<W>(need[(b - g) / (W / 2)][0], r, n0 + 16 * b);
              epi.template request<W>(need[(b - g) / (W / 2)][1], r + 8, n0 + 16 * b);
              epi.template request<W>(bias[(b - g) / (W / 2)], n0 + 16 * b);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = g; b < g + GB; b += W / 2) {
              float x[W], y[W], x1[W], y1[W];
#pragma unroll
              for (int v = 0; v < W; ++v) {
                x[v] = acc[i][b + v / 4][v % 4];
                y[v] = acc[i][b + W / 4 + v / 4][v % 4];
                if (MODE == GATED) {
                  x1[v] = acc[i][(b + 4 + v / 4) % 8][v % 4];
                  y1[v] = acc[i][(b + 4 + W / 4 + v / 4) % 8][v % 4];
                }
              }
              store_order(x, y, l);
              if (MODE == GATED) store_order(x1, y1, l);
              epi.template put<W>(r, n0 + 16 * b, s0, x, x1, need[(b - g) / (W / 2)][0], bias[(b - g) / (W / 2)]);
              __builtin_amdgcn_sched_barrier(0);
              epi.template put<W>(r + 8, n0 + 16 * b, s1, y, y1, need[(b - g) / (W / 2)][1], bias[(b - g) / (W / 2)]);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
      }
      if (grp) barrier();
    }
    if (!grp) barrier();
    __builtin_amdgcn_s_waitcnt(wait_vm(0));   // (no load into this workgroup's LDS outlives it)
    __syncthreads();
  }
}

// ----------------------------------------------------------------- few rows
// With a handful of rows per expert the cost is streaming each active
// expert's weights once, through registers: the weights take the MFMA's M side,
// the rows its N side, 16 at a time.  A workgroup takes 16 WB weight rows of
// one expert (GATED: half of them gate rows, half the up rows of the same
// columns) and up to 64 of its rows; its four waves take every fourth 64 values
// of K (whole lines of a weight row, two steps of 32) and join their sums
// through LDS in wave order.  A wave requests the weights of two such pieces
// ahead of those it multiplies; the rows come from L2.  Bound: HBM.  One token of
// eight gated experts (1024 from 4096), 134 MB: 28 us, 4.8 TB/s (6.2 is the most that
// a plain read reaches here); one row through 4096 x 1536, 12.6 MB: 8 us.
namespace b16r {
constexpr int NWV = 4, NT = 64 * NWV, PASSES = 4, TR = 16 * PASSES, NU = 2;
}

// Grid: n_nt weight-row blocks x (slots for the experts' first TR rows, then
// slots for the rest).  first: the number of those slots: E (slot = expert) or,
// with fewer rows than experts, M (slot = number among the experts with rows).
template <int MODE, bool OUT_BF16, int WB>
__global__ void __launch_bounds__(b16r::NT) k_bf16_rows(Bf16Args p, uint32_t n_nt, int64_t first) {
  using namespace b16r;
  constexpr int HB = MODE == GATED ? WB / 2 : WB;   // blocks of output columns
  __shared__ f32x4 red[NWV][WB][64];
  const int64_t slot = blockIdx.x / n_nt;
  int e = (int)slot;
  int64_t mt = 0;
  if (slot >= first) {
    if (!nth_item(p.off, p.E, slot - first, [](int m) { return (int64_t)(m > TR ? (m - 1) / TR : 0); }, e, mt)) return;
    ++mt;
  } else if (first < p.E) {
    if (!nth_item(p.off, p.E, slot, [](int m) { return (int64_t)(m > 0); }, e, mt)) return;
  }
  const uint32_t N = (uint32_t)p.N, K = (uint32_t)p.K, KB = K * 2, n0 = (blockIdx.x % n_nt) * 16 * HB;
  const int64_t r0 = (int64_t)p.off[e] + mt * TR, re = (int64_t)p.off[e + 1] < p.M ? (int64_t)p.off[e + 1] : p.M;
  if (r0 < 0 || r0 >= re) return;
  const int rows = re - r0 < TR ? (int)(re - r0) : TR;
  const int l = threadIdx.x & 63, li = l & 15, q = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int np = (rows + 15) / 16;
  const int nw = MODE == GATED ? 2 : 1;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (int64_t)e * nw * p.N * p.K, (uint64_t)nw * N * KB);
  const __amdgpu_buffer_rsrc_t ra = p.map ? make_rsrc(p.a, (uint64_t)p.a_rows * KB) : make_rsrc(p.a + r0 * p.K, (uint64_t)rows * KB);
  uint32_t wo[WB], ao[PASSES];
#pragma unroll
  for (int b = 0; b < WB; ++b) {
    const uint32_t n = n0 + 16 * (b % HB) + li;
    wo[b] = n < N ? (n + (b / HB) * N) * KB + 16 * q : t16::OOB;
  }
#pragma unroll
  for (int s = 0; s < PASSES; ++s) {
    const int r = 16 * s + li;
    ao[s] = t16::OOB;
    if (r < rows) {
      const int64_t row = p.map ? mapped_row(p.map, r0 + r, p.div, p.magic, p.a_rows, &g_dev_err) : r;
      if (row >= 0) ao[s] = (uint32_t)row * KB + 16 * q;
    }
  }
  // step h (32 values) of this wave's piece i: K chunk 8 (4 i + w) + 4 h + q
  auto at = [&](uint32_t o, uint32_t i, int h) { return 8 * (NWV * i + w) + 4 * h + q < K / 8 ? o + 128 * (NWV * i + w) + 64 * h : t16::OOB; };
  const uint32_t np64 = (K + 63) / 64, mine = np64 > (uint32_t)w ? (np64 - w + NWV - 1) / NWV : 0;
  u32x4 wq[2][NU][2][WB];
  f32x4 acc[PASSES][WB];
#pragma unroll
  for (int s = 0; s < PASSES; ++s)
#pragma unroll
    for (int b = 0; b < WB; ++b) acc[s][b] = f32x4{};
  auto weights = [&](u32x4 (&x)[NU][2][WB], uint32_t i) {   // (pieces past the wave's share: zeros)
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < WB; ++b) x[u][h][b] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, at(wo[b], i + u, h), 0, 0));
  };
  auto multiply = [&](u32x4 (&x)[NU][2][WB], uint32_t i) {
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
      if (s < np) {
        u32x4 a[NU][2];
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) a[u][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, at(ao[s], i + u, h), 0, 0));
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < WB; ++b)
              acc[s][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][h][b]), __builtin_bit_cast(bf16x8, a[u][h]), acc[s][b], 0, 0, 0);
      }
    }
  };
  weights(wq[0], 0);
  for (uint32_t i = 0; i < mine; i += 2 * NU) {
    weights(wq[1], i + NU);
    multiply(wq[0], i);
    weights(wq[0], i + 2 * NU);
    multiply(wq[1], i + NU);
  }
  typedef Bf16Epilogue<MODE, OUT_BF16, 0> Epi;
  const Epi epi(p, e, r0, rows);
#pragma unroll
  for (int s = 0; s < PASSES; ++s) {
    if (s < np) {
      if (s) __syncthreads();   // (the last pass's sums have been read)
#pragma unroll
      for (int b = 0; b < WB; ++b) red[w][b][l] = acc[s][b];
      __syncthreads();
      // wave b joins column block b: lane (li, q) holds row li of the pass, four consecutive columns
      for (int b = w; b < HB; b += NWV) {
        const f32x4 x = ((red[0][b][l] + red[1][b][l]) + red[2][b][l]) + red[3][b][l];
        const f32x4 y = MODE == GATED ? ((red[0][b + HB][l] + red[1][b + HB][l]) + red[2][b + HB][l]) + red[3][b + HB][l] : x;
        const float z[4] = {x[0], x[1], x[2], x[3]}, z1[4] = {y[0], y[1], y[2], y[3]};
        const uint32_t n = n0 + 16 * b + 4 * q;
        typename Epi::template Need<4> need;
        typename Epi::template Bias<4> bias;
        epi.template request<4>(need, 16 * s + li, n);
        epi.template request<4>(bias, n);
        epi.template put<4>(16 * s + li, n, 1.0f, z, z1, need, bias);
      }
    }
  }
}

int tile_grid() {
  static int n[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (n[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    n[dev] = v < 8 ? 8 : v / 8 * 8;
  }
  return n[dev];
}

// Whether a forward product goes to the few-rows kernel: where the tiles of the
// experts that can have rows are fewer than the CUs, the tiled kernel leaves CUs idle and
// pays a ring's start for each; but the few-rows kernel multiplies a quarter as
// fast, so only up to 16 rows times tile columns a CU.  Both, few rows / tiled in
// us (weights from memory, launches in one graph), by tiles as counted below:
//   16   one of 4096 x 1536, 1 and 256 rows             7.8 / 35.4, 23.6 / 34.6
//    6   one of 1536 x 4096, 128 rows                   27.0 / 73.8
//   12   one of 1536 x 4096 (gated), 128 rows           29.8 / 74.9
//   32   4 of 1024 x 512 (gated), 128 rows each         12.2 / 14.9; 200 (past the bound) 23.8 / 15.8
//  128   8 of 4096 x 4096, 32 rows each                 66.3 / 89.2; 64 and 128 (past it) 79.5 / 92.5, 145 / 96
//  256   16 of 4096 x 1024, 8 and 16 rows each          29.8 / 33.1, 31.6 / 33.1
//   64 to 512   1, 2, 3, 4 and 8 tokens of 8 of 384 experts of 1024 x 4096 (gated)
//               30.6 / 65.6, 55.7 / 86.5, 78.8 / 91.0, 103 / 102, 198 / 187
// With more tiles the two are alike for even loads (384 experts of 4096 x 1024, 8
// rows each 584 / 656, 16 rows 665 / 676) and the tiled one far ahead for uneven ones
// (8 and 16 rows on average, weights falling by rank: 236 / 168, 369 / 209).
static bool few_rows(const Bf16Args& p, int64_t n_nt, int cus) {
  return n_nt * (p.M < p.E ? p.M : p.E) < cus && p.M * n_nt <= 16 * cus;
}

template <int MODE, bool OUT_BF16, int WB>
static int launch_rows(const Bf16Args& p, hipStream_t stream, const char* name) {
  using namespace b16r;
  constexpr int HB = MODE == GATED ? WB / 2 : WB;
  const int64_t first = p.M < p.E ? p.M : p.E, nt = (p.N + 16 * HB - 1) / (16 * HB), slots = first + p.M / TR;
  MOE4_REQUIRE(grid_fits(nt * slots, NT), MOE4_EINVAL, std::string(name) + ": too large");
  hipLaunchKernelGGL((k_bf16_rows<MODE, OUT_BF16, WB>), dim3((unsigned)(nt * slots)), dim3(NT), 0, stream, p, (uint32_t)nt, first);
  return check_launch(name);
}

// log2 of a tile's most rows: 256, or 128 or 64 where few tiles leave CUs idle.  A slab
// of a tile with b blocks of 64 rows takes about 28 + 9 b; the rounds of tiles are
// those of even loads.  Input gradients, 256 rows / as chosen: 512 rows 4096 -> 1536 (64)
// 92.1 / 68.1 us, 8 x 500 rows 2048 -> 1024 (64) 51.6 / 39.4, 8 x 200 rows 2048 -> 4096
// (128) 54.1 / 47.0, 4096 rows 4096 -> 1536 (128) 95.5 / 76.8.
static int tile_rows(const Bf16Args& p, int64_t n_nt, int cus) {
  const int64_t e = p.M < p.E ? p.M : p.E, m = (p.M + e - 1) / e;
  int best = 8;
  int64_t least = 0;
  for (int cap = 8; cap >= 6; --cap) {
    const int64_t tiles = e * n_nt * ((m + (1 << cap) - 1) >> cap), b = ((m < (1 << cap) ? m : 1 << cap) + 63) / 64;
    const int64_t t = (tiles + cus - 1) / cus * (28 + 9 * b);
    if (cap == 8 || t < least) {
      least = t;
      best = cap;
    }
  }
  return best;
}

template <int MODE, bool OUT_BF16>
static int launch_bf16(const Bf16Args& p, void* stream, const char* name) {
  using namespace t16;
  constexpr int NW = MODE == GATED ? TN / 2 : TN;
  const int64_t nt = (p.N + NW - 1) / NW;
  const int cus = tile_grid();
  if ((MODE == FWD || MODE == GATED) && few_rows(p, nt, cus)) {
    constexpr int RM = MODE == GATED ? GATED : FWD;
    // 64 weight rows a workgroup where two of them come to each CU, else 32: 8
    // experts of 4096 x 4096 with 8 rows (512 workgroups) 45.9 / 58.1 us, one token of
    // 384 gated experts of 1024 x 4096 (256) 36.4 / 27.6 us
    const int64_t wide = (p.N * (MODE == GATED ? 2 : 1) + 63) / 64 * (p.M < p.E ? p.M : p.E);
    return wide >= 2 * cus ? launch_rows<RM, OUT_BF16, 4>(p, as_stream(stream), name) : launch_rows<RM, OUT_BF16, 2>(p, as_stream(stream), name);
  }
  const int cap = tile_rows(p, nt, cus);
  MOE4_REQUIRE(((p.M >> cap) + p.E) * nt < ((int64_t)1 << 31), MOE4_EINVAL, std::string(name) + ": too large");
  hipLaunchKernelGGL((k_bf16_tile<MODE, OUT_BF16>), dim3((unsigned)cus), dim3(NT), 0, as_stream(stream), p, cap, (uint32_t)nt);
  return check_launch(name);
}

// What the four calls check alike.  rows of a: M without a map.
static int check_bf16(const Bf16Args& p, const char* name) {
  const std::string s(name);
  MOE4_REQUIRE(p.E >= 1 && p.E <= 2048 && p.M >= 0 && p.N > 0 && p.K > 0 && p.N % 8 == 0 && p.K % 8 == 0, MOE4_EINVAL,
               s + ": need 1 <= E <= 2048 and widths that are multiples of 8");
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
  MOE4_REQUIRE(pre || M_total == 0 || (act == MOE4_ACT_NONE && !hs), MOE4_EINVAL, "moe_grouped_gemm_bf16_dgrad: an activation or hs needs pre");
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
