// Weight gradients of the BF16 expert products (gfx950): per expert
// dw = dy^T a over its rows (v_mfma_f32_16x16x32_bf16, float32 accumulation),
// and the column sums of dy for the bias.
#include "bf16_tile.h"

namespace moe4 {

static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_gemm_bf16_wgrad() { return take_device_word(&g_dev_err); }

namespace wg {
constexpr int NT = 256;                   // four waves of 64 x 128, 2 x 2
constexpr int TM = 128, TN = 256, BK = 32;   // tile (of dy's and of a's columns), rows of a slab
constexpr int HALF = BK * TM * 2, STAGE = HALF + BK * TN * 2, NS = 3;   // dy's part of a slab, a slab, the ring's slabs
constexpr int NL = 6;                     // a wave's loads of a slab: two of dy, four of a
constexpr int LIST = 128;                 // tiles listed at a time
constexpr int SLOTS = 512;                // workgroups at a time: two on each of 256 CUs
}  // namespace wg

// Slice i of n rows: whole slabs, as even as they get; rows r .. r + m - 1.
struct Slice {
  int32_t r, m;
  __device__ Slice(int32_t n, int i, int slices) {
    const uint32_t slabs = ((uint32_t)n + wg::BK - 1) / wg::BK, each = slabs / slices, more = slabs - each * slices;
    const uint32_t from = (each * i + ((uint32_t)i < more ? i : more)) * wg::BK, end = from + (each + ((uint32_t)i < more)) * wg::BK;
    r = (int32_t)(from < (uint32_t)n ? from : (uint32_t)n);
    m = (int32_t)(end < (uint32_t)n ? end : (uint32_t)n) - r;
  }
};

// An expert's first row and its rows, from offsets that need not be sound.
__device__ inline int2 expert_rows(const int32_t* off, int e, int64_t M) {
  int32_t r0 = off[e], r1 = off[e + 1];
  r0 = r0 < 0 ? 0 : (r0 < (int32_t)M ? r0 : (int32_t)M);
  r1 = r1 < (int32_t)M ? r1 : (int32_t)M;
  return make_int2(r0, r1 > r0 ? r1 - r0 : 0);
}

// A tile of a slice's sum: n-tile nt (of dy's columns), k-tile kt (of a's; at = nt
// 2^16 + kt), the slice's rows; e: its number, slices e + slice (-1: no tile).
struct WTile {
  int32_t e, at, row0, rows;
};

// The rows are the contraction: a slab is 32 rows of both operands, read
// transposed from LDS.  Two workgroups share a CU, so that one multiplies while
// the other stores: a short contraction (a few hundred rows) writes its float32
// tile in about the time that it takes to multiply.  A map's entries come through
// LDS, those of eight slabs at a time.
// Bound: 512 cycles of MFMA a slab and workgroup, 48 bytes per cycle and CU through
// the load path, and for short contractions the stores.  8192 rows each of 8 experts of
// 4096 x 4096: 1955 us, 1125 TFLOP/s (eight waves on one 256 x 256 tile: 996; torch's
// library product of that kind 1089); 341 rows each of 384 experts of 4096 x 1024:
// 2180 us (multiplication alone 1215; 6.4 GB of results at the rate of a fill 930).  Results
// stored in pieces of 64 bytes took 2820 us there, whole lines from lanes that are
// not consecutive 2550, from consecutive ones 2290, passed on to memory 2080.
// Order: the experts by falling number of rows, their tiles dealt to the workgroups
// from first to last, then from last to first, and so on, so that everyone gets as
// much to multiply; every second workgroup of an XCD (they share a CU) takes its own from
// the end, so that the experts with many rows are multiplied while those with few
// or none are stored.  (16384 tokens, 8 of 384 experts by weights that fall with
// rank, 4096 x 1024: experts visited in mixed order, each on one XCD, 2565 us, by
// falling rows 2076, half of the workgroups from the end 1960; 192 tiles 242 us
// where each CU first gets one, else 259.)
__global__ void __launch_bounds__(wg::NT, 2) k_bf16_wgrad(Bf16Wgrad p, uint32_t n_nt, uint32_t n_kt) {
  using namespace wg;
  using t16::OOB;
  using t16::lds_u8;
  using t16::s16x4;
  using t16::rsrc4;
  using t16::load_lds;
  using t16::load_lds4;
  using t16::wait_vm;
  __shared__ __attribute__((aligned(16))) uint8_t ring[NS * STAGE];
  __shared__ __attribute__((aligned(16))) WTile s_tile[LIST];   // this workgroup's next tiles
  __shared__ __attribute__((aligned(16))) uint32_t s_map[2][2][4][64];   // map entries: operand, half of them, wave, slab and row
  const int tid = threadIdx.x, l = tid & 63, li = l & 15, q = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w >> 1, wn = w & 1;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)ring);
  const uint32_t ldsm = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8)(uint8_t*)s_map);
  const int E = p.E * p.slices;      // (of here on: the slices)
  float* const dw = p.slices > 1 ? p.dw_part : p.dw;
  const float beta = p.slices > 1 ? 0.0f : p.beta;
  const bool zero_empty = p.slices == 1 && p.zero_empty && beta == 0.0f;
  const uint32_t per_e = n_nt * n_kt, total = per_e * E;
  // Neighbours in the order of tiles share operands: they are on one XCD, whose
  // workgroups 2 i and 2 i + 1 share a CU (of a round that is not full each CU first
  // gets one tile).
  const uint32_t G = gridDim.x, xcd = blockIdx.x % 8, slot = blockIdx.x / 8, rounds = (total + G - 1) / G;
  const bool back = slot % 2;
  const uint32_t N = (uint32_t)p.N, K = (uint32_t)p.K, ldd = N * 2, lda = K * 2;
  auto lane = [&]() __attribute__((always_inline)) {   // (kept from the optimiser, as in gemm_bf16.hip)
    int x = l;
    asm volatile("" : "+v"(x));
    return x;
  };

  // ------------------------------------------------------------- load stream
  // It runs two slabs ahead of the multiplication, through the tiles' ends.
  uint32_t ln = 0, n_my = 0;
  int32_t lr = 0, left = 0;          // the next slab's first row in its expert, the expert's rows from there
  u32x4 rd, ra;
  uint32_t vod[2], voa[4], cd[2], ca[4];   // offsets; with a map those of the columns
  uint32_t batch = 0;                // eight slabs' map entries that have been taken up
  auto tile = [&](uint32_t i) __attribute__((always_inline)) {
    const WTile x = s_tile[i];
    return WTile{__builtin_amdgcn_readfirstlane(x.e), __builtin_amdgcn_readfirstlane(x.at), __builtin_amdgcn_readfirstlane(x.row0),
                 __builtin_amdgcn_readfirstlane(x.rows)};
  };
  // Rows 8 w .. 8 w + 7 of a slab are this wave's to load: dy's 8 w + 4 t + l / 16,
  // a's 8 w + 2 t + l / 32; and the chunk (16 bytes) that lands in the lane's slot
  auto row_d = [&](int t, int l) __attribute__((always_inline)) { return 4 * t + (l >> 4); };
  auto row_a = [&](int t, int l) __attribute__((always_inline)) { return 2 * t + (l >> 5); };
  auto chunk_d = [&](int t, int l) __attribute__((always_inline)) { return (uint32_t)(l & 15) ^ (4 * (l >> 4)) ^ (2 * (w & 1)); };
  auto chunk_a = [&](int t, int l) __attribute__((always_inline)) { return (uint32_t)(l & 31) ^ (4 * (row_a(t, l) & 3)) ^ (2 * (w & 1)); };
  // requests the map entries of the eight slabs from row r of the expert's rows
  // (row0 .., n of them) on: this wave's of slab s to 8 s on, in the order in
  // which a lane takes them (dy: row 4 t + g to 2 g + t, a: row 2 t + h to 4 h + t).
  // (The descriptors start at row r: an offset from the slice's first row would
  // pass a descriptor's 2^31 bytes at row 2^29.)
  auto fetch = [&](int32_t row0, int32_t n, int32_t r) __attribute__((always_inline)) {
    const int x = lane();
    const uint32_t o = 4 * (BK * (x >> 3) + 8 * w);
    const int64_t at = (int64_t)row0 + r;
    const uint64_t bytes = (uint64_t)(n - r) * 4;
    __builtin_amdgcn_s_waitcnt(t16::WAIT_LGKM0);   // (the entries there have been read)
    const uint32_t to = ldsm + ((batch & 1) * 4 + w) * 256;
    if (p.dy_map) load_lds4(rsrc4(p.dy_map + at, bytes), to, o + 4 * (4 * (x & 1) + ((x >> 1) & 3)));
    if (p.a_map) load_lds4(rsrc4(p.a_map + at, bytes), to + 2048, o + 4 * (2 * (x & 3) + ((x >> 2) & 1)));
    ++batch;
  };
  // a mapped row's offset; rows that do not exist are noted in bad
  auto gather = [&](uint32_t m, bool in, uint32_t c, uint32_t rows, uint32_t ld, bool& bad) __attribute__((always_inline)) {
    const uint32_t row = udiv_magic(m, p.div, p.magic);
    const bool ok = (int32_t)m >= 0 && row < rows;
    bad |= in && !ok;
    return in && ok ? row * ld + c : OOB;
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
    // (the half being read is the one not being filled)
    const uint32_t at = (batch & 1) * 256 + w * 64 + 8 * ((lr / BK) & 7);
    bool bad = false;
    if (p.dy_map) {
      const u32x2 m = *reinterpret_cast<const u32x2*>(&s_map[0][0][0][0] + at + 2 * q);
#pragma unroll
      for (int t = 0; t < 2; ++t) vod[t] = gather(m[t], 8 * w + row_d(t, l) < left, cd[t], (uint32_t)p.dy_rows, ldd, bad);
    }
    if (p.a_map) {
      const u32x4 m = *reinterpret_cast<const u32x4*>(&s_map[1][0][0][0] + at + 4 * (l >> 5));
#pragma unroll
      for (int t = 0; t < 4; ++t) voa[t] = gather(m[t], 8 * w + row_a(t, l) < left, ca[t], (uint32_t)p.a_rows, lda, bad);
    }
    if (__any(bad) && l == 0) atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
  };
  // the loads go on with tile ln, passing over those of experts without rows
  auto bind = [&]() __attribute__((always_inline)) {
    const WTile x = lt = skip(ln);
    ++ln;
    // (its map entries were requested with the first slab of the tile before: with
    // its only one, they have not been waited for)
    if (mapped && lr <= BK && x.rows) __builtin_amdgcn_s_waitcnt(wait_vm(0));
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
      if (t < 2) {
        const uint32_t c = n0 + 8 * chunk_d(t, l);
        cd[t] = c < N ? 2 * c : OOB;
        vod[t] = (8 * w + row_d(t, l)) * ldd + cd[t];
      }
      const uint32_t c = k0 + 8 * chunk_a(t, l);
      ca[t] = c < K ? 2 * c : OOB;
      voa[t] = (8 * w + row_a(t, l)) * lda + ca[t];
    }
  };
  auto step = [&](u32x4& rs, uint32_t ld) __attribute__((always_inline)) {
    const uint64_t base = ((uint64_t)rs[1] << 32 | rs[0]) + BK * ld;
    rs = rsrc4(reinterpret_cast<const void*>(base), (uint64_t)left * ld);
  };
  // the next slab: its rows, its loads one at a time, and on
  auto ready = [&]() __attribute__((always_inline)) {
    if (left == 0) bind();
    if (mapped && left) set_rows();
  };
  auto load = [&](int t, uint32_t st) __attribute__((always_inline)) {
    if (t < 2) load_lds(rd, lds0 + st + (2 * w + t) * 1024, vod[t & 1], 0);
    else load_lds(ra, lds0 + st + HALF + (4 * w + t - 2) * 1024, voa[(t - 2) & 3], 0);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    lr += BK;
    left = left > BK ? left - BK : 0;
    if (!p.dy_map) step(rd, ldd);
    if (!p.a_map) step(ra, lda);
  };

  // --------------------------------------------------------------- fragments
  // A transposed read takes 4 rows x 32 bytes from each 16 lanes.  The 16-byte
  // chunk c of row r sits at c ^ 4 (r % 4) ^ 2 (r / 8 % 2): 32 lanes hit every bank once.
  const uint32_t sw = (4 * (li >> 2)) ^ (2 * (q & 1)), fr = 8 * q + (li >> 2);
  const uint32_t lb = HALF + fr * 512 + 16 * (16 * wn + (((li & 3) >> 1) ^ sw)) + 8 * (li & 1);
  typedef __attribute__((address_space(3))) s16x4* lp;
  auto read_tr = [&](bf16x8& f, uint32_t at, uint32_t four_rows) __attribute__((always_inline)) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(lds_u8)(ring + at + four_rows));
    f = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  for (uint32_t j0 = 0; j0 < rounds; j0 += LIST) {
    // the slices by falling rows (equal ones, and from 2^20 on, by number): a bitonic
    // sort in the ring, which is free between lists
    {
      uint32_t* key = reinterpret_cast<uint32_t*>(ring);
      auto rows_of = [&](int i) __attribute__((always_inline)) {
        const int e = i / p.slices;
        const int2 m = expert_rows(p.off, e, p.M);
        const Slice s(m.y, i - e * p.slices, p.slices);
        return make_int2(m.x + s.r, s.m);
      };
      int n = 1;
      while (n < E) n *= 2;
      for (int i = tid; i < n; i += NT) {
        const int m = i < E ? rows_of(i).y : 0;
        key[i] = i < E ? (uint32_t)(m < 0xFFFFF ? m : 0xFFFFF) << 12 | (uint32_t)(4095 - i) : 0;
      }
      for (int k = 2; k <= n; k *= 2) {
        for (int j = k / 2; j; j /= 2) {
          __syncthreads();
          for (int x = tid; x < n / 2; x += NT) {
            const int i = 2 * x - (x & (j - 1));   // (the pair's lower index)
            const uint32_t a = key[i], b = key[i + j];
            if ((a < b) == ((i & k) == 0)) {
              key[i] = b;
              key[i + j] = a;
            }
          }
        }
      }
      __syncthreads();
      if (tid < LIST && j0 + tid < rounds) {
        const uint32_t r = back ? rounds - 1 - (j0 + tid) : j0 + tid, n = total - r * G < G ? total - r * G : G;
        const uint32_t share = (n + 7) / 8, at = n == G ? slot : slot / 2 + slot % 2 * (G / 16), y = xcd * share + at;
        WTile x{-1, 0, 0, 0};
        if (at < share && y < n) {
          const uint32_t t = r * G + (r & 1 ? n - 1 - y : y), i = t / per_e, z = t - i * per_e;
          // (bands of four k-tiles, in them the n-tiles one after the other: 8192 rows each
          // for 8 experts of 4096 x 4096 1955 us, whole rows of k-tiles 2040)
          const uint32_t band = z / (4 * n_nt), wide = n_kt - 4 * band < 4 ? n_kt - 4 * band : 4, o = z - band * 4 * n_nt, nt = o / wide;
          x.e = 4095 - (int32_t)(key[i] & 4095);
          x.at = (int32_t)(nt << 16 | (4 * band + o - nt * wide));
          const int2 m = rows_of(x.e);
          x.row0 = m.x;
          x.rows = m.y;
        }
        s_tile[tid] = x;
      }
      __syncthreads();
      n_my = rounds - j0 < LIST ? rounds - j0 : LIST;
    }
    ln = 0;
    left = 0;
    if (mapped) {
      const WTile x = skip(0);
      fetch(x.row0, x.rows, 0);
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
    for (int s = 0; s < 2; ++s) {
      ready();
#pragma unroll
      for (int t = 0; t < NL; ++t) load(t, s * STAGE);
      advance();
    }
    uint32_t gs = 0, st2 = 2 * STAGE;   // the slab's place in the ring, and that of the one two slabs on
    int stored = 0;                     // memory operations of the last epilogue, at least
    for (uint32_t ct = 0; ct < n_my; ++ct) {
      const WTile m = tile(ct);
      const uint32_t nt = (uint32_t)(m.at >> 16), kt = (uint32_t)(m.at & 0xFFFF), nk = ((uint32_t)m.rows + BK - 1) / BK;
      if (nk == 0 && (!zero_empty || m.e < 0)) continue;
      const uint32_t tn = N - nt * TM < TM ? N - nt * TM : TM;
      const int mb = (int)((tn + 31) / 32);   // blocks of 16 of a wave
      f32x4 acc[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[i][n] = f32x4{};
      uint32_t ao[4];   // dy's blocks: chunks 2 mb wm + 2 i and + 1 of the row
      {
        const int x = lane() & 15, q = lane() >> 4, j = x >> 2, s = x & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) ao[i] = (8 * q + j) * 256 + 8 * (s & 1) + 16 * ((2 * mb * wm + 2 * i + (s >> 1)) ^ (4 * j) ^ (2 * (q & 1)));
      }
      for (uint32_t s = 0; s < nk; ++s) {
        // This slab has landed: newer are the next one's loads and, in a tile's
        // first two, the last tile's stores.  Past the barrier so have the other
        // waves' loads, and the slab before has been read.
        __builtin_amdgcn_sched_barrier(0);
        if (s >= 2 || stored < 8) __builtin_amdgcn_s_waitcnt(wait_vm(NL));
        else if (stored >= 32) __builtin_amdgcn_s_waitcnt(wait_vm(NL + 32));
        else if (stored >= 16) __builtin_amdgcn_s_waitcnt(wait_vm(NL + 16));
        else __builtin_amdgcn_s_waitcnt(wait_vm(NL + 8));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        bf16x8 fa[4], fb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          read_tr(fb[i], (gs + lb) ^ (32 * i), 2048);
          if (i < 4) read_tr(fa[i], gs + ao[i], 1024);
        }
        ready();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < mb) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[i], acc[i][n], 0, 0, 0);
            }
          }
          load(i, st2);
          if (i >= 2) load(i + 2, st2);
        }
        __builtin_amdgcn_s_setprio(0);
        advance();
        st2 = gs;
        gs = gs == (NS - 1) * STAGE ? 0 : gs + STAGE;
      }
      if (nk) stored = 8 * mb;
      const int64_t row0 = (int64_t)m.e * p.N + (int64_t)nt * TM;
      const __amdgpu_buffer_rsrc_t rc = make_rsrc(dw + row0 * p.K, (uint64_t)tn * K * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < mb) {
          const int l = lane();
          const uint32_t r = 16 * mb * wm + 16 * i + (l >> 3);
#pragma unroll
          for (int n = 0; n < 8; n += 2) {
            const uint32_t k = kt * TN + 128 * wn + 16 * n + 4 * (l & 7), o = k < K ? r * K + k : PAST, o8 = k < K ? o + 8 * K : PAST;
            float x[4], y[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              x[v] = acc[i][n][v];
              y[v] = acc[i][n + 1][v];
            }
            t16::store_order(x, y, l);
            if (beta != 0.0f) {
              float a[4], b[4];
              load_f32<4>(rc, o, a);
              load_f32<4>(rc, o8, b);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                x[v] = a[v] + x[v];
                y[v] = b[v] + y[v];
              }
            }
            store_f32<4, NT_STORE>(rc, o, x);
            store_f32<4, NT_STORE>(rc, o8, y);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));   // (no load into this workgroup's LDS outlives it)
    __syncthreads();
  }
}

// db: 64 columns of one slice of an expert's rows per workgroup, eight a thread;
// thread row y sums rows y, y + 128, ... in order, then the 128 sums are added in
// order.  Bound: the read of dy; 16384 x 1536, 19 slices: 10 us, 4.9 TB/s (one: 55).
__global__ void __launch_bounds__(1024) k_bias_grad_bf16(Bf16Wgrad p) {
  __shared__ float s[128][65];
  const int e = blockIdx.y / p.db_slices, i = blockIdx.y - e * p.db_slices, cx = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t n = (int64_t)blockIdx.x * 64 + 8 * cx;
  const int2 m = expert_rows(p.off, e, p.M);
  const Slice sl(m.y, i, p.db_slices);
  const int64_t r0 = m.x + (int64_t)sl.r, r1 = r0 + sl.m;
  const bool part = p.db_slices > 1;
  if (sl.m == 0 && (part || p.beta != 0.0f || !p.zero_empty)) return;
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
  float* d = part ? p.db_part + (int64_t)blockIdx.y * p.N + c : p.db + (int64_t)e * p.N + c;
  *d = !part && p.beta != 0.0f ? *d + t : t;
}

// The slices' sums [E, slices, L] joined in their order: dst [E, L] (L % 4 == 0).
// Bound: its bytes; two slices of 1536 x 4096 in 15 us, 5.1 TB/s.
__global__ void __launch_bounds__(256) k_wgrad_join(Bf16Wgrad p, const float* part, int slices, float* dst, int64_t L) {
  const int e = blockIdx.y;
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  const int32_t n = expert_rows(p.off, e, p.M).y;
  if (i >= L || (n == 0 && (p.beta != 0.0f || !p.zero_empty))) return;
  f32x4* d = reinterpret_cast<f32x4*>(dst + e * L + i);
  const f32x4* s = reinterpret_cast<const f32x4*>(part + (int64_t)e * slices * L + i);
  f32x4 t = {};
#pragma unroll 4
  for (int k = 0; k < slices; ++k) {
    const f32x4 x = s[k * (L / 4)];   // (an empty slice's is not written, and not used)
    if (Slice(n, k, slices).m) t = t + x;
  }
  *d = p.beta != 0.0f ? *d + t : t;
}

}  // namespace moe4

using namespace moe4;

// Slices of each expert's rows, for tiles (items) that are fewer than the workgroups
// at a time: where the estimate is least, in 25 ns: a slab's share, a launch to join, for
// each slice its turn there and the bytes of its sums, twice.
// 16384 rows of 1536 x 4096, 192 tiles: one slice 327 us, two 229 us with the join (five,
// two tiles a workgroup: 240).  In all, at one slice per 256 rows / as chosen: 60000
// rows of 128 x 256 (32 slices) 52 / 42 us, 8 x 2048 rows of 512 x 512 (8) 40 / 33.
static int wgrad_slices(int64_t items, int32_t E, int64_t M, int64_t slab, int64_t sums) {
  const int64_t slabs = (M / E + wg::BK - 1) / wg::BK, most = wg::SLOTS / items < 128 ? wg::SLOTS / items : 128;
  int64_t least = slab * slabs;
  int best = 1;
  for (int64_t n = 2; n <= most && n <= slabs; ++n) {
    const int64_t t = slab * ((slabs + n - 1) / n) + 320 + 10 * n + n * E * sums / 15625;
    if (t < least) {
      least = t;
      best = (int)n;
    }
  }
  return best;
}
static int dw_slices(int32_t E, int64_t M, int64_t N, int64_t K) {
  return wgrad_slices((N + wg::TM - 1) / wg::TM * ((K + wg::TN - 1) / wg::TN) * E, E, M, 36, N * K);
}
static int db_slices(int32_t E, int64_t M, int64_t N) { return wgrad_slices((N + 63) / 64 * E, E, M, 9, N); }
static size_t dw_part_bytes(int32_t E, int64_t M, int64_t N, int64_t K) {
  const int n = dw_slices(E, M, N, K);
  return n > 1 ? (size_t)n * E * N * K * 4 : 0;
}

static bool wgrad_shape(int32_t E, int64_t M, int64_t N, int64_t K) {
  return E >= 1 && E <= 2048 && M >= 0 && N > 0 && K > 0 && N % 8 == 0 && K % 8 == 0;
}
static bool wgrad_fits(int64_t M, int64_t N, int64_t K) {
  return M < ((int64_t)1 << 31) && N < ((int64_t)1 << 20) && K < ((int64_t)1 << 20) && N * K < ((int64_t)1 << 29);
}

extern "C" size_t moe_grouped_gemm_bf16_wgrad_ws_bytes(int32_t E, int64_t M_total, int64_t N, int64_t K) {
  if (!wgrad_shape(E, M_total, N, K) || !wgrad_fits(M_total, N, K)) return 0;   // (the call refuses these)
  const int n = db_slices(E, M_total, N);
  return dw_part_bytes(E, M_total, N, K) + (n > 1 ? (size_t)n * E * N * 4 : 0);
}

extern "C" int moe_grouped_gemm_bf16_wgrad(const uint16_t* dy, int64_t dy_rows, const int32_t* dy_map, const uint16_t* a, int64_t a_rows,
                                           const int32_t* a_map, int32_t map_div, const int32_t* expert_off, int32_t E, int64_t M_total,
                                           int64_t N, int64_t K, float* dw, float beta, int flags, const float* db_scale, float* db,
                                           void* ws, size_t ws_bytes, void* stream) {
  const std::string s("moe_grouped_gemm_bf16_wgrad");
  MOE4_REQUIRE(wgrad_shape(E, M_total, N, K), MOE4_EINVAL,
               s + ": need 1 <= E <= 2048 and widths that are multiples of 8");
  MOE4_REQUIRE(wgrad_fits(M_total, N, K) && dy_rows >= 0 && a_rows >= 0 && dy_rows < ((int64_t)1 << 31) && a_rows < ((int64_t)1 << 31),
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
  const size_t need = moe_grouped_gemm_bf16_wgrad_ws_bytes(E, M_total, N, K), dw_bytes = dw_part_bytes(E, M_total, N, K);
  MOE4_REQUIRE(need == 0 || (ws && ws_bytes >= need), MOE4_EWORKSPACE, s + ": workspace of moe_grouped_gemm_bf16_wgrad_ws_bytes() bytes required");
  MOE4_REQUIRE(need == 0 || aligned16(ws), MOE4_EALIGN, s + ": ws must be 16-byte aligned");
  const uint32_t magic = map_div <= 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / (uint32_t)map_div);
  const Bf16Wgrad p{dy, a, dy_map, a_map, expert_off, db_scale, dw, db, dy_rows, a_rows, M_total, N, K, (uint32_t)map_div, magic, E, beta,
                    (flags & MOE4_WGRAD_SKIP_EMPTY) == 0, dw_slices(E, M_total, N, K), db_slices(E, M_total, N), static_cast<float*>(ws),
                    reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + dw_bytes)};
  hipStream_t st = as_stream(stream);
  const int64_t nt = (N + wg::TM - 1) / wg::TM, kt = (K + wg::TN - 1) / wg::TN;
  MOE4_REQUIRE(nt * kt * E < ((int64_t)1 << 31), MOE4_EINVAL, s + ": too large");
  hipLaunchKernelGGL(k_bf16_wgrad, dim3(2 * (unsigned)tile_grid()), dim3(wg::NT), 0, st, p, (uint32_t)nt, (uint32_t)kt);
  const auto join = [&](const float* part, int slices, float* dst, int64_t L) {
    if (slices > 1) hipLaunchKernelGGL(k_wgrad_join, dim3((unsigned)((L + 1023) / 1024), (unsigned)E), dim3(256), 0, st, p, part, slices, dst, L);
  };
  join(p.dw_part, p.slices, dw, N * K);
  if (db) {
    hipLaunchKernelGGL(k_bias_grad_bf16, dim3((unsigned)((N + 63) / 64), (unsigned)(E * p.db_slices)), dim3(1024), 0, st, p);
    join(p.db_part, p.db_slices, db, N);
  }
  return check_launch(s.c_str());
}
