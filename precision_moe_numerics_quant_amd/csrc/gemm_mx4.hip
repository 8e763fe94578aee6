// Expert-grouped product of MXFP4 operands (gfx950): C[rows of e] = A[rows of
// e] . B[e]^T on the block-scaled FP4 MFMA, whose E8M0 scale per 32 values
// along K is exactly MXFP4's.  Products of two E2M1 values and their power-of-
// two scales are exact; the accumulation is float32.
#include <type_traits>

#include "gemm_common.h"
#include "moe4_internal.h"

namespace moe4 {

constexpr int FP4 = 4;  // the MFMA's operand format code of E2M1

// Raw buffer loads.  An offset of OOB is past every descriptor: 0 comes back.
constexpr uint32_t OOB = 0x80000000u;

// Descriptor of the whole dwords that hold `bytes` bytes from p on (never
// past the page that holds the last of them); ax: bytes ahead of p in it.
__device__ inline __amdgpu_buffer_rsrc_t dword_rsrc(const uint8_t* p, uint64_t bytes, uint32_t& ax) {
  ax = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)reinterpret_cast<uintptr_t>(p) & 3u));
  return make_rsrc(p - ax, bytes ? (bytes + ax + 3) / 4 * 4 : 0);
}

// ----------------------------------------------------------------- few rows
// With a handful of rows per expert the cost is streaming each active
// expert's weights once.  The weights take the MFMA's M side
// (v_mfma_scale_f32_16x16x128_f8f6f4), the expert's rows its N side, 16 at a
// time.  A workgroup takes 16 WB weight rows of one expert and up to 16 PASSES
// of its rows; its four waves split K (so that one token's eight experts
// still fill the chip) and join their sums through LDS in wave order.  A wave
// requests all the weights of its K share at once (NS steps of 128, the
// smallest of 2, 3, 4, 6 and 8 that holds it: up to K = 4096; a smaller NS has
// fewer registers and more waves), keeps them in registers for all its passes,
// and only the rows' codes, from L2, are read per pass.  No LDS for the
// operands.  HBM bounds it: 384 experts of 1536 x 4096 (1.28 GB) with 4 rows each
// in 242 us (5.3 TB/s; reads alone reach 6.2 here), one token's eight experts in
// 8 us, which is latency: a wave's loads, the join, the launch.
namespace m4s {
constexpr int NT = 256, NWV = NT / 64, WB = 2, WROWS = 16 * WB;
constexpr int KB = 128;           // K per step: lane (li, q) holds k = 128 s + 32 q .. of row li
constexpr int PASSES = 4, TR = 16 * PASSES;
}  // namespace m4s

// Grid: n_nt weight-row blocks x (slots for the experts' first TR rows, then
// slots for the rest).  first: the number of those slots: E (slot = expert) or,
// with fewer rows than experts, M_total (slot = number among the experts with
// rows).  ALIGNED: K % 128 == 0 and 4-byte aligned scales, so that a row's
// scales of a step are one dword.
template <bool OUT_BF16, bool ALIGNED, int NS>
__global__ void __launch_bounds__(m4s::NT)
    k_gemm_mx4_rows(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_sf,
                    const uint8_t* __restrict__ b_codes, const uint8_t* __restrict__ b_sf,
                    const int32_t* __restrict__ off, int E, int64_t M_total, int64_t N, int64_t K, uint32_t n_nt,
                    int64_t first, void* __restrict__ c) {
  using namespace m4s;
  __shared__ f32x4 red[NWV][WB][64];
  const int64_t slot = blockIdx.x / n_nt;
  int e = (int)slot;
  int64_t mt = 0;
  if (slot >= first) {
    if (!nth_item(off, E, slot - first, [](int m) { return (int64_t)(m > TR ? (m - 1) / TR : 0); }, e, mt)) return;
    ++mt;
  } else if (first < E) {
    if (!nth_item(off, E, slot, [](int m) { return (int64_t)(m > 0); }, e, mt)) return;
  }
  const int64_t n0 = (int64_t)(blockIdx.x % n_nt) * WROWS;
  const int64_t r0 = (int64_t)off[e] + mt * TR;
  const int64_t re = (int64_t)off[e + 1] < M_total ? (int64_t)off[e + 1] : M_total;
  const int64_t r1 = re < r0 + TR ? re : r0 + TR;
  if (r0 < 0 || r0 >= r1) return;
  const int l = threadIdx.x & 63, li = l & 15, qg = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t KH = (uint32_t)(K / 2), KS = (uint32_t)(K / 32), nst = (KS + 3) / 4;
  const uint32_t spw = (nst + NWV - 1) / NWV;                       // steps per wave
  const uint32_t s0 = spw * w, s1 = s0 + spw < nst ? s0 + spw : nst;
  const int64_t rowb = (int64_t)e * N + n0, nb = N - n0 < WROWS ? N - n0 : WROWS;
  const __amdgpu_buffer_rsrc_t rbc = make_rsrc(b_codes + rowb * KH, (uint64_t)nb * KH);
  const __amdgpu_buffer_rsrc_t rac = make_rsrc(a_codes + r0 * KH, (uint64_t)(r1 - r0) * KH);
  uint32_t ax, bx;
  const __amdgpu_buffer_rsrc_t rbs = dword_rsrc(b_sf + rowb * KS, (uint64_t)nb * KS, bx);
  const __amdgpu_buffer_rsrc_t ras = dword_rsrc(a_sf + r0 * KS, (uint64_t)(r1 - r0) * KS, ax);
  // row r's codes of step s, and its scales: the step's dword (ALIGNED) or
  // this lane's byte.  Steps past the wave's share and chunks past K count as
  // zeros, codes and scale.
  auto codes = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t r, uint32_t s) {
    const uint32_t kb = 4 * s + qg;
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, s < s1 && kb < KS ? r * KH + 16 * kb : OOB, 0, 0));
  };
  // ALIGNED: the dwords of NS steps in one load (they may reach past the
  // wave's share or the row: step_scale drops those)
  constexpr int NY = ALIGNED ? (NS + 3) / 4 * 4 : NS;
  auto scales = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t x, uint32_t r, uint32_t s, uint32_t (&y)[NY]) {
    if (ALIGNED) {
#pragma unroll
      for (int i = 0; i < NY; i += 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, r * KS + 4 * (s + i), 0, 0);
        y[i] = v[0]; y[i + 1] = v[1]; y[i + 2] = v[2]; y[i + 3] = v[3];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const uint32_t kb = 4 * (s + i) + qg;
        y[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, s + i < s1 && kb < KS ? x + r * KS + kb : OOB, 0, 0);
      }
    }
  };
  // (shifted where it is used: at the load it would wait for it)
  auto step_scale = [&](uint32_t y, uint32_t s) { return ALIGNED ? (int)(s < s1 ? y >> (8 * qg) : 0u) : (int)y; };
  i32x4 wq[NS][WB];
  uint32_t wy[WB][NY];
  auto weights = [&](uint32_t sb) {
#pragma unroll
    for (int b = 0; b < WB; ++b) {
      scales(rbs, bx, 16 * b + li, sb, wy[b]);
#pragma unroll
      for (int s = 0; s < NS; ++s) wq[s][b] = codes(rbc, 16 * b + li, sb + s);
    }
  };
  const bool held = spw <= NS;  // one batch of steps: the weights stay for all passes
  if (held) weights(s0);
  for (uint32_t p = 0; r0 + 16 * p < r1; ++p) {
    f32x4 acc[WB];
#pragma unroll
    for (int b = 0; b < WB; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t sb = s0; sb < s1; sb += NS) {
      if (!held) weights(sb);
      i32x4 xq[NS];
      uint32_t xy[NY];
      scales(ras, ax, 16 * p + li, sb, xy);
#pragma unroll
      for (int s = 0; s < NS; ++s) xq[s] = codes(rac, 16 * p + li, sb + s);
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int b = 0; b < WB; ++b)
          acc[b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              __builtin_shufflevector(wq[s][b], wq[s][b], 0, 1, 2, 3, -1, -1, -1, -1),
              __builtin_shufflevector(xq[s], xq[s], 0, 1, 2, 3, -1, -1, -1, -1), acc[b], FP4, FP4, 0,
              step_scale(wy[b][s], sb + s), 0, step_scale(xy[s], sb + s));
    }
    if (p) __syncthreads();  // (the last pass's sums have been read)
#pragma unroll
    for (int b = 0; b < WB; ++b) red[w][b][l] = acc[b];
    __syncthreads();
    // wave b joins block b: lane (li, q) holds row li of the pass and weight
    // rows n0 + 16 b + 4 q .. + 3, four consecutive output columns
    const int64_t row = r0 + 16 * p + li, col = n0 + 16 * w + 4 * qg;
    if (w < WB && row < r1 && col < N) {
      const f32x4 v = ((red[0][w][l] + red[1][w][l]) + red[2][w][l]) + red[3][w][l];
      if (OUT_BF16)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(c) + row * N + col) =
            u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      else
        *reinterpret_cast<f32x4*>(static_cast<float*>(c) + row * N + col) = v;
    }
  }
}

// ---------------------------------------------------------------- many rows
// Persistent and warp-specialised, the structure of this library's other
// grouped GEMMs: four producer waves only issue direct-to-LDS loads of a
// 256-value K slab (128 code bytes and 8 scale bytes of each row) into a ring
// of stages, TN / 32 consumer waves of 64 x 64 only read LDS, run the MFMAs
// (v_mfma_scale_f32_32x32x64_f8f6f4) and store; one barrier per slab.  128 x
// TN tiles.  (Four consumers of 64 x 128 read a quarter less from LDS but leave
// one per SIMD: 260 against 244 us at 4096 rows of 384 experts, N = 4096, K =
// 1536; before the stores were deferred 686 against 680 at 131072 rows of them,
// N = 1536, K = 4096.)
//
// What bounds it, at 131072 rows of eight experts, N = 1536, K = 4096 (502 us,
// 3.3 PFLOP/s): no one unit.  Parts of the kernel timed alone, one run each: the
// MFMAs on random operands 298 us (5.5 PFLOP/s at 1.4 GHz, where power holds the
// clock; on zeros they run at 2.4), with their LDS reads 380, the loads into LDS
// 335, loads and MFMAs 443.  384 experts under power-law routing: 593 us in a
// loop, 655 under the profiler, there at 1.85 GHz with the MFMAs busy 35 % of
// the cycles, the VALU 20 and the LDS 24.  256 x 256 tiles move a third fewer
// bytes per MFMA but leave one wave per SIMD that loads and multiplies: 1006 us.
// Ordinary instead of nontemporal stores: 510.  Float32 results (N = 4096, K =
// 1536, 2.1 GB of them, stored between tiles): 847 us, 581 at the copy rate.
//
// Every load goes through a buffer descriptor that ends with the expert's
// rows, so rows past its last or N and K chunks past K (their lanes' offsets are
// set out of range) arrive as zeros, cost no traffic and no shape needs a kernel
// of its own.
//
// Scales: a wave's load of 64 rows' scales touches 64 cache lines whatever it
// takes from each, as long as four of its whole-row code loads, so the fewest
// such loads win.  PAIR (K % 512 == 0, 16-byte aligned scales): one 16-byte
// load per row brings two slabs' scales, into a ring of their own.  Otherwise
// a 16-byte load per row and slab, from the dword that holds the first of its 8
// scale bytes, and the consumer cuts them out (TN = 128 only: 256 columns with
// a slab's scales in every stage do not fit the LDS).
namespace m4w {
constexpr int TM = 128;
constexpr int BK = 256, ROW_B = BK / 2;  // K values and code bytes of a row and slab
typedef __attribute__((address_space(3))) void* lds_ptr;
// 16-byte chunk c of a row sits at chunk c ^ ((row >> 1) & 7) (the 16 lanes of
// a fragment read hit 16 distinct bank groups); applied through the global
// address that each lane loads
__device__ inline int swz(int row, int c) { return c ^ ((row >> 1) & 7); }
// 16 bytes at each lane's offset + soff into lane-consecutive LDS from p on
__device__ __forceinline__ void load_lds(const __amdgpu_buffer_rsrc_t& rs, uint8_t* p, uint32_t off, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)p, 16, off, soff, 0, 0);
}
// Row R of B's tile in LDS is row n of the tile in memory: the MFMA columns of
// two neighbouring 32-row blocks are even and odd rows of B, so that a lane's
// two values of an output row are neighbours and 32 lanes store whole lines
__device__ inline int bmap(int R) { return (R & ~63) + 2 * (R & 31) + ((R >> 5) & 1); }
// s_waitcnt immediates (vmcnt: bits 3:0 and 15:14; expcnt 6:4; lgkmcnt 11:8)
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
constexpr int WAIT_LGKM0 = 15 | (3 << 14) | (7 << 4);
constexpr int NT_STORE = 2;                // buffer-store cache policy: nontemporal
template <int TN, bool PAIR>
struct Cfg {
  static constexpr int NCW = TN / 32, NT = 64 * (NCW + 4);  // consumer waves of 64 x 64, threads
  static constexpr int CODE_A = TM * ROW_B, CODE_B = TN * ROW_B;
  static constexpr int GRPS = (TM + TN) / 64;            // 64-row scale groups (A's first), a load each
  static constexpr int SCL = GRPS * 64 * 16;
  static constexpr int STAGE = CODE_A + CODE_B + (PAIR ? 0 : SCL);
  static constexpr int S = TN == 128 ? 4 : 3;
  // PAIR: the scales of slabs 2 p and 2 p + 1 in buffer p % NP.  Slab j is
  // requested after the barrier of slab j - S + 1, when slab j - S has been
  // read: pair p + NP (slab 2 p + 2 NP) must come after slab 2 p + 1.
  static constexpr int NP = PAIR ? (S + 2) / 2 : 0;
  static_assert(!PAIR || 2 * NP - S >= 1, "pair ring");
  static constexpr int RING = S * STAGE + NP * SCL;
  static constexpr int IC = 4 + TN / 32;                 // code loads per producer and slab
  static constexpr int NU = (GRPS + 3) / 4;              // scale loads per producer (PAIR: on even slabs)
  static_assert(RING + 16 <= 160 * 1024, "LDS");
};
}  // namespace m4w

template <bool OUT_BF16, int TN, bool PAIR>
__global__ void __launch_bounds__(64 * (TN / 32 + 4), 1)
    k_gemm_mx4_ws(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_sf,
                  const uint8_t* __restrict__ b_codes, const uint8_t* __restrict__ b_sf,
                  const int32_t* __restrict__ off, int E, int64_t M_total, int64_t N, int64_t K, DgSplit sp,
                  void* __restrict__ c) {
  using namespace m4w;
  using C = Cfg<TN, PAIR>;
  constexpr int S = C::S, STAGE = C::STAGE, QB = TN / 32, NCW = C::NCW;
  __shared__ __attribute__((aligned(16))) uint8_t ring[C::RING];
  __shared__ uint32_t s_nmt;
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // total m-tiles (before any load into LDS is in flight)
  if (w == 0) {
    uint32_t n = 0;
    for (int e = l; e < E; e += 64) {
      const int32_t m = off[e + 1] - off[e];
      n += m > 0 ? (uint32_t)((m + TM - 1) / TM) : 0u;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
    if (l == 0) s_nmt = n;
  }
  __syncthreads();
  const uint32_t n_nt = (uint32_t)((N + TN - 1) / TN), n_mt = s_nmt;
  const uint32_t KH = (uint32_t)(K / 2), KS = (uint32_t)(K / 32), nk = (KS + 7) / 8;
  // this workgroup's tiles: q = q0, q0 + stride, ... of its XCD (see DgSplit)
  const uint32_t xcd = blockIdx.x % 8, stride = (gridDim.x - xcd + 7) / 8, q0 = blockIdx.x / 8;
  const uint32_t sm = (8 / sp.xb) * sp.pm, q_end = (n_mt + sm - 1) / sm * (sp.pm * sp.pn);

  if (w >= NCW) {
    // ---- producer pw: 8-row code loads 4 pw .. of A and QB pw .. of B, scale groups NU pw ..
    const int pw = w - NCW;
    __amdgpu_buffer_rsrc_t rac = make_rsrc(a_codes, 0), ras = rac, rbc = rac, rbs = rac;
    uint32_t ax = 0, bx = 0;       // the scale descriptors' bytes ahead of the tile's first
    MtCursor<TM> cur;
    uint32_t pt = q0, ps = 0;
    bool more = false;
    auto seek = [&]() {
      uint32_t mi = 0, nt = 0;
      while (pt < q_end && !sp.tile(xcd, pt, n_mt, n_nt, mi, nt)) pt += stride;
      more = pt < q_end && cur.seek(off, E, mi);
      if (!more) return;
      const int e = cur.e;
      int64_t row0 = (int64_t)ld_const(off, e) + (int64_t)(mi - cur.first) * TM;
      const int64_t n0 = (int64_t)nt * TN;
      const int64_t end = (int64_t)ld_const(off, e + 1) < M_total ? (int64_t)ld_const(off, e + 1) : M_total;
      int64_t ra = end - row0 < TM ? end - row0 : TM;
      if (row0 < 0 || ra <= 0) {  // (offsets outside [0, M]: a row is read, none stored)
        row0 = 0;
        ra = 1;
      }
      const int64_t rb = N - n0 < TN ? N - n0 : TN, rowb = (int64_t)e * N + n0;
      rac = make_rsrc(a_codes + row0 * KH, (uint64_t)ra * KH);
      rbc = make_rsrc(b_codes + rowb * KH, (uint64_t)rb * KH);
      const uint8_t* as = a_sf + row0 * KS;
      const uint8_t* bs = b_sf + rowb * KS;
      ras = dword_rsrc(as, (uint64_t)ra * KS, ax);
      rbs = dword_rsrc(bs, (uint64_t)rb * KS, bx);
      ps = 0;
    };
    seek();
    // each load's offset into its descriptor at K = 0: the same for every tile
    // (the slab's offset goes in the scalar operand)
    uint32_t aoff[4], boff[8], soff[2];
    uint32_t chunk[2];  // the logical chunk of this lane in rows 0-7 and 8-15 of every 16
#pragma unroll
    for (int q = 0; q < 2; ++q) chunk[q] = (uint32_t)swz(8 * q + (l >> 3), l & 7);
#pragma unroll
    for (int q = 0; q < 4; ++q) aoff[q] = (uint32_t)(32 * pw + 8 * q + (l >> 3)) * KH + 16u * chunk[q & 1];
#pragma unroll
    for (int q = 0; q < QB; ++q) boff[q] = (uint32_t)bmap((TN / 4) * pw + 8 * q + (l >> 3)) * KH + 16u * chunk[q & 1];
    auto sgrp = [&](int k) {  // scale group k of this wave (the last one again: every producer issues as many loads)
      const int grp = C::NU * pw + k;
      return grp < C::GRPS ? grp : C::GRPS - 1;
    };
#pragma unroll
    for (int k = 0; k < C::NU; ++k) {
      const int grp = sgrp(k);
      soff[k] = (uint32_t)(grp < TM / 64 ? 64 * grp + l : bmap(64 * grp - TM + l)) * KS;
    }
    auto issue = [&](uint32_t j) {  // slab j of this workgroup
      uint8_t* base = ring + (j % S) * STAGE;
      const uint32_t kb = ps * (uint32_t)ROW_B, left = KS - 8 * ps;  // chunks of the row from this slab on
      // (PAIR: whole slabs only)
      auto at = [&](uint32_t o, int q) { return PAIR || chunk[q & 1] < left ? o : OOB; };
#pragma unroll
      for (int q = 0; q < 4; ++q) load_lds(rac, base + (4 * pw + q) * 1024, at(aoff[q], q), kb);
#pragma unroll
      for (int q = 0; q < QB; ++q) load_lds(rbc, base + C::CODE_A + (QB * pw + q) * 1024, at(boff[q], q), kb);
      if (!PAIR || (ps & 1) == 0) {
        uint8_t* sl = PAIR ? ring + S * STAGE + ((j >> 1) % (PAIR ? C::NP : 1)) * C::SCL : base + C::CODE_A + C::CODE_B;
#pragma unroll
        for (int k = 0; k < C::NU; ++k) {
          const int grp = sgrp(k);
          uint8_t* sb = sl + grp * 1024;
          const bool opa = grp < TM / 64;
          // (PAIR: inside the row.  Otherwise the 16 bytes may reach past the last
          // row: all of the offset in the operand that the range check sees)
          const uint32_t o = PAIR ? soff[k] : (((opa ? ax : bx) + soff[k]) & ~3u) + 8 * ps, so = PAIR ? 8 * ps : 0;
          if (opa) load_lds(ras, sb, o, so);
          else load_lds(rbs, sb, o, so);
        }
      }
      if (++ps == nk) {
        pt += stride;
        seek();
      }
    };
    uint32_t n_iss = 0;
    for (int st = 0; st < S - 1 && more; ++st) issue(n_iss++);
    for (uint32_t gs = 0; gs < n_iss; ++gs) {
      // slab gs landed (the loads of the rem later ones may still be in
      // flight: PAIR has a slab's scale loads on every second one), then the barrier
      const uint32_t rem = n_iss - 1 - gs;
      __builtin_amdgcn_sched_barrier(0);
      if (rem >= 2) __builtin_amdgcn_s_waitcnt(wait_vm(2 * C::IC + (PAIR ? 1 : 2) * C::NU));
      else if (rem == 1 && PAIR && (gs & 1) == 0) __builtin_amdgcn_s_waitcnt(wait_vm(C::IC));
      else if (rem == 1) __builtin_amdgcn_s_waitcnt(wait_vm(C::IC + C::NU));
      else __builtin_amdgcn_s_waitcnt(wait_vm(0));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      if (more) issue(n_iss++);
    }
    __builtin_amdgcn_s_barrier();  // (the consumers' barrier after their last slab)
    return;
  }
  // ---- consumers: wave w owns the 64 x 64 block (w / CWN, w % CWN)
  constexpr int MI = 2, NJ = 2, CWN = TN / 64;
  const int g = (l >> 5) & 1, li = l & 31;
  const int wm = w / CWN * 64, wn = w % CWN * 64;
  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16{};
  uint32_t sha[MI], shb[NJ];  // !PAIR: the rows' first scale byte in its dword
  // A slab is four 64-value k steps.  Lane half g supplies K block 2 ks + g and
  // its scale, byte 2 (ks % 2) of the row's scale dword ks / 2 shifted by g
  // bytes.  With one or two consumer waves per SIMD little else hides the LDS
  // latency, so the next step's fragments are read before the MFMAs of this
  // one, across slabs and tiles too: the last step of a slab runs after the next
  // slab's barrier (its fragments are in registers by then).  After the last
  // slab of all that barrier is an extra one and the reads are of no use.
  i32x4 fa[2][MI], fb[2][NJ];      // the fragments of even and odd steps
  uint32_t ya[MI][2], yb[NJ][2];   // the slab's scales
  // chunk 2 ks + g of a row sits at chunk (g ^ swizzle) ^ 2 ks: one lane offset,
  // its k steps by an XOR (kept opaque: as loop invariants they would fill the
  // registers that the accumulators need)
  uint32_t lx = (uint32_t)li * ROW_B + 16u * (uint32_t)swz(li, g);
  auto frags = [&](uint32_t j, int ks) {
    const uint8_t* st = ring + (j % S) * STAGE;
    const uint32_t o = lx ^ (32u * ks);
    const uint8_t* la = st + wm * ROW_B + o;
    const uint8_t* lb = st + C::CODE_A + wn * ROW_B + o;
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[ks & 1][i] = *reinterpret_cast<const i32x4*>(la + 32 * i * ROW_B);
#pragma unroll
    for (int n = 0; n < NJ; ++n) fb[ks & 1][n] = *reinterpret_cast<const i32x4*>(lb + 32 * n * ROW_B);
  };
  // the raw scales of slab j (row r of A, or TM + row of B), and from those
  // ya, yb; left: scale blocks from the slab on (fewer than 8: the rest 0)
  using Raw = typename std::conditional<PAIR, u32x2, u32x4>::type;
  Raw ra[MI], rb[NJ];
  auto scales = [&](uint32_t j) {
    const uint8_t* sc = PAIR ? ring + S * STAGE + ((j >> 1) % (PAIR ? C::NP : 1)) * C::SCL + 8 * (j & 1)
                             : ring + (j % S) * STAGE + C::CODE_A + C::CODE_B;
    auto get = [&](int r) { return *reinterpret_cast<const Raw*>(sc + r * 16); };
#pragma unroll
    for (int i = 0; i < MI; ++i) ra[i] = get(wm + 32 * i + li);
#pragma unroll
    for (int n = 0; n < NJ; ++n) rb[n] = get(TM + wn + 32 * n + li);
  };
  auto set_scales = [&](uint32_t left) {
    auto put = [&](const Raw& q, uint32_t sh, uint32_t (&y)[2]) {
      uint32_t d0 = q[0], d1 = q[1];
      if (!PAIR) {
        d0 = __builtin_amdgcn_alignbyte(q[1], q[0], sh);
        d1 = __builtin_amdgcn_alignbyte(q[PAIR ? 1 : 2], q[1], sh);
        if (left < 8) {  // (uniform; a slab that ends inside the row's last blocks)
          d0 &= left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
          d1 &= left > 4 ? (1u << (8 * (left - 4))) - 1u : 0u;
        }
      }
      y[0] = d0 >> (8 * g);
      y[1] = d1 >> (8 * g);
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) put(ra[i], sha[i], ya[i]);
#pragma unroll
    for (int n = 0; n < NJ; ++n) put(rb[n], shb[n], yb[n]);
  };
  auto mfmas = [&](int ks) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int n = 0; n < NJ; ++n) {
        const i32x8 xa = __builtin_shufflevector(fa[ks & 1][i], fa[ks & 1][i], 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8 xb = __builtin_shufflevector(fb[ks & 1][n], fb[ks & 1][n], 0, 1, 2, 3, -1, -1, -1, -1);
        // (the byte selector is an immediate)
        if (ks & 1)
          acc[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xa, xb, acc[i][n], FP4, FP4, 2, (int)ya[i][ks >> 1], 2,
                                                                      (int)yb[n][ks >> 1]);
        else
          acc[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xa, xb, acc[i][n], FP4, FP4, 0, (int)ya[i][ks >> 1], 0,
                                                                      (int)yb[n][ks >> 1]);
      }
  };
  auto barrier = [&]() {  // this wave's reads of the slab before are done
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  constexpr int ESZ = OUT_BF16 ? 2 : 4;
  const uint32_t ld = (uint32_t)N * ESZ;  // output row pitch in bytes
  const uint32_t lane_off = (uint32_t)(g * 4) * ld + (uint32_t)li * (2 * ESZ);
  // DEFER (bf16 results, two slabs or more to a tile): a tile's results wait in
  // half its accumulators' registers and are stored between the MFMAs of the
  // next tile's first two slabs, an eighth of them after each MFMA step (1 % at
  // K = 4096, 512 columns and K = 2048 89 - 85 us, 128 columns 44 - 38)
  constexpr bool DEFER = OUT_BF16 && PAIR;
  uint32_t pk[DEFER ? MI : 1][16];
  __amdgpu_buffer_rsrc_t prc = make_rsrc(c, 0);  // (of nothing: the stores go nowhere)
  uint32_t pvo = OOB, pfo = 0;
  auto put_pending = [&](int i, int v) {
    __builtin_amdgcn_raw_buffer_store_b32(pk[DEFER ? i : 0][v], prc, pvo, pfo + (uint32_t)(32 * i + (v >> 2) * 8 + (v & 3)) * ld, NT_STORE);
  };
  auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) put_pending(i, v);
    prc = make_rsrc(c, 0);
  };
  if (DEFER) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) pk[DEFER ? i : 0][v] = 0;
  }
  MtCursor<TM> cur;
  uint32_t gs = 0;
  // one slab of an active tile; pend: the half of the pending stores that goes with it (2: none)
  auto slab = [&](uint32_t s, int pend) {
    asm volatile("" : "+v"(lx));
    auto stores = [&](int ks) {
      if (DEFER && pend < 2) {
#pragma unroll
        for (int v = 0; v < 4; ++v) put_pending(pend, 4 * ks + v);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
      frags(gs, ks + 1);
      __builtin_amdgcn_sched_barrier(0);
      mfmas(ks);
      __builtin_amdgcn_sched_barrier(0);
      stores(ks);
    }
    barrier();
    scales(gs + 1);
    frags(gs + 1, 0);
    __builtin_amdgcn_sched_barrier(0);
    mfmas(3);
    __builtin_amdgcn_sched_barrier(0);
    stores(3);
    set_scales(KS - 8 * (s + 1));  // (after the tile's last slab: set again for the next tile)
    ++gs;
  };
#pragma unroll
  for (int i = 0; i < MI; ++i) sha[i] = 0;
#pragma unroll
  for (int n = 0; n < NJ; ++n) shb[n] = 0;
  barrier();
  scales(0);
  frags(0, 0);
  for (uint32_t q = q0; q < q_end; q += stride) {
    uint32_t mi, nt;
    if (!sp.tile(xcd, q, n_mt, n_nt, mi, nt)) continue;
    if (!cur.seek(off, E, mi)) break;
    const int e = cur.e;
    const int64_t row0 = (int64_t)ld_const(off, e) + (int64_t)(mi - cur.first) * TM, n0 = (int64_t)nt * TN;
    const int64_t row_end = (int64_t)ld_const(off, e + 1) < M_total ? (int64_t)ld_const(off, e + 1) : M_total;
    // waves whose rows or columns all lie past the tile's last skip their MFMAs
    const bool active = row0 >= 0 && row0 + wm < row_end && n0 + wn < N;
    if (!PAIR) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
        sha[i] = (uint32_t)(reinterpret_cast<uintptr_t>(a_sf) + (uint64_t)(row0 + wm + 32 * i + li) * KS) & 3u;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        shb[j] = (uint32_t)(reinterpret_cast<uintptr_t>(b_sf) + (uint64_t)((int64_t)e * N + n0 + bmap(wn + 32 * j + li)) * KS) & 3u;
    }
    if (!active) {
      if (DEFER) flush();
      for (uint32_t s = 0; s < nk; ++s, ++gs) barrier();
      scales(gs);
      frags(gs, 0);
      continue;
    }
    set_scales(KS);
    uint32_t s = 0;
    if (DEFER) {
      slab(0, 0);
      slab(1, 1);
      prc = make_rsrc(c, 0);
      s = 2;
    }
    for (; s < nk; ++s) slab(s, 2);  // (one basic block: the MFMAs stay between their reads)
    // epilogue: straight from the accumulators, a whole 128- or 256-byte row
    // segment from 32 lanes (bmap); the descriptor covers the tile's rows up to
    // the expert's last, so stores of rows past it are dropped
    // (NJ = 2: columns c0 + 2 li and + 1 of the wave's 64, N % 32 == 0: half of
    // them may be past N)
    const int64_t nrows = row_end - row0 < TM ? row_end - row0 : TM, c0 = n0 + wn;
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(static_cast<uint8_t*>(c) + row0 * (int64_t)ld, (uint64_t)nrows * ld);
    const uint32_t vo = c0 + 2 * li < N ? lane_off : OOB, fo = (uint32_t)wm * ld + (uint32_t)c0 * ESZ;
    if (DEFER) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) pk[DEFER ? i : 0][v] = bf16_pair(acc[i][0][v], acc[i][1][v]);
      prc = rC;
      pvo = vo;
      pfo = fo;
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const uint32_t so = fo + (uint32_t)(32 * i + (v >> 2) * 8 + (v & 3)) * ld;
          if (OUT_BF16)
            __builtin_amdgcn_raw_buffer_store_b32(bf16_pair(acc[i][0][v], acc[i][1][v]), rC, vo, so, NT_STORE);
          else
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(acc[i][0][v]), __float_as_uint(acc[i][1][v])}, rC, vo, so, NT_STORE);
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x16{};
  }
  if (DEFER) flush();
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
// workgroups of the tiled kernel (every XCD has one at least)
static int ws_grid() { return cu_count() < 8 ? 8 : cu_count(); }

// Whether a product goes to the few-rows kernel: up to 4 rows per expert on
// average, or up to 32 where the tiled kernel would not have a tile for every
// CU.  N = 1536, K = 4096, few-rows against tiled kernel, even routing | one power-law routing (1.1), in us:
//   384 experts, rows per expert 4: 242 - 286 | 88 - 76;  8: 254 - 284 | 130 - 83;
//   11: 261 - 285 | 163 - 86;  16: 301 - 285 | 210 - 110;  32: 405 - 293 | 363 - 162
//   (a popular expert's weights are read again for every 64 rows, past K = 4096
//   for every 16);
//   8 experts, rows per expert 8, 16, 32: 12 - 19, 12 - 19, 14 - 20
static bool few_rows(int E, int64_t M, int64_t N) {
  const int64_t tiles = ((M < E ? M : E) + M / m4w::TM) * ((N + 255) / 256);
  return M <= 4 * (int64_t)E || (M <= 32 * (int64_t)E && tiles < ws_grid());
}
// its workgroups: blocks of weight rows, and slots (see the kernel)
static int64_t rows_nt(int64_t N) { return (N + m4s::WROWS - 1) / m4s::WROWS; }
static int64_t rows_slots(int E, int64_t M) { return (M < E ? M : E) + M / m4s::TR; }

template <bool OUT_BF16>
static void launch_mx4(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, const int32_t* off, int E,
                       int64_t M, int64_t N, int64_t K, void* c, hipStream_t s) {
  const bool al = K % 128 == 0 && aligned4(as) && aligned4(bs);
  if (few_rows(E, M, N)) {
    const int64_t n_nt = rows_nt(N), first = M < E ? M : E;
    const dim3 rgrid((unsigned)(n_nt * rows_slots(E, M)));
    const int64_t spw = ((K + m4s::KB - 1) / m4s::KB + m4s::NWV - 1) / m4s::NWV;
#define MOE4_MX4S(AL, NS)                                                                                                      \
  hipLaunchKernelGGL((k_gemm_mx4_rows<OUT_BF16, AL, NS>), rgrid, dim3(m4s::NT), 0, s, ac, as, bc, bs, off, E, M, N, K,           \
                     (uint32_t)n_nt, first, c)
#define MOE4_MX4S_AL(NS)            \
  do {                              \
    if (al) MOE4_MX4S(true, NS);    \
    else MOE4_MX4S(false, NS);      \
  } while (0)
    if (spw <= 2) MOE4_MX4S_AL(2);
    else if (spw == 3) MOE4_MX4S_AL(3);
    else if (spw == 4) MOE4_MX4S_AL(4);
    else if (spw <= 6) MOE4_MX4S_AL(6);
    else MOE4_MX4S_AL(8);
#undef MOE4_MX4S_AL
#undef MOE4_MX4S
    return;
  }
  const dim3 grid((unsigned)ws_grid());
  const bool pair = K % 512 == 0 && aligned16(as) && aligned16(bs);
#define MOE4_MX4(TN, AL)                                                                                                       \
  hipLaunchKernelGGL((k_gemm_mx4_ws<OUT_BF16, TN, AL>), grid, dim3(64 * (TN / 32 + 4)), 0, s, ac, as, bc, bs, off, E, M, N, K, \
                     dg_split((N + TN - 1) / TN, m4w::TM, TN), c)
  // 256 columns unless that pads the last tile of a few: us at 131072 rows, 32
  // experts, K = 2048, TN 128 - 256 (before the results waited for the next tile):
  // N = 128 40 - 47, 384 78 - 82, 512 100 - 92, 640 124 - 118, 1536 303 - 262.
  // Without pairs of scales (TN = 128) 334 at N = 1536.
  if (!pair) MOE4_MX4(128, false);
  else if (N % 256 == 0 || N > 512) MOE4_MX4(256, true);
  else MOE4_MX4(128, true);
#undef MOE4_MX4
}

}  // namespace moe4

using namespace moe4;

extern "C" int moe_grouped_gemm_mx4(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* b_codes,
                                    const uint8_t* b_sf, const int32_t* expert_off, int32_t E, int64_t M_total, int64_t N,
                                    int64_t K, void* c, int c_dtype, void* stream) {
  MOE4_REQUIRE(c_dtype == MOE4_F32 || c_dtype == MOE4_BF16, MOE4_EINVAL, "moe_grouped_gemm_mx4: c_dtype must be F32 or BF16");
  MOE4_REQUIRE(E >= 1 && M_total >= 0 && N > 0 && K > 0 && K % 32 == 0 && N % 32 == 0, MOE4_EINVAL,
               "moe_grouped_gemm_mx4: need K % 32 == 0 and N % 32 == 0");
  MOE4_REQUIRE(M_total < ((int64_t)1 << 31) && N < ((int64_t)1 << 22) && K < ((int64_t)1 << 22) && N * K < ((int64_t)1 << 32),
               MOE4_EINVAL, "moe_grouped_gemm_mx4: M must be below 2^31, N and K below 2^22, each expert's B below 2 GiB");
  MOE4_REQUIRE(expert_off && (M_total == 0 || (a_codes && a_sf && b_codes && b_sf && c)), MOE4_EINVAL,
               "moe_grouped_gemm_mx4: NULL pointer");
  MOE4_REQUIRE(aligned16(a_codes) && aligned16(b_codes) && aligned16(c), MOE4_EALIGN,
               "moe_grouped_gemm_mx4: a_codes, b_codes and c must be 16-byte aligned");
  if (M_total == 0) return MOE4_OK;
  // (the tiled kernel's grid is fixed; its tile counts are 32-bit)
  MOE4_REQUIRE(few_rows(E, M_total, N) ? grid_fits(rows_nt(N) * rows_slots(E, M_total), m4s::NT)
                                       : (M_total / m4s::TR + E) * rows_nt(N) < ((int64_t)1 << 31),
               MOE4_EINVAL, "moe_grouped_gemm_mx4: too large");
  if (c_dtype == MOE4_BF16)
    launch_mx4<true>(a_codes, a_sf, b_codes, b_sf, expert_off, E, M_total, N, K, c, as_stream(stream));
  else
    launch_mx4<false>(a_codes, a_sf, b_codes, b_sf, expert_off, E, M_total, N, K, c, as_stream(stream));
  return check_launch("moe_grouped_gemm_mx4");
}
