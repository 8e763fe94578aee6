// Shared by the tiled BF16 expert products (gfx950): the ring in LDS, the direct
// loads and their waits, the order of stores.
#pragma once
#include "bf16_gemm.h"

namespace moe4 {
namespace t16 {

constexpr int NT = 512;                      // eight waves of 64 x 128, 4 x 2
constexpr int TN = 256, BK = 64;             // tile columns, contraction slab
constexpr int HALF = 256 * BK * 2, STAGE = 2 * HALF, RING = 2 * STAGE;   // two slabs
constexpr int MAX_E = 2048;                  // experts (their offsets are kept in LDS)
constexpr uint32_t OOB = 0x80000000u;        // past every descriptor: zeros arrive
typedef __attribute__((address_space(3))) uint8_t* lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// s_waitcnt immediates (vmcnt: bits 3:0 and 15:14; expcnt 6:4; lgkmcnt 11:8)
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
constexpr int WAIT_LGKM0 = 15 | (3 << 14) | (7 << 4);

// Buffer descriptor of a wave-uniform range as four scalar registers.
__device__ __forceinline__ u32x4 rsrc4(const void* p, uint64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t n = bytes > 0x7FFFFFF0ull ? 0x7FFFFFF0u : (uint32_t)bytes;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)n), 0x00020000u};
}

// 16 bytes at each lane's offset + soff into lane-consecutive LDS from `lds` on
// (a byte address in LDS).  Inline assembly because the compiler, which does not
// know that other stages are read meanwhile, would wait for every load in flight
// before each LDS read; it has no output register, and its completion is waited
// for by hand (wait_vm) before the barrier that hands the stage over.
// (M0 is not in the clobber list, which does not take it; nothing else in these
// kernels uses it.  It needs the one wait state.  The scalar registers need five
// behind a vector instruction that writes them, a lane read of a spilled
// descriptor say; the compiler does not see to that here, and three more in each load cost
// 1 to 3 %: the build checks the distance in the code it made, wait_states.py.)
__device__ __forceinline__ void load_lds(const u32x4& rs, uint32_t lds, uint32_t off, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(off), "s"(rs), "s"(soff) : "memory");
}

// 4 bytes at each lane's offset into lane-consecutive LDS
__device__ __forceinline__ void load_lds4(const u32x4& rs, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(rs) : "memory");
}

// Results to store: x and y are two blocks, lane 16 q + i holding W values of row
// i from column W q on.  Afterwards x is row l / 8 and y row 8 + l / 8 of lane l,
// columns W (l % 4) on of the first block for l % 8 < 4, else of the second: a store
// then takes whole lines, eight of 128 bytes, each from consecutive lanes.
// (Figures at the weight gradient.)
template <int W>
__device__ __forceinline__ void store_order(float (&x)[W], float (&y)[W], int l) {
  const bool hi = l & 8;
  const int from = 4 * (16 * (l & 3) + 8 * ((l >> 2) & 1) + (l >> 3));
#pragma unroll
  for (int v = 0; v < W; ++v) {
    const int s = __float_as_int(hi ? x[v] : y[v]);
    const float r = __int_as_float(__builtin_amdgcn_update_dpp(s, s, 0x128, 0xF, 0xF, false));   // (lane i ^ 8's)
    x[v] = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(hi ? r : x[v])));
    y[v] = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(hi ? y[v] : r)));
  }
}

// Waits until all of this wave's memory operations but the `newer` latest have
// completed (fewer may be let through).
__device__ __forceinline__ void wait_but(int newer) {
  __builtin_amdgcn_sched_barrier(0);
  if (newer >= 48) __builtin_amdgcn_s_waitcnt(wait_vm(48));
  else if (newer >= 32) __builtin_amdgcn_s_waitcnt(wait_vm(32));
  else if (newer >= 16) __builtin_amdgcn_s_waitcnt(wait_vm(16));
  else if (newer >= 8) __builtin_amdgcn_s_waitcnt(wait_vm(8));
  else if (newer >= 4) __builtin_amdgcn_s_waitcnt(wait_vm(4));
  else __builtin_amdgcn_s_waitcnt(wait_vm(0));
}

}  // namespace t16

// Workgroups of the persistent kernels: the current device's CUs, a multiple of 8.
int tile_grid();

}  // namespace moe4
