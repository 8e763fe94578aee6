// The router's balance loss and its gradient (gfx950).
//
// With z = logits + bias, p[t] = softmax(z[t]) over the E experts, token
// segments s (consecutive token ranges, one loss each) and n_s the segment's
// unmasked tokens:
//   counts[s, e] = the assignments (t, j) of those tokens with topk_idx = e
//   probs[s, e]  = the mean of p[t, e] over them
//   loss[s]      = E / (k n_s) * sum_e counts[s, e] probs[s, e]
// (1 for an even router, E / k for one that sends every token to the same k
// experts with certainty), and, the counts being constants,
//   dz[t, e] = dloss[s] E / (k n_s^2) p[t, e] (c[e] - sum_e' p[t, e'] c[e']).
//
// Every kernel reads the logits once, a row per wave: 25 MB at 16384 x 384, where
// k_balance_part takes 15 us (5 for the bytes; the rest is the latency of four
// rows in turn per wave and the exponentials), k_balance_sum 7.6 (a launch and
// a dependent chain over 256 partial rows), k_balance_bwd 17 (75 MB with
// the gradient it adds to: 4.4 TB/s).  The sums over tokens are made in a fixed
// order (no floating-point atomics): workgroup c sums the tokens of chunk c, and flushes a partial row
// at every segment boundary inside it.  The pair (c, s) takes partial row
// c + s: chunk and segment both only grow along the tokens, so the rows are
// distinct and no prefix sum over the segments is needed.
#include "moe4_internal.h"

namespace moe4 {

// This file's device-side error word (moe4_debug_check reads and clears it).
static __device__ uint32_t g_dev_err;
uint32_t take_dev_err_balance() { return take_device_word(&g_dev_err); }

namespace bl {
constexpr int MAXE = 1024, MAXK = 16;
constexpr int NW = 16, THREADS = 64 * NW;  // k_balance_part: waves per chunk
constexpr int CH_MIN = 16, CH_MAX = 64;    // tokens per chunk (bl_chunk)
constexpr int CHUNKS = 256;                // chunks that fill the chip (a constant: the workspace query names no device)
constexpr int SUM_T = 512, SUM_Q = 16;     // k_balance_sum: threads, column quads per workgroup
constexpr int BWD_W = 4;                   // k_balance_bwd: waves (tokens) per workgroup
constexpr int64_t BWD_X = 1 << 22;         // its workgroups along x (2^24 of them would be 2^32 threads)
// tokens: k_balance_part's threads, 16 per token, stay below the 2^32 of a grid dimension
constexpr int64_t MAXT = (1 << 28) - CH_MAX;
}  // namespace bl

__device__ inline float sum_xor16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ inline float sum_xor32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
// The sum over the wave, in every lane (a fixed order, without LDS).
__device__ inline float wave_sum(float v) {
  v = v + lane_xor1(v);
  v = v + lane_xor2(v);
  v = v + __uint_as_float(dpp_u<DPP_HALF_MIRROR>(__float_as_uint(v)));
  v = v + lane_xor8(v);
  v = sum_xor16(v);
  return sum_xor32(v);
}

// Row t of z (expert l + 64 i in register i; -infinity past E).
template <int PER>
__device__ inline void load_row(const float* __restrict__ logits, const float (&b)[PER], int64_t t, int E, float (&z)[PER]) {
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] = l + 64 * i < E ? logits[t * E + l + 64 * i] + b[i] : -INFINITY;
}

// The lane's biases (0 without one: z + 0 is z).
template <int PER>
__device__ inline void load_bias(const float* __restrict__ bias, int E, float (&b)[PER]) {
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = bias && l + 64 * i < E ? bias[l + 64 * i] : 0.0f;
}

// z turned into its softmax (every expert of a row of -infinities is 0).  The
// maximum passes over NaNs, so the zero is each -infinity's own and not the
// row's: a NaN beside -infinities (masked experts, the places past E) stays one
// and makes the sum, and with it the row, NaN.
// exp(d) = 2^(d log2 e): for d <= 0 the product's rounding is as large an error
// as the difference's own, and the hardware's 2^x is good to one unit (results
// below 2^-126 are zeros).
template <int PER>
__device__ inline void softmax_row(float (&z)[PER]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = fmaxf(m, z[i]);
  m = wave_max(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    z[i] = z[i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((z[i] - m) * 1.44269504f);
    s = s + z[i];
  }
  s = wave_sum(s);
  const float r = s > 0.0f ? 1.0f / s : s;  // (a NaN stays one)
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] = z[i] * r;
}

// Segment bounds; without offsets one segment of all T tokens.
__device__ inline int64_t seg_at(const int32_t* __restrict__ off, int s, int64_t T) {
  const int64_t v = off ? (int64_t)off[s] : (s ? T : 0);
  return v < 0 ? 0 : (v > T ? T : v);
}

// The first segment that ends past token t (n_seg if none), t the same in the
// whole wave: the lanes try 64 segments at a time, one load deep per factor of 64.
__device__ inline int seg_of(const int32_t* __restrict__ off, int n_seg, int64_t t, int64_t T) {
  const int l = threadIdx.x & 63;
  int lo = 0, hi = n_seg;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int i = lo + (l + 1) * step - 1;  // the last segment of lane l's stretch
    const unsigned long long past = __ballot(i < hi && seg_at(off, i + 1, T) > t);
    if (past == 0) {  // not in a whole stretch: in the last, shorter one or none
      lo = lo + (hi - lo) / step * step;
      continue;
    }
    const int f = __builtin_ctzll(past);
    hi = lo + (f + 1) * step - 1;
    lo = lo + f * step;
  }
  return lo;
}

// Tokens per chunk: the fewest (16, 32, 64) that do not make more chunks than
// CUs (1000 tokens in 37 sequences, 64 experts: 7 us with 16, 14 with 64; 8192
// tokens, 60 sequences, 256 experts: 11.5 with 32, 17 with 64).
inline int bl_chunk(int64_t T) {
  int ch = bl::CH_MIN;
  while (ch < bl::CH_MAX && (T + ch - 1) / ch > bl::CHUNKS) ch *= 2;
  return ch;
}

// One workgroup per chunk of ch tokens, a token per wave at a time, the next
// token's row in flight during this one's softmax (four waves of sixteen tokens
// each without that: 50 us against 15; more tokens per chunk leave CUs idle,
// fewer make the join longer).  Partial rows have Ep =
// 4 ceil(E / 4) columns (the last ones 0), so that the join reads 16 bytes a
// lane.
template <int PER>
__global__ void __launch_bounds__(bl::THREADS)
    k_balance_part(const float* __restrict__ logits, const float* __restrict__ bias, const int32_t* __restrict__ idx,
                   const uint8_t* __restrict__ mask, const int32_t* __restrict__ seg_off, int n_seg, int64_t T, int E,
                   int Ep, int k, int ch, float* __restrict__ psum, int32_t* __restrict__ pcnt, int32_t* __restrict__ ptok,
                   int32_t* __restrict__ arrived) {
  using namespace bl;
  __shared__ float lp[NW][64 * PER];
  __shared__ int lc[64 * PER];
  __shared__ int lt[NW];
  const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t c = blockIdx.x, t0 = c * ch, t1 = t0 + ch < T ? t0 + ch : T;
  if (c == 0)
    for (int s = tid; s < n_seg; s += THREADS) arrived[s] = 0;
  float bv[PER];
  load_bias<PER>(bias, E, bv);
  for (int s = seg_of(seg_off, n_seg, t0, T); s < n_seg; ++s) {
    const int64_t sa = seg_at(seg_off, s, T), sb = seg_at(seg_off, s + 1, T);
    if (sa >= t1) break;
    const int64_t a = sa > t0 ? sa : t0, b = sb < t1 ? sb : t1;
    if (b <= a) continue;  // (uniform over the workgroup)
    for (int e = tid; e < 64 * PER; e += THREADS) lc[e] = 0;
    __syncthreads();
    float acc[PER], z[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
    int n = 0;
    auto live = [&](int64_t t) { return t < b && (!mask || mask[t]); };
    int64_t t = a + w;
    while (t < b && !live(t)) t += NW;
    if (t < b) load_row<PER>(logits, bv, t, E, z);
    while (t < b) {
      int64_t u = t + NW;
      while (u < b && !live(u)) u += NW;
      float y[PER];
      if (u < b) load_row<PER>(logits, bv, u, E, y);
      ++n;
      if (l < k) {
        int e = idx[t * k + l];
        if (e < 0 || e >= E) {
          atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
          e = e < 0 ? 0 : E - 1;
        }
        atomicAdd(&lc[e], 1);
      }
      softmax_row<PER>(z);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        acc[i] = acc[i] + z[i];
        z[i] = y[i];
      }
      t = u;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) lp[w][l + 64 * i] = acc[i];
    if (l == 0) lt[w] = n;
    __syncthreads();
    const int64_t row = c + s;
    for (int e = tid; e < Ep; e += THREADS) {
      float v = lp[0][e];
#pragma unroll
      for (int i = 1; i < NW; ++i) v = v + lp[i][e];
      psum[row * Ep + e] = v;
      pcnt[row * Ep + e] = lc[e];
    }
    if (tid == 0) {
      int m = 0;
      for (int i = 0; i < NW; ++i) m += lt[i];
      ptok[row] = m;
    }
    __syncthreads();
  }
}

// Workgroup (column block, segment): 64 columns of the segment's partial rows,
// dealt to 32 shares of the workgroup (rows g, g + 32, ... of four columns a
// lane, eight rows in flight), which are joined in order.  The column blocks'
// parts of the loss are summed in order by the segment's last workgroup (its
// arrival count starts at 0, set by k_balance_part).
__global__ void __launch_bounds__(bl::SUM_T)
    k_balance_sum(const float* __restrict__ psum, const int32_t* __restrict__ pcnt, const int32_t* __restrict__ ptok,
                  const int32_t* __restrict__ seg_off, int64_t T, int E, int Ep, int k, int ch, float* __restrict__ loss,
                  int32_t* __restrict__ counts, int32_t* __restrict__ tokens, float* __restrict__ probs,
                  float* __restrict__ ploss, int32_t* __restrict__ arrived) {
  using namespace bl;
  constexpr int G = SUM_T / SUM_Q;
  __shared__ f32x4 lp[SUM_T];
  __shared__ i32x4 lc[SUM_T];
  __shared__ int ln;
  const int tid = threadIdx.x;
  const int s = blockIdx.y, nb = gridDim.x;
  const int64_t a = seg_at(seg_off, s, T), b = seg_at(seg_off, s + 1, T);
  const int64_t c0 = a / ch, c1 = b > a ? (b - 1) / ch + 1 : c0;
  const int Q = Ep / 4, g = tid / SUM_Q, q = blockIdx.x * SUM_Q + tid % SUM_Q;
  if (tid == 0) ln = 0;
  f32x4 ps = {0.0f, 0.0f, 0.0f, 0.0f};
  i32x4 cn = {0, 0, 0, 0};
  if (q < Q) {
    constexpr int U = 8;
    const f32x4* pp = reinterpret_cast<const f32x4*>(psum);
    const i32x4* pc = reinterpret_cast<const i32x4*>(pcnt);
    for (int64_t c = c0 + g; c < c1; c += U * G) {
      f32x4 v[U];
      i32x4 m[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = c + (int64_t)u * G;
        v[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[u] = i32x4{0, 0, 0, 0};
        if (r < c1) {
          v[u] = pp[(r + s) * Q + q];
          m[u] = pc[(r + s) * Q + q];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ps = ps + v[u];
        cn = cn + m[u];
      }
    }
  }
  int n = 0;
  for (int64_t c = c0 + tid; c < c1; c += SUM_T) n += ptok[c + s];
  lp[tid] = ps;
  lc[tid] = cn;
  __syncthreads();
  if (n) atomicAdd(&ln, n);
  if (g == 0)
    for (int i = 1; i < G; ++i) {
      ps = ps + lp[i * SUM_Q + tid];
      cn = cn + lc[i * SUM_Q + tid];
    }
  __syncthreads();
  n = ln;
  float f = 0.0f;
  if (g == 0 && q < Q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * q + i;
      if (e < E) {
        const float mean = n > 0 ? ps[i] / (float)n : 0.0f;
        counts[(int64_t)s * E + e] = cn[i];
        probs[(int64_t)s * E + e] = mean;
        f = f + (float)cn[i] * mean;
      }
    }
  }
  if (tid < 64) {  // (the first wave holds all of g = 0)
    f = wave_sum(f);
    int before = 0;
    if (tid == 0) {  // (the addition releases the store before it)
      __hip_atomic_store(ploss + (int64_t)s * nb + blockIdx.x, f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      before = __hip_atomic_fetch_add(arrived + s, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) == nb - 1) {  // (nb <= 16: a part per lane)
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      const float part = tid < nb ? __hip_atomic_load(ploss + (int64_t)s * nb + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0f;
      f = 0.0f;
      for (int i = 0; i < nb; ++i) f = f + __shfl(part, i, 64);
      if (tid == 0) {
        loss[s] = n > 0 ? f * ((float)E / ((float)k * (float)n)) : 0.0f;
        tokens[s] = n;
      }
    }
  }
}

// One wave per token; past 2^24 tokens the workgroups go on along y.
template <int PER>
__global__ void __launch_bounds__(64 * bl::BWD_W)
    k_balance_bwd(const float* __restrict__ dloss, const float* __restrict__ logits, const float* __restrict__ bias,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                  const uint8_t* __restrict__ mask, const int32_t* __restrict__ seg_off, int n_seg, int64_t T, int E,
                  int k, const float* base, float* out) {  // base may be out
  using namespace bl;
  const int64_t t = ((int64_t)blockIdx.y * BWD_X + blockIdx.x) * BWD_W + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63;
  if (t >= T) return;
  float o[PER], z[PER], bv[PER], c[PER];
  const int s = seg_of(seg_off, n_seg, t, T);
  const bool live = s < n_seg && t >= seg_at(seg_off, s, T) && (!mask || mask[t]);
  int cnt[PER], ns = 0;
  float dl = 0.0f;
  if (live) {  // (every load in flight before the first is used)
    load_bias<PER>(bias, E, bv);
#pragma unroll
    for (int i = 0; i < PER; ++i) cnt[i] = l + 64 * i < E ? counts[(int64_t)s * E + l + 64 * i] : 0;
    ns = tokens[s];
    dl = dloss[s];
    load_row<PER>(logits, bv, t, E, z);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = base && l + 64 * i < E ? base[t * E + l + 64 * i] : 0.0f;
  if (live && ns > 0) {
    const float n = (float)ns;
    // counts from their mean: the same gradient (sum_e p = 1), without the
    // cancellation of two large numbers when the router is nearly even
    const float cm = (float)k * n / (float)E;
    const float f = dl * ((float)E / ((float)k * n)) / n;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l + 64 * i < E ? (float)cnt[i] - cm : 0.0f;
    softmax_row<PER>(z);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) d = d + z[i] * c[i];
    d = wave_sum(d);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] + f * z[i] * (c[i] - d);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (l + 64 * i < E) out[t * E + l + 64 * i] = o[i];
}

// Workspace: partial rows (ceil(T / ch) + n_seg of them): Ep float32 sums, Ep
// counts, one token count; per segment the column blocks' parts of the loss
// and an arrival count.
struct BlLayout {
  int64_t rows, off_cnt, off_tok, off_loss, off_arr, bytes;
};
inline int bl_ep(int E) { return (E + 3) / 4 * 4; }
inline int bl_blocks(int E) { return (E + 4 * bl::SUM_Q - 1) / (4 * bl::SUM_Q); }
inline BlLayout bl_layout(int64_t T, int E, int n_seg) {
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  BlLayout L;
  L.rows = (T + bl_chunk(T) - 1) / bl_chunk(T) + n_seg;
  L.off_cnt = up(L.rows * bl_ep(E) * 4);
  L.off_tok = 2 * L.off_cnt;
  L.off_loss = L.off_tok + up(L.rows * 4);
  L.off_arr = L.off_loss + up((int64_t)n_seg * bl_blocks(E) * 4);
  L.bytes = L.off_arr + (int64_t)n_seg * 4;
  return L;
}

}  // namespace moe4

using namespace moe4;

// The kernel for E experts: PER logits per lane (registers and exponentials
// past the last expert cost as much as real ones)
#define MOE4_BL_PER(LAUNCH)      \
  do {                           \
    if (E <= 64) LAUNCH(1);      \
    else if (E <= 128) LAUNCH(2); \
    else if (E <= 256) LAUNCH(4); \
    else if (E <= 384) LAUNCH(6); \
    else if (E <= 512) LAUNCH(8); \
    else LAUNCH(16);             \
  } while (0)

extern "C" size_t moe_balance_loss_ws_bytes(int64_t T, int32_t E, int32_t n_seg) {
  if (T < 0 || E < 1 || n_seg < 1) return 0;
  return (size_t)bl_layout(T, E, n_seg).bytes;
}

extern "C" int moe_balance_loss(const float* logits, const float* bias, const int32_t* topk_idx,
                                const uint8_t* token_mask, const int32_t* seg_off, int32_t n_seg, int64_t T, int32_t E,
                                int32_t k, float* loss, int32_t* counts, int32_t* tokens, float* probs, void* ws,
                                size_t ws_bytes, void* stream) {
  MOE4_REQUIRE(T >= 0 && E >= 1 && E <= bl::MAXE && k >= 1 && k <= bl::MAXK && k <= E, MOE4_EINVAL,
               "moe_balance_loss: need T >= 0, 1 <= k <= min(E, 16), E <= 1024");
  MOE4_REQUIRE(T <= bl::MAXT && T * (int64_t)k < ((int64_t)1 << 31), MOE4_EINVAL,
               "moe_balance_loss: T must be at most 2^28 - 64 and T * k below 2^31");
  MOE4_REQUIRE(n_seg >= 1 && n_seg <= 65535 && (seg_off || n_seg == 1), MOE4_EINVAL,
               "moe_balance_loss: 1 <= n_seg <= 65535, with seg_off unless it is 1");
  MOE4_REQUIRE(loss && counts && tokens && probs && (T == 0 || (logits && topk_idx)), MOE4_EINVAL,
               "moe_balance_loss: NULL pointer");
  const BlLayout L = bl_layout(T, E, n_seg);
  MOE4_REQUIRE(ws != nullptr && ws_bytes >= (size_t)L.bytes, MOE4_EWORKSPACE,
               "moe_balance_loss: workspace of moe_balance_loss_ws_bytes() bytes required");
  MOE4_REQUIRE(aligned16(ws), MOE4_EALIGN, "moe_balance_loss: ws must be 16-byte aligned");
  char* base = static_cast<char*>(ws);
  float* psum = reinterpret_cast<float*>(base);
  int32_t* pcnt = reinterpret_cast<int32_t*>(base + L.off_cnt);
  int32_t* ptok = reinterpret_cast<int32_t*>(base + L.off_tok);
  float* ploss = reinterpret_cast<float*>(base + L.off_loss);
  int32_t* arrived = reinterpret_cast<int32_t*>(base + L.off_arr);
  const hipStream_t st = as_stream(stream);
  const int Ep = bl_ep(E), ch = bl_chunk(T);
#define MOE4_BL_PART(PER)                                                                                               \
  hipLaunchKernelGGL((k_balance_part<PER>), dim3((unsigned)(T > 0 ? (T + ch - 1) / ch : 1)), dim3(bl::THREADS), 0, \
                     st, logits, bias, topk_idx, token_mask, seg_off, n_seg, T, E, Ep, k, ch, psum, pcnt, ptok, arrived)
  MOE4_BL_PER(MOE4_BL_PART);
#undef MOE4_BL_PART
  hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)bl_blocks(E), (unsigned)n_seg), dim3(bl::SUM_T), 0, st, psum, pcnt, ptok,
                     seg_off, T, E, Ep, k, ch, loss, counts, tokens, probs, ploss, arrived);
  return check_launch("moe_balance_loss");
}

extern "C" int moe_balance_loss_backward(const float* dloss, const float* logits, const float* bias,
                                         const int32_t* counts, const int32_t* tokens, const uint8_t* token_mask,
                                         const int32_t* seg_off, int32_t n_seg, int64_t T, int32_t E, int32_t k,
                                         const float* dlogits_in, float* dlogits, void* stream) {
  MOE4_REQUIRE(T >= 0 && E >= 1 && E <= bl::MAXE && k >= 1 && k <= bl::MAXK && k <= E, MOE4_EINVAL,
               "moe_balance_loss_backward: need T >= 0, 1 <= k <= min(E, 16), E <= 1024");
  MOE4_REQUIRE(n_seg >= 1 && (seg_off || n_seg == 1), MOE4_EINVAL,
               "moe_balance_loss_backward: n_seg >= 1, with seg_off unless it is 1");
  MOE4_REQUIRE(T <= bl::MAXT, MOE4_EINVAL, "moe_balance_loss_backward: T must be at most 2^28 - 64");
  MOE4_REQUIRE(dloss && counts && tokens && (T == 0 || (logits && dlogits)), MOE4_EINVAL,
               "moe_balance_loss_backward: NULL pointer");
  if (T == 0) return MOE4_OK;
  const int64_t wg = (T + bl::BWD_W - 1) / bl::BWD_W, ny = (wg + bl::BWD_X - 1) / bl::BWD_X;
  const dim3 grid((unsigned)(wg < bl::BWD_X ? wg : bl::BWD_X), (unsigned)ny);
#define MOE4_BL_BWD(PER)                                                                                       \
  hipLaunchKernelGGL((k_balance_bwd<PER>), grid, dim3(64 * bl::BWD_W), 0, as_stream(stream), dloss, logits, bias, \
                     counts, tokens, token_mask, seg_off, n_seg, T, E, k, dlogits_in, dlogits)
  MOE4_BL_PER(MOE4_BL_BWD);
#undef MOE4_BL_BWD
  return check_launch("moe_balance_loss_backward");
}
