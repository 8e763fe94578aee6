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
// Every kernel reads the logits once, a row per wave, and is bound by that
// read.  The sums over tokens are made in a fixed order (no floating-point
// atomics): workgroup c sums the tokens of chunk c, and flushes a partial row
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
constexpr int PER = MAXE / 64;          // logits per lane at the most
constexpr int NW = 4, THREADS = 64 * NW;
constexpr int CH = 64;                  // tokens per chunk
constexpr int SUM_T = 1024;
}  // namespace bl

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = v + __shfl_xor(v, o, 64);
  return v;
}

// Row r of z in registers (expert l + 64 i in register i), turned into its
// softmax; the experts past E, and every expert of a row of -infinities, are 0.
__device__ inline void softmax_row(const float* __restrict__ logits, const float* __restrict__ bias, int64_t t, int E,
                                   float (&p)[bl::PER]) {
  const int l = threadIdx.x & 63;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < bl::PER; ++i) {
    const int e = l + 64 * i;
    p[i] = -INFINITY;
    if (e < E) {
      p[i] = logits[t * E + e];
      if (bias) p[i] = p[i] + bias[e];
    }
    m = fmaxf(m, p[i]);
  }
  m = wave_max(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < bl::PER; ++i) {
    p[i] = m == -INFINITY ? 0.0f : expf(p[i] - m);
    s = s + p[i];
  }
  s = wave_sum(s);
  const float r = s > 0.0f ? 1.0f / s : s;  // (a NaN stays one)
#pragma unroll
  for (int i = 0; i < bl::PER; ++i) p[i] = p[i] * r;
}

// Segment bounds; without offsets one segment of all T tokens.
__device__ inline int64_t seg_at(const int32_t* __restrict__ off, int s, int64_t T) {
  const int64_t v = off ? (int64_t)off[s] : (s ? T : 0);
  return v < 0 ? 0 : (v > T ? T : v);
}

// The first segment that ends past token t (n_seg if none).
__device__ inline int seg_of(const int32_t* __restrict__ off, int n_seg, int64_t t, int64_t T) {
  int lo = 0, hi = n_seg;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seg_at(off, mid + 1, T) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(bl::THREADS)
    k_balance_part(const float* __restrict__ logits, const float* __restrict__ bias, const int32_t* __restrict__ idx,
                   const uint8_t* __restrict__ mask, const int32_t* __restrict__ seg_off, int n_seg, int64_t T, int E,
                   int k, float* __restrict__ psum, int32_t* __restrict__ pcnt, int32_t* __restrict__ ptok) {
  using namespace bl;
  __shared__ float lp[NW][MAXE];
  __shared__ int lc[MAXE];
  __shared__ int lt[NW];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t c = blockIdx.x, t0 = c * CH, t1 = t0 + CH < T ? t0 + CH : T;
  for (int s = seg_of(seg_off, n_seg, t0, T); s < n_seg; ++s) {
    const int64_t sa = seg_at(seg_off, s, T), sb = seg_at(seg_off, s + 1, T);
    if (sa >= t1) break;
    const int64_t a = sa > t0 ? sa : t0, b = sb < t1 ? sb : t1;
    if (b <= a) continue;  // (uniform over the workgroup)
    for (int e = tid; e < E; e += THREADS) lc[e] = 0;
    __syncthreads();
    float acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
    int n = 0;
    for (int64_t t = a + w; t < b; t += NW) {
      if (mask && !mask[t]) continue;
      ++n;
      float p[PER];
      softmax_row(logits, bias, t, E, p);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = acc[i] + p[i];
      if (l < k) {
        int e = idx[t * k + l];
        if (e < 0 || e >= E) {
          atomicOr(&g_dev_err, MOE4_DEVERR_INDEX);
          e = e < 0 ? 0 : E - 1;
        }
        atomicAdd(&lc[e], 1);
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l + 64 * i < E) lp[w][l + 64 * i] = acc[i];
    if (l == 0) lt[w] = n;
    __syncthreads();
    const int64_t row = c + s;
    for (int e = tid; e < E; e += THREADS) {
      psum[row * E + e] = ((lp[0][e] + lp[1][e]) + lp[2][e]) + lp[3][e];
      pcnt[row * E + e] = lc[e];
    }
    if (tid == 0) ptok[row] = lt[0] + lt[1] + lt[2] + lt[3];
    __syncthreads();
  }
}

// One workgroup per segment: its partial rows in order.
__global__ void __launch_bounds__(bl::SUM_T)
    k_balance_sum(const float* __restrict__ psum, const int32_t* __restrict__ pcnt, const int32_t* __restrict__ ptok,
                  const int32_t* __restrict__ seg_off, int64_t T, int E, int k, float* __restrict__ loss,
                  int32_t* __restrict__ counts, int32_t* __restrict__ tokens, float* __restrict__ probs) {
  using namespace bl;
  __shared__ float lf[SUM_T / 64];
  __shared__ float lp[SUM_T];
  __shared__ int lc[SUM_T];
  __shared__ int ln;
  const int tid = threadIdx.x;
  const int s = blockIdx.x;
  const int64_t a = seg_at(seg_off, s, T), b = seg_at(seg_off, s + 1, T);
  const int64_t c0 = a / CH, c1 = b > a ? (b - 1) / CH + 1 : c0;
  // the experts side by side, the partial rows dealt over the rest of the
  // workgroup: G shares of rows g, g + G, ..., joined in order
  const int EW = (E + 63) / 64 * 64, G = SUM_T / EW, g = tid / EW, e = tid % EW;
  if (tid == 0) ln = 0;
  float ps = 0.0f;
  int cn = 0;
  if (g < G && e < E)
    for (int64_t c = c0 + g; c < c1; c += G) {
      ps = ps + psum[(c + s) * E + e];
      cn += pcnt[(c + s) * E + e];
    }
  lp[tid] = ps;
  lc[tid] = cn;
  __syncthreads();
  int n = 0;
  for (int64_t c = c0 + tid; c < c1; c += SUM_T) n += ptok[c + s];
  if (n) atomicAdd(&ln, n);
  if (g == 0 && e < E)
    for (int i = 1; i < G; ++i) {
      ps = ps + lp[i * EW + e];
      cn += lc[i * EW + e];
    }
  __syncthreads();
  n = ln;
  const float mean = n > 0 ? ps / (float)n : 0.0f;
  float v = 0.0f;
  if (g == 0 && e < E) {
    if (counts) counts[(int64_t)s * E + e] = cn;
    if (probs) probs[(int64_t)s * E + e] = mean;
    v = (float)cn * mean;
  }
  v = wave_sum(v);
  if ((tid & 63) == 0) lf[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    float f = 0.0f;
    for (int i = 0; i < SUM_T / 64; ++i) f = f + lf[i];
    loss[s] = n > 0 ? f * ((float)E / ((float)k * (float)n)) : 0.0f;
    tokens[s] = n;
  }
}

// One wave per token.
__global__ void __launch_bounds__(bl::THREADS)
    k_balance_bwd(const float* __restrict__ dloss, const float* __restrict__ logits, const float* __restrict__ bias,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                  const uint8_t* __restrict__ mask, const int32_t* __restrict__ seg_off, int n_seg, int64_t T, int E,
                  int k, const float* base, float* out) {  // base may be out
  using namespace bl;
  const int64_t t = (int64_t)blockIdx.x * NW + (threadIdx.x >> 6);
  const int l = threadIdx.x & 63;
  if (t >= T) return;
  const int s = seg_of(seg_off, n_seg, t, T);
  const bool live = s < n_seg && t >= seg_at(seg_off, s, T) && (!mask || mask[t]) && tokens[s] > 0;
  float p[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) p[i] = 0.0f;
  if (live) {
    const int32_t* cs = counts + (int64_t)s * E;
    const float n = (float)tokens[s];
    // counts from their mean: the same gradient (sum_e p = 1), without the
    // cancellation of two large numbers when the router is nearly even
    const float cm = (float)k * n / (float)E;
    const float f = dloss[s] * ((float)E / ((float)k * n)) / n;
    softmax_row(logits, bias, t, E, p);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l + 64 * i < E) d = d + p[i] * ((float)cs[l + 64 * i] - cm);
    d = wave_sum(d);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (l + 64 * i < E) p[i] = f * p[i] * (((float)cs[l + 64 * i] - cm) - d);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = l + 64 * i;
    if (e < E) out[t * E + e] = base ? base[t * E + e] + p[i] : p[i];
  }
}

// Workspace: partial rows (ceil(T / CH) + n_seg of them): E float32 sums, E
// counts, one token count.
struct BlLayout {
  int64_t rows, off_cnt, off_tok, bytes;
};
inline BlLayout bl_layout(int64_t T, int E, int n_seg) {
  BlLayout L;
  L.rows = (T + bl::CH - 1) / bl::CH + n_seg;
  L.off_cnt = (L.rows * E * 4 + 255) / 256 * 256;
  L.off_tok = 2 * L.off_cnt;
  L.bytes = L.off_tok + L.rows * 4;
  return L;
}

}  // namespace moe4

using namespace moe4;

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
  MOE4_REQUIRE(T * (int64_t)k < ((int64_t)1 << 31), MOE4_EINVAL, "moe_balance_loss: T * k must be below 2^31");
  MOE4_REQUIRE(n_seg >= 1 && (seg_off || n_seg == 1), MOE4_EINVAL, "moe_balance_loss: n_seg >= 1, with seg_off unless it is 1");
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
  const hipStream_t st = as_stream(stream);
  if (T > 0)
    hipLaunchKernelGGL(k_balance_part, dim3((unsigned)((T + bl::CH - 1) / bl::CH)), dim3(bl::THREADS), 0, st, logits, bias,
                       topk_idx, token_mask, seg_off, n_seg, T, E, k, psum, pcnt, ptok);
  hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)n_seg), dim3(bl::SUM_T), 0, st, psum, pcnt, ptok, seg_off, T, E, k,
                     loss, counts, tokens, probs);
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
  MOE4_REQUIRE(T < ((int64_t)1 << 31), MOE4_EINVAL, "moe_balance_loss_backward: T must be below 2^31");
  MOE4_REQUIRE(dloss && counts && tokens && (T == 0 || (logits && dlogits)), MOE4_EINVAL,
               "moe_balance_loss_backward: NULL pointer");
  if (T == 0) return MOE4_OK;
  hipLaunchKernelGGL(k_balance_bwd, dim3((unsigned)((T + bl::NW - 1) / bl::NW)), dim3(bl::THREADS), 0, as_stream(stream),
                     dloss, logits, bias, counts, tokens, token_mask, seg_off, n_seg, T, E, k, dlogits_in, dlogits);
  return check_launch("moe_balance_loss_backward");
}
