// Log probabilities of given tokens, entropy and the top alternatives of
// logit rows (contract in w4a16sv.h).
//
// For a row x: m = max x, S = sum exp(x - m), W = sum (x - m) exp(x - m);
// ln p(i) = (x_i - m) - ln S, entropy = ln S - W / S. All three sums merge
// over parts of the row (each part against its own maximum, then scaled by
// exp(m_part - m)), so the logits are read once.
//
// token_stats_kernel: a warp takes a window of 1024 logits in registers and
// leaves its (m, S, W) and the maxima of its four 256-logit quarters.
// token_report_kernel, one CTA per row: merges the windows; the `top`-th
// largest quarter maximum is a lower bound of the `top`-th largest logit, so
// only quarters that reach it are read again (at most `top` of them unless
// maxima tie), and the few logits at or above it are ranked in shared memory.
//
// Bound: HBM for the first kernel (one pass, 16-byte loads); the second reads
// about 1.5 % of the row's bytes in statistics and top x 256 logits, mostly
// from L2. Windows start at 16-byte boundaries of memory, not of the row, so
// that rows of any length load 16 bytes at a time.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kLpWindow = 1024;
constexpr int kLpQuarter = 256;
constexpr int kLpStatWarps = 8;
constexpr int kLpRepThreads = 256;
constexpr int kLpCand = 1024;    // logits ranked in shared memory
constexpr float kLpLog2e = 1.4426950408889634f;

struct LogprobParams {
  const void* logits;
  const int32_t* ids;
  int R, V, m, top;
  int windows;  // per row
  float *logp, *entropy;
  int32_t* top_ids;
  float* top_logp;
  float* win;      // [R][windows][4]: m, S, W, unused
  float* quarter;  // [R][windows][4]: maxima
  unsigned* err;
};

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// elements of T before the row's first one back to a 16-byte boundary
template <typename T>
__device__ __forceinline__ int lp_shift(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// the E = 16 / sizeof(T) elements at index e (a multiple of E less the shift)
// of the row as floats, -inf outside [0, V)
template <typename T>
__device__ __forceinline__ void lp_load(const T* row, int e, int V, float* x) {
  constexpr int E = 16 / sizeof(T);
  if (e >= 0 && e + E <= V) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + e));
    if constexpr (sizeof(T) == 4) {
      x[0] = __uint_as_float(w.x);
      x[1] = __uint_as_float(w.y);
      x[2] = __uint_as_float(w.z);
      x[3] = __uint_as_float(w.w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(u[k] << 16);
        x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = e + k >= 0 && e + k < V ? (float)row[e + k] : -INFINITY;
  }
}

// An order of the logits as unsigned integers: rising with the value, the
// two zeros equal, NaN above all.
__device__ __forceinline__ unsigned lp_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const unsigned b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float lp_warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float lp_warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(32 * kLpStatWarps) token_stats_kernel(const LogprobParams p) {
  constexpr int E = 16 / sizeof(T), L = 32 / E;  // loads of E elements a lane
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kLpStatWarps + (threadIdx.x >> 5);
  if (id >= (int64_t)p.R * p.windows) return;
  const int r = (int)(id / p.windows), w = (int)(id % p.windows);
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
  const int e0 = w * kLpWindow - lp_shift(row) + lane * E;
  float x[32];
#pragma unroll
  for (int k = 0; k < L; ++k) lp_load<T>(row, e0 + k * 32 * E, p.V, x + k * E);
  // quarter q: loads q L / 4 .. ; a NaN is carried apart (fmaxf drops it)
  float q[4];
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    q[k] = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[k] = fmaxf(q[k], x[8 * k + j]);
      nan |= x[8 * k + j] != x[8 * k + j];
    }
    q[k] = lp_warp_max(q[k]);
  }
  const float mx = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3]));
  // exp(x - m) = 2^((x - m) log2 e); x - m is exact or rounded once. z is kept
  // off -inf so that a masked logit adds 0 * finite to W.
  float s0 = 0.0f, s1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
  if (mx > -INFINITY || nan) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float z0 = x[j] - mx, z1 = x[j + 1] - mx;
      const float t0 = lp_ex2(z0 * kLpLog2e), t1 = lp_ex2(z1 * kLpLog2e);
      s0 += t0;
      s1 += t1;
      w0 = fmaf(fmaxf(z0, -1e30f), t0, w0);
      w1 = fmaf(fmaxf(z1, -1e30f), t1, w1);
    }
  }
  const float S = lp_warp_sum(s0 + s1), W = lp_warp_sum(w0 + w1);
  // a quarter with a NaN holds the row's largest key
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    bool n = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) n |= x[8 * k + j] != x[8 * k + j];
    if (__any_sync(0xffffffffu, nan) && __any_sync(0xffffffffu, n)) q[k] = NAN;
  }
  if (lane == 0) {
    reinterpret_cast<float4*>(p.win)[id] = make_float4(mx, S, W, 0.0f);
    if (p.top > 0) reinterpret_cast<float4*>(p.quarter)[id] = make_float4(q[0], q[1], q[2], q[3]);
  }
}

// CTA-wide radix selection (8 bits a pass, from the top): the key of the k-th
// largest (k >= 1) of the keys that each(f) hands to f, with at least k of
// them. hist: 256 words; out[0] the key's prefix, out[1] what is left of k.
template <typename Each>
__device__ unsigned lp_select(int k, int* hist, unsigned* out, Each each) {
  unsigned prefix = 0;
  int left = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kLpRepThreads) hist[i] = 0;
    __syncthreads();
    each([&](unsigned key) {
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255u], 1);
    });
    __syncthreads();
    if (threadIdx.x < 32) {  // bins from 255 down, 8 a lane
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = hist[255 - (8 * threadIdx.x + j)];
        sum += c[j];
      }
      int x = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if ((int)threadIdx.x >= d) x += y;
      }
      int before = x - sum;
      if (before < left && left <= x) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < left && left <= before + c[j]) {
            out[0] = prefix | ((unsigned)(255 - (8 * threadIdx.x + j)) << shift);
            out[1] = (unsigned)(left - before);
          }
          before += c[j];
        }
      }
    }
    __syncthreads();
    prefix = out[0];
    left = (int)out[1];
    __syncthreads();
  }
  return prefix;
}

template <typename T>
__global__ void __launch_bounds__(kLpRepThreads) token_report_kernel(const LogprobParams p) {
  __shared__ int hist[256];
  __shared__ unsigned sel[2];
  __shared__ float red[3][kLpRepThreads / 32];
  __shared__ unsigned ckey[kLpCand];
  __shared__ int cidx[kLpCand];
  __shared__ int s_count, s_ties;
  grid_launch_dependents();
  grid_dependency_wait();
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
  const float4* win = reinterpret_cast<const float4*>(p.win) + (int64_t)r * p.windows;
  // ---- the windows merged: every sum against the row's maximum
  float m = -INFINITY;
  for (int w = tid; w < p.windows; w += kLpRepThreads) m = fmaxf(m, __ldcg(&win[w]).x);
  m = lp_warp_max(m);
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kLpRepThreads / 32; ++k) m = fmaxf(m, red[0][k]);
  float S = 0.0f, W = 0.0f;
  for (int w = tid; w < p.windows; w += kLpRepThreads) {
    const float4 v = __ldcg(&win[w]);
    const float d = v.x - m, t = v.x == -INFINITY && v.y == 0.0f ? 0.0f : expf(d);
    S = fmaf(v.y, t, S);
    W += t * fmaf(fmaxf(d, -1e30f), v.y, v.z);
  }
  S = lp_warp_sum(S);
  W = lp_warp_sum(W);
  if (lane == 0) {
    red[1][warp] = S;
    red[2][warp] = W;
  }
  __syncthreads();
  S = W = 0.0f;
#pragma unroll
  for (int k = 0; k < kLpRepThreads / 32; ++k) {
    S += red[1][k];
    W += red[2][k];
  }
  const float ls = S > 0.0f ? logf(S) : NAN;  // -inf alone, or a NaN
  if (tid == 0 && p.entropy) p.entropy[r] = ls - W / S;
  for (int i = tid; i < p.m; i += kLpRepThreads) {
    const int id = p.ids[(int64_t)r * p.m + i];
    float v = 0.0f;
    if (id >= 0 && id < p.V) {
      v = ((float)row[id] - m) - ls;
    } else if (id != -1) {
      report_error(p.err, kErrInput);
      v = NAN;
    }
    p.logp[(int64_t)r * p.m + i] = v;
  }
  if (p.top == 0) return;

  // ---- the lower bound from the quarters' maxima (with fewer quarters than
  // `top`, every logit is a candidate)
  const float* qmax = p.quarter + (int64_t)r * p.windows * 4;
  const int nq = p.windows * 4, shift = lp_shift(row);
  unsigned bound = 0;
  if (nq >= p.top)
    bound = lp_select(p.top, hist, sel, [&](auto f) {
      for (int i = tid; i < nq; i += kLpRepThreads) f(lp_key(__ldcg(&qmax[i])));
    });
  if (tid == 0) s_count = 0;
  __syncthreads();
  // every logit of a quarter that reaches the bound, a warp a quarter
  auto scan = [&](auto f) {
    constexpr int E = 16 / sizeof(T), L = 8 / E;
    for (int i = warp; i < nq; i += kLpRepThreads / 32) {
      if (lp_key(__ldcg(&qmax[i])) < bound) continue;
      const int e0 = i * kLpQuarter - shift + lane * E;
      float x[8];
#pragma unroll
      for (int k = 0; k < L; ++k) lp_load<T>(row, e0 + k * 32 * E, p.V, x + k * E);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + (j / E) * 32 * E + j % E;
        if (e >= 0 && e < p.V) f(lp_key(x[j]), e);
      }
    }
  };
  scan([&](unsigned key, int e) {
    if (key >= bound) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kLpCand) {
        ckey[at] = key;
        cidx[at] = e;
      }
    }
  });
  __syncthreads();
  int n = s_count;
  if (n > kLpCand) {
    // many ties: the exact key of the `top`-th largest, all logits above it,
    // and of those equal to it the first ones in index order
    const unsigned kth = lp_select(p.top, hist, sel, [&](auto f) {
      scan([&](unsigned key, int) {
        if (key >= bound) f(key);
      });
    });
    __syncthreads();
    if (tid == 0) s_count = s_ties = 0;
    __syncthreads();
    scan([&](unsigned key, int e) {
      if (key > kth) {
        const int at = atomicAdd(&s_count, 1);  // fewer than top <= 64 of them
        ckey[at] = key;
        cidx[at] = e;
      }
    });
    __syncthreads();
    const int above = s_count, want = p.top - above;
    // the ties in index order, 256 logits at a time
    for (int e0 = 0; e0 < p.V; e0 += kLpRepThreads) {
      const int e = e0 + tid;
      const bool hit = e < p.V && lp_key((float)row[e]) == kth;
      const unsigned ball = __ballot_sync(0xffffffffu, hit);
      if (lane == 0) hist[warp] = __popc(ball);
      __syncthreads();
      int before = s_ties;
      for (int k = 0; k < warp; ++k) before += hist[k];
      const int at = before + __popc(ball & ((1u << lane) - 1u));
      if (hit && at < want) {
        ckey[above + at] = kth;
        cidx[above + at] = e;
      }
      __syncthreads();
      if (tid == 0)
        for (int k = 0; k < kLpRepThreads / 32; ++k) s_ties += hist[k];
      __syncthreads();
      if (s_ties >= want) break;
    }
    n = p.top;
    __syncthreads();
  }
  // ---- ranks: larger key first, then the lower index
  for (int i = tid; i < n; i += kLpRepThreads) {
    const unsigned key = ckey[i];
    const int e = cidx[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += ckey[j] > key || (ckey[j] == key && cidx[j] < e);
    if (rank < p.top) {
      p.top_ids[(int64_t)r * p.top + rank] = e;
      p.top_logp[(int64_t)r * p.top + rank] = ((float)row[e] - m) - ls;
    }
  }
}

static int lp_windows(int V, bool wide) { return (V + (wide ? 3 : 7) + kLpWindow - 1) / kLpWindow; }

size_t token_logprobs_ws(int R, int V) { return (size_t)R * lp_windows(V, false) * 32; }

cudaError_t launch_token_logprobs(const void* logits, bool bf16, const int32_t* ids, int R, int V, int m, int top,
                                  float* logp, float* entropy, int32_t* top_ids, float* top_logp, void* workspace,
                                  unsigned* err, cudaStream_t stream) {
  LogprobParams p;
  p.logits = logits;
  p.ids = ids;
  p.R = R;
  p.V = V;
  p.m = m;
  p.top = top;
  p.windows = lp_windows(V, !bf16);
  p.logp = logp;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logp = top_logp;
  p.win = static_cast<float*>(workspace);
  p.quarter = p.win + (size_t)R * p.windows * 4;
  p.err = err;
  const int64_t warps = (int64_t)R * p.windows;
  const dim3 grid((unsigned)((warps + kLpStatWarps - 1) / kLpStatWarps));
  const dim3 block(32 * kLpStatWarps);
  cudaError_t e = bf16 ? launch_pdl(token_stats_kernel<__nv_bfloat16>, grid, block, 0, stream, p)
                       : launch_pdl(token_stats_kernel<float>, grid, block, 0, stream, p);
  if (e != cudaSuccess) return e;
  return bf16 ? launch_pdl(token_report_kernel<__nv_bfloat16>, dim3((unsigned)R), dim3(kLpRepThreads), 0, stream, p)
              : launch_pdl(token_report_kernel<float>, dim3((unsigned)R), dim3(kLpRepThreads), 0, stream, p);
}

}  // namespace w4a16
