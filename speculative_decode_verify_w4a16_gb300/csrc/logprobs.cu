// Log probabilities of given tokens, entropy and the top alternatives of
// logit rows (contract in w4a16sv.h).
//
// For a row x: m = max x, S = sum exp(x - m), W = sum (x - m) exp(x - m);
// ln p(i) = (x_i - m) - ln S, entropy = ln S - W / S. All three sums merge
// over parts of the row (each part against its own maximum, then scaled by
// exp(m_part - m)), so the logits are read once.
//
// token_stats_kernel: a warp takes a window of 1024 logits in registers (the
// next one's loads in flight) and leaves its (m, S, W) and the maxima of its
// four 256-logit quarters as ordered integers (one reduction instruction each;
// a NaN is above all numbers, so it reaches m and with it every result).
// token_report_kernel, one CTA per row: merges the windows; the `top`-th
// largest window maximum is a lower bound of the `top`-th largest logit, so
// only quarters that reach it are read again (few more than `top`, unless
// maxima tie), and the few logits at or above it are ranked in shared memory.
// Ranks are counted (each of up to 1025 values against all), two orders of
// magnitude less latency than a sort of the row.
//
// Bound: HBM for the first kernel (one pass, 16-byte loads); the second reads
// 3 % of the row's bytes (bf16; fp32 1.6 %) in statistics and some top x 256
// logits, mostly from L2: its latency counts. Windows start at 16-byte boundaries of memory, not of the row, so
// that rows of any length load 16 bytes at a time.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kLpWindow = 1024;
constexpr int kLpQuarter = 256;
constexpr int kLpStatWarps = 8;
constexpr int kLpRepThreads = 128;
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
  float4* win;     // [R][windows]: m, S, W (in powers of two: sum of log2 terms), unused
  uint4* quarter;  // [R][windows]: the quarters' maxima (lp_key)
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

__device__ __forceinline__ uint64_t lp_2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void lp_un2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t lp_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t lp_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t lp_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// the 16 bytes at index e of the row (a multiple of 16 bytes less the shift),
// elements outside [0, V) set to -inf
template <typename T>
__device__ __forceinline__ uint4 lp_load(const T* row, int e, int V) {
  constexpr int E = 16 / sizeof(T);
  if (e >= 0 && e + E <= V) return __ldg(reinterpret_cast<const uint4*>(row + e));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[k] = e + k >= 0 && e + k < V ? reinterpret_cast<const uint32_t*>(row)[e + k] : 0xFF800000u;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
      const uint32_t lo = e + 2 * k >= 0 && e + 2 * k < V ? h[e + 2 * k] : 0xFF80u;
      const uint32_t hi = e + 2 * k + 1 >= 0 && e + 2 * k + 1 < V ? h[e + 2 * k + 1] : 0xFF80u;
      w[k] = lo | (hi << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// ... as floats
template <typename T>
__device__ __forceinline__ void lp_floats(uint4 v, float* x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      x[k] = __uint_as_float(u[k]);
    } else {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  }
}

// An order of the logits as unsigned integers: rising with the value, the
// two zeros equal, NaN above all.
__device__ __forceinline__ unsigned lp_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const unsigned b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float lp_unkey(unsigned k) {
  return k == 0xFFFFFFFFu ? NAN : __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ float lp_warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(32 * kLpStatWarps, sizeof(T) == 2 ? 4 : 2) token_stats_kernel(const LogprobParams p) {
  constexpr int E = 16 / sizeof(T), L = 32 / E;  // loads of E elements a lane
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int total = p.R * p.windows, step = gridDim.x * kLpStatWarps;
  int id = blockIdx.x * kLpStatWarps + (threadIdx.x >> 5);
  uint4 next[L];
  auto load = [&](int i) {
    const int r = i / p.windows, w = i - r * p.windows;
    const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
    const int e0 = w * kLpWindow - lp_shift(row) + lane * E;
#pragma unroll
    for (int k = 0; k < L; ++k) next[k] = lp_load<T>(row, e0 + k * 32 * E, p.V);
  };
  if (id < total) load(id);
  for (; id < total; id += step) {
    float x[32];
#pragma unroll
    for (int k = 0; k < L; ++k) lp_floats<T>(next[k], x + k * E);
    if (id + step < total) load(id + step);
    unsigned key[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // the largest as a float, unless a NaN (which compares false) is among them
      float m = x[8 * q];
      bool nan = x[8 * q] != x[8 * q];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        m = fmaxf(m, x[8 * q + j]);
        nan |= x[8 * q + j] != x[8 * q + j];
      }
      key[q] = __reduce_max_sync(0xffffffffu, nan ? 0xFFFFFFFFu : lp_key(m));
    }
    const float mx = lp_unkey(max(max(key[0], key[1]), max(key[2], key[3])));
    // z = (x - m) log2 e (kept off -inf, and off NaN: m carries that), S = sum
    // 2^z, W = sum z 2^z, two logits an instruction
    const uint64_t nm = lp_2(-mx, -mx), l2 = lp_2(kLpLog2e, kLpLog2e);
    uint64_t s2[2] = {0ull, 0ull}, w2[2] = {0ull, 0ull};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float z0, z1;
      lp_un2(lp_mul2(lp_add2(lp_2(x[j], x[j + 1]), nm), l2), z0, z1);
      z0 = fmaxf(z0, -1e30f);
      z1 = fmaxf(z1, -1e30f);
      const uint64_t t = lp_2(lp_ex2(z0), lp_ex2(z1));
      s2[(j >> 1) & 1] = lp_add2(s2[(j >> 1) & 1], t);
      w2[(j >> 1) & 1] = lp_fma2(lp_2(z0, z1), t, w2[(j >> 1) & 1]);
    }
    float a, b, c, d;
    lp_un2(lp_add2(s2[0], s2[1]), a, b);
    lp_un2(lp_add2(w2[0], w2[1]), c, d);
    const float S = lp_warp_sum(a + b), W = lp_warp_sum(c + d);
    if (lane == 0) {
      p.win[id] = make_float4(mx, S, W, 0.0f);
      if (p.top > 0) p.quarter[id] = make_uint4(key[0], key[1], key[2], key[3]);
    }
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
  __shared__ float red[2][kLpRepThreads / 32];
  __shared__ unsigned red_k[kLpRepThreads / 32];
  __shared__ unsigned ckey[kLpCand];
  __shared__ int cidx[kLpCand];
  __shared__ int s_count, s_ties, s_quarters;
  __shared__ unsigned s_bound;
  extern __shared__ __align__(16) unsigned lp_smem[];
  grid_launch_dependents();
  grid_dependency_wait();
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
  const float4* win = p.win + (int64_t)r * p.windows;
  const int nq = p.windows * 4, shift = lp_shift(row), wpad = (p.windows + 3) / 4 * 4;
  unsigned* wkey = lp_smem;                                // [wpad] keys of the windows' maxima
  unsigned* qkey = wkey + wpad;                            // [nq] ... of the quarters' (top > 0)
  int* quarters = reinterpret_cast<int*>(qkey + nq);       // [nq] those to read again
  // ---- the given tokens' logits asked for (their ids come first), then the
  // statistics; thread tid's first window stays in registers
  const int id0 = tid < p.m ? p.ids[(int64_t)r * p.m + tid] : -1;
  const float x0 = id0 >= 0 && id0 < p.V ? (float)row[id0] : 0.0f;
  float4 v0 = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
  unsigned mk = 0u;
  for (int w = tid; w < wpad; w += kLpRepThreads) {
    unsigned k = 0u;
    if (w < p.windows) {
      const float4 v = __ldcg(&win[w]);
      if (w == tid) v0 = v;
      k = lp_key(v.x);
      if (p.top > 0) reinterpret_cast<uint4*>(qkey)[w] = __ldcg(p.quarter + (int64_t)r * p.windows + w);
    }
    wkey[w] = k;
    mk = max(mk, k);
  }
  mk = __reduce_max_sync(0xffffffffu, mk);
  if (lane == 0) red_k[warp] = mk;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kLpRepThreads / 32; ++k) mk = max(mk, red_k[k]);
  const float m = lp_unkey(mk);
  // ---- the windows merged: every sum against the row's maximum
  float S = 0.0f, W = 0.0f;
  for (int w = tid; w < p.windows; w += kLpRepThreads) {
    const float4 v = w == tid ? v0 : __ldcg(&win[w]);
    const float d = fmaxf(v.x - m, -1e30f), t = expf(d);
    S = fmaf(v.y, t, S);
    W += t * fmaf(d, v.y, v.z * 0.69314718056f);
  }
  S = lp_warp_sum(S);
  W = lp_warp_sum(W);
  if (lane == 0) {
    red[0][warp] = S;
    red[1][warp] = W;
  }
  __syncthreads();
  S = W = 0.0f;
#pragma unroll
  for (int k = 0; k < kLpRepThreads / 32; ++k) {
    S += red[0][k];
    W += red[1][k];
  }
  // a NaN, +inf or -inf alone: no distribution
  const float ls = S > 0.0f && m < INFINITY && m > -INFINITY ? logf(S) : NAN;
  if (tid == 0 && p.entropy) p.entropy[r] = ls - W / S;
  if (tid < p.m) {  // m <= 64 of them
    if (id0 < -1 || id0 >= p.V) report_error(p.err, kErrInput);
    p.logp[(int64_t)r * p.m + tid] = id0 == -1 ? 0.0f : id0 >= 0 && id0 < p.V ? (x0 - m) - ls : NAN;
  }
  if (p.top == 0) return;

  // ---- the lower bound: the `top`-th largest maximum of the windows, or of
  // the quarters where there are fewer windows (with fewer quarters than `top`,
  // every logit is a candidate)
  if (tid == 0) {
    s_count = s_quarters = 0;
    s_bound = 0u;
  }
  __syncthreads();
  {
    const bool by_window = p.windows >= p.top;
    const int n = by_window ? p.windows : nq;
    const unsigned* key = by_window ? wkey : qkey;
    if (n >= p.top)
      for (int i = tid; i < n; i += kLpRepThreads) {
        const unsigned mine = key[i];
        int rank = 0;  // of value i, the earlier of equal ones first (a key of 0 past the end counts for nothing)
        for (int j = 0; j < n; j += 4) {
          const uint4 k = reinterpret_cast<const uint4*>(key)[j >> 2];
          rank += (k.x > mine || (k.x == mine && j < i)) + (k.y > mine || (k.y == mine && j + 1 < i)) +
                  (k.z > mine || (k.z == mine && j + 2 < i)) + (k.w > mine || (k.w == mine && j + 3 < i));
        }
        if (rank == p.top - 1) s_bound = mine;
      }
  }
  __syncthreads();
  const unsigned bound = s_bound;
  for (int i = tid; i < nq; i += kLpRepThreads)
    if (qkey[i] >= bound) quarters[atomicAdd(&s_quarters, 1)] = i;
  __syncthreads();
  const int again = s_quarters;
  // every logit of a quarter that reaches the bound, a warp a quarter
  auto scan = [&](auto f) {
    constexpr int E = 16 / sizeof(T), L = 8 / E;
    for (int i = warp; i < again; i += kLpRepThreads / 32) {
      const int e0 = quarters[i] * kLpQuarter - shift + lane * E;
      float x[8];
#pragma unroll
      for (int k = 0; k < L; ++k) lp_floats<T>(lp_load<T>(row, e0 + k * 32 * E, p.V), x + k * E);
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
    // the ties in index order, a logit a thread at a time
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
                                  int num_sms, unsigned* err, cudaStream_t stream) {
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
  p.win = static_cast<float4*>(workspace);
  p.quarter = reinterpret_cast<uint4*>(p.win + (size_t)R * p.windows);
  p.err = err;
  // every SM's resident CTAs (4, or 2 of fp32: see the kernel's bounds), fewer
  // when there are fewer windows
  const int64_t warps = (int64_t)R * p.windows, most = (int64_t)num_sms * (bf16 ? 4 : 2);
  const int64_t ctas = (warps + kLpStatWarps - 1) / kLpStatWarps;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  const dim3 block(32 * kLpStatWarps);
  cudaError_t e = bf16 ? launch_pdl(token_stats_kernel<__nv_bfloat16>, grid, block, 0, stream, p)
                       : launch_pdl(token_stats_kernel<float>, grid, block, 0, stream, p);
  if (e != cudaSuccess) return e;
  // window keys, quarter keys, quarter numbers (37 KB for 2^20 logits)
  const size_t smem = ((size_t)p.windows * (top > 0 ? 8 : 0) + (p.windows + 3) / 4 * 4) * 4;
  return bf16 ? launch_pdl(token_report_kernel<__nv_bfloat16>, dim3((unsigned)R), dim3(kLpRepThreads), smem, stream, p)
              : launch_pdl(token_report_kernel<float>, dim3((unsigned)R), dim3(kLpRepThreads), smem, stream, p);
}

}  // namespace w4a16
