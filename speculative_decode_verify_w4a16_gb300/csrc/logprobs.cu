// Log probabilities of given tokens, entropy and the top alternatives of
// logit rows (contract in w4a16sv.h).
//
// Everything in powers of two, with l = log2 e: for a row x and a reference
// c = rn(l max x), S = sum 2^z and W = sum z 2^z over z = l x - c (one fused
// multiply-add, so c's rounding cancels; it moves the largest z by up to
// 2^-24 |c|, so from |max x| = 2^20 on z = l (x - max x) instead); then
//   log2 p(i) = (l x_i - c) - log2 S,   entropy = (log2 S - W / S) ln 2.
// Sums over parts of the row, each against its own c, merge by 2^(c_part - c).
// So the logits are read once.
//
// A warp takes a window of 1024 logits in registers (the next one's loads in
// flight): its (c, S, W) and the maxima of its four 256-logit quarters as
// ordered integers (one reduction instruction each; a NaN is above all numbers,
// so it reaches the maximum and with it every result). The report then merges
// the windows; the `top`-th largest maximum of windows (or groups of them) is a
// lower bound of the `top`-th largest logit, so only quarters that reach it are
// read again (few more than `top`, unless maxima tie), and the few logits at or
// above it are ranked in shared memory. Ranks are counted, each of the maxima
// against all: two orders of magnitude less latency than a sort of the row.
//
// Bound: HBM (one pass, 16-byte loads), next to it the instruction issue: some
// 240 a window and warp (bf16), so pairs of logits go through packed
// instructions wherever there are any. With at least four rows an SM a CTA takes
// a row from its first load to its report (token_logprobs_kernel); with fewer,
// the windows are spread over all SMs and a second kernel reports
// (token_stats_kernel, token_report_kernel). Rows of 128256 logits with 20
// alternatives, both ways, in us: bf16, 16 rows 15.7 and 11.5, 64 rows 16.0 and
// 17.1, 228 29.1 and 26.0, 456 34.5 and 36.5, 608 35.1 and 43.3, 1024 57.5 and
// 66.9; fp32, 16 rows 16.1 and 12.7, 228 27.4 and 32.2, 456 51.4 and 50.1, 608
// 60.3 and 61.5, 1024 105 and 97: nowhere does the rule lose more than 18 %.
// A row's CTA has 256 threads, four CTAs an SM: with 1024 rows the later rows
// stream while the first ones report (57 us, 263 MB: 0.68 of the HBM copy rate;
// 58 us with every load's bounds looked at, not only those of a row's ends); 128
// threads and eight CTAs take them all at once and then report all at once, 68
// against 58; 512 threads 63; the maxima by the reduction instruction for floats
// 58 against 56. 16 rows of fp32 (8.2 MB) take 8.2 us, latency. Rows where fewer
// than `top` logits are above all others (all but a few masked, or flat) take 0.3
// ms, 1024 of them 0.9 (bf16) and 1.7 ms: every logit is then a candidate.
// Windows start at 16-byte boundaries of memory, not of the row, so that rows of
// any length load 16 bytes at a time.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kLpWindow = 1024;
constexpr int kLpQuarter = 256;
constexpr int kLpStatWarps = 8;
constexpr int kLpRowThreads = 256;  // of a row's report (and its windows, in one kernel)
constexpr int kLpCand = 1024;       // logits ranked in shared memory
constexpr float kLpLog2e = 1.4426950408889634f, kLpLn2 = 0.69314718055994531f;
constexpr float kLpNear = 1048576.0f;  // maxima below it: c is the reference, else l max x itself

struct LogprobParams {
  const void* logits;
  const int32_t* ids;
  int R, V, m, top;
  int windows;  // per row
  float *logp, *entropy;
  int32_t* top_ids;
  float* top_logp;
  float4* win;     // [R][windows]: c, S, W, unused
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

// the largest, NaN if any is
__device__ __forceinline__ float lp_max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t lp_maxh2(uint32_t a, uint32_t b) {  // of two bf16 pairs
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One window of a warp from its raw words: quarter maxima (the same in every
// lane), and c, S, W (valid in lane 0)
template <typename T>
__device__ __forceinline__ void lp_window(uint4 (&raw)[32 * sizeof(T) / 16], int lane, unsigned (&key)[4], float& c,
                                          float& S, float& W) {
  constexpr int L = 32 * sizeof(T) / 16;
  uint32_t* u = reinterpret_cast<uint32_t*>(raw);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float m;
    if constexpr (sizeof(T) == 4) {
      const float* x = reinterpret_cast<const float*>(raw) + 8 * q;
      m = lp_max3(lp_max3(lp_max3(x[0], x[1], x[2]), x[3], x[4]), lp_max3(x[5], x[6], x[7]), x[7]);
    } else {
      const uint32_t h = lp_maxh2(lp_maxh2(u[4 * q], u[4 * q + 1]), lp_maxh2(u[4 * q + 2], u[4 * q + 3]));
      const float lo = __uint_as_float(h << 16), hi = __uint_as_float(h & 0xFFFF0000u);
      m = lp_max3(lo, hi, hi);
    }
    key[q] = __reduce_max_sync(0xffffffffu, lp_key(m));
  }
  const float mx = lp_unkey(max(max(key[0], key[1]), max(key[2], key[3])));
  c = mx * kLpLog2e;
  uint64_t s2[2] = {0ull, 0ull}, w2[2] = {0ull, 0ull};
  if (fabsf(mx) < kLpNear) {
    // logits below -1e30 (masks) as -1e30: their 2^z is 0 either way, and z 2^z
    // is 0 and not -inf * 0
    const uint64_t nc = lp_2(-c, -c), l2 = lp_2(kLpLog2e, kLpLog2e);
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 low = __float2bfloat162_rn(-1e30f);
#pragma unroll
      for (int k = 0; k < 4 * L; ++k) u[k] = lp_maxh2(u[k], *reinterpret_cast<const uint32_t*>(&low));
    }
#pragma unroll
    for (int k = 0; k < L; ++k) {
      constexpr int E = 16 / sizeof(T);
      float x[E];
      lp_floats<T>(raw[k], x);
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        if constexpr (sizeof(T) == 4) {
          x[j] = fmaxf(x[j], -1e30f);
          x[j + 1] = fmaxf(x[j + 1], -1e30f);
        }
        const uint64_t z = lp_fma2(lp_2(x[j], x[j + 1]), l2, nc);
        float z0, z1;
        lp_un2(z, z0, z1);
        const uint64_t t = lp_2(lp_ex2(z0), lp_ex2(z1));
        s2[(j >> 1) & 1] = lp_add2(s2[(j >> 1) & 1], t);
        w2[(j >> 1) & 1] = lp_fma2(z, t, w2[(j >> 1) & 1]);
      }
    }
  } else if (mx == mx && fabsf(mx) < INFINITY) {
    // a maximum beyond: the differences first, then their powers
#pragma unroll
    for (int k = 0; k < L; ++k) {
      constexpr int E = 16 / sizeof(T);
      float x[E];
      lp_floats<T>(raw[k], x);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float z = fmaxf((x[j] - mx) * kLpLog2e, -1e30f), t = lp_ex2(z);
        float a, b;
        lp_un2(s2[0], a, b);
        s2[0] = lp_2(a + t, b);
        lp_un2(w2[0], a, b);
        w2[0] = lp_2(fmaf(z, t, a), b);
      }
    }
  }
  float a, b, d, e;
  lp_un2(lp_add2(s2[0], s2[1]), a, b);
  lp_un2(lp_add2(w2[0], w2[1]), d, e);
  // both sums over the warp: S in the lower lanes, W in the upper ones
  const float sl = a + b, wl = d + e;
  float v = (lane & 16 ? wl : sl) + __shfl_xor_sync(0xffffffffu, lane & 16 ? sl : wl, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  S = v;
  W = __shfl_sync(0xffffffffu, v, 16);
}

// the raw words of a window: lane's 16-byte pieces, 512 bytes apart
template <typename T>
__device__ __forceinline__ void lp_fetch(const T* row, int w, int V, int lane, uint4 (&raw)[32 * sizeof(T) / 16]) {
  constexpr int E = 16 / sizeof(T), L = 32 / E;
  const int first = w * kLpWindow - lp_shift(row), e0 = first + lane * E;
  if (first >= 0 && first + kLpWindow <= V) {  // all but the row's ends
    const uint4* p = reinterpret_cast<const uint4*>(row + e0);
#pragma unroll
    for (int k = 0; k < L; ++k) raw[k] = __ldg(p + k * 32);
  } else {
#pragma unroll
    for (int k = 0; k < L; ++k) raw[k] = lp_load<T>(row, e0 + k * 32 * E, V);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kLpStatWarps, sizeof(T) == 2 ? 4 : 2) token_stats_kernel(const LogprobParams p) {
  constexpr int L = 32 * sizeof(T) / 16;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int total = p.R * p.windows, step = gridDim.x * kLpStatWarps;
  int id = blockIdx.x * kLpStatWarps + (threadIdx.x >> 5);
  uint4 next[L];
  auto fetch = [&](int i) {
    const int r = i / p.windows;
    lp_fetch<T>(static_cast<const T*>(p.logits) + (int64_t)r * p.V, i - r * p.windows, p.V, lane, next);
  };
  if (id < total) fetch(id);
  for (; id < total; id += step) {
    uint4 raw[L];
#pragma unroll
    for (int k = 0; k < L; ++k) raw[k] = next[k];
    if (id + step < total) fetch(id + step);
    unsigned key[4];
    float c, S, W;
    lp_window<T>(raw, lane, key, c, S, W);
    if (lane == 0) {
      p.win[id] = make_float4(c, S, W, 0.0f);
      p.quarter[id] = make_uint4(key[0], key[1], key[2], key[3]);
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
    for (int i = threadIdx.x; i < 256; i += kLpRowThreads) hist[i] = 0;
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

// A row's shared arrays: every window's statistics and quarter keys, the
// windows' keys, the quarters to read again
struct LpRow {
  float4* win;
  uint4* quarter;
  unsigned* wkey;
  int* quarters;
  __device__ __forceinline__ LpRow(uint4* mem, int windows)
      : win(reinterpret_cast<float4*>(mem)), quarter(mem + windows),
        wkey(reinterpret_cast<unsigned*>(mem + 2 * windows)),
        quarters(reinterpret_cast<int*>(wkey + windows)) {}
};
static size_t lp_row_bytes(int windows, int top) {
  return (size_t)windows * 36 + (top > 0 ? (size_t)windows * 16 : 0);
}

// The report of row r by the CTA. Thread i < m has its token's id and logit;
// win and quarter are filled (and synchronised).
template <typename T>
__device__ void lp_report(const LogprobParams& p, int r, const T* row, const LpRow& s, int id0, float x0) {
  __shared__ __align__(16) int hist[256];
  __shared__ unsigned sel[2];
  __shared__ float red[2][kLpRowThreads / 32];
  __shared__ unsigned red_k[kLpRowThreads / 32];
  __shared__ unsigned ckey[kLpCand];
  __shared__ int cidx[kLpCand];
  __shared__ int s_count, s_ties, s_quarters;
  __shared__ unsigned s_bound;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nq = p.windows * 4, shift = lp_shift(row);
  const unsigned* qkey = reinterpret_cast<const unsigned*>(s.quarter);
  const unsigned* wkey = s.wkey;
  int* quarters = s.quarters;
  unsigned mk = 0u;
  for (int w = tid; w < p.windows; w += kLpRowThreads) {
    const uint4 k = s.quarter[w];
    const unsigned most = max(max(k.x, k.y), max(k.z, k.w));
    s.wkey[w] = most;
    mk = max(mk, most);
  }
  mk = __reduce_max_sync(0xffffffffu, mk);
  if (lane == 0) red_k[warp] = mk;
  if (tid == 0) {
    s_count = s_quarters = 0;
    s_bound = 0u;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kLpRowThreads / 32; ++k) mk = max(mk, red_k[k]);
  const float m = lp_unkey(mk), c = m * kLpLog2e;
  // ---- the windows merged: every sum against the row's reference
  const bool fine = fabsf(m) < INFINITY, near = fabsf(m) < kLpNear;
  float S = 0.0f, W = 0.0f;
  if (fine)
    for (int w = tid; w < p.windows; w += kLpRowThreads) {
      const float4 v = s.win[w];
      const float mx = lp_unkey(wkey[w]);
      // the window's reference less the row's, whichever form each has
      float d;
      if (fabsf(mx) < kLpNear)
        d = near ? v.x - c : -fmaf(m, kLpLog2e, -v.x);
      else
        d = near ? fmaf(mx, kLpLog2e, -c) : (mx - m) * kLpLog2e;
      d = fmaxf(d, -1e30f);
      const float t = exp2f(d);
      S = fmaf(v.y, t, S);
      W += t * fmaf(d, v.y, v.z);
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
  for (int k = 0; k < kLpRowThreads / 32; ++k) {
    S += red[0][k];
    W += red[1][k];
  }
  // a NaN, +inf or -inf alone: no distribution
  const float ls = fine ? log2f(S) : NAN;
  auto logp = [&](float x) {
    // by the same form as the sums; for a mask near the type's lowest value by
    // the difference, which does not overflow
    return near && fabsf(x) < 1e30f ? (fmaf(x, kLpLog2e, -c) - ls) * kLpLn2 : (x - m) - ls * kLpLn2;
  };
  if (tid == 0 && p.entropy) p.entropy[r] = (ls - W / S) * kLpLn2;
  if (tid < p.m) {  // m <= 64 of them
    if (id0 < -1 || id0 >= p.V) report_error(p.err, kErrInput);
    p.logp[(int64_t)r * p.m + tid] = id0 == -1 ? 0.0f : id0 >= 0 && id0 < p.V ? logp(x0) : NAN;
  }
  if (p.top == 0) return;

  // ---- the lower bound: the `top`-th largest maximum of as few groups of
  // windows as leave 2 top of them, of the windows, of the quarters, or of sixteen
  // logits each (where there are no `top` of those, every logit is a candidate).
  // Fewer maxima are quicker to rank and let few more logits through: of 63 maxima
  // the 20th is on average the 24th logit, of 126 the 22nd.
  {
    int g = 1;
    while ((p.windows + 2 * g - 1) / (2 * g) >= 2 * p.top) g *= 2;
    const bool quarters_too = p.windows < p.top;
    const int n = quarters_too ? nq : (p.windows + g - 1) / g;  // < 4 top: no more than 256
    unsigned* key = reinterpret_cast<unsigned*>(hist);
    for (int i = tid; i < (n + 3) / 4 * 4; i += kLpRowThreads) {
      unsigned most = 0u;
      if (i < n && quarters_too) most = qkey[i];
      else if (i < n)
        for (int w = i * g; w < min(i * g + g, p.windows); ++w) most = max(most, wkey[w]);
      key[i] = most;
    }
    __syncthreads();
    if (n >= p.top)
      for (int i = tid; i < n; i += kLpRowThreads) {
        const unsigned mine = key[i];
        int above = 0, equal = 0;  // (a key of 0 past the end is no larger than any)
        for (int j = 0; j < n; j += 4) {
          const uint4 k = reinterpret_cast<const uint4*>(key)[j >> 2];
          above += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
          equal += (k.x == mine) + (k.y == mine) + (k.z == mine) + (k.w == mine);
        }
        if (above < p.top && p.top <= above + equal) s_bound = mine;  // all that write it write the same
      }
    else if (p.V / 16 >= p.top) {
      // fewer quarters than that: the maxima of sixteen logits (two lanes of a
      // warp), of which there are `top` (1000 rows of 4000 logits with 32
      // alternatives: 36 us, 73 with all logits as candidates)
      constexpr int E = 16 / sizeof(T), L = 8 / E;
      for (int i = warp; i < nq; i += kLpRowThreads / 32) {  // nq < top: no more than 1008 places
        const int e0 = i * kLpQuarter - shift + lane * E;
        unsigned most = 0u;
#pragma unroll
        for (int c = 0; c < L; ++c) {
          float x[E];
          lp_floats<T>(lp_load<T>(row, e0 + c * 32 * E, p.V), x);
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const int e = e0 + c * 32 * E + j;
            if (e >= 0 && e < p.V) most = max(most, lp_key(x[j]));
          }
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        if (!(lane & 1)) ckey[16 * i + (lane >> 1)] = most;  // 0: no logit
      }
      __syncthreads();
      const unsigned least = lp_select(p.top, hist, sel, [&](auto f) {
        for (int i = tid; i < 16 * nq; i += kLpRowThreads)
          if (ckey[i]) f(ckey[i]);
      });
      if (tid == 0) s_bound = least;
    }
  }
  __syncthreads();
  const unsigned bound = s_bound;
  for (int i = tid; i < nq; i += kLpRowThreads)
    if (qkey[i] >= bound) quarters[atomicAdd(&s_quarters, 1)] = i;
  __syncthreads();
  const int again = s_quarters;
  // every logit of a quarter that reaches the bound, a warp a quarter
  auto scan = [&](auto f) {
    constexpr int E = 16 / sizeof(T), L = 8 / E;
    for (int i = warp; i < again; i += kLpRowThreads / 32) {
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
    for (int e0 = 0; e0 < p.V; e0 += kLpRowThreads) {
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
        for (int k = 0; k < kLpRowThreads / 32; ++k) s_ties += hist[k];
      __syncthreads();
      if (s_ties >= want) break;
    }
    n = p.top;
    __syncthreads();
  }
  // few quarters, and so many candidates: all against all costs n^2, so first
  // only those that reach the `top`-th key, and of many equal to it the first ones
  // (1000 rows of 1000 logits with 32 alternatives: 36 us, 834 with all of them)
#pragma unroll 1
  for (int round = 0; round < 2 && n > 4 * p.top; ++round) {
    const unsigned kth = round == 0 ? 0u : sel[0];
    const int ties = (int)sel[1];  // of the `top` largest, those equal to the last
    __syncthreads();
    const unsigned least = lp_select(round == 0 ? p.top : ties, hist, sel, [&](auto f) {
      for (int i = tid; i < n; i += kLpRowThreads) {
        if (round == 0)
          f(ckey[i]);
        else if (ckey[i] == kth)
          f(~(unsigned)cidx[i]);
      }
    });
    constexpr int kEach = kLpCand / kLpRowThreads;
    unsigned key[kEach];
    int e[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = tid + j * kLpRowThreads;
      key[j] = i < n ? ckey[i] : 0u;
      e[j] = i < n ? cidx[i] : 0;
    }
    __syncthreads();
    if (tid == 0) s_count = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (tid + j * kLpRowThreads < n &&
          (round == 0 ? key[j] >= least : key[j] > kth || ~(unsigned)e[j] >= least)) {
        const int at = atomicAdd(&s_count, 1);
        ckey[at] = key[j];
        cidx[at] = e[j];
      }
    __syncthreads();
    n = s_count;
  }
  // ---- ranks: larger key first, then the lower index
  for (int i = tid; i < n; i += kLpRowThreads) {
    const unsigned key = ckey[i];
    const int e = cidx[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += ckey[j] > key || (ckey[j] == key && cidx[j] < e);
    if (rank < p.top) {
      p.top_ids[(int64_t)r * p.top + rank] = e;
      p.top_logp[(int64_t)r * p.top + rank] = logp((float)row[e]);
    }
  }
}

// The report of rows whose windows another kernel has summed up.
template <typename T>
__global__ void __launch_bounds__(kLpRowThreads) token_report_kernel(const LogprobParams p) {
  extern __shared__ uint4 lp_smem[];
  grid_launch_dependents();
  grid_dependency_wait();
  const int r = blockIdx.x, tid = threadIdx.x;
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
  const LpRow s(lp_smem, p.windows);
  const int id0 = tid < p.m ? p.ids[(int64_t)r * p.m + tid] : -1;
  const float x0 = id0 >= 0 && id0 < p.V ? (float)row[id0] : 0.0f;
  for (int w = tid; w < p.windows; w += kLpRowThreads) {
    s.win[w] = __ldcg(&p.win[(int64_t)r * p.windows + w]);
    s.quarter[w] = __ldcg(&p.quarter[(int64_t)r * p.windows + w]);
  }
  __syncthreads();
  lp_report<T>(p, r, row, s, id0, x0);
}

// A CTA a row, from the windows to the report.
template <typename T>
__global__ void __launch_bounds__(kLpRowThreads, sizeof(T) == 2 ? 4 : 2) token_logprobs_kernel(const LogprobParams p) {
  extern __shared__ uint4 lp_smem[];
  constexpr int L = 32 * sizeof(T) / 16, kWarps = kLpRowThreads / 32;
  grid_launch_dependents();
  grid_dependency_wait();
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.V;
  const LpRow s(lp_smem, p.windows);
  const int id0 = tid < p.m ? p.ids[(int64_t)r * p.m + tid] : -1;
  uint4 next[L];
  if (warp < p.windows) lp_fetch<T>(row, warp, p.V, lane, next);
  const float x0 = id0 >= 0 && id0 < p.V ? (float)row[id0] : 0.0f;
  for (int w = warp; w < p.windows; w += kWarps) {
    uint4 raw[L];
#pragma unroll
    for (int k = 0; k < L; ++k) raw[k] = next[k];
    if (w + kWarps < p.windows) lp_fetch<T>(row, w + kWarps, p.V, lane, next);
    unsigned key[4];
    float c, S, W;
    lp_window<T>(raw, lane, key, c, S, W);
    if (lane == 0) {
      s.win[w] = make_float4(c, S, W, 0.0f);
      s.quarter[w] = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  __syncthreads();
  lp_report<T>(p, r, row, s, id0, x0);
}

static int lp_windows(int V, bool wide) { return (V + (wide ? 3 : 7) + kLpWindow - 1) / kLpWindow; }

size_t token_logprobs_ws(int R, int V) { return (size_t)R * lp_windows(V, false) * 32; }

template <typename T>
static cudaError_t launch_lp(const LogprobParams& p, int num_sms, cudaStream_t stream) {
  const size_t smem = lp_row_bytes(p.windows, p.top);  // 6 KB for 128 K logits, 49 KB for 2^20
  cudaError_t e;
  // a CTA a row when that gives every SM four of them (measured above)
  if (p.R >= 4 * num_sms) {
    if (smem > 32 * 1024) {
      e = cudaFuncSetAttribute(token_logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(token_logprobs_kernel<T>, dim3((unsigned)p.R), dim3(kLpRowThreads), smem, stream, p);
  }
  // every SM's resident CTAs (4, or 2 of fp32: see the kernel's bounds), fewer
  // when there are fewer windows
  const int64_t warps = (int64_t)p.R * p.windows, most = (int64_t)num_sms * (sizeof(T) == 2 ? 4 : 2);
  const int64_t ctas = (warps + kLpStatWarps - 1) / kLpStatWarps;
  e = launch_pdl(token_stats_kernel<T>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * kLpStatWarps), 0, stream,
                 p);
  if (e != cudaSuccess) return e;
  if (smem > 32 * 1024) {
    e = cudaFuncSetAttribute(token_report_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(token_report_kernel<T>, dim3((unsigned)p.R), dim3(kLpRowThreads), smem, stream, p);
}

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
  return bf16 ? launch_lp<__nv_bfloat16>(p, num_sms, stream) : launch_lp<float>(p, num_sms, stream);
}

}  // namespace w4a16
