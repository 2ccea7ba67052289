// Rotary positions, and the append of a step's rows to the paged 16-bit cache
// (contracts in w4a16sv.h).
//
// Pair i of a head's first `rot` elements turns by the angle a_i = p f_i, p the
// row's position: (u, v) -> factor (u cos a_i - v sin a_i, v cos a_i + u sin
// a_i). The angle is needed modulo a whole turn, and p f_i / 2 pi loses its
// fraction in fp32 for far positions, so f_i / 2 pi is kept as a 64-bit fixed
// point fraction of a turn, F_i: the low 64 bits of p F_i are the fraction, with
// the error of F_i's rounding alone (p 2^-65 turns), for every int32 position.
// An eighth of a turn at most is left for the sine and cosine once the nearest
// quarter turn is split off.
//
// Bound: HBM (each row read and written once) for prompts; launch and load
// latency for the rows of a step. A CTA takes a row: its loads go out first, the
// row's sines and cosines (one pair a thread, for all heads) are computed
// meanwhile and handed over through shared memory.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kRowThreads = 256;

// eight elements as fp32, and back: 16 bytes of bf16 or fp16, 32 of fp32
template <int TYPE>
struct Eight {
  uint4 w[TYPE == 2 ? 2 : 1];
};
template <int TYPE>
constexpr int kElt = TYPE == 2 ? 4 : 2;

template <int TYPE>
__device__ __forceinline__ Eight<TYPE> load8(const void* p, int64_t at) {
  Eight<TYPE> e;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * kElt<TYPE>);
#pragma unroll
  for (int i = 0; i < (TYPE == 2 ? 2 : 1); ++i) e.w[i] = s[i];
  return e;
}
template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t at, const Eight<TYPE>& e) {
  uint4* d = reinterpret_cast<uint4*>(static_cast<char*>(p) + at * kElt<TYPE>);
#pragma unroll
  for (int i = 0; i < (TYPE == 2 ? 2 : 1); ++i) d[i] = e.w[i];
}
template <int TYPE>
__device__ __forceinline__ void widen(const Eight<TYPE>& e, float (&f)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&e);
  if constexpr (TYPE == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == 0) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
}
template <int TYPE>
__device__ __forceinline__ Eight<TYPE> narrow(const float (&f)[8]) {
  Eight<TYPE> e;
  uint32_t* w = reinterpret_cast<uint32_t*>(&e);
  if constexpr (TYPE == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == 0) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  return e;
}

// cosine and sine of a turn's fraction in 2^-32 turns, times `factor`
__device__ __forceinline__ float2 cos_sin(uint32_t turn, float factor) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const int rest = (int)(turn - (quarter << 30));  // -2^29 .. 2^29 - 1
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);
  const float cs = (quarter & 1u) ? s : c, sn = (quarter & 1u) ? c : s;
  return make_float2((quarter == 1u || quarter == 2u) ? -cs * factor : cs * factor,
                     quarter >= 2u ? -sn * factor : sn * factor);
}

// The rotated (u, v) of unit `u` of a head: pairs 8 u .. 8 u + 7. Half layout:
// eight elements at 8 u and eight at rot / 2 + 8 u; interleaved: sixteen at 16 u.
template <int TYPE>
__device__ __forceinline__ void turn_unit(Eight<TYPE>& a, Eight<TYPE>& b, const float2* cs, int u, bool inter) {
  float x[8], y[8];
  widen<TYPE>(a, x);
  widen<TYPE>(b, y);
  const float2* c = cs + 8 * u;
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c0 = c[i], c1 = c[4 + i];
      const float u0 = x[2 * i], v0 = x[2 * i + 1], u1 = y[2 * i], v1 = y[2 * i + 1];
      x[2 * i] = u0 * c0.x - v0 * c0.y;
      x[2 * i + 1] = v0 * c0.x + u0 * c0.y;
      y[2 * i] = u1 * c1.x - v1 * c1.y;
      y[2 * i + 1] = v1 * c1.x + u1 * c1.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 ci = c[i];
      const float p = x[i], q = y[i];
      x[i] = p * ci.x - q * ci.y;
      y[i] = q * ci.x + p * ci.y;
    }
  }
  a = narrow<TYPE>(x);
  b = narrow<TYPE>(y);
}

// Where row i of a step goes: the request b with start[b] <= i < start[b + 1]
// (by a warp: 32 requests a round), its position, page and row of the page.
// Everything is checked; a bad request is reported and has page -2, a row of no
// request -1.
struct RowPlace {
  int pos, page;
};
__device__ RowPlace find_row(const RowParams& p, int i, int lane) {
  int b;
  int first, last;
  if (p.start) {
    int lo = 0, hi = p.B;  // start[lo] <= i (taken for granted at 0), start[hi] > i or hi = B
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + (lane + 1) * step;
      const bool before = at < hi && p.start[at] <= i;
      const int n = __popc(__ballot_sync(0xffffffffu, before));
      lo += n * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    first = p.start[b];
    last = p.start[b + 1];
    if (first < 0 || first > last || last > p.T) {
      if (lane == 0) report_error(p.err, kErrInput);
      return {0, -2};
    }
    if (i < first || i >= last) return {0, -1};
  } else {
    b = i / p.per;
    first = b * p.per;
    last = first + p.per;
  }
  const int len = p.lens[b];
  if (len < 0 || (int64_t)len + (last - first) > (int64_t)p.max_blocks * 64) {
    if (lane == 0) report_error(p.err, kErrInput);
    return {0, -2};
  }
  const int pos = len + (i - first);
  const int page = p.table[(int64_t)b * p.max_blocks + pos / 64];
  if (page < 0 || page >= p.pages) {
    if (lane == 0) report_error(p.err, kErrInput);
    return {pos, -3};
  }
  return {pos, page};
}

// One row a CTA. Rotated heads: x (rope) or q, then k (append); copied: v.
template <int TYPE, bool APPEND>
__global__ void __launch_bounds__(kRowThreads) rope_rows_kernel(const RowParams p) {
  extern __shared__ float2 row_cs[];  // [rot / 2]
  __shared__ RowPlace s_place;
  const int tid = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const int row = blockIdx.x;
  RowPlace place{0, 0};
  if constexpr (APPEND) {
    if (row == 0 && p.start)  // rows out of order are found wherever they are
      for (int b = tid; b < p.B; b += kRowThreads)
        if (p.start[b + 1] < p.start[b]) report_error(p.err, kErrInput);
    if (tid < 32) {
      const RowPlace r = find_row(p, row, tid);
      if (tid == 0) s_place = r;
    }
    __syncthreads();
    place = s_place;
    if (place.page == -1 || place.page == -2) return;
  } else {
    place.pos = p.positions[row];
  }
  for (int i = tid; i < p.rot / 2; i += kRowThreads) {
    const uint64_t turns = p.turns[i] * (uint64_t)(int64_t)(p.inverse ? -(int64_t)place.pos : (int64_t)place.pos);
    row_cs[i] = cos_sin((uint32_t)(turns >> 32), p.factor);
  }
  __syncthreads();
  const int D = p.D, units = p.rot / 16, rest = (D - p.rot) / 8;
  const int64_t page_row = ((int64_t)place.page * p.Hkv * 64 + place.pos % 64) * D;
  const bool stored = !APPEND || place.page >= 0;
  // head h's source and destination (null: none)
  auto head = [&](int h, const void*& src, int64_t& from, void*& dst, int64_t& to) {
    if (h < p.Hq) {
      src = p.q;
      from = (int64_t)row * p.q_stride + (int64_t)h * D;
      dst = p.q_out;
      to = (int64_t)row * p.out_stride + (int64_t)h * D;
    } else {
      const bool key = h < p.Hq + p.Hkv;
      const int g = h - p.Hq - (key ? 0 : p.Hkv);
      src = key ? p.k_new : p.v_new;
      from = (int64_t)row * (key ? p.k_stride : p.v_stride) + (int64_t)g * D;
      dst = stored ? (key ? p.k : p.v) : nullptr;
      to = page_row + (int64_t)g * 64 * D;
    }
  };
  const int turned = p.Hq + (APPEND ? p.Hkv : 0);
  const int second = p.inter ? 8 : p.rot / 2, width = p.inter ? 16 : 8;
  for (int i = tid; i < turned * units; i += kRowThreads) {
    const int h = i / units, u = i - h * units;
    const void* src;
    void* dst;
    int64_t from, to;
    head(h, src, from, dst, to);
    if (!dst) continue;
    Eight<TYPE> a = load8<TYPE>(src, from + width * u), b = load8<TYPE>(src, from + width * u + second);
    turn_unit<TYPE>(a, b, row_cs, u, p.inter != 0);
    store8<TYPE>(dst, to + width * u, a);
    store8<TYPE>(dst, to + width * u + second, b);
  }
  const int copies = turned * rest + (APPEND ? p.Hkv * (D / 8) : 0);
  for (int i = tid; i < copies; i += kRowThreads) {
    int h, at;
    if (i < turned * rest) {
      h = i / rest;
      at = p.rot + 8 * (i - h * rest);
    } else {
      const int j = i - turned * rest;
      h = j / (D / 8);
      at = 8 * (j - h * (D / 8));
      h += turned;
    }
    const void* src;
    void* dst;
    int64_t from, to;
    head(h, src, from, dst, to);
    if (dst) store8<TYPE>(dst, to + at, load8<TYPE>(src, from + at));
  }
}

template <bool APPEND>
static cudaError_t launch_rows(const RowParams& p, int type, cudaStream_t stream) {
  const dim3 grid((unsigned)p.T), block(kRowThreads);
  const size_t smem = (size_t)p.rot / 2 * sizeof(float2);
  switch (type) {
    case 0: return launch_pdl(rope_rows_kernel<0, APPEND>, grid, block, smem, stream, p);
    case 1: return launch_pdl(rope_rows_kernel<1, APPEND>, grid, block, smem, stream, p);
    default:
      if constexpr (APPEND)
        return cudaErrorInvalidValue;
      else
        return launch_pdl(rope_rows_kernel<2, false>, grid, block, smem, stream, p);
  }
}

cudaError_t launch_rope(const RowParams& p, int type, cudaStream_t stream) {
  return launch_rows<false>(p, type, stream);
}
cudaError_t launch_kv16_append(const RowParams& p, int type, cudaStream_t stream) {
  return launch_rows<true>(p, type, stream);
}

}  // namespace w4a16
