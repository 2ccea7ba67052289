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
// Measured: 16381 rows of 72 heads 92.8 us (604 MB: 0.96 of the HBM copy rate), fp32
// 179 (1.21 GB, 0.99), 4093 rows of 40 heads, half of each turned in pairs, 10.4 us (84
// MB, in part in the L2), 12.0 K rows of 64 + 16 heads into pages 105 us (655 MB,
// 0.92); 80 rows 3.1 us, 64 rows into pages 5.1. Rows of few heads leave most of a
// CTA's threads without an item: 32768 rows of one head of 64 take 34.5 us (8.5 MB:
// 0.04), of 8 heads of 128 40 (134 MB, 0.49), 12 K rows of 8 + 8 heads into pages
// without queries 26 (98 MB, 0.56), of 1 + 1 18 (0.10). What keeps the memory busy is
// bytes in flight and CTAs at once: 128 threads, five items each, eight CTAs an SM;
// against 92, 104 us there were 96, 110 with 192 threads (5 CTAs), 105, 110 with 256 and three items
// (5), 95, 101 with 256 and one (8), 130, 142 with ten CTAs (registers spilled), and
// 104, 123 with the loads behind the sines.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kRowThreads = 128;
constexpr int kRowBlocks = 8;  // CTAs an SM
// items whose loads a thread has in flight (fp32: what the registers hold)
template <int TYPE>
constexpr int kRowFlight = TYPE == 2 ? 2 : 5;

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
  for (int i = 0; i < (TYPE == 2 ? 2 : 1); ++i)
    e.w[i] = s[i];
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

// Half layout: the pairs 8 u .. 8 u + 7, a their first elements, b their second ones.
template <int TYPE>
__device__ __forceinline__ void turn_halves(Eight<TYPE>& a, Eight<TYPE>& b, const float2* cs) {
  float x[8], y[8];
  widen<TYPE>(a, x);
  widen<TYPE>(b, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 c = cs[i];
    const float u = x[i], v = y[i];
    x[i] = u * c.x - v * c.y;
    y[i] = v * c.x + u * c.y;
  }
  a = narrow<TYPE>(x);
  b = narrow<TYPE>(y);
}
// Interleaved: four pairs side by side.
template <int TYPE>
__device__ __forceinline__ void turn_pairs(Eight<TYPE>& a, const float2* cs) {
  float x[8];
  widen<TYPE>(a, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = cs[i];
    const float u = x[2 * i], v = x[2 * i + 1];
    x[2 * i] = u * c.x - v * c.y;
    x[2 * i + 1] = v * c.x + u * c.y;
  }
  a = narrow<TYPE>(x);
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

// One row a CTA. Rotated heads: x (rope) or q, then k (append); copied: v. A head
// is so many items: eight pairs (half layout) or eight elements (interleaved) to
// turn, then eight elements to copy. A thread takes every 128th item, kRowFlight at
// a time, and loads the first ones before it waits for the sines.
template <int TYPE, bool APPEND, bool INTER>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) rope_rows_kernel(const RowParams p, const FastDiv by_items,
                                                                const FastDiv by_eighths) {
  extern __shared__ float2 row_cs[];  // [rot / 2]
  __shared__ RowPlace s_place;
  const int tid = threadIdx.x, row = blockIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const int D = p.D, half = p.rot / 2, turns = INTER ? p.rot / 8 : p.rot / 16, items = (int)by_items.d;
  const int turned = (p.Hq + (APPEND ? p.Hkv : 0)) * items, total = turned + (APPEND ? p.Hkv * (D / 8) : 0);
  struct Item {
    int head, at;  // head of the row (q's, then k's, then v's), first element
    bool turn;
  };
  auto item = [&](int i) {
    Item t;
    if (!APPEND || i < turned) {
      t.head = by_items(i);
      const int u = i - t.head * items;
      t.turn = u < turns;
      t.at = t.turn ? 8 * u : p.rot + 8 * (u - turns);
    } else {
      const int h = by_eighths(i - turned);
      t.head = p.Hq + p.Hkv + h;
      t.turn = false;
      t.at = 8 * (i - turned - h * (D / 8));
    }
    return t;
  };
  Eight<TYPE> a[kRowFlight<TYPE>], b[kRowFlight<TYPE>];
  auto load = [&](int first) {
#pragma unroll
    for (int k = 0; k < kRowFlight<TYPE>; ++k) {
      const int i = first + k * kRowThreads;
      if (i >= total) break;
      const Item t = item(i);
      const void* src = p.q;
      int64_t from = (int64_t)row * p.q_stride + (int64_t)t.head * D;
      if (APPEND && t.head >= p.Hq) {
        const bool key = t.head < p.Hq + p.Hkv;
        src = key ? p.k_new : p.v_new;
        from = (int64_t)row * (key ? p.k_stride : p.v_stride) + (int64_t)(t.head - p.Hq - (key ? 0 : p.Hkv)) * D;
      }
      a[k] = load8<TYPE>(src, from + t.at);
      if (!INTER && t.turn) b[k] = load8<TYPE>(src, from + t.at + half);
    }
  };
  bool taken = true;  // (append: a row of no request is not read)
  if constexpr (APPEND) {
    if (row == 0 && p.start)  // rows out of order or outside are found wherever they are: no row of the step may lead to them
      for (int b = tid; b < p.B; b += kRowThreads) {
        const int first = p.start[b], last = p.start[b + 1];
        if (first < 0 || last < first || last > p.T) report_error(p.err, kErrInput);
      }
    taken = !p.start || row < p.start[p.B];
  }
  if (taken) load(tid);
  RowPlace place{0, 0};
  if constexpr (APPEND) {
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
  for (int i = tid; i < half; i += kRowThreads) {
    const uint64_t turn = p.turns[i] * (uint64_t)(int64_t)(p.inverse ? -(int64_t)place.pos : (int64_t)place.pos);
    row_cs[i] = cos_sin((uint32_t)(turn >> 32), p.factor);
  }
  __syncthreads();
  const int64_t page_row = ((int64_t)place.page * p.Hkv * 64 + place.pos % 64) * D;
  for (int first = tid; first < total; first += kRowFlight<TYPE> * kRowThreads) {
    if (first != tid || !taken) load(first);
#pragma unroll
    for (int k = 0; k < kRowFlight<TYPE>; ++k) {
      const int i = first + k * kRowThreads;
      if (i >= total) break;
      const Item t = item(i);
      if (t.turn) {
        if constexpr (INTER)
          turn_pairs<TYPE>(a[k], row_cs + t.at / 2);
        else
          turn_halves<TYPE>(a[k], b[k], row_cs + t.at);
      }
      void* dst = p.q_out;
      int64_t to = (int64_t)row * p.out_stride + (int64_t)t.head * D;
      if (APPEND && t.head >= p.Hq) {
        const bool key = t.head < p.Hq + p.Hkv;
        dst = key ? p.k : p.v;
        to = page_row + (int64_t)(t.head - p.Hq - (key ? 0 : p.Hkv)) * 64 * D;
        if (place.page < 0 || !in_bounds(p.err, to + t.at + (t.turn && !INTER ? half : 0) + 7,
                                         (int64_t)p.pages * p.Hkv * 64 * D))
          continue;
      }
      store8<TYPE>(dst, to + t.at, a[k]);
      if (!INTER && t.turn) store8<TYPE>(dst, to + t.at + half, b[k]);
    }
  }
}

template <int TYPE, bool APPEND>
static cudaError_t launch_rows_t(const RowParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.T), block(kRowThreads);
  const size_t smem = (size_t)p.rot / 2 * sizeof(float2);
  const int items = p.inter ? p.D / 8 : p.rot / 16 + (p.D - p.rot) / 8;
  const FastDiv by_items = fast_div((uint32_t)items), by_eighths = fast_div((uint32_t)(p.D / 8));
  if (p.inter) return launch_pdl(rope_rows_kernel<TYPE, APPEND, true>, grid, block, smem, stream, p, by_items, by_eighths);
  return launch_pdl(rope_rows_kernel<TYPE, APPEND, false>, grid, block, smem, stream, p, by_items, by_eighths);
}

cudaError_t launch_rope(const RowParams& p, int type, cudaStream_t stream) {
  return type == 0 ? launch_rows_t<0, false>(p, stream)
                   : type == 1 ? launch_rows_t<1, false>(p, stream) : launch_rows_t<2, false>(p, stream);
}
cudaError_t launch_kv16_append(const RowParams& p, int type, cudaStream_t stream) {
  return type == 0 ? launch_rows_t<0, true>(p, stream) : launch_rows_t<1, true>(p, stream);
}

}  // namespace w4a16
