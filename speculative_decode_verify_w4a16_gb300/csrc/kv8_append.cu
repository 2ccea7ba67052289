// The kept rows of a step into the paged 8-bit cache (contract in w4a16sv.h).
//
// A request's kept rows go to consecutive positions, so they fall into pieces
// of its 64-token blocks: the first one may continue the block being filled
// (its older rows are in the tail page), the last one may leave a block open.
// A piece that ends its block becomes a page: amax over the block's finite
// magnitudes, scale = 2^k with the smallest k >= -100 for which amax / 2^k is
// no larger than the largest code (0.875 * 2^T: T = 9 for e4m3, 16 for e5m2),
// codes = x * 2^-k rounded to nearest even. A power of two makes x * 2^-k and
// code * scale exact in fp32 (and bf16): one rounding per value, and nothing
// is lost against amax / largest (the codes are floating point). The other
// pieces copy their rows.
//
// Bound: HBM (each row read and written once) for prompts; for the few rows
// of a draft step over many layers the chain of dependent loads (piece ->
// source rows -> values) per CTA. A CTA therefore takes one piece and walks
// over `heads` (layer, head) pairs of it: the piece is found once, and a copy
// deals all of the pairs' rows over its threads at once.
#include <cuda_fp8.h>
#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kAppThreads = 256;  // the first half takes the keys, the second the values
constexpr int kAppD = 128;

struct AppendParams {
  const __nv_bfloat16 *k_new, *v_new;
  int64_t row_stride, layer_stride;
  const int32_t *tails, *new_tails, *new_start, *src_rows, *slots;
  int B, rows, Hkv, layers, pages, tail_pages;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  __nv_bfloat16 *k_tail, *v_tail;
  unsigned* err;
  int heads;  // (layer, head) pairs per CTA
};

// exponent k of the scale for the largest finite magnitude's bf16 bits
template <int FMT>
__device__ __forceinline__ int kv8_exponent(unsigned amax_bits) {
  constexpr int top = FMT == 0 ? 9 : 16;
  if (amax_bits == 0) return 0;
  // 1.f * 2^(e - 127) <= 1.75 * 2^(top - 1 + k), f <= .75 on the smaller side
  const int e = (int)(amax_bits >> 7) - 127, f = (int)(amax_bits & 0x7Fu);
  const int k = e + 1 - top + (f > 0x60 ? 1 : 0);
  return k < -100 ? -100 : k;
}

template <int FMT>
__device__ __forceinline__ uint32_t kv8_pack4(uint32_t a, uint32_t b, float inv) {
  // four bf16 (two words) -> four codes
  const float x0 = __uint_as_float(a << 16) * inv, x1 = __uint_as_float(a & 0xFFFF0000u) * inv;
  const float x2 = __uint_as_float(b << 16) * inv, x3 = __uint_as_float(b & 0xFFFF0000u) * inv;
  constexpr __nv_fp8_interpretation_t t = FMT == 0 ? __NV_E4M3 : __NV_E5M2;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, t);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, t);
  return lo | (hi << 16);
}

// magnitude bits of the larger finite one of a word's two bf16
__device__ __forceinline__ unsigned kv8_mag(uint32_t w) {
  const unsigned lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u);
}

template <int FMT>
__global__ void __launch_bounds__(kAppThreads, 4) kv8_append_kernel(const AppendParams p) {
  __shared__ int s_src[64];
  __shared__ unsigned s_max[2][kAppThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // ---- the request: piece numbers from new_start[b] / 64 + 2 b on are b's
  // (it has at most kept / 64 + 2 of them). Every warp searches, 32 requests
  // a step.
  const int f = blockIdx.x;
  int lo = 0, hi = p.B;  // the last b of lo .. hi - 1 whose first number is <= f
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const bool le = b < hi && p.new_start[b] / 64 + 2 * b <= f;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // a prefix of the lanes
    const int at = lo + max(c - 1, 0) * step;
    hi = min(hi, at + step);
    lo = at;
  }
  const int b = lo;
  const int i0 = p.new_start[b], i1 = p.new_start[b + 1];
  if (i0 < 0 || i1 > p.rows || i1 < i0) {
    if (tid == 0) report_error(p.err, kErrInput);
    return;
  }
  if (i1 == i0) return;
  const int piece = f - (i0 / 64 + 2 * b);
  const int first = p.slots[i0];
  const int t = first >= 0 ? first & 63 : -1 - first;  // the block's rows before this step
  if (t > 63) {  // no slot (INT_MIN: its page was bad)
    if (tid == 0) report_error(p.err, kErrInput);
    return;
  }
  const int cnt = i1 - i0;
  if (piece >= (t + cnt + 63) / 64) return;
  const int r0 = piece == 0 ? t : 0;              // the piece's new rows: r0 .. r1 - 1 of the block
  const int r1 = min(64, t + cnt - piece * 64);
  const int base = i0 + piece * 64 - t;            // kept row at block row r: base + r
  // ---- source rows and slots: all new rows agree on the page (or the tail)
  const int s0 = p.slots[base + r0];
  const bool page_piece = s0 >= 0;
  bool bad = page_piece ? r1 != 64 || (s0 >> 6) >= p.pages : false;
  if (tid < 64) {
    int src = -1;
    if (tid >= r0 && tid < r1) {
      src = p.src_rows[base + tid];
      bad = bad || src < 0 || src >= p.rows || p.slots[base + tid] != (page_piece ? (s0 & ~63) + tid : -1 - tid);
    }
    s_src[tid] = src;
  }
  const int tail_old = p.tails[b], tail_new = p.new_tails[b];
  if (page_piece ? r0 > 0 && (tail_old < 0 || tail_old >= p.tail_pages) : (tail_new < 0 || tail_new >= p.tail_pages))
    bad = true;
  if (__syncthreads_or(bad)) {
    if (tid == 0) report_error(p.err, kErrInput);
    return;
  }
  const int lh0 = blockIdx.y * p.heads, lh1 = min(p.layers * p.Hkv, lh0 + p.heads);
  if (!page_piece) {
    // ---- copy: rows r0 .. r1 - 1, 16 words of 16 bytes each, keys and values
    const int per = (r1 - r0) * 32, total = (lh1 - lh0) * per;
    constexpr int kBatch = 4;  // words a thread holds: their loads are in flight together
    for (int w0 = tid; w0 < total; w0 += kBatch * kAppThreads) {
      uint4 x[kBatch];
      int64_t to[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int w = w0 + k * kAppThreads;
        if (w < total) {
          const int lh = lh0 + w / per, rest = w % per;
          const int r = r0 + (rest >> 5), c = rest & 31;  // c: 0 .. 15 keys, 16 .. 31 values
          const int layer = lh / p.Hkv, h = lh % p.Hkv;
          x[k] = __ldg(reinterpret_cast<const uint4*>((c < 16 ? p.k_new : p.v_new) + layer * p.layer_stride +
                                                      (int64_t)s_src[r] * p.row_stride + h * kAppD + (c & 15) * 8));
          to[k] = ((((int64_t)layer * p.tail_pages + tail_new) * p.Hkv + h) * 64 + r) * kAppD + (c & 15) * 8;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (w0 + k * kAppThreads < total &&
            in_bounds(p.err, to[k] + 7, (int64_t)p.layers * p.tail_pages * p.Hkv * 64 * kAppD))
          *reinterpret_cast<uint4*>((((w0 + k * kAppThreads) & 31) < 16 ? p.k_tail : p.v_tail) + to[k]) = x[k];
    }
    return;
  }
  // ---- a page: 128 threads each for the keys and the values, thread (row
  // group, 8 columns): rows g, g + 8, .. of the block in registers
  const int half = tid >> 7, u = tid & 127, g = u >> 4, c = (u & 15) * 8;
  const __nv_bfloat16* src_new = half ? p.v_new : p.k_new;
  const __nv_bfloat16* src_tail = half ? p.v_tail : p.k_tail;
  uint8_t* codes = half ? p.v : p.k;
  float* scales = half ? p.v_scale : p.k_scale;
  const int page = s0 >> 6;
  int buf = 0;
  for (int lh = lh0; lh < lh1; ++lh, buf ^= 1) {
    const int layer = lh / p.Hkv, h = lh - layer * p.Hkv;
    const __nv_bfloat16* a = src_new + layer * p.layer_stride + h * kAppD + c;
    const __nv_bfloat16* o = src_tail + (((int64_t)layer * p.tail_pages + tail_old) * p.Hkv + h) * 64 * kAppD + c;
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 8 * k + g;
      x[k] = *reinterpret_cast<const uint4*>(r < r0 ? o + r * kAppD : a + (int64_t)s_src[r] * p.row_stride);
    }
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      m = max(m, max(max(kv8_mag(x[k].x), kv8_mag(x[k].y)), max(kv8_mag(x[k].z), kv8_mag(x[k].w))));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s_max[buf][warp] = m;
    __syncthreads();  // one a pair: the next one writes the other buffer
#pragma unroll
    for (int w = 0; w < 4; ++w) m = max(m, s_max[buf][half * 4 + w]);
    const int k2 = kv8_exponent<FMT>(m);
    const float inv = __uint_as_float((unsigned)(127 - k2) << 23);  // 2^-k2, k2 in -100 .. 119
    const int64_t at = (((int64_t)layer * p.pages + page) * p.Hkv + h);
    if (u == 0) scales[at] = __uint_as_float((unsigned)(127 + k2) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 8 * k + g;
      if (in_bounds(p.err, at, (int64_t)p.layers * p.pages * p.Hkv))
        *reinterpret_cast<uint2*>(codes + (at * 64 + r) * kAppD + c) =
            make_uint2(kv8_pack4<FMT>(x[k].x, x[k].y, inv), kv8_pack4<FMT>(x[k].z, x[k].w, inv));
    }
  }
}

cudaError_t launch_kv8_append(const void* k_new, const void* v_new, int64_t row_stride, int64_t layer_stride,
                              const int32_t* tails, const int32_t* new_tails, const int32_t* new_start,
                              const int32_t* src_rows, const int32_t* slots, int B, int rows, int Hkv, int layers,
                              int pages, int tail_pages, int fmt, void* k, void* v, float* k_scale, float* v_scale,
                              void* k_tail, void* v_tail, int num_sms, unsigned* err, cudaStream_t stream) {
  AppendParams p;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.row_stride = row_stride;
  p.layer_stride = layer_stride;
  p.tails = tails;
  p.new_tails = new_tails;
  p.new_start = new_start;
  p.src_rows = src_rows;
  p.slots = slots;
  p.B = B;
  p.rows = rows;
  p.Hkv = Hkv;
  p.layers = layers;
  p.pages = pages;
  p.tail_pages = tail_pages;
  p.k = static_cast<uint8_t*>(k);
  p.v = static_cast<uint8_t*>(v);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_tail = static_cast<__nv_bfloat16*>(k_tail);
  p.v_tail = static_cast<__nv_bfloat16*>(v_tail);
  p.err = err;
  // piece numbers: see the search in the kernel
  const int64_t numbers = rows / 64 + 2 * (int64_t)B;
  // pairs per CTA: all of a layer's heads as long as that leaves every SM
  // eight CTAs' worth of pieces, else fewer
  const int64_t pairs = (int64_t)layers * Hkv;
  int64_t heads = Hkv;
  while (heads > 1 && numbers * ((pairs + heads - 1) / heads) < 8 * (int64_t)num_sms) heads = (heads + 1) / 2;
  while ((pairs + heads - 1) / heads > 65535) heads *= 2;
  p.heads = (int)heads;
  const dim3 grid((unsigned)numbers, (unsigned)((pairs + heads - 1) / heads));
  return fmt == 0 ? launch_pdl(kv8_append_kernel<0>, grid, dim3(kAppThreads), 0, stream, p)
                  : launch_pdl(kv8_append_kernel<1>, grid, dim3(kAppThreads), 0, stream, p);
}

}  // namespace w4a16
