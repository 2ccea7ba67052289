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
// of a draft step over many layers latency. Which pieces there are is known on
// the device alone, so the CTAs (eight an SM) first sum up the requests' pages
// from the plan, each for itself, and then take (page, layer, head) items in
// turn, the even CTAs the keys and the odd ones the values, and after them the
// tail rows, (request, group of layer-heads) by (request, group): no CTA is
// launched for work that is not there (one CTA for every piece that might exist
// took 33 us for 80 layers of 16 drafts).
// Measured: prompts of 29364 rows (8 heads, 182 MB; 7344 page items, six in turn
// a CTA) 36 us, 0.74 of the HBM copy rate; 46 rows of 16 drafts in 80 layers (60
// MB, half of it the one block that completes: 1280 page items, a second one for
// 64 of the 1216 CTAs, then the tail rows) 14.9 us, 0.60; 64 rows of one layer
// 3.7 us. Against what there was at
// the time: keys and values by the same CTA (256 threads, four an SM) 37.3, 16.8
// and 4.4 us against 37.9, 16.4 and 3.8; the next item's words on their way
// meanwhile (in registers, or copied to shared memory asynchronously) 41 to 45 us
// for the prompts against 40; integer divisions for layers and tail rows 37.9 and
// 16.4 us against 36.0 and 14.9.
#include <cuda_fp8.h>
#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kAppThreads = 128;
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
  int group;   // (layer, head) pairs of a tail item
  FastDiv by_heads;
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

__device__ __forceinline__ void kv8_mul2(float a, float b, float inv, float& x, float& y) {
  asm("{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmul.rn.f32x2 v, v, s;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(inv));
}

template <int FMT>
__device__ __forceinline__ uint32_t kv8_pack4(uint32_t a, uint32_t b, float inv) {
  // four bf16 (two words) -> four codes
  float x0, x1, x2, x3;
  kv8_mul2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), inv, x0, x1);
  kv8_mul2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u), inv, x2, x3);
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
__global__ void __launch_bounds__(kAppThreads, 8) kv8_append_kernel(const AppendParams p) {
  extern __shared__ int app_smem[];
  __shared__ unsigned s_max[2][kAppThreads / 32];
  __shared__ int s_src[2][64];
  __shared__ int2 s_at[2][2];
  __shared__ int s_sum[kAppThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B;
  int* pre = app_smem;          // [B + 1] pages completed by the requests before
  int* first = pre + B + 1;     // [B] first kept row
  int* count = first + B;       // [B] kept rows, times 64, plus the block's rows before this step
  grid_launch_dependents();
  grid_dependency_wait();
  // ---- the requests: rows, the open block's fill, pages. Thread tid sums a
  // run of them
  const int per = (B + kAppThreads - 1) / kAppThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int i0 = p.new_start[b], i1 = p.new_start[b + 1];
    int n = i1 - i0, t = 0, full = 0;
    if (i0 < 0 || i1 > p.rows || n < 0) {
      if (blockIdx.x == 0) report_error(p.err, kErrInput);
      n = 0;
    }
    if (n > 0) {
      const int s = p.slots[i0];
      t = s >= 0 ? s & 63 : -1 - s;
      if (t > 63) {  // no slot (INT_MIN: its page was bad)
        if (blockIdx.x == 0) report_error(p.err, kErrInput);
        n = t = 0;
      }
      full = s >= 0 ? (t + n) / 64 : 0;
    }
    first[b] = i0;
    count[b] = n * 64 + t;
    pre[b] = full;
    mine += full;
  }
  int x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int at = x - mine, pages = 0;
#pragma unroll
  for (int w = 0; w < kAppThreads / 32; ++w) {
    at += w < warp ? s_sum[w] : 0;
    pages += s_sum[w];
  }
  for (int b = b0; b < b1; ++b) {
    const int full = pre[b];
    pre[b] = at;
    at += full;
  }
  if (tid == 0) pre[B] = pages;
  __syncthreads();
  const int pairs = p.layers * p.Hkv;

  // ---- pages: thread (row group, 8 columns), rows g, g + 8, .. of the block
  // in registers
  const int half = blockIdx.x & 1, g = tid >> 4, c = (tid & 15) * 8;
  const __nv_bfloat16* src_new = half ? p.v_new : p.k_new;
  const __nv_bfloat16* src_tail = half ? p.v_tail : p.k_tail;
  uint8_t* codes = half ? p.v : p.k;
  float* scales = half ? p.v_scale : p.k_scale;
  // item i is page i / pairs and layer-head i % pairs; a CTA's items are step
  // apart, kept as both parts
  struct Item {
    int pc, lh;
  };
  const int step = (int)gridDim.x >> 1, step_pc = step / pairs, step_lh = step - step_pc * pairs;
  auto after = [&](Item i) {
    i.pc += step_pc;
    i.lh += step_lh;
    if (i.lh >= pairs) {
      i.lh -= pairs;
      ++i.pc;
    }
    return i;
  };
  // Two warps find an item's rows (a thread a row) one item ahead of the CTA:
  // source rows, -1 - block row for those in the tail page; the page, -1 if
  // anything fits no plan
  auto find = [&](int pc, int to) {
    int b = 0;  // the request: the last one with pre[b] <= pc
    for (int hi = B - 1; b < hi;) {
      const int mid = (b + hi + 1) >> 1;
      if (pre[mid] <= pc)
        b = mid;
      else
        hi = mid - 1;
    }
    const int k0 = pc - pre[b], t = count[b] & 63;
    const int r0 = k0 == 0 ? t : 0;           // the block's new rows: r0 .. 63
    const int base = first[b] + k0 * 64 - t;  // kept row at block row r: base + r
    const int slot = p.slots[base + r0], page = slot >> 6, tail = p.tails[b];
    bool bad = slot < 0 || page >= p.pages || (r0 > 0 && (tail < 0 || tail >= p.tail_pages));
    int src = -1 - tid;
    if (tid >= r0) {
      src = p.src_rows[base + tid];
      bad = bad || src < 0 || src >= p.rows || p.slots[base + tid] != page * 64 + tid;
    }
    s_src[to][tid] = src;
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) s_at[to][warp] = make_int2(bad ? -1 : page, tail);
  };
  int buf = 0;
  Item item;
  item.pc = (int)(blockIdx.x >> 1) / pairs;
  item.lh = (int)(blockIdx.x >> 1) - item.pc * pairs;
  if (item.pc < pages && tid < 64) find(item.pc, 0);
  __syncthreads();
  for (Item next = item; item.pc < pages; item = next, buf ^= 1) {
    const int lh = item.lh, layer = p.by_heads(lh), h = lh - layer * p.Hkv;
    const int page = min(s_at[buf][0].x, s_at[buf][1].x), tail = s_at[buf][0].y;
    const __nv_bfloat16* a = src_new + layer * p.layer_stride + h * kAppD + c;
    const __nv_bfloat16* o = src_tail + (((int64_t)layer * p.tail_pages + tail) * p.Hkv + h) * 64 * kAppD + c;
    uint4 v[8];
    unsigned m = 0;
    if (page >= 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int src = s_src[buf][8 * k + g];
        v[k] = __ldg(reinterpret_cast<const uint4*>(src < 0 ? o + (-1 - src) * kAppD : a + (int64_t)src * p.row_stride));
      }
    }
    next = after(item);
    if (next.pc < pages && tid < 64) find(next.pc, buf ^ 1);
    if (page >= 0) {
      // the two halves of the words side by side; where anything is not finite
      // again, without that
      unsigned m2 = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m2 = __vimax3_u16x2(m2, v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu);
        m2 = __vimax3_u16x2(m2, v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu);
      }
      m = max(m2 & 0xFFFFu, m2 >> 16);
      if (m >= 0x7F80u) {
        m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          m = max(m, max(max(kv8_mag(v[k].x), kv8_mag(v[k].y)), max(kv8_mag(v[k].z), kv8_mag(v[k].w))));
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s_max[buf][warp] = m;
    __syncthreads();  // one an item: the next one writes the other buffers
    if (page < 0) {
      if (tid == 0) report_error(p.err, kErrInput);
      continue;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) m = max(m, s_max[buf][w]);
    const int k2 = kv8_exponent<FMT>(m);
    const float inv = __uint_as_float((unsigned)(127 - k2) << 23);  // 2^-k2, k2 in -100 .. 120
    const int64_t to = (((int64_t)layer * p.pages + page) * p.Hkv + h);
    if (!in_bounds(p.err, to, (int64_t)p.layers * p.pages * p.Hkv)) continue;
    if (tid == 0) scales[to] = __uint_as_float((unsigned)(127 + k2) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<uint2*>(codes + (to * 64 + 8 * k + g) * kAppD + c) =
          make_uint2(kv8_pack4<FMT>(v[k].x, v[k].y, inv), kv8_pack4<FMT>(v[k].z, v[k].w, inv));
  }

  // ---- tail rows: the request's last (t + n) % 64 block rows, those of them
  // that are new; 16 words of 16 bytes a row, keys and values. The last CTAs
  // first (the first ones may have had a page more).
  const int groups = (pairs + p.group - 1) / p.group;
  const int64_t tails = (int64_t)B * groups;
  for (int64_t item = gridDim.x - 1 - blockIdx.x; item < tails; item += gridDim.x) {
    const int b = (int)(item / groups), lh0 = (int)(item - (int64_t)b * groups) * p.group;
    const int n = count[b] >> 6, t = count[b] & 63, full = pre[b + 1] - pre[b];
    const int r0 = full > 0 ? 0 : t, r1 = t + n - full * 64;  // block rows
    if (n == 0 || r1 <= r0) continue;
    const int base = first[b] + full * 64 - t, tail = p.new_tails[b];
    bool bad = r1 > 64 || tail < 0 || tail >= p.tail_pages;
    if (!bad && tid >= r0 && tid < r1) {
      const int src = p.src_rows[base + tid];
      bad = src < 0 || src >= p.rows || p.slots[base + tid] != -1 - tid;
    }
    if (__syncthreads_or(bad)) {
      if (tid == 0) report_error(p.err, kErrInput);
      continue;
    }
    const int total = (r1 - r0) * 32 * min(p.group, pairs - lh0);
    // q / rows for q < 1024 by 2^20 / rows rounded up (1 to 64 rows, 16 pairs)
    const int rows = r1 - r0, inv = (1 << 20) / rows + 1;
    constexpr int kBatch = 4;  // words a thread holds: their loads are in flight together
    for (int w0 = tid; w0 < total; w0 += kBatch * kAppThreads) {
      uint4 v[kBatch];
      int64_t to[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int w = w0 + k * kAppThreads;
        if (w < total) {
          const int q = w >> 5, d = w & 31;  // d: 0 .. 15 keys, 16 .. 31 values
          const int dl = (q * inv) >> 20, r = r0 + q - dl * rows;
          const int lh = lh0 + dl, layer = p.by_heads(lh), h = lh - layer * p.Hkv;
          v[k] = __ldg(reinterpret_cast<const uint4*>((d < 16 ? p.k_new : p.v_new) + layer * p.layer_stride +
                                                      (int64_t)p.src_rows[base + r] * p.row_stride + h * kAppD +
                                                      (d & 15) * 8));
          to[k] = ((((int64_t)layer * p.tail_pages + tail) * p.Hkv + h) * 64 + r) * kAppD + (d & 15) * 8;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (w0 + k * kAppThreads < total &&
            in_bounds(p.err, to[k] + 7, (int64_t)p.layers * p.tail_pages * p.Hkv * 64 * kAppD))
          *reinterpret_cast<uint4*>(((tid & 31) < 16 ? p.k_tail : p.v_tail) + to[k]) = v[k];
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
  // eight CTAs an SM (their registers), fewer where there is less that could be
  // done: pages (one a request at most, and one for every 64 rows) and tails
  const int64_t pairs = (int64_t)layers * Hkv, most = (int64_t)num_sms * 8;
  int64_t group = (int64_t)B * pairs / (2 * most);  // tail items of two CTAs' turns, 1 .. 16 pairs each
  group = group < 1 ? 1 : group > 16 ? 16 : group;
  p.group = (int)group;
  p.by_heads = fast_div((uint32_t)Hkv);
  const int64_t items = 2 * (rows / 64 + (int64_t)B) * pairs, tail_items = B * ((pairs + group - 1) / group);
  const int64_t ctas = items > tail_items ? items : tail_items;
  const dim3 grid((unsigned)(ctas < most ? ctas + (ctas & 1) : most));
  const size_t smem = ((size_t)3 * B + 1) * sizeof(int);
  auto kernel = fmt == 0 ? kv8_append_kernel<0> : kv8_append_kernel<1>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, grid, dim3(kAppThreads), smem, stream, p);
}

}  // namespace w4a16
