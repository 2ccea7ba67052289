// Tree-masked verify attention over the paged 8-bit cache (contract in
// w4a16sv.h): the first, plain form. A warp takes one query row (request,
// node, head) and walks over its keys: the request's full blocks, its tail
// rows, the tree's own rows on the node's root path; lane l holds columns
// 4 l .. 4 l + 3. Everything in fp32.
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

constexpr int kKaD = 128;
constexpr int kKaWarps = 4;

template <int FMT>
__device__ __forceinline__ float4 ka_decode(uint32_t w) {
  constexpr __nv_fp8_interpretation_t t = FMT == 0 ? __NV_E4M3 : __NV_E5M2;
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), t));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), t));
  const float2 x = __half22float2(a), y = __half22float2(b);
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 ka_bf16(uint2 w) {
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

struct KaRow {  // the online softmax of one query row
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __device__ void add(float4 q, float4 k, float4 v) {
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s), c = mn == -INFINITY ? 1.0f : exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * c + w;
    o.x = o.x * c + w * v.x;
    o.y = o.y * c + w * v.y;
    o.z = o.z * c + w * v.z;
    o.w = o.w * c + w * v.w;
  }
};

template <int FMT>
__global__ void __launch_bounds__(32 * kKaWarps) kv8_attention_plain_kernel(const Kv8AttnParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kKaWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)p.B * p.n * p.H) return;
  const int h = (int)(row % p.H), j = (int)(row / p.H % p.n), b = (int)(row / p.H / p.n);
  const int kvh = h / (p.H / p.Hkv);
  int len = p.lens[b];
  if (len < 0 || len > p.max_len) {
    if (lane == 0) report_error(p.err, kErrInput);
    len = len < 0 ? 0 : p.max_len;
  }
  float4 q = ka_bf16(*reinterpret_cast<const uint2*>(p.q + ((int64_t)b * p.n + j) * p.q_stride + h * kKaD + 4 * lane));
  q.x *= p.scale_log2;
  q.y *= p.scale_log2;
  q.z *= p.scale_log2;
  q.w *= p.scale_log2;
  KaRow st;
  for (int blk = 0; blk < len / 64; ++blk) {
    const int page = p.table[(int64_t)b * p.max_blocks + blk];
    const bool ok = page >= 0 && page < p.pages;
    if (!ok && lane == 0) report_error(p.err, kErrInput);
    const int64_t at = ok ? (int64_t)page * p.Hkv + kvh : 0;
    const float sk = ok ? p.k_scale[at] : 0.0f, sv = ok ? p.v_scale[at] : 0.0f;
    for (int r = 0; r < 64; ++r) {
      float4 k = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = k;
      if (ok) {
        k = ka_decode<FMT>(*reinterpret_cast<const uint32_t*>(p.k + (at * 64 + r) * kKaD + 4 * lane));
        v = ka_decode<FMT>(*reinterpret_cast<const uint32_t*>(p.v + (at * 64 + r) * kKaD + 4 * lane));
      }
      st.add(q, make_float4(k.x * sk, k.y * sk, k.z * sk, k.w * sk),
             make_float4(v.x * sv, v.y * sv, v.z * sv, v.w * sv));
    }
  }
  const int tail = p.tails[b];
  if (len % 64 > 0 && (tail < 0 || tail >= p.tail_pages)) {
    if (lane == 0) report_error(p.err, kErrInput);
  } else {
    for (int r = 0; r < len % 64; ++r) {
      const int64_t at = (((int64_t)tail * p.Hkv + kvh) * 64 + r) * kKaD + 4 * lane;
      st.add(q, ka_bf16(*reinterpret_cast<const uint2*>(p.k_tail + at)),
             ka_bf16(*reinterpret_cast<const uint2*>(p.v_tail + at)));
    }
  }
  for (int a = j; a >= 0;) {
    const int64_t at = ((int64_t)b * p.n + a) * p.kv_stride + kvh * kKaD + 4 * lane;
    st.add(q, ka_bf16(*reinterpret_cast<const uint2*>(p.k_new + at)),
           ka_bf16(*reinterpret_cast<const uint2*>(p.v_new + at)));
    const int up = p.parents ? p.parents[(int64_t)b * p.n + a] : a - 1;
    if (a == 0 ? up != -1 : (up < 0 || up >= a)) {
      if (lane == 0) report_error(p.err, kErrInput);
      break;
    }
    a = up;
  }
  const float inv = 1.0f / st.l;
  __nv_bfloat16* out = p.out + row * kKaD + 4 * lane;
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(st.o.x * inv, st.o.y * inv);
  *reinterpret_cast<__nv_bfloat162*>(out + 2) = __floats2bfloat162_rn(st.o.z * inv, st.o.w * inv);
}

size_t kv8_attention_ws(int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv8_attention(const Kv8AttnParams& p, int fmt, void*, int, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.B * p.n * p.H;
  const dim3 grid((unsigned)((rows + kKaWarps - 1) / kKaWarps)), block(32 * kKaWarps);
  return fmt == 0 ? launch_pdl(kv8_attention_plain_kernel<0>, grid, block, 0, stream, p)
                  : launch_pdl(kv8_attention_plain_kernel<1>, grid, block, 0, stream, p);
}

}  // namespace w4a16
