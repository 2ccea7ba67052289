// Causal attention of a step's new rows over the paged 16-bit cache (contract in w4a16sv.h).
//
// A row at position p of its request sees the keys max(0, p - window + 1) .. p:
// out = sum_j softmax_j(scale q . k_j) v_j, a warp a row and query head, the
// running maximum and sum of the softmax in fp32.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_float(__half x) {
  return __half2float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float(float x) {
  return __float2half_rn(x);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) kv16_attention_rows_kernel(const Kv16AttnParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)p.T * p.H) return;
  if (item == 0 && p.start)  // rows out of order are found wherever they are
    for (int i = lane; i < p.B; i += 32)
      if (p.start[i + 1] < p.start[i]) report_error(p.err, kErrInput);
  const int row = (int)(item / p.H), h = (int)(item % p.H);
  int b = 0, first = 0, last = 0;
  for (; b < p.B; ++b) {
    first = p.start ? p.start[b] : b * p.per;
    last = p.start ? p.start[b + 1] : first + p.per;
    if (row >= first && row < last) break;
  }
  if (b == p.B) return;
  const int len = p.lens[b];
  if (first < 0 || last > p.T || len < 0 || (int64_t)len + (last - first) > (int64_t)p.max_blocks * 64) {
    if (lane == 0) report_error(p.err, kErrInput);
    return;
  }
  constexpr int E = D / 32;
  const int pos = len + row - first, kvh = h / (p.H / p.Hkv);
  const T* qr = static_cast<const T*>(p.q) + (int64_t)row * p.q_stride + (int64_t)h * D;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_float<T>(qr[lane + 32 * e]) * p.scale_log2;
    o[e] = 0.0f;
  }
  for (int j = p.window > 0 ? max(0, pos - p.window + 1) : 0; j <= pos; ++j) {
    const int page = p.table[(int64_t)b * p.max_blocks + j / 64];
    const bool there = page >= 0 && page < p.pages;
    if (!there && lane == 0) report_error(p.err, kErrInput);
    const int64_t at = (((int64_t)page * p.Hkv + kvh) * 64 + j % 64) * D;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s += q[e] * (there ? to_float<T>(static_cast<const T*>(p.k)[at + lane + 32 * e]) : 0.0f);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float mx = fmaxf(m, s), c = exp2f(m - mx), w = exp2f(s - mx);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * c + w * (there ? to_float<T>(static_cast<const T*>(p.v)[at + lane + 32 * e]) : 0.0f);
    m = mx;
  }
  T* out = static_cast<T*>(p.out) + ((int64_t)row * p.H + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = from_float<T>(o[e] / l);
}

size_t kv16_attention_ws(int rows, int H, int Hkv, int D, int num_sms) { return 0; }

cudaError_t launch_kv16_attention(const Kv16AttnParams& p, int type, int D, void* workspace, int num_sms,
                                  cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)p.T * p.H + 3) / 4)), block(128);
  if (type == 0)
    return D == 128 ? launch_pdl(kv16_attention_rows_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, p)
                    : launch_pdl(kv16_attention_rows_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, p);
  return D == 128 ? launch_pdl(kv16_attention_rows_kernel<__half, 128>, grid, block, 0, stream, p)
                  : launch_pdl(kv16_attention_rows_kernel<__half, 64>, grid, block, 0, stream, p);
}

}  // namespace w4a16
