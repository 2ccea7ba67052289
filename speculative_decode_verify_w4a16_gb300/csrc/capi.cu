// C-ABI layer of libw4a16sv: argument checks, dispatch, device state.
// Declarations and the contract of every entry point are in w4a16sv.h.
#include <math.h>

#include <mutex>

#include "../../include/w4a16sv.h"
#include "common.cuh"
#include "format.cuh"
#include <math.h>

#include "internal.h"

namespace w4a16 {

// Device error word (one per device that loads the library).
__device__ unsigned g_error_word;

namespace {
std::mutex g_mu;
DeviceInfo g_dev[64];
}  // namespace

cudaError_t device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_dev[dev].device != dev) {
    DeviceInfo d;
    d.device = dev;
    e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_error_word);
    if (e != cudaSuccess) return e;
    d.err = static_cast<unsigned*>(p);
    g_dev[dev] = d;
  }
  *out = g_dev[dev];
  return cudaSuccess;
}

cudaError_t linear_plan(int M, int64_t N, int64_t K, const DeviceInfo& dev, LinearPlan* plan,
                        size_t max_partial_bytes) {
  plan->use_tc = M >= kTcMinM;
  cudaError_t e;
  if (plan->use_tc) {
    e = tc_plan(M, N, K, dev, max_partial_bytes, &plan->tc);
    plan->workspace_bytes = tc_workspace_bytes(plan->tc);
  } else {
    e = skinny_plan(M, N, K, dev, max_partial_bytes, &plan->sk);
    plan->workspace_bytes = skinny_workspace_bytes(plan->sk);
  }
  return e;
}

cudaError_t launch_linear(const void* x, int M, int64_t K, const void* qw_packed, const void* sc_packed, int64_t N,
                          void* out, void* workspace, const LinearPlan& plan, const DeviceInfo& dev,
                          cudaStream_t stream) {
  if (plan.use_tc) return launch_tc(x, M, K, qw_packed, sc_packed, N, out, workspace, plan.tc, dev, stream);
  return launch_skinny(x, M, K, qw_packed, sc_packed, N, out, workspace, plan.sk, dev, stream);
}

}  // namespace w4a16

using namespace w4a16;

static inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static inline bool valid_nk(int64_t N, int64_t K) {
  return N > 0 && K > 0 && N % kUnitRows == 0 && K % kGroup == 0 && N <= (int64_t(1) << 20) &&
         K <= (int64_t(1) << 24);
}

extern "C" {

const char* w4a16_status_string(w4a16_status s) {
  switch (s) {
    case W4A16_OK: return "W4A16_OK";
    case W4A16_ERR_INVALID_ARG: return "W4A16_ERR_INVALID_ARG";
    case W4A16_ERR_UNSUPPORTED: return "W4A16_ERR_UNSUPPORTED";
    case W4A16_ERR_CUDA: return "W4A16_ERR_CUDA";
    case W4A16_ERR_DEVICE_TIMEOUT: return "W4A16_ERR_DEVICE_TIMEOUT";
    case W4A16_ERR_DEVICE_INPUT: return "W4A16_ERR_DEVICE_INPUT";
    case W4A16_ERR_WORKSPACE: return "W4A16_ERR_WORKSPACE";
    case W4A16_ERR_BOUNDS: return "W4A16_ERR_BOUNDS";
    default: return "W4A16_ERR_UNKNOWN";
  }
}

int w4a16_abi_version(void) { return 1; }

size_t w4a16_packed_weight_bytes(int64_t N, int64_t K) { return valid_nk(N, K) ? (size_t)(N * K / 2) : 0; }

size_t w4a16_packed_scale_bytes(int64_t N, int64_t K) { return valid_nk(N, K) ? (size_t)(N * K / 64) : 0; }

static bool item_args_ok(int64_t U, int C, int min_units) {
  return C >= 1 && U >= C && min_units >= 1 && U <= (int64_t(1) << 40);
}

int w4a16_item_rounds(int64_t U, int C, int min_units, int max_rounds, int64_t* rb) {
  if (!item_args_ok(U, C, min_units) || !rb) return 0;
  const ItemSched s = make_item_sched(U, C, min_units, max_rounds);
  for (int r = 0; r <= s.R; ++r) rb[r] = s.rb[r];
  return s.R;
}

int64_t w4a16_item_begin(int64_t U, int C, int min_units, int max_rounds, int i) {
  if (!item_args_ok(U, C, min_units)) return -1;
  const ItemSched s = make_item_sched(U, C, min_units, max_rounds);
  if (i < 0 || (int64_t)i > (int64_t)s.R * C) return -1;
  return item_begin(s, i);
}

int64_t w4a16_item_owner(int64_t U, int C, int min_units, int max_rounds, int64_t u) {
  if (!item_args_ok(U, C, min_units) || u < 0 || u >= U) return -1;
  return item_owner(make_item_sched(U, C, min_units, max_rounds), u);
}

w4a16_status w4a16_quantize(const float* w, int64_t N, int64_t K, uint32_t* qweight, uint16_t* scales,
                            void* stream) {
  if (!w || !qweight || !scales || !valid_nk(N, K)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(qweight, 4) || !aligned(scales, 2)) return W4A16_ERR_INVALID_ARG;
  return launch_quantize(w, N, K, qweight, scales, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

w4a16_status w4a16_prepack(const uint32_t* qweight, const uint16_t* scales, int64_t N, int64_t K,
                           void* qweight_packed, void* scales_packed, void* stream) {
  if (!qweight || !scales || !qweight_packed || !scales_packed || !valid_nk(N, K)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(qweight_packed, 16) || !aligned(scales_packed, 16) || !aligned(qweight, 4) || !aligned(scales, 2))
    return W4A16_ERR_INVALID_ARG;
  return launch_prepack(qweight, scales, N, K, static_cast<uint32_t*>(qweight_packed),
                        static_cast<uint16_t*>(scales_packed), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

static bool linear_shape_ok(int M, int64_t N, int64_t K) {
  return M >= 1 && M <= kTcMaxM && valid_nk(N, K) && K >= 1024;
}

size_t w4a16_linear_workspace_bytes(int M, int64_t N, int64_t K) {
  if (!linear_shape_ok(M, N, K)) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  LinearPlan plan;
  if (linear_plan(M, N, K, dev, &plan) != cudaSuccess) return 0;
  return plan.workspace_bytes;
}

w4a16_status w4a16_linear(const void* x, int M, int64_t K, const void* qweight_packed, const void* scales_packed,
                          int64_t N, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !qweight_packed || !scales_packed || !out) return W4A16_ERR_INVALID_ARG;
  if (M < 1 || !valid_nk(N, K)) return W4A16_ERR_INVALID_ARG;
  if (M > kTcMaxM || K < 1024) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(qweight_packed, 16) || !aligned(scales_packed, 16) || !aligned(out, 4))
    return W4A16_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return W4A16_ERR_WORKSPACE;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  LinearPlan plan;
  if (linear_plan(M, N, K, dev, &plan) != cudaSuccess) return W4A16_ERR_CUDA;
  if (workspace_bytes < plan.workspace_bytes) return W4A16_ERR_WORKSPACE;
  return launch_linear(x, M, K, qweight_packed, scales_packed, N, out, workspace, plan, dev,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

size_t w4a16_linear_logits_workspace_bytes(int M, int64_t N, int64_t K) {
  if (!linear_shape_ok(M, N, K)) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  TcPlan plan;
  if (tc_plan_fused(M, N, K, dev, &plan) != cudaSuccess) return 0;
  return tc_workspace_bytes(plan);
}

w4a16_status w4a16_linear_logits(const void* x, int M, int64_t K, const void* qweight_packed,
                                 const void* scales_packed, int64_t N, float* logits, float* row_stats,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !qweight_packed || !scales_packed || !logits || !row_stats) return W4A16_ERR_INVALID_ARG;
  if (M < 1 || !valid_nk(N, K)) return W4A16_ERR_INVALID_ARG;
  if (M > kTcMaxM || K < 1024) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(qweight_packed, 16) || !aligned(scales_packed, 16) || !aligned(logits, 4) ||
      !aligned(row_stats, 8))
    return W4A16_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return W4A16_ERR_WORKSPACE;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  TcPlan plan;
  if (tc_plan_fused(M, N, K, dev, &plan) != cudaSuccess) return W4A16_ERR_CUDA;
  if (workspace_bytes < tc_workspace_bytes(plan)) return W4A16_ERR_WORKSPACE;
  return launch_tc_fused(x, M, K, qweight_packed, scales_packed, N, logits, reinterpret_cast<float2*>(row_stats),
                         workspace, plan, dev, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

static bool accept_shape_ok(int B, int n, int V) {
  // grid rows: B * (2n + 1) statistics rows must fit one grid dimension
  return B >= 1 && B <= 32768 && n >= 1 && n <= 1024 && V >= 2 && V <= (1 << 20) &&
         (int64_t)B * (2 * n + 1) <= 65535;
}

size_t spec_accept_workspace_bytes(int B, int n, int V) {
  if (!accept_shape_ok(B, n, V)) return 0;
  return accept_plan(B, n, V).total;
}

static w4a16_status accept_impl(const float* p_logits, const float* q_logits, const int32_t* draft_ids,
                                const int32_t* tree_parents, const float* uniforms, int B, int n, int V,
                                int32_t* accepted_len, int32_t* next_token, int32_t* accepted_node, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!p_logits || !draft_ids || !accepted_len || !next_token) return W4A16_ERR_INVALID_ARG;
  if (accepted_node && !aligned(accepted_node, 4)) return W4A16_ERR_INVALID_ARG;
  if (!accept_shape_ok(B, n, V)) return W4A16_ERR_INVALID_ARG;
  if (q_logits && !uniforms) return W4A16_ERR_INVALID_ARG;
  if (q_logits && tree_parents && V > kAcceptTreeMaxV) return W4A16_ERR_UNSUPPORTED;
  if (V % 4 == 0 && (!aligned(p_logits, 16) || (q_logits && !aligned(q_logits, 16)))) return W4A16_ERR_INVALID_ARG;
  if (!aligned(p_logits, 4) || !aligned(draft_ids, 4) || !aligned(accepted_len, 4) || !aligned(next_token, 4))
    return W4A16_ERR_INVALID_ARG;
  const AcceptPlan plan = accept_plan(B, n, V);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < plan.total) return W4A16_ERR_WORKSPACE;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  cudaError_t e;
  if (q_logits && tree_parents)
    e = launch_accept_tree(p_logits, q_logits, draft_ids, tree_parents, uniforms, B, n, V, accepted_len, next_token,
                           accepted_node, dev.err, static_cast<cudaStream_t>(stream));
  else if (q_logits)
    e = launch_accept_seq(p_logits, q_logits, draft_ids, uniforms, B, n, V, accepted_len, next_token, workspace, plan,
                          dev.num_sms, dev.err, static_cast<cudaStream_t>(stream), nullptr, accepted_node);
  else
    e = launch_accept_greedy(p_logits, draft_ids, tree_parents, B, n, V, accepted_len, next_token, workspace, plan,
                             dev.err, static_cast<cudaStream_t>(stream), accepted_node);
  return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

w4a16_status spec_accept(const float* p_logits, const float* q_logits, const int32_t* draft_ids,
                         const int32_t* tree_parents, const float* uniforms, int B, int n, int V,
                         int32_t* accepted_len, int32_t* next_token, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return accept_impl(p_logits, q_logits, draft_ids, tree_parents, uniforms, B, n, V, accepted_len, next_token,
                     nullptr, workspace, workspace_bytes, stream);
}

w4a16_status spec_accept_node(const float* p_logits, const float* q_logits, const int32_t* draft_ids,
                              const int32_t* tree_parents, const float* uniforms, int B, int n, int V,
                              int32_t* accepted_len, int32_t* next_token, int32_t* accepted_node, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!accepted_node) return W4A16_ERR_INVALID_ARG;
  return accept_impl(p_logits, q_logits, draft_ids, tree_parents, uniforms, B, n, V, accepted_len, next_token,
                     accepted_node, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------- verify attention
static bool attn_shape_ok(int B, int n, int H, int Hkv, int Lcap, int max_len) {
  return B >= 1 && B <= 65535 && n >= 1 && H >= 1 && Hkv >= 1 && Hkv <= 65535 && H % Hkv == 0 && max_len >= 0 &&
         (int64_t)max_len + n <= Lcap && (int64_t)B * Hkv * Lcap <= INT32_MAX && (int64_t)n * H <= INT32_MAX;
}

size_t tree_attention_workspace_bytes(int B, int n, int H, int Hkv, int D, int Lcap, int max_len) {
  if (!attn_shape_ok(B, n, H, Hkv, Lcap, max_len) || D != 128 || n > 64) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  return attn_plan(B, n, H, Hkv, max_len, dev.num_sms).ws_bytes;
}

w4a16_status tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* lens,
                            const int32_t* tree_parents, int B, int n, int H, int Hkv, int D, int Lcap, int max_len,
                            float scale, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !lens || !out) return W4A16_ERR_INVALID_ARG;
  if (!attn_shape_ok(B, n, H, Hkv, Lcap, max_len) || !(scale > 0.0f) || !(scale < INFINITY))
    return W4A16_ERR_INVALID_ARG;
  if (D != 128 || n > 64) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lens, 4) ||
      (tree_parents && !aligned(tree_parents, 4)))
    return W4A16_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  const AttnPlan plan = attn_plan(B, n, H, Hkv, max_len, dev.num_sms);
  if (plan.ws_bytes > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < plan.ws_bytes))
    return W4A16_ERR_WORKSPACE;
  return launch_tree_attention(q, k_cache, v_cache, lens, tree_parents, B, n, H, Hkv, Lcap, max_len, scale, out,
                               workspace, plan, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

w4a16_status kv_compact(void* k_cache, void* v_cache, const int32_t* lens, const int32_t* tree_parents,
                        const int32_t* accepted_node, int B, int n, int Hkv, int D, int Lcap, int n_layers,
                        int32_t* new_lens, void* stream) {
  if (!k_cache || !v_cache || !lens || !accepted_node || !new_lens) return W4A16_ERR_INVALID_ARG;
  if (B < 1 || n < 1 || Hkv < 1 || D < 8 || D % 8 != 0 || Lcap < n || n_layers < 1 || n_layers > 65535)
    return W4A16_ERR_INVALID_ARG;
  // one tree node's keys and values of every head: at most 4096 16-byte words
  if (n > 64 || (int64_t)2 * Hkv * (D / 8) > 4096) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lens, 4) || !aligned(accepted_node, 4) ||
      !aligned(new_lens, 4) || (tree_parents && !aligned(tree_parents, 4)))
    return W4A16_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  return launch_kv_compact(k_cache, v_cache, lens, tree_parents, accepted_node, B, n, Hkv, D, Lcap, n_layers,
                           new_lens, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

w4a16_status spec_accept_prestat(const float* p_logits, const float* p_stats, const float* q_logits,
                                 const int32_t* draft_ids, const float* uniforms, int B, int n, int V,
                                 int32_t* accepted_len, int32_t* next_token, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!p_logits || !p_stats || !q_logits || !draft_ids || !uniforms || !accepted_len || !next_token)
    return W4A16_ERR_INVALID_ARG;
  if (!accept_shape_ok(B, n, V) || V % 32 != 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(p_logits, 16) || !aligned(q_logits, 16) || !aligned(p_stats, 8) || !aligned(draft_ids, 4) ||
      !aligned(uniforms, 4) || !aligned(accepted_len, 4) || !aligned(next_token, 4))
    return W4A16_ERR_INVALID_ARG;
  const AcceptPlan plan = accept_plan(B, n, V);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < plan.total) return W4A16_ERR_WORKSPACE;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  return launch_accept_seq(p_logits, q_logits, draft_ids, uniforms, B, n, V, accepted_len, next_token, workspace,
                           plan, dev.num_sms, dev.err, static_cast<cudaStream_t>(stream),
                           reinterpret_cast<const float2*>(p_stats)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

// ------------------------------------------------- paged 8-bit cache
w4a16_status kv_block_plan(const int32_t* lens, const int32_t* tails, const int32_t* row_start,
                           const int32_t* tree_parents, const int32_t* accepted_node, const int32_t* release, int B,
                           int n, int rows, int max_blocks, int ring_cap, int32_t* block_table, int32_t* free_ring,
                           const int32_t* queue, int32_t* new_lens, int32_t* new_tails, int32_t* new_start,
                           int32_t* new_queue, int32_t* src_rows, int32_t* slots, void* stream) {
  if (!lens || !tails || !block_table || !free_ring || !queue || !new_lens || !new_tails || !new_start || !new_queue)
    return W4A16_ERR_INVALID_ARG;
  if ((row_start != nullptr) == (accepted_node != nullptr) || (tree_parents && !accepted_node))
    return W4A16_ERR_INVALID_ARG;  // one of the two modes
  if (B < 1 || rows < 0 || max_blocks < 1 || ring_cap < 1 || (rows > 0 && (!src_rows || !slots)))
    return W4A16_ERR_INVALID_ARG;
  if (accepted_node && (n < 1 || (int64_t)B * n != rows)) return W4A16_ERR_INVALID_ARG;
  if (B > kPlanMaxB || (accepted_node && n > 64) || ring_cap > (1 << 25) || (int64_t)B * max_blocks > INT32_MAX ||
      max_blocks > (INT32_MAX - 63) / 64 || rows > (1 << 30))
    return W4A16_ERR_UNSUPPORTED;
  const void* all[] = {lens,  tails,    row_start, tree_parents, accepted_node, release,  block_table, free_ring,
                       queue, new_lens, new_tails, new_start,    new_queue,     src_rows, slots};
  for (const void* a : all)
    if (!aligned(a, 4)) return W4A16_ERR_INVALID_ARG;
  if (new_lens == lens || new_tails == tails || new_queue == queue) return W4A16_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  return launch_block_plan(lens, tails, row_start, tree_parents, accepted_node, release, B, n, rows, max_blocks,
                           ring_cap, block_table, free_ring, queue, new_lens, new_tails, new_start, new_queue,
                           src_rows, slots, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

// pages and heads of a cache: every index in 64-token rows fits int32
static bool kv8_cache_ok(int Hkv, int pages, int tail_pages) {
  return Hkv >= 1 && Hkv <= 65535 && pages >= 1 && pages <= (1 << 25) && tail_pages >= 1 &&
         (int64_t)pages * Hkv <= INT32_MAX && (int64_t)tail_pages * Hkv <= INT32_MAX;
}

w4a16_status kv8_append(const void* k_new, const void* v_new, int64_t row_stride, int64_t layer_stride,
                        const int32_t* tails, const int32_t* new_tails, const int32_t* new_start,
                        const int32_t* src_rows, const int32_t* slots, int B, int rows, int Hkv, int D, int layers,
                        int pages, int tail_pages, int fmt, void* k, void* v, float* k_scale, float* v_scale,
                        void* k_tail, void* v_tail, void* stream) {
  if (!k_new || !v_new || !tails || !new_tails || !new_start || !src_rows || !slots || !k || !v || !k_scale ||
      !v_scale || !k_tail || !v_tail)
    return W4A16_ERR_INVALID_ARG;
  if (B < 1 || rows < 1 || layers < 1 || !kv8_cache_ok(Hkv, pages, tail_pages) || fmt < 0 || fmt > 1 ||
      row_stride < (int64_t)Hkv * D || row_stride % 8 != 0 || layer_stride < 0 || layer_stride % 8 != 0)
    return W4A16_ERR_INVALID_ARG;
  if (D != 128 || B > kPlanMaxB || rows > (1 << 24) || (int64_t)layers * Hkv > (1 << 24)) return W4A16_ERR_UNSUPPORTED;
  const void* wide[] = {k_new, v_new, k, v, k_tail, v_tail};
  for (const void* a : wide)
    if (!aligned(a, 16)) return W4A16_ERR_INVALID_ARG;
  const void* words[] = {tails, new_tails, new_start, src_rows, slots, k_scale, v_scale};
  for (const void* a : words)
    if (!aligned(a, 4)) return W4A16_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  return launch_kv8_append(k_new, v_new, row_stride, layer_stride, tails, new_tails, new_start, src_rows, slots, B,
                           rows, Hkv, layers, pages, tail_pages, fmt, k, v, k_scale, v_scale, k_tail, v_tail,
                           dev.num_sms, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

static bool kv8_attn_shape_ok(int B, int n, int H, int Hkv, int max_len) {
  return B >= 1 && B <= 65535 && n >= 1 && H >= 1 && Hkv >= 1 && Hkv <= 65535 && H % Hkv == 0 && max_len >= 0 &&
         (int64_t)B * n * H <= INT32_MAX && (int64_t)B * Hkv <= INT32_MAX;
}

size_t kv8_tree_attention_workspace_bytes(int B, int n, int H, int Hkv, int D, int max_len) {
  if (!kv8_attn_shape_ok(B, n, H, Hkv, max_len) || D != 128 || n > 64) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  return kv8_attention_ws(n, H, Hkv, dev.num_sms);
}

w4a16_status kv8_tree_attention(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                                int64_t kv_stride, const void* k, const void* v, const float* k_scale,
                                const float* v_scale, const void* k_tail, const void* v_tail,
                                const int32_t* block_table, const int32_t* lens, const int32_t* tails,
                                const int32_t* tree_parents, int B, int n, int H, int Hkv, int D, int max_blocks,
                                int pages, int tail_pages, int max_len, int fmt, float scale, void* out,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_new || !v_new || !k || !v || !k_scale || !v_scale || !k_tail || !v_tail || !block_table || !lens ||
      !tails || !out)
    return W4A16_ERR_INVALID_ARG;
  if (!kv8_attn_shape_ok(B, n, H, Hkv, max_len) || !kv8_cache_ok(Hkv, pages, tail_pages) || fmt < 0 || fmt > 1 ||
      max_blocks < 1 || max_len / 64 > max_blocks || (int64_t)B * max_blocks > INT32_MAX || q_stride < (int64_t)H * D ||
      q_stride % 8 != 0 || kv_stride < (int64_t)Hkv * D || kv_stride % 8 != 0 || !(scale > 0.0f) || !(scale < INFINITY))
    return W4A16_ERR_INVALID_ARG;
  if (D != 128 || n > 64 || kv_stride > (int64_t(1) << 31) || !kv8_attention_fits(B, n, H, Hkv, max_len))
    return W4A16_ERR_UNSUPPORTED;
  const void* wide[] = {q, k_new, v_new, k, v, k_tail, v_tail, out};
  for (const void* a : wide)
    if (!aligned(a, 16)) return W4A16_ERR_INVALID_ARG;
  const void* words[] = {k_scale, v_scale, block_table, lens, tails, tree_parents};
  for (const void* a : words)
    if (!aligned(a, 4)) return W4A16_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  const size_t need = kv8_attention_ws(n, H, Hkv, dev.num_sms);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  Kv8AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.q_stride = q_stride;
  p.kv_stride = kv_stride;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_tail = static_cast<const __nv_bfloat16*>(k_tail);
  p.v_tail = static_cast<const __nv_bfloat16*>(v_tail);
  p.table = block_table;
  p.lens = lens;
  p.tails = tails;
  p.parents = tree_parents;
  p.B = B;
  p.n = n;
  p.H = H;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks;
  p.pages = pages;
  p.tail_pages = tail_pages;
  p.max_len = max_len;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = dev.err;
  return launch_kv8_attention(p, fmt, workspace, dev.num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

// ------------------------------------------------- rotary positions
// rows of a tensor [T][heads][D]: `stride` elements apart
static bool rows_ok(const void* p, int64_t stride, int64_t heads, int D) {
  return aligned(p, 16) && stride >= heads * D && stride % 8 == 0;
}

static bool rotation_ok(const uint64_t* turns, int D, int rot, float factor) {
  return rot >= 0 && rot <= D && (rot == 0 || turns) && aligned(turns, 8) && factor > 0.0f && factor < INFINITY;
}

w4a16_status rope_rotate(const void* x, int64_t x_stride, const int32_t* positions, const uint64_t* turns, int T,
                         int heads, int D, int rot, int interleaved, float factor, int inverse, int type, void* y,
                         int64_t y_stride, void* stream) {
  if (!x || !positions || !turns || !y || T < 1 || heads < 1 || D < 1 || rot < 2 || type < 0 || type > 2)
    return W4A16_ERR_INVALID_ARG;
  if (!rotation_ok(turns, D, rot, factor) || !rows_ok(x, x_stride, heads, D) || !rows_ok(y, y_stride, heads, D) ||
      !aligned(positions, 4) || (x == y && x_stride != y_stride))
    return W4A16_ERR_INVALID_ARG;
  if (D % 8 != 0 || rot % 16 != 0 || D > 1024 || heads > (1 << 20)) return W4A16_ERR_UNSUPPORTED;
  RowParams p = {};
  p.q = x;
  p.q_stride = x_stride;
  p.q_out = y;
  p.out_stride = y_stride;
  p.positions = positions;
  p.turns = turns;
  p.factor = factor;
  p.T = T;
  p.Hq = heads;
  p.D = D;
  p.rot = rot;
  p.inter = interleaved != 0;
  p.inverse = inverse != 0;
  return launch_rope(p, type, static_cast<cudaStream_t>(stream)) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

// ------------------------------------------------- paged 16-bit cache
// a step's rows and the cache that they go to
static bool kv16_step_ok(const int32_t* row_start, int T, int B, int Hkv, int max_blocks, int pages) {
  return T >= 1 && B >= 1 && Hkv >= 1 && Hkv <= 65535 && pages >= 1 && max_blocks >= 1 &&
         max_blocks <= (INT32_MAX - 63) / 64 && (int64_t)B * max_blocks <= INT32_MAX &&
         (int64_t)pages * Hkv <= (1 << 25) && (row_start || T % B == 0);
}

w4a16_status kv16_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride, const void* q,
                         int64_t q_stride, const uint64_t* turns, int rot, int interleaved, float factor,
                         const int32_t* block_table, const int32_t* lens, const int32_t* row_start, int T, int B,
                         int H, int Hkv, int D, int max_blocks, int pages, int type, void* k, void* v, void* q_out,
                         int64_t q_out_stride, void* stream) {
  if (!k_new || !v_new || !block_table || !lens || !k || !v || (q != nullptr) != (q_out != nullptr))
    return W4A16_ERR_INVALID_ARG;
  if (!kv16_step_ok(row_start, T, B, Hkv, max_blocks, pages) || D < 1 || type < 0 || type > 1 ||
      (q && (H < 1 || !rows_ok(q, q_stride, H, D) || !rows_ok(q_out, q_out_stride, H, D))) ||
      (q == q_out && q_stride != q_out_stride))
    return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(k_new, k_stride, Hkv, D) || !rows_ok(v_new, v_stride, Hkv, D) ||
      !rotation_ok(turns, D, rot, factor) || !aligned(k, 16) || !aligned(v, 16) || !aligned(block_table, 4) ||
      !aligned(lens, 4) || !aligned(row_start, 4))
    return W4A16_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || rot % 16 != 0 || B > kPlanMaxB || T > (1 << 24) || (q && H > (1 << 20)))
    return W4A16_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  RowParams p = {};
  p.q = q;
  p.q_stride = q_stride;
  p.q_out = q_out;
  p.out_stride = q_out_stride;
  p.k_new = k_new;
  p.v_new = v_new;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.turns = turns;
  p.factor = factor;
  p.T = T;
  p.Hq = q ? H : 0;
  p.Hkv = Hkv;
  p.D = D;
  p.rot = rot;
  p.inter = interleaved != 0;
  p.start = row_start;
  p.lens = lens;
  p.table = block_table;
  p.B = B;
  p.per = T / B;
  p.max_blocks = max_blocks;
  p.pages = pages;
  p.k = k;
  p.v = v;
  p.err = dev.err;
  return launch_kv16_append(p, type, static_cast<cudaStream_t>(stream)) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

constexpr float kLog2e = 1.4426950408889634f;  // (weights are powers of two of the scores times the scale times this)
static bool kv16_attn_shape_ok(int T, int H, int Hkv) {
  return T >= 1 && H >= 1 && Hkv >= 1 && Hkv <= 65535 && H % Hkv == 0;
}
static bool kv16_attn_size_ok(int T, int H, int D) {
  return (D == 64 || D == 128) && T <= (1 << 24) && (int64_t)T * H <= INT32_MAX;
}

size_t kv16_attention_workspace_bytes(int T, int H, int Hkv, int D) {
  if (!kv16_attn_shape_ok(T, H, Hkv) || !kv16_attn_size_ok(T, H, D)) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  return kv16_attention_ws(T, H, Hkv, D, dev.num_sms);
}

w4a16_status kv16_attention(const void* q, int64_t q_stride, const void* k, const void* v, const int32_t* block_table,
                            const int32_t* lens, const int32_t* row_start, int T, int B, int H, int Hkv, int D,
                            int max_blocks, int pages, int window, float scale, int type, void* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !block_table || !lens || !out) return W4A16_ERR_INVALID_ARG;
  if (!kv16_attn_shape_ok(T, H, Hkv) || !kv16_step_ok(row_start, T, B, Hkv, max_blocks, pages) || D < 1 || type < 0 ||
      type > 1 || window < 0 || !rows_ok(q, q_stride, H, D) || !(scale > 0.0f) ||
      !(scale * kLog2e < INFINITY))
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(lens, 4) ||
      !aligned(row_start, 4))
    return W4A16_ERR_INVALID_ARG;
  if (!kv16_attn_size_ok(T, H, D) || B > kPlanMaxB || !kv16_attention_fits(T, B, H, Hkv, max_blocks))
    return W4A16_ERR_UNSUPPORTED;
  if (q == out && q_stride != (int64_t)H * D && T > 1) return W4A16_ERR_INVALID_ARG;  // (rows would lie over later ones)
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  const size_t need = kv16_attention_ws(T, H, Hkv, D, dev.num_sms);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  Kv16AttnParams p = {};
  p.q = q;
  p.q_stride = q_stride;
  p.k = k;
  p.v = v;
  p.start = row_start;
  p.lens = lens;
  p.table = block_table;
  p.T = T;
  p.B = B;
  p.per = T / B;
  p.H = H;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks;
  p.pages = pages;
  p.window = window >= (int64_t)max_blocks * 64 ? 0 : window;  // (a window past every position is none)
  p.scale_log2 = scale * kLog2e;
  p.out = out;
  p.err = dev.err;
  return launch_kv16_attention(p, type, D, workspace, dev.num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

// ------------------------------------------------- log probabilities
static bool logprobs_shape_ok(int R, int V, int m, int top) {
  return R >= 1 && R <= (1 << 20) && V >= 1 && V <= (1 << 20) && m >= 0 && m <= 64 && top >= 0 && top <= 64 &&
         top <= V && (int64_t)R * ((V + 7 + 1023) / 1024) < (int64_t(1) << 30);
}

size_t token_logprobs_workspace_bytes(int R, int V, int top) {
  return logprobs_shape_ok(R, V, 0, top) ? token_logprobs_ws(R, V) : 0;
}

w4a16_status token_logprobs(const void* logits, int bf16, const int32_t* ids, int R, int V, int m, int top,
                            float* logp, float* entropy, int32_t* top_ids, float* top_logp, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!logits || !logprobs_shape_ok(R, V, m, top) || bf16 < 0 || bf16 > 1) return W4A16_ERR_INVALID_ARG;
  if ((m > 0 && (!ids || !logp)) || (top > 0 && (!top_ids || !top_logp))) return W4A16_ERR_INVALID_ARG;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(ids, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return W4A16_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < token_logprobs_ws(R, V)) return W4A16_ERR_WORKSPACE;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  return launch_token_logprobs(logits, bf16 != 0, ids, R, V, m, top, logp, entropy, top_ids, top_logp, workspace,
                               dev.num_sms, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? W4A16_OK
             : W4A16_ERR_CUDA;
}

unsigned long long w4a16_stream_capture_id(void* stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream while another one captures: not in a capture itself)
    return 0;
  }
  return status == cudaStreamCaptureStatusNone ? 0 : id;
}

w4a16_status w4a16_check_device_status(void* stream) {
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return W4A16_ERR_CUDA;
  unsigned word = 0;
  if (cudaMemcpy(&word, dev.err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return W4A16_ERR_CUDA;
  if (word) {
    const unsigned zero = 0;
    if (cudaMemcpy(dev.err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return W4A16_ERR_CUDA;
  }
  if (word & kErrTimeout) return W4A16_ERR_DEVICE_TIMEOUT;
  if (word & kErrBounds) return W4A16_ERR_BOUNDS;
  if (word & kErrInput) return W4A16_ERR_DEVICE_INPUT;
  return W4A16_OK;
}

}  // extern "C"
