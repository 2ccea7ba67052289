// Block tables, slot maps and the free list of a step, from the requests'
// lengths (contract in w4a16sv.h).
//
// With kept[b] rows, need[b] = (lens + kept) / 64 - lens / 64 pages; request b
// is granted iff need[b] = 0 or need[0] + .. + need[b] <= free, and the page
// of its i-th new block is ring[head + (needs before b) + i]. Everything after
// the two prefix sums over the requests (needs, then granted rows) is
// independent, row by row and page by page.
//
// Bound: latency (a few dependent loads, two block scans); the largest case,
// 64 K rows of 1021 requests, moves 0.55 MB. So every CTA computes the sums
// over all requests itself (a few KB from L2) instead of waiting for another
// kernel or CTA, and the rows and pages are dealt over the grid. Measured: 16
// requests with a draft each 4.5 us, 1021 requests with 0 to 126 rows each 7.4 us;
// nearly all of it is the launch and the chain of loads and scans.
#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {

struct BlockPlanParams {
  const int32_t *lens, *tails, *row_start, *parents, *node, *release;
  int B, n, rows, max_blocks, ring_cap;
  int32_t *table, *ring;
  const int32_t* queue;
  int32_t *new_lens, *new_tails, *new_start, *new_queue, *src_rows, *slots;
  unsigned* err;
};

constexpr int kPlanMaxPage = 1 << 25;  // page * 64 + 63 fits int32

// shared memory per request (after the fixed words)
struct PlanArrays {
  int *start, *need, *back, *first, *len;
  uint64_t* path;
};

// Exclusive sums over the requests, in place, of N arrays at once (the barriers
// are what costs): a[k][0 .. B - 1] hold the counts on entry, a[k][B] the total
// on return. Every thread of the CTA calls it.
template <int N>
__device__ __forceinline__ void plan_scan(int* const (&a)[N], int B, int2* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int per = (B + blockDim.x - 1) / blockDim.x;
  const int i0 = min(B, (int)threadIdx.x * per), i1 = min(B, i0 + per);
  __syncthreads();  // the counts are written, and scratch is free
  int sum[2] = {0, 0}, x[2];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    for (int i = i0; i < i1; ++i) sum[k] += a[k][i];
    x[k] = sum[k];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x[k], d);
      if (lane >= d) x[k] += y;
    }
  }
  if (lane == 31) scratch[warp] = make_int2(x[0], N > 1 ? x[N - 1] : 0);
  __syncthreads();
  const int2 w2 = lane < nw ? scratch[lane] : make_int2(0, 0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int w = k ? w2.y : w2.x, total = __reduce_add_sync(0xffffffffu, w);
    int o = x[k] - sum[k] + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    for (int i = i0; i < i1; ++i) {
      const int c = a[k][i];
      a[k][i] = o;
      o += c;
    }
    if (threadIdx.x == 0) a[k][B] = total;
  }
  __syncthreads();
}

// the last i of 0 .. B - 1 with a[i] <= x (a rising, a[0] <= x)
__device__ __forceinline__ int plan_find(const int* a, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// place a, 0 <= a <= cap, behind place head of the ring
__device__ __forceinline__ int plan_ring(int head, int a, int cap) {
  const int i = head + a;
  return i >= cap ? i - cap : i;
}

__global__ void __launch_bounds__(1024) kv_block_plan_kernel(const BlockPlanParams p) {
  extern __shared__ uint64_t plan_smem[];
  __shared__ int2 scratch[32];
  const int B = p.B, tid = threadIdx.x, nt = blockDim.x;
  PlanArrays s;
  s.path = plan_smem;
  s.start = reinterpret_cast<int*>(plan_smem + (p.node ? B : 0));
  s.need = s.start + B + 1;
  s.back = s.need + B + 1;
  s.first = s.back + B + 1;
  s.len = s.first + B + 1;
  grid_launch_dependents();
  grid_dependency_wait();
  const bool say = blockIdx.x == 0;  // one CTA reports what all of them find
  int head = p.queue[0], count = p.queue[1];
  if (head < 0 || head >= p.ring_cap || count < 0 || count > p.ring_cap) {
    if (say && tid == 0) report_error(p.err, kErrInput);
    head = count = 0;
  }
  // ---- rows each request would keep
  if (p.node && p.parents) {
    // a warp a request: the parents in the lanes, the walk by shuffles
    const int lane = tid & 31;
    for (int b = tid >> 5; b < B; b += nt >> 5) {
      const int32_t* par = p.parents + (int64_t)b * p.n;
      const int p0 = lane < p.n ? par[lane] : -1, p1 = lane + 32 < p.n ? par[lane + 32] : -1;
      int j = p.node[b];
      bool bad = j < 0 || j >= p.n;
      uint64_t m = 0;
      if (bad) j = -1;
      while (j >= 0) {
        m |= 1ull << j;
        const int up = __shfl_sync(0xffffffffu, j < 32 ? p0 : p1, j & 31);
        if (j == 0 ? up != -1 : (up < 0 || up >= j)) {
          bad = true;
          break;
        }
        j = up;
      }
      if (lane == 0) {
        if (bad && say) report_error(p.err, kErrInput);
        s.path[b] = bad ? 1ull : m;
      }
    }
  } else if (p.node) {
    for (int b = tid; b < B; b += nt) {
      int j = p.node[b];
      if (j < 0 || j >= p.n) {
        if (say) report_error(p.err, kErrInput);
        j = 0;
      }
      s.path[b] = j == 63 ? ~0ull : (1ull << (j + 1)) - 1ull;
    }
  }
  __syncthreads();
  bool bad_rows = false;
  const int64_t cap_tokens = (int64_t)p.max_blocks * 64 + 63;
  for (int b = tid; b < B; b += nt) {
    int len = p.lens[b], first = 0;
    int64_t cnt;
    if (p.node) {
      cnt = __popcll(s.path[b]);
    } else {
      first = p.row_start[b];
      const int next = p.row_start[b + 1];
      cnt = (int64_t)next - first;
      bad_rows |= first < 0 || next > p.rows || cnt < 0;
    }
    const bool ended = p.release && p.release[b] != 0;
    if (len < 0 || len > cap_tokens) {  // a length the table cannot hold
      if (say) report_error(p.err, kErrInput);
      cnt = 0;
      s.len[b] = -1;
      len = 0;
    } else if (!ended && (len + cnt) / 64 > p.max_blocks) {
      if (say) report_error(p.err, kErrInput);
      cnt = 0;
      s.len[b] = len;
    } else {
      s.len[b] = len;
    }
    if (ended) cnt = 0;
    s.first[b] = first;
    s.need[b] = (int)((len + cnt) / 64 - len / 64);
    s.back[b] = ended ? len / 64 : 0;
    s.start[b] = (int)cnt;
  }
  // ranges that are not one after the other: whose a row is cannot be told, so
  // nobody keeps any
  if (__syncthreads_or(bad_rows)) {
    if (say && tid == 0) report_error(p.err, kErrInput);
    for (int b = tid; b < B; b += nt) s.start[b] = s.need[b] = 0;
  }
  {
    int* const pages[2] = {s.need, s.back};
    plan_scan(pages, B, scratch);
  }
  // ---- grants: need[] and back[] are sums before each request now
  __shared__ int taken_s;
  if (tid == 0) taken_s = 0;
  __syncthreads();
  int most = 0;
  for (int b = tid; b < B; b += nt) {
    const int upto = s.need[b + 1];
    if (upto > s.need[b]) {
      if (upto <= count)
        most = max(most, upto);
      else
        s.start[b] = 0;
    }
  }
  if (most) atomicMax(&taken_s, most);
  int* const granted[1] = {s.start};
  plan_scan(granted, B, scratch);  // the rows of granted requests
  const int taken = taken_s, asked = s.need[B], back = s.back[B], kept = s.start[B];
  const int gt = blockIdx.x * nt + tid, gn = gridDim.x * nt;

  // ---- per request
  for (int b = gt; b < B; b += gn) {
    const int len = s.len[b], cnt = s.start[b + 1] - s.start[b];
    const bool ended = p.release && p.release[b] != 0;
    const bool filled = cnt > 0 && (len + cnt) / 64 > len / 64;
    p.new_lens[b] = ended ? 0 : len < 0 ? p.lens[b] : len + cnt;
    const int tail = p.tails[b];
    p.new_tails[b] = filled ? tail ^ 1 : tail;
  }
  for (int b = gt; b <= B; b += gn) p.new_start[b] = s.start[b];
  const int room = p.ring_cap - count;  // ring places behind the last free page
  if (gt == 0) {
    if (back > room) report_error(p.err, kErrInput);
    p.new_queue[0] = plan_ring(head, taken, p.ring_cap);
    p.new_queue[1] = count - taken + min(back, room);
    p.new_queue[2] = asked - taken;
  }
  // ---- pages taken, and pages returned
  for (int a = gt; a < taken; a += gn) {
    const int b = plan_find(s.need, B, a);
    const int page = p.ring[plan_ring(head, a, p.ring_cap)];
    const bool bad = page < 0 || page >= kPlanMaxPage;
    if (bad) report_error(p.err, kErrInput);
    const int64_t at = (int64_t)b * p.max_blocks + s.len[b] / 64 + (a - s.need[b]);
    if (in_bounds(p.err, at, (int64_t)(b + 1) * p.max_blocks)) p.table[at] = bad ? -1 : page;
  }
  for (int a = gt; a < min(back, room); a += gn) {
    const int b = plan_find(s.back, B, a);
    p.ring[plan_ring(plan_ring(head, count, p.ring_cap), a, p.ring_cap)] = p.table[(int64_t)b * p.max_blocks + (a - s.back[b])];
  }
  // ---- rows
  for (int r = gt; r < p.rows; r += gn) {
    if (r >= kept) {
      p.src_rows[r] = -1;
      p.slots[r] = INT_MIN;
    }
    int b, off;
    bool keep;
    if (p.node) {
      b = r / p.n;
      const int j = r - b * p.n;
      keep = (s.path[b] >> j) & 1ull;
      off = __popcll(s.path[b] & ((1ull << j) - 1ull));
    } else {
      b = plan_find(s.first, B, r);
      off = r - s.first[b];
      keep = off >= 0;
    }
    const int cnt = s.start[b + 1] - s.start[b];
    if (keep && off < cnt) {
      const int len = s.len[b], i = s.start[b] + off, pos = len + off;
      if (!in_bounds(p.err, i, p.rows)) continue;
      p.src_rows[i] = r;
      int slot = -1 - pos % 64;
      if (pos / 64 < (len + cnt) / 64) {
        const int page = p.ring[plan_ring(head, s.need[b] + (pos / 64 - len / 64), p.ring_cap)];
        slot = page < 0 || page >= kPlanMaxPage ? INT_MIN : page * 64 + pos % 64;
      }
      p.slots[i] = slot;
    }
  }
}

size_t block_plan_smem(int B, bool draft) { return (draft ? (size_t)B * 8 : 0) + ((size_t)B + 1) * 5 * sizeof(int); }

cudaError_t launch_block_plan(const int32_t* lens, const int32_t* tails, const int32_t* row_start,
                              const int32_t* parents, const int32_t* node, const int32_t* release, int B, int n,
                              int rows, int max_blocks, int ring_cap, int32_t* table, int32_t* ring,
                              const int32_t* queue, int32_t* new_lens, int32_t* new_tails, int32_t* new_start,
                              int32_t* new_queue, int32_t* src_rows, int32_t* slots, unsigned* err,
                              cudaStream_t stream) {
  const BlockPlanParams p = {lens,  tails, row_start, parents,  node,      release,   B,         n,        rows,  max_blocks,
                             ring_cap, table, ring,   queue,    new_lens,  new_tails, new_start, new_queue, src_rows, slots,
                             err};
  const int work = rows > B ? rows : B;
  const int threads = work <= 1024 ? 256 : 1024;
  const int ctas = (work + threads - 1) / threads;
  const size_t smem = block_plan_smem(B, node != nullptr);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_block_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kv_block_plan_kernel, dim3((unsigned)(ctas < 64 ? ctas : 64)), dim3((unsigned)threads), smem,
                    stream, p);
}

}  // namespace w4a16
