// Causal attention of a step's new rows over the paged 16-bit cache (contract in w4a16sv.h).
//
// A row at position p of its request sees the keys max(0, p - window + 1) .. p:
// out = sum_j softmax_j(scale q . k_j) v_j. The query rows of a key/value head
// are its G = H / Hkv query heads at every new token, row r = token * G +
// head-in-group, so that keys and values are read once for the group. A unit
// is 256 of those rows of one request and head, against 64-key tiles (pages)
// from the first key that any of its rows sees to the last.
//
// Split: the units of all requests end to end, by their estimated work, cut into
// one run a CTA (a CTA an SM), at tile boundaries. A unit that is cut leaves
// its pieces' references, sums and unnormalised outputs in the workspace, and the
// CTA that finishes last merges them, in the order of the keys: every CTA gets
// much the same work whatever the lengths are, decoding rows and prompts share a
// launch, the host needs no length, and no CTA waits for another. A cut costs some
// 10 to 18 thousand cycles (a part's start and end 3 to 9 thousand, a tile of two
// row tiles 1400, of one 600 to 800), so it moves to a unit's end where that is
// near, and few units get few CTAs. Many short units are taken whole from a queue
// instead; which CTA has a unit does not show in its rows.
//
// In a CTA (tcgen05, TMEM, TMA):
//   warp 0        the run's parts (a unit or a piece of one), published in a
//                 ring of descriptors; TMA copies of K and V tiles into a ring,
//                 K two tiles ahead of V, as they are used
//   warps 1, 2    the MMAs of slot 0 and 1: S = Q K^T (128 x 64 x D, both from
//                 shared memory) two tiles ahead of O += P V (P from TMEM, V as
//                 it was loaded: the MN-major operand)
//   warp 3        the guard: looks through the values of tiles that some row
//                 sees in part, and takes out NaN and infinities, which a weight
//                 of zero would not hide; rows that do see them get them added
//                 at the end
//   warps 4 - 11  the softmax of slot 0 and 1, one row a thread: scores from TMEM,
//                 weights and their sum in fp32, the weights rounded to the
//                 cache's type back into TMEM over the scores: the product takes
//                 both operands in one type. Each is off by half a step at most,
//                 and a row by that of its weighted magnitudes (the sum is that of
//                 the unrounded ones: it adds nothing)
// With more than 128 rows the two slots are two row tiles, which share every
// key tile; with fewer they take the key tiles in turn and are merged at the
// part's end. While one slot's softmax runs, the tensor pipe works for the other.
//
// Bound and measured (bf16, D 128, 64 heads over 8, unless said; times by events):
//   long contexts, 4 requests of 120 to 131 K, one row each: HBM, 302 us for 2.04 GB
//     (0.99 of a plain copy's rate)
//   64 and 256 requests of 1 to 8 K, one row each: 192 us for 1.18 GB (0.91), 678 for
//     4.72 (1.02); at fp16, D 64 117 and 427 (0.74, 0.81): half the bytes a tile, the
//     same hand-offs
//   16 requests of 4 to 8 K, 5 rows each: 80 us for 392 MB (0.72); a run is some 79
//     tiles, its start, end and merge a third of it
//   a chunk of 2048 rows after 30720: the tensor pipe and the softmax, 1.42 ms cold to
//     1.6 ms in a row (the clock falls): 1.5 to 1.33 PFLOP/s, 0.79 to 0.70 of the bf16
//     peak (fp16 1.46 ms; D 64, half the work, 1.11). Of some 1640 cycles a tile the
//     MMAs of both slots take 1250 (626 each, 392 of it S: with N = 64 a k-step takes 49
//     cycles for 32 of arithmetic, as shared memory gives 128 bytes a cycle), a slot's
//     softmax 1000 and its hand-offs 400; with one k-step of S in place of eight the chunk took 1.11 ms, without the softmax's
//     arithmetic no less than with it
//   7 prompts of up to 3002 rows, 16 heads of their own: 81 us, 0.45 of the peak;
//     parts of 4 to 47 tiles start and end in 7000 cycles, and masked tiles take more
//   49 requests, one in 8 a prompt, fp16, D 64, window 4096: 410 us, 0.36 of the
//     peak; softmax and hand-offs, some 1250 cycles a tile (the MMAs 700, the
//     exponentials 512)
// Tried and slower, or no better: 128-key tiles with one score buffer (chunk 1586 us
// when this form took 1500), a row's columns over two warpgroups, two warpgroups a
// slot taking its tiles in turn, one MMA warp for both slots (in turn, or whichever is
// ready), a slot's MMAs kept together (chunk 1500 -> 2010), the next scores loaded beside the store of the weights (mixed 429 -> 477),
// outputs through shared memory in whole lines (5 us of 100 for prompts), tiles that a warp
// does not see at all passed over (mixed 423 -> 435: the branch lengthens the others).
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "softmax.cuh"
#include "tcgen05.cuh"

namespace w4a16 {

constexpr int kCaThreads = 384;
constexpr int kCaKeys = 64;   // keys of a tile: a page
constexpr int kCaDesc = 4;    // parts described ahead
constexpr int kCaOk = 16;     // guarded tiles that the guard may be ahead: more than the ring holds
constexpr int kCaSpecial = 12;  // guarded tiles of a part, at most (256 tokens' own keys, and as many where a window ends)

// The weights a key tile has in the split: two row tiles, or one.
constexpr int kCaWeight2 = 8, kCaWeight1 = 5;
constexpr int kCaOverhead = 256;  // keys that a unit's start and end are worth
constexpr int kCaSnap = 16;       // tiles that a cut may move to the unit's begin or end,
constexpr int kCaSnapFew = 4;     // and where there are fewer units than CTAs
// What a cut is worth, in tiles of one row tile: by itself, and for each row of each piece (stored, fetched and added); and
// the tiles that a piece has at least. Measured: one row of 64 heads over 8 after 1003 tokens, units in 2 pieces 14.3 us, in
// 3 13.6, in 19 15.9; 300 rows of 32 heads over 8 after 1000, whole 27.6 us, in 3 pieces 64; the same after 8000 in 3 pieces
// 75 us, and 82 where cuts lay a tile or two beside the units' ends.
constexpr float kCaCut = 8.0f, kCaRowPiece = 0.056f, kCaLeast = 6.0f;

// Many short units are not cut into runs but taken from a queue, whole ones, a request's longest first: where no unit has
// more than kCaQueueTiles tiles and there are twice as many as CTAs, or four times the tiles and four times as many units.
// Measured, cut / queue, us (bf16, D 128, 64 heads over 8): 7 prompts of up to 3002 rows (16 heads of their own) 96 / 81, 64
// requests of up to 2000 tokens, one row each, 63 / 59, 32 prompts of up to 512 rows 125 / 110, 4 of 4000 rows 832 / 771, 49
// requests with a window of 4096 434 / 417; fewer and longer units, 64 requests of up to 4000 tokens (3.4 units of 32 tiles a
// CTA): 100.6 / 100.5; 256 of up to 6000 (13.5 of 47): 477 / 465.
// And where none is left to the end that is far longer than the others: with what its request's units are of a CTA's share
// taken off, the request's longest weighs no more than kCaQueueLate of them on average. (The queue has the requests in their
// order: behind the others it is what the call waits for.) 79 requests of 100 tokens and a last one of 1000 35 / 38, of 8000
// 42 / 87 (first 41 / 66); 200 of 100 and a last one of 4000 76 / 95 (first 76 / 71); 100 of 500 and a last one of 2000 56 / 66
// (first 57 / 55); 40 prompts of 100 rows and a last one of 2000 (16 heads of their own) 62 / 61 (first 62 / 51), of 3000 91 /
// 73. Sorted by length, which was tried, the queue needs no such rule, but evenly spread batches took 5 percent longer.
constexpr int kCaQueueTiles = 32;
constexpr float kCaQueueLate = 2.6f;
constexpr int kCaMany = 65535;  // units that are too many to be counted (more than any number of CTAs wants)

// Weights are taken against a reference: the largest score of the first tile that
// the row sees keys of. It is raised (and the sums so far, in TMEM, rescaled) by a
// tile whose weights, 64 at a time, add up to more than this; no weight is then
// larger, and no tile's maximum has to be found otherwise. In fp16 the reference
// itself stands for 2^8: weights fit up to 2^15, and down to 2^-22 of the
// reference they keep all their bits (2^-32: some).
template <int TYPE>
constexpr float kCaMost = TYPE == 0 ? 256.0f : 32768.0f;
template <int TYPE>
constexpr float kCaUp = TYPE == 0 ? 0.0f : 8.0f;
// A weight is 2^(s c - m), c the scale and m the reference times c, rounded, in one multiplication and addition: off by
// the rounding of m, 2^-24 |m| powers of two at most, by the same for all of a row's keys, so that it cancels. From 2^28 on in
// fp16, 2^32 in bf16, it passes what a weight holds. Rows that had a reference of this size are done over, key by key
// (ca_far_row): scores like that need not be fast (one row of 64 heads after 8000 tokens 1.25 ms), and the code for them in
// the tiles' loop cost the others 2 percent.
constexpr float kCaFar = 16777216.0f;

struct CaMaps {
  CUtensorMap k, v;  // [pages * Hkv][D / 64][64][64]: halves of 64 columns apart, as they lie in shared memory
};
struct CaWork {
  FastDiv by_g;
  int ctas, rows_cap;  // rows of a workspace slot
  int wide;            // out lies on 32 bytes
  uint64_t ctas_inv;   // floor(2^64 / ctas)
  float tiles_inv;     // a CTA's share of the split's work, in tiles by their weight, for 1
  int* done;           // [ctas] tiles of the unit that this CTA's first cut is in, finished
  int* queue;          // units taken, CTAs finished
  float2* part_ml;     // [2 * ctas][rows_cap] (reference, sum), log2 domain; a sum below zero: the row is to be done over
  float* part_o;       // [2 * ctas][rows_cap][D] unnormalised sums
};

// One part of a CTA's run: tiles lo .. hi - 1 of the nt tiles of a unit.
struct CaPart {
  int b, at, past, kvh;
  int row0, rows;    // the unit's rows (packed): row0 .. row0 + rows - 1
  int tile0, nt;     // the unit's first tile and their number
  int lo, hi;        // hi = 0: no more parts
  int gw, gc;        // tiles gw .. gc - 1 of the part are seen whole by every row; the others are masked and guarded
  int first_cut;     // cut units: the first CTA that begins inside this unit
  int last_key;      // the last key that any row sees
  int64_t u0, v;     // cut units: begin and extent in the split
};
struct CaSpecial {
  int key0;
  uint32_t keys[2];  // of the tile's 64: those with a value that is not finite
};
struct CaShared {
  uint64_t full[20], free[20];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], fin[2];
  uint64_t stat, read, stored, told;
  uint64_t landed[kCaOk], ok[kCaOk];  // guarded values: in shared memory, looked through
  uint64_t desc_full[kCaDesc], desc_free[kCaDesc], q_ready[2][kCaDesc];
  CaPart part[kCaDesc];
  int specials[kCaDesc];
  CaSpecial special[kCaDesc][kCaSpecial];
  uint32_t tmem;
  int last;
  unsigned beat;  // counts on as the producer, or a row that is done over, does
};

template <int D>
struct CaLayout {
  static constexpr int kQHalf = 128 * 128;  // 128 rows of 64 columns
  static constexpr int kQ = D / 64 * kQHalf;
  static constexpr int kHalf = kCaKeys * 128;  // 64 keys of 64 columns
  static constexpr int kTile = D / 64 * kHalf;
  static constexpr int kBufs = D == 128 ? 10 : 20;
  static constexpr int kRingOff = 2 * kQ;
  static constexpr int kSharedOff = kRingOff + kBufs * kTile;
  static constexpr int kTotal = kSharedOff + (int)sizeof(CaShared);
  static_assert(kTotal <= 227 * 1024, "shared memory");
  static_assert(kBufs <= 20 && kBufs / 2 < kCaOk, "rings");
};

// TMEM columns: a slot's two score buffers (a tile's weights over the first half of its scores), and its sums
__device__ __forceinline__ uint32_t ca_s_col(int t, int sb) { return 128u * (uint32_t)t + 64u * (uint32_t)sb; }
__device__ __forceinline__ uint32_t ca_o_col(int t) { return 256u + 128u * (uint32_t)t; }

// 16 bytes to shared memory, asynchronously; zeros where there are none.
__device__ __forceinline__ void ca_copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ca_copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The page's head z by TMA, counted on bar; by a whole warp, whose elected lane
// issues (from code that one lane alone runs, an issue takes several times as long).
__device__ __forceinline__ void ca_copy_tile(void* dst, const CUtensorMap* map, int32_t z, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%2], %4;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%5, %5, %5, %3}], "
      "[%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(z), "r"(bytes), "r"(0)
      : "memory");
}

// 32 bytes to global memory, at once where they lie on 32.
__device__ __forceinline__ void ca_store32(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Four MMAs of a k-step each, issued by one elected lane of a converged warp; the first adds to what is there if
// `accumulate`. SS: both operands from shared memory, K-major (32 bytes a step); TS: A from TMEM (8 columns a step), B
// MN-major (16 rows of 128 bytes).
__device__ __forceinline__ void ca_mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 b2, %2, 4;\n\t"
      "add.s64 a3, %1, 6;\n\tadd.s64 b3, %2, 6;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void ca_mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\tadd.u32 a2, %1, 16;\n\tadd.s64 b2, %2, 256;\n\t"
      "add.u32 a3, %1, 24;\n\tadd.s64 b3, %2, 384;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Bounded wait by a whole warp; false once it has run out: when kWaitLimitNs have passed in which the CTA's producer got no
// further. (It is not the wait itself that is bounded: the guard has nothing to do while a part's unmasked tiles pass by, which
// may be two million of them.) A test without a time answers in 45 cycles, and several at once in little more; one with a
// time takes 80, each for itself.
__device__ __noinline__ bool ca_wait_long(uint64_t* bar, uint32_t parity, unsigned* err, const unsigned* beat) {
  if (mbar_try_wait(bar, parity, 1000000u)) return true;  // (most end here: the clock is not read before)
  unsigned long long t0 = globaltimer_ns();
  unsigned last = *(volatile const unsigned*)beat;
  while (!mbar_try_wait(bar, parity, 1000000u)) {
    const unsigned long long t = globaltimer_ns();
    const unsigned now = *(volatile const unsigned*)beat;
    if (now != last) {
      last = now;
      t0 = t;
    } else if (t - t0 > kWaitLimitNs) {
      report_error(err, kErrTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool ca_wait(uint64_t* bar, uint32_t parity, unsigned* err, const unsigned* beat) {
  return mbar_try_wait(bar, parity) || ca_wait_long(bar, parity, err, beat);
}

#if W4A16_TEST_HOOKS
// Debug builds only: the producer of CTA 0 leaves out this buffer of its run (no
// copy, no arrival), so that the bounded waits run out. -1: off.
__device__ int g_test_skip_copy = -1;
__device__ __forceinline__ bool test_skip_copy(uint32_t buf) {
  return blockIdx.x == 0 && (int)buf == *(volatile int*)&g_test_skip_copy;
}
#else
__device__ __forceinline__ bool test_skip_copy(uint32_t) { return false; }
#endif

// ------------------------------------------------------------------ the split

// floor(a / b) for 0 <= a, b > 0 and a quotient below 2^22 (the fp32 estimate is
// off by less than one then, and put right); the whole number next to a * n / b for
// a < b, or one of the ends, if it is no more than `snap` from it. __fdividef: b
// below 2^126.
__device__ __forceinline__ int ca_fix(int q, int64_t a, int64_t b) {
  int64_t r = a - q * b;
  while (r < 0) r += b, --q;
  while (r >= b) r -= b, ++q;
  return q;
}
__device__ __forceinline__ int ca_quotient(int64_t a, int64_t b) { return ca_fix((int)__fdividef((float)a, (float)b), a, b); }
__device__ __forceinline__ int ca_share(int64_t a, int n, int64_t b, int snap) {
  const int q = ca_fix((int)(__fdividef((float)a, (float)b) * (float)n + 0.5f), 2 * a * n + b, 2 * b);
  return q <= min(snap, n / 2) ? 0 : n - q <= snap ? n : q;
}

// A request's rows: the first, their number (0 where it brings none or is not
// valid), and the tokens before them.
struct CaRequest {
  int at, cnt, past;
};
__device__ __forceinline__ CaRequest ca_request(const Kv16AttnParams& p, int b, bool report) {
  CaRequest r;
  r.at = p.start ? p.start[b] : b * p.per;
  const int end = p.start ? p.start[b + 1] : r.at + p.per;
  const int len = p.lens[b];  // (fetched with the others)
  r.cnt = 0;
  r.past = 0;
  if (r.at < 0 || end < r.at || end > p.T) {
    if (report) report_error(p.err, kErrInput);
    return r;
  }
  if (end == r.at) return r;
  r.past = len;
  if (r.past < 0 || (int64_t)r.past + (end - r.at) > (int64_t)p.max_blocks * 64) {
    if (report) report_error(p.err, kErrInput);
    return r;
  }
  r.cnt = end - r.at;
  return r;
}

// Estimated work of a request's units, per head: unit i has G (past + overhead) +
// 256 (i + 1), the keys of its last row times G, times a weight, and no more
// than a window's. Sums in closed form; every CTA computes the same numbers.
struct CaLoad {
  int64_t base, cap, overhead;
  int units, weight, capped;  // from unit `capped` on the window's extent
  __device__ __forceinline__ int64_t before(int i) const {  // units 0 .. i - 1
    const int64_t m = i < capped ? i : capped;
    return weight * (i * overhead + m * base + 128 * m * (m + 1) + (i - m) * cap);
  }
};
__device__ __forceinline__ CaLoad ca_load(const Kv16AttnParams& p, const CaWork& wk, const CaRequest& r) {
  const int G = (int)wk.by_g.d;
  CaLoad w;
  const int64_t rows = (int64_t)r.cnt * G;
  w.units = (int)((rows + 255) / 256);
  w.weight = rows > 128 ? kCaWeight2 : kCaWeight1;
  w.base = (int64_t)G * r.past;
  w.overhead = (int64_t)G * kCaOverhead;
  w.cap = 0;
  w.capped = w.units;
  if (p.window > 0) {
    w.cap = (int64_t)G * p.window + 256;
    const int64_t n = w.cap > w.base ? (w.cap - w.base + 255) / 256 - 1 : 0;  // units below the cap
    w.capped = n < w.units ? (int)n : w.units;
  }
  return w;
}

// The key tiles of a unit.
struct CaTiles {
  int first_pos, last_pos, tile0, nt;
};
__device__ __forceinline__ CaTiles ca_tiles(const Kv16AttnParams& p, const CaWork& wk, const CaRequest& r, int unit) {
  const int row0 = unit * 256, rows = r.cnt * (int)wk.by_g.d;
  CaTiles t;
  t.first_pos = r.past + wk.by_g(row0);
  t.last_pos = r.past + wk.by_g(min(row0 + 255, rows - 1));
  t.tile0 = p.window > 0 ? max(0, t.first_pos - p.window + 1) / kCaKeys : 0;
  t.nt = t.last_pos / kCaKeys + 1 - t.tile0;
  return t;
}

// Where a run begins: tile `cut` of a unit.
struct CaPlace {
  int b, kvh, unit, cut;
  int64_t u0, v;
  CaRequest r;
};
// The place of x in request b, whose work begins at `at` (at <= x < its end).
__device__ CaPlace ca_locate(const Kv16AttnParams& p, const CaWork& wk, int b, const CaRequest& r, int64_t at, int64_t x,
                             int snap) {
  const CaLoad w = ca_load(p, wk, r);
  const int64_t head = w.before(w.units);
  CaPlace o;
  o.b = b;
  o.kvh = ca_quotient(x - at, head);
  at += o.kvh * head;
  int lo = 0, hi = w.units;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (w.before(mid) <= x - at)
      lo = mid;
    else
      hi = mid;
  }
  o.unit = lo;
  o.u0 = at + w.before(lo);
  o.v = w.before(lo + 1) - w.before(lo);
  o.r = r;
  o.cut = ca_share(x - o.u0, ca_tiles(p, wk, r, lo).nt, o.v, snap);
  return o;
}

template <int TYPE>
__device__ __forceinline__ uint32_t ca_pack(float lo, float hi) {
  if constexpr (TYPE == 0) return pack_bf16_rn(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int TYPE>
constexpr uint32_t kCaExp = TYPE == 0 ? 0x7F807F80u : 0x7C007C00u;
template <int TYPE>
constexpr uint32_t kCaExpUnit = TYPE == 0 ? 0x00800080u : 0x04000400u;
// bit 15 and 31: the half's exponent is all ones (NaN or infinite)
template <int TYPE>
__device__ __forceinline__ uint32_t ca_not_finite(uint32_t w) {
  return ((w & kCaExp<TYPE>)+kCaExpUnit<TYPE>)&0x80008000u;
}

// two values times zero, added to acc
template <int TYPE>
__device__ __forceinline__ uint32_t ca_times_zero(uint32_t w, uint32_t acc) {
  uint32_t r;
  if constexpr (TYPE == 0)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
  return r;
}

// The values at `at` (D elements) that are not finite, added to an output row's columns c0 .. c0 + 31.
template <int TYPE>
__device__ __noinline__ void ca_add_special(const Kv16AttnParams& p, const CaShared* sh, int slot, int b, int kvh, int D,
                                            int pos, int c0, uint32_t* ov) {
  const int n = min(*(volatile const int*)&sh->specials[slot], kCaSpecial);
  for (int e = 0; e < n; ++e) {
    const CaSpecial& s = sh->special[slot][e];
    for (int r = 0; r < kCaKeys; ++r) {
      const int key = s.key0 + r;
      if (!((s.keys[r >> 5] >> (r & 31)) & 1u) || key > pos || (p.window > 0 && key <= pos - p.window)) continue;
      const int page = p.table[(int64_t)b * p.max_blocks + key / 64];
      if (page < 0 || page >= p.pages) continue;
      const uint16_t* v =
          static_cast<const uint16_t*>(p.v) + (((int64_t)page * p.Hkv + kvh) * 64 + key % 64) * D + c0;
      for (int c = 0; c < 32; ++c) {
        const uint32_t bits = v[c];
        if (!(ca_not_finite<TYPE>(bits) & 0x8000u)) continue;
        const float x = TYPE == 0 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
        ov[c] = __float_as_uint(__uint_as_float(ov[c]) + x);
      }
    }
  }
}

// the first or second value of a pair
template <int TYPE>
__device__ __forceinline__ float ca_value(uint32_t w, int half) {
  if constexpr (TYPE == 0) return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return half ? v.y : v.x;
}
// Row R of part d's request and head from the definition, by a warp, D / 32 columns a lane: differences of scores are taken
// before the scale, against the largest so far.
template <int TYPE, int D>
__device__ __noinline__ void ca_far_row(const Kv16AttnParams& p, const CaPart& d, int G, int R, int lane, unsigned* beat) {
  constexpr int W = D / 64;  // words a lane
  const int j = R / G, pos = d.past + j, head = d.kvh * G + R - j * G;
  if (!in_bounds(p.err, d.at + j, p.T)) return;
  auto words = [&](const void* base, int64_t row, uint32_t* w) {
    const uint32_t* at = static_cast<const uint32_t*>(base) + row / 2 + W * lane;
    if constexpr (W == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(at);
      w[0] = x.x;
      w[1] = x.y;
    } else {
      w[0] = *at;
    }
  };
  uint32_t q[W];
  words(p.q, (int64_t)(d.at + j) * p.q_stride + (int64_t)head * D, q);
  float acc[2 * W] = {}, m = -INFINITY, l = 0.0f;
  constexpr int N = 8;  // keys at a time, of one page
  const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
#pragma unroll 1
  for (int key0 = first / N * N; key0 <= pos; key0 += N) {
    const int page = p.table[(int64_t)d.b * p.max_blocks + key0 / 64];
    const int64_t row = (((int64_t)page * p.Hkv + d.kvh) * 64 + key0 % 64) * D;
    uint32_t k[N][W] = {}, v[N][W] = {};
    if (page >= 0 && page < p.pages) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        words(p.k, row + n * D, k[n]);
        words(p.v, row + n * D, v[n]);
      }
    }
    float s[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      s[n] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) s[n] = fmaf(ca_value<TYPE>(q[i / 2], i & 1), ca_value<TYPE>(k[n][i / 2], i & 1), s[n]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s[n] += __shfl_xor_sync(0xffffffffu, s[n], x);
    }
    const float before = m;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (key0 + n >= first && key0 + n <= pos) m = fmaxf(m, s[n]);
    const float f = before == -INFINITY ? 0.0f : ex2((before - m) * p.scale_log2);
    l *= f;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) acc[i] *= f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (key0 + n < first || key0 + n > pos) continue;
      const float w = s[n] == -INFINITY ? 0.0f : ex2((s[n] - m) * p.scale_log2);
      l += w;
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) acc[i] = fmaf(w, ca_value<TYPE>(v[n][i / 2], i & 1), acc[i]);
    }
    if (lane == 0 && key0 % 512 == 0) atomicAdd(beat, 1u);
  }
  const float inv = 1.0f / l;
  uint32_t* to = static_cast<uint32_t*>(p.out) + ((int64_t)(d.at + j) * p.H + head) * D / 2 + W * lane;
#pragma unroll
  for (int i = 0; i < W; ++i) to[i] = ca_pack<TYPE>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
}

// A cut unit's rows from its np pieces, by eight warps: warp w has the rows w, w +
// 8, .., a lane D / 32 columns; N rows and K pieces at a time, whose loads go out
// together.
template <int TYPE, int D, int N, int K>
__device__ __noinline__ void ca_merge(const Kv16AttnParams& p, const CaWork& wk, const CaPart& d, const int* list, int np,
                                      int w, int lane, unsigned* beat) {
  constexpr int V = D / 32;
  const int G = (int)wk.by_g.d, rows = d.rows;
  for (int r0 = w; r0 < rows; r0 += 8 * N) {
    float acc[N][V], M[N], S[N];
    bool far[N];  // the row is done over
#pragma unroll
    for (int q = 0; q < N; ++q) {
      far[q] = false;
      M[q] = -INFINITY;
      S[q] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[q][v] = 0.0f;
    }
    for (int k0 = 0; k0 < np; k0 += K) {
      float2 ml[N][K];
      float o[N][K][V];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int at = k0 + k < np ? list[k0 + k] : 0;
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const bool there = k0 + k < np && r0 + 8 * q < rows;
          const int64_t row = (int64_t)at + (there ? r0 + 8 * q : 0);
          ml[q][k] = there ? __ldcg(&wk.part_ml[row]) : make_float2(-INFINITY, 0.0f);
          const float* x = wk.part_o + row * D + V * lane;
          if constexpr (V == 4) {
            const float4 y = there ? __ldcg(reinterpret_cast<const float4*>(x)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            o[q][k][0] = y.x;
            o[q][k][1] = y.y;
            o[q][k][2] = y.z;
            o[q][k][3] = y.w;
          } else {
            const float2 y = there ? __ldcg(reinterpret_cast<const float2*>(x)) : make_float2(0.0f, 0.0f);
            o[q][k][0] = y.x;
            o[q][k][1] = y.y;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < N; ++q) {
        float top = M[q];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          far[q] = far[q] || ml[q][k].y < 0.0f;
          if (ml[q][k].y != 0.0f) top = fmaxf(top, ml[q][k].x);  // (a sum of zero: the piece's keys are not seen)
        }
        const float f0 = S[q] == 0.0f ? 0.0f : ex2(M[q] - top);
        S[q] *= f0;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[q][v] *= f0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float f = ml[q][k].y == 0.0f ? 0.0f : ex2(ml[q][k].x - top);
          S[q] += f * ml[q][k].y;
#pragma unroll
          for (int v = 0; v < V; ++v) acc[q][v] += f * o[q][k][v];
        }
        M[q] = top;
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int r = r0 + 8 * q;
      if (r >= rows) continue;
      const float inv = 1.0f / S[q];
      const int R = d.row0 + r, j = wk.by_g(R);
      if (!in_bounds(p.err, d.at + j, p.T)) continue;
      uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                 ((int64_t)(d.at + j) * p.H + d.kvh * G + R - j * G) * D + V * lane);
      if (far[q])
        ca_far_row<TYPE, D>(p, d, G, R, lane, beat);
      else if constexpr (V == 4)
        *reinterpret_cast<uint2*>(to) =
            make_uint2(ca_pack<TYPE>(acc[q][0] * inv, acc[q][1] * inv), ca_pack<TYPE>(acc[q][2] * inv, acc[q][3] * inv));
      else
        *to = ca_pack<TYPE>(acc[q][0] * inv, acc[q][1] * inv);
    }
  }
}

// The last position of slot t's rows, where the slots are row tiles.
__device__ __forceinline__ int ca_slot_last(const CaWork& wk, const CaPart& d, int t) {
  return d.past + wk.by_g(d.row0 + min(d.rows - 1, 128 * t + 127));
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kCaThreads, 1)
    kv16_attention_kernel(const __grid_constant__ CaMaps maps, const Kv16AttnParams p, const CaWork wk) {
  using L = CaLayout<D>;
  constexpr int NB = L::kBufs;
  extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's atoms are 1024 bytes)
  CaShared* sh = reinterpret_cast<CaShared*>(smem + L::kSharedOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = (int)wk.by_g.d, cta = (int)blockIdx.x;

  if (tid == 0) {
    sh->beat = 0u;
    for (int i = 0; i < NB; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->free[i], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->fin[t], 1);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&sh->s_full[t][k], 1);
        mbar_init(&sh->p_full[t][k], 4);
        mbar_init(&sh->pv_done[t][k], 1);
      }
    }
    mbar_init(&sh->stat, 4);
    mbar_init(&sh->read, 4);
    mbar_init(&sh->stored, 8);
    mbar_init(&sh->told, 1);
    for (int i = 0; i < kCaOk; ++i) {
      mbar_init(&sh->landed[i], 1);
      mbar_init(&sh->ok[i], 1);
    }
    for (int i = 0; i < kCaDesc; ++i) {
      for (int t = 0; t < 2; ++t) mbar_init(&sh->q_ready[t][i], 4);
      mbar_init(&sh->desc_full[i], 1);
      mbar_init(&sh->desc_free[i], 11);
    }
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512u);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
  }
  grid_dependency_wait();  // everything else in global memory may come from the kernels before

  // ---- the run: CTA c of C takes the work from about W c / C to W (c + 1) / C.
  // Each thread sums a row of requests; the scratch lies where Q will
  struct Scratch {
    int64_t sums[kCaThreads / 32];
    int units[kCaThreads / 32], longest[kCaThreads / 32], late[kCaThreads / 32];
    int64_t at[2];  // the work before the requests that the run begins and ends in
    CaPlace place[2];
  };
  Scratch* scr = reinterpret_cast<Scratch*>(smem);
  const int per = (p.B + kCaThreads - 1) / kCaThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t mine = 0;
  int units = 0, longest = 0, late = 0;
  CaRequest r = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    r = ca_request(p, b, cta == 0);
    if (r.cnt > 0) {
      const CaLoad w = ca_load(p, wk, r);
      const int64_t n = p.Hkv * w.before(w.units);
      mine += n;
      units = (int)min((int64_t)units + (int64_t)p.Hkv * w.units, (int64_t)kCaMany);
      const int nt = ca_tiles(p, wk, r, w.units - 1).nt;
      longest = max(longest, nt);
      late = max(late, w.weight * (nt + kCaOverhead / kCaKeys) - (int)((float)n * wk.tiles_inv));
    }
  }
  units = __reduce_add_sync(0xffffffffu, units);
  longest = __reduce_max_sync(0xffffffffu, longest);
  late = __reduce_max_sync(0xffffffffu, late);
  int64_t upto = mine;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, k);
    if (lane >= k) upto += o;
  }
  if (lane == 31) scr->sums[warp] = upto;
  if (lane == 31) {
    scr->units[warp] = units;
    scr->longest[warp] = longest;
    scr->late[warp] = late;
  }
  if (tid < 2) scr->place[tid] = CaPlace{p.B, 0, 0, 0, 0, 1, CaRequest{0, 0, 0}};
  __syncthreads();
  grid_launch_dependents();  // (TMEM is allocated: no later kernel can hold it while this one waits for it)
  int64_t W = 0, at = upto - mine;
  units = 0;
  for (int w = 0; w < kCaThreads / 32; ++w) {
    if (w < warp) at += scr->sums[w];
    W += scr->sums[w];
    units += scr->units[w];
    longest = max(longest, scr->longest[w]);
    late = max(late, scr->late[w]);
  }
  const bool queue = units < kCaMany &&
                     ((units >= 2 * wk.ctas && longest <= kCaQueueTiles) ||
                      (units >= 4 * wk.ctas && longest <= 4 * kCaQueueTiles)) &&
                     (float)late * (float)units <= kCaQueueLate * (float)W * (wk.tiles_inv * (float)wk.ctas);
  // Fewer units than CTAs: each in a whole number of pieces, as many as pay, unless it is done sooner with a run for every
  // CTA, nearly all of which then merge.
  int C = wk.ctas;
  uint64_t inv = wk.ctas_inv;
  int snap = kCaSnap;
  if (units > 0 && units < C) {
    const float all = (float)W / (float)(kCaWeight1 * G * kCaKeys), per_unit = all / (float)units;
    const float row = kCaRowPiece * fminf(256.0f, (float)p.T * (float)p.H / (float)units);
    int k = max(1, min(C / units, (int)fminf(sqrtf(per_unit / row), per_unit / kCaLeast)));
    float even = per_unit / (float)k + kCaCut + (float)k * row;
    if (k == 1 || per_unit <= even) {
      k = 1;
      even = per_unit + kCaCut;  // (units of different lengths are cut all the same)
    }
    // (a run for every CTA: most have a second part to start)
    if (even <= all / (float)C + 1.5f * kCaCut + ((float)C / (float)units + 2.0f) * row) {
      C = units * k;
      snap = max(1, min(kCaSnap, (int)(per_unit / (float)(4 * k))));
      inv = (uint64_t)(0xFFFFFFFFu / (uint32_t)C) << 32;  // (2^64 / C less 2^-32 C of it: a short division)
    } else {
      snap = kCaSnapFew;  // (nearly every cut is meant)
    }
  }
  auto bound = [&](int c) { return c >= C ? W : (int64_t)__umul64hi((uint64_t)W, inv * (uint64_t)c); };
#pragma unroll 1
  for (int e = 0; e < 2 && !queue; ++e) {
    const int64_t x = bound(cta + e);
    if (x < at || x >= at + mine) continue;
    int64_t a = at;
    for (int b = b0; b < b1; ++b) {
      int64_t n = mine;  // (a thread with one request knows it, and its work)
      if (per > 1) {
        r = ca_request(p, b, false);
        if (r.cnt == 0) continue;
        const CaLoad w = ca_load(p, wk, r);
        n = p.Hkv * w.before(w.units);
      }
      if (x < a + n) {
        scr->place[e].b = b;
        scr->place[e].r = r;
        scr->at[e] = a;
        break;
      }
      a += n;
    }
  }
  __syncthreads();
  if ((tid == 0 || tid == 32) && scr->place[tid >> 5].b < p.B) {  // both ends at once
    const int e = tid >> 5;
    scr->place[e] = ca_locate(p, wk, scr->place[e].b, scr->place[e].r, scr->at[e], bound(cta + e), snap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const CaPlace begin = scr->place[0], end = scr->place[1];
  const uint32_t tmem = sh->tmem;
  __syncthreads();  // the scratch becomes Q
  // A tile has the buffers 2 r (keys) and 2 r + 1 (values) of the ring, r its place among kPairs, and the phase ph.
  // (Places are stepped, not divided out: the pace hangs on these chains of instructions.)
  constexpr uint32_t kPairs = NB / 2;
  struct Place {
    uint32_t r, ph;
    __device__ __forceinline__ void step(uint32_t by) {
      r += by;
      if (r >= kPairs) r -= kPairs, ph ^= 1u;
    }
  };
  // what part of a cut unit falls to CTA c: tiles cut_at(c) .. cut_at(c + 1) - 1
  auto cut_at = [&](int c, int64_t u0, int64_t v, int nt) {
    const int64_t x = bound(c);
    return x <= u0 ? 0 : x >= u0 + v ? nt : ca_share(x - u0, nt, v, snap);
  };

  if (warp == 0) {
    // ------------------------------------------------- parts and copies
    uint32_t keys = 0, values = 0, guarded = 0;  // tiles copied so far, and guarded ones
    Place pk = {0u, 0u}, pv = {0u, 0u};
    int seq = 0;
    bool ok = true;
    int b = begin.b, kvh = begin.kvh, unit = begin.unit;
    bool first = true;
    CaRequest r = begin.r;
    CaLoad w;
    if (b < p.B) w = ca_load(p, wk, r);
    // the queue: 32 requests at a time, a lane each, of which the first has the units from `from` on
    int group = 0, from = 0, mine_units = 0, mine_upto = 0;
    CaRequest mine_r;
    auto look = [&]() {
      mine_r = group + lane < p.B ? ca_request(p, group + lane, false) : CaRequest{0, 0, 0};
      mine_units = mine_r.cnt > 0 ? ca_load(p, wk, mine_r).units * p.Hkv : 0;
      mine_upto = mine_units;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, mine_upto, k);
        if (lane >= k) mine_upto += o;
      }
    };
    if (queue) look();
    while (ok) {
      bool at_end = false;
      if (queue) {
        int u = lane == 0 ? atomicAdd(wk.queue, 1) : 0;
        u = __shfl_sync(0xffffffffu, u, 0);
        if (u >= units) break;
        int in_group;
        while (u - from >= (in_group = __shfl_sync(0xffffffffu, mine_upto, 31)) && group + 32 < p.B) {
          from += in_group;
          group += 32;
          look();
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, mine_upto > u - from)) - 1;
        if (l < 0) break;
        b = group + l;
        r.at = __shfl_sync(0xffffffffu, mine_r.at, l);
        r.cnt = __shfl_sync(0xffffffffu, mine_r.cnt, l);
        r.past = __shfl_sync(0xffffffffu, mine_r.past, l);
        const int n = __shfl_sync(0xffffffffu, mine_units, l);
        const int k = u - from - (__shfl_sync(0xffffffffu, mine_upto, l) - n);  // the last rows first, all heads of them
        kvh = k % p.Hkv;
        unit = n / p.Hkv - 1 - k / p.Hkv;
      } else {
        if (b >= p.B) break;
        at_end = b == end.b && kvh == end.kvh && unit == end.unit;
      }
      const CaTiles t = ca_tiles(p, wk, r, unit);
      const int lo = !queue && first ? begin.cut : 0, hi = at_end ? end.cut : t.nt;
      if (hi > lo) {
        const int ds = seq % kCaDesc;
        if (seq >= kCaDesc && !ca_wait(&sh->desc_free[ds], (uint32_t)(seq / kCaDesc - 1) & 1u, p.err, &sh->beat)) {
          ok = false;
          break;
        }
        // key tiles t with 64 t + 63 <= first_pos, and 64 t > last_pos - window, are seen whole by every row
        const int whole = (t.first_pos + 1) / kCaKeys - t.tile0 - lo;
        const int in_window =
            p.window > 0 && t.last_pos >= p.window ? (t.last_pos - p.window) / kCaKeys + 1 - t.tile0 - lo : 0;
        const int gw = min(max(in_window, 0), hi - lo), gc = max(min(whole, hi - lo), gw);
        if (lane == 0) {
          CaPart& d = sh->part[ds];
          d.b = b;
          d.at = r.at;
          d.past = r.past;
          d.kvh = kvh;
          d.row0 = unit * 256;
          d.rows = min(256, r.cnt * G - unit * 256);
          d.tile0 = t.tile0;
          d.nt = t.nt;
          d.lo = lo;
          d.hi = hi;
          d.gw = gw;
          d.gc = gc;
          d.last_key = t.last_pos;
          d.first_cut = 0;
          d.u0 = first ? begin.u0 : end.u0;
          d.v = first ? begin.v : end.v;
        }
        if (lo > 0 || hi < t.nt) {  // the first CTA that begins after the unit's begin, looked for from here downwards
          int cs = cta + 1;
          while (true) {
            const unsigned later = __ballot_sync(0xffffffffu, cs - lane >= 1 && bound(cs - lane) > (first ? begin.u0 : end.u0));
            const int n = later == 0xffffffffu ? 32 : __ffs(~later) - 1;
            cs -= n;
            if (n < 32) break;
          }
          if (lane == 0) sh->part[ds].first_cut = cs + 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->desc_full[ds]);
        ++seq;
        // the pages of 32 tiles at a time, a lane an entry
        const int32_t* row = p.table + (int64_t)b * p.max_blocks;
        int base = t.tile0 + lo;
        auto entries = [&]() {
          if (base + lane >= t.tile0 + hi || !in_bounds(p.err, base + lane, p.max_blocks)) return -1;
          const int page = row[base + lane];
          if (page >= 0 && page < p.pages) return page;
          report_error(p.err, kErrInput);
          return -1;
        };
        int now = entries();
        // keys two tiles before values, as they are used: a buffer is in use for no longer than it has to be
        int z1 = 0, z2 = 0;
        for (int k = lo; ok && k < hi + 2; ++k) {
          int z = 0;
          if (k < hi) {
            if (t.tile0 + k - base >= 32) {
              base += 32;
              now = entries();
              if (lane == 0) *(volatile unsigned*)&sh->beat = sh->beat + 1u;
            }
            const int page = __shfl_sync(0xffffffffu, now, t.tile0 + k - base);
            z = page >= 0 ? page * p.Hkv + kvh : p.pages * p.Hkv;  // past the last page: zeros
            ok = keys < kPairs || ca_wait(&sh->free[2u * pk.r], pk.ph ^ 1u, p.err, &sh->beat);
            if (ok && !test_skip_copy(2u * keys))
              ca_copy_tile(smem + L::kRingOff + 2u * pk.r * L::kTile, &maps.k, z, &sh->full[2u * pk.r], (uint32_t)L::kTile);
            if (ok) ++keys, pk.step(1u);
          }
          const int v = k - 2;
          if (ok && v >= lo) {
            const uint32_t x = 2u * pv.r + 1u;
            ok = values < kPairs || ca_wait(&sh->free[x], pv.ph ^ 1u, p.err, &sh->beat);
            // guarded values land at a barrier of their own: the guard tells when they may be used
            const bool guard = v - lo < gw || v - lo >= gc;
            if (ok && !test_skip_copy(2u * values + 1u)) {
              uint64_t* bar = &sh->full[x];
              if (guard) {
                if (lane == 0) mbar_arrive(bar);
                bar = &sh->landed[guarded % kCaOk];
              }
              ca_copy_tile(smem + L::kRingOff + x * L::kTile, &maps.v, z2, bar, (uint32_t)L::kTile);
            }
            if (ok) ++values, guarded += guard, pv.step(1u);
          }
          z2 = z1;
          z1 = z;
        }
      }
      if (queue) continue;
      if (at_end) break;
      first = false;
      if (++unit == w.units) {
        unit = 0;
        if (++kvh == p.Hkv) {
          kvh = 0;
          do {
            if (++b == p.B) break;
            r = ca_request(p, b, false);
          } while (r.cnt == 0);
          if (b < p.B) w = ca_load(p, wk, r);
        }
      }
    }
    // no more parts
    const int ds = seq % kCaDesc;
    if (ok && seq >= kCaDesc) ok = ca_wait(&sh->desc_free[ds], (uint32_t)(seq / kCaDesc - 1) & 1u, p.err, &sh->beat);
    if (ok && lane == 0) {
      sh->part[ds].lo = 0;
      sh->part[ds].hi = 0;
      mbar_arrive(&sh->desc_full[ds]);
    }
    // the copies in flight land before the CTA exits (some may be, if a wait of another warp ran out)
    for (uint32_t k = keys > kPairs ? keys - kPairs : 0; k < keys; ++k)
      if (!test_skip_copy(2u * k)) ca_wait(&sh->full[2u * (k % kPairs)], (k / kPairs) & 1u, p.err, &sh->beat);
    for (uint32_t k = values > kPairs ? values - kPairs : 0; k < values; ++k)
      if (!test_skip_copy(2u * k + 1u)) ca_wait(&sh->full[2u * (k % kPairs) + 1u], (k / kPairs) & 1u, p.err, &sh->beat);
    for (uint32_t k = guarded > kCaOk ? guarded - kCaOk : 0; k < guarded; ++k)
      ca_wait(&sh->landed[k % kCaOk], (k / kCaOk) & 1u, p.err, &sh->beat);
  } else if (warp <= 2) {
    // ------------------------------------------------------ MMA, slot t
    // The scores are a tile ahead of the weights, so that neither side waits for the other's latency.
    const int t = warp - 1;
    constexpr uint32_t fmt = TYPE == 0 ? 1u : 0u;
    const uint32_t idesc_s = umma_idesc(kCaKeys, fmt, fmt, 0u, 0u), idesc_o = umma_idesc(D, fmt, fmt, 0u, 1u);
    Place part0 = {0u, 0u};             // the part's first tile
    uint32_t oks = 0, sc = 0, pc = 0;   // guarded tiles, scores issued and weights used so far
    const uint32_t s_col = tmem + ca_s_col(t, 0), o_col = tmem + ca_o_col(t);
    const uint64_t ring_k = umma_desc_sw128_kmajor(smem_u32(smem + L::kRingOff));
    const uint64_t ring_v = umma_desc_sw128_mnmajor(smem_u32(smem + L::kRingOff + L::kTile), (uint32_t)L::kHalf, 1024u);
    bool ok = true, issued = false;
    for (int seq = 0; ok; ++seq) {
      const int ds = seq % kCaDesc;
      if (!ca_wait(&sh->desc_full[ds], (uint32_t)(seq / kCaDesc) & 1u, p.err, &sh->beat)) break;
      const CaPart& d = sh->part[ds];
      const int n = d.hi - d.lo, gw = d.gw, gc = d.gc;
      if (n <= 0) break;
      const bool two = d.rows > 128;
      // this slot's tiles: as far as its rows see where the slots are row tiles, every other one where they share the rows
      const int upto = two ? min(max(ca_slot_last(wk, d, t) / kCaKeys + 1 - d.tile0 - d.lo, 0), n) : n;
      const int step = two ? 1 : 2, first = two ? 0 : t;
      int i = first;  // the tile whose scores come next
      int at = 0;     // tiles before it are used or passed over
      Place pi = part0, pv;
      const uint64_t q0 = umma_desc_sw128_kmajor(smem_u32(smem + (two ? t : 0) * L::kQ));
      // Each slot releases every buffer once: those it does not use as soon as they are there (a phase is never skipped).
      auto pass = [&](int to) {
        for (; at < to; ++at, pi.step(1u))
          for (uint32_t x = 2u * pi.r, e = x + 2u; x < e; ++x) {
            if (!ca_wait(&sh->full[x], pi.ph, p.err, &sh->beat)) return false;
            if (lane == 0) mbar_arrive(&sh->free[x]);
            __syncwarp();
          }
        return true;
      };
      auto scores = [&](bool there) {  // S = Q K^T
        if (at < i) {
          if (!pass(i)) return false;
          there = false;
        }
        if (!there && !ca_wait(&sh->full[2u * pi.r], pi.ph, p.err, &sh->beat)) return false;
        tc_fence_after();
        const uint32_t sb = sc & 1u;
        const uint64_t k0 = ring_k + (uint64_t)(pi.r * (2u * L::kTile / 16));  // (the descriptors count in 16 bytes)
        ca_mma4_ss(s_col + 64u * sb, q0, k0, idesc_s, 0u);
        if constexpr (D == 128) ca_mma4_ss(s_col + 64u * sb, q0 + L::kQHalf / 16, k0 + L::kHalf / 16, idesc_s, 1u);
        umma_commit_warp(&sh->s_full[t][sb]);
        umma_commit_warp(&sh->free[2u * pi.r]);
        issued = true;
        ++sc;
        at = i + 1;
        i += step;
        pi.step(1u);
        return true;
      };
      // (slot 1's warps are done with the part before, and where the slots share the rows slot 0's have loaded them)
      if (i < upto && t == 1 && !two) ok = ca_wait(&sh->q_ready[0][ds], (uint32_t)(seq / kCaDesc) & 1u, p.err, &sh->beat);
      if (ok && i < upto) ok = ca_wait(&sh->q_ready[t][ds], (uint32_t)(seq / kCaDesc) & 1u, p.err, &sh->beat) && scores(false);
      if (ok && i < upto) ok = scores(false);
      // the scores two tiles on go out behind the product of the weights that lie in their buffer
      pv = part0;
      pv.step((uint32_t)first);
      for (int v = first; ok && v < upto; v += step, ++pc, pv.step((uint32_t)step)) {
        const uint32_t sb = pc & 1u;
        uint64_t *values = &sh->full[2u * pv.r + 1u], *weights = &sh->p_full[t][sb];
        const bool v_there = mbar_test(values, pv.ph), p_there = mbar_test(weights, (pc >> 1) & 1u);
        const bool k_there = mbar_test(&sh->full[2u * pi.r], pi.ph);  // (the tile `at`, whose last phase is waited for)
        if (!v_there) ok = ca_wait(values, pv.ph, p.err, &sh->beat);
        if (ok && (v < gw || v >= gc)) {  // the guard has looked through the values
          const uint32_t g = oks + (uint32_t)(v < gw ? v : gw + v - gc);
          ok = ca_wait(&sh->ok[g % kCaOk], (g / kCaOk) & 1u, p.err, &sh->beat);
        }
        if (ok && !p_there) ok = ca_wait(weights, (pc >> 1) & 1u, p.err, &sh->beat);
        if (!ok) break;
        tc_fence_after();
        // O += P V
        ca_mma4_ts(o_col, s_col + 64u * sb, ring_v + (uint64_t)(pv.r * (2u * L::kTile / 16)), idesc_o, v >= step ? 1u : 0u);
        umma_commit_warp(&sh->pv_done[t][sb]);
        umma_commit_warp(&sh->free[2u * pv.r + 1u]);
        if (i < upto) ok = scores(k_there);
      }
      ok = ok && pass(n);
      part0 = pi;
      oks += (uint32_t)(gw + n - gc);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->desc_free[ds]);
    }
    if (issued) {
      umma_commit_warp(&sh->fin[t]);  // tracks all of this warp's MMAs
      ca_wait(&sh->fin[t], 0u, p.err, &sh->beat);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ guard
    uint32_t buf = 0, oks = 0;
    bool ok = true;
    for (int seq = 0; ok; ++seq) {
      const int ds = seq % kCaDesc;
      if (!ca_wait(&sh->desc_full[ds], (uint32_t)(seq / kCaDesc) & 1u, p.err, &sh->beat)) break;
      const CaPart& d = sh->part[ds];
      const int lo = d.lo, n = d.hi - lo, gw = d.gw, gc = d.gc, tile0 = d.tile0, last_key = d.last_key;
      if (n <= 0) break;
      if (lane == 0) *(volatile int*)&sh->specials[ds] = 0;
      __syncwarp();
      for (int i = gw > 0 ? 0 : gc; ok && i < n; i = i + 1 < gw || i + 1 >= gc ? i + 1 : gc) {
        const uint32_t x = buf + 2u * (uint32_t)i + 1u;
        if (!ca_wait(&sh->landed[oks % kCaOk], (oks / kCaOk) & 1u, p.err, &sh->beat)) {
          ok = false;
          break;
        }
        uint8_t* v0 = smem + L::kRingOff + (x % NB) * L::kTile;
        uint32_t nil[4] = {0u, 0u, 0u, 0u};  // 0 times each value, summed up: NaN where one is not finite
#pragma unroll 8
        for (int o = lane * 16; o < L::kTile; o += 512) {
          const uint4 w = *reinterpret_cast<const uint4*>(v0 + o);
          nil[0] = ca_times_zero<TYPE>(w.x, nil[0]);
          nil[1] = ca_times_zero<TYPE>(w.y, nil[1]);
          nil[2] = ca_times_zero<TYPE>(w.z, nil[2]);
          nil[3] = ca_times_zero<TYPE>(w.w, nil[3]);
        }
        if (__any_sync(0xffffffffu, ((nil[0] | nil[1] | nil[2] | nil[3]) & 0x7FFF7FFFu) != 0u)) {
          const int e = *(volatile int*)&sh->specials[ds];
          CaSpecial& sp = sh->special[ds][min(e, kCaSpecial - 1)];
          if (lane < 2) sp.keys[lane] = 0u;
          if (lane == 2) sp.key0 = (tile0 + lo + i) * kCaKeys;
          __syncwarp();
          for (int o = lane * 4; o < L::kTile; o += 128) {
            uint32_t* w = reinterpret_cast<uint32_t*>(v0 + o);
            const uint32_t bad = ca_not_finite<TYPE>(*w);
            if (!bad) continue;
            const int r = (o % L::kHalf) / 128;
            if ((tile0 + lo + i) * kCaKeys + r <= last_key) atomicOr(&sp.keys[r >> 5], 1u << (r & 31));
            *w &= ~((bad >> 15) * 0xFFFFu);
          }
          fence_proxy_async_smem();
          __threadfence_block();
          __syncwarp();
          if (lane == 0) *(volatile int*)&sh->specials[ds] = min(e + 1, kCaSpecial);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->ok[oks % kCaOk]);
        ++oks;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->desc_free[ds]);
      buf += 2u * (uint32_t)n;
    }
  } else {
    // ---------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2, qd = warp & 3, rl = qd * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * qd) << 16);
    const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
    uint32_t sc = 0, shared_parts = 0, cut_parts = 0;
    bool ok = true, have_q = false;
    // this warp's rows of a part's Q: 128-byte swizzle, K-major, halves of 64 columns; eight lanes a row
    auto load_q = [&](const CaPart& e) {
      const int u0 = (e.rows > 128 ? 128 * t : 0) + qd * 32, c = lane & 7;
      if (e.rows <= 128 && t == 1) return;  // (slot 0's rows)
      uint8_t* qt = smem + t * L::kQ + qd * 32 * 128;
#pragma unroll 1  // (a part runs it once: the shorter code is sooner there)
      for (int k = 0; k < 8; ++k) {
        const int r = 4 * k + (lane >> 3), u = u0 + r;
        const int R2 = e.row0 + (u < e.rows ? u : 0), j2 = wk.by_g(R2);
        const bool there = u < e.rows && in_bounds(p.err, e.at + j2, p.T);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (int64_t)(e.at + j2) * p.q_stride +
                              (int64_t)(e.kvh * G + R2 - j2 * G) * D + c * 8;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          ca_copy16(qt + h * L::kQHalf + r * 128 + ((c ^ (r & 7)) << 4), there ? src + 64 * h : p.q, there);
      }
    };
    auto hand_q = [&](int ds) {
      ca_copy_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_ready[t][ds]);
    };
    for (int seq = 0; ok; ++seq) {
      const int ds = seq % kCaDesc;
      if (!ca_wait(&sh->desc_full[ds], (uint32_t)(seq / kCaDesc) & 1u, p.err, &sh->beat)) break;
      const CaPart& d = sh->part[ds];
      const int n = d.hi - d.lo;
      if (n <= 0) break;
      if (!have_q) {
        load_q(d);
        hand_q(ds);
      }
      have_q = false;
      const bool two = d.rows > 128, cut = n < d.nt;
      const int ur = (two ? 128 * t : 0) + rl;  // this thread's row of the unit
      const bool valid = ur < d.rows;
      const int R = d.row0 + (valid ? ur : 0), j = wk.by_g(R), pos = d.past + j;
      const int head = d.kvh * G + R - j * G;
      const bool any_row = __any_sync(0xffffffffu, valid);
      int nt = (n - t + 1) / 2;
      if (two) nt = min(max(ca_slot_last(wk, d, t) / kCaKeys + 1 - d.tile0 - d.lo, 0), n);
      const int gw = d.gw, gc = d.gc;
      const int rel = pos - (d.tile0 + d.lo) * kCaKeys;  // the row's position, from the part's first key on
      float m = -INFINITY, l = 0.0f;
      bool far = false;  // the row is to be done over
      for (int jt = 0; jt < nt; ++jt, ++sc) {
        const int i = two ? jt : 2 * jt + t, buf = (int)(sc & 1u);
        if (!ca_wait(&sh->s_full[t][buf], (sc >> 1) & 1u, p.err, &sh->beat)) {
          ok = false;
          break;
        }
        if (!any_row) {  // (what the weights of these rows are does not matter)
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[t][buf]);
          continue;
        }
        tc_fence_after();
        // seen: the columns bottom < c <= top (where a whole warp sees all of them, there is nothing to mask)
        const int top = rel - i * kCaKeys, bottom = p.window > 0 ? top - p.window : -1;
        bool masked = i < gw || i >= gc;
        if (masked) masked = __any_sync(0xffffffffu, top < kCaKeys - 1 || bottom >= 0);
        auto mask = [&](uint32_t (&x)[32], int first) {  // columns first .. first + 31
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (first + c > top || first + c <= bottom) x[c] = __float_as_uint(-INFINITY);
        };
        // the weights of 32 columns, as pairs of the cache's type, and their sum
        auto weigh = [&](const uint32_t (&x)[32], uint32_t* pr, float u) {
          const uint64_t nu2 = f2_pack(-u, -u);
          uint64_t la = f2_pack(0.0f, 0.0f), lb = la;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nu2), x0, x1);
            const float e0 = ex2(x0), e1 = ex2(x1);
            pr[c] = ca_pack<TYPE>(e0, e1);
            const uint64_t r2 = f2_pack(e0, e1);
            if (c & 1)
              lb = f2_add(lb, r2);
            else
              la = f2_add(la, r2);
          }
          float a0, a1;
          f2_unpack(f2_add(la, lb), a0, a1);
          return a0 + a1;
        };
        const uint32_t col = trow + ca_s_col(t, buf);
        uint32_t sa[32], sb[32], pr[32];
        auto load = [&]() {
          tmem_ld_32x32b_x32(col, sa);
          tmem_ld_32x32b_x32(col + 32u, sb);
          tmem_wait_ld(sa);
          tmem_wait_ld(sb);
          if (masked) {
            mask(sa, 0);
            mask(sb, 32);
          }
        };
        load();
        float u = (m == -INFINITY ? 0.0f : m) - kCaUp<TYPE>;
        float sum = weigh(sa, pr, u);
        sum += weigh(sb, pr + 16, u);
        const bool raise = m == -INFINITY || !(sum <= kCaMost<TYPE>);
        if (__any_sync(0xffffffffu, raise)) {
          // the reference becomes the largest score where it has to; the sums so far follow
          load();
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            m4[c & 3] = max3f(m4[c & 3], __uint_as_float(sa[2 * c]), __uint_as_float(sa[2 * c + 1]));
            m4[(c + 2) & 3] = max3f(m4[(c + 2) & 3], __uint_as_float(sb[2 * c]), __uint_as_float(sb[2 * c + 1]));
          }
          const float raw = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), mx = raw * p.scale_log2;
          float cf = 1.0f;
          if (raise && mx > m) {
            far = far || (fabsf(mx) >= kCaFar && fabsf(raw) < INFINITY);
            cf = m == -INFINITY ? 0.0f : ex2(m - mx);
            m = mx;
            l *= cf;
          }
          if (jt > 0 && __any_sync(0xffffffffu, cf < 1.0f)) {
            if (!ca_wait(&sh->pv_done[t][buf ^ 1], ((sc - 1) >> 1) & 1u, p.err, &sh->beat)) {  // the sums of the tile before
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              tmem_ld_32x32b_x32(trow + ca_o_col(t) + (uint32_t)c0, pr);
              tmem_wait_ld(pr);
#pragma unroll
              for (int c = 0; c < 32; ++c) pr[c] = __float_as_uint(__uint_as_float(pr[c]) * cf);
              tmem_st_32x32b_x32(trow + ca_o_col(t) + (uint32_t)c0, pr);
            }
          }
          u = (m == -INFINITY ? 0.0f : m) - kCaUp<TYPE>;
          sum = weigh(sa, pr, u);
          sum += weigh(sb, pr + 16, u);
        }
        l += sum;
        tmem_st_32x32b_x32(col, pr);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full[t][buf]);
      }
      // With its last scores this slot is done with its Q (row tiles: it is this slot's alone), and the next part's comes
      // in beside the last product of the weights, its scores beside this part's end. (A cut part's end needs the place.)
      if (ok && nt > 0 && two && !cut) {
        const int dn = (seq + 1) % kCaDesc;
        if (__all_sync(0xffffffffu, mbar_test(&sh->desc_full[dn], (uint32_t)((seq + 1) / kCaDesc) & 1u)) &&
            sh->part[dn].hi > 0) {
          load_q(sh->part[dn]);
          have_q = true;
        }
      }
      // ---- the part's end
      if (far) l = -1.0f;
      if (ok && nt > 0) ok = ca_wait(&sh->pv_done[t][(sc - 1) & 1u], ((sc - 1) >> 1) & 1u, p.err, &sh->beat);
      if (!ok) {
        if (have_q) ca_copy_wait();
        break;
      }
      bool to_hand = have_q;
      tc_fence_after();
      float a0 = 1.0f, a1 = 0.0f;  // factors of this slot's sums and of the other's
      if (!two) {
        if (t == 1) {  // hand over the reference and the sum through TMEM; the sums of values are there
          uint32_t st[8] = {__float_as_uint(m), __float_as_uint(l), 0u, 0u, 0u, 0u, 0u, 0u};
          tmem_st_32x32b_x8(trow + ca_s_col(1, 0), st);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->stat);
        } else {
          if (!ca_wait(&sh->stat, shared_parts & 1u, p.err, &sh->beat)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t st[8];
          tmem_ld_32x32b_x8(trow + ca_s_col(1, 0), st);
          tmem_wait_ld(st);
          const float m1 = __uint_as_float(st[0]), l1 = __uint_as_float(st[1]);
          if (n > 1 && (l < 0.0f || l1 < 0.0f)) {
            l = -1.0f;
          } else if (n > 1 && !(l1 == 0.0f)) {
            const float M = fmaxf(m, m1);
            a0 = l == 0.0f ? 0.0f : ex2(m - M);
            a1 = ex2(m1 - M);
            l = l * a0 + l1 * a1;
            m = M;
          }
        }
      }
      const int64_t slot = 2 * cta + (d.lo > 0 ? 0 : 1);
      if ((two || t == 0) && any_row) {
        const float il = 1.0f / l;
        const int64_t pi = slot * wk.rows_cap + ur;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + ((int64_t)(d.at + j) * p.H + head) * D;
        float* part = wk.part_o + pi * D;
        const bool st_ok =
            valid && (cut ? in_bounds(p.err, ur, wk.rows_cap) : !(l < 0.0f) && in_bounds(p.err, d.at + j, p.T));
        const bool looked = two ? (gw > 0 && nt > 0) || gc < nt : gw > 0 || gc < n;
        const bool specials = looked && *(volatile const int*)&sh->specials[ds] > 0;
        const bool other = __any_sync(0xffffffffu, a1 != 0.0f);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          const uint32_t col = (uint32_t)c0;
          if (to_hand && c0 > 0) {  // (behind the first columns: the rows are there by now)
            hand_q((seq + 1) % kCaDesc);
            to_hand = false;
          }
          uint32_t ov[32];
          if (nt > 0) {
            tmem_ld_32x32b_x32(trow + ca_o_col(t) + col, ov);
            tmem_wait_ld(ov);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = 0u;
          }
          if (other) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t ow[16];
              tmem_ld_32x32b<16>(trow + ca_o_col(1) + col + 16u * (uint32_t)h, ow);
              tmem_wait_ld(ow);
              if (a1 != 0.0f) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  ov[16 * h + c] = __float_as_uint(__uint_as_float(ov[16 * h + c]) * a0 + __uint_as_float(ow[c]) * a1);
              }
            }
          }
          if (specials && valid) {
            uint32_t tmp[32];  // (not ov itself: its address would put it in memory)
#pragma unroll
            for (int c = 0; c < 32; ++c) tmp[c] = ov[c];
            ca_add_special<TYPE>(p, sh, ds, d.b, d.kvh, D, pos, (int)col, tmp);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = tmp[c];
          }
          if (!st_ok) continue;
          // a lane its own row, in whole sectors (through shared memory, whole lines at once: slower by the round trip)
          if (cut) {
#pragma unroll
            for (int c = 0; c < 32; c += 8) ca_store32(part + c0 + c, ov + c, true);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c)
              w[c] = ca_pack<TYPE>(__uint_as_float(ov[2 * c]) * il, __uint_as_float(ov[2 * c + 1]) * il);
            ca_store32(dst + c0, w, wk.wide != 0);
            ca_store32(dst + c0 + 16, w + 8, wk.wide != 0);
          }
        }
        if (cut && st_ok) wk.part_ml[pi] = make_float2(m, l);
        for (unsigned over = __ballot_sync(0xffffffffu, valid && !cut && l < 0.0f); over; over &= over - 1)
          ca_far_row<TYPE, D>(p, d, G, __shfl_sync(0xffffffffu, R, __ffs(over) - 1), lane, &sh->beat);
      }
      if (to_hand) hand_q((seq + 1) % kCaDesc);
      if (!two) {  // slot 1's scores and sums may be written again
        if (t == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->read);
        } else if (!ca_wait(&sh->read, shared_parts & 1u, p.err, &sh->beat)) {
          ok = false;
          break;
        }
        ++shared_parts;
      }
      tc_fence_before();
      if (cut) {
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->stored);
        if (warp == 4) {
          if (!ca_wait(&sh->stored, cut_parts & 1u, p.err, &sh->beat)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            int* done = wk.done + (in_bounds(p.err, d.first_cut, wk.ctas) ? d.first_cut : 0);
            const bool last = atomic_add_acq_rel(done, n) + n == d.nt;
            if (last) *done = 0;
            *(volatile int*)&sh->last = last ? 1 : 0;
            mbar_arrive(&sh->told);
          }
          __syncwarp();
        }
        if (!ca_wait(&sh->told, cut_parts & 1u, p.err, &sh->beat)) {
          ok = false;
          break;
        }
        ++cut_parts;
        if (*(volatile int*)&sh->last) {
          // the unit's pieces, merged in the order of the keys: their places first, each warp for itself
          __threadfence();
          int* list = reinterpret_cast<int*>(smem + t * L::kQ + qd * 32 * 128);  // (this warp's rows of Q)
          int np = 0;
          for (int cb = d.first_cut - 1;; cb += 32) {
            const int c = cb + lane;
            const bool in = c < C && bound(c) < d.u0 + d.v;
            const int from = in ? cut_at(c, d.u0, d.v, d.nt) : 0, to = in ? cut_at(c + 1, d.u0, d.v, d.nt) : 0;
            const unsigned has = __ballot_sync(0xffffffffu, to > from);
            if (to > from) list[np + __popc(has & ((1u << lane) - 1u))] = (2 * c + (from == 0 ? 1 : 0)) * wk.rows_cap;
            np += __popc(has);
            if (!__all_sync(0xffffffffu, in)) break;
          }
          __syncwarp();
          // loads in flight along rows too, or along pieces: whichever takes fewer turns, each of them a load's latency (512
          // rows of 8 heads after 30000 tokens: 115 us; with 8 rows and 2 pieces a turn 121)
          if ((d.rows + 31) / 32 * ((np + 3) / 4) < (d.rows + 7) / 8 * ((np + 7) / 8))
            ca_merge<TYPE, D, 4, 4>(p, wk, d, list, np, warp - 4, lane, &sh->beat);
          else
            ca_merge<TYPE, D, 1, 8>(p, wk, d, list, np, warp - 4, lane, &sh->beat);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->desc_free[ds]);
    }
  }

  // ---------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (queue && tid == 0 && atomic_add_acq_rel(wk.queue + 1, 1) == wk.ctas - 1) wk.queue[0] = wk.queue[1] = 0;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512u);
  }
}

// ------------------------------------------------------------------ host
struct CaPlan {
  int ctas, rows_cap;
  size_t done_bytes, ml_bytes, total;
};
static CaPlan ca_plan(int T, int H, int Hkv, int D, int num_sms) {
  CaPlan k;
  k.ctas = num_sms > 0 ? num_sms : 1;
  const int64_t rows = (int64_t)T * (H / Hkv);
  k.rows_cap = rows < 256 ? (int)rows : 256;
  k.done_bytes = ((size_t)(k.ctas + 2) * 4 + 255) / 256 * 256;
  k.ml_bytes = ((size_t)2 * k.ctas * k.rows_cap * 8 + 255) / 256 * 256;
  k.total = k.done_bytes + k.ml_bytes + (size_t)2 * k.ctas * k.rows_cap * D * 4;
  return k;
}

size_t kv16_attention_ws(int T, int H, int Hkv, int D, int num_sms) { return ca_plan(T, H, Hkv, D, num_sms).total; }

// The split's numbers stay below 2^55 (times the CTAs: 2^63), a unit's work times its tiles too.
bool kv16_attention_fits(int T, int B, int H, int Hkv, int max_blocks) {
  const double G = H / Hkv, units = (double)T * H / 256 + (double)B * Hkv;
  return G <= 1024 && max_blocks <= (1 << 21) &&
         units * kCaWeight2 * (G * (64.0 * max_blocks + kCaOverhead) + 256.0) < 36028797018963968.0;
}

template <int TYPE, int D>
static cudaError_t launch_ca(const CaMaps& maps, const Kv16AttnParams& p, const CaWork& wk, cudaStream_t stream) {
  constexpr int smem = CaLayout<D>::kTotal;
  const cudaError_t e =
      cudaFuncSetAttribute(kv16_attention_kernel<TYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv16_attention_kernel<TYPE, D>, dim3((unsigned)wk.ctas), dim3(kCaThreads), (size_t)smem, stream, maps,
                    p, wk);
}

cudaError_t launch_kv16_attention(const Kv16AttnParams& p, int type, int D, void* workspace, int num_sms,
                                  cudaStream_t stream) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!encode) return cudaErrorNotSupported;
  const CaPlan k = ca_plan(p.T, p.H, p.Hkv, D, num_sms);
  CaMaps maps;
  const cuuint64_t dims[4] = {64, 64, (cuuint64_t)D / 64, (cuuint64_t)p.pages * p.Hkv};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 128};
  const cuuint32_t box[4] = {64u, 64u, (cuuint32_t)D / 64, 1u}, es[4] = {1u, 1u, 1u, 1u};
  for (int c = 0; c < 2; ++c)
    if (encode(c ? &maps.v : &maps.k, type == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void*>(c ? p.v : p.k), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  CaWork wk;
  wk.by_g = fast_div((uint32_t)(p.H / p.Hkv));
  wk.ctas = k.ctas;
  wk.ctas_inv = k.ctas > 1 ? ~uint64_t(0) / (uint64_t)k.ctas : ~uint64_t(0);
  wk.tiles_inv = 1.0f / ((float)k.ctas * (float)(p.H / p.Hkv * kCaKeys));
  wk.rows_cap = k.rows_cap;
  wk.wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  wk.done = reinterpret_cast<int*>(ws);
  wk.queue = wk.done + k.ctas;
  wk.part_ml = reinterpret_cast<float2*>(ws + k.done_bytes);
  wk.part_o = reinterpret_cast<float*>(ws + k.done_bytes + k.ml_bytes);
  if (D == 128)
    return type == 0 ? launch_ca<0, 128>(maps, p, wk, stream) : launch_ca<1, 128>(maps, p, wk, stream);
  return type == 0 ? launch_ca<0, 64>(maps, p, wk, stream) : launch_ca<1, 64>(maps, p, wk, stream);
}

}  // namespace w4a16

#if W4A16_TEST_HOOKS
// Debug builds only (not part of the C ABI header): see g_test_skip_copy.
extern "C" int w4a16_test_set_skip_copy(int buf) {
  return (int)cudaMemcpyToSymbol(w4a16::g_test_skip_copy, &buf, sizeof(int));
}
#endif
