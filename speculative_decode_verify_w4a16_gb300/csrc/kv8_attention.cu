// Tree-masked verify attention over the paged 8-bit cache (contract in
// w4a16sv.h).
//
// The query rows of a KV head are its G = H / Hkv query heads at every tree
// node, row R = node * G + head-in-group, in row blocks of up to NP = 64 rows.
// The keys are the M side of both products, 128 of them a tile:
//   S^T [key][row]  = K [key][d] . Q^T         (M = 128 keys, N = rows)
//   O^T [d][row]   += V^T [d][key] . P^T       (M = 128 columns, N = rows)
// so that the few rows of a draft fill the N side exactly and the work of the
// softmax is rows x keys, not 128 x keys. The 8-bit keys go from HBM through
// TMA straight into the tensor cores (kind::f8f6f4): q is the sum of two e4m3
// terms, q 2^e = q1 + q2 / 32 with e such that the row's largest magnitude is
// in [128, 256), which together hold bf16's 8 bits exactly for elements down
// to 2^-14 of that maximum (absolute error 2^-23 of it below); the terms are
// separate N columns (S = S1 + S2 / 32), so that K is read from shared memory
// once. The 8-bit values are widened to fp16, exactly, on their way: four warps
// read them transposed (ldmatrix on 8-bit elements) and store V^T in TMEM as
// the A operand, because the softmax weights need more than e4m3 holds (P is
// rounded to fp16, half a step 2^-11). Through TMEM, not through shared
// memory: a tile's 32 KB of fp16 written there and read again by the MMAs took
// most of the shared-memory bandwidth, and an MMA with A in TMEM takes 27
// cycles instead of 48 (N = 48).
//
// A page's scales are powers of two per 64 keys: the keys' multiplies the
// scores; the values' is added to the exponent. P = 2^(s + log2 sv - m) is
// what multiplies the code, and the normaliser adds P / sv, in fp32.
//
// Online softmax: m is a reference per row, 7 below the maximum of s + log2 sv
// when it was last set; it is raised again only when a weight would pass 2^15
// (fp16 holds 2^15.99; weights down to 2^-14 keep all 11 bits, that is 2^-21
// of the largest). One vote per tile over the four warps finds that; the
// maximum itself, and the rescaling of O^T in TMEM, are computed only then (at
// the first tile of a part, and seldom after it). Blocks of zeros have scale 1,
// whatever their neighbours have: they, and pages that are not there, count as
// 2^-64, so that they do not raise m.
//
// Code that runs once per part (the query rows, the first maximum, the end) is
// kept short: a CTA meets it with cold instruction caches, and straight-line
// code then costs some 20 to 40 cycles an instruction. Hence the quotients without
// integer divisions and the merge of cut units after everything else, where
// all warps take part and no registers have to be kept (both together: the
// trees 225 -> 201 us, one request of one node 14.0 -> 12.6).
//
// The tile of bf16 rows, the tail page's (rows 0 .. 63 of the tile) and the
// tree's own (64 .. 127), comes last in a request's tiles, with bf16 operands
// (kind::f16) and the mask: tail row r for r < lens % 64, node j for the rows of
// j and its descendants. Last, because m is then what the 8-bit tiles' weights
// need, in fp16 and in units of their own value scales; the bf16 weights and the
// fp32 sums have range for any such m (raised only past 2^64). With that tile
// first, m came from it, and of small values the cached ones' weights were lost
// (what the order costs: the trees 197 -> 199 us, 3 requests with trees of 17
// nodes 15.4 -> 16.6, the others nothing).
// Rows that hold nothing are zeroed in shared memory, and so are values that are
// not finite in a node (a node does not see its siblings, and 0 * NaN is NaN);
// they are added at the end to the rows that do see the node.
//
// Work: every (request, KV head, row block) unit has 1 + ceil(full blocks / 2)
// tiles. The tiles of all units are laid end to end and cut into one run per
// SM; a CTA walks over its run, which may end one unit and start others. A
// unit inside one run is finished there; one that was cut leaves (m, l, O^T)
// per run, and the CTA that finishes last of them (a counter) merges them.
//
// Measured (one layer of 64 query heads on 8, e4m3): four requests of 120 to
// 131 K tokens, one node each (1.02 GB) 159 us, 0.95 of the HBM copy rate, which
// bounds it; 16 requests of 4 to 8 K tokens, chains of 5 (198 MB) 48 us, 0.61 of
// it; 16 of 2 to 4 K tokens with trees of 64 nodes (102 GFLOP) 199 us, 0.27 of
// the bf16 rate; one request of 1003 tokens and one node 10.6 us. The chains and
// trees are bound by the softmax warps' latency: a tile takes some 1600 cycles at
// 48 rows and 1800 at 64 (the products take 460 and 600 of them, the warps issue
// in 45 to 55 % of the cycles), and a part's start and end some 8000. Measured
// and not kept, against what there was at the time: 128 rows a block with 32 a
// warpgroup, the trees in 563 us (registers); 32 rows a warpgroup at 64, no gain
// (fewer warps to hide latency with), 8 rows at 48, the chains in 55 against 48
// (64 registers); the two terms' products added up in TMEM,
// 272 against 240; the next part's query rows prepared by a warp of its own,
// 273 against 232 (it takes 2500 cycles for four rows; their loads before the
// part's end: 225); scores given back when read, and fetched a tile ahead where
// registers allow, 208 against 201 and the chains 50 against 48; cut units
// announced at the CTA's end only, 206.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace w4a16 {

#if W4A16_TEST_HOOKS
// Debug builds only: the producer of CTA 0 leaves out the keys of the 8-bit tile
// with this index in its run (no copy, no arrival for it), so that the bounded
// waits run out and the kernel reports a timeout. -1: off.
__device__ int g_test_skip_tile = -1;
__device__ __forceinline__ bool test_skip_tile(int tile) {
  return blockIdx.x == 0 && tile == *(volatile int*)&g_test_skip_tile;
}
#else
__device__ __forceinline__ bool test_skip_tile(int) { return false; }
#endif

constexpr int kKaD = 128;
constexpr int kKaTile = 128;      // keys per tile
constexpr float kKaRoom = 7.0f;    // log2 of the largest weight when m is set
constexpr float kKaLimit = 15.0f;  // ... and where m is raised
constexpr float kKaLimit16 = 64.0f;  // ... and by the bf16 tile

// Quotients without integer divisions (FastDiv, and this): code that runs once is
// met with cold instruction caches, and a division is some 25 instructions.
// a / b, a < 2^31, from the quotient of floats: a few units off at most, then exact
__device__ __forceinline__ unsigned ka_quot(unsigned a, unsigned b) {
  unsigned q = (unsigned)__fdividef((float)a, (float)b);
  int r = (int)(a - q * b);
#pragma unroll 1
  for (; r < 0; r += (int)b) --q;
#pragma unroll 1
  for (; r >= (int)b; r -= (int)b) ++q;
  return q;
}

struct KaWork {  // the cut of the tiles into runs
  int row_blocks, np, G;  // G query heads a head
  FastDiv by_g, by_blocks, by_units, by_ctas;
  int* done;        // [ctas]: finished parts of the cut unit that begins in a run; zero at rest
  float2* part_ml;  // [2 ctas][np]
  float* part_o;    // [2 ctas][np][D]
};

__device__ __forceinline__ float ka_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t ka_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t ka_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// two fp16 x as e4m3 terms: x = c1 + c2 / 32 (the difference is exact)
__device__ __forceinline__ void ka_terms(uint32_t x, uint32_t& c1, uint32_t& c2) {
  asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 y, k;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, a;\n\t"
      "sub.f16x2 y, %2, y;\n\t"
      "mov.b32 k, 0x50005000;\n\t"  // 32, twice
      "mul.f16x2 y, y, k;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 b, y;\n\t"
      "cvt.u32.u16 %0, a;\n\t"
      "cvt.u32.u16 %1, b;\n\t}"
      : "=r"(c1), "=r"(c2)
      : "r"(x));
}
// four e4m3 codes widened to fp16 (exact)
__device__ __forceinline__ void ka_widen(uint32_t in, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(in));
}
// named barrier over one softmax warpgroup
__device__ __forceinline__ void ka_bar(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
// ... and with a vote: whether p holds in any of its threads
__device__ __forceinline__ bool ka_bar_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, %2, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}
// two fp32 lanes in one 64-bit register, for the paired fp32 instructions
__device__ __forceinline__ uint64_t ka_2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void ka_un2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ka_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t ka_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t ka_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float ka_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __noinline__ bool ka_wait_long(uint64_t* bar, uint32_t parity, unsigned* err) {
  return mbar_wait(bar, parity, err);
}
// Bounded wait by a whole warp, or by one thread: every lane tests the same
// barrier (a hint of a microsecond: the hardware wakes the warp when the phase
// completes, and a polling loop takes issue slots from the other warps). Once a
// wait has run out (still false) the later ones return at once: the warps that
// meet at named barriers then walk through the rest of their work, on garbage
// and in bounds, instead of leaving the others waiting.
__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t parity, unsigned* err, bool still = true) {
  if (still && !mbar_try_wait(bar, parity, 1000u)) still = ka_wait_long(bar, parity, err);
  return still;
}

// By a whole warp: whether the lane's block of codes (8 KB at v) holds zeros
// alone, for the lanes that ask. One load tells for nearly every block.
__device__ __noinline__ bool ka_zero_block(const uint8_t* v, bool ask) {
  constexpr uint32_t kMag = 0x7F7F7F7Fu;  // (a zero may have a sign)
  const int lane = threadIdx.x & 31;
  bool zero = false;
  if (ask) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(v));
    zero = ((x.x | x.y | x.z | x.w) & kMag) == 0u;
  }
#pragma unroll 1
  for (unsigned left = __ballot_sync(0xffffffffu, zero); left; left &= left - 1) {
    const int of = __ffs((int)left) - 1;
    const uint4* at = reinterpret_cast<const uint4*>(__shfl_sync(0xffffffffu, (unsigned long long)v, of)) + lane;
    uint32_t any = 0u;
#pragma unroll 4
    for (int i = 0; i < 64 * kKaD / 512; ++i) {
      const uint4 x = __ldg(at + 32 * i);
      any |= x.x | x.y | x.z | x.w;
    }
    if (__any_sync(0xffffffffu, (any & kMag) != 0u) && lane == of) zero = false;
  }
  return zero;
}

__device__ __forceinline__ int ka_len(const Kv8AttnParams& p, int b) {
  const int l = p.lens[b];
  return l < 0 ? 0 : l > p.max_len ? p.max_len : l;
}
__device__ __forceinline__ int ka_tiles(int len) { return 1 + (len / 64 + 1) / 2; }

// One part of a run: tiles lo .. hi - 1 of the nt tiles of unit u of request
// b; tile lo is tile at of all. Tile i holds blocks 2 i and 2 i + 1, the last
// one the bf16 rows.
struct KaSeg {
  int b, u, lo, hi, nt, len;
  unsigned at;
  __device__ __forceinline__ bool ends() const { return hi == nt; }       // holds the bf16 tile
  __device__ __forceinline__ bool bf16(int i) const { return i + 1 == nt; }
};
struct KaIter {
  unsigned at, left;
  int b, u, tile, units;
  int len, nt;
};
__device__ __forceinline__ bool ka_next(const Kv8AttnParams& p, KaIter& it, KaSeg& s) {
  if (it.left == 0 || it.b >= p.B) return false;
  const unsigned take = min((unsigned)(it.nt - it.tile), it.left);
  s = KaSeg{it.b, it.u, it.tile, it.tile + (int)take, it.nt, it.len, it.at};
  it.left -= take;
  it.at += take;
  it.tile = 0;
  if (++it.u == it.units) {
    it.u = 0;
    ++it.b;
    if (it.left > 0 && it.b < p.B) {
      it.len = ka_len(p, it.b);
      it.nt = ka_tiles(it.len);
    }
  }
  return true;
}

// As many runs of the T tiles as leave `least` (1 or 2) tiles each, one an SM at
// most; run c of them begins at c per + min(c, rest). (1 <= T < 2^31: the host
// checks.)
// Single tiles where the units have 16 or fewer on average: a tile costs more
// than the merge of twice the parts (8 units of 3 tiles 8.9 us against 11.0, of
// 9 tiles 10.8 against 12.4; of 33 tiles, though, 15.3 against 12.4, and one unit
// of 33 13.9 against 10.8).
struct KaCut {
  unsigned runs, per, rest;
  KaCut() = default;
  __device__ __forceinline__ KaCut(unsigned T, unsigned units, const FastDiv& by_ctas) {
    const unsigned least = (uint64_t)T > (uint64_t)16u * units ? 2u : 1u, most = least == 2u ? T / 2 : T;
    const bool all = most >= by_ctas.d;
    runs = all ? by_ctas.d : max(most, 1u);
    per = all ? (unsigned)by_ctas((int)T) : min(T, least);
    rest = T - per * runs;
  }
  __device__ __forceinline__ unsigned begin(unsigned c) const { return c * per + min(c, rest); }
  __device__ __forceinline__ unsigned owner(unsigned f) const {  // the run that holds tile f
    const unsigned big = rest * (per + 1u);
    const bool low = f < big;
    return (low ? 0u : rest) + ka_quot(low ? f : f - big, low ? per + 1u : per);
  }
};

// Sixteen rows, a value each in every lane: reduced over the warp by halving
// the rows at each exchange; lanes 2 r and 2 r + 1 return row r.
template <bool MAX>
__device__ __forceinline__ float ka_reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int h = 8, m = 16; h >= 1; h >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? v[i + h] : v[i], got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], m);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
  return MAX ? fmaxf(v[0], got) : v[0] + got;
}

template <int NP>
struct KaCfg {
  static constexpr int kRows = 16, kGroups = NP / kRows;  // softmax warpgroups, 16 rows each
  static constexpr int kSoft0 = 4, kConv0 = 4 + 4 * kGroups;
  static constexpr int kThreads = 32 * (kConv0 + 4);
  // stages of 128 keys (16 KB), as many as fit
  static constexpr int kStages = NP > 32 ? 4 : 5, kVStages = NP > 48 ? 3 : NP > 16 ? 4 : 5;
  static constexpr int kTileBytes = kKaTile * 128;
  static constexpr int kPBytes = NP * 256;
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kXOff = kVOff + kVStages * kTileBytes;  // a bf16 tile's values: halves of 64 columns
  static constexpr int kQ8Off = kXOff + 2 * kTileBytes;       // 2 NP rows of 128 bytes
  static constexpr int kQ16Off = kQ8Off + 2 * NP * 128;       // 2 halves of NP rows of 128 bytes
  static constexpr int kPOff = kQ16Off + 2 * NP * 128;
  static constexpr int kZeroOff = kPOff + 2 * kPBytes;        // 1 KB of zeros (8 rows of 128 bytes)
  static constexpr int kMaskOff = kZeroOff + 1024;            // u64 [NP]: nodes a row sees
  static constexpr int kGmOff = kMaskOff + NP * 8;            // float4 [NP / 2]: g, g, -m, -m of two rows
  static constexpr int kPartOff = kGmOff + NP * 8;            // float [4][NP]
  static constexpr int kRowOff = kPartOff + NP * 16;          // int [NP]
  static constexpr int kScaleOff = kRowOff + NP * 4;          // float4 [16][2]: a tile's blocks
  static constexpr int kSeeOff = kScaleOff + 16 * 2 * 16;     // u16 [groups][128]
  static constexpr int kBarOff = kSeeOff + kGroups * 256;
  static constexpr int kNumBars = 2 * kStages + 2 * kVStages + 12;
  static constexpr int kTotal = kBarOff + kNumBars * 8 + 1024;
  // TMEM columns: scores (two terms) of two tiles, O^T, then V^T of two tiles
  // (fp16 pairs along the keys: 64 columns)
  static constexpr uint32_t kOCol = 4 * NP, kVCol = 5 * NP;
  static constexpr uint32_t kCols = 5 * NP + 128 <= 256 ? 256 : 512;
  static_assert(kTotal + 1024 <= 227 * 1024, "shared memory");
  static_assert(NP % 16 == 0 && NP <= 64, "row block");
};

// Values that are not finite, of nodes that a row sees, added to O^T (in TMEM):
// they were taken out of the products so as not to reach the other rows.
template <int Q>
__device__ __noinline__ void ka_add_bad(const Kv8AttnParams& p, int b, int kvh, unsigned long long bad,
                                        const uint64_t* mask, uint32_t col, int d) {
#pragma unroll 1
  for (int q0 = 0; q0 < Q; q0 += 8) {
    uint32_t o[8];
    tmem_ld_32x32b<8>(col + (uint32_t)q0, o);
    tmem_wait_ld();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
#pragma unroll 1
      for (unsigned long long m = bad & mask[q0 + q]; m; m &= m - 1) {
        const int j = __ffsll((long long)m) - 1;
        const float v = __bfloat162float(p.v_new[((int64_t)b * p.n + j) * p.kv_stride + kvh * kKaD + d]);
        if (!(fabsf(v) < INFINITY)) o[q] = __float_as_uint(__uint_as_float(o[q]) + v);
      }
    }
    tmem_st_32x32b_x8(col + (uint32_t)q0, o);
  }
  tmem_wait_st();
}

// barrier over all softmax warpgroups
template <int GROUPS>
__device__ __forceinline__ void ka_bar_all() {
  asm volatile("barrier.cta.sync 9, %0;" ::"n"(128 * GROUPS) : "memory");
}

// A cut unit whose parts are all there, for this CTA to merge
struct KaMerge {
  int b, u;
  unsigned s0, c0, parts;  // the first part in slot s0, that of run c0 + k in slot 2 (c0 + k)
};

// By the whole CTA, at its end: a warp takes 4 rows, a lane 4 columns of each;
// lane 4 k + i has (m, l) of the k-th of 8 parts in row r + i. The loads of
// kAhead parts are in flight together, the first ones' next to the (m, l): what
// costs here is the latency of L2.
template <int NP>
__device__ __forceinline__ void ka_merge(const Kv8AttnParams& p, const KaWork& wk, const KaMerge& mg, int r, int lane) {
  constexpr int kAhead = NP <= 32 ? 4 : 2;
  const unsigned parts = mg.parts;
  auto slot = [&](unsigned k) { return (size_t)(k ? 2u * (mg.c0 + k) : mg.s0) * NP + r; };
  float4 x[kAhead][4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto load = [&](unsigned k0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (k0 + a < parts) {
        const float4* src = reinterpret_cast<const float4*>(wk.part_o + slot(k0 + a) * kKaD) + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[a][i] = __ldcg(src + i * (kKaD / 4));
      }
  };
  auto stat = [&](unsigned k0) {
    const unsigned k = k0 + (lane >> 2);
    return k < parts ? __ldcg(&wk.part_ml[slot(k) + (lane & 3)]) : make_float2(-INFINITY, 0.0f);
  };
  load(0u);
  float2 ml = stat(0u);
  float M = ml.x;
#pragma unroll 1
  for (unsigned k = 8; k < parts; k += 8) M = fmaxf(M, stat(k).x);
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float l = 0.0f;
#pragma unroll 1
  for (unsigned k8 = 0; k8 < parts; k8 += 8) {
    if (k8) ml = stat(k8);
    const float w = ml.x == M ? 1.0f : ka_ex2(ml.x - M);  // 0 for a part that is not there
    l = fmaf(w, ml.y, l);
#pragma unroll 1
    for (unsigned k = k8; k < min(k8 + 8u, parts); k += kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (k + a < parts) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, (int)(4u * (k - k8 + a)) + i);
            o[i].x = fmaf(wi, x[a][i].x, o[i].x);
            o[i].y = fmaf(wi, x[a][i].y, o[i].y);
            o[i].z = fmaf(wi, x[a][i].z, o[i].z);
            o[i].w = fmaf(wi, x[a][i].w, o[i].w);
          }
        }
      if (k + kAhead < parts) load(k + kAhead);
    }
  }
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = 1.0f / l;
  const int G = wk.G, kvh = wk.by_blocks(mg.u), R0 = (mg.u - kvh * wk.row_blocks) * NP + r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = __shfl_sync(0xffffffffu, inv, i);
    const int R = R0 + i, j = wk.by_g(R), row = (mg.b * p.n + j) * p.H + kvh * G + R - j * G;
    if (R < p.n * G && in_bounds(p.err, row, (int64_t)p.B * p.n * p.H))
      reinterpret_cast<uint2*>(p.out + (int64_t)row * kKaD)[lane] =
          make_uint2(ka_bf162(o[i].x * v, o[i].y * v), ka_bf162(o[i].z * v, o[i].w * v));
  }
}

struct KaMaps {
  CUtensorMap k, v, k_tail, v_tail, k_new, v_new;
};

template <int NP, int FMT>
__global__ void __launch_bounds__(KaCfg<NP>::kThreads, 1)
    kv8_attention_kernel(const __grid_constant__ KaMaps maps, const Kv8AttnParams p, const KaWork wk) {
  using C = KaCfg<NP>;
  constexpr int S = C::kStages, SV = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  // the next 1024-byte boundary, by an offset: through an integer the compiler
  // would lose sight of the address space and load and store generically
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* mask_s = reinterpret_cast<uint64_t*>(smem + C::kMaskOff);
  float* gm_s = reinterpret_cast<float*>(smem + C::kGmOff);  // row r: g at 4 (r / 2) + r % 2, -m two on
  float* part_s = reinterpret_cast<float*>(smem + C::kPartOff);
  int* row_s = reinterpret_cast<int*>(smem + C::kRowOff);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* k_free = k_full + S;
  uint64_t* v_full = k_free + S;
  uint64_t* v_free = v_full + SV;
  uint64_t* w_full = v_free + SV;  // [2] 16-bit values ready
  uint64_t* s_full = w_full + 2;   // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* pv_done = p_full + 2;  // [2]
  uint64_t* q_ready = pv_done + 2;
  uint64_t* x_full = q_ready + 1;  // a bf16 tile's values
  uint64_t* mma_fin = x_full + 1;  // [2]
  float4* scale_s = reinterpret_cast<float4*>(smem + C::kScaleOff);  // tile tc, block half: 2 (tc % 16) + half
  uint16_t* see_s = reinterpret_cast<uint16_t*>(smem + C::kSeeOff);
  __shared__ uint32_t tmem_s;
  __shared__ unsigned scan_s[32];
  __shared__ unsigned s_pre;
  __shared__ int s_b;
  __shared__ KaCut cut_s;
  __shared__ KaMerge merge_s[2];  // a run's first and last unit
  __shared__ int par_s[64];
  __shared__ unsigned long long bad_s[4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&k_full[s], 2);  // the copies, and the scales (or nothing)
      mbar_init(&k_free[s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_free[s], 4);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&w_full[k], 4);
      mbar_init(&s_full[k], 1);
      mbar_init(&p_full[k], 4 * C::kGroups);
      mbar_init(&pv_done[k], 1);
      mbar_init(&mma_fin[k], 1);
    }
    mbar_init(q_ready, 4 * C::kGroups);
    mbar_init(x_full, 1);
    fence_mbarrier_init();
    merge_s[0].parts = merge_s[1].parts = 0u;
  }
  if (warp == 2) {
    tmem_alloc(&tmem_s, C::kCols);
    tmem_relinquish();
  }
  if (warp == 3) {
    if (lane < 6) tma_prefetch_map(&maps.k + lane);
    for (int k = lane; k < 64; k += 32) reinterpret_cast<uint4*>(smem + C::kZeroOff)[k] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  grid_dependency_wait();
  // ---- this CTA's run: sums of the requests' tiles
  const int units = p.Hkv * wk.row_blocks;
  int n0 = 0;  // request tid's
  if (tid < p.B) {
    n0 = ka_tiles(ka_len(p, tid));
    if (blockIdx.x == 0 && (unsigned)p.lens[tid] > (unsigned)p.max_len) report_error(p.err, kErrInput);
  }
  unsigned T;
  {
    unsigned x = (unsigned)n0;
#pragma unroll 1
    for (int b = tid + C::kThreads; b < p.B; b += C::kThreads) {
      x += (unsigned)ka_tiles(ka_len(p, b));
      if (blockIdx.x == 0 && (unsigned)p.lens[b] > (unsigned)p.max_len) report_error(p.err, kErrInput);
    }
    x = __reduce_add_sync(0xffffffffu, x);
    if (lane == 0) scan_s[warp] = x;
    __syncthreads();
    x = lane < C::kThreads / 32 ? scan_s[lane] : 0u;
    T = __reduce_add_sync(0xffffffffu, x) * (unsigned)units;
  }
  unsigned f0, f1;
  {
    const KaCut runs(T, (unsigned)(p.B * units), wk.by_ctas);
    f0 = runs.begin(blockIdx.x);
    f1 = blockIdx.x < runs.runs ? runs.begin(blockIdx.x + 1u) : f0;
    if (tid == 0) cut_s = runs;
  }
  {
    const unsigned target = (unsigned)wk.by_units((int)f0);  // tiles of one unit of the requests before b <= target
    unsigned before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B && before <= target; b0 += C::kThreads) {
      const int b = b0 + tid, n = b0 == 0 ? n0 : b < p.B ? ka_tiles(ka_len(p, b)) : 0;
      unsigned x = (unsigned)n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) scan_s[warp] = x;
      __syncthreads();
      const unsigned w = lane < C::kThreads / 32 ? scan_s[lane] : 0u;
      const unsigned at = before + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + x - (unsigned)n;
      before += __reduce_add_sync(0xffffffffu, w);
      if (b < p.B && target >= at && target < at + (unsigned)n) {
        s_b = b;
        s_pre = at;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  // (a CTA past the last run walks over nothing)
  KaIter it;
  {
    it.at = f0;
    it.left = f1 - f0;
    it.units = units;
    it.b = it.left > 0 ? s_b : 0;
    it.len = ka_len(p, it.b);
    it.nt = ka_tiles(it.len);
    const unsigned rel = it.left > 0 ? f0 - (unsigned)units * s_pre : 0u;
    it.u = (int)ka_quot(rel, (unsigned)it.nt);
    it.tile = (int)rel - it.u * it.nt;
  }
  KaSeg sg;
  int issued = 0;
  if (warp == 0) {
    // ---------------------------------------------------------- producer
    // K stages are used in order; a bf16 tile takes two neighbours (32 KB), and
    // passes over the last stage, which has none. Every use of a stage, a
    // passed one too, completes a phase of its full and its free barrier.
    // (A bf16 tile's values have a buffer of their own: the widening warps ask
    // for them.)
    int kc = 0, vc = 0, tc = 0;  // uses of the K and V stages, tiles so far
    int k_more = 0;      // a use of K whose tile was given up
    bool ok = true;
    auto k_wait = [&](int use) {
      return use < S || ka_wait(&k_free[use % S], (uint32_t)(use / S - 1) & 1u, p.err);
    };
    while (ok && ka_next(p, it, sg)) {
      const int kvh = wk.by_blocks(sg.u);
      // 8-bit tiles: lane 2 k + h has block h of the k-th of 16 tiles, its page and
      // scales; the next 16 tiles' are asked for ahead.
      const int full = sg.len / 64, end8 = min(sg.hi, sg.nt - 1);
      const int32_t* tab = p.table + (int64_t)sg.b * p.max_blocks;
      auto page_of = [&](int i) {  // of the 16 tiles from i on; -2: no such block
        const int blk = 2 * i + lane;
        return blk < full && blk < 2 * end8 ? max(tab[blk], -1) : -2;  // (any negative entry is a bad page)
      };
      int page_n = page_of(sg.lo), page = -2;
      float sk = 0.0f, lsv = 0.0f, isv = 1.0f, sk_n = 0.0f, sv_n = 1.0f;
      auto scales_of = [&]() {  // of the pages asked for earlier
        sk_n = 0.0f;
        sv_n = 1.0f;
        if (page_n >= 0 && page_n < p.pages) {
          sk_n = p.k_scale[(int64_t)page_n * p.Hkv + kvh];
          sv_n = p.v_scale[(int64_t)page_n * p.Hkv + kvh];
        } else if (page_n != -2) {
          report_error(p.err, kErrInput);
          page_n = -1;
        }
      };
      scales_of();
#pragma unroll 1
      for (int i = sg.lo; ok && i < end8; ++i, ++tc) {
        const int k = (i - sg.lo) & 15;
        if (k == 0) {
          page = page_n;
          page_n = page_of(i + 16);
        } else if (k == 8) {
          scales_of();
        }
        const int pa = __shfl_sync(0xffffffffu, page, 2 * k), pb = __shfl_sync(0xffffffffu, page, 2 * k + 1);
        // a page that is not there: past the tensor's end, filled with zeros
        const int none = p.pages * p.Hkv, ks = kc % S, vs = vc % SV;
        const int za = pa < 0 ? none : pa * p.Hkv + kvh, zb = pb < 0 ? none : pb * p.Hkv + kvh;
        if (lane == 0) {
          ok = k_wait(kc);
          if (ok && !test_skip_tile(tc)) {
            uint8_t* kd = smem + C::kKOff + ks * C::kTileBytes;
            mbar_arrive_expect_tx(&k_full[ks], C::kTileBytes);
            tma_load_3d(kd, &maps.k, 0, 0, za, &k_full[ks]);
            tma_load_3d(kd + 8192, &maps.k, 0, 0, zb, &k_full[ks]);
          }
        }
        // key scale, log2 of the value scale, its inverse, 1 for no block
        if (k == 0) {
          sk = sk_n;
          const bool one = page >= 0 && sv_n == 1.0f;  // perhaps a block of zeros
          bool nothing = page == -1;
          if (__any_sync(0xffffffffu, one))
            nothing |= ka_zero_block(p.v + ((int64_t)(one ? page : 0) * p.Hkv + kvh) * (64 * kKaD), one);
          lsv = nothing ? -64.0f : log2f(sv_n);
          isv = nothing ? 18446744073709551616.0f : 1.0f / sv_n;
        }
        if ((lane >> 1) == k) scale_s[2 * (tc & 15) + (lane & 1)] = make_float4(sk, lsv, isv, page == -2 ? 1.0f : 0.0f);
        __syncwarp();
        if (lane == 0) {
          if (ok) {
            mbar_arrive(&k_full[ks]);
            k_more = 1;
            if (vc >= SV) ok = ka_wait(&v_free[vs], (uint32_t)(vc / SV - 1) & 1u, p.err);
          }
          if (ok) {
            uint8_t* vd = smem + C::kVOff + vs * C::kTileBytes;
            mbar_arrive_expect_tx(&v_full[vs], C::kTileBytes);
            tma_load_3d(vd, &maps.v, 0, 0, za, &v_full[vs]);
            tma_load_3d(vd + 8192, &maps.v, 0, 0, zb, &v_full[vs]);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (ok) {
          ++kc;
          ++vc;
          k_more = 0;
        }
      }
      if (ok && sg.ends()) {
        const int t = sg.len & 63;
        const bool pass = kc % S == S - 1;
        if (lane == 0) {
          const int tail = p.tails[sg.b];
          if (pass && (ok = k_wait(kc))) {
            mbar_arrive(&k_full[S - 1]);
            mbar_arrive(&k_full[S - 1]);
          }
          const int use = kc + (pass ? 1 : 0), s = use % S;
          ok = ok && k_wait(use) && k_wait(use + 1);
          if (ok) {
            const bool tok = t > 0 && tail >= 0 && tail < p.tail_pages;
            if (t > 0 && !tok) report_error(p.err, kErrInput);
            uint8_t* kd = smem + C::kKOff + s * C::kTileBytes;
            scale_s[2 * (tc & 15)] = scale_s[2 * (tc & 15) + 1] = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
            mbar_arrive(&k_full[s + 1]);
            mbar_arrive(&k_full[s + 1]);
            mbar_arrive(&k_full[s]);
            mbar_arrive_expect_tx(&k_full[s], (uint32_t)((tok ? 64 : 0) + p.n) * 256u);
            for (int h = 0; h < 2; ++h) {
              if (tok) tma_load_3d(kd + h * C::kTileBytes, &maps.k_tail, 64 * h, 0, tail * p.Hkv + kvh, &k_full[s]);
              tma_load_4d(kd + h * C::kTileBytes + 8192, &maps.k_new, 64 * h, kvh, 0, sg.b, &k_full[s]);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (ok) kc += pass ? 3 : 2;
        ++tc;
      }
    }
    // every copy has landed before the CTA exits (it has, unless a wait ran
    // out somewhere): the last use of each stage
    if (lane == 0) {
      const int ke = kc + k_more;
      for (int u = ke > S ? ke - S : 0; u < ke; ++u) mbar_wait(&k_full[u % S], (uint32_t)(u / S) & 1u, p.err);
      for (int u = vc > SV ? vc - SV : 0; u < vc; ++u) mbar_wait(&v_full[u % SV], (uint32_t)(u / SV) & 1u, p.err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ O^T MMAs
    constexpr uint32_t id_o8 = umma_idesc(NP, 0u, 0u, 0u, 1u), id_o16 = umma_idesc(NP, 1u, 1u, 1u, 1u);
    const uint32_t xb = smem_u32(smem + C::kXOff), pb = smem_u32(smem + C::kPOff);
    int tc = 0;  // tiles so far
    bool ok = true;
    while (ok && ka_next(p, it, sg)) {
#pragma unroll 1
      for (int i = sg.lo; i < sg.hi; ++i, ++tc) {
        const int w = tc & 1;
        const uint32_t ph = (uint32_t)(tc >> 1) & 1u;
        ok = ka_wait(&w_full[w], ph, p.err) && ka_wait(&p_full[w], ph, p.err);
        if (!ok) break;
        tc_fence_after();
        // P^T: chunks of 8 rows, 16 bytes a key. 16 keys an MMA. V^T from TMEM,
        // or a bf16 tile's from shared memory: 128-byte rows of 64 columns a
        // key, the other 64 columns a half on
        const uint32_t bp = pb + (uint32_t)(w * C::kPBytes);
        if (sg.bf16(i)) {
#pragma unroll 1
          for (int k = 0; k < 8; ++k)
            umma_bf16_ss_warp(tmem + C::kOCol,
                              umma_desc_sw128_mnmajor(xb + 2048u * (uint32_t)k, (uint32_t)C::kTileBytes, 1024u),
                              umma_desc_flat_mnmajor(bp + 256u * (uint32_t)k, 128u, 2048u), id_o16,
                              (i > sg.lo || k > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16_ts_warp(tmem + C::kOCol, tmem + C::kVCol + 64u * (uint32_t)w + 8u * (uint32_t)k,
                              umma_desc_flat_mnmajor(bp + 256u * (uint32_t)k, 128u, 2048u), id_o8,
                              (i > sg.lo || k > 0) ? 1u : 0u);
        }
        umma_commit_warp(&pv_done[w]);
        issued = 1;
      }
    }
    if (issued) umma_commit_warp(&mma_fin[0]);
  } else if (warp == 3) {
    // ------------------------------------------------------------ S^T MMAs
    // (a warp of its own: a tile's scores go out when P V of two tiles before
    // is complete, so that a tile whose scores are there also has its P buffer)
    constexpr uint32_t id_s8 = umma_idesc(2 * NP, (uint32_t)FMT, 0u, 0u, 0u);
    constexpr uint32_t id_s16 = umma_idesc(NP, 1u, 1u, 0u, 0u);
    const uint32_t kb = smem_u32(smem + C::kKOff);
    const uint32_t q8 = smem_u32(smem + C::kQ8Off), q16 = smem_u32(smem + C::kQ16Off);
    const uint64_t zero = umma_desc_sw128_kmajor(smem_u32(smem + C::kZeroOff)) & ~((uint64_t)0x3FFFu << 32);
    int kc = 0, tc = 0, seg = 0;  // K stages, tiles, parts so far
    bool ok = true;
    while (ok && ka_next(p, it, sg)) {
      ok = ka_wait(q_ready, (uint32_t)seg & 1u, p.err);
#pragma unroll 1
      for (int i = sg.lo; ok && i < sg.hi; ++i, ++tc) {
        const uint32_t d = tmem + (uint32_t)(tc & 1) * 2u * NP;
        if (tc >= 2) ok = ka_wait(&pv_done[tc & 1], (uint32_t)((tc - 2) >> 1) & 1u, p.err);
        if (sg.bf16(i) && kc % S == S - 1) {  // the stage that the producer passed over
          ok = ka_wait(&k_full[S - 1], (uint32_t)(kc / S) & 1u, p.err, ok);
          umma_commit_warp(&k_free[S - 1]);
          ++kc;
        }
        const int s = kc % S;
        ok = ka_wait(&k_full[s], (uint32_t)(kc / S) & 1u, p.err, ok);
        if (sg.bf16(i)) ok = ka_wait(&k_full[s + 1], (uint32_t)((kc + 1) / S) & 1u, p.err, ok);
        issued = 1;
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = kb + (uint32_t)s * C::kTileBytes;
        if (sg.bf16(i)) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16_ss_warp(d, umma_desc_sw128_kmajor(a + (uint32_t)((k >> 2) * C::kTileBytes + 32 * (k & 3))),
                              umma_desc_sw128_kmajor(q16 + (uint32_t)((k >> 2) * NP * 128 + 32 * (k & 3))), id_s16,
                              k > 0 ? 1u : 0u);
          // the second term's columns: zeros (one 8-row group of zeros stands
          // for all of both operands: stride 0)
          umma_bf16_ss_warp(d + NP, zero, zero, id_s16, 0u);
          umma_commit_warp(&k_free[s]);
          umma_commit_warp(&k_free[s + 1]);
          kc += 2;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8_ss_warp(d, umma_desc_sw128_kmajor(a + 32u * (uint32_t)k),
                            umma_desc_sw128_kmajor(q8 + 32u * (uint32_t)k), id_s8, k > 0 ? 1u : 0u);
          umma_commit_warp(&k_free[s]);
          ++kc;
        }
        umma_commit_warp(&s_full[tc & 1]);
      }
      ++seg;
    }
    if (issued) umma_commit_warp(&mma_fin[1]);
  } else if (warp >= C::kConv0) {
    // ------------------------------------------------- values to fp16 in TMEM
    // Warp qd owns the TMEM lanes (columns d of the values) 32 qd .. + 31. A
    // 16 x 16 ldmatrix of 8-bit elements, transposed, gives a lane the codes of
    // keys 4 (l % 4) .. + 3 at d = l / 4 and l / 4 + 8: widened, the fragment of
    // a 16x256b TMEM store of 16 lanes d and 8 columns (16 keys).
    const int ct = tid - 32 * C::kConv0, qd = warp & 3;
    int vc = 0, tc = 0, xc = 0, seg = 0, last = -2;  // last: the latest bf16 tile
    bool ok = true;
    while (ka_next(p, it, sg)) {
      // The bf16 tile's values: fetched and made ready at the part's start, while
      // the softmax warps are at the last part's end and at this one's query rows,
      // once P V of the last such tile has left their buffer (and so all four warps
      // are past it)
      bool to_do = sg.ends();
      const int t = sg.len & 63, tail = p.tails[sg.b];
      const bool tok = t > 0 && tail >= 0 && tail < p.tail_pages;
      if (to_do) {
        if (last >= 0 && last >= tc - 2) ok = ka_wait(&pv_done[last & 1], (uint32_t)(last >> 1) & 1u, p.err, ok);
        last = tc + sg.hi - sg.lo - 1;
        if (ct == 0) bad_s[seg & 3] = 0ull;
        if (ct == 0 && ok) {
          const int kvh = wk.by_blocks(sg.u);
          uint8_t* w = smem + C::kXOff;
          mbar_arrive_expect_tx(x_full, (uint32_t)((tok ? 64 : 0) + p.n) * 256u);
          for (int h = 0; h < 2; ++h) {
            if (tok) tma_load_3d(w + h * C::kTileBytes, &maps.v_tail, 64 * h, 0, tail * p.Hkv + kvh, x_full);
            tma_load_4d(w + h * C::kTileBytes + 8192, &maps.v_new, 64 * h, kvh, 0, sg.b, x_full);
          }
        }
        __syncwarp();
      }
      for (int i = sg.lo; i < sg.hi; ++i, ++tc) {
        // P V (tc - 2) has left the TMEM buffer
        if (tc >= 2) ok = ka_wait(&pv_done[tc & 1], (uint32_t)((tc - 2) >> 1) & 1u, p.err, ok);
        if (to_do) {
          to_do = false;
          uint8_t* w = smem + C::kXOff;
          asm volatile("barrier.cta.sync 8, 128;" ::: "memory");  // (ids 1 .. 4 and 9: the softmax)
          ok = ka_wait(x_full, (uint32_t)xc & 1u, p.err, ok);
          ++xc;
          // thread = row of the tile: its 256 bytes, both halves
          const bool node = ct >= 64;
          const bool there = node ? ct - 64 < p.n : tok && ct < t;
          uint4* row[2] = {reinterpret_cast<uint4*>(w + ct * 128),
                           reinterpret_cast<uint4*>(w + C::kTileBytes + ct * 128)};
          bool bad = false;
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            uint4* at = row[k >> 3] + ((k + ct) & 7);
            if (!there) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else if (node) {
              uint4 x = *at;
              uint32_t* e = &x.x;
              bool any = false;
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                if ((e[m] & 0x7F80u) == 0x7F80u) {
                  e[m] &= 0xFFFF0000u;
                  any = true;
                }
                if ((e[m] & 0x7F800000u) == 0x7F800000u) {
                  e[m] &= 0xFFFFu;
                  any = true;
                }
              }
              if (any) *at = x;
              bad |= any;
            }
          }
          if (bad) atomicOr(&bad_s[seg & 3], 1ull << (ct - 64));
          fence_proxy_async_smem();
        }
        if (!sg.bf16(i)) {
          const int s = vc % SV;
          ok = ka_wait(&v_full[s], (uint32_t)(vc / SV) & 1u, p.err, ok);
          ++vc;
          const uint32_t v = smem_u32(smem + C::kVOff + s * C::kTileBytes);
#pragma unroll
          for (int dh = 0; dh < 2; ++dh) {
            uint32_t x[16];  // 16 columns d of 128 keys
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 32 * k + lane;
              ldmatrix_b8_trans_x2(v + (uint32_t)(r * 128 + (((2 * qd + dh) ^ (r & 7)) << 4)), x + 4 * k);
            }
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
              uint32_t o[16];
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const uint32_t in = x[8 * kh + m];
                if constexpr (FMT == 0) {
                  ka_widen(in, o[2 * m], o[2 * m + 1]);
                } else {  // e5m2 is the upper byte of fp16
                  o[2 * m] = __byte_perm(in, 0u, 0x1404);
                  o[2 * m + 1] = __byte_perm(in, 0u, 0x3424);
                }
              }
              tmem_st_16x256b_x4(tmem + ((uint32_t)(32 * qd + 16 * dh) << 16) + C::kVCol +
                                     64u * (uint32_t)(tc & 1) + 32u * (uint32_t)kh,
                                 o);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_free[s]);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_full[tc & 1]);
      }
      ++seg;
    }
  } else if (warp >= C::kSoft0) {
    // ------------------------------------------------------------ softmax
    constexpr int Q = C::kRows;
    const int wg = (warp - C::kSoft0) >> 2, qd = warp & 3;
    const int key = qd * 32 + lane;  // the thread's key of a tile (TMEM lane)
    const int st = tid - 32 * C::kSoft0 - 128 * wg;  // thread of the warpgroup
    const int qa = wg * Q;                           // its first row
    const uint32_t trow = tmem + ((uint32_t)(32 * qd) << 16);
    const int bar = 1 + wg;
    const int G = wk.G, rows = p.n * G;
    const float4* gm = reinterpret_cast<const float4*>(gm_s) + (qa >> 1);
    // where the thread's 16 columns of a part's query row are (eight lanes a
    // row); null for a row that does not exist
    auto q_at = [&](const KaSeg& g) {
      const int kvh = wk.by_blocks(g.u), R = (g.u - kvh * wk.row_blocks) * NP + qa + (st >> 3), j = wk.by_g(R);
      return R < rows ? p.q + ((int64_t)g.b * p.n + j) * p.q_stride + (kvh * G + R - j * G) * kKaD + 16 * (st & 7)
                      : nullptr;
    };
    int tc = 0, seg = 0;
    bool ok = true;
    uint4 v[2];  // the thread's 16 columns of a part's query row
    auto q_load = [&](const __nv_bfloat16* at) {
      v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
      if (at) {
        v[0] = reinterpret_cast<const uint4*>(at)[0];
        v[1] = reinterpret_cast<const uint4*>(at)[1];
      }
    };
    {
      KaIter first = it;
      if (ka_next(p, first, sg)) q_load(q_at(sg));
    }
    while (ka_next(p, it, sg)) {
      const int kvh = wk.by_blocks(sg.u), rb = sg.u - kvh * wk.row_blocks;
      // ---- Q: x = q 2^ex, |x| < 256, as bf16 and as two e4m3 terms
      {
        if (sg.ends() && p.parents && st < p.n) {
          // the parents (bad ones reported and cut off), for the masks; every
          // warpgroup writes the same
          int up = p.parents[(int64_t)sg.b * p.n + st];
          if (st == 0 ? up != -1 : (up < 0 || up >= st)) {
            report_error(p.err, kErrInput);
            up = -1;
          }
          par_s[st] = up;
        }
        const int r = qa + (st >> 3), c = st & 7, sw = r & 7;
        uint32_t in[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        // the largest magnitude (two side by side); without what is not finite
        unsigned m2 = 0;
#pragma unroll
        for (int e = 0; e < 8; e += 2) m2 = __vimax3_u16x2(m2, in[e] & 0x7FFF7FFFu, in[e + 1] & 0x7FFF7FFFu);
        unsigned m = max(m2 & 0xFFFFu, m2 >> 16);
        if (m >= 0x7F80u) {  // an infinity becomes a NaN, which e4m3 has; the row is NaN either way
          m = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const unsigned lo = in[e] & 0x7FFFu, hi = (in[e] >> 16) & 0x7FFFu;
            if (lo >= 0x7F80u) in[e] |= 0x7FFFu;
            if (hi >= 0x7F80u) in[e] |= 0x7FFF0000u;
            m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = min(134 - (int)(m >> 7), 120);  // |q| 2^ex in [128, 256)
        const float up = __uint_as_float((unsigned)(127 + ex) << 23);
        // x in fp16: its 8 bits are exact above 2^-16 (2^-24 of the maximum)
        uint32_t t1[4], t2[4], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = __uint_as_float(in[e] << 16) * up, x1 = __uint_as_float(in[e] & 0xFFFF0000u) * up;
          w[e] = ka_bf162(x0, x1);
          uint32_t c1, c2;
          ka_terms(ka_half2(x0, x1), c1, c2);
          t1[e >> 1] = (e & 1) ? t1[e >> 1] | (c1 << 16) : c1;
          t2[e >> 1] = (e & 1) ? t2[e >> 1] | (c2 << 16) : c2;
        }
        uint8_t* q8 = smem + C::kQ8Off + r * 128 + ((c ^ sw) << 4);
        uint8_t* q16 = smem + C::kQ16Off + (c >> 2) * NP * 128 + r * 128;
        *reinterpret_cast<uint4*>(q8) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
        *reinterpret_cast<uint4*>(q8 + NP * 128) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
        *reinterpret_cast<uint4*>(q16 + (((2 * (c & 3)) ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(q16 + (((2 * (c & 3) + 1) ^ sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        if (c == 0) {
          const int R = rb * NP + r, j = wk.by_g(R);
          gm_s[4 * (r >> 1) + (r & 1)] = __uint_as_float((unsigned)(127 - ex) << 23) * p.scale_log2;
          gm_s[4 * (r >> 1) + 2 + (r & 1)] = 0.0f;
          row_s[r] = R < rows ? (sg.b * p.n + j) * p.H + kvh * G + R - j * G : -1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
        ka_bar(bar);
        if (sg.ends()) {
          if (st < Q) {
            const int R = rb * NP + qa + st, j = wk.by_g(R);
            uint64_t mk = 0;
            if (R < rows) {
              if (p.parents)
#pragma unroll 1
                for (int k = j; k >= 0; k = par_s[k]) mk |= 1ull << k;
              else
                mk = j == 63 ? ~0ull : (1ull << (j + 1)) - 1ull;
            }
            mask_s[qa + st] = mk;
          }
          ka_bar(bar);
        }
      }
      if (sg.ends()) {
        uint32_t see = 0xFFFFu;
        if (key < 64) {
          const int tail = p.tails[sg.b];
          if (key >= (sg.len & 63) || tail < 0 || tail >= p.tail_pages) see = 0u;
        } else {
          see = 0u;
#pragma unroll 1
          for (int q = 0; q < Q; ++q) see |= (uint32_t)((mask_s[qa + q] >> (key - 64)) & 1ull) << q;
        }
        see_s[wg * 128 + key] = (uint16_t)see;
      }
      // the next part's query rows on their way to L2
      const __nv_bfloat16* q_next = nullptr;
      {
        KaIter after = it;
        KaSeg next;
        if (ka_next(p, after, next)) q_next = q_at(next);
      }
      if (q_next && !(st & 1)) asm volatile("prefetch.global.L2 [%0];" ::"l"(q_next));
      uint64_t l[Q / 2];
#pragma unroll
      for (int q = 0; q < Q / 2; ++q) l[q] = 0ull;
      const int half = qd >> 1;
#pragma unroll 1
      for (int i = sg.lo; i < sg.hi; ++i, ++tc) {
        const int buf = tc & 1;
        const bool bf = sg.bf16(i);
        ok = ka_wait(&s_full[buf], (uint32_t)(tc >> 1) & 1u, p.err, ok);
        tc_fence_after();
        // ---- t = s + log2 sv - m, two rows an instruction
        float t[Q];
        const uint32_t sc = trow + (uint32_t)buf * 2u * NP + (uint32_t)qa;
        const float4 blk = scale_s[2 * (tc & 15) + half];  // key scale, log2 value scale, its inverse
        const uint64_t sk2 = ka_2(blk.x, blk.x), lsv2 = ka_2(blk.y, blk.y), c32 = ka_2(0.03125f, 0.03125f);
#pragma unroll
        for (int q0 = 0; q0 < Q; q0 += 8) {
          uint32_t u1[8], u2[8];
          tmem_ld_32x32b<8>(sc + q0, u1);
          tmem_ld_32x32b<8>(sc + NP + q0, u2);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const float4 w = gm[(q0 + q) >> 1];
            const uint64_t x = ka_fma2(ka_2(__uint_as_float(u2[q]), __uint_as_float(u2[q + 1])), c32,
                                       ka_2(__uint_as_float(u1[q]), __uint_as_float(u1[q + 1])));
            ka_un2(ka_fma2(x, ka_mul2(ka_2(w.x, w.y), sk2), ka_add2(ka_2(w.z, w.w), lsv2)), t[q0 + q], t[q0 + q + 1]);
          }
        }
        if (blk.w != 0.0f) {  // no such block
#pragma unroll
          for (int q = 0; q < Q; ++q) t[q] = -INFINITY;
        }
        if (bf) {
          const uint32_t see = see_s[wg * 128 + key];
#pragma unroll
          for (int q = 0; q < Q; ++q)
            if (!((see >> q) & 1u)) t[q] = -INFINITY;
        }
        // ---- is m to be set, or does a weight pass the limit?
        const float limit = bf ? kKaLimit16 : kKaLimit;
        bool raise = i == sg.lo;
        if (!raise) {
          float over = -INFINITY;
#pragma unroll
          for (int q = 0; q < Q; q += 2) over = ka_max3(over, t[q], t[q + 1]);
          raise = ka_bar_any(bar, over > limit);
        }
        if (raise) {
          {
            float x[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) x[q] = t[q];
            const float mx = ka_reduce16<true>(x, lane);
            if (!(lane & 1)) part_s[qd * NP + qa + (lane >> 1)] = mx;
          }
          ka_bar(bar);
          const int r = qa + (lane & 15);  // a lane's row from here on
          const float mx = fmaxf(fmaxf(part_s[r], part_s[NP + r]), fmaxf(part_s[2 * NP + r], part_s[3 * NP + r]));
          float d = 0.0f;
          if (i == sg.lo ? mx > -INFINITY : mx > limit) d = mx - kKaRoom;
          const float f = ka_ex2(-d);
          if (qd == 0 && lane < 16) gm_s[4 * (r >> 1) + 2 + (r & 1)] -= d;
#pragma unroll
          for (int q = 0; q < Q; ++q) t[q] -= __shfl_sync(0xffffffffu, d, q);
          if (i > sg.lo) {
#pragma unroll
            for (int q = 0; q < Q; q += 2)
              l[q / 2] = ka_mul2(l[q / 2], ka_2(__shfl_sync(0xffffffffu, f, q), __shfl_sync(0xffffffffu, f, q + 1)));
            // O^T holds the sums up to tile i - 1
            ok = ka_wait(&pv_done[buf ^ 1], (uint32_t)((tc - 1) >> 1) & 1u, p.err, ok);
            tc_fence_after();
#pragma unroll 1
            for (int q0 = 0; q0 < Q; q0 += 8) {
              uint32_t o[8];
              tmem_ld_32x32b<8>(trow + C::kOCol + (uint32_t)(qa + q0), o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                o[q] = __float_as_uint(__uint_as_float(o[q]) * __shfl_sync(0xffffffffu, f, q0 + q));
              tmem_st_32x32b_x8(trow + C::kOCol + (uint32_t)(qa + q0), o);
            }
            tmem_wait_st();
          }
          ka_bar(bar);  // the new m, and part_s read
        }
        // ---- P (P V (i - 2) has left its buffer)
        uint4* pd = reinterpret_cast<uint4*>(smem + C::kPOff + buf * C::kPBytes + (qa >> 3) * 2048 + key * 16);
        const uint64_t isv2 = ka_2(blk.z, blk.z);
#pragma unroll
        for (int q = 0; q < Q; q += 2) {
          t[q] = ka_ex2(t[q]);
          t[q + 1] = ka_ex2(t[q + 1]);
          l[q / 2] = ka_fma2(ka_2(t[q], t[q + 1]), isv2, l[q / 2]);
        }
        if (bf) {
#pragma unroll
          for (int q = 0; q < Q; q += 8)
            pd[q * 16] = make_uint4(ka_bf162(t[q], t[q + 1]), ka_bf162(t[q + 2], t[q + 3]), ka_bf162(t[q + 4], t[q + 5]),
                                    ka_bf162(t[q + 6], t[q + 7]));
        } else {
#pragma unroll
          for (int q = 0; q < Q; q += 8)
            pd[q * 16] = make_uint4(ka_half2(t[q], t[q + 1]), ka_half2(t[q + 2], t[q + 3]), ka_half2(t[q + 4], t[q + 5]),
                                    ka_half2(t[q + 6], t[q + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // ---- the end of the unit's part: the rows' sums over the keys, then O^T
      q_load(q_next);
      {
        float x[Q];
#pragma unroll
        for (int q = 0; q < Q; q += 2) ka_un2(l[q / 2], x[q], x[q + 1]);
        const float y = ka_reduce16<false>(x, lane);
        if (!(lane & 1)) part_s[qd * NP + qa + (lane >> 1)] = y;
      }
      ka_bar(bar);
      float inv;  // of a lane's row
      const bool whole = sg.lo == 0 && sg.hi == sg.nt;
      // a cut unit's part: a run's first part in its first slot, else the second
      const unsigned slot = 2u * blockIdx.x + (seg == 0 ? 0u : 1u);
      {
        const int r = qa + (lane & 15);
        const float y = (part_s[r] + part_s[NP + r]) + (part_s[2 * NP + r] + part_s[3 * NP + r]);
        inv = 1.0f / y;
        if (!whole && st < Q) wk.part_ml[slot * NP + r] = make_float2(-gm_s[4 * (r >> 1) + 2 + (r & 1)], y);
      }
      ok = ka_wait(&pv_done[(tc - 1) & 1], (uint32_t)((tc - 1) >> 1) & 1u, p.err, ok);
      tc_fence_after();
      const unsigned long long bad = sg.ends() ? bad_s[seg & 3] : 0ull;
      if (bad) ka_add_bad<Q>(p, sg.b, kvh, bad, mask_s + qa, trow + C::kOCol + (uint32_t)qa, key);
      // whole: the rows as bf16 through the warpgroup's chunk of a P buffer (no
      // MMA reads it any more), 256 bytes each, and out 16 bytes a thread
      __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem + C::kPOff + (qa >> 3) * 2048);
#pragma unroll 1
      for (int q0 = 0; q0 < Q; q0 += 8) {
        uint32_t o[8];
        tmem_ld_32x32b<8>(trow + C::kOCol + (uint32_t)(qa + q0), o);
        tmem_wait_ld();
        if (whole) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            stage[(q0 + q) * kKaD + key] =
                __float2bfloat16_rn(__uint_as_float(o[q]) * __shfl_sync(0xffffffffu, inv, q0 + q));
        } else {
          float* dst = wk.part_o + ((size_t)slot * NP + qa + q0) * kKaD + key;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (in_bounds(p.err, (int64_t)slot * NP + qa + q0 + q, (int64_t)2 * wk.by_ctas.d * NP))
              dst[q * kKaD] = __uint_as_float(o[q]);
        }
      }
      if (whole) {
        ka_bar(bar);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int q = (st >> 4) + 8 * k;
          if (row_s[qa + q] >= 0 && in_bounds(p.err, row_s[qa + q], (int64_t)p.B * p.n * p.H))
            reinterpret_cast<uint4*>(p.out + (int64_t)row_s[qa + q] * kKaD)[st & 15] =
                reinterpret_cast<const uint4*>(stage)[q * 16 + (st & 15)];
        }
      }
      if (!whole) {
        // ---- the last of the unit's CTAs is to merge the parts, at its end
        ka_bar_all<C::kGroups>();  // (the counter's release covers what the barrier has gathered)
        if (warp == C::kSoft0 && lane == 0) {
          const KaCut runs = cut_s;
          const unsigned u0 = sg.at - (unsigned)sg.lo;  // the unit's first tile
          unsigned c0 = blockIdx.x, c1 = blockIdx.x;    // the runs of its first and last
#pragma unroll 1
          for (int e = 0; e < 2; ++e)
            if (e ? sg.hi < sg.nt : sg.lo > 0) {
              const unsigned c = runs.owner(e ? u0 + (unsigned)sg.nt - 1u : u0);
              e ? c1 = c : c0 = c;
            }
          const unsigned parts = c1 - c0 + 1u;
          if (atomic_add_acq_rel(&wk.done[c0], 1) == (int)parts - 1) {
            wk.done[c0] = 0;
            // the first part is its run's first only if the run begins with it
            merge_s[seg == 0 ? 0 : 1] = KaMerge{sg.b, sg.u, 2u * c0 + (runs.begin(c0) == u0 ? 0u : 1u), c0, parts};
          }
        }
      }
      tc_fence_before();
      ka_bar(bar);  // the small arrays are free for the next part
      ++seg;
    }
  }

  // ---------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  // no MMA in flight when TMEM is freed
  if ((warp == 1 || warp == 3) && lane == 0 && issued) mbar_wait(&mma_fin[warp >> 1], 0u, p.err);
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k)
    if (merge_s[k].parts > 0u && 4 * warp < NP) ka_merge<NP>(p, wk, merge_s[k], 4 * warp, lane);
}

// ------------------------------------------------------------------ host
struct KaPlan {
  int np, row_blocks, ctas;
  size_t done_bytes, ml_bytes, total;
};
static KaPlan ka_plan(int n, int H, int Hkv, int num_sms) {
  KaPlan k;
  const int rows = n * (H / Hkv);
  // row blocks of at most 64 rows, all of the same size up to a multiple of 16
  k.row_blocks = (rows + 63) / 64;
  k.np = ((rows + k.row_blocks - 1) / k.row_blocks + 15) / 16 * 16;
  k.ctas = num_sms > 0 ? num_sms : 1;
  k.done_bytes = ((size_t)k.ctas * 4 + 255) / 256 * 256;
  k.ml_bytes = (size_t)2 * k.ctas * k.np * 8;
  k.total = k.done_bytes + k.ml_bytes + (size_t)2 * k.ctas * k.np * kKaD * 4;
  return k;
}

size_t kv8_attention_ws(int n, int H, int Hkv, int num_sms) { return ka_plan(n, H, Hkv, num_sms).total; }

// an upper bound of the tiles of all units
bool kv8_attention_fits(int B, int n, int H, int Hkv, int max_len) {
  const int64_t rb = ((int64_t)n * (H / Hkv) + 63) / 64;
  return (double)B * Hkv * rb * ((double)max_len / 128.0 + 2.0) < 2147483648.0;
}

template <int NP, int FMT>
static cudaError_t launch_ka(const KaMaps& maps, const Kv8AttnParams& p, const KaWork& wk, cudaStream_t stream) {
  constexpr int smem = KaCfg<NP>::kTotal;
  const cudaError_t e =
      cudaFuncSetAttribute(kv8_attention_kernel<NP, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_attention_kernel<NP, FMT>, dim3(wk.by_ctas.d), dim3(KaCfg<NP>::kThreads), (size_t)smem,
                    stream, maps, p, wk);
}

cudaError_t launch_kv8_attention(const Kv8AttnParams& p, int fmt, void* workspace, int num_sms, cudaStream_t stream) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!encode) return cudaErrorNotSupported;
  const KaPlan k = ka_plan(p.n, p.H, p.Hkv, num_sms);
  KaMaps maps;
  const cuuint32_t es[4] = {1u, 1u, 1u, 1u};
  auto map = [&](CUtensorMap* m, CUtensorMapDataType t, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box) {
    return encode(m, t, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  bool ok = true;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)kKaD, 64, (cuuint64_t)p.pages * p.Hkv}, st[2] = {kKaD, kKaD * 64};
    const cuuint32_t box[3] = {(cuuint32_t)kKaD, 64u, 1u};
    ok = map(&maps.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.k, dims, st, box) &&
         map(&maps.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.v, dims, st, box);
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)kKaD, 64, (cuuint64_t)p.tail_pages * p.Hkv}, st[2] = {kKaD * 2, kKaD * 128};
    const cuuint32_t box[3] = {64u, 64u, 1u};
    ok = ok && map(&maps.k_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.k_tail, dims, st, box) &&
         map(&maps.v_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.v_tail, dims, st, box);
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)kKaD, (cuuint64_t)p.Hkv, (cuuint64_t)p.n, (cuuint64_t)p.B};
    const cuuint64_t st[3] = {kKaD * 2, (cuuint64_t)p.kv_stride * 2, (cuuint64_t)p.kv_stride * 2 * p.n};
    const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)p.n, 1u};
    ok = ok && map(&maps.k_new, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.k_new, dims, st, box) &&
         map(&maps.v_new, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.v_new, dims, st, box);
  }
  if (!ok) return cudaErrorInvalidValue;
  KaWork wk;
  wk.row_blocks = k.row_blocks;
  wk.np = k.np;
  wk.G = p.H / p.Hkv;
  wk.by_g = fast_div((uint32_t)wk.G);
  wk.by_blocks = fast_div((uint32_t)wk.row_blocks);
  wk.by_units = fast_div((uint32_t)(p.Hkv * wk.row_blocks));
  wk.by_ctas = fast_div((uint32_t)k.ctas);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  wk.done = reinterpret_cast<int*>(ws);
  wk.part_ml = reinterpret_cast<float2*>(ws + k.done_bytes);
  wk.part_o = reinterpret_cast<float*>(ws + k.done_bytes + k.ml_bytes);
  switch (k.np) {
    case 16: return fmt ? launch_ka<16, 1>(maps, p, wk, stream) : launch_ka<16, 0>(maps, p, wk, stream);
    case 32: return fmt ? launch_ka<32, 1>(maps, p, wk, stream) : launch_ka<32, 0>(maps, p, wk, stream);
    case 48: return fmt ? launch_ka<48, 1>(maps, p, wk, stream) : launch_ka<48, 0>(maps, p, wk, stream);
    default: return fmt ? launch_ka<64, 1>(maps, p, wk, stream) : launch_ka<64, 0>(maps, p, wk, stream);
  }
}

}  // namespace w4a16

#if W4A16_TEST_HOOKS
// Debug builds only (not part of the C ABI header): see g_test_skip_tile.
extern "C" int w4a16_test_set_skip_tile(int tile) {
  return (int)cudaMemcpyToSymbol(w4a16::g_test_skip_tile, &tile, sizeof(int));
}
#endif
