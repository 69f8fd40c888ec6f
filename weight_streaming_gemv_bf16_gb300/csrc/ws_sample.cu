// ws_sample.cu -- the next token of each row of logits, drawn from a given
// uniform number: temperature, then the top_k largest, then the smallest set of
// the largest of those that holds top_p of their mass, then those of it that
// are at least min_p times as likely as the most likely one.
//
// Each of the four keeps a prefix of the tokens in falling order (equal logits
// by the lower index), so what is kept is a border: every logit above a value,
// and the first few, by index, that equal it.  Among them the token is the first, in
// the order of indices, whose running sum of weights 2^-t, t = (max - x) log2(e) /
// temperature, passes u times their sum.
//
// Weights are held in fixed point, so that sums do not depend on their order and a
// row's borders and token are the same however it is cut.  A logit x is split at a
// grid of step g, a power of two with g log2(e) / temperature in 2^-6 .. 2^-5: x = h
// + l exactly; the weight is a table's entry for h (a pair of fp32 values, made for the
// row) times e^(l / temperature), a polynomial with its leading terms as pairs.  It is off
// by about 2^-37 of itself and rounded to 2^-41 of the most likely token's: the draw differs
// from one in 64-bit arithmetic only where u lies as near to a border.  What is summed
// are the two words that adding 24 and 1.5 2^-18 to its upper and lower part leaves.
// Where top_k has cut the row to few tokens no table is made: their weights come
// from 2^-t itself (sp_weight, 2^44 for the most likely).
//
// A cluster of up to 16 CTAs takes a row, a contiguous slice each (a short row is one
// small CTA's: k_sample_whole); what a CTA needs again it reads from L2, or where the SMs have
// one CTA each from shared memory, in which the first pass leaves it.  The first pass takes the
// maximum.  Then
//   - top_k up to 5157: a step of the grid that the top_k-th logit lies above almost surely
//     comes from a sample (every 16th piece), or from a count of all; a pass gathers what lies
//     above it and checks their number, and the first CTA finds all borders and the token
//     among them;
//   - a larger top_k: gathered as well, the border found by all CTAs (what the lists, 8800 a CTA,
//     do not hold is read again for each histogram: 400 rows of 151936 bf16, a CTA each, top_k
//     8000 305 us, 16000 1058);
//   - top_p alone: a pass adds up weights of 12 bits by steps of the grid: that names the
//     few steps that hold the border.  The next forms the exact sums of all weights and of
//     those above these steps, and gathers what lies in them, for the first CTA to search;
//   - otherwise: a pass for the exact sum of what is kept.
// A border is found through histograms over the keys of what was gathered, until one value
// is left.  Where the token's place is known by the running sums of the CTAs, and of their
// warps' runs, one CTA reads that run again.  The CTAs of a cluster add up their
// histograms and sums through distributed shared memory.
//
// Bound by instructions where there are many rows, by the chain of passes and barriers
// where there are few.  Device time, us: 256 rows of 151936 bf16 (floor 11.5): the largest 33,
// top_k 50 67, 2500 139, no border 106, top_p 0.9 165 (whole rows: 142, of which the pass for the
// exact sums 47, the coarse one 20), settings of every kind 98; 16 rows of 151936 fp32 (floor
// 1.4): 9, 20, 42, 22, 35, 36; one row of 50257 fp32: 4.5, 14, 30, 14, 24, 26.
// What it took from 203 us (top_p, 256 rows) and from 20 (one
// row): exact weights by 64-bit integer steps for every logit, once for a histogram of them and
// once for the sum, 46 instructions a logit (203 us); by the grid's table 24 (151); the border
// among few, not by rounds over the slice; 2500 of 50257 searched by one CTA and not by all (49).
// Steps as functions of their own that are not inlined: their registers pass through local
// memory, 17 us where 12 now, one row's largest.  Sorting what was gathered: 290 cycles a step
// of a bitonic network, 48000 for 2048.
#include <cfloat>
#include <cmath>
#include <cstddef>
#include <mutex>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpRuns = 4 * kSpWarps;
constexpr int kSpBins = 2048;            // of keys
constexpr int kSpGrid = 2944;            // steps of the grid down to weights of 2^-46; what lies beyond has none
constexpr int kSpSteps = 4096;           // as many bins, in whole ones for each thread
constexpr int kSpTable = 1024;           // entries of 2^(-j / 1024)
constexpr int kSpMaxCluster = 16;
constexpr int kSpMaxV = 1 << 19;
constexpr int kSpFar = 46 * kSpTable;    // steps of 1/1024 in t from which weights are 0
constexpr int kSpCoarse = 12;            // bits of the second pass's weights: 2^19 of them fit 32 bits
constexpr int kSpLimbs = 4, kSpLimb = 12;  // a weight's bits in a histogram: 2^19 of 12 fit 32 bits
constexpr int kSpList = 8800;            // gathered logits a CTA
constexpr int kSpBring = 4096;           // of a row, for the first CTA
constexpr int kSpPack = 5500;            // ... or, with their indices in the lists' place
constexpr int kSpRate = 16;              // pieces for one that the sample takes

struct SampleParams {
  const void* logits;
  long long ld;
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* token;
  float* prob;
  int rows, V, per;  // per: tokens a CTA
  int stays;         // a slice stays in shared memory, behind SpShared
  int ranked;        // rows are taken in the order of what their settings cost
};

__device__ __forceinline__ uint32_t sp_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t sp_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every CTA of the cluster comes here as often as the others: nothing that a
// CTA alone sees decides whether it does.
__device__ __forceinline__ void sp_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// this address in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t sp_at(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void sp_put(uint32_t at, uint64_t a, uint64_t b) {
  asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(at), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ uint32_t sp_get(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

struct alignas(16) SpPair {  // (written to another CTA as 16 bytes)
  uint64_t a, b;
};
struct SpBox {
  SpPair x, y;
};
// fp32 values in the order of unsigned integers, 2^31 for the two zeros; what the low bits of
// 16-bit values lack, their keys lack too
__device__ __forceinline__ uint32_t sp_key(float x) {
  const uint32_t b = __float_as_uint(x), m = b & 0x7fffffffu;
  return b & 0x80000000u ? 0x80000000u - m : b | 0x80000000u;
}
__device__ __forceinline__ float sp_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : 0x80000000u | (0x80000000u - key));
}

// A row's largest logit, and log2(e) / temperature as hi + lo.
struct SpScale {
  float top, ch, cl;
};

// The grid: logits less `ref` (0, or the largest where its size is beyond the grid's: what
// is near it is then exactly apart from it), from `least` on; adding `magic` leaves the step
// in the low bits, `first` for the largest.  1 / temperature as rh + rl.
struct SpGrid {
  float ref, least, magic, rh, rl;
  int first;
};

// (All of this by scalar instructions: two values an instruction took 101 us where one takes
// 93, 256 rows of 151936 with no border; the pairs of registers have to be put together.)
constexpr float kSpMagic = 12288.f;  // 1.5 2^13: a unit in the last place is 2^-10

__device__ __forceinline__ bool sp_near(int k) { return (unsigned)k < (unsigned)kSpFar; }

// 2^44 2^-t of a logit, t in steps of 1/1024 and what is left of it; `more` steps are added.
// With s + e = top - x exactly and ph = s ch rounded, t = ph + pl, pl = (s ch - ph) + s
// cl + e ch.
__device__ __forceinline__ uint64_t sp_weight(const SpScale& c, float x, const uint64_t* pow2, int more = 0) {
  const float s = __fsub_rn(c.top, x), ph = __fmul_rn(s, c.ch), m = __fadd_rn(kSpMagic, ph);
  const int k = __float_as_int(m) - __float_as_int(kSpMagic) + more;
  if (!sp_near(k)) return 0;
  const float v = __fsub_rn(s, c.top);
  const float e = __fsub_rn(__fsub_rn(c.top, __fsub_rn(s, v)), __fadd_rn(x, v));
  float pl = __fmaf_rn(s, c.ch, -ph);
  pl = __fmaf_rn(s, c.cl, pl);
  pl = __fmaf_rn(e, c.ch, pl);
  const float left = __fsub_rn(__fsub_rn(m, kSpMagic), ph);  // the steps less ph, exactly
  const float z = __fmul_rn(__fsub_rn(left, pl), 0.693147180559945f);
  const float q = __fmaf_rn(__fmul_rn(z, z), __fmaf_rn(z, 1.f / 6.f, 0.5f), z);  // e^z - 1, |z| < 2^-11
  constexpr float kUnit = 1.5f * 0x1p-10f;  // a unit in the last place is 2^-33
  const int n = __float_as_int(__fadd_rn(q, kUnit)) - __float_as_int(kUnit);
  const uint64_t p = pow2[k & (kSpTable - 1)];
  const uint64_t w = p + (uint64_t)(((int64_t)(int32_t)(p >> 14) * n) >> 19);
  return (((w << 1) >> (k >> 10)) + 1) >> 1;
}

// 1 / temperature = r + e: the reciprocal and its remainder; times log2(e) as two terms
__device__ __forceinline__ void sp_scale(float top, float temp, SpScale& c, float& r, float& e) {
  constexpr float kLh = 1.44269504f, kLl = 1.92596303e-8f;
  r = __fdiv_rn(1.f, temp);
  e = __fmul_rn(__fmaf_rn(-r, temp, 1.f), r);
  c.top = top;
  c.ch = __fmul_rn(r, kLh);
  c.cl = fmaf(e, kLh, fmaf(r, kLl, __fmaf_rn(r, kLh, -c.ch)));
}
// The least key that min_p keeps: (x - top) / temperature >= ln(min_p), in 64 bits
__device__ __forceinline__ uint32_t sp_floor(float top, float temp, float low) {
  const double x = low >= 1.f ? (double)top : (double)top + (double)temp * log((double)low);
  return sp_key(__double2float_ru(x));
}

// A logit's steps below the largest's, 0 .. kSpGrid (weight 0), and what is left.
__device__ __forceinline__ int sp_cell(const SpGrid& g, float x, float& l) {
  x = fmaxf(__fsub_rn(x, g.ref), g.least);
  const float h = __fadd_rn(x, g.magic);
  l = __fsub_rn(x, __fsub_rn(h, g.magic));
  return g.first - __float_as_int(h);
}
__device__ __forceinline__ int sp_cell(const SpGrid& g, float x) {
  float l;
  return sp_cell(g, x, l);
}

constexpr float kSpUp = 24.f, kSpDown = 1.5f * 0x1p-18f;  // units in the last place: 2^-19, 2^-41
// The words of a weight: kSpUp's and kSpDown's bits and as many units above them.
__device__ __forceinline__ void sp_words(const SpGrid& g, float2 entry, float l, uint32_t& up, uint32_t& down) {
  const float e = entry.x;
  const float z = __fmul_rn(l, g.rh);  // |z| < 2^-6.5
  const float zl = __fmaf_rn(l, g.rl, __fmaf_rn(l, g.rh, -z));
  const float zz = __fmul_rn(z, z), p = __fmaf_rn(__fmaf_rn(z, 1.f / 24.f, 1.f / 6.f), z, 0.5f);
  const float q = __fmaf_rn(zz, p, z);                                        // e^z - 1, rounded
  const float ql = __fadd_rn(__fmaf_rn(zz, p, __fsub_rn(z, q)), zl);          // and what that lost
  const float w = __fmaf_rn(e, q, e);
  const float wl = __fadd_rn(__fmaf_rn(e, ql, __fmaf_rn(e, q, __fsub_rn(e, w))), entry.y);
  const float u = __fadd_rn(w, kSpUp);
  up = __float_as_uint(u);
  down = __float_as_uint(__fadd_rn(__fadd_rn(__fsub_rn(w, __fsub_rn(u, kSpUp)), wl), kSpDown));
}
// A sum of words, of n weights, in units of 2^-41
__device__ __forceinline__ uint64_t sp_units(uint32_t up, uint32_t down, uint32_t n) {
  return ((uint64_t)(up - n * (uint32_t)0x41c00000) << 22) +
         (int64_t)(int32_t)(down - n * (uint32_t)0x36c00000);
}

template <int DT>
constexpr int kSpVec = DT == DT_F32 ? 4 : 8;  // logits in 16 bytes

template <int DT>
__device__ __forceinline__ void sp_unpack(const uint4& u, float (&x)[kSpVec<DT>]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_F32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == DT_BF16) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// 2^(-j / 1024) as 2^44 times it, rounded: products of the square roots of 1/2
struct SpPowers {
  uint64_t at[kSpTable];
  constexpr SpPowers() : at{} {
    // 2^64 2^(-1/2), 2^(-1/4), ..., 2^(-1/1024)
    const uint64_t root[10] = {
        0xb504f333f9de6484ull, 0xd744fccad69d6af4ull, 0xeac0c6e7dd24392eull, 0xf5257d152486cc2cull,
        0xfa83b2db722a033aull, 0xfd3e0c0cf486c174ull, 0xfe9e115c7b8f884aull, 0xff4ecb59511ec8a5ull,
        0xffa756521c8daed1ull, 0xffd3a751c0f7e10bull};
    for (int j = 0; j < kSpTable; ++j) {
      unsigned __int128 p = (unsigned __int128)1 << 64;
      for (int i = 0; i < 10; ++i)
        if (j >> (9 - i) & 1) p = p * root[i] >> 64;
      at[j] = (uint64_t)(((p >> 19) + 1) >> 1);
    }
  }
};
__device__ const SpPowers kSpPowers{};

// What SpFew's threads share.
struct SpFewShared {
  uint64_t sums[32];
  uint64_t before, all;
  uint32_t bin, lo, hi, differ;
};
// What a CTA keeps of its row, and what its threads share.
struct SpShared {
  uint64_t pow2[kSpTable];
  alignas(16) uint32_t hist[kSpLimbs * kSpBins];
  alignas(16) float2 grid[kSpGrid + 1];
  float list[kSpList];            // gathered logits
  uint8_t in_run[kSpList];        // the run that each lies in
  SpBox box[2][kSpMaxCluster];    // what the cluster's CTAs send one another, by turns
  SpPair found[2];                // ... and what one of them found
  uint4 edge[2];                  // the slice's first and last 16 bytes; what they hold of others is ruled out
  uint64_t sums[2][kSpWarps];
  uint64_t above[kSpRuns];
  uint32_t limbs[kSpRuns][kSpLimbs];
  uint32_t ties[kSpRuns];
  uint32_t lo, hi;
  SpFewShared few;
  int listed;                     // logits that were gathered
  // the row
  const char* src;   // the slice's first 16 bytes
  int skew;          // the first logit there
  int pieces, run;   // 16-byte pieces; those of a run, one after another
  uint32_t inverse;  // 2^32 / run, rounded up: the run of a piece below 2^16
  int runs;          // a warp's runs, 1 or 4, behind one another: their sums are kept
  uint32_t rank, size;
  SpScale c;
  SpGrid g;
  int table;         // weights are the grid's
  // The gathered logits: those in steps `from` to `to`.  `held` of them in the list, or
  // (-1: it did not hold them) to be read again.
  int from, to, held;
};

// The steps below are inlined where they are used, but for sp_border, which few rows come to.

// (x, y) summed over the threads before this one and, in `all`, over the CTA.
// Two barriers.
__device__ __forceinline__ SpPair sp_before(SpShared& sh, uint64_t x, uint64_t y, SpPair& all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint64_t s = x, r = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, s, o), v = __shfl_up_sync(0xffffffffu, r, o);
    if (lane >= o) s += u, r += v;
  }
  if (lane == 31) sh.sums[0][w] = s, sh.sums[1][w] = r;
  __syncthreads();
  SpPair before = {0, 0};
  all = before;
#pragma unroll 4
  for (int i = 0; i < kSpWarps; ++i) {
    if (i == w) before = all;
    all.a += sh.sums[0][i], all.b += sh.sums[1][i];
  }
  __syncthreads();
  before.a += s - x, before.b += r - y;
  return before;
}

// What this CTA gives to all: the place of CTA i's is i afterwards.  `turn` alternates.
__device__ __forceinline__ const SpBox* sp_swap(SpShared& sh, uint32_t& turn, uint64_t a, uint64_t b = 0, uint64_t c = 0) {
  SpBox* box = sh.box[turn];
  turn ^= 1;
  if (threadIdx.x < sh.size) {
    sp_put(sp_at(&box[sh.rank].x, threadIdx.x), a, b);
    sp_put(sp_at(&box[sh.rank].y, threadIdx.x), c, 0);
  }
  sp_sync();
  return box;
}

// f x for 0 <= f < 1, rounded down, or up: the product of the 24-bit fraction and x, exactly
__device__ __forceinline__ uint64_t sp_part(float f, uint64_t x, bool up) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (int)(e ? e : 1);  // 24 and more
  const uint64_t hi = __umul64hi(m, x), lo = m * x;
  uint64_t q, left;
  if (shift < 64) q = (hi << (64 - shift)) | (lo >> shift), left = lo << (64 - shift);
  else if (shift < 128) q = hi >> (shift - 64), left = lo | (shift > 64 ? hi << (128 - shift) : 0);
  else q = 0, left = hi | lo;
  return q + (up && left ? 1 : 0);
}

struct SpBorder {
  uint32_t key;
  uint64_t ties;
};
// how many of weight w reach goal
__device__ __forceinline__ uint64_t sp_count(uint64_t goal, uint64_t w) { return w ? (goal + w - 1) / w : ~0ull; }

struct SpRange {
  uint32_t hi;
  int low, bits;
};
struct SpSpot {
  uint32_t at;
  uint64_t left, all;
};
// A few logits that one CTA has in shared memory: what is kept of them, and the token.
// Source: n, key(i), index(i) and weight(key) of the logits.  hist: kSpLimbs * BINS words.
template <int THREADS, int BINS, typename Source>
struct SpFew {
  SpFewShared& sh;
  uint32_t* hist;
  const Source& at;

  // The sum of x over the threads before this one, and over all.  Two barriers.
  __device__ __forceinline__ uint64_t before(uint64_t x, uint64_t& all) const {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) sh.sums[w] = s;
    __syncthreads();
    uint64_t b = 0;
    all = 0;
#pragma unroll 4
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i == w) b = all;
      all += sh.sums[i];
    }
    __syncthreads();
    return b + s - x;
  }

  // The CTA's least lo and largest hi.  Two barriers.
  __device__ __forceinline__ void bounds(uint32_t& lo, uint32_t& hi) const {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (threadIdx.x == 0) sh.lo = 0xffffffffu, sh.hi = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&sh.lo, lo);
      atomicMax(&sh.hi, hi);
    }
    __syncthreads();
    lo = sh.lo, hi = sh.hi;
  }

  // The largest key, the low bits that all have in common, and how many bits the places below the
  // largest, in steps of those, take.
  __device__ __forceinline__ SpRange range() const {
    uint32_t lo = 0xffffffffu, hi = 0, differ = 0;
    const uint32_t one = at.key(0);
    for (int i = threadIdx.x; i < at.n; i += THREADS) {
      const uint32_t y = at.key(i);
      lo = min(lo, y), hi = max(hi, y), differ |= y ^ one;
    }
    differ = __reduce_or_sync(0xffffffffu, differ);
    if (threadIdx.x == 0) sh.differ = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) atomicOr(&sh.differ, differ);
    bounds(lo, hi);
    SpRange r;
    r.hi = hi;
    r.low = max(0, __ffs(sh.differ) - 1);
    r.bits = 32 - __clz((hi - lo) >> r.low);
    return r;
  }

  // Among those that `in` takes, in rising order of place(i) < 2^bits: the place at which their
  // running count, or weight, reaches goal (1 at least; none where it does not), what is left of goal
  // for those there, and their count, or weight.  By histograms of BINS bins, narrower each time.
  template <bool WEIGHT, typename P, typename F>
  __device__ __forceinline__ SpSpot find(uint64_t goal, int bits, P place, F in) const {
    constexpr int kHere = WEIGHT ? kSpLimbs : 1, kLog = BINS == 1024 ? 10 : 8, kEach = BINS / THREADS;
    static_assert(BINS == 1 << kLog && BINS % THREADS == 0, "whole bins a thread");
    uint32_t from = 0, wide = 0xffffffffu;
    int shift = max(0, bits - kLog);
#pragma unroll 1
    for (;;) {
#pragma unroll
      for (int i = 0; i < kHere * kEach; ++i) hist[THREADS * i + threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < at.n; i += THREADS) {
        const uint32_t x = place(i) - from;
        if (x > wide || !in(i)) continue;
        uint32_t* h = &hist[x >> shift];
        if constexpr (WEIGHT) {
          const uint64_t w = at.weight(at.key(i));
#pragma unroll
          for (int l = 0; l < kSpLimbs; ++l)
            atomicAdd(h + l * BINS, (uint32_t)(w >> (kSpLimb * l)) & ((1u << kSpLimb) - 1));
        } else {
          atomicAdd(h, 1u);
        }
      }
      __syncthreads();
      uint64_t v[kEach], s = 0, all;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        v[i] = 0;
#pragma unroll
        for (int l = 0; l < kHere; ++l) v[i] += (uint64_t)hist[l * BINS + kEach * threadIdx.x + i] << (kSpLimb * l);
        s += v[i];
      }
      uint64_t sum = before(s, all);
      if (goal > all) return {0xffffffffu, 0, 0};
      if (sum < goal && goal <= sum + s) {
        int b = 0;
#pragma unroll
        for (int i = 0; i + 1 < kEach; ++i)
          if (i == b && sum + v[i] < goal) sum += v[i], ++b;
        sh.bin = kEach * threadIdx.x + b;
        sh.before = sum;
        sh.all = v[0];
#pragma unroll
        for (int i = 1; i < kEach; ++i)
          if (i == b) sh.all = v[i];
      }
      __syncthreads();
      goal -= sh.before;
      from += sh.bin << shift;
      if (shift == 0) return {from, goal, sh.all};
      wide = (1u << shift) - 1;
      shift = max(0, shift - kLog);
      // where a pass is short, what the bin holds is worth one: mostly a single value (one row
      // of 50257, top_k 50, top_p 0.9: 17.4 us, 19.4 without; 1216 of 1000 the same)
      if (at.n > 2 * THREADS) continue;
      const uint64_t there = sh.all;
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int i = threadIdx.x; i < at.n; i += THREADS) {
        const uint32_t x = place(i);
        if (x - from <= wide && in(i)) lo = min(lo, x), hi = max(hi, x);
      }
      bounds(lo, hi);
      if (lo == hi) return {lo, goal, there};
      from = lo;
      wide = hi - lo;
      shift = max(0, 32 - __clz(wide) - kLog);
    }
  }

  // The sum of the weights that `in` takes.
  template <typename F>
  __device__ __forceinline__ uint64_t mass(F in) const {
    uint64_t w = 0, all;
    for (int i = threadIdx.x; i < at.n; i += THREADS)
      if (in(i)) w += at.weight(at.key(i));
    before(w, all);
    return all;
  }

  // The row's token, where all that top_k keeps is here (k of them, or all).  What is kept:
  // those at places before `b`, and of those there the first b.left (of b.all).
  __device__ __forceinline__ void settle(int k, float p, uint32_t floor_key, float u, int V, int* token,
                                         float* prob) const {
    const SpRange r = range();
    auto place = [&](int i) { return (r.hi - at.key(i)) >> r.low; };
    auto index = [&](int i) { return at.index(i); };
    auto key_at = [&](uint32_t d) { return r.hi - (d << r.low); };
    SpSpot b = {0xffffffffu, 0, 0};  // all of them
    if (k < at.n) b = find<false>(k, r.bits, place, [](int) { return true; });
    auto above = [&](int i) { return place(i) < b.at; };
    uint64_t sum = mass(above), one = b.left ? at.weight(key_at(b.at)) : 0;
    if (p < 1.f) {
      const uint64_t goal = max((uint64_t)1, sp_part(fmaxf(p, 0.f), sum + b.left * one, true));
      if (goal <= sum) {
        b = find<true>(goal, r.bits, place, above);
        one = at.weight(key_at(b.at));  // (above 0: the sum rises there)
        sum = goal - b.left;
        b.left = sp_count(b.left, one);
        b.all /= one;
      } else if (one) {
        b.left = min(b.left, sp_count(goal - sum, one));
      }
    }
    if (floor_key > (b.at == 0xffffffffu ? 0u : key_at(b.at))) {
      b = {((r.hi - floor_key) >> r.low) + 1, 0, 0};
      sum = mass(above);
    }
    uint32_t last = 0xffffffffu;  // of those at b.at, the index of the last that is kept
    const int bits = 32 - __clz(V - 1);
    if (b.left < b.all) last = find<false>(b.left, bits, index, [&](int i) { return place(i) == b.at; }).at;
    sum += b.left * one;
    const uint64_t want = u >= 1.f ? sum - 1 : sp_part(fmaxf(u, 0.f), sum, false);
    const SpSpot e = find<true>(want + 1, bits, index, [&](int i) {
      const uint32_t d = place(i);
      return d < b.at || (b.left && d == b.at && at.index(i) <= last);
    });
    if (threadIdx.x == 0) {
      *token = (int)e.at;
      if (prob) *prob = (float)((double)e.all / (double)sum);
    }
  }
};

// (the first CTA's are what the others add theirs to: none does before all are clear)
__device__ __forceinline__ void sp_clear(SpShared& sh, int words) {
#pragma unroll 1
  for (int i = threadIdx.x; i < words; i += kSpThreads) sh.hist[i] = 0;
  sp_sync();
}

// What the first CTA's histograms of BINS bins hold in the EACH bins from b on.  Counts (1 limb),
// weights (kSpLimbs), or (0) weights of kSpCoarse bits relative to the grid's, brought to
// units of 2^-42.  Returns their sum.
template <int BINS, int EACH>
__device__ __forceinline__ uint64_t sp_bins(const SpShared& sh, int limbs, int b, uint64_t (&v)[EACH]) {
  static_assert(EACH % 4 == 0 && kSpGrid % EACH == 0, "16 bytes a read; all of a thread's in the grid or none");
  uint64_t s = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) v[i] = 0;
  if (BINS == kSpSteps && b >= kSpGrid) return 0;
#pragma unroll
  for (int i = 0; i < EACH; i += 4) {
    const uint4 h = *reinterpret_cast<const uint4*>(sh.hist + b + i);
    v[i] = h.x, v[i + 1] = h.y, v[i + 2] = h.z, v[i + 3] = h.w;
  }
  if (BINS == kSpBins && limbs == kSpLimbs) {
#pragma unroll
    for (int l = 1; l < kSpLimbs; ++l)
#pragma unroll
      for (int i = 0; i < EACH; ++i) v[i] += (uint64_t)sh.hist[l * kSpBins + b + i] << (kSpLimb * l);
  }
  if (BINS == kSpSteps && limbs == 0) {  // times a 24-bit fraction and a power of two
#pragma unroll
    for (int i = 0; i < EACH; i += 2) {
      const float4 w = *reinterpret_cast<const float4*>(sh.grid + b + i);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x = __float_as_uint(j ? w.z : w.x), m = (x & 0x7fffffu) | 0x800000u;
        const int shift = 127 - (int)(x >> 23) - 7;  // 1 is 2^23, and has to be 2^30
        const uint64_t y = v[i + j] * m;
        v[i + j] = x < 0x800000u || shift > 63 ? 0 : shift >= 0 ? y >> shift : y << -shift;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) s += v[i];
  return s;
}

// The bins in which the cluster's running sum reaches `goal`, or with p >= 0 comes within
// 2^-11 of p times all and leaves that; BINS where it does not.  `before`: the sum before
// the first.  Ends with the histograms free again.
struct SpFound {
  int bin[2];
  uint64_t before;
};
template <int BINS>
__device__ __forceinline__ SpFound sp_find(SpShared& sh, int limbs, uint64_t goal, float p) {
  __syncthreads();
  if (sh.rank != 0) {  // to the first CTA's
    const uint32_t to = sp_at(sh.hist, 0);
    const int words = limbs > 1 ? limbs * BINS : BINS;
#pragma unroll 4
    for (int i = threadIdx.x; i < words; i += kSpThreads) {
      const uint32_t n = sh.hist[i];
      if (n) asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(to + 4 * i), "r"(n) : "memory");
    }
  }
  sp_sync();
  if (sh.rank == 0) {
    constexpr int kEach = BINS / kSpThreads;
    const int b0 = threadIdx.x * kEach;
    uint64_t v[kEach];
    const uint64_t s = sp_bins<BINS>(sh, limbs, b0, v);
    SpPair cta;
    const uint64_t start = sp_before(sh, s, 0, cta).a;
    uint64_t last = goal;
    if (p >= 0.f) {
      const uint64_t g = sp_part(p, cta.a, true), off = (g >> 11) + kSpGrid;
      goal = g > off ? g - off : 1;
      last = g + off;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t g = i ? last : goal;
      uint64_t at = start;
      int b = b0;
      if (start < g && g <= start + s) {  // in this thread's bins
#pragma unroll
        for (int j = 0; j + 1 < kEach; ++j)
          if (b == b0 + j && at + v[j] < g) at += v[j], ++b;
      } else if (threadIdx.x == 0 && g > cta.a) {
        b = BINS;
      } else {
        continue;
      }
      for (uint32_t r = 0; r < sh.size; ++r) sp_put(sp_at(&sh.found[i], r), b, at);
    }
  }
  sp_sync();
  SpFound f;
  f.bin[0] = (int)sh.found[0].a;
  f.bin[1] = (int)sh.found[1].a;
  f.before = sh.found[0].b;
  return f;
}

__device__ __forceinline__ uint64_t sp_weight_of(const SpShared& sh, float x) {
  if (!sh.table) return sp_weight(sh.c, x, sh.pow2);
  float l;
  uint32_t up, down;
  const int k = sp_cell(sh.g, x, l);
  sp_words(sh.g, sh.grid[k], l, up, down);
  return sp_units(up, down, 1);
}

// The grid's weights, for a row that needs them of many logits.
__device__ __forceinline__ void sp_table(SpShared& sh) {
  SpScale d = sh.c;
  d.top = sh.c.top - sh.g.ref;
  // (as far as the weights go: 46 / (g log2(e) / temperature) steps)
  const int n = min(kSpGrid, (int)(46.f / (d.ch * __uint_as_float((__float_as_uint(sh.g.magic) & 0x7f800000u) - (23u << 23)))) + 2);
#pragma unroll 2
  for (int i = threadIdx.x; i <= kSpGrid; i += kSpThreads) {
    float2 e = make_float2(0.f, 0.f);
    if (i < n && i < kSpGrid) {
      // half the weight, since the step that holds the largest may lie above it
      const uint64_t w = sp_weight(d, __int_as_float(sh.g.first - i) - sh.g.magic, sh.pow2, kSpTable);
      const float hi = __ull2float_rn(w);
      e = make_float2(hi * 0x1p-43f, (float)((int64_t)w - (int64_t)__float2ull_rn(hi)) * 0x1p-43f);
    }
    sh.grid[i] = e;
  }
  if (threadIdx.x == 0) sh.table = 1;
  __syncthreads();
}

// f(piece, v): the pieces from v0 + lane to v1, AHEAD loads of a lane in flight
template <int AHEAD, typename F>
__device__ __forceinline__ void sp_scan(const SpShared& sh, int v0, int v1, F f) {
  const uint4* src = reinterpret_cast<const uint4*>(sh.src);
  const int last = sh.pieces - 1;
  v1 = min(v1, last + 1);
#pragma unroll 1
  for (v0 += threadIdx.x & 31; v0 < v1; v0 += 32 * AHEAD) {
    uint4 u[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int v = v0 + 32 * i;
      const uint4* p = v == 0 ? &sh.edge[0] : v == last ? &sh.edge[1] : src + v;
      if (v < v1) u[i] = *p;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (v0 + 32 * i < v1) f(u[i], v0 + 32 * i);
  }
}
// f(v0, v1) of each run: its sums over the lanes to sh.above
template <typename F>
__device__ __forceinline__ void sp_runs(SpShared& sh, F f) {
  const int w = threadIdx.x >> 5;
#pragma unroll 1
  for (int i = 0; i < sh.runs; ++i) {
    const int r = w * sh.runs + i;
    uint64_t x = f(r * sh.run, (r + 1) * sh.run);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) sh.above[r] = x;
  }
  __syncwarp();
}
__device__ __forceinline__ int sp_run(const SpShared& sh, int v) { return (int)__umulhi((uint32_t)v, sh.inverse); }
// a warp's share of the slice: its runs
__device__ __forceinline__ int sp_mine(const SpShared& sh) { return sh.run * sh.runs; }
template <int AHEAD, typename F>
__device__ __forceinline__ void sp_scan(const SpShared& sh, F f) {
  const int n = sp_mine(sh), w = threadIdx.x >> 5;
  sp_scan<AHEAD>(sh, w * n, (w + 1) * n, f);
}

// The largest of a piece; a NaN among them is the result.
template <int DT>
__device__ __forceinline__ float sp_largest(const uint4& u) {
  if constexpr (DT == DT_F32) {
    return max_nan(max3_nan(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)), __uint_as_float(u.w));
  } else {
    uint32_t m = u.x;
    const uint32_t w[3] = {u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if constexpr (DT == DT_F16) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    if constexpr (DT == DT_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
      return max_nan(f.x, f.y);
    } else {
      return max_nan(bf16lo(m), bf16hi(m));
    }
  }
}

template <int DT>
__device__ __forceinline__ float sp_pick(const uint4& u, int j) {  // logit j of a piece
  const int w = DT == DT_F32 ? j : j >> 1;
  const uint32_t y = w < 2 ? (w ? u.y : u.x) : (w == 2 ? u.z : u.w);
  if constexpr (DT == DT_F32) return __uint_as_float(y);
  if constexpr (DT == DT_BF16) return j & 1 ? bf16hi(y) : bf16lo(y);
  return __half2float(__ushort_as_half((unsigned short)(j & 1 ? y >> 16 : y)));
}

template <int DT>
__device__ __forceinline__ float sp_one(const SpShared& sh, int i) {  // logit i of the slice's pieces
  constexpr int kVec = kSpVec<DT>;
  const int v = i / kVec;
  const uint4* p = v == 0 ? &sh.edge[0] : v == sh.pieces - 1 ? &sh.edge[1]
                                                               : reinterpret_cast<const uint4*>(sh.src) + v;
  if constexpr (DT == DT_F32) return reinterpret_cast<const float*>(p)[i % kVec];
  const uint16_t h = reinterpret_cast<const uint16_t*>(p)[i % kVec];
  return DT == DT_F16 ? __half2float(__ushort_as_half(h)) : bf16lo(h);
}

// f(x, its run): every gathered logit, one at a time
template <int DT, typename F>
__device__ __forceinline__ void sp_each(const SpShared& sh, F f) {
  constexpr int kVec = kSpVec<DT>;
  const int held = sh.held;
  if (held >= 0) {
#pragma unroll 1
    for (int i = threadIdx.x; i < held; i += kSpThreads) f(sh.list[i], (int)sh.in_run[i]);
    return;
  }
  const int from = sh.from, to = sh.to;
  sp_scan<1>(sh, [&](const uint4& u, int v) {
    const int run = sp_run(sh, v);
#pragma unroll 1
    for (int j = 0; j < kVec; ++j) {
      const float x = sp_pick<DT>(u, j);
      const int k = sp_cell(sh.g, x);
      if (k >= from && k <= to) f(x, run);
    }
  });
}

__device__ __forceinline__ void sp_gather(SpShared& sh, float x, int run) {
  const int i = atomicAdd(&sh.listed, 1);
  if (i < kSpList) {
    sh.list[i] = x;
    sh.in_run[i] = (uint8_t)run;
  }
}

// Gather the steps up to `to`.  PACK: as key << 32 | index of the row, in place of the lists.
__device__ __forceinline__ uint64_t* sp_packed(SpShared& sh) { return reinterpret_cast<uint64_t*>(sh.list); }
static_assert(offsetof(SpShared, list) % 8 == 0 && offsetof(SpShared, in_run) + sizeof(SpShared::in_run) ==
                                                       offsetof(SpShared, list) + 8 * kSpPack, "their place");
template <int DT>
__device__ __forceinline__ void sp_gather_top(SpShared& sh, int to, bool pack, int i0) {
  constexpr int kVec = kSpVec<DT>;
  const SpGrid g = sh.g;
  // the least value that may lie in them, by a whole step less
  const float least = __fadd_rn(__int_as_float(g.first - (to + 1)) - g.magic, g.ref);
  sp_scan<4>(sh, [&](const uint4& u, int v) {
    if (!(sp_largest<DT>(u) >= least)) return;
    float x[kVec];
    sp_unpack<DT>(u, x);
    uint32_t in = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (x[j] >= least) in |= 1u << j;
#pragma unroll 1
    for (; in; in &= in - 1) {
      const int j = __ffs(in) - 1;
      const float y = sp_pick<DT>(u, j);
      if (sp_cell(g, y) > to) continue;
      if (pack) {
        const int i = atomicAdd(&sh.listed, 1);
        if (i < kSpPack) sp_packed(sh)[i] = (uint64_t)sp_key(y) << 32 | (uint32_t)(i0 + v * kVec + j - sh.skew);
      } else {
        sp_gather(sh, y, sp_run(sh, v));
      }
    }
  });
}

// After a pass that gathered the steps from .. to: how many the row has of them, and
// whether the lists hold them (the same for every CTA); the cluster's sums of a and b.
struct SpGathered {
  uint64_t n;
  SpPair sum;
};
__device__ __forceinline__ SpGathered sp_gathered(SpShared& sh, uint32_t& turn, int from, int to, uint64_t a, uint64_t b,
                                                  int most = kSpList) {
  SpPair cta;
  sp_before(sh, a, b, cta);
  const int n = sh.listed;
  const SpBox* box = sp_swap(sh, turn, cta.a, cta.b, n);
  SpGathered g = {0, {0, 0}};
  bool over = false;
#pragma unroll 4
  for (uint32_t r = 0; r < sh.size; ++r) {
    g.sum.a += box[r].x.a, g.sum.b += box[r].x.b;
    g.n += box[r].y.a;
    over |= box[r].y.a > (uint64_t)most;
  }
  if (threadIdx.x == 0) sh.from = from, sh.to = to, sh.held = over ? -1 : n;
  __syncthreads();
  return g;
}

// The lists of all CTAs to the first one's histograms' place: the logits, or the packed ones (to
// the grid's place as well).  What sp_gathered gave is at most kSpBring, or kSpPack.  Ends with
// the first CTA alone going on (true).
template <bool PACK>
__device__ __forceinline__ bool sp_bring(SpShared& sh, uint32_t turn) {
  const SpBox* box = sh.box[turn ^ 1];  // the counts, swapped last
  uint32_t at = 0;
#pragma unroll 1
  for (uint32_t r = 0; r < sh.rank; ++r) at += (uint32_t)box[r].y.a;
  const uint32_t base = sp_at(sh.hist, 0);
  for (int i = threadIdx.x; i < sh.held; i += kSpThreads) {
    if constexpr (PACK)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(base + 8 * (at + i)), "l"(sp_packed(sh)[i]) : "memory");
    else
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(base + 4 * (at + i)), "f"(sh.list[i]) : "memory");
  }
  sp_sync();
  return sh.rank == 0;
}

// Gathered logits, as the first CTA searches them: packed ones, or the values.
struct SpPacked {
  const SpShared& sh;
  const uint64_t* at;
  int n;
  __device__ __forceinline__ uint32_t key(int i) const { return (uint32_t)(at[i] >> 32); }
  __device__ __forceinline__ uint32_t index(int i) const { return (uint32_t)at[i]; }
  __device__ __forceinline__ uint64_t weight(uint32_t key) const { return sp_weight_of(sh, sp_value(key)); }
};
struct SpValues {
  const SpShared& sh;
  const float* at;
  int n;
  __device__ __forceinline__ uint32_t key(int i) const { return sp_key(at[i]); }
  __device__ __forceinline__ uint64_t weight(uint32_t key) const { return sp_weight_of(sh, sp_value(key)); }
};
constexpr int kSpFewBins = 1024;
static_assert(kSpBring + kSpLimbs * kSpFewBins <= kSpLimbs * kSpBins, "the histograms lie behind them");
static_assert(sizeof(SpShared::hist) + sizeof(SpShared::grid) >= 8 * kSpPack &&
                  offsetof(SpShared, grid) == offsetof(SpShared, hist) + sizeof(SpShared::hist) &&
                  offsetof(SpShared, hist) % 8 == 0, "packed ones");

// The cluster's sum of every thread's a.
__device__ __forceinline__ uint64_t sp_sum(SpShared& sh, uint32_t& turn, uint64_t a) {
  SpPair cta;
  sp_before(sh, a, 0, cta);
  const SpBox* box = sp_swap(sh, turn, cta.a);
  uint64_t s = 0;
#pragma unroll 4
  for (uint32_t r = 0; r < sh.size; ++r) s += box[r].x.a;
  return s;
}

// The border among the gathered logits whose key is at least `lo`: the key in which their
// running count, or weight, in falling order reaches goal (1 at least, their sum at
// most), and how many of that key belong to it.
template <int DT>
__device__ __noinline__ SpBorder sp_border(SpShared& sh, uint32_t& turn, bool weights, uint32_t lo, uint64_t goal) {
  uint32_t hi = 0xffffffffu;
#pragma unroll 1
  for (;;) {
    // the smallest key and the largest
    uint32_t a = 0xffffffffu, b = 0;
    sp_each<DT>(sh, [&](float x, int) {
      const uint32_t y = sp_key(x);
      if (y >= lo && y <= hi) a = min(a, y), b = max(b, y);
    });
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    if (threadIdx.x == 0) sh.lo = 0xffffffffu, sh.hi = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&sh.lo, a);
      atomicMax(&sh.hi, b);
    }
    __syncthreads();
    const SpBox* box = sp_swap(sh, turn, sh.lo, sh.hi);
    lo = 0xffffffffu, hi = 0;
#pragma unroll 1
    for (uint32_t r = 0; r < sh.size; ++r) {
      lo = min(lo, (uint32_t)box[r].x.a);
      hi = max(hi, (uint32_t)box[r].x.b);
    }
    if (lo >= hi) break;
    const int shift = max(0, 32 - __clz(hi - lo) - 11), limbs = weights ? kSpLimbs : 1;
    sp_clear(sh, limbs * kSpBins);
    sp_each<DT>(sh, [&](float x, int) {
      const uint32_t y = sp_key(x);
      if (y < lo || y > hi) return;
      uint32_t* h = &sh.hist[(hi - y) >> shift];
      if (weights) {
        const uint64_t w = sp_weight_of(sh, x);
#pragma unroll
        for (int l = 0; l < kSpLimbs; ++l)
          atomicAdd(h + l * kSpBins, (uint32_t)(w >> (kSpLimb * l)) & ((1u << kSpLimb) - 1));
      } else {
        atomicAdd(h, 1u);
      }
    });
    const SpFound f = sp_find<kSpBins>(sh, limbs, goal, -1.f);
    if (f.bin[0] == kSpBins) break;  // (goal is their sum at most)
    goal -= f.before;
    hi -= (uint32_t)f.bin[0] << shift;
    const uint32_t wide = (1u << shift) - 1;
    lo = wide <= hi - lo ? hi - wide : lo;
  }
  SpBorder r = {hi, goal};
  if (weights) {
    r.ties = sp_count(goal, sp_weight_of(sh, sp_value(hi)));
  }
  return r;
}

// The order in which rows are taken where they do not all lie on the SMs at once: the costly ones
// first.  The row in place i of it, by counts of the classes in the 1024 rows around it.
// Both sides, us: 1024 rows of 32000 bf16, settings of every kind 125, 150 in the rows' own
// order, 437 of 8192 51 and 66; with the same settings for all rows the counts cost 1.4 a
// wave (top_p 0.9 174 and 169, the largest 41 and 36).  Where all rows are resident it gains
// nothing (256 of 151936 152 and 151): which of them share an SM is not theirs to say.
__device__ __forceinline__ int sp_class(const SampleParams& a, int row) {
  const float temp = a.temperature ? a.temperature[row] : 1.f, p = a.top_p ? a.top_p[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (!(temp > 0.f) || k == 1) return 3;
  if (k > 1 && k < a.V) return k > 1500 ? 0 : k > 300 ? 1 : 2;
  return p < 1.f ? 0 : 1;
}
__device__ __forceinline__ int sp_ranked(SpShared& sh, const SampleParams& a, int i) {
  constexpr int kHalves = 2, kWindow = kHalves * kSpThreads;
  static_assert(kHalves * kSpWarps == 32 && sizeof(sh.limbs) >= 4 * 32 * 4, "four classes' counts, a lane each");
  const int t = threadIdx.x, lane = t & 31, base = i / kWindow * kWindow;
  uint32_t* count = &sh.limbs[0][0];  // [class][half][warp]
  int kind[kHalves];
  uint32_t before[kHalves];
#pragma unroll
  for (int j = 0; j < kHalves; ++j) {
    const int r = base + j * kSpThreads + t;
    kind[j] = r < a.rows ? sp_class(a, r) : 4;
    before[j] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t all = __ballot_sync(0xffffffffu, kind[j] == q);
      if (kind[j] == q) before[j] = __popc(all & ((1u << lane) - 1));
      if (lane == 0) count[32 * q + j * kSpWarps + (t >> 5)] = __popc(all);
    }
  }
  __syncthreads();
  if (t < 32) {
    uint32_t v[4], s = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = count[4 * lane + q], s += v[q];
    const uint32_t mine = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    s -= mine;
#pragma unroll
    for (int q = 0; q < 4; ++q) count[4 * lane + q] = s, s += v[q];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kHalves; ++j)
    if (kind[j] < 4 && count[32 * kind[j] + j * kSpWarps + (t >> 5)] + before[j] == (uint32_t)(i - base))
      sh.ties[0] = base + j * kSpThreads + t;
  __syncthreads();
  return (int)sh.ties[0];
}

template <int DT>
__global__ void __launch_bounds__(kSpThreads, 2) k_sample_tokens(const __grid_constant__ SampleParams a) {
  constexpr int kVec = kSpVec<DT>, kSize = 16 / kVec;
  extern __shared__ __align__(16) unsigned char smem[];
  SpShared& sh = *reinterpret_cast<SpShared*>(smem);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t rank = sp_rank(), size = sp_size();
  uint32_t turn = 0;
#pragma unroll
  for (int i = 0; i < kSpSteps / kSpThreads; ++i) sh.hist[i * kSpThreads + t] = 0;
  // (waited for before the first write to another CTA: all have begun by then, and the
  // first one's histograms are clear)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
#pragma unroll
  for (int j = t; j < kSpTable; j += kSpThreads) sh.pow2[j] = kSpPowers.at[j];
  pdl_launch_dependents();
  pdl_wait();
  const int row = a.ranked ? sp_ranked(sh, a, blockIdx.x / size) : blockIdx.x / size;
  const int i0 = min((int)rank * a.per, a.V), n = min(a.per, a.V - i0);
  const char* src = static_cast<const char*>(a.logits) + ((long long)row * a.ld + i0) * kSize;
  const int skew = (int)((uintptr_t)src & 15) / kSize, pieces = n > 0 ? (skew + n + kVec - 1) / kVec : 0;
  if (t == 0) {
    sh.src = src - skew * kSize;
    sh.skew = skew;
    sh.pieces = pieces;
    sh.runs = pieces >= 128 * kSpRuns ? kSpRuns / kSpWarps : 1;
    sh.run = max(2, (pieces + kSpWarps * sh.runs - 1) / (kSpWarps * sh.runs));
    sh.inverse = 0xffffffffu / (uint32_t)sh.run + 1;
    sh.rank = rank;
    sh.size = size;
    sh.listed = sh.table = sh.from = sh.to = sh.held = 0;
    sh.lo = 0xffffffffu;
  }
  float temp = a.temperature ? a.temperature[row] : 1.f;
  const float p = a.top_p ? a.top_p[row] : 1.f, low = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
  int k = a.top_k ? a.top_k[row] : 0;
  if (t < 2 * kVec && pieces > 0) {
    const int e = (t < kVec ? 0 : pieces - 1) * kVec + t % kVec - skew;
    const bool mine = e >= 0 && e < n;
    if constexpr (DT == DT_F32)
      reinterpret_cast<uint32_t*>(sh.edge)[t] = mine ? reinterpret_cast<const uint32_t*>(src)[e] : 0xff800000u;
    else
      reinterpret_cast<uint16_t*>(sh.edge)[t] =
          mine ? reinterpret_cast<const uint16_t*>(src)[e] : DT == DT_F16 ? (uint16_t)0xfc00 : (uint16_t)0xff80;
  }
  __syncthreads();

  float top = -INFINITY;
  uint4* stay = reinterpret_cast<uint4*>(smem + sizeof(SpShared));
  sp_scan<4>(sh, [&](const uint4& u, int v) {
    top = max_nan(top, sp_largest<DT>(u));
    if (a.stays) stay[v] = u;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.ties[warp] = __float_as_uint(top);
  __syncthreads();
  if (a.stays && t == 0) sh.src = reinterpret_cast<const char*>(stay);  // (a barrier of the cluster follows)
#pragma unroll 1
  for (int w = 0; w < kSpWarps; ++w) top = max_nan(top, __uint_as_float(sh.ties[w]));
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  {
    const SpBox* box = sp_swap(sh, turn, __float_as_uint(top));
#pragma unroll 4
    for (uint32_t r = 0; r < size; ++r) top = max_nan(top, __uint_as_float((uint32_t)box[r].x.a));
  }

  // no distribution (a NaN, +infinity, nothing but -infinity), or a NaN among the settings
  if (!(fabsf(top) <= FLT_MAX) || temp != temp || p != p || low != low || u != u) {
    if (rank == 0 && t == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = __uint_as_float(0x7fc00000u);
    }
    sp_sync();  // no CTA ends while another may still write to it
    return;
  }
  if (!(temp > 0.f)) temp = 1.f, k = 1;
  temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
  SpGrid g;
  {
    SpScale c;
    float r, e;
    sp_scale(top, temp, c, r, e);
    g.rh = r;
    g.rl = e;
    const uint32_t step = 127 - 6 + 127 - (__float_as_uint(c.ch) >> 23);  // its exponent's bits
    const float unit = __uint_as_float(step << 23);
    g.magic = 1.5f * 8388608.f * unit;
    g.ref = fabsf(top) < 2097152.f * unit ? 0.f : top;
    const float h = __fadd_rn(__fsub_rn(top, g.ref), g.magic);
    g.first = __float_as_int(h);
    g.least = __fsub_rn(__fsub_rn(h, g.magic), kSpGrid * unit);
    if (t == 0) {
      sh.c = c;
      sh.g = g;
      if (low > 0.f) sh.ties[0] = sp_floor(top, temp, low);
    }
  }
  __syncthreads();
  const uint32_t floor_key = low > 0.f ? sh.ties[0] : 0u;

  // What is kept: every key above `key`, and the first `ties` that equal it.  The
  // weights above are those of the steps below sh.from (`above`: this thread's of its
  // warp's run), and what is gathered.
  uint32_t key = 0;
  uint64_t ties = 0, above = 0;
  bool listed = false;  // the border lies among the gathered logits
  bool made = false;    // the grid's table
  bool summed = false;  // sh.above holds the runs' sums
  bool clean = true;    // the histograms are clear
  if (k == 1) {  // the largest alone, the first of its equals
    uint32_t first = 0xffffffffu;
    sp_scan<4>(sh, [&](const uint4& u, int v) {
      if (sp_largest<DT>(u) != top) return;
#pragma unroll 1
      for (int j = 0; j < kVec; ++j)
        if (sp_pick<DT>(u, j) == top) first = min(first, (uint32_t)(i0 + v * kVec + j - skew));
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&sh.lo, first);
    __syncthreads();
    const SpBox* box = sp_swap(sh, turn, sh.lo);
    for (uint32_t r = 0; r < size; ++r) first = min(first, (uint32_t)box[r].x.a);
    if (rank == 0 && t == 0) {
      a.token[row] = (int)first;
      if (a.prob) a.prob[row] = 1.f;
    }
    return;  // (nothing is written to this CTA any more)
  } else if (k > 1 && k < a.V) {
    // The steps to gather: those that the sample says, or (where that was too few, or
    // top_k is large) those that a count of all says.
    int to = kSpGrid - 1;
    uint64_t n = 0;
    bool enough = true;
    // few: the first CTA finishes the row
    bool pack = k <= kSpPack - kSpPack / 16;
    auto gather = [&]() {
      sp_gather_top<DT>(sh, to, pack, i0);
      n = sp_gathered(sh, turn, 0, to, 0, 0, pack ? kSpPack : kSpList).n;
    };
    auto drop = [&]() {
      __syncthreads();
      if (t == 0) sh.listed = 0;
      __syncthreads();
    };
    // of a sample: as many as k of the row leave but once in some thousand rows
    const float part = (float)k / (float)kSpRate;
    const int likely = (int)(part + 4.f * sqrtf(part) + 4.f);
    const int room = pack ? kSpPack / 5 * 4 : kSpList / 5 * 4 * (int)size;
    for (int rate = a.per >= 4096 && likely * kSpRate <= room ? kSpRate : 1;; rate = 1) {
      if (!clean) sp_clear(sh, kSpSteps);
      clean = false;
      const int stride = rate == 1 ? 1 : kSpRate;
#pragma unroll 1
      for (int i = t; i * stride < pieces; i += kSpThreads) {
        const int v = min(i * stride + (stride > 1 ? (i * 7) & (kSpRate - 1) : 0), pieces - 1);
        const uint4* q = v == 0 ? &sh.edge[0] : v == pieces - 1 ? &sh.edge[1]
                                                                : reinterpret_cast<const uint4*>(sh.src) + v;
        float x[kVec];
        sp_unpack<DT>(*q, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int st = sp_cell(g, x[j]);
          if (st < kSpGrid) atomicAdd(&sh.hist[st], 1u);
        }
      }
      const SpFound f = sp_find<kSpSteps>(sh, 1, rate == 1 ? k : likely, -1.f);
      enough = f.bin[0] < kSpGrid;
      to = min(f.bin[0], kSpGrid - 1);
      if (rate == 1) break;
      if (enough) {
        gather();
        if (n >= (uint64_t)k && (pack ? n <= kSpPack : sh.held >= 0)) break;
        drop();
      }
      n = 0;
    }
    if (n == 0 && enough) {
      gather();
      if (pack && n > kSpPack) {
        pack = false;
        drop();
        gather();
      }
    }
    if (enough && pack) {
      const bool alone = size == 1;
      if (alone || sp_bring<true>(sh, turn)) {
        const SpPacked few = {sh, alone ? sp_packed(sh) : reinterpret_cast<uint64_t*>(sh.hist), (int)n};
        const SpFew<kSpThreads, kSpFewBins, SpPacked> first{
            sh.few, alone ? sh.hist : reinterpret_cast<uint32_t*>(sp_packed(sh)), few};
        first.settle(k, p, floor_key, u, a.V, &a.token[row], a.prob ? &a.prob[row] : nullptr);
      }
      return;  // (nothing is written to this CTA any more, or it is the first)
    }
    if (enough) {
      SpBorder b = sp_border<DT>(sh, turn, false, 0u, k);
      listed = true;
      if (p < 1.f) {
        uint64_t w = 0;
        sp_each<DT>(sh, [&](float x, int) {
          if (sp_key(x) > b.key) w += sp_weight_of(sh, x);
        });
        w = sp_sum(sh, turn, w);
        const uint64_t one = sp_weight_of(sh, sp_value(b.key));
        const uint64_t goal = max((uint64_t)1, sp_part(fmaxf(p, 0.f), w + b.ties * one, true));
        if (goal <= w) b = sp_border<DT>(sh, turn, true, b.key + 1, goal);
        else if (one) b.ties = min(b.ties, (goal - w + one - 1) / one);
      }
      key = b.key;
      ties = b.ties;
    } else {
      drop();
    }
  }
  if (!listed && p < 1.f) {
    // weights of kSpCoarse bits by steps: 1 + z + z^2 / 2 for e^z, |z| < 2^-6.5; a step's sum
    // is off by 2^-12.9 of itself at most.  (Beyond the grid the magic sum's bits are below
    // its last step's, or negative.)
    if (!clean) sp_clear(sh, kSpSteps);
    constexpr float kOne = (float)(1 << kSpCoarse), kUnit = 8388608.f + kOne;
    const int least = g.first - kSpGrid;
    const uint32_t base = smem_addr(sh.hist) + 4u * (uint32_t)g.first;
    sp_scan<2>(sh, [&](const uint4& u, int) {
      float x[kVec];
      sp_unpack<DT>(u, x);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float y = __fsub_rn(x[j], g.ref), h = __fadd_rn(y, g.magic);
        const float z = __fmul_rn(__fsub_rn(y, __fsub_rn(h, g.magic)), g.rh);
        const float m = __fmaf_rn(z, __fmaf_rn(z, 0.5f * kOne, kOne), kUnit);
        const int at = __float_as_int(h);
        if (at > least)
          asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(base - 4u * (uint32_t)at),
                       "r"(__float_as_uint(m) & 0x1fffu)
                       : "memory");
      }
    });
    sp_table(sh);
    made = true;
    const SpFound f = sp_find<kSpSteps>(sh, 0, 0, fmaxf(p, 0.f));
    const int from = min(f.bin[0], kSpGrid - 1), to = min(f.bin[1], kSpGrid - 1);
    if (floor_key && sp_cell(g, sp_value(floor_key)) < from) {
      // min_p rules out more than top_p
      key = floor_key - 1;
    } else {
      uint64_t total = 0;
      sp_runs(sh, [&](int v0, int v1) {
        uint32_t au = 0, ad = 0, bu = 0, bd = 0, n = 0, nb = 0;
        sp_scan<2>(sh, v0, v1, [&](const uint4& u, int v) {
          float x[kVec];
          sp_unpack<DT>(u, x);
          uint32_t in = 0;
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            float l;
            uint32_t up, down;
            const int st = sp_cell(g, x[j], l);
            sp_words(g, sh.grid[st], l, up, down);
            au += up;
            ad += down;
            if (st < from) bu += up, bd += down, ++nb;
            if ((unsigned)(st - from) <= (unsigned)(to - from)) in |= 1u << j;
          }
#pragma unroll 1
          for (; in; in &= in - 1) {
            const int j = __ffs(in) - 1;
            sp_gather(sh, sp_pick<DT>(u, j), sp_run(sh, v));
          }
          n += kVec;
        });
        total += sp_units(au, ad, n);
        return sp_units(bu, bd, nb);
      });
      summed = true;
      if (lane < sh.runs) above = sh.above[warp * sh.runs + lane];
      const SpGathered f2 = sp_gathered(sh, turn, from, to, above, total);
      // (the border lies among them: more than the sum above, no more than with theirs)
      const uint64_t goal = max((uint64_t)1, sp_part(fmaxf(p, 0.f), f2.sum.b, true)) - f2.sum.a;
      SpBorder b;
      const bool alone = size == 1 && sh.held >= 0;
      if (alone || f2.n <= kSpBring) {
        // few: the first CTA finds it and tells the others
        if (alone || sp_bring<false>(sh, turn)) {
          const SpValues few = {sh, alone ? sh.list : reinterpret_cast<float*>(sh.hist), (int)f2.n};
          const SpFew<kSpThreads, kSpFewBins, SpValues> first{sh.few, alone ? sh.hist : sh.hist + kSpBring, few};
          const SpRange r = first.range();
          const SpSpot e = first.find<true>(
              goal, r.bits, [&](int i) { return (r.hi - few.key(i)) >> r.low; }, [](int) { return true; });
          b.key = r.hi - (e.at << r.low);
          b.ties = sp_count(e.left, few.weight(b.key));
          if (t < (int)size) sp_put(sp_at(&sh.found[0], t), b.key, b.ties);
        }
        sp_sync();
        b.key = (uint32_t)sh.found[0].a;
        b.ties = sh.found[0].b;
      } else {
        b = sp_border<DT>(sh, turn, true, 0u, goal);
      }
      key = b.key;
      ties = b.ties;
      listed = true;
    }
  }
  if (floor_key > key) {  // (it is none of those above the gathered ones: all of them stay)
    key = floor_key - 1;  // all from floor_key on
    ties = 0;
  }
  if (!listed) {  // the weights of all that is kept, by runs
    __syncthreads();
    if (!made) sp_table(sh);
    if (t == 0) sh.from = kSpGrid, sh.held = 0;
    const float least = sp_value(key + 1);  // (key 0: a NaN, which no logit is below)
    sp_runs(sh, [&](int v0, int v1) {
      uint32_t bu = 0, bd = 0, nb = 0;
      sp_scan<2>(sh, v0, v1, [&](const uint4& u, int) {
        float x[kVec];
        sp_unpack<DT>(u, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          float l;
          uint32_t up, down;
          const int st = sp_cell(g, x[j], l);
          sp_words(g, sh.grid[st], l, up, down);
          if (!(x[j] < least)) bu += up, bd += down, ++nb;
        }
      });
      return sp_units(bu, bd, nb);
    });
    summed = true;
    above = lane < sh.runs ? sh.above[warp * sh.runs + lane] : 0;
    __syncthreads();
  }

  // The CTA's kept weights, its token's place among all of the row's.
  const uint64_t tie_weight = ties ? sp_weight_of(sh, sp_value(key)) : 0;
  SpPair cta;
  {
    uint64_t mine = above, eqs = 0;
    sp_each<DT>(sh, [&](float x, int) {
      const uint32_t y = sp_key(x);
      if (y > key) mine += sp_weight_of(sh, x);
      eqs += y == key;
    });
    sp_before(sh, mine, eqs, cta);
  }
  const SpBox* box = sp_swap(sh, turn, cta.a, cta.b);
  // of `eq` equal ones behind `before` others, those that are kept
  auto kept = [&](uint64_t before, uint64_t eq) {
    return before >= ties ? 0 : min(eq, ties - before);
  };
  uint64_t all = 0, base = 0, ties0 = 0, seen = 0;
#pragma unroll 1
  for (uint32_t r = 0; r < size; ++r) {
    if (r == rank) base = all, ties0 = seen;
    all += box[r].x.a + kept(seen, box[r].x.b) * tie_weight;
    seen += box[r].x.b;
  }
  const uint64_t want = u >= 1.f ? all - 1 : sp_part(fmaxf(u, 0.f), all, false);
  if (want >= base && want - base < cta.a + kept(ties0, cta.b) * tie_weight) {
    // the token lies in this CTA's slice: the runs' sums, two a lane
    const int runs = kSpWarps * sh.runs;
    for (int i = t; i < kSpRuns; i += kSpThreads) {
#pragma unroll
      for (int l = 0; l < kSpLimbs; ++l) sh.limbs[i][l] = 0;
      sh.ties[i] = 0;
      if (!summed || i >= runs) sh.above[i] = 0;
    }
    __syncthreads();
    sp_each<DT>(sh, [&](float x, int run) {
      const uint32_t y = sp_key(x);
      if (y > key) {
        const uint64_t w = sp_weight_of(sh, x);
#pragma unroll
        for (int l = 0; l < kSpLimbs; ++l)
          atomicAdd(&sh.limbs[run][l], (uint32_t)(w >> (kSpLimb * l)) & ((1u << kSpLimb) - 1));
      }
      if (y == key) atomicAdd(&sh.ties[run], 1u);
    });
    __syncthreads();
    uint64_t at, eq0;
    int run;
    {
      static_assert(kSpRuns == 64, "two a lane");
      const uint32_t e0 = sh.ties[2 * lane], e1 = sh.ties[2 * lane + 1];
      uint32_t eqs = e0 + e1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, eqs, o);
        if (lane >= o) eqs += x;
      }
      const uint64_t q0 = ties0 + eqs - e0 - e1, q1 = q0 + e0;
      uint64_t m0 = sh.above[2 * lane] + kept(q0, e0) * tie_weight;
      uint64_t m1 = sh.above[2 * lane + 1] + kept(q1, e1) * tie_weight;
#pragma unroll
      for (int l = 0; l < kSpLimbs; ++l) {
        m0 += (uint64_t)sh.limbs[2 * lane][l] << (kSpLimb * l);
        m1 += (uint64_t)sh.limbs[2 * lane + 1][l] << (kSpLimb * l);
      }
      uint64_t s = m0 + m1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
      }
      s += base - m0 - m1;
      const bool second = want - s >= m0;  // (where it is this lane's)
      const unsigned hit = __ballot_sync(0xffffffffu, want >= s && want - s < m0 + m1);
      const int o = hit ? __ffs(hit) - 1 : 31;
      at = __shfl_sync(0xffffffffu, second ? s + m0 : s, o);
      eq0 = __shfl_sync(0xffffffffu, second ? q1 : q0, o);
      run = __shfl_sync(0xffffffffu, 2 * lane + second, o);
    }
    // its pieces, a few a thread, in order; the second time round the token's own
    const int v1 = min((run + 1) * sh.run, pieces) * kVec, v0 = min(run * sh.run * kVec, v1);
    const int each = ((v1 - v0) / kVec + kSpThreads - 1) / kSpThreads * kVec;
    const int ea = min(v0 + t * each, v1), eb = min(ea + each, v1);
    uint64_t eqb = 0;
    bool here = true;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      uint64_t sum = 0, eq = 0;
      if (here) {
#pragma unroll 1
        for (int i = ea; i < eb; ++i) {
          const float x = sp_one<DT>(sh, i);
          const uint32_t y = sp_key(x);
          uint64_t wx = y > key ? sp_weight_of(sh, x) : 0;
          const bool tie = ties && y == key;
          if (round && tie) wx = kept(eqb, 1) * tie_weight, ++eqb;
          if (round && want - at < wx) {
            a.token[row] = i0 + i - skew;
            if (a.prob) a.prob[row] = (float)((double)wx / (double)all);
            break;
          }
          if (round) at += wx;
          sum += wx;
          eq += tie;
        }
      }
      if (round) break;
      SpPair x;
      eqb = eq0 + sp_before(sh, 0, eq, x).b;
      const uint64_t m = sum + kept(eqb, eq) * tie_weight;
      at += sp_before(sh, m, 0, x).a;
      here = want >= at && want - at < m;
    }
  }
  sp_sync();  // no CTA ends while another may still write to it
}

// Rows of up to kSpWhole tokens: a CTA of 128 threads each, all keys in shared memory, SpFew
// over all of them.  Ten rows lie on an SM at once, where the cluster's kernel has two.
// Both sides, us (settings of every kind; top_p 0.9): 704 rows of 52 11, 10 here, 49, 56 there;
// 304 of 1400 27, 22 and 30, 30; 1216 of 1000 36, 42 and 99, 116; one of 1400 19, 20 and 21, 21;
// but one of 2000 24, 25 and 21, 21, 304 of 2000 34, 29 and 30, 30.  (1216 of 2000 66, 77 and 91,
// 112: not taken, the kernel depends on the row's length alone, and a row's token with it.)
constexpr int kSpWhole = 1536;
constexpr int kSpWholeThreads = 128, kSpWholeBins = 256;
struct SpWhole {
  uint32_t keys[kSpWhole];
  uint32_t hist[kSpLimbs * kSpWholeBins];
  SpFewShared few;
  uint32_t top[kSpWholeThreads / 32];
  uint32_t floor_key, first;
};
struct SpRow {
  const SpWhole& sh;
  const SpScale& c;
  int n;
  __device__ __forceinline__ uint32_t key(int i) const { return sh.keys[i]; }
  __device__ __forceinline__ uint32_t index(int i) const { return (uint32_t)i; }
  __device__ __forceinline__ uint64_t weight(uint32_t key) const { return sp_weight(c, sp_value(key), kSpPowers.at); }
};

template <int DT>
__global__ void __launch_bounds__(kSpWholeThreads) k_sample_whole(const __grid_constant__ SampleParams a) {
  __shared__ SpWhole sh;
  const int t = threadIdx.x, row = blockIdx.x;
  if (t == 0) sh.first = 0xffffffffu;
  pdl_launch_dependents();
  pdl_wait();
  float temp = a.temperature ? a.temperature[row] : 1.f;
  const float p = a.top_p ? a.top_p[row] : 1.f, low = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
  int k = a.top_k ? a.top_k[row] : 0;
  float top = -INFINITY;
#pragma unroll 4
  for (int i = t; i < a.V; i += kSpWholeThreads) {
    float x;
    if constexpr (DT == DT_F32) x = static_cast<const float*>(a.logits)[(long long)row * a.ld + i];
    else if constexpr (DT == DT_BF16) x = bf16lo(static_cast<const uint16_t*>(a.logits)[(long long)row * a.ld + i]);
    else x = __half2float(__ushort_as_half(static_cast<const uint16_t*>(a.logits)[(long long)row * a.ld + i]));
    top = max_nan(top, x);
    sh.keys[i] = sp_key(x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((t & 31) == 0) sh.top[t >> 5] = __float_as_uint(top);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSpWholeThreads / 32; ++w) top = max_nan(top, __uint_as_float(sh.top[w]));
  if (!(fabsf(top) <= FLT_MAX) || temp != temp || p != p || low != low || u != u) {
    if (t == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  if (!(temp > 0.f)) temp = 1.f, k = 1;
  if (k == 1) {
    const uint32_t key = sp_key(top);
    for (int i = t; i < a.V; i += kSpWholeThreads)
      if (sh.keys[i] == key) atomicMin(&sh.first, (uint32_t)i);
    __syncthreads();
    if (t == 0) {
      a.token[row] = (int)sh.first;
      if (a.prob) a.prob[row] = 1.f;
    }
    return;
  }
  temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
  SpScale c;
  float r, e;
  sp_scale(top, temp, c, r, e);
  if (t == 0) sh.floor_key = low > 0.f ? sp_floor(top, temp, low) : 0u;
  __syncthreads();
  const SpRow all = {sh, c, a.V};
  SpFew<kSpWholeThreads, kSpWholeBins, SpRow>{sh.few, sh.hist, all}.settle(
      k > 1 && k < a.V ? k : a.V, p, sh.floor_key, u, a.V, &a.token[row], a.prob ? &a.prob[row] : nullptr);
}

static_assert(sizeof(SpShared) <= 113 * 1024, "two CTAs a SM");
constexpr int kSpStay = 227 * 1024 - (int)sizeof(SpShared);
// bytes of a slice's pieces, wherever it begins in its first one
static int sp_stay(int per, int vec) { return (per + 2 * vec - 2) / vec * 16; }

// CTAs a row and launch.  A slice stays in shared memory where it fits and each CTA finds an
// SM: the most CTAs a row, to 8, with which all clusters lie on the SMs at once (the runtime
// says how many do), slices no shorter than 2048 tokens on half of the SMs and 8192 on more; 16
// only for slices of 8192 on half of them.  Both sides, us, top_p 0.9 and settings of every kind:
// 16 rows of 151936 fp32 in six 35, 36, in five 48, 42 (its slices do not fit), in eight 43, 42 (two
// CTAs a SM); 14 rows in eight 32, 33, and 43, 39 with nothing in shared memory; 8 rows in eight 31,
// 32, in sixteen 40, 36; one row of 50257 24, 26, in sixteen 26, 28; 19 of 50257 in six 26, 27, in
// seven 33, 31.
// Else two CTAs a SM: as many as all clusters lie there at once with, slices of 8192.  64 rows of
// 151936 fp32 in four 62, 73, in two 89, 101; but 76 rows of bf16 in four, which do not fit, 87, 66,
// in two 57, 73.  Slices of 32768 also where pairs of CTAs take two waves, the costly rows first: whole
// rows are all resident, and an SM with two costly ones holds up the rest.  256 rows of 151936
// bf16 in two 163, 98, whole 142, 150 (without settings 107 and 91: whole).  160 to 300 rows of
// 65536, 100000 and 151936: settings of every kind bf16 60 to 115 in two and 83 to 158 whole, fp32
// 79 to 163 and 112 to 309; top_p 0.9 for all bf16 81 to 168 and 72 to 144, fp32 87 to 187 and 79 to
// 172; the largest of all 18 to 64 and 13 to 67: what one setting for all loses (a quarter to a half
// at 65536, little at 151936) is less than what different ones gain, and which it is only the device
// knows.  But 256 of 32000 in two 79, 56, whole 52, 67; 500 of 50257 fp32 174, 126 and 144, 104.
template <int DT>
static cudaError_t sample_launch(SampleParams p, cudaStream_t stream) {
  if (p.V <= kSpWhole) return launch_serving(k_sample_whole<DT>, dim3((unsigned)p.rows), kSpWholeThreads, 0, stream, p);
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static bool ready[kMaxDev] = {false};
  // clusters of that many CTAs on the device at once; and with an SM for each CTA
  static int fit[kMaxDev][kSpMaxCluster + 1], alone[kMaxDev][kSpMaxCluster + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDev) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSpThreads);
  cfg.attrs = at;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev]) {
      e = cudaFuncSetAttribute(k_sample_tokens<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)sizeof(SpShared) + kSpStay);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_sample_tokens<DT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      cfg.numAttrs = 1;
      for (int c = 1; c <= kSpMaxCluster && e == cudaSuccess; ++c) {
        at[0].val.clusterDim.x = c;
        cfg.gridDim = dim3((unsigned)c);
        cfg.dynamicSmemBytes = (int)sizeof(SpShared);
        e = cudaOccupancyMaxActiveClusters(&fit[dev][c], k_sample_tokens<DT>, &cfg);
        cfg.dynamicSmemBytes = (int)sizeof(SpShared) + kSpStay;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&alone[dev][c], k_sample_tokens<DT>, &cfg);
      }
      if (e != cudaSuccess) return e;
      ready[dev] = true;
    }
  }
  const bool differ = p.temperature || p.top_k || p.top_p;  // rows may differ in what they cost
  const int least = p.V > 1 << 18 ? 2 : 1;                  // (a thread's words add up 2^9 logits at most)
  // half: of the SMs, with one each
  auto half = [&](int c) { return p.rows * c <= device_sm_count() / 2; };
  auto stay = [&](int c) { return sp_stay((p.V + c - 1) / c, kSpVec<DT>); };
  int c = kSpMaxCluster;
  for (; c >= least; c = c == kSpMaxCluster ? 8 : c - 1) {
    const int per = p.V / c;
    if (p.rows <= alone[dev][c] && stay(c) <= kSpStay &&
        (c == 1 || (per >= 2048 && half(c) && c <= 8) || (per >= 8192 && (c <= 8 || half(c)))))
      break;
  }
  p.stays = c >= least;
  if (!p.stays)
    for (c = least; c < 8; c *= 2) {
      const int per = p.V / (2 * c), at_once = fit[dev][2 * c];
      if (!(per >= 2048 && half(2 * c)) && !(per >= 8192 && p.rows <= at_once) &&
          !(per >= 32768 && c == 1 && p.rows <= 2 * at_once && differ))
        break;
    }
  p.per = (p.V + c - 1) / c;
  p.ranked = differ && p.rows * c > 2 * device_sm_count();
  at[0].val.clusterDim.x = c;
  cfg.gridDim = dim3((unsigned)(p.rows * c));
  cfg.dynamicSmemBytes = (int)sizeof(SpShared) + (p.stays ? stay(c) : 0);
  cfg.stream = stream;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_sample_tokens<DT>, p);
}

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_sample_tokens(const void *logits, int dtype, long long ld, const float *u,
                           const float *temperature, const int32_t *top_k, const float *top_p,
                           const float *min_p, int32_t *token, float *prob, int rows, int V,
                           ws_stream_t stream) {
  if (!logits || !u || !token) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if (dtype != WS_DTYPE_F32 && dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) {
    set_error("unknown dtype %d", dtype);
    return WS_ERR_ARG;
  }
  if (rows < 1 || rows > 65536 || V < 1 || V > kSpMaxV || ld < V) {
    set_error("sampling: rows 1..65536, V 1..%d, ld at least V", kSpMaxV);
    return WS_ERR_SHAPE;
  }
  if ((uintptr_t)logits & (dtype == WS_DTYPE_F32 ? 3u : 1u)) {
    set_error("sampling: logits must be aligned to their type");
    return WS_ERR_ALIGN;
  }
  SampleParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.token = token;
  p.prob = prob;
  p.rows = rows;
  p.V = V;
  cudaError_t e;
  if (dtype == WS_DTYPE_F32) e = sample_launch<DT_F32>(p, (cudaStream_t)stream);
  else if (dtype == WS_DTYPE_BF16) e = sample_launch<DT_BF16>(p, (cudaStream_t)stream);
  else e = sample_launch<DT_F16>(p, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
