// ws_prompt_attention.cu -- causal attention over packed prompts with grouped
// heads: token t of a sequence attends to the sequence's tokens up to t.
//
// out = sum_j p_j v_j, p = softmax_j(q . k_j / sqrt(128)); one pass over the
// keys with a running maximum m and sum l: p_j = 2^(c s_j - m), l = sum p_j,
// out = sum p_j v_j / l, c = log2(e) / sqrt(128).  m follows the keys' maximum
// only when that is 2^8 above it, so the output accumulators are rarely
// rescaled and a p is at most 2^8.
//
// One CTA takes two tiles of 128 query rows that read the same keys and
// values: two heads of one group over the same tokens where the group is even,
// else two neighbouring runs of tokens of one head.  Sixteen warps:
//   0..3, 4..7  the softmax of tile 0 and of tile 1, a thread a row: scores out
//               of tensor memory, probabilities back into it over the scores;
//   8, 9        issue the products of tile 0 and of tile 1 (one thread each): S =
//               Q K^T from shared memory, O += P V with P from tensor memory,
//               both accumulators there (S, S, O, O: the 512 columns).  The
//               tensor cores take a product when they begin it, not before, so
//               one thread for both tiles leaves them idle while it waits;
//   10          the copies: Q once, K and V through two stages each;
//   12..15      guard the values of the last blocks, where keys are masked: a
//               probability of 0 times a value that is not finite would still
//               be NaN, so those values, and the rows behind the sequence, are
//               zeroed in shared memory before the product, and the rows that
//               do attend to such a value get its share at the end.
//
// Bound by the tensor cores, then by the chain score -> maximum -> powers ->
// product that each tile goes through (about 2200 cycles a block, 1054 of them
// in the products; two tiles a CTA overlap to 2700): one sequence of 8192
// tokens, 32 heads over 8: 320-335 us in runs of 30, 1640-1720 TFLOP/s of the
// unmasked pairs, 0.88-0.92 of the measured matrix rate; 346-358 us in long runs
// of calls, under the power cap.  A thread
// for each tile's products instead of one for both took 434 us to 341; row
// maxima with the loads (tcgen05.ld.red) and the two-part hand-over the rest.
// Prompts that fill less than one wave take as long as their longest tile's
// chain, about 1.4 us a block, with about 4.6 us before and behind it (1712 + 61
// tokens, 8/8 heads: 25.6 us, the floor 3.2; 2692 + 129 + 19: 36.4 against 8.0).
#include <cfloat>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "ws_kv_q4.cuh"
#include "ws_tcgen05.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kPromptDim = 128;
constexpr int kPaTile = 128;                       // query rows a tile, keys a block
constexpr int kPaThreads = 512;
constexpr int kPaTileBytes = kPaTile * kPromptDim * 2;
constexpr int kPaHalf = kPaTileBytes / 2;          // 128 rows of 64 values, 128-byte swizzle
constexpr int kPaStages = 2;                       // of keys, and of values
constexpr int kPaSmem = (2 + 2 * kPaStages) * kPaTileBytes + 1024;
// A block's probabilities are handed over in two parts, so that the product
// starts on the first 96 keys while the last 32 are on their way (20.9 us for
// prompts of 2252 tokens in 6 sequences, 12 heads; 22.7 with 64 and 64, 22.8
// with 32 and 96; four parts cost more in waits than they win).
constexpr int kPaParts = 2, kPaCut = 96;
constexpr float kPaLazy = 8.f;
constexpr int kPaRegsSoftmax = 216, kPaRegsOther = 40;
static_assert(256 * kPaRegsSoftmax + 256 * kPaRegsOther <= kPaThreads * 128,
              "the register shares fit what the block is launched with");

struct PromptParams {
  CUtensorMap mq, mk, mv;  // [T][heads][128], boxes of 128 tokens x 64 dimensions
  const uint16_t* q;       // the same, for the rows that need single values
  const uint16_t* k;
  const uint16_t* v;
  const int* cu;           // [n + 1]
  uint16_t* out;           // [T][nh * 128]
  float* lse;              // [T][nh] or null
  long long qs, ks, vs;
  int T, n, nh, nkv;
  int pair;                // 1: the tiles are two heads; 0: two runs of one head
  float scale;             // log2(e) / sqrt(128)
  int* err;
  unsigned long long timeout_ns;
  TestHold hold;           // copies: 0, 1 the tiles' queries, 2 + 2 j and 3 + 2 j block j's keys and values
};

struct PaShared {
  uint64_t q_full[2], k_full[kPaStages], k_empty[kPaStages], v_full[kPaStages], v_empty[kPaStages];
  uint64_t s_full[2], p_full[2][kPaParts], o_full[2], guard_go[2], guard[2];
  uint32_t tmem;
  uint32_t odd[2][4];      // values of the guarded blocks that are not finite, a bit a key
  int sent[6];             // copies started on q_full, k_full and v_full, each in turn
  int abort;
};

__device__ __forceinline__ float pa_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Wait with the library's limit; a wait that runs out ends every other one.
__device__ __forceinline__ bool pa_wait_slow(uint64_t* bar, uint32_t parity, PaShared* sh, int* err,
                                          unsigned long long timeout_ns) {
  const uint64_t t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&sh->abort) return false;
    if (global_ns() - t0 > timeout_ns) {
      *(volatile int*)&sh->abort = 1;
      atomicExch(err, (int)DERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, PaShared* sh,
                                        const PromptParams& a) {
  if (mbar_try_wait(bar, parity)) return true;
  return pa_wait_slow(bar, parity, sh, a.err, a.timeout_ns);
}

// Sequence and query block of tile `t` (units of `rows` tokens), by the whole
// warp: the tiles with the most keys first, whatever their sequence, while the
// bounds fit the lanes; sequence by sequence beyond that (33 sequences of 20 to
// 700 tokens, 16/4 heads, 66.4 us, 63.9 when the longest sequences come first; 64
// of them 110.6 and 107.5).  false: no such tile.
__device__ __forceinline__ bool pa_place(const PromptParams& a, int t, int rows, int& first,
                                         int& len, int& block) {
  const int lane = threadIdx.x & 31;
  const unsigned all = 0xffffffffu;
  for (int b0 = 0; b0 < a.n; b0 += 32) {
    const int i = b0 + lane;
    int lo = 0, hi = 0;
    if (i < a.n) {
      lo = a.cu[i];
      hi = a.cu[i + 1];
      if (lo < 0 || hi < lo || hi > a.T) {
        // (every CTA that gets this far: there is one more of them than tiles for
        // each sequence without tiles)
        if (threadIdx.x < 32) atomicExch(a.err, kDerrBadSeq);
        lo = hi = 0;
      }
    }
    const int nt = (hi - lo + rows - 1) / rows;
    const int total = __reduce_add_sync(all, nt);
    if (t >= total) {
      t -= total;
      continue;
    }
    int src;
    if (a.n <= 32) {
      // tiles of block b and up: sum max(0, nt - b); the largest b with more than t
      int lo_b = 0, hi_b = __reduce_max_sync(all, nt);
      while (hi_b - lo_b > 1) {
        const int mid = (lo_b + hi_b) >> 1;
        if (__reduce_add_sync(all, max(0, nt - mid)) > t) lo_b = mid; else hi_b = mid;
      }
      block = lo_b;
      const int rank = t - __reduce_add_sync(all, max(0, nt - block - 1));
      unsigned m = __ballot_sync(all, nt > block);
      for (int k = 0; k < rank; ++k) m &= m - 1;
      src = __ffs(m) - 1;
    } else {
      int sum = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(all, sum, o);
        if (lane >= o) sum += u;
      }
      src = __ffs(__ballot_sync(all, sum > t)) - 1;
      block = __shfl_sync(all, sum, src) - 1 - t;
    }
    first = __shfl_sync(all, lo, src);
    len = __shfl_sync(all, hi, src) - first;
    return true;
  }
  return false;
}

template <int DT>
__device__ __forceinline__ float pa_value(const uint16_t* p) {
  return DT == DT_F16 ? __half2float(__ushort_as_half(*p)) : __uint_as_float((uint32_t)*p << 16);
}
template <int DT>
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  if constexpr (DT == DT_F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The share of the guarded values that are not finite in 32 dimensions of one
// row's accumulators: p times the value for each that the row attends to.
template <int DT>
__device__ __forceinline__ void pa_odd_values(const PromptParams& a, const PaShared* sh, int first,
                                           int tok, int guard0, int head, int kvh, float m, int d0,
                                           uint32_t* o) {
  for (int e = 0; e < 2; ++e)
    for (int w = 0; w < 4; ++w) {
      uint32_t bits = sh->odd[e][w];
      while (bits) {
        const int key = (guard0 + e) * kPaTile + w * 32 + __ffs(bits) - 1;
        bits &= bits - 1;
        if (key > tok) continue;
        const uint16_t* q = a.q + (size_t)(first + tok) * a.qs + (size_t)head * kPromptDim;
        const uint16_t* k = a.k + (size_t)(first + key) * a.ks + (size_t)kvh * kPromptDim;
        const uint16_t* v = a.v + (size_t)(first + key) * a.vs + (size_t)kvh * kPromptDim + d0;
        float s = 0.f;
        for (int d = 0; d < kPromptDim; ++d) s = fmaf(pa_value<DT>(q + d), pa_value<DT>(k + d), s);
        const float p = pa_exp2(fmaf(s, a.scale, -m));
#pragma unroll
        for (int d = 0; d < 32; ++d)
          o[d] = __float_as_uint(fmaf(p, pa_value<DT>(v + d), __uint_as_float(o[d])));
      }
    }
}

template <int DT>
__global__ void __launch_bounds__(kPaThreads, 1)
    k_prompt_attention(const __grid_constant__ PromptParams a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ PaShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 10 && lane < 3) tma_prefetch_map(lane == 0 ? &a.mq : lane == 1 ? &a.mk : &a.mv);
  pdl_launch_dependents();
  pdl_wait();
  const int heads = a.pair ? a.nh / 2 : a.nh, rows = a.pair ? kPaTile : 2 * kPaTile;
  int first, len, block;
  if (!pa_place(a, blockIdx.x / heads, rows, first, len, block)) return;
  const int h0 = (blockIdx.x % heads) * (a.pair ? 2 : 1), kvh = h0 / (a.nh / a.nkv);
  // per tile: head, first row of the sequence, blocks of keys (0: no tile)
  const int row0 = block * rows, row1 = a.pair ? row0 : row0 + kPaTile;
  const int n0 = row0 / kPaTile + 1, n1 = row1 < len ? row1 / kPaTile + 1 : 0;
  const int nb = max(n0, n1), guard0 = n0 - 1;  // the blocks from guard0 on hold masked keys

  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sq = smem;
  unsigned char* sk = smem + 2 * kPaTileBytes;
  unsigned char* sv = sk + kPaStages * kPaTileBytes;

  // a tile's rows of one head: two boxes of 64 dimensions; `id` as in the
  // parameters' `hold`, `slot` the barrier's place in `sent`
  // (asked for once: a comparison of the CTA's index with the parameter ahead of
  // each copy took 8192 tokens, 32/8 heads from 321 to 333 us)
  const int hold = a.hold.here();
  auto copy = [&](unsigned char* dst, const CUtensorMap* map, int h, int tok, uint64_t* bar, int slot,
                  int id) {
    if (id == hold) return;
    mbar_arrive_expect_tx(bar, kPaTileBytes);
    tma_load_3d(dst, map, 0, h, tok, bar);
    tma_load_3d(dst + kPaHalf, map, 64, h, tok, bar);
    ++sh.sent[slot];
  };
  // the copies' warp starts the barriers and the first copies before the
  // tensor memory is there
  if (warp == 10 && elect_one()) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.s_full[i], 1);
      for (int h = 0; h < kPaParts; ++h) mbar_init(&sh.p_full[i][h], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.guard_go[i], 1);
      mbar_init(&sh.guard[i], 128);
    }
    for (int i = 0; i < kPaStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], n1 > 0 ? 2 : 1);  // both tiles are done with a stage
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], n1 > 0 ? 2 : 1);
    }
    fence_mbar_init();
    sh.abort = 0;
    for (int i = 0; i < 6; ++i) sh.sent[i] = 0;
    copy(sq, &a.mq, h0, first + row0, &sh.q_full[0], 0, 0);
    copy(sk, &a.mk, kvh, first, &sh.k_full[0], 2, 2);
    if (n1 > 0) copy(sq + kPaTileBytes, &a.mq, h0 + a.pair, first + row1, &sh.q_full[1], 1, 1);
    copy(sv, &a.mv, kvh, first, &sh.v_full[0], 4, 3);
    if (guard0 == 0) mbar_arrive(&sh.guard_go[0]);
  }
  if (threadIdx.x < 8) sh.odd[threadIdx.x >> 2][threadIdx.x & 3] = 0;
  if (warp == 8) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // every role's end; after it nothing more is issued, and `abort` stays as it is
  auto leave = [&]() {
    __syncwarp();
    tc_fence_before();
    consumer_sync(kPaThreads);
  };
  auto aborted = [&]() { return *(volatile int*)&sh.abort != 0; };

  if (warp < 8) {
    regs_raise<kPaRegsSoftmax>();
    const int tile = warp >> 2, r = (warp & 3) * 32 + lane;
    const int n = tile ? n1 : n0, head = h0 + (a.pair ? tile : 0);
    const int tok = (tile ? row1 : row0) + r;  // of the sequence
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + tile * 128 + lanes, to = tmem + 256 + tile * 128 + lanes;
    float m = -FLT_MAX;  // below every finite score
    float2 l = make_float2(0.f, 0.f);
    bool ok = true;
    // one block of keys; the last one holds the diagonal
    auto softmax = [&](int j, auto diagonal) {
      ok = pa_wait(&sh.s_full[tile], j & 1, &sh, a);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      tc_fence_after();
      uint32_t s[128], mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_max(ts + 32 * c, s + 32 * c, mx[c]);
      tmem_wait_ld();
      tmem_loaded<128>(s);
      asm volatile("" : "+r"(mx[0]), "+r"(mx[1]), "+r"(mx[2]), "+r"(mx[3]));
      if constexpr (decltype(diagonal)::value) {
        // the diagonal: of the warp's 32 rows, the 32 keys of its own number
        // are masked one by one, those after them all
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < (warp & 3)) continue;
          float y = -INFINITY;
          if (c == (warp & 3)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (i > lane) s[32 * c + i] = 0xff800000u;
              y = fmaxf(y, __uint_as_float(s[32 * c + i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * c + i] = 0xff800000u;
          }
          mx[c] = __float_as_uint(y);
        }
      }
      const float top = fmaxf(fmaxf(__uint_as_float(mx[0]), __uint_as_float(mx[1])),
                              fmaxf(__uint_as_float(mx[2]), __uint_as_float(mx[3]))) * a.scale;
      if (__any_sync(0xffffffffu, top > m + kPaLazy)) {
        const float mn = fmaxf(m, top), f = pa_exp2(m - mn);
        m = mn;
        l.x *= f, l.y *= f;
        if (j > 0) {  // the products up to block j - 1 are done: this block's scores came after
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t o[32];
            tmem_ld32(to + c, o);
            tmem_wait_ld();
            tmem_loaded<32>(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(to + c, o);
          }
        }
      }
      const float2 sc = make_float2(a.scale, a.scale), nm = make_float2(-m, -m);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 32 * h + 2 * i;
          float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, nm);
          x.x = pa_exp2(x.x);
          x.y = pa_exp2(x.y);
          l = add2(l, x);
          p[i] = pa_pack<DT>(x.x, x.y);
        }
        tmem_st16(ts + 16 * h, p);
        if (32 * (h + 1) == kPaCut || h == 3) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[tile][h == 3]);
        }
      }
    };
#pragma unroll 1
    for (int j = 0; j < n - 1 && ok; ++j) softmax(j, std::false_type());
    if (n > 0 && ok) softmax(n - 1, std::true_type());
    if (n > 0 && ok) ok = __all_sync(0xffffffffu, pa_wait(&sh.o_full[tile], 0, &sh, a) && !aborted());
    if (n > 0 && ok) {
      tc_fence_after();
      const float sum = l.x + l.y, inv = 1.f / sum;
      const uint32_t odd = sh.odd[0][0] | sh.odd[0][1] | sh.odd[0][2] | sh.odd[0][3] |
                           sh.odd[1][0] | sh.odd[1][1] | sh.odd[1][2] | sh.odd[1][3];
      // rows to the tile's query buffer (its products are done), 16-byte
      // pieces in an order that spreads over the banks, then out row by row
      unsigned char* st = sq + tile * kPaTileBytes + (warp & 3) * 32 * 256;
      uint32_t o[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(to + 32 * c, o + 32 * c);
      tmem_wait_ld();
      tmem_loaded<128>(o);
      if (odd && tok < len) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          pa_odd_values<DT>(a, &sh, first, tok, guard0, head, kvh, m, 32 * c, o + 32 * c);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pa_pack<DT>(__uint_as_float(o[8 * i + 2 * e]) * inv,
                             __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
        *reinterpret_cast<uint4*>(st + lane * 256 + (i ^ (lane & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (a.lse && tok < len)
        a.lse[(size_t)(first + tok) * a.nh + head] = (m + log2f(sum)) * 0.6931471805599453f;
      __syncwarp();
      const int base = tok - lane;  // the warp's first row
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int rr = 2 * i + (lane >> 4), piece = lane & 15;
        if (base + rr < len)
          *reinterpret_cast<uint4*>(a.out + ((size_t)(first + base + rr) * a.nh + head) * kPromptDim +
                                    piece * 8) =
              *reinterpret_cast<const uint4*>(st + rr * 256 + (piece ^ (rr & 7)) * 16);
      }
    }
    leave();
  } else {
    regs_lower<kPaRegsOther>();
    if (warp < 10) {
      const int tile = warp - 8, n = tile ? n1 : n0;
      if (n > 0 && elect_one()) {
        constexpr uint32_t qk = mma_idesc(DT == DT_BF16, false, kPaTile, kPaTile);
        constexpr uint32_t pv = mma_idesc(DT == DT_BF16, true, kPaTile, kPromptDim);
        const uint32_t ts = tmem + tile * 128, to = tmem + 256 + tile * 128;
        const uint32_t q = smem_addr(sq + tile * kPaTileBytes);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok) ok = pa_wait(bar, parity, &sh, a);
        };
        auto scores = [&](int j) {  // S = Q K^T, 16 dimensions at a time
          const uint32_t k = smem_addr(sk + (j % kPaStages) * kPaTileBytes);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = (i >> 2) * kPaHalf + (i & 3) * 32;
            mma_ss(ts, smem_desc(q + at, 16, 1024), smem_desc(k + at, 16, 1024), qk, i > 0);
          }
          mma_commit(&sh.s_full[tile]);
          if (j + kPaStages < nb) mma_commit(&sh.k_empty[j % kPaStages]);  // filled again
        };
        wait(&sh.k_full[0], 0);
        wait(&sh.q_full[tile], 0);
        if (ok) scores(0);
        for (int j = 0; j < n && ok; ++j) {
          const int s = j % kPaStages, s1 = (j + 1) % kPaStages;
          wait(&sh.v_full[s], (j / kPaStages) & 1);
          if (j >= guard0) wait(&sh.guard[j - guard0], 0);
          if (j + 1 < n) wait(&sh.k_full[s1], ((j + 1) / kPaStages) & 1);
          const uint32_t v = smem_addr(sv + s * kPaTileBytes);
#pragma unroll
          for (int h = 0; h < kPaParts; ++h) {  // O += P V, 16 keys at a time
            wait(&sh.p_full[tile][h], j & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = h ? kPaCut / 16 : 0; i < (h ? kPaTile : kPaCut) / 16; ++i)
              mma_ts(to, ts + i * 8, smem_desc(v + i * 2048, kPaHalf, 1024), pv, j > 0 || i > 0);
          }
          if (!ok) break;
          if (j + kPaStages < nb) mma_commit(&sh.v_empty[s]);
          if (j + 1 < n) scores(j + 1);
          else mma_commit(&sh.o_full[tile]);
        }
        if (!ok) mma_commit(&sh.o_full[tile]);  // either way: behind every product of the tile
      }
    } else if (warp == 10) {
      if (elect_one()) {
        for (int j = 1; j < nb; ++j) {  // block 0 is on its way
          const int s = j % kPaStages;
          const uint32_t par = (j / kPaStages + 1) & 1;
          if (j >= kPaStages && !pa_wait(&sh.k_empty[s], par, &sh, a)) break;
          copy(sk + s * kPaTileBytes, &a.mk, kvh, first + j * kPaTile, &sh.k_full[s], 2 + s, 2 + 2 * j);
          if (j >= kPaStages && !pa_wait(&sh.v_empty[s], par, &sh, a)) break;
          copy(sv + s * kPaTileBytes, &a.mv, kvh, first + j * kPaTile, &sh.v_full[s], 4 + s, 3 + 2 * j);
          // from here on the stage's phase is this block's
          if (j >= guard0) mbar_arrive(&sh.guard_go[j - guard0]);
        }
      }
    } else if (warp >= 12) {
      const int key = (warp - 12) * 32 + lane;
      for (int j = guard0; j < nb; ++j) {
        const int s = j % kPaStages;
        if (!pa_wait(&sh.guard_go[j - guard0], 0, &sh, a) ||
            !pa_wait(&sh.v_full[s], (j / kPaStages) & 1, &sh, a))
          break;
        const int valid = len - j * kPaTile;  // keys of the block inside the sequence
        uint4* half0 = reinterpret_cast<uint4*>(sv + s * kPaTileBytes + key * 128);
        uint4* half1 = reinterpret_cast<uint4*>(sv + s * kPaTileBytes + kPaHalf + key * 128);
        bool zero = key >= valid;
        if (!zero) {
          uint32_t bad = 0;
#pragma unroll 4
          for (int i = 0; i < 8; ++i) {
            const uint4 u = half0[i], x = half1[i];
            const uint32_t w[8] = {u.x, u.y, u.z, u.w, x.x, x.y, x.z, x.w};
            // an exponent of all ones carries into the sign's place
            constexpr uint32_t kExp = DT == DT_F16 ? 0x7c007c00u : 0x7f807f80u;
            constexpr uint32_t kOne = DT == DT_F16 ? 0x04000400u : 0x00800080u;
#pragma unroll
            for (int e = 0; e < 8; ++e) bad |= (w[e] & kExp) + kOne;
          }
          zero = (bad & 0x80008000u) != 0;
          if (zero) atomicOr(&sh.odd[j - guard0][key >> 5], 1u << (key & 31));
        }
        if (zero) {
#pragma unroll
          for (int i = 0; i < 8; ++i) half0[i] = half1[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // what was zeroed before the product reads it
        mbar_arrive(&sh.guard[j - guard0]);
      }
    }
    leave();
    // After a wait that ran out, whoever's it was: no product and no copy of this
    // CTA stays under way behind it.
    if (warp < 10 && aborted()) {
      if (warp == 8 || n1 > 0) mbar_wait_bounded(&sh.o_full[warp - 8], 0, a.timeout_ns);
    } else if (warp == 10 && aborted()) {
      static_assert(kPaStages == 2, "six barriers of copies");
      if (elect_one())
        for (int i = 0; i < 6; ++i) {
          uint64_t* bar = i < 2 ? &sh.q_full[i] : i < 4 ? &sh.k_full[i - 2] : &sh.v_full[i - 4];
          if (sh.sent[i]) mbar_wait_bounded(bar, (sh.sent[i] - 1) & 1, a.timeout_ns);
        }
    }
  }
  if (aborted()) __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

typedef CUresult (*PaEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                               const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                               const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, and the kernels' attribute, once per device.
static PaEncodeFn pa_setup(cudaError_t* err) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static PaEncodeFn fn = nullptr;
  static bool ready[kMaxDev] = {false};
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err == cudaSuccess && (dev < 0 || dev >= kMaxDev)) *err = cudaErrorInvalidDevice;
  if (*err != cudaSuccess) return nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    *err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                            cudaEnableDefault, &q);
    if (*err == cudaSuccess && q != cudaDriverEntryPointSuccess) *err = cudaErrorNotSupported;
    if (*err != cudaSuccess) return nullptr;
    fn = reinterpret_cast<PaEncodeFn>(ptr);
  }
  if (!ready[dev]) {
    *err = cudaFuncSetAttribute(k_prompt_attention<DT_BF16>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kPaSmem);
    if (*err == cudaSuccess)
      *err = cudaFuncSetAttribute(k_prompt_attention<DT_F16>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kPaSmem);
    if (*err != cudaSuccess) return nullptr;
    ready[dev] = true;
  }
  return fn;
}

static bool pa_map(PaEncodeFn fn, CUtensorMap* map, int dtype, const void* base, int T, int heads,
                   long long stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)kPromptDim, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {kPromptDim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {kPromptDim / 2, 1, kPaTile};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, dtype == WS_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_prompt_attention(const void *q, const void *k, const void *v, int dtype,
                              const int32_t *cu_seqlens, void *out, float *lse, int T, int n_seqs,
                              int n_heads, int n_kv_heads, int head_dim, long long q_stride,
                              long long k_stride, long long v_stride, ws_stream_t stream) {
  if (!q || !k || !v || !cu_seqlens || !out) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if (dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) {
    set_error("dtype must be WS_DTYPE_BF16 or WS_DTYPE_F16");
    return WS_ERR_ARG;
  }
  if (T < 1 || n_seqs < 1 || n_kv_heads < 1 || n_heads < 1 || n_heads > 65535 ||
      n_heads % n_kv_heads || head_dim != kPromptDim || q_stride % 8 || k_stride % 8 ||
      v_stride % 8 || q_stride < (long long)n_heads * kPromptDim ||
      k_stride < (long long)n_kv_heads * kPromptDim ||
      v_stride < (long long)n_kv_heads * kPromptDim) {
    set_error("prompt attention: T and sequences at least 1, head_dim %d, n_heads (to 65535) a "
              "multiple of n_kv_heads, token strides a multiple of 8 and at least the heads' "
              "dimensions", kPromptDim);
    return WS_ERR_SHAPE;
  }
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) & 15u) {
    set_error("prompt attention: q, k, v and out must be 16-byte aligned");
    return WS_ERR_ALIGN;
  }
  PromptParams a = {};
  a.pair = (n_heads / n_kv_heads) % 2 == 0;
  // at most: the tokens' whole tiles, and one more a sequence
  const long long rows = a.pair ? kPaTile : 2 * kPaTile;
  const long long tiles = T / rows + n_seqs, grid = tiles * (a.pair ? n_heads / 2 : n_heads);
  if (grid > 0x7fffffffll || T > 0x7fffffff - 2 * kPaTile) {
    set_error("prompt attention: too many tiles (%lld)", grid);
    return WS_ERR_SHAPE;
  }
  cudaError_t e = cudaSuccess;
  const PaEncodeFn fn = pa_setup(&e);
  if (!fn) {
    set_error("prompt attention setup failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  if (!pa_map(fn, &a.mq, dtype, q, T, n_heads, q_stride) ||
      !pa_map(fn, &a.mk, dtype, k, T, n_kv_heads, k_stride) ||
      !pa_map(fn, &a.mv, dtype, v, T, n_kv_heads, v_stride)) {
    set_error("prompt attention: tensor map encoding failed");
    return WS_ERR_CUDA;
  }
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.cu = cu_seqlens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.T = T;
  a.n = n_seqs;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.scale = (float)(1.4426950408889634 / sqrt((double)kPromptDim));
  a.timeout_ns = tuning().timeout_ns;
  a.hold = test_hold();
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  if (dtype == WS_DTYPE_F16)
    e = launch_serving(k_prompt_attention<DT_F16>, dim3((unsigned)grid), kPaThreads, kPaSmem, (cudaStream_t)stream, a);
  else
    e = launch_serving(k_prompt_attention<DT_BF16>, dim3((unsigned)grid), kPaThreads, kPaSmem, (cudaStream_t)stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
