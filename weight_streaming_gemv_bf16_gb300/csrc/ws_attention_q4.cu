// ws_attention_q4.cu -- decode attention over a 4-bit key-value cache, one new
// token per batch row: the call of ws_attention.cu on rows of 80 bytes.
//
// out_h = sum_j p_j v_j, p = softmax_j(q_h . k_j / sqrt(128)) over the slots
// 0 .. pos, k and v = s (code - 8) + z per slot and group of 32 dimensions, so
//   q . k = sum_g s_g (sum_d q_d (code_d - 8)) + z_g (sum_d q_d),
//   out   = sum_j (p_j s_j) (code_j - 8) + sum_j p_j z_j :
// the codes enter the products as exact small integers, a key's scale weighs
// each group's part of its score, and a value's scale joins the probability.
// The fp32 operands (q, and p s) enter as bf16 hi + lo pairs, their errors
// 2^-17.  Warp-level products (m16n8k16): a tile is 16 or 32 slots by 128
// dimensions for at most 8 heads, far below a tcgen05 tile, and its operands
// are made in registers.
//
// The tiles of 32 slots of all rows and heads, in fours, are cut into one equal
// run a resident CTA, whatever the rows' lengths; the CTA that shares a (row, head)
// with others leaves a partial result, and the last of each 16 and the last of
// those groups merge.  A warp streams its tiles through a ring of two stages
// (two bulk copies of 2560 bytes each).
//
// Bound by latency, with no unit full: expanding 4 bits to operands and carrying
// the scales takes about 800 instructions a warp and tile, each chain of them
// waits for its own, and registers leave 12 warps a SM (8 with 5 to 8 heads a
// group).  16 rows x 16384 slots x 8 heads (32 query heads; 257 MB): 59.9 us,
// 4.3 TB/s, 0.63 of the measured copy rate, issue 53% active, integer pipe 49%,
// DRAM 51%, tensor pipe 20%; with 64 query heads (the core for 8) 74.4 us, 3.5
// TB/s; 2 rows of 23462 and 11731 slots, 4 heads, 20.4 us with 32 query heads,
// 18.0 with 16.  What it took from 113 us (these and the figures below with the
// new rows read back, 1.4 us): nibbles masked in place and
// raised by one packed fma (no shift for every second one) 93 -> 80; products
// that start from nothing and two CTAs a SM without spills -> 73; for up to 4
// heads the operands changed over -> 67; lo terms by the mixed fma -> 63.4; runs
// cut between fours of tiles -> 61.7.
// Slower, not kept: keys as e4m3 (the masked nibbles are e4m3 numbers already,
// the sums came out exact; mixing the two product types cost more than the
// conversions) 90; nibbles as raw subnormal bf16 operands 72; four stages or
// three, 8 warps a CTA, 4 CTAs a SM.
#include <cfloat>
#include <cmath>
#include <mutex>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kQ4MaxG = 8;       // query heads per key-value head (half the MMA's 16 rows)
constexpr int kQ4MaxB = 1024;
constexpr int kQ4Tile = 32;      // slots per tile: four of the products' 8 columns
constexpr int kQ4Warps = 4;
constexpr int kQ4Threads = kQ4Warps * 32;
constexpr int kQ4Stages = 2;     // ring stages per warp
constexpr int kQ4StageBytes = 2 * kQ4Tile * kKvRow;  // keys, then values
constexpr int kQ4MaxCtas = 1024;
constexpr int kQ4Merge = 16;                         // partial results merged in one go
constexpr int kQ4Part = kKvDim + 4;                  // one partial result: acc[128], max, sum, two unused
constexpr int kQ4Ring = kQ4Warps * kQ4Stages * kQ4StageBytes;
// the running maximum follows the tile's only when that is 2^8 above it; it
// starts at the lowest number, below every finite score
constexpr float kQ4Lazy = 8.f;

struct AttnQ4Params {
  const float* q;      // [B][nh * 128]
  const float* k_new;  // [B][nkv * 128]
  const float* v_new;
  unsigned char* kc;   // [B][nkv][S][80]
  unsigned char* vc;
  const int* pos;      // [B]: slot of the new token, negative: none
  float* out_f32;
  uint16_t* out_bf16;
  int B, nh, nkv, S, G;
  float scale;         // log2(e) / sqrt(128)
  float* part;         // [CTAs][2][G][kQ4Part]
  unsigned* tick;      // [3][kQ4MaxCtas]
  int* err;
  unsigned long long timeout_ns;
};

// Tiles of a row and head in the count that the CTAs share out: a multiple of
// the warps, which take four tiles in the time of one, so that a run never ends
// among the four and short sequences get a CTA each.  Those past the last slot
// are empty.  Counting the filled ones only, four to a CTA at least: 12 rows of 3
// slots, 56/8 heads, 13.4 us against 7.2; 10 rows to 3190, 4/4, 15.4 against 14.2;
// 16 x 16384, 32/8, 63.4 against 61.7; one row of 1000, 12/2, 8.80 against 8.85.
__device__ __forceinline__ int q4_tiles(int pos, int S) {
  constexpr int kSlots = kQ4Tile * kQ4Warps;
  return pos < 0 || pos >= S ? 0 : (pos / kSlots + 1) * kQ4Warps;
}

// Two codes, nibble HI of byte 0 and of byte 2 of m, as bf16 f (code - 8) with
// f = 1/64 (HI 0) or 1/4 (HI 1).  Masked in place, a nibble is the bits of a
// number on the subnormal grid: code 2^-133 at bits 0..3 and, since the lowest
// normal binade has the same spacing, code 2^-129 at bits 4..7.  One packed fma
// by 2^127 brings it to f code and takes 8 f off, all exact; the queries and
// the results carry 1 / f.
template <int HI>
__device__ __forceinline__ uint32_t q4_pair(uint32_t m) {
  const uint32_t v = m & (HI ? 0x00f000f0u : 0x000f000fu);
  const uint32_t up = 0x7f007f00u, off = HI ? 0xc000c000u : 0xbe00be00u;  // 2^127; -2, -1/8
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(up), "r"(off));
  return r;
}
constexpr float kQ4Lo = 64.f, kQ4Hi = 4.f;

// d = A B: the product whose sum starts here, with no registers to clear first
__device__ __forceinline__ void q4_mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// v = hi + lo, hi = bf16(v), lo = bf16(v - hi), two values a word
__device__ __forceinline__ void q4_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - bf16lo(hi), b - bf16hi(hi));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// bf16 halves of a word in fp32 arithmetic by the mixed fma (one exact product,
// one rounding): v + c x, x the low or the high half, c a bf16 twice in a word.
__device__ __forceinline__ float q4_fma_low(uint32_t u, uint32_t c, float v) {
  float r;
  asm("{\n\t.reg .b16 l, h, o, p;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {o, p}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, o, %3;\n\t}" : "=f"(r) : "r"(u), "r"(c), "f"(v));
  return r;
}
__device__ __forceinline__ float q4_fma_high(uint32_t u, uint32_t c, float v) {
  float r;
  asm("{\n\t.reg .b16 l, h, o, p;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {o, p}, %2;\n\t"
      "fma.rn.f32.bf16 %0, h, p, %3;\n\t}" : "=f"(r) : "r"(u), "r"(c), "f"(v));
  return r;
}

__device__ __forceinline__ float q4_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ unsigned q4_ticket(unsigned* p) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// Where a warp's next tile lies: tile x of the CTA's range (counted from the
// range's start) is tile x - at of (row b, head g), which has nt of them.
struct Q4Cursor {
  int b, g, at, nt, pos;
};

__device__ __forceinline__ void q4_seek(const AttnQ4Params& a, Q4Cursor& c, int x) {
  while (x >= c.at + c.nt) {
    c.at += c.nt;
    if (++c.g == a.nkv) {
      c.g = 0;
      do {
        c.pos = a.pos[++c.b];
        c.nt = q4_tiles(c.pos, a.S);
      } while (c.nt == 0);
    }
  }
}

// The sequence's last tile: its n cached rows by bulk copies, then the new row,
// quantised, to its place there and in the cache, and zeros for the rows behind
// it (whatever the cache holds there).
__device__ __noinline__ void q4_stage_last(const AttnQ4Params& a, size_t seg, int n,
                                           unsigned char* kr, unsigned char* vr, unsigned char* st,
                                           uint64_t* bar, int lane, uint64_t pol) {
  if (lane == 0) {
    mbar_arrive_expect_tx(bar, 2u * n * kKvRow);
    if (n > 0) {
      bulk_copy_g2s(st, kr, n * kKvRow, bar, pol);
      bulk_copy_g2s(st + kQ4Tile * kKvRow, vr, n * kKvRow, bar, pol);
    }
  }
  const bool keys = lane < 16;
  float x[8];
  load8<DT_F32>((keys ? a.k_new : a.v_new) + seg * kKvDim + (lane & 15) * 8, x);
  uint32_t sz;
  const uint32_t w = quantize8(x, sz);
  const KvLane at(keys);
  put_row(st + ((keys ? 0 : kQ4Tile) + n) * kKvRow, w, sz, at);
  put_row((keys ? kr : vr) + n * kKvRow, w, sz, at);
  uint4* z = reinterpret_cast<uint4*>(st + (keys ? 0 : kQ4Tile * kKvRow));
  for (int i = (n + 1) * 5 + (lane & 15); i < kQ4Tile * 5; i += 16) z[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
}

// Merge of n partial results (entry i at rest + i * step, entry 0 at first) for
// head h by one warp, four dimensions a lane: M = max m, L = sum 2^(m - M) l,
// O = sum 2^(m - M) acc.  A batch's loads are all in flight together.
__device__ __forceinline__ void q4_merge(const float* first, const float* rest, size_t step, int n,
                                         int h, int lane, float4& O, float& M, float& L) {
  O = make_float4(0.f, 0.f, 0.f, 0.f);
  M = -FLT_MAX;
  L = 0.f;
  for (int i0 = 0; i0 < n; i0 += kQ4Merge) {
    float4 x[kQ4Merge];
#pragma unroll
    for (int j = 0; j < kQ4Merge; ++j) {
      const int i = min(i0 + j, n - 1);
      const float* e = (i == 0 ? first : rest + i * step) + (size_t)h * kQ4Part;
      x[j] = __ldcg(reinterpret_cast<const float4*>(e) + lane);
    }
    const int i = min(i0 + (lane & (kQ4Merge - 1)), n - 1);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(
        (i == 0 ? first : rest + i * step) + (size_t)h * kQ4Part + kKvDim));
    float mx = ml.x;
#pragma unroll
    for (int o = kQ4Merge / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx = fmaxf(mx, M);
    const float f = q4_exp2(M - mx);
    M = mx;
    float w = i0 + (lane & (kQ4Merge - 1)) < n ? q4_exp2(ml.x - mx) : 0.f;
    float lw = w * ml.y;
    if (i0 + (lane & (kQ4Merge - 1)) >= n) lw = 0.f;
#pragma unroll
    for (int o = kQ4Merge / 2; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    L = fmaf(L, f, lw);
    O.x *= f, O.y *= f, O.z *= f, O.w *= f;
#pragma unroll
    for (int j = 0; j < kQ4Merge; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      if (i0 + j < n) {
        O.x = fmaf(wj, x[j].x, O.x);
        O.y = fmaf(wj, x[j].y, O.y);
        O.z = fmaf(wj, x[j].z, O.z);
        O.w = fmaf(wj, x[j].w, O.w);
      }
    }
  }
}

// out = O / L, four dimensions a lane
__device__ __forceinline__ void q4_write(const AttnQ4Params& a, int b, int g, int lane, int h,
                                         float4 O, float L) {
  const size_t at = ((size_t)b * a.nh + (size_t)g * a.G + h) * kKvDim + 4 * lane;
  O.x /= L, O.y /= L, O.z /= L, O.w /= L;
  if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + at) = O;
  if (a.out_bf16) {
    const __nv_bfloat162 u = __floats2bfloat162_rn(O.x, O.y), v = __floats2bfloat162_rn(O.z, O.w);
    *reinterpret_cast<uint2*>(a.out_bf16 + at) = make_uint2(
        *reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
  }
}

__device__ __forceinline__ void q4_put(float* e, int lane, float4 O, float M, float L) {
  reinterpret_cast<float4*>(e)[lane] = O;
  if (lane == 0) *reinterpret_cast<float2*>(e + kKvDim) = make_float2(M, L);
}

// The two products of a warp and what it accumulates, for up to 8 heads a group:
// heads are the rows of the products, their hi terms in rows 0..7 and their lo
// terms in rows 8..15; the columns are slots, then dimensions.
struct Q4Wide {
  static constexpr int kHeads = 8;
  static constexpr int kCtas = 2;  // a SM: 245 registers; three (168, spilled) took 78 us where this takes 73.5
  struct Shared {
    uint4 qfrag[8][32];
    float qsum[kHeads][4];
  };
  float o[16][4], m;
  float zo[4];  // sum p z, column = group (the columns 4 .. 7 repeat them)
  float2 l;
  uint32_t qz[2], zmask;

  __device__ __forceinline__ void begin(const AttnQ4Params& a, int b, int g0, Shared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane >> 2, rt = lane & 3;
    // the queries as the first product's A operand, in shared memory (held in
    // registers they cost a CTA a SM its place): head rg in rows rg (hi terms)
    // and rg + 8 (lo terms); lane rt of a quad holds dimensions 32 g + 8 rt ..
    // + 7, in the order of the key row's nibbles; warp g makes group g's.  qz:
    // their sums per group, the operand against the zeros (k = group)
    {
      static_assert(kQ4Warps == 4, "a warp per group");
      const float* qr = a.q + ((size_t)b * a.nh + (size_t)g0 * a.G + (rg < a.G ? rg : 0)) * kKvDim;
      float v[8], sum = 0.f;
      load8<DT_F32>(qr + 32 * warp + 8 * rt, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = rg < a.G ? v[i] * a.scale : 0.f;
        sum += v[i];
        v[i] *= i & 1 ? kQ4Hi : kQ4Lo;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (rt == 0) sh.qsum[rg][warp] = sum;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint4 f;
        q4_split(v[2 * k], v[2 * k + 4], f.x, f.y);
        q4_split(v[2 * k + 1], v[2 * k + 5], f.z, f.w);
        sh.qfrag[2 * warp + k][lane] = f;
      }
    }
    __syncthreads();
    {
      const float2 z = rt < 2 ? *reinterpret_cast<const float2*>(&sh.qsum[rg][2 * rt]) : make_float2(0.f, 0.f);
      q4_split(z.x, z.y, qz[0], qz[1]);
    }
    zmask = rt < 2 ? 0xffffffffu : 0u;
    m = -FLT_MAX;
    l = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) zo[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }

  __device__ __forceinline__ void tile(const unsigned char* st, int slot0, int pos, const Shared& sh) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, rt = lane & 3;
    // scores: head rg, slots 8 n + 2 rt + e
    float2 s[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint4 kw[2], ks[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const unsigned char* kr = st + (16 * u + 8 * n + rg) * kKvRow;
        kw[n] = *reinterpret_cast<const uint4*>(kr + 16 * rt);
        const uint2 kz = *reinterpret_cast<const uint2*>(kr + kKvCodes + 8 * (rt & 1));
        const unsigned char* ksp = st + (16 * u + 8 * n + 2 * rt) * kKvRow + kKvCodes;
        ks[n][0] = *reinterpret_cast<const uint4*>(ksp);
        ks[n][1] = *reinterpret_cast<const uint4*>(ksp + kKvRow);
        float cz[4];
        q4_mma0(cz, qz[0], qz[1], 0u, 0u, __byte_perm(kz.x, kz.y, 0x7632) & zmask, 0u);
        s[2 * u + n] = add2(make_float2(cz[0], cz[1]), make_float2(cz[2], cz[3]));
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 q0 = sh.qfrag[2 * g][lane], q1 = sh.qfrag[2 * g + 1][lane];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(&kw[n])[g], w8 = w >> 8;
          float c[4];
          q4_mma0(c, q0.x, q0.y, q0.z, q0.w, q4_pair<0>(w), q4_pair<1>(w));
          mma_bf16_16816(c, q1.x, q1.y, q1.z, q1.w, q4_pair<0>(w8), q4_pair<1>(w8));
          s[2 * u + n] = fma2(make_float2(bf16lo(reinterpret_cast<const uint32_t*>(&ks[n][0])[g]),
                                          bf16lo(reinterpret_cast<const uint32_t*>(&ks[n][1])[g])),
                              add2(make_float2(c[0], c[1]), make_float2(c[2], c[3])),
                              s[2 * u + n]);
        }
      }
    }
    if (slot0 + kQ4Tile > pos + 1) {
      const int slot = slot0 + 2 * rt;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (slot + 8 * n > pos) s[n].x = -INFINITY;
        if (slot + 8 * n + 1 > pos) s[n].y = -INFINITY;
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(s[0].x, s[0].y), fmaxf(s[1].x, s[1].y)),
                     fmaxf(fmaxf(s[2].x, s[2].y), fmaxf(s[3].x, s[3].y)));
    if (__any_sync(0xffffffffu, mx > m + kQ4Lazy)) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m, mx), f = q4_exp2(m - mn);
      m = mn;
      l.x *= f, l.y *= f;
#pragma unroll
      for (int e = 0; e < 4; ++e) zo[e] *= f;
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= f;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      s[n].x = q4_exp2(s[n].x - m);
      s[n].y = q4_exp2(s[n].y - m);
      l = add2(l, s[n]);
    }
    // output: the probabilities times each slot's scale enter as the A
    // operand (hi rows and lo rows again), the codes as B: column rg is
    // dimension 32 g + 4 rg + i
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const unsigned char* sv = st + (kQ4Tile + 16 * u + 2 * rt) * kKvRow;
      uint2 vw[2][2];
      uint4 vs[2][2];
      uint32_t ph[2], pl[2], bz[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned char* r = sv + (8 * n + e) * kKvRow;
          vw[n][e] = *reinterpret_cast<const uint2*>(r + 8 * rg);
          vs[n][e] = *reinterpret_cast<const uint4*>(r + kKvCodes);
          z[e] = *reinterpret_cast<const uint32_t*>(r + kKvCodes + 4 * (rg & 3));
        }
        bz[n] = __byte_perm(z[0], z[1], 0x7632);
        q4_split(s[2 * u + n].x, s[2 * u + n].y, ph[n], pl[n]);
      }
      mma_bf16_16816(zo, ph[0], pl[0], ph[1], pl[1], bz[0], bz[1]);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t ah[2], al[2], m0[2], m1[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t z0 = reinterpret_cast<const uint32_t*>(&vs[n][0])[g];
          const uint32_t z1 = reinterpret_cast<const uint32_t*>(&vs[n][1])[g];
          const float2 ps = mul2(s[2 * u + n], make_float2(bf16lo(z0), bf16lo(z1)));
          q4_split(ps.x, ps.y, ah[n], al[n]);
          const uint32_t w0 = g < 2 ? vw[n][0].x : vw[n][0].y, w1 = g < 2 ? vw[n][1].x : vw[n][1].y;
          m0[n] = __byte_perm(w0, w1, g & 1 ? 0x0602 : 0x0400);
          m1[n] = __byte_perm(w0, w1, g & 1 ? 0x0703 : 0x0501);
        }
        mma_bf16_16816(o[4 * g], ah[0], al[0], ah[1], al[1], q4_pair<0>(m0[0]), q4_pair<0>(m0[1]));
        mma_bf16_16816(o[4 * g + 1], ah[0], al[0], ah[1], al[1], q4_pair<1>(m0[0]), q4_pair<1>(m0[1]));
        mma_bf16_16816(o[4 * g + 2], ah[0], al[0], ah[1], al[1], q4_pair<0>(m1[0]), q4_pair<0>(m1[1]));
        mma_bf16_16816(o[4 * g + 3], ah[0], al[0], ah[1], al[1], q4_pair<1>(m1[0]), q4_pair<1>(m1[1]));
      }
    }
  }

  // this warp's result: cm, cl [heads], comb [heads][128]
  __device__ __forceinline__ void end(int G, float* cm, float* cl, float* comb) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, rt = lane & 3;
    // dimensions 32 g + 8 rt .. + 7
    float lsum = l.x + l.y, zs[4];
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 1);
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      zs[g] = __shfl_sync(0xffffffffu, zo[g & 1] + zo[2 + (g & 1)], (lane & 28) + (g >> 1));
    if (rt == 0) cm[rg] = m, cl[rg] = lsum;
    float* cw = comb + rg * kKvDim + 8 * rt;
    if (rg < G) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(cw + 32 * g + 4 * e) =
              make_float4(fmaf(o[4 * g + 0][e] + o[4 * g + 0][2 + e], kQ4Lo, zs[g]),
                          fmaf(o[4 * g + 1][e] + o[4 * g + 1][2 + e], kQ4Hi, zs[g]),
                          fmaf(o[4 * g + 2][e] + o[4 * g + 2][2 + e], kQ4Lo, zs[g]),
                          fmaf(o[4 * g + 3][e] + o[4 * g + 3][2 + e], kQ4Hi, zs[g]));
    }
  }
};

__device__ __forceinline__ uint32_t q4_transpose(uint32_t a) {  // an 8x8 matrix of 16-bit values
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The same for up to 4 heads a group, with the operands changed over: the codes
// are the rows (16 slots, then 16 dimensions), the columns the heads' hi terms
// and, from 4 on, their lo terms.  Half as many products and accumulators, so
// that more CTAs fit; the probabilities pass from rows to columns by a
// transposition between the two products.
struct Q4Narrow {
  static constexpr int kHeads = 4;
  static constexpr int kCtas = 3;  // a SM: 62.8 us, two or four 64 and 67 (the latter spilled)
  struct Shared {};
  // lane: heads 2 (rt & 1) + e; o[2 g + i / 2]: dimensions 32 g + 4 rg + i, hi
  // terms for rt < 2, lo terms for the others
  float o[8][4], zo[4][2], m[2], l[2];
  uint32_t qb[8][2], qz;

  __device__ __forceinline__ void begin(const AttnQ4Params& a, int b, int g0, Shared&) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, rt = lane & 3;
    const int h = rg & 3;  // column rg: head h's hi term, or its lo term
    const float* qr = a.q + ((size_t)b * a.nh + (size_t)g0 * a.G + (h < a.G ? h : 0)) * kKvDim;
    float sums[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8], sum = 0.f;
      load8<DT_F32>(qr + 32 * g + 8 * rt, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = h < a.G ? v[i] * a.scale : 0.f;
        sum += v[i];
        v[i] *= i & 1 ? kQ4Hi : kQ4Lo;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sums[g] = sum;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t hi, lo;
        q4_split(v[2 * k], v[2 * k + 4], hi, lo);
        qb[2 * g + k][0] = rg < 4 ? hi : lo;
        q4_split(v[2 * k + 1], v[2 * k + 5], hi, lo);
        qb[2 * g + k][1] = rg < 4 ? hi : lo;
      }
    }
    uint32_t hi, lo;
    q4_split(rt == 0 ? sums[0] : rt == 1 ? sums[2] : 0.f, rt == 0 ? sums[1] : rt == 1 ? sums[3] : 0.f,
             hi, lo);
    qz = rg < 4 ? hi : lo;
#pragma unroll
    for (int e = 0; e < 2; ++e) m[e] = -FLT_MAX, l[e] = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) zo[g][0] = zo[g][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }

  __device__ __forceinline__ void tile(const unsigned char* st, int slot0, int pos, const Shared&) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, rt = lane & 3;
    const uint32_t zmask = rt < 2 ? 0xffffffffu : 0u, minus = rt < 2 ? 0x80008000u : 0xbf80bf80u;
    // scores: slots 16 u + 8 n + rg, heads 2 (rt & 1) + e
    float s[2][2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint4 kw[2], ks[2];
      uint32_t z[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const unsigned char* r = st + (16 * u + 8 * n + rg) * kKvRow;
        kw[n] = *reinterpret_cast<const uint4*>(r + 16 * rt);
        ks[n] = *reinterpret_cast<const uint4*>(r + kKvCodes);
        z[n] = (rt & 1 ? __byte_perm(ks[n].z, ks[n].w, 0x7632) : __byte_perm(ks[n].x, ks[n].y, 0x7632)) &
               zmask;
      }
      float sum[4];
      q4_mma0(sum, z[0], z[1], 0u, 0u, qz, 0u);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kw[0])[g];
        const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kw[1])[g];
        float c[4];
        q4_mma0(c, q4_pair<0>(w0), q4_pair<0>(w1), q4_pair<1>(w0), q4_pair<1>(w1), qb[2 * g][0], qb[2 * g][1]);
        mma_bf16_16816(c, q4_pair<0>(w0 >> 8), q4_pair<0>(w1 >> 8), q4_pair<1>(w0 >> 8),
                       q4_pair<1>(w1 >> 8), qb[2 * g + 1][0], qb[2 * g + 1][1]);
        const float s0 = bf16lo(reinterpret_cast<const uint32_t*>(&ks[0])[g]);
        const float s1 = bf16lo(reinterpret_cast<const uint32_t*>(&ks[1])[g]);
        sum[0] = fmaf(s0, c[0], sum[0]);
        sum[1] = fmaf(s0, c[1], sum[1]);
        sum[2] = fmaf(s1, c[2], sum[2]);
        sum[3] = fmaf(s1, c[3], sum[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)  // hi and lo terms
        s[u][i >> 1][i & 1] = sum[i] + __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    if (slot0 + kQ4Tile > pos + 1) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (slot0 + 16 * u + 8 * n + rg > pos) s[u][n][0] = s[u][n][1] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) mx[e] = fmaxf(fmaxf(s[0][0][e], s[0][1][e]), fmaxf(s[1][0][e], s[1][1][e]));
    if (__any_sync(0xffffffffu, mx[0] > m[0] + kQ4Lazy || mx[1] > m[1] + kQ4Lazy)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], i));
        const float mn = fmaxf(m[e], mx[e]), f = q4_exp2(m[e] - mn);
        m[e] = mn;
        l[e] *= f;
#pragma unroll
        for (int g = 0; g < 4; ++g) zo[g][e] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][e] *= f, o[i][2 + e] *= f;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[u][n][e] = q4_exp2(s[u][n][e] - m[e]);
          l[e] += s[u][n][e];
        }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const unsigned char* sv = st + (kQ4Tile + 16 * u) * kKvRow;
      uint2 vw[2][2];
      uint4 vs[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          vw[n][e] = *reinterpret_cast<const uint2*>(sv + (8 * n + 2 * rt + e) * kKvRow + 8 * rg);
        vs[n] = *reinterpret_cast<const uint4*>(sv + (8 * n + rg) * kKvRow + kKvCodes);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t pb[2], m0[2], m1[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t sz = reinterpret_cast<const uint32_t*>(&vs[n])[g];
          const float sc = bf16lo(sz), z = bf16hi(sz);
          // hi terms in the lanes rt < 2; the others take them off first
          const float p0 = s[u][n][0] * sc, p1 = s[u][n][1] * sc;
          const __nv_bfloat162 hi = __floats2bfloat162_rn(p0, p1);
          const uint32_t h = *reinterpret_cast<const uint32_t*>(&hi);
          const __nv_bfloat162 part =
              __floats2bfloat162_rn(q4_fma_low(h, minus, p0), q4_fma_high(h, minus, p1));
          pb[n] = q4_transpose(*reinterpret_cast<const uint32_t*>(&part));
          zo[g][0] = fmaf(s[u][n][0], z, zo[g][0]);
          zo[g][1] = fmaf(s[u][n][1], z, zo[g][1]);
          const uint32_t w0 = g < 2 ? vw[n][0].x : vw[n][0].y, w1 = g < 2 ? vw[n][1].x : vw[n][1].y;
          m0[n] = __byte_perm(w0, w1, g & 1 ? 0x0602 : 0x0400);
          m1[n] = __byte_perm(w0, w1, g & 1 ? 0x0703 : 0x0501);
        }
        mma_bf16_16816(o[2 * g], q4_pair<0>(m0[0]), q4_pair<1>(m0[0]), q4_pair<0>(m0[1]),
                       q4_pair<1>(m0[1]), pb[0], pb[1]);
        mma_bf16_16816(o[2 * g + 1], q4_pair<0>(m1[0]), q4_pair<1>(m1[0]), q4_pair<0>(m1[1]),
                       q4_pair<1>(m1[1]), pb[0], pb[1]);
      }
    }
  }

  __device__ __forceinline__ void end(int G, float* cm, float* cl, float* comb) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, rt = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], i);
#pragma unroll
        for (int g = 0; g < 4; ++g) zo[g][e] += __shfl_xor_sync(0xffffffffu, zo[g][e], i);
      }
      if (rg == 0 && rt < 2) cm[2 * rt + e] = m[e], cl[2 * rt + e] = l[e];
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = o[2 * g + (i >> 1)][2 * (i & 1) + e];
          v[i] = fmaf(x + __shfl_xor_sync(0xffffffffu, x, 2), i & 1 ? kQ4Hi : kQ4Lo, zo[g][e]);
        }
        if (rt < 2 && 2 * rt + e < G)
          *reinterpret_cast<float4*>(comb + (2 * rt + e) * kKvDim + 32 * g + 4 * rg) =
              make_float4(v[0], v[1], v[2], v[3]);
      }
  }
};

template <class Core>
__global__ void __launch_bounds__(kQ4Threads, Core::kCtas)
    k_decode_attention_q4(const __grid_constant__ AttnQ4Params a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kQ4Warps][kQ4Stages];
  __shared__ float cm[kQ4Warps][Core::kHeads], cl[kQ4Warps][Core::kHeads];
  __shared__ typename Core::Shared shared;
  __shared__ int last;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, G = a.G;

  pdl_wait();
  // the tiles of all rows and heads, cut into as many equal runs as there are
  // CTAs; every warp finds the run's place by itself
  // (fewer than 2^31 of them: the caller's bound of 2^30, and three empty ones for
  // each of 1024 * 65535 rows and heads at most)
  int total = 0, p0 = -1;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int p = b0 + lane < a.B ? a.pos[b0 + lane] : -1;
    if (b0 == 0) p0 = p;
    if (p >= a.S && blockIdx.x == 0 && warp == 0) atomicExch(a.err, kDerrBadSlot);
    total += q4_tiles(p, a.S);
  }
  total = __reduce_add_sync(0xffffffffu, total) * a.nkv;
  const int per = ((int)((total + gridDim.x - 1) / gridDim.x) + kQ4Warps - 1) / kQ4Warps * kQ4Warps;
  const int start = blockIdx.x * per, run = min(per, total - start);
  if (run <= 0) return;
  Q4Cursor cur;
  {
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int p = b0 == 0 ? p0 : b0 + lane < a.B ? a.pos[b0 + lane] : -1;
      const int nt = q4_tiles(p, a.S);
      int sum = nt * a.nkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > start);
      if (hit) {
        const int l = __ffs(hit) - 1;
        cur.b = b0 + l;
        cur.pos = __shfl_sync(0xffffffffu, p, l);
        cur.nt = __shfl_sync(0xffffffffu, nt, l);
        const int in = start - before - (__shfl_sync(0xffffffffu, sum, l) - cur.nt * a.nkv);
        cur.g = in / cur.nt;
        cur.at = -(in % cur.nt);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  unsigned char* ring = smem + warp * kQ4Stages * kQ4StageBytes;
  float* comb = reinterpret_cast<float*>(smem + kQ4Ring);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kQ4Stages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const uint64_t pol = l2_policy_evict_first();
  // the next tile to stage: its segment, and its rows' addresses there
  Q4Cursor ic = cur;
  int xi = warp, ni = 0, nc = 0;
  unsigned char *ikr = nullptr, *ivr = nullptr;
  int ilast = -1;  // the last tile of the segment, counted as x
  auto issue = [&]() {
    for (; xi < run; xi += kQ4Warps) {
      if (xi > ilast) {
        q4_seek(a, ic, xi);
        const int tile = xi - ic.at;
        if (tile > ic.pos / kQ4Tile) continue;  // empty: on to the next row or head
        ilast = ic.at + ic.pos / kQ4Tile;
        const size_t row = ((size_t)ic.b * a.nkv + ic.g) * a.S + (size_t)tile * kQ4Tile;
        ikr = a.kc + row * kKvRow;
        ivr = a.vc + row * kKvRow;
      }
      unsigned char* st = ring + ni * kQ4StageBytes;
      uint64_t* bar = &full[warp][ni];
      fence_proxy_async_smem();  // what the lanes read and wrote there before the copies
      __syncwarp();
      if (xi == ilast) {
        q4_stage_last(a, (size_t)ic.b * a.nkv + ic.g, ic.pos - (xi - ic.at) * kQ4Tile, ikr, ivr, st,
                      bar, lane, pol);
      } else if (lane == 0) {
        mbar_arrive_expect_tx(bar, kQ4StageBytes);
        bulk_copy_g2s(st, ikr, kQ4Tile * kKvRow, bar, pol);
        bulk_copy_g2s(st + kQ4Tile * kKvRow, ivr, kQ4Tile * kKvRow, bar, pol);
      }
      ni ^= 1;
      ikr += kQ4Warps * kQ4Tile * kKvRow;
      ivr += kQ4Warps * kQ4Tile * kKvRow;
      xi += kQ4Warps;
      return;
    }
  };
  static_assert(kQ4Stages == 2, "stage indices flip");
  issue();
  issue();

  int x = warp, x0 = 0;
  uint32_t par = 0;
  bool abort = false;
  while (x0 < run) {  // one (row, head) at a time
    q4_seek(a, cur, x0);
    const int x1 = min(run, cur.at + cur.nt);
    Core core;
    core.begin(a, cur.b, cur.g, shared);
    const int xe = min(x1, cur.at + cur.pos / kQ4Tile + 1);
    for (; x < xe; x += kQ4Warps) {
      const unsigned char* st = ring + nc * kQ4StageBytes;
      bool ok = abort || mbar_try_wait(&full[warp][nc], par);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = ok || mbar_wait_bounded(&full[warp][nc], par, a.timeout_ns);
        if (__any_sync(0xffffffffu, !ok)) {
          abort = true;  // nothing more is issued; what is under way ends first
          if (lane == 0) atomicExch(a.err, (int)DERR_TIMEOUT);
          // (both stages when the next to fill is the one waited for, else that one)
          for (int i = 0; i < 2 - (ni ^ nc); ++i)
            mbar_wait_bounded(&full[warp][nc ^ i], par ^ (nc & i), a.timeout_ns);
        }
      }
      if (!abort) core.tile(st, (x - cur.at) * kQ4Tile, cur.pos, shared);
      nc ^= 1;
      par ^= nc == 0;
      if (!abort) issue();
    }
    if (x < x1) x += kQ4Warps;  // an empty tile ends the row and head

    // (let go any earlier, the next kernel's CTAs take from this one's loads: 65.2
    // against 63.4 us over 16 x 16384 slots)
    if (x1 >= run) pdl_launch_dependents();
    // the four warps' results, then this CTA's
    core.end(G, cm[warp], cl[warp], comb + (size_t)warp * Core::kHeads * kKvDim);
    __syncthreads();
    const int seg0 = start + cur.at;  // the segment's first tile among all
    const int c0 = seg0 / per, n = (seg0 + cur.nt - 1) / per - c0 + 1;
    const int me = blockIdx.x - c0;
    const size_t slot = (size_t)2 * G * kQ4Part;  // floats of a CTA's two partials
    float* mine = a.part + (size_t)blockIdx.x * slot + (me == 0 ? slot / 2 : 0);
    for (int h = warp; h < G; h += kQ4Warps) {
      float M = cm[0][h], L = 0.f;
#pragma unroll
      for (int w = 1; w < kQ4Warps; ++w) M = fmaxf(M, cm[w][h]);
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kQ4Warps; ++w) {
        const float f = q4_exp2(cm[w][h] - M);
        const float4 v = reinterpret_cast<const float4*>(comb + ((size_t)w * Core::kHeads + h) * kKvDim)[lane];
        O.x = fmaf(f, v.x, O.x);
        O.y = fmaf(f, v.y, O.y);
        O.z = fmaf(f, v.z, O.z);
        O.w = fmaf(f, v.w, O.w);
        L = fmaf(f, cl[w][h], L);
      }
      if (n == 1) q4_write(a, cur.b, cur.g, lane, h, O, L);
      else q4_put(mine + h * kQ4Part, lane, O, M, L);
    }
    if (n > 1) {
      // the last CTA of each 16 merges them into the first one's place, the
      // last of the groups merges the groups
      const int grp = me / kQ4Merge, in = min(kQ4Merge, n - grp * kQ4Merge);
      const int groups = (n + kQ4Merge - 1) / kQ4Merge;
      float* base = a.part + (size_t)c0 * slot;  // CTA c0's entry is its second one
      float* first = base + (grp ? (size_t)grp * kQ4Merge * slot : slot / 2);
      __syncthreads();
      if (t == 0) {
        unsigned* tk = a.tick + (grp ? kQ4MaxCtas : 0) + c0 + grp * kQ4Merge;
        last = q4_ticket(tk) == (unsigned)(in - 1);
        if (last) *tk = 0;
      }
      __syncthreads();
      if (last) {
        // head h is the same warp's from the partials to the result
        for (int h = warp; h < G; h += kQ4Warps) {
          float4 O;
          float M, L;
          q4_merge(first, base + (size_t)grp * kQ4Merge * slot, slot, in, h, lane, O, M, L);
          if (groups == 1) {
            q4_write(a, cur.b, cur.g, lane, h, O, L);
          } else {
            __syncwarp();  // every lane has read the first entry
            q4_put(first + h * kQ4Part, lane, O, M, L);
          }
        }
        if (groups > 1) {
          __syncthreads();
          if (t == 0) {
            unsigned* tk = a.tick + 2 * kQ4MaxCtas + c0;
            last = q4_ticket(tk) == (unsigned)(groups - 1);
            if (last) *tk = 0;
          }
          __syncthreads();
          if (last)
            for (int h = warp; h < G; h += kQ4Warps) {
              float4 O;
              float M, L;
              q4_merge(base + slot / 2, base, kQ4Merge * slot, groups, h, lane, O, M, L);
              q4_write(a, cur.b, cur.g, lane, h, O, L);
            }
        }
      }
    }
    __syncthreads();  // cm, cl and comb are free again
    x0 = x1;
  }
}

template <class Core>
constexpr int kQ4Smem = kQ4Ring + kQ4Warps * Core::kHeads * kKvDim * 4;

// Resident CTAs of the device: the grid, set up once per device.
template <class Core>
static int q4_grid(cudaError_t* err) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static int grid[kMaxDev] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDev) {
    *err = e != cudaSuccess ? e : cudaErrorInvalidDevice;
    return 0;
  }
  std::lock_guard<std::mutex> lk(mu);
  if (!grid[dev]) {
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_decode_attention_q4<Core>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kQ4Smem<Core>);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_decode_attention_q4<Core>,
                                                        kQ4Threads, kQ4Smem<Core>);
    if (e != cudaSuccess || per_sm < 1) {
      *err = e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
      return 0;
    }
    grid[dev] = sms * per_sm < kQ4MaxCtas ? sms * per_sm : kQ4MaxCtas;
  }
  return grid[dev];
}

template <class Core>
static cudaError_t q4_launch(const AttnQ4Params& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const int grid = q4_grid<Core>(&e);
  if (!grid) return e;
  e = launch_serving(k_decode_attention_q4<Core>, dim3(grid), kQ4Threads, kQ4Smem<Core>, stream, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

static size_t q4_workspace(int nh, int nkv) {
  return 3 * kQ4MaxCtas * 4 + (size_t)kQ4MaxCtas * 2 * (nh / nkv) * kQ4Part * 4;
}

static bool q4_shape_ok(int B, int nh, int nkv, int d, int S) {
  return B >= 1 && B <= kQ4MaxB && nkv >= 1 && nkv <= 65535 && nh >= 1 && nh % nkv == 0 &&
         nh / nkv <= kQ4MaxG && d == kKvDim && S >= 1 &&
         (long long)B * nkv * (S / kQ4Tile + 1) < (1ll << 30);
}

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_attention_q4_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim,
                                       int s_max) {
  if (!q4_shape_ok(B, n_heads, n_kv_heads, head_dim, s_max)) return 0;
  return q4_workspace(n_heads, n_kv_heads);
}

ws_status ws_decode_attention_q4(const float *q, const float *k_new, const float *v_new,
                                 void *k_cache, void *v_cache, const int32_t *pos, float *out_f32,
                                 void *out_bf16, int B, int n_heads, int n_kv_heads, int head_dim,
                                 int s_max, void *workspace, size_t workspace_bytes,
                                 ws_stream_t stream) {
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !pos || (!out_f32 && !out_bf16) ||
      !workspace) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if (!q4_shape_ok(B, n_heads, n_kv_heads, head_dim, s_max)) {
    set_error("4-bit decode attention: B 1..%d, head_dim %d, n_heads 1 to %d times n_kv_heads, "
              "s_max at least 1, fewer than 2^30 tiles of 32 slots", kQ4MaxB, kKvDim, kQ4MaxG);
    return WS_ERR_SHAPE;
  }
  const void* al[] = {q, k_new, v_new, k_cache, v_cache, workspace, out_f32, out_bf16};
  for (const void* p : al)
    if ((uintptr_t)p & 15u) {
      set_error("4-bit decode attention: device pointers must be 16-byte aligned");
      return WS_ERR_ALIGN;
    }
  const size_t need = ws_attention_q4_workspace_bytes(B, n_heads, n_kv_heads, head_dim, s_max);
  if (workspace_bytes < need) {
    set_error("workspace too small: need %zu bytes, got %zu", need, workspace_bytes);
    return WS_ERR_ARG;
  }
  AttnQ4Params a = {};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.kc = static_cast<unsigned char*>(k_cache);
  a.vc = static_cast<unsigned char*>(v_cache);
  a.pos = pos;
  a.B = B;
  a.out_f32 = out_f32;
  a.out_bf16 = static_cast<uint16_t*>(out_bf16);
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.S = s_max;
  a.G = n_heads / n_kv_heads;
  a.scale = (float)(1.4426950408889634 / sqrt((double)kKvDim));
  a.tick = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(a.tick + 3 * kQ4MaxCtas);
  a.timeout_ns = tuning().timeout_ns;
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  const cudaError_t e = a.G <= Q4Narrow::kHeads ? q4_launch<Q4Narrow>(a, (cudaStream_t)stream)
                                                : q4_launch<Q4Wide>(a, (cudaStream_t)stream);
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
