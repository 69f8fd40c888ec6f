// ws_attention_paged.cu -- decode attention over a paged key-value cache, one
// new token per batch row: slot j of a sequence is slot j % ps of the page that
// entry j / ps of its table row names.
//
// out_h = sum_j p_j v_j, p = softmax_j(q_h . k_j / sqrt(128)), j = 0 .. pos; one
// pass with a running maximum m and sum l in log2 units: p_j = 2^(c s_j - m).
// A unit is 16 slots of one key-value head: both products are warp-level
// m16n8k16 with the cached rows as the 16-row operand, the heads (up to 8) as
// the columns: S = K q, O^T = V^T P.  fp32 queries enter as the terms of the
// cache's type that they take (three in bf16, two in fp16: relative error 2^-24 and
// 2^-22), so that the log-sum-exp is as good as fp32; the probabilities as hi + lo pairs
// (2^-17, 2^-22), as in the decode attention over contiguous caches: bf16 outputs before their
// rounding (2^-9) are off by 2e-6 of themselves (root mean square, rows of 2111).  A third bf16
// term was built: 3e-7, half as many value products again, 0.4 to 1.1% of the time of the batches
// below.
//
// A unit never crosses a page (page sizes are multiples of 16), so one tiled
// bulk copy brings its 16 keys and one its 16 values, as two halves of 64
// dimensions in the 128-byte swizzle that the ldmatrix reads want.  Each warp
// streams its own units through its own ring; the table's entries are read 32
// units ahead, a lane each.  All units of all rows and heads are cut into one
// equal run a resident CTA, whatever the rows' lengths; a CTA that shares a
// (row, head) with others leaves a partial result, and the last of them merges (of
// more than 48: the last of each 16, then the last of those groups).
//
// Bound by DRAM where the cache is long: 16 rows to 32768 slots, 32/8 heads, 239 us,
// 6.9 TB/s read, the copy rate.  Short and ragged rows by the fixed part of a segment (the
// place among the rows, first copies through a page's entry, the four warps' join and
// the merge of the splits, 8 us together): 13 rows to 4099, 8/8, 28 us for a floor of
// 20; 64 rows to 2111, 28/4 and fp32 queries, 44 for 31; one row of 1000, 12/2, 9.
#include <cfloat>
#include <cmath>
#include <mutex>

#include "ws_kv_q4.cuh"
#include "ws_paged.cuh"
#include "ws_split_merge.cuh"
#include "ws_tcgen05.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kPgHeads = 8;    // query heads a CTA takes at once: the products' columns
constexpr int kPgMaxB = 1024;
constexpr int kPgUnit = 16;    // slots
constexpr int kPgWarps = 4;
constexpr int kPgThreads = kPgWarps * 32;
// Ring stages a warp, CTAs a SM.  fp32 queries take the registers of a third CTA: with it
// 64 rows to 2111 slots, 28/4 heads, 48.1 us against 45.1 (before kPgTail), one row of 8192, 32/8, 21.9
// against 15.4.  16-bit ones: 16 rows to 32768, 32/8, 245.5 us against 251.9 with two, 256
// rows of 200 51.2 against 57.4.
template <bool LO>
constexpr int kPgStages = LO ? 3 : 2;
template <bool LO>
constexpr int kPgCtas = LO ? 2 : 3;
constexpr int kPgHalf = kPgUnit * 128;              // bytes of a unit's keys, 64 dimensions
constexpr int kPgStageBytes = 4 * kPgHalf;          // keys, then values
constexpr int kPgComb = kSplitDim + 4;              // floats from head to head: a warp's lanes in 32 banks
template <bool LO>
constexpr int kPgRing = kPgWarps * kPgStages<LO> * kPgStageBytes;
template <bool LO>
constexpr int kPgSmem = kPgRing<LO> + kPgWarps / 2 * kPgHeads * kPgComb * 4 + 1024;
constexpr int kPgMaxCtas = 1024;
constexpr int kPgOnce = 48;     // CTAs of a (row, head) that are merged in one go
// the running maximum follows a unit's only when that is 2^8 above it; it starts
// at the lowest number, below every finite score
constexpr float kPgLazy = 8.f;
// fp16 probabilities are held 2^7 times as large (at most 2^15), so that the lo
// terms reach down to 2^-31 of the maximum's
template <int DT>
constexpr float kPgUp = DT == DT_F16 ? 7.f : 0.f;

struct PagedParams {
  CUtensorMap mk, mv;  // [2 halves][rows of 16-bit 128][64], boxes of 2 x 16 x 64
  const void* q;       // [B][nh * 128], fp32 or the cache's type
  const void* k_new;   // [B][nkv * 128] of q's type, or null
  const void* v_new;
  uint16_t* k;         // [n_pages][nkv][ps][128]
  uint16_t* v;
  const int* table;    // [n_rows][max_pages]
  const int* rows;     // [B] or null
  const int* pos;      // [B]: slot of the new token, negative: none
  float* out_f32;      // [B][nh * 128]
  uint16_t* out_16;
  float* lse;          // [B][nh]
  int B, n_rows, max_pages, n_pages, ps, nh, nkv;
  int slots, upp;      // of a table row; units a page
  unsigned inv;        // 2^32 / upp rounded up, 0 for one unit
  int G, parts, hc;    // heads a key-value head; cut into `parts` of at most hc
  float scale;         // log2(e) / sqrt(128)
  float* part;         // [CTAs][2][hc][kSplitPart]
  unsigned* tick;      // [3][kPgMaxCtas]
  int* err;
  unsigned long long timeout_ns;
  TestHold hold;       // copies: the units of a row and part
};

// A batch row's sequence: its table row and last slot; pos < 0: none.
struct PgRow {
  int pos, row;
};
__device__ __forceinline__ PgRow pg_row(const PagedParams& a, int b, bool flag) {
  PgRow r = {-1, 0};
  if (b >= a.B) return r;
  r.pos = a.pos[b];
  if (r.pos < 0) return r;
  r.row = a.rows ? a.rows[b] : b;
  if (r.row < 0 || r.row >= a.n_rows || r.pos >= a.slots) {
    r.pos = -1;
    if (flag) atomicExch(a.err, kDerrBadSlot);
  }
  return r;
}

// Units of a row and head in the count that the CTAs share out: a multiple of
// the warps, so that a run never ends among the four and short sequences get a
// CTA each; those past the last slot are empty.  kPgTail more stand for what the end of a row
// and head costs the CTA that comes to it (2 to 3 us, in which the others stream on): none, 12,
// 16 and 20: 13 ragged rows 30.9, 29.0, 28.3, 28.1 us; 16 rows to 4096, 12/2, 23.1, 17.8, 17.9,
// 17.8; one row of 8192 15.0, 15.6, 14.7, 15.7; 30 of 500, 28/4, -, 14.6, 15.6, 15.2.
constexpr int kPgTail = 16;
__device__ __forceinline__ int pg_units(int pos) {
  constexpr int kSlots = kPgUnit * kPgWarps;
  return pos < 0 ? 0 : (pos / kSlots + 1) * kPgWarps + kPgTail;
}

// The page (its place in the table's row) of unit u of a row, below 2^26; upp is 64 at
// most.  Divisions by run-time numbers are 30 instructions each, and fourteen of them stood between
// the launch and its first copies.
__device__ __forceinline__ int pg_page(const PagedParams& a, int u) {
  return a.inv ? (int)__umulhi((unsigned)u, a.inv) : u;
}
__device__ __forceinline__ int pg_head(const PagedParams& a, int g) {  // key-value head of part g
  return a.parts == 1 ? g : g / a.parts;
}

// Where a warp's next unit lies: unit x of the CTA's range (counted from the
// range's start) is unit x - at of (row b, part g), which has nt of them.
struct PgCursor {
  int b, g, at, nt;
  PgRow r;
};

__device__ __forceinline__ void pg_seek(const PagedParams& a, PgCursor& c, int x) {
  while (x >= c.at + c.nt) {
    c.at += c.nt;
    if (++c.g == a.nkv * a.parts) {
      c.g = 0;
      do {
        c.r = pg_row(a, ++c.b, false);
        c.nt = pg_units(c.r.pos);
      } while (c.nt == 0);
    }
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pg_pack(float a, float b) {
  if constexpr (DT == DT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int DT>
__device__ __forceinline__ float2 pg_unpack(uint32_t u) {
  if constexpr (DT == DT_F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  else return make_float2(bf16lo(u), bf16hi(u));
}
// v = hi + lo, two values a word
template <int DT>
__device__ __forceinline__ void pg_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pg_pack<DT>(a, b);
  const float2 h = pg_unpack<DT>(hi);
  lo = pg_pack<DT>(a - h.x, b - h.y);
}

template <int DT>
__device__ __forceinline__ void pg_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == DT_F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ void pg_ldsm(uint32_t addr, uint32_t (&r)[4]) {
  ldsm_x4(addr, r[0], r[1], r[2], r[3]);
}
// the same with each 8x8 matrix transposed
__device__ __forceinline__ void pg_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pg_transpose(uint32_t a) {  // an 8x8 matrix of 16-bit values
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The two products of a warp and what it accumulates, for up to 8 heads.
// Lane 4 r + t: heads 2 t, 2 t + 1 of the results, head r of the queries.
// LO: the queries have lower terms (they are fp32).
template <int DT, bool LO>
struct PgCore {
  static constexpr int kTerms = !LO ? 1 : DT == DT_F16 ? 2 : 3;
  float o[8][4];  // o[i]: dimensions 16 i + r (+ 8), heads 2 t + e
  float m[2], l[2], sc[2];
  uint32_t q[kTerms][8][2];
  uint32_t ka, va;  // this lane's row in a unit's keys, and in its values
  uint32_t kx, vx;

  // The queries of n heads from h0 on, as they lie in memory: head r's (column r;
  // those from n on are zero), this lane's dimensions 16 i + 8 e + 2 t, + 1
  float2 x[LO ? 8 : 1][2];
  __device__ __forceinline__ void fetch(const PagedParams& a, int b, int h0, int n) {
    const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const size_t at = ((size_t)b * a.nh + h0 + (r < n ? r : 0)) * kSplitDim + 2 * t;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (LO) {
          x[i][e] = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + 16 * i + 8 * e);
          if (r >= n) x[i][e] = make_float2(0.f, 0.f);
        } else {
          q[0][i][e] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at + 16 * i + 8 * e);
          if (r >= n) q[0][i][e] = 0u;
        }
      }
  }

  // The fetched queries as operands; nothing summed up yet.
  __device__ __forceinline__ void begin(const PagedParams& a) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float up = 1.f;
    if constexpr (LO) {
      if constexpr (DT == DT_F16) {
        // fp32 queries may lie outside fp16: each head by the power of two that brings its
        // largest value to 1 .. 2 (2 .. 4 from 2^127 on; 2^126 is the largest whose reciprocal is normal)
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) top = fmaxf(top, fmaxf(fabsf(x[i][e].x), fabsf(x[i][e].y)));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 126);
        up = __uint_as_float((uint32_t)(ex + 127) << 23);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) x[i][e].x *= down, x[i][e].y *= down;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            q[k][i][e] = pg_pack<DT>(x[i][e].x, x[i][e].y);
            const float2 h = pg_unpack<DT>(q[k][i][e]);
            x[i][e].x -= h.x, x[i][e].y -= h.y;
          }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sc[e] = a.scale * __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
      m[e] = -FLT_MAX;
      l[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // ldmatrix: lane 8 j + i gives row i of matrix j.  Keys: matrices (rows 0..7,
    // 8..15) x (8 dimensions, the next 8); values, transposed: (8 dimensions, the next 8) x (rows
    // 0..7, 8..15).
    const int kr = (lane & 7) + (lane & 8), vr = (lane & 7) + ((lane & 16) >> 1);
    ka = kr * 128;
    kx = (((lane >> 4) ^ (kr & 7)) << 4);
    va = vr * 128;
    vx = ((((lane >> 3) & 1) ^ (vr & 7)) << 4);
  }

  // one unit at st: slots slot0 .. slot0 + 15, those after pos masked
  __device__ __forceinline__ void unit(uint32_t st, int slot0, int pos) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    // one sum a term, and two for the only one
    constexpr int kSums = kTerms == 1 ? 2 : kTerms;
    float c[kSums][4];
#pragma unroll
    for (int j = 0; j < kSums; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[j][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t f[4];
      pg_ldsm(st + ka + (i >> 2) * kPgHalf + (kx ^ ((i & 3) << 5)), f);
#pragma unroll
      for (int k = 0; k < kTerms; ++k) pg_mma<DT>(c[kTerms == 1 ? i & 1 : k], f, q[k][i][0], q[k][i][1]);
    }
    float s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = c[kSums - 1][e];
#pragma unroll
      for (int j = kSums - 2; j >= 0; --j) s[e] += c[j][e];
      s[e] *= sc[e & 1];
    }
    if (slot0 + kPgUnit > pos + 1) {
      if (slot0 + r > pos) s[0] = s[1] = -INFINITY;
      if (slot0 + r + 8 > pos) s[2] = s[3] = -INFINITY;
    }
    float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
    if (__any_sync(0xffffffffu, mx[0] > m[0] + kPgLazy || mx[1] > m[1] + kPgLazy)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], x));
        const float mn = fmaxf(m[e], mx[e]), f = split_exp2(m[e] - mn);
        m[e] = mn;
        l[e] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][e] *= f, o[i][2 + e] *= f;
      }
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = split_exp2(s[e] - (m[e & 1] - kPgUp<DT>));
    l[0] += p[0] + p[2];
    l[1] += p[1] + p[3];
    uint32_t ph[2], pl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      pg_split<DT>(p[2 * j], p[2 * j + 1], ph[j], pl[j]);
      ph[j] = pg_transpose(ph[j]);
      pl[j] = pg_transpose(pl[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t f[4];
      pg_ldsm_t(st + 2 * kPgHalf + va + (i >> 2) * kPgHalf + (vx ^ ((i & 3) << 5)), f);
      pg_mma<DT>(o[i], f, ph[0], ph[1]);
      pg_mma<DT>(o[i], f, pl[0], pl[1]);
    }
  }

  // this warp's maxima and sums: cm, cl [heads]
  __device__ __forceinline__ void sums(float* cm, float* cl) {
    const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
      if (r == 0) cm[2 * t + e] = m[e], cl[2 * t + e] = l[e];
    }
  }
  // its outputs, brought to the CTA's maxima M of its two heads, to comb [heads][kPgComb]
  template <bool ADD>
  __device__ __forceinline__ void put(float M0, float M1, float* comb) {
    const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const float f[2] = {split_exp2(m[0] - M0), split_exp2(m[1] - M1)};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* c = comb + (2 * t + (e & 1)) * kPgComb + 16 * i + 8 * (e >> 1) + r;
        *c = ADD ? fmaf(o[i][e], f[e & 1], *c) : o[i][e] * f[e & 1];
      }
  }
};

// Eight values of the new row as two words a pair in the cache's type.
template <int DT>
__device__ __forceinline__ uint4 pg_new8(const void* src, bool f32, size_t at) {
  if (!f32) return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + at);
  float x[8];
  load8<DT_F32>(static_cast<const float*>(src) + at, x);
  return make_uint4(pg_pack<DT>(x[0], x[1]), pg_pack<DT>(x[2], x[3]), pg_pack<DT>(x[4], x[5]),
                    pg_pack<DT>(x[6], x[7]));
}

// The sequence's last unit, its copies done: the new row to its place there
// and (`store`) in the page, and zeros for the values behind it, whatever the
// page holds there.
template <int DT>
__device__ __noinline__ void pg_last(const PagedParams& a, unsigned char* st, size_t row0, int n,
                                     size_t from, bool f32, bool store, int lane) {
  const bool keys = lane < 16;
  const int c = lane & 15;
  unsigned char* half = st + (keys ? 0 : 2 * kPgHalf) + (c >> 3) * kPgHalf;
  if (a.k_new) {
    const uint4 x = pg_new8<DT>(keys ? a.k_new : a.v_new, f32, from + 8 * c);
    *reinterpret_cast<uint4*>(half + n * 128 + (((c & 7) ^ (n & 7)) << 4)) = x;
    if (store) *reinterpret_cast<uint4*>((keys ? a.k : a.v) + (row0 + n) * kSplitDim + 8 * c) = x;
  }
  if (!keys)
    for (int i = n + 1; i < kPgUnit; ++i)
      *reinterpret_cast<uint4*>(half + i * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
  __syncwarp();
}

// out = O / L, four dimensions a lane
template <int DT>
__device__ __forceinline__ void pg_write(const PagedParams& a, int b, int h, int lane, float4 O,
                                         float M, float L) {
  const size_t at = ((size_t)b * a.nh + h) * kSplitDim + 4 * lane;
  O.x /= L, O.y /= L, O.z /= L, O.w /= L;
  if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + at) = O;
  if (a.out_16)
    *reinterpret_cast<uint2*>(a.out_16 + at) = make_uint2(pg_pack<DT>(O.x, O.y), pg_pack<DT>(O.z, O.w));
  if (a.lse && lane == 0)
    a.lse[(size_t)b * a.nh + h] = (M - kPgUp<DT> + log2f(L)) * 0.6931471805599453f;
}

template <int DT, bool LO>
__global__ void __launch_bounds__(kPgThreads, kPgCtas<LO>)
    k_decode_attention_paged(const __grid_constant__ PagedParams a) {
  constexpr int kStages = kPgStages<LO>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kPgWarps][kStages];
  __shared__ float cm[kPgWarps][kPgHeads], cl[kPgWarps][kPgHeads];
  __shared__ int last;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr unsigned all = 0xffffffffu;

  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
    tma_prefetch_map(&a.mk);
    tma_prefetch_map(&a.mv);
  }
  __syncwarp();
  pdl_wait();
  // the units of all rows and parts, cut into as many equal runs as there are
  // CTAs; every warp finds the run's place by itself
  const int np = a.nkv * a.parts;
  int total = 0;
  PgRow r0 = {-1, 0};
#pragma unroll 4
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const PgRow r = pg_row(a, b0 + lane, blockIdx.x == 0 && warp == 0);
    if (b0 == 0) r0 = r;
    total += pg_units(r.pos);
  }
  total = __reduce_add_sync(all, total) * np;
  const int per = ((total + (int)gridDim.x - 1) / (int)gridDim.x + kPgWarps - 1) / kPgWarps * kPgWarps;
  const int start = blockIdx.x * per, run = min(per, total - start);
  if (run <= 0) return;
  PgCursor cur;
  {
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
      const PgRow r = b0 == 0 ? r0 : pg_row(a, b0 + lane, false);
      const int nt = pg_units(r.pos);
      int sum = nt * np;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(all, sum, o);
        if (lane >= o) sum += u;
      }
      const unsigned hit = __ballot_sync(all, before + sum > start);
      if (hit) {
        const int l = __ffs(hit) - 1;
        cur.b = b0 + l;
        cur.r.pos = __shfl_sync(all, r.pos, l);
        cur.r.row = __shfl_sync(all, r.row, l);
        cur.nt = __shfl_sync(all, nt, l);
        const int in = start - before - (__shfl_sync(all, sum, l) - cur.nt * np);
        cur.g = in / cur.nt;
        cur.at = -(in % cur.nt);
        break;
      }
      before += __shfl_sync(all, sum, 31);
    }
  }
  int x0 = 0;
  if (cur.at + cur.nt <= kPgTail) {  // only the end of the run's first row and part: not its work
    x0 = cur.at + cur.nt;
    if (x0 >= run) return;
    pg_seek(a, cur, x0);
  }
  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* ring = smem + warp * kStages * kPgStageBytes;
  float* comb = reinterpret_cast<float*>(smem + kPgRing<LO>);

  // The next units to stage: up to 32 of the warp's in one segment, their pages a lane
  // each; and those behind them, whose pages are read ahead (behind the copies in
  // flight a read takes 3 us).
  struct Block {
    PgCursor c;
    int unit, n;  // the first of them, how many
  };
  auto block_at = [&](PgCursor c, int x) {  // from unit x of the run on
    Block k = {c, 0, 0};
    for (; x < run; x += kPgWarps) {
      pg_seek(a, k.c, x);
      k.unit = x - k.c.at;
      const int left = min(k.c.r.pos / kPgUnit, run - 1 - k.c.at) - k.unit;
      if (left < 0) continue;  // empty: on to the next row or part
      k.n = min(left / kPgWarps + 1, 32);
      break;
    }
    return k;
  };
  auto pages_of = [&](const Block& k) {
    const int u = k.unit + kPgWarps * lane;
    return lane < k.n ? a.table[(size_t)k.c.r.row * a.max_pages + pg_page(a, u)] : 0;
  };
  Block next = block_at(cur, x0 + warp);
  int ent = 0, ent_next = pages_of(next), left = 0, unit = 0, part = 0;  // of the units at hand
  int ni = 0, nc = 0;
  int at_page[kStages];  // of each stage's unit
  uint32_t bad = 0;        // stages whose unit has no page
  auto issue = [&]() {
    if (left == 0) {
      if (!next.n) return;
      ent = ent_next;
      left = next.n;
      unit = next.unit;
      part = next.c.g;
      next = block_at(next.c, next.c.at + unit + left * kPgWarps);
      ent_next = pages_of(next);
    }
    const int page = __shfl_sync(all, ent, 0), in = (unit - pg_page(a, unit) * a.upp) * kPgUnit;
    const bool held = unit == a.hold.here();
    ent = __shfl_down_sync(all, ent, 1);
    --left;
    unit += kPgWarps;
    unsigned char* st = ring + ni * kPgStageBytes;
    uint64_t* bar = &full[warp][ni];
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (s == ni) at_page[s] = page;
    fence_proxy_async_smem();  // what the lanes read and wrote there before the copies
    __syncwarp();
    if ((unsigned)page >= (unsigned)a.n_pages) {
      bad |= 1u << ni;
      if (lane == 0) atomicExch(a.err, kDerrBadSlot);
    } else if (lane == 0 && !held) {
      const int row = (page * a.nkv + pg_head(a, part)) * a.ps + in;
      mbar_arrive_expect_tx(bar, kPgStageBytes);
      tma_load_3d(st, &a.mk, 0, row, 0, bar);
      tma_load_3d(st + 2 * kPgHalf, &a.mv, 0, row, 0, bar);
    }
    ni = ni + 1 == kStages ? 0 : ni + 1;
  };
  // the first queries ahead of the copies, the next segments' behind their last units
  PgCore<DT, LO> core;
  auto fetch = [&](const PgCursor& c) {
    const int kvh = pg_head(a, c.g), pt = c.g - kvh * a.parts;
    core.fetch(a, c.b, kvh * a.G + pt * a.hc, min(a.hc, a.G - pt * a.hc));
    if (a.k_new) {  // the new row's lines, for the segment's end
      const size_t at = ((size_t)c.b * a.nkv + kvh) * kSplitDim + 8 * (lane & 15);
      const char* p = static_cast<const char*>(lane < 16 ? a.k_new : a.v_new) + at * (LO ? 4 : 2);
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
    }
  };
  fetch(cur);
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) issue();

  int x = x0 + warp;
  uint32_t par = 0;  // a bit a stage
  bool abort = false;
  while (x0 < run) {  // one (row, part) at a time
    const int x1 = min(run, cur.at + cur.nt);
    const int kvh = pg_head(a, cur.g), pt = cur.g - kvh * a.parts;
    const int h0 = kvh * a.G + pt * a.hc, nhd = min(a.hc, a.G - pt * a.hc);
    core.begin(a);
    const int xe = min(x1, cur.at + cur.r.pos / kPgUnit + 1);
    bool poison = false;
    for (; x < xe; x += kPgWarps) {
      unsigned char* st = ring + nc * kPgStageBytes;
      if (bad >> nc & 1) {  // nothing was copied: the stage's phase stays as it is
        bad &= ~(1u << nc);
        poison = true;
      } else {
        bool ok = abort || mbar_try_wait(&full[warp][nc], par >> nc & 1);
        if (!__all_sync(all, ok)) {
          ok = ok || mbar_wait_bounded(&full[warp][nc], par >> nc & 1, a.timeout_ns);
          if (__any_sync(all, !ok)) {
            abort = true;  // nothing more is issued; what is under way ends first
            if (lane == 0) atomicExch(a.err, (int)DERR_TIMEOUT);
            int i = nc;
            do {  // the stages from this one to the last filled
              if (!(bad >> i & 1)) mbar_wait_bounded(&full[warp][i], par >> i & 1, a.timeout_ns);
              i = i + 1 == kStages ? 0 : i + 1;
            } while (i != ni);
          }
        }
        par ^= 1u << nc;
        if (!abort) {
          const int slot0 = (x - cur.at) * kPgUnit;
          if (slot0 + kPgUnit > cur.r.pos) {
            int page = at_page[0];
#pragma unroll
            for (int s = 1; s < kStages; ++s)
              if (s == nc) page = at_page[s];
            const int u = x - cur.at;
            pg_last<DT>(a, st, ((size_t)page * a.nkv + kvh) * a.ps + slot0 - pg_page(a, u) * a.ps, cur.r.pos - slot0,
                        ((size_t)cur.b * a.nkv + kvh) * kSplitDim, LO, pt == 0, lane);
          }
          core.unit(smem_addr(st), slot0, cur.r.pos);
        }
      }
      nc = nc + 1 == kStages ? 0 : nc + 1;
      if (!abort) issue();
    }
    x = x1 + warp;
    PgCursor then = cur;
    if (x1 < run) {
      pg_seek(a, then, x1);
      fetch(then);
    }
    if (poison) core.l[0] = core.l[1] = __uint_as_float(0x7fc00000u);

    if (x1 >= run) pdl_launch_dependents();
    // the four warps' results, then this CTA's
    core.sums(cm[warp], cl[warp]);
    __syncthreads();
    {
      static_assert(kPgWarps == 4, "two warps' outputs side by side, the other two added to them");
      float M[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * (lane & 3) + e;
        M[e] = fmaxf(fmaxf(cm[0][h], cm[1][h]), fmaxf(cm[2][h], cm[3][h]));
      }
      float* c = comb + (warp & 1) * kPgHeads * kPgComb;
      if (warp < 2) core.template put<false>(M[0], M[1], c);
      __syncthreads();
      if (warp >= 2) core.template put<true>(M[0], M[1], c);
      __syncthreads();
    }
    const int seg0 = start + cur.at;  // the segment's first unit among all
    const int c0 = seg0 / per, n = (seg0 + cur.nt - kPgTail - 1) / per - c0 + 1;
    const int me = blockIdx.x - c0;
    const size_t slot = (size_t)2 * a.hc * kSplitPart;  // floats of a CTA's two partials
    float* mine = a.part + (size_t)blockIdx.x * slot + (me == 0 ? slot / 2 : 0);
    for (int h = warp; h < nhd; h += kPgWarps) {
      float M = cm[0][h], L = 0.f;
#pragma unroll
      for (int w = 1; w < kPgWarps; ++w) M = fmaxf(M, cm[w][h]);
      float4 O = reinterpret_cast<const float4*>(comb + h * kPgComb)[lane];
      const float4 v = reinterpret_cast<const float4*>(comb + (kPgHeads + h) * kPgComb)[lane];
      O.x += v.x, O.y += v.y, O.z += v.z, O.w += v.w;
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) L = fmaf(split_exp2(cm[w][h] - M), cl[w][h], L);
      if (n == 1) pg_write<DT>(a, cur.b, h0 + h, lane, O, M, L);
      else split_put(mine + h * kSplitPart, lane, O, M, L);
    }
    if (n > 1) {
      // up to kPgOnce: the last CTA merges all.  More: the last of each 16 merges
      // them into the first one's place, the last of the groups merges the groups.
      const bool once = n <= kPgOnce;
      const int grp = once ? 0 : me / kSplitMerge, in = once ? n : min(kSplitMerge, n - grp * kSplitMerge);
      const int groups = once ? 1 : (n + kSplitMerge - 1) / kSplitMerge;
      float* base = a.part + (size_t)c0 * slot;  // CTA c0's entry is its second one
      float* first = base + (grp ? (size_t)grp * kSplitMerge * slot : slot / 2);
      __syncthreads();
      if (t == 0) {
        unsigned* tk = a.tick + (grp ? kPgMaxCtas : 0) + c0 + grp * kSplitMerge;
        last = split_ticket(tk) == (unsigned)(in - 1);
        if (last) *tk = 0;
      }
      __syncthreads();
      if (last) {
        // head h is the same warp's from the partials to the result
        for (int h = warp; h < nhd; h += kPgWarps) {
          float4 O;
          float M, L;
          split_merge(first, base + (size_t)grp * kSplitMerge * slot, slot, in, h, lane, O, M, L);
          if (groups == 1) {
            pg_write<DT>(a, cur.b, h0 + h, lane, O, M, L);
          } else {
            __syncwarp();  // every lane has read the first entry
            split_put(first + h * kSplitPart, lane, O, M, L);
          }
        }
        if (groups > 1) {
          __syncthreads();
          if (t == 0) {
            unsigned* tk = a.tick + 2 * kPgMaxCtas + c0;
            last = split_ticket(tk) == (unsigned)(groups - 1);
            if (last) *tk = 0;
          }
          __syncthreads();
          if (last)
            for (int h = warp; h < nhd; h += kPgWarps) {
              float4 O;
              float M, L;
              split_merge(base + slot / 2, base, kSplitMerge * slot, groups, h, lane, O, M, L);
              pg_write<DT>(a, cur.b, h0 + h, lane, O, M, L);
            }
        }
      }
    }
    __syncthreads();  // cm, cl and comb are free again
    x0 = x1;
    cur = then;
  }
}

// Resident CTAs of the device: the grid, set up once per device.
template <int DT, bool LO>
static int pg_grid(cudaError_t* err) {
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
      e = cudaFuncSetAttribute(k_decode_attention_paged<DT, LO>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmem<LO>);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_decode_attention_paged<DT, LO>,
                                                        kPgThreads, kPgSmem<LO>);
    if (e != cudaSuccess || per_sm < 1) {
      *err = e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
      return 0;
    }
    grid[dev] = sms * per_sm < kPgMaxCtas ? sms * per_sm : kPgMaxCtas;
  }
  return grid[dev];
}

template <int DT, bool LO>
static cudaError_t pg_launch(const PagedParams& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const int grid = pg_grid<DT, LO>(&e);
  if (!grid) return e;
  e = launch_serving(k_decode_attention_paged<DT, LO>, dim3(grid), kPgThreads, kPgSmem<LO>, stream, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

static bool pg_shape_ok(int B, int nh, int nkv, int d) {
  return B >= 1 && B <= kPgMaxB && nkv >= 1 && nkv <= 65535 && nh >= 1 && nh <= 65535 &&
         nh % nkv == 0 && d == kSplitDim;
}
static int pg_parts(int G) { return (G + kPgHeads - 1) / kPgHeads; }
static int pg_heads(int G) { return (G + pg_parts(G) - 1) / pg_parts(G); }

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_attention_paged_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim) {
  if (!pg_shape_ok(B, n_heads, n_kv_heads, head_dim)) return 0;
  return 3 * kPgMaxCtas * 4 + (size_t)kPgMaxCtas * 2 * pg_heads(n_heads / n_kv_heads) * kSplitPart * 4;
}

ws_status ws_decode_attention_paged(const void *q, int q_dtype, const void *k_new,
                                    const void *v_new, void *k_pages, void *v_pages, int dtype,
                                    const int32_t *table, const int32_t *rows, const int32_t *pos,
                                    float *out_f32, void *out_16, float *lse, int B, int n_rows,
                                    int max_pages, int n_pages, int page_size, int n_heads,
                                    int n_kv_heads, int head_dim, void *workspace,
                                    size_t workspace_bytes, ws_stream_t stream) {
  if (!q || !k_pages || !v_pages || !table || !pos || !workspace || (!out_f32 && !out_16) ||
      !k_new != !v_new) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if ((dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) ||
      (q_dtype != WS_DTYPE_F32 && q_dtype != dtype)) {
    set_error("paged decode attention: pages in bf16 or fp16, q and the new rows in fp32 or the "
              "pages' type");
    return WS_ERR_ARG;
  }
  if (!pg_shape_ok(B, n_heads, n_kv_heads, head_dim) ||
      !paged_shape_ok(n_rows, max_pages, n_pages, page_size, n_kv_heads) ||
      (!rows && n_rows < B) ||
      (long long)B * n_kv_heads * pg_parts(n_heads / n_kv_heads) *
              ((long long)max_pages * page_size / kPgUnit + kPgWarps + kPgTail) >= (1ll << 31) - 4 * kPgMaxCtas) {
    set_error("paged decode attention: B 1..%d (at most n_rows without rows), head_dim %d, n_heads "
              "(to 65535) a multiple of n_kv_heads, page_size a multiple of 16 to 1024, "
              "max_pages * page_size at most 2^30, n_pages * n_kv_heads * page_size and the units "
              "of 16 slots below 2^31", kPgMaxB, kSplitDim);
    return WS_ERR_SHAPE;
  }
  const void* al[] = {q, k_new, v_new, k_pages, v_pages, workspace, out_f32, out_16};
  for (const void* p : al)
    if ((uintptr_t)p & 15u) {
      set_error("paged decode attention: q, new rows, pages, workspace and out must be 16-byte aligned");
      return WS_ERR_ALIGN;
    }
  const size_t need = ws_attention_paged_workspace_bytes(B, n_heads, n_kv_heads, head_dim);
  if (workspace_bytes < need) {
    set_error("workspace too small: need %zu bytes, got %zu", need, workspace_bytes);
    return WS_ERR_ARG;
  }
  PagedParams a = {};
  cudaError_t e = cudaSuccess;
  const long long slots = (long long)n_pages * n_kv_heads * page_size;
  if (!paged_map(&a.mk, dtype, k_pages, slots, &e) || !paged_map(&a.mv, dtype, v_pages, slots, &e)) {
    set_error("paged decode attention: tensor map: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k = static_cast<uint16_t*>(k_pages);
  a.v = static_cast<uint16_t*>(v_pages);
  a.table = table;
  a.rows = rows;
  a.pos = pos;
  a.out_f32 = out_f32;
  a.out_16 = static_cast<uint16_t*>(out_16);
  a.lse = lse;
  a.B = B;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  a.slots = max_pages * page_size;
  a.upp = page_size / kPgUnit;
  a.inv = a.upp == 1 ? 0u : (unsigned)(((1ull << 32) + a.upp - 1) / a.upp);
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.G = n_heads / n_kv_heads;
  a.parts = pg_parts(a.G);
  a.hc = pg_heads(a.G);
  a.scale = (float)(1.4426950408889634 / sqrt((double)kSplitDim));
  a.tick = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(a.tick + 3 * kPgMaxCtas);
  a.timeout_ns = tuning().timeout_ns;
  a.hold = test_hold();
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  const bool lo = q_dtype == WS_DTYPE_F32;
  if (dtype == WS_DTYPE_F16)
    e = lo ? pg_launch<DT_F16, true>(a, (cudaStream_t)stream) : pg_launch<DT_F16, false>(a, (cudaStream_t)stream);
  else
    e = lo ? pg_launch<DT_BF16, true>(a, (cudaStream_t)stream) : pg_launch<DT_BF16, false>(a, (cudaStream_t)stream);
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
