// ws_logprobs.cu -- log-probabilities of given tokens over rows of logits,
// with the row's entropy and its most likely tokens.
//
// With m = max x, Z = sum e^(x - m): log p_i = x_i - m - log Z, and the
// entropy -sum p log p = log Z - sum e^(x - m) (x - m) / Z.  One pass, a running
// maximum per thread (2^x by the special-function unit, which takes x log2 e).
//
// Bound by the latencies of its instructions and the barrier of each step, with
// no unit full: 2048 rows x 151665 bf16 with 20 alternatives: 150 us, 4.14 TB/s,
// 0.61 of the measured copy rate, issue 61% active, integer pipe 50%, DRAM 51%;
// the sums alone are 6 instructions a value, the search about as much again (1300
// rows: 64 us without it, 0.91 of the copy rate; 117 with it).  Shorter rows pay
// for the search's start and end, in which no copy is under way: 700 x 50257, 23.2
// us without, 42.1 with 20 alternatives, the floor 10.4; 5000 x 8000, 23.6 and 46.0
// against 11.8; 558 x 75974, 21.9 and 39.9 against 12.5.  A small
// batch's rows are cut into steps over up to 48 CTAs, the last of which merges:
// 16 x 151936 fp32 11.9 us, 1 x 50257 10.7 us, all of it latency (a CTA a row:
// 196 and 207 us).
#include <cmath>
#include <cstddef>
#include <mutex>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kMaxTop = 32;         // alternatives a row: one a lane
constexpr int kMaxVocab = 1 << 28;  // a row's bytes fit 32 bits
constexpr int kLpThreads = 128;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpBytes = 64;        // of values that a thread takes at once
constexpr int kLpStep = kLpThreads * kLpBytes / 2;  // values a step at most
constexpr int kLpStages = 2;        // steps on their way or worked on
constexpr int kLpCompact = 64;      // candidates that make the CTA sort out the best ones
constexpr int kLpBuf = 512;         // candidates there is room for
constexpr int kLpSplits = 48;       // CTAs a row at most
constexpr int kLpCtas = 8 * 152;    // CTAs that a batch's rows are cut into: all that are resident
constexpr float kLpFar = -1e4f;     // e^y is 0 long before: stands for -infinity in sums
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobParams {
  const void* x;  // [rows][ld], the first V of each row
  const int* targets;
  float* logprob;
  float* entropy;
  int* top_idx;
  float* top_lp;
  long long ld;
  int V, k;
  int splits, chunk;           // CTAs a row, values a CTA
  unsigned* tick;              // [rows]
  float4* stat;                // [rows][splits]: max, sum, sum e y
  unsigned long long* keys;    // [rows][splits][k]
  int* err;
  unsigned long long timeout_ns;
  TestHold hold;               // copies: the CTA's steps
};

// A key that orders as (value, lower index): the value's bits made monotone,
// then the complement of the index.  0 below every key; NaN has none.
__device__ __forceinline__ unsigned long long top_key(float v, int i) {
  if (v != v) return 0;
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 with +0
  return ((unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) |
         (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return (int)(0xffffffffu - (uint32_t)k);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float lp_exp2(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// Largest, sum of e^(x - max) and sum of e^(x - max) log2 e (x - max) of some
// values.  m starts at the lowest number, so that x - m is defined for every x
// but +infinity and NaN, which make the sums NaN.
struct LpSum {
  float m, z, t;
  __device__ __forceinline__ void raise(float to) {  // m to `to` >= m
    const float d = fmaxf(m - to, kLpFar) * kLog2e, f = lp_exp2(d);
    t = z > 0.f ? f * fmaf(z, d, t) : t;
    z *= f;
    m = to;
  }
  __device__ __forceinline__ void add_diff(float d) {  // one value, x - m given
    const float y = max_nan(d, kLpFar) * kLog2e, e = lp_exp2(y);
    z += e;
    t = fmaf(e, y, t);
  }
  __device__ __forceinline__ void join(const LpSum& o) {
    if (o.m > m) raise(o.m);
    const float d = o.m == m ? 0.f : fmaxf(o.m - m, kLpFar) * kLog2e, f = lp_exp2(d);
    z = fmaf(o.z, f, z);
    if (o.z != 0.f) t = fmaf(f, fmaf(o.z, d, o.t), t);
  }
  // over `n` lanes (a power of two); the lanes agree to the bit
  __device__ __forceinline__ void join_lanes(int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      if (o >= n) break;
      LpSum p;
      p.m = __shfl_xor_sync(0xffffffffu, m, o);
      p.z = __shfl_xor_sync(0xffffffffu, z, o);
      p.t = __shfl_xor_sync(0xffffffffu, t, o);
      if (lane & o) {
        p.join(*this);
        *this = p;
      } else {
        join(p);
      }
    }
  }
};

// 64 bytes of values in registers as they came
template <int DT>
struct LpRegs {
  static constexpr int kVec = DT == DT_F32 ? 4 : 8;  // values a 16-byte load
  static constexpr int kEach = kLpBytes / 16 * kVec;
  uint4 u[kLpBytes / 16];
  __device__ __forceinline__ uint32_t word(int i) const {
    return reinterpret_cast<const uint32_t*>(u)[i];
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == DT_F32) return __uint_as_float(word(i));
    const uint32_t h = word(i >> 1);
    if constexpr (DT == DT_F16) {
      const __half2 v = *reinterpret_cast<const __half2*>(&h);
      return i & 1 ? __high2float(v) : __low2float(v);
    }
    return i & 1 ? bf16hi(h) : bf16lo(h);
  }
  __device__ __forceinline__ float largest() const {  // NaN only where nothing else is there
    if constexpr (DT == DT_F32) {
      float m = value(0);
#pragma unroll
      for (int i = 1; i < kEach; ++i) m = fmaxf(m, value(i));
      return m;
    } else if constexpr (DT == DT_BF16) {
      __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&u[0].x);
#pragma unroll
      for (int i = 1; i < kEach / 2; ++i) {
        const uint32_t w = word(i);
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
      }
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      __half2 m = *reinterpret_cast<const __half2*>(&u[0].x);
#pragma unroll
      for (int i = 1; i < kEach / 2; ++i) {
        const uint32_t w = word(i);
        m = __hmax2(m, *reinterpret_cast<const __half2*>(&w));
      }
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
  // whether value 2 i or 2 i + 1 is at least thr (`packed`: thr rounded down, twice)
  __device__ __forceinline__ bool pair_reaches(int i, float thr, uint32_t packed) const {
    if constexpr (DT == DT_F32) {
      return fmaxf(value(2 * i), value(2 * i + 1)) >= thr;
    } else {
      const uint32_t w = word(i);
      if constexpr (DT == DT_BF16)
        return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w),
                           *reinterpret_cast<const __nv_bfloat162*>(&packed)) != 0;
      else
        return __hge2_mask(*reinterpret_cast<const __half2*>(&w),
                           *reinterpret_cast<const __half2*>(&packed)) != 0;
    }
  }
  static __device__ __forceinline__ uint32_t pack_down(float thr) {
    if constexpr (DT == DT_F32) return 0;
    uint32_t h;
    if constexpr (DT == DT_BF16) h = __bfloat16_as_ushort(__float2bfloat16_rd(thr));
    else h = __half_as_ushort(__float2half_rd(thr));
    return h | (h << 16);
  }
  // x - m, one rounding: for the 16-bit types by the mixed fma 1 x + (-m)
  __device__ __forceinline__ float diff(int i, float neg_m) const {
    if constexpr (DT == DT_F32) {
      return value(i) + neg_m;
    } else {
      const uint32_t h = word(i >> 1);
      float r;
      if constexpr (DT == DT_BF16) {
        if (i & 1)
          asm("{\n\t.reg .b16 l, h, o;\n\tmov.b32 {l, h}, %1;\n\tmov.b16 o, 0x3f80;\n\t"
              "fma.rn.f32.bf16 %0, h, o, %2;\n\t}" : "=f"(r) : "r"(h), "f"(neg_m));
        else
          asm("{\n\t.reg .b16 l, h, o;\n\tmov.b32 {l, h}, %1;\n\tmov.b16 o, 0x3f80;\n\t"
              "fma.rn.f32.bf16 %0, l, o, %2;\n\t}" : "=f"(r) : "r"(h), "f"(neg_m));
      } else {
        if (i & 1)
          asm("{\n\t.reg .b16 l, h, o;\n\tmov.b32 {l, h}, %1;\n\tmov.b16 o, 0x3c00;\n\t"
              "fma.rn.f32.f16 %0, h, o, %2;\n\t}" : "=f"(r) : "r"(h), "f"(neg_m));
        else
          asm("{\n\t.reg .b16 l, h, o;\n\tmov.b32 {l, h}, %1;\n\tmov.b16 o, 0x3c00;\n\t"
              "fma.rn.f32.f16 %0, l, o, %2;\n\t}" : "=f"(r) : "r"(h), "f"(neg_m));
      }
      return r;
    }
  }
};

template <int DT>
__device__ __forceinline__ float lp_value(const void* row, int i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(row)[i];
  const uint16_t u = static_cast<const uint16_t*>(row)[i];
  if constexpr (DT == DT_F16) return __half2float(__ushort_as_half(u));
  return __uint_as_float((uint32_t)u << 16);
}

// The lanes' keys in falling order; then merged with a list in falling order.
template <typename K>
__device__ __forceinline__ K lp_exchange(K k, int o, bool keep_max) {
  const K p = __shfl_xor_sync(0xffffffffu, k, o);
  return (p > k) == keep_max ? p : k;
}
template <typename K>
__device__ __forceinline__ K lp_sort(K k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o > 0; o >>= 1)
      k = lp_exchange(k, o, ((lane & o) == 0) == ((lane & n) == 0 || n == 32));
  return k;
}
template <typename K>
__device__ __forceinline__ K lp_merge(K a, K b, int lane) {
  const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = a > r ? a : r;  // the 32 largest of both, rising then falling
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = lp_exchange(a, o, (lane & o) == 0);
  return a;
}

struct LpShared {
  uint64_t full[kLpStages];
  unsigned long long thr;   // a candidate's key is at least this
  LpSum sums[kLpWarps];
  int n;                    // candidates
  int last, abort;
  unsigned long long list[kLpWarps][32];
  unsigned long long buf[kLpBuf];  // (not there without alternatives)
};
constexpr int kLpRing = kLpStages * kLpThreads * kLpBytes;

// The whole CTA: the 32 largest keys of the warps' lists (`mine`, in falling
// order; those of the first `lists` warps are not empty) become the only
// candidates, in falling order, and the threshold the k-th of them plus 1.
__device__ __forceinline__ void lp_gather(LpShared& sh, unsigned long long mine, int lists, int k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
  for (int o = 1; o < lists; o <<= 1) {
    if ((warp & (2 * o - 1)) == o) sh.list[warp][lane] = mine;
    __syncthreads();
    if (!(warp & (2 * o - 1)) && warp + o < lists) mine = lp_merge(mine, sh.list[warp + o][lane], lane);
  }
  __syncthreads();
  if (warp == 0) {
    sh.buf[lane] = mine;
    if (lane == k - 1) sh.thr = mine ? mine + 1 : 0;
    const int have = __popc(__ballot_sync(0xffffffffu, mine != 0));
    if (lane == 0) sh.n = have;
  }
  __syncthreads();
}

// The same of the n candidates so far.
__device__ __noinline__ void lp_compact(LpShared& sh, int n, int k) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  unsigned long long mine = 0;
  for (int i = warp * 32; i < n; i += kLpThreads) {
    const unsigned long long key = i + lane < n ? sh.buf[i + lane] : 0;
    if (__any_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, mine, k - 1)))
      mine = lp_merge(mine, lp_sort(key, lane), lane);
  }
  lp_gather(sh, mine, min(kLpWarps, (n + 31) / 32), k);
}

// One CTA per (split, row).  A ring of two steps of 8 KB in shared memory filled
// by bulk copies, so that registers hold one step and eight CTAs share a SM
// (three steps and fewer CTAs were slower: the other CTAs cover the steps'
// barrier.  A ring for each warp, no barrier a step and the candidates looked at
// every 1, 2, 4, 8 steps: 163, 160, 157, 157 us against 150 for the 2048 rows;
// the clamp on pairs of 16 bits 156; the search in two levels 150).  The best `k` are found in the same pass:
// the k-th of the threads' largest values of the first step bounds the k-th of
// all from below, so that only the values from there on become candidates, few
// in most rows; their best ones raise the bound when there are many.  An order
// that keeps rising makes that slower but not wrong, and so does a row in which
// fewer than k of those largest values are above -infinity: every value ruled out
// then reaches the bound and is looked at by its index (2048 x 151936 bf16, 20
// alternatives: 149 us, with 1504 tokens allowed 157, with 18 allowed 479; 16 rows
// fp32 with 16 allowed 26 against 12).
template <int DT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 8) k_token_logprobs(const __grid_constant__ LogprobParams a) {
  extern __shared__ __align__(128) unsigned char smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem + kLpRing);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = blockIdx.x / a.splits, sp = blockIdx.x - r * a.splits;
  constexpr int kSize = DT == DT_F32 ? 4 : 2, kVec = LpRegs<DT>::kVec;
  const char* row = static_cast<const char*>(a.x) + (size_t)r * a.ld * kSize;
  const int c0 = sp * a.chunk, c1 = min(a.V, c0 + a.chunk);
  // values before the first 16-byte boundary and behind the last: one a thread
  const int pre = min(c1 - c0, (int)((16 - ((uintptr_t)(row + (size_t)c0 * kSize) & 15)) & 15) / kSize);
  const int v0 = c0 + pre, nv = (c1 - v0) / kVec, rest = (c1 - v0) - nv * kVec;
  const char* body = row + (size_t)v0 * kSize;

  constexpr int kLoads = kLpBytes / 16, kEach = LpRegs<DT>::kEach;
  constexpr uint32_t kNegInf = DT == DT_F32 ? 0xff800000u : DT == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  constexpr int kStepVec = kLpThreads * kLoads, kStepBytes = kStepVec * 16;
  const int steps = (nv + kStepVec - 1) / kStepVec;
  const int hold = a.hold.here();
  auto fill = [&](int step) {  // one thread
    if (step == hold) return;
    const int bytes = min(kStepBytes, (nv - step * kStepVec) * 16);
    uint64_t* bar = &sh.full[step % kLpStages];
    mbar_arrive_expect_tx(bar, bytes);
    bulk_copy_g2s(smem + (step % kLpStages) * kStepBytes, body + (size_t)step * kStepBytes, bytes, bar,
                  l2_policy_evict_first());
  };
  if (t == 0) {
    for (int i = 0; i < kLpStages; ++i) mbar_init(&sh.full[i], 1);
    fence_mbar_init();
    sh.n = 0;
    sh.abort = 0;
  }
  pdl_launch_dependents();
  pdl_wait();
  if (t == 0) {
    for (int i = 0; i < kLpStages && i < steps; ++i) fill(i);
  }
  __syncthreads();

  // the target's logit, in time for the end
  const int target = t == 0 && a.targets ? a.targets[r] : -1;
  const float target_x = target >= 0 && target < a.V ? lp_value<DT>(row, target) : 0.f;

  LpSum s = {-FLT_MAX, 0.f, 0.f};
  unsigned long long thr = 0;
  float thrv = -INFINITY;
  int over = 0;  // the place of this thread's last candidate
  auto candidate = [&](float v, int i, bool again) {
    const unsigned long long key = top_key(v, i);
    if (key < thr || !key) return;
    if (again)  // one of those kept already?
#pragma unroll 1
      for (int e = 0; e < 32; ++e)
        if (sh.buf[e] == key) return;
    over = atomicAdd(&sh.n, 1);
    if (over < kLpBuf) sh.buf[over] = key;
  };
  if (t < pre + rest) {
    const int i = t < pre ? c0 + t : v0 + nv * kVec + (t - pre);
    const float x = lp_value<DT>(row, i);
    if (x > s.m) s.m = x;
    s.add_diff(x - s.m);
    if (TOP) candidate(x, i, false);
  }
  for (int step = 0; step < steps; ++step) {
    const int at = step * kStepVec;
    const bool ok = mbar_wait_bounded(&sh.full[step % kLpStages], (step / kLpStages) & 1, a.timeout_ns);
    if (!ok) sh.abort = 1;
    LpRegs<DT> cur;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {  // -infinity behind the end
      cur.u[j] = reinterpret_cast<const uint4*>(smem + (step % kLpStages) * kStepBytes)[j * kLpThreads + t];
      if (at + j * kLpThreads + t >= nv) cur.u[j] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
    }
    const float mx = cur.largest();
    if (mx > s.m) s.raise(mx);
    {
      const float nm = -s.m;
      float2 z = make_float2(0.f, 0.f), e2 = z;
#pragma unroll
      for (int i = 0; i < kEach; i += 2) {
        const float2 y = mul2(make_float2(max_nan(cur.diff(i, nm), kLpFar),
                                          max_nan(cur.diff(i + 1, nm), kLpFar)),
                              make_float2(kLog2e, kLog2e));
        const float2 e = make_float2(lp_exp2(y.x), lp_exp2(y.y));
        z = add2(z, e);
        e2 = fma2(e, y, e2);
      }
      s.z += z.x + z.y;
      s.t += e2.x + e2.y;
    }
    if (TOP) {
      if (at == 0) {
        // the k-th of the threads' largest values: at least k values reach it
        const uint32_t u = __float_as_uint(mx + 0.f);
        uint32_t top = mx == mx ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
        top = lp_sort(top, lane);
        uint32_t* lists = reinterpret_cast<uint32_t*>(sh.list);
#pragma unroll
        for (int o = 1; o < kLpWarps; o <<= 1) {
          if ((warp & (2 * o - 1)) == o) lists[warp * 32 + lane] = top;
          __syncthreads();
          if (!(warp & (2 * o - 1))) top = lp_merge(top, lists[(warp + o) * 32 + lane], lane);
        }
        if (warp == 0 && lane == a.k - 1) sh.thr = (unsigned long long)top << 32;
        __syncthreads();
        thr = sh.thr;
        thrv = thr >> 32 ? key_value(thr) : -INFINITY;
      }
    }
    // one barrier a step: the stage is free again, and whether the candidates
    // are many (more than there is room for: their best raise the bound, and
    // the step's values are gone through again) or a wait ran out
    bool again = false, lost = false;
    do {
      if (TOP && mx >= thrv) {
        const uint32_t packed = LpRegs<DT>::pack_down(thrv);
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i)
          if (cur.pair_reaches(i, thrv, packed)) hits |= 1u << i;
        while (hits) {  // few: from the ring again, so that this code is there once
          const int i = 2 * (__ffs(hits) - 1), vec = i / kVec * kLpThreads + t;
          hits &= hits - 1;
          if (at + vec >= nv) continue;
          const char* w = reinterpret_cast<const char*>(smem) + (step % kLpStages) * kStepBytes +
                          vec * 16 + i % kVec * kSize;
#pragma unroll 1
          for (int e = 0; e < 2; ++e)
            candidate(lp_value<DT>(w, e), v0 + (at + vec) * kVec + i % kVec + e, again);
        }
      }
      again = false;
      if (__syncthreads_or(!ok || (TOP && over >= kLpCompact))) {
        if (sh.abort) {
          // the row comes out as NaN; this part of it has no candidates, and its
          // ticket is taken below as ever
          if (t == 0) {
            atomicExch(a.err, (int)DERR_TIMEOUT);
            for (int i = step; i < steps && i < step + kLpStages; ++i)  // copies under way
              if (i != hold) mbar_wait_bounded(&sh.full[i % kLpStages], (i / kLpStages) & 1, a.timeout_ns);
            sh.n = 0;
          }
          s.z = s.t = NAN;
          lost = true;
          break;
        }
        if (TOP) {
          const int n = sh.n;
          again = n > kLpBuf;
          lp_compact(sh, min(n, kLpBuf), a.k);
          thr = sh.thr;
          thrv = thr >> 32 ? key_value(thr) : -INFINITY;
          over = 0;
          __syncthreads();
        }
      }
    } while (TOP && again);
    if (lost) break;
    if (t == 0 && step + kLpStages < steps) {
      fence_proxy_async_smem();  // the reads of this stage before the copy into it
      fill(step + kLpStages);
    }
  }
  if (TOP) {
    __syncthreads();
    lp_compact(sh, sh.n, a.k);
  }
  s.join_lanes(32);
  if (lane == 0) sh.sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = sh.sums[lane & (kLpWarps - 1)];
    s.join_lanes(kLpWarps);
  }
  if (a.splits > 1) {
    const size_t at = (size_t)r * a.splits;
    if (t == 0) a.stat[at + sp] = make_float4(s.m, s.z, s.t, 0.f);
    if (TOP && t < a.k) a.keys[(at + sp) * a.k + t] = sh.buf[t];
    __syncthreads();
    if (t == 0) {
      unsigned old;
      asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.tick + r) : "memory");
      sh.last = old == (unsigned)(a.splits - 1);
      if (sh.last) a.tick[r] = 0;
    }
    __syncthreads();
    if (!sh.last) return;
    // the row's last CTA: the splits' sums in their order, and the best of
    // their best
    if (warp == 0) {
      static_assert(kLpSplits <= 64, "two splits a lane");
      const float4 v = lane < a.splits ? __ldcg(a.stat + at + lane) : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
      const float4 w =
          lane + 32 < a.splits ? __ldcg(a.stat + at + lane + 32) : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
      s = {v.x, v.y, v.z};
      s.join({w.x, w.y, w.z});
      s.join_lanes(32);
    }
    if (TOP) {
      // lists in falling order already, four on their way at a time; short ones
      // are sorted again, 32 keys at once (a sort and a merge take as long as
      // four merges)
      unsigned long long mine = 0;
      const int n = a.splits * a.k;
      if (a.k <= 8)
        for (int i = warp * 32; i < n; i += kLpThreads)
          mine = lp_merge(mine, lp_sort(i + lane < n ? __ldcg(a.keys + at * a.k + i + lane) : 0ull, lane), lane);
      else
        for (int i0 = warp; i0 < a.splits; i0 += 4 * kLpWarps) {
          unsigned long long key[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kLpWarps;
            key[u] = i < a.splits && lane < a.k ? __ldcg(a.keys + (at + i) * a.k + lane) : 0;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) mine = lp_merge(mine, key[u], lane);
        }
      lp_gather(sh, mine, min(kLpWarps, a.k <= 8 ? (n + 31) / 32 : a.splits), a.k);
    }
  }
  if (warp > 0) return;
  // the alternatives are at most 32: one a lane of the first warp
  const float lz = logf(s.z);
  if (t == 0) {
    if (a.entropy) a.entropy[r] = lz - s.t / s.z / kLog2e;
    if (a.targets) {
      float lp = 0.f;
      if (target >= a.V) {
        atomicExch(a.err, kDerrBadToken);
        lp = NAN;
      } else if (target >= 0) {
        lp = target_x - s.m - lz;
      }
      a.logprob[r] = lp;
    }
  }
  if (TOP && t < a.k) {
    const unsigned long long key = sh.buf[t];
    if (a.top_idx) a.top_idx[(size_t)r * a.k + t] = key ? key_index(key) : -1;
    if (a.top_lp) a.top_lp[(size_t)r * a.k + t] = key ? key_value(key) - s.m - lz : NAN;
  }
}

// Splits of a row, and values a split: whole steps, and no more than fill
// kLpCtas CTAs with all rows, one wave (a row alone on one CTA takes 20 times as
// long).  With 608, 1216 and 1824 CTAs: 64 x 151936 bf16, 20 alternatives, 23.4,
// 17.0, 17.0 us; 377 x 20034 fp32, 5 alternatives, 19.5, 15.9, 16.1; 558 x 75974
// fp16 without, 26.1, 19.9, 23.6.  More rows are not cut, to even out their waves
// either: 2048 x 151665, 20 alternatives, 151.5 us whole, 174.8 in halves.
static void lp_split(int rows, int V, int& splits, int& chunk) {
  const int steps = (V + kLpStep - 1) / kLpStep;
  int want = kLpCtas / rows;
  if (want > kLpSplits) want = kLpSplits;
  if (want < 1) want = 1;
  const int per = (steps + want - 1) / want;
  chunk = per * kLpStep;
  splits = (steps + per - 1) / per;
}

// rows on several CTAs are at most kLpCtas / 2; the tickets' place is the same
// for every shape, so that no call finds another's results there
constexpr size_t kLpTick = (kLpCtas / 2 * 4 + 255) / 256 * 256;

static size_t lp_align(size_t v) { return (v + 255) / 256 * 256; }

constexpr int kLpSmemTop = kLpRing + (int)sizeof(LpShared);
constexpr int kLpSmem = kLpRing + (int)offsetof(LpShared, buf);

// The kernels' shared memory, once per device.
static cudaError_t lp_setup() {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static bool ready[kMaxDev] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (ready[dev]) return cudaSuccess;
  auto set = [&](const void* f) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmemTop);
  };
  set((const void*)k_token_logprobs<DT_F32, true>);
  set((const void*)k_token_logprobs<DT_BF16, true>);
  set((const void*)k_token_logprobs<DT_F16, true>);
  ready[dev] = e == cudaSuccess;
  return e;
}

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_logprobs_workspace_bytes(int rows, int V, int topk) {
  if (rows < 1 || V < 1 || V > kMaxVocab || topk < 0 || topk > kMaxTop || topk > V) return 0;
  int splits, chunk;
  lp_split(rows, V, splits, chunk);
  if (splits == 1) return 256;
  return kLpTick + lp_align((size_t)rows * splits * 16) + (size_t)rows * splits * topk * 8;
}

ws_status ws_token_logprobs(const void *logits, int dtype, long long ld, const int32_t *targets,
                            float *logprob, float *entropy, int32_t *top_idx, float *top_logprob,
                            int rows, int V, int topk, void *workspace, size_t workspace_bytes,
                            ws_stream_t stream) {
  if (!logits || !workspace || (!targets != !logprob) || (topk > 0 && !top_idx && !top_logprob) ||
      (!logprob && !entropy && topk == 0)) {
    set_error("null argument (targets and logprob go together; topk needs an output)");
    return WS_ERR_ARG;
  }
  if (dtype != WS_DTYPE_F32 && dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) {
    set_error("dtype must be WS_DTYPE_F32, WS_DTYPE_BF16 or WS_DTYPE_F16");
    return WS_ERR_ARG;
  }
  if (rows < 1 || V < 1 || V > kMaxVocab || ld < V || topk < 0 || topk > kMaxTop || topk > V) {
    set_error("log-probabilities: rows and V at least 1 (V to 2^28), ld at least V, topk 0..%d and "
              "at most V", kMaxTop);
    return WS_ERR_SHAPE;
  }
  if (((uintptr_t)logits & (dtype == WS_DTYPE_F32 ? 3u : 1u)) || ((uintptr_t)workspace & 15u)) {
    set_error("log-probabilities: logits aligned to their type, workspace to 16 bytes");
    return WS_ERR_ALIGN;
  }
  const size_t need = ws_logprobs_workspace_bytes(rows, V, topk);
  if (workspace_bytes < need) {
    set_error("workspace too small: need %zu bytes, got %zu", need, workspace_bytes);
    return WS_ERR_ARG;
  }
  cudaError_t e = lp_setup();
  if (e != cudaSuccess) {
    set_error("log-probabilities setup failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  LogprobParams a = {};
  a.x = logits;
  a.timeout_ns = tuning().timeout_ns;
  a.hold = test_hold();
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_idx = top_idx;
  a.top_lp = top_logprob;
  a.ld = ld;
  a.V = V;
  a.k = topk;
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  lp_split(rows, V, a.splits, a.chunk);
  char* w = static_cast<char*>(workspace);
  a.tick = reinterpret_cast<unsigned*>(w);
  w += kLpTick;
  a.stat = reinterpret_cast<float4*>(w);
  a.keys = reinterpret_cast<unsigned long long*>(w + lp_align((size_t)rows * a.splits * 16));
  cudaStream_t st = (cudaStream_t)stream;
  const int grid = rows * a.splits;
  const int sm = topk ? kLpSmemTop : kLpSmem;
  if (dtype == WS_DTYPE_F32) {
    if (topk) e = launch_serving(k_token_logprobs<DT_F32, true>, dim3(grid), kLpThreads, sm, st, a);
    else e = launch_serving(k_token_logprobs<DT_F32, false>, dim3(grid), kLpThreads, sm, st, a);
  } else if (dtype == WS_DTYPE_BF16) {
    if (topk) e = launch_serving(k_token_logprobs<DT_BF16, true>, dim3(grid), kLpThreads, sm, st, a);
    else e = launch_serving(k_token_logprobs<DT_BF16, false>, dim3(grid), kLpThreads, sm, st, a);
  } else {
    if (topk) e = launch_serving(k_token_logprobs<DT_F16, true>, dim3(grid), kLpThreads, sm, st, a);
    else e = launch_serving(k_token_logprobs<DT_F16, false>, dim3(grid), kLpThreads, sm, st, a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
