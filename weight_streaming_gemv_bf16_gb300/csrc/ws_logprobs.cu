// ws_logprobs.cu -- log-probabilities of given tokens over rows of logits,
// with the row's entropy and its most likely tokens.
//
// With m = max x, Z = sum e^(x - m): log p_i = x_i - m - log Z, and the
// entropy -sum p log p = log Z - sum e^(x - m) (x - m) / Z.
#include <cmath>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kMaxTop = 32;         // alternatives a row: one a lane
constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpEach = 16;         // values a thread takes at once
constexpr int kLpStep = kLpThreads * kLpEach;
constexpr int kLpCompact = 64;      // candidates that make the CTA sort out the best ones
constexpr int kLpBuf = kLpCompact + kLpStep + 2 * kLpEach;
static_assert(kLpBuf >= 64 * kMaxTop, "the splits' best fit");
constexpr int kLpSplits = 64;       // CTAs a row at most
constexpr int kLpCtas = 608;        // CTAs that a small batch's rows are cut into
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

// 16 values in registers as they came; the largest; x - m of each; each value
template <int DT>
struct LpRegs {
  static constexpr int kVec = DT == DT_F32 ? 4 : 8;  // values a 16-byte load
  uint4 u[kLpEach / kVec];
  __device__ __forceinline__ float value(int i) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
    if constexpr (DT == DT_F32) return __uint_as_float(w[i]);
    const uint32_t h = w[i >> 1];
    if constexpr (DT == DT_F16) {
      const __half2 v = *reinterpret_cast<const __half2*>(&h);
      return i & 1 ? __high2float(v) : __low2float(v);
    }
    return i & 1 ? bf16hi(h) : bf16lo(h);
  }
  __device__ __forceinline__ float largest() const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
    if constexpr (DT == DT_F32) {
      float m = value(0);
#pragma unroll
      for (int i = 1; i < kLpEach; ++i) m = fmaxf(m, value(i));
      return m;
    } else if constexpr (DT == DT_BF16) {
      __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0]);
#pragma unroll
      for (int i = 1; i < kLpEach / 2; ++i)
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      __half2 m = *reinterpret_cast<const __half2*>(&w[0]);
#pragma unroll
      for (int i = 1; i < kLpEach / 2; ++i) m = __hmax2(m, *reinterpret_cast<const __half2*>(&w[i]));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
  // x - m, one rounding: for the 16-bit types by the mixed fma 1 x + (-m)
  __device__ __forceinline__ float diff(int i, float neg_m) const {
    if constexpr (DT == DT_F32) {
      return value(i) + neg_m;
    } else {
      const uint32_t h = reinterpret_cast<const uint32_t*>(u)[i >> 1];
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

// The lanes' keys in falling order; then merged with a list in falling order.
__device__ __forceinline__ unsigned long long lp_exchange(unsigned long long k, int o, bool keep_max) {
  const unsigned long long p = __shfl_xor_sync(0xffffffffu, k, o);
  return (p > k) == keep_max ? p : k;
}
__device__ __forceinline__ unsigned long long lp_sort(unsigned long long k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o > 0; o >>= 1)
      k = lp_exchange(k, o, ((lane & o) == 0) == ((lane & n) == 0 || n == 32));
  return k;
}
__device__ __forceinline__ unsigned long long lp_merge(unsigned long long a, unsigned long long b,
                                                       int lane) {
  const unsigned long long r = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = a > r ? a : r;  // the 32 largest of both, rising then falling
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = lp_exchange(a, o, (lane & o) == 0);
  return a;
}

struct LpShared {
  unsigned long long buf[kLpBuf];
  unsigned long long list[kLpWarps][32];
  unsigned long long thr;   // a candidate's key is at least this
  int n;                    // candidates
  LpSum sums[kLpWarps];
  int last;
};

// The whole CTA: the 32 largest of the candidates, in falling order, become
// the only ones.  bar: the threshold becomes the k-th of them, plus `plus`.
__device__ __forceinline__ void lp_compact(LpShared& sh, int n, int k, int plus) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  unsigned long long mine = 0;
  for (int i = warp * 32; i < n; i += kLpThreads) {
    const unsigned long long key = i + lane < n ? sh.buf[i + lane] : 0;
    if (__any_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, mine, k - 1)))
      mine = lp_merge(mine, lp_sort(key, lane), lane);
  }
  // the warps' lists in pairs; those past the candidates are empty
  const int lists = min(kLpWarps, (n + 31) / 32);
#pragma unroll 1
  for (int o = 1; o < lists; o <<= 1) {
    if ((warp & (2 * o - 1)) == o) sh.list[warp][lane] = mine;
    __syncthreads();
    if (!(warp & (2 * o - 1)) && warp + o < lists) mine = lp_merge(mine, sh.list[warp + o][lane], lane);
  }
  __syncthreads();
  if (warp == 0) {
    sh.buf[lane] = mine;
    if (lane == k - 1) sh.thr = mine ? mine + plus : 0;
    const int have = __popc(__ballot_sync(0xffffffffu, mine != 0));
    if (lane == 0) sh.n = have;
  }
  __syncthreads();
}

// One CTA per (split, row).  DRAM bound: 64 bytes (32 of the 16-bit types) a
// thread are in flight while the last ones are worked on, one barrier for
// every 4096 values.  The best `k` are found in the same pass: the k-th of the
// threads' best values of the first step bounds the k-th of all from below, so
// that only the few values from there on become candidates; their best ones
// raise the bound when there are many, which an order that keeps rising makes
// slower but not wrong.
template <int DT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) k_token_logprobs(const __grid_constant__ LogprobParams a) {
  extern __shared__ __align__(16) unsigned char smem[];
  LpShared& sh = *reinterpret_cast<LpShared*>(smem);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = blockIdx.x / a.splits, sp = blockIdx.x - r * a.splits;
  constexpr int kSize = DT == DT_F32 ? 4 : 2, kVec = LpRegs<DT>::kVec;
  const char* row = static_cast<const char*>(a.x) + (size_t)r * a.ld * kSize;
  const int c0 = sp * a.chunk, c1 = min(a.V, c0 + a.chunk);
  // values before the first 16-byte boundary and behind the last: one a thread
  const int pre = min(c1 - c0, (int)((16 - ((uintptr_t)(row + (size_t)c0 * kSize) & 15)) & 15) / kSize);
  const int v0 = c0 + pre, nv = (c1 - v0) / kVec, rest = (c1 - v0) - nv * kVec;
  const uint4* body = reinterpret_cast<const uint4*>(row + (size_t)v0 * kSize);

  constexpr int kAhead = DT == DT_F32 ? 1 : 2;  // steps in flight: 64 bytes a thread
  LpRegs<DT> cur, nxt[kAhead];
  constexpr int kLoads = kLpEach / kVec;
  constexpr uint32_t kNegInf = DT == DT_F32 ? 0xff800000u : DT == DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  auto load = [&](LpRegs<DT>& g, int at) {  // vectors at + j * 256 + t; -infinity behind the end
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = at + j * kLpThreads + t;
      g.u[j] = i < nv ? __ldcs(body + i) : make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
    }
  };
  constexpr int kStepVec = kLpThreads * kLoads;
  load(cur, 0);
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) load(nxt[i], (i + 1) * kStepVec);

  LpSum s = {-FLT_MAX, 0.f, 0.f};
  unsigned long long thr = 0;
  float thrv = -INFINITY;
  if (TOP) {
    if (t == 0) sh.n = 0;
    __syncthreads();
  }
  int over = 0;
  auto candidate = [&](float v, int i) {
    const unsigned long long key = top_key(v, i);
    if (key >= thr && key) {
      const int at = atomicAdd(&sh.n, 1);
      sh.buf[at] = key;
      over = at;
    }
  };
  if (t < pre + rest) {
    const int i = t < pre ? c0 + t : v0 + nv * kVec + (t - pre);
    float x;
    if constexpr (DT == DT_F32) x = reinterpret_cast<const float*>(row)[i];
    else if constexpr (DT == DT_F16) x = __half2float(reinterpret_cast<const __half*>(row)[i]);
    else x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
    if (x > s.m) s.m = x;
    s.add_diff(x - s.m);
    if (TOP) candidate(x, i);
  }
  for (int at = 0; at < nv; at += kStepVec) {
    if (at + kAhead * kStepVec < nv) load(nxt[kAhead - 1], at + kAhead * kStepVec);
    const float mx = cur.largest();
    if (mx > s.m) s.raise(mx);
    {
      const float nm = -s.m;
      float2 z = make_float2(0.f, 0.f), e2 = z;
#pragma unroll
      for (int i = 0; i < kLpEach; i += 2) {
        const float2 y = make_float2(max_nan(cur.diff(i, nm), kLpFar) * kLog2e,
                                     max_nan(cur.diff(i + 1, nm), kLpFar) * kLog2e);
        const float2 e = make_float2(lp_exp2(y.x), lp_exp2(y.y));
        z = add2(z, e);
        e2 = fma2(e, y, e2);
      }
      s.z += z.x + z.y;
      s.t += e2.x + e2.y;
    }
    if (TOP) {
      if (at == 0) {
        // the threads' best values, over what the candidates will hold
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < kLpEach; ++i) {
          const int e = v0 + ((i / kVec) * kLpThreads + t) * kVec + i % kVec;
          const float v = cur.value(i);
          const unsigned long long key = v == mx && (i / kVec) * kLpThreads + t < nv ? top_key(v, e) : 0;
          best = key > best ? key : best;
        }
        const int have = sh.n;  // the odd values at the ends, kept behind
        unsigned long long odd = 0;
        __syncthreads();
        if (t < have) odd = sh.buf[t];
        __syncthreads();
        sh.buf[t] = best;
        __syncthreads();
        lp_compact(sh, kLpThreads, a.k, 0);
        thr = sh.thr;
        thrv = thr ? key_value(thr) : -INFINITY;
        __syncthreads();
        if (t < have) sh.buf[t] = odd;
        if (t == 0) sh.n = have;
        __syncthreads();
      }
      if (mx >= thrv) {
#pragma unroll
        for (int i = 0; i < kLpEach; ++i) {
          const float v = cur.value(i);
          const int vec = at + (i / kVec) * kLpThreads + t;
          if (v >= thrv && vec < nv) candidate(v, v0 + vec * kVec + i % kVec);
        }
      }
      if (__syncthreads_or(over >= kLpCompact)) {
        lp_compact(sh, sh.n, a.k, 1);
        thr = sh.thr;
        thrv = thr ? key_value(thr) : -INFINITY;
        over = 0;
        __syncthreads();
      }
    }
    cur = nxt[0];
#pragma unroll
    for (int i = 1; i < kAhead; ++i) nxt[i - 1] = nxt[i];
  }
  if (TOP) {
    __syncthreads();
    lp_compact(sh, sh.n, a.k, 1);
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
      static_assert(kLpSplits == 64, "two splits a lane");
      const float4 v = lane < a.splits ? __ldcg(a.stat + at + lane) : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
      const float4 w =
          lane + 32 < a.splits ? __ldcg(a.stat + at + lane + 32) : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
      s = {v.x, v.y, v.z};
      s.join({w.x, w.y, w.z});
      s.join_lanes(32);
    }
    if (TOP) {
      const int n = a.splits * a.k;
      for (int i = t; i < n; i += kLpThreads) sh.buf[i] = __ldcg(a.keys + at * a.k + i);
      __syncthreads();
      lp_compact(sh, n, a.k, 1);
    }
  }
  if (warp > 0) return;
  // the alternatives are at most 32: one a lane of the first warp
  const float lz = logf(s.z);
  if (t == 0) {
    if (a.entropy) a.entropy[r] = lz - s.t / s.z / kLog2e;
    if (a.targets) {
      const int i = a.targets[r];
      float lp = 0.f;
      if (i >= a.V) {
        atomicExch(a.err, kDerrBadToken);
        lp = NAN;
      } else if (i >= 0) {
        float x;
        if constexpr (DT == DT_F32) x = reinterpret_cast<const float*>(row)[i];
        else if constexpr (DT == DT_F16) x = __half2float(reinterpret_cast<const __half*>(row)[i]);
        else x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
        lp = x - s.m - lz;
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
// kLpCtas CTAs with all rows (a row alone on one CTA takes 40 times as long).
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

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_logprobs_workspace_bytes(int rows, int V, int topk) {
  if (rows < 1 || V < 1 || topk < 0 || topk > kMaxTop || topk > V) return 0;
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
  if (rows < 1 || V < 1 || ld < V || topk < 0 || topk > kMaxTop || topk > V) {
    set_error("log-probabilities: rows and V at least 1, ld at least V, topk 0..%d and at most V",
              kMaxTop);
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
  LogprobParams a = {};
  a.x = logits;
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
  const int sm = sizeof(LpShared);
  if (dtype == WS_DTYPE_F32) {
    if (topk) k_token_logprobs<DT_F32, true><<<grid, kLpThreads, sm, st>>>(a);
    else k_token_logprobs<DT_F32, false><<<grid, kLpThreads, sm, st>>>(a);
  } else if (dtype == WS_DTYPE_BF16) {
    if (topk) k_token_logprobs<DT_BF16, true><<<grid, kLpThreads, sm, st>>>(a);
    else k_token_logprobs<DT_BF16, false><<<grid, kLpThreads, sm, st>>>(a);
  } else {
    if (topk) k_token_logprobs<DT_F16, true><<<grid, kLpThreads, sm, st>>>(a);
    else k_token_logprobs<DT_F16, false><<<grid, kLpThreads, sm, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
