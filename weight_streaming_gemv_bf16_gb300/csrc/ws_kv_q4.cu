// ws_kv_q4.cu -- rows into the 4-bit key-value cache and out of it: packed
// prompts, or one token per cache row, as keys and values in fp32, bf16 or
// fp16; and the cached rows back as the values they stand for.
//
// Bound by DRAM: a token and key-value head reads 512 bytes (16-bit) and
// writes 160.  A warp takes a token and head at a time, lanes 0..15 its key row
// and 16..31 its value row, eight dimensions a lane, so that a group of 32 is a
// quad: its minimum and maximum are two shuffles away and nothing passes
// through shared memory.  For 56195 tokens x 8 heads in bf16 the store takes 77
// us, 3.9 TB/s: 154 instructions a row pair and their latencies (issue 66%
// active, integer pipe 55%, DRAM 40%); the load 62-64 us, 4.7 TB/s: the latency of
// its reads, two of 2 bytes and one of 4 a lane.  fp32: 119 and 130 us, 4.5 and 4.1
// TB/s.  A CTA's warps take consecutive tokens of one head: their rows are
// neighbours in the cache.
#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

struct KvRowsParams {
  const void* k;  // [T] tokens of [nkv][128], strides in elements
  const void* v;
  void* k_out;  // load: contiguous [T][nkv][128]
  void* v_out;
  const int* cu;     // [n + 1] token bounds of the sequences; null: token i is sequence i
  const int* rows;   // [n] cache row of each sequence; null: row i
  const int* start;  // [n] slot of its first token, negative: none
  unsigned char* kc;  // [n_rows][nkv][S][80]
  unsigned char* vc;
  long long ks, vs;
  int T, n, n_rows, nkv, S;
  int per;  // tokens a warp
  int* err;
};

// Where the tokens of one sequence go, in one head's cache rows.
struct KvPlace {
  int lo, hi;     // its tokens
  int lim;        // those before lim have a slot
  bool over;      // those from lim on lack one that they should have
  size_t at;      // row (of 80 bytes) of token lo
  __host__ __device__ bool holds(int t) const { return t >= lo && t < hi; }
  // row of token t < lim (a bound may be as low as an int goes: t - lo in 64 bits)
  __host__ __device__ size_t row(int t) const { return at + (size_t)((long long)t - lo); }
};

// The place of the sequence that token t is in (t alone where it is in none).
// No access is made outside the cache, whatever the bounds: a row or slot there
// only sets `over`.
__host__ __device__ __forceinline__ void kv_find(const KvRowsParams& a, int t, int g, KvPlace& p) {
  int i = t;
  p = {t, t + 1, t, false, 0};
  if (a.cu) {
    int lo = 0, hi = a.n;  // the last bound at or before t
    if (a.cu[0] > t) return;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    if (lo >= a.n || a.cu[lo + 1] <= t) return;
    i = lo;
    p.lo = p.lim = a.cu[lo];
    p.hi = a.cu[lo + 1];
  }
  const int s0 = a.start[i], row = a.rows ? a.rows[i] : i;
  if (s0 < 0) return;
  if (row >= 0 && row < a.n_rows && s0 < a.S) {
    // the tokens' count may pass 32 bits, that of the slots does not
    const long long tokens = (long long)p.hi - p.lo, slots = a.S - s0;
    p.lim = (int)(p.lo + (tokens < slots ? tokens : slots));
    p.at = ((size_t)row * a.nkv + g) * a.S + s0;
  }
  p.over = p.lim < p.hi;
}

constexpr int kKvWarps = 8;
constexpr int kKvBatch = 4;  // tokens whose loads a warp has in flight together

// A warp takes `per` tokens of one head, kKvWarps apart.
template <int DT>
__global__ void __launch_bounds__(kKvWarps * 32, 4) k_kv_store_q4(const __grid_constant__ KvRowsParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
  const int base = blockIdx.x * kKvWarps * a.per + warp;
  const bool keys = lane < 16;
  constexpr size_t es = DT == DT_F32 ? 4 : 2;
  const char* src = static_cast<const char*>(keys ? a.k : a.v) + ((size_t)g * kKvDim + (lane & 15) * 8) * es;
  const size_t stride = (size_t)(keys ? a.ks : a.vs) * es;
  unsigned char* cache = keys ? a.kc : a.vc;
  const KvLane at(keys);
  src += (size_t)base * stride;
  KvPlace place = {0, 0, 0, false, 0};
  for (int i = 0; i < a.per; i += kKvBatch, src += kKvBatch * kKvWarps * stride) {
    uint4 raw[kKvBatch][DT == DT_F32 ? 2 : 1];
    unsigned char* dst[kKvBatch];
#pragma unroll
    for (int u = 0; u < kKvBatch; ++u) {
      const int t = base + (i + u) * kKvWarps;
      dst[u] = nullptr;
      if (i + u < a.per && t < a.T) {
#pragma unroll
        for (int e = 0; e < (DT == DT_F32 ? 2 : 1); ++e)
          raw[u][e] = __ldcs(reinterpret_cast<const uint4*>(src + u * kKvWarps * stride) + e);
        if (!place.holds(t)) kv_find(a, t, g, place);
        if (t < place.lim) dst[u] = cache + place.row(t) * kKvRow;
        else if (place.over && lane == 0) atomicExch(a.err, kDerrBadSlot);
      }
    }
#pragma unroll
    for (int u = 0; u < kKvBatch; ++u) {
      if (!dst[u]) continue;  // alike in the whole warp
      float x[8];
      load8<DT>(raw[u], x);
      uint32_t sz;
      const uint32_t w = quantize8(x, sz);
      put_row(dst[u], w, sz, at);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kKvWarps * 32, 8) k_kv_load_q4(const __grid_constant__ KvRowsParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
  const int base = blockIdx.x * kKvWarps * a.per + warp;
  const bool keys = lane < 16;
  constexpr size_t es = DT == DT_F32 ? 4 : 2;
  const unsigned char* cache = keys ? a.kc : a.vc;
  const size_t stride = (size_t)a.nkv * kKvDim * es;
  char* out = static_cast<char*>(keys ? a.k_out : a.v_out) + (size_t)base * stride +
              ((size_t)g * kKvDim + (lane & 15) * 8) * es;
  const KvLane at(keys);
  KvPlace place = {0, 0, 0, false, 0};
  for (int i = 0; i < a.per; i += kKvBatch, out += kKvBatch * kKvWarps * stride) {
    KvWord word[kKvBatch];
    bool there[kKvBatch];
#pragma unroll
    for (int u = 0; u < kKvBatch; ++u) {
      const int t = base + (i + u) * kKvWarps;
      there[u] = i + u < a.per && t < a.T;
      if (!there[u]) continue;
      if (!place.holds(t)) kv_find(a, t, g, place);
      there[u] = t < place.lim;
      if (there[u]) word[u] = get_word(cache + place.row(t) * kKvRow, at);
      else if (place.over && lane == 0) atomicExch(a.err, kDerrBadSlot);
    }
#pragma unroll
    for (int u = 0; u < kKvBatch; ++u) {
      if (!there[u]) continue;
      float x[8];
      word_values(word[u], x);
      store8<DT>(out + u * kKvWarps * stride, x);
    }
  }
}

static bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

static ws_status kv_rows(KvRowsParams& a, int dtype, int head_dim, bool store,
                         cudaStream_t stream) {
  const void* k = store ? a.k : a.k_out;
  const void* v = store ? a.v : a.v_out;
  if (!k || !v || !a.kc || !a.vc || !a.start) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if (dtype != WS_DTYPE_F32 && dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) {
    set_error("dtype must be WS_DTYPE_F32, WS_DTYPE_BF16 or WS_DTYPE_F16");
    return WS_ERR_ARG;
  }
  if (a.T < 1 || a.T > (1 << 30) || a.n < 1 || a.n_rows < 1 || a.nkv < 1 || a.nkv > 65535 || a.S < 1 ||
      head_dim != kKvDim || (!a.cu && a.T != a.n) ||
      (store && (a.ks < (long long)a.nkv * kKvDim || a.vs < (long long)a.nkv * kKvDim ||
                 a.ks % 8 || a.vs % 8))) {
    set_error("4-bit rows: T (to 2^30), sequences, rows, key-value heads (to 65535) and s_max at least 1, "
              "head_dim %d, T = sequences without bounds, token strides a multiple of 8 and at "
              "least n_kv_heads * %d", kKvDim, kKvDim);
    return WS_ERR_SHAPE;
  }
  if (misaligned(k) || misaligned(v) || misaligned(a.kc) || misaligned(a.vc)) {
    set_error("4-bit rows: keys, values and caches must be 16-byte aligned");
    return WS_ERR_ALIGN;
  }
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  // few rows: a warp each, for the shortest time; many: 16 a warp, so that the
  // search for a token's sequence is made once and four loads are in flight
  a.per = (long long)a.T * a.nkv > 16 * 1024 ? 16 : 1;
  const dim3 grid((a.T + kKvWarps * a.per - 1) / (kKvWarps * a.per), a.nkv);
  cudaError_t e;
  if (store) {
    if (dtype == WS_DTYPE_F32) e = launch_serving(k_kv_store_q4<DT_F32>, grid, kKvWarps * 32, 0, stream, a);
    else if (dtype == WS_DTYPE_BF16) e = launch_serving(k_kv_store_q4<DT_BF16>, grid, kKvWarps * 32, 0, stream, a);
    else e = launch_serving(k_kv_store_q4<DT_F16>, grid, kKvWarps * 32, 0, stream, a);
  } else {
    if (dtype == WS_DTYPE_F32) e = launch_serving(k_kv_load_q4<DT_F32>, grid, kKvWarps * 32, 0, stream, a);
    else if (dtype == WS_DTYPE_BF16) e = launch_serving(k_kv_load_q4<DT_BF16>, grid, kKvWarps * 32, 0, stream, a);
    else e = launch_serving(k_kv_load_q4<DT_F16>, grid, kKvWarps * 32, 0, stream, a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_kv_q4_row_bytes(int head_dim) { return head_dim == kKvDim ? kKvRow : 0; }

ws_status ws_kv_store_q4(const void *k, const void *v, int dtype, const int32_t *cu_seqlens,
                         const int32_t *rows, const int32_t *start, void *k_cache, void *v_cache,
                         int T, int n_seqs, int n_rows, int n_kv_heads, int head_dim, int s_max,
                         long long k_stride, long long v_stride, ws_stream_t stream) {
  KvRowsParams a = {};
  a.k = k;
  a.v = v;
  a.cu = cu_seqlens;
  a.rows = rows;
  a.start = start;
  a.kc = static_cast<unsigned char*>(k_cache);
  a.vc = static_cast<unsigned char*>(v_cache);
  a.ks = k_stride;
  a.vs = v_stride;
  a.T = T;
  a.n = n_seqs;
  a.n_rows = n_rows;
  a.nkv = n_kv_heads;
  a.S = s_max;
  return kv_rows(a, dtype, head_dim, true, (cudaStream_t)stream);
}

ws_status ws_kv_load_q4(const void *k_cache, const void *v_cache, const int32_t *cu_seqlens,
                        const int32_t *rows, const int32_t *start, void *k, void *v, int dtype,
                        int T, int n_seqs, int n_rows, int n_kv_heads, int head_dim, int s_max,
                        ws_stream_t stream) {
  KvRowsParams a = {};
  a.k_out = k;
  a.v_out = v;
  a.cu = cu_seqlens;
  a.rows = rows;
  a.start = start;
  a.kc = static_cast<unsigned char*>(const_cast<void*>(k_cache));
  a.vc = static_cast<unsigned char*>(const_cast<void*>(v_cache));
  a.T = T;
  a.n = n_seqs;
  a.n_rows = n_rows;
  a.nkv = n_kv_heads;
  a.S = s_max;
  return kv_rows(a, dtype, head_dim, false, (cudaStream_t)stream);
}

long ws_debug_kv_places(const int32_t *cu_seqlens, const int32_t *rows, const int32_t *start, int T,
                        int n_seqs, int n_rows, int s_max, long long *places) {
  if (!start || !places || T < 1 || n_seqs < 1 || n_rows < 1 || s_max < 1 ||
      (!cu_seqlens && T != n_seqs))
    return -1;
  KvRowsParams a = {};
  a.cu = cu_seqlens;
  a.rows = rows;
  a.start = start;
  a.T = T;
  a.n = n_seqs;
  a.n_rows = n_rows;
  a.nkv = 1;
  a.S = s_max;
  KvPlace place = {0, 0, 0, false, 0};
  long found = 0;
  for (int t = 0; t < T; ++t) {
    if (!place.holds(t)) kv_find(a, t, 0, place);
    places[t] = t < place.lim ? (long long)place.row(t) : place.over ? -2 : -1;
    found += t < place.lim;
  }
  return found;
}

}  // extern "C"
