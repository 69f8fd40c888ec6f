// ws_logprobs.cu -- log-probabilities of given tokens over rows of logits,
// with the row's entropy and its most likely tokens.
//
// With m = max x, Z = sum e^(x - m): log p_i = x_i - m - log Z, and the
// entropy -sum p log p = log Z - sum e^(x - m) (x - m) / Z.
#include <cmath>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kMaxTop = 32;

struct LogprobParams {
  const void* x;  // [rows][ld], the first V of each row
  const int* targets;
  float* logprob;
  float* entropy;
  int* top_idx;
  float* top_lp;
  long long ld;
  int V, k;
  int* err;
};

template <int DT>
__device__ __forceinline__ float logit(const void* row, int i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(row)[i];
  const uint16_t u = static_cast<const uint16_t*>(row)[i];
  if constexpr (DT == DT_F16) return __half2float(__ushort_as_half(u));
  return __uint_as_float((uint32_t)u << 16);
}

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

template <typename T, typename F>
__device__ __forceinline__ T cta_reduce(T v, F f, T* red) {
  const int t = threadIdx.x;
  red[t] = v;
  __syncthreads();
  for (int o = blockDim.x >> 1; o > 0; o >>= 1) {
    if (t < o) red[t] = f(red[t], red[t + o]);
    __syncthreads();
  }
  const T r = red[0];
  __syncthreads();
  return r;
}

// One CTA per row: the maximum, the sums, then one pass per alternative.
template <int DT>
__global__ void __launch_bounds__(256) k_token_logprobs(const __grid_constant__ LogprobParams a) {
  __shared__ float red[256];
  __shared__ unsigned long long kred[256];
  const int r = blockIdx.x, t = threadIdx.x, V = a.V;
  const char* row = static_cast<const char*>(a.x) + (size_t)r * a.ld * (DT == DT_F32 ? 4 : 2);
  float m = -INFINITY;
  for (int i = t; i < V; i += 256) m = max_nan(m, logit<DT>(row, i));
  m = cta_reduce(m, [](float x, float y) { return max_nan(x, y); }, red);
  float z = 0.f, e = 0.f;
  for (int i = t; i < V; i += 256) {
    const float y = logit<DT>(row, i) - m, p = expf(y);
    z += p;
    if (p != 0.f) e = fmaf(p, y, e);
  }
  z = cta_reduce(z, [](float x, float y) { return x + y; }, red);
  e = cta_reduce(e, [](float x, float y) { return x + y; }, red);
  const float lz = logf(z);
  if (t == 0) {
    if (a.entropy) a.entropy[r] = lz - e / z;
    if (a.targets && a.logprob) {
      const int i = a.targets[r];
      if (i >= V) atomicExch(a.err, kDerrBadToken);
      a.logprob[r] = i < 0 ? 0.f : i >= V ? NAN : logit<DT>(row, i) - m - lz;
    }
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0;
    for (int i = t; i < V; i += 256) {
      const unsigned long long key = top_key(logit<DT>(row, i), i);
      if (key < last && key > best) best = key;
    }
    best = cta_reduce(best, [](unsigned long long x, unsigned long long y) { return x > y ? x : y; },
                      kred);
    last = best;
    if (t == 0) {
      if (a.top_idx) a.top_idx[(size_t)r * a.k + j] = best ? key_index(best) : -1;
      if (a.top_lp) a.top_lp[(size_t)r * a.k + j] = best ? key_value(best) - m - lz : NAN;
    }
  }
}

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_logprobs_workspace_bytes(int rows, int V, int topk) {
  if (rows < 1 || V < 1 || topk < 0 || topk > kMaxTop || topk > V) return 0;
  return 256;
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
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == WS_DTYPE_F32) k_token_logprobs<DT_F32><<<rows, 256, 0, st>>>(a);
  else if (dtype == WS_DTYPE_BF16) k_token_logprobs<DT_BF16><<<rows, 256, 0, st>>>(a);
  else k_token_logprobs<DT_F16><<<rows, 256, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
