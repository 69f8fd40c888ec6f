// ws_prompt_attention.cu -- causal attention over packed prompts with grouped
// heads: token t of a sequence attends to the sequence's tokens up to t.
//
// out = sum_j p_j v_j, p = softmax_j(q . k_j / sqrt(128)).
#include <cmath>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kPromptDim = 128;

struct PromptParams {
  const uint16_t* q;  // [T][nh][128], token strides in elements
  const uint16_t* k;  // [T][nkv][128]
  const uint16_t* v;
  const int* cu;      // [n + 1]
  uint16_t* out;      // [T][nh * 128]
  float* lse;         // [T][nh] or null
  long long qs, ks, vs;
  int T, n, nh, nkv;
  float scale;
  int* err;
};

// One warp per (token, head), four dimensions a lane, the keys one by one.
template <int DT>
__global__ void __launch_bounds__(128) k_prompt_attention(const __grid_constant__ PromptParams a) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && h == 0)
    for (int i = threadIdx.x; i < a.n; i += 128)
      if (a.cu[i] < 0 || a.cu[i + 1] < a.cu[i] || a.cu[i + 1] > a.T) atomicExch(a.err, kDerrBadSeq);
  if (t >= a.T) return;
  int lo = 0, hi = a.n;
  if (a.cu[0] > t) return;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  if (lo >= a.n || a.cu[lo + 1] <= t) return;
  const int j0 = a.cu[lo], g = h / (a.nh / a.nkv);
  if (j0 < 0 || a.cu[lo + 1] > a.T) return;
  auto get = [&](const uint16_t* p, long long stride, int tok, int head, float (&x)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + (size_t)tok * stride +
                                                    (size_t)head * kPromptDim + lane * 4);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (DT == DT_F16) {
        const __half2 y = *reinterpret_cast<const __half2*>(&w[i]);
        x[2 * i] = __low2float(y);
        x[2 * i + 1] = __high2float(y);
      } else {
        x[2 * i] = bf16lo(w[i]);
        x[2 * i + 1] = bf16hi(w[i]);
      }
    }
  };
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  get(a.q, a.qs, t, h, q);
  for (int j = j0; j <= t; ++j) {
    float k[4], v[4];
    get(a.k, a.ks, j, g, k);
    get(a.v, a.vs, j, g, v);
    const float s = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * a.scale;
    const float mn = s == -INFINITY ? m : fmaxf(m, s);
    const float f = m == mn ? 1.f : expf(m - mn);
    const float p = s == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(p, v[i], o[i] * f);
  }
  uint16_t* out = a.out + ((size_t)t * a.nh + h) * kPromptDim + lane * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = o[i] / l;
    out[i] = DT == DT_F16 ? __half_as_ushort(__float2half_rn(v))
                          : __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
  if (a.lse && lane == 0) a.lse[(size_t)t * a.nh + h] = m + logf(l);
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
  a.scale = 1.0f / sqrtf((float)kPromptDim);
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  const dim3 grid((T + 3) / 4, n_heads);
  if (dtype == WS_DTYPE_F16)
    k_prompt_attention<DT_F16><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
  else
    k_prompt_attention<DT_BF16><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
