// ws_attention_q4.cu -- decode attention over a 4-bit key-value cache, one new
// token per batch row: the call of ws_attention.cu on rows of 80 bytes.
//
// out_h = sum_j p_j v_j, p = softmax_j(q_h . k_j / sqrt(128)) over the slots
// 0 .. pos, k and v = s (code - 8) + z per slot and group of 32 dimensions.
#include <cmath>

#include "ws_kv_q4.cuh"

#include "wsgemv.h"

namespace ws {

constexpr int kQ4MaxG = 8;       // query heads per key-value head
constexpr int kQ4MaxB = 1024;
constexpr int kQ4Tile = 128;

struct AttnQ4Params {
  const float* q;      // [B][nh * 128]
  const float* k_new;  // [B][nkv * 128]
  const float* v_new;
  unsigned char* kc;   // [B][nkv][S][80]
  unsigned char* vc;
  const int* pos;      // [B]: slot of the new token, negative: none
  float* out_f32;
  uint16_t* out_bf16;
  int nh, nkv, S, G;
  float scale;
  int* err;
};

// One CTA per (key-value head, batch row): the slots in tiles of 128; a thread
// is a slot in the scores and a dimension in the output.
__global__ void __launch_bounds__(128)
    k_decode_attention_q4(const __grid_constant__ AttnQ4Params a) {
  const int g = blockIdx.x, b = blockIdx.y, G = a.G, t = threadIdx.x;
  const int pos = a.pos[b];
  if (pos < 0) return;
  if (pos >= a.S) {
    if (t == 0) atomicExch(a.err, kDerrBadSlot);
    return;
  }
  __shared__ float qs[kQ4MaxG][kKvDim], sc[kQ4MaxG][kQ4Tile];
  const size_t bg = (size_t)b * a.nkv + g;
  unsigned char* kr = a.kc + bg * a.S * kKvRow;
  unsigned char* vr = a.vc + bg * a.S * kKvRow;
  if (t < 32) {
    float x[8];
    const bool keys = t < 16;
    load8<DT_F32>((keys ? a.k_new : a.v_new) + bg * kKvDim + (t & 15) * 8, x);
    uint32_t sz;
    const uint32_t w = quantize8(x, sz);
    put_row((keys ? kr : vr) + (size_t)pos * kKvRow, w, sz, keys, true);
  }
  for (int h = 0; h < G; ++h)
    qs[h][t] = a.q[((size_t)b * a.nh + (size_t)g * G + h) * kKvDim + t] * a.scale;
  __syncthreads();
  float m[kQ4MaxG], l[kQ4MaxG], o[kQ4MaxG];
#pragma unroll
  for (int h = 0; h < kQ4MaxG; ++h) m[h] = -INFINITY, l[h] = 0.f, o[h] = 0.f;
  const int unit = 4 * ((t & 31) >> 2) + (t >> 5), nib = 4 * (t & 3);
  for (int j0 = 0; j0 <= pos; j0 += kQ4Tile) {
    const int n = min(kQ4Tile, pos + 1 - j0);
    __syncthreads();
    if (t < n) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(kr + (size_t)(j0 + t) * kKvRow);
      float s[kQ4MaxG];
#pragma unroll
      for (int h = 0; h < kQ4MaxG; ++h) s[h] = 0.f;
      for (int w = 0; w < 16; ++w) {
        const uint32_t c = row[w], sz = row[16 + (w & 3)];
        const int d0 = 32 * (w & 3) + 8 * (w >> 2);
        for (int i = 0; i < 8; ++i) {
          const float x = bf16lo(sz) * (float)((int)((c >> (4 * i)) & 15) - 8) + bf16hi(sz);
#pragma unroll
          for (int h = 0; h < kQ4MaxG; ++h)
            if (h < G) s[h] = fmaf(x, qs[h][d0 + i], s[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < kQ4MaxG; ++h)
        if (h < G) sc[h][t] = s[h];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kQ4MaxG; ++h) {
      if (h >= G) continue;
      float mx = m[h];
      for (int j = 0; j < n; ++j) mx = fmaxf(mx, sc[h][j]);
      const float f = expf(m[h] - mx);
      m[h] = mx;
      l[h] *= f;
      o[h] *= f;
    }
    for (int j = 0; j < n; ++j) {
      const unsigned char* row = vr + (size_t)(j0 + j) * kKvRow;
      const uint32_t c = reinterpret_cast<const uint16_t*>(row)[unit];
      const uint32_t sz = reinterpret_cast<const uint32_t*>(row)[16 + (t >> 5)];
      const float x = bf16lo(sz) * (float)((int)((c >> nib) & 15) - 8) + bf16hi(sz);
#pragma unroll
      for (int h = 0; h < kQ4MaxG; ++h) {
        if (h >= G) continue;
        const float p = expf(sc[h][j] - m[h]);
        l[h] += p;
        o[h] = fmaf(p, x, o[h]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kQ4MaxG; ++h) {
    if (h >= G) continue;
    const size_t at = ((size_t)b * a.nh + (size_t)g * G + h) * kKvDim + t;
    const float v = o[h] / l[h];
    if (a.out_f32) a.out_f32[at] = v;
    if (a.out_bf16) a.out_bf16[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

static bool q4_shape_ok(int B, int nh, int nkv, int d, int S) {
  return B >= 1 && B <= kQ4MaxB && nkv >= 1 && nkv <= 65535 && nh >= 1 && nh % nkv == 0 &&
         nh / nkv <= kQ4MaxG && d == kKvDim && S >= 1;
}

}  // namespace ws

using namespace ws;

extern "C" {

size_t ws_attention_q4_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim,
                                       int s_max) {
  if (!q4_shape_ok(B, n_heads, n_kv_heads, head_dim, s_max)) return 0;
  return 256;
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
              "s_max at least 1", kQ4MaxB, kKvDim, kQ4MaxG);
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
  a.out_f32 = out_f32;
  a.out_bf16 = static_cast<uint16_t*>(out_bf16);
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.S = s_max;
  a.G = n_heads / n_kv_heads;
  a.scale = 1.0f / sqrtf((float)kKvDim);
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  k_decode_attention_q4<<<dim3(n_kv_heads, B), 128, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("launch failed: %s", cudaGetErrorString(e));
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

}  // extern "C"
