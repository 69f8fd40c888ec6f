// ws_kv_q4.cuh -- the 4-bit key-value row: its layout and its quantiser,
// shared by the row store and load (ws_kv_q4.cu) and the decode attention
// over such a cache (ws_attention_q4.cu); and what all serving kernels share:
// their launch, packed fp32 arithmetic, 8 values a lane and the error codes.
//
// A row is one slot of one key-value head: 128 values in four groups of 32
// consecutive dimensions, each with a bf16 scale s and zero z; code q (0..15)
// stands for s (q - 8) + z, the reading of the library's 4-bit weights at a
// finer group (a key's channels differ more than a weight's columns, and 32
// values is as many as one quad of lanes quantises without leaving its
// registers).  64 bytes of codes, then four (s, z) pairs: 80 bytes, an odd
// multiple of 16, so that the 16-byte pieces of 8 rows lie in distinct
// shared-memory banks.  The order of the codes is that of the decode
// attention's matrix products, so that their operands come from few wide
// loads with no exchange between lanes:
//   keys:   32-bit word 4 t + g holds dimensions 32 g + 8 t .. + 7 (t, g in
//           0..3; lane t of a quad reads its words of all four groups as 16
//           bytes), bits 4 i .. 4 i + 3 dimension i of the eight;
//   values: 16-bit unit 4 r + g holds dimensions 32 g + 4 r .. + 3 (r in
//           0..7; lane r reads its units of all four groups as 8 bytes), bits
//           4 i .. 4 i + 3 dimension i of the four.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "ws_common.cuh"
#include "ws_device.cuh"

namespace ws {

// A launch that may begin while the kernel before it on the stream drains: its
// setup (barriers, tensor memory, its place in the grid) overlaps that kernel's
// last CTAs.  The kernels launched so wait for everything before them
// (pdl_wait) ahead of their first access to memory, in every thread.
template <typename P>
inline cudaError_t launch_serving(void (*kernel)(const P), dim3 grid, int threads, int smem,
                                  cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

constexpr int kKvDim = 128;
constexpr int kKvGroup = 32;
constexpr int kKvCodes = kKvDim / 2;                              // bytes of codes
constexpr int kKvRow = kKvCodes + kKvDim / kKvGroup * 4;          // 80
constexpr int kDerrBadSlot = 2;                                   // a position or slot outside the cache
constexpr int kDerrBadSeq = 3;                                    // sequence bounds out of order or range
constexpr int kDerrBadToken = 4;                                  // a token outside the vocabulary
constexpr uint32_t kBf16Nan = 0x7fc0u;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two fp32 values a register pair: one instruction for both.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Eight consecutive values (dimensions 8 l .. 8 l + 7 of a row, l = lane % 16,
// 16 lanes a row; both halves of the warp take part) to their codes, nibble i
// dimension i, and the group's (s, z) as bits s | z << 16.  Every decision in
// fp32: s = bf16((max - min) / 15), taken as 0 below 2^-126; z = bf16(min +
// 8 s); q = clamp(rint((x - z) / s) + 8, 0, 15), 8 where s is 0.  A group
// with a value that is not finite stands for NaN as a whole.
__device__ __forceinline__ uint32_t quantize8(float (&x)[8], uint32_t& sz) {
  float lo = min_nan(min3_nan(x[0], x[1], x[2]), min3_nan(x[3], x[4], x[5]));
  float hi = max_nan(max3_nan(x[0], x[1], x[2]), max3_nan(x[3], x[4], x[5]));
  lo = min3_nan(lo, x[6], x[7]);
  hi = max3_nan(hi, x[6], x[7]);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  // (max - min) / 15, corrected once by its exact remainder (Markstein's
  // quotient: with the rounded reciprocal that is the rounded quotient)
  const float range = __fsub_rn(hi, lo), y = 1.f / 15.f, s0 = __fmul_rn(range, y);
  const float s32 = __fmaf_rn(__fmaf_rn(-s0, 15.f, range), y, s0);
  if (!(s32 <= FLT_MAX)) {  // a NaN or an infinity in the group
    sz = kBf16Nan | (kBf16Nan << 16);
    return 0x88888888u;
  }
  float s = __bfloat162float(__float2bfloat16_rn(s32));
  if (s < 1.17549435e-38f) s = 0.f;
  float z = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, 8.f * s)));
  sz = (__float_as_uint(s) >> 16) | (__float_as_uint(z) & 0xffff0000u);
  if (s == 0.f) return 0x88888888u;
  if (s < 0x1p-90f) {  // away from the subnormals, where the remainder would be rounded
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
    z *= 0x1p64f;
    s *= 0x1p64f;
  }
  // rint(d / s), d = x - z: d times an approximate 1 / s, corrected by the exact
  // remainder.  That is within 2^-45 of d / s before it is rounded, so a tie
  // comes out as one, and nothing else does: d next to (n + 1/2) s, which has 12
  // bits, is more than (1 + 2^-12) 2^-24 of it away, half a unit of n + 1/2 at
  // most 2^-24.  Adding 1.5 2^23 + 8 rounds to even and leaves rint + 8 in the
  // low bits.
  constexpr float kMagic = 12582912.f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 d = add2(make_float2(x[i], x[i + 1]), make_float2(-z, -z)), rr = make_float2(r, r);
    const float2 q = mul2(d, rr), e = fma2(q, make_float2(-s, -s), d);
    const float2 n = add2(fma2(e, rr, q), make_float2(kMagic + 8.f, kMagic + 8.f));
    c[i] = n.x;
    c[i + 1] = n.y;
  }
  // two codes at a time, clamped to 4 bits, above the ones before them
  uint32_t w = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2)
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %0;"
        : "+r"(w) : "r"(__float_as_int(c[i + 1]) - 0x4b400000), "r"(__float_as_int(c[i]) - 0x4b400000));
  return w;
}

// Where lane l = 4 g + t of a row's 16 lanes finds and leaves its codes: the
// same instructions for keys and values, which lanes of one warp may hold both.
// Keys: 32-bit word 4 t + g.  Values: units 8 t + g and 8 t + 4 + g to read; to
// write, the pair of groups (g, g ^ 1) trades halves, so that each lane has the
// two units of one r, a word.
struct KvLane {
  int read0, read1;  // bytes of the two 16-bit units
  int write;         // word
  uint32_t pick;     // byte selector of (own, partner's) codes
  int sz;            // word of the group's (s, z)
  __device__ __forceinline__ KvLane(bool keys) {
    const int l = threadIdx.x & 15, g = l >> 2, t = l & 3;
    read0 = keys ? 4 * (4 * t + g) : 2 * (8 * t + g);
    read1 = keys ? read0 + 2 : read0 + 8;
    write = keys ? 4 * t + g : (2 * t + (g & 1)) * 2 + (g >> 1);
    pick = keys ? 0x3210 : g & 1 ? 0x3276 : 0x5410;
    sz = kKvCodes / 4 + g;
  }
};

// The row's 80 bytes from 16 lanes' quantize8 results.  `row` in global or
// shared memory, 4-byte aligned.
__device__ __forceinline__ void put_row(unsigned char* row, uint32_t w, uint32_t sz, const KvLane& at) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 4);
  uint32_t* r = reinterpret_cast<uint32_t*>(row);
  r[at.write] = __byte_perm(w, other, at.pick);
  if ((threadIdx.x & 3) == 0) r[at.sz] = sz;
}

// What lane l of a row's 16 lanes reads: its eight codes and their (s, z); and
// the values they stand for.
struct KvWord {
  uint32_t w, sz;
};
__device__ __forceinline__ KvWord get_word(const unsigned char* row, const KvLane& at) {
  KvWord r;
  r.w = *reinterpret_cast<const uint16_t*>(row + at.read0) |
        ((uint32_t)*reinterpret_cast<const uint16_t*>(row + at.read1) << 16);
  r.sz = reinterpret_cast<const uint32_t*>(row)[at.sz];
  return r;
}
__device__ __forceinline__ void word_values(const KvWord& r, float (&x)[8]) {
  const float s = bf16lo(r.sz), z = bf16hi(r.sz);
  const uint32_t even = r.w & 0x0f0f0f0fu, odd = (r.w >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 2^23 + code, a byte into the mantissa; s (code - 8) is exact, so the fma
    // rounds where the sum does
    const float2 c = make_float2(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7540 | i)),
                                 __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7540 | i)));
    const float2 v = fma2(make_float2(s, s), add2(c, make_float2(-8388616.f, -8388616.f)), make_float2(z, z));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, float (&x)[8]) {
  if constexpr (DT == DT_F32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == DT_F16) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[j]);
        x[2 * j] = __low2float(h);
        x[2 * j + 1] = __high2float(h);
      } else {
        x[2 * j] = bf16lo(w[j]);
        x[2 * j + 1] = bf16hi(w[j]);
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, const float (&x)[8]) {
  if constexpr (DT == DT_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == DT_F16) {
        const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace ws
