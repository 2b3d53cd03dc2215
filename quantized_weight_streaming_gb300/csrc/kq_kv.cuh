// The 4-bit paged key/value cache: layout, element access and the 16/32-bit
// activation types, shared by the kernels that write it (kq_kv.cu) and read it
// (kq_attn.cu).
//
// A page of one key head is page_size / 16 granules.  A granule holds 16
// tokens: key codes, value codes, key scales, value scales, 18 bytes per head
// dimension in all.  Its order is that of the tensor-core operands that
// attention builds from it, so that a warp takes both operands of 8 tokens as
// one 16-byte word per lane (8 bytes at a head dimension of 64):
//  - The head dimension is cut into slabs of 128 (one slab of 64), a slab into
//    G groups of 32 that share a scale.
//  - Keys [slab][token][c = 0..3][group] 32-bit: the nibbles of dimensions
//    32 group + 8 c + 0..7.  Lane 4 token + c of a warp holds a quarter of
//    every group of its token: the B operand of queries x keys, group by group.
//  - Values [slab][token / 8][r = 0..7][token % 8 / 2][group][token % 2]
//    16-bit: the nibbles of dimensions 32 group + 4 r + 0..3.  Lane 4 r + pair
//    holds, in one 32-bit word per group, four dimensions of two successive
//    tokens: the A operand of values x probabilities.
//  - Scales fp16 [slab][token][group]; a code q stands for scale * (q - 8).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kq.h"

namespace kq {
namespace kv {

constexpr int kGranule = 16;  // tokens

template <int D>
struct Layout {
  static constexpr int kSlabs = D >= 128 ? D / 128 : 1;
  static constexpr int kSlabDim = D / kSlabs;
  static constexpr int kGroups = kSlabDim / 32;          // groups of a slab
  static constexpr int kKeySlab = kGranule * kSlabDim / 2;  // bytes of a slab's key (or value) codes
  static constexpr int kBlock = 8 * kSlabDim / 2;        // bytes of 8 tokens of a slab
  static constexpr int kCodes = kGranule * D / 2;
  static constexpr int kKeys = 0;
  static constexpr int kValues = kCodes;
  static constexpr int kKeyScales = 2 * kCodes;
  static constexpr int kValueScales = 2 * kCodes + D;    // 16 tokens x D/32 groups x 2 bytes = D
  static constexpr int kBytes = 2 * kCodes + 2 * D;
  static constexpr int kScaleSlab = kGranule * kGroups * 2;

  // Byte of the 32-bit key word of dimensions 8 w .. 8 w + 7 (w = 0 .. D/8 - 1) of a token.
  __device__ static int key_word(int token, int w) {
    const int s = w / (kSlabDim / 8), g = w % (kSlabDim / 8) / 4, c = w % 4;
    return kKeys + s * kKeySlab + token * (kSlabDim / 2) + (c * kGroups + g) * 4;
  }
  // Byte of the 16-bit value unit of dimensions 4 u .. 4 u + 3 of a token.
  __device__ static int value_unit(int token, int u) {
    const int s = u / (kSlabDim / 4), g = u % (kSlabDim / 4) / 8, r = u % 8;
    return kValues + s * kKeySlab + (token / 8) * kBlock +
           (((r * 4 + token % 8 / 2) * kGroups + g) * 2 + token % 2) * 2;
  }
  // Byte of the key scale of group q (of D/32) of a token; value scales lie D bytes further.
  __device__ static int key_scale(int token, int q) {
    return kKeyScales + (q / kGroups) * kScaleSlab + (token * kGroups + q % kGroups) * 2;
  }
};

// What a kernel needs of a kq_kv_cache.
struct Cache {
  uint8_t* data;
  int64_t block_bytes;  // of one page of one head
  int64_t pages;
  int32_t page_size;
  int32_t kv_heads;
};

// ---- activation types --------------------------------------------------------

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    union { uint4 u; T t[8]; } x;
    x.u = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(x.t[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    union { uint4 u; T t[8]; } x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.t[i] = from_float<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = x.u;
  }
}

// Four or eight consecutive elements as they are in memory, to be held while others load.
template <typename T, int N>
struct Raw {
  uint32_t u[N * sizeof(T) / 4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 4); ++i) u[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {
    constexpr int kBytes = N * sizeof(T);
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      u[0] = v.x, u[1] = v.y;
    }
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        union { uint32_t w; T t[2]; } y;
        y.t[0] = from_float<T>(v[2 * i]), y.t[1] = from_float<T>(v[2 * i + 1]);
        u[i] = y.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    constexpr int kBytes = N * sizeof(T);
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    }
  }
  __device__ __forceinline__ void get(float* v) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        union { uint32_t w; T t[2]; } y;
        y.w = u[i];
        v[2 * i] = to_float(y.t[0]), v[2 * i + 1] = to_float(y.t[1]);
      }
    }
  }
};

// Four consecutive elements, aligned to their size.
template <typename T>
__device__ __forceinline__ void load4(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    union { uint2 u; T t[4]; } x;
    x.u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_float(x.t[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    union { uint2 u; T t[4]; } x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.t[i] = from_float<T>(v[i]);
    *reinterpret_cast<uint2*>(p) = x.u;
  }
}

}  // namespace kv

// ---- host side -----------------------------------------------------------------

// Checks an activation type / a cache descriptor / a heads view of `dtype` elements (kq_kv.cu).
int check_dtype(int dtype);
int check_cache(const kq_kv_cache* c);
int check_heads(const kq_heads* h, const char* name, int dtype);
kv::Cache cache_view(const kq_kv_cache* c);
int read_kv_status(int clear);
int read_attn_status(int clear);

}  // namespace kq
