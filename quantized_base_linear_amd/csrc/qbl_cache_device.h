// Device helpers shared by the cache kernels (gfx950, wave64).  Internal.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "qbl_cache_kernels.h"

namespace qbl {
namespace {

// First byte of the tile that holds token position pos of head h in page p.
template <int DIM>
__device__ __forceinline__ uint8_t* tile_ptr(const qbl_kv& kv, int layer, int p, int h, int pos, int page_shift) {
  return static_cast<uint8_t*>(kv.store) + tile_offset(kv, layer, p, h, pos, page_shift, DIM);
}

__device__ __forceinline__ float half_bits(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }

// Element i of an activation array of type T (QBL_T_*), as float.
template <int T>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (T == QBL_T_F32) return static_cast<const float*>(p)[i];
  if constexpr (T == QBL_T_F16) return half_bits(static_cast<const uint16_t*>(p)[i]);
  if constexpr (T == QBL_T_BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Eight consecutive elements from i as floats; vec: p + i is 16-byte aligned.
template <int T>
__device__ __forceinline__ void load8(const void* p, int64_t i, bool vec, float (&x)[8]) {
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = load_elem<T>(p, i + j);
    return;
  }
  if constexpr (T == QBL_T_F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T == QBL_T_F16) {
        x[2 * j] = half_bits(w[j] & 0xFFFFu);
        x[2 * j + 1] = half_bits(w[j] >> 16);
      } else {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

template <int T>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (T == QBL_T_F32) static_cast<float*>(p)[i] = v;
  if constexpr (T == QBL_T_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  if constexpr (T == QBL_T_BF16) static_cast<__hip_bfloat16*>(p)[i] = __float2bfloat16(v);
}

// Four consecutive elements from i; vec: p + i is aligned to all four.
template <int T>
__device__ __forceinline__ void store4(void* p, int64_t i, bool vec, const float (&x)[4]) {
  if (!vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) store_elem<T>(p, i + k, x[k]);
    return;
  }
  if constexpr (T == QBL_T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (T == QBL_T_F16) w[k] = __half_as_ushort(__float2half_rn(x[k]));
      else w[k] = __builtin_bit_cast(unsigned short, (__bf16)x[k]);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
}

}  // namespace
}  // namespace qbl
