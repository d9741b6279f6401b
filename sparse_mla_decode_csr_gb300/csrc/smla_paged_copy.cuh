// Values of the token tensors and of the records, as the paged cache's writer, reader
// and append kernels handle them: 16-byte chunks of 8 values of a 16-bit type, 4 of f32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "smla_internal.h"

namespace smla {

template <int kDtype>
struct Elem {
  static constexpr int kPer = kDtype == SMLA_DTYPE_F32 ? 4 : 8;  // values of a 16-byte chunk
  static constexpr int kSteps = kLatent / (32 * kPer);           // chunk steps of a latent row
  static constexpr int kRopeLanes = kRope / kPer;
  static constexpr int kBytes = 16 / kPer;
};

// The kPer values of a chunk as f32, and back.
template <int kDtype>
__device__ __forceinline__ void unpack(const uint4& c, float (&x)[Elem<kDtype>::kPer]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == SMLA_DTYPE_F32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (kDtype == SMLA_DTYPE_BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int kDtype>
__device__ __forceinline__ uint4 pack(const float (&x)[Elem<kDtype>::kPer]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == SMLA_DTYPE_F32) {
      w[i] = __float_as_uint(x[i]);
    } else if constexpr (kDtype == SMLA_DTYPE_BF16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Scale of a block with largest magnitude amax, and its reciprocal: the
// smallest power of two that is not below max(amax, 1e-4) / 448.  (An infinite amax
// counts as the largest f32, so that the reciprocal stays a normal power of two.)
__device__ __forceinline__ float block_scale(float amax, float* inv) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(amax, 1e-4f), FLT_MAX) / 448.0f);
  const uint32_t e = (b >> 23) + ((b & 0x7FFFFFu) ? 1u : 0u);
  *inv = __uint_as_float((254u - e) << 23);
  return __uint_as_float(e << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// A record's codes and scales by a warp, lane l from the chunks l, l + 32, ... of the row.
template <int kDtype>
__device__ __forceinline__ void write_latent(uint8_t* rec, const uint4 (&lat)[Elem<kDtype>::kSteps]) {
  using E = Elem<kDtype>;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < E::kSteps; ++i) {
    float x[E::kPer];
    unpack<kDtype>(lat[i], x);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < E::kPer; ++k) amax = fmaxf(amax, fabsf(x[k]));
    constexpr int kLanes = 128 / E::kPer;  // lanes of a scale block
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float inv;
    const float scale = block_scale(amax, &inv);
    const uint32_t c0 = e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    const int chunk = lane + 32 * i;
    if constexpr (E::kPer == 8) {
      const uint32_t c1 = e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
      *reinterpret_cast<uint2*>(rec + chunk * 8) = make_uint2(c0, c1);
    } else {
      *reinterpret_cast<uint32_t*>(rec + chunk * 4) = c0;
    }
    if ((lane & (kLanes - 1)) == 0) *reinterpret_cast<float*>(rec + kScaleOffset + 4 * (chunk / kLanes)) = scale;
  }
}

}  // namespace smla
